// Launch arguments of the gated linear recurrence's kernels.
#pragma once

#include "gdn_common.cuh"

namespace gdn {

constexpr int kStateRows = 64;  // rows between the states that the backward pass starts from

struct RecArgs {
    const void *x, *g, *dout;
    const float *s0, *dfinal;  // [num_seqs, hv, 128] or null
    const int32_t *cu;         // [num_seqs + 1] or null: sequences of dense_seqlen rows
    void *out, *dx, *dg;
    float *final_state, *dinitial;
    float *states;  // [ceil(total_tokens / kStateRows), hv, 128]; written forward (or null), read backward
    int total_tokens, num_seqs, dense_seqlen, hv;
    int *status;
    unsigned long long wait_ns;  // limit of a wait
};

cudaError_t launch_linrec(const RecArgs &a, int io_dtype, bool channel, cudaStream_t s);
cudaError_t launch_linrec_bwd(const RecArgs &a, int io_dtype, bool channel, cudaStream_t s);
cudaError_t launch_linrec_step(const void *x, const void *g, float *state, const int32_t *idx, void *out, int seqs,
                               int hv, int slots, int io_dtype, bool channel, int *status, cudaStream_t s);

}  // namespace gdn
