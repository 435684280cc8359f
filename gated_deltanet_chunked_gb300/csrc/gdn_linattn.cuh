// Linear attention with a decay for each head: what its translation units
// share. One form serves the forward pass and the three products of the
// backward pass. Over a sequence's tokens, in time or against it,
//   S = lambda S + b_t^T c_t,  out_t = a_t S   (lambda = exp(decay of the head))
// with (a, b, c, out) and the initial and final S in these roles:
//   forward       (q, k, v, out)    in time       S0 -> final state
//   d_q           (dout, v, k, dq)  in time       S0^T
//   d_v           (k, q, dout, dv)  against time  dfinal -> (times lambda) dinitial
//   d_k           (v, dout, q, dk)  against time  dfinal^T
// Sequences are cut into segments so that all SMs have work: a first kernel
// sums up each segment alone, a second one chains the sums to the state that
// enters each segment, a third one walks the segments and writes the output.
#pragma once

#include <math.h>

#include "gdn_common.cuh"
#include "gdn_vec.cuh"

namespace gdn {
namespace la {

constexpr int kState = kHeadDim * kHeadDim;

// A segment of a sequence: rows [start, start + len).
struct Seg {
    int seq, start, len;
    int flags;  // kFirst, kLast: the first, the last of its sequence
};
constexpr int kFirst = 1, kLast = 2;

struct Role {
    const void *a, *b, *c;
    void *out;          // io type, or f32 with `partial`
    const float *init;  // [seqs, hv, 128, 128] or null for zeros
    float *fin;         // the state that leaves each sequence, or null
    float *states;      // workspace [max_segs, hv, b 128, c 128]: sums, then entering states, of the segments
    float scale_in, scale_out;  // of a's products with b and of b in the state; of the output
    int ga, gb, gc;     // value heads to a head of a, b, c (out has one for each value head)
    int against;        // against time
    int swapped;        // init is [c, b] (no role with a fin)
    int partial;        // out is f32 [tokens, hv, 128], to be summed over the group's heads
    int sectors;        // out starts at a multiple of 32 bytes
};

struct Args {
    Role role[3];
    int roles;
    const float *decay;
    const int *cu;
    int hv, num_seqs, total_tokens, dense_seqlen;
    int seg_len, max_segs;
    int *n_segs;     // [1]; 0 after a failed check
    int *seq_first;  // [num_seqs + 1] first segment of each sequence
    Seg *segs;       // [max_segs]
    int *status;
    unsigned long long wait_ns;
};

// lambda^n for a whole n >= 0 (below 2^24): the product's rounding goes into
// the exponential as a factor, so that what is left is about one rounding of
// the result. A decay of -inf forgets everything before the token itself.
__device__ __forceinline__ float power(float decay, int n) {
    if (n == 0) return 1.f;
    const float f = float(n), hi = decay * f;
    if (hi < -104.f) return 0.f;  // below the smallest f32
    const float lo = fmaf(decay, f, -hi);
    const float e = vec::exp_exact2(make_float2(hi, hi)).x;
    return fmaf(e, lo, e);
}

// Exponents of a row's decays for role `r`: what the state that enters a
// segment's first walked chunk is multiplied with on its way to a row, and over
// a whole chunk. Against time the sequence's own initial state is that behind
// the last token, not decayed on its way to it.
__device__ __forceinline__ int entry_offset(const Role &r, const Seg &s, bool first_chunk) {
    return r.against && first_chunk && (s.flags & kLast) ? 0 : 1;
}

// The kernels of a call follow one another closely: each lets the next one
// start when all of its CTAs have, and that one reads nothing its predecessors
// wrote before they have ended (each waits for the one before it, so for all).
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t s, A &&...args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = grid, c.blockDim = dim3(block), c.dynamicSmemBytes = smem, c.stream = s, c.attrs = &attr, c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

cudaError_t launch_tc(const Args &a, cudaStream_t s);
cudaError_t launch_simt(const Args &a, cudaStream_t s);
cudaError_t launch_table(const Args &a, cudaStream_t s);
cudaError_t launch_chain(const Args &a, cudaStream_t s);
cudaError_t launch_group_sums(const float *x0, void *y0, const float *x1, void *y1, long long rows, int heads, int group,
                              const int *n_segs, int io_dtype, cudaStream_t s);
// rows a segment may have: those with the least estimated time
int segment_rows(long long total_tokens, long long num_seqs, int hv, int roles, int io_dtype);

}  // namespace la

cudaError_t launch_linattn_step(const gdn_problem &p, const void *q, const void *k, const void *v, const float *decay,
                                float scale, void *state, const int32_t *state_indices, void *out, int *status,
                                cudaStream_t s);
}  // namespace gdn
