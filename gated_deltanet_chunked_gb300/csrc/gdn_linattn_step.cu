// Decode step of linear attention with a decay for each head: one token of
// each sequence, S = lambda S + k^T v in place, o = scale q S.
//
// Bound by memory: each (sequence, value head) has its 64 KiB f32 state (32 KiB
// in bf16) read and written once. One CTA a pair; a thread holds 16 bytes of a
// row and all its rows in flight at once, writes each updated, and adds it into
// its columns' outputs, which are summed over the CTA's rows at the end.
// 157 us for 256 x 32 pairs (1.08 GB: 6.9 TB/s, 1.01 of the measured copy rate).
#include "gdn_linattn.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;

template <typename T, typename ST>
__global__ void __launch_bounds__(kThreads) k_linattn_step(const T *__restrict__ q, const T *__restrict__ k,
                                                          const T *__restrict__ v, const float *__restrict__ decay,
                                                          float scale, ST *__restrict__ state,
                                                          const int32_t *__restrict__ idx, T *__restrict__ out, int hq,
                                                          int hv, int slots, int *status) {
    constexpr int kCols = 16 / sizeof(ST), kLanes = kHeadDim / kCols, kRowsAtOnce = kThreads / kLanes,
                  kRows = kHeadDim / kRowsAtOnce;
    using Words = vec::Pack<ST, kCols>;
    __shared__ float qs[kHeadDim], ks[kHeadDim];
    __shared__ __align__(16) float red[kThreads / 32][kHeadDim];
    const int pair = blockIdx.x, n = pair / hv, h = pair % hv, hk = h / (hv / hq);
    const int tid = threadIdx.x, col = tid % kLanes * kCols, row0 = tid / kLanes;
    const int slot = idx ? idx[n] : n;
    if (slot < 0) return;  // nothing read, nothing written
    if (slot >= slots) {
        if (tid == 0) record_status(status, GDN_EDEVICE_INPUT);
        return;
    }
    ST *S = state + (size_t(slot) * hv + h) * kHeadDim * kHeadDim;
    float small = 0.f;
    if (tid < kHeadDim) small = to_f32(k[(size_t(n) * hq + hk) * kHeadDim + tid]);
    else small = to_f32(q[(size_t(n) * hq + hk) * kHeadDim + tid - kHeadDim]);
    float2 vv[kCols / 2];
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) {
        const T *p = v + size_t(pair) * kHeadDim + col + 2 * i;
        vv[i] = make_float2(to_f32(p[0]), to_f32(p[1]));
    }
    Words s[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) s[i].load(S + (row0 + i * kRowsAtOnce) * kHeadDim + col);
    (tid < kHeadDim ? ks[tid] : qs[tid - kHeadDim]) = small;
    const float keep = la::power(decay[h], 1);
    __syncthreads();
    float2 o[kCols / 2] = {};
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = row0 + i * kRowsAtOnce;
        const float2 kr = vec::both(ks[row]), qr = vec::both(qs[row]);
#pragma unroll
        for (int c = 0; c < kCols / 2; ++c) {
            const float2 x = vec::fma2(kr, vv[c], vec::mul2(vec::both(keep), s[i].f2(c)));
            s[i].set2(c, x);
            o[c] = vec::fma2(qr, x, o[c]);
        }
        s[i].store(S + row * kHeadDim + col);
    }
    // the lanes of a warp that hold the same columns, then the warps
    if constexpr (kLanes < 32) {
#pragma unroll
        for (int c = 0; c < kCols / 2; ++c) {
            o[c].x += __shfl_xor_sync(0xffffffffu, o[c].x, kLanes);
            o[c].y += __shfl_xor_sync(0xffffffffu, o[c].y, kLanes);
        }
    }
    if (tid % 32 < kLanes)
#pragma unroll
        for (int c = 0; c < kCols / 2; ++c) *reinterpret_cast<float2 *>(&red[tid / 32][col + 2 * c]) = o[c];
    __syncthreads();
    if (tid < kHeadDim) {
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) y += red[w][tid];
        out[size_t(pair) * kHeadDim + tid] = from_f32<T>(scale * y);
    }
}

template <typename T, typename ST>
void run(const gdn_problem &p, const void *q, const void *k, const void *v, const float *decay, float scale, void *state,
         const int32_t *idx, void *out, int *status, cudaStream_t s) {
    k_linattn_step<T, ST><<<unsigned(p.num_seqs) * unsigned(p.hv), kThreads, 0, s>>>(
        static_cast<const T *>(q), static_cast<const T *>(k), static_cast<const T *>(v), decay, scale,
        static_cast<ST *>(state), idx, static_cast<T *>(out), p.hq, p.hv, p.num_state_slots, status);
}

}  // namespace

cudaError_t launch_linattn_step(const gdn_problem &p, const void *q, const void *k, const void *v, const float *decay,
                                float scale, void *state, const int32_t *state_indices, void *out, int *status,
                                cudaStream_t s) {
    if (p.num_seqs == 0) return cudaSuccess;
    LaunchScope scope(GDN_K_LINATTN_STEP, s);
    const bool bf_state = p.flags & GDN_FLAG_STATE_BF16;
    auto *go = p.io_dtype == GDN_DT_BF16
                   ? (bf_state ? run<__nv_bfloat16, __nv_bfloat16> : run<__nv_bfloat16, float>)
                   : (bf_state ? run<float, __nv_bfloat16> : run<float, float>);
    go(p, q, k, v, decay, scale, state, state_indices, out, status, s);
    return cudaGetLastError();
}

}  // namespace gdn
