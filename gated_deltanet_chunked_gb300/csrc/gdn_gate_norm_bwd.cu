// Output gate, backward pass (gdn_gated_rmsnorm_bwd).
//
// Per (token, head) row of 128 channels, with r = 1 / sqrt(mean o^2 + eps),
// n = o r, s = sigmoid(z) and u = dy w z s:
//   d_o = r (u - n mean(u n)),  d_z = dy n w (s + z s (1 - s)),
//   d_weight = sum over rows of dy n z s.
//
// HBM-bound: three rows in, two out. A thread owns eight (bf16: 16 lanes a
// row) or four (f32: 32 lanes a row) channels, so that every access is 16
// bytes; its sum over rows stays in registers and each CTA writes one partial
// row, added by a second launch in a fixed order. Three CTAs an SM, each with
// one row ahead in registers, keep enough loads under way.
// Measured, bf16, 32 heads, of the copy rate (6783 GB/s): T = 16384 107 us
// (0.93), T = 4096 32 us (0.77, 3 us of it the second launch); f32, T = 16384
// 204 us (0.97).
#include "gdn_vec.cuh"

namespace gdn {
namespace {

using vec::Pack;

constexpr int kBThreads = 256;
constexpr int kMaxCtas = 456;  // three CTAs on each of 152 SMs: what registers allow

struct GateBwdArgs {
    const void *dy, *o, *z;
    const float *weight;
    float eps;
    void *d_o, *d_z;
    float *part;  // [gridDim.x, 128] or null
    long long rows;
};

template <typename T>
__global__ void __launch_bounds__(kBThreads, 3) k_gated_rmsnorm_bwd(const GateBwdArgs a) {
    constexpr int VE = 16 / int(sizeof(T)), G = kHeadDim / VE, kGroups = kBThreads / G;
    const int tid = threadIdx.x % G, group = threadIdx.x / G;
    const T *dy = static_cast<const T *>(a.dy) + tid * VE, *o = static_cast<const T *>(a.o) + tid * VE,
            *z = static_cast<const T *>(a.z) + tid * VE;
    T *d_o = static_cast<T *>(a.d_o) + tid * VE, *d_z = static_cast<T *>(a.d_z) + tid * VE;
    constexpr int H = VE / 2;  // pairs of a thread
    float2 w[H], dw[H];
#pragma unroll
    for (int k = 0; k < H; ++k) {
        w[k] = reinterpret_cast<const float2 *>(a.weight + tid * VE)[k];
        dw[k] = make_float2(0.f, 0.f);
    }
    const long long step = (long long)gridDim.x * kGroups;
    long long row = (long long)blockIdx.x * kGroups + group;
    const long long first = row - (threadIdx.x & 31) / G;  // the warp's rows advance together
    Pack<T, VE> po, pz, py;
    po.zero();
    pz.zero();
    py.zero();
    auto fetch = [&](long long r) {
        po.load(o + r * kHeadDim);
        pz.load(z + r * kHeadDim);
        py.load(dy + r * kHeadDim);
    };
    if (row < a.rows) fetch(row);
    using vec::both;
    using vec::fma2;
    using vec::mul2;
    for (long long base = first; base < a.rows; base += step, row += step) {
        float2 n[H], zz[H], g[H], ss = both(0.f);
#pragma unroll
        for (int k = 0; k < H; ++k) {
            n[k] = po.f2(k);
            zz[k] = pz.f2(k);
            g[k] = py.f2(k);
            ss = fma2(n[k], n[k], ss);
        }
        if (row + step < a.rows) fetch(row + step);
        const bool live = row < a.rows;
        const float r = rsqrtf(fmaf(vec::group_sum<G>(vec::sum2(ss)), 1.f / kHeadDim, a.eps));
        float2 u[H], uns = both(0.f);
#pragma unroll
        for (int k = 0; k < H; ++k) {
            const float2 sig = vec::sigmoid2(zz[k]), silu = mul2(zz[k], sig);
            n[k] = mul2(n[k], both(r));
            const float2 gn = mul2(g[k], n[k]);
            if (live) dw[k] = fma2(gn, silu, dw[k]);
            u[k] = mul2(mul2(g[k], w[k]), silu);
            uns = fma2(u[k], n[k], uns);
            // silu' = s + silu (1 - s)
            zz[k] = mul2(mul2(gn, w[k]), fma2(silu, vec::add2(both(1.f), make_float2(-sig.x, -sig.y)), sig));
        }
        const float un = vec::group_sum<G>(vec::sum2(uns)) * (1.f / kHeadDim);
        if (live) {
            Pack<T, VE> q, t;
#pragma unroll
            for (int k = 0; k < H; ++k) {
                q.set2(k, mul2(fma2(n[k], both(-un), u[k]), both(r)));
                t.set2(k, zz[k]);
            }
            q.store(d_o + row * kHeadDim);
            t.store(d_z + row * kHeadDim);
        }
    }
    if (!a.part) return;
    __shared__ float sums[kGroups][kHeadDim];
#pragma unroll
    for (int k = 0; k < H; ++k) *reinterpret_cast<float2 *>(&sums[group][tid * VE + 2 * k]) = dw[k];
    __syncthreads();
    if (threadIdx.x < kHeadDim) {
        float t = 0.f;
        for (int k = 0; k < kGroups; ++k) t += sums[k][threadIdx.x];
        a.part[blockIdx.x * kHeadDim + threadIdx.x] = t;
    }
}

// CTAs of a launch (a bound that does not depend on the device)
int ctas_of(long long rows, int io_dtype) {
    const int groups = kBThreads / (io_dtype == GDN_DT_BF16 ? 16 : 32);
    const long long c = (rows + groups - 1) / groups;
    return int(c < kMaxCtas ? c : kMaxCtas);
}

}  // namespace

size_t gated_rmsnorm_bwd_workspace(long long rows, int io_dtype) {
    return size_t(ctas_of(rows, io_dtype)) * kHeadDim * sizeof(float);  // a multiple of 256
}

cudaError_t launch_gated_rmsnorm_bwd(const void *dy, const void *o, const void *z, const float *weight, float eps,
                                     void *d_o, void *d_z, float *d_weight, void *workspace, long long rows,
                                     int io_dtype, cudaStream_t s) {
    const int ctas = ctas_of(rows, io_dtype);
    float *part = d_weight ? static_cast<float *>(workspace) : nullptr;
    if (rows > 0) {
        const GateBwdArgs a{dy, o, z, weight, eps, d_o, d_z, part, rows};
        LaunchScope scope(GDN_K_GATED_RMSNORM_BWD, s);
        if (io_dtype == GDN_DT_BF16)
            k_gated_rmsnorm_bwd<__nv_bfloat16><<<unsigned(ctas), kBThreads, 0, s>>>(a);
        else
            k_gated_rmsnorm_bwd<float><<<unsigned(ctas), kBThreads, 0, s>>>(a);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return launch_row_sums(part, nullptr, ctas, kHeadDim, d_weight, nullptr, s);
}

}  // namespace gdn
