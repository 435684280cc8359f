// Linear attention with a decay for each head, f32, on the FMA units.
//
// Blocks of 32 tokens, one CTA a segment and head, the state in shared memory.
// With tab[n] = lambda^n, for the block's rows i, j (in time; against it the
// exponents are mirrored):
//   out_i = scale_out (lambda^(i+1) a_i S + sum_{j<=i} lambda^(i-j) (a_i b_j) c_j)
//   S     = lambda^len S + sum_j lambda^(len-1-j) b_j^T c_j
// All arithmetic is f32 (f32 inputs want more than the tensor cores' 11 bits),
// the decays are powers taken from the exponent, not products over tokens,
// whose errors would add up over the state's memory.
// Bound by the FMA units and by the loads from shared memory that feed them. A CTA
// has an SM to itself: 4 us for its start and end, 10.5 us a block in the walk and
// 4.4 in the sum (1.2 M and 0.5 M multiply-adds, 5 and 2 us on the units alone).
// With the scores over a's rows two fit: 21 us a block and 10 each, no gain, and
// alone on its SM, where there are few segments, such a CTA takes 12.3 and 6.0,
// for its 128 registers. 27 us for 200 tokens x 2 heads with all four kernels.
#include <type_traits>

#include "gdn_linattn.cuh"

namespace gdn {
namespace la {
namespace {

constexpr int kB = 32;  // tokens of a block
constexpr int kThreads = 256;
constexpr int kPitch = kHeadDim + 4;  // of b's rows, which neighbouring lanes read

struct SimtShared {
    float state[kState];
    float a[kB][kHeadDim], b[kB][kPitch], c[kB][kHeadDim], p[kB][kB];
    float tab[kB + 1], w[kB];
};

__device__ __forceinline__ float2 lo2(const float4 &v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 hi2(const float4 &v) { return make_float2(v.z, v.w); }

// kWalk: the segment's output and the state that leaves it; else its sum alone
template <bool kWalk>
__global__ void __launch_bounds__(kThreads, 1) k_la_simt(const __grid_constant__ Args p) {
    extern __shared__ __align__(16) uint8_t raw[];
    SimtShared &s = *reinterpret_cast<SimtShared *>(raw);
    const int role = blockIdx.x % p.roles, h = blockIdx.x / p.roles % p.hv, index = blockIdx.x / (p.roles * p.hv);
    next_may_start();
    wait_for_previous();
    if (index >= *p.n_segs) return;
    const Role &r = p.role[role];
    const Seg seg = p.segs[index];
    const bool leaves = seg.flags & (r.against ? kFirst : kLast), enters = seg.flags & (r.against ? kLast : kFirst);
    if (!kWalk && leaves) return;  // no segment follows
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float decay = p.decay[h];
    if (tid <= kB) s.tab[tid] = power(decay, tid);
    const size_t per_head = size_t(p.hv) * kState;
    float *mine = r.states + size_t(index) * per_head + size_t(h) * kState;
    const float *init = kWalk && enters ? r.init ? r.init + size_t(seg.seq) * per_head + size_t(h) * kState : nullptr : mine;
    if (kWalk && init && enters && r.swapped) {
#pragma unroll 16
        for (int k = 0; k < kState / kThreads; ++k) {
            const int e = k * kThreads + tid;
            s.state[e] = init[e % kHeadDim * kHeadDim + e / kHeadDim];
        }
    } else {
#pragma unroll 8
        for (int k = 0; k < kState / 4 / kThreads; ++k) {
            const int e = k * kThreads + tid;
            reinterpret_cast<float4 *>(s.state)[e] =
                kWalk && init ? reinterpret_cast<const float4 *>(init)[e] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }

    const int blocks = (seg.len + kB - 1) / kB;
    const int ha = p.hv / r.ga, hb = p.hv / r.gb, hc = p.hv / r.gc;
    const float *ga = static_cast<const float *>(r.a) + size_t(h / r.ga) * kHeadDim;
    const float *gb = static_cast<const float *>(r.b) + size_t(h / r.gb) * kHeadDim;
    const float *gc = static_cast<const float *>(r.c) + size_t(h / r.gc) * kHeadDim;
    auto block_from = [&](int n) { return (r.against ? blocks - 1 - n : n) * kB; };
    // rows 4 warp .. 4 warp + 3, channels 4 lane .. 4 lane + 3 of each: the next block's, while this one is worked on
    float4 na[4], nb[4], nc[4];
    auto fetch = [&](int n) {
        const int from = block_from(n), len = min(kB, seg.len - from);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = 4 * warp + k;
            const size_t t = size_t(seg.start + from + i);
            na[k] = nb[k] = nc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < len) {
                if (kWalk) na[k] = *reinterpret_cast<const float4 *>(ga + t * ha * kHeadDim + 4 * lane);
                nb[k] = *reinterpret_cast<const float4 *>(gb + t * hb * kHeadDim + 4 * lane);
                nc[k] = *reinterpret_cast<const float4 *>(gc + t * hc * kHeadDim + 4 * lane);
            }
        }
    };
    if (blocks > 0) fetch(0);
    for (int n = 0; n < blocks; ++n) {
        const int from = block_from(n), len = min(kB, seg.len - from);
        const int off = entry_offset(r, seg, n == 0);
        __syncthreads();  // the block before has been read; the state and the powers are there
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = 4 * warp + k;
            if (kWalk) *reinterpret_cast<float4 *>(&s.a[i][4 * lane]) = na[k];
            *reinterpret_cast<float4 *>(&s.b[i][4 * lane]) = nb[k];
            *reinterpret_cast<float4 *>(&s.c[i][4 * lane]) = nc[k];
        }
        if (tid < kB) s.w[tid] = tid < len ? r.scale_in * s.tab[r.against ? tid : len - 1 - tid] : 0.f;
        __syncthreads();
        if (n + 1 < blocks) fetch(n + 1);
        if constexpr (kWalk) {
            // scores of rows 4 warp + k with column `lane`
            float2 acc[4] = {};
#pragma unroll 4
            for (int d = 0; d < kHeadDim; d += 4) {
                const float4 y = *reinterpret_cast<const float4 *>(&s.b[lane][d]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 x = *reinterpret_cast<const float4 *>(&s.a[4 * warp + k][d]);
                    acc[k] = vec::fma2(lo2(x), lo2(y), acc[k]);
                    acc[k] = vec::fma2(hi2(x), hi2(y), acc[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = 4 * warp + k, d = r.against ? lane - i : i - lane;
                const bool in = d >= 0 && lane < len;
                s.p[i][lane] = in ? vec::sum2(acc[k]) * (r.scale_in * s.tab[max(d, 0)]) : 0.f;
            }
            __syncwarp();
            // rows 4 warp + k, columns 4 lane ..: with the state, then inside the block
            float2 x0[4] = {}, x1[4] = {};
#pragma unroll 4
            for (int d = 0; d < kHeadDim; d += 4) {
                float4 y[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) y[q] = *reinterpret_cast<const float4 *>(&s.state[(d + q) * kHeadDim + 4 * lane]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 x = *reinterpret_cast<const float4 *>(&s.a[4 * warp + k][d]);
                    const float f[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        x0[k] = vec::fma2(vec::both(f[q]), lo2(y[q]), x0[k]);
                        x1[k] = vec::fma2(vec::both(f[q]), hi2(y[q]), x1[k]);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = 4 * warp + k;
                const float f = i < len ? s.tab[r.against ? len - 1 - i + off : i + off] : 0.f;
                x0[k] = vec::mul2(vec::both(f), x0[k]);
                x1[k] = vec::mul2(vec::both(f), x1[k]);
            }
            // Rows of c that a row's sum has, and no other: a score of 0 times an infinity or NaN is no number. Beside the
            // warp's own four, which see a part of one another, they are the same for all four.
            auto add = [&](int j, auto own) {
                float4 y[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) y[q] = *reinterpret_cast<const float4 *>(&s.c[j + q][4 * lane]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float4 x = *reinterpret_cast<const float4 *>(&s.p[4 * warp + k][j]);
                    const float f[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (own && (r.against ? q < k : q > k)) continue;
                        x0[k] = vec::fma2(vec::both(f[q]), lo2(y[q]), x0[k]);
                        x1[k] = vec::fma2(vec::both(f[q]), hi2(y[q]), x1[k]);
                    }
                }
            };
            const int own4 = 4 * warp;
            if (r.against) add(own4, std::true_type{});
#pragma unroll 2
            for (int j = r.against ? own4 + 4 : 0; j < (r.against ? kB : own4); j += 4) add(j, std::false_type{});
            if (!r.against) add(own4, std::true_type{});
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = 4 * warp + k;
                if (i < len) {
                    float *to = static_cast<float *>(r.out) + (size_t(seg.start + from + i) * p.hv + h) * kHeadDim + 4 * lane;
                    *reinterpret_cast<float4 *>(to) = make_float4(r.scale_out * x0[k].x, r.scale_out * x0[k].y,
                                                                  r.scale_out * x1[k].x, r.scale_out * x1[k].y);
                }
            }
            if (n + 1 == blocks && !(leaves && r.fin)) break;  // the state goes nowhere
            __syncthreads();  // the state has been read
        }
        // the state: rows 8 (tid / 16) .., columns 4 (tid % 16) .. and 64 behind
        const int b0 = tid / 16 * 8, c0 = tid % 16 * 4;
        const float keep = s.tab[len - 1 + off];
        float2 acc[8][4];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float4 u = *reinterpret_cast<const float4 *>(&s.state[(b0 + q) * kHeadDim + c0]);
            const float4 v = *reinterpret_cast<const float4 *>(&s.state[(b0 + q) * kHeadDim + c0 + 64]);
            acc[q][0] = vec::mul2(vec::both(keep), lo2(u));
            acc[q][1] = vec::mul2(vec::both(keep), hi2(u));
            acc[q][2] = vec::mul2(vec::both(keep), lo2(v));
            acc[q][3] = vec::mul2(vec::both(keep), hi2(v));
        }
#pragma unroll 2
        for (int j = 0; j < kB; ++j) {
            const float w = s.w[j];
            const float4 x = *reinterpret_cast<const float4 *>(&s.b[j][b0]), y = *reinterpret_cast<const float4 *>(&s.b[j][b0 + 4]);
            const float4 u = *reinterpret_cast<const float4 *>(&s.c[j][c0]), v = *reinterpret_cast<const float4 *>(&s.c[j][c0 + 64]);
            const float f[8] = {w * x.x, w * x.y, w * x.z, w * x.w, w * y.x, w * y.y, w * y.z, w * y.w};
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                acc[q][0] = vec::fma2(vec::both(f[q]), lo2(u), acc[q][0]);
                acc[q][1] = vec::fma2(vec::both(f[q]), hi2(u), acc[q][1]);
                acc[q][2] = vec::fma2(vec::both(f[q]), lo2(v), acc[q][2]);
                acc[q][3] = vec::fma2(vec::both(f[q]), hi2(v), acc[q][3]);
            }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            *reinterpret_cast<float4 *>(&s.state[(b0 + q) * kHeadDim + c0]) =
                make_float4(acc[q][0].x, acc[q][0].y, acc[q][1].x, acc[q][1].y);
            *reinterpret_cast<float4 *>(&s.state[(b0 + q) * kHeadDim + c0 + 64]) =
                make_float4(acc[q][2].x, acc[q][2].y, acc[q][3].x, acc[q][3].y);
        }
    }
    __syncthreads();
    if (!kWalk) {
#pragma unroll 8
        for (int k = 0; k < kState / 4 / kThreads; ++k) {
            const int e = k * kThreads + tid;
            reinterpret_cast<float4 *>(mine)[e] = reinterpret_cast<const float4 *>(s.state)[e];
        }
    } else if (leaves && r.fin) {
        const float f = r.against && seg.len > 0 ? s.tab[1] : 1.f;  // to the gradient of the state before the first token
        float *to = r.fin + size_t(seg.seq) * per_head + size_t(h) * kState;
#pragma unroll 4
        for (int e = tid; e < kState; e += kThreads) to[e] = f == 1.f ? s.state[e] : f * s.state[e];
    }
}

}  // namespace

cudaError_t launch_simt(const Args &a, cudaStream_t s) {
    constexpr int kBytes = sizeof(SimtShared);
    cudaError_t e = cudaFuncSetAttribute(k_la_simt<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k_la_simt<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess || (e = launch_table(a, s)) != cudaSuccess) return e;
    const unsigned items = unsigned(a.max_segs) * unsigned(a.hv) * unsigned(a.roles);
    if (a.seg_len < a.total_tokens) {
        {
            LaunchScope scope(GDN_K_LINATTN_SUM, s);
            e = launch_behind(k_la_simt<false>, dim3(items), kThreads, kBytes, s, a);
        }
        if (e != cudaSuccess || (e = launch_chain(a, s)) != cudaSuccess) return e;
    }
    LaunchScope scope(GDN_K_LINATTN_WALK, s);
    return launch_behind(k_la_simt<true>, dim3(items), kThreads, kBytes, s, a);
}

}  // namespace la
}  // namespace gdn
