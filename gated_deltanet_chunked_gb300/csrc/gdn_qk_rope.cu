// Norm of every query and key head and the rotation by position in one pass
// (gdn_qk_norm_rope), and its backward pass. For a head's row x of 128 channels
//   n = x / sqrt(mean x^2 + eps) * weight,
//   (y_a, y_b) = (n_a cos t - n_b sin t, n_a sin t + n_b cos t)
// for each of the rotated pairs (a, b), t = position * frequency of the pair.
// Backward, with dn the gradient turned back, xhat = x r, u = dn weight:
//   dx = r (u - xhat mean(u xhat)),  dweight = sum over rows of dn xhat.
//
// Each row is read and written once, 16 bytes a lane. A CTA takes the rows of a
// few tokens at a time and has their angles' sines and cosines in shared memory,
// once for all heads of a token. Bound by latency, no unit is full: 0.56 to 0.59
// of the issue slots, DRAM at 31 to 47%, a third of the warps. To the 16 bytes of
// a bf16 row that a lane reads come six loads of 16 bytes from shared memory
// (weight, cos and +-sin), anew for each head of a token, and a step's rows are
// asked for when the step before has been stored, so that with one batch a step
// only the two other CTAs have loads under way during the arithmetic. 65536 tokens
// of 32 + 4 heads, bf16, take 256 us (1.21 GB: 4.7 TB/s, 0.69 of the measured copy
// rate), 4096 tokens of 16 + 16 heads 21 us and 35 backward with the sums (0.46
// and 0.43). What made it faster: values in an order without bank conflicts and
// no division a row (35 -> 24 us), a partner's channels by shuffles after the
// norm, not before (24 -> 23), steps whose rows fill the lane groups (36 heads:
// 336 -> 272 us).
//
// Angles. A position has up to 31 bits and t is wanted to 2^-24 of a turn:
// frequency / 2 pi is held in three f32, the position in two whole f32, and the
// parts' products, exact by FMA, lose their whole turns before they are added.
// Remainders of up to half a turn are added with what each sum's rounding loses
// (2^-25 of a turn, 3.1 x 2^-24 radian a sum), so that one rounding is left:
// 2^-26 of a turn up to half a one, 2^-25 just above it, where 2^-22 radian is
// promised. Without that angles were off by up to 9.4 x 2^-24 radian.
#include "gdn_common.cuh"
#include "gdn_vec.cuh"

namespace gdn {
namespace {

using vec::both;
using vec::fma2;
using vec::mul2;

constexpr int kThreads = 256;
constexpr int kMaxPairs = kHeadDim / 2;
constexpr int kMaxTokens = 16;  // of a CTA's step
constexpr int kCtas = 3;        // on an SM: with four the forward pass spills and is 5% slower

struct RopeArgs {
    const void *x[2];         // q, k: [tokens, heads, 128], tokens `stride` elements apart
    const void *dy[2];        // backward
    void *y[2];               // forward: y; backward: dx
    long long xs[2], ds[2], ys[2];
    const float *weight[2];   // [128] or null for ones
    const float *inv_freq;    // [pairs]
    const int *positions;     // [axes, tokens]
    const int *pair_axis;     // [pairs] or null
    float *partial[2];        // backward: [CTAs, 128] sums of dweight, or null
    float eps;
    int tokens, heads[2], pairs, axes;
    int step;                 // tokens of a CTA's step
    int *status;
};

// How a row's pairs lie: next to each other, or half a rotation apart, whole
// 16-byte lanes from lane to lane or not.
enum Pairs { kNeighbours, kLanes, kAnywhere };

__device__ __forceinline__ float less_turns(float x) { return x - rintf(x); }

// a + b and what its rounding lost
__device__ __forceinline__ float2 sum_exact(float a, float b) {
    const float s = a + b, v = s - a;
    return make_float2(s, (a - (s - v)) + (b - v));
}

// cos and sin of position * frequency
__device__ __forceinline__ float2 angle(int pos, const float3 &f) {
    const float p1 = float(pos & ~0xfff), p0 = float(pos & 0xfff);
    const float a = p1 * f.x, b = p0 * f.x, c = p1 * f.y;
    // up to half a turn each, and what is small beside them
    const float2 hi = sum_exact(less_turns(a), less_turns(b));
    const float2 lo = sum_exact(less_turns(fmaf(p1, f.x, -a)), less_turns(c));
    const float2 t = sum_exact(less_turns(hi.x), less_turns(lo.x));
    const float rest = (hi.y + lo.y + t.y) + (fmaf(p0, f.x, -b) + fmaf(p1, f.y, -c) + (p0 * f.y + p1 * f.z));
    float s, co;
    sincospif(2.f * (less_turns(t.x) + rest), &s, &co);
    return make_float2(co, s);
}

template <typename T>
struct Layout {
    static constexpr int kVe = 16 / sizeof(T), kLanesOfRow = kHeadDim / kVe, kRows = kThreads / kLanesOfRow;
};

// frequency / 2 pi in three parts: 1 / 2 pi in three, their products with the
// frequency exact by FMA, the middle ones added exactly
__device__ __forceinline__ float3 turns_of(float f) {
    const float h = 0.15915493667125702f, l = 6.4206382432985265e-09f, l2 = 7.342738699078887e-17f;
    const float a = f * h, e = fmaf(f, h, -a), g = f * l, b = e + g, v = b - e;
    return make_float3(a, b, (e - (b - v)) + (g - v) + fmaf(f, l, -g) + f * l2);
}

struct RopeShared {
    float turn[2][3][kMaxTokens * kMaxPairs];  // cos, sin, -sin
    float weight[2][kHeadDim];
};

// Where element i of a row of values lies that lanes read 4 VE bytes each of
// (with `lanes`, else in order): a lane's first 16 bytes beside the other lanes'
// first ones, so that a load meets every bank once.
template <int VE>
__device__ __forceinline__ int place(int i, bool lanes) {
    return lanes && VE == 8 ? (i & 4) * (kMaxPairs / 8) + (i >> 3) * 4 + (i & 3) : i;
}
template <int VE>
__device__ __forceinline__ int weight_place(int i) {
    return VE == 8 ? (i & 4) * (kHeadDim / 8) + (i >> 3) * 4 + (i & 3) : i;
}
// a lane's VE of them (those of lane `lane`, `rest` elements from the first 16 bytes to the next)
template <int VE>
__device__ __forceinline__ void load_lane(const float *row, int lane, int rest, float2 *v) {
#pragma unroll
    for (int i = 0; i < VE / 4; ++i) {
        const float4 x = *reinterpret_cast<const float4 *>(row + i * rest + lane * 4);
        v[2 * i] = make_float2(x.x, x.y), v[2 * i + 1] = make_float2(x.z, x.w);
    }
}

// the values of lane `other` of the row
template <int Lanes, int N>
__device__ __forceinline__ void from_lane(const float2 (&v)[N], int other, float2 (&o)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i)
        o[i] = make_float2(__shfl_sync(0xffffffffu, v[i].x, other, Lanes), __shfl_sync(0xffffffffu, v[i].y, other, Lanes));
}

// The partner's channels of a lane's VE channels in a row of f32 values, for
// pairs that do not lie in whole lanes: through shared memory.
template <int VE>
__device__ __forceinline__ void partners(float *row, int ch, int pairs, const float2 *v, float2 *o) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < VE / 2; ++i) *reinterpret_cast<float2 *>(row + ch + 2 * i) = v[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < VE; ++i) {
        const int c = ch + i;
        const float w = c < 2 * pairs ? row[c < pairs ? c + pairs : c - pairs] : 0.f;
        (i & 1 ? o[i / 2].y : o[i / 2].x) = w;
    }
}

// Turns a lane's VE channels v (partners' o) by the token's cos, sin and -sin
// (kBack: back); channels behind the rotated ones stay.
template <int VE, int P, bool kBack>
__device__ __forceinline__ void rotate(const float *co, const float *si, const float *minus, int lane, int pairs, float2 *v,
                                       const float2 *o) {
    const int ch = lane * VE;
    if (ch >= 2 * pairs) return;
    if constexpr (P == kNeighbours) {
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) {
            const int p = ch / 2 + i;
            if (p >= pairs) break;
            const float c = co[p], s = kBack ? minus[p] : si[p];
            v[i] = make_float2(v[i].x * c - v[i].y * s, v[i].x * s + v[i].y * c);
        }
    } else if constexpr (P == kLanes) {
        const bool first = ch < pairs;
        const int at = first ? lane : lane - pairs / VE;
        float2 c[VE / 2], s[VE / 2];
        load_lane<VE>(co, at, kMaxPairs / 2, c);
        load_lane<VE>(first != kBack ? minus : si, at, kMaxPairs / 2, s);
#pragma unroll
        for (int i = 0; i < VE / 2; ++i) v[i] = fma2(v[i], c[i], mul2(o[i], s[i]));
    } else {
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            const int c = ch + i;
            if (c >= 2 * pairs) break;
            const bool first = c < pairs;
            const int p = first ? c : c - pairs;
            float &a = i & 1 ? v[i / 2].y : v[i / 2].x;
            const float b = i & 1 ? o[i / 2].y : o[i / 2].x;
            a = fmaf(a, co[p], b * (first != kBack ? minus[p] : si[p]));
        }
    }
}

template <typename T, int P, bool kBwd>
__global__ void __launch_bounds__(kThreads, kCtas) k_qk_rope(const __grid_constant__ RopeArgs a) {
    using L = Layout<T>;
    // rows a lane group has under way: 16 bytes a lane of each
    constexpr int VE = L::kVe, R = kBwd ? 2 : 4;
    using Row = vec::Pack<T, VE>;
    __shared__ __align__(16) RopeShared s;
    __shared__ __align__(16) float swap[P == kAnywhere ? L::kRows : 1][kHeadDim];
    const int tid = threadIdx.x, lane = tid % L::kLanesOfRow, group = tid / L::kLanesOfRow, ch = lane * VE;
    const int heads = a.heads[0] + a.heads[1];
    for (int i = tid; i < 2 * kHeadDim; i += kThreads) {
        const int w = i / kHeadDim, c = i % kHeadDim;
        s.weight[w][weight_place<VE>(c)] = a.weight[w] ? a.weight[w][c] : 1.f;
    }
    // this thread's pair of the angles (kMaxPairs divides the CTA's threads)
    const int pair = tid % kMaxPairs;
    int axis = 0;
    float3 f = make_float3(0.f, 0.f, 0.f);
    if (pair < a.pairs) {
        if (a.pair_axis) axis = a.pair_axis[pair];
        f = turns_of(a.inv_freq[pair]);
    }
    if (__syncthreads_or(axis < 0 || axis >= a.axes)) {
        if (tid == 0) record_status(a.status, GDN_EDEVICE_INPUT);
        if (kBwd && tid < kHeadDim)
            for (int w = 0; w < 2; ++w)
                if (a.partial[w]) a.partial[w][size_t(blockIdx.x) * kHeadDim + tid] = 0.f;
        return;
    }
    const int *pos = a.positions + size_t(axis) * a.tokens;
    const int pair_at = place<VE>(pair, P == kLanes);
    // from one of a lane group's rows to its next: tokens and heads
    const int next_t = L::kRows / heads, next_h = L::kRows % heads;
    // partner's lane, for pairs in whole lanes
    const int off = a.pairs / VE, other = lane < off ? lane + off : lane < 2 * off ? lane - off : lane;
    float2 dw[2][VE / 2] = {};
    int which = 0;
    for (long long t0 = (long long)blockIdx.x * a.step; t0 < a.tokens; t0 += (long long)gridDim.x * a.step, which ^= 1) {
        const int step = int(min((long long)a.step, a.tokens - t0));
        float(*turn)[kMaxTokens * kMaxPairs] = s.turn[which];  // two in turn, so that one barrier a step is enough
        int t = group / heads, h = group % heads;
        bool angles = false;
        const T *x0[2], *d0[2];
        T *y0[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // k's first head counts on from q's
            const int from = ch - (k ? a.heads[0] * kHeadDim : 0);
            x0[k] = static_cast<const T *>(a.x[k]) + t0 * a.xs[k] + from;
            if (kBwd) d0[k] = static_cast<const T *>(a.dy[k]) + t0 * a.ds[k] + from;
            y0[k] = static_cast<T *>(a.y[k]) + t0 * a.ys[k] + from;
        }
        // R rows at a time; the first loads are under way while the angles are taken
        for (int r0 = 0; r0 < step * heads; r0 += R * L::kRows) {
            Row x[R], d[kBwd ? R : 1];
            int token[R];
            bool w[R];
            T *to[R];
#pragma unroll
            for (int k = 0; k < R; ++k) {
                token[k] = t;
                w[k] = h >= a.heads[0];
                to[k] = (w[k] ? y0[1] : y0[0]) + t * (w[k] ? a.ys[1] : a.ys[0]) + h * kHeadDim;
                x[k].zero();
                if (kBwd) d[k].zero();
                if (t < step) {
                    x[k].load((w[k] ? x0[1] : x0[0]) + t * (w[k] ? a.xs[1] : a.xs[0]) + h * kHeadDim);
                    if (kBwd) d[k].load((w[k] ? d0[1] : d0[0]) + t * (w[k] ? a.ds[1] : a.ds[0]) + h * kHeadDim);
                }
                t += next_t, h += next_h;
                if (h >= heads) h -= heads, ++t;
            }
            if (!angles) {
                if (pair < a.pairs)
                    for (int k = tid / kMaxPairs; k < step; k += kThreads / kMaxPairs) {
                        const float2 v = angle(pos[t0 + k], f);
                        turn[0][k * kMaxPairs + pair_at] = v.x;
                        turn[1][k * kMaxPairs + pair_at] = v.y;
                        turn[2][k * kMaxPairs + pair_at] = -v.y;
                    }
                __syncthreads();
                angles = true;
            }
#pragma unroll
            for (int k = 0; k < R; ++k) {
                const bool has = token[k] < step;
                const float *weight = s.weight[w[k]];
                const int tt = has ? token[k] * kMaxPairs : 0;
                const float *co = turn[0] + tt, *si = turn[1] + tt, *minus = turn[2] + tt;
                float2 v[VE / 2], o[VE / 2], wt[VE / 2], ss = both(0.f);
                load_lane<VE>(weight, lane, kHeadDim / 2, wt);
#pragma unroll
                for (int i = 0; i < VE / 2; ++i) {
                    v[i] = x[k].f2(i);
                    ss = fma2(v[i], v[i], ss);
                }
                if constexpr (!kBwd) {
                    const float2 r = both(rsqrtf(vec::group_sum<L::kLanesOfRow>(vec::sum2(ss)) * (1.f / kHeadDim) + a.eps));
#pragma unroll
                    for (int i = 0; i < VE / 2; ++i) v[i] = mul2(mul2(v[i], r), wt[i]);
                    if constexpr (P == kLanes) from_lane<L::kLanesOfRow>(v, other, o);
                    if constexpr (P == kAnywhere) partners<VE>(swap[group], ch, a.pairs, v, o);
                    rotate<VE, P, false>(co, si, minus, lane, a.pairs, v, o);
#pragma unroll
                    for (int i = 0; i < VE / 2; ++i) x[k].set2(i, v[i]);
                } else {
                    float2 n[VE / 2];
#pragma unroll
                    for (int i = 0; i < VE / 2; ++i) n[i] = d[k].f2(i);
                    if constexpr (P == kLanes) from_lane<L::kLanesOfRow>(n, other, o);
                    if constexpr (P == kAnywhere) partners<VE>(swap[group], ch, a.pairs, n, o);
                    rotate<VE, P, true>(co, si, minus, lane, a.pairs, n, o);
                    float2 u[VE / 2], ux = both(0.f);
#pragma unroll
                    for (int i = 0; i < VE / 2; ++i) {
                        u[i] = mul2(n[i], wt[i]);
                        ux = fma2(u[i], v[i], ux);
                    }
                    const float2 sums = vec::group_sum2<L::kLanesOfRow>(vec::sum2(ss), vec::sum2(ux));
                    const float r = rsqrtf(sums.x * (1.f / kHeadDim) + a.eps);
                    const float m = sums.y * r * (1.f / kHeadDim);  // mean(u xhat)
#pragma unroll
                    for (int i = 0; i < VE / 2; ++i) {
                        const float2 xhat = mul2(v[i], both(r));
                        x[k].set2(i, mul2(both(r), fma2(xhat, both(-m), u[i])));
                        if (has) {
                            if (w[k]) dw[1][i] = fma2(n[i], xhat, dw[1][i]);
                            else dw[0][i] = fma2(n[i], xhat, dw[0][i]);
                        }
                    }
                }
                if (has) x[k].store(to[k]);
            }
        }
    }
    if constexpr (kBwd) {
        float(*sums)[2][kHeadDim] = reinterpret_cast<float(*)[2][kHeadDim]>(s.turn);  // [lane groups]
        static_assert(sizeof s.turn >= L::kRows * 2 * kHeadDim * sizeof(float), "sums over the lane groups");
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int i = 0; i < VE / 2; ++i) *reinterpret_cast<float2 *>(&sums[group][w][ch + 2 * i]) = dw[w][i];
        __syncthreads();
        const int w = tid / kHeadDim, c = tid % kHeadDim;
        if (a.partial[w]) {
            float v = 0.f;
            for (int g = 0; g < L::kRows; ++g) v += sums[g][w][c];
            a.partial[w][size_t(blockIdx.x) * kHeadDim + c] = v;
        }
    }
}

constexpr int kSms = 152;

int ctas_of(long long tokens, int step) {
    const long long steps = (tokens + step - 1) / step, most = kSms * kCtas;
    return int(steps < most ? steps : most);
}

// Tokens of a CTA's step (angles and a barrier come once a step): those whose
// rows fill the lane groups best, four at a time, but not so many that SMs are
// without work.
int step_of(long long tokens, int heads, int io_dtype) {
    const int at_once = 4 * (io_dtype == GDN_DT_BF16 ? Layout<__nv_bfloat16>::kRows : Layout<float>::kRows);
    const long long most = tokens / (kSms * kCtas) < kMaxTokens ? tokens / (kSms * kCtas) : kMaxTokens;
    int best = 1;
    double full = 0;
    for (int n = 1; n <= most; ++n) {
        const long long rows = (long long)n * heads;
        const double f = double(rows) / double((rows + at_once - 1) / at_once * at_once);
        if (f > full + 0.02) full = f, best = n;
    }
    return best;
}

template <typename T, bool kBwd>
void go(const RopeArgs &a, int interleaved, int ctas, cudaStream_t s) {
    if (interleaved) k_qk_rope<T, kNeighbours, kBwd><<<ctas, kThreads, 0, s>>>(a);
    else if (a.pairs % Layout<T>::kVe == 0) k_qk_rope<T, kLanes, kBwd><<<ctas, kThreads, 0, s>>>(a);
    else k_qk_rope<T, kAnywhere, kBwd><<<ctas, kThreads, 0, s>>>(a);
}

}  // namespace

size_t qk_rope_bwd_workspace(long long tokens, int heads, int io_dtype) {
    return size_t(ctas_of(tokens, step_of(tokens, heads, io_dtype))) * 2 * kHeadDim * sizeof(float);
}

cudaError_t launch_qk_rope(const gdn_qk_rope &r, const QkRopeTensors &t, void *workspace, int *status, cudaStream_t s) {
    const int heads = r.hq + r.hk;
    const bool bwd = t.dy[0] != nullptr || t.dy[1] != nullptr || t.dweight[0] || t.dweight[1];
    RopeArgs a{};
    a.xs[0] = r.q_stride, a.xs[1] = r.k_stride;
    a.ds[0] = r.dout_q_stride, a.ds[1] = r.dout_k_stride;
    a.ys[0] = r.out_q_stride, a.ys[1] = r.out_k_stride;
    a.heads[0] = r.hq, a.heads[1] = r.hk;
    a.step = step_of(r.tokens, heads, r.io_dtype);
    const int ctas = ctas_of(r.tokens, a.step);
    float *const parts = static_cast<float *>(workspace), *const *dweight = t.dweight;
    for (int w = 0; w < 2; ++w) {
        a.x[w] = t.x[w], a.dy[w] = t.dy[w], a.y[w] = t.y[w], a.weight[w] = t.weight[w];
        if (dweight[w]) a.partial[w] = parts + size_t(w) * ctas * kHeadDim;
    }
    a.inv_freq = t.inv_freq, a.positions = t.positions, a.pair_axis = t.pair_axis;
    a.eps = r.eps;
    a.tokens = r.tokens, a.pairs = r.rotary / 2, a.axes = r.axes;
    a.status = status;
    if (ctas > 0) {
        LaunchScope scope(bwd ? GDN_K_QK_NORM_ROPE_BWD : GDN_K_QK_NORM_ROPE, s);
        if (r.io_dtype == GDN_DT_BF16)
            bwd ? go<__nv_bfloat16, true>(a, r.interleaved, ctas, s) : go<__nv_bfloat16, false>(a, r.interleaved, ctas, s);
        else
            bwd ? go<float, true>(a, r.interleaved, ctas, s) : go<float, false>(a, r.interleaved, ctas, s);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (bwd && (dweight[0] || dweight[1]))
        return launch_row_sums(a.partial[0], a.partial[1], ctas, kHeadDim, dweight[0], dweight[1], s);
    return cudaSuccess;
}

}  // namespace gdn
