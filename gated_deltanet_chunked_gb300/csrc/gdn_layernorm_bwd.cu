// Layer norm, backward pass (gdn_layernorm_bwd), and the sum of partial rows
// that ends it and gdn_gated_rmsnorm_bwd.
//
//   xhat = (x - mean) rstd, u = dy * weight
//   dx = rstd (u - mean_j u - xhat mean_j (u xhat))
//   dweight = sum over rows of dy xhat, dbias = sum over rows of dy
//
// HBM-bound: dy and x are read once, dx written once. A thread owns the same
// columns of every row that its CTA takes, so the two sums over rows stay in
// its registers; each CTA writes one partial row of each at its end, and a
// second launch adds those in a fixed order (no atomics: the same call gives
// the same bits).
#include "gdn_layernorm.cuh"

namespace gdn {
namespace {

using vec::Pack;

struct LnBwdArgs {
    const void *dy, *x;
    const float *mean, *rstd, *weight;
    void *dx;
    float *dw_part, *db_part;  // [gridDim.x, width] each, or null
    bool sums;                 // whether either is wanted
    int rows, width;
};

// The thread's sums over rows: in registers, or (IN_SMEM) in shared memory, four
// columns at a time at a thread's own place.
template <int NV, int VE, bool IN_SMEM>
struct Sums {
    float2 v[NV][VE / 2];
    __device__ __forceinline__ explicit Sums(float4 *) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < VE / 2; ++k) v[i][k] = make_float2(0.f, 0.f);
    }
    // each pair k of vector i becomes f(k, itself)
    template <typename F>
    __device__ __forceinline__ void add(int i, F f) {
#pragma unroll
        for (int k = 0; k < VE / 2; ++k) v[i][k] = f(k, v[i][k]);
    }
    __device__ __forceinline__ float get(int i, int j) const { return j & 1 ? v[i][j / 2].y : v[i][j / 2].x; }
};
template <int NV, int VE>
struct Sums<NV, VE, true> {
    float4 *p;
    __device__ __forceinline__ explicit Sums(float4 *base) : p(base + threadIdx.x) {
#pragma unroll
        for (int k = 0; k < NV * VE / 4; ++k) p[k * blockDim.x] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    template <typename F>
    __device__ __forceinline__ void add(int i, F f) {
#pragma unroll
        for (int q = 0; q < VE / 4; ++q) {
            float4 &r = p[(i * VE / 4 + q) * blockDim.x];
            const float4 t = r;
            const float2 lo = f(2 * q, make_float2(t.x, t.y)), hi = f(2 * q + 1, make_float2(t.z, t.w));
            r = make_float4(lo.x, lo.y, hi.x, hi.y);
        }
    }
    __device__ __forceinline__ float get(int i, int j) const {
        return reinterpret_cast<const float *>(p + (i * VE + j) / 4 * blockDim.x)[j % 4];
    }
};

// MT, the most threads of a CTA: with 1024 a thread has 64 registers, too few
// for its sums and its weights, which then are in shared memory and read again
// for every row.
template <typename T, int NV, int G, bool ALIGNED, int MT>
__global__ void __launch_bounds__(G ? ln::kRowThreads : MT) k_layernorm_bwd(const LnBwdArgs a) {
    using L = ln::Place<T, NV, G, ALIGNED>;
    constexpr int VE = L::VE;
    constexpr bool kWide = MT == 1024;
    extern __shared__ __align__(16) uint8_t smem[];  // rows ahead; then, kWide: two sums for every column of a thread
    __shared__ __align__(16) float2 red[2][32];
    if (!G) {
        if (threadIdx.x < 64) red[threadIdx.x / 32][threadIdx.x % 32] = make_float2(0.f, 0.f);
        __syncthreads();
    }
    const L at(a.width);
    using F = ln::Feed<T, 2, NV, G, ALIGNED, !kWide>;
    const T *const src[2] = {static_cast<const T *>(a.x), static_cast<const T *>(a.dy)};
    F feed(at, src, a.rows, smem);
    float4 *wide_sums = reinterpret_cast<float4 *>(smem + F::smem(int(blockDim.x)));
    T *dx = static_cast<T *>(a.dx);
    constexpr int H = VE / 2;  // pairs of a vector
    float2 w[NV][H];
    if (!kWide) at.load_columns(w, a.weight, 1.f);
    Sums<NV, VE, kWide> dw(wide_sums), db(wide_sums + NV * VE / 4 * blockDim.x);
    const float inv_width = 1.f / float(a.width);
    int row = at.row;
    // one row; its statistics are given, and those of the row after the next
    // take their place (two rows ahead, without a move that would wait for
    // them; kWide, short of registers: of the next row)
    const int ahead = (kWide ? 1 : 2) * at.step;
    auto one_row = [&](float2 &stats, float2 *buf) {
        const bool live = row < a.rows;
        const float mean = stats.x, rstd = stats.y;
        if (row + ahead < a.rows) stats = make_float2(a.mean[row + ahead], a.rstd[row + ahead]);
        Pack<T, VE> in[2][NV];
        feed.get(in);
        float2 xhat[NV][H], g[NV][H], a1 = make_float2(0.f, 0.f), a2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < H; ++k) {
                xhat[i][k] = vec::mul2(vec::add2(in[0][i].f2(k), vec::both(-mean)), vec::both(rstd));
                g[i][k] = in[1][i].f2(k);
            }
        if (live) {  // outside the row g is zero
            if (kWide) at.load_columns(w, a.weight, 1.f);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                dw.add(i, [&](int k, float2 s) { return vec::fma2(g[i][k], xhat[i][k], s); });
                db.add(i, [&](int k, float2 s) { return vec::add2(g[i][k], s); });
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    g[i][k] = vec::mul2(g[i][k], w[i][k]);
                    a1 = vec::add2(a1, g[i][k]);
                    a2 = vec::fma2(g[i][k], xhat[i][k], a2);
                }
            }
        }
        float s1 = vec::sum2(a1), s2 = vec::sum2(a2);
        if (G) {
            const float2 t = vec::group_sum2<G ? G : 2>(s1, s2);
            s1 = t.x, s2 = t.y;
        } else {
            const float2 t = vec::block_sum2(s1, s2, buf);
            s1 = t.x, s2 = t.y;
        }
        s1 = __fmul_rn(s1, inv_width);
        s2 = __fmul_rn(s2, inv_width);
        if (live) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                Pack<T, VE> o;
#pragma unroll
                for (int k = 0; k < H; ++k)
                    o.set2(k, vec::mul2(vec::fma2(xhat[i][k], vec::both(-s2), vec::add2(g[i][k], vec::both(-s1))),
                                        vec::both(rstd)));
                at.store(o, i, dx + (long long)row * a.width);
            }
        }
        row += at.step;
    };
    float2 even = make_float2(0.f, 0.f), odd = even;
    if (row < a.rows) even = make_float2(a.mean[row], a.rstd[row]);
    if (!kWide && row + at.step < a.rows) odd = make_float2(a.mean[row + at.step], a.rstd[row + at.step]);
    int turn = 0;
    for (int base = at.base; base < a.rows; base += ahead, turn ^= 1) {
        one_row(even, red[kWide ? turn : 0]);
        if (!kWide && base + at.step < a.rows) one_row(odd, red[1]);
    }
    if (!a.sums) return;
    float *dwp = a.dw_part ? a.dw_part + (long long)blockIdx.x * a.width : nullptr;
    float *dbp = a.db_part ? a.db_part + (long long)blockIdx.x * a.width : nullptr;
    if (!G && ALIGNED) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!at.full(i)) continue;
#pragma unroll
            for (int j = 0; j < VE; j += 4) {
                if (dwp)
                    *reinterpret_cast<float4 *>(dwp + at.col[i] + j) =
                        make_float4(dw.get(i, j), dw.get(i, j + 1), dw.get(i, j + 2), dw.get(i, j + 3));
                if (dbp)
                    *reinterpret_cast<float4 *>(dbp + at.col[i] + j) =
                        make_float4(db.get(i, j), db.get(i, j + 1), db.get(i, j + 2), db.get(i, j + 3));
            }
        }
    } else if (!G) {
        // columns that no thread has 16 bytes of: through shared memory, so that the stores are whole lines
        float *line = reinterpret_cast<float *>(smem);
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            float *out = pass ? dbp : dwp;
            if (!out) continue;
            if (kWide) {  // which holds the sums: no room for a line
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < VE; ++j)
                        if (at.has(i, j)) out[at.col[i] + j] = pass ? db.get(i, j) : dw.get(i, j);
                continue;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < VE; ++j)
                    if (at.has(i, j)) line[at.col[i] + j] = pass ? db.get(i, j) : dw.get(i, j);
            __syncthreads();
            for (int c = threadIdx.x; c < a.width; c += blockDim.x) out[c] = line[c];
        }
    } else {
        // the CTA's row groups, added in order; one of the two sums at a time
        constexpr int kCols = (G ? G : 1) * VE * NV;
        constexpr int kGroups = ln::kRowThreads / (G ? G : 1);
        __shared__ float part[G ? kGroups * kCols : 1];
        const int group = int(threadIdx.x) / (G ? G : 1);
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < VE; ++j)
                    if (at.has(i, j)) part[group * kCols + at.col[i] + j] = pass ? db.get(i, j) : dw.get(i, j);
            __syncthreads();
            float *out = pass ? dbp : dwp;
            if (!out) continue;
            for (int c = threadIdx.x; c < a.width; c += blockDim.x) {
                float t = 0.f;
#pragma unroll
                for (int k = 0; k < kGroups; ++k) t += part[k * kCols + c];
                out[c] = t;
            }
        }
    }
}

// Most CTAs of a launch, one partial row each: what the SMs hold of CTAs of
// that size, as a constant of the width, so that the workspace does not depend
// on the device.
int max_parts(int threads) { return ln::kSms * (threads <= 128 ? 8 : threads <= 256 ? 4 : threads <= 512 ? 2 : 1); }

template <typename T>
size_t workspace_of(int rows, int width) {
    const int most = max_parts(ln::shape_of<T>(rows, width).threads);
    return (2 * size_t(rows < most ? rows : most) * size_t(width) * sizeof(float) + 255) & ~size_t(255);
}

template <typename T, int NV, int G, bool ALIGNED>
struct Run {
    template <int MT>
    static cudaError_t go(const ln::Shape &sh, LnBwdArgs &a, int &parts, cudaStream_t s) {
        const auto fn = k_layernorm_bwd<T, NV, G, ALIGNED, MT>;
        struct Key;
        const size_t smem = ln::Feed<T, 2, NV, G, ALIGNED, MT != 1024>::smem(sh.threads) +
                            (MT == 1024     ? size_t(sh.threads) * NV * 16 / sizeof(T) * 2 * sizeof(float)
                             : !ALIGNED && !G ? size_t(a.width) * sizeof(float)
                                              : 0);
        const cudaError_t e = ln::allow_smem(reinterpret_cast<const void *>(fn), smem);
        if (e != cudaSuccess) return e;
        const long long ctas = ((long long)a.rows + sh.rows_per_cta - 1) / sh.rows_per_cta;
        long long most = (long long)ln::kSms * ln::ctas_per_sm<Key>(reinterpret_cast<const void *>(fn), sh.threads, smem);
        if (most > max_parts(sh.threads)) most = max_parts(sh.threads);
        // few rows: four at least a CTA, which writes two f32 rows of sums, while every SM has two CTAs
        if (a.sums && ctas < 4 * most) most = ctas / 4 > 2 * ln::kSms ? ctas / 4 / 8 * 8 : 2 * ln::kSms;
        parts = int(ctas < most ? ctas : most);
        if (a.dw_part && a.db_part) a.db_part = a.dw_part + size_t(parts) * a.width;
        fn<<<unsigned(parts), sh.threads, smem, s>>>(a);
        return cudaGetLastError();
    }
    static cudaError_t run(const ln::Shape &sh, LnBwdArgs &a, int &parts, cudaStream_t s) {
        // more than 512 threads only with the most elements a thread
        constexpr int kMost = !G && NV * 16 / int(sizeof(T)) >= 16 ? 1024 : 512;
        return sh.threads <= 512 ? go<512>(sh, a, parts, s) : go<kMost>(sh, a, parts, s);
    }
};

constexpr int kSumWarps = 16;

// grid (ceil(width / 32), 2): 32 columns of one of the two arrays a CTA, each
// warp every kSumWarps-th row.
__global__ void __launch_bounds__(32 * kSumWarps) k_row_sums(const float *a, const float *b, int parts, int width,
                                                             float *out_a, float *out_b) {
    const float *in = blockIdx.y ? b : a;
    float *out = blockIdx.y ? out_b : out_a;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    __shared__ float t[kSumWarps][32];
    if (!out) return;
    float sum = 0.f;
    if (c < width)
#pragma unroll 10
        for (int r = w; r < parts; r += kSumWarps) sum += in[(long long)r * width + c];
    t[w][lane] = sum;
    __syncthreads();
    if (w == 0 && c < width) {
#pragma unroll
        for (int k = 1; k < kSumWarps; ++k) sum += t[k][lane];
        out[c] = sum;
    }
}

}  // namespace

cudaError_t launch_row_sums(const float *a, const float *b, int parts, int width, float *out_a, float *out_b,
                            cudaStream_t s) {
    if (!out_a && !out_b) return cudaSuccess;
    LaunchScope scope(GDN_K_ROW_SUMS, s);
    k_row_sums<<<dim3(unsigned((width + 31) / 32), out_b ? 2 : 1), 32 * kSumWarps, 0, s>>>(a, b, parts, width, out_a,
                                                                                           out_b);
    return cudaGetLastError();
}

size_t layernorm_bwd_workspace(int rows, int width, int io_dtype) {
    return io_dtype == GDN_DT_BF16 ? workspace_of<__nv_bfloat16>(rows, width) : workspace_of<float>(rows, width);
}

cudaError_t launch_layernorm_bwd(const void *dy, const void *x, const float *mean, const float *rstd,
                                 const float *weight, void *dx, float *dweight, float *dbias, void *workspace,
                                 int rows, int width, int io_dtype, cudaStream_t s) {
    int parts = 0;
    float *ws = static_cast<float *>(workspace);
    LnBwdArgs a{dy,   x,    mean, rstd, weight, dx, dweight ? ws : nullptr, dbias ? ws : nullptr, dweight || dbias,
                rows, width};
    if (rows > 0) {
        LaunchScope scope(GDN_K_LAYERNORM_BWD, s);
        const cudaError_t e =
            io_dtype == GDN_DT_BF16
                ? ln::dispatch<__nv_bfloat16, Run>(ln::shape_of<__nv_bfloat16>(rows, width), a, parts, s)
                : ln::dispatch<float, Run>(ln::shape_of<float>(rows, width), a, parts, s);
        if (e != cudaSuccess) return e;
    }
    return launch_row_sums(a.dw_part, a.db_part, parts, width, dweight, dbias, s);
}

}  // namespace gdn
