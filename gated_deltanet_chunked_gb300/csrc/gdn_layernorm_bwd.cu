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
// the same bits). Rows too wide for the registers of 512 threads, with weights
// and sums, are on a cluster of two CTAs (3000 x 16384 bf16: 71 us; on 1024
// threads of one CTA, with the sums in shared memory, 118).
// Measured, bf16, of the copy rate (6783 GB/s): 16384 x 4096 66 us (0.90),
// 32768 x 2048 66 (0.90), 524288 x 128 68 (0.87), 8000 x 8192 74 (0.79);
// 4096 x 4096 24 (0.63), 17 of them without the sums: partial rows and their
// second launch cost 5 to 7 us whatever the rows.
#include "gdn_layernorm.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace {

using vec::Pack;

struct LnBwdArgs {
    const void *dy, *x;
    const float *mean, *rstd, *weight;
    void *dx;
    float *dw_part, *db_part;  // [CTAs (or pairs), width] each, or null
    bool sums;                 // whether either is wanted
    int rows, width;
    int *status;
    unsigned long long wait_ns;  // limit of a pair's wait
};

// PAIR: a row is on two CTAs, each the same half of all its rows. MT: the most
// threads of a CTA. Short aligned rows are held to 80 registers, with which
// three CTAs fit an SM (524288 x 128 bf16: 68 us, 76 with two).
template <typename T, int NV, int G, bool ALIGNED, bool PAIR, int MT>
__global__ void __launch_bounds__(MT, G && NV == 1 && ALIGNED ? 3 : 1)
k_layernorm_bwd(const LnBwdArgs a) {
    using L = ln::Place<T, NV, G, ALIGNED>;
    constexpr int VE = L::VE;
    extern __shared__ __align__(16) uint8_t smem[];  // rows ahead
    __shared__ __align__(16) float2 red[2][32];
    __shared__ ln::Pair<float2> pair;
    if (!G) {
        if (threadIdx.x < 64) red[threadIdx.x / 32][threadIdx.x % 32] = make_float2(0.f, 0.f);
        if (PAIR && threadIdx.x == 0) pair.init();
        __syncthreads();
    }
    if (PAIR) tc::cluster_arrive();
    const int rank = PAIR ? int(tc::cluster_ctarank()) : 0;
    const L at(a.width, rank, PAIR ? 2 : 1);
    const T *const src[2] = {static_cast<const T *>(a.x), static_cast<const T *>(a.dy)};
    ln::Feed<T, 2, NV, G, ALIGNED> feed(at, src, a.rows, smem);
    T *dx = static_cast<T *>(a.dx);
    constexpr int H = VE / 2;  // pairs of a vector
    // Outside the row x and g are zero, and so is what they add, unless mean rstd
    // is infinite. Such rows are looked for, and their normalised values outside
    // the row cleared; or (kOnce) rstd is taken once, for a row's sum of g (x -
    // mean) in the place of that of g xhat: 649350 x 77 96 us, 103 with the other,
    // 3000 x 16383 135 and 143; but 150150 x 333 113 and 107, 8000 x 4095 68 and 66.
    constexpr bool kOnce = !ALIGNED && (PAIR || (G && NV == 1));
    float2 w[NV][H], dw[NV][H], db[NV][H];  // the columns' weights, their sums over rows
    at.load_columns(w, a.weight, 1.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < H; ++k) dw[i][k] = db[i][k] = make_float2(0.f, 0.f);
    if (PAIR) tc::cluster_wait();  // both CTAs are ready
    bool ok = true;
    const float inv_width = 1.f / float(a.width);
    int row = at.row;
    // one row; its statistics are given, and those of the row after the next
    // take their place (two rows ahead, without a move that would wait for
    // them). It is the use-th row with this `buf`.
    auto one_row = [&](float2 &stats, int buf, int use) {
        const bool live = row < a.rows;
        const float mean = stats.x, rstd = stats.y;
        // PAIR: not before the exchange, whose fence waits for loads under way
        // (3000 x 16384 bf16: 75 us, 88 before it); of unaligned rows they
        // are better late too (8000 x 4095: 66, 74), of aligned ones early (16384 x 4096: 66, 71)
        auto next_stats = [&] {
            if (row + 2 * at.step < a.rows) stats = make_float2(a.mean[row + 2 * at.step], a.rstd[row + 2 * at.step]);
        };
        if (!PAIR && ALIGNED) next_stats();
        Pack<T, VE> in[2][NV];
        feed.get(in);
        float2 xhat[NV][H], g[NV][H], a1 = make_float2(0.f, 0.f), a2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < H; ++k) {
                xhat[i][k] = vec::add2(in[0][i].f2(k), vec::both(-mean));  // kOnce: without rstd
                if (!kOnce) xhat[i][k] = vec::mul2(xhat[i][k], vec::both(rstd));
                g[i][k] = in[1][i].f2(k);
            }
        if (!kOnce && !(fabsf(__fmul_rn(mean, rstd)) < INFINITY)) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    if (!feed.in_row(i, 2 * k)) xhat[i][k].x = 0.f;
                    if (!feed.in_row(i, 2 * k + 1)) xhat[i][k].y = 0.f;
                }
        }
        if (live) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    dw[i][k] = vec::fma2(kOnce ? vec::mul2(g[i][k], vec::both(rstd)) : g[i][k], xhat[i][k], dw[i][k]);
                    db[i][k] = vec::add2(g[i][k], db[i][k]);
                    g[i][k] = vec::mul2(g[i][k], w[i][k]);
                    a1 = vec::add2(a1, g[i][k]);
                    a2 = vec::fma2(g[i][k], xhat[i][k], a2);
                }
        }
        float s1 = vec::sum2(a1), s2 = vec::sum2(a2);
        const float2 t = G ? vec::group_sum2<G ? G : 2>(s1, s2) : vec::block_sum2(s1, s2, red[buf]);
        s1 = t.x, s2 = t.y;
        if (PAIR) {
            pair.send(t, buf, rank, ok);
            float2 low, up;
            pair.receive(low, up, buf, use, a.wait_ns, ok);
            s1 = low.x + up.x, s2 = low.y + up.y;
        }
        if (PAIR || !ALIGNED) next_stats();
        s1 = __fmul_rn(s1, inv_width);
        s2 = __fmul_rn(s2, inv_width);
        if (kOnce) s2 = __fmul_rn(__fmul_rn(s2, rstd), rstd);
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
    if (row + at.step < a.rows) odd = make_float2(a.mean[row + at.step], a.rstd[row + at.step]);
    int use = 0;
    for (int base = at.base; base < a.rows; base += 2 * at.step, ++use) {
        one_row(even, 0, use);
        if (base + at.step < a.rows) one_row(odd, 1, use);
    }
    if (PAIR) pair.leave(ok, at.rows_of(a.rows), rank, a.status);
    if (!a.sums) return;
    const long long part_row = int(blockIdx.x) / (PAIR ? 2 : 1);
    float *dwp = a.dw_part ? a.dw_part + part_row * a.width : nullptr;
    float *dbp = a.db_part ? a.db_part + part_row * a.width : nullptr;
    auto value = [&](int pass, int i, int j) {
        const float2 v = pass ? db[i][j / 2] : dw[i][j / 2];
        return j & 1 ? v.y : v.x;
    };
    if (!G) {
        float *line = reinterpret_cast<float *>(smem);  // unaligned rows: the CTA's sums on their way to whole lines
        const int lo = at.col[0] - int(threadIdx.x) * VE, hi = min(lo + NV * int(blockDim.x) * VE, a.width);
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            float *out = pass ? dbp : dwp;
            if (!out) continue;
            if (!ALIGNED) __syncthreads();
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < VE; j += ALIGNED ? 4 : 1) {
                    if (ALIGNED && at.full(i))
                        *reinterpret_cast<float4 *>(out + at.col[i] + j) =
                            make_float4(value(pass, i, j), value(pass, i, j + 1), value(pass, i, j + 2), value(pass, i, j + 3));
                    else if (!ALIGNED && at.has(i, j))
                        line[at.col[i] + j - lo] = value(pass, i, j);
                }
            if (!ALIGNED) {
                __syncthreads();
                for (int c = max(lo, 0) + int(threadIdx.x); c < hi; c += int(blockDim.x)) out[c] = line[c - lo];
            }
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
                    if (at.has(i, j)) part[group * kCols + at.col[i] + j] = value(pass, i, j);
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

// Most partial rows of a launch (a CTA's or a cluster's one each): what the SMs
// hold of CTAs of that size, as a constant of the width, so that the workspace
// does not depend on the device.
int max_parts(const ln::Shape &sh) {
    return ln::kSms * (sh.threads <= 128 ? 8 : sh.threads <= 256 ? 4 : 2) / sh.ctas();
}

template <typename T>
size_t workspace_of(int rows, int width) {
    const int most = max_parts(ln::shape_of<T, false>(rows, width));
    return (2 * size_t(rows < most ? rows : most) * size_t(width) * sizeof(float) + 255) & ~size_t(255);
}

template <typename T, int NV, int G, bool ALIGNED, bool PAIR>
struct Run {
    template <int MT>
    static cudaError_t go(const ln::Shape &sh, LnBwdArgs &a, int &parts, cudaStream_t s) {
        const auto fn = k_layernorm_bwd<T, NV, G, ALIGNED, PAIR, MT>;
        struct Key;
        size_t smem = vec::RowsAhead<2, NV>::smem(sh.threads);
        const size_t line = size_t(sh.threads) * NV * 16 / sizeof(T) * sizeof(float);
        if (!ALIGNED && !G && smem < line) smem = line;
        const cudaError_t e = ln::allow_smem(reinterpret_cast<const void *>(fn), smem);
        if (e != cudaSuccess) return e;
        // CTAs, or pairs: a partial row each
        const long long units = ((long long)a.rows + sh.rows_per_cta - 1) / sh.rows_per_cta;
        const int ctas = ln::kSms * ln::ctas_per_sm<Key>(reinterpret_cast<const void *>(fn), sh.threads, smem);
        int most = ctas / sh.ctas();
        if (most > max_parts(sh)) most = max_parts(sh);
        // few rows: four at least a unit, which writes two f32 rows of sums, while every SM has two CTAs (if it can)
        const int least = 2 * ln::kSms / sh.ctas();
        if (a.sums && most > least && units < 4 * most) most = units / 4 > least ? int(units / 4) : least;
        if (!ALIGNED && most > 8) most = most / 8 * 8;  // keeps a thread's rows at one misalignment
        parts = int(units < most ? units : most);
        if (a.dw_part && a.db_part) a.db_part = a.dw_part + size_t(parts) * a.width;
        return ln::launch(fn, sh, parts, smem, s, a);
    }
    static cudaError_t run(const ln::Shape &sh, LnBwdArgs &a, int &parts, cudaStream_t s) {
        // a few elements of the widest unaligned rows take a warp more, and then registers that others need
        // (3000 x 16383 bf16: 134 us, 16375: 94; spills)
        if constexpr (PAIR && !ALIGNED)
            if (sh.threads > 512) return go<544>(sh, a, parts, s);
        return go<G ? ln::kRowThreads : 512>(sh, a, parts, s);
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
                                 int rows, int width, int io_dtype, int *status, unsigned long long wait_ns,
                                 cudaStream_t s) {
    int parts = 0;
    float *ws = static_cast<float *>(workspace);
    LnBwdArgs a{dy,   x,    mean, rstd, weight, dx, dweight ? ws : nullptr, dbias ? ws : nullptr, dweight || dbias,
                rows, width, status, wait_ns};
    if (rows > 0) {
        LaunchScope scope(GDN_K_LAYERNORM_BWD, s);
        const cudaError_t e =
            io_dtype == GDN_DT_BF16
                ? ln::dispatch<__nv_bfloat16, false, Run>(ln::shape_of<__nv_bfloat16, false>(rows, width), a, parts, s)
                : ln::dispatch<float, false, Run>(ln::shape_of<float, false>(rows, width), a, parts, s);
        if (e != cudaSuccess) return e;
    }
    return launch_row_sums(a.dw_part, a.db_part, parts, width, dweight, dbias, s);
}

}  // namespace gdn
