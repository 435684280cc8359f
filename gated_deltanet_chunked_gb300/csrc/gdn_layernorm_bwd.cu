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
    int rows, width;
};

template <typename T, int VE, int NV, int G, int MT>
__global__ void __launch_bounds__(G ? ln::kRowThreads : MT) k_layernorm_bwd(const LnBwdArgs a) {
    __shared__ float2 red[2][32];
    const int per_row = G ? G : int(blockDim.x);
    const int tid = G ? int(threadIdx.x) % (G ? G : 1) : int(threadIdx.x);
    const long long step = (long long)gridDim.x * (G ? int(blockDim.x) / (G ? G : 1) : 1);
    long long row = G ? (long long)blockIdx.x * (int(blockDim.x) / (G ? G : 1)) + int(threadIdx.x) / (G ? G : 1)
                      : (long long)blockIdx.x;
    const long long first = G ? row - (threadIdx.x & 31) / (G ? G : 1) : row;
    const T *x = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy);
    T *dx = static_cast<T *>(a.dx);
    float w[NV][VE], dw[NV][VE], db[NV][VE];
    bool has[NV];
    int col[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        col[i] = (tid + i * per_row) * VE;
        has[i] = col[i] < a.width;
#pragma unroll
        for (int j = 0; j < VE; ++j) {
            w[i][j] = has[i] && a.weight ? a.weight[col[i] + j] : 1.f;
            dw[i][j] = db[i][j] = 0.f;
        }
    }
    const float inv_width = 1.f / float(a.width);
    Pack<T, VE> nx[NV], ny[NV];
    float nmean = 0.f, nrstd = 0.f;
    auto fetch = [&](long long r) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (has[i]) {
                nx[i].load(x + r * a.width + col[i]);
                ny[i].load(dy + r * a.width + col[i]);
            }
        nmean = a.mean[r];
        nrstd = a.rstd[r];
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        nx[i].zero();
        ny[i].zero();
    }
    if (row < a.rows) fetch(row);
    int turn = 0;
    for (long long base = first; base < a.rows; base += step, row += step, turn ^= 1) {
        const bool live = row < a.rows;
        const float rstd = nrstd, mean = nmean;
        float xhat[NV][VE], g[NV][VE], s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                xhat[i][j] = __fmul_rn(nx[i].f(j) - mean, rstd);
                g[i][j] = ny[i].f(j);
            }
        if (row + step < a.rows) fetch(row + step);
        if (live) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!has[i]) continue;
#pragma unroll
                for (int j = 0; j < VE; ++j) {
                    dw[i][j] = fmaf(g[i][j], xhat[i][j], dw[i][j]);
                    db[i][j] += g[i][j];
                    g[i][j] = __fmul_rn(g[i][j], w[i][j]);
                    s1 += g[i][j];
                    s2 = fmaf(g[i][j], xhat[i][j], s2);
                }
            }
        }
        if (G) {
            s1 = vec::group_sum<G ? G : 1>(s1);
            s2 = vec::group_sum<G ? G : 1>(s2);
        } else {
            const float2 t = vec::block_sum2(s1, s2, red[turn]);
            s1 = t.x, s2 = t.y;
        }
        s1 = __fmul_rn(s1, inv_width);
        s2 = __fmul_rn(s2, inv_width);
        if (live) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!has[i]) continue;
                Pack<T, VE> o;
#pragma unroll
                for (int j = 0; j < VE; ++j) o.set(j, rstd * fmaf(-xhat[i][j], s2, g[i][j] - s1));
                o.store(dx + row * a.width + col[i]);
            }
        }
    }
    if (!a.dw_part) return;
    if (!G) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!has[i]) continue;
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                a.dw_part[(long long)blockIdx.x * a.width + col[i] + j] = dw[i][j];
                a.db_part[(long long)blockIdx.x * a.width + col[i] + j] = db[i][j];
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
                for (int j = 0; j < VE; ++j) part[group * kCols + col[i] + j] = pass ? db[i][j] : dw[i][j];
            __syncthreads();
            float *out = (pass ? a.db_part : a.dw_part) + (long long)blockIdx.x * a.width;
            for (int c = threadIdx.x; c < a.width; c += blockDim.x) {
                float t = 0.f;
                for (int k = 0; k < kGroups; ++k) t += part[k * kCols + c];
                out[c] = t;
            }
        }
    }
}

// CTAs of a launch, one partial row each. Short rows: enough CTAs to fill the
// SMs with warps; long rows: two CTAs an SM, so that the partial rows stay few.
// The bound is a constant of the width, so the workspace does not depend on
// the device.
int max_parts(int width) { return width <= ln::kWarpWidth ? 1216 : 304; }

template <typename T>
int parts_of(int rows, int width) {
    const ln::Shape sh = ln::shape_of<T>(width);
    const long long ctas = ((long long)rows + sh.rows_per_cta - 1) / sh.rows_per_cta;
    return int(ctas < max_parts(width) ? ctas : max_parts(width));
}

template <typename T, int VE, int NV, int G>
void launch(const LnBwdArgs &a, const ln::Shape &sh, int parts, cudaStream_t s) {
    if (sh.threads <= 512)
        k_layernorm_bwd<T, VE, NV, G, 512><<<unsigned(parts), sh.threads, 0, s>>>(a);
    else if (!G)
        k_layernorm_bwd<T, VE, NV, G, G ? 512 : 1024><<<unsigned(parts), sh.threads, 0, s>>>(a);
}

template <typename T>
void dispatch(const LnBwdArgs &a, int parts, cudaStream_t s) {
    const ln::Shape sh = ln::shape_of<T>(a.width);
    GDN_LN_DISPATCH(T, sh, launch, a, sh, parts, s);
}

constexpr int kSumLanes = 32;  // rows of partial sums in work at a time

// grid (ceil(width / 32), 2): 32 columns of one of the two arrays a CTA
__global__ void __launch_bounds__(32 * kSumLanes) k_row_sums(const float *a, const float *b, int parts, int width,
                                                             float *out_a, float *out_b) {
    const float *in = blockIdx.y ? b : a;
    float *out = blockIdx.y ? out_b : out_a;
    if (!out) return;
    __shared__ float t[kSumLanes][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float sum = 0.f;
    if (c < width)
        for (int r = threadIdx.y; r < parts; r += kSumLanes) sum += in[(long long)r * width + c];
    t[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    // warp y adds the kSumLanes partial sums of column y
    const float v = vec::group_sum<32>(t[threadIdx.x][threadIdx.y]);
    const int co = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && co < width) out[co] = v;
}

}  // namespace

cudaError_t launch_row_sums(const float *a, const float *b, int parts, int width, float *out_a, float *out_b,
                            cudaStream_t s) {
    if (!out_a && !out_b) return cudaSuccess;
    LaunchScope scope(GDN_K_ROW_SUMS, s);
    k_row_sums<<<dim3(unsigned((width + 31) / 32), 2), dim3(32, kSumLanes), 0, s>>>(a, b, parts, width, out_a, out_b);
    return cudaGetLastError();
}

size_t layernorm_bwd_workspace(int rows, int width) {
    const size_t parts = size_t(rows < max_parts(width) ? rows : max_parts(width));
    return (2 * parts * size_t(width) * sizeof(float) + 255) & ~size_t(255);
}

cudaError_t launch_layernorm_bwd(const void *dy, const void *x, const float *mean, const float *rstd,
                                 const float *weight, void *dx, float *dweight, float *dbias, void *workspace,
                                 int rows, int width, int io_dtype, cudaStream_t s) {
    const bool bf = io_dtype == GDN_DT_BF16;
    const int parts = bf ? parts_of<__nv_bfloat16>(rows, width) : parts_of<float>(rows, width);
    float *dw = static_cast<float *>(workspace), *db = dw + size_t(parts) * width;
    const bool sums = dweight || dbias;
    if (rows > 0) {
        const LnBwdArgs a{dy, x, mean, rstd, weight, dx, sums ? dw : nullptr, sums ? db : nullptr, rows, width};
        LaunchScope scope(GDN_K_LAYERNORM_BWD, s);
        if (bf)
            dispatch<__nv_bfloat16>(a, parts, s);
        else
            dispatch<float>(a, parts, s);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return launch_row_sums(dw, db, parts, width, dweight, dbias, s);
}

}  // namespace gdn
