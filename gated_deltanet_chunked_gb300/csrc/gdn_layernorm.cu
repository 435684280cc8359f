// Layer norm over the last dimension (gdn_layernorm).
//
//   y = (x - mean) * rstd * weight + bias,  rstd = 1 / sqrt(mean (x - mean)^2 + eps)
//
// HBM-bound: a row is read once, held in registers through both statistics
// (the mean first, then the squares about it: no cancellation whatever the
// row's offset) and written once. Threads keep their columns' weight and bias
// in registers over all their rows, and the next row's loads are issued
// before the current row's reductions. Roundings are written out (fmaf,
// __fmul_rn): the same row gives the same bits with and without the optional
// outputs, which the compiler may turn into separate copies of the loop.
#include "gdn_layernorm.cuh"

namespace gdn {
namespace {

using vec::Pack;

struct LnArgs {
    const void *x;
    const float *weight, *bias;
    float eps;
    void *y;
    float *mean, *rstd;
    int rows, width;
};

template <typename T, int VE, int NV, int G, int MT>
__global__ void __launch_bounds__(G ? ln::kRowThreads : MT) k_layernorm(const LnArgs a) {
    __shared__ float red[2][32];
    const int per_row = G ? G : int(blockDim.x);
    const int tid = G ? int(threadIdx.x) % (G ? G : 1) : int(threadIdx.x);
    const long long step = (long long)gridDim.x * (G ? int(blockDim.x) / (G ? G : 1) : 1);
    long long row = G ? (long long)blockIdx.x * (int(blockDim.x) / (G ? G : 1)) + int(threadIdx.x) / (G ? G : 1)
                      : (long long)blockIdx.x;
    // a warp's (a CTA's) rows advance together: all of its lanes take part in
    // every reduction, with zeros where a row is past the end
    const long long first = G ? row - (threadIdx.x & 31) / (G ? G : 1) : row;
    const T *x = static_cast<const T *>(a.x);
    T *y = static_cast<T *>(a.y);
    float w[NV][VE], b[NV][VE];
    bool has[NV];
    int col[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        col[i] = (tid + i * per_row) * VE;
        has[i] = col[i] < a.width;
#pragma unroll
        for (int j = 0; j < VE; ++j) {
            w[i][j] = has[i] && a.weight ? a.weight[col[i] + j] : 1.f;
            b[i][j] = has[i] && a.bias ? a.bias[col[i] + j] : 0.f;
        }
    }
    const float inv_width = 1.f / float(a.width);
    Pack<T, VE> next[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        next[i].zero();
        if (has[i] && row < a.rows) next[i].load(x + row * a.width + col[i]);
    }
    for (long long base = first; base < a.rows; base += step, row += step) {
        float v[NV][VE], sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VE; ++j) sum += (v[i][j] = next[i].f(j));
        if (row + step < a.rows) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (has[i]) next[i].load(x + (row + step) * a.width + col[i]);
        }
        const float mean = __fmul_rn(G ? vec::group_sum<G ? G : 1>(sum) : vec::block_sum(sum, red[0]), inv_width);
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VE; ++j) {
                v[i][j] -= mean;
                if (has[i]) sq = fmaf(v[i][j], v[i][j], sq);
            }
        const float var = __fmul_rn(G ? vec::group_sum<G ? G : 1>(sq) : vec::block_sum(sq, red[1]), inv_width);
        const float rstd = 1.f / sqrtf(__fadd_rn(var, a.eps));
        if (row < a.rows) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!has[i]) continue;
                Pack<T, VE> o;
#pragma unroll
                for (int j = 0; j < VE; ++j) o.set(j, fmaf(__fmul_rn(v[i][j], rstd), w[i][j], b[i][j]));
                o.store(y + row * a.width + col[i]);
            }
            if (tid == 0) {
                if (a.mean) a.mean[row] = mean;
                if (a.rstd) a.rstd[row] = rstd;
            }
        }
    }
}

template <typename T, int VE, int NV, int G>
void launch(const LnArgs &a, const ln::Shape &sh, int sms, cudaStream_t s) {
    const long long ctas = ((long long)a.rows + sh.rows_per_cta - 1) / sh.rows_per_cta;
    const long long most = (long long)sms * (2048 / sh.threads);
    const unsigned grid = unsigned(ctas < most ? ctas : most);
    if (sh.threads <= 512)
        k_layernorm<T, VE, NV, G, 512><<<grid, sh.threads, 0, s>>>(a);
    else if (!G)
        k_layernorm<T, VE, NV, G, G ? 512 : 1024><<<grid, sh.threads, 0, s>>>(a);
}

template <typename T>
void dispatch(const LnArgs &a, int sms, cudaStream_t s) {
    const ln::Shape sh = ln::shape_of<T>(a.width);
    GDN_LN_DISPATCH(T, sh, launch, a, sh, sms, s);
}

}  // namespace

cudaError_t launch_layernorm(const void *x, const float *weight, const float *bias, float eps, void *y, float *mean,
                             float *rstd, int rows, int width, int io_dtype, cudaStream_t s) {
    if (rows == 0) return cudaSuccess;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const LnArgs a{x, weight, bias, eps, y, mean, rstd, rows, width};
    LaunchScope scope(GDN_K_LAYERNORM, s);
    if (io_dtype == GDN_DT_BF16)
        dispatch<__nv_bfloat16>(a, sms, s);
    else
        dispatch<float>(a, sms, s);
    return cudaGetLastError();
}

}  // namespace gdn
