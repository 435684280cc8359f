// Layer norm over the last dimension (gdn_layernorm).
//
//   y = (x - mean) * rstd * weight + bias,  rstd = 1 / sqrt(mean (x - mean)^2 + eps)
//
// HBM-bound: a row is read once, held in registers through both statistics
// (the mean first, then the squares about it: no cancellation whatever the
// row's offset) and written once. Threads keep their columns' weight and bias
// in registers over all their rows, and the next row's loads are issued
// before the current row's reductions. Arithmetic is on pairs (two values an
// instruction), and its roundings are written out: the same row gives the same
// bits with and without the optional outputs, which the compiler may turn into
// separate copies of the loop.
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

constexpr int kMaxThreads = 576;  // 544 for the widest rows

template <typename T, int NV, int G, bool ALIGNED>
__global__ void __launch_bounds__(G ? ln::kRowThreads : kMaxThreads) k_layernorm(const LnArgs a) {
    using L = ln::Place<T, NV, G, ALIGNED>;
    constexpr int VE = L::VE;
    __shared__ __align__(16) float red[2][32];
    if (!G) {
        if (threadIdx.x < 64) red[threadIdx.x / 32][threadIdx.x % 32] = 0.f;
        __syncthreads();
    }
    const L at(a.width);
    extern __shared__ __align__(16) uint8_t smem[];
    const T *const src[1] = {static_cast<const T *>(a.x)};
    ln::Feed<T, 1, NV, G, ALIGNED, true> feed(at, src, a.rows, smem);
    T *y = static_cast<T *>(a.y);
    constexpr int H = VE / 2;  // pairs of a vector
    // 32 elements a thread leave no registers for weight and bias: read for every row
    constexpr bool kReread = NV * VE > 16;
    float2 w[NV][H], b[NV][H];
    if (!kReread) {
        at.load_columns(w, a.weight, 1.f);
        at.load_columns(b, a.bias, 0.f);
    }
    const float inv_width = 1.f / float(a.width);
    int row = at.row;
    for (int base = at.base; base < a.rows; base += at.step, row += at.step) {
        Pack<T, VE> in[1][NV];
        feed.get(in);
        float2 v[NV][H], acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < H; ++k) acc = vec::add2(acc, v[i][k] = in[0][i].f2(k));
        const float sum = vec::sum2(acc);
        const float mean = __fmul_rn(G ? vec::group_sum<G ? G : 1>(sum) : vec::block_sum(sum, red[0]), inv_width);
        acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int k = 0; k < H; ++k) v[i][k] = vec::add2(v[i][k], vec::both(-mean));
            if (!at.full(i)) {  // outside the row: not in the squares
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    if (!at.has(i, 2 * k)) v[i][k].x = 0.f;
                    if (!at.has(i, 2 * k + 1)) v[i][k].y = 0.f;
                }
            }
#pragma unroll
            for (int k = 0; k < H; ++k) acc = vec::fma2(v[i][k], v[i][k], acc);
        }
        const float sq = vec::sum2(acc);
        const float var = __fmul_rn(G ? vec::group_sum<G ? G : 1>(sq) : vec::block_sum(sq, red[1]), inv_width);
        const float rstd = rsqrtf(__fadd_rn(var, a.eps));
        if (row < a.rows) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (kReread) {
                    at.load_column(w[i], i, a.weight, 1.f);
                    at.load_column(b[i], i, a.bias, 0.f);
                }
                Pack<T, VE> o;
#pragma unroll
                for (int k = 0; k < H; ++k)
                    o.set2(k, vec::fma2(vec::mul2(v[i][k], vec::both(rstd)), w[i][k], b[i][k]));
                at.store(o, i, y + (long long)row * a.width);
            }
            if (at.tid == 0) {
                if (a.mean) a.mean[row] = mean;
                if (a.rstd) a.rstd[row] = rstd;
            }
        }
    }
}

template <typename T, int NV, int G, bool ALIGNED>
struct Run {
    static cudaError_t run(const ln::Shape &sh, const LnArgs &a, cudaStream_t s) {
        const auto fn = k_layernorm<T, NV, G, ALIGNED>;
        const void *f = reinterpret_cast<const void *>(fn);
        struct Key;
        const size_t smem = ln::Feed<T, 1, NV, G, ALIGNED, true>::smem(sh.threads);
        const cudaError_t e = ln::allow_smem(f, smem);
        if (e != cudaSuccess) return e;
        const long long ctas = ((long long)a.rows + sh.rows_per_cta - 1) / sh.rows_per_cta;
        // all CTAs at once; a multiple of eight, which keeps a CTA's rows at one misalignment
        const long long most = (long long)ln::kSms * ln::ctas_per_sm<Key>(f, sh.threads, smem);
        fn<<<unsigned(ctas < most ? ctas : most), sh.threads, smem, s>>>(a);
        return cudaGetLastError();
    }
};

}  // namespace

cudaError_t launch_layernorm(const void *x, const float *weight, const float *bias, float eps, void *y, float *mean,
                             float *rstd, int rows, int width, int io_dtype, cudaStream_t s) {
    if (rows == 0) return cudaSuccess;
    const LnArgs a{x, weight, bias, eps, y, mean, rstd, rows, width};
    LaunchScope scope(GDN_K_LAYERNORM, s);
    if (io_dtype == GDN_DT_BF16)
        return ln::dispatch<__nv_bfloat16, Run>(ln::shape_of<__nv_bfloat16>(rows, width, 32), a, s);
    return ln::dispatch<float, Run>(ln::shape_of<float>(rows, width, 32), a, s);
}

}  // namespace gdn
