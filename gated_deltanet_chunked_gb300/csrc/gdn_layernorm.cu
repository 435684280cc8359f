// Layer norm over the last dimension (gdn_layernorm).
//
//   y = (x - mean) * rstd * weight + bias,  rstd = 1 / sqrt(mean (x - mean)^2 + eps)
//
// HBM-bound: a row is read once, held in registers through both statistics and
// written once. The mean comes first, then the squares about it. Where the mean
// is more than 4 deviations, what rounding left in it counts (6e-5 in a row that
// is 1000 all over, which 1 / sqrt(eps) makes 0.02): there the values about it
// are summed too, and correct it. So whatever the row's offset, errors are small
// beside its deviations. (Summed in every row that takes 48 us at 16384 x 4096,
// where 44 are taken.) Threads keep their columns' weight and bias
// in registers over all their rows, and the next rows are on their way to
// shared memory meanwhile. Arithmetic is on pairs (two values an instruction),
// and its roundings are written out: the same row gives the same bits with and
// without the optional outputs, which the compiler may turn into separate
// copies of the loop.
// Measured, bf16, of the copy rate (6783 GB/s): 16384 x 4096 44 us (0.90),
// 32768 x 2048 45 (0.88), 524288 x 128 46 (0.86), 8000 x 8192 46 (0.84); where
// rows are odd a third of the time goes into their ragged ends (20000 x 1001
// 20 us, 0.60); a single row takes 2.3 us. What bounds the widest rows is
// their two reductions, with one CTA on an SM: 3000 x 16384 43 us (0.67). f32:
// 65536 x 1024 92 us (0.86), 524288 x 128 98 (0.81), 4000 x 16384 82 (0.94).
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
    int *status;
    unsigned long long wait_ns;  // limit of a pair's wait
};

// PAIR: a row is on two CTAs, each the same half of all its rows. (Threads: 544
// for the widest unaligned rows; 576 holds the others to 96 registers, with
// which more CTAs fit: 20000 x 1001 20 us, with a bound of 512 23.)
template <typename T, int NV, int G, bool ALIGNED, bool PAIR>
__global__ void __launch_bounds__(G ? ln::kRowThreads : PAIR ? 544 : 576) k_layernorm(const LnArgs a) {
    using L = ln::Place<T, NV, G, ALIGNED>;
    constexpr int VE = L::VE;
    __shared__ __align__(16) float red[3][32];
    __shared__ ln::Pair<float4> pair;
    if (!G) {
        if (threadIdx.x < 32) red[0][threadIdx.x] = red[1][threadIdx.x] = red[2][threadIdx.x] = 0.f;
        if (PAIR && threadIdx.x == 0) pair.init();
        __syncthreads();
    }
    if (PAIR) tc::cluster_arrive();
    const int rank = PAIR ? int(tc::cluster_ctarank()) : 0;
    const L at(a.width, rank, PAIR ? 2 : 1);
    extern __shared__ __align__(16) uint8_t smem[];
    const T *const src[1] = {static_cast<const T *>(a.x)};
    ln::Feed<T, 1, NV, G, ALIGNED> feed(at, src, a.rows, smem);
    T *y = static_cast<T *>(a.y);
    constexpr int H = VE / 2;  // pairs of a vector
    // 32 elements a thread leave no registers for weight and bias: at the
    // thread's own place in shared memory, or, where the rows ahead (f32) leave
    // none of that either, read for every row
    constexpr bool kShared = NV * VE > 16 && sizeof(T) == 2, kReread = NV * VE > 16 && !kShared;
    float4 *const shared = reinterpret_cast<float4 *>(smem + vec::RowsAhead<1, NV>::smem(int(blockDim.x))) + threadIdx.x;
    float2 w[NV][H], b[NV][H];
    if (!kReread) {
        at.load_columns(w, a.weight, 1.f);
        at.load_columns(b, a.bias, 0.f);
    }
    if (kShared) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < H; ++k)
                shared[(i * H + k) * blockDim.x] = make_float4(w[i][k].x, w[i][k].y, b[i][k].x, b[i][k].y);
    }
    const float inv_width = 1.f / float(a.width);
    // PAIR: the columns of the lower CTA, and what mean and squares are first taken over
    const int lower = min(NV * int(blockDim.x) * VE - at.offset(), a.width), mine = rank ? a.width - lower : lower;
    const float inv_mine = PAIR ? 1.f / float(mine) : inv_width;
    if (PAIR) tc::cluster_wait();  // both CTAs are ready
    bool ok = true;
    int row = at.row, n = 0;
    for (int base = at.base; base < a.rows; base += at.step, row += at.step) {
        Pack<T, VE> in[1][NV];
        feed.get(in);
        float2 v[NV][H], acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int k = 0; k < H; ++k) acc = vec::add2(acc, v[i][k] = in[0][i].f2(k));
        const float sum = vec::sum2(acc);
        float mean = __fmul_rn(G ? vec::group_sum<G ? G : 1>(sum) : vec::block_sum(sum, red[0]), inv_mine);
        acc = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int k = 0; k < H; ++k) v[i][k] = vec::add2(v[i][k], vec::both(-mean));
            if (!at.full(i)) {  // outside the row: in neither sum
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
        float squares = G ? vec::group_sum<G ? G : 1>(sq) : vec::block_sum(sq, red[1]);
        float off = 0.f;  // the mean is `mean` + off, the squares about it sum v^2 - (sum v) off
        const bool far = __fmul_rn(mean, mean) > __fmul_rn(16.f * inv_mine, squares);  // the same in all of the row's threads
        if (G ? __any_sync(0xffffffffu, far) : far) {
            acc = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int k = 0; k < H; ++k) acc = vec::add2(acc, v[i][k]);
            const float left = G ? vec::group_sum<G ? G : 1>(vec::sum2(acc)) : vec::block_sum(vec::sum2(acc), red[2]);
            if (far) {
                off = __fmul_rn(left, inv_mine);
                // rounding may leave less than 0 where all values are one
                squares = fmaxf(fmaf(-left, off, squares), 0.f);
            }
        }
        float shift = -off;  // v + shift: the values about the mean
        if (PAIR) {
            // squares about the row's mean: those about each half's, and
            // (difference of the means)^2 for each of its columns
            float4 low, up;
            pair.send(make_float4(mean, off, squares, 0.f), n & 1, rank, ok);
            pair.receive(low, up, n & 1, n >> 1, a.wait_ns, ok);
            const float part = __fmul_rn(float(lower), inv_width), rest = __fadd_rn(1.f, -part);
            const float apart = __fadd_rn(__fadd_rn(low.x, -up.x), __fadd_rn(low.y, -up.y));
            shift = fmaf(rank ? -part : rest, apart, shift);
            squares = fmaf(__fmul_rn(float(lower), rest), __fmul_rn(apart, apart), __fadd_rn(low.z, up.z));
            mean = __fadd_rn(up.x, fmaf(part, apart, up.y));
            ++n;
        } else {
            mean = __fadd_rn(mean, off);
        }
        const float var = __fmul_rn(squares, inv_width);
        const float rstd = rsqrtf(__fadd_rn(var, a.eps)), shifted = __fmul_rn(shift, rstd);
        if (row < a.rows) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (kReread) {
                    at.load_column(w[i], i, a.weight, 1.f);
                    at.load_column(b[i], i, a.bias, 0.f);
                }
                Pack<T, VE> o;
#pragma unroll
                for (int k = 0; k < H; ++k) {
                    if (kShared) {
                        const float4 t = shared[(i * H + k) * blockDim.x];
                        w[i][k] = make_float2(t.x, t.y), b[i][k] = make_float2(t.z, t.w);
                    }
                    o.set2(k, vec::fma2(vec::fma2(v[i][k], vec::both(rstd), vec::both(shifted)), w[i][k], b[i][k]));
                }
                at.store(o, i, y + (long long)row * a.width);
            }
            if (at.tid == 0 && rank == 0) {
                if (a.mean) a.mean[row] = mean;
                if (a.rstd) a.rstd[row] = rstd;
            }
        }
    }
    if (PAIR) pair.leave(ok, at.rows_of(a.rows), rank, a.status);
}

template <typename T, int NV, int G, bool ALIGNED, bool PAIR>
struct Run {
    static cudaError_t run(const ln::Shape &sh, const LnArgs &a, cudaStream_t s) {
        const auto fn = k_layernorm<T, NV, G, ALIGNED, PAIR>;
        const void *f = reinterpret_cast<const void *>(fn);
        struct Key;
        constexpr int kElements = NV * 16 / int(sizeof(T));  // of a thread
        size_t smem = vec::RowsAhead<1, NV>::smem(sh.threads);
        if (kElements > 16 && sizeof(T) == 2) smem += size_t(sh.threads) * kElements * 2 * sizeof(float);
        const cudaError_t e = ln::allow_smem(f, smem);
        if (e != cudaSuccess) return e;
        const long long units = ((long long)a.rows + sh.rows_per_cta - 1) / sh.rows_per_cta;
        // all CTAs at once
        int most = ln::kSms * ln::ctas_per_sm<Key>(f, sh.threads, smem) / sh.ctas();
        if (!ALIGNED) most = most / 8 * 8;  // keeps a thread's rows at one misalignment
        return ln::launch(fn, sh, units < most ? units : most, smem, s, a);
    }
};

}  // namespace

cudaError_t launch_layernorm(const void *x, const float *weight, const float *bias, float eps, void *y, float *mean,
                             float *rstd, int rows, int width, int io_dtype, int *status, unsigned long long wait_ns,
                             cudaStream_t s) {
    if (rows == 0) return cudaSuccess;
    const LnArgs a{x, weight, bias, eps, y, mean, rstd, rows, width, status, wait_ns};
    LaunchScope scope(GDN_K_LAYERNORM, s);
    if (io_dtype == GDN_DT_BF16)
        return ln::dispatch<__nv_bfloat16, true, Run>(ln::shape_of<__nv_bfloat16, true>(rows, width), a, s);
    return ln::dispatch<float, true, Run>(ln::shape_of<float, true>(rows, width), a, s);
}

}  // namespace gdn
