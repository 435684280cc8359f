// Gated linear recurrence (gdn_linear_recurrence, its backward pass and its
// decode step).
//
//   s_t = exp(g_t) s_{t-1} + x_t per channel, out = s
//   backward: ds_t = dout_t + e_{t+1}, e_t = exp(g_t) ds_t,
//             dx_t = ds_t, dg_t = exp(g_t) s_{t-1} ds_t
//
// One thread walks one channel of one sequence. The backward pass takes the
// state at every kRecTile-th row of the packed axis from the forward pass and
// recomputes the rows between, last tile first.
#include "gdn_linrec.cuh"
#include "gdn_vec.cuh"

namespace gdn {
namespace {

using vec::Pack;

// range of sequence n; false (and recorded) if the offsets are bad
__device__ __forceinline__ bool sequence(const RecArgs &a, int n, int &start, int &end) {
    if (!a.cu) {
        start = n * a.dense_seqlen;
        end = start + a.dense_seqlen;
        return true;
    }
    int bad = 0;
    for (int i = threadIdx.x; i < a.num_seqs; i += blockDim.x) bad |= a.cu[i] > a.cu[i + 1];
    if (a.cu[0] != 0 || a.cu[a.num_seqs] != a.total_tokens) bad = 1;
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) record_status(a.status, GDN_EDEVICE_INPUT);
        return false;
    }
    start = a.cu[n];
    end = a.cu[n + 1];
    return true;
}

template <typename T, bool CHANNEL>
__device__ __forceinline__ float decay(const RecArgs &a, int t, int h) {
    const long long row = (long long)t * a.hv + h;
    return expf(CHANNEL ? to_f32<T>(static_cast<const T *>(a.g)[row * kHeadDim + threadIdx.x])
                        : static_cast<const float *>(a.g)[row]);
}

template <typename T, bool CHANNEL>
__global__ void __launch_bounds__(kHeadDim) k_linrec(const RecArgs a) {
    const int h = blockIdx.x, n = blockIdx.y, c = threadIdx.x;
    int start, end;
    if (!sequence(a, n, start, end)) return;
    const T *x = static_cast<const T *>(a.x);
    T *out = static_cast<T *>(a.out);
    const long long srow = ((long long)n * a.hv + h) * kHeadDim + c;
    float s = a.s0 ? a.s0[srow] : 0.f;
    for (int t = start; t < end; ++t) {
        if (a.states && t % kRecTile == 0) a.states[((long long)(t / kRecTile) * a.hv + h) * kHeadDim + c] = s;
        const long long i = ((long long)t * a.hv + h) * kHeadDim + c;
        s = fmaf(decay<T, CHANNEL>(a, t, h), s, to_f32<T>(x[i]));
        out[i] = from_f32<T>(s);
    }
    if (a.final_state) a.final_state[srow] = s;
}

template <typename T, bool CHANNEL>
__global__ void __launch_bounds__(kHeadDim) k_linrec_bwd(const RecArgs a) {
    const int h = blockIdx.x, n = blockIdx.y, c = threadIdx.x;
    int start, end;
    if (!sequence(a, n, start, end)) return;
    const T *x = static_cast<const T *>(a.x), *dout = static_cast<const T *>(a.dout);
    T *dx = static_cast<T *>(a.dx);
    __shared__ float sums[4];
    const long long srow = ((long long)n * a.hv + h) * kHeadDim + c;
    float e = a.dfinal ? a.dfinal[srow] : 0.f;
    float before[kRecTile];  // the state before each row of the tile
    for (int t1 = end; t1 > start;) {
        const int tile = (t1 - 1) / kRecTile, t0 = max(start, tile * kRecTile);
        float s = t0 == start ? (a.s0 ? a.s0[srow] : 0.f) : a.states[((long long)tile * a.hv + h) * kHeadDim + c];
        for (int t = t0; t < t1; ++t) {
            before[t - t0] = s;
            s = fmaf(decay<T, CHANNEL>(a, t, h), s, to_f32<T>(x[((long long)t * a.hv + h) * kHeadDim + c]));
        }
        for (int t = t1 - 1; t >= t0; --t) {
            const long long i = ((long long)t * a.hv + h) * kHeadDim + c;
            const float ds = to_f32<T>(dout[i]) + e;
            dx[i] = from_f32<T>(ds);
            e = decay<T, CHANNEL>(a, t, h) * ds;
            const float dg = e * before[t - t0];
            if (CHANNEL) {
                static_cast<T *>(a.dg)[i] = from_f32<T>(dg);
            } else {
                const float w = vec::group_sum<32>(dg);
                __syncthreads();
                if ((c & 31) == 0) sums[c >> 5] = w;
                __syncthreads();
                if (c == 0)
                    static_cast<float *>(a.dg)[(long long)t * a.hv + h] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
            }
        }
        t1 = t0;
    }
    if (a.dinitial) a.dinitial[srow] = e;
}

// Decode step: a warp takes one (sequence, head) row, four channels a lane.
// HBM-bound (state read and written, x and out); every access of a warp is
// contiguous.
constexpr int kStepWarps = 4;

template <typename T, bool CHANNEL>
__global__ void __launch_bounds__(32 * kStepWarps)
k_linrec_step(const void *x_, const void *g_, float *state, const int32_t *idx, void *out_, int rows, int hv, int slots,
              int *status) {
    const int row = blockIdx.x * kStepWarps + (threadIdx.x >> 5), c = (threadIdx.x & 31) * 4;
    if (row >= rows) return;
    const int n = row / hv, h = row - n * hv;
    const int slot = idx ? idx[n] : n;
    if (slot < 0 || slot >= slots) {
        if (slot >= slots && c == 0) record_status(status, GDN_EDEVICE_INPUT);
        return;
    }
    const long long i = (long long)row * kHeadDim + c;
    Pack<T, 4> px, pg;
    px.load(static_cast<const T *>(x_) + i);
    float a[4];
    if (CHANNEL) {
        pg.load(static_cast<const T *>(g_) + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = expf(pg.f(j));
    } else {
        a[0] = a[1] = a[2] = a[3] = expf(static_cast<const float *>(g_)[row]);
    }
    Pack<float, 4> s;
    float *ps = state + ((long long)slot * hv + h) * kHeadDim + c;
    s.load(ps);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        s.e[j] = fmaf(a[j], s.e[j], px.f(j));
        px.set(j, s.e[j]);
    }
    s.store(ps);
    px.store(static_cast<T *>(out_) + i);
}

// calls F<T, CHANNEL> for the io dtype and the gate's form
template <template <typename, bool> class F, typename... A>
void for_type(int io_dtype, bool channel, A... args) {
    if (io_dtype == GDN_DT_BF16)
        channel ? F<__nv_bfloat16, true>::run(args...) : F<__nv_bfloat16, false>::run(args...);
    else
        channel ? F<float, true>::run(args...) : F<float, false>::run(args...);
}

template <typename T, bool CHANNEL>
struct Forward {
    static void run(const RecArgs &a, cudaStream_t s) {
        k_linrec<T, CHANNEL><<<dim3(unsigned(a.hv), unsigned(a.num_seqs)), kHeadDim, 0, s>>>(a);
    }
};
template <typename T, bool CHANNEL>
struct Backward {
    static void run(const RecArgs &a, cudaStream_t s) {
        k_linrec_bwd<T, CHANNEL><<<dim3(unsigned(a.hv), unsigned(a.num_seqs)), kHeadDim, 0, s>>>(a);
    }
};
template <typename T, bool CHANNEL>
struct Step {
    static void run(const void *x, const void *g, float *state, const int32_t *idx, void *out, int rows, int hv,
                    int slots, int *status, cudaStream_t s) {
        k_linrec_step<T, CHANNEL><<<unsigned((rows + kStepWarps - 1) / kStepWarps), 32 * kStepWarps, 0, s>>>(
            x, g, state, idx, out, rows, hv, slots, status);
    }
};

}  // namespace

cudaError_t launch_linrec(const RecArgs &a, int io_dtype, bool channel, cudaStream_t s) {
    LaunchScope scope(GDN_K_LINREC, s);
    for_type<Forward, const RecArgs &>(io_dtype, channel, a, s);
    return cudaGetLastError();
}

cudaError_t launch_linrec_bwd(const RecArgs &a, int io_dtype, bool channel, cudaStream_t s) {
    LaunchScope scope(GDN_K_LINREC_BWD, s);
    for_type<Backward, const RecArgs &>(io_dtype, channel, a, s);
    return cudaGetLastError();
}

cudaError_t launch_linrec_step(const void *x, const void *g, float *state, const int32_t *idx, void *out, int seqs,
                               int hv, int slots, int io_dtype, bool channel, int *status, cudaStream_t s) {
    if (seqs == 0) return cudaSuccess;
    LaunchScope scope(GDN_K_LINREC_STEP, s);
    for_type<Step>(io_dtype, channel, x, g, state, idx, out, seqs * hv, hv, slots, status, s);
    return cudaGetLastError();
}

}  // namespace gdn
