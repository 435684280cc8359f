// Linear attention with a decay for each head: segments of the sequences, the
// chain of their sums, sums over a group's heads, and how long segments are.
#include "gdn_linattn.cuh"

namespace gdn {
namespace la {
namespace {

constexpr int kTableThreads = 1024;

__device__ __forceinline__ int seq_begin(const Args &a, int n) { return a.cu ? a.cu[n] : n * a.dense_seqlen; }
// an empty sequence has one empty segment: its state passes through
__device__ __forceinline__ int seq_segs(int len, int seg_len) { return len > 0 ? (len - 1) / seg_len + 1 : 1; }

// One CTA: checks the offsets (start at 0, do not decrease, end at the token
// count), counts each sequence's segments, and lists them.
__global__ void __launch_bounds__(kTableThreads) k_la_table(const __grid_constant__ Args a) {
    __shared__ int wsum[32];
    __shared__ int bad;
    next_may_start();
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, N = a.num_seqs;
    if (tid == 0) bad = 0;
    __syncthreads();
    const int per = (N + kTableThreads - 1) / kTableThreads;
    const int n0 = min(N, tid * per), n1 = min(N, n0 + per);
    int local = 0, last = n0 < n1 ? seq_begin(a, n0) : 0;
    if (n0 == 0 && n0 < n1 && last != 0) bad = 1;
    for (int n = n0; n < n1; ++n) {
        const int e = seq_begin(a, n + 1);
        if (e < last || last < 0 || e > a.total_tokens) bad = 1;
        else local += seq_segs(e - last, a.seg_len);
        last = e;
    }
    if (n0 < n1 && n1 == N && last != a.total_tokens) bad = 1;
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) wsum[wid] = incl;
    __syncthreads();
    if (bad) {  // the same for all behind the barrier
        if (tid == 0) {
            record_status(a.status, GDN_EDEVICE_INPUT);
            *a.n_segs = 0;
        }
        return;
    }
    if (wid == 0) {
        int x = wsum[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += t;
        }
        wsum[lane] = x;
    }
    __syncthreads();
    int first = (wid > 0 ? wsum[wid - 1] : 0) + incl - local;
    const int total = wsum[31];
    if (tid == 0) {
        *a.n_segs = total;
        a.seq_first[N] = total;
    }
    for (int n = n0; n < n1; ++n) {
        a.seq_first[n] = first;
        first += seq_segs(seq_begin(a, n + 1) - seq_begin(a, n), a.seg_len);
    }
    __syncthreads();
    for (int i = tid; i < total; i += kTableThreads) {
        int lo = 0, hi = N - 1;  // the last sequence whose first segment is at most i
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.seq_first[mid] <= i) lo = mid;
            else hi = mid - 1;
        }
        const int b = seq_begin(a, lo), len = seq_begin(a, lo + 1) - b, k = i - a.seq_first[lo];
        const int rest = len - k * a.seg_len;
        a.segs[i] = Seg{lo, b + k * a.seg_len, min(a.seg_len, rest),
                        (k == 0 ? kFirst : 0) | (rest <= a.seg_len ? kLast : 0)};
    }
}

// Chains the segments' sums: behind it, states[seg] is the state that enters
// the segment (of those that another one comes before). Four elements a
// thread; a sequence's segments one after the other. Bound by memory: each sum is
// read and replaced (9 us for 19 segments of 32 heads). The sums of eight
// segments are on their way together: one at a time took 120 us for 57 segments,
// eight 17.
constexpr int kChainThreads = 256, kChainCtas = kState / 4 / kChainThreads, kChainBatch = 8;

__global__ void __launch_bounds__(kChainThreads) k_la_chain(const __grid_constant__ Args a) {
    next_may_start();
    wait_for_previous();
    if (*a.n_segs == 0) return;
    const int part = blockIdx.x % kChainCtas, rest = blockIdx.x / kChainCtas, h = rest % a.hv;
    const Role &r = a.role[rest / a.hv];
    const float decay = a.decay[h];
    const int e = (part * kChainThreads + threadIdx.x) * 4;
    const size_t per_head = size_t(a.hv) * kState;
    for (int n = blockIdx.y; n < a.num_seqs; n += gridDim.y) {
        const int s0 = a.seq_first[n], s1 = a.seq_first[n + 1];
        if (s1 - s0 < 2) continue;
        const int step = r.against ? -1 : 1, from = r.against ? s1 - 1 : s0, count = s1 - s0;
        float *states = r.states + size_t(h) * kState + e;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f), left = s;
        if (r.init) {
            const float *init = r.init + size_t(n) * per_head + size_t(h) * kState;
            if (r.swapped) {
                const int b = e / kHeadDim, c = e % kHeadDim;
                s = make_float4(init[c * kHeadDim + b], init[(c + 1) * kHeadDim + b], init[(c + 2) * kHeadDim + b],
                                init[(c + 3) * kHeadDim + b]);
            } else {
                s = *reinterpret_cast<const float4 *>(init + e);
            }
        }
        // the sums come in batches, whose loads are under way together
        for (int k = 1; k < count; k += kChainBatch) {
            float4 sum[kChainBatch];
            float keep[kChainBatch];
#pragma unroll
            for (int i = 0; i < kChainBatch; ++i) {
                if (k + i >= count) break;
                const int at = from + (k + i - 1) * step;  // the segment left
                sum[i] = k + i == 1 || i > 0 ? *reinterpret_cast<const float4 *>(states + size_t(at) * per_head) : left;
                const Seg seg = a.segs[at];
                keep[i] = power(decay, seg.len - 1 + entry_offset(r, seg, true));
            }
            // (the batch's last place is read before the state goes there: it is the next one's first sum)
            if (k + kChainBatch < count)
                left = *reinterpret_cast<const float4 *>(states + size_t(from + (k + kChainBatch - 1) * step) * per_head);
#pragma unroll
            for (int i = 0; i < kChainBatch; ++i) {
                if (k + i >= count) break;
                s.x = fmaf(keep[i], s.x, sum[i].x), s.y = fmaf(keep[i], s.y, sum[i].y);
                s.z = fmaf(keep[i], s.z, sum[i].z), s.w = fmaf(keep[i], s.w, sum[i].w);
                *reinterpret_cast<float4 *>(states + size_t(from + (k + i) * step) * per_head) = s;
            }
        }
    }
}

// y[t, hq] = sum over the group's heads of x[t, hv], in their order, rounded once; of two tensors; nothing after a failed
// check, whose x nobody wrote. Bound by memory: 25 us for 4096 tokens x 32 heads on 16 (168 MB, 6.7 TB/s).
template <typename T>
__global__ void __launch_bounds__(256) k_la_group_sums(const float *__restrict__ x0, T *__restrict__ y0,
                                                       const float *__restrict__ x1, T *__restrict__ y1, long long items,
                                                       int group, const int *n_segs) {
    wait_for_previous();
    if (*n_segs == 0) return;
    const float *x = blockIdx.y ? x1 : x0;
    T *y = blockIdx.y ? y1 : y0;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;  // four channels of a (token, query head)
    if (i >= items) return;
    const float *from = x + (i / 32 * group) * kHeadDim + (i % 32) * 4;
    float4 s = *reinterpret_cast<const float4 *>(from);
    for (int g = 1; g < group; ++g) {
        const float4 v = *reinterpret_cast<const float4 *>(from + g * kHeadDim);
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    vec::Pack<T, 4> out;
    out.set2(0, make_float2(s.x, s.y));
    out.set2(1, make_float2(s.z, s.w));
    out.store(y + i * 4);
}

}  // namespace

cudaError_t launch_table(const Args &a, cudaStream_t s) {
    LaunchScope scope(GDN_K_LINATTN_TABLE, s);
    k_la_table<<<1, kTableThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_chain(const Args &a, cudaStream_t s) {
    LaunchScope scope(GDN_K_LINATTN_CHAIN, s);
    return launch_behind(k_la_chain, dim3(unsigned(kChainCtas) * unsigned(a.hv) * unsigned(a.roles),
                                          unsigned(a.num_seqs < 1024 ? a.num_seqs : 1024)),
                         kChainThreads, 0, s, a);
}

cudaError_t launch_group_sums(const float *x0, void *y0, const float *x1, void *y1, long long rows, int heads, int group,
                              const int *n_segs, int io_dtype, cudaStream_t s) {
    const long long items = rows * heads * 32;
    if (items == 0) return cudaSuccess;
    LaunchScope scope(GDN_K_LINATTN_GROUP_SUM, s);
    const dim3 ctas(unsigned((items + 255) / 256), 2);
    if (io_dtype == GDN_DT_BF16)
        return launch_behind(k_la_group_sums<__nv_bfloat16>, ctas, 256, 0, s, x0, static_cast<__nv_bfloat16 *>(y0), x1,
                             static_cast<__nv_bfloat16 *>(y1), items, group, n_segs);
    return launch_behind(k_la_group_sums<float>, ctas, 256, 0, s, x0, static_cast<float *>(y0), x1,
                         static_cast<float *>(y1), items, group, n_segs);
}

// Rows of a segment: those with the least estimated time. Microseconds of a
// chunk (bf16: 128 rows, f32: blocks of 32) in the walk and in the sum, of a
// CTA's start and end, and of the two kernels that several segments need. bf16:
// as measured at 4096 and 65536 tokens x 32 heads; f32: on 76 to 608 CTAs of 1 to
// 32 blocks; both with a CTA an SM.
// Against the best of 2 to 17 lengths the choice took up to 9% longer for 47 of 50
// calls: one sequence of 200 to 16384 tokens and sets of 2 to 64, 2 to 40 heads,
// forward and backward. The others, bf16, are a sequence of 4000 tokens with one
// of 60 (11%), ten of 0 to 1000 backward (16%), 8000 with two of 100 backward (23%).
int segment_rows(long long total_tokens, long long num_seqs, int hv, int roles, int io_dtype) {
    const bool tc = io_dtype == GDN_DT_BF16;
    const int unit = tc ? 128 : 32;
    const double slots = 152, walk = tc ? 2.8 : 10.5, sum = tc ? 1.3 : 4.4, start = tc ? 14.0 : 4.0, kernels = 8.0;
    const long long units = (total_tokens + unit - 1) / unit;
    const double heads = double(hv) * roles;
    auto waves = [&](double items) { return ceil(items / slots); };
    long long best = 1;
    double least = 0;
    for (long long u = 1;; u = u < 16 ? u + 1 : u + u / 8) {
        if (u > units && u > 1) u = units;
        const bool cut = u < units;
        const double t = waves(double((units + u - 1) / u + num_seqs - 1) * heads) * (start + double(u) * (cut ? walk + sum : walk)) +
                         (cut ? kernels : 0);
        if (u == 1 || t < least) least = t, best = u;
        if (u >= units || u * unit >= 65536) break;
    }
    // Several sequences (their lengths are on the device): segments of twice the mean length leave most of them whole,
    // and those need no sums. Lengths that differ cost a quarter where CTAs take several, half where they take one; equal
    // ones whole rounds (bf16 8 prompts x 32 heads 278 us whole and 347 to 438 cut, 64 short ones 258 and 281 to 567; f32
    // 4 x 1500 tokens x 40 heads 982 whole and 792 cut).
    if (num_seqs > 1) {
        const double mean = double(units) / double(num_seqs), items = double(num_seqs) * heads;
        const double rounds = fmax(waves(items), 1.25 * items / slots);
        const double whole = (items > slots ? rounds * (start + mean * walk) : start + 1.5 * mean * walk) + kernels;
        const long long u = (2 * units + num_seqs - 1) / num_seqs;
        if (whole < least && u > 0 && u * unit < 65536) best = u;
    }
    return int(best * unit);
}

}  // namespace la
}  // namespace gdn
