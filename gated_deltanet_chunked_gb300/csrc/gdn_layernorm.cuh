// How the layer norm's kernels divide a row of `width` elements.
//
// A row is held in registers, so that it is read once; every load is 16 bytes,
// VE elements, NV of them a thread. Rows whose width is no multiple of VE do
// not start on 16 bytes: such a row's vectors begin up to VE - 1 elements
// before it, at the last aligned address; of its first and last vector the
// elements outside the row are read with the others (not past the tensor's
// end), replaced by zeros and not written. A CTA's rows are a multiple of eight
// apart, so all rows of a thread have the same misalignment and it owns the
// same columns of all.
// G lanes of a warp share a row where it is short, so that no lane is without
// elements; longer rows take a whole CTA (G = 0).
#pragma once

#include <atomic>

#include "gdn_async.cuh"
#include "gdn_common.cuh"

namespace gdn {
namespace ln {

constexpr int kSms = 152;
constexpr int kRowThreads = 256;  // threads of a CTA whose warps take rows of their own, and wanted of others

struct Shape {
    bool aligned;      // every row starts on 16 bytes
    int nv, g;         // loads per thread, lanes per row (0: the CTA, or a pair)
    int threads;       // of a CTA
    int rows_per_cta;  // rows in work at a time
    bool pair;         // a row is on a cluster of two CTAs
    int ctas() const { return pair ? 2 : 1; }
};

// Long rows: 16 elements a thread, which is the least of reductions and
// barriers for an element; few rows (latency counts) over as many threads as
// help. Rows that so take more than 512 threads are on two CTAs, which tell
// each other their sums; or (LONG, the forward pass) on 512 threads with 32
// elements each where they are aligned: 3000 x 16384 43 us, on two CTAs 57;
// unaligned, 3000 x 16383, 126 and 77. Many bf16 rows of more than 400 such
// threads are better on half of them too, so that an SM has two CTAs: 8000 x
// 8192 46 us against 57, 7000 wide 46 and 59, but 6000 wide 30 and 29, and 400
// rows of 8192 5.9 and 5.2.
template <typename T, bool LONG>
inline Shape shape_of(int rows, int width) {
    constexpr int VE = 16 / int(sizeof(T)), kMost = 16 / VE;  // at most 16 elements a thread
    Shape s;
    s.aligned = width % VE == 0;
    const int vecs = s.aligned ? width / VE : (width + VE - 1 + VE - 1) / VE;  // for any misalignment
    s.g = vecs <= 16 ? 16 : vecs <= 32 * kMost ? 32 : 0;
    s.nv = 1;
    if (!s.g && rows > 16 * kSms) {
        s.nv = kMost;
        // LONG, bf16: not where three warps with one vector a lane do and two
        // with two would have three tenths of their places empty (83333 x 600:
        // 45 us for 49, 71428 x 700: 56 for 63; the backward pass and f32 lose
        // as much, and so does 1040 wide with five warps for three)
        if (LONG && sizeof(T) == 2 && vecs < 90) s.nv = 1;
    }
    while (s.nv < kMost && vecs > (s.g ? s.g : kRowThreads) * s.nv) s.nv *= 2;
    const bool more = LONG && s.aligned;  // elements a thread
    const bool wide = !s.g && vecs > (more && sizeof(T) == 2 && rows > 4 * kSms ? 400 : 512) * s.nv;
    s.pair = wide && !more;
    if (wide && !s.pair) s.nv *= 2;
    const int each = s.nv * s.ctas();  // vectors of a thread, and of that at its place in the other CTA
    s.threads = s.g ? kRowThreads : ((vecs + each - 1) / each + 31) / 32 * 32;
    s.rows_per_cta = s.g ? kRowThreads / s.g : 1;
    return s;
}

// calls F<T, NV, G, ALIGNED, PAIR>(...) for the shape
template <typename T, bool LONG, template <typename, int, int, bool, bool> class F, bool ALIGNED, typename... A>
inline cudaError_t dispatch_nv(const Shape &s, A &...a) {
    constexpr int kMost = 4 * int(sizeof(T)) / 4;  // 16 / VE: 2 for bf16, 4 for f32
    if (s.g == 16) return F<T, 1, 16, ALIGNED, false>::run(s, a...);
    if (s.g == 32) {
        if (s.nv == 1) return F<T, 1, 32, ALIGNED, false>::run(s, a...);
        if (s.nv == 2) return F<T, 2, 32, ALIGNED, false>::run(s, a...);
        return F<T, kMost, 32, ALIGNED, false>::run(s, a...);
    }
    if constexpr (LONG && ALIGNED) {
        if (s.nv > kMost) return F<T, 2 * kMost, 0, ALIGNED, false>::run(s, a...);
    } else {
        if (s.pair) return F<T, kMost, 0, ALIGNED, true>::run(s, a...);
    }
    if (s.nv == 1) return F<T, 1, 0, ALIGNED, false>::run(s, a...);
    if (s.nv == 2) return F<T, 2, 0, ALIGNED, false>::run(s, a...);
    return F<T, kMost, 0, ALIGNED, false>::run(s, a...);
}
template <typename T, bool LONG, template <typename, int, int, bool, bool> class F, typename... A>
inline cudaError_t dispatch(const Shape &s, A &...a) {
    return s.aligned ? dispatch_nv<T, LONG, F, true>(s, a...) : dispatch_nv<T, LONG, F, false>(s, a...);
}

// Launches `units` CTAs, or pairs of CTAs.
template <typename... P, typename... A>
inline cudaError_t launch(void (*fn)(P...), const Shape &sh, long long units, size_t smem, cudaStream_t s,
                          const A &...a) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at = {};
    cfg.gridDim = dim3(unsigned(units * sh.ctas()));
    cfg.blockDim = dim3(unsigned(sh.threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = unsigned(sh.ctas());
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = sh.pair ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, fn, a...);
}

// Sums that the two CTAs of a pair tell each other, one row after the other, in
// shared memory: two buffers in turn. A buffer's next sums come when both CTAs
// have sent the other's, and so have read these. ok is each thread's own: it
// turns false when its wait runs out, and the rows go on on what is there,
// without waits of that thread. Thread 0 sends, and none after its own.
// V: float2 or float4.
template <typename V>
struct Pair {
    V sums[2][2];  // by buffer, CTA
    uint64_t bar[2];
    tc::GiveUp<2> gave_up;
    int sent;  // rows, by a CTA whose thread 0 gave up

    __device__ __forceinline__ void init() {  // by one thread, before a cluster barrier
        tc::mbar_init(&bar[0], 1);
        tc::mbar_init(&bar[1], 1);
        tc::fence_mbar_init();
        gave_up.sent[0] = gave_up.sent[1] = 0;
    }
    // tells both CTAs v, the same in all threads of one
    __device__ __forceinline__ void send(V v, int buf, int rank, bool ok) {
        using namespace tc;
        if (threadIdx.x || !ok) return;
        mbar_arrive_expect_tx(&bar[buf], 2 * sizeof(V));
#pragma unroll
        for (int r = 0; r < 2; ++r)
            cluster_st_async(cluster_map(&sums[buf][rank], r), v, cluster_map(&bar[buf], r));
    }
    // what both have sent, for the use-th time to buffer `buf`
    __device__ __forceinline__ void receive(V &lower, V &upper, int buf, int use, unsigned long long wait_ns, bool &ok) {
        if (ok && !tc::mbar_wait_cluster(&bar[buf], uint32_t(use) & 1, wait_ns)) {
            ok = false;
            if (threadIdx.x == 0) sent = 2 * use + buf + 1;
        }
        lower = sums[buf][0], upper = sums[buf][1];
    }
    // after the last of `rows` rows
    __device__ __forceinline__ void leave(bool ok, int rows, int rank, int *status) {
        using namespace tc;
        if (__any_sync(0xffffffffu, !ok) && (threadIdx.x & 31) == 0) record_status(status, GDN_ETIMEOUT);
        if (__shfl_sync(0xffffffffu, int(threadIdx.x == 0 && !ok), 0)) {
            if (threadIdx.x == 0) gave_up.tell(sent, rank, 2);
            cluster_arrive();
        } else {
            cluster_arrive_relaxed();
        }
        cluster_wait();  // neither CTA sends any more, and none leaves while the other may
        if (threadIdx.x < 32) gave_up.settle(bar, rows, rank, 2, sizeof(V));
    }
};

// CTAs of kernel `fn` that an SM holds at `threads` each, asked once a kernel
// (K: a type of its own, whose shared memory is a function of the threads),
// thread count and device.
template <typename K>
inline int ctas_per_sm(const void *fn, int threads, size_t smem) {
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices][33];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) dev = -1;
    int n = dev < 0 ? 0 : known[dev][threads / 32].load(std::memory_order_relaxed);
    if (n > 0) return n;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, threads, smem) != cudaSuccess || n < 1) n = 1;
    if (dev >= 0) known[dev][threads / 32].store(n, std::memory_order_relaxed);
    return n;
}

// Lets `fn` have so much dynamic shared memory; a kernel's static variables (up
// to 16 KB here) count against the 48 KB that need no leave.
inline cudaError_t allow_smem(const void *fn, size_t bytes) {
    return bytes <= 24 << 10 ? cudaSuccess
                             : cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
}

// A thread's place: its row group, and its vectors' columns.
template <typename T, int NV, int G, bool ALIGNED>
struct Place {
    static constexpr int VE = 16 / int(sizeof(T));
    using P = vec::Pack<T, VE>;
    int tid;
    int row, base, step;  // first row; first row of the warp (CTA), which decides when it ends; rows apart
    int col[NV];
    int width;

    // a row on `ctas` CTAs, of which this is the rank-th
    __device__ __forceinline__ Place(int w, int rank, int ctas) : width(w) {
        constexpr int g = G ? G : 1;
        const int groups = G ? int(blockDim.x) / g : 1, group = G ? int(threadIdx.x) / g : 0;
        tid = G ? int(threadIdx.x) % g : int(threadIdx.x);
        row = int(blockIdx.x) / ctas * groups + group;
        base = G ? row - (threadIdx.x & 31) / g : row;
        step = int(gridDim.x) / ctas * groups;
        const int off = offset();
#pragma unroll
        for (int i = 0; i < NV; ++i)
            col[i] = (tid + (rank * NV + i) * (G ? G : int(blockDim.x))) * VE - off;
    }
    // how many of `rows` rows are its CTA's (G = 0)
    __device__ __forceinline__ int rows_of(int rows) const { return base < rows ? (rows - 1 - base) / step + 1 : 0; }
    // elements before the row in its first vector
    __device__ __forceinline__ int offset() const { return ALIGNED ? 0 : int((long long)row * width % VE); }
    __device__ __forceinline__ bool full(int i) const {
        return ALIGNED ? col[i] < width : col[i] >= 0 && col[i] + VE <= width;
    }
    // whether element j of vector i is in the row
    __device__ __forceinline__ bool has(int i, int j) const {
        return ALIGNED ? col[i] < width : unsigned(col[i] + j) < unsigned(width);
    }
    // of the row at p
    __device__ __forceinline__ void store(const P &v, int i, T *p) const {
        if (full(i)) {
            v.store(p + col[i]);
        } else if (!ALIGNED) {
#pragma unroll
            for (int j = 0; j < VE; ++j)
                if (has(i, j)) p[col[i] + j] = v.e[j];
        }
    }
    // pairs of a per-column f32 array (null: `otherwise`); what it gives
    // outside the row is not used
    __device__ __forceinline__ void load_column(float2 (&w)[VE / 2], int i, const float *p, float otherwise) const {
#pragma unroll
        for (int j = 0; j < VE; j += 4) {
            if (ALIGNED) {
                float4 t = make_float4(otherwise, otherwise, otherwise, otherwise);
                if (p && full(i)) t = *reinterpret_cast<const float4 *>(p + col[i] + j);
                w[j / 2] = make_float2(t.x, t.y);
                w[j / 2 + 1] = make_float2(t.z, t.w);
            } else {
                float t[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) t[m] = !has(i, j + m) ? 0.f : p ? p[col[i] + j + m] : otherwise;
                w[j / 2] = make_float2(t[0], t[1]);
                w[j / 2 + 1] = make_float2(t[2], t[3]);
            }
        }
    }
    __device__ __forceinline__ void load_columns(float2 (&w)[NV][VE / 2], const float *p, float otherwise) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) load_column(w[i], i, p, otherwise);
    }
};

// The thread's vectors of its rows of NT tensors in turn, read ahead through
// its own place in shared memory.
template <typename T, int NT, int NV, int G, bool ALIGNED>
struct Feed {
    using L = Place<T, NV, G, ALIGNED>;
    using A = vec::RowsAhead<NT, NV>;
    using P = typename L::P;

    const L &at;
    const T *src[NT];  // of the next row to ask for, at the thread's first vector
    long long pitch;   // elements between this thread's rows
    long long rest;    // elements from src to the tensor's end (unaligned rows)
    int left;          // rows still to ask for
    bool any[NV];      // whether the vector has elements of the row
    // Its bits that are of the row, the same for all rows; not in the forward
    // pass of long rows, which has no registers left for them (4095 wide 61 us
    // for 53; where they are, 150150 x 333 backward takes 100 for 131, forward
    // 62 for 71)
    static constexpr bool kMasks = !ALIGNED && (NT > 1 || G);
    uint32_t keep[kMasks ? NV : 1][4];
    A a;

    __device__ __forceinline__ Feed(const L &place, const T *const (&from)[NT], int rows, void *smem)
        : at(place), pitch((long long)place.step * place.width), a(smem) {
        left = at.row < rows ? (rows - 1 - at.row) / at.step + 1 : 0;
        rest = (long long)(rows - at.row) * at.width - at.col[0];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            any[i] = at.col[i] < at.width;
            if constexpr (kMasks) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    constexpr int kOf = 4 / int(sizeof(T));  // elements of a word
                    keep[i][k] = (at.has(i, k * kOf) ? sizeof(T) == 4 ? ~0u : 0xffffu : 0u) |
                                 (kOf == 2 && at.has(i, k * kOf + kOf - 1) ? 0xffff0000u : 0u);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) src[t] = from[t] + (long long)at.row * at.width + at.col[0];
#pragma unroll
        for (int s = 0; s < A::kAhead; ++s) ask();
    }
    // whether element j of vector i is in the row
    __device__ __forceinline__ bool in_row(int i, int j) const {
        constexpr int kOf = 4 / int(sizeof(T));
        return kMasks ? keep[kMasks ? i : 0][j / kOf] >> (j % kOf * 16) & 1 : at.has(i, j);
    }
    __device__ __forceinline__ void ask() {
        if (left > 0) {
            constexpr int VE = L::VE;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int off = (G ? G * VE : int(blockDim.x) * VE) * i;
                    if (!any[i]) continue;
                    if (ALIGNED || rest - off >= VE) a.copy(t * NV + i, src[t] + off);
                    else a.copy_part(t * NV + i, src[t] + off, int(rest - off) * int(sizeof(T)));
                }
        }
        if (!ALIGNED) rest -= pitch;
#pragma unroll
        for (int t = 0; t < NT; ++t) src[t] += pitch;
        --left;
        a.commit();
    }
    // the next row's vectors: zeros outside the row, anything where there is no row
    __device__ __forceinline__ void get(P (&v)[NT][NV]) {
        ask();
        a.wait();
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (kMasks) {
                    const uint32_t(&m)[4] = keep[kMasks ? i : 0];
                    const uint4 r = a.take(t * NV + i);  // where the vector has none of the row, what happens to be there
                    v[t][i].r = make_uint4(r.x & m[0], r.y & m[1], r.z & m[2], r.w & m[3]);
                    continue;
                }
                if (any[i]) v[t][i].r = a.take(t * NV + i);
                else v[t][i].zero();
                if (!ALIGNED && any[i] && !at.full(i)) {
#pragma unroll
                    for (int j = 0; j < L::VE; ++j)
                        if (!at.has(i, j)) v[t][i].set(j, 0.f);
                }
            }
        a.taken();
    }
};

}  // namespace ln
}  // namespace gdn
