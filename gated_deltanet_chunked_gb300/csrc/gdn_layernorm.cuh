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

namespace gdn {
namespace ln {

constexpr int kSms = 152;
constexpr int kRowThreads = 256;  // threads of a CTA whose warps take rows of their own, and wanted of others

struct Shape {
    bool aligned;      // every row starts on 16 bytes
    int nv, g;         // loads per thread, lanes per row (0: the CTA)
    int threads;       // of a CTA
    int rows_per_cta;  // rows in work at a time
};

// Long rows: 16 elements a thread, which is the least of reductions and
// barriers for an element; few rows (latency counts) over as many threads as
// help. Where that takes more than 512 threads, `most` = 32 elements a thread
// keep two CTAs on an SM, whose reductions overlap (3000 x 16384 bf16 forward:
// 56 us with 1024 threads, 51 with 512).
template <typename T>
inline Shape shape_of(int rows, int width, int most = 16) {
    constexpr int VE = 16 / int(sizeof(T)), kMost = 16 / VE;  // at most 16 elements a thread
    Shape s;
    s.aligned = width % VE == 0;
    const int vecs = s.aligned ? width / VE : (width + VE - 1 + VE - 1) / VE;  // for any misalignment
    s.g = vecs <= 16 ? 16 : vecs <= 32 * kMost ? 32 : 0;
    s.nv = 1;
    if (!s.g && rows > 16 * kSms) s.nv = kMost;
    while (s.nv < kMost && vecs > (s.g ? s.g : kRowThreads) * s.nv) s.nv *= 2;
    // (also the widest unaligned rows, by a few elements one vector too many for 1024 threads)
    if (!s.g && vecs > (most > 16 ? 512 : 1024) * s.nv) s.nv *= 2;
    s.threads = s.g ? kRowThreads : ((vecs + s.nv - 1) / s.nv + 31) / 32 * 32;
    s.rows_per_cta = s.g ? kRowThreads / s.g : 1;
    return s;
}

// calls F<T, NV, G, ALIGNED>(...) for the shape
template <typename T, template <typename, int, int, bool> class F, bool ALIGNED, typename... A>
inline cudaError_t dispatch_nv(const Shape &s, A &...a) {
    constexpr int kMost = 4 * int(sizeof(T)) / 4;  // 16 / VE: 2 for bf16, 4 for f32
    if (s.g == 16) return F<T, 1, 16, ALIGNED>::run(s, a...);
    if (s.g == 32) {
        if (s.nv == 1) return F<T, 1, 32, ALIGNED>::run(s, a...);
        if (s.nv == 2) return F<T, 2, 32, ALIGNED>::run(s, a...);
        return F<T, kMost, 32, ALIGNED>::run(s, a...);
    }
    if (s.nv == 1) return F<T, 1, 0, ALIGNED>::run(s, a...);
    if (s.nv == 2) return F<T, 2, 0, ALIGNED>::run(s, a...);
    if (s.nv == kMost) return F<T, kMost, 0, ALIGNED>::run(s, a...);
    return F<T, 2 * kMost, 0, ALIGNED>::run(s, a...);
}
template <typename T, template <typename, int, int, bool> class F, typename... A>
inline cudaError_t dispatch(const Shape &s, A &...a) {
    return s.aligned ? dispatch_nv<T, F, true>(s, a...) : dispatch_nv<T, F, false>(s, a...);
}

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

    __device__ __forceinline__ Place(int w) : width(w) {
        constexpr int g = G ? G : 1;
        const int groups = G ? int(blockDim.x) / g : 1, group = G ? int(threadIdx.x) / g : 0;
        tid = G ? int(threadIdx.x) % g : int(threadIdx.x);
        row = int(blockIdx.x) * groups + group;
        base = G ? row - (threadIdx.x & 31) / g : row;
        step = int(gridDim.x) * groups;
        const int off = ALIGNED ? 0 : int((long long)row * width % VE);
#pragma unroll
        for (int i = 0; i < NV; ++i) col[i] = (tid + i * (G ? G : int(blockDim.x))) * VE - off;
    }
    __device__ __forceinline__ bool full(int i) const {
        return ALIGNED ? col[i] < width : col[i] >= 0 && col[i] + VE <= width;
    }
    // whether element j of vector i is in the row
    __device__ __forceinline__ bool has(int i, int j) const {
        return ALIGNED ? col[i] < width : unsigned(col[i] + j) < unsigned(width);
    }
    // vector i of the row at p; zeros outside the row
    __device__ __forceinline__ void load(P &v, int i, const T *p) const {
        if (full(i)) {
            v.load(p + col[i]);
        } else if (!ALIGNED) {
#pragma unroll
            for (int j = 0; j < VE; ++j)
                if (has(i, j)) v.e[j] = p[col[i] + j];
        }
    }
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

// The thread's vectors of its rows of NT tensors in turn, read ahead: through
// its own place in shared memory, or (IN_SMEM false: a CTA of 1024 threads)
// one row ahead in registers.
template <typename T, int NT, int NV, int G, bool ALIGNED, bool IN_SMEM>
struct Feed {
    using L = Place<T, NV, G, ALIGNED>;
    using A = vec::RowsAhead<NT, NV>;
    using P = typename L::P;
    static __host__ __device__ size_t smem(int threads) { return IN_SMEM ? A::smem(threads) : 0; }

    const L &at;
    const T *src[NT];  // of the next row to ask for, at the thread's first vector
    long long pitch;   // elements between this thread's rows
    long long rest;    // elements from src to the tensor's end (unaligned rows)
    int left;          // rows still to ask for
    bool any[NV];      // whether the vector has elements of the row
    A a;
    P next[IN_SMEM ? 1 : NT][IN_SMEM ? 1 : NV];

    __device__ __forceinline__ Feed(const L &place, const T *const (&from)[NT], int rows, void *smem)
        : at(place), pitch((long long)place.step * place.width), a(smem) {
        left = at.row < rows ? (rows - 1 - at.row) / at.step + 1 : 0;
        rest = (long long)(rows - at.row) * at.width - at.col[0];
#pragma unroll
        for (int i = 0; i < NV; ++i) any[i] = at.col[i] < at.width;
#pragma unroll
        for (int t = 0; t < NT; ++t) src[t] = from[t] + (long long)at.row * at.width + at.col[0];
        if (IN_SMEM) {
#pragma unroll
            for (int s = 0; s < A::kAhead; ++s) ask();
        } else {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < NV; ++i) next[IN_SMEM ? 0 : t][IN_SMEM ? 0 : i].zero();
            ask();
        }
    }
    __device__ __forceinline__ void ask() {
        if (left > 0) {
            constexpr int VE = L::VE;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int off = (G ? G * VE : int(blockDim.x) * VE) * i;
                    if (!IN_SMEM) {
                        at.load(next[IN_SMEM ? 0 : t][IN_SMEM ? 0 : i], i, src[t] - at.col[0]);
                    } else if (any[i]) {
                        if (ALIGNED || rest - off >= VE) a.copy(t * NV + i, src[t] + off);
                        else a.copy_part(t * NV + i, src[t] + off, int(rest - off) * int(sizeof(T)));
                    }
                }
        }
        if (!ALIGNED) rest -= pitch;
#pragma unroll
        for (int t = 0; t < NT; ++t) src[t] += pitch;
        --left;
        if (IN_SMEM) a.commit();
    }
    // the next row's vectors: zeros outside the row, anything where there is no row
    __device__ __forceinline__ void get(P (&v)[NT][NV]) {
        if (IN_SMEM) {
            ask();
            a.wait();
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!IN_SMEM) v[t][i] = next[IN_SMEM ? 0 : t][IN_SMEM ? 0 : i];
                else if (any[i]) v[t][i].r = a.take(t * NV + i);
                else v[t][i].zero();
                if (IN_SMEM && !ALIGNED && any[i] && !at.full(i)) {
#pragma unroll
                    for (int j = 0; j < L::VE; ++j)
                        if (!at.has(i, j)) v[t][i].set(j, 0.f);
                }
            }
        if (IN_SMEM) a.taken();
        else ask();
    }
};

}  // namespace ln
}  // namespace gdn
