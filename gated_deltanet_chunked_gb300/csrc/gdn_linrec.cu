// Gated linear recurrence (gdn_linear_recurrence, its backward pass and its
// decode step).
//
//   s_t = exp(g_t) s_{t-1} + x_t per channel, out = s
//   backward: ds_t = dout_t + e_{t+1}, e_t = exp(g_t) ds_t,
//             dx_t = ds_t, dg_t = e_t s_{t-1}
//
// HBM-bound: the forward pass reads x and g and writes out, the backward pass
// reads x, g and dout and writes dx and dg, each once. What has to be won is
// parallelism along the time axis. A row's map s -> a s + x composes: a
// segment of rows is s -> A s + B with A the product of its decays. A cluster
// of CTAs takes one head and walks the packed token axis in rounds; in a round
// each CTA takes the next tile of kRecTile rows, each of its warps a segment
// of kSeg rows, each lane four channels:
//  1. every warp composes its segment's rows (tile in shared memory by TMA,
//     kept in registers from here on);
//  2. the CTA composes its segments and writes the result into every CTA of
//     the cluster (distributed shared memory);
//  3. one cluster barrier; then every CTA knows the state at its tile's first
//     row and, all in the same order, the state that the next round starts from;
//  4. every warp walks its segment again from its state and writes its rows.
// So a round costs one barrier instead of a chain of flags through global
// memory, needs no workspace, and adds in a fixed order: the same call gives
// the same bits. While a round runs, the next tiles are on their way.
//
// Sequences are boundaries on the one axis. A segment that holds a sequence's
// first row (for the backward pass: last row) does not depend on what comes
// before: that is marked in A (kReset) instead of multiplying by zero, so that
// an infinity or NaN of one sequence cannot reach the next.
//
// The backward pass walks the rounds from the last to the first with e in the
// place of s. It needs s_{t-1} too: the forward pass left the state before
// every tile in `states` (1/64 of x's rows), from which each CTA recomputes
// its tile's states by the same steps 1, 2 and 4 without any exchange.
// s and e are f32 throughout; only out, dx and dg are rounded.
#include "gdn_linrec.cuh"
#include "gdn_vec.cuh"
#include "tc_ptx.cuh"
#include "tma_host.cuh"

namespace gdn {
namespace {

using vec::Pack;

constexpr int kSeg = 8;                     // rows of a warp in a round
constexpr int kRecWarps = kRecTile / kSeg;  // 8
constexpr int kRecThreads = 32 * kRecWarps;
constexpr int kMaxCluster = 8;
constexpr float kReset = -1.f;  // in the place of a product of decays (never negative)

static_assert(kRecThreads == 2 * kHeadDim, "two threads a channel between the barriers");

// (a, b) followed by (a2, b2)
__device__ __forceinline__ void compose(float &a, float &b, float a2, float b2) {
    if (a2 < 0.f) {
        a = kReset;
        b = b2;
    } else {
        b = fmaf(a2, b, b2);
        a = a < 0.f ? kReset : a * a2;
    }
}

__device__ __forceinline__ float apply(float a, float b, float s) { return a < 0.f ? b : fmaf(a, s, b); }

// The sequences' boundaries on the token axis.
struct Bounds {
    const int32_t *cu;
    int n, seqlen, total;
    int next;  // packed: first offset not below the last segment asked for (monotone use)

    __device__ __forceinline__ int start(int i) const { return cu ? cu[i] : i * seqlen; }

    // bit i (0 .. kSeg): a sequence ends before, or starts at, row t0 + i.
    // Called by whole warps; packed: the offsets are searched 32 at a time on
    // from the last call's place (forward: t0 rises from call to call;
    // backward: t0 falls).
    template <bool FORWARD>
    __device__ __forceinline__ uint32_t mask(int t0) {
        uint32_t m = 0;
        if (!cu) {
            for (int b = (t0 + seqlen - 1) / seqlen * seqlen; b <= t0 + kSeg && b <= total; b += seqlen)
                m |= 1u << (b - t0);
            return m;
        }
        const int lane = threadIdx.x & 31;
        if (FORWARD) {
            for (;;) {
                const int v = next + lane <= n ? cu[next + lane] : INT_MAX;
                const uint32_t below = __ballot_sync(0xffffffffu, v < t0);
                next += __popc(below);
                if (below != 0xffffffffu) break;
            }
        } else {
            for (;;) {  // next: an offset index from which on all are >= t0 of the last call
                const int v = next - 1 - lane >= 0 ? cu[next - 1 - lane] : INT_MIN;
                const uint32_t above = __ballot_sync(0xffffffffu, v >= t0);
                next -= __popc(above);
                if (above != 0xffffffffu) break;
            }
        }
        for (int k = next;; k += 32) {
            const int v = k + lane <= n ? cu[k + lane] : INT_MAX;
            const bool in = v <= t0 + kSeg;
            m |= __reduce_or_sync(0xffffffffu, in ? 1u << (v - t0) : 0u);
            if (__ballot_sync(0xffffffffu, in) != 0xffffffffu) return m;
        }
    }

    // the sequence that starts at row t (some sequence with rows does)
    __device__ __forceinline__ int starting(int t) const {
        if (!cu) return t / seqlen;
        int lo = 0, hi = n - 1;  // the last i with cu[i] <= t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (cu[mid] <= t) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    }

    // the sequence whose last row is t
    __device__ __forceinline__ int ending(int t) const {
        if (!cu) return t / seqlen;
        int lo = 1, hi = n;  // the first i with cu[i] > t
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] > t) hi = mid;
            else lo = mid + 1;
        }
        return lo - 1;
    }
};

// Offsets start at 0, do not fall and end at the last row; the same answer in
// every CTA. A bad one is recorded.
__device__ __forceinline__ bool offsets_ok(const RecArgs &a) {
    if (!a.cu) return true;
    int bad = 0;
    for (int i = threadIdx.x; i < a.num_seqs; i += blockDim.x) bad |= a.cu[i] > a.cu[i + 1];
    if (a.cu[0] != 0 || a.cu[a.num_seqs] != a.total_tokens) bad = 1;
    if (!__syncthreads_or(bad)) return true;
    if (threadIdx.x == 0) record_status(a.status, GDN_EDEVICE_INPUT);
    return false;
}

// Sequences without rows: `to` gets `from` (null: zeros). One cluster per head.
__device__ __forceinline__ void copy_empty(const RecArgs &a, const Bounds &bd, const float *from, float *to, int h,
                                           int rank, int ctas) {
    if (!to) return;
    const int c = (threadIdx.x & 31) * 4;
    for (int i = rank * kRecWarps + (threadIdx.x >> 5); i < a.num_seqs; i += ctas * kRecWarps) {
        if (bd.start(i) != bd.start(i + 1)) continue;
        const long long o = ((long long)i * a.hv + h) * kHeadDim + c;
        *reinterpret_cast<float4 *>(to + o) =
            from ? *reinterpret_cast<const float4 *>(from + o) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}

__device__ __forceinline__ void load4(float (&v)[4], const float *p) {
    const float4 t = *reinterpret_cast<const float4 *>(p);
    v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
}
__device__ __forceinline__ void store4(float *p, const float (&v)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// Shared memory between the barriers of a round.
struct Exchange {
    float seg_a[kRecWarps][kHeadDim], seg_b[kRecWarps][kHeadDim];  // segments; seg_b then the state at each
    float cta[2][kMaxCluster][2][kHeadDim];  // by round parity: every CTA's composed segments (a, b)
};

// Steps 2 and 3 for two threads a channel: composes this CTA's segments, hands
// them to the cluster and, with everyone's, moves `carry` (the value before
// the round) on to the next round's. seg_b becomes the value that each
// segment starts from; returns the one that the CTA's first segment starts
// from. REVERSE: segments and CTAs from the last to the first.
template <bool REVERSE>
__device__ __forceinline__ float exchange(Exchange &ex, float &carry, int parity, int rank, int ctas) {
    using namespace tc;
    const int c = threadIdx.x % kHeadDim, half = threadIdx.x / kHeadDim;
    {
        const int w0 = REVERSE ? kRecWarps - 1 : 0;
        float a = ex.seg_a[w0][c], b = ex.seg_b[w0][c];
#pragma unroll
        for (int i = 1; i < kRecWarps; ++i) {
            const int w = REVERSE ? kRecWarps - 1 - i : i;
            compose(a, b, ex.seg_a[w][c], ex.seg_b[w][c]);
        }
        float *slot = &ex.cta[parity][rank][half][c];
        const float v = half ? b : a;
        if (ctas == 1) {
            *slot = v;
        } else {
            for (int r = 0; r < ctas; ++r) cluster_st(cluster_map(slot, r), v);
        }
    }
    if (ctas == 1) __syncthreads();
    else cluster_sync();
    float in = carry, s = carry;
    for (int i = 0; i < ctas; ++i) {
        const int r = REVERSE ? ctas - 1 - i : i;
        if (r == rank) in = s;
        s = apply(ex.cta[parity][r][0][c], ex.cta[parity][r][1][c], s);
    }
    carry = s;
    if (half == 0) {
        s = in;
#pragma unroll
        for (int i = 0; i < kRecWarps; ++i) {
            const int w = REVERSE ? kRecWarps - 1 - i : i;
            const float b = ex.seg_b[w][c];
            ex.seg_b[w][c] = s;
            s = apply(ex.seg_a[w][c], b, s);
        }
    }
    return in;
}

// Bytes of one stage: the tiles of x (and dout) and, with gates per channel, of g.
template <typename T, bool CHANNEL, bool BACKWARD>
constexpr uint32_t stage_bytes() {
    return uint32_t(kRecTile * kHeadDim * sizeof(T)) * (1 + CHANNEL + BACKWARD);
}
template <bool BACKWARD>
constexpr int stages() { return BACKWARD ? 1 : 2; }

// Tile loads through a ring of stages: one thread issues, everyone waits.
template <typename T, bool CHANNEL, bool BACKWARD>
struct Ring {
    static constexpr int kStages = stages<BACKWARD>();
    static constexpr uint32_t kTile = kRecTile * kHeadDim * sizeof(T);
    uint8_t *base;
    uint64_t *full;
    bool dead;  // a wait ran out: later ones are skipped

    __device__ __forceinline__ const T *x(int i) const {
        return reinterpret_cast<const T *>(base + (i % kStages) * stage_bytes<T, CHANNEL, BACKWARD>());
    }
    __device__ __forceinline__ const T *g(int i) const { return x(i) + kRecTile * kHeadDim; }
    __device__ __forceinline__ const T *dout(int i) const { return x(i) + (1 + CHANNEL) * kRecTile * kHeadDim; }

    // by one thread: tile i of this CTA's walk, rows from t0 of head h
    __device__ __forceinline__ void load(int i, const CUtensorMap *mx, const CUtensorMap *mg, const CUtensorMap *md,
                                         int h, int t0) {
        uint64_t *bar = &full[i % kStages];
        tc::mbar_arrive_expect_tx(bar, stage_bytes<T, CHANNEL, BACKWARD>());
        tc::tma_load_3d(const_cast<T *>(x(i)), mx, 0, h, t0, bar);
        if (CHANNEL) tc::tma_load_3d(const_cast<T *>(g(i)), mg, 0, h, t0, bar);
        if (BACKWARD) tc::tma_load_3d(const_cast<T *>(dout(i)), md, 0, h, t0, bar);
    }
    __device__ __forceinline__ void wait(int i, unsigned long long limit) {
        if (!dead && !tc::mbar_wait(&full[i % kStages], uint32_t((i / kStages) & 1), limit)) dead = true;
    }
};

// Gate per head of row t0 + lane (lanes 0 .. kSeg - 1; 0, which passes the
// state on, past the end). Loaded a round ahead of its use.
__device__ __forceinline__ float head_gate(const RecArgs &a, int t0, int h) {
    const int lane = threadIdx.x & 31;
    return lane < kSeg && t0 + lane < a.total_tokens ? static_cast<const float *>(a.g)[(long long)(t0 + lane) * a.hv + h]
                                                     : 0.f;
}

// Decays of a segment's rows, from the tile of gates per channel or from head_gate's value.
template <typename T, bool CHANNEL>
__device__ __forceinline__ void decays(float (&a)[kSeg][4], const T *g_tile, float g_head) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float v = CHANNEL ? 0.f : expf(g_head);
#pragma unroll
    for (int i = 0; i < kSeg; ++i) {
        if (CHANNEL) {
            Pack<T, 4> p;
            p.load(g_tile + (w * kSeg + i) * kHeadDim + lane * 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) a[i][j] = expf(p.f(j));
        } else {
            a[i][0] = a[i][1] = a[i][2] = a[i][3] = __shfl_sync(0xffffffffu, v, i);
        }
    }
}

template <typename T, bool CHANNEL>
__global__ void __launch_bounds__(kRecThreads)
k_linrec(const RecArgs a, const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mg, int ctas) {
    using namespace tc;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Exchange ex;
    __shared__ uint64_t full[stages<false>()];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane * 4;
    const int rank = ctas == 1 ? 0 : int(cluster_ctarank()), h = int(blockIdx.x) / ctas;
    if (!offsets_ok(a)) return;  // the same in every CTA
    Bounds bd{a.cu, a.num_seqs, a.dense_seqlen, a.total_tokens, 0};
    copy_empty(a, bd, a.s0, a.final_state, h, rank, ctas);
    const int tiles = (a.total_tokens + kRecTile - 1) / kRecTile;
    const int rounds = (tiles + ctas - 1) / ctas;
    if (!rounds) return;
    Ring<T, CHANNEL, false> ring{reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem) + 127) & ~uintptr_t(127)),
                                 full, false};
    if (threadIdx.x == 0) {
        for (int i = 0; i < ring.kStages; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
        for (int i = 0; i < ring.kStages && i < rounds; ++i)
            ring.load(i, &mx, &mg, nullptr, h, (i * ctas + rank) * kRecTile);
    }
    __syncthreads();
    if (ctas > 1) cluster_sync();  // every CTA of the cluster runs before its shared memory is written
    float carry = 0.f;  // of channel threadIdx.x % 128, before the round
    float gate = CHANNEL ? 0.f : head_gate(a, rank * kRecTile + w * kSeg, h);
    for (int round = 0; round < rounds; ++round) {
        const int tile = round * ctas + rank, t0 = tile * kRecTile + w * kSeg;
        const uint32_t starts = t0 < a.total_tokens ? bd.mask<true>(t0) : 0u;  // bit kSeg: before the next segment
        ring.wait(round, a.wait_ns);
        float d[kSeg][4];
        Pack<T, 4> x[kSeg];
        decays<T, CHANNEL>(d, ring.g(round), gate);
        if (!CHANNEL) gate = head_gate(a, t0 + ctas * kRecTile, h);
        const T *xt = ring.x(round) + w * kSeg * kHeadDim + c;
        float A[4] = {1.f, 1.f, 1.f, 1.f}, B[4] = {0.f, 0.f, 0.f, 0.f};
        bool reset = false;
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
            x[i].load(xt + i * kHeadDim);
            if ((starts >> i & 1) && t0 + i < a.total_tokens) {
                reset = true;
                if (a.s0)
                    load4(B, a.s0 + ((long long)bd.starting(t0 + i) * a.hv + h) * kHeadDim + c);
                else
                    B[0] = B[1] = B[2] = B[3] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                B[j] = fmaf(d[i][j], B[j], x[i].f(j));
                A[j] *= d[i][j];
            }
        }
        if (reset) A[0] = A[1] = A[2] = A[3] = kReset;
        store4(&ex.seg_a[w][c], A);
        store4(&ex.seg_b[w][c], B);
        __syncthreads();
        // the tile is in registers: its stage takes a later one
        if (threadIdx.x == 0 && round + ring.kStages < rounds)
            ring.load(round + ring.kStages, &mx, &mg, nullptr, h, (tile + ring.kStages * ctas) * kRecTile);
        const float in = exchange<false>(ex, carry, round & 1, rank, ctas);
        if (a.states && tile < tiles && threadIdx.x < kHeadDim)
            a.states[((long long)tile * a.hv + h) * kHeadDim + threadIdx.x] = in;
        __syncthreads();
        float s[4];
        load4(s, &ex.seg_b[w][c]);
        T *out = static_cast<T *>(a.out) + ((long long)t0 * a.hv + h) * kHeadDim + c;
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
            if (t0 + i >= a.total_tokens) break;
            if (starts >> i & 1) {
                if (a.s0)
                    load4(s, a.s0 + ((long long)bd.starting(t0 + i) * a.hv + h) * kHeadDim + c);
                else
                    s[0] = s[1] = s[2] = s[3] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[j] = fmaf(d[i][j], s[j], x[i].f(j));
                x[i].set(j, s[j]);
            }
            x[i].store(out + (long long)i * a.hv * kHeadDim);
            if (a.final_state && (starts >> (i + 1) & 1))
                store4(a.final_state + ((long long)bd.ending(t0 + i) * a.hv + h) * kHeadDim + c, s);
        }
    }
    if (ring.dead && lane == 0) record_status(a.status, GDN_ETIMEOUT);
}

template <typename T, bool CHANNEL>
__global__ void __launch_bounds__(kRecThreads)
k_linrec_bwd(const RecArgs a, const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mg,
             const __grid_constant__ CUtensorMap md, int ctas) {
    using namespace tc;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Exchange ex;
    __shared__ float fwd_a[kRecWarps][kHeadDim], fwd_b[kRecWarps][kHeadDim];
    __shared__ uint64_t full[stages<true>()];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane * 4;
    const int rank = ctas == 1 ? 0 : int(cluster_ctarank()), h = int(blockIdx.x) / ctas;
    if (!offsets_ok(a)) return;
    Bounds bd{a.cu, a.num_seqs, a.dense_seqlen, a.total_tokens, a.num_seqs + 1};
    copy_empty(a, bd, a.dfinal, a.dinitial, h, rank, ctas);
    const int tiles = (a.total_tokens + kRecTile - 1) / kRecTile;
    const int rounds = (tiles + ctas - 1) / ctas;
    if (!rounds) return;
    Ring<T, CHANNEL, true> ring{reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem) + 127) & ~uintptr_t(127)),
                                full, false};
    if (threadIdx.x == 0) {
        for (int i = 0; i < ring.kStages; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
        for (int i = 0; i < ring.kStages && i < rounds; ++i)
            ring.load(i, &mx, &mg, &md, h, ((rounds - 1 - i) * ctas + rank) * kRecTile);
    }
    __syncthreads();
    if (ctas > 1) cluster_sync();
    float carry = 0.f;
    float gate = CHANNEL ? 0.f : head_gate(a, ((rounds - 1) * ctas + rank) * kRecTile + w * kSeg, h);
    for (int round = 0; round < rounds; ++round) {
        const int tile = (rounds - 1 - round) * ctas + rank, t0 = tile * kRecTile + w * kSeg;
        const uint32_t bounds = t0 < a.total_tokens ? bd.mask<false>(t0) : 0u;
        // the state before the tile, of this thread's channel (unused where the tile starts a sequence)
        float state = 0.f;
        if (threadIdx.x >= kHeadDim && tile < tiles)
            state = a.states[((long long)tile * a.hv + h) * kHeadDim + threadIdx.x - kHeadDim];
        ring.wait(round, a.wait_ns);
        float d[kSeg][4];
        Pack<T, 4> x[kSeg], dy[kSeg];
        decays<T, CHANNEL>(d, ring.g(round), gate);
        if (!CHANNEL && round + 1 < rounds) gate = head_gate(a, t0 - ctas * kRecTile, h);
        const T *xt = ring.x(round) + w * kSeg * kHeadDim + c, *yt = ring.dout(round) + w * kSeg * kHeadDim + c;
        // the rows' maps: forward for s, in reverse for e
        {
            float A[4] = {1.f, 1.f, 1.f, 1.f}, B[4] = {0.f, 0.f, 0.f, 0.f};
            bool reset = false;
#pragma unroll
            for (int i = 0; i < kSeg; ++i) {
                x[i].load(xt + i * kHeadDim);
                dy[i].load(yt + i * kHeadDim);
                if ((bounds >> i & 1) && t0 + i < a.total_tokens) {
                    reset = true;
                    if (a.s0)
                        load4(B, a.s0 + ((long long)bd.starting(t0 + i) * a.hv + h) * kHeadDim + c);
                    else
                        B[0] = B[1] = B[2] = B[3] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    B[j] = fmaf(d[i][j], B[j], x[i].f(j));
                    A[j] *= d[i][j];
                }
            }
            float R[4] = {A[0], A[1], A[2], A[3]};
            if (reset) A[0] = A[1] = A[2] = A[3] = kReset;
            store4(&fwd_a[w][c], A);
            store4(&fwd_b[w][c], B);
            float E[4] = {0.f, 0.f, 0.f, 0.f};
            reset = false;
#pragma unroll
            for (int i = kSeg - 1; i >= 0; --i) {
                if (bounds >> (i + 1) & 1) {
                    reset = true;
                    if (a.dfinal && t0 + i < a.total_tokens)
                        load4(E, a.dfinal + ((long long)bd.ending(t0 + i) * a.hv + h) * kHeadDim + c);
                    else
                        E[0] = E[1] = E[2] = E[3] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) E[j] = d[i][j] * (dy[i].f(j) + E[j]);
            }
            if (reset) R[0] = R[1] = R[2] = R[3] = kReset;
            store4(&ex.seg_a[w][c], R);
            store4(&ex.seg_b[w][c], E);
        }
        __syncthreads();
        if (threadIdx.x == 0 && round + ring.kStages < rounds)
            ring.load(round + ring.kStages, &mx, &mg, &md, h, (tile - ring.kStages * ctas) * kRecTile);
        exchange<true>(ex, carry, round & 1, rank, ctas);
        if (threadIdx.x >= kHeadDim) {  // the other half of the threads: the state at every segment
            const int ch = threadIdx.x - kHeadDim;
#pragma unroll
            for (int i = 0; i < kRecWarps; ++i) {
                const float b = fwd_b[i][ch];
                fwd_b[i][ch] = state;
                state = apply(fwd_a[i][ch], b, state);
            }
        }
        __syncthreads();
        float before[kSeg][4], s[4];
        load4(s, &fwd_b[w][c]);
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
            if ((bounds >> i & 1) && t0 + i < a.total_tokens) {
                if (a.s0)
                    load4(s, a.s0 + ((long long)bd.starting(t0 + i) * a.hv + h) * kHeadDim + c);
                else
                    s[0] = s[1] = s[2] = s[3] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                before[i][j] = s[j];
                s[j] = fmaf(d[i][j], s[j], x[i].f(j));
            }
        }
        float e[4], sums[kSeg];
        load4(e, &ex.seg_b[w][c]);
        const long long row0 = ((long long)t0 * a.hv + h) * kHeadDim + c;
#pragma unroll
        for (int i = kSeg - 1; i >= 0; --i) {
            const bool live = t0 + i < a.total_tokens;
            if (bounds >> (i + 1) & 1) {
                if (a.dfinal && live)
                    load4(e, a.dfinal + ((long long)bd.ending(t0 + i) * a.hv + h) * kHeadDim + c);
                else
                    e[0] = e[1] = e[2] = e[3] = 0.f;
            }
            sums[i] = 0.f;
            Pack<T, 4> q;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float ds = dy[i].f(j) + e[j];
                dy[i].set(j, ds);
                e[j] = d[i][j] * ds;
                const float dg = e[j] * before[i][j];
                if (CHANNEL) q.set(j, dg);
                else sums[i] += dg;
            }
            if (live) {
                const long long row = row0 + (long long)i * a.hv * kHeadDim;
                dy[i].store(static_cast<T *>(a.dx) + row);
                if (CHANNEL) q.store(static_cast<T *>(a.dg) + row);
                if (a.dinitial && (bounds >> i & 1))
                    store4(a.dinitial + ((long long)bd.starting(t0 + i) * a.hv + h) * kHeadDim + c, e);
            }
        }
        if (!CHANNEL) {
            // eight rows' sums over the head's channels: lanes halve the rows they add, lane 4 r ends with row r
#pragma unroll
            for (int m = 16, k = kSeg / 2; k; m >>= 1, k >>= 1) {
                const bool up = lane & m;
#pragma unroll
                for (int i = 0; i < k; ++i) {
                    const float send = up ? sums[i] : sums[i + k], keep = up ? sums[i + k] : sums[i];
                    sums[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
                }
            }
            sums[0] += __shfl_xor_sync(0xffffffffu, sums[0], 2);
            sums[0] += __shfl_xor_sync(0xffffffffu, sums[0], 1);
            const int r = lane >> 2;
            if ((lane & 3) == 0 && t0 + r < a.total_tokens)
                static_cast<float *>(a.dg)[(long long)(t0 + r) * a.hv + h] = sums[0];
        }
    }
    if (ring.dead && lane == 0) record_status(a.status, GDN_ETIMEOUT);
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

// CTAs of a cluster: as many as there are tiles, at most the portable eight
int cluster_of(int total) {
    const int tiles = (total + kRecTile - 1) / kRecTile;
    int c = 1;
    while (c < kMaxCluster && c < tiles) c *= 2;
    return c;
}

// launches `fn` with one cluster of `ctas` CTAs a head
template <typename... P, typename... A>
cudaError_t launch_clusters(void (*fn)(P...), int hv, int ctas, size_t smem, cudaStream_t s, const A &...args) {
    cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(fn),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(hv) * unsigned(ctas));
    cfg.blockDim = dim3(kRecThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = unsigned(ctas);
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, P(args)...);
}

template <typename T, bool CHANNEL>
cudaError_t forward(const RecArgs &a, cudaStream_t s) {
    CUtensorMap mx = {}, mg = {};
    if (a.total_tokens > 0) {
        const bool f32 = sizeof(T) == 4;
        if (!make_tmap_head_rows(&mx, a.x, f32, a.hv, a.total_tokens, kRecTile)) return cudaErrorInvalidValue;
        if (CHANNEL && !make_tmap_head_rows(&mg, a.g, f32, a.hv, a.total_tokens, kRecTile))
            return cudaErrorInvalidValue;
    }
    const size_t smem = stages<false>() * size_t(stage_bytes<T, CHANNEL, false>()) + 128;
    const int ctas = cluster_of(a.total_tokens);
    LaunchScope scope(GDN_K_LINREC, s);
    return launch_clusters(k_linrec<T, CHANNEL>, a.hv, ctas, smem, s, a, mx, mg, ctas);
}

template <typename T, bool CHANNEL>
cudaError_t backward(const RecArgs &a, cudaStream_t s) {
    CUtensorMap mx = {}, mg = {}, md = {};
    if (a.total_tokens > 0) {
        const bool f32 = sizeof(T) == 4;
        if (!make_tmap_head_rows(&mx, a.x, f32, a.hv, a.total_tokens, kRecTile) ||
            !make_tmap_head_rows(&md, a.dout, f32, a.hv, a.total_tokens, kRecTile))
            return cudaErrorInvalidValue;
        if (CHANNEL && !make_tmap_head_rows(&mg, a.g, f32, a.hv, a.total_tokens, kRecTile))
            return cudaErrorInvalidValue;
    }
    const size_t smem = stages<true>() * size_t(stage_bytes<T, CHANNEL, true>()) + 128;
    const int ctas = cluster_of(a.total_tokens);
    LaunchScope scope(GDN_K_LINREC_BWD, s);
    return launch_clusters(k_linrec_bwd<T, CHANNEL>, a.hv, ctas, smem, s, a, mx, mg, md, ctas);
}

}  // namespace

cudaError_t launch_linrec(const RecArgs &a, int io_dtype, bool channel, cudaStream_t s) {
    if (io_dtype == GDN_DT_BF16) return channel ? forward<__nv_bfloat16, true>(a, s) : forward<__nv_bfloat16, false>(a, s);
    return channel ? forward<float, true>(a, s) : forward<float, false>(a, s);
}

cudaError_t launch_linrec_bwd(const RecArgs &a, int io_dtype, bool channel, cudaStream_t s) {
    if (io_dtype == GDN_DT_BF16)
        return channel ? backward<__nv_bfloat16, true>(a, s) : backward<__nv_bfloat16, false>(a, s);
    return channel ? backward<float, true>(a, s) : backward<float, false>(a, s);
}

cudaError_t launch_linrec_step(const void *x, const void *g, float *state, const int32_t *idx, void *out, int seqs,
                               int hv, int slots, int io_dtype, bool channel, int *status, cudaStream_t s) {
    if (seqs == 0) return cudaSuccess;
    const int rows = seqs * hv;
    const unsigned grid = unsigned((rows + kStepWarps - 1) / kStepWarps);
    constexpr int kThreads = 32 * kStepWarps;
    LaunchScope scope(GDN_K_LINREC_STEP, s);
    if (io_dtype == GDN_DT_BF16) {
        if (channel)
            k_linrec_step<__nv_bfloat16, true><<<grid, kThreads, 0, s>>>(x, g, state, idx, out, rows, hv, slots, status);
        else
            k_linrec_step<__nv_bfloat16, false><<<grid, kThreads, 0, s>>>(x, g, state, idx, out, rows, hv, slots, status);
    } else {
        if (channel)
            k_linrec_step<float, true><<<grid, kThreads, 0, s>>>(x, g, state, idx, out, rows, hv, slots, status);
        else
            k_linrec_step<float, false><<<grid, kThreads, 0, s>>>(x, g, state, idx, out, rows, hv, slots, status);
    }
    return cudaGetLastError();
}

}  // namespace gdn
