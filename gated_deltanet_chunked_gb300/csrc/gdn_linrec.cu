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
// of CTAs takes half of a head's channels and walks the packed token axis in
// rounds; in a round each CTA takes the next tile of 128 rows, each of its warps
// a segment of 16 rows, each lane two channels:
//  1. every warp composes its segment's rows (tile in shared memory by TMA,
//     kept in registers from here on);
//  2. the CTA composes its segments and stores the result into every CTA of
//     the cluster (distributed shared memory, asynchronous stores that count
//     on the receiver's mbarrier);
//  3. when all have arrived, every CTA knows the state at its tile's first row
//     and, all in the same order, the state that the next round starts from;
//  4. every warp walks its segment again from its state and writes its rows.
// So a round costs one exchange inside the cluster instead of a chain of
// flags through global memory, needs no workspace, and adds in a fixed order:
// the same call gives the same bits. While a round runs, the next tiles are on
// their way. (A cluster barrier in the place of the counted stores has to be a
// release, and then waits for the rows written in the round before.)
// A round takes about 2 us, whatever it carries: walk over the tile 1050
// cycles, the exchange 1200 to 2000 (clusters of 4 to 16), second walk and
// stores 570, and the wait for the tile 240. Long axes with gates per channel
// fill the memory pipe all the same (two CTAs an SM); gates per head carry
// fewer bytes a round and do not.
// Measured, bf16, 32 heads, of the copy rate (6783 GB/s) by a call's own bytes:
// gates per channel, T = 65536: forward 260 us (0.91), backward 443 (0.90);
// T = 4096: 25 (0.60), 37 (0.67); gates per head, 38429 packed rows: 136
// (0.69), 264 (0.53). f32, 16 heads x 8000, per channel: 37 (0.79), 58 (0.83).
// Few heads on a long axis leave SMs idle (launch_clusters): 4 heads x 65536
// per channel 82 (0.36), 117 (0.42), per head 67 (0.30), 169 (0.18).
//
// Sequences are boundaries on the one axis. A segment that holds a sequence's
// first row (for the backward pass: last row) does not depend on what comes
// before: that is marked in A (kReset) instead of multiplying by zero, so that
// an infinity or NaN of one sequence cannot reach the next.
//
// The backward pass walks the rounds from the last to the first with e in the
// place of s. It needs s_{t-1} too: the forward pass left the state before
// every tile in `states`, from which each CTA recomputes its tile's states by
// the same steps without any exchange. With gates per head dg is a sum over
// the head, so there a CTA takes all 128 channels of tiles of 64 rows.
// s and e are f32 throughout; only out, dx and dg are rounded.
#include <atomic>
#include <type_traits>

#include "gdn_linrec.cuh"
#include "gdn_vec.cuh"
#include "tc_ptx.cuh"
#include "tma_host.cuh"

namespace gdn {
namespace {

using vec::Pack;

constexpr int kRecWarps = 8;
constexpr int kRecThreads = 32 * kRecWarps;
constexpr int kPart = 8;  // rows whose states the backward pass holds at a time
constexpr int kMaxCluster = 16;  // above the portable eight
constexpr float kReset = -1.f;  // in the place of a product of decays (never negative)

// A CTA's tile: 64 channels x 8 segments of 16 rows, or (WIDE) 128 x 4. A
// warp has 64 channels, two a lane, of one segment.
template <bool WIDE>
struct Tile {
    static constexpr int kSeg = 16;
    static constexpr int kCh = WIDE ? 128 : 64;
    static constexpr int kSegs = WIDE ? 4 : 8;
    static constexpr int kRows = kSegs * kSeg;
    static constexpr int kParts = kHeadDim / kCh;  // clusters of a head
    static_assert(kRows % kStateRows == 0 && kStateRows % kSeg == 0 && kSeg % kPart == 0, "");

    static __device__ __forceinline__ int seg() { return (threadIdx.x >> 5) % kSegs; }
    // the lane's first channel in the tile
    static __device__ __forceinline__ int channel() { return (threadIdx.x >> 5) / kSegs * 64 + (threadIdx.x & 31) * 2; }
};

using vec::both;
using vec::fma2;
using vec::mul2;

// (a, b) followed by (a2, b2)
__device__ __forceinline__ void compose(float &a, float &b, float a2, float b2) {
    const float nb = fmaf(a2, b, b2), na = a * a2;
    b = a2 < 0.f ? b2 : nb;
    a = a < 0.f || a2 < 0.f ? kReset : na;
}

__device__ __forceinline__ float apply(float a, float b, float s) { return a < 0.f ? b : fmaf(a, s, b); }

// Where sequences start and end in a tile, for all of its warps: bit i of
// starts[k] (ends[k]) says that row i of segment k is a sequence's first
// (last), `first` (`last`) at that row which sequence it is.
template <typename S>
struct Marks {
    uint32_t starts[S::kSegs], ends[S::kSegs];
    int first[S::kRows], last[S::kRows];
};

// The sequences' boundaries on the token axis.
struct Bounds {
    const int32_t *cu;
    int n, seqlen, total;

    __device__ __forceinline__ int start(int i) const { return cu ? cu[i] : i * seqlen; }

    // Where the last mark() left off.
    struct Cursor {
        int next;    // the offsets before it are below that tile's first row, the others not
        int offset;  // FORWARD: the first not below that tile's end; else: the last not above its first row
    };
    // FORWARD: t0 rises from call to call; else it falls
    template <bool FORWARD>
    __device__ __forceinline__ Cursor begin() const { return FORWARD ? Cursor{0, 0} : Cursor{n + 1, INT_MAX}; }

    // Marks the tile from row t0, by one warp. Packed: the offsets are searched
    // 32 at a time from the cursor on, unless its offset says that there is
    // none in this tile (the reads depend on each other, and the CTA waits for
    // them). Sequences without rows share an offset with their neighbours and
    // are left out.
    template <bool FORWARD, typename S>
    __device__ __forceinline__ void mark(int t0, Cursor &cursor, Marks<S> &m) const {
        const int lane = threadIdx.x & 31, end = min(t0 + S::kRows, total);
        if (lane < S::kSegs) m.starts[lane] = m.ends[lane] = 0;
        __syncwarp();
        if (t0 < 0 || t0 >= total) return;  // seqlen is not 0 where there are rows
        auto start_at = [&](int r, int seq) {
            if (r >= S::kRows || t0 + r >= total) return;
            atomicOr(&m.starts[r / S::kSeg], 1u << (r % S::kSeg));
            m.first[r] = seq;
        };
        auto end_at = [&](int r, int seq) {
            if (r < 0) return;
            atomicOr(&m.ends[r / S::kSeg], 1u << (r % S::kSeg));
            m.last[r] = seq;
        };
        if (!cu) {
            for (long long k = ((long long)t0 + seqlen - 1) / seqlen + lane; k * seqlen <= end; k += 32) {
                const int r = int(k * seqlen) - t0;
                start_at(r, int(k));
                end_at(r - 1, int(k) - 1);
            }
            return;
        }
        if (FORWARD ? cursor.offset > end : cursor.offset < t0) return;
        int &next = cursor.next;
        uint32_t moved;
        do {  // next becomes the first offset that is not below t0
            if (FORWARD) {
                moved = __ballot_sync(0xffffffffu, next + lane <= n && cu[next + lane] < t0);
                next += __popc(moved);
            } else {
                moved = __ballot_sync(0xffffffffu, next - 1 - lane >= 0 && cu[next - 1 - lane] >= t0);
                next -= __popc(moved);
            }
        } while (moved == 0xffffffffu);
        if (FORWARD) cursor.offset = -1;
        uint32_t in = 0xffffffffu;
        for (int k = next + lane; in == 0xffffffffu; k += 32) {
            const int v = k <= n ? cu[k] : INT_MAX;
            in = __ballot_sync(0xffffffffu, v <= end);
            if (FORWARD && cursor.offset < 0) {
                const int below = __popc(__ballot_sync(0xffffffffu, v < end));  // offsets rise
                if (below < 32) cursor.offset = __shfl_sync(0xffffffffu, v, below);
            }
            if (v > end) continue;
            if (k < n && cu[k + 1] != v) start_at(v - t0, k);    // the last sequence of those that start here
            if (k > 0 && cu[k - 1] != v) end_at(v - t0 - 1, k - 1);  // the first of those that end here
        }
        if (!FORWARD) cursor.offset = next <= n && cu[next] == t0 ? t0 : cu[next - 1];  // the first offset is 0
    }
};

// A lane's two channels of sequence `seq` in per-sequence states [num_seqs, hv, 128] (null: zeros).
__device__ __forceinline__ float2 state_of(const float *from, int seq, int width, int hc) {
    return from ? *reinterpret_cast<const float2 *>(from + (long long)seq * width + hc) : make_float2(0.f, 0.f);
}
__device__ __forceinline__ void set_state(float *to, int seq, int width, int hc, float2 v) {
    *reinterpret_cast<float2 *>(to + (long long)seq * width + hc) = v;
}

__device__ __forceinline__ float2 &pair(float *p) { return *reinterpret_cast<float2 *>(p); }

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

// Sequences without rows: `to` gets `from` (null: zeros).
template <typename S>
__device__ __forceinline__ void copy_empty(const RecArgs &a, const Bounds &bd, const float *from, float *to, int hc,
                                           int rank, int ctas) {
    if (!to) return;
    for (int i = rank * S::kSegs + S::seg(); i < a.num_seqs; i += ctas * S::kSegs) {
        if (bd.start(i) != bd.start(i + 1)) continue;
        const long long o = (long long)i * a.hv * kHeadDim + hc;
        *reinterpret_cast<float2 *>(to + o) =
            from ? *reinterpret_cast<const float2 *>(from + o) : make_float2(0.f, 0.f);
    }
}

// Shared memory of a round's exchange.
template <typename S>
struct Exchange {
    float seg_a[S::kSegs][S::kCh], seg_b[S::kSegs][S::kCh];  // segments; seg_b then the state at each
    float2 cta[2][kMaxCluster][S::kCh];  // by round parity: every CTA's composed segments (a, b)
    uint64_t bar[2];
    Marks<S> marks[2];          // by round parity
    // of gates per head, by round parity: every row's decay, twice (for packed
    // arithmetic), and their product in parts of kPart rows
    float2 decays[2][S::kRows];
    float2 products[2][S::kRows / kPart];
    tc::GiveUp<kMaxCluster> gave_up;
    int stop;  // set where a wait of the exchange has run out
};

// A channel's segments of a tile in walking order.
template <typename S, bool REVERSE>
struct Segments {
    float a[S::kSegs], b[S::kSegs];

    static __device__ __forceinline__ int seg(int i) { return REVERSE ? S::kSegs - 1 - i : i; }
    __device__ __forceinline__ Segments(const float (*sa)[S::kCh], const float (*sb)[S::kCh], int ch) {
#pragma unroll
        for (int i = 0; i < S::kSegs; ++i) a[i] = sa[seg(i)][ch], b[i] = sb[seg(i)][ch];
    }
    __device__ __forceinline__ float2 composed() const {
        float ca = a[0], cb = b[0];
#pragma unroll
        for (int i = 1; i < S::kSegs; ++i) compose(ca, cb, a[i], b[i]);
        return make_float2(ca, cb);
    }
    // writes the value that each segment starts from, `s` at the first, and
    // calls at(segment, value) for each
    template <typename F>
    __device__ __forceinline__ void finish(float (*sb)[S::kCh], int ch, float s, F at) {
#pragma unroll
        for (int i = 0; i < S::kSegs; ++i) {
            sb[seg(i)][ch] = s;
            at(seg(i), s);
            s = apply(a[i], b[i], s);
        }
    }
};

// Steps 2 and 3, the first kCh threads, one a channel, after the segments are
// in shared memory: moves `carry` (the value before the round) on to the next
// round's; seg_b becomes the value that each segment starts from, which
// at(segment, value) gets too. REVERSE: segments and CTAs from the last to the
// first. When the wait runs out the round is finished on what is there and the
// CTA leaves after it: all of its threads see `stop` alike, which is set between
// the round's two barriers and read behind the second. One
// thread a channel is the fewest instructions; the other warps have the
// forward states of the backward pass, the next tiles' boundaries and gates
// to see to meanwhile.
template <bool REVERSE, typename S, typename F>
__device__ __forceinline__ void exchange(Exchange<S> &ex, float &carry, int round, int rank, int ctas,
                                         unsigned long long wait_ns, bool &ok, F at) {
    using namespace tc;
    const int ch = threadIdx.x, p = round & 1;
    if (threadIdx.x == 0) mbar_arrive_expect_tx(&ex.bar[p], uint32_t(ctas) * S::kCh * 8);
    Segments<S, REVERSE> sg(ex.seg_a, ex.seg_b, ch);
    const float2 mine = sg.composed();
#pragma unroll 4
    for (int r = 0; r < ctas; ++r)
        cluster_st_async(cluster_map(&ex.cta[p][rank][ch], r), mine.x, mine.y, cluster_map(&ex.bar[p], r));
    if (!mbar_wait_cluster(&ex.bar[p], uint32_t(round >> 1) & 1, wait_ns)) ex.stop = 1, ok = false;
    float s = carry, in = carry;
#pragma unroll 4
    for (int i = 0; i < ctas; ++i) {
        const int r = REVERSE ? ctas - 1 - i : i;
        const float2 v = ex.cta[p][r][ch];
        if (r == rank) in = s;
        s = apply(v.x, v.y, s);
    }
    carry = s;
    sg.finish(ex.seg_b, ch, in, at);
}

// The CTA's way out, all threads, after `round` of `rounds` rounds. Where a wait
// has run out, tiles and gates on their way land first, and the cluster settles
// its exchange.
template <typename S, typename R>
__device__ __forceinline__ void leave(Exchange<S> &ex, R &ring, bool ok, bool stop, int round, int rounds, int rank,
                                      int ctas, bool feeder, int *status) {
    using namespace tc;
    if ((!ok || stop) && feeder) ring.drain();
    if (__any_sync(0xffffffffu, !ok) && (threadIdx.x & 31) == 0) record_status(status, GDN_ETIMEOUT);
    if (stop) {
        async_copy_wait_all();
        if (threadIdx.x == 0) ex.gave_up.tell(round, rank, ctas);
        cluster_arrive();
    } else {
        cluster_arrive_relaxed();
    }
    cluster_wait();  // no CTA sends any more, and none leaves while another may
    if (threadIdx.x < 32) ex.gave_up.settle(ex.bar, rounds, rank, ctas, S::kCh * 8);
}

// Tile loads through a ring of stages: one thread issues, everyone waits.
template <typename T, bool CHANNEL, bool BACKWARD>
struct Ring {
    using S = Tile<BACKWARD && !CHANNEL>;
    static constexpr int kTile = S::kRows * S::kCh;                                 // elements of one tensor's tile
    static constexpr uint32_t kTiles = kTile * sizeof(T) * (1 + CHANNEL + BACKWARD);  // x, g per channel, dout
    static constexpr uint32_t kState = BACKWARD ? S::kCh * 4 : 0;                     // the state before the tile
    static constexpr uint32_t kBytes = kTiles + kState;
    // CTAs of an SM that registers allow, and stages that shared memory then
    // allows. The smallest tiles (bf16, gates per head) leave room for three
    // (8 heads x 700 rows 6.6 us, with two of twice the rows 8.4; 32 heads x
    // 38429 136 against 135).
    static constexpr int kCtasPerSm = BACKWARD && sizeof(T) == 4 ? 1 : kTiles <= 16384 ? 3 : 2;
    static constexpr int kStages = kCtasPerSm == 1 || kTiles <= 32768 ? 2 : 1;
    static constexpr size_t kSmem = size_t(kStages) * kBytes + 128;
    uint8_t *base;
    uint64_t *full;
    int asked = 0;  // tiles, by the issuing thread

    __device__ __forceinline__ const T *x(int i) const { return reinterpret_cast<const T *>(base + (i % kStages) * kBytes); }
    __device__ __forceinline__ const T *g(int i) const { return x(i) + kTile; }
    __device__ __forceinline__ const T *dout(int i) const { return x(i) + (1 + CHANNEL) * kTile; }

    __device__ __forceinline__ const float *state(int i) const {
        return reinterpret_cast<const float *>(base + (i % kStages) * kBytes + kTiles);
    }

    // by one thread: tile i of this CTA's walk, rows from t0, channels from c0 of head h
    __device__ __forceinline__ void load(int i, const CUtensorMap *mx, const CUtensorMap *mg, const CUtensorMap *md,
                                         const RecArgs &a, int c0, int h, int t0) {
        uint64_t *bar = &full[i % kStages];
        asked = i + 1;
        const bool state = BACKWARD && t0 < a.total_tokens;
        tc::mbar_arrive_expect_tx(bar, state ? kBytes : kTiles);
        if (state)
            tc::bulk_load(base + (i % kStages) * kBytes + kTiles,
                          a.states + ((long long)(t0 / kStateRows) * a.hv + h) * kHeadDim + c0, kState, bar);
        tc::tma_load_3d(const_cast<T *>(x(i)), mx, c0, h, t0, bar);
        if (CHANNEL) tc::tma_load_3d(const_cast<T *>(g(i)), mg, c0, h, t0, bar);
        if (BACKWARD) tc::tma_load_3d(const_cast<T *>(dout(i)), md, c0, h, t0, bar);
    }
    __device__ __forceinline__ void wait(int i, unsigned long long wait_ns, bool &ok) {
        if (ok && !tc::mbar_wait_for(&full[i % kStages], uint32_t((i / kStages) & 1), wait_ns)) ok = false;
    }
    // by the issuing thread of a CTA that leaves early: the last tiles asked
    // for land (2 s each at most) before it exits
    __device__ __forceinline__ void drain() {
        for (int i = asked > kStages ? asked - kStages : 0; i < asked; ++i)
            tc::mbar_wait(&full[i % kStages], uint32_t((i / kStages) & 1));
    }
};

// Gates per head of a tile's rows, a round ahead, by the last warps of the CTA,
// 64 rows each: load() asks for a tile's, each lane's to its own place in shared
// memory (in registers they would hold up the warp's next walk until they are
// there, and with it the CTA), store() turns what the last load() brought into
// decays (rows past the end pass the state on). One warp for all took longer
// than the exchange beside it.
template <int ROWS>
struct HeadGates {
    float g[ROWS ? ROWS : 1];
    static __device__ __forceinline__ bool mine() { return int(threadIdx.x) >= kRecThreads - ROWS / 2; }
    static __device__ __forceinline__ int row() {
        return (int(threadIdx.x) - (kRecThreads - ROWS / 2)) / 32 * 64 + int(threadIdx.x & 31);
    }
    __device__ __forceinline__ void load(const RecArgs &a, int t0, int h) {
#pragma unroll
        for (int k = 0; k < 64; k += 32) {
            const int r = row() + k, t = t0 + r;
            if (t >= 0 && t < a.total_tokens)
                tc::async_copy_4(&g[r], static_cast<const float *>(a.g) + (long long)t * a.hv + h);
            else
                g[r] = 0.f;
        }
        tc::async_copy_commit();
    }
    __device__ __forceinline__ void store(float2 *to, float2 *products) const {
        const int r = row();
        tc::async_copy_wait_all();
        float2 d = vec::exp_exact2(make_float2(g[r], g[r + 32]));
        to[r] = vec::both(d.x);
        to[r + 32] = vec::both(d.y);
#pragma unroll
        for (int m = 1; m < kPart; m *= 2) {
            d.x *= __shfl_xor_sync(0xffffffffu, d.x, m);
            d.y *= __shfl_xor_sync(0xffffffffu, d.y, m);
        }
        if (r % kPart == 0) {
            products[r / kPart] = vec::both(d.x);
            products[(r + 32) / kPart] = vec::both(d.y);
        }
    }
};

// Decays of a segment's rows for the lane's two channels: pairs of their own,
// in registers, or the head's one value, in shared memory. A decay's error is
// taken as often as the state remembers rows: gates per head (few) and f32
// gates are exact to a rounding (with u = 2^-24, 1.1 u at most; the state is off
// by 2e-7 where it remembers 55 rows, 7e-7 at 1000). For bf16 gates per channel
// that would cost a quarter of the forward pass's time (T = 65536 x 32 heads:
// 327 us against 260), and the base-2 unit is taken instead. Over all bf16 gates
// from -4 on it is off by 1.9 u at most, 0.5 to 0.85 u in the mean square and
// -0.1 to -0.5 u in the mean; expf, which the decode step takes, by 1.9, 0.5 to
// 0.7 and -0.1 to 0.4 u. States that remember 36, 92 and 667 rows are then off
// by 6e-7, 1.4e-6 and 4e-6 (with expf 2e-7, 3e-7 and 7e-6). Below -4, where the
// state is forgotten, log2 e's own rounding adds up to |g| / 4.5 u.
template <typename T, bool CHANNEL, typename S>
struct Decays;
template <typename T, typename S>
struct Decays<T, true, S> {
    float2 d[S::kSeg];
    __device__ __forceinline__ Decays(const T *g_tile, const float2 *, const float2 *) {
#pragma unroll
        for (int i = 0; i < S::kSeg; ++i) {
            Pack<T, 2> p;
            p.load(g_tile + i * S::kCh);
            d[i] = sizeof(T) == 4 ? vec::exp_exact2(p.f2(0)) : vec::exp2_of(p.f2(0));
        }
    }
    __device__ __forceinline__ float2 operator()(int i) const { return d[i]; }
    __device__ __forceinline__ float2 product() const {
        float2 p = d[0];
#pragma unroll
        for (int i = 1; i < S::kSeg; ++i) p = mul2(p, d[i]);
        return p;
    }
};
template <typename T, typename S>
struct Decays<T, false, S> {
    const float2 *d, *parts;
    __device__ __forceinline__ Decays(const T *, const float2 *decays, const float2 *products)
        : d(decays), parts(products) {}
    __device__ __forceinline__ float2 operator()(int i) const { return d[i]; }
    __device__ __forceinline__ float2 part(int k) const { return parts[k]; }
    __device__ __forceinline__ float2 product() const {
        float2 p = parts[0];
#pragma unroll
        for (int k = 1; k < S::kSeg / kPart; ++k) p = mul2(p, parts[k]);
        return p;
    }
};

// A walk over a segment, one body(row, checked) a row: most segments hold no
// boundary and no row past the end, and run without the checks for them.
template <int FROM, int TO, typename F>
__device__ __forceinline__ void walk(bool plain, F body) {
    constexpr int kStep = FROM <= TO ? 1 : -1, kCount = (FROM <= TO ? TO - FROM : FROM - TO) + 1;
    if (plain) {
#pragma unroll
        for (int n = 0; n < kCount; ++n) body(FROM + kStep * n, std::false_type{});
    } else {
#pragma unroll
        for (int n = 0; n < kCount; ++n) body(FROM + kStep * n, std::true_type{});
    }
}

__device__ __forceinline__ float2 f2(const Pack<float, 2> &p) { return make_float2(p.e[0], p.e[1]); }
__device__ __forceinline__ float2 f2(const Pack<__nv_bfloat16, 2> &p) {
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&p.r));
}
// row i from `base`: rows are `pitch` bytes apart
template <typename T>
__device__ __forceinline__ T *row_at(T *base, unsigned pitch, int i) {
    return reinterpret_cast<T *>(reinterpret_cast<char *>(base) + (unsigned long long)pitch * unsigned(i));
}

template <typename T>
__device__ __forceinline__ void store2(T *to, float2 v);
template <>
__device__ __forceinline__ void store2<float>(float *to, float2 v) { *reinterpret_cast<float2 *>(to) = v; }
template <>
__device__ __forceinline__ void store2<__nv_bfloat16>(__nv_bfloat16 *to, float2 v) {
    *reinterpret_cast<__nv_bfloat162 *>(to) = __floats2bfloat162_rn(v.x, v.y);
}

template <typename T, bool CHANNEL>
__global__ void __launch_bounds__(kRecThreads, Ring<T, CHANNEL, false>::kCtasPerSm)
k_linrec(const RecArgs a, const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mg, int ctas) {
    using namespace tc;
    using R = Ring<T, CHANNEL, false>;
    using S = typename R::S;
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kSeg = S::kSeg;
    __shared__ Exchange<S> ex;
    using Gates = HeadGates<CHANNEL ? 0 : S::kRows>;
    __shared__ Gates gates;
    __shared__ uint64_t full[R::kStages];
    const int w = S::seg(), c = S::channel();
    const bool last_warp = threadIdx.x >= kRecThreads - 32, feeder = threadIdx.x == kRecThreads - 1;
    const int rank = int(cluster_ctarank()), unit = int(blockIdx.x) / ctas;
    const int h = unit / S::kParts, c0 = unit % S::kParts * S::kCh;
    const int hc = h * kHeadDim + c0 + c;  // this lane's first channel in a row [hv, 128]
    const int tiles = (a.total_tokens + S::kRows - 1) / S::kRows;
    const int rounds = (tiles + ctas - 1) / ctas;
    R ring{reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem) + 127) & ~uintptr_t(127)), full};
    ex.gave_up.init();
    if (threadIdx.x == 0) ex.stop = 0;
    if (feeder) {
        for (int i = 0; i < R::kStages; ++i) mbar_init(&full[i], 1);
        mbar_init(&ex.bar[0], 1);
        mbar_init(&ex.bar[1], 1);
        fence_mbar_init();
        for (int i = 0; i < R::kStages && i < rounds; ++i)
            ring.load(i, &mx, &mg, nullptr, a, c0, h, (i * ctas + rank) * S::kRows);
    }
    __syncthreads();
    cluster_arrive();  // this CTA's barriers are ready
    bool ok = true;
    if (!offsets_ok(a)) {  // the same in every CTA: nothing is written
        if (feeder) ring.drain();
        cluster_wait();
        return;
    }
    const Bounds bd{a.cu, a.num_seqs, a.dense_seqlen, a.total_tokens};
    Bounds::Cursor next = bd.begin<true>();
    if (last_warp && rounds) bd.mark<true>(rank * S::kRows, next, ex.marks[0]);
    if (!CHANNEL && Gates::mine()) {
        gates.load(a, rank * S::kRows, h);
        gates.store(ex.decays[0], ex.products[0]);
        gates.load(a, (ctas + rank) * S::kRows, h);
    }
    copy_empty<S>(a, bd, a.s0, a.final_state, hc, rank, ctas);
    __syncthreads();
    float carry = 0.f;  // of this thread's channel in the exchange, before the round
    const int width = a.hv * kHeadDim;  // of a row
    const unsigned pitch = unsigned(width) * sizeof(T);
    bool stop = false;
    int round = 0;
    while (round < rounds && !stop) {
        const int t0 = (round * ctas + rank) * S::kRows, tw = t0 + w * kSeg;  // the tile's and the warp's first row
        const int rows = min(kSeg, a.total_tokens - tw);                     // may be negative
        const Marks<S> &marks = ex.marks[round & 1];
        const uint32_t starts = marks.starts[w], ends = marks.ends[w];
        const int *first = marks.first + w * kSeg, *last = marks.last + w * kSeg;
        ring.wait(round, a.wait_ns, ok);
        Pack<T, 2> x[kSeg];
        const int o = w * kSeg * S::kCh + c;
#pragma unroll
        for (int i = 0; i < kSeg; ++i) x[i].load(ring.x(round) + o + i * S::kCh);
        const Decays<T, CHANNEL, S> d(ring.g(round) + o, ex.decays[round & 1] + w * kSeg,
                                        ex.products[round & 1] + w * (kSeg / kPart));
        const bool plain = !(starts | ends) && rows == kSeg;
        {
            float2 A = d.product(), B = make_float2(0.f, 0.f);
            walk<0, kSeg - 1>(plain, [&](int i, auto checked) {
                if (checked && (starts >> i & 1)) B = state_of(a.s0, first[i], width, hc);
                B = fma2(d(i), B, f2(x[i]));
            });
            if (starts) A = make_float2(kReset, kReset);
            pair(&ex.seg_a[w][c]) = A;
            pair(&ex.seg_b[w][c]) = B;
        }
        __syncthreads();
        if (round == 0) cluster_wait();  // every CTA's barriers are ready
        if (threadIdx.x < S::kCh)
            exchange<false>(ex, carry, round, rank, ctas, a.wait_ns, ok, [&](int seg, float s) {
                const int t = t0 + seg * kSeg;
                if (seg % (kStateRows / kSeg) == 0 && a.states && t < a.total_tokens)
                    a.states[(long long)(t / kStateRows) * width + h * kHeadDim + c0 + threadIdx.x] = s;
            });
        if (last_warp && round + 1 < rounds) {
            // the tile is in registers: its stage takes a later one
            if (feeder && ok && round + R::kStages < rounds)
                ring.load(round + R::kStages, &mx, &mg, nullptr, a, c0, h, t0 + R::kStages * ctas * S::kRows);
            __syncwarp();
            bd.mark<true>(t0 + ctas * S::kRows, next, ex.marks[(round + 1) & 1]);
        }
        if (!CHANNEL && Gates::mine() && round + 1 < rounds) {
            gates.store(ex.decays[(round + 1) & 1], ex.products[(round + 1) & 1]);
            gates.load(a, t0 + 2 * ctas * S::kRows, h);
        }
        __syncthreads();
        stop = ex.stop;
        float2 s = pair(&ex.seg_b[w][c]);
        T *out = static_cast<T *>(a.out) + (long long)tw * width + hc;
        walk<0, kSeg - 1>(plain, [&](int i, auto checked) {
            if (checked) {
                if (i >= rows) return;
                if (starts >> i & 1) s = state_of(a.s0, first[i], width, hc);
            }
            s = fma2(d(i), s, f2(x[i]));
            store2(row_at(out, pitch, i), s);
            if (checked && a.final_state && (ends >> i & 1)) set_state(a.final_state, last[i], width, hc, s);
        });
        ++round;
    }
    if (!rounds) cluster_wait();
    leave(ex, ring, ok, stop, round, rounds, rank, ctas, feeder, a.status);
}

template <typename T, bool CHANNEL>
__global__ void __launch_bounds__(kRecThreads, Ring<T, CHANNEL, true>::kCtasPerSm)
k_linrec_bwd(const RecArgs a, const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mg,
             const __grid_constant__ CUtensorMap md, int ctas) {
    using namespace tc;
    using R = Ring<T, CHANNEL, true>;
    using S = typename R::S;
    constexpr int kSeg = S::kSeg;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ Exchange<S> ex;
    using Gates = HeadGates<CHANNEL ? 0 : S::kRows>;
    __shared__ Gates gates;
    __shared__ float fwd_a[S::kSegs][S::kCh], fwd_b[S::kSegs][S::kCh];
    __shared__ float head_sums[CHANNEL ? 1 : 2][2][CHANNEL ? 1 : S::kRows];  // by round parity, half of the head, row
    __shared__ uint64_t full[R::kStages];
    const int w = S::seg(), c = S::channel(), lane = threadIdx.x & 31;
    const bool last_warp = threadIdx.x >= kRecThreads - 32, feeder = threadIdx.x == kRecThreads - 1;
    const int rank = int(cluster_ctarank()), unit = int(blockIdx.x) / ctas;
    const int h = unit / S::kParts, c0 = unit % S::kParts * S::kCh;
    const int hc = h * kHeadDim + c0 + c;
    const int tiles = (a.total_tokens + S::kRows - 1) / S::kRows;
    const int rounds = (tiles + ctas - 1) / ctas;
    const int t_first = ((rounds - 1) * ctas + rank) * S::kRows, t_step = ctas * S::kRows;
    R ring{reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem) + 127) & ~uintptr_t(127)), full};
    ex.gave_up.init();
    if (threadIdx.x == 0) ex.stop = 0;
    if (feeder) {
        for (int i = 0; i < R::kStages; ++i) mbar_init(&full[i], 1);
        mbar_init(&ex.bar[0], 1);
        mbar_init(&ex.bar[1], 1);
        fence_mbar_init();
        for (int i = 0; i < R::kStages && i < rounds; ++i)
            ring.load(i, &mx, &mg, &md, a, c0, h, t_first - i * t_step);
    }
    __syncthreads();
    cluster_arrive();
    bool ok = true;
    if (!offsets_ok(a)) {
        if (feeder) ring.drain();
        cluster_wait();
        return;
    }
    const Bounds bd{a.cu, a.num_seqs, a.dense_seqlen, a.total_tokens};
    Bounds::Cursor next = bd.begin<false>();
    if (last_warp && rounds) bd.mark<false>(t_first, next, ex.marks[0]);  // without rows there is no first tile
    if (!CHANNEL && Gates::mine()) {
        gates.load(a, t_first, h);
        gates.store(ex.decays[0], ex.products[0]);
        gates.load(a, t_first - t_step, h);
    }
    copy_empty<S>(a, bd, a.dfinal, a.dinitial, hc, rank, ctas);
    __syncthreads();
    float carry = 0.f;
    const int width = a.hv * kHeadDim;  // of a row
    const unsigned pitch = unsigned(width) * sizeof(T);
    // dg per head of the tile at row t: the sums of the head's two halves
    auto write_head_sums = [&](int parity, int t) {
        const int r = threadIdx.x;
        if (r < S::kRows && t + r < a.total_tokens)
            static_cast<float *>(a.dg)[(long long)(t + r) * a.hv + h] = head_sums[parity][0][r] + head_sums[parity][1][r];
    };
    bool stop = false;
    int round = 0;
    while (round < rounds && !stop) {
        const int t0 = t_first - round * t_step, tw = t0 + w * kSeg;
        const int rows = min(kSeg, a.total_tokens - tw);
        // the segment's rows that start (s is reset) and end (e is reset) a sequence
        const Marks<S> &marks = ex.marks[round & 1];
        const uint32_t starts = marks.starts[w], ends = marks.ends[w];
        const int *first = marks.first + w * kSeg, *last = marks.last + w * kSeg;
        const bool plain = !(starts | ends) && rows == kSeg;
        ring.wait(round, a.wait_ns, ok);
        const float state = ring.state(round)[threadIdx.x % S::kCh];  // unused where the tile starts a sequence
        Pack<T, 2> x[kSeg], dy[kSeg];
        const int o = w * kSeg * S::kCh + c;
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
            x[i].load(ring.x(round) + o + i * S::kCh);
            dy[i].load(ring.dout(round) + o + i * S::kCh);
        }
        const Decays<T, CHANNEL, S> d(ring.g(round) + o, ex.decays[round & 1] + w * kSeg,
                                        ex.products[round & 1] + w * (kSeg / kPart));
        // the rows' maps: forward for s, in reverse for e
        float2 to_part[kSeg / kPart];  // from the segment's first row with s = 0 to every part's
        {
            const float2 A = d.product();
            float2 B = make_float2(0.f, 0.f), E = make_float2(0.f, 0.f);
            walk<0, kSeg - 1>(plain, [&](int i, auto checked) {
                if (!CHANNEL && i % kPart == 0) to_part[i / kPart] = B;
                if (checked && (starts >> i & 1)) B = state_of(a.s0, first[i], width, hc);
                B = fma2(d(i), B, f2(x[i]));
            });
            walk<kSeg - 1, 0>(plain, [&](int i, auto checked) {
                if (checked && (ends >> i & 1)) E = state_of(a.dfinal, last[i], width, hc);
                E = mul2(d(i), vec::add2(f2(dy[i]), E));
            });
            const float2 reset = make_float2(kReset, kReset);
            pair(&fwd_a[w][c]) = starts ? reset : A;
            pair(&fwd_b[w][c]) = B;
            pair(&ex.seg_a[w][c]) = ends ? reset : A;
            pair(&ex.seg_b[w][c]) = E;
        }
        __syncthreads();
        if (feeder && ok && round + R::kStages < rounds)
            ring.load(round + R::kStages, &mx, &mg, &md, a, c0, h, t0 - R::kStages * t_step);
        if (!CHANNEL && round) write_head_sums((round - 1) & 1, t0 + t_step);
        if (round == 0) cluster_wait();
        __syncwarp();
        if (threadIdx.x < S::kCh) {
            exchange<true>(ex, carry, round, rank, ctas, a.wait_ns, ok, [](int, float) {});
        } else if (threadIdx.x < 2 * S::kCh) {
            const int ch = threadIdx.x - S::kCh;
            Segments<S, false> sg(fwd_a, fwd_b, ch);
            sg.finish(fwd_b, ch, state, [](int, float) {});
        }
        if (last_warp && round + 1 < rounds) {
            __syncwarp();
            bd.mark<false>(t0 - t_step, next, ex.marks[(round + 1) & 1]);
        }
        if (!CHANNEL && Gates::mine() && round + 1 < rounds) {
            __syncwarp();
            gates.store(ex.decays[(round + 1) & 1], ex.products[(round + 1) & 1]);
            gates.load(a, t0 - 2 * t_step, h);
        }
        __syncthreads();
        stop = ex.stop;
        // The segment's states are kept for kPart rows at a time, the last part
        // first: from the states at the parts' first rows each part is walked
        // again.
        constexpr int kParts = kSeg / kPart;
        float2 e = pair(&ex.seg_b[w][c]), at_part[kParts];
        {
            float2 s = pair(&fwd_b[w][c]);
            at_part[0] = s;
            if constexpr (CHANNEL) {
                walk<0, kSeg - kPart - 1>(plain, [&](int i, auto checked) {
                    if (checked && (starts >> i & 1)) s = state_of(a.s0, first[i], width, hc);
                    s = fma2(d(i), s, f2(x[i]));
                    if (i % kPart == kPart - 1) at_part[i / kPart + 1] = s;
                });
            } else {  // the parts' products are at hand: s is A s + what it would be from zero
                float2 A = both(1.f);
#pragma unroll
                for (int k = 1; k < kParts; ++k) {
                    A = mul2(A, d.part(k - 1));
                    at_part[k] = starts & ((1u << (k * kPart)) - 1) ? to_part[k] : fma2(A, s, to_part[k]);
                }
            }
        }
        T *dx = static_cast<T *>(a.dx) + (long long)tw * width + hc;
        T *dgc = static_cast<T *>(a.dg) + (long long)tw * width + hc;  // per channel
        auto part_walk = [&](auto part_) {
            constexpr int part = decltype(part_)::value;
            float2 s = at_part[part], before[kPart];
            walk<part * kPart, part * kPart + kPart - 1>(plain, [&](int i, auto checked) {
                if (checked && (starts >> i & 1)) s = state_of(a.s0, first[i], width, hc);
                before[i % kPart] = s;
                s = fma2(d(i), s, f2(x[i]));
            });
            float sums[kPart];
            walk<part * kPart + kPart - 1, part * kPart>(plain, [&](int i, auto checked) {
                if (checked && (ends >> i & 1)) e = state_of(a.dfinal, last[i], width, hc);
                const float2 ds = vec::add2(f2(dy[i]), e);
                e = mul2(d(i), ds);
                const float2 dg = mul2(e, before[i % kPart]);
                if (!CHANNEL) sums[i % kPart] = dg.x + dg.y;
                if (!checked || i < rows) {
                    store2(row_at(dx, pitch, i), ds);
                    if (CHANNEL) store2(row_at(dgc, pitch, i), dg);
                    if (checked && a.dinitial && (starts >> i & 1))
                        set_state(a.dinitial, first[i], width, hc, e);
                }
            });
            if (!CHANNEL) {
                // eight rows' sums over the warp's channels: lanes halve the
                // rows they add, lane 4 r ends with row r
#pragma unroll
                for (int m = 16, k = kPart / 2; k; m >>= 1, k >>= 1) {
                    const bool up = lane & m;
#pragma unroll
                    for (int i = 0; i < k; ++i) {
                        const float send = up ? sums[i] : sums[i + k], keep = up ? sums[i + k] : sums[i];
                        sums[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
                    }
                }
                sums[0] += __shfl_xor_sync(0xffffffffu, sums[0], 2);
                sums[0] += __shfl_xor_sync(0xffffffffu, sums[0], 1);
                // written out after the next round's first barrier
                if ((lane & 3) == 0) head_sums[round & 1][c / 64][w * kSeg + part * kPart + (lane >> 2)] = sums[0];
            }
        };
        part_walk(std::integral_constant<int, 1>{});
        part_walk(std::integral_constant<int, 0>{});
        ++round;
    }
    if (!CHANNEL && rounds) {
        __syncthreads();
        if (!stop) write_head_sums((rounds - 1) & 1, rank * S::kRows);
    }
    if (!rounds) cluster_wait();
    leave(ex, ring, ok, stop, round, rounds, rank, ctas, feeder, a.status);
}

static_assert(kPart == 8, "the sums over a head's channels take eight rows at a time");

// Decode step: a warp takes one (sequence, head) row, four channels a lane.
// HBM-bound (state read and written, x and out); every access of a warp is
// contiguous. bf16, 32 heads: 1024 sequences 10.5 us (0.82 of the copy rate),
// 256 3.0 us (0.72: launch and one latency).
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

void launch_shape(cudaLaunchConfig_t &cfg, cudaLaunchAttribute &at, int grid, int ctas, size_t smem) {
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(kRecThreads);
    cfg.dynamicSmemBytes = smem;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = unsigned(ctas);
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
}

// Clusters of `ctas` CTAs of kernel `fn` that the current device runs at once.
// Asked once for each size (it takes the driver some microseconds).
template <typename R, typename F>
cudaError_t active_clusters(F *fn, int ctas, int &clusters) {
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices][kMaxCluster + 1];  // 0: not asked yet; one array a kernel
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kDevices && (clusters = known[dev][ctas].load(std::memory_order_relaxed)) > 0) {
        clusters -= 1;
        return cudaSuccess;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at = {};
    launch_shape(cfg, at, ctas, ctas, R::kSmem);
    e = cudaOccupancyMaxActiveClusters(&clusters, fn, &cfg);
    if (e != cudaSuccess) return e;
    if (dev < kDevices) known[dev][ctas].store(clusters + 1, std::memory_order_relaxed);
    return cudaSuccess;
}

// Launches `units` clusters of kernel `fn`, each over the whole token axis.
// The more CTAs a cluster has, the more of the axis is in work: as many as
// there are tiles, as kMaxCluster, and as lets all clusters run at once (a
// second wave would start on the whole axis when the first is done: at
// T = 65536 with 64 units, 262 us with clusters of 4 against 289 with 8). So a
// unit has at most kMaxCluster CTAs: with few heads most SMs are without work,
// and the time goes with the rounds (1 head x 65536 rows 61 us forward, 32 CTAs
// of 128 rows; its bytes would take 7).
template <typename R, typename... P, typename... A>
cudaError_t launch_clusters(void (*fn)(P...), const RecArgs &a, cudaStream_t s, const A &...maps) {
    using S = typename R::S;
    const void *f = reinterpret_cast<const void *>(fn);
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, int(R::kSmem));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    const int units = a.hv * S::kParts, tiles = (a.total_tokens + S::kRows - 1) / S::kRows;
    int ctas = tiles < kMaxCluster ? tiles : kMaxCluster;
    for (; ctas > 1; --ctas) {
        int clusters = 0;
        e = active_clusters<R>(fn, ctas, clusters);
        if (e != cudaSuccess) return e;
        if (clusters >= units) break;
    }
    if (ctas < 1) ctas = 1;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at = {};
    launch_shape(cfg, at, units * ctas, ctas, R::kSmem);
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, fn, a, maps..., ctas);
}

// the tensor map of a [total_tokens, hv, 128] tensor's tiles
template <typename S, typename T>
bool tile_map(CUtensorMap *map, const void *base, const RecArgs &a) {
    return make_tmap_head_rows(map, base, sizeof(T) == 4, a.hv, a.total_tokens, S::kCh, S::kRows);
}

template <typename T, bool CHANNEL>
cudaError_t forward(const RecArgs &a, cudaStream_t s) {
    using R = Ring<T, CHANNEL, false>;
    using S = typename R::S;
    CUtensorMap mx = {}, mg = {};
    if (a.total_tokens > 0) {
        if (!tile_map<S, T>(&mx, a.x, a)) return cudaErrorInvalidValue;
        if (CHANNEL && !tile_map<S, T>(&mg, a.g, a)) return cudaErrorInvalidValue;
    }
    LaunchScope scope(GDN_K_LINREC, s);
    return launch_clusters<R>(k_linrec<T, CHANNEL>, a, s, mx, mg);
}

template <typename T, bool CHANNEL>
cudaError_t backward(const RecArgs &a, cudaStream_t s) {
    using R = Ring<T, CHANNEL, true>;
    using S = typename R::S;
    CUtensorMap mx = {}, mg = {}, md = {};
    if (a.total_tokens > 0) {
        if (!tile_map<S, T>(&mx, a.x, a) || !tile_map<S, T>(&md, a.dout, a)) return cudaErrorInvalidValue;
        if (CHANNEL && !tile_map<S, T>(&mg, a.g, a)) return cudaErrorInvalidValue;
    }
    LaunchScope scope(GDN_K_LINREC_BWD, s);
    return launch_clusters<R>(k_linrec_bwd<T, CHANNEL>, a, s, mx, mg, md);
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
