// Linear attention with a decay for each head, bf16, on the tensor cores.
//
// Chunks of 128 tokens. With tab[n] = lambda^n, for the chunk's rows i, j and
// the state S that enters it, in time:
//   out_i = scale_out (lambda^(i+1) a_i S + sum_{j<=i} lambda^(i-j) (a_i b_j) c_j)
//   S'    = lambda^len S + sum_j lambda^(len-1-j) b_j^T c_j
// and against time with the mirrored exponents. Four products of 128^3 a chunk:
//   P = A B^T, intra = (P o decays) C, inter = A S, sum = (decayed B)^T C.
// A, B and C are exact in bf16. Roundings to bf16 are those of the decayed
// scores and of the state as an operand of `inter`: each is of the size of the
// output's own rounding. The state itself stays f32 in registers, and what is
// added to it is exact to 2^-24: with the decay in three bf16 parts
// w = w1 + w2 + w3, decayed B goes in as four (fl rounds to bf16),
//   h = fl(w1 b),  w1 b - h,  m = fl(w2 b),  fl(w3 b + (w2 b - m)),
// where the differences are exact, so that each takes one bf16x2 FMA for two
// elements. (Two parts would leave 3e-6 in a final state that is f32, one 2e-3;
// three of f32 arithmetic take 12 instructions a pair instead of 5.)
#include <string.h>

#include "gdn_linattn.cuh"
#include "tc_ptx.cuh"
#include "tma_host.cuh"

namespace gdn {
namespace la {
namespace {

constexpr int kC = 128;                  // tokens of a chunk
constexpr uint32_t kTile = kC * 128 * 2;  // bytes of a bf16 tile: two halves of 64 columns, 128-byte swizzled rows
constexpr uint32_t kHalf = kTile / 2;
constexpr uint32_t kTmem = 0;  // where an allocation of all 512 columns starts
constexpr uint64_t kDrainNs = 100000000ull;

struct Maps {
    CUtensorMap a[3], b[3], c[3], o[3];
};

// Segment, head and role of a CTA.
struct Item {
    Seg seg;
    int index, h, role;
    __device__ __forceinline__ explicit Item(const Args &p)
        : index(blockIdx.x / (p.roles * p.hv)), h(blockIdx.x / p.roles % p.hv), role(blockIdx.x % p.roles) {}
};
__device__ __forceinline__ bool segment_of(const Args &p, uint32_t smem, Item &it) {
    wait_for_previous();
    it.seg = p.segs[it.index];  // (beside the count, not behind it)
    if (it.index >= *p.n_segs) return false;
    if (smem & 1023u) {  // (dynamic shared memory alone starts at a multiple: the tiles' swizzle counts on it)
        record_status(p.status, GDN_ECUDA);
        return false;
    }
    return true;
}

// Bounded waits: one that runs out marks the CTA, and every other wait of it
// ends then. The limit is one of cycles, of which there is more than one a
// nanosecond: little code, since the roles' loops have to stay in the
// instruction cache together (521 us of walk with 77 KB of code, 436 with 58).
// The warp that issues the products polls; the many that wait for it suspend,
// which leaves the issue slots to those at work (5% of the walk).
struct Waiter {
    volatile int *dead;
    long long limit;
    template <bool kPoll>
    __device__ __forceinline__ bool one(uint64_t *bar, uint32_t parity) const {
        const long long t0 = clock64();
        while (!(kPoll || limit < (long long)tc::kShortLimitNs ? tc::mbar_test_wait(bar, parity) : tc::mbar_try_wait(bar, parity)))
            if (*dead || clock64() - t0 > limit) {
                *dead = 1;
                return false;
            }
        return true;
    }
    __device__ __forceinline__ bool one(uint64_t *bar, uint32_t parity) const { return one<false>(bar, parity); }
    // of a whole warp, which goes on as one
    __device__ __forceinline__ bool warp(uint64_t *bar, uint32_t parity) const {
        return __all_sync(0xffffffffu, one<false>(bar, parity));
    }
    __device__ __forceinline__ bool poll(uint64_t *bar, uint32_t parity) const {
        return __all_sync(0xffffffffu, one<true>(bar, parity));
    }
};

__device__ __forceinline__ uint32_t pack2(float x, float y) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float2 unpack2(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// Address inside one column half of a tile of row `row`'s 16-byte group `g`
__device__ __forceinline__ uint8_t *at(uint8_t *half, int row, int g) { return half + tc::sw128_offset(row, g); }

// The decays of a pair of rows of B in three bf16 parts.
struct PairDecay {
    uint32_t w[3];
};
__device__ __forceinline__ PairDecay pair_decay(float2 w) {
    PairDecay d;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        d.w[i] = pack2(w.x, w.y);
        const float2 u = unpack2(d.w[i]);
        w.x -= u.x, w.y -= u.y;
    }
    return d;
}

__device__ __forceinline__ __nv_bfloat162 bf2(uint32_t u) { return *reinterpret_cast<const __nv_bfloat162 *>(&u); }
__device__ __forceinline__ uint32_t raw2(__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t *>(&v); }

// B's rows row0 .. row0 + 15 of a tile, transposed, decayed and in four parts,
// into tensor-memory columns to + step q .. + 7 for part q. w[i][j]: part i of
// the decays of rows row0 + 2 j and the next. Rows behind `len` count as zeros
// whatever they hold. The warp's lanes are B's columns 32 (warp % 4) ...
__device__ __forceinline__ void split_rows(const uint8_t *tile, int row0, const uint32_t *w0, const uint32_t *w1,
                                           const uint32_t *w2, int len, uint32_t to, uint32_t step) {
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
    const uint32_t from = tc::smem_u32(tile) + (quarter >> 1) * kHalf;
    // this lane's row of the blocks: of (columns 0-7, 8-15) x (rows 0-7, 8-15)
    const int block = lane >> 3, trow = row0 + (block >> 1) * 8 + (lane & 7);
    uint32_t x[8], y[8], d[3][2];
#pragma unroll
    for (int c = 0; c < 2; ++c)  // 16 columns of B
        tc::ldmatrix_x4_trans(from + tc::sw128_offset(trow, (quarter & 1) * 4 + 2 * c + (block & 1)), x + 4 * c);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int j = 4 * k + (lane & 3);
        d[0][k] = w0[j], d[1][k] = w1[j], d[2][k] = w2[j];
    }
    if (row0 + 16 > len) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int row = row0 + 8 * (k >> 1 & 1) + 2 * (lane & 3);
            if (row >= len) x[k] = 0;
            else if (row + 1 >= len) x[k] &= 0xffffu;
        }
    }
    const uint32_t lanes = tc::tmem_addr(to, quarter * 32, 0);
    auto store = [&](int part) {
        tc::tmem_st_16x8(lanes + part * step, y);
        tc::tmem_st_16x8(lanes + (16 << 16) + part * step, y + 4);
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = raw2(__hmul2_rn(bf2(d[i][k >> 1 & 1]), bf2(x[k])));
        store(2 * i);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            __nv_bfloat162 v = __hfma2(bf2(d[i][k >> 1 & 1]), bf2(x[k]), __hneg2(bf2(y[k])));
            if (i) v = __hfma2(bf2(d[2][k >> 1 & 1]), bf2(x[k]), v);
            y[k] = raw2(v);
        }
        store(2 * i + 1);
    }
}

// zeros in the rows of a tile behind the sequence, by 256 threads
__device__ __forceinline__ void zero_behind(uint8_t *tile, int len, int t) {
    const int row = t & 127;
    if (row >= len) {
#pragma unroll
        for (int g = 0; g < 8; ++g) *reinterpret_cast<uint4 *>(at(tile + (t >> 7) * kHalf, row, g)) = make_uint4(0, 0, 0, 0);
    }
    tc::fence_proxy_async_smem();
}

// a tile, counted on `full`
__device__ __forceinline__ void load_tile(uint8_t *dst, const CUtensorMap *map, int head, int row, uint64_t *full) {
    tc::tma_load_3d(dst, map, 0, head, row, full);
    tc::tma_load_3d(dst + kHalf, map, 64, head, row, full);
}

// brings a tile into L2
__device__ __forceinline__ void prefetch_tile(const CUtensorMap *map, int head, int row) {
    tc::tma_prefetch_3d(map, 0, head, row);
    tc::tma_prefetch_3d(map, 64, head, row);
}

// operand descriptors: of a whole tile, and what k-step `k` (16 of the product's inner dimension) adds to it
__device__ __forceinline__ uint64_t k_major(const void *tile) { return tc::sdesc_sw128(tc::smem_u32(tile), 0, 1024); }
__device__ __forceinline__ uint64_t mn_major(const void *tile) { return tc::sdesc_sw128(tc::smem_u32(tile), kHalf, 1024); }
__host__ __device__ constexpr uint32_t k_step(int k) { return ((k >> 2) * kHalf + (k & 3) * 32) >> 4; }
__host__ __device__ constexpr uint32_t mn_step(int k) { return k * 2048 >> 4; }
constexpr uint32_t kIdKK = tc::idesc_bf16_f32(128, 128, false, false);
constexpr uint32_t kIdKM = tc::idesc_bf16_f32(128, 128, false, true);

// sum (+)= the four parts' products with C's rows row0 .. row0 + 16 K - 1
template <int K>
__device__ __forceinline__ void mma_parts(uint32_t sum, uint32_t part, uint32_t step, uint64_t c, int row0, bool fresh) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int k = 0; k < K; ++k)
            tc::mma_bf16_ts(sum, part + q * step + 8 * k, c + mn_step(row0 / 16 + k), kIdKM, !(fresh && q == 0 && k == 0));
}

// ---------------------------------------------------------------------------
// Sum of one segment: states[seg] = sum_j lambda^(distance to the segment's
// end that the walk leaves by) b_j^T c_j. 16 warps split B (32 rows each group
// of four) and add up the chunks' sums (32 columns each group), one copies, one
// issues the products.
// The tensor cores cut what they add to an accumulator instead of rounding it:
// 32 additions a chunk in one accumulator over 57 chunks left a sum 2e-5 too
// small, one chunk leaves 4e-7. So each chunk has an accumulator of its own, of
// two in turn, and the chunks' sums are added in f32 registers.
// ---------------------------------------------------------------------------
// Bound by latency between HBM and the products (1.1 us of a chunk): 178 us at
// 65536 tokens x 32 heads (256 segments of 57 chunks on 152 SMs, 1.56 us a chunk;
// 717 MB at 4.0 TB/s). With one accumulator for all chunks it took 168 us, with
// one for two chunks 174 us and errors of 9e-7.
constexpr int kSumThreads = 576, kSumSplit = 16;  // warps that split B
constexpr uint32_t kSumParts = 256;  // tensor-memory columns of the parts: 4 sets of 4 x 16, behind two accumulators

struct SumShared {
    uint8_t b[3][kTile], c[3][kTile];
    uint32_t w[kSumSplit][3][16];  // decays of a warp's rows
    float tab[kC + 4];
    uint64_t b_full[3], b_free[3], c_full[3], c_clean[3], c_free[3], part_full[4], part_free[4], sum_full[2], sum_free[2], done;
    uint32_t tmem;
    int dead;
};

__global__ void __launch_bounds__(kSumThreads, 1) k_la_sum_tc(const __grid_constant__ Args p,
                                                              const __grid_constant__ Maps m) {
    extern __shared__ __align__(1024) uint8_t raw[];
    SumShared &s = *reinterpret_cast<SumShared *>(raw);
    Item it(p);
    const Role &r = p.role[it.role];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    next_may_start();
    const float decay = p.decay[it.h];
    if (tid <= kC) s.tab[tid] = power(decay, tid);
    if (warp == kSumSplit && lane == 0) {
        for (int i = 0; i < 3; ++i) {
            tc::mbar_init(&s.b_full[i], 1);
            tc::mbar_init(&s.b_free[i], kSumSplit);
            tc::mbar_init(&s.c_full[i], 1);
            tc::mbar_init(&s.c_clean[i], kSumSplit);
            tc::mbar_init(&s.c_free[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            tc::mbar_init(&s.part_full[i], 4);
            tc::mbar_init(&s.part_free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&s.sum_full[i], 1);
            tc::mbar_init(&s.sum_free[i], kSumSplit);
        }
        tc::mbar_init(&s.done, 1);
        s.dead = 0;
        tc::fence_mbar_init();
    }
    if (!segment_of(p, tc::smem_u32(raw), it)) return;
    const Seg seg = it.seg;
    if (seg.flags & (r.against ? kFirst : kLast)) return;  // no segment follows
    const int chunks = (seg.len + kC - 1) / kC;
    auto load = [&](int n) {
        const int u = n % 3;
        tc::mbar_arrive_expect_tx(&s.b_full[u], kTile);
        tc::mbar_arrive_expect_tx(&s.c_full[u], kTile);
        load_tile(s.b[u], &m.b[it.role], it.h / r.gb, seg.start + n * kC, &s.b_full[u]);
        load_tile(s.c[u], &m.c[it.role], it.h / r.gc, seg.start + n * kC, &s.c_full[u]);
    };
    int asked = 0;  // chunks whose tiles the copying thread has asked for
    if (warp == kSumSplit && lane == 0)
        for (; asked < min(3, chunks); ++asked) load(asked);
    if (warp == kSumSplit + 1) {
        tc::tmem_alloc(&s.tmem, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const Waiter wait{&s.dead, (long long)p.wait_ns};
    // a set of parts for each quarter of a chunk's rows
    auto part_of = [&](int quarter) { return kTmem + kSumParts + quarter * 64; };
    auto sum_of = [&](int n) { return kTmem + (n & 1) * 128; };

    if (warp == kSumSplit) {
        if (lane == 0) {
            for (; asked < chunks; ++asked) {
                const uint32_t ph = (asked / 3 - 1) & 1;
                if (!wait.one(&s.b_free[asked % 3], ph) || !wait.one(&s.c_free[asked % 3], ph)) break;
                load(asked);
            }
        }
    } else if (warp == kSumSplit + 1) {
        const bool leader = tc::elect_one();
        const uint64_t tiles = mn_major(s.c[0]);
        bool ok = true;
        for (int n = 0; n < chunks && ok; ++n) {
            const int u = n % 3;
            ok = wait.poll(&s.c_full[u], (n / 3) & 1) && wait.poll(&s.c_clean[u], (n / 3) & 1) &&
                 (n < 2 || wait.poll(&s.sum_free[n & 1], ((n >> 1) - 1) & 1));
            const uint64_t c = tiles + u * (kTile >> 4);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                if (!(ok = ok && wait.poll(&s.part_full[g], n & 1))) break;
                tc::tc_fence_after();
                if (leader) {
                    mma_parts<2>(sum_of(n), part_of(g), 16, c, 32 * g, g == 0);
                    tc::mma_commit(&s.part_free[g]);
                    if (g == 3) {
                        tc::mma_commit(&s.c_free[u]);
                        tc::mma_commit(&s.sum_full[n & 1]);
                    }
                }
            }
        }
        if (leader) {
            tc::mma_commit(&s.done);  // all products have ended
            tc::mbar_wait(&s.done, 0, kDrainNs);
        }
    } else {
        const int group = warp >> 2, row0 = group * 32;
        float sum[32] = {};  // lane: b, columns 32 group ..: c
        auto add_sum = [&](int n) {
            if (!wait.warp(&s.sum_full[n & 1], (n >> 1) & 1)) return false;
            tc::tc_fence_after();
            float v[32];
            tc::tmem_ld32(tc::tmem_addr(sum_of(n), (warp & 3) * 32, 32 * group), v);
            tc::tmem_ld_wait();
            tc::tc_fence_before();
            tc::warp_arrive(&s.sum_free[n & 1]);
#pragma unroll
            for (int i = 0; i < 32; ++i) sum[i] += v[i];
            return true;
        };
        bool ok = true;
        for (int n = 0; n < chunks && ok; ++n) {
            const int u = n % 3, from = n * kC, len = min(kC, seg.len - from);
            const uint32_t ph = (n / 3) & 1;
            if (len < kC) {
                if (!(ok = wait.warp(&s.c_full[u], ph))) break;
                if (warp < 8) zero_behind(s.c[u], len, tid);
            }
            tc::warp_arrive(&s.c_clean[u]);
            const float over = r.scale_in * power(decay, r.against ? from : seg.len - from - len);
            const int row = row0 + 2 * lane;
            uint32_t(*w)[16] = s.w[warp];
            __syncwarp();
            if (lane < 16) {
                const PairDecay d = pair_decay(r.against ? make_float2(over * s.tab[row], over * s.tab[row + 1])
                                                         : make_float2(over * s.tab[max(len - 1 - row, 0)],
                                                                       over * s.tab[max(len - 2 - row, 0)]));
                w[0][lane] = d.w[0], w[1][lane] = d.w[1], w[2][lane] = d.w[2];
            }
            __syncwarp();
            if (n > 1 && !(ok = add_sum(n - 2))) break;  // (while the last chunk's products run)
            if (!(ok = wait.warp(&s.b_full[u], ph))) break;
            if (n > 0 && !(ok = wait.warp(&s.part_free[group], (n - 1) & 1))) break;
            tc::tc_fence_after();
#pragma unroll 1
            for (int t = 0; t < 2; ++t)
                split_rows(s.b[u], row0 + 16 * t, w[0] + 8 * t, w[1] + 8 * t, w[2] + 8 * t, len, part_of(group) + 8 * t, 16);
            tc::warp_arrive(&s.b_free[u]);
            tc::tmem_st_wait();
            tc::tc_fence_before();
            tc::warp_arrive(&s.part_full[group]);
        }
        if (ok && (chunks < 2 || add_sum(chunks - 2)) && add_sum(chunks - 1)) {
            float *to = r.states + (size_t(it.index) * p.hv + it.h) * kState + ((warp & 3) * 32 + lane) * kHeadDim + 32 * group;
#pragma unroll
            for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4 *>(to + i) = make_float4(sum[i], sum[i + 1], sum[i + 2], sum[i + 3]);
        }
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    if (tid == 0 && s.dead) record_status(p.status, GDN_ETIMEOUT);
    if (warp == kSumSplit && lane == 0 && s.dead)
        // tiles on their way have to land before the CTA ends, whichever warp gave up (behind the barrier: none will)
        for (int k = max(0, asked - 3); k < asked; ++k) {
            tc::mbar_wait(&s.b_full[k % 3], (k / 3) & 1, kDrainNs);
            tc::mbar_wait(&s.c_full[k % 3], (k / 3) & 1, kDrainNs);
        }
    if (warp == kSumSplit + 1) tc::tmem_dealloc(kTmem, 512);
}

// ---------------------------------------------------------------------------
// The walk of one segment. Warps 0-3 take the scores' decays, warps 4-11 split
// B (each group of four every other 16 rows), warps 12-19 hold the state (row
// b, 64 columns c a thread) and finish the output, warps 20 and 22 copy in and
// out, warp 21 issues the products (23 fills their group of four, whose registers
// the others get). The products' order, P, sum, inter, intra of each chunk, leaves
// each of the other warps the time of five products or more.
// inter and intra have one accumulator: both are taken over the row's
// e = max(lambda^(i+1), 2^-64), which the finished row is multiplied with.
// Where a decay is below 2^-64 the state's part is 2^-64 of the undecayed one
// instead.
// What bounds a chunk is shared memory as much as the products: 56 products of
// 128 x 128 x 16 take 67 cycles each, an operand in shared memory is 4 KiB of
// its 128 bytes a cycle, and both operands there would fill it. So the parts of
// B and the scores are operands in tensor memory (for B's parts alone that gave
// nothing, 535 and 534 us of walk, while other steps bound it). Descriptors are in uniform registers: products
// under `lane == 0` instead of an elected lane cost 8%.
// Measured: 375 to 385 us at 65536 tokens x 32 heads (1.6 GB of its own at
// 4.2 TB/s), 37 us at 4096: 3.5 us a chunk and SM, 1.94 of it products. The rest is the
// latency of about ten hand-offs a chunk (250 to 600 cycles each) around P ->
// scores -> intra -> output. Tried and left: a second issuing warp for the sums,
// and warps of their own for the output (375 -> 390 to 424 us: as many again
// wait, and take issue slots), products in rolled loops (400 us).
// ---------------------------------------------------------------------------
constexpr int kWalkThreads = 768;
constexpr uint32_t kColP = 0, kColOut = 128, kColSum = 256, kColPart = 384;  // parts: 4 sets of 4 x 8 columns
constexpr float kLeast = 5.421010862427522e-20f;                             // 2^-64

struct WalkShared {
    uint8_t a[2][kTile], b[2][kTile], c[2][kTile], state[kTile];
    float between[2 * kC];  // [128 + d]: lambda^|d|, d from -128 to 127
    uint32_t w[2][3][kC / 2];  // decays of B's rows, of a whole chunk and of the sequence's last one
    uint64_t ab_full[2], c_full[2], a_free[2], b_free[2], c_clean, c_free[2], part_full[4], part_free[4], p_full,
        scores_full, sum_full, sum_free, state_full, state_free, out_full, out_free, staged[2], drain;
    uint32_t tmem;
    int dead;
};

// 32 bytes to global memory: one sector a thread
__device__ __forceinline__ void store_sector(void *to, const uint32_t *w, bool whole) {
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4 *>(to)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4 *>(to)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

__global__ void __launch_bounds__(kWalkThreads, 1) k_la_walk_tc(const __grid_constant__ Args p,
                                                                const __grid_constant__ Maps m) {
    extern __shared__ __align__(1024) uint8_t raw[];
    WalkShared &s = *reinterpret_cast<WalkShared *>(raw);
    Item it(p);
    const Role &r = p.role[it.role];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    next_may_start();
    const float decay = p.decay[it.h];
    if (tid <= kC) {
        const float f = power(decay, tid);
        s.between[kC - tid] = f;
        if (tid < kC) s.between[kC + tid] = f;
    }
    if (warp == 20 && lane == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&s.ab_full[i], 1);
            tc::mbar_init(&s.c_full[i], 1);
            tc::mbar_init(&s.a_free[i], 1);
            tc::mbar_init(&s.b_free[i], 9);
            tc::mbar_init(&s.c_free[i], 1);
            tc::mbar_init(&s.staged[i], 8);
        }
        for (int i = 0; i < 4; ++i) {
            tc::mbar_init(&s.part_full[i], 4);
            tc::mbar_init(&s.part_free[i], 1);
        }
        tc::mbar_init(&s.p_full, 1);
        tc::mbar_init(&s.scores_full, 4);
        tc::mbar_init(&s.sum_full, 1);
        tc::mbar_init(&s.sum_free, 8);
        tc::mbar_init(&s.state_full, 8);
        tc::mbar_init(&s.state_free, 1);
        tc::mbar_init(&s.out_full, 1);
        tc::mbar_init(&s.out_free, 8);
        tc::mbar_init(&s.c_clean, 8);
        tc::mbar_init(&s.drain, 1);
        s.dead = 0;
        tc::fence_mbar_init();
    }
    if (!segment_of(p, tc::smem_u32(raw), it)) return;
    const Seg seg = it.seg;
    const int chunks = (seg.len + kC - 1) / kC;
    const bool leaves = r.fin && (seg.flags & (r.against ? kFirst : kLast));  // the state behind the last chunk is wanted
    // the walk's n-th chunk
    auto chunk_from = [&](int n) { return (r.against ? chunks - 1 - n : n) * kC; };
    auto chunk_len = [&](int n) { return min(kC, seg.len - chunk_from(n)); };
    auto sums = [&](int n) { return n + 1 < chunks || leaves; };
    // tiles of the n-th chunk; A and B are counted on one barrier
    auto row_of = [&](int n) { return seg.start + chunk_from(n); };
    auto load_b = [&](int n) {
        tc::mbar_arrive_expect_tx(&s.ab_full[n & 1], 2 * kTile);
        load_tile(s.b[n & 1], &m.b[it.role], it.h / r.gb, row_of(n), &s.ab_full[n & 1]);
    };
    auto load_a = [&](int n) { load_tile(s.a[n & 1], &m.a[it.role], it.h / r.ga, row_of(n), &s.ab_full[n & 1]); };
    auto load_c = [&](int n) {
        tc::mbar_arrive_expect_tx(&s.c_full[n & 1], kTile);
        load_tile(s.c[n & 1], &m.c[it.role], it.h / r.gc, row_of(n), &s.c_full[n & 1]);
    };
    // the chunk after those under way comes from HBM meanwhile
    auto prefetch = [&](int n) {
        if (n >= chunks) return;
        prefetch_tile(&m.b[it.role], it.h / r.gb, row_of(n));
        prefetch_tile(&m.a[it.role], it.h / r.ga, row_of(n));
        prefetch_tile(&m.c[it.role], it.h / r.gc, row_of(n));
    };
    int na = min(2, chunks), nc = na;  // chunks whose A and B, and whose C the copying thread has asked for
    if (warp == 20 && lane == 0) {
        for (int n = 0; n < na; ++n) load_b(n), load_a(n), load_c(n);
        prefetch(2);
    }
    if (tid >= 256 && tid < 256 + kC) {  // B's decays, of a whole chunk and of the one that ends the segment
        const int which = (tid - 256) / (kC / 2), pair = tid % (kC / 2), row = 2 * pair;
        const int len = which ? seg.len - (chunks - 1) * kC : kC;
        float2 f = make_float2(0.f, 0.f);
        if (row < len) f.x = r.scale_in * power(decay, r.against ? row : len - 1 - row);
        if (row + 1 < len) f.y = r.scale_in * power(decay, r.against ? row + 1 : len - 2 - row);
        const PairDecay d = pair_decay(f);
#pragma unroll
        for (int i = 0; i < 3; ++i) s.w[which][i][pair] = d.w[i];
    }
    if (warp == 21) {
        tc::tmem_alloc(&s.tmem, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const Waiter wait{&s.dead, (long long)p.wait_ns};
    auto power_of = [&](int n) { return s.between[kC - n]; };  // lambda^n, n from 0 to 128

    // 768 threads are launched with 80 registers each: 128 x (56 + 40) + 256 x (64 + 128) is the same
    if (warp >= 20) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 20 && lane == 0) {
            for (int n = 2; n < chunks; ++n) {
                const int u = n & 1;
                const uint32_t ph = ((n >> 1) - 1) & 1;
                if (!wait.one(&s.b_free[u], ph) || !wait.one(&s.a_free[u], ph)) break;
                load_b(n), load_a(n), ++na;
                prefetch(n + 1);
                if (!wait.one(&s.c_free[u], ph)) break;
                load_c(n), ++nc;
            }
        } else if (warp == 22 && lane == 0) {  // finished chunks out, and their C's place back
            // (of the two barriers the one of chunk n is not arrived at again before C's place is: chunk n + 2 needs it)
            for (int n = 0; n < chunks; ++n) {
                if (!wait.one(&s.staged[n & 1], (n >> 1) & 1)) break;
                if (chunk_len(n) == kC) {
                    const int boxes = r.partial ? 4 : 2;  // of 128 bytes a row
                    for (int q = 0; q < boxes; ++q)
                        tc::tma_store_3d(&m.o[it.role], q * 64, it.h, row_of(n), (q < 2 ? s.c : s.a)[n & 1] + (q & 1) * kHalf);
                    tc::bulk_commit_group();
                    tc::bulk_wait_group_read<0>();
                }
                tc::mbar_arrive(&s.c_free[n & 1]);
                if (r.partial) tc::mbar_arrive(&s.a_free[n & 1]);
            }
            tc::bulk_wait_group_all();
        } else if (warp == 21 && chunks > 0) {
            const bool leader = tc::elect_one();
            const uint64_t a0 = k_major(s.a[0]), b0 = k_major(s.b[0]), c0 = mn_major(s.c[0]), st = mn_major(s.state);
            auto tile = [](int n) { return uint64_t(n & 1) * (kTile >> 4); };
            auto scores = [&](int n) {
                if (!wait.poll(&s.ab_full[n & 1], (n >> 1) & 1)) return false;
                tc::tc_fence_after();
                const uint64_t a = a0 + tile(n), b = b0 + tile(n);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) tc::mma_bf16(kTmem + kColP, a + k_step(k), b + k_step(k), kIdKK, k > 0);
                    tc::mma_commit(&s.p_full);
                    tc::mma_commit(&s.b_free[n & 1]);
                }
                return true;
            };
            bool ok = true;
            for (int n = 0; ok && n < chunks; ++n) {
                const uint32_t ph = n & 1, before = (n - 1) & 1;
                const uint64_t c = c0 + tile(n), a = a0 + tile(n);
                const bool more = sums(n);
                if (!(ok = scores(n) && wait.poll(&s.c_full[n & 1], (n >> 1) & 1) &&
                           (chunk_len(n) == kC || wait.poll(&s.c_clean, 0))))
                    break;
                if (more) {
                    if (n > 0 && !(ok = wait.poll(&s.sum_free, before))) break;
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        if (!(ok = ok && wait.poll(&s.part_full[t & 3], t >> 2))) break;
                        tc::tc_fence_after();
                        if (leader) {
                            mma_parts<1>(kTmem + kColSum, kTmem + kColPart + (t & 3) * 32, 8, c, 16 * t, t == 0);
                            tc::mma_commit(&s.part_free[t & 3]);
                            if (t == 7) tc::mma_commit(&s.sum_full);
                        }
                    }
                    if (!ok) break;
                }
                if (!(ok = wait.poll(&s.state_full, ph) && (n == 0 || wait.poll(&s.out_free, before)))) break;
                tc::tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) tc::mma_bf16(kTmem + kColOut, a + k_step(k), st + mn_step(k), kIdKM, k > 0);
                    tc::mma_commit(&s.state_free);
                    if (!r.partial) tc::mma_commit(&s.a_free[n & 1]);
                }
                if (!(ok = wait.poll(&s.scores_full, ph))) break;
                tc::tc_fence_after();
                if (leader) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) tc::mma_bf16_ts(kTmem + kColOut, kTmem + kColP + k * 8, c + mn_step(k), kIdKM, 1);
                    tc::mma_commit(&s.out_full);
                }
            }
            if (leader) {
                tc::mma_commit(&s.drain);
                tc::mbar_wait(&s.drain, 0, kDrainNs);
            }
        }
    } else if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        // decayed scores: row i of the chunk, bf16 over the scores' own columns. Beside the diagonal block of
        // 32 the decay is one factor of the row times one of the column (at most 1), in it one of i - j.
        const int i = tid, i0 = warp * 32;
        const uint32_t mine = tc::tmem_addr(kTmem + kColP, i0, 0);
        const float row_in = r.against ? power_of(i0 + 32 - i) : power_of(i - i0);
        const float *diagonal = s.between + kC - i, *beside = s.between + kC - i0 - (r.against ? 32 : 0);
#pragma unroll 1
        for (int n = 0; n < chunks; ++n) {
            const int len = chunk_len(n), off = entry_offset(r, seg, n == 0);
            const float over = r.scale_in / fmaxf(power_of(r.against ? max(len - 1 - i, 0) + off : i + off), kLeast);
            const float2 over2 = make_float2(over, over), row2 = make_float2(row_in * over, row_in * over);
            if (!wait.warp(&s.p_full, n & 1)) break;
            tc::tc_fence_after();
#pragma unroll 1
            for (int j0 = 0; j0 < kC; j0 += 16) {
                uint32_t w[8];
                const int x = j0 >> 5;
                if (r.against ? x < warp || j0 >= len : x > warp) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) w[k] = 0;
                } else {
                    float v[16];
                    tc::tmem_ld16(mine + j0, v);
                    tc::tmem_ld_wait();
                    if (x == warp) {
                        const float *f = diagonal + j0;
                        const int at = r.against ? j0 - i : i - j0, step = r.against ? 1 : -1;
#pragma unroll
                        for (int k = 0; k < 16; k += 2) {
                            const float2 y = __fmul2_rn(make_float2(v[k], v[k + 1]), __fmul2_rn(over2, make_float2(f[k], f[k + 1])));
                            v[k] = at + step * k >= 0 ? y.x : 0.f;
                            v[k + 1] = at + step * (k + 1) >= 0 ? y.y : 0.f;
                        }
                    } else {
                        const float *f = beside + j0;
#pragma unroll
                        for (int k = 0; k < 16; k += 4) {
                            const float4 g = *reinterpret_cast<const float4 *>(f + k);
                            const float2 v0 = __fmul2_rn(make_float2(v[k], v[k + 1]), __fmul2_rn(row2, make_float2(g.x, g.y)));
                            const float2 v1 = __fmul2_rn(make_float2(v[k + 2], v[k + 3]), __fmul2_rn(row2, make_float2(g.z, g.w)));
                            v[k] = v0.x, v[k + 1] = v0.y, v[k + 2] = v1.x, v[k + 3] = v1.y;
                        }
                    }
                    if (j0 + 16 > len) {  // columns behind the sequence
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            if (j0 + k >= len) v[k] = 0.f;
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) w[k] = pack2(v[2 * k], v[2 * k + 1]);
                }
                tc::tmem_st8(mine + j0 / 2, w);
            }
            tc::tmem_st_wait();
            tc::tc_fence_before();
            tc::warp_arrive(&s.scores_full);
        }
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        // B, decayed, in parts, every other 16 rows; C's rows behind the sequence
        const int group = (warp - 4) >> 2;
        bool ok = true;
#pragma unroll 1
        for (int n = 0; n < chunks && ok; ++n) {
            const int len = chunk_len(n);
            if (len < kC) {
                if (!(ok = wait.warp(&s.c_full[n & 1], (n >> 1) & 1))) break;
                zero_behind(s.c[n & 1], len, tid - 128);
                tc::warp_arrive(&s.c_clean);  // (one chunk of a segment at most is not whole)
            }
            if (!sums(n)) break;  // the last chunk
            if (!(ok = wait.warp(&s.ab_full[n & 1], (n >> 1) & 1))) break;
            const uint32_t(*w)[kC / 2] = s.w[len < kC];
#pragma unroll 1
            for (int t = group; t < 8; t += 2) {
                const int set = t & 3;
                if (8 * n + t >= 4 && !(ok = wait.warp(&s.part_free[set], (t >> 2) ^ 1))) break;
                tc::tc_fence_after();
                split_rows(s.b[n & 1], 16 * t, w[0] + 8 * t, w[1] + 8 * t, w[2] + 8 * t, len, kTmem + kColPart + set * 32, 8);
                if (t >= 6) tc::warp_arrive(&s.b_free[n & 1]);
                tc::tmem_st_wait();
                tc::tc_fence_before();
                tc::warp_arrive(&s.part_full[set]);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 128;");
        const int half = (warp - 12) >> 2, row = tid & 127, lane0 = (warp & 3) * 32, c0 = half * 64;
        const uint32_t sum = tc::tmem_addr(kTmem + kColSum, lane0, c0), acc = tc::tmem_addr(kTmem + kColOut, lane0, c0);
        const size_t per_head = size_t(p.hv) * kState;
        float2 st[32];  // row b of the state, columns c0 ..
        // the state that enters: the sequence's own, or the chained sum of the segments before
        const bool own = seg.flags & (r.against ? kLast : kFirst);
        const float *enters = own ? r.init : r.states;
        if (enters) {
            enters += size_t(own ? seg.seq : it.index) * per_head + size_t(it.h) * kState;
            if (own && r.swapped) {
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    st[k] = make_float2(enters[(c0 + 2 * k) * kHeadDim + row], enters[(c0 + 2 * k + 1) * kHeadDim + row]);
            } else {
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                    const float4 v = *reinterpret_cast<const float4 *>(enters + row * kHeadDim + c0 + 2 * k);
                    st[k] = make_float2(v.x, v.y), st[k + 1] = make_float2(v.z, v.w);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) st[k] = make_float2(0.f, 0.f);
        }
        bool ok = true;
#pragma unroll 1
        for (int n = 0; n <= chunks; ++n) {
            const uint32_t before = (n - 1) & 1;
            if (n > 0 && sums(n - 1)) {  // S = lambda^len S + the chunk's sum
                if (!(ok = wait.warp(&s.sum_full, before))) break;
                tc::tc_fence_after();
                const float keep = power_of(chunk_len(n - 1) - 1 + entry_offset(r, seg, n == 1));
#pragma unroll
                for (int x = 0; x < 64; x += 16) {
                    float v[16];
                    tc::tmem_ld16(sum + x, v);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        st[x / 2 + k] = __ffma2_rn(make_float2(keep, keep), st[x / 2 + k], make_float2(v[2 * k], v[2 * k + 1]));
                }
                tc::tc_fence_before();
                tc::warp_arrive(&s.sum_free);
            }
            if (n < chunks) {
                if (n > 0 && !(ok = wait.warp(&s.state_free, before))) break;
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    const float2 *x = st + 4 * g;
                    *reinterpret_cast<uint4 *>(at(s.state + half * kHalf, row, g)) =
                        make_uint4(pack2(x[0].x, x[0].y), pack2(x[1].x, x[1].y), pack2(x[2].x, x[2].y), pack2(x[3].x, x[3].y));
                }
                tc::fence_proxy_async_smem();
                tc::warp_arrive(&s.state_full);
            }
            if (n > 0) {  // the output of the chunk before
                const int c = n - 1, len = chunk_len(c), from = seg.start + chunk_from(c);
                const int off = entry_offset(r, seg, c == 0);
                const float f = r.scale_out * fmaxf(power_of(r.against ? max(len - 1 - row, 0) + off : row + off), kLeast);
                const float2 f2 = make_float2(f, f);
                const size_t at_out = (size_t(from + row) * p.hv + it.h) * kHeadDim + c0;
                if (!(ok = wait.warp(&s.out_full, before))) break;
                tc::tc_fence_after();
                // a whole chunk's rows go through the place of its C (f32 ones' second half through that of its A), and
                // out by copies
                const bool staged = len == kC;
                uint8_t *stage = r.partial ? (half ? s.a : s.c)[c & 1] : s.c[c & 1] + half * kHalf;
#pragma unroll 1
                for (int x = 0; x < 64; x += 16) {
                    float v[16];
                    tc::tmem_ld16(acc + x, v);
                    tc::tmem_ld_wait();
                    if (x == 48) {
                        tc::tc_fence_before();
                        tc::warp_arrive(&s.out_free);
                    }
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float2 y = __fmul2_rn(f2, make_float2(v[2 * k], v[2 * k + 1]));
                        if (r.partial) w[2 * k] = __float_as_uint(y.x), w[2 * k + 1] = __float_as_uint(y.y);
                        else w[k] = pack2(y.x, y.y);
                    }
                    if (staged) {
                        uint8_t *box = r.partial ? stage + (x >> 5) * kHalf : stage;
                        const int g = r.partial ? (x & 31) / 4 : x / 8;
                        *reinterpret_cast<uint4 *>(at(box, row, g)) = make_uint4(w[0], w[1], w[2], w[3]);
                        *reinterpret_cast<uint4 *>(at(box, row, g + 1)) = make_uint4(w[4], w[5], w[6], w[7]);
                        if (r.partial) {
                            *reinterpret_cast<uint4 *>(at(box, row, g + 2)) = make_uint4(w[8], w[9], w[10], w[11]);
                            *reinterpret_cast<uint4 *>(at(box, row, g + 3)) = make_uint4(w[12], w[13], w[14], w[15]);
                        }
                    } else if (row < len) {
                        if (r.partial) {
                            float *to = static_cast<float *>(r.out) + at_out + x;
                            store_sector(to, w, r.sectors);
                            store_sector(to + 8, w + 8, r.sectors);
                        } else {
                            store_sector(static_cast<__nv_bfloat16 *>(r.out) + at_out + x, w, r.sectors);
                        }
                    }
                }
                if (staged) tc::fence_proxy_async_smem();
                tc::warp_arrive(&s.staged[c & 1]);
            }
        }
        if (leaves && ok) {
            const float f = r.against && seg.len > 0 ? power_of(1) : 1.f;  // to the gradient of the state before the first token
            float *to = r.fin + size_t(seg.seq) * per_head + size_t(it.h) * kState;
            if (f != 1.f) {
#pragma unroll
                for (int k = 0; k < 32; ++k) st[k] = __fmul2_rn(make_float2(f, f), st[k]);
            }
#pragma unroll
            for (int k = 0; k < 32; k += 2)
                *reinterpret_cast<float4 *>(to + row * kHeadDim + c0 + 2 * k) =
                    make_float4(st[k].x, st[k].y, st[k + 1].x, st[k + 1].y);
        }
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    if (tid == 0 && s.dead) record_status(p.status, GDN_ETIMEOUT);
    if (warp == 20 && lane == 0 && s.dead) {
        // tiles on their way have to land before the CTA ends, whichever warp gave up (behind the barrier: none will)
        for (int k = max(0, na - 2); k < na; ++k) tc::mbar_wait(&s.ab_full[k & 1], (k >> 1) & 1, kDrainNs);
        for (int k = max(0, nc - 2); k < nc; ++k) tc::mbar_wait(&s.c_full[k & 1], (k >> 1) & 1, kDrainNs);
    }
    if (warp == 21) tc::tmem_dealloc(kTmem, 512);
}

// Boxes of 128 rows and 64 bf16 of a head (of f32 rows, `wide` 2, 32 elements as pairs of bf16: copies only)
bool tile_map(CUtensorMap *map, const void *base, int heads, int tokens, int wide = 1) {
    const uint64_t row = 256 * uint64_t(wide);
    return make_tmap_bf16_3d(map, base, 128 * wide, uint64_t(heads), uint64_t(tokens), row, uint64_t(heads) * row, 64, 1, kC);
}

}  // namespace

cudaError_t launch_tc(const Args &args, cudaStream_t s) {
    Args a = args;
    for (int i = 0; i < a.roles; ++i) a.role[i].sectors = (reinterpret_cast<uintptr_t>(a.role[i].out) & 31) == 0;
    Maps m;
    memset(&m, 0, sizeof m);
    if (a.total_tokens > 0)
        for (int i = 0; i < a.roles; ++i) {
            const Role &r = a.role[i];
            if (!tile_map(&m.a[i], r.a, a.hv / r.ga, a.total_tokens) || !tile_map(&m.b[i], r.b, a.hv / r.gb, a.total_tokens) ||
                !tile_map(&m.c[i], r.c, a.hv / r.gc, a.total_tokens) ||
                !tile_map(&m.o[i], r.out, a.hv, a.total_tokens, r.partial ? 2 : 1))
                return cudaErrorInvalidValue;
        }
    constexpr int kSumBytes = sizeof(SumShared), kWalkBytes = sizeof(WalkShared);
    static_assert(kSumBytes <= 232448 && kWalkBytes <= 232448, "shared memory of a CTA");
    cudaError_t e = cudaFuncSetAttribute(k_la_sum_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, kSumBytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k_la_walk_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, kWalkBytes);
    if (e != cudaSuccess) return e;
    const unsigned items = unsigned(a.max_segs) * unsigned(a.hv) * unsigned(a.roles);
    if ((e = launch_table(a, s)) != cudaSuccess) return e;
    if (a.seg_len < a.total_tokens) {
        {
            LaunchScope scope(GDN_K_LINATTN_SUM, s);
            e = launch_behind(k_la_sum_tc, dim3(items), kSumThreads, kSumBytes, s, a, m);
        }
        if (e != cudaSuccess || (e = launch_chain(a, s)) != cudaSuccess) return e;
    }
    LaunchScope scope(GDN_K_LINATTN_WALK, s);
    return launch_behind(k_la_walk_tc, dim3(items), kWalkThreads, kWalkBytes, s, a, m);
}

}  // namespace la
}  // namespace gdn
