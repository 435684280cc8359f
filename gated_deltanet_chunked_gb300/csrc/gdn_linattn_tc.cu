// Linear attention with a decay for each head, bf16, on the tensor cores.
//
// Chunks of 128 tokens. With tab[n] = lambda^n, for the chunk's rows i, j and
// the state S that enters it, in time:
//   out_i = scale_out (lambda^(i+1) a_i S + sum_{j<=i} lambda^(i-j) (a_i b_j) c_j)
//   S'    = lambda^len S + sum_j lambda^(len-1-j) b_j^T c_j
// and against time with the mirrored exponents. Four products of 128^3 a chunk:
//   P = A B^T, intra = (P o decays) C, inter = A S, sum = C^T (decayed B).
// A, B and C are exact in bf16. Roundings to bf16 are those of the decayed
// scores and of the state as an operand of `inter`: each is of the size of the
// output's own rounding. The state itself stays f32 in registers, and what is
// added to it is exact to 2^-26: decayed B goes in as three bf16 parts (two
// leave 3e-6 in a final state that is f32, one 2e-3).
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
constexpr uint64_t kDrainNs = 100000000ull;

struct Maps {
    CUtensorMap a[3], b[3], c[3], o[3];
};

// Segment, head and role of CTA `item`.
struct Item {
    Seg seg;
    int index, h, role;
};
__device__ __forceinline__ bool item_of(const Args &p, Item &it) {
    const int i = blockIdx.x;
    it.role = i % p.roles;
    it.h = (i / p.roles) % p.hv;
    it.index = i / (p.roles * p.hv);
    if (it.index >= *p.n_segs) return false;
    it.seg = p.segs[it.index];
    return true;
}

// Bounded waits of one thread: one that runs out marks the CTA, and every other
// wait of it ends then.
struct Waiter {
    volatile int *dead;
    int *status;
    unsigned long long limit;
    __device__ __forceinline__ bool one(uint64_t *bar, uint32_t parity) const {
        if (limit >= tc::kShortLimitNs && tc::mbar_try_wait(bar, parity)) return true;
        const uint64_t t0 = tc::globaltimer_ns();
        for (;;) {
#pragma unroll 1
            for (int i = 0; i < 16; ++i)
                if (tc::mbar_test_wait(bar, parity)) return true;
            if (*dead) return false;
            if (tc::globaltimer_ns() - t0 > limit) {
                *dead = 1;
                record_status(status, GDN_ETIMEOUT);
                return false;
            }
        }
    }
    // of a whole warp, which goes on as one
    __device__ __forceinline__ bool warp(uint64_t *bar, uint32_t parity) const {
        return __all_sync(0xffffffffu, one(bar, parity));
    }
};

__device__ __forceinline__ uint32_t pack2(float x, float y) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float2 unpack2(uint32_t u) {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// w times two bf16, as three bf16 parts (each the nearest to what is left)
__device__ __forceinline__ void split3(uint32_t x, float w, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    float2 v = __fmul2_rn(unpack2(x), make_float2(w, w));
    hi = pack2(v.x, v.y);
    float2 u = unpack2(hi);
    v = __fadd2_rn(v, make_float2(-u.x, -u.y));
    mid = pack2(v.x, v.y);
    u = unpack2(mid);
    v = __fadd2_rn(v, make_float2(-u.x, -u.y));
    lo = pack2(v.x, v.y);
}

// Address inside one half of a tile of row `row`'s 16-byte group `g`
__device__ __forceinline__ uint8_t *at(uint8_t *half, int row, int g) { return half + tc::sw128_offset(row, g); }

// this thread's row (64 columns) of decayed B in three parts; w 0: zeros
// whatever the row holds
__device__ __forceinline__ void split_row(uint8_t *b_half, int row, float w, uint4 *hi, uint4 *mid, uint4 *lo) {
#pragma unroll
    for (int g = 0; g < 8; ++g) {
        uint4 x = *reinterpret_cast<const uint4 *>(at(b_half, row, g));
        if (w == 0.f) x = make_uint4(0, 0, 0, 0);
        split3(x.x, w, hi[g].x, mid[g].x, lo[g].x);
        split3(x.y, w, hi[g].y, mid[g].y, lo[g].y);
        split3(x.z, w, hi[g].z, mid[g].z, lo[g].z);
        split3(x.w, w, hi[g].w, mid[g].w, lo[g].w);
    }
}
__device__ __forceinline__ void store_row(uint8_t *half, int row, const uint4 *x) {
#pragma unroll
    for (int g = 0; g < 8; ++g) *reinterpret_cast<uint4 *>(at(half, row, g)) = x[g];
}

__device__ __forceinline__ void load_tile(uint8_t *dst, const CUtensorMap *map, int head, int row, uint64_t *full) {
    tc::mbar_arrive_expect_tx(full, kTile);
    tc::tma_load_3d(dst, map, 0, head, row, full);
    tc::tma_load_3d(dst + kHalf, map, 64, head, row, full);
}

// operand descriptors of k-step `k` (16 of the product's inner dimension) of a tile
__device__ __forceinline__ uint64_t k_major(uint32_t tile, int k) {
    return tc::sdesc_sw128(tile + (k >> 2) * kHalf + (k & 3) * 32, 0, 1024);
}
__device__ __forceinline__ uint64_t mn_major(uint32_t tile, int k) {
    return tc::sdesc_sw128(tile + k * 2048, kHalf, 1024);
}
constexpr uint32_t kIdKK = tc::idesc_bf16_f32(128, 128, false, false);
constexpr uint32_t kIdMM = tc::idesc_bf16_f32(128, 128, true, true);
constexpr uint32_t kIdKM = tc::idesc_bf16_f32(128, 128, false, true);

__device__ __forceinline__ uint32_t smem_base(const uint8_t *p) { return tc::smem_u32(p); }

// sum[tmem] (+)= C^T part
__device__ __forceinline__ void mma_sum(uint32_t d, const uint8_t *c, const uint8_t *part, bool fresh) {
    const uint32_t ca = smem_base(c), pa = smem_base(part);
#pragma unroll
    for (int k = 0; k < 8; ++k) tc::mma_bf16(d, mn_major(ca, k), mn_major(pa, k), kIdMM, !(fresh && k == 0));
}

// ---------------------------------------------------------------------------
// Sum of one segment: states[seg] = sum_j lambda^(distance to the segment's
// end that the walk leaves by) b_j^T c_j, accumulated in tensor memory over
// all chunks. 8 warps split B, one copies, one issues the products.
// ---------------------------------------------------------------------------
constexpr int kSumThreads = 320;

struct SumShared {
    uint8_t b[2][kTile], c[2][kTile], part[3][kTile];
    float tab[kC + 4];
    uint64_t b_full[2], b_free[2], c_full[2], c_free[2], part_full[3], part_free[3], done;
    uint32_t tmem;
    int dead;
};

__global__ void __launch_bounds__(kSumThreads, 1) k_la_sum_tc(const __grid_constant__ Args p,
                                                              const __grid_constant__ Maps m) {
    extern __shared__ __align__(1024) uint8_t raw[];
    SumShared &s = *reinterpret_cast<SumShared *>(raw + (-tc::smem_u32(raw) & 1023u));
    Item it;
    if (!item_of(p, it)) return;
    const Role &r = p.role[it.role];
    const Seg seg = it.seg;
    if (seg.flags & (r.against ? kFirst : kLast)) return;  // no segment follows
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float decay = p.decay[it.h];
    for (int n = tid; n <= kC; n += kSumThreads) s.tab[n] = power(decay, n);
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&s.b_full[i], 1);
            tc::mbar_init(&s.b_free[i], 8);
            tc::mbar_init(&s.c_full[i], 1);
            tc::mbar_init(&s.c_free[i], 1);
        }
        for (int i = 0; i < 3; ++i) {
            tc::mbar_init(&s.part_full[i], 8);
            tc::mbar_init(&s.part_free[i], 1);
        }
        tc::mbar_init(&s.done, 1);
        s.dead = 0;
        tc::fence_mbar_init();
    }
    if (warp == 9) {
        tc::tmem_alloc(&s.tmem, 128);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = s.tmem;
    const Waiter wait{&s.dead, p.status, p.wait_ns};
    const int chunks = (seg.len + kC - 1) / kC;

    if (warp == 8) {
        if (lane == 0) {
            int n = 0;
            for (; n < chunks; ++n) {
                const int u = n & 1;
                const uint32_t ph = ((n >> 1) - 1) & 1;
                if (n >= 2 && (!wait.one(&s.b_free[u], ph) || !wait.one(&s.c_free[u], ph))) break;
                load_tile(s.b[u], &m.b[it.role], it.h / r.gb, seg.start + n * kC, &s.b_full[u]);
                load_tile(s.c[u], &m.c[it.role], it.h / r.gc, seg.start + n * kC, &s.c_full[u]);
            }
            if (s.dead)  // what is on its way has to land before the CTA ends
                for (int k = max(0, n - 2); k < n; ++k) {
                    tc::mbar_wait(&s.b_full[k & 1], (k >> 1) & 1, kDrainNs);
                    tc::mbar_wait(&s.c_full[k & 1], (k >> 1) & 1, kDrainNs);
                }
        }
    } else if (warp == 9) {
        if (lane == 0) {
            bool ok = true;
            for (int n = 0; n < chunks && ok; ++n) {
                const int u = n & 1;
                if (!(ok = wait.one(&s.c_full[u], (n >> 1) & 1))) break;
                for (int q = 0; q < 3; ++q) {
                    if (!(ok = wait.one(&s.part_full[q], n & 1))) break;
                    tc::tc_fence_after();
                    mma_sum(tmem, s.c[u], s.part[q], n == 0 && q == 0);
                    tc::mma_commit(&s.part_free[q]);
                }
                if (ok) tc::mma_commit(&s.c_free[u]);
            }
            tc::mma_commit(&s.done);  // all products have ended
            tc::mbar_wait(&s.done, 0, kDrainNs);
        }
    } else {
        const int half = warp >> 2, row = tid & 127;
        bool ok = true;
        for (int n = 0; n < chunks && ok; ++n) {
            const int u = n & 1, from = n * kC, len = min(kC, seg.len - from);
            const uint32_t ph = (n >> 1) & 1;
            float w = 0.f;
            if (row < len)
                w = r.scale_in * (r.against ? power(decay, from) * s.tab[row]
                                            : power(decay, seg.len - from - len) * s.tab[len - 1 - row]);
            if (!(ok = wait.warp(&s.b_full[u], ph))) break;
            uint4 part[3][8];
            split_row(s.b[u] + half * kHalf, row, w, part[0], part[1], part[2]);
            tc::warp_arrive(&s.b_free[u]);
            if (len < kC) {  // rows of the next sequence, or behind the tensor's end
                if (!(ok = wait.warp(&s.c_full[u], ph))) break;
                if (row >= len) {
                    const uint4 zero[8] = {};
                    store_row(s.c[u] + half * kHalf, row, zero);
                }
            }
#pragma unroll
            for (int q = 0; q < 3; ++q) {
                if (ok && n > 0) ok = wait.warp(&s.part_free[q], (n - 1) & 1);
                if (ok) {
                    store_row(s.part[q] + half * kHalf, row, part[q]);
                    tc::fence_proxy_async_smem();
                    tc::warp_arrive(&s.part_full[q]);
                }
            }
        }
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    if (warp < 8 && !s.dead) {  // lane: c, columns: b
        const int c = tid & 127, b0 = (warp >> 2) * 64;
        float *to = r.states + (size_t(it.index) * p.hv + it.h) * kState + c;
#pragma unroll
        for (int x = 0; x < 64; x += 16) {
            float v[16];
            tc::tmem_ld16(tc::tmem_addr(tmem, (warp & 3) * 32, b0 + x), v);
            tc::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) to[(b0 + x + i) * kHeadDim] = v[i];
        }
        tc::tc_fence_before();
    }
    __syncthreads();
    if (warp == 9) tc::tmem_dealloc(tmem, 128);
}

// ---------------------------------------------------------------------------
// The walk of one segment. Warps 0-3 take the scores' decays, warps 4-11 hold
// the state (row c, 64 columns b a thread), split B and finish the output,
// warp 12 copies, warp 13 issues the products (14 and 15 fill a group of four
// warps, to which registers are dealt).
// ---------------------------------------------------------------------------
constexpr int kWalkThreads = 512;
constexpr uint32_t kColP = 0, kColIntra = 128, kColInter = 256, kColSum = 384;

struct WalkShared {
    uint8_t a[2][kTile], b[kTile], c[kTile], part[2][kTile], state[kTile];
    float tab[kC + 4];   // lambda^n
    float down[kC + 4];  // lambda^(128 - n)
    uint64_t a_full[2], a_free[2], b_full, b_free, c_full, c_free, part_full, third_full, first_free, p_full, scores_full,
        sum_full, sum_free, state_full, state_free, out_full, out_free, staged[2], drain;
    uint32_t tmem;
    int dead;
};

__global__ void __launch_bounds__(kWalkThreads, 1) k_la_walk_tc(const __grid_constant__ Args p,
                                                                const __grid_constant__ Maps m) {
    extern __shared__ __align__(1024) uint8_t raw[];
    WalkShared &s = *reinterpret_cast<WalkShared *>(raw + (-tc::smem_u32(raw) & 1023u));
    Item it;
    if (!item_of(p, it)) return;
    const Role &r = p.role[it.role];
    const Seg seg = it.seg;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float decay = p.decay[it.h];
    for (int n = tid; n <= kC; n += kWalkThreads) {
        const float f = power(decay, n);
        s.tab[n] = f;
        s.down[kC - n] = f;
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&s.a_full[i], 1);
            tc::mbar_init(&s.a_free[i], 2);
            tc::mbar_init(&s.staged[i], 4);
        }
        tc::mbar_init(&s.b_full, 1);
        tc::mbar_init(&s.b_free, 9);
        tc::mbar_init(&s.c_full, 1);
        tc::mbar_init(&s.c_free, 1);
        tc::mbar_init(&s.part_full, 8);
        tc::mbar_init(&s.third_full, 8);
        tc::mbar_init(&s.first_free, 1);
        tc::mbar_init(&s.p_full, 1);
        tc::mbar_init(&s.scores_full, 4);
        tc::mbar_init(&s.sum_full, 1);
        tc::mbar_init(&s.sum_free, 8);
        tc::mbar_init(&s.state_full, 8);
        tc::mbar_init(&s.state_free, 1);
        tc::mbar_init(&s.out_full, 1);
        tc::mbar_init(&s.out_free, 8);
        tc::mbar_init(&s.drain, 1);
        s.dead = 0;
        tc::fence_mbar_init();
    }
    if (warp == 13) {
        tc::tmem_alloc(&s.tmem, 512);
        tc::tmem_relinquish();
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = s.tmem;
    const Waiter wait{&s.dead, p.status, p.wait_ns};
    const int chunks = (seg.len + kC - 1) / kC;
    const bool leaves = r.fin && (seg.flags & (r.against ? kFirst : kLast));  // the state behind the last chunk is wanted
    // the walk's n-th chunk
    auto chunk_from = [&](int n) { return (r.against ? chunks - 1 - n : n) * kC; };
    auto chunk_len = [&](int n) { return min(kC, seg.len - chunk_from(n)); };
    auto sums = [&](int n) { return n + 1 < chunks || leaves; };

    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 12 && lane == 0) {
            int n = 0;
            for (; n < chunks; ++n) {
                const int u = n & 1, row = seg.start + chunk_from(n);
                if (n >= 2 && !wait.one(&s.a_free[u], ((n >> 1) - 1) & 1)) break;
                load_tile(s.a[u], &m.a[it.role], it.h / r.ga, row, &s.a_full[u]);
                if (n >= 1 && !wait.one(&s.b_free, (n - 1) & 1)) { ++n; break; }
                load_tile(s.b, &m.b[it.role], it.h / r.gb, row, &s.b_full);
                if (n >= 1 && !wait.one(&s.c_free, (n - 1) & 1)) { ++n; break; }
                load_tile(s.c, &m.c[it.role], it.h / r.gc, row, &s.c_full);
            }
            if (s.dead && n > 0) {  // what is on its way has to land before the CTA ends
                for (int k = max(0, n - 2); k < n; ++k) tc::mbar_wait(&s.a_full[k & 1], (k >> 1) & 1, kDrainNs);
                tc::mbar_wait(&s.b_full, (n - 1) & 1, kDrainNs);
                tc::mbar_wait(&s.c_full, (n - 1) & 1, kDrainNs);
            }
        } else if (warp == 13 && lane == 0) {
            const uint32_t b = smem_base(s.b), c = smem_base(s.c), st = smem_base(s.state);
            for (int n = 0; n < chunks; ++n) {
                const uint32_t ph = n & 1, before = (n - 1) & 1, a = smem_base(s.a[n & 1]);
                if (!wait.one(&s.a_full[n & 1], (n >> 1) & 1) || !wait.one(&s.b_full, ph)) break;
                tc::tc_fence_after();
#pragma unroll
                for (int k = 0; k < 8; ++k) tc::mma_bf16(tmem + kColP, k_major(a, k), k_major(b, k), kIdKK, k > 0);
                tc::mma_commit(&s.p_full);
                tc::mma_commit(&s.b_free);
                if (!wait.one(&s.c_full, ph)) break;
                if (sums(n)) {
                    if (!wait.one(&s.part_full, ph) || (n > 0 && !wait.one(&s.sum_free, before))) break;
                    tc::tc_fence_after();
                    mma_sum(tmem + kColSum, s.c, s.part[0], true);
                    tc::mma_commit(&s.first_free);
                    mma_sum(tmem + kColSum, s.c, s.part[1], false);
                    if (!wait.one(&s.third_full, ph)) break;
                    tc::tc_fence_after();
                    mma_sum(tmem + kColSum, s.c, s.part[0], false);
                    tc::mma_commit(&s.sum_full);
                }
                // (a chunk's rows behind its sequence are zeroed in C before the state is handed over)
                if (!wait.one(&s.scores_full, ph) || (chunk_len(n) < kC && !wait.one(&s.state_full, ph)) ||
                    (n > 0 && !wait.one(&s.out_free, before)))
                    break;
                tc::tc_fence_after();
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    tc::mma_bf16_ts(tmem + kColIntra, tmem + kColP + k * 8, mn_major(c, k), kIdKM, k > 0);
                tc::mma_commit(&s.c_free);
                if (!wait.one(&s.state_full, ph)) break;
                tc::tc_fence_after();
#pragma unroll
                for (int k = 0; k < 8; ++k) tc::mma_bf16(tmem + kColInter, k_major(a, k), k_major(st, k), kIdKK, k > 0);
                tc::mma_commit(&s.state_free);
                tc::mma_commit(&s.out_full);
            }
            tc::mma_commit(&s.drain);
            tc::mbar_wait(&s.drain, 0, kDrainNs);
        }
    } else if (warp < 4) {
        // decayed scores: row i of the chunk, bf16 over the scores' own columns. Left of the diagonal block of
        // 32 the decay is one factor of the row times one of the column (both at most 1), in it one of i - j.
        const int i = tid, i0 = warp * 32;
        const uint32_t mine = tc::tmem_addr(tmem + kColP, i0, 0);
        for (int n = 0; n < chunks; ++n) {
            if (!wait.warp(&s.p_full, n & 1)) break;
            tc::tc_fence_after();
            const int len = chunk_len(n);
            const float row = r.scale_in * (r.against ? s.tab[i0 + 32 - i] : s.tab[i - i0]);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                uint32_t w[16];
                const int j0 = 32 * x;
                if (r.against ? x < warp || j0 >= len : x > warp) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) w[k] = 0;
                } else {
                    float v[32];
                    tc::tmem_ld32(mine + j0, v);
                    tc::tmem_ld_wait();
                    if (x == warp) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const int d = r.against ? k - lane : lane - k;
                            v[k] = d >= 0 && (!r.against || j0 + k < len) ? v[k] * (r.scale_in * s.tab[max(d, 0)]) : 0.f;
                        }
                    } else {
                        const float *col = r.against ? s.tab + (j0 - i0 - 32) : s.down + (kC - i0 + j0);
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(col + k);
                            v[k] *= row * f.x, v[k + 1] *= row * f.y, v[k + 2] *= row * f.z, v[k + 3] *= row * f.w;
                        }
                        if (r.against && j0 + 32 > len) {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (j0 + k >= len) v[k] = 0.f;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 16; ++k) w[k] = pack2(v[2 * k], v[2 * k + 1]);
                }
                tc::tmem_st16(mine + 16 * x, w);
            }
            tc::tmem_st_wait();
            tc::tc_fence_before();
            tc::warp_arrive(&s.scores_full);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        const int half = (warp - 4) >> 2, row = tid & 127, lane0 = (warp & 3) * 32, b0 = half * 64;
        const uint32_t sum = tc::tmem_addr(tmem + kColSum, lane0, b0), intra = tc::tmem_addr(tmem + kColIntra, lane0, b0),
                       inter = tc::tmem_addr(tmem + kColInter, lane0, b0);
        const size_t per_head = size_t(p.hv) * kState;
        float st[64];
        // the state that enters: the sequence's own, or the chained sum of the segments before
        const bool enters = seg.flags & (r.against ? kLast : kFirst);
        if (!enters) {
            const float *from = r.states + size_t(it.index) * per_head + size_t(it.h) * kState + row;
#pragma unroll
            for (int k = 0; k < 64; ++k) st[k] = from[(b0 + k) * kHeadDim];
        } else if (r.init) {
            const float *from = r.init + size_t(seg.seq) * per_head + size_t(it.h) * kState;
#pragma unroll
            for (int k = 0; k < 64; ++k) st[k] = r.swapped ? from[row * kHeadDim + b0 + k] : from[(b0 + k) * kHeadDim + row];
        } else {
#pragma unroll
            for (int k = 0; k < 64; ++k) st[k] = 0.f;
        }
        // S = lambda^len S + the chunk's sum
        auto advance = [&](int n) {
            const float keep = s.tab[chunk_len(n) - 1 + entry_offset(r, seg, n == 0)];
#pragma unroll
            for (int x = 0; x < 64; x += 16) {
                float v[16];
                tc::tmem_ld16(sum + x, v);
                tc::tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; ++k) st[x + k] = fmaf(keep, st[x + k], v[k]);
            }
            tc::tc_fence_before();
        };
        uint32_t stores = 0;
        // the output of chunk n, through the place of its A tile when it is whole
        auto finish = [&](int n) {
            const int len = chunk_len(n), from = seg.start + chunk_from(n);
            const int off = entry_offset(r, seg, n == 0);
            const float f = row < len ? r.scale_out * s.tab[r.against ? len - 1 - row + off : row + off] : 0.f;
            const bool staged = len == kC && !r.partial;
            uint8_t *half_tile = s.a[n & 1] + half * kHalf;
            const size_t at_out = (size_t(from + row) * p.hv + it.h) * kHeadDim + b0;
#pragma unroll
            for (int x = 0; x < 64; x += 16) {
                float u[16], v[16];
                tc::tmem_ld16(intra + x, u);
                tc::tmem_ld16(inter + x, v);
                tc::tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 16; ++k) u[k] = fmaf(f, v[k], r.scale_out * u[k]);
                if (r.partial) {
                    if (row < len) {
                        float4 *to = reinterpret_cast<float4 *>(static_cast<float *>(r.out) + at_out + x);
#pragma unroll
                        for (int k = 0; k < 4; ++k) to[k] = make_float4(u[4 * k], u[4 * k + 1], u[4 * k + 2], u[4 * k + 3]);
                    }
                } else {
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const float *w = u + 8 * g;
                        const uint4 y = make_uint4(pack2(w[0], w[1]), pack2(w[2], w[3]), pack2(w[4], w[5]), pack2(w[6], w[7]));
                        if (staged) *reinterpret_cast<uint4 *>(at(half_tile, row, x / 8 + g)) = y;
                        else if (row < len)
                            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(r.out) + at_out + x + 8 * g) = y;
                    }
                }
            }
            tc::tc_fence_before();
            tc::warp_arrive(&s.out_free);
            if (staged) {
                tc::fence_proxy_async_smem();
                tc::warp_arrive(&s.staged[half]);
                if (row == 0 && wait.one(&s.staged[half], stores++ & 1)) {
                    tc::tma_store_3d(&m.o[it.role], b0, it.h, from, half_tile);
                    tc::bulk_commit_group();
                }
                __syncwarp();
            }
        };
        uint8_t *b_half = s.b + half * kHalf;
        int n = 0;
        for (; n < chunks; ++n) {
            const uint32_t ph = n & 1, before = (n - 1) & 1;
            const int len = chunk_len(n);
            const bool more = sums(n);
            if (n > 0) {
                if (!wait.warp(&s.sum_full, before)) break;
                tc::tc_fence_after();
                advance(n - 1);
                tc::warp_arrive(&s.sum_free);
            }
            if (len < kC) {
                if (!wait.warp(&s.c_full, ph)) break;
                if (row >= len) {
                    const uint4 zero[8] = {};
                    store_row(s.c + half * kHalf, row, zero);
                }
            }
            uint4 lo[8];
            if (more) {
                if (!wait.warp(&s.b_full, ph)) break;
                const float w = row < len ? r.scale_in * s.tab[r.against ? row : len - 1 - row] : 0.f;
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    uint4 x = *reinterpret_cast<const uint4 *>(at(b_half, row, g)), hi, mid;
                    if (w == 0.f) x = make_uint4(0, 0, 0, 0);
                    split3(x.x, w, hi.x, mid.x, lo[g].x);
                    split3(x.y, w, hi.y, mid.y, lo[g].y);
                    split3(x.z, w, hi.z, mid.z, lo[g].z);
                    split3(x.w, w, hi.w, mid.w, lo[g].w);
                    *reinterpret_cast<uint4 *>(at(s.part[0] + half * kHalf, row, g)) = hi;
                    *reinterpret_cast<uint4 *>(at(s.part[1] + half * kHalf, row, g)) = mid;
                }
                tc::fence_proxy_async_smem();
                tc::warp_arrive(&s.part_full);
            }
            tc::warp_arrive(&s.b_free);
            if (n > 0 && !wait.warp(&s.state_free, before)) break;
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                const float *x = st + 8 * g;
                *reinterpret_cast<uint4 *>(at(s.state + half * kHalf, row, g)) =
                    make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
            }
            tc::fence_proxy_async_smem();
            tc::warp_arrive(&s.state_full);
            if (n > 0) {
                if (!wait.warp(&s.out_full, before)) break;
                tc::tc_fence_after();
                finish(n - 1);
            }
            if (more) {
                if (!wait.warp(&s.first_free, ph)) break;
                store_row(s.part[0] + half * kHalf, row, lo);
                tc::fence_proxy_async_smem();
                tc::warp_arrive(&s.third_full);
            }
            if (n > 0 && row == 0) {  // the output's copy has read the tile that the next A goes to
                tc::bulk_wait_group_read<0>();
                tc::mbar_arrive(&s.a_free[(n - 1) & 1]);
            }
            __syncwarp();
        }
        if (n == chunks) {
            bool ok = true;
            if (leaves && chunks > 0) {
                ok = wait.warp(&s.sum_full, (chunks - 1) & 1);
                if (ok) {
                    tc::tc_fence_after();
                    advance(chunks - 1);
                }
            }
            if (chunks > 0 && ok && wait.warp(&s.out_full, (chunks - 1) & 1)) {
                tc::tc_fence_after();
                finish(chunks - 1);
            }
            if (leaves && ok) {
                const float f = r.against && seg.len > 0 ? s.tab[1] : 1.f;  // to the gradient of the state before the first token
                float *to = r.fin + size_t(seg.seq) * per_head + size_t(it.h) * kState;
#pragma unroll
                for (int k = 0; k < 64; ++k) {
                    const float x = f == 1.f ? st[k] : f * st[k];
                    if (r.swapped) to[row * kHeadDim + b0 + k] = x;
                    else to[(b0 + k) * kHeadDim + row] = x;
                }
            }
        }
        if (row == 0) tc::bulk_wait_group_all();
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 13) tc::tmem_dealloc(tmem, 512);
}

bool tile_map(CUtensorMap *map, const void *base, int heads, int tokens) {
    return make_tmap_bf16_3d(map, base, 128, uint64_t(heads), uint64_t(tokens), 256, uint64_t(heads) * 256, 64, 1, kC);
}

}  // namespace

cudaError_t launch_tc(const Args &a, cudaStream_t s) {
    Maps m;
    memset(&m, 0, sizeof m);
    if (a.total_tokens > 0)
        for (int i = 0; i < a.roles; ++i) {
            const Role &r = a.role[i];
            if (!tile_map(&m.a[i], r.a, a.hv / r.ga, a.total_tokens) || !tile_map(&m.b[i], r.b, a.hv / r.gb, a.total_tokens) ||
                !tile_map(&m.c[i], r.c, a.hv / r.gc, a.total_tokens) ||
                (!r.partial && !tile_map(&m.o[i], r.out, a.hv, a.total_tokens)))
                return cudaErrorInvalidValue;
        }
    constexpr int kSumBytes = sizeof(SumShared) + 1024, kWalkBytes = sizeof(WalkShared) + 1024;
    static_assert(kSumBytes <= 232448 && kWalkBytes <= 232448, "shared memory of a CTA");
    cudaError_t e = cudaFuncSetAttribute(k_la_sum_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, kSumBytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k_la_walk_tc, cudaFuncAttributeMaxDynamicSharedMemorySize, kWalkBytes);
    if (e != cudaSuccess) return e;
    const unsigned items = unsigned(a.max_segs) * unsigned(a.hv) * unsigned(a.roles);
    if ((e = launch_table(a, s)) != cudaSuccess) return e;
    if (a.seg_len < a.total_tokens) {
        {
            LaunchScope scope(GDN_K_LINATTN_SUM, s);
            k_la_sum_tc<<<items, kSumThreads, kSumBytes, s>>>(a, m);
        }
        if ((e = cudaGetLastError()) != cudaSuccess || (e = launch_chain(a, s)) != cudaSuccess) return e;
    }
    LaunchScope scope(GDN_K_LINATTN_WALK, s);
    k_la_walk_tc<<<items, kWalkThreads, kWalkBytes, s>>>(a, m);
    return cudaGetLastError();
}

}  // namespace la
}  // namespace gdn
