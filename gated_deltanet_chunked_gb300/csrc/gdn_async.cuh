// Rows of NT tensors on their way to a thread's own place in shared memory
// (cp.async, 16 bytes each): kAhead rows ahead of the one in work, so that the
// bytes in flight do not depend on how long a row's reductions take and cost
// no registers. A thread reads only what it copied itself, so no barrier is
// involved: it waits for its own copies.
#pragma once

#include "gdn_vec.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace vec {

template <int NT, int NV>
struct RowsAhead {
    // rows in shared memory: 48 to 128 bytes of a thread in flight
    static constexpr int kStages = NT * NV >= 8 ? 2 : NT * NV >= 3 ? 3 : 4;
    static constexpr int kAhead = kStages - 1;
    static __host__ __device__ size_t smem(int threads) { return size_t(kStages) * NT * NV * 16 * threads; }

    // [kStages][NT * NV][threads] vectors, addresses in the shared window
    uint32_t base, pitch, put, got;
    __device__ __forceinline__ explicit RowsAhead(void *smem)
        : base(tc::smem_u32(smem) + threadIdx.x * 16), pitch(blockDim.x * 16), put(base), got(base) {}
    __device__ __forceinline__ void copy(int v, const void *from) const {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(put + v * pitch), "l"(from) : "memory");
    }
    // only the first `bytes` (1 to 16), zeros after them
    __device__ __forceinline__ void copy_part(int v, const void *from, int bytes) const {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(put + v * pitch), "l"(from), "r"(bytes)
                     : "memory");
    }
    __device__ __forceinline__ void advance(uint32_t &at) const {
        at += NT * NV * pitch;
        if (at == base + kStages * NT * NV * pitch) at = base;
    }
    // ends a row's copies; every row has one, copies or not
    __device__ __forceinline__ void commit() {
        asm volatile("cp.async.commit_group;" ::: "memory");
        advance(put);
    }
    // the oldest row's copies have landed
    __device__ __forceinline__ void wait() const { asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory"); }
    __device__ __forceinline__ uint4 take(int v) const {
        uint4 r;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                     : "r"(got + v * pitch)
                     : "memory");
        return r;
    }
    __device__ __forceinline__ void taken() { advance(got); }
};

}  // namespace vec
}  // namespace gdn
