// Vectors of VE consecutive elements of one row (2 to 16 bytes) between
// memory and f32 registers, for the row-wise kernels (norms and their
// backward passes) and the recurrence's decode step.
#pragma once

#include "gdn_common.cuh"

namespace gdn {
namespace vec {

template <int BYTES>
struct Raw;
template <>
struct Raw<16> { using type = uint4; };
template <>
struct Raw<8> { using type = uint2; };
template <>
struct Raw<4> { using type = uint32_t; };
template <>
struct Raw<2> { using type = uint16_t; };

// VE elements of T as they lie in memory
template <typename T, int VE>
struct Pack {
    using raw = typename Raw<int(sizeof(T)) * VE>::type;
    union {
        raw r;
        T e[VE];
    };
    __device__ __forceinline__ Pack() {}
    __device__ __forceinline__ void load(const T *p) { r = *reinterpret_cast<const raw *>(p); }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<raw *>(p) = r; }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < VE; ++i) e[i] = from_f32<T>(0.f);
    }
    __device__ __forceinline__ float f(int i) const { return to_f32<T>(e[i]); }
    __device__ __forceinline__ void set(int i, float v) { e[i] = from_f32<T>(v); }
};

// sum over the G lanes (a power of two, lane-aligned) of each group of a warp
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int m = G / 2; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// sum over the CTA (blockDim.x a multiple of 32); every thread gets it. `buf`
// holds 32 floats; calls in turn use two buffers alternately, so that one
// barrier a call is enough.
__device__ __forceinline__ float block_sum(float v, float *buf) {
    v = group_sum<32>(v);
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    return group_sum<32>(lane < warps ? buf[lane] : 0.f);
}

__device__ __forceinline__ float2 block_sum2(float a, float b, float2 *buf) {
    a = group_sum<32>(a);
    b = group_sum<32>(b);
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) buf[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    const float2 t = lane < warps ? buf[lane] : make_float2(0.f, 0.f);
    return make_float2(group_sum<32>(t.x), group_sum<32>(t.y));
}

}  // namespace vec

// Sums `parts` rows of partial sums [parts, width] in a fixed order: a -> out_a
// and b -> out_b (either output may be null). `parts` 0 writes zeros.
cudaError_t launch_row_sums(const float *a, const float *b, int parts, int width, float *out_a, float *out_b,
                            cudaStream_t s);

}  // namespace gdn
