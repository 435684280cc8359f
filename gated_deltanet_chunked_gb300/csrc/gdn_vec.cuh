// Vectors of VE consecutive elements of one row (4 to 16 bytes) between
// memory and f32 registers, for the row-wise kernels (norms and their
// backward passes) and the recurrence's decode step.
#pragma once

#include <type_traits>

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
    // elements 2 k and 2 k + 1
    __device__ __forceinline__ float2 f2(int k) const { return pair_f(reinterpret_cast<const Pair *>(e)[k]); }
    __device__ __forceinline__ void set2(int k, float2 v) { reinterpret_cast<Pair *>(e)[k] = pair_t(v); }

  private:
    using Pair = typename std::conditional<sizeof(T) == 2, __nv_bfloat162, float2>::type;
    static __device__ __forceinline__ float2 pair_f(float2 v) { return v; }
    static __device__ __forceinline__ float2 pair_f(__nv_bfloat162 v) { return __bfloat1622float2(v); }
    static __device__ __forceinline__ Pair pair_t(float2 v) {
        if constexpr (sizeof(T) == 2) return __floats2bfloat162_rn(v.x, v.y);
        else return v;
    }
};

// Packed f32 arithmetic, two values an instruction (each as the scalar one
// rounds): these kernels are as much bound by instructions as by memory.
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float sum2(float2 v) { return __fadd_rn(v.x, v.y); }

// exp of two values on the base-2 unit: with y = v log2 e rounded and r what
// the rounding left, exp v = 2^y (1 + r ln 2), so that the only errors are
// the unit's (2 steps) and one rounding. v is at most 88; below -200 (and at
// -inf, where r would be NaN) the result is the same zero.
__device__ __forceinline__ float2 exp2_of(float2 v) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(v.x) : "f"(-200.f));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(v.y) : "f"(-200.f));
    const float2 l = both(1.4426950408889634f);
    const float2 y = mul2(v, l);
    const float2 r = mul2(fma2(v, l, make_float2(-y.x, -y.y)), both(0.6931471805599453f));
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(y.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(y.y));
    return fma2(e, r, e);
}

// exp of two values to within a rounding of the last product: with n the
// integer next to v log2 e, exp v = 2^n exp r for r = v - n ln 2 (ln 2 in two
// parts, the first short enough that n times it is exact: the reduction of
// Cody and Waite), |r| <= 0.35, where exp's Taylor polynomial of degree 7 is off
// by 5e-9; 2^n is exact on the base-2 unit. NaN and underflow as exp2_of.
__device__ __forceinline__ float2 exp_exact2(float2 v) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(v.x) : "f"(-200.f));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(v.y) : "f"(-200.f));
    const float big = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
    const float2 n = add2(fma2(v, both(1.4426950408889634f), both(big)), both(-big));
    const float ln2_hi = 0.693145751953125f, ln2_lo = 1.4286068203094173e-06f;  // 16 bits of ln 2, and the rest
    const float2 r = fma2(n, both(-ln2_lo), fma2(n, both(-ln2_hi), v));
    float2 p = fma2(r, both(1.f / 5040.f), both(1.f / 720.f));
    p = fma2(p, r, both(1.f / 120.f));
    p = fma2(p, r, both(1.f / 24.f));
    p = fma2(p, r, both(1.f / 6.f));
    p = fma2(p, r, both(0.5f));
    p = fma2(p, r, both(1.f));
    p = fma2(p, r, both(1.f));
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(n.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(n.y));
    return mul2(e, p);
}

// 1 / (1 + exp(-z)) of two values: below -88 as at -88 (less than the
// smallest normal number)
__device__ __forceinline__ float2 sigmoid2(float2 z) {
    float2 v = make_float2(-z.x, -z.y), s;
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(v.x) : "f"(88.f));
    asm("min.NaN.f32 %0, %0, %1;" : "+f"(v.y) : "f"(88.f));
    v = add2(exp2_of(v), both(1.f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(v.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(v.y));
    return s;
}

// sum over the G lanes (a power of two, lane-aligned) of each group of a warp
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int m = G / 2; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// two such sums: after the first step half of the lanes go on with either
template <int G>
__device__ __forceinline__ float2 group_sum2(float a, float b) {
    const bool up = threadIdx.x & (G / 2);
    const float send = up ? a : b;
    float v = (up ? b : a) + __shfl_xor_sync(0xffffffffu, send, G / 2);
#pragma unroll
    for (int m = G / 4; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    const float o = __shfl_xor_sync(0xffffffffu, v, G / 2);
    return up ? make_float2(o, v) : make_float2(v, o);
}

// sum over the CTA (blockDim.x a multiple of 32); every thread gets it. `buf`
// holds 32 floats (pairs), 16-byte aligned and zero where no warp writes; calls
// in turn use two buffers alternately, so that one barrier a call is enough. The warps' sums are read by every
// thread, four at a time: fewer instructions than a second round of shuffles.
__device__ __forceinline__ float block_sum(float v, float *buf) {
    v = group_sum<32>(v);
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float4 s = *reinterpret_cast<const float4 *>(buf);
    for (int w = 4; w < warps; w += 4) {
        const float4 t = *reinterpret_cast<const float4 *>(buf + w);
        s.x += t.x, s.y += t.y, s.z += t.z, s.w += t.w;
    }
    return (s.x + s.y) + (s.z + s.w);
}

__device__ __forceinline__ float2 block_sum2(float a, float b, float2 *buf) {
    const float2 v = group_sum2<32>(a, b);
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float4 s = *reinterpret_cast<const float4 *>(buf);
    for (int w = 2; w < warps; w += 2) {
        const float4 t = *reinterpret_cast<const float4 *>(buf + w);
        s.x += t.x, s.y += t.y, s.z += t.z, s.w += t.w;
    }
    return make_float2(s.x + s.z, s.y + s.w);
}

}  // namespace vec

// Sums `parts` rows of partial sums [parts, width] in a fixed order: a -> out_a
// and b -> out_b (either output may be null). `parts` 0 writes zeros.
cudaError_t launch_row_sums(const float *a, const float *b, int parts, int width, float *out_a, float *out_b,
                            cudaStream_t s);

}  // namespace gdn
