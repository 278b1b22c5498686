// Blocks of floats held as e4m3 (4 exponent bits, 3 mantissa bits, largest value 448) with one
// float32 scale each, shared by the quantiser, the 8-bit product and the 8-bit K/V cache.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace tlb {

constexpr int kFp8Block = 128;      // columns that share a scale

// Whether a pointer is aligned to elements of this many bytes.
inline bool aligned_to(const void *p, size_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// Magnitude of x as an integer that orders as the floats do, NaN above infinity: the largest of a
// block is an integer maximum, which keeps a NaN (a float maximum drops it).
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// The scale of a block whose largest magnitude is `top` (bits): the smallest power of two 2^e,
// e >= -126, with top <= 448 * 2^e, and its reciprocal.  448 = 1.75 * 2^8.  Dividing by a power of
// two is exact, so each value is rounded once.  A block that holds an infinity or a NaN gets the
// scale NaN: all its values are NaN.
__device__ __forceinline__ float block_scale(uint32_t top, float &inv) {
    if (top >= 0x7F800000u) {
        inv = __uint_as_float(0x7FC00000u);
        return inv;
    }
    const int e = max(int(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0), 1);   // 1 .. 247
    inv = __uint_as_float(uint32_t(254 - e) << 23);
    return __uint_as_float(uint32_t(e) << 23);
}

// Two floats to e4m3 (nearest, ties to even; |x| <= 448 here, NaN stays NaN): a in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
    return to_e4m3x2(a, b) | (to_e4m3x2(c, d) << 16);
}

// Two e4m3 values (the low 16 bits of v) as a pair of halves, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t v) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(v));
    return r;
}
// Four e4m3 values as two pairs of halves: the lower two, the upper two.
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t v, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t v) {
    const uint32_t h = e4m3x2_to_half2(v);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Element loads of the two float types that are quantised from and read back to.
template <typename T> __device__ __forceinline__ float load_float(const T *p);
template <> __device__ __forceinline__ float load_float<float>(const float *p) { return __ldg(p); }
template <> __device__ __forceinline__ float load_float<__nv_bfloat16>(const __nv_bfloat16 *p) {
    return __uint_as_float(uint32_t(__ldg(reinterpret_cast<const unsigned short *>(p))) << 16);
}
// Four consecutive elements, aligned to their size.
__device__ __forceinline__ float4 load_float4(const float *p) { return ld_stream(reinterpret_cast<const float4 *>(p)); }
__device__ __forceinline__ float4 load_float4(const __nv_bfloat16 *p) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
}
__device__ __forceinline__ void store_float4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store_float4(__nv_bfloat16 *p, float4 v) {
    *reinterpret_cast<uint2 *>(p) = pack_bf16x4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ void store_float(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_float(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

}  // namespace tlb
