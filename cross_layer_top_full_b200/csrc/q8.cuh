// q8.cuh -- the row format of the quantised cache (include/indexcache.h) and
// its arithmetic, shared by the kernels that write, read and attend over it.
#pragma once

#include "common.cuh"

namespace ic {
namespace q8 {

constexpr int ROW = IC_Q8_ROW_BYTES;   // bytes of a latent row
constexpr int DV = 512;                // quantised columns (the values)
constexpr int DR = 64;                 // columns kept as bfloat16, divided by the scale
constexpr int KVW = DV + DR;
constexpr int DI = 128;                // an indexer key
constexpr int OFF_ROPE = DV;
static_assert(OFF_ROPE + 2 * DR == ROW && ROW % 128 == 0, "row format");

// Bits of |x| where x is finite, else 0: what a row's maximum is taken of
// (non-negative floats order like their bits).
__device__ __forceinline__ uint32_t finite_abs_bits(float x) {
    const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
    return u < 0x7f800000u ? u : 0u;
}

// Exponent e of a row's scale 2^e: the smallest with max <= 448 * 2^e, at
// least -32; 0 for a row of zeros.  448 = 1.75 * 2^8, so with max = m * 2^E,
// m in [1, 2): e = E - 8 for m <= 1.75, else E - 7.
__device__ __forceinline__ int scale_exponent(uint32_t max_bits) {
    if (max_bits == 0) return 0;
    const int e = (int)(max_bits >> 23) - 127 - 8 + ((max_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e > -32 ? e : -32;
}

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Two codes: x * inv (exact, inv a power of two) rounded to the nearest e4m3
// value, ties to even, saturating at 448; the first in the low byte.
__device__ __forceinline__ uint32_t encode2(float a, float b, float inv) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a * inv, b * inv), __NV_SATFINITE, __NV_E4M3);
}

// Two codes (low byte first) as floats.
__device__ __forceinline__ float2 decode2(uint32_t codes) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xffffu), __NV_E4M3);
    return __half22float2(__half2(h));
}

}  // namespace q8
}  // namespace ic
