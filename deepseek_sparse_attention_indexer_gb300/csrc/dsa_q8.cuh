// dsa_q8.cuh -- the 8-bit cache row and its conversions, shared by the kernels
// that write, read and attend over it.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "dsa_internal.h"
#include "dsa_ptx.cuh"

namespace dsa {

constexpr int kQ8Row = DSA_Q8_ROW_BYTES;       // 512 e4m3 | 64 bf16
constexpr int kQ8Latent = DSA_V_DIM;           // 512
constexpr int kQ8Rope = DSA_QK_DIM - DSA_V_DIM;  // 64
static_assert(kQ8Row == kQ8Latent + 2 * kQ8Rope, "an 8-bit cache row");

// (lo, hi) -> two e4m3 codes, nearest even, saturating at 448 (NaN stays NaN); lo in the low byte
__device__ __forceinline__ uint16_t pack_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
    return (uint32_t)pack_e4m3x2(a, b) | ((uint32_t)pack_e4m3x2(c, d) << 16);
}
// two e4m3 codes -> their values (every e4m3 number is exact in half precision)
__device__ __forceinline__ float2 unpack_e4m3x2(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Smallest k with amax <= 448 * 2^k, clamped to [-64, 64]; 0 for amax = 0.  448 = 1.75 * 2^8, so k
// is the exponent less 8, and one more where the fraction passes .75: no logarithm, no rounding.
__device__ __forceinline__ int e4m3_scale_exponent(float amax) {
    if (!(amax > 0.f)) return 0;
    const uint32_t b = __float_as_uint(amax);
    const int k = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(-64, min(64, k));
}
__device__ __forceinline__ float exp2_int(int k) { return __uint_as_float((uint32_t)(k + 127) << 23); }

// Four values as hi + lo / 16 in e4m3 (|x| <= 448): the four hi bytes, the four lo bytes.  The half-precision step
// between keeps 11 bits, the difference x - hi is exact.
__device__ __forceinline__ void split_e4m3x4(float x, float y, float z, float w, uint32_t& hi, uint32_t& lo) {
    asm("{\n\t.reg .b32 a, b, p, q;\n\t.reg .b16 s, t;\n\t"
        "cvt.rn.f16x2.f32 a, %3, %2;\n\t"
        "cvt.rn.f16x2.f32 b, %5, %4;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 s, a;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 t, b;\n\t"
        "mov.b32 %0, {s, t};\n\t"
        "cvt.rn.f16x2.e4m3x2 p, s;\n\t"
        "cvt.rn.f16x2.e4m3x2 q, t;\n\t"
        "sub.rn.f16x2 a, a, p;\n\t"
        "sub.rn.f16x2 b, b, q;\n\t"
        "mul.rn.f16x2 a, a, %6;\n\t"
        "mul.rn.f16x2 b, b, %6;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 s, a;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 t, b;\n\t"
        "mov.b32 %1, {s, t};\n\t}\n"
        : "=&r"(hi), "=&r"(lo)
        : "f"(x), "f"(y), "f"(z), "f"(w), "r"(0x4c004c00u));   // 16, twice
}

// Pool row of key j of sequence b, -1 when its page lies outside the pool.
__device__ __forceinline__ int64_t paged_row(const PageTable& pt, int b, int j) {
    const int page = __ldg(pt.table + (int64_t)b * pt.stride + (j >> pt.shift));
    if (page < 0 || page >= pt.num_pages) return -1;
    return ((int64_t)page << pt.shift) + (j & ((1 << pt.shift) - 1));
}

}  // namespace dsa
