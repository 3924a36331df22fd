// latent_row.cuh -- a new token's latent row from its projection, shared by the
// kernels that write the 8-bit and the 4-bit cache: RMS norm of the 512 latent
// dims, rotation of the 64 rope dims, one warp a row.
#pragma once
#include "dsa_q8.cuh"

namespace dsa {

// The latent dims are computed as unevaluated sums of two floats (Knuth's two-sum, products' errors by fma), about
// 2^-44 relative: a code is then the nearest of the formula's value, not of a float32 chain's, and does not hang on
// the order of a sum.  In float32 alone a few codes in a million fall on the other side of a midpoint.
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two add(Two a, Two b) {
    const Two s = two_sum(a.hi, b.hi);
    return two_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
// 1 / sqrt(x): one Newton step from the unit's value, its residual 1 - x r^2 without cancellation
__device__ __forceinline__ Two two_rsqrt(Two x) {
    const float r = rsqrtf(x.hi);
    const float t = __fmul_rn(r, r), tl = __fmaf_rn(r, r, -t);
    const float p = __fmul_rn(x.hi, t), pl = __fmaf_rn(x.hi, t, -p);
    const float e = __fsub_rn(__fsub_rn(__fsub_rn(1.f, p), pl), __fmaf_rn(x.hi, tl, __fmul_rn(x.lo, t)));
    return {r, __fmul_rn(__fmul_rn(0.5f, r), e)};
}
// c * r * w as one float rounded to odd: the float below it in magnitude with its last bit set unless the value is
// a float, so that rounding it once more to fewer bits, or comparing it, is as rounding or comparing the value
__device__ __forceinline__ float scaled_to_odd(float c, Two r, float w) {
    const float a = __fmul_rn(c, r.hi), al = __fmaf_rn(c, r.lo, __fmaf_rn(c, r.hi, -a));
    const float u = __fmul_rn(a, w), ul = __fmaf_rn(al, w, __fmaf_rn(a, w, -u));
    const float s = __fadd_rn(u, ul), t = __fsub_rn(ul, __fsub_rn(s, u));
    uint32_t b = __float_as_uint(s);
    if (fabsf(t) > 0.f) b = (b - ((__float_as_uint(t) ^ b) >> 31)) | 1u;
    return fabsf(u) < INFINITY ? __uint_as_float(b) : u;
}

// A row and eps far from 1 are taken at 2^-e and 2^-2e times their size, which leaves the quotient as it is, so that
// neither a sum of squares nor 1 / sqrt leaves float32's range.  0 where the larger of the row's top and sqrt(eps) lies
// within 2^-40 .. 2^40: their squares and 2^-80 of them are floats.
__device__ __forceinline__ int range_exponent(float top, float eps) {
    const float m = fmaxf(top, sqrtf(eps));
    if (m >= 0x1p-40f && m <= 0x1p40f) return 0;
    return max(-126, min(126, (int)(__float_as_uint(m) >> 23) - 127));
}

// Arguments of a write: R tokens to rows of a cache (include/dsa.h).
struct CacheWriteParams {
    const __nv_bfloat16* kv_a;
    int64_t stride;
    const float* norm_w;
    float eps;
    const float* cos_sin;
    int max_pos;
    const int32_t* pos;
    const int32_t* slots;
    int R;
    uint8_t* cache;
    float* scale;
    int cache_rows;
    int32_t* status;
};

// The token's slot, -1 where it is left out: padding, or out of range (recorded).
__device__ __forceinline__ int write_slot(const CacheWriteParams& p, int r, int& pos, int lane) {
    const int slot = __ldg(p.slots + r);
    if (slot < 0) return -1;
    pos = __ldg(p.pos + r);
    if (slot < p.cache_rows && pos >= 0 && pos < p.max_pos) return slot;
    if (lane == 0) raise_dev_error(p.status, DEV_ERR_BOUNDS);
    return -1;
}

// x[0..7]: latent dims 8l..8l+7, x[8..15]: 256+8l..256+8l+7 of lane l, so that every load of the warp is one contiguous
// span; normalised and rounded to odd.  pe: rope dims 2l, 2l + 1 as they are.
__device__ __forceinline__ void normed_row(const CacheWriteParams& p, int r, int lane, float (&x)[16], uint32_t& pe) {
    const __nv_bfloat16* src = p.kv_a + (int64_t)r * p.stride;
    uint4 raw[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) raw[h] = ldg_nc_v4(src + 256 * h + 8 * lane);
    pe = __ldg(reinterpret_cast<const uint32_t*>(src + kQ8Latent) + lane);

    float top = 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t w[4] = {raw[h].x, raw[h].y, raw[h].z, raw[h].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[8 * h + 2 * i] = bf16_lo(w[i]);
            x[8 * h + 2 * i + 1] = bf16_hi(w[i]);
            top = fmaxf(top, fmaxf(fabsf(x[8 * h + 2 * i]), fabsf(x[8 * h + 2 * i + 1])));
        }
    }
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));   // magnitudes compare as their bits
    float eps = p.eps;
    const int e = range_exponent(top, eps);
    if (e != 0) {
        const float f = exp2_int(-e);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] *= f;
        eps = eps * f * f;
        if (top == 0.f) eps = 1.f;            // zeros, also over eps = 0
    }
    Two ss{0.f, 0.f};                         // a bf16 number's square is a float
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const Two s = two_sum(ss.hi, __fmul_rn(x[i], x[i]));
        ss = {s.hi, __fadd_rn(ss.lo, s.lo)};
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        ss = add(ss, {__shfl_xor_sync(0xffffffffu, ss.hi, o), __shfl_xor_sync(0xffffffffu, ss.lo, o)});
    const Two rstd = two_rsqrt(add({ss.hi * (1.f / kQ8Latent), ss.lo * (1.f / kQ8Latent)}, {eps, 0.f}));
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 w = __ldg(reinterpret_cast<const float4*>(p.norm_w + 256 * h + 8 * lane) + i);
            float* y = x + 8 * h + 4 * i;
            y[0] = scaled_to_odd(y[0], rstd, w.x);
            y[1] = scaled_to_odd(y[1], rstd, w.y);
            y[2] = scaled_to_odd(y[2], rstd, w.z);
            y[3] = scaled_to_odd(y[3], rstd, w.w);
        }
}

// Rope dims 2l, 2l + 1 of lane l turned by their pairs' angles (cs: 32 cosines | 32 sines), as two bf16.
template <bool INTERLEAVE>
__device__ __forceinline__ uint32_t turned_rope(uint32_t pe, const float* cs, int lane) {
    float a = bf16_lo(pe), b = bf16_hi(pe);   // rope dims 2l, 2l + 1
    if (INTERLEAVE) {                         // the pair itself
        const float c = __ldg(cs + lane), s = __ldg(cs + 32 + lane);
        const float u = a * c - b * s, v = b * c + a * s;
        a = u;
        b = v;
    } else {                                  // dims 2l, 2l + 1 pair with those of lane l ^ 16
        const int i = 2 * (lane & 15);
        const float2 c = __ldg(reinterpret_cast<const float2*>(cs + i));
        const float2 s = __ldg(reinterpret_cast<const float2*>(cs + 32 + i));
        const float a2 = __shfl_xor_sync(0xffffffffu, a, 16), b2 = __shfl_xor_sync(0xffffffffu, b, 16);
        const float sign = lane < 16 ? -1.f : 1.f;
        a = a * c.x + sign * (a2 * s.x);
        b = b * c.y + sign * (b2 * s.y);
    }
    return pack_bf16x2(a, b);
}

}  // namespace dsa
