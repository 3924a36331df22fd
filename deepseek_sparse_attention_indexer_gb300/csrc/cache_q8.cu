// cache_q8.cu -- writing the 8-bit latent cache and reading it back.
//
// Write (SlimServe "GLM52_PIPELINE_TRACE.md", section 4: the projection's 576
// outputs split into kv_cmpr 512 | k_pe 64, k_pe rotated, kv_cmpr
// RMS-normalised), with the quantisation of this library's cache row:
//   u = c * rsqrt(mean(c^2) + eps) * w,  2^k >= max|u| / 448,  row = e4m3(u 2^-k) | bf16(turned k_pe)
// Read: out = bf16(e4m3 * scale) | k_pe.
// Both move about 1.8 KB a token: a warp a row, every load and store of it one contiguous span.  Reading is bound by HBM
// (65,536 rows 20.8 us: 118 MB, 5.7 TB/s; eight uneven contexts of up to 4096 rows through their pages 6.0 us).  Writing
// 4096 rows takes 4.7 us (7.9 MB, 1.7 TB/s): a launch's start, one wave of loads and the norm in pairs of floats (see
// Two; 3.0 us with float32 alone).  8 rows take 2.5 us, the host 9 us for the call.
#include "dsa_q8.cuh"

namespace dsa {

namespace {

constexpr int kWarps = 8;   // rows in flight a CTA: one warp a row

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

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

struct WriteParams {
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

// One warp a row: lane l holds latent dims 8l..8l+7 and 256+8l..256+8l+7 and rope dims 2l, 2l+1,
// so that every load and store of the warp is one contiguous span.
template <bool INTERLEAVE>
__global__ void __launch_bounds__(kWarps * 32, 4) cache_write_q8_kernel(const WriteParams p) {
    griddep_wait();
    const int r = blockIdx.x * kWarps + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    if (r >= p.R) return;
    const int slot = __ldg(p.slots + r);
    if (slot < 0) return;
    const int pos = __ldg(p.pos + r);
    if (slot >= p.cache_rows || pos < 0 || pos >= p.max_pos) {
        if (lane == 0) raise_dev_error(p.status, DEV_ERR_BOUNDS);
        return;
    }
    const __nv_bfloat16* src = p.kv_a + (int64_t)r * p.stride;
    uint4 raw[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) raw[h] = ldg_nc_v4(src + 256 * h + 8 * lane);
    const uint32_t pe = __ldg(reinterpret_cast<const uint32_t*>(src + kQ8Latent) + lane);
    const float* cs = p.cos_sin + (int64_t)pos * kQ8Rope;

    float x[16], top = 0.f;
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
    float amax = 0.f;
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
            amax = fmaxf(amax, fmaxf(fmaxf(fabsf(y[0]), fabsf(y[1])), fmaxf(fabsf(y[2]), fabsf(y[3]))));
        }
    const int k = e4m3_scale_exponent(warp_max(amax));
    const float inv = exp2_int(-k);
    uint8_t* dst = p.cache + (int64_t)slot * kQ8Row;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float* y = x + 8 * h;
        *reinterpret_cast<uint2*>(dst + 256 * h + 8 * lane) =
            make_uint2(pack_e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                       pack_e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv));
    }
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
    reinterpret_cast<uint32_t*>(dst + kQ8Latent)[lane] = pack_bf16x2(a, b);
    if (lane == 0) p.scale[slot] = exp2_int(k);
}

// One warp a row: lane l widens latent dims 16l..16l+15 and copies rope dims 2l, 2l+1.
__device__ __forceinline__ void read_row(const uint8_t* cache, const float* scale, int64_t row, __nv_bfloat16* dst,
                                         int lane) {
    uint32_t o[8], pe = 0;
    if (row >= 0) {
        const uint8_t* src = cache + row * kQ8Row;
        const uint4 c = ldg_nc_v4(src + 16 * lane);
        pe = __ldg(reinterpret_cast<const uint32_t*>(src + kQ8Latent) + lane);
        const float s = __ldg(scale + row);
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 lo = unpack_e4m3x2(w[i] & 0xffffu), hi = unpack_e4m3x2(w[i] >> 16);
            o[2 * i] = pack_bf16x2(lo.x * s, lo.y * s);
            o[2 * i + 1] = pack_bf16x2(hi.x * s, hi.y * s);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = 0;
    }
    uint4* d = reinterpret_cast<uint4*>(dst + 16 * lane);
    d[0] = make_uint4(o[0], o[1], o[2], o[3]);
    d[1] = make_uint4(o[4], o[5], o[6], o[7]);
    reinterpret_cast<uint32_t*>(dst + kQ8Latent)[lane] = pe;
}

__global__ void __launch_bounds__(kWarps * 32)
    cache_read_q8_kernel(const uint8_t* cache, const float* scale, int cache_rows, const int32_t* slots, int R,
                         __nv_bfloat16* out, int32_t* status) {
    griddep_wait();
    const int r = blockIdx.x * kWarps + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    if (r >= R) return;
    int64_t row = __ldg(slots + r);
    if (row >= cache_rows) {
        if (lane == 0) raise_dev_error(status, DEV_ERR_BOUNDS);
        row = -1;
    }
    read_row(cache, scale, row, out + (int64_t)r * DSA_QK_DIM, lane);
}

__global__ void __launch_bounds__(kWarps * 32)
    cache_read_q8_paged_kernel(const uint8_t* cache, const float* scale, const int32_t* kv_len, int Nmax, int B,
                               __nv_bfloat16* out, const PageTable pt, int32_t* status) {
    griddep_wait();
    const int j = blockIdx.x * kWarps + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    for (int b = blockIdx.y; b < B; b += gridDim.y) {
        if (j >= min(__ldg(kv_len + b), Nmax)) continue;
        const int64_t row = paged_row(pt, b, j);
        if (row < 0 && lane == 0) raise_dev_error(status, DEV_ERR_BOUNDS);
        read_row(cache, scale, row, out + ((int64_t)b * Nmax + j) * DSA_QK_DIM, lane);
    }
}

}  // namespace

dsa_status_t launch_cache_write_q8(const void* kv_a, int64_t kv_a_stride, const float* norm_w, float eps,
                                   const float* cos_sin, int max_pos, int interleave, const int32_t* pos,
                                   const int32_t* slots, int R, void* cache, float* cache_scale, int cache_rows,
                                   cudaStream_t stream) {
    const WriteParams p{static_cast<const __nv_bfloat16*>(kv_a), kv_a_stride, norm_w, eps, cos_sin, max_pos, pos,
                        slots, R, static_cast<uint8_t*>(cache), cache_scale, cache_rows, device_status_ptr()};
    auto kern = interleave ? cache_write_q8_kernel<true> : cache_write_q8_kernel<false>;
    if (launch_pdl(kern, dim3(ceil_div(R, kWarps)), dim3(kWarps * 32), 0, stream, p) != cudaSuccess)
        return DSA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

dsa_status_t launch_cache_read_q8(const void* cache, const float* cache_scale, int cache_rows, const int32_t* slots,
                                  int R, void* out, cudaStream_t stream) {
    if (launch_pdl(cache_read_q8_kernel, dim3(ceil_div(R, kWarps)), dim3(kWarps * 32), 0, stream,
                   static_cast<const uint8_t*>(cache), cache_scale, cache_rows, slots, R,
                   static_cast<__nv_bfloat16*>(out), device_status_ptr()) != cudaSuccess)
        return DSA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

dsa_status_t launch_cache_read_q8_paged(const void* cache, const float* cache_scale, const int32_t* kv_len, int B,
                                        int Nmax, void* out, const PageTable& pages, cudaStream_t stream) {
    const dim3 grid(ceil_div(Nmax, kWarps), B < 65535 ? B : 65535);
    if (launch_pdl(cache_read_q8_paged_kernel, grid, dim3(kWarps * 32), 0, stream, static_cast<const uint8_t*>(cache),
                   cache_scale, kv_len, Nmax, B, static_cast<__nv_bfloat16*>(out), pages,
                   device_status_ptr()) != cudaSuccess)
        return DSA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
