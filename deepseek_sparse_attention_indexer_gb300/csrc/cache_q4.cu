// cache_q4.cu -- writing the 4-bit latent cache and reading it back.
//
// Write: u, the normalised latent row, and the turned rope dims as in cache_q8.cu; then
//   s_b = the smallest (1 + m/4) 2^j, m < 3, with max|u| of block b <= 6 s_b;  c = 2^(J - 5), J the largest j of the row
//   block byte = s_b / c (see dsa_q4.cuh; no less than 2^-6), code = u / s_b to the nearest magnitude, ties to the even
// Read: out = bf16(code * block * scale) | k_pe.
// A warp a row, as in cache_q8.cu; both move about 1.6 KB a token.  Writing is bound by the norm's and the codes' instructions
// (4096 rows 5.7 us, a million 0.96 ms: 1.7 TB/s; with the codes counted by seven comparisons 7.1 us, 1.26 ms; the 8-bit rows,
// 0.79), reading by HBM (65,536 rows 19.6 us, a million 0.32 ms: 5.1 TB/s); 8 rows take 2.5 and 1.4 us.
#include <cuda_fp4.h>

#include "dsa_q4.cuh"
#include "latent_row.cuh"

namespace dsa {

namespace {

constexpr int kWarps = 8;   // rows in flight a CTA: one warp a row

// exponent j and fraction m of the smallest (1 + m/4) 2^j >= amax / 6: 6, 7.5 and 9 are 1.5, 1.875 and 1.125 times a
// power of two
__device__ __forceinline__ void block_step(float amax, int& j, int& m) {
    const uint32_t b = __float_as_uint(amax), f = b & 0x7fffffu;
    j = (int)(b >> 23) - 127 - (f <= 0x100000u ? 3 : 2);
    m = f <= 0x100000u ? 2 : f <= 0x400000u ? 0 : f <= 0x700000u ? 1 : 2;
    if (!(amax > 0.f)) j = -1000;
}

// u / step, inv = 1 / step rounded, on the side of every midpoint between two magnitudes, or on it, that u / step is on.
// A midpoint's multiple of the step has at most six significant bits, so u is first rounded to odd at twelve: it is the
// multiple then or 2^-12 of it away.  The product with inv (1, 0.8 (1 + 2^-26) or 2/3 (1 + 2^-25) times a power of two) is
// within 2^-25 of the quotient: nowhere near another midpoint, and where u is the multiple less than half a float's step
// (2^-24 / 1.75) off the midpoint, which it is rounded to.  Zero for -0 and NaN.
__device__ __forceinline__ float quotient(float u, float inv) {
    const uint32_t b = __float_as_uint(u);
    const float v = __uint_as_float((b | ((b & 0xfffu) + 0xfffu)) & ~0xfffu);
    return u == u ? __fmaf_rn(v, inv, 0.f) : 0.f;
}
// The nearest codes of eight numbers, ties to the even one, four bits each, and the signs of four at bits 8 i + 7
__device__ __forceinline__ uint32_t codes(const float* q) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = __nv_cvt_float2_to_fp4x2(make_float2(q[2 * i], q[2 * i + 1]), __NV_E2M1, cudaRoundNearest);
    return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}
__device__ __forceinline__ uint32_t signs(const float* q) {
    const uint32_t a = __byte_perm(__float_as_uint(q[0]), __float_as_uint(q[1]), 0x0073);
    return __byte_perm(a, __byte_perm(__float_as_uint(q[2]), __float_as_uint(q[3]), 0x0073), 0x5410) & 0x80808080u;
}

template <bool INTERLEAVE>
__global__ void __launch_bounds__(kWarps * 32, 4) cache_write_q4_kernel(const CacheWriteParams p) {
    griddep_wait();
    const int r = blockIdx.x * kWarps + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    if (r >= p.R) return;
    int pos;
    const int slot = write_slot(p, r, pos, lane);
    if (slot < 0) return;
    float x[16];
    uint32_t pe;
    normed_row(p, r, lane, x, pe);
    int j[2], m[2];                            // a block is two lanes' eight dims
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[8 * h + i]));
        block_step(fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1)), j[h], m[h]);
    }
    const int k = max(-64, min(64, __reduce_max_sync(0xffffffffu, max(j[0], j[1])) - 5));
    uint8_t* dst = p.cache + (int64_t)slot * kQ4Row;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int a = j[h] - k + 6;
        if (a < 0 || a > 11) m[h] = a < 0 ? 0 : 2;
        a = max(0, min(11, a));
        const float inv = (m[h] == 0 ? 1.f : m[h] == 1 ? 0.8f : 2.f / 3.f) * exp2_int(6 - k - a);
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = quotient(x[8 * h + i], inv);
        reinterpret_cast<uint32_t*>(dst)[32 * h + lane] =
            (codes(q) & kQ4Magnitudes) | signs(q) | signs(q + 4) >> 4;
        if ((lane & 1) == 0) dst[kQ4Codes + 16 * h + lane / 2] = (uint8_t)(3 * a + m[h]);
    }
    reinterpret_cast<uint32_t*>(dst + kQ4Rope)[lane] =
        turned_rope<INTERLEAVE>(pe, p.cos_sin + (int64_t)pos * kQ8Rope, lane);
    if (lane == 0) p.scale[slot] = exp2_int(k);
}

// One warp a row: lane l widens block l and copies rope dims 2l, 2l+1.
__device__ __forceinline__ void read_row(const uint8_t* cache, const float* scale, int64_t row, __nv_bfloat16* dst,
                                         int lane) {
    uint32_t o[8], pe = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = 0;
    if (row >= 0) {
        const uint8_t* src = cache + row * kQ4Row;
        const uint2 c = __ldg(reinterpret_cast<const uint2*>(src) + lane);
        const uint32_t b = __ldg(src + kQ4Codes + lane);
        pe = __ldg(reinterpret_cast<const uint32_t*>(src + kQ4Rope) + lane);
        const float s = __ldg(scale + row);
        if (b < kQ4Scales) {
            const float f = q4_block_scale(b);
            const uint2 unit = make_uint2(0x3c383000u, 0x4c484440u);   // the magnitudes as e4m3
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint2 v = q4_expand(h ? c.y : c.x, unit);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 t = unpack_e4m3x2((i < 2 ? v.x : v.y) >> (16 * (i & 1)) & 0xffffu);
                    o[4 * h + i] = pack_bf16x2(t.x * f * s, t.y * f * s);   // t f is exact
                }
            }
        }
    }
    uint4* d = reinterpret_cast<uint4*>(dst + 16 * lane);
    d[0] = make_uint4(o[0], o[1], o[2], o[3]);
    d[1] = make_uint4(o[4], o[5], o[6], o[7]);
    reinterpret_cast<uint32_t*>(dst + kQ8Latent)[lane] = pe;
}

__global__ void __launch_bounds__(kWarps * 32)
    cache_read_q4_kernel(const uint8_t* cache, const float* scale, int cache_rows, const int32_t* slots, int R,
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
    cache_read_q4_paged_kernel(const uint8_t* cache, const float* scale, const int32_t* kv_len, int Nmax, int B,
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

// One warp a row: lane l expands block l to 16 e4m3 bytes and copies rope dims 2l, 2l+1: row j of the 8-bit cache.
__global__ void __launch_bounds__(kWarps * 32)
    cache_expand_q4_kernel(const uint8_t* cache, const float* scale, int N, uint8_t* out, float* out_scale,
                           const PageTable pt) {
    griddep_wait();
    const int j = blockIdx.x * kWarps + threadIdx.x / 32;
    const int lane = threadIdx.x & 31;
    if (j >= N) return;
    const int64_t row = pt.table ? paged_row(pt, 0, j) : j;
    if (row < 0) return;                       // a page outside the pool: the attention does not read its rows
    const uint8_t* src = cache + row * kQ4Row;
    uint8_t* dst = out + (int64_t)j * kQ8Row;
    const uint2 c = __ldg(reinterpret_cast<const uint2*>(src) + lane);
    const uint32_t b = __ldg(src + kQ4Codes + lane);
    const uint32_t pe = __ldg(reinterpret_cast<const uint32_t*>(src + kQ4Rope) + lane);
    const float s = __ldg(scale + row);
    const uint2 t = b < kQ4Scales ? q4_table(q4_block_scale(b)) : make_uint2(0, 0);
    const uint2 x = q4_expand(c.x, t), y = q4_expand(c.y, t);
    reinterpret_cast<uint4*>(dst)[lane] = make_uint4(x.x, x.y, y.x, y.y);
    reinterpret_cast<uint32_t*>(dst + kQ8Latent)[lane] = pe;
    if (lane == 0) out_scale[j] = s;
}

}  // namespace

dsa_status_t launch_cache_expand_q4(const void* cache, const float* cache_scale, int N, void* out, float* out_scale,
                                    const PageTable& pages, cudaStream_t stream) {
    if (launch_pdl(cache_expand_q4_kernel, dim3(ceil_div(N, kWarps)), dim3(kWarps * 32), 0, stream,
                   static_cast<const uint8_t*>(cache), cache_scale, N, static_cast<uint8_t*>(out), out_scale,
                   pages) != cudaSuccess)
        return DSA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

dsa_status_t launch_cache_write_q4(const void* kv_a, int64_t kv_a_stride, const float* norm_w, float eps,
                                   const float* cos_sin, int max_pos, int interleave, const int32_t* pos,
                                   const int32_t* slots, int R, void* cache, float* cache_scale, int cache_rows,
                                   cudaStream_t stream) {
    const CacheWriteParams p{static_cast<const __nv_bfloat16*>(kv_a), kv_a_stride, norm_w, eps, cos_sin, max_pos, pos,
                             slots, R, static_cast<uint8_t*>(cache), cache_scale, cache_rows, device_status_ptr()};
    auto kern = interleave ? cache_write_q4_kernel<true> : cache_write_q4_kernel<false>;
    if (launch_pdl(kern, dim3(ceil_div(R, kWarps)), dim3(kWarps * 32), 0, stream, p) != cudaSuccess)
        return DSA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

dsa_status_t launch_cache_read_q4(const void* cache, const float* cache_scale, int cache_rows, const int32_t* slots,
                                  int R, void* out, cudaStream_t stream) {
    if (launch_pdl(cache_read_q4_kernel, dim3(ceil_div(R, kWarps)), dim3(kWarps * 32), 0, stream,
                   static_cast<const uint8_t*>(cache), cache_scale, cache_rows, slots, R,
                   static_cast<__nv_bfloat16*>(out), device_status_ptr()) != cudaSuccess)
        return DSA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

dsa_status_t launch_cache_read_q4_paged(const void* cache, const float* cache_scale, const int32_t* kv_len, int B,
                                        int Nmax, void* out, const PageTable& pages, cudaStream_t stream) {
    const dim3 grid(ceil_div(Nmax, kWarps), B < 65535 ? B : 65535);
    if (launch_pdl(cache_read_q4_paged_kernel, grid, dim3(kWarps * 32), 0, stream, static_cast<const uint8_t*>(cache),
                   cache_scale, kv_len, Nmax, B, static_cast<__nv_bfloat16*>(out), pages,
                   device_status_ptr()) != cudaSuccess)
        return DSA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
