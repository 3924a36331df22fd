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
// latent_row.cuh; 3.0 us with float32 alone).  8 rows take 2.5 us, the host 9 us for the call.
#include "latent_row.cuh"

namespace dsa {

namespace {

constexpr int kWarps = 8;   // rows in flight a CTA: one warp a row

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

template <bool INTERLEAVE>
__global__ void __launch_bounds__(kWarps * 32, 4) cache_write_q8_kernel(const CacheWriteParams p) {
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
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
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
    reinterpret_cast<uint32_t*>(dst + kQ8Latent)[lane] =
        turned_rope<INTERLEAVE>(pe, p.cos_sin + (int64_t)pos * kQ8Rope, lane);
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
    const CacheWriteParams p{static_cast<const __nv_bfloat16*>(kv_a), kv_a_stride, norm_w, eps, cos_sin, max_pos, pos,
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
