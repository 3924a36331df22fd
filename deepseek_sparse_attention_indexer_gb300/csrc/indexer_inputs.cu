// indexer_inputs.cu -- the indexer's queries and keys from their projections:
// norm of each 128-wide head, rotation of its first 64 dims, and the scatter of
// the keys to their cache, in one pass (SlimServe "GLM52_PIPELINE_TRACE.md",
// section 5: indexer_rope_interleave).
//   y = (x - [mean]) * rsqrt(mean((x - [mean])^2) + eps) * w + b,
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin) for the 32 pairs of dims 0..63
// 16.9 KB a token in and out, a few operations an element.
#include "dsa_q8.cuh"

namespace dsa {

namespace {

constexpr int kThreads = 256;
constexpr int kHeadsPerToken = DSA_INDEXER_HEADS + 1;   // 32 query heads, then the key
constexpr int kD = DSA_INDEXER_DIM;

struct NormRopeParams {
    const __nv_bfloat16 *q, *k;
    int64_t q_stride, k_stride;
    const float *q_w, *q_b, *k_w, *k_b;
    float eps;
    const float* cos_sin;
    int max_pos;
    const int32_t *pos, *slots;
    int units;              // R * 33
    __nv_bfloat16 *q_out, *k_cache;
    int cache_rows;
    int32_t* status;
};

// Sum over the 16 lanes of a half warp.
__device__ __forceinline__ float half_sum(float x) {
#pragma unroll
    for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__device__ __forceinline__ void load8(const float* w, float (&v)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(w)), b = __ldg(reinterpret_cast<const float4*>(w) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Half a warp a head: lane l of it holds dims 8l..8l+7 (16 bytes).  Lanes 0..7 hold the turned dims.
// Every lane of a warp takes part in the shuffles; a half warp without work stores nothing.
template <bool LAYER, bool INTERLEAVE>
__global__ void __launch_bounds__(kThreads) indexer_norm_rope_kernel(const NormRopeParams p) {
    griddep_wait();
    const int unit = blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4);
    const int l = threadIdx.x & 15;
    const int token = unit / kHeadsPerToken, h = unit % kHeadsPerToken;
    const bool is_k = h == DSA_INDEXER_HEADS;
    bool live = unit < p.units;
    int pos = 0, slot = 0;
    if (live) {
        pos = __ldg(p.pos + token);
        if (is_k) slot = __ldg(p.slots + token);
        if (pos < 0 || pos >= p.max_pos || slot >= p.cache_rows) {
            if (l == 0) raise_dev_error(p.status, DEV_ERR_BOUNDS);
            live = false;
        }
        live = live && slot >= 0;
    }
    float x[8];
    {
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (live)
            raw = *reinterpret_cast<const uint4*>((is_k ? p.k + (int64_t)token * p.k_stride
                                                        : p.q + (int64_t)token * p.q_stride + h * kD) + 8 * l);
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(w[i]);
            x[2 * i + 1] = bf16_hi(w[i]);
        }
    }
    const float* nw = is_k ? p.k_w : p.q_w;
    const float* nb = is_k ? p.k_b : p.q_b;
    float mean = 0.f;
    if (LAYER) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += x[i];
        mean = half_sum(s) * (1.f / kD);
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i] - mean, x[i] - mean, ss);
    const float rstd = rsqrtf(half_sum(ss) * (1.f / kD) + p.eps);
    if (nw) {
        float w[8];
        load8(nw + 8 * l, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (x[i] - mean) * rstd * w[i];
        if (nb) {
            load8(nb + 8 * l, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] += w[i];
        }
    }
    const float* cs = p.cos_sin + (int64_t)(live ? pos : 0) * 64;
    if (INTERLEAVE) {          // lane l < 8 holds pairs 4l..4l+3
        if (l < 8) {
            const float4 c = __ldg(reinterpret_cast<const float4*>(cs) + l);
            const float4 s = __ldg(reinterpret_cast<const float4*>(cs + 32) + l);
            const float cc[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = x[2 * i], b = x[2 * i + 1];
                x[2 * i] = a * cc[i] - b * sn[i];
                x[2 * i + 1] = b * cc[i] + a * sn[i];
            }
        }
    } else {                   // dims 8l..8l+7 of lane l < 4 pair with those of lane l + 4
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __shfl_xor_sync(0xffffffffu, x[i], 4);
        if (l < 8) {
            float c[8], s[8];
            load8(cs + 8 * (l & 3), c);
            load8(cs + 32 + 8 * (l & 3), s);
            const float sign = l < 4 ? -1.f : 1.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * c[i] + sign * (y[i] * s[i]);
        }
    }
    if (!live) return;
    __nv_bfloat16* dst = is_k ? p.k_cache + (int64_t)slot * kD
                              : p.q_out + (int64_t)token * (DSA_INDEXER_HEADS * kD) + h * kD;
    *reinterpret_cast<uint4*>(dst + 8 * l) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                        pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

}  // namespace

dsa_status_t launch_indexer_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int norm,
                                      const float* q_w, const float* q_b, const float* k_w, const float* k_b,
                                      float eps, const float* cos_sin, int max_pos, int interleave,
                                      const int32_t* pos, const int32_t* slots, int R, void* q_out, void* k_cache,
                                      int cache_rows, cudaStream_t stream) {
    const NormRopeParams p{static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k), q_stride,
                           k_stride, q_w, q_b, k_w, k_b, eps, cos_sin, max_pos, pos, slots, R * kHeadsPerToken,
                           static_cast<__nv_bfloat16*>(q_out), static_cast<__nv_bfloat16*>(k_cache), cache_rows,
                           device_status_ptr()};
    auto kern = norm == DSA_NORM_LAYER
                    ? (interleave ? indexer_norm_rope_kernel<true, true> : indexer_norm_rope_kernel<true, false>)
                    : (interleave ? indexer_norm_rope_kernel<false, true> : indexer_norm_rope_kernel<false, false>);
    const int grid = ceil_div(p.units, kThreads / 16);
    if (launch_pdl(kern, dim3(grid), dim3(kThreads), 0, stream, p) != cudaSuccess) return DSA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
