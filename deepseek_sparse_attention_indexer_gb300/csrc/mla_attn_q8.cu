// mla_attn_q8.cu -- sparse absorbed-MLA attention over the 8-bit latent cache.
//
//   s[h,t] = scale * (q[h, :512] . (c_t * e4m3_t) + q[h, 512:] . rope_t),  p = softmax_t(s) in float32,
//   out[h,:] = sum_t p[h,t] * c_t * e4m3_t
// over the query's selected rows t, c_t the row's scale (the method's passages are cited in mla_attn.cu).
// This form: one CTA per (query, 16 heads), float32 arithmetic on the CUDA cores, keys in tiles of 32
// widened to float32 in shared memory, online softmax over the tiles.
#include <cmath>

#include "dsa_q8.cuh"

namespace dsa {

namespace {

constexpr int kThreads = 256;
constexpr int kHG = 16;            // heads a CTA
constexpr int kT = 32;             // keys a tile
constexpr int kPitch = DSA_QK_DIM + 1;   // floats, odd: a warp's 32 keys fall into 32 banks

struct AttnQ8Params {
    const __nv_bfloat16* q;
    const uint8_t* cache;
    const float* cache_scale;
    const int32_t* idx;
    const int32_t* kv_len;     // [B], or nullptr: every row may use Nmax keys
    void* out;
    int out_f32;
    float* lse;
    int prefill;               // 1: all rows read sequence 0; 0: row r reads sequence r
    int Nmax, top_k;
    float scale;
    int32_t* status;
    PageTable pages;
};

constexpr int kSmem = (kHG * DSA_QK_DIM + kT * kPitch + kHG * kT + 3 * kHG) * 4;

__global__ void __launch_bounds__(kThreads) attn_q8_kernel(const AttnQ8Params p) {
    extern __shared__ float sm[];
    float* sq = sm;                              // [16][576]
    float* skv = sq + kHG * DSA_QK_DIM;          // [32][577]
    float* sp = skv + kT * kPitch;               // [16][32] scores, then probabilities
    float* sm_m = sp + kHG * kT;                 // running maxima
    float* sm_l = sm_m + kHG;                    // running sums
    float* sm_a = sm_l + kHG;                    // rescale factors
    griddep_wait();
    const int row = blockIdx.x >> 2, h0 = (blockIdx.x & 3) * kHG, tid = threadIdx.x;
    const int b = p.prefill ? 0 : row;
    const int bound = p.kv_len ? min(__ldg(p.kv_len + b), p.Nmax) : p.Nmax;
    const __nv_bfloat16* q = p.q + ((int64_t)row * DSA_HEADS + h0) * DSA_QK_DIM;
    for (int i = tid; i < kHG * DSA_QK_DIM; i += kThreads) sq[i] = __bfloat162float(q[i]);
    if (tid < kHG) {
        sm_m[tid] = -INFINITY;
        sm_l[tid] = 0.f;
    }
    float acc[kHG][2];                           // heads x dims tid, tid + 256
#pragma unroll
    for (int h = 0; h < kHG; ++h) acc[h][0] = acc[h][1] = 0.f;
    for (int t0 = 0; t0 < p.top_k; t0 += kT) {
        __syncthreads();
        for (int k = tid / 32; k < kT; k += kThreads / 32) {     // a warp a key
            const int lane = tid & 31;
            int j = t0 + k < p.top_k ? __ldg(p.idx + (int64_t)row * p.top_k + t0 + k) : -1;
            int64_t at = -1;
            if (j >= bound) {
                if (lane == 0) raise_dev_error(p.status, DEV_ERR_BOUNDS);
                j = -1;
            }
            if (j >= 0) {
                at = p.pages.table ? paged_row(p.pages, b, j) : (int64_t)b * p.Nmax + j;
                if (at < 0 && lane == 0) raise_dev_error(p.status, DEV_ERR_BOUNDS);
            }
            const bool have = j >= 0;            // a page outside the pool is a row of zeros
            const float c = at >= 0 ? __ldg(p.cache_scale + at) : 0.f;
            for (int d = lane; d < DSA_QK_DIM; d += 32) {
                float v = 0.f;
                if (at >= 0) {
                    const uint8_t* r = p.cache + at * kQ8Row;
                    v = d < kQ8Latent ? unpack_e4m3x2(r[d]).x * c
                                      : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(r + kQ8Latent)[d - kQ8Latent]);
                }
                skv[k * kPitch + d] = v;
            }
            if (lane < kHG) sp[lane * kT + k] = have ? 0.f : -INFINITY;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kHG * kT / kThreads; ++i) {
            const int k = tid & 31, h = tid / 32 + i * (kThreads / 32);
            float s = 0.f;
            for (int d = 0; d < DSA_QK_DIM; ++d) s = fmaf(sq[h * DSA_QK_DIM + d], skv[k * kPitch + d], s);
            sp[h * kT + k] += s * p.scale;       // -inf where nothing is selected
        }
        __syncthreads();
        if (tid < kHG) {
            float m = sm_m[tid];
            for (int k = 0; k < kT; ++k) m = fmaxf(m, sp[tid * kT + k]);
            const float mm = m == -INFINITY ? 0.f : m;
            float l = 0.f;
            for (int k = 0; k < kT; ++k) {
                const float e = expf(sp[tid * kT + k] - mm);
                sp[tid * kT + k] = e;
                l += e;
            }
            const float a = expf(sm_m[tid] - mm);
            sm_a[tid] = a;
            sm_l[tid] = sm_l[tid] * a + l;
            sm_m[tid] = m;
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < kHG; ++h) {
            acc[h][0] *= sm_a[h];
            acc[h][1] *= sm_a[h];
        }
        for (int k = 0; k < kT; ++k) {
            const float v0 = skv[k * kPitch + tid], v1 = skv[k * kPitch + tid + 256];
#pragma unroll
            for (int h = 0; h < kHG; ++h) {
                const float e = sp[h * kT + k];
                acc[h][0] = fmaf(e, v0, acc[h][0]);
                acc[h][1] = fmaf(e, v1, acc[h][1]);
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kHG; ++h) {
        const float inv = sm_l[h] > 0.f ? 1.f / sm_l[h] : 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int64_t o = ((int64_t)row * DSA_HEADS + h0 + h) * DSA_V_DIM + tid + 256 * i;
            if (p.out_f32)
                static_cast<float*>(p.out)[o] = acc[h][i] * inv;
            else
                static_cast<__nv_bfloat16*>(p.out)[o] = __float2bfloat16_rn(acc[h][i] * inv);
        }
    }
    if (p.lse && tid < kHG)
        p.lse[(int64_t)row * DSA_HEADS + h0 + tid] = sm_l[tid] > 0.f ? sm_m[tid] + logf(sm_l[tid]) : -INFINITY;
}

dsa_status_t launch(int rows, const AttnQ8Params& p, cudaStream_t stream) {
    dsa_status_t st = ensure_smem_attr(reinterpret_cast<const void*>(attn_q8_kernel), kSmem);
    if (st != DSA_OK) return st;
    if (launch_pdl(attn_q8_kernel, dim3(rows * (DSA_HEADS / kHG)), dim3(kThreads), kSmem, stream, p) != cudaSuccess)
        return DSA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace

dsa_status_t launch_attn_q8_prefill(const void* q, const void* cache, const float* cache_scale, const int32_t* idx,
                                    int L, int N, int top_k, float scale, void* out, int out_f32, float* lse,
                                    const PageTable& pages, cudaStream_t stream) {
    const AttnQ8Params p{static_cast<const __nv_bfloat16*>(q), static_cast<const uint8_t*>(cache), cache_scale, idx,
                         nullptr, out, out_f32, lse, 1, N, top_k, scale, device_status_ptr(), pages};
    return launch(L, p, stream);
}

dsa_status_t launch_attn_q8_decode(const void* q, const void* cache, const float* cache_scale, const int32_t* kv_len,
                                   const int32_t* idx, int B, int Nmax, int top_k, float scale, void* out,
                                   int out_f32, float* lse, void* workspace, const PageTable& pages,
                                   cudaStream_t stream) {
    (void)workspace;
    const AttnQ8Params p{static_cast<const __nv_bfloat16*>(q), static_cast<const uint8_t*>(cache), cache_scale, idx,
                         kv_len, out, out_f32, lse, 0, Nmax, top_k, scale, device_status_ptr(), pages};
    return launch(B, p, stream);
}

}  // namespace dsa
