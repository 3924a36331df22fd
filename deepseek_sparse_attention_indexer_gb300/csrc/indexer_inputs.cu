// indexer_inputs.cu -- the indexer's queries and keys from their projections:
// norm of each 128-wide head, rotation of its first 64 dims, and the scatter of
// the keys to their cache, in one pass (SlimServe "GLM52_PIPELINE_TRACE.md",
// section 5: indexer_rope_interleave).
//   y = (x - [mean]) * rsqrt(mean((x - [mean])^2) + eps) * w + b,
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin) for the 32 pairs of dims 0..63
// 16.9 KB a token in and out, a few operations an element.  4096 tokens with both norms (69 MB) take 13.1 us, 5.3 TB/s,
// eight 16-byte loads of a lane in flight: with four 14.0, with two 16.3, with one 24; CTAs of 64 threads, so that
// a token's end leaves few lanes waiting (256 threads: 14.5 against 14.0, four loads).  8 tokens take 2.1 us, 1.7
// with two loads: less than the time the host needs to issue the call, so one form serves both.
#include "dsa_q8.cuh"

namespace dsa {

namespace {

constexpr int kThreads = 64;
constexpr int kHalves = kThreads / 16;                // half warps a CTA
constexpr int kHeads = DSA_INDEXER_HEADS;             // query heads of a token, beside its one key
constexpr int kD = DSA_INDEXER_DIM;
constexpr int kN = 8;                                 // query heads a half warp
static_assert(kHeads % kN == 0, "a half warp's heads are of one token");

struct NormRopeParams {
    const __nv_bfloat16 *q, *k;
    int64_t q_stride, k_stride;
    const float *q_w, *q_b, *k_w, *k_b;
    float eps;
    const float* cos_sin;
    int max_pos;
    const int32_t *pos, *slots;
    int R;
    __nv_bfloat16 *q_out, *k_cache;
    int cache_rows;
    int q_blocks;           // CTAs of queries; those behind them turn keys
    int32_t* status;
};

// Sum over the 16 lanes of a half warp.
__device__ __forceinline__ float half_sum(float x) {
#pragma unroll
    for (int o = 8; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Half a lane's dims of a head: 4, at `at` and at `at + gap`.
__device__ __forceinline__ void load8(const float* at, int gap, float2 (&v)[4]) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(at)), b = __ldg(reinterpret_cast<const float4*>(at + gap));
    v[0] = make_float2(a.x, a.y); v[1] = make_float2(a.z, a.w);
    v[2] = make_float2(b.x, b.y); v[3] = make_float2(b.z, b.w);
}

// N heads of one token by half a warp; every lane of the warp takes part in the shuffles, a half warp without
// work stores nothing.  Lanes 0..7 hold the turned dims, both dims of a pair on one lane: interleaved, lane l has
// dims 8l..8l+7 (16 bytes); split in halves, lane l < 8 has dims 4l..4l+3 and 32 more (8 bytes each), lane l >= 8
// dims 8l..8l+7.  The pairs of lane l are 4l..4l+3 either way.  Arithmetic in pairs of floats: the instructions'
// issue bounds the kernel beside HBM.
template <bool LAYER, bool INTERLEAVE, int N>
__device__ __forceinline__ void turn_heads(const __nv_bfloat16* src, __nv_bfloat16* dst, const float* nw, const float* nb,
                                           const float* cs, float eps, int l, bool live) {
    const int at = !INTERLEAVE && l < 8 ? 4 * l : 8 * l;        // the lane's first 4 dims
    const int gap = !INTERLEAVE && l < 8 ? 32 : 4;              // and how much further its last 4 lie
    uint2 raw[N][2];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        if (INTERLEAVE) {
            const uint4 v = live ? *reinterpret_cast<const uint4*>(src + n * kD + at) : make_uint4(0, 0, 0, 0);
            raw[n][0] = make_uint2(v.x, v.y);
            raw[n][1] = make_uint2(v.z, v.w);
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j)
                raw[n][j] = live ? *reinterpret_cast<const uint2*>(src + n * kD + at + j * gap) : make_uint2(0, 0);
        }
    }
    float c[4], s[4];
    if (l < 8) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(cs) + l);
        const float4 b = __ldg(reinterpret_cast<const float4*>(cs + 32) + l);
        c[0] = a.x; c[1] = a.y; c[2] = a.z; c[3] = a.w;
        s[0] = b.x; s[1] = b.y; s[2] = b.z; s[3] = b.w;
    }
    float2 w[4], wb[4];
    if (nw) load8(nw + at, gap, w);
    if (nb) load8(nb + at, gap, wb);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const uint32_t words[4] = {raw[n][0].x, raw[n][0].y, raw[n][1].x, raw[n][1].y};
        float2 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = make_float2(bf16_lo(words[i]), bf16_hi(words[i]));
        if (nw) {
            if (LAYER) {
                const float2 sum = __fadd2_rn(__fadd2_rn(x[0], x[1]), __fadd2_rn(x[2], x[3]));
                const float mean = half_sum(sum.x + sum.y) * (1.f / kD);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = __fadd2_rn(x[i], make_float2(-mean, -mean));
            }
            float2 ss = __fmul2_rn(x[0], x[0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) ss = __ffma2_rn(x[i], x[i], ss);
            const float rstd = rsqrtf(half_sum(ss.x + ss.y) * (1.f / kD) + eps);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = __fmul2_rn(x[i], make_float2(rstd, rstd));
                x[i] = nb ? __ffma2_rn(x[i], w[i], wb[i]) : __fmul2_rn(x[i], w[i]);
            }
        }
        if (l < 8) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = x[i].x;
                v[2 * i + 1] = x[i].y;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float &va = v[INTERLEAVE ? 2 * i : i], &vb = v[INTERLEAVE ? 2 * i + 1 : i + 4];
                const float a = va, b = vb;
                va = a * c[i] - b * s[i];
                vb = b * c[i] + a * s[i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = make_float2(v[2 * i], v[2 * i + 1]);
        }
        if (live) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(x[i].x, x[i].y);
            if (INTERLEAVE) {
                *reinterpret_cast<uint4*>(dst + n * kD + at) = make_uint4(o[0], o[1], o[2], o[3]);
            } else {
                *reinterpret_cast<uint2*>(dst + n * kD + at) = make_uint2(o[0], o[1]);
                *reinterpret_cast<uint2*>(dst + n * kD + at + gap) = make_uint2(o[2], o[3]);
            }
        }
    }
}

// Query CTAs: a half warp has kN heads of a token, whose loads are in flight together and share weights
// and angles.  Key CTAs: a half warp a token.
template <bool LAYER, bool INTERLEAVE>
__global__ void __launch_bounds__(kThreads) indexer_norm_rope_kernel(const NormRopeParams p) {
    griddep_wait();
    const int l = threadIdx.x & 15;
    const bool is_k = (int)blockIdx.x >= p.q_blocks;
    const int unit = (is_k ? (int)blockIdx.x - p.q_blocks : (int)blockIdx.x) * kHalves + (threadIdx.x >> 4);
    const int token = is_k ? unit : unit / (kHeads / kN);
    bool live = token < p.R;
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
    const float* cs = p.cos_sin + (int64_t)(live ? pos : 0) * 64;
    if (is_k) {
        turn_heads<LAYER, INTERLEAVE, 1>(p.k + (int64_t)token * p.k_stride, p.k_cache + (int64_t)slot * kD, p.k_w, p.k_b,
                                         cs, p.eps, l, live);
    } else {
        const int h = unit % (kHeads / kN) * kN;
        turn_heads<LAYER, INTERLEAVE, kN>(p.q + (int64_t)token * p.q_stride + h * kD,
                                          p.q_out + ((int64_t)token * kHeads + h) * kD, p.q_w, p.q_b, cs, p.eps, l, live);
    }
}

}  // namespace

dsa_status_t launch_indexer_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int norm,
                                      const float* q_w, const float* q_b, const float* k_w, const float* k_b,
                                      float eps, const float* cos_sin, int max_pos, int interleave,
                                      const int32_t* pos, const int32_t* slots, int R, void* q_out, void* k_cache,
                                      int cache_rows, cudaStream_t stream) {
    const int q_blocks = ceil_div(R * (kHeads / kN), kHalves);
    const NormRopeParams p{static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k), q_stride,
                           k_stride, q_w, q_b, k_w, k_b, eps, cos_sin, max_pos, pos, slots, R,
                           static_cast<__nv_bfloat16*>(q_out), static_cast<__nv_bfloat16*>(k_cache), cache_rows,
                           q_blocks, device_status_ptr()};
    auto kern = norm == DSA_NORM_LAYER
                    ? (interleave ? indexer_norm_rope_kernel<true, true> : indexer_norm_rope_kernel<true, false>)
                    : (interleave ? indexer_norm_rope_kernel<false, true> : indexer_norm_rope_kernel<false, false>);
    if (launch_pdl(kern, dim3(q_blocks + ceil_div(R, kHalves)), dim3(kThreads), 0, stream, p) != cudaSuccess) return DSA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
