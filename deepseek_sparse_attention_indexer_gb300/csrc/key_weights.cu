// key_weights.cu -- the attention weight that each key of a latent cache received: what an eviction goes by.
//
//   W[j] = sum over the queries that selected key j, over their 64 heads, of exp(scale * q . k_j - lse)
//
// with the lse that the attention of the same queries returned: the probabilities again, summed over heads instead of
// spent on values.  A pass of the scores alone (576 products a key and head, against 1088 for the attention).
//
// How (GB300 design):
//   * Keys sit on the 128 lanes of tensor memory, S^T = K . Q^T (M = 128 keys, N = 64 heads), so that a thread of the
//     epilogue has one key's 64 scores and its sum over heads needs no other thread.
//   * The rows of every format go through registers into tensor memory as bf16, as the A operand of the MMA, 64 dims
//     (32 columns) a slot of a ring of eight: e4m3 and 4-bit numbers times their block's scale are bf16 numbers, and the
//     row's scale is applied to the sum (the rope dims, which it does not scale, have an accumulator of their own).
//     Shared memory holds queries only, and its port is free for the MMA's reads of them.
//   * Four lanes load a row's 64 dims, 16 each, and store them with the 16-lane shape, whose columns a thread holds in
//     pairs: the MMA sees a chunk's dims in another order, four at a time transposed, and so does the query, which is
//     brought into that order on its way to shared memory.  (A lane a row is the order of the 32-lane shape, and a
//     load instruction then touches 32 lines in place of 8.)
//   * Roles: warp 0 issues MMAs, warps 1-3 load queries, 16 warps gather, 8 do the epilogue (4 a tile, in turn).
//   * Decode adds a key's weight to its float32 sum: one thread a key (the same key twice adds the same number twice).
//     A prefill's queries meet at keys in any order, so they add whole numbers, 2^-shift each, in 64 bits, and a second
//     kernel makes floats of them: the same bits every time.
#include <cuda.h>

#include <atomic>
#include <cmath>

#include "dsa_q4.cuh"
#include "mla_attn_common.cuh"

namespace dsa {

namespace {

constexpr int kQDim = DSA_QK_DIM;                  // 576
constexpr int kDims = 64;                          // dims of a chunk
constexpr int kChunks = kQDim / kDims;             // 9, the last one the rope dims
constexpr int kQBlk = kH * 128;                    // 8 KB: 64 heads x 64 dims
constexpr int kSlots = 8;                          // chunks in tensor memory
constexpr int kLoadWarps = 3, kGatherWarps = 16, kEpiWarps = 8;
constexpr int kFirstGather = 1 + kLoadWarps;
constexpr int kFirstEpi = kFirstGather + kGatherWarps;
constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
constexpr int kGroups = kGatherWarps / 4;          // four warps, one a lane quadrant, fill a chunk

constexpr int OFF_Q = 0;                           // 2 queries
constexpr int OFF_LSE = OFF_Q + 2 * kChunks * kQBlk;   // float [2][64]: -lse log2(e)
constexpr int OFF_BAR = OFF_LSE + 2 * kH * 4;
// barriers: full[8], empty[8], acc_full[2], acc_free[2], q_full[2], q_free[2]
constexpr int kBars = 2 * kSlots + 8;
constexpr int OFF_TMEM = OFF_BAR + kBars * 8;
constexpr int OFF_ABORT = OFF_TMEM + 4;
constexpr int kSmemBytes = OFF_ABORT + 4;

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t TM_A = 0;                       // ring: 8 x 32 columns
constexpr uint32_t TM_D = 256;                     // 2 x (64 latent, 64 rope)
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);   // 128-byte swizzle, 8-row groups 1 KB apart
constexpr uint32_t IDESC = idesc_bf16_f32(128, 64, false, false);

constexpr float kMostWeight = 128.f;               // of a query: 64 heads' probabilities, and room for their rounding

struct WeightParams : AttnShape {
    const __nv_bfloat16* q;    // [rows][64][576]
    const uint8_t* cache;      // rows of the format's bytes
    const float* cache_scale;  // q8, q4
    const float* lse;          // [rows][64]
    float scale_log2;          // scale * log2(e)
    float* acc;                // decode: [B][Nmax]
    unsigned long long* sums;  // prefill: [N], units of 2^-shift
    float unit;                // 2^shift
    int32_t* status;
    PageTable pages;
};

template <int FMT>
struct Row {
    static constexpr int kBytes = FMT == DSA_ROWS_BF16 ? 2 * kQDim : FMT == DSA_ROWS_Q8 ? kQ8Row : kQ4Row;
};

__device__ __forceinline__ Item item_at(const WeightParams& p, int item) {
    Item it{item / p.nsplit, item % p.nsplit, 0, 0, 0, 0};
    it.slot0 = it.split * p.split_len;
    it.slot_end = min(p.top_k, it.slot0 + p.split_len);
    it.batch = p.prefill ? 0 : it.row;
    it.bound = p.kv_len ? min(__ldg(p.kv_len + it.batch), p.Nmax) : p.Nmax;
    return it;
}

// Cache row of key j, -1 where there is none.
__device__ __forceinline__ int64_t key_row(const WeightParams& p, const Item& I, int j) {
    if (j < 0 || j >= I.bound) return -1;
    if (!p.pages.table) return (int64_t)I.batch * p.Nmax + j;
    return paged_row(p.pages, I.batch, j);
}

__device__ __forceinline__ void tmem_st_16x256b_x4(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// four e4m3 codes as bf16: exponent and fraction in place, then the exponent's bias (a product with 2^120, exact, also
// of the subnormal numbers)
__device__ __forceinline__ void e4m3_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t m = w & 0x7f7f7f7fu;
    constexpr uint32_t k2_120 = 0x7b807b80u;
    lo = mul_bf16x2((__byte_perm(w, 0, 0x1404) & 0x80008000u) | (__byte_perm(m, 0, 0x1404) >> 4), k2_120);
    hi = mul_bf16x2((__byte_perm(w, 0, 0x3424) & 0x80008000u) | (__byte_perm(m, 0, 0x3424) >> 4), k2_120);
}
// eight 4-bit codes as bf16, times their block's scale (twice in `scale`)
__device__ __forceinline__ void q4_to_bf16(uint32_t w, uint32_t scale, uint32_t* out) {
    const uint32_t sel = w & kQ4Magnitudes;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t s = h ? sel >> 16 : sel;
        const uint32_t top = __byte_perm(0x3f3f3f00u, 0x40404040u, s) | ((h ? w << 4 : w) & 0x80808080u);
        const uint32_t low = __byte_perm(0xc0800000u, 0xc0804000u, s);
        out[2 * h] = mul_bf16x2(__byte_perm(low, top, 0x5140), scale);
        out[2 * h + 1] = mul_bf16x2(__byte_perm(low, top, 0x7362), scale);
    }
}

// dims 16 j .. 16 j + 15 of chunk c of a row, as they lie in the cache; zeros without a row
template <int FMT>
__device__ __forceinline__ void load_dims(const WeightParams& p, int64_t row, int c, int j, uint32_t (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0;
    if (row < 0) return;
    const uint8_t* src = p.cache + row * Row<FMT>::kBytes;
    if (FMT == DSA_ROWS_BF16) {
        ldg_nc_v8(src + 128 * c + 32 * j, x);
    } else if (c == kChunks - 1) {                 // the rope dims of the other formats are bf16, too
        ldg_nc_v8(src + (FMT == DSA_ROWS_Q8 ? kQ8Latent : kQ4Rope) + 32 * j, x);
    } else if (FMT == DSA_ROWS_Q8) {
        const uint4 v = ldg_nc_v4(src + 64 * c + 16 * j);
        x[0] = v.x;
        x[1] = v.y;
        x[2] = v.z;
        x[3] = v.w;
    } else {
        ldg_nc_v2(src + 32 * c + 8 * j, x[0], x[1]);
        x[2] = ldg_nc_u8(src + kQ4Codes + 4 * c + j);
    }
}
// the same as bf16
template <int FMT>
__device__ __forceinline__ void widen(int c, uint32_t (&x)[8]) {
    if (FMT == DSA_ROWS_BF16 || c == kChunks - 1) return;
    if (FMT == DSA_ROWS_Q8) {
        const uint32_t w[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int i = 0; i < 4; ++i) e4m3_to_bf16(w[i], x[2 * i], x[2 * i + 1]);
    } else {
        const uint32_t w0 = x[0], w1 = x[1], b = x[2];
        // (1 + m/4) 2^(a - 6) as bf16: exponent 121 + a, fraction m/4
        const uint32_t a = b / 3, m = b - 3 * a;
        const uint32_t s = b < kQ4Scales ? (121 + a) << 7 | m << 5 : 0;
        q4_to_bf16(w0, s | s << 16, x);
        q4_to_bf16(w1, s | s << 16, x + 4);
    }
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1) key_weights_kernel(const WeightParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {   // the operand's swizzle counts from 1 KB boundaries
        if (threadIdx.x == 0) raise_dev_error(p.status, DEV_ERR_TIMEOUT);
        return;
    }
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    uint64_t* empty = full + kSlots;
    uint64_t* acc_full = empty + kSlots;
    uint64_t* acc_free = acc_full + 2;
    uint64_t* q_full = acc_free + 2;
    uint64_t* q_free = q_full + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_TMEM);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);
    const int warp = threadIdx.x / 32;
    const uint32_t lane = lane_id();

    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&full[i], 4);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_free[i], 4);
            mbar_init(&q_full[i], kLoadWarps);
            mbar_init(&q_free[i], 1 + kEpiWarps);  // the MMAs, and every warp of the epilogue once an item
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    griddep_wait();

    // One lane polls for its warp.
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        bool ok = true;
        if (lane == 0) ok = mbar_poll(bar, parity, abort_flag, p.status);
        return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    };
    // Items with tiles, in the same order for every role: f(item, tiles) until it returns false.
    auto items = [&](auto f) {
        for (int s = 0;; ++s) {
            const int it = nth_item(p, s);
            if (it == -1) return;
            if (it < 0) continue;
            const Item I = item_at(p, it);
            const int T = item_tiles(p, I, lane);
            if (T > 0 && !f(I, T)) return;
        }
    };

    if (warp == 0) {
        // ------------------------------------------------------------ MMA issuer
        int n = 0, gt = 0, qi = 0;
        items([&](const Item&, int T) {
            bool ok = wait(&q_full[qi & 1], (qi >> 1) & 1);
            const uint32_t q_lo = ((smem_u32(smem + OFF_Q) + (qi & 1) * (kChunks * kQBlk)) >> 4) | ((16u >> 4) << 16);
            for (int t = 0; ok && t < T; ++t, ++gt) {
                ok = wait(&acc_free[gt & 1], ((gt >> 1) & 1) ^ 1);
                const uint32_t d = tmem_base + TM_D + 128 * (gt & 1);
                for (int c = 0; ok && c < kChunks; ++c, ++n) {
                    ok = wait(&full[n % kSlots], (n / kSlots) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (lane == 0) {
                        const bool rope = FMT != DSA_ROWS_BF16 && c == kChunks - 1;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16_ts_lo(d + (rope ? 64 : 0), tmem_base + TM_A + 32 * (n % kSlots) + 8 * k,
                                           q_lo + c * (kQBlk >> 4) + 2 * k, kDescHi, IDESC, ((c && !rope) || k) ? 1u : 0u);
                        mma_commit(&empty[n % kSlots]);
                        if (c == kChunks - 1) {
                            mma_commit(&acc_full[gt & 1]);
                            if (t == T - 1) mma_commit(&q_free[qi & 1]);
                        }
                    }
                    __syncwarp();
                }
            }
            ++qi;
            return ok;
        });
    } else if (warp < kFirstGather) {
        // ------------------------------------------------------------ queries
        const int lt = (warp - 1) * 32 + (int)lane;
        int qi = 0;
        items([&](const Item& I, int) {
            if (!wait(&q_free[qi & 1], ((qi >> 1) & 1) ^ 1)) return false;
            const __nv_bfloat16* src = p.q + (int64_t)I.row * (kH * kQDim);
            uint8_t* dst = smem + OFF_Q + (qi & 1) * (kChunks * kQBlk);
            // 16 dims a step: head h, chunk c, piece j; its four dims 4 b.. go to 8-byte unit 4 b + j of the row
#pragma unroll 4
            for (int i = lt; i < kH * kChunks * 4; i += kLoadWarps * 32) {
                const int h = i / (kChunks * 4), r = i % (kChunks * 4), c = r / 4, j = r % 4;
                const uint4 u = ldg_nc_v4(src + h * kQDim + 16 * r), v = ldg_nc_v4(src + h * kQDim + 16 * r + 8);
                const uint2 w[4] = {{u.x, u.y}, {u.z, u.w}, {v.x, v.y}, {v.z, v.w}};
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    *reinterpret_cast<uint2*>(dst + c * kQBlk + h * 128 + (((2 * b + (j >> 1)) ^ (h & 7)) << 4) + 8 * (j & 1)) = w[b];
            }
            if (lt < kH)
                reinterpret_cast<float*>(smem + OFF_LSE)[(qi & 1) * kH + lt] =
                    -1.4426950408889634f * __ldg(p.lse + (int64_t)I.row * kH + lt);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[qi & 1]);
            ++qi;
            return true;
        });
    } else if (warp < kFirstEpi) {
        // ------------------------------------------------------------ gather
        const int quad = warp & 3, group = (warp - kFirstGather) >> 2;
        const int j = (int)(lane & 3);
        const uint32_t at = tmem_base + TM_A + (static_cast<uint32_t>(quad * 32) << 16);
        int n0 = 0;                                // chunks of the tiles before
        items([&](const Item& I, int T) {
            for (int t = 0; t < T; ++t, n0 += kChunks) {
                int64_t row[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {      // rows l / 4 + 8 i of the quadrant
                    const int slot = I.slot0 + t * kTile + quad * 32 + 8 * i + (int)(lane >> 2);
                    row[i] = key_row(p, I, slot < I.slot_end ? __ldg(p.idx + (int64_t)I.row * p.top_k + slot) : -1);
                }
                for (int c = (group - n0 % kGroups + kGroups) % kGroups; c < kChunks; c += kGroups) {
                    const int n = n0 + c;
                    uint32_t x[4][8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) load_dims<FMT>(p, row[i], c, j, x[i]);
                    if (!wait(&empty[n % kSlots], ((n / kSlots) & 1) ^ 1)) return false;
                    tc_fence_after();
#pragma unroll
                    for (int i = 0; i < 4; ++i) widen<FMT>(c, x[i]);
#pragma unroll
                    for (int f = 0; f < 2; ++f) {  // 16 lanes: rows of i = 2 f and 2 f + 1
                        uint32_t r[16];
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            r[4 * b] = x[2 * f][2 * b];
                            r[4 * b + 1] = x[2 * f][2 * b + 1];
                            r[4 * b + 2] = x[2 * f + 1][2 * b];
                            r[4 * b + 3] = x[2 * f + 1][2 * b + 1];
                        }
                        tmem_st_16x256b_x4(at + 32 * (n % kSlots) + (16u * f << 16), r);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[n % kSlots]);
                }
            }
            return true;
        });
    } else {
        // ------------------------------------------------------------ epilogue
        const int quad = warp & 3, set = (warp - kFirstEpi) >> 2;
        const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
        int gt = 0, qi = 0;
        items([&](const Item& I, int T) {
            // also of an item whose only tile is the other set's: no arrival ahead of its phase
            if (!wait(&q_full[qi & 1], (qi >> 1) & 1)) return false;
            for (int t = 0; t < T; ++t, ++gt) {
                if ((gt & 1) != set) continue;
                const int slot = I.slot0 + t * kTile + quad * 32 + (int)lane;
                const int key = slot < I.slot_end ? __ldg(p.idx + (int64_t)I.row * p.top_k + slot) : -1;
                const int64_t row = key_row(p, I, key);
                if (key >= 0 && row < 0) raise_dev_error(p.status, DEV_ERR_BOUNDS);
                float c = 1.f;
                if (FMT != DSA_ROWS_BF16 && row >= 0) c = __ldg(p.cache_scale + row);
                const float2 sc = make_float2(p.scale_log2 * c, p.scale_log2 * c), sr = make_float2(p.scale_log2, p.scale_log2);
                if (!wait(&acc_full[gt & 1], (gt >> 1) & 1)) return false;
                tc_fence_after();
                const float2* nl = reinterpret_cast<const float2*>(smem + OFF_LSE + (qi & 1) * kH * 4);
                const uint32_t d = tmem_base + lane_addr + TM_D + 128 * (gt & 1);
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int h = 0; h < kH; h += 16) {
                    uint32_t v[16], r[16];
                    tmem_ld16(d + h, v);
                    if (FMT != DSA_ROWS_BF16) tmem_ld16(d + 64 + h, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        float2 x = nl[h / 2 + k];
                        if (FMT != DSA_ROWS_BF16)
                            x = __ffma2_rn(make_float2(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1])), sr, x);
                        x = __ffma2_rn(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), sc, x);
                        sum = __fadd2_rn(sum, make_float2(ex2_approx(x.x), ex2_approx(x.y)));
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_free[gt & 1]);
                const float s = sum.x + sum.y;
                const float w = s > 0.f ? fminf(s, kMostWeight) : 0.f;   // NaN: 0
                if (row >= 0) {
                    if (p.prefill)
                        atomicAdd(p.sums + key, (unsigned long long)__float2ull_rn(w * p.unit));
                    else
                        atomicAdd(p.acc + (int64_t)I.batch * p.Nmax + key, w);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_free[qi & 1]);
            ++qi;
            return true;
        });
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

// acc (+)= the sums in units of 1 / unit
__global__ void __launch_bounds__(256)
    key_weights_finish_kernel(const unsigned long long* sums, int N, double per_unit, int accumulate, float* acc) {
    griddep_wait();
    const int j = blockIdx.x * 256 + threadIdx.x;
    if (j >= N) return;
    const float w = (float)((double)sums[j] * per_unit);
    acc[j] = accumulate ? acc[j] + w : w;
}

template <int FMT>
dsa_status_t launch(const WeightParams& p, cudaStream_t stream) {
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> done[kMaxDevices];
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return DSA_ERR_CUDA;
    if (!done[dev].load(std::memory_order_acquire)) {
        const dsa_status_t st = ensure_smem_attr(reinterpret_cast<const void*>(key_weights_kernel<FMT>), kSmemBytes);
        if (st != DSA_OK) return st;
        done[dev].store(true, std::memory_order_release);
    }
    const int sms = device_sm_count();
    if (launch_pdl(key_weights_kernel<FMT>, dim3(p.n_items < sms ? p.n_items : sms), dim3(kThreads), kSmemBytes, stream,
                   p) != cudaSuccess)
        return DSA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

dsa_status_t launch_format(int format, const WeightParams& p, cudaStream_t stream) {
    return format == DSA_ROWS_BF16 ? launch<DSA_ROWS_BF16>(p, stream)
           : format == DSA_ROWS_Q8 ? launch<DSA_ROWS_Q8>(p, stream)
                                   : launch<DSA_ROWS_Q4>(p, stream);
}

// Parts of a query's tiles: whole queries where they fill the SMs, else so many parts that the items do.
void split(WeightParams& p, int rows) {
    const int sms = device_sm_count(), tiles = ceil_div(p.top_k, kTile);
    int parts = rows >= sms || sms < 1 ? 1 : sms / rows;
    if (parts > tiles) parts = tiles;
    const int each = ceil_div(tiles, parts);
    p.rows = rows;
    p.split_len = each * kTile;
    p.nsplit = ceil_div(tiles, each);
    p.n_items = rows * p.nsplit;
}

WeightParams base_params(const void* q, const void* cache, const float* cache_scale, const int32_t* idx,
                         const float* lse, int Nmax, int top_k, float scale, const PageTable& pages) {
    WeightParams p{};
    p.idx = idx;
    p.Nmax = Nmax;
    p.top_k = top_k;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.cache = static_cast<const uint8_t*>(cache);
    p.cache_scale = cache_scale;
    p.lse = lse;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.status = device_status_ptr();
    p.pages = pages;
    return p;
}

}  // namespace

dsa_status_t launch_key_weights_prefill(int format, const void* q, const void* cache, const float* cache_scale,
                                        const int32_t* idx, const float* lse, int L, int N, int top_k, float scale,
                                        float* acc, int accumulate, void* workspace, const PageTable& pages,
                                        cudaStream_t stream) {
    WeightParams p = base_params(q, cache, cache_scale, idx, lse, N, top_k, scale, pages);
    p.prefill = 1;
    p.sums = static_cast<unsigned long long*>(workspace);
    // the largest sum, L queries of kMostWeight = 2^7, stays below 2^62 units
    int shift = 55;
    while (shift > 0 && ((long long)L >> (55 - shift)) > 0) --shift;
    p.unit = ldexpf(1.f, shift);
    split(p, L);
    if (cudaMemsetAsync(workspace, 0, (size_t)N * 8, stream) != cudaSuccess) return DSA_ERR_CUDA;
    const dsa_status_t st = launch_format(format, p, stream);
    if (st != DSA_OK) return st;
    if (launch_pdl(key_weights_finish_kernel, dim3(ceil_div(N, 256)), dim3(256), 0, stream,
                   static_cast<const unsigned long long*>(workspace), N, ldexp(1.0, -shift), accumulate, acc) != cudaSuccess)
        return DSA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

dsa_status_t launch_key_weights_decode(int format, const void* q, const void* cache, const float* cache_scale,
                                       const int32_t* kv_len, const int32_t* idx, const float* lse, int B, int Nmax,
                                       int top_k, float scale, float* acc, int accumulate, const PageTable& pages,
                                       cudaStream_t stream) {
    WeightParams p = base_params(q, cache, cache_scale, idx, lse, Nmax, top_k, scale, pages);
    p.kv_len = kv_len;
    p.acc = acc;
    split(p, B);
    if (!accumulate && cudaMemsetAsync(acc, 0, (size_t)B * Nmax * 4, stream) != cudaSuccess) return DSA_ERR_CUDA;
    return launch_format(format, p, stream);
}

}  // namespace dsa
