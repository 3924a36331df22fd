// key_weights.cu -- the attention weight that each key of a latent cache received: what an eviction goes by.
//
//   W[j] = sum over the queries that selected key j, over their 64 heads, of exp(scale * q . k_j - lse)
//
// with the lse that the attention of the same queries returned: the probabilities again, summed over heads instead of
// spent on values.  A pass of the scores alone (576 products a key and head, against 1088 for the attention).
//
// How (GB300 design):
//   * S^T = K . Q^T with the keys on the 128 lanes of tensor memory (M = 128 keys, N = 64 heads), so that a thread of the
//     epilogue has one key's 64 scores and its sum over heads needs no other thread.
//   * A tile's rows go to shared memory as bf16, 64 dims a slot, nine slots for the 576: bf16 rows by cp.async, whose
//     copies in flight hold no registers, e4m3 and 4-bit rows through registers.  Their numbers, times their block's
//     scale, are bf16 numbers; the row's scale is applied to the sum, and the rope dims, which it does not scale, have
//     an accumulator of their own.  (Rows through registers into tensor memory, as the MMA's A operand, left too few
//     bytes in flight: 1.24 ms for 4096 queries of 2048 bf16 rows.)
//   * One query stands in shared memory; a chunk of the next one is loaded when the last tile's MMAs have read it.
//   * An MMA of N = 64 takes its issuer 57 cycles, whatever N, a commit 200 and a look at the barriers 550: two issuers,
//     each with an accumulator of its own for its dims, and barriers for four groups of chunks in place of nine.
//   * Roles: warps 0 and 2 issue MMAs, warp 1 loads queries (TMA), 8 warps gather bf16 rows, 16 the others, 8 do the
//     epilogue, 4 a tile, in turn.
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
constexpr int kBlk = 128 * 128;                    // 16 KB: 128 keys x 64 dims
constexpr int kEpiWarps = 8;
template <int FMT>
struct Roles {                                     // warps 0 and 2 MMA, 1 queries, 3 none, then gather, then epilogue
    static constexpr int kGather = FMT == DSA_ROWS_BF16 ? 8 : 16;
    static constexpr int kFirstEpi = 4 + kGather;
    static constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
};

constexpr int OFF_Q = 0;
constexpr int OFF_K = OFF_Q + kChunks * kQBlk;
constexpr int OFF_LSE = OFF_K + kChunks * kBlk;    // float [8][64]: -lse log2(e), a copy an epilogue warp
constexpr int OFF_BAR = OFF_LSE + kEpiWarps * kH * 4;
// barriers: full[4], empty[4], q_full[4], q_free[4], acc_full[2], acc_free[2]
constexpr int kParts = 4;                          // chunks 0 1, 2 3 (first issuer); 4 5, 6 7 8 (second)
constexpr int kBars = 4 * kParts + 4;
__device__ __forceinline__ constexpr int part_begin(int g) { return 2 * g; }
__device__ __forceinline__ constexpr int part_end(int g) { return g == kParts - 1 ? kChunks : 2 * g + 2; }
constexpr int OFF_TMEM = OFF_BAR + kBars * 8;
constexpr int OFF_ABORT = OFF_TMEM + 4;
constexpr int kSmemBytes = OFF_ABORT + 4;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");

// accumulators of a tile, two tiles: chunks 0 to 3, chunks 4 and up, and, where it is not among those, the rope chunk
template <int FMT>
struct Acc {
    static constexpr uint32_t kCols = FMT == DSA_ROWS_BF16 ? 128 : 192, kAlloc = FMT == DSA_ROWS_BF16 ? 256 : 512;
};
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

// Dims 16 j .. 16 j + 15 of chunk c of a row of the 8-bit or 4-bit cache as they lie there; zeros without a row.
template <int FMT>
__device__ __forceinline__ void load_dims(const WeightParams& p, int row, int c, int j, uint32_t (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0;
    if (row < 0) return;
    const uint8_t* src = p.cache + (int64_t)row * Row<FMT>::kBytes;
    if (c == kChunks - 1) {                        // the rope dims, bf16
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
    if (c == kChunks - 1) return;
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
__global__ void __launch_bounds__(Roles<FMT>::kThreads, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tmap_q, const WeightParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {   // the operands' swizzle counts from 1 KB boundaries
        if (threadIdx.x == 0) raise_dev_error(p.status, DEV_ERR_TIMEOUT);
        return;
    }
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    uint64_t* empty = full + kParts;
    uint64_t* q_full = empty + kParts;
    uint64_t* q_free = q_full + kParts;
    uint64_t* acc_full = q_free + kParts;
    uint64_t* acc_free = acc_full + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_TMEM);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);
    constexpr int kFirstEpi = Roles<FMT>::kFirstEpi, kGroups = Roles<FMT>::kGather / 4;
    const int warp = threadIdx.x / 32;
    const uint32_t lane = lane_id();

    if (threadIdx.x == 0) {
        for (int i = 0; i < kParts; ++i) {
            mbar_init(&full[i], FMT == DSA_ROWS_BF16 ? 128 : 4);   // the copies' arrivals, or a warp's
            mbar_init(&empty[i], 1);
            mbar_init(&q_full[i], 1);
            mbar_init(&q_free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 2);
            mbar_init(&acc_free[i], 4);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, Acc<FMT>::kAlloc);
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

    // Chunk c of every tile lies in slot c; the slots' barriers are in the phase of the tile, gt, the query's of the item, qi.
    if (warp == 0 || warp == 2) {
        // ------------------------------------------------------------ MMA issuers
        // One look at all barriers, a lane each (a poll between MMAs waits until the tensor core has taken those before
        // it): lanes 0, 1 the keys' parts, 2, 3 the query's, 4 the accumulator.
        const int g0 = warp;                       // the issuer's parts g0, g0 + 1
        int gt = 0, qi = 0;
        const uint32_t base = (smem_u32(smem) >> 4) | ((16u >> 4) << 16);
        items([&](const Item&, int T) {
            for (int t = 0; t < T; ++t, ++gt) {
                const uint32_t acc = tmem_base + Acc<FMT>::kCols * (gt & 1), d = acc + (g0 ? 64 : 0);
                uint64_t* mine = lane < 2 ? &full[g0 + lane] : lane < 4 ? &q_full[g0 + lane - 2] : &acc_free[gt & 1];
                const uint32_t parity = lane < 2 ? gt & 1 : lane < 4 ? qi & 1 : ((gt >> 1) & 1) ^ 1;
                uint32_t got = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t need = 5u << h | 16u;
                    if ((got & need) != need) {
                        got = mbar_poll_warp(mine, parity, lane, 5, need, abort_flag, p.status);
                        if (got == 0) return false;
                        fence_proxy_async_smem();  // of every lane that saw a barrier, before the lane that issues
                        tc_fence_after();
                        __syncwarp();
                    }
                    if (lane == 0) {
                        const int g = g0 + h;
                        for (int c = part_begin(g); c < part_end(g); ++c) {
                            const bool rope = FMT != DSA_ROWS_BF16 && c == kChunks - 1;
                            const bool first = c == part_begin(g0) || rope;
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_bf16_ss_lo(rope ? acc + 128 : d, base + ((OFF_K + c * kBlk) >> 4) + 2 * k, kDescHi,
                                               base + ((OFF_Q + c * kQBlk) >> 4) + 2 * k, kDescHi, IDESC, first && k == 0 ? 0u : 1u);
                        }
                        mma_commit(&empty[g]);
                        if (t == T - 1) mma_commit(&q_free[g]);
                    }
                    __syncwarp();
                }
                if (lane == 0) mma_commit(&acc_full[gt & 1]);
                __syncwarp();
            }
            ++qi;
            return true;
        });
    } else if (warp == 1) {
        // ------------------------------------------------------------ queries (TMA)
        int qi = 0;
        items([&](const Item& I, int) {
            for (int g = 0; g < kParts; ++g) {
                if (!wait(&q_free[g], (qi & 1) ^ 1)) return false;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&q_full[g], (part_end(g) - part_begin(g)) * kQBlk);
                    for (int c = part_begin(g); c < part_end(g); ++c)
                        tma_load_2d(smem + OFF_Q + c * kQBlk, &tmap_q, &q_full[g], c * kDims, I.row * kH);
                }
                __syncwarp();
            }
            ++qi;
            return true;
        });
    } else if (warp >= 4 && warp < kFirstEpi) {
        // ------------------------------------------------------------ gather
        // Four warps, 32 rows each, fill a chunk: bf16 rows eight lanes a row, 16 bytes each, two sets of warps with two
        // parts each; the others four lanes a row, 16 dims each, a set a part.
        constexpr int kLanes = FMT == DSA_ROWS_BF16 ? 8 : 4, kRows = kLanes;
        constexpr int kOwn = kParts / kGroups;
        const int quad = warp & 3, g0 = ((warp - 4) >> 2) * kOwn;
        const int j = (int)lane % kLanes, r0 = quad * 32 + (int)lane / kLanes;   // rows r0 + 32 / kLanes * i
        int gt = 0;
        items([&](const Item& I, int T) {
            const int32_t* idx = p.idx + (int64_t)I.row * p.top_k;
            for (int t = 0; t < T; ++t, ++gt) {
                int row[kRows];
#pragma unroll
                for (int i = 0; i < kRows; ++i) {
                    const int slot = I.slot0 + t * kTile + r0 + 32 / kLanes * i;
                    row[i] = slot < I.slot_end ? __ldg(idx + slot) : -1;
                }
#pragma unroll
                for (int i = 0; i < kRows; ++i) row[i] = (int)key_row(p, I, row[i]);
                if constexpr (FMT == DSA_ROWS_BF16) {
#pragma unroll 1
                    for (int g = g0; g < g0 + kOwn; ++g) {
                        if (!wait(&empty[g], (gt & 1) ^ 1)) return false;
                        for (int c = part_begin(g); c < part_end(g); ++c) {
                            const uint32_t dst = smem_u32(smem + OFF_K) + c * kBlk + r0 * 128;
#pragma unroll
                            for (int i = 0; i < kRows; ++i) {
                                const uint8_t* src = p.cache + (int64_t)max(row[i], 0) * Row<FMT>::kBytes + 128 * c + 16 * j;
                                cp_async_16(dst + i * 512 + ((j ^ ((r0 + 4 * i) & 7)) << 4), src, row[i] >= 0 ? 16u : 0u);
                            }
                        }
                        cp_async_arrive_noinc(&full[g]);
                    }
                } else {
                    uint32_t x[kRows][8];
                    const int g = g0, r = (int)lane / kLanes;   // row % 8
                    for (int c = part_begin(g); c < part_end(g); ++c) {
#pragma unroll
                        for (int i = 0; i < kRows; ++i) load_dims<FMT>(p, row[i], c, j, x[i]);
                        if (c == part_begin(g) && !wait(&empty[g], (gt & 1) ^ 1)) return false;
                        uint8_t* dst = smem + OFF_K + c * kBlk + r0 * 128;
#pragma unroll
                        for (int i = 0; i < kRows; ++i) {
                            widen<FMT>(c, x[i]);
                            *reinterpret_cast<uint4*>(dst + i * 1024 + (((2 * j) ^ r) << 4)) = make_uint4(x[i][0], x[i][1], x[i][2], x[i][3]);
                            *reinterpret_cast<uint4*>(dst + i * 1024 + (((2 * j + 1) ^ r) << 4)) = make_uint4(x[i][4], x[i][5], x[i][6], x[i][7]);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[g]);
                }
            }
            return true;
        });
        cp_async_wait_all();
    } else if (warp >= kFirstEpi) {
        // ------------------------------------------------------------ epilogue
        const int quad = warp & 3, set = (warp - kFirstEpi) >> 2;
        const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
        float2* nl = reinterpret_cast<float2*>(smem + OFF_LSE) + (warp - kFirstEpi) * (kH / 2);
        int gt = 0;
        items([&](const Item& I, int T) {
            const float* lse = p.lse + (int64_t)I.row * kH + 2 * lane;
            const float l0 = __ldg(lse), l1 = __ldg(lse + 1);
            __syncwarp();
            nl[lane] = make_float2(-1.4426950408889634f * l0, -1.4426950408889634f * l1);
            __syncwarp();
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
                const uint32_t d = tmem_base + lane_addr + Acc<FMT>::kCols * (gt & 1);
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int h = 0; h < kH; h += 16) {
                    uint32_t u[16], v[16], r[16];
                    tmem_ld16(d + h, u);
                    tmem_ld16(d + 64 + h, v);
                    if (FMT != DSA_ROWS_BF16) tmem_ld16(d + 128 + h, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        float2 x = nl[h / 2 + k];
                        if (FMT != DSA_ROWS_BF16)
                            x = __ffma2_rn(make_float2(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1])), sr, x);
                        x = __ffma2_rn(make_float2(__uint_as_float(u[2 * k]), __uint_as_float(u[2 * k + 1])), sc, x);
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
            return true;
        });
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem_base, Acc<FMT>::kAlloc);
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
    CUtensorMap tq;
    const dsa_status_t st = make_tmap_bf16_2d(&tq, p.q, kQDim, (uint64_t)p.rows * kH, kQDim * 2, kDims, kH);
    if (st != DSA_OK) return st;
    const int sms = device_sm_count();
    if (launch_pdl(key_weights_kernel<FMT>, dim3(p.n_items < sms ? p.n_items : sms), dim3(Roles<FMT>::kThreads), kSmemBytes,
                   stream, tq, p) != cudaSuccess)
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
