// key_weights.cu -- the attention weight that each key of a latent cache received: what an eviction goes by.
//
//   W[j] = sum over the queries that selected key j, over their 64 heads, of exp(scale * q . k_j - lse)
//
// with the lse that the attention of the same queries returned: the probabilities again, summed over heads instead of
// spent on values.  A pass of the scores alone (576 products a key and head, against 1088 for the attention).
//
// How (GB300 design):
//   * S^T = K . Q^T with the keys on the 128 lanes of tensor memory (M = 128 keys, heads as N), so that a thread of the
//     epilogue has one key's 64 scores and its sum over heads needs no other thread.
//   * The gathered rows go to shared memory by cp.async, whose copies in flight hold no registers; the query stands there.
//     (Rows through registers into tensor memory, as the MMA's A operand, left too few bytes in flight: 1.24 ms for 4096
//     queries of 2048 bf16 rows.)
//   * bf16 rows: nine chunks of 64 dims, a tile's in nine slots.  An MMA of N = 64 takes its issuer 57 cycles, whatever
//     N, and a look at the barriers 550: two issuers, and barriers for four groups of chunks, each with an accumulator
//     of its own, in place of nine (1.22 -> 0.91 ms).
//   * 8-bit and 4-bit rows: e4m3 products, the query as two e4m3 numbers, as in the attention over them (mla_attn_q8.cu):
//     four chunks of 128 dims and the rope dims, 20 MMAs a tile in place of 36, two issuers with a tile in turn.  The
//     row's scale and the query head's are applied to the sums.  4-bit rows are expanded on their way, a lane its own row.
//   * Decode adds a key's weight to its float32 sum: one thread a key (the same key twice adds the same number twice).
//     A prefill's queries meet at keys in any order, so they add whole numbers, 2^-shift each, in 64 bits, and a second
//     kernel makes floats of them: the same bits every time.
//   * Measured: 4096 queries of 2048 of 16k keys 0.76 ms over bf16 rows (0.42 of the bf16 matrix peak, 12.7 TB/s gathered from
//     L2), 0.70 over 8-bit and 4-bit rows; decode of 128 sequences of up to 8192 keys 52 us over 4-bit, 38 over 8-bit, 54 over
//     bf16 rows, of 8 over bf16 rows 7.5.  What bounds it (traces): bf16 rows the bytes in flight, one tile's 147 KB for the 3500
//     cycles of copy (2000), MMA and barriers; 8-bit rows the MMA phases of the two issuers, which fall together and then
//     wait together for the epilogue (3100 cycles a tile); 4-bit rows in decode the expansion.
#include <cuda.h>

#include <atomic>
#include <cmath>
#include <type_traits>

#include "dsa_q4.cuh"
#include "mla_attn_common.cuh"

namespace dsa {

namespace {

constexpr int kQDim = DSA_QK_DIM;                  // 576
constexpr int kBlk = 128 * 128;                    // 16 KB: 128 keys x 128 bytes
constexpr int kQBlk = kH * 128;                    // 8 KB: 64 heads x 64 bf16 dims
constexpr int kEpiWarps = 8;                       // four a tile, in turn
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);   // 128-byte swizzle, 8-row groups 1 KB apart
constexpr uint32_t IDESC_BF16 = idesc_bf16_f32(128, 64, false, false);
constexpr uint32_t IDESC_E4M3 = idesc_e4m3_f32(128, 128, false, false);
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMostWeight = 128.f;               // of a query: 64 heads' probabilities, and room for their rounding

struct WeightParams : AttnShape {
    const __nv_bfloat16* q;    // [rows][64][576]
    const uint8_t* cache;      // rows of the format's bytes
    const float* cache_scale;  // 8-bit, 4-bit
    const float* lse;          // [rows][64]
    float scale_log2;          // scale * log2(e)
    float* acc;                // decode: [B][Nmax]
    unsigned long long* sums;  // prefill: [N], units of 2^-shift
    float unit;                // 2^shift
    int32_t* status;
    PageTable pages;           // of `cache`
    PageTable given;           // of the caller's cache, where `cache` holds its rows expanded and dense; else the same
};

__device__ __forceinline__ Item item_at(const WeightParams& p, int item) {
    Item it{item / p.nsplit, item % p.nsplit, 0, 0, 0, 0};
    it.slot0 = it.split * p.split_len;
    it.slot_end = min(p.top_k, it.slot0 + p.split_len);
    it.batch = p.prefill ? 0 : it.row;
    it.bound = p.kv_len ? min(__ldg(p.kv_len + it.batch), p.Nmax) : p.Nmax;
    return it;
}

// Selected key `slot` of the item, -1 where there is none; and the cache row of a key, -1 where there is none.
__device__ __forceinline__ int key_at(const WeightParams& p, const Item& I, int slot) {
    return slot < I.slot_end ? __ldg(p.idx + (int64_t)I.row * p.top_k + slot) : -1;
}
__device__ __forceinline__ int key_row(const WeightParams& p, const PageTable& pages, const Item& I, int key) {
    if (key < 0 || key >= I.bound) return -1;
    if (!pages.table) return (int)((int64_t)I.batch * p.Nmax + key);
    return (int)paged_row(pages, I.batch, key);
}

// Items with tiles, in the same order for every role: f(item, tiles) until it returns false.
template <typename F>
__device__ __forceinline__ void for_items(const WeightParams& p, uint32_t lane, F f) {
    for (int s = 0;; ++s) {
        const int it = nth_item(p, s);
        if (it == -1) return;
        if (it < 0) continue;
        const Item I = item_at(p, it);
        const int T = item_tiles(p, I, lane);
        if (T > 0 && !f(I, T)) return;
    }
}

// The row of a gathering lane, one a tile, tile after tile over all items, in two steps so that the loads of one are in
// flight while the warp copies: fetch() loads the key of the next tile, resolve() makes a cache row of it (a page lookup
// when paged).
struct Feed {
    int s = 0, tiles = 0;              // next item; tiles of the current one still to fetch
    int slot = 0;                      // of the lane's row in the next tile
    Item I{};
    int key = -1, batch = 0, bound = 0;

    __device__ __forceinline__ bool fetch(const WeightParams& p, uint32_t lane, int r) {
        while (tiles == 0) {
            const int it = nth_item(p, s++);
            if (it == -1) return false;
            if (it < 0) continue;
            I = item_at(p, it);
            tiles = item_tiles(p, I, lane);
            slot = I.slot0 + r;
        }
        key = key_at(p, I, slot);
        batch = I.batch;
        bound = I.bound;
        slot += kTile;
        --tiles;
        return true;
    }
    __device__ __forceinline__ int resolve(const WeightParams& p) const {
        Item at{};
        at.batch = batch;
        at.bound = bound;
        return key_row(p, p.pages, at, key);
    }
};

// All lanes look once; where the phase has not come, one lane polls for its warp.
__device__ __forceinline__ bool warp_poll(uint64_t* bar, uint32_t parity, uint32_t lane, volatile int* abort, int32_t* status) {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    bool ok = true;
    if (lane == 0) ok = mbar_poll(bar, parity, abort, status);
    return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}

__device__ __align__(16) uint8_t g_no_row[2 * kQDim];   // zeros, the row of a key that is not there

// 128 bytes of each of the lane's rows (r0 + 4 i of the tile, eight lanes a row, this lane's 16 bytes the j-th: src) to a
// slot.  One instruction a row, and a row looked up by one lane: the gathering warps' instructions are what a tile of bf16
// or 8-bit rows waits for.
struct RowCopy {
    const uint8_t* src[8];
    uint32_t even, odd;                            // offsets in a slot of the rows of even and of odd i, less 512 i

    __device__ __forceinline__ RowCopy(int r0, int j)
        : even(r0 * 128 + ((j ^ (r0 & 7)) << 4)), odd(r0 * 128 + ((j ^ (r0 & 7) ^ 4) << 4)) {}
    // row: the cache row of the warp's lane-th row of the tile
    __device__ __forceinline__ void point(const WeightParams& p, int row, int bytes, int j, uint32_t lane) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int r = __shfl_sync(0xffffffffu, row, 4 * i + (int)(lane >> 3));
            src[i] = (r < 0 ? g_no_row : p.cache + (int64_t)r * bytes) + 16 * j;
        }
    }
    __device__ __forceinline__ void copy(int at, uint32_t slot) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) cp_async_16(slot + ((i & 1) ? odd : even) + i * 512, src[i] + at);
    }
};

__device__ __forceinline__ void add_weight(const WeightParams& p, const Item& I, int key, int row, float2 sum) {
    const float s = sum.x + sum.y;
    const float w = s > 0.f ? fminf(s, kMostWeight) : 0.f;   // NaN: 0
    if (row < 0) return;
    if (p.prefill)
        atomicAdd(p.sums + key, (unsigned long long)__float2ull_rn(w * p.unit));
    else
        atomicAdd(p.acc + (int64_t)I.batch * p.Nmax + key, w);
}

// A copy of -lse log2(e) of the item's heads for the calling warp.  The exponent is s (scale log2(e)) - lse log2(e), both factors
// rounded: up to 2^-23 (|scale s| + |lse|) of a weight, of the size of what the rounding of lse to float32 itself leaves open
// (2^-24 |lse|).  (scale s - lse) log2(e) has one rounding of the difference; it took 4096 queries over 8-bit rows 704 -> 737 us and
// over bf16 rows 758 -> 763, and left the error against float64 of 1024 queries at 3.5e-7 (bf16: the tensor core cuts sums) and 6e-8.
__device__ __forceinline__ void stage_lse(const WeightParams& p, const Item& I, float2* nl, uint32_t lane) {
    const float* lse = p.lse + (int64_t)I.row * kH + 2 * lane;
    const float l0 = __ldg(lse), l1 = __ldg(lse + 1);
    __syncwarp();
    nl[lane] = make_float2(-kLog2e * l0, -kLog2e * l1);
    __syncwarp();
}

template <int N>
__device__ __forceinline__ float2 pair(const uint32_t (&v)[N], int k) {
    return make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]));
}

// ------------------------------------------------------------------------------------------------ bf16 rows

namespace wide {

constexpr int kChunks = kQDim / 64;                // 9
constexpr int kParts = 4;                          // chunks 0 1, 2 3 (first issuer); 4 5, 6 7 8 (second)
__device__ __forceinline__ constexpr int part_begin(int g) { return 2 * g; }
__device__ __forceinline__ constexpr int part_end(int g) { return g == kParts - 1 ? kChunks : 2 * g + 2; }
// warps 0 and 2 MMA, 1 queries, 3 none, 4-11 gather, 12-19 epilogue
constexpr int kFirstGather = 4, kFirstEpi = 12, kThreads = 32 * (kFirstEpi + kEpiWarps);

constexpr int OFF_Q = 0;
constexpr int OFF_K = OFF_Q + kChunks * kQBlk;
constexpr int OFF_LSE = OFF_K + kChunks * kBlk;    // float [8][64], a copy an epilogue warp
constexpr int OFF_BAR = OFF_LSE + kEpiWarps * kH * 4;
constexpr int kBars = 4 * kParts + 4;              // full[4], empty[4], q_full[4], q_free[4], acc_full[2], acc_free[2]
constexpr int OFF_TMEM = OFF_BAR + kBars * 8;
constexpr int OFF_ABORT = OFF_TMEM + 4;
constexpr int kSmemBytes = OFF_ABORT + 4;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");
// An accumulator a part, two tiles: the tensor core cuts a sum where it adds to it, and 8 to 12 additions each, summed here
// rounded to nearest, are nearer than 16 to 20 (error against float64, 8 sequences, 1.1e-6 -> 5e-7, for 4% of the time).
constexpr uint32_t kAccCols = 64 * kParts, kTmemCols = 2 * kAccCols;

}  // namespace wide

__global__ void __launch_bounds__(wide::kThreads, 1)
    key_weights_bf16_kernel(const __grid_constant__ CUtensorMap tmap_q, const WeightParams p) {
    using namespace wide;
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
    const int warp = threadIdx.x / 32;
    const uint32_t lane = lane_id();

    if (threadIdx.x == 0) {
        for (int i = 0; i < kParts; ++i) {
            mbar_init(&full[i], 128);              // the copies' arrivals, one a lane of four warps
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
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    griddep_wait();
    auto wait = [&](uint64_t* bar, uint32_t parity) { return warp_poll(bar, parity, lane, abort_flag, p.status); };

    // Chunk c of every tile lies in slot c; the slots' barriers are in the phase of the tile, gt, the query's of the item, qi.
    if (warp == 0 || warp == 2) {
        // ------------------------------------------------------------ MMA issuers
        // One look at all barriers, a lane each (a poll between MMAs waits until the tensor core has taken those before
        // it): lanes 0, 1 the keys' parts, 2, 3 the query's, 4 the accumulator.
        const int g0 = warp;                       // the issuer's parts g0, g0 + 1
        int gt = 0, qi = 0;
        const uint32_t base = (smem_u32(smem) >> 4) | ((16u >> 4) << 16);
        for_items(p, lane, [&](const Item&, int T) {
            for (int t = 0; t < T; ++t, ++gt) {
                const uint32_t d = tmem_base + kAccCols * (gt & 1);
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
                        for (int c = part_begin(g); c < part_end(g); ++c)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_bf16_ss_lo(d + 64 * g, base + ((OFF_K + c * kBlk) >> 4) + 2 * k, kDescHi,
                                               base + ((OFF_Q + c * kQBlk) >> 4) + 2 * k, kDescHi, IDESC_BF16,
                                               c == part_begin(g) && k == 0 ? 0u : 1u);
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
        for_items(p, lane, [&](const Item& I, int) {
            for (int g = 0; g < kParts; ++g) {
                if (!wait(&q_free[g], (qi & 1) ^ 1)) return false;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&q_full[g], (part_end(g) - part_begin(g)) * kQBlk);
                    for (int c = part_begin(g); c < part_end(g); ++c)
                        tma_load_2d(smem + OFF_Q + c * kQBlk, &tmap_q, &q_full[g], 64 * c, I.row * kH);
                }
                __syncwarp();
            }
            ++qi;
            return true;
        });
    } else if (warp >= kFirstGather && warp < kFirstEpi) {
        // ------------------------------------------------------------ gather: two sets of four warps, two parts each
        const int quad = warp & 3, g0 = (warp - kFirstGather) >> 2 << 1;
        const int j = (int)lane & 7, r0 = quad * 32 + (int)(lane >> 3);
        const uint32_t keys = smem_u32(smem) + OFF_K;
        const int r = quad * 32 + (int)lane;       // the row the lane looks up
        Feed feed;
        RowCopy rows(r0, j);
        int row = -1;
        bool has = feed.fetch(p, lane, r), more = has;
        if (has) {
            row = feed.resolve(p);
            more = feed.fetch(p, lane, r);
        }
        for (int gt = 0; has; ++gt) {
            rows.point(p, row, 2 * kQDim, j, lane);
            if (more) row = feed.resolve(p);
            has = more;
            more = more && feed.fetch(p, lane, r);
            bool ok = true;
            auto part = [&](auto which) {          // the chunks as constants: offsets in the instructions
                constexpr int g = decltype(which)::value;
                ok = ok && wait(&empty[g], (gt & 1) ^ 1);
                if (!ok) return;
#pragma unroll
                for (int c = part_begin(g); c < part_end(g); ++c) rows.copy(128 * c, keys + c * kBlk);
                cp_async_arrive_noinc(&full[g]);
            };
            if (g0 == 0) {
                part(std::integral_constant<int, 0>{});
                part(std::integral_constant<int, 1>{});
            } else {
                part(std::integral_constant<int, 2>{});
                part(std::integral_constant<int, 3>{});
            }
            if (!ok) break;
        }
        cp_async_wait_all();
    } else if (warp >= kFirstEpi) {
        // ------------------------------------------------------------ epilogue
        const int quad = warp & 3, set = (warp - kFirstEpi) >> 2;
        const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
        float2* nl = reinterpret_cast<float2*>(smem + OFF_LSE) + (warp - kFirstEpi) * (kH / 2);
        const float2 sc = make_float2(p.scale_log2, p.scale_log2);
        int gt = 0;
        for_items(p, lane, [&](const Item& I, int T) {
            stage_lse(p, I, nl, lane);
            for (int t = 0; t < T; ++t, ++gt) {
                if ((gt & 1) != set) continue;
                const int key = key_at(p, I, I.slot0 + t * kTile + quad * 32 + (int)lane), row = key_row(p, p.pages, I, key);
                if (key >= 0 && row < 0) raise_dev_error(p.status, DEV_ERR_BOUNDS);
                if (!wait(&acc_full[gt & 1], (gt >> 1) & 1)) return false;
                tc_fence_after();
                const uint32_t d = tmem_base + lane_addr + kAccCols * (gt & 1);
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int h = 0; h < kH; h += 16) {
                    uint32_t u[16], v[16];
                    float2 s[8];
                    tmem_ld16(d + h, u);
                    tmem_ld16(d + 64 + h, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 8; ++k) s[k] = __fadd2_rn(pair(u, k), pair(v, k));
                    tmem_ld16(d + 128 + h, u);
                    tmem_ld16(d + 192 + h, v);
                    tmem_ld_wait();
                    if (h == kH - 16) {            // all read: free before the last exponentials
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&acc_free[gt & 1]);
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float2 x = __ffma2_rn(__fadd2_rn(s[k], __fadd2_rn(pair(u, k), pair(v, k))), sc, nl[h / 2 + k]);
                        sum = __fadd2_rn(sum, make_float2(ex2_approx(x.x), ex2_approx(x.y)));
                    }
                }
                add_weight(p, I, key, row, sum);
            }
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

// ------------------------------------------------------------------------------------------------ 8-bit and 4-bit rows

namespace low {

constexpr int kChunks = 5;                         // four of 128 latent dims, the rope dims
constexpr int kSlots = 9;                          // chunk n of the CTA lies in slot n % 9
constexpr int kQueryWarps = 8;                     // eight heads each
// Places of the query heads' scales.  Those of item n are written when the MMAs of item n - 2 are known to be done.  With items
// of one tile these waited only for accumulators that the epilogue gives free before its last reads of the scales: of items
// n - 4 and, by the other set of warps, n - 5.  So six places at least.
constexpr int kScalePlaces = 8;
// warps 0 and 2 MMA, 1 and 3 none, 4-11 gather, 12-19 queries, 20-27 epilogue
constexpr int kFirstGather = 4, kFirstQuery = 12, kFirstEpi = kFirstQuery + kQueryWarps;
constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
// registers by warpgroups of what the launch holds
constexpr int kLaunchRegs = 72, kIssueRegs = 56, kGatherRegs = 72, kQueryRegs = 88, kEpiRegs = 64;
static_assert(32 * (4 * kIssueRegs + 8 * kGatherRegs + 8 * kQueryRegs + 8 * kEpiRegs) <= kThreads * kLaunchRegs, "registers of the CTA");

constexpr int OFF_QHL = 0;                         // 4 chunks x (64 hi rows, 64 lo rows) x 128 B
constexpr int OFF_QR = OFF_QHL + 4 * kBlk;         // rope dims of 64 heads, bf16
constexpr int OFF_K = OFF_QR + kQBlk;
constexpr int OFF_LSE = OFF_K + kSlots * kBlk;     // float [8][64], a copy an epilogue warp
constexpr int OFF_QS = OFF_LSE + kEpiWarps * kH * 4;   // float [8][64]: scale log2(e) 2^k of a query's heads
constexpr int OFF_TABLE = OFF_QS + kScalePlaces * kH * 4;   // uint2 [256]: the magnitudes of 4-bit codes as e4m3, by block byte
constexpr int OFF_BAR = OFF_TABLE + 256 * 8;
constexpr int kBars = 2 * kSlots + 3 + 4;          // full[9], empty[9], q_full, qr_full, q_free, acc_full[2], acc_free[2]
constexpr int OFF_TMEM = OFF_BAR + kBars * 8;
constexpr int OFF_ABORT = OFF_TMEM + 4;
constexpr int kSmemBytes = OFF_ABORT + 4;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");
constexpr uint32_t kAccCols = 192, kTmemCols = 512;   // 64 hi, 64 lo, 64 rope of a tile, two tiles

}  // namespace low

template <bool Q4>
__global__ void __launch_bounds__(low::kThreads, 1)
    key_weights_e4m3_kernel(const __grid_constant__ CUtensorMap tmap_q, const WeightParams p) {
    using namespace low;
    constexpr int kBytes = Q4 ? kQ4Row : kQ8Row;
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {   // the operands' swizzle counts from 1 KB boundaries
        if (threadIdx.x == 0) raise_dev_error(p.status, DEV_ERR_TIMEOUT);
        return;
    }
    float* qs_s = reinterpret_cast<float*>(smem + OFF_QS);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    uint64_t* empty = full + kSlots;
    uint64_t* q_full = empty + kSlots;
    uint64_t* qr_full = q_full + 1;
    uint64_t* q_free = q_full + 2;
    uint64_t* acc_full = q_full + 3;
    uint64_t* acc_free = acc_full + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_TMEM);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);
    const int warp = threadIdx.x / 32;
    const uint32_t lane = lane_id();

    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&full[i], 128);              // one arrival a lane of four warps: the copies', or its own
            mbar_init(&empty[i], 1);
        }
        mbar_init(q_full, kQueryWarps);
        mbar_init(qr_full, 1);
        mbar_init(q_free, 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 2);              // the issuer: its commit, and that it has seen the query's scales
            mbar_init(&acc_free[i], 4);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    if (Q4 && threadIdx.x < 256)
        reinterpret_cast<uint2*>(smem + OFF_TABLE)[threadIdx.x] =
            threadIdx.x < kQ4Scales ? q4_table(q4_block_scale(threadIdx.x)) : make_uint2(0, 0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    griddep_wait();
    auto wait = [&](uint64_t* bar, uint32_t parity) { return warp_poll(bar, parity, lane, abort_flag, p.status); };

    if (warp < kFirstGather) setmaxnreg_dec<kIssueRegs>();
    if (warp == 0 || warp == 2) {
        // ------------------------------------------------------------ MMA issuers, tiles in turn
        // One look at all barriers: lanes 0-4 the chunks, 5 the query, 6 its rope dims, 7 the accumulator.
        const int mine_of = warp >> 1;
        int gt = 0, qi = 0;
        const uint32_t base = (smem_u32(smem) >> 4) | ((16u >> 4) << 16);
        for_items(p, lane, [&](const Item&, int T) {
            bool used = false;
            for (int t = 0; t < T; ++t, ++gt) {
                if ((gt & 1) != mine_of) continue;
                used = true;
                const int n = kChunks * gt, at = n + (int)lane;
                const uint32_t d = tmem_base + kAccCols * (gt & 1);
                uint64_t* mine = lane < kChunks ? &full[at % kSlots] : lane == 5 ? q_full : lane == 6 ? qr_full : &acc_free[gt & 1];
                const uint32_t parity = lane < kChunks ? at / kSlots & 1 : lane < 7 ? qi & 1 : ((gt >> 1) & 1) ^ 1;
                const int slot0 = n % kSlots;
                uint32_t got = 0;
                bool ok = true;
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    const uint32_t need = 0xe0u | 1u << c;
                    if (ok && (got & need) != need) {
                        got = mbar_poll_warp(mine, parity, lane, 8, need, abort_flag, p.status);
                        ok = got != 0;
                        fence_proxy_async_smem();  // of every lane that saw a barrier, before the lane that issues
                        tc_fence_after();
                        __syncwarp();
                    }
                    if (lane == 0 && ok) {
                        const int slot = slot0 + c - (slot0 + c >= kSlots ? kSlots : 0);
                        const uint32_t a = base + (OFF_K >> 4) + slot * (kBlk >> 4);
                        if (c < 4) {
#pragma unroll
                            for (int k = 0; k < 4; ++k)   // 32 dims a step
                                mma_e4m3_ss_lo(d, a + 2 * k, kDescHi, base + ((OFF_QHL + c * kBlk) >> 4) + 2 * k, kDescHi,
                                               IDESC_E4M3, (c | k) ? 1u : 0u);
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k)   // 16 dims a step
                                mma_bf16_ss_lo(d + 128, a + 2 * k, kDescHi, base + (OFF_QR >> 4) + 2 * k, kDescHi, IDESC_BF16,
                                               k ? 1u : 0u);
                        }
                        mma_commit(&empty[slot]);
                    }
                    __syncwarp();
                }
                if (!ok) return false;
                if (lane == 0) {
                    mbar_arrive(&acc_full[gt & 1]);
                    mma_commit(&acc_full[gt & 1]);
                    if (t >= T - 2) mma_commit(q_free);   // the issuer's last tile of the item
                }
                __syncwarp();
            }
            if (!used) {                           // an item of one tile, the other's: no arrival ahead of its phase
                if (!wait(q_full, qi & 1)) return false;
                if (lane == 0) mbar_arrive(q_free);
                __syncwarp();
            }
            ++qi;
            return true;
        });
    } else if (warp >= kFirstGather && warp < kFirstQuery) {
        // ------------------------------------------------------------ gather: two sets of four warps
        // 8-bit rows: the sets copy every other chunk, eight lanes a row.  4-bit rows: the first expands chunks 0 and 2, the
        // second 1 and 3, a lane its own row.
        setmaxnreg_dec<kGatherRegs>();
        const int quad = warp & 3, set = (warp - kFirstGather) >> 2;
        const uint32_t ring = smem_u32(smem) + OFF_K;
        int n = 0;                                 // the tile's first chunk
        auto free = [&](int c) { return wait(&empty[(n + c) % kSlots], ((n + c) / kSlots & 1) ^ 1); };
        if constexpr (!Q4) {
            const int j = (int)lane & 7, r0 = quad * 32 + (int)(lane >> 3);
            const int r = quad * 32 + (int)lane;   // the row the lane looks up
            Feed feed;
            RowCopy rows(r0, j);
            int row = -1;
            bool has = feed.fetch(p, lane, r), more = has;
            if (has) {
                row = feed.resolve(p);
                more = feed.fetch(p, lane, r);
            }
            for (; has; n += kChunks) {
                rows.point(p, row, kBytes, j, lane);
                if (more) row = feed.resolve(p);
                has = more;
                more = more && feed.fetch(p, lane, r);
                bool ok = true;
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {   // the rope dims follow the latent dims, 128 bytes too
                    if (((n + c) & 1) != set) continue;
                    if (!(ok = ok && free(c))) break;
                    rows.copy(128 * c, ring + (n + c) % kSlots * kBlk);
                    cp_async_arrive_noinc(&full[(n + c) % kSlots]);
                }
                if (!ok) break;
            }
        } else {
            const int r = quad * 32 + (int)lane;   // the lane's row of a tile
            const uint32_t table = smem_u32(smem) + OFF_TABLE;
            Feed feed;
            int row = -1, next = -1;
            uint32_t x[2][16], b[2][2];
            auto load = [&] {                      // both chunks' codes, ahead of the waits for their places
                const uint8_t* src = p.cache + (int64_t)max(row, 0) * kBytes;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = set + 2 * h;
                    ldg_nc_v8(src + 64 * c, x[h]);
                    ldg_nc_v8(src + 64 * c + 32, x[h] + 8);
                    ldg_nc_v2(src + kQ4Codes + 8 * c, b[h][0], b[h][1]);
                }
            };
            bool has = feed.fetch(p, lane, r), more = has;
            if (has) {
                row = feed.resolve(p);
                more = feed.fetch(p, lane, r);
            }
            for (; has; n += kChunks) {
                load();                            // (at the loop's end the loads were waited for there: 56 us for 52)
                if (more) next = feed.resolve(p);
                has = more;
                more = more && feed.fetch(p, lane, r);
                bool ok = true;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int c = set + 2 * h;
                    if (!(ok = ok && free(c))) break;
                    if (row < 0) b[h][0] = b[h][1] = 0xffffffffu;   // zeros
                    const uint32_t dst = ring + (n + c) % kSlots * kBlk + r * 128 + ((r & 7) << 4);
                    uint2 tb = lds_v2(table + 8 * (b[h][0] & 0xff));
#pragma unroll
                    for (int i = 0; i < 8; ++i) {  // a table's load is ahead of the store before it
                        uint2 ahead = tb;
                        if (i < 7) ahead = lds_v2(table + 8 * __byte_perm(b[h][(i + 1) >> 2], 0, 0x4440 + ((i + 1) & 3)));
                        const uint2 u = q4_expand(x[h][2 * i], tb), v = q4_expand(x[h][2 * i + 1], tb);
                        sts_v4(dst ^ (i << 4), u.x, u.y, v.x, v.y);
                        tb = ahead;
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(&full[(n + c) % kSlots]);
                }
                if (ok && ((n ^ set) & 1) == 0) {  // the rope dims by the sets in turn
                    if ((ok = free(4))) {
                        const uint8_t* src = p.cache + (int64_t)max(row, 0) * kBytes + kQ4Rope;
                        const uint32_t dst = ring + (n + 4) % kSlots * kBlk + r * 128 + ((r & 7) << 4);
#pragma unroll
                        for (int i = 0; i < 8; ++i) cp_async_16(dst ^ (i << 4), src + 16 * i, row >= 0 ? 16u : 0u);
                        cp_async_arrive_noinc(&full[(n + 4) % kSlots]);
                    }
                }
                if (!ok) break;
                row = next;
            }
        }
        cp_async_wait_all();
    } else if (warp >= kFirstQuery && warp < kFirstEpi) {
        // ------------------------------------------------------------ queries
        // Eight heads a warp, dims 16 l .. 16 l + 15 a lane, loaded and split before their place comes free.
        setmaxnreg_inc<kQueryRegs>();
        constexpr int kOwn = kH / kQueryWarps;
        const int h0 = (warp - kFirstQuery) * kOwn;
        int qi = 0;
        for_items(p, lane, [&](const Item& I, int) {
            const __nv_bfloat16* src = p.q + ((int64_t)I.row * kH + h0) * kQDim + 16 * lane;
            uint32_t hi[kOwn][4], lo[kOwn][4];
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                const uint4 a = ldg_nc_v4(src + i * kQDim), b = ldg_nc_v4(src + i * kQDim + 8);
                hi[i][0] = a.x, hi[i][1] = a.y, hi[i][2] = a.z, hi[i][3] = a.w;
                lo[i][0] = b.x, lo[i][1] = b.y, lo[i][2] = b.z, lo[i][3] = b.w;
            }
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                const uint32_t w[8] = {hi[i][0], hi[i][1], hi[i][2], hi[i][3], lo[i][0], lo[i][1], lo[i][2], lo[i][3]};
                float amax = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));
                // magnitudes compare as their bit patterns do
                const int e = e4m3_scale_exponent(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax))));
                const float inv = exp2_int(-e);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    split_e4m3x4(bf16_lo(w[2 * k]) * inv, bf16_hi(w[2 * k]) * inv, bf16_lo(w[2 * k + 1]) * inv,
                                 bf16_hi(w[2 * k + 1]) * inv, hi[i][k], lo[i][k]);
                if (lane == 0) qs_s[(qi & (kScalePlaces - 1)) * kH + h0 + i] = p.scale_log2 * exp2_int(e);
            }
            if (!wait(q_free, (qi & 1) ^ 1)) return false;
            if (warp == kFirstQuery && lane == 0) {
                mbar_arrive_expect_tx(qr_full, kQBlk);
                tma_load_2d(smem + OFF_QR, &tmap_q, qr_full, kQ8Latent, I.row * kH);
            }
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                const int h = h0 + i;
                uint8_t* d = smem + OFF_QHL + (int)(lane >> 3) * kBlk + h * 128 + (((int)(lane & 7) ^ (h & 7)) << 4);
                *reinterpret_cast<uint4*>(d) = make_uint4(hi[i][0], hi[i][1], hi[i][2], hi[i][3]);
                *reinterpret_cast<uint4*>(d + kH * 128) = make_uint4(lo[i][0], lo[i][1], lo[i][2], lo[i][3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
            ++qi;
            return true;
        });
    } else if (warp >= kFirstEpi) {
        // ------------------------------------------------------------ epilogue
        setmaxnreg_dec<kEpiRegs>();
        const int quad = warp & 3, set = (warp - kFirstEpi) >> 2;
        const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
        float2* nl = reinterpret_cast<float2*>(smem + OFF_LSE) + (warp - kFirstEpi) * (kH / 2);
        const float2 sr = make_float2(p.scale_log2, p.scale_log2), sixteenth = make_float2(0.0625f, 0.0625f);
        int gt = 0, qi = 0;
        for_items(p, lane, [&](const Item& I, int T) {
            stage_lse(p, I, nl, lane);
            const float2* qs = reinterpret_cast<const float2*>(qs_s + (qi & (kScalePlaces - 1)) * kH);
            for (int t = 0; t < T; ++t, ++gt) {
                if ((gt & 1) != set) continue;
                const int key = key_at(p, I, I.slot0 + t * kTile + quad * 32 + (int)lane);
                int row = key_row(p, p.given, I, key);
                if (key >= 0 && row < 0) raise_dev_error(p.status, DEV_ERR_BOUNDS);
                if (row >= 0 && !p.pages.table) row = (int)((int64_t)I.batch * p.Nmax + key);
                const float c = row >= 0 ? __ldg(p.cache_scale + row) : 0.f;
                if (!wait(&acc_full[gt & 1], (gt >> 1) & 1)) return false;
                tc_fence_after();
                const uint32_t d = tmem_base + lane_addr + kAccCols * (gt & 1);
                float2 sum = make_float2(0.f, 0.f);
                // Eight heads' columns are loaded while those before are summed, and the accumulator is free when the last have
                // come (4096 queries 0.75 -> 0.70 ms).  (The registers pass through an empty statement after the wait, so that no use comes before it.)
                uint32_t v[2][3][8];
                auto load = [&](int h) {
#pragma unroll
                    for (int part = 0; part < 3; ++part) tmem_ld8(d + 64 * part + h, v[h / 8 & 1][part]);
                };
                load(0);
#pragma unroll
                for (int h = 0; h < kH; h += 8) {
                    uint32_t (&u)[3][8] = v[h / 8 & 1];
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 24; ++k) asm volatile("" : "+r"(u[k / 8][k % 8]));
                    if (h < kH - 8) {
                        load(h + 8);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&acc_free[gt & 1]);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 x = __ffma2_rn(__ffma2_rn(pair(u[1], k), sixteenth, pair(u[0], k)),
                                                    __fmul2_rn(qs[h / 2 + k], make_float2(c, c)),
                                                    __ffma2_rn(pair(u[2], k), sr, nl[h / 2 + k]));
                        sum = __fadd2_rn(sum, make_float2(ex2_approx(x.x), ex2_approx(x.y)));
                    }
                }
                add_weight(p, I, key, row, sum);
            }
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

using Kernel = void (*)(const CUtensorMap, const WeightParams);

template <Kernel KERNEL, int THREADS, int SMEM>
dsa_status_t launch(const WeightParams& p, cudaStream_t stream) {
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> done[kMaxDevices];
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return DSA_ERR_CUDA;
    if (!done[dev].load(std::memory_order_acquire)) {
        const dsa_status_t st = ensure_smem_attr(reinterpret_cast<const void*>(KERNEL), SMEM);
        if (st != DSA_OK) return st;
        done[dev].store(true, std::memory_order_release);
    }
    CUtensorMap tq;
    const dsa_status_t st = make_tmap_bf16_2d(&tq, p.q, kQDim, (uint64_t)p.rows * kH, kQDim * 2, 64, kH);
    if (st != DSA_OK) return st;
    const int sms = device_sm_count();
    if (launch_pdl(KERNEL, dim3(p.n_items < sms ? p.n_items : sms), dim3(THREADS), SMEM, stream, tq, p) != cudaSuccess)
        return DSA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

dsa_status_t launch_format(int format, const WeightParams& p, cudaStream_t stream) {
    return format == DSA_ROWS_BF16 ? launch<key_weights_bf16_kernel, wide::kThreads, wide::kSmemBytes>(p, stream)
           : format == DSA_ROWS_Q8 ? launch<key_weights_e4m3_kernel<false>, low::kThreads, low::kSmemBytes>(p, stream)
                                   : launch<key_weights_e4m3_kernel<true>, low::kThreads, low::kSmemBytes>(p, stream);
}

// Parts of a query's tiles: as many as give each SM one item at most; whole queries where they are more than half as many as the
// SMs.  A cut costs another load of the query and no merge, so finer ones could even out what this leaves idle: half of the
// SMs at 77 queries on 152, almost all of a second round at 153 (decode over bf16 / 8-bit / 4-bit rows, us: 77 sequences
// 45 / 32 / 43, 152 65 / 44 / 51, 153 95 / 65 / 87, 304 123 / 79 / 96).
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
    p.scale_log2 = scale * kLog2e;
    p.status = device_status_ptr();
    p.pages = p.given = pages;
    return p;
}

}  // namespace

// A prefill over the 4-bit cache expands its rows to 8-bit ones first where the queries select each key six times or more:
// a selected key then costs 0.085 ns in place of 0.125, a key of the cache 0.2 ns and the launch 2 us.  Direct / expanded, us: 16
// queries of 2048 of 2k keys 13.0 / 13.0, 32 17.7 / 15.6; 64 of 8k 26 / 22; 304 of 16k 80 / 59, of 65k (9.5 times each) 82 / 68;
// 608 of 131k (9.5) 167 / 138, of 262k (4.8) 183 / 168, of 524k (2.4) 196 / 222; 2432 of 262k 698 / 507; 4096 of 2M (4) 1391 / 1396.
bool key_weights_expands(int format, int L, int N, int top_k) {
    return format == DSA_ROWS_Q4 && (long long)L * top_k >= 6LL * N + 49152;
}

size_t key_weights_workspace(bool expand, int N) {
    const size_t sums = (size_t)N * 8;
    return expand ? round_up(sums) + round_up((size_t)N * kQ8Row) + (size_t)N * sizeof(float) : sums;
}

dsa_status_t launch_key_weights_prefill(int format, bool expand, const void* q, const void* cache, const float* cache_scale,
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
    dsa_status_t st = DSA_OK;
    if (expand) {
        uint8_t* rows = static_cast<uint8_t*>(workspace) + round_up((size_t)N * 8);
        float* scales = reinterpret_cast<float*>(rows + round_up((size_t)N * kQ8Row));
        if ((st = launch_cache_expand_q4(cache, cache_scale, N, rows, scales, pages, stream)) != DSA_OK) return st;
        p.cache = rows;
        p.cache_scale = scales;
        p.pages = PageTable{};
        format = DSA_ROWS_Q8;
    }
    if ((st = launch_format(format, p, stream)) != DSA_OK) return st;
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
