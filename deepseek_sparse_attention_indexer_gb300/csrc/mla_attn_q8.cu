// mla_attn_q8.cu -- sparse absorbed-MLA attention over the 8-bit latent cache.
//
// What it computes (the method's passages are cited in mla_attn.cu): with the row's scale c_t,
//   s[h,t] = scale * (c_t * q[h,0:512] . e4m3_t + q[h,512:576] . rope_t),  p = softmax_t(s) in float32,
//   out[h,:] = sum_t p[h,t] * c_t * e4m3_t.
//
// How (GB300 design):
//   * The rows go to the tensor core as they lie in the cache: both products run on e4m3 operands,
//     nothing is widened.  As in the bf16 kernel, keys sit on the 128 TMEM lanes: S^T = K . Q^T and
//     O^T = V^T . P^T (M = 128 keys / latent dims), the gathered tile is stored once with the 128-byte
//     swizzle and read K-major by QK and MN-major by PV.
//   * A bf16 query has 8 significant bits, an e4m3 number 4: a query is the sum of two e4m3 numbers,
//     hi + lo / 16 (times a power of two a head), exactly so down to 2^-14 of the head's largest
//     element and within 2^-22 of it below.  hi and lo of the 64 heads stand next to each other as one
//     N = 128 operand, so QK over 32 dims is one MMA; the softmax adds the two halves.  The rope
//     dims are a bf16 product of their own (their rows are not scaled).
//   * The probabilities are split the same way, P' = hi + lo / 16, lo's factor applied by the
//     block-scaled MMA (constant scale bytes in TMEM), both into one accumulator: 8 significant bits, as
//     the bf16 kernel's probabilities have.  The row's scale is folded in before the split:
//     P' = 2^(t - m) with t = log2(e) s + log2(c), so that e4m3's range (2^-9 .. 448, and 2^-13 with
//     lo) is spent on the weights that the value sum sees; the row sum divides it out again.
//   * The reference m of a head is set from the query's first tile so that its largest P' is 2^5.5,
//     and moved when a later one would pass 2^8.75 (e4m3 ends at 448): a higher start would leave
//     less room and rescale O^T more often, a lower one would lose the small weights sooner (a
//     weight keeps 8 bits down to 2^-11.5 of the largest at worst, 2^-14.8 at best).
//   * Shared memory holds 7 latent chunks (128 keys x 128 dims, 16 KB) as a ring, one rope block and
//     one P^T block beside the 72 KB query: tile t + 1 is gathered, and its QK issued, while tile t is
//     in its softmax and PV.  Chunk 3 of tile t + 1 takes the place of chunk 0 of tile t.
//   * Roles (19 warps): warp 0 issues QK, warps 1 and 2 PV (chunks 0, 2 and 1, 3), 16 worker warps
//     gather (cp.async), convert the query, do the softmax and write the output.  Two PV issuers: one
//     thread reaches an N = 64 scaled MMA every ~80 cycles, two one every ~52, which is the rate of the
//     operands' shared-memory reads (6 KB at 128 B a cycle); one N = 128 issuer reaches its 64.
//   * Decode splits a sequence's selected keys over CTAs and writes partial (normalised output, lse)
//     pairs; the bf16 path's merge kernel joins them.
#include <cuda.h>

#include <cmath>

#include "dsa_q8.cuh"
#include "mla_attn_common.cuh"

namespace dsa {

namespace {

constexpr int kBlk = 128 * 128;                    // 16 KB: 128 rows of 128 bytes
constexpr int kChunks = kQ8Latent / 128;           // 4 latent chunks of 128 dims a tile
constexpr int kStages = 2;                         // tiles in shared memory
constexpr int kRopeHalf = 128 * 64;                // 8 KB: 128 rows of 32 rope dims
constexpr int kPvIssuers = 2;
constexpr int kGatherWarps = 8;                    // rows and query
constexpr int kWorkerWarps = 16;                   // softmax and output
constexpr int kWorkers = kWorkerWarps * 32;
// warp 0 QK, warps 1-2 PV, warp 3 none; warps 4-11 gather; warps 12-27 workers.  The register split is by
// warpgroups of four warps out of what the launch holds: 896 threads of 72 registers.
constexpr int kFirstGather = 4;
constexpr int kFirstWorker = kFirstGather + kGatherWarps;
constexpr int kThreads = 32 * (kFirstWorker + kWorkerWarps);
constexpr int kLaunchRegs = 72, kIssueRegs = 56, kGatherRegs = 64, kWorkerRegs = 80;
static_assert(kThreads * kLaunchRegs >=
                  32 * (kFirstGather * kIssueRegs + kGatherWarps * kGatherRegs + kWorkerWarps * kWorkerRegs),
              "registers of the CTA");
constexpr int kRowsPerWarp = kTile / kGatherWarps; // 16 rows of a tile, 8 query heads a gather warp
constexpr int kHG = kH / (kWorkerWarps / 4);       // 16 heads a worker warp
constexpr int kGroupThreads = 4 * 32;              // the four warps sharing a head group
constexpr uint32_t kGatherBar = 7;                 // named barriers: 1, 2 workers, 3-6 head groups, 7 gather
static_assert(kHG == 16 && kWorkerWarps == 16, "warp_transpose_reduce16 takes a head group of 16");

constexpr float kFirstTop = 5.5f;                  // log2 of the first tile's largest P'
constexpr float kMostTop = 8.75f;                  // log2 of the largest P' (430 <= 448)
constexpr float kNoRef = 3.0e38f;                  // -m before the reference is set (finite: see mla_attn.cu)

// smem layout
constexpr int OFF_QHL = 0;                         // 4 chunks x (64 hi rows, 64 lo rows) x 128 B
constexpr int OFF_QR = OFF_QHL + kChunks * kBlk;   // rope dims of 64 heads: two halves of 64 rows x 64 B
constexpr int OFF_LAT = OFF_QR + kH * 128;         // 2 tiles x 4 latent chunks
constexpr int OFF_ROPE = OFF_LAT + kStages * kChunks * kBlk;   // half of a tile's rope dims
constexpr int OFF_P = OFF_ROPE + kRopeHalf;        // 128 keys x (64 hi | 64 lo)
constexpr int OFF_SC = OFF_P + kBlk;               // float [128]: scales of the tile's rows, 0 = no key
constexpr int OFF_QS = OFF_SC + kTile * 4;         // float [3][64]: scale * log2(e) * 2^k of a query's heads
constexpr int OFF_RED = OFF_QS + 3 * kH * 4;       // float [4][64]
constexpr int OFF_MNEG = OFF_RED + 4 * kH * 4;     // float [64]: minus the references
constexpr int OFF_ALPHA = OFF_MNEG + kH * 4;       // float [64]: rescale factors; at an item's end 1 / l
constexpr int OFF_BAR = OFF_ALPHA + kH * 4;
// barriers: full[8], free[8], rope_full, rope_free, s_full, s_free, p_full, q_full
constexpr int kSlots = kStages * kChunks;
constexpr int kBars = 2 * kSlots + 6;
constexpr int OFF_TMEM = OFF_BAR + kBars * 8;
constexpr int OFF_ABORT = OFF_TMEM + 4;
constexpr int kSmemBytes = OFF_ABORT + 4;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t TM_S = 0;                       // S^T: 64 columns hi, 64 lo
constexpr uint32_t TM_R = 128;                     // the rope product, 64 columns
constexpr uint32_t TM_O = 192;                     // O^T chunk c at TM_O + 64 c
constexpr uint32_t TM_ONE = 448;                   // scale bytes 2^0
constexpr uint32_t TM_LO = 464;                    // scale bytes 2^-4

// Operands: 128-byte swizzle, 8-row groups 1 KB apart.  The descriptors' high words are the same; the
// low words (address, leading offset) are sums that stay below the address field's end (see sdesc).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescHiRope = (512u >> 4) | (1u << 14) | (4u << 29);   // rope halves: 64-byte rows and swizzle
constexpr uint32_t IDESC_QK = idesc_e4m3_f32(128, 128, false, false);
constexpr uint32_t IDESC_ROPE = idesc_bf16_f32(128, 64, false, false);
constexpr uint32_t IDESC_PV = idesc_e4m3_scaled_f32(128, 64, true, true);

__device__ float g_unit_scale = 1.f;               // scale of a row whose page lies outside the pool (zeros)

struct AttnQ8Params : AttnShape {
    const __nv_bfloat16* q;    // [rows][64][576]
    const uint8_t* cache;      // 640-byte rows
    const float* cache_scale;
    void* out;                 // final: [rows][64][512], float32 or bf16 (out_f32)
    int out_f32;
    float* lse;                // final: [rows][64] or nullptr
    float* part_o;             // partial: [rows][nsplit][64][512]
    float* part_lse;           // partial: [rows][nsplit][64]
    float scale_log2;          // scale * log2(e)
    int32_t* status;           // device error word
    PageTable pages;           // paged cache (pages.table == nullptr: dense rows)
};

// log2 on the special-function unit; exact for the powers of two that the cache holds.
__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two values as hi + lo / 16 in e4m3 (|x| <= 448): hi in the low 16 bits of the result, lo in the
// high ones.  The half-precision step between keeps 11 bits, the difference x - hi is exact.
__device__ __forceinline__ uint32_t split_e4m3x2(float x, float y) {
    uint32_t h, back, r;
    uint16_t hi, lo;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(y), "f"(x));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(h));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(hi));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(back));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(0x4c004c00u));   // 16
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lo) : "r"(r));
    return (uint32_t)hi | ((uint32_t)lo << 16);
}
__device__ __forceinline__ uint32_t lows(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
__device__ __forceinline__ uint32_t highs(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }

// Transposes over groups of G lanes.  Lane j of a group holds N words (N / G to each lane of the group, in
// order); afterwards word i * (N / G) + k is word j * (N / G) + k of the group's lane i.
template <int N, int G>
__device__ __forceinline__ void transpose_words(uint32_t (&v)[N], uint32_t lane) {
    constexpr int K = N / G;
#pragma unroll
    for (int s = G / 2; s; s >>= 1) {        // swap the off-diagonal halves of every 2s x 2s block
        const bool up = lane & s;
#pragma unroll
        for (int b = 0; b < G; ++b) {
            if (b & s) continue;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                uint32_t &lo = v[b * K + k], &hi = v[(b + s) * K + k];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, s);
                if (up) lo = got; else hi = got;
            }
        }
    }
}

template <bool PARTIAL>
__global__ void __launch_bounds__(kThreads, 1) mla_attn_q8_kernel(const AttnQ8Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {   // the operands' swizzle counts from 1 KB boundaries; there is no room to round up
        if (threadIdx.x == 0) raise_dev_error(p.status, DEV_ERR_TIMEOUT);
        return;
    }
    float* sc_s = reinterpret_cast<float*>(smem + OFF_SC);
    float* qs_s = reinterpret_cast<float*>(smem + OFF_QS);
    float* red = reinterpret_cast<float*>(smem + OFF_RED);
    float* m_neg = reinterpret_cast<float*>(smem + OFF_MNEG);
    float* alpha_s = reinterpret_cast<float*>(smem + OFF_ALPHA);
    float* invl_s = alpha_s;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    uint64_t* freed = full + kSlots;
    uint64_t* rope_full = freed + kSlots;
    uint64_t* rope_free = rope_full + 1;
    uint64_t* s_full = rope_full + 2;
    uint64_t* s_free = rope_full + 3;
    uint64_t* p_full = rope_full + 4;
    uint64_t* q_full = rope_full + 5;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_TMEM);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);

    const int warp = threadIdx.x / 32;
    const uint32_t lane = lane_id();

    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&full[i], kGatherWarps * 32);   // one cp.async arrival per gather thread
            mbar_init(&freed[i], 1);                  // the commit of the PV issuer that consumed the chunk
        }
        mbar_init(rope_full, kGatherWarps * 32);
        mbar_init(rope_free, 1);
        mbar_init(s_full, 2);                   // the QK issuer: its commit, and that it has seen the rows' scales
        mbar_init(s_free, kWorkerWarps);
        mbar_init(p_full, kWorkerWarps);
        mbar_init(q_full, kGatherWarps);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    if (warp >= kFirstWorker && warp < kFirstWorker + 4) {   // four warps: all four lane quadrants
        uint32_t v[16];
        const uint32_t a = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0x7f7f7f7fu;
        tmem_st16(a + TM_ONE, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0x7b7b7b7bu;
        tmem_st16(a + TM_LO, v);
        tmem_st_wait();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();                 // inputs and outputs may belong to the previous kernel until here

    // Chunk c of the CTA's g-th tile lies in slot 4 (g % 2) + c; the slot's barriers are in their use g / 2.
    if (warp < kFirstGather) setmaxnreg_dec<kIssueRegs>();
    if (warp == 0) {
        // ------------------------------------------------------------ QK issuer
        int gt = 0, qi = 0;
        bool ok = true;
        for (int s = 0; ok; ++s) {
            const int item = nth_item(p, s);
            if (item == -1) break;
            if (item < 0) continue;
            const Item I = decode_item(p, item);
            const int T = item_tiles(p, I, lane);
            if (T == 0) continue;
            if (lane == 0) {
                const uint32_t base = (smem_u32(smem) >> 4) | ((16u >> 4) << 16);   // leading offset: one atom wide
                ok = mbar_wait_clk<true>(q_full, qi & 1, abort_flag, p.status);
                for (int t = 0; ok && t < T; ++t, ++gt) {
                    // the workers have read the previous tile's S^T
                    if (!(ok = mbar_wait_clk<true>(s_free, (gt & 1) ^ 1, abort_flag, p.status))) break;
                    tc_fence_after();
                    const uint32_t lat = base + (OFF_LAT >> 4) + (gt & 1) * (kChunks * kBlk >> 4);
                    // first half of the rope dims; the second half takes its place while the chunks run
#pragma unroll
                    for (int j = 0; j < 2 + kChunks; ++j) {
                        if (j == 0 || j == 1 + kChunks) {
                            const int half = j ? 1 : 0;
                            if (!(ok = mbar_wait_clk<true>(rope_full, half, abort_flag, p.status))) break;
                            if (half) mbar_arrive(s_full);
                            fence_proxy_async_smem();
#pragma unroll
                            for (int kk = 0; kk < 2; ++kk)
                                mma_bf16_ss_lo(tmem_base + TM_R, base + (OFF_ROPE >> 4) + 2 * kk, kDescHiRope,
                                               base + ((OFF_QR + half * kH * 64) >> 4) + 2 * kk, kDescHiRope, IDESC_ROPE,
                                               (half | kk) ? 1u : 0u);
                            if (!half) mma_commit(rope_free);
                        } else {
                            const int c = j - 1;
                            if (!(ok = mbar_wait_clk<true>(&full[4 * (gt & 1) + c], (gt >> 1) & 1, abort_flag, p.status))) break;
                            fence_proxy_async_smem();
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)   // 32 dims a step
                                mma_e4m3_ss_lo(tmem_base + TM_S, lat + c * (kBlk >> 4) + 2 * kk, kDescHi,
                                               base + (OFF_QHL >> 4) + c * (kBlk >> 4) + 2 * kk, kDescHi, IDESC_QK,
                                               (c | kk) ? 1u : 0u);
                        }
                    }
                    if (ok) mma_commit(s_full);
                }
                ++qi;
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        }
    } else if (warp <= kPvIssuers) {
        // ------------------------------------------------------------ PV issuers
        const int iss = warp - 1;
        int gt = 0;
        bool ok = true;
        for (int s = 0; ok; ++s) {
            const int item = nth_item(p, s);
            if (item == -1) break;
            if (item < 0) continue;
            const Item I = decode_item(p, item);
            const int T = item_tiles(p, I, lane);
            if (lane == 0) {
                // A = V^T MN-major: 128 dims a row, 8-key groups 1 KB apart; B = P^T MN-major, hi at byte 0 of a
                // row, lo at byte 64
                const uint32_t base = (smem_u32(smem) >> 4) | ((uint32_t)(kBlk >> 4) << 16);
                for (int t = 0; ok && t < T; ++t, ++gt) {
                    if (!(ok = mbar_wait_clk<true>(p_full, gt & 1, abort_flag, p.status))) break;
                    tc_fence_after();
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int c = iss + 2 * j;
                        const uint32_t slot = 4u * (uint32_t)(gt & 1) + (uint32_t)c;
                        const uint32_t a = base + (OFF_LAT >> 4) + slot * (kBlk >> 4);
                        const uint32_t d = tmem_base + TM_O + 64 * (uint32_t)c;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {     // 32 keys (four 8-key groups, 4 KB) a step
                            const uint32_t b = base + (OFF_P >> 4) + kk * (4096 >> 4);
                            mma_e4m3_scaled_ss_lo(d, a + kk * (4096 >> 4), kDescHi, b, kDescHi, IDESC_PV,
                                                  tmem_base + TM_ONE, tmem_base + TM_ONE, (t | kk) ? 1u : 0u);
                            mma_e4m3_scaled_ss_lo(d, a + kk * (4096 >> 4), kDescHi, b + (64 >> 4), kDescHi, IDESC_PV,
                                                  tmem_base + TM_ONE, tmem_base + TM_LO, 1u);
                        }
                        mma_commit(&freed[slot]);
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        }
    } else if (warp >= kFirstGather && warp < kFirstWorker) {
        // ------------------------------------------------------------ gather
        setmaxnreg_dec<kGatherRegs>();
        const int gw = warp - kFirstGather;       // 0..7: rows 16 gw .. 16 gw + 15 of a tile, query heads 8 gw ..
        const uint32_t smem_base = smem_u32(smem);
        // One thread polls, a named barrier releases the eight warps.  (A thread suspended in try_wait was seen
        // to resume 800 to 3400 cycles after the phase had completed; threads that all poll take the issue slots
        // of the softmax.)  The answer is the same in every warp: all leave together when a wait gives up.
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            bool ok = true;
            if (threadIdx.x == 32 * kFirstGather) ok = mbar_wait_clk<true>(bar, parity, abort_flag, p.status);
            return named_bar_and(kGatherBar, kGatherWarps * 32, ok);
        };
        // Lanes 0..15 carry their row through three stages: the selected key (fetch), its cache row (resolve: a
        // page lookup when paged), the copies.  Each stage runs one tile ahead of the next, so that its loads
        // are in flight during the copies of the tile before.
        int f_s = 0, f_T = 0;                     // next item of the CTA; tiles of the current one still to fetch
        const int32_t* f_idx = p.idx;             // this lane's next slot, and how many slots are left from it on
        int f_left = 0, f_batch = 0, f_bound = 0;
        int f_key = -1, f_first = -1;             // the fetched tile's key; its query when it is an item's first tile
        auto fetch = [&]() -> bool {
            f_first = -1;
            while (f_T == 0) {
                const int it = nth_item(p, f_s++);
                if (it == -1) return false;
                if (it < 0) continue;
                const Item I = decode_item(p, it);
                f_T = item_tiles(p, I, lane);
                f_idx = p.idx + (int64_t)I.row * p.top_k + I.slot0 + kRowsPerWarp * gw + (int)lane;
                f_left = lane < kRowsPerWarp ? I.slot_end - I.slot0 - kRowsPerWarp * gw - (int)lane : 0;
                f_batch = I.batch;
                f_bound = I.bound;
                f_first = I.row;
                if (lane == 0)                    // the warp's heads of the query, into L2
                    l2_prefetch_bulk(p.q + ((int64_t)I.row * kH + kH / kGatherWarps * gw) * DSA_QK_DIM,
                                     kH / kGatherWarps * DSA_QK_DIM * 2);
            }
            f_key = f_left > 0 ? __ldg(f_idx) : -1;
            f_idx += kTile;
            f_left -= kTile;
            --f_T;
            return true;
        };
        // cache row of the fetched key; -1: no key, -2: a page outside the pool (a row of zeros)
        auto resolve = [&]() -> int {
            const int j = f_key;
            if (j < 0) return -1;
            if (j >= f_bound) {
                raise_dev_error(p.status, DEV_ERR_BOUNDS);
                return -1;
            }
            if (p.pages.table) {
                const int row = (int)paged_row(p.pages, f_batch, j);
                if (row < 0) raise_dev_error(p.status, DEV_ERR_BOUNDS);
                return row < 0 ? -2 : row;
            }
            return (int)((int64_t)f_batch * p.Nmax + j);
        };
        // One 128-byte block (blk 0..3 latent, 4 rope) of the warp's 16 rows: a warp instruction copies a block of
        // four different rows, 8 lanes a row.
        const int ci = (int)(lane >> 3), cc = (int)(lane & 7);
        const uint32_t dst0 = smem_base + (uint32_t)((kRowsPerWarp * gw + ci) * 128);
        auto copy_chunk = [&](int row, int g, int c) -> bool {      // chunk c of the CTA's g-th tile
            const uint32_t slot = 4u * (uint32_t)(g & 1) + (uint32_t)c;
            if (!wait(&freed[slot], ((g >> 1) & 1) ^ 1)) return false;
#pragma unroll
            for (int i = 0; i < kRowsPerWarp / 4; ++i) {
                const int r = __shfl_sync(0xffffffffu, row, 4 * i + ci);
                cp_async_16(dst0 + OFF_LAT + slot * kBlk + i * 512 + ((cc ^ (4 * (i & 1) + ci)) << 4),
                            p.cache + (r < 0 ? 0 : (int64_t)r * kQ8Row + c * 128 + cc * 16), r < 0 ? 0u : 16u);
            }
            cp_async_arrive_noinc(&full[slot]);
            return true;
        };
        // half of the rope dims: 64-byte rows, 4 lanes a row, 8 rows a warp instruction
        auto copy_rope = [&](int row, int half) {
#pragma unroll
            for (int i = 0; i < kRowsPerWarp / 8; ++i) {
                const int tr = 8 * i + (int)(lane >> 2);
                const int r = __shfl_sync(0xffffffffu, row, tr);
                const int pc = (int)(lane & 3);
                cp_async_16(smem_base + OFF_ROPE + (kRowsPerWarp * gw + tr) * 64 + ((pc ^ ((tr >> 1) & 3)) << 4),
                            p.cache + (r < 0 ? 0 : (int64_t)r * kQ8Row + kQ8Latent + half * 64 + pc * 16), r < 0 ? 0u : 16u);
            }
        };
        // Query head h: lane l holds dims 8l.. and 256 + 8l.., and rope dims 2l, 2l + 1.
        struct Head {
            uint4 w[2];
            uint32_t pe;
        };
        auto load_head = [&](int row, int h) -> Head {
            const __nv_bfloat16* src = p.q + ((int64_t)row * kH + h) * DSA_QK_DIM;
            Head q;
            q.w[0] = ldg_nc_v4(src + 8 * lane);
            q.w[1] = ldg_nc_v4(src + 256 + 8 * lane);
            q.pe = __ldg(reinterpret_cast<const uint32_t*>(src + kQ8Latent) + lane);
            return q;
        };
        auto convert_head = [&](const Head& q, int qbuf, int h) {
            const uint32_t w[8] = {q.w[0].x, q.w[0].y, q.w[0].z, q.w[0].w, q.w[1].x, q.w[1].y, q.w[1].z, q.w[1].w};
            float amax = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));
            // magnitudes compare as their bit patterns do
            const int e = e4m3_scale_exponent(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax))));
            const float inv = exp2_int(-e);
            const uint32_t swz = (uint32_t)((((lane & 15) >> 1) ^ (h & 7)) << 4) + (lane & 1) * 8;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t s[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) s[k] = split_e4m3x2(bf16_lo(w[4 * b + k]) * inv, bf16_hi(w[4 * b + k]) * inv);
                uint8_t* d = smem + OFF_QHL + (2 * b + (int)(lane >> 4)) * kBlk + h * 128 + swz;
                *reinterpret_cast<uint2*>(d) = make_uint2(lows(s[0], s[1]), lows(s[2], s[3]));
                *reinterpret_cast<uint2*>(d + 64 * 128) = make_uint2(highs(s[0], s[1]), highs(s[2], s[3]));
            }
            *reinterpret_cast<uint32_t*>(smem + OFF_QR + (lane >> 4) * (kH * 64) + h * 64 +
                                         ((((lane & 15) >> 2) ^ ((h >> 1) & 3)) << 4) + (lane & 3) * 4) = q.pe;
            if (lane == 0) qs_s[qbuf * kH + h] = p.scale_log2 * exp2_int(e);
        };

        bool has0 = fetch(), has1;                // tile being copied; tile fetched
        int row0 = has0 ? resolve() : -1, first0 = f_first;
        has1 = has0 && fetch();
        int qbuf = 0;
        for (int g = 0; has0; ++g) {
            const int row1 = has1 ? resolve() : -1, first1 = f_first;
            bool ok = true;
#pragma unroll
            for (int c = 0; c < kChunks; ++c) ok = ok && copy_chunk(row0, g, c);
            // QK of the previous tile is complete: the rope block, and after an item's last tile the query, are free
            if (ok && g > 0) ok = wait(s_full, (g - 1) & 1);
            if (!ok) break;
            copy_rope(row0, 0);
            cp_async_arrive_noinc(rope_full);
            if (first0 >= 0) {
                constexpr int kHeads = kH / kGatherWarps;
                Head q = load_head(first0, kHeads * gw);
#pragma unroll 1
                for (int i = 0; i < kHeads; ++i) {
                    const Head next = load_head(first0, kHeads * gw + min(i + 1, kHeads - 1));
                    convert_head(q, qbuf, kHeads * gw + i);
                    q = next;
                }
                qbuf = qbuf == 2 ? 0 : qbuf + 1;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(q_full);
            }
            // the first half is consumed: QK of this tile has begun, so the workers have read the scales before
            if (!wait(rope_free, g & 1)) break;
            copy_rope(row0, 1);
            if (lane < kRowsPerWarp)
                cp_async_4(smem_base + OFF_SC + (kRowsPerWarp * gw + lane) * 4,
                           row0 >= 0 ? p.cache_scale + row0 : &g_unit_scale, row0 == -1 ? 0u : 4u);
            cp_async_arrive_noinc(rope_full);
            row0 = row1;
            has0 = has1;
            first0 = first1;
            has1 = has1 && fetch();
        }
        cp_async_wait_all();
    } else if (warp >= kFirstWorker) {
        // ------------------------------------------------------------ workers
        setmaxnreg_inc<kWorkerRegs>();
        const int ww = warp - kFirstWorker;       // 0..15
        const int quad = warp & 3;                // TMEM lane quadrant this warp may access
        const int hg = ww >> 2;                   // head group: heads h0 .. h0 + 15
        const int h0 = hg * kHG;
        const uint32_t group_bar = 3 + (uint32_t)hg;
        const int tid = ww * 32 + (int)lane;      // 0..511
        const int key = quad * 32 + (int)lane;    // TMEM lane == key row of the tile == dim row of O^T
        const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
        // Spinning waits, as in the gather: of one thread for all workers (the answer is common), or of one lane for
        // its warp.
        auto wait_all = [&](uint64_t* bar, uint32_t parity) -> bool {
            bool ok = true;
            if (tid == 0) ok = mbar_wait_clk<true>(bar, parity, abort_flag, p.status);
            return named_bar_and(1, kWorkers, ok);
        };
        auto pv_done = [&](int g) -> bool {           // both PV issuers' last chunk of tile g is consumed
            bool ok = true;
            if (lane == 0) {
                const uint32_t par = (g >> 1) & 1;
                ok = mbar_wait_clk<true>(&freed[4 * (g & 1) + 2], par, abort_flag, p.status) &&
                     mbar_wait_clk<true>(&freed[4 * (g & 1) + 3], par, abort_flag, p.status);
            }
            __syncwarp();
            return ok;
        };

        // ---- items.  One without a selected key gets zeros and lse = -inf here.
        int n_s = 0;
        Item nI{};
        int nT = 0;
        auto store_lse = [&](const Item& I, int h, float v) {
            if (PARTIAL)
                p.part_lse[((int64_t)I.row * p.nsplit + I.split) * kH + h] = v;
            else if (p.lse)
                p.lse[(int64_t)I.row * kH + h] = v;
        };
        auto next_item = [&]() -> bool {
            for (;;) {
                const int it = nth_item(p, n_s++);
                if (it == -1) return false;
                if (it < 0) continue;
                nI = decode_item(p, it);
                nT = item_tiles(p, nI, lane);
                if (nT > 0) return true;
                if (tid < kH) store_lse(nI, tid, -INFINITY);
                if (PARTIAL) {
                    float* d = p.part_o + ((int64_t)nI.row * p.nsplit + nI.split) * (kH * kDv);
                    for (int i = tid; i < kH * kDv; i += kWorkers) d[i] = 0.f;
                } else if (p.out_f32) {
                    float* d = static_cast<float*>(p.out) + (int64_t)nI.row * (kH * kDv);
                    for (int i = tid; i < kH * kDv; i += kWorkers) d[i] = 0.f;
                } else {
                    __nv_bfloat16* d = static_cast<__nv_bfloat16*>(p.out) + (int64_t)nI.row * (kH * kDv);
                    for (int i = tid; i < kH * kDv; i += kWorkers) d[i] = __float2bfloat16_rn(0.f);
                }
            }
        };

        // `gok` is the thread's wait status: a wait that gives up does not change the control flow inside an item
        // (all workers keep meeting the same named barriers); the consensus barrier at the item's end takes all
        // out together.
        bool gok = true;
        bool more = next_item();
        bool failed = false;
        int gt = 0;                               // tiles done by this CTA
        int qbuf = 0;                             // the item's query scales
        while (more && !failed) {
            const Item I = nI;
            const int T = nT;
            more = next_item();
            named_bar_sync(1, kWorkers);          // the previous item's readers of m_neg / invl are done
            if (tid < kH) m_neg[tid] = kNoRef;
            float2 l2[kHG / 2];                   // row sums of heads (h0 + 2i, h0 + 2i + 1)
#pragma unroll
            for (int i = 0; i < kHG / 2; ++i) l2[i] = make_float2(0.f, 0.f);
            named_bar_sync(1, kWorkers);
            for (int t = 0; t < T; ++t, ++gt) {
                gok = wait_all(s_full, gt & 1) && gok;
                tc_fence_after();
                float2 t2[kHG / 2];               // log2(e) s + log2(c): the exponents before the reference
                const float c = sc_s[key];
                {
                    uint32_t hi[kHG], lo[kHG], ro[kHG];
                    tmem_ld16(tmem_base + lane_addr + TM_S + h0, hi);
                    tmem_ld16(tmem_base + lane_addr + TM_S + 64 + h0, lo);
                    tmem_ld16(tmem_base + lane_addr + TM_R + h0, ro);
                    tmem_ld_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_free);
                    const float lc = c > 0.f ? lg2_approx(c) : -INFINITY;   // no key: weight 0
                    const float2 lc2 = make_float2(lc, lc), c2 = make_float2(c, c);
                    const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
                    const float2 sixteenth = make_float2(0.0625f, 0.0625f);
#pragma unroll
                    for (int i = 0; i < kHG / 2; ++i) {
                        const float2 a = make_float2(__uint_as_float(hi[2 * i]), __uint_as_float(hi[2 * i + 1]));
                        const float2 b = make_float2(__uint_as_float(lo[2 * i]), __uint_as_float(lo[2 * i + 1]));
                        const float2 r = make_float2(__uint_as_float(ro[2 * i]), __uint_as_float(ro[2 * i + 1]));
                        const float2 qs = reinterpret_cast<const float2*>(qs_s + qbuf * kH + h0)[i];
                        t2[i] = __ffma2_rn(__ffma2_rn(b, sixteenth, a), __fmul2_rn(qs, c2), __ffma2_rn(r, sl2, lc2));
                    }
                }
                float2 e2[kHG / 2];
                auto shift = [&]() {
#pragma unroll
                    for (int h4 = 0; h4 < kHG / 4; ++h4) {
                        const float4 n4 = reinterpret_cast<const float4*>(m_neg + h0)[h4];
                        e2[2 * h4] = __fadd2_rn(t2[2 * h4], make_float2(n4.x, n4.y));
                        e2[2 * h4 + 1] = __fadd2_rn(t2[2 * h4 + 1], make_float2(n4.z, n4.w));
                    }
                };
                shift();
                // The vote on moving a reference, and the rare move, involve the group's four warps only.
                bool viol = false;
#pragma unroll
                for (int i = 0; i < kHG / 2; ++i) viol |= (e2[i].x > kMostTop) || (e2[i].y > kMostTop);
                bool any_upd = false;
                if (named_bar_or(group_bar, kGroupThreads, viol)) {
                    float xm[kHG];
#pragma unroll
                    for (int i = 0; i < kHG / 2; ++i) {
                        xm[2 * i] = t2[i].x;
                        xm[2 * i + 1] = t2[i].y;
                    }
                    const float r = warp_transpose_reduce16<true>(xm, lane);
                    if ((lane & 1u) == 0) red[quad * kH + h0 + (int)(lane >> 1)] = r;
                    named_bar_sync(group_bar, kGroupThreads);
                    bool upd = false;
                    if (ww == 4 * hg && lane < kHG) {   // one lane per head of the group
                        const int h = h0 + (int)lane;
                        const float mt = fmaxf(fmaxf(red[h], red[kH + h]), fmaxf(red[2 * kH + h], red[3 * kH + h])) - kFirstTop;
                        const bool unset = (m_neg[h] == kNoRef);
                        const float mo = -m_neg[h];
                        float a = 1.f;
                        if (mt > -INFINITY && (unset || mt > mo + (kMostTop - kFirstTop))) {
                            a = unset ? 0.f : ex2_approx(mo - mt);
                            m_neg[h] = -mt;
                            upd = !unset;
                        }
                        alpha_s[h] = a;
                    }
                    any_upd = named_bar_or(group_bar, kGroupThreads, upd);
                    shift();
                    if (any_upd) {
#pragma unroll
                        for (int h4 = 0; h4 < kHG / 4; ++h4) {
                            const float4 a4 = reinterpret_cast<const float4*>(alpha_s + h0)[h4];
                            l2[2 * h4] = __fmul2_rn(l2[2 * h4], make_float2(a4.x, a4.y));
                            l2[2 * h4 + 1] = __fmul2_rn(l2[2 * h4 + 1], make_float2(a4.z, a4.w));
                        }
                    }
                }
                // P' and its two e4m3 parts; the row sum takes the float32 weight with the row's scale divided out
                const float ic = c > 0.f ? __frcp_rn(c) : 0.f;
                uint32_t w[kHG / 2];
#pragma unroll
                for (int i = 0; i < kHG / 2; ++i) {
                    const float2 pr = make_float2(ex2_approx(e2[i].x), ex2_approx(e2[i].y));
                    l2[i] = __ffma2_rn(pr, make_float2(ic, ic), l2[i]);
                    w[i] = split_e4m3x2(pr.x, pr.y);
                }
                if (gt > 0) gok = gok && pv_done(gt - 1);   // P^T and O^T are free
                if (any_upd && t > 0) {
                    tc_fence_after();
#pragma unroll 1
                    for (int ch = 0; ch < kChunks; ++ch) {
                        uint32_t v[kHG];
                        const uint32_t a = tmem_base + lane_addr + TM_O + 64 * ch + h0;
                        tmem_ld16(a, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < kHG; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha_s[h0 + k]);
                        tmem_st16(a, v);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                }
                {   // P^T row `key`: 16 heads hi at 16-byte piece hg of the swizzled row, lo at piece 4 + hg
                    uint8_t* d = smem + OFF_P + key * 128;
                    *reinterpret_cast<uint4*>(d + ((hg ^ (key & 7)) << 4)) =
                        make_uint4(lows(w[0], w[1]), lows(w[2], w[3]), lows(w[4], w[5]), lows(w[6], w[7]));
                    *reinterpret_cast<uint4*>(d + (((4 + hg) ^ (key & 7)) << 4)) =
                        make_uint4(highs(w[0], w[1]), highs(w[2], w[3]), highs(w[4], w[5]), highs(w[6], w[7]));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
            }
            qbuf = qbuf == 2 ? 0 : qbuf + 1;
            // ---------------- final: l = sum of partial row sums; out = O^T / l
            {
                float l_part[kHG];
#pragma unroll
                for (int i = 0; i < kHG / 2; ++i) {
                    l_part[2 * i] = l2[i].x;
                    l_part[2 * i + 1] = l2[i].y;
                }
                const float r = warp_transpose_reduce16<false>(l_part, lane);
                if ((lane & 1u) == 0) red[quad * kH + h0 + (int)(lane >> 1)] = r;
            }
            if (!named_bar_and(2, kWorkers, gok && pv_done(gt - 1))) {
                failed = true;
                break;
            }
            tc_fence_after();
            if (tid < kH) {
                const float l = red[tid] + red[kH + tid] + red[2 * kH + tid] + red[3 * kH + tid];
                // l = 0: every selected key was outside the cache
                invl_s[tid] = (l > 0.f) ? 1.f / l : (l == 0.f ? 0.f : l);
                store_lse(I, tid, (l > 0.f) ? (log2f(l) - m_neg[tid]) * 0.6931471805599453f : (l == 0.f ? -INFINITY : l));
            }
            named_bar_sync(1, kWorkers);
            // A lane holds one dim of 16 heads; the lanes of a group exchange them so that each stores 16
            // contiguous bytes of a head (with a store of one element a lane an item's output took 5 us).
#pragma unroll 1
            for (int ch = 0; ch < kChunks; ++ch) {
                uint32_t v[kHG];
                tmem_ld16(tmem_base + lane_addr + TM_O + 64 * ch + h0, v);
                tmem_ld_wait();
#pragma unroll
                for (int h = 0; h < kHG; ++h) v[h] = __float_as_uint(__uint_as_float(v[h]) * invl_s[h0 + h]);
                const int dim0 = ch * 128 + quad * 32;
                if (PARTIAL || p.out_f32) {       // groups of 4 lanes: lane j gets heads 4j.. of the group's 4 dims
                    float* base = PARTIAL ? p.part_o + (((int64_t)I.row * p.nsplit + I.split) * kH + h0) * kDv
                                          : static_cast<float*>(p.out) + ((int64_t)I.row * kH + h0) * kDv;
                    transpose_words<16, 4>(v, lane);
                    float* dst = base + (int)(lane & 3) * 4 * kDv + dim0 + (int)(lane & ~3u);
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        *reinterpret_cast<uint4*>(dst + h * kDv) = make_uint4(v[h], v[4 + h], v[8 + h], v[12 + h]);
                } else {                          // groups of 8 lanes: lane j gets heads 2j, 2j + 1 of the group's 8 dims
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                    transpose_words<8, 8>(w, lane);
                    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) +
                                         ((int64_t)I.row * kH + h0 + (int)(lane & 7) * 2) * kDv + dim0 + (int)(lane & ~7u);
                    *reinterpret_cast<uint4*>(dst) =
                        make_uint4(lows(w[0], w[1]), lows(w[2], w[3]), lows(w[4], w[5]), lows(w[6], w[7]));
                    *reinterpret_cast<uint4*>(dst + kDv) =
                        make_uint4(highs(w[0], w[1]), highs(w[2], w[3]), highs(w[4], w[5]), highs(w[6], w[7]));
                }
            }
            tc_fence_before();
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, kTmemCols);
    }
}

template <bool PARTIAL>
dsa_status_t launch(const AttnQ8Params& p, cudaStream_t stream) {
    auto kern = mla_attn_q8_kernel<PARTIAL>;
    dsa_status_t st = ensure_smem_attr(reinterpret_cast<const void*>(kern), kSmemBytes);
    if (st != DSA_OK) return st;
    const int sms = device_sm_count();
    if (launch_pdl(kern, dim3(p.n_items < sms ? p.n_items : sms), dim3(kThreads), kSmemBytes, stream, p) != cudaSuccess)
        return DSA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

AttnQ8Params base_params(const void* q, const void* cache, const float* cache_scale, const int32_t* idx, int rows,
                         int Nmax, int top_k, float scale, const PageTable& pages) {
    AttnQ8Params p{};
    p.idx = idx;
    p.rows = rows;
    p.Nmax = Nmax;
    p.top_k = top_k;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.cache = static_cast<const uint8_t*>(cache);
    p.cache_scale = cache_scale;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.status = device_status_ptr();
    p.pages = pages;
    return p;
}

}  // namespace

dsa_status_t launch_attn_q8_prefill(const void* q, const void* cache, const float* cache_scale, const int32_t* idx,
                                    int L, int N, int top_k, float scale, void* out, int out_f32, float* lse,
                                    const PageTable& pages, cudaStream_t stream) {
    AttnQ8Params p = base_params(q, cache, cache_scale, idx, L, N, top_k, scale, pages);
    p.prefill = 1;
    p.nsplit = 1;
    p.split_len = ceil_div(top_k, kTile) * kTile;
    p.n_items = L;
    p.out = out;
    p.out_f32 = out_f32;
    p.lse = lse;
    return launch<false>(p, stream);
}

dsa_status_t launch_attn_q8_decode(const void* q, const void* cache, const float* cache_scale, const int32_t* kv_len,
                                   const int32_t* idx, int B, int Nmax, int top_k, float scale, void* out,
                                   int out_f32, float* lse, void* workspace, const PageTable& pages,
                                   cudaStream_t stream) {
    AttnQ8Params p = base_params(q, cache, cache_scale, idx, B, Nmax, top_k, scale, pages);
    p.kv_len = kv_len;
    p.split_len = ceil_div(ceil_div(top_k, kTile), decode_splits(B, top_k)) * kTile;
    p.nsplit = ceil_div(top_k, p.split_len);
    p.n_items = B * p.nsplit;
    p.part_o = static_cast<float*>(workspace);
    p.part_lse = p.part_o + (size_t)B * p.nsplit * kH * kDv;
    dsa_status_t st = launch<true>(p, stream);
    if (st != DSA_OK) return st;
    return launch_decode_combine(p.part_o, p.part_lse, B, p.nsplit, out, out_f32, lse, stream);
}

}  // namespace dsa
