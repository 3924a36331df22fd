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
constexpr int kRing = 7;                           // chunk slots
constexpr int kWorkerWarps = 16;
constexpr int kWorkers = kWorkerWarps * 32;
constexpr int kPvIssuers = 2;
constexpr int kFirstWorker = 1 + kPvIssuers;       // warp 0 QK, warps 1-2 PV, warps 3.. workers
constexpr int kThreads = 32 * kFirstWorker + kWorkers;
constexpr int kMaxRegs = 96;                       // 19 warps: 5 share one 16K-register sub-partition
constexpr int kHG = kH / (kWorkerWarps / 4);       // 16 heads a worker warp
constexpr int kGroupThreads = 4 * 32;              // the four warps sharing a head group
static_assert(kHG == 16 && kWorkerWarps == 16, "a worker warp: 16 heads, 8 rows of a tile, 4 query heads");

constexpr float kFirstTop = 5.5f;                  // log2 of the first tile's largest P'
constexpr float kMostTop = 8.75f;                  // log2 of the largest P' (430 <= 448)
constexpr float kNoRef = 3.0e38f;                  // -m before the reference is set (finite: see mla_attn.cu)

// smem layout (1024-aligned base)
constexpr int OFF_QHL = 0;                         // 4 chunks x (64 hi rows, 64 lo rows) x 128 B
constexpr int OFF_QR = OFF_QHL + kChunks * kBlk;   // 64 heads x 64 bf16
constexpr int OFF_LAT = OFF_QR + kH * 128;         // ring of latent chunks
constexpr int OFF_ROPE = OFF_LAT + kRing * kBlk;   // 128 keys x 64 bf16
constexpr int OFF_P = OFF_ROPE + kBlk;             // 128 keys x (64 hi | 64 lo)
constexpr int OFF_SC = OFF_P + kBlk;               // float [2][128]: scales of the tile's rows, 0 = no key
constexpr int OFF_QS = OFF_SC + 2 * kTile * 4;     // float [2][64]: scale * log2(e) * 2^k of the query's heads
constexpr int OFF_RED = OFF_QS + 2 * kH * 4;       // float [4][64]
constexpr int OFF_MNEG = OFF_RED + 4 * kH * 4;     // float [64]: minus the references
constexpr int OFF_ALPHA = OFF_MNEG + kH * 4;       // float [64]
constexpr int OFF_INVL = OFF_ALPHA + kH * 4;       // float [64]
constexpr int OFF_BAR = OFF_INVL + kH * 4;
// barriers: full[7], free[7], rope_full, s_full, s_free, p_full, q_full
constexpr int kBars = 2 * kRing + 5;
constexpr int OFF_TMEM = OFF_BAR + kBars * 8;
constexpr int OFF_ABORT = OFF_TMEM + 4;
constexpr int kSmemBytes = OFF_ABORT + 4 + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory of a CTA");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t TM_S = 0;                       // S^T: 64 columns hi, 64 lo
constexpr uint32_t TM_R = 128;                     // the rope product, 64 columns
constexpr uint32_t TM_O = 192;                     // O^T chunk c at TM_O + 64 c
constexpr uint32_t TM_ONE = 448;                   // scale bytes 2^0
constexpr uint32_t TM_LO = 464;                    // scale bytes 2^-4

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

template <bool PARTIAL>
__global__ void __maxnreg__(kMaxRegs)   // kThreads threads, one CTA per SM
    mla_attn_q8_kernel(const AttnQ8Params p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* sc_s = reinterpret_cast<float*>(smem + OFF_SC);
    float* qs_s = reinterpret_cast<float*>(smem + OFF_QS);
    float* red = reinterpret_cast<float*>(smem + OFF_RED);
    float* m_neg = reinterpret_cast<float*>(smem + OFF_MNEG);
    float* alpha_s = reinterpret_cast<float*>(smem + OFF_ALPHA);
    float* invl_s = reinterpret_cast<float*>(smem + OFF_INVL);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    uint64_t* freed = full + kRing;
    uint64_t* rope_full = freed + kRing;
    uint64_t* s_full = rope_full + 1;
    uint64_t* s_free = rope_full + 2;
    uint64_t* p_full = rope_full + 3;
    uint64_t* q_full = rope_full + 4;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_TMEM);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);

    const int warp = threadIdx.x / 32;
    const uint32_t lane = lane_id();

    if (threadIdx.x == 0) {
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&full[i], kWorkers);      // one cp.async arrival per worker thread
            mbar_init(&freed[i], 1);            // the commit of the PV issuer that consumed the chunk
        }
        mbar_init(rope_full, kWorkers);
        mbar_init(s_full, 1);
        mbar_init(s_free, kWorkerWarps);
        mbar_init(p_full, kWorkerWarps);
        mbar_init(q_full, kWorkerWarps);
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

    // Chunk n = 4 g + c of the CTA's g-th tile lies in slot n % 7; its slot's barriers are in use n / 7.
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
                const uint64_t lat = sdesc_sw128(smem_u32(smem + OFF_LAT), 16, 1024);
                const uint64_t qhl = sdesc_sw128(smem_u32(smem + OFF_QHL), 16, 1024);
                const uint64_t rope = sdesc_sw128(smem_u32(smem + OFF_ROPE), 16, 1024);
                const uint64_t qr = sdesc_sw128(smem_u32(smem + OFF_QR), 16, 1024);
                ok = mbar_wait_spin(q_full, qi & 1, abort_flag, p.status);
                for (int t = 0; ok && t < T; ++t, ++gt) {
                    // the workers have read the previous tile's S^T
                    if (!(ok = mbar_wait_spin(s_free, (gt & 1) ^ 1, abort_flag, p.status))) break;
                    tc_fence_after();
#pragma unroll
                    for (int j = 0; j < 5; ++j) {   // chunks 0, 1, 2, the rope block, chunk 3 (its copy comes last)
                        if (j == 3) {
                            if (!(ok = mbar_wait_spin(rope_full, gt & 1, abort_flag, p.status))) break;
                            fence_proxy_async_smem();
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_bf16_ss_lo(tmem_base + TM_R, (uint32_t)rope + 2 * kk, (uint32_t)(rope >> 32),
                                               (uint32_t)qr + 2 * kk, (uint32_t)(qr >> 32), IDESC_ROPE, kk ? 1u : 0u);
                        } else {
                            const int c = j < 3 ? j : 3;
                            const uint32_t n = 4u * (uint32_t)gt + (uint32_t)c, slot = n % kRing;
                            if (!(ok = mbar_wait_spin(&full[slot], (n / kRing) & 1, abort_flag, p.status))) break;
                            fence_proxy_async_smem();
                            const uint32_t a = (uint32_t)lat + slot * (kBlk >> 4);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)   // 32 dims a step
                                mma_e4m3_ss_lo(tmem_base + TM_S, a + 2 * kk, (uint32_t)(lat >> 32),
                                               (uint32_t)qhl + c * (kBlk >> 4) + 2 * kk, (uint32_t)(qhl >> 32), IDESC_QK,
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
                const uint64_t lat = sdesc_sw128(smem_u32(smem + OFF_LAT), kBlk, 1024);
                const uint64_t pt = sdesc_sw128(smem_u32(smem + OFF_P), kBlk, 1024);
                for (int t = 0; ok && t < T; ++t, ++gt) {
                    if (!(ok = mbar_wait_spin(p_full, gt & 1, abort_flag, p.status))) break;
                    tc_fence_after();
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int c = iss + 2 * j;
                        const uint32_t slot = (4u * (uint32_t)gt + (uint32_t)c) % kRing;
                        const uint32_t a = (uint32_t)lat + slot * (kBlk >> 4);
                        const uint32_t d = tmem_base + TM_O + 64 * (uint32_t)c;
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {     // 32 keys (four 8-key groups, 4 KB) a step
                            mma_e4m3_scaled_ss_lo(d, a + kk * (4096 >> 4), (uint32_t)(lat >> 32),
                                                  (uint32_t)pt + kk * (4096 >> 4), (uint32_t)(pt >> 32), IDESC_PV,
                                                  tmem_base + TM_ONE, tmem_base + TM_ONE, (t | kk) ? 1u : 0u);
                            mma_e4m3_scaled_ss_lo(d, a + kk * (4096 >> 4), (uint32_t)(lat >> 32),
                                                  (uint32_t)pt + kk * (4096 >> 4) + (64 >> 4), (uint32_t)(pt >> 32), IDESC_PV,
                                                  tmem_base + TM_ONE, tmem_base + TM_LO, 1u);
                        }
                        mma_commit(&freed[slot]);
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        }
    } else {
        // ------------------------------------------------------------ workers
        const int ww = warp - kFirstWorker;       // 0..15
        const int quad = warp & 3;                // TMEM lane quadrant this warp may access
        const int hg = ww >> 2;                   // head group: heads h0 .. h0 + 15
        const int h0 = hg * kHG;
        const uint32_t group_bar = 3 + (uint32_t)hg;
        const int tid = ww * 32 + (int)lane;      // 0..511
        const int key = quad * 32 + (int)lane;    // TMEM lane == key row of the tile == dim row of O^T
        const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
        const uint32_t smem_base = smem_u32(smem);
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            return mbar_wait(bar, parity, abort_flag, p.status);
        };
        auto chunk_free = [&](uint32_t n) -> bool {   // PV has consumed chunk n
            return wait(&freed[n % kRing], (n / kRing) & 1);
        };
        auto pv_done = [&](int g) -> bool { return chunk_free(4u * g + 2) && chunk_free(4u * g + 3); };

        // ---- gather.  The warp copies rows 64 h + 4 ww + i (h < 2, i < 4) of every tile; lanes 0..7 carry
        // row 4 h + i of them through three stages: the selected key (fetch), its cache row (resolve: a page
        // lookup when paged), the copies.  Each stage runs one tile ahead of the next, so that its loads
        // are in flight during a softmax.
        int f_s = 0, f_t = 0, f_T = 0;            // fetch cursor: next tile to fetch
        Item fI{};
        bool f_open = true;
        auto fetch = [&](int& j, int& batch, int& bound) -> bool {   // false: no more tiles
            while (f_open && f_t >= f_T) {
                const int it = nth_item(p, f_s++);
                if (it == -1) {
                    f_open = false;
                } else if (it >= 0) {
                    fI = decode_item(p, it);
                    f_T = item_tiles(p, fI, lane);
                    f_t = 0;
                }
            }
            if (!f_open) return false;
            const int slot = fI.slot0 + f_t * kTile + 64 * (int)(lane >> 2) + 4 * ww + (int)(lane & 3);
            j = (lane < 8 && slot < fI.slot_end) ? __ldg(p.idx + (int64_t)fI.row * p.top_k + slot) : -1;
            batch = fI.batch;
            bound = fI.bound;
            ++f_t;
            return true;
        };
        // cache row of key j; -1: no key, -2: a page outside the pool (a row of zeros)
        auto resolve = [&](int j, int batch, int bound) -> int {
            if (j < 0) return -1;
            if (j >= bound) {
                raise_dev_error(p.status, DEV_ERR_BOUNDS);
                return -1;
            }
            if (p.pages.table) {
                const int row = (int)paged_row(p.pages, batch, j);
                if (row < 0) raise_dev_error(p.status, DEV_ERR_BOUNDS);
                return row < 0 ? -2 : row;
            }
            return (int)((int64_t)batch * p.Nmax + j);
        };
        const int ci = (int)(lane >> 3);          // the warp's row i of a half this lane copies for
        const int cc = (int)(lane & 7);           // 16-byte piece of the 128-byte block
        uint32_t dst_h[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = 64 * h + 4 * ww + ci;
            dst_h[h] = (uint32_t)(r * 128 + ((cc ^ (r & 7)) << 4));
        }
        // one 128-byte block (blk 0..3 latent, 4 rope) of the warp's 8 rows, row8 held by lanes 0..7
        auto copy_block = [&](int row8, int blk, uint32_t dst) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = __shfl_sync(0xffffffffu, row8, 4 * h + ci);
                cp_async_16(dst + dst_h[h], p.cache + (r < 0 ? 0 : (int64_t)r * kQ8Row + blk * 128 + cc * 16),
                            r < 0 ? 0u : 16u);
            }
        };
        auto copy_chunk = [&](int row8, int g, int c) -> bool {      // chunk c of the CTA's g-th tile
            const uint32_t n = 4u * (uint32_t)g + (uint32_t)c, slot = n % kRing;
            const bool ok = __all_sync(0xffffffffu, wait(&freed[slot], ((n / kRing) & 1) ^ 1));
            if (ok) copy_block(row8, c, smem_base + OFF_LAT + slot * kBlk);
            if (ok) cp_async_arrive_noinc(&full[slot]);
            return ok;
        };
        auto copy_rope = [&](int row8, int g) {   // the rope block and the scales: QK of tile g - 1 is complete
            copy_block(row8, kChunks, smem_base + OFF_ROPE);
            if (lane < 8) {
                const int r = 64 * (int)(lane >> 2) + 4 * ww + (int)(lane & 3);
                cp_async_4(smem_base + OFF_SC + ((g & 1) * kTile + r) * 4,
                           row8 >= 0 ? p.cache_scale + row8 : &g_unit_scale, row8 == -1 ? 0u : 4u);
            }
            cp_async_arrive_noinc(rope_full);
        };

        // ---- query: the warp converts heads 4 ww .. 4 ww + 3.  Lane l holds dims 8l.. and 256 + 8l.. of a head.
        auto q_head = [&](int row, int qpar, int i) {
            const int h = 4 * ww + i;
            const __nv_bfloat16* src = p.q + ((int64_t)row * kH + h) * DSA_QK_DIM;
            uint4 raw[2];
            raw[0] = ldg_nc_v4(src + 8 * lane);
            raw[1] = ldg_nc_v4(src + 256 + 8 * lane);
            const uint32_t pe = __ldg(reinterpret_cast<const uint32_t*>(src + kQ8Latent) + lane);
            const uint32_t w[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w, raw[1].x, raw[1].y, raw[1].z, raw[1].w};
            float amax = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));
#pragma unroll
            for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const int e = e4m3_scale_exponent(amax);
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
            *reinterpret_cast<uint32_t*>(smem + OFF_QR + h * 128 + (((lane >> 2) ^ (h & 7)) << 4) + (lane & 3) * 4) = pe;
            if (lane == 0) qs_s[qpar * kH + h] = p.scale_log2 * exp2_int(e);
        };
        auto q_ready = [&]() {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
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

        // ---- prologue: tile 0 whole, chunks 0-2 of tile 1, the query of the first item.  `gok` is this thread's
        // wait status: a wait that gives up does not change the control flow inside an item (all workers keep
        // meeting the same named barriers); the consensus barrier at the item's end takes all out together.
        bool gok = true;
        int fj, fb, fl;                           // fetched: key, batch, bound of the tile three ahead
        int rowA, rowR = -1;                      // rows of the next tile to copy whole, of the one after it
        bool hasA, hasR, hasF;
        hasA = fetch(fj, fb, fl);
        {
            int j1, b1, l1;
            hasR = fetch(j1, b1, l1);
            rowA = hasA ? resolve(fj, fb, fl) : -1;
            if (hasA) {
#pragma unroll
                for (int c = 0; c < kChunks; ++c) gok = copy_chunk(rowA, 0, c) && gok;
                copy_rope(rowA, 0);
            }
            rowA = hasR ? resolve(j1, b1, l1) : -1;
            hasA = hasR;
            if (hasA)
#pragma unroll
                for (int c = 0; c < 3; ++c) gok = copy_chunk(rowA, 1, c) && gok;
        }
        hasR = fetch(fj, fb, fl);
        rowR = hasR ? resolve(fj, fb, fl) : -1;
        hasF = fetch(fj, fb, fl);
        bool more = next_item();
        if (more) {
#pragma unroll 1
            for (int i = 0; i < 4; ++i) q_head(nI.row, 0, i);
            q_ready();
        }
        bool failed = false;
        int gt = 0;                               // tiles done by this CTA
        int qpar = 0;                             // parity of the item's query scales
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
                gok = gok && wait(s_full, gt & 1);
                gok = gok && wait(rope_full, gt & 1);   // complete (QK needed it): makes the scales visible here
                tc_fence_after();
                if (hasA && __all_sync(0xffffffffu, gok)) copy_rope(rowA, gt + 1);
                float2 t2[kHG / 2];               // log2(e) s + log2(c): the exponents before the reference
                const float c = sc_s[(gt & 1) * kTile + key];
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
                        const float2 qs = reinterpret_cast<const float2*>(qs_s + qpar * kH + h0)[i];
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
                // copies of chunk 3 of the next tile and chunks 0-2 of the one after it, as PV frees their slots;
                // after an item's last tile its QK is complete: the next query is converted between them
                const bool conv = more && t == T - 1;
#pragma unroll
                for (int k = 0; k < kChunks; ++k) {
                    if (conv) q_head(nI.row, qpar ^ 1, k);
                    if (k == 0) {
                        if (hasA) gok = copy_chunk(rowA, gt + 1, 3) && gok;
                    } else if (hasR) {
                        gok = copy_chunk(rowR, gt + 2, k - 1) && gok;
                    }
                }
                if (conv) q_ready();
                rowA = rowR;
                hasA = hasR;
                rowR = hasF ? resolve(fj, fb, fl) : -1;
                hasR = hasF;
                if (hasF) hasF = fetch(fj, fb, fl);
            }
            qpar ^= 1;
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
#pragma unroll 1
            for (int ch = 0; ch < kChunks; ++ch) {
                uint32_t v[kHG];
                tmem_ld16(tmem_base + lane_addr + TM_O + 64 * ch + h0, v);
                tmem_ld_wait();
                float o[kHG];
#pragma unroll
                for (int h = 0; h < kHG; ++h) o[h] = __uint_as_float(v[h]) * invl_s[h0 + h];
                const int dim = ch * 128 + key;
                if (PARTIAL) {
                    float* dst = p.part_o + (((int64_t)I.row * p.nsplit + I.split) * kH + h0) * kDv + dim;
#pragma unroll
                    for (int h = 0; h < kHG; ++h) dst[h * kDv] = o[h];
                } else if (p.out_f32) {
                    float* dst = static_cast<float*>(p.out) + ((int64_t)I.row * kH + h0) * kDv + dim;
#pragma unroll
                    for (int h = 0; h < kHG; ++h) dst[h * kDv] = o[h];
                } else {
                    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + ((int64_t)I.row * kH + h0) * kDv + dim;
#pragma unroll
                    for (int h = 0; h < kHG; ++h) dst[h * kDv] = __float2bfloat16_rn(o[h]);
                }
            }
            tc_fence_before();
        }
        cp_async_wait_all();
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
