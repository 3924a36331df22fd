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
//     hi + lo / 16 (times a power of two a head), exactly so down to 2^-13 of the head's largest
//     element and within 2^-21 of it below.  hi and lo of the 64 heads stand next to each other as one
//     N = 128 operand, so QK over 32 dims is one MMA; the softmax adds the two halves.  The rope
//     dims are a bf16 product of their own (their rows are not scaled).
//   * The probabilities are split the same way, P' = hi + lo / 16, lo's factor applied by the
//     block-scaled MMA (constant scale bytes in TMEM), both into one accumulator: 8 significant bits, as
//     the bf16 kernel's probabilities have.  The row's scale is folded in before the split:
//     P' = 2^(t - m) with t = log2(e) s + log2(c), so that e4m3's range (2^-9 .. 448, and 2^-13 with
//     lo) is spent on the weights that the value sum sees; the row sum divides it out again (and takes the
//     weight without c where c makes P' smaller than float32's numbers).
//   * The reference m of a head is set from the query's first tile so that its largest P' is 2^4.5,
//     and moved when a later one would pass 2^8.75 (e4m3 ends at 448): a higher start would leave
//     less room and rescale O^T more often, a lower one would lose the small weights sooner (a
//     weight keeps 8 bits down to 2^-10.5 of the largest at worst, 2^-14.8 at best).
//   * Shared memory holds two tiles' latent rows (64 KB each), the 72 KB query and one P^T block.  The rope
//     rows go through registers into tensor memory, as the A operand of their MMA: shared memory is what the
//     kernel runs short of, and the operand reads of a tile's other MMAs alone take it 2750 cycles.
//   * Roles (28 warps, registers moved to the workers by setmaxnreg): warp 0 issues QK, warps 1 and 2 PV
//     (chunks 0, 2 and 1, 3), warp 3 the query's TMA; 4 warps gather latent rows (cp.async), 4 the rope rows and
//     scales, 16 worker warps do the softmax and write the output; the query, read as bf16, is split in place
//     by the eight gathering warps when its predecessor's last QK has read the old one.  Two PV issuers: one
//     thread reaches an N = 64 scaled MMA every 80 cycles, two one every 52; one N = 128 issuer reaches its 64.
//     Spinning waits are one thread's a role (with a poller in each gathering warp 1.18 ms became 1.40).
//   * Queries run whole on persistent CTAs; those behind the last full round of the SMs (all, for few) have
//     their selected keys cut into parts, one a CTA, which write partial (normalised output, lse) pairs for the
//     bf16 path's merge kernel.  Merging inside a thread-block cluster was slower: reading the other CTAs' parts from
//     distributed shared memory took 13 thousand cycles, storing them there 20 thousand, and a cluster barrier
//     with the parts in global memory made a call of 8 sequences 18.2 us, against 14.9 with the merge kernel.
//   * Measured: 4096 queries of 2048 keys 1.12 ms (0.52 of the bf16 matrix peak for the 1088 products a key and
//     head), decode of 256 sequences 99 us, of 8 14.4 us, of one 12.9 us.  About 5000 cycles a tile of 128 keys:
//     the loop copy, QK, softmax, PV of a stage is 10 thousand, and two stages fit.  Leaving out the vote and the
//     softmax's reads of shared memory took 1.18 to 1.11 ms, half of PV or of QK 1.25 to 1.15.
//   * The same kernel over the 4-bit cache (Q4): every stored value is an e4m3 number, so only the gather differs.  The four
//     latent warps expand chunks 0 and 1, the four rope warps 2 and 3 ahead of their rope rows, a lane its own row: codes in
//     registers before their place comes free, a block's eight magnitudes from a table in shared memory, a byte selection
//     a half word.  A prefill that selects each key several times expands the cache once instead (attn_q4_expands) and
//     takes the 8-bit kernel's time, 4096 queries 1.13 ms.  Decode of 256 sequences of up to 8192 keys 145 us (99 over 8-bit
//     rows), of 37 20.6, of one 13.4: the latent warps are never idle (a trace: of 8300 cycles a tile the L2 prefetch of 32
//     rows takes 2000, lookups 900, expanding 2300, the loads' latency 1500).  The table in shared memory left out would give
//     17 us, all of the expansion 24.
#include <cuda.h>

#include <atomic>
#include <cmath>
#include <type_traits>

#include "dsa_q4.cuh"
#include "mla_attn_common.cuh"

namespace dsa {

namespace {

constexpr int kBlk = 128 * 128;                    // 16 KB: 128 rows of 128 bytes
constexpr int kChunks = kQ8Latent / 128;           // 4 latent chunks of 128 dims a tile
constexpr int kStages = 2;                         // tiles in shared memory
constexpr int kPvIssuers = 2;
constexpr int kGatherWarps = 4;                    // latent rows, half of the query
constexpr int kQueryWarp = 1 + kPvIssuers;
constexpr int kRopeWarps = 4;                      // rope rows, scales, the other half of the query
constexpr int kWorkerWarps = 16;                   // softmax and output
constexpr int kWorkers = kWorkerWarps * 32;
// warp 0 QK, warps 1-2 PV, warp 3 the query's TMA; warps 4-7 latent rows, 8-11 rope rows; 12-27 workers.
// The register split is by warpgroups of four warps out of what the launch holds: 896 threads of 72 registers.
constexpr int kFirstGather = 4;
constexpr int kFirstRope = kFirstGather + kGatherWarps;
constexpr int kFirstWorker = kFirstRope + kRopeWarps;
constexpr int kThreads = 32 * (kFirstWorker + kWorkerWarps);
constexpr int kLaunchRegs = 72, kIssueRegs = 56, kGatherRegs = 64, kWorkerRegs = 80;
static_assert(kThreads * kLaunchRegs >=
                  32 * (kFirstGather * kIssueRegs + (kGatherWarps + kRopeWarps) * kGatherRegs + kWorkerWarps * kWorkerRegs),
              "registers of the CTA");
static_assert(kGatherWarps == 4 && kRopeWarps == 4, "a warp of either kind has 32 rows of a tile, one a lane");
constexpr int kHG = kH / (kWorkerWarps / 4);       // 16 heads a worker warp
constexpr int kGroupThreads = 4 * 32;              // the four warps sharing a head group
constexpr uint32_t kGatherBar = 7;                 // named barriers: 1, 2 workers, 3-6 head groups, 7 gather, 8 rope
static_assert(kHG == 16 && kWorkerWarps == 16, "a warp's loads of S^T take a head group of 16");

constexpr float kFirstTop = 4.5f;                  // log2 of the first tile's largest P'
constexpr float kMostTop = 8.75f;                  // log2 of the largest P' (430 <= 448)
constexpr float kLeastExponent = -126.f;           // ex2_approx gives 0 below
constexpr float kSmallScale = 0x1p-20f;            // below it the row sum looks at P' < 2^-126
// A row of zeros is written with scale 1, but any scale stands for the same row: taken is the smallest, so that the
// row, which adds nothing to the value sum, takes none of e4m3's range from the others.  Only rows of scale 1 or more,
// few among a normalised latent's (about 2^-6), are looked at.  4096 queries, ms: 1.13, with every hundredth row of zeros
// 1.14, every tenth 1.34, zeros alone 3.97; a cache whose every row has scale 1, float32 output, 1.17 -> 1.32.  A look
// at every row's first codes took 1.22; a lane alone at its row of zeros, after the wait, 2.19 for every hundredth.
constexpr float kZeroRowScale = 0x1p-64f;

// smem layout
constexpr int OFF_QHL = 0;                         // 4 chunks x (64 hi rows, 64 lo rows) x 128 B
constexpr int OFF_QR = OFF_QHL + kChunks * kBlk;   // rope dims of 64 heads: 64 rows x 128 B
constexpr int OFF_LAT = OFF_QR + kH * 128;         // 2 tiles x 4 latent chunks
constexpr int OFF_P = OFF_LAT + kStages * kChunks * kBlk;   // 128 keys x (64 hi | 64 lo)
// A tile's rows: c, log2 c (0, -inf: no key), of two tiles, and 1 / c (0) and whether there are small scales, of four:
// the workers read the first before they give S^T free, the second after, while the rows of later tiles come in.  The slot of tile g is
// next written for tile g + 4, behind QK of g + 3, which waits for every worker's reading of S^T of g + 2.
constexpr int OFF_SC = OFF_P + kBlk;               // float2 [2][128]
constexpr int OFF_IC = OFF_SC + 2 * kTile * 8;     // float [4][128]
constexpr int OFF_SMALL = OFF_IC + 4 * kTile * 4;    // int [4][4]: one of a quarter of the tile's rows has a small scale
constexpr int OFF_QS = OFF_SMALL + 4 * 4 * 4;        // float [4][64]: scale * log2(e) * 2^k of a query's heads
constexpr int OFF_RED = OFF_QS + 4 * kH * 4;       // float [4][64]
constexpr int OFF_MNEG = OFF_RED + 4 * kH * 4;     // float [64]: minus the references
constexpr int OFF_DELTA = OFF_MNEG + kH * 4;       // float [64]: how far a reference has just risen
constexpr int OFF_INVL = OFF_DELTA + kH * 4;       // float [64]
constexpr int OFF_TABLE = OFF_INVL + kH * 4;       // uint2 [256]: the magnitudes of 4-bit codes as e4m3, by block byte
constexpr int OFF_BAR = OFF_TABLE + 256 * 8;
// barriers: full[8], free[4], rope_full, s_full, s_free, p_full, q_free, q_raw, q_full
constexpr int kSlots = kStages * kChunks;
constexpr int kBars = kSlots + 2 * kStages + 7;
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
constexpr uint32_t TM_K = 480;                     // the tile's rope rows, 32 columns of two bf16
static_assert(TM_K + kQ8Rope / 2 <= kTmemCols, "tensor memory columns");

// Operands: 128-byte swizzle, 8-row groups 1 KB apart.  The descriptors' high words are the same; the
// low words (address, leading offset) are sums that stay below the address field's end (see sdesc).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t IDESC_QK = idesc_e4m3_f32(128, 128, false, false);
constexpr uint32_t IDESC_ROPE = idesc_bf16_f32(128, 64, false, false);
constexpr uint32_t IDESC_PV = idesc_e4m3_scaled_f32(128, 64, true, true);

__device__ __align__(32) uint8_t g_no_row[kQ8Latent];   // zeros, the latent dims of a slot without a row

// The two caches: bytes of a row, where its rope dims begin.
template <bool Q4>
struct Rows {
    static constexpr int kBytes = Q4 ? kQ4Row : kQ8Row;
    static constexpr int kRope = Q4 ? kQ4Rope : kQ8Latent;
    // the lane's share of a row's codes, and whether they stand for zeros of either sign
    static constexpr int kLaneCodes = Q4 ? kQ4Codes / 32 : kQ8Latent / 32;
};
static_assert(kQ4Rope <= kQ8Latent, "g_no_row holds the codes and blocks of a 4-bit row");

struct AttnQ8Params : AttnShape {
    const __nv_bfloat16* q;    // [rows][64][576]
    const uint8_t* cache;      // 640-byte or 416-byte rows
    const float* cache_scale;
    void* out;                 // final: [rows][64][512], float32 or bf16 (out_f32)
    int out_f32;
    float* lse;                // final: [rows][64] or nullptr
    int whole;                 // queries that are one item each; the others have nsplit each (parts)
    float* part_o;             // [parts][64][512] normalised partial outputs
    float* part_lse;           // [parts][64]
    float scale_log2;          // scale * log2(e)
    int32_t* status;           // device error word
    PageTable pages;           // paged cache (pages.table == nullptr: dense rows)
    int l2_prefetch;           // 1: rows go into L2 a tile before their copy (want_l2_prefetch)
    int dense;                 // 1: key j is row j, though its page is looked up (rows expanded from a paged cache)
};

// P^T, and so O^T, hold a group's 16 heads in another order than S^T: position p is head head_at(p).  A thread that
// holds heads 2 a, 2 a + 1, 8 + 2 a, 9 + 2 a of S^T (a = lane % 4) writes them as four neighbouring bytes.  Four
// heads of four keys a thread, in place of 16 heads of one key: the heads' scales and references stay in registers
// (prefill of 4096 queries 1148 -> 1140 us, of 333 112.7 -> 110.7).
__device__ __forceinline__ constexpr int head_at(int p) { return 8 * ((p >> 1) & 1) + 2 * (p >> 2) + (p & 1); }

// Items: the whole queries, then the parts of the others; Item::split is the part's number, -1 for a whole query.
__device__ __forceinline__ Item item_at(const AttnQ8Params& p, int item) {
    Item it{item, -1, 0, 0, p.top_k, 0};
    if (item >= p.whole) {
        it.split = item - p.whole;
        it.row = p.whole + it.split / p.nsplit;
        it.slot0 = it.split % p.nsplit * p.split_len;
        it.slot_end = min(p.top_k, it.slot0 + p.split_len);
    }
    it.batch = p.prefill ? 0 : it.row;
    it.bound = p.kv_len ? min(__ldg(p.kv_len + it.batch), p.Nmax) : p.Nmax;
    return it;
}

// log2 on the special-function unit; exact for the powers of two that the cache holds.
__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The rows of this CTA's tiles, tile after tile, one a lane (row `base` of a tile), in two steps so that the
// loads of one are in flight while the caller works: fetch() loads the selected key of the next tile,
// resolve() turns it into a cache row (a page lookup when paged).
struct RowStream {
    int s = 0, tiles = 0;               // next item of the CTA; tiles of the current one still to fetch
    const int32_t* at = nullptr;        // this lane's slot of the next tile, and the slots from it to the item's end
    int left = 0, batch = 0, bound = 0;
    int key = -1;
    bool first = false;                 // the fetched tile is its item's first

    __device__ __forceinline__ bool fetch(const AttnQ8Params& p, uint32_t lane, int base) {
        first = false;
        while (tiles == 0) {
            const int it = nth_item(p, s++);
            if (it == -1) return false;
            if (it < 0) continue;
            const Item I = item_at(p, it);
            at = p.idx + (int64_t)I.row * p.top_k + I.slot0 + base;
            left = I.slot_end - I.slot0 - base;
            batch = I.batch;
            bound = I.bound;
            first = true;
            key = left > 0 ? __ldg(at) : -1;    // beside the loads of item_tiles
            tiles = item_tiles(p, I, lane);
        }
        if (!first) key = left > 0 ? __ldg(at) : -1;
        at += kTile;
        left -= kTile;
        --tiles;
        return true;
    }
    // cache row of the fetched key; -1: no key, -2: a page outside the pool (a row of zeros)
    __device__ __forceinline__ int resolve(const AttnQ8Params& p) const {
        if (key < 0) return -1;
        if (key >= bound) {
            raise_dev_error(p.status, DEV_ERR_BOUNDS);
            return -1;
        }
        if (!p.pages.table) return (int)((int64_t)batch * p.Nmax + key);
        const int row = (int)paged_row(p.pages, batch, key);
        if (row >= 0) return p.dense ? key : row;
        raise_dev_error(p.status, DEV_ERR_BOUNDS);
        return -2;
    }
};

template <bool Q4>
__device__ __forceinline__ bool codes_are_zero(const uint8_t* at) {   // kLaneCodes bytes, zeros of either sign
    if (Q4) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
        return ((v.x | v.y) & kQ4Magnitudes) == 0;
    }
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(at));
    return ((v.x | v.y | v.z | v.w) & 0x7f7f7f7fu) == 0;
}

// The scale sc of the lane's row, or kZeroRowScale where the row's latent dims are zeros, by a warp: each lane looks at
// its row's first codes, and the warp together at the rows that begin with zeros.  (Two or four rows at once took
// registers that the kernel has not: 1.13 -> 1.15, 1.17 ms without any such row.)
template <bool Q4>
__device__ __forceinline__ float row_scale(const uint8_t* cache, int row, float sc, uint32_t lane) {
    constexpr int kBytes = Rows<Q4>::kBytes;
    const bool maybe = sc >= 1.f && codes_are_zero<Q4>(cache + (int64_t)row * kBytes);
    for (uint32_t m = __ballot_sync(0xffffffffu, maybe); m; m &= m - 1) {
        const int l = __ffs(m) - 1;
        const int64_t r = __shfl_sync(0xffffffffu, row, l);
        const bool zero = codes_are_zero<Q4>(cache + r * kBytes + Rows<Q4>::kLaneCodes * lane);
        if (__all_sync(0xffffffffu, zero) && (int)lane == l) sc = kZeroRowScale;
    }
    return sc;
}

// Query head h from its bf16 dims to its e4m3 parts, in place, by a warp: lane l holds dims 16 l .. 16 l + 15.
__device__ __forceinline__ void convert_head(uint8_t* smem, int qbuf, int h, float scale_log2, uint32_t lane) {
    const int j = (int)(lane >> 2), pc = 2 * (int)(lane & 3);
    const uint8_t* raw = smem + OFF_QHL + (j & 3) * kBlk + ((j >> 2) * kH + h) * 128;
    const uint4 a = *reinterpret_cast<const uint4*>(raw + ((pc ^ (h & 7)) << 4));
    const uint4 b = *reinterpret_cast<const uint4*>(raw + (((pc + 1) ^ (h & 7)) << 4));
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));
    // magnitudes compare as their bit patterns do; every lane has read its dims when this returns
    const int e = e4m3_scale_exponent(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax))));
    const float inv = exp2_int(-e);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        split_e4m3x4(bf16_lo(w[2 * k]) * inv, bf16_hi(w[2 * k]) * inv, bf16_lo(w[2 * k + 1]) * inv,
                     bf16_hi(w[2 * k + 1]) * inv, hi[k], lo[k]);
    uint8_t* d = smem + OFF_QHL + (int)(lane >> 3) * kBlk + h * 128 + (((int)(lane & 7) ^ (h & 7)) << 4);
    __syncwarp();
    *reinterpret_cast<uint4*>(d) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(d + kH * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    if (lane == 0) reinterpret_cast<float*>(smem + OFF_QS)[qbuf * kH + h] = scale_log2 * exp2_int(e);
}

__device__ __forceinline__ void store_lse(const AttnQ8Params& p, int row, int split, int h, float v) {
    if (split >= 0)
        p.part_lse[(int64_t)split * kH + h] = v;
    else if (p.lse)
        p.lse[(int64_t)row * kH + h] = v;
}

// An item without a selected key: zeros and lse = -inf, by all workers.
__device__ __noinline__ void zero_item(const AttnQ8Params& p, int row, int split, int tid) {
    if (tid < kH) store_lse(p, row, split, tid, -INFINITY);
    const int n = kH * kDv * (split >= 0 || p.out_f32 ? 4 : 2) / 16;
    uint4* d = split >= 0 ? reinterpret_cast<uint4*>(p.part_o) + (int64_t)split * n
                          : static_cast<uint4*>(p.out) + (int64_t)row * n;
#pragma unroll 1
    for (int i = tid; i < n; i += kWorkers) d[i] = make_uint4(0, 0, 0, 0);
}

// SPLIT: one item a CTA, a part of a query; else persistent CTAs, whole queries and then parts.
// Q4: the 4-bit cache, whose rows are expanded to the same e4m3 tile on their way to shared memory.
template <bool SPLIT, bool Q4>
__global__ void __launch_bounds__(kThreads, 1) mla_attn_q8_kernel(const __grid_constant__ CUtensorMap tmap_q, const AttnQ8Params p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023u) {   // the operands' swizzle counts from 1 KB boundaries; there is no room to round up
        if (threadIdx.x == 0) raise_dev_error(p.status, DEV_ERR_TIMEOUT);
        return;
    }
    // warps that convert a whole query: latent and rope warps; the rope warps of the 4-bit cache have no registers for it
    constexpr int kConverters = Q4 ? kGatherWarps : kGatherWarps + kRopeWarps;
    float2* sc_s = reinterpret_cast<float2*>(smem + OFF_SC);
    float* ic_s = reinterpret_cast<float*>(smem + OFF_IC);
    int* small_s = reinterpret_cast<int*>(smem + OFF_SMALL);
    float* qs_s = reinterpret_cast<float*>(smem + OFF_QS);
    float* red = reinterpret_cast<float*>(smem + OFF_RED);
    float* m_neg = reinterpret_cast<float*>(smem + OFF_MNEG);
    float* delta_s = reinterpret_cast<float*>(smem + OFF_DELTA);
    float* invl_s = reinterpret_cast<float*>(smem + OFF_INVL);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    uint64_t* freed = full + kSlots;
    uint64_t* rope_full = freed + 2 * kStages;
    uint64_t* s_full = rope_full + 1;
    uint64_t* s_free = rope_full + 2;
    uint64_t* p_full = rope_full + 3;
    uint64_t* q_free = rope_full + 4;
    uint64_t* q_raw = rope_full + 5;
    uint64_t* q_full = rope_full + 6;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_TMEM);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_ABORT);

    const int warp = threadIdx.x / 32;
    const uint32_t lane = lane_id();

    if (threadIdx.x == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&full[i], Q4 ? kGatherWarps : kGatherWarps * 32);   // one cp.async arrival per gather thread
        }
        for (int i = 0; i < 2 * kStages; ++i) mbar_init(&freed[i], kPvIssuers);   // both issuers' commits of a chunk
        mbar_init(rope_full, kRopeWarps);
        mbar_init(s_full, 2);                   // the QK issuer: its commit, and that it has seen the rows' scales
        mbar_init(s_free, kWorkerWarps);
        mbar_init(p_full, kWorkerWarps);
        mbar_init(q_free, 1);
        mbar_init(q_raw, 1);
        mbar_init(q_full, SPLIT ? kWorkerWarps : kConverters);
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
    if (Q4 && threadIdx.x < 256)
        reinterpret_cast<uint2*>(smem + OFF_TABLE)[threadIdx.x] =
            threadIdx.x < kQ4Scales ? q4_table(q4_block_scale(threadIdx.x)) : make_uint2(0, 0);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();                 // inputs and outputs may belong to the previous kernel until here

    // Chunk c of the CTA's g-th tile lies in slot 4 (g % 2) + c; the slots' barriers are in their use g / 2.  PV frees
    // them by pairs: chunks 0 and 1 (one of each issuer), then 2 and 3.
    if (warp < kFirstGather) setmaxnreg_dec<kIssueRegs>();
    if (warp == 0) {
        // ------------------------------------------------------------ QK issuer
        int gt = 0, qi = 0;
        bool ok = true;
        for (int s = 0; ok; ++s) {
            const int item = nth_item(p, s);
            if (item == -1) break;
            if (item < 0) continue;
            const Item I = item_at(p, item);
            const int T = item_tiles(p, I, lane);
            if (T == 0) continue;
            const uint32_t base = (smem_u32(smem) >> 4) | ((16u >> 4) << 16);   // leading offset: one atom wide
            for (int t = 0; ok && t < T; ++t, ++gt) {
                // A poll between MMAs waits until the tensor core has taken those before it (about 300 cycles), and each
                // of several in a row takes its own time: a lane a barrier, the warp looks at all of them at once.
                // Lanes 0-3: the rope rows, chunks 0 and 1, that the workers have read the previous tile's S^T; lane 4:
                // the query; 5, 6: chunks 2 and 3, whose coming may be waited for between the MMAs.
                uint64_t* ch = full + 4 * (gt & 1);
                const uint32_t par = (gt >> 1) & 1;
                uint64_t* mine = lane == 0 ? rope_full : lane == 3 ? s_free : lane == 4 ? q_full
                                 : lane < 3 ? ch + lane - 1 : lane < 7 ? ch + lane - 3 : ch;
                const uint32_t mpar = lane == 0 ? gt & 1 : lane == 3 ? (gt & 1) ^ 1 : lane == 4 ? qi & 1 : par;
                auto poll = [&](uint32_t need) { return mbar_poll_warp(mine, mpar, lane, 7, need, abort_flag, p.status); };
                // 4-bit rows: the warps that bring the rope rows expand chunks 2 and 3 before them, so the rope product is last.
                constexpr uint32_t kFirst = Q4 ? 0x1e : 0x1f, kRest = Q4 ? 0x61 : 0x60;
                const uint32_t got = poll(kFirst);
                ok = got != 0;
                if (!ok) break;
                const uint32_t lat = base + (OFF_LAT >> 4) + (gt & 1) * (kChunks * kBlk >> 4);
                auto chunk = [&](int c) {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)       // 32 dims a step
                        mma_e4m3_ss_lo(tmem_base + TM_S, lat + c * (kBlk >> 4) + 2 * kk, kDescHi,
                                       base + (OFF_QHL >> 4) + c * (kBlk >> 4) + 2 * kk, kDescHi, IDESC_QK, (c | kk) ? 1u : 0u);
                };
                fence_proxy_async_smem();   // of every lane that saw a barrier, before the lane that issues
                __syncwarp();
                tc_fence_after();
                auto rope = [&] {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)       // 16 dims a step, the keys from tensor memory
                        mma_bf16_ts_lo(tmem_base + TM_R, tmem_base + TM_K + 8 * kk, base + (OFF_QR >> 4) + 2 * kk, kDescHi,
                                       IDESC_ROPE, kk ? 1u : 0u);
                };
                if (lane == 0) {
                    chunk(0);
                    chunk(1);
                    if (!Q4) rope();
                }
                __syncwarp();
                if ((got & kRest) != kRest) {
                    ok = poll(kRest) != 0;
                    if (!ok) break;
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (Q4) tc_fence_after();
                if (lane == 0) {
                    chunk(2);
                    chunk(3);
                    if (Q4) rope();
                    mbar_arrive(s_full);
                    mma_commit(s_full);
                    if (t == T - 1) mma_commit(q_free);
                }
                __syncwarp();
            }
            ++qi;
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
            const Item I = item_at(p, item);
            const int T = item_tiles(p, I, lane);
            if (lane == 0) {
                // A = V^T MN-major: 128 dims a row, 8-key groups 1 KB apart; B = P^T MN-major, hi at byte 0 of a
                // row, lo at byte 64
                const uint32_t base = (smem_u32(smem) >> 4) | ((uint32_t)(kBlk >> 4) << 16);
                for (int t = 0; ok && t < T; ++t, ++gt) {
                    if (!(ok = mbar_poll(p_full, gt & 1, abort_flag, p.status))) break;
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
                        mma_commit(&freed[2 * (gt & 1) + j]);
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        }
    } else if (warp == kQueryWarp) {
        // ------------------------------------------------------------ queries (TMA)
        int qi = 0;
        bool ok = true;
        for (int s = 0; ok; ++s) {
            const int item = nth_item(p, s);
            if (item == -1) break;
            if (item < 0) continue;
            const Item I = item_at(p, item);
            if (item_tiles(p, I, lane) == 0) continue;
            if (lane == 0) {
                if (qi > 0) l2_prefetch_bulk(p.q + (int64_t)I.row * (kH * DSA_QK_DIM), kH * DSA_QK_DIM * 2);
                // QK of the item before is complete: its query's place is free
                ok = mbar_poll(q_free, (qi & 1) ^ 1, abort_flag, p.status);
                if (ok) {
                    // the query as it is, into the place of its e4m3 parts: dims 64 j.. of the heads go where the rows
                    // of chunk j % 4 will be, hi rows for j < 4, lo rows for the others
                    mbar_arrive_expect_tx(q_raw, kH * DSA_QK_DIM * 2);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        tma_load_2d(smem + OFF_QHL + (j & 3) * kBlk + (j >> 2) * (kH * 128), &tmap_q, q_raw, 64 * j, I.row * kH);
                    tma_load_2d(smem + OFF_QR, &tmap_q, q_raw, kQ8Latent, I.row * kH);
                }
                ++qi;
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        }
    } else if (warp >= kFirstGather && warp < kFirstWorker) {
        // ------------------------------------------------------------ gather: latent rows, rope rows, queries
        constexpr int kBytes = Rows<Q4>::kBytes;
        const bool is_rope = warp >= kFirstRope;
        const int gw = (warp - kFirstGather) & 3; // rows 32 gw .. 32 gw + 31 of a tile
        constexpr int kQHeads = kH / kConverters;   // a warp's
        const int qh0 = kQHeads * (warp - kFirstGather);
        const uint32_t smem_base = smem_u32(smem);
        // One thread polls (the roles' pollers on different schedulers), a named barrier releases the four warps.  (A
        // thread suspended in try_wait was seen to resume 800 to 3400 cycles after the phase had completed; warps that
        // poll for themselves copy out of step.)  The answer is the same in every warp: all leave together when a wait gives up.
        auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            bool ok = true;
            if (gw == (is_rope ? 2 : 1) && lane == 0) ok = mbar_poll(bar, parity, abort_flag, p.status);
            return named_bar_and(kGatherBar + (is_rope ? 1 : 0), 128, ok);
        };
        int qi = 0;
        auto convert = [&]() -> bool {            // the warp's heads of the item's query, once it has landed
            if (!wait(q_raw, qi & 1)) return false;
#pragma unroll 2
            for (int i = 0; i < kQHeads; ++i) convert_head(smem, qi & 3, qh0 + i, p.scale_log2, lane);
            ++qi;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
            return true;
        };

        auto gather = [&](auto role) {            // of the latent rows, or the rope rows
            const bool rope = role;
            RowStream rs;
            const int base = 32 * gw + (int)lane;
            // `has`: there is a tile to copy, `row` its row; `more`: one is fetched behind it
            bool has = rs.fetch(p, lane, base);
            int row = has ? rs.resolve(p) : -1;
            bool first = rs.first, more = has && rs.fetch(p, lane, base);
            // latent rows: a warp instruction copies a 128-byte block of four different rows, 8 lanes a row; this lane's
            // rows are 32 gw + 4 i + l / 8
            const int ci = (int)(lane >> 3), cc = (int)(lane & 7);
            const uint32_t dst0 = smem_base + OFF_LAT + (uint32_t)((32 * gw + ci) * 128);
            const uint32_t sw0 = (uint32_t)((cc ^ ci) << 4), sw1 = (uint32_t)((cc ^ (4 + ci)) << 4);
            // 4-bit rows: the latent warps expand chunks 0 and 1, the rope warps 2 and 3, a lane its own row.  Its codes and
            // block bytes are in registers when their place comes free.  (A row's pieces on eight lanes, as the copies of
            // 8-bit rows have them, took 16 shuffles and twice the loads.)  The eight lanes of a store's phase have eight
            // different rows mod 8: by the swizzle no bank twice.
            const int kChunk = rope ? 2 : 0;          // the first of the warp's two
            uint32_t x0[16], x1[16], block[4];
            auto load = [&](uint32_t (&x)[16], const uint8_t* src, int c) {
                ldg_nc_v8(src + 64 * c, x);
                ldg_nc_v8(src + 64 * c + 32, x + 8);
            };
            auto expand = [&](const uint32_t (&x)[16], int g, int c) {
                const uint32_t table = smem_base + OFF_TABLE;
                const uint32_t dst = smem_base + OFF_LAT + (g & 1) * (kChunks * kBlk) + c * kBlk + base * 128 + ((base & 7) << 4);
                // A table's load is ahead of the store before it.
                uint2 t = lds_v2(table + 8 * (block[2 * (c - kChunk)] & 0xff));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint2 u = t;
                    if (i < 7) u = lds_v2(table + 8 * __byte_perm(block[2 * (c - kChunk) + ((i + 1) >> 2)], 0, 0x4440 + ((i + 1) & 3)));
                    const uint2 a = q4_expand(x[2 * i], t), b = q4_expand(x[2 * i + 1], t);
                    sts_v4(dst ^ (i << 4), a.x, a.y, b.x, b.y);
                    t = u;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[4 * (g & 1) + c]);
            };
            constexpr int kEarly = 2;                 // quarters of the rope dims loaded while a chunk is expanded
            float sc1 = kZeroRowScale;                // the scale of the rope warps' next row
            auto load_row = [&](int row) {
                const uint8_t* src = row < 0 ? g_no_row : p.cache + (int64_t)row * kBytes;
                // (a sector that the latent and the rope warps share: without L1, decode of 256 sequences 145 -> 148.5 us)
                ldg_nc_v4(src + kQ4Codes + 8 * kChunk, block);
                load(x0, src, kChunk);
                load(x1, src, kChunk + 1);
                if (rope) sc1 = row >= 0 ? ldg_nc_f32(p.cache_scale + row) : kZeroRowScale;
            };
            if constexpr (Q4) load_row(row);
            for (int g = 0; has; ++g) {
                const int row1 = more ? rs.resolve(p) : -1;
                const bool first1 = rs.first, has1 = more;
                // a row of a large cache into L2 a tile before it is copied (by the time of the copy HBM has answered)
                if (p.l2_prefetch && !rope && row1 >= 0) l2_prefetch_bulk(p.cache + (int64_t)row1 * kBytes, kBytes);
                more = more && rs.fetch(p, lane, base);
                if (rope) {
                    // A lane carries one key's 64 rope dims (128 bytes) through registers into its lane of tensor memory:
                    // the loads run ahead, and only the store waits for QK of the tile before.
                    uint32_t k[32];
                    float sc = kZeroRowScale;         // of a page outside the pool
                    const uint8_t* src = row < 0 ? g_no_row : p.cache + (int64_t)row * kBytes + Rows<Q4>::kRope;
                    auto load_k = [&](int from, int to) {
#pragma unroll
                        for (int i = from; i < to; ++i) ldg_nc_v8(src + 32 * i, k + 8 * i);
                    };
                    if constexpr (Q4) {
                        if (!wait(&freed[2 * (g & 1) + 1], ((g >> 1) & 1) ^ 1)) break;
                        expand(x0, g, 2);
                        load_k(0, kEarly);
                        expand(x1, g, 3);
                        load_k(kEarly, 4);
                        sc = sc1;
                    } else {
                        load_k(0, 4);
                        if (row >= 0) sc = __ldg(p.cache_scale + row);
                    }
                    sc = row_scale<Q4>(p.cache, row, sc, lane);
                    if (g > 0 && !wait(s_full, (g - 1) & 1)) break;   // QK of the tile before is complete
                    tc_fence_after();
                    __syncwarp();
                    tmem_st32(tmem_base + TM_K + (static_cast<uint32_t>(32 * gw) << 16), k);
                    sc_s[(g & 1) * kTile + base] = row == -1 ? make_float2(0.f, -INFINITY) : make_float2(sc, lg2_approx(sc));
                    ic_s[(g & 3) * kTile + base] = row == -1 ? 0.f : 1.f / sc;
                    const bool small = __any_sync(0xffffffffu, row != -1 && sc < kSmallScale);
                    if (lane == 0) small_s[(g & 3) * 4 + gw] = small;
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(rope_full);
                } else if constexpr (Q4) {
                    if (!wait(&freed[2 * (g & 1)], ((g >> 1) & 1) ^ 1)) break;
                    expand(x0, g, 0);
                    expand(x1, g, 1);
                } else {
                    const uint8_t* mine = row < 0 ? g_no_row : p.cache + (int64_t)row * kQ8Row;
                    const uint8_t* src[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        src[i] = reinterpret_cast<const uint8_t*>(__shfl_sync(
                                     0xffffffffu, reinterpret_cast<unsigned long long>(mine), 4 * i + ci)) + cc * 16;
                    const uint32_t dst = dst0 + (g & 1) * (kChunks * kBlk);
                    bool ok = true;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        ok = ok && wait(&freed[2 * (g & 1) + half], ((g >> 1) & 1) ^ 1);
                        if (ok) {
#pragma unroll
                            for (int c = 2 * half; c < 2 * half + 2; ++c) {
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    cp_async_16(dst + c * kBlk + i * 512 + ((i & 1) ? sw1 : sw0), src[i] + c * 128);
                                cp_async_arrive_noinc(&full[4 * (g & 1) + c]);
                            }
                        }
                    }
                    if (!ok) break;
                }
                if (!(Q4 && rope) && !SPLIT && first && !convert()) break;   // split: the workers, idle so far, convert the only query
                row = row1;
                first = first1;
                has = has1;
                if constexpr (Q4) load_row(row);
            }
        };
        // 8-bit rows: one loop for both kinds of warps (a loop each: decode of 256 sequences 99 -> 104 us, of 37 18.7 -> 19.2).
        // 4-bit rows: a loop each, in which the role is a constant.
        if constexpr (!Q4) {
            setmaxnreg_dec<kGatherRegs>();
            gather(is_rope);
        } else if (is_rope) {
            setmaxnreg_dec<kGatherRegs>();
            gather(std::true_type{});
        } else {
            setmaxnreg_dec<kGatherRegs>();
            gather(std::false_type{});
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
            if (tid == 3 * 32) ok = mbar_poll(bar, parity, abort_flag, p.status);
            return named_bar_and(1, kWorkers, ok);
        };
        auto pv_done = [&](int g) -> bool {           // PV has consumed tile g (most often it has: every lane looks)
            return mbar_poll(&freed[2 * (g & 1) + 1], (g >> 1) & 1, abort_flag, p.status);
        };

        // ---- items.  One without a selected key gets zeros and lse = -inf here.
        int n_s = 0, n_item = 0, nT = 0;
        auto next_item = [&]() -> bool {
            for (;;) {
                n_item = nth_item(p, n_s++);
                if (n_item == -1) return false;
                if (n_item < 0) continue;
                const Item nI = item_at(p, n_item);
                nT = item_tiles(p, nI, lane);
                if (nT > 0) return true;
                zero_item(p, nI.row, nI.split, tid);
            }
        };

        // `gok` is the thread's wait status: a wait that gives up does not change the control flow inside an item
        // (all workers keep meeting the same named barriers); the consensus barrier at the item's end takes all
        // out together.
        bool gok = true;
        bool more = next_item();
        bool failed = false;
        if (SPLIT && more) {
            gok = wait_all(q_raw, 0);
#pragma unroll 1
            for (int i = 0; i < kH / kWorkerWarps; ++i)
                convert_head(smem, 0, kH / kWorkerWarps * ww + i, p.scale_log2, lane);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_full);
        }
        int gt = 0;                               // tiles done by this CTA
        int qbuf = 0;                             // the item's query scales
        while (more && !failed) {
            const int item = n_item, T = nT;
            named_bar_sync(1, kWorkers);          // the previous item's readers of m_neg / invl are done
            if (tid < kH) m_neg[tid] = 0.f;
            bool unset = true;
            // of the thread's heads h0 + 8 b + 2 (l % 4), + 1: row sums, scales, minus the references
            float2 l2[2], qs2[2], mn2[2];
#pragma unroll
            for (int b = 0; b < 2; ++b) l2[b] = qs2[b] = mn2[b] = make_float2(0.f, 0.f);
            named_bar_sync(1, kWorkers);
            for (int t = 0; t < T; ++t, ++gt) {
                gok = wait_all(s_full, gt & 1) && gok;
                tc_fence_after();
                if (t == 0)
#pragma unroll
                    for (int b = 0; b < 2; ++b)
                        qs2[b] = reinterpret_cast<const float2*>(qs_s + qbuf * kH + h0)[4 * b + (lane & 3)];
                // The exponents e = log2(e) s + log2(c) - m of the thread's 16 weights: keys 16 f + 8 r + l / 4 of the warp's
                // 32 (their scales sc[2 f + r]) with the heads above: e2[4 f + 2 b + r].
                const float2* my_sc = sc_s + (gt & 1) * kTile + quad * 32 + (int)(lane >> 2);
                const float* my_ic = ic_s + (gt & 3) * kTile + quad * 32 + (int)(lane >> 2);
                float2 e2[kHG / 2];
                {
                    float2 sc[4];                 // c and log2 c
                    uint32_t hi[2][8], lo[2][8], ro[2][8];
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        const uint32_t at = tmem_base + lane_addr + (16u * f << 16) + h0;
                        tmem_ld_16x256b_x2(at + TM_S, hi[f]);
                        tmem_ld_16x256b_x2(at + TM_S + 64, lo[f]);
                        tmem_ld_16x256b_x2(at + TM_R, ro[f]);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) sc[k] = my_sc[8 * k];
                    tmem_ld_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_free);
                    const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
                    const float2 sixteenth = make_float2(0.0625f, 0.0625f);
#pragma unroll
                    for (int f = 0; f < 2; ++f)
#pragma unroll
                        for (int b = 0; b < 2; ++b)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const int i = 4 * b + 2 * r;
                                const float2 s = sc[2 * f + r];
                                const float2 x = make_float2(__uint_as_float(hi[f][i]), __uint_as_float(hi[f][i + 1]));
                                const float2 y = make_float2(__uint_as_float(lo[f][i]), __uint_as_float(lo[f][i + 1]));
                                const float2 z = make_float2(__uint_as_float(ro[f][i]), __uint_as_float(ro[f][i + 1]));
                                e2[4 * f + 2 * b + r] =
                                    __ffma2_rn(__ffma2_rn(y, sixteenth, x), __fmul2_rn(qs2[b], make_float2(s.x, s.x)),
                                               __ffma2_rn(z, sl2, __fadd2_rn(make_float2(s.y, s.y), mn2[b])));
                            }
                }
                // The vote on moving a reference, and the rare move, involve the group's four warps only.  While no key
                // has been seen (`unset`, the same in the whole group: a padding slot is one for every head) the
                // reference is 0 and there is nothing to vote on.
                bool any_upd = false;
                bool move = unset;
                if (!unset) {
                    float top = e2[0].x;
#pragma unroll
                    for (int i = 0; i < kHG / 2; ++i) top = fmaxf(fmaxf(top, e2[i].x), e2[i].y);
                    move = named_bar_or(group_bar, kGroupThreads, top > kMostTop);
                }
                if (move) {
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        float2 x = e2[2 * b];
#pragma unroll
                        for (int k = 1; k < 4; ++k) {
                            const float2 y = e2[4 * (k >> 1) + 2 * b + (k & 1)];
                            x = make_float2(fmaxf(x.x, y.x), fmaxf(x.y, y.y));
                        }
#pragma unroll
                        for (int o = 4; o < 32; o *= 2) {
                            x.x = fmaxf(x.x, __shfl_xor_sync(0xffffffffu, x.x, o));
                            x.y = fmaxf(x.y, __shfl_xor_sync(0xffffffffu, x.y, o));
                        }
                        if (lane < 4) reinterpret_cast<float2*>(red + quad * kH + h0)[4 * b + lane] = x;
                    }
                    named_bar_sync(group_bar, kGroupThreads);
                    bool seen = false;
                    if (ww == 4 * hg && lane < kHG) {   // one lane per head of the group
                        const int h = h0 + (int)lane;
                        const float top = fmaxf(fmaxf(red[h], red[kH + h]), fmaxf(red[2 * kH + h], red[3 * kH + h]));
                        float d = 0.f;                  // how far the reference rises
                        if (top > (unset ? -INFINITY : kMostTop)) d = top - kFirstTop;
                        m_neg[h] -= d;
                        delta_s[h] = d;
                        seen = top > -INFINITY;
                    }
                    // any key at all: the references are set; from then on a move scales the sums
                    seen = named_bar_or(group_bar, kGroupThreads, seen);
                    any_upd = !unset;
                    unset = unset && !seen;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const float2 d = reinterpret_cast<const float2*>(delta_s + h0)[4 * b + (lane & 3)];
                        mn2[b] = make_float2(mn2[b].x - d.x, mn2[b].y - d.y);
                        if (any_upd) {            // in two steps: a sum of up to 2^84 outlives a rise past 126
                            const float2 h = make_float2(ex2_approx(-0.5f * d.x), ex2_approx(-0.5f * d.y));
                            l2[b] = __fmul2_rn(__fmul2_rn(l2[b], h), h);
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float2& e = e2[4 * (k >> 1) + 2 * b + (k & 1)];
                            e = make_float2(e.x - d.x, e.y - d.y);
                        }
                    }
                }
                // looked at before the exponentials, so that the poll's time does not follow theirs
                const bool early = gt == 0 || mbar_test_wait(&freed[2 * ((gt - 1) & 1) + 1], ((gt - 1) >> 1) & 1);
                // A row of small scale may have its part in the sum though its P' is below float32's numbers: the weight
                // without the scale, then.  (Without a row below kSmallScale nothing is lost: what P' < 2^-126 adds is
                // below 2^-106, and the sum at least 2^(4.5 - 64).)
                if (small_s[(gt & 3) * 4 + quad]) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float c1 = my_ic[8 * k];
                        if (c1 > 1.f / kSmallScale) {
                            const float lc1 = lg2_approx(c1);
#pragma unroll
                            for (int b = 0; b < 2; ++b) {
                                const float2 x = e2[4 * (k >> 1) + 2 * b + (k & 1)];
                                if (x.x < kLeastExponent) l2[b].x += ex2_approx(x.x + lc1);
                                if (x.y < kLeastExponent) l2[b].y += ex2_approx(x.y + lc1);
                            }
                        }
                    }
                }
                // P' and its two e4m3 parts; the row sum takes the float32 weight with the row's scale divided out
                uint32_t whi[4], wlo[4];          // four heads of each of the thread's keys
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 x0 = e2[4 * (k >> 1) + (k & 1)], x1 = e2[4 * (k >> 1) + 2 + (k & 1)];
                    const float2 p0 = make_float2(ex2_approx(x0.x), ex2_approx(x0.y));
                    const float2 p1 = make_float2(ex2_approx(x1.x), ex2_approx(x1.y));
                    const float c1 = my_ic[8 * k];
                    const float2 ic = make_float2(c1, c1);
                    l2[0] = __ffma2_rn(p0, ic, l2[0]);
                    l2[1] = __ffma2_rn(p1, ic, l2[1]);
                    split_e4m3x4(p0.x, p0.y, p1.x, p1.y, whi[k], wlo[k]);
                }
                if (!early) gok = gok && pv_done(gt - 1);   // P^T and O^T are free
                if (any_upd) {                    // t > 0: some key came before
                    tc_fence_after();
#pragma unroll 1
                    for (int ch = 0; ch < kChunks; ++ch) {
                        uint32_t v[kHG];
                        const uint32_t a = tmem_base + lane_addr + TM_O + 64 * ch + h0;
                        tmem_ld16(a, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < kHG; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * ex2_approx(-delta_s[h0 + head_at(k)]));
                        tmem_st16(a, v);
                    }
                    tmem_st_wait();
                    tc_fence_before();
                }
                {   // P^T row `key`: 16 heads hi at 16-byte piece hg of the swizzled row, lo at piece 4 + hg
                    const uint32_t d = smem_u32(smem + OFF_P + key * 128);
                    __syncwarp();
                    stmatrix_x4(d + ((hg ^ (key & 7)) << 4), whi);
                    stmatrix_x4(d + (((4 + hg) ^ (key & 7)) << 4), wlo);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full);
                if (t == 0) more = next_item();   // its loads beside PV
            }
            qbuf = (qbuf + 1) & 3;
            // ---------------- final: l = sum of partial row sums; out = O^T / l
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int o = 4; o < 32; o *= 2) {
                    l2[b].x += __shfl_xor_sync(0xffffffffu, l2[b].x, o);
                    l2[b].y += __shfl_xor_sync(0xffffffffu, l2[b].y, o);
                }
                if (lane < 4) reinterpret_cast<float2*>(red + quad * kH + h0)[4 * b + lane] = l2[b];
            }
            if (!named_bar_and(2, kWorkers, gok && pv_done(gt - 1))) {
                failed = true;
                break;
            }
            tc_fence_after();
            const Item I = item_at(p, item);
            if (tid < kH) {
                const float l = red[tid] + red[kH + tid] + red[2 * kH + tid] + red[3 * kH + tid];
                // l = 0: every selected key was outside the cache
                invl_s[tid] = (l > 0.f) ? 1.f / l : (l == 0.f ? 0.f : l);
                store_lse(p, I.row, I.split, tid,
                          (l > 0.f) ? (log2f(l) - m_neg[tid]) * 0.6931471805599453f : (l == 0.f ? -INFINITY : l));
            }
            named_bar_sync(1, kWorkers);
            if (SPLIT) {                          // the CTA's part, float32: a store of a warp is 128 bytes of a head
                float* part = p.part_o + ((int64_t)I.split * kH + h0) * kDv + key;
#pragma unroll 2
                for (int ch = 0; ch < kChunks; ++ch) {
                    uint32_t v[kHG];
                    tmem_ld16(tmem_base + lane_addr + TM_O + 64 * ch + h0, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int h = 0; h < kHG; ++h) __stcg(part + head_at(h) * kDv + ch * 128, __uint_as_float(v[h]) * invl_s[h0 + head_at(h)]);
                }
                tc_fence_before();
                continue;
            }
            // P^T is consumed: each warp takes 1 KB of its block to turn its 32 dims x 16 heads so that a store
            // writes 16 contiguous bytes of a head a lane.
            uint8_t* stage = smem + OFF_P + ww * 1024;
            const bool f32 = p.out_f32 || I.split >= 0;
            float* out32 = (I.split >= 0 ? p.part_o + (int64_t)I.split * kH * kDv
                                         : static_cast<float*>(p.out) + (int64_t)I.row * kH * kDv) + h0 * kDv;
            __nv_bfloat16* out16 = static_cast<__nv_bfloat16*>(p.out) + ((int64_t)I.row * kH + h0) * kDv;
#pragma unroll 1
            for (int ch = 0; ch < kChunks; ++ch) {
                const int dim0 = ch * 128 + quad * 32;
                if (f32) {                        // a lane a dim, 8 heads at a time: rows of 32 dims
                    uint32_t v[kHG];
                    tmem_ld16(tmem_base + lane_addr + TM_O + 64 * ch + h0, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        __syncwarp();
#pragma unroll
                        for (int h = 0; h < 8; ++h)
                            reinterpret_cast<float*>(stage)[h * 32 + lane] =
                                __uint_as_float(v[8 * half + h]) * invl_s[h0 + head_at(8 * half + h)];
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int h = 4 * i + (int)(lane >> 3);
                            *reinterpret_cast<float4*>(out32 + head_at(8 * half + h) * kDv + dim0 + (int)(lane & 7) * 4) =
                                reinterpret_cast<const float4*>(stage)[h * 8 + (lane & 7)];
                        }
                    }
                } else {                          // 8 x 8 blocks (dims x heads) stored transposed: rows of 32 dims
                    uint32_t v[2][8];
#pragma unroll
                    for (int half = 0; half < 2; ++half)   // 16 dims: a lane has dims l / 4 and l / 4 + 8, heads 2 (l % 4), + 1
                        tmem_ld_16x256b_x2(tmem_base + lane_addr + (16u * half << 16) + TM_O + 64 * ch + h0, v[half]);
                    tmem_ld_wait();
                    __syncwarp();
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t w[4];            // blocks: dims 0-7 / 8-15 of heads 0-7, then of heads 8-15
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const float2 il = *reinterpret_cast<const float2*>(invl_s + h0 + head_at(8 * b + 2 * (int)(lane & 3)));
#pragma unroll
                            for (int r = 0; r < 2; ++r)
                                w[2 * b + r] = pack_bf16x2(__uint_as_float(v[half][4 * b + 2 * r]) * il.x,
                                                           __uint_as_float(v[half][4 * b + 2 * r + 1]) * il.y);
                        }
                        // row of block m that this lane addresses: head 8 (m / 2) + l % 8, dims 16 half + 8 (m % 2)
                        const int m = (int)(lane >> 3), h = 8 * (m >> 1) + (int)(lane & 7), pc = 2 * half + (m & 1);
                        stmatrix_x4_trans(smem_u32(stage) + h * 64 + ((pc ^ ((h >> 1) & 3)) << 4), w);
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int h = 8 * i + (int)(lane >> 2), pc = (int)(lane & 3);
                        *reinterpret_cast<uint4*>(out16 + head_at(h) * kDv + dim0 + pc * 8) =
                            *reinterpret_cast<const uint4*>(stage + h * 64 + ((pc ^ ((h >> 1) & 3)) << 4));
                    }
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

// Shared-memory limit of a kernel, raised once a device.
template <bool SPLIT, bool Q4>
dsa_status_t prepare_kernel() {
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> done[kMaxDevices];
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return DSA_ERR_CUDA;
    if (done[dev].load(std::memory_order_acquire)) return DSA_OK;
    const dsa_status_t st = ensure_smem_attr(reinterpret_cast<const void*>(mla_attn_q8_kernel<SPLIT, Q4>), kSmemBytes);
    if (st == DSA_OK) done[dev].store(true, std::memory_order_release);
    return st;
}

template <bool SPLIT, bool Q4>
dsa_status_t launch(const AttnQ8Params& p, cudaStream_t stream) {
    dsa_status_t st = prepare_kernel<SPLIT, Q4>();
    if (st != DSA_OK) return st;
    CUtensorMap tq;
    if ((st = make_tmap_bf16_2d(&tq, p.q, DSA_QK_DIM, (uint64_t)p.rows * kH, DSA_QK_DIM * 2, 64, kH)) != DSA_OK) return st;
    const int sms = device_sm_count();
    if (launch_pdl(mla_attn_q8_kernel<SPLIT, Q4>, dim3(p.n_items < sms ? p.n_items : sms), dim3(kThreads), kSmemBytes, stream,
                   tq, p) != cudaSuccess)
        return DSA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

// How a launch's queries are cut: `whole` of them run whole, the `cut` others in `splits` parts of `each` tiles,
// at most one part a CTA (SM), into the workspace, and are merged.
struct Cut {
    int whole, cut, splits, each;
};

// The queries behind the last full round of the SMs are cut when that is no slower: they would take an item's
// tiles (2.6 us each) with most SMs idle, and take, cut, a part's tiles and the merge, whose time grows with the
// queries (1 tile's for a few, 3 tiles' for 70; one more behind whole queries, whose CTAs lose the overlap with a
// next one).  Whole / cut, us: 1 query of 16 tiles 45.7 / 12.7; 4 of 2 tiles 15.5 / 12.9; 40 of 3 18.4 / 17.0; 70
// of 4 21.1 / 22.2, of 5 23.5 / 25.1, of 6 26.0 / 25.3; behind a full round, 1 of 16 tiles 87.8 / 56.4, 76 of 16
// 89.1 / 80.4, 8 of 3 tiles 30.0 / 27.1, 38 of 4 34.1 / 33.3, 68 of 6 43.9 / 45.2, of 8 52.5 / 51.7.
Cut cut_rows(int rows, int top_k) {
    const int sms = device_sm_count(), tiles = ceil_div(top_k, kTile);
    if (sms < 1) return Cut{rows, 0, 1, tiles};
    const int rest = rows % sms, most = rest > 0 ? sms / rest : 1;
    if (most < 2 || tiles < 2) return Cut{rows, 0, 1, tiles};
    const int n = ceil_div(tiles, most < tiles ? most : tiles);   // tiles a part
    if (n + 1 + rest / 32 + (rows > rest ? 1 : 0) > tiles) return Cut{rows, 0, 1, tiles};
    return Cut{rows - rest, rest, ceil_div(tiles, n), n};
}

// Rows go into L2 a tile before their copy when the keys of the call are more than half of L2 and an item has 8
// tiles or more to run ahead in; a prefetch of rows that L2 holds, or of few tiles, only takes from the copies.
// Without / with, us: 1216 queries at 16k keys (10 MB) 349 / 355, at 131k (84 MB) 379 / 375, at 1M 412 / 397;
// decode of 152 sequences of 8k 63.3 / 62.8, of 304 of 32k 122.4 / 120.0, of 32 of 131k (4 tiles an item) 29.7 / 30.4.
int want_l2_prefetch(int64_t keys, int split_len, int row_bytes) {
    return split_len >= 8 * kTile && (size_t)keys * row_bytes > device_l2_bytes() / 2 ? 1 : 0;
}

AttnQ8Params base_params(const void* q, const void* cache, const float* cache_scale, const int32_t* idx, int Nmax,
                         int top_k, float scale, void* out, int out_f32, float* lse, const PageTable& pages) {
    AttnQ8Params p{};
    p.idx = idx;
    p.Nmax = Nmax;
    p.top_k = top_k;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.cache = static_cast<const uint8_t*>(cache);
    p.cache_scale = cache_scale;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.out = out;
    p.out_f32 = out_f32;
    p.lse = lse;
    p.status = device_status_ptr();
    p.pages = pages;
    return p;
}

template <bool Q4>
dsa_status_t launch_rows(AttnQ8Params p, int rows, void* workspace, cudaStream_t stream) {
    const Cut c = cut_rows(rows, p.top_k);
    p.rows = rows;
    p.whole = c.whole;
    p.nsplit = c.splits;
    p.split_len = c.each * kTile;
    p.n_items = c.whole + c.cut * c.splits;
    p.l2_prefetch = want_l2_prefetch((p.prefill ? 1 : (int64_t)rows) * p.Nmax, c.whole > 0 ? p.top_k : p.split_len,
                                    Rows<Q4>::kBytes);
    p.part_o = static_cast<float*>(workspace);
    p.part_lse = p.part_o + (size_t)c.cut * c.splits * kH * kDv;
    const dsa_status_t st = c.whole > 0 ? launch<false, Q4>(p, stream) : launch<true, Q4>(p, stream);
    if (st != DSA_OK || c.cut == 0) return st;
    void* out = static_cast<char*>(p.out) + (int64_t)c.whole * kH * kDv * (p.out_f32 ? 4 : 2);
    float* lse = p.lse ? p.lse + (int64_t)c.whole * kH : nullptr;
    return launch_decode_combine(p.part_o, p.part_lse, c.cut, c.splits, out, p.out_f32, lse, stream);
}

}  // namespace

// A prefill over the 4-bit cache expands the cache's rows to 8-bit ones first, once for all its queries, where they
// select each key three times or more: a selected key then costs 0.13 ns in place of 0.19, a key of the cache 0.2 ns and
// the launch 2 us.  Direct / expanded, us: 8 queries of 2048 of 2k keys 15.3 / 15.9; 32 of 4k 26.2 / 24.1; 152 of 16k 64 / 51,
// of 131k (2.4 times each) 68 / 73; 608 of 131k 267 / 203, of 524k (2.4) 278 / 270; 4096 of 16k 1584 / 1111, of 2M (4)
// 1891 / 1545.
bool attn_q4_expands(int rows, int top_k, int N) { return N > 0 && (long long)rows * top_k >= 3LL * N + 24576; }

size_t attn_q8_workspace(int rows, int top_k) {
    const Cut c = cut_rows(rows, top_k);
    return (size_t)c.cut * c.splits * kH * (kDv + 1) * sizeof(float);
}

size_t attn_q4_workspace(int rows, int top_k, int N) {
    const size_t cut = attn_q8_workspace(rows, top_k);
    if (!attn_q4_expands(rows, top_k, N)) return cut;
    return round_up(cut) + round_up((size_t)N * kQ8Row) + (size_t)N * sizeof(float);
}

dsa_status_t launch_attn_q8_prefill(const void* q, const void* cache, const float* cache_scale, bool q4, bool expand,
                                    const int32_t* idx, int L, int N, int top_k, float scale, void* out, int out_f32,
                                    float* lse, void* workspace, const PageTable& pages, cudaStream_t stream) {
    AttnQ8Params p = base_params(q, cache, cache_scale, idx, N, top_k, scale, out, out_f32, lse, pages);
    p.prefill = 1;
    if (!q4) return launch_rows<false>(p, L, workspace, stream);
    if (!expand) return launch_rows<true>(p, L, workspace, stream);
    uint8_t* rows = static_cast<uint8_t*>(workspace) + round_up(attn_q8_workspace(L, top_k));
    float* scales = reinterpret_cast<float*>(rows + round_up((size_t)N * kQ8Row));
    const dsa_status_t st = launch_cache_expand_q4(cache, cache_scale, N, rows, scales, pages, stream);
    if (st != DSA_OK) return st;
    p.cache = rows;
    p.cache_scale = scales;
    p.dense = 1;
    return launch_rows<false>(p, L, workspace, stream);
}

dsa_status_t launch_attn_q8_decode(const void* q, const void* cache, const float* cache_scale, bool q4,
                                   const int32_t* kv_len, const int32_t* idx, int B, int Nmax, int top_k, float scale,
                                   void* out, int out_f32, float* lse, void* workspace, const PageTable& pages,
                                   cudaStream_t stream) {
    AttnQ8Params p = base_params(q, cache, cache_scale, idx, Nmax, top_k, scale, out, out_f32, lse, pages);
    p.kv_len = kv_len;
    return q4 ? launch_rows<true>(p, B, workspace, stream) : launch_rows<false>(p, B, workspace, stream);
}

}  // namespace dsa
