// mla_attn_common.cuh -- what the two attention kernels (bf16 rows, 8-bit rows)
// share: the split of a launch into items of one query's selected keys, their
// assignment to persistent CTAs.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

#include "dsa_internal.h"
#include "dsa_ptx.cuh"

namespace dsa {

constexpr int kH = DSA_HEADS;          // 64
constexpr int kDv = DSA_V_DIM;         // 512
constexpr int kTile = 128;             // keys per tile (MMA M)

// The queries, their selections and the split into items.
struct AttnShape {
    const int32_t* idx;        // [rows][top_k]
    const int32_t* kv_len;     // [B] or nullptr (then every row may use Nmax keys)
    int rows;                  // queries (prefill) or sequences (decode)
    int prefill;               // 1: all rows read batch 0 of kv; 0: row r reads batch r
    int Nmax;
    int top_k;
    int nsplit, split_len;     // slots per item = split_len (multiple of 128)
    int n_items;               // rows * nsplit
};

struct Item {
    int row, split, batch, slot0, slot_end, bound;
};

__device__ __forceinline__ int nth_item(const AttnShape& p, int s) {
    int base = s * (int)gridDim.x;
    if (base >= p.n_items) return -1;
    int k = (s & 1) ? ((int)gridDim.x - 1 - (int)blockIdx.x) : (int)blockIdx.x;
    int item = base + k;
    return item < p.n_items ? item : -2;
}

// Number of 128-slot tiles up to the last non-negative index of the item's
// slot range (warp-collective; every lane gets the same answer).  A full
// selection ends with a valid index, so the last 32 slots are looked at first;
// otherwise (a query with fewer causal keys than top_k: a valid prefix, then
// -1) the range is scanned backwards 512 slots a round, 16 independent loads a
// lane, so that a short item costs a few L2 round trips rather than one per 32
// slots.
__device__ __forceinline__ int item_tiles(const AttnShape& p, const Item& I, uint32_t lane) {
    const int32_t* ir = p.idx + (int64_t)I.row * p.top_k;
    int hi = I.slot_end - 32;   // slots [hi, slot_end) first
    {
        const int s = hi + (int)lane;
        const bool v = (s >= I.slot0) && (s < I.slot_end) && (__ldg(ir + s) >= 0);
        const uint32_t m = __ballot_sync(0xffffffffu, v);
        if (m) return (hi + 31 - __clz(m) - I.slot0) / kTile + 1;
    }
    for (; hi > I.slot0; hi -= 512) {   // slots [max(slot0, hi - 512), hi)
        const int lo = hi - 512;
        int last = -1;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int s = lo + 32 * k + (int)lane;
            if (s >= I.slot0 && s < hi && __ldg(ir + s) >= 0) last = s;
        }
        last = __reduce_max_sync(0xffffffffu, last);
        if (last >= 0) return (last - I.slot0) / kTile + 1;
    }
    return 0;
}

}  // namespace dsa
