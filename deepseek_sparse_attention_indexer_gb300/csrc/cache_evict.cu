// cache_evict.cu -- which keys of each sequence stay when its cache is cut to a budget, and the moves that close the gaps.
//
// Plan: of a sequence with more than `keep` keys stay the protected ones (the `recent` latest positions, positions below
// `sink`) and the heaviest others, `keep` in all, equal weights the lower index first.  Only the keys behind the budget's
// end move: the i-th place below `keep` whose key goes is filled from the i-th key from `keep` on that stays.  Sources
// and destinations are then different rows, so all moves run at once and in place.
//
// How: a sequence is a thread-block cluster (one block for short ones), a block a contiguous part of its keys.  Weights
// are order-preserving 32-bit keys in shared memory, protected ones the largest; a radix select (11 + 11 + 10 bits,
// the blocks' histograms summed through distributed shared memory) finds the last one that stays, and two scans give each
// thread, which has a run of keys, the ranks of its equal keys, its gaps and its movers.  No sort, no atomics whose order
// shows.  It is a chain of latencies: three histograms, four cluster barriers (8 sequences of 4096 keys 12.8 us, 64 of up to
// 16k 19.5).
//
// Moves: all tensors of the call in one launch of as many warps as the SMs hold.  The rows lie apart in HBM, so it is bytes
// in flight that count: 32 entries' indices and pages are looked up at once, a lane each, and a lane loads its pieces of two
// moves, all tensors, before it stores the first.  Most entries lie behind a sequence's last move, and sequences have few
// or many, so a warp takes entries from all over.  79,491 moves of 1416 bytes in 64 sequences' 524,288 entries 43 us (225 MB,
// 5.2 TB/s; a run of eight entries a warp 53, an entry a warp 99), 8175 in 8 sequences' 16,384 4.8 us (a warp an entry 7.6);
// four blocks an SM, which spill, 44 and 5.0, two with four moves in flight 45 and 4.7.
#include <cooperative_groups.h>

#include <atomic>
#include <cstdint>

#include "dsa_q8.cuh"

namespace cg = cooperative_groups;

namespace dsa {

namespace {

constexpr int kThreads = 1024;
constexpr int kBins = 2048;
constexpr int kKeysInSmem = 48 * 1024;             // keys of a block held in shared memory; longer parts are read again

struct PlanParams {
    const float* acc;
    const int32_t* pos;
    const int32_t* kv_len;
    int Nmax, keep, recent, sink, most;            // most: moves a sequence can have
    int smem_keys;
    int32_t* src;
    int32_t* dst;
    int32_t* left;
};

// Keys that compare as the weights do: -0 as 0, NaN below all others.
__device__ __forceinline__ uint32_t order_key(float w) {
    const uint32_t b = __float_as_uint(w + 0.f);
    if ((b & 0x7fffffffu) > 0x7f800000u) return 0;
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ int padded(int i) { return i + (i >> 5); }   // runs of a power of two start in different banks

// Sums of x and y over the threads before this one, in their place; the totals over all.
__device__ __forceinline__ int2 scan_block(int2& x, int2* warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto scan_warp = [&](int2 v) {
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int a = __shfl_up_sync(0xffffffffu, v.x, o), b = __shfl_up_sync(0xffffffffu, v.y, o);
            if (lane >= o) v = make_int2(v.x + a, v.y + b);
        }
        return v;
    };
    const int2 own = scan_warp(x);
    __syncthreads();                               // readers of the last scan are done
    if (lane == 31) warp_sums[warp] = own;
    __syncthreads();
    const int2 w = scan_warp(warp_sums[lane]);     // of kThreads / 32 = 32 warps
    const int before = max(warp - 1, 0);
    const int bx = __shfl_sync(0xffffffffu, w.x, before), by = __shfl_sync(0xffffffffu, w.y, before);
    x = make_int2(own.x - x.x + (warp ? bx : 0), own.y - x.y + (warp ? by : 0));
    return make_int2(__shfl_sync(0xffffffffu, w.x, 31), __shfl_sync(0xffffffffu, w.y, 31));
}

__global__ void __launch_bounds__(kThreads, 1) evict_plan_kernel(const PlanParams p) {
    extern __shared__ uint32_t keys_s[];
    __shared__ int hist[2][kBins];
    __shared__ int2 warp_sums[32];
    __shared__ int share[4];                       // read by the other blocks: largest position, gaps, movers
    __shared__ int found[2];                       // bin, keys of larger digits
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int b = blockIdx.x / C, t = threadIdx.x;
    griddep_wait();
    const int n = min(__ldg(p.kv_len + b), p.Nmax);
    int32_t* src = p.src + (int64_t)b * p.most;
    int32_t* dst = p.dst + (int64_t)b * p.most;
    if (n <= p.keep) {                             // the same for the whole cluster
        for (int i = rank * kThreads + t; i < p.most; i += C * kThreads) src[i] = dst[i] = -1;
        if (rank == 0 && t == 0) p.left[b] = max(n, 0);
        return;
    }
    const int part = (n - 1) / C + 1;              // n > keep >= 1, up to 2^31 - 1
    const int j0 = (int)min((int64_t)n, (int64_t)rank * part), len = min(part, n - j0);
    const float* acc = p.acc + (int64_t)b * p.Nmax + j0;
    const int32_t* pos = p.pos + (int64_t)b * p.Nmax + j0;

    // Largest position; the weights' keys beside it where they are held.
    const bool held = len <= p.smem_keys;
    int newest = INT32_MIN;
    for (int i = t; i < len; i += kThreads) {
        if (held) keys_s[padded(i)] = order_key(__ldg(acc + i));
        newest = max(newest, __ldg(pos + i));
    }
    if (p.recent > 0) {
        newest = __reduce_max_sync(0xffffffffu, newest);
        if ((t & 31) == 0) warp_sums[t >> 5].x = newest;
        __syncthreads();
        if (t < 32) {
            const int m = __reduce_max_sync(0xffffffffu, warp_sums[t].x);
            if (t == 0) share[0] = m;
        }
        cluster.sync();
        for (int r = 0; r < C; ++r) newest = max(newest, cluster.map_shared_rank(share, r)[0]);
    }
    const int64_t oldest_recent = (int64_t)newest - p.recent;   // positions above it are protected
    auto make = [&](int i) -> uint32_t {           // a thread's own keys, as it wrote them
        const int at = __ldg(pos + i);
        if ((p.recent > 0 && at > oldest_recent) || at < p.sink) return 0xffffffffu;
        return held ? keys_s[padded(i)] : order_key(__ldg(acc + i));
    };
    auto key = [&](int i) -> uint32_t { return held ? keys_s[padded(i)] : make(i); };

    // Radix select: `prefix` the digits found so far, `want` how many of the keys that share them stay.
    uint32_t prefix = 0;
    int want = p.keep, equal_before = 0;
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        int* h = hist[pass & 1];                   // the other one is still read by the blocks of the pass before
        for (int i = t; i < kBins; i += kThreads) h[i] = 0;
        __syncthreads();
        for (int i = t; i < len; i += kThreads) {
            uint32_t k;
            if (pass == 0) {
                k = make(i);
                if (held) keys_s[padded(i)] = k;
            } else {
                k = key(i);
                if ((k >> (shift + bits)) != prefix) continue;
            }
            atomicAdd(&h[(k >> shift) & ((1u << bits) - 1)], 1);
        }
        cluster.sync();
        // bins from the largest on, two a thread: sums over the cluster
        int own[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int bin = kBins - 1 - (2 * t + i);
            own[i] = 0;
            for (int r = 0; r < C; ++r) own[i] += cluster.map_shared_rank(h, r)[bin];
        }
        int2 before = make_int2(own[0] + own[1], 0);
        scan_block(before, warp_sums);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (before.x < want && before.x + own[i] >= want) {
                found[0] = kBins - 1 - (2 * t + i);
                found[1] = before.x;
            }
            before.x += own[i];
        }
        __syncthreads();
        const int bin = found[0];
        want -= found[1];
        prefix = prefix << bits | (uint32_t)bin;
        if (pass == 2)                             // keys equal to the last that stays, in the blocks before
            for (int r = 0; r < rank; ++r) equal_before += cluster.map_shared_rank(h, r)[bin];
    }

    // A run of keys a thread: ranks of the equal ones, then what goes below `keep` and what stays behind it.
    const int run = (len + kThreads - 1) / kThreads, r0 = min(len, t * run), r1 = min(len, r0 + run);
    int2 eq = make_int2(0, 0);
    for (int i = r0; i < r1; ++i) eq.x += key(i) == prefix;
    scan_block(eq, warp_sums);
    const int eq0 = equal_before + eq.x;
    auto each = [&](auto f) {
        int e = eq0;
        for (int i = r0; i < r1; ++i) {
            const uint32_t k = key(i);
            const bool stays = k > prefix || (k == prefix && e++ < want);
            f(j0 + i, stays);
        }
    };
    int2 own = make_int2(0, 0);                    // gaps, movers
    each([&](int j, bool stays) {
        own.x += j < p.keep && !stays;
        own.y += j >= p.keep && stays;
    });
    const int2 all = scan_block(own, warp_sums);
    int gap = own.x, mover = own.y;
    if (t == 0) {
        share[1] = all.x;
        share[2] = all.y;
    }
    cluster.sync();
    int count = 0;
    for (int r = 0; r < C; ++r) {
        const int* s = cluster.map_shared_rank(share, r);
        if (r < rank) {
            gap += s[1];
            mover += s[2];
        }
        count += s[2];
    }
    each([&](int j, bool stays) {
        if (j < p.keep && !stays) dst[gap++] = j;
        if (j >= p.keep && stays) src[mover++] = j;
    });
    for (int i = count + rank * kThreads + t; i < p.most; i += C * kThreads) src[i] = dst[i] = -1;
    if (rank == 0 && t == 0) p.left[b] = p.keep;
    cluster.sync();                                // no block leaves while its shared memory is read
}

constexpr int kMoveWarps = 8, kMoveBlocks = 3;     // warps a block, blocks an SM
constexpr int kAhead = 3;                          // pieces of 16 bytes of a move that a lane loads before it stores

struct MoveParams {
    const int32_t* src;
    const int32_t* dst;
    int B, most, Nmax, count;
    uint8_t* base[DSA_MAX_MOVED];                  // tensors of 16-byte pieces first
    int bytes[DSA_MAX_MOVED];
    int paged[DSA_MAX_MOVED];                      // 1: rows of a pool
    int wide;                                      // tensors whose rows are whole 16-byte pieces
    int pieces, words;                             // of a row of all those; 4-byte words of a row of the others
    PageTable pages;
    int32_t* status;
};

// Piece (or word) u of a move: its tensor and the offset in the row, bytes of `size`; false behind the last.
__device__ __forceinline__ bool find_piece(const MoveParams& p, int u, int first, int last, int size, int& tensor, int& at) {
    for (int i = first; i < last; ++i) {
        const int n = p.bytes[i] / size;
        if (u < n) {
            tensor = i;
            at = u * size;
            return true;
        }
        u -= n;
    }
    return false;
}

__global__ void __launch_bounds__(kMoveWarps * 32, kMoveBlocks) move_rows_kernel(const __grid_constant__ MoveParams p) {
    const int lane = threadIdx.x & 31;
    griddep_wait();
    // The lane's pieces, the same of every move: where they lie in row 0 of their tensors, the tensors' bytes a row.
    uint8_t* at[kAhead + 1];
    int bytes[kAhead + 1];
    bool paged[kAhead + 1];
#pragma unroll
    for (int k = 0; k <= kAhead; ++k) {
        int i, o;
        const bool mine = k < kAhead ? find_piece(p, lane + 32 * k, 0, p.wide, 16, i, o) : find_piece(p, lane, p.wide, p.count, 4, i, o);
        at[k] = mine ? p.base[i] + o : nullptr;
        bytes[k] = mine ? p.bytes[i] : 0;
        paged[k] = mine && p.paged[i];
    }
    struct Move {                                  // rows of the dense tensors and of the pools; from[0] -1: left out
        int from[2], to[2];
    };
    auto from = [](const Move& v, bool paged) { return paged ? v.from[1] : v.from[0]; };
    auto to = [](const Move& v, bool paged) { return paged ? v.to[1] : v.to[0]; };
    // Entry e is the (e / B)-th of a sequence; a warp's are as many apart as there are warps, 32 looked up at a time.  The
    // sequences in turn, one further at each place, so that a warp meets all of them whatever the number of warps.
    const uint32_t warps = gridDim.x * kMoveWarps, B = p.B, entries = B * p.most;   // entries < 2^31
    for (uint32_t e0 = blockIdx.x * kMoveWarps + threadIdx.x / 32; e0 < entries; e0 += 32 * warps) {
        const uint32_t e = e0 + lane * warps;
        Move own{{-1, -1}, {-1, -1}};
        if (e < entries) {
            const uint32_t m = e / B;
            const int b = (int)((e + m) % B);
            const int from = __ldg(p.src + (int64_t)b * p.most + m), to = __ldg(p.dst + (int64_t)b * p.most + m);
            bool bad = false;
            if (from >= 0 && to >= 0 && !(bad = from >= p.Nmax || to >= p.Nmax)) {
                own.from[0] = b * p.Nmax + from;   // below 2^31, as the rows of a pool
                own.to[0] = b * p.Nmax + to;
                if (p.pages.table) {
                    own.from[1] = (int)paged_row(p.pages, b, from);
                    own.to[1] = (int)paged_row(p.pages, b, to);
                    bad = own.from[1] < 0 || own.to[1] < 0;
                    if (bad) own.from[0] = -1;     // in no tensor, so that a key's rows stay together
                }
            }
            if (bad) raise_dev_error(p.status, DEV_ERR_BOUNDS);
        }
        uint32_t left = __ballot_sync(0xffffffffu, own.from[0] >= 0);
        while (left) {
            Move mv[2];
            uint4 v[2][kAhead];
            uint32_t w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int l = left ? __ffs(left) - 1 : 0;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int f = __shfl_sync(0xffffffffu, own.from[j], l);
                    mv[i].from[j] = left ? f : -1;
                    mv[i].to[j] = __shfl_sync(0xffffffffu, own.to[j], l);
                }
                left &= left - 1;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (at[k] && from(mv[i], paged[k]) >= 0)
                        v[i][k] = *reinterpret_cast<const uint4*>(at[k] + (int64_t)from(mv[i], paged[k]) * bytes[k]);
                if (at[kAhead] && from(mv[i], paged[kAhead]) >= 0)
                    w[i] = *reinterpret_cast<const uint32_t*>(at[kAhead] + (int64_t)from(mv[i], paged[kAhead]) * bytes[kAhead]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (at[k] && from(mv[i], paged[k]) >= 0)
                        *reinterpret_cast<uint4*>(at[k] + (int64_t)to(mv[i], paged[k]) * bytes[k]) = v[i][k];
                if (at[kAhead] && from(mv[i], paged[kAhead]) >= 0)
                    *reinterpret_cast<uint32_t*>(at[kAhead] + (int64_t)to(mv[i], paged[kAhead]) * bytes[kAhead]) = w[i];
                for (int u = lane + 32 * kAhead; u < p.pieces; u += 32) {   // longer rows
                    int j, o;
                    if (!find_piece(p, u, 0, p.wide, 16, j, o) || from(mv[i], p.paged[j]) < 0) continue;
                    *reinterpret_cast<uint4*>(p.base[j] + (int64_t)to(mv[i], p.paged[j]) * p.bytes[j] + o) =
                        *reinterpret_cast<const uint4*>(p.base[j] + (int64_t)from(mv[i], p.paged[j]) * p.bytes[j] + o);
                }
                for (int u = lane + 32; u < p.words; u += 32) {
                    int j, o;
                    if (!find_piece(p, u, p.wide, p.count, 4, j, o) || from(mv[i], p.paged[j]) < 0) continue;
                    *reinterpret_cast<uint32_t*>(p.base[j] + (int64_t)to(mv[i], p.paged[j]) * p.bytes[j] + o) =
                        *reinterpret_cast<const uint32_t*>(p.base[j] + (int64_t)from(mv[i], p.paged[j]) * p.bytes[j] + o);
                }
            }
        }
    }
}

}  // namespace

dsa_status_t launch_evict_plan(const float* acc, const int32_t* pos, const int32_t* kv_len, int B, int Nmax, int keep,
                               int recent, int sink, int32_t* src, int32_t* dst, int32_t* left, cudaStream_t stream) {
    PlanParams p{acc, pos, kv_len, Nmax, keep, recent, sink, keep < Nmax - keep ? keep : Nmax - keep, 0, src, dst, left};
    // Blocks a sequence: one for 4096 keys, two for 8192, four for 32k, eight beyond (a sequence of 4k / 8k / 16k / 32k / 64k
    // keys, us: 1 block 13.1 / 16.9 / 25.6 / 42.3 / -, 2 13.1 / 14.7 / 18.6 / 27.2 / 44.3, 4 14.5 / 15.8 / 17.3 / 21.2 / 30.1, 8
    // 21.2 / 21.7 / 23.0 / 24.7 / 28.6), but no more than one block an SM at once (64 sequences of 16k: 1 block 26, 2 18.8, 4
    // 36, 8 118), and enough that a part fits shared memory (one of 64k in one block 305).
    const int sms = device_sm_count();
    int cluster = Nmax <= 4096 ? 1 : Nmax <= 8192 ? 2 : Nmax <= 32768 ? 4 : 8;
    while (cluster > 1 && (long long)B * cluster * 9 > sms * 8) cluster /= 2;   // (clusters leave some SMs)
    while (cluster < 8 && ceil_div(Nmax, cluster) >= kKeysInSmem) cluster *= 2;
    const int part = ceil_div(Nmax, cluster);
    p.smem_keys = part < kKeysInSmem ? part : 0;
    const int smem = p.smem_keys ? (p.smem_keys + p.smem_keys / 32 + 1) * 4 : 0;
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> done[kMaxDevices];
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return DSA_ERR_CUDA;
    if (!done[dev].load(std::memory_order_acquire)) {
        const dsa_status_t st = ensure_smem_attr(reinterpret_cast<const void*>(evict_plan_kernel),
                                                 (kKeysInSmem + kKeysInSmem / 32 + 1) * 4);
        if (st != DSA_OK) return st;
        done[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(B * cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, evict_plan_kernel, p) != cudaSuccess) return DSA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

dsa_status_t launch_move_rows(const int32_t* src, const int32_t* dst, int B, int most, int Nmax, int count,
                              void* const* tensors, const int* row_bytes, const int* paged, const PageTable& pages,
                              cudaStream_t stream) {
    MoveParams p{};
    p.src = src;
    p.dst = dst;
    p.B = B;
    p.most = most;
    p.Nmax = Nmax;
    for (int pass = 0; pass < 2; ++pass) {         // the tensors of whole 16-byte pieces, then the others
        for (int i = 0; i < count; ++i) {
            const bool wide = row_bytes[i] % 16 == 0 && aligned16(tensors[i]);
            if (wide != (pass == 0)) continue;
            const int at = p.count++;
            p.base[at] = static_cast<uint8_t*>(tensors[i]);
            p.bytes[at] = row_bytes[i];
            p.paged[at] = paged[i];
            (wide ? p.pieces : p.words) += row_bytes[i] / (wide ? 16 : 4);
            if (wide) p.wide = p.count;
        }
    }
    p.pages = pages;
    p.status = device_status_ptr();
    const int blocks = kMoveBlocks * device_sm_count(), need = (int)(((long long)B * most + kMoveWarps - 1) / kMoveWarps);
    if (launch_pdl(move_rows_kernel, dim3(need < blocks ? need : blocks), dim3(kMoveWarps * 32), 0, stream, p) != cudaSuccess)
        return DSA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
