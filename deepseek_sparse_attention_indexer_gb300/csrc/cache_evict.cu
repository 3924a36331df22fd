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
// shows.  It is a chain of latencies: three histograms, four cluster barriers.
//
// Moves: a warp a move, all tensors of the call in one launch.
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

// Sum of x over the threads before this one; total over all.
__device__ __forceinline__ int scan_block(int x, int* warp_sums, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = x;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    __syncthreads();                               // readers of the last scan are done
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    int w = warp_sums[lane];                       // kThreads / 32 = 32 warps
    int before = 0, all = 0;
#pragma unroll
    for (int o = 0; o < 32; ++o) {
        const int v = __shfl_sync(0xffffffffu, w, o);
        if (o < warp) before += v;
        all += v;
    }
    total = all;
    return before + s - x;
}

__global__ void __launch_bounds__(kThreads, 1) evict_plan_kernel(const PlanParams p) {
    extern __shared__ uint32_t keys_s[];
    __shared__ int hist[2][kBins];
    __shared__ int warp_sums[32];
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
    const int part = (n + C - 1) / C;
    const int j0 = min(n, rank * part), len = min(n, j0 + part) - j0;
    const float* acc = p.acc + (int64_t)b * p.Nmax + j0;
    const int32_t* pos = p.pos + (int64_t)b * p.Nmax + j0;

    int newest = INT32_MIN;
    if (p.recent > 0) {
        for (int i = t; i < len; i += kThreads) newest = max(newest, __ldg(pos + i));
        newest = __reduce_max_sync(0xffffffffu, newest);
        if ((t & 31) == 0) warp_sums[t >> 5] = newest;
        __syncthreads();
        if (t < 32) {
            const int m = __reduce_max_sync(0xffffffffu, warp_sums[t]);
            if (t == 0) share[0] = m;
        }
        cluster.sync();
        for (int r = 0; r < C; ++r) newest = max(newest, cluster.map_shared_rank(share, r)[0]);
    }
    const int64_t oldest_recent = (int64_t)newest - p.recent;   // positions above it are protected
    auto make = [&](int i) -> uint32_t {
        const int at = __ldg(pos + i);
        if ((p.recent > 0 && at > oldest_recent) || at < p.sink) return 0xffffffffu;
        return order_key(__ldg(acc + i));
    };
    const bool held = len <= p.smem_keys;
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
        int total;
        int before = scan_block(own[0] + own[1], warp_sums, total);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (before < want && before + own[i] >= want) {
                found[0] = kBins - 1 - (2 * t + i);
                found[1] = before;
            }
            before += own[i];
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
    int eq = 0, total;
    for (int i = r0; i < r1; ++i) eq += key(i) == prefix;
    const int eq0 = equal_before + scan_block(eq, warp_sums, total);
    auto each = [&](auto f) {
        int e = eq0;
        for (int i = r0; i < r1; ++i) {
            const uint32_t k = key(i);
            const bool stays = k > prefix || (k == prefix && e++ < want);
            f(j0 + i, stays);
        }
    };
    int gaps = 0, movers = 0;
    each([&](int j, bool stays) {
        gaps += j < p.keep && !stays;
        movers += j >= p.keep && stays;
    });
    int all_gaps, all_movers;
    int gap = scan_block(gaps, warp_sums, all_gaps), mover = scan_block(movers, warp_sums, all_movers);
    if (t == 0) {
        share[1] = all_gaps;
        share[2] = all_movers;
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

constexpr int kMoveWarps = 8;

struct MoveParams {
    const int32_t* src;
    const int32_t* dst;
    int most, Nmax, count;
    uint8_t* base[DSA_MAX_MOVED];
    int bytes[DSA_MAX_MOVED];
    int paged[DSA_MAX_MOVED];                      // 1: rows of a pool
    PageTable pages;
    int32_t* status;
};

__global__ void __launch_bounds__(kMoveWarps * 32) move_rows_kernel(const __grid_constant__ MoveParams p) {
    griddep_wait();
    const int m = blockIdx.x * kMoveWarps + threadIdx.x / 32, lane = threadIdx.x & 31;
    if (m >= p.most) return;
    const int b = blockIdx.y;
    const int from = __ldg(p.src + (int64_t)b * p.most + m), to = __ldg(p.dst + (int64_t)b * p.most + m);
    if (from < 0 || to < 0) return;
    if (from >= p.Nmax || to >= p.Nmax) {
        if (lane == 0) raise_dev_error(p.status, DEV_ERR_BOUNDS);
        return;
    }
    int64_t pf = -1, pt = -1;
    if (p.pages.table) {
        pf = paged_row(p.pages, b, from);
        pt = paged_row(p.pages, b, to);
    }
    for (int i = 0; i < p.count; ++i) {
        const int64_t f = p.paged[i] ? pf : (int64_t)b * p.Nmax + from, t = p.paged[i] ? pt : (int64_t)b * p.Nmax + to;
        if (f < 0 || t < 0) {
            if (lane == 0) raise_dev_error(p.status, DEV_ERR_BOUNDS);
            continue;
        }
        const int bytes = p.bytes[i];
        const uint8_t* s = p.base[i] + f * bytes;
        uint8_t* d = p.base[i] + t * bytes;
        if (bytes % 16 == 0 && (reinterpret_cast<uintptr_t>(p.base[i]) & 15) == 0) {
            int at = lane * 16;
            for (; at + 1024 < bytes; at += 1536) {   // three loads in flight
                uint4 v[3];
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    if (at + 512 * k < bytes) v[k] = *reinterpret_cast<const uint4*>(s + at + 512 * k);
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    if (at + 512 * k < bytes) *reinterpret_cast<uint4*>(d + at + 512 * k) = v[k];
            }
            for (; at < bytes; at += 512) *reinterpret_cast<uint4*>(d + at) = *reinterpret_cast<const uint4*>(s + at);
        } else {
            for (int at = lane * 4; at < bytes; at += 128)
                *reinterpret_cast<uint32_t*>(d + at) = *reinterpret_cast<const uint32_t*>(s + at);
        }
    }
}

}  // namespace

dsa_status_t launch_evict_plan(const float* acc, const int32_t* pos, const int32_t* kv_len, int B, int Nmax, int keep,
                               int recent, int sink, int32_t* src, int32_t* dst, int32_t* left, cudaStream_t stream) {
    PlanParams p{acc, pos, kv_len, Nmax, keep, recent, sink, keep < Nmax - keep ? keep : Nmax - keep, 0, src, dst, left};
    int cluster = 1;
    while (cluster < 8 && Nmax > 2048 * cluster) cluster *= 2;
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
    p.most = most;
    p.Nmax = Nmax;
    p.count = count;
    for (int i = 0; i < count; ++i) {
        p.base[i] = static_cast<uint8_t*>(tensors[i]);
        p.bytes[i] = row_bytes[i];
        p.paged[i] = paged[i];
    }
    p.pages = pages;
    p.status = device_status_ptr();
    if (launch_pdl(move_rows_kernel, dim3(ceil_div(most, kMoveWarps), B), dim3(kMoveWarps * 32), 0, stream, p) != cudaSuccess)
        return DSA_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace dsa
