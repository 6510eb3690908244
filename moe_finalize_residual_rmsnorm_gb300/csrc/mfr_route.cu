// Route: a stable counting sort of the N = T * k (token, slot) pairs by expert
// id, giving the index maps of the expert-grouped layout that the dispatch,
// the finalize and their gradients read.
//
//   c_e = pairs of expert e,  p_e = c_e rounded up to `align`
//   offset_e = p_0 + ... + p_{e-1}
//   row(s) = offset_{id_s} + #{s' < s : id_s' = id_s},   slot_of[row(s)] = s
//
// A pair's rank among its expert's pairs is the sum of four counts, each in
// pair order, so the result is the stable one whatever the schedule, and no
// atomic is used: the lanes before it in its warp's round (a match over the
// warp), the rounds before in its warp (a 16-bit counter per warp and expert
// in shared memory), the warps before in its CTA (a scan over the warps'
// counters), and the CTAs before.
//
// The bytes (12 a pair) are few: 262144 pairs are 3 MB, 0.5 us at the copy
// rate, so the time is latency, and the one-launch form is one cluster of up
// to 16 CTAs that exchange their E totals through distributed shared memory
// instead of three launches.  Past 16384 pairs a CTA three launches count,
// scan and write.
#include <cooperative_groups.h>

#include "moe_layer_ops.h"
#include "mfr_device.cuh"
#include "mfr_layer.h"

namespace cg = cooperative_groups;

namespace mfr {
namespace {

// Counters of one warp: 16 bits per expert (a CTA holds at most 16384 pairs).
// The pitch is 2 mod 4 counters, so that the 32 warps' counters of one expert
// lie in 32 banks.
__host__ __device__ constexpr int count_pitch(int E) { return (E + 1) / 4 * 4 + 2; }

// Dynamic shared memory: int tot[E], start[E + 1], before[E]; uint16 cnt[warps][pitch].
int route_smem(int threads, int E) { return (3 * E + 1) * 4 + threads / 32 * count_pitch(E) * 2; }

struct RouteShared {
    int* tot;       // pairs of each expert in this CTA
    int* start;     // [E + 1] first row of each expert
    int* before;    // first row of this CTA's pairs of each expert
    uint16_t* cnt;  // [warps][pitch]
};

__device__ __forceinline__ RouteShared route_shared(unsigned char* smem, int E) {
    RouteShared s;
    s.tot = reinterpret_cast<int*>(smem);
    s.start = s.tot + E;
    s.before = s.start + E + 1;
    s.cnt = reinterpret_cast<uint16_t*>(s.before + E);
    return s;
}

// Ranks this CTA's pairs [first, first + threads * I) within the CTA.  Thread
// order is pair order: warp w holds 32 * I consecutive pairs, lane l the pairs
// l, 32 + l, ...  On return id[i] is the pair's expert (-1: none), rank[i] its
// rank within its warp, sh.cnt[warp][e] the CTA's pairs of e in earlier warps
// and sh.tot[e] the CTA's pairs of e; the CTA is synchronised.
template <int I>
__device__ __forceinline__ void rank_pairs(const RouteParams& p, const RouteShared& sh, int64_t first, int (&id)[I],
                                           int (&rank)[I]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int pitch = count_pitch(p.E);
    const int64_t s0 = first + static_cast<int64_t>(warp) * 32 * I + lane;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const int64_t s = s0 + 32 * i;
        id[i] = -1;
        if (s < p.N) {
            const int32_t e = p.ids[s];
            const bool ok = e >= 0 && e < p.E;
            id[i] = ok ? e : -1;
            bad |= !ok && !(p.sentinel && e < 0);
        }
    }
    uint16_t* mine = sh.cnt + warp * pitch;
    for (int e = lane; e < p.E; e += 32) mine[e] = 0;
    if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicOr(p.status, MFR_STATUS_BAD_INDEX);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, id[i]);
        const uint32_t lower = same & ((1u << lane) - 1u);
        const int base = id[i] >= 0 ? mine[id[i]] : 0;
        rank[i] = base + __popc(lower);
        __syncwarp();
        if (id[i] >= 0 && lower == 0) mine[id[i]] = static_cast<uint16_t>(base + __popc(same));
        __syncwarp();
    }
    __syncthreads();
    // exclusive scan over the warps, one expert per warp step, lane = warp
    for (int e = warp; e < p.E; e += warps) {
        const int v = lane < warps ? sh.cnt[lane * pitch + e] : 0;
        int incl = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
            if (lane >= off) incl += o;
        }
        if (lane < warps) sh.cnt[lane * pitch + e] = static_cast<uint16_t>(incl - v);
        if (lane == 31) sh.tot[e] = incl;
    }
    __syncthreads();
}

// Exclusive scan by warp 0 of the E padded totals: start[e], and start[E] the
// rows in all.  total(e) gives an expert's pairs.
template <typename Total>
__device__ __forceinline__ void scan_experts(int* start, int E, int align, Total total) {
    const int lane = threadIdx.x & 31;
    const int per = (E + 31) / 32;
    const int e0 = lane * per;
    int sum = 0;
    for (int i = 0; i < per; ++i)
        if (e0 + i < E) sum += (total(e0 + i) + align - 1) / align * align;
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
        if (lane >= off) incl += o;
    }
    int run = incl - sum;
    for (int i = 0; i < per; ++i)
        if (e0 + i < E) {
            start[e0 + i] = run;
            run += (total(e0 + i) + align - 1) / align * align;
        }
    if (lane == 31) start[E] = incl;
}

// Marks the rows that carry no pair: the padding of each expert's block and
// the rows behind the last block.  Shared among `n` threads, this one `i`
// (both in whole warps).
__device__ __forceinline__ void mark_empty_rows(int32_t* slot_of, int64_t R, int E, const int* start,
                                                const int32_t* counts, int64_t i, int64_t n) {
    const int lane = static_cast<int>(i & 31);
    for (int64_t e = i >> 5; e < E; e += n >> 5)
        for (int r = start[e] + counts[e] + lane; r < start[e + 1]; r += 32) slot_of[r] = MFR_ROW_PADDING;
    for (int64_t r = start[E] + i; r < R; r += n) slot_of[r] = MFR_ROW_UNUSED;
}

template <int I>
__device__ __forceinline__ void write_maps(const RouteParams& p, const RouteShared& sh, int64_t first,
                                           const int (&id)[I], const int (&rank)[I]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint16_t* mine = sh.cnt + warp * count_pitch(p.E);
    const int64_t s0 = first + static_cast<int64_t>(warp) * 32 * I + lane;
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const int64_t s = s0 + 32 * i;
        if (s >= p.N) continue;
        const int e = id[i];
        const int row = e >= 0 ? sh.before[e] + mine[e] + rank[i] : -1;
        p.row_of[s] = row;
        if (row >= 0) p.slot_of[row] = static_cast<int32_t>(s);
    }
}

// ---- one launch: a cluster of CTAs -----------------------------------------------
template <int I>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteParams p, const int csize) {
    extern __shared__ __align__(16) unsigned char smem[];
    const RouteShared sh = route_shared(smem, p.E);
    const int rank_in_cluster = static_cast<int>(blockIdx.x);   // the grid is one cluster
    const int64_t first = static_cast<int64_t>(blockIdx.x) * blockDim.x * I;
    int id[I], rank[I];
    // No early trigger: the maps written here are inputs that a finalize with
    // dependent launch reads before its own wait.
    pdl_wait();
    rank_pairs<I>(p, sh, first, id, rank);
    int* total = sh.tot;          // pairs of each expert in all CTAs
    if (csize > 1) {
        cg::cluster_group cl = cg::this_cluster();
        cl.sync();                // every CTA's totals are written
        total = sh.start;         // E + 1 ints; start[] is made from it below, in place
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
            int sum = 0, mine = 0;
            for (int c = 0; c < csize; ++c) {
                if (c == rank_in_cluster) mine = sum;
                sum += cl.map_shared_rank(sh.tot, c)[e];
            }
            sh.before[e] = mine;
            total[e] = sum;
        }
        cl.barrier_arrive();      // this CTA has read the others' totals
        __syncthreads();
    } else {
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) sh.before[e] = 0;
        __syncthreads();
    }
    if (rank_in_cluster == 0)
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) p.counts[e] = total[e];
    if (csize > 1) cg::this_cluster().barrier_wait();   // before tot is reused
    if (total != sh.tot) {
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) sh.tot[e] = total[e];
        __syncthreads();
    }
    if (threadIdx.x < 32) scan_experts(sh.start, p.E, p.align, [&](int e) { return sh.tot[e]; });
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) sh.before[e] += sh.start[e];
    if (rank_in_cluster == 0)
        for (int e = threadIdx.x; e <= p.E; e += blockDim.x) p.offsets[e] = sh.start[e];
    __syncthreads();
    write_maps<I>(p, sh, first, id, rank);
    mark_empty_rows(p.slot_of, p.R, p.E, sh.start, sh.tot,
                    static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x,
                    static_cast<int64_t>(csize) * blockDim.x);
}

// ---- three launches --------------------------------------------------------------
__global__ void __launch_bounds__(kRouteThreads) route_count_kernel(const RouteParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    const RouteShared sh = route_shared(smem, p.E);
    int id[kRouteMaxItems], rank[kRouteMaxItems];
    pdl_wait();
    rank_pairs<kRouteMaxItems>(p, sh, blockIdx.x * kRouteBlockPairs, id, rank);
    for (int e = threadIdx.x; e < p.E; e += blockDim.x)
        p.block_counts[static_cast<int64_t>(blockIdx.x) * p.E + e] = sh.tot[e];
}

// One CTA: block_counts[b][e] becomes the pairs of e before block b; counts and offsets.
__global__ void __launch_bounds__(kRouteThreads) route_scan_kernel(const RouteParams p, const int blocks) {
    __shared__ int s_total[kMaxExperts];
    __shared__ int s_start[kMaxExperts + 1];
    pdl_wait();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        int run = 0;
        int b = 0;
        for (; b + 8 <= blocks; b += 8) {      // eight loads in flight
            int v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = p.block_counts[static_cast<int64_t>(b + i) * p.E + e];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p.block_counts[static_cast<int64_t>(b + i) * p.E + e] = run;
                run += v[i];
            }
        }
        for (; b < blocks; ++b) {
            const int v = p.block_counts[static_cast<int64_t>(b) * p.E + e];
            p.block_counts[static_cast<int64_t>(b) * p.E + e] = run;
            run += v;
        }
        s_total[e] = run;
        p.counts[e] = run;
    }
    __syncthreads();
    if (threadIdx.x < 32) scan_experts(s_start, p.E, p.align, [&](int e) { return s_total[e]; });
    __syncthreads();
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) p.offsets[e] = s_start[e];
}

__global__ void __launch_bounds__(kRouteThreads) route_write_kernel(const RouteParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    const RouteShared sh = route_shared(smem, p.E);
    int id[kRouteMaxItems], rank[kRouteMaxItems];
    pdl_wait();
    rank_pairs<kRouteMaxItems>(p, sh, blockIdx.x * kRouteBlockPairs, id, rank);
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) sh.start[e] = p.offsets[e];
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        sh.before[e] = p.offsets[e] + p.block_counts[static_cast<int64_t>(blockIdx.x) * p.E + e];
        sh.tot[e] = p.counts[e];
    }
    __syncthreads();
    write_maps<kRouteMaxItems>(p, sh, blockIdx.x * kRouteBlockPairs, id, rank);
    mark_empty_rows(p.slot_of, p.R, p.E, sh.start, sh.tot,
                    static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x,
                    static_cast<int64_t>(gridDim.x) * blockDim.x);
}

__global__ void route_empty_kernel(const RouteParams p) {
    pdl_wait();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int64_t n = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t e = i; e <= p.E; e += n) p.offsets[e] = 0;
    for (int64_t e = i; e < p.E; e += n) p.counts[e] = 0;
}

using RouteKernel = void (*)(const RouteParams, int);
RouteKernel route_kernel_for(int items) {
    return items <= 1 ? route_kernel<1> : items <= 2 ? route_kernel<2> : items <= 4 ? route_kernel<4>
         : items <= 8 ? route_kernel<8> : route_kernel<16>;
}

cudaError_t allow_smem(const void* f, int bytes) {
    return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

}  // namespace

cudaError_t route_prepare(const RouteLaunch& l, int) {
    // the attribute is per kernel, shared by every plan: always the most any plan needs
    const int most = route_smem(kRouteThreads, kMaxExperts);
    if (l.cluster == 0) {
        cudaError_t e = allow_smem(reinterpret_cast<const void*>(route_count_kernel), most);
        return e != cudaSuccess ? e : allow_smem(reinterpret_cast<const void*>(route_write_kernel), most);
    }
    const void* f = reinterpret_cast<const void*>(route_kernel_for(l.items));
    cudaError_t e = allow_smem(f, most);
    if (e == cudaSuccess && l.cluster > 8)
        e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e;
}

cudaError_t route_launch(const RouteParams& p, const RouteLaunch& l, cudaStream_t s) {
    if (l.cluster > 0)
        return layer_launch(route_kernel_for(l.items), l.cluster, l.threads, route_smem(l.threads, p.E), l.cluster, l.pdl,
                            s, p, l.cluster);
    const int smem = route_smem(kRouteThreads, p.E);
    cudaError_t e = layer_launch(route_count_kernel, l.blocks, kRouteThreads, smem, 1, l.pdl, s, p);
    if (e == cudaSuccess) e = layer_launch(route_scan_kernel, 1, kRouteThreads, 0, 1, l.pdl, s, p, l.blocks);
    if (e == cudaSuccess) e = layer_launch(route_write_kernel, l.blocks, kRouteThreads, smem, 1, l.pdl, s, p);
    return e;
}

cudaError_t route_empty_launch(const RouteParams& p, int pdl, cudaStream_t s) {
    return layer_launch(route_empty_kernel, 1, 256, 0, 1, pdl, s, p);
}

}  // namespace mfr
