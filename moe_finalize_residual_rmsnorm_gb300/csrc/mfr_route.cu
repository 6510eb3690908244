// Route: a stable counting sort of the N = T * k (token, slot) pairs by expert
// id, giving the index maps of the expert-grouped layout that the dispatch,
// the finalize and their gradients read.
//
//   c_e = pairs of expert e,  p_e = c_e rounded up to `align`
//   offset_e = p_0 + ... + p_{e-1}
//   row(s) = offset_{id_s} + #{s' < s : id_s' = id_s},   slot_of[row(s)] = s
//
// A pair's rank among its expert's pairs is the sum of four counts, each in
// pair order, so the result is the stable one whatever the schedule: the
// lanes before it in its warp's round, the rounds before in its warp (a 16-bit
// counter per warp and expert in shared memory), the warps before in its CTA
// (a scan over the warps' counters), and the CTAs before.
//
// The bytes (12 a pair) are few: 262144 pairs are 3 MB, 0.5 us at the copy
// rate, so the time is latency and the counting.  Few pairs are one cluster
// of CTAs that exchange their E totals through distributed shared memory, in
// one launch; more are two launches over all SMs, the first of which counts
// each CTA's pairs and the second sums the counts before its own and writes.
// Measured on GB300: 64 pairs of 128 experts 1.9 us, 8192 pairs 3.6 us, 32768
// pairs 5.7 us, 262144 pairs of 256 experts in 128-row blocks 8.2 us (28 us in
// one cluster of 16 CTAs with warp matches), 524288 pairs of 128 experts 10.7 us,
// of 1024 experts 16.2 us, 2 M pairs of 256 experts 32 us.  These large calls
// count: every CTA sums the counts of all blocks (blocks^2 * E * 4 bytes out of
// L2), and from 4096 pairs an SM up a CTA's rounds run one after another, with a
// barrier around each scan and a thread per expert in it.
#include <cooperative_groups.h>

#include "moe_layer_ops.h"
#include "mfr_device.cuh"
#include "mfr_layer.h"

namespace cg = cooperative_groups;

namespace mfr {
namespace {

// Counters of one warp: 16 bits per expert (a CTA ranks at most 4096 pairs at
// a time).
__host__ __device__ constexpr int count_pitch(int E) { return (E + 1) / 2 * 2; }

// Dynamic shared memory: int tot[E], before[E], all[E], start[E + 1]; uint16 cnt[warps][pitch].
int route_smem(int threads, int E) { return (4 * E + 1) * 4 + threads / 32 * count_pitch(E) * 2; }

struct RouteShared {
    int* tot;       // pairs of each expert among those this CTA ranks
    int* before;    // first row of this CTA's pairs of each expert
    int* all;       // pairs of each expert in the call
    int* start;     // [E + 1] first row of each expert
    uint16_t* cnt;  // [warps][pitch]
};

__device__ __forceinline__ RouteShared route_shared(unsigned char* smem, int E) {
    RouteShared s;
    s.tot = reinterpret_cast<int*>(smem);
    s.before = s.tot + E;
    s.all = s.before + E;
    s.start = s.all + E;
    s.cnt = reinterpret_cast<uint16_t*>(s.start + E + 1);
    return s;
}

// The expert of pair s, or E: none.
__device__ __forceinline__ int expert_of(const RouteParams& p, int64_t s, bool& bad) {
    if (s >= p.N) return p.E;
    const int32_t e = p.ids[s];
    if (e >= 0 && e < p.E) return e;
    bad |= !(p.sentinel && e < 0);
    return p.E;
}

// Ranks this CTA's pairs [first, first + threads * I) within the CTA.  Thread
// order is pair order: warp w holds 32 * I consecutive pairs, lane l the pairs
// l, 32 + l, ...  On return id[i] is the pair's expert (E: none), rank[i] its
// rank within its warp, sh.cnt[warp][e] the CTA's pairs of e in earlier warps
// and sh.tot[e] the CTA's pairs of e; the CTA is synchronised.
// The lanes of a round with the same expert are found from one ballot per
// bit of the id: measured on GB300, a match instruction takes 60 cycles of
// its SM and the 9 ballots of 256 experts 30.
template <int I>
__device__ __forceinline__ void rank_pairs(const RouteParams& p, const RouteShared& sh, int64_t first, int (&id)[I],
                                           int (&rank)[I]) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int pitch = count_pitch(p.E);
    const int bits = 32 - __clz(p.E);          // ids are 0 .. E
    const int64_t s0 = first + static_cast<int64_t>(warp) * 32 * I + lane;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < I; ++i) id[i] = expert_of(p, s0 + 32 * i, bad);
    uint16_t* mine = sh.cnt + warp * pitch;
    for (int e = lane; e < pitch / 2; e += 32) reinterpret_cast<uint32_t*>(mine)[e] = 0;
    if (__any_sync(0xFFFFFFFFu, bad) && lane == 0) atomicOr(p.status, MFR_STATUS_BAD_INDEX);
    uint32_t same[I];
#pragma unroll
    for (int i = 0; i < I; ++i) same[i] = 0xFFFFFFFFu;
    for (int b = 0; b < bits; ++b) {
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const bool on = (id[i] >> b) & 1;
            const uint32_t with = __ballot_sync(0xFFFFFFFFu, on);
            same[i] &= on ? with : ~with;
        }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < I; ++i) {
        const uint32_t lower = same[i] & ((1u << lane) - 1u);
        const bool has = id[i] < p.E;
        const int base = has ? mine[id[i]] : 0;
        rank[i] = base + __popc(lower);
        __syncwarp();
        if (has && lower == 0) mine[id[i]] = static_cast<uint16_t>(base + __popc(same[i]));
        __syncwarp();
    }
    __syncthreads();
    // exclusive scan over the warps, a thread per expert, eight loads at a time
    for (int e = tid; e < p.E; e += blockDim.x) {
        int run = 0;
        for (int w0 = 0; w0 < warps; w0 += 8) {
            int v[8];
#pragma unroll
            for (int w = 0; w < 8; ++w) v[w] = w0 + w < warps ? sh.cnt[(w0 + w) * pitch + e] : 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                if (w0 + w < warps) sh.cnt[(w0 + w) * pitch + e] = static_cast<uint16_t>(run);
                run += v[w];
            }
        }
        sh.tot[e] = run;
    }
    __syncthreads();
}

// start[] from all[], a thread per expert (blockDim.x >= E); the CTA is
// synchronised on return.
__device__ __forceinline__ void scan_experts(const RouteParams& p, const RouteShared& sh) {
    __shared__ int s_warp[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    int v = 0;
    if (tid < p.E) {
        v = sh.all[tid];
        if (p.align > 1) v = (v + p.align - 1) / p.align * p.align;
    }
    int incl = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, incl, off);
        if (lane >= off) incl += o;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int base = lane < warp && lane < warps ? s_warp[lane] : 0;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) base += __shfl_xor_sync(0xFFFFFFFFu, base, off);
    if (tid < p.E) sh.start[tid] = base + incl - v;
    if (tid == p.E - 1) sh.start[p.E] = base + incl;
    __syncthreads();
}

// Marks the rows that carry no pair: the padding of each expert's block and
// the rows behind the last block.  Shared among `n` threads, this one `i`
// (both in whole warps).
__device__ __forceinline__ void mark_empty_rows(const RouteParams& p, const RouteShared& sh, int64_t i, int64_t n) {
    const int lane = static_cast<int>(i & 31);
    if (p.align > 1)
        for (int64_t e = i >> 5; e < p.E; e += n >> 5)
            for (int64_t r = sh.start[e] + sh.all[e] + lane; r < sh.start[e + 1]; r += 32) p.slot_of[r] = MFR_ROW_PADDING;
    for (int64_t r = sh.start[p.E] + i; r < p.R; r += n) p.slot_of[r] = MFR_ROW_UNUSED;
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
        const int row = e < p.E ? sh.before[e] + mine[e] + rank[i] : -1;
        p.row_of[s] = row;
        if (row >= 0) p.slot_of[row] = static_cast<int32_t>(s);
    }
}

// ---- one launch: a cluster of CTAs -----------------------------------------------
template <int I>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteParams p, const int csize) {
    extern __shared__ __align__(16) unsigned char smem[];
    const RouteShared sh = route_shared(smem, p.E);
    const int cta = static_cast<int>(blockIdx.x);   // the grid is one cluster
    const int64_t first = static_cast<int64_t>(cta) * blockDim.x * I;
    int id[I], rank[I];
    // No early trigger: the maps written here are inputs that a finalize with
    // dependent launch reads before its own wait.
    pdl_wait();
    rank_pairs<I>(p, sh, first, id, rank);
    if (csize > 1) {
        cg::cluster_group cl = cg::this_cluster();
        cl.sync();                // every CTA's totals are written
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
            int sum = 0, mine = 0;
            for (int c = 0; c < csize; ++c) {
                if (c == cta) mine = sum;
                sum += cl.map_shared_rank(sh.tot, c)[e];
            }
            sh.before[e] = mine;
            sh.all[e] = sum;
        }
        cl.barrier_arrive();      // this CTA has read the others' totals
    } else {
        for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
            sh.before[e] = 0;
            sh.all[e] = sh.tot[e];
        }
    }
    // scan_experts: thread e reads only its own all[e] before it synchronises
    scan_experts(p, sh);
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        sh.before[e] += sh.start[e];
        if (cta == 0) {
            p.counts[e] = sh.all[e];
            p.offsets[e] = sh.start[e];
        }
    }
    if (cta == 0 && threadIdx.x == 0) p.offsets[p.E] = sh.start[p.E];
    __syncthreads();
    write_maps<I>(p, sh, first, id, rank);
    mark_empty_rows(p, sh, static_cast<int64_t>(cta) * blockDim.x + threadIdx.x, static_cast<int64_t>(csize) * blockDim.x);
    if (csize > 1) cg::this_cluster().barrier_wait();   // no CTA leaves while its totals may be read
}

// ---- two launches -------------------------------------------------------------------
// CTA b's pairs are [b, b + 1) * rounds * kRouteThreads * I.
constexpr int kCountGroups = 32;

// Counts of one block in the workspace: whole groups of four.
__host__ __device__ constexpr int block_pitch(int E) { return (E + 3) / 4 * 4; }
static_assert(kMaxExperts % 4 == 0 && kMaxExperts <= kRouteThreads, "a thread per expert, four experts a load");

__global__ void __launch_bounds__(kRouteThreads) route_count_kernel(const RouteParams p, const int64_t per_cta) {
    __shared__ int s_count[kMaxExperts];
    for (int e = threadIdx.x; e < block_pitch(p.E); e += blockDim.x) s_count[e] = 0;
    pdl_wait();
    // The second launch may start: it reads the ids, which are complete, and
    // waits for this one before it reads or writes anything else.
    pdl_launch_dependents();
    __syncthreads();
    const int64_t first = blockIdx.x * per_cta;
    for (int64_t i = threadIdx.x; i < per_cta; i += blockDim.x) {
        bool bad = false;
        const int e = expert_of(p, first + i, bad);
        if (e < p.E) atomicAdd(&s_count[e], 1);      // whole numbers: any order gives the same
        if (bad) atomicOr(p.status, MFR_STATUS_BAD_INDEX);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < block_pitch(p.E); e += blockDim.x)
        p.block_counts[static_cast<int64_t>(blockIdx.x) * block_pitch(p.E) + e] = s_count[e];
}

template <int I>
__global__ void __launch_bounds__(kRouteThreads) route_write_kernel(const RouteParams p, const int rounds) {
    extern __shared__ __align__(16) unsigned char smem[];
    const RouteShared sh = route_shared(smem, p.E);
    const int tid = threadIdx.x;
    int id[I], rank[I];
    int64_t first = static_cast<int64_t>(blockIdx.x) * rounds * kRouteThreads * I;
    rank_pairs<I>(p, sh, first, id, rank);
    pdl_wait();
    // pairs of each expert in the blocks before, and in all: a thread takes
    // four experts of every `groups`-th block, eight loads at a time (at most
    // kCountGroups groups: measured for 262144 pairs of 256 experts, 4: 10.9
    // us, 8: 8.6, 16: 8.1; of 8 experts, 8: 7.0, 32: 5.9)
    const int quads = block_pitch(p.E) / 4, groups = min(static_cast<int>(blockDim.x) / quads, kCountGroups);
    const int group = tid / quads, e0 = (tid - group * quads) * 4;
    for (int e = tid; e < p.E; e += blockDim.x) sh.before[e] = sh.all[e] = 0;
    __syncthreads();
    if (group < groups) {
        int before[4] = {0, 0, 0, 0}, all[4] = {0, 0, 0, 0};
        const int blocks = static_cast<int>(gridDim.x), mine = static_cast<int>(blockIdx.x);
        for (int b0 = group; b0 < blocks; b0 += 8 * groups) {
            int4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int b = b0 + i * groups;
                v[i] = b < blocks ? *reinterpret_cast<const int4*>(p.block_counts + static_cast<int64_t>(b) * block_pitch(p.E) + e0)
                                  : make_int4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    all[q] += w[q];
                    if (b0 + i * groups < mine) before[q] += w[q];
                }
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (e0 + q < p.E) {
                atomicAdd(&sh.before[e0 + q], before[q]);
                atomicAdd(&sh.all[e0 + q], all[q]);
            }
    }
    __syncthreads();
    scan_experts(p, sh);
    for (int e = tid; e < p.E; e += blockDim.x) {
        sh.before[e] += sh.start[e];
        if (blockIdx.x == 0) {
            p.counts[e] = sh.all[e];
            p.offsets[e] = sh.start[e];
        }
    }
    if (blockIdx.x == 0 && tid == 0) p.offsets[p.E] = sh.start[p.E];
    __syncthreads();
    for (int r = 0;;) {
        write_maps<I>(p, sh, first, id, rank);
        if (++r == rounds) break;
        __syncthreads();
        for (int e = tid; e < p.E; e += blockDim.x) sh.before[e] += sh.tot[e];
        __syncthreads();
        first += kRouteThreads * I;
        rank_pairs<I>(p, sh, first, id, rank);
    }
    mark_empty_rows(p, sh, static_cast<int64_t>(blockIdx.x) * blockDim.x + tid, static_cast<int64_t>(gridDim.x) * blockDim.x);
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
    return items <= 1 ? route_kernel<1> : items <= 2 ? route_kernel<2> : route_kernel<4>;
}

RouteKernel route_write_for(int items) { return items <= 2 ? route_write_kernel<2> : route_write_kernel<4>; }

cudaError_t allow_smem(const void* f, int bytes) {
    return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

}  // namespace

int64_t route_workspace(const RouteLaunch& l, int E) { return l.cluster ? 0 : static_cast<int64_t>(l.blocks) * block_pitch(E) * 4; }

RouteLaunch route_choose(int64_t N, int64_t R, int E, int forced, int sms) {
    RouteLaunch l{};
    const int c_most = forced ? forced : 16;
    const bool one = forced < 0 ? false : forced ? N <= int64_t(forced) * kRouteThreads * kRouteMaxItems : N <= kRouteOneLaunchPairs;
    if (!one) {
        // one CTA an SM, in one round of two or four pairs a thread where that
        // is enough (524288 pairs, 128 experts: 10.7 us; 14.4 with two CTAs an SM)
        l.items = N <= int64_t(2) * kRouteThreads * sms ? 2 : 4;
        const int64_t round = int64_t(kRouteThreads) * l.items, want = (N + round - 1) / round, most = sms;
        l.rounds = static_cast<int>((want + most - 1) / most);
        l.blocks = static_cast<int>((want + l.rounds - 1) / l.rounds);
        return l;
    }
    int c = forced ? forced : 1;
    // Up to 512 pairs one CTA, then 256 a CTA; where blocks are padded, also
    // enough CTAs to mark 1024 padding rows each.  Measured, us by CTAs:
    //   512 pairs   1: 2.34   2: 2.85         1024 pairs  2: 3.23   4: 2.87
    //   8192 pairs  4: 5.5  8: 4.6  16: 3.7   32768 pairs  16: 5.7  two launches: 6.6
    //   64 pairs, 512 experts, 128-row blocks  1: 5.06   8: 4.63   16: 5.08
    while (!forced && c < c_most && ((N > 512 && N > c * int64_t(256)) || R - N > c * int64_t(1024))) c *= 2;
    // a thread per pair and per expert
    const int64_t pairs = (N + c - 1) / c;
    int64_t threads = pairs > E ? pairs : E;
    threads = threads < 128 ? 128 : threads > kRouteThreads ? kRouteThreads : (threads + 31) / 32 * 32;
    l.cluster = c;
    l.threads = static_cast<int>(threads);
    l.items = 1;
    while (int64_t(l.items) * threads * c < N) l.items *= 2;
    return l;
}

cudaError_t route_prepare(const RouteLaunch& l) {
    // the attribute is per kernel, shared by every plan: always the most any plan needs
    const int most = route_smem(kRouteThreads, kMaxExperts);
    cudaError_t e = preload(route_empty_kernel);
    if (e == cudaSuccess) e = preload(route_count_kernel);
    if (e != cudaSuccess) return e;
    if (l.cluster == 0) return allow_smem(reinterpret_cast<const void*>(route_write_for(l.items)), most);
    const void* f = reinterpret_cast<const void*>(route_kernel_for(l.items));
    e = allow_smem(f, most);
    if (e == cudaSuccess && l.cluster > 8)
        e = cudaFuncSetAttribute(f, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e;
}

bool route_resident(const RouteLaunch& l, int E) {
    if (l.cluster <= 1) return true;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(l.cluster), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(l.threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(route_smem(l.threads, E));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(l.cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, reinterpret_cast<const void*>(route_kernel_for(l.items)), &cfg) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return n >= 1;
}

cudaError_t route_launch(const RouteParams& p, const RouteLaunch& l, int pdl, cudaStream_t s) {
    if (l.cluster > 0)
        return layer_launch(route_kernel_for(l.items), l.cluster, l.threads, route_smem(l.threads, p.E), l.cluster, pdl,
                            s, p, l.cluster);
    cudaError_t e = layer_launch(route_count_kernel, l.blocks, kRouteThreads, 0, 1, pdl, s, p,
                                 static_cast<int64_t>(l.rounds) * kRouteThreads * l.items);
    if (e == cudaSuccess)
        e = layer_launch(route_write_for(l.items), l.blocks, kRouteThreads, route_smem(kRouteThreads, p.E), 1, pdl, s, p, l.rounds);
    return e;
}

cudaError_t route_empty_launch(const RouteParams& p, int pdl, cudaStream_t s) {
    return layer_launch(route_empty_kernel, 1, 256, 0, 1, pdl, s, p);
}

}  // namespace mfr
