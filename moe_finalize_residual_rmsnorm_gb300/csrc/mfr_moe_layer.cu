// A whole MoE layer for a few tokens:
//
//   h[t, j] = silu(G_e x[t]) * (U_e x[t]),   e = expert of token t's slot j
//   out[t]  = sum_j w[t, j] * (D_e h[t, j])
//
// with the rows of G_e and U_e stacked in w13[e] [2 I, H] and D_e in w2[e] [H, I],
// in bf16, or in E4M3 with FP32 scales (a scale per 128 x 128 weights and per 128
// columns of x and h; h is quantised per 128 columns as moe_residual_rmsnorm does).
//
// Every chosen expert's weights are read once, and up to about a hundred pairs an
// expert those bytes bound the layer, so the weights are the streamed operand:
// they are the 128 rows of the product's A, and the expert's pairs its 16 .. 128
// columns (B).  One warp keeps a ring of stages of 32 KB of weights filled by
// tensor-map copies, one loads the pairs' rows next to them (x by gathers of four; h,
// which the first launch leaves in the sorted order, 16 a copy), one thread issues tcgen05
// products into tensor memory, and eight warps finish one unit while the next one is
// multiplied.
//
// Each CTA sorts the pairs by expert itself (at most 4096, from L2), so that no
// launch before it is needed; up to 32 of them are one warp's, which asks for its first
// weights before the others are ready (5 tokens of 384 x 368: 11.7 -> 10.9 us).  A unit is
// (tile of weight rows, chunk of an expert's pairs) over all of K, in turns over persistent
// CTAs; chunks of one expert are neighbours, so that its weights come from DRAM once.
//   first launch:  64 rows of G and the same 64 of U (E4M3: 128 and 128, a group of
//                  h's scales), h to the workspace
//   second launch: 256 rows of D, products to y[pair] in FP32; it loads weights
//                  before it waits for the first launch
//   then the pairs of every token are added in slot order, by a small third launch:
//                  no atomics, the same bits in every call
// bf16 calls with many pairs an expert have a launch before these, which copies their rows
// of x in the sorted order.  Where units are few and long, the CTAs of a cluster take a part of K each.
// Measured on GB300 (4096 x 1024 weights an expert, bf16, copy rate 6782 GB/s): 16 tokens
// of 128 experts 293 to 320 us (78 to 82 of them chosen; 0.95 to 1.0 of the copy rate), 64 of
// 64 experts 247 us (0.96), one token of 64 experts 38.5 us (0.77: two launches' starts, sorts
// and first loads, 8 us); 128 tokens of 64 experts of 8192 x 1024 in E4M3 270 us (0.88: 512
// units are 3.4 turns of the SMs).  With units for few SMs one SM takes 60-70 GB/s: a stage's eight products are
// 330 cycles whatever their columns (the weights are read from shared memory for each), and
// hand-overs 200 more.
// Not taken: dividing the steps along K evenly over the CTAs, with partial sums put
// together by the last to arrive (every piece's end is a fence, an atomic and a round
// trip: one token 54 us that way and 42 this, 37 tokens 85 and 51, 128 in E4M3 378 and
// 289); adding the pairs in the second launch by the last CTA of a tile (128 tokens: 50
// us at its end); two CTAs an SM, so that the launches overlap (half the ring each: one
// token 52 us); fetching w2 to L2 at the first launch's end (no difference) or further
// ahead of the ring while waiting for it (8 to 64 stages: 2 to 4 % slower); units of 32
// or 64 columns of h and 128 rows of D, in E4M3 with clusters that share a group's
// largest magnitude (25 shapes 5 % slower: more copies, and in E4M3 more steps, a byte);
// clusters of two for every call, which divide the last, partial turn (3 % slower); units
// of three or two quarters of the rows where they fill that turn better (2 % faster
// for 37 tokens, calls of a few tokens 1 us slower).
//
// bf16: h is kept as the sum of two bf16 values (16 bits of it), two products of the
// same weights, which cost nothing where bytes bound it; rounded once it alone would
// put the output 1.4 times as far from the exact one as its own rounding does.  So held
// the output is as far from it as with all 24 bits (0.00166 of its rms), and one in 200
// is the neighbouring bf16 value of the one that 24 bits give.
// E4M3: products of 128 columns of K are one accumulation in tensor memory, which
// the finishing warps scale and add in FP32 registers.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <mutex>

#include "moe_step_ops.h"
#include "mfr_layer.h"
#include "mfr_step.h"
#include "mfr_tcgen05.cuh"

namespace mfr {
namespace {

constexpr int kWarps = kMoeThreads / 32;
constexpr int kFinishWarps = 8;
constexpr int kPanel = kMoeRows * 128;             // 128 weight rows of 128 bytes of K; a stage has two
constexpr int kRingStages = 6;
constexpr float kAmaxFloor = 0x1p-100f;
constexpr float kBf16Max = 0x1.FEp127f;            // the largest finite bf16 value

// Rows of pairs in a stage.  bf16: two panels, of the two steps of K in a stage of the
// first launch, or of the two parts of h in the second.
template <bool FP8, int NB>
constexpr int stage_bytes() { return 2 * kPanel + NB * 128 * (FP8 ? 1 : 2); }

// Accumulators of a unit: gate and up rows in one (bf16), or two of 128 rows.
template <bool FP8, bool DOWN>
constexpr int accumulators() { return FP8 || DOWN ? 2 : 1; }

// The two parts of h are columns of one product, side by side, where tensor memory
// holds that twice; else two products.
template <bool FP8, bool DOWN, int NB>
constexpr bool stacked() { return DOWN && !FP8 && NB <= 64; }

// Accumulators in turn: two units', in E4M3 four steps' (128 tokens of 64 experts 287 ->
// 278 us).
constexpr int kMaxTurns = 4;
template <bool FP8, int NB>
constexpr int turns() { return FP8 ? 4 : 2; }

// Columns of an accumulator, and of all.
template <bool FP8, bool DOWN, int NB>
constexpr int columns() { return stacked<FP8, DOWN, NB>() ? 2 * NB : NB; }
template <bool FP8, bool DOWN, int NB>
constexpr uint32_t tmem_columns() {
    constexpr int n = turns<FP8, NB>() * accumulators<FP8, DOWN>() * columns<FP8, DOWN, NB>();
    return n < 32 ? 32 : n;
}

// Behind the ring.
template <bool FP8, int NB>
struct Shared {
    uint64_t full[kRingStages], empty[kRingStages];
    uint64_t done[kMaxTurns], taken[kMaxTurns];       // an accumulator is complete; its values are in registers
    uint64_t drain;
    uint64_t parts[kFinishWarps];     // the other parts' sums of this warp's values are in the workspace
    uint32_t tmem;
    int dead;                         // a wait ran out: every role leaves
    int issued[2];                    // stages that the loading warps have begun
    int scan[kWarps];
    union {
        struct {                      // E4M3
            alignas(16) float sx[kFinishWarps][2][NB / 2];   // factors of a warp's columns, for both accumulators
            uint32_t top[2][4][NB / 2];       // largest magnitudes, by side, warp and column
        };
        // bf16: products that gate and up rows' lanes exchange, by side, turn and column;
        // two turns, so that one barrier does, where there are several
        float other[2][!FP8 && NB > 16 ? 2 : 1][8][FP8 ? 1 : 64];
    };
};

__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ void shared_proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void group_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" :: "r"(id), "r"(threads) : "memory");
}

// Whether all of the finishing warps are well: they leave together, or none does.
__device__ __forceinline__ bool finishers_well(bool ok) {
    uint32_t all;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 4, %2, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(all) : "r"(static_cast<uint32_t>(ok)), "n"(32 * kFinishWarps) : "memory");
    return all != 0;
}

// A role's wait for another.  It gives up after p.wait_limit cycles (0: at once, whatever
// there is), or when another has given up.
template <bool CLUSTER = false>
__device__ bool role_wait(int* dead_word, const MoeParams& p, uint32_t bar, uint32_t parity) {
    auto test = [&] { return CLUSTER ? mbar_test_cluster(bar, parity) : mbar_test_parity(bar, parity); };
    if (p.wait_limit > 0 && test()) return true;
    volatile int* dead = dead_word;
    const long long t0 = clock64();
    while (p.wait_limit == 0 || !test()) {
        if (*dead) return false;
        if (clock64() - t0 >= p.wait_limit) {
            *dead = 1;
            atomicOr(p.status, MFR_STATUS_TIMEOUT);
            return false;
        }
    }
    return true;
}

// A chunk of an expert's pairs: (expert, first place in the sorted list, pairs).
struct Entry {
    int expert, start, n;
};
__device__ __forceinline__ uint32_t pack_entry(int expert, int start, int n) {
    return static_cast<uint32_t>(expert) | (static_cast<uint32_t>(start) << 10) | (static_cast<uint32_t>(n - 1) << 22);
}
__device__ __forceinline__ Entry unpack_entry(uint32_t v) {
    return {static_cast<int>(v & 1023u), static_cast<int>((v >> 10) & 4095u), static_cast<int>(v >> 22) + 1};
}

__device__ __forceinline__ bool valid_expert(int id, int E) { return static_cast<uint32_t>(id) < static_cast<uint32_t>(E); }

// Stable counting sort of the pairs by expert, the same in every CTA: `list` gets
// the pairs, `entries` the chunks of at most NB of them; returns their number.
// `hist`: [kWarps + 1][E], and behind it the pairs' ids and their places among their
// warp's pairs of the same expert.  All threads call it.
template <bool FP8, int NB>
__device__ int sort_pairs(const MoeParams& p, Shared<FP8, NB>* s, uint16_t* list, uint32_t* entries, int* hist, bool report) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = p.T * p.k, E = p.E;
    const int seg = ((P + kWarps - 1) / kWarps + 31) & ~31, first = warp * seg, last = min(P, first + seg);
    const int warps = (P + seg - 1) / seg;            // that have pairs
    int* ids = hist + (kWarps + 1) * E;
    uint16_t* place = reinterpret_cast<uint16_t*>(ids + P);
    for (int i = tid; i < P; i += kMoeThreads) ids[i] = __ldg(p.ids + i);
    for (int i = tid; i < warps * E; i += kMoeThreads) hist[i] = 0;
    __syncthreads();
    bool bad = false;
    for (int i0 = first; i0 < last; i0 += 32) {
        const int i = i0 + lane, e = i < last ? ids[i] : -1;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
        const bool ok = valid_expert(e, E);
        if (ok) place[i] = static_cast<uint16_t>(hist[warp * E + e] + __popc(same & ((1u << lane) - 1)));
        else bad |= i < last && !(p.sentinel && e < 0);
        __syncwarp();
        if (ok && lane == __ffs(same) - 1) hist[warp * E + e] += __popc(same);
        __syncwarp();
    }
    if (report && bad) atomicOr(p.status, MFR_STATUS_BAD_INDEX);
    __syncthreads();
    // each thread: a run of experts; pairs in the low half, chunks in the high half
    const int per = (E + kMoeThreads - 1) / kMoeThreads, e0 = min(E, tid * per), e1 = min(E, e0 + per);
    uint32_t sum = 0;
    for (int e = e0; e < e1; ++e) {
        int n = 0;
        for (int w = 0; w < warps; ++w) {
            const int c = hist[w * E + e];
            hist[w * E + e] = n;
            n += c;
        }
        hist[kWarps * E + e] = n;
        sum += static_cast<uint32_t>(n) + (static_cast<uint32_t>((n + NB - 1) / NB) << 16);
    }
    uint32_t incl = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, off);
        if (lane >= off) incl += v;
    }
    if (lane == 31) s->scan[warp] = static_cast<int>(incl);
    __syncthreads();
    uint32_t base = incl - sum, all = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) base += static_cast<uint32_t>(s->scan[w]);
        all += static_cast<uint32_t>(s->scan[w]);
    }
    int at = static_cast<int>(base & 0xFFFFu), chunk = static_cast<int>(base >> 16);
    for (int e = e0; e < e1; ++e) {
        const int n = hist[kWarps * E + e];
        if (n == 0) continue;
        for (int w = 0; w < warps; ++w) hist[w * E + e] += at;
        for (int c = 0; c < n; c += NB) entries[chunk++] = pack_entry(e, at + c, min(NB, n - c));
        at += n;
    }
    __syncthreads();
    for (int i = first + lane; i < last; i += 32)
        if (valid_expert(ids[i], E)) list[hist[warp * E + ids[i]] + place[i]] = static_cast<uint16_t>(i);
    return static_cast<int>(all >> 16);               // the caller's barrier ends it
}

// The same for at most 32 pairs by one warp, which needs no other.
template <int NB>
__device__ __forceinline__ int sort_few(const MoeParams& p, uint16_t* list, uint32_t* entries, bool report) {
    const int lane = threadIdx.x & 31, P = p.T * p.k;
    const int id = lane < P ? __ldg(p.ids + lane) : -1;
    const bool ok = valid_expert(id, p.E);
    if (report && lane < P && !ok && !(p.sentinel && id < 0)) atomicOr(p.status, MFR_STATUS_BAD_INDEX);
    const int key = ok ? id : kMaxExperts;            // pairs without an expert come last
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, key);
    const int before = __popc(same & ((1u << lane) - 1)), total = __popc(same);
    const bool leads = ok && before % NB == 0;        // a chunk
    const uint32_t leaders = __ballot_sync(0xFFFFFFFFu, leads);
    int rank = 0, chunk = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const int other = __shfl_sync(0xFFFFFFFFu, key, j);
        const bool first = other < key || (other == key && j < lane);
        rank += first;
        chunk += first && (leaders >> j & 1u);
    }
    if (ok) list[rank] = static_cast<uint16_t>(lane);
    if (leads) entries[chunk] = pack_entry(id, rank, min(NB, total - before));
    __syncwarp();
    return __popc(leaders);
}

// __expf is off by 2 + 1.2 |g| units of 2^-23 at most, which nothing after it shows: h is held to
// 2^-16, in E4M3 to 2^-4.
__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.f + __expf(-g)) * u; }

// bf16 with many pairs an expert: their rows of x are put in the sorted order by a launch
// of their own, because gathers of four rows take 23 ns each, 128 rows of a stage 1.5 us
// (256 tokens of 16 experts of 4096 x 1024: 269 us with gathers and 140 so, of 8 of 1024 x
// 1024: 63 and 41; with 64 columns between 5 % faster and 4 % slower, and slower in E4M3,
// whose stages take half the gathers).
constexpr bool copied(bool fp8, int columns) { return !fp8 && columns == 128; }

__global__ void __launch_bounds__(kMoeThreads, 1) moe_rows_kernel(const MoeParams p, const uint8_t* x) {
    extern __shared__ __align__(16) unsigned char raw[];
    Shared<false, 128>* s = reinterpret_cast<Shared<false, 128>*>(raw);
    uint32_t* entries = reinterpret_cast<uint32_t*>(raw + sizeof(Shared<false, 128>));
    int* hist = reinterpret_cast<int*>(entries + p.entries);
    uint16_t* list = reinterpret_cast<uint16_t*>(hist + (kWarps + 1) * p.E) + 3 * p.T * p.k;       // behind the ids and places
    pdl_wait();
    pdl_launch_dependents();
    const int M = sort_pairs<false, 128>(p, s, list, entries, hist, false);
    __syncthreads();
    if (M == 0) return;
    const Entry last = unpack_entry(entries[M - 1]);
    const int lane = threadIdx.x & 31, pairs = last.start + last.n, bytes = p.H * 2;
    for (int i = blockIdx.x * kWarps + (threadIdx.x >> 5); i < pairs; i += gridDim.x * kWarps) {
        const uint8_t* from = x + static_cast<int64_t>(list[i] / p.k) * bytes;
        uint8_t* to = p.rows + static_cast<int64_t>(i) * bytes;
        for (int b = lane * 16; b < bytes; b += 4 * 512) {
            uint4 v[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) v[n] = ld_stream_u4_if(from + b + n * 512, b + n * 512 < bytes);
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (b + n * 512 < bytes) *reinterpret_cast<uint4*>(to + b + n * 512) = v[n];
        }
    }
}

// One launch of products.  DOWN: the second one.  JOINT: the CTAs of a cluster have one
// unit, a part of K each, and the first adds the others' sums to its own.
template <bool FP8, bool DOWN, int NB, bool JOINT>
__global__ void __launch_bounds__(kMoeThreads, 1)
moe_layer_kernel(const MoeParams p, const __grid_constant__ CUtensorMap weights, const __grid_constant__ CUtensorMap rows) {
    constexpr bool GATES = !FP8 && !DOWN;            // gate and up rows in one accumulator, two steps of K a stage
    constexpr bool LATER = DOWN || copied(FP8, NB);     // a launch before it writes its rows, in the list's order
    constexpr int KE = FP8 ? 128 : 64;               // elements of 128 bytes of K
    constexpr int KS = GATES ? 2 * KE : KE;          // of a stage
    constexpr int HALF = NB / 2;                     // columns that one finishing warp holds at most
    constexpr bool STACKED = stacked<FP8, DOWN, NB>();
    constexpr int COLS = columns<FP8, DOWN, NB>();   // of an accumulator
    constexpr int ACC = accumulators<FP8, DOWN>() * COLS;
    constexpr int STAGE = stage_bytes<FP8, NB>();
    constexpr int TURNS = turns<FP8, NB>();
    constexpr int ROWS = GATES ? kMoeRows / 2 : DOWN ? 2 * kMoeRows : kMoeRows;     // of a tile
    extern __shared__ unsigned char raw[];
    const uint32_t ring = (smem_addr(raw) + 1023u) & ~1023u;
    const int S = p.stages;
    unsigned char* behind = raw + (ring - smem_addr(raw)) + S * STAGE;
    Shared<FP8, NB>* s = reinterpret_cast<Shared<FP8, NB>*>(behind);
    uint32_t* entries = reinterpret_cast<uint32_t*>(behind + sizeof(Shared<FP8, NB>));
    uint16_t* list = reinterpret_cast<uint16_t*>(entries + p.entries);
    int* hist = reinterpret_cast<int*>(raw + (ring - smem_addr(raw)));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(smem_addr(&s->full[i]), 2);
            mbar_init(smem_addr(&s->empty[i]), 1);
        }
        for (int i = 0; i < kMaxTurns; ++i) {
            mbar_init(smem_addr(&s->done[i]), 1);
            mbar_init(smem_addr(&s->taken[i]), kFinishWarps);
        }
        mbar_init(smem_addr(&s->drain), 1);
        if (JOINT)
            for (int i = 0; i < kFinishWarps; ++i) mbar_init(smem_addr(&s->parts[i]), p.cluster - 1);
        s->dead = s->issued[0] = s->issued[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&weights);
        prefetch_map(&rows);
    }
    if (warp == 1) tmem_alloc(smem_addr(&s->tmem), tmem_columns<FP8, DOWN, NB>());
    // A later launch starts when every CTA of the one before has waited for what lay
    // before it, so only what that one writes is still to come: the ids, the weights
    // and their scales are there.
    if (!LATER) {
        pdl_wait();
        pdl_launch_dependents();
    }
    const int H = p.H, I = p.I, K = DOWN ? I : H, P = p.T * p.k;
    const int KB = (K + KS - 1) / KS;                // stages of a unit
    // this CTA's units, and its stages of them
    const int part = JOINT ? blockIdx.x % p.cluster : 0, parts = JOINT ? p.cluster : 1;
    const int U0 = blockIdx.x / parts, G = gridDim.x / parts, K0 = KB * part / parts, K1 = KB * (part + 1) / parts;

    // The weights: stages up to number `until`, from where the last call ended.
    struct {
        int u, kb, i, st, parity;
        bool ok;
    } feed{U0, K0, 0, 0, 1, true};
    auto load_weights = [&](int M, int units, int until) {
        for (; feed.u < units; feed.u += G) {
            const int tile = feed.u / M, expert = unpack_entry(entries[feed.u - tile * M]).expert;
            const int c1a = tile * ROWS, c1b = DOWN ? c1a + kMoeRows : I + c1a;
            for (; feed.kb < K1; ++feed.kb, ++feed.i) {
                if (feed.i == until) return;
                if (feed.i >= S) feed.ok = __all_sync(0xFFFFFFFFu, role_wait(&s->dead, p, smem_addr(&s->empty[feed.st]), feed.parity));
                if (!feed.ok) return;
                const uint32_t bar = smem_addr(&s->full[feed.st]), a = ring + feed.st * STAGE;
                const int c0 = feed.kb * KS;
                if (elect_lane()) {
                    mbar_arrive_expect_tx(bar, 2 * kPanel);
                    map_load3(a, &weights, c0, c1a, expert, bar);
                    if constexpr (GATES) {           // 64 rows a box; a box behind the end of K reads zeros
                        map_load3(a + kPanel / 2, &weights, c0, c1b, expert, bar);
                        map_load3(a + kPanel, &weights, c0 + KE, c1a, expert, bar);
                        map_load3(a + kPanel + kPanel / 2, &weights, c0 + KE, c1b, expert, bar);
                    } else {
                        map_load3(a + kPanel, &weights, c0, c1b, expert, bar);
                    }
                }
                __syncwarp();
                if (++feed.st == S) {
                    feed.st = 0;
                    feed.parity ^= 1;
                }
            }
            feed.kb = K0;
        }
    };

    const int tiles = ((DOWN ? H : I) + ROWS - 1) / ROWS;
    const bool report = !DOWN && blockIdx.x == 0;
    int M;
    if (P <= 32) {
        // nothing of the ring is in use, so that the first stages are asked for at once
        if (warp == 0) {
            M = sort_few<NB>(p, list, entries, report);
            if (lane == 0) s->scan[0] = M;
            load_weights(M, M * tiles, S);
        }
    } else {
        M = sort_pairs<FP8, NB>(p, s, list, entries, hist, report);
        shared_proxy_fence();         // the ring's memory held the counts
    }
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    if (P <= 32) M = s->scan[0];
    const uint32_t tmem = s->tmem;
    const int units = M * tiles;
    if (JOINT) cluster_arrive();
    bool met = false;                                // this thread has seen the cluster's arrivals

    if (warp == 0) {
        load_weights(M, units, INT_MAX);
        if (lane == 0) s->issued[0] = feed.i;
    } else if (warp == kWarps - 1) {  // the pairs' rows
        if (LATER) {
            pdl_wait();
            pdl_launch_dependents();
            proxy_fence();
        }
        bool ok = true;
        int i = 0, st = 0, parity = 1;
        for (int u = U0; ok && u < units; u += G) {
            const Entry en = unpack_entry(entries[u % M]);
            // x by tokens, four rows a copy (lane n: 4 n and on); in the list's order 16 a copy
            int4 r = make_int4(0, 0, 0, 0);
            if constexpr (!LATER) {
                int v[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) v[n] = list[en.start + min(4 * lane + n, en.n - 1)] / p.k;
                r = make_int4(v[0], v[1], v[2], v[3]);
            }
            const int copies = LATER ? (en.n + 15) >> 4 : (en.n + 3) >> 2;
            constexpr int COPY = LATER ? 2048 : 512;
            const uint32_t second = ring + 2 * kPanel + (STACKED ? (en.n + 15) & ~15 : NB) * 128;
            for (int kb = K0; kb < K1; ++kb, ++i) {
                if (i >= S) ok = role_wait(&s->dead, p, smem_addr(&s->empty[st]), parity);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const uint32_t bar = smem_addr(&s->full[st]), b = ring + st * STAGE + 2 * kPanel;
                if (lane == 0) mbar_arrive_expect_tx(bar, copies * COPY * (FP8 ? 1 : 2));
                __syncwarp();
                if (lane < copies) {
                    const uint32_t b2 = second + st * STAGE + lane * COPY;
                    if constexpr (LATER) {
                        map_load2(b + lane * COPY, &rows, kb * KS, en.start + lane * 16, bar);
                        // the other step of K, or the lower parts of h
                        if constexpr (!FP8) map_load2(b2, &rows, kb * KS + (GATES ? KE : 0), (DOWN ? P : 0) + en.start + lane * 16, bar);
                    } else {
                        map_gather4(b + lane * COPY, &rows, kb * KS, r, bar);
                        if constexpr (!FP8) map_gather4(b2, &rows, kb * KS + KE, r, bar);
                    }
                }
                if (++st == S) {
                    st = 0;
                    parity ^= 1;
                }
            }
        }
        if (lane == 0) s->issued[1] = i;
    } else if (warp == 1) {           // the products
        bool ok = true;
        int st = 0, parity = 0, uses = 0;
        for (int u = U0; ok && u < units; u += G) {
            const int n = (unpack_entry(entries[u % M]).n + 15) & ~15;
            const uint32_t desc = mma_desc(FP8, STACKED ? 2 * n : n);
            for (int kb = K0; kb < K1; ++kb) {
                // the stage is full, and (lane 1) the accumulator's values are in registers
                const bool again = lane == 1 && (FP8 || kb == K0) && uses >= TURNS;
                ok = __all_sync(0xFFFFFFFFu, role_wait(&s->dead, p, again ? smem_addr(&s->taken[uses % TURNS]) : smem_addr(&s->full[st]),
                                                       again ? (uses / TURNS - 1) & 1 : parity));
                if (!ok) break;
                tcgen05_fence_after();
                const bool last = FP8 || kb == K1 - 1;
                if (elect_lane()) {
                    const uint32_t a = ring + st * STAGE, d = tmem + uses % TURNS * ACC;
                    const uint64_t da = operand_desc(a), db = operand_desc(a + 2 * kPanel);
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint64_t from = da + half * (kPanel >> 4) + i * 2;
                            const bool more = i > 0 || (!FP8 && kb > K0) || (GATES && half > 0);
                            mma_issue<FP8>(d + (GATES ? 0 : half * COLS), from, db + (GATES ? half * (NB * 128 >> 4) : 0) + i * 2, desc, more);
                            if constexpr (DOWN && !FP8 && !STACKED)
                                mma_issue<FP8>(d + half * COLS, from, db + (NB * 128 >> 4) + i * 2, desc, true);
                        }
                    mma_commit(smem_addr(&s->empty[st]));
                    if (last) mma_commit(smem_addr(&s->done[uses % TURNS]));
                }
                __syncwarp();
                if (last) ++uses;
                if (++st == S) {
                    st = 0;
                    parity ^= 1;
                }
            }
        }
        if (!ok) {                    // products may be in flight
            if (elect_lane()) mma_commit(smem_addr(&s->drain));
            __syncwarp();
            mbar_wait(smem_addr(&s->drain), 0);
        }
    } else {                          // the ends of the units
        if (LATER) pdl_wait();
        const int quad = warp & 3, side = (warp - 2) >> 2, row = quad * 32 + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16) + side * 8;
        int uses = 0;
        bool ok = true;
        // where this warp's values of a part lie, 16 of a thread for each group of columns
        float* mine = p.parts + (static_cast<int64_t>(blockIdx.x) * kFinishWarps + (warp - 2)) * (NB / 16) * 512 + lane;
        auto put_part = [&](int q, const float (&a)[8], const float (&b)[8]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                mine[q * 512 + j * 32] = a[j];
                mine[q * 512 + 256 + j * 32] = b[j];
            }
        };
        auto add_parts = [&](int q, float (&a)[8], float (&b)[8]) {
            for (int r = 1; r < parts; ++r) {
                const float* from = mine + static_cast<int64_t>(r) * kFinishWarps * (NB / 16) * 512 + q * 512;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    a[j] += __ldcg(from + j * 32);
                    b[j] += __ldcg(from + 256 + j * 32);
                }
            }
        };
        // this part's sums are in the workspace
        auto hand_over = [&] {
            __threadfence();
            cluster_wait();
            met = true;
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(smem_addr(&s->parts[warp - 2]), 0);
        };
        // whether the others' are, for all of the finishing warps
        auto parts_there = [&] {
            cluster_wait();
            met = true;
            const bool there = role_wait<true>(&s->dead, p, smem_addr(&s->parts[warp - 2]), 0);
            __threadfence();
            return finishers_well(there);
        };
        for (int u = U0; ok && u < units; u += G) {
            const int tile = u / M;
            const Entry en = unpack_entry(entries[u - tile * M]);
            const uint16_t* pairs = list + en.start;
            // this warp's columns: eight from side * 8 on, from side * 8 + 16 on, ...
            const int groups = (en.n - side * 8 + 15) >> 4;
            // Columns c0 .. c0 + 7 of the second launch: products to y.
            auto to_y = [&](int c0, const float (&a)[8], const float (&b)[8]) {
                const int h0 = tile * ROWS + row, h1 = h0 + kMoeRows;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (c0 + j >= en.n) break;
                    float* y = p.y + static_cast<int64_t>(pairs[c0 + j]) * H;
                    if (h0 < H) y[h0] = a[j];
                    if (h1 < H) y[h1] = b[j];
                }
            };
            if constexpr (FP8) {
                const int HB = (H + 127) / 128, IB = I / 128;        // scale blocks
                float d0[NB / 16][8], d1[NB / 16][8];
                float(*sx)[HALF] = s->sx[warp - 2];
                // this lane's column's row of scales
                const int own = lane & (HALF - 1), at_own = min((own >> 3) * 16 + side * 8 + (own & 7), en.n - 1);
                const float* from = DOWN ? p.act_sf + static_cast<int64_t>(en.start + at_own) * KB
                                         : p.x_sf + static_cast<int64_t>(pairs[at_own] / p.k) * KB;
                const float* w0 = DOWN ? p.w2_sf + (static_cast<int64_t>(en.expert) * HB + 2 * tile) * IB
                                       : p.w13_sf + (static_cast<int64_t>(en.expert) * 2 * IB + tile) * HB;
                const float* w1 = DOWN ? w0 + (2 * tile + 1 < HB ? IB : 0) : w0 + static_cast<int64_t>(IB) * HB;
#pragma unroll
                for (int q = 0; q < NB / 16; ++q)
#pragma unroll
                    for (int i = 0; i < 8; ++i) d0[q][i] = d1[q][i] = 0.f;
                // the scales of four steps, and the next four on their way
                constexpr int AHEAD = 4;
                float sw0[AHEAD], sw1[AHEAD], f[AHEAD], nw0[AHEAD], nw1[AHEAD], nf[AHEAD];
                auto load_scales = [&](int kb) {
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i) {
                        const int at = min(kb + i, K1 - 1);
                        nw0[i] = __ldg(w0 + at);
                        nw1[i] = __ldg(w1 + at);
                        nf[i] = __ldcg(from + at);
                    }
                };
                load_scales(K0);
                for (int kb0 = K0; ok && kb0 < K1; kb0 += AHEAD) {
#pragma unroll
                    for (int i = 0; i < AHEAD; ++i) {
                        sw0[i] = nw0[i];
                        sw1[i] = nw1[i];
                        f[i] = nf[i];
                    }
                    load_scales(kb0 + AHEAD);
#pragma unroll
                    for (int step = 0; step < AHEAD; ++step) {
                        if (kb0 + step >= K1) break;
                        __syncwarp();
                        if (lane < HALF) {
                            sx[0][lane] = f[step] * sw0[step];
                            sx[1][lane] = f[step] * sw1[step];
                        }
                        __syncwarp();
                        ok = role_wait(&s->dead, p, smem_addr(&s->done[uses % TURNS]), uses / TURNS & 1);
                        ok = __all_sync(0xFFFFFFFFu, ok);
                        if (!ok) break;
                        tcgen05_fence_after();
                        const uint32_t acc = lanes + uses % TURNS * ACC;
                        constexpr int TWO = NB > 16 ? 2 : 1;           // groups on their way at once
#pragma unroll
                        for (int q0 = 0; q0 < NB / 16; q0 += TWO) {
                            if (q0 >= groups) break;
                            uint32_t a[TWO][8], b[TWO][8];
#pragma unroll
                            for (int n = 0; n < TWO; ++n) {            // one behind the last: columns that nothing uses
                                tmem_load8(acc + (q0 + n) * 16, a[n]);
                                tmem_load8(acc + COLS + (q0 + n) * 16, b[n]);
                            }
#pragma unroll
                            for (int n = 0; n < TWO; ++n) {
                                const int q = q0 + n;
                                tmem_wait_load(a[n], b[n]);
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    d0[q][i] = fmaf(__uint_as_float(a[n][i]), sx[0][q * 8 + i], d0[q][i]);
                                    d1[q][i] = fmaf(__uint_as_float(b[n][i]), sx[1][q * 8 + i], d1[q][i]);
                                }
                            }
                        }
                        tcgen05_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_addr(&s->taken[uses % TURNS]));
                        ++uses;
                    }
                }
                ok = finishers_well(ok);
                if (!ok) break;
                if (JOINT && part > 0) {
#pragma unroll
                    for (int q = 0; q < NB / 16; ++q)
                        if (q < groups) put_part(q, d0[q], d1[q]);
                    hand_over();
                    continue;
                }
                if (JOINT) {
                    ok = parts_there();
                    if (!ok) break;
#pragma unroll
                    for (int q = 0; q < NB / 16; ++q)
                        if (q < groups) add_parts(q, d0[q], d1[q]);
                }
                if constexpr (DOWN) {
#pragma unroll
                    for (int q = 0; q < NB / 16; ++q) {
                        if (q >= groups) break;
                        to_y(q * 16 + side * 8, d0[q], d1[q]);
                    }
                } else {
                    uint32_t(*top)[HALF] = s->top[side];      // the last unit's were read before finishers_well
                    const int i = tile * ROWS + row;
#pragma unroll
                    for (int q = 0; q < NB / 16; ++q) {
                        if (q >= groups) break;
                        uint32_t largest = 0;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            d0[q][j] = swiglu(d0[q][j], d1[q][j]);
                            const float m = fabsf(d0[q][j]);
                            const uint32_t t = __reduce_max_sync(0xFFFFFFFFu, m == m ? __float_as_uint(m) : 0u);
                            if (lane == j) largest = t;
                        }
                        if (lane < 8) top[quad][q * 8 + lane] = largest;
                    }
                    group_sync(1 + side, 128);
                    if (const int col = (lane >> 3) * 16 + side * 8 + (lane & 7); lane < HALF && col < en.n) {
                        const uint32_t t = max(max(top[0][lane], top[1][lane]), max(top[2][lane], top[3][lane]));
                        const float amax = fminf(fmaxf(__uint_as_float(t), kAmaxFloor), FLT_MAX);
                        sx[0][lane] = 448.f / amax;
                        if (quad == 0) p.act_sf[static_cast<int64_t>(en.start + col) * IB + tile] = amax / 448.f;
                    }
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < NB / 16; ++q) {
                        if (q >= groups) break;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int col = q * 16 + side * 8 + j;
                            if (col >= en.n) break;
                            p.act[static_cast<int64_t>(en.start + col) * I + i] = static_cast<uint8_t>(e4m3_rn_sat(d0[q][j] * sx[0][q * 8 + j]));
                        }
                    }
                }
            } else {
                ok = role_wait(&s->dead, p, smem_addr(&s->done[uses % TURNS]), uses / TURNS & 1);
                ok = finishers_well(ok);
                if (JOINT && part == 0 && ok) ok = parts_there();
                if (!ok) break;
                tcgen05_fence_after();
                const uint32_t acc = lanes + uses % TURNS * ACC;
#pragma unroll 1
                for (int q = 0; q < groups; ++q) {
                    const int c0 = q * 16 + side * 8;
                    uint32_t a[8], b[8];
                    float v0[8], v1[8];
                    tmem_load8(acc + q * 16, a);
                    tmem_load8(acc + (GATES ? 0 : COLS) + q * 16, b);
                    tmem_wait_load(a, b);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        v0[i] = __uint_as_float(a[i]);
                        v1[i] = __uint_as_float(b[i]);
                    }
                    if constexpr (STACKED) {
                        const int n16 = (en.n + 15) & ~15;
                        tmem_load8(acc + n16 + q * 16, a);
                        tmem_load8(acc + COLS + n16 + q * 16, b);
                        tmem_wait_load(a, b);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            v0[i] += __uint_as_float(a[i]);
                            v1[i] += __uint_as_float(b[i]);
                        }
                    }
                    if (JOINT && part > 0) {
                        put_part(q, v0, v1);
                        continue;
                    }
                    if (JOINT) add_parts(q, v0, v1);
                    if constexpr (DOWN) {
                        to_y(c0, v0, v1);
                    } else {
                        // lanes 0 .. 63 hold gate rows and finish columns 0 .. 3, lanes 64 .. 127 hold up
                        // rows and finish 4 .. 7
                        float(*other)[64] = s->other[side][NB > 16 ? q & 1 : 0];
                        const bool gates = row < 64;
                        const int r = row & 63, i = tile * ROWS + r;
#pragma unroll
                        for (int j = 0; j < 4; ++j) other[gates ? 4 + j : j][r] = gates ? v0[4 + j] : v0[j];
                        group_sync(1 + side, 128);
                        if (i < I) {
                            __nv_bfloat16* act = reinterpret_cast<__nv_bfloat16*>(p.act);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int col = c0 + (gates ? j : 4 + j);
                                if (col >= en.n) break;
                                const float h = gates ? swiglu(v0[j], other[j][r]) : swiglu(other[4 + j][r], v0[4 + j]);
                                const int64_t at = en.start + col;
                                const bool finite = fabsf(h) < INFINITY;
                                // an infinity is whole in its upper part, and no other h is made one
                                const __nv_bfloat16 high = __float2bfloat16_rn(finite ? fminf(fmaxf(h, -kBf16Max), kBf16Max) : h);
                                act[at * I + i] = high;
                                act[(at + P) * I + i] = __float2bfloat16_rn(finite ? h - __bfloat162float(high) : 0.f);
                            }
                        }
                    }
                }
                tcgen05_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&s->taken[uses % TURNS]));
                ++uses;
                if (JOINT && part > 0) hand_over();
            }
        }
    }
    __syncwarp();
    tcgen05_fence_before();
    __syncthreads();
    if (s->dead && tid == 0) {
        // Copies still in flight when the roles gave up: a stage that one of the two
        // loading warps did not come to gets its arrival, so that its phase can end.
        const int lo = min(s->issued[0], s->issued[1]), hi = max(s->issued[0], s->issued[1]);
        for (int i = lo; i < hi; ++i) mbar_arrive(smem_addr(&s->full[i % S]));
        for (int i = max(0, hi - S); i < hi; ++i) mbar_wait(smem_addr(&s->full[i % S]), (i / S) & 1);
    }
    __syncwarp();
    if (warp == 1) {
        tcgen05_fence_after();
        tmem_free(tmem, tmem_columns<FP8, DOWN, NB>());
    }
    if (JOINT) {                      // nobody leaves while another may still arrive on its barriers
        if (!met) cluster_wait();
        cluster_arrive();
        cluster_wait();
    }
}

// out[t] from y, a thread for four columns of a token: the pairs in slot order, eight
// rows in flight.
constexpr int kSumThreads = 128;
__global__ void __launch_bounds__(kSumThreads) moe_sum_kernel(const MoeParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int t = blockIdx.y, h = (blockIdx.x * kSumThreads + threadIdx.x) * 4;
    if (h >= p.H) return;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    const float* y = p.y + static_cast<int64_t>(t) * p.k * p.H + h;
    for (int j0 = 0; j0 < p.k; j0 += 8) {
        float4 v[8];
        float w[8];
        uint32_t on = 0;                              // a row without an expert holds anything: not added
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int pair = t * p.k + j0 + j;
            const bool in = j0 + j < p.k;
            v[j] = in ? __ldcg(reinterpret_cast<const float4*>(y + static_cast<int64_t>(j0 + j) * p.H)) : sum;
            w[j] = in ? __ldg(p.w + pair) : 0.f;
            if (in && valid_expert(__ldg(p.ids + pair), p.E)) on |= 1u << j;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (!(on >> j & 1u)) continue;
            sum.x = fmaf(w[j], v[j].x, sum.x);
            sum.y = fmaf(w[j], v[j].y, sum.y);
            sum.z = fmaf(w[j], v[j].z, sum.z);
            sum.w = fmaf(w[j], v[j].w, sum.w);
        }
    }
    st_u2(p.out + static_cast<int64_t>(t) * p.H + h, make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w)));
}

using Kernel = void (*)(const MoeParams, const CUtensorMap, const CUtensorMap);

template <bool FP8, int NB>
Kernel kernel_of(bool down, bool joint) {
    if (joint) return down ? moe_layer_kernel<FP8, true, NB, true> : moe_layer_kernel<FP8, false, NB, true>;
    return down ? moe_layer_kernel<FP8, true, NB, false> : moe_layer_kernel<FP8, false, NB, false>;
}

template <int NB>
Kernel kernel_of(bool fp8, bool down, bool joint) { return fp8 ? kernel_of<true, NB>(down, joint) : kernel_of<false, NB>(down, joint); }

Kernel kernel_for(const MoeLayerShape& s, bool down, bool joint) {
    switch (s.columns) {
        case 16: return kernel_of<16>(s.fp8, down, joint);
        case 32: return kernel_of<32>(s.fp8, down, joint);
        case 64: return kernel_of<64>(s.fp8, down, joint);
        default: return kernel_of<false, 128>(down, joint);
    }
}

constexpr int kMaxSmem = 227 * 1024;

template <bool FP8>
int shared_bytes(int columns) {
    return static_cast<int>(columns == 16 ? sizeof(Shared<FP8, 16>) : columns == 32 ? sizeof(Shared<FP8, 32>)
                            : columns == 64 ? sizeof(Shared<FP8, 64>) : sizeof(Shared<FP8, 128>));
}
int shared_bytes(const MoeLayerShape& s) { return s.fp8 ? shared_bytes<true>(s.columns) : shared_bytes<false>(s.columns); }

bool encode(void* encoder, CUtensorMap* map, bool fp8, int rank, const void* base, const uint64_t* dims, const uint32_t* box) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    cuuint64_t d[3], strides[2];
    cuuint32_t b[3], ones[3] = {1, 1, 1};
    uint64_t pitch = fp8 ? 1 : 2;
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        pitch *= dims[i];
        if (i + 1 < rank) strides[i] = pitch;
    }
    return reinterpret_cast<Encode>(encoder)(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
                                             const_cast<void*>(base), d, strides, b, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t align256(int64_t v) { return (v + 255) & ~int64_t(255); }

}  // namespace

// Chunks of experts' pairs that there can be.
static int most_entries(const MoeLayerShape& s) {
    const int P = s.T * s.k;
    return std::min(P, std::min(P, s.E) + P / s.columns);
}

void moe_layer_choose(MoeLayerShape& s) {
    const int64_t P = static_cast<int64_t>(s.T) * s.k;
    // columns for most experts' pairs, were they drawn evenly: fewer leave more of the ring to
    // the weights, and a popular expert's further chunks read its weights from L2
    const double mean = static_cast<double>(P) / s.E;
    int64_t want = static_cast<int64_t>(mean + 3.0 * std::sqrt(mean) + 4.0);
    if (want > s.T) want = s.T;
    // E4M3: 64 at most, whose accumulators and sums a finishing warp holds in registers
    // (256 tokens of 16 experts of 4096 x 1024: 215 us with 128, 98 with 64, 126 where more than
    // 38 chunks are a third turn of the SMs)
    s.columns = want <= 16 ? 16 : want <= 32 ? 32 : want <= 64 || s.fp8 ? 64 : 128;
    s.entries = (most_entries(s) + 3) & ~3;
    const int behind = shared_bytes(s) + s.entries * 4 + static_cast<int>((P * 2 + 15) & ~15);
    const int stage = 2 * kPanel + s.columns * 128 * (s.fp8 ? 1 : 2);
    s.stages = (kMaxSmem - 1024 - behind) / stage;
    if (s.stages > kRingStages) s.stages = kRingStages;
    s.smem = 1024 + behind + s.stages * stage;
    s.act = 0;
    s.act_sf = align256(P * s.I * (s.fp8 ? 1 : 4));
    s.y = s.act_sf + (s.fp8 ? align256(P * (s.I / 128) * 4) : 0);
    s.rows = s.y + align256(P * s.H * 4);
    s.parts = s.rows + (copied(s.fp8, s.columns) ? align256(P * s.H * 2) : 0);
}

void* moe_layer_encoder() {
    static std::once_flag once;
    static void* fn = nullptr;
    std::call_once(once, [] {
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess) {
            fn = nullptr;
            cudaGetLastError();
        }
    });
    return fn;
}

template <typename F>
static cudaError_t prepare(F* kernel) {
    const void* k = reinterpret_cast<const void*>(kernel);
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, k);
    // the attribute is per kernel, shared by every plan: always the most
    return e == cudaSuccess ? cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) : e;
}

// Units are divided where a part saves at least `worth` stages (of 0.4 us; the launch in
// clusters and the handing over cost 4 us) and the most units that there can be still
// leave a third of the SMs idle: there the second launch loads ahead (one token of E4M3
// experts, 4096 x 1024: 31.3 us as 64 units and 33.1 as 128 halves).  86 tokens of 8
// experts of 5936 x 256 in E4M3: 47 -> 31 us; 2 of 304 x 1248: 15.0 -> 12.2.
cudaError_t moe_layer_prepare(MoeLayerShape& s, int sms) {
    constexpr int worth = 10;
    s.bytes = s.parts;
    for (int down = 0; down < 2; ++down) {
        const int rows = down ? 2 * kMoeRows : s.fp8 ? kMoeRows : kMoeRows / 2, step = s.fp8 ? 128 : down ? 64 : 128;
        const int64_t units = static_cast<int64_t>(most_entries(s)) * (((down ? s.H : s.I) + rows - 1) / rows);
        const int steps = ((down ? s.I : s.H) + step - 1) / step;
        s.cluster[down] = 1;
        s.grid[down] = sms;
        cudaError_t e;
        for (int c = 8; c > 1; c /= 2) {
            if (units * c * 3 > sms * 2 || steps - steps / c < worth) continue;
            const Kernel kernel = kernel_for(s, down != 0, true);
            if ((e = prepare(kernel)) != cudaSuccess) return e;
            cudaLaunchConfig_t cfg{};
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = static_cast<unsigned>(c);
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.gridDim = dim3(static_cast<unsigned>(units * c), 1, 1);
            cfg.blockDim = dim3(kMoeThreads, 1, 1);
            cfg.dynamicSmemBytes = static_cast<size_t>(s.smem);
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            int n = 0;
            if ((e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) != cudaSuccess) return e;
            if (n < units) continue;                  // they do not all find room at once
            s.cluster[down] = c;
            s.grid[down] = static_cast<int>(units) * c;
            s.bytes = std::max(s.bytes, s.parts + int64_t(s.grid[down]) * kFinishWarps * (s.columns / 16) * 512 * 4);
            break;
        }
        if (s.cluster[down] == 1 && (e = prepare(kernel_for(s, down != 0, false))) != cudaSuccess) return e;
    }
    if (copied(s.fp8, s.columns)) {
        const cudaError_t e = prepare(moe_rows_kernel);
        if (e != cudaSuccess) return e;
    }
    return preload(moe_sum_kernel);
}

cudaError_t moe_layer_launch(const MoeLayerShape& s, const MoeParams& p, const void* x, const void* w13, const void* w2,
                             int pdl, cudaStream_t st) {
    void* enc = moe_layer_encoder();
    if (!enc) return cudaErrorNotSupported;
    const uint64_t T = s.T, H = s.H, I = s.I, E = s.E, P = T * s.k * (s.fp8 ? 1 : 2);
    const uint32_t ke = s.fp8 ? 128 : 64;
    const uint64_t dx[] = {H, T}, d13[] = {H, 2 * I, E}, da[] = {I, P}, d2[] = {I, H, E};
    const uint32_t row[] = {ke, 1}, box13[] = {ke, static_cast<uint32_t>(s.fp8 ? kMoeRows : kMoeRows / 2), 1}, box2[] = {ke, kMoeRows, 1};
    const uint32_t rows16[] = {ke, 16};
    CUtensorMap mx, m13, ma, m2;
    const bool copy = copied(s.fp8, s.columns);
    const uint64_t dr[] = {H, static_cast<uint64_t>(s.T) * s.k};
    if (!encode(enc, &mx, s.fp8, 2, copy ? p.rows : x, copy ? dr : dx, copy ? rows16 : row) || !encode(enc, &m13, s.fp8, 3, w13, d13, box13) ||
        !encode(enc, &ma, s.fp8, 2, p.act, da, rows16) || !encode(enc, &m2, s.fp8, 3, w2, d2, box2))
        return cudaErrorInvalidValue;
    MoeParams up = p, down = p;
    up.cluster = s.cluster[0];
    down.cluster = s.cluster[1];
    cudaError_t e = cudaSuccess;
    if (copy) {
        const int pairs = s.T * s.k, smem = shared_bytes(s) + s.entries * 4 + (kWarps + 1) * s.E * 4 + pairs * 8;
        e = layer_launch(moe_rows_kernel, std::min(s.grid[0], (pairs + kWarps - 1) / kWarps),
                         kMoeThreads, smem, 1, pdl, st, p, static_cast<const uint8_t*>(x));
    }
    if (e == cudaSuccess) e = layer_launch(kernel_for(s, false, up.cluster > 1), s.grid[0], kMoeThreads, s.smem, up.cluster, pdl, st, up, m13, mx);
    if (e == cudaSuccess) e = layer_launch(kernel_for(s, true, down.cluster > 1), s.grid[1], kMoeThreads, s.smem, down.cluster, pdl, st, down, m2, ma);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((s.H + 4 * kSumThreads - 1) / (4 * kSumThreads), s.T, 1);
    cfg.blockDim = dim3(kSumThreads, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, moe_sum_kernel, p);
}

}  // namespace mfr
