// A whole MoE layer for a few tokens, in two launches:
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
// columns (B).  A warp keeps a ring of stages of 128 bytes of K filled by
// tensor-map copies (two boxes of 128 weight rows, the pairs' rows gathered four
// at a time), one thread issues tcgen05 products into tensor memory, and eight
// warps finish one tile while the next one is multiplied.
//
// Each CTA sorts the pairs by expert itself (at most 4096, from L2), so that no
// launch before it is needed; work is (expert, chunk of its pairs) x (tile of
// weight rows), in turns over persistent CTAs.
//   first launch:  a tile is 128 rows of G and the same 128 of U, so that a thread
//                  holds both halves of an element of h
//   second launch: a tile is 256 rows of D; the products go to y[pair] in FP32, and
//                  the CTA that finishes the last expert of a tile adds the pairs of
//                  each token in slot order: no atomics on values, the same bits in
//                  every call
//
// E4M3: products of 128 columns of K are one accumulation in tensor memory, which
// the finishing warps scale and add in FP32 registers.
#include <cfloat>
#include <mutex>

#include "moe_step_ops.h"
#include "mfr_layer.h"
#include "mfr_step.h"
#include "mfr_tcgen05.cuh"

namespace mfr {
namespace {

constexpr int kWarps = kMoeThreads / 32;
constexpr int kFinishWarps = 8;
constexpr int kTileBytes = 2 * kMoeRows * 128;     // weights of a stage
constexpr int kRingStages = 6;
constexpr float kAmaxFloor = 0x1p-100f;

template <int NB>
constexpr int stage_bytes() { return kTileBytes + NB * 128; }

// Behind the ring.
struct Shared {
    uint64_t full[kRingStages], empty[kRingStages];
    uint64_t done[2], taken[2];       // an accumulator is complete; its values are in registers
    uint64_t drain;
    uint32_t tmem;
    int dead;                         // a wait ran out: every role leaves
    int last;                         // this CTA finished the last piece of a tile
    int entries;
    int scan[kWarps];
    float sx[kFinishWarps][64];       // E4M3: scales of a warp's columns
    uint32_t top[2][4][64];           // E4M3: largest magnitudes, by half, warp and column
};

__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async;" ::: "memory"); }
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

// A role's wait for another.  It gives up after kWaitCycles, or when another has given up.
__device__ bool role_wait(Shared* s, int* status, uint32_t bar, uint32_t parity) {
    if (mbar_test_parity(bar, parity)) return true;
    volatile int* dead = &s->dead;
    const long long t0 = clock64();
    while (!mbar_test_parity(bar, parity)) {
        if (*dead) return false;
        if (clock64() - t0 > kWaitCycles) {
            *dead = 1;
            atomicOr(status, MFR_STATUS_TIMEOUT);
            return false;
        }
    }
    return true;
}

// (expert, first place in the sorted list, pairs) of a chunk of pairs.
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
// `hist`: [kWarps + 1][E].  All threads call it.
template <int NB>
__device__ int sort_pairs(const MoeParams& p, Shared* s, uint16_t* list, uint32_t* entries, int* hist, bool report) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = p.T * p.k, E = p.E;
    const int seg = ((P + kWarps - 1) / kWarps + 31) & ~31, first = warp * seg, last = min(P, first + seg);
    for (int i = tid; i < kWarps * E; i += kMoeThreads) hist[i] = 0;
    __syncthreads();
    bool bad = false;
    for (int i = first + lane; i < last; i += 32) {
        const int id = p.ids[i];
        if (valid_expert(id, E)) atomicAdd(&hist[warp * E + id], 1);
        else bad |= !(p.sentinel && id < 0);
    }
    if (report && bad) atomicOr(p.status, MFR_STATUS_BAD_INDEX);
    __syncthreads();
    // each thread: a run of experts; pairs in the low half, chunks in the high half
    const int per = (E + kMoeThreads - 1) / kMoeThreads, e0 = min(E, tid * per), e1 = min(E, e0 + per);
    uint32_t sum = 0;
    for (int e = e0; e < e1; ++e) {
        int n = 0;
        for (int w = 0; w < kWarps; ++w) {
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
    uint32_t base = incl - sum;
    for (int w = 0; w < warp; ++w) base += static_cast<uint32_t>(s->scan[w]);
    int at = static_cast<int>(base & 0xFFFFu), chunk = static_cast<int>(base >> 16);
    for (int e = e0; e < e1; ++e) {
        for (int w = 0; w < kWarps; ++w) hist[w * E + e] += at;
        const int n = hist[kWarps * E + e];
        for (int c = 0; c < n; c += NB) entries[chunk++] = pack_entry(e, at + c, min(NB, n - c));
        at += n;
    }
    if (tid == kMoeThreads - 1) s->entries = chunk;
    __syncthreads();
    for (int i0 = first; i0 < last; i0 += 32) {
        const int i = i0 + lane, id = i < last ? p.ids[i] : -1;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, id);
        const bool ok = valid_expert(id, E);
        if (ok) list[hist[warp * E + id] + __popc(same & ((1u << lane) - 1))] = static_cast<uint16_t>(i);
        __syncwarp();
        if (ok && lane == __ffs(same) - 1) hist[warp * E + id] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    return s->entries;
}

__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.f + __expf(-g)) * u; }

// One launch of the layer.  DOWN: the second one.
template <bool FP8, bool DOWN, int NB>
__global__ void __launch_bounds__(kMoeThreads, 1)
moe_layer_kernel(const MoeParams p, const __grid_constant__ CUtensorMap weights, const __grid_constant__ CUtensorMap rows) {
    constexpr int KE = FP8 ? 128 : 64;               // elements of K in a stage
    constexpr int HALF = NB / 2;                     // columns that one finishing warp holds at most
    extern __shared__ unsigned char raw[];
    const uint32_t ring = (smem_addr(raw) + 1023u) & ~1023u;
    unsigned char* behind = raw + (ring - smem_addr(raw)) + p.stages * stage_bytes<NB>();
    Shared* s = reinterpret_cast<Shared*>(behind);
    uint32_t* entries = reinterpret_cast<uint32_t*>(behind + sizeof(Shared));
    uint16_t* list = reinterpret_cast<uint16_t*>(entries + p.entries);
    int* hist = reinterpret_cast<int*>(raw + (ring - smem_addr(raw)));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int S = p.stages;

    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(smem_addr(&s->full[i]), 1);
            mbar_init(smem_addr(&s->empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&s->done[i]), 1);
            mbar_init(smem_addr(&s->taken[i]), kFinishWarps);
        }
        mbar_init(smem_addr(&s->drain), 1);
        s->dead = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        prefetch_map(&weights);
        prefetch_map(&rows);
    }
    if (warp == 1) tmem_alloc(smem_addr(&s->tmem), 4 * NB < 32 ? 32 : 4 * NB);
    pdl_wait();
    pdl_launch_dependents();
    const int M = sort_pairs<NB>(p, s, list, entries, hist, !DOWN && blockIdx.x == 0);
    proxy_fence();                    // the ring's memory held the counts
    tcgen05_fence_before();
    __syncthreads();
    tcgen05_fence_after();
    const uint32_t tmem = s->tmem;

    const int H = p.H, I = p.I, K = DOWN ? I : H;
    const int KB = (K + KE - 1) / KE;
    const int tiles = DOWN ? (H + 2 * kMoeRows - 1) / (2 * kMoeRows) : (I + kMoeRows - 1) / kMoeRows;
    const int units = M * tiles;
    const int HB = (H + 127) / 128, IB = I / 128;    // scale blocks
    if (!DOWN && blockIdx.x == 0)
        for (int i = tid; i < (H + 2 * kMoeRows - 1) / (2 * kMoeRows); i += kMoeThreads) p.counters[i] = 0;
    int issued = 0;                   // stages that the loading warp has begun

    if (warp == 0) {
        bool ok = true;
        for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
            const Entry en = unpack_entry(entries[u / tiles]);
            const int tile = u % tiles;
            const int c1a = DOWN ? tile * 2 * kMoeRows : tile * kMoeRows;
            const int c1b = DOWN ? c1a + kMoeRows : I + c1a;
            const int gathers = (en.n + 3) >> 2;
            int r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int pair = list[en.start + min(4 * lane + i, en.n - 1)];
                r[i] = DOWN ? pair : pair / p.k;
            }
            for (int kb = 0; kb < KB; ++kb, ++issued) {
                const int st = issued % S, turn = issued / S;
                if (turn > 0) ok = role_wait(s, p.status, smem_addr(&s->empty[st]), (turn - 1) & 1);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const uint32_t bar = smem_addr(&s->full[st]), a = ring + st * stage_bytes<NB>();
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar, kTileBytes + gathers * 512);
                    map_load3(a, &weights, kb * KE, c1a, en.expert, bar);
                    map_load3(a + kMoeRows * 128, &weights, kb * KE, c1b, en.expert, bar);
                }
                __syncwarp();
                if (lane < gathers)
                    map_gather4(a + kTileBytes + lane * 512, &rows, kb * KE, make_int4(r[0], r[1], r[2], r[3]), bar);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            bool ok = true;
            int stage = 0, uses = 0;
            for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
                const Entry en = unpack_entry(entries[u / tiles]);
                const uint32_t desc = mma_desc(FP8, (en.n + 15) & ~15);
                for (int kb = 0; kb < KB; ++kb, ++stage) {
                    const int st = stage % S;
                    if (FP8 || kb == 0) {
                        if (uses > 1) ok = role_wait(s, p.status, smem_addr(&s->taken[uses & 1]), ((uses >> 1) - 1) & 1);
                        if (!ok) break;
                        tcgen05_fence_after();
                    }
                    ok = role_wait(s, p.status, smem_addr(&s->full[st]), (stage / S) & 1);
                    if (!ok) break;
                    tcgen05_fence_after();
                    const uint32_t a = ring + st * stage_bytes<NB>(), d = tmem + (uses & 1) * 2 * NB;
                    const uint64_t da = operand_desc(a), db = operand_desc(a + kTileBytes);
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_issue<FP8>(d + half * NB, da + half * (kMoeRows * 128 >> 4) + i * 2, db + i * 2, desc,
                                           i > 0 || (!FP8 && kb > 0));
                    mma_commit(smem_addr(&s->empty[st]));
                    if (FP8 || kb == KB - 1) {
                        mma_commit(smem_addr(&s->done[uses & 1]));
                        ++uses;
                    }
                }
            }
            if (!ok) {                // products may be in flight
                mma_commit(smem_addr(&s->drain));
                mbar_wait(smem_addr(&s->drain), 0);
            }
        }
    } else {
        const int quad = warp & 3, side = (warp - 2) >> 2, row = quad * 32 + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16) + side * 8;
        int uses = 0;
        bool ok = true;
        // column j of this warp is column (j / 8) * 16 + side * 8 + j % 8 of the accumulator
        for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
            const Entry en = unpack_entry(entries[u / tiles]);
            const int tile = u % tiles;
            float d0[HALF], d1[HALF];
            if constexpr (FP8) {
                float* sx = s->sx[warp - 2];
                int from[2];          // this lane's columns' rows of scales
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int j = lane + 32 * i, c = (j >> 3) * 16 + side * 8 + (j & 7);
                    const int pair = list[en.start + min(c, en.n - 1)];
                    from[i] = DOWN ? pair : pair / p.k;
                }
                const float* scales = DOWN ? p.act_sf : p.x_sf;
                const float* w0 = DOWN ? p.w2_sf + (static_cast<int64_t>(en.expert) * HB + 2 * tile) * IB
                                       : p.w13_sf + (static_cast<int64_t>(en.expert) * 2 * IB + tile) * HB;
                const float* w1 = DOWN ? w0 + (2 * tile + 1 < HB ? IB : 0) : w0 + static_cast<int64_t>(IB) * HB;
#pragma unroll
                for (int j = 0; j < HALF; ++j) d0[j] = d1[j] = 0.f;
                for (int kb = 0; kb < KB; ++kb, ++uses) {
                    const float sw0 = w0[kb], sw1 = w1[kb];
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (lane + 32 * i < HALF) sx[lane + 32 * i] = scales[static_cast<int64_t>(from[i]) * KB + kb];
                    __syncwarp();
                    ok = role_wait(s, p.status, smem_addr(&s->done[uses & 1]), (uses >> 1) & 1);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    tcgen05_fence_after();
                    const uint32_t at = lanes + (uses & 1) * 2 * NB;
#pragma unroll
                    for (int q = 0; q < NB / 16; ++q) {
                        if (q * 16 + side * 8 >= en.n) break;
                        uint32_t a[8], b[8];
                        tmem_load8(at + q * 16, a);
                        tmem_load8(at + NB + q * 16, b);
                        tmem_wait_load(a, b);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float f = sx[q * 8 + i];
                            d0[q * 8 + i] = fmaf(__uint_as_float(a[i]), f * sw0, d0[q * 8 + i]);
                            d1[q * 8 + i] = fmaf(__uint_as_float(b[i]), f * sw1, d1[q * 8 + i]);
                        }
                    }
                    tcgen05_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&s->taken[uses & 1]));
                }
            } else {
                ok = role_wait(s, p.status, smem_addr(&s->done[uses & 1]), (uses >> 1) & 1);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (ok) {
                    tcgen05_fence_after();
                    const uint32_t at = lanes + (uses & 1) * 2 * NB;
#pragma unroll
                    for (int q = 0; q < NB / 16; ++q) {
                        if (q * 16 + side * 8 >= en.n) break;
                        uint32_t a[8], b[8];
                        tmem_load8(at + q * 16, a);
                        tmem_load8(at + NB + q * 16, b);
                        tmem_wait_load(a, b);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            d0[q * 8 + i] = __uint_as_float(a[i]);
                            d1[q * 8 + i] = __uint_as_float(b[i]);
                        }
                    }
                    tcgen05_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&s->taken[uses & 1]));
                    ++uses;
                }
            }
            ok = finishers_well(ok);
            if (!ok) break;
            if constexpr (!DOWN) {
                const int i = tile * kMoeRows + row;
#pragma unroll
                for (int j = 0; j < HALF; ++j) d0[j] = swiglu(d0[j], d1[j]);
                if constexpr (FP8) {
                    uint32_t(*top)[64] = s->top[side];
#pragma unroll
                    for (int j = 0; j < HALF; ++j) {
                        if ((j >> 3) * 16 + side * 8 + (j & 7) >= en.n) continue;
                        const float m = fabsf(d0[j]);
                        const uint32_t t = __reduce_max_sync(0xFFFFFFFFu, m == m ? __float_as_uint(m) : 0u);
                        if (lane == (j & 31)) top[quad][j] = t;
                    }
                    group_sync(1 + side, 128);
#pragma unroll
                    for (int j = 0; j < HALF; ++j) {
                        const int c = (j >> 3) * 16 + side * 8 + (j & 7);
                        if (c < en.n) {
                            const uint32_t t = max(max(top[0][j], top[1][j]), max(top[2][j], top[3][j]));
                            const float amax = fminf(fmaxf(__uint_as_float(t), kAmaxFloor), FLT_MAX);
                            const int pair = list[en.start + c];
                            p.act[static_cast<int64_t>(pair) * I + i] = static_cast<uint8_t>(e4m3_rn_sat(d0[j] * (448.f / amax)));
                            if (row == 0) p.act_sf[static_cast<int64_t>(pair) * IB + tile] = amax / 448.f;
                        }
                    }
                    group_sync(1 + side, 128);
                } else {
                    if (i < I)
#pragma unroll
                        for (int j = 0; j < HALF; ++j) {
                            const int c = (j >> 3) * 16 + side * 8 + (j & 7);
                            if (c < en.n)
                                reinterpret_cast<__nv_bfloat16*>(p.act)[static_cast<int64_t>(list[en.start + c]) * I + i] =
                                    __float2bfloat16_rn(d0[j]);
                        }
                }
            } else {
                const int h0 = tile * 2 * kMoeRows + row, h1 = h0 + kMoeRows;
#pragma unroll
                for (int j = 0; j < HALF; ++j) {
                    const int c = (j >> 3) * 16 + side * 8 + (j & 7);
                    if (c < en.n) {
                        float* y = p.y + static_cast<int64_t>(list[en.start + c]) * H;
                        if (h0 < H) y[h0] = d0[j];
                        if (h1 < H) y[h1] = d1[j];
                    }
                }
                __threadfence();
                group_sync(3, 32 * kFinishWarps);
                if (tid == 64) s->last = atomicAdd(&p.counters[tile], 1) == M - 1;
                group_sync(3, 32 * kFinishWarps);
                if (s->last) {        // every pair's products for these columns are there
                    __threadfence();
                    const int q = (tid - 64) & 63, h = tile * 2 * kMoeRows + q * 4;
                    if (h < H)
                        for (int t = (tid - 64) >> 6; t < p.T; t += 4) {
                            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
                            for (int j = 0; j < p.k; ++j) {
                                const int pair = t * p.k + j;
                                if (!valid_expert(p.ids[pair], p.E)) continue;
                                const float w = p.w[pair];
                                const float4 v = __ldcg(reinterpret_cast<const float4*>(p.y + static_cast<int64_t>(pair) * H + h));
                                sum.x = fmaf(w, v.x, sum.x);
                                sum.y = fmaf(w, v.y, sum.y);
                                sum.z = fmaf(w, v.z, sum.z);
                                sum.w = fmaf(w, v.w, sum.w);
                            }
                            st_u2(p.out + static_cast<int64_t>(t) * H + h,
                                  make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w)));
                        }
                }
            }
        }
    }
    if (DOWN && M == 0)               // no pair has an expert here
        for (int64_t i = (static_cast<int64_t>(blockIdx.x) * kMoeThreads + tid) * 4; i < static_cast<int64_t>(p.T) * H;
             i += static_cast<int64_t>(gridDim.x) * kMoeThreads * 4)
            st_u2(p.out + i, make_uint2(0, 0));
    __syncwarp();
    if (warp == 0) {
        // copies still in flight, when a role gave up before it took their stage
        if (s->dead && lane == 0)
            for (int i = max(0, issued - S); i < issued; ++i) mbar_wait(smem_addr(&s->full[i % S]), (i / S) & 1);
        __syncwarp();
    }
    tcgen05_fence_before();
    __syncthreads();
    if (warp == 1) {
        tcgen05_fence_after();
        tmem_free(tmem, 4 * NB < 32 ? 32 : 4 * NB);
    }
}

using Kernel = void (*)(const MoeParams, const CUtensorMap, const CUtensorMap);

template <int NB>
Kernel kernel_of(bool fp8, bool down) {
    if (fp8) return down ? moe_layer_kernel<true, true, NB> : moe_layer_kernel<true, false, NB>;
    return down ? moe_layer_kernel<false, true, NB> : moe_layer_kernel<false, false, NB>;
}

Kernel kernel_for(const MoeLayerShape& s, bool down) {
    switch (s.columns) {
        case 16: return kernel_of<16>(s.fp8, down);
        case 32: return kernel_of<32>(s.fp8, down);
        case 64: return kernel_of<64>(s.fp8, down);
        default: return kernel_of<128>(s.fp8, down);
    }
}

constexpr int kMaxSmem = 227 * 1024;

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

void moe_layer_choose(MoeLayerShape& s, int sms) {
    const int64_t P = static_cast<int64_t>(s.T) * s.k, elem = s.fp8 ? 1 : 2;
    s.columns = s.T <= 16 ? 16 : s.T <= 32 ? 32 : s.T <= 64 ? 64 : 128;
    const int stage = kTileBytes + s.columns * 128;
    const int64_t entries = (P < s.E ? P : s.E) + P / s.columns;
    s.entries = static_cast<int>((entries < P ? entries : P) + 1) & ~1;
    const int behind = static_cast<int>(sizeof(Shared)) + s.entries * 4 + static_cast<int>((P * 2 + 15) & ~15);
    s.stages = (kMaxSmem - 1024 - behind) / stage;
    if (s.stages > kRingStages) s.stages = kRingStages;
    s.smem = 1024 + behind + s.stages * stage;
    s.grid = sms;
    s.act = 0;
    s.act_sf = align256(P * s.I * elem);
    s.y = s.act_sf + (s.fp8 ? align256(P * (s.I / 128) * 4) : 0);
    s.counters = s.y + align256(P * s.H * 4);
    s.bytes = s.counters + align256((s.H + 2 * kMoeRows - 1) / (2 * kMoeRows) * 4);
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

cudaError_t moe_layer_prepare(const MoeLayerShape& s) {
    for (int down = 0; down < 2; ++down) {
        const void* k = reinterpret_cast<const void*>(kernel_for(s, down != 0));
        cudaFuncAttributes a;
        cudaError_t e = cudaFuncGetAttributes(&a, k);
        // the attribute is per kernel, shared by every plan: always the most
        if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t moe_layer_launch(const MoeLayerShape& s, const MoeParams& p, const void* x, const void* w13, const void* w2,
                             int pdl, cudaStream_t st) {
    void* enc = moe_layer_encoder();
    if (!enc) return cudaErrorNotSupported;
    const uint64_t T = s.T, H = s.H, I = s.I, E = s.E, P = T * s.k;
    const uint32_t ke = s.fp8 ? 128 : 64;
    const uint64_t dx[] = {H, T}, d13[] = {H, 2 * I, E}, da[] = {I, P}, d2[] = {I, H, E};
    const uint32_t row[] = {ke, 1}, box[] = {ke, kMoeRows, 1};
    CUtensorMap mx, m13, ma, m2;
    if (!encode(enc, &mx, s.fp8, 2, x, dx, row) || !encode(enc, &m13, s.fp8, 3, w13, d13, box) ||
        !encode(enc, &ma, s.fp8, 2, p.act, da, row) || !encode(enc, &m2, s.fp8, 3, w2, d2, box))
        return cudaErrorInvalidValue;
    cudaError_t e = layer_launch(kernel_for(s, false), s.grid, kMoeThreads, s.smem, 1, pdl, st, p, m13, mx);
    if (e == cudaSuccess) e = layer_launch(kernel_for(s, true), s.grid, kMoeThreads, s.smem, 1, pdl, st, p, m2, ma);
    return e;
}

}  // namespace mfr
