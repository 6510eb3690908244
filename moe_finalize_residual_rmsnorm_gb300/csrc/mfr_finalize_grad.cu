// Gradient of the finalize's weighted sum, for the pairs (t, j) that have a row r:
//
//   d_expert_out[r, h]   = bf16( w[t, j] * d_out[t, h] )
//   d_topk_weights[t, j] = sum_h d_out[t, h] * expert_out[r, h]
//
// Both come from one pass: a token's gradient is read once and, chunk by chunk
// in registers, multiplied into its k rows, while the k rows' dot products
// run beside.  It reads a row and writes a row per pair (2.35 GB at 16384 x
// 4096, k = 8), so bytes bound it, and what counts is that enough of them are
// in flight: eight 16-byte row loads a thread (with few slots from two chunks,
// k = 2 at 16384 x 4096: 126 us with one, 99 with two; with more than eight
// slots sixteen loads and two CTAs of 256 threads an SM, k = 16: 653 us, 820 in
// two groups of eight), and 768 threads an SM (measured at k = 8: 344 us, 1.01
// of the copy rate, and with an FP32 gradient 362 us, 1.01; with 512 threads and
// more registers 430 us and more, with 1024 and fewer 380).  At the registers
// that 768 threads leave, three of the bf16 forms (k = 3 and 4, and k = 5 to 8 with
// and without a cluster) spill 12 bytes a thread.
// Rows are written past L1.  The dot products are summed per thread in column
// order, over the lanes by a reduce-scatter butterfly and over the warps in
// order, all in FP32, so a call gives the same bits every time; a token's
// threads, turns and CTAs go by T, so in another batch its sums may be added in
// another order.  A row's gradient is rounded once, from the FP32 product to
// bf16, the type of the rows that the experts' GEMMs take their gradients in.
#include <cooperative_groups.h>

#include "mfr_maps.cuh"

namespace cg = cooperative_groups;

namespace mfr {
namespace {

constexpr int kThreads = 256;

template <bool F32>
__device__ __forceinline__ void load_grad(const void* d_out, int64_t at, float (&g)[8]) {
    if constexpr (F32) {
        const float* f = static_cast<const float*>(d_out) + at;
        const float4 a = ld_once_f4(f), b = ld_once_f4(f + 4);
        g[0] = a.x; g[1] = a.y; g[2] = a.z; g[3] = a.w;
        g[4] = b.x; g[5] = b.y; g[6] = b.z; g[7] = b.w;
    } else {
        unpack8(ld_stream_u4(static_cast<const uint16_t*>(d_out) + at), g);
    }
}

// One token a CTA, thread i of it the chunks i, i + blockDim.x, ... of the
// token's rows, U of them at a time; SG: slots at most.  SPLIT: a token has a
// cluster of csize CTAs, each a share of the chunks, whose dot products meet in
// the first one's shared memory.  The row_ctas CTAs (whole clusters) before the
// tokens' look after the rows' side of the maps, `rpw` rows a warp.
template <bool F32, int SG, int U, bool SPLIT>
__global__ void __launch_bounds__(kThreads, SG > 8 ? 2 : 3) finalize_grad_kernel(const FinalizeGradParams p, const int row_ctas,
                                                                                   const int rpw, const int csize) {
    __shared__ int s_row[kMaxK];      // -1: the pair has no row
    __shared__ float s_w[kMaxK];
    __shared__ float s_part[kThreads / 32][SG > 8 ? 16 : 8];
    __shared__ float s_split[8][SPLIT ? kMaxK : 1];
    const MapParams& m = p.m;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int chunks = p.H >> 3;
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x < row_ctas) {
        const int64_t r0 = (static_cast<int64_t>(blockIdx.x) * warps + warp) * rpw;
        const bool pad = lane < rpw && r0 + lane < m.R && row_is_padding(m, r0 + lane);
        for (uint32_t todo = __ballot_sync(0xFFFFFFFFu, pad); todo; todo &= todo - 1) {
            uint16_t* row = p.d_expert_out + (r0 + __ffs(todo) - 1) * p.H;
            for (int c = lane; c < chunks; c += 32) st_stream_u4(row + c * 8, make_uint4(0, 0, 0, 0));
        }
        return;
    }
    const int64_t t = (blockIdx.x - row_ctas) / csize;
    const int rank = SPLIT ? static_cast<int>(blockIdx.x - row_ctas) % csize : 0;
    if constexpr (SPLIT) cg::this_cluster().barrier_arrive();
    if (tid < m.k) {
        s_row[tid] = pair_row(m, t, tid, rank == 0);
        s_w[tid] = p.w[t * m.k + tid];
    }
    float dot[SG > 8 ? 16 : 8];
#pragma unroll
    for (int j = 0; j < (SG > 8 ? 16 : 8); ++j) dot[j] = 0.f;
    __syncthreads();
    const int first = SPLIT ? chunks * rank / csize : 0, nck = SPLIT ? chunks * (rank + 1) / csize : chunks;   // this CTA's
    for (int c0 = first + tid; c0 - tid < nck; c0 += U * blockDim.x) {     // as many turns for every thread
        uint4 v[SG][U];
        float g[U][8];
#pragma unroll
        for (int j = 0; j < SG; ++j) {
            const int row = j < m.k ? s_row[j] : -1;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * blockDim.x;
                if (row >= 0 && c < nck) v[j][u] = ld_stream_u4(p.expert_out + static_cast<int64_t>(row) * p.H + c * 8);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + u * blockDim.x < nck) load_grad<F32>(p.d_out, t * p.H + (c0 + u * blockDim.x) * 8, g[u]);
#pragma unroll
        for (int j = 0; j < SG; ++j) {
            const int row = j < m.k ? s_row[j] : -1;
            if (row < 0) continue;
            const float w = s_w[j];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * blockDim.x;
                if (c >= nck) continue;
                float e[8];
                unpack8(v[j][u], e);
#pragma unroll
                for (int q = 0; q < 8; ++q) dot[j] = fmaf(g[u][q], e[q], dot[j]);
                st_stream_u4(p.d_expert_out + static_cast<int64_t>(row) * p.H + c * 8,
                             make_uint4(pack_bf16x2(w * g[u][0], w * g[u][1]), pack_bf16x2(w * g[u][2], w * g[u][3]),
                                        pack_bf16x2(w * g[u][4], w * g[u][5]), pack_bf16x2(w * g[u][6], w * g[u][7])));
            }
        }
    }
#pragma unroll
    for (int a = 0; a < (SG > 8 ? 2 : 1); ++a) {
        float d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = dot[a * 8 + j];
        const float sum = warp_reduce_scatter8(d, lane);
        if ((lane & 3) == 0) s_part[warp][a * 8 + (lane >> 2)] = sum;
    }
    __syncthreads();
    float total = 0.f;
    if (tid < m.k)
        for (int i = 0; i < warps; ++i) total += s_part[i][tid];
    if constexpr (SPLIT) {
        cg::cluster_group cl = cg::this_cluster();
        cl.barrier_wait();          // the first CTA runs
        if (tid < m.k) cl.map_shared_rank(&s_split[0][0], 0)[rank * kMaxK + tid] = total;
        cl.sync();
        total = 0.f;
        if (rank == 0 && tid < m.k)
            for (int i = 0; i < csize; ++i) total += s_split[i][tid];
    }
    if (rank == 0 && tid < m.k) p.d_w[t * m.k + tid] = total;
}

using GradKernel = void (*)(const FinalizeGradParams, int, int, int);

template <bool F32, bool SPLIT>
GradKernel kernel_for(int k) {
    return k <= 2 ? finalize_grad_kernel<F32, 2, 2, SPLIT> : k <= 4 ? finalize_grad_kernel<F32, 4, 2, SPLIT>
         : k <= 8 ? finalize_grad_kernel<F32, 8, 1, SPLIT> : finalize_grad_kernel<F32, 16, 1, SPLIT>;
}

}  // namespace

cudaError_t finalize_grad_prepare(int k, int fp32) {
    cudaError_t e = preload(fp32 ? kernel_for<true, false>(k) : kernel_for<false, false>(k));
    return e != cudaSuccess ? e : preload(fp32 ? kernel_for<true, true>(k) : kernel_for<false, true>(k));
}

cudaError_t finalize_grad_launch(const FinalizeGradParams& p, int sms, int pdl, cudaStream_t s) {
    const int nck = p.H / 8;
    // A CTA's threads divide a token's chunks evenly: no turn in which a few
    // have one (333 x 2056, 257 chunks: 160 threads twice, 5.2 us; 256 threads,
    // of which one has a second, 6.3).  Where tokens are plenty, smaller CTAs of more
    // turns: the more CTAs an SM holds, the less the phases of each show
    // (16384 x 4096, us by turns: k = 8 2: 340, 4: 335; k = 3 4: 152, 8: 145; k =
    // 16 2: 677, 4: 653), but two warps at least for five rows or more (32768 x
    // 1024, k = 8: one warp 177, two 172).
    int turns = (nck + kThreads - 1) / kThreads;
    const int least = p.m.k <= 4 ? 8 : 4;
    if (p.m.T > 12 * static_cast<int64_t>(sms) && turns < least) turns = least;
    int block = ((nck + turns - 1) / turns + 31) / 32 * 32;
    if (p.m.k > 4 && block < 64 && nck > 32) block = 64;
    // Few tokens of more than two turns: a cluster per token, while its CTAs find
    // an SM each (us with one CTA a token and with the cluster: T = 1, H = 4096
    // 3.4, 3.4; 8192 5.3, 3.4; 16384 9.0, 3.6; T = 38, H = 8192 5.6, 4.3).
    int csize = 1;
    if (nck > 2 * kThreads)
        while (csize < 8 && p.m.T * 2 * csize <= sms) csize *= 2;
    if (csize > 1) {
        const int share = (nck + csize - 1) / csize;
        turns = (share + kThreads - 1) / kThreads;
        block = ((share + turns - 1) / turns + 31) / 32 * 32;
    }
    const int rpw = rows_per_warp(p.m.T, p.m.R, sms);
    const int64_t per = static_cast<int64_t>(block / 32) * rpw;
    const int row_ctas = static_cast<int>((p.m.R + per * csize - 1) / (per * csize)) * csize;
    const GradKernel kernel = csize > 1 ? (p.fp32 ? kernel_for<true, true>(p.m.k) : kernel_for<false, true>(p.m.k))
                                        : (p.fp32 ? kernel_for<true, false>(p.m.k) : kernel_for<false, false>(p.m.k));
    return layer_launch(kernel, row_ctas + p.m.T * csize, block, 0, csize, pdl, s, p, row_ctas, rpw, csize);
}

}  // namespace mfr
