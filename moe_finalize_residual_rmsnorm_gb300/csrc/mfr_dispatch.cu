// Dispatch: the rows of x copied into expert order.
//
//   rows_out[permuted_row_of[t, j], :] = x[t, :]   for the pairs (t, j) that have a row
//
// A pure copy: it reads each token's row once and writes it k times, so DRAM
// writes bound it.  The work is split by token, not by output row: by row
// each token's row would be read k times at unrelated moments, which at 134
// MB of tokens no longer comes from L2.  One warp holds a segment of a row in
// registers and stores it to the k rows; nothing waits on anything but the
// map entries, whose two dependent loads (the row, then the row's pair) run
// behind the segment's own loads.
//
// Measured on GB300 at 16384 x 4096 bf16 rows, k = 8, blocks padded to 128
// rows (1.27 GB): 190 us, the copy rate of half reads and half writes (a plain
// fill of as many bytes runs at 0.6 of it); 4096 x 8192 8-bit rows with scales
// 44.7 us (0.92).  Copies through shared memory (a bulk load and k bulk stores a
// segment, 4 or 8 warps with 2 or 3 stages) took 6 % longer; stores that keep
// L1 lines 7 % longer at 4096 x 8192 bytes.
#include "mfr_maps.cuh"

namespace mfr {
namespace {

constexpr int kThreads = 256;

// A token's row of scales to the rows of its pairs, by one warp: lane j < k
// holds the row of pair j.  Word is the unit the row divides into.
template <typename Word>
__device__ __forceinline__ void copy_scales(const DispatchParams& p, int64_t t, int row, int lane) {
    const int words = p.sf_bytes / static_cast<int>(sizeof(Word));
    const Word* src = reinterpret_cast<const Word*>(p.sf) + t * words;
    for (int c0 = 0; c0 < words; c0 += 32) {
        const int c = c0 + lane;
        const Word v = c < words ? src[c] : Word(0);
        for (int j = 0; j < p.m.k; ++j) {
            const int r = __shfl_sync(0xFFFFFFFFu, row, j);
            if (r >= 0 && c < words) reinterpret_cast<Word*>(p.sf_out)[static_cast<int64_t>(r) * words + c] = v;
        }
    }
}

// One warp per (token, segment of C * 32 chunks of 16 bytes), behind the warps
// that look after the rows' side of the maps, `rpw` rows each.  Segments of 2
// KB where the call fills the GPU, fewer map reads a byte, else of 512 bytes.
// Measured with segments of 512 bytes, 1, 2 and 4 KB: 16384 x 4096 in blocks of 128
// 187, 188, 190, 192 us, 4096 x 8192 8-bit rows with scales 43.8, 44.2, 44.8,
// 46.3; so where the rows' warps come first, 512 bytes would do for every
// call (with them last: 208, 204, 208, 207 us).
template <int C>
__global__ void __launch_bounds__(kThreads) dispatch_kernel(const DispatchParams p, const int segs, const int64_t row_warps,
                                                            const int rpw) {
    const int lane = threadIdx.x & 31;
    int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const MapParams& m = p.m;
    const int nck = p.row_bytes >> 4;
    pdl_wait();
    pdl_launch_dependents();
    if (warp < row_warps) {
        const int64_t r0 = warp * rpw;
        const bool pad = lane < rpw && r0 + lane < m.R && row_is_padding(m, r0 + lane);
        for (uint32_t todo = __ballot_sync(0xFFFFFFFFu, pad); todo; todo &= todo - 1) {
            const int64_t r = r0 + __ffs(todo) - 1;
            for (int c = lane; c < nck; c += 32) st_stream_u4(p.out + r * p.row_bytes + c * 16, make_uint4(0, 0, 0, 0));
            for (int c = lane; c < p.sf_bytes; c += 32) p.sf_out[r * p.sf_bytes + c] = 0;
        }
        return;
    }
    warp -= row_warps;
    if (warp >= m.T * segs) return;
    const int64_t t = warp / segs;
    const int seg = static_cast<int>(warp - t * segs);
    const int c0 = seg * C * 32 + lane;
    const uint8_t* src = p.x + t * p.row_bytes;
    uint4 v[C];
#pragma unroll
    for (int i = 0; i < C; ++i)
        v[i] = c0 + 32 * i < nck ? ld_stream_u4(src + (c0 + 32 * i) * 16) : make_uint4(0, 0, 0, 0);
    const int row = lane < m.k ? pair_row(m, t, lane, seg == 0) : -1;
    for (int j = 0; j < m.k; ++j) {
        const int r = __shfl_sync(0xFFFFFFFFu, row, j);
        if (r < 0) continue;
        uint8_t* dst = p.out + static_cast<int64_t>(r) * p.row_bytes;
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (c0 + 32 * i < nck) st_stream_u4(dst + (c0 + 32 * i) * 16, v[i]);
    }
    if (p.sf_bytes > 0 && seg == segs - 1) {
        if (p.sf_bytes % 4 == 0) copy_scales<uint32_t>(p, t, row, lane);
        else copy_scales<uint8_t>(p, t, row, lane);
    }
}

// ---- the gradient ---------------------------------------------------------------------
// d_x[t, :] = bf16( sum_j d_rows[permuted_row_of[t, j], :] ), summed in FP32 in
// slot order and rounded once, to the type of the rows.  Reads k rows and writes
// one a token, nothing else: bytes bound it.  One warp per (token, segment of C *
// 32 chunks), SG rows' loads in flight.  Measured on GB300: 4097 x 8192, k = 8
// 90.7 us (0.98 of the copy rate; the persistent ring kernel of the finalize
// with unit weights took 94.5), 24651 x 1328, k = 5 63 us (0.92; 116).  The
// loads are predicated, not branched over: in branches they went one by one
// (101 us).
template <int SG, int C>
__global__ void __launch_bounds__(kThreads) dispatch_grad_kernel(const DispatchGradParams p, const int segs) {
    const int lane = threadIdx.x & 31;
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const MapParams& m = p.m;
    const int nck = p.H >> 3;
    pdl_wait();
    pdl_launch_dependents();
    if (warp >= m.T * segs) return;
    const int64_t t = warp / segs;
    const int seg = static_cast<int>(warp - t * segs);
    const int c0 = seg * C * 32 + lane;
    int row = lane < m.k ? m.row_of[t * m.k + lane] : -1;
    if (static_cast<int64_t>(row) >= m.R || row < 0) {
        if (lane < m.k && seg == 0 && !(m.sentinel && row < 0)) atomicOr(m.status, MFR_STATUS_BAD_INDEX);
        row = -1;
    }
    float acc[C][8];
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[i][q] = 0.f;
#pragma unroll 1
    for (int j0 = 0; j0 < m.k; j0 += SG) {
        uint4 v[SG][C];
#pragma unroll
        for (int j = 0; j < SG; ++j) {
            const int r = __shfl_sync(0xFFFFFFFFu, row, (j0 + j) & 31);      // lanes past the slots hold -1
#pragma unroll
            for (int i = 0; i < C; ++i)
                v[j][i] = ld_stream_u4_if(p.d_rows + static_cast<int64_t>(r) * p.H + (c0 + 32 * i) * 8,
                                          r >= 0 && c0 + 32 * i < nck);
        }
#pragma unroll
        for (int j = 0; j < SG; ++j)
#pragma unroll
            for (int i = 0; i < C; ++i) {
                float e[8];
                unpack8(v[j][i], e);
#pragma unroll
                for (int q = 0; q < 8; ++q) acc[i][q] += e[q];
            }
    }
#pragma unroll
    for (int i = 0; i < C; ++i)
        if (c0 + 32 * i < nck)
            st_u4(p.d_x + t * p.H + (c0 + 32 * i) * 8,
                  make_uint4(pack_bf16x2(acc[i][0], acc[i][1]), pack_bf16x2(acc[i][2], acc[i][3]),
                             pack_bf16x2(acc[i][4], acc[i][5]), pack_bf16x2(acc[i][6], acc[i][7])));
}

using DispatchGradKernel = void (*)(const DispatchGradParams, int);
DispatchGradKernel grad_kernel_for(int k) {
    return k <= 2 ? dispatch_grad_kernel<2, 2> : k <= 4 ? dispatch_grad_kernel<4, 2>
         : k <= 6 ? dispatch_grad_kernel<6, 1> : dispatch_grad_kernel<8, 1>;
}

}  // namespace

cudaError_t dispatch_prepare() {
    cudaError_t e = preload(dispatch_kernel<4>);
    if (e == cudaSuccess) e = preload(dispatch_kernel<1>);
    for (int k = 1; k <= kMaxK && e == cudaSuccess; ++k) e = preload(grad_kernel_for(k));
    return e;
}

cudaError_t dispatch_grad_launch(const DispatchGradParams& p, int pdl, cudaStream_t s) {
    const int nck = p.H / 8;
    // as many loads as there are slots, at least four: two chunks a lane of few slots
    const int c = p.m.k <= 4 ? 2 : 1;
    const int segs = (nck + 32 * c - 1) / (32 * c);
    const int64_t grid = (p.m.T * segs + kThreads / 32 - 1) / (kThreads / 32);
    return layer_launch(grad_kernel_for(p.m.k), grid, kThreads, 0, 1, pdl, s, p, segs);
}

cudaError_t dispatch_launch(const DispatchParams& p, int sms, int pdl, cudaStream_t s) {
    const int nck = p.row_bytes / 16;
    const bool wide = fills_gpu(p.m.T * nck, sms);
    const int rpw = rows_per_warp(p.m.T, p.m.R, sms);
    const int chunks = wide ? 128 : 32;
    const int segs = (nck + chunks - 1) / chunks;
    const int64_t row_warps = (p.m.R + rpw - 1) / rpw;
    const int64_t grid = (row_warps + p.m.T * segs + kThreads / 32 - 1) / (kThreads / 32);
    return wide ? layer_launch(dispatch_kernel<4>, grid, kThreads, 0, 1, pdl, s, p, segs, row_warps, rpw)
                : layer_launch(dispatch_kernel<1>, grid, kThreads, 0, 1, pdl, s, p, segs, row_warps, rpw);
}

}  // namespace mfr
