// Dispatch: the rows of x copied into expert order.
#include "mfr_maps.cuh"

namespace mfr {
namespace {

constexpr int kDispatchThreads = 256;
constexpr int kRowsPerWarp = 32;      // rows whose padding one warp looks after

__device__ __forceinline__ void copy_small(const uint8_t* src, uint8_t* dst, int bytes, int i, int n) {
    if (bytes % 4 == 0) {
        for (int c = i; c < bytes / 4; c += n)
            reinterpret_cast<uint32_t*>(dst)[c] = reinterpret_cast<const uint32_t*>(src)[c];
    } else {
        for (int c = i; c < bytes; c += n) dst[c] = src[c];
    }
}

// One warp per (token, column segment); the warps behind the pairs' warps look
// after the rows' side of the maps.
__global__ void __launch_bounds__(kDispatchThreads) dispatch_kernel(const DispatchParams p, const int segs,
                                                                    const int seg_chunks) {
    const int lane = threadIdx.x & 31;
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const MapParams& m = p.m;
    const int nck = p.row_bytes >> 4;
    pdl_wait();
    pdl_launch_dependents();
    if (warp < m.T * segs) {
        const int64_t t = warp / segs;
        const int seg = static_cast<int>(warp - t * segs);
        const int c0 = seg * seg_chunks, c1 = min(nck, c0 + seg_chunks);
        const uint8_t* src = p.x + t * p.row_bytes;
        const int row = lane < m.k ? pair_row(m, t, lane, seg == 0) : -1;
        for (int c = c0 + lane; c - lane < c1; c += 32) {
            const bool mine = c < c1;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (mine) v = ld_stream_u4(src + static_cast<int64_t>(c) * 16);
            for (int j = 0; j < m.k; ++j) {
                const int r = __shfl_sync(0xFFFFFFFFu, row, j);
                if (r >= 0 && mine) st_u4(p.out + static_cast<int64_t>(r) * p.row_bytes + static_cast<int64_t>(c) * 16, v);
            }
        }
        if (p.sf_bytes > 0 && seg == segs - 1) {
            for (int j = 0; j < m.k; ++j) {
                const int r = __shfl_sync(0xFFFFFFFFu, row, j);
                if (r >= 0)
                    copy_small(p.sf + t * p.sf_bytes, p.sf_out + static_cast<int64_t>(r) * p.sf_bytes, p.sf_bytes, lane, 32);
            }
        }
        return;
    }
    const int64_t r0 = (warp - m.T * segs) * kRowsPerWarp;
    if (r0 >= m.R) return;
    const bool pad = r0 + lane < m.R && row_is_padding(m, r0 + lane);
    for (uint32_t todo = __ballot_sync(0xFFFFFFFFu, pad); todo; todo &= todo - 1) {
        const int64_t r = r0 + __ffs(todo) - 1;
        for (int c = lane; c < nck; c += 32) st_u4(p.out + r * p.row_bytes + static_cast<int64_t>(c) * 16, make_uint4(0, 0, 0, 0));
        for (int c = lane; c < p.sf_bytes; c += 32) p.sf_out[r * p.sf_bytes + c] = 0;
    }
}

__global__ void fill_ones_kernel(float* w, int64_t n) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x)
        w[i] = 1.f;
}

}  // namespace

cudaError_t fill_ones_launch(float* w, int64_t n) {
    return layer_launch(fill_ones_kernel, 256, 256, 0, 1, 0, nullptr, w, n);
}

cudaError_t dispatch_launch(const DispatchParams& p, int sms, int pdl, cudaStream_t s) {
    const int nck = p.row_bytes / 16;
    int seg_chunks = nck;
    if (seg_chunks > 128) seg_chunks = 128;
    const int segs = (nck + seg_chunks - 1) / seg_chunks;
    const int64_t warps = p.m.T * segs + (p.m.R + kRowsPerWarp - 1) / kRowsPerWarp;
    const int wpb = kDispatchThreads / 32;
    (void)sms;
    return layer_launch(dispatch_kernel, (warps + wpb - 1) / wpb, kDispatchThreads, 0, 1, pdl, s, p, segs, seg_chunks);
}

}  // namespace mfr
