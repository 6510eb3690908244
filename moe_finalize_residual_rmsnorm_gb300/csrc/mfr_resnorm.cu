// Residual addition + RMSNorm with an 8-bit output:
//
//   r = residual + x,  y = r * rsqrt(mean(r^2) + eps) * gamma,
//   a group's scale from its largest |y|,  q = E4M3(y / scale)
//
// y is quantised from its FP32 value, not from its bf16 rounding, so that each
// code carries one rounding.
//
// One pass over DRAM: a token's r stays on the chip from its sum to its
// output, so bytes bound it (2 + 4 read, 4 + 1 (+ 2) written an element) and
// one CTA per token is enough, as long as several are resident on an SM, each
// in another phase of load, sum and store.  The launch bounds below hold that
// up, at 4 and 20 bytes of spills a thread in the two one-chunk forms with a
// scale per token; CTAs are at most 512 threads of one to four chunks (8 columns).
// Measured on GB300, of the copy rate: 16384 x 4096 107 us (1.03), with bf16
// output and MX scales 127 us (1.02); 8192 x 8192 109 us (1.00; 117 with 1024
// threads of a chunk, 121 with two 512-thread CTAs an SM); 4096 x 16384 119
// us (0.92).
//   three or four chunks (H > 8192): r waits in shared memory, three CTAs an SM
//     (16384 columns: 148 us with r in the registers of 1024 threads, 119 with a
//     ring of stages as in the gradient; 9000 columns: 127 us with three chunks a
//     thread, 150 with four, 150 with the ring)
//   few tokens of wide rows: a cluster of 4 or 8 CTAs per token, which
//     exchange their sums through distributed shared memory (T = 1: H = 4096
//     1.96 -> 1.71 us, 8192 2.98 -> 1.86, 16384 5.24 -> 2.03)
//   H <= 512: a warp per token, no barrier; under 256 columns lanes are idle
//     (of the copy rate at 256, 128 and 64 columns: 0.96, 0.74, 0.42)
#include <cfloat>

#include <cooperative_groups.h>

#include "moe_layer_ops.h"
#include "mfr_device.cuh"
#include "mfr_layer.h"

namespace cg = cooperative_groups;

namespace mfr {
namespace {

constexpr float kAmaxFloor = 0x1p-100f;
constexpr float kE4m3Max = 448.f;
constexpr int kWarpTokens = 8;

// Two E4M3 codes (nearest even, saturating at 448): lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2_rn_sat(float lo, float hi) {
    uint16_t q;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(q) : "f"(hi), "f"(lo));
    return q;
}

__device__ __forceinline__ uint2 e4m3x8(const float (&y)[8], float enc) {
    uint2 q;
    q.x = e4m3x2_rn_sat(y[0] * enc, y[1] * enc) | (e4m3x2_rn_sat(y[2] * enc, y[3] * enc) << 16);
    q.y = e4m3x2_rn_sat(y[4] * enc, y[5] * enc) | (e4m3x2_rn_sat(y[6] * enc, y[7] * enc) << 16);
    return q;
}

__device__ __forceinline__ float max_over(float v, int lanes) {
    for (int off = 1; off < lanes; off <<= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
    return v;
}

// E8M0 byte of the smallest power of two 2^(byte - 127) that brings amax, in
// [2^-100, FLT_MAX], to 448 = 1.75 * 2^8 or below: from amax = m * 2^x, 1 <= m <
// 2, the exponent x - 8, one more where m > 1.75.
__device__ __forceinline__ uint32_t mx_scale_byte(float amax) {
    const uint32_t u = __float_as_uint(amax);
    return (u >> 23) - 8u + ((u & 0x7FFFFFu) > 0x600000u ? 1u : 0u);
}

// Sum over the CTA in a fixed order; every thread gets it.  `s` holds one float per warp.
__device__ __forceinline__ float block_sum(float v, float* s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    v = warp_allreduce_sum(v);
    if (lane == 0) s[warp] = v;
    __syncthreads();
    float sum = 0.f;
    for (int i = 0; i < warps; ++i) sum += s[i];
    return sum;
}

// A token belongs to one CTA, or (WARP) to one warp of a CTA of kWarpTokens
// warps, or (SPLIT) to a cluster of csize CTAs; chunk c (8 columns) to thread
// c % nt of its nt threads (SPLIT: of CTA c / nt).  A group of columns lies in
// consecutive lanes of one warp, 16 or 4 of them.
template <int CPT, int QUANT, bool WARP, bool SPLIT = false>
__global__ void __launch_bounds__(WARP ? 32 * kWarpTokens : 512, WARP ? 1 : CPT == 1 ? 4 : 3)
resnorm_kernel(const ResNormParams p, const int csize) {
    __shared__ float s_sum[32];
    __shared__ float s_max[32];
    __shared__ float s_split[2][16];      // SPLIT: every CTA's sum and largest magnitude
    const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x;
    const int rank = SPLIT ? static_cast<int>(blockIdx.x) % csize : 0;
    const int64_t t = WARP ? static_cast<int64_t>(blockIdx.x) * kWarpTokens + (threadIdx.x >> 5)
                    : SPLIT ? blockIdx.x / csize : blockIdx.x;
    // chunk 0 of this CTA, and the chunks of the row (whole groups of 16 a CTA)
    const int first = SPLIT ? rank * nt : 0, nck = p.H >> 3;
    const int64_t base = t * p.H;
    if constexpr (SPLIT) cg::this_cluster().barrier_arrive();
    pdl_wait();
    pdl_launch_dependents();
    if (WARP && t >= p.T) return;
    // Rows wider than 8192 columns wait for the sum in shared memory: their
    // registers would leave one CTA an SM.
    constexpr bool STASH = !WARP && CPT > 2;
    extern __shared__ float4 stash[];     // [2 CPT][nt]
    float r[CPT][8];
    uint4 g[CPT];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        const int c = first + tid + i * nt;
        if (c < nck) {
            const uint4 xv = ld_stream_u4(p.x + base + c * 8);
            const float4 a = ld_once_f4(p.residual_in + base + c * 8), b = ld_once_f4(p.residual_in + base + c * 8 + 4);
            if constexpr (!STASH) g[i] = *reinterpret_cast<const uint4*>(p.gamma + c * 8);
            unpack8(xv, r[i]);
            r[i][0] += a.x; r[i][1] += a.y; r[i][2] += a.z; r[i][3] += a.w;
            r[i][4] += b.x; r[i][5] += b.y; r[i][6] += b.z; r[i][7] += b.w;
            st_f4(p.residual_out + base + c * 8, make_float4(r[i][0], r[i][1], r[i][2], r[i][3]));
            st_f4(p.residual_out + base + c * 8 + 4, make_float4(r[i][4], r[i][5], r[i][6], r[i][7]));
        } else {
            g[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < 8; ++q) r[i][q] = 0.f;
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) ss = fmaf(r[i][q], r[i][q], ss);
        if constexpr (STASH) {
            stash[(2 * i) * nt + tid] = make_float4(r[i][0], r[i][1], r[i][2], r[i][3]);
            stash[(2 * i + 1) * nt + tid] = make_float4(r[i][4], r[i][5], r[i][6], r[i][7]);
        }
    }
    ss = WARP ? warp_allreduce_sum(ss) : block_sum(ss, s_sum);
    if constexpr (SPLIT) {
        cg::cluster_group cl = cg::this_cluster();
        cl.barrier_wait();                // every CTA of the token runs
        if (tid < csize) cl.map_shared_rank(s_split[0], tid)[rank] = ss;
        cl.sync();
        ss = 0.f;
        for (int i = 0; i < csize; ++i) ss += s_split[0][i];
    }
    const float inv = rsqrtf(ss / static_cast<float>(p.H) + p.eps);
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        const int c = first + tid + i * nt;
        float gf[8];
        if constexpr (STASH) {
            const float4 a = stash[(2 * i) * nt + tid], b = stash[(2 * i + 1) * nt + tid];
            r[i][0] = a.x; r[i][1] = a.y; r[i][2] = a.z; r[i][3] = a.w;
            r[i][4] = b.x; r[i][5] = b.y; r[i][6] = b.z; r[i][7] = b.w;
            g[i] = c < nck ? *reinterpret_cast<const uint4*>(p.gamma + c * 8) : make_uint4(0, 0, 0, 0);
        }
        unpack8(g[i], gf);
        float amax = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            r[i][q] = (c < nck) ? (r[i][q] * inv) * gf[q] : 0.f;
            amax = fmaxf(amax, fabsf(r[i][q]));
        }
        if (c < nck && p.out)
            st_u4(p.out + base + c * 8, make_uint4(pack_bf16x2(r[i][0], r[i][1]), pack_bf16x2(r[i][2], r[i][3]),
                                                   pack_bf16x2(r[i][4], r[i][5]), pack_bf16x2(r[i][6], r[i][7])));
        if constexpr (QUANT == MFR_QUANT_TOKEN) {
            top = fmaxf(top, amax);
            if constexpr (STASH) {
                stash[(2 * i) * nt + tid] = make_float4(r[i][0], r[i][1], r[i][2], r[i][3]);
                stash[(2 * i + 1) * nt + tid] = make_float4(r[i][4], r[i][5], r[i][6], r[i][7]);
            }
        }
        if constexpr (QUANT == MFR_QUANT_GROUP128) {
            amax = fminf(fmaxf(max_over(amax, 16), kAmaxFloor), FLT_MAX);
            if (c < nck) {
                st_u2(p.q + base + c * 8, e4m3x8(r[i], kE4m3Max / amax));
                if ((c & 15) == 0) static_cast<float*>(p.sf)[t * ((p.H + 127) / 128) + (c >> 4)] = amax / kE4m3Max;
            }
        }
        if constexpr (QUANT == MFR_QUANT_MX32) {
            amax = fminf(fmaxf(max_over(amax, 4), kAmaxFloor), FLT_MAX);
            const uint32_t byte = mx_scale_byte(amax);
            if (c < nck) {
                st_u2(p.q + base + c * 8, e4m3x8(r[i], __uint_as_float((254u - byte) << 23)));
                if ((c & 3) == 0)
                    static_cast<uint8_t*>(p.sf)[nvfp4_sf_index(t, c >> 2, (p.H + 31) / 32, p.sf_tiled)] =
                        static_cast<uint8_t>(byte);
            }
        }
    }
    if constexpr (QUANT == MFR_QUANT_TOKEN) {
        top = max_over(top, 32);
        if constexpr (!WARP) {
            if ((tid & 31) == 0) s_max[tid >> 5] = top;
            __syncthreads();
            for (int i = 0; i < nt / 32; ++i) top = fmaxf(top, s_max[i]);
        }
        if constexpr (SPLIT) {
            cg::cluster_group cl = cg::this_cluster();
            if (tid < csize) cl.map_shared_rank(s_split[1], tid)[rank] = top;
            cl.sync();
            for (int i = 0; i < csize; ++i) top = fmaxf(top, s_split[1][i]);
        }
        top = fminf(fmaxf(top, kAmaxFloor), FLT_MAX);
        const float enc = kE4m3Max / top;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int c = first + tid + i * nt;
            if constexpr (STASH) {
                const float4 a = stash[(2 * i) * nt + tid], b = stash[(2 * i + 1) * nt + tid];
                r[i][0] = a.x; r[i][1] = a.y; r[i][2] = a.z; r[i][3] = a.w;
                r[i][4] = b.x; r[i][5] = b.y; r[i][6] = b.z; r[i][7] = b.w;
            }
            if (c < nck) st_u2(p.q + base + c * 8, e4m3x8(r[i], enc));
        }
        if (tid == 0 && rank == 0) static_cast<float*>(p.sf)[t] = top / kE4m3Max;
    }
}

// CTAs per token: 8 or 4 where that many find an SM each and the row is wide
// enough to pay for the exchange (us for T = 1 by CTAs: H = 2048 1: 1.51, 2:
// 1.83; H = 4096 1: 1.96, 4: 1.73, 8: 1.71; T = 38, H = 8192 1: 3.05, 4: 2.42).
int split_ctas(int64_t T, int H, int sms) {
    if (H < 4096) return 1;
    return T * 8 <= sms ? 8 : T * 4 <= sms ? 4 : 1;
}

// A call's kernel and launch geometry.
struct Form {
    void (*kernel)(const ResNormParams, int);
    int64_t grid;
    int block;
    int smem;
    int csize;
};

template <int CPT, bool WARP, bool SPLIT = false>
void (*kernel_for(int quant))(const ResNormParams, int) {
    switch (quant) {
        case MFR_QUANT_TOKEN: return resnorm_kernel<CPT, MFR_QUANT_TOKEN, WARP, SPLIT>;
        case MFR_QUANT_GROUP128: return resnorm_kernel<CPT, MFR_QUANT_GROUP128, WARP, SPLIT>;
        case MFR_QUANT_MX32: return resnorm_kernel<CPT, MFR_QUANT_MX32, WARP, SPLIT>;
        default: return resnorm_kernel<CPT, MFR_QUANT_NONE, WARP, SPLIT>;
    }
}

Form form_for(int64_t T, int H, int quant, int sms) {
    const int nck = H / 8;
    auto threads = [&](int n) { return ((nck + n - 1) / n + 31) / 32 * 32; };     // each with at most n chunks
    const int csize = split_ctas(T, H, sms);
    if (csize > 1) return {kernel_for<1, false, true>(quant), T * csize, threads(csize), 0, csize};
    if (H <= 512) {
        const int64_t grid = (T + kWarpTokens - 1) / kWarpTokens;
        return {H <= 256 ? kernel_for<1, true>(quant) : kernel_for<2, true>(quant), grid, 32 * kWarpTokens, 0, 1};
    }
    if (H <= 4096) return {kernel_for<1, false>(quant), T, threads(1), 0, 1};
    if (H <= 8192) return {kernel_for<2, false>(quant), T, threads(2), 0, 1};
    if (H <= 12288) return {kernel_for<3, false>(quant), T, threads(3), 2 * 3 * 16 * threads(3), 1};
    return {kernel_for<4, false>(quant), T, threads(4), 2 * 4 * 16 * threads(4), 1};
}

}  // namespace

cudaError_t resnorm_prepare(int64_t T, int H, int quant, int sms) {
    const Form f = form_for(T, H, quant, sms);
    const cudaError_t e = preload(f.kernel);
    if (e != cudaSuccess || f.smem == 0) return e;
    // the attribute is per kernel, shared by every plan: always the most any
    // plan needs, which the widest rows of each form do
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(f.kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                2 * (H <= 12288 ? 3 : 4) * 16 * 512);
}

cudaError_t resnorm_launch(const ResNormParams& p, int sms, int pdl, cudaStream_t s) {
    const Form f = form_for(p.T, p.H, p.quant, sms);
    return layer_launch(f.kernel, f.grid, f.block, f.smem, f.csize, pdl, s, p, f.csize);
}

}  // namespace mfr
