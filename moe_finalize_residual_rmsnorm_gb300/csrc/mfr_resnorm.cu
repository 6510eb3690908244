// Residual addition + RMSNorm with an 8-bit output.
#include <cfloat>

#include "moe_layer_ops.h"
#include "mfr_device.cuh"
#include "mfr_layer.h"

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

// E8M0 byte of the smallest power of two 2^(byte - 127) with amax / 2^.. <= 448 = 1.75 * 2^8,
// for amax in [2^-100, FLT_MAX]: from amax = m * 2^x, 1 <= m < 2, the exponent x - 8, one more where m > 1.75.
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
// warps; chunk c (8 columns) to thread c % nt of its nt threads.
template <int CPT, int QUANT, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarpTokens : 1024) resnorm_kernel(const ResNormParams p) {
    __shared__ float s_sum[32];
    __shared__ float s_max[32];
    const int tid = WARP ? threadIdx.x & 31 : threadIdx.x, nt = WARP ? 32 : blockDim.x, nck = p.H >> 3;
    const int64_t t = WARP ? static_cast<int64_t>(blockIdx.x) * kWarpTokens + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t base = t * p.H;
    pdl_wait();
    pdl_launch_dependents();
    if (WARP && t >= p.T) return;
    float r[CPT][8];
    uint4 g[CPT];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        const int c = tid + i * nt;
        if (c < nck) {
            const uint4 xv = ld_stream_u4(p.x + base + c * 8);
            const float4 a = ld_once_f4(p.residual_in + base + c * 8), b = ld_once_f4(p.residual_in + base + c * 8 + 4);
            g[i] = *reinterpret_cast<const uint4*>(p.gamma + c * 8);
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
    }
    ss = WARP ? warp_allreduce_sum(ss) : block_sum(ss, s_sum);
    const float inv = rsqrtf(ss / static_cast<float>(p.H) + p.eps);
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        const int c = tid + i * nt;
        float gf[8];
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
        if constexpr (QUANT == MFR_QUANT_TOKEN) top = fmaxf(top, amax);
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
        top = fminf(fmaxf(top, kAmaxFloor), FLT_MAX);
        const float enc = kE4m3Max / top;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int c = tid + i * nt;
            if (c < nck) st_u2(p.q + base + c * 8, e4m3x8(r[i], enc));
        }
        if (tid == 0) static_cast<float*>(p.sf)[t] = top / kE4m3Max;
    }
}

template <int CPT, bool WARP>
cudaError_t launch_quant(const ResNormParams& p, int pdl, cudaStream_t s) {
    const int64_t grid = WARP ? (p.T + kWarpTokens - 1) / kWarpTokens : p.T;
    const int threads = ((p.H / 8 + CPT - 1) / CPT + 31) / 32 * 32;
    const int block = WARP ? 32 * kWarpTokens : threads;
    switch (p.quant) {
        case MFR_QUANT_TOKEN: return layer_launch(resnorm_kernel<CPT, MFR_QUANT_TOKEN, WARP>, grid, block, 0, 1, pdl, s, p);
        case MFR_QUANT_GROUP128:
            return layer_launch(resnorm_kernel<CPT, MFR_QUANT_GROUP128, WARP>, grid, block, 0, 1, pdl, s, p);
        case MFR_QUANT_MX32: return layer_launch(resnorm_kernel<CPT, MFR_QUANT_MX32, WARP>, grid, block, 0, 1, pdl, s, p);
        default: return layer_launch(resnorm_kernel<CPT, MFR_QUANT_NONE, WARP>, grid, block, 0, 1, pdl, s, p);
    }
}

}  // namespace

cudaError_t resnorm_launch(const ResNormParams& p, int pdl, cudaStream_t s) {
    if (p.H <= 256) return launch_quant<1, true>(p, pdl, s);
    if (p.H <= 512) return launch_quant<2, true>(p, pdl, s);
#ifdef RN2
    if (p.H > 2048) return launch_quant<2, false>(p, pdl, s);
#endif
    if (p.H <= 8192) return launch_quant<1, false>(p, pdl, s);
    return launch_quant<2, false>(p, pdl, s);
}

}  // namespace mfr
