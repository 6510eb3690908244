// Residual addition + RMSNorm with an 8-bit output, and its gradient.
#include <cfloat>

#include "moe_layer_ops.h"
#include "mfr_device.cuh"
#include "mfr_layer.h"

namespace mfr {
namespace {

constexpr float kAmaxFloor = 0x1p-100f;
constexpr float kE4m3Max = 448.f;

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

// One CTA per token; chunk c (8 columns) belongs to thread c % blockDim.x.
template <int CPT, int QUANT>
__global__ void __launch_bounds__(1024) resnorm_kernel(const ResNormParams p) {
    __shared__ float s_sum[32];
    __shared__ float s_max[32];
    const int tid = threadIdx.x, nt = blockDim.x, nck = p.H >> 3;
    const int64_t t = blockIdx.x, base = t * p.H;
    pdl_wait();
    pdl_launch_dependents();
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
    const float inv = rsqrtf(block_sum(ss, s_sum) / static_cast<float>(p.H) + p.eps);
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
        if ((tid & 31) == 0) s_max[tid >> 5] = top;
        __syncthreads();
        for (int i = 0; i < nt / 32; ++i) top = fmaxf(top, s_max[i]);
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

template <int CPT>
cudaError_t launch_quant(const ResNormParams& p, int block, int pdl, cudaStream_t s) {
    switch (p.quant) {
        case MFR_QUANT_TOKEN: return layer_launch(resnorm_kernel<CPT, MFR_QUANT_TOKEN>, p.T, block, 0, 1, pdl, s, p);
        case MFR_QUANT_GROUP128: return layer_launch(resnorm_kernel<CPT, MFR_QUANT_GROUP128>, p.T, block, 0, 1, pdl, s, p);
        case MFR_QUANT_MX32: return layer_launch(resnorm_kernel<CPT, MFR_QUANT_MX32>, p.T, block, 0, 1, pdl, s, p);
        default: return layer_launch(resnorm_kernel<CPT, MFR_QUANT_NONE>, p.T, block, 0, 1, pdl, s, p);
    }
}

// ---- gradient ------------------------------------------------------------------------
// Persistent CTAs; a thread owns the same columns of every token, so the
// gamma gradient is a running sum in its registers, written once per CTA.
template <int CPT>
__global__ void __launch_bounds__(1024) resnorm_grad_kernel(const ResNormGradParams p) {
    __shared__ float2 s_sum[2][32];
    const int tid = threadIdx.x, nt = blockDim.x, nck = p.H >> 3;
    const int lane = tid & 31, warp = tid >> 5, warps = nt >> 5;
    float dg[CPT][8];
#pragma unroll
    for (int i = 0; i < CPT; ++i)
#pragma unroll
        for (int q = 0; q < 8; ++q) dg[i][q] = 0.f;
    pdl_wait();
    pdl_launch_dependents();
    int turn = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, turn ^= 1) {
        const int64_t base = t * p.H;
        float r[CPT][8], dy[CPT][8], dres[CPT][8];
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int c = tid + i * nt;
#pragma unroll
            for (int q = 0; q < 8; ++q) r[i][q] = dy[i][q] = dres[i][q] = 0.f;
            if (c < nck) {
                const float4 a = ld_once_f4(p.r + base + c * 8), b = ld_once_f4(p.r + base + c * 8 + 4);
                unpack8(ld_stream_u4(p.d_out + base + c * 8), dy[i]);
                if (p.d_res) {
                    const float4 u = ld_once_f4(p.d_res + base + c * 8), v = ld_once_f4(p.d_res + base + c * 8 + 4);
                    dres[i][0] = u.x; dres[i][1] = u.y; dres[i][2] = u.z; dres[i][3] = u.w;
                    dres[i][4] = v.x; dres[i][5] = v.y; dres[i][6] = v.z; dres[i][7] = v.w;
                }
                float g[8];
                unpack8(*reinterpret_cast<const uint4*>(p.gamma + c * 8), g);
                r[i][0] = a.x; r[i][1] = a.y; r[i][2] = a.z; r[i][3] = a.w;
                r[i][4] = b.x; r[i][5] = b.y; r[i][6] = b.z; r[i][7] = b.w;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    ss = fmaf(r[i][q], r[i][q], ss);
                    dot = fmaf(g[q] * dy[i][q], r[i][q], dot);
                }
            }
        }
        ss = warp_allreduce_sum(ss);
        dot = warp_allreduce_sum(dot);
        if (lane == 0) s_sum[turn][warp] = make_float2(ss, dot);
        __syncthreads();
        ss = dot = 0.f;
        for (int i = 0; i < warps; ++i) {
            ss += s_sum[turn][i].x;
            dot += s_sum[turn][i].y;
        }
        const float n = static_cast<float>(p.H);
        const float inv = rsqrtf(ss / n + p.eps);
        const float back = inv * (dot * inv / n);     // times r * inv: no power of inv that could underflow
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int c = tid + i * nt;
            if (c < nck) {
                float g[8];
                unpack8(*reinterpret_cast<const uint4*>(p.gamma + c * 8), g);
                float d[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float unit = r[i][q] * inv;
                    d[q] = dres[i][q] + (inv * (g[q] * dy[i][q]) - unit * back);
                    dg[i][q] = fmaf(dy[i][q], unit, dg[i][q]);
                }
                st_f4(p.d_in + base + c * 8, make_float4(d[0], d[1], d[2], d[3]));
                st_f4(p.d_in + base + c * 8 + 4, make_float4(d[4], d[5], d[6], d[7]));
                if (p.d_x)
                    st_u4(p.d_x + base + c * 8, make_uint4(pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3]),
                                                           pack_bf16x2(d[4], d[5]), pack_bf16x2(d[6], d[7])));
            }
        }
    }
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        const int c = tid + i * nt;
        if (c < nck) {
            float* out = p.partial + static_cast<int64_t>(blockIdx.x) * p.H + c * 8;
            st_f4(out, make_float4(dg[i][0], dg[i][1], dg[i][2], dg[i][3]));
            st_f4(out + 4, make_float4(dg[i][4], dg[i][5], dg[i][6], dg[i][7]));
        }
    }
}

// Sum of the partial gamma gradients: a CTA owns 32 columns, warp w the rows w, w + 8, ...
constexpr int kSumWarps = 8;
__global__ void __launch_bounds__(32 * kSumWarps) gamma_sum_kernel(const float* partial, int rows, int H, float* d_gamma) {
    __shared__ float s[kSumWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    pdl_wait();
    pdl_launch_dependents();
    float sum = 0.f;
    if (col < H) {
#pragma unroll 8
        for (int i = warp; i < rows; i += kSumWarps) sum += partial[static_cast<int64_t>(i) * H + col];
    }
    s[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && col < H) {
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < kSumWarps; ++i) sum += s[i][lane];
        d_gamma[col] = sum;
    }
}

int chunk_threads(int H, int cpt, int most) {
    const int nck = H / 8;
    const int want = ((nck + cpt - 1) / cpt + 31) / 32 * 32;
    return want < most ? want : most;
}

}  // namespace

cudaError_t resnorm_launch(const ResNormParams& p, int pdl, cudaStream_t s) {
    if (p.H <= 8192) return launch_quant<1>(p, chunk_threads(p.H, 1, 1024), pdl, s);
    return launch_quant<2>(p, chunk_threads(p.H, 2, 1024), pdl, s);
}

int resnorm_grad_partials(int64_t T, int H, int sms) {
    const int64_t most = static_cast<int64_t>(sms) * (H <= 4096 ? 2 : 1);
    return static_cast<int>(T < most ? T : most);
}

cudaError_t resnorm_grad_launch(const ResNormGradParams& p, int sms, int pdl, cudaStream_t s) {
    const int grid = resnorm_grad_partials(p.T, p.H, sms);
    cudaError_t e = cudaSuccess;
    if (grid > 0)
        e = p.H <= 8192 ? layer_launch(resnorm_grad_kernel<1>, grid, chunk_threads(p.H, 1, 1024), 0, 1, pdl, s, p)
                        : layer_launch(resnorm_grad_kernel<2>, grid, chunk_threads(p.H, 2, 1024), 0, 1, pdl, s, p);
    if (e == cudaSuccess)
        e = layer_launch(gamma_sum_kernel, (p.H + 31) / 32, 32 * kSumWarps, 0, 1, pdl, s, p.partial, grid, p.H, p.d_gamma);
    return e;
}

}  // namespace mfr
