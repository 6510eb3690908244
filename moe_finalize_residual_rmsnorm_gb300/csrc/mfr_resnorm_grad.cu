// Gradient of residual addition + RMSNorm.  With unit = r * inv,
// inv = (mean(r^2) + eps)^-1/2, for every token:
//   d_r     = d_res + inv * (gamma * d_out) - unit * inv * mean(gamma * d_out * unit)
//   d_gamma = sum over the tokens of d_out * unit
// (inv^3 of the plain formula is never formed: it leaves the FP32 range for
// rows around 1e13.)  Sums and outputs are FP32; d_x is d_r rounded once to
// bf16, the type of x.
//
// Bytes bound it: 4 + 4 + 2 read and 4 (+ 2) written an element.  Measured on
// GB300, of the copy rate: 8192 x 8192 166 us (0.96; 224 us a token at a time
// without the ring below), 16384 x 4096 160 us (0.99), 32768 x 2048 164 us
// (0.96), 4096 x 16384 164 us (0.97), 32768 x 1024 86 us (0.92); 511 x 4104
// 11.5 us (0.43), of which the second launch is 2.3: its last tile holds 8 columns
// but costs a stage and a wait like a full one, and 511 tokens are four turns
// of 152 CTAs.
//
// Wide rows: persistent CTAs, whose GT consumer threads own the same columns
// of every token, so that d_gamma is a running sum in registers, written once
// per CTA and summed over the CTAs by a second small kernel in a fixed order.
// A token is two sums over its columns and then an output that needs them, so
// a CTA that loads, sums and stores one token after another leaves the memory
// idle between; a producer warp therefore keeps a ring of shared-memory
// stages filled with the next tokens' column tiles by bulk copies, and the
// consumers read a tile twice from shared memory.
// Narrow rows: a warp per token, several CTAs per SM.
#include "moe_layer_ops.h"
#include "mfr_device.cuh"
#include "mfr_layer.h"

namespace mfr {
namespace {

// ---- wide rows ---------------------------------------------------------------------------
// GT consumer threads, four columns of a tile each; NT tiles at most.
template <int GT>
constexpr int tile_cols() { return GT * 4; }
template <int GT>
constexpr int stage_bytes() { return tile_cols<GT>() * (4 + 4 + 2); }   // r, d_res, d_out
constexpr int kRingHeader = 256;                  // the barriers
constexpr int kMaxStages = 11;
// The ring holds the current token's tiles, which are read twice, and `ahead`
// more.  More bytes in flight are slower, not faster: reads then run ahead of
// the writes that share the DRAM.  Measured, times in us by stages in all:
//   H = 8192 (4 tiles of 20 KB, 1 CTA an SM)    5: 192   6: 178   7: 164   8: 178   11: 184
//   H = 4096 (4 tiles of 10 KB, 2 CTAs an SM)   5: 181   6: 167   7: 161   8: 179   11: 186
//   H = 2048 (4 tiles of 5 KB, 4 CTAs an SM)    5: 177   6: 164   7: 177   8: 187   11: 188
//   H = 16384 (8 tiles of 20 KB, 1 CTA an SM)   9: 190  11: 168
template <int GT>
constexpr int stages_ahead() { return GT == 128 ? 2 : 3; }
template <int GT>
int ring_smem(int stages) { return kRingHeader + stages * stage_bytes<GT>(); }

// One side's wait for the other.  When it runs out the CTA's producer stops
// filling, its consumers leave together at the next sum, without their row of
// the partial sums, and MFR_STATUS_TIMEOUT says so.
// LIMITED: the limit is the call's, at 0 none waits (a kernel of its own: as an
// argument of the usual one the limit cost 4096 x 16384 2 %).
template <bool LIMITED>
__device__ __forceinline__ bool ring_wait(const ResNormGradParams& p, uint32_t bar, uint32_t parity) {
    if constexpr (LIMITED) return p.wait_limit > 0 && mbar_wait_bounded(bar, parity, p.wait_limit);
    return mbar_wait(bar, parity);
}

template <int GT, int NT, bool LIMITED>
__global__ void __launch_bounds__(GT + 32, 512 / GT) resnorm_grad_ring(const ResNormGradParams p) {
    constexpr int CB = tile_cols<GT>(), WARPS = GT / 32;
    static_assert(NT + stages_ahead<GT>() <= kMaxStages && 16 * kMaxStages <= kRingHeader, "the barriers fit the header");
    extern __shared__ __align__(128) unsigned char smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem);        // S full, S empty
    unsigned char* ring = smem + kRingHeader;
    __shared__ float2 s_sum[2][WARPS];
    const int tid = threadIdx.x, lane = tid & 31;
    const int H = p.H, ntiles = (H + CB - 1) / CB, S = ntiles + stages_ahead<GT>();
    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_addr(&bars[s]), 1);
            mbar_init(smem_addr(&bars[S + s]), WARPS);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    if (tid >= GT) {
        // ---- producer: lanes 0, 1, 2 copy a tile's r, d_res and d_out ----
        int64_t fill = 0;
        int s = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int64_t t = blockIdx.x; t < p.T && ok; t += gridDim.x) {
            for (int b = 0; b < ntiles; ++b) {
                const bool freed = fill < S || ring_wait<LIMITED>(p, smem_addr(&bars[S + s]), phase ^ 1u);
                if (!__all_sync(0xFFFFFFFFu, freed)) {
                    if (lane == 0) atomicOr(p.status, MFR_STATUS_TIMEOUT);
                    ok = false;
                    break;
                }
                const uint32_t st = smem_addr(ring + s * stage_bytes<GT>());
                const int c0 = b * CB;
                const uint32_t cb = static_cast<uint32_t>(min(CB, H - c0));
                const uint32_t bar = smem_addr(&bars[s]);
                const int64_t at = t * H + c0;
                if (lane == 0) mbar_arrive_expect_tx(bar, cb * (p.d_res ? 10 : 6));
                __syncwarp();
                if (lane == 0) bulk_load(st, p.r + at, cb * 4, bar);
                if (lane == 1 && p.d_res) bulk_load(st + CB * 4, p.d_res + at, cb * 4, bar);
                if (lane == 2) bulk_load(st + CB * 8, p.d_out + at, cb * 2, bar);
                ++fill;
                if (++s == S) { s = 0; phase ^= 1u; }
            }
        }
        // every copy has landed before the CTA exits (they need no one else: the
        // full limit, whatever the ring's)
        if (lane == 0)
            for (int64_t f = fill > S ? fill - S : 0; f < fill; ++f)
                if (!mbar_wait(smem_addr(&bars[f % S]), static_cast<uint32_t>(f / S) & 1u)) {
                    atomicOr(p.status, MFR_STATUS_TIMEOUT);
                    break;
                }
        return;
    }
    // ---- consumers: thread i owns the columns 4 i .. 4 i + 3 of every tile ----
    const int warp = tid >> 5;
    uint2 g[NT];
    float dg[NT][4];
#pragma unroll
    for (int b = 0; b < NT; ++b) {
        const int col = b * CB + tid * 4;
        g[b] = col < H ? *reinterpret_cast<const uint2*>(p.gamma + col) : make_uint2(0, 0);
#pragma unroll
        for (int q = 0; q < 4; ++q) dg[b][q] = 0.f;
    }
    const float n = static_cast<float>(H);
    int s = 0, turn = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, turn ^= 1) {
        const int s0 = s;
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int b = 0; b < NT; ++b) {
            if (b >= ntiles) break;
            ok = ok && ring_wait<LIMITED>(p, smem_addr(&bars[s]), phase);
            const unsigned char* st = ring + s * stage_bytes<GT>();
            if (b * CB + tid * 4 < H) {
                const float4 r = *reinterpret_cast<const float4*>(st + tid * 16);
                const uint2 d = *reinterpret_cast<const uint2*>(st + CB * 8 + tid * 8);
                ss = fmaf(r.x, r.x, ss);
                ss = fmaf(r.y, r.y, ss);
                ss = fmaf(r.z, r.z, ss);
                ss = fmaf(r.w, r.w, ss);
                dot = fmaf(bf16_lo(g[b].x) * bf16_lo(d.x), r.x, dot);
                dot = fmaf(bf16_hi(g[b].x) * bf16_hi(d.x), r.y, dot);
                dot = fmaf(bf16_lo(g[b].y) * bf16_lo(d.y), r.z, dot);
                dot = fmaf(bf16_hi(g[b].y) * bf16_hi(d.y), r.w, dot);
            }
            if (++s == S) { s = 0; phase ^= 1u; }
        }
        ss = warp_allreduce_sum(ss);
        dot = warp_allreduce_sum(dot);
        // a wait that ran out anywhere in the CTA ends it: the sum carries the news
        if (lane == 0) s_sum[turn][warp] = make_float2(ss, dot);
        if (!__all_sync(0xFFFFFFFFu, ok) && lane == 0) atomicOr(p.status, MFR_STATUS_TIMEOUT);
        int all_ok;
        asm volatile("{\n\t.reg .pred q, r;\n\tsetp.ne.u32 q, %1, 0;\n\t"
                     "barrier.cta.red.and.pred r, 1, %2, q;\n\tselp.u32 %0, 1, 0, r;\n\t}"
                     : "=r"(all_ok) : "r"(static_cast<int>(ok)), "n"(GT) : "memory");
        if (!all_ok) return;
        ss = dot = 0.f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) {
            ss += s_sum[turn][i].x;
            dot += s_sum[turn][i].y;
        }
        const float inv = rsqrtf(ss / n + p.eps);
        const float back = inv * (dot * inv / n);
        int s2 = s0;
#pragma unroll
        for (int b = 0; b < NT; ++b) {
            if (b >= ntiles) break;
            const unsigned char* st = ring + s2 * stage_bytes<GT>();
            const int col = b * CB + tid * 4;
            if (col < H) {
                const float4 r = *reinterpret_cast<const float4*>(st + tid * 16);
                const uint2 d = *reinterpret_cast<const uint2*>(st + CB * 8 + tid * 8);
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
                if (p.d_res) a = *reinterpret_cast<const float4*>(st + CB * 4 + tid * 16);
                const float u0 = r.x * inv, u1 = r.y * inv, u2 = r.z * inv, u3 = r.w * inv;
                const float y0 = bf16_lo(d.x), y1 = bf16_hi(d.x), y2 = bf16_lo(d.y), y3 = bf16_hi(d.y);
                a.x += inv * (bf16_lo(g[b].x) * y0) - u0 * back;
                a.y += inv * (bf16_hi(g[b].x) * y1) - u1 * back;
                a.z += inv * (bf16_lo(g[b].y) * y2) - u2 * back;
                a.w += inv * (bf16_hi(g[b].y) * y3) - u3 * back;
                dg[b][0] = fmaf(y0, u0, dg[b][0]);
                dg[b][1] = fmaf(y1, u1, dg[b][1]);
                dg[b][2] = fmaf(y2, u2, dg[b][2]);
                dg[b][3] = fmaf(y3, u3, dg[b][3]);
                st_f4(p.d_in + t * H + col, a);
                if (p.d_x) st_u2(p.d_x + t * H + col, make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w)));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&bars[S + s2]));
            if (++s2 == S) s2 = 0;
        }
    }
#pragma unroll
    for (int b = 0; b < NT; ++b) {
        const int col = b * CB + tid * 4;
        if (col < H)
            st_f4(p.partial + static_cast<int64_t>(blockIdx.x) * H + col, make_float4(dg[b][0], dg[b][1], dg[b][2], dg[b][3]));
    }
}

// ---- narrow rows ------------------------------------------------------------------------------
// A warp per token, lane l owning the chunks (8 columns) l, l + 32, ...
// Measured: 32768 x 512 46 us (0.86 of the copy rate), 32768 x 256 25 us (0.78),
// 65536 x 256 46 us (0.86), 131072 x 128 51 us (0.78), 262144 x 64 85 us (0.47);
// above, the ring is faster (32768 x 1024 85 us, 92 with a warp per token).
constexpr int kNarrowWarps = 8;
constexpr int kNarrowMaxH = 512;

template <int CPT>
__global__ void __launch_bounds__(32 * kNarrowWarps) resnorm_grad_narrow(const ResNormGradParams p) {
    __shared__ float s_dg[kNarrowWarps][CPT * 256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nck = p.H >> 3;
    const float n = static_cast<float>(p.H);
    float dg[CPT][8];
#pragma unroll
    for (int i = 0; i < CPT; ++i)
#pragma unroll
        for (int q = 0; q < 8; ++q) dg[i][q] = 0.f;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t step = static_cast<int64_t>(gridDim.x) * kNarrowWarps;
    // the next token's values are loaded while this one's sums and stores are under way
    float4 nr[CPT][2], na[CPT][2];
    uint4 nd[CPT];
    auto load = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int c = lane + 32 * i;
            const int64_t at = t * p.H + c * 8;
            nr[i][0] = nr[i][1] = na[i][0] = na[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
            nd[i] = make_uint4(0, 0, 0, 0);
            if (t < p.T && c < nck) {
                nr[i][0] = ld_once_f4(p.r + at);
                nr[i][1] = ld_once_f4(p.r + at + 4);
                nd[i] = ld_stream_u4(p.d_out + at);
                if (p.d_res) {
                    na[i][0] = ld_once_f4(p.d_res + at);
                    na[i][1] = ld_once_f4(p.d_res + at + 4);
                }
            }
        }
    };
    int64_t t = static_cast<int64_t>(blockIdx.x) * kNarrowWarps + warp;
    load(t);
    for (; t < p.T; t += step) {
        float r[CPT][8], a[CPT][8];
        uint4 d[CPT];
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const float4 u = nr[i][0], v = nr[i][1], x = na[i][0], w = na[i][1];
            r[i][0] = u.x; r[i][1] = u.y; r[i][2] = u.z; r[i][3] = u.w;
            r[i][4] = v.x; r[i][5] = v.y; r[i][6] = v.z; r[i][7] = v.w;
            a[i][0] = x.x; a[i][1] = x.y; a[i][2] = x.z; a[i][3] = x.w;
            a[i][4] = w.x; a[i][5] = w.y; a[i][6] = w.z; a[i][7] = w.w;
            d[i] = nd[i];
        }
        load(t + step);
        float g[8], y[8];
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int c = lane + 32 * i;
            if (c >= nck) continue;
            unpack8(*reinterpret_cast<const uint4*>(p.gamma + c * 8), g);
            unpack8(d[i], y);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                ss = fmaf(r[i][q], r[i][q], ss);
                dot = fmaf(g[q] * y[q], r[i][q], dot);
            }
        }
        ss = warp_allreduce_sum(ss);
        dot = warp_allreduce_sum(dot);
        const float inv = rsqrtf(ss / n + p.eps);
        const float back = inv * (dot * inv / n);
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int c = lane + 32 * i;
            if (c >= nck) continue;
            unpack8(*reinterpret_cast<const uint4*>(p.gamma + c * 8), g);
            unpack8(d[i], y);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float unit = r[i][q] * inv;
                a[i][q] += inv * (g[q] * y[q]) - unit * back;
                dg[i][q] = fmaf(y[q], unit, dg[i][q]);
            }
            const int64_t at = t * p.H + c * 8;
            st_f4(p.d_in + at, make_float4(a[i][0], a[i][1], a[i][2], a[i][3]));
            st_f4(p.d_in + at + 4, make_float4(a[i][4], a[i][5], a[i][6], a[i][7]));
            if (p.d_x)
                st_u4(p.d_x + at, make_uint4(pack_bf16x2(a[i][0], a[i][1]), pack_bf16x2(a[i][2], a[i][3]),
                                             pack_bf16x2(a[i][4], a[i][5]), pack_bf16x2(a[i][6], a[i][7])));
        }
    }
    // the warps' sums of a column in warp order
#pragma unroll
    for (int i = 0; i < CPT; ++i)
#pragma unroll
        for (int q = 0; q < 8; ++q) s_dg[warp][(lane + 32 * i) * 8 + q] = dg[i][q];
    __syncthreads();
    for (int col = threadIdx.x; col < p.H; col += blockDim.x) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kNarrowWarps; ++w) sum += s_dg[w][col];
        p.partial[static_cast<int64_t>(blockIdx.x) * p.H + col] = sum;
    }
}

// ---- the partial sums of d_gamma ------------------------------------------------------------
// A CTA owns 32 columns, warp w the rows w, w + 32, ..., then a butterfly over the
// warps.  It costs 2.5 to 3 us of a call; small CTAs of 8 columns that wait beside
// the first kernel's took longer (511 x 4104 12.5 us instead of 11.7, 32768 x
// 2048 181 instead of 164).
__global__ void __launch_bounds__(1024) gamma_sum_kernel(const float* partial, int rows, int H, float* d_gamma) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    pdl_wait();
    pdl_launch_dependents();
    float sum = 0.f;
    if (col < H) {
        for (int i0 = warp; i0 < rows; i0 += 32 * 10) {      // ten loads in flight
            float v[10];
#pragma unroll
            for (int i = 0; i < 10; ++i) v[i] = i0 + 32 * i < rows ? partial[static_cast<int64_t>(i0 + 32 * i) * H + col] : 0.f;
#pragma unroll
            for (int i = 0; i < 10; ++i) sum += v[i];
        }
    }
    s[warp][lane] = sum;
    __syncthreads();
    const float v = warp_allreduce_sum(s[lane][warp]);       // column `warp` of the 32
    if (lane == 0 && blockIdx.x * 32 + warp < H) d_gamma[blockIdx.x * 32 + warp] = v;
}

// The kernel for rows of H columns, its threads, shared memory and CTAs per SM.
struct Form {
    void (*kernel)(const ResNormGradParams);
    int threads;
    int smem;
    int per_sm;
    int tokens;   // of a CTA at a time
};

template <int GT, int NT>
Form ring_form(int H, bool limited) {
    const int tiles = (H + tile_cols<GT>() - 1) / tile_cols<GT>();
    return {limited ? resnorm_grad_ring<GT, NT, true> : resnorm_grad_ring<GT, NT, false>, GT + 32, ring_smem<GT>(tiles + stages_ahead<GT>()), 512 / GT, 1};
}

// limited: the call has a wait limit of its own (rows that pass through the ring).
Form form_for(int H, bool limited) {
    if (H <= 256) return {resnorm_grad_narrow<1>, 32 * kNarrowWarps, 0, 3, kNarrowWarps};
    if (H <= kNarrowMaxH) return {resnorm_grad_narrow<2>, 32 * kNarrowWarps, 0, 2, kNarrowWarps};
    if (H <= 2048) return ring_form<128, 4>(H, limited);
    if (H <= 4096) return ring_form<256, 4>(H, limited);
    if (H <= 8192) return ring_form<512, 4>(H, limited);
    return ring_form<512, 8>(H, limited);
}

}  // namespace

cudaError_t resnorm_grad_prepare(int H, bool limited) {
    const Form f = form_for(H, limited);
    cudaError_t e = preload(gamma_sum_kernel);
    if (e == cudaSuccess) e = preload(f.kernel);
    if (e != cudaSuccess || f.smem == 0) return e;
    // the attribute is per kernel, shared by every plan: always the most any
    // plan needs, which the widest rows of each form do
    const int widest = H <= 2048 ? 2048 : H <= 4096 ? 4096 : H <= 8192 ? 8192 : kMaxH;
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(f.kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                form_for(widest, limited).smem);
}

int resnorm_grad_partials(int64_t T, int H, int sms) {
    const Form f = form_for(H, false);
    const int64_t want = (T + f.tokens - 1) / f.tokens, most = static_cast<int64_t>(sms) * f.per_sm;
    return static_cast<int>(want < most ? want : most);
}

cudaError_t resnorm_grad_launch(const ResNormGradParams& p, int sms, int pdl, cudaStream_t s) {
    const Form f = form_for(p.H, p.wait_limit != kWaitCycles);
    const int grid = resnorm_grad_partials(p.T, p.H, sms);
    cudaError_t e = cudaSuccess;
    if (grid > 0) e = layer_launch(f.kernel, grid, f.threads, f.smem, 1, pdl, s, p);
    if (e == cudaSuccess)
        e = layer_launch(gamma_sum_kernel, (p.H + 31) / 32, 1024, 0, 1, pdl, s, p.partial, grid, p.H, p.d_gamma);
    return e;
}

}  // namespace mfr
