// RMSNorm of every query and key head with the position rotation in the same
// pass, and its gradient.  For a head x of D elements at position t:
//
//   n = x * rsqrt(mean(x^2) + eps) * gamma
//   a pair (n_a, n_b) of the first `rotary` elements turns by its angle:
//     out_a = n_a cos - n_b sin,  out_b = n_a sin + n_b cos
//   pairs: (i, i + rotary / 2), or interleaved (2 i, 2 i + 1)
//
// and back, with d turned by the opposite angle:
//   d_x = inv * (gamma d - unit * mean(gamma d * unit)),  unit = x * inv
//   d_gamma = sum over tokens and heads of d * unit
//
// Bytes bound both: every head is read once (the gradient: twice) and written
// once.  A lane holds 16 elements of a head, both members of each of its pairs, so
// that nothing is exchanged but the sums; a head takes 1 to 32 lanes and a warp a
// group of 32 to 1 heads of one token.  A warp's unit of work is a run of groups of one
// token, whose cosines and sines stay in registers, and it has several groups' loads in
// flight (four, the gradient two): with one ahead, an iteration was as long as a
// load.  Queries and keys belong to different CTAs, so that a lane's gamma and its
// running sum of d_gamma stay where they are.
#include "moe_step_ops.h"
#include "mfr_device.cuh"
#include "mfr_layer.h"
#include "mfr_step.h"

namespace mfr {
namespace {

constexpr int kQkWarps = 8;

template <bool F16>
__device__ __forceinline__ void widen(uint4 v, float* f) {
    if constexpr (F16) {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            f[2 * i] = x.x;
            f[2 * i + 1] = x.y;
        }
    } else {
        f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
        f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
    }
}

template <bool F16>
__device__ __forceinline__ uint32_t narrow2(float a, float b) {
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        return pack_bf16x2(a, b);
    }
}

template <bool F16>
__device__ __forceinline__ uint4 narrow(const float* f) {
    return make_uint4(narrow2<F16>(f[0], f[1]), narrow2<F16>(f[2], f[3]), narrow2<F16>(f[4], f[5]), narrow2<F16>(f[6], f[7]));
}

// Which elements of a head a lane holds: eight from `a` and eight from `b` (-1: none).
struct Place {
    int a, b;
    bool turns;       // both halves belong to pairs; cosines and sines 8 u and on
    int u;
};

__device__ __forceinline__ Place place_of(int u, int D, int rotary, bool interleaved) {
    Place p;
    const int turning = rotary / 16, chunks = D / 8;
    p.u = u;
    p.turns = u < turning;
    int a, b;
    if (p.turns && !interleaved) {
        a = u;
        b = u + turning;
    } else {
        a = 2 * u;
        b = 2 * u + 1;
    }
    p.a = a < chunks ? a * 8 : -1;
    p.b = b < chunks ? b * 8 : -1;
    return p;
}

// The pairs of x turned by the angles, or back.
template <bool BACK, bool PAIRED>
__device__ __forceinline__ void turn(float (&x)[16], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int ia = PAIRED ? 2 * i : i, ib = PAIRED ? 2 * i + 1 : i + 8;
        const float sn = BACK ? -s[i] : s[i], a = x[ia], b = x[ib];
        x[ia] = a * c[i] - b * sn;
        x[ib] = a * sn + b * c[i];
    }
}

template <int L>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

// Units of work: CTA b < blocks_q has queries' units, the others keys'.  A group is HPW =
// 32 / L heads; a token's per_token groups are `slices` runs of `run` groups, and
// unit u is run u % slices of token u / slices.  A warp takes every stride-th unit.
struct QkRuns {
    int blocks_q;
    int run[2];
    int per_token[2];
    int slices[2];
    int64_t stride[2];
};

// PAIRED: pairs (2 i, 2 i + 1).
template <bool F16, int L, bool GRAD, bool PAIRED>
__global__ void __launch_bounds__(32 * kQkWarps, GRAD ? 2 : 3) qk_kernel(const QkParams p, const QkRuns r) {
    constexpr int HPW = 32 / L;
    constexpr int BATCH = GRAD ? 2 : 4;       // groups whose loads are in flight
    __shared__ float s_gamma[GRAD ? kQkWarps : 1][GRAD ? 16 * L : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int which = static_cast<int>(blockIdx.x) < r.blocks_q ? 0 : 1;
    const QkSide& side = p.side[which];
    const int per = r.per_token[which], slices = r.slices[which], run = r.run[which];
    const int64_t units = p.T * slices;
    const Place pl = place_of(lane % L, p.D, p.rotary, PAIRED);
    const float per_element = 1.f / static_cast<float>(p.D);
    pdl_wait();
    pdl_launch_dependents();
    float sum[GRAD ? 16 : 1];
    const uint4 none = make_uint4(0, 0, 0, 0);
    const uint4 gamma_a = pl.a >= 0 ? *reinterpret_cast<const uint4*>(side.gamma + pl.a) : none;
    const uint4 gamma_b = pl.b >= 0 ? *reinterpret_cast<const uint4*>(side.gamma + pl.b) : none;
    if constexpr (GRAD)
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[i] = 0.f;
    for (int64_t unit = (blockIdx.x - (which ? r.blocks_q : 0)) * int64_t(kQkWarps) + warp; unit < units; unit += r.stride[which]) {
        const int64_t t = unit / slices;
        const int g0 = static_cast<int>(unit - t * slices) * run, g1 = min(g0 + run, per);
        const int pos = p.positions[t];
        const uint16_t* xs = side.x + t * side.x_token;
        const uint16_t* ds = GRAD ? side.d_out + t * side.d_token : nullptr;
        float c[8], s[8];
        bool known = false, good = false;
        for (int g = g0; g < g1; g += BATCH) {
            uint4 xa[BATCH], xb[BATCH], da[GRAD ? BATCH : 1], db[GRAD ? BATCH : 1];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const int head = (g + i) * HPW + lane / L;
                const bool on = g + i < g1 && head < side.heads;
                const uint16_t* x = xs + head * side.x_head;
                xa[i] = ld_stream_u4_if(x + pl.a, on && pl.a >= 0);
                xb[i] = ld_stream_u4_if(x + pl.b, on && pl.b >= 0);
                if constexpr (GRAD) {
                    const uint16_t* d = ds + head * side.d_head;
                    da[i] = ld_stream_u4_if(d + pl.a, on && pl.a >= 0);
                    db[i] = ld_stream_u4_if(d + pl.b, on && pl.b >= 0);
                }
            }
            if (!known) {
                known = true;
                good = static_cast<uint32_t>(pos) < static_cast<uint32_t>(p.max_positions);
                if (!good && lane == 0) atomicOr(p.status, MFR_STATUS_BAD_INDEX);
                const float4* row = reinterpret_cast<const float4*>(p.table + static_cast<int64_t>(pos) * p.rotary + 8 * pl.u);
                const bool on = good && pl.turns;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 a = on ? __ldg(row + i) : make_float4(1.f, 1.f, 1.f, 1.f);
                    const float4 b = on ? __ldg(row + p.rotary / 8 + i) : make_float4(0.f, 0.f, 0.f, 0.f);
                    c[4 * i] = a.x; c[4 * i + 1] = a.y; c[4 * i + 2] = a.z; c[4 * i + 3] = a.w;
                    s[4 * i] = b.x; s[4 * i + 1] = b.y; s[4 * i + 2] = b.z; s[4 * i + 3] = b.w;
                }
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                if (g + i >= g1) break;
                const int head = (g + i) * HPW + lane / L;
                float x[16], gamma[16];
                widen<F16>(gamma_a, gamma);
                widen<F16>(gamma_b, gamma + 8);
                widen<F16>(xa[i], x);
                widen<F16>(xb[i], x + 8);
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
                const float inv = rsqrtf(fmaf(head_sum<L>(ss), per_element, p.eps));
                if constexpr (!GRAD) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = x[e] * inv * gamma[e];
                    if (pl.turns) turn<false, PAIRED>(x, c, s);
                } else {
                    float d[16];
                    widen<F16>(da[i], d);
                    widen<F16>(db[i], d + 8);
                    if (pl.turns) turn<true, PAIRED>(d, c, s);
                    float dot = 0.f;
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        x[e] *= inv;                                  // unit
                        if (good) sum[e] = fmaf(d[e], x[e], sum[e]);
                        d[e] *= gamma[e];
                        dot = fmaf(d[e], x[e], dot);
                    }
                    const float mean = head_sum<L>(dot) * per_element;
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = inv * (d[e] - x[e] * mean);
                }
                if (good && head < side.heads) {
                    uint16_t* o = side.out + t * side.out_token + head * side.out_head;
                    if (pl.a >= 0) st_stream_u4(o + pl.a, narrow<F16>(x));
                    if (pl.b >= 0) st_stream_u4(o + pl.b, narrow<F16>(x + 8));
                }
            }
        }
    }
    if constexpr (GRAD) {
        // this warp's heads, then the CTA's warps, in a fixed order
#pragma unroll
        for (int i = 0; i < 16; ++i) {
#pragma unroll
            for (int off = L; off < 32; off <<= 1) sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], off);
            if (lane < L) s_gamma[warp][i * L + lane] = sum[i];
        }
        __syncthreads();
        for (int j = threadIdx.x; j < 16 * L; j += 32 * kQkWarps) {
            const int i = j / L;
            const Place q = place_of(j % L, p.D, p.rotary, PAIRED);
            const int at = i < 8 ? q.a : q.b;
            if (at < 0) continue;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kQkWarps; ++w) v += s_gamma[w][j];
            p.partial[static_cast<int64_t>(blockIdx.x) * p.D + at + (i & 7)] = v;
        }
    }
}

// d_gamma from the CTAs' partial sums: a CTA for 32 columns of one side.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps) qk_gamma_kernel(const QkParams p, const QkRuns r, int blocks) {
    __shared__ float s_sum[kSumWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tiles = (p.D + 31) / 32;
    const int which = static_cast<int>(blockIdx.x) / tiles, col = static_cast<int>(blockIdx.x) % tiles * 32 + lane;
    pdl_wait();
    pdl_launch_dependents();
    const int first = which ? r.blocks_q : 0, last = which ? blocks : r.blocks_q;
    float v[4] = {0.f, 0.f, 0.f, 0.f};                // four rows in flight
    if (col < p.D)
        for (int b = first + warp; b < last; b += 4 * kSumWarps)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (b + i * kSumWarps < last) v[i] += __ldcg(p.partial + static_cast<int64_t>(b + i * kSumWarps) * p.D + col);
    s_sum[warp][lane] = (v[0] + v[1]) + (v[2] + v[3]);
    __syncthreads();
    if (warp == 0 && col < p.D) {
        float total = 0.f;
        for (int w = 0; w < kSumWarps; ++w) total += s_sum[w][lane];
        p.side[which].d_gamma[col] = total;
    }
}

using Kernel = void (*)(const QkParams, const QkRuns);

int lanes_for(int D) {
    int l = 1;
    while (l * 16 < D) l *= 2;
    return l;
}

template <bool F16, bool GRAD, bool PAIRED>
Kernel kernel_of(int D) {
    switch (lanes_for(D)) {
        case 1: return qk_kernel<F16, 1, GRAD, PAIRED>;
        case 2: return qk_kernel<F16, 2, GRAD, PAIRED>;
        case 4: return qk_kernel<F16, 4, GRAD, PAIRED>;
        case 8: return qk_kernel<F16, 8, GRAD, PAIRED>;
        case 16: return qk_kernel<F16, 16, GRAD, PAIRED>;
        default: return qk_kernel<F16, 32, GRAD, PAIRED>;
    }
}

template <bool GRAD>
Kernel kernel_of(const QkShape& s) {
    if (s.fp16) return s.interleaved ? kernel_of<true, GRAD, true>(s.D) : kernel_of<true, GRAD, false>(s.D);
    return s.interleaved ? kernel_of<false, GRAD, true>(s.D) : kernel_of<false, GRAD, false>(s.D);
}

Kernel kernel_for(const QkShape& s, bool grad) { return grad ? kernel_of<true>(s) : kernel_of<false>(s); }

// A warp's run is a token's groups where tokens are many, fewer where that leaves
// SMs without work.  The gradient's warps stay for several units, two CTAs an SM, so
// that there are few partial sums of d_gamma.
QkRuns runs_for(const QkShape& s, int64_t T, bool grad, int sms, int* blocks) {
    const int hpw = 32 / lanes_for(s.D), heads[2] = {s.heads_q, s.heads_k};
    QkRuns r;
    int64_t units[2];
    for (int i = 0; i < 2; ++i) {
        const int per = (heads[i] + hpw - 1) / hpw;
        int run = per < 16 ? per : 16;
        while (run > 1 && T * ((per + run - 1) / run) < static_cast<int64_t>(sms) * 8) run = (run + 1) / 2;
        r.per_token[i] = per;
        r.run[i] = run;
        r.slices[i] = (per + run - 1) / run;
        units[i] = T * r.slices[i];
    }
    const int64_t all = units[0] * r.run[0] + units[1] * r.run[1], most = static_cast<int64_t>(sms) * 2;
    int64_t b[2];
    for (int i = 0; i < 2; ++i) {
        b[i] = (units[i] + kQkWarps - 1) / kQkWarps;
        if (grad && all > 0) {
            // shares of the CTAs in the proportion of the work
            int64_t share = most * (units[i] * r.run[i]) / all;
            if (share < 1) share = 1;
            if (b[i] > share) b[i] = share;
        }
        r.stride[i] = b[i] * kQkWarps;
    }
    r.blocks_q = static_cast<int>(b[0]);
    *blocks = static_cast<int>(b[0] + b[1]);
    return r;
}

}  // namespace

cudaError_t qk_prepare(const QkShape& s) {
    cudaError_t e = preload(kernel_for(s, false));
    if (e == cudaSuccess) e = preload(kernel_for(s, true));
    if (e == cudaSuccess) e = preload(qk_gamma_kernel);
    return e;
}

int qk_grad_partials(const QkShape& s, int64_t T, int sms) {
    int blocks;
    runs_for(s, T, true, sms, &blocks);
    return blocks;
}

cudaError_t qk_launch(const QkShape& s, const QkParams& p, bool grad, int sms, int pdl, cudaStream_t st) {
    int blocks;
    const QkRuns r = runs_for(s, p.T, grad, sms, &blocks);
    cudaError_t e = cudaSuccess;
    if (blocks > 0) e = layer_launch(kernel_for(s, grad), blocks, 32 * kQkWarps, 0, 1, pdl, st, p, r);
    if (e == cudaSuccess && grad)
        e = layer_launch(qk_gamma_kernel, 2 * ((s.D + 31) / 32), 32 * kSumWarps, 0, 1, pdl, st, p, r, blocks);
    return e;
}

}  // namespace mfr
