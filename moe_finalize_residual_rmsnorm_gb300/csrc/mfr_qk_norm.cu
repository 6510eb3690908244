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
// that nothing is exchanged but the sums; a head takes 1 to 32 lanes and a
// warp 32 to 1 heads of one token.  A warp works on a run of such groups of heads,
// token after token, with the next group's loads in flight and a token's cosines
// and sines in registers while it lasts.  Queries and keys are runs of different
// CTAs, so that a lane's gamma and its running sum of d_gamma stay where they are.
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
template <bool BACK>
__device__ __forceinline__ void turn(float (&x)[16], const float (&c)[8], const float (&s)[8], bool interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float sn = BACK ? -s[i] : s[i];
        if (interleaved) {
            const float a = x[2 * i], b = x[2 * i + 1];
            x[2 * i] = a * c[i] - b * sn;
            x[2 * i + 1] = a * sn + b * c[i];
        } else {
            const float a = x[i], b = x[i + 8];
            x[i] = a * c[i] - b * sn;
            x[i + 8] = a * sn + b * c[i];
        }
    }
}

template <int L>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

// Runs of groups: CTA b < blocks_q has queries' groups, the others keys'.  A group is
// HPW = 32 / L heads of one token, group g of a side belongs to token g / per_token.
struct QkRuns {
    int blocks_q;
    int run[2];             // groups a warp
    int per_token[2];
};

template <bool F16, int L, bool GRAD>
__global__ void __launch_bounds__(32 * kQkWarps) qk_kernel(const QkParams p, const QkRuns r) {
    constexpr int HPW = 32 / L;
    __shared__ float s_gamma[GRAD ? kQkWarps : 1][GRAD ? 16 * L : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int which = static_cast<int>(blockIdx.x) < r.blocks_q ? 0 : 1;
    const QkSide& side = p.side[which];
    const int64_t block = blockIdx.x - (which ? r.blocks_q : 0);
    const int per = r.per_token[which];
    const int64_t groups = p.T * per;
    const int64_t g0 = (block * kQkWarps + warp) * r.run[which];
    const int64_t g1 = g0 + r.run[which] < groups ? g0 + r.run[which] : groups;
    const Place pl = place_of(lane % L, p.D, p.rotary, p.interleaved != 0);
    const bool interleaved = p.interleaved != 0;
    pdl_wait();
    pdl_launch_dependents();
    float gamma[16], sum[GRAD ? 16 : 1];
    const uint4 none = make_uint4(0, 0, 0, 0);
    widen<F16>(pl.a >= 0 ? *reinterpret_cast<const uint4*>(side.gamma + pl.a) : none, gamma);
    widen<F16>(pl.b >= 0 ? *reinterpret_cast<const uint4*>(side.gamma + pl.b) : none, gamma + 8);
    if constexpr (GRAD)
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[i] = 0.f;
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) { c[i] = 1.f; s[i] = 0.f; }
    int64_t t = per > 0 ? g0 / per : 0;
    int in_token = static_cast<int>(g0 - t * per);
    bool known = false;                       // c and s are those of token t
    bool good = false;
    // the next group's loads: x, and for the gradient d_out
    uint4 xa = none, xb = none, da = none, db = none;
    auto load = [&](int64_t tok, int grp) {
        const int head = grp * HPW + lane / L;
        const bool on = head < side.heads;
        const uint16_t* x = side.x + tok * side.x_token + head * side.x_head;
        xa = on && pl.a >= 0 ? ld_stream_u4(x + pl.a) : none;
        xb = on && pl.b >= 0 ? ld_stream_u4(x + pl.b) : none;
        if constexpr (GRAD) {
            const uint16_t* d = side.d_out + tok * side.d_token + head * side.d_head;
            da = on && pl.a >= 0 ? ld_stream_u4(d + pl.a) : none;
            db = on && pl.b >= 0 ? ld_stream_u4(d + pl.b) : none;
        }
    };
    if (g0 < g1) load(t, in_token);
    for (int64_t g = g0; g < g1; ++g) {
        const uint4 va = xa, vb = xb, ea = da, eb = db;
        if (!known) {
            const int pos = p.positions[t];
            good = static_cast<uint32_t>(pos) < static_cast<uint32_t>(p.max_positions);
            if (!good && lane == 0) atomicOr(p.status, MFR_STATUS_BAD_INDEX);
            if (good && pl.turns) {
                const float* row = p.table + static_cast<int64_t>(pos) * p.rotary + 8 * pl.u;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    c[i] = __ldg(row + i);
                    s[i] = __ldg(row + p.rotary / 2 + i);
                }
            }
            known = true;
        }
        const int64_t t_now = t;
        const int head = in_token * HPW + lane / L;
        const bool good_now = good;
        if (++in_token == per) {
            in_token = 0;
            ++t;
        }
        if (g + 1 < g1) load(t, in_token);
        float x[16];
        widen<F16>(va, x);
        widen<F16>(vb, x + 8);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
        const float inv = rsqrtf(head_sum<L>(ss) / static_cast<float>(p.D) + p.eps);
        if constexpr (!GRAD) {
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = x[i] * inv * gamma[i];
            if (pl.turns) turn<false>(x, c, s, interleaved);
        } else {
            float d[16];
            widen<F16>(ea, d);
            widen<F16>(eb, d + 8);
            if (pl.turns) turn<true>(d, c, s, interleaved);
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                x[i] *= inv;                                  // unit
                if (good_now) sum[i] = fmaf(d[i], x[i], sum[i]);
                d[i] *= gamma[i];
                dot = fmaf(d[i], x[i], dot);
            }
            const float mean = head_sum<L>(dot) / static_cast<float>(p.D);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = inv * (d[i] - x[i] * mean);
        }
        if (good_now && head < side.heads) {
            uint16_t* o = side.out + t_now * side.out_token + head * side.out_head;
            if (pl.a >= 0) st_stream_u4(o + pl.a, narrow<F16>(x));
            if (pl.b >= 0) st_stream_u4(o + pl.b, narrow<F16>(x + 8));
        }
        if (t != t_now) known = false;
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
            const Place q = place_of(j % L, p.D, p.rotary, interleaved);
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
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(32 * kSumWarps) qk_gamma_kernel(const QkParams p, const QkRuns r, int blocks) {
    __shared__ float s_sum[kSumWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tiles = (p.D + 31) / 32;
    const int which = static_cast<int>(blockIdx.x) / tiles, col = static_cast<int>(blockIdx.x) % tiles * 32 + lane;
    pdl_wait();
    pdl_launch_dependents();
    const int first = which ? r.blocks_q : 0, last = which ? blocks : r.blocks_q;
    float v = 0.f;
    if (col < p.D)
        for (int b = first + warp; b < last; b += kSumWarps) v += __ldcg(p.partial + static_cast<int64_t>(b) * p.D + col);
    s_sum[warp][lane] = v;
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

template <bool F16, bool GRAD>
Kernel kernel_of(int D) {
    switch (lanes_for(D)) {
        case 1: return qk_kernel<F16, 1, GRAD>;
        case 2: return qk_kernel<F16, 2, GRAD>;
        case 4: return qk_kernel<F16, 4, GRAD>;
        case 8: return qk_kernel<F16, 8, GRAD>;
        case 16: return qk_kernel<F16, 16, GRAD>;
        default: return qk_kernel<F16, 32, GRAD>;
    }
}

Kernel kernel_for(const QkShape& s, bool grad) {
    if (s.fp16) return grad ? kernel_of<true, true>(s.D) : kernel_of<true, false>(s.D);
    return grad ? kernel_of<false, true>(s.D) : kernel_of<false, false>(s.D);
}

// A warp's run: as few groups as keep every SM in work, so that small calls have
// many warps and large ones few partial sums and token changes.
QkRuns runs_for(const QkShape& s, int64_t T, bool grad, int sms, int* blocks) {
    const int hpw = 32 / lanes_for(s.D);
    QkRuns r;
    r.per_token[0] = (s.heads_q + hpw - 1) / hpw;
    r.per_token[1] = (s.heads_k + hpw - 1) / hpw;
    const int64_t groups = T * (r.per_token[0] + r.per_token[1]);
    const int64_t warps = static_cast<int64_t>(sms) * kQkWarps * (grad ? 3 : 16);
    int64_t run = (groups + warps - 1) / warps;
    if (!grad && run > 16) run = 16;
    if (run < 1) run = 1;
    int64_t b[2];
    for (int i = 0; i < 2; ++i) {
        r.run[i] = static_cast<int>(run);
        const int64_t per_block = run * kQkWarps;
        b[i] = (T * r.per_token[i] + per_block - 1) / per_block;
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
