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
// once.  A lane holds 16 elements of a head, both members of each of its pairs, as
// pairs of FP32 values that one instruction works on, so that nothing is exchanged but
// the sums; a head takes as many lanes as it needs (D / 16) and a warp as many
// heads of one token as it holds.  A warp's unit of work is a run of such groups of
// heads, whose cosines and sines stay in registers, two groups' loads in flight.
// Queries and keys belong to different CTAs, so that a lane's gamma and its running sum
// of d_gamma stay where they are; the gradient's warps stay for several units, and a
// second launch adds their sums in a fixed order.
// Measured on GB300, of the copy rate: 16384 x 40 heads x 128 out of a packed tensor 58.5
// us (0.87; 61 without the prefetch to L2), its gradient at 8192 tokens 48.5 us (0.78); 4097
// x 28 x 80 gradient 21 us (0.39: 2.5 units a warp, whose first loads nothing covers, 390
// instructions a group of heads, and 3 us for the second launch).  Loads wait: 22 warps an
// SM have 24 KB in flight in registers.  Three or four groups at a time (64, 67 us), more
// warps of fewer registers (67), refilling a group's registers as soon as it is in use
// (63) and copies into shared memory four groups ahead (80) were no faster, nor was
// prefetching in the gradient (50, and 24 for 23.5).
#include "moe_step_ops.h"
#include "mfr_device.cuh"
#include "mfr_layer.h"
#include "mfr_step.h"

namespace mfr {
namespace {

constexpr int kQkWarps = 4;
constexpr int kQkCtas = 6, kQkGradCtas = 4;      // an SM

// Two FP32 values that one instruction works on.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pair(float lo, float hi) {
    f2 v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
    return v;
}
__device__ __forceinline__ float2 halves(f2 v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ f2 both(float v) { return pair(v, v); }
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f2 swapped(f2 v) {
    const float2 f = halves(v);
    return pair(f.y, f.x);
}
__device__ __forceinline__ float sum2(f2 v) {
    const float2 f = halves(v);
    return f.x + f.y;
}

// Eight 16-bit values as four pairs, and back.
template <bool F16>
__device__ __forceinline__ void widen(uint4 v, f2* f) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (F16) {
            const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            f[i] = pair(x.x, x.y);
        } else {
            f[i] = pair(bf16_lo(u[i]), bf16_hi(u[i]));
        }
    }
}

template <bool F16>
__device__ __forceinline__ uint32_t narrow2(f2 v) {
    const float2 f = halves(v);
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(f.x, f.y);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        return pack_bf16x2(f.x, f.y);
    }
}

template <bool F16>
__device__ __forceinline__ uint4 narrow(const f2* f) {
    return make_uint4(narrow2<F16>(f[0]), narrow2<F16>(f[1]), narrow2<F16>(f[2]), narrow2<F16>(f[3]));
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" :: "l"(p)); }

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

// A lane's cosines and sines, as `turn` takes them: for pairs (i, i + rotary / 2) four
// pairs each of neighbours, for pairs (2 i, 2 i + 1) eight of (cos, cos) and of (-sin, sin),
// or back (sin, -sin).
template <bool BACK, bool PAIRED>
struct Angles {
    f2 c[PAIRED ? 8 : 4], s[PAIRED ? 8 : 4];
    __device__ __forceinline__ void set(int i, float c0, float c1, float s0, float s1) {      // angles 2 i and 2 i + 1
        if constexpr (PAIRED) {
            c[2 * i] = both(c0);
            c[2 * i + 1] = both(c1);
            s[2 * i] = BACK ? pair(s0, -s0) : pair(-s0, s0);
            s[2 * i + 1] = BACK ? pair(s1, -s1) : pair(-s1, s1);
        } else {
            c[i] = pair(c0, c1);
            s[i] = pair(s0, s1);
        }
    }
};

// The pairs of x turned by the angles, or back.
template <bool BACK, bool PAIRED>
__device__ __forceinline__ void turn(f2 (&x)[8], const Angles<BACK, PAIRED>& t) {
    if constexpr (PAIRED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fma2(swapped(x[i]), t.s[i], mul2(x[i], t.c[i]));
    } else {
        const f2 minus = both(-1.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const f2 a = x[i], b = x[i + 4], less = mul2(BACK ? a : b, minus);
            x[i] = fma2(BACK ? b : less, t.s[i], mul2(a, t.c[i]));
            x[i + 4] = fma2(BACK ? less : a, t.s[i], mul2(b, t.c[i]));
        }
    }
}

// Sum over a head's lanes, L or (L = 0) `lanes` of them from `base` on.
template <int L>
__device__ __forceinline__ float head_sum(float v, int lanes, int base) {
    if constexpr (L > 0 && (L & (L - 1)) == 0) {
#pragma unroll
        for (int off = L / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
        return v;
    } else {
        float sum = 0.f;
        if constexpr (L > 0) {
#pragma unroll
            for (int i = 0; i < L; ++i) sum += __shfl_sync(0xFFFFFFFFu, v, base + i);
        } else {
            for (int i = 0; i < lanes; ++i) sum += __shfl_sync(0xFFFFFFFFu, v, base + i);
        }
        return sum;
    }
}

// Units of work: CTA b < blocks_q has queries' units, the others keys'.  A group is HPW =
// 32 / lanes heads; a token's per_token groups are `slices` runs of `run` groups, and
// unit u is run u % slices of token u / slices.  A warp takes every stride-th unit:
// step_t tokens and step_s runs further.
struct QkRuns {
    int lanes;              // of a head
    int blocks_q;
    int run[2];
    int per_token[2];
    int slices[2];
    int step_t[2];
    int step_s[2];
};

// L: lanes of a head, 0: as many as r says.  PAIRED: pairs (2 i, 2 i + 1).
template <bool F16, int L, bool GRAD, bool PAIRED>
__global__ void __launch_bounds__(32 * kQkWarps, GRAD ? kQkGradCtas : kQkCtas) qk_kernel(const __grid_constant__ QkParams p, const __grid_constant__ QkRuns r) {
    constexpr int BATCH = 2;                  // groups whose loads are in flight
    __shared__ float s_gamma[GRAD ? kQkWarps : 1][GRAD ? 32 * 16 : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lanes = L > 0 ? L : r.lanes, heads_a_warp = 32 / lanes;
    const int which = static_cast<int>(blockIdx.x) < r.blocks_q ? 0 : 1;
    const QkSide& side = p.side[which];
    const int per = r.per_token[which], slices = r.slices[which], run = r.run[which];
    const int of_head = lane / lanes, base = of_head * lanes;
    const bool used = of_head < heads_a_warp;             // lanes behind the last whole head have none
    const Place pl = place_of(lane - base, p.D, p.rotary, PAIRED);
    const bool has_a = used && pl.a >= 0, has_b = used && pl.b >= 0;
    const float per_element = 1.f / static_cast<float>(p.D);
    pdl_wait();
    pdl_launch_dependents();
    const uint4 none = make_uint4(0, 0, 0, 0);
    f2 gamma[8], sum[GRAD ? 8 : 1];
    widen<F16>(has_a ? *reinterpret_cast<const uint4*>(side.gamma + pl.a) : none, gamma);
    widen<F16>(has_b ? *reinterpret_cast<const uint4*>(side.gamma + pl.b) : none, gamma + 4);
    if constexpr (GRAD)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] = 0;
    // T * slices is the number of 16 heads at most that an output holds: far below 2^32
    const uint32_t unit = (blockIdx.x - (which ? r.blocks_q : 0)) * kQkWarps + warp;
    int64_t t = unit / static_cast<uint32_t>(slices);
    int slice = static_cast<int>(unit - static_cast<uint32_t>(t) * slices);
    int next_pos = t < p.T ? p.positions[t] : 0;
    while (t < p.T) {
        int next_slice = slice + r.step_s[which];
        int64_t next = t + r.step_t[which];
        if (next_slice >= slices) {
            next_slice -= slices;
            ++next;
        }
        const int g0 = slice * run, g1 = min(g0 + run, per);
        const int pos = next_pos;
        if (next < p.T) next_pos = p.positions[next];     // long before its cosines are asked for
        const int first = g0 * heads_a_warp + of_head;
        const uint16_t* xs = side.x + t * side.x_token + first * side.x_head;
        const uint16_t* ds = GRAD ? side.d_out + t * side.d_token + first * side.d_head : nullptr;
        uint16_t* os = side.out + t * side.out_token + first * side.out_head;
        const int64_t x_step = heads_a_warp * side.x_head, d_step = GRAD ? heads_a_warp * side.d_head : 0;
        const int64_t o_step = heads_a_warp * side.out_head;
        int heads = side.heads - first;                   // from this lane's first on
        Angles<GRAD, PAIRED> angles;
        bool known = false, good = false;
        for (int g = g0; g < g1; g += BATCH) {
            uint4 xa[BATCH], xb[BATCH], da[GRAD ? BATCH : 1], db[GRAD ? BATCH : 1];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const bool on = g + i < g1 && i * heads_a_warp < heads;
                xa[i] = xb[i] = none;
                if (on && has_a) xa[i] = ld_stream_u4(xs + i * x_step + pl.a);
                if (on && has_b) xb[i] = ld_stream_u4(xs + i * x_step + pl.b);
                if constexpr (GRAD) {
                    da[i] = db[i] = none;
                    if (on && has_a) da[i] = ld_stream_u4(ds + i * d_step + pl.a);
                    if (on && has_b) db[i] = ld_stream_u4(ds + i * d_step + pl.b);
                }
            }
            if (!known) {
                known = true;
                // the rest of the run to L2: more bytes in flight than registers hold
                if constexpr (!GRAD)
                    for (int i = BATCH; i < g1 - g0; ++i) {
                        const bool on = i * heads_a_warp < heads;
                        if (on && has_a) prefetch_l2(xs + i * x_step + pl.a);
                        if (on && has_b) prefetch_l2(xs + i * x_step + pl.b);
                    }
                good = static_cast<uint32_t>(pos) < static_cast<uint32_t>(p.max_positions);
                if (!good && lane == 0) atomicOr(p.status, MFR_STATUS_BAD_INDEX);
                const float4* row = reinterpret_cast<const float4*>(p.table + static_cast<int64_t>(pos) * p.rotary + 8 * pl.u);
                const bool on = good && pl.turns;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float4 a = on ? __ldg(row + i) : make_float4(1.f, 1.f, 1.f, 1.f);
                    const float4 b = on ? __ldg(row + p.rotary / 8 + i) : make_float4(0.f, 0.f, 0.f, 0.f);
                    angles.set(2 * i, a.x, a.y, b.x, b.y);
                    angles.set(2 * i + 1, a.z, a.w, b.z, b.w);
                }
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                if (g + i >= g1) break;
                const bool here = good && i * heads_a_warp < heads;      // this lane's head counts
                f2 x[8], square = 0;
                widen<F16>(xa[i], x);
                widen<F16>(xb[i], x + 4);
#pragma unroll
                for (int e = 0; e < 8; ++e) square = fma2(x[e], x[e], square);
                const float inv = rsqrtf(fmaf(head_sum<L>(sum2(square), lanes, base), per_element, p.eps));
                const f2 inv2 = both(inv);
                if constexpr (!GRAD) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = mul2(mul2(x[e], inv2), gamma[e]);
                    if (pl.turns) turn<false, PAIRED>(x, angles);
                } else {
                    f2 d[8], dot2 = 0;
                    widen<F16>(da[i], d);
                    widen<F16>(db[i], d + 4);
                    if (pl.turns) turn<true, PAIRED>(d, angles);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x[e] = mul2(x[e], inv2);                      // unit
                        // zeros of a lane without a head are NaN here when eps is 0
                        if (here) sum[e] = fma2(d[e], x[e], sum[e]);
                        d[e] = mul2(d[e], gamma[e]);
                        dot2 = fma2(d[e], x[e], dot2);
                    }
                    const f2 less = both(-(head_sum<L>(sum2(dot2), lanes, base) * per_element));
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = mul2(inv2, fma2(x[e], less, d[e]));
                }
                if (here) {
                    if (has_a) st_stream_u4(os + i * o_step + pl.a, narrow<F16>(x));
                    if (has_b) st_stream_u4(os + i * o_step + pl.b, narrow<F16>(x + 4));
                }
            }
            heads -= BATCH * heads_a_warp;
            xs += BATCH * x_step;
            os += BATCH * o_step;
            if constexpr (GRAD) ds += BATCH * d_step;
        }
        t = next;
        slice = next_slice;
    }
    if constexpr (GRAD) {
        // the CTA's warps' heads, in a fixed order
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = halves(sum[i]);
            s_gamma[warp][(2 * i) * 32 + lane] = f.x;
            s_gamma[warp][(2 * i + 1) * 32 + lane] = f.y;
        }
        __syncthreads();
        for (int j = threadIdx.x; j < 16 * lanes; j += 32 * kQkWarps) {
            const int i = j / lanes, u = j % lanes;
            const Place q = place_of(u, p.D, p.rotary, PAIRED);
            const int at = i < 8 ? q.a : q.b;
            if (at < 0) continue;
            float v = 0.f;
            for (int w = 0; w < kQkWarps; ++w)
                for (int h = 0; h < heads_a_warp; ++h) v += s_gamma[w][i * 32 + h * lanes + u];
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
    float sum = 0.f;
    if (col < p.D)
        for (int b = first + warp; b < last; b += 8 * kSumWarps) {
            float v[8];                               // eight rows in flight
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = b + i * kSumWarps < last ? __ldcg(p.partial + static_cast<int64_t>(b + i * kSumWarps) * p.D + col) : 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += v[i];
        }
    s_sum[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && col < p.D) {
        float total = 0.f;
        for (int w = 0; w < kSumWarps; ++w) total += s_sum[w][lane];
        p.side[which].d_gamma[col] = total;
    }
}

using Kernel = void (*)(const QkParams, const QkRuns);

int lanes_for(int D) { return (D + 15) / 16; }

// A head's lanes are known to the kernel up to 8 and for powers of two (4097 x 28 heads of 80,
// gradient: 23.5 us with a loop over them, 21 so).
template <bool F16, bool GRAD, bool PAIRED>
Kernel kernel_of(int D) {
    switch (lanes_for(D)) {
        case 1: return qk_kernel<F16, 1, GRAD, PAIRED>;
        case 2: return qk_kernel<F16, 2, GRAD, PAIRED>;
        case 3: return qk_kernel<F16, 3, GRAD, PAIRED>;
        case 4: return qk_kernel<F16, 4, GRAD, PAIRED>;
        case 5: return qk_kernel<F16, 5, GRAD, PAIRED>;
        case 6: return qk_kernel<F16, 6, GRAD, PAIRED>;
        case 7: return qk_kernel<F16, 7, GRAD, PAIRED>;
        case 8: return qk_kernel<F16, 8, GRAD, PAIRED>;
        case 16: return qk_kernel<F16, 16, GRAD, PAIRED>;
        case 32: return qk_kernel<F16, 32, GRAD, PAIRED>;
        default: return qk_kernel<F16, 0, GRAD, PAIRED>;
    }
}

template <bool GRAD>
Kernel kernel_of(const QkShape& s) {
    if (s.fp16) return s.interleaved ? kernel_of<true, GRAD, true>(s.D) : kernel_of<true, GRAD, false>(s.D);
    return s.interleaved ? kernel_of<false, GRAD, true>(s.D) : kernel_of<false, GRAD, false>(s.D);
}

Kernel kernel_for(const QkShape& s, bool grad) { return grad ? kernel_of<true>(s) : kernel_of<false>(s); }

// A warp's run is a token's groups where tokens are many, fewer where that leaves
// SMs without work.  The gradient's CTAs are as many as find room at once, so that there
// are few partial sums of d_gamma.
QkRuns runs_for(const QkShape& s, int64_t T, bool grad, int sms, int* blocks) {
    QkRuns r;
    r.lanes = lanes_for(s.D);
    const int hpw = 32 / r.lanes, heads[2] = {s.heads_q, s.heads_k};
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
    // a unit's work: its groups, and about two more for its first loads, which nothing covers
    const int64_t work[2] = {units[0] * (r.run[0] + 2), units[1] * (r.run[1] + 2)};
    const int64_t all = work[0] + work[1], most = static_cast<int64_t>(sms) * kQkGradCtas;
    int64_t b[2];
    for (int i = 0; i < 2; ++i) {
        b[i] = (units[i] + kQkWarps - 1) / kQkWarps;
        if (grad && all > 0) {
            // shares of the CTAs in the proportion of the work
            int64_t share = most * work[i] / all;
            if (share < 1) share = 1;
            if (b[i] > share) b[i] = share;
        }
        r.step_t[i] = static_cast<int>(b[i] * kQkWarps / r.slices[i]);
        r.step_s[i] = static_cast<int>(b[i] * kQkWarps % r.slices[i]);
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
