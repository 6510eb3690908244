// The router's choice and its gradient.
//
//   scores   p = softmax(l) over the E experts, or sigmoid(l)
//   choice   the k largest l, or sigmoid(l) + bias where there is a bias; among
//            equals the lowest index
//   weights  w_j = scale * p_j, or scale * p_j / (p_1 + .. + p_k)
//
// A warp per token, its logits in registers (E / 32 a lane) as order-preserving integer
// keys.  k maxima over the lanes' largest keys give a bound that the k chosen reach and
// few others do; those few (up to 32, else they are taken one by one) are compared
// with each other.  With softmax scores, and with sigmoid ones without a bias, the keys
// are the logits themselves (both functions rise), so the choice is exact.  With a bias the FP32 keys are off by some of their last
// bits: neighbours in the order that lie closer than those errors reach (about a
// token in a thousand) are chosen once more by keys in 64 bits.
//
// Bytes would bound both directions (32768 x 256: 5 us), but the choice's instructions
// do: 22 us with a bias, 17 without (k = 8; taking the k experts one by one: 50).  The
// gradient of renormalised softmax weights reads the chosen logits alone (16385 x 128:
// 5.8 us, 2.6 of bytes, bound by its instructions as well).
#include <cfloat>

#include "moe_step_ops.h"
#include "mfr_device.cuh"
#include "mfr_layer.h"
#include "mfr_step.h"

namespace mfr {
namespace {

constexpr int kGateWarps = 4;
constexpr int kGateCtas = 8;           // an SM, of the choice (10 or 12 spill registers: 25, 29 us)

// Rises with f; 0 for -infinity and NaN, which are never chosen.
__device__ __forceinline__ uint32_t order_key(float f) {
    f += 0.f;                                             // -0 counts as 0
    const uint32_t u = __float_as_uint(f);
    return f > -INFINITY ? u ^ ((static_cast<int32_t>(u) >> 31) | 0x80000000u) : 0u;
}
// That of a key with a bias.
__device__ __forceinline__ uint32_t order_key(float l, float key) {
    const uint32_t u = __float_as_uint(key);              // never -0: a sigmoid is not
    return l > -INFINITY && key > -INFINITY ? u ^ ((static_cast<int32_t>(u) >> 31) | 0x80000000u) : 0u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

template <bool B16>
__device__ __forceinline__ float logit_at(const void* l, int64_t i) {
    if constexpr (B16) return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(l)[i]) << 16);
    else return static_cast<const float*>(l)[i];
}

// This lane's N logits of row `at`, from expert lane * N on: lower lanes have lower
// experts.  V: logits a load, where rows start on such a boundary.
template <bool B16, int V, int N>
__device__ __forceinline__ void load_row(const void* l, int64_t at, int E, int lane, float (&f)[N]) {
#pragma unroll
    for (int v = 0; v < N; v += V) {
        const int e = lane * N + v;
        if constexpr (V == 4) {
            float4 x = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (e < E) {
                if constexpr (B16) {
                    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(l) + at + e);
                    x = make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
                } else {
                    x = *reinterpret_cast<const float4*>(static_cast<const float*>(l) + at + e);
                }
            }
            f[v] = x.x; f[v + 1] = x.y; f[v + 2] = x.z; f[v + 3] = x.w;
        } else {
            f[v] = e < E ? logit_at<B16>(l, at + e) : -INFINITY;
        }
    }
}

// Off by 2^-23 (one ulp); 0 from 2^126 on, where 1 / v is no normal number.  In place of
// divisions, whose instructions bound the choice: weights of 32768 x 256 with a bias are
// off by 6.5e-8 with it (rms of the error by that of the weights; FP32 divisions 5.3e-8),
// gradients of 16385 x 128 by 6.9e-8 (6.6e-8).
__device__ __forceinline__ float reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float sigmoid(float l) { return reciprocal(1.f + expf(-l)); }

// For keys, off by less than 6.25 u (u = 2^-24): ex2.approx is off by 2^-22 and its
// rounded argument by 2 u |l|, which the sigmoid's slope makes 1.25 u at most (where
// |l| is large it is flat); the sum by u, rcp.approx by 2^-23.
__device__ __forceinline__ float near_sigmoid(float l) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * -1.4426950408889634f));
    return reciprocal(1.f + e);
}

__device__ __forceinline__ float warp_max(float v) {
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
    return v;
}

// Sum over a token's slots, a lane each, for the lanes that may have one.
__device__ __forceinline__ float slots_sum(float v) {
#pragma unroll
    for (int off = kMaxK / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

// sigmoid(l) times a factor that the token's chosen logits share (top: the largest),
// 1 where one of them is positive: far negative ones still have their proportions.
__device__ __forceinline__ float shared_sigmoid(float l, float top) {
    return top > 0.f ? sigmoid(l) : expf(l - fmaxf(top, -FLT_MAX)) * reciprocal(1.f + expf(l));
}

// Rises with f, a double that is no NaN; above 0.
__device__ __forceinline__ unsigned long long order_key64(double f) {
    const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(f + 0.0));
    return u ^ ((static_cast<long long>(u) >> 63) | 0x8000000000000000ull);
}

// An expert's key in 64 bits.  FP64 instructions are slow on this chip (a warp's takes 16
// cycles), so that few are computed, a lane each where that goes.
__device__ __noinline__ unsigned long long exact_key(float l, float bias) {
    return order_key64(1.0 / (1.0 + exp(-static_cast<double>(l))) + static_cast<double>(bias));
}

// The least FP32 key whose exact one may be as large as that of `key`; infinity, an
// infinite bias, is exact.
__device__ __forceinline__ float reach(float key) { return key < INFINITY ? key - 0x1p-20f * (1.f + fabsf(key)) : key; }

// The choice by keys in 64 bits among the experts whose FP32 key is at least `from`;
// lane j gets the j-th one.
template <bool B16>
__device__ __noinline__ int choose_in_64_bits(const GateParams& p, int64_t at, float from, int lane) {
    unsigned long long keys[kMaxExperts / 32];
    const int n = (p.E + 31) / 32;
    for (int i = 0; i < n; ++i) {
        const int e = i * 32 + lane;
        const float l = e < p.E ? logit_at<B16>(p.logits, at + e) : -INFINITY;
        keys[i] = 0;
        if (!(l > -INFINITY)) continue;
        const float bias = p.bias[e];
        if (near_sigmoid(l) + bias >= from) keys[i] = exact_key(l, bias);
    }
    int mine = -1;
    for (int j = 0; j < p.k; ++j) {
        unsigned long long best = 0;
        int best_i = 0;
        for (int i = 0; i < n; ++i)
            if (keys[i] > best) {
                best = keys[i];
                best_i = i;
            }
        unsigned long long top = best;
        int e = best_i * 32 + lane;
        for (int off = 16; off > 0; off >>= 1) {
            const unsigned long long k2 = __shfl_xor_sync(0xFFFFFFFFu, top, off);
            const int e2 = __shfl_xor_sync(0xFFFFFFFFu, e, off);
            if (k2 > top || (k2 == top && e2 < e)) {
                top = k2;
                e = e2;
            }
        }
        if (top == 0) break;
        if (e % 32 == lane) keys[e / 32] = 0;
        if (lane == j) mine = e;
    }
    return mine;
}

// A warp's tokens are t, t + all warps, ...: the next one's logits are on their way
// while this one's experts are chosen.
template <bool B16, int V, int N>
__global__ void __launch_bounds__(32 * kGateWarps, N <= 8 ? kGateCtas : 1) gate_kernel(const GateParams p) {
    constexpr bool KEPT = N <= 8;                         // biases in registers
    __shared__ __align__(16) unsigned long long s_key[kGateWarps][36], s_sorted[kGateWarps][32];
    const int lane = threadIdx.x & 31;
    unsigned long long* keys = s_key[threadIdx.x >> 5];
    unsigned long long* sorted = s_sorted[threadIdx.x >> 5];
    const int64_t warps = static_cast<int64_t>(gridDim.x) * kGateWarps;
    int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_dependents();
    float bias[KEPT ? N : 1];
    if constexpr (KEPT)
#pragma unroll
        for (int i = 0; i < N; ++i) bias[i] = p.bias && lane * N + i < p.E ? __ldg(p.bias + lane * N + i) : 0.f;
    float next[N];
    if (t < p.T) load_row<B16, V, N>(p.logits, t * p.E, p.E, lane, next);
    for (; t < p.T; t += warps) {
        const int64_t at = t * p.E;
        float l[N];
#pragma unroll
        for (int i = 0; i < N; ++i) l[i] = next[i];
        if (t + warps < p.T) load_row<B16, V, N>(p.logits, at + warps * p.E, p.E, lane, next);
        float denominator = 1.f, top = 0.f;
        if (!p.sigmoid && !p.renormalize) {
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < N; ++i) m = fmaxf(m, l[i]);
            m = warp_max(m);
            top = fminf(fmaxf(m, -FLT_MAX), FLT_MAX);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) sum += l[i] > -INFINITY ? expf(fminf(l[i], FLT_MAX) - top) : 0.f;
            denominator = warp_allreduce_sum(sum);
        }
        uint32_t key[N], best = 0;                        // this lane's largest
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (p.bias) {
                float b;
                if constexpr (KEPT) b = bias[i];
                else b = lane * N + i < p.E ? __ldg(p.bias + lane * N + i) : 0.f;
                key[i] = order_key(l[i], near_sigmoid(l[i]) + b);
            } else {
                key[i] = order_key(l[i]);
            }
            best = max(best, key[i]);
        }
        int mine = -1;
        float x = 0.f;                                    // its logit
        // one more: whether the first left out is close; and another, so that the bound lies
        // below what may be among the chosen (32768 x 256, k = 8: 32 -> 26 us then; with k = 16 more
        // than 32 experts reach it too often: 33 -> 43)
        const int wanted = p.bias ? p.k + (p.k <= 8 ? 2 : 1) : p.k;
        // A bound below the last of the wanted keys: that many lanes' largest reach it.
        uint32_t bound = 0, left = best;
        for (int j = 0; j < wanted; ++j) {
            bound = __reduce_max_sync(0xFFFFFFFFu, left);
            if (left == bound) left = 0;
        }
        bound = max(bound, 1u);
        int own_count = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) own_count += key[i] >= bound;
        int upto = own_count;                             // of the lanes to this one
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, upto, off);
            if (lane >= off) upto += v;
        }
        const int count = __shfl_sync(0xFFFFFFFFu, upto, 31);
        bool known = false;                               // x is
        if (count <= 32) {
            // The few experts that reach it, one a lane, find their ranks by comparing.
            int to = upto - own_count;
#pragma unroll
            for (int i = 0; i < N; ++i)
                // falling order of these: keys, then rising experts
                if (key[i] >= bound) keys[to++] = (static_cast<unsigned long long>(key[i]) << 32) | (0xFFFFFFFFu - (lane * N + i));
            if (lane < 4) keys[count + lane] = 0;         // four are compared at a time
            __syncwarp();
            const unsigned long long own = lane < count ? keys[lane] : 0;
            int rank = 0;
            for (int j = 0; j < count; j += 4) {
                const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(keys + j), b = *reinterpret_cast<const ulonglong2*>(keys + j + 2);
                rank += (a.x > own) + (a.y > own) + (b.x > own) + (b.y > own);
            }
            if (lane < count) sorted[rank] = own;
            __syncwarp();
            const unsigned long long at_rank = lane < count ? sorted[lane] : 0x8000000000000000ull;
            const int e = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(at_rank));
            const float v = key_value(static_cast<uint32_t>(at_rank >> 32));
            if (lane < min(p.k, count)) mine = e;
            if (!p.bias) {
                x = v;
                known = true;
            } else {
                // Neighbours in the order that are closer than their keys' errors, two of less
                // than 2^-21 (1 + |key|) each (6.25 u for the sigmoid, u |key| for the sum):
                // keys in 64 bits decide, unless experts below the bound may be among them.
                const float after = __shfl_down_sync(0xFFFFFFFFu, v, 1);
                const bool close = lane < p.k && lane + 1 < count && !(v - after > 0x1p-20f * (1.f + fabsf(after)));
                if (__any_sync(0xFFFFFFFFu, close)) {
                    const float from = reach(__shfl_sync(0xFFFFFFFFu, v, max(0, min(p.k, count) - 1)));
                    if (bound > 1 && !(key_value(bound) < from)) {
                        mine = choose_in_64_bits<B16>(p, at, from, lane);
                    } else {
                        unsigned long long exact = 0;
                        if (lane < count) keys[lane] = exact = exact_key(logit_at<B16>(p.logits, at + e), __ldg(p.bias + e));
                        __syncwarp();
                        rank = 0;
                        for (int j = 0; j < count; ++j) {
                            // equal ones: the lower expert, of which the FP32 order tells nothing
                            const int other = __shfl_sync(0xFFFFFFFFu, e, j);
                            rank += keys[j] > exact || (keys[j] == exact && other < e);
                        }
                        if (lane < count) sorted[rank] = static_cast<unsigned long long>(e);
                        __syncwarp();
                        if (lane < min(p.k, count)) mine = static_cast<int>(sorted[lane]);
                    }
                }
            }
            __syncwarp();
        } else {
            uint32_t before = 0;
            bool close = false;
            float least = -INFINITY;
            for (int j = 0; j < (p.bias ? p.k + 1 : p.k); ++j) {
                const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, best);
                if (m == 0) break;
                const int owner = __ffs(__ballot_sync(0xFFFFFFFFu, best == m)) - 1;
                int e = 0;
                if (lane == owner) {
                    // its first expert with this key goes
                    best = 0;
                    bool found = false;
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const bool hit = !found && key[i] == m;
                        if (hit) {
                            e = i;
                            key[i] = 0;
                        }
                        found |= hit;
                        best = max(best, key[i]);
                    }
                }
                e = __shfl_sync(0xFFFFFFFFu, e, owner) + owner * N;
                if (lane == j && j < p.k) mine = e;
                if (p.bias) {
                    const float v = key_value(m);
                    close |= j > 0 && !(key_value(before) - v > 0x1p-20f * (1.f + fabsf(v)));
                    before = m;
                    if (j < p.k) least = v;
                }
            }
            // the least key that may be among the chosen: that of the k-th, less both errors
            if (close) mine = choose_in_64_bits<B16>(p, at, reach(least), lane);
        }
        if (!known && mine >= 0) x = logit_at<B16>(p.logits, at + mine);
        float w = mine >= 0 ? fminf(x, FLT_MAX) : 0.f;
        if (p.sigmoid) {
            if (!p.renormalize || __any_sync(0xFFFFFFFFu, w > 0.f)) {
                w = mine >= 0 ? sigmoid(w) : 0.f;
            } else {
                top = warp_max(mine >= 0 ? w : -INFINITY);
                w = mine >= 0 ? shared_sigmoid(w, top) : 0.f;
            }
        } else {
            if (p.renormalize) top = __shfl_sync(0xFFFFFFFFu, w, 0);   // the first chosen is the largest
            w = mine >= 0 ? expf(w - top) : 0.f;
        }
        if (p.renormalize) denominator = slots_sum(w);
        if (lane < p.k) {
            p.ids[t * p.k + lane] = mine;
            p.w[t * p.k + lane] = w > 0.f ? p.scale * (w * reciprocal(denominator)) : 0.f;
        }
    }
}

// d_logits: what every expert gets, then the chosen ones once more with their own part.
// Vector v of a lane holds experts (v * 32 + lane) * V and on.
template <bool B16, int V, int NV>
__global__ void __launch_bounds__(32 * kGateWarps) gate_grad_kernel(const GateParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_dependents();
    if (t >= p.T) return;
    const int64_t at = t * p.E;
    const bool full = !p.sigmoid && !p.renormalize;       // every expert gets something
    float l[NV * V];
    if (full)
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float x[V];
            load_row<B16, V, V>(p.logits, at + v * 32 * V, p.E - v * 32 * V, lane, x);
#pragma unroll
            for (int i = 0; i < V; ++i) l[v * V + i] = x[i];
        }
    // lane j: the j-th chosen expert, its logit and the gradient of its weight
    int e = lane < p.k ? p.ids_in[t * p.k + lane] : -1;
    const float d_w = lane < p.k ? p.d_w[t * p.k + lane] : 0.f;
    if (e >= p.E || e < -1) {
        atomicOr(p.status, MFR_STATUS_BAD_INDEX);
        e = -1;
    }
    const bool on = e >= 0;
    const float x = on ? logit_at<B16>(p.logits, at + e) : -INFINITY, le = fminf(x, FLT_MAX);
    const float g = on ? p.scale * d_w : 0.f;
    float d, all = 0.f, own = 0.f;                        // of the chosen; factor of the others' scores; that of the chosen
    if (p.sigmoid) {
        float q = on ? sigmoid(le) : 0.f;
        d = g;
        if (p.renormalize) {
            const float m = warp_max(x);                  // all lanes, those without a slot too
            q = on ? shared_sigmoid(le, m) : 0.f;
            const float total = slots_sum(q);
            q = total > 0.f ? q * reciprocal(total) : 0.f;
            d = g - slots_sum(g * q);
        }
        d = on ? d * q * sigmoid(-le) : 0.f;
    } else if (p.renormalize) {
        float m = warp_max(x);
        m = fminf(fmaxf(m, -FLT_MAX), FLT_MAX);
        float q = x > -INFINITY ? expf(le - m) : 0.f;
        const float total = slots_sum(q);
        q = total > 0.f ? q * reciprocal(total) : 0.f;
        d = q * (g - slots_sum(g * q));
    } else {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV * V; ++i) m = fmaxf(m, l[i]);
        m = warp_max(m);
        m = fminf(fmaxf(m, -FLT_MAX), FLT_MAX);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV * V; ++i) {
            l[i] = l[i] > -INFINITY ? expf(fminf(l[i], FLT_MAX) - m) : 0.f;
            sum += l[i];
        }
        const float inv = reciprocal(fmaxf(warp_allreduce_sum(sum), FLT_MIN));
        const float q = x > -INFINITY ? expf(le - m) * inv : 0.f;
        const float mean = warp_allreduce_sum(g * q);      // every lane wants it
        all = -mean * inv;
        own = -mean * q;
        d = q * g;
    }
    // the same expert in several slots: the first of them has the sum
    float mine = d;
    uint32_t same = 0;                                    // slots
    for (int j = 0; j < p.k; ++j) same |= (__shfl_sync(0xFFFFFFFFu, e, j) == e ? 1u : 0u) << j;
    const bool first = on && lane == __ffs(same) - 1;
    if (__any_sync(0xFFFFFFFFu, on && (same & (same - 1)) != 0))
        for (int j = 0; j < p.k; ++j) {
            const float v = __shfl_sync(0xFFFFFFFFu, d, j);
            if ((same >> j & 1u) && j != lane) mine += v;
        }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int from = (v * 32 + lane) * V;
        if (from >= p.E) continue;
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = full ? all * l[v * V + i] : 0.f;
        if constexpr (V == 4) {
            if constexpr (B16)
                st_u2(static_cast<uint16_t*>(p.d_logits) + at + from, make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])));
            else
                st_f4(static_cast<float*>(p.d_logits) + at + from, make_float4(o[0], o[1], o[2], o[3]));
        } else if constexpr (B16) {
            static_cast<__nv_bfloat16*>(p.d_logits)[at + from] = __float2bfloat16_rn(o[0]);
        } else {
            static_cast<float*>(p.d_logits)[at + from] = o[0];
        }
    }
    __syncwarp();                                         // the warp's own stores come in this order
    if (first) {
        if constexpr (B16) static_cast<__nv_bfloat16*>(p.d_logits)[at + e] = __float2bfloat16_rn(mine + own);
        else static_cast<float*>(p.d_logits)[at + e] = mine + own;
    }
}

using Kernel = void (*)(const GateParams);

template <bool B16, int V, int N>
Kernel pick(bool grad) { return grad ? gate_grad_kernel<B16, V, N / V> : gate_kernel<B16, V, N>; }

// N logits a lane; four a load where rows start on such a boundary, else one.
template <bool B16>
Kernel kernel_for(int E, bool grad) {
    if (E % 4 == 0) {
        if (E <= 128) return pick<B16, 4, 4>(grad);
        if (E <= 256) return pick<B16, 4, 8>(grad);
        if (E <= 512) return pick<B16, 4, 16>(grad);
        return pick<B16, 4, 32>(grad);
    }
    if (E <= 32) return pick<B16, 1, 1>(grad);
    if (E <= 128) return pick<B16, 1, 4>(grad);
    if (E <= 512) return pick<B16, 1, 16>(grad);
    return pick<B16, 1, 32>(grad);
}

Kernel kernel_for(int E, bool b16, bool grad) { return b16 ? kernel_for<true>(E, grad) : kernel_for<false>(E, grad); }

}  // namespace

cudaError_t gate_prepare(int E, int b16) {
    const cudaError_t e = preload(kernel_for(E, b16 != 0, false));
    return e == cudaSuccess ? preload(kernel_for(E, b16 != 0, true)) : e;
}

cudaError_t gate_launch(const GateParams& p, int b16, bool grad, int sms, int pdl, cudaStream_t s) {
    const int64_t ctas = (p.T + kGateWarps - 1) / kGateWarps, most = static_cast<int64_t>(sms) * kGateCtas;
    return layer_launch(kernel_for(p.E, b16 != 0, grad), grad || ctas < most ? ctas : most, 32 * kGateWarps, 0, 1, pdl, s, p);
}

}  // namespace mfr
