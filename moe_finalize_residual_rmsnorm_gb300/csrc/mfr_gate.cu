// The router's choice and its gradient.
//
//   scores   p = softmax(l) over the E experts, or sigmoid(l)
//   choice   the k largest l, or sigmoid(l) + bias where there is a bias; among
//            equals the lowest index
//   weights  w_j = scale * p_j, or scale * p_j / (p_1 + .. + p_k)
//
// A warp per token, its logits in registers (E / 32 a lane).  Each of the k
// rounds is one maximum over the warp of order-preserving integer keys and one
// minimum over the indices that hold it.  With softmax scores, and with sigmoid
// ones without a bias, the keys are the logits themselves (both functions rise),
// so the choice is exact.  With a bias the FP32 keys are off by some of their last
// bits: neighbours in the order that lie closer than those errors reach (about a
// token in a thousand) are chosen once more by keys in 64 bits.
//
// Bytes bound neither direction on paper (32768 x 256: 5 us); the rounds'
// instructions do.  The gradient of renormalised softmax weights reads the chosen
// logits alone.
#include <cfloat>

#include "moe_step_ops.h"
#include "mfr_device.cuh"
#include "mfr_layer.h"
#include "mfr_step.h"

namespace mfr {
namespace {

constexpr int kGateWarps = 4;

// Rises with f; 0 for -infinity and NaN, which are never chosen.
__device__ __forceinline__ uint32_t order_key(float f) {
    f += 0.f;                                             // -0 counts as 0
    const uint32_t u = __float_as_uint(f);
    return f > -INFINITY ? u ^ ((static_cast<int32_t>(u) >> 31) | 0x80000000u) : 0u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

template <bool B16>
__device__ __forceinline__ float logit_at(const void* l, int64_t i) {
    if constexpr (B16) return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(l)[i]) << 16);
    else return static_cast<const float*>(l)[i];
}

// This lane's logits of row `at`: vector v holds experts (v * 32 + lane) * V and on.
template <bool B16, int V, int NV>
__device__ __forceinline__ void load_row(const void* l, int64_t at, int E, int lane, float (&f)[NV * V]) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int e = (v * 32 + lane) * V;
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
            f[v * 4] = x.x; f[v * 4 + 1] = x.y; f[v * 4 + 2] = x.z; f[v * 4 + 3] = x.w;
        } else {
            f[v] = e < E ? logit_at<B16>(l, at + e) : -INFINITY;
        }
    }
}

__device__ __forceinline__ float sigmoid(float l) { return 1.f / (1.f + expf(-l)); }

__device__ __forceinline__ float warp_max(float v) {
    for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
    return v;
}

// sigmoid(l) times a factor that the token's chosen logits share (top: the largest),
// 1 where one of them is positive: far negative ones still have their proportions.
__device__ __forceinline__ float shared_sigmoid(float l, float top) {
    return top > 0.f ? sigmoid(l) : expf(l - fmaxf(top, -FLT_MAX)) / (1.f + expf(l));
}

// Rises with f, a double that is no NaN; above 0.
__device__ __forceinline__ unsigned long long order_key64(double f) {
    const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(f + 0.0));
    return u ^ ((static_cast<long long>(u) >> 63) | 0x8000000000000000ull);
}

// The choice by keys in 64 bits among the experts whose FP32 key is at least `from`;
// lane j gets the j-th one.  FP64 instructions are rare on this chip (a warp's takes 16
// cycles), so that only those few experts' keys are computed, once.
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
        if (sigmoid(l) + bias >= from)
            keys[i] = order_key64(1.0 / (1.0 + exp(-static_cast<double>(l))) + static_cast<double>(bias));
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

template <bool B16, int V, int NV>
__global__ void __launch_bounds__(32 * kGateWarps) gate_kernel(const GateParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_dependents();
    if (t >= p.T) return;
    const int64_t at = t * p.E;
    float l[NV * V];
    load_row<B16, V, NV>(p.logits, at, p.E, lane, l);
    float denominator = 1.f, top = 0.f;
    if (!p.sigmoid && !p.renormalize) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV * V; ++i) m = fmaxf(m, l[i]);
        m = warp_max(m);
        top = fminf(fmaxf(m, -FLT_MAX), FLT_MAX);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV * V; ++i) sum += l[i] > -INFINITY ? expf(fminf(l[i], FLT_MAX) - top) : 0.f;
        denominator = warp_allreduce_sum(sum);
    }
    uint32_t key[NV * V];
#pragma unroll
    for (int i = 0; i < NV * V; ++i) {
        const int e = (i / V * 32 + lane) * V + i % V;
        key[i] = order_key(l[i]);
        if (p.bias && key[i]) key[i] = order_key(sigmoid(l[i]) + p.bias[e]);
    }
    int mine = -1;
    uint32_t before = 0;
    bool close = false;
    float least = -INFINITY;
    const int rounds = p.bias ? p.k + 1 : p.k;            // one more: whether the first left out is close
    for (int j = 0; j < rounds; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < NV * V; ++i) m = max(m, key[i]);
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if (m == 0) break;
        uint32_t e = UINT32_MAX;
#pragma unroll
        for (int i = NV * V - 1; i >= 0; --i)
            if (key[i] == m) e = static_cast<uint32_t>((i / V * 32 + lane) * V + i % V);
        e = __reduce_min_sync(0xFFFFFFFFu, e);
#pragma unroll
        for (int i = 0; i < NV * V; ++i)
            if (e == static_cast<uint32_t>((i / V * 32 + lane) * V + i % V)) key[i] = 0;
        if (lane == j && j < p.k) mine = static_cast<int>(e);
        if (p.bias) {
            // an FP32 key is off by at most 4 u for the sigmoid (exp, sum, quotient)
            // and u |key| for the sum: two of them by less than 2^-20 (1 + |key|)
            const float v = key_value(m);
            close |= j > 0 && !(key_value(before) - v > 0x1p-20f * (1.f + fabsf(v)));
            before = m;
            if (j < p.k) least = v;
        }
    }
    // the least key that may be among the chosen: that of the k-th, less both errors
    if (close) mine = choose_in_64_bits<B16>(p, at, least - 0x1p-20f * (1.f + fabsf(least)), lane);
    float w = mine >= 0 ? fminf(logit_at<B16>(p.logits, at + mine), FLT_MAX) : 0.f;
    if (p.sigmoid) {
        if (p.renormalize) top = warp_max(mine >= 0 ? w : -INFINITY);
        w = mine < 0 ? 0.f : p.renormalize ? shared_sigmoid(w, top) : sigmoid(w);
    } else {
        if (p.renormalize) top = __shfl_sync(0xFFFFFFFFu, w, 0);   // the first chosen is the largest
        w = mine >= 0 ? expf(w - top) : 0.f;
    }
    if (p.renormalize) denominator = warp_allreduce_sum(w);
    if (p.sigmoid && !p.renormalize) denominator = 1.f;
    if (lane < p.k) {
        p.ids[t * p.k + lane] = mine;
        p.w[t * p.k + lane] = w > 0.f ? p.scale * (w / denominator) : 0.f;
    }
}

// d_logits: what every expert gets, then the chosen ones once more with their own part.
template <bool B16, int V, int NV>
__global__ void __launch_bounds__(32 * kGateWarps) gate_grad_kernel(const GateParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kGateWarps + (threadIdx.x >> 5);
    pdl_wait();
    pdl_launch_dependents();
    if (t >= p.T) return;
    const int64_t at = t * p.E;
    // lane j: the j-th chosen expert, its logit and the gradient of its weight
    int e = lane < p.k ? p.ids_in[t * p.k + lane] : -1;
    if (e >= p.E || (e < 0 && e != -1)) {
        atomicOr(p.status, MFR_STATUS_BAD_INDEX);
        e = -1;
    }
    const bool on = e >= 0;
    const float x = on ? logit_at<B16>(p.logits, at + e) : -INFINITY, le = fminf(x, FLT_MAX);
    const float g = on ? p.scale * p.d_w[t * p.k + lane] : 0.f;
    float d, all = 0.f;                                   // of the chosen; factor of p_e for every expert
    float l[NV * V];
    float top = 0.f, denominator = 1.f;
    if (p.sigmoid) {
        float q = on ? sigmoid(le) : 0.f;
        d = g;
        if (p.renormalize) {
            const float m = warp_max(x);              // all lanes, those without a slot too
            q = on ? shared_sigmoid(le, m) : 0.f;
            const float total = warp_allreduce_sum(q);
            q = total > 0.f ? q / total : 0.f;
            d = g - warp_allreduce_sum(g * q);
        }
        d = on ? d * q * sigmoid(-le) : 0.f;
    } else if (p.renormalize) {
        float m = warp_max(x);
        m = fminf(fmaxf(m, -FLT_MAX), FLT_MAX);
        float q = x > -INFINITY ? expf(le - m) : 0.f;
        const float total = warp_allreduce_sum(q);
        q = total > 0.f ? q / total : 0.f;
        d = q * (g - warp_allreduce_sum(g * q));
    } else {
        load_row<B16, V, NV>(p.logits, at, p.E, lane, l);
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NV * V; ++i) m = fmaxf(m, l[i]);
        m = warp_max(m);
        top = fminf(fmaxf(m, -FLT_MAX), FLT_MAX);
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV * V; ++i) {
            l[i] = l[i] > -INFINITY ? expf(fminf(l[i], FLT_MAX) - top) : 0.f;
            sum += l[i];
        }
        denominator = fmaxf(warp_allreduce_sum(sum), FLT_MIN);
        const float q = x > -INFINITY ? expf(le - top) / denominator : 0.f;
        all = -warp_allreduce_sum(g * q);
        d = q * g;
    }
    // the same expert in several slots: the first of them has the sum
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    float mine = d;
    for (int j = 0; j < p.k; ++j) {
        const float v = __shfl_sync(0xFFFFFFFFu, d, j);
        if (j != lane && (same >> j & 1u)) mine += v;
    }
    const float own = !p.sigmoid && !p.renormalize && on ? all * (x > -INFINITY ? expf(le - top) / denominator : 0.f) : 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int first = (v * 32 + lane) * V;
        if (first >= p.E) continue;
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = all != 0.f ? all * (l[v * V + i] / denominator) : 0.f;
        if constexpr (V == 4) {
            if constexpr (B16)
                st_u2(static_cast<uint16_t*>(p.d_logits) + at + first, make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])));
            else
                st_f4(static_cast<float*>(p.d_logits) + at + first, make_float4(o[0], o[1], o[2], o[3]));
        } else if constexpr (B16) {
            static_cast<__nv_bfloat16*>(p.d_logits)[at + first] = __float2bfloat16_rn(o[0]);
        } else {
            static_cast<float*>(p.d_logits)[at + first] = o[0];
        }
    }
    __syncwarp();                                         // the warp's own stores come in this order
    if (on && lane == __ffs(same) - 1) {
        if constexpr (B16) static_cast<__nv_bfloat16*>(p.d_logits)[at + e] = __float2bfloat16_rn(mine + own);
        else static_cast<float*>(p.d_logits)[at + e] = mine + own;
    }
}

using Kernel = void (*)(const GateParams);

template <bool B16, int V, int NV>
Kernel pick(bool grad) { return grad ? gate_grad_kernel<B16, V, NV> : gate_kernel<B16, V, NV>; }

// Four logits a load where rows start on such a boundary, else one.
template <bool B16>
Kernel kernel_for(int E, bool grad) {
    if (E % 4 == 0) {
        if (E <= 128) return pick<B16, 4, 1>(grad);
        if (E <= 256) return pick<B16, 4, 2>(grad);
        if (E <= 512) return pick<B16, 4, 4>(grad);
        return pick<B16, 4, 8>(grad);
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

cudaError_t gate_launch(const GateParams& p, int b16, bool grad, int pdl, cudaStream_t s) {
    return layer_launch(kernel_for(p.E, b16 != 0, grad), (p.T + kGateWarps - 1) / kGateWarps, 32 * kGateWarps, 0, 1, pdl, s, p);
}

}  // namespace mfr
