// The L2 norm of many tensors together, and the tensors scaled to a largest norm:
//
//   norm = sqrt(sum of all squares),  out = in * min(1, max_norm / (norm + eps))
//
// Bytes bound it: everything is read for the norm, then read again and written.
// Two launches over the same pieces of the tensors (up to 64 KB each): the first
// leaves a sum of squares a CTA, the second adds those in a fixed order, each CTA
// for itself, and scales the pieces from the last to the first, so that what the
// first launch read last still lies in L2.
// A thread adds up to 130 squares of a piece in FP32 in four chains, and where their
// sum leaves FP32 adds them once more at a smaller scale; its pieces' sums and
// everything above are 64 bits.  No atomics: the same bits in every call.
// Measured on GB300: 60 tensors of 700 M elements, 1.85 GB, in place, 847 to 860 us: the
// first launch 252 us (7.3 TB/s), the second 557 (6.65 TB/s, of a copy rate of 6.78).
// Tensors beyond kClipGroup are further pairs of launches, and every CTA of each second
// launch adds the sums of all first ones: 2000 tensors of 65536 FP32 elements 167 us, 8192
// of 16384 558 us (three passes: 238), 65536 of 4096 16.8 ms (475 us).
#include "moe_step_ops.h"
#include "mfr_device.cuh"
#include "mfr_layer.h"
#include "mfr_step.h"

namespace mfr {
namespace {

constexpr int kClipThreads = 256;
constexpr int kClipCtas = 6;             // an SM

// The tensor that piece c belongs to.
template <int N>
__device__ __forceinline__ int tensor_of(const ClipList<N>& l, uint32_t c) {
    int lo = 0, hi = l.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (l.first[mid] <= c) lo = mid;
        else hi = mid;
    }
    return lo;
}

// What a piece covers: whole 16-byte vectors behind the tensor's first boundary, and
// for the first and the last piece of a tensor the elements before and behind them.
struct Piece {
    int64_t head;          // elements before the first boundary
    int64_t v0, v1;        // vectors of this piece
    int64_t tail;          // first element behind the last vector
    bool first, last;
};

__device__ __forceinline__ Piece piece_of(const void* in, int64_t n, bool f32, uint32_t index, int64_t vectors) {
    Piece p;
    const int to = static_cast<int>(16 - (reinterpret_cast<uintptr_t>(in) & 15)) & 15;
    const int head = f32 ? to >> 2 : to >> 1, shift = f32 ? 2 : 3;      // elements of a vector: 4 or 8
    p.head = head < n ? head : n;
    const int64_t all = (n - p.head) >> shift;
    p.tail = p.head + (all << shift);
    p.v0 = index * vectors;
    p.v1 = p.v0 + vectors < all ? p.v0 + vectors : all;
    p.first = index == 0;
    // the count of pieces is fixed by n alone, so the last piece may hold no vector
    p.last = ((static_cast<int64_t>(index) + 1) * vectors << shift) >= n;
    return p;
}

__device__ __forceinline__ float element(const void* p, int64_t i, int type) {
    if (type == MFR_GRAD_F32) return static_cast<const float*>(p)[i];
    const uint16_t u = static_cast<const uint16_t*>(p)[i];
    return type == MFR_GRAD_BF16 ? __uint_as_float(static_cast<uint32_t>(u) << 16) : __half2float(__ushort_as_half(u));
}

__device__ __forceinline__ void set_element(void* p, int64_t i, int type, float v) {
    if (type == MFR_GRAD_F32) static_cast<float*>(p)[i] = v;
    else if (type == MFR_GRAD_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// The values of a vector: 4 or 8.
__device__ __forceinline__ void unpack(uint4 v, int type, float (&f)[8]) {
    if (type == MFR_GRAD_F32) {
        f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
        f[4] = f[5] = f[6] = f[7] = 0.f;
    } else if (type == MFR_GRAD_BF16) {
        unpack8(v, f);
    } else {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            f[2 * i] = x.x;
            f[2 * i + 1] = x.y;
        }
    }
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint4 pack(const float (&f)[8], int type) {
    if (type == MFR_GRAD_F32)
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    if (type == MFR_GRAD_BF16)
        return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    return make_uint4(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]), pack_half2(f[4], f[5]), pack_half2(f[6], f[7]));
}

// With a factor of 1 the bits are copied as they are, NaNs too.
__device__ __forceinline__ void scale_element(const void* in, void* out, int64_t i, int type, float scale) {
    if (scale != 1.f) set_element(out, i, type, element(in, i, type) * scale);
    else if (type == MFR_GRAD_F32) static_cast<uint32_t*>(out)[i] = static_cast<const uint32_t*>(in)[i];
    else static_cast<uint16_t*>(out)[i] = static_cast<const uint16_t*>(in)[i];
}

__device__ __forceinline__ uint4 scaled(uint4 v, int type, float scale) {
    if (scale == 1.f) return v;
    float f[8];
    unpack(v, type, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= scale;
    return pack(f, type);
}

__device__ __forceinline__ double warp_sum(double v) {
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

// Sum over the CTA in a fixed order; every thread gets it.
__device__ __forceinline__ double block_sum(double v, double* s) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    double sum = 0.0;
    for (int i = 0; i < kClipThreads / 32; ++i) sum += s[i];
    return sum;
}

// This thread's squares of a piece once more, where their FP32 sum is infinite though each
// of them may be finite: at 2^-8, which 130 of them at most do not leave.
__device__ __forceinline__ double wide_sum(const void* in, int64_t n, int type, const Piece& q) {
    const int per = type == MFR_GRAD_F32 ? 4 : 8;
    float a = 0.f;
    const auto add = [&](int64_t i) {
        const float f = element(in, i, type);
        a = fmaf(f * f, 0x1p-8f, a);
    };
#pragma unroll 1
    for (int64_t at = q.v0 + threadIdx.x; at < q.v1; at += kClipThreads)
#pragma unroll 1
        for (int e = 0; e < per; ++e) add(q.head + at * per + e);
    if (q.first && threadIdx.x < q.head) add(threadIdx.x);
    if (q.last && q.tail + threadIdx.x < n) add(q.tail + threadIdx.x);
    return 256.0 * static_cast<double>(a);
}

template <int N>
__global__ void __launch_bounds__(kClipThreads, kClipCtas) squares_kernel(const __grid_constant__ ClipList<N> l, const ClipParams p) {
    __shared__ double s[kClipThreads / 32];
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    double sum = 0.0;
    for (uint32_t c = blockIdx.x; c < l.first[l.n]; c += gridDim.x) {
        const int i = tensor_of(l, c), type = l.type[i], size = type == MFR_GRAD_F32 ? 4 : 2;
        const void* in = l.in[i];
        const int64_t n = l.numel[i];
        const Piece q = piece_of(in, n, type == MFR_GRAD_F32, c - l.first[i], p.vectors);
        const uint4* v = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(in) + q.head * size);
        float a[4] = {0.f, 0.f, 0.f, 0.f};
        int64_t at = q.v0 + tid;
        for (; at + 3 * kClipThreads < q.v1; at += 4 * kClipThreads) {
            uint4 x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = ld_stream_u4(v + at + k * kClipThreads);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float f[8];
                unpack(x[k], type, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) a[k] = fmaf(f[e], f[e], a[k]);
            }
        }
        for (; at < q.v1; at += kClipThreads) {
            float f[8];
            unpack(ld_stream_u4(v + at), type, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) a[0] = fmaf(f[e], f[e], a[0]);
        }
        if (q.first && tid < q.head) {
            const float f = element(in, tid, type);
            a[1] = fmaf(f, f, a[1]);
        }
        if (q.last && q.tail + tid < n) {
            const float f = element(in, q.tail + tid, type);
            a[2] = fmaf(f, f, a[2]);
        }
        const float chains = (a[0] + a[1]) + (a[2] + a[3]);
        sum += chains < INFINITY || chains != chains ? static_cast<double>(chains) : wide_sum(in, n, type, q);
    }
    sum = block_sum(sum, s);
    if (tid == 0) p.partial[p.partial_at + blockIdx.x] = sum;
}

template <int N>
__global__ void __launch_bounds__(kClipThreads, kClipCtas) scale_kernel(const __grid_constant__ ClipList<N> l, const ClipParams p) {
    __shared__ double s[kClipThreads / 32];
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    double sum = 0.0;
    for (int i = tid; i < p.partials; i += kClipThreads) sum += __ldcg(p.partial + i);
    sum = block_sum(sum, s);
    const float norm = static_cast<float>(sqrt(sum));
    if (blockIdx.x == 0 && tid == 0 && p.partial_at == 0) *p.norm = norm;
    // not finite: the tensors keep their values
    float scale = 1.f;
    if (norm < INFINITY) scale = fminf(p.max_norm / (norm + p.eps), 1.f);
    const uint32_t pieces = l.first[l.n];
    for (uint32_t r = blockIdx.x; r < pieces; r += gridDim.x) {
        const uint32_t c = pieces - 1 - r;
        const int i = tensor_of(l, c), type = l.type[i], size = type == MFR_GRAD_F32 ? 4 : 2;
        const void* in = l.in[i];
        void* out = l.out[i];
        if (in == out && scale == 1.f) continue;
        const int64_t n = l.numel[i];
        const Piece q = piece_of(in, n, type == MFR_GRAD_F32, c - l.first[i], p.vectors);
        if (q.first && tid < q.head) scale_element(in, out, tid, type, scale);
        if (q.last && q.tail + tid < n) scale_element(in, out, q.tail + tid, type, scale);
        if (((reinterpret_cast<uintptr_t>(in) ^ reinterpret_cast<uintptr_t>(out)) & 15) != 0) {
            const int per = 16 / size;
            for (int64_t e = q.head + q.v0 * per + tid; e < q.head + q.v1 * per; e += kClipThreads)
                scale_element(in, out, e, type, scale);
            continue;
        }
        const uint4* v = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(in) + q.head * size);
        uint4* o = reinterpret_cast<uint4*>(static_cast<uint8_t*>(out) + q.head * size);
        int64_t at = q.v0 + tid;
        for (; at + 3 * kClipThreads < q.v1; at += 4 * kClipThreads) {
            uint4 x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = ld_stream_u4(v + at + k * kClipThreads);
#pragma unroll
            for (int k = 0; k < 4; ++k) st_stream_u4(o + at + k * kClipThreads, scaled(x[k], type, scale));
        }
        for (; at < q.v1; at += kClipThreads) st_stream_u4(o + at, scaled(ld_stream_u4(v + at), type, scale));
    }
}

template <int N>
cudaError_t launch_group(const ClipShape& s, const ClipParams& base, const void* const* in, void* const* out, int from, int n,
                         int group, bool scale, int pdl, cudaStream_t st) {
    ClipList<N> l;
    l.n = n;
    uint32_t pieces = 0;
    for (int i = 0; i < n; ++i) {
        l.in[i] = in[from + i];
        l.out[i] = out[from + i];
        l.numel[i] = s.numel[from + i];
        l.type[i] = s.type[from + i];
        l.first[i] = pieces;
        pieces += s.pieces[from + i];
    }
    l.first[n] = pieces;
    ClipParams p = base;
    p.partial_at = group * s.grid;
    return scale ? layer_launch(scale_kernel<N>, s.grid, kClipThreads, 0, 1, pdl, st, l, p)
                 : layer_launch(squares_kernel<N>, s.grid, kClipThreads, 0, 1, pdl, st, l, p);
}

}  // namespace

// Pieces of 64 KB; smaller ones, to 4 KB, where that many would leave SMs idle.
void clip_choose(ClipShape& s, int sms) {
    int64_t bytes = 0;
    for (int i = 0; i < s.n; ++i) bytes += s.numel[i] * (s.type[i] == MFR_GRAD_F32 ? 4 : 2);
    s.vectors = kClipMaxVectors;
    while (s.vectors > kClipThreads && bytes < static_cast<int64_t>(s.vectors) * 16 * sms * 4) s.vectors /= 2;
    for (int i = 0; i < s.n; ++i) {
        const int64_t per = static_cast<int64_t>(s.vectors) * (s.type[i] == MFR_GRAD_F32 ? 4 : 8);
        s.pieces[i] = static_cast<uint32_t>((s.numel[i] + per - 1) / per);
    }
    s.groups = s.n <= kClipGroup ? 1 : (s.n + kClipGroup - 1) / kClipGroup;
    int64_t most = 1;
    for (int g = 0; g < s.groups; ++g) {
        int64_t pieces = 0;
        for (int i = g * kClipGroup; i < s.n && i < (g + 1) * kClipGroup; ++i) pieces += s.pieces[i];
        if (pieces > most) most = pieces;
    }
    s.grid = static_cast<int>(most < sms * kClipCtas ? most : sms * kClipCtas);
}

cudaError_t clip_prepare() {
    cudaError_t e = preload(squares_kernel<kClipFew>);
    if (e == cudaSuccess) e = preload(scale_kernel<kClipFew>);
    if (e == cudaSuccess) e = preload(squares_kernel<kClipGroup>);
    if (e == cudaSuccess) e = preload(scale_kernel<kClipGroup>);
    return e;
}

cudaError_t clip_launch(const ClipShape& s, const ClipParams& p, const void* const* in, void* const* out, int pdl, cudaStream_t st) {
    for (int scale = 0; scale < 2; ++scale)
        for (int g = 0; g < s.groups; ++g) {
            const int from = g * kClipGroup, n = s.n - from < kClipGroup ? s.n - from : kClipGroup;
            const cudaError_t e = n <= kClipFew ? launch_group<kClipFew>(s, p, in, out, from, n, g, scale != 0, pdl, st)
                                                : launch_group<kClipGroup>(s, p, in, out, from, n, g, scale != 0, pdl, st);
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}

}  // namespace mfr
