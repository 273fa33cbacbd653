// kda_rotary.cuh -- rotary positions of q and k, in one memory-bound pass.
//
// Channels (x, y) of pair i of a head turn by the angle pos * f_i:
//   x' = scale (x cos - y sin),   y' = scale (x sin + y cos)
// over the first `rot` channels of each head; the others are copied (or left,
// when the output is the input).  Pairs are neighbours (2 i, 2 i + 1), or the
// two halves (i, i + rot / 2).  The inverse turns by the negated angle, which is
// also the gradient.
//
// Angles of far positions: fp32 loses pos * f to 0.06 rad at a million tokens, so
// the product is formed in revolutions in fp64, with what its roundings leave (at
// 2^31 alone they are off by 5e-7 rad), reduced to [-1/2, 1/2] there, and only then
// given to sincospi in fp32 (2e-7 rad).  A block computes the rot / 2 angles of its
// tokens once, into shared memory, for all of its heads: with H heads that is one
// angle per 2 H values.
//
// Measured: q and k of 8,192 tokens, 96 heads of 128 139 us (5.8 TB/s); a step of 256
// tokens, 96 and 8 heads, half of 128 channels turned 5.3 us, most of it the fp64
// angles and the latency of one wave.
//
// A work item is two 16-byte vectors (the two halves of pairs, or 8 bf16 / 4 fp32
// consecutive pairs members); sizes that do not allow 16-byte accesses take the
// same kernel with single elements.
#pragma once

#include "kda_common.cuh"

namespace kda {
namespace rotary {

constexpr int kThreads = 256;
constexpr int kMaxHalf = 128;          // rot / 2 at most
constexpr int kMaxTokens = 32;         // tokens of a block

struct Args {
    const int32_t *pos;                // [T], or NULL: the index in the sequence
    const int32_t *cu;
    int N;
    int64_t T;
    int Hq, Hk, d, rot;
    int inverse;
    float scale;
    int64_t q_stride, k_stride, qo_stride, ko_stride;   // elements between tokens
    int tokens;                        // of a block
    int heads;                         // of a block, over q then k
};

template <typename T, int V>
struct Vec;
template <typename T>
struct Vec<T, 1> {
    static __device__ __forceinline__ void ld(const T *p, float (&x)[1]) { x[0] = IO<T>::ld(p); }
    static __device__ __forceinline__ void st(T *p, const float (&x)[1]) { IO<T>::st(p, x[0]); }
};
template <>
struct Vec<__nv_bfloat16, 2> {
    static __device__ __forceinline__ void ld(const __nv_bfloat16 *p, float (&x)[2]) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
        x[0] = __uint_as_float(w << 16);
        x[1] = __uint_as_float(w & 0xffff0000u);
    }
    static __device__ __forceinline__ void st(__nv_bfloat16 *p, const float (&x)[2]) {
        *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(x[0], x[1]);
    }
};
template <>
struct Vec<float, 4> {
    static __device__ __forceinline__ void ld(const float *p, float (&x)[4]) {
        const float4 a = *reinterpret_cast<const float4 *>(p);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    }
    static __device__ __forceinline__ void st(float *p, const float (&x)[4]) {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    }
};
template <>
struct Vec<__nv_bfloat16, 8> {
    static __device__ __forceinline__ void ld(const __nv_bfloat16 *p, float (&x)[8]) {
        const uint4 r = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void st(__nv_bfloat16 *p, const float (&x)[8]) {
        uint4 r;
        uint32_t *w = reinterpret_cast<uint32_t *>(&r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<uint32_t *>(&b);
        }
        *reinterpret_cast<uint4 *>(p) = r;
    }
};

// Position of token t: given, or its index in its sequence.
__device__ __forceinline__ int64_t position(const Args &a, int64_t t) {
    if (a.pos != nullptr) return a.pos[t];
    if (a.cu == nullptr) return t % (a.T / a.N);
    int lo = 0, hi = a.N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)a.cu[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return t - a.cu[lo];
}

// pos * f / 2 pi less its nearest whole number: 1 / 2 pi and both products as sums of
// two doubles.
__device__ __forceinline__ double turns(int64_t pos, float f) {
    constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
    const double x = f, p = (double)pos;
    const double hi = x * kHi, lo = fma(x, kHi, -hi) + x * kLo;
    const double t = p * hi;
    return (t - rint(t)) + (fma(p, hi, -t) + p * lo);
}

// grid (token tiles, head slices).  V = 1 or a full 16-byte vector; kPairs:
// neighbours are paired.  One work item of a head is V pairs: for halves the
// vectors at i and i + rot / 2, for neighbours the 2 V values at 2 i (two
// vectors).  Items behind the pairs copy one vector each.
template <typename T, int V, bool kPairs>
__global__ void __launch_bounds__(kThreads)
rotary_kernel(const T *q, const T *k, const float *__restrict__ freq, Args a, T *qo, T *ko) {
    __shared__ float2 cs[kMaxTokens * kMaxHalf];
    const int half = a.rot / 2;
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
    const int nt = (int)(a.T - t0 < a.tokens ? a.T - t0 : a.tokens);
    if (a.pos == nullptr && a.cu != nullptr && blockIdx.x == 0 && blockIdx.y == 0) {
        bool ok = true;
        for (int i = threadIdx.x; i < a.N; i += kThreads) ok = ok && a.cu[i] <= a.cu[i + 1];
        if (threadIdx.x == 0) ok = ok && a.cu[0] == 0 && (int64_t)a.cu[a.N] == a.T;
        if (!ok) raise_error(kErrSeqlens);
    }
    for (int e = threadIdx.x; e < nt * half; e += kThreads) {
        float s, c;
        sincospif((float)(2.0 * turns(position(a, t0 + e / half), freq[e % half])), &s, &c);
        cs[e] = make_float2(c * a.scale, (a.inverse ? -s : s) * a.scale);
    }
    __syncthreads();
    const int h0 = blockIdx.y * a.heads, heads = a.Hq + a.Hk;
    const int nh = heads - h0 < a.heads ? heads - h0 : a.heads;
    const int turn = half / V;                       // items that turn, per head
    const int items = turn + (a.d - a.rot) / V;
    for (int e = threadIdx.x; e < nt * nh * items; e += kThreads) {
        const int i = e % items, w = e / items;
        const int h = h0 + w % nh, lt = w / nh;
        const int64_t t = t0 + lt;
        const bool is_q = h < a.Hq;
        const T *src = is_q ? q + t * a.q_stride + (int64_t)h * a.d
                            : k + t * a.k_stride + (int64_t)(h - a.Hq) * a.d;
        T *dst = is_q ? qo + t * a.qo_stride + (int64_t)h * a.d
                      : ko + t * a.ko_stride + (int64_t)(h - a.Hq) * a.d;
        float x[V], y[V];
        if (i >= turn) {                             // channels that do not turn
            if (src != dst) {
                const int c = a.rot + (i - turn) * V;
                Vec<T, V>::ld(src + c, x);
                Vec<T, V>::st(dst + c, x);
            }
            continue;
        }
        const float2 *p = cs + lt * half + i * V;
        const int c = kPairs ? 2 * i * V : i * V, c2 = kPairs ? c + V : c + half;
        Vec<T, V>::ld(src + c, x);
        Vec<T, V>::ld(src + c2, y);
        if (kPairs && V > 1) {                       // x, y hold 2 V values, pairs adjacent
#pragma unroll
            for (int j = 0; j < V; j += 2) {
                const float2 f = p[j / 2], f2 = p[V / 2 + j / 2];
                const float x0 = x[j], x1 = x[(j + 1) % V], y0 = y[j], y1 = y[(j + 1) % V];
                x[j] = x0 * f.x - x1 * f.y;
                x[(j + 1) % V] = x0 * f.y + x1 * f.x;
                y[j] = y0 * f2.x - y1 * f2.y;
                y[(j + 1) % V] = y0 * f2.y + y1 * f2.x;
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float2 f = p[j];
                const float x0 = x[j], y0 = y[j];
                x[j] = x0 * f.x - y0 * f.y;
                y[j] = x0 * f.y + y0 * f.x;
            }
        }
        Vec<T, V>::st(dst + c, x);
        Vec<T, V>::st(dst + c2, y);
    }
}

}  // namespace rotary
}  // namespace kda
