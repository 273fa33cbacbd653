// kda_layernorm.cuh -- layer norm of rows of D values, forward and backward.
//
//   y = (x - m) r w + b,   m = mean x,   r = (mean (x - m)^2 + eps)^{-1/2}
//   dx = r (u - mean u - xh mean(u xh)),   u = dy w,   xh = (x - m) r
//   dw = sum dy xh,   db = sum dy     over the rows that share a weight row
//
// Rows are [T, G, D] with weights [G, D]: G = 1 is the norm of a stream, G = H
// that of each head's output.  Bound by memory: a row is read once into
// registers, where the mean and then the centred square are summed in fp32 (two
// passes over registers, so no cancellation in the variance).
//
// A row is shared by kTpr threads (a part of a warp, a warp, or a block) with up
// to kNV vectors of V elements each.  Backward: a block keeps to one group g and
// walks tokens, so a thread always meets the same columns and sums dw, db in
// registers; the row groups of a block meet in shared memory, one partial per
// block goes to the workspace, and a second kernel adds the partials in order (no
// atomics: results do not depend on the schedule).
#pragma once

#include "kda_rotary.cuh"

namespace kda {
namespace ln {

using rotary::Vec;

template <int kTpr>
struct Block {
    static constexpr int kThreads = kTpr < 256 ? 256 : kTpr;
    static constexpr int kRows = kThreads / kTpr;
};

// Sum of two values over the kTpr threads of a row.
template <int kTpr>
__device__ __forceinline__ float2 row_sum2(float2 x, float2 *red) {
#pragma unroll
    for (int o = (kTpr < 32 ? kTpr : 32) / 2; o > 0; o >>= 1) {
        x.x += __shfl_xor_sync(0xffffffffu, x.x, o);
        x.y += __shfl_xor_sync(0xffffffffu, x.y, o);
    }
    if (kTpr > 32) {
        constexpr int W = kTpr / 32;
        const int w = threadIdx.x / 32, first = threadIdx.x / kTpr * W;
        __syncthreads();                                // the last use of red is over
        if (threadIdx.x % 32 == 0) red[w] = x;
        __syncthreads();
        x = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            x.x += red[first + i].x;
            x.y += red[first + i].y;
        }
    }
    return x;
}

template <typename T, int V, int kTpr, int kNV>
__global__ void __launch_bounds__(Block<kTpr>::kThreads)
fwd_kernel(const T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ b,
           int64_t rows, int G, int D, float eps, T *__restrict__ y, float *__restrict__ mean,
           float *__restrict__ rstd) {
    __shared__ float2 red[Block<kTpr>::kThreads / 32];
    const int64_t row = (int64_t)blockIdx.x * Block<kTpr>::kRows + threadIdx.x / kTpr;
    const int lane = threadIdx.x % kTpr;
    const bool live = row < rows;
    float v[kNV][V];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        const int c = (lane + i * kTpr) * V;
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] = 0.f;
        if (live && c < D) {
            Vec<T, V>::ld(x + row * D + c, v[i]);
#pragma unroll
            for (int j = 0; j < V; ++j) s += v[i][j];
        }
    }
    const float m = row_sum2<kTpr>(make_float2(s, 0.f), red).x / (float)D;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i)
        if ((lane + i * kTpr) * V < D)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[i][j] -= m;
                s = fmaf(v[i][j], v[i][j], s);
            }
    const float r = rsqrtf(row_sum2<kTpr>(make_float2(s, 0.f), red).x / (float)D + eps);
    if (!live) return;
    const size_t wrow = (size_t)(row % G) * D;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
        const int c = (lane + i * kTpr) * V;
        if (c >= D) continue;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            v[i][j] *= r;
            if (w != nullptr) v[i][j] *= w[wrow + c + j];
            if (b != nullptr) v[i][j] += b[wrow + c + j];
        }
        Vec<T, V>::st(y + row * D + c, v[i]);
    }
    if (lane == 0) {
        mean[row] = m;
        rstd[row] = r;
    }
}

// grid (blocks along T, G).  part: [blocks][2][G][D], dw then db.
template <typename T, int V, int kTpr, int kNV>
__global__ void __launch_bounds__(Block<kTpr>::kThreads)
bwd_kernel(const T *__restrict__ dy, const T *__restrict__ x, const float *__restrict__ mean,
           const float *__restrict__ rstd, const float *__restrict__ w, int64_t tokens, int G,
           int D, T *__restrict__ dx, float *__restrict__ part) {
    using B = Block<kTpr>;
    __shared__ float2 red[B::kThreads / 32];
    extern __shared__ float acc[];                      // [kRows][D] where kRows > 1
    const int g = blockIdx.y, lane = threadIdx.x % kTpr, rg = threadIdx.x / kTpr;
    float dw[kNV][V], db[kNV][V], wv[kNV][V];
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int c = (lane + i * kTpr) * V + j;
            dw[i][j] = db[i][j] = 0.f;
            wv[i][j] = c < D ? (w != nullptr ? w[(size_t)g * D + c] : 1.f) : 0.f;
        }
    const int64_t step = (int64_t)gridDim.x * B::kRows;
    const int64_t trips = (tokens + step - 1) / step;   // the same for every thread
    for (int64_t it = 0; it < trips; ++it) {
        const int64_t t = it * step + (int64_t)blockIdx.x * B::kRows + rg;
        const bool live = t < tokens;
        const int64_t row = t * G + g;
        const float m = live ? mean[row] : 0.f, r = live ? rstd[row] : 0.f;
        float xh[kNV][V], u[kNV][V];
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            const int c = (lane + i * kTpr) * V;
#pragma unroll
            for (int j = 0; j < V; ++j) xh[i][j] = u[i][j] = 0.f;
            if (live && c < D) {
                Vec<T, V>::ld(x + row * D + c, xh[i]);
                Vec<T, V>::ld(dy + row * D + c, u[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < kNV; ++i)
            if (live && (lane + i * kTpr) * V < D)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    xh[i][j] = (xh[i][j] - m) * r;
                    dw[i][j] = fmaf(u[i][j], xh[i][j], dw[i][j]);
                    db[i][j] += u[i][j];
                    u[i][j] *= wv[i][j];
                    s.x += u[i][j];
                    s.y = fmaf(u[i][j], xh[i][j], s.y);
                }
        s = row_sum2<kTpr>(s, red);
        s.x /= (float)D;
        s.y /= (float)D;
        if (live)
#pragma unroll
            for (int i = 0; i < kNV; ++i) {
                const int c = (lane + i * kTpr) * V;
                if (c >= D) continue;
#pragma unroll
                for (int j = 0; j < V; ++j) u[i][j] = r * (u[i][j] - s.x - xh[i][j] * s.y);
                Vec<T, V>::st(dx + row * D + c, u[i]);
            }
    }
    if (part == nullptr) return;
    float *out = part + ((size_t)blockIdx.x * 2 * G + g) * D;
#pragma unroll
    for (int which = 0; which < 2; ++which, out += (size_t)G * D) {
        if (B::kRows == 1) {
#pragma unroll
            for (int i = 0; i < kNV; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int c = (lane + i * kTpr) * V + j;
                    if (c < D) out[c] = which ? db[i][j] : dw[i][j];
                }
            continue;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kNV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int c = (lane + i * kTpr) * V + j;
                if (c < D) acc[rg * D + c] = which ? db[i][j] : dw[i][j];
            }
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += B::kThreads) {
            float a = 0.f;
            for (int i = 0; i < B::kRows; ++i) a += acc[i * D + c];
            out[c] = a;
        }
    }
}

// dw[e] = sum over blocks of part[block][0][e], db alike.  A block owns 32
// columns; 8 warps sum every eighth partial and meet in shared memory.
__global__ void __launch_bounds__(256)
weight_sum_kernel(const float *__restrict__ part, int blocks, int64_t n, float *__restrict__ dw,
                  float *__restrict__ db) {
    __shared__ float red[8][33];
    const int64_t e = (int64_t)blockIdx.x * 32 + threadIdx.x % 32;
    const int wrp = threadIdx.x / 32;
    const float *p = part + (blockIdx.y ? n : 0);
    float *out = blockIdx.y ? db : dw;
    float s = 0.f;
    if (e < n)
        for (int i = wrp; i < blocks; i += 8) s += p[(size_t)i * 2 * n + e];
    red[wrp][threadIdx.x % 32] = s;
    __syncthreads();
    if (wrp == 0 && e < n && out != nullptr) {
        float a = 0.f;
        for (int i = 0; i < 8; ++i) a += red[i][threadIdx.x];
        out[e] = a;
    }
}

}  // namespace ln
}  // namespace kda
