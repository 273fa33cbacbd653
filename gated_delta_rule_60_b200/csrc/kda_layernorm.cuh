// kda_layernorm.cuh -- layer norm of rows of D values, forward and backward.
//
//   y = (x - m) r w + b,   m = mean x,   r = (mean (x - m)^2 + eps)^{-1/2}
//   dx = r (u - mean u - xh mean(u xh)),   u = dy w,   xh = (x - m) r
//   dw = sum dy xh,   db = sum dy     over the rows that share a weight row
//
// Rows are [T, G, D] with weights [G, D]: G = 1 is the norm of a stream, G = H
// that of each head's output.  Bound by memory: a row is read once into registers.
//
// A row is shared by kTpr threads (a part of a warp, a warp, or a block) with up
// to kNV vectors of V elements each; a block of kRows such rows takes kGs
// neighbouring groups of kRows / kGs tokens at a time (rows that are neighbours in
// memory), always the same groups, and walks along the tokens with the loads of two
// steps in flight.  So a thread always meets the same columns, and the gradient sums
// dw and db in registers; the tokens of a block meet in shared memory, one partial
// per block goes to the workspace, and a second kernel adds the partials in order
// (no atomics: results do not depend on the schedule).
//
// The work per value is small, so instructions bound it before memory does unless
// they are few: packed fp32 pairs, pointers that advance by a constant, rows of up to
// 512 values with their weights (and, for the gradient, both factors of a row) in
// registers.  Longer rows take 64 bytes a thread (32 bf16 or 16 fp32 values, so that
// two blocks' rows fit an SM) and are read a second time from where they lie.  The
// mean, then the centred square, are summed over the row's values: none of the
// cancellation of sum x^2 - (sum x)^2 / D.
//
// Measured (bf16): 8,192 x 96 rows of 128, forward 68 us (5.9 TB/s), backward 102 us
// (5.9 TB/s); 4,099 rows of 5,000, forward 30 us (2.8 TB/s), backward 47 us (2.6 TB/s:
// two barriers a row and few rows a block to hide them), the sum of its partials 5 us.
#pragma once

#include "kda_rotary.cuh"

namespace kda {
namespace ln {

using rotary::Vec;

template <int kTpr>
struct Block {
    static constexpr int kThreads = kTpr < 256 ? 256 : kTpr;
    static constexpr int kRows = kThreads / kTpr;
    static constexpr int kWarps = kThreads / 32;
    static constexpr bool kShort = kTpr <= 32;
};

// A thread's vectors of kArrays rows, two steps ahead: asynchronous copies into
// places of shared memory that only this thread reads (no barrier; registers hold
// the row that is being worked on alone).  Single 16-bit elements (odd D), which
// cannot be copied so, are loaded when they are needed.
constexpr int kStages = 3;

template <typename T, int V, int kNV, int kThreads, int kArrays>
struct Feed {
    static constexpr int kBytes = V * (int)sizeof(T);
    static constexpr bool kAsync = kBytes >= 4;
    static constexpr size_t kSmem = kAsync ? (size_t)kStages * kArrays * kNV * kThreads * kBytes : 0;
    unsigned char *at;
    __device__ __forceinline__ explicit Feed(unsigned char *smem) : at(smem + threadIdx.x * kBytes) {}
    __device__ __forceinline__ unsigned char *slot(int stage, int array, int i) {
        return at + ((stage * kArrays + array) * kNV + i) * kThreads * kBytes;
    }
    __device__ __forceinline__ void ask(int stage, int array, int i, const T *p) {
        if (kAsync) {
            const uint32_t d = (uint32_t)__cvta_generic_to_shared(slot(stage, array, i));
            if (kBytes == 16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(p) : "memory");
            else
                asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(p), "n"(kBytes)
                             : "memory");
        }
    }
    __device__ __forceinline__ void close() {
        if (kAsync) asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // everything but the two latest groups is there
    __device__ __forceinline__ void wait() {
        if (kAsync) asm volatile("cp.async.wait_group 2;" ::: "memory");
    }
    __device__ __forceinline__ void get(int stage, int array, int i, const T *p, float (&x)[V]) {
        Vec<T, V>::ld(kAsync ? reinterpret_cast<const T *>(slot(stage, array, i)) : p, x);
    }
};

// The columns of a thread: vector i at (lane + i kTpr) V.  kFull: all below D.
template <int V, int kTpr, int kNV, bool kFull>
struct Columns {
    int lane, D;
    __device__ __forceinline__ int at(int i) const { return (lane + i * kTpr) * V; }
    __device__ __forceinline__ bool in(int i) const { return kFull || at(i) < D; }
    // fp32 values of vector i's columns (fill without an array)
    __device__ __forceinline__ void weights(const float *w, float fill, int i, float *x) const {
#pragma unroll
        for (int j = 0; j < V; j += V < 4 ? V : 4) {
            if (w == nullptr || !in(i)) {
#pragma unroll
                for (int k = 0; k < (V < 4 ? V : 4); ++k) x[j + k] = fill;
            } else if (V < 4) {
#pragma unroll
                for (int k = 0; k < (V < 4 ? V : 4); ++k) x[j + k] = w[at(i) + k];
            } else {
                const float4 f = *reinterpret_cast<const float4 *>(w + at(i) + j);
                x[j] = f.x;
                x[j + 1] = f.y;
                x[j + 2] = f.z;
                x[j + 3] = f.w;
            }
        }
    }
};

// Sum over the threads of a row; red: a place per warp of its own for every use
// that another may still be reading.
template <int kTpr>
__device__ __forceinline__ float row_sum(float x, float *red) {
#pragma unroll
    for (int o = (kTpr < 32 ? kTpr : 32) / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (kTpr <= 32) return x;
    constexpr int W = kTpr < 32 ? 1 : kTpr / 32;
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) x += red[threadIdx.x / kTpr * W + i];
    return x;
}

// Where a row group walks: tokens first, first + step, ...
struct Rows {
    int64_t first, step;
    int g;
};
template <int kTpr>
__device__ __forceinline__ Rows make_rows(int gs) {
    const int rg = threadIdx.x / kTpr, ts = Block<kTpr>::kRows / gs;
    return {(int64_t)blockIdx.x * ts + rg / gs, (int64_t)gridDim.x * ts, (int)blockIdx.y * gs + rg % gs};
}

// Arithmetic on V values: packed pairs where V is even.
template <int V, typename F2, typename F1>
__device__ __forceinline__ void each(F2 two, F1 one) {
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int j = 0; j < V; j += 2) two(j);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) one(j);
    }
}
__device__ __forceinline__ float2 pair(const float *x) { return make_float2(x[0], x[1]); }
__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }
__device__ __forceinline__ void put(float *x, float2 v) {
    x[0] = v.x;
    x[1] = v.y;
}

// Blocks an SM that the registers are to allow.
template <int kTpr, bool kBwd>
constexpr int min_blocks() {
    return kTpr > 256 ? (kBwd ? 1 : 2) : Block<kTpr>::kShort ? (kBwd ? 2 : 3) : (kBwd ? 2 : 4);
}

template <typename T, int V, int kTpr, int kNV, bool kFull>
__global__ void __launch_bounds__(Block<kTpr>::kThreads, (min_blocks<kTpr, false>()))
fwd_kernel(const T *x, const float *__restrict__ w, const float *__restrict__ b, int64_t tokens,
           int G, int gs, int D, float eps, T *y, float *__restrict__ mean, float *__restrict__ rstd) {
    using B = Block<kTpr>;
    using namespace sm100;
    constexpr int N = kNV * V, K = B::kShort ? N : V;  // values kept: all, or a vector at a time
    __shared__ float red[2][2][B::kWarps];
    extern __shared__ __align__(16) unsigned char raw[];
    const Rows rows = make_rows<kTpr>(gs);
    const Columns<V, kTpr, kNV, kFull> col = {(int)threadIdx.x % kTpr, D};
    const float *wg = w == nullptr ? nullptr : w + (size_t)rows.g * D;
    const float *bg = b == nullptr ? nullptr : b + (size_t)rows.g * D;
    float wv[K], bv[K];
    if (B::kShort)
#pragma unroll
        for (int i = 0; i < kNV; ++i) {
            col.weights(wg, 1.f, i, wv + i * V % K);
            col.weights(bg, 0.f, i, bv + i * V % K);
        }
    Feed<T, V, kNV, B::kThreads, 1> feed(raw);
    const int64_t ahead = rows.step * G * D;
    const T *px = x + (rows.first * G + rows.g) * (int64_t)D, *pf = px;
    T *py = y + (rows.first * G + rows.g) * (int64_t)D;
    int64_t row = rows.first * G + rows.g;
    auto fetch = [&](int64_t t, int stage) {
        if (t < tokens)
#pragma unroll
            for (int i = 0; i < kNV; ++i)
                if (col.in(i)) feed.ask(stage, 0, i, pf + col.at(i));
        pf += ahead;
        feed.close();
    };
    const int64_t trips = (tokens + rows.step - 1) / rows.step;       // the same for every thread
    const float inv_d = 1.f / (float)D;
    fetch(rows.first, 0);
    fetch(rows.first + rows.step, 1);
    int stage = 0;
    int64_t t = rows.first;
    for (int64_t it = 0; it < trips; ++it, t += rows.step) {
        const bool live = t < tokens;
        fetch(t + 2 * rows.step, stage == 0 ? kStages - 1 : stage - 1);
        feed.wait();
        float v[K];
        float2 s = twice(0.f), q = twice(0.f);
#pragma unroll
        for (int i = 0; i < kNV; ++i)
            if (live && col.in(i)) {
                float *a = v + i * V % K;
                feed.get(stage, 0, i, px + col.at(i), *reinterpret_cast<float(*)[V]>(a));
                each<V>([&](int j) { s = fadd2(s, pair(a + j)); }, [&](int j) { s.x += a[j]; });
            }
        const float m = row_sum<kTpr>(s.x + s.y, red[it & 1][0]) * inv_d;
#pragma unroll
        for (int i = 0; i < kNV; ++i)
            if (live && col.in(i)) {
                float *a = v + i * V % K;
                if (!B::kShort) feed.get(stage, 0, i, px + col.at(i), *reinterpret_cast<float(*)[V]>(a));
                each<V>(
                    [&](int j) {
                        const float2 c = fadd2(pair(a + j), twice(-m));
                        put(a + j, c);
                        q = ffma2(c, c, q);
                    },
                    [&](int j) {
                        a[j] -= m;
                        q.x = fmaf(a[j], a[j], q.x);
                    });
            }
        const float r = rsqrtf(row_sum<kTpr>(q.x + q.y, red[it & 1][1]) * inv_d + eps);
        if (live) {
#pragma unroll
            for (int i = 0; i < kNV; ++i)
                if (col.in(i)) {
                    float *a = v + i * V % K, *w1 = wv + i * V % K, *b1 = bv + i * V % K;
                    if (!B::kShort) {
                        feed.get(stage, 0, i, px + col.at(i), *reinterpret_cast<float(*)[V]>(a));
                        col.weights(wg, 1.f, i, w1);
                        col.weights(bg, 0.f, i, b1);
                        each<V>([&](int j) { put(a + j, fadd2(pair(a + j), twice(-m))); }, [&](int j) { a[j] -= m; });
                    }
                    each<V>([&](int j) { put(a + j, ffma2(fmul2(pair(a + j), twice(r)), pair(w1 + j), pair(b1 + j))); },
                            [&](int j) { a[j] = fmaf(a[j] * r, w1[j], b1[j]); });
                    Vec<T, V>::st(py + col.at(i), *reinterpret_cast<float(*)[V]>(a));
                }
            if (col.lane == 0) {
                mean[row] = m;
                rstd[row] = r;
            }
        }
        px += ahead;
        py += ahead;
        row += rows.step * G;
        stage = stage == kStages - 1 ? 0 : stage + 1;
    }
}

// grid (blocks along T, G / gs).  part: [blocks][2][G][D], dw then db (kBias).
//   dx = r u - r mean(u) - xh r mean(u xh)
template <typename T, int V, int kTpr, int kNV, bool kFull, bool kBias>
__global__ void __launch_bounds__(Block<kTpr>::kThreads, (min_blocks<kTpr, true>()))
bwd_kernel(const T *dy, const T *__restrict__ x, const float *__restrict__ mean,
           const float *__restrict__ rstd, const float *__restrict__ w, int64_t tokens, int G, int gs,
           int D, T *dx, float *__restrict__ part) {
    using B = Block<kTpr>;
    using namespace sm100;
    constexpr int N = kNV * V, K = B::kShort ? N : V;
    __shared__ float red[2][2][B::kWarps];
    extern __shared__ __align__(16) unsigned char raw[];
    float *acc = reinterpret_cast<float *>(raw);        // [kRows][D], when the rows are done
    const Rows rows = make_rows<kTpr>(gs);
    const Columns<V, kTpr, kNV, kFull> col = {(int)threadIdx.x % kTpr, D};
    const float *wg = w == nullptr ? nullptr : w + (size_t)rows.g * D;
    float wv[K], dw[N], db[kBias ? N : 1];
#pragma unroll
    for (int e = 0; e < N; ++e) dw[e] = db[kBias ? e : 0] = 0.f;
    if (B::kShort)
#pragma unroll
        for (int i = 0; i < kNV; ++i) col.weights(wg, 1.f, i, wv + i * V % K);
    Feed<T, V, kNV, B::kThreads, 2> feed(raw);
    const int64_t ahead = rows.step * G * D;
    int64_t row = rows.first * G + rows.g, at = row * D, at_f = at;
    auto fetch = [&](int64_t t, int stage) {
        if (t < tokens)
#pragma unroll
            for (int i = 0; i < kNV; ++i)
                if (col.in(i)) {
                    feed.ask(stage, 0, i, x + at_f + col.at(i));
                    feed.ask(stage, 1, i, dy + at_f + col.at(i));
                }
        at_f += ahead;
        feed.close();
    };
    float nm = 0.f, nr = 0.f;                           // mean and rstd of the next row
    auto fetch_stats = [&](int64_t t, int64_t of) {
        if (t < tokens) {
            nm = mean[of];
            nr = rstd[of];
        }
    };
    const int64_t trips = (tokens + rows.step - 1) / rows.step;
    const float inv_d = 1.f / (float)D;
    fetch(rows.first, 0);
    fetch(rows.first + rows.step, 1);
    fetch_stats(rows.first, row);
    int stage = 0;
    int64_t t = rows.first;
    for (int64_t it = 0; it < trips; ++it, t += rows.step) {
        const bool live = t < tokens;
        const float m = nm, r = nr;
        fetch(t + 2 * rows.step, stage == 0 ? kStages - 1 : stage - 1);
        fetch_stats(t + rows.step, row + rows.step * G);
        feed.wait();
        float xh[K], u[K];                              // (x - m) r and dy w
        float2 sx = twice(0.f), sy = twice(0.f);
        auto get = [&](int i, float *a, float *b) {
            feed.get(stage, 0, i, x + at + col.at(i), *reinterpret_cast<float(*)[V]>(a));
            feed.get(stage, 1, i, dy + at + col.at(i), *reinterpret_cast<float(*)[V]>(b));
            each<V>([&](int j) { put(a + j, fmul2(fadd2(pair(a + j), twice(-m)), twice(r))); },
                    [&](int j) { a[j] = (a[j] - m) * r; });
        };
#pragma unroll
        for (int i = 0; i < kNV; ++i)
            if (live && col.in(i)) {
                float *a = xh + i * V % K, *b = u + i * V % K, *w1 = wv + i * V % K, *d = dw + i * V;
                get(i, a, b);
                if (!B::kShort) col.weights(wg, 1.f, i, w1);
                each<V>(
                    [&](int j) {
                        put(d + j, ffma2(pair(b + j), pair(a + j), pair(d + j)));
                        if constexpr (kBias) put(db + i * V + j, fadd2(pair(b + j), pair(db + i * V + j)));
                        const float2 c = fmul2(pair(b + j), pair(w1 + j));
                        put(b + j, c);
                        sx = fadd2(sx, c);
                        sy = ffma2(c, pair(a + j), sy);
                    },
                    [&](int j) {
                        d[j] = fmaf(b[j], a[j], d[j]);
                        if constexpr (kBias) db[i * V + j] += b[j];
                        b[j] *= w1[j];
                        sx.x += b[j];
                        sy.x = fmaf(b[j], a[j], sy.x);
                    });
            }
        const float k0 = -r * inv_d * row_sum<kTpr>(sx.x + sx.y, red[it & 1][0]);
        const float k1 = -r * inv_d * row_sum<kTpr>(sy.x + sy.y, red[it & 1][1]);
        if (live)
#pragma unroll
            for (int i = 0; i < kNV; ++i)
                if (col.in(i)) {
                    float *a = xh + i * V % K, *b = u + i * V % K, *w1 = wv + i * V % K;
                    if (!B::kShort) {                   // again, rather than 64 registers over the sums
                        get(i, a, b);
                        col.weights(wg, 1.f, i, w1);
                        each<V>([&](int j) { put(b + j, fmul2(pair(b + j), pair(w1 + j))); },
                                [&](int j) { b[j] *= w1[j]; });
                    }
                    each<V>([&](int j) { put(b + j, ffma2(pair(b + j), twice(r),
                                                          ffma2(pair(a + j), twice(k1), twice(k0)))); },
                            [&](int j) { b[j] = fmaf(b[j], r, fmaf(a[j], k1, k0)); });
                    Vec<T, V>::st(dx + at + col.at(i), *reinterpret_cast<float(*)[V]>(b));
                }
        at += ahead;
        row += rows.step * G;
        stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    if (part == nullptr) return;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    float *out = part + (size_t)blockIdx.x * 2 * G * D;
    const int rg = threadIdx.x / kTpr;
#pragma unroll
    for (int which = 0; which < (kBias ? 2 : 1); ++which, out += (size_t)G * D) {
        if (B::kRows == gs) {                           // one row for each group
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (col.in(e / V)) out[(size_t)rows.g * D + col.at(e / V) + e % V] = which ? db[kBias ? e : 0] : dw[e];
            continue;
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (col.in(e / V)) acc[rg * D + col.at(e / V) + e % V] = which ? db[kBias ? e : 0] : dw[e];
        __syncthreads();
        for (int e = threadIdx.x; e < gs * D; e += B::kThreads) {
            float a = 0.f;
            for (int i = e / D; i < B::kRows; i += gs) a += acc[i * D + e % D];
            out[(size_t)(blockIdx.y * gs + e / D) * D + e % D] = a;
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
