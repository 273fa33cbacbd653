// kda_linear_simt.cuh -- decayed linear attention on CUDA cores, all in fp32:
// segment states, outputs, and the two halves of the gradient.
//
// Serves fp32 inputs (held to 1e-5) at every head size.  32-token chunks: their
// products and the state update cost the same order of work, and the chunk's tiles and
// the state fit shared memory at every head size.  Every product is a register tile
// over operands in shared memory whose rows are padded by four floats, so that reads
// of 16 bytes along rows and of 4 across them are free of bank conflicts.  Bound by
// shared-memory reads and FMAs where there are heads enough, by the latency of a
// chunk's steps where there are few.
//
// Measured: 96 heads of 128 x 2,048 tokens, outputs 0.94 ms, gradient 2.11 ms (20 TFLOP/s
// of products, of the 71 that these cores have; with operands read 4 bytes at a time
// 1.68 and 4.38 ms); 211 tokens of 3 heads of 64 in 5 sequences 20 us (30 us).
//
// Gradient of L = <dO, O> + <dhT, hT>, per chunk with E = dL/dS at its end:
//   P = Q K^T . D scale,   dP = dO V^T,   dA = dP . D scale
//   dQ = dA K + Diag(scale e^b) dO S0^T
//   dK = dA^T Q + Diag(e^{b_C - b}) V E^T
//   dV = P^T dO + Diag(e^{b_C - b}) K E
//   dL/dS0 = e^{b_C} E + (Diag(scale e^b) Q)^T dO
//   dg_t = sum_{i >= t} (q_i . dq_i - k_i . dk_i) + <S_end, E_end>
// S is needed for dQ alone and E for dK, dV alone, so one kernel walks forward
// with S (dQ) and one backward with E (dK, dV, dg): no state is stored per chunk.
// q_i . dq_i and k_i . dk_i are formed from the fp32 products (the part inside
// the chunk as row and column sums of P . dP), not from rounded dq, dk.
#pragma once

#include "kda_linear_common.cuh"

namespace kda {
namespace lin {

constexpr int kC = 32;                 // tokens of a chunk
constexpr int kThreads = 256;
constexpr int kPad = 4;                // floats behind a row in shared memory

// A register tile of an M x N product over 256 threads: lanes run along N, a thread's
// rows are neighbours.
template <int M, int N>
struct Tile {
    static constexpr int kNT = N < 32 ? N : 32;
    static constexpr int kRows = kThreads / kNT;       // rows covered at once
    static constexpr int kI = M / kRows, kJ = N / kNT;
    static_assert(M % kRows == 0 && N % kNT == 0, "tile");
    float v[kI][kJ];
    static __device__ __forceinline__ int m(int i) { return threadIdx.x / kNT * kI + i; }
    static __device__ __forceinline__ int n(int j) { return threadIdx.x % kNT + j * kNT; }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kI; ++i)
#pragma unroll
            for (int j = 0; j < kJ; ++j) v[i][j] = 0.f;
    }
    // v += A B, A(m, k) = A[m lda + k] (or A[k lda + m] if TA), B alike, one k after
    // the other.  Four k at a time: along k both operands are read as 16 bytes (A by
    // all lanes of a row at once, B without bank conflicts, since rows are 4 floats
    // apart modulo the banks), and so are a thread's rows of A if TA.
    template <int K, bool TA, bool TB>
    __device__ __forceinline__ void mac(const float *A, int lda, const float *B, int ldb) {
        constexpr int kV = kI % 4 == 0 ? 4 : kI % 2 == 0 ? 2 : 1;
        A += TA ? m(0) : m(0) * lda;
        B += TB ? n(0) * ldb : n(0);
        // small tiles have few sums, and need more loads in flight
        constexpr int kUnroll = kI * kJ <= 4 ? 8 : kI * kJ <= 16 ? 4 : 2;
#pragma unroll kUnroll
        for (int k = 0; k < K; k += 4) {
            float b[4][kJ];
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                if (TB) {
                    const float4 x = *reinterpret_cast<const float4 *>(B + j * kNT * ldb + k);
                    b[0][j] = x.x; b[1][j] = x.y; b[2][j] = x.z; b[3][j] = x.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) b[i][j] = B[(k + i) * ldb + j * kNT];
                }
            }
            if (TA) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < kI; i += kV) {
                        float a[kV];
                        const float *p = A + (k + c) * lda + i;
                        if constexpr (kV == 4) {
                            const float4 x = *reinterpret_cast<const float4 *>(p);
                            a[0] = x.x; a[1] = x.y; a[2] = x.z; a[3] = x.w;
                        } else if constexpr (kV == 2) {
                            const float2 x = *reinterpret_cast<const float2 *>(p);
                            a[0] = x.x; a[1] = x.y;
                        } else {
                            a[0] = *p;
                        }
#pragma unroll
                        for (int r = 0; r < kV; ++r)
#pragma unroll
                            for (int j = 0; j < kJ; ++j) v[i + r][j] = fmaf(a[r], b[c][j], v[i + r][j]);
                    }
            } else {
#pragma unroll
                for (int i = 0; i < kI; ++i) {
                    const float4 x = *reinterpret_cast<const float4 *>(A + i * lda + k);
                    const float a[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int j = 0; j < kJ; ++j) v[i][j] = fmaf(a[c], b[c][j], v[i][j]);
                }
            }
        }
    }
};

// Sum over the kNT lanes that share a row of a tile.
template <int NT>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = NT / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// [kC][W] tile of rows t0 .. t0 + len of x [T, heads, D], columns c0 .. c0 + W,
// zero behind len (a row of zeros with log-decay 0 leaves every result alone).
template <int W>
__device__ __forceinline__ void load_tile(float *dst, const float *x, int64_t t0, int len, int heads,
                                          int head, int D, int c0) {
    for (int e = threadIdx.x; e < kC * W / 4; e += kThreads) {
        const int r = e / (W / 4), c = e % (W / 4) * 4;
        const size_t row = t0 + (r < len ? r : 0);
        cp_async16(sm100::smem_u32(dst + r * (W + kPad) + c), x + (row * heads + head) * D + c0 + c, r < len);
    }
}

// The decays of a chunk, by warp 0: sums b_i in fp64, and the factors e^{b_i} and
// e^{b_C - b_i} of its rows.
struct Decays {
    double b[kC], tot;
    float row[kC], col[kC];
};
__device__ __forceinline__ void chunk_decays(Decays &d, const float *g, int per_token, int64_t t0,
                                             int len, int h, int H) {
    if (threadIdx.x < 32) {
        const int i = threadIdx.x;
        const double b = warp_scan(i < len ? (double)load_decay(g, per_token, t0 + i, h, H) : 0.0);
        const double tot = __shfl_sync(0xffffffffu, b, 31);
        d.b[i] = b;
        d.row[i] = expf((float)b);
        d.col[i] = expf((float)(tot - b));
        if (i == 0) d.tot = tot;
    }
}
// What the chunk's loads and decays are waited for with.
__device__ __forceinline__ void chunk_ready() {
    cp_commit();                                       // a copy in no group is not waited for
    cp_wait_all();
    __syncthreads();
}

// ------------------------------------------------------- segment states
// Forward: R = sum_j e^{b_end - b_j} k_j v_j^T over the segment (skipped for the
// last segment of a sequence).  Reverse: R = sum_i scale e^{b_i} q_i dO_i^T, b
// counted from the segment's start (skipped for the first).
template <int D>
struct StateSmem {
    static constexpr int kW = D < 64 ? D : 64;         // value columns of a block
    float x[kC * (D + kPad)], y[kC * (kW + kPad)];
    Decays d;
};

template <int D, bool kReverse>
__global__ void __launch_bounds__(kThreads)
state_kernel(const float *__restrict__ x, const float *__restrict__ y, const float *__restrict__ g,
             int per_token, SegMap m, int Hk, int H, float scale, float *__restrict__ ws,
             float *__restrict__ total) {
    using Sm = StateSmem<D>;
    constexpr int W = Sm::kW;
    extern __shared__ __align__(16) unsigned char raw[];
    Sm &sm = *reinterpret_cast<Sm *>(raw);
    const int h = blockIdx.y, c0 = blockIdx.z * W;
    Segment sg;
    if (!find_body(m, blockIdx.x, kReverse, sg)) return;
    Tile<D, W> S;
    S.zero();
    double sum = 0.0;
    const int64_t len = sg.t1 - sg.t0;
    const int64_t chunks = (len + kC - 1) / kC;
    for (int64_t c = 0; c < chunks; ++c) {
        const int64_t t = sg.t0 + (kReverse ? chunks - 1 - c : c) * kC;
        const int L = (int)(sg.t1 - t < kC ? sg.t1 - t : kC);
        __syncthreads();
        load_tile<D>(sm.x, x, t, L, Hk, h / (H / Hk), D, 0);
        load_tile<W>(sm.y, y, t, L, H, h, D, c0);
        chunk_decays(sm.d, g, per_token, t, L, h, H);
        chunk_ready();
        const double tot = sm.d.tot;
        sum += tot;
        for (int e = threadIdx.x; e < kC * W; e += kThreads) {
            const int r = e / W;
            sm.y[r * (W + kPad) + e % W] *=
                kReverse ? scale * sm.d.row[r] : sm.d.col[r];
        }
        const float a = expf((float)tot);
#pragma unroll
        for (int i = 0; i < S.kI; ++i)
#pragma unroll
            for (int j = 0; j < S.kJ; ++j) S.v[i][j] *= a;
        __syncthreads();
        S.template mac<kC, true, false>(sm.x, D + kPad, sm.y, W + kPad);
    }
    float *out = ws + ((size_t)sg.slot * H + h) * D * D + c0;
#pragma unroll
    for (int i = 0; i < S.kI; ++i)
#pragma unroll
        for (int j = 0; j < S.kJ; ++j) out[(size_t)S.m(i) * D + S.n(j)] = S.v[i][j];
    if (c0 == 0 && threadIdx.x == 0) total[(size_t)sg.slot * H + h] = expf((float)sum);
}

// -------------------------------------------------------------- outputs
template <int D>
struct OutSmem {
    static constexpr int kW = D < 64 ? D : 64;
    float S[D * (kW + kPad)];
    float q[kC * (D + kPad)], k[kC * (D + kPad)], v[kC * (kW + kPad)], P[kC * (kC + kPad)];
    Decays d;
};

// grid (units, H, D / kW): value columns are independent, so a head is split
// over blocks of 64 columns (the chunk's 32 x 32 products are formed in each).
template <int D>
__global__ void __launch_bounds__(kThreads)
out_kernel(const float *__restrict__ q, const float *__restrict__ k, const float *__restrict__ v,
           const float *__restrict__ g, int per_token, const float *h0, SegMap m, int Hk, int H,
           float scale, const float *__restrict__ ws, float *__restrict__ o, float *hT) {
    using Sm = OutSmem<D>;
    constexpr int W = Sm::kW;
    extern __shared__ __align__(16) unsigned char raw[];
    Sm &sm = *reinterpret_cast<Sm *>(raw);
    const int u = blockIdx.x, h = blockIdx.y, c0 = blockIdx.z * W;
    if (u == 0 && h == 0 && c0 == 0) check_seqlens(m);
    Segment sg;
    if (!find_segment(m, u, sg)) return;
    const float *from = ws != nullptr && sg.count > 1 ? ws + ((size_t)sg.slot * H + h) * D * D
                        : h0 != nullptr ? h0 + ((size_t)sg.n * H + h) * D * D : nullptr;
    Tile<D, W> S;
#pragma unroll
    for (int i = 0; i < S.kI; ++i)
#pragma unroll
        for (int j = 0; j < S.kJ; ++j) {
            S.v[i][j] = from != nullptr ? from[(size_t)S.m(i) * D + c0 + S.n(j)] : 0.f;
            sm.S[S.m(i) * (W + kPad) + S.n(j)] = S.v[i][j];
        }
    for (int64_t t = sg.t0; t < sg.t1; t += kC) {
        const int L = (int)(sg.t1 - t < kC ? sg.t1 - t : kC);
        __syncthreads();
        load_tile<D>(sm.q, q, t, L, Hk, h / (H / Hk), D, 0);
        load_tile<D>(sm.k, k, t, L, Hk, h / (H / Hk), D, 0);
        load_tile<W>(sm.v, v, t, L, H, h, D, c0);
        chunk_decays(sm.d, g, per_token, t, L, h, H);
        chunk_ready();
        Tile<kC, kC> P;
        P.zero();
        P.template mac<D, false, true>(sm.q, D + kPad, sm.k, D + kPad);
#pragma unroll
        for (int i = 0; i < P.kI; ++i)
#pragma unroll
            for (int j = 0; j < P.kJ; ++j) {
                const int r = P.m(i), c = P.n(j);
                sm.P[r * (kC + kPad) + c] = r >= c ? P.v[i][j] * expf((float)(sm.d.b[r] - sm.d.b[c])) : 0.f;
            }
        Tile<kC, W> O;
        O.zero();
        O.template mac<D, false, false>(sm.q, D + kPad, sm.S, W + kPad);
#pragma unroll
        for (int i = 0; i < O.kI; ++i) {
            const float a = sm.d.row[O.m(i)];
#pragma unroll
            for (int j = 0; j < O.kJ; ++j) O.v[i][j] *= a;
        }
        __syncthreads();
        O.template mac<kC, false, false>(sm.P, kC + kPad, sm.v, W + kPad);
#pragma unroll
        for (int i = 0; i < O.kI; ++i)
            if (O.m(i) < L)
#pragma unroll
                for (int j = 0; j < O.kJ; ++j)
                    o[((size_t)(t + O.m(i)) * H + h) * D + c0 + O.n(j)] = O.v[i][j] * scale;
        __syncthreads();
        const double tot = sm.d.tot;
        for (int e = threadIdx.x; e < kC * W; e += kThreads)
            sm.v[e / W * (W + kPad) + e % W] *= sm.d.col[e / W];
        const float a = expf((float)tot);
#pragma unroll
        for (int i = 0; i < S.kI; ++i)
#pragma unroll
            for (int j = 0; j < S.kJ; ++j) S.v[i][j] *= a;
        __syncthreads();
        S.template mac<kC, true, false>(sm.k, D + kPad, sm.v, W + kPad);
#pragma unroll
        for (int i = 0; i < S.kI; ++i)
#pragma unroll
            for (int j = 0; j < S.kJ; ++j) sm.S[S.m(i) * (W + kPad) + S.n(j)] = S.v[i][j];
    }
    if (hT != nullptr && sg.s == sg.count - 1) {
        float *out = hT + ((size_t)sg.n * H + h) * D * D + c0;
#pragma unroll
        for (int i = 0; i < S.kI; ++i)
#pragma unroll
            for (int j = 0; j < S.kJ; ++j) out[(size_t)S.m(i) * D + S.n(j)] = S.v[i][j];
    }
}

// ------------------------------------------------------------- gradient
template <int D>
struct GradSmem {
    float S[D * (D + kPad)];                              // S (dQ) or E (dK, dV)
    float q[kC * (D + kPad)], k[kC * (D + kPad)], v[kC * (D + kPad)], dO[kC * (D + kPad)];
    float P[kC * (kC + kPad)], A[kC * (kC + kPad)];
    Decays d;
    float r[kC];
    double red[kThreads / 32];
};

// Loads a chunk and forms P = (Q K^T . D) scale and dA = (dO V^T . D) scale in
// shared memory; kW: P is replaced by W = P . dO V^T.
template <int D, bool kW>
__device__ __forceinline__ void grad_chunk(GradSmem<D> &sm, const float *q, const float *k, const float *v,
                                           const float *dO, const float *g, int per_token, int64_t t,
                                           int L, int Hk, int H, int h, float scale) {
    load_tile<D>(sm.q, q, t, L, Hk, h / (H / Hk), D, 0);
    load_tile<D>(sm.k, k, t, L, Hk, h / (H / Hk), D, 0);
    load_tile<D>(sm.v, v, t, L, H, h, D, 0);
    load_tile<D>(sm.dO, dO, t, L, H, h, D, 0);
    chunk_decays(sm.d, g, per_token, t, L, h, H);
    chunk_ready();
    Tile<kC, kC> P, dP;
    P.zero();
    dP.zero();
    P.template mac<D, false, true>(sm.q, D + kPad, sm.k, D + kPad);
    dP.template mac<D, false, true>(sm.dO, D + kPad, sm.v, D + kPad);
#pragma unroll
    for (int i = 0; i < P.kI; ++i)
#pragma unroll
        for (int j = 0; j < P.kJ; ++j) {
            const int r = P.m(i), c = P.n(j);
            const float e = r >= c ? scale * expf((float)(sm.d.b[r] - sm.d.b[c])) : 0.f;
            const float p = P.v[i][j] * e;
            sm.P[r * (kC + kPad) + c] = r >= c ? (kW ? p * dP.v[i][j] : p) : 0.f;
            sm.A[r * (kC + kPad) + c] = r >= c ? dP.v[i][j] * e : 0.f;
        }
}

// A gradient row of a head that shares q and k with others goes out as a part (to
// be summed over the group).
__device__ __forceinline__ void store_shared(float *out, float *part, size_t e, float x) {
    (part != nullptr ? part : out)[e] = x;
}

// dQ, the decay term of every row (rowsum W - colsum W + q . dq from the state),
// and <S_end, E_end> of the segment.
template <int D>
__global__ void __launch_bounds__(kThreads)
grad_q_kernel(const float *__restrict__ q, const float *__restrict__ k, const float *__restrict__ v,
              const float *__restrict__ dO, const float *__restrict__ g, int per_token,
              const float *__restrict__ h0, const float *__restrict__ dhT, SegMap m, int Hk, int H,
              float scale, const float *__restrict__ wsS, const float *__restrict__ wsE,
              float *__restrict__ dq, float *__restrict__ part, float *__restrict__ term,
              double *__restrict__ anchor) {
    extern __shared__ __align__(16) unsigned char raw[];
    GradSmem<D> &sm = *reinterpret_cast<GradSmem<D> *>(raw);
    const int u = blockIdx.x, h = blockIdx.y;
    if (u == 0 && h == 0) check_seqlens(m);
    Segment sg;
    if (!find_segment(m, u, sg)) return;
    const size_t seg = ((size_t)sg.slot * H + h) * D * D, seq = ((size_t)sg.n * H + h) * D * D;
    const float *from = wsS != nullptr && sg.count > 1 ? wsS + seg : h0 != nullptr ? h0 + seq : nullptr;
    Tile<D, D> S;
#pragma unroll
    for (int i = 0; i < S.kI; ++i)
#pragma unroll
        for (int j = 0; j < S.kJ; ++j) {
            S.v[i][j] = from != nullptr ? from[(size_t)S.m(i) * D + S.n(j)] : 0.f;
            sm.S[S.m(i) * (D + kPad) + S.n(j)] = S.v[i][j];
        }
    for (int64_t t = sg.t0; t < sg.t1; t += kC) {
        const int L = (int)(sg.t1 - t < kC ? sg.t1 - t : kC);
        __syncthreads();
        grad_chunk<D, true>(sm, q, k, v, dO, g, per_token, t, L, Hk, H, h, scale);
        Tile<kC, D> X;                                 // dO S^T
        X.zero();
        X.template mac<D, false, true>(sm.dO, D + kPad, sm.S, D + kPad);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < X.kI; ++i) {
            const int r = X.m(i);
            const float a = scale * sm.d.row[r];
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < X.kJ; ++j) {
                X.v[i][j] *= a;
                s = fmaf(X.v[i][j], sm.q[r * (D + kPad) + X.n(j)], s);
            }
            s = row_sum<X.kNT>(s);
            if (threadIdx.x % X.kNT == 0) sm.r[r] = s;
        }
        X.template mac<kC, false, false>(sm.A, kC + kPad, sm.k, D + kPad);
#pragma unroll
        for (int i = 0; i < X.kI; ++i)
            if (X.m(i) < L)
#pragma unroll
                for (int j = 0; j < X.kJ; ++j) {
                    const size_t row = (size_t)(t + X.m(i)) * H + h;
                    store_shared(dq, part, row * D + X.n(j), X.v[i][j]);
                }
        const double tot = sm.d.tot;
        for (int e = threadIdx.x; e < kC * D; e += kThreads)
            sm.v[e / D * (D + kPad) + e % D] *= sm.d.col[e / D];
        const float a = expf((float)tot);
#pragma unroll
        for (int i = 0; i < S.kI; ++i)
#pragma unroll
            for (int j = 0; j < S.kJ; ++j) S.v[i][j] *= a;
        __syncthreads();
        if (threadIdx.x < L) {
            float s = sm.r[threadIdx.x];
            for (int c = 0; c < kC; ++c)
                s += sm.P[threadIdx.x * (kC + kPad) + c] - sm.P[c * (kC + kPad) + threadIdx.x];
            term[(size_t)(t + threadIdx.x) * H + h] = s;
        }
        S.template mac<kC, true, false>(sm.k, D + kPad, sm.v, D + kPad);
#pragma unroll
        for (int i = 0; i < S.kI; ++i)
#pragma unroll
            for (int j = 0; j < S.kJ; ++j) sm.S[S.m(i) * (D + kPad) + S.n(j)] = S.v[i][j];
    }
    const float *to = wsE != nullptr && sg.count > 1 ? wsE + seg : dhT != nullptr ? dhT + seq : nullptr;
    double s = 0.0;
    if (to != nullptr)
#pragma unroll
        for (int i = 0; i < S.kI; ++i)
#pragma unroll
            for (int j = 0; j < S.kJ; ++j)
                s += (double)S.v[i][j] * (double)to[(size_t)S.m(i) * D + S.n(j)];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (threadIdx.x % 32 == 0) sm.red[threadIdx.x / 32] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        s = 0.0;
        for (int i = 0; i < kThreads / 32; ++i) s += sm.red[i];
        anchor[(size_t)u * H + h] = s;
    }
}

// dK, dV, dg and dh0, chunks last to first.
template <int D>
__global__ void __launch_bounds__(kThreads)
grad_kv_kernel(const float *__restrict__ q, const float *__restrict__ k, const float *__restrict__ v,
               const float *__restrict__ dO, const float *__restrict__ g, int per_token,
               const float *__restrict__ dhT, SegMap m, int Hk, int H, float scale,
               const float *__restrict__ wsE, const float *__restrict__ term,
               const double *__restrict__ anchor, float *__restrict__ dk, float *__restrict__ part,
               float *__restrict__ dv, float *__restrict__ dg, double *__restrict__ head_sum,
               float *__restrict__ dh0) {
    extern __shared__ __align__(16) unsigned char raw[];
    GradSmem<D> &sm = *reinterpret_cast<GradSmem<D> *>(raw);
    const int u = blockIdx.x, h = blockIdx.y;
    Segment sg;
    if (!find_segment(m, u, sg)) {
        if (!per_token && threadIdx.x == 0) head_sum[(size_t)u * H + h] = 0.0;
        return;
    }
    const size_t seg = ((size_t)sg.slot * H + h) * D * D, seq = ((size_t)sg.n * H + h) * D * D;
    const float *from = wsE != nullptr && sg.count > 1 ? wsE + seg : dhT != nullptr ? dhT + seq : nullptr;
    Tile<D, D> E;
#pragma unroll
    for (int i = 0; i < E.kI; ++i)
#pragma unroll
        for (int j = 0; j < E.kJ; ++j) {
            E.v[i][j] = from != nullptr ? from[(size_t)E.m(i) * D + E.n(j)] : 0.f;
            sm.S[E.m(i) * (D + kPad) + E.n(j)] = E.v[i][j];
        }
    double carry = anchor[(size_t)u * H + h], sum = 0.0;   // warp 0
    const int64_t chunks = (sg.t1 - sg.t0 + kC - 1) / kC;
    for (int64_t c = chunks - 1; c >= 0; --c) {
        const int64_t t = sg.t0 + c * kC;
        const int L = (int)(sg.t1 - t < kC ? sg.t1 - t : kC);
        __syncthreads();
        grad_chunk<D, false>(sm, q, k, v, dO, g, per_token, t, L, Hk, H, h, scale);
        const double tot = sm.d.tot;
        Tile<kC, D> X;                                 // V E^T
        X.zero();
        X.template mac<D, false, true>(sm.v, D + kPad, sm.S, D + kPad);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < X.kI; ++i) {
            const int r = X.m(i);
            const float a = sm.d.col[r];
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < X.kJ; ++j) {
                X.v[i][j] *= a;
                s = fmaf(X.v[i][j], sm.k[r * (D + kPad) + X.n(j)], s);
            }
            s = row_sum<X.kNT>(s);
            if (threadIdx.x % X.kNT == 0) sm.r[r] = s;
        }
        X.template mac<kC, true, false>(sm.A, kC + kPad, sm.q, D + kPad);
#pragma unroll
        for (int i = 0; i < X.kI; ++i)
            if (X.m(i) < L)
#pragma unroll
                for (int j = 0; j < X.kJ; ++j) {
                    const size_t row = (size_t)(t + X.m(i)) * H + h;
                    store_shared(dk, part, row * D + X.n(j), X.v[i][j]);
                }
        X.zero();                                      // K E
        X.template mac<D, false, false>(sm.k, D + kPad, sm.S, D + kPad);
#pragma unroll
        for (int i = 0; i < X.kI; ++i) {
            const float a = sm.d.col[X.m(i)];
#pragma unroll
            for (int j = 0; j < X.kJ; ++j) X.v[i][j] *= a;
        }
        X.template mac<kC, true, false>(sm.P, kC + kPad, sm.dO, D + kPad);
#pragma unroll
        for (int i = 0; i < X.kI; ++i)
            if (X.m(i) < L)
#pragma unroll
                for (int j = 0; j < X.kJ; ++j)
                    dv[((size_t)(t + X.m(i)) * H + h) * D + X.n(j)] = X.v[i][j];
        __syncthreads();
        for (int e = threadIdx.x; e < kC * D; e += kThreads)
            sm.dO[e / D * (D + kPad) + e % D] *= scale * sm.d.row[e / D];
        if (threadIdx.x < 32) {                        // sums from the chunk's end
            const int i = threadIdx.x, r = 31 - i;
            double x = 0.0;
            if (r < L) x = (double)term[(size_t)(t + r) * H + h] - (double)sm.r[r];
            x = warp_scan(x) + carry;
            if (r < L) {
                if (per_token) dg[(size_t)(t + r) * H + h] = (float)x;
                sum += x;
            }
            carry = __shfl_sync(0xffffffffu, x, 31);
        }
        const float a = expf((float)tot);
#pragma unroll
        for (int i = 0; i < E.kI; ++i)
#pragma unroll
            for (int j = 0; j < E.kJ; ++j) E.v[i][j] *= a;
        __syncthreads();
        E.template mac<kC, true, false>(sm.q, D + kPad, sm.dO, D + kPad);
#pragma unroll
        for (int i = 0; i < E.kI; ++i)
#pragma unroll
            for (int j = 0; j < E.kJ; ++j) sm.S[E.m(i) * (D + kPad) + E.n(j)] = E.v[i][j];
    }
    if (!per_token && threadIdx.x < 32) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (threadIdx.x == 0) head_sum[(size_t)u * H + h] = sum;
    }
    if (dh0 != nullptr && sg.s == 0) {
        float *out = dh0 + seq;
#pragma unroll
        for (int i = 0; i < E.kI; ++i)
#pragma unroll
            for (int j = 0; j < E.kJ; ++j) out[(size_t)E.m(i) * D + E.n(j)] = E.v[i][j];
    }
}

// out[t][hk][c] = sum over the group of part[t][hk r + i][c], in fp32 and in the
// order of the heads; a thread owns 4 channels of one (t, hk).  Bound by memory: 2 x
// 8 heads of 10,824 tokens 20.7 us (5.4 TB/s).
template <typename T>
__global__ void __launch_bounds__(kThreads)
group_sum_kernel(const float *__restrict__ part, T *__restrict__ out, int64_t rows, int rep, int D) {
    const int64_t e = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;
    if (e >= rows * D) return;
    const int64_t row = e / D;
    const float *p = part + row * rep * D + e % D;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < rep; ++i) {
        const float4 x = *reinterpret_cast<const float4 *>(p + (size_t)i * D);
        s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    IO<T>::st(out + e, s.x);
    IO<T>::st(out + e + 1, s.y);
    IO<T>::st(out + e + 2, s.z);
    IO<T>::st(out + e + 3, s.w);
}

// dg[h] of a constant decay: the units' sums in order.
__global__ void __launch_bounds__(kThreads)
head_sum_kernel(const double *__restrict__ head_sum, float *__restrict__ dg, int units, int H) {
    __shared__ double red[kThreads];
    double s = 0.0;
    for (int u = threadIdx.x; u < units; u += kThreads) s += head_sum[(size_t)u * H + blockIdx.x];
    red[threadIdx.x] = s;
    __syncthreads();
    for (int o = kThreads / 2; o > 0; o >>= 1) {
        if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
        __syncthreads();
    }
    if (threadIdx.x == 0) dg[blockIdx.x] = (float)red[0];
}

}  // namespace lin
}  // namespace kda
