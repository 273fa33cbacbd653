// kda_linear_mma.cuh -- decayed linear attention in bf16 on warp-level matrix
// instructions (m16n8k16, fp32 accumulators): segment states, outputs for head
// sizes below 128, and the gradient for every head size.
//
// Why warp-level.  The gradient of the decays is a small difference of large sums
// and goes out in fp32, so its products with the state need the state to 24 bits:
// three bf16 terms.  Here the state is a register accumulator whose fragments are
// the next product's left operand as they are, and are cut into terms in registers.
// On tcgen05 each term would be written to tensor memory for every chunk, as the
// prefill writes those of V' (192 columns of 512 at d = 128): another kernel, which
// is not built.  Rounded to bf16 once each, on top of the outputs' own rounding: P, dA,
// the state that the queries of a prefill read, and E where dV reads it.
//
// The state X (D x D, fp32) is spread over NW = D / 16 warps, 16 rows each.  With
// 64-token chunks, tiles of tokens in shared memory (rows padded by 16 bytes: every
// ldmatrix is free of bank conflicts), filled by asynchronous copies a chunk ahead:
//   X (+)= (Diag(c) A)^T B     A^T by transposing loads, scaled and cut in registers
//   Y^T = X B^T                X's accumulators as the left operand
// What bounds the gradient: at d = 128 a block has 8 warps of 255 registers (two a scheduler),
// and the tensor pipe is busy for 40 to 43 % of the time; the rest waits for
// shared memory and for one matrix instruction after another.  96 heads x 2,048
// tokens: dQ 194 us, dK and dV 240 us.
// Formulas of the gradient: kda_linear_simt.cuh.  One walk forward with S gives dQ
// and x_i = q_i . dq_i, one walk backward with E = dL/dS gives dK, dV, y_j = k_j . dk_j
// and dg_t = sum_{i >= t} (x_i - y_i) + <S_end, E_end>; x and y are formed from fp32:
// the part inside the chunk as row and column sums of P . dP, the other as
// q_i . (S dO_i) before it is rounded.
#pragma once

#include "kda_linear_simt.cuh"

namespace kda {
namespace lin {
namespace mm {

using bf16 = __nv_bfloat16;
constexpr int kTok = 64;               // tokens of a chunk
constexpr int kPp = kTok + 8;          // pitch of a token x token tile

template <int D>
struct Shape {
    static constexpr int kWarps = D / 16, kThreads = 32 * kWarps;
    static constexpr int kPitch = D + 8;
    static constexpr int kTile = kTok * kPitch;        // elements
    static constexpr int kN = D / 8, kK = D / 16;      // n-tiles and k-steps over D
};

struct __align__(16) Factors {
    float hi[kTok], lo[kTok];          // b_i / ln 2, a sum of two floats
    float row[kTok];                   // scale e^{b_i}
    float col[kTok];                   // e^{b_C - b_j}
    float gamma;                       // e^{b_C}
    float end_hi, end_lo;
};
static_assert(sizeof(Factors) % 16 == 0, "copied in 16-byte pieces");

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Fragments from a tile X [rows][pitch] in shared memory (byte address).
// Left operand, rows r0 .. + 15, k = columns k0 .. + 15.
__device__ __forceinline__ void frag_a(uint32_t x, int pitch, int r0, int k0, uint32_t (&r)[4]) {
    const int l = threadIdx.x & 31;
    ldmatrix(x + 2u * ((r0 + (l & 15)) * pitch + k0 + 8 * (l >> 4)), r);
}
// Left operand X^T: rows = columns c0 .. + 15 of X, k = rows k0 .. + 15.
__device__ __forceinline__ void frag_at(uint32_t x, int pitch, int c0, int k0, uint32_t (&r)[4]) {
    const int l = threadIdx.x & 31;
    ldmatrix_trans(x + 2u * ((k0 + (l & 7) + 8 * (l >> 4)) * pitch + c0 + 8 * ((l >> 3) & 1)), r);
}
// Right operands of two n-tiles: n = rows n0 .. + 15 of X, k = columns k0 .. + 15.
// Tile i takes r[2 i], r[2 i + 1].
__device__ __forceinline__ void frag_b(uint32_t x, int pitch, int n0, int k0, uint32_t (&r)[4]) {
    const int l = threadIdx.x & 31;
    ldmatrix(x + 2u * ((n0 + (l & 7) + 8 * (l >> 4)) * pitch + k0 + 8 * ((l >> 3) & 1)), r);
}
// The same of X^T: n = columns n0 .. + 15, k = rows k0 .. + 15.
__device__ __forceinline__ void frag_bt(uint32_t x, int pitch, int n0, int k0, uint32_t (&r)[4]) {
    const int l = threadIdx.x & 31;
    ldmatrix_trans(x + 2u * ((k0 + (l & 15)) * pitch + n0 + 8 * (l >> 4)), r);
}

// 64 token rows of one head; rows behind L become zero (and are not read).
template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const bf16 *x, int64_t t, int L, int heads, int head) {
    using Sh = Shape<D>;
    // a thread keeps its column: rows r0, r0 + kStep, ...
    constexpr int kStep = Sh::kThreads / (D / 8);
    const int r0 = threadIdx.x / (D / 8), c = threadIdx.x % (D / 8) * 8;
    const bf16 *base = x + ((size_t)t * heads + head) * D + c, *p = base + (size_t)r0 * heads * D;
    const size_t step = (size_t)kStep * heads * D;
    dst += 2u * (r0 * Sh::kPitch + c);
#pragma unroll
    for (int i = 0; i < kTok / kStep; ++i, p += step) {
        const bool live = r0 + i * kStep < L;
        cp_async16(dst + 2u * (i * kStep * Sh::kPitch), live ? p : base, live);
    }
}

// The two decays a lane of warp 0 holds: tokens 2 lane, 2 lane + 1 of a chunk.
__device__ __forceinline__ float2 fetch_decays(const float *g, int per_token, int64_t t, int L, int h, int H) {
    const int i = 2 * (threadIdx.x & 31);
    return make_float2(i < L ? load_decay(g, per_token, t + i, h, H) : 0.f,
                       i + 1 < L ? load_decay(g, per_token, t + i + 1, h, H) : 0.f);
}

__device__ __forceinline__ void make_factors(Factors &f, float2 g, float scale) {
    const int lane = threadIdx.x & 31;
    Sum2 run = add2({g.x, 0.f}, {g.y, 0.f});
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sum2 up = {__shfl_up_sync(0xffffffffu, run.hi, o), __shfl_up_sync(0xffffffffu, run.lo, o)};
        if (lane >= o) run = add2(up, run);
    }
    const Sum2 end = {__shfl_sync(0xffffffffu, run.hi, 31), __shfl_sync(0xffffffffu, run.lo, 31)};
    Sum2 b0 = {__shfl_up_sync(0xffffffffu, run.hi, 1), __shfl_up_sync(0xffffffffu, run.lo, 1)};
    if (lane == 0) b0 = {0.f, 0.f};
    b0 = add2(b0, {g.x, 0.f});
    const Sum2 b[2] = {b0, run};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float h2 = b[i].hi * kLog2e;             // log2 e = kLog2e + 1.9e-8
        const Sum2 c = add2({h2, fmaf(b[i].hi, kLog2e, -h2)},
                            {fmaf(b[i].lo, kLog2e, b[i].hi * 1.92596299e-8f), 0.f});
        f.hi[2 * lane + i] = c.hi;
        f.lo[2 * lane + i] = c.lo;
        f.row[2 * lane + i] = scale * exp_sum(b[i]);
        f.col[2 * lane + i] = exp_sum(add2(end, minus(b[i])));
    }
    if (lane == 0) {
        f.gamma = exp_sum(end);
        f.end_hi = end.hi;
        f.end_lo = end.lo;
    }
}

// The factors of every chunk, one warp each, before the kernels that use them: what
// they take is latency (a scan and a dozen exponentials), which one warp of a block
// would make all others wait for at every chunk: 5 us for 96 heads x 2,048 tokens,
// whose gradient took 746 us with the factors and dg in the kernels, and 700 without.  Chunk c of sequence n has the slot
// start_n / 64 + n + c, as segments have their units.
__global__ void __launch_bounds__(256)
factor_kernel(const float *__restrict__ g, int per_token, SegMap chunks, int H, float scale,
              Factors *__restrict__ out) {
    const int64_t i = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    if (i >= (int64_t)chunks.units * H) return;
    const int h = (int)(i % H);
    Segment c;
    if (!find_segment(chunks, (int)(i / H), c)) return;
    make_factors(out[i], fetch_decays(g, per_token, c.t0, (int)(c.t1 - c.t0), h, H), scale);
}

// The slot of a segment's first chunk.
__device__ __forceinline__ int64_t first_slot(const SegMap &m, const Segment &s) {
    return (s.t0 - (int64_t)s.s * m.L) / kTok + s.n + (int64_t)s.s * (m.L / kTok);
}

__device__ __forceinline__ void load_factors(Factors &f, const Factors *from) {
    if (threadIdx.x < 32)
        for (unsigned e = threadIdx.x; e < sizeof(Factors) / 16; e += 32)
            cp_async16(sm100::smem_u32(&f) + 16 * e, reinterpret_cast<const char *>(from) + 16 * e, true);
}

// e^{b_i - b_j} from both sums
__device__ __forceinline__ float spread(float2 i, float2 j) {
    return sm100::ex2_approx((i.x - j.x) + (i.y - j.y));
}
__device__ __forceinline__ float2 sum_at(const Factors &f, int i) { return make_float2(f.hi[i], f.lo[i]); }

// acc += (rows of X in registers) B^T, X = hi (+ mid + lo) terms of its
// accumulators, B [64 tokens][D] in shared memory: out^T [16 rows][64 tokens].
// With three terms the two small ones of all of D go first: every addition to an
// accumulator loses up to a unit of its last place, and this way D / 16 of them
// meet it at its full size instead of 3 D / 16 (the error of dg, a difference of
// such sums, fell by half).
template <int D, int kTerms>
__device__ __forceinline__ void state_times_tile(float (&acc)[8][4], const float (&X)[D / 8][4], uint32_t b) {
    using Sh = Shape<D>;
#pragma unroll
    for (int pass = kTerms == 3 ? 0 : 1; pass < 2; ++pass) {
#pragma unroll
        for (int k = 0; k < Sh::kK; ++k) {
            uint32_t a[3][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {              // (row, k half): (g, 0), (g + 8, 0), (g, 8), (g + 8, 8)
                const float2 x = make_float2(X[2 * k + (i >> 1)][2 * (i & 1)], X[2 * k + (i >> 1)][2 * (i & 1) + 1]);
                if (kTerms == 3) split3(x, a[0][i], a[1][i], a[2][i]);
                else a[0][i] = sm100::pack_bf16(x.x, x.y);
            }
            uint32_t r[2][2][4];
            frag_b(b, Sh::kPitch, 0, 16 * k, r[0][0]);
            frag_b(b, Sh::kPitch, 16, 16 * k, r[0][1]);
#pragma unroll
            for (int n = 0; n < 2; ++n) {              // four accumulators between two uses of one
                if (n == 0) {
                    frag_b(b, Sh::kPitch, 32, 16 * k, r[1][0]);
                    frag_b(b, Sh::kPitch, 48, 16 * k, r[1][1]);
                }
#pragma unroll
                for (int t = 2; t >= 0; --t)
                    if ((pass == 0) == (t > 0))
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma(acc[4 * n + i], a[t], r[n][i >> 1][2 * (i & 1)], r[n][i >> 1][2 * (i & 1) + 1]);
            }
        }
    }
}

// X = gamma X + (Diag(c) A)^T B over a chunk: rows 16 warp .. of X are channels of A.
template <int D>
__device__ __forceinline__ void update_state(float (&X)[D / 8][4], uint32_t a_tile, uint32_t b_tile,
                                             const float *c, float gamma) {
    using Sh = Shape<D>;
    const int r0 = 16 * (threadIdx.x / 32), lane = threadIdx.x & 31;
    float add[D / 8][4];
#pragma unroll
    for (int n = 0; n < Sh::kN; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) add[n][i] = 0.f;
#pragma unroll
    for (int k = 0; k < kTok / 16; ++k) {
        constexpr int kB = Sh::kN >= 4 ? 2 : 1;        // pairs of n-tiles at once
        constexpr int kG = Sh::kN / 2 / kB;
        uint32_t r[4], a[3][4], b[2][kB][4];
        frag_at(a_tile, Sh::kPitch, r0, 16 * k, r);
#pragma unroll
        for (int i = 0; i < kB; ++i) frag_bt(b_tile, Sh::kPitch, 16 * i, 16 * k, b[0][i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = *reinterpret_cast<const float2 *>(c + 16 * k + 8 * (i >> 1) + 2 * (lane & 3));
            split3(sm100::fmul2(sm100::bf16x2_to_float2(r[i]), f), a[0][i], a[1][i], a[2][i]);
        }
#pragma unroll
        for (int n = 0; n < kG; ++n) {
            if (n + 1 < kG)
#pragma unroll
                for (int i = 0; i < kB; ++i)
                    frag_bt(b_tile, Sh::kPitch, 16 * (kB * (n + 1) + i), 16 * k, b[(n + 1) & 1][i]);
#pragma unroll
            for (int t = 2; t >= 0; --t)
#pragma unroll
                for (int i = 0; i < 2 * kB; ++i)
                    mma(add[2 * kB * n + i], a[t], b[n & 1][i >> 1][2 * (i & 1)], b[n & 1][i >> 1][2 * (i & 1) + 1]);
        }
    }
#pragma unroll
    for (int n = 0; n < Sh::kN; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) X[n][i] = fmaf(gamma, X[n][i], add[n][i]);
}

// out^T accumulators [16 channels][64 tokens] of this warp to rows of `out`
// ([T, heads, D] bf16, or fp32 partial sums of `part`).
template <int D>
__device__ __forceinline__ void store_transposed(const float (&acc)[8][4], bf16 *out, float *part, int64_t t,
                                                 int L, int heads, int head, float scale) {
    const int lane = threadIdx.x & 31, c0 = 16 * (threadIdx.x / 32);
    if (part != nullptr) {
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 8 * n + 2 * (lane & 3) + (i & 1);
                if (r < L)
                    part[((size_t)(t + r) * heads + head) * D + c0 + (lane >> 2) + 8 * (i >> 1)] = acc[n][i] * scale;
            }
        return;
    }
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const uint32_t x = transpose8(sm100::pack_bf16(acc[n][2 * hf] * scale, acc[n][2 * hf + 1] * scale));
            const int r = 8 * n + (lane >> 2);
            if (r < L)
                *reinterpret_cast<uint32_t *>(out + ((size_t)(t + r) * heads + head) * D + c0 + 8 * hf +
                                              2 * (lane & 3)) = x;
        }
}

__device__ __forceinline__ void zero8(float (&acc)[8][4]) {
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
}

// One 16 x 32 unit of the 64 x 64 products inside a chunk: C = A B^T over D.
template <int D>
__device__ __forceinline__ void unit_product(float (&c)[4][4], uint32_t a_tile, uint32_t b_tile, int r0, int n0) {
    using Sh = Shape<D>;
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[n][i] = 0.f;
#pragma unroll
    for (int k = 0; k < Sh::kK; ++k) {
        uint32_t a[4], b[4];
        frag_a(a_tile, Sh::kPitch, r0, 16 * k, a);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            frag_b(b_tile, Sh::kPitch, n0 + 16 * n, 16 * k, b);
            mma(c[2 * n], a, b[0], b[1]);
            mma(c[2 * n + 1], a, b[2], b[3]);
        }
    }
}

// The 64-token walk of a segment, forward or backward: chunk index -> first token.
struct Walk {
    int64_t t0, t1;
    int chunks, reverse;
    __device__ __forceinline__ int chunk(int i) const { return reverse ? chunks - 1 - i : i; }
    __device__ __forceinline__ int64_t first(int i) const { return t0 + (int64_t)chunk(i) * kTok; }
    __device__ __forceinline__ int rows(int i) const {
        const int64_t n = t1 - first(i);
        return (int)(n < kTok ? n : kTok);
    }
};

__device__ __forceinline__ Walk make_walk(const Segment &s, bool reverse) {
    return {s.t0, s.t1, (int)((s.t1 - s.t0 + kTok - 1) / kTok), reverse};
}

// State fragments: element (n, i) of a warp is row 16 warp + lane / 4 + 8 (i / 2),
// column 8 n + 2 (lane % 4) + i % 2.
template <int D, bool kTransposed>
__device__ __forceinline__ void load_state(float (&X)[D / 8][4], const float *from) {
    const int lane = threadIdx.x & 31, r0 = 16 * (threadIdx.x / 32) + (lane >> 2), c0 = 2 * (lane & 3);
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + 8 * (i >> 1), c = 8 * n + c0 + (i & 1);
            X[n][i] = from == nullptr ? 0.f : kTransposed ? from[(size_t)c * D + r] : from[(size_t)r * D + c];
        }
}
template <int D, bool kTransposed>
__device__ __forceinline__ void store_state(const float (&X)[D / 8][4], float *to) {
    const int lane = threadIdx.x & 31, r0 = 16 * (threadIdx.x / 32) + (lane >> 2), c0 = 2 * (lane & 3);
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = r0 + 8 * (i >> 1), c = 8 * n + c0 + (i & 1);
            to[kTransposed ? (size_t)c * D + r : (size_t)r * D + c] = X[n][i];
        }
}

// ------------------------------------------------------- segment states
template <int D>
struct StateSmem {
    bf16 a[2][Shape<D>::kTile], b[2][Shape<D>::kTile];
    Factors f[2];
};

template <int D, bool kReverse>
__global__ void __launch_bounds__(Shape<D>::kThreads)
state_kernel(const bf16 *__restrict__ x, const bf16 *__restrict__ y, const Factors *__restrict__ factors,
             SegMap m, int Hk, int H, float *__restrict__ ws, float *__restrict__ total) {
    extern __shared__ __align__(16) unsigned char raw[];
    StateSmem<D> &sm = *reinterpret_cast<StateSmem<D> *>(raw);
    const int h = blockIdx.x % H;
    Segment sg;
    if (!find_body(m, blockIdx.x / H, kReverse, sg)) return;
    const Walk w = make_walk(sg, kReverse);
    const int hk = h / (H / Hk);
    const int64_t slot = first_slot(m, sg);
    float X[D / 8][4];
    load_state<D, false>(X, nullptr);
    Sum2 sum = {0.f, 0.f};
    auto load = [&](int i) {
        load_tile<D>(sm100::smem_u32(sm.a[i & 1]), x, w.first(i), w.rows(i), Hk, hk);
        load_tile<D>(sm100::smem_u32(sm.b[i & 1]), y, w.first(i), w.rows(i), H, h);
        load_factors(sm.f[i & 1], factors + (slot + w.chunk(i)) * H + h);
        cp_commit();
    };
    load(0);
    for (int i = 0; i < w.chunks; ++i) {
        cp_wait_all();
        __syncthreads();
        if (i + 1 < w.chunks) load(i + 1);
        const Factors &f = sm.f[i & 1];
        update_state<D>(X, sm100::smem_u32(sm.a[i & 1]), sm100::smem_u32(sm.b[i & 1]), kReverse ? f.row : f.col,
                        f.gamma);
        sum = add2(sum, {f.end_hi, f.end_lo});
    }
    store_state<D, false>(X, ws + ((size_t)sg.slot * H + h) * D * D);
    if (threadIdx.x == 0) total[(size_t)sg.slot * H + h] = exp_sum(sum);
}

// -------------------------------------------------------------- outputs
template <int D>
struct OutSmem {
    bf16 q[2][Shape<D>::kTile], k[2][Shape<D>::kTile], v[2][Shape<D>::kTile];
    bf16 p[kTok * kPp];
    Factors f[2];
};

// Rows of the state are value channels here (S^T): O^T = S^T Q^T + V^T P^T.
template <int D>
__global__ void __launch_bounds__(Shape<D>::kThreads)
out_kernel(const bf16 *__restrict__ q, const bf16 *__restrict__ k, const bf16 *__restrict__ v,
           const Factors *__restrict__ factors, const float *h0, SegMap m, int Hk, int H,
           float scale, const float *__restrict__ ws, bf16 *__restrict__ o, float *hT) {
    using Sh = Shape<D>;
    extern __shared__ __align__(16) unsigned char raw[];
    OutSmem<D> &sm = *reinterpret_cast<OutSmem<D> *>(raw);
    const int h = blockIdx.x % H;
    const int u = blockIdx.x / H;
    if (blockIdx.x == 0) check_seqlens(m);
    Segment sg;
    if (!find_segment(m, u, sg)) return;
    const Walk w = make_walk(sg, false);
    const int hk = h / (H / Hk), warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int64_t slot = first_slot(m, sg);
    const float *from = ws != nullptr && sg.count > 1 ? ws + ((size_t)sg.slot * H + h) * D * D
                        : h0 != nullptr ? h0 + ((size_t)sg.n * H + h) * D * D : nullptr;
    float X[D / 8][4];
    load_state<D, true>(X, from);
    auto load = [&](int i) {
        const int64_t t = w.first(i);
        const int L = w.rows(i);
        load_tile<D>(sm100::smem_u32(sm.q[i & 1]), q, t, L, Hk, hk);
        load_tile<D>(sm100::smem_u32(sm.k[i & 1]), k, t, L, Hk, hk);
        load_tile<D>(sm100::smem_u32(sm.v[i & 1]), v, t, L, H, h);
        load_factors(sm.f[i & 1], factors + (slot + w.chunk(i)) * H + h);
        cp_commit();
    };
    if (w.chunks > 0) load(0);
    const uint32_t tp = sm100::smem_u32(sm.p);
    for (int i = 0; i < w.chunks; ++i) {
        cp_wait_all();
        __syncthreads();
        if (i + 1 < w.chunks) load(i + 1);
        const Factors &f = sm.f[i & 1];
        const uint32_t tq = sm100::smem_u32(sm.q[i & 1]), tk = sm100::smem_u32(sm.k[i & 1]),
                       tv = sm100::smem_u32(sm.v[i & 1]);
#pragma unroll 1
        for (int x = warp; x < 8; x += Sh::kWarps) {
            const int r0 = 16 * (x >> 1), n0 = 32 * (x & 1);
            if (n0 > r0 + 15) continue;                // never read
            float c[4][4];
            unit_product<D>(c, tq, tk, r0, n0);
            const float2 br[2] = {sum_at(f, r0 + (lane >> 2)), sum_at(f, r0 + (lane >> 2) + 8)};
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int j = n0 + 8 * n + 2 * (lane & 3);
                const float2 b0 = sum_at(f, j), b1 = sum_at(f, j + 1);
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int r = r0 + (lane >> 2) + 8 * hf;
                    const float a = r >= j ? c[n][2 * hf] * spread(br[hf], b0) : 0.f;
                    const float b = r >= j + 1 ? c[n][2 * hf + 1] * spread(br[hf], b1) : 0.f;
                    *reinterpret_cast<uint32_t *>(&sm.p[r * kPp + j]) = sm100::pack_bf16(a, b);
                }
            }
        }
        float acc[8][4];
        zero8(acc);
        state_times_tile<D, 1>(acc, X, tq);
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const float2 e = *reinterpret_cast<const float2 *>(&f.row[8 * n + 2 * (lane & 3)]);
            acc[n][0] *= e.x; acc[n][1] *= e.y; acc[n][2] *= e.x; acc[n][3] *= e.y;
        }
        __syncthreads();
        float in[8][4];                                // P carries no scale
        zero8(in);
#pragma unroll
        for (int kk = 0; kk < kTok / 16; ++kk) {
            uint32_t a[4], b[4];
            frag_at(tv, Sh::kPitch, 16 * warp, 16 * kk, a);
#pragma unroll
            for (int n = kk; n < 4; ++n) {             // tokens 16 n .. see those from 16 kk on
                frag_b(tp, kPp, 16 * n, 16 * kk, b);
                mma(in[2 * n], a, b[0], b[1]);
                mma(in[2 * n + 1], a, b[2], b[3]);
            }
        }
#pragma unroll
        for (int n = 0; n < 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[n][e] = fmaf(in[n][e], scale, acc[n][e]);
        store_transposed<D>(acc, o, nullptr, w.first(i), w.rows(i), H, h, 1.f);
        update_state<D>(X, tv, tk, f.col, f.gamma);
    }
    if (hT != nullptr && sg.s == sg.count - 1)
        store_state<D, true>(X, hT + ((size_t)sg.n * H + h) * D * D);
}

// ------------------------------------------------------------- gradient
template <int D>
struct GradSmem {
    bf16 q[2][Shape<D>::kTile], k[2][Shape<D>::kTile], v[2][Shape<D>::kTile], dO[2][Shape<D>::kTile];
    bf16 p[kTok * kPp], a[kTok * kPp];
    Factors f[2];
    float inner[4][kTok];              // parts of the row or column sums of W
    float outer[Shape<D>::kWarps][kTok];
    double red[Shape<D>::kWarps];
};
template <int D>
struct GradKvSmem : GradSmem<D> {
    // its rows are read by ldmatrix; without the alignment they may start in the
    // padding at the end of the base
    __align__(16) bf16 e[D * Shape<D>::kPitch];
};

// P, dA and W = P . dP of a chunk: P (scaled) and dA as bf16 tiles, and the sums of
// W's rows (kRows: inner[half][row]) or columns (inner[row block][column]).
template <int D, bool kRows>
__device__ __forceinline__ void inside_chunk(GradSmem<D> &sm, int buf, const Factors &f, float scale) {
    using Sh = Shape<D>;
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const uint32_t tq = sm100::smem_u32(sm.q[buf]), tk = sm100::smem_u32(sm.k[buf]),
                   tv = sm100::smem_u32(sm.v[buf]), td = sm100::smem_u32(sm.dO[buf]);
#pragma unroll 1
    for (int x = warp; x < 8; x += Sh::kWarps) {
        const int r0 = 16 * (x >> 1), n0 = 32 * (x & 1);
        if (n0 > r0 + 15) {                            // above the diagonal: sums of nothing
            if (kRows && (lane & 3) == 0) sm.inner[x & 1][r0 + (lane >> 2)] = sm.inner[x & 1][r0 + 8 + (lane >> 2)] = 0.f;
            if (!kRows) sm.inner[x >> 1][n0 + lane] = 0.f;
            continue;
        }
        float c[4][4], d[4][4];
        unit_product<D>(c, tq, tk, r0, n0);
        unit_product<D>(d, td, tv, r0, n0);
        float sum[2] = {0.f, 0.f};
        const float2 br[2] = {sum_at(f, r0 + (lane >> 2)), sum_at(f, r0 + (lane >> 2) + 8)};
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int j = n0 + 8 * n + 2 * (lane & 3);
            const float2 bj[2] = {sum_at(f, j), sum_at(f, j + 1)};
            float col[2] = {0.f, 0.f};
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int r = r0 + (lane >> 2) + 8 * hf;
                float p[2], da[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float e = scale * spread(br[hf], bj[i]);
                    const bool in = r >= j + i;        // above the diagonal e may be anything
                    p[i] = in ? c[n][2 * hf + i] * e : 0.f;
                    da[i] = in ? d[n][2 * hf + i] * e : 0.f;
                    const float w = in ? p[i] * d[n][2 * hf + i] : 0.f;
                    sum[hf] += w;
                    col[i] += w;
                }
                if (!kRows) *reinterpret_cast<uint32_t *>(&sm.p[r * kPp + j]) = sm100::pack_bf16(p[0], p[1]);
                *reinterpret_cast<uint32_t *>(&sm.a[r * kPp + j]) = sm100::pack_bf16(da[0], da[1]);
            }
            if (!kRows) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) col[i] += __shfl_xor_sync(0xffffffffu, col[i], o);
                    if (lane < 4) sm.inner[x >> 1][j + i] = col[i];
                }
            }
        }
        if (kRows)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) sum[hf] += __shfl_xor_sync(0xffffffffu, sum[hf], o);
                if ((lane & 3) == 0) sm.inner[x & 1][r0 + (lane >> 2) + 8 * hf] = sum[hf];
            }
    }
}

// acc [16 channels][64 tokens] scaled by the tokens' factors; the dot of each
// token's 16 channels with those of `tile` goes to outer[warp][token].
template <int D>
__device__ __forceinline__ void scale_and_dot(float (&acc)[8][4], const float *factor, uint32_t tile, float *outer) {
    using Sh = Shape<D>;
    const int lane = threadIdx.x & 31, c0 = 16 * (threadIdx.x / 32);
#pragma unroll
    for (int n = 0; n < 8; n += 2) {
        uint32_t x[4];                                 // tile^T: (n, rows 0-7), (n, 8-15), (n + 1, ..)
        const int l = lane;
        ldmatrix_trans(tile + 2u * ((8 * n + (l & 7) + 8 * (l >> 4)) * Sh::kPitch + c0 + 8 * ((l >> 3) & 1)), x);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            float(&a)[4] = acc[n + s];
            const float2 e = *reinterpret_cast<const float2 *>(&factor[8 * (n + s) + 2 * (lane & 3)]);
            a[0] *= e.x; a[1] *= e.y; a[2] *= e.x; a[3] *= e.y;
            const float2 lo = sm100::bf16x2_to_float2(x[2 * s]), hi = sm100::bf16x2_to_float2(x[2 * s + 1]);
            float d0 = fmaf(a[0], lo.x, a[2] * hi.x), d1 = fmaf(a[1], lo.y, a[3] * hi.y);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                d0 += __shfl_xor_sync(0xffffffffu, d0, o);
                d1 += __shfl_xor_sync(0xffffffffu, d1, o);
            }
            if (lane < 4) {
                outer[8 * (n + s) + 2 * lane] = d0;
                outer[8 * (n + s) + 2 * lane + 1] = d1;
            }
        }
    }
}

// One block per SM takes the longest units first (6 documents of 100 to 3,000 tokens,
// 16 heads of 128: 738 -> 678 us).  Where an SM has several, that would put the long
// ones together on the same SMs (the same with heads of 64: 278 -> 296 us).
template <int D>
__device__ __forceinline__ int grad_unit(const SegMap &m, int i, unsigned char *smem) {
    if constexpr (D == 128) return ranked_unit<Shape<D>::kThreads>(m, i, reinterpret_cast<int *>(smem));
    return i;
}

// dQ, x_i = q_i . dq_i (term) and <S_end, E_end> (anchor).  194 us for 96 heads x
// 2,048 tokens, 210 us for 10,824 packed tokens of 16 heads.
template <int D>
__global__ void __launch_bounds__(Shape<D>::kThreads)
grad_q_kernel(const bf16 *__restrict__ q, const bf16 *__restrict__ k, const bf16 *__restrict__ v,
              const bf16 *__restrict__ dO, const Factors *__restrict__ factors,
              const float *__restrict__ h0, const float *__restrict__ dhT, SegMap m, int Hk, int H,
              float scale, const float *__restrict__ wsS, const float *__restrict__ wsE,
              bf16 *__restrict__ dq, float *__restrict__ part, float *__restrict__ term,
              double *__restrict__ anchor) {
    using Sh = Shape<D>;
    extern __shared__ __align__(16) unsigned char raw[];
    GradSmem<D> &sm = *reinterpret_cast<GradSmem<D> *>(raw);
    const int h = blockIdx.x % H;
    const int u = grad_unit<D>(m, blockIdx.x / H, raw);
    if (blockIdx.x == 0) check_seqlens(m);
    Segment sg;
    if (!find_segment(m, u, sg)) return;
    const Walk w = make_walk(sg, false);
    const int hk = h / (H / Hk), warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int64_t slot = first_slot(m, sg);
    const size_t seg = ((size_t)sg.slot * H + h) * D * D, seq = ((size_t)sg.n * H + h) * D * D;
    float X[D / 8][4];
    load_state<D, false>(X, wsS != nullptr && sg.count > 1 ? wsS + seg : h0 != nullptr ? h0 + seq : nullptr);
    auto load = [&](int i) {
        const int64_t t = w.first(i);
        const int L = w.rows(i);
        load_tile<D>(sm100::smem_u32(sm.q[i & 1]), q, t, L, Hk, hk);
        load_tile<D>(sm100::smem_u32(sm.k[i & 1]), k, t, L, Hk, hk);
        load_tile<D>(sm100::smem_u32(sm.v[i & 1]), v, t, L, H, h);
        load_tile<D>(sm100::smem_u32(sm.dO[i & 1]), dO, t, L, H, h);
        load_factors(sm.f[i & 1], factors + (slot + w.chunk(i)) * H + h);
        cp_commit();
    };
    if (w.chunks > 0) load(0);
    const uint32_t ta = sm100::smem_u32(sm.a);
    for (int i = 0; i < w.chunks; ++i) {
        cp_wait_all();
        __syncthreads();
        if (i + 1 < w.chunks) load(i + 1);
        const Factors &f = sm.f[i & 1];
        const uint32_t tq = sm100::smem_u32(sm.q[i & 1]), tk = sm100::smem_u32(sm.k[i & 1]),
                       tv = sm100::smem_u32(sm.v[i & 1]), td = sm100::smem_u32(sm.dO[i & 1]);
        inside_chunk<D, true>(sm, i & 1, f, scale);
        float acc[8][4];                               // dQ^T
        zero8(acc);
        state_times_tile<D, 3>(acc, X, td);
        scale_and_dot<D>(acc, f.row, tq, sm.outer[warp]);
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < kTok / 16; ++kk) {
            uint32_t a[4], b[4];
            frag_at(tk, Sh::kPitch, 16 * warp, 16 * kk, a);
#pragma unroll
            for (int n = kk; n < 4; ++n) {
                frag_b(ta, kPp, 16 * n, 16 * kk, b);
                mma(acc[2 * n], a, b[0], b[1]);
                mma(acc[2 * n + 1], a, b[2], b[3]);
            }
        }
        const int64_t t = w.first(i);
        const int L = w.rows(i);
        store_transposed<D>(acc, dq, part, t, L, H, h, 1.f);
        for (int r = threadIdx.x; r < L; r += Sh::kThreads) {
            float s = sm.inner[0][r] + sm.inner[1][r];
#pragma unroll
            for (int x = 0; x < Sh::kWarps; ++x) s += sm.outer[x][r];
            term[(size_t)(t + r) * H + h] = s;
        }
        update_state<D>(X, tk, tv, f.col, f.gamma);
    }
    const float *to = wsE != nullptr && sg.count > 1 ? wsE + seg : dhT != nullptr ? dhT + seq : nullptr;
    double s = 0.0;
    if (to != nullptr) {
        float E[D / 8][4];
        load_state<D, false>(E, to);
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) s += (double)X[n][i] * (double)E[n][i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) sm.red[warp] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        s = 0.0;
        for (int i = 0; i < Sh::kWarps; ++i) s += sm.red[i];
        anchor[(size_t)u * H + h] = s;
    }
}

// dK, dV, y_j = k_j . dk_j and dh0, chunks last to first.  240 us for 96 heads x 2,048
// tokens, 260 us for 10,824 packed tokens of 16 heads.
template <int D>
__global__ void __launch_bounds__(Shape<D>::kThreads)
grad_kv_kernel(const bf16 *__restrict__ q, const bf16 *__restrict__ k, const bf16 *__restrict__ v,
               const bf16 *__restrict__ dO, const Factors *__restrict__ factors,
               const float *__restrict__ dhT, SegMap m, int Hk, int H, float scale,
               const float *__restrict__ wsE, bf16 *__restrict__ dk, float *__restrict__ part,
               bf16 *__restrict__ dv, float *__restrict__ term, float *__restrict__ dh0) {
    using Sh = Shape<D>;
    extern __shared__ __align__(16) unsigned char raw[];
    GradKvSmem<D> &sm = *reinterpret_cast<GradKvSmem<D> *>(raw);
    const int h = blockIdx.x % H;
    const int u = grad_unit<D>(m, blockIdx.x / H, raw);
    Segment sg;
    if (!find_segment(m, u, sg)) return;
    const Walk w = make_walk(sg, true);
    const int hk = h / (H / Hk), warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int64_t slot = first_slot(m, sg);
    const size_t seg = ((size_t)sg.slot * H + h) * D * D, seq = ((size_t)sg.n * H + h) * D * D;
    float X[D / 8][4];
    load_state<D, false>(X, wsE != nullptr && sg.count > 1 ? wsE + seg : dhT != nullptr ? dhT + seq : nullptr);
    auto load = [&](int i) {
        const int64_t t = w.first(i);
        const int L = w.rows(i);
        load_tile<D>(sm100::smem_u32(sm.q[i & 1]), q, t, L, Hk, hk);
        load_tile<D>(sm100::smem_u32(sm.k[i & 1]), k, t, L, Hk, hk);
        load_tile<D>(sm100::smem_u32(sm.v[i & 1]), v, t, L, H, h);
        load_tile<D>(sm100::smem_u32(sm.dO[i & 1]), dO, t, L, H, h);
        load_factors(sm.f[i & 1], factors + (slot + w.chunk(i)) * H + h);
        cp_commit();
    };
    if (w.chunks > 0) load(0);
    const uint32_t ta = sm100::smem_u32(sm.a), tp = sm100::smem_u32(sm.p), te = sm100::smem_u32(sm.e);
    for (int i = 0; i < w.chunks; ++i) {
        const int64_t t = w.first(i);
        const int L = w.rows(i);
        cp_wait_all();
        __syncthreads();
        if (i + 1 < w.chunks) load(i + 1);
        const Factors &f = sm.f[i & 1];
        const uint32_t tq = sm100::smem_u32(sm.q[i & 1]), tk = sm100::smem_u32(sm.k[i & 1]),
                       tv = sm100::smem_u32(sm.v[i & 1]), td = sm100::smem_u32(sm.dO[i & 1]);
        inside_chunk<D, false>(sm, i & 1, f, scale);
#pragma unroll
        for (int n = 0; n < Sh::kN; ++n)               // E in bf16, for dV alone
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
                *reinterpret_cast<uint32_t *>(&sm.e[(16 * warp + (lane >> 2) + 8 * hf) * Sh::kPitch + 8 * n +
                                                    2 * (lane & 3)]) =
                    sm100::pack_bf16(X[n][2 * hf], X[n][2 * hf + 1]);
        {
            float acc[8][4];                           // dK^T
            zero8(acc);
            state_times_tile<D, 3>(acc, X, tv);
            scale_and_dot<D>(acc, f.col, tk, sm.outer[warp]);
            __syncthreads();
#pragma unroll
            for (int kk = 0; kk < kTok / 16; ++kk) {
                uint32_t a[4], b[4];
                frag_at(tq, Sh::kPitch, 16 * warp, 16 * kk, a);
#pragma unroll
                for (int n = 0; n <= kk; ++n) {        // keys 16 n .. are seen from 16 kk on
                    frag_bt(ta, kPp, 16 * n, 16 * kk, b);
                    mma(acc[2 * n], a, b[0], b[1]);
                    mma(acc[2 * n + 1], a, b[2], b[3]);
                }
            }
            store_transposed<D>(acc, dk, part, t, L, H, h, 1.f);
        }
        constexpr int kCols = D < 32 ? D : 32, kUnits = 4 * (D / kCols);
#pragma unroll 1
        for (int x = warp; x < kUnits; x += Sh::kWarps) {
            const int r0 = 16 * (x & 3), n0 = kCols * (x >> 2);
            float c[kCols / 8][4];
#pragma unroll
            for (int n = 0; n < kCols / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) c[n][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < Sh::kK; ++kk) {      // K E
                uint32_t a[4], b[4];
                frag_a(tk, Sh::kPitch, r0, 16 * kk, a);
#pragma unroll
                for (int n = 0; n < kCols / 16; ++n) {
                    frag_bt(te, Sh::kPitch, n0 + 16 * n, 16 * kk, b);
                    mma(c[2 * n], a, b[0], b[1]);
                    mma(c[2 * n + 1], a, b[2], b[3]);
                }
            }
            const float f0 = f.col[r0 + (lane >> 2)], f1 = f.col[r0 + 8 + (lane >> 2)];
#pragma unroll
            for (int n = 0; n < kCols / 8; ++n) {
                c[n][0] *= f0; c[n][1] *= f0; c[n][2] *= f1; c[n][3] *= f1;
            }
#pragma unroll 1
            for (int kk = r0 / 16; kk < kTok / 16; ++kk) {   // P^T dO, rows from r0 on
                uint32_t a[4], b[4];
                frag_at(tp, kPp, r0, 16 * kk, a);
#pragma unroll
                for (int n = 0; n < kCols / 16; ++n) {
                    frag_bt(td, Sh::kPitch, n0 + 16 * n, 16 * kk, b);
                    mma(c[2 * n], a, b[0], b[1]);
                    mma(c[2 * n + 1], a, b[2], b[3]);
                }
            }
#pragma unroll
            for (int n = 0; n < kCols / 8; ++n)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int r = r0 + (lane >> 2) + 8 * hf;
                    if (r < L)
                        *reinterpret_cast<uint32_t *>(dv + ((size_t)(t + r) * H + h) * D + n0 + 8 * n +
                                                      2 * (lane & 3)) =
                            sm100::pack_bf16(c[n][2 * hf], c[n][2 * hf + 1]);
                }
        }
        for (int r = threadIdx.x; r < L; r += Sh::kThreads) {
            float y = 0.f;
#pragma unroll
            for (int z = 0; z < 4; ++z) y += sm.inner[z][r];
#pragma unroll
            for (int z = 0; z < Sh::kWarps; ++z) y += sm.outer[z][r];
            term[(size_t)(t + r) * H + h] -= y;        // x of the other walk, minus y
        }
        update_state<D>(X, tq, td, f.row, f.gamma);
    }
    if (dh0 != nullptr && sg.s == 0) store_state<D, false>(X, dh0 + seq);
}

// dg_t = sum over the segment's tokens from t on of (x - y), plus <S_end, E_end>:
// lanes are heads, the warps of a block take an equal share of the tokens each (their
// totals first), sums in fp64.  With a constant decay the segment's sum goes out.
// A few blocks with a chain of loads and sums each: latency alone, 13.5 us for 96
// heads x 3 segments of 683 tokens (18.2 us with eight loads at a time).
constexpr int kDecayWarps = 32, kDecayAhead = 16;
__global__ void __launch_bounds__(32 * kDecayWarps)
decay_grad_kernel(const float *__restrict__ term, const double *__restrict__ anchor, int per_token, SegMap m,
                  int H, float *__restrict__ dg, double *__restrict__ head_sum) {
    __shared__ double total[kDecayWarps][33];
    const int u = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int h = blockIdx.y * 32 + lane;
    Segment sg;
    const bool live = find_segment(m, u, sg);
    if (!live) {
        if (!per_token && warp == 0 && h < H) head_sum[(size_t)u * H + h] = 0.0;
        return;
    }
    const int len = (int)(sg.t1 - sg.t0), per = (len + kDecayWarps - 1) / kDecayWarps;
    const int a = min(warp * per, len), b = min(a + per, len);
    // the shares' terms from the last token on, sixteen loads at a time
    auto walk = [&](auto visit) {
        if (h >= H) return;
        const float *p = term + (size_t)sg.t0 * H + h;
        for (int t = b - 1; t >= a; t -= kDecayAhead) {
            float x[kDecayAhead];
#pragma unroll
            for (int i = 0; i < kDecayAhead; ++i)
                if (t - i >= a) x[i] = p[(size_t)(t - i) * H];
#pragma unroll
            for (int i = 0; i < kDecayAhead; ++i)
                if (t - i >= a) visit(t - i, (double)x[i]);
        }
    };
    double s = 0.0;
    walk([&](int, double x) { s += x; });
    total[warp][lane] = s;
    __syncthreads();
    s = h < H ? anchor[(size_t)u * H + h] : 0.0;
    for (int i = kDecayWarps - 1; i > warp; --i) s += total[i][lane];
    double all = 0.0;
    float *out = dg + (size_t)(per_token ? sg.t0 : 0) * H + h;
    walk([&](int t, double x) {
        s += x;
        if (per_token) out[(size_t)t * H] = (float)s;
        all += s;
    });
    if (per_token) return;
    __syncthreads();
    total[warp][lane] = all;
    __syncthreads();
    if (warp == 0 && h < H) {
        all = 0.0;
        for (int i = 0; i < kDecayWarps; ++i) all += total[i][lane];
        head_sum[(size_t)u * H + h] = all;
    }
}

}  // namespace mm
}  // namespace lin
}  // namespace kda
