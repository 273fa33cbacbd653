// kda_linear_sm100.cuh -- decayed linear attention, bf16, d = 128, on the 5th-gen
// tensor cores: outputs and segment states.
//
// One CTA walks one segment of one (sequence, head) in chunks of C = 128 tokens.
// With b_i the decay sum inside the chunk and m a level between its extremes:
//
//   O = Diag(r) ( P' V + Q S'' ),   P'_ij = (Q K^T)_ij e^{m - b_j} for i >= j,
//   S'' = e^m S0,                   r_i = scale e^{b_i - m}
//   S = e^{b_C} S0 + V'^T K,        V'_j = e^{b_C - b_j} v_j     (S held as [value][key])
//
// so both products of O share one accumulator and the decay costs one multiply
// per element of P' and one per element of O.  The level is the middle of the
// extremes, and a chunk whose b stays within 60 of it keeps every factor inside
// e^{+-60}, far inside the range of bf16 and fp32.  A chunk that decays further
// takes the slow form: P'_ij e^{b_i - b_j} by an exponential of its own, the rows
// of Q scaled by e^{b_i} in place, m = 0.
//
// Precision.  O rounds P' and S'' to bf16 once each (2^-8 of a term); its sum and
// the row factor are fp32.  S is fp32 in registers and must not take a bf16
// rounding per token, so V' goes to the tensor cores as three bf16 terms (24
// bits) whose products with K are exact, accumulated in fp32 from the smallest
// term up; each chunk's sum starts from zero and is added to S with rounding to
// nearest.
//
// Roles of the 16 warps: 0 loads and stores tiles (TMA); 1 issues Q K^T, P' V and
// Q S''; 2 forms the decay factors a chunk ahead; 3 issues V'^T K; 4-7 (thread =
// token) turn Q K^T into P' and write O; 8-15 (thread = value channel, half of the
// key channels each) form V' and carry S.  The two halves of a chunk's V' have
// buffers of their own, so the next chunk's first half is formed while the tensor
// cores work on this one's second, and only S'' ties a chunk to the one before.
// Tensor memory (512 columns): Q K^T, then O 128 | P' 64 | V'^T K 128 | V' 2 x 96.
// Shared memory: two stages of Q, K, V (96 KB each; O leaves through Q's tile) and
// S'' (32 KB).
#pragma once

#include "kda_linear_common.cuh"
#include "sm100_ptx.cuh"

namespace kda {
namespace lin {
namespace tc {

using namespace kda::sm100;

constexpr int kD = 128, kTok = 128, kThreads = 512, kStages = 2;
constexpr uint32_t kTile = kTok * kD * 2;              // 32 KB; two halves of 64 channels
constexpr uint32_t kHalf = kTile / 2;
constexpr uint32_t kStageBytes = 3 * kTile;            // Q, K, V
constexpr uint32_t kOffS = kStages * kStageBytes;      // S''
constexpr uint32_t kOffSmall = kOffS + kTile;

// Tensor-memory columns.
constexpr uint32_t kColX = 0, kColP = 128, kColD = 192, kColV = 320, kVBuf = 96, kVPart = 32;

constexpr float kRange = 60.f;                         // |b - m| of the fast form
constexpr unsigned long long kWaitLimit = 4000000000ull;   // about 2 s of SM clock

struct __align__(16) Decay {
    float x[kTok], y[kTok];    // fast: e^{m - b}, r;  slow: b as a sum of two floats
    float kv;                  // fast: e^{b_C - m}
    float em;                  // e^m (slow: 1)
    float gamma;               // e^{b_C}
    float end_hi, end_lo;      // slow: b_C
    int slow;
};

struct Small {
    Decay dec[kStages];
    uint64_t full[kStages], dec_full[kStages], dec_free[kStages];
    uint64_t staged[kStages], k_free[kStages];
    uint64_t d1_full, p_ready, o_full, x_free, s_ready;
    uint64_t v_full[2], v_free[2], ds_full, ds_free;
    uint64_t drain[2];
    uint32_t tmem;
    volatile int abort;
};

constexpr uint32_t kSmem = kOffSmall + sizeof(Small);
static_assert(kSmem <= 232448, "shared memory");

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// A wait that every lane polls; false after the limit, or once another role gave up.
__device__ __forceinline__ bool wait(Small &sm, uint64_t *bar, uint32_t parity) {
    const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, &sm.abort, kWaitLimit));
    if (!ok) {
        if (!sm.abort) raise_error(kErrTimeout);
        sm.abort = 1;
    }
    return ok;
}

// One arrival of a warp, after all of its lanes.
__device__ __forceinline__ void arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// tcgen05.st 16 lanes x 128 bits, four times: 16 columns.  Register 2 c + r holds
// row lane / 4 + 8 r, column 4 c + lane % 4: the fragments of ldmatrix.
__device__ __forceinline__ void tmem_st_frag(uint32_t addr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

__device__ __forceinline__ void ldmatrix_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// x = hi + mid + lo in bf16 pairs; what is left is below 2^-24 of x.
__device__ __forceinline__ void split3(float2 x, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    hi = pack_bf16(x.x, x.y);
    float2 h = bf16x2_to_float2(hi);
    x = fadd2(x, make_float2(-h.x, -h.y));
    mid = pack_bf16(x.x, x.y);
    h = bf16x2_to_float2(mid);
    x = fadd2(x, make_float2(-h.x, -h.y));
    lo = pack_bf16(x.x, x.y);
}

struct Params {
    const float *g, *h0;
    const float *ws;           // start states of segments, or NULL
    float *out;                // hT, or the segments' R
    float *total;              // R: the segments' decays
    __nv_bfloat16 *o;
    SegMap m;
    int per_token, Hk, H;
    float scale;
};

// Decay factors of chunk tokens 4 lane .. 4 lane + 3 (warp 2); returns b_C.
__device__ __forceinline__ double decay_factors(Decay &d, const float (&g)[4], float scale) {
    const int lane = threadIdx.x & 31;
    double b[4], run = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = run += (double)g[i];
    const double before = warp_scan(run) - run;
    float top, low;
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] += before;
    top = fmaxf(fmaxf((float)b[0], (float)b[1]), fmaxf((float)b[2], (float)b[3]));
    low = fminf(fminf((float)b[0], (float)b[1]), fminf((float)b[2], (float)b[3]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
    }
    const double end = __shfl_sync(0xffffffffu, b[3], 31);
    const double m = 0.5 * ((double)top + (double)low);
    const bool slow = !(top - low <= 2.f * kRange);    // NaN: slow
    if (slow) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            d.x[4 * lane + i] = (float)b[i];
            d.y[4 * lane + i] = (float)(b[i] - (double)(float)b[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            d.x[4 * lane + i] = expf((float)(m - b[i]));
            d.y[4 * lane + i] = scale * expf((float)(b[i] - m));
        }
    }
    if (lane == 0) {
        d.kv = slow ? 1.f : expf((float)(end - m));
        d.em = slow ? 1.f : expf((float)m);
        d.gamma = expf((float)end);
        d.end_hi = (float)end;
        d.end_lo = (float)(end - (double)(float)end);
        d.slow = slow;
    }
    return end;
}

// Longest first.  Blocks start in index order, so with the units of a batch in
// decreasing length the last to start are the short ones; each block ranks the
// units itself (ties by index, so the ranks are a permutation).  Up to one unit a
// thread; above that there are enough of them for their order not to matter.
__device__ __forceinline__ int ranked_unit(const SegMap &m, int rank, int *len) {
    const int t = threadIdx.x;
    if (t < m.units) {
        Segment g;
        len[t] = find_segment(m, t, g) ? (int)(g.t1 - g.t0) : -1;
    }
    if (t == 0) len[kThreads] = 0;
    __syncthreads();
    if (t < m.units) {
        const int mine = len[t];
        int r = 0;
        for (int j = 0; j < m.units; ++j) r += (len[j] > mine) | ((len[j] == mine) & (j < t));
        if (r == rank) len[kThreads] = t;
    }
    __syncthreads();
    const int u = len[kThreads];
    __syncthreads();
    return u;
}

// kStates: only S is wanted, from zero; R and the decay of the segment go out.
template <bool kStates>
__global__ void __launch_bounds__(kThreads, 1)
linear_sm100_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o,
                    const Params p) {
    extern __shared__ __align__(1024) unsigned char sh[];
    Small &sm = *reinterpret_cast<Small *>(sh + kOffSmall);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int h = blockIdx.x % p.H;
    int u = blockIdx.x / p.H;
    if (!kStates && blockIdx.x == 0) check_seqlens(p.m);
    if (p.m.cu != nullptr && p.m.units > 1 && p.m.units <= kThreads)
        u = ranked_unit(p.m, u, reinterpret_cast<int *>(sh + kOffS));
    Segment sg;
    if (!find_segment(p.m, u, sg)) return;
    if (kStates && sg.s == sg.count - 1) return;
    const int chunks = (int)((sg.t1 - sg.t0 + kTok - 1) / kTok);
    const int hk = h / (p.H / p.Hk);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.dec_full[i], 1);
            mbar_init(&sm.dec_free[i], kStates ? 8 : 12);
            mbar_init(&sm.staged[i], 4);
            mbar_init(&sm.k_free[i], 1);
            mbar_init(&sm.v_full[i], 8);
            mbar_init(&sm.v_free[i], 1);
        }
        mbar_init(&sm.d1_full, 1);
        mbar_init(&sm.p_ready, 4);
        mbar_init(&sm.o_full, 1);
        mbar_init(&sm.x_free, 4);
        mbar_init(&sm.s_ready, 8);
        mbar_init(&sm.ds_full, 1);
        mbar_init(&sm.ds_free, 8);
        mbar_init(&sm.drain[0], 1);
        mbar_init(&sm.drain[1], 1);
        sm.abort = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sm.tmem;
    const uint32_t base = smem_u32(sh);
    auto rows_of = [&](int c) { return (int)(sg.t1 - sg.t0 - (int64_t)c * kTok < kTok
                                                 ? sg.t1 - sg.t0 - (int64_t)c * kTok : kTok); };

    if (warp == 0) {
        // ------------------------------------------------------------ tiles
        auto load = [&](int c) {
            if (elect_one()) {
                unsigned char *st = sh + (c & 1) * kStageBytes;
                uint64_t *bar = &sm.full[c & 1];
                const int t = (int)(sg.t0 + (int64_t)c * kTok);
                mbar_expect_tx(bar, kStates ? 2 * kTile : 3 * kTile);
                tma_load_3d(st + kTile, &map_k, bar, 0, hk, t);
                tma_load_3d(st + kTile + kHalf, &map_k, bar, 64, hk, t);
                if (!kStates) {
                    tma_load_3d(st, &map_q, bar, 0, hk, t);
                    tma_load_3d(st + kHalf, &map_q, bar, 64, hk, t);
                }
                tma_load_3d(st + 2 * kTile, &map_v, bar, 0, h, t);
                tma_load_3d(st + 2 * kTile + kHalf, &map_v, bar, 64, h, t);
            }
            __syncwarp();
        };
        for (int c = 0; c < kStages && c < chunks; ++c) load(c);
        int c = 0;
        for (; c < chunks; ++c) {
            if (!kStates) {
                if (!wait(sm, &sm.staged[c & 1], (c >> 1) & 1)) break;
                if (rows_of(c) == kTok) {
                    if (elect_one()) {
                        const unsigned char *st = sh + (c & 1) * kStageBytes;
                        const int t = (int)(sg.t0 + (int64_t)c * kTok);
                        tma_store_3d(&map_o, st, 0, h, t);
                        tma_store_3d(&map_o, st + kHalf, 64, h, t);
                        bulk_commit_group();
                        bulk_wait_group_read<0>();
                    }
                    __syncwarp();
                }
            }
            if (!wait(sm, &sm.k_free[c & 1], (c >> 1) & 1)) break;
            if (c + kStages < chunks) load(c + kStages);
        }
        if (c < chunks) {                              // gave up: let the copies in flight land
            const int issued = c + kStages < chunks ? c + kStages : chunks;
            for (int i = c; i < issued; ++i) mbar_wait_drain(&sm.full[i & 1], (i >> 1) & 1, kWaitLimit);
        }
        if (elect_one()) bulk_wait_group<0>();
        __syncwarp();
    } else if (warp == 1 && !kStates) {
        // ------------------------------------------- Q K^T, then P' V + Q S''
        constexpr uint32_t id_kk = idesc_bf16(128, 128, false, false);
        constexpr uint32_t id_kn = idesc_bf16(128, 128, false, true);
        const uint64_t ds = sdesc(base + kOffS, kHalf, 1024, kLayoutSW128);
        int c = 0;
        for (; c < chunks; ++c) {
            const uint32_t st = base + (c & 1) * kStageBytes;
            const uint64_t dq = sdesc(st, kHalf, 1024, kLayoutSW128);
            const uint64_t dk = sdesc(st + kTile, kHalf, 1024, kLayoutSW128);
            const uint64_t dv = sdesc(st + 2 * kTile, kHalf, 1024, kLayoutSW128);
            if (!wait(sm, &sm.full[c & 1], (c >> 1) & 1)) break;
            if (c > 0 && !wait(sm, &sm.x_free, (c - 1) & 1)) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t off = (k & 3) * 32 + (k >> 2) * kHalf;
                    mma_ss(tm + kColX, sdesc_at(dq, off), sdesc_at(dk, off), id_kk, k > 0);
                }
                tc_commit(&sm.d1_full);
            }
            __syncwarp();
            if (!wait(sm, &sm.s_ready, c & 1)) break;
            if (!wait(sm, &sm.p_ready, c & 1)) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint32_t off = (k & 3) * 32 + (k >> 2) * kHalf;
                    mma_ss(tm + kColX, sdesc_at(dq, off), sdesc_at(ds, off), id_kk, k > 0);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    mma_ts(tm + kColX, tm + kColP + 8 * k, sdesc_at(dv, 2048 * k), id_kn, 1);
                tc_commit(&sm.o_full);
            }
            __syncwarp();
        }
    } else if (warp == 2) {
        // ----------------------------------------------------------- decays
        float g[4], next[4];
        auto fetch = [&](int c, float (&x)[4]) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t t = sg.t0 + (int64_t)c * kTok + 4 * lane + i;
                x[i] = t < sg.t1 ? load_decay(p.g, p.per_token, t, h, p.H) : 0.f;
            }
        };
        double sum = 0.0;
        if (chunks > 0) fetch(0, next);
        for (int c = 0; c < chunks; ++c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) g[i] = next[i];
            if (c + 1 < chunks) fetch(c + 1, next);
            if (c >= kStages && !wait(sm, &sm.dec_free[c & 1], ((c >> 1) - 1) & 1)) break;
            sum += decay_factors(sm.dec[c & 1], g, p.scale);
            arrive(&sm.dec_full[c & 1]);
        }
        if (kStates && lane == 0) p.total[(size_t)u * p.H + h] = expf((float)sum);
    } else if (warp == 3) {
        // ------------------------------------------------------------ V'^T K
        constexpr uint32_t id = idesc_bf16(128, 128, false, true);
        for (int c = 0; c < chunks; ++c) {
            const uint64_t dk = sdesc(base + (c & 1) * kStageBytes + kTile, kHalf, 1024, kLayoutSW128);
            bool ok = true;
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                if (!ok) break;
                ok = wait(sm, &sm.v_full[hf], c & 1);
                if (ok && hf == 0 && c > 0) ok = wait(sm, &sm.ds_free, (c - 1) & 1);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int part = 2; part >= 0; --part)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_ts(tm + kColD, tm + kColV + hf * kVBuf + part * kVPart + 8 * k,
                                   sdesc_at(dk, 2048 * (4 * hf + k)), id, hf > 0 || part < 2 || k > 0);
                    tc_commit(&sm.v_free[hf]);
                    if (hf == 1) {
                        tc_commit(&sm.ds_full);
                        tc_commit(&sm.k_free[c & 1]);
                    }
                }
                __syncwarp();
            }
            if (!ok) break;
        }
    } else if (warp < 8 && !kStates && warp >= 4) {
        // ------------------------------------------------ P' and O (thread = token)
        const int w = warp - 4, row = 32 * w + lane;
        const uint32_t tq = tm + ((uint32_t)(32 * w) << 16);
        uint32_t z[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = 0u;
        for (int jb = w + 1; jb < 4; ++jb) tmem_st16(tq + kColP + 16 * jb, z);   // stays zero
        tmem_wait_st();
        for (int c = 0; c < chunks; ++c) {
            const Decay &d = sm.dec[c & 1];
            unsigned char *st = sh + (c & 1) * kStageBytes;
            const int L = rows_of(c);
            if (!wait(sm, &sm.dec_full[c & 1], (c >> 1) & 1)) break;
            if (!wait(sm, &sm.d1_full, c & 1)) break;
            tc_fence_after();
            const bool slow = d.slow;
#pragma unroll 1
            for (int jb = 0; jb <= w; ++jb) {
                uint32_t r[32];
                tmem_ld32(tq + kColX + 32 * jb, r);
                float e[32];
                if (!slow) {
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(&d.x[32 * jb + j]);
                        e[j] = f.x; e[j + 1] = f.y; e[j + 2] = f.z; e[j + 3] = f.w;
                    }
                } else {
                    const float hi = d.x[row], lo = d.y[row];
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        e[j] = expf((hi - d.x[32 * jb + j]) + (lo - d.y[32 * jb + j]));
                }
                tmem_wait_ld();
                uint32_t o[16];
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    float2 x = fmul2(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])),
                                     make_float2(e[j], e[j + 1]));
                    if (jb == w) {
                        x.x = lane >= j ? x.x : 0.f;
                        x.y = lane >= j + 1 ? x.y : 0.f;
                    }
                    o[j / 2] = pack_bf16(x.x, x.y);
                }
                tmem_st16(tq + kColP + 16 * jb, o);
            }
            if (slow) {                                // Q has been read by Q K^T
                const float a = expf(d.x[row] + d.y[row]);
#pragma unroll 1
                for (int i = 0; i < 16; ++i) {
                    uint4 *x = reinterpret_cast<uint4 *>(st + (i >> 3) * kHalf + sw128_off(row, 8 * (i & 7)));
                    uint4 y = *x;
                    uint32_t *yw = reinterpret_cast<uint32_t *>(&y);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = bf16x2_to_float2(yw[j]);
                        yw[j] = pack_bf16(f.x * a, f.y * a);
                    }
                    *x = y;
                }
            }
            if (row >= L) {                            // another sequence's values, never multiplied
                unsigned char *v = st + 2 * kTile;
#pragma unroll 1
                for (int i = 0; i < 16; ++i)
                    *reinterpret_cast<uint4 *>(v + (i >> 3) * kHalf + sw128_off(row, 8 * (i & 7))) =
                        make_uint4(0, 0, 0, 0);
            }
            if (slow || L < kTok) fence_proxy_async_smem();
            tmem_wait_st();
            tc_fence_before();
            arrive(&sm.p_ready);

            if (!wait(sm, &sm.o_full, c & 1)) break;
            tc_fence_after();
            const float a = slow ? p.scale : d.y[row];
            __nv_bfloat16 *og = p.o + ((size_t)(sg.t0 + (int64_t)c * kTok + row) * p.H + h) * kD;
#pragma unroll 1
            for (int jb = 0; jb < 4; ++jb) {
                uint32_t r[32];
                tmem_ld32(tq + kColX + 32 * jb, r);
                tmem_wait_ld();
                if (jb == 3) {
                    tc_fence_before();
                    arrive(&sm.x_free);
                    arrive(&sm.dec_free[c & 1]);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint4 y;
                    uint32_t *yw = reinterpret_cast<uint32_t *>(&y);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 x = fmul2(make_float2(__uint_as_float(r[8 * j + 2 * i]),
                                                           __uint_as_float(r[8 * j + 2 * i + 1])),
                                               make_float2(a, a));
                        yw[i] = pack_bf16(x.x, x.y);
                    }
                    if (L == kTok)
                        *reinterpret_cast<uint4 *>(st + (jb >> 1) * kHalf +
                                                   sw128_off(row, 32 * (jb & 1) + 8 * j)) = y;
                    else if (row < L)
                        *reinterpret_cast<uint4 *>(og + 32 * jb + 8 * j) = y;
                }
            }
            fence_proxy_async_smem();
            arrive(&sm.staged[c & 1]);
        }
    } else if (warp >= 8) {
        // ------------------------------------------ V' and S (thread = value channel)
        const int q = warp & 3, side = (warp - 8) >> 2;
        const int dv = 32 * q + lane, dk0 = 64 * side;
        const uint32_t tq = tm + ((uint32_t)(32 * q) << 16);
        float S[64];
        const float *from = nullptr;
        if (!kStates) {
            if (p.ws != nullptr && sg.count > 1) from = p.ws + ((size_t)u * p.H + h) * kD * kD;
            else if (p.h0 != nullptr) from = p.h0 + ((size_t)sg.n * p.H + h) * kD * kD;
        }
#pragma unroll
        for (int i = 0; i < 64; ++i) S[i] = from != nullptr ? from[(size_t)(dk0 + i) * kD + dv] : 0.f;

        // one half (64 tokens) of V' of chunk c; this warp: 32 channels x 32 tokens
        auto produce = [&](int c, int hf) -> bool {
            const Decay &d = sm.dec[c & 1];
            unsigned char *st = sh + (c & 1) * kStageBytes;
            const int L = rows_of(c);
            if (hf == 0) {
                if (!wait(sm, &sm.full[c & 1], (c >> 1) & 1)) return false;
                if (!wait(sm, &sm.dec_full[c & 1], (c >> 1) & 1)) return false;
                if (L < kTok) {                        // K rows of another sequence
                    const int r = 8 * (warp - 8) * 2 + (lane >> 1);
                    if (r >= L)
#pragma unroll 1
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<uint4 *>(st + kTile + (lane & 1) * kHalf + sw128_off(r, 8 * i)) =
                                make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
            }
            if (c > 0 && !wait(sm, &sm.v_free[hf], (c - 1) & 1)) return false;
            tc_fence_after();
            const int t0 = 64 * hf + 32 * side;        // tokens t0 .. t0 + 31
            float2 f[4];                               // factors of tokens t0 + 8 i + 2 (lane % 4)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = t0 + 8 * i + 2 * (lane & 3);
                if (!d.slow) {
                    const float2 x = *reinterpret_cast<const float2 *>(&d.x[t]);
                    f[i] = fmul2(x, make_float2(d.kv, d.kv));
                } else {
                    f[i].x = expf((d.end_hi - d.x[t]) + (d.end_lo - d.y[t]));
                    f[i].y = expf((d.end_hi - d.x[t + 1]) + (d.end_lo - d.y[t + 1]));
                }
            }
            const uint32_t vt = base + (c & 1) * kStageBytes + 2 * kTile;
            const uint32_t col = kColV + hf * kVBuf + 16 * side;
#pragma unroll
            for (int a = 0; a < 2; ++a) {              // 16 channels
                uint32_t hi[8], mid[8], lo[8];
#pragma unroll
                for (int b = 0; b < 2; ++b) {          // 16 tokens
                    // matrices: (tokens 0-7, channels 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15)
                    const int t = t0 + 16 * b + 8 * (lane >> 4) + (lane & 7);
                    const int ch = 32 * q + 16 * a + 8 * ((lane >> 3) & 1);
                    uint32_t x[4];
                    ldmatrix_trans(vt + (ch >> 6) * kHalf + sw128_off(t, ch & 63), x);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {      // register 4 b + j: column pair 2 b + j / 2
                        const int i = 2 * b + (j >> 1);
                        float2 v = fmul2(bf16x2_to_float2(x[j]), f[i]);
                        if (L < kTok) {                // 0 times whatever is there is not 0
                            const int tt = t0 + 8 * i + 2 * (lane & 3);
                            v.x = tt < L ? v.x : 0.f;
                            v.y = tt + 1 < L ? v.y : 0.f;
                        }
                        split3(v, hi[4 * b + j], mid[4 * b + j], lo[4 * b + j]);
                    }
                }
                const uint32_t at = tq + ((uint32_t)(16 * a) << 16) + col;
                tmem_st_frag(at, hi);
                tmem_st_frag(at + kVPart, mid);
                tmem_st_frag(at + 2 * kVPart, lo);
            }
            tmem_wait_st();
            tc_fence_before();
            arrive(&sm.v_full[hf]);
            return true;
        };
        // S'' of chunk c into shared memory: row = value channel, this warp's key half
        auto publish = [&](int c) {
            const float em = sm.dec[c & 1].em;
            unsigned char *t = sh + kOffS + side * kHalf;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint4 y;
                uint32_t *yw = reinterpret_cast<uint32_t *>(&y);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 x = fmul2(make_float2(S[8 * i + 2 * j], S[8 * i + 2 * j + 1]),
                                           make_float2(em, em));
                    yw[j] = pack_bf16(x.x, x.y);
                }
                *reinterpret_cast<uint4 *>(t + sw128_off(dv, 8 * i)) = y;
            }
            fence_proxy_async_smem();
            arrive(&sm.s_ready);
        };
        bool ok = true;
        if (chunks > 0) {
            ok = produce(0, 0);
            if (ok && !kStates) publish(0);
        }
        for (int c = 0; ok && c < chunks; ++c) {
            ok = produce(c, 1);
            if (ok && c + 1 < chunks) ok = produce(c + 1, 0);
            if (ok) ok = wait(sm, &sm.ds_full, c & 1);
            if (!ok) break;
            tc_fence_after();
            const float gamma = sm.dec[c & 1].gamma;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t r[32];
                tmem_ld32(tq + kColD + dk0 + 32 * i, r);
                tmem_wait_ld();
                if (i == 1) {
                    tc_fence_before();
                    arrive(&sm.ds_free);
                    arrive(&sm.dec_free[c & 1]);
                }
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float2 y = ffma2(make_float2(S[32 * i + j], S[32 * i + j + 1]), make_float2(gamma, gamma),
                                           make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])));
                    S[32 * i + j] = y.x;
                    S[32 * i + j + 1] = y.y;
                }
            }
            if (!kStates && c + 1 < chunks) {
                ok = wait(sm, &sm.o_full, c & 1);      // S'' has been read
                if (ok) publish(c + 1);
            }
        }
        float *to = nullptr;
        if (kStates) to = p.out + ((size_t)u * p.H + h) * kD * kD;
        else if (p.out != nullptr && sg.s == sg.count - 1) to = p.out + ((size_t)sg.n * p.H + h) * kD * kD;
        if (ok && to != nullptr)
#pragma unroll
            for (int i = 0; i < 64; ++i) to[(size_t)(dk0 + i) * kD + dv] = S[i];
    }

    // every product has been waited for by its reader; after a wait that ran out,
    // its issuer waits for what it has started
    __syncwarp();
    if (sm.abort && (warp == 1 || warp == 3)) {
        if (elect_one()) {
            tc_commit(&sm.drain[warp >> 1]);
            mbar_wait_drain(&sm.drain[warp >> 1], 0, kWaitLimit);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tm, 512);
}

// [T, heads, 128] bf16 as (128, heads, T) in boxes of 64 channels x 128 tokens.
inline bool make_map(CUtensorMap *map, const void *base, int heads, int64_t T) {
    EncodeTiledFn fn = encode_tiled_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {kD, (cuuint64_t)heads, (cuuint64_t)T};
    cuuint64_t strides[2] = {kD * 2, (cuuint64_t)heads * kD * 2};
    cuuint32_t box[3] = {64, 1, kTok};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc
}  // namespace lin
}  // namespace kda
