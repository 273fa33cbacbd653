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
// e^{+-60}, inside the range of bf16 and fp32 for q.k v and states below 1e11 (P' may
// be e^{60} of them) and down to 1e-11 (bf16 ends in steps of 2^-133, e^{-60} times
// 1e-14).  Within 40 the limits would be nine decades further out, and 96 heads x
// 8,192 tokens take 270 us instead of 246, as more heads leave the fast form.  A chunk
// that decays by more than e^{-120} takes a level for each 32 tokens, all of them
// powers of two: P'_ij gains the ratio of its row's level to its column's, and the rows
// of Q are scaled in place by the ratio of theirs to the first (exact).  Levels of
// neighbouring blocks may be 2^173 apart while the last token of one and the first
// of the next still see each other, and fp32 ends at 2^-149: what a ratio has below
// 2^-63 goes to P' behind e^{m - b_j}, so that no step leaves the range before P'
// itself does (which has decayed by e^{-27} at least then).  A row of Q has a ratio
// below 2^-126 only where S0 has decayed by e^{-27} too.  Where 32 tokens decay by
// more than e^{-120}, every row takes a level, m = 0 for S'', and P'_ij an exponential
// of its own.  All tokens alike, 96 heads x 8,192: 226 us in the first form (e^{-0.8} a
// token), 280 us in the second (e^{-3}), 394 us in the third (e^{-4}).
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
//
// Measured: 96 heads x 8,192 tokens 246 us (3.3 TB/s; 125 us of it are the bytes at
// the rate of a copy), 87,469 packed tokens of 32 heads 577 us behind 11 us of states
// and scan, 16 heads x 131,072 tokens 430 us behind 235 us of states.  Neither memory
// nor the tensor cores bound it (half and a quarter busy): a chunk takes 6 to 7
// thousand cycles of dependent steps, S to S'' to O and V' to S, and in this division
// of tensor memory Q K^T of the next chunk waits until O has been read.  An O with
// columns of its own (P' over what Q K^T leaves, V' in quarters) is not built; two
// terms of V' instead of three would make the room too, and leave the final state with
// an error of 2.7e-6.
#pragma once

#include "kda_linear_common.cuh"
#include "sm100_ptx.cuh"

namespace kda {
namespace lin {
namespace tc {

using namespace kda::sm100;

constexpr int kD = 128, kTok = 128, kThreads = 512;
constexpr uint32_t kTile = kTok * kD * 2;              // 32 KB; two halves of 64 channels
constexpr uint32_t kHalf = kTile / 2;

// Shared memory.  Outputs: two stages of Q, K, V, then S''.  States: three stages of
// K and V (with two, the tiles of a chunk were asked for 1,400 cycles before they
// were needed, less than a copy from L2 takes).
template <bool kStates>
struct Space {
    static constexpr int kStages = kStates ? 3 : 2;
    static constexpr uint32_t kStage = (kStates ? 2 : 3) * kTile;
    static constexpr uint32_t kK = kStates ? 0 : kTile, kV = kK + kTile;   // in a stage; Q at 0
    static constexpr uint32_t kS = kStages * kStage;
    static constexpr uint32_t kSmall = kS + (kStates ? 0 : kTile);
};

// Tensor-memory columns.
constexpr uint32_t kColX = 0, kColP = 128, kColD = 192, kColV = 320, kVBuf = 96, kVPart = 32;

constexpr float kRange = 60.f;                         // |b - m| of the fast form
constexpr unsigned long long kWaitLimit = 4000000000ull;   // about 2 s of SM clock

// How the decay of a chunk is split into factors (b, m of the comment above).
enum : int { kOneLevel = 0, kFourLevels = 1, kDirect = 2 };

struct __align__(16) Decay {
    float x[kTok], y[kTok];    // e^{m - b}, r;  direct: b as a sum of two floats
    float kv[4];               // e^{b_C - m} for the m of 32 tokens
    int level[4];              // m = level ln 2
    float em;                  // e^m of the first (direct: 1)
    float gamma;               // e^{b_C}
    float end_hi, end_lo;      // direct: b_C
    int mode;
};

template <int kStages>
struct Small {
    Decay dec[kStages];
    uint64_t full[kStages], dec_free[kStages];
    uint64_t staged[kStages], k_free[kStages];
    uint64_t d1_full, p_ready, o_full, x_free;
    uint64_t v_full[2], v_free, ds_full, ds_free, cleared;
    uint64_t drain[2];
    uint32_t tmem;
    volatile int abort;
};

template <bool kStates>
constexpr uint32_t smem_bytes() {
    return Space<kStates>::kSmall + (uint32_t)sizeof(Small<Space<kStates>::kStages>);
}
static_assert(smem_bytes<false>() <= 232448 && smem_bytes<true>() <= 232448, "shared memory");

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// A wait that every lane polls (each poll may suspend the warp for up to 10 us);
// false once another role gave up, or after kPolls polls: 2 s at most, and 4 ms
// at least where a poll returns at once.  The loop is kept short: sixteen warps
// in six roles share the instruction caches.
constexpr int kPolls = 1 << 18;
template <typename S>
__device__ __forceinline__ bool wait(S &sm, uint64_t *bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
#pragma unroll 1
    for (int n = 0; n < kPolls; ++n) {
        if (__all_sync(0xffffffffu, mbar_try_wait_hint(bar, parity, 10000))) return true;
        if (sm.abort) return false;
    }
    raise_error(kErrTimeout);
    sm.abort = 1;
    return false;
}

// One arrival of a warp, after all of its lanes.
__device__ __forceinline__ void arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// tcgen05.st 16 lanes x 128 bits, twice: 8 columns.  Register 2 c + r holds row
// lane / 4 + 8 r, column 4 c + lane % 4: the fragments of ldmatrix.
__device__ __forceinline__ void tmem_st_frag(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}

// level ln 2, with ln 2 split in two parts (Cody and Waite): the first has 10 bits,
// and what its product with a large level does not hold is kept too.
__device__ __forceinline__ Sum2 level_sum(int level) {
    const float l = (float)level, hi = l * 0.693359375f;
    return add2({hi, fmaf(l, 0.693359375f, -hi)}, {l * -2.12194440054690583e-4f, 0.f});
}

// Direct form: every row has a level of its own.
__device__ __forceinline__ int row_level(const Decay &d, int row) {
    const float l = rintf(d.x[row] * kLog2e);
    return l < -4e6f ? -4000000 : (int)l;
}
__device__ __noinline__ float direct_row_factor(const Decay &d, int row, float scale) {
    return scale * exp_sum(add2({d.x[row], d.y[row]}, minus(level_sum(row_level(d, row)))));
}

// One 32 x 32 block of P' in the direct form, an exponential for every element.
__device__ __noinline__ void direct_block(const Decay &d, uint32_t from, uint32_t to, int row, int j0) {
    const Sum2 m = level_sum(row_level(d, row));
#pragma unroll 1
    for (int c = 0; c < 32; c += 8, from += 8, to += 4) {
        uint32_t r[8], o[4];
        prefill::tmem_ld8(from, r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = j0 + c + i;
            const float x = __uint_as_float(r[i]) * __expf((m.hi - d.x[j]) + (m.lo - d.y[j]));
            r[i] = __float_as_uint(row >= j ? x : 0.f);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = pack_bf16(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(to), "r"(o[0]),
                     "r"(o[1]), "r"(o[2]), "r"(o[3])
                     : "memory");
    }
}

// 32 elements of P' times 2^e
__device__ __forceinline__ void times_pow2(uint32_t (&o)[16], int e) {
    const __nv_bfloat162 f = __float2bfloat162_rn(exp2f((float)e));
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        __nv_bfloat162 *x = reinterpret_cast<__nv_bfloat162 *>(&o[i]);
        *x = __hmul2(*x, f);
    }
}

// Row `row` of a tile of 128 channels times a, in place.
__device__ __noinline__ void scale_row(unsigned char *tile, int row, float a) {
    const __nv_bfloat162 f = __float2bfloat162_rn(a);
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
        uint4 *x = reinterpret_cast<uint4 *>(tile + (i >> 3) * kHalf + sw128_off(row, 8 * (i & 7)));
        uint4 y = *x;
        __nv_bfloat162 *yw = reinterpret_cast<__nv_bfloat162 *>(&y);
#pragma unroll
        for (int j = 0; j < 4; ++j) yw[j] = __hmul2(yw[j], f);
        *x = y;
    }
}

// Rows L .. of K and V (the tile behind it) are another sequence's, or nobody's:
// zero times a NaN there would still be one.  By the 8 warps of S, who wait for one
// another (`cleared`), read V next and publish S'' (which every product of V waits
// for) after it.
__device__ __noinline__ void clear_tail(unsigned char *k, int L) {
    const int t = threadIdx.x - 256, row = t >> 1;
    if (row >= L)
        for (int i = 0; i < 8; ++i) {
            uint4 *x = reinterpret_cast<uint4 *>(k + (t & 1) * kHalf + sw128_off(row, 8 * i));
            x[0] = make_uint4(0, 0, 0, 0);
            x[kTile / sizeof(uint4)] = make_uint4(0, 0, 0, 0);
        }
    fence_proxy_async_smem();
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

// Decay factors of chunk tokens 4 lane .. 4 lane + 3 (warp 2), formed before the
// slot they go to is free.
struct LaneDecay {
    float x[4], y[4], kv, em, gamma;
    Sum2 end;
    int level, mode;
};

// kReverse: x is r, and kv the level's own factor: x kv = scale e^{b_i}.
template <bool kReverse>
__device__ __forceinline__ void decay_factors(LaneDecay &d, const float (&g)[4], float scale) {
    const int lane = threadIdx.x & 31;
    Sum2 b[4];
    b[0] = {g[0], 0.f};
#pragma unroll
    for (int i = 1; i < 4; ++i) b[i] = add2(b[i - 1], {g[i], 0.f});
    Sum2 run = b[3], before = {0.f, 0.f};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sum2 up = {__shfl_up_sync(0xffffffffu, run.hi, o), __shfl_up_sync(0xffffffffu, run.lo, o)};
        if (lane >= o) {
            run = add2(up, run);
            before = add2(up, before);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = add2(before, b[i]);
    d.end = {__shfl_sync(0xffffffffu, b[3].hi, 31), __shfl_sync(0xffffffffu, b[3].lo, 31)};
    // extremes of 32 tokens (8 lanes), then of the chunk
    float top = fmaxf(fmaxf(b[0].hi, b[1].hi), fmaxf(b[2].hi, b[3].hi));
    float low = fminf(fminf(b[0].hi, b[1].hi), fminf(b[2].hi, b[3].hi));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
    }
    const bool near32 = __all_sync(0xffffffffu, top - low <= 2.f * kRange);      // NaN: no
    float top_c = top, low_c = low;
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
        top_c = fmaxf(top_c, __shfl_xor_sync(0xffffffffu, top_c, o));
        low_c = fminf(low_c, __shfl_xor_sync(0xffffffffu, low_c, o));
    }
    const bool near_c = top_c - low_c <= 2.f * kRange;
    d.mode = near_c ? kOneLevel : near32 ? kFourLevels : kDirect;
    if (near_c) {
        top = top_c;
        low = low_c;
    }
    const bool direct = d.mode == kDirect;
    d.level = direct ? 0 : __float2int_rn(0.5f * (top + low) * kLog2e);
    const Sum2 m = level_sum(d.level);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const Sum2 t = add2(m, minus(b[i]));
        d.x[i] = direct ? b[i].hi : kReverse ? scale * exp_sum(minus(t)) : exp_sum(t);
        d.y[i] = direct ? b[i].lo : scale * exp_sum(minus(t));
    }
    d.kv = direct ? 1.f : kReverse ? exp_sum(m) : exp_sum(add2(d.end, minus(m)));
    d.em = direct ? 1.f : exp_sum(m);
    d.gamma = exp_sum(d.end);
}

__device__ __forceinline__ void store_decay(Decay &o, const LaneDecay &d) {
    const int lane = threadIdx.x & 31;
    *reinterpret_cast<float4 *>(&o.x[4 * lane]) = make_float4(d.x[0], d.x[1], d.x[2], d.x[3]);
    *reinterpret_cast<float4 *>(&o.y[4 * lane]) = make_float4(d.y[0], d.y[1], d.y[2], d.y[3]);
    if ((lane & 7) == 0) {
        o.kv[lane >> 3] = d.kv;
        o.level[lane >> 3] = d.level;
    }
    if (lane == 0) {
        o.em = d.em;
        o.gamma = d.gamma;
        o.end_hi = d.end.hi;
        o.end_lo = d.end.lo;
        o.mode = d.mode;
    }
}
// kOutputs: o and the final state.  kStates: only S is wanted, from zero; R and the
// decay of the segment go out.  kReverse: the same for the gradient of the state,
// R = sum_i scale e^{b_i} q_i dO_i^T, chunks last to first (map_k is that of q,
// map_v that of dO).
enum : int { kOutputs = 0, kForwardStates = 1, kReverseStates = 2 };

template <int kMode>
__global__ void __launch_bounds__(kThreads, 1)
linear_sm100_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o,
                    const Params p) {
    constexpr bool kStates = kMode != kOutputs, kReverse = kMode == kReverseStates;
    extern __shared__ __align__(1024) unsigned char sh[];
    using Sp = Space<kStates>;
    constexpr int kStages = Sp::kStages;
    Small<kStages> &sm = *reinterpret_cast<Small<kStages> *>(sh + Sp::kSmall);
    auto slot = [](int c) { return kStages == 2 ? c & 1 : c % kStages; };
    auto phase = [](int c) { return kStages == 2 ? (c >> 1) & 1 : (c / kStages) & 1; };
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int h = blockIdx.x % p.H;
    const int i = blockIdx.x / p.H;
    if (!kStates && blockIdx.x == 0) check_seqlens(p.m);
    Segment sg;
    if (kStates) {                                     // all of one length, but for sequence ends
        if (!find_body(p.m, i, kReverse, sg)) return;
    } else {
        if (!find_segment(p.m, ranked_unit<kThreads>(p.m, i, reinterpret_cast<int *>(sh)), sg)) return;
    }
    const int len = (int)(sg.t1 - sg.t0);
    const int chunks = (len + kTok - 1) / kTok;
    const int hk = h / (p.H / p.Hk);

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sm.full[i], 2);                 // the tiles, and the decay factors
            mbar_init(&sm.dec_free[i], kStates ? 8 : 12);
            mbar_init(&sm.staged[i], 4);
            mbar_init(&sm.k_free[i], 1);
            mbar_init(&sm.v_full[i], 8);
        }
        mbar_init(&sm.v_free, 1);
        mbar_init(&sm.d1_full, 1);
        mbar_init(&sm.p_ready, 12);
        mbar_init(&sm.o_full, 1);
        mbar_init(&sm.x_free, 4);
        mbar_init(&sm.ds_full, 1);
        mbar_init(&sm.ds_free, 8);
        mbar_init(&sm.cleared, 8);
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
    const int t_first = (int)sg.t0;                    // tokens stay below 2^31
    // first token of the c-th chunk of the walk, counted from the segment's
    auto first = [&](int c) { return (kReverse ? chunks - 1 - c : c) * kTok; };

    if (warp == 0) {
        // ------------------------------------------------------------ tiles
        auto load = [&](int c) {
            if (elect_one()) {
                unsigned char *st = sh + slot(c) * Sp::kStage;
                uint64_t *bar = &sm.full[slot(c)];
                const int t = t_first + first(c);
                mbar_expect_tx(bar, kStates ? 2 * kTile : 3 * kTile);
                tma_load_3d(st + Sp::kK, &map_k, bar, 0, hk, t);
                tma_load_3d(st + Sp::kK + kHalf, &map_k, bar, 64, hk, t);
                if (!kStates) {
                    tma_load_3d(st, &map_q, bar, 0, hk, t);
                    tma_load_3d(st + kHalf, &map_q, bar, 64, hk, t);
                }
                tma_load_3d(st + Sp::kV, &map_v, bar, 0, h, t);
                tma_load_3d(st + Sp::kV + kHalf, &map_v, bar, 64, h, t);
            }
            __syncwarp();
        };
        // the tiles of the chunk after are brought to L2, so that a stage that becomes
        // free is filled from there
        auto prefetch = [&](int c) {
            if (c < chunks && elect_one()) {
                const int t = t_first + first(c);
#pragma unroll
                for (int x = 0; x < kD; x += 64) {
                    tma_prefetch_3d(&map_k, x, hk, t);
                    if (!kStates) tma_prefetch_3d(&map_q, x, hk, t);
                    tma_prefetch_3d(&map_v, x, h, t);
                }
            }
            __syncwarp();
        };
        for (int c = 0; c < kStages && c < chunks; ++c) load(c);
        prefetch(kStages);
        int c = 0;
        for (; c < chunks; ++c) {
            if (!kStates) {
                if (!wait(sm, &sm.staged[slot(c)], phase(c))) break;
                if (len - c * kTok >= kTok) {
                    if (elect_one()) {
                        const unsigned char *st = sh + slot(c) * Sp::kStage;
                        const int t = t_first + first(c);
                        tma_store_3d(&map_o, st, 0, h, t);
                        tma_store_3d(&map_o, st + kHalf, 64, h, t);
                        bulk_commit_group();
                        bulk_wait_group_read<0>();
                    }
                    __syncwarp();
                }
            }
            if (!wait(sm, &sm.k_free[slot(c)], phase(c))) break;
            if (c + kStages < chunks) load(c + kStages);
            prefetch(c + kStages + 1);
        }
        if (c < chunks) {                              // gave up: let the copies in flight land
            const int issued = c + kStages < chunks ? c + kStages : chunks;
            for (int i = c; i < issued; ++i) mbar_wait_drain(&sm.full[slot(i)], phase(i), kWaitLimit);
        }
        if (elect_one()) bulk_wait_group<0>();
        __syncwarp();
    } else if (warp == 1 && !kStates) {
        // ------------------------------------------- Q K^T, then P' V + Q S''
        constexpr uint32_t id_kk = idesc_bf16(128, 128, false, false);
        constexpr uint32_t id_kn = idesc_bf16(128, 128, false, true);
        const uint64_t ds = sdesc(base + Sp::kS, kHalf, 1024, kLayoutSW128);
        int c = 0;
        for (; c < chunks; ++c) {
            const uint32_t st = base + slot(c) * Sp::kStage;
            const uint64_t dq = sdesc(st, kHalf, 1024, kLayoutSW128);
            const uint64_t dk = sdesc(st + Sp::kK, kHalf, 1024, kLayoutSW128);
            const uint64_t dv = sdesc(st + Sp::kV, kHalf, 1024, kLayoutSW128);
            if (!wait(sm, &sm.full[slot(c)], phase(c))) break;
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
            if (!wait(sm, &sm.p_ready, c & 1)) break;  // P' and S''
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
                const int t = first(c) + 4 * lane + i;
                x[i] = t < len ? load_decay(p.g, p.per_token, sg.t0 + t, h, p.H) : 0.f;
            }
        };
        Sum2 sum = {0.f, 0.f};
        if (chunks > 0) fetch(0, next);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) g[i] = next[i];
            if (c + 1 < chunks) fetch(c + 1, next);
            LaneDecay d;
            decay_factors<kReverse>(d, g, p.scale);
            if (kStates) sum = add2(sum, d.end);
            if (c >= kStages && !wait(sm, &sm.dec_free[slot(c)], phase(c - kStages))) break;
            store_decay(sm.dec[slot(c)], d);
            arrive(&sm.full[slot(c)]);
        }
        if (kStates && lane == 0) p.total[(size_t)sg.slot * p.H + h] = exp_sum(sum);
    } else if (warp == 3) {
        // ------------------------------------------------------------ V'^T K
        constexpr uint32_t id = idesc_bf16(128, 128, false, true);
        for (int c = 0; c < chunks; ++c) {
            const uint64_t dk = sdesc(base + slot(c) * Sp::kStage + Sp::kK, kHalf, 1024, kLayoutSW128);
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
                    if (hf == 0) {
                        tc_commit(&sm.v_free);
                    } else {
                        tc_commit(&sm.ds_full);
                        tc_commit(&sm.k_free[slot(c)]);
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
        uint32_t below[16];                            // of a diagonal block: row >= column
#pragma unroll
        for (int i = 0; i < 16; ++i)
            below[i] = (lane >= 2 * i ? 0xffffu : 0u) | (lane >= 2 * i + 1 ? 0xffff0000u : 0u);
        for (int c = 0; c < chunks; ++c) {
            const Decay &d = sm.dec[slot(c)];
            unsigned char *st = sh + slot(c) * Sp::kStage;
            const bool whole_chunk = len - c * kTok >= kTok;
            if (!wait(sm, &sm.d1_full, c & 1)) break;
            tc_fence_after();
            const int mode = d.mode;
            const int level = d.level[w];
#pragma unroll 1
            for (int jb = 0; jb <= w; ++jb) {
                if (mode == kDirect) {
                    direct_block(d, tq + kColX + 32 * jb, tq + kColP + 16 * jb, row, 32 * jb);
                    continue;
                }
                uint32_t r[32], o[16];
                tmem_ld32(tq + kColX + 32 * jb, r);
                const uint32_t whole = jb < w ? 0xffffffffu : 0u;
                const int dl = level - d.level[jb], near = max(dl, -63);   // 0 on one level
                const float ratio = exp2f((float)near);
                tmem_wait_ld();
                if (mode == kFourLevels)
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float2 x = fmul2(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])),
                                               make_float2(ratio, ratio));
                        r[j] = __float_as_uint(x.x);
                        r[j + 1] = __float_as_uint(x.y);
                    }
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(&d.x[32 * jb + j]);
                    const float2 x = fmul2(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])),
                                           make_float2(f.x, f.y));
                    const float2 y = fmul2(make_float2(__uint_as_float(r[j + 2]), __uint_as_float(r[j + 3])),
                                           make_float2(f.z, f.w));
                    o[j / 2] = pack_bf16(x.x, x.y) & (below[j / 2] | whole);
                    o[j / 2 + 1] = pack_bf16(y.x, y.y) & (below[j / 2 + 1] | whole);
                }
                if (dl < near) times_pow2(o, dl - near);
                tmem_st16(tq + kColP + 16 * jb, o);
            }
            // Q has been read by Q K^T
            if (mode == kDirect) scale_row(st, row, exp2f((float)row_level(d, row)));
            else if (level != d.level[0]) scale_row(st, row, exp2f((float)(level - d.level[0])));
            if (mode != kOneLevel) fence_proxy_async_smem();
            tmem_wait_st();
            tc_fence_before();
            arrive(&sm.p_ready);

            if (!wait(sm, &sm.o_full, c & 1)) break;
            tc_fence_after();
            const float a = mode == kDirect ? direct_row_factor(d, row, p.scale) : d.y[row];
            __nv_bfloat16 *og = p.o + ((size_t)(sg.t0 + c * kTok + row) * p.H + h) * kD;
#pragma unroll 1
            for (int jb = 0; jb < 2; ++jb) {           // 64 columns at once: two loads in flight
                uint32_t r[2][32];
                tmem_ld32(tq + kColX + 64 * jb, r[0]);
                tmem_ld32(tq + kColX + 64 * jb + 32, r[1]);
                tmem_wait_ld();
                if (jb == 1) {
                    tc_fence_before();
                    arrive(&sm.x_free);
                    arrive(&sm.dec_free[slot(c)]);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint4 y;
                    uint32_t *yw = reinterpret_cast<uint32_t *>(&y);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 x = fmul2(make_float2(__uint_as_float(r[j >> 2][8 * (j & 3) + 2 * i]),
                                                           __uint_as_float(r[j >> 2][8 * (j & 3) + 2 * i + 1])),
                                               make_float2(a, a));
                        yw[i] = pack_bf16(x.x, x.y);
                    }
                    if (whole_chunk)
                        *reinterpret_cast<uint4 *>(st + jb * kHalf + sw128_off(row, 8 * j)) = y;
                    else if (c * kTok + row < len)
                        *reinterpret_cast<uint4 *>(og + 64 * jb + 8 * j) = y;
                }
            }
            fence_proxy_async_smem();
            arrive(&sm.staged[slot(c)]);
        }
    } else if (warp >= 8) {
        // ------------------------------------------ V' and S (thread = value channel)
        const int q = warp & 3, side = (warp - 8) >> 2;
        const int dv = 32 * q + lane, dk0 = 64 * side;
        const uint32_t tq = tm + ((uint32_t)(32 * q) << 16);
        float S[64];
        const float *from = nullptr;
        if (!kStates) {
            if (p.ws != nullptr && sg.count > 1) from = p.ws + ((size_t)sg.slot * p.H + h) * kD * kD;
            else if (p.h0 != nullptr) from = p.h0 + ((size_t)sg.n * p.H + h) * kD * kD;
        }
#pragma unroll
        for (int i = 0; i < 64; ++i) S[i] = from != nullptr ? from[(size_t)(dk0 + i) * kD + dv] : 0.f;

        // one half (64 tokens) of V' of chunk c; this warp: 32 channels x 32 tokens
        auto produce = [&](int c, int hf) -> bool {
            const Decay &d = sm.dec[slot(c)];
            unsigned char *st = sh + slot(c) * Sp::kStage;
            if (hf == 0) {
                if (!wait(sm, &sm.full[slot(c)], phase(c))) return false;
                if (len - first(c) < kTok) {           // one chunk of a segment
                    clear_tail(st + Sp::kK, len - first(c));
                    arrive(&sm.cleared);
                    if (!wait(sm, &sm.cleared, 0)) return false;
                }
            }
            // the second half's buffer was free once the last chunk's V'^T K was done
            if (hf == 0 && c > 0 && !wait(sm, &sm.v_free, (c - 1) & 1)) return false;
            tc_fence_after();
            const int t0 = 64 * hf + 32 * side;        // tokens t0 .. t0 + 31
            const uint32_t vt = base + slot(c) * Sp::kStage + Sp::kV;
            const uint32_t col = kColV + hf * kVBuf + 16 * side;
            // 16 tokens a step, both halves of the channels.  Matrices: (tokens 0-7,
            // channels 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15)
            const int ch = 32 * q + 8 * ((lane >> 3) & 1);
            const float kv = d.kv[t0 >> 5];
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                const int tr = t0 + 16 * b + 8 * (lane >> 4) + (lane & 7), tt = t0 + 16 * b + 2 * (lane & 3);
                uint32_t x[2][4];
#pragma unroll
                for (int a = 0; a < 2; ++a)
                    ldmatrix_trans(vt + (ch >> 6) * kHalf + sw128_off(tr, (ch + 16 * a) & 63), x[a]);
                float2 f[2];                           // factors of tokens tt, tt + 1 and tt + 8, tt + 9
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int t = tt + 8 * i;
                    const float2 dx = *reinterpret_cast<const float2 *>(&d.x[t]);
                    if (d.mode != kDirect) {
                        f[i] = fmul2(dx, make_float2(kv, kv));
                    } else {
                        f[i].x = kReverse ? p.scale * __expf(dx.x + d.y[t])
                                          : __expf((d.end_hi - dx.x) + (d.end_lo - d.y[t]));
                        f[i].y = kReverse ? p.scale * __expf(dx.y + d.y[t + 1])
                                          : __expf((d.end_hi - dx.y) + (d.end_lo - d.y[t + 1]));
                    }
                }
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    uint32_t hi[4], mid[4], lo[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 v = fmul2(bf16x2_to_float2(x[a][j]), f[j >> 1]);
                        split3(v, hi[j], mid[j], lo[j]);
                    }
                    const uint32_t at = tq + ((uint32_t)(16 * a) << 16) + col + 8 * b;
                    tmem_st_frag(at, hi);
                    tmem_st_frag(at + kVPart, mid);
                    tmem_st_frag(at + 2 * kVPart, lo);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            arrive(&sm.v_full[hf]);
            return true;
        };
        // S'' of chunk c into shared memory: row = value channel, this warp's key half
        auto publish = [&](int c) {
            const float em = sm.dec[slot(c)].em;
            unsigned char *t = sh + Sp::kS + side * kHalf;
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
            arrive(&sm.p_ready);
        };
        bool ok = true;
#pragma unroll 1
        for (int i = 0; ok && i <= 2 * chunks; ++i) {
            if (i < 2 * chunks) ok = produce(i >> 1, i & 1);
            if (!ok || (i & 1)) continue;
            const int c = (i >> 1) - 1;                // the chunk whose V'^T K is due
            if (c >= 0) {
                ok = wait(sm, &sm.ds_full, c & 1);
                if (!ok) continue;
                tc_fence_after();
                const float gamma = sm.dec[slot(c)].gamma;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    uint32_t r[32];
                    tmem_ld32(tq + kColD + dk0 + 32 * b, r);
                    tmem_wait_ld();
                    if (b == 1) {
                        tc_fence_before();
                        arrive(&sm.ds_free);
                        arrive(&sm.dec_free[slot(c)]);
                    }
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float2 y = ffma2(make_float2(S[32 * b + j], S[32 * b + j + 1]),
                                               make_float2(gamma, gamma),
                                               make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])));
                        S[32 * b + j] = y.x;
                        S[32 * b + j + 1] = y.y;
                    }
                }
                if (!kStates && c + 1 < chunks) ok = wait(sm, &sm.o_full, c & 1);   // S'' has been read
            }
            if (!kStates && ok && c + 1 < chunks) publish(c + 1);
        }
        float *to = nullptr;
        if (kStates) to = p.out + ((size_t)sg.slot * p.H + h) * kD * kD;
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
