// kda_linear_api.cuh -- entry points of the decayed linear attention: argument
// checks, the split into segments, workspaces, launches.  Included by kda_api.cu.
#pragma once

namespace kda {
namespace lin {

inline size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

struct Plan {
    SegMap map;
    bool split;
    size_t state_bytes, total_bytes;                   // of one direction
    size_t factor_bytes;                               // warp-level path: decay factors of the chunks
    int bodies;                                        // T_tot / L: segments whose states are formed
};

inline Plan make_plan(const int32_t *cu, int32_t N, int64_t T_tot, int32_t H, int32_t d, int64_t L,
                      bool factors) {
    Plan p;
    p.map.cu = cu;
    p.map.N = N;
    p.map.T_tot = T_tot;
    p.map.L = L;
    p.map.units = (int)(T_tot / L + N);
    p.map.per = (int)(T_tot / N);
    p.split = L != kNoSplit;
    p.bodies = p.split ? (int)(T_tot / L) : 0;
    const size_t n = (size_t)state_slots(T_tot, L, N) * H;
    p.state_bytes = p.split ? align256(n * d * d * sizeof(float)) : 0;
    p.total_bytes = p.split ? align256(n * sizeof(float)) : 0;
    p.factor_bytes = factors ? align256((size_t)(T_tot / mm::kTok + N) * H * sizeof(mm::Factors)) : 0;
    return p;
}

// bf16 at d = 128 runs on tcgen05 (prefill), other bf16 on warp-level matrix
// instructions, fp32 on CUDA cores.
inline bool tensor_path(int32_t d, kda_dtype dt) { return d == 128 && dt == KDA_BF16; }

// The scan reads and writes a state of every segment, at about 3.5 TB/s.
inline double scan_us(int32_t d) { return 8.0 * d * d / 3.5e6; }

inline Costs fwd_costs(int32_t d, kda_dtype dt) {
    if (tensor_path(d, dt)) return {tc::kTok, 148, 3.6, 2.1, scan_us(d)};
    if (dt == KDA_BF16) return {mm::kTok, 148 * (d == 64 ? 3 : 6), d == 64 ? 2.5 : 1.5, d == 64 ? 1.2 : 0.8, scan_us(d)};
    return {kC, 148 * (d >= 64 ? 2 : 4), 4.0, 1.5, scan_us(d)};
}

inline Costs bwd_costs(int32_t d, kda_dtype dt) {
    if (dt == KDA_BF16)
        return {mm::kTok, 148 * (d == 128 ? 1 : d == 64 ? 2 : 3), d == 128 ? 20.0 : 6.0, 2.4, 2 * scan_us(d)};
    return {kC, 148 * (d == 128 ? 1 : 2), d == 128 ? 16.0 : 8.0, d == 128 ? 6.0 : 3.0, 2 * scan_us(d)};
}

// The workspace query does not know whether cu_seqlens is given: with several
// sequences it takes the larger of the two plans.
inline int64_t fwd_length(int32_t N, bool equal, int64_t T_tot, int32_t H, int32_t d, kda_dtype dt) {
    return segment_length(N, equal, T_tot, (int64_t)H * (dt == KDA_FP32 && d == 128 ? 2 : 1), fwd_costs(d, dt));
}

inline size_t fwd_bytes(const Plan &p) { return p.state_bytes + p.total_bytes + p.factor_bytes; }

inline bool fwd_factors(int32_t d, kda_dtype dt) { return dt == KDA_BF16 && !tensor_path(d, dt); }

inline int64_t bwd_length(int32_t N, bool equal, int64_t T_tot, int32_t H, int32_t d, kda_dtype dt) {
    return segment_length(N, equal, T_tot, H, bwd_costs(d, dt));
}

struct BwdSizes {
    size_t states, totals, terms, anchors, sums, parts, all;
};

inline BwdSizes bwd_sizes(const Plan &p, int64_t T_tot, int32_t Hk, int32_t H, int32_t d) {
    BwdSizes s;
    const size_t n = (size_t)p.map.units * H;
    s.states = p.state_bytes;
    s.totals = p.total_bytes;
    s.terms = align256((size_t)T_tot * H * sizeof(float));
    s.anchors = align256(n * sizeof(double));
    s.sums = align256(n * sizeof(double));
    s.parts = Hk != H ? align256((size_t)T_tot * H * d * sizeof(float)) : 0;
    s.all = 2 * s.states + 2 * s.totals + s.terms + s.anchors + s.sums + s.parts + p.factor_bytes;
    return s;
}

inline bool supported_d(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

// Sizes that the prefill and its gradient take.
inline kda_status check_sizes(int32_t N, int64_t T_tot, int32_t Hk, int32_t H, int32_t d, kda_dtype dt) {
    if (N < 0 || T_tot < 0 || H <= 0 || Hk <= 0 || H > 65535 || H % Hk != 0)
        return KDA_ERR_INVALID_ARGUMENT;
    if (dt != KDA_BF16 && dt != KDA_FP32) return KDA_ERR_UNSUPPORTED;
    if (!supported_d(d)) return KDA_ERR_UNSUPPORTED;
    if (T_tot > kMaxTokensSm100) return KDA_ERR_UNSUPPORTED;
    if ((int64_t)N * H > 0x7fffffff || T_tot / 64 + N > 0x7fffffff) return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

// The rest of their checks; KDA_OK leaves `empty` true when there is nothing to do.
inline kda_status check_shapes(int32_t N, int64_t T_tot, int32_t Hk, int32_t H, int32_t d,
                               kda_dtype dt, const int32_t *cu, float scale, bool &empty) {
    empty = false;
    const kda_status st = check_sizes(N, T_tot, Hk, H, d, dt);
    if (st != KDA_OK) return st;
    if (!(scale - scale == 0.f)) return KDA_ERR_INVALID_ARGUMENT;       // inf or NaN
    if (N == 0) {
        empty = true;
        return T_tot == 0 ? KDA_OK : KDA_ERR_INVALID_ARGUMENT;
    }
    if (cu == nullptr && (T_tot % N) != 0) return KDA_ERR_INVALID_ARGUMENT;
    if (cu != nullptr && !aligned16(cu)) return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

inline bool all_given(const void *const *p, int n) {
    for (int i = 0; i < n; ++i)
        if (p[i] == nullptr || !aligned16(p[i])) return false;
    return true;
}

// Arrays that kernels read value by value (decays, positions, statistics) need
// no more than the alignment of a value: they are often rows of larger ones.
inline bool given4(const void *p) {
    return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0;
}

inline bool ok16(const void *p) { return p == nullptr || aligned16(p); }

template <typename K>
inline bool set_smem(K kern, size_t bytes) {
    if (bytes <= 40 * 1024) return true;               // 48 KB, static arrays included, need no asking
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) ==
           cudaSuccess;
}

inline kda_status launched() { return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

template <bool kReverse>
inline kda_status launch_scan(const Plan &p, int H, int d, const float *init, const float *total,
                              float *ws, cudaStream_t s) {
    const int dd = d * d;
    const int64_t z = scan_blocks(p.map);
    const dim3 grid((unsigned)((dd + 4 * kScanThreads - 1) / (4 * kScanThreads)), (unsigned)H,
                    (unsigned)(z < 65535 ? z : 65535));
    segment_scan_kernel<kReverse><<<grid, kScanThreads, 0, s>>>(p.map, H, dd, init, total, ws);
    return launched();
}

struct FwdArgs {
    const void *q, *k, *v;
    const float *g, *h0;
    int per_token;
    int32_t Hk, H;
    float scale;
    void *o;
    float *hT;
    unsigned char *ws;
};

template <int D>
kda_status fwd_simt(const Plan &p, const FwdArgs &a, cudaStream_t s) {
    float *states = nullptr, *total = nullptr;
    const dim3 grid((unsigned)p.map.units, (unsigned)a.H, (unsigned)(D / OutSmem<D>::kW));
    const float *q = (const float *)a.q, *k = (const float *)a.k, *v = (const float *)a.v;
    if (p.split) {
        states = reinterpret_cast<float *>(a.ws);
        total = reinterpret_cast<float *>(a.ws + p.state_bytes);
        auto kern = state_kernel<D, false>;
        const size_t smem = sizeof(StateSmem<D>);
        const dim3 bodies((unsigned)p.bodies, grid.y, grid.z);
        if (!set_smem(kern, smem)) return KDA_ERR_CUDA;
        kern<<<bodies, kThreads, smem, s>>>(k, v, a.g, a.per_token, p.map, a.Hk, a.H, 1.f, states, total);
        kda_status st = launched();
        if (st == KDA_OK) st = launch_scan<false>(p, a.H, D, a.h0, total, states, s);
        if (st != KDA_OK) return st;
    }
    auto kern = out_kernel<D>;
    const size_t smem = sizeof(OutSmem<D>);
    if (!set_smem(kern, smem)) return KDA_ERR_CUDA;
    kern<<<grid, kThreads, smem, s>>>(q, k, v, a.g, a.per_token, a.h0, p.map, a.Hk, a.H, a.scale, states,
                                      (float *)a.o, a.hT);
    return launched();
}

inline kda_status launch_factors(const Plan &p, const float *g, int per_token, int H, float scale,
                                 mm::Factors *out, cudaStream_t s) {
    SegMap c = p.map;
    c.L = mm::kTok;
    c.units = (int)(c.T_tot / mm::kTok + c.N);
    const int64_t blocks = ((int64_t)c.units * H + 7) / 8;
    mm::factor_kernel<<<(unsigned)blocks, 256, 0, s>>>(g, per_token, c, H, scale, out);
    return launched();
}

// bf16 below d = 128
template <int D>
kda_status fwd_mma(const Plan &p, const FwdArgs &a, cudaStream_t s) {
    float *states = nullptr, *total = nullptr;
    const unsigned blocks = (unsigned)((int64_t)p.map.units * a.H), threads = mm::Shape<D>::kThreads;
    const __nv_bfloat16 *q = (const __nv_bfloat16 *)a.q, *k = (const __nv_bfloat16 *)a.k,
                        *v = (const __nv_bfloat16 *)a.v;
    mm::Factors *f = reinterpret_cast<mm::Factors *>(a.ws + p.state_bytes + p.total_bytes);
    kda_status st = launch_factors(p, a.g, a.per_token, a.H, a.scale, f, s);
    if (st != KDA_OK) return st;
    if (p.split) {
        states = reinterpret_cast<float *>(a.ws);
        total = reinterpret_cast<float *>(a.ws + p.state_bytes);
        auto kern = mm::state_kernel<D, false>;
        const size_t smem = sizeof(mm::StateSmem<D>);
        if (!set_smem(kern, smem)) return KDA_ERR_CUDA;
        kern<<<(unsigned)((int64_t)p.bodies * a.H), threads, smem, s>>>(k, v, f, p.map, a.Hk, a.H, states, total);
        st = launched();
        if (st == KDA_OK) st = launch_scan<false>(p, a.H, D, a.h0, total, states, s);
        if (st != KDA_OK) return st;
    }
    auto kern = mm::out_kernel<D>;
    const size_t smem = sizeof(mm::OutSmem<D>);
    if (!set_smem(kern, smem)) return KDA_ERR_CUDA;
    kern<<<blocks, threads, smem, s>>>(q, k, v, f, a.h0, p.map, a.Hk, a.H, a.scale, states,
                                       (__nv_bfloat16 *)a.o, a.hT);
    return launched();
}

inline tc::Params tensor_params(const Plan &p, const float *g, int per_token, int32_t Hk, int32_t H, float scale) {
    tc::Params t = {};
    t.g = g;
    t.m = p.map;
    t.per_token = per_token;
    t.Hk = Hk;
    t.H = H;
    t.scale = scale;
    return t;
}

// The segments' states on tcgen05: R and decays of `x` (Hk heads) and `y` (H heads).
template <int kMode>
kda_status tensor_states(const Plan &p, const CUtensorMap &x, const CUtensorMap &y, tc::Params t, float *out,
                         float *total, cudaStream_t s) {
    constexpr size_t smem = tc::smem_bytes<true>();
    auto kern = tc::linear_sm100_kernel<kMode>;
    t.out = out;
    t.total = total;
    if (!set_smem(kern, smem)) return KDA_ERR_CUDA;
    kern<<<(unsigned)((int64_t)p.bodies * t.H), tc::kThreads, smem, s>>>(x, x, y, y, t);
    return launched();
}

// [T, heads, 128] maps; with no tokens no tile is copied, and the maps describe
// a row of hT, which the caller has then given.
inline kda_status fwd_tensor(const Plan &p, const FwdArgs &a, cudaStream_t s) {
    const int64_t T = p.map.T_tot;
    CUtensorMap mq, mk, mv, mo;
    auto base = [&](const void *x) { return T > 0 ? x : (const void *)a.hT; };
    const int64_t rows = T > 0 ? T : 1;
    if (!tc::make_map(&mq, base(a.q), a.Hk, rows) || !tc::make_map(&mk, base(a.k), a.Hk, rows) ||
        !tc::make_map(&mv, base(a.v), a.H, rows) || !tc::make_map(&mo, base(a.o), a.H, rows))
        return KDA_ERR_CUDA;
    tc::Params t = tensor_params(p, a.g, a.per_token, a.Hk, a.H, a.scale);
    t.h0 = a.h0;
    t.out = a.hT;
    t.o = (__nv_bfloat16 *)a.o;
    if (p.split) {
        float *states = reinterpret_cast<float *>(a.ws), *total = reinterpret_cast<float *>(a.ws + p.state_bytes);
        kda_status st = tensor_states<tc::kForwardStates>(p, mk, mv, t, states, total, s);
        if (st == KDA_OK) st = launch_scan<false>(p, a.H, tc::kD, a.h0, total, states, s);
        if (st != KDA_OK) return st;
        t.ws = states;
    }
    constexpr size_t smem = tc::smem_bytes<false>();
    auto kern = tc::linear_sm100_kernel<tc::kOutputs>;
    if (!set_smem(kern, smem)) return KDA_ERR_CUDA;
    kern<<<(unsigned)((int64_t)p.map.units * a.H), tc::kThreads, smem, s>>>(mq, mk, mv, mo, t);
    return launched();
}

struct BwdArgs {
    const void *q, *k, *v, *dO;
    const float *g, *h0, *dhT;
    int per_token;
    int32_t Hk, H;
    float scale;
    void *dq, *dk, *dv;
    float *dg, *dh0;
    unsigned char *ws;
};

template <typename T>
kda_status launch_group_sum(const float *part, void *out, int64_t T_tot, int32_t Hk, int32_t H,
                            int32_t d, cudaStream_t s) {
    const int64_t rows = T_tot * Hk;
    const int64_t blocks = (rows * d / 4 + kThreads - 1) / kThreads;
    group_sum_kernel<T><<<(unsigned)blocks, kThreads, 0, s>>>(part, (T *)out, rows, H / Hk, d);
    return launched();
}

// Where a gradient call's workspace has what.
struct BwdSpace {
    float *S, *E, *totS, *totE, *term, *part;
    double *anchor, *sums;
    mm::Factors *factors;
};

inline BwdSpace bwd_space(const Plan &p, const BwdSizes &z, unsigned char *w) {
    BwdSpace b;
    auto take = [&](size_t n) {
        unsigned char *at = w;
        w += n;
        return at;
    };
    b.S = p.split ? (float *)take(z.states) : nullptr;
    b.E = p.split ? (float *)take(z.states) : nullptr;
    b.totS = (float *)take(z.totals);
    b.totE = (float *)take(z.totals);
    b.term = (float *)take(z.terms);
    b.anchor = (double *)take(z.anchors);
    b.sums = (double *)take(z.sums);
    b.part = z.parts ? (float *)take(z.parts) : nullptr;
    b.factors = (mm::Factors *)w;
    return b;
}

// The launches of a gradient: states of both directions and their scans when the
// sequences are split, dQ, then dK and dV; shared heads' parts are added after each.
template <int D>
kda_status bwd_simt(const Plan &p, const BwdArgs &a, cudaStream_t s) {
    const BwdSpace b = bwd_space(p, bwd_sizes(p, p.map.T_tot, a.Hk, a.H, D), a.ws);
    const float *q = (const float *)a.q, *k = (const float *)a.k, *v = (const float *)a.v, *dO = (const float *)a.dO;
    kda_status st = KDA_OK;
    if (p.split) {
        const dim3 grid((unsigned)p.bodies, (unsigned)a.H, (unsigned)(D / StateSmem<D>::kW));
        const size_t smem = sizeof(StateSmem<D>);
        auto fs = state_kernel<D, false>;
        auto rs = state_kernel<D, true>;
        if (!set_smem(fs, smem) || !set_smem(rs, smem)) return KDA_ERR_CUDA;
        fs<<<grid, kThreads, smem, s>>>(k, v, a.g, a.per_token, p.map, a.Hk, a.H, 1.f, b.S, b.totS);
        rs<<<grid, kThreads, smem, s>>>(q, dO, a.g, a.per_token, p.map, a.Hk, a.H, a.scale, b.E, b.totE);
        st = launched();
        if (st == KDA_OK) st = launch_scan<false>(p, a.H, D, a.h0, b.totS, b.S, s);
        if (st == KDA_OK) st = launch_scan<true>(p, a.H, D, a.dhT, b.totE, b.E, s);
        if (st != KDA_OK) return st;
    }
    const dim3 grid((unsigned)p.map.units, (unsigned)a.H);
    const size_t smem = sizeof(GradSmem<D>);
    auto kq = grad_q_kernel<D>;
    auto kkv = grad_kv_kernel<D>;
    if (!set_smem(kq, smem) || !set_smem(kkv, smem)) return KDA_ERR_CUDA;
    kq<<<grid, kThreads, smem, s>>>(q, k, v, dO, a.g, a.per_token, a.h0, a.dhT, p.map, a.Hk, a.H, a.scale, b.S, b.E,
                                    (float *)a.dq, b.part, b.term, b.anchor);
    st = launched();
    if (st == KDA_OK && b.part) st = launch_group_sum<float>(b.part, a.dq, p.map.T_tot, a.Hk, a.H, D, s);
    if (st != KDA_OK) return st;
    kkv<<<grid, kThreads, smem, s>>>(q, k, v, dO, a.g, a.per_token, a.dhT, p.map, a.Hk, a.H, a.scale, b.E, b.term,
                                     b.anchor, (float *)a.dk, b.part, (float *)a.dv, a.dg, b.sums, a.dh0);
    st = launched();
    if (st == KDA_OK && b.part) st = launch_group_sum<float>(b.part, a.dk, p.map.T_tot, a.Hk, a.H, D, s);
    if (st == KDA_OK && !a.per_token) {
        head_sum_kernel<<<(unsigned)a.H, kThreads, 0, s>>>(b.sums, a.dg, p.map.units, a.H);
        st = launched();
    }
    return st;
}

template <int D>
kda_status bwd_mma(const Plan &p, const BwdArgs &a, cudaStream_t s) {
    using T = __nv_bfloat16;
    const BwdSpace b = bwd_space(p, bwd_sizes(p, p.map.T_tot, a.Hk, a.H, D), a.ws);
    const T *q = (const T *)a.q, *k = (const T *)a.k, *v = (const T *)a.v, *dO = (const T *)a.dO;
    const unsigned grid = (unsigned)((int64_t)p.map.units * a.H), threads = mm::Shape<D>::kThreads;
    kda_status st = launch_factors(p, a.g, a.per_token, a.H, a.scale, b.factors, s);
    if (st != KDA_OK) return st;
    if (p.split) {
        if constexpr (D == tc::kD) {
            CUtensorMap mq, mk, mv, md;
            const int64_t T = p.map.T_tot;
            if (!tc::make_map(&mq, q, a.Hk, T) || !tc::make_map(&mk, k, a.Hk, T) ||
                !tc::make_map(&mv, v, a.H, T) || !tc::make_map(&md, dO, a.H, T))
                return KDA_ERR_CUDA;
            const tc::Params t = tensor_params(p, a.g, a.per_token, a.Hk, a.H, a.scale);
            st = tensor_states<tc::kForwardStates>(p, mk, mv, t, b.S, b.totS, s);
            if (st == KDA_OK) st = tensor_states<tc::kReverseStates>(p, mq, md, t, b.E, b.totE, s);
        } else {
            const size_t smem = sizeof(mm::StateSmem<D>);
            auto fs = mm::state_kernel<D, false>;
            auto rs = mm::state_kernel<D, true>;
            if (!set_smem(fs, smem) || !set_smem(rs, smem)) return KDA_ERR_CUDA;
            const unsigned bodies = (unsigned)((int64_t)p.bodies * a.H);
            fs<<<bodies, threads, smem, s>>>(k, v, b.factors, p.map, a.Hk, a.H, b.S, b.totS);
            rs<<<bodies, threads, smem, s>>>(q, dO, b.factors, p.map, a.Hk, a.H, b.E, b.totE);
            st = launched();
        }
        if (st == KDA_OK) st = launch_scan<false>(p, a.H, D, a.h0, b.totS, b.S, s);
        if (st == KDA_OK) st = launch_scan<true>(p, a.H, D, a.dhT, b.totE, b.E, s);
        if (st != KDA_OK) return st;
    }
    auto kq = mm::grad_q_kernel<D>;
    auto kkv = mm::grad_kv_kernel<D>;
    const size_t q_smem = sizeof(mm::GradSmem<D>), kv_smem = sizeof(mm::GradKvSmem<D>);
    if (!set_smem(kq, q_smem) || !set_smem(kkv, kv_smem)) return KDA_ERR_CUDA;
    kq<<<grid, threads, q_smem, s>>>(q, k, v, dO, b.factors, a.h0, a.dhT, p.map, a.Hk, a.H, a.scale, b.S, b.E,
                                     (T *)a.dq, b.part, b.term, b.anchor);
    st = launched();
    if (st == KDA_OK && b.part) st = launch_group_sum<T>(b.part, a.dq, p.map.T_tot, a.Hk, a.H, D, s);
    if (st != KDA_OK) return st;
    kkv<<<grid, threads, kv_smem, s>>>(q, k, v, dO, b.factors, a.dhT, p.map, a.Hk, a.H, a.scale, b.E, (T *)a.dk,
                                       b.part, (T *)a.dv, b.term, a.dh0);
    st = launched();
    if (st == KDA_OK && b.part) st = launch_group_sum<T>(b.part, a.dk, p.map.T_tot, a.Hk, a.H, D, s);
    if (st != KDA_OK) return st;
    mm::decay_grad_kernel<<<dim3((unsigned)p.map.units, (unsigned)((a.H + 31) / 32)), 32 * mm::kDecayWarps, 0, s>>>(
        b.term, b.anchor, a.per_token, p.map, a.H, a.dg, b.sums);
    st = launched();
    if (st == KDA_OK && !a.per_token) {
        head_sum_kernel<<<(unsigned)a.H, kThreads, 0, s>>>(b.sums, a.dg, p.map.units, a.H);
        st = launched();
    }
    return st;
}

template <typename T, int D>
kda_status step(const void *q, const void *k, const void *v, const float *g, int per_token,
                float *S, void *o, int64_t units, int Hk, int H, float scale, cudaStream_t s) {
    using Sh = StepShape<D>;
    const int64_t blocks = (units + Sh::kUnits - 1) / Sh::kUnits;
    step_kernel<T, D><<<(unsigned)blocks, Sh::kThreads, 0, s>>>(
        (const T *)q, (const T *)k, (const T *)v, g, per_token, S, (T *)o, units, Hk, H, scale);
    return launched();
}

// f<D>(...) by the run-time head size.
#define KDA_LIN_BY_D(f, d, ...)            \
    ((d) == 16   ? f<16>(__VA_ARGS__)      \
     : (d) == 32 ? f<32>(__VA_ARGS__)      \
     : (d) == 64 ? f<64>(__VA_ARGS__)      \
                 : f<128>(__VA_ARGS__))

inline kda_status fwd(int d, kda_dtype dt, const Plan &p, const FwdArgs &a, cudaStream_t s) {
    if (dt == KDA_FP32) return KDA_LIN_BY_D(fwd_simt, d, p, a, s);
    return d == 16   ? fwd_mma<16>(p, a, s)
           : d == 32 ? fwd_mma<32>(p, a, s)
           : d == 64 ? fwd_mma<64>(p, a, s)
                     : fwd_tensor(p, a, s);
}

inline kda_status bwd(int d, kda_dtype dt, const Plan &p, const BwdArgs &a, cudaStream_t s) {
    if (dt == KDA_FP32) return KDA_LIN_BY_D(bwd_simt, d, p, a, s);
    return KDA_LIN_BY_D(bwd_mma, d, p, a, s);
}

template <int D>
kda_status step_any(kda_dtype dt, const void *q, const void *k, const void *v, const float *g, int per_token,
                    float *S, void *o, int64_t units, int Hk, int H, float scale, cudaStream_t s) {
    return dt == KDA_BF16 ? step<__nv_bfloat16, D>(q, k, v, g, per_token, S, o, units, Hk, H, scale, s)
                          : step<float, D>(q, k, v, g, per_token, S, o, units, Hk, H, scale, s);
}

}  // namespace lin
}  // namespace kda

extern "C" KDA_API size_t kda_linear_chunk_fwd_workspace_size(int32_t N, int64_t T_tot, int32_t H,
                                                              int32_t d, kda_dtype dt) {
    using namespace kda::lin;
    if (N <= 0 || check_sizes(N, T_tot, 1, H, d, dt) != KDA_OK) return 0;
    const size_t a = fwd_bytes(make_plan(nullptr, N, T_tot, H, d, fwd_length(N, false, T_tot, H, d, dt), fwd_factors(d, dt)));
    const size_t b = fwd_bytes(make_plan(nullptr, N, T_tot, H, d, fwd_length(N, true, T_tot, H, d, dt), fwd_factors(d, dt)));
    return a > b ? a : b;
}

extern "C" KDA_API kda_status kda_linear_chunk_fwd(
    const void *q, const void *k, const void *v, const float *g, const float *h0,
    const int32_t *cu_seqlens, int32_t N, int64_t T_tot, int32_t Hk, int32_t H, int32_t d,
    kda_dtype dt, int32_t g_per_token, float scale, void *o, float *hT, void *workspace,
    size_t workspace_bytes, void *stream) {
    bool empty;
    kda_status st = kda::lin::check_shapes(N, T_tot, Hk, H, d, dt, cu_seqlens, scale, empty);
    if (st != KDA_OK || empty) return st;
    const void *req[] = {q, k, v, o};
    if (T_tot > 0 && (!kda::lin::all_given(req, 4) || !kda::lin::given4(g)))
        return KDA_ERR_INVALID_ARGUMENT;
    if (!kda::lin::ok16(h0) || !kda::lin::ok16(hT)) return KDA_ERR_INVALID_ARGUMENT;
    if (T_tot == 0 && hT == nullptr) return KDA_OK;
    const kda::lin::Plan p = kda::lin::make_plan(
        cu_seqlens, N, T_tot, H, d,
        kda::lin::fwd_length(N, cu_seqlens == nullptr, T_tot, H, d, dt), kda::lin::fwd_factors(d, dt));
    if ((int64_t)p.map.units * H > 0x7fffffff) return KDA_ERR_INVALID_ARGUMENT;
    const size_t need = kda_linear_chunk_fwd_workspace_size(N, T_tot, H, d, dt);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need ||
                     (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return KDA_ERR_WORKSPACE;
    const kda::lin::FwdArgs a = {q, k, v, g, h0, g_per_token, Hk, H, scale, o, hT,
                                 (unsigned char *)workspace};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return kda::lin::fwd(d, dt, p, a, s);
}

extern "C" KDA_API kda_status kda_linear_decode_step(
    const void *q, const void *k, const void *v, const float *g, float *S, void *o, int32_t B,
    int32_t Hk, int32_t H, int32_t d, kda_dtype dt, int32_t g_per_token, float scale,
    void *stream) {
    if (B < 0 || H <= 0 || Hk <= 0 || H % Hk != 0) return KDA_ERR_INVALID_ARGUMENT;
    if (dt != KDA_BF16 && dt != KDA_FP32) return KDA_ERR_UNSUPPORTED;
    if (!kda::lin::supported_d(d)) return KDA_ERR_UNSUPPORTED;
    if (!(scale - scale == 0.f)) return KDA_ERR_INVALID_ARGUMENT;
    if (B == 0) return KDA_OK;
    if ((int64_t)B * H > 0x7fffffff) return KDA_ERR_INVALID_ARGUMENT;
    const void *req[] = {q, k, v, S, o};
    if (!kda::lin::all_given(req, 5) || !kda::lin::given4(g)) return KDA_ERR_INVALID_ARGUMENT;
    return KDA_LIN_BY_D(kda::lin::step_any, d, dt, q, k, v, g, g_per_token, S, o, (int64_t)B * H, Hk,
                        H, scale, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" KDA_API size_t kda_linear_chunk_bwd_workspace_size(int32_t N, int64_t T_tot,
                                                              int32_t Hk, int32_t H, int32_t d,
                                                              kda_dtype dt) {
    using namespace kda::lin;
    if (N <= 0 || check_sizes(N, T_tot, Hk, H, d, dt) != KDA_OK) return 0;
    size_t most = 0;
    for (int equal = 0; equal < 2; ++equal) {
        const Plan p = make_plan(nullptr, N, T_tot, H, d, bwd_length(N, equal, T_tot, H, d, dt), dt == KDA_BF16);
        const size_t n = bwd_sizes(p, T_tot, Hk, H, d).all;
        most = n > most ? n : most;
    }
    return most;
}

extern "C" KDA_API kda_status kda_linear_chunk_bwd(
    const void *q, const void *k, const void *v, const float *g, const float *h0,
    const int32_t *cu_seqlens, int32_t N, int64_t T_tot, int32_t Hk, int32_t H, int32_t d,
    kda_dtype dt, int32_t g_per_token, float scale, const void *dO, const float *dhT, void *dq,
    void *dk, void *dv, float *dg, float *dh0, void *workspace, size_t workspace_bytes,
    void *stream) {
    bool empty;
    kda_status st = kda::lin::check_shapes(N, T_tot, Hk, H, d, dt, cu_seqlens, scale, empty);
    if (st != KDA_OK) return st;
    // a constant decay's gradient is written whatever the number of tokens
    if ((T_tot > 0 || !g_per_token) && !kda::lin::given4(dg))
        return KDA_ERR_INVALID_ARGUMENT;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (empty) {
        if (!g_per_token && cudaMemsetAsync(dg, 0, sizeof(float) * H, s) != cudaSuccess)
            return KDA_ERR_CUDA;
        return KDA_OK;
    }
    const void *req[] = {q, k, v, dO, dq, dk, dv};
    if (T_tot > 0 && (!kda::lin::all_given(req, 7) || !kda::lin::given4(g)))
        return KDA_ERR_INVALID_ARGUMENT;
    if (!kda::lin::ok16(h0) || !kda::lin::ok16(dhT) || !kda::lin::ok16(dh0))
        return KDA_ERR_INVALID_ARGUMENT;
    const kda::lin::Plan p = kda::lin::make_plan(
        cu_seqlens, N, T_tot, H, d,
        kda::lin::bwd_length(N, cu_seqlens == nullptr, T_tot, H, d, dt), dt == KDA_BF16);
    if ((int64_t)p.map.units * H > 0x7fffffff) return KDA_ERR_INVALID_ARGUMENT;
    const size_t need = kda_linear_chunk_bwd_workspace_size(N, T_tot, Hk, H, d, dt);
    if (workspace == nullptr || workspace_bytes < need ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return KDA_ERR_WORKSPACE;
    const kda::lin::BwdArgs a = {q, k, v, dO, g, h0, dhT, g_per_token, Hk, H, scale,
                                 dq, dk, dv, dg, dh0, (unsigned char *)workspace};
    return kda::lin::bwd(d, dt, p, a, s);
}
