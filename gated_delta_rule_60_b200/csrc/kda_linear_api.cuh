// kda_linear_api.cuh -- entry points of the decayed linear attention: argument
// checks, the split into segments, workspaces, launches.  Included by kda_api.cu.
#pragma once

namespace kda {
namespace lin {

constexpr int64_t kNoSplit = int64_t(1) << 40;         // segment length of "one segment each"

inline size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

// Tokens of a segment.  With chains = (sequence, head, column block) triples,
// no split is made when they fill the GPU and their lengths are known to be
// equal; else a segment is a quarter of an SM's even share of the tokens, so
// that no long sequence is left over at the end.
inline int64_t segment_length(int32_t N, bool equal, int64_t T_tot, int64_t chains_per_seq, int chunk) {
    const int64_t kSMs = 148;
    if (N <= 0 || T_tot <= 0) return kNoSplit;
    if ((equal || N == 1) && N * chains_per_seq >= 2 * kSMs) return kNoSplit;
    int64_t L = (T_tot * chains_per_seq + 4 * kSMs - 1) / (4 * kSMs);
    if (L < 256) L = 256;
    L = (L + chunk - 1) / chunk * chunk;
    return L >= T_tot ? kNoSplit : L;
}

struct Plan {
    SegMap map;
    bool split;
    size_t state_bytes, total_bytes;                   // of one direction
};

inline Plan make_plan(const int32_t *cu, int32_t N, int64_t T_tot, int32_t H, int32_t d, int64_t L) {
    Plan p;
    p.map.cu = cu;
    p.map.N = N;
    p.map.T_tot = T_tot;
    p.map.L = L;
    p.map.units = (int)(T_tot / L + N);
    p.split = L != kNoSplit;
    const size_t n = (size_t)p.map.units * H;
    p.state_bytes = p.split ? align256(n * d * d * sizeof(float)) : 0;
    p.total_bytes = p.split ? align256(n * sizeof(float)) : 0;
    return p;
}

// The tensor-core kernels: one block an SM, a chunk of 128 tokens takes about
// 1.7 us there, and 0.9 us where only states are wanted.
inline bool tensor_path(int32_t d, kda_dtype dt) { return d == 128 && dt == KDA_BF16; }

// Equal lengths: the number of segments that minimises the waves of both passes
// (the first over all segments but the last) and the two further launches.
// Lengths that the host does not know: an SM's even share of the tokens, which
// bounds what one long sequence can leave over.
inline int64_t tensor_length(int32_t N, bool equal, int64_t T_tot, int32_t H) {
    const int64_t kSMs = 148;
    if (N <= 0 || T_tot <= 0) return kNoSplit;
    if (!equal) {
        int64_t L = (T_tot * H + kSMs - 1) / kSMs;
        if (L < 1024) L = 1024;
        L = (L + tc::kTok - 1) / tc::kTok * tc::kTok;
        return L >= T_tot ? kNoSplit : L;
    }
    const int64_t len = (T_tot + N - 1) / N, chunks = (len + tc::kTok - 1) / tc::kTok;
    auto waves = [&](int64_t blocks) { return (double)((blocks + kSMs - 1) / kSMs); };
    double best = waves((int64_t)N * H) * 1.7 * (double)chunks;
    int64_t L = kNoSplit;
    for (int64_t G = 2; G <= 64 && G * 4 <= chunks; ++G) {
        const int64_t per = (chunks + G - 1) / G;
        const double t = ((double)per) * (waves((int64_t)N * H * G) * 1.7 + waves((int64_t)N * H * (G - 1)) * 0.9) + 8.0;
        if (t < best) {
            best = t;
            L = per * tc::kTok;
        }
    }
    return L;
}

// The workspace query does not know whether cu_seqlens is given: with several
// sequences it takes the larger of the two plans.
inline int64_t fwd_length(int32_t N, bool equal, int64_t T_tot, int32_t H, int32_t d, kda_dtype dt) {
    return tensor_path(d, dt) ? tensor_length(N, equal || N == 1, T_tot, H)
                              : segment_length(N, false, T_tot, (int64_t)H * (d < 64 ? 1 : d / 64), kC);
}

inline size_t fwd_bytes(const Plan &p) { return p.state_bytes + p.total_bytes; }

inline int64_t bwd_length(int32_t N, int64_t T_tot, int32_t H, int32_t d) {
    (void)d;
    return segment_length(N, false, T_tot, H, kC);
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
    s.all = 2 * s.states + 2 * s.totals + s.terms + s.anchors + s.sums + s.parts;
    return s;
}

inline bool supported_d(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

// Checks that the prefill and its gradient share; KDA_OK leaves `empty` true
// when there is nothing to do.
inline kda_status check_shapes(int32_t N, int64_t T_tot, int32_t Hk, int32_t H, int32_t d,
                               kda_dtype dt, const int32_t *cu, float scale, bool &empty) {
    empty = false;
    if (N < 0 || T_tot < 0 || H <= 0 || Hk <= 0 || H > 65535 || H % Hk != 0)
        return KDA_ERR_INVALID_ARGUMENT;
    if (dt != KDA_BF16 && dt != KDA_FP32) return KDA_ERR_UNSUPPORTED;
    if (!supported_d(d)) return KDA_ERR_UNSUPPORTED;
    if (T_tot > kMaxTokensSm100) return KDA_ERR_UNSUPPORTED;
    if (!(scale - scale == 0.f)) return KDA_ERR_INVALID_ARGUMENT;       // inf or NaN
    if (N == 0) {
        empty = true;
        return T_tot == 0 ? KDA_OK : KDA_ERR_INVALID_ARGUMENT;
    }
    if (cu == nullptr && (T_tot % N) != 0) return KDA_ERR_INVALID_ARGUMENT;
    if (cu != nullptr && !aligned16(cu)) return KDA_ERR_INVALID_ARGUMENT;
    if ((int64_t)N * H > 0x7fffffff || T_tot / 256 + N > 0x7fffffff) return KDA_ERR_INVALID_ARGUMENT;
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
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) ==
           cudaSuccess;
}

inline kda_status launched() { return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

template <bool kReverse>
inline kda_status launch_scan(const Plan &p, int H, int d, const float *init, const float *total,
                              float *ws, cudaStream_t s) {
    const int dd = d * d;
    const dim3 grid((unsigned)((dd + 4 * kScanThreads - 1) / (4 * kScanThreads)), (unsigned)H,
                    (unsigned)(p.map.N < 65535 ? p.map.N : 65535));
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

template <typename T, int D>
kda_status fwd_simt(const Plan &p, const FwdArgs &a, cudaStream_t s) {
    float *states = nullptr, *total = nullptr;
    const dim3 grid((unsigned)p.map.units, (unsigned)a.H, (unsigned)(D / OutSmem<D>::kW));
    if (p.split) {
        states = reinterpret_cast<float *>(a.ws);
        total = reinterpret_cast<float *>(a.ws + p.state_bytes);
        auto kern = state_kernel<T, D, false>;
        const size_t smem = sizeof(StateSmem<D>);
        if (!set_smem(kern, smem)) return KDA_ERR_CUDA;
        kern<<<grid, kThreads, smem, s>>>((const T *)a.k, (const T *)a.v, a.g, a.per_token, p.map,
                                          a.Hk, a.H, 1.f, states, total);
        kda_status st = launched();
        if (st == KDA_OK) st = launch_scan<false>(p, a.H, D, a.h0, total, states, s);
        if (st != KDA_OK) return st;
    }
    auto kern = out_kernel<T, D>;
    const size_t smem = sizeof(OutSmem<D>);
    if (!set_smem(kern, smem)) return KDA_ERR_CUDA;
    kern<<<grid, kThreads, smem, s>>>((const T *)a.q, (const T *)a.k, (const T *)a.v, a.g,
                                      a.per_token, a.h0, p.map, a.Hk, a.H, a.scale, states,
                                      (T *)a.o, a.hT);
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
    tc::Params t;
    t.g = a.g;
    t.h0 = a.h0;
    t.ws = nullptr;
    t.out = a.hT;
    t.total = nullptr;
    t.o = (__nv_bfloat16 *)a.o;
    t.m = p.map;
    t.per_token = a.per_token;
    t.Hk = a.Hk;
    t.H = a.H;
    t.scale = a.scale;
    const unsigned blocks = (unsigned)((int64_t)p.map.units * a.H);
    if (p.split) {
        tc::Params r = t;
        r.out = reinterpret_cast<float *>(a.ws);
        r.total = reinterpret_cast<float *>(a.ws + p.state_bytes);
        if (!set_smem(tc::linear_sm100_kernel<true>, tc::kSmem)) return KDA_ERR_CUDA;
        tc::linear_sm100_kernel<true><<<blocks, tc::kThreads, tc::kSmem, s>>>(mq, mk, mv, mo, r);
        kda_status st = launched();
        if (st == KDA_OK) st = launch_scan<false>(p, a.H, tc::kD, a.h0, r.total, r.out, s);
        if (st != KDA_OK) return st;
        t.ws = r.out;
    }
    if (!set_smem(tc::linear_sm100_kernel<false>, tc::kSmem)) return KDA_ERR_CUDA;
    tc::linear_sm100_kernel<false><<<blocks, tc::kThreads, tc::kSmem, s>>>(mq, mk, mv, mo, t);
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

template <typename T, int D>
kda_status bwd_simt(const Plan &p, const BwdArgs &a, cudaStream_t s) {
    const BwdSizes z = bwd_sizes(p, p.map.T_tot, a.Hk, a.H, D);
    unsigned char *w = a.ws;
    float *wsS = p.split ? (float *)w : nullptr;
    w += z.states;
    float *wsE = p.split ? (float *)w : nullptr;
    w += z.states;
    float *totS = (float *)w;
    w += z.totals;
    float *totE = (float *)w;
    w += z.totals;
    float *term = (float *)w;
    w += z.terms;
    double *anchor = (double *)w;
    w += z.anchors;
    double *sums = (double *)w;
    w += z.sums;
    float *part = z.parts ? (float *)w : nullptr;
    kda_status st = KDA_OK;
    if (p.split) {
        const dim3 grid((unsigned)p.map.units, (unsigned)a.H, (unsigned)(D / StateSmem<D>::kW));
        const size_t smem = sizeof(StateSmem<D>);
        auto f = state_kernel<T, D, false>;
        auto r = state_kernel<T, D, true>;
        if (!set_smem(f, smem) || !set_smem(r, smem)) return KDA_ERR_CUDA;
        f<<<grid, kThreads, smem, s>>>((const T *)a.k, (const T *)a.v, a.g, a.per_token, p.map,
                                       a.Hk, a.H, 1.f, wsS, totS);
        r<<<grid, kThreads, smem, s>>>((const T *)a.q, (const T *)a.dO, a.g, a.per_token, p.map,
                                       a.Hk, a.H, a.scale, wsE, totE);
        st = launched();
        if (st == KDA_OK) st = launch_scan<false>(p, a.H, D, a.h0, totS, wsS, s);
        if (st == KDA_OK) st = launch_scan<true>(p, a.H, D, a.dhT, totE, wsE, s);
        if (st != KDA_OK) return st;
    }
    const dim3 grid((unsigned)p.map.units, (unsigned)a.H);
    const size_t smem = sizeof(GradSmem<D>);
    auto kq = grad_q_kernel<T, D>;
    auto kkv = grad_kv_kernel<T, D>;
    if (!set_smem(kq, smem) || !set_smem(kkv, smem)) return KDA_ERR_CUDA;
    kq<<<grid, kThreads, smem, s>>>((const T *)a.q, (const T *)a.k, (const T *)a.v,
                                    (const T *)a.dO, a.g, a.per_token, a.h0, a.dhT, p.map, a.Hk,
                                    a.H, a.scale, wsS, wsE, (T *)a.dq, part, term, anchor);
    st = launched();
    if (st == KDA_OK && part) st = launch_group_sum<T>(part, a.dq, p.map.T_tot, a.Hk, a.H, D, s);
    if (st != KDA_OK) return st;
    kkv<<<grid, kThreads, smem, s>>>((const T *)a.q, (const T *)a.k, (const T *)a.v,
                                     (const T *)a.dO, a.g, a.per_token, a.dhT, p.map, a.Hk, a.H,
                                     a.scale, wsE, term, anchor, (T *)a.dk, part, (T *)a.dv, a.dg,
                                     sums, a.dh0);
    st = launched();
    if (st == KDA_OK && part) st = launch_group_sum<T>(part, a.dk, p.map.T_tot, a.Hk, a.H, D, s);
    if (st == KDA_OK && !a.per_token) {
        head_sum_kernel<<<(unsigned)a.H, kThreads, 0, s>>>(sums, a.dg, p.map.units, a.H);
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

// f<T, D>(...) by the run-time type and head size.
#define KDA_LIN_DISPATCH(f, dt, d, ...)                                                     \
    ((dt) == KDA_BF16                                                                       \
         ? ((d) == 16   ? f<__nv_bfloat16, 16>(__VA_ARGS__)                                 \
            : (d) == 32 ? f<__nv_bfloat16, 32>(__VA_ARGS__)                                 \
            : (d) == 64 ? f<__nv_bfloat16, 64>(__VA_ARGS__)                                 \
                        : f<__nv_bfloat16, 128>(__VA_ARGS__))                               \
         : ((d) == 16   ? f<float, 16>(__VA_ARGS__)                                         \
            : (d) == 32 ? f<float, 32>(__VA_ARGS__)                                         \
            : (d) == 64 ? f<float, 64>(__VA_ARGS__)                                         \
                        : f<float, 128>(__VA_ARGS__)))

}  // namespace lin
}  // namespace kda

extern "C" KDA_API size_t kda_linear_chunk_fwd_workspace_size(int32_t N, int64_t T_tot, int32_t H,
                                                              int32_t d, kda_dtype dt) {
    using namespace kda::lin;
    if (N <= 0 || T_tot < 0 || H <= 0 || !supported_d(d)) return 0;
    if (dt != KDA_BF16 && dt != KDA_FP32) return 0;
    const size_t a = fwd_bytes(make_plan(nullptr, N, T_tot, H, d, fwd_length(N, false, T_tot, H, d, dt)));
    const size_t b = fwd_bytes(make_plan(nullptr, N, T_tot, H, d, fwd_length(N, true, T_tot, H, d, dt)));
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
        kda::lin::fwd_length(N, cu_seqlens == nullptr, T_tot, H, d, dt));
    if ((int64_t)p.map.units * H > 0x7fffffff) return KDA_ERR_INVALID_ARGUMENT;
    const size_t need = kda_linear_chunk_fwd_workspace_size(N, T_tot, H, d, dt);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need ||
                     (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return KDA_ERR_WORKSPACE;
    const kda::lin::FwdArgs a = {q, k, v, g, h0, g_per_token, Hk, H, scale, o, hT,
                                 (unsigned char *)workspace};
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (kda::lin::tensor_path(d, dt)) return kda::lin::fwd_tensor(p, a, s);
    return KDA_LIN_DISPATCH(kda::lin::fwd_simt, dt, d, p, a, s);
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
    return KDA_LIN_DISPATCH(kda::lin::step, dt, d, q, k, v, g, g_per_token, S, o, (int64_t)B * H,
                            Hk, H, scale, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" KDA_API size_t kda_linear_chunk_bwd_workspace_size(int32_t N, int64_t T_tot,
                                                              int32_t Hk, int32_t H, int32_t d,
                                                              kda_dtype dt) {
    if (N <= 0 || T_tot < 0 || H <= 0 || Hk <= 0 || !kda::lin::supported_d(d)) return 0;
    if (dt != KDA_BF16 && dt != KDA_FP32) return 0;
    const kda::lin::Plan p = kda::lin::make_plan(nullptr, N, T_tot, H, d,
                                                 kda::lin::bwd_length(N, T_tot, H, d));
    return kda::lin::bwd_sizes(p, T_tot, Hk, H, d).all;
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
    const kda::lin::Plan p = kda::lin::make_plan(cu_seqlens, N, T_tot, H, d,
                                                 kda::lin::bwd_length(N, T_tot, H, d));
    const size_t need = kda::lin::bwd_sizes(p, T_tot, Hk, H, d).all;
    if (workspace == nullptr || workspace_bytes < need ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return KDA_ERR_WORKSPACE;
    const kda::lin::BwdArgs a = {q, k, v, dO, g, h0, dhT, g_per_token, Hk, H, scale,
                                 dq, dk, dv, dg, dh0, (unsigned char *)workspace};
    return KDA_LIN_DISPATCH(kda::lin::bwd_simt, dt, d, p, a, s);
}
