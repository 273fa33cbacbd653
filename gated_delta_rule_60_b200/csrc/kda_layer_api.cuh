// kda_layer_api.cuh -- entry points of the steps around the operator: rotary
// positions and layer norm.  Included by kda_api.cu.
#pragma once

#include <algorithm>
#include <cmath>

namespace kda {
namespace rotary {

template <typename T, int V>
kda_status launch_v(const void *q, const void *k, const float *freq, const Args &a, bool pairs,
                    void *qo, void *ko, dim3 grid, cudaStream_t s) {
    if (pairs)
        rotary_kernel<T, V, true><<<grid, kThreads, 0, s>>>((const T *)q, (const T *)k, freq, a,
                                                            (T *)qo, (T *)ko);
    else
        rotary_kernel<T, V, false><<<grid, kThreads, 0, s>>>((const T *)q, (const T *)k, freq, a,
                                                             (T *)qo, (T *)ko);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

template <typename T, int V>
kda_status launch(const void *q, const void *k, const float *freq, Args a, bool pairs, void *qo,
                  void *ko, cudaStream_t s) {
    const int heads = a.Hq + a.Hk, half = a.rot / 2;
    // 16-byte accesses need every vector of every row on a 16-byte boundary
    const bool wide = half % V == 0 && a.d % V == 0 && a.q_stride % V == 0 &&
                      a.k_stride % V == 0 && a.qo_stride % V == 0 && a.ko_stride % V == 0;
    const int v = wide ? V : 1;
    const int64_t items = (int64_t)heads * (half / v + (a.d - a.rot) / v);
    // a block takes about 4 items a thread: several tokens of few heads, or some
    // of many heads while that still gives every SM its blocks
    a.tokens = (int)(items >= 4 * kThreads ? 1 : (4 * kThreads) / items);
    if (a.tokens > kMaxTokens) a.tokens = kMaxTokens;
    const int64_t spread = (a.T + 147) / 148;           // tokens per SM
    if (a.tokens > spread) a.tokens = (int)spread;
    const int64_t tiles = (a.T + a.tokens - 1) / a.tokens;
    int slices = 1;
    while (tiles * slices < 2 * 148 && slices < heads && items / slices > kThreads) slices *= 2;
    a.heads = (heads + slices - 1) / slices;
    slices = (heads + a.heads - 1) / a.heads;
    const dim3 grid((unsigned)tiles, (unsigned)slices);
    return wide ? launch_v<T, V>(q, k, freq, a, pairs, qo, ko, grid, s)
                : launch_v<T, 1>(q, k, freq, a, pairs, qo, ko, grid, s);
}

}  // namespace rotary

namespace ln {

constexpr int kMaxD = 8192;

// The smallest row share that holds D values, and the values of a thread: 16 up to
// 512, then 64 bytes of them.  The widest rows take 256 threads in bf16, 512 in fp32.
template <typename T>
constexpr int long_per() { return 64 / (int)sizeof(T); }
template <typename T>
constexpr int widest() { return kMaxD / long_per<T>(); }
#define KDA_LN_DISPATCH(T, D, CALL)                         \
    ((D) <= 32                   ? CALL(2, 16)              \
     : (D) <= 128                ? CALL(8, 16)              \
     : (D) <= 512                ? CALL(32, 16)             \
     : (D) <= 64 * long_per<T>() ? CALL(64, long_per<T>())  \
     : (D) <= 128 * long_per<T>() ? CALL(128, long_per<T>()) \
     : (D) <= 256 * long_per<T>() ? CALL(256, long_per<T>()) \
                                  : CALL(widest<T>(), long_per<T>()))

// Threads that share a row.
inline int row_share(int D, kda_dtype dt) {
#define KDA_LN_TPR(TPR, PER) TPR
    return dt == KDA_BF16 ? KDA_LN_DISPATCH(__nv_bfloat16, D, KDA_LN_TPR) : KDA_LN_DISPATCH(float, D, KDA_LN_TPR);
#undef KDA_LN_TPR
}

// How rows fall on blocks: gs groups of a block (the largest power of two that G
// and the block's rows share), and blocks along the tokens, so that all groups
// together have about `per_sm` blocks on every SM.
struct Grid {
    int gs, blocks;
};
inline Grid make_grid(int64_t tokens, int G, int tpr, int per_sm) {
    const int rows = tpr < 256 ? 256 / tpr : 1;
    int gs = 1;
    while (2 * gs <= rows && G % (2 * gs) == 0) gs *= 2;
    const int ts = rows / gs;
    const int64_t most = (tokens + ts - 1) / ts;
    const int64_t want = std::max(148 * per_sm / (G / gs), 1);
    return {gs, (int)(want < most ? want : most < 1 ? 1 : most)};
}
// About as many as are resident, so that a block walks along its tokens with the next
// rows on their way.
constexpr int kFwdPerSm = 3, kBwdPerSm = 2;

// A row can fill its share only where D is a multiple of a full vector.
template <typename T, int V>
constexpr bool may_fill() { return V * sizeof(T) == 16; }

template <typename T, int V, int kTpr, int kPer>
kda_status fwd_at(const void *x, const float *w, const float *b, int64_t tokens, int G, int D,
                  float eps, void *y, float *mean, float *rstd, cudaStream_t s) {
    constexpr int kNV = kPer / V, kThreads = Block<kTpr>::kThreads;
    const Grid g = make_grid(tokens, G, kTpr, kFwdPerSm);
    auto kern = fwd_kernel<T, V, kTpr, kNV, false>;
    if constexpr (may_fill<T, V>())
        if (D == kTpr * V * kNV) kern = fwd_kernel<T, V, kTpr, kNV, true>;
    const size_t smem = Feed<T, V, kNV, kThreads, 1>::kSmem;
    if (!lin::set_smem(kern, smem)) return KDA_ERR_CUDA;
    kern<<<dim3((unsigned)g.blocks, (unsigned)(G / g.gs)), kThreads, smem, s>>>(
        (const T *)x, w, b, tokens, G, g.gs, D, eps, (T *)y, mean, rstd);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

template <typename T, int V>
kda_status fwd(const void *x, const float *w, const float *b, int64_t tokens, int G, int D,
               float eps, void *y, float *mean, float *rstd, cudaStream_t s) {
#define KDA_LN_FWD(TPR, PER) fwd_at<T, V, TPR, PER>(x, w, b, tokens, G, D, eps, y, mean, rstd, s)
    return KDA_LN_DISPATCH(T, D, KDA_LN_FWD);
#undef KDA_LN_FWD
}

template <typename T, int V, int kTpr, int kPer, bool kBias>
kda_status bwd_at(const void *dy, const void *x, const float *mean, const float *rstd,
                  const float *w, int64_t tokens, int G, int D, void *dx, float *part,
                  cudaStream_t s) {
    constexpr int kNV = kPer / V, kRows = Block<kTpr>::kRows, kThreads = Block<kTpr>::kThreads;
    const Grid g = make_grid(tokens, G, kTpr, kBwdPerSm);
    const size_t sums = kRows != g.gs && part ? (size_t)kRows * D * sizeof(float) : 0;
    const size_t rows = Feed<T, V, kNV, kThreads, 2>::kSmem, smem = std::max(rows, sums);
    auto kern = bwd_kernel<T, V, kTpr, kNV, false, kBias>;
    if constexpr (may_fill<T, V>())
        if (D == kTpr * V * kNV) kern = bwd_kernel<T, V, kTpr, kNV, true, kBias>;
    if (!lin::set_smem(kern, smem)) return KDA_ERR_CUDA;
    kern<<<dim3((unsigned)g.blocks, (unsigned)(G / g.gs)), kThreads, smem, s>>>(
        (const T *)dy, (const T *)x, mean, rstd, w, tokens, G, g.gs, D, (T *)dx, part);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

template <typename T, int V>
kda_status bwd(const void *dy, const void *x, const float *mean, const float *rstd, const float *w,
               int64_t tokens, int G, int D, void *dx, float *part, bool bias, cudaStream_t s) {
#define KDA_LN_BWD(TPR, PER)                                                                   \
    (bias ? bwd_at<T, V, TPR, PER, true>(dy, x, mean, rstd, w, tokens, G, D, dx, part, s)      \
          : bwd_at<T, V, TPR, PER, false>(dy, x, mean, rstd, w, tokens, G, D, dx, part, s))
    return KDA_LN_DISPATCH(T, D, KDA_LN_BWD);
#undef KDA_LN_BWD
}

inline kda_status check(int64_t T, int32_t G, int32_t D, kda_dtype dt) {
    if (T < 0 || G <= 0 || D <= 0 || G > 65535) return KDA_ERR_INVALID_ARGUMENT;
    if (dt != KDA_BF16 && dt != KDA_FP32) return KDA_ERR_UNSUPPORTED;
    if (D > kMaxD) return KDA_ERR_UNSUPPORTED;
    if (T > (int64_t(1) << 40) / G / D) return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

}  // namespace ln
}  // namespace kda

extern "C" KDA_API kda_status kda_rotary_frequencies(int32_t rot, double base, kda_rope_scaling scaling,
                                                     double factor, double original_length,
                                                     double beta_fast, double beta_slow,
                                                     float *inv_freq, float *scale) {
    if (rot <= 0 || rot % 2 != 0 || rot > 2 * kda::rotary::kMaxHalf || inv_freq == nullptr ||
        scale == nullptr || !(base > 1.0) || !std::isfinite(base))
        return KDA_ERR_INVALID_ARGUMENT;
    if (scaling != KDA_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
        return KDA_ERR_INVALID_ARGUMENT;
    *scale = 1.f;
    const double pi2 = 6.283185307179586476925;
    switch (scaling) {
    case KDA_ROPE_NONE:
    case KDA_ROPE_LINEAR:
    case KDA_ROPE_BASE:
        if (scaling == KDA_ROPE_BASE && rot > 2) base *= std::pow(factor, (double)rot / (rot - 2));
        for (int i = 0; i < rot / 2; ++i) {
            const double f = std::pow(base, -2.0 * i / rot);
            inv_freq[i] = (float)(scaling == KDA_ROPE_LINEAR ? f / factor : f);
        }
        return KDA_OK;
    case KDA_ROPE_PARTS:
        if (!(original_length > 0.0) || !(beta_fast > beta_slow) || !(beta_slow >= 0.0) ||
            !std::isfinite(original_length) || !std::isfinite(beta_fast))
            return KDA_ERR_INVALID_ARGUMENT;
        for (int i = 0; i < rot / 2; ++i) {
            const double f = std::pow(base, -2.0 * i / rot);
            double keep = (original_length * f / pi2 - beta_slow) / (beta_fast - beta_slow);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            inv_freq[i] = (float)(f * keep + f / factor * (1.0 - keep));
        }
        *scale = (float)(1.0 + 0.1 * std::log(factor));
        return KDA_OK;
    }
    return KDA_ERR_UNSUPPORTED;
}

extern "C" KDA_API kda_status kda_rotary(const void *q, const void *k, const float *inv_freq,
                                         const int32_t *positions, const int32_t *cu_seqlens,
                                         int32_t N, int64_t T_tot, int32_t Hq, int32_t Hk,
                                         int32_t d, int32_t rot, kda_dtype dt, int32_t interleaved,
                                         int32_t inverse, float scale, int64_t q_stride,
                                         int64_t k_stride, void *q_out, void *k_out,
                                         int64_t q_out_stride, int64_t k_out_stride, void *stream) {
    if (T_tot < 0 || Hq <= 0 || Hk < 0 || d <= 0 || rot < 0 || rot % 2 != 0 || rot > d ||
        Hq > 65535 || Hk > 65535)
        return KDA_ERR_INVALID_ARGUMENT;
    if (dt != KDA_BF16 && dt != KDA_FP32) return KDA_ERR_UNSUPPORTED;
    if (d > 1024 || rot > 2 * kda::rotary::kMaxHalf) return KDA_ERR_UNSUPPORTED;
    if (!(scale - scale == 0.f)) return KDA_ERR_INVALID_ARGUMENT;
    const int64_t qw = (int64_t)Hq * d, kw = (int64_t)Hk * d;
    if (q_stride < qw || q_out_stride < qw || k_stride < kw || k_out_stride < kw)
        return KDA_ERR_INVALID_ARGUMENT;
    if (positions == nullptr && (N <= 0 || (cu_seqlens == nullptr && T_tot % N != 0)))
        return N == 0 && T_tot == 0 ? KDA_OK : KDA_ERR_INVALID_ARGUMENT;
    if (T_tot == 0) return KDA_OK;
    if (T_tot > 0x7fffffff) return KDA_ERR_UNSUPPORTED;
    const void *req[] = {q, q_out};
    if (!kda::lin::all_given(req, 2)) return KDA_ERR_INVALID_ARGUMENT;
    if (Hk > 0 && (k == nullptr || k_out == nullptr || !aligned16(k) || !aligned16(k_out)))
        return KDA_ERR_INVALID_ARGUMENT;
    if (rot > 0 && !kda::lin::given4(inv_freq)) return KDA_ERR_INVALID_ARGUMENT;
    if ((positions && !kda::lin::given4(positions)) || (cu_seqlens && !aligned16(cu_seqlens)))
        return KDA_ERR_INVALID_ARGUMENT;
    // in place only over the whole layout
    if ((q == q_out && q_stride != q_out_stride) || (k && k == k_out && k_stride != k_out_stride))
        return KDA_ERR_INVALID_ARGUMENT;
    // an output that starts where the other one, or the other input, does
    if (Hk > 0 && (q_out == k_out || q_out == k || k_out == q)) return KDA_ERR_INVALID_ARGUMENT;
    kda::rotary::Args a;
    a.pos = positions;
    a.cu = cu_seqlens;
    a.N = N;
    a.T = T_tot;
    a.Hq = Hq;
    a.Hk = Hk;
    a.d = d;
    a.rot = rot;
    a.inverse = inverse;
    a.scale = scale;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.qo_stride = q_out_stride;
    a.ko_stride = k_out_stride;
    a.tokens = a.heads = 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dt == KDA_BF16
               ? kda::rotary::launch<__nv_bfloat16, 8>(q, k, inv_freq, a, interleaved != 0, q_out, k_out, s)
               : kda::rotary::launch<float, 4>(q, k, inv_freq, a, interleaved != 0, q_out, k_out, s);
}

extern "C" KDA_API kda_status kda_layernorm_fwd(const void *x, const float *weight,
                                                const float *bias, int64_t T, int32_t G, int32_t D,
                                                kda_dtype dt, float eps, void *y, float *mean,
                                                float *rstd, void *stream) {
    const kda_status st = kda::ln::check(T, G, D, dt);
    if (st != KDA_OK) return st;
    if (!(eps >= 0.f) || !(eps - eps == 0.f)) return KDA_ERR_INVALID_ARGUMENT;
    if (T == 0) return KDA_OK;
    const void *req[] = {x, y};
    if (!kda::lin::all_given(req, 2) || !kda::lin::given4(mean) || !kda::lin::given4(rstd) ||
        !kda::lin::ok16(weight) || !kda::lin::ok16(bias))
        return KDA_ERR_INVALID_ARGUMENT;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    using namespace kda::ln;
    if (dt == KDA_BF16)
        return D % 8 == 0   ? fwd<__nv_bfloat16, 8>(x, weight, bias, T, G, D, eps, y, mean, rstd, s)
               : D % 2 == 0 ? fwd<__nv_bfloat16, 2>(x, weight, bias, T, G, D, eps, y, mean, rstd, s)
                            : fwd<__nv_bfloat16, 1>(x, weight, bias, T, G, D, eps, y, mean, rstd, s);
    return D % 4 == 0 ? fwd<float, 4>(x, weight, bias, T, G, D, eps, y, mean, rstd, s)
                      : fwd<float, 1>(x, weight, bias, T, G, D, eps, y, mean, rstd, s);
}

extern "C" KDA_API size_t kda_layernorm_bwd_workspace_size(int64_t T, int32_t G, int32_t D,
                                                           kda_dtype dt) {
    if (kda::ln::check(T, G, D, dt) != KDA_OK || T == 0) return 0;
    const kda::ln::Grid g = kda::ln::make_grid(T, G, kda::ln::row_share(D, dt), kda::ln::kBwdPerSm);
    return (size_t)g.blocks * 2 * G * D * sizeof(float);
}

extern "C" KDA_API kda_status kda_layernorm_bwd(const void *dy, const void *x, const float *mean,
                                                const float *rstd, const float *weight, int64_t T,
                                                int32_t G, int32_t D, kda_dtype dt, void *dx,
                                                float *dweight, float *dbias, void *workspace,
                                                size_t workspace_bytes, void *stream) {
    const kda_status st0 = kda::ln::check(T, G, D, dt);
    if (st0 != KDA_OK) return st0;
    if (!kda::lin::ok16(weight) || !kda::lin::ok16(dweight) || !kda::lin::ok16(dbias))
        return KDA_ERR_INVALID_ARGUMENT;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) {                                       // no rows: the sums are zero
        const size_t n = (size_t)G * D * sizeof(float);
        if ((dweight && cudaMemsetAsync(dweight, 0, n, s) != cudaSuccess) ||
            (dbias && cudaMemsetAsync(dbias, 0, n, s) != cudaSuccess))
            return KDA_ERR_CUDA;
        return KDA_OK;
    }
    const void *req[] = {dy, x, dx};
    if (!kda::lin::all_given(req, 3) || !kda::lin::given4(mean) || !kda::lin::given4(rstd))
        return KDA_ERR_INVALID_ARGUMENT;
    const bool sums = dweight != nullptr || dbias != nullptr;
    const size_t need = sums ? kda_layernorm_bwd_workspace_size(T, G, D, dt) : 0;
    if (sums && (workspace == nullptr || workspace_bytes < need ||
                 (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return KDA_ERR_WORKSPACE;
    float *part = sums ? (float *)workspace : nullptr;
    using namespace kda::ln;
    const int blocks = make_grid(T, G, row_share(D, dt), kBwdPerSm).blocks;
    const bool b = dbias != nullptr;
    kda_status st;
    if (dt == KDA_BF16)
        st = D % 8 == 0   ? bwd<__nv_bfloat16, 8>(dy, x, mean, rstd, weight, T, G, D, dx, part, b, s)
             : D % 2 == 0 ? bwd<__nv_bfloat16, 2>(dy, x, mean, rstd, weight, T, G, D, dx, part, b, s)
                          : bwd<__nv_bfloat16, 1>(dy, x, mean, rstd, weight, T, G, D, dx, part, b, s);
    else
        st = D % 4 == 0 ? bwd<float, 4>(dy, x, mean, rstd, weight, T, G, D, dx, part, b, s)
                        : bwd<float, 1>(dy, x, mean, rstd, weight, T, G, D, dx, part, b, s);
    if (st != KDA_OK || !sums) return st;
    const int64_t n = (int64_t)G * D;
    weight_sum_kernel<<<dim3((unsigned)((n + 31) / 32), dbias != nullptr ? 2 : 1), 256, 0, s>>>(
        part, blocks, n, dweight, dbias);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
