// kda_linear_decode.cuh -- one token of the decayed linear attention for each
// (sequence, head), the fp32 state updated in place:
//   S = e^g S + k v^T,   o = scale S^T q
//
// Bound by memory: 2 x 4 d^2 bytes of state per (sequence, head) against a few
// rows of d values.  A thread owns kR rows x 4 columns: 16-byte accesses, each element
// read once and written once with the streaming hint (the state of a batch is far
// larger than L2), and the write does not wait for the output's reduction, which meets
// once in shared memory.  A thread has few of its loads in flight (32 registers in all
// at d = 128); what hides their latency is that 95 % of an SM's warps are there.
//
// Measured: 256 x 96 states of 128 x 128 509 us, 6.4 TB/s, the rate of a plain copy;
// one sequence of 16 heads of 64 2.7 us, the latency of one block.
#pragma once

#include "kda_decode.cuh"
#include "kda_linear_common.cuh"

namespace kda {
namespace lin {

template <int D>
struct StepShape {
    static constexpr int kR = D == 128 ? 16 : D >= 32 ? 8 : 4;    // rows of a thread
    static constexpr int kGroups = D / kR;                        // row groups of a unit
    static constexpr int kUnitThreads = kGroups * D / 4;
    static constexpr int kThreads = kUnitThreads < 128 ? 128 : kUnitThreads;
    static constexpr int kUnits = kThreads / kUnitThreads;        // (sequence, head) of a block
};

template <typename T, int D>
__global__ void __launch_bounds__(StepShape<D>::kThreads)
step_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
            const float *__restrict__ g, int per_token, float *__restrict__ S, T *__restrict__ o,
            int64_t units, int Hk, int H, float scale) {
    using Sh = StepShape<D>;
    constexpr int R = Sh::kR;
    __shared__ float4 part[Sh::kUnits][Sh::kGroups][D / 4];
    const int x = threadIdx.x / Sh::kUnitThreads, t = threadIdx.x % Sh::kUnitThreads;
    const int rg = t / (D / 4), c4 = t % (D / 4);
    const int64_t u = (int64_t)blockIdx.x * Sh::kUnits + x;
    if (u < units) {
        float *Su = S + (size_t)u * D * D + (size_t)(rg * R) * D + 4 * c4;
        float4 s[R];
#pragma unroll
        for (int i = 0; i < R; ++i) s[i] = ld_stream_f4(Su + (size_t)i * D);
        const int64_t b = u / H;
        const int h = (int)(u % H);
        const size_t shared_row = ((size_t)b * Hk + h / (H / Hk)) * D + rg * R;
        const float a = expf(load_decay(g, per_token, b, h, H));
        const T *vp = v + (size_t)u * D + 4 * c4;
        const float4 vv = make_float4(IO<T>::ld(vp), IO<T>::ld(vp + 1), IO<T>::ld(vp + 2), IO<T>::ld(vp + 3));
        float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float kk = IO<T>::ld(k + shared_row + i), qq = IO<T>::ld(q + shared_row + i);
            s[i].x = fmaf(kk, vv.x, a * s[i].x); s[i].y = fmaf(kk, vv.y, a * s[i].y);
            s[i].z = fmaf(kk, vv.z, a * s[i].z); s[i].w = fmaf(kk, vv.w, a * s[i].w);
            r.x = fmaf(qq, s[i].x, r.x); r.y = fmaf(qq, s[i].y, r.y);
            r.z = fmaf(qq, s[i].z, r.z); r.w = fmaf(qq, s[i].w, r.w);
            st_stream_f4(Su + (size_t)i * D, s[i]);
        }
        part[x][rg][c4] = r;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < Sh::kUnits * D; e += Sh::kThreads) {
        const int64_t w = (int64_t)blockIdx.x * Sh::kUnits + e / D;
        if (w >= units) break;
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < Sh::kGroups; ++i) y += reinterpret_cast<const float *>(part[e / D][i])[e % D];
        IO<T>::st(o + (size_t)w * D + e % D, y * scale);
    }
}

}  // namespace lin
}  // namespace kda
