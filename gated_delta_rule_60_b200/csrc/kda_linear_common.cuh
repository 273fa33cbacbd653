// kda_linear_common.cuh -- decayed linear attention: the segment map, the
// decay sums, and the scan over segment states that every path shares.
//
// Per head, with a log-decay g_t <= 0 (one per token, or one constant):
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale * S_t^T q_t
// A chunk of C tokens starting from S0, with b_i = g_1 + .. + g_i inside it and
// D_ij = e^{b_i - b_j} for i >= j:
//   O  = scale * ( Diag(e^b) Q S0 + (Q K^T . D) V )
//   S  = e^{b_C} S0 + (Diag(e^{b_C - b}) K)^T V
// The composition of two stretches of tokens is S -> gamma S + R with a scalar
// gamma, so a sequence can be cut into segments: every segment's R from a zero
// start (in parallel), an elementwise scan of the R of one (sequence, head),
// then every segment's outputs from its true start state (in parallel).
//
// Segment map.  Sequence lengths are known on the device only.  A segment is L
// tokens of one sequence (the last one shorter); segment s of sequence n gets
// the unit number  start_n / L + n + s.  Because ceil(len / L) <=
// (start + len) / L - start / L + 1, the numbers of different sequences never
// meet, the largest is below T_tot / L + N, and a unit finds its sequence by a
// binary search of cu_seqlens: no table, no launch to build one.  At most N
// units have no segment and return at once.
//
// State slots.  Only a segment of a sequence that is longer than L has a state in
// the workspace, so segment s of such a sequence has the slot  j + s + min(n, j)
// with j = start_n / L.  The next such sequence has j' >= j + count - 1 > j and
// n' > n, so its first slot is behind this one's last; and as j + count - 1 <=
// T_tot / L, all lie below T_tot / L + min(N, T_tot / L).  (With a state for every
// unit, the workspace of 4,096 sequences of 96 heads of 128 was 26 GB.)
#pragma once

#include "kda_common.cuh"
#include "sm100_ptx.cuh"

namespace kda {
namespace lin {

struct SegMap {
    const int32_t *cu;
    int N;
    int64_t T_tot;
    int64_t L;      // tokens of a segment, at most kNoSplit
    int units;      // T_tot / L + N
    int per;        // tokens of each sequence where cu is NULL
};

// Token numbers stay below 2^31, so that a block finds its segment with 32-bit
// divisions (64-bit ones took 8 us of 253 at 96 heads x 8,192 tokens, 23 of 620 packed).
constexpr int64_t kNoSplit = int64_t(1) << 31;         // segment length of "one segment each"

struct Segment {
    int n;                 // sequence
    int s, count;          // index of the segment, segments of the sequence
    int slot;              // of its state (count > 1)
    int64_t t0, t1;        // its tokens
};

__host__ __device__ __forceinline__ int64_t seq_begin(const SegMap &m, int n) {
    return m.cu == nullptr ? (int64_t)n * m.per : (int64_t)m.cu[n];
}

__host__ __device__ __forceinline__ int64_t by_length(const SegMap &m, int64_t t) {
    return (uint32_t)t / (uint32_t)m.L;
}

__host__ __device__ __forceinline__ int64_t unit_base(const SegMap &m, int n) {
    return by_length(m, seq_begin(m, n)) + n;
}

__host__ __device__ inline int64_t state_slots(int64_t T_tot, int64_t L, int64_t N) {
    const int64_t j = T_tot / L;
    return j + (N < j ? N : j);
}
__host__ __device__ __forceinline__ int state_slot(int n, int j, int s) { return j + s + (n < j ? n : j); }

// The segments of sequence n; false when its bounds are malformed.  With good
// bounds every unit of the sequence lies in [0, m.units).
__host__ __device__ __forceinline__ bool seq_segments(const SegMap &m, int n, int64_t &start, int64_t &end,
                                                      int &base, int &count) {
    start = seq_begin(m, n);
    end = start + m.per;
    if (m.cu != nullptr && !seq_bounds(m.cu, n, m.N, m.T_tot, start, end)) return false;
    base = (int)(by_length(m, start) + n);
    count = end > start ? (int)by_length(m, end - start + m.L - 1) : 1;
    return true;
}

// The segment of unit u; false when it has none.
__host__ __device__ __forceinline__ bool find_segment(const SegMap &m, int u, Segment &g) {
    int lo = 0, hi = m.N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (unit_base(m, mid) <= u) lo = mid;
        else hi = mid - 1;
    }
    int64_t start, end;
    int base;
    g.n = lo;
    if (!seq_segments(m, lo, start, end, base, g.count)) return false;
    g.s = u - base;
    if (g.s < 0 || g.s >= g.count) return false;
    g.slot = state_slot(lo, base - lo, g.s);
    g.t0 = start + (int64_t)g.s * m.L;
    g.t1 = g.t0 + m.L < end ? g.t0 + m.L : end;
    return true;
}

// Longest first.  Blocks start in index order, so with the units of a batch in
// decreasing length the last to start are the short ones; each block ranks the
// units itself (ties by index, so the ranks are a permutation).  Up to one unit a
// thread; above that there are enough of them for their order not to matter.
// len: kBlock + 1 words of shared memory that nobody uses yet.
template <int kBlock>
__device__ __forceinline__ int ranked_unit(const SegMap &m, int rank, int *len) {
    if (m.cu == nullptr || m.units <= 1 || m.units > kBlock) return rank;
    const int t = threadIdx.x;
    if (t < m.units) {
        Segment g;
        len[t] = find_segment(m, t, g) ? (int)(g.t1 - g.t0) : -1;
    }
    if (t == 0) len[kBlock] = 0;
    __syncthreads();
    if (t < m.units) {
        const int mine = len[t];
        int r = 0;
        for (int j = 0; j < m.units; ++j) r += (len[j] > mine) | ((len[j] == mine) & (j < t));
        if (r == rank) len[kBlock] = t;
    }
    __syncthreads();
    const int u = len[kBlock];
    __syncthreads();
    return u;
}

// The segments whose own states are wanted, all but one of each sequence (the last,
// or in reverse the first), are numbered without gaps for short sequences:
// segment i of them has the number start_n / L + i.  A sequence with any is longer
// than L, so the numbers never meet, all lie below T_tot / L, and the owner of a
// number is the last sequence that starts at or below it.
__host__ __device__ __forceinline__ bool find_body(const SegMap &m, int64_t j, bool reverse, Segment &g) {
    int lo = 0, hi = m.N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (by_length(m, seq_begin(m, mid)) <= j) lo = mid;
        else hi = mid - 1;
    }
    int64_t start, end;
    int base;
    g.n = lo;
    if (!seq_segments(m, lo, start, end, base, g.count)) return false;
    const int64_t i = j - by_length(m, start);
    if (i < 0 || i >= g.count - 1) return false;
    g.s = (int)i + (reverse ? 1 : 0);
    g.slot = state_slot(lo, base - lo, g.s);
    g.t0 = start + (int64_t)g.s * m.L;
    g.t1 = g.t0 + m.L < end ? g.t0 + m.L : end;
    return true;
}

// What a plan is made for: how many blocks run at once, and about what a chunk of
// `tok` tokens costs a block in the main passes and in those that form the segments'
// states, and what a segment costs the scan (microseconds on a B200; only their ratios
// and the 8 us of two further launches matter).
struct Costs {
    int tok, slots;
    double main_us, state_us, scan_us;
};

// Tokens of a segment, for `chains` blocks per sequence.  Equal lengths: the number
// of segments that minimises the waves of both passes (the first over all segments
// but the last).  Lengths that the host does not know: a slot's even share of the
// tokens, which bounds what one long sequence can leave over; sequences below it
// stay whole.  16 x 131,072 tokens: 9 segments 0.66 ms, 37 0.71 ms, unsplit 3.9 ms; 96 x 8,192:
// unsplit 0.25 ms, any split adds a pass over all but the last segment.  Half of
// that share fits one packed batch better and another worse (gradient, 6 documents,
// 16 heads: 678 -> 640 us; 2 documents, 8 heads: 344 -> 450 us).
inline int64_t segment_length(int32_t N, bool equal, int64_t T_tot, int64_t chains, const Costs &c) {
    if (N <= 0 || T_tot <= 0) return kNoSplit;
    if (!equal && N > 1) {
        int64_t L = (T_tot * chains + c.slots - 1) / c.slots;
        if (L < 8 * c.tok) L = 8 * c.tok;
        L = (L + c.tok - 1) / c.tok * c.tok;
        return L >= T_tot ? kNoSplit : L;
    }
    const int64_t len = (T_tot + N - 1) / N, chunks = (len + c.tok - 1) / c.tok;
    auto waves = [&](int64_t blocks) { return (double)((blocks + c.slots - 1) / c.slots); };
    double best = waves(N * chains) * c.main_us * (double)chunks;
    int64_t L = kNoSplit;
    for (int64_t G = 2; G <= 64 && G * 4 <= chunks; ++G) {
        const int64_t per = (chunks + G - 1) / G;
        const double t = (double)per * (waves(N * chains * G) * c.main_us + waves(N * chains * (G - 1)) * c.state_us) +
                         8.0 + (double)(N * chains * G) * c.scan_us;
        if (t < best) {
            best = t;
            L = per * c.tok;
        }
    }
    return L;
}

// The whole of cu_seqlens is checked by one block (every other access relies on
// the bounds of its own sequence alone): a descent between sequences that no
// unit looks at is reported too.
__device__ __forceinline__ void check_seqlens(const SegMap &m) {
    if (m.cu == nullptr) return;
    bool ok = true;
    for (int i = threadIdx.x; i < m.N; i += blockDim.x) ok = ok && m.cu[i] <= m.cu[i + 1];
    if (threadIdx.x == 0) ok = ok && m.cu[0] == 0 && (int64_t)m.cu[m.N] == m.T_tot;
    if (!ok) raise_error(kErrSeqlens);
}

// One log-decay.  Anything below -1e4 forgets everything in every format, and a
// finite stand-in for -inf keeps differences of sums free of inf - inf; NaN stays.
__device__ __forceinline__ float clamp_decay(float g) {
    return g < -1e4f ? -1e4f : g;
}

__device__ __forceinline__ float load_decay(const float *g, int per_token, int64_t t, int h, int H) {
    return clamp_decay(per_token ? g[(size_t)t * H + h] : g[h]);
}

// Inclusive sum over the lanes of a warp, in fp64: sums of up to C log-decays
// are subtracted from one another, and fp32 would leave the differences between
// tokens behind a strong decay with its rounding error.
__device__ __forceinline__ double warp_scan(double x) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// A decay sum as two floats, hi the nearest to the whole: 48 bits, as differences of
// sums behind a strong decay need (fp64 arithmetic would do, at several times the
// latency, where a warp forms the factors that others wait for).
struct Sum2 {
    float hi, lo;
};
__device__ __forceinline__ Sum2 add2(Sum2 a, Sum2 b) {
    const float s = a.hi + b.hi, t = s - a.hi;
    const float e = (a.hi - (s - t)) + (b.hi - t) + (a.lo + b.lo);
    const float r = s + e;
    return {r, e - (r - s)};
}
__device__ __forceinline__ Sum2 minus(Sum2 a) { return {-a.hi, -a.lo}; }
// e^t without the rounding of t
__device__ __forceinline__ float exp_sum(Sum2 t) {
    const float e = expf(t.hi);
    return fmaf(e, t.lo, e);
}

__device__ __forceinline__ void ldmatrix_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// 16 bytes to shared memory, zeros (and nothing read) if not live
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait_all() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// x = hi + mid + lo in bf16 pairs, each the leading 8 bits of what is left: cut,
// not rounded, so that a part costs a byte permute instead of a conversion.  What
// is left over is below 2^-24 of x.
__device__ __forceinline__ float2 cut_bf16(float2 x) {
    return make_float2(__uint_as_float(__float_as_uint(x.x) & 0xffff0000u),
                                 __uint_as_float(__float_as_uint(x.y) & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack_cut(float2 x) {
    return __byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x7632);
}
__device__ __forceinline__ void split3(float2 x, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    const float2 minus = make_float2(-1.f, -1.f);
    hi = pack_cut(x);
    x = sm100::ffma2(cut_bf16(x), minus, x);
    mid = pack_cut(x);
    x = sm100::ffma2(cut_bf16(x), minus, x);
    lo = pack_cut(x);
}

// Scan over the segments of one (sequence, head): on entry ws[slot][h] holds the
// segment's R, on return the state it starts from (forward) or the gradient of
// the state it ends in (reverse).  Elementwise, so bound by memory: one read and
// one write of each R.  grid (elements / 1024, H, scan_blocks): equal sequences one
// each; packed ones the numbers of find_body, of which the first segment's count (a
// sequence of a single segment starts from `init` itself).  A thread owns 4 elements
// and asks for the R of 4 segments at once (of 8, a third of the registers' blocks
// are lost: 96 heads x 3 segments 15.2 -> 18.2 us, 16 x 9 segments 6.6 -> 7.9 us).
constexpr int kScanThreads = 256, kScanAhead = 4;

__host__ __device__ inline int64_t scan_blocks(const SegMap &m) {
    return m.cu == nullptr ? m.N : m.T_tot / m.L;
}

template <bool kReverse>
__global__ void __launch_bounds__(kScanThreads)
segment_scan_kernel(SegMap m, int H, int dd, const float *init, const float *__restrict__ total,
                    float *ws) {
    const int h = blockIdx.y;
    const int e = (blockIdx.x * kScanThreads + threadIdx.x) * 4;
    if (e >= dd) return;
    const ptrdiff_t dir = kReverse ? -1 : 1, step = dir * H * dd, tstep = dir * H;
    const int64_t blocks = scan_blocks(m);
    for (int64_t j = blockIdx.z; j < blocks; j += gridDim.z) {
        Segment g;
        if (m.cu != nullptr) {
            if (!find_body(m, j, false, g) || g.s != 0) continue;
        } else {
            int base;
            g.n = (int)j;
            if (!seq_segments(m, g.n, g.t0, g.t1, base, g.count)) continue;
            g.slot = state_slot(g.n, base - g.n, 0);
        }
        const int first = kReverse ? g.slot + g.count - 1 : g.slot;
        float *p = ws + ((size_t)first * H + h) * dd + e;
        const float *t = total + (size_t)first * H + h;
        float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
        if (init != nullptr) S = *reinterpret_cast<const float4 *>(init + ((size_t)g.n * H + h) * dd + e);
        for (int left = g.count; left > 0; left -= kScanAhead) {
            float4 R[kScanAhead];
            float a[kScanAhead];
#pragma unroll
            for (int i = 0; i < kScanAhead; ++i)       // nothing starts from the last one's end
                if (i + 1 < left) {
                    R[i] = *reinterpret_cast<const float4 *>(p + i * step);
                    a[i] = t[i * tstep];
                }
#pragma unroll
            for (int i = 0; i < kScanAhead; ++i) {
                if (i < left) *reinterpret_cast<float4 *>(p + i * step) = S;
                if (i + 1 < left) {
                    S.x = fmaf(a[i], S.x, R[i].x); S.y = fmaf(a[i], S.y, R[i].y);
                    S.z = fmaf(a[i], S.z, R[i].z); S.w = fmaf(a[i], S.w, R[i].w);
                }
            }
            p += kScanAhead * step;
            t += kScanAhead * tstep;
        }
    }
}

}  // namespace lin
}  // namespace kda
