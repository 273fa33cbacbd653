// The linear attention's segment numbers, as its kernels find them, on the host.
#include "kda_linear_common.cuh"

using namespace kda::lin;

namespace {
SegMap make(const int32_t *cu, int N, int64_t T, int64_t L) { return {cu, N, T, L, (int)(T / L + N), (int)(T / N)}; }
void put(int64_t *row, const Segment &g) {
    const int64_t v[6] = {g.n, g.s, g.count, g.count > 1 ? g.slot : -1, g.t0, g.t1};
    for (int i = 0; i < 6; ++i) row[i] = v[i];
}
}  // namespace

extern "C" __attribute__((visibility("default"))) int64_t length(int32_t N, int equal, int64_t T, int64_t chains,
                                                                 int tok, int slots, double main_us,
                                                                 double state_us, double scan_us) {
    return segment_length(N, equal != 0, T, chains, Costs{tok, slots, main_us, state_us, scan_us});
}

extern "C" __attribute__((visibility("default"))) int64_t slots(int64_t T, int64_t L, int64_t N) {
    return state_slots(T, L, N);
}

// rows of (sequence, segment, segments, slot, first token, end), -1 where there is none
extern "C" __attribute__((visibility("default"))) void units(const int32_t *cu, int N, int64_t T, int64_t L,
                                                             int64_t *out) {
    const SegMap m = make(cu, N, T, L);
    for (int u = 0; u < m.units; ++u) {
        Segment g;
        if (find_segment(m, u, g)) put(out + 6 * u, g);
    }
}

extern "C" __attribute__((visibility("default"))) void bodies(const int32_t *cu, int N, int64_t T, int64_t L,
                                                              int reverse, int64_t *out) {
    const SegMap m = make(cu, N, T, L);
    for (int64_t j = 0; j < T / L; ++j) {
        Segment g;
        if (find_body(m, j, reverse != 0, g)) put(out + 6 * j, g);
    }
}
