"""The segment numbers and state slots of the linear attention: the functions that its
kernels call, compiled for the host, over packed and equal batches, with the lengths
that the split takes and others, and with malformed bounds; and the workspace that
follows from the slots (CPU)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from gated_delta_rule_60_b200 import binding, build

HERE = os.path.dirname(os.path.abspath(__file__))
I64 = ctypes.POINTER(ctypes.c_int64)


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    build.build()
    out = str(tmp_path_factory.mktemp("segments") / "libsegments.so")
    subprocess.run([build._nvcc(), *build.ARCH, "-O1", "-std=c++17", "-shared", "-Xcompiler", "-fPIC",
                    "-I", build.CSRC, "-o", out, os.path.join(HERE, "linear_segments_driver.cu")], check=True)
    lib = ctypes.CDLL(out)
    i32, i64, f64, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_double, ctypes.c_void_p
    lib.length.restype = lib.slots.restype = i64
    lib.length.argtypes = [i32, i32, i64, i64, i32, i32, f64, f64, f64]
    lib.slots.argtypes = [i64, i64, i64]
    lib.units.argtypes, lib.units.restype = [vp, i32, i64, i64, I64], None
    lib.bodies.argtypes, lib.bodies.restype = [vp, i32, i64, i64, i32, I64], None
    return lib


def _rows(lib, name, cu, N, T, L, *more):
    n = T // L + (N if name == "units" else 0)
    out = np.full((max(n, 1), 6), -1, dtype=np.int64)
    c = None if cu is None else np.asarray(cu, dtype=np.int32)
    getattr(lib, name)(None if c is None else c.ctypes.data, N, T, L, *more, out.ctypes.data_as(I64))
    return [tuple(r) for r in out[:n].tolist()]


def _check(lib, lens, L, equal):
    """All segments once, each with the bounds that it has; every state slot once and
    below the bound that the workspace is made for; the bodies are the segments but the
    last (in reverse, but the first) of each sequence, and a sequence's slots follow
    one another, as the scan takes them."""
    N, T = len(lens), sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    want, split = set(), {}
    for n, ln in enumerate(lens):
        count = max(1, -(-ln // L))
        for s in range(count):
            t = int(cu[n]) + s * L
            want.add((n, s, count, t, min(t + L, int(cu[n + 1]))))
    rows = [r for r in _rows(lib, "units", None if equal else cu, N, T, L) if r[0] >= 0]
    assert len(rows) == len(want) and {r[:3] + r[4:] for r in rows} == want
    slot = {r[:2]: r[3] for r in rows if r[2] > 1}
    bound = lib.slots(T, L, N)
    assert bound == T // L + min(N, T // L)
    assert len(set(slot.values())) == len(slot) and all(0 <= s < bound for s in slot.values())
    for (n, s), at in slot.items():
        assert at == slot[n, 0] + s
    for reverse in (0, 1):
        got = [r for r in _rows(lib, "bodies", None if equal else cu, N, T, L, reverse) if r[0] >= 0]
        assert len(got) == len(set(got))
        assert set(got) == {r for r in rows if r[2] > 1 and (r[1] > 0 if reverse else r[1] < r[2] - 1)}


def _batch(rng, L):
    n = int(rng.integers(1, 40))
    lens = rng.integers(0, 4 * L, n) * rng.integers(0, 2, n) + rng.integers(0, 3, n)
    lens[rng.random(n) < 0.3] = L * int(rng.integers(0, 4))
    lens[rng.random(n) < 0.2] += 1
    return [int(x) for x in lens]


@pytest.mark.parametrize("seed", range(60))
def test_packed_sequences(lib, seed):
    rng = np.random.default_rng(seed)
    L = int(rng.choice([32, 64, 128, 1024, 4096]))
    lens = _batch(rng, L)
    _check(lib, lens, L, False)
    T = sum(lens)
    if T:
        chosen = lib.length(len(lens), 0, T, int(rng.integers(1, 17)), 64, 148, 3.6, 2.1, 0.02)
        _check(lib, lens, chosen, False)


@pytest.mark.parametrize("seed", range(30))
def test_equal_sequences(lib, seed):
    rng = np.random.default_rng(1000 + seed)
    n, ln = int(rng.integers(1, 9)), int(rng.integers(1, 20000))
    L = lib.length(n, 1, n * ln, int(rng.integers(1, 5)), 64, 148, 3.6, 2.1, 0.02)
    assert L % 64 == 0
    _check(lib, [ln] * n, L, True)
    _check(lib, [ln] * n, 128, True)
    _check(lib, [ln] * n, 1 << 31, True)


def test_far_tokens(lib):
    """Token numbers near 2^31."""
    T = 0x7fffffc0
    for lens in ([T], [5, T - 12, 0, 7], [T // 2, T - T // 2]):
        L = lib.length(len(lens), 0, T, 1, 128, 148, 3.6, 2.1, 0.04)
        assert L < T
        _check(lib, lens, L, False)
        _check(lib, lens, 1 << 31, False)


@pytest.mark.parametrize("cu", [[0, 700, 600, 1280], [0, 640, 1000], [50, 640, 1280], [0, 2000, 1280], [0, -40, 1280],
                                [0, 1280, 0, 1280], [0, 2147483647, -2147483648, 1280]])
def test_malformed_bounds_stay_inside(lib, cu):
    T, N = 1280, len(cu) - 1
    for L in (64, 128, 512, 1 << 31):
        found = _rows(lib, "units", cu, N, T, L)
        for reverse in (0, 1):
            found += _rows(lib, "bodies", cu, N, T, L, reverse)
        for n, s, count, slot, t0, t1 in found:
            if n < 0:
                continue
            assert 0 <= n < N and 0 <= s < count and 0 <= t0 <= t1 <= T and t1 - t0 <= L
            assert slot < lib.slots(T, L, N) and (slot >= 0 or count == 1)


def test_workspace_does_not_grow_with_short_sequences(lib):
    """Sequences that are not split need no state in the workspace: what the states of
    many short sequences took (64 KB a head and sequence here) is not asked for."""
    state = 96 * 128 * 128 * 4
    for dt in (torch.bfloat16, torch.float32):
        one = binding.kda_linear_chunk_fwd_workspace_size(1, 1 << 17, 96, 128, dt)
        for N in (2, 256, 4096):
            assert binding.kda_linear_chunk_fwd_workspace_size(N, 1 << 17, 96, 128, dt) <= max(one, 8 * state) + (1 << 20)
        # and what stays of a gradient's: decay terms, two sums for each unit, decay
        # factors of 64 tokens (1.1 KB), all of them small beside a state
        few = binding.kda_linear_chunk_bwd_workspace_size(2, 1 << 17, 96, 96, 128, dt)
        many = binding.kda_linear_chunk_bwd_workspace_size(4096, 1 << 17, 96, 96, 128, dt)
        assert many - few <= 4096 * 96 * (16 + 1200) + 2 * 8 * state


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(torch.bfloat16, 128), (torch.bfloat16, 32), (torch.float32, 64)])
def test_long_sequences_among_many_short_ones(dtype, d):
    """Split sequences whose slots are not their units."""
    from linear_testutil import make
    from test_linear_gpu import _check_bwd, _check_fwd
    lens = [3] * 40 + [1900] + [0, 1, 2] * 9 + [1300, 1] + [5] * 11 + [1030]
    x, cu = make(lens, 1, 1, d, dtype, seed=73)
    _check_fwd(x, cu)
    _check_bwd(x, cu)
