"""The numbers of segments that the linear attention's blocks turn back into
(sequence, segment) by a binary search, restated here (CPU), and packed batches
whose sequences end at, before and behind the ends of segments (GPU)."""
import numpy as np
import pytest
import torch

BF, FP = torch.bfloat16, torch.float32


def _owner(starts, length, u, step):
    """The last sequence whose first number is at or below u."""
    return max(n for n, s in enumerate(starts) if s // length + step * n <= u)


@pytest.mark.parametrize("seed", range(40))
def test_numbers_of_segments(seed):
    """Every segment has a number of its own that its sequence is found by, below
    T / L + N; and so have the ones whose states are formed, all but one of each
    sequence, below T / L."""
    rng = np.random.default_rng(seed)
    length = int(rng.choice([64, 256, 1024]))
    n = int(rng.integers(1, 30))
    lens = rng.integers(0, 4 * length, n) * rng.integers(0, 2, n) + rng.integers(0, 3, n)
    lens[rng.random(n) < 0.3] = length * int(rng.integers(0, 4))
    starts = np.concatenate([[0], np.cumsum(lens)[:-1]])
    total = int(lens.sum())
    units, bodies = {}, {}
    for i, (s, ln) in enumerate(zip(starts.tolist(), lens.tolist())):
        count = max(1, -(-ln // length))
        for j in range(count):
            u = s // length + i + j
            assert u not in units and u < total // length + n
            assert _owner(starts.tolist(), length, u, 1) == i
            units[u] = (i, j)
        for j in range(count - 1):
            u = s // length + j
            assert u not in bodies and u < total // length
            assert _owner(starts.tolist(), length, u, 0) == i
            bodies[u] = (i, j)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 32), (FP, 64)])
def test_sequences_end_around_segment_ends(dtype, d):
    from test_linear_gpu import _check_bwd, _check_fwd
    from linear_testutil import make
    lens = [1, 1024, 1025, 0, 1023, 512, 2, 513, 1, 256, 511, 1, 0, 1281]
    x, cu = make(lens, 1, 1, d, dtype, seed=71)
    _check_fwd(x, cu)
    _check_bwd(x, cu)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (FP, 32)])
def test_equal_sequences_of_several_segments(dtype, d):
    """Without cu_seqlens, as many sequences as a batch has, each split; the same
    numbers as one sequence at a time, within the bounds of the sums."""
    from gated_delta_rule_60_b200 import binding
    from linear_testutil import cuda, make
    x, cu = make([2304] * 3, 1, 2, d, dtype, seed=72)
    c = cuda(x)
    args = [c[n] for n in ("q", "k", "v", "g")]
    o, hT = binding.kda_linear_chunk_fwd(*args, c["h0"], num_seqs=3)
    got = binding.kda_linear_chunk_bwd(*args, c["dO"], c["h0"], dhT=c["dhT"], num_seqs=3)
    assert binding.kda_stream_status() == binding.KDA_OK
    o2, hT2 = binding.kda_linear_chunk_fwd(*args, c["h0"], cu.cuda())
    got2 = binding.kda_linear_chunk_bwd(*args, c["dO"], c["h0"], cu.cuda(), c["dhT"])
    # two results, each within half a step of bf16 and within 2^-8 of a row's size from
    # the two roundings of the products (fp32: 1e-5 of it)
    rel = 1e-5 if dtype == FP else 4 * 2.0 ** -8
    for a, b in [(o, o2)] + [(got[n], got2[n]) for n in ("dq", "dk", "dv")]:
        assert float((a.double() - b.double()).norm() / b.double().norm()) < rel
    for a, b in [(hT, hT2)] + [(got[n], got2[n]) for n in ("dg", "dh0")]:
        assert float((a.double() - b.double()).norm() / b.double().norm()) < 1e-5
