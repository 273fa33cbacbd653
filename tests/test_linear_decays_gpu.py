"""Strong decays in bf16 at d = 128, whose kernel splits the decay of a chunk into
factors in one of three forms: around one level while the chunk's sums stay within
120, around one for each 32 tokens while those do, else one for each row.  Every input
here says which forms it takes.  Against the fp64 definition, element by element,
with queries that look for the key of the token before (a lost product of the last
token of 32 with the first of the next shows as one lost row, which random queries
hide).  The bounds are derived in linear_testutil."""
import numpy as np
import pytest
import torch

from gated_delta_rule_60_b200 import binding
from linear_testutil import BF16, SUM, close, make, sizes
from oracle import linear_ops as lo
from test_linear_gpu import _check_bwd, _check_fwd, _fwd

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
INF = float("inf")


def _forms(g, lengths):
    """{form: number of (chunk, head)} of log-decays g [T, H] or [H]."""
    T = sum(lengths)
    g = g.double().numpy()
    g = np.maximum(np.broadcast_to(g, (T, g.shape[-1])), -1e4)
    count = {"one": 0, "four": 0, "rows": 0}
    t = 0
    for n in lengths:
        for c in range(0, n, 128):
            x = np.zeros((128, g.shape[1]))
            m = min(128, n - c)
            x[:m] = g[t + c:t + c + m]
            b = x.cumsum(0)
            span = np.ptp(b, 0)
            near = np.ptp(b.reshape(4, 32, -1), 1).max(0)
            count["one"] += int((span <= 120).sum())
            count["four"] += int(((span > 120) & (near <= 120)).sum())
            count["rows"] += int((near > 120).sum())
        t += n
    return count


def _make(lengths, H, *, h0, seed):
    x, cu = make(lengths, 1, H, 128, BF, h0=h0, seed=seed)
    k = x["k"].float()
    q = torch.cat([k[:1], k[:-1]]) + 0.25 * x["q"].float()
    x["q"] = (q / q.norm(dim=-1, keepdim=True)).to(BF)
    return x, cu


CONSTANT = (-0.5, -1.0, -1.5, -2.0, -2.5, -3.0, -3.1, -3.2, -3.3, -3.5, -3.6, -3.8, -3.87, -3.9, -4.0, -20.0)


@pytest.mark.parametrize("h0", [False, True])
@pytest.mark.parametrize("lengths", [[300], [256, 33, 100]])
def test_constant_decays(lengths, h0):
    x, cu = _make(lengths, len(CONSTANT), h0=h0, seed=201)
    x["g"] = torch.tensor(CONSTANT)
    forms = _forms(x["g"], lengths)
    assert min(forms.values()) > 0, forms
    _check_fwd(x, cu)


@pytest.mark.parametrize("h0", [False, True])
@pytest.mark.parametrize("spread", [0.05, 0.3])
def test_decays_of_tokens_around_the_borders(spread, h0):
    x, cu = _make([389], len(CONSTANT), h0=h0, seed=202)
    gen = torch.Generator().manual_seed(5)
    at = torch.tensor(CONSTANT)
    x["g"] = (at * (1.0 + spread * torch.randn(389, len(CONSTANT), generator=gen))).clamp(max=0.0)
    forms = _forms(x["g"], [389])
    assert min(forms.values()) > 0, forms
    _check_fwd(x, cu)


# (token, log-decay) of a chunk, nothing forgotten elsewhere: two drops in neighbouring
# blocks of 32, early in one and late in the next (the levels are then as far apart as
# they get, and every token between the drops still sees all others between them); at
# and behind block ends; one in every block; all that a block may have in one token
DROPS = [
    [(1, -110.0), (63, -110.0)], [(1, -119.0), (63, -119.0)], [(33, -100.0), (95, -100.0)], [(65, -90.0), (127, -90.0)],
    [(31, -119.0), (32, -1.0)], [(32, -119.0), (63, -119.0)], [(0, -119.0), (31, -0.5), (32, -0.5), (63, -118.0)],
    [(15, -119.0), (47, -119.0), (79, -119.0), (111, -119.0)], [(1, -60.0), (31, -59.0), (33, -60.0), (63, -59.0)],
    [(1, -118.0), (63, -118.0), (65, -118.0), (127, -118.0)], [(64, -119.0), (95, -119.0), (96, -119.0), (127, -119.0)],
    [(20, -87.0), (40, -87.0)],
]


@pytest.mark.parametrize("h0", [False, True])
def test_single_drops(h0):
    x, cu = _make([256, 128], len(DROPS), h0=h0, seed=203)
    g = torch.zeros(384, len(DROPS))
    for h, drops in enumerate(DROPS):
        for t, a in drops:
            g[t::128, h] = a
    x["g"] = g
    forms = _forms(g, [256, 128])
    assert forms["rows"] == 0 and forms["four"] >= 2 * len(DROPS), forms
    _check_fwd(x, cu)


def test_forms_across_segments():
    """All forms in sequences that are split, so that the passes over segments, forward
    and in reverse, take them too."""
    T = 2600
    x, cu = _make([T], 4, h0=True, seed=204)
    gen = torch.Generator().manual_seed(6)
    g = torch.empty(T, 4)
    g[:, 0] = -3.5
    g[:, 1] = (-3.2 * (1.0 + 0.3 * torch.randn(T, generator=gen))).clamp(max=0.0)
    g[:, 2] = -1e-3
    g[::37, 2] = -1000.0
    g[5::119, 2] = -INF
    g[:, 3] = -0.01
    g[1::64, 3] = -110.0
    g[62::64, 3] = -100.0
    x["g"] = g
    forms = _forms(g, [T])
    assert min(forms["four"], forms["rows"]) > 8, forms
    states = 4 * 128 * 128 * 4
    assert binding.kda_linear_chunk_fwd_workspace_size(1, T, 4, 128, BF) >= 2 * states
    assert binding.kda_linear_chunk_bwd_workspace_size(1, T, 1, 4, 128, BF) >= 4 * states
    _check_fwd(x, cu)
    _check_bwd(x, cu, plain_decay=False)


def test_constant_decays_across_segments():
    T = 2304
    x, cu = _make([T], 3, h0=False, seed=205)
    x["g"] = torch.tensor([-0.9, -3.5, -1000.0])
    forms = _forms(x["g"], [T])
    assert min(forms.values()) > 8, forms
    _check_fwd(x, cu)
    _check_bwd(x, cu, plain_decay=False)


@pytest.mark.parametrize("size", [1e-11, 1e11])
def test_the_range_of_the_values(size):
    """Values and states of the smallest and largest size that the forms are promised
    for.  The state that queries read is rounded to bf16 behind a factor of e^{-60} at
    least, and bf16 ends in steps of 2^-133: half of one is 2^-134 e^{60} = 5.2e-15 of
    an output for every unit of |q|, of which a query has sqrt(128) at most: 5.9e-14.
    Products end in steps of 2^-149 in fp32: 256 of 1.6e-19 are 4e-17 besides."""
    decays = (-0.3, -0.9, -0.93, -3.0, -3.7, -5.0)
    x, cu = _make([300], len(decays), h0=True, seed=206)
    x["g"] = torch.tensor(decays)
    x["v"] = (x["v"].float() * size).to(BF)
    x["h0"] = x["h0"] * size
    o, hT = _fwd(x, cu)
    ro, rh = lo.linear_forward(x["q"], x["k"], x["v"], x["g"], cu, x["h0"])
    a = sizes(x)
    so, sh = lo.linear_forward(a["q"], a["k"], a["v"], a["g"], cu, a["h0"])
    got = o.double().cpu().numpy()
    assert np.all(np.abs(got - ro) <= SUM * so + BF16 * (np.abs(ro) + so) + 6e-14)
    close(hT, rh, sh, torch.float32, "hT")
