"""A sequence of NaN and infinities among others of a packed batch: everything that
belongs to the others is bit for bit what it is without them (tiles reach behind a
sequence's end into the next one's tokens)."""
import pytest
import torch

from gated_delta_rule_60_b200 import binding
from linear_testutil import cuda, make

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 32), (BF, 16), (FP, 128), (FP, 64), (FP, 16)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_others_do_not_see_it(dtype, d, bad):
    lens = [100, 37, 300, 5, 1, 64, 1300, 20]
    x, cu = make(lens, 1, 2, d, dtype, seed=301)
    clean, dirty, c = cuda(x), cuda(x), cu.cuda()
    out = torch.ones(sum(lens), dtype=torch.bool, device="cuda")
    keep = torch.ones(len(lens), dtype=torch.bool, device="cuda")
    for n in (1, 4, 5):
        rows = slice(int(cu[n]), int(cu[n + 1]))
        out[rows] = False
        keep[n] = False
        for name in ("q", "k", "v", "dO"):
            dirty[name][rows] = bad
        dirty["g"][rows] = bad if bad < 0 else float("nan")
        dirty["h0"][n] = bad
        dirty["dhT"][n] = bad

    def both(z):
        o, hT = binding.kda_linear_chunk_fwd(z["q"], z["k"], z["v"], z["g"], z["h0"], c)
        return o, hT, binding.kda_linear_chunk_bwd(z["q"], z["k"], z["v"], z["g"], z["dO"], z["h0"], c, z["dhT"])

    a, b = both(clean), both(dirty)
    assert torch.equal(a[0][out], b[0][out]) and torch.equal(a[1][keep], b[1][keep])
    for n in ("dq", "dk", "dv", "dg"):
        assert torch.equal(a[2][n][out], b[2][n][out]), n
    assert torch.equal(a[2]["dh0"][keep], b[2]["dh0"][keep])
    assert not torch.isfinite(b[0][~out]).all()
    assert binding.kda_stream_status() == binding.KDA_OK


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (FP, 64)])
def test_split_states_carried_in_place(dtype, d):
    """hT = h0 where long sequences are split and short ones are not."""
    lens = [1900, 3, 0, 1300]
    x, cu = make(lens, 1, 2, d, dtype, seed=302)
    z, c = cuda(x), cu.cuda()
    o, hT = binding.kda_linear_chunk_fwd(z["q"], z["k"], z["v"], z["g"], z["h0"], c)
    S = z["h0"].clone()
    o2, S2 = binding.kda_linear_chunk_fwd(z["q"], z["k"], z["v"], z["g"], S, c, hT=S)
    assert S2.data_ptr() == S.data_ptr() and torch.equal(o, o2) and torch.equal(S, hT)
    S = z["h0"].clone()
    o3, S3 = binding.kda_linear_chunk_fwd(z["q"][:1900], z["k"][:1900], z["v"][:1900], z["g"][:1900], S[:1],
                                          num_seqs=1, hT=S[:1])
    S = z["h0"].clone()[:1]
    o4, S4 = binding.kda_linear_chunk_fwd(z["q"][:1900], z["k"][:1900], z["v"][:1900], z["g"][:1900], S, num_seqs=1)
    assert torch.equal(o3, o4) and torch.equal(S3, S4)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (FP, 64)])
def test_gradient_with_one_of_the_two_states(dtype, d):
    """h0 without dhT and dhT without h0, against a zero state in its place."""
    x, cu = make([700, 0, 90], 1, 2, d, dtype, seed=303)
    z, c = cuda(x), cu.cuda()
    call = lambda h0, dhT: binding.kda_linear_chunk_bwd(z["q"], z["k"], z["v"], z["g"], z["dO"], h0, c, dhT)
    zero = torch.zeros_like(z["h0"])
    for a, b in ((call(z["h0"], None), call(z["h0"], zero)), (call(None, z["dhT"]), call(zero, z["dhT"])),
                 (call(None, None), call(zero, zero))):
        assert all(torch.equal(a[n], b[n]) for n in a)
