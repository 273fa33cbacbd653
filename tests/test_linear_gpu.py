"""The decayed linear attention on the GPU against its fp64 definition: prefill,
single tokens, gradient, and a run of them as a model would make it.  The bounds
are derived in linear_testutil."""
import numpy as np
import pytest
import torch

from gated_delta_rule_60_b200 import binding
from guard_bands import guarded, margins_intact
from linear_testutil import close, cuda, decay_sizes, make, near, sizes
from oracle import linear_ops as lo

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32

# lengths, Hk, H, d: one token; around the chunk lengths 32, 64 and 128; empty
# sequences; sequences longer than a segment (256 tokens at these sizes); shared q, k
SHAPES = [
    ([1], 1, 1, 16), ([31, 32, 33], 2, 2, 32), ([0, 5, 0, 64, 1, 0], 1, 3, 64),
    ([127, 128, 129, 63, 65], 2, 4, 128), ([700], 2, 2, 64), ([0, 611, 3, 257, 256], 1, 2, 128),
    ([1], 3, 6, 128), ([1000], 1, 1, 128), ([2] * 40, 1, 2, 16),
]


def _fwd(x, cu, **kw):
    d = cuda(x)
    out = binding.kda_linear_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"], cu.cuda(), **kw)
    assert binding.kda_stream_status() == binding.KDA_OK
    return out


def _check_fwd(x, cu, scale=1.0):
    dt = x["v"].dtype
    o, hT = _fwd(x, cu, scale=scale)
    a = sizes(x)
    ro, rh = lo.linear_forward(x["q"], x["k"], x["v"], x["g"], cu, x["h0"], scale)
    so, sh = lo.linear_forward(a["q"], a["k"], a["v"], a["g"], cu, a["h0"], abs(scale))
    close(o, ro, so, dt, "o")
    close(hT, rh, sh, FP, "hT")


def _check_bwd(x, cu, scale=1.0, plain_decay=True):
    dt = x["v"].dtype
    d = cuda(x)
    got = binding.kda_linear_chunk_bwd(d["q"], d["k"], d["v"], d["g"], d["dO"], d["h0"], cu.cuda(),
                                       d["dhT"], scale=scale)
    assert binding.kda_stream_status() == binding.KDA_OK
    ref = lo.linear_backward(x["q"], x["k"], x["v"], x["g"], x["dO"], cu, x["h0"], x["dhT"], scale)
    size, size_g = decay_sizes(x, cu, abs(scale))
    for n in ("dq", "dk", "dv"):
        close(got[n], ref[n], size[n], dt, n)
    close(got["dh0"], ref["dh0"], size["dh0"], FP, "dh0")
    close(got["dg"], ref["dg"], size_g, FP, "dg")
    if plain_decay:
        near(got["dg"], ref["dg"], 1e-5, "dg")
    return got


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_prefill(i, dtype):
    lengths, Hk, H, d = SHAPES[i]
    x, cu = make(lengths, Hk, H, d, dtype, const=i % 3 == 1, h0=i % 2 == 0, seed=i)
    _check_fwd(x, cu, 1.0 if i % 2 else d ** -0.5)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_gradient(i, dtype):
    lengths, Hk, H, d = SHAPES[i]
    x, cu = make(lengths, Hk, H, d, dtype, const=i % 3 == 1, h0=i % 2 == 0, seed=100 + i)
    _check_bwd(x, cu, 1.0 if i % 2 else d ** -0.5)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 32), (BF, 16), (FP, 128), (FP, 32)])
def test_sequences_of_several_segments(dtype, d):
    """Long enough to be split on every path (256 to 1,024 tokens a segment at
    these sizes), packed with short and empty ones, and alone."""
    x, cu = make([1300, 0, 70, 2100], 1, 2, d, dtype, seed=d)
    _check_fwd(x, cu)
    _check_bwd(x, cu)
    x, cu = make([2700], 1, 1, d, dtype, h0=False, seed=d + 1)
    _check_fwd(x, cu)
    _check_bwd(x, cu)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (FP, 64), (BF, 32)])
def test_extreme_decays(dtype, d):
    """Forgetting at once (-inf), decays far below any format's range, none at
    all, and mixes of them within a chunk and across segments."""
    x, cu = make([300, 40], 1, 4, d, dtype, seed=7)
    g = x["g"]
    g[:, 0] = 0.0
    g[:, 1] = -1000.0
    g[::7, 2] = -float("inf")
    g[::5, 3] = -88.0
    g[130, :] = -float("inf")
    _check_fwd(x, cu)
    _check_bwd(x, cu, plain_decay=False)


def test_slow_decay_over_many_segments():
    x, cu = make([5000], 1, 1, 128, BF, seed=8, rate=1e-4)
    _check_fwd(x, cu)
    x, cu = make([2000], 1, 1, 128, BF, seed=9, rate=1e-4)
    _check_bwd(x, cu)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (FP, 128), (BF, 64)])
def test_states_carry_in_place_and_gradient_is_optional(dtype, d):
    """Two halves with the state carried in place give the whole; without hT and
    without h0 nothing else changes."""
    x, cu = make([600], 1, 2, d, dtype, h0=False, seed=11)
    o, hT = _fwd(x, cu)
    half = lambda s: {n: None if t is None else t[s].contiguous() for n, t in x.items()}
    a, b = cuda(half(slice(0, 333))), cuda(half(slice(333, 600)))
    S = torch.zeros_like(hT)
    o1, S1 = binding.kda_linear_chunk_fwd(a["q"], a["k"], a["v"], a["g"], S, hT=S)
    o2, S2 = binding.kda_linear_chunk_fwd(b["q"], b["k"], b["v"], b["g"], S, hT=S)
    assert S1.data_ptr() == S2.data_ptr() == S.data_ptr()
    size = lo.linear_forward(x["q"].abs(), x["k"].abs(), x["v"].abs(), x["g"], cu)
    close(torch.cat([o1, o2]), o.double().cpu().numpy(), 2 * size[0], dtype, "o")
    close(S, hT.double().cpu().numpy(), 2 * size[1], FP, "hT")
    o3, none = _fwd(x, cu, output_final_state=False)
    assert none is None and torch.equal(o3, o)


@pytest.mark.parametrize("dtype,d,Hk,H,B", [(BF, 128, 2, 6, 5), (FP, 64, 3, 3, 3), (BF, 32, 1, 2, 9),
                                            (FP, 16, 1, 1, 1), (FP, 128, 1, 4, 2), (BF, 64, 4, 8, 7)])
def test_single_tokens_follow_the_prefill(dtype, d, Hk, H, B):
    """Eight tokens one at a time, against the definition, within guard bands."""
    n = 8
    x, cu = make([n] * B, Hk, H, d, dtype, const=B == 9, seed=B)
    buf, S = guarded((B, H, d, d), FP, 7.0, "cuda")
    S.copy_(x["h0"])
    obuf, o = guarded((B, H, d), dtype, 3.0, "cuda")
    dx = cuda(x)
    at = lambda t, i: t.view(B, n, *t.shape[1:])[:, i].contiguous()
    ro, rh = lo.linear_forward(x["q"], x["k"], x["v"], x["g"], cu, x["h0"], 0.5)
    a = sizes(x)
    so, sh = lo.linear_forward(a["q"], a["k"], a["v"], a["g"], cu, a["h0"], 0.5)
    for i in range(n):
        g = dx["g"] if dx["g"].dim() == 1 else at(dx["g"], i)
        got = binding.kda_linear_decode_step(at(dx["q"], i), at(dx["k"], i), at(dx["v"], i), g, S,
                                             scale=0.5, o=o)
        rows = slice(i, None, n)
        close(got, ro[rows], so[rows], dtype, i)
    close(S, rh, sh, FP, "S")
    assert margins_intact(buf, 7.0) and margins_intact(obuf, 3.0)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (FP, 64)])
def test_nothing_outside_the_outputs_is_written(dtype, d):
    lengths = [300, 0, 33, 129]
    x, cu = make(lengths, 1, 2, d, dtype, seed=21)
    T, N = sum(lengths), len(lengths)
    ob, o = guarded((T, 2, d), dtype, 3.0, "cuda")
    hb, hT = guarded((N, 2, d, d), FP, 7.0, "cuda")
    need = binding.kda_linear_chunk_fwd_workspace_size(N, T, 2, d, dtype)
    ws = torch.full((need + 512,), 5, dtype=torch.uint8, device="cuda")
    off = (-ws.data_ptr()) % 256
    _fwd(x, cu, o=o, hT=hT, workspace=ws[off:off + need])
    assert margins_intact(ob, 3.0) and margins_intact(hb, 7.0)
    assert bool((ws[off + need:] == 5).all()) and bool((ws[:off] == 5).all())
    ref = _fwd(x, cu)
    assert torch.equal(ref[0], o) and torch.equal(ref[1], hT)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (FP, 32)])
def test_packing_and_repetition_change_nothing(dtype, d):
    """Equal lengths with and without cu_seqlens, the same call twice."""
    x, cu = make([96] * 4, 2, 2, d, dtype, seed=31)
    o, hT = _fwd(x, cu)
    dx = cuda(x)
    o2, h2 = binding.kda_linear_chunk_fwd(dx["q"], dx["k"], dx["v"], dx["g"], dx["h0"], num_seqs=4)
    o3, h3 = _fwd(x, cu)
    assert torch.equal(o, o3) and torch.equal(hT, h3)
    assert torch.equal(o, o2) and torch.equal(hT, h2)
    call = lambda: binding.kda_linear_chunk_bwd(dx["q"], dx["k"], dx["v"], dx["g"], dx["dO"], dx["h0"],
                                                cu.cuda(), dx["dhT"])
    a, b = call(), call()
    assert all(torch.equal(a[n], b[n]) for n in a)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (FP, 64)])
def test_streams_and_graphs(dtype, d):
    """On another stream, two streams at once, and two captured graphs that are
    replayed with new inputs in the same buffers."""
    x, cu = make([400, 77], 1, 2, d, dtype, seed=41)
    y, _ = make([400, 77], 1, 2, d, dtype, seed=42)
    want = [[*_fwd(z, cu)] for z in (x, y)]
    dx, dy, dcu = cuda(x), cuda(y), cu.cuda()
    grad = lambda z: binding.kda_linear_chunk_bwd(z["q"], z["k"], z["v"], z["g"], z["dO"], z["h0"], dcu,
                                                  z["dhT"])
    wantg = [grad(dx), grad(dy)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [binding.kda_linear_chunk_fwd(z["q"], z["k"], z["v"], z["g"], z["h0"], dcu, stream=s)
           for z, s in zip((dx, dy), streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    bufs = cuda(x)
    side = torch.cuda.Stream()
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for f in (lambda: binding.kda_linear_chunk_fwd(bufs["q"], bufs["k"], bufs["v"], bufs["g"],
                                                       bufs["h0"], dcu),
                  lambda: grad(bufs)):
            f()
            side.synchronize()
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=side):
                outs.append(f())
            graphs.append(gr)
    torch.cuda.synchronize()
    for z, w, wg in ((dy, want[1], wantg[1]), (dx, want[0], wantg[0])):
        for n, t in bufs.items():
            t.copy_(z[n])
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0][0], w[0]) and torch.equal(outs[0][1], w[1])
        assert all(torch.equal(outs[1][n], wg[n]) for n in wg)


def test_malformed_sequences_are_reported():
    x, _ = make([64, 64], 1, 2, 128, BF, seed=51)
    dx = cuda(x)
    for cu in ([0, 70, 60, 128], [0, 64, 100], [5, 64, 128], [0, 200, 128], [0, -4, 128]):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        binding.kda_linear_chunk_fwd(dx["q"], dx["k"], dx["v"], dx["g"], None, c)
        assert binding.kda_stream_status() == binding.KDA_ERR_BAD_SEQLENS, cu
        binding.kda_linear_chunk_bwd(dx["q"], dx["k"], dx["v"], dx["g"], dx["dO"], None, c)
        assert binding.kda_stream_status() == binding.KDA_ERR_BAD_SEQLENS, cu
    assert binding.kda_stream_status() == binding.KDA_OK


def test_no_tokens():
    z = torch.zeros(0, 2, 64, device="cuda", dtype=BF)
    g = torch.zeros(0, 2, device="cuda")
    h0 = torch.randn(3, 2, 64, 64, device="cuda")
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    o, hT = binding.kda_linear_chunk_fwd(z, z, z, g, h0, cu)
    assert o.shape == (0, 2, 64) and torch.equal(hT, h0)
    got = binding.kda_linear_chunk_bwd(z, z, z, g, z, h0, cu, h0)
    assert torch.equal(got["dh0"], h0)
    got = binding.kda_linear_chunk_bwd(z, z, z, g[:0, 0].new_zeros(2) - 1, z, h0, cu)
    assert bool((got["dg"] == 0).all()) and bool((got["dh0"] == 0).all())
    assert binding.kda_stream_status() == binding.KDA_OK


def test_gradient_against_differences():
    """<gradient, direction> against a central difference of the GPU's own
    forward in fp32.  L is linear in q, in k, in v and in h0, so a wide step has
    no truncation error there; in g the step of 2^-11 leaves (2^-11 |z|)^2 / 6.
    L is a sum of 4e4 terms of size 1 whose roundings (about 1e-6 each, of
    random sign) leave 2e-4, over a step of 2^-10 at least: 0.2, against
    gradients along z whose terms' root sum square is 30 and more."""
    x, cu = make([150, 60], 1, 2, 64, FP, seed=61)
    dx, dcu = cuda(x), cu.cuda()
    got = binding.kda_linear_chunk_bwd(dx["q"], dx["k"], dx["v"], dx["g"], dx["dO"], dx["h0"], dcu, dx["dhT"])

    def loss(y):
        o, hT = binding.kda_linear_chunk_fwd(y["q"], y["k"], y["v"], y["g"], y["h0"], dcu)
        return float((o.double() * dx["dO"].double()).sum() + (hT.double() * dx["dhT"].double()).sum())

    gen = torch.Generator(device="cuda").manual_seed(1)
    for n in ("q", "k", "v", "g", "h0"):
        z = torch.randn(dx[n].shape, generator=gen, device="cuda")
        e = 2.0 ** -8 if n in ("q", "k", "g") else 2.0 ** -4
        e /= 8 if n == "g" else 1
        num = (loss({**dx, n: dx[n] + e * z}) - loss({**dx, n: dx[n] - e * z})) / (2 * e)
        dot = float((got["d" + n].double() * z.double()).sum())
        size = float((got["d" + n].double() * z.double()).square().sum().sqrt())
        assert abs(num - dot) <= 2e-2 * max(size, abs(dot)), (n, num, dot, size)


def test_layer_of_the_operators_together():
    """Rotary positions, a prompt, its norm, then tokens one by one from the
    carried state: the same as the whole sequence at once, and the gradient
    back through all of it against the definitions."""
    T, H, d, extra = 150, 3, 64, 5
    gen = torch.Generator().manual_seed(3)
    randn = lambda *s: torch.randn(*s, generator=gen)
    L = T + extra
    q, k, v = (randn(L, H, d) * d ** -0.25 for _ in range(3))
    g, w, b, dy = -0.1 * randn(L, H).abs(), 1 + 0.1 * randn(H, d), 0.1 * randn(H, d), randn(L, H, d)
    inv, sc = binding.kda_rotary_frequencies(32, 10000.0, binding.KDA_ROPE_PARTS, 4.0, 64.0, device="cpu")
    pos = np.arange(L)
    rq, rk = (lo.rotary(t, inv, pos, True, scale=sc) for t in (q, k))
    ro, _ = lo.linear_forward(rq, rk, v, g, [0, L])
    ry, _, _ = lo.layernorm(ro, w, b)
    c = lambda t: t.cuda().contiguous()
    p = torch.arange(L, dtype=torch.int32, device="cuda")
    gq, gk = binding.kda_rotary(c(q), c(k), c(inv), p, interleaved=True, scale=sc)
    o1, S = binding.kda_linear_chunk_fwd(gq[:T].contiguous(), gk[:T].contiguous(), c(v)[:T].contiguous(),
                                         c(g)[:T].contiguous())
    outs = [o1]
    for t in range(T, L):
        outs.append(binding.kda_linear_decode_step(*(z[t:t + 1].contiguous() for z in (gq, gk, c(v), c(g))), S))
    o = torch.cat(outs)
    y, mean, rstd = binding.kda_layernorm_fwd(o, c(w), c(b))
    near(o, ro, 1e-5, "o")
    near(y, ry, 1e-5, "y")
    n = binding.kda_layernorm_bwd(c(dy), o, mean, rstd, c(w), bias=True)
    a = binding.kda_linear_chunk_bwd(gq, gk, c(v), c(g), n["dx"])
    dq, dk = binding.kda_rotary(a["dq"], a["dk"], c(inv), p, interleaved=True, inverse=True, scale=sc)
    rn = lo.layernorm_backward(dy, ro, w, groups=H)
    ra = lo.linear_backward(rq, rk, v, g, rn["dx"], [0, L])
    for got, ref, name in ((n["dweight"], rn["dweight"], "dw"), (n["dbias"], rn["dbias"], "db"),
                           (a["dv"], ra["dv"], "dv"), (a["dg"], ra["dg"], "dg"),
                           (dq, lo.rotary(ra["dq"], inv, pos, True, True, sc), "dq"),
                           (dk, lo.rotary(ra["dk"], inv, pos, True, True, sc), "dk")):
        near(got, ref, 1e-4, name)
    assert binding.kda_stream_status() == binding.KDA_OK
