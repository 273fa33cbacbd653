"""Rotary positions and layer norm on the GPU against their fp64 definitions.

Bounds.  One rounding to the storage type: 2^-8 (bf16) or 2^-24 (fp32) of the
value.  Rotary in fp32: cos and sin are off by 2e-7 (the angle) plus two
roundings, so 5e-7 of |x| + |y| of the pair.  Layer norm: sums of D fp32 terms
are off by D 2^-24 of the terms' sizes at most; the trees here are at most 16 +
9 + 16 additions deep, so 41 2^-24 = 2.5e-6, and y, dx are a few such values."""
import numpy as np
import pytest
import torch

from gated_delta_rule_60_b200 import binding
from oracle import linear_ops as lo

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float32


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def _rotary_close(got, x, ref, dtype, scale, rot):
    got, x = got.double().cpu().numpy(), lo._f64(x)
    size = np.sqrt((x ** 2).sum(-1, keepdims=True)) * scale
    assert np.all(np.abs(got - ref) <= _half(dtype) * np.abs(ref) * (1 + 1e-6) + 1e-6 * size + 1e-30)
    assert np.array_equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,d,rot", [(1, 1, 1, 2, 2), (3, 2, 1, 64, 64), (70, 5, 2, 80, 34),
                                           (33, 96, 96, 128, 128), (129, 4, 0, 128, 64),
                                           (600, 1, 1, 256, 256), (17, 3, 3, 7, 6), (9, 2, 2, 128, 0),
                                           (5, 2, 1, 1024, 160)])
def test_rotary(T, Hq, Hk, d, rot, pairs, dtype):
    gen = torch.Generator().manual_seed(T + d)
    q, k = torch.randn(T, Hq, d, generator=gen).to(dtype), torch.randn(T, max(Hk, 1), d, generator=gen).to(dtype)
    inv = torch.rand(rot // 2, generator=gen) ** 4
    pos = torch.randint(-5, 1 << 20, (T,), generator=gen).to(torch.int32)
    pos[0] = 2147483647
    dev = (lambda t: t.cuda())
    for inverse in (False, True):
        a, b = binding.kda_rotary(dev(q), dev(k) if Hk else None, dev(inv) if rot else None, dev(pos),
                                  interleaved=pairs, inverse=inverse, scale=1.25)
        _rotary_close(a, q, lo.rotary(q, inv, pos, pairs, inverse, 1.25), dtype, 1.25, rot)
        if Hk:
            _rotary_close(b, k, lo.rotary(k, inv, pos, pairs, inverse, 1.25), dtype, 1.25, rot)
        else:
            assert b is None


@pytest.mark.parametrize("dtype", [BF, FP])
def test_rotary_of_slices_in_place_and_by_sequence(dtype):
    """q and k as slices of one projection (aligned, and by an odd offset),
    turned in place; v between the tokens stays; positions from cu_seqlens."""
    for width, off in ((5 * 64 + 64, 0), (5 * 64 + 65, 0), (5 * 64 + 72, 8)):
        gen = torch.Generator().manual_seed(width)
        p = torch.randn(50, width, generator=gen).to(dtype).cuda()
        keep = p.clone()
        q = p[:, off:off + 192].unflatten(1, (3, 64))
        k = p[:, off + 192:off + 320].unflatten(1, (2, 64))
        cu = torch.tensor([0, 7, 7, 50], dtype=torch.int32)
        inv, _ = binding.kda_rotary_frequencies(48)
        want_q = lo.rotary(q.cpu(), inv.cpu(), lo.sequence_positions(cu))
        q0, k0 = q.cpu().clone(), k.cpu().clone()
        want_k = lo.rotary(k0, inv.cpu(), lo.sequence_positions(cu))
        a, b = binding.kda_rotary(q, k, inv, None, cu.cuda(), q_out=q, k_out=k)
        assert a.data_ptr() == q.data_ptr() and b.data_ptr() == k.data_ptr()
        _rotary_close(a, q0, want_q, dtype, 1.0, 48)
        _rotary_close(b, k0, want_k, dtype, 1.0, 48)
        assert torch.equal(p[:, off + 320:], keep[:, off + 320:]) and torch.equal(p[:, :off], keep[:, :off])
        back, _ = binding.kda_rotary(q[:49], None, inv, num_seqs=7)
        _rotary_close(back, q[:49].cpu(), lo.rotary(q[:49].cpu(), inv.cpu(), np.arange(49) % 7), dtype, 1.0, 48)
    assert binding.kda_stream_status() == binding.KDA_OK
    binding.kda_rotary(q, None, inv, None, torch.tensor([0, 60, 50], dtype=torch.int32).cuda())
    assert binding.kda_stream_status() == binding.KDA_ERR_BAD_SEQLENS


def _norm_case(shape, w_shape, dtype, bias, seed):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(*shape, generator=gen) * 2 + 3).to(dtype)
    dy = torch.randn(*shape, generator=gen).to(dtype)
    w = 1 + 0.3 * torch.randn(*w_shape, generator=gen)
    return x, dy, w, torch.randn(*w_shape, generator=gen) if bias else None


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("shape,groups", [((1, 1), 0), ((3, 2), 0), ((2, 7, 8), 0), ((5, 3, 16), 3),
                                          ((130, 4, 128), 4), ((33, 96, 64), 96), ((700, 100), 0),
                                          ((9, 1000), 0), ((4, 1001), 0), ((6, 5000), 0), ((2, 8192), 0),
                                          ((3, 8191), 0), ((4000, 32), 0), ((40, 5, 2050), 5), ((2500, 512), 0)])
def test_layernorm(shape, groups, dtype):
    bias = shape[0] % 2 == 0
    w_shape = shape[-2:] if groups else shape[-1:]
    x, dy, w, b = _norm_case(shape, w_shape, dtype, bias, sum(shape))
    dev = (lambda t: None if t is None else t.cuda())
    y, mean, rstd = binding.kda_layernorm_fwd(dev(x), dev(w), dev(b), eps=1e-5)
    ry, rm, rr = lo.layernorm(x, w, b)
    f = (lambda t: t.double().cpu().numpy())
    eps = 41 * 2.0 ** -24
    mag = np.abs(lo._f64(x)).max(-1)
    assert np.all(np.abs(f(mean) - rm) <= eps * mag + 1e-30)
    # the mean's error shifts every centred value: relative to the deviation 1 / rstd
    assert np.all(np.abs(f(rstd) - rr) <= rr * (4 * eps + eps * mag * rr) + 1e-30)
    # x - mean is off by the mean's error, times rstd and the weight
    span = 1 + np.abs(ry) + (mag * rr)[..., None] * np.abs(w.double().numpy())
    assert np.all(np.abs(f(y) - ry) <= _half(dtype) * np.abs(ry) + 4 * eps * span)
    got = binding.kda_layernorm_bwd(dev(dy), dev(x), mean, rstd, dev(w), bias=bias)
    ref = lo.layernorm_backward(dy, x, w, groups=groups)
    xh = np.abs((lo._f64(x) - rm[..., None]) * rr[..., None])
    u = np.abs(lo._f64(dy) * w.double().numpy())
    exh = 4 * eps * (1 + xh + (mag * rr)[..., None])                 # error of xh
    big = rr[..., None] * (u + u.mean(-1, keepdims=True) + xh * (u * xh).mean(-1, keepdims=True))
    err = rr[..., None] * (exh * (u * xh).mean(-1, keepdims=True) + xh * (u * exh).mean(-1, keepdims=True))
    assert np.all(np.abs(f(got["dx"]) - ref["dx"]) <= _half(dtype) * np.abs(ref["dx"]) + 8 * eps * big + err + 1e-30)
    g = (-1, groups, shape[-1]) if groups else (-1, shape[-1])
    rows = int(np.prod(shape)) // int(np.prod(w_shape))
    deep = (rows + 41) * 2.0 ** -24                                  # a sum of `rows` terms, in any order
    ady = np.abs(lo._f64(dy))
    size = ((ady * xh).reshape(g).sum(0), ady.reshape(g).sum(0))
    slip = (ady * exh).reshape(g).sum(0)
    assert np.all(np.abs(f(got["dweight"]) - ref["dweight"]) <= deep * size[0] + slip + 1e-30)
    if bias:
        assert np.all(np.abs(f(got["dbias"]) - ref["dbias"]) <= deep * size[1] + 1e-30)
    else:
        assert "dbias" not in got
    again = binding.kda_layernorm_bwd(dev(dy), dev(x), mean, rstd, dev(w), bias=bias)
    assert all(torch.equal(again[n], got[n]) for n in got)
    assert binding.kda_stream_status() == binding.KDA_OK


def test_layernorm_variants():
    """No weight, no bias, in place, constant rows, no rows, large offsets."""
    x, dy, w, b = _norm_case((50, 256), (256,), FP, True, 5)
    X, DY = x.cuda(), dy.cuda()
    y, m, r = binding.kda_layernorm_fwd(X)
    assert np.abs(y.double().cpu().numpy() - lo.layernorm(x)[0]).max() <= 1e-5
    yb, _, _ = binding.kda_layernorm_fwd(X, None, b.cuda())
    assert np.abs(yb.double().cpu().numpy() - lo.layernorm(x, None, b)[0]).max() <= 1e-5
    got = binding.kda_layernorm_bwd(DY, X, m, r)
    assert set(got) == {"dx"}
    got2 = binding.kda_layernorm_bwd(DY, X, m, r, bias=True)
    assert torch.equal(got2["dx"], got["dx"]) and got2["dbias"].shape == (256,)
    Z = X.clone()
    out, _, _ = binding.kda_layernorm_fwd(Z, y=Z)
    assert out.data_ptr() == Z.data_ptr() and torch.equal(Z, y)
    D = DY.clone()
    binding.kda_layernorm_bwd(D, X, m, r, dx=D)
    assert torch.equal(D, got["dx"])
    flat = torch.full((4, 64), 3.0, device="cuda")
    y, m, r = binding.kda_layernorm_fwd(flat)
    assert bool((y == 0).all()) and bool((m == 3).all())
    none = torch.zeros(0, 3, 64, device="cuda")
    wz = torch.ones(3, 64, device="cuda")
    y, m, r = binding.kda_layernorm_fwd(none, wz)
    got = binding.kda_layernorm_bwd(none, none, m, r, wz, bias=True)
    assert got["dx"].shape == (0, 3, 64) and bool((got["dweight"] == 0).all()) and bool((got["dbias"] == 0).all())
    far = torch.randn(8, 512, device="cuda") + 1000.0
    y, _, _ = binding.kda_layernorm_fwd(far)
    # x - mean is exact to a rounding of x (2^-24 1000) and the mean's (41 2^-24 1000)
    assert np.abs(y.double().cpu().numpy() - lo.layernorm(far)[0]).max() <= 42 * 2.0 ** -24 * 1004 * 1.2


def test_rotary_and_norm_on_a_stream_and_in_a_graph():
    gen = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(64, 4, 128, device="cuda", generator=gen).to(BF)
    w = torch.randn(4, 128, device="cuda", generator=gen)
    inv, _ = binding.kda_rotary_frequencies(128)
    pos = torch.arange(64, dtype=torch.int32, device="cuda")

    def both(stream=None):
        a, _ = binding.kda_rotary(q, None, inv, pos, stream=stream)
        y, m, r = binding.kda_layernorm_fwd(a, w, stream=stream)
        return y, binding.kda_layernorm_bwd(q, a, m, r, w, bias=True, stream=stream)

    y, g = both()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    y2, g2 = both(s)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(g[n], g2[n]) for n in g)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        y3, g3 = both()
    q.add_(1.0)
    gr.replay()
    y4, g4 = both()
    torch.cuda.synchronize()
    assert torch.equal(y3, y4) and all(torch.equal(g3[n], g4[n]) for n in g3)
