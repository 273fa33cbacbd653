"""Host-side refusals of the linear attention, rotary and layer-norm entry
points: bad calls return a status before any launch (the pointers below are
never dereferenced), and the frequency tables (CPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from gated_delta_rule_60_b200 import binding, build

P = ctypes.c_void_p
INV, UNS, WS, OK = (binding.KDA_ERR_INVALID_ARGUMENT, binding.KDA_ERR_UNSUPPORTED,
                    binding.KDA_ERR_WORKSPACE, binding.KDA_OK)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


def _p(x):
    return None if x is None else P(x)


def _fwd(lib, q=256, k=256, v=256, g=256, h0=None, cu=None, N=1, T=64, Hk=2, H=4, d=64, dt=0, tok=1, scale=1.0,
         o=256, hT=None, ws=None, wsb=0):
    return lib.kda_linear_chunk_fwd(_p(q), _p(k), _p(v), _p(g), _p(h0), _p(cu), N, T, Hk, H, d, dt, tok, scale,
                                    _p(o), _p(hT), _p(ws), wsb, None)


def test_prefill_refusals(lib):
    for name in ("q", "k", "v", "o"):
        assert _fwd(lib, **{name: None}) == INV and _fwd(lib, **{name: 264}) == INV, name
    assert _fwd(lib, g=None) == INV and _fwd(lib, g=258) == INV
    assert _fwd(lib, h0=8) == INV and _fwd(lib, hT=8) == INV and _fwd(lib, cu=8) == INV
    assert _fwd(lib, N=-1) == INV and _fwd(lib, T=-1) == INV and _fwd(lib, H=0) == INV and _fwd(lib, Hk=0) == INV
    assert _fwd(lib, Hk=3) == INV and _fwd(lib, H=70000, Hk=1) == INV and _fwd(lib, N=3) == INV
    assert _fwd(lib, d=48) == UNS and _fwd(lib, d=256) == UNS and _fwd(lib, dt=2) == UNS
    assert _fwd(lib, scale=math.inf) == INV and _fwd(lib, scale=math.nan) == INV
    assert _fwd(lib, N=0) == INV and _fwd(lib, N=0, T=0) == OK and _fwd(lib, T=0) == OK
    assert _fwd(lib, N=1 << 30, T=1 << 30) == INV
    assert _fwd(lib, T=(1 << 31) - 1) == UNS
    T, H = 1 << 16, 2
    need = lib.kda_linear_chunk_fwd_workspace_size(1, T, H, 64, 0)
    assert need > 0
    big = dict(T=T, Hk=1, H=H)
    assert _fwd(lib, **big) == WS and _fwd(lib, **big, ws=256, wsb=need - 1) == WS
    assert _fwd(lib, **big, ws=272, wsb=need) == WS
    assert lib.kda_linear_chunk_fwd_workspace_size(1, 64, 2, 128, 0) == 0
    assert lib.kda_linear_chunk_fwd_workspace_size(1, 1 << 16, 2, 48, 0) == 0


def test_decode_refusals(lib):
    def step(q=256, g=256, S=256, o=256, B=2, Hk=2, H=4, d=64, dt=0, scale=1.0):
        return lib.kda_linear_decode_step(_p(q), P(256), P(256), _p(g), _p(S), _p(o), B, Hk, H, d, dt, 1, scale, None)

    assert step(q=None) == INV and step(g=None) == INV and step(S=None) == INV and step(o=258) == INV
    assert step(B=-1) == INV and step(H=0) == INV and step(Hk=3) == INV and step(B=1 << 30) == INV
    assert step(d=24) == UNS and step(dt=9) == UNS and step(scale=math.nan) == INV and step(B=0) == OK


def test_gradient_refusals(lib):
    def bwd(dO=256, dg=256, dq=256, T=64, N=1, Hk=2, d=64, dt=1, dh0=None, ws=256, wsb=1 << 40, tok=1):
        return lib.kda_linear_chunk_bwd(P(256), P(256), P(256), P(256), None, None, N, T, Hk, 4, d, dt, tok, 1.0,
                                        _p(dO), None, _p(dq), P(256), P(256), _p(dg), _p(dh0), _p(ws), wsb, None)

    assert bwd(dO=None) == INV and bwd(dg=None) == INV and bwd(dq=260) == INV and bwd(dh0=4) == INV
    assert bwd(T=0, dg=None, tok=0) == INV and bwd(Hk=3) == INV and bwd(d=8) == UNS and bwd(dt=5) == UNS
    need = lib.kda_linear_chunk_bwd_workspace_size(1, 64, 2, 4, 64, 1)
    assert need > 0 and bwd(ws=None) == WS and bwd(wsb=need - 1) == WS and bwd(ws=384) == WS
    assert bwd(N=0, T=0) == OK
    # shared heads need room for each head's own part
    assert need > lib.kda_linear_chunk_bwd_workspace_size(1, 64, 4, 4, 64, 1)


def test_rotary_refusals(lib):
    def rot(q=256, k=256, f=256, pos=256, cu=None, N=1, T=64, Hq=4, Hk=2, d=64, rot=32, dt=0, scale=1.0, sq=256,
            sk=128, qo=512, ko=512, sqo=256, sko=128):
        return lib.kda_rotary(_p(q), _p(k), _p(f), _p(pos), _p(cu), N, T, Hq, Hk, d, rot, dt, 0, 0, scale, sq, sk,
                              _p(qo), _p(ko), sqo, sko, None)

    assert rot(q=None) == INV and rot(k=None) == INV and rot(f=None) == INV and rot(qo=None) == INV
    assert rot(q=258) == INV and rot(pos=258) == INV and rot(cu=260) == INV
    assert rot(rot=33) == INV and rot(rot=66) == INV and rot(rot=-2) == INV and rot(T=-1) == INV
    assert rot(Hq=0) == INV and rot(Hk=-1) == INV and rot(Hq=70000) == INV and rot(scale=math.inf) == INV
    assert rot(sq=255) == INV and rot(sko=127) == INV
    assert rot(pos=None, N=3) == INV and rot(pos=None, N=0) == INV
    assert rot(q=512, sq=512) == INV                           # in place with another stride
    assert rot(d=2048, sq=1 << 20, sk=1 << 20, sqo=1 << 20, sko=1 << 20) == UNS
    assert rot(d=512, rot=512, sq=1 << 20, sk=1 << 20, sqo=1 << 20, sko=1 << 20) == UNS
    assert rot(dt=3) == UNS and rot(T=1 << 31) == UNS and rot(T=0) == OK


def test_layernorm_refusals(lib):
    def fwd(x=256, y=256, m=256, w=None, T=4, G=1, D=64, dt=0, eps=1e-5):
        return lib.kda_layernorm_fwd(_p(x), _p(w), None, T, G, D, dt, eps, _p(y), _p(m), P(256), None)

    assert fwd(x=None) == INV and fwd(y=None) == INV and fwd(m=None) == INV and fwd(w=8) == INV
    assert fwd(T=-1) == INV and fwd(G=0) == INV and fwd(D=0) == INV and fwd(G=70000) == INV
    assert fwd(eps=-1.0) == INV and fwd(eps=math.nan) == INV and fwd(T=1 << 40) == INV
    assert fwd(D=8193) == UNS and fwd(dt=4) == UNS and fwd(T=0) == OK

    def bwd(dy=256, dx=256, dw=256, ws=256, wsb=1 << 40, T=4, D=64):
        return lib.kda_layernorm_bwd(_p(dy), P(256), P(256), P(256), None, T, 1, D, 0, _p(dx), _p(dw), None,
                                     _p(ws), wsb, None)

    need = lib.kda_layernorm_bwd_workspace_size(4, 1, 64, 0)
    assert need > 0 and bwd(dy=None) == INV and bwd(dx=None) == INV and bwd(dw=4) == INV
    assert bwd(ws=None) == WS and bwd(wsb=need - 1) == WS and bwd(ws=264) == WS and bwd(D=9000) == UNS


def test_frequencies():
    f = lambda *a, **k: binding.kda_rotary_frequencies(*a, device="cpu", **k)
    inv, s = f(64)
    want = 10000.0 ** (-np.arange(32) / 32)
    np.testing.assert_allclose(inv.numpy(), want, rtol=1e-7)
    assert s == 1.0 and inv.dtype == torch.float32
    np.testing.assert_allclose(f(64, 10000.0, binding.KDA_ROPE_LINEAR, 8.0)[0].numpy(), want / 8, rtol=1e-7)
    ntk = f(64, 10000.0, binding.KDA_ROPE_BASE, 8.0)[0].numpy()
    np.testing.assert_allclose([ntk[0], ntk[-1]], [1.0, want[-1] / 8], rtol=1e-6)
    by, s = f(64, 10000.0, binding.KDA_ROPE_PARTS, 8.0, 4096.0)
    turns = 4096 * want / (2 * np.pi)
    assert abs(s - (1 + 0.1 * math.log(8))) < 1e-6
    np.testing.assert_allclose(by.numpy()[turns >= 32], want[turns >= 32], rtol=1e-7)
    np.testing.assert_allclose(by.numpy()[turns <= 1], want[turns <= 1] / 8, rtol=1e-7)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and np.all((by.numpy()[mid] < want[mid]) & (by.numpy()[mid] > want[mid] / 8))
    for bad in (dict(rot=3), dict(rot=0), dict(rot=258), dict(rot=64, base=1.0),
                dict(rot=64, scaling=1, factor=0.5), dict(rot=64, scaling=3, factor=2.0),
                dict(rot=64, scaling=3, factor=2.0, original_length=10.0, beta_fast=1.0, beta_slow=2.0),
                dict(rot=64, scaling=9)):
        with pytest.raises(binding.KdaError):
            f(**bad)


def test_host_tensors_are_refused(lib):
    z, g = torch.zeros(4, 2, 64), torch.zeros(4, 2)
    S = torch.zeros(4, 2, 64, 64)
    for call in (lambda: binding.kda_linear_chunk_fwd(z, z, z, g),
                 lambda: binding.kda_linear_chunk_bwd(z, z, z, g, z),
                 lambda: binding.kda_linear_decode_step(z, z, z, g, S),
                 lambda: binding.kda_rotary(z, None, None, g[:, 0].int()),
                 lambda: binding.kda_layernorm_fwd(z),
                 lambda: binding.kda_layernorm_bwd(z, z, g, g)):
        with pytest.raises(ValueError, match="must be on"):
            call()
