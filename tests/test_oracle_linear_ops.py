"""The fp64 definitions of the linear attention, rotary positions and layer norm
(oracle/linear_ops.py) against closed forms and central differences (CPU)."""
import numpy as np
import pytest

from oracle import linear_ops as lo


def _case(lengths, Hk, H, d, const=False, seed=0):
    r = np.random.RandomState(seed)
    T, N = sum(lengths), len(lengths)
    cu = np.concatenate([[0], np.cumsum(lengths)])
    x = dict(q=r.randn(T, Hk, d), k=r.randn(T, Hk, d), v=r.randn(T, H, d),
             g=-np.abs(r.randn(H)) if const else -np.abs(r.randn(T, H)), h0=r.randn(N, H, d, d))
    return x, cu, r.randn(T, H, d), r.randn(N, H, d, d)


def test_quadratic_form():
    x, cu, _, _ = _case([5, 0, 3], 1, 2, 4)
    o, hT = lo.linear_forward(x["q"], x["k"], x["v"], x["g"], cu, x["h0"], 0.5)
    for n in range(3):
        for h in range(2):
            b = np.cumsum(x["g"][cu[n]:cu[n + 1], h])
            for i, t in enumerate(range(cu[n], cu[n + 1])):
                y = np.exp(b[i]) * x["q"][t, 0] @ x["h0"][n, h]
                for j, s in enumerate(range(cu[n], t + 1)):
                    y = y + np.exp(b[i] - b[j]) * (x["q"][t, 0] @ x["k"][s, 0]) * x["v"][s, h]
                np.testing.assert_allclose(o[t, h], 0.5 * y, rtol=1e-12, atol=1e-12)
    np.testing.assert_array_equal(hT[1], x["h0"][1])


def test_forgetting_and_no_decay():
    x, cu, _, _ = _case([6], 1, 1, 3)
    g = np.zeros((6, 1))
    _, hT = lo.linear_forward(x["q"], x["k"], x["v"], g, cu)
    np.testing.assert_allclose(hT[0, 0], x["k"][:, 0].T @ x["v"][:, 0], rtol=1e-12)
    g[4] = -np.inf
    _, hT = lo.linear_forward(x["q"], x["k"], x["v"], g, cu, x["h0"])
    np.testing.assert_allclose(hT[0, 0], x["k"][4:, 0].T @ x["v"][4:, 0], rtol=1e-12)


@pytest.mark.parametrize("const", [False, True])
def test_gradient_against_differences(const):
    x, cu, dO, dhT = _case([4, 0, 3], 2, 4, 3, const)
    loss = lambda y: sum((a * b).sum() for a, b in zip(
        lo.linear_forward(y["q"], y["k"], y["v"], y["g"], cu, y["h0"], 0.7), (dO, dhT)))
    got = lo.linear_backward(x["q"], x["k"], x["v"], x["g"], dO, cu, x["h0"], dhT, 0.7)
    r = np.random.RandomState(5)
    for name in ("q", "k", "v", "g", "h0"):
        z = r.randn(*x[name].shape)
        e = 1e-6
        d = (loss({**x, name: x[name] + e * z}) - loss({**x, name: x[name] - e * z})) / (2 * e)
        assert abs(d - (got["d" + name] * z).sum()) <= 1e-7 * max(1.0, abs(d)), name


@pytest.mark.parametrize("pairs", [False, True])
def test_rotary(pairs):
    r = np.random.RandomState(1)
    x, f = r.randn(5, 2, 10), r.rand(3)
    pos = np.array([0, 1, 7, 100000, -3])
    y = lo.rotary(x, f, pos, pairs, scale=1.5)
    np.testing.assert_allclose(y[0, :, :6], 1.5 * x[0, :, :6])
    np.testing.assert_array_equal(y[..., 6:], x[..., 6:])
    i, j = (2, 3) if pairs else (1, 4)
    c, s = np.cos(7 * f[1]), np.sin(7 * f[1])
    np.testing.assert_allclose(y[2, 1, i], 1.5 * (x[2, 1, i] * c - x[2, 1, j] * s))
    np.testing.assert_allclose(y[2, 1, j], 1.5 * (x[2, 1, i] * s + x[2, 1, j] * c))
    z = lo.rotary(y, f, pos, pairs, inverse=True, scale=1 / 1.5)
    np.testing.assert_allclose(z, x, rtol=1e-12)
    np.testing.assert_array_equal(lo.sequence_positions([0, 2, 2, 5]), [0, 1, 0, 1, 2])


def test_layernorm_gradient_against_differences():
    r = np.random.RandomState(2)
    x, w, b, dy = r.randn(6, 3, 7) + 2, r.randn(3, 7), r.randn(3, 7), r.randn(6, 3, 7)
    y, m, _ = lo.layernorm(x)
    np.testing.assert_allclose(y.mean(-1), 0, atol=1e-12)
    np.testing.assert_allclose((y ** 2).mean(-1), 1, atol=1e-4)
    got = lo.layernorm_backward(dy, x, w, groups=3)
    loss = lambda x, w, b: (lo.layernorm(x, w, b)[0] * dy).sum()
    for i, name in enumerate(("dx", "dweight", "dbias")):
        at = [x, w, b]
        z = r.randn(*at[i].shape)
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + 1e-6 * z, at[i] - 1e-6 * z
        d = (loss(*up) - loss(*down)) / 2e-6
        assert abs(d - (got[name] * z).sum()) <= 1e-6 * max(1.0, abs(d)), name
