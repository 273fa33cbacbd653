"""Inputs and bounds for the tests of the decayed linear attention.

Bounds.  A rounding to bf16 is off by at most 2^-8 of the value.  The bf16 path
rounds once the operands that carry a decay (the products inside a chunk, the
state that the queries read) and once the result, so every term of an output is
off by at most 2^-8 of its size: |x - ref| <= 2^-8 |ref| + 2^-8 A, with A the
same sums of the terms' sizes (the definition on absolute values).  Sums of up
to 128 + 128 fp32 terms add 256 2^-24 = 1.5e-5 of A at most; in fp32 that is the
whole bound.  States and decay gradients are fp32 in both."""
import numpy as np
import torch

from oracle import linear_ops as lo

BF16 = 2.0 ** -8
SUM = 256 * 2.0 ** -24


def make(lengths, Hk, H, d, dtype, *, const=False, h0=True, seed=0, rate=None):
    """(inputs, cu): unit q, k; heads that remember a few to a thousand tokens."""
    gen = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=gen)
    T, N = sum(lengths), len(lengths)
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dtype)
    r = torch.exp(-6.0 * torch.rand(H, generator=gen)) if rate is None else torch.full((H,), float(rate))
    x = dict(q=unit(randn(T, Hk, d)), k=unit(randn(T, Hk, d)), v=randn(T, H, d).to(dtype),
             g=-r if const else -r * randn(T, H).abs(), h0=0.3 * randn(N, H, d, d) if h0 else None,
             dO=randn(T, H, d).to(dtype), dhT=0.3 * randn(N, H, d, d) if h0 else None)
    cu = torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int32)
    return x, cu


def cuda(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def sizes(x):
    return {n: None if t is None else (t if n == "g" else t.abs()) for n, t in x.items()}


def close(got, ref, size, dtype, what):
    """Elementwise bound of an output held in dtype."""
    got = got.detach().cpu().double().numpy()
    assert got.shape == ref.shape, what
    bound = SUM * size + 1e-30
    if dtype == torch.bfloat16:
        bound = bound + BF16 * (np.abs(ref) + size)
    over = np.abs(got - ref) - bound
    assert np.all(np.isfinite(got)), what
    assert over.size == 0 or over.max() <= 0, (what, float(over.max()), float(np.abs(got - ref).max()))


def near(got, ref, most, what):
    got = got.detach().cpu().double().numpy()
    n = np.linalg.norm(ref)
    assert np.linalg.norm(got - ref) <= most * n + 1e-30, (what, np.linalg.norm(got - ref) / max(n, 1e-30))


def decay_sizes(x, cu, scale):
    """What dg_t is a sum of: q . dq and k . dk of the tokens from t on, and
    <S, E> at the sequence's end; by size."""
    a = sizes(x)
    g = lo.linear_backward(a["q"], a["k"], a["v"], a["g"], a["dO"], cu, a["h0"], a["dhT"], scale)
    hT = lo.linear_forward(a["q"], a["k"], a["v"], a["g"], cu, a["h0"], scale)[1]
    rep = x["v"].shape[1] // x["q"].shape[1]
    H = x["v"].shape[1]
    per = [np.repeat((lo._f64(a[n]) * g["d" + n]).sum(-1), rep, 1) for n in ("q", "k")]
    t = per[0] + per[1]
    out = np.zeros((x["v"].shape[0], H))
    for n in range(len(cu) - 1):
        s, e = int(cu[n]), int(cu[n + 1])
        end = np.zeros(H) if a["dhT"] is None else (hT[n] * lo._f64(a["dhT"][n])).sum((-1, -2))
        out[s:e] = t[s:e][::-1].cumsum(0)[::-1] + end
    return g, (out.sum(0) if x["g"].dim() == 1 else out)
