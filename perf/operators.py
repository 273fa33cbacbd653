"""Measured cases of the decayed linear attention and of the steps around it.

Five passes, each as a user's program makes it:

  prefill   linear attention with a decay for each head over packed prompts:
            S_t = e^{g_t} S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t
  decode    one token of it per (sequence, head), the state updated in place
  grad      the gradient of the prefill for L = <dO, o> + <dhT, hT>
  rotary    rotary positions on the first `rot` channels of q and k
  norm      layer norm of rows, forward and backward, weight gradients included

With ``own`` false, run() computes them in plain torch operations (32 bits,
64 for the decay sums and the angles); with ``own`` true it calls the
library's entry points on the same inputs.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
CHUNK = 64                     # chunk length of the plain form


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one long prompt on 96 heads: the headline prefill shape of the library's benchmark
        dict(name="prefill_96x8192", op="prefill", dtype="bf16", n=1, lo=8192, hi=8192, H=96, Hk=96, d=128,
             decay="token", h0=False, scale=1.0),
        # a batch of packed prompts with carried states, q and k shared by four heads
        dict(name="prefill_packed", op="prefill", dtype="bf16", n=24, lo=256, hi=8192, H=32, Hk=8, d=128,
             decay="token", h0=True, scale=0.08838834764831845),
        # one very long document on few heads, with a constant decay for each head
        dict(name="prefill_16x131072", op="prefill", dtype="bf16", n=1, lo=131072, hi=131072, H=16, Hk=16, d=128,
             decay="head", h0=False, scale=1.0),
        # a few short ragged prompts in full precision: latency
        dict(name="prefill_short_fp32", op="prefill", dtype="fp32", n=5, lo=1, hi=77, H=3, Hk=3, d=64,
             decay="token", h0=True, scale=0.125),
        # the library's batched-decode shape: 256 sequences on 96 heads
        dict(name="decode_256x96", op="decode", dtype="bf16", n=256, H=96, Hk=96, d=128, decay="token", scale=1.0),
        # one user, one token: latency
        dict(name="decode_1x16", op="decode", dtype="bf16", n=1, H=16, Hk=4, d=64, decay="head", scale=0.125),
        # the training shape of the library's benchmark
        dict(name="grad_96x2048", op="grad", dtype="bf16", n=1, lo=2048, hi=2048, H=96, Hk=96, d=128,
             decay="token", h0=False, scale=1.0),
        # packed training documents, carried state, q and k shared by two heads
        dict(name="grad_packed", op="grad", dtype="bf16", n=6, lo=100, hi=3000, H=16, Hk=8, d=128,
             decay="token", h0=True, scale=0.08838834764831845),
        # q and k of the long prompt, whole heads, first and second half paired
        dict(name="rotary_8192x96", op="rotary", dtype="bf16", T=8192, H=96, Hk=96, d=128, rot=128,
             interleaved=False, last=8192, factor=1.0),
        # one decode step far into long contexts: neighbours paired, half of the head, scaled
        dict(name="rotary_step", op="rotary", dtype="bf16", T=256, H=96, Hk=8, d=128, rot=64,
             interleaved=True, last=1000000, factor=32.0),
        # the norm of the operator's output, a weight row for each of 96 heads
        dict(name="norm_heads", op="norm", dtype="bf16", T=8192, G=96, D=128, bias=False),
        # the norm of a residual stream, ragged width
        dict(name="norm_wide", op="norm", dtype="bf16", T=4099, G=1, D=5000, bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("prefill", "prefill", "decode", "grad", "rotary", "norm"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    d = rng.choice((16, 32, 64, 128, 128))
    Hk = _log(rng, 1, 48)
    H = Hk * rng.choice((1, 1, 2, 4) if Hk <= 24 else (1, 2))
    if op in ("prefill", "grad"):
        n = _log(rng, 1, 24)
        most = 500000 if op == "prefill" else 150000      # tokens times heads
        if dtype == "fp32":
            most //= 4
        hi = max(2, min(_log(rng, 2, 16384), most // (n * H)))
        lo = max(0, hi // rng.choice((1, 2, 8, 40)) - rng.choice((0, 0, 1)))
        return dict(op=op, dtype=dtype, n=n, lo=lo, hi=hi, H=H, Hk=Hk, d=d, decay=rng.choice(("token", "token", "head")),
                    h0=rng.random() < 0.5, scale=rng.choice((1.0, 1.0 / math.sqrt(d))))
    if op == "decode":
        return dict(op=op, dtype=dtype, n=_log(rng, 1, 256), H=H, Hk=Hk, d=d, decay=rng.choice(("token", "head")),
                    scale=rng.choice((1.0, 1.0 / math.sqrt(d))))
    if op == "rotary":
        d = rng.choice((64, 80, 128, 192, 256))
        T = _log(rng, 1, 8192)
        H, Hk = min(H, 64), min(Hk, 32)
        return dict(op=op, dtype=dtype, T=T, H=H, Hk=Hk, d=d, rot=2 * rng.randint(d // 16, d // 2),
                    interleaved=rng.random() < 0.5, last=_log(rng, 100, 1000000) + T,
                    factor=rng.choice((1.0, 4.0, 32.0)))
    G = rng.choice((1, 1, 4, 16, 96))
    D = _log(rng, 32, 8192) if G == 1 else rng.choice((16, 32, 64, 128, 100, 256))
    return dict(op="norm", dtype=dtype, T=max(1, min(_log(rng, 1, 20000), 40000000 // (G * D))), G=G, D=D,
                bias=rng.random() < 0.5)


def _lengths(case):
    r = random.Random(1000003 * case["n"] + 1009 * case["lo"] + case["hi"])
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["n"])]
    return lens if sum(lens) else [1] + lens[1:]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("prefill", "grad"):
        lens = _lengths(case)
        T, N, H, Hk, d = sum(lens), len(lens), case["H"], case["Hk"], case["d"]
        g = 4 * T * H if case["decay"] == "token" else 4 * H
        state = 4 * N * H * d * d
        if case["op"] == "prefill":
            # q, k, v, g in; o and the final states out; the two products with the state
            return {"bytes": e * T * d * (2 * Hk + 2 * H) + g + state * (2 if case["h0"] else 1) + 4 * (N + 1),
                    "flops": 4 * T * H * d * d}
        # q, k, v, dO, g in; dq, dk, dv, dg out; both recurrences and their reads
        return {"bytes": e * T * d * (4 * Hk + 3 * H) + 2 * g + state * (3 if case["h0"] else 2) + 4 * (N + 1),
                "flops": 10 * T * H * d * d}
    if case["op"] == "decode":
        B, H, Hk, d = case["n"], case["H"], case["Hk"], case["d"]
        return {"bytes": 8 * B * H * d * d + e * B * d * (2 * Hk + 2 * H) + 4 * H * (B if case["decay"] == "token" else 1),
                "flops": 5 * B * H * d * d}
    if case["op"] == "rotary":
        T, heads = case["T"], case["H"] + case["Hk"]
        return {"bytes": 2 * e * T * heads * case["d"] + 4 * T, "flops": 3 * T * heads * case["rot"]}
    T, G, D = case["T"], case["G"], case["D"]
    # x and dy in, y and dx out; mean and rstd kept; the weights and their gradients
    return {"bytes": 4 * e * T * G * D + 8 * T * G + 4 * G * D * (4 if case["bias"] else 2), "flops": 20 * T * G * D}


# ----------------------------------------------------------------- inputs
def _plan(lens, dev):
    """Where the tokens of each chunk lie, and the chunks of each sequence."""
    idx, seq, first, last, cu = [], [], [], [], [0]
    for n, L in enumerate(lens):
        first.append(len(seq))
        for c in range(0, L, CHUNK):
            idx.append((cu[-1] + c, min(CHUNK, L - c)))
            seq.append(n)
        last.append(len(seq) - 1)
        cu.append(cu[-1] + L)
    start = torch.tensor([a for a, _ in idx])[:, None] + torch.arange(CHUNK)
    live = torch.arange(CHUNK) < torch.tensor([b for _, b in idx])[:, None]
    T = cu[-1]
    back = torch.empty(T, dtype=torch.long)
    back[start[live]] = torch.arange(live.numel()).reshape(live.shape)[live]
    full = torch.tensor([L > 0 for L in lens])
    return dict(idx=torch.where(live, start, T).to(dev), back=back.to(dev), seq=torch.tensor(seq).to(dev),
                first=torch.tensor(first).clamp(max=len(seq) - 1).to(dev),
                last=torch.tensor(last).clamp(min=0).to(dev), full=full.to(dev),
                cu=torch.tensor(cu, dtype=torch.int32).to(dev), lens=lens)


def _frequencies(rot, factor, last):
    """Angles per position; a factor above 1 stretches the slow channels by it, the
    fast ones not at all, and those between by a linear ramp (scaled by parts)."""
    inv = torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    if factor == 1.0:
        return inv.float(), 1.0
    turns = 4096.0 * inv / (2.0 * math.pi)
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
    return (inv * keep + inv / factor * (1.0 - keep)).float(), 1.0 + 0.1 * math.log(factor)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def unit(*shape):
        x = randn(*shape)
        return (x / x.norm(dim=-1, keepdim=True)).to(dt)

    s = dict(case=case)
    op = case["op"]
    if op in ("prefill", "grad", "decode"):
        H, Hk, d = case["H"], case["Hk"], case["d"]
        if op == "decode":
            T = N = case["n"]
        else:
            s["plan"] = _plan(_lengths(case), dev)
            T, N = sum(s["plan"]["lens"]), len(s["plan"]["lens"])
        s["q"], s["k"], s["v"] = unit(T, Hk, d), unit(T, Hk, d), randn(T, H, d).to(dt)
        # heads remember from a few tokens to about a thousand
        rate = torch.exp(torch.rand(H, generator=gen, device=dev) * math.log(500.0) - math.log(500.0))
        if case["decay"] == "head":
            s["g"] = -rate
        else:
            s["g"] = -rate * torch.nn.functional.softplus(randn(T, H) + 0.5)
        state = (lambda: randn(N, H, d, d) * 0.3)
        if op == "decode":
            s["S"] = state()
        else:
            s["h0"] = state() if case["h0"] else None
        if op == "grad":
            s["dO"] = randn(T, H, d).to(dt)
            s["dhT"] = state() if case["h0"] else None
    elif op == "rotary":
        T, d = case["T"], case["d"]
        s["q"], s["k"] = randn(T, case["H"], d).to(dt), randn(T, case["Hk"], d).to(dt)
        if T <= 1024:          # a step: every row at a place of its own
            s["pos"] = torch.randint(0, case["last"], (T,), generator=gen, device=dev).to(torch.int32)
        else:                  # a prompt
            s["pos"] = torch.arange(case["last"] - T, case["last"], device=dev, dtype=torch.int32)
        inv, s["scale"] = _frequencies(case["rot"], case["factor"], case["last"])
        s["inv"] = inv.to(dev)
    else:
        T, G, D = case["T"], case["G"], case["D"]
        shape = (T, D) if G == 1 else (T, G, D)
        s["x"] = (randn(*shape) * 2.0 + 0.5).to(dt)
        s["dy"] = randn(*shape).to(dt)
        s["w"] = 1.0 + 0.2 * randn(*shape[1:])
        s["b"] = 0.1 * randn(*shape[1:]) if case["bias"] else None
    return s


# ------------------------------------------------------------- plain forms
def _chunks(x, plan):
    """[T, H, ...] -> [H, chunks, CHUNK, ...] in fp32, zero behind each end."""
    x = torch.cat([x.float(), x.new_zeros((1,) + tuple(x.shape[1:]), dtype=torch.float32)])
    return x[plan["idx"]].movedim(2, 0).contiguous()


def _decays(g, T, H, plan):
    """The log-decay sums in 64 bits: from the chunk's start to each token, of
    whole chunks, and from the first chunk's start to each chunk's end."""
    g = g.double() if g.dim() == 2 else g.double().expand(T, H)
    g = torch.cat([g, g.new_zeros(1, H)])[plan["idx"]].movedim(2, 0)
    b = g.cumsum(-1)
    total = b[..., -1]
    return b, total, total.cumsum(-1)


def _across(total, cum, plan):
    """M[c, c'] = decay from the end of chunk c' to the start of chunk c, c' < c in
    one sequence; `begin`: from the sequence's start to the start of chunk c."""
    start = cum - total
    seq = plan["seq"]
    n = seq.numel()
    before = (seq[:, None] == seq[None, :]) & torch.ones(n, n, dtype=torch.bool, device=seq.device).tril(-1)
    M = torch.where(before, start[:, :, None] - cum[:, None, :], -math.inf).exp_().float()
    begin = (start - start[:, plan["first"]][:, seq]).exp().float()
    end = (cum[:, plan["last"]][:, seq] - cum).exp().float()
    return M, begin, end


def _spread(b):
    """D[i, j] = e^{b_i - b_j} for i >= j, else 0."""
    keep = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=b.device).tril()
    return torch.where(keep, b[..., :, None] - b[..., None, :], -math.inf).exp_().float()


def _states(k, v, b, total, M, begin, h0, plan):
    d = k.shape[-1]
    add = (k * (total[..., None] - b).exp().float()[..., None]).transpose(-1, -2) @ v
    S = (M @ add.flatten(2)).unflatten(-1, (d, d))
    if h0 is not None:
        S = S + begin[..., None, None] * h0.movedim(1, 0)[:, plan["seq"]]
    return S, add


def _whole(x, plan):
    """[H, chunks, CHUNK, ...] -> [T, H, ...]."""
    return x.flatten(1, 2)[:, plan["back"]].movedim(0, 1)


def _plain_prefill(s):
    case, plan = s["case"], s["plan"]
    dt, rep = DTYPES[case["dtype"]], case["H"] // case["Hk"]
    T, H = s["v"].shape[:2]
    q, k, v = _chunks(s["q"], plan), _chunks(s["k"], plan), _chunks(s["v"], plan)
    q, k = q.repeat_interleave(rep, 0), k.repeat_interleave(rep, 0)
    b, total, cum = _decays(s["g"], T, H, plan)
    M, begin, _ = _across(total, cum, plan)
    S, add = _states(k, v, b, total, M, begin, s["h0"], plan)
    o = b.exp().float()[..., None] * (q @ S) + ((q @ k.transpose(-1, -2)) * _spread(b)) @ v
    end = total.exp().float()[..., None, None] * S + add
    hT = end[:, plan["last"]].movedim(0, 1)
    empty = torch.zeros_like(hT) if s["h0"] is None else s["h0"]
    hT = torch.where(plan["full"][:, None, None, None], hT, empty)
    return {"o": (_whole(o, plan) * case["scale"]).to(dt), "hT": hT}


def _plain_decode(s):
    case = s["case"]
    rep = case["H"] // case["Hk"]
    q, k = s["q"].float().repeat_interleave(rep, 1), s["k"].float().repeat_interleave(rep, 1)
    S = s["S"]
    S.mul_(s["g"].exp()[..., None, None]).add_(k[..., :, None] * s["v"].float()[..., None, :])
    o = (q[..., None, :] @ S)[..., 0, :] * case["scale"]
    return {"o": o.to(s["q"].dtype), "S": S}


def _plain_grad(s):
    case, plan = s["case"], s["plan"]
    dt, rep, scale = DTYPES[case["dtype"]], case["H"] // case["Hk"], case["scale"]
    T, H = s["v"].shape[:2]
    q, k, v, dO = (_chunks(s[n], plan) for n in ("q", "k", "v", "dO"))
    q, k = q.repeat_interleave(rep, 0), k.repeat_interleave(rep, 0)
    d = q.shape[-1]
    b, total, cum = _decays(s["g"], T, H, plan)
    M, begin, end = _across(total, cum, plan)
    S, _ = _states(k, v, b, total, M, begin, s["h0"], plan)
    eb, ee, D = b.exp().float()[..., None] * scale, (total[..., None] - b).exp().float()[..., None], _spread(b)
    # the gradient of the state at each chunk's end, from the chunks after it
    R = (q * eb).transpose(-1, -2) @ dO
    E = (M.transpose(-1, -2) @ R.flatten(2)).unflatten(-1, (d, d))
    if s["dhT"] is not None:
        E = E + end[..., None, None] * s["dhT"].movedim(1, 0)[:, plan["seq"]]
    # inside a chunk
    P, dP = (q @ k.transpose(-1, -2)) * D * scale, dO @ v.transpose(-1, -2)
    dA, W = dP * D * scale, P * dP
    dq_s, dk_s = eb * (dO @ S.transpose(-1, -2)), ee * (v @ E.transpose(-1, -2))
    dq, dk = dA @ k + dq_s, dA.transpose(-1, -2) @ q + dk_s
    dv = P.transpose(-1, -2) @ dO + ee * (k @ E)
    # the decays: of the chunk's inner sums, then of each token in them
    rq, rk = (q.double() * dq_s).sum(-1), (k.double() * dk_s).sum(-1)
    db = W.double().sum(-1) - W.double().sum(-2) + rq - rk
    dG = total.exp() * (S.double() * E).sum((-1, -2)) + rk.sum(-1)
    dg = _whole(db.flip(-1).cumsum(-1).flip(-1) + dG[..., None], plan)
    dg = (dg if case["decay"] == "token" else dg.sum(0)).float()
    dS = (R + total.exp().float()[..., None, None] * E)[:, plan["first"]].movedim(0, 1)
    none = torch.zeros_like(dS) if s["dhT"] is None else s["dhT"]
    dh0 = torch.where(plan["full"][:, None, None, None], dS, none)
    shared = (lambda x: _whole(x, plan).unflatten(1, (case["Hk"], rep)).sum(2).to(dt))
    return {"dq": shared(dq), "dk": shared(dk), "dv": _whole(dv, plan).to(dt), "dg": dg, "dh0": dh0}


def _plain_rotary(s):
    rot, half, pairs = s["case"]["rot"], s["case"]["rot"] // 2, s["case"]["interleaved"]
    angle = s["pos"].double()[:, None] * s["inv"].double()
    cos, sin = (angle.cos() * s["scale"]).float()[:, None], (angle.sin() * s["scale"]).float()[:, None]

    def turn(x):
        y = x.float()
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if pairs else (y[..., :half], y[..., half:rot])
        a, b = a * cos - b * sin, a * sin + b * cos
        z = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
        return torch.cat([z, y[..., rot:]], -1).to(x.dtype)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


EPS = 1e-5


def _plain_norm(s):
    x, dy, w = s["x"].float(), s["dy"].float(), s["w"]
    mean = x.mean(-1, keepdim=True)
    u = x - mean
    rstd = (u.square().mean(-1, keepdim=True) + EPS).rsqrt()
    xh = u * rstd
    y = xh * w
    if s["b"] is not None:
        y = y + s["b"]
    gw = dy * w
    dx = rstd * (gw - gw.mean(-1, keepdim=True) - xh * (gw * xh).mean(-1, keepdim=True))
    out = {"y": y.to(s["x"].dtype), "mean": mean[..., 0], "rstd": rstd[..., 0], "dx": dx.to(s["x"].dtype),
           "dw": (dy * xh).sum(0)}
    if s["b"] is not None:
        out["db"] = dy.sum(0)
    return out


PLAIN = {"prefill": _plain_prefill, "decode": _plain_decode, "grad": _plain_grad, "rotary": _plain_rotary,
         "norm": _plain_norm}


# --------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return PLAIN[op](s)
    import gated_delta_rule_60_b200 as kda
    if op == "prefill":
        o, hT = kda.kda_linear_chunk_fwd(s["q"], s["k"], s["v"], s["g"], s["h0"], s["plan"]["cu"],
                                         scale=case["scale"])
        return {"o": o, "hT": hT}
    if op == "decode":
        return {"o": kda.kda_linear_decode_step(s["q"], s["k"], s["v"], s["g"], s["S"], scale=case["scale"]),
                "S": s["S"]}
    if op == "grad":
        return kda.kda_linear_chunk_bwd(s["q"], s["k"], s["v"], s["g"], s["dO"], s["h0"], s["plan"]["cu"], s["dhT"],
                                        scale=case["scale"])
    if op == "rotary":
        q, k = kda.kda_rotary(s["q"], s["k"], s["inv"], s["pos"], interleaved=case["interleaved"], scale=s["scale"])
        return {"q": q, "k": k}
    y, mean, rstd = kda.kda_layernorm_fwd(s["x"], s["w"], s["b"], eps=EPS)
    got = kda.kda_layernorm_bwd(s["dy"], s["x"], mean, rstd, s["w"], bias=case["bias"])
    out = {"y": y, "mean": mean, "rstd": rstd, "dx": got["dx"], "dw": got["dweight"]}
    if case["bias"]:
        out["db"] = got["dbias"]
    return out


# ------------------------------------------------- the definitions, 64 bits
def _padded(x, plan):
    """[T, H, ...] -> [Lmax, N, H, ...] in fp64, zero behind each end."""
    L = max(plan["lens"])
    out = torch.zeros((L, len(plan["lens"])) + tuple(x.shape[1:]), dtype=torch.float64, device=x.device)
    at = 0
    for n, m in enumerate(plan["lens"]):
        out[:m, n] = x[at:at + m].double()
        at += m
    return out


def _packed(x, plan):
    return torch.cat([x[:m, n] for n, m in enumerate(plan["lens"])])


def _exact_linear(s):
    """Token by token, every sequence side by side; behind a sequence's end the
    decay is 1 and nothing is written."""
    case, plan = s["case"], s["plan"]
    rep, scale = case["H"] // case["Hk"], case["scale"]
    T, H = s["v"].shape[:2]
    g = s["g"] if s["g"].dim() == 2 else s["g"].expand(T, H)
    a = _padded(g, plan).exp()
    q, k, v = _padded(s["q"].repeat_interleave(rep, 1), plan), _padded(s["k"].repeat_interleave(rep, 1), plan), \
        _padded(s["v"], plan)
    L, N, _, d = q.shape
    S = torch.zeros(N, H, d, d, dtype=torch.float64, device=q.device) if s["h0"] is None else s["h0"].double()
    step = (lambda S, t: torch.addcmul(a[t, ..., None, None] * S, k[t, ..., :, None], v[t, ..., None, :]))
    if case["op"] == "prefill":
        o = torch.empty_like(v)
        for t in range(L):
            S = step(S, t)
            o[t] = torch.einsum("nhij,nhi->nhj", S, q[t])
        return {"o": _packed(o, plan) * scale, "hT": S}
    dO = _padded(s["dO"], plan) * scale
    keep = {}
    for t in range(L):
        if t % 64 == 0:
            keep[t] = S
        S = step(S, t)
    dS = torch.zeros_like(S) if s["dhT"] is None else s["dhT"].double()
    dq, dk, dv, dg = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q), torch.empty_like(a)
    for t0 in sorted(keep, reverse=True):
        block = [keep.pop(t0)]
        for t in range(t0, min(t0 + 64, L)):
            block.append(step(block[-1], t))
        for t in reversed(range(t0, min(t0 + 64, L))):
            dq[t] = torch.einsum("nhij,nhj->nhi", block[t - t0 + 1], dO[t])
            dS = torch.addcmul(dS, q[t, ..., :, None], dO[t, ..., None, :])
            dk[t] = torch.einsum("nhij,nhj->nhi", dS, v[t])
            dv[t] = torch.einsum("nhij,nhi->nhj", dS, k[t])
            dS = dS * a[t, ..., None, None]
            dg[t] = (dS * block[t - t0]).sum((-1, -2))
    shared = (lambda x: _packed(x, plan).unflatten(1, (case["Hk"], rep)).sum(2))
    dg = _packed(dg, plan)
    return {"dq": shared(dq), "dk": shared(dk), "dv": _packed(dv, plan),
            "dg": dg if case["decay"] == "token" else dg.sum(0), "dh0": dS}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("prefill", "grad"):
        return _exact_linear(s)
    if op == "decode":
        rep = case["H"] // case["Hk"]
        q, k = s["q"].double().repeat_interleave(rep, 1), s["k"].double().repeat_interleave(rep, 1)
        S = s["S"].double() * s["g"].double().exp()[..., None, None]
        S += torch.einsum("bhi,bhj->bhij", k, s["v"].double())
        return {"o": torch.einsum("bhij,bhi->bhj", S, q) * case["scale"], "S": S}
    if op == "rotary":
        rot = case["rot"]
        angle = s["pos"].double()[:, None] * s["inv"].double()
        by = torch.polar(torch.full_like(angle, s["scale"]), angle)[:, None]

        def turn(x):
            y = x.double()
            z = y[..., :rot]
            if case["interleaved"]:
                z = torch.view_as_real(torch.view_as_complex(z.unflatten(-1, (rot // 2, 2)).contiguous()) * by).flatten(-2)
            else:
                w = torch.complex(z[..., :rot // 2].contiguous(), z[..., rot // 2:].contiguous()) * by
                z = torch.cat([w.real, w.imag], -1)
            return torch.cat([z, y[..., rot:]], -1)

        return {"q": turn(s["q"]), "k": turn(s["k"])}
    # layer norm from its definition, the gradients by automatic differentiation
    x, w = s["x"].double().requires_grad_(), s["w"].double().requires_grad_()
    b = None if s["b"] is None else s["b"].double().requires_grad_()
    mean = x.sum(-1, keepdim=True) / x.shape[-1]
    var = ((x - mean) ** 2).sum(-1, keepdim=True) / x.shape[-1]
    rstd = 1.0 / torch.sqrt(var + EPS)
    y = (x - mean) * rstd * w if b is None else (x - mean) * rstd * w + b
    grads = torch.autograd.grad(y, [x, w] + ([] if b is None else [b]), s["dy"].double())
    out = {"y": y.detach(), "mean": mean.detach()[..., 0], "rstd": rstd.detach()[..., 0], "dx": grads[0],
           "dw": grads[1]}
    if b is not None:
        out["db"] = grads[2]
    return out
