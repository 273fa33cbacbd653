"""A bias without a weight, for a stream and for each of G groups: the backward takes
what the forward takes.  Bounds: dx and dbias are sums of at most rows + 41 fp32 terms
one after the other (see test_rotary_norm_gpu)."""
import numpy as np
import pytest
import torch

from gated_delta_rule_60_b200 import binding
from oracle import linear_ops as lo

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape,groups", [((37, 4, 64), 4), ((5, 3, 100), 3), ((29, 96), 0), ((2, 11, 5, 16), 5)])
def test_gradient_of_a_bias_alone(shape, groups):
    gen = torch.Generator().manual_seed(sum(shape))
    x, dy = torch.randn(*shape, generator=gen), torch.randn(*shape, generator=gen)
    b = torch.randn(*(shape[-2:] if groups else shape[-1:]), generator=gen)
    y, mean, rstd = binding.kda_layernorm_fwd(x.cuda(), None, b.cuda())
    got = binding.kda_layernorm_bwd(dy.cuda(), x.cuda(), mean, rstd, bias=b.cuda())
    assert set(got) == {"dx", "dbias"} and got["dbias"].shape == b.shape
    rows = x.numel() // b.numel()
    flat = (-1,) + tuple(b.shape)
    ref, size = (t.reshape(flat).sum(0) for t in (lo._f64(dy), np.abs(lo._f64(dy))))
    assert np.all(np.abs(got["dbias"].double().cpu().numpy() - ref) <= (rows + 41) * 2.0 ** -24 * size)
    none = binding.kda_layernorm_bwd(dy.cuda(), x.cuda(), mean, rstd)
    assert set(none) == {"dx"} and torch.equal(none["dx"], got["dx"])
    # with a weight of ones of the same shape: the same, and the weight's gradient besides
    w = torch.ones_like(b).cuda()
    both = binding.kda_layernorm_bwd(dy.cuda(), x.cuda(), mean, rstd, w, bias=b.cuda())
    flag = binding.kda_layernorm_bwd(dy.cuda(), x.cuda(), mean, rstd, w, bias=True)
    assert torch.equal(both["dbias"], got["dbias"]) and all(torch.equal(both[n], flag[n]) for n in both)


def test_a_bias_of_another_shape_is_refused():
    x = torch.randn(6, 4, 64, device="cuda")
    y, m, r = binding.kda_layernorm_fwd(x)
    w = torch.ones(4, 64, device="cuda")
    for bias, weight in ((torch.zeros(64, device="cuda"), w), (torch.zeros(3, 64, device="cuda"), None),
                         (torch.zeros(4, 32, device="cuda"), None), (w, torch.ones(64, device="cuda")),
                         (torch.zeros(4, 64), w)):
        with pytest.raises(ValueError):
            binding.kda_layernorm_bwd(x, x, m, r, weight, bias=bias)
    with pytest.raises(TypeError):
        binding.kda_layernorm_bwd(x, x, m, r, bias=w.to(torch.bfloat16))
