"""Angles of the farthest positions.  Pairs (1, 0) become (cos, sin) of the angle in
fp32.  The angle is promised to 2e-7 rad, and sincospi is off by up to one unit of
the last place, 2^-24 below 1: |error| <= 2e-7 + 6e-8.  The reference is the 80-bit
product of position and frequency, exact in its 64 bits, reduced there."""
import numpy as np
import pytest
import torch

from gated_delta_rule_60_b200 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("low,high", [(-1 << 31, -(1 << 31) + 100000), ((1 << 31) - 100000, (1 << 31) - 1),
                                      (1 << 28, 1 << 29), (-5, 100)])
def test_far_positions(low, high, pairs):
    gen = torch.Generator().manual_seed(9)
    T, half = 600, 128
    pos = torch.randint(low, high + 1, (T,), generator=gen)
    pos[0], pos[1] = low, high
    inv = 0.5 + 0.5 * torch.rand(half, generator=gen)
    inv[0] = 1.0
    q = torch.zeros(T, 1, 2 * half)
    even = slice(0, None, 2) if pairs else slice(0, half)
    odd = slice(1, None, 2) if pairs else slice(half, None)
    q[..., even] = 1.0
    got, _ = binding.kda_rotary(q.cuda(), None, inv.cuda(), pos.to(torch.int32).cuda(), interleaved=pairs)
    got = got[:, 0].double().cpu().numpy()
    angle = pos.numpy().astype(np.longdouble)[:, None] * inv.numpy().astype(np.longdouble)
    two_pi = 2 * np.longdouble("3.14159265358979323846264338327950288")
    angle = (angle - two_pi * np.rint(angle / two_pi)).astype(np.float64)
    most = 2e-7 + 2.0 ** -24
    assert np.abs(got[:, even] - np.cos(angle)).max() <= most
    assert np.abs(got[:, odd] - np.sin(angle)).max() <= most
