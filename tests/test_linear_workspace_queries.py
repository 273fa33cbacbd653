"""The workspace queries of the linear attention ask for nothing where the call itself
is refused, whatever the sizes (CPU)."""
import pytest

from gated_delta_rule_60_b200 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load_library()


GOOD = dict(N=3, T=1 << 20, Hk=2, H=4, d=64, dt=0)
REFUSED = [dict(T=1 << 31), dict(T=1 << 40), dict(T=(1 << 63) - 1), dict(T=-1), dict(H=70000), dict(N=1 << 30),
           dict(N=(1 << 31) - 1), dict(N=-5), dict(N=0), dict(d=48), dict(d=0), dict(dt=7), dict(H=0), dict(H=-4)]


@pytest.mark.parametrize("case", REFUSED)
def test_nothing_for_refused_sizes(lib, case):
    c = {**GOOD, **case}
    assert lib.kda_linear_chunk_fwd_workspace_size(c["N"], c["T"], c["H"], c["d"], c["dt"]) == 0
    assert lib.kda_linear_chunk_bwd_workspace_size(c["N"], c["T"], c["Hk"], c["H"], c["d"], c["dt"]) == 0


def test_something_for_the_others(lib):
    c = GOOD
    assert lib.kda_linear_chunk_fwd_workspace_size(c["N"], c["T"], c["H"], c["d"], c["dt"]) > 0
    assert lib.kda_linear_chunk_bwd_workspace_size(c["N"], c["T"], c["Hk"], c["H"], c["d"], c["dt"]) > 0
    for Hk in (0, 3, -2):
        assert lib.kda_linear_chunk_bwd_workspace_size(c["N"], c["T"], Hk, c["H"], c["d"], c["dt"]) == 0
