"""The roles of the tensor-core kernel give up their waits (a limit of polls, then an
error status), each at a point of its own.  So a role must not stand at a barrier that
others reach only while all is well: it would wait there for good (CPU; read from the
source, as no GPU is to be hung to see it)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_delta_rule_60_b200", "csrc")


def _code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def test_roles_wait_with_a_limit_only():
    code = _code("kda_linear_sm100.cuh")
    kernel = code[code.index("linear_sm100_kernel("):]
    roles = kernel[kernel.index("if (warp == 0) {\n", kernel.index("auto first")):kernel.index("if (sm.abort &&")]
    assert len(roles) > 10000
    assert "__syncthreads" not in roles
    assert not re.search(r"bar(rier)?(\.cta)?\.sync|bar(rier)?(\.cta)?\.red|named_barrier", code)
    # a wait's answer is looked at wherever it is made
    for m in re.finditer(r"[^\n]*\bwait\(sm,[^\n]*", roles):
        assert re.search(r"if \(|ok = |return", m.group(0)), m.group(0)
