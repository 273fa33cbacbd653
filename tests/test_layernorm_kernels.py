"""Every layer-norm kernel in the library is one that some width asks for, and the
other way round (CPU; kernels by the names of their host stubs)."""
import re
import subprocess

from gated_delta_rule_60_b200 import build


def _wanted():
    """(type, vector, threads of a row, vectors of a thread, row fills its share)."""
    out = set()
    for D in range(1, 8193):
        for name, size in (("__nv_bfloat16", 2), ("float", 4)):
            full = 16 // size
            V = full if D % full == 0 else 2 if size == 2 and D % 2 == 0 else 1
            long = 64 // size
            tpr, per = next((t, p) for t, p in [(2, 16), (8, 16), (32, 16)] + [(1 << i, long) for i in range(6, 10)]
                            if D <= t * p)
            out.add((name, V, tpr, per // V, D == tpr * per))
    return out


def test_kernels_are_those_that_widths_ask_for():
    names = subprocess.run(["nm", "-C", build.build()], check=True, capture_output=True, text=True).stdout
    got = {"fwd": set(), "bwd": set()}
    for which, args in re.findall(r"void kda::ln::(fwd|bwd)_kernel<([^>]*)>", names):
        a = [x.strip() for x in args.split(",")]
        got[which].add((a[0], *map(int, a[1:4]), a[4] == "true", *a[5:]))
    want = _wanted()
    assert got["fwd"] == want
    assert got["bwd"] == {w + (b,) for w in want for b in ("true", "false")}
