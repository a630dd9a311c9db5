"""The plain forms of perf/operators.py against its definitions in 64 bits, on the CPU; its lists, draws and counts of work."""
import random

import pytest

import operator_cases as oc

SMALL = [dict(op="norm", T=5, H=96, ld=96, residual=True, quant="mxfp8"), dict(op="norm", T=3, H=77, ld=90, residual=False, quant="none"),
         dict(op="norm", T=4, H=130, ld=130, residual=True, quant="fp8"),
         dict(op="route", T=9, E=48, k=5, scoring="softmax", bias=False, groups=1, top=1, best=1, masked=7, dtype="bf16"),
         dict(op="route", T=9, E=48, k=5, scoring="sigmoid", bias=True, groups=4, top=2, best=2, masked=0, dtype="fp32"),
         dict(op="quant", rows=7, K=160), dict(op="linear", M=5, N=33, K=96, bias=True, dynamic=True),
         dict(op="linear", M=17, N=40, K=288, bias=False, dynamic=False)]


@pytest.mark.parametrize("case", SMALL, ids=lambda c: "-".join(str(v) for v in c.values()))
def test_plain_forms(case):
    for seed in range(3):
        oc.check(oc.load("cpu", own=False), case, seed)


def test_lists_draws_and_work():
    mod = oc.load("cpu", own=False)
    listed = mod.listed()
    names = [c["name"] for c in listed]
    assert 4 <= len(listed) <= 12 and len(set(names)) == len(names)
    assert all(sum(c["op"] == op for c in listed) >= 2 for op in ("norm", "route", "quant", "linear"))
    rng = random.Random(1)
    drawn = [mod.draw(rng) for _ in range(300)]
    keys = {c["op"]: set(c) - {"name"} for c in listed}
    assert all(set(c) == keys[c["op"]] for c in drawn) and {c["op"] for c in drawn} == set(keys)
    most = {op: max(mod.work(c)["flops"] for c in listed if c["op"] == op) for op in keys}
    for c in drawn:
        w = mod.work(c)
        assert w["bytes"] > 0 and 0 < w["flops"] <= most["linear"]
        if c["op"] in ("norm", "quant"):
            assert w["flops"] <= most[c["op"]]
