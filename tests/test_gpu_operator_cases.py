"""perf/operators.py on the GPU: the package's calls and the plain forms against the definitions in 64 bits."""
import random

import pytest

import operator_cases as oc
from test_operator_cases_cpu import SMALL

pytestmark = pytest.mark.gpu


def _some():
    mod, rng = oc.load("cuda", own=True), random.Random(7)
    listed = [c for c in mod.listed() if mod.work(c)["flops"] < 1e10]
    drawn = [c for c in (mod.draw(rng) for _ in range(60)) if mod.work(c)["flops"] < 2e9]
    return SMALL + listed + drawn


@pytest.mark.parametrize("own", [True, False])
def test_cases(lib, own):
    mod = oc.load("cuda", own)
    for i, case in enumerate(_some()):
        oc.check(mod, case, 100 + i)
    assert lib.device_status() == 0
