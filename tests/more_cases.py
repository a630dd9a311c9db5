"""What perf/more_operators.py computes for a case, held against its definitions in 64 bits."""
import importlib.util
import os

import torch

import rows_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load(device, own):
    """A fresh copy of the module, its inputs on `device`."""
    spec = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.DEV, mod.own = device, own
    return mod


def small(mod, rng, op, most=3e7):
    """A drawn case of this operator, halved until it has little work."""
    case = mod.draw(rng)
    while case["op"] != op:
        case = mod.draw(rng)
    least = dict(T=1, N=16, K=64, H=16)
    while mod.work(case)["flops"] > most or mod.work(case)["bytes"] > most:
        key = rng.choice([k for k in least if k in case])
        case[key] = max(least[key], case[key] // 16 * 8 if key == "K" else case[key] // 2)
    return case


def check(mod, case, seed):
    got, want = mod.run(mod.prepare(case, seed)), mod.exact(case, seed)
    s = mod.prepare(case, seed)
    if case["op"] == "group":
        for k in want:
            assert got[k].dtype == torch.int32 and torch.equal(got[k], want[k]), (case, k)
        return
    if case["op"] == "experts":
        y, slack = ref.grouped(s["x"], s["w"], s["offsets"], s["bias"], s["rows"], case["swiglu"])
    elif case["op"] == "combine":
        y, slack = ref.combine(s["y"], s["place"], s["weights"], s["addend"])
    else:
        y, slack = ref.lora(s["x"], s["w"], s["a"], s["b"], s["ids"], s["bias"], s["scale"])
    assert got.dtype == torch.bfloat16 and (want - y).abs().max() <= 1e-9 * y.abs().max()
    ref.check(got, want, slack, str(case))
