"""What perf/operators.py computes for a case, held against its definitions in 64 bits."""
import importlib.util
import os

import numpy as np
import torch

import moe_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SLACK = 2.0 ** -17   # of |y|, the norm in fp32 (tests/test_gpu_norm.py)
WEIGHT = 2.0 ** -17  # of a routing weight (tests/test_gpu_route.py)


def load(device, own):
    """A fresh copy of the module, its inputs on `device`."""
    spec = importlib.util.spec_from_file_location("operators", os.path.join(ROOT, "perf", "operators.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.DEV, mod.own = device, own
    return mod


def _norm(mod, case, got, want):
    y = ref.f64(want["out"])
    assert (np.abs(ref.f64(got["out"]) - y) <= ref.half_ulp(np.abs(y) * (1 + SLACK)) + SLACK * np.abs(y)).all()
    if case["residual"]:  # the sum of two bf16 values, rounded once (f64 holds it exactly)
        assert torch.equal(got["residual"], want["residual"].float().to(torch.bfloat16))
    if case["quant"] == "none":
        return
    u, c = ref.f64(want["codes"]), ref.f64(got["codes"].float())
    near = np.abs(c - u) <= (2.0 ** -4 + 2 * SLACK) * np.abs(u) + 2.0 ** -10
    if case["quant"] == "mxfp8":
        e = np.log2(ref.f64(want["scales"])).astype(np.int64)
        b = y.reshape(*e.shape, 32)
        lo, hi = (ref.scale_exponents(b * f, 8) for f in (1 - SLACK, 1 + SLACK))
        g = np.log2(ref.f64(got["scales"].float())).astype(np.int64)
        assert ((g == lo) | (g == hi)).all() and ((e == lo) | (e == hi)).all()
        near |= np.repeat(g != e, 32, axis=-1)  # a largest magnitude within SLACK of a power of two: other codes
    assert near.all()


def _route(mod, case, got, want, state):
    w, ids = ref.f64(got["weights"]), got["ids"].cpu().numpy().astype(np.int64)
    key, score, allowed = ref.route(ref.f64(state["logits"]), case["k"], case["scoring"],
                                    None if state["bias"] is None else ref.f64(state["bias"]), case["groups"], case["top"],
                                    case["best"], True, 1.0)
    masked = np.where(allowed, key, -np.inf)
    order = np.argsort(-masked, axis=-1, kind="stable")[:, :case["k"]]
    if case["scoring"] == "softmax":
        assert np.array_equal(ids, order)
    picked = np.take_along_axis(masked, ids, 1)
    assert (np.abs(picked - np.take_along_axis(masked, order, 1)) <= 2.0 ** -18).all()
    s = np.take_along_axis(score, ids, 1)
    s = s / s.sum(-1, keepdims=True)
    assert (np.abs(w - s) <= WEIGHT * s).all()
    same = (ids == order).all(-1)
    assert (np.abs(w - ref.f64(want["weights"])) <= WEIGHT * s)[same].all()


def _linear(mod, case, got, want, state):
    x = mod._exact_fp4(state["x"]) if case["dynamic"] else mod._exact_values(state["xq"], state["xs"])
    sabs = x.abs() @ mod._exact_values(state["wq"], state["ws"]).abs().t()
    if state["bias"] is not None:
        sabs = sabs + state["bias"].double().abs()
    y, sabs = ref.f64(want), ref.f64(sabs)
    bound = ref.linear_bound(y, sabs, case["K"])
    if not mod.own:  # K sums in fp32, in any order
        acc = case["K"] * 2.0 ** -24 * sabs
        bound = ref.half_ulp(np.abs(y) + acc) + acc
    assert (np.abs(ref.f64(got) - y) <= bound).all()


def check(mod, case, seed):
    state = mod.prepare(case, seed)
    got, want = mod.run(state), mod.exact(case, seed)
    if case["op"] == "norm":
        _norm(mod, case, got, want)
    elif case["op"] == "quant":  # values that bf16 holds
        assert np.array_equal(ref.f64(got), ref.f64(want))
    elif case["op"] == "route":
        _route(mod, case, got, want, state)
    else:
        _linear(mod, case, got, want, state)
