"""examples/moe_block.py: each step of the block against the 64-bit forms, on what the step before gave."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import moe_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.mark.parametrize("tokens", [1, 13, 70])
def test_block(lib, tokens):
    import moe_block
    H, width, E = 512, 160, 16
    w = moe_block.make_weights(H, width, E, seed=tokens)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x, r = (torch.randn(tokens, H, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    out, residual, mid = moe_block.moe_block(x, r, w)
    h, y = ref.norm(ref.f64(x), ref.f64(r), ref.f64(w["norm"]), 1e-6)
    assert np.array_equal(ref.f64(residual), h)
    n = mid["norm"]
    assert (np.abs(ref.f64(n.out) - y) <= ref.half_ulp(np.abs(y) * (1 + 2.0 ** -17)) + 2.0 ** -17 * np.abs(y)).all()
    lg = ref.f64(n.out) @ ref.f64(w["router"]).T
    assert np.allclose(ref.f64(mid["logits"]), lg, rtol=0, atol=2.0 ** -14 * np.abs(ref.f64(n.out)).sum(1).max() / H ** 0.5)
    key, score, allowed = ref.route(ref.f64(mid["logits"]), 4, "sigmoid", ref.f64(w["bias"]), 4, 2, 2, True, 1.0)
    ids = mid["ids"].cpu().numpy().astype(np.int64)
    picked = np.take_along_axis(np.where(allowed, key, -9.0), ids, 1)
    rest = np.where(allowed, key, -9.0)
    np.put_along_axis(rest, ids, -9.0, 1)
    assert (picked.min(1) + 2.0 ** -18 >= rest.max(1)).all()
    s = np.take_along_axis(score, ids, 1)
    s /= s.sum(1, keepdims=True)
    assert np.allclose(ref.f64(mid["weights"]), s, rtol=2.0 ** -17, atol=0)
    yv = ref.values_mxfp4(n.codes.cpu().numpy(), n.scales.cpu().numpy())
    total = np.zeros((tokens, H))
    for e, (token, slot, act, down) in mid["experts"].items():
        t = token.cpu().numpy()
        gu = yv[t] @ ref.values_mxfp4(*(v.cpu().numpy() for v in w["gate_up"][e])).T
        a = gu[:, :width] / (1 + np.exp(-gu[:, :width])) * gu[:, width:]
        assert np.allclose(ref.f64(act), a, rtol=2.0 ** -5, atol=2.0 ** -5 * np.sqrt((a * a).mean()))
        q = ref.values_mxfp4(*ref.quant_mxfp4(ref.f64(act)))
        ref.check_linear(down, q, ref.values_mxfp4(*(v.cpu().numpy() for v in w["down"][e])), None, width, f"expert {e}")
        np.add.at(total, t, ref.f64(down) * ref.f64(mid["weights"])[t, slot.cpu().numpy(), None])
    assert np.allclose(ref.f64(out), total, rtol=2.0 ** -7, atol=2.0 ** -18 * np.abs(total).max())


def test_command_line(lib):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "moe_block.py"), "--tokens", "5", "--hidden", "256",
                        "--width", "64", "--experts", "8"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "5 tokens through" in r.stdout
