"""examples/moe_block.py with experts in bf16: each step against the 64-bit forms, on what the step before gave."""
import os
import subprocess
import sys

import pytest
import torch

import rows_ref as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.mark.parametrize("tokens", [1, 13, 300])
def test_block(lib, tokens):
    import moe_block
    H, width, E, k = 512, 160, 16, 4
    w = moe_block.make_bf16_weights(H, width, E, seed=tokens)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x, r = (torch.randn(tokens, H, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    out, residual, mid = moe_block.bf16_moe_block(x, r, w, k)
    assert torch.equal(residual, (x.float() + r.float()).to(torch.bfloat16))
    for a, b in zip(mid["by"], ref.group(mid["ids"].cpu(), E)):
        assert torch.equal(a.cpu(), b)
    ref.check(mid["act"], *ref.grouped(mid["norm"].out, w["gate_up"], mid["by"].offsets, None, mid["by"].rows, True))
    ref.check(mid["down"], *ref.grouped(mid["act"], w["down"], mid["by"].offsets, None, None, False))
    ref.check(out, *ref.combine(mid["down"], mid["by"].place, mid["weights"], None))
    graph = torch.cuda.CUDAGraph()  # nothing on the way leaves the device
    with torch.cuda.graph(graph):
        again = moe_block.bf16_moe_block(x, r, w, k)[0]
    graph.replay()
    assert torch.equal(again, out) and lib.device_status() == 0


def test_command_line(lib):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "moe_block.py"), "--tokens", "5", "--hidden", "256",
                        "--width", "64", "--experts", "8", "--bf16"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "5 tokens through" in r.stdout
