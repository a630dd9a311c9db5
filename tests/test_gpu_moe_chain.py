"""Calls that feed one another: back to back on a stream, with both launch flags, and in a graph, they give what the same
calls give with the device idle between any two.  Every launch may start while the one before it still runs, so a read or a
write before the grid-dependency wait would show here."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
STEPS = 12


def _weights(H, E, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    w = lambda n, k: (torch.randn(n, k, generator=g, device=DEV) * k ** -0.5).to(torch.bfloat16)  # noqa: E731
    return w(H, H), w(E, H), (1 + 0.1 * torch.randn(H, generator=g, device=DEV)).to(torch.bfloat16), g


def _chain(m, x, r, wq, ws, router, norm, bufs, flags, pause):
    """Each step's input and residual are overwritten by the step, its buffers are those of the step before."""
    picked = []
    for _ in range(STEPS):
        m.rmsnorm(x, norm, r, quant="mxfp4", out=bufs["y"], residual_out=r, codes=bufs["q"], scales=bufs["s"], flags=flags)
        pause()
        m.bf16_linear_mxfp4(bufs["q"], bufs["s"], wq, ws, out=x, flags=flags)
        pause()
        logits = m.bf16_linear_f32out(bufs["y"], router, flags=flags)
        pause()
        picked += m.route(logits, 4, scoring="sigmoid", groups=4, top_groups=2, group_best=2, flags=flags)
        pause()
        m.bf16_linear_mxfp4_dynamic(x, wq, ws, out=bufs["y"], workspace=bufs["w"], flags=flags)
        pause()
        m.quant_mxfp4(bufs["y"], out=bufs["q"], scales=bufs["s"], flags=flags)
        pause()
        m.dequant_mxfp4(bufs["q"], bufs["s"], out=x, flags=flags)
        pause()
    return [x, r, bufs["y"], *picked]


@pytest.mark.parametrize("T,H", [(1, 2048), (16, 1536), (40, 2048), (700, 2048)])
def test_chain(lib, T, H):
    W, router, norm, g = _weights(H, 64, T)
    wq, ws = lib.quant_mxfp4(W)
    x0, r0 = (torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2))

    def run(flags, pause, graph=False):
        x, r = x0.clone(), r0.clone()
        bufs = dict(y=torch.empty_like(x), q=torch.empty(T, H // 2, dtype=torch.uint8, device=DEV),
                    s=torch.empty(T, H // 32, dtype=torch.uint8, device=DEV),
                    w=torch.empty(max(256, lib.mxfp4_dynamic_workspace(T, H, H)), dtype=torch.uint8, device=DEV))
        if not graph:
            got = _chain(lib, x, r, wq, ws, router, norm, bufs, flags, pause)
        else:
            cg = torch.cuda.CUDAGraph()
            with torch.cuda.graph(cg):
                got = _chain(lib, x, r, wq, ws, router, norm, bufs, flags, pause)
            x.copy_(x0)
            r.copy_(r0)
            cg.replay()
        torch.cuda.synchronize()
        return [t.clone() for t in got]

    want = run(0, torch.cuda.synchronize)
    for _ in range(3):
        for flags in (0, lib.FLAG_PDL, lib.FLAG_SERIAL):
            got = run(flags, lambda: None)
            assert all(torch.equal(a, b) for a, b in zip(want, got)), f"flags {flags}"
    assert all(torch.equal(a, b) for a, b in zip(want, run(0, lambda: None, graph=True)))
    assert lib.device_status() == 0


@pytest.mark.parametrize("T,H", [(16, 1440), (40, 1440), (1300, 2080)])
def test_chain_with_scale_rows_off_16_byte_boundaries(lib, T, H):
    test_chain(lib, T, H)
