"""The calls that csrc/torch_calls.cpp marshals give what the ctypes path gives, and leave the same errors."""
import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(params=["compiled", "ctypes"])
def path(lib, monkeypatch, request):
    from moe_router_gemm_gb300 import _binding
    if request.param == "ctypes":
        monkeypatch.setattr(_binding, "_calls", None)
    elif _binding._calls is None:
        pytest.skip("the marshalling module is not built for this PyTorch")
    return lib


def _work(m):
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(21, 640, generator=g, device=DEV).to(torch.bfloat16)
    r, w = x.flip(0).contiguous(), x[0].contiguous()
    logits, bias = torch.randn(21, 64, generator=g, device=DEV), torch.randn(64, generator=g, device=DEV)
    one = torch.full((1,), 0.02, device=DEV)
    wq, ws = m.quant_mxfp4(torch.randn(96, 640, generator=g, device=DEV).to(torch.bfloat16))
    xq, xs = m.quant_mxfp4(x)
    wide = torch.randn(21, 900, generator=g, device=DEV).to(torch.bfloat16)[:, 5:645]
    b = bias.to(torch.bfloat16).repeat(2)[:96].contiguous()
    got = [*m.rmsnorm(x, w), *m.rmsnorm(x, w, r, quant="mxfp8"), *m.rmsnorm(wide, w, r, quant="mxfp4", bf16_out=False),
           *m.rmsnorm(x, w, quant="fp8", scale=one, eps=1e-3), *m.route(logits, 5), xq, xs, m.dequant_mxfp4(xq, xs),
           *m.route(logits.to(torch.bfloat16)[:, :48], 3, scoring="sigmoid", bias=bias[:48], groups=4, top_groups=2,
                    group_best=2, renormalize=False, scale=1.5),
           m.bf16_linear_mxfp4(xq, xs, wq, ws), m.bf16_linear_mxfp4(xq, xs, wq, ws, b),
           m.bf16_linear_mxfp4_dynamic(x, wq, ws, b), m.bf16_linear_mxfp4_dynamic(x[:3], wq, ws),
           m.rmsnorm(x[:0], w).out, m.bf16_linear_mxfp4_dynamic(x[:0], wq, ws)]
    return [t for t in got if t is not None]


def test_same_results(lib, monkeypatch):
    from moe_router_gemm_gb300 import _binding
    a = _work(lib)
    monkeypatch.setattr(_binding, "_calls", None)
    b = _work(lib)
    assert len(a) == len(b) == 23
    for p, q in zip(a, b):
        assert p.dtype == q.dtype and p.shape == q.shape and p.is_contiguous() and torch.equal(p, q)


def test_current_stream(path):
    """A call goes to the stream that is current, behind what that stream still has to do."""
    x = torch.zeros(64, 4096, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(4096, dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        x.fill_(3.0)
        out = path.rmsnorm(x, w).out
    s.synchronize()
    assert (out == 1.0).all()


def test_refusals(path):
    m = path
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    q, s = m.quant_mxfp4(x)
    for f, err in ((lambda: m.rmsnorm(x.float(), w), TypeError), (lambda: m.rmsnorm(x, w[:32]), ValueError),
                   (lambda: m.rmsnorm(x, w.cpu()), ValueError), (lambda: m.rmsnorm(x.cpu(), w), ValueError),
                   (lambda: m.rmsnorm(x, w, quant="fp8"), ValueError), (lambda: m.rmsnorm(x, w, bf16_out=False), ValueError),
                   (lambda: m.rmsnorm(x, w, quant="mxfp8", scale=w.float()[:1]), ValueError),
                   (lambda: m.route(x.double(), 2), TypeError), (lambda: m.route(x, 2, scoring="tanh"), ValueError),
                   (lambda: m.route(x, 2, bias=w), ValueError), (lambda: m.quant_mxfp4(x.float()), ValueError),
                   (lambda: m.quant_mxfp4(x[:, :32]), ValueError), (lambda: m.dequant_mxfp4(q, s[:2]), ValueError),
                   (lambda: m.bf16_linear_mxfp4(q, s, q, s[:, :1]), ValueError),
                   (lambda: m.bf16_linear_mxfp4_dynamic(x, q, s, bias=w.float()), ValueError)):
        with pytest.raises(err):
            f()
    for f, status in ((lambda: m.rmsnorm(x, w, eps=-1.0), -1), (lambda: m.rmsnorm(x[:, :40].contiguous(), w[:40], quant="mxfp4"), -6),
                      (lambda: m.route(x, 0), -1), (lambda: m.route(x, 40), -6), (lambda: m.route(x, 2, groups=3), -1),
                      (lambda: m.quant_mxfp4(x[:, :48].contiguous()), -6), (lambda: m.rmsnorm(x, w, flags=3), -1)):
        with pytest.raises(m.BF16LinearError) as e:
            f()
        assert e.value.status == status


def test_sizes_past_32_bits_are_refused(path):
    """Arguments that no C int holds are errors and not what their low 32 bits say."""
    m, wide = path, (1 << 32) + 64
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device=DEV)
    w, (q, s) = torch.ones(64, dtype=torch.bfloat16, device=DEV), m.quant_mxfp4(x)
    row, codes = torch.zeros(1, wide, dtype=torch.bfloat16, device=DEV), torch.zeros(1, wide // 2, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(1, wide // 32, dtype=torch.uint8, device=DEV)
    calls = [lambda: m.rmsnorm(row, row[0]), lambda: m.rmsnorm(row, row[0], quant="mxfp4", bf16_out=False),
             lambda: m.quant_mxfp4(row), lambda: m.dequant_mxfp4(codes, scales),
             lambda: m.bf16_linear_mxfp4(codes, scales, codes, scales),
             lambda: m.bf16_linear_mxfp4_dynamic(row, codes, scales),
             lambda: m.route(row, 2), lambda: m.route(x, (1 << 32) + 2)]
    for over in (1 << 32, 1 << 70):
        calls += [lambda o=o: m.route(x, 2, **o) for o in (dict(groups=over + 1), dict(top_groups=over + 1), dict(group_best=over + 1))]
        calls += [lambda f=f: m.rmsnorm(x, w, flags=f) for f in (over, -over)]
        calls += [lambda f=f: f(over) for f in (lambda v: m.quant_mxfp4(x, flags=v), lambda v: m.dequant_mxfp4(q, s, flags=v),
                                                lambda v: m.bf16_linear_mxfp4(q, s, q, s, flags=v),
                                                lambda v: m.bf16_linear_mxfp4_dynamic(x, q, s, flags=v),
                                                lambda v: m.route(x, 2, flags=v))]
    for f in calls:
        with pytest.raises(m.BF16LinearError) as e:
            f()
        assert e.value.status in (-1, -6)
    assert m.mxfp4_dynamic_workspace(17, 64, wide) == 0


def test_other_threads_run_while_a_launch_waits(path):
    """A launch waits when the stream has as many as it takes; the interpreter is free meanwhile."""
    x = torch.ones(4, 256, dtype=torch.bfloat16, device=DEV)
    w, logits = x[0].contiguous(), torch.zeros(4, 64, device=DEV)
    q, sc = path.quant_mxfp4(x)
    calls = [lambda: path.rmsnorm(x, w), lambda: path.route(logits, 2), lambda: path.quant_mxfp4(x),
             lambda: path.dequant_mxfp4(q, sc), lambda: path.bf16_linear_mxfp4(q, sc, q, sc),
             lambda: path.bf16_linear_mxfp4_dynamic(x, q, sc)]
    stream = torch.cuda.Stream()
    for call in calls:
        took = []

        def work():
            with torch.cuda.stream(stream):
                torch.cuda._sleep(1_200_000_000)  # most of a second
                for _ in range(3000):
                    t = time.perf_counter()
                    call()
                    took.append(time.perf_counter() - t)

        torch.cuda.synchronize()
        worker = threading.Thread(target=work)
        worker.start()
        gap, last = 0.0, time.perf_counter()
        while worker.is_alive():
            time.sleep(0.001)
            now = time.perf_counter()
            gap, last = max(gap, now - last), now
        worker.join()
        torch.cuda.synchronize()
        assert len(took) == 3000 and max(took) > 0.1, "no launch had to wait"
        assert gap < max(took) / 2, f"{gap:.3f} s without the interpreter, in a call of {max(took):.3f} s"
