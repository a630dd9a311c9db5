"""Measurement cases of the operators around the linear layers: norm, routing, and 4-bit quantisation and product.

Four operators that a mixture-of-experts block needs next to its router and dense linears:

  norm    root-mean-square norm of rows, with the residual's addition before it and,
          where asked, an output in 8 bits with scales beside the bf16 one;
  route   the k experts of each token and their weights, from the router's logits;
  quant   a bf16 matrix into MXFP4 (32 elements share a power-of-two scale) and
          back into the bf16 values that the codes stand for;
  linear  out = x @ W^T (+ bias) with both operands in MXFP4, x either given in
          MXFP4 or given in bf16 and quantised by the call.

Each has a plain form here (elementary torch operations in 32 bits) and, where ``own``
is true, the package's calls.  ``exact`` restates each in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32  # elements along K that share a scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of the 4-bit codes 0..7; code 8 + i is minus code i
EPS = 1e-6


def listed():
    return [
        # A decode step's norm before the smallest router (hidden 2048): a launch's latency.
        dict(name="norm 4x2048", op="norm", T=4, H=2048, ld=2048, residual=True, quant="none"),
        # The 1536 query columns of the concatenated attention-input projection (row stride 2112),
        # normed on their own, no residual; prefill of 2048 tokens.
        dict(name="norm 2048x1536 of 2112", op="norm", T=2048, H=1536, ld=2112, residual=False, quant="none"),
        # A long prefill's norm before the experts: bf16 for the router, MXFP8 for the products, and the new residual.
        dict(name="norm 8192x7168 mxfp8", op="norm", T=8192, H=7168, ld=7168, residual=True, quant="mxfp8"),
        # Routing of a full decode batch over 256 experts, softmax scores.
        dict(name="route 16x256 softmax", op="route", T=16, E=256, k=8, scoring="softmax", bias=False, groups=1, top=1,
             best=1, masked=0, dtype="fp32"),
        # 384 experts of which some are out of service (logits of -inf), bf16 logits, an odd number of tokens.
        dict(name="route 2047x384 masked", op="route", T=2047, E=384, k=6, scoring="softmax", bias=False, groups=1, top=1,
             best=1, masked=37, dtype="bf16"),
        # A long prefill over 256 experts in 8 groups of which 4 stay, sigmoid scores with a balance bias.
        dict(name="route 8192x256 groups", op="route", T=8192, E=256, k=8, scoring="sigmoid", bias=True, groups=8, top=4,
             best=2, masked=0, dtype="fp32"),
        # One expert's activations, a ragged handful of tokens.
        dict(name="quant 37x2880", op="quant", rows=37, K=2880),
        # A square projection's weight, quantised once at load time.
        dict(name="quant 7168x7168", op="quant", rows=7168, K=7168),
        # One decode token through the attention-input projection, quantised by the call.
        dict(name="linear 1x2112x7168", op="linear", M=1, N=2112, K=7168, bias=False, dynamic=True),
        # An odd decode batch through a hidden size that no tile divides.
        dict(name="linear 13x5760x2880", op="linear", M=13, N=5760, K=2880, bias=True, dynamic=True),
        # A speculative or multi-user decode batch through a dense MLP with bias, x from the norm already quantised.
        dict(name="linear 64x14336x4096", op="linear", M=64, N=14336, K=4096, bias=True, dynamic=False),
        # Prefill of 8192 tokens through a square projection.
        dict(name="linear 8192x7168x7168", op="linear", M=8192, N=7168, K=7168, bias=False, dynamic=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _k(rng, blocks):
    """A row length in whole blocks: one of the hidden sizes in use, or an odd number of blocks."""
    if rng.random() < 0.4:
        return rng.choice([2048, 2880, 4096, 6144, 7168])
    return BLOCK * (2 * _log(rng, 1, blocks // 2) - 1)


def draw(rng):
    op = rng.choice(["norm", "route", "quant", "linear", "linear"])
    if op == "norm":
        T, quant, residual = _log(rng, 1, 8192), rng.choice(["none", "none", "fp8", "mxfp8"]), rng.random() < 0.7
        H = _k(rng, 224) if quant == "mxfp8" else _log(rng, 64, 7168)
        ld = H if residual or rng.random() < 0.5 else H + rng.randint(1, 640)
        return dict(op=op, T=T, H=H, ld=ld, residual=residual, quant=quant)
    if op == "route":
        T, scoring = _log(rng, 1, 8192), rng.choice(["softmax", "sigmoid"])
        if rng.random() < 0.4:  # limited to the best groups
            groups = rng.choice([2, 4, 8, 16])
            each = _log(rng, 2, 384 // groups)
            top = rng.randint(1, groups - 1)
            k, E = rng.randint(1, min(16, top * each)), groups * each
            best = 2 if scoring == "sigmoid" else 1
            masked = 0
        else:
            groups, top, best = 1, 1, 1
            E = _log(rng, 8, 512)
            k = rng.randint(1, min(16, E // 2))
            masked = rng.randint(0, E // 4)
        return dict(op=op, T=T, E=E, k=k, scoring=scoring, bias=scoring == "sigmoid", groups=groups, top=top, best=best,
                    masked=masked, dtype=rng.choice(["fp32", "bf16"]))
    if op == "quant":
        return dict(op=op, rows=_log(rng, 1, 7168), K=_k(rng, 224))
    M, N, K = _log(rng, 1, 8192), _log(rng, 16, 14336), _k(rng, 224)
    while M * N * K > 8192 * 7168 * 7168:
        N = max(16, N // 2)
    return dict(op=op, M=M, N=N, K=K, bias=rng.random() < 0.5, dynamic=rng.random() < 0.5)


# ---- inputs ----

def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _activations(g, rows, K):
    """A hidden state: rows of differing size, and a few channels that run far above the others."""
    x = _randn(g, rows, K)
    x *= torch.exp2(2.0 * _randn(g, rows, 1))
    x *= torch.where(torch.rand(1, K, generator=g, device=DEV) < 0.01, 20.0, 1.0)
    return x.to(torch.bfloat16)


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case=case)
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        s["x"] = _activations(g, T, case["ld"])[:, :H]
        s["residual"] = _activations(g, T, H) if case["residual"] else None
        s["weight"] = (1.0 + 0.2 * _randn(g, H)).to(torch.bfloat16)
        s["scale"] = torch.full((1,), 0.02, device=DEV) if case["quant"] == "fp8" else None
    elif case["op"] == "route":
        T, E = case["T"], case["E"]
        logits = 1.5 * _randn(g, T, E) + 0.5 * _randn(g, 1, E)
        if case["masked"]:
            logits[:, torch.randperm(E, generator=g, device=DEV)[: case["masked"]]] = float("-inf")
        s["logits"] = logits.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        s["bias"] = 0.1 * _randn(g, E) if case["bias"] else None
    elif case["op"] == "quant":
        s["x"] = (_randn(g, case["rows"], case["K"]) * case["K"] ** -0.5).to(torch.bfloat16)
    else:
        M, N, K = case["M"], case["N"], case["K"]
        x = _activations(g, M, K)
        if case["dynamic"]:
            s["x"] = x
        else:
            s["xq"], s["xs"] = _pack(*_encode(x))
        s["wq"], s["ws"] = _pack(*_encode((_randn(g, N, K) * K ** -0.5).to(torch.bfloat16)))
        s["bias"] = (0.2 * torch.rand(N, generator=g, device=DEV) - 0.1).to(torch.bfloat16) if case["bias"] else None
    return s


# ---- plain forms: elementary operations in 32 bits ----

def _pow2(e):
    """2^e in fp32 for whole e in -127..127, exactly (a power function may be off by an ulp, which moves ties)."""
    e = e.int()
    return torch.where(e > -127, ((e.clamp_min(-126) + 127) << 23).view(torch.float32), 2.0 ** -127)


def _exponents(v, top):
    """floor(log2) of each block's largest magnitude, less the format's top exponent, at least -127."""
    amax = v.abs().amax(-1)
    e = torch.frexp(amax).exponent - 1 - top
    return torch.where(amax == 0, torch.full_like(e, -127), e.clamp_min(-127))


def _encode(x):
    """MXFP4 codes (0..15) and scale exponents of x[rows, K]."""
    v = x.float().view(x.shape[0], -1, BLOCK)
    e = _exponents(v, 2)
    y = v * _pow2(-e).unsqueeze(-1)
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return (code + 8 * (y < 0).to(torch.uint8)).view(x.shape), e


def _pack(code, e):
    """Two codes to a byte, the even element in the low half; scale bytes e + 127."""
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous(), (e + 127).to(torch.uint8)


def _unpack(q, s):
    """The fp32 values of packed codes and scale bytes."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=q.device)
    code = torch.stack([q & 15, q >> 4], -1).view(q.shape[0], -1)
    v = table[code.long()].view(q.shape[0], -1, BLOCK)
    return (v * _pow2(s.int() - 127).unsqueeze(-1)).view(q.shape[0], -1)


def _plain_norm(s):
    h = s["x"].float()
    out = {}
    if s["residual"] is not None:
        out["residual"] = (h + s["residual"].float()).to(torch.bfloat16)
        h = out["residual"].float()
    y = h * (1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)) * s["weight"].float()
    out["out"] = y.to(torch.bfloat16)
    if s["case"]["quant"] == "fp8":
        out["codes"] = (y * (1.0 / s["scale"])).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    elif s["case"]["quant"] == "mxfp8":
        v = y.view(y.shape[0], -1, BLOCK)
        e = _exponents(v, 8)
        out["codes"] = (v * _pow2(-e).unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(y.shape)
        out["scales"] = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return out


def _plain_route(s):
    c, x = s["case"], s["logits"].float()
    if c["scoring"] == "softmax":
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x - torch.where(m == float("-inf"), torch.zeros_like(m), m))
        total = p.sum(-1, keepdim=True)
        score = p / torch.where(total == 0, torch.ones_like(total), total)
        key = x  # the scores' order, with no ties that rounding made
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
        key = score if s["bias"] is None else score + s["bias"]
        key = torch.where(x == float("-inf"), x, key)  # an expert out of service, whatever its bias
    if c["groups"] > 1:
        g = key.view(key.shape[0], c["groups"], -1)
        best = g.sort(dim=-1, descending=True, stable=True).values[..., : c["best"]].sum(-1)
        order = best.sort(dim=-1, descending=True, stable=True).indices
        keep = torch.zeros_like(best, dtype=torch.bool).scatter(1, order[:, : c["top"]], True)
        key = torch.where(keep.unsqueeze(-1), g, torch.full_like(g, float("-inf"))).view(key.shape)
    ids = key.sort(dim=-1, descending=True, stable=True).indices[:, : c["k"]]
    w = score.gather(1, ids)
    total = w.sum(-1, keepdim=True)
    return {"weights": w / torch.where(total == 0, torch.ones_like(total), total), "ids": ids.int()}


def _plain_linear(s):
    x = _unpack(*(_pack(*_encode(s["x"])) if s["case"]["dynamic"] else (s["xq"], s["xs"])))
    y = x @ _unpack(s["wq"], s["ws"]).t()
    return (y if s["bias"] is None else y + s["bias"].float()).to(torch.bfloat16)


# ---- one pass ----

def run(state):
    op = state["case"]["op"]
    if own:
        return _own[op](state)
    if op == "quant":
        return _unpack(*_pack(*_encode(state["x"]))).to(torch.bfloat16)
    return {"norm": _plain_norm, "route": _plain_route, "linear": _plain_linear}[op](state)


def _own_norm(s):
    import moe_router_gemm_gb300 as m
    quant = s["case"]["quant"]
    r = m.rmsnorm(s["x"], s["weight"], s["residual"], eps=EPS, quant=None if quant == "none" else quant, scale=s["scale"])
    out = {"out": r.out}
    if s["residual"] is not None:
        out["residual"] = r.residual
    if quant != "none":
        out["codes"] = r.codes.view(torch.float8_e4m3fn)
    if quant == "mxfp8":
        out["scales"] = r.scales.view(torch.float8_e8m0fnu)
    return out


def _own_route(s):
    import moe_router_gemm_gb300 as m
    c = s["case"]
    w, ids = m.route(s["logits"], c["k"], scoring=c["scoring"], bias=s["bias"], groups=c["groups"], top_groups=c["top"],
                     group_best=c["best"])
    return {"weights": w, "ids": ids}


def _own_quant(s):
    import moe_router_gemm_gb300 as m
    return m.dequant_mxfp4(*m.quant_mxfp4(s["x"]))


def _own_linear(s):
    import moe_router_gemm_gb300 as m
    if s["case"]["dynamic"]:
        return m.bf16_linear_mxfp4_dynamic(s["x"], s["wq"], s["ws"], s["bias"])
    return m.bf16_linear_mxfp4(s["xq"], s["xs"], s["wq"], s["ws"], s["bias"])


_own = {"norm": _own_norm, "route": _own_route, "quant": _own_quant, "linear": _own_linear}


# ---- what a pass cannot do without ----

def work(case):
    if case["op"] == "norm":
        n = case["T"] * case["H"]
        b = 2 * n + 2 * case["H"] + 2 * n + (4 * n if case["residual"] else 0)  # x, weight, out, residual in and out
        b += {"none": 0, "fp8": n, "mxfp8": n + n // BLOCK}[case["quant"]]
        return {"bytes": b, "flops": 5 * n}
    if case["op"] == "route":
        n = case["T"] * case["E"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + 8 * case["T"] * case["k"], "flops": 4 * n}
    if case["op"] == "quant":  # bf16 in, codes and scales out and in again, bf16 out
        n = case["rows"] * case["K"]
        return {"bytes": 4 * n + 2 * (n // 2 + n // BLOCK), "flops": 4 * n}
    M, N, K = case["M"], case["N"], case["K"]
    x = 2 * M * K if case["dynamic"] else M * K // 2 + M * K // BLOCK
    return {"bytes": x + N * K // 2 + N * K // BLOCK + 2 * M * N + (2 * N if case["bias"] else 0), "flops": 2 * M * N * K}


# ---- the definitions in 64 bits ----

def _exp2(e):
    """2^e in fp64 for whole e, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _log2_floor(a):
    """floor(log2(a)) of positive fp64 values."""
    return ((a.view(torch.int64) >> 52) & 2047) - 1023


def _exact_fp4(x):
    """The values that MXFP4 keeps of x: each element rounded to its binade's step (half to even), largest 6 times the scale."""
    v = x.double().view(x.shape[0], -1, BLOCK)
    amax = v.abs().amax(-1, keepdim=True)
    scale = _exp2((_log2_floor(amax.clamp_min(2.0 ** -140)) - 2).clamp_min(-127))
    u = v / scale
    step = _exp2(_log2_floor(u.abs().clamp_min(1.0)) - 1)
    return (torch.round(u / step) * step).clamp(-6.0, 6.0).mul(scale).view(x.shape)


def _exact_values(q, s):
    code = torch.stack([q.int() & 15, q.int() >> 4], -1).view(q.shape[0], -1)
    mant, ex = (code & 1).double(), (code >> 1) & 3
    v = torch.where(ex == 0, 0.5 * mant, (1.0 + 0.5 * mant) * _exp2(ex - 1))
    v = torch.where(code > 7, -v, v)
    return v * _exp2(s.long() - 127).repeat_interleave(BLOCK, -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double()
        out = {}
        if s["residual"] is not None:
            out["residual"] = h + s["residual"].double()
            h = out["residual"].to(torch.bfloat16).double()  # the residual stream is bf16 by definition
        y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].double()
        out["out"] = y
        if case["quant"] == "fp8":
            out["codes"] = (y / s["scale"].double()).clamp(-448.0, 448.0)
        elif case["quant"] == "mxfp8":
            v = y.view(y.shape[0], -1, BLOCK)
            scale = _exp2((_log2_floor(v.abs().amax(-1).clamp_min(2.0 ** -140)) - 8).clamp_min(-127))
            out["codes"] = (v / scale.unsqueeze(-1)).clamp(-448.0, 448.0).view(y.shape)
            out["scales"] = scale
        return out
    if case["op"] == "route":
        x = s["logits"].double()
        score = torch.softmax(x, -1) if case["scoring"] == "softmax" else torch.sigmoid(x)
        key = score if s["bias"] is None else score + s["bias"].double()
        if case["scoring"] == "softmax":
            key = x
        key = key.masked_fill(x == float("-inf"), float("-inf"))
        if case["groups"] > 1:
            g = key.view(key.shape[0], case["groups"], -1)
            best = g.topk(min(case["best"], g.shape[-1]), -1).values.sum(-1)
            kept = torch.argsort(best, dim=-1, descending=True, stable=True)[:, : case["top"]]
            away = torch.ones_like(best).scatter_(1, kept, 0.0).bool()
            key = g.masked_fill(away.unsqueeze(-1), float("-inf")).view(key.shape)
        order = torch.argsort(key, dim=-1, descending=True, stable=True)[:, : case["k"]]
        w = torch.gather(score, 1, order)
        return {"weights": w / w.sum(-1, keepdim=True), "ids": None}
    if case["op"] == "quant":
        return _exact_fp4(s["x"])
    x = _exact_fp4(s["x"]) if case["dynamic"] else _exact_values(s["xq"], s["xs"])
    y = x @ _exact_values(s["wq"], s["ws"]).t()
    return y if s["bias"] is None else y + s["bias"].double()
