"""Measurement cases of the products whose weight depends on the row: experts' and adapters' linears, and what moves their rows.

Four operators that stand between a router's choice and the block's output:

  group    the pairs of a token and an expert, ordered by expert: where each expert's rows start,
           which token each row is of, and where each pair went;
  experts  out[p] = x[row of p] @ W[e]^T (+ bias[e]) for the rows p of each expert e, their number
           known on the device alone; with `swiglu`, W holds gate and up projections and
           out = silu(gate) * up;
  combine  a token's output from its rows: the weighted sum (+ what a shared expert gave);
  lora     out = x @ W^T (+ bias) + scale_a * (x @ A_a^T) @ B_a^T, each row with the low-rank
           adapter a of its request, or none.

Each has a plain form here (elementary torch operations in 32 bits) and, where ``own``
is true, the package's calls.  ``exact`` restates each in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # A decode batch's choice of experts: a launch's latency.
        dict(name="group 16x8 of 256", op="group", T=16, k=8, E=256, dropped=0.0),
        # A long prefill's, some pairs dropped (experts that live elsewhere).
        dict(name="group 8192x8 of 256", op="group", T=8192, k=8, E=256, dropped=0.1),
        # One decode token through its experts' gate and up projections: eight weights are read, each for one row.
        dict(name="experts 1x8 of 128 up", op="experts", T=1, k=8, E=128, N=2048, K=7168, swiglu=True, gather=True, bias=False),
        # An odd decode batch over few experts, sizes that no tile divides, with bias.
        dict(name="experts 13x4 of 32 up", op="experts", T=13, k=4, E=32, N=2880, K=2880, swiglu=True, gather=True, bias=True),
        # A multi-user decode batch's down projection: nearly all experts' weights, a few rows each.
        dict(name="experts 64x8 of 128 down", op="experts", T=64, k=8, E=128, N=7168, K=2048, swiglu=False, gather=False,
             bias=False),
        # A long prefill's gate and up projections: rows by the hundred for each expert.
        dict(name="experts 8192x8 of 128 up", op="experts", T=8192, k=8, E=128, N=2048, K=7168, swiglu=True, gather=True,
             bias=False),
        # The outputs of a small decode batch.
        dict(name="combine 4x8x2048", op="combine", T=4, k=8, H=2048, addend=False, dropped=0.0),
        # A long prefill's, with a shared expert's output.
        dict(name="combine 8192x8x7168", op="combine", T=8192, k=8, H=7168, addend=True, dropped=0.0),
        # One decode token, one of many small adapters, a square projection.
        dict(name="lora 1x4096x4096 r16", op="lora", T=1, N=4096, K=4096, R=16, L=64, runs=False, bare=0.0, bias=False),
        # An odd decode batch, requests of many adapters and some of none, the attention-input projection.
        dict(name="lora 61x2112x7168 r32", op="lora", T=61, N=2112, K=7168, R=32, L=24, runs=False, bare=0.2, bias=False),
        # A large decode batch through a dense MLP with bias.
        dict(name="lora 256x14336x4096 r16", op="lora", T=256, N=14336, K=4096, R=16, L=64, runs=False, bare=0.1, bias=True),
        # A prefill of several requests, one after another, each with its adapter.
        dict(name="lora 8192x7168x7168 r64", op="lora", T=8192, N=7168, K=7168, R=64, L=8, runs=True, bare=0.1, bias=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo=64):
    """A row length: one of the hidden sizes in use, or any multiple of 8."""
    if rng.random() < 0.4:
        return rng.choice([2048, 2880, 4096, 6144, 7168])
    return 8 * _log(rng, lo // 8, 7168 // 8)


def draw(rng):
    op = rng.choice(["group", "experts", "experts", "combine", "lora", "lora"])
    if op == "group":
        E = _log(rng, 2, 512)
        return dict(op=op, T=_log(rng, 1, 8192), k=rng.randint(1, min(8, E)), E=E, dropped=rng.choice([0.0, 0.0, 0.3]))
    if op == "combine":
        return dict(op=op, T=_log(rng, 1, 8192), k=rng.randint(1, 8), H=_log(rng, 64, 7168), addend=rng.random() < 0.5,
                    dropped=rng.choice([0.0, 0.2]))
    T, K, bias = _log(rng, 1, 8192), _width(rng), rng.random() < 0.3
    if op == "experts":
        E, swiglu = _log(rng, 2, 128), rng.random() < 0.5
        N = _log(rng, 32, 2048) if swiglu else _log(rng, 32, 7168)
        while E * N * (2 if swiglu else 1) > 128 * 2048:
            N = max(32, N // 2)
        return dict(op=op, T=T, k=rng.randint(1, min(8, E)), E=E, N=N, K=K, swiglu=swiglu, gather=rng.random() < 0.6, bias=bias)
    L, N = _log(rng, 1, 64), _log(rng, 64, 14336)
    while T * N * K > 8192 * 7168 * 7168:
        N = max(64, N // 2)
    return dict(op=op, T=T, N=N, K=K, R=8 * _log(rng, 1, 8), L=L, runs=rng.random() < 0.4, bare=rng.choice([0.0, 0.2]), bias=bias)


# ---- inputs ----

def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _weight(g, *shape):
    """A weight of unit gain; made in bf16, since a layer's experts are billions of elements."""
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16).mul_(shape[-1] ** -0.5)


def _activations(g, rows, K):
    """A hidden state: rows of differing size, and a few channels that run far above the others."""
    x = _randn(g, rows, K)
    x *= torch.exp2(0.5 * _randn(g, rows, 1))
    x *= torch.where(torch.rand(1, K, generator=g, device=DEV) < 0.01, 10.0, 1.0)
    return x.to(torch.bfloat16)


def _choice(g, T, k, E, dropped=0.0):
    """k different experts a token, some experts sought more than others; -1 where the pair is dropped."""
    ids = (_randn(g, T, E) + 0.5 * _randn(g, 1, E)).topk(k, -1).indices.int()
    return torch.where(torch.rand(T, k, generator=g, device=DEV) < dropped, -1, ids) if dropped else ids


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case=case)
    T = case["T"]
    if case["op"] == "group":
        s["ids"] = _choice(g, T, case["k"], case["E"], case["dropped"])
    elif case["op"] == "experts":
        k, E, N, K = case["k"], case["E"], case["N"], case["K"]
        ids = _choice(g, T, k, E).view(-1).long()
        s["offsets"] = torch.cat([ids.new_zeros(1), torch.bincount(ids, minlength=E).cumsum(0)]).int()
        s["rows"] = (torch.argsort(ids, stable=True) // k).int() if case["gather"] else None
        s["x"] = _activations(g, T if case["gather"] else T * k, K)
        s["w"] = _weight(g, E, 2 * N if case["swiglu"] else N, K)
        s["bias"] = (0.2 * _randn(g, *s["w"].shape[:2])).to(torch.bfloat16) if case["bias"] else None
    elif case["op"] == "combine":
        k, H = case["k"], case["H"]
        s["y"] = _activations(g, T * k, H)
        place = torch.randperm(T * k, generator=g, device=DEV).int().view(T, k)
        s["place"] = torch.where(torch.rand(T, k, generator=g, device=DEV) < case["dropped"], -1, place)
        w = torch.rand(T, k, generator=g, device=DEV) + 0.05
        s["weights"] = w / w.sum(-1, keepdim=True)
        s["addend"] = _activations(g, T, H) if case["addend"] else None
    else:
        N, K, R, L = case["N"], case["K"], case["R"], case["L"]
        s["x"], s["w"] = _activations(g, T, K), _weight(g, N, K)
        s["a"], s["b"] = _weight(g, L, R, K), _weight(g, L, N, R)
        s["scale"] = 0.5 + torch.rand(L, generator=g, device=DEV)
        s["bias"] = (0.2 * _randn(g, N)).to(torch.bfloat16) if case["bias"] else None
        requests = max(1, T // 512) if case["runs"] else T  # runs: tokens of a request stand together
        ends = torch.randint(0, T, (requests,), generator=g, device=DEV).sort().values
        of = torch.searchsorted(ends, torch.arange(T, device=DEV)).clamp_max(requests - 1) if case["runs"] else torch.arange(T, device=DEV)
        ids = torch.randint(0, L, (requests,), generator=g, device=DEV)
        ids = torch.where(torch.rand(requests, generator=g, device=DEV) < case["bare"], -1, ids)
        s["ids"] = ids[of].int()
    return s


# ---- plain forms: elementary operations in 32 bits ----

def _plain_group(s):
    ids, E, k = s["ids"].view(-1).long(), s["case"]["E"], s["case"]["k"]
    kept = (ids >= 0) & (ids < E)
    key = torch.where(kept, ids, E)
    order = key.sort(stable=True).indices
    counts = (key.unsqueeze(0) == torch.arange(E, device=key.device).unsqueeze(1)).sum(-1)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    at = torch.arange(key.numel(), device=key.device)
    place = torch.empty_like(order).scatter(0, order, at)
    return {"offsets": offsets.int(), "rows": torch.where(at < offsets[-1], order // k, -1).int(),
            "place": torch.where(kept, place, -1).int().view(s["ids"].shape)}


def _plain_experts(s):
    off, w = s["offsets"].long(), s["w"]
    x = s["x"].float() if s["rows"] is None else s["x"][s["rows"].long()].float()
    at = torch.arange(x.shape[0], device=x.device)
    e = (at.unsqueeze(1) >= off[1:].unsqueeze(0)).sum(-1)  # the expert of each row
    if x.shape[0] <= w.shape[0]:  # a weight for each row
        y = torch.bmm(w[e].float(), x.unsqueeze(-1)).squeeze(-1)
    else:  # every expert's rows in a block of the longest's size (a plain program asks the device for it)
        i = at - off[e]
        block = x.new_zeros(w.shape[0], int((off[1:] - off[:-1]).max()), x.shape[1])
        block[e, i] = x
        y = torch.bmm(block, w.float().transpose(1, 2))[e, i]
    if s["bias"] is not None:
        y = y + s["bias"][e].float()
    if s["case"]["swiglu"]:
        gate, up = y.chunk(2, -1)
        y = gate / (1.0 + torch.exp(-gate)) * up
    return y.to(torch.bfloat16)


def _plain_combine(s):
    y = s["y"][s["place"].clamp_min(0).long()].float()  # [T, k, H]
    y = (torch.where(s["place"] >= 0, s["weights"], 0.0).unsqueeze(-1) * y).sum(1)
    return (y if s["addend"] is None else y + s["addend"].float()).to(torch.bfloat16)


def _plain_lora(s):
    x, ids, (L, N, R) = s["x"].float(), s["ids"].long(), s["b"].shape
    y = x @ s["w"].float().t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    # Every adapter's inner values, those of a row's own adapter kept, and all adapters' second halves as one.
    mine = ids.unsqueeze(1) == torch.arange(L, device=ids.device).unsqueeze(0)
    h = (x @ s["a"].float().view(L * R, -1).t()).view(-1, L, R)
    h = torch.where(mine.unsqueeze(-1), h * s["scale"].view(1, L, 1), 0.0)
    return (y + h.view(-1, L * R) @ s["b"].float().transpose(1, 2).reshape(L * R, N)).to(torch.bfloat16)


# ---- one pass ----

def run(state):
    if own:
        return _own[state["case"]["op"]](state)
    return _plain[state["case"]["op"]](state)


def _own_group(s):
    import moe_router_gemm_gb300 as m
    r = m.group_rows(s["ids"], s["case"]["E"])
    return {"offsets": r.offsets, "rows": r.rows, "place": r.place}


def _own_experts(s):
    import moe_router_gemm_gb300 as m
    return m.bf16_linear_grouped(s["x"], s["w"], s["offsets"], s["bias"], rows=s["rows"], swiglu=s["case"]["swiglu"])


def _own_combine(s):
    import moe_router_gemm_gb300 as m
    return m.combine_rows(s["y"], s["place"], s["weights"], s["addend"])


def _own_lora(s):
    import moe_router_gemm_gb300 as m
    return m.bf16_linear_lora(s["x"], s["w"], s["a"], s["b"], s["ids"], s["bias"], scale=s["scale"])


_plain = {"group": _plain_group, "experts": _plain_experts, "combine": _plain_combine, "lora": _plain_lora}
_own = {"group": _own_group, "experts": _own_experts, "combine": _own_combine, "lora": _own_lora}


# ---- what a pass cannot do without ----

def work(case):
    T = case["T"]
    if case["op"] == "group":
        n = T * case["k"]
        return {"bytes": 12 * n + 4 * (case["E"] + 1), "flops": n}
    if case["op"] == "combine":
        n = T * case["H"]
        kept = case["k"] * (1.0 - case["dropped"])
        return {"bytes": int(2 * n * (kept + 1 + case["addend"])) + 8 * T * case["k"], "flops": int(2 * n * kept)}
    K, N = case["K"], case["N"]
    if case["op"] == "experts":
        E, P = case["E"], T * case["k"]
        used = E * (1.0 - (1.0 - case["k"] / E) ** T)  # experts that any token chose, were all sought alike
        wide = 2 * N if case["swiglu"] else N
        b = int(used) * wide * (2 * K + (2 if case["bias"] else 0)) + 2 * (T if case["gather"] else P) * K + 2 * P * N
        return {"bytes": b + 4 * (E + 1) + (4 * P if case["gather"] else 0), "flops": 2 * P * wide * K}
    R, L = case["R"], case["L"]
    requests = max(1, T // 512) if case["runs"] else T
    used = int(L * (1.0 - (1.0 - (1.0 - case["bare"]) / L) ** requests))  # adapters that any row has
    b = 2 * (T * K + N * K + T * N + used * R * (N + K)) + 4 * (T + L) + (2 * N if case["bias"] else 0)
    return {"bytes": b, "flops": 2 * T * N * K + int(2 * T * (1.0 - case["bare"]) * R * (N + K))}


# ---- the definitions in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "group":  # whole numbers; each pair's key is its own, so that any sort orders them
        ids, k, E = s["ids"].reshape(-1).long(), case["k"], case["E"]
        n = ids.numel()
        pairs = torch.nonzero((ids >= 0) & (ids < E)).view(-1)
        at = torch.sort(ids[pairs] * n + pairs).values
        rows, place = ids.new_full((n,), -1), ids.new_full((n,), -1)
        rows[: at.numel()] = at % n // k
        place[at % n] = torch.arange(at.numel(), device=DEV)
        offsets = torch.searchsorted(at // n, torch.arange(E + 1, device=DEV))
        return {"offsets": offsets.int(), "rows": rows.int(), "place": place.int().view(s["ids"].shape)}
    if case["op"] == "experts":
        ends = s["offsets"].tolist()
        out = torch.zeros(ends[-1], case["N"], dtype=torch.float64, device=DEV)
        for e in range(case["E"]):
            lo, hi = ends[e], ends[e + 1]
            if lo == hi:
                continue
            x = s["x"][lo:hi] if s["rows"] is None else s["x"].index_select(0, s["rows"][lo:hi].long())
            y = x.double() @ s["w"][e].double().t()
            if case["bias"]:
                y += s["bias"][e].double()
            if case["swiglu"]:
                y = y[:, : case["N"]] * torch.sigmoid(y[:, : case["N"]]) * y[:, case["N"]:]
            out[lo:hi] = y
        return out
    if case["op"] == "combine":
        out = torch.zeros(case["T"], case["H"], dtype=torch.float64, device=DEV) if s["addend"] is None else s["addend"].double()
        for j in range(case["k"]):
            have = (s["place"][:, j] >= 0).nonzero().view(-1)
            out[have] += s["weights"][have, j, None].double() * s["y"][s["place"][have, j].long()].double()
        return out
    out = s["x"].double() @ s["w"].double().t()
    if case["bias"]:
        out += s["bias"].double()
    for a in range(case["L"]):
        mine = (s["ids"] == a).nonzero().view(-1)
        if mine.numel():
            h = s["x"][mine].double() @ s["a"][a].double().t()
            out[mine] += s["scale"][a].double() * (h @ s["b"][a].double().t())
    return out
