"""bf16_route against its 64-bit form.

Ids: the keys of the picks, in f64, must run downwards and none may lie below a key left out, to within KEY: scores and
bias below 2 in magnitude, an exponential of 2 ulp, a sum of at most 37 terms in a row and a few roundings stay below
64 * 2^-24 = 2^-18.  Where the keys are exact (logits as keys, values that fp32 holds), ids must be equal.  Weights: an
argument l - m of magnitude at most 30 off by 2^-24 of itself, the sums and roundings: 30 + 37 + 16 times 2^-24 < 2^-17.
"""
import numpy as np
import pytest
import torch

import moe_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KEY, WEIGHT = 2.0 ** -18, 2.0 ** -17


def _check(lib, logits, k, exact_ids=False, **kw):
    w, ids = lib.route(logits, k, **kw)
    T, E = logits.shape
    full = dict(scoring="softmax", bias=None, groups=1, top_groups=1, group_best=1, renormalize=True, scale=1.0)
    full.update(kw)
    scale = full["scale"]
    if full["bias"] is not None:
        full["bias"] = ref.f64(full["bias"])
    key, score, allowed = ref.route(ref.f64(logits), k, **full)
    i = ids.cpu().numpy().astype(np.int64)
    assert i.shape == (T, k) and (i >= 0).all() and (i < E).all()
    assert all(len(set(r)) == k for r in i.tolist())
    assert np.take_along_axis(allowed, i, 1).all()
    masked = np.where(allowed, key, -np.inf)
    if exact_ids:
        order = np.array([sorted(range(E), key=lambda e: (not allowed[t, e], -key[t, e], e))[:k] for t in range(T)])
        assert np.array_equal(i, order)
    else:
        got = np.take_along_axis(masked, i, 1)
        with np.errstate(invalid="ignore"):
            assert (np.diff(got, axis=1)[np.isfinite(got[:, 1:])] <= KEY).all()
        rest = masked.copy()
        np.put_along_axis(rest, i, -np.inf, 1)
        assert (rest.max(-1) <= got.min(-1) + KEY).all()
    s = np.take_along_axis(score, i, 1)
    if full["renormalize"]:
        total = s.sum(-1, keepdims=True)
        s = s / np.where(total == 0, 1.0, total)
    want = s * scale
    assert (np.abs(ref.f64(w) - want) <= WEIGHT * np.abs(want) + 2.0 ** -126).all()
    return w, ids


def _logits(T, E, seed, dtype=torch.float32, ld=None):
    g = torch.Generator().manual_seed(seed)
    return (2 * torch.randn(T, ld or E, generator=g)).to(dtype).to(DEV)[:, :E]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (5, 8, 2), (7, 33, 5), (16, 128, 4), (31, 100, 32),
                                   (65, 384, 6), (3, 512, 10), (2, 1000, 16), (2, 1024, 1), (1, 32, 32), (9, 160, 6), (5, 96, 3), (6, 192, 7), (40, 384, 8), (3, 700, 12), (8, 383, 8)])
def test_softmax(lib, T, E, k, dtype):
    _check(lib, _logits(T, E, T + E, dtype), k, exact_ids=True)
    _check(lib, _logits(T, E, T + E + 1, dtype, ld=E + 3), k, exact_ids=True, renormalize=False, scale=2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 8, 3), (33, 256, 8), (4, 77, 7), (2, 1024, 32)])
def test_bias_ranks_but_does_not_weigh(lib, T, E, k, scoring):
    g = torch.Generator().manual_seed(E)
    bias = (0.3 * torch.randn(E, generator=g)).to(DEV)
    _check(lib, _logits(T, E, T), k, scoring=scoring, bias=bias)
    _check(lib, _logits(T, E, T, torch.bfloat16), k, scoring=scoring, bias=bias, renormalize=False)


@pytest.mark.parametrize("scoring,best", [("softmax", 1), ("softmax", 2), ("sigmoid", 1), ("sigmoid", 2)])
@pytest.mark.parametrize("T,E,k,groups,top", [(33, 256, 8, 8, 4), (5, 64, 6, 4, 1), (3, 160, 6, 8, 3), (9, 96, 5, 32, 3),
                                              (4, 15, 2, 5, 2), (2, 1024, 8, 8, 2), (70, 384, 8, 8, 3), (9, 384, 6, 4, 2), (5, 192, 4, 2, 1),
                                              (8, 96, 4, 3, 2), (11, 768, 9, 16, 5), (3, 160, 5, 4, 2), (6, 24, 12, 2, 1), (7, 14, 4, 7, 2)])
def test_groups(lib, T, E, k, groups, top, scoring, best):
    g = torch.Generator().manual_seed(E + groups)
    bias = (0.2 * torch.randn(E, generator=g)).to(DEV) if scoring == "sigmoid" else None
    _check(lib, _logits(T, E, E + T), k, scoring=scoring, bias=bias, groups=groups, top_groups=top, group_best=best,
           exact_ids=scoring == "softmax" and best == 1)


@pytest.mark.parametrize("scoring,best", [("softmax", 1), ("sigmoid", 2)])
@pytest.mark.parametrize("T,E,k,groups,top", [(50, 240, 14, 16, 9), (7, 336, 10, 16, 1), (9, 272, 4, 8, 5), (6, 288, 11, 8, 1),
                                              (5, 382, 8, 2, 1), (8, 300, 8, 12, 4), (4, 1023, 9, 3, 2), (3, 1000, 9, 20, 7),
                                              (9, 34, 3, 17, 4), (5, 62, 30, 31, 29), (3, 1023, 31, 31, 30), (6, 40, 6, 4, 3)])
@pytest.mark.parametrize("dtype,pad", [(torch.float32, 0), (torch.bfloat16, 4), (torch.float32, 1)])
def test_groups_of_any_size(lib, T, E, k, groups, top, scoring, best, dtype, pad):
    g = torch.Generator().manual_seed(E + groups)
    bias = (0.2 * torch.randn(E, generator=g)).to(DEV) if scoring == "sigmoid" else None
    _check(lib, _logits(T, E, E + T, dtype, ld=E + pad), k, scoring=scoring, bias=bias, groups=groups, top_groups=top,
           group_best=best, exact_ids=scoring == "softmax" and best == 1)


def test_ties_go_to_the_lowest_index(lib):
    g = torch.Generator().manual_seed(0)
    for E, groups, top in [(256, 1, 1), (256, 8, 3), (100, 1, 1), (60, 5, 2), (1024, 1, 1)]:
        logits = torch.randint(-2, 3, (40, E), generator=g).float().to(DEV)
        _check(lib, logits, 8, exact_ids=True, groups=groups, top_groups=top)
        zero = logits * 0.0
        zero[:, ::2] = -0.0  # equal to +0
        _check(lib, zero, 8, exact_ids=True, groups=groups, top_groups=top)
        w, ids = lib.route(zero, 8, scoring="sigmoid", groups=groups, top_groups=top)
        assert (ids == torch.arange(8, device=DEV)).all() and (w == 0.125).all()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [48, 256])
def test_masked_experts(lib, E, scoring):
    logits = _logits(12, E, 4)
    bias = torch.full((E,), 3.0, device=DEV)
    logits[:, 5:E - 3] = -float("inf")     # eight are left
    kw = dict(scoring=scoring, bias=bias if scoring == "sigmoid" else None)
    _check(lib, logits, 8, exact_ids=scoring == "softmax", **kw)
    w, ids = _check(lib, logits, 10, **kw)  # two of the masked ones have to join, lowest first, without weight
    assert (ids[:, 8:] == torch.tensor([5, 6], device=DEV)).all() and (w[:, 8:] == 0).all()
    logits[3] = -float("inf")              # a row whose mask leaves nothing
    w, ids = lib.route(logits, 4, **kw)
    assert (w[3] == 0).all() and ids[3].tolist() == [0, 1, 2, 3]
    w, ids = lib.route(logits, 4, renormalize=False, **kw)
    assert (w[3] == 0).all()


def test_lowest_value_masks_and_extremes(lib):
    low = torch.finfo(torch.float32).min
    logits = _logits(6, 64, 9)
    logits[0] = low                        # the type's lowest value throughout: all equal, none out
    logits[1, 10:] = low
    logits[2] = 1e30 * logits[2].sign() + torch.arange(64, device=DEV)
    w, ids = lib.route(logits, 4)
    assert ids[0].tolist() == [0, 1, 2, 3] and (w[0] == 0.25).all()
    assert (ids[1] < 10).all() and torch.isfinite(w).all()
    w, ids = lib.route(logits, 4, scoring="sigmoid")
    assert torch.isfinite(w).all() and (w[0] == 0).all()


def test_nan_logits(lib):
    logits = _logits(4, 64, 6)
    clean, cids = lib.route(logits, 4)
    logits[1, 20] = float("nan")
    w, ids = lib.route(logits, 4)
    assert w[1].isnan().all() and torch.equal(w[[0, 2, 3]], clean[[0, 2, 3]])
    assert all(len(set(r)) == 4 for r in ids.tolist()) and 20 not in ids[1].tolist()
    ws, ids = lib.route(logits, 4, scoring="sigmoid")
    assert torch.isfinite(ws).all() and 20 not in ids[1].tolist()
    logits[2] = float("nan")
    _, ids = lib.route(logits, 4)
    assert ids[2].tolist() == [0, 1, 2, 3]


def test_many_tokens_equal_few(lib):
    """Every token's answer is its own: a long batch, another stream, and each row alone."""
    logits = _logits(30001, 256, 12)
    bias = 0.1 * torch.randn(256, device=DEV)
    kw = dict(scoring="sigmoid", bias=bias, groups=8, top_groups=4, group_best=2)
    w, ids = lib.route(logits, 8, **kw)
    for at in (0, 17, 29999, 30000):
        w1, i1 = lib.route(logits[at:at + 1].clone(), 8, **kw)
        assert torch.equal(w1[0], w[at]) and torch.equal(i1[0], ids[at])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    w2, i2 = lib.route(logits, 8, stream=s, **kw)
    s.synchronize()
    assert torch.equal(w, w2) and torch.equal(ids, i2)


def test_offsets_past_32_bits(lib):
    T, ld = 17000, 260000
    logits = torch.empty(T, ld, dtype=torch.bfloat16, device=DEV)
    logits[:, :64] = torch.randn(T, 64, device=DEV).to(torch.bfloat16)
    assert T * ld > 2 ** 32
    w, ids = lib.route(logits[:, :64], 4)
    w1, i1 = lib.route(logits[:, :64].contiguous(), 4)
    assert torch.equal(w, w1) and torch.equal(ids, i1)


def test_empty_and_refusals(lib):
    w, ids = lib.route(_logits(1, 64, 1)[:0], 4)
    assert w.shape == (0, 4) and ids.shape == (0, 4)
    x = _logits(4, 64, 1)
    for kw in (dict(k=0), dict(k=65), dict(k=4, groups=5), dict(k=4, groups=8, top_groups=9),
               dict(k=17, groups=4, top_groups=1), dict(k=1, group_best=3), dict(k=1, groups=64, group_best=2)):
        k = kw.pop("k")
        with pytest.raises(lib.BF16LinearError) as e:
            lib.route(x, k, **kw)
        assert e.value.status in (-1, -6)
    with pytest.raises(lib.BF16LinearError) as e:
        lib.route(_logits(1, 1025, 1), 2)
    assert e.value.status == -6
    with pytest.raises(ValueError):
        lib.route(x, 2, scoring="relu")
    with pytest.raises(ValueError):
        lib.route(x, 2, bias=torch.zeros(63, device=DEV))
    with pytest.raises(TypeError):
        lib.route(x.double(), 2)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_scores_without_a_value(lib, bad):
    """A NaN or +inf logit leaves a softmax row no scores: ranked by logits the choice stands, ranked by scores it is the lowest."""
    logits = _logits(3, 64, 2)
    logits[1, 20] = bad
    best = torch.where(torch.isnan(logits[1]), -float("inf"), logits[1]).sort(descending=True, stable=True).indices[:4]
    w, ids = lib.route(logits, 4)
    assert w[1].isnan().all() and ids[1].tolist() == best.tolist() and not w[[0, 2]].isnan().any()
    for kw in (dict(bias=torch.rand(64, device=DEV)), dict(groups=8, top_groups=2, group_best=2)):
        w, ids = lib.route(logits, 4, **kw)
        assert w[1].isnan().all() and ids[1].tolist() == [0, 1, 2, 3] and not w[[0, 2]].isnan().any()
