"""The checks of arguments of the grouping, the grouped and the adapters' linears and the combination, which need no GPU; the
tests' own 64-bit forms; the plain forms of perf/more_operators.py against its definitions."""
import ctypes as C
import random

import pytest
import torch

import more_cases
import rows_ref as ref

P = [C.c_void_p(v << 24) for v in range(1, 12)]
EINVAL, EALIGN, EUNSUPPORTED = -1, -2, -6
MAX_ROWS = (1 << 31) - 1 - 65536


def at(p, d):
    return C.c_void_p(p.value + d)


def test_group_rows_checks(lib):
    f = lib.load().bf16_group_rows
    i, o, r, p = P[:4]

    def call(i=i, T=4, k=2, g=8, o=o, r=r, p=None, flags=0):
        return f(i, T, k, g, o, r, p, flags, None)

    for bad in (dict(T=-1), dict(k=0), dict(k=-1), dict(g=0), dict(g=-5), dict(flags=3), dict(flags=4), dict(i=None), dict(o=None),
                dict(r=None), dict(r=i), dict(o=i), dict(p=i), dict(p=r), dict(o=r), dict(T=MAX_ROWS // 2 + 1), dict(T=1 << 62),
                dict(o=at(r, 28))):
        assert call(**bad) == EINVAL, bad
    assert call(g=1025) == EUNSUPPORTED
    for bad in (dict(i=at(i, 2)), dict(o=at(o, 1)), dict(r=at(r, 2)), dict(p=at(p, 3))):
        assert call(**bad) == EALIGN, bad


def test_linear_grouped_checks(lib):
    f = lib.load().bf16_linear_grouped
    x, w, b, o, r, y = P[:6]

    def call(x=x, xr=16, w=w, b=None, o=o, r=r, y=y, n=32, g=4, N=24, K=64, s=0, ws=None, wn=0, flags=0):
        return f(x, xr, w, b, o, r, y, n, g, N, K, s, ws, wn, flags, None)

    for bad in (dict(n=-1), dict(xr=-1), dict(g=0), dict(N=0), dict(K=0), dict(K=-8), dict(flags=3), dict(x=None), dict(w=None),
                dict(o=None), dict(y=None), dict(xr=0), dict(r=None), dict(y=x), dict(y=w), dict(y=at(o, -16)), dict(b=y), dict(r=y),
                dict(n=MAX_ROWS + 1), dict(xr=MAX_ROWS + 1), dict(xr=1 << 40), dict(g=1024, N=1 << 20, K=1 << 14)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(K=60), dict(g=1025), dict(N=(1 << 24) + 1), dict(K=(1 << 24) + 8)):
        assert call(**bad) == EUNSUPPORTED, bad
    for bad in (dict(x=at(x, 2)), dict(w=at(w, 8)), dict(b=at(b, 2)), dict(y=at(y, 4)), dict(o=at(o, 2)), dict(r=at(r, 2))):
        assert call(**bad) == EALIGN, bad
    assert call(n=0, x=None, y=None) == 0 and call(n=0, xr=0, r=None, s=1) == 0
    few = dict(n=2, g=4, N=64, K=7168)  # two tiles: K in parts
    need, ws = lib.grouped_workspace(*few.values()), P[6]
    assert need >= 2 * 4 * 2 * 64 and lib.grouped_workspace(*few.values(), True) >= 2 * 4 * 2 * 128
    assert call(**few) == call(**few, ws=ws, wn=need - 1) == call(**few, ws=y, wn=need) == call(**few, ws=x, wn=need) == EINVAL
    assert call(**few, ws=at(ws, 64), wn=need) == EALIGN
    assert lib.grouped_workspace(65536, 128, 4096, 7168) == lib.grouped_workspace(0, 4, 64, 7168) == 0
    assert lib.grouped_workspace(2, 1025, 64, 7168) == lib.grouped_workspace(1 << 40, 4, 64, 7168) == 0


def test_combine_rows_checks(lib):
    f = lib.load().bf16_combine_rows
    y, p, w, a, o = P[:5]

    def call(y=y, yr=32, p=p, w=w, a=None, o=o, T=4, k=8, H=64, flags=0):
        return f(y, yr, p, w, a, o, T, k, H, flags, None)

    for bad in (dict(T=-1), dict(yr=-1), dict(k=0), dict(H=0), dict(flags=3), dict(y=None), dict(p=None), dict(o=None), dict(o=y),
                dict(o=p), dict(o=w), dict(a=at(o, 16)), dict(T=1 << 60), dict(yr=1 << 60)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(y=at(y, 2)), dict(o=at(o, 2)), dict(a=at(a, 8)), dict(p=at(p, 2)), dict(w=at(w, 1))):
        assert call(**bad) == EALIGN, bad
    assert call(T=0, p=None, o=None) == 0


def test_linear_lora_checks(lib):
    f, need = lib.load().bf16_linear_lora, lib.lora_workspace(16, 24, 64, 8, 4)
    x, w, bi, a, b, s, i, o, ws = P[:9]

    def call(x=x, w=w, bi=None, a=a, b=b, s=None, i=i, o=o, M=16, N=24, K=64, R=8, L=4, ws=ws, n=need, flags=0):
        return f(x, w, bi, a, b, s, i, o, M, N, K, R, L, ws, n, flags, None)

    assert need > 0
    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(R=0), dict(L=0), dict(flags=3), dict(x=None), dict(w=None), dict(a=None),
                dict(b=None), dict(i=None), dict(o=None), dict(ws=None), dict(n=need - 1), dict(o=x), dict(o=w), dict(o=a), dict(o=b),
                dict(o=i), dict(ws=o), dict(ws=x), dict(s=o), dict(bi=o)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(K=60), dict(R=12), dict(R=136), dict(L=1025), dict(N=(1 << 24) + 1)):
        assert call(**bad) == EUNSUPPORTED, bad
    for bad in (dict(x=at(x, 2)), dict(w=at(w, 2)), dict(bi=at(bi, 2)), dict(a=at(a, 8)), dict(b=at(b, 4)), dict(o=at(o, 2)),
                dict(s=at(s, 2)), dict(i=at(i, 1)), dict(ws=at(ws, 16))):
        assert call(**bad) == EALIGN, bad
    assert call(M=0, x=None, o=None, ws=None, n=0) == 0
    assert lib.lora_workspace(16, 24, 60, 8, 4) == lib.lora_workspace(16, 24, 64, 12, 4) == lib.lora_workspace(-1, 24, 64, 8, 4) == 0
    assert lib.lora_workspace(16, 24, 1 << 32, 8, 4) == 0


def test_tensors_of_the_wrong_kind(lib):
    """What the Python side refuses before any call, on CPU tensors."""
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d)  # noqa: E731
    i32, f32 = torch.int32, torch.float32
    for f, err in ((lambda: lib.group_rows(z(4, 2, d=torch.int64), 8), TypeError), (lambda: lib.group_rows(z(4, 2, d=i32), 8), ValueError),
                   (lambda: lib.bf16_linear_grouped(z(4, 64, d=f32), z(2, 8, 64), z(3, d=i32)), TypeError),
                   (lambda: lib.bf16_linear_grouped(z(4, 64), z(2, 8, 64), z(3, d=i32)), ValueError),
                   (lambda: lib.combine_rows(z(4, 64), z(2, 2, d=i32)), ValueError),
                   (lambda: lib.bf16_linear_lora(z(4, 64), z(8, 64, d=f32), z(2, 8, 64), z(2, 8, 8), z(4, d=i32)), TypeError),
                   (lambda: lib.bf16_linear_lora(z(4, 64), z(8, 64), z(2, 8, 64), z(2, 8, 8), z(4, d=i32)), ValueError)):
        with pytest.raises(err):
            f()


def test_the_reference_forms():
    off, rows, place = ref.group(torch.tensor([[2, 0], [7, 2], [0, -1]], dtype=torch.int32), 4)
    assert off.tolist() == [0, 2, 2, 4, 4] and rows.tolist() == [0, 2, 0, 1, -1, -1]
    assert place.tolist() == [[2, 0], [-1, 3], [1, -1]]
    x, w = torch.tensor([[1.0, 2.0], [3.0, 4.0]]), torch.tensor([[[1.0, 0.0]], [[0.0, 2.0]]])
    y, _ = ref.grouped(x, w, torch.tensor([0, 1, 3]), None, torch.tensor([1, 0, 1]), False)
    assert y.tolist() == [[3.0], [4.0], [8.0]]
    y, _ = ref.grouped(x, torch.tensor([[[1.0, 0.0], [0.0, 1.0]]]), torch.tensor([0, 2]), torch.tensor([[0.0, 1.0]]), None, True)
    assert torch.allclose(y.view(-1), torch.tensor([3 / (1 + 2.718281828459045 ** -1), 15 / (1 + 2.718281828459045 ** -3)]).double())
    c, _ = ref.combine(x, torch.tensor([[0, 1], [5, 1]]), torch.tensor([[0.5, 2.0], [1.0, 1.0]]), torch.ones(2, 2))
    assert c.tolist() == [[7.5, 10.0], [4.0, 5.0]]
    y, _ = ref.lora(x, torch.eye(2), torch.ones(1, 1, 2), torch.tensor([[[1.0], [0.0]]]), torch.tensor([0, -1]), None,
                    torch.tensor([2.0]))
    assert y.tolist() == [[7.0, 2.0], [3.0, 4.0]]


@pytest.mark.parametrize("op", ["group", "experts", "combine", "lora"])
def test_plain_forms_of_the_cases(op):
    mod = more_cases.load("cpu", own=False)
    rng = random.Random(op)
    for i in range(6):
        case = more_cases.small(mod, rng, op)
        more_cases.check(mod, case, 11 + i)


def test_cases_are_what_they_say():
    mod = more_cases.load("cpu", own=False)
    listed = mod.listed()
    assert len({c["name"] for c in listed}) == len(listed) == 12
    most = {k: max(mod.work(c)[k] for c in listed) for k in ("bytes", "flops")}
    rng = random.Random(3)
    for _ in range(300):
        w = mod.work(mod.draw(rng))
        assert 0 < w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]


def test_lora_workspace_of_refused_sizes(lib):
    """No bytes for the sizes that the call refuses, on either side of each bound."""
    f = lib.lora_workspace
    top, wide = MAX_ROWS, 1 << 24
    assert f(16, 24, 64, 8, 1024) > 0 and f(16, wide, 64, 8, 4) > 0 and f(16, 24, wide, 8, 4) > 0 and f(top, 24, 64, 8, 4) > 0
    for sizes in ((16, 24, 64, 8, 1025), (16, wide + 1, 64, 8, 4), (16, 24, wide + 8, 8, 4), (top + 1, 24, 64, 8, 4), ((1 << 31) - 1, 24, 64, 8, 4),
                  (100, (1 << 31) - 1, 64, 16, 4), (16, 24, (1 << 31) - 8, 8, 4), (16, 24, 64, 8, (1 << 31) - 1), (16, wide, 64, 128, 1024),
                  (1 << 20, (1 << 20) + 1, 64, 8, 4), (16, 24, 64, 136, 4), (0, 24, 64, 8, 4)):
        assert f(*sizes) == 0, sizes


def test_grouped_workspace_of_refused_sizes(lib):
    """As above, at sizes of few tiles, whose K would go in parts."""
    f = lib.grouped_workspace
    assert f(2, 4, 64, 7168) > 0 and f(1, 1024, 4096, 1 << 18) > 0 and f(1, 1, 64, 1 << 24) > 0 and f(1, 1024, 2048, 1 << 18, True) > 0
    for sizes in ((2, 4, 64, 7164), (2, 4, 64, 7167), (1, 1024, 4096, (1 << 18) + 8), (1, 1024, 2048, 1 << 19, True), (1, 1, 64, (1 << 24) + 8),
                  (2, 1025, 64, 7168), (0, 4, 64, 7168), (2, 4, 0, 7168), (-2, 4, 64, 7168), (2, -4, 64, 7168)):
        assert f(*sizes) == 0, sizes


@pytest.mark.parametrize("off", [-1 << 32, 1 << 32, -1 << 40])
def test_workspaces_of_sizes_that_no_int_holds(lib, off):
    """Their low 32 bits are a size that has a workspace."""
    for f, sizes in ((lib.lora_workspace, (16, 24, 64, 8, 4)), (lib.grouped_workspace, (2, 4, 64, 7168)),
                     (lib.mxfp4_dynamic_workspace, (64, 256, 64))):
        assert f(*sizes) > 0
        for i, v in enumerate(sizes):
            assert f(*sizes[:i], v + off, *sizes[i + 1:]) == 0, (f.__name__, i)
