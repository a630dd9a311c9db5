"""Grouping, the grouped linear, the combination and the adapters' linear on the GPU, against the 64-bit forms of rows_ref."""
import random

import pytest
import torch

import more_cases
import rows_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _bf16(g, *shape, scale=1.0):
    return (scale * torch.randn(*shape, generator=g, device=DEV)).to(torch.bfloat16)


# ---- grouping ----

@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 8), (3, 2, 5), (16, 8, 256), (33, 6, 384), (100, 1, 64), (512, 8, 256), (513, 8, 256),
                                   (1000, 4, 1024), (2047, 6, 384), (8192, 8, 256), (40000, 7, 3), (100, 300, 17)])
@pytest.mark.parametrize("out", [0.0, 0.3, 1.0])
def test_group_rows(lib, T, k, E, out):
    g = _gen(T + k + E)
    ids = torch.randint(0, E, (T, k), generator=g, device=DEV, dtype=torch.int32)
    away = torch.rand(T, k, generator=g, device=DEV)
    ids = torch.where(away < out, torch.where(away < out / 2, -1 - ids, E + ids), ids)
    got = lib.group_rows(ids, E)
    for name, a, b in zip(got._fields, got, ref.group(ids.cpu(), E)):
        assert a.dtype == torch.int32 and torch.equal(a.cpu(), b), name


def test_group_rows_extremes(lib):
    ids = torch.tensor([-2 ** 31, 2 ** 31 - 1, 0, 1023, 1024, -1], dtype=torch.int32, device=DEV)
    got = lib.group_rows(ids, 1024)
    assert got.place.tolist() == [-1, -1, 0, 1, -1, -1] and got.rows.tolist() == [2, 3, -1, -1, -1, -1]
    assert got.offsets.tolist() == [0] + [1] * 1023 + [2]
    same = lib.group_rows(torch.full((70000,), 5, dtype=torch.int32, device=DEV), 9)  # one group has all
    assert torch.equal(same.place, torch.arange(70000, device=DEV, dtype=torch.int32)) and torch.equal(same.rows, same.place)
    assert same.offsets.tolist() == [0] * 6 + [70000] * 4
    none = lib.group_rows(torch.empty(0, 3, dtype=torch.int32, device=DEV), 6)
    assert none.offsets.tolist() == [0] * 7 and none.rows.numel() == none.place.numel() == 0


# ---- the grouped linear ----

def _problem(T, k, E, N, K, seed, swiglu=False, bias=False, gather=True, counts=None):
    """Rows of E groups (their counts given, or by chance), with x either the tokens or the rows themselves."""
    g = _gen(seed)
    if counts is None:
        ids = torch.rand(T, E, generator=g, device=DEV).topk(k, -1).indices.view(-1)
        rows = (ids.argsort(stable=True) // k).int()
        off = torch.cat([ids.new_zeros(1), torch.bincount(ids, minlength=E).cumsum(0)]).int()
    else:
        off = torch.tensor([0] + counts, device=DEV).cumsum(0).int()
        rows = torch.randint(0, T, (int(off[-1]),), generator=g, device=DEV, dtype=torch.int32)
    wide = 2 * N if swiglu else N
    x = _bf16(g, T if gather else rows.numel(), K)
    return dict(x=x, w=_bf16(g, E, wide, K, scale=K ** -0.5), offsets=off, bias=_bf16(g, E, wide) if bias else None,
                rows=rows if gather else None, swiglu=swiglu)


def _check(lib, p, what=""):
    got = lib.bf16_linear_grouped(p["x"], p["w"], p["offsets"], p["bias"], rows=p["rows"], swiglu=p["swiglu"])
    want, slack = ref.grouped(**p)
    ref.check(got[: want.shape[0]], want, slack, what)
    assert lib.device_status() == 0
    return got


SHAPES = [(1, 1, 1, 1, 8), (1, 8, 8, 64, 64), (1, 8, 128, 300, 2048), (3, 2, 5, 33, 72), (13, 4, 32, 288, 2880), (16, 8, 16, 128, 7168),
          (64, 8, 24, 256, 512), (70, 3, 4, 130, 136), (200, 2, 3, 257, 640), (513, 4, 7, 640, 1024), (1000, 1, 1, 384, 256),
          (700, 6, 6, 95, 200), (2048, 2, 5, 512, 320), (40, 8, 1024, 40, 64), (300, 1, 300, 16, 16)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("gather", [False, True])
def test_linear_grouped(lib, shape, swiglu, gather):
    T, k, E, N, K = shape
    _check(lib, _problem(T, k, E, N, K, sum(shape), swiglu, bias=(T + swiglu) % 2 == 0, gather=gather), str(shape))


COUNTS = [[0, 0, 0], [1], [0, 1, 0], [5, 0, 0, 7], [255, 257, 0, 1, 256], [31, 33, 32, 1, 63, 65], [1000, 0, 3], [15, 16, 17, 127, 128, 129],
          [0] * 40 + [9] + [0] * 40, [511, 513, 512], [3] * 90, [1, 2000, 1]]


@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c))[:40])
@pytest.mark.parametrize("swiglu", [False, True])
def test_ragged_groups(lib, counts, swiglu):
    for gather in (True, False):
        _check(lib, _problem(max(1, sum(counts) // 2), 0, len(counts), 200, 328, len(counts), swiglu, True, gather, counts), str(counts))


def test_rows_of_no_group_stay(lib):
    p = _problem(50, 0, 4, 72, 128, 1, counts=[9, 0, 20, 4])
    rows = torch.cat([p["rows"], torch.full((17,), -1, dtype=torch.int32, device=DEV)])
    out = torch.full((50, 72), 7.0, dtype=torch.bfloat16, device=DEV)
    lib.bf16_linear_grouped(p["x"], p["w"], p["offsets"], rows=rows, out=out)
    want, slack = ref.grouped(**p)
    ref.check(out[:33], want, slack)
    assert (out[33:] == 7.0).all()
    # rows before the first group, too
    lib.bf16_linear_grouped(p["x"], p["w"], p["offsets"] + 3, rows=torch.cat([rows[:3], rows[:-3]]), out=out.fill_(7.0))
    ref.check(out[3:36], want, slack)
    assert (out[:3] == 7.0).all() and (out[36:] == 7.0).all()


def test_offsets_and_rows_out_of_range_stay_inside(lib):
    """Offsets that fall or pass the end, rows outside x: taken as the contract says, nothing else is read or written."""
    p = _problem(20, 0, 5, 40, 64, 2, counts=[4, 4, 4, 4, 4])
    full = torch.full((24, 40), 7.0, dtype=torch.bfloat16, device=DEV)
    out = full[2:22]
    off = torch.tensor([-5, 6, 3, 10, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV)
    lib.bf16_linear_grouped(p["x"], p["w"], off, rows=p["rows"], out=out)
    assert (full[:2] == 7.0).all() and (full[22:] == 7.0).all()
    rows = p["rows"].clone()
    rows[3], rows[5] = -9, 1000
    got = lib.bf16_linear_grouped(p["x"], p["w"], p["offsets"], rows=rows)
    want, slack = ref.grouped(**{**p, "rows": rows.clamp(0, 19)})
    ref.check(got, want, slack)
    assert lib.device_status() == 0


def test_not_finite_rows_stay_their_own(lib):
    """A NaN or an infinity in a row of x shows in that row's outputs alone; an infinite gate goes through SwiGLU."""
    for swiglu in (False, True):
        p = _problem(64, 2, 6, 100, 192, 5, swiglu, gather=False)
        clean = lib.bf16_linear_grouped(p["x"], p["w"], p["offsets"], swiglu=swiglu)
        x = p["x"].clone()
        x[7, 100], x[20, 5], x[41] = float("nan"), float("inf"), 3e38
        got = lib.bf16_linear_grouped(x, p["w"], p["offsets"], swiglu=swiglu)
        keep = torch.ones(128, dtype=torch.bool, device=DEV)
        keep[[7, 20, 41]] = False
        assert torch.equal(got[keep], clean[keep]) and got[7].isnan().all()
        assert not got[20].isfinite().any() if not swiglu else True


def test_swiglu_of_large_gates(lib):
    """Gates from -200 to 200: the exponential overflows and underflows without NaN."""
    g = torch.linspace(-200, 200, 41, device=DEV)
    x = torch.eye(8, device=DEV).to(torch.bfloat16)[:1]
    w = torch.zeros(1, 82, 8, device=DEV)
    w[0, :41, 0], w[0, 41:, 0] = g, 2.0
    w = w.to(torch.bfloat16)
    off = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    got = lib.bf16_linear_grouped(x, w, off, swiglu=True)
    want, slack = ref.grouped(x, w, off, None, None, True)
    ref.check(got, want, slack)


def test_groups_do_not_touch_one_another(lib):
    """A group's rows give the same bits alone and among others."""
    p = _problem(90, 0, 6, 264, 520, 9, True, True, counts=[40, 3, 300, 0, 17, 140])
    whole = lib.bf16_linear_grouped(p["x"], p["w"], p["offsets"], p["bias"], rows=p["rows"], swiglu=True)
    ends = p["offsets"].tolist()
    for e in range(6):
        off = p["offsets"].clone()
        off[: e + 1], off[e + 1:] = ends[e], ends[e + 1]
        alone = torch.zeros_like(whole)
        lib.bf16_linear_grouped(p["x"], p["w"], off, p["bias"], rows=p["rows"], swiglu=True, out=alone)
        assert torch.equal(alone[ends[e]:ends[e + 1]], whole[ends[e]:ends[e + 1]])
        assert (alone[: ends[e]] == 0).all() and (alone[ends[e + 1]:] == 0).all()


@pytest.mark.parametrize("T,k,E,N,K", [(1, 1, 1, 64, 7168), (2, 2, 10, 41, 7168), (1, 4, 8, 300, 2888), (60, 1, 2, 530, 1024), (20, 7, 15, 85, 6792)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_few_tiles(lib, T, k, E, N, K, swiglu):
    """K in parts, through a workspace whose contents do not matter; rows of no group stay."""
    for gather in (True, False):
        p = _problem(T, k, E, N, K, T + k, swiglu, True, gather)
        got = _check(lib, p, str((T, k, E, N, K)))
        need = lib.grouped_workspace(T * k, E, N, K, swiglu)
        assert need > 0
        space = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
        again = lib.bf16_linear_grouped(p["x"], p["w"], p["offsets"], p["bias"], rows=p["rows"], swiglu=swiglu, workspace=space)
        assert torch.equal(again, got)
    p = _problem(12, 0, 3, N, K, 3, swiglu, counts=[2, 0, 5])
    out = torch.full((12, N), 7.0, dtype=torch.bfloat16, device=DEV)
    rows = torch.cat([p["rows"], p["rows"][:5]])
    assert lib.grouped_workspace(12, 3, N, K, swiglu) > 0
    lib.bf16_linear_grouped(p["x"], p["w"], p["offsets"] + 2, rows=torch.cat([rows[:2], rows[:10]]), swiglu=swiglu, out=out)
    want, slack = ref.grouped(**p)
    ref.check(out[2:9], want, slack)
    assert (out[:2] == 7.0).all() and (out[9:] == 7.0).all()


def test_many_weights(lib):
    """Weights past 2^31 elements: an expert far into them."""
    E, N, K = 40, 8192, 7168
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device=DEV)
    w[37] = _bf16(_gen(1), N, K, scale=K ** -0.5)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[38:] = 5
    x = _bf16(_gen(2), 5, K)
    got = lib.bf16_linear_grouped(x, w, off)
    want, slack = ref.grouped(x, w[37:38], torch.tensor([0, 5]), None, None, False)
    ref.check(got, want, slack)


def test_long_out(lib):
    """Rows of out past 2^31 elements, in a group of 270,000 rows, and from x as it stands."""
    counts, N, K = [3, 269997], 8200, 64
    for gather in (True, False):
        p = _problem(1000, 0, 2, N, K, 6, gather=gather, counts=counts)
        got = lib.bf16_linear_grouped(p["x"], p["w"], p["offsets"], rows=p["rows"])
        at = torch.tensor([0, 2, 3, 131071, 262144, 269744, 269999], device=DEV)
        x = p["x"][p["rows"][at].long()] if gather else p["x"][at]
        off = torch.tensor([0, 2, 7], device=DEV)
        ref.check(got[at], *ref.grouped(x, p["w"], off, None, None, False))
        del got, p


def test_long_combine(lib):
    """Rows of y past 2^31 elements."""
    H = 8192
    y = torch.zeros(270000, H, dtype=torch.bfloat16, device=DEV)
    y[269990:] = _bf16(_gen(3), 10, H)
    place = torch.arange(269990, 270000, device=DEV, dtype=torch.int32).view(5, 2)
    w = torch.rand(5, 2, generator=_gen(4), device=DEV)
    got = lib.combine_rows(y, place, w)
    ref.check(got, *ref.combine(y[269990:], place - 269990, w, None))


# ---- combination ----

@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (1, 8, 2048), (4, 8, 7168), (7, 3, 33), (100, 6, 130), (33, 32, 2884), (1000, 2, 66), (2000, 8, 1024)])
@pytest.mark.parametrize("addend", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_combine_rows(lib, T, k, H, addend, weighted):
    g = _gen(T + k + H)
    y = _bf16(g, T * k + 3, H)
    place = torch.randint(-2, T * k + 6, (T, k), generator=g, device=DEV, dtype=torch.int32)  # some outside, some twice
    w = torch.rand(T, k, generator=g, device=DEV) if weighted else None
    a = _bf16(g, T, H) if addend else None
    got = lib.combine_rows(y, place, w, a)
    want, slack = ref.combine(y, place, w, a)
    ref.check(got, want, slack)
    if addend:  # in place
        lib.combine_rows(y, place, w, a, out=a)
        assert torch.equal(a, got)


def test_combine_of_nothing(lib):
    y = torch.full((2, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    away = torch.tensor([[-1, 2], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device=DEV)
    assert (lib.combine_rows(y, away) == 0).all()  # rows outside are not read, whatever they hold
    assert (lib.combine_rows(y[:0], away) == 0).all()
    assert lib.combine_rows(y, away[:0]).shape == (0, 64)


# ---- adapters ----

def _lora_problem(M, N, K, R, L, seed, bare=0.2, bias=False, scale=True, runs=False):
    g = _gen(seed)
    ids = torch.randint(0, L, (M,), generator=g, device=DEV, dtype=torch.int32)
    if runs:
        ids = ids.sort().values[torch.arange(M, device=DEV).flip(0)].contiguous()
    away = torch.rand(M, generator=g, device=DEV)
    ids = torch.where(away < bare, torch.where(away < bare / 2, -1 - ids, L + ids), ids)
    return dict(x=_bf16(g, M, K), w=_bf16(g, N, K, scale=K ** -0.5), a=_bf16(g, L, R, K, scale=K ** -0.5),
                b=_bf16(g, L, N, R, scale=R ** -0.5), ids=ids, bias=_bf16(g, N) if bias else None,
                scale=torch.randn(L, generator=g, device=DEV) if scale else None)


def _check_lora(lib, p, what="", **kw):
    got = lib.bf16_linear_lora(p["x"], p["w"], p["a"], p["b"], p["ids"], p["bias"], scale=p["scale"], **kw)
    ref.check(got, *ref.lora(**p), what)
    assert lib.device_status() == 0
    return got


LORA = [(1, 1, 8, 8, 1), (2, 333, 7168, 40, 3), (4, 1001, 9000, 128, 5), (4, 70, 16384, 16, 2), (1, 515, 4104, 8, 4), (3, 64, 16384, 64, 9), (2, 130, 12288, 128, 3), (2, 65, 12296, 8, 3), (1, 77, 24576, 16, 4), (1, 4096, 4096, 16, 64), (3, 33, 72, 8, 2), (8, 256, 2880, 32, 5), (16, 2112, 7168, 64, 8), (61, 300, 1024, 24, 7),
        (64, 1000, 512, 128, 70), (129, 257, 320, 40, 3), (200, 640, 136, 16, 200), (513, 520, 256, 72, 4), (1030, 384, 640, 64, 9),
        (2048, 130, 64, 96, 1000), (300, 77, 2048, 8, 1), (2000, 1024, 1024, 128, 2), (65, 5000, 136, 24, 30), (300, 9999, 72, 8, 100),
        (1500, 4100, 320, 128, 40), (435, 377, 5944, 32, 2), (90, 905, 7168, 16, 12), (1081, 116, 2048, 16, 4), (300, 250, 1536, 104, 300), (700, 4104, 2056, 48, 500), (256, 14336, 256, 16, 64), (520, 6144, 640, 80, 3)]


@pytest.mark.parametrize("shape", LORA, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("runs", [False, True])
def test_linear_lora(lib, shape, runs):
    M, N, K, R, L = shape
    for i, bare in enumerate((0.2, 0.0, 1.0)):
        p = _lora_problem(M, N, K, R, L, sum(shape) + i, bare, bias=(M + i) % 2 == 1, scale=i != 1, runs=runs)
        got = _check_lora(lib, p, f"{shape} {bare}")
        space = torch.full((lib.lora_workspace(M, N, K, R, L),), 255, dtype=torch.uint8, device=DEV)  # its contents do not matter
        assert torch.equal(_check_lora(lib, p, workspace=space), got)


@pytest.mark.parametrize("R", range(8, 129, 8))
@pytest.mark.parametrize("M,N", [(3, 777), (17, 130), (64, 5001)])
def test_lora_of_every_rank(lib, R, M, N):
    _check_lora(lib, _lora_problem(M, N, 264, R, 6, R, bias=M == 17))


@pytest.mark.parametrize("shape", [(65, 4096, 512, 16, 9), (128, 333, 4096, 8, 3), (129, 6, 8, 128, 2), (160, 1001, 2056, 32, 5),
                                   (160, 700, 72, 128, 1), (161, 700, 72, 128, 1), (100, 5001, 4096, 40, 30), (97, 1, 7168, 104, 4)],
                         ids=lambda s: "x".join(map(str, s)))
def test_lora_of_about_a_hundred_rows(lib, shape):
    M, N, K, R, L = shape
    for bare in (0.2, 1.0):
        p = _lora_problem(M, N, K, R, L, sum(shape), bare, bias=bare < 1, scale=bare < 1)
        got = _check_lora(lib, p, f"{shape} {bare}")
        space = torch.full((lib.lora_workspace(M, N, K, R, L),), 255, dtype=torch.uint8, device=DEV)
        assert torch.equal(_check_lora(lib, p, workspace=space), got)
    p = _lora_problem(M, N, K, R, 4, 3, bare=0.3, scale=False)
    clean = _check_lora(lib, p)
    a, b = p["a"].clone(), p["b"].clone()
    a[1, 3, 7], b[2] = float("nan"), float("inf")
    got = lib.bf16_linear_lora(p["x"], p["w"], a, b, p["ids"], p["bias"])
    keep = (p["ids"] != 1) & (p["ids"] != 2)
    assert torch.equal(got[keep], clean[keep]) and got[p["ids"] == 1].isnan().all()
    assert not got[p["ids"] == 2].isfinite().any()


def test_lora_not_finite(lib):
    """A NaN in one adapter reaches its rows alone; rows without an adapter have none of them."""
    for M, N in ((12, 72), (600, 72), (600, 5000), (2000, 1000)):
        p = _lora_problem(M, N, 128, 16, 4, 3, bare=0.3, scale=False)
        clean = _check_lora(lib, p)
        a, b = p["a"].clone(), p["b"].clone()
        a[1, 3, 7], b[2] = float("nan"), float("inf")
        got = lib.bf16_linear_lora(p["x"], p["w"], a, b, p["ids"], p["bias"])
        keep = (p["ids"] != 1) & (p["ids"] != 2)
        assert torch.equal(got[keep], clean[keep]) and got[p["ids"] == 1].isnan().all()
        assert not got[p["ids"] == 2].isfinite().any()


# ---- together ----

@pytest.mark.parametrize("flags", [0, 1, 2])
@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 128, 16, 4), (37, 512, 200, 24, 6), (600, 384, 320, 8, 2)])
def test_a_block_of_experts(lib, T, H, I, E, k, flags):
    """Router, choice, grouping, both projections, combination: each from what the one before gave, then all in a graph."""
    g = _gen(T + H)
    x, wr = _bf16(g, T, H), _bf16(g, E, H, scale=H ** -0.5)
    w1, w2 = _bf16(g, E, 2 * I, H, scale=H ** -0.5), _bf16(g, E, H, I, scale=I ** -0.5)
    shared = _bf16(g, T, H)

    def block():
        w, ids = lib.route(lib.bf16_linear_f32out(x, wr, flags=flags), k, flags=flags)
        r = lib.group_rows(ids, E, flags=flags)
        h = lib.bf16_linear_grouped(x, w1, r.offsets, rows=r.rows, swiglu=True, flags=flags)
        y = lib.bf16_linear_grouped(h, w2, r.offsets, flags=flags)
        return w, ids, r, h, y, lib.combine_rows(y, r.place, w, shared, flags=flags)

    w, ids, r, h, y, out = got = block()
    for a, b in zip(r, ref.group(ids.cpu(), E)):
        assert torch.equal(a.cpu(), b)
    ref.check(h, *ref.grouped(x, w1, r.offsets, None, r.rows, True))
    ref.check(y, *ref.grouped(h, w2, r.offsets, None, None, False))
    ref.check(out, *ref.combine(y, r.place, w, shared))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        block()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = block()
    x.copy_(x.flip(0))
    shared.copy_(shared.flip(0))
    for _ in range(2):
        graph.replay()
    want = block()
    for a, b in zip((*again[:2], *again[2], *again[3:]), (*want[:2], *want[2], *want[3:])):
        assert torch.equal(a, b)
    assert lib.device_status() == 0


def test_streams_and_graphs_of_the_adapters(lib):
    p = _lora_problem(70, 200, 256, 16, 5, 1)
    q = _lora_problem(900, 200, 256, 16, 5, 2)
    want = [_check_lora(lib, v) for v in (p, q)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [[lib.bf16_linear_lora(v["x"], v["w"], v["a"], v["b"], v["ids"], scale=v["scale"], stream=st) for v in (p, q)]
            for st in (s, None) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = [lib.bf16_linear_lora(v["x"], v["w"], v["a"], v["b"], v["ids"], scale=v["scale"]) for v in (p, q)]
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(o, want))


@pytest.mark.parametrize("flags", [0, 2])
@pytest.mark.parametrize("M,N,K", [(1, 2000, 4096), (2, 2000, 2048), (16, 2000, 2048), (60, 1100, 2048), (100, 1100, 2048), (700, 500, 520)])
def test_operands_written_just_before(lib, M, N, K, flags):
    """What the kernel before writes (each operand in turn comes last) is what the adapters' linear reads, on one workspace
    and with calls right behind one another, eager and in a graph."""
    R, L = 16, 5
    problems = [_lora_problem(M, N, K, R, L, seed) for seed in (1, 2, 3)]
    names = ("x", "w", "a", "b")
    space = torch.empty(lib.lora_workspace(M, N, K, R, L), dtype=torch.uint8, device=DEV)

    def call(v, ids, scale, out=None):
        return lib.bf16_linear_lora(v["x"], v["w"], v["a"], v["b"], ids, scale=scale, out=out, workspace=space, flags=flags)

    want = [call(v, v["ids"], v["scale"]) for v in problems]
    torch.cuda.synchronize()
    now = {n: torch.zeros_like(problems[0][n]) for n in names}
    ids = torch.zeros_like(problems[0]["ids"])
    scale = torch.zeros_like(problems[0]["scale"])
    one = {n: torch.arange(now[n].numel() // now[n].shape[-1], device=DEV, dtype=torch.int32)[:, None] for n in names}

    def copy(name, v):  # by a kernel that lets the next one start early
        lib.combine_rows(v[name].reshape(-1, v[name].shape[-1]), one[name], out=now[name].view(-1, now[name].shape[-1]), flags=flags)

    outs = [torch.zeros_like(want[0]) for _ in range(4 * len(problems))]

    def chain():
        i = 0
        for last in names:
            for v in problems:
                ids.copy_(v["ids"])
                scale.copy_(v["scale"])
                for n in names:
                    if n != last:
                        copy(n, v)
                copy(last, v)
                call(now, ids, scale, outs[i])
                i += 1

    for _ in range(3):
        chain()
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            assert torch.equal(o, want[i % len(problems)]), i
            o.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % len(problems)]), i
    assert lib.device_status() == 0


def test_groups_are_tensors_of_their_own(lib):
    ids = torch.randint(0, 5, (67, 3), generator=_gen(1), device=DEV, dtype=torch.int32)
    got = lib.group_rows(ids, 5)
    assert [tuple(v.shape) for v in got] == [(6,), (201,), (67, 3)] and all(v.is_contiguous() for v in got)
    kept = [v.clone() for v in got]
    for i, v in enumerate(got):  # one filled, the others stay
        v.fill_(-7)
        assert all(torch.equal(a, b) for a, b in zip(got[i + 1:], kept[i + 1:]))
    with torch.inference_mode():
        assert all(torch.equal(a, b) for a, b in zip(lib.group_rows(ids, 5), kept))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = lib.group_rows(ids, 5)
    ids.copy_(ids.flip(0))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(again, lib.group_rows(ids, 5)))
    got = lib.group_rows(ids[:0], 5)
    assert [tuple(v.shape) for v in got] == [(6,), (0,), (0, 3)] and not got.offsets.any()


def test_two_streams_at_once(lib):
    """Calls on two streams, each with its own workspace, give what they give one after the other."""
    p = [_problem(T, 4, 9, 500, 712, T, True, True) for T in (300, 3)]
    q = [_lora_problem(M, 500, 712, 48, 6, M, bias=True) for M in (2, 50, 700)]

    def calls():
        return ([lib.bf16_linear_grouped(v["x"], v["w"], v["offsets"], v["bias"], rows=v["rows"], swiglu=True) for v in p]
                + [lib.bf16_linear_lora(v["x"], v["w"], v["a"], v["b"], v["ids"], v["bias"], scale=v["scale"]) for v in q]
                + [v for n in (5, 5000) for v in lib.group_rows(torch.arange(n, device=DEV, dtype=torch.int32) % 7, 6)])

    want = calls()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(calls())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for r in got for a, b in zip(r, want))
    assert lib.device_status() == 0


def test_same_bits_again(lib):
    p, q = _problem(300, 4, 9, 500, 712, 4, True, True), _lora_problem(300, 500, 712, 48, 6, 4, bias=True)
    first = None
    for _ in range(5):
        r = (lib.bf16_linear_grouped(p["x"], p["w"], p["offsets"], p["bias"], rows=p["rows"], swiglu=True),
             lib.bf16_linear_lora(q["x"], q["w"], q["a"], q["b"], q["ids"], q["bias"], scale=q["scale"]))
        first = first or r
        assert all(torch.equal(a, b) for a, b in zip(r, first))


@pytest.fixture(params=["compiled", "ctypes"])
def path(lib, monkeypatch, request):
    from moe_router_gemm_gb300 import _binding
    if request.param == "ctypes":
        monkeypatch.setattr(_binding, "_calls", None)
    elif _binding._calls is None:
        pytest.skip("the marshalling module is not built for this PyTorch")
    return lib


def test_both_paths(path):
    p, q = _problem(30, 2, 6, 100, 192, 4, True, True), _lora_problem(30, 100, 192, 16, 4, 6, bias=True)
    _check(path, p)
    _check(path, _problem(30, 2, 6, 100, 192, 5, gather=False))
    _check_lora(path, q)
    ids = torch.randint(0, 6, (30, 2), device=DEV, dtype=torch.int32)
    for i in (ids, ids[:, 0].contiguous()):
        for a, b in zip(path.group_rows(i, 6), ref.group(i.cpu(), 6)):
            assert torch.equal(a.cpu(), b) and a.is_contiguous()
    y = _bf16(_gen(1), 60, 100)
    ref.check(path.combine_rows(y, ids), *ref.combine(y, ids, None, None))


def test_refusals(path):
    m = path
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device=DEV)  # noqa: E731
    i32, f32 = torch.int32, torch.float32
    x, w, off, ids = z(4, 64), z(2, 8, 64), z(3, d=i32), z(4, 2, d=i32)
    a, b, sh = z(3, 8, 64), z(3, 16, 8), z(16, 64)
    for f, err in ((lambda: m.group_rows(ids.long(), 8), TypeError), (lambda: m.group_rows(ids[:, :1], 8), ValueError),
                   (lambda: m.group_rows(z(2, 2, 2, d=i32), 8), ValueError), (lambda: m.group_rows(ids, 8, place=z(4, d=i32)), ValueError),
                   (lambda: m.bf16_linear_grouped(x.float(), w, off), TypeError), (lambda: m.bf16_linear_grouped(x, w, off[:2]), ValueError),
                   (lambda: m.bf16_linear_grouped(x, w[0], off), ValueError), (lambda: m.bf16_linear_grouped(x, w[:, :7].contiguous(), off, swiglu=True), ValueError),
                   (lambda: m.bf16_linear_grouped(x[:, :32], w, off), ValueError), (lambda: m.bf16_linear_grouped(x, w, off.long()), ValueError),
                   (lambda: m.bf16_linear_grouped(x, w, off, rows=off.long()), ValueError),
                   (lambda: m.bf16_linear_grouped(x, w, off, z(2, 7)), ValueError), (lambda: m.bf16_linear_grouped(x, w, off.cpu()), ValueError),
                   (lambda: m.bf16_linear_grouped(x, w, off, out=z(4, 9)), ValueError),
                   (lambda: m.combine_rows(x.float(), ids), ValueError), (lambda: m.combine_rows(x, ids[:, 0]), ValueError),
                   (lambda: m.combine_rows(x, ids, z(4, 2)), ValueError), (lambda: m.combine_rows(x, ids, None, z(4, 32)), ValueError),
                   (lambda: m.bf16_linear_lora(x, sh.float(), a, b, ids[:, 0].contiguous()), TypeError),
                   (lambda: m.bf16_linear_lora(x, sh, a, b, ids), ValueError), (lambda: m.bf16_linear_lora(x, sh, a, b[:2], ids[:, 0].contiguous()), ValueError),
                   (lambda: m.bf16_linear_lora(x, sh, a, b, ids[:, 0].contiguous(), scale=z(2, d=f32)), ValueError),
                   (lambda: m.bf16_linear_lora(x, sh, a, b, ids[:, 0].contiguous(), z(15)), ValueError)):
        with pytest.raises(err):
            f()
    one = ids[:, 0].contiguous()
    for f, status in ((lambda: m.group_rows(ids, 0), -1), (lambda: m.group_rows(ids, 2000), -6), (lambda: m.group_rows(ids, 1 << 32), -1),
                      (lambda: m.group_rows(ids, 8, flags=3), -1), (lambda: m.group_rows(z(4, 0, d=i32), 8), -1),
                      (lambda: m.bf16_linear_grouped(z(4, 60), z(2, 8, 60), off), -6), (lambda: m.bf16_linear_grouped(x, w, off, flags=1 << 33), -1),
                      (lambda: m.bf16_linear_grouped(x, z(1025, 1, 64), z(1026, d=i32)), -6),
                      (lambda: m.bf16_linear_grouped(z(2, 7168), z(2, 8, 7168), off, workspace=z(64, d=torch.uint8)), -1),
                      (lambda: m.combine_rows(x, z(4, 0, d=i32)), -1), (lambda: m.combine_rows(x, ids, flags=3), -1),
                      (lambda: m.bf16_linear_lora(x, sh, z(3, 4, 64), z(3, 16, 4), one), -6),
                      (lambda: m.bf16_linear_lora(x, sh, a, b, one, workspace=z(64, d=torch.uint8)), -1)):
        with pytest.raises(m.BF16LinearError) as e:
            f()
        assert e.value.status == status


def test_the_measured_cases(lib):
    mod = more_cases.load(DEV, own=True)
    rng = random.Random(17)
    for i in range(40):
        case = more_cases.small(mod, rng, ("group", "experts", "combine", "lora")[i % 4], most=3e9)
        more_cases.check(mod, case, 100 + i)
    assert lib.device_status() == 0
