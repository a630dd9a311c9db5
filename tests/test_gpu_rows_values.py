"""Values at the ends of their range in the grouped and the adapters' linears: infinities in an adapter's B, gates whose
exponential nearly overflows, scales that overflow a part of a sum; and rows too long for the form of one or two rows."""
import pytest
import torch

import rows_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF = float("inf")


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _bf16(g, *shape, scale=1.0):
    return (scale * torch.randn(*shape, generator=g, device=DEV)).to(torch.bfloat16)


def _check_lora(lib, p, what=""):
    got = lib.bf16_linear_lora(p["x"], p["w"], p["a"], p["b"], p["ids"], p["bias"], scale=p["scale"])
    ref.check(got, *ref.lora(**p), what)
    assert lib.device_status() == 0
    return got


def _adapters(M, N, K, R, L, seed):
    g = _gen(seed)
    return dict(x=_bf16(g, M, K), w=_bf16(g, N, K, scale=K ** -0.5), a=_bf16(g, L, R, K, scale=K ** -0.5),
                b=_bf16(g, L, N, R, scale=R ** -0.5), ids=torch.randint(-1, L, (M,), generator=g, device=DEV, dtype=torch.int32),
                bias=None, scale=torch.randn(L, generator=g, device=DEV))


# Every form: one and two rows, few rows, about a hundred, and tiles (inner values by row or on tensor cores; K whole or in
# parts; one block of 64 ranks or two).
FORMS = [(1, 200, 128, 8), (2, 200, 128, 8), (12, 200, 128, 8), (60, 1100, 256, 24), (100, 200, 128, 8), (300, 200, 128, 8), (300, 200, 2048, 16),
         (700, 9000, 72, 8), (2500, 300, 512, 64), (520, 260, 512, 128)]


@pytest.mark.parametrize("shape", FORMS, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("exact", [False, True])
def test_infinities_in_b(lib, shape, exact):
    """An infinite element of B gives its output the sign of the inner value that it meets, whatever the number of rows; two
    that meet with different signs give NaN, as does one that meets a zero.  `exact`: inner values that bf16 holds."""
    M, N, K, R = shape
    p = _adapters(M, N, K, R, 5, M + N)
    if exact:
        p["x"] = torch.zeros_like(p["x"])
        p["x"][:, 3] = 1.0
        p["scale"] = None
    b, last = p["b"], R - 1
    b[0, 7, 0], b[1, 0, last], b[2, N - 1, R // 2] = INF, -INF, INF  # one each
    b[3, 5, 0], b[3, 5, last], b[3, 6, 1], b[3, 6, 2] = INF, INF, -INF, INF
    p["a"][4, 1] = 0.0  # an inner value of zero
    b[4, 9, 1] = INF
    p["ids"][: min(M, 5)] = torch.arange(min(M, 5), device=DEV, dtype=torch.int32)
    got = _check_lora(lib, p, f"{shape}")
    if M >= 5:
        assert got[0, 7].isinf() and got[1, 0].isinf() and got[2, N - 1].isinf() and got[4, 9].isnan()


@pytest.mark.parametrize("shape", FORMS, ids=lambda s: "x".join(map(str, s)))
def test_infinite_inner_values(lib, shape):
    """An infinity in A, against finite elements of B, infinite ones and zeros."""
    M, N, K, R = shape
    p = _adapters(M, N, K, R, 3, M + N)
    p["x"][:, 3] = 1.0
    p["a"][0, 1, 3], p["a"][1, R - 1, 3] = INF, -INF
    p["b"][0, 4, 1], p["b"][0, 5, 1], p["b"][0, 6, 1], p["b"][1, 2, R - 1] = INF, -INF, 0.0, INF
    p["ids"][: min(M, 2)] = torch.arange(min(M, 2), device=DEV, dtype=torch.int32)
    _check_lora(lib, p, f"{shape}")


@pytest.mark.parametrize("M", [1, 2, 3, 20, 64, 70, 150, 300])
def test_scales_that_overflow_parts_of_a_sum(lib, M):
    """scale * (x @ A^T) is finite, scale times a part of that sum is not; and an infinite scale."""
    K, N, R, L = 8192, 1100, 8, 3
    p = _adapters(M, N, K, R, L, M)
    p["x"] = torch.ones_like(p["x"])
    a = torch.ones(K, device=DEV)
    a[K // 2:] = -1.0
    a[K - 1] = -0.875  # the sum is 0.125, in any order exact
    p["a"] = a.to(torch.bfloat16).expand(L, R, K).contiguous()
    p["b"] = p["b"].abs()  # (so that no infinities of both signs meet)
    p["scale"] = torch.tensor([1e37, INF, -2.5e37], device=DEV)
    p["ids"] = (torch.arange(M, device=DEV) % L).int()
    _check_lora(lib, p, f"{M} rows")


@pytest.mark.parametrize("shape", [(1, 1100, 24584, 16, 3), (1, 2100, 24584, 16, 3), (1, 2048, 26000, 16, 3), (1, 1100, 28040, 8, 3), (1, 5001, 30000, 128, 2), (2, 1100, 12296, 16, 3),
                                   (2, 1025, 20000, 40, 3), (1, 4100, 27000, 16, 2)], ids=lambda s: "x".join(map(str, s)))
def test_one_or_two_long_rows(lib, shape):
    """Rows past what the form of one or two rows takes, with weights of enough rows for the plan by the fill of the SMs."""
    M, N, K, R, L = shape
    p = _adapters(M, N, K, R, L, K)
    p["ids"].clamp_(min=0)
    p["bias"] = _bf16(_gen(1), N)
    _check_lora(lib, p, f"{shape}")


# ---- SwiGLU ----

# silu's steps, relative errors: the exponential's instruction 2^-22.5 and the correction's rounding 2^-24, the sum 2^-24, the
# reciprocal 2^-23, the product by g 2^-24, the product by up 2^-24: below 2^-20 in all.
SILU = 2.0 ** -20


def _gates(lib, gate, frac, up, K):
    """SwiGLU of one row whose gates are gate + frac (a bf16 product by one, and a bf16 bias: exact in fp32 where the sum has
    24 bits) and whose up values are `up`."""
    n = gate.numel()
    x = torch.zeros(1, K, dtype=torch.bfloat16, device=DEV)
    x[0, 0] = 1.0
    w = torch.zeros(1, 2 * n, K, dtype=torch.bfloat16, device=DEV)
    w[0, :n, 0], w[0, n:, 0] = gate, up
    bias = torch.zeros(1, 2 * n, dtype=torch.bfloat16, device=DEV)
    bias[0, :n] = frac
    off = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    assert (lib.grouped_workspace(1, 1, n, K, True) > 0) == (K >= 1024)  # K in parts, or whole
    got = lib.bf16_linear_grouped(x, w, off, bias, swiglu=True)
    assert lib.device_status() == 0
    return got[0]


@pytest.mark.parametrize("K", [8, 7168])
@pytest.mark.parametrize("power", [0, 100, -20])
def test_silu_over_its_range(lib, K, power):
    """From the most negative gates whose exponential fp32 holds (exp(88.72) < 2^128) to large ones: off by half a bf16 step
    and SILU."""
    whole = torch.arange(-88, 89, device=DEV).repeat_interleave(16).float()
    frac = (torch.arange(16, device=DEV) / 16.0).repeat(177) * torch.where(whole < 0, -1.0, 1.0)
    keep = (whole + frac > -88.72)
    gate, frac = whole[keep].to(torch.bfloat16), (frac[keep] + 2.0 ** -7).to(torch.bfloat16)
    g = gate.double() + frac.double()
    assert torch.equal(g.float().double(), g) and (g > -88.7228).all()
    up = torch.full_like(gate, 2.0 ** power)
    got = _gates(lib, gate, frac, up, K)
    want = g / (1 + torch.exp(-g)) * up.double()
    ref.check(got, want, SILU * want.abs() + 2.0 ** -133, f"2^{power}, K {K}")


@pytest.mark.parametrize("K", [8, 7168])
def test_silu_at_its_ends(lib, K):
    """Infinite gates and up values, and gates past the exponential's range, as g / (1 + exp(-g)) * u in fp32 has them."""
    rows = [(-88.0, -0.5, INF, -INF), (-88.0, -0.5, -INF, INF), (-87.0, -0.25, 2.0 ** 120, None), (-88.0, -0.5, 2.0 ** 127, None),
            (-89.0, 0.0, 3.0, 0.0), (-200.0, 0.0, 2.0 ** 100, 0.0), (-3e38, 0.0, 1.0, 0.0), (-89.0, 0.0, INF, float("nan")),
            (INF, 0.0, 2.0, INF), (INF, 0.0, -2.0, -INF), (INF, 0.0, 0.0, float("nan")), (-INF, 0.0, 1.0, float("nan")),
            (3e38, 0.0, 1.0, None), (0.0, 0.0, INF, float("nan")), (0.0, 0.0, 5.0, 0.0), (2.0 ** -120, 0.0, 1.0, None),
            (float("nan"), 0.0, 1.0, float("nan")), (1.0, 0.0, float("nan"), float("nan"))]
    col = lambda i: torch.tensor([r[i] for r in rows], device=DEV).to(torch.bfloat16)  # noqa: E731
    gate, frac, up = col(0), col(1), col(2)
    g = gate.double() + frac.double()
    want = g / (1 + torch.exp(-g)) * up.double()
    said = torch.tensor([float("nan") if r[3] is None else r[3] for r in rows], device=DEV, dtype=torch.float64)
    want = torch.where(torch.tensor([r[3] is None for r in rows], device=DEV), want, said)
    got = _gates(lib, gate, frac, up, K)
    ref.check(got, want, SILU * want.abs().nan_to_num(0.0, 0.0, 0.0) + 2.0 ** -133, f"K {K}")


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("K", [192, 4096])
def test_infinite_and_huge_rows(lib, swiglu, K):
    """A row with an infinity, and one whose only element is huge, against the definition: infinities of the weights' signs,
    and with SwiGLU what silu makes of them."""
    g = _gen(5)
    E, N, T = 3, 100, 24
    x = _bf16(g, T, K)
    w = _bf16(g, E, 2 * N if swiglu else N, K, scale=K ** -0.5)
    off = torch.tensor([0, 9, 9, T], dtype=torch.int32, device=DEV)
    x[4, 5], x[17, 5] = INF, -INF
    x[20], x[8] = 0.0, 0.0
    x[20, 1], x[8, 2] = 3e38, -3e38
    got = lib.bf16_linear_grouped(x, w, off, swiglu=swiglu)
    want, slack = ref.grouped(x, w, off, None, None, swiglu)
    past = want.abs() > 3.4e38 * (1 + 2.0 ** -8)  # (products of two sums of about 1e37)
    want = torch.where(past, torch.copysign(torch.full_like(want, INF), want), want)
    ref.check(got, want, slack, f"swiglu {swiglu}")
    if swiglu:
        assert got[4].isinf().any() and got[4].isnan().any() and got[20].isinf().any() and (got[20] == 0).any()
    else:
        assert got[4].isinf().all() and got[17].isinf().all()
