"""Values at the ends of their range in the adapters' linear: infinities in A and B."""
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
