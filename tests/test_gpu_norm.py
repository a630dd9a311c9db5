"""bf16_rmsnorm against its 64-bit form.

Bounds, derived from the arithmetic: h is bf16(x + residual), compared bit for bit.  y in fp32 is off by the sum of
squares (every partial sum at most 2^-24 of it, at most H / 512 + 69 in a row, halved by the root) and a handful of
roundings: below 2^-17 of |y| up to H = 32768.  bf16 adds half its spacing at y; e4m3 2^-4 of |y| (2^-10 of the block's scale below
its normal range), e2m1 1/4 of |y| (1/4 of the scale below 1).  A scale byte must be the one of the block's largest |y|,
or of one 2^-17 of it away.
"""
import numpy as np
import pytest
import torch

import moe_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SLACK = 2.0 ** -17
E4M3 = torch.float8_e4m3fn


def _inputs(rows, H, seed, ld=None, residual=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, ld or H, generator=g).mul(torch.exp2(4 * torch.randn(rows, 1, generator=g))).to(torch.bfloat16)
    r = torch.randn(rows, H, generator=g).to(torch.bfloat16) if residual else None
    w = (1 + 0.3 * torch.randn(H, generator=g)).to(torch.bfloat16)
    return x.to(DEV)[:, :H], (r.to(DEV) if residual else None), w.to(DEV)


def _check(lib, x, r, w, eps, quant, res, scale=None):
    h, y = ref.norm(ref.f64(x), None if r is None else ref.f64(r), ref.f64(w), eps)
    if r is not None:
        assert np.array_equal(ref.f64(res.residual), h)
    if res.out is not None:
        g = ref.f64(res.out)
        assert (np.abs(g - y) <= ref.half_ulp(np.abs(y) * (1 + SLACK)) + SLACK * np.abs(y)).all()
    if quant == "fp8":
        v = ref.f64(res.codes.view(E4M3))
        u = y / scale
        lim = np.clip(u, -448, 448)
        assert (np.abs(v - lim) <= (2.0 ** -4 + 2 * SLACK) * np.abs(lim) + 2.0 ** -10).all()
    elif quant in ("mxfp8", "mxfp4"):
        top, peak = (8, 448.0) if quant == "mxfp8" else (2, 6.0)
        rows, H = y.shape
        e = res.scales.cpu().numpy().astype(np.int64) - 127
        blocks = y.reshape(rows, H // 32, 32)
        lo = ref.scale_exponents(blocks * (1 - SLACK), top)
        hi = ref.scale_exponents(blocks * (1 + SLACK), top)
        assert ((e == lo) | (e == hi)).all()
        s = np.exp2(e.astype(np.float64))[..., None]
        u = np.clip(blocks / s, -peak, peak)
        if quant == "mxfp8":
            v = ref.f64(res.codes.view(E4M3)).reshape(blocks.shape)
            tol = (2.0 ** -4 + 2 * SLACK) * np.abs(u) + 2.0 ** -10
        else:
            v = ref.values_mxfp4(res.codes.cpu().numpy(), np.full((rows, H // 32), 127, np.uint8)).reshape(blocks.shape)
            tol = (0.25 + 2 * SLACK) * np.maximum(np.abs(u), 1.0)
        assert (np.abs(v - u) <= tol).all()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,H", [(1, 1), (3, 7), (1, 33), (5, 64), (2, 1000), (1, 2048), (17, 2880), (4, 4097),
                                    (33, 7168), (700, 67), (1000, 1501), (2000, 2881), (300, 8189), (2, 16384), (9, 16383), (1, 32768), (2, 33000), (1, 40009)])
def test_bf16(lib, rows, H, residual):
    x, r, w = _inputs(rows, H, rows + H, residual=residual)
    res = lib.rmsnorm(x, w, r)
    assert (res.residual is None) == (r is None) and res.codes is None and res.scales is None
    _check(lib, x, r, w, 1e-6, None, res)


@pytest.mark.parametrize("quant", ["fp8", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("rows,H,ld", [(1, 32, 32), (3, 96, 96), (700, 7168, 7169), (300, 1536, 2113), (9, 64, 70),
                                       (40, 16384, 16390), (3, 16416, 16417), (7, 1536, 2112), (5, 2880, 2881), (16, 7168, 7168),
                                       (2, 512, 515)])
@pytest.mark.parametrize("residual", [False, True])
def test_quantised(lib, rows, H, ld, quant, residual):
    x, r, w = _inputs(rows, H, rows + H, ld=ld, residual=residual)
    scale = torch.full((1,), 0.015625, device=DEV) if quant == "fp8" else None
    both = lib.rmsnorm(x, w, r, quant=quant, scale=scale)
    _check(lib, x, r, w, 1e-6, quant, both, 0.015625)
    alone = lib.rmsnorm(x, w, r, quant=quant, scale=scale, bf16_out=False)
    assert alone.out is None and torch.equal(alone.codes, both.codes)
    if quant != "fp8":
        assert torch.equal(alone.scales, both.scales)


@pytest.mark.parametrize("rows,H,ld", [(900, 188, 516), (5, 99, 107), (800, 2001, 2009), (3, 4099, 4099), (2000, 65, 65),
                                       (5, 983, 1235), (900, 1501, 1800), (400, 7168, 7300), (3, 64, 67), (77, 8191, 8195)])
@pytest.mark.parametrize("residual", [False, True])
def test_odd_rows_in_fp8(lib, rows, H, ld, residual):
    x, r, w = _inputs(rows, H, rows + H, ld=ld, residual=residual)
    scale = torch.full((1,), 0.03125, device=DEV)
    res = lib.rmsnorm(x, w, r, quant="fp8", scale=scale)
    _check(lib, x, r, w, 1e-6, "fp8", res, 0.03125)


@pytest.mark.parametrize("start", [0, 1, 3, 8, 1536])
def test_column_ranges(lib, start):
    """A column range of a wider matrix, at even and odd offsets."""
    x, _, w = _inputs(9, 2112, 5, residual=False)
    part, pw = x[:, start:start + 512], w[:512]
    res = lib.rmsnorm(part, pw, quant="mxfp8")
    _check(lib, part, None, pw, 1e-6, "mxfp8", res)


def test_in_place_residual_and_outputs(lib):
    x, r, w = _inputs(6, 1024, 3)
    want = lib.rmsnorm(x, w, r, quant="mxfp4")
    r2 = r.clone()
    out = torch.empty_like(x.contiguous())
    got = lib.rmsnorm(x, w, r2, quant="mxfp4", out=out, residual_out=r2)
    assert got.residual is r2 and got.out is out
    assert torch.equal(r2, want.residual) and torch.equal(out, want.out) and torch.equal(got.codes, want.codes)


@pytest.mark.parametrize("H", [256, 255])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_bad_values_stay_in_their_row(lib, H, bad):
    x, r, w = _inputs(5, H, 11)
    clean = lib.rmsnorm(x, w, r)
    x[2, 7] = bad
    res = lib.rmsnorm(x, w, r)
    others = [0, 1, 3, 4]
    assert torch.equal(res.out[others], clean.out[others])
    if np.isnan(bad):
        assert res.out[2].isnan().all()
    else:  # h / inf is 0, inf / inf NaN
        assert res.out[2, 7].isnan() and (res.out[2, :7] == 0).all()
    if H % 32 == 0:
        q = lib.rmsnorm(x, w, r, quant="mxfp4")
        v = lib.dequant_mxfp4(q.codes, q.scales)
        assert v[2, :32].isnan().all() and not v[others].isnan().any()


def test_zero_rows_and_epsilon(lib):
    x = torch.zeros(3, 128, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    res = lib.rmsnorm(x, w, quant="mxfp8")
    assert (res.out == 0).all() and (res.codes == 0).all() and (res.scales == 0).all()
    x[1] = 2.0
    assert torch.equal(lib.rmsnorm(x, w, eps=0.0).out[1], w)
    assert (lib.rmsnorm(x, w, eps=12.0).out[1] == 0.5).all()
    empty = lib.rmsnorm(x[:0], w, x[:0], quant="mxfp4")
    assert empty.out.shape == (0, 128) and empty.codes.shape == (0, 64)


def test_extreme_magnitudes(lib):
    """Squares that stay inside fp32 at both ends of what bf16 rows hold."""
    for mag in (2.0 ** -45, 2.0 ** 45):
        x, _, w = _inputs(4, 512, 8, residual=False)
        x = (x.float() * mag).to(torch.bfloat16)
        _check(lib, x, None, w, 0.0, None, lib.rmsnorm(x, w, eps=0.0))


def test_repeats_bit_for_bit_and_on_another_stream(lib):
    x, r, w = _inputs(64, 2880, 2)
    a = lib.rmsnorm(x, w, r, quant="mxfp8")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = lib.rmsnorm(x, w, r, quant="mxfp8", stream=s)
    s.synchronize()
    assert torch.equal(a.out, b.out) and torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


def test_offsets_past_32_bits(lib):
    """rows * ldx past 2^32 elements: the last rows of a strided view equal the same rows alone."""
    rows, H, ld = 33600, 512, 128000
    x = torch.empty(rows, ld, dtype=torch.bfloat16, device=DEV)
    x[-3:] = torch.randn(3, ld, device=DEV).to(torch.bfloat16)
    x[:-3, :H] = 1.0
    w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    assert rows * ld > 2 ** 32
    res = lib.rmsnorm(x[:, :H], w, quant="mxfp8")
    last = lib.rmsnorm(x[-3:, :H].contiguous(), w, quant="mxfp8")
    assert torch.equal(res.out[-3:], last.out) and torch.equal(res.codes[-3:], last.codes)


def test_refusals(lib):
    x, r, w = _inputs(4, 64, 1)
    for bad in (dict(quant="int8"), dict(quant="fp8"), dict(scale=torch.ones(1, device=DEV)), dict(bf16_out=False),
                dict(residual_out=r), dict(quant="mxfp8", codes=torch.empty(4, 63, dtype=torch.uint8, device=DEV))):
        with pytest.raises(ValueError):
            lib.rmsnorm(x, w, **bad)
    with pytest.raises(ValueError):
        lib.rmsnorm(x, w[:63], r)
    with pytest.raises(ValueError):
        lib.rmsnorm(x.t(), w)
    with pytest.raises(TypeError):
        lib.rmsnorm(x.float(), w)
    y, _, v = _inputs(4, 48, 1)
    with pytest.raises(lib.BF16LinearError) as e:
        lib.rmsnorm(y, v, quant="mxfp4", codes=torch.empty(4, 24, dtype=torch.uint8, device=DEV))
    assert e.value.status == -6
    with pytest.raises(lib.BF16LinearError) as e:
        lib.rmsnorm(x, w, out=x)  # an output over an input
    assert e.value.status == -1


def test_the_longest_rows(lib):
    """H within a block's threads of 2^31.  Ones have a norm of one exactly, so y is the weight, which bf16 holds."""
    H = (1 << 31) - 40
    x = torch.ones(1, H, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    w[-700:] = (1 + torch.rand(700, device=DEV)).to(torch.bfloat16)
    w[1 << 30] = 3.0
    assert torch.equal(lib.rmsnorm(x, w, eps=0.0).out[0], w)


@pytest.mark.parametrize("H", [40, 512, 2001, 40000])
def test_squares_past_fp32(lib, H):
    """Rows whose squares fp32 does not hold: zeros above, infinities below where eps is 0, and only in those rows."""
    x, _, w = _inputs(4, H, 8, residual=False)
    x = x.sign() + (x == 0)
    clean = lib.rmsnorm(x, w, eps=0.0).out
    x[1] *= 2.0 ** 64
    x[2] *= 2.0 ** -76
    y = lib.rmsnorm(x, w, eps=0.0).out
    assert (y[1] == 0).all() and torch.equal(y[2], torch.inf * (x[2].float() * w.float()).sign().to(y.dtype))
    assert torch.equal(y[[0, 3]], clean[[0, 3]])
    y = lib.rmsnorm(x, w).out
    assert (y[1] == 0).all()
    _check(lib, x[2:3], None, w, 1e-6, None, lib.rmsnorm(x[2:3], w))
