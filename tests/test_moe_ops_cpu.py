"""The norm's, the routing's and MXFP4's checks of arguments, which need no GPU, and the tests' own 64-bit forms."""
import ctypes as C

import numpy as np
import torch

import moe_ref as ref
from test_oracle_mxfp8 import floor_log2
from fractions import Fraction

P = [C.c_void_p(v << 24) for v in range(1, 9)]
EINVAL, EALIGN, EUNSUPPORTED = -1, -2, -6


def test_rmsnorm_checks(lib):
    f = lib.load().bf16_rmsnorm
    x, r, w, o, ro, c, s, sc = P

    def call(x=x, ldx=64, r=None, w=w, o=o, ro=None, c=None, s=None, sc=None, rows=4, H=64, eps=1e-6, quant=0, flags=0):
        return f(x, ldx, r, w, o, ro, c, s, sc, rows, H, eps, quant, flags, None)

    for bad in (dict(rows=-1), dict(H=0), dict(ldx=63), dict(flags=3), dict(quant=4), dict(quant=-1), dict(eps=-1.0),
                dict(eps=float("nan")), dict(x=None), dict(w=None), dict(o=None), dict(r=r), dict(ro=ro), dict(quant=1, c=c),
                dict(quant=2, c=c), dict(quant=3, s=s), dict(o=x), dict(r=r, ro=o), dict(quant=2, c=o, s=s),
                dict(rows=1 << 62)):
        assert call(**bad) == EINVAL, bad
    assert call(H=48, quant=2, c=c, s=s) == EUNSUPPORTED
    at = lambda p, d: C.c_void_p(p.value + d)  # noqa: E731
    for bad in (dict(x=at(x, 1)), dict(w=at(w, 8)), dict(o=at(o, 2)), dict(r=at(r, 4), ro=ro), dict(quant=1, c=at(c, 1), sc=sc),
                dict(quant=1, c=c, sc=at(sc, 2))):
        assert call(**bad) == EALIGN, bad
    assert call(rows=0, x=None, o=None) == 0


def test_route_checks(lib):
    f = lib.load().bf16_route
    lg, b, w, i = P[:4]

    def call(lg=lg, ld=64, b=None, w=w, i=i, T=4, E=64, k=4, sc=0, g=1, tg=1, gb=1, flags=0):
        return f(lg, ld, b, w, i, T, E, k, sc, g, tg, gb, 1, 1.0, 0, flags, None)

    for bad in (dict(T=-1), dict(E=0), dict(ld=63), dict(k=0), dict(sc=2), dict(g=0), dict(g=5), dict(tg=0), dict(g=4, tg=5),
                dict(g=16, tg=1, k=5), dict(gb=0), dict(gb=3), dict(flags=3),
                dict(lg=None), dict(w=None), dict(i=None), dict(i=w), dict(w=lg), dict(b=w)):
        assert call(**bad) == EINVAL, bad
    for bad in (dict(E=1025, ld=1025), dict(k=33), dict(g=64)):
        assert call(**bad) == EUNSUPPORTED, bad
    at = lambda p, d: C.c_void_p(p.value + d)  # noqa: E731
    assert call(lg=at(lg, 2)) == EALIGN and call(w=at(w, 1)) == EALIGN and call(b=at(b, 2)) == EALIGN
    assert call(T=0, lg=None) == 0


def test_mxfp4_checks(lib):
    L = lib.load()
    a, s, b, t, o, x = P[:6]
    f = L.bf16_linear_mxfp4
    assert f(a, s, b, t, None, o, 4, 8, 80, 0, None) == EUNSUPPORTED
    assert f(a, s, b, t, None, o, -1, 8, 64, 0, None) == EINVAL
    assert f(a, s, b, t, None, o, 4, 8, 64, 3, None) == EINVAL
    assert f(None, s, b, t, None, o, 4, 8, 64, 0, None) == EINVAL
    assert f(a, s, b, t, None, a, 4, 8, 64, 0, None) == EINVAL
    assert f(C.c_void_p(a.value + 8), s, b, t, None, o, 4, 8, 64, 0, None) == EALIGN
    assert f(a, s, b, t, None, o, 0, 8, 64, 0, None) == 0
    d = L.bf16_linear_mxfp4_dynamic
    need = lib.mxfp4_dynamic_workspace(4000, 4000, 64)
    assert need >= 4000 * 34
    assert d(x, b, t, None, o, 4000, 4000, 64, None, 0, 0, None) == EINVAL
    assert d(x, b, t, None, o, 4000, 4000, 64, a, need - 1, 0, None) == EINVAL
    assert d(x, b, t, None, o, 4000, 4000, 64, C.c_void_p(a.value + 16), need, 0, None) == EALIGN
    assert d(x, b, t, None, o, 4000, 4000, 64, x, need, 0, None) == EINVAL
    assert d(x, b, t, None, o, 4, 8, 80, a, 1 << 20, 0, None) == EUNSUPPORTED
    assert d(None, b, t, None, o, 0, 8, 64, None, 0, 0, None) == 0
    for q in (L.bf16_quant_mxfp4, lambda x, r, k, c, s, fl, st: L.bf16_dequant_mxfp4(c, s, r, k, x, fl, st)):
        assert q(x, 4, 48, a, s, 0, None) == EUNSUPPORTED
        assert q(x, -1, 64, a, s, 0, None) == EINVAL
        assert q(x, 4, 64, x, s, 0, None) == EINVAL
        assert q(C.c_void_p(x.value + 2), 4, 64, a, s, 0, None) == EALIGN
        assert q(x, 1 << 62, 64, a, s, 0, None) == EINVAL
        assert q(None, 0, 64, None, None, 0, None) == 0
    assert lib.mxfp4_dynamic_workspace(4, 8, 80) == 0 and lib.mxfp4_dynamic_workspace(-1, 8, 64) == 0


def test_the_reference_quantisation_is_the_definition():
    """Exact rationals: the scale exponent by integer arithmetic, each code the nearest value, ties to the even code."""
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((6, 64)) * np.exp2(rng.integers(-130, 100, (6, 2))).repeat(32, 1))
    x = ref.f64(ref.bf16(x))
    x[0, :32] = 0
    q, s = ref.quant_mxfp4(x)
    mags = [Fraction(v) for v in (0, "1/2", 1, "3/2", 2, 3, 4, 6)]
    for r in range(6):
        for b in range(2):
            vals = [Fraction(float(v)) for v in x[r, 32 * b:32 * b + 32]]
            amax = max(abs(v) for v in vals)
            e = -127 if amax == 0 else max(floor_log2(amax) - 2, -127)
            assert s[r, b] == e + 127
            for j, v in enumerate(vals):
                y = abs(v) / Fraction(2) ** e
                best = min(range(8), key=lambda c: (abs(mags[c] - y), c % 2))
                code = (q[r, 16 * b + j // 2] >> (4 * (j % 2))) & 15
                assert code & 7 == best
    v = ref.values_mxfp4(q, s)
    assert np.array_equal(ref.quant_mxfp4(v)[0] & 0x77, q & 0x77)


def test_the_reference_forms_of_norm_and_route():
    t = torch.tensor([[3.0, 4.0, 0.0, 0.0]], dtype=torch.float64).numpy()
    h, y = ref.norm(t, None, np.ones(4), 0.0)
    assert np.allclose(y, [[1.2, 1.6, 0, 0]])
    key, score, allowed = ref.route(np.log(np.array([[1.0, 2.0, 3.0, 2.0]])), 2, "softmax", None, 2, 1, 1, True, 1.0)
    assert np.allclose(score, [[0.125, 0.25, 0.375, 0.25]]) and allowed.tolist() == [[False, False, True, True]]



def test_mxfp4_workspace_at_long_k(lib):
    """Up to the largest K there is, a call whose x does not fit shared memory asks for room for its codes and scales."""
    up = lambda v: (v + 255) // 256 * 256  # noqa: E731
    for M in (1, 16, 17, 300):
        for K in (262144, 1 << 26, 1 << 28, 2_000_000_000, 2_021_027_872, 2_147_483_392, (1 << 31) - 32):
            for N in (128, 2112):
                assert lib.mxfp4_dynamic_workspace(M, N, K) == up(M * K // 2) + up(M * K // 32), (M, N, K)
