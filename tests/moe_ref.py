"""Plain 64-bit forms of the norm, the routing and MXFP4, for the tests (numpy, no code of the package)."""
import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def bf16(a) -> torch.Tensor:
    return torch.as_tensor(np.asarray(a, dtype=np.float64)).to(torch.bfloat16)


def scale_exponents(v, top):
    """max(floor(log2 max|v|) - top, -127) of each 32-value block of v[..., 32] (frexp: m * 2^e, m in [0.5, 1))."""
    amax = np.abs(v).max(-1)
    _, e = np.frexp(amax)
    return np.where(amax == 0, -127, np.maximum(e - 1 - top, -127)).astype(np.int64)


def quant_mxfp4(x):
    """(packed codes, scale bytes) of finite x[rows, K] (f64): nearest e2m1, ties to the even code, from the definition."""
    rows, K = x.shape
    v = x.reshape(rows, K // 32, 32)
    e = scale_exponents(v, 2)
    y = v / np.exp2(e.astype(np.float64))[..., None]
    d = np.abs(np.abs(y)[..., None] - E2M1)  # distance to each magnitude
    lo = d.argmin(-1)                        # the nearest, the lower of two at the same distance
    hi = 7 - d[..., ::-1].argmin(-1)         # ... the higher
    code = np.where(lo % 2 == 0, lo, hi) + 8 * np.signbit(y)
    code = code.reshape(rows, K).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e + 127).astype(np.uint8)


def values_mxfp4(q, s):
    """The f64 values [rows, K] of packed codes and scale bytes (255: NaN)."""
    code = np.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1)
    v = E2M1[code & 7] * np.where(code > 7, -1.0, 1.0)
    scale = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127.0))
    return v * np.repeat(scale, 32, axis=-1)


def half_ulp(v):
    """Half the distance between bf16 values around v: the most that rounding to nearest moves it."""
    _, e = np.frexp(np.maximum(np.abs(v), 2.0 ** -126))
    return np.exp2(e - 9.0)


def linear_bound(y, sabs, K):
    """How far a bf16 result may be from the f64 sum y of products whose magnitudes sum to sabs: the one rounding to bf16,
    and fp32 accumulation over K / 64 steps and the joins of at most 16 parts, each step off by at most
    2^-22 of the running magnitude (a tensor core aligns and cuts its addends rather than rounding their sum)."""
    acc = (K / 64 + 16) * 2.0 ** -22 * sabs
    return half_ulp(np.abs(y) + acc) + acc


def check_linear(got, xv, wv, bias, K, what=""):
    y = xv @ wv.T
    sabs = np.abs(xv) @ np.abs(wv).T
    if bias is not None:
        y, sabs = y + bias, sabs + np.abs(bias)
    g = f64(got)
    assert g.shape == y.shape
    assert np.array_equal(np.isnan(g), np.isnan(y)), f"{what}: NaN in other places"
    fine = ~np.isnan(y)
    bad = np.abs(g - y)[fine] > linear_bound(y, sabs, K)[fine]
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} outside, worst {np.abs(g - y)[fine].max()}"


def norm(x, residual, weight, eps):
    """(h, y) in f64; h holds bf16 values."""
    h = x
    if residual is not None:
        h = f64((torch.from_numpy(x) + torch.from_numpy(residual)).float().to(torch.bfloat16))
    with np.errstate(all="ignore"):
        return h, h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * weight


def route(logits, k, scoring, bias, groups, top_groups, group_best, renormalize, scale):
    """For each token: (keys f64, scores f64, allowed experts as a boolean row), groups chosen by exact f64 keys."""
    T, E = logits.shape
    if scoring == "softmax":
        m = logits.max(-1, keepdims=True)
        p = np.exp(logits - np.where(np.isinf(m), 0.0, m))
        total = p.sum(-1, keepdims=True)
        score = p / np.where(total == 0, 1.0, total)
    else:
        with np.errstate(over="ignore"):
            score = 1.0 / (1.0 + np.exp(-logits))
    key = score + (0.0 if bias is None else bias)
    if scoring == "softmax" and bias is None and group_best == 1:
        key = logits.copy()
    key = np.where(np.isneginf(logits), -np.inf, key)
    allowed = np.ones((T, E), bool)
    if groups > 1:
        g = np.sort(key.reshape(T, groups, -1), -1)[..., ::-1][..., :group_best].sum(-1)
        order = np.argsort(-g, axis=-1, kind="stable")[:, :top_groups]
        keep = np.zeros((T, groups), bool)
        np.put_along_axis(keep, order, True, 1)
        allowed = np.repeat(keep, E // groups, axis=1)
    return key, score, allowed
