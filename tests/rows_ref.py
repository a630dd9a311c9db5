"""Plain 64-bit forms of the operators whose weight depends on the row, for the tests (torch on any device, no code of the
package), with how far a result may be from them.

ACC: fp32 accumulation of K products whose magnitudes sum to s is off by at most (K / 64 + 16) * 2^-22 * s, as in
moe_ref.linear_bound.  A result rounded once to bf16 is off by half a step more.
"""
import torch


def half_ulp(v):
    """Half the distance between bf16 values around v."""
    _, e = torch.frexp(v.abs().clamp_min(2.0 ** -126))
    return torch.ldexp(torch.ones_like(v), e - 9)


def acc(K, s):
    return (K / 64 + 16) * 2.0 ** -22 * s


def check(got, want, slack, what=""):
    """got (bf16) is the rounding of a value within `slack` of want; NaN and infinities in the same places."""
    g = got.double()
    assert g.shape == want.shape, f"{what}: {tuple(g.shape)} {tuple(want.shape)}"
    assert torch.equal(g.isnan(), want.isnan()), f"{what}: NaN in other places"
    inf = want.isinf()
    assert torch.equal(g[inf], want[inf]), f"{what}: infinities"
    fine = ~(want.isnan() | inf)
    w, s = want[fine], slack[fine]
    off = (g[fine] - w).abs()
    bad = off > half_ulp(w.abs() + s) + s
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {off[bad].max()} at {w[bad][off[bad].argmax()]}"


def group(ids, groups):
    """(offsets, rows, place) by a loop over the pairs."""
    flat = ids.reshape(-1).tolist()
    k = ids.shape[1] if ids.dim() == 2 else 1
    of = [[i for i, e in enumerate(flat) if e == g] for g in range(groups)] if groups * len(flat) < 1 << 22 else None
    if of is None:
        of = [[] for _ in range(groups)]
        for i, e in enumerate(flat):
            if 0 <= e < groups:
                of[e].append(i)
    offsets, rows, place = [0], [-1] * len(flat), [-1] * len(flat)
    p = 0
    for g in of:
        for i in g:
            rows[p], place[i] = i // k, p
            p += 1
        offsets.append(p)
    t = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return t(offsets), t(rows), t(place).reshape(ids.shape)


def silu(g):
    return g / (1 + torch.exp(-g))


def grouped(x, w, offsets, bias, rows, swiglu):
    """(out, slack) in f64 for the positions 0 .. offsets[-1] - 1."""
    x, ends = x.double(), offsets.tolist()
    K = x.shape[1]
    outs, slacks = [], []
    for e in range(w.shape[0]):
        lo, hi = ends[e], ends[e + 1]
        v = x[lo:hi] if rows is None else x[rows[lo:hi].long()]
        we = w[e].double()
        y, s = v @ we.T, v.abs() @ we.abs().T
        if bias is not None:
            y, s = y + bias[e].double(), s + bias[e].double().abs()
        s = acc(K, s)
        if swiglu:
            N = y.shape[1] // 2
            g, u, f = y[:, :N], y[:, N:], silu(y[:, :N])
            # silu's slope is at most 1.1; the exponential (2 ulp), the sum, the quotient and the product: 8 * 2^-24 of it
            y, s = f * u, 1.1 * s[:, :N] * (u.abs() + s[:, N:]) + f.abs() * s[:, N:] + 2.0 ** -21 * (f * u).abs() + 2.0 ** -126
        outs.append(y)
        slacks.append(s)
    return torch.cat(outs), torch.cat(slacks)


def combine(y, place, weights, addend):
    """(out, slack): k products and an addend, each sum rounded by 2^-24 of the running magnitude."""
    T, k = place.shape
    out = torch.zeros(T, y.shape[1], dtype=torch.float64, device=y.device)
    mag = torch.zeros_like(out)
    for j in range(k):
        have = ((place[:, j] >= 0) & (place[:, j] < y.shape[0])).nonzero().view(-1)
        v = y[place[have, j].long()].double()
        if weights is not None:
            v = v * weights[have, j, None].double()
        out[have] += v
        mag[have] += v.abs()
    if addend is not None:
        out, mag = out + addend.double(), mag + addend.double().abs()
    return out, (k + 2) * 2.0 ** -24 * mag


def lora(x, w, a, b, ids, bias, scale):
    """(out, slack).  The inner values may go on as a sum of two bf16 values, which is off by at most 2^-18 of them (2^-9 of
    2^-9), and times the scale in fp32: 2^-17 of them in all."""
    x = x.double()
    K, (L, N, R) = x.shape[1], b.shape
    wd = w.double()
    y, s = x @ wd.T, x.abs() @ wd.abs().T
    if bias is not None:
        y, s = y + bias.double(), s + bias.double().abs()
    s = acc(K, s)
    for e in range(L):
        mine = (ids == e).nonzero().view(-1)
        if not mine.numel():
            continue
        ad, bd, f = a[e].double(), b[e].double(), 1.0 if scale is None else scale[e].double()
        h = f * (x[mine] @ ad.T)
        hs = abs(f) * acc(K, x[mine].abs() @ ad.abs().T) + 2.0 ** -17 * h.abs()
        y[mine] += h @ bd.T
        s[mine] += (hs + acc(R, h.abs() + hs)) @ bd.abs().T
    return y, s + 2.0 ** -22 * y.abs()
