"""Float64 references and error bounds of the dense training step's operators.

Bounds.  u = 2^-24 is the rounding unit of fp32, 2^-8 that of bf16.  A sum of n
products in fp32, in any order, is off by at most about n u times the sum of
their magnitudes; (n + 8) u covers the operations around it.  An operand that is
rounded to bf16 between two products carries 2^-8 of its value through the second
one's magnitudes.  TINY covers results below the fp32 range.

Everything works on float64 tensors of any device and returns (value, bound of
the absolute error before the output's own rounding); ``close`` adds that.
"""
import math

import torch

U = 2.0 ** -24
UB = 2.0 ** -8
TINY = 2.0 ** -100
SUM = 96  # depth of a row's sum (see norm_ref.py)


def close(got, ref, bound):
    """|got - ref| <= bound and the rounding of got's type, element by element."""
    unit = UB if got.dtype == torch.bfloat16 else U
    got = got.to(torch.float64)
    off = (got - ref).abs()
    most = bound * (1 + unit) + unit * ref.abs() + TINY
    bad = ~(off <= most)
    if bad.any():
        i = int((off / most).nan_to_num(math.inf).argmax())
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()} outside the bound; the worst is "
                             f"{got.flatten()[i]} for {ref.flatten()[i]}, bound {most.flatten()[i]}")
    return True


def mm(a, b):
    return torch.matmul(a, b.contiguous())


# ------------------------------------------------------------------ RMS norm --
def rms(z, gamma, eps, added):
    """z float64; `added`: z is a sum that fp32 rounds once."""
    rstd = (z.square().mean(1) + eps).rsqrt()
    y = z * rstd[:, None] * gamma
    rel = (SUM + 4 + 2 * added) * U  # squares, their sum, the root; the row's own rounding
    return y, rel * y.abs(), rstd, rel * rstd


def rms_bwd(dy, x, gamma, rstd, dres):
    """The formula on a given rstd; dx, its bound, dgamma, its bound."""
    r, K = rstd[:, None], x.shape[1]
    n = x * r
    t = dy * gamma
    dx = r * (t - n * (t * n).sum(1, keepdim=True) / K)
    mag = r * (t.abs() + n.abs() * (t * n).abs().sum(1, keepdim=True) / K)
    if dres is not None:
        dx, mag = dx + dres, mag + dres.abs()
    rows = x.shape[0]
    return dx, SUM * U * mag, (dy * n).sum(0), (rows + 8) * U * (dy * n).abs().sum(0)


# ----------------------------------------------------------------- gated FFN --
C = 2.0 * math.sqrt(2.0 / math.pi)


def act(name, g):
    """act(g), its derivative, and the error of their fp32 evaluation.  s = 1 /
    (1 + e^-a): the exponent's error of at most (10 |a| + 10) u reaches s times
    (1 - s)."""
    if name == "relu":
        on = (g > 0).to(g.dtype)
        return g * on, on, torch.zeros_like(g), torch.zeros_like(g)
    a = g if name == "silu" else C * (g + 0.044715 * g ** 3)
    da = torch.ones_like(g) if name == "silu" else C * (1 + 3 * 0.044715 * g ** 2)
    s, c = torch.sigmoid(a), torch.sigmoid(-a)
    es = s * (c * (10 * a.abs() + 10) * U + 4 * U)
    t = s * c
    slope = s + g * t * da
    e = g.abs() * es + 2 * U * (g * s).abs()
    # 1 - s is off by es and a rounding of a number near 1
    ed = es + (g * da).abs() * (es + s * U + 8 * U * t) + 4 * U * slope.abs()
    return g * s, slope, e, ed


def ffn(x, wg, wu, wd, name):
    """Returns y, its bound, g, its bound, u, its bound."""
    K, N = x.shape[1], wg.shape[0]
    g, u = mm(x, wg.T), mm(x, wu.T)
    eg = (K + 8) * U * mm(x.abs(), wg.T.abs())
    eu = (K + 8) * U * mm(x.abs(), wu.T.abs())
    a, _, ea, _ = act(name, g)
    # |act'| <= 1.13 for all three
    ea = ea + 1.13 * eg
    h = a * u
    eh = ea * (u.abs() + eu) + a.abs() * eu + 2 * U * h.abs()
    eh = eh + UB * (h.abs() + eh)
    y = mm(h, wd)
    return y, mm(eh, wd.abs()) + (N + 8) * U * mm(h.abs() + eh, wd.abs()), g, eg, u, eu


def ffn_bwd(dy, x, wg, wu, wd, g, u, name):
    """The formula on given g and u; a dict of (value, bound)."""
    M, K = x.shape
    N = wg.shape[0]
    a, da, ea, eda = act(name, g)
    dh = mm(dy, wd.T)
    edh = (K + 8) * U * mm(dy.abs(), wd.T.abs())

    def rounded(v, e):
        e = e + 4 * U * v.abs()
        return v, e + UB * (v.abs() + e)

    dz, ez = rounded(dh * u * da, edh * (u * da).abs() + (dh.abs() + edh) * u.abs() * eda)
    du, eu = rounded(dh * a, edh * a.abs() + (dh.abs() + edh) * ea)
    h, eh = rounded(a * u, ea * u.abs())

    def product(v, e, w, n):
        return mm(v, w), mm(e, w.abs()) + (n + 8) * U * mm(v.abs() + e, w.abs())

    dxg, exg = product(dz, ez, wg, 2 * N)
    dxu, exu = product(du, eu, wu, 2 * N)
    return {"dx": (dxg + dxu, exg + exu), "dwg_t": product(dz.T, ez.T, x, M),
            "dwu_t": product(du.T, eu.T, x, M), "dwd": product(h.T, eh.T, dy, M)}


# -------------------------------------------------------------- cross entropy --
def logits(x, w):
    l = mm(x, w.T)
    return l, (x.shape[1] + 8) * U * mm(x.abs(), w.T.abs())


def ce(x, w, target):
    """loss, its bound, lse, its bound.  A sum of exponentials is off by the
    logits' errors (which the log takes as they are), by the exponents' roundings
    (3 u of the largest magnitude) and by its own additions."""
    l, e = logits(x, w)
    V = w.shape[0]
    has = (target >= 0) & (target < V)
    lse = torch.logsumexp(l, 1)
    at = l.gather(1, target.clamp(0, V - 1).long()[:, None])[:, 0]
    top, most = e.max(1).values, l.abs().max(1).values
    e_lse = top + (4 * most + 128 + 4 * math.log(V) + 4 * lse.abs()) * U
    loss = torch.where(has, lse - at, 0.0)
    return loss, torch.where(has, e_lse + top + U * most, 0.0), lse, e_lse


def ce_bwd(dloss, x, w, target, lse):
    """The formula on a given lse; a dict of (value, bound)."""
    M, K = x.shape
    V = w.shape[0]
    l, e = logits(x, w)
    has = (target >= 0) & (target < V)
    p = (l - lse[:, None]).exp()
    ep = p * (e + (4 * l.abs() + 4 * lse.abs()[:, None] + 8) * U)
    d = p.clone()
    rows = torch.arange(M, device=x.device)[has]
    d[rows, target[has].long()] -= 1.0
    s = torch.where(has, dloss, 0.0)[:, None]
    d, ed = d * s, (ep + 2 * U * d.abs()) * s.abs()
    ed = ed + UB * (d.abs() + ed)

    def product(v, b, n):
        return mm(v[0], b), mm(v[1], b.abs()) + (n + 8) * U * mm(v[0].abs() + v[1], b.abs())

    return {"dx": product((d, ed), w, V + 64), "dw": product((d.T, ed.T), x, M)}
