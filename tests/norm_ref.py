"""Float64 references and error bounds of the layer norm and the int8 rows.

Bounds.  u = 2^-24 is the rounding unit of fp32, 2^-8 that of bf16 (8 significant bits).  A sum
of K terms that the kernels take in any tree of depth D has an error of at
most about D u times the sum of the magnitudes; a row is summed by up to 1024
threads, each over at most 64 values one after the other, so D is at most
64 + 16 (tree) and SUM = 96 covers it and the divisions around it.
"""
import numpy as np

U = 2.0 ** -24
UB = 2.0 ** -8
SUM = 96


def out_unit(bf16):
    """Rounding of the stored value on top of the fp32 arithmetic."""
    return UB * (1 + 2 ** -8) if bf16 else U


def norm(z, gamma, beta, eps, bf16):
    """z, gamma, beta float64; returns y, mean, rstd and their bounds."""
    mean = z.mean(1)
    d = z - mean[:, None]
    var = (d * d).mean(1)
    rstd = 1.0 / np.sqrt(var + eps)
    scaled = d * rstd[:, None] * gamma
    y = scaled if beta is None else scaled + beta
    e_mean = SUM * U * np.abs(z).mean(1)
    # d is off by u |z| and the mean's error; the mean of d^2 then by the sum
    # and by twice that (Cauchy-Schwarz over the row), over var + eps
    e_d = 2 * U * np.abs(z) + e_mean[:, None]
    rms_ed = np.sqrt((e_d * e_d).mean(1))
    rel_r = SUM * U + rstd * rms_ed * (1 + rstd * rms_ed)
    e_y = (np.abs(gamma) * rstd[:, None] * e_d + np.abs(scaled) * (rel_r[:, None] + 4 * U)
           + 2 * U * np.abs(y))
    return y, mean, rstd, e_y + out_unit(bf16) * np.abs(y), e_mean + U * np.abs(mean), rstd * rel_r


def norm_bwd(dy, x, gamma, mean, rstd, dres):
    """Formula of the gradient on given statistics; returns dx, dgamma, dbeta
    and the magnitudes their errors are proportional to."""
    r = rstd[:, None]
    n = (x - mean[:, None]) * r
    mag_n = (np.abs(x) + np.abs(mean)[:, None]) * np.abs(r)
    t = dy * gamma
    dx = r * (t - t.mean(1, keepdims=True) - n * (t * n).mean(1, keepdims=True))
    mag = np.abs(r) * (np.abs(t) + np.abs(t).mean(1, keepdims=True)
                       + mag_n * (np.abs(t) * mag_n).mean(1, keepdims=True))
    if dres is not None:
        dx = dx + dres
        mag = mag + np.abs(dres)
    return (dx, (dy * n).sum(0), dy.sum(0), mag, (np.abs(dy) * mag_n).sum(0), np.abs(dy).sum(0))


def quantise(x32):
    """The rows of a float32 array exactly as tw_quant_rows defines them, in
    float32 arithmetic: every operation is one IEEE rounding, so codes and
    scales are expected to the bit."""
    x32 = np.asarray(x32, dtype=np.float32)
    top = np.abs(x32).max(1) if x32.shape[1] else np.zeros(x32.shape[0], np.float32)
    bad = ~np.isfinite(x32).all(1)
    some = ~bad & (top >= np.float32(2.0 ** -100))
    safe = np.where(some, top, np.float32(1)).astype(np.float32)
    inv = np.float32(1) / safe * np.float32(127)
    with np.errstate(invalid="ignore"):
        q = np.rint((np.where(np.isfinite(x32), x32, 0) * inv[:, None]).astype(np.float32))
    q = np.where(some[:, None], q, 0).astype(np.int8)
    scale = np.where(some, safe / np.float32(127), np.float32(0)).astype(np.float32)
    scale[bad] = np.nan
    return q, scale


def product(q, xs, w, ws, bias=None):
    """Exact value of the int8 product and the magnitude its three roundings
    act on (the integer sum to fp32 and two multiplications, plus the add)."""
    s = q.astype(np.float64) @ w.astype(np.float64).T
    v = s * xs.astype(np.float64)[:, None] * ws.astype(np.float64)
    e = 4 * U * np.abs(v)
    if bias is not None:
        v = v + bias.astype(np.float64)
        e = e + U * np.abs(v)
    return v, e
