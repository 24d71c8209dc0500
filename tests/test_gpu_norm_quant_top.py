"""The scale of a normed and quantised row comes from that row's elements
alone: rows that do not fill the threads that hold them, with a beta whose
largest entry the norm cancels, against float64."""
import numpy as np
import pytest

import norm_ref as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8


@pytest.fixture(scope="module")
def tw():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from activation_sparse_feed_gate_amd import tw as mod

    return mod


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def cancelled(M, K, dtype, gain):
    """Rows with one late channel far below the rest, gamma about ``gain``,
    and a beta that is large on that channel alone: |beta| there exceeds every
    |y|.  (The channel is among the last 8; its norm is near -sqrt(K - 1) or
    -9, whichever is nearer to zero.)"""
    g = torch.Generator().manual_seed(K)
    x = torch.randn(M, K, generator=g)
    gamma = gain * (1 + 0.1 * torch.rand(K, generator=g))
    beta = 0.01 * gain * torch.randn(K, generator=g)
    x[:, K - 3] = -30.0 if K < 100 else -9.0
    beta[K - 3] = 6.0 * gain
    return x.to(dtype).cuda(), gamma.cuda(), beta.cuda()


def reference(x, add, gamma, beta):
    """y in float64 and the bound of the kernels' own y."""
    z = f64(x) + (0 if add is None else f64(add))
    y, _, rstd, e_y, _, _ = R.norm(z, f64(gamma), f64(beta), 1e-5, False)
    return y, e_y + R.U * np.abs(z) * np.abs(f64(gamma)) * rstd[:, None]


# rows of whole vectors that leave lanes without elements (and two that do not:
# 512, 2048), in every number of threads and vectors
@pytest.mark.parametrize("K", [8, 264, 512, 768, 1536, 2048, 3000, 5632, 9000, 12288])
@pytest.mark.parametrize("gain", [1.0, 0.01])
@pytest.mark.parametrize("at", [None, BF, F32])
def test_scale_is_the_rows_own(tw, K, gain, at):
    x, gamma, beta = cancelled(5, K, F32 if K % 16 else BF, gain)
    add = None if at is None else (0.01 * torch.randn(5, K, generator=torch.Generator().manual_seed(1))).to(at).cuda()
    y, e_y = reference(x, add, gamma, beta)
    top, e_top = np.abs(y).max(1), e_y.max(1)
    assert (np.abs(f64(beta)[K - 8:]).max() > 1.2 * top).all(), "beta is to exceed every |y|"
    out = tw.layernorm_quantize(x, gamma, beta, add=add)
    scale, q = f64(out["scale"]), f64(out["q"])
    assert (np.abs(scale * 127 - top) <= e_top + 2 * R.U * top).all()
    assert (np.abs(q).max(1) == 127).all()
    assert (np.abs(q * scale[:, None] - y) <= scale[:, None] * (0.5 + 127 * 4 * R.U) + e_y + e_top[:, None]).all()


@pytest.mark.parametrize("M", [1, 2, 4, 5, 9, 40])
@pytest.mark.parametrize("K", [16, 768, 1536, 5632])
def test_gateup_from_the_float64_norm(tw, M, K):
    """The gate and up products of codes taken from the float64 norm, at row
    counts that norm in the product's kernel and at those that do not.  A code
    whose value lies within the kernels' own error of half way may be the next
    one: it moves a sum by at most its weight."""
    N = 70
    x, gamma, beta = cancelled(M, K, BF, 1.0)
    y, e_y = reference(x, None, gamma, beta)
    top, e_top = np.abs(y).max(1), e_y.max(1)
    step = top / 127
    v = y / step[:, None]
    # error of a value in codes: the norm's, the row's scale's, three fp32 roundings
    e_v = e_y / step[:, None] + 127 * (e_top / top)[:, None] + 127 * 4 * R.U
    q = np.rint(v)
    unsure = (np.abs(np.abs(v - q) - 0.5) <= e_v).astype(np.float64)
    assert unsure.sum() < 0.02 * unsure.size + 2
    g = torch.Generator().manual_seed(7)
    wg, wu = (torch.randint(-127, 128, (N, K), generator=g, dtype=I8) for _ in range(2))
    gs, us = (torch.rand(N, generator=g) * 0.05 + 1e-3 for _ in range(2))
    h = f64(tw.quant_gateup(x, wg.cuda(), gs.cuda(), wu.cuda(), us.cuda(), gamma=gamma, beta=beta, out_dtype=F32))

    def product(w, s):
        W = f64(w)
        p = (q @ W.T) * step[:, None] * f64(s)
        e = (unsure @ np.abs(W).T) * step[:, None] * f64(s)
        return p, e + np.abs(p) * ((e_top / top)[:, None] + 6 * R.U)

    (pg, eg), (pu, eu) = product(wg, gs), product(wu, us)
    pg = np.maximum(pg, 0)
    ref = pg * pu
    bound = eg * (np.abs(pu) + eu) + eu * pg + 2 * R.U * np.abs(ref)
    assert (np.abs(h - ref) <= bound).all(), np.abs(h - ref).max()
