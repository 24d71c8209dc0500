"""Layer-norm gradient of rows that do not fill the threads that hold them,
where the mean times 1/std passes the range of fp32: the threads' unused
places take no part in the row's sums."""
import numpy as np
import pytest

import norm_ref as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def tw():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from activation_sparse_feed_gate_amd import tw as mod

    return mod


# (512, 2048: rows that fill the threads) whole vectors and odd rows
@pytest.mark.parametrize("K", [5, 200, 512, 768, 1001, 1536, 2048, 2500, 5000, 9000])
@pytest.mark.parametrize("xt", [BF, F32])
@pytest.mark.parametrize("power,eps", [(110, 1e-12), (120, 1e-5)])
def test_constant_row_far_from_zero(tw, K, xt, power, eps):
    """A constant row has variance 0, so rstd = 1 / sqrt(eps) and n = 0, and
    dx = rstd (t - mean(t)) for t = dy gamma: finite, whatever the row's value."""
    g = torch.Generator().manual_seed(K)
    x = torch.randn(3, K, generator=g)
    x[1] = 2.0 ** power
    dy = torch.randn(3, K, generator=g)
    gamma = 1 + 0.2 * torch.randn(K, generator=g)
    mean, rstd = torch.zeros(3), torch.ones(3)
    mean[1], rstd[1] = 2.0 ** power, 1 / eps ** 0.5
    assert (mean[1] * rstd[1]).isinf()
    out = tw.layernorm_backward(dy.cuda(), x.to(xt).cuda(), gamma.cuda(), mean.cuda(), rstd.cuda())
    t = dy.double().numpy() * gamma.double().numpy()
    r = rstd.double().numpy()[1]
    ref = r * (t[1] - t[1].mean())
    bound = R.SUM * R.U * r * (np.abs(t[1]) + np.abs(t[1]).mean())
    got = out["dx"].double().cpu().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got[1] - ref) <= bound).all()
    n = x.to(xt).double().numpy()
    n[1] = 0
    d = dy.double().numpy()
    assert (np.abs(out["dgamma"].double().cpu().numpy() - (d * n).sum(0)) <= R.SUM * R.U * np.abs(d * n).sum(0)).all()
    assert (np.abs(out["dbeta"].double().cpu().numpy() - d.sum(0)) <= R.SUM * R.U * np.abs(d).sum(0)).all()
