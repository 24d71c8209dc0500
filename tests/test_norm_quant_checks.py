"""Layer norm and int8 entry points on the CPU: every rejection of the C ABI
happens on the host before any device call (fake addresses), the binding
rejects tensors the kernels could not take, and the float64 references the
GPU tests use agree with autograd, with differences and with hand-worked
values."""
import numpy as np
import pytest
import torch

import norm_ref as R

BF, F32, I8, U8 = torch.bfloat16, torch.float32, torch.int8, torch.uint8
P = 0x100000  # a 16-byte-aligned address that is never read


@pytest.fixture(scope="module")
def tw():
    import os

    from activation_sparse_feed_gate_amd import build as b

    srcs = [os.path.join(b.CSRC, s) for s in b.SOURCES] + [os.path.join(b.INCLUDE, "tw.h")]
    if not os.path.exists(b.LIBRARY) or any(
            os.path.getmtime(s) > os.path.getmtime(b.LIBRARY) for s in srcs):
        b.build()
    from activation_sparse_feed_gate_amd import tw as mod

    return mod


# ------------------------------------------------------------------- C ABI --
def fwd(tw, **kw):
    a = dict(x=P, xt=0, xs=64, add=None, at=0, gamma=P, beta=P, eps=1e-5, M=4, K=64, sum=None, y=P,
             yt=0, mean=None, rstd=None)
    a.update(kw)
    return tw._lib.tw_layernorm_fwd(a["x"], a["xt"], a["xs"], a["add"], a["at"], a["gamma"],
                                    a["beta"], a["eps"], a["M"], a["K"], a["sum"], a["y"],
                                    a["yt"], a["mean"], a["rstd"], None, None)


def lnq(tw, **kw):
    a = dict(x=P, xt=0, xs=64, add=None, at=0, gamma=P, beta=P, eps=1e-5, M=4, K=64, sum=None, q=P,
             scale=P)
    a.update(kw)
    return tw._lib.tw_layernorm_quant(a["x"], a["xt"], a["xs"], a["add"], a["at"], a["gamma"],
                                      a["beta"], a["eps"], a["M"], a["K"], a["sum"], a["q"],
                                      a["scale"], None, None)


NORM_BAD = [(dict(M=-1), 1), (dict(K=0), 1), (dict(K=16385, xs=16385), 2), (dict(xt=2), 1),
            (dict(xt=7), 1), (dict(xs=63), 1), (dict(xs=-64), 1), (dict(xs=1 << 41), 2),
            (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(x=None), 1),
            (dict(x=P + 8), 1), (dict(gamma=None), 1), (dict(gamma=P + 4), 1),
            (dict(beta=P + 4), 1), (dict(add=P, at=2), 1), (dict(add=P + 2), 1),
            (dict(sum=P), 1), (dict(add=P, sum=P + 4), 1)]


@pytest.mark.parametrize("kw,code", NORM_BAD + [(dict(y=None), 1), (dict(yt=2), 1), (dict(y=P + 2), 1),
                                                (dict(mean=P + 4), 1), (dict(rstd=P + 4), 1)])
def test_layernorm_fwd_rejects(tw, kw, code):
    assert fwd(tw, **kw) == code and tw._lib.tw_last_error()


@pytest.mark.parametrize("kw,code", NORM_BAD + [(dict(q=None), 1), (dict(scale=None), 1),
                                                (dict(q=P + 8), 1), (dict(scale=P + 4), 1)])
def test_layernorm_quant_rejects(tw, kw, code):
    assert lnq(tw, **kw) == code and tw._lib.tw_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 1), (dict(K=0), 1), (dict(K=20000, xs=20000), 2), (dict(xs=3), 1), (dict(dt=2), 1),
    (dict(xt=2), 1), (dict(ot=2), 1), (dict(dy=None), 1), (dict(x=None), 1), (dict(gamma=None), 1),
    (dict(mean=None), 1), (dict(rstd=None), 1), (dict(dx=None), 1), (dict(dx=P + 4), 1),
    (dict(dres=P + 4), 1), (dict(dg=P + 4), 1), (dict(db=P + 4), 1), (dict(ws=None), 1),
    (dict(wsb=16), 1)])
def test_layernorm_bwd_rejects(tw, kw, code):
    a = dict(dy=P, dt=0, x=P, xt=0, xs=64, gamma=P, mean=P, rstd=P, dres=None, M=4, K=64, dx=P,
             ot=1, dg=P, db=P, ws=P, wsb=1 << 24)
    a.update(kw)
    st = tw._lib.tw_layernorm_bwd(a["dy"], a["dt"], a["x"], a["xt"], a["xs"], a["gamma"],
                                  a["mean"], a["rstd"], a["dres"], a["M"], a["K"], a["dx"],
                                  a["ot"], a["dg"], a["db"], a["ws"], a["wsb"], None, None)
    assert st == code and tw._lib.tw_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 1), (dict(K=0), 1), (dict(K=65537, xs=65537), 2), (dict(xt=2), 1), (dict(xs=5), 1),
    (dict(x=None), 1), (dict(q=None), 1), (dict(scale=None), 1), (dict(q=P + 1), 1)])
def test_quant_rows_rejects(tw, kw, code):
    a = dict(x=P, xt=0, xs=64, M=4, K=64, q=P, scale=P)
    a.update(kw)
    st = tw._lib.tw_quant_rows(a["x"], a["xt"], a["xs"], a["M"], a["K"], a["q"], a["scale"], None,
                               None)
    assert st == code and tw._lib.tw_last_error()


PRODUCT_BAD = [
    (dict(M=-1), 1), (dict(K=0), 1), (dict(N=0), 1), (dict(K=72, xs=72), 2),
    (dict(K=65552, xs=65552), 2), (dict(M=(1 << 24) + 1), 2), (dict(N=(1 << 24) + 1), 2),
    (dict(M=1 << 24, N=1 << 16), 2), (dict(yt=2), 1), (dict(xt=3), 1), (dict(x=None), 1),
    (dict(x=P + 8), 1), (dict(y=None), 1), (dict(xs=8), 1), (dict(ws=None), 1), (dict(wsb=8), 1),
    (dict(xsc=P), 1),                      # scales for a float x
    (dict(xt=2), 1),                       # int8 rows without scales
    (dict(xt=2, xsc=P, xs=128), 1)]        # int8 rows apart


@pytest.mark.parametrize("kw,code", PRODUCT_BAD + [(dict(w=None), 1), (dict(wsc=None), 1),
                                                   (dict(w=P + 8), 1), (dict(bias=P + 4), 1)])
def test_quant_linear_rejects(tw, kw, code):
    a = dict(x=P, xt=0, xs=64, xsc=None, w=P, wsc=P, bias=None, M=4, K=64, N=64, y=P, yt=0, ws=P,
             wsb=1 << 30)
    a.update(kw)
    st = tw._lib.tw_quant_linear(a["x"], a["xt"], a["xs"], a["xsc"], a["w"], a["wsc"], a["bias"],
                                 a["M"], a["K"], a["N"], a["y"], a["yt"], a["ws"], a["wsb"], None,
                                 None)
    assert st == code and tw._lib.tw_last_error()


@pytest.mark.parametrize("kw,code", PRODUCT_BAD + [
    (dict(wg=None), 1), (dict(wu=None), 1), (dict(gs=None), 1), (dict(us=None), 1),
    (dict(beta=P), 1), (dict(gamma=P, eps=-1.0), 1), (dict(gamma=P + 4), 1),
    (dict(gamma=P, beta=P + 4), 1), (dict(gamma=P, xt=2, xsc=P), 1),
    (dict(gamma=P, K=16400, xs=16400), 2)])
def test_quant_gateup_rejects(tw, kw, code):
    a = dict(x=P, xt=0, xs=64, xsc=None, gamma=None, beta=None, eps=1e-5, wg=P, gs=P, wu=P, us=P,
             M=4, K=64, N=64, y=P, yt=0, ws=P, wsb=1 << 30)
    a.update(kw)
    st = tw._lib.tw_quant_gateup(a["x"], a["xt"], a["xs"], a["xsc"], a["gamma"], a["beta"],
                                 a["eps"], a["wg"], a["gs"], a["wu"], a["us"], a["M"], a["K"],
                                 a["N"], a["y"], a["yt"], a["ws"], a["wsb"], None, None)
    assert st == code and tw._lib.tw_last_error()


def test_workspace_queries(tw):
    assert tw.tw_quant_workspace_bytes(100, 64) >= 100 * 64 + 400
    assert tw.tw_quant_workspace_bytes(1 << 24, 65536) >= 1 << 40
    for bad in ((-1, 64), (4, 0), (4, 8), (4, 1 << 20), ((1 << 24) + 1, 64)):
        assert tw.tw_quant_workspace_bytes(*bad) == 0
    assert tw.tw_layernorm_bwd_workspace_bytes(1, 64) >= 2 * 64 * 4
    assert tw.tw_layernorm_bwd_workspace_bytes(0, 64) >= 2 * 64 * 4
    for bad in ((-1, 64), (4, 0), (4, 16385)):
        assert tw.tw_layernorm_bwd_workspace_bytes(*bad) == 0


# ------------------------------------------------------------------ binding --
def e(*shape, dtype=F32):
    return torch.empty(shape, dtype=dtype)


M, K, N = 6, 64, 48
BAD = (TypeError, ValueError)


@pytest.mark.parametrize("over,what", [
    (dict(x=e(M, K, dtype=torch.float16)), "x"), (dict(x=e(M * K)), "two-dimensional"),
    (dict(gamma=e(K + 1)), "gamma"), (dict(gamma=e(K, dtype=BF)), "gamma"), (dict(gamma=None), "gamma is required"),
    (dict(beta=e(K - 1)), "beta"), (dict(y=e(M, K + 1)), "y"), (dict(y=e(M, K, dtype=I8)), "y"),
    (dict(add=e(M, K, dtype=I8)), "add"), (dict(add=e(M - 1, K)), "add"),
    (dict(add=e(M, K), total=e(M, K, dtype=BF)), "total"), (dict(mean=e(M, 1)), "mean"),
    (dict(rstd=e(M, dtype=BF)), "rstd"), (dict(x=e(K, M).t()), "contiguous rows"), ({}, "device tensor")])
def test_layernorm_binding(tw, over, what):
    a = dict(x=e(M, K), gamma=e(K), beta=e(K), eps=1e-5, y=e(M, K))
    a.update(over)
    with pytest.raises(BAD, match=what):
        tw.tw_layernorm_fwd(**a)


@pytest.mark.parametrize("over,what", [
    (dict(dy=e(M, K + 1)), "dy"), (dict(mean=e(M + 1)), "mean"), (dict(rstd=None), "rstd is required"),
    (dict(dx=e(M, K, dtype=I8)), "dx"), (dict(dres=e(M, K, dtype=BF)), "dres"),
    (dict(dgamma=e(K, dtype=BF)), "dgamma"), (dict(dbeta=e(1)), "dbeta")])
def test_layernorm_bwd_binding(tw, over, what):
    a = dict(dy=e(M, K), x=e(M, K), gamma=e(K), mean=e(M), rstd=e(M), dx=e(M, K), dgamma=e(K),
             dbeta=e(K), ws=e(16))
    a.update(over)
    with pytest.raises(BAD, match=what):
        tw.tw_layernorm_bwd(**a)


@pytest.mark.parametrize("over,what", [
    (dict(w=e(N, K)), "w"), (dict(w=e(N, K + 16, dtype=I8)), "w"), (dict(w_scale=e(K)), "w_scale"),
    (dict(bias=e(N, dtype=BF)), "bias"), (dict(y=e(N, M)), "y"), (dict(x_scale=e(M)), "x is not int8"),
    (dict(w=e(N * K, dtype=I8)), "two-dimensional")])
def test_quant_linear_binding(tw, over, what):
    a = dict(x=e(M, K), w=e(N, K, dtype=I8), w_scale=e(N), y=e(M, N), ws=e(16))
    a.update(over)
    with pytest.raises(BAD, match=what):
        tw.tw_quant_linear(**a)


@pytest.mark.parametrize("over,what", [
    (dict(wu=e(N + 1, K, dtype=I8)), "wu"), (dict(u_scale=e(N + 1)), "u_scale"),
    (dict(gamma=e(K + 1)), "gamma"), (dict(h=e(M, K)), "h")])
def test_quant_gateup_binding(tw, over, what):
    a = dict(x=e(M, K), wg=e(N, K, dtype=I8), g_scale=e(N), wu=e(N, K, dtype=I8), u_scale=e(N),
             h=e(M, N), ws=e(16))
    a.update(over)
    with pytest.raises(BAD, match=what):
        tw.tw_quant_gateup(**a)


# --------------------------------------------------------------- references --
def test_norm_reference_matches_autograd():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(5, 37, generator=g, dtype=torch.float64, requires_grad=True)
    gamma = torch.randn(37, generator=g, dtype=torch.float64, requires_grad=True)
    beta = torch.randn(37, generator=g, dtype=torch.float64, requires_grad=True)
    dy, dres = (torch.randn(5, 37, generator=g, dtype=torch.float64) for _ in range(2))
    y = torch.nn.functional.layer_norm(x, (37,), gamma, beta, 1e-5)
    ((y * dy).sum() + (x * dres).sum()).backward()
    X, G, B = x.detach().numpy(), gamma.detach().numpy(), beta.detach().numpy()
    yr, mean, rstd, *_ = R.norm(X, G, B, 1e-5, False)
    assert np.allclose(yr, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    dx, dg, db, *_ = R.norm_bwd(dy.numpy(), X, G, mean, rstd, dres.numpy())
    assert np.allclose(dx, x.grad.numpy(), rtol=1e-11, atol=1e-11)
    assert np.allclose(dg, gamma.grad.numpy(), rtol=1e-11, atol=1e-11)
    assert np.allclose(db, beta.grad.numpy(), rtol=1e-11, atol=1e-11)


def test_norm_backward_reference_by_differences():
    rng = np.random.default_rng(2)
    X, DY = rng.standard_normal((4, 9)), rng.standard_normal((4, 9))
    G, B = rng.standard_normal(9), rng.standard_normal(9)
    y, mean, rstd, *_ = R.norm(X, G, B, 1e-5, False)
    dx, dg, db, *_ = R.norm_bwd(DY, X, G, mean, rstd, None)
    h = 1e-6
    for i in range(4):
        for k in range(9):
            d = np.zeros_like(X)
            d[i, k] = h
            num = ((R.norm(X + d, G, B, 1e-5, False)[0] - R.norm(X - d, G, B, 1e-5, False)[0]) * DY).sum() / (2 * h)
            assert abs(num - dx[i, k]) < 1e-7
    for k in range(9):
        d = np.zeros(9)
        d[k] = h
        num = ((R.norm(X, G + d, B, 1e-5, False)[0] - R.norm(X, G - d, B, 1e-5, False)[0]) * DY).sum() / (2 * h)
        assert abs(num - dg[k]) < 1e-7
        num = ((R.norm(X, G, B + d, 1e-5, False)[0] - R.norm(X, G, B - d, 1e-5, False)[0]) * DY).sum() / (2 * h)
        assert abs(num - db[k]) < 1e-7


def test_quantise_reference_by_hand():
    x = np.array([[127.0, -63.5, 0.5, 1.5, -1.5, 0.25, 0.0, 126.6],
                  [0, 0, 0, 0, 0, 0, 0, 0],
                  [2.0 ** -101, 0, 0, 0, 0, 0, 0, 0],
                  [1, np.inf, 0, 0, 0, 0, 0, 0],
                  [np.nan, 5, 0, 0, 0, 0, 0, 0]], dtype=np.float32)
    q, s = R.quantise(x)
    assert q[0].tolist() == [127, -64, 0, 2, -2, 0, 0, 127]
    assert s[0] == 1.0 and s[1] == 0.0 and s[2] == 0.0 and np.isnan(s[3:]).all()
    assert not q[1:].any()


def test_product_reference_by_hand():
    q = np.array([[1, -2, 127]], dtype=np.int8)
    w = np.array([[3, 4, 127], [-1, 0, 2]], dtype=np.int8)
    v, _ = R.product(q, np.array([0.5]), w, np.array([2.0, 0.25]), np.array([1.0, -1.0]))
    assert v.tolist() == [[(3 - 8 + 16129) * 1.0 + 1.0, (-1 + 254) * 0.125 - 1.0]]


def test_native_calls_leave_bad_arguments_to_the_checked_path(tw):
    """On the CPU every argument is unusable: the native functions answer
    None (no exception, no call) and the binding's own checks raise."""
    c = tw._calls
    x, g, w = e(4, 64), e(64), e(8, 64, dtype=I8)
    assert c.layernorm(x, g, None, 1e-5, None, BF) is None
    assert c.layernorm(None, "gamma", 3, object(), x, BF) is None
    assert c.layernorm() is None and c.layernorm(x) is None
    assert c.layernorm_backward(x, x, g, e(4), e(4), None, F32) is None
    assert c.quant_linear(x, w, e(8), None, None, BF, None) is None
    assert c.quant_linear(x, w, e(8), None, None, "bf16", None) is None
    assert c.quant_gateup(x, w, e(8), w, e(8), None, None, 1e-5, None, BF, None) is None
    with pytest.raises(ValueError, match="device tensor"):
        tw.layernorm(x, g)
