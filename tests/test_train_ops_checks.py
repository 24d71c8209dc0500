"""The dense training step's entry points on the CPU: every rejection of the C
ABI happens on the host before any device call (fake addresses), the binding
rejects tensors the kernels could not take, and the float64 references that the
GPU tests use agree with autograd."""
import ctypes
import os

import pytest
import torch

import train_ref as R

BF, F32, I8, I64 = torch.bfloat16, torch.float32, torch.int8, torch.int64
P = 0x100000  # a 16-byte-aligned address that is never read
Q = 0x200000


@pytest.fixture(scope="module")
def tw():
    from activation_sparse_feed_gate_amd import build as b

    srcs = [os.path.join(b.CSRC, s) for s in b.SOURCES] + [os.path.join(b.INCLUDE, "tw.h")]
    if not os.path.exists(b.LIBRARY) or any(
            os.path.getmtime(s) > os.path.getmtime(b.LIBRARY) for s in srcs):
        b.build()
    from activation_sparse_feed_gate_amd import tw as mod

    return mod


def call(f, order, base, kw):
    a = dict(base)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return f(*[a[k] for k in order.split()], None, None)


# ------------------------------------------------------------------ RMS norm --
RMS_BAD = [(dict(M=-1), 1), (dict(K=0), 1), (dict(K=16385, xs=16385), 2), (dict(xt=2), 1), (dict(xt=7), 1),
           (dict(xs=63), 1), (dict(xs=1 << 41), 2), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
           (dict(x=None), 1), (dict(x=P + 8), 1), (dict(gamma=None), 1), (dict(gamma=P + 4), 1),
           (dict(add=P, at=2), 1), (dict(add=P + 2), 1), (dict(sum=P), 1), (dict(add=P, sum=P + 4), 1)]


@pytest.mark.parametrize("kw,code", RMS_BAD + [(dict(y=None), 1), (dict(yt=2), 1), (dict(y=P + 2), 1),
                                               (dict(rstd=P + 4), 1)])
def test_rmsnorm_fwd_rejects(tw, kw, code):
    base = dict(x=P, xt=0, xs=64, add=None, at=0, gamma=P, eps=1e-5, M=4, K=64, sum=None, y=P, yt=0,
                rstd=None)
    assert call(tw._lib.tw_rmsnorm_fwd, "x xt xs add at gamma eps M K sum y yt rstd", base, kw) == code
    assert tw._lib.tw_last_error()


@pytest.mark.parametrize("kw,code", RMS_BAD + [(dict(q=None), 1), (dict(scale=None), 1), (dict(q=P + 8), 1)])
def test_rmsnorm_quant_rejects(tw, kw, code):
    base = dict(x=P, xt=0, xs=64, add=None, at=0, gamma=P, eps=1e-5, M=4, K=64, sum=None, q=P, scale=P)
    assert call(tw._lib.tw_rmsnorm_quant, "x xt xs add at gamma eps M K sum q scale", base, kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), 1), (dict(K=0), 1), (dict(K=20000, xs=20000), 2), (dict(xs=3), 1), (dict(dt=2), 1),
    (dict(xt=2), 1), (dict(ot=2), 1), (dict(dy=None), 1), (dict(x=None), 1), (dict(gamma=None), 1),
    (dict(rstd=None), 1), (dict(dx=None), 1), (dict(dx=P + 4), 1), (dict(dres=P + 4), 1),
    (dict(dg=P + 4), 1), (dict(ws=None), 1), (dict(wsb=16), 1)])
def test_rmsnorm_bwd_rejects(tw, kw, code):
    base = dict(dy=P, dt=0, x=P, xt=0, xs=64, gamma=P, rstd=P, dres=None, M=4, K=64, dx=P, ot=1, dg=P,
                ws=P, wsb=1 << 24)
    order = "dy dt x xt xs gamma rstd dres M K dx ot dg ws wsb"
    assert call(tw._lib.tw_rmsnorm_bwd, order, base, kw) == code


# ----------------------------------------------------------------- gated FFN --
FFN_BAD = [(dict(M=-1), 1), (dict(K=0), 1), (dict(N=0), 1), (dict(K=60, xs=64), 2), (dict(N=100), 2),
           (dict(K=(1 << 20) + 8, xs=(1 << 20) + 8), 2), (dict(N=(1 << 20) + 8), 2), (dict(M=(1 << 24) + 1), 2),
           (dict(xs=56), 1), (dict(xs=0), 1), (dict(xs=-64), 1), (dict(xs=66), 2), (dict(xs=(1 << 20) + 8), 2),
           (dict(act=-1), 1), (dict(act=3), 1), (dict(x=None), 1), (dict(x=P + 2), 1), (dict(wg=None), 1),
           (dict(wu=None), 1), (dict(wd=None), 1), (dict(wg=P + 8), 1), (dict(ws=None), 1), (dict(wsb=64), 1),
           (dict(ws=P + 4), 1), (dict(g=P + 2), 1), (dict(u=P + 2), 1)]


@pytest.mark.parametrize("kw,code", FFN_BAD + [(dict(y=None), 1), (dict(yt=2), 1), (dict(y=P + 8), 1)])
def test_gated_ffn_fwd_rejects(tw, kw, code):
    base = dict(x=P, xs=64, wg=P, wu=P, wd=P, act=1, M=4, K=64, N=128, g=None, u=None, y=P, yt=0, ws=P,
                wsb=1 << 30)
    order = "x xs wg wu wd act M K N g u y yt ws wsb"
    assert call(tw._lib.tw_gated_ffn_fwd, order, base, kw) == code
    assert tw._lib.tw_last_error()


@pytest.mark.parametrize("kw,code", FFN_BAD + [
    (dict(dy=None), 1), (dict(dy=P + 8), 1), (dict(g=None), 1), (dict(u=None), 1), (dict(dx=P + 2), 1),
    (dict(dxt=2), 1), (dict(dwt=2), 1), (dict(dwg=None), 1), (dict(dwu=None), 1), (dict(dwd=None), 1),
    (dict(dwd=P + 4), 1)])
def test_gated_ffn_bwd_rejects(tw, kw, code):
    base = dict(dy=P, x=P, xs=64, wg=P, wu=P, wd=P, act=1, g=P, u=P, M=4, K=64, N=128, dx=P, dxt=0, dwg=P,
                dwu=P, dwd=P, dwt=0, ws=P, wsb=1 << 30)
    order = "dy x xs wg wu wd act g u M K N dx dxt dwg dwu dwd dwt ws wsb"
    assert call(tw._lib.tw_gated_ffn_bwd, order, base, kw) == code


# -------------------------------------------------------------- cross entropy --
CE_BAD = [(dict(M=-1), 1), (dict(K=0), 1), (dict(V=0), 1), (dict(V=-5), 1), (dict(K=60, xs=64), 2),
          (dict(V=(1 << 24) + 1), 2), (dict(M=(1 << 24) + 1), 2), (dict(xs=56), 1), (dict(xs=68), 2),
          (dict(x=None), 1), (dict(w=None), 1), (dict(w=P + 8), 1), (dict(t=None), 1), (dict(t=P + 8), 1),
          (dict(tt=0), 1), (dict(tt=5), 1), (dict(lse=None), 1), (dict(lse=P + 4), 1), (dict(ws=None), 1),
          (dict(wsb=16), 1)]


@pytest.mark.parametrize("kw,code", CE_BAD + [(dict(loss=None), 1)])
def test_linear_ce_fwd_rejects(tw, kw, code):
    base = dict(x=P, xs=64, w=P, t=P, tt=4, M=4, K=64, V=1001, loss=P, lse=P, ws=P, wsb=1 << 40)
    assert call(tw._lib.tw_linear_ce_fwd, "x xs w t tt M K V loss lse ws wsb", base, kw) == code
    assert tw._lib.tw_last_error()


@pytest.mark.parametrize("kw,code", CE_BAD + [(dict(dl=None), 1), (dict(dx=P + 4), 1), (dict(dxt=3), 1),
                                              (dict(dw=P + 4), 1), (dict(dwt=3), 1)])
def test_linear_ce_bwd_rejects(tw, kw, code):
    base = dict(dl=P, x=P, xs=64, w=P, t=P, tt=4, lse=P, M=4, K=64, V=1001, dx=P, dxt=0, dw=P, dwt=0, ws=P,
                wsb=1 << 40)
    assert call(tw._lib.tw_linear_ce_bwd, "dl x xs w t tt lse M K V dx dxt dw dwt ws wsb", base, kw) == code


def test_workspace_queries(tw):
    """0 for what the calls reject, and no error message left behind."""
    L = tw._lib
    assert L.tw_gated_ffn_fwd(None, 0, None, None, None, 0, -1, 0, 0, None, None, None, 0, None, 0, None,
                              None) == 1
    message = L.tw_last_error()
    assert tw.tw_gated_ffn_workspace_bytes(4, 60, 64) == 0 and tw.tw_gated_ffn_bwd_workspace_bytes(4, 64, 3) == 0
    assert tw.tw_linear_ce_workspace_bytes(4, 64, 0) == 0 and tw.tw_linear_ce_bwd_workspace_bytes(-4, 64, 8) == 0
    assert tw.tw_rmsnorm_bwd_workspace_bytes(4, 0) == 0
    assert L.tw_last_error() == message
    assert tw.tw_gated_ffn_workspace_bytes(100, 64, 72) >= 100 * 72 * 2
    assert tw.tw_gated_ffn_bwd_workspace_bytes(100, 64, 72) >= 3 * 100 * 72 * 2
    # a piece of D is bounded whatever the vocabulary
    assert tw.tw_linear_ce_bwd_workspace_bytes(4096, 64, 1 << 24) < (1 << 30)
    assert tw.tw_linear_ce_bwd_workspace_bytes(4096, 64, 1000) >= 4096 * 1000 * 2
    assert L.tw_grad_norm_workspace_bytes(-1, None) == 0 and L.tw_grad_norm_workspace_bytes(3, None) == 0


# ------------------------------------------------------------------- clipping --
def clip(tw, g=(P, Q), n=(100, 50), gt=(1, 1), out=None, ot=None, most=1.0, eps=1e-6, norm=0x300000,
         ws=0x400000, wsb=1 << 20, count=None):
    out, ot = g if out is None else out, gt if ot is None else ot
    k = len(g)
    return tw._lib.tw_grad_clip(k if count is None else count, (ctypes.c_void_p * k)(*g),
                                (ctypes.c_int64 * k)(*n), (ctypes.c_int * k)(*gt), (ctypes.c_void_p * k)(*out),
                                (ctypes.c_int * k)(*ot), most, eps, norm, ws, wsb, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(count=-1), 1), (dict(count=(1 << 20) + 1), 2), (dict(gt=(1, 2)), 1), (dict(n=(-1, 5)), 1),
    (dict(n=(5, (1 << 34) + 1)), 2), (dict(g=(P, None)), 1), (dict(g=(P + 2, Q)), 1),
    (dict(g=(P + 1, Q), gt=(0, 1)), 1), (dict(most=-1.0), 1), (dict(most=float("nan")), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(norm=None), 1), (dict(norm=P + 2), 1), (dict(ws=None), 1),
    (dict(wsb=4), 1), (dict(out=(P, None)), 1), (dict(ot=(1, 3)), 1),
    # outputs that overlap: each other, another gradient, their own at another place or of another type
    (dict(out=(P, P)), 1), (dict(out=(0x500000, 0x500000 + 396)), 1), (dict(out=(Q, P)), 1),
    (dict(out=(P + 4, Q)), 1), (dict(out=(P, Q), ot=(0, 1)), 1), (dict(out=(0x500000, P + 8)), 1),
    (dict(g=(P, P), n=(100, 100)), 1)])
def test_grad_clip_rejects(tw, kw, code):
    assert clip(tw, **kw) == code
    assert tw._lib.tw_last_error()


@pytest.mark.parametrize("kw", [dict(g=None), dict(n=None), dict(gt=None), dict(norm=None)])
def test_grad_norm_rejects(tw, kw):
    a = dict(g=(ctypes.c_void_p * 1)(P), n=(ctypes.c_int64 * 1)(8), gt=(ctypes.c_int * 1)(1), norm=P)
    a.update(kw)
    assert tw._lib.tw_grad_norm(1, a["g"], a["n"], a["gt"], a["norm"], P, 1 << 20, None, None) == 1


# -------------------------------------------------------------------- binding --
def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_cpu_and_wrong_tensors(tw):
    x, gamma, w = z(4, 64), z(64, dtype=F32), z(128, 64)
    t, v = z(4, dtype=I64), z(4, dtype=F32)
    for f in (lambda: tw.rmsnorm(x, gamma), lambda: tw.rmsnorm_quantize(x, gamma),
              lambda: tw.rmsnorm_backward(x, x, gamma, v), lambda: tw.gated_ffn(x, w, w, w),
              lambda: tw.gated_ffn_backward(x, x, w, w, w, z(4, 128), z(4, 128)),
              lambda: tw.linear_ce(x, w, t), lambda: tw.linear_ce_backward(v, x, w, t, v),
              lambda: tw.grad_norm([x]), lambda: tw.clip_grads([x], 1.0)):
        with pytest.raises(ValueError, match="device tensors"):
            f()
    bad = [lambda: tw.rmsnorm(z(4), gamma), lambda: tw.rmsnorm(x, z(65, dtype=F32)),
           lambda: tw.rmsnorm(x, z(64)), lambda: tw.rmsnorm(x, gamma, add=z(4, 65)),
           lambda: tw.rmsnorm(x, gamma, out_dtype=I8), lambda: tw.rmsnorm(x.int(), gamma),
           lambda: tw.rmsnorm_backward(z(5, 64), x, gamma, v),
           lambda: tw.rmsnorm_backward(x, x, gamma, z(5, dtype=F32)),
           lambda: tw.gated_ffn(x.float(), w, w, w), lambda: tw.gated_ffn(x, w, w, z(128, 72)),
           lambda: tw.gated_ffn(x, w, w.float(), w), lambda: tw.gated_ffn(x, w, w, w, act="tanh"),
           lambda: tw.gated_ffn(x, w, w, w, out_dtype=torch.float16),
           lambda: tw.gated_ffn(x.t(), z(128, 4), z(128, 4), z(128, 4)),
           lambda: tw.gated_ffn_backward(x, x, w, w, w, z(4, 120), z(4, 128)),
           lambda: tw.gated_ffn_backward(x.float(), x, w, w, w, z(4, 128), z(4, 128)),
           lambda: tw.linear_ce(x, w, z(5, dtype=I64)), lambda: tw.linear_ce(x, w, v),
           lambda: tw.linear_ce(x, z(128, 72), t),
           lambda: tw.linear_ce_backward(z(4), x, w, t, v), lambda: tw.grad_norm([]),
           lambda: tw.grad_norm([1.0]), lambda: tw.clip_grads([x, z(3, dtype=I64)], 1.0),
           lambda: tw.clip_grads([x], 1.0, out=[z(4, 65)]), lambda: tw.clip_grads([x], 1.0, out=[])]
    for f in bad:
        with pytest.raises((ValueError, TypeError)):
            f()


# ----------------------------------------------------------------- references --
def grad_of(f, *ts):
    ts = [t.clone().requires_grad_() for t in ts]
    f(*ts).backward()
    return [t.grad for t in ts]


def test_references_agree_with_autograd():
    g = torch.Generator().manual_seed(0)

    def r(*shape):
        return torch.randn(*shape, generator=g, dtype=torch.float64)

    M, K, N = 5, 8, 16
    x, gamma, dy = r(M, K), r(K), r(M, K)
    dx, dg = grad_of(lambda x, gamma: (torch.nn.functional.rms_norm(x, (K,), gamma, 1e-5) * dy).sum(), x, gamma)
    y, _, rstd, _ = R.rms(x, gamma, 1e-5, False)
    assert torch.allclose(y, torch.nn.functional.rms_norm(x, (K,), gamma, 1e-5))
    got = R.rms_bwd(dy, x, gamma, rstd, None)
    assert torch.allclose(got[0], dx) and torch.allclose(got[2], dg)
    w = [r(N, K), r(N, K), r(N, K)]
    F = torch.nn.functional
    for name, f in (("relu", torch.relu), ("silu", F.silu), ("gelu", lambda v: F.gelu(v, approximate="tanh"))):
        def ffn(x, wg, wu, wd):
            return (f(x @ wg.T) * (x @ wu.T)) @ wd

        y, _, gate, _, up, _ = R.ffn(x, *w, name)
        assert torch.allclose(y, ffn(x, *w))
        ref = grad_of(lambda *a: (ffn(*a) * dy).sum(), x, *w)
        got = R.ffn_bwd(dy, x, *w, gate, up, name)
        for k, v in zip(("dx", "dwg_t", "dwu_t", "dwd"), ref):
            assert torch.allclose(got[k][0], v), (name, k)
    t, dloss = torch.tensor([3, -100, 0, 15, 7]), r(M)
    loss, _, lse, _ = R.ce(x, w[0], t)
    assert torch.allclose(loss, F.cross_entropy(x @ w[0].T, t, reduction="none", ignore_index=-100))
    ref = grad_of(lambda x, w: (F.cross_entropy(x @ w.T, t, reduction="none", ignore_index=-100) * dloss).sum(),
                  x, w[0])
    got = R.ce_bwd(dloss, x, w[0], t, lse)
    assert torch.allclose(got["dx"][0], ref[0]) and torch.allclose(got["dw"][0], ref[1])


def test_bounds_catch_mistakes():
    """A dropped row, a wrong derivative and a missing target leave the bounds."""
    g = torch.Generator().manual_seed(0)

    def r(*shape):
        return torch.randn(*shape, generator=g, dtype=torch.float64)

    M, K, N = 33, 64, 72
    x, dy, w = r(M, K), r(M, K), [r(N, K) / 8 for _ in range(3)]
    y, ey, gate, _, up, _ = R.ffn(x, *w, "silu")
    assert R.close(y.float(), y, ey)
    with pytest.raises(AssertionError):
        R.close(R.ffn(x, *w, "gelu")[0].float(), y, ey)
    ref = R.ffn_bwd(dy, x, *w, gate, up, "silu")
    short = R.ffn_bwd(dy[1:], x[1:], *w, gate[1:], up[1:], "silu")
    for k in ("dwg_t", "dwu_t", "dwd"):
        with pytest.raises(AssertionError):
            R.close(short[k][0].float(), *ref[k])
    t = torch.randint(0, N, (M,), generator=g)
    lse = R.ce(x, w[0], t)[2]
    ref = R.ce_bwd(dy[:, 0], x, w[0], t, lse)
    other = R.ce_bwd(dy[:, 0], x, w[0], torch.where(torch.arange(M) == 3, -100, t), lse)
    for k in ("dx", "dw"):
        with pytest.raises(AssertionError):
            R.close(other[k][0].float(), *ref[k])
