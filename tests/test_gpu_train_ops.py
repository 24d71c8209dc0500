"""The dense training step's operators on the GPU against float64, with error
bounds derived in train_ref.py: RMS norm, gated FFN, cross entropy, gradient
clipping; odd sizes, strides, empty and extreme rows, streams, graphs,
repeatability."""
import math

import numpy as np
import pytest

import norm_ref as NR
import train_ref as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def tw():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from activation_sparse_feed_gate_amd import tw as mod

    return mod


def d64(t):
    return t.detach().to(torch.float64)


def rnd(seed, *shape, std=1.0, dtype=BF, pad=0):
    g = torch.Generator().manual_seed(seed)
    t = torch.randn(*shape[:-1], shape[-1] + pad, generator=g) * std
    return t.to(dtype).cuda()[..., :shape[-1]]


def same(a, b):
    """Bit-equal dicts of tensors (None where there is none)."""
    assert a.keys() == b.keys()
    for k in a:
        assert (a[k] is None) == (b[k] is None), k
        if a[k] is not None:
            assert torch.equal(a[k].view(torch.uint8) if a[k].dim() else a[k],
                               b[k].view(torch.uint8) if b[k].dim() else b[k]), k


# ------------------------------------------------------------------ RMS norm --
# one element, below, at and above a vector, each kernel's largest and next
WIDTHS = [1, 2, 7, 8, 9, 100, 511, 512, 513, 1001, 1024, 1025, 2048, 2056, 4096, 4097, 9999, 16384]


def check_rms(x, add, gamma, out, eps=1e-5):
    z = d64(x) if add is None else d64(x) + d64(add)
    y, ey, rstd, er = R.rms(z, d64(gamma), eps, add is not None)
    R.close(out["y"], y, ey)
    R.close(out["rstd"], rstd, er)
    if add is None:
        assert out["sum"] is None
    else:
        assert torch.equal(out["sum"], (x.float() + add.float()).to(x.dtype))


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("xt,at,yt", [(BF, None, BF), (F32, F32, BF), (BF, F32, F32), (F32, BF, F32),
                                      (BF, BF, BF), (F32, None, F32)])
def test_rms_forward(tw, K, xt, at, yt):
    M = 7 if K > 4096 else 13
    x, gamma = rnd(K, M, K, dtype=xt), 1 + 0.2 * rnd(K + 1, K, dtype=F32)
    add = None if at is None else rnd(K + 2, M, K, dtype=at)
    print(f"case M={M} K={K} {xt} {at} {yt}", flush=True)
    check_rms(x, add, gamma, tw.rmsnorm(x, gamma, add=add, out_dtype=yt))


@pytest.mark.parametrize("M", [0, 1, 2, 5, 1000, 4099])
@pytest.mark.parametrize("K", [64, 333, 5000])
def test_rms_rows(tw, M, K):
    x, gamma = rnd(M + K, M, K), 1 + 0.2 * rnd(1, K, dtype=F32)
    out = tw.rmsnorm(x, gamma)
    assert out["y"].shape == (M, K)
    if M:
        check_rms(x, None, gamma, out)
    dy = rnd(3, M, K, dtype=F32)
    got = tw.rmsnorm_backward(dy, x, gamma, out["rstd"])
    dx, ex, dg, eg = R.rms_bwd(d64(dy), d64(x), d64(gamma), d64(out["rstd"]), None)
    R.close(got["dx"], dx, ex)
    R.close(got["dgamma"], dg, eg)


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("dt,xt,ot,res", [(BF, BF, BF, False), (F32, BF, F32, True), (BF, F32, BF, True),
                                          (F32, F32, F32, False)])
def test_rms_backward(tw, K, dt, xt, ot, res):
    M = 29
    x, gamma = rnd(K, M, K, dtype=xt, std=3.0), 1 + 0.2 * rnd(K + 1, K, dtype=F32)
    dy = rnd(K + 2, M, K, dtype=dt)
    dres = rnd(K + 3, M, K, dtype=ot) if res else None
    rstd = tw.rmsnorm(x, gamma)["rstd"]
    got = tw.rmsnorm_backward(dy, x, gamma, rstd, dres=dres, dx_dtype=ot)
    dx, ex, dg, eg = R.rms_bwd(d64(dy), d64(x), d64(gamma), d64(rstd), None if dres is None else d64(dres))
    R.close(got["dx"], dx, ex)
    R.close(got["dgamma"], dg, eg)


@pytest.mark.parametrize("K", [1, 8, 100, 1024, 2048, 4100, 16384])
@pytest.mark.parametrize("xt,at", [(BF, None), (F32, BF)])
def test_rms_quantize(tw, K, xt, at):
    """Codes are the norm's values to within half a step and the norm's error."""
    x, gamma = rnd(K, 9, K, dtype=xt), 1 + 0.2 * rnd(K + 1, K, dtype=F32)
    add = None if at is None else rnd(K + 2, 9, K, dtype=at)
    out = tw.rmsnorm_quantize(x, gamma, add=add)
    z = d64(x) if add is None else d64(x) + d64(add)
    y, ey, _, _ = R.rms(z, d64(gamma), 1e-5, add is not None)
    step = y.abs().amax(1) / 127
    R.close(out["scale"], step, ey.amax(1) / 127 + 2 * R.U * step)
    got = d64(out["q"]) * d64(out["scale"])[:, None]
    # half a step, and the codes' own products of three roundings
    assert ((got - y).abs() <= 0.5 * step[:, None] + ey + 130 * 4 * R.U * step[:, None] + R.TINY).all()
    assert int(out["q"].abs().max()) <= 127
    if add is not None:
        assert torch.equal(out["sum"], (x.float() + add.float()).to(x.dtype))


@pytest.mark.parametrize("pad", [1, 3, 8])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rms_strided(tw, pad, dtype):
    x, gamma = rnd(5, 9, 1001, dtype=dtype, pad=pad), 1 + 0.2 * rnd(1, 1001, dtype=F32)
    a, b = tw.rmsnorm(x, gamma), tw.rmsnorm(x.contiguous(), gamma)
    same(a, b)
    same(tw.rmsnorm_quantize(x, gamma), tw.rmsnorm_quantize(x.contiguous(), gamma))
    dy = rnd(6, 9, 1001)
    same(tw.rmsnorm_backward(dy, x, gamma, a["rstd"]), tw.rmsnorm_backward(dy, x.contiguous(), gamma, a["rstd"]))


@pytest.mark.parametrize("K", [9, 64, 1001, 2048, 2056])
def test_rms_extreme_rows(tw, K):
    """Rows of zeros (with eps and without), of NaN and infinities: their
    neighbours are as they are without them."""
    x, gamma = rnd(K, 8, K, dtype=F32), 1 + 0.2 * rnd(1, K, dtype=F32)
    plain = tw.rmsnorm(x, gamma, out_dtype=F32)
    odd = x.clone()
    odd[1], odd[3, K // 2], odd[5, 0] = 0.0, float("nan"), float("inf")
    out, q = tw.rmsnorm(odd, gamma, out_dtype=F32), tw.rmsnorm_quantize(odd, gamma)
    keep = [0, 2, 4, 6, 7]
    assert torch.equal(out["y"][keep], plain["y"][keep])
    assert (out["y"][1] == 0).all() and (q["q"][1] == 0).all() and q["scale"][1] == 0
    assert out["y"][3].isnan().all() and q["scale"][3].isnan()
    assert out["y"][5, 0].isnan() and (out["y"][5, 1:] == 0).all() and q["scale"][5].isnan()
    # without eps a row of zeros has an infinite rstd: 0 times it is NaN there, and nowhere else
    bare = tw.rmsnorm(odd, gamma, eps=0.0, out_dtype=F32)
    assert bare["y"][1].isnan().all() and bare["rstd"][1].isinf()
    R.close(bare["y"][keep], *R.rms(d64(x[keep]), d64(gamma), 0.0, False)[:2])


def test_rms_sum_in_place(tw):
    x, add, gamma = rnd(1, 33, 2048), rnd(2, 33, 2048, dtype=F32), 1 + 0.2 * rnd(3, 2048, dtype=F32)
    ref = tw.rmsnorm(x, gamma, add=add)
    y = torch.empty_like(x)
    tw.tw_rmsnorm_fwd(x, gamma, 1e-5, y, add=add, total=x)
    assert torch.equal(y, ref["y"]) and torch.equal(x, ref["sum"])


def test_rms_gradient_by_differences(tw):
    """dx and dgamma against central differences of the kernel's own forward, in fp32."""
    x, gamma, dy = rnd(1, 3, 24, dtype=F32), 1 + 0.2 * rnd(2, 24, dtype=F32), rnd(3, 3, 24, dtype=F32)

    def loss(x, gamma):
        return float((d64(tw.rmsnorm(x, gamma, out_dtype=F32)["y"]) * d64(dy)).sum())

    got = tw.rmsnorm_backward(dy, x, gamma, tw.rmsnorm(x, gamma)["rstd"])
    h = 2.0 ** -6
    # the third derivative's term h^2, and 72 values off by 1e-5 of their size over 2 h
    tol = 24 * h * h + 72 * 4 * 100 * R.U / (2 * h)
    for i, j in [(0, 0), (1, 7), (2, 23)]:
        a, b = x.clone(), x.clone()
        a[i, j] += h
        b[i, j] -= h
        step = float(d64(a[i, j]) - d64(b[i, j]))
        assert abs((loss(a, gamma) - loss(b, gamma)) / step - float(got["dx"][i, j])) < tol
    for j in (0, 11):
        a, b = gamma.clone(), gamma.clone()
        a[j] += h
        b[j] -= h
        step = float(d64(a[j]) - d64(b[j]))
        assert abs((loss(x, a) - loss(x, b)) / step - float(got["dgamma"][j])) < tol


# ----------------------------------------------------------------- gated FFN --
# (M, K, N): one token, few, tiles' edges, sizes no tile divides, one vector wide
SHAPES = [(1, 8, 8), (1, 2048, 5632), (2, 136, 264), (3, 1024, 4096), (5, 1000, 2728), (8, 512, 1032),
          (16, 2048, 1024), (17, 264, 520), (32, 1024, 72), (64, 1016, 1000), (127, 128, 128),
          (128, 128, 256), (129, 136, 136), (200, 8, 1000), (300, 1000, 8), (777, 1000, 2728),
          (1024, 1024, 1024), (2048, 520, 1096),
          # enough for the larger tiles: whole ones, and ragged in every size
          (4096, 2048, 2048), (4100, 2056, 2104), (4104, 72, 4168), (520, 4104, 4104)]


def weights(K, N, seed=0):
    return (rnd(seed + 1, N, K, std=K ** -0.5), rnd(seed + 2, N, K, std=K ** -0.5),
            rnd(seed + 3, N, K, std=N ** -0.5))


def check_ffn(x, w, act, out):
    y, ey, g, eg, u, eu = R.ffn(d64(x), *(d64(t) for t in w), act)
    R.close(out["y"], y, ey)
    if out["g"] is not None:
        R.close(out["g"], g, eg)
        R.close(out["u"], u, eu)


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("act,keep,yt", [("silu", True, BF), ("gelu", False, F32), ("relu", True, F32)])
def test_ffn_forward(tw, M, K, N, act, keep, yt):
    print(f"case {M}x{K}x{N} {act}", flush=True)
    x, w = rnd(M, M, K), weights(K, N)
    check_ffn(x, w, act, tw.gated_ffn(x, *w, act=act, keep=keep, out_dtype=yt))


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("act,xt,wt", [("silu", BF, BF), ("gelu", F32, BF), ("relu", BF, F32)])
def test_ffn_backward(tw, M, K, N, act, xt, wt):
    print(f"case {M}x{K}x{N} {act}", flush=True)
    x, w, dy = rnd(M, M, K), weights(K, N), rnd(M + 1, M, K)
    g, u = rnd(M + 2, M, N, std=1.5), rnd(M + 3, M, N)
    got = tw.gated_ffn_backward(dy, x, *w, g, u, act=act, dx_dtype=xt, dw_dtype=wt)
    ref = R.ffn_bwd(d64(dy), d64(x), *(d64(t) for t in w), d64(g), d64(u), act)
    for k, (v, e) in ref.items():
        R.close(got[k], v, e)


@pytest.mark.parametrize("M", [1, 16, 100, 300])
@pytest.mark.parametrize("pad", [8, 24])
def test_ffn_strided(tw, M, pad):
    """Rows of a wider buffer whose other columns are NaN: the same bits as a
    contiguous copy's."""
    K, N = 264, 520
    wide = torch.full((M, K + pad), float("nan"), dtype=BF, device="cuda")
    x = wide[:, :K]
    x.copy_(rnd(1, M, K))
    w, dy = weights(K, N), rnd(2, M, K)
    a, b = tw.gated_ffn(x, *w, keep=True), tw.gated_ffn(x.contiguous(), *w, keep=True)
    same(a, b)
    same(tw.gated_ffn_backward(dy, x, *w, a["g"], a["u"]),
         tw.gated_ffn_backward(dy, x.contiguous(), *w, a["g"], a["u"]))


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_ffn_no_rows(tw, act):
    x, w = rnd(1, 0, 64), weights(64, 72)
    out = tw.gated_ffn(x, *w, act=act, keep=True)
    assert out["y"].shape == (0, 64) and out["g"].shape == (0, 72)
    for wt in (BF, F32):
        got = tw.gated_ffn_backward(x, x, *w, out["g"], out["u"], act=act, dw_dtype=wt)
        assert got["dx"].shape == (0, 64) and all((got[k] == 0).all() for k in ("dwg_t", "dwu_t", "dwd"))


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("M", [4, 150])
def test_ffn_nan_stays_in_its_row(tw, act, M):
    K, N = 136, 264
    x, w = rnd(1, M, K), weights(K, N)
    odd = x.clone()
    odd[M - 2, 5] = float("nan")
    a, b = tw.gated_ffn(x, *w, act=act), tw.gated_ffn(odd, *w, act=act)
    keep = [i for i in range(M) if i != M - 2]
    assert torch.equal(a["y"][keep], b["y"][keep]) and b["y"][M - 2].isnan().all()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_ffn_saturated_gates(tw, act):
    """Gates far past the logistic function's range, infinities among them in
    the gradient's input: no NaN where the formula's limit is a number."""
    M, K, N = 6, 64, 72
    w, x, dy = weights(K, N), rnd(1, M, K), rnd(2, M, K)
    g = torch.tensor([-3e38, -1e20, -200.0, -90.0, 90.0, 200.0, 1e20, 3e38], dtype=BF).cuda()
    g = g.repeat(M, N // 8).contiguous()
    u = rnd(3, M, N, std=1e-3)
    wide = d64(g).requires_grad_()
    f = torch.nn.functional.silu(wide) if act == "silu" else wide * (wide > 0)
    slope = torch.autograd.grad(f.sum(), wide)[0]
    dh = R.mm(d64(dy), d64(w[2]).T)
    got = tw.gated_ffn_backward(dy, x, *w, g, u, act=act, dw_dtype=F32)
    dz = dh * d64(u) * slope
    e = 0.02 * R.mm(dz.abs().T, d64(x).abs())
    assert ((d64(got["dwg_t"]) - R.mm(dz.T, d64(x))).abs() <= e + 1e-20).all()


def test_ffn_gradient_by_differences(tw):
    """The float64 formula's gradient by differences; the kernel is held to the
    formula above."""
    M, K, N = 3, 8, 16
    for act in ("silu", "gelu", "relu"):
        x, w = d64(rnd(1, M, K)), [d64(t) for t in weights(K, N)]
        dy = d64(rnd(4, M, K))

        def loss(x, w):
            return (R.ffn(x, *w, act)[0] * dy).sum()

        _, _, g, _, u, _ = R.ffn(x, *w, act)
        ref = R.ffn_bwd(dy, x, *w, g, u, act)
        h = 1e-5
        for name, t in (("dx", x), ("dwg_t", w[0]), ("dwu_t", w[1]), ("dwd", w[2])):
            keep = t[1, 3].item()
            t[1, 3] = keep + h
            up = loss(x, w)
            t[1, 3] = keep - h
            down = loss(x, w)
            t[1, 3] = keep
            assert abs(((up - down) / (2 * h) - ref[name][0][1, 3]).item()) < 1e-6


# -------------------------------------------------------------- cross entropy --
CE = [(1, 8, 1), (1, 64, 2), (1, 1024, 32768), (2, 136, 127), (4, 1024, 5000), (5, 72, 128), (16, 520, 129),
      (17, 64, 1000), (33, 256, 333), (64, 1000, 2049), (127, 128, 257), (129, 136, 4097),
      (300, 520, 1000), (777, 256, 5003), (1025, 64, 2000), (2048, 1024, 8192), (1029, 72, 9001),
      (2100, 2056, 4099)]


def ce_case(M, K, V, wide=True, seed=0):
    x, w = rnd(seed + M, M, K), rnd(seed + V, V, K, std=2 * K ** -0.5)
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(0, V, (M,), generator=g)
    t[torch.rand(M, generator=g) < 0.2] = -100
    return x, w, t.cuda() if wide else t.int().cuda()


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("M,K,V", CE)
def test_ce_forward(tw, M, K, V, wide):
    print(f"case {M}x{K}x{V}", flush=True)
    x, w, t = ce_case(M, K, V, wide)
    out = tw.linear_ce(x, w, t)
    loss, el, lse, es = R.ce(d64(x), d64(w), t)
    R.close(out["lse"], lse, es)
    R.close(out["loss"], loss, el)
    assert (out["loss"] >= 0).all() and (out["loss"][t < 0] == 0).all()


@pytest.mark.parametrize("M,K,V", CE)
@pytest.mark.parametrize("xt,wt", [(BF, BF), (F32, F32)])
def test_ce_backward(tw, M, K, V, xt, wt):
    print(f"case {M}x{K}x{V}", flush=True)
    x, w, t = ce_case(M, K, V, xt == BF)
    lse = torch.logsumexp(d64(x) @ d64(w).T, 1).float()
    dloss = rnd(7, M, dtype=F32)
    got = tw.linear_ce_backward(dloss, x, w, t, lse, dx_dtype=xt, dw_dtype=wt)
    for k, (v, e) in R.ce_bwd(d64(dloss), d64(x), d64(w), t, d64(lse)).items():
        R.close(got[k], v, e)


def test_ce_pieces(tw):
    """More than one piece of the vocabulary, the last a ragged one."""
    M, K, V = 8200, 64, 50001
    x, w, t = ce_case(M, K, V)
    assert tw.tw_linear_ce_bwd_workspace_bytes(M, K, V) < 2 * M * V
    lse = torch.logsumexp(x.float() @ w.float().T, 1)
    dloss = rnd(7, M, dtype=F32)
    got = tw.linear_ce_backward(dloss, x, w, t, lse, dw_dtype=F32)
    for k, (v, e) in R.ce_bwd(d64(dloss), d64(x), d64(w), t, d64(lse)).items():
        R.close(got[k], v, e)


@pytest.mark.parametrize("M", [1, 4, 40, 200])
def test_ce_strided(tw, M):
    K, V = 264, 1001
    wide = torch.full((M, K + 16), float("nan"), dtype=BF, device="cuda")
    x = wide[:, :K]
    _, w, t = ce_case(M, K, V)
    x.copy_(rnd(1, M, K))
    a = tw.linear_ce(x, w, t)
    same(a, tw.linear_ce(x.contiguous(), w, t))
    dloss = rnd(7, M, dtype=F32)
    same(tw.linear_ce_backward(dloss, x, w, t, a["lse"]),
         tw.linear_ce_backward(dloss, x.contiguous(), w, t, a["lse"]))


@pytest.mark.parametrize("M", [3, 200])
def test_ce_targets_outside(tw, M):
    """Targets below 0, at V and past 32 bits: left out."""
    K, V = 136, 300
    x, w, t = ce_case(M, K, V)
    t[0], t[1], t[2] = V, -1, (1 << 40) + 5
    out = tw.linear_ce(x, w, t)
    assert (out["loss"][:3] == 0).all() and out["lse"].isfinite().all()
    got = tw.linear_ce_backward(torch.ones(M, device="cuda"), x, w, t, out["lse"])
    assert (got["dx"][:3] == 0).all()
    none = torch.full_like(t, -100)
    out = tw.linear_ce(x, w, none)
    got = tw.linear_ce_backward(torch.ones(M, device="cuda"), x, w, none, out["lse"])
    assert (out["loss"] == 0).all() and (got["dx"] == 0).all() and (got["dw"] == 0).all()


@pytest.mark.parametrize("M", [6, 300])
def test_ce_rows_left_out_hold_anything(tw, M):
    """NaN and infinities in rows that are left out, or whose dloss is 0: their dx is 0
    and the others' as it was."""
    K, V = 136, 700
    x, w, t = ce_case(M, K, V)
    t[:] = t.clamp(min=0)
    t[0], t[M - 1] = -100, -100
    dloss = rnd(7, M, dtype=F32)
    dloss[2] = 0.0
    lse = tw.linear_ce(x, w, t)["lse"]
    ws = torch.empty(tw.tw_linear_ce_bwd_workspace_bytes(M, K, V), dtype=torch.uint8, device="cuda")
    a, b = torch.empty_like(x), torch.empty_like(x)
    tw.tw_linear_ce_bwd(dloss, x, w, t, lse, ws, dx=a)
    odd = x.clone()
    odd[0, 3], odd[2, 7], odd[M - 1] = float("nan"), float("inf"), float("-inf")
    lse = tw.linear_ce(odd, w, t)["lse"]
    tw.tw_linear_ce_bwd(dloss, odd, w, t, lse, ws, dx=b)
    assert torch.equal(a, b) and (b[[0, 2, M - 1]] == 0).all() and (b[1] != 0).any()


def test_ce_no_rows(tw):
    x, w, t = rnd(1, 0, 64), rnd(2, 100, 64), torch.empty(0, dtype=torch.int64, device="cuda")
    out = tw.linear_ce(x, w, t)
    assert out["loss"].shape == (0,)
    got = tw.linear_ce_backward(out["loss"], x, w, t, out["lse"])
    assert got["dx"].shape == (0, 64) and (got["dw"] == 0).all()


@pytest.mark.parametrize("M", [4, 150])
def test_ce_extreme_logits(tw, M):
    """Logits of thousands, one far above the rest; a row of NaN and one of an
    infinity leave the others as they are; weights of minus infinity are words
    that never come."""
    K, V = 64, 700
    x, w, t = ce_case(M, K, V, seed=3)
    x, w = x * 30, w * 30
    out = tw.linear_ce(x, w, t)
    loss, el, lse, es = R.ce(d64(x), d64(w), t)
    R.close(out["lse"], lse, es)
    R.close(out["loss"], loss, el)
    odd = x.clone()
    odd[0, 3], odd[2, 7] = float("nan"), float("inf")
    got = tw.linear_ce(odd, w, t)
    keep = [i for i in range(M) if i not in (0, 2)]
    assert torch.equal(got["lse"][keep], out["lse"][keep]) and got["lse"][0].isnan()
    x2, w2 = x.abs() + 1, w.clone()
    w2[256:512] = -float("inf")  # whole tiles of logits of minus infinity
    w2[5] = -float("inf")
    t2 = torch.zeros_like(t)
    got = tw.linear_ce(x2, w2, t2)
    live = torch.cat([w[:5], w[6:256], w[512:]])
    loss, el, lse, es = R.ce(d64(x2), d64(live), t2)
    R.close(got["lse"], lse, es)
    R.close(got["loss"], loss, el)


def test_ce_gradient_by_differences(tw):
    """The float64 formula's gradient by differences, on the formula that the
    kernel is held to."""
    x, w, t = d64(rnd(1, 4, 8)), d64(rnd(2, 11, 8)), torch.tensor([0, 10, -100, 3]).cuda()
    dloss = d64(rnd(3, 4, dtype=F32))
    ref = R.ce_bwd(dloss, x, w, t, R.ce(x, w, t)[2])
    h = 1e-5
    for name, v in (("dx", x), ("dw", w)):
        for at in ((0, 1), (3, 7)):
            keep = v[at].item()
            v[at] = keep + h
            up = (R.ce(x, w, t)[0] * dloss).sum()
            v[at] = keep - h
            down = (R.ce(x, w, t)[0] * dloss).sum()
            v[at] = keep
            assert abs(((up - down) / (2 * h) - ref[name][0][at]).item()) < 1e-6


@pytest.mark.parametrize("M", [16, 17, 32, 33, 64, 65, 256, 257])
def test_at_the_rules_row_counts(tw, M):
    """Row counts on both sides of where another kernel takes over."""
    K, N, V = 264, 1040, 1000
    x, w, dy = rnd(M, M, K), weights(K, N), rnd(M + 1, M, K)
    out = tw.gated_ffn(x, *w, keep=True)
    check_ffn(x, w, "silu", out)
    got = tw.gated_ffn_backward(dy, x, *w, out["g"], out["u"])
    for k, (v, e) in R.ffn_bwd(d64(dy), d64(x), *(d64(t) for t in w), d64(out["g"]),
                               d64(out["u"]), "silu").items():
        R.close(got[k], v, e)
    x, w, t = ce_case(M, K, V)
    out = tw.linear_ce(x, w, t)
    loss, el, lse, es = R.ce(d64(x), d64(w), t)
    R.close(out["lse"], lse, es)
    R.close(out["loss"], loss, el)


# ---------------------------------------------------------- past 32-bit offsets --
def test_ffn_past_32_bits(tw):
    """Hidden rows past 2^31 elements: the last rows' outputs, and the weight gradients of
    the first and last neurons, which every row enters."""
    M, K, N = 540_000, 64, 4096
    assert M * N > 1 << 31
    x, dy, w = rnd(1, M, K), rnd(2, M, K), weights(K, N)
    out = tw.gated_ffn(x, *w, keep=True)
    g, u = out["g"], out["u"]
    for rows in (slice(0, 40), slice(M - 300, M)):
        check_ffn(x[rows], w, "silu", {k: v[rows] for k, v in out.items()})
    got = tw.gated_ffn_backward(dy, x, *w, g, u, dx_dtype=F32, dw_dtype=F32)
    for rows in (slice(0, 40), slice(M - 300, M)):
        ref = R.ffn_bwd(d64(dy[rows]), d64(x[rows]), *(d64(t) for t in w), d64(g[rows]),
                        d64(u[rows]), "silu")
        R.close(got["dx"][rows], *ref["dx"])
    for of in (slice(0, 8), slice(N - 8, N)):
        ref = R.ffn_bwd(d64(dy), d64(x), *(d64(t[of]) for t in w), d64(g[:, of]), d64(u[:, of]),
                        "silu")
        for k in ("dwg_t", "dwu_t", "dwd"):
            R.close(got[k][of], *ref[k])
    del out, g, u, got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M", [3, 70])
def test_ce_past_32_bits(tw, M):
    """A projection of more than 2^31 elements, words at its end."""
    K, V = 2048, 1_060_000
    assert K * V > 1 << 31
    g = torch.Generator("cuda").manual_seed(M)
    w = torch.empty(V, K, dtype=BF, device="cuda").normal_(0, 2 * K ** -0.5, generator=g)
    x = rnd(M, M, K)
    t = torch.arange(V - M, V, device="cuda")
    t[1] = 5
    out = tw.linear_ce(x, w, t)
    wide = d64(w)
    loss, el, lse, es = R.ce(d64(x), wide, t)
    R.close(out["lse"], lse, es)
    R.close(out["loss"], loss, el)
    dloss = rnd(7, M, dtype=F32)
    got = tw.linear_ce_backward(dloss, x, w, t, out["lse"])
    for k, (v, e) in R.ce_bwd(d64(dloss), d64(x), wide, t, d64(out["lse"])).items():
        R.close(got[k], v, e)
    del w, wide, got, loss, el, v, e
    torch.cuda.empty_cache()


def test_rms_past_32_bits(tw):
    M, K = 1_050_000, 2048
    assert M * K > 1 << 31
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.empty(M, K, dtype=BF, device="cuda").normal_(generator=g)
    gamma = rnd(3, K, dtype=F32)
    out = tw.rmsnorm(x, gamma)
    q = tw.rmsnorm_quantize(x, gamma)
    back = tw.rmsnorm_backward(x, x, gamma, out["rstd"])
    for rows in (slice(0, 5), slice(M - 100, M)):
        a = tw.rmsnorm(x[rows], gamma)
        assert torch.equal(a["y"], out["y"][rows]) and torch.equal(a["rstd"], out["rstd"][rows])
        assert torch.equal(tw.rmsnorm_quantize(x[rows], gamma)["q"], q["q"][rows])
        assert torch.equal(tw.rmsnorm_backward(x[rows], x[rows], gamma, a["rstd"])["dx"],
                           back["dx"][rows])
    del x, out, q, back
    torch.cuda.empty_cache()


def test_clip_past_32_bits(tw):
    n = (1 << 31) + 5001
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.empty(n, dtype=BF, device="cuda").normal_(generator=g)
    ends = [x[:1000].clone(), x[-9000:].clone()]
    ref = math.sqrt(sum(float((d64(c) ** 2).sum()) for c in x.split(1 << 28)))
    # at most 2048 x 256 threads with 8 sums each, and the tree
    rel = (n / (2048 * 256 * 8) + 64) * R.U
    norm = tw.clip_grads([x], 1.0)
    assert abs(float(norm) - ref) <= rel * ref
    for was, now in zip(ends, (x[:1000], x[-9000:])):
        want = d64(was) / (ref + 1e-6)
        R.close(now, want, (2 * rel + 4 * R.U) * want.abs())
    del x
    torch.cuda.empty_cache()


# ------------------------------------------------------------------- clipping --
def check_clip(grads, out, norm, most, eps=1e-6):
    """grads: as they were.  The squares are summed 8 ways a thread."""
    total = sum(float((d64(g) ** 2).sum()) for g in grads)
    ref = math.sqrt(total)
    longest = max([g.numel() for g in grads] + [1])
    rel = (longest / (256 * 8) + 64) * R.U  # additions one after another, and the tree
    assert abs(float(norm) - ref) <= rel * ref + R.TINY
    by = most / (ref + eps)
    by, slack = (1.0, 0.0) if by > 1 + 2 * rel else (by, 2 * rel + 4 * R.U)
    for g, o in zip(grads, out):
        want = d64(g) * by
        R.close(o, want, slack * want.abs() + (0 if by != 1.0 else 0))


SIZES = [[(1,)], [(7,)], [(8192,)], [(8193,)], [(1001, 256), (256,), (0,), (3, 5, 7), (8191,)],
         [(100000,), (1,), (65536, 3)]]


@pytest.mark.parametrize("shapes", SIZES)
@pytest.mark.parametrize("gt,ot", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("by", [0.25, 4.0])
def test_clip(tw, shapes, gt, ot, by):
    grads = [rnd(i, *s, dtype=gt) for i, s in enumerate(shapes)]
    norm = math.sqrt(sum(float((d64(g) ** 2).sum()) for g in grads))
    out = [torch.full(s, 7.0, dtype=ot, device="cuda") for s in shapes]
    before = [g.clone() for g in grads]
    check_clip(before, out, tw.clip_grads(grads, by * norm, out=out), by * norm)
    assert all(torch.equal(a, b) for a, b in zip(before, grads))
    assert abs(float(tw.grad_norm(grads)) - norm) <= 1e-5 * norm


@pytest.mark.parametrize("by", [0.25, 4.0])
def test_clip_in_place(tw, by):
    grads = [rnd(1, 513, 129), rnd(2, 1000, dtype=F32), rnd(3, 33, dtype=F32)]
    before = [g.clone() for g in grads]
    norm = math.sqrt(sum(float((d64(g) ** 2).sum()) for g in grads))
    got = tw.clip_grads(grads, by * norm)
    check_clip(before, grads, got, by * norm)
    if by > 1:
        assert all(torch.equal(a, b) for a, b in zip(before, grads))


def test_clip_views_of_one_buffer(tw):
    """Neighbouring pieces of one buffer, at addresses aligned only to their
    type; what lies between and around them stays."""
    for dtype in (BF, F32):
        flat = rnd(4, 40000, dtype=dtype)
        cuts = [(1, 5000), (5003, 8192 + 17), (20001, 9), (20011, 19000)]
        grads = [flat[a:a + n] for a, n in cuts]
        before, whole = [g.clone() for g in grads], flat.clone()
        norm = math.sqrt(sum(float((d64(g) ** 2).sum()) for g in before))
        check_clip(before, grads, tw.clip_grads(grads, norm / 3), norm / 3)
        for a, n in cuts:
            whole[a:a + n] = flat[a:a + n]
        assert torch.equal(whole, flat)


@pytest.mark.parametrize("count,n", [(97, 10), (300, 33), (289, 180000)])
def test_clip_many(tw, count, n):
    """More buffers than a launch takes, and more parts than a workgroup adds
    itself."""
    flat = rnd(5, count * n)
    grads = list(flat.split(n))
    before = [g.clone() for g in grads]
    norm = float(d64(flat).norm())
    check_clip(before, grads, tw.clip_grads(grads, norm / 7), norm / 7)


def test_clip_extremes(tw):
    g = [rnd(1, 100, dtype=F32), rnd(2, 50)]
    g[0][3] = float("nan")
    assert tw.clip_grads(g, 1.0).isnan() and all(t.isnan().all() for t in g)
    g = [rnd(1, 100, dtype=F32)]
    g[0][3] = float("inf")
    assert tw.clip_grads(g, 1.0).isinf()
    assert g[0][3].isnan() and (g[0][:3] == 0).all()
    zero = [torch.zeros(1000, device="cuda")]
    assert tw.clip_grads(zero, 1.0) == 0 and (zero[0] == 0).all()
    empty = [torch.zeros(0, device="cuda")]
    assert tw.clip_grads(empty, 1.0) == 0 and tw.grad_norm(empty) == 0


# ------------------------------------------------- streams, graphs, the step --
def all_calls(tw):
    """One call of each operator on inputs of its own; f() -> dict of tensors."""
    x, gamma, add = rnd(1, 150, 264), 1 + 0.2 * rnd(2, 264, dtype=F32), rnd(3, 150, 264, dtype=F32)
    w, dy = weights(264, 520), rnd(4, 150, 264)
    g, u = rnd(5, 150, 520), rnd(6, 150, 520)
    few = rnd(7, 3, 264)
    cx, cw, ct = ce_case(150, 264, 1001)
    dloss = rnd(8, 150, dtype=F32)
    lse = tw.linear_ce(cx, cw, ct)["lse"].clone()
    rstd = tw.rmsnorm(x, gamma)["rstd"].clone()
    grads = [rnd(9, 300, 77), rnd(10, 12345, dtype=F32)]
    out = [torch.empty(t.shape, device="cuda") for t in grads]

    def clip():
        norm = tw.clip_grads(grads, 1.0, out=out)
        return {"norm": norm, "a": out[0], "b": out[1]}

    return {
        "rmsnorm": lambda: tw.rmsnorm(x, gamma, add=add),
        "rmsnorm_quantize": lambda: tw.rmsnorm_quantize(x, gamma, add=add),
        "rmsnorm_backward": lambda: tw.rmsnorm_backward(dy, x, gamma, rstd),
        "gated_ffn": lambda: tw.gated_ffn(x, *w, keep=True),
        "gated_ffn_few": lambda: tw.gated_ffn(few, *w, keep=True),
        "gated_ffn_backward": lambda: tw.gated_ffn_backward(dy, x, *w, g, u),
        "linear_ce": lambda: tw.linear_ce(cx, cw, ct),
        "linear_ce_few": lambda: tw.linear_ce(cx[:3], cw, ct[:3]),
        "linear_ce_backward": lambda: tw.linear_ce_backward(dloss, cx, cw, ct, lse),
        "clip": clip,
    }


NAMES = ["rmsnorm", "rmsnorm_quantize", "rmsnorm_backward", "gated_ffn", "gated_ffn_few",
         "gated_ffn_backward", "linear_ce", "linear_ce_few", "linear_ce_backward", "clip"]


def copied(d):
    return {k: None if v is None else v.clone() for k, v in d.items()}


@pytest.mark.parametrize("name", NAMES)
def test_repeatable_and_on_another_stream(tw, name):
    f = all_calls(tw)[name]
    first = copied(f())
    same(first, f())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = f()
    s.synchronize()
    same(first, got)


@pytest.mark.parametrize("name", NAMES)
def test_native_call_equals_the_checked_one(tw, name, monkeypatch):
    """The native part of the binding takes the call, and the checked Python way
    gives the same bits."""
    f = all_calls(tw)[name]
    native, taken = tw._calls, []

    class Spy:
        def __getattr__(self, k):
            def run(*a):
                got = getattr(native, k)(*a)
                taken.append((k, got is not None))
                return got
            return run

    class Never:
        def __getattr__(self, k):
            return lambda *a: None

    monkeypatch.setattr(tw, "_calls", Spy())
    first = copied(f())
    assert taken and all(ok for _, ok in taken), taken
    monkeypatch.setattr(tw, "_calls", Never())
    same(first, f())


@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(tw, name):
    f = all_calls(tw)[name]
    first = copied(f())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = f()
    for i in range(3):
        for v in got.values():
            if v is not None:
                v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        same(first, got)
        same(first, f())


def test_two_graphs_and_two_streams_at_once(tw):
    """Captured calls with workspaces of their own, replayed on two streams at
    the same time, with eager calls between."""
    calls = all_calls(tw)
    names = ["gated_ffn_backward", "linear_ce_backward", "clip", "linear_ce"]
    first = {n: copied(calls[n]()) for n in names}
    torch.cuda.synchronize()
    graphs = {}
    for n in names[:2]:
        graphs[n] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[n]):
            first[n + " got"] = calls[n]()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(a):
            graphs[names[0]].replay()
        with torch.cuda.stream(b):
            graphs[names[1]].replay()
        eager = {n: copied(calls[n]()) for n in names[2:]}
        torch.cuda.synchronize()
        for n in names[:2]:
            same(first[n], first[n + " got"])
        for n in names[2:]:
            same(first[n], eager[n])


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_training_step(tw, act):
    """A stack of sublayers, loss, gradients and clipping, as a program would
    use them, against float64 (bf16 operands: a per cent of a gradient's
    norm).

    ReLU's derivative jumps at 0, so a gate whose sign differs changes a gradient by
    its whole entry.  Gates are standard normal; the norm's output, rounded to
    bf16 (2^-9 of a value, over sqrt(3), on average), and the stream before it, off
    by about as much, move them by up to d = 2^-8 or so: a share f = 2 d 0.4 = 0.0031
    of them lies that close to 0, against the half that is on, and the gradient's
    norm moves by up to sqrt(f / 0.5) = 0.08."""
    from activation_sparse_feed_gate_amd import block

    off = block.dense_main(act=act)
    assert off.pop("loss") < 2e-3 and off.pop("served loss") < 2e-3, off
    assert all(v < (0.08 if act == "relu" else 0.02) for v in off.values()), off


def test_serving_on_rms_norms(tw):
    """block.serve with RMS norms, the int8 sublayer in float64 on the same
    codes' definition: half a code a value through two products."""
    from activation_sparse_feed_gate_amd import block

    M, K, N = 5, 256, 512
    x = rnd(1, M, K, dtype=F32)
    w = weights(K, N)
    layers = [(1 + 0.1 * rnd(i, K, dtype=F32), None, block.quantize_ffn(*w)) for i in (2, 3)]
    y, stream = block.serve(x, layers, layers[0][0], norm="rms")
    z = d64(x)
    for gamma, _, _ in layers:
        n = R.rms(z, d64(gamma), 1e-5, False)[0]
        z = z + R.mm(torch.relu(R.mm(n, d64(w[0]).T)) * R.mm(n, d64(w[1]).T), d64(w[2]))
    assert float((d64(stream) - z).norm() / z.norm()) < 0.03
    ref = R.rms(z, d64(layers[0][0]), 1e-5, False)[0]
    assert y.dtype == BF and float((d64(y) - ref).norm() / ref.norm()) < 0.03
    with pytest.raises(ValueError):
        block.serve(x, [(layers[0][0], layers[0][0], layers[0][2])], layers[0][0], norm="rms")
    with pytest.raises(ValueError):
        block.serve(x, layers, layers[0][0], norm="none")
