"""Layer norm (forward, backward, int8) on the GPU against float64, with
error bounds derived in norm_ref.py; strides, odd rows, extreme rows,
gradients by differences, streams, graphs and repeatability."""
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


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def rows(M, K, dtype, seed, offset=0.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K + pad, generator=g) * (1 + torch.rand(K + pad, generator=g)) + offset
    return x.to(dtype).cuda()[:, :K]


def params(K, seed, beta=True):
    g = torch.Generator().manual_seed(seed)
    gamma = (1 + 0.2 * torch.randn(K, generator=g)).cuda()
    return gamma, (0.3 * torch.randn(K, generator=g)).cuda() if beta else None


# rows of one element, below and above a vector, each kernel's largest and
# next sizes (512, 1024, 2048, 4096, 16384), odd ones
WIDTHS = [1, 2, 7, 8, 9, 100, 511, 512, 513, 1001, 1024, 1025, 2047, 2048, 2056, 4095, 4096, 4097,
          9999, 16384]


def check_forward(x, add, gamma, beta, out, eps=1e-5):
    z32 = x.float() + add.float() if add is not None else x.float()
    z = f64(x) + f64(add) if add is not None else f64(x)
    y, mean, rstd, e_y, e_m, e_r = R.norm(z, f64(gamma), None if beta is None else f64(beta), eps,
                                          out["y"].dtype == BF)
    # where there is an add, z itself is rounded to fp32 once
    slack = R.U * np.abs(z) * np.abs(f64(gamma)) * rstd[:, None] if add is not None else 0.0
    assert (np.abs(f64(out["y"]) - y) <= e_y + slack).all()
    assert (np.abs(f64(out["mean"]) - mean) <= e_m).all()
    assert (np.abs(f64(out["rstd"]) - rstd) <= e_r).all()
    if add is not None:
        assert torch.equal(out["sum"], z32.to(x.dtype))


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("xt,at,yt", [(BF, None, BF), (F32, F32, BF), (BF, F32, F32), (F32, BF, F32),
                                      (BF, BF, BF), (F32, None, F32)])
def test_forward(tw, K, xt, at, yt):
    M = 7 if K > 4096 else 13
    x = rows(M, K, xt, K, offset=0.5)
    add = None if at is None else rows(M, K, at, K + 1)
    gamma, beta = params(K, K + 2, beta=K % 2 == 0)
    print(f"case M={M} K={K} {xt} {at} {yt}", flush=True)
    check_forward(x, add, gamma, beta, tw.layernorm(x, gamma, beta, add=add, out_dtype=yt))


@pytest.mark.parametrize("M", [0, 1, 2, 3, 4, 5, 1000, 4099])
@pytest.mark.parametrize("K", [64, 333, 5000])
def test_row_counts(tw, M, K):
    x = rows(M, K, BF, M + K)
    gamma, beta = params(K, 1)
    out = tw.layernorm(x, gamma, beta)
    assert out["y"].shape == (M, K)
    if M:
        check_forward(x, None, gamma, beta, out)


@pytest.mark.parametrize("pad", [1, 3, 8])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [96, 1001, 4100])
def test_strided_rows(tw, pad, dtype, K):
    """Rows of a wider buffer: the same bits as a contiguous copy's."""
    x = rows(9, K, dtype, K, pad=pad)
    gamma, beta = params(K, 2)
    a, b = tw.layernorm(x, gamma, beta), tw.layernorm(x.contiguous(), gamma, beta)
    for k in ("y", "mean", "rstd"):
        assert torch.equal(a[k], b[k]), k
    qa, qb = tw.layernorm_quantize(x, gamma, beta), tw.layernorm_quantize(x.contiguous(), gamma, beta)
    assert torch.equal(qa["q"], qb["q"]) and torch.equal(qa["scale"], qb["scale"])
    dy = rows(9, K, F32, 5)
    ga = tw.layernorm_backward(dy, x, gamma, a["mean"], a["rstd"])
    gb = tw.layernorm_backward(dy, x.contiguous(), gamma, a["mean"], a["rstd"])
    for k in ga:
        assert torch.equal(ga[k], gb[k]), k


def test_last_token_of_each_sequence(tw):
    """A strided view with a row distance past 32 bits."""
    stride = (1 << 31) + 64
    buf = torch.empty(2 * stride, dtype=BF, device="cuda")
    x = buf.as_strided((2, 256), (stride, 1))
    x.copy_(rows(2, 256, BF, 3))
    gamma, beta = params(256, 4)
    check_forward(x, None, gamma, beta, tw.layernorm(x, gamma, beta))
    q, scale = tw.quantize_rows(x)
    qr, sr = R.quantise(x.float().cpu().numpy())
    assert (q.cpu().numpy() == qr).all() and (scale.cpu().numpy() == sr).all()


def test_more_than_2_31_elements(tw):
    M, K = (1 << 31) // 1024 + 5, 1024
    x = torch.zeros(M, K, dtype=BF, device="cuda")
    x[-3:] = rows(3, K, BF, 8)
    gamma, beta = params(K, 9)
    out = tw.layernorm(x, gamma, beta)
    tail = {k: v[-3:].clone() for k, v in out.items() if v is not None}
    check_forward(x[-3:], None, gamma, beta, tail)
    assert torch.equal(out["y"][0].float(), beta.to(BF).float())
    dy = torch.zeros(M, K, dtype=BF, device="cuda")
    dy[-3:] = rows(3, K, BF, 10)
    g = tw.layernorm_backward(dy, x, gamma, out["mean"], out["rstd"], dx_dtype=BF)
    small = tw.layernorm_backward(dy[-3:], x[-3:], gamma, tail["mean"], tail["rstd"], dx_dtype=BF)
    assert torch.equal(g["dx"][-3:], small["dx"])
    assert not g["dx"][:-3].any()


def test_far_from_zero(tw):
    """Rows whose mean is 1000 times their spread: the variance is taken over
    centred values."""
    x = rows(11, 777, F32, 1, offset=2000.0)
    gamma, beta = params(777, 2)
    check_forward(x, None, gamma, beta, tw.layernorm(x, gamma, beta, out_dtype=F32))


def test_extreme_rows(tw):
    K = 600
    x = rows(8, K, F32, 1)
    x[1] = 3.5                      # constant: variance 0
    x[2] = 0.0
    x[3, 17] = float("nan")
    x[4, 5] = float("inf")
    x[5] *= 1e-30                   # variance far below eps
    x[6] *= 1e15
    gamma, beta = params(K, 3)
    out = tw.layernorm(x, gamma, beta, out_dtype=F32)
    y = out["y"]
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).all()
    assert torch.equal(y[2], beta)
    assert (y[1] - beta).abs().max() <= 3.5 * 96 * 2.0 ** -24 * 1.1 / 1e-5 ** 0.5 * gamma.abs().max()
    keep = [0, 2, 5, 6, 7]
    check_forward(x[keep], None, gamma, beta, {k: v[keep] for k, v in out.items() if v is not None})
    assert torch.isnan(tw.layernorm(x, gamma, beta)["y"][3:5]).all()  # bf16 keeps NaN
    q = tw.layernorm_quantize(x, gamma, beta)
    assert torch.isnan(q["scale"][3:5]).all() and not q["q"][3:5].any()
    assert torch.isfinite(q["scale"][keep]).all()


def test_sum_in_place(tw):
    x, add = rows(33, 1000, F32, 1), rows(33, 1000, F32, 2)
    gamma, beta = params(1000, 3)
    ref = tw.layernorm(x, gamma, beta, add=add)
    for target in ("x", "add"):
        xc, ac = x.clone(), add.clone()
        y = torch.empty(33, 1000, dtype=BF, device="cuda")
        tw.tw_layernorm_fwd(xc, gamma, beta, 1e-5, y, add=ac, total=xc if target == "x" else ac)
        assert torch.equal(y, ref["y"])
        assert torch.equal(xc if target == "x" else ac, ref["sum"])


# ---------------------------------------------------------------- backward --
def check_backward(dy, x, gamma, mean, rstd, dres, out):
    M = x.shape[0]
    dx, dg, db, mag, mag_g, mag_b = R.norm_bwd(f64(dy), f64(x), f64(gamma), f64(mean), f64(rstd),
                                               None if dres is None else f64(dres))
    e = R.SUM * R.U * mag + R.out_unit(out["dx"].dtype == BF) * np.abs(dx)
    assert (np.abs(f64(out["dx"]) - dx) <= e).all()
    # a column is summed over the rows a wave walks, then over waves and
    # workgroups: at most M / 256 + 4 + 64 additions in sequence
    depth = M / 256 + R.SUM
    assert (np.abs(f64(out["dgamma"]) - dg) <= depth * R.U * mag_g).all()
    assert (np.abs(f64(out["dbeta"]) - db) <= depth * R.U * mag_b).all()


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("dt,xt,ot,res", [(BF, BF, BF, False), (F32, BF, F32, False),
                                          (F32, F32, F32, True), (BF, F32, BF, True)])
def test_backward(tw, K, dt, xt, ot, res):
    M = 9 if K > 4096 else 37
    x, dy = rows(M, K, xt, K, offset=0.3), rows(M, K, dt, K + 1)
    dres = rows(M, K, ot, K + 2) if res else None
    gamma, beta = params(K, K + 3)
    f = tw.layernorm(x, gamma, beta)
    print(f"case M={M} K={K} {dt} {xt} {ot}", flush=True)
    out = tw.layernorm_backward(dy, x, gamma, f["mean"], f["rstd"], dres=dres, dx_dtype=ot)
    check_backward(dy, x, gamma, f["mean"], f["rstd"], dres, out)


@pytest.mark.parametrize("M", [0, 1, 3, 4, 5, 255, 2049, 10007])
@pytest.mark.parametrize("K", [40, 1001, 2500])
def test_backward_row_counts(tw, M, K):
    x, dy = rows(M, K, BF, M + 1), rows(M, K, F32, M + 2)
    gamma, beta = params(K, 1)
    f = tw.layernorm(x, gamma, beta)
    out = tw.layernorm_backward(dy, x, gamma, f["mean"], f["rstd"])
    if M == 0:
        assert not out["dgamma"].any() and not out["dbeta"].any()
    else:
        check_backward(dy, x, gamma, f["mean"], f["rstd"], None, out)


def test_backward_optional_outputs(tw):
    M, K = 50, 700
    x, dy = rows(M, K, BF, 1), rows(M, K, BF, 2)
    gamma, beta = params(K, 3)
    f = tw.layernorm(x, gamma, beta)
    full = tw.layernorm_backward(dy, x, gamma, f["mean"], f["rstd"], dx_dtype=BF)
    ws = torch.empty(tw.tw_layernorm_bwd_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    for want in ((), ("dgamma",), ("dbeta",)):
        bufs = {k: torch.full((K,), 7.0, device="cuda") for k in want}
        dx = torch.empty(M, K, dtype=BF, device="cuda")
        tw.tw_layernorm_bwd(dy, x, gamma, f["mean"], f["rstd"], dx, ws=ws if want else None, **bufs)
        assert torch.equal(dx, full["dx"])
        for k, v in bufs.items():
            assert torch.equal(v, full[k])


@pytest.mark.parametrize("K", [5, 300, 2100])
def test_gradient_by_differences(tw, K):
    """dx, dgamma and dbeta against central differences of the forward's
    formula in float64 along random directions."""
    M, eps, h = 6, 1e-5, 1e-6
    x, dy = rows(M, K, F32, K), rows(M, K, F32, K + 1)
    dres = rows(M, K, F32, K + 2)
    gamma, beta = params(K, K + 3)
    f = tw.layernorm(x, gamma, beta, eps=eps, out_dtype=F32)
    out = tw.layernorm_backward(dy, x, gamma, f["mean"], f["rstd"], dres=dres)
    X, DY, G, B, DR = f64(x), f64(dy), f64(gamma), f64(beta), f64(dres)

    def loss(X, G, B):  # dres: the gradient of a second path that reads x itself
        return (R.norm(X, G, B, eps, False)[0] * DY).sum() + (X * DR).sum()

    rng = np.random.default_rng(K)
    for name, base in (("dx", X), ("dgamma", G), ("dbeta", B)):
        for _ in range(3):
            d = rng.standard_normal(base.shape)
            at = {"dx": X, "dgamma": G, "dbeta": B}
            hi, lo = dict(at), dict(at)
            hi[name], lo[name] = base + h * d, base - h * d
            num = (loss(*hi.values()) - loss(*lo.values())) / (2 * h)
            g = f64(out[name])
            # fp32 gradient (SUM u of its magnitudes, here against the norms),
            # truncation h^2 and the difference's own rounding 2^-52 loss / h
            tol = (R.SUM * R.U * 8 * np.abs(g * d).sum() + 1e-4 * np.linalg.norm(g) * np.linalg.norm(d) / K
                   + 2.0 ** -50 * (np.abs(DY).sum() * 8 + np.abs(X * DR).sum()) / h)
            assert abs(num - (g * d).sum()) <= tol, (name, num, (g * d).sum(), tol)


# ------------------------------------------------------- int8 rows, streams --
@pytest.mark.parametrize("K", [1, 7, 16, 100, 512, 513, 2048, 4100, 16384, 16400, 20001, 65536])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_rows_to_the_bit(tw, K, dtype):
    x = rows(6, K, dtype, K)
    x[1] = 0
    x[2] *= 1e-36
    x[3, K // 2] = float("inf") if K % 2 else float("nan")
    x[4] *= 1e-20
    q, scale = tw.quantize_rows(x)
    qr, sr = R.quantise(x.float().cpu().numpy())
    assert np.array_equal(scale.cpu().numpy(), sr, equal_nan=True)
    assert np.array_equal(q.cpu().numpy(), qr)


def test_quantize_ties_and_range(tw):
    """Values half way between codes go to the even one, and the ends are
    +-127 exactly."""
    x = torch.arange(-254, 255, dtype=torch.float32)[None] / 2  # top 127: codes are the halves
    q, scale = tw.quantize_rows(x.cuda())
    assert scale.item() == 1.0
    assert np.array_equal(q.cpu().numpy()[0], np.rint(x.numpy()[0]).astype(np.int8))
    big = torch.full((1, 64), 3.3e38)
    big[0, ::2] *= -1
    q, scale = tw.quantize_rows(big.cuda())
    assert (q.abs() == 127).all() and torch.isfinite(scale).all()


@pytest.mark.parametrize("K", [8, 500, 1024, 3000, 9000])
@pytest.mark.parametrize("at", [None, BF, F32])
def test_layernorm_quantize(tw, K, at):
    x = rows(21, K, F32 if K % 16 else BF, K)
    add = None if at is None else rows(21, K, at, 1)
    gamma, beta = params(K, 2)
    out = tw.layernorm_quantize(x, gamma, beta, add=add)
    z = f64(x) + f64(add) if add is not None else f64(x)
    y, _, rstd, e_y, _, _ = R.norm(z, f64(gamma), f64(beta), 1e-5, False)
    e_y = e_y + R.U * np.abs(z) * np.abs(f64(gamma)) * rstd[:, None]
    scale = f64(out["scale"])
    top, e_top = np.abs(y).max(1), e_y.max(1)
    assert (np.abs(scale * 127 - top) <= e_top + 2 * R.U * top).all()
    q = f64(out["q"])
    assert (np.abs(q).max(1) == 127).all()
    # half a step, the norm's error, and the fp32 roundings of the factor
    assert (np.abs(q * scale[:, None] - y) <= scale[:, None] * (0.5 + 127 * 4 * R.U) + e_y + e_top[:, None]).all()
    if add is not None:
        assert torch.equal(out["sum"], (x.float() + add.float()).to(x.dtype))


def test_side_stream_and_repeatability(tw):
    M, K = 3001, 1111
    x, dy = rows(M, K, BF, 1), rows(M, K, F32, 2)
    gamma, beta = params(K, 3)

    def both():
        f = tw.layernorm(x, gamma, beta)
        g = tw.layernorm_backward(dy, x, gamma, f["mean"], f["rstd"])
        return [f["y"], f["mean"], f["rstd"], g["dx"], g["dgamma"], g["dbeta"]]

    ref = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = both()
    s.synchronize()
    again = both()
    for a, b, c in zip(ref, side, again):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_graph_replays(tw):
    M, K = 513, 1024
    x, dy = rows(M, K, BF, 1), rows(M, K, F32, 2)
    gamma, beta = params(K, 3)
    y = torch.empty(M, K, dtype=BF, device="cuda")
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    dx = torch.empty(M, K, device="cuda")
    dg, db = torch.empty(K, device="cuda"), torch.empty(K, device="cuda")
    ws = torch.empty(tw.tw_layernorm_bwd_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")

    def step():
        tw.tw_layernorm_fwd(x, gamma, beta, 1e-5, y, mean=mean, rstd=rstd)
        tw.tw_layernorm_bwd(dy, x, gamma, mean, rstd, dx, dg, db, ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (11, 12, 13):
        x.copy_(rows(M, K, BF, seed))
        dy.copy_(rows(M, K, F32, seed + 100))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, mean, rstd, dx, dg, db)]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (y, mean, rstd, dx, dg, db)):
            assert torch.equal(a, b)


def test_events(tw):
    M, K = 64, 512
    x, dy = rows(M, K, BF, 1), rows(M, K, BF, 2)
    gamma, beta = params(K, 3)
    f = tw.layernorm(x, gamma, beta)
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    for e in ev:
        e.record()
    ids = [e.cuda_event for e in ev]
    y = torch.empty(M, K, dtype=BF, device="cuda")
    tw.tw_layernorm_fwd(x, gamma, beta, 1e-5, y, events=ids[:2])
    ws = torch.empty(tw.tw_layernorm_bwd_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    dg, db = torch.empty(K, device="cuda"), torch.empty(K, device="cuda")
    tw.tw_layernorm_bwd(dy, x, gamma, f["mean"], f["rstd"], torch.empty_like(dy), dg, db, ws=ws,
                        events=ids)
    torch.cuda.synchronize()
    assert ev[0].elapsed_time(ev[1]) >= 0 and ev[1].elapsed_time(ev[2]) >= 0
