"""int8 products on the GPU: the integer sums are exact, so outputs are held
to the few fp32 roundings after them (norm_ref.product); ragged sizes,
strided inputs, extreme rows, streams, graphs."""
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


def codes(M, K, seed, full=False):
    """int8 codes over the whole range, ends included; ``full``: all +-127,
    which gives the largest sums."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-127, 128, (M, K), generator=g, dtype=I8)
    if full:
        q = torch.where(q >= 0, torch.tensor(127, dtype=I8), torch.tensor(-127, dtype=I8))
    return q.cuda()


def scales(n, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.rand(n, generator=g) * 0.05 + 1e-3).cuda()


def num(t):
    return t.cpu().numpy() if t.dtype != BF else t.float().cpu().numpy()


def check(y, ref, e):
    ref_y = num(y).astype(np.float64)
    bound = e + R.out_unit(y.dtype == BF) * np.abs(ref)
    assert ref_y.shape == ref.shape
    assert (np.abs(ref_y - ref) <= bound).all(), np.abs(ref_y - ref).max()


def gate_ref(q, xs, wg, gs, wu, us):
    g, eg = R.product(q, xs, wg, gs)
    u, eu = R.product(q, xs, wu, us)
    g = np.maximum(g, 0)
    return g * u, eg * np.abs(u) + eu * g + 2 * R.U * np.abs(g * u)


# every kernel's row counts: few rows (to 16, to 32), tiles of 64, 128, 256
SHAPES = [(1, 16, 1), (1, 2048, 5), (2, 48, 16), (7, 80, 127), (16, 256, 250), (17, 1008, 33),
          (32, 64, 1001), (33, 2048, 128), (64, 96, 63), (65, 4096, 65), (77, 1008, 1001),
          (128, 128, 4096), (129, 160, 2500), (300, 272, 700), (1025, 80, 1300), (2000, 1040, 2100),
          (4100, 144, 3300), (5000, 64, 4097), (2900, 400, 4700), (4200, 656, 5000),
          (16001, 384, 300)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("yt,bias", [(BF, True), (F32, False), (F32, True)])
def test_linear_int8(tw, M, K, N, yt, bias):
    q, w = codes(M, K, 1), codes(N, K, 2)
    xs, ws = scales(M, 3), scales(N, 4)
    b = torch.randn(N, generator=torch.Generator().manual_seed(5)).cuda() if bias else None
    print(f"case {M} {K} {N} {yt} bias={bias}", flush=True)
    y = tw.quant_linear(q, w, ws, bias=b, x_scale=xs, out_dtype=yt)
    check(y, *R.product(num(q), num(xs), num(w), num(ws), num(b) if bias else None))


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("yt", [BF, F32])
def test_gateup_int8(tw, M, K, N, yt):
    q, wg, wu = codes(M, K, 1), codes(N, K, 2), codes(N, K, 3)
    xs, gs, us = scales(M, 4), scales(N, 5), scales(N, 6)
    print(f"case {M} {K} {N} {yt}", flush=True)
    h = tw.quant_gateup(q, wg, gs, wu, us, x_scale=xs, out_dtype=yt)
    check(h, *gate_ref(num(q), num(xs), num(wg), num(gs), num(wu), num(us)))


@pytest.mark.parametrize("M", [3, 40, 700])
def test_largest_sums(tw, M):
    """All codes +-127 at the longest reduction: |sum| up to 127^2 65536."""
    K, N = 65536, 48
    q, w = codes(M, K, 1, full=True), codes(N, K, 2, full=True)
    w[0] = q[0]
    w[1] = -q[0]
    xs, ws = scales(M, 3), scales(N, 4)
    y = tw.quant_linear(q, w, ws, x_scale=xs, out_dtype=F32)
    check(y, *R.product(num(q), num(xs), num(w), num(ws)))


def test_every_k_tail(tw):
    """Each remainder of K over a stage, in every kernel."""
    for K in range(16, 200, 16):
        for M, N in ((5, 40), (20, 40), (70, 90), (130, 6400), (2100, 4600)):
            q, w = codes(M, K, K), codes(N, K, K + 1)
            xs, ws = scales(M, 3), scales(N, 4)
            y = tw.quant_linear(q, w, ws, x_scale=xs, out_dtype=F32)
            check(y, *R.product(num(q), num(xs), num(w), num(ws)))


def rows(M, K, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(M, K + pad, generator=g) * (0.2 + torch.rand(K + pad, generator=g))).to(dtype).cuda()[:, :K]


@pytest.mark.parametrize("M,K,N", [(0, 64, 64), (1, 512, 300), (1, 16, 16), (3, 5632, 70), (4, 2048, 333), (9, 1024, 64), (16, 8192, 40),
                                   (31, 96, 100), (90, 2048, 600), (1500, 256, 1500)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_linear_quantises_its_input(tw, M, K, N, dtype, pad):
    """A float input gives what its rows' exact codes give."""
    x, w, ws = rows(M, K, dtype, 1, pad), codes(N, K, 2), scales(N, 3)
    y = tw.quant_linear(x, w, ws, out_dtype=F32)
    q, xs = R.quantise(x.float().cpu().numpy())
    check(y, *R.product(q, xs, num(w), num(ws)))


@pytest.mark.parametrize("M,K,N", [(0, 64, 64), (1, 512, 300), (2, 16, 16), (4, 2048, 333), (5, 5632, 48), (16, 1024, 64), (33, 1024, 600),
                                   (1500, 256, 1500)])
@pytest.mark.parametrize("dtype,pad", [(BF, 0), (F32, 0), (BF, 3)])
@pytest.mark.parametrize("norm", ["no", "gamma", "gamma, beta"])
def test_gateup_norms_its_input(tw, M, K, N, dtype, pad, norm):
    """A float input gives the gate and up products of its quantised norm
    (or of its quantised rows): the same bits as the two calls, or within
    what one code of difference in the norm can do."""
    x = rows(M, K, dtype, 1, pad)
    wg, wu, gs, us = codes(N, K, 2), codes(N, K, 3), scales(N, 4), scales(N, 5)
    gamma = beta = None
    if norm != "no":
        gamma = (1 + 0.1 * torch.randn(K, generator=torch.Generator().manual_seed(6))).cuda()
    if norm == "gamma, beta":
        beta = (0.1 * torch.randn(K, generator=torch.Generator().manual_seed(7))).cuda()
    h = tw.quant_gateup(x, wg, gs, wu, us, gamma=gamma, beta=beta, out_dtype=F32)
    if norm == "no":
        q, xs = tw.quantize_rows(x)
    else:
        n = tw.layernorm_quantize(x, gamma, beta)
        q, xs = n["q"], n["scale"]
    ref, e = gate_ref(num(q), num(xs), num(wg), num(gs), num(wu), num(us))
    if norm != "no":
        # the norm's own error (SUM u) may move a code that lies that near a
        # boundary, and moves the scale by as much: allow four codes' worth
        step = 4 * 127 * num(xs).astype(np.float64)[:, None]
        g = np.maximum(R.product(num(q), num(xs), num(wg), num(gs))[0], 0)
        u = R.product(num(q), num(xs), num(wu), num(us))[0]
        sg, su = step * num(gs), step * num(us)
        e = e + sg * (np.abs(u) + su) + su * g + 4 * R.SUM * R.U * np.abs(ref)
    check(h, ref, e)


def test_extreme_rows(tw):
    """Rows of NaN or infinity give NaN, rows of zeros give the bias, and
    neither touches another row."""
    for M in (6, 40, 300):
        K, N = 256, 200
        x = rows(M, K, BF, 1)
        w, ws = codes(N, K, 2), scales(N, 3)
        b = torch.randn(N, generator=torch.Generator().manual_seed(5)).cuda()
        ref = tw.quant_linear(x, w, ws, bias=b)
        bad = x.clone()
        bad[1, 7], bad[2, 9], bad[3] = float("nan"), float("-inf"), 0.0
        y = tw.quant_linear(bad, w, ws, bias=b)
        assert torch.isnan(y[1:3]).all()
        assert torch.equal(y[3], b.to(BF))
        assert torch.equal(y[0], ref[0]) and torch.equal(y[4:], ref[4:])
        h = tw.quant_gateup(bad, w, ws, w.flip(0).contiguous(), ws)
        assert torch.isnan(h[1:3]).all() and not h[3].any() and torch.isfinite(h[4:].float()).all()


def test_input_past_4_gib(tw):
    """Row offsets past 32 bits in the tiles and in the quantiser."""
    M, K, N = 70001, 65536, 40
    x = torch.zeros(M, K, dtype=I8, device="cuda")
    x[-200:] = codes(200, K, 1)
    xs, w, ws = scales(M, 2), codes(N, K, 3), scales(N, 4)
    y = tw.quant_linear(x, w, ws, x_scale=xs, out_dtype=F32)
    check(y[-200:], *R.product(num(x[-200:]), num(xs[-200:]), num(w), num(ws)))
    assert not y[:-200].any()


@pytest.mark.parametrize("M", [1, 40, 700])
def test_repeatable_on_any_stream(tw, M):
    K, N = 1024, 900
    x, w, ws = rows(M, K, BF, 1), codes(N, K, 2), scales(N, 3)
    gamma = torch.ones(K, device="cuda")

    def both():
        return tw.quant_linear(x, w, ws), tw.quant_gateup(x, w, ws, w, ws, gamma=gamma)

    ref = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        side = both()
    s.synchronize()
    for a, b, c in zip(ref, side, both()):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("M", [1, 40, 700])
def test_graph_replays(tw, M):
    K, N = 512, 640
    x, w, ws = rows(M, K, BF, 1), codes(N, K, 2), scales(N, 3)
    wd, ds = codes(K, N, 4), scales(K, 5)
    gamma = torch.ones(K, device="cuda")
    h, y = torch.empty(M, N, dtype=BF, device="cuda"), torch.empty(M, K, device="cuda")
    wk = torch.empty(tw.tw_quant_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    wn = torch.empty(tw.tw_quant_workspace_bytes(M, N), dtype=torch.uint8, device="cuda")

    def step():
        tw.tw_quant_gateup(x, w, ws, w, ws, h, gamma=gamma, ws=wk)
        tw.tw_quant_linear(h, wd, ds, y, ws=wn)

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
        graph.replay()
        torch.cuda.synchronize()
        got = h.clone(), y.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], h) and torch.equal(got[1], y)


def test_quantised_ffn_near_the_float_one(tw):
    """The int8 gate/up and down projections against the same FFN in float64
    on the unquantised operands: both roundings of 8 bits are independent
    errors of at most half a step, a few per cent of y altogether."""
    M, K, N = 200, 512, 1024
    g = torch.Generator().manual_seed(1)
    x = torch.randn(M, K, generator=g)
    W = [torch.randn(N, K, generator=g) / K ** 0.5 for _ in range(2)] + [torch.randn(K, N, generator=g) / N ** 0.5]
    (wg, gs), (wu, us), (wd, ds) = (tw.quantize_rows(w.cuda()) for w in W)
    h = tw.quant_gateup(x.cuda(), wg, gs, wu, us)
    y = tw.quant_linear(h, wd, ds, out_dtype=F32)
    X, G, Up, D = (t.double() for t in (x, *W))
    ref = (torch.relu(X @ G.T) * (X @ Up.T)) @ D.T
    assert ((y.cpu().double() - ref).norm() / ref.norm()).item() < 0.05
