"""The dense training step's operators where a formula's limit is a number and its terms
are not: gates of plus and minus infinity.  Bounds are train_ref.py's."""
import pytest

import train_ref as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")
ACTS = ["silu", "gelu", "relu"]
ROWS = [6, 100]  # the kernels of few rows, the tiles


@pytest.fixture(scope="module")
def tw():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from activation_sparse_feed_gate_amd import tw as mod

    return mod


def d64(t):
    return t.detach().to(torch.float64)


def rnd(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(BF).cuda()


def weights(K, N):
    return rnd(1, N, K, std=K ** -0.5), rnd(2, N, K, std=K ** -0.5), rnd(3, N, K, std=N ** -0.5)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", ROWS)
def test_gradient_at_gates_of_minus_infinity(tw, act, M):
    """The activation and its slope are 0 there: the neuron adds nothing to any gradient."""
    K, N = 64, 72
    w, x, dy, u = weights(K, N), rnd(4, M, K), rnd(5, M, K), rnd(6, M, N)
    g = rnd(7, M, N, std=1.5)
    g[:, ::5] = -INF  # whole neurons
    g[1::3, 2] = -INF
    got = tw.gated_ffn_backward(dy, x, *w, g, u, act=act, dx_dtype=F32, dw_dtype=F32)
    # (at -10^4 the float64 activation, its slope and their errors are 0)
    ref = R.ffn_bwd(d64(dy), d64(x), *(d64(t) for t in w), d64(g).clamp(min=-1e4), d64(u), act)
    for k, (v, e) in ref.items():
        R.close(got[k], v, e)
    for k in ("dwg_t", "dwu_t", "dwd"):
        assert (got[k][::5] == 0).all(), k


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", ROWS)
def test_gate_gradient_at_gates_of_infinity(tw, act, M):
    """The slope is 1 there: dz = dh u, whatever becomes of du."""
    K, N = 64, 72
    w, x, dy, u = weights(K, N), rnd(4, M, K), rnd(5, M, K), rnd(6, M, N)
    g = torch.full((M, N), INF, dtype=BF, device="cuda")
    got = tw.gated_ffn_backward(dy, x, *w, g, u, act=act, dw_dtype=F32)["dwg_t"]
    dh = R.mm(d64(dy), d64(w[2]).T)
    dz = dh * d64(u)
    e = (K + 8) * R.U * R.mm(d64(dy).abs(), d64(w[2]).T.abs()) * d64(u).abs() + 4 * R.U * dz.abs()
    e = e + R.UB * (dz.abs() + e)
    R.close(got, R.mm(dz.T, d64(x)),
            R.mm(e.T, d64(x).abs()) + (M + 8) * R.U * R.mm((dz.abs() + e).T, d64(x).abs()))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", ROWS)
def test_every_gradient_at_saturated_gates(tw, act, M):
    """Finite gates far past the logistic function's range: all four gradients."""
    K, N = 64, 72
    w, x, dy, u = weights(K, N), rnd(4, M, K), rnd(5, M, K), rnd(6, M, N)
    g = torch.tensor([-3e38, -1e20, -200.0, -129.0, -127.0, -90.0, -17.0, -16.0, 16.0, 17.0, 90.0,
                      127.0, 129.0, 200.0, 1e4, 1e20, 0.0, -0.0], dtype=BF).cuda()
    g = g.repeat(M, N // 18).contiguous()
    got = tw.gated_ffn_backward(dy, x, *w, g, u, act=act, dx_dtype=F32, dw_dtype=F32)
    ref = R.ffn_bwd(d64(dy), d64(x), *(d64(t) for t in w), d64(g), d64(u), act)
    for k, (v, e) in ref.items():
        R.close(got[k], v, e)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", ROWS)
def test_forward_at_gates_of_minus_infinity(tw, act, M):
    """Gate sums past the fp32 range: those neurons add nothing, y is the others'."""
    K, N = 64, 72
    w, x = weights(K, N), rnd(4, M, K)
    x[:, 0] = 2.0 ** 127
    for t in w[:2]:
        t[:, 0] = 0
    off = torch.zeros(N, dtype=torch.bool, device="cuda")
    off[::5] = True
    w[0][off, 0] = -4.0
    out = tw.gated_ffn(x, *w, act=act, keep=True)
    assert (out["g"][:, off] == -INF).all() and out["g"][:, ~off].isfinite().all()
    y, ey = R.ffn(d64(x), *(d64(t[~off]) for t in w), act)[:2]
    R.close(out["y"], y, ey)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", ROWS)
def test_gates_of_nan_stay_nan(tw, act, M):
    K, N = 64, 72
    w, x, dy, u = weights(K, N), rnd(4, M, K), rnd(5, M, K), rnd(6, M, N)
    g = rnd(7, M, N)
    g[:, 3] = float("nan")
    got = tw.gated_ffn_backward(dy, x, *w, g, u, act=act)
    assert got["dwu_t"][3].isnan().all() and got["dwd"][3].isnan().all() and got["dx"].isnan().all()
    assert got["dwu_t"][4].isfinite().all()
