"""The dense training step's operators at the largest sizes and row distances that the
header names, against float64 (train_ref.py)."""
import pytest

import train_ref as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def tw():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from activation_sparse_feed_gate_amd import tw as mod

    yield mod
    torch.cuda.empty_cache()


def d64(t):
    return t.detach().to(torch.float64)


def rnd(seed, *shape, std=1.0, dtype=BF):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def far(x, stride):
    """The rows of x, `stride` elements apart among NaN."""
    wide = torch.full((x.shape[0], stride), float("nan"), dtype=x.dtype, device="cuda")
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def same(a, b):
    assert a.keys() == b.keys()
    for k in a:
        assert (a[k] is None and b[k] is None) or torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("M", [3, 20, 60, 300])
def test_rows_as_far_apart_as_they_may_be(tw, M):
    K, N, V = 264, 520, 1001
    print(f"case {M}x{K}, rows 2^20 apart", flush=True)
    x = rnd(M, M, K)
    y = far(x, 1 << 20)
    w = [rnd(i, N, K, std=0.05) for i in (1, 2, 3)]
    a = tw.gated_ffn(x, *w, keep=True)
    same(a, tw.gated_ffn(y, *w, keep=True))
    dy = rnd(4, M, K)
    same(tw.gated_ffn_backward(dy, x, *w, a["g"], a["u"]), tw.gated_ffn_backward(dy, y, *w, a["g"], a["u"]))
    wo, t = rnd(5, V, K, std=0.1), torch.arange(M, device="cuda")
    c = tw.linear_ce(x, wo, t)
    same(c, tw.linear_ce(y, wo, t))
    dloss = rnd(6, M, dtype=F32)
    same(tw.linear_ce_backward(dloss, x, wo, t, c["lse"]), tw.linear_ce_backward(dloss, y, wo, t, c["lse"]))


@pytest.mark.parametrize("M", [2, 70, 300])
@pytest.mark.parametrize("K,N", [(1 << 20, 24), (24, 1 << 20)])
def test_longest_rows_of_the_ffn(tw, M, K, N):
    print(f"case {M}x{K}x{N}", flush=True)
    x, dy = rnd(M, M, K), rnd(M + 1, M, K)
    w = [rnd(i, N, K, std=K ** -0.5) for i in (1, 2)] + [rnd(3, N, K, std=N ** -0.5)]
    out = tw.gated_ffn(x, *w, keep=True)
    wide = [d64(t) for t in w]
    y, ey, g, eg, u, eu = R.ffn(d64(x), *wide, "silu")
    for k, v, e in (("y", y, ey), ("g", g, eg), ("u", u, eu)):
        R.close(out[k], v, e)
    got = tw.gated_ffn_backward(dy, x, *w, out["g"], out["u"])
    for k, (v, e) in R.ffn_bwd(d64(dy), d64(x), *wide, d64(out["g"]), d64(out["u"]), "silu").items():
        R.close(got[k], v, e)


@pytest.mark.parametrize("M", [2, 20, 70, 300])
def test_longest_rows_of_the_loss(tw, M):
    K, V = 1 << 20, 129
    print(f"case {M}x{K}x{V}", flush=True)
    x, w = rnd(M, M, K), rnd(1, V, K, std=2 * K ** -0.5)
    t = torch.arange(M, device="cuda") % V
    t[1] = -100
    out = tw.linear_ce(x, w, t)
    loss, el, lse, es = R.ce(d64(x), d64(w), t)
    R.close(out["lse"], lse, es)
    R.close(out["loss"], loss, el)
    dloss = rnd(7, M, dtype=F32)
    got = tw.linear_ce_backward(dloss, x, w, t, out["lse"])
    for k, (v, e) in R.ce_bwd(d64(dloss), d64(x), d64(w), t, d64(out["lse"])).items():
        R.close(got[k], v, e)


def test_most_rows(tw):
    M, K, N, V = 1 << 24, 8, 8, 3
    print(f"case {M} rows", flush=True)
    x, dy = rnd(1, M, K), rnd(2, M, K)
    w = [rnd(i, N, K, std=K ** -0.5) for i in (3, 4, 5)]
    wide = [d64(t) for t in w]
    out = tw.gated_ffn(x, *w, keep=True)
    y, ey, g, eg, u, eu = R.ffn(d64(x), *wide, "silu")
    for k, v, e in (("y", y, ey), ("g", g, eg), ("u", u, eu)):
        R.close(out[k], v, e)
    del y, ey, g, eg, u, eu
    got = tw.gated_ffn_backward(dy, x, *w, out["g"], out["u"], dw_dtype=F32)
    for k, (v, e) in R.ffn_bwd(d64(dy), d64(x), *wide, d64(out["g"]), d64(out["u"]), "silu").items():
        R.close(got[k], v, e)
        if k != "dx":  # (2^24 additions leave no bound; each rounding apart, they average out)
            assert float((d64(got[k]) - v).norm() / v.norm()) < 0.01, k
    del out, got
    w = rnd(6, V, K)
    t = torch.arange(M, device="cuda") % (V + 1)  # every fourth row is left out
    out = tw.linear_ce(x, w, t)
    loss, el, lse, es = R.ce(d64(x), d64(w), t)
    R.close(out["lse"], lse, es)
    R.close(out["loss"], loss, el)
    dloss = rnd(7, M, dtype=F32)
    got = tw.linear_ce_backward(dloss, x, w, t, out["lse"], dw_dtype=F32)
    for k, (v, e) in R.ce_bwd(d64(dloss), d64(x), d64(w), t, d64(out["lse"])).items():
        R.close(got[k], v, e)
