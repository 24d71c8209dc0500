"""Clipping at the ends of its arguments: a norm or a largest norm of 0, an infinite largest
norm."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module")
def tw():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from activation_sparse_feed_gate_amd import tw as mod

    return mod


# one buffer; more parts than a workgroup of the clipping adds itself
SIZES = [[100], [8193, 7], [8192 * 1100]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("most", [0.0, 1.0])
@pytest.mark.parametrize("apart", [False, True])
def test_zeros_without_eps_stay_zeros(tw, sizes, dtype, most, apart):
    g = [torch.zeros(n, dtype=dtype, device="cuda") for n in sizes]
    out = [torch.full_like(t, 7.0) for t in g] if apart else None
    norm = tw.clip_grads(g, most, eps=0.0, out=out)
    assert norm == 0 and all((t == 0).all() for t in (out or g))


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_a_largest_norm_of_zero_makes_zeros(tw, sizes, eps):
    g = [torch.ones(n, device="cuda") for n in sizes]
    norm = tw.clip_grads(g, 0.0, eps=eps)
    assert norm > 0 and all((t == 0).all() for t in g)
    # squares below the fp32 range: the norm is 0, the gradients are not
    g = [torch.full((n,), 1e-30, device="cuda") for n in sizes]
    assert tw.clip_grads(g, 0.0, eps=eps) == 0 and all((t == 0).all() for t in g)
    g[0][3] = float("nan")
    assert tw.clip_grads(g, 0.0, eps=eps).isnan() and all(t.isnan().all() for t in g)


@pytest.mark.parametrize("sizes", SIZES)
def test_an_infinite_largest_norm_leaves_them(tw, sizes):
    g = [torch.randn(n, device="cuda") for n in sizes]
    was = [t.clone() for t in g]
    assert tw.clip_grads(g, INF).isfinite()
    assert all(torch.equal(a, b) for a, b in zip(was, g))
