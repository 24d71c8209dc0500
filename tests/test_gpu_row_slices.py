"""Per-row inputs (targets, log-sum-exps, loss gradients, norms' factors) that begin at any
row of a longer tensor, as tokens[1:] does: the bits of an aligned copy's call."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF, F32 = torch.bfloat16, torch.float32
M, K, V = 37, 264, 1001


@pytest.fixture(scope="module")
def tw():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from activation_sparse_feed_gate_amd import tw as mod

    return mod


class Never:
    """The binding without its native part."""

    def __getattr__(self, k):
        return lambda *a: None


@pytest.fixture(params=["native", "checked"])
def way(request, tw, monkeypatch):
    if request.param == "native":
        native = tw._calls

        class Must:
            def __getattr__(self, k):
                def run(*a):
                    got = getattr(native, k)(*a)
                    assert got is not None, k
                    return got
                return run

        monkeypatch.setattr(tw, "_calls", Must())
    else:
        monkeypatch.setattr(tw, "_calls", Never())
    return tw


def rnd(seed, *shape, std=1.0, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def case(dtype=torch.int64, seed=0):
    x, w = rnd(seed + 1, M, K), rnd(seed + 2, V, K, std=2 * K ** -0.5)
    t = torch.randint(0, V, (M,), generator=torch.Generator().manual_seed(seed))
    t[::6] = -100
    return x, w, t.to(dtype).cuda()


def shifted(t, by):
    """t as rows by, by + 1, ... of a longer tensor."""
    long = torch.full((len(t) + by + 3,), 7, dtype=t.dtype, device="cuda")
    long[by:by + len(t)] = t
    s = long[by:by + len(t)]
    assert s.data_ptr() % 16 == by * t.element_size() % 16
    return s


def same(a, b):
    assert a.keys() == b.keys() and all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("by", [1, 2, 3])
@pytest.mark.parametrize("dtype", [torch.int64, torch.int32])
def test_loss_and_its_gradient(way, by, dtype):
    x, w, t = case(dtype)
    dloss = rnd(3, M, dtype=F32)
    out = way.linear_ce(x, w, t)
    same(out, way.linear_ce(x, w, shifted(t, by)))
    ref = way.linear_ce_backward(dloss, x, w, t, out["lse"])
    same(ref, way.linear_ce_backward(shifted(dloss, by), x, w, shifted(t, by), shifted(out["lse"], by)))


@pytest.mark.parametrize("by", [1, 2, 3])
def test_norm_gradient(way, by):
    x, dy, gamma = rnd(1, M, K), rnd(2, M, K), 1 + 0.1 * rnd(3, K, dtype=F32)
    rstd = way.rmsnorm(x, gamma)["rstd"]
    same(way.rmsnorm_backward(dy, x, gamma, rstd), way.rmsnorm_backward(dy, x, gamma, shifted(rstd, by)))


def test_rows_that_do_not_lie_together_are_refused(tw):
    x, w, t = case()
    with pytest.raises(ValueError):
        tw.linear_ce(x, w, t.repeat_interleave(2)[1::2])
    with pytest.raises(ValueError):
        tw.linear_ce_backward(torch.ones((), device="cuda").expand(M), x, w, t, rnd(3, M, dtype=F32))


def test_captured_and_replayed(tw):
    """A replay reads the targets that are there then, not those of the capture."""
    x, w, t = case()
    tokens, dloss = shifted(t, 1), shifted(rnd(3, M, dtype=F32), 1)
    lse = shifted(tw.linear_ce(x, w, t)["lse"], 1)

    def calls():
        return {**tw.linear_ce(x, w, tokens), **tw.linear_ce_backward(dloss, x, w, tokens, lse)}

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for i in range(4):
        tokens.copy_(case(seed=10 + i)[2])
        dloss.mul_(1.5)
        for v in got.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        same(got, calls())


def test_on_another_stream(tw):
    x, w, t = case()
    ref = tw.linear_ce(x, w, t)
    tokens = shifted(t, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = tw.linear_ce(x, w, tokens)
    s.synchronize()
    same(ref, got)


def test_a_training_step_on_the_next_tokens(tw):
    from activation_sparse_feed_gate_amd import block

    x, w, t = case()
    layers = [(1 + 0.1 * rnd(4, K, dtype=F32), *(rnd(5 + i, 520, K, std=0.05) for i in range(3)))]
    gamma = 1 + 0.1 * rnd(9, K, dtype=F32)
    a = block.dense_train_step(x, layers, gamma, w, t)
    b = block.dense_train_step(x, layers, gamma, w, shifted(t, 1))
    assert torch.equal(a["loss"], b["loss"]) and torch.equal(a["dw_out"], b["dw_out"])
    same(a["layers"][0], b["layers"][0])
    assert torch.equal(block.dense_serve(x, layers, gamma, w, t),
                       block.dense_serve(x, layers, gamma, w, shifted(t, 1)))
