"""The pre-norm FFN sublayer that runs the norm, the int8 projections and the
hybrid training FFN together, and the native part of the binding."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mods():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from activation_sparse_feed_gate_amd import block, tw

    return block, tw


def test_block_against_float64(mods):
    """8-bit rounding (half a step of 127 levels in each of four operands): a
    few per cent.  Training: the norm's output, the gradient of y and the
    stored backup are bf16 (2^-8 each), every sum fp32: under 2 per cent."""
    r = mods[0].main()
    assert r.pop("int8 FFN output") < 0.05
    for k, v in r.items():
        assert v < 0.02, (k, v)


@pytest.mark.parametrize("M", [1, 3, 150])
def test_serving_stack(mods, M):
    """Three sublayers and a last norm: each FFN's output joins the stream in
    the next norm; within the 8-bit rounding of the same stack in float64."""
    block, tw = mods
    K, N = 512, 1536
    g = torch.Generator().manual_seed(M)
    x = torch.randn(M, K, generator=g)
    layers, ref = [], x.double()
    for _ in range(3):
        gamma, beta = 1 + 0.1 * torch.randn(K, generator=g), 0.1 * torch.randn(K, generator=g)
        w = [(torch.randn(N, K, generator=g) * s).bfloat16() for s in (K ** -0.5, K ** -0.5, N ** -0.5)]
        layers.append((gamma.cuda(), beta.cuda(), block.quantize_ffn(*(t.cuda() for t in w))))
        ref = block._reference(ref, gamma.double(), beta.double(), *(t.double() for t in w))
    gamma = torch.ones(K)
    y, stream = block.serve(x.cuda(), layers, gamma.cuda())
    assert stream.dtype == F32
    assert ((stream.double().cpu() - ref).norm() / ref.norm()).item() < 0.05
    d = ref - ref.mean(1, keepdim=True)
    n = d / (d.square().mean(1, keepdim=True) + 1e-5).sqrt()
    assert ((y.double().cpu() - n).norm() / n.norm()).item() < 0.05


# ------------------------------------------------- native part of the binding --
def calls(tw):
    """(name, function of the public binding, its arguments) over types,
    strides and optional arguments."""
    g = torch.Generator().manual_seed(5)

    def r(*shape, dtype=F32):
        return torch.randn(*shape, generator=g).to(dtype).cuda()

    M, K, N = 9, 64, 40
    gamma, beta, mean, rstd = r(K), r(K), r(M), r(M).abs()
    w = torch.randint(-127, 128, (N, K), dtype=torch.int8, generator=g).cuda()
    w2 = w.flip(0).contiguous()
    q = torch.randint(-127, 128, (M, K), dtype=torch.int8, generator=g).cuda()
    ws, xs, bias = r(N).abs(), r(M).abs(), r(N)
    space = torch.empty(tw.tw_quant_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    out = []
    for t in (BF, F32):
        x = r(M, K, dtype=t)
        wide = r(M, K + 3, dtype=t)[:, :K]
        out += [("layernorm", tw.layernorm, (x, gamma)), ("layernorm", tw.layernorm, (wide, gamma, beta)),
                ("layernorm", tw.layernorm, (x, gamma, beta, 1e-6, r(M, K), F32)),
                ("layernorm", tw.layernorm, (x, gamma, None, 0.5, r(M, K, dtype=BF), BF)),
                ("layernorm_backward", tw.layernorm_backward, (r(M, K, dtype=t), wide, gamma, mean, rstd)),
                ("layernorm_backward", tw.layernorm_backward, (r(M, K), x, gamma, mean, rstd, r(M, K, dtype=t), t)),
                ("quant_linear", tw.quant_linear, (x, w, ws)), ("quant_linear", tw.quant_linear, (wide, w, ws, bias, None, t, space)),
                ("quant_gateup", tw.quant_gateup, (x, w, ws, w2, ws, gamma, beta)),
                ("quant_gateup", tw.quant_gateup, (wide, w, ws, w2, ws, None, None, 1e-5, None, t, space))]
    out += [("quant_linear", tw.quant_linear, (q, w, ws, bias, xs)),
            ("quant_gateup", tw.quant_gateup, (q, w, ws, w2, ws, None, None, 1e-5, xs, F32))]
    return out


def flat(v):
    return v if isinstance(v, dict) else {"out": v}


def test_native_calls_equal_the_checked_ones(mods, monkeypatch):
    tw = mods[1]

    class Native:
        seen = []

        def __getattr__(self, name):
            def call(*a):
                v = getattr(native, name)(*a)
                self.seen.append((name, v is not None))
                return v
            return call

    class Never:
        def __getattr__(self, name):
            return lambda *a: None

    native = tw._calls
    for name, f, args in calls(tw):
        spy = Native()
        monkeypatch.setattr(tw, "_calls", spy)
        a = flat(f(*args))
        assert spy.seen == [(name, True)]
        spy.seen.clear()
        monkeypatch.setattr(tw, "_calls", Never())
        b = flat(f(*args))
        assert a.keys() == b.keys()
        for k in a:
            assert (a[k] is None) == (b[k] is None), k
            if a[k] is not None:
                assert a[k].dtype == b[k].dtype and torch.equal(a[k], b[k]), (name, k)


def test_bad_arguments_raise_through_the_allocating_calls(mods):
    tw = mods[1]
    x, gamma = torch.randn(4, 64, device="cuda"), torch.ones(64, device="cuda")
    w, ws = torch.zeros(32, 64, dtype=torch.int8, device="cuda"), torch.ones(32, device="cuda")
    for call, error, what in [
            (lambda: tw.layernorm(x.half(), gamma), TypeError, "x"),
            (lambda: tw.layernorm(x, gamma[:32]), ValueError, "gamma"),
            (lambda: tw.layernorm(x, gamma.cpu()), ValueError, "gamma"),
            (lambda: tw.layernorm(x, gamma, out_dtype=torch.float16), TypeError, "y"),
            (lambda: tw.layernorm(x, gamma, eps=-1.0), tw.TwError, "eps"),
            (lambda: tw.layernorm(x.t(), torch.ones(4, device="cuda")), ValueError, "contiguous rows"),
            (lambda: tw.layernorm(x[:, 1:], gamma[1:].contiguous()), tw.TwError, "aligned"),
            (lambda: tw.layernorm(torch.empty(2, 16385, device="cuda"), torch.ones(16385, device="cuda")), tw.TwError, "at most"),
            (lambda: tw.layernorm_backward(x, x, gamma, ws, ws), ValueError, "mean"),
            (lambda: tw.quant_linear(x, w.float(), ws), TypeError, "w"),
            (lambda: tw.quant_linear(x, w, ws, x_scale=ws[:4]), ValueError, "x is not int8"),
            (lambda: tw.quant_linear(x[:, :24].contiguous(), w[:, :24].contiguous(), ws), tw.TwError, "multiple of 16"),
            (lambda: tw.quant_linear(x, w, ws, ws=torch.empty(8, dtype=torch.uint8, device="cuda")), tw.TwError, "workspace"),
            (lambda: tw.quant_gateup(x, w, ws, w, ws, beta=gamma), tw.TwError, "beta"),
            (lambda: tw.quant_gateup(w, w, ws, w, ws, gamma=gamma, x_scale=ws), tw.TwError, "gamma")]:
        with pytest.raises(error, match=what):
            call()


def test_expanded_rows_are_refused(mods):
    """A broadcast row (distance 0) is not rows of memory: refused."""
    tw = mods[1]
    x = torch.randn(1, 64, device="cuda").expand(5, 64)
    with pytest.raises(tw.TwError, match="x_stride"):
        tw.layernorm(x, torch.ones(64, device="cuda"))
