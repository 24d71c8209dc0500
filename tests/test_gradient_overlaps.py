"""Backward passes whose outputs would overwrite what a later kernel of the same call reads
are refused; the overlaps that leave every result as it is are not."""
import pytest
import torch

BF, F32 = torch.bfloat16, torch.float32
M, K, N, V = 5, 64, 72, 64


@pytest.fixture(scope="module")
def tw():
    from activation_sparse_feed_gate_amd import tw as mod

    return mod


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def ffn(tw, **kw):
    a = dict(dy=z(M, K), x=z(M, K), wg_t=z(N, K), wu_t=z(N, K), wd=z(N, K), g=z(M, N), u=z(M, N),
             ws=z(1 << 20), dx=z(M, K), dwg_t=z(N, K), dwu_t=z(N, K), dwd=z(N, K))
    a.update({k: a[v] if isinstance(v, str) else v for k, v in kw.items()})
    return tw.tw_gated_ffn_bwd(**a)


def ce(tw, **kw):
    a = dict(dloss=z(M, dtype=F32), x=z(M, K), w=z(V, K), target=z(M, dtype=torch.int64), lse=z(M, dtype=F32),
             ws=z(1 << 20), dx=z(M, K), dw=z(V, K))
    a.update({k: a[v] if isinstance(v, str) else v for k, v in kw.items()})
    return tw.tw_linear_ce_bwd(**a)


def parts():
    """Two [M][K] that share rows."""
    flat = z(2 * M * K)
    return flat[:M * K].view(M, K), flat[K:K + M * K].view(M, K)


NO_DW = dict(dwg_t=None, dwu_t=None, dwd=None)


@pytest.mark.parametrize("kw", [
    dict(dx="dy"), dict(dx="x"), dict(dwg_t="dwu_t"), dict(dwu_t="dwd"), dict(dwg_t="dwd"),
    dict(x=z(N, K)[:M], dwd=None)], ids=lambda kw: "-".join(kw))
def test_ffn(tw, kw):
    if "dwd" in kw and kw["dwd"] is None:  # x lies in a weight gradient
        big = z(N, K)
        kw = dict(x=big[:M], dwd=big)
    with pytest.raises(ValueError, match="overlap"):
        ffn(tw, **kw)


def test_ffn_parts(tw):
    a, b = parts()
    for kw in (dict(dx=a, dy=b), dict(dx=b, x=a)):
        with pytest.raises(ValueError, match="overlap"):
            ffn(tw, **kw)
    w = z(N * K + 8)
    with pytest.raises(ValueError, match="overlap"):
        ffn(tw, wg_t=w[8:].view(N, K), dx=w[:M * K].view(M, K), **NO_DW)


@pytest.mark.parametrize("kw", [dict(dx="x")], ids=["dx"])
def test_ce(tw, kw):
    with pytest.raises(ValueError, match="overlap"):
        ce(tw, **kw)
    w = z(V, K)
    flat = z(V * K + 8)
    for kw in (dict(w=w, dx=w[:M]), dict(w=w, dx=w[:M], dw=None), dict(dw=w, x=w[:M]), dict(dw=w, dx=w[-M:]),
               dict(w=flat[:-8].view(V, K), dw=flat[8:].view(V, K))):
        with pytest.raises(ValueError, match="overlap"):
            ce(tw, **kw)


def test_others_reach_the_library(tw):
    """(Which refuses the CPU's tensors.)"""
    flat = z(2 * M * K)
    a, b = flat[:M * K].view(M, K), flat[M * K:].view(M, K)
    for call in (lambda: ffn(tw), lambda: ffn(tw, dx="dy", **NO_DW), lambda: ffn(tw, dx="x", **NO_DW),
                 lambda: ffn(tw, dx=a, dy=b), lambda: ffn(tw, dx=b, x=a), lambda: ce(tw),
                 lambda: ce(tw, dx="x", dw=None), lambda: ce(tw, dx=b, x=a), lambda: ce(tw, dw="w"),
                 lambda: ffn(tw, dx=None),
                 lambda: ce(tw, dx=None)):
        with pytest.raises(ValueError, match="device tensors"):
            call()


@pytest.mark.gpu
def test_in_place_where_nothing_reads_them_again(tw):
    """dx over dy or x, without weight gradients: the bits of a buffer of its own."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator().manual_seed(1)

    def r(*shape, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(BF).cuda()

    for rows in (5, 300):
        x, dy, w = r(rows, K), r(rows, K), [r(N, K, std=0.1) for _ in range(3)]
        gate, up = r(rows, N), r(rows, N)
        ws = torch.empty(tw.tw_gated_ffn_bwd_workspace_bytes(rows, K, N), dtype=torch.uint8, device="cuda")
        ref = tw.gated_ffn_backward(dy, x, *w, gate, up)["dx"]
        tw.tw_gated_ffn_bwd(dy, x, *w, gate, up, ws, dx=dy)
        assert torch.equal(dy, ref)
        out, t = r(V, K, std=0.2), torch.arange(rows, device="cuda") % V
        lse, dloss = tw.linear_ce(x, out, t)["lse"], torch.ones(rows, device="cuda")
        ws = torch.empty(tw.tw_linear_ce_bwd_workspace_bytes(rows, K, V), dtype=torch.uint8, device="cuda")
        ref = tw.linear_ce_backward(dloss, x, out, t, lse)["dx"]
        both = tw.linear_ce_backward(dloss, x, out, t, lse)
        was, w = x.clone(), out.clone()
        tw.tw_linear_ce_bwd(dloss, x, w, t, lse, ws, dw=w)
        assert torch.equal(w, both["dw"]) and torch.equal(x, was)
        tw.tw_linear_ce_bwd(dloss, x, out, t, lse, ws, dx=x)
        assert torch.equal(x, ref)
