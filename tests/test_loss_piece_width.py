"""Pieces of the vocabulary in the loss's backward pass: their rows stay within the limit
that 32-bit offsets of a tile's rows set, 2^22 words."""
import pytest
import torch

import train_ref as R

BF, F32 = torch.bfloat16, torch.float32
WIDTH = 1 << 22


@pytest.fixture(scope="module")
def tw():
    from activation_sparse_feed_gate_amd import tw as mod

    return mod


@pytest.mark.parametrize("M", [17, 20, 33, 48, 63])
def test_a_pieces_rows_are_bounded(tw, M):
    """17 to 63 rows against a vocabulary whose D takes more than 512 MB: D's piece is M
    rows of 2^22 words at most, and parts of dx and dw beside it."""
    K, V = 8, 1 << 24
    assert M * V * 2 > 512 << 20
    assert tw.tw_linear_ce_bwd_workspace_bytes(M, K, V) <= M * WIDTH * 2 + (9 << 20)


@pytest.mark.parametrize("M", [1, 16, 64])
def test_one_piece_where_few_rows_take_it_whole(tw, M):
    K, V = 8, 1 << 22
    assert tw.tw_linear_ce_bwd_workspace_bytes(M, K, V) >= M * V * 2


@pytest.mark.gpu
@pytest.mark.parametrize("M,V", [(20, (1 << 24) - 3), (17, 1 << 24)])
def test_a_long_vocabulary_in_pieces(tw, M, V):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    K = 8
    g = torch.Generator("cuda").manual_seed(M)
    w = torch.empty(V, K, dtype=BF, device="cuda").normal_(0, 0.7, generator=g)
    x = torch.randn(M, K, generator=torch.Generator().manual_seed(M)).to(BF).cuda()
    t = torch.arange(V - M, V, device="cuda")
    t[1], t[2], t[3] = 5, -100, WIDTH
    print(f"case {M}x{K}x{V}", flush=True)
    out = tw.linear_ce(x, w, t)
    dloss = torch.randn(M, generator=torch.Generator().manual_seed(1)).cuda()
    got = tw.linear_ce_backward(dloss, x, w, t, out["lse"], dx_dtype=F32, dw_dtype=F32)
    lse, wide, xd, off = out["lse"].double()[:, None], w.double(), x.double(), 0
    scale = torch.where(t >= 0, dloss.double(), 0.0)[:, None]
    dx, ex = torch.zeros_like(xd), torch.zeros_like(xd)
    for c in wide.split(1 << 22):
        # D of these words and its error as in train_ref.ce_bwd, which takes whole vocabularies
        l, e = R.logits(xd, c)
        d = (l - lse).exp()
        e = d * (e + (4 * l.abs() + 4 * lse.abs() + 8) * R.U)
        here = (t >= off) & (t < off + len(c))
        rows = torch.arange(M, device="cuda")[here]
        d[rows, t[here] - off] -= 1.0
        d, e = d * scale, (e + 2 * R.U * d.abs()) * scale.abs()
        e = e + R.UB * (d.abs() + e)
        R.close(got["dw"][off:off + len(c)], R.mm(d.T, xd),
                R.mm(e.T, xd.abs()) + (M + 8) * R.U * R.mm((d.abs() + e).T, xd.abs()))
        dx += R.mm(d, c)
        ex += R.mm(e, c.abs()) + (V + 72) * R.U * R.mm(d.abs() + e, c.abs())
        off += len(c)
    R.close(got["dx"], dx, ex)
    del w, wide, got, out
    torch.cuda.empty_cache()
