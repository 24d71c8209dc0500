"""The loss's gradient for 2^23 rows and a vocabulary in pieces: dx's parts are added by as
many workgroups as one grid dimension of 256 threads holds."""
import pytest

import train_ref as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF = torch.bfloat16


def test_rows_past_a_launch():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from activation_sparse_feed_gate_amd import tw

    M, K, V = 1 << 23, 2048, 300
    ws_bytes = tw.tw_linear_ce_bwd_workspace_bytes(M, K, V)
    if torch.cuda.mem_get_info()[0] < ws_bytes + 5 * M * K:
        pytest.skip("needs about 150 GB of device memory")
    print(f"case {M}x{K}x{V}", flush=True)
    x = torch.empty(M, K, dtype=BF, device="cuda")
    for i, c in enumerate(x.split(M // 16)):
        c.normal_(generator=torch.Generator("cuda").manual_seed(i))
    g = torch.Generator().manual_seed(1)
    w = (torch.randn(V, K, generator=g) * 2 * K ** -0.5).to(BF).cuda()
    t = torch.randint(0, V, (M,), generator=g).cuda()
    t[::9] = -100
    dloss = torch.randn(M, generator=g).cuda()
    lse = tw.linear_ce(x, w, t)["lse"]
    dx = torch.empty_like(x)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device="cuda")
    tw.tw_linear_ce_bwd(dloss, x, w, t, lse, ws, dx=dx)
    for rows in (slice(0, 300), slice(M // 2 - 100, M // 2 + 100), slice(M - 300, M)):
        ref = R.ce_bwd(dloss[rows].double(), x[rows].double(), w.double(), t[rows], lse[rows].double())
        R.close(dx[rows], *ref["dx"])
    del x, dx, ws, t, lse, dloss
    torch.cuda.empty_cache()
