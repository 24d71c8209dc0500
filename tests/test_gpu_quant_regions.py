"""Large-tile int8 products whose tile grids split into regions of the XCDs:
every output of every split (8 x 1, 4 x 2, 2 x 4 row by column regions, and
the undivided walk), with remainder rows and columns, on fewer and on more
tiles than workgroups."""
import numpy as np
import pytest

import norm_ref as R
from test_gpu_quant import check, codes, gate_ref, num, scales, tw  # noqa: F401  (tw: the fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF, F32 = torch.bfloat16, torch.float32


# tile grids (linear, 256 x 256): 64x8, 16x16, 8x22, 8x17, 20x17 (none divides), 32x8 with one row left over
@pytest.mark.parametrize("M,N", [(16384, 2048), (16380, 2045), (4096, 4096), (4093, 4090), (2048, 5632), (2041, 4352),
                                 (5000, 4200), (8192 - 255, 2048)])
@pytest.mark.parametrize("K", [64, 272])
def test_linear(tw, M, N, K):
    q, w, xs, ws = codes(M, K, 1), codes(N, K, 2), scales(M, 3), scales(N, 4)
    b = torch.randn(N, generator=torch.Generator().manual_seed(5)).cuda()
    print(f"case {M} {K} {N}", flush=True)
    for yt, bias in ((BF, None), (F32, b)):
        y = tw.quant_linear(q, w, ws, bias=bias, x_scale=xs, out_dtype=yt)
        check(y, *R.product(num(q), num(xs), num(w), num(ws), None if bias is None else num(b)))


# gate/up, 256 x 128: 64x16, 16x32, 8x34, 8x33, 12x21 (none divides)
@pytest.mark.parametrize("M,N", [(16384, 2048), (16383, 2047), (4096, 4096), (2048, 4352), (2040, 4100), (2900, 2600)])
@pytest.mark.parametrize("K", [64, 272])
def test_gateup(tw, M, N, K):
    q, wg, wu = codes(M, K, 1), codes(N, K, 2), codes(N, K, 3)
    xs, gs, us = scales(M, 4), scales(N, 5), scales(N, 6)
    print(f"case {M} {K} {N}", flush=True)
    h = tw.quant_gateup(q, wg, gs, wu, us, x_scale=xs, out_dtype=BF)
    check(h, *gate_ref(num(q), num(xs), num(wg), num(gs), num(wu), num(us)))
    assert np.isfinite(num(h)).all()
