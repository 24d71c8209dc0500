"""Gradient clipping: the norm and the workspace may overlap no buffer of the call.  The
refusals happen on the host (fake addresses); the GPU takes neighbours that touch."""
import ctypes
import math

import pytest
import torch

G, OUT, NORM, WS = 0x100000, 0x200000, 0x300000, 0x400000
N = 100  # fp32 elements: 400 bytes


@pytest.fixture(scope="module")
def tw():
    from activation_sparse_feed_gate_amd import tw as mod

    return mod


def call(tw, f, g=G, out=OUT, norm=NORM, ws=WS):
    arr = (ctypes.c_void_p * 2)(g, 0), (ctypes.c_int64 * 2)(N, 0), (ctypes.c_int * 2)(1, 1)
    need = tw.tw_grad_norm_workspace_bytes([N, 0])
    assert need == 8
    if f == "norm":
        return tw._lib.tw_grad_norm(2, *arr, norm, ws, 1 << 20, None, None)
    o = (ctypes.c_void_p * 2)(out, 0)
    return tw._lib.tw_grad_clip(2, *arr, o, arr[2], 1.0, 0.0, norm, ws, 1 << 20, None, None)


@pytest.mark.parametrize("f", ["norm", "clip"])
@pytest.mark.parametrize("kw,words", [
    (dict(norm=G), ("g[0]", "norm")), (dict(norm=G + 396), ("g[0]", "norm")),
    (dict(ws=G), ("g[0]", "workspace")), (dict(ws=G + 384), ("g[0]", "workspace")),
    (dict(norm=WS), ("norm", "workspace")), (dict(norm=WS + 4), ("norm", "workspace"))])
def test_the_norm_and_the_workspace_overlap_nothing(tw, f, kw, words):
    assert call(tw, f, **kw) == 1
    message = tw._lib.tw_last_error().decode()
    assert all(w in message for w in words) and "overlap" in message, message


@pytest.mark.parametrize("kw,word", [(dict(norm=OUT), "norm"), (dict(norm=OUT + 396), "norm"),
                                     (dict(ws=OUT), "workspace"), (dict(ws=OUT + 384), "workspace"),
                                     (dict(out=G, norm=G + 4), "norm"), (dict(out=G, ws=G + 16), "workspace")])
def test_nor_an_output(tw, kw, word):
    assert call(tw, "clip", **kw) == 1
    message = tw._lib.tw_last_error().decode()
    assert word in message and "overlap" in message, message


@pytest.mark.gpu
def test_neighbours_that_touch(tw):
    """One buffer: the workspace, the gradients, the norm, the outputs, end to end."""
    flat = torch.zeros(1 << 12, device="cuda")
    ws, g, norm, out = flat[:4], flat[4:4 + N], flat[4 + N], flat[5 + N:5 + 2 * N]
    g.copy_(torch.randn(N, generator=torch.Generator().manual_seed(1)))
    was = g.clone()
    ref = math.sqrt(float((g.double() ** 2).sum()))
    assert tw.tw_grad_norm_workspace_bytes([N]) <= 16
    tw.tw_grad_norm([g], norm, ws)
    assert abs(float(norm) - ref) < 1e-5 * ref
    norm.zero_()
    tw.tw_grad_clip([g], [out], 0.5 * ref, 0.0, norm, ws)
    assert abs(float(norm) - ref) < 1e-5 * ref and torch.equal(g, was)
    assert (out - 0.5 * g).abs().max() < 1e-5 * g.abs().max() and (flat[5 + 2 * N:] == 0).all()
    # a workspace longer than the call needs may run on into the gradients
    long = flat[:64]
    tw.tw_grad_norm([g], norm, long)
    assert abs(float(norm) - ref) < 1e-5 * ref and torch.equal(g, was)
