"""A pre-norm FFN sublayer, y = x + FFN(norm(x)), on the library's kernels.

Serving, ``ffn_int8``: the layer norm, gate, up and down projections on 8-bit
integers (weights quantised once by ``quantize_ffn``); the FFN's output joins
the residual stream in the next layer norm.

Training, ``train_forward`` and ``train_backward``: the layer norm, the TwELL
gate and the hybrid sparse FFN, and their gradients.

``python -m activation_sparse_feed_gate_amd.block`` runs both on a GPU at a small
shape and compares them with the same sublayer in float64.
"""
from __future__ import annotations

import torch

from . import tw


def quantize_ffn(wg_t, wu_t, wd):
    """int8 weights of an FFN given in the library's layout ([N][K] each: W_g
    and W_u transposed, W_d itself), one scale per output channel: per hidden
    neuron for gate and up, per model channel for down."""
    q = {}
    for name, w in (("g", wg_t), ("u", wu_t), ("d", wd.t().contiguous())):
        q["w" + name], q[name + "_scale"] = tw.quantize_rows(w)
    return q


def ffn_int8(x, gamma, beta, q, eps=1e-5):
    """FFN(norm(x)) on int8 operands, fp32 [M][K] (``x``: the residual stream,
    bf16 or fp32; ``q``: from ``quantize_ffn``)."""
    h = tw.quant_gateup(x, q["wg"], q["g_scale"], q["wu"], q["u_scale"], gamma=gamma, beta=beta,
                        eps=eps)
    return tw.quant_linear(h, q["wd"], q["d_scale"], out_dtype=torch.float32)


def serve(x, layers, gamma_out, beta_out=None, eps=1e-5):
    """A stack of sublayers (gamma, beta, q) on rows x, ending in a last norm:
    every FFN's output is added to the stream by a norm kernel.  Returns
    (normed bf16, stream)."""
    stream, add = x, None
    for gamma, beta, q in layers:
        if add is None:
            add = ffn_int8(stream, gamma, beta, q, eps)
            continue
        n = tw.layernorm_quantize(stream, gamma, beta, eps, add=add)
        stream = n["sum"]
        h = tw.quant_gateup(n["q"], q["wg"], q["g_scale"], q["wu"], q["u_scale"],
                            x_scale=n["scale"])
        add = tw.quant_linear(h, q["wd"], q["d_scale"], out_dtype=torch.float32)
    out = tw.layernorm(stream, gamma_out, beta_out, eps, add=add)
    return out["y"], stream if add is None else out["sum"]


def train_forward(x, gamma, beta, wg_t, wu_t, wd, T=128, C=128, P=128, R_max=None, eps=1e-5):
    """y = x + FFN(norm(x)) for training (fp32 [M][K]); x fp32 or bf16, weights
    bf16.  Returns (y, what ``train_backward`` needs).

    A row with more than P active neurons, or more than C in one tile of T (at
    random initialisation about half of N are active), lives in the dense
    backup of R_max rows: by default there is one for every row.  For a smaller
    backup the call waits for the number of rows that need it and raises where
    they do not fit, since such a row would have no output."""
    M, N = x.shape[0], wg_t.shape[0]
    # the backup's own limit is 2^31 elements
    R_max = min(M, (2 ** 31 - 1) // N if R_max is None else R_max)
    n = tw.layernorm(x, gamma, beta, eps)
    packed = tw.pack_gate(n["y"], wg_t, T, C, 0)
    f, hy = tw.hybrid_forward(n["y"], wg_t, wu_t, wd, packed, P=P, R_max=R_max)
    if R_max < M:
        need = int(hy["bk_count"])
        if need > R_max:
            raise RuntimeError(f"train_forward: {need} rows have more active neurons than a "
                               f"sparse row holds, the dense backup has room for {R_max}")
    return x.float() + f, dict(x=x, n=n, hy=hy, gamma=gamma, weights=(wg_t, wu_t, wd))


def train_backward(dy, saved, l1=0.0):
    """Gradients of ``train_forward`` for dy = dLoss/dy (fp32 [M][K]): dx,
    dgamma, dbeta and those of the weights (``hybrid_backward``'s names)."""
    n = saved["n"]
    g = tw.hybrid_backward(n["y"], *saved["weights"], dy.to(torch.bfloat16), saved["hy"], l1)
    out = tw.layernorm_backward(g["dx"], saved["x"], saved["gamma"], n["mean"], n["rstd"],
                                dres=dy)
    for k in ("dwg_t", "dwu_t", "dwd"):
        out[k] = g[k]
    return out


def _reference(x, gamma, beta, wg_t, wu_t, wd, eps=1e-5):
    """x + FFN(norm(x)) in torch, in the tensors' own precision but for the
    norm's output, which the FFN reads as bf16: rounded here too (gradients
    pass it unchanged), so that ReLU cuts the same gate entries."""
    d = x - x.mean(1, keepdim=True)
    n = d / (d.square().mean(1, keepdim=True) + eps).sqrt() * gamma + beta
    n = n + (n.bfloat16().to(n.dtype) - n).detach()
    return x + (torch.relu(n @ wg_t.T) * (n @ wu_t.T)) @ wd


def main(M=200, K=256, N=1024):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(M, K, generator=g)
    gamma, beta = 1 + 0.1 * torch.randn(K, generator=g), 0.1 * torch.randn(K, generator=g)
    w = [(torch.randn(N, K, generator=g) * s).bfloat16() for s in (K ** -0.5, K ** -0.5, N ** -0.5)]
    dy = torch.randn(M, K, generator=g)
    wide = [t.double().requires_grad_() for t in (x, gamma, beta, *w)]
    y_ref = _reference(*wide)
    (y_ref * dy).sum().backward()
    grads = dict(zip(("dx", "dgamma", "dbeta", "dwg_t", "dwu_t", "dwd"), (t.grad for t in wide)))
    dev = [t.cuda() for t in (x, gamma, beta, *w)]

    def off(a, b):
        return ((a.double().cpu() - b).norm() / b.norm()).item()

    result = {"int8 FFN output": off(ffn_int8(*dev[:3], quantize_ffn(*dev[3:])),
                                     (y_ref - wide[0]).detach())}
    y, saved = train_forward(*dev, R_max=M)
    result["training output"] = off(y, y_ref.detach())
    got = train_backward(dy.cuda(), saved)
    for k, v in grads.items():
        result[k] = off(got[k], v)
    for k, v in result.items():
        print(f"{k:>18}: {v:.2e} of its norm from float64")
    return result


if __name__ == "__main__":
    main()
