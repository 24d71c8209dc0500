"""A pre-norm FFN sublayer, y = x + FFN(norm(x)), on the library's kernels.

Serving, ``ffn_int8``: the layer norm, gate, up and down projections on 8-bit
integers (weights quantised once by ``quantize_ffn``); the FFN's output joins
the residual stream in the next layer norm.

Training, ``train_forward`` and ``train_backward``: the layer norm, the TwELL
gate and the hybrid sparse FFN, and their gradients.

The dense baseline, ``dense_train_step``: a stack of RMS norm and gated FFN
sublayers, the output projection's cross entropy and the clipped gradients;
``dense_serve`` scores tokens with the same weights.

``python -m activation_sparse_feed_gate_amd.block`` runs them on a GPU at a small
shape and compares them with the same computation in float64.
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


def serve(x, layers, gamma_out, beta_out=None, eps=1e-5, norm="layer"):
    """A stack of sublayers (gamma, beta, q) on rows x, ending in a last norm:
    every FFN's output is added to the stream by a norm kernel.  Returns
    (normed bf16, stream).  ``norm`` "rms": RMS norms, whose beta is None."""
    if norm not in ("layer", "rms"):
        raise ValueError(f'serve: norm must be "layer" or "rms", got {norm!r}')
    if norm == "rms":
        return _serve_rms(x, layers, gamma_out, beta_out, eps)
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


def _serve_rms(x, layers, gamma_out, beta_out, eps):
    if beta_out is not None or any(beta is not None for _, beta, _ in layers):
        raise ValueError("serve: an RMS norm has no beta")
    stream, add = x, None
    for gamma, _, q in layers:
        n = tw.rmsnorm_quantize(stream, gamma, eps, add=add)
        stream = stream if add is None else n["sum"]
        h = tw.quant_gateup(n["q"], q["wg"], q["g_scale"], q["wu"], q["u_scale"],
                            x_scale=n["scale"])
        add = tw.quant_linear(h, q["wd"], q["d_scale"], out_dtype=torch.float32)
    out = tw.rmsnorm(stream, gamma_out, eps, add=add)
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


def _dense_forward(x, layers, gamma_out, act, eps, keep):
    """Stack of (gamma, wg_t, wu_t, wd) sublayers on the stream x, ending in a
    last norm: every norm adds the FFN's output before it.  Returns the last
    norm's dict and, with ``keep``, what each sublayer's gradient reads."""
    stream, add, saved = x, None, []
    for gamma, wg_t, wu_t, wd in layers:
        n = tw.rmsnorm(stream, gamma, eps, add=add)
        stream = stream if add is None else n["sum"]
        f = tw.gated_ffn(n["y"], wg_t, wu_t, wd, act=act, keep=keep, out_dtype=x.dtype)
        add = f["y"]
        if keep:
            saved.append((n["y"], stream, n["rstd"], f["g"], f["u"]))
    n = tw.rmsnorm(stream, gamma_out, eps, add=add)
    if add is None:
        n["sum"] = stream
    return n, saved


def dense_serve(x, layers, gamma_out, w_out, target, act="silu", eps=1e-5):
    """Log-probabilities (fp32 [M]) of ``target`` after the rows x: 0 where a row
    has no target (outside [0, V))."""
    n, _ = _dense_forward(x, layers, gamma_out, act, eps, False)
    return -tw.linear_ce(n["y"], w_out, target)["loss"]


def dense_train_step(x, layers, gamma_out, w_out, target, act="silu", eps=1e-5, max_norm=1.0):
    """Loss and clipped gradients of a stack of pre-norm sublayers under the cross
    entropy of an output projection, averaged over the rows that have a target.

    x [M][K] bf16 or fp32, layers a list of (gamma, wg_t, wu_t, wd), w_out [V][K].
    Returns a dict: loss and norm (scalar tensors; the norm before clipping), dx,
    layers (a list of dicts dgamma, dwg_t, dwu_t, dwd), dgamma_out, dw_out."""
    n, saved = _dense_forward(x, layers, gamma_out, act, eps, True)
    ce = tw.linear_ce(n["y"], w_out, target)
    has = ((target >= 0) & (target < w_out.shape[0])).float()
    dloss = has / has.sum().clamp(min=1.0)
    out = {"loss": (ce["loss"] * dloss).sum(), "layers": []}
    g = tw.linear_ce_backward(dloss, n["y"], w_out, target, ce["lse"])
    out["dw_out"] = g["dw"]
    b = tw.rmsnorm_backward(g["dx"], n["sum"], gamma_out, n["rstd"], dx_dtype=x.dtype)
    out["dgamma_out"], d = b["dgamma"], b["dx"]
    for (gamma, *weights), (y, stream, rstd, gate, up) in zip(reversed(layers), reversed(saved)):
        f = tw.gated_ffn_backward(d.to(torch.bfloat16), y, *weights, gate, up, act=act)
        b = tw.rmsnorm_backward(f.pop("dx"), stream, gamma, rstd, dres=d, dx_dtype=x.dtype)
        d = b["dx"]
        out["layers"].insert(0, {"dgamma": b["dgamma"], **f})
    out["dx"] = d
    grads = [out["dw_out"], out["dgamma_out"], *(t for f in out["layers"] for t in f.values())]
    out["norm"] = tw.clip_grads(grads, max_norm)
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


def _dense_reference(x, layers, gamma_out, w_out, target, act, eps=1e-5):
    """Mean loss of ``dense_train_step`` in torch, in the tensors' own precision."""
    def norm(z, gamma):
        return z * (z.square().mean(1, keepdim=True) + eps).rsqrt() * gamma

    f = {"relu": torch.relu, "silu": torch.nn.functional.silu,
         "gelu": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[act]
    for gamma, wg_t, wu_t, wd in layers:
        n = norm(x, gamma)
        x = x + (f(n @ wg_t.T) * (n @ wu_t.T)) @ wd
    return torch.nn.functional.cross_entropy(norm(x, gamma_out) @ w_out.T, target,
                                             ignore_index=-100)


def dense_main(M=200, K=256, N=688, V=1001, depth=2, act="silu"):
    g = torch.Generator().manual_seed(2)

    def matrix(rows, std):
        return (torch.randn(rows, K, generator=g) * std).bfloat16()

    def gamma():
        return 1 + 0.1 * torch.randn(K, generator=g)

    x = torch.randn(M, K, generator=g)
    layers = [(gamma(), matrix(N, K ** -0.5), matrix(N, K ** -0.5), matrix(N, N ** -0.5))
              for _ in range(depth)]
    gamma_out, w_out = gamma(), matrix(V, 2 * K ** -0.5)
    target = torch.randint(0, V, (M,), generator=g)
    target[::7] = -100
    wide = [x, *(t for layer in layers for t in layer), gamma_out, w_out]
    wide = [t.double().requires_grad_() for t in wide]
    stack = [tuple(wide[1 + 4 * i:5 + 4 * i]) for i in range(depth)]
    loss = _dense_reference(wide[0], stack, wide[-2], wide[-1], target, act)
    loss.backward()
    norm = torch.stack([t.grad.square().sum() for t in wide[1:]]).sum().sqrt()
    most = 0.5 * norm.item()
    got = dense_train_step(x.cuda(), [tuple(t.cuda() for t in layer) for layer in layers],
                           gamma_out.cuda(), w_out.cuda(), target.cuda(), act=act, max_norm=most)

    def off(a, b):
        return ((a.double().cpu() - b).norm() / b.norm()).item()

    result = {"loss": off(got["loss"], loss.detach()), "norm": off(got["norm"], norm),
              "dx": off(got["dx"], wide[0].grad),
              "dgamma_out": off(got["dgamma_out"], 0.5 * wide[-2].grad),
              "dw_out": off(got["dw_out"], 0.5 * wide[-1].grad)}
    for i, layer in enumerate(got["layers"]):
        for j, (k, v) in enumerate(layer.items()):
            result[f"{k} {i}"] = off(v, 0.5 * stack[i][j].grad)
    logp = dense_serve(x.cuda(), [tuple(t.cuda() for t in layer) for layer in layers],
                       gamma_out.cuda(), w_out.cuda(), target.cuda(), act=act)
    result["served loss"] = off(-logp.sum() / (target >= 0).sum(), loss.detach())
    for k, v in result.items():
        print(f"{k:>18}: {v:.2e} of its norm from float64")
    return result


if __name__ == "__main__":
    main()
    dense_main()
