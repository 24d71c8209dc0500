"""Cases of the operators of a dense training step and its serving form: the root-mean-square norm,
the gated FFN with its backward pass, the cross entropy of the output projection, gradient clipping.

Operators
  rms       z = x (+ add), y = z / sqrt(mean(z^2) + eps) * gamma; the sum z is an output where `add` is
            given; y in bf16, or in 8-bit integers with a scale a row
  rms_bwd   dx (+ the gradient arriving at z past the norm) and dgamma
  ffn       y = (act(x Wg) * (x Wu)) Wd, act SiLU, GELU (tanh form) or ReLU; a training step keeps the
            gate and up values before the activation
  ffn_bwd   dx, dWg, dWu, dWd from dy and those values
  ce        loss and log-sum-exp of every row of x W^T over a vocabulary; rows without a target are left out
  ce_bwd    dx and dW from the gradient of every row's loss
  clip      the norm over many gradients, and the gradients times min(1, most / norm)

``run`` computes them in plain torch operations, or (``own``) through this repository's binding.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
EPS = 1e-5
TINY = 2.0 ** -100  # a row whose largest magnitude is below this quantises to zeros


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # the norm in front of the next FFN while 8 sequences decode: latency is all there is
        dict(name="rms decode 8x2048", op="rms", M=8, K=2048, x="bf16", add="f32", y="bf16", pad=0),
        # a long prompt's float32 stream takes the FFN's output in; the int8 projections read the norm
        dict(name="rms int8 16384x2048", op="rms", M=16384, K=2048, x="f32", add="bf16", y="int8", pad=0),
        # the 2B block's norm in a training step's backward pass, the residual's gradient added
        dict(name="rms_bwd 16384x2048", op="rms_bwd", M=16384, K=2048, dy="bf16", x="bf16", res="yes", dx="bf16"),
        # one decoded token through the paper's block width
        dict(name="ffn decode 1x2048x5632", op="ffn", M=1, K=2048, N=5632, act="silu", keep=False, pad=0),
        # a ragged batch at sizes that no tile divides, rows of a wider buffer
        dict(name="ffn ragged 777x1000x2728", op="ffn", M=777, K=1000, N=2728, act="gelu", keep=False, pad=24),
        # the 2B block's training forward
        dict(name="ffn train 16384x2048x8192", op="ffn", M=16384, K=2048, N=8192, act="silu", keep=True, pad=0),
        # the 0.5B block's training backward
        dict(name="ffn_bwd 4096x1024x4096", op="ffn_bwd", M=4096, K=1024, N=4096, act="silu", pad=0),
        # log-probabilities of 4 decoded tokens
        dict(name="ce score 4x1024x32768", op="ce", M=4, K=1024, V=32768, pad=0),
        # the 0.5B model's loss over a batch of 4096 tokens
        dict(name="ce train 4096x1024x32768", op="ce", M=4096, K=1024, V=32768, pad=0),
        # its gradient, a vocabulary of odd size
        dict(name="ce_bwd 4096x1024x49999", op="ce_bwd", M=4096, K=1024, V=49999, pad=0),
        # a small model's gradients: matrices and vectors, some of odd sizes
        dict(name="clip small 26 tensors", op="clip", layers=4, K=256, N=1001, g="f32", out="f32", over=True),
        # a 0.5B model's bf16 gradients, clipped into the optimizer's float32 ones
        dict(name="clip 0.5B 146 tensors", op="clip", layers=24, K=1024, N=4096, g="bf16", out="f32", over=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _of(rng, *values):
    return values[rng.randrange(len(values))]


def _eights(rng, lo, hi):
    n = _log(rng, lo, hi)
    return 8 * n if rng.random() < 0.5 else -(-n // 16) * 128


def draw(rng):
    op = _of(rng, "rms", "rms_bwd", "ffn", "ffn_bwd", "ce", "ce_bwd", "clip")
    M = _log(rng, 1, 16384)
    if op in ("rms", "rms_bwd"):
        K = _log(rng, 64, 8192)
        K = K if rng.random() < 0.5 else -(-K // 64) * 64
        M = max(1, min(M, 16384 * 2048 // K))
        if op == "rms":
            return dict(op=op, M=M, K=K, x=_of(rng, "bf16", "f32"), add=_of(rng, "no", "bf16", "f32"),
                        y=_of(rng, "bf16", "f32", "int8"), pad=_of(rng, 0, 0, 8, 3))
        return dict(op=op, M=M, K=K, dy=_of(rng, "bf16", "f32"), x=_of(rng, "bf16", "f32"),
                    res=_of(rng, "no", "yes"), dx=_of(rng, "bf16", "f32"))
    if op in ("ffn", "ffn_bwd"):
        K, N = _eights(rng, 16, 512), _eights(rng, 16, 1024)
        M = max(1, min(M, 16384 * 2048 * 8192 // (2 * K * N)))
        c = dict(op=op, M=M, K=K, N=N, act=_of(rng, "silu", "gelu", "relu"), pad=_of(rng, 0, 0, 8, 40))
        if op == "ffn":
            c["keep"] = rng.random() < 0.4
        return c
    if op in ("ce", "ce_bwd"):
        K, V = _eights(rng, 16, 256), _log(rng, 500, 60000)
        M = max(1, min(M, 4096 * 1024 * 49999 // (K * V)))
        return dict(op=op, M=M, K=K, V=V, pad=_of(rng, 0, 0, 8, 40))
    g = _of(rng, "bf16", "f32")
    return dict(op=op, layers=_log(rng, 1, 24), K=_log(rng, 32, 1024), N=_log(rng, 64, 4096), g=g,
                out=_of(rng, g, "f32"), over=rng.random() < 0.8)


def _shapes(c):
    """Gradients of a model of c["layers"] blocks: two norms' and four matrices' each, then the output's."""
    K, N = c["K"], c["N"]
    return [(K,), (K, K), (N, K), (N, K), (N, K), (K,)] * c["layers"] + [(K,), (2 * N, K)]


def work(c):
    if c["op"] == "clip":
        n = sum(math.prod(s) for s in _shapes(c))
        return {"bytes": n * (2 * SIZE[c["g"]] + SIZE[c["out"]]), "flops": 3 * n}
    M, K = c["M"], c["K"]
    if c["op"] == "rms":
        add = SIZE.get(c["add"], 0)
        row = SIZE[c["x"]] + add + (SIZE[c["x"]] if add else 0) + SIZE.get(c["y"], 1)
        return {"bytes": M * K * row + 4 * M + 4 * K, "flops": 4 * M * K}
    if c["op"] == "rms_bwd":
        dx = SIZE[c["dx"]]
        row = SIZE[c["dy"]] + SIZE[c["x"]] + dx + (dx if c["res"] == "yes" else 0)
        return {"bytes": M * K * row + 4 * M + 8 * K, "flops": 9 * M * K}
    if c["op"] == "ffn":
        return {"bytes": 2 * (2 * M * K + 3 * K * c["N"] + (2 * M * c["N"] if c["keep"] else 0)),
                "flops": 6 * M * K * c["N"]}
    if c["op"] == "ffn_bwd":
        return {"bytes": 2 * (3 * M * K + 2 * M * c["N"] + 6 * K * c["N"]), "flops": 12 * M * K * c["N"]}
    V = c["V"]
    if c["op"] == "ce":
        return {"bytes": 2 * (M + V) * K + 16 * M, "flops": 2 * M * K * V}
    return {"bytes": 4 * (M + V) * K + 16 * M, "flops": 6 * M * K * V}


# ------------------------------------------------------------------ inputs --
def _padded(x, pad):
    """The rows of x; with `pad`, as the first columns of a wider buffer."""
    if not pad:
        return x
    wide = torch.zeros(x.shape[0], x.shape[1] + pad, dtype=x.dtype, device=DEV)
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def _stream(g, M, K, dtype, pad=0):
    """Rows of a residual stream: a few channels far larger than the rest."""
    channel = torch.exp(0.3 * torch.randn(K, generator=g, device=DEV))
    channel[torch.randint(0, K, (max(1, K // 256),), generator=g, device=DEV)] *= 12.0
    x = torch.randn(M, K, generator=g, device=DEV).mul_(channel)
    return _padded(x.to(dtype), pad)


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device=DEV).mul_(std).to(dtype)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = dict(case=c)
    if c["op"] == "clip":
        s["grads"] = [_normal(g, *shape, std=1e-3, dtype=TYPES[c["g"]]) for shape in _shapes(c)]
        n = sum(t.numel() for t in s["grads"])
        s["flat"] = torch.empty(n, dtype=TYPES[c["out"]], device=DEV)  # the optimizer's one buffer
        s["out"] = [v.view(t.shape) for v, t in zip(s["flat"].split([t.numel() for t in s["grads"]]), s["grads"])]
        s["most"] = (0.3 if c["over"] else 3.0) * 1e-3 * math.sqrt(n)
        return s
    M, K = c["M"], c["K"]
    if c["op"] in ("rms", "rms_bwd"):
        s["gamma"] = 1.0 + 0.1 * torch.randn(K, generator=g, device=DEV)
        s["x"] = _stream(g, M, K, TYPES[c["x"]], c.get("pad", 0))
        if c["op"] == "rms":
            s["add"] = None if c["add"] == "no" else _normal(g, M, K, dtype=TYPES[c["add"]])
            return s
        s["dy"] = _normal(g, M, K, dtype=TYPES[c["dy"]])
        s["res"] = _normal(g, M, K, dtype=TYPES[c["dx"]]) if c["res"] == "yes" else None
        s["rstd"] = torch.rsqrt(s["x"].double().square().mean(1) + EPS).float()
        return s
    s["x"] = _padded(_normal(g, M, K), c["pad"])
    if c["op"] in ("ffn", "ffn_bwd"):
        N = c["N"]
        s["wg"], s["wu"] = (_normal(g, N, K, std=K ** -0.5) for _ in "gu")
        s["wd"] = _normal(g, N, K, std=N ** -0.5)
        if c["op"] == "ffn_bwd":
            s["dy"] = _normal(g, M, K)
            x = s["x"].float()
            s["g"], s["u"] = ((x @ s[w].float().T).to(torch.bfloat16) for w in ("wg", "wu"))
        return s
    V = c["V"]
    s["w"] = _normal(g, V, K, std=2.0 * K ** -0.5)
    # most targets are as unlikely as any word, some are what the model expects; padding has none
    t = torch.randint(0, V, (M,), generator=g, device=DEV)
    some = torch.rand(M, generator=g, device=DEV)
    s["x"][some < 0.3] += 2.5 * s["w"][t[some < 0.3]]
    s["target"] = torch.where(some > 0.93, torch.full_like(t, -100), t)
    if c["op"] == "ce_bwd":
        s["dloss"] = (torch.rand(M, generator=g, device=DEV) + 0.5) / M
        top = s["x"].float() @ s["w"].float().T
        s["lse"] = torch.logsumexp(top, 1)
    return s


# -------------------------------------------------------------- plain forms --
def _activated(act, g):
    """act(g) and its derivative."""
    if act == "relu":
        return g.clamp(min=0.0), (g > 0).float()
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def _bf16(t):
    return t.to(torch.bfloat16)


def _plain_rms(s):
    c = s["case"]
    z = s["x"].float()
    if s["add"] is not None:
        z = z + s["add"].float()
    rstd = torch.rsqrt((z * z).mean(1, keepdim=True) + EPS)
    y = z * rstd * s["gamma"]
    if c["y"] == "int8":
        top = y.abs().amax(1, keepdim=True)
        some = top >= TINY
        q = torch.round(y * torch.where(some, 127.0 / top, 0.0))
        scale = torch.where(some, top / 127.0, 0.0)
        out = {"values": _bf16(q * scale), "scale": scale[:, 0]}
    else:
        out = {"y": y.to(TYPES[c["y"]]), "rstd": rstd[:, 0]}
    if s["add"] is not None:
        out["sum"] = z.to(TYPES[c["x"]])
    return out


def _plain_rms_bwd(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    n = s["x"].float() * rstd
    t = dy * s["gamma"]
    dx = rstd * (t - n * (t * n).mean(1, keepdim=True))
    if s["res"] is not None:
        dx = dx + s["res"].float()
    return {"dx": dx.to(TYPES[s["case"]["dx"]]), "dgamma": (dy * n).sum(0)}


def _plain_ffn(s):
    x = s["x"].float()
    g, u = x @ s["wg"].float().T, x @ s["wu"].float().T
    y = _bf16((_activated(s["case"]["act"], g)[0] * u) @ s["wd"].float())
    return {"y": y, "g": _bf16(g), "u": _bf16(u)} if s["case"]["keep"] else {"y": y}


def _plain_ffn_bwd(s):
    x, dy, g, u = (s[k].float() for k in ("x", "dy", "g", "u"))
    a, da = _activated(s["case"]["act"], g)
    dh = dy @ s["wd"].float().T
    dg, du = dh * u * da, dh * a
    return {"dx": _bf16(dg @ s["wg"].float() + du @ s["wu"].float()), "dwg_t": _bf16(dg.T @ x),
            "dwu_t": _bf16(du.T @ x), "dwd": _bf16((a * u).T @ dy)}


def _plain_ce(s):
    logits = s["x"].float() @ s["w"].float().T
    top = logits.amax(1, keepdim=True)
    lse = (top + torch.log(torch.exp(logits - top).sum(1, keepdim=True)))[:, 0]
    has = s["target"] >= 0
    at = logits.gather(1, s["target"].clamp(min=0)[:, None])[:, 0]
    return {"loss": torch.where(has, lse - at, 0.0), "lse": lse}


def _plain_ce_bwd(s):
    x, w = s["x"].float(), s["w"].float()
    d = torch.exp(x @ w.T - s["lse"][:, None])
    has = s["target"] >= 0
    rows = torch.arange(d.shape[0], device=DEV)
    d[rows, s["target"].clamp(min=0)] -= 1.0
    d = d * torch.where(has, s["dloss"], 0.0)[:, None]
    return {"dx": _bf16(d @ w), "dw": _bf16(d.T @ x)}


def _plain_clip(s):
    norm = torch.sqrt(torch.stack([(g.float() * g.float()).sum() for g in s["grads"]]).sum())
    by = (s["most"] / (norm + 1e-6)).clamp(max=1.0)
    return {"norm": norm, "out": torch.cat([(g.float() * by).to(s["flat"].dtype).reshape(-1)
                                            for g in s["grads"]])}


_PLAIN = dict(rms=_plain_rms, rms_bwd=_plain_rms_bwd, ffn=_plain_ffn, ffn_bwd=_plain_ffn_bwd,
              ce=_plain_ce, ce_bwd=_plain_ce_bwd, clip=_plain_clip)


# --------------------------------------------------------------------- run --
def _own(s):
    from activation_sparse_feed_gate_amd import tw

    c, op = s["case"], s["case"]["op"]
    if op == "rms" and c["y"] == "int8":
        out = tw.rmsnorm_quantize(s["x"], s["gamma"], EPS, add=s["add"])
        got = {"values": _bf16(out["q"] * out["scale"][:, None]), "scale": out["scale"]}
        return got if s["add"] is None else {**got, "sum": out["sum"]}
    if op == "rms":
        out = tw.rmsnorm(s["x"], s["gamma"], EPS, add=s["add"], out_dtype=TYPES[c["y"]])
        return {k: v for k, v in out.items() if v is not None}
    if op == "rms_bwd":
        return tw.rmsnorm_backward(s["dy"], s["x"], s["gamma"], s["rstd"], dres=s["res"],
                                   dx_dtype=TYPES[c["dx"]])
    if op == "ffn":
        out = tw.gated_ffn(s["x"], s["wg"], s["wu"], s["wd"], act=c["act"], keep=c["keep"])
        return {k: v for k, v in out.items() if v is not None}
    if op == "ffn_bwd":
        return tw.gated_ffn_backward(s["dy"], s["x"], s["wg"], s["wu"], s["wd"], s["g"], s["u"],
                                     act=c["act"])
    if op == "ce":
        return tw.linear_ce(s["x"], s["w"], s["target"])
    if op == "ce_bwd":
        return tw.linear_ce_backward(s["dloss"], s["x"], s["w"], s["target"], s["lse"])
    norm = tw.clip_grads(s["grads"], s["most"], out=s["out"])
    return {"norm": norm, "out": s["flat"]}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------- exact --
def exact(case, seed):
    """The operators' definition in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        wide = [t.to(torch.float64) for t in s["grads"]]
        total = sum(torch.dot(t.flatten(), t.flatten()) for t in wide)
        norm = total.sqrt()
        factor = torch.minimum(s["most"] / (norm + 1e-6), torch.ones_like(norm))
        return {"norm": norm, "out": torch.cat([t.flatten() for t in wide]).mul_(factor)}
    f = {k: v.to(torch.float64) for k, v in s.items() if isinstance(v, torch.Tensor) and k != "target"}
    K = case["K"]
    if op == "rms":
        z = f["x"] + f["add"] if "add" in f else f["x"]
        r = (torch.linalg.vector_norm(z, dim=1).square() / K + EPS).rsqrt()
        y = torch.einsum("mk,m,k->mk", z, r, f["gamma"])
        if case["y"] == "int8":
            step = y.abs().max(dim=1).values / 127.0
            q = torch.round(y / step.clamp(min=1e-300).unsqueeze(1))
            live = step * 127.0 >= TINY
            out = {"values": torch.where(live.unsqueeze(1), q * step.unsqueeze(1), 0.0),
                   "scale": torch.where(live, step, 0.0)}
        else:
            out = {"y": y, "rstd": r}
        return {**out, "sum": z} if "add" in f else out
    if op == "rms_bwd":
        # through y = z r gamma with r = rstd: dr/dz = -z r^3 / K
        r = f["rstd"].unsqueeze(1)
        dg = f["dy"] * f["gamma"]
        dr = (dg * f["x"]).sum(dim=1, keepdim=True)
        dx = dg * r - f["x"] * r.pow(3) * dr / K + f.get("res", 0.0)
        return {"dx": dx, "dgamma": (f["dy"] * f["x"] * r).sum(dim=0)}

    def product(a, b):  # a b^T
        return torch.matmul(a, b.t().contiguous())

    def act(v):
        if case["act"] == "relu":
            return torch.relu(v)
        if case["act"] == "silu":
            return v * torch.sigmoid(v)
        return torch.nn.functional.gelu(v, approximate="tanh")

    if op == "ffn":
        g, u = product(f["x"], f["wg"]), product(f["x"], f["wu"])
        y = torch.matmul(act(g) * u, f["wd"])
        return {"y": y, "g": g, "u": u} if case["keep"] else {"y": y}
    if op == "ffn_bwd":
        g = f["g"].requires_grad_()
        a = act(g)
        da, = torch.autograd.grad(a.sum(), g)
        a = a.detach()
        dh = product(f["dy"], f["wd"])
        dz, du = dh * f["u"] * da, dh * a
        t = [v.t().contiguous() for v in (dz, du, a * f["u"])]
        return {"dx": torch.matmul(dz, f["wg"]).add_(torch.matmul(du, f["wu"])),
                "dwg_t": torch.matmul(t[0], f["x"]), "dwu_t": torch.matmul(t[1], f["x"]),
                "dwd": torch.matmul(t[2], f["dy"])}
    logits = product(f["x"], f["w"])
    t = s["target"]
    if op == "ce":
        logp = torch.log_softmax(logits, dim=1)
        loss = torch.nn.functional.nll_loss(logp, t, ignore_index=-100, reduction="none")
        return {"loss": loss, "lse": torch.logsumexp(logits, dim=1)}
    p = logits.sub_(f["lse"].unsqueeze(1)).exp_()
    keep = (t != -100).to(torch.float64)
    p.scatter_add_(1, t.clamp(min=0).unsqueeze(1), -torch.ones_like(keep).unsqueeze(1))
    p.mul_((keep * f["dloss"]).unsqueeze(1))
    return {"dx": torch.matmul(p, f["w"]), "dw": torch.matmul(p.t().contiguous(), f["x"])}
