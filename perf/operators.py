"""Measured cases of the operators around the sketched layers: checkpoints in 8 bits, norms, cross entropy.

Three sets, as one fine-tuning step uses them together (plus their forms for a few tokens):

* ``ckpt``  activations kept for the backward pass as 8-bit codes with a power-of-two scale per 32 columns,
  read back, and the table gradient of a sketched layer taken from them;
* ``norm``  layer norm and root-mean-square norm in front of a sketched layer, forward and backward, the
  forward also writing the layer's 8-bit checkpoint;
* ``xent``  softmax cross entropy of a sketched vocabulary projection that never keeps its logits: loss and
  log-sum-exp per token, gradients of the hidden states and of the tables.

``own`` chooses between elementary torch operations in 32 bits (False) and this repository's kernels (True).
"""
import math

import torch

own = False

_T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
_IGNORE = -100


def _skm():
    import lut_sketched_matmul_amd
    return lut_sketched_matmul_amd


# ---------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one batch of 16 tokens of a 4096-wide layer written and read back: latency
        dict(name="ckpt_roundtrip_m16", op="ckpt", m=16, d=4096, x="f16"),
        # the largest activation of a 7B layer's step: the input of its down projection, 8192 tokens
        dict(name="ckpt_roundtrip_m8192", op="ckpt", m=8192, d=11008, x="bf16"),
        # both gradients of a 4096 x 4096 projection from its checkpoint, a short ragged batch
        dict(name="ckpt_bwd_m1000", op="ckpt_bwd", m=1000, n=4096, d=4096, b=3, gpr=8, x="f16", lut="f16", dx=True),
        # the table gradient of the 7B down projection at a training step's 8192 tokens
        dict(name="ckpt_dlut_m8192", op="ckpt_bwd", m=8192, n=4096, d=11008, b=4, gpr=8, x="bf16", lut="f16", dx=False),
        # the norm in front of one token's projection (decode)
        dict(name="norm_fwd_m1", op="norm_fwd", m=1, d=4096, x="f16", kind="rms", bias=False, ckpt=False),
        # forward with the checkpoint written along, 8192 tokens of a 4096-wide layer
        dict(name="norm_fwd_ckpt_m8192", op="norm_fwd", m=8192, d=4096, x="bf16", kind="rms", bias=False, ckpt=True),
        # backward of a layer norm with weight and bias gradients, its incoming gradient in fp32
        dict(name="norm_bwd_m8192", op="norm_bwd", m=8192, d=4096, x="bf16", kind="layer", bias=True, dy="f32"),
        # odd sizes: rows that are not a whole number of vectors
        dict(name="norm_bwd_odd", op="norm_bwd", m=777, d=1001, x="f16", kind="layer", bias=True, dy="f16"),
        # scoring four tokens against a 32000-word vocabulary (decode-sized)
        dict(name="xent_fwd_m4", op="xent_fwd", m=4, V=32000, d=4096, b=4, gpr=8, x="f16", lut="f16", prompt=0.0, seq=4),
        # evaluation loss of 2001 tokens, no gradients
        dict(name="xent_fwd_m2001", op="xent_fwd", m=2001, V=32000, d=4096, b=4, gpr=8, x="bf16", lut="f16",
             prompt=0.0, seq=2001),
        # a frozen head over a large vocabulary: hidden-state gradient only
        dict(name="xent_bwd_frozen_m2048", op="xent_bwd", m=2048, V=128256, d=4096, b=4, gpr=4, x="bf16", lut="bf16",
             prompt=0.0, seq=2048, dlut=False),
        # one training step of a trained head, sequences of 1024 whose first quarter (the prompt) is not scored
        dict(name="xent_train_m4096", op="xent_train", m=4096, V=32000, d=4096, b=4, gpr=8, x="f16", lut="f16",
             prompt=0.25, seq=1024, dlut=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ckpt", "ckpt_bwd", "norm_fwd", "norm_bwd", "xent_fwd", "xent_bwd", "xent_train"])
    x = rng.choice(["f16", "bf16"])
    if op == "ckpt":
        return dict(op=op, m=_log(rng, 1, 8192), d=32 * _log(rng, 2, 344), x=x)
    if op == "norm_fwd":
        kind = rng.choice(["rms", "layer"])
        ckpt = rng.random() < 0.5
        d = 32 * _log(rng, 2, 172) if ckpt else _log(rng, 64, 5504)
        return dict(op=op, m=_log(rng, 1, 8192), d=d, x=x, kind=kind, bias=kind == "layer", ckpt=ckpt)
    if op == "norm_bwd":
        kind = rng.choice(["rms", "layer"])
        return dict(op=op, m=_log(rng, 1, 8192), d=_log(rng, 64, 4096), x=x, kind=kind, bias=kind == "layer",
                    dy=rng.choice(["f32", x]))
    b, gpr = rng.choice([2, 3, 4]), rng.choice([1, 2, 4, 8])
    d = 32 * gpr * max(1, _log(rng, 256, 4096) // (32 * gpr))
    lut = "f16" if x == "f16" else rng.choice(["f16", "bf16"])
    if op == "ckpt_bwd":
        return dict(op=op, m=_log(rng, 1, 8192), n=_log(rng, 128, 8192), d=d, b=b, gpr=gpr, x=x, lut=lut,
                    dx=rng.random() < 0.5)
    m = _log(rng, 1, 4096)
    c = dict(op=op, m=m, V=_log(rng, 500, 64000), d=d, b=b, gpr=gpr, x=x, lut=lut,
             prompt=rng.choice([0.0, 0.3]), seq=max(2, m // 2))
    if op != "xent_fwd":
        c["dlut"] = rng.random() < 0.5
    if m * c["V"] > 4096 * 32000:
        c["V"] = 4096 * 32000 // m
    return c


def _scored(c):
    """Tokens with a target: all but the first `prompt` share of every sequence of `seq` tokens."""
    skip = int(c["prompt"] * c["seq"])
    return sum(1 for t in range(c["m"]) if t % c["seq"] >= skip)


def work(case):
    c, op = case, case["op"]
    m, d = c["m"], c["d"]
    xb = _BYTES[c["x"]]
    if op == "ckpt":  # X in, codes and scales out and in again, values out
        return {"bytes": m * d * (2 * xb + 2 + 2 / 32), "flops": 4.0 * m * d}
    if op == "norm_fwd":
        b = m * d * 2 * xb + 8 * m + 4 * d * (2 if c["bias"] else 1)
        if c["ckpt"]:  # codes and scales out, then read back as values
            b += m * d * (2 + 2 / 32 + xb)
        return {"bytes": b, "flops": 8.0 * m * d}
    if op == "norm_bwd":
        return {"bytes": m * d * (2 * xb + _BYTES[c["dy"]]) + 8 * m + 4 * d * (3 if c["bias"] else 2), "flops": 12.0 * m * d}
    b, gpr = c["b"], c["gpr"]
    rows = c["n"] if op == "ckpt_bwd" else c["V"]
    tables = rows * gpr * (1 << b)
    weights = rows * d * b / 8 + 2 * tables
    if op == "ckpt_bwd":
        byt = m * rows * xb + m * d * (1 + 1 / 32) + rows * d * b / 8 + 4 * tables
        if c["dx"]:
            byt += 2 * tables + 4 * m * d
        return {"bytes": byt, "flops": 2.0 * m * rows * d * (2 if c["dx"] else 1)}
    k = _scored(c)
    gemm = 2.0 * k * rows * d
    if op == "xent_fwd":
        return {"bytes": k * d * xb + weights + 16 * m, "flops": gemm}
    byt = k * d * xb + m * d * xb + weights + 20 * m + (4 * tables if c["dlut"] else 0)
    return {"bytes": byt, "flops": gemm * (3 if c["dlut"] else 2)}


# --------------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, sigma, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)


def _sketch(g, n, d, b, gpr, dtype):
    idx = torch.randint(0, 256, (n, d * b // 8), generator=g, device="cuda", dtype=torch.uint8)
    lut = torch.sort(torch.randn((n, gpr, 1 << b), generator=g, device="cuda") * 0.02, dim=-1).values.to(dtype)
    return idx, lut


def _activations(g, m, d, dtype):
    """Rows of different scale with a few large columns, as the inputs of a layer have them."""
    x = torch.randn((m, d), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((m, 1), generator=g, device="cuda"))
    x[:, :: max(1, d // 7)] *= 8.0
    return x.to(dtype)


def prepare(case, seed):
    c, op, g = case, case["op"], _gen(seed)
    m, d, x = c["m"], c["d"], _T[c["x"]]
    s = dict(c)
    if op == "ckpt":
        s["X"] = _activations(g, m, d, x)
        return s
    if op in ("norm_fwd", "norm_bwd"):
        s["X"] = (_activations(g, m, d, torch.float32) + 0.3).to(x)
        s["w"] = 1.0 + 0.2 * torch.randn(d, generator=g, device="cuda")
        s["bias_"] = 0.1 * torch.randn(d, generator=g, device="cuda") if c["bias"] else None
        if op == "norm_bwd":
            s["dY"] = _normal(g, (m, d), 0.01, _T[c["dy"]])
            mean, rstd = _norm_stats(s["X"].float(), c["kind"])
            s["mean"] = mean.reshape(-1).contiguous() if mean is not None else None
            s["rstd"] = rstd.reshape(-1).contiguous()
        return s
    if op == "ckpt_bwd":
        s["idx"], s["lut_"] = _sketch(g, c["n"], d, c["b"], c["gpr"], _T[c["lut"]])
        s["dY"] = _normal(g, (m, c["n"]), 0.01, x)
        s["codes"], s["scales"] = _quantise(_activations(g, m, d, x))
        return s
    s["idx"], s["lut_"] = _sketch(g, c["V"], d, c["b"], c["gpr"], _T[c["lut"]])
    scale = torch.where(torch.rand((m, 1), generator=g, device="cuda") < 0.5, 1.0, 2.5)
    s["X"] = (torch.randn((m, d), generator=g, device="cuda") * scale).to(x)
    t = torch.randint(0, c["V"], (m,), generator=g, device="cuda")
    pos = torch.arange(m, device="cuda") % c["seq"]
    s["targets"] = torch.where(pos < int(c["prompt"] * c["seq"]), _IGNORE, t)
    # gradient of the mean loss; f16 steps scale their loss so that gradients stay in f16's normal range
    s["dloss"] = torch.full((m,), (4096.0 if c["x"] == "f16" else 1.0) / max(1, _scored(c)), device="cuda")
    if op == "xent_bwd":
        s["lse"] = torch.logsumexp(s["X"].float() @ _weights(s, c["V"]).T, dim=1)
    return s


# ----------------------------------------------------------------------------------------------- plain forms

def _quantise(X):
    """int8 codes q and biased exponents s per 32 columns: q 2^(s - 127), the smallest step that reaches the
    block's largest magnitude with 127 (bounded so that every value is a finite number of X's type)."""
    lo, hi = (-24, 9) if X.dtype == torch.float16 else (-126, 121)
    v = X.float().reshape(X.shape[0], -1, 32)
    top = v.abs().amax(2, keepdim=True)
    _, e = torch.frexp(top / 127.0)
    e = torch.where(torch.ldexp(torch.full_like(top, 127.0), e - 1) >= top, e - 1, e)
    e = torch.where(top > 0, e, lo).clamp(lo, hi)
    q = torch.round(torch.ldexp(v, -e)).clamp(-127, 127)
    return q.reshape(X.shape).to(torch.int8), (e + 127).reshape(X.shape[0], -1).to(torch.uint8)


def _values(codes, scales):
    q = codes.float().reshape(codes.shape[0], -1, 32)
    return torch.ldexp(q, scales.int()[..., None] - 127).reshape(codes.shape)


def _norm_stats(x, kind, eps=1e-5):
    if kind == "layer":
        mean = x.mean(1, keepdim=True)
        return mean, torch.rsqrt((x - mean).square().mean(1, keepdim=True) + eps)
    return None, torch.rsqrt(x.square().mean(1, keepdim=True) + eps)


def _codes(idx, d, b):
    """The b-bit indices of every row, [n, d] int64."""
    n = idx.shape[0]
    if b == 3:
        w = idx.reshape(n, -1, 3).int()
        w = w[..., 0] | (w[..., 1] << 8) | (w[..., 2] << 16)
        f = (w[..., None] >> (3 * torch.arange(8, device=idx.device, dtype=torch.int32))) & 7
    else:
        f = (idx[..., None] >> (b * torch.arange(8 // b, device=idx.device, dtype=torch.uint8))) & ((1 << b) - 1)
    return f.reshape(n, d).long()


def _weights(s, n):
    c = _codes(s["idx"], s["d"], s["b"]).reshape(n, s["gpr"], -1)
    return s["lut_"].float().gather(2, c).reshape(n, s["d"])


def _bins(dW, s, n):
    """Sums of a weight gradient over the columns that share a table entry."""
    c = _codes(s["idx"], s["d"], s["b"]).reshape(n, s["gpr"], -1)
    return torch.zeros((n, s["gpr"], 1 << s["b"]), device=dW.device).scatter_add_(2, c, dW.reshape(c.shape))


def _plain(s):
    op = s["op"]
    if op == "ckpt":
        return {"values": _values(*_quantise(s["X"])).to(s["X"].dtype)}
    if op == "norm_fwd":
        x = s["X"].float()
        mean, rstd = _norm_stats(x, s["kind"])
        y = (x if mean is None else x - mean) * rstd * s["w"]
        y = (y if s["bias_"] is None else y + s["bias_"]).to(s["X"].dtype)
        out = {"y": y, "rstd": rstd.reshape(-1)}
        if mean is not None:
            out["mean"] = mean.reshape(-1)
        if s["ckpt"]:
            out["values"] = _values(*_quantise(y)).to(y.dtype)
        return out
    if op == "norm_bwd":
        x, dy, rstd = s["X"].float(), s["dY"].float(), s["rstd"][:, None]
        xh = (x if s["mean"] is None else x - s["mean"][:, None]) * rstd
        gw = dy * s["w"]
        t = gw - xh * (gw * xh).mean(1, keepdim=True)
        dx = rstd * (t if s["mean"] is None else t - gw.mean(1, keepdim=True))
        out = {"dX": dx.to(s["X"].dtype), "dw": (dy * xh).sum(0)}
        if s["bias_"] is not None:
            out["db"] = dy.sum(0)
        return out
    if op == "ckpt_bwd":
        dy, xv = s["dY"].float(), _values(s["codes"], s["scales"])
        out = {"dLUT": _bins(dy.T @ xv, s, s["n"])}
        if s["dx"]:
            out["dX"] = dy @ _weights(s, s["n"])
        return out
    V = s["V"]
    x, W = s["X"].float(), _weights(s, V)
    logits = x @ W.T
    t = s["targets"]
    live = t != _IGNORE
    at = torch.where(live, t, 0)[:, None]
    out = {}
    if op == "xent_bwd":
        lse = s["lse"]
    else:
        top = logits.amax(1, keepdim=True)
        lse = (top + torch.log(torch.exp(logits - top).sum(1, keepdim=True))).reshape(-1)
        out["lse"] = torch.where(live, lse, 0.0)
        out["loss"] = torch.where(live, lse - logits.gather(1, at).reshape(-1), 0.0)
    if op != "xent_fwd":
        g = torch.exp(logits - lse[:, None])
        g.scatter_add_(1, at, torch.full_like(at, -1, dtype=torch.float32))
        g = g * torch.where(live, s["dloss"], 0.0)[:, None]
        out["dX"] = (g @ W).to(s["X"].dtype)
        if s["dlut"]:
            out["dLUT"] = _bins(g.T @ x, s, V)
    return out


# ------------------------------------------------------------------------------------ this repository's calls

def _own(s):
    skm, op = _skm(), s["op"]
    if op == "ckpt":
        codes, scales = skm.sketch_act_quant(s["X"])
        return {"values": skm.sketch_act_dequant(codes, scales, s["X"].dtype)}
    if op == "norm_fwd":
        y, mean, rstd, codes, scales = skm.sketch_norm_fwd(s["X"], s["w"], s["bias_"], kind=s["kind"], eps=1e-5,
                                                           checkpoint=s["ckpt"])
        out = {"y": y, "rstd": rstd}
        if mean is not None:
            out["mean"] = mean
        if s["ckpt"]:
            out["values"] = skm.sketch_act_dequant(codes, scales, y.dtype)
        return out
    if op == "norm_bwd":
        dX, dw, db = skm.sketch_norm_bwd(s["dY"], s["X"], s["w"], s["mean"], s["rstd"], kind=s["kind"],
                                         need_db=s["bias_"] is not None)
        out = {"dX": dX, "dw": dw}
        if db is not None:
            out["db"] = db
        return out
    if op == "ckpt_bwd":
        dX, dLUT = skm.sketch_matmul_bwd_ckpt(s["dY"], s["codes"], s["scales"], s["idx"], s["lut_"], s["b"], s["gpr"],
                                              need_dx=s["dx"])
        return {"dLUT": dLUT, "dX": dX} if s["dx"] else {"dLUT": dLUT}
    out = {}
    lse = s.get("lse")
    if op != "xent_bwd":
        loss, lse = skm.sketch_xent_fwd(s["X"], s["idx"], s["lut_"], s["targets"], s["b"], s["gpr"], ignore_index=_IGNORE)
        out.update(lse=lse, loss=loss)
    if op != "xent_fwd":
        dX, dLUT = skm.sketch_xent_bwd(s["X"], s["idx"], s["lut_"], s["targets"], lse, s["dloss"], s["b"], s["gpr"],
                                       ignore_index=_IGNORE, need_dlut=s["dlut"])
        out["dX"] = dX
        if s["dlut"]:
            out["dLUT"] = dLUT
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------- in 64 bits

def _w64(s, n):
    """Dense weights from the bit stream's definition: index j sits at bits b j .. b j + b - 1 of its row."""
    d, b = s["d"], s["b"]
    idx = s["idx"].long()
    p = b * torch.arange(d, device=idx.device)
    lo = idx[:, p >> 3]
    hi = idx[:, torch.clamp((p >> 3) + 1, max=idx.shape[1] - 1)]
    code = ((lo + 256 * hi) >> (p & 7)) % (1 << b)
    group = torch.arange(d, device=idx.device) // (d // s["gpr"])
    return code, s["lut_"].double()[torch.arange(n, device=idx.device)[:, None], group[None, :], code]


def _bins64(dW, code, s):
    n, K = dW.shape[0], 1 << s["b"]
    code, dW = code.reshape(n, s["gpr"], -1), dW.reshape(n, s["gpr"], -1)
    return torch.stack([torch.where(code == k, dW, 0.0).sum(2) for k in range(K)], dim=2)


def _grid64(v, dtype):
    """v (exact numbers of `dtype`) on the 8-bit grid of its 32-column block."""
    lo, hi = (-24, 9) if dtype == torch.float16 else (-126, 121)
    b = v.double().reshape(v.shape[0], -1, 32)
    top = b.abs().amax(2, keepdim=True)
    e = torch.ceil(torch.log2(torch.clamp(top, min=2.0 ** -140) / 127.0)).clamp(lo, hi)
    step = torch.exp2(e)
    return ((b / step).round().clamp(-127, 127) * step).reshape(v.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "ckpt":
        return {"values": _grid64(s["X"], s["X"].dtype)}
    if op in ("norm_fwd", "norm_bwd"):
        x, w, n = s["X"].double(), s["w"].double(), s["d"]
        if op == "norm_fwd":
            mean = x.sum(1) / n if s["kind"] == "layer" else torch.zeros_like(x[:, 0])
            rstd = 1.0 / torch.sqrt(((x - mean[:, None]) ** 2).sum(1) / n + 1e-5)
            y = (x - mean[:, None]) * rstd[:, None] * w
            if s["bias_"] is not None:
                y = y + s["bias_"].double()
            out = {"y": y, "rstd": rstd}
            if s["kind"] == "layer":
                out["mean"] = mean
            if s["ckpt"]:
                out["values"] = _grid64(y.to(s["X"].dtype), s["X"].dtype)
            return out
        dy, r = s["dY"].double(), s["rstd"].double()[:, None]
        xh = (x - (s["mean"].double()[:, None] if s["mean"] is not None else 0.0)) * r
        a = dy * w
        dx = a - xh * ((a * xh).sum(1, keepdim=True) / n)
        if s["kind"] == "layer":
            dx = dx - a.sum(1, keepdim=True) / n
        out = {"dX": dx * r, "dw": (dy * xh).sum(0)}
        if s["bias_"] is not None:
            out["db"] = dy.sum(0)
        return out
    if op == "ckpt_bwd":
        code, W = _w64(s, s["n"])
        dy = s["dY"].double()
        q = s["codes"].double().reshape(s["m"], -1, 32) * torch.exp2(s["scales"].double() - 127.0)[..., None]
        out = {"dLUT": _bins64(dy.T.contiguous() @ q.reshape(s["m"], -1), code, s)}
        if s["dx"]:
            out["dX"] = dy @ W
        return out
    code, W = _w64(s, s["V"])
    x, t = s["X"].double(), s["targets"]
    live = t != _IGNORE
    z = x @ W.T
    out = {}
    if op == "xent_bwd":
        lse = s["lse"].double()
    else:
        lse = torch.logsumexp(z, dim=1)
        zt = z[torch.arange(s["m"], device=z.device), torch.where(live, t, 0)]
        out["lse"] = torch.where(live, lse, 0.0)
        out["loss"] = torch.where(live, lse - zt, 0.0)
    if op != "xent_fwd":
        g = torch.exp(z - lse[:, None])
        g[torch.arange(s["m"], device=z.device), torch.where(live, t, 0)] -= 1.0
        g *= torch.where(live, s["dloss"].double(), 0.0)[:, None]
        out["dX"] = g @ W
        if s["dlut"]:
            out["dLUT"] = _bins64(g.T.contiguous() @ x, code, s)
    return out
