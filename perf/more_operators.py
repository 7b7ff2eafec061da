"""Measured cases of the operators at a sketched projection's output: low-rank adapters, dropout, head rotation.

Three operators, as one attention layer of a fine-tuned model uses them on its sketched q/k/v projection:

* ``adapter`` low-rank adapters of many requests beside one shared projection: every token names the adapter whose
  product is added to the projection's output; in training with dropout in front and all gradients;
* ``dropout`` dropout (with the residual it is added to) whose mask comes from a counter and is never stored;
* ``rotary``  norms of the query and key heads and their position rotation in one pass, forward and backward, on the
  heads where the joined q/k/v projection leaves them.

``own`` chooses between elementary torch operations in 32 bits (False) and this repository's kernels (True).
"""
import math

import numpy as np
import torch

own = False

_T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2}
_EPS = 1e-6


def _skm():
    import lut_sketched_matmul_amd
    return lut_sketched_matmul_amd


# ---------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # the inputs of 16 tokens of a 4096-wide layer: latency
        dict(name="dropout_m16", op="dropout", m=16, d=4096, x="bf16", p=0.1, residual=False, grad=False),
        # the block output of a 7B training step (8192 tokens) dropped and added to its residual, and its gradient
        dict(name="dropout_residual_m8192", op="dropout", m=8192, d=4096, x="bf16", p=0.1, residual=True, grad=True),
        # an odd number of fp32 values
        dict(name="dropout_odd", op="dropout", m=2001, d=4097, x="f32", p=0.5, residual=False, grad=False),
        # one request's token with its adapter beside a 7B attention projection (decode): latency
        dict(name="adapter_m1", op="adapter", m=1, d=4096, n=4096, r=16, S=8, x="f16", kind="mixed"),
        # a decode batch of 64 requests over 64 adapters beside the 7B gate projection
        dict(name="adapter_m64_s64", op="adapter", m=64, d=4096, n=11008, r=16, S=64, x="bf16", kind="mixed"),
        # a 70B MLP prefill of 2048 tokens: requests of ragged lengths, 8 adapters of rank 64, some requests with none
        dict(name="adapter_prefill_m2048", op="adapter", m=2048, d=8192, n=28672, r=64, S=8, x="bf16", kind="ragged"),
        # a training step of one adapter on a 7B attention projection, dropout in front, all gradients
        dict(name="adapter_train_m8192", op="adapter_train", m=8192, d=4096, n=4096, r=16, S=1, x="bf16", kind="one", p=0.05),
        # five tasks' adapters trained in one ragged batch; odd token count, width and rank
        dict(name="adapter_train_odd", op="adapter_train", m=4001, d=4096, n=4095, r=12, S=5, x="f16", kind="ragged", p=0.0),
        # one token's 32 query and 8 key heads (decode): latency
        dict(name="rotary_m1", op="rotary", m=1, hq=32, hk=8, dh=128, rot=128, x="f16", norm=True, pairs="halves", far=5000),
        # a prefill of 8192 tokens at far positions, 64 query and 8 key heads
        dict(name="rotary_m8192", op="rotary", m=8192, hq=64, hk=8, dh=128, rot=128, x="bf16", norm=True, pairs="halves",
             far=131072),
        # a training step's 4096 tokens with 32 + 32 heads: outputs, gradients of heads and of both norms' weights
        dict(name="rotary_train_m4096", op="rotary_train", m=4096, hq=32, hk=32, dh=128, rot=128, x="f16", norm=True,
             pairs="halves", far=0),
        # partly rotated fp32 heads of 80 with neighbouring pairs, no norm; a ragged token count
        dict(name="rotary_train_odd", op="rotary_train", m=777, hq=6, hk=2, dh=80, rot=36, x="f32", norm=False,
             pairs="neighbours", far=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    c = _draw(rng)
    while work(c)["bytes"] > 500e6 or work(c)["flops"] > 9e9:
        c["m"] = max(1, c["m"] * 2 // 3)
    return c


def _draw(rng):
    op = rng.choice(["dropout", "adapter", "adapter", "adapter_train", "adapter_train", "rotary", "rotary_train"])
    if op == "dropout":
        m = _log(rng, 1, 8192)
        return dict(op=op, m=m, d=min(_log(rng, 32, 16384), 8192 * 4096 // m), x=rng.choice(["f16", "bf16", "f32"]),
                    p=rng.choice([0.05, 0.1, 0.5, round(rng.uniform(0.0, 0.9), 3)]), residual=rng.random() < 0.5,
                    grad=rng.random() < 0.5)
    if op in ("adapter", "adapter_train"):
        kind = rng.choice(["one", "ragged", "mixed"])
        m = _log(rng, 1, 8192)
        d, n = 32 * _log(rng, 8, 256), _log(rng, 64, 28672)
        if m * (d + n) > 8192 * 8192:
            n = max(64, 8192 * 8192 // m - d)
        S = 1 if kind == "one" else _log(rng, 1, 64)
        r = rng.choice([4, 8, 16, 16, 32, 64, rng.randint(1, 64)])
        c = dict(op=op, m=m, d=d, n=n, r=r, S=S, x=rng.choice(["f16", "bf16"]), kind=kind)
        if op == "adapter_train":
            c["p"] = rng.choice([0.0, 0.05, 0.1])
        return c
    dh = rng.choice([64, 128, 128, 256, 2 * _log(rng, 8, 128)])
    hq = rng.choice([1, 8, 32, 40, 64, rng.randint(1, 64)])
    hk = rng.choice([hq, max(1, hq // 4), max(1, hq // 8)])
    return dict(op=op, m=_log(rng, 1, 8192), hq=hq, hk=hk, dh=dh, rot=rng.choice([dh, dh, 2 * max(1, dh // 4)]),
                x=rng.choice(["f16", "bf16", "f32"]), norm=rng.random() < 0.6, pairs=rng.choice(["halves", "neighbours"]),
                far=rng.choice([0, 4096, 131072]))


def work(case):
    c, op = case, case["op"]
    xb, m = _BYTES[c["x"]], c["m"]
    if op == "dropout":  # values in, values out (and the residual in; and the same for the gradient)
        count = m * c["d"]
        passes = 2 + (1 if c["residual"] else 0) + (2 if c["grad"] else 0)
        return {"bytes": count * xb * passes, "flops": count * (2.0 if c["grad"] else 1.0)}
    if op in ("adapter", "adapter_train"):
        d, n, r = c["d"], c["n"], c["r"]
        weights = min(c["S"], m) * r * (d + n) * xb
        byt = m * (d + 2 * n) * xb + weights  # X, the projection's output in and out
        flops = 2.0 * m * r * (d + n)
        if op == "adapter_train":  # dY and X once each for the gradients, dX from fp32 to X's type, dA and dB in fp32
            byt += m * (n + d) * xb + m * d * (4 + xb) + c["S"] * r * (d + n) * 4 + weights
            flops *= 3.0
        return {"bytes": byt, "flops": flops}
    rows = m * (c["hq"] + c["hk"]) * c["dh"]
    if op == "rotary":
        return {"bytes": 2 * rows * xb + 8 * m, "flops": rows * (7.0 if c["norm"] else 3.0)}
    # heads in and out; their gradients in and out, and with a norm the heads once more
    return {"bytes": rows * xb * (5 if c["norm"] else 4) + 8 * m, "flops": rows * (20.0 if c["norm"] else 6.0)}


# --------------------------------------------------------------------------------------------------- inputs

def _normal(g, shape, sigma, dtype):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(dtype)


def _activations(g, m, d, dtype):
    """Rows of different scale with a few large columns, as the inputs of a layer have them."""
    x = torch.randn((m, d), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((m, 1), generator=g, device="cuda"))
    x[:, :: max(1, d // 7)] *= 8.0
    return x.to(dtype)


def _requests(rng, m, S, kind):
    """The adapter of every token: requests of ragged lengths one after the other, or one token each; -1 is none."""
    if kind == "mixed":
        ids = rng.integers(-1 if m > 1 else 0, S, m)
    else:
        cuts = np.sort(rng.integers(0, m + 1, max(2, S)))
        ids = rng.integers(-1, S, cuts.size + 1)[np.searchsorted(cuts, np.arange(m), side="right")]
    return torch.from_numpy(ids.astype(np.int32)).to("cuda")


def prepare(case, seed):
    c, op = case, case["op"]
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    rng = np.random.default_rng(int(seed) % (1 << 63))
    m, x = c["m"], _T[c["x"]]
    s = dict(c)
    # the dropout's key and stream number, on the GPU so that a captured step can move on
    s["seed_"] = torch.from_numpy(rng.integers(0, 1 << 62, 2)).to("cuda")
    if op == "dropout":
        s["X"] = _activations(g, m, c["d"], x)
        s["res"] = _activations(g, m, c["d"], x) if c["residual"] else None
        s["dY"] = _normal(g, (m, c["d"]), 0.01, x) if c["grad"] else None
        return s
    if op in ("adapter", "adapter_train"):
        d, n, r, S = c["d"], c["n"], c["r"], c["S"]
        s["X"] = _activations(g, m, d, x)
        s["A"] = _normal(g, (S, r, d), 1.0 / math.sqrt(d), x)
        s["B"] = _normal(g, (S, n, r), 0.05, x)
        s["base"] = _normal(g, (m, n), 1.0, x)
        s["ids"] = None if c["kind"] == "one" else _requests(rng, m, S, c["kind"])
        s["scale"] = (0.5 + 1.5 * torch.rand(S, generator=g, device="cuda"))
        if op == "adapter_train":
            s["dY"] = _normal(g, (m, n), 0.01, x)
            s["base_dx"] = _normal(g, (m, d), 0.01, torch.float32)
        return s
    hq, hk, dh = c["hq"], c["hk"], c["dh"]
    # q, k and v side by side, as one projection of all three writes them
    s["qkv"] = _activations(g, m, (hq + 2 * hk) * dh, x)
    s["q"] = s["qkv"][:, :hq * dh].unflatten(1, (hq, dh))
    s["k"] = s["qkv"][:, hq * dh:(hq + hk) * dh].unflatten(1, (hk, dh))
    start = rng.integers(0, c["far"] + 1, 4)
    s["pos"] = torch.from_numpy(start[np.arange(m) * 4 // m] + np.arange(m) % (m // 4 + 1)).to("cuda")
    s["inv_freq"] = 10000.0 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"])
    s["qw"] = s["kw"] = None
    if c["norm"]:
        s["qw"] = 1.0 + 0.2 * torch.randn(dh, generator=g, device="cuda")
        s["kw"] = 1.0 + 0.2 * torch.randn(dh, generator=g, device="cuda")
    if op == "rotary_train":
        s["dq"] = _normal(g, (m, hq, dh), 0.01, x)
        s["dk"] = _normal(g, (m, hk, dh), 0.01, x)
    return s


# ----------------------------------------------------------------------------------------------- plain forms

_M32 = 0xFFFFFFFF


def _keep(count, seed, p):
    """Which of `count` values stay: 16 random bits each, eight to a call of Philox4x32-10 (Salmon et al., 2011)
    with the key seed[0] and the counter (number of the eight, seed[1])."""
    block = torch.arange((count + 7) // 8, device=seed.device)
    x = [block & _M32, block >> 32, (seed[1] & _M32).expand_as(block), ((seed[1] >> 32) & _M32).expand_as(block)]
    k0, k1 = seed[0] & _M32, (seed[0] >> 32) & _M32
    for _ in range(10):
        a, b = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57  # (the low 64 bits, whatever the sign)
        x = [((b >> 32) & _M32) ^ x[1] ^ k0, b & _M32, ((a >> 32) & _M32) ^ x[3] ^ k1, a & _M32]
        k0, k1 = (k0 + 0x9E3779B9) & _M32, (k1 + 0xBB67AE85) & _M32
    u = torch.stack([h for w in x for h in (w & 0xFFFF, w >> 16)], dim=1).reshape(-1)[:count]
    return u >= _threshold(p)


def _threshold(p):
    return int(round(p * 65536))


def _dropped(x, seed, p):
    """fp32: values that stay, divided by the share that does; zeros elsewhere."""
    stay = (65536 - _threshold(p)) / 65536
    return torch.where(_keep(x.numel(), seed, p).reshape(x.shape), x.float() / stay, 0.0)


def _rows_of(s):
    """(adapter, its tokens) for every adapter that has any."""
    if s["ids"] is None:
        return [(0, slice(None))]
    found = [(a, torch.nonzero(s["ids"] == a).reshape(-1)) for a in range(s["S"])]
    return [(a, t) for a, t in found if t.numel()]


def _adapter(s):
    train = s["op"] == "adapter_train"
    x = _dropped(s["X"], s["seed_"], s["p"]) if train and s["p"] else s["X"].float()
    y = s["base"].float()
    A, B = s["A"].float(), s["B"].float()
    if train:
        dy, dx = s["dY"].float(), torch.zeros_like(x)
        dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    for a, t in _rows_of(s):
        h = x[t] @ A[a].T
        y[t] += s["scale"][a] * (h @ B[a].T)
        if train:
            g = dy[t] * s["scale"][a]
            dh = g @ B[a]
            dB[a] = g.T @ h
            dA[a] = dh.T @ x[t]
            dx[t] = dh @ A[a]
    out = {"Y": y.to(s["base"].dtype)}
    if train:
        if s["p"]:
            dx = _dropped(dx, s["seed_"], s["p"])
        out.update(dX=(s["base_dx"] + dx).to(s["X"].dtype), dA=dA, dB=dB)
    return out


def _turned(x, cos, sin, pairs):
    """Heads x [m, h, dh] with the pairs of their first columns turned by the angles, [m, rot / 2]."""
    rot = 2 * cos.shape[1]
    c, s = cos[:, None], sin[:, None]
    if pairs == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        return torch.cat([a * c - b * s, a * s + b * c, x[..., rot:]], dim=2)
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    return torch.cat([torch.stack([a * c - b * s, a * s + b * c], dim=3).flatten(2), x[..., rot:]], dim=2)


def _rotary(s):
    angle = s["pos"].double()[:, None] * s["inv_freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    out = {}
    for name, x, w in (("q", s["q"], s["qw"]), ("k", s["k"], s["kw"])):
        v = x.float()
        if w is not None:
            rstd = torch.rsqrt(v.square().mean(2, keepdim=True) + _EPS)
            xh = v * rstd
            v = xh * w
        out[name] = _turned(v, cos, sin, s["pairs"]).to(x.dtype)
        if s["op"] == "rotary_train":
            g = _turned(s["d" + name].float(), cos, -sin, s["pairs"])
            if w is not None:
                out["d" + name + "w"] = (g * xh).sum((0, 1))
                g = g * w
                g = rstd * (g - xh * (g * xh).mean(2, keepdim=True))
            out["d" + name] = g.to(x.dtype)
    return out


def _plain(s):
    if s["op"] == "dropout":
        y = _dropped(s["X"], s["seed_"], s["p"])
        out = {"Y": (y if s["res"] is None else s["res"].float() + y).to(s["X"].dtype)}
        if s["dY"] is not None:
            out["dX"] = _dropped(s["dY"], s["seed_"], s["p"]).to(s["X"].dtype)
        return out
    return _adapter(s) if s["op"].startswith("adapter") else _rotary(s)


# ------------------------------------------------------------------------------------ this repository's calls

def _own(s):
    skm, op = _skm(), s["op"]
    if op == "dropout":
        out = {"Y": skm.sketch_dropout(s["X"], s["p"], s["seed_"], residual=s["res"])}
        if s["dY"] is not None:
            out["dX"] = skm.sketch_dropout(s["dY"], s["p"], s["seed_"])
        return out
    if op == "adapter":
        Y, _ = skm.sketch_adapter_fwd(s["X"], s["A"], s["B"], s["base"], adapter=s["ids"], scale=s["scale"])
        return {"Y": Y}
    if op == "adapter_train":
        Y, H = skm.sketch_adapter_fwd(s["X"], s["A"], s["B"], s["base"], adapter=s["ids"], scale=s["scale"], p=s["p"],
                                      seed=s["seed_"], need_h=True)
        dX, dA, dB = skm.sketch_adapter_bwd(s["dY"], s["X"], H, s["A"], s["B"], s["base_dx"], adapter=s["ids"],
                                            scale=s["scale"], p=s["p"], seed=s["seed_"])
        return {"Y": Y, "dX": dX, "dA": dA, "dB": dB}
    at = dict(eps=_EPS if s["norm"] else None, pairs=s["pairs"])
    q, k = skm.sketch_rotary_fwd(s["q"], s["k"], s["pos"], s["inv_freq"], s["qw"], s["kw"], **at)
    out = {"q": q, "k": k}
    if op == "rotary_train":
        dq, dk, dqw, dkw = skm.sketch_rotary_bwd(s["dq"], s["dk"], s["q"], s["k"], s["pos"], s["inv_freq"], s["qw"],
                                                 s["kw"], **at)
        out.update(dq=dq, dk=dk)
        if s["norm"]:
            out.update(dqw=dqw, dkw=dkw)
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------------------------- in 64 bits

def _stay64(count, seed, p):
    """1 / share for the values that stay, 0 for the others (numpy's unsigned 64-bit products)."""
    key, stream = (int(v) & ((1 << 64) - 1) for v in seed.tolist())
    low = np.uint64(_M32)
    n = np.arange((count + 7) // 8, dtype=np.uint64)
    c0, c1 = n & low, n >> np.uint64(32)
    c2, c3 = np.full_like(n, stream & _M32), np.full_like(n, stream >> 32)
    for i in range(10):
        p0, p1 = np.uint64(0xD2511F53) * c0, np.uint64(0xCD9E8D57) * c2
        k0, k1 = ((key & _M32) + i * 0x9E3779B9) & _M32, ((key >> 32) + i * 0xBB67AE85) & _M32
        c0, c1, c2, c3 = ((p1 >> np.uint64(32)) ^ c1 ^ np.uint64(k0), p1 & low,
                          (p0 >> np.uint64(32)) ^ c3 ^ np.uint64(k1), p0 & low)
    words = np.stack([c0, c1, c2, c3], axis=1).astype("<u4")
    u = np.ascontiguousarray(words).view("<u2").reshape(-1)[:count]
    t = int(math.floor(p * 65536 + 0.5))
    return torch.from_numpy(u >= t).to("cuda").double() * (65536.0 / (65536.0 - t))


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "dropout":
        mask = _stay64(s["X"].numel(), s["seed_"], s["p"]).reshape(s["X"].shape)
        y = s["X"].double() * mask
        out = {"Y": y if s["res"] is None else y + s["res"].double()}
        if s["dY"] is not None:
            out["dX"] = s["dY"].double() * mask
        return out
    if op.startswith("adapter"):
        m, S = s["m"], s["S"]
        ids = torch.zeros(m, device="cuda", dtype=torch.int32) if s["ids"] is None else s["ids"]
        x, y = s["X"].double(), s["base"].double()
        train = op == "adapter_train"
        if train:
            mask = _stay64(x.numel(), s["seed_"], s["p"]).reshape(x.shape) if s["p"] else torch.ones_like(x)
            x = x * mask
            dx, dA, dB = s["base_dx"].double(), [], []
        for a in range(S):
            on = (ids == a).double()[:, None]
            A, B = s["A"][a].double(), s["B"][a].double()
            w = float(s["scale"][a])
            if not bool(on.any()):
                if train:
                    dA.append(torch.zeros_like(A))
                    dB.append(torch.zeros_like(B))
                continue
            h = (x @ A.T) * on * w
            y = y + h @ B.T
            if train:
                dy = s["dY"].double()
                dh = (dy @ B) * on * w
                dx = dx + (dh @ A) * mask
                dA.append(dh.T @ x)
                dB.append(dy.T @ h)
        out = {"Y": y}
        if train:
            out.update(dX=dx, dA=torch.stack(dA), dB=torch.stack(dB))
        return out
    # pairs as complex numbers, turned by exp(i angle)
    turn = torch.polar(torch.ones((), device="cuda", dtype=torch.float64),
                       s["pos"].double()[:, None] * s["inv_freq"][None, :])[:, None, :]
    rot, dh = s["rot"], s["dh"]
    at = torch.arange(rot // 2, device="cuda")
    first, second = (at, at + rot // 2) if s["pairs"] == "halves" else (2 * at, 2 * at + 1)

    def turned(v, by):
        z = torch.complex(v[..., first], v[..., second]) * by
        v = v.clone()
        v[..., first], v[..., second] = z.real, z.imag
        return v

    out = {}
    for name, w in (("q", s["qw"]), ("k", s["kw"])):
        x = s[name].double()
        if w is None:
            out[name] = turned(x, turn)
        else:
            r = 1.0 / torch.sqrt((x * x).sum(2, keepdim=True) / dh + _EPS)
            out[name] = turned(x * r * w.double(), turn)
        if op == "rotary_train":
            gr = turned(s["d" + name].double(), turn.conj())
            if w is not None:
                out["d" + name + "w"] = (gr * x * r).sum(1).sum(0)
                gr = gr * w.double()
                gr = r * gr - x * r ** 3 * ((gr * x).sum(2, keepdim=True) / dh)
            out["d" + name] = gr
    return out
