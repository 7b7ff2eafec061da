"""Plain 64-bit definitions of dropout, the low-rank adapters and head rotation, for the tests (any device)."""
import math

import numpy as np
import torch

U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}   # half steps, relative
SUB = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}              # and of f16's subnormals
E = 2.0 ** -24
INF = float("inf")
T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def philox(key, block, stream):
    """The four words of one call, by Python's whole numbers."""
    M = (1 << 32) - 1
    c = [block & M, block >> 32, stream & M, stream >> 32]
    k = [key & M, key >> 32]
    for _ in range(10):
        a, b = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(b >> 32) ^ c[1] ^ k[0], b & M, (a >> 32) ^ c[3] ^ k[1], a & M]
        k = [(k[0] + 0x9E3779B9) & M, (k[1] + 0xBB67AE85) & M]
    return c


def halves(first, count, seed):
    """The 16 random bits of values first .. first + count - 1 (first a multiple of 8), numpy."""
    key, stream = (int(v) & ((1 << 64) - 1) for v in seed)
    M = np.uint64((1 << 32) - 1)
    s = np.uint64(32)
    n = np.arange(first // 8, first // 8 + (count + 7) // 8, dtype=np.uint64)
    c = [n & M, n >> s, np.full_like(n, stream & int(M)), np.full_like(n, stream >> 32)]
    for i in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        k0 = np.uint64(((key & int(M)) + i * 0x9E3779B9) & int(M))
        k1 = np.uint64(((key >> 32) + i * 0xBB67AE85) & int(M))
        c = [(b >> s) ^ c[1] ^ k0, b & M, (a >> s) ^ c[3] ^ k1, a & M]
    w = np.stack(c, 1)
    return np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], 2).reshape(-1)[:count].astype(np.int64)


def threshold(p):
    return int(math.floor(p * 65536 + 0.5))


def multiplier(shape, p, seed, device):
    """1 / (1 - p) where a value stays, 0 where it goes."""
    t = threshold(p)
    count = int(np.prod(shape))
    keep = torch.from_numpy(halves(0, count, seed) >= t) if t else torch.ones(count, dtype=torch.bool)
    return (keep.to(device).double() * (65536.0 / (65536 - t) if t < 65536 else 0.0)).reshape(shape)


def adapter64(c):
    """Values of a forward and backward in float64 and the bounds of their rounding, for inputs c (a dict).

    Bounds, element by element, with a = absolute values: a sum of L products of exact operands in fp32 is off by at
    most (L + 8) 2^-24 of the sum of their magnitudes (one rounding per addition, 8 for the partial sums of waves and
    ranges and the factors); an operand taken in terms adds its remainder: 2^-16 (two bf16 terms), 2^-21 of the
    token's largest (two f16 terms: 2^-22, and twice for f16's subnormals), 2^-23 (three bf16 terms).
    """
    x, A, B = c["X"].double(), c["A"].double(), c["B"].double()
    m, d = x.shape
    S, r, _ = A.shape
    n = B.shape[1]
    dev = x.device
    ids = torch.zeros(m, dtype=torch.int64, device=dev) if c["ids"] is None else c["ids"].long()
    scale = torch.ones(S, device=dev).double() if c["scale"] is None else c["scale"].double()
    mul = multiplier((m, d), c["p"], c["seed"], dev) if c["p"] else torch.ones_like(x)
    xd = torch.where(mul > 0, x, 0.0) * mul
    f16 = c["X"].dtype == torch.float16
    y = c["base"].double() if c["base"] is not None else torch.zeros((m, n), device=dev).double()
    yb, H, Hb = torch.zeros_like(y), torch.zeros((m, r), device=dev).double(), torch.zeros((m, r), device=dev).double()
    back = c.get("dY") is not None
    out = {}
    if back:
        dy = c["dY"].double()
        dx = c["base_dx"].double() if c["base_dx"] is not None else torch.zeros_like(x)
        dxb = torch.zeros_like(x)
        dA, dB = torch.zeros_like(A), torch.zeros_like(B)
        dAb, dBb = torch.zeros_like(A), torch.zeros_like(B)
    for s in range(S):
        t = torch.nonzero(ids == s).reshape(-1)
        if not t.numel():
            continue
        w, a, b = scale[s], A[s], B[s]
        h = xd[t] @ a.T
        hb = (d + 8) * E * (xd[t].abs() @ a.abs().T)
        H[t], Hb[t] = h, hb
        y[t] += w * (h @ b.T)
        two = 2.0 ** -21 * h.abs().amax(1, keepdim=True).expand_as(h) if f16 else 2.0 ** -16 * h.abs()
        yb[t] = w.abs() * ((hb + two + (2 * r + 8) * E * h.abs()) @ b.abs().T)
        if back:
            g = dy[t]
            dh = w * (g @ b)
            dhb = (n + 8) * E * w.abs() * (g.abs() @ b.abs())
            k = t.numel()
            three = 2.0 ** -23 + (3 * k + 8) * E
            dB[s] = w * (g.T @ h)
            dBb[s] = w.abs() * (g.abs().T @ (hb + three * h.abs()))
            dA[s] = dh.T @ xd[t]
            dAb[s] = (dhb + three * dh.abs()).T @ xd[t].abs()
            dx[t] += (dh @ a) * mul[t]
            two = 2.0 ** -21 * dh.abs().amax(1, keepdim=True).expand_as(dh) if f16 else 2.0 ** -16 * dh.abs()
            dxb[t] = ((dhb + two + (2 * r + 8) * E * dh.abs()) @ a.abs()) * mul[t]
    u, sub = U[c["X"].dtype], SUB[c["X"].dtype]
    out["Y"] = (y, yb + u * y.abs() * (1 + 2.0 ** -7) + sub + 2 * E * y.abs())
    out["H"] = (H, Hb)
    if back:
        out["dX"] = (dx, dxb + u * dx.abs() * (1 + 2.0 ** -7) + sub + 2 * E * dx.abs())
        out["dA"], out["dB"] = (dA, dAb), (dB, dBb)
    return out


def turned(v, angle, pairs, back=False):
    rot = 2 * angle.shape[1]
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    if back:
        s = -s
    i = torch.arange(rot // 2, device=v.device)
    a, b = (i, i + rot // 2) if pairs == "halves" else (2 * i, 2 * i + 1)
    o = v.clone()
    o[..., a] = v[..., a] * c - v[..., b] * s
    o[..., b] = v[..., a] * s + v[..., b] * c
    return o


def rotary64(x, w, pos, freq, eps, pairs, dy=None):
    """(y, bound) of one side, and with dy (dx, bound), (dw, bound). x [m, h, dh] of any dtype.

    Bounds: the mean square of dh values is off by (dh + 2) 2^-24 of itself, its root by half, quotients and products by
    2^-24 each; sine and cosine by 2^-23 (the angle's rest rounded, the Taylor sum); a turned value is the sum of two
    products, bounded by the pair's magnitudes.
    """
    m, h, dh = x.shape
    u, sub = U[x.dtype], SUB[x.dtype]
    v = x.double()
    angle = pos.double()[:, None] * freq
    rel = E * (16 + ((dh + 2) / 2 if eps is not None else 0))
    i = torch.arange(angle.shape[1], device=x.device)
    a, b = (i, i + angle.shape[1]) if pairs == "halves" else (2 * i, 2 * i + 1)

    def pair_size(z):
        s = z.abs().clone()
        s[..., a] = s[..., b] = z[..., a].abs() + z[..., b].abs()
        return s

    ww = torch.ones(dh, device=x.device).double() if w is None else w.double()
    r = torch.ones((m, h, 1), device=x.device).double()
    if eps is not None:
        r = 1.0 / torch.sqrt((v * v).mean(2, keepdim=True) + eps)
    z = v * r * ww if eps is not None else v
    y = turned(z, angle, pairs)
    out = {"y": (y, u * y.abs() * (1 + 2.0 ** -7) + sub + rel * pair_size(z))}
    if dy is not None:
        g0 = dy.double()
        g = turned(g0, angle, pairs, back=True)
        gs = pair_size(g0)
        if eps is None:
            out["dx"] = (g, u * g.abs() * (1 + 2.0 ** -7) + sub + rel * gs)
        else:
            xh = v * r
            out["dw"] = ((g * xh).sum((0, 1)), (m * h + 40 + dh) * E * (gs * xh.abs()).sum((0, 1)))
            q = (g * ww * xh).mean(2, keepdim=True)
            qs = (gs * ww.abs() * xh.abs()).mean(2, keepdim=True)
            dx = r * (g * ww - xh * q)
            size = r * (gs * ww.abs() + xh.abs() * qs)
            out["dx"] = (dx, u * dx.abs() * (1 + 2.0 ** -7) + sub + (2 * rel + (dh + 8) * E) * size)
    return out


def off(got, want_bound):
    """How far `got` is outside its bound (<= 0: inside). A value whose magnitude is at least the type's largest plus half
    of its last step rounds to an infinity: that is its result, and either is where the bound reaches that border."""
    want, bound = want_bound
    if not got.numel():
        return 0.0
    far = (got.double() - want).abs() - bound
    if got.dtype in (torch.float16, torch.bfloat16):
        top = torch.finfo(got.dtype).max
        border = top * (1 + U[got.dtype] / (2 - 2 * U[got.dtype]))
        infinite = torch.isinf(got) & (torch.sign(got.double()) == torch.sign(want))
        far = torch.where(infinite & (want.abs() + bound >= border), -1.0, far)
        far = torch.where(~infinite & (want.abs() - bound >= border), INF, far)
    return float(far.max())
