"""GPU parity of the 8-bit checkpoints, norms and cross entropy of a sketched head against float64.

Tolerances are bounds by arithmetic, elementwise. u = 2^-24 is half a step of fp32, h(t) = finfo(t).eps / 2
half a relative step of a 16-bit type. A sum of k terms added in chains of c additions is off by at most
(c + 1) u of the sum of the terms' magnitudes (to first order); each bound counts the additions of the longest
chain the kernels can have and is applied to the float64 sum of magnitudes.
"""
import numpy as np
import pytest

import oracle
from lut_sketched_matmul_amd import synthetic as syn
from oracle import train_oracle as to

from gpu_util import to_dev, to_f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
H = {"f32": U, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}   # half a relative step
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}     # half a step of the subnormals that matter here


def skm():
    import lut_sketched_matmul_amd as m
    return m


def torch():
    import torch as _t
    return _t


def tdtype(name):
    t = torch()
    return {"f32": t.float32, "f16": t.float16, "bf16": t.bfloat16}[name]


def within(got, ref, bound, what):
    assert got.shape == ref.shape, what
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN at other places"
    off = np.abs(got - ref)[~nan] - np.broadcast_to(bound, ref.shape)[~nan]
    assert off.size == 0 or off.max() <= 0.0, f"{what}: {int((off > 0).sum())} of {off.size} over the bound by up to {off.max():.3e}"


def dev(name, shape, sigma, dtype):
    a = syn.random_normal(name, shape, sigma, dtype)
    return to_dev(a, dtype), syn.to_float64(a, dtype)


# ---------------------------------------------------------------------------------------------------------
# 8-bit checkpoints: exact
# ---------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,d", [(1, 32), (3, 64), (5, 160), (2, 4096), (33, 1376)])
def test_act_quant_exact(m, d, dtype):
    """Codes, exponent bytes and the values read back, bit for bit; blocks of many scales, zeros, non-finite."""
    a = syn.random_normal(f"ckpt/{m}/{d}", (m, d), 1.0, "f32").astype(np.float64)
    e = syn.rng_for(f"ckpt/scale/{m}/{d}").integers(-14, 5, size=(m, d // 32))
    a = a * np.repeat(2.0 ** e, 32, axis=1)
    a[0, :32] = 0.0
    s = syn.to_storage(a.astype(np.float32), dtype)
    a = syn.to_float64(s, dtype)
    if d > 64:
        a[m - 1, d - 1], a[0, 40], a[m // 2, 70] = np.inf, np.nan, -np.inf
        s = syn.to_storage(a.astype(np.float32), dtype)
    X = to_dev(s, dtype)
    codes, scales = skm().sketch_act_quant(X)
    qc, qs = to.act_quant(a, dtype)
    assert np.array_equal(scales.cpu().numpy(), qs)
    assert np.array_equal(codes.cpu().numpy(), qc)
    back = to_f64(skm().sketch_act_dequant(codes, scales, tdtype(dtype)))
    assert np.array_equal(back, to.act_dequant(qc, qs), equal_nan=True)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_act_quant_ends_of_the_range(dtype):
    """The largest and smallest values of every type, ties, and both sides of a step's change."""
    big = {"f16": 65504.0, "bf16": (2 - 2.0 ** -7) * 2.0 ** 127, "f32": (2 - 2.0 ** -23) * 2.0 ** 127}[dtype]
    tops = [big, 127.0, 127.5, 128.0, 126.5, 63.5, 2.0 ** -14, 2.0 ** -24, 1.984375, 1.9921875, 1.9765625]
    if dtype != "f16":
        tops += [2.0 ** -126, 2.0 ** -120, 1e30, 1e-30, 2.0 ** 121 * 127, 2.0 ** -130]
    a = np.zeros((len(tops), 32))
    for i, t in enumerate(tops):
        with np.errstate(over="ignore"):
            a[i, :8] = [t, -t, t / 2, t / 254, 3 * t / 254, -5 * t / 254, t / 508, -t / 127]
    s = syn.to_storage(a.astype(np.float32), dtype)
    a = syn.to_float64(s, dtype)
    codes, scales = skm().sketch_act_quant(to_dev(s, dtype))
    qc, qs = to.act_quant(a, dtype)
    assert np.array_equal(scales.cpu().numpy(), qs) and np.array_equal(codes.cpu().numpy(), qc)
    back = to_f64(skm().sketch_act_dequant(codes, scales, tdtype(dtype)))
    assert np.isfinite(back).all() and np.array_equal(back, to.act_dequant(qc, qs))


def test_act_quant_empty_and_outputs():
    t = torch()
    X = t.zeros((0, 64), dtype=t.float16, device="cuda")
    codes, scales = skm().sketch_act_quant(X)
    assert codes.shape == (0, 64) and scales.shape == (0, 2)
    assert skm().sketch_act_dequant(codes, scales, t.float16).shape == (0, 64)
    X = t.randn((4, 64), device="cuda").half()
    buf = t.full((6, 64), 7, dtype=t.int8, device="cuda")
    skm().sketch_act_quant(X, codes=buf[1:5])
    assert (buf[0] == 7).all() and (buf[5] == 7).all()     # rows outside the output stay as they were


PAIRS = [("f16", "f16"), ("bf16", "f16"), ("bf16", "bf16"), ("f16", "bf16"), ("f32", "f32")]


@pytest.mark.parametrize("io,ldt", PAIRS)
@pytest.mark.parametrize("m,n,d,b,gpr", [
    (1, 136, 512, 2, 1), (33, 136, 512, 3, 4), (96, 136, 512, 4, 8), (31, 131, 96, 4, 1), (64, 1, 64, 3, 1),
    (40, 1000, 256, 4, 1), (5, 1100, 2048, 2, 2), (290, 520, 1088, 4, 2), (300, 77, 640, 3, 20),
])
def test_bwd_from_checkpoint(m, n, d, b, gpr, io, ldt):
    """Both gradients of the values the checkpoint stands for against float64; ragged tokens, rows and columns."""
    t = torch()
    name = f"bwdck/{m}/{n}/{d}/{io}/{ldt}/{b}"
    idx = syn.random_packed_indices(name + "/i", n, d, b)
    lut = syn.random_lut(name + "/l", n, gpr, b, 0.02, ldt)
    X, _ = dev(name + "/x", (m, d), 1.0, io)
    dY, dY64 = dev(name + "/y", (m, n), 0.1, io)
    gi, gl = to_dev(idx, "u8"), to_dev(lut, ldt)
    codes, scales = skm().sketch_act_quant(X)
    x64 = to.act_dequant(codes.cpu().numpy(), scales.cpu().numpy())
    dX, dL = skm().sketch_matmul_bwd_ckpt(dY, codes, scales, gi, gl, b, gpr)
    ref = oracle.backward_dlut(dY64, x64, idx, b, gpr)
    mag = oracle.backward_dlut(np.abs(dY64), np.abs(x64), idx, b, gpr)
    # tokens in chains of at most m, a bin's entries in chains of at most d / gpr, split sums
    tol = (m + d // gpr + 80) * U * mag
    within(to_f64(dL), ref, tol, "dLUT")
    W = oracle.dequantize(idx, syn.to_float64(lut, ldt), d, b, gpr)
    sx = (np.abs(dY64) @ np.abs(W)) * (n + 80) * U
    if (io, ldt) == ("bf16", "f16"):       # operands below 2^-14 of f16: 2^-23 of the row's largest
        sx = sx + 2.0 ** -23 * np.abs(dY64).max(1, keepdims=True) * np.abs(W).sum(0)
    elif (io, ldt) == ("f16", "bf16"):     # dY is rounded to the tables' dtype
        sx = sx + H["bf16"] * (np.abs(dY64) @ np.abs(W))
    within(to_f64(dX), dY64 @ W, sx, "dX")
    one = skm().sketch_matmul_bwd_ckpt(dY, codes, scales, gi, gl, b, gpr, need_dlut=False)
    assert one[1] is None and t.equal(one[0], dX)
    acc = t.ones_like(dL)
    two = skm().sketch_matmul_bwd_ckpt(dY, codes, scales, gi, gl, b, gpr, need_dx=False, dlut_out=acc, accumulate=True)
    assert two[0] is None and two[1] is acc
    within(to_f64(acc), to_f64(dL) + 1.0, 80 * U * (mag + 1.0), "accumulate")


@pytest.mark.parametrize("m", [33, 64])
def test_bwd_from_checkpoint_infinite_gradient_stays_in_its_row(m):
    """Padding rows are zeros, not copies: an infinity in the last token's dY stays an infinity of its table row."""
    t = torch()
    n, d = 136, 64
    idx = syn.random_packed_indices("bwdinf/i", n, d, 4)
    gi, gl = to_dev(idx, "u8"), t.randn((n, 1, 16), device="cuda").half()
    codes, scales = skm().sketch_act_quant(t.ones((m, d), device="cuda").half())
    dY = t.ones((m, n), device="cuda").half()
    dY[m - 1, 5] = float("inf")
    dL = to_f64(skm().sketch_matmul_bwd_ckpt(dY, codes, scales, gi, gl, 4, 1)[1])
    used = oracle.backward_dlut(np.ones((1, n)), np.ones((1, d)), idx, 4, 1)
    assert np.isposinf(dL[5][used[5] > 0]).all()
    rest = [i for i in range(n) if i != 5]
    assert np.array_equal(dL[rest], m * used[rest])


# ---------------------------------------------------------------------------------------------------------
# norms
# ---------------------------------------------------------------------------------------------------------

SHAPES = [(1, 1), (2, 7), (3, 32), (5, 100), (4, 513), (7, 512), (9, 1001), (6, 1024), (3, 1025), (3, 2048), (2, 2056), (3, 4096),
          (2, 5000), (2, 8224), (1, 16384), (2, 17000), (1, 65536), (300, 64)]


@pytest.mark.parametrize("params", ["f32", "same", "none"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,d", SHAPES)
def test_norm_forward_backward(m, d, dtype, kind, params):
    t = torch()
    name = f"norm/{m}/{d}/{kind}"
    eps = 1e-5
    a = syn.to_float64(syn.random_normal(name, (m, d), 1.0, "f32"), "f32") * 2.0 + 1.5
    s = syn.to_storage(a.astype(np.float32), dtype)
    X, x = to_dev(s, dtype), syn.to_float64(s, dtype)
    pd = {"f32": "f32", "same": dtype, "none": None}[params]
    W = B = w = b = None
    if pd:
        W, w = dev(name + "/w", (d,), 1.0, pd)
        if kind == "layer":
            B, b = dev(name + "/b", (d,), 0.5, pd)
    Y, mean, rstd, codes, scales = skm().sketch_norm_fwd(X, W, B, kind=kind, eps=eps)
    assert codes is None and scales is None and (mean is None) == (kind == "rms")
    ry, rm, rr = to.norm_fwd(x, w, b, kind, eps)
    # chains: at most 64 elements per thread, 6 + 16 sums over lanes and waves
    c = 96 * U
    top = np.abs(x).max(1)
    dm = c * np.abs(x).sum(1) / d + U * top if kind == "layer" else np.zeros(m)      # error of the mean
    if mean is not None:
        within(to_f64(mean), rm, dm, "mean")
    # relative error of the variance: its own chain, twice that of x - mean, and the mean's
    sd = 1.0 / rr
    dr = rr * (c + 4 * U + dm * dm * rr * rr + 2 * (dm + U * top) / sd)
    within(to_f64(rstd), rr, dr, "rstd")
    aw = np.abs(w) if w is not None else 1.0
    xh = np.abs(x - (rm[:, None] if kind == "layer" else 0.0)) * rr[:, None]
    arith = aw * (xh * (dr / rr + 4 * U)[:, None] + ((dm + U * top) * rr)[:, None]) + U * np.abs(ry)
    within(to_f64(Y), ry, arith * 1.01 + H[dtype] * (np.abs(ry) + arith) + TINY[dtype], "Y")

    for dyt in {"f32", dtype}:
        G, g = dev(name + "/dy", (m, d), 1.0, dyt)
        dX, dw, db = skm().sketch_norm_bwd(G, X, W, mean, rstd, kind=kind)
        mu, rs = (to_f64(mean) if mean is not None else np.zeros(m)), to_f64(rstd)
        rx, rw, rb = to.norm_bwd(g, x, w, mu, rs, kind)
        xh = (x - (mu[:, None] if kind == "layer" else 0.0)) * rs[:, None]
        axh = np.abs(xh) + U * (np.abs(x) + np.abs(mu)[:, None]) * rs[:, None]
        gw = np.abs(g if w is None else g * w)
        # each term of dx = r (g - mean(g) - xh mean(g xh)), its products and the two chains
        e = rs[:, None] * (4 * U * gw + (c + 4 * U) * gw.mean(1, keepdims=True)
                           + (c + 8 * U) * axh * (gw * axh).mean(1, keepdims=True)
                           + 2 * U * (np.abs(x) + np.abs(mu)[:, None]) * rs[:, None] * (gw * axh).mean(1, keepdims=True)
                           + 2 * U * axh * ((np.abs(x) + np.abs(mu)[:, None]) * rs[:, None] * gw).mean(1, keepdims=True))
        within(to_f64(dX), rx, e * 1.01 + H[dtype] * (np.abs(rx) + e) + TINY[dtype], f"dX {dyt}")
        # rows in chains of at most m, then the partial sums of at most 2048 blocks in 16 slices
        k = (min(m, 4096) + 160) * U
        within(to_f64(dw), rw, k * (np.abs(g) * axh).sum(0)
               + 2 * U * (np.abs(g) * (np.abs(x) + np.abs(mu)[:, None]) * rs[:, None]).sum(0), f"dw {dyt}")
        within(to_f64(db), rb, k * np.abs(g).sum(0), f"db {dyt}")
        # the outputs one by one, and added to what is there
        one = skm().sketch_norm_bwd(G, X, W, mean, rstd, kind=kind, need_dw=False, need_db=False)
        assert t.equal(one[0], dX) and one[1] is None and one[2] is None
        w1 = t.ones(d, device="cuda")
        two = skm().sketch_norm_bwd(G, X, W, mean, rstd, kind=kind, need_dx=False, need_db=False, dw_out=w1,
                                    accumulate=True)
        assert two[0] is None and two[1] is w1
        within(to_f64(w1), to_f64(dw) + 1.0, 8 * U * (1.0 + np.abs(to_f64(dw))), "accumulate")


@pytest.mark.parametrize("m,d,dtype,kind", [(600, 16392, "bf16", "layer"), (70, 16385, "f16", "rms"),
                                            (130, 8232, "bf16", "layer")])
def test_norm_many_long_rows(m, d, dtype, kind):
    """Blocks that walk several long rows, and slabs of several rows per column sum."""
    test_norm_forward_backward(m, d, dtype, kind, "f32")


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,d", [(1, 32), (5, 96), (3, 2048), (6, 4096), (2, 8224), (2, 17024)])
def test_norm_checkpoint(m, d, dtype, kind):
    """The checkpoint written along is that of Y as stored, and the backward reads X from a checkpoint."""
    t = torch()
    X, _ = dev(f"normck/{m}/{d}", (m, d), 1.0, dtype)
    W, _ = dev(f"normck/w/{d}", (d,), 1.0, "f32")
    Y, mean, rstd, codes, scales = skm().sketch_norm_fwd(X, W, kind=kind, checkpoint=True)
    plain = skm().sketch_norm_fwd(X, W, kind=kind)
    assert t.equal(Y, plain[0]) and t.equal(rstd, plain[2])
    c, s = skm().sketch_act_quant(Y)
    assert t.equal(codes, c) and t.equal(scales, s)
    xc = skm().sketch_act_quant(X)
    xq = skm().sketch_act_dequant(*xc, X.dtype)
    G, _ = dev(f"normck/dy/{m}/{d}", (m, d), 1.0, "f32")
    want = skm().sketch_norm_bwd(G, xq, W, mean, rstd, kind=kind)
    got = skm().sketch_norm_bwd(G, xc, W, mean, rstd, kind=kind, x_dtype=X.dtype)
    for p, q in zip(got, want):
        assert t.equal(p, q)


def test_norm_rows_apart():
    """A row of NaN, of infinities or of zeros changes no other row; zeros give y = bias and dx = 0 for dy = 0."""
    t = torch()
    X = t.randn((6, 4096), device="cuda").bfloat16()
    W, B = t.randn(4096, device="cuda"), t.randn(4096, device="cuda")
    base = skm().sketch_norm_fwd(X, W, B)
    Z = X.clone()
    Z[1] = float("nan")
    Z[3, 5] = float("inf")
    Z[4] = 0.0
    Y, mean, rstd, codes, scales = skm().sketch_norm_fwd(Z, W, B, checkpoint=True)
    for r in (0, 2, 5):
        assert t.equal(Y[r], base[0][r])
    assert t.isnan(Y[1].float()).all() and t.equal(Y[4], B.bfloat16())
    assert (scales[1] == 255).all()
    G = t.zeros_like(X)
    dX, dw, db = skm().sketch_norm_bwd(G, X, W, base[1], base[2])
    assert (dX == 0).all() and (dw == 0).all() and (db == 0).all()


def test_norm_empty():
    t = torch()
    X = t.zeros((0, 64), dtype=t.float16, device="cuda")
    Y, mean, rstd, codes, scales = skm().sketch_norm_fwd(X, checkpoint=True)
    assert Y.shape == (0, 64) and mean.numel() == 0 and codes.shape == (0, 64)
    dX, dw, db = skm().sketch_norm_bwd(X, X, None, mean, rstd)
    assert dX.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


def test_norm_many_rows_is_deterministic():
    """More rows than blocks: chains of rows per block, the same bits every time."""
    t = torch()
    m, d = 5003, 264
    X, x = dev("normmany", (m, d), 1.0, "bf16")
    G, g = dev("normmany/g", (m, d), 1.0, "bf16")
    Y, mean, rstd, _, _ = skm().sketch_norm_fwd(X)
    a = skm().sketch_norm_bwd(G, X, None, mean, rstd)
    b = skm().sketch_norm_bwd(G, X, None, mean, rstd)
    assert all(t.equal(p, q) for p, q in zip(a, b))
    mu, rs = to_f64(mean), to_f64(rstd)
    _, rw, rb = to.norm_bwd(g, x, None, mu, rs, "layer")
    xh = np.abs(x - mu[:, None]) * rs[:, None]
    k = (m / 500 + 200) * U
    within(to_f64(a[1]), rw, k * (np.abs(g) * (xh + 2.0)).sum(0), "dw")
    within(to_f64(a[2]), rb, k * np.abs(g).sum(0), "db")


# ---------------------------------------------------------------------------------------------------------
# cross entropy of a sketched head
# ---------------------------------------------------------------------------------------------------------

def head(name, V, d, b, gpr, ldt, sigma=0.05):
    idx = syn.random_packed_indices(name + "/i", V, d, b)
    lut = syn.random_lut(name + "/l", V, gpr, b, sigma, ldt)
    W = oracle.dequantize(idx, syn.to_float64(lut, ldt), d, b, gpr)
    return to_dev(idx, "u8"), to_dev(lut, ldt), idx, W


def targets_for(name, m, V, ignored):
    g = syn.rng_for(name)
    t = g.integers(0, V, size=m)
    if ignored == "some":
        t[g.random(m) < 0.4] = -100
    elif ignored == "all":
        t[:] = -100
    return t


def check_xent(name, m, V, d, b, gpr, io, ldt, ignored="some", sigma=1.0, dscale=1.0, x=None, need=(True, True)):
    t = torch()
    gi, gl, idx, W = head(name, V, d, b, gpr, ldt)
    if x is None:
        X, x = dev(name + "/x", (m, d), sigma, io)
    else:
        s = syn.to_storage(x.astype(np.float32), io)
        X, x = to_dev(s, io), syn.to_float64(s, io)
    tg = targets_for(name + "/t", m, V, ignored)
    T = t.from_numpy(tg).cuda()
    live = tg != -100
    xl = np.where(live[:, None], x, 0.0)
    loss, lse = skm().sketch_xent_fwd(X, gi, gl, T, b, gpr)
    Z = xl @ W.T
    rl, rs = to.xent_fwd(Z, tg)
    S = (np.abs(xl) @ np.abs(W).T).max(1)
    # logits: products of d columns, 16 (or 32) at a time; bf16 -> f16 operands lose at most 2^-23 of the row's top
    dz = (d / 16 + 24) * U * S
    if (io, ldt) == ("bf16", "f16"):
        dz = dz + 2.0 ** -23 * np.abs(xl).max(1) * np.abs(W).sum(1).max()
    # exp of arguments down to -A: relative error (1.5 A + 8) u, where terms below e^-30 of the largest count nothing;
    # chains of 32 + 8 + V / 4096 + 32 additions
    rel = (45 + 8 + 72 + V / 4096) * U
    bound = np.where(live, dz + rel + 8 * U * np.abs(rs), 0.0)
    within(to_f64(lse), rs, bound, "lse")
    within(to_f64(loss), rl, np.where(live, 2 * bound + 4 * U * np.abs(rl), 0.0), "loss")

    w = np.abs(syn.to_float64(syn.random_normal(name + "/w", (m,), 1.0, "f32"), "f32")) * dscale
    w = w.astype(np.float32).astype(np.float64)
    DL = t.from_numpy(w.astype(np.float32)).cuda()
    dX, dL = skm().sketch_xent_bwd(X, gi, gl, T, lse, DL, b, gpr, need_dx=need[0], need_dlut=need[1])
    lse64 = to_f64(lse)
    dZ = to.xent_dz(Z, tg, lse64, w)
    P = np.exp(np.where(live[:, None], Z - lse64[:, None], -np.inf))
    # error of dZ before its rounding: the softmax's argument and exp, and the subtraction
    e = w[:, None] * (P * (dz[:, None] + 2 * U * np.abs(lse64)[:, None] + 60 * U) + 4 * U)
    top = (w * live).max() if live.any() else 0.0
    if need[0]:
        # operands rounded once in the tables' dtype (f16: a floor of 2^-39 of the largest dloss), fp32 sums of V terms
        op = H[ldt] * (np.abs(dZ) + e) + (2.0 ** -38 * top if ldt == "f16" else 0.0)
        err = (e + op) @ np.abs(W) + (V / 16 + 64) * U * (np.abs(dZ) @ np.abs(W))
        ref = dZ @ W
        within(to_f64(dX), ref, 1.01 * err + H[io] * (np.abs(ref) + err) + TINY[io], "dX")
        assert (to_f64(dX)[~live] == 0).all()
    else:
        assert dX is None
    if need[1]:
        split = {"f16": 2.0 ** -22, "bf16": 2.0 ** -16}[io]
        op = e + split * np.abs(dZ) + (2.0 ** -38 * top if io == "f16" else 0.0)
        ref = oracle.backward_dlut(dZ, xl, idx, b, gpr)
        err = oracle.backward_dlut(op, np.abs(xl), idx, b, gpr)
        mag = oracle.backward_dlut(np.abs(dZ), np.abs(xl), idx, b, gpr)
        within(to_f64(dL), ref, 1.01 * err + (2 * m / 16 + d / gpr + 40) * U * mag, "dLUT")
    else:
        assert dL is None
    return loss, lse, dX, dL


@pytest.mark.parametrize("io,ldt", [("f16", "f16"), ("bf16", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("m,V,d,b,gpr", [
    (1, 1, 32, 4, 1), (1, 7, 64, 2, 1), (2, 255, 64, 3, 2), (3, 256, 96, 4, 1), (16, 257, 128, 4, 4),
    (17, 300, 512, 4, 1), (31, 1000, 256, 3, 2), (33, 520, 576, 2, 2), (64, 129, 512, 4, 8), (257, 1001, 320, 4, 1),
    (300, 2050, 512, 3, 1),
    # few tokens: activations per slot (below and from 8 tokens on, ragged slots), many tokens, tables too large for
    # the decode
    (5, 300, 8192, 4, 4), (16, 130, 2112, 2, 1), (64, 100, 1024, 3, 4), (65, 257, 128, 4, 2), (4, 90, 512, 4, 16),
])
def test_xent(m, V, d, b, gpr, io, ldt):
    check_xent(f"xent/{m}/{V}/{d}/{b}/{io}/{ldt}", m, V, d, b, gpr, io, ldt, ignored="some" if m > 2 else "none")


@pytest.mark.parametrize("need", [(True, False), (False, True)])
@pytest.mark.parametrize("io,ldt", [("f16", "f16"), ("bf16", "f16"), ("bf16", "bf16")])
def test_xent_one_gradient(io, ldt, need):
    check_xent(f"xent1/{io}/{ldt}", 70, 400, 256, 4, 2, io, ldt, need=need)


@pytest.mark.parametrize("ignored", ["none", "all"])
def test_xent_ignored(ignored):
    loss, lse, dX, dL = check_xent(f"xenti/{ignored}", 40, 300, 256, 4, 1, "bf16", "f16", ignored=ignored)
    if ignored == "all":
        assert (loss == 0).all() and (lse == 0).all() and (dX == 0).all() and (dL == 0).all()


@pytest.mark.parametrize("io,ldt", [("f16", "f16"), ("bf16", "f16"), ("bf16", "bf16")])
def test_xent_far_scales(io, ldt):
    """Logits in the hundreds beside rows of zeros and tiny ones: no row's statistics spoil another's."""
    m, d = 48, 256
    x = syn.to_float64(syn.random_normal("xents", (m, d), 1.0, "f32"), "f32")
    x *= np.exp(np.linspace(-12, 4, m))[:, None]
    x[7] = 0.0
    check_xent(f"xents/{io}/{ldt}", m, 600, d, 4, 1, io, ldt, ignored="none", x=x)


@pytest.mark.parametrize("dscale", [1e-6, 1e-3, 4096.0])
@pytest.mark.parametrize("io", ["f16", "bf16"])
def test_xent_gradient_scales(io, dscale):
    check_xent(f"xentg/{io}/{dscale}", 50, 777, 256, 4, 1, io, io, dscale=dscale)


def test_xent_pieces_of_the_vocabulary():
    """4096 tokens: 256 MiB of dZ is 16384 words with dLUT, so this vocabulary takes two pieces, the last ragged."""
    check_xent("xentp", 4096, 16650, 64, 4, 1, "bf16", "f16")


def test_xent_nonfinite_in_ignored_rows():
    """Rows of ignored tokens may hold anything; a bad target is NaN in its own row and in dLUT, not elsewhere."""
    t = torch()
    gi, gl, idx, _ = head("xentn", 300, 256, 4, 2, "f16")
    X = t.randn((40, 256), device="cuda").bfloat16()
    T = t.randint(0, 300, (40,), device="cuda")
    T[[3, 20, 39]] = -100
    DL = t.ones(40, device="cuda")
    base = skm().sketch_xent_fwd(X, gi, gl, T, 4, 2)
    grads = skm().sketch_xent_bwd(X, gi, gl, T, base[1], DL, 4, 2)
    Z = X.clone()
    Z[3], Z[20, 7], Z[39] = float("nan"), float("inf"), float("-inf")
    DL[3], DL[20] = float("nan"), float("inf")
    got = skm().sketch_xent_fwd(Z, gi, gl, T, 4, 2)
    assert t.equal(got[0], base[0]) and t.equal(got[1], base[1])
    g2 = skm().sketch_xent_bwd(Z, gi, gl, T, base[1], DL, 4, 2)
    assert t.equal(g2[0], grads[0]) and t.equal(g2[1], grads[1])
    T[5] = 300
    loss, lse = skm().sketch_xent_fwd(Z, gi, gl, T, 4, 2)
    keep = [i for i in range(40) if i != 5]
    assert t.isnan(loss[5]) and t.equal(loss[keep], base[0][keep]) and t.equal(lse, base[1])
    dX, dL = skm().sketch_xent_bwd(Z, gi, gl, T, lse, DL, 4, 2)
    assert t.isnan(dX[5].float()).all() and t.equal(dX[keep], grads[0][keep])
    used = oracle.backward_dlut(np.ones((1, 300)), np.ones((1, 256)), idx, 4, 2) > 0     # entries some column maps to
    assert np.array_equal(np.isnan(to_f64(dL)), used)


def test_xent_other_ignore_index_and_accumulate():
    t = torch()
    gi, gl, _, _ = head("xenta", 200, 128, 4, 1, "f16")
    X = t.randn((33, 128), device="cuda").half()
    T = t.randint(1, 200, (33,), device="cuda")
    DL = t.full((33,), 0.5, device="cuda")
    T2 = T.clone()
    T[::3], T2[::3] = -100, 0
    a = skm().sketch_xent_fwd(X, gi, gl, T, 4, 1)
    b = skm().sketch_xent_fwd(X, gi, gl, T2, 4, 1, ignore_index=0)
    assert t.equal(a[0], b[0]) and t.equal(a[1], b[1])
    ga = skm().sketch_xent_bwd(X, gi, gl, T, a[1], DL, 4, 1)
    acc = t.full_like(ga[1], 2.0)
    gb = skm().sketch_xent_bwd(X, gi, gl, T2, a[1], DL, 4, 1, ignore_index=0, dlut_out=acc, accumulate=True)
    assert t.equal(ga[0], gb[0]) and gb[1] is acc
    within(to_f64(acc), to_f64(ga[1]) + 2.0, 4 * U * (2.0 + np.abs(to_f64(ga[1]))), "accumulate")


@pytest.mark.parametrize("V", [40, 20000])
def test_xent_table_gradient_keeps_fp32_of_bf16(V):
    """dLUT takes bf16 activations' dZ as precisely as f16's.

    Activations of +-1 are exact in both types and scaling them by a power of two changes no logit, so both calls start
    from the same dZ, and an entry is dZ times a whole number: each side is off by 2^-23 (two f16 values) and by the
    rounding of three fp32 operations at the most. (f16's floor: 2^-39 of the gradient, 1.)
    """
    t = torch()
    d = 256
    gi, gl, idx, _ = head(f"xentq/{V}", V, d, 4, 1, "f16")
    X = t.sign(t.randn((1, d), device="cuda") + 0.1)
    T = t.full((1,), V - 3, device="cuda", dtype=t.int64)
    DL = t.ones(1, device="cuda")
    _, lse = skm().sketch_xent_fwd(X.half(), gi, gl, T, 4, 1)
    a = skm().sketch_xent_bwd(X.half(), gi, gl, T, lse, DL, 4, 1, need_dx=False)[1]
    b = skm().sketch_xent_bwd(X.bfloat16(), gi, gl, T, lse, DL, 4, 1, need_dx=False)[1]
    ref = to_f64(a)
    within(to_f64(b), ref, 2 * (2.0 ** -23 + 3 * U) * np.abs(ref) + 2 * d * 2.0 ** -39, "dLUT")


@pytest.mark.parametrize("m,V,d,b,gpr", [
    # many groups of 16 tokens in one launch: a last group of 4 and of 15 tokens, row blocks that are no whole number
    # of 8, activations in LDS and from memory; and the first shapes past them, which take the tiles
    (500, 130, 256, 4, 2), (175, 1000, 1056, 3, 3), (300, 2048, 1536, 2, 2), (120, 3300, 2048, 4, 1),
    (1000, 2048, 320, 4, 1), (48, 12000, 256, 4, 2),
])
@pytest.mark.parametrize("io,ldt", [("f16", "f16"), ("bf16", "f16"), ("bf16", "bf16")])
def test_xent_groups_of_tokens(m, V, d, b, gpr, io, ldt):
    check_xent(f"xentgr/{m}/{V}/{io}/{ldt}", m, V, d, b, gpr, io, ldt)


@pytest.mark.parametrize("m,V,d,ignored", [
    # 144 dX tiles, cut 3 : 1; as many that 0.6 of them are equal ranges; 297, the last 41 in halves; too few words to
    # cut; a single tile in ranges; more tokens than one round of the list's scan
    (4400, 2100, 2048, "none"), (4400, 2100, 2048, "some"), (8200, 2100, 2304, "none"), (4400, 1000, 2048, "none"),
    (300, 1500, 256, "some"), (17000, 300, 64, "some"),
])
def test_xent_ranges_of_dx(m, V, d, ignored):
    check_xent(f"xentdx/{m}/{V}/{ignored}", m, V, d, 4, 1, "f16", "f16", ignored=ignored, need=(True, False))


def test_xent_pieces_with_cut_tiles():
    """Two pieces of 36 steps (the second ragged), 160 dX tiles of each in two ranges."""
    check_xent("xentcut", 10000, 4590, 1024, 4, 1, "bf16", "bf16", ignored="none")


@pytest.mark.parametrize("io,ldt", [("f16", "f16"), ("bf16", "f16"), ("bf16", "bf16")])
def test_xent_zero_rows_have_gradients(io, ldt):
    """A row of zeros (or nearly) gives the tables nothing but takes the gradient sum_v (1/V - [target]) W itself."""
    m, d = 40, 256
    x = syn.to_float64(syn.random_normal("xentz", (m, d), 1.0, "f32"), "f32")
    x[::3] = 0.0
    x[1::6] *= 2.0 ** -60 if io == "bf16" else 2.0 ** -12
    dX = check_xent(f"xentz/{io}/{ldt}", m, 500, d, 4, 1, io, ldt, ignored="none", x=x)[2]
    assert (to_f64(dX)[::3] != 0).any(1).all()


def test_xent_empty_batch():
    t = torch()
    gi, gl, _, _ = head("xente", 64, 64, 4, 1, "f16")
    X = t.zeros((0, 64), dtype=t.float16, device="cuda")
    T = t.zeros(0, dtype=t.int64, device="cuda")
    loss, lse = skm().sketch_xent_fwd(X, gi, gl, T, 4, 1)
    assert loss.numel() == 0 and lse.numel() == 0
    dX, dL = skm().sketch_xent_bwd(X, gi, gl, T, lse, lse, 4, 1)
    assert dX.shape == (0, 64) and (dL == 0).all()


# ---------------------------------------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------------------------------------

def test_another_stream():
    """Outputs and workspaces belong to the stream that is given."""
    t = torch()
    gi, gl, _, _ = head("xentst", 500, 256, 4, 2, "f16")
    X = t.randn((100, 256), device="cuda").half()
    T = t.randint(0, 500, (100,), device="cuda")
    DL = t.ones(100, device="cuda")
    want = skm().sketch_xent_fwd(X, gi, gl, T, 4, 2)
    wg = skm().sketch_xent_bwd(X, gi, gl, T, want[1], DL, 4, 2)
    wn = skm().sketch_norm_fwd(X, checkpoint=True)
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    got = skm().sketch_xent_fwd(X, gi, gl, T, 4, 2, stream=s)
    junk = [t.full((1 << 18,), 7.0, device="cuda") for _ in range(4)]
    gg = skm().sketch_xent_bwd(X, gi, gl, T, got[1], DL, 4, 2, stream=s)
    gn = skm().sketch_norm_fwd(X, checkpoint=True, stream=s)
    t.cuda.current_stream().wait_stream(s)
    for p, q in zip((*got, *gg, gn[0], *gn[3:]), (*want, *wg, wn[0], *wn[3:])):
        assert t.equal(p, q)
    assert all((j == 7.0).all() for j in junk)


def test_captured_step_replays():
    """norm with checkpoint, layer, loss and all gradients in one graph, replayed on new inputs between eager work."""
    t = torch()
    m, d, n, V = 64, 256, 256, 500
    gi, gl, _, _ = head("cap/w", n, d, 4, 2, "f16")
    hi, hl, _, _ = head("cap/h", V, n, 4, 2, "f16")
    W = t.randn(d, device="cuda")
    X = t.randn((m, d), device="cuda").half()
    T = t.randint(0, V, (m,), device="cuda")
    DL = t.full((m,), 1.0 / m * 1024, device="cuda")

    def step():
        k = skm()
        Y, mean, rstd, codes, scales = k.sketch_norm_fwd(X, W, kind="rms", checkpoint=True)
        Hd = k.sketch_matmul_fwd(Y, gi, gl, 4, 2)
        loss, lse = k.sketch_xent_fwd(Hd, hi, hl, T, 4, 2)
        dH, dLh = k.sketch_xent_bwd(Hd, hi, hl, T, lse, DL, 4, 2)
        dY, dLw = k.sketch_matmul_bwd_ckpt(dH, codes, scales, gi, gl, 4, 2)
        dX, dw, _ = k.sketch_norm_bwd(dY, X, W, mean, rstd, kind="rms", need_db=False)
        return loss, lse, dLh, dLw, dX, dw

    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        step()
    t.cuda.current_stream().wait_stream(side)
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        outs = step()
    for k in range(4):
        X.copy_(t.randn((m, d), device="cuda").half())
        T.copy_(t.randint(0, V, (m,), device="cuda"))
        T[k::7] = -100
        g.replay()
        got = [o.clone() for o in outs]
        want = step()
        t.cuda.synchronize()
        for p, q in zip(got, want):
            assert t.equal(p, q)


def test_offsets_past_32_bits():
    """More than 2^32 elements: the last rows of the whole give what those rows alone give."""
    t, k = torch(), skm()
    m, d = 131200, 32768
    X = t.zeros((m, d), dtype=t.bfloat16, device="cuda")
    X[-3:] = t.randn((3, d), device="cuda").bfloat16()
    Y, mean, rstd, codes, scales = k.sketch_norm_fwd(X, kind="rms", checkpoint=True)
    y, _, r, c, s = k.sketch_norm_fwd(X[-3:].contiguous(), kind="rms", checkpoint=True)
    assert t.equal(Y[-3:], y) and t.equal(rstd[-3:], r) and t.equal(codes[-3:], c) and t.equal(scales[-3:], s)
    back = k.sketch_act_dequant(codes, scales, t.bfloat16, out=Y)
    assert t.equal(back[-3:], k.sketch_act_dequant(c, s, t.bfloat16)) and not back[:-3].any()
    dX, dw, db = k.sketch_norm_bwd(X, X, None, None, rstd, kind="rms")
    dx = k.sketch_norm_bwd(X[-3:].contiguous(), X[-3:].contiguous(), None, None, r, kind="rms")
    assert t.equal(dX[-3:], dx[0]) and not dX[:-3].any()


def test_two_graphs_share_a_workspace():
    """A workspace holds nothing between calls: two captured calls of different sizes take turns on one."""
    t, k = torch(), skm()
    calls = []
    for name, m, V, d, b in (("a", 96, 700, 256, 4), ("b", 40, 300, 128, 3)):
        gi, gl, _, _ = head("share/" + name, V, d, b, 1, "f16")
        X = t.randn((m, d), device="cuda").half()
        T = t.randint(0, V, (m,), device="cuda")
        T[::5] = -100
        calls.append((X, gi, gl, T, b, 1))
    need = max(k.sketch_xent_bwd_workspace(X.shape[0], gi.shape[0], X.shape[1], b, 1, 1, 1)
               for X, gi, gl, T, b, _ in calls)
    need = max([need] + [k.sketch_xent_fwd_workspace(X.shape[0], gi.shape[0], X.shape[1], b, 1, 1, 1)
                         for X, gi, gl, T, b, _ in calls])
    ws = t.full((need,), 255, dtype=t.uint8, device="cuda")          # (NaN wherever a call reads before it writes)

    def run(c):
        loss, lse = k.sketch_xent_fwd(*c, workspace=ws)
        return (loss, lse, *k.sketch_xent_bwd(c[0], c[1], c[2], c[3], lse, t.ones_like(loss), c[4], c[5], workspace=ws))

    want = [[o.clone() for o in run(c)] for c in calls]
    graphs, outs = [], []
    for c in calls:
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            outs.append(run(c))
        graphs.append(g)
    for i in (0, 1, 1, 0, 1, 0):
        ws.fill_(255)
        graphs[i].replay()
        t.cuda.synchronize()
        assert all(t.equal(p, q) for p, q in zip(outs[i], want[i]))


def test_two_streams_at_once():
    """Calls on two streams with their own workspaces do not disturb each other."""
    t, k = torch(), skm()
    gi, gl, _, _ = head("two", 1000, 512, 4, 1, "f16")
    sets = []
    for i in range(2):
        X = t.randn((300, 512), device="cuda").half()
        T = t.randint(0, 1000, (300,), device="cuda")
        sets.append((X, gi, gl, T, 4, 1))
    DL = t.ones(300, device="cuda")
    want = []
    for c in sets:
        loss, lse = k.sketch_xent_fwd(*c)
        want.append((loss, *k.sketch_xent_bwd(c[0], gi, gl, c[3], lse, DL, 4, 1)))
    t.cuda.synchronize()
    streams = [t.cuda.Stream() for _ in sets]
    got = []
    for _ in range(3):
        got = []
        for c, s in zip(sets, streams):
            loss, lse = k.sketch_xent_fwd(*c, stream=s)
            got.append((loss, *k.sketch_xent_bwd(c[0], gi, gl, c[3], lse, DL, 4, 1, stream=s)))
    t.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(t.equal(p, q) for p, q in zip(g, w))
