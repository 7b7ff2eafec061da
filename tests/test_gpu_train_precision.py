"""GPU tests of what the training operators keep of their operands: bounds derived term by term, in float64.

U = 2^-24 is half a step of fp32, h(t) = finfo(t).eps / 2 half a relative step of a 16-bit type. An f16 operand that
was scaled so that the largest factor lies in [2^14, 2^15) is off by h(f16) of itself or, below 2^-14, by 2^-25, which
is at most 2^-39 of that factor.
"""
import numpy as np
import pytest

import oracle
from lut_sketched_matmul_amd import synthetic as syn
from oracle import train_oracle as to

from gpu_util import to_dev, to_f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
H = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 0.0}
PAIRS = [("f16", "f16"), ("bf16", "f16"), ("bf16", "bf16")]


def skm():
    import lut_sketched_matmul_amd as m
    return m


def torch():
    import torch as _t
    return _t


def head(name, V, d, b, gpr, ldt, sigma=0.05):
    idx = syn.random_packed_indices(name + "/i", V, d, b)
    lut = syn.random_lut(name + "/l", V, gpr, b, sigma, ldt)
    W = oracle.dequantize(idx, syn.to_float64(lut, ldt), d, b, gpr)
    return to_dev(idx, "u8"), to_dev(lut, ldt), idx, W


def inputs(x, io):
    s = syn.to_storage(x.astype(np.float32), io)
    return to_dev(s, io), syn.to_float64(s, io)


def within(got, ref, bound, what):
    assert got.shape == ref.shape and np.isfinite(got).all(), what
    off = np.abs(got - ref) - bound
    assert off.max() <= 0.0, f"{what}: {int((off > 0).sum())} of {off.size} over the bound by up to {off.max():.3e}"


def logit_error(x, W, io, ldt, d):
    """Of every token's logits: fp32 sums of d products, and f16 operands of prescaled bf16 rows."""
    dz = (d / 16 + 24) * U * (np.abs(x) @ np.abs(W).T).max(1)
    if (io, ldt) == ("bf16", "f16"):
        dz = dz + 2.0 ** -23 * np.abs(x).max(1) * np.abs(W).sum(1).max()
    return dz


def dz_error(P, w, lse, dz, T):
    """Of dZ in fp32: the softmax's argument and exp, relative to the softmax; the target's also the subtraction."""
    e = w[:, None] * P * (dz + 2 * U * np.abs(lse) + 60 * U)[:, None]
    e[np.arange(len(T)), T] += 4 * U * w
    return e


@pytest.mark.parametrize("ldt", ["f16", "bf16"])
@pytest.mark.parametrize("m", [24, 300])
@pytest.mark.parametrize("big", ["half", "one"])
def test_table_gradient_of_rows_around_a_quarter(m, ldt, big):
    """Every bf16 row gives the tables its dZ to 22 bits, whether its largest value lies just below or above 2^-2."""
    t = torch()
    V, d, b, gpr = 12000, 64, 4, 1
    name = f"quarter/{m}/{ldt}"
    gi, gl, idx, W = head(name, V, d, b, gpr, ldt)
    x = syn.to_float64(syn.random_normal(name + "/x", (m, d), 1.0, "f32"), "f32")
    top = np.where(np.arange(m) % 2 == 1, 0.26, 0.24) if big == "half" else np.where(np.arange(m) == m // 2, 0.26, 0.24)
    X, x = inputs(x * (top / np.abs(x).max(1))[:, None], "bf16")
    T = syn.rng_for(name + "/t").integers(0, V, size=m)
    w = np.ones(m)
    gt = t.from_numpy(T).cuda()
    _, lse = skm().sketch_xent_fwd(X, gi, gl, gt, b, gpr)
    dL = skm().sketch_xent_bwd(X, gi, gl, gt, lse, t.ones(m, device="cuda"), b, gpr, need_dx=False)[1]
    l64 = to_f64(lse)
    Z = x @ W.T
    dZ = to.xent_dz(Z, T, l64, w)
    e = dz_error(np.exp(Z - l64[:, None]), w, l64, logit_error(x, W, "bf16", ldt, d), T)
    # the scale of an operand's row: its largest value in [2^14, 2^15); of dZ's row: the inverse, times one power of two
    step = np.exp2(np.floor(np.log2(np.abs(x).max(1))) - 14)
    op = e + 2.0 ** -22 * np.abs(dZ) + (2.0 ** -39 * (w * step).max() / step)[:, None]
    ref = oracle.backward_dlut(dZ, x, idx, b, gpr)
    mag = oracle.backward_dlut(np.abs(dZ), np.abs(x), idx, b, gpr)
    err = oracle.backward_dlut(op, np.abs(x), idx, b, gpr)
    err += oracle.backward_dlut(np.abs(dZ), np.repeat(2.0 ** -25 * step[:, None], d, 1), idx, b, gpr)
    within(to_f64(dL), ref, 1.01 * err + (2 * m / 16 + d // gpr + 40) * U * mag, "dLUT")


def check_dx(name, m, V, d, b, gpr, io, ldt, w, sigma=0.05, x=None, weights=None, need_dlut=False, others=None):
    """dX against float64, every token by its own dloss: H[ldt] of each term (`others` if given) but the target's (2^-22:
    it keeps its remainder in fp32) or 2^-39 of the token's |dloss|, where dX has an operand of its own."""
    t = torch()
    gi, gl, idx, W = weights if weights is not None else head(name, V, d, b, gpr, ldt, sigma)
    if x is None:
        x = syn.to_float64(syn.random_normal(name + "/x", (m, d), 1.0, "f32"), "f32")
    X, x = inputs(x, io)
    T = syn.rng_for(name + "/t").integers(0, V, size=m)
    gt = t.from_numpy(T).cuda()
    w = w.astype(np.float32).astype(np.float64)
    _, lse = skm().sketch_xent_fwd(X, gi, gl, gt, b, gpr)
    dX = skm().sketch_xent_bwd(X, gi, gl, gt, lse, t.from_numpy(w.astype(np.float32)).cuda(), b, gpr,
                               need_dlut=need_dlut)[0]
    l64 = to_f64(lse)
    Z = x @ W.T
    dZ = to.xent_dz(Z, T, l64, w)
    e = dz_error(np.exp(Z - l64[:, None]), np.abs(w), l64, logit_error(x, W, io, ldt, d), T)
    keep = np.full(dZ.shape, H[ldt] if others is None else others)
    keep[np.arange(m), T] = 2.0 ** -22
    op = e + keep * (np.abs(dZ) + e) + (2.0 ** -39 * np.abs(w)[:, None] if ldt == "f16" else 0.0)
    ref = dZ @ W
    # fp32 sums of V terms: 16 at a time, the pieces, the ranges
    err = op @ np.abs(W) + (V / 16 + 64) * U * (np.abs(dZ) @ np.abs(W))
    bound = 1.01 * err + H[io] * (np.abs(ref) + err) + TINY[io]
    within(to_f64(dX), ref, bound, "dX")
    return dZ[np.arange(m), T], W[T], bound


@pytest.mark.parametrize("m", [24, 300])
@pytest.mark.parametrize("io,ldt,need_dlut,hi,lo", [
    ("f16", "f16", False, 15, -12), ("bf16", "f16", False, 20, -60), ("bf16", "f16", True, 20, -60),
    ("bf16", "bf16", False, 20, -60),
])
def test_dx_of_tokens_with_far_weights(io, ldt, need_dlut, hi, lo, m):
    """A token's dX is as precise beside a token of 2^80 times its weight as alone."""
    w = np.exp2(np.linspace(hi, lo, m))
    w[1::2] *= -1.0
    check_dx(f"farw/{io}/{ldt}/{m}", m, 9000, 64, 4, 1, io, ldt, w, need_dlut=need_dlut)


@pytest.mark.parametrize("m", [20, 700])
@pytest.mark.parametrize("io,ldt,V", [("f16", "f16", 4096), ("bf16", "f16", 4096), ("bf16", "bf16", 1024)])
def test_dx_keeps_the_targets_remainder(io, ldt, V, m):
    """Rows of zeros against words near 4: dX = mean(W) - W[target], the small difference of two large terms. The
    softmax 1 / V is exact in 16 bits and 1 / V - 1 is not, so only its remainder saves the difference."""
    d, b = 64, 4
    g = syn.rng_for(f"rest/{ldt}")
    idx = syn.random_packed_indices(f"rest/{ldt}/i", V, d, b)
    lut = syn.to_storage((4.0 + g.integers(-2, 3, size=(V, 1, 16)) * 2.0 ** -5).astype(np.float32), ldt)
    W = oracle.dequantize(idx, syn.to_float64(lut, ldt), d, b, 1)
    dz, wt, bound = check_dx(f"rest/{io}/{ldt}/{m}", m, V, d, b, 1, io, ldt, np.ones(m), x=np.zeros((m, d)),
                             weights=(to_dev(idx, "u8"), to_dev(lut, ldt), idx, W), need_dlut=m == 20, others=0.0)
    # (the bound tells: the target's term rounded like the others would be outside it)
    r = syn.to_float64(syn.to_storage((dz * 0.999999).astype(np.float32), ldt), ldt) - dz
    assert (np.abs(r[:, None] * wt) > 2 * bound).all()


@pytest.mark.parametrize("d", [7, 41, 56, 97, 112, 1001, 1792, 4280, 4512, 8560, 9024, 14336, 16826, 20000])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_norm_of_constant_rows_is_exact(d, dtype):
    """The sums of 1000s and 4s are exact, so their means are, wherever the mean is a quotient rounded once: no
    variance, y = bias, 1 / rms = 1 / 2; and the backward's mean of a constant g takes all of it away."""
    t = torch()
    X = to_dev(syn.to_storage(np.full((5, d), 1000.0, np.float32), dtype), dtype)
    B = to_dev(syn.random_normal(f"const/{d}", (d,), 1.0, "f32"), "f32")
    Y, mean, rstd, _, _ = skm().sketch_norm_fwd(X, None, B, kind="layer", eps=1e-5)
    assert (mean == 1000.0).all() and t.equal(Y, B.to(Y.dtype).expand(5, d))
    assert (rstd == rstd[0]).all() and abs(float(rstd[0]) * 1e-5 ** 0.5 - 1.0) <= 4 * U
    dX, dw, db = skm().sketch_norm_bwd(t.full((5, d), 3.0, device="cuda"), X, None, mean, rstd, kind="layer")
    assert (dX == 0).all() and (dw == 0).all() and (db == 15.0).all()
    X = to_dev(syn.to_storage(np.full((5, d), -2.0, np.float32), dtype), dtype)
    Y, mean, rstd, _, _ = skm().sketch_norm_fwd(X, kind="rms", eps=0.0)
    assert mean is None and (rstd == 0.5).all() and (Y == -1.0).all()
    # g xh = -3 in every column: mean(g xh) = -3 and dx = r (g - xh mean(g xh)) = 0
    dX = skm().sketch_norm_bwd(t.full((5, d), 3.0, device="cuda"), X, None, None, rstd, kind="rms")[0]
    assert (dX == 0).all()
