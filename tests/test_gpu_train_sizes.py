"""GPU tests of the training operators at the ends of their ranges: the most tokens, more than 2^32 values."""
import numpy as np
import pytest

import oracle
from lut_sketched_matmul_amd import synthetic as syn

from gpu_util import to_dev, to_f64

pytestmark = pytest.mark.gpu


def skm():
    import lut_sketched_matmul_amd as m
    return m


def torch():
    import torch as _t
    return _t


def near(got, want, rel, what):
    got, want = to_f64(got), np.asarray(want)
    assert np.linalg.norm(got - want) <= rel * np.linalg.norm(want), what


@pytest.mark.parametrize("m,V,d", [
    ((1 << 22) - 16, 3, 1056),      # few words: 16 tokens per block
    (1 << 22, 3, 1056),             # the most tokens
    ((1 << 20) + 8, 40, 4160),      # 256 x 256 tiles
])
def test_xent_of_more_than_2_32_values(m, V, d):
    """Rows of zeros but the last three: their results are the formula's, the others' those of equal logits."""
    t, k = torch(), skm()
    idx = syn.random_packed_indices(f"sizes/{V}/i", V, d, 4)
    lut = syn.random_lut(f"sizes/{V}/l", V, 1, 4, 0.05, "f16")
    W = oracle.dequantize(idx, syn.to_float64(lut, "f16"), d, 4, 1)
    gi, gl = to_dev(idx, "u8"), to_dev(lut, "f16")
    X = t.zeros((m, d), dtype=t.float16, device="cuda")
    X[-3:] = to_dev(syn.random_normal(f"sizes/{V}/x", (3, d), 1.0, "f16"), "f16")
    x = to_f64(X[-3:])
    T = t.arange(m, device="cuda") % V
    loss, lse = k.sketch_xent_fwd(X, gi, gl, T, 4, 1)
    last = T[-3:].cpu().numpy()
    Z = x @ W.T
    rl = np.log(np.exp(Z - Z.max(1, keepdims=True)).sum(1)) + Z.max(1)
    near(lse[-3:], rl, 2.0 ** -18, "lse")
    near(loss[-3:], rl - Z[np.arange(3), last], 2.0 ** -16, "loss")
    assert (loss[:-3] == loss[0]).all() and abs(float(loss[0]) - np.log(V)) <= 2.0 ** -22 * np.log(V)
    dX, dL = k.sketch_xent_bwd(X, gi, gl, T, lse, t.ones(m, device="cuda"), 4, 1)
    P = np.exp(Z - rl[:, None])
    P[np.arange(3), last] -= 1.0
    # three roundings to 16 bits at the most: a norm of 2^-10
    near(dX[-3:], P @ W, 2.0 ** -10, "dX")
    for r in (0, 1, m // 2, m - 4):
        near(dX[r], W.mean(0) - W[r % V], 2.0 ** -10, f"dX of row {r}")
    assert t.equal(dX[(m // 2) // V * V], dX[0])
    near(dL, oracle.backward_dlut(P, x, idx, 4, 1), 2.0 ** -16, "dLUT")


def test_norm_gradients_of_more_than_2_32_values():
    """dw and db of rows of zeros but the last three are those of the three."""
    t, k = torch(), skm()
    m, d = 131200, 32768
    X = t.zeros((m, d), dtype=t.bfloat16, device="cuda")
    X[-3:] = to_dev(syn.random_normal("sizes/norm", (3, d), 1.0, "bf16"), "bf16")
    rstd = t.ones(m, device="cuda")
    dX, dw, db = k.sketch_norm_bwd(X, X, None, None, rstd, kind="rms")
    x = to_f64(X[-3:])
    near(dw, (x * x).sum(0), 2.0 ** -22, "dw")
    near(db, x.sum(0), 2.0 ** -22, "db")
    m, d = 1 << 21, 2056
    X = t.zeros((m, d), dtype=t.bfloat16, device="cuda")
    X[-3:] = to_dev(syn.random_normal("sizes/norm2", (3, d), 1.0, "bf16"), "bf16")
    dX, dw, db = k.sketch_norm_bwd(X, X, None, None, t.ones(m, device="cuda"), kind="rms")
    x = to_f64(X[-3:])
    near(dw, (x * x).sum(0), 2.0 ** -22, "dw")
    near(db, x.sum(0), 2.0 ** -22, "db")
    assert not dX[:-3].any()
