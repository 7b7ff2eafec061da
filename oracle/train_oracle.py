"""CPU oracle of the operators around the sketched layers (float64, numpy).

TEST INFRASTRUCTURE, like ``sketch_oracle``: only the tests import it, and it
shares no code with the library.

* 8-bit checkpoint: per block of 32 columns the smallest integer e with
  127 2^e >= max|x| (bounded by the dtype), q = rint(x 2^-e) in [-127, 127].
* Layer norm and root-mean-square norm, their gradients from the definition.
* Softmax cross entropy of logits Z = X W^T: lse, loss, dZ.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
NAN_BLOCK = 255
RANGE = {"f16": (-24, 9), "bf16": (-126, 121), "f32": (-126, 121)}


def act_quant(X: np.ndarray, dtype: str):
    """(codes int8 [m, d], scales uint8 [m, d/32]) of X (float64 values of `dtype`)."""
    lo, hi = RANGE[dtype]
    m, d = X.shape
    codes = np.zeros((m, d), np.int8)
    scales = np.zeros((m, d // BLOCK), np.uint8)
    for t in range(m):
        for g in range(d // BLOCK):
            x = X[t, g * BLOCK:(g + 1) * BLOCK]
            if not np.all(np.isfinite(x)):
                scales[t, g] = NAN_BLOCK
                continue
            top = float(np.max(np.abs(x)))
            e = lo
            while e < hi and np.ldexp(127.0, e) < top:
                e += 1
            q = np.clip(np.rint(np.ldexp(x, -e)), -127, 127)
            codes[t, g * BLOCK:(g + 1) * BLOCK] = q.astype(np.int8)
            scales[t, g] = e + 127
    return codes, scales


def act_dequant(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    m, d = codes.shape
    s = np.repeat(scales.astype(np.int64), BLOCK, axis=1)
    v = np.ldexp(codes.astype(np.float64), s - 127)
    return np.where(s == NAN_BLOCK, np.nan, v)


def norm_fwd(X, weight=None, bias=None, kind="layer", eps=1e-5):
    """(Y, mean, rstd); mean is zeros for kind "rms"."""
    d = X.shape[1]
    mean = X.sum(1) / d if kind == "layer" else np.zeros(X.shape[0])
    c = X - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).sum(1) / d + eps)
    Y = c * rstd[:, None]
    if weight is not None:
        Y = Y * weight
    if bias is not None:
        Y = Y + bias
    return Y, mean, rstd


def norm_bwd(dY, X, weight, mean, rstd, kind="layer"):
    """(dX, dweight, dbias) from the given statistics."""
    d = X.shape[1]
    xh = (X - (mean[:, None] if kind == "layer" else 0.0)) * rstd[:, None]
    g = dY if weight is None else dY * weight
    t = g - xh * ((g * xh).sum(1, keepdims=True) / d)
    if kind == "layer":
        t = t - g.sum(1, keepdims=True) / d
    return t * rstd[:, None], (dY * xh).sum(0), dY.sum(0)


def xent_fwd(Z, targets, ignore_index=-100):
    """(loss, lse) per token of the logits Z [m, V]."""
    m, V = Z.shape
    loss, lse = np.zeros(m), np.zeros(m)
    for t in range(m):
        if targets[t] == ignore_index:
            continue
        top = Z[t].max()
        lse[t] = top + np.log(np.exp(Z[t] - top).sum())
        loss[t] = lse[t] - Z[t, targets[t]] if 0 <= targets[t] < V else np.nan
    return loss, lse


def xent_dz(Z, targets, lse, dloss, ignore_index=-100):
    """dZ [m, V]: dloss (softmax - onehot), zeros for ignored tokens, NaN for targets outside [0, V)."""
    m, V = Z.shape
    dZ = np.zeros((m, V))
    for t in range(m):
        if targets[t] == ignore_index:
            continue
        if not 0 <= targets[t] < V:
            dZ[t] = np.nan
            continue
        p = np.exp(Z[t] - lse[t])
        p[targets[t]] -= 1.0
        dZ[t] = dloss[t] * p
    return dZ
