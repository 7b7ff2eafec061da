"""Pins of ``oracle/train_oracle.py`` (CPU): hand-worked cases, differences, torch's own modules in float64."""
import numpy as np
import pytest
import torch

from oracle import train_oracle as to


def rng(seed):
    return np.random.default_rng(seed)


def test_checkpoint_hand_worked():
    """127 needs step 1, 127.5 and 128 step 2 (64 codes of 2), 63.5 step 1/2; ties round to even."""
    x = np.zeros((1, 128))
    x[0, :4] = [127.0, 0.5, 1.5, -2.5]
    x[0, 32:36] = [128.0, 1.0, 3.0, -5.0]
    x[0, 64:66] = [63.5, 0.25]
    codes, scales = to.act_quant(x, "bf16")
    assert list(scales[0]) == [127, 128, 126, 1]
    assert list(codes[0, :4]) == [127, 0, 2, -2]
    assert list(codes[0, 32:36]) == [64, 0, 2, -2]
    assert list(codes[0, 64:66]) == [127, 0]
    assert np.array_equal(to.act_dequant(codes, scales)[0, 32:36], [128.0, 0.0, 4.0, -4.0])


def test_checkpoint_bounds_of_the_range():
    """f16: 65504 takes step 2^9 and the largest code; the smallest subnormal is kept; bf16's largest stays finite."""
    x = np.zeros((1, 64))
    x[0, 0], x[0, 32] = 65504.0, 2.0 ** -24
    codes, scales = to.act_quant(x, "f16")
    assert list(scales[0]) == [136, 103] and codes[0, 0] == 127 and codes[0, 32] == 1
    assert to.act_dequant(codes, scales)[0, 0] == 65024.0
    x[0, 0], x[0, 32] = (2.0 - 2.0 ** -7) * 2.0 ** 127, 2.0 ** -130
    codes, scales = to.act_quant(x, "bf16")
    v = to.act_dequant(codes, scales)
    assert v[0, 0] == 127 * 2.0 ** 121 and v[0, 32] == 0.0


def test_checkpoint_error_is_half_a_step_and_nonfinite_blocks_are_nan():
    x = rng(1).standard_normal((7, 96)) * np.exp(3 * rng(2).standard_normal((7, 1)))
    codes, scales = to.act_quant(x, "f32")
    step = np.repeat(2.0 ** (scales.astype(float) - 127), 32, axis=1)
    v = to.act_dequant(codes, scales)
    assert np.all(np.abs(v - x) <= step / 2)
    assert np.all(np.abs(x).reshape(7, 3, 32).max(2) > 127 * 2.0 ** (scales.astype(float) - 128))  # smallest such step
    x[3, 40] = np.inf
    x[5, 95] = np.nan
    codes, scales = to.act_quant(x, "f32")
    v = to.act_dequant(codes, scales)
    assert np.isnan(v[3, 32:64]).all() and np.isnan(v[5, 64:]).all()
    assert np.isfinite(v).sum() == v.size - 64


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_matches_torch_and_differences(kind):
    g = rng(3)
    X, w, b, dY = g.standard_normal((5, 17)), g.standard_normal(17), g.standard_normal(17), g.standard_normal((5, 17))
    b = b if kind == "layer" else None
    Y, mean, rstd = to.norm_fwd(X, w, b, kind, 1e-3)
    xt, wt = torch.tensor(X, requires_grad=True), torch.tensor(w, requires_grad=True)
    bt = torch.tensor(b, requires_grad=True) if b is not None else None
    if kind == "layer":
        y = torch.nn.functional.layer_norm(xt, (17,), wt, bt, 1e-3)
    else:
        y = torch.nn.functional.rms_norm(xt, (17,), wt, 1e-3)
    assert np.allclose(Y, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    y.backward(torch.tensor(dY))
    dX, dw, db = to.norm_bwd(dY, X, w, mean, rstd, kind)
    assert np.allclose(dX, xt.grad.numpy(), rtol=1e-11, atol=1e-12)
    assert np.allclose(dw, wt.grad.numpy(), rtol=1e-11, atol=1e-12)
    if bt is not None:
        assert np.allclose(db, bt.grad.numpy(), rtol=1e-11, atol=1e-12)
    h = 1e-6
    for t, j in ((0, 0), (2, 9), (4, 16)):
        P, M = X.copy(), X.copy()
        P[t, j] += h
        M[t, j] -= h
        num = ((to.norm_fwd(P, w, b, kind, 1e-3)[0] - to.norm_fwd(M, w, b, kind, 1e-3)[0]) * dY).sum() / (2 * h)
        assert abs(num - dX[t, j]) < 1e-7


def test_xent_matches_torch_and_differences():
    g = rng(4)
    Z = g.standard_normal((6, 11)) * 3
    targets = np.array([0, 10, -100, 4, 4, -100])
    loss, lse = to.xent_fwd(Z, targets)
    zt = torch.tensor(Z, requires_grad=True)
    ref = torch.nn.functional.cross_entropy(zt, torch.tensor(targets), reduction="none", ignore_index=-100)
    assert np.allclose(loss, ref.detach().numpy(), rtol=1e-13, atol=1e-13)
    w = g.standard_normal(6)
    ref.backward(torch.tensor(w))
    dZ = to.xent_dz(Z, targets, lse, w)
    assert np.allclose(dZ, zt.grad.numpy(), rtol=1e-12, atol=1e-14)
    h = 1e-6
    for t, v in ((0, 0), (1, 3), (3, 4)):
        P, M = Z.copy(), Z.copy()
        P[t, v] += h
        M[t, v] -= h
        num = ((to.xent_fwd(P, targets)[0] - to.xent_fwd(M, targets)[0]) * w).sum() / (2 * h)
        assert abs(num - dZ[t, v]) < 1e-8


def test_xent_targets_outside_the_vocabulary_are_nan():
    Z = np.zeros((3, 4))
    targets = np.array([4, -1, 2])
    loss, lse = to.xent_fwd(Z, targets)
    assert np.isnan(loss[:2]).all() and abs(loss[2] - np.log(4)) < 1e-15 and np.allclose(lse, np.log(4))
    dZ = to.xent_dz(Z, targets, lse, np.ones(3))
    assert np.isnan(dZ[:2]).all() and np.allclose(dZ[2], [0.25, 0.25, -0.75, 0.25])
