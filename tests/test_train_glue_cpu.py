"""The autograd functions around checkpoints, norms and the head loss, without a GPU: the library's calls are replaced
by stand-ins that compute the same with torch and refuse what the library refuses (tensors that do not start at a
multiple of 16 bytes)."""
import pytest
import torch

from lut_sketched_matmul_amd import finetune


class Calls:
    """Stand-ins for the binding's calls; `log` names those that were made."""

    def __init__(self):
        self.log = []

    def made(self, name, *tensors):
        self.log.append(name)
        for t in tensors:
            if t is not None:
                assert t.is_contiguous() and t.data_ptr() % 16 == 0, f"{name}: pointer not 16-byte aligned"

    @staticmethod
    def weights(idx, lut, b, gpr):
        assert b == 4
        code = torch.stack([idx & 15, idx >> 4], 2).reshape(idx.shape[0], gpr, -1).long()
        return lut.float().gather(2, code).reshape(idx.shape[0], -1), code

    def sketch_matmul_fwd(self, X, idx, lut, b, gpr):
        self.made("matmul_fwd", X, idx, lut)
        return (X.float() @ self.weights(idx, lut, b, gpr)[0].T).to(X.dtype)

    def sketch_matmul_bwd(self, dY, X, idx, lut, b, gpr, d=None, need_dx=True, need_dlut=True):
        self.made("matmul_bwd", dY, X, idx, lut)
        W, code = self.weights(idx, lut, b, gpr)
        dL = None
        if need_dlut:
            dL = torch.zeros(lut.shape).scatter_add_(2, code, (dY.float().T @ X.float()).reshape(code.shape))
        return dY.float() @ W if need_dx else None, dL

    def sketch_act_quant(self, X):
        self.made("quant", X)
        return X.clone(), torch.zeros(1)

    def sketch_matmul_bwd_ckpt(self, dY, codes, scales, idx, lut, b, gpr, need_dx=True):
        self.made("bwd_ckpt", dY, codes)
        return self.sketch_matmul_bwd(dY, codes, idx, lut, b, gpr, need_dx=need_dx)

    def sketch_norm_fwd(self, X, weight=None, bias=None, kind="layer", eps=1e-5, checkpoint=False):
        self.made("norm_fwd_ckpt" if checkpoint else "norm_fwd", X, weight, bias)
        x = X.float()
        rstd = torch.rsqrt((x * x).mean(1) + eps)
        Y = (x * rstd[:, None] * weight).to(X.dtype)
        return Y, None, rstd, Y.clone() if checkpoint else None, torch.zeros(1) if checkpoint else None

    def sketch_norm_bwd(self, dY, X, weight, mean, rstd, kind="layer", need_dx=True, need_dw=True, need_db=True,
                        x_dtype=None):
        self.made("norm_bwd_ckpt" if isinstance(X, tuple) else "norm_bwd", dY, X[0] if isinstance(X, tuple) else X)
        x = (X[0] if isinstance(X, tuple) else X).float()
        xh, g = x * rstd[:, None], dY.float() * weight
        dX = rstd[:, None] * (g - xh * (g * xh).mean(1, keepdim=True))
        return (dX.to(x_dtype or (X[0] if isinstance(X, tuple) else X).dtype) if need_dx else None,
                (dY.float() * xh).sum(0) if need_dw else None, None)

    def sketch_xent_fwd(self, X, idx, lut, targets, b, gpr, ignore_index=-100):
        self.made("xent_fwd", X, idx, lut)
        Z = X.float() @ self.weights(idx, lut, b, gpr)[0].T
        lse = torch.logsumexp(Z, 1)
        return lse - Z.gather(1, targets[:, None])[:, 0], lse

    def sketch_xent_bwd(self, X, idx, lut, targets, lse, dloss, b, gpr, ignore_index=-100, need_dx=True,
                        need_dlut=True):
        self.made("xent_bwd", X, idx, lut, lse, dloss)
        W, code = self.weights(idx, lut, b, gpr)
        dZ = torch.exp(X.float() @ W.T - lse[:, None])
        dZ = (dZ - torch.nn.functional.one_hot(targets, idx.shape[0])) * dloss[:, None]
        dL = torch.zeros(lut.shape).scatter_add_(2, code, (dZ.T @ X.float()).reshape(code.shape)) if need_dlut else None
        return (dZ @ W).to(X.dtype) if need_dx else None, dL


@pytest.fixture
def calls(monkeypatch):
    c = Calls()
    for name in dir(Calls):
        if name.startswith("sketch_"):
            monkeypatch.setattr(finetune._lib, name, getattr(c, name))
    return c


def sketch(n, d, gpr, seed):
    g = torch.Generator().manual_seed(seed)
    idx = torch.randint(0, 256, (n, d // 2), generator=g, dtype=torch.uint8)
    return idx, torch.randn((n, gpr, 16), generator=g)


def normal(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def apart(t):
    """The same values in a contiguous tensor that starts 4 bytes after a multiple of 16."""
    buf = torch.empty(t.numel() + 4 // t.element_size(), dtype=t.dtype)
    buf[4 // t.element_size():] = t.reshape(-1)
    v = buf[4 // t.element_size():].reshape(t.shape)
    assert v.is_contiguous() and v.data_ptr() % 16 == 4
    return v


def test_losses_of_two_batches_joined(calls):
    """autograd gives the second batch the rest of one vector, 3 floats after its start."""
    idx, lut = sketch(11, 32, 1, 0)
    head = finetune.SketchedHead(idx, lut, 32, 4, 1)
    A, B = normal((3, 32), 1).half().requires_grad_(), normal((5, 32), 2).half().requires_grad_()
    T = torch.arange(8)
    w = normal((8,), 3)
    (torch.cat([head.token_losses(A, T[:3]), head.token_losses(B, T[3:])]) * w).sum().backward()
    ga, gb, gl = A.grad, B.grad, head.lut_master.grad
    head.lut_master.grad = None
    both = torch.cat([A, B]).detach().requires_grad_()
    (head.token_losses(both, T) * w).sum().backward()
    assert torch.equal(torch.cat([ga, gb]), both.grad)
    assert torch.allclose(gl, head.lut_master.grad, rtol=1e-5, atol=1e-6)
    assert calls.log.count("xent_bwd") == 3


@pytest.mark.parametrize("checkpoint", [False, True])
def test_layers_of_two_batches_joined(calls, checkpoint):
    """7 outputs a row: the second batch's output gradient starts 21 values after the first one's."""
    idx, lut = sketch(7, 32, 1, 4)
    layer = finetune.SketchedLinear(idx, lut, 32, 4, 1, compute_dtype=torch.float32, checkpoint=checkpoint)
    normed = finetune.SketchedLinear(idx, lut, 32, 4, 1, compute_dtype=torch.float32, checkpoint=checkpoint,
                                     norm=finetune.SketchNorm(32, "rms", device="cpu"))
    for f in (layer, normed):
        A, B = normal((3, 32), 5).requires_grad_(), normal((5, 32), 6).requires_grad_()
        torch.autograd.backward([torch.cat([f(A), f(B)])], [normal((8, 7), 7)])
        both = torch.cat([A, B]).detach().requires_grad_()
        f(both).backward(normal((8, 7), 7))
        assert torch.allclose(torch.cat([A.grad, B.grad]), both.grad, rtol=1e-5, atol=1e-6)


def test_norms_of_two_batches_joined(calls):
    norm = finetune.SketchNorm(7, "rms", device="cpu")
    A, B = normal((3, 7), 8).requires_grad_(), normal((5, 7), 9).requires_grad_()
    torch.autograd.backward([torch.cat([norm(A), norm(B)])], [normal((8, 7), 10)])
    both = torch.cat([A, B]).detach().requires_grad_()
    norm(both).backward(normal((8, 7), 10))
    assert torch.allclose(torch.cat([A.grad, B.grad]), both.grad, rtol=1e-5, atol=1e-6)


def test_inputs_that_start_anywhere(calls):
    idx, lut = sketch(8, 32, 1, 11)
    x = normal((3, 32), 12)
    for f in (finetune.SketchedLinear(idx, lut, 32, 4, 1, compute_dtype=torch.float32),
              finetune.SketchedLinear(idx, lut, 32, 4, 1, compute_dtype=torch.float32, checkpoint=True),
              finetune.SketchedLinear(idx, lut, 32, 4, 1, compute_dtype=torch.float32, checkpoint=True,
                                      norm=finetune.SketchNorm(32, "rms", device="cpu")),
              finetune.SketchNorm(32, "rms", device="cpu")):
        X, want = apart(x).requires_grad_(), x.clone().requires_grad_()
        Y, Z = f(X), f(want)
        assert torch.equal(Y, Z)
        Y.backward(apart(torch.ones_like(Y)))
        Z.backward(torch.ones_like(Z))
        assert torch.equal(X.grad, want.grad)
    h = x.half()
    head = finetune.SketchedHead(idx, lut, 32, 4, 1)
    X, want = apart(h).requires_grad_(), h.clone().requires_grad_()
    T = torch.arange(3)
    head.token_losses(X, T).sum().backward()
    head.token_losses(want, T).sum().backward()
    assert torch.equal(X.grad, want.grad)


def test_checkpoint_is_for_the_table_gradient(calls):
    """Frozen tables: nothing is quantised and the gradients of X and of the norm are those of X itself."""
    idx, lut = sketch(8, 32, 1, 13)
    x, dY = normal((4, 32), 14), normal((4, 8), 15)
    grads = []
    for checkpoint in (False, True):
        norm = finetune.SketchNorm(32, "rms", device="cpu")
        layer = finetune.SketchedLinear(idx, lut, 32, 4, 1, compute_dtype=torch.float32, checkpoint=checkpoint, norm=norm)
        layer.lut_master.requires_grad_(False)
        X = x.clone().requires_grad_()
        layer(X).backward(dY)
        grads.append((X.grad, norm.weight.grad))
    assert all(torch.equal(p, q) for p, q in zip(*grads))
    assert "norm_bwd" in calls.log and not {"quant", "norm_fwd_ckpt", "norm_bwd_ckpt"} & set(calls.log)
    # trained tables: both checkpoints, as asked for
    layer.lut_master.requires_grad_(True)
    layer(x.clone().requires_grad_()).backward(dY)
    assert {"quant", "norm_fwd_ckpt", "norm_bwd_ckpt"} <= set(calls.log)


def test_nothing_is_kept_without_gradients(calls):
    """Under no_grad a checkpointed layer does the plain layer's calls: there is no backward to keep anything for."""
    idx, lut = sketch(8, 32, 1, 16)
    x = normal((4, 32), 17)
    layer = finetune.SketchedLinear(idx, lut, 32, 4, 1, compute_dtype=torch.float32, checkpoint=True)
    normed = finetune.SketchedLinear(idx, lut, 32, 4, 1, compute_dtype=torch.float32, checkpoint=True,
                                     norm=finetune.SketchNorm(32, "rms", device="cpu"))
    with torch.no_grad():
        layer(x)
        normed(x)
    assert calls.log == ["matmul_fwd", "norm_fwd", "matmul_fwd"]


def test_head_of_an_empty_batch(calls, monkeypatch):
    """No token is scored: loss 0, gradients 0, as for a batch whose every target is ignored."""
    monkeypatch.setattr(finetune._lib, "sketch_xent_mean", lambda *a, **k: pytest.fail("takes at least one token"))
    idx, lut = sketch(8, 32, 1, 18)
    head = finetune.SketchedHead(idx, lut, 32, 4, 1)
    X = torch.zeros((0, 32), dtype=torch.float16, requires_grad=True)
    loss = head(X, torch.zeros(0, dtype=torch.int64))
    assert loss.dim() == 0 and loss.dtype == torch.float32 and float(loss.detach()) == 0.0
    loss.backward()
    assert X.grad.shape == (0, 32) and (head.lut_master.grad == 0).all()
