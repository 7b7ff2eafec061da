"""GPU tests of the fine-tuning modules on the tensors autograd and slicing hand out (contiguous, starting anywhere)."""
import pytest

from lut_sketched_matmul_amd import synthetic as syn

from gpu_util import to_dev

pytestmark = pytest.mark.gpu


def torch():
    import torch as _t
    return _t


def ft():
    from lut_sketched_matmul_amd import finetune
    return finetune


def sketch(name, n, d, b, gpr):
    return (to_dev(syn.random_packed_indices(name + "/i", n, d, b), "u8"),
            to_dev(syn.random_lut(name + "/l", n, gpr, b, 0.05, "f16"), "f16"))


def test_losses_of_two_batches_joined():
    t = torch()
    gi, gl = sketch("joined", 300, 128, 4, 1)
    head = ft().SketchedHead(gi, gl, 128, 4, 1)
    X = to_dev(syn.random_normal("joined/x", (8, 128), 1.0, "f16"), "f16")
    T = t.arange(8, device="cuda") * 7
    w = to_dev(syn.random_normal("joined/w", (8,), 1.0, "f32"), "f32")
    A, B, both = X[:3].clone().requires_grad_(), X[3:].clone().requires_grad_(), X.clone().requires_grad_()
    (t.cat([head.token_losses(A, T[:3]), head.token_losses(B, T[3:])]) * w).sum().backward()
    tables, head.lut_master.grad = head.lut_master.grad, None
    (head.token_losses(both, T) * w).sum().backward()
    want = head.lut_master.grad
    # one sum of 8 tokens instead of two of 3 and 5, and f16 operands under another power of two: bits at the end
    assert float((t.cat([A.grad, B.grad]) - both.grad).float().norm()) <= 2.0 ** -10 * float(both.grad.float().norm())
    assert float((tables - want).norm()) <= 2.0 ** -18 * float(want.norm())


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_of_slices_of_a_ragged_width(kind):
    """Rows of 1001 f16 values: a slice of the input and the second batch's gradient start at odd rows."""
    t = torch()
    norm = ft().SketchNorm(1001, kind)
    X = to_dev(syn.random_normal("slices/x", (8, 1001), 1.0, "f16"), "f16")
    G = to_dev(syn.random_normal("slices/g", (8, 1001), 1.0, "f16"), "f16")
    both = X.clone().requires_grad_()
    norm(both).backward(G)
    want = norm.weight.grad
    norm.weight.grad = None
    parts = X.clone().requires_grad_()
    t.cat([norm(parts[:3]), norm(parts[3:])]).backward(G)
    assert t.equal(parts.grad, both.grad)
    assert float((norm.weight.grad - want).norm()) <= 2.0 ** -20 * float(want.norm())


def test_layer_of_an_odd_number_of_outputs():
    t = torch()
    gi, gl = sketch("oddout", 7, 256, 3, 2)
    layer = ft().SketchedLinear(gi, gl, 256, 3, 2, checkpoint=True, norm=ft().SketchNorm(256, "rms"))
    X = to_dev(syn.random_normal("oddout/x", (8, 256), 1.0, "f16"), "f16")
    G = to_dev(syn.random_normal("oddout/g", (8, 7), 1.0, "f16"), "f16")
    both, parts = X.clone().requires_grad_(), X.clone().requires_grad_()
    layer(both).backward(G)
    want, layer.lut_master.grad = layer.lut_master.grad, None
    t.cat([layer(parts[:3]), layer(parts[3:])]).backward(G)
    assert float((parts.grad - both.grad).float().norm()) <= 2.0 ** -10 * float(both.grad.float().norm())
    assert float((layer.lut_master.grad - want).norm()) <= 2.0 ** -18 * float(want.norm())


def test_head_of_an_empty_batch():
    t = torch()
    gi, gl = sketch("emptyhead", 40, 64, 4, 1)
    head = ft().SketchedHead(gi, gl, 64, 4, 1, norm=ft().SketchNorm(64))
    X = t.zeros((0, 64), dtype=t.float16, device="cuda", requires_grad=True)
    loss = head(X, t.zeros(0, dtype=t.int64, device="cuda"))
    loss.backward()
    assert float(loss.detach()) == 0.0 and X.grad.shape == (0, 64)
    assert (head.lut_master.grad == 0).all() and (head.norm.weight.grad == 0).all()
