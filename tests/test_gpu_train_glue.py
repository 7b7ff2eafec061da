"""GPU tests of the fine-tuning modules around norms, 8-bit checkpoints and the head loss.

The library calls are scored against float64 in ``test_gpu_train.py``; here the modules must give exactly what
those calls give, gradients must agree with central differences, and a whole step must run, train its
parameters with the fused optimizers and agree with a float64 model.
"""
import numpy as np
import pytest

import oracle
from lut_sketched_matmul_amd import synthetic as syn

from gpu_util import to_dev, to_f64

pytestmark = pytest.mark.gpu


def skm():
    import lut_sketched_matmul_amd as m
    return m


def ft():
    from lut_sketched_matmul_amd import finetune
    return finetune


def torch():
    import torch as _t
    return _t


def tdtype(name):
    t = torch()
    return {"f32": t.float32, "f16": t.float16, "bf16": t.bfloat16}[name]


def sketch(name, n, d, b, gpr, ldt="f16", sigma=0.05):
    idx = syn.random_packed_indices(name + "/i", n, d, b)
    lut = syn.random_lut(name + "/l", n, gpr, b, sigma, ldt)
    return idx, lut, to_dev(idx, "u8"), to_dev(lut, ldt)


def normal(name, shape, dtype, sigma=1.0):
    return to_dev(syn.random_normal(name, shape, sigma, dtype), dtype)


PAIRS = [("f16", "f16"), ("bf16", "f16"), ("bf16", "bf16"), ("f32", "f32")]


@pytest.mark.parametrize("io,ldt", PAIRS)
def test_checkpointed_linear_is_its_calls(io, ldt):
    t = torch()
    n, d, b, gpr, m = 96, 256, 4, 2, 37
    _, _, gi, gl = sketch(f"ckl/{ldt}", n, d, b, gpr, ldt)
    X, dY = normal("ckl/x", (m, d), io).requires_grad_(), normal("ckl/y", (m, n), io)
    plain = ft().SketchedLinear(gi, gl, d, b, gpr, compute_dtype=tdtype(ldt))
    layer = ft().SketchedLinear(gi, gl, d, b, gpr, compute_dtype=tdtype(ldt), checkpoint=True)
    assert t.equal(layer(X), plain(X))
    layer(X).backward(dY)
    codes, scales = skm().sketch_act_quant(X.detach())
    dX, dL = skm().sketch_matmul_bwd_ckpt(dY, codes, scales, gi, layer.compute_tables(), b, gpr)
    assert t.equal(X.grad, dX.to(X.dtype)) and t.equal(layer.lut_master.grad, dL)
    # frozen tables: no checkpoint, the same input gradient up to the order of its sums
    X.grad = None
    layer.lut_master.requires_grad_(False)
    layer(X).backward(dY)
    want = skm().sketch_matmul_bwd(dY, None, gi, layer.compute_tables(), b, gpr, d=d, need_dlut=False)[0]
    assert t.equal(X.grad, want.to(X.dtype))
    # the input needs no gradient
    layer.lut_master.requires_grad_(True)
    layer.lut_master.grad = None
    layer(X.detach()).backward(dY)
    assert t.equal(layer.lut_master.grad, dL)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("io,ldt", PAIRS)
def test_normed_layers_are_their_calls(io, ldt, checkpoint, kind):
    t, k = torch(), skm()
    n, d, b, gpr, m = 96, 256, 3, 2, 33
    _, _, gi, gl = sketch(f"nml/{ldt}", n, d, b, gpr, ldt)
    X, dY = normal("nml/x", (m, d), io).requires_grad_(), normal("nml/y", (m, n), io)
    w = 1.0 + 0.3 * normal("nml/w", (d,), "f32")
    norm = ft().SketchNorm(d, kind=kind, eps=1e-4, weight=w)
    assert (norm.bias is None) == (kind == "rms")
    group = ft().GroupedSketchedLinear([gi[:32], gi[32:]], [gl[:32], gl[32:]], d, b, gpr, compute_dtype=tdtype(ldt),
                                       checkpoint=checkpoint, norm=norm)
    ya, yb = group(X)
    Xn, mean, rstd, codes, scales = k.sketch_norm_fwd(X.detach(), norm.weight.detach(),
                                                      norm.bias.detach() if norm.bias is not None else None,
                                                      kind=kind, eps=1e-4, checkpoint=True)
    lut = group.inner.compute_tables()
    assert t.equal(t.cat([ya, yb], 1), k.sketch_matmul_fwd(Xn, gi, lut, b, gpr))
    t.autograd.backward([ya, yb], [dY[:, :32], dY[:, 32:]])
    if checkpoint:
        dXn, dL = k.sketch_matmul_bwd_ckpt(dY, codes, scales, gi, lut, b, gpr)
        x = k.sketch_act_quant(X.detach())
    else:
        dXn, dL = k.sketch_matmul_bwd(dY, Xn, gi, lut, b, gpr)
        x = X.detach()
    dX, dw, db = k.sketch_norm_bwd(dXn, x, norm.weight.detach(), mean, rstd, kind=kind, x_dtype=X.dtype)
    assert t.equal(X.grad, dX) and t.equal(group.lut_master.grad, dL) and t.equal(norm.weight.grad, dw)
    assert norm.bias is None or t.equal(norm.bias.grad, db)
    # the norm alone
    X.grad = norm.weight.grad = None
    norm(X).backward(dXn.to(X.dtype))
    want = k.sketch_norm_bwd(dXn.to(X.dtype), X.detach(), norm.weight.detach(), mean, rstd, kind=kind)
    assert t.equal(norm(X), Xn) and t.equal(X.grad, want[0]) and t.equal(norm.weight.grad, want[1])
    # without gradients nothing is kept and the outputs are the same
    with t.no_grad():
        za, zb = group(X)
    assert t.equal(za, ya) and t.equal(zb, yb)


@pytest.mark.parametrize("io,ldt", PAIRS[:3])
def test_head_is_its_calls(io, ldt):
    t, k = torch(), skm()
    V, d, b, gpr, m = 301, 128, 4, 1, 50
    _, _, gi, gl = sketch(f"head/{ldt}", V, d, b, gpr, ldt)
    X = normal("head/x", (m, d), io).requires_grad_()
    T = t.from_numpy(syn.rng_for("head/t").integers(0, V, size=m)).cuda()
    T[::4] = -100
    head = ft().SketchedHead(gi, gl, d, b, gpr, compute_dtype=tdtype(ldt))
    loss = head(X, T)
    tok, lse = k.sketch_xent_fwd(X.detach(), gi, head.lut, T, b, gpr)
    count = int((T != -100).sum())
    assert loss.dim() == 0 and abs(float(loss.detach()) - float(tok.double().sum()) / count) <= 64 * 2.0 ** -24 * float(loss.detach())
    assert t.equal(head.token_losses(X, T), tok)
    (3.0 * loss).backward()
    weight = t.where(T != -100, t.tensor(1.0, device="cuda") / count, t.tensor(0.0, device="cuda"))
    dX, dL = k.sketch_xent_bwd(X.detach(), gi, head.lut, T, lse, weight * 3.0, b, gpr)
    assert t.equal(X.grad, dX) and t.equal(head.lut_master.grad, dL)
    assert t.equal(head.logits(X), k.sketch_matmul_fwd(X.detach(), gi, head.lut, b, gpr))
    head.lut_master.requires_grad_(False)
    X.grad = None
    (3.0 * head(X, T)).backward()
    assert t.equal(X.grad, dX)
    # no token scored: loss 0, gradients 0
    X.grad = None
    none = head(X, t.full_like(T, -100))
    none.backward()
    assert float(none.detach()) == 0.0 and (X.grad == 0).all()
    with pytest.raises(TypeError, match="float16 or bfloat16"):
        ft().SketchedHead(gi, gl, d, b, gpr, compute_dtype=t.float32)
    with pytest.raises(ValueError, match="norm of 64"):
        ft().SketchedLinear(gi, gl, d, b, gpr, norm=ft().SketchNorm(64))


@pytest.mark.parametrize("m", [8, 100])
def test_head_gradients_agree_with_differences(m):
    """Central differences along directions whose steps are exact in f16. The loss is off by at most
    S u (its fp32 sums), the difference by the third derivative times h^2 / 6."""
    t, k = torch(), skm()
    V, d, b, gpr = 70, 64, 4, 2
    g = syn.rng_for(f"diff/{m}")
    idx, lut, gi, gl = sketch("diff", V, d, b, gpr, "f16")
    gl = (t.round(gl.float() * 256) / 256).half()                       # tables on a grid of 2^-8
    x = g.integers(-64, 65, size=(m, d)) / 64.0
    X = t.from_numpy(x.astype(np.float16)).cuda()
    T = t.from_numpy(g.integers(0, V, size=m)).cuda()
    DL = t.ones(m, device="cuda")
    _, lse = k.sketch_xent_fwd(X, gi, gl, T, b, gpr)
    dX, dL = k.sketch_xent_bwd(X, gi, gl, T, lse, DL, b, gpr)

    def total(Xv, lv):
        return float(k.sketch_xent_fwd(Xv, gi, lv, T, b, gpr)[0].double().sum())

    noise = m * 16 * 2.0 ** -24 * 64                                     # every loss within 1024 u
    h = 2.0 ** -6
    D = t.from_numpy(g.integers(-1, 2, size=(m, d)).astype(np.float16)).cuda()
    num = (total(X + h * D, gl) - total(X - h * D, gl)) / (2 * h)
    ana, mag = float((dX.double() * D).sum()), float((dX.double() * D).abs().sum())
    # d logits / dh <= 16 in sum over 64 columns of at most 0.25: |third derivative| <= 16^3, times m h^2 / 6
    assert abs(num - ana) <= 2.0 ** -10 * mag + noise / h + m * 16.0 ** 3 / 6 * h * h * 0.05
    h = 2.0 ** -8
    E = t.from_numpy(g.integers(-1, 2, size=tuple(gl.shape)).astype(np.float16)).cuda()
    num = (total(X, gl + h * E) - total(X, gl - h * E)) / (2 * h)
    ana, mag = float((dL.double() * E).sum()), float((dL.double() * E).abs().sum())
    assert abs(num - ana) <= 2.0 ** -16 * mag + noise / h + m * 64.0 ** 3 / 6 * h * h * 0.05


def float64_step(p, T, eps):
    """The float64 model of the step below: losses and gradients from dense weights."""
    t = torch()
    q = {k: v.double().requires_grad_() for k, v in p.items()}

    def norm(x, w):
        return x * t.rsqrt((x * x).mean(1, keepdim=True) + eps) * w

    h = norm(q["x"], q["n1"]) @ q["w1"].T
    y = q["x"] + h @ q["w2"].T
    z = norm(y, q["n2"]) @ q["wh"].T
    loss = t.nn.functional.cross_entropy(z, T, ignore_index=-100)
    loss.backward()
    return float(loss), {k: v.grad for k, v in q.items()}


@pytest.mark.parametrize("checkpoint", [False, True])
@pytest.mark.parametrize("m", [5, 70])
def test_one_training_step(m, checkpoint):
    """norm -> layer -> layer -> residual -> norm -> head loss, its backward and the fused optimizers."""
    t, f = torch(), ft()
    d, n, V, b, gpr, eps = 256, 512, 700, 4, 2, 1e-5
    parts = {}
    for name, rows, cols in (("w1", n, d), ("w2", d, n), ("wh", V, d)):
        idx, lut, gi, gl = sketch(f"step/{name}", rows, cols, b, gpr, "bf16")
        parts[name] = (gi, gl, t.from_numpy(oracle.dequantize(idx, syn.to_float64(lut, "bf16"), cols, b, gpr)), idx)
    n1 = f.SketchNorm(d, kind="rms", eps=eps)
    n2 = f.SketchNorm(d, kind="rms", eps=eps)
    bf = t.bfloat16
    l1 = f.SketchedLinear(parts["w1"][0], parts["w1"][1], d, b, gpr, bf, checkpoint=checkpoint, norm=n1)
    l2 = f.SketchedLinear(parts["w2"][0], parts["w2"][1], n, b, gpr, bf, checkpoint=checkpoint)
    head = f.SketchedHead(parts["wh"][0], parts["wh"][1], d, b, gpr, bf, norm=n2)
    X = normal(f"step/x/{m}", (m, d), "bf16").requires_grad_()
    T = t.from_numpy(syn.rng_for(f"step/t/{m}").integers(0, V, size=m)).cuda()
    T[1::3] = -100
    loss = head(X + l2(l1(X)), T)
    loss.backward()
    ref, grads = float64_step({"x": X.detach().cpu(), "n1": t.ones(d), "n2": t.ones(d), "w1": parts["w1"][2],
                               "w2": parts["w2"][2], "wh": parts["wh"][2]}, T.cpu(), eps)
    # Six roundings to bf16 (h = 2^-8) lie between X and the loss, four more on the way back; each moves a
    # gradient by at most h of its norm and the checkpoint's steps (2^-7 of a block's largest) by about as much
    # again: 10 h + 2 * 2^-7 < 2^-4
    tol = 2.0 ** -4
    assert abs(float(loss) - ref) <= tol * ref

    def near(got, want, what):
        got, want = got.double().cpu(), want.double()
        assert float((got - want).norm()) <= tol * float(want.norm()), what

    near(X.grad, grads["x"], "dX")
    near(n1.weight.grad, grads["n1"], "norm 1")
    near(n2.weight.grad, grads["n2"], "norm 2")
    for layer, name in ((l1, "w1"), (l2, "w2"), (head, "wh")):
        idx = parts[name][3]
        dw = grads[name].numpy()
        near(layer.lut_master.grad, t.from_numpy(_bin(dw, idx, layer.d, b, gpr)), name)
    opt = f.LutAdam([l1.lut_master, l2.lut_master, head.lut_master, n1.weight, n2.weight], lr=1e-3)
    before = [p.detach().clone() for g in opt.param_groups for p in g["params"]]
    opt.step()
    after = [p for g in opt.param_groups for p in g["params"]]
    assert all(not t.equal(p, q) for p, q in zip(before, after))
    for layer in (l1, l2, head):
        assert t.equal(layer.lut, layer.lut_master.detach().to(bf))
    assert t.isfinite(head(X + l2(l1(X)), T))


def _bin(dW, idx, d, b, gpr):
    """Sums of a dense weight gradient over the columns that share an entry."""
    code = oracle.unpack_indices(idx, d, b)
    out = np.zeros((dW.shape[0], gpr, 1 << b))
    g = np.arange(d) // (d // gpr)
    for i in range(dW.shape[0]):
        np.add.at(out[i], (g, code[i]), dW[i])
    return out


def test_mean_of_many_tokens():
    t, k = torch(), skm()
    g = syn.rng_for("mean")
    loss = t.from_numpy(g.random(20003).astype(np.float32) * 5).cuda()
    T = t.from_numpy(g.integers(0, 3, size=20003)).cuda()
    mean, weight = k.sketch_xent_mean(loss, T, ignore_index=1)
    on = (T != 1).cpu().numpy()
    ref = to_f64(loss)[on].mean()
    # chains of 20 and 26 additions, one division
    assert abs(float(mean) - ref) <= 50 * 2.0 ** -24 * ref
    want = np.where(on, np.float32(1.0) / np.float32(on.sum()), np.float32(0.0))
    assert np.array_equal(weight.cpu().numpy(), want)
    with pytest.raises(ValueError, match="at least one"):
        k.sketch_xent_mean(loss[:0], T[:0])
