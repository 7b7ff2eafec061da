"""The modules around adapters, dropout and head rotation, without a GPU: the library's calls are replaced by
stand-ins that compute the same with torch and refuse what the library refuses."""
import copy
import pickle
import threading

import pytest
import torch
from torch.utils.checkpoint import checkpoint

from lut_sketched_matmul_amd import finetune


class Calls:
    def __init__(self):
        self.log = []

    @staticmethod
    def packed(*tensors):
        for t in tensors:
            if t is not None:
                assert t.is_contiguous() and t.data_ptr() % 16 == 0

    @staticmethod
    def weights(idx, lut, gpr):
        code = torch.stack([idx & 15, idx >> 4], 2).reshape(idx.shape[0], gpr, -1).long()
        return lut.float().gather(2, code).reshape(idx.shape[0], -1), code

    def sketch_matmul_fwd(self, X, idx, lut, b, gpr):
        self.packed(X)
        return (X.float() @ self.weights(idx, lut, gpr)[0].T).to(X.dtype)

    def sketch_matmul_bwd(self, dY, X, idx, lut, b, gpr, d=None, need_dx=True, need_dlut=True):
        self.packed(dY, X)
        self.log.append(("matmul_bwd", need_dx, need_dlut))
        W, code = self.weights(idx, lut, gpr)
        dL = torch.zeros(lut.shape).scatter_add_(2, code, (dY.float().T @ X.float()).reshape(code.shape)) if need_dlut else None
        return dY.float() @ W if need_dx else None, dL

    @staticmethod
    def mask(shape, p, seed):
        if not p:
            return torch.ones(shape)
        g = torch.Generator().manual_seed(int(seed[0] % 1000 * 1000 + seed[1]))
        return (torch.rand(shape, generator=g) >= p).float() / (1 - p)

    def sketch_dropout(self, X, p, seed=None, residual=None):
        self.packed(X, residual)
        self.log.append(("dropout", p, None if seed is None else seed.tolist()))
        y = X.float() * self.mask(X.shape, p, seed)
        return (y if residual is None else y + residual.float()).to(X.dtype)

    def sketch_adapter_fwd(self, X, A, B, base=None, adapter=None, scale=None, p=0.0, seed=None, out=None, need_h=False):
        self.packed(X, A, B, base)
        self.log.append(("adapter_fwd", p, need_h, out is base))
        ids = torch.zeros(X.shape[0], dtype=torch.int64) if adapter is None else adapter.long()
        ok = ((ids >= 0) & (ids < A.shape[0])).float()[:, None]
        i = ids.clamp(0, A.shape[0] - 1)
        H = torch.einsum("td,trd->tr", X.float() * self.mask(X.shape, p, seed), A.float()[i]) * ok
        Y = (base.float() + scale[i][:, None] * torch.einsum("tr,tnr->tn", H, B.float()[i])).to(X.dtype)
        if out is not None:
            out.copy_(Y)
            Y = out
        return Y, H if need_h else None

    def sketch_adapter_bwd(self, dY, X, H, A, B, base_dx=None, adapter=None, scale=None, p=0.0, seed=None, need_dx=True,
                           need_da=True, need_db=True):
        self.packed(dY, X, H, base_dx)
        self.log.append(("adapter_bwd", need_dx, need_da, need_db))
        ids = torch.zeros(X.shape[0], dtype=torch.int64) if adapter is None else adapter.long()
        ok = ((ids >= 0) & (ids < A.shape[0])).float()[:, None]
        i = ids.clamp(0, A.shape[0] - 1)
        g = dY.float() * scale[i][:, None] * ok
        dh = torch.einsum("tn,tnr->tr", g, B.float()[i])
        mask = self.mask(X.shape, p, seed)
        dX = dA = dB = None
        if need_dx:
            dX = torch.einsum("tr,trd->td", dh, A.float()[i]) * mask
            dX = (dX if base_dx is None else dX + base_dx).to(X.dtype)
        if need_da:
            dA = torch.zeros(A.shape).index_add_(0, i, dh[:, :, None] * (X.float() * mask)[:, None])
        if need_db:
            dB = torch.zeros(B.shape).index_add_(0, i, g[:, :, None] * H[:, None])
        return dX, dA, dB

    @staticmethod
    def turn(x, pos, f, back=False):
        c, s = (fn(pos.double()[:, None] * f).float()[:, None] for fn in (torch.cos, torch.sin))
        if back:
            s = -s
        a, b = x[..., :f.numel()], x[..., f.numel():2 * f.numel()]
        return torch.cat([a * c - b * s, a * s + b * c, x[..., 2 * f.numel():]], 2)

    @staticmethod
    def side_by_side(*ts):
        for t in ts:
            if t is not None:
                assert t.stride(2) == 1 and t.stride(1) == t.shape[2]

    def sketch_rotary_fwd(self, q, k, pos, f, qw=None, kw=None, eps=None, pairs="halves"):
        self.side_by_side(q, k)

        def side(x, w):
            if x is None:
                return None
            v = x.float()
            if eps is not None:
                v = v * torch.rsqrt(v.square().mean(2, keepdim=True) + eps) * w
            return self.turn(v, pos, f).to(x.dtype)

        return side(q, qw), side(k, kw)

    def sketch_rotary_bwd(self, dq, dk, q, k, pos, f, qw=None, kw=None, eps=None, pairs="halves", need_dw=True):
        self.side_by_side(dq, dk, q, k)
        self.log.append(("rotary_bwd", need_dw))

        def side(dy, x, w):
            if x is None:
                return None, None
            g, v = self.turn(dy.float(), pos, f, back=True), x.float()
            if eps is None:
                return g.to(x.dtype), None
            r = torch.rsqrt(v.square().mean(2, keepdim=True) + eps)
            dw = (g * v * r).sum((0, 1))
            g = g * w
            return (r * g - v * r ** 3 * (g * v).mean(2, keepdim=True)).to(x.dtype), dw

        (a, c), (b, d) = side(dq, q, qw), side(dk, k, kw)
        return a, b, c if need_dw else None, d if need_dw else None


@pytest.fixture
def calls(monkeypatch):
    c = Calls()
    for name in dir(Calls):
        if name.startswith("sketch_"):
            monkeypatch.setattr(finetune._lib, name, getattr(c, name))
    return c


def sketch(n, d, gpr, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, 256, (n, d // 2), generator=g, dtype=torch.uint8), torch.randn((n, gpr, 16), generator=g) * 0.1


def normal(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def adapter(n, d, r, S, p=0.0, dtype=torch.bfloat16):
    a = finetune.SketchAdapter(n, d, r, S, alpha=2 * r, dropout=p, compute_dtype=dtype, seed=5, device="cpu")
    with torch.no_grad():
        a.B_master.copy_(normal(a.B_master.shape, 3))
    a.refresh_copies()
    return a


@pytest.mark.parametrize("p", [0.0, 0.3])
@pytest.mark.parametrize("norm", [False, True])
def test_adapted_layer_against_autograd(calls, p, norm, monkeypatch):
    """Every gradient against torch's own of the same formula, with fp32 copies in place of the 16-bit ones."""
    n, d, r, S, m = 12, 64, 4, 3, 9
    idx, lut = sketch(n, d, 2, 1)
    a = adapter(n, d, r, S, p)
    a.A, a.B = a.A_master.detach().clone(), a.B_master.detach().clone()
    nm = torch.nn.Identity() if norm else None
    if norm:
        nm.weight = torch.ones(d)
    layer = finetune.SketchedLinear(idx, lut, d, 4, 2, compute_dtype=torch.float32, norm=nm, adapter=a)
    ids = torch.tensor([0, 1, 1, -1, 2, 0, 7, 1, 2], dtype=torch.int32)
    X = normal((m, d), 2).requires_grad_()
    Y = layer(X, ids)
    dY = normal((m, n), 4)
    Y.backward(dY)
    W, _ = calls.weights(idx, layer.lut_master, 2)
    x2 = X.detach().clone().requires_grad_()
    A, B, L = (t.detach().clone().requires_grad_() for t in (a.A_master, a.B_master, layer.lut_master))
    mask = calls.mask((m, d), p, torch.tensor([5, 0]))
    W, _ = calls.weights(idx, L, 2)
    ok = ((ids >= 0) & (ids < S)).float()[:, None]
    i = ids.long().clamp(0, S - 1)
    want = x2 @ W.T + 2.0 * ok * torch.einsum("tr,tnr->tn", torch.einsum("td,trd->tr", x2 * mask, A[i]), B[i])
    want.backward(dY)
    for got, ref in ((Y, want), (X.grad, x2.grad), (a.A_master.grad, A.grad), (a.B_master.grad, B.grad),
                     (layer.lut_master.grad, L.grad)):
        assert torch.allclose(got, ref, rtol=1e-4, atol=1e-5)


def test_only_what_is_asked_for(calls):
    n, d = 12, 64
    idx, lut = sketch(n, d, 2, 1)
    a = adapter(n, d, 4, 2)
    layer = finetune.SketchedLinear(idx, lut, d, 4, 2, compute_dtype=torch.bfloat16, adapter=a)
    layer.lut_master.requires_grad_(False)
    X = normal((5, d), 2).bfloat16()
    layer(X).float().sum().backward()                       # the adapters alone: the tables' kernels do not run
    assert calls.log == [("adapter_fwd", 0.0, True, True), ("adapter_bwd", False, True, True)]
    calls.log.clear()
    a.A_master.requires_grad_(False), a.B_master.requires_grad_(False)
    X = X.requires_grad_()
    layer(X).float().sum().backward()                       # all frozen: neither X nor H is kept
    assert calls.log == [("adapter_fwd", 0.0, False, True), ("matmul_bwd", True, False), ("adapter_bwd", True, False, False)]
    calls.log.clear()
    a.A_master.requires_grad_(True), a.B_master.requires_grad_(True)
    with torch.no_grad():
        layer(X)
    assert calls.log == [("adapter_fwd", 0.0, False, True)]


def test_dropout_streams(calls):
    """Each forward its own mask, backward the forward's; eval mode none; the state travels with the module."""
    drop = finetune.SketchDropout(0.5, seed=9, device="cpu")
    X, res = normal((4, 32), 1).requires_grad_(), normal((4, 32), 2).requires_grad_()
    y1, y2 = drop(X, res), drop(X, res)
    assert not torch.equal(y1, y2)
    y2.backward(torch.ones(4, 32))
    assert torch.equal(X.grad, calls.mask((4, 32), 0.5, torch.tensor([9, 1]))) and torch.equal(res.grad, torch.ones(4, 32))
    assert drop.state_dict()["seed.state"].tolist() == [9, 2]
    drop.eval()
    assert torch.equal(drop(X), X) and torch.equal(drop(X, res), X + res)
    assert drop.seed.state.tolist() == [9, 2]
    torch.manual_seed(1)
    a, b = (finetune.SketchDropout(0.1, device="cpu").seed.state for _ in range(2))
    assert a[0] != b[0]
    torch.manual_seed(1)
    assert finetune.SketchDropout(0.1, device="cpu").seed.state[0] == a[0]
    ad = adapter(8, 64, 4, 1, p=0.1)
    assert ad.arguments()[1].tolist() == [5, 0] and ad.arguments()[1].tolist() == [5, 1]
    assert ad.eval().arguments() == (0.0, None)


@pytest.mark.parametrize("norm", [False, True])
def test_rotary_on_views_of_a_joined_projection(calls, norm):
    m, hq, hk, dh = 6, 4, 2, 16
    rot = finetune.SketchRotary(dh, norm=norm, device="cpu", q_weight=normal(dh, 8) if norm else None)
    x = normal((m, (hq + 2 * hk) * dh), 1).requires_grad_()
    pos = torch.arange(m) + 3
    q, k, v = torch.split(x, [hq * dh, hk * dh, hk * dh], 1)
    yq, yk = rot(q.unflatten(1, (hq, dh)), k.unflatten(1, (hk, dh)), pos)
    gq, gk = normal(yq.shape, 2), normal(yk.shape, 3)
    ((yq * gq).sum() + (yk.transpose(0, 1) * gk.transpose(0, 1)).sum() + v.sum()).backward()
    x2 = x.detach().clone().requires_grad_()
    w = [t.detach().clone().requires_grad_() for t in (rot.q_weight, rot.k_weight)] if norm else [None, None]
    a, b = x2[:, :hq * dh].unflatten(1, (hq, dh)), x2[:, hq * dh:(hq + hk) * dh].unflatten(1, (hk, dh))
    outs = calls.sketch_rotary_fwd(a, b, pos, rot.inv_freq, *w, eps=rot.eps)
    ((outs[0] * gq).sum() + (outs[1] * gk).sum() + x2[:, (hq + hk) * dh:].sum()).backward()
    assert torch.allclose(yq, outs[0]) and torch.allclose(yk, outs[1]) and torch.allclose(x.grad, x2.grad, atol=1e-5)
    if norm:
        assert torch.allclose(rot.q_weight.grad, w[0].grad, atol=1e-5) and torch.allclose(rot.k_weight.grad, w[1].grad, atol=1e-5)
    one, none = rot(q.unflatten(1, (hq, dh)).detach(), None, pos)
    assert none is None and torch.equal(one, yq)


def test_refusals(calls):
    idx, lut = sketch(12, 64, 2, 1)
    make = lambda **k: finetune.SketchedLinear(idx, lut, 64, 4, 2, compute_dtype=torch.bfloat16, **k)
    with pytest.raises(ValueError):
        make(adapter=adapter(12, 64, 4, 1), checkpoint=True)
    with pytest.raises(ValueError):
        make(adapter=adapter(11, 64, 4, 1))
    with pytest.raises(ValueError):
        make(adapter=adapter(12, 32, 4, 1))
    with pytest.raises(ValueError):
        make()(normal((3, 64), 1).bfloat16(), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(TypeError):
        adapter(8, 64, 4, 1, dtype=torch.float32)
    for r in (0, 129):
        with pytest.raises(ValueError):
            finetune.SketchAdapter(8, 64, r, device="cpu")
    with pytest.raises(ValueError):
        finetune.SketchDropout(1.5, device="cpu")
    for bad in (dict(rot_dim=3), dict(rot_dim=18), dict(pairs="both"), dict(q_weight=torch.ones(16)),
                dict(norm=True, q_weight=torch.ones(8)), dict(inv_freq=torch.ones(4), rot_dim=16)):
        with pytest.raises(ValueError):
            finetune.SketchRotary(16, device="cpu", **bad)


# ---- activations that are computed again in the backward pass -------------------------------------------


def dropping_parts():
    """A run of an adapted layer with dropout in front, and a dropout used twice, all from the same seeds every time."""
    n, d = 64, 64
    idx, lut = sketch(n, d, 2, 1)
    torch.manual_seed(3)
    layer = finetune.SketchedLinear(idx, lut, d, 4, 2, compute_dtype=torch.bfloat16, adapter=adapter(n, d, 4, 2, p=0.3))
    drop = finetune.SketchDropout(0.5, seed=9, device="cpu")
    ids = torch.tensor([0, 1, -1, 1, 0], dtype=torch.int32)
    return layer, drop, ids


def step(parts, around, runs=1):
    """(output, gradients) of layer -> dropout -> tanh -> dropout + residual, each run handed to `around(fn, X)`."""
    layer, drop, ids = parts

    def fn(X):
        return drop(torch.tanh(drop(layer(X, ids))), X)

    X = normal((5, 64), 2).bfloat16().requires_grad_()
    Y = X
    for _ in range(runs):
        Y = around(fn, Y)
    Y.backward(normal((5, 64), 4).bfloat16())
    return [Y.detach(), X.grad, layer.adapter.A_master.grad, layer.adapter.B_master.grad, layer.lut_master.grad]


def replayed(fn, X):
    return checkpoint(fn, X, use_reentrant=False, context_fn=finetune.replay_masks)


@pytest.mark.parametrize("around", [replayed, lambda fn, X: replayed(lambda x: replayed(fn, x), X)])
@pytest.mark.parametrize("runs", [1, 3])
def test_recomputed_forward_has_its_own_masks(calls, around, runs):
    """Run again in the backward pass, once or in nested checkpoints, a forward has the masks that it had."""
    want, got = (step(dropping_parts(), a, runs) for a in (lambda fn, X: fn(X), around))
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_recomputed_twice(calls):
    """A graph that is kept and gone through again."""
    drop = finetune.SketchDropout(0.5, seed=9, device="cpu")
    X = normal((4, 32), 1).requires_grad_()
    Y = replayed(lambda x: drop(torch.tanh(drop(x))), X)
    one, = torch.autograd.grad(Y.sum(), X, retain_graph=True)
    two, = torch.autograd.grad(Y.sum(), X)
    assert torch.equal(one, two) and drop.seed.state.tolist() == [9, 2]


@pytest.mark.parametrize("reentrant", [False, True])
def test_recomputation_without_the_masks_is_refused(calls, reentrant):
    """It would draw other masks than the output had."""
    with pytest.raises(RuntimeError, match="recomputed"):
        step(dropping_parts(), lambda fn, X: checkpoint(fn, X, use_reentrant=reentrant))
    parts = dropping_parts()  # (nothing is drawn here)
    parts[0].eval(), parts[1].eval()
    step(parts, lambda fn, X: checkpoint(fn, X, use_reentrant=reentrant))


@pytest.mark.parametrize("reentrant", [False, True])
def test_masks_given_by_their_seeds(calls, reentrant):
    layer, drop, ids = dropping_parts()
    X = normal((5, 64), 2).bfloat16().requires_grad_()
    dY = normal((5, 64), 4).bfloat16()
    want = drop(layer(X, ids), X)
    want.backward(dY)
    first, X.grad = X.grad, None
    layer, drop, ids = dropping_parts()

    def fn(X, a, b):
        return drop(layer(X, ids, seed=a), X, seed=b)

    got = checkpoint(fn, X, layer.adapter.seed.next(), drop.seed.next(), use_reentrant=reentrant)
    got.backward(dY)
    assert torch.equal(got, want) and torch.equal(X.grad, first)
    assert drop.seed.state.tolist() == [9, 1]
    with pytest.raises(ValueError):
        finetune.SketchedLinear(*sketch(64, 64, 2, 1), 64, 4, 2, compute_dtype=torch.bfloat16)(X, seed=drop.seed.next())


def test_contexts_left_late_and_from_another_thread():
    """A forward that raises leaves its context when it is collected: whenever, wherever."""
    drop = finetune.SketchDropout(0.5, seed=9, device="cpu")
    (a, again), (b, _) = finetune.replay_masks(), finetune.replay_masks()
    a.__enter__()
    one = drop.seed.next()
    b.__enter__()
    two = drop.seed.next()
    t = threading.Thread(target=a.__exit__, args=(None, None, None))
    t.start(), t.join()
    three = drop.seed.next()
    b.__exit__(None, None, None)
    drop.seed.next()
    assert [s.tolist() for _, s in a.drawn] == [one.tolist(), two.tolist()]
    assert [s.tolist() for _, s in b.drawn] == [two.tolist(), three.tolist()]
    for _ in range(2):
        with again:
            assert torch.equal(drop.seed.next(), one) and torch.equal(drop.seed.next(), two)
            with pytest.raises(RuntimeError, match="other dropouts"):
                drop.seed.next()
    with again, pytest.raises(RuntimeError, match="other dropouts"):
        finetune.SketchDropout(0.5, seed=9, device="cpu").seed.next()
    assert drop.seed.next().tolist() == [9, 4]


def test_copied_layers_have_keys_of_their_own(calls):
    """Layers stacked as deep copies of one drop different values; a module shared within a copy stays shared."""
    first = torch.nn.ModuleDict(dict(a=finetune.SketchDropout(0.5, seed=9, device="cpu"), ad=adapter(8, 64, 4, 1, p=0.1)))
    first["b"] = first["a"]
    first.eval()["a"].train()
    torch.manual_seed(2)
    second, third = copy.deepcopy(first), copy.deepcopy(first)
    keys = {int(m["a"].seed.state[0]) for m in (first, second, third)} | {int(m["ad"].seed.state[0]) for m in (first, second, third)}
    assert len(keys) == 6
    assert second["a"] is second["b"] and second["a"].training and second["a"].seed.training and not second["ad"].seed.training
    assert second["a"].seed.state.tolist()[1] == 0 and second["a"].seed.state.device == first["a"].seed.state.device
    torch.manual_seed(2)
    assert torch.equal(copy.deepcopy(first)["a"].seed.state, second["a"].seed.state)
    X = torch.ones(4, 32)
    assert not torch.equal(second["a"](X), third["a"](X))
    again = pickle.loads(pickle.dumps(first))  # (saved and loaded it goes on where it was)
    assert torch.equal(again["a"].seed.state, first["a"].seed.state)


@pytest.mark.parametrize("which", ["dropout", "adapter", "rotary", "matmul"])
def test_second_derivatives_are_refused(calls, which, monkeypatch):
    """The library's gradients carry no graph: a second derivative through them would miss its terms without a word."""
    for name in dir(Calls):  # (as the library, the stand-ins then give tensors without a graph)
        if name.startswith("sketch_"):
            monkeypatch.setattr(finetune._lib, name, torch.no_grad()(getattr(calls, name)))
    n = d = 64
    idx, lut = sketch(n, d, 2, 1)
    X = normal((5, d), 2).bfloat16().requires_grad_()
    if which == "rotary":
        rot = finetune.SketchRotary(16, norm=True, device="cpu")
        run = lambda x: rot(x.unflatten(1, (4, 16)), None, torch.arange(5))[0].flatten(1)
    elif which == "dropout":
        run = finetune.SketchDropout(0.5, seed=1, device="cpu")
    else:
        run = finetune.SketchedLinear(idx, lut, d, 4, 2, compute_dtype=torch.bfloat16,
                                      adapter=adapter(n, d, 4, 1) if which == "adapter" else None)
    Y = run(X)
    g, = torch.autograd.grad((Y * X).float().square().sum(), X, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.float().square().sum().backward()
    run(X).float().square().sum().backward()  # (the first derivatives stay)
