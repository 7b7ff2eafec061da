"""Fine-tuning glue: autograd, trainable sketched layers and table optimizers.

Fine-tuning trains only the table values; the mapping stays frozen (SpaLLM,
section 2.3). A :class:`SketchedLinear` keeps the trained values as an fp32
master :class:`torch.nn.Parameter` and a 16-bit compute copy that the forward
and backward kernels read. Its gradient is the fp32 table gradient of the
backward kernel. :class:`LutAdam` and :class:`LutSGD` update the master and
refresh the copy in one fused pass. The pages list the learning rates they
tried (SpaLLM, appendix B.1, Table 7) but name no optimizer.

A layer can keep its input for the table gradient as an 8-bit checkpoint
(``checkpoint=True``) and take the norm in front of it (``norm=``), which then
writes that checkpoint in its own pass (and keeps its own input in 8 bits for
its backward: dX is then that of the checkpoint). :class:`SketchedHead` is the vocabulary
projection with its cross entropy loss, whose logits are never stored.

Beside a layer can stand low-rank adapters of many requests (``adapter=SketchAdapter(...)``, with dropout in front
while training). :class:`SketchDropout` drops and adds a residual, :class:`SketchRotary` norms and turns the query and
key heads of a projection; no mask and no angle is stored.

Every compute step runs in the HIP library (forward, dX, dLUT, norms, loss,
optimizer step); this module only marshals arguments. Three small torch
operations remain in the glue: the fp32 input gradient is cast to the
activations' dtype (autograd requires a gradient in its input's dtype),
inputs and output gradients that are not contiguous or not aligned to 16 bytes
are copied, and the gradient of a mean loss is multiplied by the tokens' weights. A dropout's two whole numbers (key
and number of the mask) are copied and counted on.

The library's gradients carry no graph, so a second derivative through them is refused.
"""
from __future__ import annotations

import threading
from typing import Iterable, List, Optional, Sequence

import torch
from torch.autograd.function import once_differentiable

from . import _lib


def _packed(t):
    """t as the library takes it: contiguous, from a multiple of 16 bytes on.

    Slices start anywhere, and so do the gradients autograd hands out: those of the parts of a concatenation are
    contiguous views into one tensor.
    """
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class SketchMatmulFunction(torch.autograd.Function):
    """Y = X Wᵀ with W[i, j] = lut[i, j // G, idx[i, j]]; gradients for X and the master tables.

    Inputs: X [m, d]; lut_master [n, gpr, 2^b] fp32 (receives dLUT); lut [n, gpr, 2^b], the compute
    copy the kernels read (fp32 for the fp32 path, else f16/bf16); idx_packed [n, d*b/8] uint8.
    """

    @staticmethod
    def forward(ctx, X, lut_master, lut, idx_packed, b: int, gpr: int):
        Y = _lib.sketch_matmul_fwd(_packed(X), idx_packed, lut, b, gpr)
        ctx.save_for_backward(X, lut, idx_packed)
        ctx.b, ctx.gpr = b, gpr
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        X, lut, idx_packed = ctx.saved_tensors
        need_dx, need_dlut = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        if not (need_dx or need_dlut):
            return None, None, None, None, None, None
        dY = _packed(dY)
        if dY.dtype != X.dtype:
            raise TypeError("the output gradient must have the activations' dtype")
        dX, dL = _lib.sketch_matmul_bwd(dY, _packed(X) if need_dlut else None, idx_packed, lut, ctx.b, ctx.gpr,
                                        d=X.shape[1], need_dx=need_dx, need_dlut=need_dlut)
        if dX is not None and dX.dtype != X.dtype:
            dX = dX.to(X.dtype)
        return dX, dL, None, None, None, None


def sketch_matmul(X, lut_master, lut, idx_packed, b: int, gpr: int):
    """Functional form of :class:`SketchMatmulFunction`."""
    return SketchMatmulFunction.apply(X, lut_master, lut, idx_packed, b, gpr)


def _check_dy(dY, dtype):
    if dY.dtype != dtype:
        raise TypeError("the output gradient must have the activations' dtype")
    return _packed(dY)


class CheckpointedMatmulFunction(torch.autograd.Function):
    """:class:`SketchMatmulFunction` that keeps X as its 8-bit checkpoint for the table gradient.

    dX is unchanged; dLUT is that of the checkpoint's values. Nothing of X is kept when the tables need no
    gradient.
    """

    @staticmethod
    def forward(ctx, X, lut_master, lut, idx_packed, b: int, gpr: int):
        X = _packed(X)
        Y = _lib.sketch_matmul_fwd(X, idx_packed, lut, b, gpr)
        codes, scales = _lib.sketch_act_quant(X) if ctx.needs_input_grad[1] else (None, None)
        ctx.save_for_backward(codes, scales, lut, idx_packed)
        ctx.b, ctx.gpr, ctx.d, ctx.dtype = b, gpr, X.shape[1], X.dtype
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        codes, scales, lut, idx_packed = ctx.saved_tensors
        dX, dL = _matmul_bwd(_check_dy(dY, ctx.dtype), codes, scales, idx_packed, lut, ctx)
        return dX.to(ctx.dtype) if dX is not None else None, dL, None, None, None, None


def _matmul_bwd(dY, codes, scales, idx_packed, lut, ctx, need_dx=None):
    """(dX fp32, dLUT) from a checkpoint, or dX alone when none was kept."""
    need_dx = ctx.needs_input_grad[0] if need_dx is None else need_dx
    if codes is not None:
        return _lib.sketch_matmul_bwd_ckpt(dY, codes, scales, idx_packed, lut, ctx.b, ctx.gpr, need_dx=need_dx)
    if not need_dx:
        return None, None
    return _lib.sketch_matmul_bwd(dY, None, idx_packed, lut, ctx.b, ctx.gpr, d=ctx.d, need_dlut=False)


class NormFunction(torch.autograd.Function):
    """Layer norm or root-mean-square norm of the rows of X [m, d]; weight and bias fp32 [d] (or None)."""

    @staticmethod
    def forward(ctx, X, weight, bias, kind: str, eps: float):
        X = _packed(X)
        Y, mean, rstd, _, _ = _lib.sketch_norm_fwd(X, weight, bias, kind=kind, eps=eps)
        ctx.save_for_backward(X, weight, mean, rstd)
        ctx.kind = kind
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        X, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        dX, dw, db = _lib.sketch_norm_bwd(_packed(dY), X, weight, mean, rstd, kind=ctx.kind, need_dx=need[0],
                                          need_dw=need[1], need_db=need[2])
        return dX, dw, db, None, None


class NormMatmulFunction(torch.autograd.Function):
    """Y = norm(X) Wᵀ in two launches; its backward hands the matmul's fp32 dX to the norm without a cast.

    checkpoint: keep the normed input (written by the norm's own pass) and X as 8-bit checkpoints instead of
    16-bit copies, 16.5 bits per value for both. The table gradient is then that of the normed input's checkpoint,
    and the norm's backward (dX, dweight, dbias) that of X's. Without a table gradient nothing is quantised.
    """

    @staticmethod
    def forward(ctx, X, weight, bias, lut_master, lut, idx_packed, b: int, gpr: int, kind: str, eps: float,
                checkpoint: bool):
        X = _packed(X)
        need = ctx.needs_input_grad
        Xn, mean, rstd, codes, scales = _lib.sketch_norm_fwd(X, weight, bias, kind=kind, eps=eps,
                                                             checkpoint=checkpoint and need[3])
        Y = _lib.sketch_matmul_fwd(Xn, idx_packed, lut, b, gpr)
        x0, x1 = X, None
        if not any(need[:3]):
            x0 = None
        elif checkpoint and need[3]:
            x0, x1 = _lib.sketch_act_quant(X)
        ctx.save_for_backward(x0, x1, weight, mean, rstd, codes, scales,
                              Xn if need[3] and not checkpoint else None, lut, idx_packed)
        ctx.b, ctx.gpr, ctx.d, ctx.dtype, ctx.kind = b, gpr, X.shape[1], X.dtype, kind
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        x0, x1, weight, mean, rstd, codes, scales, Xn, lut, idx_packed = ctx.saved_tensors
        need = ctx.needs_input_grad
        dY = _check_dy(dY, ctx.dtype)
        need_dxn = any(need[:3])
        if Xn is not None:
            dXn, dL = _lib.sketch_matmul_bwd(dY, Xn, idx_packed, lut, ctx.b, ctx.gpr, need_dx=need_dxn)
        else:
            dXn, dL = _matmul_bwd(dY, codes, scales, idx_packed, lut, ctx, need_dx=need_dxn)
        dX = dw = db = None
        if need_dxn:
            dX, dw, db = _lib.sketch_norm_bwd(dXn, x0 if x1 is None else (x0, x1), weight, mean, rstd, kind=ctx.kind,
                                              need_dx=need[0], need_dw=need[1], need_db=need[2], x_dtype=ctx.dtype)
        return dX, dw, db, dL, None, None, None, None, None, None, None


class CrossEntropyFunction(torch.autograd.Function):
    """Per-token softmax cross entropy (fp32 [m]) of the logits X Wᵀ, which are never stored; gradients for X
    and the master tables. Tokens whose target is ignore_index have loss 0 and no gradient."""

    @staticmethod
    def forward(ctx, X, lut_master, lut, idx_packed, targets, b: int, gpr: int, ignore_index: int):
        X, targets = _packed(X), targets.contiguous()
        loss, lse = _lib.sketch_xent_fwd(X, idx_packed, lut, targets, b, gpr, ignore_index=ignore_index)
        ctx.save_for_backward(X, lut, idx_packed, targets, lse)
        ctx.b, ctx.gpr, ctx.ignore_index = b, gpr, ignore_index
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        X, lut, idx_packed, targets, lse = ctx.saved_tensors
        need_dx, need_dlut = ctx.needs_input_grad[0], ctx.needs_input_grad[1]
        dX, dL = _lib.sketch_xent_bwd(X, idx_packed, lut, targets, lse, _packed(dloss), ctx.b, ctx.gpr,
                                      ignore_index=ctx.ignore_index, need_dx=need_dx, need_dlut=need_dlut)
        return dX, dL, None, None, None, None, None, None


class _MeanFunction(torch.autograd.Function):
    """Mean of the losses of the tokens that are scored (0 when none is)."""

    @staticmethod
    def forward(ctx, loss, targets, ignore_index: int):
        mean, weight = _lib.sketch_xent_mean(loss, targets, ignore_index=ignore_index)
        ctx.save_for_backward(weight)
        return mean

    @staticmethod
    def backward(ctx, dmean):
        (weight,) = ctx.saved_tensors
        return weight * dmean, None, None


class DropoutFunction(torch.autograd.Function):
    """residual + dropout(X); the mask is computed again from the seed in the backward pass."""

    @staticmethod
    def forward(ctx, X, residual, p: float, seed):
        ctx.save_for_backward(seed)
        ctx.p = p
        return _lib.sketch_dropout(_packed(X), p, seed, residual=None if residual is None else _packed(residual))

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        (seed,) = ctx.saved_tensors
        dX = _lib.sketch_dropout(_packed(dY), ctx.p, seed) if ctx.needs_input_grad[0] else None
        return dX, dY if ctx.needs_input_grad[1] else None, None, None


class AdapterMatmulFunction(torch.autograd.Function):
    """Y = X Wᵀ + the adapters' products; gradients for X, the master tables and the adapters' masters.

    The matmul's fp32 dX goes into the adapters' backward, which adds its part and rounds once.
    """

    @staticmethod
    def forward(ctx, X, lut_master, lut, idx_packed, b: int, gpr: int, A_master, B_master, A, B, ids, scale,
                p: float, seed, back: bool):
        X = _packed(X)
        Y = _lib.sketch_matmul_fwd(X, idx_packed, lut, b, gpr)
        Y, H = _lib.sketch_adapter_fwd(X, A, B, Y, adapter=ids, scale=scale, p=p, seed=seed, out=Y,
                                       need_h=back and ctx.needs_input_grad[7])
        need = ctx.needs_input_grad
        ctx.save_for_backward(X if need[1] or need[6] else None, H, lut, idx_packed, A, B, ids, scale, seed)
        ctx.b, ctx.gpr, ctx.p, ctx.shape, ctx.dtype = b, gpr, p, X.shape, X.dtype
        return Y

    @staticmethod
    @once_differentiable
    def backward(ctx, dY):
        X, H, lut, idx_packed, A, B, ids, scale, seed = ctx.saved_tensors
        need = ctx.needs_input_grad
        dY = _check_dy(dY, ctx.dtype)
        base_dx = dL = None
        if need[0] or need[1]:
            base_dx, dL = _lib.sketch_matmul_bwd(dY, X if need[1] else None, idx_packed, lut, ctx.b, ctx.gpr,
                                                 d=ctx.shape[1], need_dx=need[0], need_dlut=need[1])
        if X is None:  # (not read, its shape and dtype are)
            X = dY.new_empty(ctx.shape)
        dX, dA, dB = _lib.sketch_adapter_bwd(dY, X, H, A, B, base_dx, adapter=ids, scale=scale, p=ctx.p, seed=seed,
                                             need_dx=need[0], need_da=need[6], need_db=need[7])
        return (dX, dL, None, None, None, None, dA, dB) + (None,) * 7


class RotaryFunction(torch.autograd.Function):
    """Heads q [m, heads, head_dim] and k (or None), normed (eps given) and turned; gradients for both and the weights."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, inv_freq, eps, pairs: str):
        q, k = _heads(q), _heads(k)
        out = _lib.sketch_rotary_fwd(q, k, positions, inv_freq, q_weight, k_weight, eps=eps, pairs=pairs)
        kept = (q, k) if eps is not None else (None, None)  # (the rotation alone reads no heads going back)
        ctx.save_for_backward(*kept, q_weight, k_weight, positions, inv_freq)
        ctx.eps, ctx.pairs = eps, pairs
        return out

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        q, k, q_weight, k_weight, positions, inv_freq = ctx.saved_tensors
        need = ctx.needs_input_grad
        dq, dk = _heads(dq), _heads(dk)
        if ctx.eps is None:
            q, k = dq, dk  # (not read, their shape and dtype are)
        out = _lib.sketch_rotary_bwd(dq, dk, q, k, positions, inv_freq, q_weight, k_weight, eps=ctx.eps,
                                     pairs=ctx.pairs, need_dw=need[2] or need[3])
        return tuple(g if n else None for g, n in zip(out, need)) + (None,) * 4


def _heads(t):
    """t [m, heads, head_dim] with every token's heads side by side, as the library takes them."""
    if t is None or (t.stride(2) == 1 and t.stride(1) == t.shape[2] and t.stride(0) >= t.shape[1] * t.shape[2]):
        return t
    return t.contiguous()


_masks = threading.local()  # .stack: the contexts of replay_masks that this thread is in, innermost last


class _Masks:
    """One of the two contexts of :func:`replay_masks`: seeds that forwards draw in it are noted in order, or (replay)
    handed out again from the first one. It may be left out of turn and from another thread: a checkpointed forward
    that raises leaves it when its frame is collected."""

    def __init__(self, drawn: list, replay: bool):
        self.drawn, self.replay, self.open = drawn, replay, []

    def __enter__(self):
        stack = _masks.__dict__.setdefault("stack", [])
        entry = [self.drawn, iter(self.drawn) if self.replay else None]
        stack.append(entry)
        self.open.append((stack, entry))

    def __exit__(self, *exc):
        stack, entry = self.open.pop()
        stack[:] = [e for e in stack if e is not entry]


def replay_masks():
    """``context_fn=replay_masks`` of ``torch.utils.checkpoint.checkpoint(.., use_reentrant=False, ..)``: where a
    forward with dropout is recomputed in the backward pass, it drops what it dropped the first time.

    Without it such a recomputation is refused (it would draw other masks than the output had, whatever the state of
    torch's generators), also with use_reentrant=True: there, draw the seed outside (``module.seed.next()``) and
    hand it in as an argument of the checkpointed function, on to ``forward(.., seed=seed)``.
    """
    drawn = []
    return _Masks(drawn, False), _Masks(drawn, True)


class _Seed(torch.nn.Module):
    """A dropout's random numbers: a key and the number of the next mask, on the GPU and in the state dict.

    seed: the key (None = from torch's generator, so that modules differ and torch.manual_seed repeats them). The
    number moves on in the stream's order, in replays of a captured step too. A deep copy has a key of its own, from
    torch's generator: layers that are copies of one must not drop the same values.
    """

    def __init__(self, seed: Optional[int], device):
        super().__init__()
        key = int(torch.randint(0, (1 << 63) - 1, ()).item()) if seed is None else int(seed)
        self.register_buffer("state", torch.tensor([key, 0], dtype=torch.int64, device=device))

    def __deepcopy__(self, memo):
        new = memo[id(self)] = type(self)(None, self.state.device)
        return new.train(self.training)

    @torch.no_grad()
    def next(self):
        """The seed of the next mask, int64 [2]; where :func:`replay_masks` runs a forward again, of the mask it had."""
        seen, stack = [], _masks.__dict__.get("stack", ())
        for drawn, again in reversed(stack):  # (checkpoints inside a recomputed function record what it replays)
            if again is not None:
                owner, seed = next(again, (None, None))
                if owner is not self:
                    raise RuntimeError("a recomputed forward went through other dropouts than the first time")
                break
            seen.append(drawn)
        else:
            if torch._C._current_graph_task_id() != -1:
                raise RuntimeError("dropout in a forward that is recomputed in the backward pass: give checkpoint() "
                                   "context_fn=replay_masks, or the forward its seed")
            seed = self.state.clone()
            self.state[1:] += 1
        for drawn in seen:
            drawn.append((self, seed))
        return seed


def _check_p(p: float) -> float:
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p = {p} is not a probability")
    return float(p)


class SketchDropout(torch.nn.Module):
    """residual + dropout(X) while training, residual + X else (the residual may be left out).

    Every forward has the next mask, or that of `seed` (int64 [2] on the GPU, e.g. from ``module.seed.next()``). A
    forward that is recomputed in the backward pass needs :func:`replay_masks` or its seed given. A deep copy has masks
    of its own.
    """

    def __init__(self, p: float, seed: Optional[int] = None, device="cuda"):
        super().__init__()
        self.p = _check_p(p)
        self.seed = _Seed(seed, device)

    def forward(self, X, residual=None, seed=None):
        if self.training and self.p > 0.0:
            return DropoutFunction.apply(X, residual, self.p, self.seed.next() if seed is None else seed)
        return X if residual is None else DropoutFunction.apply(X, residual, 0.0, None)


class SketchAdapter(torch.nn.Module):
    """Low-rank adapters of rank r beside a sketched layer of n rows and d columns.

    A [n_adapters, r, d] and B [n_adapters, n, r] are fp32 parameters with a 16-bit copy that the kernels read, as a
    layer's tables (trained by :class:`LutAdam` / :class:`LutSGD`, which refresh the copy). A starts uniform in
    +-1 / sqrt(d), B with zeros. scale: alpha / r for every adapter (alpha = r unless given). dropout: of the layer's
    input in front of A, while training, with masks as :class:`SketchDropout` (a forward that is recomputed needs
    :func:`replay_masks` or its seed given). compute_dtype must be the activations' dtype. A backward pass takes at most
    4096 adapters; the forward alone 2^20.
    """

    def __init__(self, n: int, d: int, r: int, n_adapters: int = 1, alpha: Optional[float] = None,
                 dropout: float = 0.0, compute_dtype=torch.float16, seed: Optional[int] = None, device="cuda"):
        super().__init__()
        if compute_dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("adapters compute in float16 or bfloat16")
        if not 1 <= r <= 128 or n_adapters < 1:
            raise ValueError(f"{n_adapters} adapters of rank {r}: at least one, of rank 1 to 128")
        self.p = _check_p(dropout)
        self.A_master = torch.nn.Parameter((torch.rand((n_adapters, r, d), device=device) * 2 - 1) / d ** 0.5)
        self.B_master = torch.nn.Parameter(torch.zeros((n_adapters, n, r), device=device))
        self.register_buffer("A", self.A_master.detach().to(compute_dtype))
        self.register_buffer("B", self.B_master.detach().to(compute_dtype))
        scale = (r if alpha is None else float(alpha)) / r
        self.register_buffer("scale", torch.full((n_adapters,), scale, dtype=torch.float32, device=device))
        self.seed = _Seed(seed, device)
        self._link_copies()

    def _link_copies(self) -> None:
        # (as SketchedLinear._link_copy)
        self.A_master._skm_copy, self.B_master._skm_copy = self.A, self.B

    def refresh_copies(self) -> None:
        """Round the masters into the compute copies (after changing them outside the optimizers)."""
        self.A.copy_(self.A_master.detach())
        self.B.copy_(self.B_master.detach())

    def arguments(self, seed=None):
        """(p, seed) of this pass: dropout while training only, with the next mask unless its seed is given."""
        self._link_copies()
        if not self.training or self.p == 0.0:
            return 0.0, None
        return self.p, self.seed.next() if seed is None else seed


class SketchRotary(torch.nn.Module):
    """Norm (optional) and position rotation of the query and key heads of a projection, in one pass.

    theta: frequencies theta^(-2 i / rot_dim), or give inv_freq (float64 [rot_dim / 2]). rot_dim: leading columns of a
    head that turn (all unless given). norm: root-mean-square norm of every head, with fp32 weights for query and key
    heads (ones unless given). pairs: "halves" or "neighbours". forward(q, k, positions): heads [m, heads, head_dim],
    also as strided views of a joined projection (``q.unflatten(1, (heads, head_dim))``), positions int64 [m].
    """

    def __init__(self, head_dim: int, theta: float = 10000.0, rot_dim: Optional[int] = None, inv_freq=None,
                 norm: bool = False, eps: float = 1e-6, pairs: str = "halves", q_weight=None, k_weight=None,
                 device="cuda"):
        super().__init__()
        _lib._pairs(pairs)
        if inv_freq is None:
            rot = head_dim if rot_dim is None else rot_dim
            if rot % 2 or not 2 <= rot <= head_dim:
                raise ValueError(f"rot_dim = {rot} of {head_dim} columns: an even number of them")
            inv_freq = float(theta) ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
        elif rot_dim is not None and rot_dim != 2 * inv_freq.numel():
            raise ValueError(f"{inv_freq.numel()} frequencies for {rot_dim} columns")
        if not norm and (q_weight is not None or k_weight is not None):
            raise ValueError("weights belong to a norm")
        self.pairs, self.eps = pairs, float(eps) if norm else None
        self.register_buffer("inv_freq", inv_freq.to(device=device, dtype=torch.float64).contiguous().clone())

        def param(t):
            if not norm:
                return None
            if t is None:
                return torch.nn.Parameter(torch.ones(head_dim, dtype=torch.float32, device=device))
            if tuple(t.shape) != (head_dim,):
                raise ValueError(f"heads of {head_dim} columns given {tuple(t.shape)} weights")
            return torch.nn.Parameter(t.detach().to(torch.float32).contiguous().clone())

        self.q_weight, self.k_weight = param(q_weight), param(k_weight)

    def forward(self, q, k, positions):
        return RotaryFunction.apply(q, k, self.q_weight, self.k_weight if k is not None else None, positions.contiguous(),
                                    self.inv_freq, self.eps, self.pairs)


class SketchNorm(torch.nn.Module):
    """Layer norm (kind "layer", with a bias) or root-mean-square norm (kind "rms") of rows of d columns.

    weight and bias are fp32 parameters (ones and zeros unless given), trained by :class:`LutAdam` /
    :class:`LutSGD` like any fp32 tensor.
    """

    def __init__(self, d: int, kind: str = "layer", eps: float = 1e-5, weight=None, bias=None, device="cuda"):
        super().__init__()
        _lib._norm_kind(kind)
        self.kind, self.eps = kind, float(eps)

        def param(t, fill):
            if t is None:
                return torch.nn.Parameter(torch.full((d,), fill, dtype=torch.float32, device=device))
            if tuple(t.shape) != (d,):
                raise ValueError(f"a norm of {d} columns given {tuple(t.shape)} weights")
            return torch.nn.Parameter(t.detach().to(torch.float32).contiguous().clone())

        self.weight = param(weight, 1.0)
        self.bias = param(bias, 0.0) if kind == "layer" or bias is not None else None

    def forward(self, X):
        return NormFunction.apply(X, self.weight, self.bias, self.kind, self.eps)


class SketchedLinear(torch.nn.Module):
    """A linear layer whose weight is a frozen mapping into trainable per-group tables.

    idx_packed: [n, d*b/8] uint8 on the GPU (frozen). lut: [n, gpr, 2^b] initial table values.
    compute_dtype: dtype of the copy the kernels read (torch.float16 / torch.bfloat16, or torch.float32
    for the fp32 path, where the master itself is read). checkpoint: keep the input for the table gradient as
    its 8-bit checkpoint (8.25 bits per value). norm: a :class:`SketchNorm` applied to the input first (its
    pass then writes the checkpoint).

    With checkpoint alone the table gradient is that of the 8-bit input and dX is unchanged. With both, the norm's
    own input is kept in 8 bits too, so dX and the gradients of the norm's weight and bias are those of that
    checkpoint (each value off by at most half a step of its 32-column block). While the tables need no gradient
    (``lut_master.requires_grad_(False)``) checkpoint changes nothing.

    adapter: a :class:`SketchAdapter` whose products are added to the output; forward then takes the adapter of every
    token too (int32 [m], outside [0, n_adapters) = none; left out: the first one), and the seed of its dropout's mask
    (left out: the next one). It reads the layer's input in full, so it does not go with checkpoint. With a norm in front
    as well, the normed input's gradient is rounded to the activations' dtype on its way to the norm's backward (the
    adapters' backward sums it in fp32 and rounds once; without an adapter the norm takes it in fp32).
    """

    def __init__(self, idx_packed, lut, d: int, b: int, gpr: int, compute_dtype=torch.float16,
                 checkpoint: bool = False, norm: Optional[SketchNorm] = None,
                 adapter: Optional[SketchAdapter] = None):
        super().__init__()
        if adapter is not None:
            if checkpoint:
                raise ValueError("an adapter reads its layer's input in full: not with checkpoint")
            if adapter.A.shape[2] != d or adapter.B.shape[1] != idx_packed.shape[0]:
                raise ValueError(f"an adapter of {adapter.B.shape[1]} x {adapter.A.shape[2]} beside a layer of "
                                 f"{idx_packed.shape[0]} x {d}")
        if norm is not None and norm.weight.numel() != d:
            raise ValueError(f"a norm of {norm.weight.numel()} columns in front of a layer of {d}")
        n = idx_packed.shape[0]
        if tuple(lut.shape) != (n, gpr, 1 << b) or idx_packed.shape[1] * 8 != d * b:
            raise ValueError("table or index shape does not match (n, gpr, 2^b) / (n, d*b/8)")
        self.d, self.b, self.gpr = d, b, gpr
        self.checkpoint, self.norm, self.adapter = bool(checkpoint), norm, adapter
        self.register_buffer("idx_packed", _packed(idx_packed))
        self.lut_master = torch.nn.Parameter(lut.detach().to(torch.float32).contiguous().clone())
        if compute_dtype == torch.float32:
            self.lut = None
        else:
            self.register_buffer("lut", self.lut_master.detach().to(compute_dtype))
        self._link_copy()

    def _link_copy(self) -> None:
        # the optimizers below find the compute copy through this attribute (set again on every
        # forward, since moving the module replaces its buffers but keeps the parameter object)
        self.lut_master._skm_copy = self.lut

    @property
    def out_features(self) -> int:
        return self.idx_packed.shape[0]

    def compute_tables(self):
        return self.lut if self.lut is not None else self.lut_master.detach()

    def refresh_copy(self) -> None:
        """Round the master into the compute copy (after changing the master outside the optimizers)."""
        if self.lut is not None:
            self.lut.copy_(self.lut_master.detach())

    def forward(self, X, adapter_ids=None, seed=None):
        self._link_copy()
        if self.adapter is not None:
            a = self.adapter
            p, seed = a.arguments(seed)
            # (a function of its own: its backward takes the adapters' 16-bit dX, half a step of the activations' type)
            X = X if self.norm is None else self.norm(X)
            if adapter_ids is not None:
                adapter_ids = adapter_ids.contiguous()
            return AdapterMatmulFunction.apply(X, self.lut_master, self.compute_tables(), self.idx_packed, self.b,
                                               self.gpr, a.A_master, a.B_master, a.A, a.B, adapter_ids, a.scale, p,
                                               seed, torch.is_grad_enabled())
        if adapter_ids is not None or seed is not None:
            raise ValueError("adapter_ids or a seed for a layer without adapters")
        # (a function's needs_input_grad names parameters under no_grad too, where no backward will come)
        checkpoint = self.checkpoint and torch.is_grad_enabled()
        if self.norm is not None:
            n = self.norm
            return NormMatmulFunction.apply(X, n.weight, n.bias, self.lut_master, self.compute_tables(),
                                            self.idx_packed, self.b, self.gpr, n.kind, n.eps, checkpoint)
        if checkpoint:
            return CheckpointedMatmulFunction.apply(X, self.lut_master, self.compute_tables(), self.idx_packed,
                                                    self.b, self.gpr)
        return sketch_matmul(X, self.lut_master, self.compute_tables(), self.idx_packed, self.b, self.gpr)


class GroupedSketchedLinear(torch.nn.Module):
    """Several sketched projections of the same input (q/k/v, gate/up) in one launch per pass.

    The projections' rows are stored back to back (indices and tables), so the forward, dX and dLUT
    each run as one launch over all rows; forward returns one view per projection. An adapter spans all
    of the rows.
    """

    def __init__(self, idx_list: Sequence, lut_list: Sequence, d: int, b: int, gpr: int,
                 compute_dtype=torch.float16, checkpoint: bool = False, norm: Optional[SketchNorm] = None,
                 adapter: Optional[SketchAdapter] = None):
        super().__init__()
        self.sizes = [int(i.shape[0]) for i in idx_list]
        self.inner = SketchedLinear(torch.cat([i.contiguous() for i in idx_list], 0),
                                    torch.cat([t.detach() for t in lut_list], 0), d, b, gpr, compute_dtype,
                                    checkpoint=checkpoint, norm=norm, adapter=adapter)

    @property
    def lut_master(self):
        return self.inner.lut_master

    def table_slices(self) -> List:
        """The master tables of each projection (views into the shared parameter)."""
        return list(torch.split(self.inner.lut_master, self.sizes, 0))

    def forward(self, X, adapter_ids=None, seed=None):
        Y = self.inner(X, adapter_ids, seed)
        return tuple(torch.split(Y, self.sizes, dim=1))


class SketchedHead(SketchedLinear):
    """The vocabulary projection of a model with its cross entropy loss: forward(X, targets) is the mean loss.

    A :class:`SketchedLinear` of n words (16-bit compute copy; its tables are frozen by
    ``head.lut_master.requires_grad_(False)``). The logits are never stored; :meth:`logits` computes them for
    generation. norm: applied to the hidden states first, in the loss and in the logits.
    """

    def __init__(self, idx_packed, lut, d: int, b: int, gpr: int, compute_dtype=torch.float16,
                 ignore_index: int = -100, norm: Optional[SketchNorm] = None):
        if compute_dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("a sketched head computes in float16 or bfloat16")
        super().__init__(idx_packed, lut, d, b, gpr, compute_dtype, norm=norm)
        self.ignore_index = ignore_index

    def token_losses(self, X, targets):
        """The loss of every token, fp32 [m] (0 where the target is ignore_index)."""
        self._link_copy()
        if self.norm is not None:
            X = self.norm(X)
        return CrossEntropyFunction.apply(X, self.lut_master, self.compute_tables(), self.idx_packed, targets, self.b,
                                          self.gpr, self.ignore_index)

    def forward(self, X, targets):
        """Mean loss over the tokens whose target is not ignore_index (0 when there is none)."""
        losses = self.token_losses(X, targets)
        if losses.numel() == 0:
            return losses.sum()
        return _MeanFunction.apply(losses, targets.contiguous(), self.ignore_index)

    def logits(self, X):
        """X Wᵀ [m, n] in X's dtype."""
        return SketchedLinear.forward(self, X)


def _copy_of(p):
    return getattr(p, "_skm_copy", None)


class LutAdam(torch.optim.Optimizer):
    """Adam with decoupled weight decay on fp32 master tables, fused with the refresh of their compute copy.

    Parameters must be fp32 CUDA tensors; a master created by :class:`SketchedLinear` carries its copy.
    grad_scale multiplies every gradient (dLUT is a sum over tokens; e.g. 1/tokens gives a mean).
    """

    def __init__(self, params: Iterable, lr: float = 1e-5, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.0, grad_scale: float = 1.0):
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay,
                                      grad_scale=grad_scale))

    @torch.no_grad()
    def step(self, closure=None):
        loss = closure() if closure is not None else None
        for group in self.param_groups:
            b1, b2 = group["betas"]
            for p in group["params"]:
                if p.grad is None:
                    continue
                st = self.state[p]
                if not st:
                    st["step"] = 0
                    st["exp_avg"] = torch.zeros_like(p, memory_format=torch.contiguous_format)
                    st["exp_avg_sq"] = torch.zeros_like(p, memory_format=torch.contiguous_format)
                st["step"] += 1
                _lib.sketch_lut_adam_step(p, _packed(p.grad), st["exp_avg"], st["exp_avg_sq"], st["step"],
                                          group["lr"], b1, b2, group["eps"], group["weight_decay"],
                                          group["grad_scale"], lut=_copy_of(p))
        return loss


class LutSGD(torch.optim.Optimizer):
    """SGD (heavy-ball momentum, L2 weight decay) on fp32 master tables, fused with the copy refresh."""

    def __init__(self, params: Iterable, lr: float = 1e-3, momentum: float = 0.0, weight_decay: float = 0.0,
                 grad_scale: float = 1.0):
        super().__init__(params, dict(lr=lr, momentum=momentum, weight_decay=weight_decay, grad_scale=grad_scale))

    @torch.no_grad()
    def step(self, closure=None):
        loss = closure() if closure is not None else None
        for group in self.param_groups:
            for p in group["params"]:
                if p.grad is None:
                    continue
                st = self.state[p]
                buf: Optional[torch.Tensor] = None
                if group["momentum"] != 0.0:
                    if "momentum_buffer" not in st:
                        st["momentum_buffer"] = torch.zeros_like(p, memory_format=torch.contiguous_format)
                    buf = st["momentum_buffer"]
                _lib.sketch_lut_sgd_step(p, _packed(p.grad), group["lr"], group["momentum"],
                                         group["weight_decay"], group["grad_scale"], momentum_buf=buf,
                                         lut=_copy_of(p))
        return loss
