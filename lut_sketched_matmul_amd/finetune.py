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

Every compute step runs in the HIP library (forward, dX, dLUT, norms, loss,
optimizer step); this module only marshals arguments. Three small torch
operations remain in the glue: the fp32 input gradient is cast to the
activations' dtype (autograd requires a gradient in its input's dtype),
inputs and output gradients that are not contiguous or not aligned to 16 bytes
are copied, and the gradient of a mean loss is multiplied by the tokens' weights.
"""
from __future__ import annotations

from typing import Iterable, List, Optional, Sequence

import torch

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
    """

    def __init__(self, idx_packed, lut, d: int, b: int, gpr: int, compute_dtype=torch.float16,
                 checkpoint: bool = False, norm: Optional[SketchNorm] = None):
        super().__init__()
        if norm is not None and norm.weight.numel() != d:
            raise ValueError(f"a norm of {norm.weight.numel()} columns in front of a layer of {d}")
        n = idx_packed.shape[0]
        if tuple(lut.shape) != (n, gpr, 1 << b) or idx_packed.shape[1] * 8 != d * b:
            raise ValueError("table or index shape does not match (n, gpr, 2^b) / (n, d*b/8)")
        self.d, self.b, self.gpr = d, b, gpr
        self.checkpoint, self.norm = bool(checkpoint), norm
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

    def forward(self, X):
        self._link_copy()
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
    each run as one launch over all rows; forward returns one view per projection.
    """

    def __init__(self, idx_list: Sequence, lut_list: Sequence, d: int, b: int, gpr: int,
                 compute_dtype=torch.float16, checkpoint: bool = False, norm: Optional[SketchNorm] = None):
        super().__init__()
        self.sizes = [int(i.shape[0]) for i in idx_list]
        self.inner = SketchedLinear(torch.cat([i.contiguous() for i in idx_list], 0),
                                    torch.cat([t.detach() for t in lut_list], 0), d, b, gpr, compute_dtype,
                                    checkpoint=checkpoint, norm=norm)

    @property
    def lut_master(self):
        return self.inner.lut_master

    def table_slices(self) -> List:
        """The master tables of each projection (views into the shared parameter)."""
        return list(torch.split(self.inner.lut_master, self.sizes, 0))

    def forward(self, X):
        Y = self.inner(X)
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
