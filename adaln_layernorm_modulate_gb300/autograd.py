"""Autograd nodes over libadaln. First the fused AdaLN (LayerNorm-Modulate) operator of the
AdaptiveLoad technical summary, section 2.B, as one forward launch and one backward call
(fused dx + D-tile partials, then the fixed-order reduce) in a PyTorch graph.

    y = (x - mean) * rstd * (1 + scale[m]) + shift[m],  rstd = 1 / sqrt(var + eps)

Dense input: x [Bt, N, D], shift and scale [Bt, D]; token (b, n) uses row b.
Packed input: x [R, D] with ``cu_seqlens`` [nseg + 1] and ``mod_idx`` [nseg] (int32, on the
device); segment s uses row ``mod_idx[s]`` of shift and scale [nmod, D].

The node saves x, scale and the fp32 row statistics (8 bytes a row), not y or xhat; with
``save_stats=False`` it keeps no statistics (the forward's are dropped with its outputs) and
the backward recomputes them from x (one more read of x, bitwise the same statistics and
gradients). Every
step runs in the library's kernels; this module only allocates outputs and workspaces
through PyTorch's allocator and passes pointers. dshift and dscale come out of the
library in fp32; autograd wants gradients in the parameters' dtype, so they are rounded
once to it (a no-op for fp32 parameters).

Between two such nodes: the norms of queries and keys for each head with their rotation by positions
(``qk_norm_rope``, ``QKNormRope``), and attention over packed or dense sequences (``attention``).

Then the end of such a network: the affine layer norm (``layer_norm``, ``LayerNorm``) and the
vocabulary loss without its logits (``linear_cross_entropy``).
"""
from __future__ import annotations

import contextlib
import math
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import (ADALN_BF16, ADALN_F32, AdalnError, adaln_attention_bwd, adaln_attention_bwd_workspace_size,
               adaln_attention_fwd, adaln_attention_fwd_workspace_size, adaln_bwd, adaln_bwd_recompute,
               adaln_bwd_recompute_workspace_size, adaln_bwd_varlen, adaln_bwd_varlen_recompute,
               adaln_bwd_varlen_recompute_workspace_size, adaln_bwd_varlen_workspace_size,
               adaln_bwd_workspace_size, adaln_fwd, adaln_fwd_varlen, adaln_fwd_varlen_workspace_size,
               adaln_layernorm_bwd, adaln_layernorm_bwd_workspace_size, adaln_layernorm_fwd,
               adaln_linear_xent_bwd, adaln_linear_xent_bwd_workspace_size, adaln_linear_xent_fwd,
               adaln_linear_xent_fwd_workspace_size, adaln_qk_norm_rope_bwd,
               adaln_qk_norm_rope_bwd_workspace_size, adaln_qk_norm_rope_fwd, adaln_read_status)

__all__ = ["AdaLNModulateFunction", "AdaLNModulate", "adaln_modulate", "LayerNormFunction", "LayerNorm",
           "layer_norm", "LinearCrossEntropyFunction", "linear_cross_entropy", "QKNormRopeFunction",
           "QKNormRope", "qk_norm_rope", "AttentionFunction", "attention"]


def _code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return ADALN_BF16
    if t.dtype == torch.float32:
        return ADALN_F32
    raise TypeError("AdaLN-Modulate supports bfloat16 and float32 tensors, got %s" % t.dtype)


def _workspace(nbytes: int, device) -> torch.Tensor:
    if nbytes <= 0:
        raise AdalnError("workspace size", 2)
    # The caching allocator returns 512-byte aligned blocks; the library needs 256.
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _on(t: torch.Tensor):
    """The library plans for the current device and launches on its current stream: a context in
    which that is t's device."""
    if t.device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(t.device)


def _check_status(ws: torch.Tensor, what: str) -> None:
    st = adaln_read_status(ws)
    if st != 0:
        raise AdalnError(what, st)


class AdaLNModulateFunction(torch.autograd.Function):
    """y = LayerNorm(x) * (1 + scale) + shift with saved fp32 mean/rstd.

    ``check_tables`` reads the packed call's device status after each launch (it
    synchronises the stream): set it while validating new ``cu_seqlens``/``mod_idx``.
    ``save_stats=False``: keep no statistics; the backward recomputes them from x."""

    @staticmethod
    def forward(ctx, x, shift, scale, cu_seqlens=None, mod_idx=None, eps: float = 1e-6,
                check_tables: bool = False, save_stats: bool = True):
        if not x.is_cuda:
            raise ValueError("AdaLN-Modulate runs on CUDA tensors")
        x = x.contiguous()
        shift = shift.contiguous()
        scale = scale.contiguous()
        if shift.dtype != x.dtype or scale.dtype != x.dtype:
            raise TypeError("x, shift and scale must share one dtype")
        if shift.device != x.device or scale.device != x.device:
            raise ValueError("x, shift and scale must be on one device")
        dt = _code(x)
        D = x.shape[-1]
        packed = cu_seqlens is not None
        y = torch.empty_like(x)
        if packed:
            if x.dim() != 2 or mod_idx is None:
                raise ValueError("packed input: x [R, D] with cu_seqlens and mod_idx")
            if cu_seqlens.dim() != 1 or mod_idx.shape != (cu_seqlens.shape[0] - 1,):
                raise ValueError("packed input: cu_seqlens [nseg + 1] and mod_idx [nseg]")
            if shift.dim() != 2 or shift.shape[1] != D or scale.shape != shift.shape:
                raise ValueError("packed input: shift and scale [nmod, D]")
            cu = cu_seqlens.to(device=x.device, dtype=torch.int32).contiguous()
            mod = mod_idx.to(device=x.device, dtype=torch.int32).contiguous()
            R, nseg, nmod = x.shape[0], mod.numel(), shift.shape[0]
            mean = torch.empty(R, dtype=torch.float32, device=x.device)
            rstd = torch.empty(R, dtype=torch.float32, device=x.device)
            with _on(x):
                nb = adaln_fwd_varlen_workspace_size(R, nseg, D, dt)
                ws = _workspace(nb, x.device)
                adaln_fwd_varlen(x, shift, scale, y, mean, rstd, cu, mod, nseg, R, nmod, D, eps, ws, nb, dt)
                if check_tables:
                    _check_status(ws, "adaln_fwd_varlen")
            kept = (mean, rstd) if save_stats else (mean[:0], rstd[:0])
            ctx.save_for_backward(x, scale, *kept, cu, mod)
        else:
            if x.dim() != 3 or shift.shape != (x.shape[0], D) or scale.shape != (x.shape[0], D):
                raise ValueError("dense input: x [Bt, N, D], shift and scale [Bt, D]")
            Bt, N = x.shape[0], x.shape[1]
            mean = torch.empty((Bt, N), dtype=torch.float32, device=x.device)
            rstd = torch.empty((Bt, N), dtype=torch.float32, device=x.device)
            with _on(x):
                adaln_fwd(x, shift, scale, y, mean, rstd, Bt, N, D, eps, dt)
            kept = (mean, rstd) if save_stats else (mean[:0], rstd[:0])
            ctx.save_for_backward(x, scale, *kept)
        ctx.packed = packed
        ctx.check_tables = check_tables
        ctx.save_stats = save_stats
        ctx.eps = eps
        ctx.shift_dtype = shift.dtype
        ctx.mark_non_differentiable(mean, rstd)
        return y, mean, rstd

    @staticmethod
    def backward(ctx, dy, _dmean, _drstd):
        x, scale, mean, rstd = ctx.saved_tensors[:4]
        dy = dy.contiguous()
        dt = _code(x)
        D = x.shape[-1]
        nmod = scale.shape[0]
        dx = torch.empty_like(x)
        dshift = torch.empty((nmod, D), dtype=torch.float32, device=x.device)
        dscale = torch.empty((nmod, D), dtype=torch.float32, device=x.device)
        with _on(x):
            if ctx.packed:
                cu, mod = ctx.saved_tensors[4:]
                R, nseg = x.shape[0], mod.numel()
                if ctx.save_stats:
                    nb = adaln_bwd_varlen_workspace_size(R, nseg, nmod, D, dt)
                    ws = _workspace(nb, x.device)
                    adaln_bwd_varlen(dy, x, mean, rstd, scale, dx, dshift, dscale, cu, mod, nseg, R, nmod,
                                     D, ws, nb, dt)
                else:
                    nb = adaln_bwd_varlen_recompute_workspace_size(R, nseg, nmod, D, dt)
                    ws = _workspace(nb, x.device)
                    adaln_bwd_varlen_recompute(dy, x, scale, dx, dshift, dscale, cu, mod, nseg, R, nmod, D,
                                               ctx.eps, ws, nb, dt)
                if ctx.check_tables:
                    _check_status(ws, "adaln_bwd_varlen")
            else:
                Bt, N = x.shape[0], x.shape[1]
                if ctx.save_stats:
                    nb = adaln_bwd_workspace_size(Bt, N, D, dt)
                    ws = _workspace(nb, x.device)
                    adaln_bwd(dy, x, mean, rstd, scale, dx, dshift, dscale, ws, nb, Bt, N, D, dt)
                else:
                    nb = adaln_bwd_recompute_workspace_size(Bt, N, D, dt)
                    ws = _workspace(nb, x.device)
                    adaln_bwd_recompute(dy, x, scale, dx, dshift, dscale, ws, nb, Bt, N, D, ctx.eps, dt)
        return (dx, dshift.to(ctx.shift_dtype), dscale.to(ctx.shift_dtype), None, None, None, None, None)


def adaln_modulate(x: torch.Tensor, shift: torch.Tensor, scale: torch.Tensor,
                   cu_seqlens: Optional[torch.Tensor] = None, mod_idx: Optional[torch.Tensor] = None,
                   eps: float = 1e-6, check_tables: bool = False, save_stats: bool = True) -> torch.Tensor:
    """Differentiable fused AdaLN-Modulate; returns y (the statistics stay in the graph)."""
    y, _, _ = AdaLNModulateFunction.apply(x, shift, scale, cu_seqlens, mod_idx, eps, check_tables,
                                          save_stats)
    return y


class AdaLNModulate(torch.nn.Module):
    """Module form: ``AdaLNModulate(eps)(x, shift, scale[, cu_seqlens, mod_idx])``. It has no
    parameters of its own: shift and scale come from the conditioning branch."""

    def __init__(self, eps: float = 1e-6, save_stats: bool = True):
        super().__init__()
        self.eps = float(eps)
        self.save_stats = bool(save_stats)

    def forward(self, x, shift, scale, cu_seqlens=None, mod_idx=None):
        return adaln_modulate(x, shift, scale, cu_seqlens, mod_idx, self.eps, save_stats=self.save_stats)

    def extra_repr(self) -> str:
        return "eps=%g, save_stats=%s" % (self.eps, self.save_stats)


class LayerNormFunction(torch.autograd.Function):
    """y = (x - mean) * rstd * weight + bias over the last dimension of x [..., D], weight and
    bias [D] (either may be None). Saves x, weight and the fp32 row statistics. Gradients that
    autograd does not ask for are not computed, except that dx always is."""

    @staticmethod
    def forward(ctx, x, weight=None, bias=None, eps: float = 1e-6):
        if not x.is_cuda:
            raise ValueError("layer_norm runs on CUDA tensors")
        if x.dim() < 1:
            raise ValueError("layer_norm input: x [..., D]")
        D = x.shape[-1]
        for p in (weight, bias):
            if p is not None and p.shape != (D,):
                raise ValueError("layer_norm: weight and bias are [D]")
            if p is not None and p.dtype != x.dtype:
                raise TypeError("x, weight and bias must share one dtype")
            if p is not None and p.device != x.device:
                raise ValueError("x, weight and bias must be on one device")
        dt = _code(x)
        x = x.contiguous()
        weight = None if weight is None else weight.contiguous()
        R = x.numel() // D if D else 0
        y = torch.empty_like(x)
        mean = torch.empty(R, dtype=torch.float32, device=x.device)
        rstd = torch.empty(R, dtype=torch.float32, device=x.device)
        with _on(x):
            adaln_layernorm_fwd(x, weight, None if bias is None else bias.contiguous(), y, mean, rstd, R, D,
                                eps, dt)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        dt, D, R = _code(x), x.shape[-1], mean.numel()
        dy = dy.contiguous()
        dx = torch.empty_like(x)
        want_w, want_b = weight is not None and ctx.needs_input_grad[1], ctx.needs_input_grad[2]
        dweight = torch.empty(D, dtype=torch.float32, device=x.device) if want_w else None
        dbias = torch.empty(D, dtype=torch.float32, device=x.device) if want_b else None
        with _on(x):
            nb = adaln_layernorm_bwd_workspace_size(R, D, dt)
            ws = _workspace(nb, x.device)
            adaln_layernorm_bwd(dy, x, mean, rstd, weight, dx, dweight, dbias, ws, nb, R, D, dt)
        return (dx, dweight.to(x.dtype) if want_w else None, dbias.to(x.dtype) if want_b else None, None)


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-6) -> torch.Tensor:
    """Differentiable affine layer norm over the last dimension."""
    return LayerNormFunction.apply(x, weight, bias, eps)


class LayerNorm(torch.nn.Module):
    """Layer norm with a learned weight (ones) and bias (zeros), each optional."""

    def __init__(self, D: int, eps: float = 1e-6, weight: bool = True, bias: bool = True, device=None,
                 dtype=None):
        super().__init__()
        self.eps = float(eps)
        self.D = int(D)
        self.weight = torch.nn.Parameter(torch.ones(D, device=device, dtype=dtype)) if weight else None
        self.bias = torch.nn.Parameter(torch.zeros(D, device=device, dtype=dtype)) if bias else None

    def forward(self, x):
        return layer_norm(x, self.weight, self.bias, self.eps)

    def extra_repr(self) -> str:
        return "%d, eps=%g, weight=%s, bias=%s" % (self.D, self.eps, self.weight is not None,
                                                   self.bias is not None)


class LinearCrossEntropyFunction(torch.autograd.Function):
    """(loss, lse) of each row of x [..., D] under the vocabulary head weight [V, D]:
    loss = lse - z_target, lse = log sum exp z, z = x weight^T, both fp32 and differentiable.
    Rows with target == ignore_index have loss and lse 0. Saves x, weight, target and lse, no
    logits. ``check_targets`` reads the call's device status (it synchronises the stream)."""

    @staticmethod
    def forward(ctx, x, weight, target, ignore_index: int = -100, check_targets: bool = False):
        if not x.is_cuda:
            raise ValueError("linear_cross_entropy runs on CUDA tensors")
        if x.dim() < 1 or weight.dim() != 2 or weight.shape[1] != x.shape[-1]:
            raise ValueError("linear_cross_entropy: x [..., D] and weight [V, D]")
        if target.shape != x.shape[:-1] or target.dtype != torch.int64:
            raise ValueError("linear_cross_entropy: target [...] of int64, one per row of x")
        if weight.device != x.device or target.device != x.device:
            raise ValueError("x, weight and target must be on one device")
        if x.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16:
            raise TypeError("linear_cross_entropy takes bfloat16 x and weight, got %s and %s"
                            % (x.dtype, weight.dtype))
        x, weight, target = x.contiguous(), weight.contiguous(), target.contiguous()
        V, D = weight.shape
        N = target.numel()
        loss = torch.empty(target.shape, dtype=torch.float32, device=x.device)
        lse = torch.empty(target.shape, dtype=torch.float32, device=x.device)
        with _on(x):
            nb = adaln_linear_xent_fwd_workspace_size(N, V, D, ADALN_BF16)
            ws = _workspace(nb, x.device)
            adaln_linear_xent_fwd(x, weight, target, loss, lse, N, V, D, ignore_index, ws, nb, ADALN_BF16)
            if check_targets:
                _check_status(ws, "adaln_linear_xent_fwd")
        ctx.save_for_backward(x, weight, target, lse)
        ctx.ignore_index = ignore_index
        ctx.set_materialize_grads(False)
        return loss, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, dlse):
        x, weight, target, lse = ctx.saved_tensors
        want_x, want_w = ctx.needs_input_grad[:2]
        if dloss is None and dlse is None:
            return None, None, None, None, None
        V, D = weight.shape
        N = target.numel()
        dloss = torch.zeros_like(lse) if dloss is None else dloss.contiguous()
        dlse = None if dlse is None else dlse.contiguous()
        dx = torch.empty_like(x) if want_x else None
        dweight = torch.empty_like(weight) if want_w else None
        with _on(x):
            nb = adaln_linear_xent_bwd_workspace_size(N, V, D, ADALN_BF16)
            ws = _workspace(nb, x.device)
            adaln_linear_xent_bwd(x, weight, target, lse, dloss, dlse, dx, dweight, N, V, D, ctx.ignore_index,
                                  ws, nb, ADALN_BF16)
        return dx, dweight, None, None, None


def linear_cross_entropy(x: torch.Tensor, weight: torch.Tensor, target: torch.Tensor,
                         ignore_index: int = -100, reduction: str = "mean", z_loss: float = 0.0,
                         check_targets: bool = False) -> torch.Tensor:
    """Softmax cross entropy of the vocabulary head ``x @ weight.T`` without its logits.

    reduction: "none" (a loss per row), "sum", or "mean" over the rows that carry a loss, those whose
    target is a word and not ignore_index (0 if there is none). z_loss adds z_loss * lse^2 to each
    such row's loss. A target that is neither a word nor ignore_index carries none either, and raises
    an error with ``check_targets``."""
    if reduction not in ("none", "sum", "mean"):
        raise ValueError("reduction must be none, sum or mean, got %r" % (reduction,))
    loss, lse = LinearCrossEntropyFunction.apply(x, weight, target, ignore_index, check_targets)
    if z_loss:
        loss = loss + z_loss * lse * lse
    if reduction == "none":
        return loss
    total = loss.sum()
    if reduction == "sum":
        return total
    V = weight.shape[0]
    counts = target.clamp(0, V - 1) == target
    if 0 <= ignore_index < V:
        counts = counts & (target != ignore_index)
    return total / counts.sum().clamp(min=1)


def _rows(t: torch.Tensor) -> torch.Tensor:
    """t [R, H, d] with heads side by side in rows the library takes, copied only if they are not:
    parts of a joint projection's rows go as they are."""
    R, H, d = t.shape
    if ((d <= 1 or t.stride(2) == 1) and (H <= 1 or t.stride(1) == d) and t.data_ptr() % 16 == 0
            and (R <= 1 or (t.stride(0) >= H * d and t.stride(0) % 8 == 0))):
        return t
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone(memory_format=torch.contiguous_format)


def _ld(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


class QKNormRopeFunction(torch.autograd.Function):
    """(q', k') of q [..., Hq, d] and k [..., Hk, d] (the same leading sizes): an RMS norm of each head
    with the weights [d], then the rotation by positions [..., axes]. Saves q, k (as they come: parts of
    a projection's rows are not copied), the weights and positions."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, axes, theta: float, eps: float, norm: bool):
        if not q.is_cuda:
            raise ValueError("qk_norm_rope runs on CUDA tensors")
        if q.dim() < 2 or k.dim() != q.dim() or k.shape[:-2] != q.shape[:-2] or k.shape[-1] != q.shape[-1]:
            raise ValueError("qk_norm_rope: q [..., Hq, d] and k [..., Hk, d] with the same leading sizes")
        Hq, Hk, d = q.shape[-2], k.shape[-2], q.shape[-1]
        for w in (q_weight, k_weight):
            if w is not None and w.shape != (d,):
                raise ValueError("qk_norm_rope: weights are [d]")
            if w is not None and not norm:
                raise ValueError("qk_norm_rope: weights go with the norm")
        if any(t is not None and t.device != q.device for t in (k, q_weight, k_weight, positions)):
            raise ValueError("q, k, weights and positions must be on one device")
        if any(t is not None and t.dtype != q.dtype for t in (k, q_weight, k_weight)):
            raise TypeError("q, k and the weights must share one dtype")
        dt = _code(q)
        axes = tuple(int(w) for w in axes) if axes is not None else ()
        if positions is not None:
            if positions.dtype.is_floating_point or positions.dtype.is_complex or positions.dtype == torch.bool:
                raise TypeError("qk_norm_rope: positions are whole numbers")
            if positions.shape != q.shape[:-2] + (len(axes),) or not axes:
                raise ValueError("qk_norm_rope: positions [..., axes], one width of `axes` each")
            positions = positions.to(torch.int32).contiguous()
        lead = q.shape[:-2]
        R = math.prod(lead)
        qr, kr = _rows(q.reshape(R, Hq, d)), _rows(k.reshape(R, Hk, d))
        q_weight = None if q_weight is None else q_weight.contiguous()
        k_weight = None if k_weight is None else k_weight.contiguous()
        # (In their own shape, and not saved: views would refuse to be changed in place.)
        qo, ko = (torch.empty(t.shape, dtype=q.dtype, device=q.device) for t in (q, k))
        with _on(q):
            adaln_qk_norm_rope_fwd(qr, kr, q_weight, k_weight, positions, qo, ko, R, Hq, Hk, d, _ld(qr), _ld(kr),
                                   Hq * d, Hk * d, axes, theta, eps, norm, dt)
        ctx.save_for_backward(*((qr, kr) if norm else (None, None)), q_weight, k_weight, positions)
        ctx.sizes = lead, R, Hq, Hk, d
        ctx.args = axes, theta, eps, norm
        return qo, ko

    @staticmethod
    @once_differentiable
    def backward(ctx, dqo, dko):
        q, k, q_weight, k_weight, positions = ctx.saved_tensors
        lead, R, Hq, Hk, d = ctx.sizes
        axes, theta, eps, norm = ctx.args
        dt = _code(dqo)
        dqo, dko = _rows(dqo.reshape(R, Hq, d)), _rows(dko.reshape(R, Hk, d))
        dq = torch.empty((R, Hq, d), dtype=dqo.dtype, device=dqo.device)
        dk = torch.empty((R, Hk, d), dtype=dqo.dtype, device=dqo.device)
        dwq, dwk = (torch.empty(d, dtype=torch.float32, device=dqo.device) if w is not None and need else None
                    for w, need in ((q_weight, ctx.needs_input_grad[2]), (k_weight, ctx.needs_input_grad[3])))
        with _on(dqo):
            nb = adaln_qk_norm_rope_bwd_workspace_size(R, Hq, Hk, d, dt)
            ws = _workspace(nb, dqo.device)
            adaln_qk_norm_rope_bwd(dqo, dko, q, k, q_weight, k_weight, positions,
                                   dq, dk, dwq, dwk, ws, nb, R, Hq, Hk, d, _ld(dqo), _ld(dko), _ld(q) if norm else 0,
                                   _ld(k) if norm else 0, Hq * d, Hk * d, axes, theta, eps, norm, dt)
        return (dq.view(*lead, Hq, d), dk.view(*lead, Hk, d), None if dwq is None else dwq.to(dq.dtype),
                None if dwk is None else dwk.to(dq.dtype), None, None, None, None, None)


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: Optional[torch.Tensor] = None, axes=None,
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                 theta: float = 10000.0, eps: float = 1e-6, norm: bool = True):
    """Differentiable norms of each head of q [..., Hq, d] and k [..., Hk, d] and their rotation by
    positions [..., len(axes)] (whole numbers of 32 bits): pairs of neighbouring elements turn, the first axes[0]
    elements with the first position, and so on; elements behind the axes do not turn. Returns (q', k').
    norm=False: the rotation alone; positions=None: the norms alone."""
    return QKNormRopeFunction.apply(q, k, q_weight, k_weight, positions, axes, float(theta), float(eps), bool(norm))


class QKNormRope(torch.nn.Module):
    """``QKNormRope(d, axes)(q, k, positions)``: head norms with learned weights (ones), and the
    rotation."""

    def __init__(self, d: int, axes=None, theta: float = 10000.0, eps: float = 1e-6, device=None, dtype=None):
        super().__init__()
        self.axes = None if axes is None else tuple(int(w) for w in axes)
        self.theta, self.eps, self.d = float(theta), float(eps), int(d)
        self.q_weight = torch.nn.Parameter(torch.ones(d, device=device, dtype=dtype))
        self.k_weight = torch.nn.Parameter(torch.ones(d, device=device, dtype=dtype))

    def forward(self, q, k, positions=None):
        axes = self.axes if positions is not None else None
        return qk_norm_rope(q, k, positions, axes, self.q_weight, self.k_weight, self.theta, self.eps)

    def extra_repr(self) -> str:
        return "%d, axes=%s, theta=%g, eps=%g" % (self.d, self.axes, self.theta, self.eps)


class AttentionFunction(torch.autograd.Function):
    """(o, lse) of packed q [Rq, Hq, d], k and v [Rk, Hk, d] (see ``attention``). lse [Hq, Rq] fp32 carries no
    gradient. Saves q, k, v (as they come), o and lse, no scores."""

    @staticmethod
    def forward(ctx, q, k, v, cu_q, cu_k, nseg: int, causal: bool, scale: float, check_tables: bool):
        (Rq, Hq, d), (Rk, Hk, _) = q.shape, k.shape
        q, k, v = _rows(q), _rows(k), _rows(v)
        o = torch.empty((Rq, Hq, d), dtype=q.dtype, device=q.device)
        lse = torch.empty((Hq, Rq), dtype=torch.float32, device=q.device)
        with _on(q):
            nb = adaln_attention_fwd_workspace_size(nseg, Rq, Rk, Hq, Hk, d, ADALN_BF16)
            ws = _workspace(nb, q.device)
            adaln_attention_fwd(q, k, v, o, lse, cu_q, cu_k, nseg, Rq, Rk, Hq, Hk, d, _ld(q), _ld(k), _ld(v), Hq * d,
                                scale, causal, ws, nb, ADALN_BF16)
            if check_tables:
                _check_status(ws, "adaln_attention_fwd")
        ctx.save_for_backward(q, k, v, o, lse, cu_q, cu_k)
        ctx.args = nseg, causal, scale, check_tables
        ctx.mark_non_differentiable(lse)
        return o, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, _dlse):
        q, k, v, o, lse, cu_q, cu_k = ctx.saved_tensors
        nseg, causal, scale, check_tables = ctx.args
        (Rq, Hq, d), (Rk, Hk, _) = q.shape, k.shape
        dout = _rows(dout)
        want_q, want_kv = ctx.needs_input_grad[0], ctx.needs_input_grad[1] or ctx.needs_input_grad[2]
        dq = torch.empty((Rq, Hq, d), dtype=q.dtype, device=q.device) if want_q else None
        dk, dv = (torch.empty((Rk, Hk, d), dtype=q.dtype, device=q.device) if want_kv else None for _ in range(2))
        with _on(q):
            nb = adaln_attention_bwd_workspace_size(nseg, Rq, Rk, Hq, Hk, d, ADALN_BF16)
            ws = _workspace(nb, q.device)
            adaln_attention_bwd(dout, q, k, v, o, lse, dq, dk, dv, cu_q, cu_k, nseg, Rq, Rk, Hq, Hk, d, _ld(dout),
                                _ld(q), _ld(k), _ld(v), Hq * d, Hq * d, Hk * d, Hk * d, scale, causal, ws, nb,
                                ADALN_BF16)
            if check_tables:
                _check_status(ws, "adaln_attention_bwd")
        return dq, dk, dv, None, None, None, None, None, None


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
              cu_seqlens_k: Optional[torch.Tensor] = None, causal: bool = False, scale: Optional[float] = None,
              check_tables: bool = False, return_lse: bool = False):
    """Differentiable softmax attention (bfloat16).

    Packed: q [Rq, Hq, d], k and v [Rk, Hk, d] with cu_seqlens [nseg + 1] of the queries and cu_seqlens_k
    of the keys (the queries' if absent). Dense: q [B, N, Hq, d], k and v [B, M, Hk, d], no tables. Hq is a
    multiple of Hk, d a multiple of 8 up to 128. causal: query i of n sees keys j <= i + m - n. scale:
    d ** -0.5 if None. Returns o like q; with return_lse also lse, [Hq, Rq] or [Hq, B, N], which carries no
    gradient. Sums and lse are fp32; probabilities and their gradients are rounded to bfloat16 for the next
    product, and the backward takes the bfloat16 o: errors of 1.4 roundings in o and dv, 1.4 to 1.8 in dq and dk.
    q, k and v whose heads or rows the library cannot take as they lie (a slice of a dense batch's rows among
    them) are copied. ``check_tables`` reads the call's device status (it synchronises the stream); without it
    malformed tables leave the outputs unwritten."""
    if not q.is_cuda:
        raise ValueError("attention runs on CUDA tensors")
    if any(t.dtype != torch.bfloat16 for t in (q, k, v)):
        raise TypeError("attention takes bfloat16 q, k and v, got %s, %s and %s" % (q.dtype, k.dtype, v.dtype))
    packed = cu_seqlens is not None
    n = 3 if packed else 4
    if q.dim() != n or k.dim() != n or v.shape != k.shape or k.shape[-1] != q.shape[-1] or (
            not packed and k.shape[0] != q.shape[0]):
        raise ValueError("attention: packed q [Rq, Hq, d], k and v [Rk, Hk, d] with cu_seqlens, or dense "
                         "q [B, N, Hq, d], k and v [B, M, Hk, d]")
    if any(t is not None and t.device != q.device for t in (k, v, cu_seqlens, cu_seqlens_k)):
        raise ValueError("q, k, v and the tables must be on one device")
    scale = q.shape[-1] ** -0.5 if scale is None else float(scale)
    if packed:
        cu_seqlens_k = cu_seqlens if cu_seqlens_k is None else cu_seqlens_k
        if cu_seqlens.dim() != 1 or cu_seqlens.shape != cu_seqlens_k.shape or cu_seqlens.numel() == 0:
            raise ValueError("attention: cu_seqlens and cu_seqlens_k are [nseg + 1]")
        cu_q, cu_k = (c.to(torch.int32).contiguous() for c in (cu_seqlens, cu_seqlens_k))
        o, lse = AttentionFunction.apply(q, k, v, cu_q, cu_k, cu_q.numel() - 1, bool(causal), scale, check_tables)
        return (o, lse) if return_lse else o
    if cu_seqlens_k is not None:
        raise ValueError("attention: cu_seqlens_k goes with cu_seqlens")
    B, N = q.shape[:2]
    o, lse = AttentionFunction.apply(q.flatten(0, 1), k.flatten(0, 1), v.flatten(0, 1), None, None, B, bool(causal),
                                     scale, check_tables)
    o = o.view(B, N, *o.shape[1:])
    return (o, lse.view(lse.shape[0], B, N)) if return_lse else o
