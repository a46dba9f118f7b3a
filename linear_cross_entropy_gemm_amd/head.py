"""The operators around the vocabulary projection, on torch tensors: dropout
with its residual add and the final layer norm in front of it, with their
backward passes, and drawing tokens from the logits behind it.  Every step
of the computation runs in the library's HIP kernels on torch's current
stream of the tensors' device; nothing synchronises, and every function can
be captured in a graph.  The differentiable ones have a backward pass;
forward-mode derivatives are refused (NotImplementedError).  (A captured
backward pass may meet leaves of which a graph built on another side stream is
alive, but none built on the default stream; where one of these functions
built it, the pass is refused.)"""
from __future__ import annotations

import dataclasses
import operator
from typing import Optional, Union

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .mx import MX_BLOCK, Mx4Weight, Mx8Rows, logits_mx4
from .torch_api import (_DTYPES, _enqueue, _ptr, _workspace, check_backward, has_tangent, linear_cross_entropy,
                        logits as _logits, note_leaves)

_U64 = (1 << 64) - 1


@dataclasses.dataclass
class LayerNormForward:
    y: torch.Tensor      # shape and dtype of x
    mean: torch.Tensor   # [...] fp32, one per row
    rstd: torch.Tensor   # [...] fp32, one per row


@dataclasses.dataclass
class LayerNormGrads:
    grad_x: Optional[torch.Tensor]        # shape and dtype of x
    grad_weight: Optional[torch.Tensor]   # [H] dtype of the weight
    grad_bias: Optional[torch.Tensor]     # [H] dtype of the weight


@dataclasses.dataclass
class RmsNormForward:
    y: torch.Tensor                   # shape and dtype of x
    residual: Optional[torch.Tensor]  # x + residual, shape and dtype of x (None without a residual)
    rstd: torch.Tensor                # [...] fp32, one per row


@dataclasses.dataclass
class RmsNormMx8:
    rows: Mx8Rows                     # y in 8 bits
    residual: Optional[torch.Tensor]  # x + residual, shape and dtype of x (None without a residual)


@dataclasses.dataclass
class RmsNormGrads:
    grad_x: Optional[torch.Tensor]       # shape and dtype of x; also the gradient of the residual
    grad_weight: Optional[torch.Tensor]  # [H] dtype of the weight


@dataclasses.dataclass
class SampleOutputs:
    tokens: torch.Tensor                     # [...] int64; -1: nothing to draw
    logprobs: Optional[torch.Tensor] = None  # [...] fp32, of the filtered distribution


@dataclasses.dataclass
class VerifyOutputs:
    tokens: torch.Tensor                     # [..., K + 1] int64: the accepted, one drawn, then -1
    accepted: torch.Tensor                   # [...] int64: how many of the drafted tokens
    logprobs: Optional[torch.Tensor] = None  # [..., K + 1] fp32 of the target's distributions


def _rows(x: torch.Tensor) -> torch.Tensor:
    """x as [M, H] with unit column stride: a view where the strides allow
    one, so a slice of a wider buffer is read in place."""
    x2 = x if x.dim() == 2 else x.reshape(-1, x.shape[-1])
    return x2 if x2.stride(1) == 1 or x2.shape[1] == 1 else x2.contiguous()


def _like(x: torch.Tensor) -> torch.Tensor:
    """A new contiguous tensor of x's shape and dtype (a shape read from
    Python and passed back takes twice as long)."""
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def _check_tensor(name: str, x: torch.Tensor) -> None:
    if x.dtype not in _DTYPES:
        raise TypeError(f"{name} must be bfloat16 or float32 (got {x.dtype})")
    if not x.is_cuda:
        raise ValueError(f"{name} must be on the GPU")


def _check_rows(name: str, x: torch.Tensor) -> None:
    _check_tensor(name, x)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"{name} must have a last dimension of at least one element")


def _check_params(x: torch.Tensor, weight: Optional[torch.Tensor], bias: Optional[torch.Tensor]):
    """Contiguous weight and bias (None stays None) and their common dtype."""
    def one(name, t):
        if t.dtype not in _DTYPES:
            raise TypeError(f"{name} must be bfloat16 or float32 (got {t.dtype})")
        if t.dim() != 1 or t.shape[0] != x.shape[-1]:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, this call needs {(x.shape[-1],)}")
        if t.device != x.device:
            raise ValueError(f"{name} is on {t.device}, x is on {x.device}")
        return t.contiguous()

    w_dtype = x.dtype
    if bias is not None:
        bias = one("bias", bias)
        w_dtype = bias.dtype
    if weight is not None:
        weight = one("weight", weight)
        if bias is not None and weight.dtype != w_dtype:
            raise TypeError(f"weight and bias must have one dtype (got {weight.dtype}, {w_dtype})")
        w_dtype = weight.dtype
    return weight, bias, w_dtype


def _layer_norm_fwd(x, weight, bias, eps, stats: bool):
    _check_rows("x", x)
    w, b, w_dtype = _check_params(x, weight, bias)
    eps = float(eps)
    x2 = _rows(x)
    M, H = x2.shape
    dev = x.device
    y = _like(x)
    mean = rstd = None
    if stats:
        mean = torch.empty(M if x.dim() == 2 else x.shape[:-1], dtype=torch.float32, device=dev)
        rstd = torch.empty_like(mean)
    rc = _enqueue(dev, lambda stream: _lib.flce_layer_norm_fwd(
        x2.data_ptr(), x2.stride(0), _ptr(w), _ptr(b), M, H, eps, y.data_ptr(), H, _ptr(mean), _ptr(rstd), stream,
        _DTYPES[x.dtype], _DTYPES[w_dtype]))
    if rc != _lib.FLCE_OK:
        raise _lib.FlceError(rc, "flce_layer_norm_fwd")
    return y, mean, rstd


def layer_norm_fwd(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                   eps: float = 1e-5) -> LayerNormForward:
    """One call of ``flce_layer_norm_fwd`` over the last dimension of ``x``:
    y and the row statistics that ``layer_norm_bwd`` takes.  ``weight`` and
    ``bias`` [H] may be absent and may be float32 next to a bfloat16 ``x``."""
    return LayerNormForward(*_layer_norm_fwd(x, weight, bias, eps, True))


def layer_norm_bwd(grad_y: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], mean: torch.Tensor,
                   rstd: torch.Tensor, workspace: Optional[torch.Tensor] = None, *, need_x: bool = True,
                   need_params: bool = True, param_dtype: Optional[torch.dtype] = None) -> LayerNormGrads:
    """One call of ``flce_layer_norm_bwd``: the gradients of ``x``, of the
    weight and of the bias (in the weight's dtype; without a weight in
    ``param_dtype``, that of ``x`` by default).  ``mean`` and ``rstd`` are those of ``layer_norm_fwd``.  A
    caller-owned ``workspace`` (uint8, ``flce_layer_norm_bwd_workspace_size``)
    may be reused by ordered calls."""
    _check_rows("x", x)
    w, _, w_dtype = _check_params(x, weight, None)
    if param_dtype is not None and param_dtype != w_dtype:
        if w is not None or param_dtype not in _DTYPES:
            raise TypeError(f"param_dtype must be the weight's dtype, or bfloat16 or float32 without one (got "
                            f"{param_dtype})")
        w_dtype = param_dtype
    if grad_y.shape != x.shape or grad_y.dtype != x.dtype or grad_y.device != x.device:
        raise ValueError(f"grad_y must match x: {tuple(x.shape)} {x.dtype} on {x.device} (got "
                         f"{tuple(grad_y.shape)} {grad_y.dtype} on {grad_y.device})")
    x2, g2 = _rows(x), _rows(grad_y)
    M, H = x2.shape
    dev = x.device
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t.dtype != torch.float32 or t.numel() != M or t.device != dev or not t.is_contiguous():
            raise ValueError(f"{name} must hold one contiguous float32 value per row of x on its device")
    gx = _like(x) if need_x else None
    gw = gb = None
    ws_bytes = 0
    if need_params:
        gw = torch.empty(H, dtype=w_dtype, device=dev)
        gb = torch.empty_like(gw)
        ws_bytes = _lib.flce_layer_norm_bwd_workspace_size(M, H, _DTYPES[x.dtype])
        if ws_bytes == 0:
            raise _lib.FlceError(_lib.FLCE_EUNSUPPORTED, "flce_layer_norm_bwd_workspace_size")
        workspace = _workspace(workspace, ws_bytes, dev)
        ws_bytes = workspace.numel()
    rc = _enqueue(dev, lambda stream: _lib.flce_layer_norm_bwd(
        g2.data_ptr(), g2.stride(0), x2.data_ptr(), x2.stride(0), _ptr(w), mean.data_ptr(), rstd.data_ptr(), M, H,
        _ptr(gx), H, _ptr(gw), _ptr(gb), stream, _DTYPES[x.dtype], _DTYPES[w_dtype],
        _ptr(workspace) if need_params else None, ws_bytes))
    if rc != _lib.FLCE_OK:
        raise _lib.FlceError(rc, "flce_layer_norm_bwd")
    return LayerNormGrads(gx, gw, gb)


def _needs_grad(*tensors) -> bool:
    """Whether the call has to go through its autograd function: for a backward
    pass, or because an input carries a forward-mode tangent (in grad mode or
    not), which the function refuses and a plain call would drop."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        return True
    return has_tangent(*tensors)


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        o = layer_norm_fwd(x, weight, bias, eps)
        ctx.save_for_backward(x, weight, o.mean, o.rstd)
        ctx.b_dtype = None if bias is None else bias.dtype
        return o.y

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y):
        check_backward(ctx, grad_y)
        x, weight, mean, rstd = ctx.saved_tensors
        need_x, need_w, need_b, _ = ctx.needs_input_grad
        g = layer_norm_bwd(grad_y, x, weight, mean, rstd, need_x=need_x, need_params=need_w or need_b,
                           param_dtype=ctx.b_dtype)
        return g.grad_x, g.grad_weight if need_w else None, g.grad_bias if need_b else None, None


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5) -> torch.Tensor:
    """Differentiable layer norm over the last dimension of ``x``.  A row's
    statistics are kept for the backward pass, the normalised values are not:
    they are formed again from ``x``, in the gradients with the mean as one
    fp32 number (off by up to 2^-24 |mean| / std there, not in the output)."""
    if not _needs_grad(x, weight, bias):
        return _layer_norm_fwd(x, weight, bias, eps, False)[0]
    y = _LayerNorm.apply(x, weight, bias, eps)
    note_leaves(y)
    return y


def _check_like(name: str, t: torch.Tensor, x: torch.Tensor, of: str = "x") -> None:
    if t.shape != x.shape or t.dtype != x.dtype or t.device != x.device:
        raise ValueError(f"{name} must match {of}: {tuple(x.shape)} {x.dtype} on {x.device} (got {tuple(t.shape)} "
                         f"{t.dtype} on {t.device})")


def _rms_norm_fwd(x, weight, eps, residual, offset, stats: bool, mx8: bool = False):
    """(y or (data, scales), s, rstd): one call of the forward kernels."""
    _check_rows("x", x)
    w, _, w_dtype = _check_params(x, weight, None)
    eps, offset = float(eps), float(offset)
    x2 = _rows(x)
    M, H = x2.shape
    dev = x.device
    s = r2 = None
    if residual is not None:
        _check_like("residual", residual, x)
        r2 = _rows(residual)
        s = _like(x)
    rstd = torch.empty(M if x.dim() == 2 else x.shape[:-1], dtype=torch.float32, device=dev) if stats else None
    ld_r = 0 if r2 is None else r2.stride(0)
    if mx8:
        nb = (H + MX_BLOCK - 1) // MX_BLOCK
        y = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=dev)
        scales = torch.empty((*x.shape[:-1], nb), dtype=torch.float8_e8m0fnu, device=dev)
        rc = _enqueue(dev, lambda stream: _lib.flce_rms_norm_mx(
            x2.data_ptr(), x2.stride(0), _ptr(r2), ld_r, _ptr(w), offset, M, H, eps, y.data_ptr(), H,
            scales.data_ptr(), nb, _ptr(s), H, _ptr(rstd), stream, _DTYPES[x.dtype], _DTYPES[w_dtype]))
        y = Mx8Rows(y, scales)
    else:
        y = _like(x)
        rc = _enqueue(dev, lambda stream: _lib.flce_rms_norm_fwd(
            x2.data_ptr(), x2.stride(0), _ptr(r2), ld_r, _ptr(w), offset, M, H, eps, y.data_ptr(), H, _ptr(s), H,
            _ptr(rstd), stream, _DTYPES[x.dtype], _DTYPES[w_dtype]))
    if rc != _lib.FLCE_OK:
        raise _lib.FlceError(rc, "flce_rms_norm_mx" if mx8 else "flce_rms_norm_fwd")
    return y, s, rstd


def rms_norm_fwd(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6, *,
                 residual: Optional[torch.Tensor] = None, offset: float = 0.0) -> RmsNormForward:
    """One call of ``flce_rms_norm_fwd`` over the last dimension of ``x`` (plus
    ``residual``): y, the new residual stream (the sum rounded to its type,
    which is what is normed) and the row statistic that ``rms_norm_bwd``
    takes.  ``weight`` [H] may be absent and may be float32 next to a bfloat16
    ``x``; ``offset`` is added to it (1 for weights kept around zero)."""
    return RmsNormForward(*_rms_norm_fwd(x, weight, eps, residual, offset, True))


def rms_norm_mx8(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6, *,
                 residual: Optional[torch.Tensor] = None, offset: float = 0.0) -> RmsNormMx8:
    """``rms_norm_fwd`` with y in 8 bits, one scale for 32 elements
    (``flce_rms_norm_mx``), as ``logits_mx4`` takes it."""
    y, s, _ = _rms_norm_fwd(x, weight, eps, residual, offset, False, mx8=True)
    return RmsNormMx8(y, s)


def rms_norm_bwd(grad_y: torch.Tensor, s: torch.Tensor, weight: Optional[torch.Tensor], rstd: torch.Tensor,
                 workspace: Optional[torch.Tensor] = None, *, offset: float = 0.0,
                 grad_residual: Optional[torch.Tensor] = None, need_x: bool = True,
                 need_weight: bool = True) -> RmsNormGrads:
    """One call of ``flce_rms_norm_bwd``: the gradient of ``x`` (and alike of the
    residual) and of the weight.  ``s`` and ``rstd`` are those of
    ``rms_norm_fwd`` (``s``: its residual output, or ``x`` itself without one);
    ``grad_residual`` is the gradient that reaches the residual stream from
    elsewhere.  Without a weight there is no gradient of it.  A caller-owned
    ``workspace`` (uint8, ``flce_rms_norm_bwd_workspace_size``) may be reused by
    ordered calls."""
    _check_rows("s", s)
    w, _, w_dtype = _check_params(s, weight, None)
    _check_like("grad_y", grad_y, s, "s")
    s2, g2 = _rows(s), _rows(grad_y)
    a2 = None
    if grad_residual is not None:
        _check_like("grad_residual", grad_residual, s, "s")
        a2 = _rows(grad_residual)
    M, H = s2.shape
    dev = s.device
    if rstd.dtype != torch.float32 or rstd.numel() != M or rstd.device != dev or not rstd.is_contiguous():
        raise ValueError("rstd must hold one contiguous float32 value per row of s on its device")
    gx = _like(s) if need_x else None
    gw = None
    ws_bytes = 0
    if need_weight and w is not None:
        gw = torch.empty(H, dtype=w_dtype, device=dev)
        ws_bytes = _lib.flce_rms_norm_bwd_workspace_size(M, H, _DTYPES[s.dtype])
        if ws_bytes == 0:
            raise _lib.FlceError(_lib.FLCE_EUNSUPPORTED, "flce_rms_norm_bwd_workspace_size")
        workspace = _workspace(workspace, ws_bytes, dev)
        ws_bytes = workspace.numel()
    rc = _enqueue(dev, lambda stream: _lib.flce_rms_norm_bwd(
        g2.data_ptr(), g2.stride(0), s2.data_ptr(), s2.stride(0), _ptr(a2), 0 if a2 is None else a2.stride(0), _ptr(w),
        float(offset), rstd.data_ptr(), M, H, _ptr(gx), H, _ptr(gw), stream, _DTYPES[s.dtype], _DTYPES[w_dtype],
        _ptr(workspace) if gw is not None else None, ws_bytes))
    if rc != _lib.FLCE_OK:
        raise _lib.FlceError(rc, "flce_rms_norm_bwd")
    return RmsNormGrads(gx, gw)


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps, offset):
        o = rms_norm_fwd(x, weight, eps, residual=residual, offset=offset)
        ctx.set_materialize_grads(False)
        ctx.offset = offset
        ctx.save_for_backward(x if residual is None else o.residual, weight, o.rstd)
        return o.y if residual is None else (o.y, o.residual)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_y, grad_s=None):
        need_x, need_r, need_w = ctx.needs_input_grad[:3]
        for g in (grad_y, grad_s):
            if g is not None:
                check_backward(ctx, g)
        if grad_y is None:   # only the residual stream goes on
            return grad_s if need_x else None, grad_s if need_r else None, None, None, None
        s, weight, rstd = ctx.saved_tensors
        g = rms_norm_bwd(grad_y, s, weight, rstd, offset=ctx.offset, grad_residual=grad_s, need_x=need_x or need_r,
                         need_weight=need_w)
        return g.grad_x if need_x else None, g.grad_x if need_r else None, g.grad_weight, None, None


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6, *,
             residual: Optional[torch.Tensor] = None, offset: float = 0.0):
    """Differentiable RMS norm over the last dimension of ``x``: y, or with a
    ``residual`` (y of x + residual, the new residual stream x + residual).
    Kept for the backward pass are the stream and one number per row."""
    if not _needs_grad(x, residual, weight):
        y, s, _ = _rms_norm_fwd(x, weight, eps, residual, offset, False)
        return y if residual is None else (y, s)
    out = _RmsNorm.apply(x, residual, weight, float(eps), float(offset))
    note_leaves(out if residual is None else out[0])
    return out


def _dropout(x, p, seed, offset, residual) -> torch.Tensor:
    xc = x.contiguous()
    res = None if residual is None else residual.contiguous()
    dev = x.device
    y = _like(x)
    tensor = torch.is_tensor(offset)
    rc = _enqueue(dev, lambda stream: _lib.flce_dropout(
        xc.data_ptr(), _ptr(res), y.data_ptr(), xc.numel(), p, seed, 0 if tensor else offset,
        offset.data_ptr() if tensor else None, stream, _DTYPES[x.dtype]))
    if rc != _lib.FLCE_OK:
        raise _lib.FlceError(rc, "flce_dropout")
    return y


class _Dropout(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, offset):
        if torch.is_tensor(offset):
            # kept as autograd state: changing it in place before the backward
            # pass raises there instead of drawing another mask
            ctx.save_for_backward(offset)
            ctx.args = (p, seed, None)
        else:
            ctx.args = (p, seed, offset)
        return _dropout(x, p, seed, offset, residual)

    @staticmethod
    def backward(ctx, grad_y):
        check_backward(ctx, grad_y)
        # the same map on the upstream gradient, itself differentiable
        p, seed, offset = ctx.args
        gx = None
        if ctx.needs_input_grad[0]:
            gx = dropout(grad_y, p, seed, ctx.saved_tensors[0] if offset is None else offset)
        return gx, grad_y if ctx.needs_input_grad[1] else None, None, None, None


def dropout(x: torch.Tensor, p: float, seed: int, offset: Union[int, torch.Tensor] = 0,
            residual: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Differentiable dropout, ``[residual +] keep * x / (1 - p)``
    (``flce_dropout``); the mask is a function of the element's position in
    row-major order, of ``seed`` and of ``offset`` and is formed again in the
    backward pass.  Draw each layer's and step's mask with a (seed, offset) of
    its own.  ``offset`` may be an int64 tensor of one element on the device
    of ``x``: a captured graph draws a new mask on each replay when the
    program advances it in between."""
    _check_tensor("x", x)
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must lie in [0, 1] (got {p})")
    seed = operator.index(seed)
    if not 0 <= seed <= _U64:
        raise ValueError("seed must be an unsigned 64-bit integer")
    if torch.is_tensor(offset):
        if offset.dtype != torch.int64 or offset.numel() != 1 or offset.device != x.device:
            raise ValueError("a tensor offset must be one int64 on the device of x")
    else:
        offset = operator.index(offset)
        if not 0 <= offset <= _U64:
            raise ValueError("offset must be an unsigned 64-bit integer")
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype
                                 or residual.device != x.device):
        raise ValueError(f"residual must match x: {tuple(x.shape)} {x.dtype} on {x.device} (got "
                         f"{tuple(residual.shape)} {residual.dtype} on {residual.device})")
    if not _needs_grad(x, residual):
        return _dropout(x, float(p), seed, offset, residual)
    y = _Dropout.apply(x, residual, float(p), seed, offset)
    note_leaves(y)
    return y


def _check_norm(norm: str, bias, offset: float) -> None:
    if norm not in ("layer", "rms"):
        raise ValueError(f"norm must be 'layer' or 'rms' (got {norm!r})")
    if norm == "rms" and bias is not None:
        raise ValueError("an RMS norm has no bias")
    if norm == "layer" and offset != 0.0:
        raise ValueError("norm_offset is that of an RMS norm")


def lm_head_loss(x: torch.Tensor, W: torch.Tensor, labels: torch.Tensor, norm_weight: Optional[torch.Tensor],
                 norm_bias: Optional[torch.Tensor] = None, eps: float = 1e-5, *,
                 residual: Optional[torch.Tensor] = None, dropout_p: float = 0.0, seed: int = 0,
                 offset: Union[int, torch.Tensor] = 0, ignore_index: int = -100, softcap: Optional[float] = None,
                 multiplier: float = 1.0, reduction: str = "mean", workspace: Optional[torch.Tensor] = None,
                 check: bool = False, norm: str = "layer", norm_offset: float = 0.0):
    """The whole head of a training step, differentiable: the last block's
    output ``x`` through dropout onto the ``residual`` stream (when either is
    asked for), the final norm (``norm``: "layer", or "rms" with
    ``norm_offset`` added to its weight and no bias), and the fused linear
    cross-entropy.  Returns (loss, n_correct) as ``linear_cross_entropy``
    does."""
    _check_norm(norm, norm_bias, norm_offset)
    if norm == "rms" and residual is not None and dropout_p == 0.0:
        y = rms_norm(x, norm_weight, eps, residual=residual, offset=norm_offset)[0]
    else:
        if dropout_p != 0.0 or residual is not None:
            x = dropout(x, dropout_p, seed, offset, residual)
        if norm == "rms":
            y = rms_norm(x, norm_weight, eps, offset=norm_offset)
        else:
            y = layer_norm(x, norm_weight, norm_bias, eps)
    return linear_cross_entropy(y, W, labels, ignore_index, softcap, multiplier, reduction, workspace, check)


def _sample_param(name: str, v, dtype, N: int, dev, prm) -> Optional[torch.Tensor]:
    """A scalar goes into the parameter block, a tensor's address into its
    per-row field; the tensor is returned to be kept alive for the call."""
    if not torch.is_tensor(v):
        if dtype == torch.int64:
            v = operator.index(v)
            if not -1 << 63 <= v < 1 << 63:   # the C field would take it modulo 2^64
                raise ValueError(f"{name} must fit 64 bits (got {v})")
            setattr(prm, name, v)
        else:
            setattr(prm, name, float(v))
        return None
    if v.dtype != dtype or v.device != dev or v.numel() != N:
        raise ValueError(f"{name} must be a number or one {dtype} per row on {dev}")
    v = v.contiguous()
    setattr(prm, name + "_rows", _ptr(v))
    return v


def sample(logits: torch.Tensor, u: torch.Tensor, temperature: Union[float, torch.Tensor] = 1.0,
           top_k: Union[int, torch.Tensor] = 0, top_p: Union[float, torch.Tensor] = 1.0,
           min_p: Union[float, torch.Tensor] = 0.0, *, logprobs: bool = False,
           workspace: Optional[torch.Tensor] = None) -> SampleOutputs:
    """One call of ``flce_sample``: a token for every row of ``logits``
    [..., V] (which may be a row-padded view) from the random numbers ``u``
    [...], float32 in [0, 1).  ``temperature`` (0: the first maximum),
    ``top_k`` (0: off), ``top_p`` (1: off) and ``min_p`` (0: off) are numbers,
    or tensors with one value per row (float32; int64 for ``top_k``) on the
    device of ``logits``; they apply in that order, min-p relative to the
    largest probability.  A row without a logit above -inf, or with a per-row
    value out of range, gets token -1.  A caller-owned ``workspace`` (uint8,
    ``flce_sample_workspace_size``) may be reused by ordered calls."""
    _check_rows("logits", logits)
    z = _rows(logits)
    N, V = z.shape
    dev = logits.device
    if u.dtype != torch.float32 or u.device != dev or u.numel() != N:
        raise ValueError(f"u must hold one float32 per row of logits on {dev}")
    u = u.contiguous()
    prm, keep = _sample_params(temperature, top_k, top_p, min_p, N, dev)
    dtype = _DTYPES[logits.dtype]
    ws_bytes = _lib.flce_sample_workspace_size(N, V, dtype)
    if ws_bytes == 0:
        raise _lib.FlceError(_lib.FLCE_EUNSUPPORTED, "flce_sample_workspace_size")
    workspace = _workspace(workspace, ws_bytes, dev)
    shape = N if logits.dim() == 2 else logits.shape[:-1]
    res = SampleOutputs(torch.empty(shape, dtype=torch.int64, device=dev),
                        torch.empty(shape, dtype=torch.float32, device=dev) if logprobs else None)
    rc = _enqueue(dev, lambda stream: _lib.flce_sample(
        z.data_ptr(), z.stride(0), u.data_ptr(), N, V, prm, res.tokens.data_ptr(), _ptr(res.logprobs), stream, dtype,
        workspace.data_ptr(), workspace.numel()))
    del keep
    if rc != _lib.FLCE_OK:
        raise _lib.FlceError(rc, "flce_sample")
    return res


def _sample_params(temperature, top_k, top_p, min_p, N, dev):
    """The parameter block, and the tensors to be kept alive for the call."""
    prm = _lib.flce_sample_params_t()
    keep = [_sample_param(n, v, d, N, dev, prm) for n, v, d in (
        ("temperature", temperature, torch.float32), ("top_k", top_k, torch.int64),
        ("top_p", top_p, torch.float32), ("min_p", min_p, torch.float32))]
    return prm, keep


def verify(target_logits: torch.Tensor, draft_tokens: torch.Tensor, u: torch.Tensor, u_draw: torch.Tensor, *,
           draft_logits: Optional[torch.Tensor] = None, draft_lens: Optional[torch.Tensor] = None,
           temperature: Union[float, torch.Tensor] = 1.0, top_k: Union[int, torch.Tensor] = 0,
           top_p: Union[float, torch.Tensor] = 1.0, min_p: Union[float, torch.Tensor] = 0.0,
           draft_temperature: Union[None, float, torch.Tensor] = None,
           draft_top_k: Union[None, int, torch.Tensor] = None, draft_top_p: Union[None, float, torch.Tensor] = None,
           draft_min_p: Union[None, float, torch.Tensor] = None, logprobs: bool = False,
           workspace: Optional[torch.Tensor] = None) -> VerifyOutputs:
    """One call of ``flce_verify``: which of the ``draft_tokens`` [..., K] (int64)
    stand, and one token more, distributed as if ``sample`` had drawn them all
    from ``target_logits`` [..., K + 1, V].  ``draft_logits`` [..., K, V] are
    what the tokens were drawn from (None: they were certain); ``u`` [..., K]
    and ``u_draw`` [...] are float32 random numbers in [0, 1); ``draft_lens``
    [...] (int64) says how many tokens of each sequence were drafted.  The
    sampling parameters are numbers, or tensors with one value per sequence;
    the draft's are those of the target where not given.  (With more than 256
    rows, flat ones under top-p alone take less time with ``top_p`` as a number
    than as a tensor.)  A caller-owned ``workspace`` (uint8,
    ``flce_verify_workspace_size``) may be reused by ordered calls."""
    _check_rows("target_logits", target_logits)
    if target_logits.dim() < 2 or target_logits.shape[-2] < 1:
        raise ValueError(f"target_logits must be [..., K + 1, V] (got {tuple(target_logits.shape)})")
    lead, K, V = target_logits.shape[:-2], target_logits.shape[-2] - 1, target_logits.shape[-1]
    dev = target_logits.device
    z = _rows(target_logits)
    B = z.shape[0] // (K + 1)

    def check(name, t, dtype, shape):
        if t.dtype != dtype or t.device != dev or t.shape != shape:
            raise ValueError(f"{name} must be {tuple(shape)} {dtype} on {dev} (got {tuple(t.shape)} {t.dtype} on "
                             f"{t.device})")
        return t.contiguous()

    x = check("draft_tokens", draft_tokens, torch.int64, (*lead, K))
    u = check("u", u, torch.float32, (*lead, K))
    u_draw = check("u_draw", u_draw, torch.float32, lead)
    lens = None if draft_lens is None else check("draft_lens", draft_lens, torch.int64, lead)
    d = None
    if draft_logits is not None:
        if draft_logits.shape != (*lead, K, V) or draft_logits.dtype != z.dtype or draft_logits.device != dev:
            raise ValueError(f"draft_logits must be {(*lead, K, V)} {z.dtype} on {dev} (got "
                             f"{tuple(draft_logits.shape)} {draft_logits.dtype} on {draft_logits.device})")
        d = _rows(draft_logits) if K > 0 else None
    prm, keep = _sample_params(temperature, top_k, top_p, min_p, B, dev)
    prm2 = None
    if not (draft_temperature is None and draft_top_k is None and draft_top_p is None and draft_min_p is None):
        prm2, keep2 = _sample_params(
            temperature if draft_temperature is None else draft_temperature, top_k if draft_top_k is None else
            draft_top_k, top_p if draft_top_p is None else draft_top_p, min_p if draft_min_p is None else draft_min_p,
            B, dev)
        keep += keep2
    dtype = _DTYPES[z.dtype]
    ws_bytes = _lib.flce_verify_workspace_size(B, K, V, dtype, 0 if d is None else 1)
    if ws_bytes == 0:
        raise _lib.FlceError(_lib.FLCE_EUNSUPPORTED, "flce_verify_workspace_size")
    workspace = _workspace(workspace, ws_bytes, dev)
    shape = (*lead, K + 1)
    res = VerifyOutputs(torch.empty(shape, dtype=torch.int64, device=dev),
                        torch.empty(lead, dtype=torch.int64, device=dev),
                        torch.empty(shape, dtype=torch.float32, device=dev) if logprobs else None)
    rc = _enqueue(dev, lambda stream: _lib.flce_verify(
        z.data_ptr(), z.stride(0), _ptr(d), 0 if d is None else d.stride(0), x.data_ptr(), _ptr(lens), u.data_ptr(),
        u_draw.data_ptr(), B, K, V, prm, prm2, res.tokens.data_ptr(), res.accepted.data_ptr(), _ptr(res.logprobs),
        stream, dtype, workspace.data_ptr(), workspace.numel()))
    del keep
    if rc != _lib.FLCE_OK:
        raise _lib.FlceError(rc, "flce_verify")
    return res


def _head_logits(x, W, norm_weight, norm_bias, eps, norm, norm_offset, residual, mx8, softcap, multiplier):
    """([N, V] logits of x's rows, the new residual stream): the final norm and
    the projection in bf16, fp32 or 4 bits."""
    _check_norm(norm, norm_bias, norm_offset)
    if residual is not None and norm != "rms":
        raise ValueError("a residual is added by an RMS norm")
    packed = isinstance(W, Mx4Weight)
    if mx8 and not (packed and norm == "rms"):
        raise ValueError("8-bit rows are those of an RMS norm in front of a projection in 4 bits")
    H = x.shape[-1]
    s = None
    if norm == "rms":
        y, s, _ = _rms_norm_fwd(x, norm_weight, eps, residual, norm_offset, False, mx8)
    else:
        y = _layer_norm_fwd(x, norm_weight, norm_bias, eps, False)[0]
    if mx8:
        y = Mx8Rows(y.data.reshape(-1, H), y.scales.reshape(-1, y.scales.shape[-1]))
    else:
        y = y.reshape(-1, H)
    return (logits_mx4 if packed else _logits)(y, W, softcap, multiplier), s


def lm_head_sample(x: torch.Tensor, W: Union[torch.Tensor, Mx4Weight], u: torch.Tensor,
                   norm_weight: Optional[torch.Tensor], norm_bias: Optional[torch.Tensor] = None, eps: float = 1e-5, *,
                   softcap: Optional[float] = None, multiplier: float = 1.0,
                   temperature: Union[float, torch.Tensor] = 1.0, top_k: Union[int, torch.Tensor] = 0,
                   top_p: Union[float, torch.Tensor] = 1.0, min_p: Union[float, torch.Tensor] = 0.0,
                   logprobs: bool = False, norm: str = "layer", norm_offset: float = 0.0,
                   residual: Optional[torch.Tensor] = None, mx8: bool = False) -> SampleOutputs:
    """The whole head of a decoding step: the final norm of the hidden states
    ``x`` [..., H] (``norm``: "layer", or "rms" of ``x`` plus ``residual`` with
    ``norm_offset`` added to its weight), the materialised logits (``logits``,
    or ``logits_mx4`` where ``W`` is in 4 bits, with ``mx8`` from 8-bit rows),
    and one token per row (``sample``)."""
    z, _ = _head_logits(x, W, norm_weight, norm_bias, eps, norm, norm_offset, residual, mx8, softcap, multiplier)
    o = sample(z, u, temperature, top_k, top_p, min_p, logprobs=logprobs)
    shape = x.shape[:-1]
    return SampleOutputs(o.tokens.reshape(shape), o.logprobs.reshape(shape) if logprobs else None)


def lm_head_verify(x: torch.Tensor, W: Union[torch.Tensor, Mx4Weight], draft_tokens: torch.Tensor, u: torch.Tensor,
                   u_draw: torch.Tensor, norm_weight: Optional[torch.Tensor],
                   norm_bias: Optional[torch.Tensor] = None, eps: float = 1e-5, *, softcap: Optional[float] = None,
                   multiplier: float = 1.0, norm: str = "layer", norm_offset: float = 0.0,
                   residual: Optional[torch.Tensor] = None, mx8: bool = False, **kwargs) -> VerifyOutputs:
    """The whole head of a step that verifies drafted tokens: the final norm of
    the hidden states ``x`` [..., K + 1, H], the materialised logits (both as
    in ``lm_head_sample``) and ``verify``, which takes the other arguments."""
    z, _ = _head_logits(x, W, norm_weight, norm_bias, eps, norm, norm_offset, residual, mx8, softcap, multiplier)
    return verify(z.reshape(*x.shape[:-1], z.shape[1]), draft_tokens, u, u_draw, **kwargs)
