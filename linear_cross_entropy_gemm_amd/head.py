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
class SampleOutputs:
    tokens: torch.Tensor                     # [...] int64; -1: nothing to draw
    logprobs: Optional[torch.Tensor] = None  # [...] fp32, of the filtered distribution


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


def lm_head_loss(x: torch.Tensor, W: torch.Tensor, labels: torch.Tensor, norm_weight: Optional[torch.Tensor],
                 norm_bias: Optional[torch.Tensor] = None, eps: float = 1e-5, *,
                 residual: Optional[torch.Tensor] = None, dropout_p: float = 0.0, seed: int = 0,
                 offset: Union[int, torch.Tensor] = 0, ignore_index: int = -100, softcap: Optional[float] = None,
                 multiplier: float = 1.0, reduction: str = "mean", workspace: Optional[torch.Tensor] = None,
                 check: bool = False):
    """The whole head of a training step, differentiable: the last block's
    output ``x`` through dropout onto the ``residual`` stream (when either is
    asked for), the final layer norm, and the fused linear cross-entropy.
    Returns (loss, n_correct) as ``linear_cross_entropy`` does."""
    if dropout_p != 0.0 or residual is not None:
        x = dropout(x, dropout_p, seed, offset, residual)
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
    prm = _lib.flce_sample_params_t()
    keep = [_sample_param(n, v, d, N, dev, prm) for n, v, d in (
        ("temperature", temperature, torch.float32), ("top_k", top_k, torch.int64),
        ("top_p", top_p, torch.float32), ("min_p", min_p, torch.float32))]
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


def lm_head_sample(x: torch.Tensor, W: torch.Tensor, u: torch.Tensor, norm_weight: Optional[torch.Tensor],
                   norm_bias: Optional[torch.Tensor] = None, eps: float = 1e-5, *, softcap: Optional[float] = None,
                   multiplier: float = 1.0, temperature: Union[float, torch.Tensor] = 1.0,
                   top_k: Union[int, torch.Tensor] = 0, top_p: Union[float, torch.Tensor] = 1.0,
                   min_p: Union[float, torch.Tensor] = 0.0, logprobs: bool = False) -> SampleOutputs:
    """The whole head of a decoding step: the final layer norm of the hidden
    states ``x`` [..., H], the materialised logits (``logits``), and one token
    per row (``sample``)."""
    y = _layer_norm_fwd(x, norm_weight, norm_bias, eps, False)[0]
    H = x.shape[-1]
    z = _logits(y.reshape(-1, H), W, softcap, multiplier)
    o = sample(z, u, temperature, top_k, top_p, min_p, logprobs=logprobs)
    shape = x.shape[:-1]
    return SampleOutputs(o.tokens.reshape(shape), o.logprobs.reshape(shape) if logprobs else None)
