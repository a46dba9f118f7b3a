"""The projection in the block formats of the OCP Microscaling specification,
on torch tensors: weights in 4 bits (MXFP4, E2M1), rows in 8 bits (MXFP8,
E4M3).  32 elements along a row share a scale, a power of two held as an E8M0
exponent."""
from __future__ import annotations

import dataclasses
from typing import Optional, Union

import torch

from . import _lib
from .torch_api import _DTYPES, _enqueue, _ptr, _workspace

MX_BLOCK = 32
MX_STEP = 128   # packed rows are padded to whole steps


@dataclasses.dataclass
class Mx8Rows:
    """Rows in 8 bits: element h of a row stands for data[..., h] *
    scales[..., h // 32]."""
    data: torch.Tensor     # [..., H] float8_e4m3fn
    scales: torch.Tensor   # [..., ceil(H / 32)] float8_e8m0fnu


@dataclasses.dataclass
class Mx4Weight:
    """A projection [V, hidden] in 4 bits, rows padded with zeros to Kp, a
    multiple of 128: two elements a byte, the first in the low half; element k
    of a row has the scale scales[v, k // 32]."""
    data: torch.Tensor     # [V, Kp / 2] uint8
    scales: torch.Tensor   # [V, Kp / 32] float8_e8m0fnu
    hidden: int


def _padded(H: int) -> int:
    return (H + MX_STEP - 1) // MX_STEP * MX_STEP


def mx4_pack(W: torch.Tensor) -> Mx4Weight:
    """``W`` [V, H] (bfloat16 or float32) in 4 bits (``flce_pack_mx``): each
    block's scale is the least power of two that holds it, its elements are
    rounded to nearest."""
    if W.dtype not in _DTYPES:
        raise TypeError(f"W must be bfloat16 or float32 (got {W.dtype})")
    if not W.is_cuda:
        raise ValueError("W must be on the GPU")
    if W.dim() != 2 or W.shape[1] < 1:
        raise ValueError(f"W must be [V, H] (got {tuple(W.shape)})")
    if W.stride(1) != 1:
        W = W.contiguous()
    V, H = W.shape
    kp = _padded(H)
    out = Mx4Weight(torch.empty((V, kp // 2), dtype=torch.uint8, device=W.device),
                    torch.empty((V, kp // MX_BLOCK), dtype=torch.float8_e8m0fnu, device=W.device), H)
    rc = _enqueue(W.device, lambda stream: _lib.flce_pack_mx(
        W.data_ptr(), W.stride(0), V, H, out.data.data_ptr(), out.scales.data_ptr(), stream, _DTYPES[W.dtype]))
    if rc != _lib.FLCE_OK:
        raise _lib.FlceError(rc, "flce_pack_mx")
    return out


def _check_weight(w: Mx4Weight) -> None:
    kp = _padded(w.hidden)
    for name, t, dtype, cols in (("data", w.data, torch.uint8, kp // 2),
                                 ("scales", w.scales, torch.float8_e8m0fnu, kp // MX_BLOCK)):
        if t.dtype != dtype or t.dim() != 2 or t.shape[1] != cols or t.shape[0] != w.data.shape[0] \
                or not t.is_contiguous():
            raise ValueError(f"weight.{name} must be a contiguous [V, {cols}] {dtype} tensor (got {tuple(t.shape)} "
                             f"{t.dtype})")
    if w.data.device != w.scales.device:
        raise ValueError(f"weight.data is on {w.data.device}, weight.scales on {w.scales.device}")


def logits_mx4(x: Union[torch.Tensor, Mx8Rows], weight: Mx4Weight, softcap: Optional[float] = None,
               multiplier: float = 1.0, out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Materialised logits z = cap(m x W^T) from a projection in 4 bits
    (``flce_logits_mx``), [..., V]; ``x`` [..., H] is bfloat16 or float32 (so
    are the logits), or rows in 8 bits (bfloat16 logits).  ``out``, when given,
    is [N, ld >= V] with unit column stride, bfloat16 or float32; float32 logits
    of bfloat16 rows are as exact, and take as long, as those of float32 rows.  As with
    ``logits`` the returned rows may have a stride padded to 16 bytes.  A
    caller-owned ``workspace`` (uint8, ``flce_logits_mx_workspace_size``) may be
    reused by ordered calls."""
    mx8 = isinstance(x, Mx8Rows)
    data = x.data if mx8 else x
    if mx8:
        if data.dtype != torch.float8_e4m3fn or x.scales.dtype != torch.float8_e8m0fnu:
            raise TypeError(f"rows in 8 bits are float8_e4m3fn with float8_e8m0fnu scales (got {data.dtype}, "
                            f"{x.scales.dtype})")
    elif data.dtype not in _DTYPES:
        raise TypeError(f"x must be bfloat16, float32 or Mx8Rows (got {data.dtype})")
    if not data.is_cuda:
        raise ValueError("x must be on the GPU")
    _check_weight(weight)
    H, V = weight.hidden, weight.data.shape[0]
    if data.dim() < 1 or data.shape[-1] != H:
        raise ValueError(f"x must be [..., {H}] (got {tuple(data.shape)})")
    dev = data.device
    if weight.data.device != dev:
        raise ValueError(f"the weight is on {weight.data.device}, x is on {dev}")
    x2 = data.reshape(-1, H)
    if x2.stride(1) != 1 and H > 1:
        x2 = x2.contiguous()
    N = x2.shape[0]
    s2 = None
    if mx8:
        nb = (H + MX_BLOCK - 1) // MX_BLOCK
        if x.scales.shape != (*data.shape[:-1], nb) or x.scales.device != dev:
            raise ValueError(f"x.scales must be {(*data.shape[:-1], nb)} on {dev} (got {tuple(x.scales.shape)} on "
                             f"{x.scales.device})")
        s2 = x.scales.reshape(N, nb)
        if s2.stride(1) != 1 and nb > 1:
            s2 = s2.contiguous()
    if out is None:
        dtype = torch.bfloat16 if mx8 else data.dtype
        per = 16 // dtype.itemsize
        out = torch.empty((N, (V + per - 1) // per * per), dtype=dtype, device=dev)
    if out.dim() != 2 or out.shape[0] != N or out.shape[1] < V or out.stride(1) != 1 or out.stride(0) < V:
        raise ValueError("out must be [N, ld >= V] with unit column stride")
    if out.dtype not in _DTYPES or out.device != dev:
        raise ValueError(f"out is {out.dtype} on {out.device}, must be bfloat16 or float32 on {dev}")
    x_dtype = _lib.FLCE_DTYPE_MX8 if mx8 else _DTYPES[data.dtype]
    ws_bytes = _lib.flce_logits_mx_workspace_size(N, H, x_dtype)
    if ws_bytes == 0:
        raise _lib.FlceError(_lib.FLCE_EUNSUPPORTED, "flce_logits_mx_workspace_size")
    workspace = _workspace(workspace, ws_bytes, dev)
    rc = _enqueue(dev, lambda stream: _lib.flce_logits_mx(
        x2.data_ptr(), x2.stride(0), _ptr(s2), s2.stride(0) if mx8 else 0, weight.data.data_ptr(),
        weight.scales.data_ptr(), N, H, V, float(softcap) if softcap else 0.0, float(multiplier), out.data_ptr(),
        out.stride(0), stream, x_dtype, _DTYPES[out.dtype], workspace.data_ptr(), workspace.numel()))
    if rc != _lib.FLCE_OK:
        raise _lib.FlceError(rc, "flce_logits_mx")
    return out[:, :V].reshape(*data.shape[:-1], V)
