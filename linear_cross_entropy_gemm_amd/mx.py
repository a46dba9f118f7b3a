"""Block formats of the OCP Microscaling specification on torch tensors: rows
in 8 bits (MXFP8, E4M3).  32 elements along a row share a scale, a power of
two held as an E8M0 exponent."""
from __future__ import annotations

import dataclasses

import torch

MX_BLOCK = 32


@dataclasses.dataclass
class Mx8Rows:
    """Rows in 8 bits: element h of a row stands for data[..., h] *
    scales[..., h // 32]."""
    data: torch.Tensor     # [..., H] float8_e4m3fn
    scales: torch.Tensor   # [..., ceil(H / 32)] float8_e8m0fnu
