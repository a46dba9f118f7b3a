"""Layer norm of rows far from zero, or with values far apart, on every kernel
shape, against the fp64 definition (``oracle/head.py``).

Tolerance of a row with standard deviation 1 around `shift`, u = 2^-24: a mean
is first rounded in a sum of at most 54 + `wide` additions of terms that add up
to `shift`, so it is off by at most d = (54 + wide) u shift.  Deviations from it
are exact (both numbers lie within a factor of two), at most |xh| + d in size,
and so are their sums' errors the ordinary ones times at most (1 + d)^2 (the
squares).  What is left of the mean is added back in its own fp32 number.
"""
import numpy as np
import pytest

from gpu_util import log
from oracle import head as O
from test_head_gpu import EPS, U, _check, _np, _rand, _wide

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("require_gpu")]


@pytest.mark.parametrize("shift", [1e3, -1e4, 1e5])
@pytest.mark.parametrize("M,H", [(6, 200), (6, 500), (6, 1000), (6, 1025), (1600, 2000), (6, 2049), (900, 4000),
                                 (6, 4097), (6, 5003), (300, 6145), (6, 8000), (6, 8192), (6, 8193), (3, 20001)])
def test_layer_norm_far_from_zero(M, H, shift):
    import linear_cross_entropy_gemm_amd as L
    log(f"[ln] far rows M={M} H={H} shift={shift}")
    x = _rand((M, H), "f32", 100 + H, 1.0, shift, pad=H % 3, off=1)
    b = _rand((1, H), "f32", 101)[0].clone()
    o = L.layer_norm_fwd(x, None, b, EPS)
    X = _np(x)
    y, mean, rstd = O.layer_norm(X, None, _np(b), EPS)
    xh = np.abs((X - mean[:, None]) * rstd[:, None])
    k = _wide(H, "f32")
    grow = (1 + (54 + k) * U * abs(shift) * rstd.max()) ** 2
    _check("y", o.y, y, grow * U * (60 + k + (44 + k) * xh) + 4 * U * np.abs(y))
    _check("mean", o.mean, mean, U * (np.abs(mean) + grow * (60 + k) / rstd))
    _check("rstd", o.rstd, rstd, grow * U * (40 + k) * rstd)


@pytest.mark.parametrize("H", [5, 700, 2000, 5003, 8192, 20001])
@pytest.mark.parametrize("c", [1e21, 1e35, 1e37, 1.6e38])
def test_layer_norm_of_values_far_apart(H, c):
    """Squares of the deviations overflow (1e21^2 does), the mean does not:
    rstd is 0 and y is the bias, however the two signs lie in the row.  The
    mean's sums round at most 54 + 20 times a number of at most c: 2^-17 c."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    x = torch.full((4, H), c, device="cuda")
    x[0, :H // 2] = -c
    x[1, ::2] = -c
    x[2, 1:] = -c
    x[3] *= torch.rand(H, generator=torch.Generator().manual_seed(H)).cuda() * 2 - 1
    b = _rand((1, H), "f32", 102)[0].clone()
    o = L.layer_norm_fwd(x, None, b, EPS)
    log(f"[ln] values far apart H={H} c={c}")
    ref = _np(x).mean(1)
    assert np.all(np.abs(_np(o.mean) - ref) <= 2.0 ** -17 * c)
    assert not o.rstd.any() and torch.equal(o.y, b.expand(4, H))
