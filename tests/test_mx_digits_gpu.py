"""fp32 logits from 4-bit weights: rows in bf16 or fp32 enter as digits, whose
products the matrix unit adds exactly, so neither loses what an fp32 sum keeps.

The bound: with U = 2^-24, block maxima bx and block sums bw of |w|, S = sum |x
w| and s = Kp / 128 steps,
  * the five digits hold an element to U of its block's largest: U bx bw;
  * an instruction cuts 17 addends (16 sums of 8, exact, and the accumulator)
    below 2 U of the largest: 34 U of what the step has summed by then, at most
    S + bx bw / 16 with the first digits (half a unit each, 8 to 16 of which are
    the largest) and 2 bx bw (2^-5 + 2^-10 + ...) with those below;
  * each step's sum is added with one rounding: U s S.
Together below U (8 bx bw + (34 + s) S); the output's own half step (the
multiplier, the cap's tanh at 1e-6) comes on top.
"""
import numpy as np
import pytest

from gpu_util import log
from test_mx_gpu import U, _groups, _np, _rand, _weights

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("require_gpu")]


def _bound(x, w):
    s = (w.shape[1] + 127) // 128
    bx, bw = np.abs(_groups(x, 32)).max(2), np.abs(_groups(w, 32)).sum(2)
    return U * (8 * bx @ bw.T + (34 + s) * (np.abs(x) @ np.abs(w).T))


# across the kernels' borders: rows in LDS split by the work-groups (1, 2), brought
# to parts by a launch, and tiles of 16, 32 and 48 tokens
@pytest.mark.parametrize("N,H,V", [(1, 100, 129), (1, 8192, 500), (2, 4096, 1003), (2, 20001, 70), (3, 4096, 500),
                                   (16, 1001, 300), (17, 2049, 400), (33, 1001, 2001), (48, 130, 77), (100, 4096, 300)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_fp32_logits(N, H, V, kind):
    import torch
    import linear_cross_entropy_gemm_amd as L
    log(f"[mx4] N={N} H={H} V={V} {kind}")
    q = L.mx4_pack(_rand((V, H), "f32", 21, 0.05))
    w, x = _weights(q), _rand((N, H), kind, 22, pad=H % 3, off=1)
    x[:, 3::101] *= 300.0   # a few channels far above the rest
    for cap, mult in ((0.0, 1.0), (30.0, 0.5)):
        z = _np(L.logits_mx4(x, q, cap, mult, out=torch.empty(N, V, device="cuda")))
        ref, tol = _np(x) @ w.T * mult, _bound(_np(x), w) * mult
        if cap:
            ref = cap * np.tanh(ref / cap)
            tol = tol + 1e-6 * np.abs(ref)
        bad = np.abs(z - ref) - tol - 3 * U * np.abs(ref)
        log(f"  worst error minus bound {bad.max():.2e}, relative {np.linalg.norm(z - ref) / np.linalg.norm(ref):.1e}")
        assert bad.max() <= 0.0


@pytest.mark.parametrize("N,H,V", [(1, 6656, 4099), (2, 129, 300), (2, 16000, 70), (5, 4096, 500), (16, 640, 257),
                                   (20, 2049, 400), (40, 1001, 3001), (300, 512, 200)])
def test_bf16_rows_count_as_the_same_fp32_rows(N, H, V):
    """Bit for bit: the digits are those of the same values."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    q = L.mx4_pack(_rand((V, H), "f32", 23, 0.05))
    x = _rand((N, H), "bf16", 24)
    x[:, 5::97] *= 1000.0
    x[0, :40] = 0.0
    z = L.logits_mx4(x, q, 30.0, 0.5, out=torch.empty(N, V, device="cuda"))
    assert torch.equal(z, L.logits_mx4(x.float(), q, 30.0, 0.5))
    x[N - 1, H // 2] = float("nan")   # (and a block that is not finite)
    z = L.logits_mx4(x, q, out=torch.empty(N, V, device="cuda"))
    assert z[N - 1].isnan().all() and not z[:N - 1].isnan().any()


@pytest.mark.parametrize("N,H,V", [(33, 130, 32768), (33, 130, 32769), (48, 1001, 40001), (40, 257, 65537), (48, 64, 80001),
                                   (35, 129, 104003)])
def test_tokens_by_48_and_by_32(N, H, V):
    """Which tiles take 33 to 48 rows goes by how many rounds of work-groups they
    make; a row's logits do not depend on it."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    q = L.mx4_pack(_rand((V, H), "f32", 25, 0.05))
    x = _rand((N, H), "f32", 26)
    z = L.logits_mx4(x, q)
    assert torch.equal(z, torch.cat([L.logits_mx4(x[i:i + 24], q) for i in range(0, N, 24)]))
    some = slice(V - 300, V)
    w = _weights(L.Mx4Weight(q.data[some].contiguous(), q.scales[some].contiguous(), H))
    ref = _np(x) @ w.T
    assert (np.abs(_np(z)[:, some] - ref) <= _bound(_np(x), w) + 2 * U * np.abs(ref)).all()
