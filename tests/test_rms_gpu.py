"""GPU parity of RMS norm against the fp64 definitions (``oracle/head.py``) on
exactly the values the GPU reads.

Tolerances, with u = 2^-24 (fp32 rounding) and e = eps/2 of the storage dtype:

* the residual's sum is exact before its one rounding for bf16 (8-bit
  significands whose sum needs more than 24 bits round to the larger term), and
  one fp32 addition otherwise: it has to be equal;
* a row's sum of squares adds at most 32 values in a thread and 6 + 16 more in
  joining, all positive: relative error 54 u, halved by the root; with the
  mean, the root and the reciprocal rstd is off by at most 32 u, and y by 36 u
  + e with the weight's offset and two products.  A wide row adds H / 4096
  sequential vectors of 4 per thread: counted by `wide`;
* the gradients take rstd as an input: xh is off by u, the row's sum of g xh by
  60 u times the sum of magnitudes, and the sums over M rows by (M + 8) u times
  theirs whatever their order;
* 8 bits: the scale fits the block's maximum within 40 u, and every element is
  the nearest value within 40 u of y.
"""
import numpy as np
import pytest

from gpu_util import log
from oracle import head as O

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("require_gpu")]

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}
EPS = 1e-6


def _dt(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _rand(shape, dtype, seed, scale=1.0, shift=0.0, pad=0, off=0):
    """A seeded tensor; its rows lie `pad` elements apart in a buffer that
    starts `off` elements past an aligned address."""
    import torch
    g = torch.Generator().manual_seed(seed)
    v = (torch.randn(shape, generator=g) * scale + shift).to(_dt(dtype))
    M, H = shape
    buf = torch.zeros(M * (H + pad) + off + 8, dtype=_dt(dtype), device="cuda")
    out = buf[off:off + M * (H + pad)].view(M, H + pad)[:, :H]
    out.copy_(v)
    return out


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _wide(H, dtype):
    return 4.0 * H / 4096 if H > (16384 if dtype == "bf16" else 8192) else 0.0


def _check(name, got, ref, tol):
    bad = np.abs(_np(got) - ref) - tol
    i = int(np.argmax(bad)) if bad.size else 0
    log(f"  {name}: worst error minus bound {bad.max() if bad.size else 0:.2e}")
    assert bad.size == 0 or bad.max() <= 0.0, (name, np.unravel_index(i, bad.shape))


def _sum(x, r):
    """x + r rounded once, as the stream keeps it."""
    import torch
    return (x.float() + r.float()).to(x.dtype) if r is not None else x


# one column, one vector and its neighbours, the borders between the kernels'
# widths (512, 1024, 2048, 4096, 8192, 16384 in bf16, half of that in fp32),
# rows kept out of registers, few and many rows
SHAPES = [(1, 1), (5, 3), (3, 8), (130, 37), (1, 511), (1030, 512), (9, 513), (4101, 600), (7, 1024), (64, 1025),
          (5, 2047), (700, 2049), (3, 4096), (2, 4099), (1, 6656), (300, 6656), (530, 8192), (2, 8193), (5, 16383),
          (3, 16385), (67, 20001)]


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("M,H", SHAPES)
def test_rms_norm(M, H, dtype, wdtype):
    import torch
    import linear_cross_entropy_gemm_amd as L
    log(f"[rms] M={M} H={H} {dtype}/{wdtype}")
    x = _rand((M, H), dtype, 1, 1.5, 0.3, pad=H % 3, off=1)
    r = _rand((M, H), dtype, 4, 2.0, pad=H % 2, off=3) if H % 2 else None
    dy = _rand((M, H), dtype, 2, 1.0, 0.1, pad=(H + 1) % 2, off=3)
    ds = _rand((M, H), dtype, 5, 0.7, pad=1) if H % 4 else None
    offset = float(M % 2)
    w = _rand((1, H), wdtype, 3, 0.3, 1.0 - offset, off=1)[0]
    o = L.rms_norm_fwd(x, w, EPS, residual=r, offset=offset)
    s = _sum(x, r)
    assert (o.residual is None) == (r is None) and (r is None or torch.equal(o.residual, s))
    sn, wn = _np(s), _np(w)
    y, rstd = O.rms_norm(sn, wn, offset, EPS)
    k = 36 + _wide(H, dtype)
    _check("y", o.y, y, HALF[dtype] * np.abs(y) + k * U * np.abs(y))
    _check("rstd", o.rstd, rstd, k * U * rstd)
    g = L.rms_norm_bwd(dy, s, w, o.rstd, offset=offset, grad_residual=ds)
    dn, an, rs = _np(dy), None if ds is None else _np(ds), _np(o.rstd)
    dx, dw = O.rms_norm_grads(dn, sn, wn, offset, rs, an)
    xh, gg = sn * rs[:, None], dn * (wn + offset)
    mean = np.abs(gg * xh).mean(1, keepdims=True)
    tol = rs[:, None] * (6 * np.abs(gg) + (66 + _wide(H, dtype)) * np.abs(xh) * mean) * U
    tol += HALF[dtype] * np.abs(dx) + 2 * U * (np.abs(dx) + (0 if an is None else np.abs(an)))
    _check("grad_x", g.grad_x, dx, tol)
    tol = (M + 8) * U * np.abs(dn * xh).sum(0) + HALF[wdtype] * np.abs(dw)
    _check("grad_weight", g.grad_weight, dw, tol)
    # either output alone is the same
    assert torch.equal(L.rms_norm_bwd(dy, s, w, o.rstd, offset=offset, grad_residual=ds, need_weight=False).grad_x,
                       g.grad_x)
    assert torch.equal(L.rms_norm_bwd(dy, s, w, o.rstd, offset=offset, need_x=False).grad_weight, g.grad_weight)


def _check_mx8(rows, y):
    """Every block's scale and elements against y (fp64)."""
    M, H = y.shape
    nb = (H + 31) // 32
    code = rows.scales.view(__import__("torch").uint8).cpu().numpy().reshape(M, nb).astype(np.float64)
    q = rows.data.double().cpu().numpy().reshape(M, H)
    full = np.zeros((M, nb * 32))
    full[:, :H] = np.abs(y)
    amax = full.reshape(M, nb, 32).max(2)
    scale = 2.0 ** (code - 127)
    assert np.all(amax * (1 - 40 * U) <= 448 * scale)
    assert np.all((code == 0) | (amax * (1 + 40 * U) > 224 * scale))
    sc = np.repeat(scale, 32, 1)[:, :H]
    v = np.abs(y) / sc
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(v, 1e-30))), -6) - 3)
    assert np.all(np.abs(q * sc - y) <= sc * (step / 2 * (1 + 1e-12) + 40 * U * v))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,H", [(1, 1), (5, 31), (3, 32), (130, 37), (9, 513), (64, 1025), (700, 2049), (1, 6656),
                                 (300, 6656), (2, 8193), (3, 16385), (9, 20001)])
def test_rms_norm_mx8(M, H, dtype):
    import torch
    import linear_cross_entropy_gemm_amd as L
    log(f"[rms mx8] M={M} H={H} {dtype}")
    x = _rand((M, H), dtype, 1, 1.5, pad=H % 3, off=1) * (10.0 ** torch.linspace(-6, 6, M, device="cuda"))[:, None]
    x = x.to(_dt(dtype))
    x[:, ::77] *= 40
    r = _rand((M, H), dtype, 4, 1e-3, pad=1) if H % 2 else None
    w = _rand((1, H), "f32", 3, 2.0)[0]
    w[: H // 3] *= 1e-3
    o = L.rms_norm_mx8(x, w, EPS, residual=r)
    s = _sum(x, r)
    assert (o.residual is None) == (r is None) and (r is None or torch.equal(o.residual, s))
    assert o.rows.data.shape == (M, H) and o.rows.scales.shape == (M, (H + 31) // 32)
    _check_mx8(o.rows, O.rms_norm(_np(s), _np(w), 0.0, EPS)[0])


def test_mx8_special_blocks():
    """Zeros, tiny values, and what is not finite: its block alone is NaN."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    x = torch.ones(4, 100, device="cuda")
    w = torch.ones(100, device="cuda")
    w[40] = float("inf")
    w[64:96] = 0.0
    w[96:] = 1e-42
    o = L.rms_norm_mx8(x, w, EPS).rows
    code = o.scales.view(torch.uint8).cpu()
    assert code[:, 1].eq(255).all() and code[:, 2].eq(0).all() and code[:, 3].eq(0).all()
    q = o.data.float().cpu()
    assert q[:, 32:64].isnan().all() and q[:, 64:96].eq(0).all() and not q[:, :32].isnan().any()
    y = x.cpu().double()[0, 96] * 1e-42
    assert abs(q[0, 96].item() * 2.0 ** -127 - y.item()) <= 2.0 ** -127 * 2.0 ** -10 * 1.001
    x[2, 7] = float("nan")
    o = L.rms_norm_mx8(x, None, EPS).rows
    assert o.scales.view(torch.uint8)[2].eq(255).all() and o.data[2].float().isnan().all()
    assert not o.data[[0, 1, 3]].float().isnan().any()


def test_far_and_special_rows():
    import torch
    import linear_cross_entropy_gemm_amd as L
    for H in (100, 6656, 20001):
        x = torch.zeros(6, H, device="cuda")
        x[1] = 1e-20                   # far below eps
        x[2] = 1e17
        x[3, H // 2] = float("nan")
        x[4] = 3e30                    # its squares overflow
        x[5] = -2.0
        o = L.rms_norm_fwd(x, None, EPS)
        y, rstd = O.rms_norm(_np(x), None, 0.0, EPS)
        for i in (0, 1, 2, 5):
            _check(f"row {i}", o.y[i], y[i], 40 * U * np.abs(y[i]))
            assert abs(o.rstd[i].item() - rstd[i]) <= (40 + _wide(H, "f32")) * U * rstd[i]
        assert o.y[3].isnan().all() and o.rstd[4].item() == 0.0 and o.y[4].eq(0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [77, 6656, 20000])
def test_in_place_and_canaries(H, dtype):
    """The residual stream updated in place, y in the place of x, and not a
    byte behind the rows touched."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    M, ld, dt = 37, H + 5, _dt(dtype)
    x, r = _rand((M, ld), dtype, 1), _rand((M, ld), dtype, 2)
    x0, r0 = x.clone(), r.clone()
    w = _rand((1, H), dtype, 3, 0.2, 1.0)[0]
    ref = L.rms_norm_fwd(x0[:, :H], w, EPS, residual=r0[:, :H])
    st = torch.cuda.current_stream().cuda_stream
    d = L.FLCE_DTYPE_BF16 if dtype == "bf16" else L.FLCE_DTYPE_F32
    assert L.flce_rms_norm_fwd(x.data_ptr(), ld, r.data_ptr(), ld, w.data_ptr(), 0.0, M, H, EPS, x.data_ptr(), ld,
                               r.data_ptr(), ld, None, st, d, d) == L.FLCE_OK
    assert torch.equal(x[:, :H], ref.y) and torch.equal(r[:, :H], ref.residual)
    assert torch.equal(x[:, H:], x0[:, H:]) and torch.equal(r[:, H:], r0[:, H:])
    # 8 bits: canaries between the rows and behind them
    nb = (H + 31) // 32
    y8 = torch.full((M + 1, H + 3), 99, dtype=torch.uint8, device="cuda")
    sc = torch.full((M + 1, nb + 2), 99, dtype=torch.uint8, device="cuda")
    assert L.flce_rms_norm_mx(x0.data_ptr(), ld, None, 0, w.data_ptr(), 0.0, M, H, EPS, y8.data_ptr(), H + 3,
                              sc.data_ptr(), nb + 2, None, 0, None, st, d, d) == L.FLCE_OK
    rows = L.rms_norm_mx8(x0[:, :H], w, EPS).rows
    assert torch.equal(y8[:M, :H], rows.data.view(torch.uint8)) and y8[:, H:].eq(99).all() and y8[M].eq(99).all()
    assert torch.equal(sc[:M, :nb], rows.scales.view(torch.uint8)) and sc[:, nb:].eq(99).all() and sc[M].eq(99).all()
    assert dt == x.dtype


def test_layouts_and_empty():
    import torch
    import linear_cross_entropy_gemm_amd as L
    x = _rand((6, 64), "bf16", 1)
    w = _rand((1, 64), "f32", 2, 0.2, 1.0)[0]
    ref = L.rms_norm_fwd(x.contiguous(), w, EPS, residual=x.contiguous())
    o = L.rms_norm_fwd(x.view(2, 3, 64), w, EPS, residual=x.view(2, 3, 64))
    assert o.y.shape == (2, 3, 64) and o.rstd.shape == (2, 3) and torch.equal(o.y.view(6, 64), ref.y)
    t = x.t().contiguous().t()   # columns are not adjacent: copied
    assert torch.equal(L.rms_norm_fwd(t, w, EPS).y, L.rms_norm_fwd(x, w, EPS).y)
    b = x[:1].expand(5, 64)      # one row, read five times
    assert torch.equal(L.rms_norm_fwd(b, w, EPS).y, L.rms_norm_fwd(x[:1], w, EPS).y.expand(5, 64))
    e = L.rms_norm_fwd(x[:0], w, EPS, residual=x[:0])
    assert e.y.shape == (0, 64) and e.residual.shape == (0, 64) and e.rstd.shape == (0,)
    g = L.rms_norm_bwd(x[:0], x[:0], w, e.rstd)
    assert g.grad_x.shape == (0, 64) and g.grad_weight.eq(0).all()
    assert L.rms_norm_mx8(x[:0], w, EPS).rows.data.shape == (0, 64)
    for bad in (dict(residual=x[:3]), dict(residual=x.float())):
        with pytest.raises(ValueError, match="residual"):
            L.rms_norm_fwd(x, w, EPS, **bad)
    with pytest.raises(ValueError, match="weight"):
        L.rms_norm_fwd(x, w[:5], EPS)
    with pytest.raises(ValueError, match="grad_y"):
        L.rms_norm_bwd(x[:2], x, w, ref.rstd)
    with pytest.raises(ValueError, match="rstd"):
        L.rms_norm_bwd(x, x, w, ref.rstd[:2])
    with pytest.raises(ValueError, match="workspace"):
        L.rms_norm_bwd(x, x, w, ref.rstd, torch.empty(8, dtype=torch.uint8, device="cuda"))


def test_rows_far_apart():
    """Rows more than 2^31 elements from the first."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    ld = (1 << 30) + 12345
    buf = torch.zeros(2 * ld + 64, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((3, 64), (ld, 1))
    v = _rand((3, 64), "bf16", 1)
    x.copy_(v)
    assert torch.equal(L.rms_norm_fwd(x, None, EPS).y, L.rms_norm_fwd(v, None, EPS).y)


@pytest.mark.parametrize("H,dtype", [(600, "bf16"), (5003, "f32"), (6656, "bf16"), (7173, "bf16"), (16384, "bf16")])
def test_many_rows_as_few(H, dtype):
    """Calls that move more than the caches hold, with many rows for each
    work-group: every row comes out as from a call of 100 rows, bit for bit, and
    the weight's gradient within its bound."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    M = max(2100, (300 << 20) // (H * 8))
    g = torch.Generator(device="cuda").manual_seed(H)
    x, r, dy, ds = (torch.randn(M * H + 1, device="cuda", generator=g).to(_dt(dtype))[1:].view(M, H) for _ in range(4))
    w = torch.randn(H, device="cuda", generator=g).to(_dt(dtype))
    o = L.rms_norm_fwd(x, w, EPS, residual=r, offset=1.0)
    m = L.rms_norm_mx8(x, w, EPS, residual=r, offset=1.0)
    b = L.rms_norm_bwd(dy, o.residual, w, o.rstd, offset=1.0, grad_residual=ds)
    for i in list(range(0, M, max(100, M // 23 // 100 * 100))) + [M - 100]:
        c = slice(i, min(i + 100, M))
        few = L.rms_norm_fwd(x[c], w, EPS, residual=r[c], offset=1.0)
        assert few.y.equal(o.y[c]) and few.residual.equal(o.residual[c]) and few.rstd.equal(o.rstd[c])
        fm = L.rms_norm_mx8(x[c], w, EPS, residual=r[c], offset=1.0)
        assert fm.rows.data.view(torch.uint8).equal(m.rows.data[c].view(torch.uint8))
        assert fm.rows.scales.view(torch.uint8).equal(m.rows.scales[c].view(torch.uint8))
        assert fm.residual.equal(m.residual[c])
        fb = L.rms_norm_bwd(dy[c], o.residual[c], w, o.rstd[c], offset=1.0, grad_residual=ds[c])
        assert fb.grad_x.equal(b.grad_x[c])
    dw, mag = torch.zeros(H, dtype=torch.float64, device="cuda"), torch.zeros(H, dtype=torch.float64, device="cuda")
    for i in range(0, M, 1000):
        t = dy[i:i + 1000].double() * (o.residual[i:i + 1000].double() * o.rstd[i:i + 1000, None].double())
        dw += t.sum(0)
        mag += t.abs().sum(0)
    tol = (M + 9) * U * mag
    assert ((b.grad_weight.double() - dw).abs() <= tol + HALF[dtype] * (dw.abs() + tol)).all()


@pytest.mark.parametrize("residual", [False, True])
def test_autograd(residual):
    """Gradients through both outputs, against the formula's."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    M, H = 70, 513
    x, r, w = _rand((M, H), "f32", 1), _rand((M, H), "f32", 2), _rand((1, H), "f32", 3, 0.3)[0]
    dy, ds = _rand((M, H), "f32", 4), _rand((M, H), "f32", 5)
    leaves = [t.clone().requires_grad_() for t in ((x, r, w) if residual else (x, w))]
    if residual:
        y, s = L.rms_norm(leaves[0], leaves[2], EPS, residual=leaves[1], offset=1.0)
        torch.autograd.backward((y, s), (dy, ds))
    else:
        s = leaves[0]
        L.rms_norm(s, leaves[1], EPS, offset=1.0).backward(dy)
    sn, wn, dn = _np(s), _np(w), _np(dy)
    rstd = O.rms_norm(sn, wn, 1.0, EPS)[1]
    dx, dw = O.rms_norm_grads(dn, sn, wn, 1.0, rstd, _np(ds) if residual else None)
    xh = sn * rstd[:, None]
    big = 1 + rstd[:, None] * (np.abs(dn * (wn + 1)) + np.abs(xh) * np.abs(dn * (wn + 1) * xh).mean(1, keepdims=True))
    for t in leaves[:-1]:
        _check("grad", t.grad, dx, 140 * U * big)   # with rstd's own 32 u twice
    _check("grad_w", leaves[-1].grad, dw, (M + 48) * U * np.abs(dn * xh).sum(0))
    if residual:
        assert leaves[0].grad.data_ptr() != leaves[1].grad.data_ptr()
        # the stream's gradient alone, and y's alone
        y, s = L.rms_norm(leaves[0], leaves[2], EPS, residual=leaves[1], offset=1.0)
        g = torch.autograd.grad(s, leaves[:2], ds, retain_graph=True)
        assert torch.equal(g[0], ds) and torch.equal(g[1], ds)
        g = torch.autograd.grad(y, leaves[0], dy)[0]
        _check("grad", g, dx - _np(ds), 140 * U * big)
    # forward without gradients is the same
    with torch.no_grad():
        out = L.rms_norm(x, w, EPS, residual=r if residual else None, offset=1.0)
        assert torch.equal(out[0] if residual else out, y if residual else L.rms_norm_fwd(x, w, EPS, offset=1.0).y)


def test_gradient_against_differences():
    """The kernels' gradient against differences of the kernels' forward (fp32,
    step 2^-6: truncation below 1e-4 of the gradient's scale, rounding 2^6 32 u)."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    x, w, dy = _rand((4, 40), "f32", 1), _rand((1, 40), "f32", 2, 0.3, 1.0)[0], _rand((4, 40), "f32", 3)
    leaf = x.clone().requires_grad_()
    L.rms_norm(leaf, w, EPS).backward(dy)
    d, h = _rand((4, 40), "f32", 4), 2.0 ** -6
    up, down = (L.rms_norm(x + k * h * d, w, EPS).double() for k in (1, -1))
    diff = ((up - down) * dy.double()).sum() / (2 * h)
    size = (dy.abs() * w.abs()).sum().item()
    assert abs(diff.item() - (leaf.grad.double() * d.double()).sum().item()) <= 2e-3 * size


def test_captured_step_replays():
    import torch
    import linear_cross_entropy_gemm_amd as L
    x, r, w = _rand((33, 1000), "bf16", 1), _rand((33, 1000), "bf16", 2), _rand((1, 1000), "f32", 3)[0]
    dy = _rand((33, 1000), "bf16", 4)

    def step():
        o = L.rms_norm_fwd(x, w, EPS, residual=r)
        g = L.rms_norm_bwd(dy, o.residual, w, o.rstd, grad_residual=dy)
        q = L.rms_norm_mx8(x, w, EPS, residual=r)
        return o.y, o.residual, g.grad_x, g.grad_weight, q.rows.data.view(torch.uint8), q.rows.scales.view(torch.uint8)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        x.copy_(_rand((33, 1000), "bf16", 10 + k))
        ref = [t.clone() for t in step()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, ref):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dropout", [0.0, 0.2])
def test_head_loss_with_rms_norm(dropout):
    """The training head's path against its operators one by one."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    N, H, V = 60, 96, 300
    x, r = _rand((N, H), "bf16", 1), _rand((N, H), "bf16", 2)
    W, w = _rand((V, H), "bf16", 3, 0.1), _rand((1, H), "f32", 4, 0.2)[0]
    lab = torch.arange(N, device="cuda") * 5
    a = [t.clone().requires_grad_() for t in (x, r, W, w)]
    loss, n = L.lm_head_loss(a[0], a[2], lab, a[3], residual=a[1], dropout_p=dropout, seed=3, norm="rms",
                             norm_offset=1.0, eps=EPS)
    loss.backward()
    b = [t.clone().requires_grad_() for t in (x, r, W, w)]
    if dropout:
        y = L.rms_norm(L.dropout(b[0], dropout, 3, 0, b[1]), b[3], EPS, offset=1.0)
    else:
        y, _ = L.rms_norm(b[0], b[3], EPS, residual=b[1], offset=1.0)
    ref, m = L.linear_cross_entropy(y, b[2], lab)
    ref.backward()
    assert torch.equal(loss, ref) and torch.equal(n, m)
    for s, t in zip(a, b):
        assert torch.equal(s.grad, t.grad)
