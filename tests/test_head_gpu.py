"""GPU parity of layer norm and dropout against the fp64 definitions
(``oracle/head.py``) on exactly the values the GPU reads.

Tolerances, with u = 2^-24 (fp32 rounding) and e = eps/2 of the storage dtype:

* layer norm: a thread sums at most 32 values in sequence and the row's
  threads join in at most 6 + 16 more additions, so a row sum is off by at
  most 54 u times the sum of magnitudes.  With sd = 1/rstd the mean's and the
  deviations' errors stay below 60 u sd, rstd's below 40 u relative, hence
  |dy| <= e |y| + u (|w| (60 + 44 |xh|) + 4 |y|).  A wide row adds
  H / 4096 sequential vectors of 4 per thread: counted by `wide`.
* its gradients take mean and rstd as inputs, so xh is off by 2 u |xh|; the
  row sums as above; sums over rows by at most (M + 4) u times the sum of
  magnitudes, whatever their order.
* dropout: the mask is exact; a kept value has the scale's rounding, the
  product's (or the fused multiply-add's) and the store's.
"""
import numpy as np
import pytest

from gpu_util import log
from oracle import head as O

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("require_gpu")]

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}
EPS = 1e-5


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


# one column, one vector and its neighbours, the borders between the kernels'
# widths (512, 1024, 2048, 4096, 8192, 16384 in bf16, half of that in fp32),
# rows kept out of registers, few and many rows
SHAPES = [(1, 1), (5, 3), (3, 8), (130, 37), (1, 511), (1030, 512), (9, 513), (4101, 600), (7, 1024), (64, 1025),
          (5, 2047), (700, 2049), (3, 4096), (2, 4099), (1, 6656), (300, 6656), (530, 8192), (2, 8193), (5, 16383),
          (3, 16385), (67, 20001)]


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("M,H", SHAPES)
def test_layer_norm(M, H, dtype, wdtype):
    import torch
    import linear_cross_entropy_gemm_amd as L
    log(f"[ln] M={M} H={H} {dtype}/{wdtype}")
    x = _rand((M, H), dtype, 1, 1.5, 0.7, pad=H % 3, off=1)
    dy = _rand((M, H), dtype, 2, 1.0, 0.1, pad=(H + 1) % 2, off=3)
    w = _rand((1, H), wdtype, 3, 0.3, 1.0, off=1)[0]
    b = _rand((1, H), wdtype, 4, 0.2)[0]
    o = L.layer_norm_fwd(x, w, b, EPS)
    torch.cuda.synchronize()
    k = _wide(H, dtype)
    yr, mean, rstd = O.layer_norm(_np(x), _np(w), _np(b), EPS)
    xh = (_np(x) - mean[:, None]) * rstd[:, None]
    _check("y", o.y, yr, HALF[dtype] * np.abs(yr) + U * (np.abs(_np(w)) * (60 + k + (44 + k) * np.abs(xh))
                                                         + 4 * np.abs(yr)) + 1e-30)
    _check("mean", o.mean, mean, U * (np.abs(mean) + (60 + k) / rstd))
    _check("rstd", o.rstd, rstd, U * (40 + k) * rstd)

    g = L.layer_norm_bwd(dy, x, w, o.mean, o.rstd)
    torch.cuda.synchronize()
    m_, r_ = _np(o.mean), _np(o.rstd)
    dx, dw, db = O.layer_norm_grads(_np(dy), _np(x), _np(w), m_, r_)
    xh = np.abs((_np(x) - m_[:, None]) * r_[:, None])
    ga = np.abs(_np(dy) * _np(w))
    a1, a2 = ga.mean(1, keepdims=True), (ga * xh).mean(1, keepdims=True)
    tol = HALF[dtype] * np.abs(dx) + U * (r_[:, None] * (4 * ga + (60 + k) * (a1 + xh * a2)) + 4 * np.abs(dx)) + 1e-30
    _check("dx", g.grad_x, dx, tol)
    _check("dw", g.grad_weight, dw, HALF[wdtype] * np.abs(dw) + (M + 4) * U * (np.abs(_np(dy)) * xh).sum(0) + 1e-30)
    _check("db", g.grad_bias, db, HALF[wdtype] * np.abs(db) + (M + 4) * U * np.abs(_np(dy)).sum(0) + 1e-30)
    # parts of the gradients alone are the same bits, and so is a second call
    only = L.layer_norm_bwd(dy, x, w, o.mean, o.rstd, need_params=False)
    par = L.layer_norm_bwd(dy, x, w, o.mean, o.rstd, need_x=False)
    assert only.grad_weight is None and par.grad_x is None
    assert torch.equal(only.grad_x, g.grad_x)
    assert torch.equal(par.grad_weight, g.grad_weight) and torch.equal(par.grad_bias, g.grad_bias)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layer_norm_without_parameters_and_in_shapes(dtype):
    import torch
    import linear_cross_entropy_gemm_amd as L
    x = _rand((6, 40), dtype, 5).reshape(2, 3, 40)
    plain = L.layer_norm_fwd(x)
    ones = torch.ones(40, device="cuda", dtype=_dt(dtype))
    full = L.layer_norm_fwd(x, ones, torch.zeros_like(ones))
    assert plain.y.shape == x.shape and plain.mean.shape == (2, 3)
    assert torch.equal(plain.y, full.y) and torch.equal(plain.rstd, full.rstd)
    # one dimension, a transposed view, a broadcast row
    assert torch.equal(L.layer_norm_fwd(x[0, 0]).y, plain.y[0, 0])
    t = x.reshape(6, 40).t().contiguous().t()
    assert torch.equal(L.layer_norm_fwd(t).y, plain.y.reshape(6, 40))
    assert torch.equal(L.layer_norm_fwd(x[0, :1].expand(5, 40)).y, plain.y[0, :1].expand(5, 40))
    g = L.layer_norm_bwd(x[0, :1].expand(5, 40), x[0, :1].expand(5, 40), None, full.mean[0, :1].repeat(5),
                         full.rstd[0, :1].repeat(5))
    assert torch.equal(g.grad_x[0], g.grad_x[4])
    # no rows
    e = L.layer_norm_fwd(x[:0], ones, ones)
    assert e.y.shape == (0, 3, 40)
    g = L.layer_norm_bwd(x[:0], x[:0], ones, e.mean, e.rstd)
    torch.cuda.synchronize()
    assert g.grad_x.shape == (0, 3, 40) and not g.grad_weight.any() and not g.grad_bias.any()


def test_layer_norm_offset_rows_keep_their_deviations():
    """A row far from zero: the first mean's rounding (2^-24 of 1000) is
    taken out again, so y keeps fp32 accuracy relative to the deviations; a
    constant row normalises to the bias, a row with an infinity or a NaN is
    NaN and leaves its neighbours alone."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    x = _rand((4, 1000), "f32", 6, 1.0, 1000.0)
    x[1] = 7.0
    x[2, 17] = float("inf")
    b = torch.full((1000,), 0.25, device="cuda")
    o = L.layer_norm_fwd(x, None, b, EPS)
    torch.cuda.synchronize()
    y, _, _ = O.layer_norm(_np(x)[[0, 3]], None, _np(b), EPS)
    # x - mean0 is exact to u of the deviation; the rest as in the header
    _check("y", o.y[[0, 3]], y, U * (60 + 44 * np.abs(y) + 4 * np.abs(y)))
    assert torch.equal(o.y[1], b) and o.y[2].isnan().all()


@pytest.mark.parametrize("dtype,wdtype,M,H", [("f32", "f32", 7, 130), ("bf16", "f32", 40, 700), ("bf16", "bf16", 3, 64)])
def test_layer_norm_autograd_matches_the_formula_and_differences(dtype, wdtype, M, H):
    import torch
    import linear_cross_entropy_gemm_amd as L
    x = _rand((M, H), dtype, 7, 2.0, 0.5).requires_grad_()
    w = _rand((1, H), wdtype, 8, 0.3, 1.0)[0].clone().requires_grad_()
    b = _rand((1, H), wdtype, 9)[0].clone().requires_grad_()
    dy = _rand((M, H), dtype, 10)
    y = L.layer_norm(x, w, b, 0.1)
    gx, gw, gb = torch.autograd.grad(y, (x, w, b), dy)
    o = L.layer_norm_fwd(x.detach(), w.detach(), b.detach(), 0.1)
    g = L.layer_norm_bwd(dy, x.detach(), w.detach(), o.mean, o.rstd)
    assert torch.equal(y, o.y) and torch.equal(gx, g.grad_x)
    assert torch.equal(gw, g.grad_weight) and torch.equal(gb, g.grad_bias)
    assert gx.dtype == x.dtype and gw.dtype == w.dtype and gb.dtype == b.dtype
    # central differences of the fp64 definition along random directions: the
    # step 1e-5 leaves 1e-9; the gradients' own errors are bounded as above,
    # here by their storage rounding and 80 u of the magnitudes involved
    X, W, B, D = _np(x), _np(w), _np(b), _np(dy)
    r = np.random.default_rng(11)
    vx, vw, vb = r.normal(size=X.shape), r.normal(size=H), r.normal(size=H)
    h = 1e-5
    f = lambda s: float((D * O.layer_norm(X + s * h * vx, W + s * h * vw, B + s * h * vb, 0.1)[0]).sum())
    num = (f(1) - f(-1)) / (2 * h)
    ana = float((_np(gx) * vx).sum() + (_np(gw) * vw).sum() + (_np(gb) * vb).sum())
    _, mean, rstd = O.layer_norm(X, W, B, 0.1)
    mag = rstd[:, None] * np.abs(D * W) + np.abs(_np(gx))
    tol = (np.abs(_np(gx) * vx).sum() * HALF[dtype] * 1.01 + (np.abs(_np(gw) * vw).sum() + np.abs(_np(gb) * vb).sum())
           * HALF[wdtype] * 1.01 + 80 * U * (mag * np.abs(vx)).sum() * (1 + np.sqrt(H))
           + (M + 80) * U * (np.abs(D) * (4 + np.abs(X - mean[:, None]) * rstd[:, None])).sum() + 1e-6 * (1 + abs(num)))
    log(f"[ln] differences {num:.6f} gradient {ana:.6f} bound {tol:.2e}")
    assert abs(num - ana) <= tol


@pytest.mark.parametrize("use", ["x", "w", "b", "wb"])
def test_layer_norm_autograd_computes_what_is_asked(use):
    import torch
    import linear_cross_entropy_gemm_amd as L
    x, w, b = _rand((5, 96), "bf16", 12), _rand((1, 96), "f32", 13)[0].clone(), _rand((1, 96), "f32", 14)[0].clone()
    dy = _rand((5, 96), "bf16", 15)
    leaves = {"x": x, "w": w, "b": b}
    for k in use:
        leaves[k].requires_grad_()
    got = torch.autograd.grad(L.layer_norm(x, w, b), [leaves[k] for k in use], dy)
    o = L.layer_norm_fwd(x.detach(), w.detach(), b.detach())
    g = L.layer_norm_bwd(dy, x.detach(), w.detach(), o.mean, o.rstd)
    want = {"x": g.grad_x, "w": g.grad_weight, "b": g.grad_bias}
    assert all(torch.equal(a, want[k]) for a, k in zip(got, use))
    # a bias without a weight, of another dtype than x
    bb = b.detach().clone().requires_grad_()
    gb, = torch.autograd.grad(L.layer_norm(x.detach(), None, bb), bb, dy)
    assert gb.dtype == torch.float32


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,p,seed,offset", [(1, 0.5, 0, 0), (7, 0.3, 1, 2), (1024, 0.0, 5, 1), (4099, 0.1, 2 ** 64 - 1, 0),
                                             (100003, 0.9, 3 << 40, 7 << 40), (2049, 1.0, 4, 4),
                                             (33333, 0.25, 12345, 2 ** 64 - 1)])
def test_dropout(n, p, seed, offset, dtype):
    import torch
    import linear_cross_entropy_gemm_amd as L
    log(f"[dropout] n={n} p={p} seed={seed} offset={offset} {dtype}")
    x = _rand((1, n), dtype, 20, 2.0, off=1)[0]
    res = _rand((1, n), dtype, 21, off=3)[0]
    if n > 10:
        x[3], x[5], x[8] = float("inf"), float("nan"), 0.0
    xn = _np(x)
    keep = O.dropout_keep(n, p, seed, offset)
    for r in (None, res):
        y = L.dropout(x, p, seed, offset, residual=r)
        torch.cuda.synchronize()
        got = _np(y)
        base = np.zeros(n) if r is None else _np(r)
        assert np.array_equal(got[~keep], base[~keep])
        with np.errstate(invalid="ignore"):
            ref = base + xn / (1.0 - p) if p < 1.0 else base
        fin = keep & np.isfinite(ref)
        assert np.array_equal(np.isnan(got[keep]), np.isnan(ref[keep]))
        assert np.array_equal(np.isinf(got[keep]), np.isinf(ref[keep]))
        tol = HALF[dtype] * (1 + 4 * U) * np.abs(ref) + 3 * U * (np.abs(xn) / max(1 - p, 1e-9) + np.abs(ref))
        assert (np.abs(got[fin] - ref[fin]) <= tol[fin]).all()
        y2 = L.dropout(x, p, seed, torch.tensor([offset - 2 ** 64 if offset >= 2 ** 63 else offset], device="cuda"), r)
        assert torch.equal(y2.view(torch.int16 if dtype == "bf16" else torch.int32),
                           y.view(torch.int16 if dtype == "bf16" else torch.int32))


def test_dropout_gradients_and_shapes():
    import torch
    import linear_cross_entropy_gemm_amd as L
    x = _rand((6, 50), "bf16", 22).reshape(2, 3, 50).requires_grad_()
    r = _rand((6, 50), "bf16", 23).reshape(2, 3, 50).requires_grad_()
    g = _rand((6, 50), "bf16", 24).reshape(2, 3, 50)
    y = L.dropout(x, 0.4, 9, 1, residual=r)
    gx, gr = torch.autograd.grad(y, (x, r), g)
    assert torch.equal(gr, g) and torch.equal(gx, L.dropout(g, 0.4, 9, 1))
    # the map is linear in x: its difference along any direction is the kept
    # share of that direction, which the mask gives exactly
    keep = O.dropout_keep(300, 0.4, 9, 1).reshape(2, 3, 50)
    assert np.array_equal(_np(gx) != 0, keep & (_np(g) != 0))
    # a transposed view counts elements in its own row-major order
    t = x.detach().reshape(6, 50).t()
    assert torch.equal(L.dropout(t, 0.4, 9, 1), L.dropout(t.contiguous(), 0.4, 9, 1))
    assert L.dropout(x.detach()[:0], 0.4, 9).shape == (0, 3, 50)
    s = torch.ones((), device="cuda")
    assert L.dropout(s, 0.0, 9).item() == 1.0
    with pytest.raises(ValueError, match="residual"):
        L.dropout(x, 0.4, 9, 1, residual=r[:1])
    for bad in (dict(p=1.5), dict(seed=-1), dict(offset=-1), dict(offset=torch.zeros(2, dtype=torch.int64, device="cuda")),
                dict(offset=torch.zeros(1, dtype=torch.int64))):
        with pytest.raises(ValueError):
            L.dropout(x, **{"p": 0.4, "seed": 9, **bad})


def test_dropout_second_derivative():
    """The map is linear, so the gradient of its gradient with respect to the
    upstream gradient is the map again."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    x, v = _rand((3, 70), "f32", 26).requires_grad_(), _rand((3, 70), "f32", 27)
    g = _rand((3, 70), "f32", 28).requires_grad_()
    gx, = torch.autograd.grad(L.dropout(x, 0.3, 5), x, g, create_graph=True)
    gg, = torch.autograd.grad(gx, g, v)
    assert torch.equal(gg, L.dropout(v, 0.3, 5))


def test_dropout_offset_changed_before_the_backward_pass_raises():
    import torch
    import linear_cross_entropy_gemm_amd as L
    off = torch.zeros(1, dtype=torch.int64, device="cuda")
    x = _rand((2, 64), "f32", 25).requires_grad_()
    y = L.dropout(x, 0.5, 3, off)
    off.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("H", [5, 700, 6656, 20001])
@pytest.mark.parametrize("c", [-3e38, 1e38, 1e30])
def test_layer_norm_of_a_huge_constant_row(H, c):
    """The row's sum overflows fp32, its mean does not: y is the bias.  (Exactly:
    the rounding of the mean leaves deviations of 0, or of at least one step of
    c, whose squares overflow and make rstd 0.)"""
    import torch
    import linear_cross_entropy_gemm_amd as L
    x = torch.full((3, H), c, dtype=torch.float32, device="cuda")
    b = _rand((1, H), "f32", 60)[0].clone()
    o = L.layer_norm_fwd(x, None, b)
    assert torch.all((o.mean.double() - x[0, 0].double()).abs() <= 2.0 ** -18 * abs(c))
    assert torch.equal(o.y, b.expand(3, H))


def test_layer_norm_bias_gradient_without_a_weight():
    """A float32 bias beside bfloat16 rows: its gradient is not rounded to
    bfloat16 on the way."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    M, H = 200, 300
    x, dy = _rand((M, H), "bf16", 61), _rand((M, H), "bf16", 62)
    b = torch.zeros(H, device="cuda", requires_grad=True)
    gb, = torch.autograd.grad(L.layer_norm(x, None, b), b, dy)
    assert gb.dtype == torch.float32
    _check("db", gb, _np(dy).sum(0), (M + 4) * U * np.abs(_np(dy)).sum(0))
    o = L.layer_norm_fwd(x)
    g = L.layer_norm_bwd(dy, x, None, o.mean, o.rstd, param_dtype=torch.float32)
    assert torch.equal(g.grad_bias, gb) and g.grad_weight.dtype == torch.float32
    for weight, d in ((b.detach(), torch.bfloat16), (None, torch.float16)):
        with pytest.raises(TypeError):
            L.layer_norm_bwd(dy, x, weight, o.mean, o.rstd, param_dtype=d)


def test_step_replays_from_a_captured_graph():
    """Dropout, layer norm and their gradients in one captured graph, four
    replays with eager work in between; the dropout offset advances on the
    device, so each replay draws the mask of its step."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    x, r = _rand((130, 700), "bf16", 30), _rand((130, 700), "bf16", 31)
    w, b = _rand((1, 700), "f32", 32, 0.2, 1.0)[0].clone(), _rand((1, 700), "f32", 33)[0].clone()
    dy = _rand((130, 700), "bf16", 34)
    off = torch.zeros(1, dtype=torch.int64, device="cuda")
    ws = torch.empty(L.flce_layer_norm_bwd_workspace_size(130, 700, L.FLCE_DTYPE_BF16), dtype=torch.uint8,
                     device="cuda")

    def step(offset):
        z = L.dropout(x, 0.2, 77, offset, residual=r)
        o = L.layer_norm_fwd(z, w, b)
        g = L.layer_norm_bwd(dy, z, w, o.mean, o.rstd, ws)
        return o.y, g.grad_weight, g.grad_bias, g.grad_x, L.dropout(g.grad_x, 0.2, 77, offset)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(off)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(off)
    torch.cuda.synchronize()
    seen = []
    for rep in range(4):
        off.fill_(rep)
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = step(rep)       # the program's own eager work between replays
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(got, want)), rep
        seen.append(got[0])
    assert not torch.equal(seen[0], seen[1])


def test_autograd_step_replays_from_a_captured_graph():
    """The differentiable functions and their backward pass in one captured
    graph; eager steps of the same leaves run before it and between replays."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    x, r = (_rand((70, 900), "bf16", 63 + i).requires_grad_() for i in range(2))
    w, b = (_rand((1, 900), "f32", 65 + i, 0.2, 1.0)[0].clone().requires_grad_() for i in range(2))
    dy = _rand((70, 900), "bf16", 67)
    off = torch.zeros(1, dtype=torch.int64, device="cuda")

    def step(offset):
        y = L.layer_norm(L.dropout(x, 0.2, 78, offset, residual=r), w, b)
        return (y.detach(), *torch.autograd.grad(y, (x, r, w, b), dy))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(off)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(off)
    torch.cuda.synchronize()
    for rep in range(4):
        off.fill_(rep)
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        want = step(rep)
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(got, want)), rep


def test_two_streams_match_separate_calls():
    import torch
    import linear_cross_entropy_gemm_amd as L
    xs = [_rand((600, 900), "bf16", 40 + i) for i in range(2)]
    dys = [_rand((600, 900), "bf16", 50 + i) for i in range(2)]

    def call(i):
        o = L.layer_norm_fwd(xs[i])
        g = L.layer_norm_bwd(dys[i], xs[i], None, o.mean, o.rstd)
        return o.y, g.grad_x, g.grad_weight, L.dropout(xs[i], 0.3, i)

    alone = [call(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    both = [None, None]
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            both[i] = call(i)
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, c) for a, c in zip(alone[i], both[i]))


def test_outputs_end_where_their_rows_end():
    """Canaries behind strided outputs, in-place forms, through the C ABI."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    st = torch.cuda.current_stream().cuda_stream
    M, H = 6, 37
    x = _rand((M, H), "bf16", 60, pad=4)
    want = L.layer_norm_fwd(x)
    buf = torch.full((M, H + 5), 3.0, dtype=torch.bfloat16, device="cuda")
    assert L.flce_layer_norm_fwd(x.data_ptr(), H + 4, None, None, M, H, EPS, buf.data_ptr(), H + 5, None, None, st, 0,
                                 0) == L.FLCE_OK
    gx = torch.full((M, H + 3), 3.0, dtype=torch.bfloat16, device="cuda")
    g = L.layer_norm_bwd(x, x, None, want.mean, want.rstd, need_params=False)
    assert L.flce_layer_norm_bwd(x.data_ptr(), H + 4, x.data_ptr(), H + 4, None, want.mean.data_ptr(),
                                 want.rstd.data_ptr(), M, H, gx.data_ptr(), H + 3, None, None, st, 0, 0, None,
                                 0) == L.FLCE_OK
    torch.cuda.synchronize()
    assert torch.equal(buf[:, :H], want.y) and (buf[:, H:] == 3.0).all()
    assert torch.equal(gx[:, :H], g.grad_x) and (gx[:, H:] == 3.0).all()
    y = x.clone(memory_format=torch.contiguous_format)
    assert L.flce_layer_norm_fwd(y.data_ptr(), H, None, None, M, H, EPS, y.data_ptr(), H, None, None, st, 0,
                                 0) == L.FLCE_OK
    d = torch.full((45,), 2.0, device="cuda")
    assert L.flce_dropout(d.data_ptr(), None, d.data_ptr(), 41, 1.0, 0, 0, None, st, 1) == L.FLCE_OK
    torch.cuda.synchronize()
    assert torch.equal(y, want.y) and not d[:41].any() and (d[41:] == 2.0).all()


@pytest.mark.parametrize("reduction", ["mean", "none"])
def test_lm_head_loss_runs_the_operators_together(reduction):
    """The head's path equals its operators called one by one, loss and
    gradients bitwise, and the fp64 composition of the oracles within bf16
    rounding of the intermediate states."""
    import torch
    import oracle
    import linear_cross_entropy_gemm_amd as L
    N, H, V = 70, 96, 530
    x, r = (_rand((N, H), "bf16", 70 + i).requires_grad_() for i in range(2))
    w = _rand((1, H), "f32", 72, 0.2, 1.0)[0].clone().requires_grad_()
    b = _rand((1, H), "f32", 73, 0.2)[0].clone().requires_grad_()
    W = (_rand((V, H), "bf16", 74) * 0.1).requires_grad_()
    lab = torch.randint(0, V, (N,), generator=torch.Generator().manual_seed(5)).cuda()
    lab[::9] = -100
    kw = dict(residual=r, dropout_p=0.15, seed=11, offset=6, softcap=30.0, multiplier=0.5, reduction=reduction)
    loss, nc = L.lm_head_loss(x, W, lab, w, b, **kw)
    up = torch.rand(loss.shape, generator=torch.Generator().manual_seed(6)).cuda()
    got = torch.autograd.grad(loss, (x, r, W, w, b), up)
    xs, rs, Ws, w2, b2 = (t.detach().requires_grad_() for t in (x, r, W, w, b))
    y = L.layer_norm(L.dropout(xs, 0.15, 11, 6, rs), w2, b2)
    loss2, nc2 = L.linear_cross_entropy(y, Ws, lab, -100, 30.0, 0.5, reduction)
    want = torch.autograd.grad(loss2, (xs, rs, Ws, w2, b2), up)
    assert torch.equal(loss, loss2) and torch.equal(nc, nc2)
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    z = O.dropout(_np(x), 0.15, 11, 6, _np(r))
    yr, mean, rstd = O.layer_norm(z, _np(w), _np(b), 1e-5)
    ref = oracle.flce_reference(yr, _np(W), lab.cpu().numpy(), -100, 30.0, 0.5, "sum" if reduction == "none" else "mean")
    mine = float(loss.detach().sum())
    rel = abs(mine - ref["loss"]) / abs(ref["loss"])
    log(f"[head] {reduction}: loss {mine:.5f} oracle {ref['loss']:.5f}")
    # z and y are rounded to bf16 (2^-8 each, and y's deviations shift by as
    # much): a logit sums H products of |y| ~ 1 and |W| ~ 0.1 with m = 0.5, so
    # its error is at most 3 * 2^-8 * 0.5 * sum |y W| and the loss moves by no
    # more than twice the largest of those
    la = 0.5 * (np.abs(yr) @ np.abs(_np(W)).T).max()
    assert abs(mine - ref["loss"]) <= 2 * 3 * 2.0 ** -8 * la * (1 if reduction == "mean" else N) and rel < 0.05


def test_layer_norm_rows_far_apart():
    """Row offsets past 2^31 elements, in every tensor."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    ld, H = (1 << 31) + 8191, 700
    st = torch.cuda.current_stream().cuda_stream
    bufs = [torch.empty(ld + H, dtype=torch.bfloat16, device="cuda").as_strided((2, H), (ld, 1)) for _ in range(4)]
    x, dy, y, gx = bufs
    x.copy_(_rand((2, H), "bf16", 80))
    dy.copy_(_rand((2, H), "bf16", 81))
    want = L.layer_norm_fwd(x.contiguous())
    g = L.layer_norm_bwd(dy.contiguous(), x.contiguous(), None, want.mean, want.rstd)
    log("[ln] rows far apart")
    assert L.flce_layer_norm_fwd(x.data_ptr(), ld, None, None, 2, H, EPS, y.data_ptr(), ld, None, None, st, 0,
                                 0) == L.FLCE_OK
    assert L.flce_layer_norm_bwd(dy.data_ptr(), ld, x.data_ptr(), ld, None, want.mean.data_ptr(), want.rstd.data_ptr(),
                                 2, H, gx.data_ptr(), ld, None, None, st, 0, 0, None, 0) == L.FLCE_OK
    o = L.layer_norm_fwd(x)
    torch.cuda.synchronize()
    assert torch.equal(y, want.y) and torch.equal(gx, g.grad_x) and torch.equal(o.y, want.y)


def test_dropout_past_2_to_the_32_elements():
    """The last elements of a tensor of more than 2^32: their words come from
    counters past 2^30 (elements / 4)."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    n, tail = (1 << 32) + 1001, 4001
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    log("[dropout] 2^32 + 1001 elements")
    y = L.dropout(x, 0.25, 5, 6)
    torch.cuda.synchronize()
    first = (n - tail) // 4
    blk = np.arange(first, (n + 3) // 4, dtype=np.uint64)
    ctr = np.zeros((blk.size, 4), dtype=np.uint64)
    ctr[:, 0], ctr[:, 1], ctr[:, 2] = blk & np.uint64(0xFFFFFFFF), blk >> np.uint64(32), 6
    keep = (O.philox4x32_10(ctr, (5, 0)).reshape(-1) >= np.uint64(1 << 30))[:n - first * 4]
    got = _np(y[first * 4:])
    assert np.array_equal(got != 0, keep) and set(got[keep]) == {float(torch.tensor(4 / 3).bfloat16())}
    assert 0.745 < float((y[::4099] != 0).float().mean()) < 0.755


def test_operators_take_numpy_scalars_and_empty_batches():
    import torch
    import linear_cross_entropy_gemm_amd as L
    x = _rand((4, 96), "bf16", 90)
    assert torch.equal(L.dropout(x, np.float32(0.5), np.int64(3), np.uint32(2)), L.dropout(x, 0.5, 3, 2))
    u = torch.rand(4, device="cuda")
    a = L.sample(x, u, np.float32(0.5), np.int32(7), np.float64(0.5), np.float32(0.25)).tokens
    assert torch.equal(a, L.sample(x, u, 0.5, 7, 0.5, 0.25).tokens)
    assert torch.equal(L.layer_norm(x, eps=np.float32(0.5)), L.layer_norm(x, eps=0.5))
    W = _rand((50, 96), "bf16", 91).clone()
    w = torch.ones(96, device="cuda")
    o = L.lm_head_sample(x[:0], W, u[:0], w)
    assert o.tokens.shape == (0,)
    loss, n = L.lm_head_loss(x[:0], W, torch.zeros(0, dtype=torch.int64, device="cuda"), w)
    assert loss.item() == 0.0 and n.item() == 0
