"""GPU parity of the 4-bit projection against its fp64 definition on exactly the
values the GPU reads.

Packing is exact arithmetic (a maximum's exponent, a division by a power of
two, comparisons): codes and scales have to be equal.

Logits: with u = 2^-24, a sum of Kp products (3 Kp with fp32) that adds them one
by one is off by at most 2 u of the running sum each time:
|dz| <= 2 u Kp parts sum|x w| m.  What the matrix unit cuts comes on top for bf16
and 8-bit rows: of the 8 products that it adds at a time each may lose 2^-13 of
the largest, and a bf16 element below 2^-14 of its block's largest is off by
2^-22 of that largest.  fp32 rows' digits are whole numbers of 2^-24 of their
block's largest, off by half of one, and their sums lose nothing but the fp32
roundings.
The softcap adds 1e-6 of its value, the store half a step.
"""
import numpy as np
import pytest

from gpu_util import log
from oracle import head as O

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("require_gpu")]

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": U}


def _dt(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _rand(shape, dtype, seed, scale=1.0, pad=0, off=0):
    """A seeded tensor; its rows lie `pad` elements apart in a buffer that
    starts `off` elements past an aligned address."""
    import torch
    g = torch.Generator().manual_seed(seed)
    v = (torch.randn(shape, generator=g) * scale).to(_dt(dtype))
    M, H = shape
    buf = torch.zeros(M * (H + pad) + off + 8, dtype=_dt(dtype), device="cuda")
    out = buf[off:off + M * (H + pad)].view(M, H + pad)[:, :H]
    out.copy_(v)
    return out


def _np(t):
    return t.detach().double().cpu().numpy()


def _codes(w):
    b = w.data.cpu().numpy()
    return np.stack((b & 15, b >> 4), 2).reshape(b.shape[0], -1)


def _weights(w):
    """[V, hidden] in fp64."""
    import torch
    c = _codes(w)
    v = O.E2M1[c & 7] * (1 - 2.0 * (c >> 3))
    e = w.scales.view(torch.uint8).cpu().numpy().astype(np.float64) - 127
    return (v * np.repeat(2.0 ** e, 32, 1))[:, :w.hidden]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,H", [(1, 1), (3, 31), (7, 32), (5, 100), (40, 128), (33, 1001), (300, 513), (1000, 2048)])
def test_pack_is_exact(V, H, dtype):
    import torch
    import linear_cross_entropy_gemm_amd as L
    W = _rand((V, H), dtype, 1, 0.02, pad=H % 3, off=1) * (10.0 ** torch.linspace(-8, 8, V, device="cuda"))[:, None]
    W = W.to(_dt(dtype))
    W[V // 2, : H // 2] = 0
    # ties and borders of the scale
    W[0, : min(H, 8)] = torch.tensor([6.0, 5.0, -2.5, 0.25, 0.75, 1.25, 1.75, 3.5], device="cuda")[:min(H, 8)].to(W.dtype)
    q = L.mx4_pack(W)
    code, e = O.mx_quantize(_np(W), O.E2M1)
    assert np.array_equal(_codes(q)[:, :H], code) and not _codes(q)[:, H:].any()
    s = q.scales.view(torch.uint8).cpu().numpy()
    assert np.array_equal(s[:, :e.shape[1]], e + 127) and not s[:, e.shape[1]:].any()


def test_pack_special_blocks():
    import torch
    import linear_cross_entropy_gemm_amd as L
    W = torch.ones(3, 96, device="cuda")
    W[0, 40], W[1, 3], W[2, 95] = float("inf"), float("nan"), 3.4e38
    s = L.mx4_pack(W).scales.view(torch.uint8).cpu()
    assert s[:, :3].tolist() == [[125, 255, 125], [255, 125, 125], [125, 125, 253]]
    e = L.mx4_pack(W[:0])
    assert e.data.shape == (0, 64) and L.mx4_pack(W.t().contiguous().t()).scales.view(torch.uint8).cpu().equal(s)


def _groups(a, n):
    """[rows, K] padded to whole groups of n: [rows, K / n, n]."""
    pad = -a.shape[1] % n
    return np.pad(a, ((0, 0), (0, pad))).reshape(a.shape[0], -1, n)


def _cut(x, w, fp32):
    """What the rounding of the rows' parts and the matrix unit's sums of 8 may
    cost, [N, V]; of the latter a bound: the largest product of 8 is at most the
    largest |x| times the largest |w|, and the products beside it are 7."""
    bx, bw = np.abs(_groups(x, 32)).max(2), np.abs(_groups(w, 32)).sum(2)
    if fp32:
        return U * bx @ bw.T
    return 2.0 ** -22 * bx @ bw.T + 7 * 2.0 ** -13 * np.abs(_groups(x, 8)).max(2) @ np.abs(_groups(w, 8)).max(2).T


def _check_logits(z, x, w, cap, mult, out, parts):
    z, ref = _np(z), x @ w.T * mult
    tol = 2 * U * parts * ((w.shape[1] + 127) // 128 * 128) * (np.abs(x) @ np.abs(w).T) * abs(mult)
    tol = tol + _cut(x, w, parts == 3) * abs(mult)
    if cap:
        ref = cap * np.tanh(ref / cap)
        tol = tol + 1e-6 * np.abs(ref)
    tol = tol + HALF[out] * (np.abs(ref) + tol) + 2 * U * np.abs(ref)
    bad = np.abs(z - ref) - tol
    log(f"  worst error minus bound {bad.max():.2e}, relative {np.linalg.norm(z - ref) / np.linalg.norm(ref):.1e}")
    assert bad.max() <= 0.0, np.unravel_index(int(np.argmax(bad)), bad.shape)


# one column, a block, a step and their neighbours, several chunks; one vocabulary
# entry, a tile, ragged ones; tokens across every border between the kernels
SHAPES = [(1, 1, 1), (2, 31, 15), (5, 32, 64), (1, 100, 129), (16, 128, 130), (17, 129, 1000), (3, 255, 70),
          (33, 1001, 2001), (64, 512, 300), (65, 640, 77), (1, 6656, 4099), (130, 2049, 1003), (5, 7168, 515)]


@pytest.mark.parametrize("kind", ["bf16", "f32", "mx8"])
@pytest.mark.parametrize("N,H,V", SHAPES)
def test_logits(N, H, V, kind):
    import torch
    import linear_cross_entropy_gemm_amd as L
    log(f"[mx4] N={N} H={H} V={V} {kind}")
    q = L.mx4_pack(_rand((V, H), "f32", 1, 0.05))
    w = _weights(q)
    cap, mult = (3.0, 0.5) if H % 2 else (0.0, 1.0)
    out = "f32" if kind == "f32" else "bf16"
    if kind == "mx8":
        x = L.rms_norm_mx8(_rand((N, H), "bf16", 2), None, 1e-6).rows
        xn = _np(x.data) * np.repeat(_np(x.scales), 32, 1)[:, :H]
    else:
        x = _rand((N, H), kind, 2, pad=H % 3, off=1)
        xn = _np(x)
    z = L.logits_mx4(x, q, cap, mult)
    assert z.shape == (N, V) and z.dtype == _dt(out)
    _check_logits(z, xn, w, cap, mult, out, 3 if kind == "f32" else 1)
    # the other output type, rows of a wider buffer, not a byte behind them
    other = "bf16" if out == "f32" else "f32"
    buf = torch.full((N, V + 3), 7.0, dtype=_dt(other), device="cuda")
    z2 = L.logits_mx4(x, q, cap, mult, out=buf)
    _check_logits(z2, xn, w, cap, mult, other, 3 if kind == "f32" else 1)
    assert buf[:, V:].eq(7.0).all()


@pytest.mark.parametrize("N,H,V", [(1, 1024, 2000), (1, 8192, 500), (5, 4096, 500), (20, 2049, 400), (40, 1001, 3001),
                                   (100, 4096, 300), (300, 7168, 200)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_logits_accuracy(N, H, V, kind):
    """Over random rows the errors are independent, so they are held to their
    root mean square.  fp32: Kp / 128 sums rounded to nearest (u / sqrt 3 of a
    running sum that reaches the rms z only at the end: below u sqrt(64) / 2),
    2 u for the last instruction of each, u / sqrt 3 x 2.5 for the digits (the
    largest of 32 is 2.5 of their rms): below 8 u in all, 16 u allowed.  bf16:
    7 of 8 products lose up to 2^-13 of the group's largest (2.2 rms of a
    product), on average half, of which an rms of 2^-13 2.2 / sqrt 3 x 2^-3 at
    most is behind the value's own last bit (a product of 8 by 2 significant
    bits lies below 2^-13 of the largest with 3 or fewer of its bits): 2^-15.6 of
    a product, and both sums grow with sqrt Kp; 2^-15 allowed."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    q = L.mx4_pack(_rand((V, H), "f32", 3, 0.02))
    x = _rand((N, H), kind, 4)
    ref = _np(x) @ _weights(q).T
    z = _np(L.logits_mx4(x, q, out=torch.empty(N, V, device="cuda")))
    err = np.sqrt(np.mean((z - ref) ** 2) / np.mean(ref ** 2))
    log(f"[mx4] N={N} H={H} V={V} {kind}: relative rms error {err:.2e}")
    assert err <= (16 * U if kind == "f32" else 2.0 ** -15)


def _outlier_rows(N, H, kind):
    x = _rand((N, H), kind, 6)
    x[:, 5::97] *= 1000.0
    return x


@pytest.mark.parametrize("kind", ["bf16", "f32", "mx8"])
@pytest.mark.parametrize("N", [1, 3, 16, 20, 48, 64, 200])
@pytest.mark.parametrize("H,V", [(130, 700), (385, 257), (1500, 4100), (2560, 16)])
def test_logits_outliers_and_borders(N, H, V, kind):
    """Few columns a thousand times the others; steps that are no multiple of
    four, token counts of every kernel, vocabularies of few tiles and of more
    than the work-groups have."""
    import linear_cross_entropy_gemm_amd as L
    q = L.mx4_pack(_rand((V, H), "f32", 5, 0.05))
    x = _outlier_rows(N, H, "bf16" if kind == "mx8" else kind)
    if kind == "mx8":
        x = L.rms_norm_mx8(x, None, 1e-6).rows
        xn = _np(x.data) * np.repeat(_np(x.scales), 32, 1)[:, :H]
    else:
        xn = _np(x)
    z = L.logits_mx4(x, q)
    assert z.equal(L.logits_mx4(x, q))
    _check_logits(z, xn, _weights(q), 0.0, 1.0, "f32" if kind == "f32" else "bf16", 3 if kind == "f32" else 1)


@pytest.mark.parametrize("H", [512, 1024, 1536])
@pytest.mark.parametrize("N", [5, 40, 130])
def test_mx8_rows_of_every_alignment(N, H):
    """Rows that the products read in place and rows that are brought to a
    workspace first: the same logits, bit for bit."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    q = L.mx4_pack(_rand((333, H), "f32", 7, 0.05))
    rows = L.rms_norm_mx8(_rand((N, H), "bf16", 8), None, 1e-6).rows
    z = L.logits_mx4(rows, q)
    wide = torch.zeros(N, H + 48, dtype=torch.uint8, device="cuda")
    codes = torch.zeros(N, H // 32 + 3, dtype=torch.uint8, device="cuda")
    for off in (0, 1, 16):
        d, s = wide[:, off:off + H].view(torch.float8_e4m3fn), codes[:, off % 3:off % 3 + H // 32].view(torch.float8_e8m0fnu)
        d.copy_(rows.data)
        s.copy_(rows.scales)
        assert L.logits_mx4(L.Mx8Rows(d, s), q).equal(z)


@pytest.mark.parametrize("kind", ["bf16", "f32", "mx8"])
@pytest.mark.parametrize("N", [2, 7, 40, 130])
def test_rows_that_overlap(N, kind):
    """One row for all tokens, and windows that lie closer than their length:
    the logits of the same rows apart, bit for bit."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    H = 1024
    q = L.mx4_pack(_rand((333, H), "f32", 9, 0.05))
    for step in (0, 16, 512):
        x = _rand((1, step * (N - 1) + H), "bf16" if kind == "mx8" else kind, 10)[0]
        if kind == "mx8":
            s = torch.randint(120, 130, (step // 32 * (N - 1) + H // 32 + 512,), dtype=torch.uint8, device="cuda")
            x = x.clamp(-400, 400).to(torch.float8_e4m3fn)
            data = torch.as_strided(x, (N, H), (step, 1))
            scales = torch.as_strided(s.view(torch.float8_e8m0fnu), (N, H // 32), (step // 32, 1))
            rows = L.Mx8Rows(data, scales)
            apart = L.Mx8Rows(data.view(torch.uint8).clone().view(data.dtype).contiguous(),
                              scales.view(torch.uint8).clone().view(scales.dtype).contiguous())
        else:
            rows = torch.as_strided(x, (N, H), (step, 1))
            apart = rows.clone().contiguous()
        z = L.logits_mx4(rows, q)
        assert z.equal(L.logits_mx4(apart, q))
        assert step or (z == z[:1]).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_far_scales(kind):
    """Tokens and weights near both ends of the exponent's range, whose products
    are ordinary numbers."""
    import linear_cross_entropy_gemm_amd as L
    for up in (100, -90):
        q = L.mx4_pack(_rand((200, 300), "f32", 11, 2.0 ** up))
        x = _rand((20, 300), kind, 12, 2.0 ** -up)
        _check_logits(L.logits_mx4(x, q), _np(x), _weights(q), 0.0, 1.0, kind, 3 if kind == "f32" else 1)


@pytest.mark.parametrize("kind", ["bf16", "f32", "mx8"])
def test_special_values(kind):
    """What is not finite stays in its row, and in its vocabulary entry."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    W = _rand((200, 300), "f32", 1, 0.05)
    W[77, 100] = float("nan")
    W[5] = 0.0
    q = L.mx4_pack(W)
    x = _rand((20, 300), "bf16" if kind == "mx8" else kind, 2)
    x[3, 7], x[4, 9] = float("nan"), float("inf")
    x[6] = 0.0
    if kind == "mx8":
        data = x.float().to(torch.float8_e4m3fn)
        s = torch.full((20, 10), 127, dtype=torch.uint8, device="cuda")
        s[4, 0] = 255
        x = L.Mx8Rows(data, s.view(torch.float8_e8m0fnu))
    z = L.logits_mx4(x, q).float().cpu()
    fine = [i for i in range(20) if i not in (3, 4)]
    cols = [i for i in range(200) if i not in (77,)]
    assert z[3].isnan().all() and not z[4, cols].isfinite().any()
    assert z[:, 77].isnan().all() and z[fine][:, cols].isfinite().all()
    assert z[fine, 5].eq(0).all() and z[6, cols].eq(0).all()
    # the far ends of the scale
    c = q.scales.view(torch.uint8).clone()
    c[:, 0], c[:, 1] = 0, 252
    far = L.Mx4Weight(q.data, c.view(torch.float8_e8m0fnu), 300)
    one = torch.zeros(1, 300, dtype=torch.bfloat16, device="cuda")
    one[0, 2] = 2.0 ** 100
    assert np.array_equal(_np(L.logits_mx4(one.float(), far))[0, cols], _weights(far)[cols, 2] * 2.0 ** 100)
    one.zero_()
    one[0, 33] = 2.0 ** -100
    assert np.array_equal(_np(L.logits_mx4(one, far))[0, cols], _weights(far)[cols, 33] * 2.0 ** -100)


def test_fp32_parts_are_exact():
    """One nonzero column and a weight of 1 return x itself, over its range: the
    last digit's unit is 2^-136 at least, a 24th bit of 2^-113."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    W = torch.zeros(16, 128, device="cuda")
    W[3, 17] = 1.0
    q = L.mx4_pack(W)
    v = torch.randn(1000, device="cuda") * 10.0 ** torch.linspace(-30, 37.9, 1000, device="cuda")
    v[0], v[1], v[2] = 3.4028234663852886e38, -3.4028234663852886e38, 1.0 + 2.0 ** -23
    v = torch.where(v.isfinite() & (v.abs() >= 2.0 ** -113), v, 1.5)
    x = torch.zeros(1000, 128, device="cuda")
    x[:, 17] = v
    assert torch.equal(L.logits_mx4(x, q)[:, 3], v)


def test_layouts_and_refusals():
    import torch
    import linear_cross_entropy_gemm_amd as L
    q = L.mx4_pack(_rand((70, 96), "bf16", 1, 0.05))
    x = _rand((6, 96), "bf16", 2)
    ref = L.logits_mx4(x, q)
    assert torch.equal(L.logits_mx4(x.view(2, 3, 96), q), ref.view(2, 3, 70))
    assert torch.equal(L.logits_mx4(x.t().contiguous().t(), q), ref)
    assert torch.equal(L.logits_mx4(x[2:3].expand(4, 96), q), ref[2:3].expand(4, 70))
    assert L.logits_mx4(x[:0], q).shape == (0, 70)
    r = L.rms_norm_mx8(x.view(2, 3, 96), None).rows
    assert torch.equal(L.logits_mx4(r, q).view(6, 70), L.logits_mx4(L.rms_norm_mx8(x, None).rows, q))
    for bad in (lambda: L.logits_mx4(x[:, :95], q), lambda: L.logits_mx4(x, q, out=ref[:, :69]),
                lambda: L.logits_mx4(x, q, out=ref.half()), lambda: L.logits_mx4(L.Mx8Rows(r.data, r.scales[:1]), q),
                lambda: L.logits_mx4(x, L.Mx4Weight(q.data.cpu(), q.scales.cpu(), 96))):
        with pytest.raises(ValueError):
            bad()


def test_rows_far_apart():
    """Rows of x and of the logits more than 2^31 elements from the first."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    q = L.mx4_pack(_rand((70, 96), "bf16", 1, 0.05))
    ld = (1 << 30) + 12345
    v = _rand((3, 96), "bf16", 2)
    x = torch.zeros(2 * ld + 128, dtype=torch.bfloat16, device="cuda").as_strided((3, 96), (ld, 1))
    out = torch.zeros(2 * ld + 128, dtype=torch.bfloat16, device="cuda").as_strided((3, 70), (ld, 1))
    x.copy_(v)
    L.logits_mx4(x, q, out=out)
    assert torch.equal(out, L.logits_mx4(v, q))


@pytest.mark.parametrize("N,kind", [(3, "bf16"), (12, "mx8"), (40, "bf16"), (70, "mx8"), (20, "f32")])
def test_weights_beyond_32_bits(N, kind):
    """More than 2^32 bytes of weights: the last entries' logits as from those
    entries alone, bit for bit (an entry's sums do not depend on its tile)."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    V, H, last = (1 << 20) + 5000, 8192, 4321
    g = torch.Generator(device="cuda").manual_seed(13)
    data = torch.randint(0, 256, (V, H // 2), dtype=torch.uint8, device="cuda", generator=g)
    scales = torch.randint(115, 122, (V, H // 32), dtype=torch.uint8, device="cuda", generator=g)
    x = _rand((N, H), "bf16" if kind == "mx8" else kind, 14)
    if kind == "mx8":
        x = L.rms_norm_mx8(x, None, 1e-6).rows
    z = L.logits_mx4(x, L.Mx4Weight(data, scales.view(torch.float8_e8m0fnu), H))
    few = L.Mx4Weight(data[-last:].clone(), scales[-last:].clone().view(torch.float8_e8m0fnu), H)
    assert z.isfinite().all() and L.logits_mx4(x, few).equal(z[:, -last:])


def test_captured_and_on_two_streams():
    import torch
    import linear_cross_entropy_gemm_amd as L
    q = L.mx4_pack(_rand((3000, 640), "bf16", 1, 0.05))
    x = [_rand((n, 640), "bf16", n) for n in (1, 40)]
    ref = [L.logits_mx4(v, q) for v in x]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    out = [None, None]
    for k in range(2):
        with torch.cuda.stream(s[k]):
            out[k] = L.logits_mx4(x[k], q)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = L.rms_norm_mx8(x[1], None).rows
        z = L.logits_mx4(r, q)
    for k in range(3):
        x[1].copy_(_rand((40, 640), "bf16", 50 + k))
        ref = L.logits_mx4(L.rms_norm_mx8(x[1], None).rows, q)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, ref)


@pytest.mark.parametrize("mx8", [False, True])
def test_decoding_head(mx8):
    """lm_head_sample over an RMS norm and a 4-bit projection is its operators
    one by one."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    x, r = _rand((10, 192), "bf16", 1), _rand((10, 192), "bf16", 2)
    w = _rand((1, 192), "f32", 3, 0.2)[0]
    W = _rand((5000, 192), "bf16", 4, 0.1)
    q = L.mx4_pack(W)
    u = torch.rand(10, device="cuda")
    o = L.lm_head_sample(x, q, u, w, eps=1e-6, temperature=0.8, top_p=0.9, logprobs=True, norm="rms", norm_offset=1.0,
                         residual=r, mx8=mx8)
    f = L.rms_norm_mx8 if mx8 else L.rms_norm_fwd
    y = f(x, w, 1e-6, residual=r, offset=1.0)
    t = L.sample(L.logits_mx4(y.rows if mx8 else y.y, q), u, temperature=0.8, top_p=0.9, logprobs=True)
    assert torch.equal(o.tokens, t.tokens) and torch.equal(o.logprobs, t.logprobs)
    # with bf16 weights, and behind a layer norm
    o = L.lm_head_sample(x, W, u, w, eps=1e-6, norm="rms", residual=r)
    y = L.rms_norm_fwd(x, w, 1e-6, residual=r).y
    assert torch.equal(o.tokens, L.sample(L.logits(y, W), u).tokens)
    o = L.lm_head_sample(x.view(2, 5, 192), q, u.view(2, 5), w)
    t = L.sample(L.logits_mx4(L.layer_norm(x, w), q), u)
    assert torch.equal(o.tokens.view(-1), t.tokens)
