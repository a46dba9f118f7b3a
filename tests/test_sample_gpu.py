"""GPU parity of token sampling with the fp64 definition
(``oracle.head.sample_row``) on exactly the logits the GPU reads.

Tokens have to be equal.  The kernels' weights are off by at most 2^-39 of the
largest (an integer rounding) and the oracle's sums by V 2^-53, so a random
number closer than 1e-9 to the end of its token's interval could differ; the
seeded inputs stay clear of that (checked).  logprob is a 64-bit logarithm
rounded to fp32: half a unit of its size, plus 1e-9 of the sum.
"""
import numpy as np
import pytest

from gpu_util import log
from oracle import head as O

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("require_gpu")]


def _dt(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _logits(N, V, dtype, kind, seed, pad=0, off=0):
    """Seeded logits whose rows lie `pad` elements apart (the gap holds NaN
    and +inf: reading it would show) at `off` elements past alignment."""
    import torch
    r = np.random.default_rng(seed)
    z = r.normal(size=(N, V)) * {"flat": 1.6, "peaked": 2.5, "masked": 2.0, "ties": 0.0}[kind]
    if kind == "peaked":
        for i in range(N):
            c = r.permutation(V)[:max(1, min(V // 4, 40))]
            z[i, c] = 6 + 8 * r.random(c.size)
    if kind == "masked":
        z[r.random((N, V)) < 0.8] = -np.inf
        z[:, V // 2] = 0.5
    if kind == "ties":
        z = r.integers(-2, 3, size=(N, V)).astype(np.float64)
    buf = torch.full((N * (V + pad) + off + 16,), float("inf"), dtype=_dt(dtype), device="cuda")
    buf[::2] = float("nan")
    out = buf[off:off + N * (V + pad)].view(N, V + pad)[:, :V]
    out.copy_(torch.from_numpy(z).to(_dt(dtype)))
    return out


def _u(N, seed):
    import torch
    return torch.rand(N, generator=torch.Generator().manual_seed(seed)).cuda()


def _rowval(v, i):
    return float(v[i]) if hasattr(v, "shape") and v.dim() else float(np.float32(v))


def _compare(z, u, o, t=1.0, k=0, p=1.0, q=0.0):
    import torch
    torch.cuda.synchronize()
    zn = z.float().cpu().numpy().astype(np.float64)
    tok, lp = o.tokens.cpu().numpy(), o.logprobs.cpu().numpy()
    for i in range(zn.shape[0]):
        want, wl, border = O.sample_row(zn[i], float(u[i]), _rowval(t, i), int(_rowval(k, i)), _rowval(p, i),
                                        _rowval(q, i))
        assert border > 1e-9 or want == -1, (i, border)
        assert tok[i] == want, (i, tok[i], want)
        assert lp[i] == wl or abs(lp[i] - wl) <= 2.0 ** -24 * abs(wl) + 1e-9, (i, lp[i], wl)


PARAMS = {
    "plain": dict(), "greedy": dict(temperature=0.0), "cold": dict(temperature=0.01), "hot": dict(temperature=50.0),
    "k1": dict(top_k=1), "k5": dict(top_k=5, temperature=0.8), "k50p95": dict(top_k=50, top_p=0.95, temperature=0.8),
    "k300": dict(top_k=300), "k5000": dict(top_k=5000, top_p=0.8), "kall": dict(top_k=1 << 40),
    "p50": dict(top_p=0.5), "p90": dict(top_p=0.9), "p99": dict(top_p=0.99, temperature=1.3), "p0": dict(top_p=1e-30),
    "q5": dict(min_p=0.05), "q100": dict(min_p=1.0), "all": dict(top_k=200, top_p=0.9, min_p=0.02, temperature=1.2),
}


def _kw(prm):
    names = {"temperature": "t", "top_k": "k", "top_p": "p", "min_p": "q"}
    return {names[a]: b for a, b in prm.items()}


@pytest.mark.parametrize("kind", ["flat", "peaked", "masked", "ties"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V", [(2, 1), (3, 2), (5, 37), (4, 64), (3, 65), (4, 256), (3, 257),
                                 (6, 1000), (3, 1024), (3, 1025), (3, 2048), (3, 2049), (3, 3001), (3, 8191), (2, 8193), (2, 33001)])
def test_sample(N, V, dtype, kind):
    import linear_cross_entropy_gemm_amd as L
    z = _logits(N, V, dtype, kind, N * V, pad=V % 5, off=1)
    u = _u(N, V)
    for name, prm in PARAMS.items():
        log(f"[sample] N={N} V={V} {dtype} {kind} {name}")
        _compare(z, u, L.sample(z, u, **prm, logprobs=True), **_kw(prm))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["flat", "peaked", "ties"])
def test_sample_large_vocabulary_with_row_parameters(dtype, kind):
    import torch
    import linear_cross_entropy_gemm_amd as L
    N, V = 12, 202048
    z, u = _logits(N, V, dtype, kind, 5, pad=1), _u(N, 6)
    g = torch.Generator().manual_seed(7)
    t = (0.5 + torch.rand(N, generator=g)).cuda()
    t[3] = 0.0
    k = torch.tensor([0, 1, 40, 200, 0, 300, 1000, 50000, 0, 17, 0, 0]).cuda()
    p = torch.tensor([1.0, 0.9, 0.8, 1.0, 0.5, 0.95, 1.0, 0.9, 0.99, 1.0, 0.3, 1.0]).cuda()
    q = torch.tensor([0.0, 0.0, 0.1, 0.0, 0.0, 0.01, 0.3, 0.0, 0.0, 0.0, 0.0, 0.001]).cuda()
    log(f"[sample] N={N} V={V} {dtype} {kind} row parameters")
    o = L.sample(z, u, t, k, p, q, logprobs=True)
    _compare(z, u, o, t, k, p, q)
    # rows do not depend on one another, nor on the outputs asked for
    for i in (0, 4, 7):
        one = L.sample(z[i:i + 1], u[i:i + 1], t[i:i + 1], k[i:i + 1], p[i:i + 1], q[i:i + 1])
        assert one.logprobs is None and one.tokens.item() == o.tokens[i].item()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [9, 700, 20000])
def test_sample_special_values(dtype, V):
    """Rows the mask leaves empty, infinities, NaN, the type's lowest value,
    zeros of both signs, one candidate, and the ends of u's range."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    inf = float("inf")
    z = _logits(10, V, dtype, "flat", V)
    z[0] = -inf
    z[1] = float("nan")
    z[2, 3], z[2, 7] = inf, inf
    z[3, ::2] = float("nan")
    z[4] = torch.finfo(z.dtype).min
    z[5] = torch.finfo(z.dtype).min
    z[5, 5] = 0.0
    z[6] = 0.0
    z[6, ::2] = -0.0
    z[7] = -inf
    z[7, V - 1] = -3.0
    z[8] = torch.finfo(z.dtype).max
    z[8, 1] = torch.finfo(z.dtype).min
    z[9, 4] = torch.finfo(z.dtype).tiny / 2
    for lo in (True, False):
        u = torch.full((10,), 2.0 ** -20 if lo else 1.0 - 2.0 ** -24, device="cuda")
        for name in ("plain", "greedy", "k5", "k300", "p50", "q5", "all"):
            prm = PARAMS[name]
            log(f"[sample] special V={V} {dtype} {name} u={u[0].item():.8f}")
            o = L.sample(z, u, **prm, logprobs=True)
            torch.cuda.synchronize()
            zn = z.float().cpu().numpy().astype(np.float64)
            for i in range(10):
                want = O.sample_row(zn[i], float(u[i]), *(float(np.float32(prm.get(a, b))) if a != "top_k" else
                                                          prm.get(a, b) for a, b in (("temperature", 1.0), ("top_k", 0),
                                                                                     ("top_p", 1.0), ("min_p", 0.0))))
                assert o.tokens[i].item() == want[0], (i, name)
            assert o.logprobs[0].item() == -inf and o.tokens[0].item() == o.tokens[1].item() == -1
    # u = 0 draws the first kept token
    u = torch.zeros(10, device="cuda")
    o = L.sample(z, u)
    assert o.tokens.tolist()[2:8] == [3, 1, 0, 5, 0, V - 1]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sample_masked_pieces_and_extreme_temperatures(dtype):
    """Long stretches without a candidate, and temperatures at which every
    weight is the same or all but the largest vanish."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    V = 41000
    z = _logits(6, V, dtype, "peaked", 31)
    z[0, :8192 * 4] = float("-inf")
    z[1, 8192:] = float("-inf")
    z[2, 9000:40000] = float("-inf")
    z[3] *= 1e30
    z[4] *= 1e-30
    z[5, ::2] = torch.finfo(z.dtype).min
    u = _u(6, 32)
    for t in (1e-30, 1e-5, 1e25, 3e38):
        for name in ("plain", "k5", "k300", "p90", "q5", "all"):
            prm = dict(PARAMS[name], temperature=t)
            log(f"[sample] masked pieces {dtype} {name} t={t}")
            _compare(z, u, L.sample(z, u, **prm, logprobs=True), **_kw(prm))
    for name, prm in PARAMS.items():
        log(f"[sample] masked pieces {dtype} {name}")
        _compare(z, u, L.sample(z, u, **prm, logprobs=True), **_kw(prm))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["flat", "peaked", "masked", "ties"])
@pytest.mark.parametrize("V", [2049, 9001, 40000])
def test_sample_more_rows_than_compute_units(V, dtype, kind):
    """A batch of 300 equals its rows in smaller batches, all of them, and the
    definition on every 37th."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    N = 300
    z, u = _logits(N, V, dtype, kind, V), _u(N, V)
    pick = slice(0, N, 37)
    for name in ("plain", "greedy", "k5", "k300", "k5000", "p50", "p90", "q5", "all"):
        prm = PARAMS[name]
        log(f"[sample] N={N} V={V} {dtype} {kind} {name}")
        o = L.sample(z, u, **prm, logprobs=True)
        parts = [L.sample(z[i:i + 100], u[i:i + 100], **prm, logprobs=True) for i in range(0, N, 100)]
        assert torch.equal(o.tokens, torch.cat([q.tokens for q in parts]))
        assert torch.allclose(o.logprobs, torch.cat([q.logprobs for q in parts]), rtol=2.0 ** -23, atol=1e-9)
        _compare(z[pick], u[pick], L.SampleOutputs(o.tokens[pick], o.logprobs[pick]), **_kw(prm))


def test_sample_many_short_rows():
    import linear_cross_entropy_gemm_amd as L
    z, u = _logits(70001, 5, "f32", "flat", 33), _u(70001, 34)
    o = L.sample(z, u, 0.9, 3, 0.8, logprobs=True)
    _compare(z[::997], u[::997], L.SampleOutputs(o.tokens[::997], o.logprobs[::997]), 0.9, 3, 0.8)
    # the lowest logit of five is never among the first three
    assert not (o.tokens == z.argmin(1)).any()


@pytest.mark.parametrize("V", [700, 20000])
def test_sample_rows_far_apart(V):
    """Row offsets past 2^32 bytes and past 2^31 elements."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    ld = (1 << 31) + 12345
    buf = torch.empty(ld + V, dtype=torch.bfloat16, device="cuda")
    z = buf.as_strided((2, V), (ld, 1))
    z.copy_(_logits(2, V, "bf16", "peaked", 35))
    u = _u(2, 36)
    for prm in ({}, dict(top_k=40, top_p=0.9), dict(top_p=0.9), dict(temperature=0.0)):
        log(f"[sample] rows far apart V={V} {prm}")
        _compare(z, u, L.sample(z, u, **prm, logprobs=True), **_kw(prm))


def test_sample_bad_row_values_give_no_token():
    import torch
    import linear_cross_entropy_gemm_amd as L
    z = _logits(12, 100, "f32", "flat", 1)
    nan, inf = float("nan"), float("inf")
    u = torch.tensor([0.5] * 8 + [1.0, -0.1, nan, 0.5], device="cuda")
    t = torch.tensor([-1.0, nan, inf] + [1.0] * 9, device="cuda")
    p = torch.tensor([1.0] * 3 + [0.0, 1.1, nan] + [1.0] * 6, device="cuda")
    q = torch.tensor([0.0] * 6 + [2.0, -0.1] + [0.0] * 4, device="cuda")
    k = torch.zeros(12, dtype=torch.int64, device="cuda")
    o = L.sample(z, u, t, k, p, q, logprobs=True)
    assert o.tokens.tolist()[:11] == [-1] * 11 and o.tokens[11].item() >= 0
    k[11] = -4
    assert L.sample(z, u, t, k, p, q).tokens[11].item() == -1


def test_sample_shapes_and_refusals():
    import torch
    import linear_cross_entropy_gemm_amd as L
    z = _logits(6, 50, "bf16", "flat", 2).clone()
    u = _u(6, 3)
    flat = L.sample(z, u).tokens
    assert torch.equal(L.sample(z.view(2, 3, 50), u.view(2, 3)).tokens, flat.view(2, 3))
    assert torch.equal(L.sample(z.t().contiguous().t(), u).tokens, flat)
    assert L.sample(z[0], u[:1]).tokens.shape == () and L.sample(z[0], u[:1]).tokens.item() == flat[0].item()
    assert L.sample(z[:0], u[:0]).tokens.shape == (0,)
    # one row of logits for many random numbers
    many = _u(40, 4)
    o = L.sample(z[:1].expand(40, 50), many, logprobs=True)
    _compare(z[:1].expand(40, 50), many, o)
    for bad in (dict(u=u[:5]), dict(u=u.double()), dict(u=u.cpu()), dict(top_k=torch.zeros(6, device="cuda")),
                dict(top_p=torch.ones(5, device="cuda")), dict(min_p=torch.zeros(6)),
                dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            L.sample(**{"logits": z, "u": u, **bad})
    for bad in (dict(temperature=-1.0), dict(top_k=-1), dict(top_p=0.0), dict(min_p=1.5)):
        with pytest.raises(L.FlceError):
            L.sample(z, u, **bad)


def test_sample_replays_from_a_captured_graph():
    import torch
    import linear_cross_entropy_gemm_amd as L
    z, u = _logits(5, 30011, "bf16", "peaked", 8), _u(5, 9)
    ws = torch.empty(L.flce_sample_workspace_size(5, 30011, L.FLCE_DTYPE_BF16), dtype=torch.uint8, device="cuda")
    call = lambda: L.sample(z, u, 0.9, 40, 0.9, 0.01, logprobs=True, workspace=ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = call()
    for rep in range(4):
        u.copy_(_u(5, 20 + rep))
        z.mul_(-1.0)
        o.tokens.fill_(-7)
        graph.replay()
        torch.cuda.synchronize()
        _compare(z, u, o, 0.9, 40, 0.9, 0.01)
        got = o.tokens.clone()
        want = L.sample(z, u, 0.9, 40, 0.9, 0.01)     # eager, a workspace of its own
        assert torch.equal(got, want.tokens)


def test_sample_on_two_streams():
    import torch
    import linear_cross_entropy_gemm_amd as L
    zs = [_logits(40, 20000, "f32", k, 10) for k in ("peaked", "flat")]
    us = [_u(40, 11), _u(40, 12)]
    call = lambda i: L.sample(zs[i], us[i], 1.1, 0, 0.9, logprobs=True)
    alone = [call(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    both = [None, None]
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            both[i] = call(i)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        assert torch.equal(a.tokens, b.tokens) and torch.equal(a.logprobs, b.logprobs)


def test_sample_outputs_end_where_their_rows_end():
    import torch
    import linear_cross_entropy_gemm_amd as L
    z, u = _logits(3, 777, "bf16", "flat", 13), _u(3, 14)
    tok = torch.full((5,), -9, dtype=torch.int64, device="cuda")
    lp = torch.full((5,), 9.0, device="cuda")
    need = L.flce_sample_workspace_size(3, 777, 0)
    ws = torch.full((need + 256,), 7, dtype=torch.uint8, device="cuda")
    prm = L.flce_sample_params_t(temperature=1.0, top_p=0.9, top_k=30)
    st = torch.cuda.current_stream().cuda_stream
    assert L.flce_sample(z.data_ptr(), 777, u.data_ptr(), 3, 777, prm, tok.data_ptr(), lp.data_ptr(), st, 0,
                         ws.data_ptr(), need) == L.FLCE_OK
    torch.cuda.synchronize()
    assert (tok[:3] >= 0).all() and (tok[3:] == -9).all() and (lp[3:] == 9.0).all() and (ws[need:] == 7).all()


@pytest.mark.parametrize("V", [530, 4099])
def test_lm_head_sample_runs_the_operators_together(V):
    import torch
    import linear_cross_entropy_gemm_amd as L
    g = torch.Generator().manual_seed(15)
    x = torch.randn((2, 3, 96), generator=g).to(torch.bfloat16).cuda()
    W = (torch.randn((V, 96), generator=g) * 0.2).to(torch.bfloat16).cuda()
    w, b = (torch.randn(96, generator=g).cuda() for _ in range(2))
    u = torch.rand((2, 3), generator=g).cuda()
    kw = dict(temperature=0.8, top_k=40, top_p=0.9, logprobs=True)
    o = L.lm_head_sample(x, W, u, w, b, softcap=30.0, multiplier=0.5, **kw)
    z = L.logits(L.layer_norm(x, w, b).reshape(6, 96), W, 30.0, 0.5)
    want = L.sample(z, u.reshape(6), **kw)
    assert o.tokens.shape == (2, 3) and torch.equal(o.tokens.reshape(6), want.tokens)
    assert torch.equal(o.logprobs.reshape(6), want.logprobs)
    _compare(z, u.reshape(6), want, 0.8, 40, 0.9)
