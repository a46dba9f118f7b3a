"""GPU parity of draft verification with the fp64 definition
(``oracle.head.verify``) on exactly the logits the GPU reads.

Tokens and counts have to be equal.  A kernel's probability is a 64-bit
exponential (relative error 2^-38) over a sum of such (2^-38): u q against p is
decided within 2^-36 of them, and a sum of r, of terms at most 2^-37 (p + q) +
2^-52 off, within 2^-35 = 2.9e-11.  1e-10 is above all of these: the seeded inputs
stay clear of it (checked), but for draws from an r of next to no weight, as a
token leaves that no draft would draw: those have to be possible ones.  logprob is a 64-bit logarithm rounded to fp32: half a
unit of its size, plus 1e-9.
"""
import numpy as np
import pytest

from gpu_util import log
from oracle import head as O

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("require_gpu")]


def _dt(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def _padded(z, dtype, pad, off):
    """z [R, V] on the GPU, rows `pad` elements apart (the gap holds NaN and
    +inf: reading it would show) at `off` elements past alignment."""
    import torch
    R, V = z.shape
    buf = torch.full((R * (V + pad) + off + 16,), float("inf"), dtype=_dt(dtype), device="cuda")
    buf[::2] = float("nan")
    out = buf[off:off + R * (V + pad)].view(R, V + pad)[:, :V]
    out.copy_(torch.from_numpy(z).to(_dt(dtype)))
    return out


def _case(B, K, V, dtype, kind, seed, pad=0, off=0):
    """(target, draft, tokens, lens, u, u_draw): tokens that the draft makes
    likely, a few others, and one out of range."""
    import torch
    r = np.random.default_rng(seed)
    z = r.normal(size=(B, K + 1, V)) * {"flat": 1.6, "peaked": 2.5, "masked": 2.0, "ties": 0.0}[kind]
    if kind == "peaked":
        for i in np.ndindex(B, K + 1):
            c = r.permutation(V)[:max(1, min(V // 4, 40))]
            z[i][c] = 6 + 8 * r.random(c.size)
    d = z[:, :K] + 0.5 * r.normal(size=(B, K, V))
    if kind == "masked":
        z[r.random(z.shape) < 0.8] = -np.inf
        d[r.random(d.shape) < 0.5] = -np.inf
        z[:, :, V // 2] = 0.5
        if B > 2:
            z[1, min(1, K)] = -np.inf
            d[2] = -np.inf
    if kind == "ties":
        z = r.integers(-2, 3, size=z.shape).astype(np.float64)
        d = np.where(r.random(d.shape) < 0.9, z[:, :K], r.integers(-2, 3, size=d.shape))
    x = np.zeros((B, K), dtype=np.int64)
    for i in np.ndindex(B, K):
        live = np.flatnonzero(d[i] > -np.inf)
        best = live[np.argsort(-d[i][live])][:5]
        x[i] = r.choice(best) if best.size and r.random() < 0.9 else r.integers(0, V)
    if B > 3 and K:
        x[3, K - 1] = V if V % 2 else -5
    t = _padded(z.reshape(-1, V), dtype, pad, off).unflatten(0, (B, K + 1))
    q = _padded(d.reshape(-1, V), dtype, pad + 1, off + 1).unflatten(0, (B, K)) if K else None
    lens = torch.from_numpy(r.integers(-1, K + 3, size=B)).cuda()
    u = torch.from_numpy(r.random((B, K)).astype(np.float32) * 0.999).cuda()
    ud = torch.from_numpy(r.random(B).astype(np.float32) * 0.999).cuda()
    return t, q, torch.from_numpy(x).cuda(), lens, u, ud


NAMES = ("temperature", "top_k", "top_p", "min_p")


def _of(prm, b, default=(1.0, 0, 1.0, 0.0)):
    out = []
    for n, dflt in zip(NAMES, default):
        v = prm.get(n, dflt)
        out.append(v[b].item() if hasattr(v, "dim") else v if n == "top_k" else float(np.float32(v)))
    return tuple(out)


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _compare(case, o, prm, dprm=None, with_draft=True, with_lens=True):
    t, q, x, lens, u, ud = case
    zt, zq = _np(t), _np(q) if with_draft and q is not None else None
    B, K = x.shape
    tok, acc, lp = o.tokens.cpu().numpy(), o.accepted.cpu().numpy(), o.logprobs.cpu().numpy()
    counts = 0
    for b in range(B):
        length = lens[b].item() if with_lens else K
        mine = _of(prm, b)
        want, n, wl, (border, turn, left) = O.verify(zt[b], None if zq is None else zq[b], x[b].cpu().numpy(), length,
                                       u[b].double().cpu().numpy(), ud[b].item(), mine,
                                       None if dprm is None else _of(dprm, b, mine))
        assert border > 1e-10 and (turn > 1e-10 or left < 1e-7), (b, border, turn, left)
        assert acc[b] == n, (b, acc[b], n)
        if turn <= 1e-10:
            p = O.row_distribution(zt[b, n], *mine)
            assert tok[b, :n].tolist() == want[:n].tolist() and p[tok[b, n]] > 0 and (tok[b, n + 1:] == -1).all()
            want, wl[n] = tok[b], np.log(p[tok[b, n]])
        assert tok[b].tolist() == want.tolist(), (b, tok[b], want)
        for a, w in zip(lp[b], wl):
            assert a == w or abs(a - w) <= 2.0 ** -24 * abs(w) + 1e-9, (b, lp[b], wl)
        counts += n
    log(f"  {counts} accepted of {B * K}")


PARAMS = {
    "plain": dict(), "greedy": dict(temperature=0.0), "cold": dict(temperature=0.05), "hot": dict(temperature=20.0),
    "k1": dict(top_k=1), "k5": dict(top_k=5, temperature=0.8), "k50p95": dict(top_k=50, top_p=0.95, temperature=0.8),
    "k300": dict(top_k=300), "kall": dict(top_k=1 << 40), "p50": dict(top_p=0.5), "p90": dict(top_p=0.9),
    "p99": dict(top_p=0.99, temperature=1.3), "q5": dict(min_p=0.05), "q100": dict(min_p=1.0),
    "q5p90": dict(min_p=0.05, top_p=0.9), "all": dict(top_k=200, top_p=0.9, min_p=0.02, temperature=1.2),
}


@pytest.mark.parametrize("kind", ["flat", "peaked", "masked", "ties"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,K,V", [(2, 1, 1), (4, 2, 2), (5, 3, 37), (4, 1, 64), (6, 4, 257), (5, 3, 1000), (4, 2, 2048),
                                   (4, 3, 2049), (5, 2, 4097), (4, 2, 8193), (4, 1, 20001)])
def test_verify(B, K, V, dtype, kind):
    import linear_cross_entropy_gemm_amd as L
    case = _case(B, K, V, dtype, kind, B * V + K, pad=V % 5, off=1)
    t, q, x, lens, u, ud = case
    for k, (name, prm) in enumerate(PARAMS.items()):
        log(f"[verify] B={B} K={K} V={V} {dtype} {kind} {name}")
        d, n = k % 3 != 1, k % 2 == 0
        o = L.verify(t, x, u, ud, draft_logits=q if d else None, draft_lens=lens if n else None, **prm, logprobs=True)
        _compare(case, o, prm, with_draft=d, with_lens=n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["flat", "peaked", "masked"])
def test_large_vocabulary_with_parameters_per_sequence(dtype, kind):
    import torch
    import linear_cross_entropy_gemm_amd as L
    B, K, V = 10, 3, 129279
    case = _case(B, K, V, dtype, kind, 5, pad=1)
    t, q, x, lens, u, ud = case
    g = torch.Generator().manual_seed(7)
    temperature = (0.5 + torch.rand(B, generator=g)).cuda()
    temperature[4] = 0.0
    prm = dict(temperature=temperature, top_k=torch.tensor([0, 1, 40, 200, 0, 300, 1000, 50000, 0, 17]).cuda(),
               top_p=torch.tensor([1.0, 0.9, 0.8, 1.0, 0.5, 0.95, 1.0, 0.9, 0.99, 1.0]).cuda(),
               min_p=torch.tensor([0.0, 0.0, 0.1, 0.0, 0.0, 0.01, 0.3, 0.0, 0.0, 0.0]).cuda())
    log(f"[verify] {dtype} {kind} parameters per sequence")
    o = L.verify(t, x, u, ud, draft_logits=q, draft_lens=lens, **prm, logprobs=True)
    _compare(case, o, prm)
    # a draft with parameters of its own
    own = dict(temperature=temperature.flip(0) + 0.1, top_p=0.7)
    o = L.verify(t, x, u, ud, draft_logits=q, **prm, draft_temperature=own["temperature"], draft_top_p=0.7,
                 logprobs=True)
    _compare(case, o, prm, dprm={**prm, **own}, with_lens=False)


@pytest.mark.parametrize("V", [50, 5000])
def test_many_drafted_tokens(V):
    """More positions than a wave has lanes, all accepted and not."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    B, K = 3, 200
    case = _case(B, K, V, "f32", "peaked", 3)
    t, q, x, lens, u, ud = case
    u[0] = 0.0
    x[0] = t[0, :K].argmax(1)
    u[1, :100] = 0.0
    x[1] = t[1, :K].argmax(1)
    lens[:] = torch.tensor([K, K, 70])
    o = L.verify(t, x, u, ud, draft_logits=q, draft_lens=lens, logprobs=True)
    _compare(case, o, {})
    assert o.accepted[0].item() == K and o.accepted[1].item() >= 100


@pytest.mark.parametrize("V", [300, 30001])
def test_without_drafted_tokens_it_is_sample(V):
    """K = 0, and sequences whose draft is empty."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    case = _case(20, 0, V, "bf16", "peaked", 3)
    t, _, x, _, u, ud = case
    for prm in PARAMS.values():
        o = L.verify(t, x, u, ud, **prm, logprobs=True)
        s = L.sample(t[:, 0], ud, **prm, logprobs=True)
        assert torch.equal(o.tokens[:, 0], s.tokens) and o.accepted.eq(0).all()
        assert torch.allclose(o.logprobs[:, 0], s.logprobs, rtol=2.0 ** -22, atol=1e-9)
    case = _case(20, 3, V, "bf16", "peaked", 4)
    t, q, x, lens, u, ud = case
    lens.zero_()
    o = L.verify(t, x, u, ud, draft_logits=q, draft_lens=lens, top_p=0.9)
    assert torch.equal(o.tokens[:, 0], L.sample(t[:, 0], ud, top_p=0.9).tokens) and o.tokens[:, 1:].eq(-1).all()


def test_special_logits_and_numbers():
    import torch
    import linear_cross_entropy_gemm_amd as L
    inf, nan = float("inf"), float("nan")
    for V in (6, 4100):
        t = torch.full((8, 2, V), -inf, device="cuda")
        t[:, :, :3] = torch.tensor([1.0, 2.0, 0.0])
        d = t[:, :1].clone()
        t[1, 0, 4] = inf                 # the whole weight
        t[2, 0] = -inf                   # nothing to draw
        d[3] = -inf                      # a draft that says nothing
        t[4, 0, 1] = nan
        t[5] = torch.finfo(torch.float32).min   # a mask of lowest values: all alike
        x = torch.tensor([1, 4, 1, 1, 1, 1, 1, 1], device="cuda")[:, None]
        u = torch.zeros(8, 1, device="cuda")
        ud = torch.full((8,), 0.5, device="cuda")
        u[6], ud[7], u[7] = nan, 1.0, 1.0
        o = L.verify(t, x, u, ud, draft_logits=d, logprobs=True)
        tok, n = o.tokens.cpu(), o.accepted.cpu().tolist()
        assert n == [1, 1, 0, 1, 0, 1, 0, 0]
        assert tok[:, 0].tolist()[:6] == [1, 4, -1, 1, 0, 1] and tok[0, 1] == 1
        assert tok[2].tolist() == [-1, -1] and tok[7].tolist() == [-1, -1] and tok[6, 0] >= 0
        assert o.logprobs[1, 0].item() == 0.0 and o.logprobs[2, 0].item() == -inf
        # parameters out of range in one sequence
        bad = torch.ones(8, device="cuda")
        bad[0] = -1.0
        o = L.verify(t, x, u, ud, draft_logits=d, temperature=bad)
        assert o.tokens[0].eq(-1).all() and o.accepted[0].item() == 0 and o.tokens[3, 0].item() == 1


def test_the_same_distribution_accepts_everything():
    import torch
    import linear_cross_entropy_gemm_amd as L
    for V, dtype in ((1000, "f32"), (50001, "bf16")):
        t = _case(40, 4, V, dtype, "flat", 9)[0]
        u = torch.full((40, 4), 1.0 - 2.0 ** -24, device="cuda")
        ud = torch.rand(40, device="cuda")
        for prm in (dict(), dict(top_p=0.9), dict(top_k=40, temperature=0.7), dict(min_p=0.01)):
            x = L.sample(t[:, :4], torch.rand(40, 4, device="cuda"), **prm).tokens
            o = L.verify(t, x, u, ud, draft_logits=t[:, :4], **prm)
            assert o.accepted.eq(4).all() and torch.equal(o.tokens[:, :4], x)


@pytest.mark.parametrize("top_p", [0.9, 1.0])
def test_tokens_follow_the_target(top_p):
    """By frequency over 40000 sequences of one draft and one target, within
    five standard deviations of a frequency."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    N, V = 40000, 12
    g = torch.Generator(device="cuda").manual_seed(1)
    t, d = torch.randn(2, V, generator=g, device="cuda") * 1.5, torch.randn(1, V, generator=g, device="cuda") * 1.5
    rnd = lambda *s: torch.rand(*s, generator=g, device="cuda") * (1 - 2.0 ** -24)  # noqa: E731
    t, d = t.expand(N, 2, V), d.expand(N, 1, V)
    kw = dict(top_p=top_p, temperature=0.8)
    x = L.sample(d, rnd(N, 1), **kw).tokens
    o = L.verify(t, x, rnd(N, 1), rnd(N), draft_logits=d, **kw)
    dist = lambda z: O.row_distribution(_np(z), float(np.float32(0.8)), 0, float(np.float32(top_p)))  # noqa: E731
    p, second, q = dist(t[0, 0]), dist(t[0, 1]), dist(d[0, 0])
    freq = lambda x: torch.bincount(x, minlength=V).double().cpu().numpy() / max(1, x.numel())  # noqa: E731
    assert np.abs(freq(o.tokens[:, 0]) - p).max() < 5 * np.sqrt(0.25 / N)
    assert abs(o.accepted.double().mean().item() - np.minimum(p, q).sum()) < 5 * np.sqrt(0.25 / N)
    both = o.tokens[o.accepted == 1, 1]
    if top_p == 1.0:
        assert both.numel() > 1000
    assert both.numel() == 0 or np.abs(freq(both) - second).max() < 5 * np.sqrt(0.25 / both.numel())


@pytest.mark.parametrize("V", [1500, 9000])
def test_rows_far_apart(V):
    """Rows of both sets of logits more than 2^31 elements from the first."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    B, K, ld = 2, 1, (1 << 30) + 12345
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn(B, K + 1, V, device="cuda", generator=g).bfloat16()
    d = torch.randn(B, K, V, device="cuda", generator=g).bfloat16()
    far = torch.zeros((B * (K + 1) - 1) * ld + V, dtype=torch.bfloat16, device="cuda")
    fz = far.as_strided((B, K + 1, V), ((K + 1) * ld, ld, 1))
    fz.copy_(z)
    fard = torch.zeros(3 * ld + V, dtype=torch.bfloat16, device="cuda")
    fd = fard.as_strided((B, K, V), (3 * ld, ld, 1))
    fd.copy_(d)
    x = torch.randint(0, V, (B, K), device="cuda", generator=g)
    u, ud = torch.rand(B, K, device="cuda", generator=g), torch.rand(B, device="cuda", generator=g)
    for prm in (dict(), dict(top_k=40, top_p=0.9), dict(top_p=0.8)):
        a = L.verify(z, x, u, ud, draft_logits=d, logprobs=True, **prm)
        b = L.verify(fz, x, u, ud, draft_logits=fd, logprobs=True, **prm)
        assert a.tokens.equal(b.tokens) and a.accepted.equal(b.accepted) and a.logprobs.equal(b.logprobs)


def test_layouts_workspaces_and_refusals():
    import torch
    import linear_cross_entropy_gemm_amd as L
    B, K, V = 6, 3, 5000
    t, q, x, lens, u, ud = _case(B, K, V, "f32", "peaked", 3)
    kw = dict(top_p=0.9, logprobs=True)
    ref = L.verify(t, x, u, ud, draft_logits=q, draft_lens=lens, **kw)
    o = L.verify(t.unflatten(0, (2, 3)), x.view(2, 3, K), u.view(2, 3, K), ud.view(2, 3),
                 draft_logits=q.unflatten(0, (2, 3)), draft_lens=lens.view(2, 3), **kw)
    assert o.tokens.shape == (2, 3, K + 1) and o.accepted.shape == (2, 3)
    assert torch.equal(o.tokens.view(B, -1), ref.tokens) and torch.equal(o.logprobs.view(B, -1), ref.logprobs)
    o = L.verify(t[0], x[0], u[0], ud[0], draft_logits=q[0], draft_lens=lens[0], **kw)
    assert torch.equal(o.tokens, ref.tokens[0]) and o.accepted.shape == ()
    # other layouts of the same logits; a workspace with anything in it
    ws = torch.full((L.flce_verify_workspace_size(B, K, V, L.FLCE_DTYPE_F32, 1),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        o = L.verify(t.transpose(0, 1).contiguous().transpose(0, 1), x.t().contiguous().t(), u, ud,
                     draft_logits=q.contiguous(), draft_lens=lens, workspace=ws, **kw)
        assert torch.equal(o.tokens, ref.tokens) and torch.equal(o.logprobs, ref.logprobs)
    e = L.verify(t[:0], x[:0], u[:0], ud[:0], draft_logits=q[:0])
    assert e.tokens.shape == (0, K + 1) and e.accepted.shape == (0,)
    for bad in (dict(draft_logits=q[:, :2]), dict(draft_logits=q.bfloat16()), dict(draft_lens=lens.int()),
                dict(draft_lens=lens[:2]), dict(temperature=ud[:3]), dict(workspace=ws[:512])):
        with pytest.raises(ValueError):
            L.verify(t, x, u, ud, **{"draft_logits": q, **bad})
    for args in ((t, x[:, :2], u, ud), (t, x.int(), u, ud), (t, x, u.double(), ud), (t, x, u, ud[:3]), (t, x, u, u)):
        with pytest.raises(ValueError):
            L.verify(*args)


def test_captured_and_on_two_streams():
    import torch
    import linear_cross_entropy_gemm_amd as L
    B, K, V = 5, 3, 20001
    cases = [_case(B, K, V, "bf16", kind, k) for k, kind in enumerate(("peaked", "flat"))]

    def call(c):
        return L.verify(c[0], c[2], c[4], c[5], draft_logits=c[1], draft_lens=c[3], top_p=0.9, logprobs=True)

    ref = [call(c) for c in cases]
    torch.cuda.synchronize()
    streams, out = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None]
    for k in range(2):
        with torch.cuda.stream(streams[k]):
            out[k] = call(cases[k])
    torch.cuda.synchronize()
    for a, b in zip(out, ref):
        assert torch.equal(a.tokens, b.tokens) and torch.equal(a.logprobs, b.logprobs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = call(cases[0])
    for k in range(4):
        new = _case(B, K, V, "bf16", "peaked", 20 + k)
        for a, b in zip(cases[0], new):
            a.copy_(b)
        ref = call(cases[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o.tokens, ref.tokens) and torch.equal(o.accepted, ref.accepted)
        assert torch.equal(o.logprobs, ref.logprobs)


def test_speculative_step_of_the_head():
    """Draft, verify, and the whole head in one call: RMS norm, 4-bit projection
    and verification, against the operators one by one."""
    import torch
    import linear_cross_entropy_gemm_amd as L
    B, K, H, V = 4, 3, 192, 5001
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, r = rnd(B, K + 1, H).bfloat16(), rnd(B, K + 1, H).bfloat16()
    w, W = rnd(H) * 0.2, (rnd(V, H) * 0.1).bfloat16()
    q = L.mx4_pack(W)
    d = L.logits_mx4(L.rms_norm(x[:, :K], w, 1e-6, residual=r[:, :K], offset=1.0)[0], q)
    tokens = L.sample(d, torch.rand(B, K, device="cuda"), temperature=0.8).tokens
    u, ud = torch.rand(B, K, device="cuda"), torch.rand(B, device="cuda")
    for mx8 in (False, True):
        o = L.lm_head_verify(x, q, tokens, u, ud, w, eps=1e-6, norm="rms", norm_offset=1.0, residual=r, mx8=mx8,
                             draft_logits=d, temperature=0.8, logprobs=True)
        y = (L.rms_norm_mx8 if mx8 else L.rms_norm_fwd)(x, w, 1e-6, residual=r, offset=1.0)
        z = L.logits_mx4(y.rows if mx8 else y.y, q)
        ref = L.verify(z, tokens, u, ud, draft_logits=d, temperature=0.8, logprobs=True)
        assert torch.equal(o.tokens, ref.tokens) and torch.equal(o.accepted, ref.accepted)
        assert torch.equal(o.logprobs, ref.logprobs)
        if not mx8:
            assert o.accepted.eq(K).all()   # the draft was this very head
    o = L.lm_head_verify(x, W, tokens, u, ud, w.abs())
    z = L.logits(L.layer_norm(x, w.abs()).view(-1, H), W).reshape(B, K + 1, V)
    assert torch.equal(o.tokens, L.verify(z, tokens, u, ud).tokens)
