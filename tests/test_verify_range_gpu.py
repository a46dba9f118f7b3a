"""Verification of more rows than compute units over long vocabularies, where
two rows share a compute unit, and beyond the rows that such a work-group has
room for: against the fp64 definition, and against the same sequences in
batches that are too small for it.

Both ways through the kernels agree to 2^-37 of a row's weight, far below the
distance of the seeded inputs from where a decision turns (checked where the
definition is computed); log-probabilities are fp32 numbers that differ by a
rounding, 2^-23 of their size, at most.
"""
import pytest

from gpu_util import log
from test_verify_gpu import _case, _compare

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("require_gpu")]


def _part(case, prm, s):
    """The sequences of a slice, with their parameters."""
    t, q, x, lens, u, ud = case
    return (t[s], None if q is None else q[s], x[s], lens[s], u[s], ud[s]), \
        {k: v[s] if hasattr(v, "dim") else v for k, v in prm.items()}


def _run(case, prm):
    import linear_cross_entropy_gemm_amd as L
    t, q, x, lens, u, ud = case
    return L.verify(t, x, u, ud, draft_logits=q, draft_lens=lens, **prm, logprobs=True)


def _same_as_in_small_batches(case, prm, whole, most):
    import torch
    B = case[2].shape[0]
    for b in range(0, B, most):
        s = slice(b, min(b + most, B))
        o = _run(*_part(case, prm, s))
        assert torch.equal(o.tokens, whole.tokens[s]) and torch.equal(o.accepted, whole.accepted[s]), s
        same = (o.logprobs == whole.logprobs[s]) | \
            ((o.logprobs - whole.logprobs[s]).abs() <= 2.0 ** -23 * o.logprobs.abs() + 1e-9)
        assert same.all(), s


def _per_sequence(B, seed, **which):
    import torch
    g = torch.Generator().manual_seed(seed)
    out = {}
    if "temperature" in which:
        out["temperature"] = 0.5 + torch.rand(B, generator=g)
        out["temperature"][4::9] = 0.0
    if "top_k" in which:
        out["top_k"] = torch.tensor([0, 1, 40, 200, 7000])[torch.randint(0, 5, (B,), generator=g)]
    if "top_p" in which:
        out["top_p"] = 0.5 + 0.5 * torch.rand(B, generator=g)
        out["top_p"][::3] = 1.0
    if "min_p" in which:
        out["min_p"] = 0.1 * torch.rand(B, generator=g)
        out["min_p"][::2] = 0.0
    return {k: v.cuda() for k, v in out.items()}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["flat", "peaked", "masked"])
@pytest.mark.parametrize("V", [70001, 129279])
def test_two_rows_a_compute_unit(V, dtype, kind):
    """R = 400 rows: 16 sequences against the definition, each five times."""
    import torch
    K, times = 2, 5
    few = _case(16, K, V, dtype, kind, V + len(kind), pad=V % 7, off=1)
    many = tuple(torch.cat([v] * times) for v in few)
    for name, prm in (("mixed", _per_sequence(16, 3, temperature=1, top_k=1, top_p=1, min_p=1)), ("plain", {}),
                      ("top_p", _per_sequence(16, 4, top_p=1)), ("k50p95", dict(top_k=50, top_p=0.95, temperature=0.8)),
                      ("k7000", dict(top_k=7000)), ("q5p90", dict(min_p=0.05, top_p=0.9))):
        log(f"[verify] 80 x {V} {dtype} {kind} {name}")
        wide = {k: v.repeat(times) if torch.is_tensor(v) else v for k, v in prm.items()}
        o = _run(many, wide)
        first = type(o)(o.tokens[:16], o.accepted[:16], o.logprobs[:16])
        _compare(few, first, prm)
        for k in range(1, times):
            s = slice(16 * k, 16 * k + 16)
            assert torch.equal(o.tokens[s], o.tokens[:16]) and torch.equal(o.accepted[s], o.accepted[:16])
            assert torch.equal(o.logprobs[s], o.logprobs[:16])
        _same_as_in_small_batches(many, wide, o, 16)


@pytest.mark.parametrize("kind", ["flat", "peaked"])
@pytest.mark.parametrize("V,dtype", [(2097152, "f32"), (2097153, "bf16"), (2097153, "f32"), (1 << 23, "bf16"),
                                     (1 << 24, "f32")])
def test_more_than_256_rows_of_any_length(V, dtype, kind):
    """All sequences read one target row and one row of the draft (strides of
    0); numbers and parameters are their own."""
    import torch
    B, K = 90, 1   # 270 rows, 1024 threads a row in batches of 30 sequences
    g = torch.Generator().manual_seed(V + len(kind))
    z = 1.6 * torch.randn(V, generator=g) if kind == "flat" else 2.5 * torch.randn(V, generator=g)
    if kind == "peaked":
        z[torch.randint(0, V, (40,), generator=g)] = 12.0 + 8.0 * torch.rand(40, generator=g)
    d = z + 0.5 * torch.randn(V, generator=g)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    t, q = z.to(dt).cuda().expand(B, K + 1, V), d.to(dt).cuda().expand(B, K, V)
    x = d.topk(20).indices[torch.randint(0, 20, (B, K), generator=g)].cuda()
    lens = torch.randint(0, K + 1, (B,), generator=g).cuda()
    u, ud = torch.rand(B, K, generator=g).cuda(), 0.999 * torch.rand(B, generator=g).cuda()
    case = t, q, x, lens, u, ud
    for name, prm in (("plain", {}), ("top_p", _per_sequence(B, 5, top_p=1)), ("q1p90", dict(min_p=0.01, top_p=0.9)),
                      ("mixed", _per_sequence(B, 6, temperature=1, top_k=1, top_p=1, min_p=1))):
        log(f"[verify] 90 x {V} {dtype} {kind} {name}")
        o = _run(case, prm)
        assert o.tokens[torch.arange(B), o.accepted.cpu()].ge(0).all()
        _same_as_in_small_batches(case, prm, o, 30)
        if V == 2097153:
            s = slice(7, 9)
            small, sprm = _part(case, prm, s)
            _compare(small, type(o)(o.tokens[s], o.accepted[s], o.logprobs[s]), sprm)
