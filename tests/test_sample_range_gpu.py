"""Token sampling over the whole range of vocabularies (up to 2^24, where the
candidates of a row are gathered in more than one batch of groups) and on rows
with more candidates than the list holds, against the fp64 definition.

Tokens have to be equal: the kernels' weights are off by a relative 2^-38.8 and
half a unit of 2^-38 of the largest, so a sum over a row moves by less than
1e-10 of itself; random numbers closer than 1e-9 to the end of their token's
interval, or a nucleus that close to its border, would be ambiguous, and the
seeded inputs stay clear of that (checked).
"""
import numpy as np
import pytest

from gpu_util import log
from oracle import head as O

NAMES = ("temperature", "top_k", "top_p", "min_p")
DEFAULT = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)


def by_weight(z):
    """Indices by descending logit, equal ones ascending."""
    return np.argsort(-z, kind="stable")


def reference(z, u, order, temperature, top_k, top_p, min_p):
    """oracle.head.sample_row of a row without NaN, vectorised, sums in
    extended precision: (token, logprob, distance from the nearest border).
    The parameters are what the library takes them as, fp32 numbers."""
    temperature, top_p, min_p = (float(np.float32(v)) for v in (temperature, top_p, min_p))
    if temperature == 0.0:
        return int(z.argmax()), 0.0, 1.0
    w = np.exp((z - z.max()) / temperature)
    clear = 1.0
    if top_k > 0:
        order = order[:top_k]
    if top_p < 1.0:
        c = np.cumsum(w[order], dtype=np.longdouble)
        c /= c[-1]
        n = int(np.searchsorted(c, np.longdouble(top_p)))
        clear = float(min(abs(c[n] - top_p), abs((c[n - 1] if n else 0.0) - top_p)))
        order = order[:n + 1]
    kept = np.sort(order)
    kept = kept[(w[kept] >= min_p) & (w[kept] > 0.0)]
    c = np.cumsum(w[kept], dtype=np.longdouble)
    s = c[-1]
    c /= s
    j = min(int(np.searchsorted(c, np.longdouble(u), side="right")), kept.size - 1)
    lo = float(u - (c[j - 1] if j else -1.0))
    hi = float((c[j] if j + 1 < kept.size else 2.0) - u)
    return int(kept[j]), float(np.log(w[kept[j]] / s)), min(lo, hi, clear)


def rows(N, V, dtype, sd, seed, far=0.0):
    """Seeded normal logits of a standard deviation; `far` of the row (its
    front) lies 40 below, so the candidates are in its last groups."""
    import torch
    z = torch.from_numpy(np.random.default_rng(seed).normal(size=(N, V)) * sd)
    z[:, :int(far * V)] -= 40.0
    return z.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


def numbers(N, seed):
    import torch
    return torch.rand(N, generator=torch.Generator().manual_seed(seed))


# (N, V, dtype, sd, far, seed) with the parameters each is drawn with
LONG = [
    (2, 262145, "bf16", 1.6, 0.0, 1), (2, 300001, "f32", 1.6, 0.99, 2), (2, 600007, "bf16", 0.8, 0.0, 3),
    (1, (1 << 24) - 5, "f32", 1.6, 0.0, 4), (1, 1 << 24, "bf16", 1.6, 0.999, 5),
]
LONG_PARAMS = [dict(), dict(temperature=0.0), dict(top_k=50, top_p=0.95, temperature=0.8), dict(top_k=3000, top_p=0.8),
               dict(top_k=20000), dict(top_p=0.9), dict(top_p=0.3, temperature=0.7), dict(min_p=0.05),
               dict(min_p=0.002, top_p=0.9), dict(top_k=200, top_p=0.9, min_p=0.02, temperature=1.2)]

# more candidates than the list of 12288 (6144 from 257 rows on) holds
FLAT = [(1, 202048, "bf16", 0.8, 0.0, 6), (3, 202048, "f32", 0.8, 0.0, 7), (1, 202048, "bf16", 1.6, 0.0, 8),
        (260, 40001, "bf16", 0.8, 0.0, 9), (260, 65536, "f32", 0.3, 0.0, 10)]
FLAT_PARAMS = [dict(min_p=0.05), dict(top_p=0.9, temperature=1.5), dict(top_p=0.9), dict(min_p=0.05, temperature=2.0),
               dict(min_p=0.05, top_p=0.95), dict(top_k=13000, top_p=0.9), dict(top_k=30000, min_p=0.1)]


def test_vectorised_definition_is_the_oracles():
    for V, dtype in ((1, "f32"), (50, "bf16"), (3001, "f32"), (5000, "bf16")):
        z = rows(1, V, dtype, 1.6, V)[0].double().numpy()
        for i, prm in enumerate(LONG_PARAMS + FLAT_PARAMS):
            p = {**DEFAULT, **prm}
            u = float(numbers(1, 50 + i))
            want = O.sample_row(z, u, *(float(np.float32(p[n])) if n != "top_k" else p[n] for n in NAMES))
            got = reference(z, u, by_weight(z), **p)
            assert got[0] == want[0] and abs(got[1] - want[1]) < 1e-12, (V, prm)


@pytest.mark.gpu
@pytest.mark.usefixtures("require_gpu")
@pytest.mark.parametrize("shape", LONG + FLAT, ids=lambda s: "-".join(map(str, s)))
def test_sample_long_and_flat_rows(shape):
    import torch
    import linear_cross_entropy_gemm_amd as L
    N, V, dtype, sd, far, seed = shape
    zc, uc = rows(N, V, dtype, sd, seed, far), numbers(N, seed)
    z, u = zc.cuda(), uc.cuda()
    pick = {i: zc[i].double().numpy() for i in (range(N) if N < 10 else range(0, N, 97))}
    order = {i: by_weight(pick[i]) for i in pick}
    for prm in (LONG_PARAMS if shape in LONG else FLAT_PARAMS):
        log(f"[sample] {shape} {prm}")
        o = L.sample(z, u, **prm, logprobs=True)
        torch.cuda.synchronize()
        for i in pick:
            want, wl, border = reference(pick[i], float(uc[i]), order[i], **{**DEFAULT, **prm})
            assert border > 1e-9, (i, border)
            assert o.tokens[i].item() == want, (i, o.tokens[i].item(), want)
            got = o.logprobs[i].item()
            assert abs(got - wl) <= 2.0 ** -24 * abs(wl) + 1e-9, (i, got, wl)
