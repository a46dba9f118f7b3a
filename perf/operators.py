"""The operators around the vocabulary head, as they are measured: layer norm
(forward and backward), dropout whose mask is regenerated instead of stored,
and drawing a token from the logits.

``run`` computes an operator in its plain form (elementary torch operations),
or with ``own`` set through this package's entry points.  ``exact`` computes
the same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decoded token's final norm in front of the vocabulary projection: latency
        {"name": "ln_fwd_token", "op": "ln_fwd", "rows": 1, "hidden": 6656, "dtype": "bf16", "wdtype": "bf16",
         "pad": 0},
        # the final norm of a training step (8192 tokens), parameters kept in fp32
        {"name": "ln_fwd_train", "op": "ln_fwd", "rows": 8192, "hidden": 6656, "dtype": "bf16", "wdtype": "f32",
         "pad": 0},
        # an odd width in fp32, rows taken from a wider buffer
        {"name": "ln_fwd_ragged", "op": "ln_fwd", "rows": 1537, "hidden": 1001, "dtype": "f32", "wdtype": "f32",
         "pad": 3},
        # its backward pass, with the reduction of the weight and bias gradients over 8192 rows
        {"name": "ln_bwd_train", "op": "ln_bwd", "rows": 8192, "hidden": 6656, "dtype": "bf16", "wdtype": "f32",
         "pad": 0},
        # a ragged batch of valid tokens at an odd width
        {"name": "ln_bwd_ragged", "op": "ln_bwd", "rows": 4099, "hidden": 5003, "dtype": "f32", "wdtype": "f32",
         "pad": 0},
        # the backward pass of a long-context step (32768 tokens)
        {"name": "ln_bwd_long", "op": "ln_bwd", "rows": 32768, "hidden": 7168, "dtype": "bf16", "wdtype": "bf16",
         "pad": 0},
        # the smallest parity workload's residual branch: latency
        {"name": "dropout_small", "op": "dropout_fwd", "rows": 256, "hidden": 128, "dtype": "f32", "p": 0.1,
         "residual": True},
        # residual + dropout(branch) of a training step, forward and backward
        {"name": "dropout_train", "op": "dropout_train", "rows": 8192, "hidden": 6656, "dtype": "bf16", "p": 0.1,
         "residual": True},
        # a long-context batch, no residual
        {"name": "dropout_long", "op": "dropout_fwd", "rows": 32768, "hidden": 7168, "dtype": "bf16", "p": 0.2,
         "residual": False},
        # one decoded token, usual serving parameters, peaked logits
        {"name": "sample_token", "op": "sample", "rows": 1, "vocab": 202048, "dtype": "bf16", "logits": "peaked",
         "params": "k50p95", "pad": 0},
        # a serving batch, every row with parameters of its own, fp32 logits with a padded row stride
        {"name": "sample_batch", "op": "sample", "rows": 64, "vocab": 129279, "dtype": "f32", "logits": "peaked",
         "params": "mixed", "pad": 1},
        # a large batch of a freshly initialised model: nearly flat logits, the nucleus holds tens of thousands
        {"name": "sample_flat", "op": "sample", "rows": 256, "vocab": 202048, "dtype": "bf16", "logits": "flat",
         "params": "p90", "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "dropout_fwd", "dropout_train", "sample", "sample"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "sample":
        vocab = _log_int(rng, 32, 202048)
        rows = min(_log_int(rng, 1, 1024), max(1, 256 * 202048 // vocab * 2 // _ES[dtype]))
        return {"op": op, "rows": rows, "vocab": vocab, "dtype": dtype,
                "logits": rng.choice(["peaked", "flat", "banned"]),
                "params": rng.choice(["plain", "greedy", "k50p95", "k1000", "p90", "minp", "mixed"]),
                "pad": rng.choice([0, 0, 1, 8])}
    hidden = _log_int(rng, 8, 16384)
    rows = min(_log_int(rng, 1, 32768), max(1, 32768 * 7168 // hidden * 2 // _ES[dtype]))
    case = {"op": op, "rows": rows, "hidden": hidden, "dtype": dtype}
    if op.startswith("ln"):
        case["wdtype"] = rng.choice([dtype, "f32"])
        case["pad"] = rng.choice([0, 0, 1, 8])
    else:
        # dropout_train moves up to four times the bytes of a forward pass
        if op == "dropout_train":
            case["rows"] = max(1, rows // 2)
        case["p"] = rng.choice([0.05, 0.1, 0.2, 0.5])
        case["residual"] = rng.choice([True, False])
    return case


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(g, rows, hidden, dtype, pad):
    """Hidden states: unit-scale values, each row with a scale and offset of its
    own, and a few channels that are much larger than the rest."""
    x = torch.randn((rows, hidden + pad), device="cuda", generator=g)
    x *= 0.5 + torch.rand((rows, 1), device="cuda", generator=g)
    x += 0.3 * torch.randn((rows, 1), device="cuda", generator=g)
    big = torch.randint(0, hidden + pad, (max(1, hidden // 512),), device="cuda", generator=g)
    x[:, big] *= 8.0
    return x.to(dtype)[:, :hidden]


def _logits(g, case):
    N, V = case["rows"], case["vocab"]
    z = torch.randn((N, V + case["pad"]), device="cuda", generator=g)
    if case["logits"] == "flat":
        z *= 1.6          # 0.02 * sqrt(6656): the spread at initialisation
    else:
        z *= 2.5
        # about 48 tokens of a row (a quarter of a small vocabulary) stand out
        peak = torch.rand(z.shape, device="cuda", generator=g) < min(0.25, 48.0 / V)
        z = torch.where(peak, 6.0 + 8.0 * torch.rand(z.shape, device="cuda", generator=g), z)
    if case["logits"] == "banned":
        # a grammar or a list of banned tokens leaves a part of the vocabulary
        z.masked_fill_(torch.rand(z.shape, device="cuda", generator=g) < 0.7, float("-inf"))
        z[:, 0] = 0.0
    return z.to(_DT[case["dtype"]])[:, :V]


def _params(g, case):
    N = case["rows"]
    kind = case["params"]
    fixed = {"plain": (1.0, 0, 1.0, 0.0), "greedy": (0.0, 0, 1.0, 0.0), "k50p95": (0.8, 50, 0.95, 0.0),
             "k1000": (1.2, 1000, 1.0, 0.0), "p90": (1.0, 0, 0.9, 0.0), "minp": (1.0, 0, 1.0, 0.05)}
    if kind != "mixed":
        return fixed[kind]
    temperature = 0.5 + torch.rand(N, device="cuda", generator=g)
    temperature[::7] = 0.0
    top_k = torch.randint(0, 4, (N,), device="cuda", generator=g)
    top_k = torch.tensor([0, 1, 40, 200], device="cuda")[top_k]
    top_p = 0.5 + 0.5 * torch.rand(N, device="cuda", generator=g)
    top_p[::3] = 1.0
    min_p = 0.1 * torch.rand(N, device="cuda", generator=g)
    min_p[::2] = 0.0
    return temperature, top_k, top_p, min_p


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op == "sample":
        s["z"] = _logits(g, case)
        s["u"] = torch.rand(case["rows"], device="cuda", generator=g)
        s["params"] = _params(g, case)
        return s
    dt = _DT[case["dtype"]]
    rows, hidden = case["rows"], case["hidden"]
    if op.startswith("ln"):
        wdt = _DT[case["wdtype"]]
        s["eps"] = 1e-5
        s["x"] = _rows(g, rows, hidden, dt, case["pad"])
        s["w"] = (1.0 + 0.2 * torch.randn(hidden, device="cuda", generator=g)).to(wdt)
        s["b"] = (0.1 * torch.randn(hidden, device="cuda", generator=g)).to(wdt)
        if op == "ln_bwd":
            s["dy"] = torch.randn((rows, hidden), device="cuda", generator=g).to(dt)
            # the statistics that the forward pass kept
            x = s["x"].double()
            mean = x.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = torch.rsqrt((x - mean[:, None]).square().mean(1) + s["eps"]).float()
        return s
    s["p"] = case["p"]
    s["seed"] = seed * 7919 + 12345
    s["offset"] = seed + (1 << 33)
    s["x"] = torch.randn((rows, hidden), device="cuda", generator=g).to(dt)
    s["residual"] = torch.randn((rows, hidden), device="cuda", generator=g).to(dt) if case["residual"] else None
    if op == "dropout_train":
        s["x"].requires_grad_()
        if case["residual"]:
            s["residual"].requires_grad_()
        s["dy"] = torch.randn((rows, hidden), device="cuda", generator=g).to(dt)
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _plain_ln_fwd(s):
    x = s["x"].float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = torch.rsqrt(d.square().mean(1) + s["eps"])
    y = d * rstd[:, None] * s["w"].float() + s["b"].float()
    return y.to(s["x"].dtype), mean, rstd


def _plain_ln_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["w"].float()
    dx = (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
    wdt = s["w"].dtype
    return dx.to(s["x"].dtype), (dy * xh).sum(0).to(wdt), dy.sum(0).to(wdt)


def _plain_words(n, seed, offset):
    """Random words of elements 0..n-1: Philox4x32-10 (Salmon et al. 2011) on
    the counter (element / 4, offset) under the key ``seed``."""
    m = 0xFFFFFFFF
    blk = torch.arange((n + 3) // 4, device="cuda", dtype=torch.int64)
    c0, c1 = blk & m, blk >> 32
    c2 = torch.full_like(blk, offset & m)
    c3 = torch.full_like(blk, (offset >> 32) & m)
    k0, k1 = seed & m, (seed >> 32) & m
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & m) ^ c1 ^ k0, b & m, ((a >> 32) & m) ^ c3 ^ k1, a & m
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    return torch.stack((c0, c1, c2, c3), 1).reshape(-1)[:n]


def _plain_dropout(s, x, residual):
    keep = (_plain_words(x.numel(), s["seed"], s["offset"]) >= int(s["p"] * 2.0 ** 32)).reshape(x.shape)
    y = torch.where(keep, x.detach().float() * (1.0 / (1.0 - s["p"])), 0.0)
    if residual is not None:
        y = residual.detach().float() + y
    return y.to(x.dtype)


def _plain_sample(s):
    z = s["z"].double()
    z = torch.where(z.isnan(), float("-inf"), z)
    N, V = z.shape
    t, k, p, q = (v[:, None].double() if torch.is_tensor(v) else torch.full((N, 1), float(v), device="cuda",
                                                                           dtype=torch.float64)
                  for v in s["params"])
    if not torch.is_tensor(s["params"][2]):
        p = p.float().double()
    if not torch.is_tensor(s["params"][3]):
        q = q.float().double()
    if not torch.is_tensor(s["params"][0]):
        t = t.float().double()
    rank = torch.arange(V, device="cuda")[None, :]
    zmax = z.amax(1, keepdim=True)
    first = torch.where(z == zmax, rank, V).amin(1)
    greedy = t == 0.0
    w = torch.where(z == zmax, 1.0, torch.exp((z - zmax) / torch.where(greedy, 1.0, t)))
    val, idx = torch.sort(z, dim=1, descending=True, stable=True)
    ws = w.gather(1, idx)
    keep = (rank < k) | (k == 0)
    ws = torch.where(keep, ws, 0.0)
    cum = ws.cumsum(1)
    before = torch.cat((torch.zeros((N, 1), device="cuda", dtype=torch.float64), cum[:, :-1]), 1)
    keep = keep & ((before < p * cum[:, -1:]) | (p >= 1.0)) & (ws >= q)
    wf = torch.zeros_like(w).scatter_(1, idx, torch.where(keep, ws, 0.0))
    cum = wf.cumsum(1)
    total = cum[:, -1:]
    tok = (cum <= s["u"][:, None].double() * total).sum(1)
    last = torch.where(wf > 0, rank, 0).amax(1)
    tok = torch.minimum(tok, last)
    tok = torch.where(greedy[:, 0], first, tok)
    logprob = torch.log(wf.gather(1, tok[:, None]) / total)[:, 0]
    logprob = torch.where(greedy[:, 0], 0.0, logprob)
    none = zmax[:, 0] == float("-inf")
    return torch.where(none, -1, tok), torch.where(none, float("-inf"), logprob).float()


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    op = s["op"]
    if own:
        import linear_cross_entropy_gemm_amd as L
        if op == "ln_fwd":
            o = L.layer_norm_fwd(s["x"], s["w"], s["b"], s["eps"])
            return o.y, o.mean, o.rstd
        if op == "ln_bwd":
            o = L.layer_norm_bwd(s["dy"], s["x"], s["w"], s["mean"], s["rstd"])
            return o.grad_x, o.grad_weight, o.grad_bias
        if op == "dropout_fwd":
            return L.dropout(s["x"], s["p"], s["seed"], s["offset"], residual=s["residual"])
        if op == "dropout_train":
            y = L.dropout(s["x"], s["p"], s["seed"], s["offset"], residual=s["residual"])
            leaves = (s["x"],) if s["residual"] is None else (s["x"], s["residual"])
            return (y.detach(), *torch.autograd.grad(y, leaves, s["dy"]))
        t, k, p, q = s["params"]
        o = L.sample(s["z"], s["u"], temperature=t, top_k=k, top_p=p, min_p=q, logprobs=True)
        return o.tokens, o.logprobs
    if op == "ln_fwd":
        return _plain_ln_fwd(s)
    if op == "ln_bwd":
        return _plain_ln_bwd(s)
    if op == "dropout_fwd":
        return _plain_dropout(s, s["x"], s["residual"])
    if op == "dropout_train":
        y = _plain_dropout(s, s["x"], s["residual"])
        dx = _plain_dropout(s, s["dy"], None)
        return (y, dx) if s["residual"] is None else (y, dx, s["dy"])
    return _plain_sample(s)


def work(case):
    op, es = case["op"], _ES[case["dtype"]]
    if op == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * es + case["rows"] * 16, "flops": 4 * n}
    n = case["rows"] * case["hidden"]
    if op == "ln_fwd":
        return {"bytes": 2 * n * es + 8 * case["rows"] + 2 * case["hidden"] * _ES[case["wdtype"]], "flops": 8 * n}
    if op == "ln_bwd":
        return {"bytes": 3 * n * es + 8 * case["rows"] + 3 * case["hidden"] * _ES[case["wdtype"]], "flops": 16 * n}
    per = 3 if case["residual"] else 2
    if op == "dropout_train":
        per += 2
    return {"bytes": per * n * es, "flops": (2 if case["residual"] else 1) * n + (n if op == "dropout_train" else 0)}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _exact_ln(s, backward):
    x = s["x"].to(torch.float64)
    H = x.shape[1]
    w = s["w"].to(torch.float64)
    if not backward:
        mean = x.sum(1) / H
        var = ((x - mean.unsqueeze(1)) ** 2).sum(1) / H
        rstd = 1.0 / (var + s["eps"]).sqrt()
        return (x - mean.unsqueeze(1)) * (w * rstd.unsqueeze(1)) + s["b"].to(torch.float64), mean, rstd
    xh = (x - s["mean"].to(torch.float64).unsqueeze(1)).mul_(s["rstd"].to(torch.float64).unsqueeze(1))
    del x
    dy = s["dy"].to(torch.float64)
    db = dy.sum(0)
    dw = torch.zeros(H, dtype=torch.float64, device=dy.device)
    dx = torch.empty_like(dy)
    for i in range(0, dy.shape[0], 4096):
        a, b = dy[i:i + 4096], xh[i:i + 4096]
        dw += (a * b).sum(0)
        g = a * w
        inner = (g * b).sum(1, keepdim=True) / H
        dx[i:i + 4096] = s["rstd"][i:i + 4096].to(torch.float64).unsqueeze(1) * (g - g.sum(1, keepdim=True) / H
                                                                                 - b * inner)
    return dx, dw, db


def _exact_keep(n, seed, offset, p):
    """Kept elements 0..n-1, word by word with numpy's unsigned integers."""
    keep = np.empty(n, dtype=bool)
    lim = np.uint64(int(math.floor(p * 4294967296.0)))
    mask, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    for lo in range(0, n, 1 << 24):
        hi = min(n, lo + (1 << 24))
        ctr = np.arange(lo // 4, (hi + 3) // 4, dtype=np.uint64)
        x = [ctr & mask, ctr >> sh, np.full_like(ctr, offset & 0xFFFFFFFF), np.full_like(ctr, (offset >> 32) & 0xFFFFFFFF)]
        key = [seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF]
        for _ in range(10):
            u, v = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
            x = [(v >> sh) ^ x[1] ^ np.uint64(key[0]), v & mask, (u >> sh) ^ x[3] ^ np.uint64(key[1]), u & mask]
            key = [(key[0] + 0x9E3779B9) % 4294967296, (key[1] + 0xBB67AE85) % 4294967296]
        keep[lo:hi] = (np.stack(x, 1).reshape(-1) >= lim)[:hi - lo]
    return keep


def _exact_dropout(s):
    x = s["x"].detach()
    if x.numel() > 60_000_000:
        return None
    keep = torch.from_numpy(_exact_keep(x.numel(), s["seed"], s["offset"], s["p"])).to(x.device).reshape(x.shape)
    factor = keep.to(torch.float64) / (1.0 - s["p"])
    y = x.to(torch.float64) * factor
    if s["residual"] is not None:
        y = y + s["residual"].detach().to(torch.float64)
    if s["op"] == "dropout_fwd":
        return y
    dx = s["dy"].to(torch.float64) * factor
    return (y, dx) if s["residual"] is None else (y, dx, s["dy"].to(torch.float64))


def _exact_sample(s):
    z_all = s["z"].float().cpu().numpy().astype(np.float64)
    u = s["u"].double().cpu().numpy()
    N = z_all.shape[0]
    par = [v.cpu().numpy() if torch.is_tensor(v) else np.full(N, v, dtype=np.float32) for v in s["params"]]
    tokens, logs = np.empty(N, dtype=np.int64), np.empty(N, dtype=np.float64)
    for r in range(N):
        z = z_all[r]
        t, k, p, q = (float(v[r]) for v in par)
        live = np.flatnonzero(z > -np.inf)
        if live.size == 0:
            tokens[r], logs[r] = -1, -np.inf
            continue
        top = z[live].max()
        if t == 0.0:
            tokens[r], logs[r] = live[z[live] == top][0], 0.0
            continue
        if k > 0 or p < 1.0:
            order = live[np.argsort(-z[live], kind="stable")]
            if k > 0:
                order = order[:int(k)]
            w = np.exp((z[order] - top) / t)
            if p < 1.0:
                mass = np.cumsum(w)
                order = order[:int(np.searchsorted(mass, p * mass[-1], side="left")) + 1]
            live = np.sort(order)
        w = np.exp((z[live] - top) / t)
        live, w = live[w >= q], w[w >= q]
        mass = np.cumsum(w)
        j = min(int(np.searchsorted(mass, u[r] * mass[-1], side="right")), live.size - 1)
        tokens[r], logs[r] = live[j], math.log(w[j] / mass[-1])
    return torch.from_numpy(tokens).to(s["z"].device), torch.from_numpy(logs).to(s["z"].device)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        return _exact_sample(s)
    if case["op"].startswith("ln"):
        return _exact_ln(s, case["op"] == "ln_bwd")
    return _exact_dropout(s)
