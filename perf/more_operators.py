"""The operators of a head that serves in small types, as they are measured:
RMS norm with the residual's addition (forward, backward, and with an 8-bit
output), products with 4-bit weights, and the verification of drafted tokens.

``run`` computes an operator in its plain form (elementary torch operations),
or with ``own`` set through this package's entry points.  ``exact`` computes
the same outputs from the definitions in 64 bits.

Small types are the block formats of the OCP Microscaling specification
(v1.0): 32 elements along a row share a scale, a power of two held as an
E8M0 exponent; the elements are E4M3 (8 bits) or E2M1 (4 bits).
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4, "mx8": 1}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decoded token's final norm, the residual stream updated on the way: latency
        {"name": "rms_fwd_token", "op": "rms_fwd", "rows": 1, "hidden": 6656, "dtype": "bf16", "wdtype": "bf16",
         "residual": True, "offset": 0.0, "pad": 0},
        # the final norm of a training step (8192 tokens), parameters kept in fp32
        {"name": "rms_fwd_train", "op": "rms_fwd", "rows": 8192, "hidden": 6656, "dtype": "bf16", "wdtype": "f32",
         "residual": True, "offset": 0.0, "pad": 0},
        # its backward pass, with the gradient that arrives on the residual stream
        {"name": "rms_bwd_train", "op": "rms_bwd", "rows": 8192, "hidden": 6656, "dtype": "bf16", "wdtype": "f32",
         "residual": True, "offset": 0.0, "pad": 0},
        # a ragged batch of valid tokens at an odd width in fp32, weights kept around zero
        {"name": "rms_bwd_ragged", "op": "rms_bwd", "rows": 4099, "hidden": 5003, "dtype": "f32", "wdtype": "f32",
         "residual": False, "offset": 1.0, "pad": 0},
        # the norm in front of 8-bit products over a whole prompt
        {"name": "rms_mx8_prompt", "op": "rms_mx8", "rows": 8192, "hidden": 7168, "dtype": "bf16", "wdtype": "bf16",
         "residual": True, "offset": 0.0, "pad": 0},
        # one decoded token's logits from 4-bit weights: the largest read of a decoding step
        {"name": "mx4_token", "op": "mx4", "rows": 1, "hidden": 6656, "vocab": 202048, "dtype": "bf16", "cap": 30.0},
        # four drafted tokens of one sequence and the one they follow, hidden states in 8 bits
        {"name": "mx4_draft", "op": "mx4", "rows": 5, "hidden": 7168, "vocab": 129280, "dtype": "mx8", "cap": 0.0},
        # the drafted tokens of 64 sequences
        {"name": "mx4_batch", "op": "mx4", "rows": 320, "hidden": 4096, "vocab": 128256, "dtype": "bf16", "cap": 0.0},
        # odd sizes in fp32
        {"name": "mx4_ragged", "op": "mx4", "rows": 33, "hidden": 1001, "vocab": 50001, "dtype": "f32", "cap": 0.0},
        # four drafted tokens of one sequence, usual serving parameters: latency
        {"name": "verify_token", "op": "verify", "seqs": 1, "drafted": 4, "vocab": 202048, "dtype": "bf16",
         "logits": "peaked", "params": "k50p95", "draft": "logits", "lens": "full", "pad": 0},
        # a serving batch, every sequence with parameters and a number of drafted tokens of its own
        {"name": "verify_batch", "op": "verify", "seqs": 64, "drafted": 4, "vocab": 129279, "dtype": "f32",
         "logits": "peaked", "params": "mixed", "draft": "logits", "lens": "ragged", "pad": 1},
        # long drafts without filters, from flat distributions
        {"name": "verify_flat", "op": "verify", "seqs": 32, "drafted": 7, "vocab": 202048, "dtype": "bf16",
         "logits": "flat", "params": "plain", "draft": "logits", "lens": "full", "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rms_fwd", "rms_bwd", "rms_mx8", "mx4", "mx4", "verify", "verify"])
    if op == "mx4":
        hidden = _log_int(rng, 32, 8192)
        vocab = min(_log_int(rng, 64, 202048), 202048 * 6656 // hidden)
        rows = min(_log_int(rng, 1, 512), max(1, 320 * 4096 * 128256 // (hidden * vocab)))
        return {"op": op, "rows": rows, "hidden": hidden, "vocab": vocab, "dtype": rng.choice(["bf16", "bf16", "f32", "mx8"]),
                "cap": rng.choice([0.0, 0.0, 30.0])}
    dtype = rng.choice(["bf16", "f32"])
    if op == "verify":
        vocab, drafted = _log_int(rng, 32, 202048), rng.choice([1, 2, 3, 4, 5, 7])
        most = 32 * 15 * 202048 * 2 // _ES[dtype]
        seqs = min(_log_int(rng, 1, 256), max(1, most // (vocab * (2 * drafted + 1))))
        return {"op": op, "seqs": seqs, "drafted": drafted, "vocab": vocab, "dtype": dtype,
                "logits": rng.choice(["peaked", "flat", "banned"]),
                "params": rng.choice(["plain", "greedy", "k50p95", "p90", "minp", "mixed"]),
                "draft": rng.choice(["logits", "logits", "none"]), "lens": rng.choice(["full", "ragged"]),
                "pad": rng.choice([0, 0, 1, 8])}
    hidden = _log_int(rng, 8, 16384)
    rows = min(_log_int(rng, 1, 32768), max(1, 8192 * 7168 // hidden * 2 // _ES[dtype]))
    return {"op": op, "rows": rows, "hidden": hidden, "dtype": dtype, "wdtype": rng.choice([dtype, "f32"]),
            "residual": rng.choice([True, False]), "offset": rng.choice([0.0, 1.0]), "pad": rng.choice([0, 0, 1, 8])}


# --------------------------------------------------------------------------
# the block formats
# --------------------------------------------------------------------------
def _exponents(amax, top, most):
    """E8M0 codes of the least power of two s for which amax / s is at most
    ``top`` = most / 2^ceil: from the exponent and the mantissa in [0.5, 1)."""
    mant, e = torch.frexp(amax)
    e = e - most + (mant > top).to(e.dtype)
    return torch.where(amax > 0, e + 127, 0).clamp(0, 254).to(torch.int32)


def _power(codes, dtype):
    return torch.ldexp(torch.ones((), dtype=dtype, device=codes.device), codes.to(torch.int32) - 127)


def _e2m1_codes(v):
    """Nearest E2M1 values, ties to the even code, as 4-bit codes."""
    a = v.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return c | ((v < 0) & (c > 0)).to(torch.uint8) << 3


def _mx4_weights(g, vocab, hidden):
    """Weights of a trained projection's scale, in the 4-bit format: rows of
    ``hidden`` elements, padded with zeros to whole steps of 128, two elements a
    byte (the first in the low half), and one scale for every 32."""
    kp = (hidden + 127) // 128 * 128
    data = torch.empty((vocab, kp // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((vocab, kp // 32), dtype=torch.uint8, device="cuda")
    per = max(1, (1 << 28) // kp)
    for i in range(0, vocab, per):
        n = min(per, vocab - i)
        w = torch.zeros((n, kp), device="cuda")
        w[:, :hidden] = torch.randn((n, hidden), device="cuda", generator=g)
        w *= 0.02 * (0.5 + torch.rand((n, 1), device="cuda", generator=g))
        b = w.view(n, kp // 32, 32)
        e = _exponents(b.abs().amax(2), 0.75, 3)
        c = _e2m1_codes(b / _power(e, torch.float32)[:, :, None]).view(n, kp // 2, 2)
        data[i:i + n] = c[:, :, 0] | c[:, :, 1] << 4
        scales[i:i + n] = e.to(torch.uint8)
    return data, scales.view(torch.float8_e8m0fnu)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(g, rows, hidden, dtype, pad):
    """Hidden states: unit-scale values, each row with a scale of its own, and a
    few channels that are much larger than the rest."""
    x = torch.randn((rows, hidden + pad), device="cuda", generator=g)
    x *= 0.5 + torch.rand((rows, 1), device="cuda", generator=g)
    big = torch.randint(0, hidden + pad, (max(1, hidden // 512),), device="cuda", generator=g)
    x[:, big] *= 8.0
    return x.to(dtype)[:, :hidden]


def _verify_inputs(g, case):
    B, K, V, pad = case["seqs"], case["drafted"], case["vocab"], case["pad"]
    z = torch.randn((B, K + 1, V + pad), device="cuda", generator=g)
    if case["logits"] == "flat":
        z *= 1.6          # 0.02 * sqrt(6656): the spread at initialisation
    else:
        z *= 2.5
        # about 48 tokens of a row (a quarter of a small vocabulary) stand out
        peak = torch.rand(z.shape, device="cuda", generator=g) < min(0.25, 48.0 / V)
        z = torch.where(peak, 6.0 + 8.0 * torch.rand(z.shape, device="cuda", generator=g), z)
    # the draft model comes near the target's logits
    d = z[:, :K] + 0.5 * torch.randn((B, K, V + pad), device="cuda", generator=g)
    if case["logits"] == "banned":
        # a grammar or a list of banned tokens leaves a part of the vocabulary
        ban = torch.rand((B, 1, V + pad), device="cuda", generator=g) < 0.7
        ban[:, :, 0] = False
        z, d = z.masked_fill(ban, float("-inf")), d.masked_fill(ban, float("-inf"))
    dt = _DT[case["dtype"]]
    s = {"target": z.to(dt)[:, :, :V]}
    # drawn among the draft's most likely tokens
    val, idx = d[:, :, :V].topk(min(V, 8 if case["params"] == "mixed" else 64), dim=2)
    gumbel = -torch.log(-torch.log(torch.rand(val.shape, device="cuda", generator=g).clamp(1e-9, 1 - 1e-7)))
    best = torch.zeros_like(val[:, :, :1], dtype=torch.int64) if case["params"] == "greedy" or case["draft"] == "none" \
        else (val + gumbel).argmax(2, keepdim=True)
    s["tokens"] = idx.gather(2, best)[:, :, 0].contiguous()
    s["draft"] = d.to(dt)[:, :, :V] if case["draft"] == "logits" else None
    s["lens"] = None
    if case["lens"] == "ragged":
        s["lens"] = torch.randint(0, K + 1, (B,), device="cuda", generator=g)
    s["u"] = torch.rand((B, K), device="cuda", generator=g)
    s["u_draw"] = torch.rand(B, device="cuda", generator=g)
    kind = case["params"]
    fixed = {"plain": (1.0, 0, 1.0, 0.0), "greedy": (0.0, 0, 1.0, 0.0), "k50p95": (0.8, 50, 0.95, 0.0),
             "p90": (1.0, 0, 0.9, 0.0), "minp": (1.0, 0, 1.0, 0.05)}
    if kind != "mixed":
        s["params"] = fixed[kind]
        return s
    temperature = 0.5 + torch.rand(B, device="cuda", generator=g)
    temperature[::7] = 0.0
    top_k = torch.tensor([0, 1, 40, 200], device="cuda")[torch.randint(0, 4, (B,), device="cuda", generator=g)]
    top_p = 0.5 + 0.5 * torch.rand(B, device="cuda", generator=g)
    top_p[::3] = 1.0
    min_p = 0.1 * torch.rand(B, device="cuda", generator=g)
    min_p[::2] = 0.0
    s["params"] = temperature, top_k, top_p, min_p
    return s


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "verify":
        return {"op": op, **_verify_inputs(g, case)}
    s = {"op": op}
    rows, hidden = case["rows"], case["hidden"]
    if op == "mx4":
        s["cap"], s["mult"], s["hidden"] = case["cap"], 0.5 if case["cap"] else 1.0, hidden
        s["w"], s["ws"] = _mx4_weights(g, case["vocab"], hidden)
        x = _rows(g, rows, hidden, torch.float32, 0)
        if case["dtype"] == "mx8":
            s["x"], s["xs"] = _plain_mx8(x)
        else:
            s["x"], s["xs"] = x.to(_DT[case["dtype"]]), None
        return s
    dt, wdt = _DT[case["dtype"]], _DT[case["wdtype"]]
    s["eps"], s["offset"] = 1e-6, case["offset"]
    s["x"] = _rows(g, rows, hidden, dt, case["pad"])
    s["w"] = (1.0 - case["offset"] + 0.2 * torch.randn(hidden, device="cuda", generator=g)).to(wdt)
    s["residual"] = None
    if op == "rms_bwd":
        s["dy"] = torch.randn((rows, hidden), device="cuda", generator=g).to(dt)
        s["ds"] = torch.randn((rows, hidden), device="cuda", generator=g).to(dt) if case["residual"] else None
        # the statistic that the forward pass kept
        s["rstd"] = torch.rsqrt(s["x"].double().square().mean(1) + s["eps"]).float()
    elif case["residual"]:
        s["residual"] = torch.randn((rows, hidden), device="cuda", generator=g).to(dt)
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _plain_rms(s):
    """y in fp32, the new residual stream (rounded to its type, then normed),
    and 1 / root mean square."""
    x = s["x"]
    res = None
    if s["residual"] is not None:
        x = res = (x.float() + s["residual"].float()).to(x.dtype)
    x = x.float()
    rstd = torch.rsqrt(x.square().mean(1) + s["eps"])
    return x * rstd[:, None] * (s["w"].float() + s["offset"]), res, rstd


def _plain_rms_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    xh = x * s["rstd"][:, None]
    g = dy * (s["w"].float() + s["offset"])
    dx = (g - xh * (g * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["ds"] is not None:
        dx = dx + s["ds"].float()
    return dx.to(s["x"].dtype), (dy * xh).sum(0).to(s["w"].dtype)


def _plain_mx8(y):
    """Rows in E4M3 with one scale for every 32 elements (the last block of a
    row may be shorter)."""
    M, H = y.shape
    nb = (H + 31) // 32
    b = torch.nn.functional.pad(y, (0, nb * 32 - H)).view(M, nb, 32)
    e = _exponents(b.abs().amax(2), 0.875, 9)
    q = (b / _power(e, torch.float32)[:, :, None]).reshape(M, nb * 32)[:, :H].contiguous()
    return q.to(torch.float8_e4m3fn), e.to(torch.uint8).view(torch.float8_e8m0fnu)


def _dequant4(data, scales, hidden, dtype):
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=dtype, device=data.device)
    w = torch.stack((table[(data & 15).int()], table[(data >> 4).int()]), 2).reshape(data.shape[0], -1)
    return (w.view(w.shape[0], -1, 32) * scales.to(dtype)[:, :, None]).reshape(w.shape)[:, :hidden]


def _dequant8(x, scales, dtype):
    return x.to(dtype) * scales.to(dtype).repeat_interleave(32, 1)[:, :x.shape[1]]


def _plain_mx4(s):
    x = s["x"].float() if s["xs"] is None else _dequant8(s["x"], s["xs"], torch.float32)
    z = torch.mm(x, _dequant4(s["w"], s["ws"], s["hidden"], torch.float32).t()) * s["mult"]
    if s["cap"]:
        z = s["cap"] * torch.tanh(z / s["cap"])
    return z.to(torch.bfloat16 if s["xs"] is not None else s["x"].dtype)


def _plain_dist(z, params):
    """The distribution that a row's token is drawn from (index order): softmax
    at a temperature, then top-k, top-p within it, min-p relative to the largest
    probability; all zero where nothing is left to draw."""
    z = z.double()
    z = torch.where(z.isnan(), float("-inf"), z)
    B, L, V = z.shape
    t, k, p, q = (v.double()[:, None, None] if torch.is_tensor(v)
                  else torch.full((1, 1, 1), float(v), device="cuda").double() for v in params)
    rank = torch.arange(V, device="cuda")
    zmax = z.amax(2, keepdim=True)
    first = torch.where(z == zmax, rank, V).amin(2, keepdim=True)
    w = torch.where(z == zmax, 1.0, torch.exp((z - zmax) / torch.where(t == 0.0, 1.0, t)))
    val, idx = torch.sort(z, dim=2, descending=True, stable=True)
    ws = torch.where((rank < k) | (k == 0), w.gather(2, idx), 0.0)
    cum = ws.cumsum(2)
    before = torch.cat((torch.zeros_like(cum[:, :, :1]), cum[:, :, :-1]), 2)
    ws = torch.where(((before < p * cum[:, :, -1:]) | (p >= 1.0)) & (ws >= q), ws, 0.0)
    w = torch.zeros_like(w).scatter_(2, idx, ws)
    w = torch.where(t == 0.0, (rank == first).double(), w)
    w = torch.where(zmax == float("-inf"), 0.0, w)
    return w / w.sum(2, keepdim=True).clamp(min=1e-300)


def _plain_verify(s):
    p = _plain_dist(s["target"], s["params"])
    x, (B, K), V = s["tokens"], s["tokens"].shape, p.shape[2]
    n = torch.full((B,), K, device="cuda") if s["lens"] is None else s["lens"]
    at = torch.arange(K + 1, device="cuda")
    drafted = (at[:K] < n[:, None])[:, :, None]
    if s["draft"] is None:
        q = torch.zeros_like(p[:, :K]).scatter_(2, x[:, :, None], 1.0)
    else:
        q = _plain_dist(s["draft"], s["params"])
    px, qx = p[:, :K].gather(2, x[:, :, None]), q.gather(2, x[:, :, None])
    ok = (s["u"].double()[:, :, None] * qx < px) & drafted
    acc = ok[:, :, 0].long().cumprod(1).sum(1)
    # the draft says nothing behind its end
    q = torch.cat((torch.where(drafted, q, 0.0), torch.zeros_like(p[:, :1])), 1)
    here = acc[:, None, None].expand(B, 1, V)
    pn, qn = p.gather(1, here)[:, 0], q.gather(1, here)[:, 0]
    r = (pn - qn).clamp(min=0.0)
    r = torch.where(r.sum(1, keepdim=True) > 0.0, r, pn)
    cum = r.cumsum(1)
    tok = (cum <= s["u_draw"].double()[:, None] * cum[:, -1:]).sum(1)
    tok = torch.minimum(tok, torch.where(r > 0.0, torch.arange(V, device="cuda"), 0).amax(1))
    tok = torch.where(cum[:, -1] > 0.0, tok, -1)
    out = torch.where(at < acc[:, None], torch.cat((x, x[:, :1]), 1), torch.where(at == acc[:, None], tok[:, None], -1))
    logp = torch.log(p.gather(2, out.clamp(min=0)[:, :, None]))[:, :, 0]
    return out, acc, torch.where(out >= 0, logp, float("-inf")).float()


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    op = s["op"]
    if own:
        import linear_cross_entropy_gemm_amd as L
        if op == "rms_fwd":
            o = L.rms_norm_fwd(s["x"], s["w"], s["eps"], residual=s["residual"], offset=s["offset"])
            return o.y, o.residual, o.rstd
        if op == "rms_bwd":
            o = L.rms_norm_bwd(s["dy"], s["x"], s["w"], s["rstd"], offset=s["offset"], grad_residual=s["ds"])
            return o.grad_x, o.grad_weight
        if op == "rms_mx8":
            o = L.rms_norm_mx8(s["x"], s["w"], s["eps"], residual=s["residual"], offset=s["offset"])
            return o.rows.data, o.rows.scales, o.residual
        if op == "mx4":
            x = s["x"] if s["xs"] is None else L.Mx8Rows(s["x"], s["xs"])
            return L.logits_mx4(x, L.Mx4Weight(s["w"], s["ws"], s["hidden"]), s["cap"], s["mult"])
        t, k, p, q = s["params"]
        o = L.verify(s["target"], s["tokens"], s["u"], s["u_draw"], draft_logits=s["draft"], draft_lens=s["lens"],
                     temperature=t, top_k=k, top_p=p, min_p=q, logprobs=True)
        return o.tokens, o.accepted, o.logprobs
    if op == "rms_fwd":
        y, res, rstd = _plain_rms(s)
        return y.to(s["x"].dtype), res, rstd
    if op == "rms_bwd":
        return _plain_rms_bwd(s)
    if op == "rms_mx8":
        y, res, _ = _plain_rms(s)
        return (*_plain_mx8(y), res)
    if op == "mx4":
        return _plain_mx4(s)
    return _plain_verify(s)


def work(case):
    op, es = case["op"], _ES[case["dtype"]]
    if op == "verify":
        rows = case["seqs"] * ((case["drafted"] + 1) + (case["drafted"] if case["draft"] == "logits" else 0))
        n = rows * case["vocab"]
        return {"bytes": n * es + case["seqs"] * (case["drafted"] + 1) * 24, "flops": 4 * n}
    rows, hidden = case["rows"], case["hidden"]
    n = rows * hidden
    if op == "mx4":
        blocks = (hidden + 31) // 32
        out = 2 if es < 4 else 4
        return {"bytes": case["vocab"] * blocks * 17 + n * es + rows * case["vocab"] * out,
                "flops": 2 * n * case["vocab"]}
    ws = _ES[case["wdtype"]] * hidden
    if op == "rms_bwd":
        return {"bytes": (4 if case["residual"] else 3) * n * es + 4 * rows + 2 * ws, "flops": 11 * n}
    res = 2 if case["residual"] else 0
    if op == "rms_mx8":
        return {"bytes": (1 + res) * n * es + n + rows * ((hidden + 31) // 32) + ws, "flops": 8 * n}
    return {"bytes": (2 + res) * n * es + 4 * rows + ws, "flops": 5 * n}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _exact_rms(s):
    x, f = s["x"].to(torch.float64), torch.float64
    res = None
    if s["residual"] is not None:
        res = x + s["residual"].to(f)
        x = res.to(s["x"].dtype).to(f)   # the stream as it is kept
    rstd = 1.0 / ((x ** 2).sum(1) / x.shape[1] + s["eps"]).sqrt()
    return (x * rstd.unsqueeze(1)) * (s["w"].to(f) + s["offset"]), res, rstd


def _exact_rms_bwd(s):
    f = torch.float64
    w, rstd = s["w"].to(f) + s["offset"], s["rstd"].to(f).unsqueeze(1)
    H = w.numel()
    dw = torch.zeros(H, dtype=f, device=w.device)
    dx = torch.empty(s["x"].shape, dtype=f, device=w.device)
    for i in range(0, dx.shape[0], 4096):
        xh = s["x"][i:i + 4096].to(f) * rstd[i:i + 4096]
        d = s["dy"][i:i + 4096].to(f)
        dw += (d * xh).sum(0)
        d = d * w
        dx[i:i + 4096] = rstd[i:i + 4096] * (d - xh * ((d * xh).sum(1, keepdim=True) / H))
    if s["ds"] is not None:
        dx += s["ds"].to(f)
    return dx, dw


def _exact_mx8(y):
    """Block by block: s = 2^ceil(log2(amax / 448)), elements rounded to steps of
    2^(exponent - 3), at least 2^-9."""
    M, H = y.shape
    full = torch.zeros((M, (H + 31) // 32 * 32), dtype=y.dtype, device=y.device)
    full[:, :H] = y
    full = full.reshape(M, -1, 32)
    amax = full.abs().max(2).values
    e = torch.ceil(torch.log2(amax / 448.0))
    e = torch.where(amax / torch.exp2(e) > 448.0, e + 1, e)
    e = torch.where(amax <= 448.0 * torch.exp2(e - 1), e - 1, e)
    scale = torch.exp2(torch.clamp(torch.where(amax > 0, e, -127.0), -127.0, 127.0))
    v = full / scale.unsqueeze(2)
    step = torch.exp2(torch.clamp(torch.floor(torch.log2(v.abs().clamp(min=1e-30))), min=-6.0) - 3.0)
    v = torch.round(v / step) * step
    return v.reshape(M, -1)[:, :H], scale


def _exact_mx4(s):
    x = s["x"].to(torch.float64)
    if s["xs"] is not None:
        x = _dequant8(s["x"], s["xs"], torch.float64)
    V = s["w"].shape[0]
    z = torch.empty((x.shape[0], V), dtype=torch.float64, device=x.device)
    mag = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device=x.device) / 2
    for i in range(0, V, 8192):
        c = s["w"][i:i + 8192]
        c = torch.stack((c & 15, c >> 4), dim=-1).flatten(1).long()
        w = mag[c & 7] * (1 - 2 * (c >> 3)).double()
        e = s["ws"][i:i + 8192].view(torch.uint8).double() - 127.0
        w = (w.unflatten(1, (-1, 32)) * torch.exp2(e).unsqueeze(2)).flatten(1)[:, :s["hidden"]]
        z[:, i:i + 8192] = x @ w.t()
    z *= s["mult"]
    return s["cap"] * torch.tanh(z / s["cap"]) if s["cap"] else z


def _exact_dist(z, t, k, p, q):
    """{index: probability} as two arrays, indices ascending."""
    live = np.flatnonzero(z > -np.inf)
    if live.size == 0:
        return live, np.zeros(0)
    top = z[live].max()
    if t == 0.0:
        return live[z[live] == top][:1], np.ones(1)
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
    return live, w / w.sum()


def _exact_verify(s):
    """Sequence by sequence, up to the first rejection."""
    B, K = s["tokens"].shape
    x, u, ud = (s[n].cpu().numpy().astype(np.float64 if n != "tokens" else np.int64) for n in ("tokens", "u", "u_draw"))
    lens = np.full(B, K) if s["lens"] is None else s["lens"].cpu().numpy()
    par = [v.cpu().numpy() if torch.is_tensor(v) else np.full(B, v, dtype=np.float32) for v in s["params"]]
    row = lambda t, b, i: t[b, i].float().cpu().numpy().astype(np.float64)  # noqa: E731
    V = s["target"].shape[2]
    tokens, acc = np.full((B, K + 1), -1), np.zeros(B, dtype=np.int64)
    logs = np.full((B, K + 1), -np.inf)
    for b in range(B):
        a = [float(v[b]) for v in par]
        for i in range(K + 1):
            p = np.zeros(V)
            at, pr = _exact_dist(row(s["target"], b, i), *a)
            p[at] = pr
            q = np.zeros(V)
            if i < lens[b]:
                if s["draft"] is None:
                    q[x[b, i]] = 1.0
                else:
                    at, pr = _exact_dist(row(s["draft"], b, i), *a)
                    q[at] = pr
                if u[b, i] * q[x[b, i]] < p[x[b, i]]:
                    tokens[b, i], logs[b, i] = x[b, i], math.log(p[x[b, i]])
                    continue
            acc[b] = i
            r = np.maximum(p - q, 0.0)
            r = r if r.sum() > 0.0 else p
            mass = np.cumsum(r)
            if mass[-1] > 0.0:
                j = min(int(np.searchsorted(mass, ud[b] * mass[-1], side="right")), int(np.flatnonzero(r)[-1]))
                tokens[b, i], logs[b, i] = j, math.log(p[j])
            break
    return tuple(torch.from_numpy(v).to(s["target"].device) for v in (tokens, acc, logs))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "verify":
        return _exact_verify(s)
    if op == "mx4":
        return _exact_mx4(s)
    if op == "rms_bwd":
        return _exact_rms_bwd(s)
    y, res, rstd = _exact_rms(s)
    return (y, res, rstd) if op == "rms_fwd" else (*_exact_mx8(y), res)
