"""fp64 definitions of the operators around the vocabulary projection: layer
norm and its gradients, and dropout from a counter-based generator.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Pinned by
``tests/test_head_oracle.py``: central differences for the gradients, the
published known answers for the generator.
"""
from __future__ import annotations

import numpy as np


def layer_norm(x, w, b, eps):
    """(y, mean, rstd) of rows x [M, H]; w, b [H] or None."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if w is not None:
        y = y * np.asarray(w, dtype=np.float64)
    if b is not None:
        y = y + np.asarray(b, dtype=np.float64)
    return y, mean, rstd


def layer_norm_grads(dy, x, w, mean, rstd):
    """(dx, dw, db) of sum(dy * y) for given row statistics."""
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    mean, rstd = np.asarray(mean, dtype=np.float64)[:, None], np.asarray(rstd, dtype=np.float64)[:, None]
    xh = (x - mean) * rstd
    g = dy if w is None else dy * np.asarray(w, dtype=np.float64)
    dx = rstd * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def philox4x32_10(ctr, key):
    """Philox4x32-10 (Salmon et al., SC 2011): ctr [..., 4] and key (2 words)
    of uint32 values -> [..., 4] words."""
    m = 0xFFFFFFFF
    c = [np.asarray(ctr)[..., i].astype(np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        hi, lo = np.uint64(32), np.uint64(m)
        c = [(b >> hi) ^ c[1] ^ np.uint64(k[0]), b & lo, (a >> hi) ^ c[3] ^ np.uint64(k[1]), a & lo]
        k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
    return np.stack(c, -1)


def dropout_keep(n, p, seed, offset):
    """Which of n elements survive: word i % 4 of counter (i // 4, offset)
    under the key `seed` is at least floor(p 2^32)."""
    blk = np.arange((n + 3) // 4, dtype=np.uint64)
    ctr = np.zeros((blk.size, 4), dtype=np.uint64)
    ctr[:, 0], ctr[:, 1] = blk & np.uint64(0xFFFFFFFF), blk >> np.uint64(32)
    ctr[:, 2], ctr[:, 3] = offset & 0xFFFFFFFF, (offset >> 32) & 0xFFFFFFFF
    words = philox4x32_10(ctr, (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF)).reshape(-1)[:n]
    return words >= np.uint64(int(p * 4294967296.0))


def dropout(x, p, seed, offset, residual=None):
    x = np.asarray(x, dtype=np.float64)
    keep = dropout_keep(x.size, p, seed, offset).reshape(x.shape)
    y = np.zeros_like(x)
    if p < 1.0:
        y[keep] = x[keep] / (1.0 - p)
    return y if residual is None else y + np.asarray(residual, dtype=np.float64)


def sample_row(z, u, t=1.0, k=0, p=1.0, q=0.0):
    """(token, logprob, border) of one row of logits: the definition step by
    step.  `border` is the distance of u from the nearest end of the token's
    interval, for tests that must stay clear of it."""
    z = np.asarray(z, dtype=np.float64).copy()
    z[np.isnan(z)] = -np.inf
    zm = z.max()
    if zm == -np.inf:
        return -1, -np.inf, 1.0
    if t == 0.0:
        return int(np.flatnonzero(z == zm)[0]), 0.0, 1.0
    with np.errstate(invalid="ignore"):
        w = np.where(z == zm, 1.0, np.exp((z - zm) / t))
    order = sorted(range(z.size), key=lambda i: (-z[i], i))
    if k > 0:
        order = order[:k]
    if p < 1.0:
        total, run, prefix = float(np.cumsum(w[order])[-1]), 0.0, []
        for i in order:
            prefix.append(i)
            run += w[i]
            if run >= p * total:
                break
        order = prefix
    kept = sorted(i for i in order if w[i] >= q and w[i] > 0.0)
    c = np.cumsum(w[kept])
    j = min(int(np.searchsorted(c, u * c[-1], side="right")), len(kept) - 1)
    lo, hi = (c[j - 1] if j else 0.0) / c[-1], c[j] / c[-1]
    border = min(u - lo if j else 1.0, hi - u if j + 1 < len(kept) else 1.0)
    return kept[j], float(np.log(w[kept[j]] / c[-1])), border


def row_distribution(z, t=1.0, k=0, p=1.0, q=0.0):
    """Probabilities [V] of a row of logits under the sampler's parameters (all
    zero where nothing can be drawn), as sample_row draws from them."""
    z = np.asarray(z, dtype=np.float64).copy()
    z[np.isnan(z)] = -np.inf
    out = np.zeros(z.size)
    zm = z.max()
    if zm == -np.inf:
        return out
    if t == 0.0:
        out[np.flatnonzero(z == zm)[0]] = 1.0
        return out
    with np.errstate(invalid="ignore"):
        w = np.where(z == zm, 1.0, np.exp((z - zm) / t))
    order = np.lexsort((np.arange(z.size), -z))
    if k > 0:
        order = order[:k]
    if p < 1.0:
        run = np.cumsum(w[order])
        order = order[:np.flatnonzero(run >= p * run[-1])[0] + 1]
    kept = order[w[order] >= q]
    out[kept] = w[kept]
    return out / out.sum()


def verify(target, draft, x, length, u, u_draw, params, draft_params=None):
    """(tokens, accepted, logprobs, borders) of one sequence: target [K + 1, V]
    logits, draft [K, V] logits or None, drafted tokens x [K].  `borders` are
    the distances from where a decision turns, of u q from p relative to them
    and of u_draw from the ends of its token's interval in weight of r, and the
    whole weight of r."""
    K, V = len(x), target.shape[1]
    tokens, logs, border, turn = np.full(K + 1, -1), np.full(K + 1, -np.inf), 1.0, 1.0
    length = min(max(int(length), 0), K)
    for i in range(K + 1):
        p, q = row_distribution(target[i], *params), np.zeros(V)
        if i < length:
            if draft is not None:
                q = row_distribution(draft[i], *(params if draft_params is None else draft_params))
            elif 0 <= x[i] < V:
                q[x[i]] = 1.0
            if 0 <= x[i] < V and 0.0 <= u[i] < 1.0:
                if p[x[i]] > 0.0:
                    border = min(border, abs(u[i] * q[x[i]] - p[x[i]]) / max(u[i] * q[x[i]], p[x[i]]))
                if u[i] * q[x[i]] < p[x[i]]:
                    tokens[i], logs[i] = x[i], np.log(p[x[i]])
                    continue
        r = np.maximum(p - q, 0.0)
        r = r if r.sum() > 0.0 else p
        c = np.cumsum(r)
        if c[-1] > 0.0 and 0.0 <= u_draw < 1.0:
            kept = np.flatnonzero(r)
            j = min(int(np.searchsorted(c, u_draw * c[-1], side="right")), kept[-1])
            lo = c[j] - r[j]
            turn = min(u_draw * c[-1] - lo if j != kept[0] else 1.0,
                       c[j] - u_draw * c[-1] if j != kept[-1] else 1.0)
            tokens[i], logs[i] = j, np.log(p[j])
        return tokens, i, logs, (border, turn, c[-1])


def rms_norm(s, w, offset, eps):
    """(y, rstd) of rows s [M, H]; w [H] or None."""
    s = np.asarray(s, dtype=np.float64)
    rstd = 1.0 / np.sqrt((s ** 2).mean(1) + eps)
    y = s * rstd[:, None]
    return (y if w is None else y * (np.asarray(w, dtype=np.float64) + offset)), rstd


def rms_norm_grads(dy, s, w, offset, rstd, ds=None):
    """(dx, dw) of sum(dy * y) + sum(ds * s) for given row statistics."""
    dy, s = np.asarray(dy, dtype=np.float64), np.asarray(s, dtype=np.float64)
    rstd = np.asarray(rstd, dtype=np.float64)[:, None]
    xh = s * rstd
    g = dy if w is None else dy * (np.asarray(w, dtype=np.float64) + offset)
    dx = rstd * (g - xh * (g * xh).mean(1, keepdims=True))
    if ds is not None:
        dx = dx + np.asarray(ds, dtype=np.float64)
    return dx, (dy * xh).sum(0)


E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values():
    """The 128 non-negative codes' values (code 127 is NaN): 4 exponent bits of
    bias 7, 3 mantissa bits, subnormal steps of 2^-9."""
    c = np.arange(128)
    e, m = c >> 3, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[127] = np.nan
    return v


def mx_quantize(y, values):
    """Blocks of 32 along the rows of y [M, H]: (codes into `values` with the
    sign in the bit above, scale exponents).  The scale is the least power of
    two, at least 2^-127, under which the block's magnitudes fit the largest
    value; elements go to the nearest one, ties to the even code."""
    y = np.asarray(y, dtype=np.float64)
    M, H = y.shape
    nb = (H + 31) // 32
    full = np.zeros((M, nb * 32))
    full[:, :H] = y
    blocks = full.reshape(M, nb, 32)
    values = values[~np.isnan(values)]
    top, amax = values[-1], np.abs(blocks).max(2)
    e = np.full(amax.shape, -127, dtype=np.int64)
    for x in range(-126, 128):
        e = np.where(amax > top * 2.0 ** (x - 1), x, e)
    v = np.abs(blocks) / 2.0 ** e[:, :, None].astype(np.float64)
    hi = np.clip(np.searchsorted(values, v, side="left"), 0, values.size - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = values[hi] - v, v - values[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where((blocks < 0) & (code > 0), code | 1 << int(np.log2(values.size + 1)), code)
    return code.reshape(M, nb * 32)[:, :H], e
