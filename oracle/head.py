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
