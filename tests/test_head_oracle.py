"""Pins of the fp64 definitions in ``oracle/head.py`` (CPU)."""
import numpy as np
import pytest

from oracle import head as O


def test_philox_known_answers():
    """The generator's published known answers (zero, all-ones and pi words)."""
    cases = [
        ([0, 0, 0, 0], [0, 0], [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]),
        ([0xffffffff] * 4, [0xffffffff] * 2, [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]),
        ([0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344], [0xa4093822, 0x299f31d0],
         [0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1]),
    ]
    for ctr, key, want in cases:
        got = O.philox4x32_10(np.array(ctr, dtype=np.uint64), key)
        assert [int(v) for v in got] == want


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout_keep_rate(p):
    keep = O.dropout_keep(200001, p, (7 << 32) | 5, (3 << 32) | 1)
    # five standard deviations of a binomial share
    assert abs(keep.mean() - (1.0 - p)) <= 5.0 * np.sqrt(p * (1.0 - p) / keep.size)


def test_dropout_masks_differ_by_seed_and_offset():
    base = O.dropout_keep(4096, 0.5, 1, 2)
    for seed, off in [(2, 2), (1, 3), (1 | 1 << 32, 2), (1, 2 | 1 << 32)]:
        other = O.dropout_keep(4096, 0.5, seed, off)
        assert 0.4 < (base == other).mean() < 0.6


@pytest.mark.parametrize("M,H", [(3, 7), (5, 1), (1, 33)])
def test_layer_norm_gradients_against_differences(M, H):
    """Central differences of sum(dy * y): h = 1e-5 leaves h^2 = 1e-10 of the
    third derivative and 1e-16 / h = 1e-11 of rounding."""
    r = np.random.default_rng(3)
    x, dy = r.normal(size=(M, H)) * 2 + 1, r.normal(size=(M, H))
    w, b, eps, h = r.normal(size=H), r.normal(size=H), 0.1, 1e-5

    def f(x_, w_, b_):
        return float((dy * O.layer_norm(x_, w_, b_, eps)[0]).sum())

    _, mean, rstd = O.layer_norm(x, w, b, eps)
    dx, dw, db = O.layer_norm_grads(dy, x, w, mean, rstd)
    for _ in range(4):
        vx, vw, vb = r.normal(size=(M, H)), r.normal(size=H), r.normal(size=H)
        num = (f(x + h * vx, w + h * vw, b + h * vb) - f(x - h * vx, w - h * vw, b - h * vb)) / (2 * h)
        ana = float((dx * vx).sum() + (dw * vw).sum() + (db * vb).sum())
        assert abs(num - ana) <= 1e-7 * (1.0 + abs(ana))


def test_layer_norm_closed_form():
    y, mean, rstd = O.layer_norm([[1.0, 3.0]], [2.0, 2.0], [0.5, 0.5], 3.0)
    assert mean[0] == 2.0 and rstd[0] == 0.5 and y.tolist() == [[-0.5, 1.5]]


def test_sample_row_by_hand():
    """Weights 1, 1/2, 1/4, 1/4 (base-2 logits at t = 1 / ln 2)."""
    z, t = np.array([-1.0, 0.0, -2.0, -2.0]), 1.0 / np.log(2.0)
    pick = lambda u, **kw: O.sample_row(z, u, t, **kw)[0]
    # index order: token 0 holds [0, 1/4), 1 [1/4, 3/4), 2 [3/4, 7/8), 3 the rest
    assert [pick(u) for u in (0.0, 0.24, 0.26, 0.74, 0.76, 0.87, 0.88, 0.99)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert abs(O.sample_row(z, 0.0, t)[1] - np.log(0.25)) < 1e-15
    assert pick(0.99, k=1) == 1 and pick(0.99, k=2) == 1 and pick(0.99, k=3) == 2   # ties: lowest index stays
    assert pick(0.99, p=0.5) == 1 and pick(0.01, p=0.51) == 0 and pick(0.99, p=0.8) == 2 and pick(0.99, p=0.9) == 3
    assert pick(0.01, q=0.6) == 1 and pick(0.01, q=0.5) == 0 and pick(0.99, q=0.2) == 3
    # top-p counts within the top-k: 2/3 of (1, 1/2) is the first alone
    assert pick(0.01, k=2, p=0.66) == 1 and pick(0.01, k=2, p=0.67) == 0
    assert O.sample_row(z, 0.5, 0.0)[:2] == (1, 0.0)
    assert O.sample_row([-np.inf] * 3, 0.5)[:2] == (-1, -np.inf)
    assert O.sample_row([np.inf, 0.0, np.inf], 0.6)[0] == 2
    assert O.sample_row([np.nan, 0.0], 0.0)[0] == 1


def test_sample_row_frequencies():
    """Over evenly spaced random numbers a token is drawn in proportion to its
    probability, to one draw."""
    r = np.random.default_rng(9)
    z = r.normal(size=20)
    n = 4000
    drawn = np.bincount([O.sample_row(z, (i + 0.5) / n, 0.7)[0] for i in range(n)], minlength=20)
    w = np.exp(z / 0.7)
    assert np.abs(drawn - n * w / w.sum()).max() <= 1.0
