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
