"""Pins of the fp64 definition of draft verification."""
import numpy as np

from oracle import head as O


def test_distribution_is_what_sample_row_draws_from():
    g = np.random.default_rng(1)
    z = g.normal(size=40) * 2
    z[3], z[5] = -np.inf, np.nan
    for prm in [(1.0, 0, 1.0, 0.0), (0.7, 5, 1.0, 0.0), (1.0, 0, 0.6, 0.0), (1.0, 20, 0.9, 0.1), (0.0, 0, 1.0, 0.0)]:
        p = O.row_distribution(z, *prm)
        assert abs(p.sum() - 1) < 1e-12
        c = np.cumsum(p)
        for u in g.random(50):
            tok, lp, border = O.sample_row(z, u, *prm)
            if border > 1e-9:
                assert tok == int(np.searchsorted(c, u, side="right")) and abs(lp - np.log(p[tok])) < 1e-12
    assert not O.row_distribution(np.full(4, -np.inf)).any()


def test_by_hand():
    # p = (1/2, 1/4, 1/4), q = (1/4, 1/2, 1/4)
    t, d = np.log([[0.5, 0.25, 0.25]] * 2), np.log([[0.25, 0.5, 0.25]])
    one = (1.0, 0, 1.0, 0.0)
    tok, n, lp, _ = O.verify(t, d, [1], 1, [0.49], 0.6, one)      # 0.49 / 2 < 1/4
    assert tok.tolist() == [1, 1] and n == 1 and np.allclose(lp, np.log([0.25, 0.25]))
    tok, n, lp, _ = O.verify(t, d, [1], 1, [0.51], 0.99, one)     # what is left is token 0 alone
    assert tok.tolist() == [0, -1] and n == 0 and lp[1] == -np.inf
    tok, n, _, _ = O.verify(t, d, [1], 0, [0.0], 0.99, one)       # no draft: from p
    assert tok.tolist() == [2, -1] and n == 0
    tok, n, _, _ = O.verify(t, None, [0], 1, [0.51], 0.49, one)   # a certain token: p without it
    assert tok.tolist() == [1, -1] and n == 0
    tok, n, _, _ = O.verify(t, d, [7], 1, [0.0], 0.0, one)
    assert tok.tolist() == [0, -1] and n == 0
    t[0] = -np.inf
    assert O.verify(t, d, [1], 1, [0.0], 0.0, one)[0].tolist() == [-1, -1]


def test_first_token_is_distributed_as_the_target():
    """Exactly: the probability of each outcome, integrated over u and u_draw."""
    g = np.random.default_rng(2)
    for prm, dprm in [((1.0, 0, 1.0, 0.0), (1.0, 0, 1.0, 0.0)), ((0.7, 4, 0.9, 0.0), (1.3, 0, 0.8, 0.0))]:
        t, d = g.normal(size=(2, 6)) * 2, g.normal(size=(1, 6)) * 2
        p, q = O.row_distribution(t[0], *prm), O.row_distribution(d[0], *dprm)
        got = np.zeros(6)
        m = 400
        for x in np.flatnonzero(q):
            a = min(1.0, p[x] / q[x])   # accepted for u below a
            for u, weight in ((0.5 * a, a), (0.5 * (1 + a), 1 - a)):
                if weight < 1e-12:
                    continue
                for ud in (np.arange(m) + 0.5) / m:
                    tok, n, _, _ = O.verify(t, d, [x], 1, [u], ud, prm, dprm)
                    got[tok[0]] += q[x] * weight / m
        assert np.abs(got - p).max() < 6 / m


def test_sampling_and_verification_together_by_frequency():
    g = np.random.default_rng(3)
    t, d, one = g.normal(size=(3, 5)), g.normal(size=(2, 5)), (1.0, 0, 1.0, 0.0)
    N, counts = 6000, np.zeros((5, 5))
    p = [O.row_distribution(r) for r in t]
    for _ in range(N):
        x = [O.sample_row(r, g.random())[0] for r in d]
        tok, n, _, _ = O.verify(t, d, x, 2, g.random(2), g.random(), one)
        if n >= 1:
            counts[tok[0], tok[1]] += 1
    # given the first is accepted, the second follows p_1 whatever the first was
    for row in counts:
        if row.sum() > 300:
            assert np.abs(row / row.sum() - p[1]).max() < 4 * np.sqrt(0.25 / row.sum())
