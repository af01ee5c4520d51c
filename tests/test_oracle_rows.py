"""Pins of oracle/rows_oracle.py: hand-worked values, properties that hold by
definition, and a check of the distillation gradient against differences,
each where it can with a variant that must fail."""
import math

import numpy as np
import pytest

from oracle import rows_oracle as RO


def test_filters_on_a_worked_row():
    # weights 8, 4, 2, 1 (T = 1 / ln 2 turns the logits' steps into halvings)
    z, T = np.array([1.0, 3.0, 0.0, 2.0]), 1 / math.log(2)
    ids, p = RO.filtered(z, T)
    assert ids.tolist() == [1, 3, 0, 2] and np.allclose(p, np.array([8, 4, 2, 1]) / 15)
    assert RO.filtered(z, T, top_k=2)[0].tolist() == [1, 3]
    # sums before the entries: 0, 8, 12, 14 of 15
    assert RO.filtered(z, T, top_p=0.5)[0].tolist() == [1]
    assert RO.filtered(z, T, top_p=0.54)[0].tolist() == [1, 3]
    assert RO.filtered(z, T, top_p=0.81)[0].tolist() == [1, 3, 0]
    # after top-k = 3 the sum is 14: 8 < 0.6 * 14 but 12 >= 0.85 * 14
    assert RO.filtered(z, T, top_k=3, top_p=0.6)[0].tolist() == [1, 3]
    assert RO.filtered(z, T, top_k=3, top_p=0.85)[0].tolist() == [1, 3]
    assert RO.filtered(z, T, top_p=0.85)[0].tolist() == [1, 3, 0]   # over all 15, it is kept
    assert RO.filtered(z, T, min_p=0.2)[0].tolist() == [1, 3, 0]
    assert RO.filtered(z, T, min_p=0.26)[0].tolist() == [1, 3]
    assert RO.filtered(z, T, top_p=0.0)[0].tolist() == [1]
    assert RO.filtered(z, 0.0)[0].tolist() == [1]


def test_ties_go_to_the_lowest_index():
    z = np.array([1.0, 2.0, 2.0, 2.0, -0.0, 0.0])
    assert RO.row_order(z).tolist() == [1, 2, 3, 0, 4, 5]
    assert RO.filtered(z, 1.0, top_k=2)[0].tolist() == [1, 2]
    assert RO.sample(z, 1.0, np.full(6, 0.5))[0] == 1
    assert RO.top_logits(z, 3)[1].tolist() == [1, 2, 3]


def test_masked_entries_and_empty_rows():
    lowest = float(np.finfo(np.float32).min)
    z = np.array([np.nan, -np.inf, lowest, 0.0])
    assert RO.row_order(z).tolist() == [3, 2]
    assert RO.sample(np.array([np.nan, -np.inf]), 1.0, np.full(2, 0.5))[:2] == (-1, -math.inf)
    ids, p = RO.filtered(np.array([lowest, lowest]), 1.0)
    assert p.tolist() == [0.5, 0.5]
    val, idx, lse = RO.top_logits(z, 4)
    assert idx.tolist() == [3, 2, -1, -1] and val[2] == -np.inf and lse == 0.0


def test_draws_follow_the_distribution():
    rng = np.random.default_rng(1)
    z = rng.normal(0, 1, 6)
    ids, p = RO.filtered(z, 0.8, top_k=4)
    n = 20000
    u = rng.random((n, 6))
    got = np.bincount([RO.gumbel_draw(ids, p, u[i])[0] for i in range(n)], minlength=6)
    e = np.zeros(6)
    e[ids] = p * n
    assert got[e == 0].sum() == 0
    chi = lambda e: float(((got[ids] - e[ids]) ** 2 / e[ids]).sum())
    assert chi(e) < 16.27  # 3 degrees of freedom, 99.9 %
    flat = np.zeros(6)
    flat[ids] = n / 4
    assert chi(flat) > 16.27


def test_accept_is_greedy_verification_at_zero_temperature():
    from oracle import dflash_oracle as O
    rng = np.random.default_rng(2)
    for _ in range(20):
        z = rng.normal(0, 1, (5, 7)).astype(np.float32)
        draft = z.argmax(1)[:4].copy()
        draft[rng.integers(0, 4)] = rng.integers(0, 7)
        n, c, em, nx = RO.verify_accept_filtered(z, draft, 0.0, rng.random(4), rng.random(7))
        rn, rc, rem, rnx = O.verify_accept(z, draft)
        assert (n, c, nx) == (rn, rc, rnx) and em.tolist() == list(rem)


def test_accept_without_filters_is_the_temperature_accept():
    from oracle import dflash_oracle as O
    rng = np.random.default_rng(3)
    for _ in range(20):
        z = rng.normal(0, 2, (4, 9)).astype(np.float32)
        draft = z.argmax(1)[:3].astype(np.int32)
        ua, us = rng.random(3).astype(np.float32), rng.random(9).astype(np.float32)
        n, c, em, nx = RO.verify_accept_filtered(z, draft, 0.7, ua, us)
        rn, rc, rem, rnx, _ = O.verify_accept_sample(z, draft, 0.7, ua, us)
        assert (n, c, nx) == (rn, rc, rnx) and em.tolist() == list(rem)


def test_a_rejected_draft_is_never_drawn_and_a_missing_one_is_rejected():
    z = np.array([[0.0, 0.0, -np.inf], [1.0, 0.0, 0.0]])
    n, c, em, nx = RO.verify_accept_filtered(z, np.array([0]), 1.0, [0.9], np.full(3, 0.5))
    assert (n, c, em.tolist(), nx) == (0, 1, [1, -1], 1)
    n, c, em, nx = RO.verify_accept_filtered(z, np.array([-1]), 1.0, [0.0], np.full(3, 0.5))
    assert (n, c) == (0, 0)


def test_distill_worked_values():
    # uniform student over 4, teacher all on one token: ln 4; gradient q - p
    loss, g = RO.distill(np.zeros(4), [2.0], [1])
    assert abs(loss - math.log(4)) < 1e-15 and np.allclose(g, [0.25, -0.75, 0.25, 0.25])
    # the student equals the teacher: nothing to learn, with the rest too
    z = np.array([1.0, 2.0, 0.5, -1.0])
    loss, g = RO.distill(z, z[[1, 0]], [1, 0], t_lse=RO._lse(z))
    assert abs(loss) < 1e-12 and np.abs(g).max() < 1e-12
    # without the rest's entry the tokens outside are pushed down
    loss, g = RO.distill(z, z[[1, 0]], [1, 0])
    assert loss > 0.05 and g[2] > 0 and g[3] > 0


@pytest.mark.parametrize("rest", [False, True])
def test_distill_gradient_against_differences(rest):
    rng = np.random.default_rng(4)
    z, t, ids = rng.normal(0, 1, 9), rng.normal(0, 1, 4), np.array([7, -1, 2, 0])
    T = 1.7
    tl = RO._lse(t[ids >= 0] / T) + 0.2 if rest else None
    f = lambda z: RO.distill(z, t, ids, T, tl, 0.6)[0]
    g = RO.distill(z, t, ids, T, tl, 0.6)[1]
    h = 1e-5
    num = np.array([(f(z + h * e) - f(z - h * e)) / (2 * h) for e in np.eye(9)])
    assert np.abs(num - g).max() < 1e-9
    assert np.abs(num - RO.distill(z, t, ids, T, None if rest else 5.0, 0.6)[1]).max() > 1e-3


def test_distill_rows_left_out_and_refused():
    z = np.arange(4.0)
    for args in (([1.0], [-1]), ([-np.inf], [2])):
        loss, g = RO.distill(z, *args)
        assert loss == 0 and not g.any()
    assert RO.distill(z, [1.0], [0], weight=0.0)[0] == 0
    for ids in ([1, 1], [4, 0], [-2, 0]):
        loss, g = RO.distill(z, [1.0, 2.0], ids)
        assert math.isnan(loss) and not g.any()


def test_distill_ignores_a_rest_that_rounding_explains():
    # 30 allowed tokens, all listed, log-sum-exp in fp32: about half of the rows
    # leave a p_r above 0 that meets a student without the other tokens
    rng = np.random.default_rng(5)
    positive = 0
    for _ in range(50):
        t, z = np.full(100, -np.inf), np.full(100, -np.inf)
        at = rng.choice(100, 30, replace=False)
        t[at], z[at] = rng.normal(15, 3, 30), rng.normal(0, 1, 30)
        val, idx, lse = RO.top_logits(t, 64)
        lse = float(np.float32(lse))
        positive += np.exp(val - lse).sum() < 1
        whole, gw = RO.distill(z, val, idx)
        loss, g = RO.distill(z, val, idx, t_lse=lse)
        # sum p differs from 1 by 2^-19 at most, and ln p by as much
        assert abs(loss - whole) < 2.0 ** -19 * (2 + abs(whole)) and np.abs(g - gw).max() < 2.0 ** -18
        z[np.isinf(z)] = -1e9
        assert abs(RO.distill(z, val, idx, t_lse=lse)[0] - loss) < 1e-12
        z[np.abs(z) > 1e8] = -np.inf
        assert RO.distill(z, val, idx, t_lse=lse + 0.01)[0] == math.inf
    assert 5 < positive < 45


def test_distill_refuses_a_teacher_that_is_no_number():
    z = np.arange(4.0)
    for t, lse in (([1.0, math.nan], None), ([math.inf, 1.0], None), ([1.0, 2.0], math.nan), ([1.0, 2.0], math.inf)):
        loss, g = RO.distill(z, t, [1, 2], t_lse=lse)
        assert math.isnan(loss) and not g.any()
        assert RO.distill(z, t, [1, 2], t_lse=lse, weight=0.0)[0] == 0
    assert RO.distill(z, [1.0, math.nan], [1, -1])[0] > 0 and RO.distill(z, [math.nan], [-1], t_lse=math.nan)[0] == 0
