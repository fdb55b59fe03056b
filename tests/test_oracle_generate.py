"""Pins of the generation oracle (8-bit product, sampler) to cases fixed by hand and to
library routines."""
import numpy as np
import pytest
import torch

from oracle import generate as og


def test_quantize_by_hand():
    x = np.array([[127.0, -63.5, 0.4, 0.6], [0, 0, 0, 0], [1.0, np.nan, 2.0, 3.0], [np.inf, 1, 1, 1],
                  [254.0, 1.0, 3.0, -5.0]], dtype=np.float32)
    q, s = og.quantize_int8(x)
    assert q[0].tolist() == [127, -64, 0, 1]     # -63.5 / 1 rounds to even
    assert q[4].tolist() == [127, 0, 2, -2]      # 0.5, 1.5 and -2.5 round to even
    assert s[0] == np.float32(127) * (np.float32(1) / np.float32(127)) and s[1] == 0
    assert np.isnan(s[2]) and np.isnan(s[3])
    assert not q[1:4].any()


def test_product_matches_integers():
    rng = np.random.default_rng(0)
    a = rng.integers(-128, 128, (5, 48)).astype(np.int8)
    b = rng.integers(-128, 128, (7, 48)).astype(np.int8)
    y = og.int8_matmul(a, np.ones(5), b, np.ones(7))
    np.testing.assert_array_equal(y, a.astype(np.int64) @ b.astype(np.int64).T)
    y2 = og.int8_matmul(a, np.arange(5.0), b, np.full(7, 0.5))
    np.testing.assert_allclose(y2, y * np.arange(5.0)[:, None] * 0.5)


def test_full_draw_inverts_the_cdf():
    rng = np.random.default_rng(1)
    row = rng.standard_normal(50).astype(np.float32)
    p = torch.softmax(torch.tensor(row, dtype=torch.float64), 0).numpy()
    c = np.cumsum(p)
    for v in (0, 7, 31, 49):
        u = np.float32(c[v] - 0.5 * p[v])
        found = og.sample_row(row, u)
        assert list(found) == [v]
        assert found[v] == pytest.approx((np.log(p[v]),) * 2, abs=1e-6)


def test_filters_by_hand():
    # probabilities 0.5, 0.25, 0.125, 0.125 at ids 2, 0, 1, 3 (a tie of ids 1 and 3)
    row = np.log(np.array([0.25, 0.125, 0.5, 0.125])).astype(np.float32)

    def keep(**kw):
        a = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
        a.update(kw)
        sure, may = og.kept_ids(row, **a, tol=1e-9)
        return np.flatnonzero(sure).tolist(), np.flatnonzero(may).tolist()

    assert keep() == ([0, 1, 2, 3],) * 2
    assert keep(top_k=3) == ([0, 1, 2],) * 2           # the tie keeps the lower id
    assert keep(top_p=0.6) == ([0, 2],) * 2
    assert keep(top_p=0.0) == ([2],) * 2
    assert keep(min_p=0.4) == ([0, 2],) * 2
    assert keep(min_p=2.0) == ([2],) * 2
    assert keep(temperature=0.0) == ([2],) * 2
    assert keep(top_k=2, top_p=0.7) == ([0, 2],) * 2    # 2/3 < 0.7 of the two kept
    assert keep(top_k=2, top_p=0.6) == ([2],) * 2       # 2/3 >= 0.6
    assert og.sample_row(row, 0.99, temperature=0.0) == {2: (0.0, 0.0)}


def test_rows_with_infinities():
    assert list(og.sample_row(np.full(5, -np.inf), 0.3)) == [-1]
    assert list(og.sample_row(np.array([np.nan, -np.inf, 1.0]), 0.9)) == [2]
    both = np.array([1.0, np.inf, 3.0, np.inf])
    assert list(og.sample_row(both, 0.25)) == [1] and list(og.sample_row(both, 0.75)) == [3]


@pytest.mark.parametrize("k,p", [(0, 0.9), (10, 1.0), (10, 0.7)])
def test_matches_a_sorted_softmax(k, p):
    rng = np.random.default_rng(5)
    row = (3 * rng.standard_normal(200)).astype(np.float32)
    sure, may = og.kept_ids(row, 1.0, k, p, 0.0, 1e-9)
    assert (sure == may).all()
    val, idx = torch.sort(torch.tensor(row, dtype=torch.float64), descending=True)
    n = k or 200
    prob = torch.softmax(val[:n], 0)
    n_keep = n if p >= 1 else int((prob.cumsum(0) - prob < p).sum())
    assert sorted(idx[:n_keep].tolist()) == np.flatnonzero(sure).tolist()


def test_planted_mistakes_are_seen():
    """The comparison used on the GPU's tokens refuses draws with a filter left out, the strict
    inequality of the draw reversed, or the draw taken in ranked order."""
    rng = np.random.default_rng(6)
    row = (2 * rng.standard_normal(300)).astype(np.float32)
    z, w = og.sample_weights(row, 1.0)
    order = og.ranked(row)
    us = rng.random(200)
    wrong = {"no top_k": 0, "no top_p": 0, "ranked order": 0}
    for u in us:
        ok = og.sample_row(row, u, 1.0, 20, 0.8, 0.0)
        sure, _ = og.kept_ids(row, 1.0, 20, 0.8, 0.0)
        wrong["no top_k"] += list(og.sample_row(row, u, 1.0, 0, 0.8, 0.0, 0.0))[0] not in ok
        wrong["no top_p"] += list(og.sample_row(row, u, 1.0, 20, 1.0, 0.0, 0.0))[0] not in ok
        c = np.cumsum(w[order] * sure[order])
        wrong["ranked order"] += int(order[np.flatnonzero(c > u * c[-1])[0]]) not in ok
    assert all(n > 50 for n in wrong.values()), wrong
