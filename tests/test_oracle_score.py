"""Pins of the scoring and cache oracle: library routines, finite differences, hand-made records."""
import numpy as np
import pytest
import torch

from oracle import score as o


def rows(B=5, V=37, seed=0):
    r = np.random.default_rng(seed)
    return r.standard_normal((B, V)) * 3, r.integers(0, V, B)


@pytest.mark.parametrize("T", [1.0, 0.5, 3.0])
def test_score_is_torchs(T):
    x, tok = rows()
    logprob, entropy, logq, q = o.score(x, tok, T)
    d = torch.distributions.Categorical(logits=torch.tensor(x) / T)
    assert np.allclose(logprob, d.log_prob(torch.tensor(tok)).numpy(), rtol=1e-13)
    assert np.allclose(entropy, d.entropy().numpy(), rtol=1e-13)


def test_gradient_is_autograds_and_a_difference():
    x, tok = rows()
    r = np.random.default_rng(1)
    a, b = r.standard_normal(5), r.standard_normal(5)
    T = np.array([1.0, 0.5, 2.0, 1.5, 0.7])
    lp, ent, logq, q = o.score(x, tok, T)
    dx = o.score_gradient(logq, q, ent, tok, a, b, T)
    t = torch.tensor(x, requires_grad=True)
    ls = torch.log_softmax(t / torch.tensor(T)[:, None], 1)
    lpt = ls[torch.arange(5), torch.tensor(tok)]
    ((torch.tensor(a) * lpt).sum() - (torch.tensor(b)[:, None] * ls.exp() * ls).sum()).backward()
    assert np.allclose(dx, t.grad.numpy(), rtol=1e-12, atol=1e-14)

    def value(y):
        p, h, _, _ = o.score(y, tok, T)
        return (a * p + b * h).sum()

    for i, j in ((0, 3), (2, tok[2]), (4, 36)):
        e = np.zeros_like(x)
        e[i, j] = 1e-5
        assert abs((value(x + e) - value(x - e)) / 2e-5 - dx[i, j]) < 1e-8


def test_special_rows():
    inf, nan = np.inf, np.nan
    x = np.array([[-inf, 1.0, -inf, 1.0], [-inf] * 4, [inf, 0.0, inf, 1.0], [nan, 2.0, -inf, nan], [0.0, 0, 0, 0]])
    lp, ent, logq, q = o.score(x, np.array([1, 0, 2, 1, 7]))
    assert np.isclose(lp[0], -np.log(2)) and np.isclose(ent[0], np.log(2))
    assert np.isnan(lp[1]) and np.isnan(ent[1])
    assert np.isclose(lp[2], -np.log(2)) and np.isclose(ent[2], np.log(2))
    assert lp[3] == 0 and ent[3] == 0
    assert np.isnan(lp[4]) and np.isclose(ent[4], np.log(4))
    lp, ent, _, _ = o.score(x, np.zeros(5, int), 1.0, np.zeros(5, bool))
    assert (lp == 0).all() and (ent == 0).all()
    assert o.alternatives([1.0, 3.0, -inf, 3.0, nan], 4).tolist() == [1, 3, 0, -1]
    assert o.alternatives([0.0, -0.0, 0.0], 2).tolist() == [0, 1]


def test_cache_record_by_hand():
    # 2 bits short of a word: K = 3, V = 5 (3 bits an id), 4 bits a logit: levels 14, top 7, low 0, step 0.5
    rec = o.cache_pack([[4, 0, 9]], [[7.0, 0.0, 3.6]], 5, 4)
    assert o.cache_words(3, 5, 4) == 4 and rec.shape == (1, 4)
    assert rec[0, :2].view(np.float32).tolist() == [7.0, 0.5]
    assert rec[0, 2] == (0 | 14 << 4 | 7 << 8)  # (7 - 3.6) * 2 = 6.8 -> 7
    assert rec[0, 3] == (4 | 0 << 3 | 7 << 6)   # an id outside [0, 5) is 7
    ids, z = o.cache_unpack(rec, 3, 5, 4)
    assert ids.tolist() == [[4, 0, -1]] and z.tolist() == [[7.0, 0.0, 3.5]]


@pytest.mark.parametrize("K,V,bits", [(1, 1, 8), (31, 7, 4), (33, 8, 8), (100, 201088, 8), (70, 2 ** 30, 4)])
def test_cache_round_trip(K, V, bits):
    r = np.random.default_rng(K)
    ids = r.integers(0, V, (4, K))
    z = (r.standard_normal((4, K)) * 3).astype(np.float32)
    z[1, K // 2] = -np.inf
    z[2] = -np.inf
    got, back = o.cache_unpack(o.cache_pack(ids, z, V, bits), K, V, bits)
    assert (got == ids).all()
    for k in range(0, K, 32):
        part, b = z[:, k:k + 32], back[:, k:k + 32]
        assert ((b == -np.inf) == (part == -np.inf)).all()
        for t in range(4):
            f = part[t] > -np.inf
            if f.any():
                half = (part[t][f].max() - part[t][f].min()) / (2 ** bits - 2) / 2
                # half a step, and three float roundings of at most |top| + 2^bits steps
                assert np.abs(part[t][f] - b[t][f]).max() <= half + 2.0 ** -22 * np.abs(part[t][f]).max() + 2.0 ** -20 * half
                assert b[t][f].max() == part[t][f].max()


def test_cache_special_logits():
    inf, nan = np.inf, np.nan
    z = np.array([[10.0, 5998.0, -3.4e38], [1.0, nan, 2.0], [1.0, inf, 2.0]], dtype=np.float32)
    ids, back = o.cache_unpack(o.cache_pack(np.zeros((3, 3), int), z, 4, 8), 3, 4, 8)
    assert back[0].tolist() == [-inf, 5998.0, -inf]  # more than 4096 below
    assert np.isnan(back[1:]).all()
