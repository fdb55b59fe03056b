"""Scores and gradients from hidden states at temperatures far from 1, against the float64 oracle.

Hidden states and head hold multiples of 1/16 and 1/32, so that every logit and every partial sum of it is a whole number of
1/512 below 2^24 of them: the tensor cores' logits are exact, and no tolerance below is divided by the temperature.

Tolerances.  A weight is 2^a with a = (s - m) log2(e) / tau: the difference is exact, the constant and the product round
(2^-23 |a| ln 2, at most 2^-22 ln V where q counts), the exponential is off by 2^-22.  fp32 sums lose 2^-24 at each
addition: V / 32 of them in a row, 16 in a chunk and across splits.  That is tol(V), of the sum and of log q;
what log q itself is large in rounds relatively (2^-22).
"""
import math

import numpy as np
import pytest
import torch

from oracle import score as oracle

pytestmark = pytest.mark.gpu

LOW = [1e-1, 1e-2, 1e-3, 1e-4, 1e-5, 1e-6]


@pytest.fixture(scope="module")
def fkl(cuda_device):
    from lm_head_top_tcgen05_gb300 import build

    build.build()
    import lm_head_top_tcgen05_gb300 as m

    return m


def tol(V):
    return 2.0 ** -22 * (4 + math.log(V)) + (V / 32 + 16) * 2.0 ** -24


def make(T, d, V, seed):
    """Exact logits up to about 40; half of the vocabulary twice, so that the likeliest token mostly shares its
    logit; half of the tokens the likeliest."""
    g = torch.Generator().manual_seed(seed)
    H = torch.randint(-128, 129, (T, d), generator=g).float() / 16
    W = torch.randint(-16, 17, (V, d), generator=g).float() / 32
    W[V // 2:V // 2 * 2] = W[:V // 2]
    x = H.double() @ W.double().t()
    tok = torch.where(torch.rand(T, generator=g) < 0.5, x.argmax(1), torch.randint(0, V, (T,), generator=g))
    assert (H.bfloat16().float() == H).all() and (W.bfloat16().float() == W).all()
    return H.bfloat16().cuda(), W.bfloat16().cuda(), tok.cuda(), x.numpy()


def check_scores(x, tok, tau, lp, ent):
    V = x.shape[1]
    want_lp, want_ent, logq, q = oracle.score(x, tok.cpu().numpy(), float(np.float32(tau)))
    lp, ent = lp.detach().cpu().double().numpy(), ent.detach().cpu().double().numpy()
    assert (lp <= 0).all() and (ent >= 0).all()
    assert (np.abs(lp - want_lp) <= tol(V) + 2.0 ** -22 * np.abs(want_lp)).all(), np.abs(lp - want_lp).max()
    # entropy = E[-log q]: the error of log q, and that of the weights times the spread of log q around it
    assert (np.abs(ent - want_ent) <= tol(V) * (4 + 2 * math.log(V))).all(), np.abs(ent - want_ent).max()
    return logq, q, want_ent


@pytest.mark.parametrize("tau", [1.0, *LOW, 1e-9, 1e-20, 1e-35, 1e4, 1e36, 3e38])
@pytest.mark.parametrize("T,V", [(70, 32), (300, 1504), (70, 20000), (70, 1), (5, 33), (300, 1505), (70, 20001)])
def test_scores(fkl, T, V, tau):
    H, W, tok, x = make(T, 64, V, seed=V)
    lp, ent = fkl.fused_logprobs(H, W, tok, tau=tau)
    check_scores(x, tok, tau, lp, ent)
    if V == 1:
        assert (lp == 0).all() and (ent == 0).all()


@pytest.mark.parametrize("T", [5, 300])
def test_not_finite_logits(fkl, T):
    """What a hidden state of 2^127 makes of a head with signs: -inf has no weight, +inf and NaN make the row NaN."""
    H, W, tok, _ = make(T, 64, 1505, seed=4)
    W[:, 0] = 0.0
    W[3:40, 0], W[200, 0] = -8.0, -8.0
    tok[:] = 1
    want = fkl.fused_logprobs(H, W, tok)
    H[:, 0] = 0.0
    H[2, 0] = 2.0 ** 127
    lp, ent = fkl.fused_logprobs(H, W, tok)
    x = H.cpu().double().numpy() @ W.cpu().double().numpy().T
    x[2, np.abs(x[2]) > 3e38] = -np.inf
    e_lp, e_ent, _, _ = oracle.score(x, tok.cpu().numpy())
    assert abs(lp[2].item() - e_lp[2]) < 1e-4 and abs(ent[2].item() - e_ent[2]) < 1e-4
    W[300, 0] = 8.0
    lp, ent = fkl.fused_logprobs(H, W, tok)
    assert lp[2].isnan() and ent[2].isnan() and torch.isfinite(lp[:2]).all() and torch.isfinite(lp[3:]).all()
    assert torch.isfinite(want[0]).all()


def check_gradients(x, H, W, tok, tau, a, b, logq, q, ent, got, half):
    H, W = H.float().cpu().double().numpy(), W.float().cpu().double().numpy()
    a, b, tau = a.cpu().double().numpy(), b.cpu().double().numpy(), float(np.float32(tau))
    dS = oracle.score_gradient(logq, q, ent, tok.cpu().numpy(), a, b, tau)
    lq = np.where(q > 0, np.abs(logq), 0)
    terms = (np.abs(a)[:, None] + np.abs(b)[:, None] * (lq + ent[:, None] + 1)) / tau
    # q's relative error is log q's; dS is rounded to bf16 (2^-8) but where the token is; there a (1 - q) / tau is a
    # difference in fp32; products are summed in fp32, 16 deep
    room = q * terms * (4 * tol(x.shape[1]) + 2.0 ** -22 * lq) + 2.0 ** -8 * np.abs(dS)
    rows = np.arange(len(a))
    t = tok.cpu().numpy()
    room[rows, t] += 2.0 ** -22 * terms[rows, t] - 2.0 ** -8 * np.abs(dS[rows, t])
    room += 2.0 ** -18 * np.abs(dS)
    for g, want, lim in zip(got, (dS @ W, dS.T @ H), (room @ np.abs(W), room.T @ np.abs(H))):
        g = g.float().cpu().double().numpy()
        lim = lim + (2.0 ** -8 if half else 2.0 ** -22) * np.abs(want) + 1e-30
        assert (np.abs(g - want) <= lim).all(), (np.abs(g - want) / lim).max()


@pytest.mark.parametrize("tau", [1.0, *LOW])
@pytest.mark.parametrize("T,V", [(5, 33), (300, 1505)])
def test_gradients(fkl, T, V, tau):
    H, W, tok, x = make(T, 64, V, seed=V + 1)
    g = torch.Generator().manual_seed(3)
    a, b = torch.randn(T, generator=g).cuda(), torch.randn(T, generator=g).cuda() * 0.3
    Hl, Wl = H.clone().requires_grad_(), W.clone().requires_grad_()
    lp, ent = fkl.fused_logprobs(Hl, Wl, tok, tau=tau)
    logq, q, want_ent = check_scores(x, tok, tau, lp, ent)
    got = torch.autograd.grad((lp, ent), (Hl, Wl), (a, b))
    check_gradients(x, H, W, tok, tau, a, b, logq, q, want_ent, got, True)


@pytest.mark.parametrize("tau", [1.0, 1e-3, 1e-6])
def test_explicit_gradients(fkl, tau):
    """The explicit calls hand the row's statistics on; from lse alone a row whose lse no longer tells q is NaN."""
    T, V = 300, 1505
    H, W, tok, x = make(T, 64, V, seed=9)
    a, b = torch.randn(T).cuda(), torch.randn(T).cuda() * 0.3
    stats = torch.empty(T, 2, device="cuda")
    lp, ent, lse = fkl.logprob_forward(H, W, tok, tau=tau, stats=stats)
    logq, q, want_ent = check_scores(x, tok, tau, lp, ent)
    want = torch.logsumexp(torch.tensor(x) / float(np.float32(tau)), 1)
    assert ((lse.cpu().double() - want).abs() <= tol(V) + 2.0 ** -22 * want.abs()).all()
    # the reference is a logit at most 10 binary orders below the row's largest, and the sum is the one above it
    m, log_sum = stats.cpu().double().unbind(1)
    top = torch.tensor(x).amax(1)
    assert ((m <= top) & (top - m <= 10 * math.log(2) * tau + 1e-9)).all()
    assert ((m / float(np.float32(tau)) + log_sum - want).abs() <= tol(V) + 2.0 ** -22 * want.abs()).all()
    got = fkl.logprob_backward(H, W, tok, None, lp, ent, lse, a, b, tau, stats=stats)
    check_gradients(x, H, W, tok, tau, a, b, logq, q, want_ent, got, False)
    plain = fkl.logprob_backward(H, W, tok, None, lp, ent, lse, a, b, tau)
    off = lse.abs() > 2 ** 15
    assert (tau < 1e-4) == bool(off.all()) and plain[0].isnan().any(1).equal(off)
    if tau == 1.0:
        check_gradients(x, H, W, tok, tau, a, b, logq, q, want_ent, plain, False)
    # a row that takes no part is not spoiled by its lse
    mask = torch.zeros(T, dtype=torch.bool, device="cuda")
    none = fkl.logprob_backward(H, W, tok, mask, lp, ent, lse, a, b, tau)
    assert (none[0] == 0).all() and (none[1] == 0).all()
    with pytest.raises(ValueError):
        fkl.logprob_forward(H, W, tok, tau=tau, stats=stats[:, :1])
    with pytest.raises(ValueError):
        fkl.logprob_backward(H, W, tok, None, lp, ent, lse, a, b, tau, stats=stats[:5])


@pytest.mark.parametrize("T", [5, 300])
def test_gradients_beside_logits_of_minus_infinity(fkl, T):
    H, W, tok, _ = make(T, 64, 1505, seed=4)
    W[:, 0] = 0.0
    W[3:40, 0], W[200, 0] = -8.0, -8.0
    tok[:] = 1
    H[:, 0] = 0.0
    H[2, 0] = 2.0 ** 127
    for b in (0.0, 1.0):
        Hl = H.clone().requires_grad_()
        lp, ent = fkl.fused_logprobs(Hl, W, tok)
        dH, = torch.autograd.grad(lp.sum() + b * ent.sum(), Hl)
        assert torch.isfinite(dH).all()


@pytest.mark.parametrize("T", [1, 300])
def test_a_row_without_scores_has_no_gradient_either(fkl, T):
    """A NaN in the head, or an lse that tells nothing: NaN in all of the head's gradient, the tokens' own rows too."""
    H, W, tok, _ = make(T, 64, 900, seed=6)
    tok[:] = 17
    one = torch.ones(T, device="cuda")
    lp, ent, lse = fkl.logprob_forward(H, W, tok, tau=1e-6)
    for got in fkl.logprob_backward(H, W, tok, None, lp, ent, lse, one, one, tau=1e-6):
        assert got.isnan().all()
    W[5] = float("nan")
    Wl = W.clone().requires_grad_()
    lp, ent = fkl.fused_logprobs(H, Wl, tok)
    assert lp.isnan().all() and ent.isnan().all()
    assert torch.autograd.grad(lp.sum(), Wl)[0].isnan().all()
    # rows that take no part in the sum stay out of it
    lp, ent, lse = fkl.logprob_forward(H, W, tok)
    none = fkl.logprob_backward(H, W, tok, None, lp, ent, lse, 0 * one, None, out=(None, torch.empty(900, 64, device="cuda")))
    assert (none[1] == 0).all()
