"""Scores and gradients from hidden states and the LM head (fused_logprobs) against the float64 oracle.

Tolerances.  The tensor cores add products in fp32, 16 deep: each step loses at most 2^-23 of the partial sum, which
is below sum |h w|, so a logit is off by s_tol = (d / 16 + 2) 2^-22 max sum |h w|, and log q by twice that over tau
and the sums' error (2^-20).  dS is rounded to bf16 (half a step: 2^-8; not its entries at the tokens), its
products are summed in fp32.
"""
import numpy as np
import pytest
import torch

from oracle import score as oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fkl(cuda_device):
    from lm_head_top_tcgen05_gb300 import build

    build.build()
    import lm_head_top_tcgen05_gb300 as m

    return m


def make(T, d, V, seed=0):
    g = torch.Generator().manual_seed(seed)
    W = torch.randn(V, d, generator=g) / d ** 0.5
    tok = torch.randint(0, V, (T,), generator=g)
    H = torch.randn(T, d, generator=g) * 1.5 + 6 * torch.rand(T, 1, generator=g) * W[tok]
    return H.bfloat16().cuda(), W.bfloat16().cuda(), tok.cuda(), (torch.rand(T, generator=g) > 0.2).cuda()


class Exact:
    def __init__(self, H, W, tok, mask, tau):
        self.H, self.W = H.float().cpu().double().numpy(), W.float().cpu().double().numpy()
        self.tok, self.tau = tok.cpu().numpy(), float(np.float32(tau))
        self.keep = None if mask is None else mask.cpu().numpy().astype(bool)
        T, d = self.H.shape
        self.x = self.H @ self.W.T
        self.lp, self.ent, self.logq, self.q = oracle.score(self.x, self.tok, self.tau, self.keep)
        size = (np.abs(self.H) @ np.abs(self.W).T).max() if T else 0.0
        self.log_tol = 2 * (d / 16 + 2) * 2.0 ** -22 * size / self.tau + 2.0 ** -20 * (2 + np.log(W.shape[0] + 1))

    def check_scores(self, lp, ent):
        lp, ent = lp.cpu().double().numpy(), ent.cpu().double().numpy()
        ok = np.isfinite(self.lp)
        assert (np.isnan(lp) == np.isnan(self.lp)).all() and (np.isnan(ent) == np.isnan(self.ent)).all()
        assert (np.abs(lp - self.lp)[ok] <= self.log_tol + 2.0 ** -22 * np.abs(self.lp[ok])).all()
        ok = np.isfinite(self.ent)
        # entropy = E[-log q]: log q's error, and that of the weights, relative, times the spread of log q
        spread = 1 + self.ent[ok] + np.log(self.q.shape[1] + 1)
        assert (np.abs(ent - self.ent)[ok] <= self.log_tol * (1 + spread)).all()

    def check_gradients(self, dH, dW, a, b, bf16, base=(0.0, 0.0)):
        a, b = a.cpu().double().numpy(), b.cpu().double().numpy()
        dS = oracle.score_gradient(self.logq, self.q, self.ent, self.tok, a, b, self.tau, self.keep)
        keep = np.ones(len(a), bool) if self.keep is None else self.keep
        lq = np.where(self.q > 0, np.abs(np.nan_to_num(self.logq)), 0)
        terms = (np.abs(a)[:, None] + np.abs(b)[:, None] * (lq + np.nan_to_num(self.ent)[:, None] + 1)) / self.tau
        off = np.where(keep[:, None], np.nan_to_num(self.q) * terms * 4 * self.log_tol, 0) + 2.0 ** -18 * np.abs(dS)
        # what rounding takes from the tokens' own entries is added back: in dW where at most 4 tokens share a row
        rows, used = np.arange(len(a))[keep], self.tok[keep]
        round_h, round_w = 2.0 ** -8 * np.abs(dS), 2.0 ** -8 * np.abs(dS)
        round_h[rows, used] = 0
        few = np.bincount(used, minlength=dS.shape[1])[used] <= 4
        round_w[rows[few], used[few]] = 0
        for got, want, room, start in ((dH, dS @ self.W, (off + round_h) @ np.abs(self.W), base[0]),
                                       (dW, dS.T @ self.H, (off + round_w).T @ np.abs(self.H), base[1])):
            if got is None:
                continue
            got = got.float().cpu().double().numpy()
            want = want + start
            lim = room + (2.0 ** -8 if bf16 else 2.0 ** -22) * np.abs(want) + 1e-30
            assert (np.abs(got - want) <= lim).all(), (np.abs(got - want) / lim).max()


@pytest.mark.parametrize("T,d,V,tau", [(1, 8, 1, 1.0), (1, 64, 300, 0.5), (3, 8, 17, 2.0), (130, 64, 257, 1.0),
                                       (257, 72, 1000, 0.8), (300, 128, 4099, 1.0), (64, 256, 30011, 1.3),
                                       (700, 40, 513, 1.0), (0, 16, 50, 1.0), (63, 160, 1500, 1.0),
                                       (64, 576, 900, 0.9), (65, 136, 769, 1.0), (256, 48, 2000, 1.0),
                                       (513, 192, 300, 1.0)])
def test_scores_and_gradients(fkl, T, d, V, tau):
    H, W, tok, mask = make(T, d, V, seed=T + V)
    for m, ids in ((None, tok), (mask, tok.int())):
        e = Exact(H, W, tok, m, tau)
        Hl, Wl = H.clone().requires_grad_(), W.clone().requires_grad_()
        lp, ent = fkl.fused_logprobs(Hl, Wl, ids, m, tau=tau, chunk=128)
        e.check_scores(lp.detach(), ent.detach())
        a, b = torch.randn(T).cuda(), torch.randn(T).cuda() * 0.3
        dH, dW = torch.autograd.grad((lp, ent), (Hl, Wl), (a, b))
        assert dH.dtype == dW.dtype == torch.bfloat16
        e.check_gradients(dH, dW, a, b, True)


def test_explicit_calls(fkl):
    """fp32 gradients, accumulation, one gradient alone, chunks of every size, a workspace that is kept."""
    T, d, V, tau = 520, 96, 3001, 0.9
    H, W, tok, mask = make(T, d, V, seed=1)
    e = Exact(H, W, tok, mask, tau)
    ws = fkl.Workspace()
    lp, ent, lse = fkl.logprob_forward(H, W, tok, mask, tau, workspace=ws)
    e.check_scores(lp, ent)
    want = torch.logsumexp(torch.tensor(e.x) / tau, 1)
    assert (lse.cpu().double() - want).abs().max() <= e.log_tol + 2.0 ** -22 * want.abs().max()
    a, b = torch.randn(T).cuda(), torch.randn(T).cuda()
    first = None
    for chunk in (1, 64, 2048, 10 ** 6):
        dH, dW = fkl.logprob_backward(H, W, tok, mask, lp, ent, lse, a, b, tau, chunk, workspace=ws)
        e.check_gradients(dH, dW, a, b, False)
        if chunk == 2048:
            first = dH, dW
    again = fkl.logprob_backward(H, W, tok, mask, lp, ent, lse, a, b, tau, 2048)
    assert all(torch.equal(x, y) for x, y in zip(first, again))  # the same bits
    half = fkl.logprob_backward(H, W, tok, mask, lp, ent, lse, a, b, tau, 2048, grad_dtype=torch.bfloat16)
    assert all(torch.equal(x.bfloat16(), y) for x, y in zip(first, half))  # fp32 sums rounded once
    base = torch.randn(T, d).cuda(), torch.randn(V, d).cuda()
    out = base[0].clone(), base[1].clone()
    fkl.logprob_backward(H, W, tok, mask, lp, ent, lse, a, b, tau, 512, out=out, accumulate=True)
    e.check_gradients(*out, a, b, False, base=tuple(x.cpu().double().numpy() for x in base))
    for only in (0, 1):
        out = [torch.full((T, d), 7.0).cuda(), torch.full((V, d), 7.0).cuda()]
        out[1 - only] = None
        got = fkl.logprob_backward(H, W, tok, mask, lp, ent, lse, a, b, tau, 2048, out=tuple(out))
        assert torch.equal(got[only], first[only]) and got[1 - only] is None
    dH, dW = fkl.logprob_backward(H, W, tok, mask, lp, ent, lse, a, None, tau)
    e.check_gradients(dH, dW, a, torch.zeros(T), False)
    dH, dW = fkl.logprob_backward(H, W, tok, mask, lp, ent, lse, None, b, tau)
    e.check_gradients(dH, dW, torch.zeros(T), b, False)
    assert fkl.read_status(ws) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_at_any_16_bytes(fkl, dtype):
    """Outputs that start 16 bytes into a 32-byte unit, and what lies around them."""
    T, d, V = 100, 64, 777
    H, W, tok, mask = make(T, d, V, seed=13)
    lp, ent, lse = fkl.logprob_forward(H, W, tok, mask)
    a, b = torch.randn(T).cuda(), torch.randn(T).cuda()
    want = fkl.logprob_backward(H, W, tok, mask, lp, ent, lse, a, b, grad_dtype=dtype)
    off = 16 // want[0].element_size()
    bufs = [torch.full((n * d + 2 * off,), 7.0, dtype=dtype, device="cuda") for n in (T, V)]
    out = tuple(x[off:-off].view(-1, d) for x in bufs)
    fkl.logprob_backward(H, W, tok, mask, lp, ent, lse, a, b, grad_dtype=dtype, out=out)
    for x, y, z in zip(out, want, bufs):
        assert torch.equal(x, y) and (z[:off] == 7).all() and (z[-off:] == 7).all()


def test_tokens_that_many_share(fkl):
    """One to many tokens of a vocabulary row, the same bits each time."""
    T, d, V = 600, 64, 40
    H, W, tok, mask = make(T, d, V, seed=2)
    tok = torch.arange(T).cuda() % 3
    tok[:30] = torch.arange(30).cuda() // 4 + 10  # rows of 4 tokens, one of 2
    tok[30:35] = 30                               # one of 5
    a, b = torch.randn(T).cuda(), torch.randn(T).cuda()
    for m in (None, mask):
        e = Exact(H, W, tok, m, 1.0)
        lp, ent, lse = fkl.logprob_forward(H, W, tok, m)
        for dtype in (torch.float32, torch.bfloat16):
            got = fkl.logprob_backward(H, W, tok, m, lp, ent, lse, a, b, grad_dtype=dtype)
            e.check_gradients(*got, a, b, dtype == torch.bfloat16)
            again = fkl.logprob_backward(H, W, tok, m, lp, ent, lse, a, b, grad_dtype=dtype)
            assert all(torch.equal(x, y) for x, y in zip(got, again))


def test_frozen_head_and_frozen_states(fkl):
    H, W, tok, _ = make(90, 64, 700, seed=3)
    Hl, Wl = H.clone().requires_grad_(), W.clone().requires_grad_()
    lp, ent = fkl.fused_logprobs(Hl, Wl, tok)
    both = torch.autograd.grad(lp.sum() + ent.mean(), (Hl, Wl))
    lp, ent = fkl.fused_logprobs(Hl, W, tok)
    (lp.sum() + ent.mean()).backward()
    assert torch.equal(Hl.grad, both[0])
    lp, ent = fkl.fused_logprobs(H, Wl, tok)
    (lp.sum() + ent.mean()).backward()
    assert torch.equal(Wl.grad, both[1])
    lp, ent = fkl.fused_logprobs(H, Wl, tok)
    assert torch.autograd.grad(lp.sum(), Wl)[0].shape == W.shape  # entropy unused


def test_several_token_blocks(fkl):
    """A long batch against a small vocabulary: the backward takes several token blocks, in either loop order."""
    T, d, V = 9000, 64, 900
    H, W, tok, mask = make(T, d, V, seed=5)
    lp, ent, lse = fkl.logprob_forward(H, W, tok, mask)
    e = Exact(H, W, tok, mask, 1.0)
    e.check_scores(lp, ent)
    a, b = torch.randn(T).cuda() / 30, torch.randn(T).cuda() / 90
    for dtype in (torch.float32, torch.bfloat16):
        for chunk in (100, 4096):
            dH, dW = fkl.logprob_backward(H, W, tok, mask, lp, ent, lse, a, b, chunk=chunk, grad_dtype=dtype)
            e.check_gradients(dH, dW, a, b, dtype == torch.bfloat16)


def test_sharp_rows(fkl):
    """Logits far above the rest: the reference moves, probabilities underflow."""
    H, W, tok, _ = make(200, 128, 5000, seed=9)
    H = (H.float() * 3).bfloat16()
    e = Exact(H, W, tok, None, 0.5)
    lp, ent = fkl.fused_logprobs(H, W, tok, tau=0.5)
    e.check_scores(lp, ent)


def test_tokens_outside_and_rows_left_out(fkl):
    H, W, tok, _ = make(300, 64, 500, seed=4)
    tok[7], tok[8] = -1, 500
    ws = fkl.Workspace()
    lp, ent, lse = fkl.logprob_forward(H, W, tok, workspace=ws)
    assert fkl.read_status(ws) == 6
    assert torch.isnan(lp[7:9]).all() and torch.isfinite(lp[:7]).all() and torch.isfinite(lp[9:]).all()
    assert torch.isfinite(ent).all()
    one = torch.ones(300).cuda()
    dH, dW = fkl.logprob_backward(H, W, tok, None, lp, ent, lse, one, None, workspace=ws)
    assert fkl.read_status(ws) == 6 and torch.isnan(dH).all() and torch.isnan(dW).all()
    mask = torch.ones(300, dtype=torch.uint8).cuda()
    mask[7:9] = 0
    lp, ent, lse = fkl.logprob_forward(H, W, tok, mask, workspace=ws)
    assert fkl.read_status(ws) == 0 and (lp[7:9] == 0).all() and (ent[7:9] == 0).all()
    dH, dW = fkl.logprob_backward(H, W, tok, mask, lp, ent, lse, one, one, workspace=ws)
    assert fkl.read_status(ws) == 0 and (dH[7:9] == 0).all() and torch.isfinite(dW).all()
    none = torch.zeros(300, dtype=torch.bool).cuda()
    lp, ent, lse = fkl.logprob_forward(H, W, tok, none)
    dH, dW = fkl.logprob_backward(H, W, tok, none, lp, ent, lse, one, one)
    assert (lp == 0).all() and (ent == 0).all() and (dH == 0).all() and (dW == 0).all()


@pytest.mark.parametrize("T,V", [(300, 500), (9000, 900)])
def test_rows_left_out_may_hold_anything(fkl, T, V):
    """NaN and infinities in the hidden states of masked rows reach neither the other rows nor dW."""
    H, W, tok, mask = make(T, 64, V, seed=12)
    a, b = torch.randn(T).cuda(), torch.randn(T).cuda()
    bad = H.clone()
    bad[~mask] = torch.tensor([float("nan"), float("inf")], device="cuda").bfloat16().repeat(32)
    for dtype in (torch.float32, torch.bfloat16):
        for chunk in (100, 4096):
            outs = []
            for h in (H, bad):
                lp, ent, lse = fkl.logprob_forward(h, W, tok, mask)
                outs.append((lp, ent) + fkl.logprob_backward(h, W, tok, mask, lp, ent, lse, a, b, chunk=chunk, grad_dtype=dtype))
            for x, y in zip(*outs):
                assert torch.isfinite(y).all() and torch.equal(x, y)


@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("start,n", [(0, 32), (0, 256), (256, 64), (1000, 1), (2990, 10)])
def test_nan_in_the_head_is_not_lost(fkl, T, start, n):
    """A NaN among a row's logits makes its scores NaN, also where it is all that the row begins with."""
    H, W, tok, _ = make(T, 64, 3000, seed=15)
    W[start:start + n] = float("nan")
    lp, ent = fkl.fused_logprobs(H, W, tok)
    assert lp.isnan().all() and ent.isnan().all()


@pytest.mark.parametrize("T", [5, 300])
def test_nan_in_one_row_stays_there(fkl, T):
    H, W, tok, _ = make(T, 64, 3000, seed=16)
    want = fkl.fused_logprobs(H, W, tok)
    H[2, 3] = float("nan")
    got = fkl.fused_logprobs(H, W, tok)
    rest = torch.arange(T, device="cuda") != 2
    for g, w in zip(got, want):
        assert g[2].isnan() and torch.equal(g[rest], w[rest])


def test_empty_batch_with_a_frozen_head(fkl):
    H, W, tok, _ = make(0, 16, 50)
    Hl = H.requires_grad_()
    lp, ent = fkl.fused_logprobs(Hl, W, tok)
    lp.sum().backward()
    assert Hl.grad.shape == (0, 16)
    Wl = W.clone().requires_grad_()
    lp, ent = fkl.fused_logprobs(H.detach(), Wl, tok)
    lp.sum().backward()
    assert (Wl.grad == 0).all()


def test_a_second_derivative_is_refused(fkl):
    H, W, tok, _ = make(20, 64, 100)
    Hl = H.clone().requires_grad_()
    dH, = torch.autograd.grad(fkl.fused_logprobs(Hl, W, tok)[0].sum(), Hl, create_graph=True)
    with pytest.raises(RuntimeError):
        dH.float().sum().backward()


def test_refusals(fkl):
    H, W, tok, mask = make(20, 64, 100)
    with pytest.raises(TypeError):
        fkl.fused_logprobs(H.float(), W, tok)
    with pytest.raises(ValueError):
        fkl.fused_logprobs(H, W[:, :32], tok)
    with pytest.raises(ValueError):
        fkl.fused_logprobs(H, W, tok[:5])
    with pytest.raises(ValueError):
        fkl.fused_logprobs(H, W, tok, mask[:5])
    with pytest.raises(fkl.FklError):
        fkl.fused_logprobs(H, W, tok, tau=0.0)
    with pytest.raises(fkl.FklError):
        fkl.fused_logprobs(H[:, :12].contiguous(), W[:, :12].contiguous(), tok)
    lp, ent, lse = fkl.logprob_forward(H, W, tok)
    with pytest.raises(ValueError):
        fkl.logprob_backward(H, W, tok, None, lp, ent, lse[:3])
    with pytest.raises(ValueError):
        fkl.logprob_backward(H, W, tok, None, lp, ent, lse, ent.double())
    with pytest.raises(fkl.FklError):
        fkl.logprob_backward(H, W, tok, None, lp, ent, lse, ent, chunk=0)
    with pytest.raises(fkl.FklError):
        fkl.logprob_backward(H, W, tok, None, lp, ent, lse, ent, out=(None, None))


def test_another_stream_and_a_graph(fkl):
    H, W, tok, mask = make(300, 64, 2000, seed=6)
    want = fkl.fused_logprobs(H, W, tok, mask)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = fkl.fused_logprobs(H, W, tok, mask)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    a, b = torch.randn(300).cuda(), torch.randn(300).cuda()
    h = H.clone()

    def step(h):
        lp, ent, lse = fkl.logprob_forward(h, W, tok, mask)
        return (lp, ent) + fkl.logprob_backward(h, W, tok, mask, lp, ent, lse, a, b, grad_dtype=torch.bfloat16)

    step(h)  # one eager call of the shape, as for the loss
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for g in graphs:  # two graphs share no scratch
        with torch.cuda.graph(g):
            outs.append(step(h))
    for seed in (1, 2):
        h.copy_(make(300, 64, 2000, seed=seed)[0])
        for g in graphs:
            g.replay()
        eager = step(h)
        for o in outs:
            assert all(torch.equal(x, y) for x, y in zip(o, eager))


def test_several_threads(fkl):
    """Threads on streams of their own, and on one stream, share no scratch."""
    import threading

    H, W, tok, mask = make(200, 64, 3000, seed=14)
    x = (H.float() @ W.float().t()).bfloat16()
    a = torch.randn(200).cuda()

    def step():
        Hl, Wl = H.clone().requires_grad_(), W.clone().requires_grad_()
        lp, ent = fkl.fused_logprobs(Hl, Wl, tok, mask)
        return (lp.detach(),) + torch.autograd.grad((lp, ent), (Hl, Wl), (a, a)) + tuple(fkl.token_logprobs(x, tok, top_n=7))

    want = step()
    torch.cuda.synchronize()
    wrong = []

    def work(stream):
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = step()
                stream.synchronize()
                wrong.extend(1 for u, v in zip(got, want) if not torch.equal(u, v))

    shared = torch.cuda.Stream()
    threads = [threading.Thread(target=work, args=(s,)) for s in (torch.cuda.Stream(), torch.cuda.Stream(), shared, shared)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


# ---------------------------------------------------------------- together
def test_draw_score_and_train(fkl):
    """What a server and an on-policy step do: draw through an 8-bit head, score from its logits, then a policy gradient
    from the hidden states whose scores agree with the logits'."""
    g = torch.Generator(device="cuda").manual_seed(1)
    T, d, V = 256, 128, 4000
    H = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    W = (torch.randn(V, d, generator=g, device="cuda") * 0.2).bfloat16()
    wq, ws = fkl.quantize_int8(W)
    logits = torch.empty(T, V, device="cuda")
    token, drawn = fkl.draw_token(H, wq, ws, torch.rand(T, generator=g, device="cuda"), temperature=0.8, logits=logits)
    r = fkl.token_logprobs(logits, token, temperature=0.8, top_n=5)
    # without filters the sampler's log-probability is the scored one: whole weights of 2^-40 and fp32 sums
    assert (r.logprob - drawn).abs().max() < 2.0 ** -24 * 64 + 2 * (2.0 ** -22 + 32 * 2.0 ** -23 + 44 * 2.0 ** -24)
    assert (r.top_logprobs[:, 0] >= r.logprob).all()
    Hl, Wl = H.clone().requires_grad_(), W.clone().requires_grad_()
    lp, ent = fkl.fused_logprobs(Hl, Wl, token, tau=0.8)
    x = H.float() @ W.float().t()
    full = fkl.token_logprobs(x, token, temperature=0.8)
    e = Exact(H, W, token.long(), None, 0.8)
    e.check_scores(lp.detach(), ent.detach())
    assert (full.logprob - lp.detach()).abs().max() < 2 * e.log_tol + 2.0 ** -22 * 20
    adv = torch.randn(T, generator=g, device="cuda")
    (-(adv * lp).mean() - 0.01 * ent.mean()).backward()
    e.check_gradients(Hl.grad, Wl.grad, -adv / T, torch.full((T,), -0.01 / T), True)
