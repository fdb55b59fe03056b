"""The head's gradient where many tokens share a vocabulary row, as the frequent tokens of a text do.

A cross-entropy gives every token the same weight, so that tokens of small q have entries that round to the same bf16
value: their rounding errors have one sign and add up.  What rounding takes from a token's own entry is added back, whatever
the number of tokens.

Tolerances.  Entries of other tokens in the row are bf16 (2^-8 of each).  A token's own entry a (1 - q) is fp32 (2^-22), with
q off by log q's error.  Sums are made in the tensor cores, 16 products at a time: each product and the sum so far are cut off
(towards zero) at 2^-25 of the largest one's binary order.  (1 + n products of 2^-26 comes to 1, with n products of
2^-24 or 2^-25 to their sum; the results have fp32's 24 bits.)  A step so loses at most 16 * 2^-25 = 2^-21 and the cut of its
result, 2^-23, of the terms' size.  (A step that rounded once would lose 2^-23 at most: T = 3000 tokens lost 1.05
of T / 16 times that.)  What was taken adds one rounding a token, itself at most 2^-8 of the entry.
"""
import numpy as np
import pytest
import torch

from tests.test_gpu_score_fused import Exact

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fkl(cuda_device):
    from lm_head_top_tcgen05_gb300 import build

    build.build()
    import lm_head_top_tcgen05_gb300 as m

    return m


def make(T, d, V, shared, seed=0):
    """`shared` tokens of row 7, the others spread; positive hidden states, so that errors of one sign add up."""
    g = torch.Generator().manual_seed(seed)
    H = torch.randn(T, d, generator=g).abs() + 0.5
    W = torch.randn(V, d, generator=g) * 0.3 * (64 / d) ** 0.5
    tok = torch.randint(0, V, (T,), generator=g)
    tok[tok == 7] = 8
    tok[torch.randperm(T, generator=g)[:shared]] = 7
    return H.bfloat16().cuda(), W.bfloat16().cuda(), tok.cuda()


def check(e, dW, a, half, accumulated=0.0):
    a = a.cpu().double().numpy()
    keep = np.ones(len(a), bool) if e.keep is None else e.keep
    dS = -a[:, None] * np.nan_to_num(e.q)
    rows = np.arange(len(a))
    dS[rows, e.tok] += a
    dS[~keep] = 0
    size = np.abs(dS)
    room = np.nan_to_num(e.q) * np.abs(a)[:, None] * 4 * e.log_tol + 2.0 ** -8 * size
    room[rows, e.tok] -= 2.0 ** -8 * size[rows, e.tok]
    room += (2.0 ** -21 + (len(a) / 16 + 8) * (2.0 ** -21 + 2.0 ** -23) + len(a) * 2.0 ** -32) * size
    room[~keep] = 0
    want = dS.T @ e.H + accumulated
    lim = room.T @ np.abs(e.H) + (2.0 ** -8 if half else 2.0 ** -23) * np.abs(want) + 1e-30
    off = np.abs(dW.float().cpu().double().numpy() - want)
    assert (off <= lim).all(), (off / lim).max()


@pytest.mark.parametrize("T,d,V,shared", [(600, 64, 3001, 500), (600, 64, 3001, 5), (64, 8, 900, 40), (9, 2056, 300, 8),
                                          (2500, 136, 700, 2100), (300, 4104, 64, 200), (2600, 64, 40, 5)])
def test_one_weight_for_all(fkl, T, d, V, shared):
    H, W, tok = make(T, d, V, shared, seed=T + d)
    a = torch.full((T,), 1 / 3001).cuda()
    keep = torch.rand(T, generator=torch.Generator().manual_seed(1)) > 0.2
    for mask in (None, keep.cuda()):
        e = Exact(H, W, tok, mask, 1.0)
        lp, ent, lse = fkl.logprob_forward(H, W, tok, mask)
        both = fkl.logprob_backward(H, W, tok, mask, lp, ent, lse, a)
        check(e, both[1], a, False)
        again = fkl.logprob_backward(H, W, tok, mask, lp, ent, lse, a)
        assert torch.equal(both[1], again[1]) and torch.equal(both[0], again[0])
        only = fkl.logprob_backward(H, W, tok, mask, lp, ent, lse, a, out=(None, torch.empty_like(both[1])))
        assert torch.equal(only[1], both[1])
        half = fkl.logprob_backward(H, W, tok, mask, lp, ent, lse, a, grad_dtype=torch.bfloat16)
        assert torch.equal(half[1], both[1].bfloat16())
        base = torch.randn(V, d).cuda() * 1e-3
        sums = fkl.logprob_backward(H, W, tok, mask, lp, ent, lse, a, out=(torch.zeros_like(both[0]), base.clone()),
                                    accumulate=True)
        check(e, sums[1], a, False, base.cpu().double().numpy())


def test_ids_with_the_frequencies_of_text(fkl):
    """Ids drawn with 1 / rank: rows of one to hundreds of tokens, several token blocks, both types."""
    T, d, V = 3000, 64, 2000
    g = torch.Generator().manual_seed(8)
    H, W, _ = make(T, d, V, 0)
    tok = torch.multinomial(1 / (1 + torch.arange(V).double()), T, replacement=True, generator=g).cuda()
    a = torch.full((T,), 1 / 3001).cuda()
    e = Exact(H, W, tok, None, 1.0)
    lp, ent, lse = fkl.logprob_forward(H, W, tok)
    for chunk in (300, 1000, 4096):
        for dtype in (torch.float32, torch.bfloat16):
            _, dW = fkl.logprob_backward(H, W, tok, None, lp, ent, lse, a, chunk=chunk, grad_dtype=dtype)
            check(e, dW, a, dtype == torch.bfloat16)


def test_a_nan_in_a_shared_row_stays_there(fkl):
    """A hidden state that is NaN, in a row left out, does not come into the sums of the others."""
    H, W, tok = make(200, 64, 500, 100)
    mask = torch.ones(200, dtype=torch.bool, device="cuda")
    mask[(tok == 7).nonzero()[:20, 0]] = False
    a = torch.full((200,), 1 / 3001).cuda()
    lp, ent, lse = fkl.logprob_forward(H, W, tok, mask)
    want = fkl.logprob_backward(H, W, tok, mask, lp, ent, lse, a)
    H[~mask] = float("nan")
    lp, ent, lse = fkl.logprob_forward(H, W, tok, mask)
    got = fkl.logprob_backward(H, W, tok, mask, lp, ent, lse, a)
    assert torch.equal(want[1], got[1]) and torch.equal(want[0], got[0])


def test_a_row_of_thousands_of_tokens(fkl):
    """Longer than one look through the tokens of a CTA's share, beside rows of few and of tens of tokens."""
    T, d, V = 12000, 24, 800
    H, W, tok = make(T, d, V, 9000, seed=3)
    tok[:70] = 9
    a = torch.full((T,), 1 / 3001).cuda()
    e = Exact(H, W, tok, None, 1.0)
    lp, ent, lse = fkl.logprob_forward(H, W, tok)
    got = fkl.logprob_backward(H, W, tok, None, lp, ent, lse, a)
    check(e, got[1], a, False)
    half = fkl.logprob_backward(H, W, tok, None, lp, ent, lse, a, grad_dtype=torch.bfloat16)
    assert torch.equal(half[1], got[1].bfloat16())


def test_shared_rows_in_a_graph(fkl):
    """A captured step follows the tokens that it is replayed with: other rows are shared then, or none."""
    T, d, V = 400, 64, 900
    H, W, tok = make(T, d, V, 200)
    a = torch.randn(T).cuda()
    stats = torch.empty(T, 2, device="cuda")

    def step():
        lp, ent, lse = fkl.logprob_forward(H, W, tok, tau=0.01, stats=stats)
        return (lp, ent) + fkl.logprob_backward(H, W, tok, None, lp, ent, None, a, tau=0.01, stats=stats,
                                                grad_dtype=torch.bfloat16)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed, shared in ((1, 5), (2, 0), (3, 350)):
        h, w, t = make(T, d, V, shared, seed)
        H.copy_(h)
        W.copy_(w)
        tok.copy_(t)
        graph.replay()
        for x, y in zip(outs, step()):
            assert torch.equal(x, y)


def test_shared_rows_on_several_streams(fkl):
    import threading

    H, W, tok = make(700, 64, 900, 300, seed=4)
    a = torch.randn(700).cuda()

    def step():
        Hl, Wl = H.clone().requires_grad_(), W.clone().requires_grad_()
        lp, ent = fkl.fused_logprobs(Hl, Wl, tok, tau=0.05)
        return torch.autograd.grad((lp, ent), (Hl, Wl), (a, a))

    want = step()
    torch.cuda.synchronize()
    wrong = []

    def work(stream):
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = step()
                stream.synchronize()
                wrong.extend(1 for u, v in zip(got, want) if not torch.equal(u, v))

    threads = [threading.Thread(target=work, args=(torch.cuda.Stream(),)) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
