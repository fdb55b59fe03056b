"""Scores of given tokens from logits in memory (token_logprobs) against the float64 oracle.

Tolerances.  A row's sums are fp32: each weight 2^a has the exponential's 2^-22 and its argument's two
roundings (2^-23 |a| ln 2, |a| <= 32 where the weight matters), each addition 2^-24, at most V / 1024 of them in
a row in one thread and 40 across threads.  That is sum_tol(V), relative.  log q adds the roundings of its own terms.
"""
import math

import numpy as np
import pytest
import torch

from oracle import score as oracle

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def fkl(cuda_device):
    from lm_head_top_tcgen05_gb300 import build

    build.build()
    import lm_head_top_tcgen05_gb300 as m

    return m


def sum_tol(V):
    return 2.0 ** -22 + 32 * 2.0 ** -23 + (V / 1024 + 40) * 2.0 ** -24


def make(B, V, dtype, seed=0, pad=0, offset=0, sharp=1.0):
    """Logits [B, V] inside rows of V + pad, the first `offset` elements into their buffer."""
    g = torch.Generator().manual_seed(seed)
    buf = torch.randn(offset + B * (V + pad), generator=g) * 2 * sharp
    hot = torch.randint(0, max(1, buf.numel()), (max(1, buf.numel() // 50),), generator=g)
    buf[hot[:buf.numel()]] += 8
    buf = buf.to(dtype).cuda()
    x = buf[offset:].view(B, V + pad)[:, :V]
    return x, torch.randint(0, V, (B,), generator=g).cuda()


def check(fkl, x, tok, temperature=1.0, top_n=0, mask=None):
    B, V = x.shape
    r = fkl.token_logprobs(x, tok, temperature=temperature, top_n=top_n, mask=mask)
    T = temperature.cpu().double().numpy() if isinstance(temperature, torch.Tensor) else float(np.float32(temperature))
    xs = x.float().cpu().double().numpy()
    keep = None if mask is None else mask.cpu().numpy().astype(bool)
    lp, ent, logq, q = oracle.score(xs, tok.cpu().numpy(), T, keep)
    lp[lp < -float(np.finfo(np.float32).max)] = -np.inf  # no float32: 3e38 / 1e-3 below the largest
    Tb = np.broadcast_to(T, (B,))
    tol = sum_tol(V)
    got_lp, got_ent = r.logprob.cpu().double().numpy(), r.entropy.cpu().double().numpy()
    for b in range(B):
        assert np.isnan(lp[b]) == np.isnan(got_lp[b]) and np.isnan(ent[b]) == np.isnan(got_ent[b]), b
        if np.isfinite(lp[b]):
            # (x - m) / T: a subtraction, a product, 1 / T; then log L and the last subtraction
            lim = tol + 2.0 ** -24 * (4 * abs(lp[b]) + 4 * math.log(V + 1))
            assert abs(got_lp[b] - lp[b]) <= lim, (b, got_lp[b], lp[b], lim)
        elif not np.isnan(lp[b]):
            assert got_lp[b] == lp[b]
        if not np.isnan(ent[b]):
            # log L and U / L (both at most log V), each with the sums' error twice
            lim = 2 * tol * (1 + math.log(V + 1)) + 2.0 ** -22 * abs(ent[b])
            assert abs(got_ent[b] - ent[b]) <= lim, (b, got_ent[b], ent[b], lim)
    if top_n:
        ids, logs = r.top_ids.cpu().numpy(), r.top_logprobs.cpu().double().numpy()
        for b in range(B):
            if keep is not None and not keep[b]:
                assert (ids[b] == -1).all() and (logs[b] == -np.inf).all()
                continue
            if not (np.isfinite(Tb[b]) and Tb[b] > 0):
                assert (ids[b] == -1).all() and np.isnan(logs[b]).all()
                continue
            want = oracle.alternatives(xs[b], top_n)
            assert (ids[b] == want).all(), (b, ids[b], want)
            for i, v in enumerate(want):
                if np.isnan(ent[b]):
                    assert np.isnan(logs[b, i])
                elif v < 0 or logq[b, v] < -float(np.finfo(np.float32).max):
                    assert logs[b, i] == -np.inf
                else:
                    assert abs(logs[b, i] - logq[b, v]) <= tol + 2.0 ** -24 * (4 * abs(logq[b, v]) + 4 * math.log(V + 1))
    else:
        assert r.top_ids is None and r.top_logprobs is None
    return r


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,V,pad,offset,top_n", [
    (1, 1, 0, 0, 1), (3, 2, 1, 1, 2), (2, 7, 0, 3, 5), (5, 8, 0, 0, 8), (4, 33, 3, 5, 20), (1, 1000, 0, 0, 128),
    (7, 4097, 0, 1, 20), (2, 8191, 9, 0, 100), (1, 8192, 0, 0, 1), (3, 50261, 43, 0, 128), (1, 201088, 0, 0, 20),
    (40, 32768, 0, 0, 5), (311, 4099, 0, 0, 3), (0, 100, 0, 0, 4)])
def test_scores(fkl, dtype, B, V, pad, offset, top_n):
    x, tok = make(B, V, dtype, seed=V + B, pad=pad, offset=offset)
    check(fkl, x, tok, 0.8, top_n)
    check(fkl, x, tok.int(), 1.0, 0)


def test_slices_of_every_size(fkl):
    """Rows around the sizes at which a cluster gets another CTA, a thread another vector."""
    for V in (8190, 8193, 16383, 16389, 32767, 65541, 65536 + 7):
        for offset in (0, 1, 3):
            x, tok = make(2, V, torch.float16, seed=V, offset=offset, pad=offset)
            check(fkl, x, tok, 1.0, 40)


def test_rows_with_their_own_settings(fkl):
    x, tok = make(9, 5000, torch.float32, seed=3)
    T = torch.tensor([1.0, 0.3, 5.0, 0.0, -1.0, float("nan"), float("inf"), 1e-3, 2.0]).cuda()
    mask = torch.tensor([1, 1, 0, 1, 1, 1, 1, 1, 0], dtype=torch.uint8).cuda()
    for m in (None, mask, mask.bool()):
        check(fkl, x, tok, T, 7, m)


def test_special_values(fkl):
    inf, nan, low = float("inf"), float("nan"), torch.finfo(torch.float32).min
    V = 9000
    x = torch.randn(16, V, generator=torch.Generator().manual_seed(1))
    x[0] = -inf                        # nothing to produce
    x[1, 5:] = -inf                    # fewer ids than alternatives
    x[2] = nan
    x[3, ::2] = nan                    # NaN counts as -inf
    x[4, 100:] = low                   # masked with the type's lowest value
    x[5] = low
    x[6, [3, 4000]] = inf
    x[7] = 0.25                        # all equal
    x[8] = torch.randint(0, 3, (V,)).float()   # three values
    x[9, :] = -inf
    x[9, 8999] = -7.0                  # one id
    x[10, 11] = 3e38
    x[11] += 1e6                       # a large common offset
    x[12] = torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0)
    x[13] = torch.arange(V).float() / 100      # ascending
    x[14, :4096] = 5.0                 # more ties than the list holds, at the boundary
    x[15, 17] = -inf
    tok = torch.zeros(16, dtype=torch.int64)
    tok[6], tok[15] = 4000, 17
    x, tok = x.cuda(), tok.cuda()
    for n in (1, 20, 128):
        check(fkl, x, tok, 1.0, n)
    check(fkl, x, tok, 1e-3, 4)
    check(fkl, x, tok, 1e4, 4)
    for t in (torch.bfloat16, torch.float16):
        check(fkl, x.clamp(min=torch.finfo(t).min).where(x > -inf, x).to(t), tok, 1.0, 50)


def test_sharp_rows_keep_their_entropy(fkl):
    """Rows of entropy down to 1e-7: log L and -U / L have one sign, so only their own errors are left.

    L is 1 and a small rest.  Each addition that has the largest weight in it rounds at 1, by 2^-24 at most: V / 1024 in
    its thread, 5 across the warp, 16 across warps, and log L passes that on as an absolute error (at L = 1 its
    slope is 1).  The rest of both terms is off by the sums' relative error."""
    V = 3000
    x = torch.randn(6, V, dtype=torch.float64, generator=torch.Generator().manual_seed(2)).float()
    for b, top in enumerate([8.0, 12.0, 16.0, 20.0, 24.0, 28.0]):
        x[b, 77] = top
    tok = torch.full((6,), 77)
    r = fkl.token_logprobs(x.cuda(), tok.cuda())
    lp, ent, _, _ = oracle.score(x.numpy(), tok.numpy())
    got = r.entropy.cpu().double().numpy()
    at_one = (V / 1024 + 5 + 16) * 2.0 ** -24
    assert (np.abs(got - ent) <= 4 * sum_tol(V) * ent + at_one).all(), (got, ent)
    assert (np.abs(r.logprob.cpu().double().numpy() - lp) <= 4 * sum_tol(V) * np.abs(lp) + at_one).all()


def test_tokens_outside_the_row(fkl):
    x, _ = make(4, 100, torch.float32)
    tok = torch.tensor([-1, 100, 2 ** 33, 5]).cuda()
    r = fkl.token_logprobs(x, tok, top_n=2)
    assert torch.isnan(r.logprob[:3]).all() and torch.isfinite(r.logprob[3]) and torch.isfinite(r.entropy).all()
    r = fkl.token_logprobs(x, tok, mask=torch.tensor([False, False, False, True]).cuda())
    assert (r.logprob[:3] == 0).all() and (r.entropy[:3] == 0).all()


def test_same_bits_again_and_rows_alone(fkl):
    """The same inputs give the same bits; a row does not depend on its neighbours."""
    x, tok = make(300, 20011, torch.bfloat16, seed=4)
    a, b = fkl.token_logprobs(x, tok, top_n=30), fkl.token_logprobs(x, tok, top_n=30)
    for s, t in zip(a, b):
        assert torch.equal(s, t)
    x2 = x.clone()
    x2[1::2] = 0
    c = fkl.token_logprobs(x2, tok, top_n=30)
    for s, t in zip(a, c):
        assert torch.equal(s[::2], t[::2])


# ---------------------------------------------------------------- gradient
def check_gradient(fkl, x, tok, temperature=1.0, mask=None, entropy=True, logprob=True, top_n=0, seed=0):
    B, V = x.shape
    leaf = x.detach().requires_grad_()
    r = fkl.token_logprobs(leaf, tok, temperature=temperature, top_n=top_n, mask=mask)
    g = torch.Generator().manual_seed(seed)
    a, b = torch.randn(B, generator=g) * logprob, torch.randn(B, generator=g) * entropy
    outs = ([(r.logprob, a)] if logprob else []) + ([(r.entropy, b)] if entropy else [])
    dx, = torch.autograd.grad([o for o, _ in outs], (leaf,), [w.cuda() for _, w in outs])
    assert dx.dtype == x.dtype and dx.shape == x.shape
    T = temperature.cpu().double().numpy() if isinstance(temperature, torch.Tensor) else float(np.float32(temperature))
    keep = None if mask is None else mask.cpu().numpy().astype(bool)
    lp, ent, logq, q = oracle.score(x.float().cpu().double().numpy(), tok.cpu().numpy(), T, keep)
    want = oracle.score_gradient(logq, q, ent, tok.cpu().numpy(), a.numpy(), b.numpy(), T, keep)
    got = dx.float().cpu().double().numpy()
    assert (np.isnan(got) == np.isnan(want)).all()
    info = torch.finfo(x.dtype)
    Tb = np.broadcast_to(T, (B,))
    for i in range(B):
        if np.isnan(want[i]).any() or (keep is not None and not keep[i]):
            assert np.isnan(want[i]).all() or (got[i] == 0).all()
            continue
        lq = np.where(q[i] > 0, np.abs(logq[i]), 0)
        # q: its exponent's roundings (2^-23 of |log q| and of log L), the exponential's, the sums';
        # the factor c0 + c1 log2 q: the entropy's error and three roundings of its terms
        rel = 2.0 ** -21 + 2 * sum_tol(V) + 2.0 ** -22 * (lq + math.log(V + 1))
        terms = abs(float(a[i])) + abs(float(b[i])) * (lq + abs(ent[i]) + 1)
        lim = (q[i] * terms * rel + abs(float(b[i])) * q[i] * 2 * sum_tol(V) * (1 + math.log(V + 1))) / Tb[i]
        lim += 2.0 ** -23 * np.abs(want[i]) + 2.0 ** -126  # the sum at the token; fp32 below its normal range
        lim += (info.eps / 2 * np.abs(want[i]) if x.dtype != torch.float32 else 0) + info.smallest_normal * info.eps
        bad = np.abs(got[i] - want[i]) > lim
        assert not bad.any(), (i, np.flatnonzero(bad)[:5], got[i][bad][:5], want[i][bad][:5])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,V,pad,offset", [
    (1, 1, 0, 0), (3, 2, 1, 1), (2, 7, 0, 3), (5, 64, 0, 0), (3, 4097, 0, 0), (2, 8191, 9, 1), (4, 50261, 43, 0),
    (2, 50261, 0, 0), (1, 201088, 0, 0), (700, 130, 0, 0), (0, 10, 0, 0)])
def test_gradient(fkl, dtype, B, V, pad, offset):
    x, tok = make(B, V, dtype, seed=V, pad=pad, offset=offset)
    check_gradient(fkl, x, tok, 0.7)
    check_gradient(fkl, x, tok.int(), 1.0, entropy=False, top_n=min(V, 3))
    check_gradient(fkl, x, tok, 1.3, logprob=False)


def test_gradient_of_masked_and_odd_rows(fkl):
    inf = float("inf")
    x, tok = make(12, 3001, torch.float32, seed=8)
    x = x.clone()
    x[0] = -inf
    x[1, 7:] = -inf
    x[2, [3, 9]] = inf
    x[3, 5::2] = float("nan")
    x[4, 100:] = torch.finfo(torch.float32).min
    x[5] += 1e6
    x[6] = torch.finfo(torch.float32).min
    tok[2], tok[7], tok[8] = 9, -1, 3001
    T = torch.full((12,), 0.9).cuda()
    T[9] = 0.0
    mask = torch.ones(12, dtype=torch.bool).cuda()
    mask[10] = False
    for m in (None, mask):
        check_gradient(fkl, x, tok, T, m)
    off = torch.zeros(12, dtype=torch.bool).cuda()  # every odd row left out: no NaN is left
    check_gradient(fkl, x, tok, T, off)


def test_gradient_is_a_difference(fkl):
    """Central differences of the operator's own outputs."""
    x, tok = make(3, 500, torch.float32, seed=11)
    leaf = x.clone().requires_grad_()
    r = fkl.token_logprobs(leaf, tok, temperature=0.9)
    (r.logprob.sum() + 0.5 * r.entropy.sum()).backward()
    h = 2.0 ** -5
    for b, v in ((0, int(tok[0])), (1, 3), (2, int(x[2].argmax()))):
        vals = []
        for s in (1, -1):
            y = x.clone()
            y[b, v] += s * h
            q = fkl.token_logprobs(y, tok, temperature=0.9)
            vals.append((q.logprob[b] + 0.5 * q.entropy[b]).double().item())
        # h^2 / 6 of a third derivative of at most 10, and the outputs' fp32 error over 2 h
        assert abs((vals[0] - vals[1]) / (2 * h) - leaf.grad[b, v].item()) < 10 * h * h / 6 + 2.0 ** -20 * 16 / (2 * h)


def test_gradient_in_place_of_the_logits(fkl):
    """dlogits may be the logits' own memory (C ABI)."""
    from lm_head_top_tcgen05_gb300._lib import lib

    x, tok = make(5, 7777, torch.bfloat16, seed=5)
    leaf = x.clone().requires_grad_()
    r = fkl.token_logprobs(leaf, tok)
    ga = torch.randn(5).cuda()
    want, = torch.autograd.grad(r.logprob, leaf, ga)
    y = x.clone()
    lp, ent = torch.empty(5).cuda(), torch.empty(5).cuda()
    stats = torch.empty(5, 2).cuda()
    s = torch.cuda.current_stream().cuda_stream
    L = lib()
    assert L.fkl_token_logprobs(y.data_ptr(), 1, 5, 7777, 7777, tok.data_ptr(), 8, None, 1.0, None, 0, lp.data_ptr(),
                                ent.data_ptr(), stats.data_ptr(), None, None, s) == 0
    assert L.fkl_token_logprobs_backward(y.data_ptr(), 1, 5, 7777, 7777, tok.data_ptr(), 8, None, 1.0, None,
                                         stats.data_ptr(), ent.data_ptr(), ga.data_ptr(), None, y.data_ptr(), 7777, s) == 0
    assert torch.equal(y, want)


def test_offsets_beyond_32_bits(fkl):
    """A row whose elements lie beyond 2^31 elements, and bytes beyond 2^32, into the logits."""
    V, B = 2 ** 21 + 1, 1100
    x = torch.zeros(B, V, dtype=torch.bfloat16, device="cuda")
    small, tok1 = make(1, 1000, torch.bfloat16, seed=2)
    x[B - 1, V - 1000:] = small[0]
    x[B - 1, :V - 1000] = -math.inf
    tok = torch.full((B,), V - 1000, device="cuda") + tok1
    r = fkl.token_logprobs(x, tok, top_n=5, mask=torch.arange(B, device="cuda") == B - 1)
    s = fkl.token_logprobs(small, tok1, top_n=5)
    tol = 2 * sum_tol(V)
    assert abs(r.logprob[-1] - s.logprob[0]) < tol * 8 and abs(r.entropy[-1] - s.entropy[0]) < tol * 20
    assert torch.equal(r.top_ids[-1].long() - (V - 1000), s.top_ids[0].long())


def test_more_rows_than_a_grid_has(fkl):
    x, tok = make(70000, 5, torch.bfloat16, seed=3)
    r = fkl.token_logprobs(x, tok, top_n=2)
    rows = torch.tensor([0, 1, 65534, 65535, 65536, 69999]).cuda()
    s = fkl.token_logprobs(x[rows].contiguous(), tok[rows], top_n=2)
    for a, b in zip(r, s):
        assert torch.equal(a[rows], b)
    leaf = x.clone().requires_grad_()
    few = x[rows].clone().requires_grad_()
    da, = torch.autograd.grad(fkl.token_logprobs(leaf, tok).logprob.sum(), leaf)
    db, = torch.autograd.grad(fkl.token_logprobs(few, tok[rows]).logprob.sum(), few)
    assert torch.equal(da[rows], db)


def test_refusals(fkl):
    x, tok = make(3, 50, torch.float32)
    with pytest.raises(ValueError):
        fkl.token_logprobs(x, tok[:2])
    with pytest.raises(ValueError):
        fkl.token_logprobs(x, tok.short())
    with pytest.raises(ValueError):
        fkl.token_logprobs(x.t(), tok)
    with pytest.raises(TypeError):
        fkl.token_logprobs(x.double(), tok)
    with pytest.raises(ValueError):
        fkl.token_logprobs(x, tok, mask=torch.ones(2, dtype=torch.bool).cuda())
    with pytest.raises(ValueError):
        fkl.token_logprobs(x, tok, temperature=torch.ones(3, dtype=torch.float64).cuda())
    with pytest.raises(fkl.FklError):
        fkl.token_logprobs(x, tok, temperature=0.0)
    with pytest.raises(fkl.FklError):
        fkl.token_logprobs(x, tok, top_n=51)
    with pytest.raises(ValueError):
        fkl.token_logprobs(x, tok.cpu())


# ---------------------------------------------------------------- streams and graphs
def test_on_another_stream_and_in_a_graph(fkl):
    x, tok = make(6, 30011, torch.float16, seed=6)
    want = fkl.token_logprobs(x, tok, top_n=9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = fkl.token_logprobs(x, tok, top_n=9)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    y = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        leaf = y.detach().requires_grad_()
        r = fkl.token_logprobs(leaf, tok, top_n=9)
        dx, = torch.autograd.grad(r.logprob.sum() + r.entropy.sum(), leaf)
    for seed in (1, 2):
        new, _ = make(6, 30011, torch.float16, seed=seed)
        y.copy_(new)
        graph.replay()
        leaf = new.clone().requires_grad_()
        e = fkl.token_logprobs(leaf, tok, top_n=9)
        de, = torch.autograd.grad(e.logprob.sum() + e.entropy.sum(), leaf)
        for a, b in zip(r, e):
            assert torch.equal(a, b)
        assert torch.equal(dx, de)


def test_a_second_derivative_is_refused(fkl):
    x, tok = make(3, 100, torch.float32)
    leaf = x.clone().requires_grad_()
    r = fkl.token_logprobs(leaf, tok)
    dx, = torch.autograd.grad(r.logprob.sum(), leaf, create_graph=True)
    want, = torch.autograd.grad(fkl.token_logprobs(leaf, tok).logprob.sum(), leaf)
    assert torch.equal(dx.detach(), want)
    with pytest.raises(RuntimeError):
        dx.sum().backward()
