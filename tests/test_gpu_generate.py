"""The generation operators on the GPU against the float64 oracle (oracle/generate.py).

Tolerances, derived: the quantised integers and scales are IEEE float32 arithmetic and are
compared exactly.  A product's integer sum is exact while its partial sums stay below 2^24;
otherwise each of the K / 16 accumulation steps loses at most 2^-23 of the largest partial sum.
The two scales add a rounding each (2^-24), the output type its own half unit in the last
place.  Sampled tokens must be among those the oracle allows when exponentials are off by
2^-22 (CUDA's expf is within 2 units in the last place, 2^-22), the log-probability within
2^-20 relative plus 1e-6.
"""
import numpy as np
import pytest
import torch

from oracle import generate as og

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
HALF_ULP = {t: torch.finfo(t).eps / 2 for t in TYPES}


@pytest.fixture(scope="module")
def fkl(cuda_device):
    from lm_head_top_tcgen05_gb300 import build

    build.build()
    import lm_head_top_tcgen05_gb300 as m

    return m


# ---------------------------------------------------------------- quantisation
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K", [(1, 1), (1, 16), (3, 17), (5, 2880), (2, 4100), (70, 48), (2, 40000)])
def test_quantize(fkl, dtype, M, K):
    g = torch.Generator().manual_seed(M * 1000 + K)
    x = (torch.randn(M, K, generator=g) * 3).to(dtype)
    q, s = fkl.quantize_int8(x.cuda())
    rq, rs = og.quantize_int8(x.float().numpy())
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_special_rows_and_strides(fkl, dtype):
    x = torch.randn(8, 100, generator=torch.Generator().manual_seed(1)).to(dtype)
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 5] = float("-inf")
    x[3] = torch.finfo(dtype).tiny * 2.0 ** -3      # subnormal values
    x[4] = torch.finfo(dtype).max
    x[5, 1:] = 0
    for view in (x, x[:, 1:], x[:, :64], x[::2, 3:51]):
        v = x.cuda()[tuple(slice(*i) for i in _slices(x, view))]
        q, s = fkl.quantize_int8(v)
        rq, rs = og.quantize_int8(view.float().numpy())
        np.testing.assert_array_equal(s.cpu().numpy(), rs)
        np.testing.assert_array_equal(q.cpu().numpy(), rq)


def _slices(x, view):
    off = view.storage_offset()
    r0, c0 = divmod(off, x.shape[1])
    step = view.stride(0) // x.shape[1]
    return (r0, r0 + view.shape[0] * step, step), (c0, c0 + view.shape[1], 1)


def test_quantize_empty(fkl):
    q, s = fkl.quantize_int8(torch.empty(0, 64, device="cuda"))
    assert q.shape == (0, 64) and s.shape == (0,)


# ---------------------------------------------------------------- product
def operands(M, N, K, seed):
    rng = np.random.default_rng(seed)
    xq = rng.integers(-128, 128, (M, K)).astype(np.int8)
    wq = rng.integers(-128, 128, (N, K)).astype(np.int8)
    # scales that keep every output a normal float16
    xs = (rng.uniform(0.5, 2.0, M) / 256).astype(np.float32)
    ws = (rng.uniform(0.5, 2.0, N) / 256).astype(np.float32)
    return xq, xs, wq, ws


def dev(*arrays):
    return [torch.from_numpy(a).cuda() for a in arrays]


def assert_product(got, ops, dtype):
    xq, xs, wq, ws = ops
    ref = og.int8_matmul(xq, xs, wq, ws)
    K = xq.shape[1]
    mag = og.int8_matmul(np.abs(xq.astype(np.int16)), xs, np.abs(wq.astype(np.int16)), ws)
    exact_sum = K <= 1024
    tol = np.abs(ref) * (3 * 2.0 ** -24 + HALF_ULP[dtype]) + (2.0 ** -24 if dtype == torch.float16 else 0)
    if not exact_sum:
        tol = tol + mag * (K / 16) * 2.0 ** -23
    err = np.abs(got.double().cpu().numpy() - ref)
    assert got.dtype == dtype
    assert (err <= tol).all(), (float((err - tol).max()), np.argwhere(err > tol)[:4])


MATMUL_SHAPES = [(1, 1, 16), (1, 5, 48), (1, 130, 2880), (2, 4099, 64), (3, 128, 144), (4, 1000, 4096), (5, 77, 160),
                 (7, 129, 272), (8, 1024, 512), (9, 300, 1040), (15, 257, 128), (16, 256, 256), (17, 640, 2880),
                 (31, 515, 1456), (33, 1001, 96), (64, 384, 1024), (65, 2000, 320), (100, 133, 208), (127, 260, 112),
                 (128, 512, 640), (129, 383, 784), (192, 1030, 176), (200, 700, 1456), (255, 129, 64), (256, 256, 2880),
                 (257, 513, 272), (300, 2100, 512), (513, 300, 400), (1000, 1000, 1040), (40, 30000, 128), (1, 60001, 32)]


@pytest.mark.parametrize("M,N,K", MATMUL_SHAPES)
def test_int8_matmul(fkl, M, N, K):
    ops = operands(M, N, K, M * 7 + N * 3 + K)
    t = dev(*ops)
    for dtype in TYPES:
        assert_product(fkl.int8_matmul(*t, out_dtype=dtype), ops, dtype)


# More tiles than run at once, with several tiles of up to 128 tokens.
@pytest.mark.parametrize("M,N,K", [(129, 12001, 144), (200, 12000, 256), (250, 10100, 48), (256, 19456, 272),
                                   (257, 13001, 128), (300, 13057, 400), (400, 12290, 272), (513, 8000, 256)])
def test_int8_matmul_wide(fkl, M, N, K):
    ops = operands(M, N, K, M + N + K)
    t = dev(*ops)
    for dtype in TYPES:
        assert_product(fkl.int8_matmul(*t, out_dtype=dtype), ops, dtype)


# Wide and deep enough for tiles of 129 to 256 tokens: one and several of them, an odd last one, and a
# last wave that is cut (the last two).
@pytest.mark.parametrize("M,N,K", [(129, 12001, 2064), (200, 12000, 1456), (250, 10100, 1296), (257, 13001, 4096),
                                   (400, 12290, 2880), (513, 8000, 4112), (140, 19500, 8000), (200, 19500, 9008)])
def test_int8_matmul_large_tiles(fkl, M, N, K):
    ops = operands(M, N, K, M + N + K)
    assert_product(fkl.int8_matmul(*dev(*ops), out_dtype=torch.bfloat16), ops, torch.bfloat16)


# One tile more than run at once (256 channels and tokens each, 76 at once): it is cut, into fewer
# blocks than there are pairs to share them.
@pytest.mark.parametrize("M,N,K", [(16, 19500, 8192), (9, 19460, 4112), (5, 38913, 8192), (140, 19500, 8000)])
def test_int8_matmul_cut_into_few_blocks(fkl, M, N, K):
    ops = operands(M, N, K, M + N + K)
    assert_product(fkl.int8_matmul(*dev(*ops)), ops, torch.float32)


@pytest.mark.parametrize("M", [1, 6, 40, 300])
def test_int8_matmul_largest_values(fkl, M):
    # every product 128 * 128: the largest sums that K = 4096 can give
    xq = np.full((M, 4096), -128, dtype=np.int8)
    wq = np.full((200, 4096), -128, dtype=np.int8)
    wq[::3] = 127
    ops = (xq, np.full(M, 0.25, np.float32), wq, np.ones(200, np.float32))
    assert_product(fkl.int8_matmul(*dev(*ops)), ops, torch.float32)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [1, 5, 20, 270])
def test_int8_matmul_into_strided_output(fkl, dtype, M):
    ops = operands(M, 301, 256, 4 + M)
    big = torch.full((M, 333), 7.0, dtype=dtype, device="cuda")
    out = big[:, 5:306]
    got = fkl.int8_matmul(*dev(*ops), out_dtype=dtype, out=out)
    assert got.data_ptr() == out.data_ptr()
    assert_product(out, ops, dtype)
    assert (big[:, :5] == 7).all() and (big[:, 306:] == 7).all()


@pytest.mark.parametrize("M", [2, 33])
def test_int8_matmul_special_scales(fkl, M):
    ops = list(operands(M, 150, 128, 9))
    ops[1][0] = np.nan
    ops[3][3] = 0.0
    y = fkl.int8_matmul(*dev(*ops)).cpu().numpy()
    assert np.isnan(y[0]).all()
    assert (y[1:, 3] == 0).all() and np.isfinite(y[1:]).all()


@pytest.mark.parametrize("x_dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(1, 500, 2880), (2, 129, 48), (8, 1000, 256), (9, 300, 1456), (50, 257, 512),
                                   (300, 400, 1024)])
def test_int8_linear(fkl, x_dtype, M, N, K):
    g = torch.Generator().manual_seed(M + N + K)
    x = torch.randn(M, K, generator=g).to(x_dtype)
    W = torch.randn(N, K, generator=g) * 0.02
    wq, ws = og.quantize_int8(W.numpy())
    xq, xs = og.quantize_int8(x.float().numpy())
    for dtype in TYPES:
        y = fkl.int8_linear(x.cuda(), *dev(wq, ws), out_dtype=dtype)
        ref = og.int8_matmul(xq, xs, wq, ws)
        tol = np.abs(ref) * (3 * 2.0 ** -24 + HALF_ULP[dtype]) + (2.0 ** -24 if dtype == torch.float16 else 0)
        if K > 1024:
            tol = tol + og.int8_matmul(np.abs(xq), xs, np.abs(wq), ws) * (K / 16) * 2.0 ** -23
        assert (np.abs(y.double().cpu().numpy() - ref) <= tol).all()
    assert fkl.int8_linear(x.cuda(), *dev(wq, ws)).dtype == x_dtype


@pytest.mark.parametrize("M", [1, 7, 40])
def test_int8_linear_strided_and_special_rows(fkl, M):
    # the last token of each sequence of a batch; rows that are zero or hold a NaN
    g = torch.Generator().manual_seed(M)
    h = torch.randn(M, 5, 320, generator=g).to(torch.bfloat16)
    h[0, -1] = 0
    if M > 1:
        h[1, -1, 7] = float("nan")
    x = h[:, -1]
    W = torch.randn(333, 320, generator=g) * 0.02
    wq, ws = og.quantize_int8(W.numpy())
    y = fkl.int8_linear(h.cuda()[:, -1], *dev(wq, ws), out_dtype=torch.float32).cpu().numpy()
    xq, xs = og.quantize_int8(x.float().numpy())
    ref = og.int8_matmul(xq, xs, wq, ws)
    assert (y[0] == 0).all()
    if M > 1:
        assert np.isnan(y[1]).all()
    ok = [0] + list(range(2, M))
    assert (np.abs(y[ok] - ref[ok]) <= np.abs(ref[ok]) * 4 * 2.0 ** -24).all()


def test_products_of_no_tokens(fkl):
    wq, ws = torch.zeros(50, 64, dtype=torch.int8, device="cuda"), torch.ones(50, device="cuda")
    assert fkl.int8_linear(torch.empty(0, 64, device="cuda"), wq, ws).shape == (0, 50)
    xq = torch.empty(0, 64, dtype=torch.int8, device="cuda")
    assert fkl.int8_matmul(xq, torch.empty(0, device="cuda"), wq, ws).shape == (0, 50)


@pytest.mark.parametrize("M", [1, 30, 300])
def test_product_status_and_repeat(fkl, M):
    ops = dev(*operands(M, 3000, 1456, 2))
    ws = fkl.Workspace("cuda")
    a = fkl.int8_matmul(*ops, workspace=ws)
    b = fkl.int8_matmul(*ops, workspace=ws)
    assert fkl.read_status(ws) == 0
    assert torch.equal(a, b)


# ---------------------------------------------------------------- sampler
def check_sample(fkl, logits, u, **kw):
    """logits: CPU tensor; settings: numbers or CPU tensors [B]."""
    B = logits.shape[0]
    dk = {n: (v.cuda() if isinstance(v, torch.Tensor) else v) for n, v in kw.items()}
    lg = logits.cuda() if logits.is_contiguous() else _on_gpu_strided(logits)
    token, logprob = fkl.sample(lg, u.cuda(), **dk)
    token2, logprob2 = fkl.sample(lg, u.cuda(), **dk)
    assert token.dtype == torch.int32 and logprob.dtype == torch.float32
    assert torch.equal(token, token2)
    assert torch.equal(logprob.nan_to_num(7), logprob2.nan_to_num(7))
    token, logprob = token.cpu().tolist(), logprob.cpu().tolist()
    rows = logits.float().numpy()
    for b in range(B):
        a = {n: (v[b].item() if isinstance(v, torch.Tensor) else v) for n, v in kw.items()}
        ok = og.sample_row(rows[b], u[b].item(), **a)
        assert token[b] in ok, (b, token[b], ok, a)
        if token[b] < 0:
            assert np.isnan(logprob[b])
        else:
            lo, hi = ok[token[b]]
            margin = 2.0 ** -20 * abs(lo) + 1e-6
            assert lo - margin <= logprob[b] <= hi + margin, (b, logprob[b], lo, hi)
    return token


def _on_gpu_strided(t):
    big = torch.zeros(t.shape[0], t.stride(0), dtype=t.dtype)
    out = big.cuda()[:, :t.shape[1]]
    out.copy_(t)
    return out


def lm_logits(B, V, seed, dtype=torch.float32, hot=10):
    g = torch.Generator().manual_seed(seed)
    x = 2.0 * torch.randn(B, V, generator=g)
    if V > 4 * hot:
        x.scatter_add_(1, torch.randint(0, V, (B, hot), generator=g), 5 + 4 * torch.rand(B, hot, generator=g))
    return x.to(dtype), torch.rand(B, generator=g)


SETTINGS = [dict(), dict(temperature=0.0), dict(temperature=0.7, top_k=50, top_p=0.95), dict(top_k=1), dict(top_k=5),
            dict(top_p=0.9), dict(top_p=0.999), dict(top_p=0.0), dict(min_p=0.05), dict(min_p=2.0),
            dict(temperature=1.5, top_k=3000), dict(temperature=1.3, top_k=2000, top_p=0.8, min_p=0.001),
            dict(temperature=8.0, top_p=0.5), dict(temperature=0.05, top_p=0.9), dict(top_k=10 ** 6),
            dict(temperature=100.0, top_p=0.99)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kw", SETTINGS, ids=lambda k: ",".join(f"{a}={b}" for a, b in k.items()) or "plain")
def test_sample_settings(fkl, dtype, kw):
    logits, u = lm_logits(6, 20011, 3, dtype)
    check_sample(fkl, logits, u, **kw)


@pytest.mark.parametrize("V", [1, 2, 3, 31, 32, 33, 255, 1000, 1024, 1025, 4096, 50261, 201088, 300007])
def test_sample_sizes(fkl, V):
    for seed, kw in enumerate((dict(), dict(top_k=7), dict(top_p=0.8), dict(top_k=40, top_p=0.9, min_p=0.01))):
        logits, u = lm_logits(3, V, V + seed)
        check_sample(fkl, logits, u, **kw)


def test_sample_largest_vocabulary(fkl):
    V = 2 ** 22
    logits, u = lm_logits(2, V, 1, torch.bfloat16)
    check_sample(fkl, logits, u)
    check_sample(fkl, logits, u, top_p=0.7)
    check_sample(fkl, torch.zeros(2, V), u)
    check_sample(fkl, torch.zeros(2, V), u, top_k=V - 3, top_p=0.5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad", [1, 3, 8])
def test_sample_strided_rows(fkl, dtype, pad):
    logits, u = lm_logits(7, 3001 + pad, 8, dtype)
    check_sample(fkl, logits[:, :3001], u, top_k=20)
    check_sample(fkl, logits[:, :3001], u, top_p=0.9)
    # a view that starts inside a row
    t, _ = fkl.sample(logits.cuda()[:, pad:], u.cuda(), top_p=0.9)
    t2, _ = fkl.sample(logits[:, pad:].contiguous().cuda(), u.cuda(), top_p=0.9)
    assert torch.equal(t, t2)


@pytest.mark.parametrize("B", [1, 2, 19, 37, 40, 77, 160, 333])
def test_sample_batches_with_settings_per_row(fkl, B):
    logits, u = lm_logits(B, 5003, B, torch.bfloat16)
    g = torch.Generator().manual_seed(B)
    t = torch.rand(B, generator=g) * 1.5
    t[::5] = 0
    k = torch.randint(0, 60, (B,), generator=g, dtype=torch.int32)
    p = torch.rand(B, generator=g) * 1.2
    m = torch.rand(B, generator=g) * 0.2 - 0.05
    check_sample(fkl, logits, u, temperature=t, top_k=k, top_p=p, min_p=m)


@pytest.mark.parametrize("kw", [dict(), dict(top_k=3), dict(top_p=0.5), dict(top_k=700, top_p=0.5), dict(min_p=0.5),
                                dict(temperature=0.0)])
@pytest.mark.parametrize("V", [40, 9001])
def test_sample_ties(fkl, V, kw):
    u = torch.tensor([0.0, 0.3, 0.999, 0.5])
    check_sample(fkl, torch.zeros(4, V), u, **kw)                       # all equal
    x = torch.zeros(4, V)
    x[:, 1::2] = -0.0                                                   # -0 and +0 are the same logit
    check_sample(fkl, x, u, **kw)
    x = torch.full((4, V), -1.0)
    x[:, 7::3] = 2.0                                                    # a third tied at the top
    check_sample(fkl, x, u, **kw)
    x = (torch.randint(0, 4, (4, V), generator=torch.Generator().manual_seed(V))).float()
    check_sample(fkl, x, u, **kw)                                       # four values


@pytest.mark.parametrize("kw", [dict(), dict(top_k=3), dict(top_p=0.5), dict(min_p=0.1), dict(temperature=0.0)])
def test_sample_special_values(fkl, kw):
    V = 3000
    x = torch.randn(12, V, generator=torch.Generator().manual_seed(4))
    inf, nan = float("inf"), float("nan")
    x[0] = -inf
    x[1] = nan
    x[2, :] = -inf
    x[2, 1234] = -5.0                              # one id left
    x[3, 100:] = -inf
    x[4, ::2] = nan
    x[5, 17] = inf
    x[6, [17, 2000]] = inf
    x[7] = torch.finfo(torch.float32).min          # masked with the type's lowest value
    x[7, 5] = 1.0
    x[8] = torch.finfo(torch.float32).min
    x[9, 0] = torch.finfo(torch.float32).max
    x[10] = -inf
    x[10, [V - 1, 0]] = 3.0
    x[11] *= 1e30
    u = torch.linspace(0, 0.99, 12)
    token = check_sample(fkl, x, u, **kw)
    assert token[0] == -1 and token[1] == -1 and token[2] == 1234 and token[5] == 17 and token[7] == 5


def test_sample_random_numbers_out_of_range(fkl):
    logits, _ = lm_logits(5, 500, 2)
    u = torch.tensor([-1.0, 1.0, 2.0, float("nan"), float("inf")])
    token, _ = fkl.sample(logits.cuda(), u.cuda())
    first, _ = fkl.sample(logits.cuda(), torch.zeros(5, device="cuda"))
    assert token[0] == first[0] and token[3] == first[3]
    assert ((token >= 0) & (token < 500)).all()


def test_sample_frequencies(fkl):
    # 40000 draws of one row: every id's share within 5 standard deviations of its probability
    V, B = 12, 40000
    x = torch.randn(V, generator=torch.Generator().manual_seed(1))
    u = torch.rand(B, generator=torch.Generator().manual_seed(2))
    token, logprob = fkl.sample(x.cuda().expand(B, V).contiguous(), u.cuda(), temperature=0.8)
    p = torch.softmax(x.double() / 0.8, 0)
    share = torch.bincount(token.cpu().long(), minlength=V).double() / B
    assert ((share - p).abs() <= 5 * (p * (1 - p) / B).sqrt()).all()
    assert (logprob.cpu().double() - p.log()[token.cpu().long()]).abs().max() < 2e-6


def test_sample_empty_batch(fkl):
    t, lp = fkl.sample(torch.empty(0, 100, device="cuda"), torch.empty(0, device="cuda"))
    assert t.shape == (0,) and lp.shape == (0,)


# ---------------------------------------------------------------- the step as a whole
def test_draw_token_streams_and_graph(fkl):
    g = torch.Generator().manual_seed(5)
    W = torch.randn(5000, 256, generator=g) * 0.05
    wq, ws = fkl.quantize_int8(W.cuda())
    for M in (1, 12, 40, 300):
        h = torch.randn(M, 256, generator=g).to(torch.bfloat16).cuda()
        u = torch.rand(M, generator=g).cuda()
        ref = fkl.draw_token(h, wq, ws, u, temperature=0.9, top_k=40, top_p=0.95)
        torch.cuda.synchronize()
        side = [torch.cuda.Stream() for _ in range(2)]
        got = []
        for s in side:
            with torch.cuda.stream(s):
                got.append(fkl.draw_token(h, wq, ws, u, temperature=0.9, top_k=40, top_p=0.95))
        torch.cuda.synchronize()
        for t, lp in got:
            assert torch.equal(t, ref[0]) and torch.equal(lp, ref[1])
        work = fkl.Workspace("cuda")
        logits = torch.empty(M, 5000, device="cuda")
        hs, us = h.clone(), u.clone()
        s = side[0]
        with torch.cuda.stream(s):
            fkl.draw_token(hs, wq, ws, us, temperature=0.9, top_k=40, top_p=0.95, logits=logits, workspace=work)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                out = fkl.draw_token(hs, wq, ws, us, temperature=0.9, top_k=40, top_p=0.95, logits=logits,
                                     workspace=work)
        torch.cuda.synchronize()
        for _ in range(2):
            h2 = torch.randn(M, 256, generator=g).to(torch.bfloat16).cuda()
            hs.copy_(h2)
            graph.replay()
            torch.cuda.synchronize()
            want = fkl.draw_token(h2, wq, ws, u, temperature=0.9, top_k=40, top_p=0.95)
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


# ---------------------------------------------------------------- refusals
def test_refusals(fkl):
    c = dict(device="cuda")
    x = torch.zeros(4, 64, **c)
    wq, ws = torch.zeros(10, 64, dtype=torch.int8, **c), torch.zeros(10, **c)
    xq, xs = torch.zeros(4, 64, dtype=torch.int8, **c), torch.zeros(4, **c)
    u = torch.zeros(4, **c)
    with pytest.raises(ValueError):
        fkl.quantize_int8(x[0])
    with pytest.raises(ValueError):
        fkl.quantize_int8(x.t())
    with pytest.raises(TypeError):
        fkl.quantize_int8(x.double())
    with pytest.raises(ValueError):
        fkl.quantize_int8(x.cpu())
    with pytest.raises(ValueError):
        fkl.int8_linear(x, wq[:, :32], ws)
    with pytest.raises(ValueError):
        fkl.int8_linear(x, wq.float(), ws)
    with pytest.raises(ValueError):
        fkl.int8_linear(x, wq, ws.double())
    with pytest.raises(ValueError):
        fkl.int8_linear(x, wq, ws[:5])
    with pytest.raises(TypeError):
        fkl.int8_linear(x, wq, ws, out_dtype=torch.int32)
    with pytest.raises(ValueError):
        fkl.int8_linear(x, wq, ws, out=torch.zeros(4, 11, **c))
    with pytest.raises(ValueError):
        fkl.int8_linear(x, wq, ws, out=torch.zeros(10, 4, **c).t())
    with pytest.raises(fkl.FklError):  # K not a multiple of 16
        fkl.int8_linear(torch.zeros(4, 40, **c), torch.zeros(10, 40, dtype=torch.int8, **c), ws)
    with pytest.raises(fkl.FklError) as e:  # rows of a view that do not start on 16 bytes
        flat = torch.zeros(10 * 64 + 1, dtype=torch.int8, **c)[1:].view(10, 64)
        fkl.int8_linear(x, flat, ws)
    assert e.value.status == 2
    with pytest.raises(ValueError):
        fkl.int8_matmul(xq.float(), xs, wq, ws)
    with pytest.raises(ValueError):
        fkl.int8_matmul(xq, xs[:3], wq, ws)
    with pytest.raises(ValueError):
        fkl.sample(x, u[:3])
    with pytest.raises(ValueError):
        fkl.sample(x, u.double())
    with pytest.raises(ValueError):
        fkl.sample(x, u.cpu())
    with pytest.raises(ValueError):
        fkl.sample(x.t(), u)
    with pytest.raises(ValueError):
        fkl.sample(x[:1].expand(4, 64), u)
    with pytest.raises(TypeError):
        fkl.sample(x.to(torch.int32), u)
    with pytest.raises(ValueError):
        fkl.sample(x, u, top_k=torch.zeros(4, **c))
    with pytest.raises(ValueError):
        fkl.sample(x, u, temperature=torch.zeros(3, **c))
    with pytest.raises(fkl.FklError):
        fkl.sample(torch.zeros(1, 2 ** 22 + 1, **c), u[:1])
    with pytest.raises(fkl.FklError):
        fkl.sample(torch.zeros(4, 0, **c), u)


def test_host_memory_is_refused(fkl):
    import ctypes

    from lm_head_top_tcgen05_gb300._lib import FklSampleParams, lib

    L = lib()
    x = torch.zeros(4, 64, device="cuda")
    host = torch.zeros(4, pin_memory=True)
    tok = torch.zeros(4, dtype=torch.int32, device="cuda")
    p = FklSampleParams(temperature=1.0, top_p=1.0)
    st = L.fkl_sample(x.data_ptr(), 0, 4, 64, 64, host.data_ptr(), ctypes.byref(p), tok.data_ptr(), None, None)
    assert st == 1 and b"u is not" in L.fkl_last_error()
    q = torch.zeros(4, 64, dtype=torch.int8, device="cuda")
    st = L.fkl_quantize_int8(x.data_ptr(), 0, 4, 64, 64, q.data_ptr(), host.data_ptr(), None)
    assert st == 1 and b"scale" in L.fkl_last_error()
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    s = torch.zeros(4, device="cuda")
    st = L.fkl_int8_matmul(q.data_ptr(), s.data_ptr(), q.data_ptr(), host.data_ptr(), 4, 4, 64, 0, x.data_ptr(), 4,
                           ws.data_ptr(), ws.numel(), None)
    assert st == 1 and b"w_scale" in L.fkl_last_error()


# ---------------------------------------------------------------- paths that sizes and values choose
@pytest.mark.parametrize("kw", [dict(temperature=1000.0, top_p=0.5), dict(temperature=1000.0, top_k=9000),
                                dict(temperature=1e-3, top_p=0.9), dict(top_k=600, top_p=0.7, min_p=1e-4),
                                dict(top_k=513), dict(top_k=512, top_p=0.3), dict(top_p=1e-6), dict(min_p=1e-6, top_p=0.9),
                                dict(temperature=1e30, top_p=0.4), dict(temperature=float("inf"), top_p=0.4),
                                dict(temperature=1e-30)])
@pytest.mark.parametrize("V,dtype", [(20011, torch.float32), (151936, torch.bfloat16), (700001, torch.float16),
                                     (700001, torch.float32)])
def test_sample_paths(fkl, V, dtype, kw):
    # lists, histograms in z, exact histograms, rows too long for shared memory
    logits, u = lm_logits(2, V, V % 1000, dtype)
    if kw.get("temperature", 1.0) > 1e20 and dtype == torch.float32:
        logits[0, 5] = 3e38                      # z underflows to 0 for all others
    check_sample(fkl, logits, u, **kw)


@pytest.mark.parametrize("scale", [0.0, 1e-6, 0.01, 1.0, 30.0])
@pytest.mark.parametrize("p", [0.05, 0.5, 0.9, 0.999])
def test_sample_top_p_of_flat_and_sharp_rows(fkl, scale, p):
    g = torch.Generator().manual_seed(int(p * 1000))
    logits = torch.randn(4, 30011, generator=g) * scale
    check_sample(fkl, logits, torch.rand(4, generator=g), top_p=p)


def test_sample_rows_do_not_disturb_each_other(fkl):
    # the same row alone and inside a batch with rows of other kinds
    logits, u = lm_logits(12, 9001, 3)
    logits[3] = float("-inf")
    logits[5] = 0
    kw = dict(temperature=torch.linspace(0, 2, 12), top_k=torch.arange(12, dtype=torch.int32) * 100,
              top_p=torch.linspace(0.5, 1.1, 12), min_p=torch.linspace(0, 0.1, 12))
    dk = {n: v.cuda() for n, v in kw.items()}
    t, lp = fkl.sample(logits.cuda(), u.cuda(), **dk)
    for b in range(12):
        t1, lp1 = fkl.sample(logits[b:b + 1].cuda(), u[b:b + 1].cuda(), **{n: v[b:b + 1] for n, v in dk.items()})
        assert t1[0] == t[b] and (lp1[0] == lp[b] or (t[b] == -1 and torch.isnan(lp[b])))


@pytest.mark.parametrize("N", [1, 255, 256, 257, 19456, 19457, 20000, 40000])
@pytest.mark.parametrize("M", [1, 4, 5, 16])
def test_int8_matmul_waves(fkl, M, N):
    # around whole waves of CTA pairs (76 x 256 channels) and of the streaming kernel's warps
    ops = operands(M, N, 144, N + M)
    assert_product(fkl.int8_matmul(*dev(*ops)), ops, torch.float32)


@pytest.mark.parametrize("M,N,K", [(1, 300, 98304), (2, 70, 49168), (3, 40, 131072), (20, 300, 131072), (4, 17, 24592)])
def test_int8_matmul_deep(fkl, M, N, K):
    # the streaming kernel's tokens no longer fit shared memory beyond M * K = 96 K
    rng = np.random.default_rng(K)
    xq = rng.integers(-3, 4, (M, K)).astype(np.int8)   # sums stay below 2^24: exact
    wq = rng.integers(-3, 4, (N, K)).astype(np.int8)
    one, w1 = np.full(M, 0.5, np.float32), np.full(N, 0.25, np.float32)
    y = fkl.int8_matmul(*dev(xq, one, wq, w1)).double().cpu().numpy()
    np.testing.assert_array_equal(y, og.int8_matmul(xq, one, wq, w1))


def test_int8_linear_default_workspaces_of_two_streams(fkl):
    # calls queued on two streams do not share the module's workspace
    g = torch.Generator().manual_seed(9)
    wq, ws = fkl.quantize_int8((torch.randn(6000, 512, generator=g) * 0.02).cuda())
    xs = [torch.randn(64, 512, generator=g).cuda() for _ in range(2)]
    ref = [fkl.int8_linear(x, wq, ws) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(fkl.int8_linear(xs[i], wq, ws))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, ref[i]) for y in got[i])


def test_int8_linear_from_threads_of_one_stream(fkl):
    # two threads on the default stream, tiles that are cut along K: each gets its own product
    import threading

    g = torch.Generator().manual_seed(10)
    wq, ws = fkl.quantize_int8((torch.randn(4096, 2880, generator=g) * 0.02).cuda())
    xs = [torch.randn(9, 2880, generator=g).cuda() for _ in range(2)]
    ref = [fkl.int8_linear(x, wq, ws) for x in xs]
    torch.cuda.synchronize()
    got, start = [[], []], threading.Barrier(2)

    def work(i):
        start.wait()
        for _ in range(300):
            got[i].append(fkl.int8_linear(xs[i], wq, ws, out=torch.full((9, 4096), 7.0, device="cuda")))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 300 and all(torch.equal(y, ref[i]) for y in got[i])


def test_graph_with_the_default_workspace(fkl):
    # captured after a warm-up, replayed after a larger call and with the memory that the warm-up's
    # workspace had in other hands
    g = torch.Generator().manual_seed(11)
    wq, ws = fkl.quantize_int8((torch.randn(4096, 2880, generator=g) * 0.02).cuda())
    x, u = torch.randn(9, 2880, generator=g).cuda(), torch.rand(9, generator=g).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(s):
        fkl.draw_token(x, wq, ws, u, top_k=40)
        for _ in range(2):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1], stream=s):
                out = fkl.draw_token(x, wq, ws, u, top_k=40), fkl.int8_linear(x, wq, ws)
        many = torch.randn(2000, 2880, generator=g).cuda()
        fkl.int8_linear(many, wq, ws)
        others = [torch.full((2 ** 20,), 5, dtype=torch.int32, device="cuda") for _ in range(64)]
    s.synchronize()
    for _ in range(2):
        x.copy_(torch.randn(9, 2880, generator=g))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        (token, logprob), y = out
        want = fkl.draw_token(x, wq, ws, u, top_k=40)
        assert torch.equal(token, want[0]) and torch.equal(logprob, want[1])
        assert torch.equal(y, fkl.int8_linear(x, wq, ws))
        assert all((t == 5).all() for t in others)


def _late(fkl, ops, dtype, out, workspace, limit_ms, late_ms):
    from lm_head_top_tcgen05_gb300._lib import DTYPES, lib

    (M, K), N = ops[0].shape, ops[2].shape[0]
    buf = workspace.get(lib().fkl_int8_matmul_workspace_size(M, N, K), "cuda")
    st = lib().fkl_test_int8_matmul_late(*[t.data_ptr() for t in ops], M, N, K, DTYPES[dtype], out.data_ptr(),
                                         out.stride(0), limit_ms * 10 ** 6, late_ms * 10 ** 6, buf.data_ptr(),
                                         buf.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0


# Few tokens with cut tiles, whole tiles in several rounds, tiles of more than 128 tokens.
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(9, 4096, 2880), (5, 21001, 272), (300, 513, 1040), (200, 19500, 1456)])
def test_product_whose_tokens_come_too_late(fkl, M, N, K, dtype):
    # every wait runs out after 20 ms; the tokens are there after 200
    ops = operands(M, N, K, M + N)
    t, ws = dev(*ops), fkl.Workspace("cuda")
    big = torch.full((M, N + 6), 7.0, dtype=dtype, device="cuda")
    _late(fkl, t, dtype, big[:, 3:N + 3], ws, 20, 200)
    assert fkl.read_status(ws) == 8  # FKL_ERR_TIMEOUT
    assert torch.isnan(big[:, 3:N + 3]).all()
    assert (big[:, :3] == 7).all() and (big[:, N + 3:] == 7).all()
    token, logprob = fkl.sample(big[:, 3:N + 3], torch.rand(M, device="cuda"))
    assert (token == -1).all() and torch.isnan(logprob).all()
    # in time, and the usual call in the same workspace
    _late(fkl, t, dtype, big[:, 3:N + 3], ws, 1000, 1)
    assert fkl.read_status(ws) == 0
    assert_product(big[:, 3:N + 3], ops, dtype)
    assert_product(fkl.int8_matmul(*t, out_dtype=dtype, workspace=ws), ops, dtype)
    assert fkl.read_status(ws) == 0


def test_status_of_the_default_workspace(fkl, monkeypatch):
    monkeypatch.setattr(fkl, "_default_ws", {})  # no loss call before
    ops = dev(*operands(8, 300, 64, 1))
    fkl.int8_matmul(*ops)
    buf = fkl.default_workspace(torch.device("cuda", torch.cuda.current_device()))
    buf[0] = 4                                   # the bit that a wait that runs out sets
    assert fkl.read_status(device="cuda") == 8
    fkl.int8_matmul(*ops)
    assert buf[0] == 0


@pytest.mark.parametrize("kw", [dict(top_k=600), dict(top_k=17000), dict(top_p=0.02), dict(top_p=0.5), dict(top_p=0.97),
                                dict(top_k=9000, top_p=0.3, min_p=0.9)])
def test_sample_logits_at_the_edges_of_bins(fkl, kw):
    # logits at the edges of 1/2048 of a histogram's bin (1/64 of a halving), and next to them;
    # some thousands to a bin, more than one list holds
    V, width = 40000, np.log(2.0) / 64
    g = torch.Generator().manual_seed(12)
    x = (-torch.randint(0, 8 * 2048, (4, V), generator=g).double() * width / 2048).float()
    step = torch.randint(-1, 2, (4, V), generator=g)
    x = torch.where(step == 0, x, torch.nextafter(x, torch.where(step > 0, 1.0, -1.0))).clamp(max=0)
    x[:, 5] = 0
    check_sample(fkl, x, torch.rand(4, generator=g), **kw)
