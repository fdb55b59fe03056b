"""The teacher cache in few bits: records bit by bit against the oracle, and the loss that reads them."""
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


def make(T, K, V, seed=0):
    r = np.random.default_rng(seed)
    z = np.sort((r.standard_normal((T, K)) * 3 + 8).astype(np.float32), axis=1)[:, ::-1].copy()
    z[r.random((T, K)) < 0.02] = -np.inf
    return r.integers(0, V, (T, K)).astype(np.int32), z


def check(fkl, ids, z, V, bits):
    cache = fkl.quantize_cache(torch.tensor(ids).cuda(), torch.tensor(z).cuda(), V, bits)
    want = oracle.cache_pack(ids, z, V, bits)
    got = cache.data.cpu().numpy().view(np.uint32)
    nan = np.isnan(want[:, :2 * -(-ids.shape[1] // 32)].view(np.float32))
    same = got == want
    same[:, :nan.shape[1]] |= nan & np.isnan(got[:, :nan.shape[1]].view(np.float32))  # a NaN's payload is free
    assert same.all(), np.argwhere(~same)[:5]
    got_ids, got_z = fkl.dequantize_cache(cache)
    ids2, z2 = oracle.cache_unpack(want, ids.shape[1], V, bits)
    assert (got_ids.cpu().numpy() == ids2).all()
    np.testing.assert_array_equal(got_z.cpu().numpy(), z2)
    return cache


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("T,K,V", [(1, 1, 1), (3, 5, 2), (9, 31, 7), (8, 32, 8), (7, 33, 255), (20, 64, 65535),
                                   (33, 100, 201088), (5, 257, 50261), (2, 1024, 2 ** 30), (4, 1000, 2 ** 30 - 1)])
def test_records(fkl, T, K, V, bits):
    check(fkl, *make(T, K, V, seed=K), V, bits)


@pytest.mark.parametrize("bits", [4, 8])
def test_special_rows(fkl, bits):
    inf, nan = np.inf, np.nan
    ids, z = make(16, 70, 100, seed=3)
    z[0] = -inf
    z[1, 40:] = -inf                      # a group without a logit
    z[2, 3] = nan
    z[3, 66] = inf
    z[4] = 2.5                            # one value
    z[5, 1:] = -3.4e38                    # the type's lowest value does not widen the steps
    z[6, 0], z[6, 1] = 5000.0, 5000.0 - 4096.0
    z[7] = np.arange(70, dtype=np.float32)             # every logit a level or a tie between two
    z[8] = np.arange(70, dtype=np.float32) * 0.5
    z[9] *= np.float32(1e-38)             # subnormal differences
    z[10] *= np.float32(1e-44)
    z[11] = 3e38
    z[12] = -3e38
    z[13] = -0.0
    z[14, ::2] = 0.0
    ids[15, :3] = [-1, 100, 2 ** 31 - 1]
    check(fkl, ids, z, 100, bits)


def test_levels_next_to_a_tie(fkl):
    """Logits next to the middle of two levels, at either side of it, and on it."""
    step = np.float32(0.125)
    half = (np.arange(32 * 40, dtype=np.float32) % 254 + np.float32(0.5)) * step
    z = np.empty((40, 32), dtype=np.float32)
    for i, (lo, up) in enumerate([(0, 0), (1, 0), (0, 1)]):
        v = half.reshape(40, 32).copy()
        v = np.nextafter(v, np.float32(-np.inf)) if lo else np.nextafter(v, np.float32(np.inf)) if up else v
        z[:] = -v
        z[:, 0], z[:, 1] = 0.0, -254 * step
        check(fkl, np.zeros((40, 32), np.int32), z, 10, 8)
        check(fkl, np.zeros((40, 32), np.int32), z, 10, 4)


def test_many_rows(fkl):
    """The largest long-context cache: sampled rows against the oracle, the error of all of them."""
    T, K, V = 262144, 100, 201088
    g = torch.Generator(device="cuda").manual_seed(0)
    z = torch.sort(torch.randn(T, K, generator=g, device="cuda") * 3 + 8, dim=1, descending=True).values
    ids = torch.randint(0, V, (T, K), generator=g, device="cuda").int()
    cache = fkl.quantize_cache(ids, z, V)
    got_ids, got = fkl.dequantize_cache(cache)
    assert torch.equal(got_ids, ids)
    for a in range(0, K, 32):
        part, back = z[:, a:a + 32], got[:, a:a + 32]
        half = (part.amax(1) - part.amin(1)) / 508
        # half a step, and three float roundings of at most the largest magnitude
        assert ((part - back).abs().amax(1) <= half * (1 + 2.0 ** -20) + part.abs().amax(1) * 2.0 ** -22).all()
        assert torch.equal(part.amax(1), back.amax(1))
    rows = torch.tensor([0, 1, T // 2, T - 2, T - 1])
    want = oracle.cache_pack(ids[rows.cuda()].cpu().numpy(), z[rows.cuda()].cpu().numpy(), V, 8)
    assert (cache.data[rows.cuda()].cpu().numpy().view(np.uint32) == want).all()
    part = cache[1000:1003]
    i2, z2 = fkl.dequantize_cache(part)
    assert torch.equal(i2, ids[1000:1003]) and torch.equal(z2, got[1000:1003])


@pytest.mark.parametrize("K", [4, 7, 100])
def test_any_alignment(fkl, K):
    """Tensors and records that start anywhere."""
    T, V = 37, 5000
    ids, z = make(T, K, V, seed=K)
    want = oracle.cache_pack(ids, z, V, 8)
    W = want.shape[1]
    for off in (0, 1, 2, 3):
        i = torch.empty(off + T * K, dtype=torch.int32, device="cuda")[off:].view(T, K)
        f = torch.empty(off + T * K, device="cuda")[off:].view(T, K)
        i.copy_(torch.tensor(ids))
        f.copy_(torch.tensor(z))
        got = fkl.quantize_cache(i, f, V)
        assert (got.data.cpu().numpy().view(np.uint32) == want).all()
        data = torch.empty(off + T * W, dtype=torch.int32, device="cuda")[off:].view(T, W)
        data.copy_(got.data)
        i.zero_()
        f.zero_()
        fkl.dequantize_cache(fkl.QuantizedCache(data, K, V, 8), out=(i, f))
        assert (i.cpu().numpy() == ids).all()
        np.testing.assert_array_equal(f.cpu().numpy(), oracle.cache_unpack(want, K, V, 8)[1])


def test_empty_and_out(fkl):
    cache = fkl.quantize_cache(torch.zeros(0, 5, dtype=torch.int32).cuda(), torch.zeros(0, 5).cuda(), 10)
    assert len(cache) == 0 and fkl.dequantize_cache(cache)[0].shape == (0, 5)
    ids, z = make(6, 40, 50)
    cache = fkl.quantize_cache(torch.tensor(ids).cuda(), torch.tensor(z).cuda(), 50)
    big = torch.full((8, 40), 7, dtype=torch.int32).cuda(), torch.full((8, 40), 7.0).cuda()
    fkl.dequantize_cache(cache, out=(big[0][:6], big[1][:6]))
    assert (big[0][6:] == 7).all() and (big[1][6:] == 7).all()  # rows behind the last stay as they were
    assert torch.equal(big[0][:6].cpu(), torch.tensor(ids))


def test_refusals(fkl):
    i, z = torch.zeros(2, 3, dtype=torch.int32).cuda(), torch.zeros(2, 3).cuda()
    with pytest.raises(TypeError):
        fkl.quantize_cache(i.long(), z, 10)
    with pytest.raises(TypeError):
        fkl.quantize_cache(i, z.half(), 10)
    with pytest.raises(ValueError):
        fkl.quantize_cache(i, z[:, :2], 10)
    with pytest.raises(ValueError):
        fkl.quantize_cache(i.t().contiguous().t(), z, 10)
    with pytest.raises(fkl.FklError):
        fkl.quantize_cache(i, z, 10, bits=5)
    with pytest.raises(fkl.FklError):
        fkl.quantize_cache(i, z, 0)
    c = fkl.quantize_cache(i, z, 10)
    with pytest.raises(ValueError):
        fkl.dequantize_cache(c, out=(i[:1], z[:1]))
    with pytest.raises(ValueError):
        fkl.fused_kl(torch.zeros(2, 8).bfloat16().cuda(), torch.zeros(10, 8).bfloat16().cuda(), c, z)


# ---------------------------------------------------------------- with the loss
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("divergence", ["kl", "jsd"])
def test_the_loss_reads_it(fkl, bits, divergence):
    """teacher_cache -> fused_kl: bit for bit the loss of the unpacked slots, and near that of the teacher's own."""
    g = torch.Generator(device="cuda").manual_seed(bits)
    T, d, V, K = 300, 128, 5003, 50
    Ht, Wt = (torch.randn(n, d, generator=g, device="cuda").bfloat16() for n in (T, V))
    H0, W0 = torch.randn(T, d, generator=g, device="cuda").bfloat16(), (torch.randn(V, d, generator=g, device="cuda") * 0.1).bfloat16()
    mask = torch.rand(T, generator=g, device="cuda") > 0.2
    cache = fkl.teacher_cache(Ht, Wt, K, bits=bits)
    assert cache.K == K and cache.V == V and len(cache) == T
    idx, z = fkl.teacher_topk(Ht, Wt, K)
    assert torch.equal(fkl.dequantize_cache(cache)[0], idx)

    def step(*teacher):
        H, W = H0.clone().requires_grad_(), W0.clone().requires_grad_()
        loss = fkl.fused_kl(H, W, *teacher, mask=mask, divergence=divergence)
        loss.backward()
        return loss.detach(), H.grad, W.grad

    a, b, c = step(cache), step(*fkl.dequantize_cache(cache)), step(idx, z)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    # Each slot's logit is off by e <= half its 32 slots' step, so the teacher's probabilities are off by a factor within
    # exp(+-2e) and the divergence by at most 2e times the spread of log(p/q), which is below 60 here.
    step_of = max(((z[:, k:k + 32].amax(1) - z[:, k:k + 32].amin(1)).max().item() for k in range(0, K, 32))) / (2 ** bits - 2)
    assert abs(a[0] - c[0]) <= np.expm1(step_of) * 60
    loss, lse = fkl.forward(H0, W0, cache, mask=mask, divergence=divergence)
    assert torch.equal(loss, a[0])
    # a micro-batch takes its rows of the cache
    n = fkl.local_count(mask, T)
    parts = [fkl.fused_kl(H0[s].contiguous(), W0, cache[s], mask=mask[s].contiguous(), divergence=divergence, global_count=n)
             for s in (slice(0, 130), slice(130, T))]
    assert abs(sum(parts).item() - a[0].item()) <= 1e-3 * a[0].item()


def test_a_failed_row_reaches_the_loss(fkl):
    H, W = torch.randn(4, 16).bfloat16().cuda(), torch.randn(40, 16).bfloat16().cuda()
    ids, z = torch.randint(0, 40, (4, 6)).int().cuda(), torch.randn(4, 6).cuda()
    bad = ids.clone()
    bad[2, 3] = -1
    ws = fkl.Workspace()
    loss, _ = fkl.forward(H, W, fkl.quantize_cache(bad, z, 40), workspace=ws)
    assert torch.isnan(loss) and fkl.read_status(ws) == 6
    nan = z.clone()
    nan[1, 0] = float("nan")
    loss, _ = fkl.forward(H, W, fkl.quantize_cache(ids, nan, 40), workspace=ws)
    assert torch.isnan(loss)
