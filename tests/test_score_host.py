"""The scoring and cache entry points refuse bad arguments on the host, before touching CUDA."""
import pytest
import torch

INVALID, ALIGN, WS = 1, 2, 4
HUGE = 2 ** 31


@pytest.fixture(scope="module")
def L():
    from lm_head_top_tcgen05_gb300 import build
    from lm_head_top_tcgen05_gb300._lib import lib

    build.build()
    return lib()


def test_token_logprobs_is_checked(L):
    def call(x=16, t=0, B=4, V=100, ld=100, tok=16, size=8, mask=16, T=1.0, rows=None, n=5, lp=16, ent=16, stats=None,
             ids=16, logs=16):
        return L.fkl_token_logprobs(x, t, B, V, ld, tok, size, mask, T, rows, n, lp, ent, stats, ids, logs, None)

    assert call(t=3) == INVALID and call(t=-1) == INVALID
    assert call(B=-1) == INVALID and call(B=HUGE) == INVALID
    assert call(V=0, ld=0) == INVALID and call(V=2 ** 22 + 1, ld=2 ** 23) == INVALID and call(ld=99) == INVALID
    for name in ("x", "tok", "lp", "ent", "ids", "logs"):
        assert call(**{name: None}) == INVALID, name
    assert call(size=2) == INVALID and call(size=0) == INVALID
    assert call(n=-1) == INVALID and call(n=129, V=1000, ld=1000) == INVALID and call(n=6, V=5, ld=5) == INVALID
    for T in (0.0, -1.0, float("inf"), float("nan")):
        assert call(T=T) == INVALID
    assert call(x=18) == ALIGN and call(x=17, t=1) == ALIGN and call(tok=20) == ALIGN and call(tok=18, size=4) == ALIGN
    assert call(rows=18) == ALIGN and call(lp=18) == ALIGN and call(stats=18) == ALIGN and call(ids=18) == ALIGN


def test_token_logprobs_backward_is_checked(L):
    def call(x=16, t=1, B=4, V=100, ld=100, tok=16, size=4, mask=None, T=1.0, rows=None, stats=16, ent=16, ga=16, gb=None,
             dx=16, ldd=100):
        return L.fkl_token_logprobs_backward(x, t, B, V, ld, tok, size, mask, T, rows, stats, ent, ga, gb, dx, ldd, None)

    assert call(t=7) == INVALID and call(ldd=99) == INVALID and call(ld=99) == INVALID and call(size=3) == INVALID
    for name in ("x", "tok", "stats", "ent", "dx"):
        assert call(**{name: None}) == INVALID, name
    assert call(T=0.0) == INVALID
    assert call(dx=17) == ALIGN and call(ga=18) == ALIGN and call(gb=18) == ALIGN and call(stats=18) == ALIGN


def test_fused_sizes_and_checks(L):
    n, nb = L.fkl_logprob_workspace_size, L.fkl_logprob_backward_workspace_size
    assert n(256, 256, 4096) > 0 and n(0, 8, 1) > 0 and nb(256, 256, 4096, 64, 0) > 0
    assert n(256, 12, 4096) == 0 and n(-1, 16, 4096) == 0 and n(4, 16, 0) == 0 and nb(4, 16, 10, 0, 0) == 0
    assert nb(256, 256, 4096, 64, 1) > nb(256, 256, 4096, 64, 0)  # the fp32 sums of dH
    # no T x V tensor: far below one of bf16
    assert n(32768, 2880, 201088) < 2 ** 25 and nb(32768, 2880, 201088, 2048, 1) < 32768 * 201088 * 2 / 8

    def fwd(H=16, W=16, tok=16, size=4, mask=None, T=256, d=256, V=4096, tau=1.0, lp=16, ent=16, lse=16, ws=256,
            nbytes=1 << 30):
        return L.fkl_logprob_forward(H, W, tok, size, mask, T, d, V, tau, lp, ent, lse, ws, nbytes, None)

    def bwd(H=16, W=16, tok=16, size=4, mask=None, lp=16, ent=16, lse=16, ga=16, gb=16, T=256, d=256, V=4096, tau=1.0, chunk=64,
            bf16=0, acc=0, dH=16, dW=16, ws=256, nbytes=1 << 40):
        return L.fkl_logprob_backward(H, W, tok, size, mask, lp, ent, lse, ga, gb, T, d, V, tau, chunk, bf16, acc, dH, dW, ws,
                                      nbytes, None)

    for f in (fwd, bwd):
        assert f(d=12) == INVALID and f(T=-1) == INVALID and f(V=0) == INVALID and f(tau=0.0) == INVALID
        assert f(tau=float("nan")) == INVALID and f(size=1) == INVALID
        assert f(H=None) == INVALID and f(W=None) == INVALID and f(tok=None) == INVALID and f(lse=None) == INVALID
        assert f(H=24) == ALIGN and f(W=24) == ALIGN and f(tok=18) == ALIGN and f(lse=18) == ALIGN
        assert f(ws=None) == WS and f(nbytes=64) == WS and f(ws=128) == ALIGN
        assert f(lp=None) == INVALID and f(ent=None) == INVALID and f(lp=18) == ALIGN
    assert bwd(chunk=0) == INVALID and bwd(bf16=2) == INVALID and bwd(acc=4) == INVALID and bwd(bf16=1, acc=1) == INVALID
    assert bwd(dH=None, dW=None) == INVALID and bwd(dH=24) == ALIGN and bwd(dW=24) == ALIGN and bwd(ga=18) == ALIGN


def test_cache_is_checked(L):
    w = L.fkl_cache_words
    assert w(100, 201088, 8) * 4 == 360 and w(100, 201088, 4) * 4 == 312
    assert w(0, 10, 8) == 0 and w(1025, 10, 8) == 0 and w(5, 0, 8) == 0 and w(5, 2 ** 30 + 1, 8) == 0 and w(5, 10, 6) == 0

    def pack(i=16, z=16, T=4, K=10, V=100, bits=8, r=16):
        return L.fkl_cache_pack(i, z, T, K, V, bits, r, None)

    def unpack(i=16, z=16, T=4, K=10, V=100, bits=8, r=16):
        return L.fkl_cache_unpack(r, T, K, V, bits, i, z, None)

    for f in (pack, unpack):
        assert f(T=-1) == INVALID and f(T=HUGE) == INVALID and f(K=0) == INVALID and f(K=1025) == INVALID
        assert f(V=0) == INVALID and f(bits=2) == INVALID
        for name in ("i", "z", "r"):
            assert f(**{name: None}) == INVALID and f(**{name: 18}) == ALIGN, name


@pytest.mark.parametrize("K,V,bits", [(1, 1, 8), (32, 255, 4), (33, 256, 8), (1024, 2 ** 30, 4)])
def test_cache_words_are_the_oracles(L, K, V, bits):
    from oracle import score

    assert L.fkl_cache_words(K, V, bits) == score.cache_words(K, V, bits)


def test_binding_refuses_on_the_host():
    import lm_head_top_tcgen05_gb300 as fkl

    x, tok = torch.zeros(2, 5), torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError):
        fkl.token_logprobs(x, tok)  # host tensors
    with pytest.raises(ValueError):
        fkl.token_logprobs(x, tok, top_n=129)
    with pytest.raises(TypeError):
        fkl.fused_logprobs(torch.zeros(2, 8), torch.zeros(5, 8), tok)
    with pytest.raises(ValueError):
        fkl.logprob_backward(x, x, tok, None, x, x, x, accumulate=True)
    with pytest.raises(ValueError):
        fkl.logprob_backward(x, x, tok, None, x, x, x, grad_dtype=torch.float16)
    with pytest.raises(ValueError):
        fkl.quantize_cache(torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3), 10)
    data = torch.zeros(6, 4, dtype=torch.int32)
    cache = fkl.QuantizedCache(data, K=3, V=5, bits=4)
    assert len(cache) == 6 and len(cache[2:5]) == 3 and cache[2:5].data.data_ptr() == data[2].data_ptr()
    assert fkl.QuantizedCache(**cache.state()).K == 3
    with pytest.raises(ValueError):
        fkl.QuantizedCache(data, K=40, V=5, bits=4)  # another record length
    with pytest.raises(ValueError):
        fkl.dequantize_cache(cache)  # on the host
    with pytest.raises(TypeError):
        cache[1]
    with pytest.raises(TypeError):
        cache[::2]
    with pytest.raises(ValueError):
        fkl.forward(x, x, cache, torch.zeros(6, 3))  # logits beside a cache
