"""Gradients from hidden states where the backward has several token blocks and several vocabulary slabs at once, in
either loop order, with and without a last block that is padded.  Tolerances as in test_gpu_score_fused.py."""
import ctypes

import pytest
import torch

from tests.test_gpu_score_fused import Exact, make

D = 64
# tokens, vocabulary, chunk, tokens of the last block (below 64: padded)
SHAPES = [(1000, 1500, 300, 488), (1100, 2000, 200, 332), (1056, 1800, 300, 32), (1068, 2700, 200, 44)]


def plan(T, V, chunk):
    """(tokens of a block, blocks, slabs, whether the slabs are the outer loop with bf16 gradients)."""
    from lm_head_top_tcgen05_gb300._lib import lib

    out = (ctypes.c_int64 * 5)()
    assert lib().fkl_test_backward_plan(T, D, V, 1, chunk, 152, ctypes.cast(out, ctypes.c_void_p)) == 0
    Ct, nt, _, nslabs, Vmax = out
    # the fp32 sums of bf16 gradients: all of dH and a slab of dW, or a block of dH and all of dW
    return Ct, nt, nslabs, nt > 1 and T + Vmax < Ct + V


@pytest.fixture(scope="module")
def fkl():
    from lm_head_top_tcgen05_gb300 import build

    build.build()
    import lm_head_top_tcgen05_gb300 as m

    return m


@pytest.mark.parametrize("T,V,chunk,last", SHAPES)
def test_the_shapes_have_blocks_and_slabs(fkl, T, V, chunk, last):
    Ct, nt, nslabs, outer = plan(T, V, chunk)
    assert T > chunk and nt > 1 and nslabs > 1 and outer and T - (nt - 1) * Ct == last


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])  # slabs outer; token blocks outer
@pytest.mark.parametrize("T,V,chunk,last", SHAPES)
def test_blocks_and_slabs(fkl, cuda_device, T, V, chunk, last, dtype):
    H, W, tok, mask = make(T, D, V, seed=T)
    tok[:40] = 11  # a row that many tokens of several blocks share
    tok[-40:] = 11
    a, b = torch.randn(T).cuda(), torch.randn(T).cuda() * 0.3
    for m in (None, mask):
        e = Exact(H, W, tok, m, 1.0)
        lp, ent, lse = fkl.logprob_forward(H, W, tok, m)
        e.check_scores(lp, ent)
        got = fkl.logprob_backward(H, W, tok, m, lp, ent, lse, a, b, chunk=chunk, grad_dtype=dtype)
        e.check_gradients(*got, a, b, dtype == torch.bfloat16)
        if dtype == torch.float32:
            half = fkl.logprob_backward(H, W, tok, m, lp, ent, lse, a, b, chunk=chunk, grad_dtype=torch.bfloat16)
            assert all(torch.equal(x.bfloat16(), y) for x, y in zip(got, half))  # the same sums in either order
            base = torch.randn(T, D).cuda(), torch.randn(V, D).cuda()
            out = fkl.logprob_backward(H, W, tok, m, lp, ent, lse, a, b, chunk=chunk, accumulate=True,
                                       out=(base[0].clone(), base[1].clone()))
            e.check_gradients(*out, a, b, False, base=tuple(x.cpu().double().numpy() for x in base))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V,chunk,last", SHAPES)
def test_rows_left_out_may_hold_anything(fkl, cuda_device, T, V, chunk, last, dtype):
    H, W, tok, mask = make(T, D, V, seed=T + 1)
    a, b = torch.randn(T).cuda(), torch.randn(T).cuda()
    bad = H.clone()
    bad[~mask] = torch.tensor([float("nan"), float("inf")], device="cuda").bfloat16().repeat(D // 2)
    outs = []
    for h in (H, bad):
        lp, ent, lse = fkl.logprob_forward(h, W, tok, mask)
        outs.append((lp, ent) + fkl.logprob_backward(h, W, tok, mask, lp, ent, lse, a, b, chunk=chunk, grad_dtype=dtype))
    for x, y in zip(*outs):
        assert torch.isfinite(y).all() and torch.equal(x, y)
