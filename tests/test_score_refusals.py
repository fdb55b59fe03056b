"""What the scoring operators cannot take is refused by the call that is given it."""
import pytest
import torch

INVALID, ALIGN = 1, 2


@pytest.fixture(scope="module")
def fkl():
    from lm_head_top_tcgen05_gb300 import build

    build.build()
    import lm_head_top_tcgen05_gb300 as m

    return m


def test_the_backward_needs_lse_or_statistics(fkl):
    from lm_head_top_tcgen05_gb300._lib import lib

    L = lib()

    def fwd(lse=None, stats=None):
        return L.fkl_logprob_forward_ex(16, 16, 16, 4, None, 256, 256, 4096, 1.0, 16, 16, lse, stats, 256, 1 << 30, None)

    def bwd(lse=None, stats=None):
        return L.fkl_logprob_backward_ex(16, 16, 16, 4, None, 16, 16, lse, stats, 16, 16, 256, 256, 4096, 1.0, 64, 0, 0, 16,
                                         16, 256, 1 << 40, None)

    assert bwd() == INVALID and b"stats" in L.fkl_last_error()
    for f in (fwd, bwd):
        assert f(stats=18) == ALIGN and f(lse=18) == ALIGN and f(lse=16, stats=18) == ALIGN


def test_a_temperature_that_wants_a_gradient(fkl):
    """It would get none: the scores are differentiable in the logits alone."""
    x, tok = torch.zeros(2, 5), torch.zeros(2, dtype=torch.int64)
    T = torch.ones(2, requires_grad=True)
    for logits in (x, x.clone().requires_grad_()):
        with pytest.raises(ValueError, match="temperature.*gradient"):
            fkl.token_logprobs(logits, tok, temperature=T)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):  # only the host tensor is wrong here
        fkl.token_logprobs(x, tok, temperature=T)


@pytest.mark.gpu
def test_a_chunk_that_the_backward_would_refuse(fkl, cuda_device):
    H = torch.randn(20, 64).bfloat16().cuda().requires_grad_()
    W, tok = torch.randn(100, 64).bfloat16().cuda(), torch.zeros(20, dtype=torch.int64).cuda()
    with pytest.raises(fkl.FklError):
        fkl.fused_logprobs(H, W, tok, chunk=0)
    with pytest.raises(fkl.FklError):
        fkl.fused_logprobs(H, W, tok, chunk=-5)


@pytest.mark.parametrize("T", [1e-39, 1e-45, 4e-39])
def test_a_temperature_whose_inverse_is_infinite(fkl, T):
    """log2(e) / T is what logits are multiplied by: from 4.25e-39 down it is no float."""
    from lm_head_top_tcgen05_gb300._lib import lib

    L = lib()

    def refused(status):
        return status == INVALID and b"inverse" in L.fkl_last_error()

    assert refused(L.fkl_token_logprobs(16, 0, 4, 100, 100, 16, 8, None, T, None, 0, 16, 16, None, None, None, None))
    assert refused(L.fkl_token_logprobs_backward(16, 0, 4, 100, 100, 16, 8, None, T, None, 16, 16, 16, None, 16, 100, None))
    assert refused(L.fkl_logprob_forward(16, 16, 16, 4, None, 256, 256, 4096, T, 16, 16, 16, 256, 1 << 30, None))
    assert refused(L.fkl_logprob_backward(16, 16, 16, 4, None, 16, 16, 16, 16, 16, 256, 256, 4096, T, 64, 0, 0, 16, 16, 256,
                                          1 << 40, None))
