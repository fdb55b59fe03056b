"""The on-policy example with the teacher's cache in few bits and an entropy bonus."""
import pytest

pytestmark = pytest.mark.gpu

SMALL = ["--steps", "2", "--batch", "6", "--length", "20", "--vocab", "3000", "--width", "128"]


@pytest.mark.parametrize("more", [["--cache-bits", "8"], ["--cache-bits", "4", "--entropy", "0.01"]])
def test_on_policy_example(cuda_device, more):
    from lm_head_top_tcgen05_gb300 import build

    build.build()
    from examples import on_policy

    losses = on_policy.main(SMALL + more)
    assert len(losses) == 2
    assert all(l == l and l > 0 for l in losses)
