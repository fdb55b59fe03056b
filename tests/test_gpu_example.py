"""The on-policy example runs the generation operators and the loss together."""
import pytest

pytestmark = pytest.mark.gpu


def test_on_policy_example(cuda_device):
    from lm_head_top_tcgen05_gb300 import build

    build.build()
    from examples import on_policy

    losses = on_policy.main(["--steps", "4", "--batch", "6", "--length", "20", "--vocab", "3000", "--width", "128"])
    assert len(losses) == 4
    assert all(l == l and l > 0 for l in losses)
