"""The example that runs the low-bit projections, the rotation, the 8-bit cache and its
attention together."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [
    dict(), dict(hidden=1024, heads=8, kv_heads=8, page=16, prompts=(5, 130, 17), steps=10, seed=3),
])
def test_layer_serves_prompts_and_steps(kw):
    """A block's values are off by up to half a step of its largest / 127 (about 4.5 standard deviations):
    1% of their size, keys and values alike, and up to as much again where a block's step grew
    token by token: below 3% of the outputs."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from examples import attention_layer

    error, same = attention_layer.main(verbose=False, **kw)
    assert same
    assert error < 0.03
