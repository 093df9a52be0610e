"""The example that runs the router, the experts' packed products and the way back together."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [
    dict(), dict(hidden=320, inner=192, experts=40, k=6, tokens=65, steps=6, seed=3),
    dict(hidden=256, inner=128, experts=4, k=1, tokens=1500, steps=3, seed=5),
])
def test_layer_serves_a_prompt_and_steps(kw):
    """Roundings to bf16, 2^-8 of a value at most, 2^-8 / sqrt(3) in the mean of many: of h, of the experts' rows
    and of the result, which is up to 6 times the experts' share.  sqrt(1 + 1 + 36) 2^-8 / sqrt(3) < 5 2^-8."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from examples import experts_layer

    error, same = experts_layer.main(verbose=False, **kw)
    assert same
    assert error < 5 * 2.0 ** -8
