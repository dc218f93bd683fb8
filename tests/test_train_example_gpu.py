"""The training example: layer norm, the GEMMs, layer norm's gradient and the
orthogonalised update in one loop, which has to learn its target."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width,batch", [(256, 512), (200, 304)])
def test_example_learns(dtype, width, batch):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_projection
    finally:
        sys.path.pop(0)
    losses = train_projection.train(steps=80, width=width, batch=batch, dtype=dtype)
    # Weight and target start as independent matrices of equal size: a loss of
    # about 2.  Steps of singular values near lr, shrinking to zero, cover the
    # distance of at most 2 in each direction: 0.02 * 80 / 2 = 0.8 of it.
    assert 1.0 < losses[0] < 4.0
    assert losses[-1] < 0.5 * losses[0]
