"""GPU: the example that runs the operators around the layer together."""
import os
import runpy

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_residual_block_learns_and_serves():
    main = runpy.run_path(os.path.join(ROOT, "examples", "residual_block.py"))["main"]
    losses, off = main(steps=20, verbose=False)
    # steps against the gradient: each lowers the loss, together by a tenth at least
    assert all(b < a for a, b in zip(losses, losses[1:])) and losses[-1] < 0.9 * losses[0], losses
    # 16 levels over a group's range of about 4.5 sigma: an error of 0.087 sigma a weight, three products in a row
    assert off < 0.25, off
