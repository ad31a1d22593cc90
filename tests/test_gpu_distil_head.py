"""The layer operators together: a ZeRO-3 unit gathered in 4 bits, its forward
and backward, and its chained step (examples/distil_head.py)."""
import math
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_the_loss_falls_at_every_step():
    """The same batches every step and a small learning rate: Adam descends."""
    import distil_head
    losses, chain = distil_head.run(steps=20)
    assert all(math.isfinite(x) for x in losses)
    assert all(b < a for a, b in zip(losses, losses[1:]))
    assert chain.applied == 20 and chain.skipped == 0

