"""What the layer operators promise around their calls, on the host: which
workspaces they ask for, which calls they refuse or take, and how the binding
behaves without torch and beside a stream capture."""
import ctypes
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

dp = pytest.importorskip("gradient_reduce_adam_amd")
from gradient_reduce_adam_amd import layers as L  # noqa: E402


def test_norm_workspace_holds_the_sums_of_biases():
    """A bias needs two more column sums a workgroup, whether or not the mean is subtracted."""
    with dp.Plan((10,) * 5, 2) as plan:
        ask = lambda centered, **b: plan.block_norm_workspace(  # noqa: E731
            dp.BlockNorm(pre_w=0, post_w=2, centered=centered, **b), 10, 64)
        plain, full = ask(False), ask(True)
        assert full == 2 * plain
        for b in (dict(pre_b=1), dict(post_b=3), dict(pre_b=1, post_b=3, gate=4)):
            assert ask(False, **b) == full and ask(True, **b) == full
        assert ask(False, gate=4) == plain
