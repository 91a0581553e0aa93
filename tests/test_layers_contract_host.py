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


WITHOUT_TORCH = """
import sys
sys.modules["torch"] = None  # import torch raises ImportError
import gradient_reduce_adam_amd as dp

destroyed = []
real = dp.dp_plan_destroy
dp.dp_plan_destroy = lambda handle: (destroyed.append(handle), real(handle))
p = dp.Plan((60, 10, 10), 1)
norms = dp.BlockNorm(pre_w=1, pre_b=2, centered=True)
assert p.embed_workspace(0, 6, 40) > 0 and p.linear_workspace(64, 6, 10, 0) == 0
assert p.block_norm_workspace(norms, 10, 4) > 0
for call in (lambda: p.embed(0, None, None), lambda: p.block_norm(norms, None, None, None),
             lambda: p.accumulate_embed(0, [None], [None], True, None),
             lambda: p.accumulate_block_norm(norms, None, None, None, None, None, None, True, None),
             lambda: p.accumulate_linear(0, [None], [None], [None], True),
             lambda: dp.dpl_pack_activations(None, None, None), lambda: dp.dpl_unpack_activations(None, None, None)):
    try:
        call()
    except ImportError as e:
        assert "torch" in str(e)
    else:
        raise AssertionError("no ImportError")
handle = p.handle
del p
assert destroyed == [handle] and dp._abandoned == []
print("fine")
"""


def test_the_package_works_without_torch():
    """Without torch the package imports, plans and workspace queries work, a finalised plan is destroyed, and
    the calls that take torch tensors say what they lack."""
    r = subprocess.run([sys.executable, "-c", WITHOUT_TORCH], capture_output=True, text=True, cwd=ROOT, timeout=120)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr


def test_an_abandoned_plan_that_another_thread_destroys_first(monkeypatch):
    """Between the look at the list and the pop another thread may have emptied it."""
    monkeypatch.setattr(dp, "_abandoned", [0])

    def other_thread():
        dp._abandoned.clear()
        return False

    monkeypatch.setattr(dp, "_capturing", other_thread)
    with dp.Plan((4,), 1) as p:
        assert p.handle


def test_abandoned_plans_are_destroyed_at_the_next_call_that_synchronises(monkeypatch):
    """Not only where another plan is made: closing a plan and reading its state do it too."""
    destroyed = []
    monkeypatch.setattr(dp, "_abandoned", [])
    monkeypatch.setattr(dp, "_capturing", lambda: False)
    monkeypatch.setattr(dp, "dp_read_state", lambda handle, stream: {"t": 3})
    plan, other = dp.Plan((4,), 1), dp.Plan((5,), 1)
    real = dp.dp_plan_destroy
    monkeypatch.setattr(dp, "dp_plan_destroy", lambda h: (destroyed.append(h), real(h)))
    for call in (lambda: plan.read_state(), lambda: plan.close()):
        h = dp.dp_plan_create((6,), 1, "bf16", "bf16")
        dp._abandoned.append(h)
        call()
        assert h in destroyed and dp._abandoned == []
    other.close()
    assert len(destroyed) == 4


def test_block_norm_of_no_rows_takes_any_strides():
    """Without rows the addresses may all be null, which makes s no tensor in place of h or y."""
    with dp.Plan((8, 8), 1) as plan:
        plan.bind("param", 1 << 20)
        norms = ctypes.byref(L.Norms(-1, -1, -1, 0, -1, 0, 8, 1e-5, 1.0))
        for lds in (8, 9):
            status = dp.lib.dpl_block_norm(plan.handle, norms, 0, dp.DP_BF16, None, 8, None, 8, None, lds, None, 8, None)
            assert status != dp.DP_ERR_INVALID_ARG, dp.lib.dp_last_error()
