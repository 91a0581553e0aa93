"""The step driver's layer steps on the host: under which stream the caller's
backward pass runs and what orders it, and what a capture refuses.  The step is
assembled around stand-ins for the plan and the streams; nothing touches a
GPU."""
import contextlib

import pytest

driver = pytest.importorskip("gradient_reduce_adam_amd.driver")


class Stream:
    def __init__(self, name, log, handle):
        self.name, self.log, self.cuda_stream = name, log, handle

    def wait_stream(self, other):
        self.log.append(f"{self.name} waits for {other.name}")


class Plan:
    def __init__(self, log):
        self.log = log

    def __getattr__(self, name):
        return lambda *args, **kw: self.log.append(name)


def step_on(monkeypatch, same=False, n=2, a=2, scaler="none"):
    log = []
    mine = Stream("step", log, 7)
    current = [mine if same else Stream("caller", log, 0)]

    @contextlib.contextmanager
    def stream(s):
        before, current[0] = current[0], s
        try:
            yield
        finally:
            current[0] = before

    monkeypatch.setattr(driver.torch.cuda, "stream", stream)
    monkeypatch.setattr(driver.torch.cuda, "current_stream", lambda *device: current[0])
    d = object.__new__(driver.DPStep)
    d.n, d.a, d.partials, d.single_pass, d.offload = n, a, False, False, "direct"
    d.lr, d.eps, d.weight_decay, d.max_norm = 1e-3, 1e-8, 0.0, 0.0
    d.scaler, d.scale, d.steps_done = scaler, 1.0, 0
    d.plan, d.stream, d.device, d.shards = Plan(log), mine, None, [(0, 4)]
    return d, log, current


def test_a_capture_under_a_dynamic_loss_scale_is_refused(monkeypatch):
    """The recorded backward pass would keep the loss scale of the capture, while the update divides by the
    device's, which an overflow or a growth interval changes."""
    d, log, _ = step_on(monkeypatch, scaler="dynamic")
    monkeypatch.setattr(driver.torch.cuda, "CUDAGraph", lambda: pytest.fail("a capture began"))
    with pytest.raises(ValueError, match="dynamic"):
        d.capture_layers(lambda *args: log.append("backward"))
    assert log == []


def test_backward_runs_on_the_steps_stream_in_the_callers_order(monkeypatch):
    """The calls of a backward pass that names no stream go to the step's stream, behind what the caller issued
    before the step; what the caller issues after it waits for the step."""
    d, log, current = step_on(monkeypatch)
    d.issue_layers(lambda step, k, first, scale: log.append(f"backward {k} on {current[0].name}"), 1)
    assert log == ["step waits for caller", "backward 1 on step", "backward 2 on step", "reduce_replicas",
                   "grad_stats", "adam_step", "caller waits for step"]
    assert current[0].name == "caller"


def test_a_step_on_the_current_stream_waits_for_nothing(monkeypatch):
    """Also the form that a capture on the step's stream records: no stream waits for itself."""
    d, log, current = step_on(monkeypatch, same=True, n=1, a=1)
    d.issue_layers(lambda step, k, first, scale: log.append(f"backward {k} on {current[0].name}"), 1)
    assert log == ["backward 1 on step", "grad_stats", "adam_step"]


def test_the_caller_waits_for_a_step_that_failed_half_way(monkeypatch):
    """Its buffers may still be read on the step's stream when the exception reaches it."""
    d, log, current = step_on(monkeypatch)

    def backward(step, k, first, scale):
        if k == 2:
            raise RuntimeError("lost")
        log.append("backward")

    with pytest.raises(RuntimeError, match="lost"):
        d.issue_layers(backward, 1)
    assert log == ["step waits for caller", "backward", "caller waits for step"] and current[0].name == "caller"
