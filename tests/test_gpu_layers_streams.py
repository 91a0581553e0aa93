"""Layer steps on a stream of their own whose backward pass names no stream:
eager steps and captured ones treat it alike, and both are ordered with the
caller's stream."""
import pytest
import torch

from test_gpu_layers_step import AT, Model, NAMES

pytestmark = pytest.mark.gpu


class Plain(Model):
    """The model's backward pass as a caller writes it who leaves streams to the step."""

    def backward(self, step, k, first, loss_scale):
        assert torch.cuda.current_stream() == self.stream
        mine, self.stream = self.stream, torch.cuda.current_stream()
        super().backward(step, k, first, loss_scale)
        self.stream = mine


def test_step_against_autodiff_without_naming_a_stream():
    m = Plain(2, 2, 130, True, seed=21)
    # the gradients of this step are written on the caller's stream right before it, behind a long wait there
    fresh = torch.randn(m.dout.shape, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    m.dout.fill_(float("nan"))
    torch.cuda.synchronize()
    torch.cuda._sleep(int(5e7))
    m.dout.copy_(fresh)
    m.d.step_layers(m.backward, sync_scale=False)
    got = m.d.gbar.double()  # on the caller's stream, without a synchronisation
    m.dout.zero_()           # and the caller may write the step's inputs again
    torch.cuda.synchronize()
    m.dout.copy_(fresh)
    want = m.want()
    for k in NAMES:
        x, y = m.tensor(got, k), m.tensor(want, k)
        assert (x - y).norm() <= 1e-3 * y.norm(), (k, AT[k])
    m.d.close()


def test_eager_and_captured_steps_agree_without_naming_a_stream():
    eager, graph = Plain(2, 2, 100, True, seed=9), Plain(2, 2, 100, True, seed=9)
    for m in (eager, graph):
        m.d.step_layers(m.backward)
    replay = graph.d.capture_layers(graph.backward)
    for k in range(3):
        fresh = torch.randn(graph.dout.shape, generator=torch.Generator().manual_seed(k)).bfloat16().cuda()
        torch.cuda.synchronize()
        for m in (eager, graph):
            m.dout.copy_(fresh)
        torch.cuda.synchronize()
        replay.replay()
        eager.d.step_layers(eager.backward, sync_scale=False)
        torch.cuda.synchronize()
        assert torch.equal(eager.d.master, graph.d.master) and torch.equal(eager.d.param, graph.d.param)
    assert graph.d.read_state()["t"] == 4
    eager.d.close()
    graph.d.close()
