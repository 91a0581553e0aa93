"""Layer steps under a loss scale: eager ones follow the dynamic scaler through
an overflow, captured ones take a static scale and refuse a dynamic one."""
import pytest
import torch

from gradient_reduce_adam_amd import driver

pytestmark = pytest.mark.gpu

V, D, T = 20, 16, 50


class Table:
    """One embedding whose f16 gradient rows are multiplied by the loss scale."""

    def __init__(self, scaler, init_scale, n=1):
        g = torch.Generator().manual_seed(1)
        self.d = driver.DPStep((V * D,), n, 1, "f16", "f16", scaler=scaler, init_scale=init_scale, backoff=0.5,
                               growth_interval=1000, weight_decay=0.0, stream=torch.cuda.Stream())
        self.ids = [torch.randint(0, V, (T,), generator=g).cuda() for _ in range(n)]
        # multiples of 1/8 up to 1.75: exact under every power-of-two scale below the overflow, and so are their sums
        self.dy = [(torch.randint(-14, 15, (T, D), generator=g) / 8).half().cuda() for _ in range(n)]
        self.ws = torch.empty(self.d.plan.embed_workspace(0, D, T), dtype=torch.uint8, device="cuda")
        self.scales = []
        torch.cuda.synchronize()

    def backward(self, step, k, first, scale):
        self.scales.append(scale)
        with torch.cuda.stream(self.d.stream):
            self.d.plan.accumulate_embed(0, self.ids, [x * scale for x in self.dy], first, self.ws)

    def want(self):
        total = torch.zeros((V, D), dtype=torch.float64, device="cuda")
        for ids, dy in zip(self.ids, self.dy):
            total.index_add_(0, ids, dy.double())
        return total.flatten() / len(self.ids)


def test_eager_steps_follow_the_dynamic_scale():
    m = Table("dynamic", 2.0 ** 16)  # 1.75 * 2^16 is beyond f16
    first = m.d.step_layers(m.backward)
    assert first["found_inf"] and first["t"] == 0 and first["scale"] == 2.0 ** 15
    second = m.d.step_layers(m.backward)
    assert m.scales == [2.0 ** 16, 2.0 ** 15]
    assert not second["found_inf"] and second["t"] == 1
    assert torch.equal(m.d.gbar.double() / 2.0 ** 15, m.want())
    assert abs(second["norm"] - m.want().norm().item()) <= 1e-6 * second["norm"]
    with pytest.raises(ValueError, match="dynamic"):
        m.d.capture_layers(m.backward)
    assert m.d.step_layers(m.backward)["t"] == 2  # the refusal left the step as it was
    m.d.close()


def test_captured_steps_keep_a_static_scale():
    eager, graph = Table("static", 256.0, n=2), Table("static", 256.0, n=2)
    for m in (eager, graph):
        m.d.step_layers(m.backward)
    replay = graph.d.capture_layers(graph.backward)
    for k in range(3):
        torch.cuda.synchronize()
        for m in (eager, graph):
            for x in m.dy:
                x.neg_()
        torch.cuda.synchronize()
        replay.replay()
        eager.d.step_layers(eager.backward)
        torch.cuda.synchronize()
        assert torch.equal(eager.d.gbar, graph.d.gbar) and torch.equal(eager.d.master, graph.d.master)
        assert torch.equal(graph.d.gbar.double() / 256.0, graph.want())
    assert graph.d.read_state()["t"] == 4
    eager.d.close()
    graph.d.close()
