"""Plans destroyed while a stream capture is under way, by another thread or
under a side stream that is no part of it: the capture stays whole, and the
destruction waits for the plan's work as ever."""
import threading

import pytest
import torch

import gradient_reduce_adam_amd as dp

pytestmark = pytest.mark.gpu

V, D, T = 16, 8, 40


class Table:
    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.plan, self.acc = dp.Plan((V * D,), 1, "bf16", "bf16"), torch.full((V * D,), -7.0, device="cuda")
        self.param = torch.ones(V * D, dtype=torch.bfloat16, device="cuda")
        self.plan.bind("acc", self.acc)
        self.plan.bind("param", self.param)
        self.ids = torch.randint(0, V, (T,), generator=g).cuda()
        self.dy = torch.randn((T, D), generator=g).bfloat16().cuda()
        self.ws = torch.zeros(self.plan.embed_workspace(0, D, T), dtype=torch.uint8, device="cuda")

    def call(self):
        self.plan.accumulate_embed(0, [self.ids], [self.dy], True, self.ws)


def forward_only(t):
    t.plan.embed(0, t.ids, torch.empty((T, D), dtype=torch.bfloat16, device="cuda"))


def with_memory(t):
    t.plan.bind_tensors("param", [t.param])  # a pointer-table ring: device and pinned memory
    t.call()


def in_another_thread(plan):
    error = []

    def run():
        try:
            plan.__del__()
        except Exception as e:  # pragma: no cover
            error.append(e)

    thread = threading.Thread(target=run)
    thread.start()
    thread.join()
    assert not error


def under_a_side_stream(plan):
    with torch.cuda.stream(torch.cuda.Stream()):
        plan.__del__()


@pytest.mark.parametrize("how", [in_another_thread, under_a_side_stream], ids=["thread", "side-stream"])
@pytest.mark.parametrize("use", [forward_only, with_memory], ids=["forward-only", "with-memory"])
def test_a_capture_survives_a_plan_destroyed_beside_it(use, how):
    kept, old = Table(1), Table(2)
    use(old)
    kept.call()
    torch.cuda.synchronize()
    want = kept.acc.clone()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        kept.call()
        how(old.plan)
        kept.call()
    assert old.plan.handle == 0
    for _ in range(3):
        kept.acc.fill_(-7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept.acc, want)
    kept.plan.close()


@pytest.mark.parametrize("use", [forward_only, with_memory], ids=["forward-only", "with-memory"])
def test_destruction_waits_for_the_device(use):
    t = Table(3)
    use(t)
    stream, event = torch.cuda.Stream(), torch.cuda.Event()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        torch.cuda._sleep(int(5e7))
        event.record()
    t.plan.close()
    assert event.query()
