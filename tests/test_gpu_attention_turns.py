"""Queries that see many keys beside others of their workgroup that see none: more queries than keys under a causal mask, in
workgroups of eight waves whose halves take turns.  The definition on the GPU."""
import pytest

from test_gpu_attention import Case, cut

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("spans,spans_k,H,K,D,dt,window", [
    (cut(4000), cut(3600), 48, 2, 72, "bf16", 0), (cut(4200), cut(3700), 32, 4, 128, "f16", 1800),
    (cut(3900), cut(3599), 40, 1, 96, "bf16", 0), (cut(300, 8000), cut(7000, 300), 16, 1, 104, "bf16", 0)])
def test_queries_that_see_none_beside_others(spans, spans_k, H, K, D, dt, window):
    c = Case(spans, H, K, D, dt, seed=D, spans_k=spans_k, causal=True, window=window, device="cuda")
    c.check(**c.places())
    for (a, b), (e, f) in zip(spans, spans_k):
        none = max(0, (b - a) - (f - e))
        assert (c.out[a:a + none] == 0).all() and (c.lse[:, a:a + none] == -float("inf")).all() and (c.dq[a:a + none] == 0).all()
