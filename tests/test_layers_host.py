"""The layer operators' C interface on the host: the header is plain C, every
symbol is exported, workspace sizes are sane, and calls that the
documentation does not allow are refused before anything touches a GPU (the
addresses here are made up)."""
import copy
import ctypes
import dataclasses
import os
import pickle
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

dp = pytest.importorskip("gradient_reduce_adam_amd")
from gradient_reduce_adam_amd import layers as L  # noqa: E402

A = 1 << 20  # an aligned address that is never used
BIG = 1 << 40


@pytest.fixture
def plan():
    with dp.Plan((0, 60, 10, 10, 10, 1 << 20), 2, "bf16", "bf16") as p:
        p.bind("param", A)
        for r in range(2):
            p.bind("acc", A, r)
        yield p


def refused(status, call, *args):
    with pytest.raises(dp.DpError) as e:
        dp._check(call(*args))
    assert e.value.status == status, e.value
    return e.value.message


def bad(call, *args):
    return refused(dp.DP_ERR_INVALID_ARG, call, *args)


def ptrs(*xs):
    return (ctypes.c_void_p * len(xs))(*xs)


def test_header_is_plain_c_and_exports_match(tmp_path):
    text = open(os.path.join(ROOT, "include", "dplayer.h")).read()
    names = sorted(set(re.findall(r"^dp_status (dpl_\w+)\(", text, re.M)))
    assert sorted(L.EXPORTS) == names and len(names) == 10
    for n in names:
        assert hasattr(dp.lib, n)
    for k in ("DPL_MAX_NORM_DIM", "DPL_GROUP"):
        assert int(re.search(rf"#define {k} (\d+)", text).group(1)) == getattr(L, k)
    assert "INT64_C(1) << 24" in text and L.DPL_MAX_TOKENS == 1 << 24
    gcc = shutil.which("gcc")
    if not gcc:
        pytest.skip("needs gcc")
    src = tmp_path / "c.c"
    src.write_text('#include "dplayer.h"\nint main(void) { return (int)sizeof(dpl_norms) - (int)sizeof(dpl_norms); }\n')
    r = subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-fsyntax-only", "-D__HIP_PLATFORM_AMD__",
                        "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"), str(src)], capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stderr


def test_embed_refusals(plan):
    def call(tensor=1, id_bytes=8, dim=6, scale=1.0, tokens=3, ids=A, dtype=dp.DP_BF16, out=A, ld=6, handle=None):
        return dp.lib.dpl_embed(plan.handle if handle is None else handle,
                                ctypes.byref(L.Table(tensor, id_bytes, dim, scale)), tokens, ids, dtype, out, ld, None)

    for kw in (dict(handle=0), dict(tensor=-1), dict(tensor=6), dict(tensor=0), dict(dim=7), dict(dim=0), dict(dim=-6),
               dict(id_bytes=2), dict(scale=float("inf")), dict(scale=float("nan")), dict(scale=1e39),
               dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(dtype=3), dict(dtype=-1), dict(ids=None),
               dict(ids=A + 4), dict(ids=A + 2, id_bytes=4), dict(out=None), dict(out=A + 1), dict(ld=5),
               dict(ld=1 << 41)):
        assert "dpl_embed" in bad(lambda: call(**kw)), kw
    with dp.Plan((60,), 1) as unbound:
        refused(dp.DP_ERR_UNBOUND, lambda: call(handle=unbound.handle, tensor=0))


def test_accumulate_embed_refusals(plan):
    want = plan.embed_workspace(1, 6, 3)
    assert want > 0 and plan.embed_workspace(1, 6, 0) >= 0

    def call(ids=(A, A), dy=(A, A), tokens=3, dtype=dp.DP_BF16, ld=6, first=1, more=0, ws=A, size=want, p=plan, dim=6):
        return dp.lib.dpl_accumulate_embed(p.handle, ctypes.byref(L.Table(1, 8, dim, 1.0)), tokens,
                                           ptrs(*ids) if ids else None, dtype, ptrs(*dy) if dy else None, ld, first,
                                           more, ws, size, None)

    for kw in (dict(ids=None), dict(dy=None), dict(ids=(A, None)), dict(dy=(None, A)), dict(dy=(A, A + 1)),
               dict(dtype=7), dict(ld=5), dict(size=want - 1), dict(ws=None), dict(ws=A + 128), dict(tokens=-2),
               dict(dim=11)):
        bad(lambda: call(**kw))
    refused(dp.DP_ERR_STATE, lambda: call(first=0))  # no first micro-step yet
    with dp.Plan((1, 60), 2) as unbound:
        refused(dp.DP_ERR_UNBOUND, lambda: call(p=unbound))


def norms(post_w=-1, post_b=-1, gate=-1, pre_w=2, pre_b=-1, centered=0, dim=10, eps=1e-5, scale=1.0):
    return ctypes.byref(L.Norms(post_w, post_b, gate, pre_w, pre_b, centered, dim, eps, scale))


BAD_NORMS = (dict(dim=0), dict(dim=8193), dict(dim=11), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")),
             dict(eps=1e-60), dict(eps=float("inf")), dict(scale=float("inf")), dict(pre_w=1), dict(pre_w=6),
             dict(gate=2), dict(post_w=3, post_b=3), dict(post_b=3), dict(pre_w=-1, pre_b=3))


def test_block_norm_refusals(plan):
    def call(dtype=dp.DP_BF16, tokens=4, h=A, ldh=10, y=A, ldy=10, s=A, lds=10, x=2 * A, ldx=10, p=plan, **kw):
        return dp.lib.dpl_block_norm(p.handle, norms(**kw), tokens, dtype, h, ldh, y, ldy, s, lds, x, ldx, None)

    for kw in BAD_NORMS + (dict(dtype=dp.DP_F16), dict(dtype=9), dict(tokens=-1), dict(h=None), dict(y=None),
                           dict(s=None), dict(x=None), dict(ldh=9), dict(lds=11), dict(ldx=1), dict(x=A),
                           dict(pre_w=-1), dict(y=A + 1), dict(dtype=dp.DP_F32, s=A + 2, lds=10)):
        bad(lambda: call(**kw))
    with dp.Plan((1, 1, 10), 1) as unbound:
        refused(dp.DP_ERR_UNBOUND, lambda: call(p=unbound))


def test_block_norm_gradient_refusals(plan):
    size = ctypes.c_size_t()
    dp._check(dp.lib.dpl_block_norm_workspace(plan.handle, norms(gate=3), 4, ctypes.byref(size)))
    assert size.value > 0
    for kw in BAD_NORMS:
        bad(lambda: dp.lib.dpl_block_norm_workspace(plan.handle, norms(**kw), 4, ctypes.byref(size)))

    def call(rows=None, ld=10, tokens=4, dtype=dp.DP_BF16, ws=A, n=size.value, first=1, **kw):
        one = dict(s=A, y=2 * A, dx=3 * A, ds=4 * A, dh=5 * A, dy=6 * A)
        rows = [dict(one, **(r or {})) for r in (rows or (None, None))]
        arr = (L.NormRows * 2)(*[L.NormRows(**r) for r in rows])
        return dp.lib.dpl_accumulate_block_norm(plan.handle, norms(**dict(dict(gate=3), **kw)), tokens, dtype, arr, ld,
                                                first, 0, ws, n, None)

    both = lambda **kw: dict(rows=(kw, kw))  # noqa: E731
    for kw in (both(s=None), both(y=None), both(dx=None), dict(rows=(None, dict(ds=None))), dict(rows=(dict(dh=None), None)),
               both(dh=6 * A), both(dy=A), both(dh=2 * A), both(dx=3 * A + 1), dict(ld=9), dict(tokens=-1),
               dict(dtype=dp.DP_F16), dict(ws=None), dict(ws=A + 1), dict(n=size.value - 1),
               dict(pre_w=-1, **both(dx=None, ds=None)), dict(pre_w=-1), dict(pre_w=-1, gate=-1)):
        bad(lambda: call(**kw))
    refused(dp.DP_ERR_STATE, lambda: call(first=0))


def test_pack_refusals():
    def call(fn, tokens=3, dim=40, dtype=dp.DP_BF16, x=A, ld=40, codes=A, ldc=40, scales=A, lds=2):
        if fn == "pack":
            return dp.lib.dpl_pack_activations(tokens, dim, dtype, x, ld, codes, ldc, scales, lds, None)
        return dp.lib.dpl_unpack_activations(tokens, dim, dtype, codes, ldc, scales, lds, x, ld, None)

    for fn in ("pack", "unpack"):
        for kw in (dict(tokens=-1), dict(tokens=(1 << 24) + 1), dict(dim=0), dict(dim=(1 << 24) + 1), dict(dtype=5),
                   dict(x=None), dict(x=A + 1), dict(ld=39), dict(codes=None), dict(ldc=39), dict(scales=None),
                   dict(lds=1), dict(tokens=1 << 24, dim=1 << 12, ld=1 << 12, ldc=1 << 12, lds=1 << 7)):
            bad(lambda: call(fn, **kw))


def test_workspaces_serve_fewer_tokens(plan):
    """A workspace queried for some number of tokens is enough for any smaller one."""
    ts = [0, 1, 2, 63, 64, 65, 127, 128, 200, 512, 1000, 4095, 4096, 5000, 16384, 16385, 70000, 1 << 20, 1 << 24]
    for sizes in ([plan.embed_workspace(1, 6, t) for t in ts],
                  [plan.linear_workspace(t, 1024, 1024) for t in ts], [plan.linear_workspace(t, 6, 10, 1) for t in ts],
                  [plan.block_norm_workspace(dp.BlockNorm(pre_w=2, centered=True), 10, t) for t in ts]):
        assert sizes == sorted(sizes)
    assert plan.linear_workspace(1 << 24, 1024, 1024) <= 64 << 20


def test_norm_descriptions_copy_and_pickle():
    n = dp.BlockNorm(pre_w=2, gate=3, eps=1e-6, residual_scale=0.5)
    n.ref(10)
    for m in (copy.deepcopy(n), pickle.loads(pickle.dumps(n)), dataclasses.replace(n)):
        assert m == n and m.ref(10) is not n.ref(10)


def test_linear_refusals(plan):
    size = ctypes.c_size_t()
    ok = ctypes.byref(L.Linear(1, 0, 6, 10))
    dp._check(dp.lib.dpl_linear_workspace(plan.handle, ok, 4, ctypes.byref(size)))
    assert size.value == 0
    # few tiles and many tokens: split over workgroups, a copy of the matrix for each
    split = ctypes.byref(L.Linear(5, 0, 1024, 1024))
    dp._check(dp.lib.dpl_linear_workspace(plan.handle, split, 8192, ctypes.byref(size)))
    assert size.value % (4 * 2 << 20) == 0 and size.value > 4 * 2 << 20
    assert plan.linear_workspace(8192, 1024, 1024) == size.value

    def call(d=(1, 0, 6, 10), rows=((A, A, A), (A, A, A)), tokens=4, dtype=dp.DP_BF16, ldc=6, lds=1, ldd=10, first=1,
             ws=None, n=0):
        arr = (L.LinearRows * 2)(*[L.LinearRows(*r) for r in rows]) if rows else None
        return dp.lib.dpl_accumulate_linear(plan.handle, ctypes.byref(L.Linear(*d)), tokens, dtype, arr, ldc, lds, ldd,
                                            first, 0, ws, n, None)

    for kw in (dict(d=(1, 0, 6, 9)), dict(d=(1, 0, 0, 60)), dict(d=(1, 0, -6, -10)), dict(d=(0, 0, 1, 1)),
               dict(d=(6, 0, 6, 10)), dict(tokens=-1), dict(dtype=dp.DP_F32), dict(rows=None), dict(ldc=5),
               dict(lds=0), dict(ldd=9), dict(rows=((A, A, A), (None, A, A))), dict(rows=((A, None, A), (A, A, A))),
               dict(rows=((A, A, A + 1), (A, A, A))),
               dict(d=(5, 0, 1024, 1024), tokens=8192, ldc=1024, lds=32, ldd=1024, ws=A, n=size.value - 1),
               dict(d=(5, 0, 1024, 1024), tokens=8192, ldc=1024, lds=32, ldd=1024, ws=None, n=size.value)):
        bad(lambda: call(**kw))
    refused(dp.DP_ERR_STATE, lambda: call(first=0))


def test_a_plan_finalised_during_a_capture_is_destroyed_after_it(monkeypatch):
    plan = dp.Plan((4,), 1)
    handle = plan.handle
    monkeypatch.setattr(dp, "_capturing", lambda: True)
    plan.__del__()
    assert plan.handle == 0 and dp._abandoned == [handle]
    with dp.Plan((5,), 1):  # still within it
        assert dp._abandoned == [handle]
    monkeypatch.setattr(dp, "_capturing", lambda: False)
    with dp.Plan((6,), 1):
        assert dp._abandoned == []
