"""The C interfaces of the attention, its positions and the distillation loss on the host: the headers are plain C,
every symbol is exported, and calls that the documentation does not allow are refused before anything touches a GPU
(the addresses here are made up)."""
import copy
import ctypes
import os
import pickle
import re
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

dp = pytest.importorskip("gradient_reduce_adam_amd")
from gradient_reduce_adam_amd import attention as A  # noqa: E402
from gradient_reduce_adam_amd import distill as D  # noqa: E402

P = 1 << 20  # an aligned address that is never used


def refused(status):
    assert status == dp.DP_ERR_INVALID_ARG, dp.lib.dp_last_error()
    return dp.lib.dp_last_error().decode()


@pytest.mark.parametrize("header,module,count", [("dpattn.h", A, 4), ("dploss.h", D, 1)])
def test_headers_are_plain_c_and_exports_match(tmp_path, header, module, count):
    text = open(os.path.join(ROOT, "include", header)).read()
    names = sorted(set(re.findall(r"^dp_status (dp[ad]_\w+)\(", text, re.M)))
    assert sorted(module.EXPORTS) == names and len(names) == count
    for n in names:
        assert hasattr(dp.lib, n)
    for name, shift, plain in re.findall(r"#define (DP[AD]_MAX_\w+) (?:\(INT64_C\(1\) << (\d+)\)|(\d+))", text):
        assert getattr(module, name) == (1 << int(shift) if shift else int(plain)), name
    gcc = shutil.which("gcc")
    if not gcc:
        pytest.skip("needs gcc")
    src = tmp_path / "c.c"
    sizes = {"dpattn.h": ("dpa_rows", "dpa_rotary_desc", "dpa_rotary_rows", "dpa_attention_desc"), "dploss.h": ("dpd_distill_desc",)}
    structs = {"dpa_rows": A.Rows, "dpa_rotary_desc": A.RotaryDesc, "dpa_rotary_rows": A.RotaryRows,
               "dpa_attention_desc": A.AttentionDesc, "dpd_distill_desc": D.DistillDesc}
    checks = "".join(f"typedef char ok_{s}[sizeof({s}) == {ctypes.sizeof(structs[s])} ? 1 : -1];\n" for s in sizes[header])
    src.write_text(f'#include "{header}"\n{checks}int main(void) {{ return 0; }}\n')
    r = subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-Wno-unused-local-typedefs", "-fsyntax-only",
                        "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"), str(src)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_packed_structs_have_the_layout_of_c():
    """The binding packs the structs of a call as bytes."""
    assert A._DESC.size == ctypes.sizeof(A.AttentionDesc) and A._ROWS.size == ctypes.sizeof(A.Rows)
    assert A._ROTARY_ROWS.size == ctypes.sizeof(A.RotaryRows) and D._DESC.size == ctypes.sizeof(D.DistillDesc)
    assert [x.size for x in A._ROTARY_CALL] == [i * ctypes.sizeof(A.RotaryRows) for i in range(A.DPA_MAX_TENSORS + 1)]
    d = A.AttentionDesc.from_buffer_copy(A._DESC.pack(8, 2, 64, 1, 100, 0.5, 7, 9, 3, 40, 48, 4, 2))
    assert [getattr(d, k) for k, _ in d._fields_] == [8, 2, 64, 1, 100, 0.5, 7, 9, 3, 40, 48, 4, 2]


def desc(heads=4, kv_heads=2, dim=64, causal=1, window=0, scale=0.125, tokens=32, tokens_k=32, sequences=1, offsets=None,
         offsets_k=None, offset_bytes=4, step=1):
    return A.AttentionDesc(heads, kv_heads, dim, causal, window, scale, tokens, tokens_k, sequences, offsets, offsets_k,
                           offset_bytes, step)


def rows(n, d=64, p=P, ld=None, head=None):
    return A.Rows(p, n * d if ld is None else ld, d if head is None else head)


BAD_DESC = (dict(heads=0), dict(heads=1025, kv_heads=1), dict(kv_heads=0), dict(heads=3), dict(heads=-4, kv_heads=-2), dict(dim=0),
            dict(dim=-8), dict(dim=60), dict(dim=136), dict(window=-1), dict(scale=0.0), dict(scale=-1.0),
            dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e-46), dict(scale=1e39), dict(tokens=-1),
            dict(tokens=(1 << 24) + 1), dict(tokens_k=-1), dict(sequences=-1), dict(sequences=5), dict(sequences=(1 << 24) + 1),
            dict(offsets=P, tokens_k=31), dict(offsets=P, offset_bytes=3), dict(offsets=P, step=3), dict(offsets=P + 2),
            dict(offsets_k=P + 4, offset_bytes=8), dict(tokens_k=33, sequences=2), dict(tokens=1 << 24, tokens_k=1 << 24, heads=1024),
            dict(offsets=P, sequences=1 << 23, heads=1, kv_heads=1), dict(offsets=P, sequences=1 << 17, heads=64, kv_heads=64, dim=128))


def forward(d=None, dtype=dp.DP_BF16, q=None, k=None, v=None, out=None, lse=P, handle=True):
    # an address each, for the rows of one call lie side by side only in the packed buffers
    r = [q or rows(4), k or rows(2, p=2 * P), v or rows(2, p=3 * P), out or rows(4, p=4 * P)]
    return dp.lib.dpa_attention(ctypes.addressof(d or desc()) if handle else None, dtype, *[ctypes.addressof(x) for x in r], lse, None)


def test_attention_refusals():
    for kw in BAD_DESC:
        d = desc(**kw)
        assert "dpa_attention" in refused(forward(d)), kw
    for kw in (dict(dtype=dp.DP_F32), dict(dtype=3), dict(handle=False), dict(lse=None), dict(lse=P + 2), dict(q=rows(4, p=None)),
               dict(k=rows(2, p=P + 1)), dict(v=rows(2, ld=-1)), dict(q=rows(4, head=-64)), dict(q=rows(4, ld=1 << 31)),
               dict(out=rows(4, p=4 * P, ld=255)), dict(out=rows(4, p=4 * P, head=63)), dict(out=rows(4, p=4 * P, ld=0)),
               dict(out=rows(4)), dict(out=rows(4, p=2 * P)), dict(out=rows(4, p=3 * P)), dict(q=rows(4, head=1 << 37))):
        assert "dpa_attention" in refused(forward(**kw)), kw
    # null arguments
    d = desc()
    assert refused(dp.lib.dpa_attention(ctypes.addressof(d), dp.DP_BF16, None, None, None, None, P, None))


def backward(d=None, change=None, ws=9 * P, size=4 * 4 * 32, lse=P, dtype=dp.DP_F16):
    r = [rows(4), rows(2), rows(2), rows(4), rows(4), rows(4), rows(2), rows(2)]
    for i, x in enumerate(r):
        x.p = (i + 1) * P
    if change:
        r[change[0]] = change[1]
    a = [ctypes.addressof(x) for x in r]
    return dp.lib.dpa_attention_backward(ctypes.addressof(d or desc()), dtype, *a[:4], lse, *a[4:], ws, size, None)


def test_backward_refusals():
    for kw in BAD_DESC:
        d = desc(**kw)
        assert "dpa_attention_backward" in refused(backward(d)), kw
    for kw in (dict(ws=None), dict(size=511), dict(ws=9 * P + 128), dict(lse=None), dict(dtype=dp.DP_F32),
               dict(change=(0, rows(4, p=None))), dict(change=(4, rows(4, p=P + 1))), dict(change=(5, rows(4, p=P))),
               dict(change=(5, rows(4, p=5 * P))), dict(change=(6, rows(2, p=8 * P))), dict(change=(7, rows(2, p=4 * P))),
               dict(change=(6, rows(2, p=7 * P, ld=64))), dict(change=(5, rows(4, p=6 * P, head=32)))):
        assert "dpa_attention_backward" in refused(backward(**kw)), kw


def test_workspace():
    assert dp.dpa_attention_workspace(0, 4) == 0 and dp.dpa_attention_workspace(1000, 32) == 128000
    n = ctypes.c_size_t()
    for args in ((-1, 4), ((1 << 24) + 1, 4), (10, 0), (10, 1025)):
        refused(dp.lib.dpa_attention_workspace(*args, ctypes.byref(n)))
    refused(dp.lib.dpa_attention_workspace(10, 4, None))


def test_rotary_refusals():
    def call(sections=(16, 16), axes=None, interleaved=0, base=1e4, tokens=5, dim=64, positions=P, size=8, ld=2, axis=1, count=1,
             x=None, y=None, heads=4, dtype=dp.DP_F32, handle=True):
        d = A.RotaryDesc(len(sections) if axes is None else axes, (ctypes.c_int32 * 4)(*sections), interleaved, 0, 0, base)
        r = (A.RotaryRows * 5)(*[A.RotaryRows(x or rows(4, p=(2 + 2 * i) * P), y or rows(4, p=(3 + 2 * i) * P), heads, 0)
                                 for i in range(5)])
        return dp.lib.dpa_rotary(ctypes.addressof(d) if handle else None, tokens, dim, positions, size, ld, axis, count,
                                 ctypes.addressof(r), dtype, 0, None)

    for kw in (dict(handle=False), dict(axes=0), dict(axes=5), dict(sections=(-1, 8)), dict(sections=(33,)), dict(sections=(257,), dim=600),
               dict(base=0.0), dict(base=-2.0), dict(base=float("nan")), dict(base=float("inf")), dict(tokens=-1),
               dict(tokens=(1 << 24) + 1), dict(dim=0), dict(dim=4097), dict(positions=None), dict(positions=P + 4), dict(size=2),
               dict(ld=-1), dict(axis=-1), dict(count=0), dict(count=5), dict(heads=0), dict(heads=1025), dict(dtype=3),
               dict(x=rows(4, p=None)), dict(y=rows(4, p=3 * P + 2)), dict(y=rows(4, p=3 * P, ld=255)),
               dict(y=rows(4, p=3 * P, head=63)), dict(x=rows(4, p=3 * P, ld=300), y=rows(4, p=3 * P)), dict(y=rows(4, p=3 * P), count=2)):
        assert "dpa_rotary" in refused(call(**kw)), kw


def test_distill_refusals():
    def call(tau=1.0, soft=1.0, hard=0.5, scale=1.0, vocab=100, top=8, id_bytes=8, tokens=4, dtype=dp.DP_BF16, logits=P, ld=100,
             tdt=dp.DP_F32, teacher=P, ld_t=8, ids=P, ld_i=8, total=P, labels=P, weight=P, loss=P, dlogits=2 * P, ld_d=100, handle=True):
        d = D.DistillDesc(tau, soft, hard, scale, vocab, top, id_bytes)
        return dp.lib.dpd_distill(ctypes.addressof(d) if handle else None, tokens, dtype, logits, ld, tdt, teacher, ld_t, ids, ld_i,
                                  total, labels, weight, loss, dlogits, ld_d, None)

    inf, nan = float("inf"), float("nan")
    for kw in (dict(handle=False), dict(tau=0.0), dict(tau=-1.0), dict(tau=nan), dict(tau=inf), dict(tau=1e-46), dict(tau=1e30),
               dict(soft=nan), dict(hard=inf), dict(scale=1e39), dict(vocab=0), dict(vocab=(1 << 18) + 1), dict(top=-1), dict(top=1025),
               dict(id_bytes=2), dict(tokens=-1), dict(tokens=(1 << 21) + 1), dict(dtype=3), dict(tdt=-1), dict(logits=None),
               dict(logits=P + 1), dict(ld=99), dict(ld=1 << 39), dict(teacher=None), dict(teacher=P + 2), dict(ld_t=7), dict(ids=None),
               dict(ids=P + 4), dict(ld_i=7), dict(total=P + 2), dict(labels=P + 4), dict(weight=P + 1), dict(loss=P + 2),
               dict(dlogits=P + 1), dict(ld_d=99), dict(dlogits=P, ld_d=101), dict(loss=None, dlogits=None)):
        assert "dpd_distill" in refused(call(**kw)), kw


def test_descriptions_copy_and_pickle():
    r = dp.Rotary((8, 4), 500000.0, True, True)
    r.ref()
    for x in (copy.copy(r), copy.deepcopy(r), pickle.loads(pickle.dumps(r))):
        assert x == r and hash(x) == hash(r) and x._refs == []
    for d in (dp.Attention(True, 5, 0.3), dp.Distillation(2.0, 0.5, 0.5)):
        assert pickle.loads(pickle.dumps(d)) == d


WITHOUT_TORCH = """
import sys
sys.modules["torch"] = None
import gradient_reduce_adam_amd as dp
assert dp.dpa_attention_workspace(10, 4) == 160
for call in (lambda: dp.dpa_rotary(dp.Rotary((4,)), None, None, None),
             lambda: dp.dpa_attention(dp.Attention(), *[None] * 5),
             lambda: dp.dpa_attention_backward(dp.Attention(), *[None] * 10),
             lambda: dp.dpd_distill(dp.Distillation(), *[None] * 4)):
    try:
        call()
    except ImportError as e:
        assert "torch" in str(e)
    else:
        raise AssertionError("no ImportError")
print("fine")
"""


def test_without_torch():
    r = subprocess.run([sys.executable, "-c", WITHOUT_TORCH], capture_output=True, text=True, cwd=ROOT, timeout=120)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr
