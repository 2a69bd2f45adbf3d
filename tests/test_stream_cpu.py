"""The calls for long streams in a paged cache without a GPU: struct layouts, refusals before any
device is touched, planning, the oracle's own checks."""

import ctypes

import numpy as np
import pytest

from oracle import paged as op
from oracle import stream as os_
from quantized_position_split_gb300 import _native as N
from tests.test_paged_cpu import INVALID, UNSUPPORTED, _attn, _kv, lib  # noqa: F401


@pytest.mark.parametrize("change", [dict(window=-1), dict(sinks=-1, window=4), dict(sinks=-1), dict(window=9, n_q=2, q_batch_stride=16 * 128)])
def test_window_refusals(lib, change):  # noqa: F811
    a = _attn(**change)
    assert lib.qps_attn_paged_plan(ctypes.byref(a), None) == INVALID
    assert lib.qps_attn_decode_paged(ctypes.byref(a), None) == INVALID
    assert b"window" in lib.qps_last_error()


def _prompt(kv=None, **kw):
    a = N.PagedPromptArgs()
    a.q, a.q_tok_stride, a.tokens = 0x10000, 8 * 128, 50
    a.batch, a.hq, a.q_starts = 3, 8, 0x18000
    a.kv = kv or _kv()
    a.page_table, a.table_stride, a.table_width, a.kv_lens = 0x20000, 16, 16, 0x30000
    a.scale = 0.1
    a.o, a.lse, a.workspace, a.workspace_bytes = 0x40000000, 0x41000000, 0x50000000, 1 << 28
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(q=0x10008), INVALID), (dict(tokens=-1), INVALID), (dict(batch=0), INVALID), (dict(batch=65536), INVALID),
    (dict(hq=7), INVALID), (dict(hq=0), INVALID), (dict(hq=65536, q_tok_stride=65536 * 128), UNSUPPORTED),
    (dict(tokens=1 << 28), UNSUPPORTED), (dict(q_tok_stride=8 * 128 + 4), INVALID), (dict(q_tok_stride=128), INVALID),
    (dict(q_tok_stride=1 << 33), INVALID), (dict(q_starts=None), INVALID), (dict(q_starts=0x18002), INVALID), (dict(page_table=None), INVALID),
    (dict(kv_lens=0x30002), INVALID), (dict(table_width=0), INVALID), (dict(table_width=1 << 25, table_stride=1 << 25), INVALID),
    (dict(table_stride=15), INVALID), (dict(o_dtype=3), INVALID), (dict(scale=float("inf")), INVALID), (dict(softcap=float("nan")), INVALID),
    (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(reserved0=1), INVALID),
])
def test_prompt_refusals(lib, change, status):  # noqa: F811
    a = _prompt(**change)
    assert lib.qps_attn_prompt_plan(ctypes.byref(a), None) == status
    assert lib.qps_attn_prompt_paged(ctypes.byref(a), None) == status
    assert b"attn_prompt_paged" in lib.qps_last_error()
    assert lib.qps_attn_prompt_plan(None, None) == INVALID and lib.qps_attn_prompt_paged(None, None) == INVALID


def test_prompt_struct_layout(tmp_path):
    import os
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    pairs = [("qps_paged_prompt_args", N.PagedPromptArgs)]
    fields = [(c, t, f[0]) for c, t in pairs for f in t._fields_]
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "qps.h"\nint main(void){\n' +
                   "".join('printf("%%zu\\n", sizeof(%s));\n' % c for c, _ in pairs) +
                   "".join('printf("%%zu\\n", offsetof(%s, %s));\n' % (c, f) for c, _, f in fields) + "return 0;}\n")
    exe = tmp_path / "l"
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run(["gcc", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    out = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert out == [ctypes.sizeof(t) for _, t in pairs] + [getattr(t, f).offset for _, t, f in fields]


def test_oracle_window():
    """Against the definition, one query and position at a time, and against the plain oracle."""
    for n, n_q, window, sinks in ((9, 3, 2, 1), (5, 5, 1, 0), (20, 1, 7, 30), (7, 2, 100, 3), (6, 2, 0, 0)):
        seen = os_.visible(n, n_q, window, sinks)
        for i in range(n_q):
            q = n - n_q + i
            for t in range(n):
                assert seen[i, t] == (t <= q and (window == 0 or t > q - window or t < sinks))
    r = np.random.default_rng(0)
    page, hkv, d, n = 16, 2, 64, 45
    planes = [[r.standard_normal((6, hkv, page, d)).astype(np.float16)] for _ in range(2)]
    q = r.standard_normal((1, 3, 4, d))
    want = op.decode(q, "f16", planes[0], "f16", planes[1], np.array([[4, 0, 2]]), [n], 0.2, 5.0, True)
    got = os_.attention(q[0], [0, 3], "f16", planes[0], "f16", planes[1], np.array([[4, 0, 2]]), [n], 0.2, 5.0)
    assert np.allclose(got[0], want[0][0], atol=1e-13) and np.allclose(got[1], want[1][0], atol=1e-13)
    # a window reads nothing of the pages that it has left
    a = os_.attention(q[0], [0, 3], "f16", planes[0], "f16", planes[1], np.array([[4, -1, 2]]), [n], 0.2, window=11, sinks=16)
    assert np.isfinite(a[0]).all() and np.isfinite(a[1]).all()
