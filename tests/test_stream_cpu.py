"""The calls for long streams in a paged cache without a GPU: struct layouts, refusals before any
device is touched, planning, the oracle's own checks."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import paged as op
from oracle import stream as os_
from quantized_position_split_gb300 import _native as N
from tests.test_paged_cpu import INVALID, ROOT, UNSUPPORTED, _attn, _kv, lib  # noqa: F401


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


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")
def test_struct_layouts(tmp_path):
    pairs = [("qps_paged_prompt_args", N.PagedPromptArgs), ("qps_paged_seqs", N.PagedSeqsStruct),
             ("qps_paged_extend_args", N.PagedExtendArgs), ("qps_paged_fork_args", N.PagedForkArgs),
             ("qps_paged_compact_args", N.PagedCompactArgs)]
    fields = [(c, t, f[0]) for c, t in pairs for f in t._fields_]
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "qps.h"\nint main(void){\n' +
                   "".join('printf("%%zu\\n", sizeof(%s));\n' % c for c, _ in pairs) +
                   "".join('printf("%%zu\\n", offsetof(%s, %s));\n' % (c, f) for c, _, f in fields) + "return 0;}\n")
    exe = tmp_path / "l"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert out == [ctypes.sizeof(t) for _, t in pairs] + [getattr(t, f).offset for _, t, f in fields]


def _seqs(of, **kw):
    s = N.PagedSeqsStruct()
    s.caches, s.n_caches, s.batch = of, len(of), 3
    s.page_table, s.table_stride, s.table_width = 0x20000, 16, 16
    s.kv_lens, s.refs = 0x30000, 0x31000
    for k, v in kw.items():
        setattr(s, k, v)
    return s


def _page_calls(lib, caches=None, seqs=None, only=None, **kw):  # noqa: F811
    """The statuses of the three calls (or of one of them) and of their plans for one state, with
    fields changed.  (Only calls that are refused are made: the addresses are of nothing.)"""
    caches = caches or (N.PagedKvStruct * 2)(_kv(), _kv(N.FMT_Q8_0, N.FMT_Q8_0))
    out = {}
    for cls, name in ((N.PagedExtendArgs, "extend"), (N.PagedForkArgs, "fork"), (N.PagedCompactArgs, "compact")):
        if only not in (None, name):
            continue
        a = cls()
        a.seqs = _seqs(caches, **(seqs or {}))
        a.workspace, a.workspace_bytes = 0x50000000, 1 << 24
        for k, v in {**dict(n_new=0x32000, max_tokens=100, q_starts=0x33000, slots=0x34000, positions=0x35000, src=0x36000,
                            dst=0x37000, n=2, new_ids=0x38000, live=0x39000), **kw}.items():
            if hasattr(a, k):
                setattr(a, k, v)
        call, plan = getattr(lib, f"qps_kv_{name}_paged"), getattr(lib, f"qps_kv_{name}_plan")
        out[name] = (call(ctypes.byref(a), None), plan(ctypes.byref(a), None))
        assert call(None, None) == INVALID and plan(None, None) == INVALID
    return out


@pytest.mark.parametrize("change,status", [
    (dict(n_caches=0), INVALID), (dict(caches=None), INVALID), (dict(batch=0), INVALID), (dict(batch=4097), INVALID),
    (dict(page_table=None), INVALID), (dict(page_table=0x20002), INVALID), (dict(kv_lens=None), INVALID), (dict(refs=0x31001), INVALID),
    (dict(table_width=0), INVALID), (dict(table_width=1 << 25, table_stride=1 << 25), INVALID), (dict(table_stride=15), INVALID),
    (dict(reserved0=1), INVALID)])
def test_sequence_refusals(lib, change, status):  # noqa: F811
    for got in _page_calls(lib, seqs=change).values():
        assert got == (status, status)


def test_caches_of_one_shape(lib):  # noqa: F811
    for field, value in (("page_size", 32), ("n_pages", 11)):
        kv = _kv()
        setattr(kv, field, value)
        for got in _page_calls(lib, (N.PagedKvStruct * 2)(_kv(), kv)).values():
            assert got == (INVALID, INVALID)
    kv = _kv()
    kv.d = 96
    for got in _page_calls(lib, (N.PagedKvStruct * 1)(kv)).values():
        assert got == (UNSUPPORTED, UNSUPPORTED)


@pytest.mark.parametrize("name,change", [
    ("extend", dict(n_new=None)), ("extend", dict(n_new=0x32001)), ("extend", dict(window=-1)), ("extend", dict(sinks=-1)),
    ("extend", dict(max_tokens=-1)), ("extend", dict(max_tokens=1 << 31)), ("fork", dict(n=-1)), ("fork", dict(n=4097)),
    ("fork", dict(src=None)), ("fork", dict(dst=0x37002)), ("fork", dict(reserved0=1))])
def test_page_call_refusals(lib, name, change):  # noqa: F811
    assert _page_calls(lib, only=name, **change)[name] == (INVALID, INVALID)


@pytest.mark.parametrize("name,change", [
    ("extend", dict(q_starts=None)), ("extend", dict(slots=None)), ("extend", dict(slots=0x34004)), ("extend", dict(positions=None)),
    ("extend", dict(workspace=None)), ("extend", dict(workspace_bytes=64)), ("extend", dict(workspace=0x50000080)),
    ("extend", dict(slots=0x35008)), ("extend", dict(n_new=0x33000)), ("extend", dict(q_starts=0x30000)), ("extend", dict(positions=0x20000)),
    ("fork", dict(workspace=None)), ("fork", dict(workspace_bytes=0)), ("fork", dict(src=0x20000)), ("fork", dict(dst=0x31000)),
    ("compact", dict(new_ids=None)), ("compact", dict(live=0x39001)), ("compact", dict(new_ids=0x31000)), ("compact", dict(live=0x30008)),
    ("compact", dict(workspace=0x20000))])
def test_page_call_outputs(lib, name, change):  # noqa: F811
    assert _page_calls(lib, only=name, **change)[name] == (INVALID, N.QPS_OK)


def test_page_plans(lib):  # noqa: F811
    """Workspaces grow with what they hold, not with the lengths; n == 0 is a no-op."""
    caches = (N.PagedKvStruct * 1)(_kv())
    need = ctypes.c_size_t()
    sizes = []
    for tokens in (0, 100, 10 ** 6):
        a = N.PagedExtendArgs()
        a.seqs, a.n_new, a.max_tokens = _seqs(caches), 0x32000, tokens
        assert lib.qps_kv_extend_plan(ctypes.byref(a), ctypes.byref(need)) == N.QPS_OK
        sizes.append(need.value)
    assert 0 < sizes[0] <= sizes[1] <= sizes[2] < 1 << 20
    a = N.PagedForkArgs()
    a.seqs = _seqs(caches)
    assert lib.qps_kv_fork_paged(ctypes.byref(a), None) == N.QPS_OK


def test_oracle_pages():
    """Counts stay those of the entries, free pages are the lowest, copies hold the rows."""
    r = np.random.default_rng(3)
    page, batch, width, pages = 4, 4, 9, 20
    x = os_.Pages(page, np.full((batch, width), -1), [0] * batch, [0] * pages, [r.integers(0, 255, (pages, 2, page, 3))])
    rows = {b: [] for b in range(batch)}  # what each position holds, followed on its own
    for step in range(200):
        if step % 5 < 3:
            new = [int(n) for n in r.integers(-5, 6, batch)]
            starts, slots, pos = x.extend(new, max_tokens=24)
            for b, n in enumerate(new):
                rows[b] = rows[b][:x.lens[b]]
                for i in range(starts[b], starts[b + 1]):
                    if slots[i] >= 0:
                        mark = r.integers(0, 255, (2, 3))
                        x.planes[0][slots[i] // page, :, slots[i] % page] = mark
                        rows[b].append(mark)
        elif step % 5 == 3:
            a, b = (int(n) for n in r.integers(0, batch, 2))
            x.fork([a - (step % 2)], [b])
            if a - (step % 2) != b:
                rows[b] = (list(rows[a - (step % 2)]) if a - (step % 2) >= 0 else [])[:x.lens[b]]
        else:
            x.compact()
            assert all((c > 0) == (p < sum(n > 0 for n in x.refs)) for p, c in enumerate(x.refs))
        count = [0] * pages
        for b in range(batch):
            assert len(rows[b]) == x.lens[b]
            for j in range(-(-x.lens[b] // page)):
                count[x.table[b][j]] += 1
            for t, mark in enumerate(rows[b]):
                assert (x.planes[0][x.table[b][t // page], :, t % page] == mark).all()
        assert count == x.refs


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
