"""The calls around a paged cache without a GPU: struct layouts, what the library refuses
before it touches a device, what the binding refuses, and the oracle's definitions."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

from oracle import paged as op
from quantized_position_split_gb300 import _native as N

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED = N.QPS_ERR_INVALID_ARG, N.QPS_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(N.LIB_PATH):
        from quantized_position_split_gb300 import build
        build.build()
    return N.load()


@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")
def test_struct_layouts(tmp_path):
    pairs = [("qps_rows", N.Rows), ("qps_head_norm", N.HeadNorm), ("qps_rotation", N.RotationArgs),
             ("qps_qk_rope_args", N.QkRopeArgs), ("qps_paged_kv", N.PagedKvStruct),
             ("qps_paged_append_args", N.PagedAppendArgs), ("qps_paged_attn_args", N.PagedAttnArgs)]
    fields = [(c, t, f[0]) for c, t in pairs for f in t._fields_]
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "qps.h"\nint main(void){\n' +
                   "".join('printf("%%zu\\n", sizeof(%s));\n' % c for c, _ in pairs) +
                   "".join('printf("%%zu\\n", offsetof(%s, %s));\n' % (c, f) for c, _, f in fields) + "return 0;}\n")
    exe = tmp_path / "l"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert out == [ctypes.sizeof(t) for _, t in pairs] + [getattr(t, f).offset for _, t, f in fields]


def _rows(data, dtype=0, heads=2, tok=None, head=128):
    return N.Rows(data, dtype, heads, heads * 128 if tok is None else tok, head)


def _rope(**kw):
    a = N.QkRopeArgs()
    a.tokens, a.d = 4, 128
    a.q, a.k = _rows(0x10000), _rows(0x20000)
    a.q_out, a.k_out = _rows(0x30000), _rows(0x40000)
    a.rot = N.RotationArgs(0x50000, 100, 128, 0)
    a.positions = 0x60000
    for k, v in kw.items():
        o = a
        path = k.split("__")
        for p in path[:-1]:
            o = getattr(o, p)
        setattr(o, path[-1], v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), INVALID), (dict(d=96), UNSUPPORTED), (dict(d=1024), UNSUPPORTED), (dict(reserved0=1), INVALID),
    (dict(q__data=None), INVALID), (dict(q__data=0x10008), INVALID), (dict(q__dtype=3), INVALID),
    (dict(q__heads=-1), INVALID), (dict(q__heads=3), INVALID), (dict(q__tok_stride=257), INVALID),
    (dict(q__head_stride=64), INVALID), (dict(q__tok_stride=-256), INVALID), (dict(k__dtype=1), INVALID),
    (dict(q_out__dtype=2), UNSUPPORTED), (dict(k_out__dtype=1), INVALID), (dict(q_out__tok_stride=0), INVALID),
    (dict(rot__dim=136), INVALID), (dict(rot__dim=24), INVALID), (dict(rot__dim=144), INVALID),
    (dict(rot__pairs=2), INVALID), (dict(rot__table=None), INVALID), (dict(rot__table=0x50004), INVALID),
    (dict(rot__len=0), INVALID), (dict(positions=None), INVALID),
    (dict(q_norm__on=1, q_norm__eps=-1.0), INVALID), (dict(q_norm__on=1, q_norm__eps=float("nan")), INVALID),
    (dict(k_norm__on=1, k_norm__offset=float("inf")), INVALID), (dict(k_norm__on=1, k_norm__w=0x71, k_norm__w_dtype=0), INVALID),
    (dict(k_norm__on=1, k_norm__w=0x70, k_norm__w_dtype=9), INVALID),
    (dict(q_out__data=0x10010), INVALID),                 # shifted over the input
    (dict(q_out__data=0x20000), INVALID),                 # over the other side's input
    (dict(k_out__data=0x30000), INVALID),                 # both outputs in one place
    (dict(q_out__data=0x10000, q_out__dtype=1, k_out__dtype=1), INVALID),  # in place, of another type
    (dict(q_out__data=0x10000, q_out__tok_stride=512), INVALID),
])
def test_rope_refusals(lib, change, status):
    a = _rope(**change)
    assert lib.qps_qk_norm_rope(ctypes.byref(a), None) == status
    assert lib.qps_last_error()


def test_rope_no_ops(lib):
    assert lib.qps_qk_norm_rope(None, None) == INVALID
    assert lib.qps_qk_norm_rope(ctypes.byref(_rope(tokens=0)), None) == N.QPS_OK
    a = _rope(q__heads=0, q_out__heads=0, k__heads=0, k_out__heads=0)
    assert lib.qps_qk_norm_rope(ctypes.byref(a), None) == N.QPS_OK


def _kv(kf=N.FMT_F16, vf=N.FMT_F16):
    kv = N.PagedKvStruct()
    kv.k_fmt, kv.v_fmt, kv.hkv, kv.d, kv.page_size, kv.n_pages = kf, vf, 2, 128, 64, 10
    for i, f in enumerate(("k_data", "k_aux", "k_aux2", "v_data", "v_aux", "v_aux2")):
        setattr(kv, f, 0x100000 * (i + 1))
    return kv


KV_REFUSALS = [
    (dict(d=96), UNSUPPORTED), (dict(d=32), UNSUPPORTED), (dict(hkv=0), INVALID), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=48), UNSUPPORTED), (dict(page_size=2048), UNSUPPORTED), (dict(n_pages=0), INVALID),
    (dict(n_pages=1 << 26), INVALID), (dict(k_fmt=7), INVALID), (dict(v_fmt=-1), INVALID), (dict(k_data=None), INVALID),
    (dict(v_data=0x400008), INVALID), (dict(reserved0=1), INVALID), (dict(reserved1=1), INVALID),
    (dict(k_fmt=N.FMT_Q8_0, k_aux=None), INVALID), (dict(k_fmt=N.FMT_TQ3), UNSUPPORTED),
    (dict(v_fmt=N.FMT_TQ3), INVALID),  # no signs
]


def _append(kv=None, **kw):
    a = N.PagedAppendArgs()
    a.kv = kv or _kv()
    a.tokens = 4
    a.k, a.v = _rows(0x10000), _rows(0x20000)
    a.slots = 0x60000
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", KV_REFUSALS)
def test_cache_refusals(lib, change, status):
    kv = _kv()
    for k, v in change.items():
        setattr(kv, k, v)
    assert lib.qps_kv_append_paged(ctypes.byref(_append(kv)), None) == status
    assert lib.qps_attn_paged_plan(ctypes.byref(_attn(kv=kv)), None) == status


def test_cache_rotation_refusals(lib):
    words = (ctypes.c_uint32 * 4)()
    for block, ok in ((48, False), (16, False), (256, False)):
        kv = _kv(vf=N.FMT_TQ3)
        kv.signs1 = ctypes.cast(words, ctypes.POINTER(ctypes.c_uint32))
        kv.tq_block = block
        assert lib.qps_kv_append_paged(ctypes.byref(_append(kv)), None) == INVALID


@pytest.mark.parametrize("change", [
    dict(tokens=-1), dict(k=_rows(0x10000, heads=3)), dict(v=_rows(0x20000, heads=0)), dict(v=_rows(0x20000, dtype=1)),
    dict(k=_rows(0x10004)), dict(slots=None), dict(slots=0x60004), dict(rot=N.RotationArgs(0x50000, 9, 128, 0)),
])
def test_append_refusals(lib, change):
    assert lib.qps_kv_append_paged(ctypes.byref(_append(**change)), None) == INVALID
    assert lib.qps_kv_append_paged(None, None) == INVALID
    assert lib.qps_kv_append_paged(ctypes.byref(_append(tokens=0)), None) == N.QPS_OK


def _attn(kv=None, **kw):
    a = N.PagedAttnArgs()
    a.q, a.q_batch_stride = 0x10000, 8 * 128
    a.batch, a.n_q, a.hq = 3, 1, 8
    a.kv = kv or _kv()
    a.page_table, a.table_stride, a.table_width, a.kv_lens = 0x20000, 16, 16, 0x30000
    a.scale = 0.1
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(q=None), INVALID), (dict(q=0x10008), INVALID), (dict(batch=0), INVALID), (dict(batch=65536), INVALID),
    (dict(n_q=0), INVALID), (dict(n_q=65), INVALID), (dict(hq=7), INVALID), (dict(hq=0), INVALID),
    (dict(hq=4096, q_batch_stride=4096 * 128), UNSUPPORTED), (dict(q_batch_stride=8 * 128 + 4), INVALID),
    (dict(q_batch_stride=128), INVALID), (dict(page_table=None), INVALID), (dict(kv_lens=0x30002), INVALID),
    (dict(table_width=0), INVALID), (dict(table_width=1 << 25, table_stride=1 << 25), INVALID),
    (dict(table_width=(1 << 25) - 16, table_stride=1 << 25), INVALID),
    (dict(batch=17, table_width=(1 << 25) - 17, table_stride=1 << 25), UNSUPPORTED),
    (dict(table_stride=15), INVALID), (dict(shared_len=-64), INVALID), (dict(shared_len=32), INVALID),
    (dict(shared_len=17 * 64), INVALID), (dict(o_dtype=3), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(softcap=float("nan")), INVALID),
])
def test_attention_refusals(lib, change, status):
    a = _attn(**change)
    assert lib.qps_attn_paged_plan(ctypes.byref(a), None) == status
    assert lib.qps_attn_decode_paged(ctypes.byref(a), None) == status
    assert lib.qps_attn_paged_plan(None, None) == INVALID


def test_binding_refusals():
    """The binding names what it was given wrongly (here: host tensors) before any call."""
    import quantized_position_split_gb300 as qps
    x = torch.zeros((2, 4, 128), dtype=torch.float16)
    with pytest.raises(qps.QpsError, match="CUDA"):
        qps.qk_rope_args(x)
    with pytest.raises(qps.QpsError, match="CUDA"):
        qps.PagedKV("f16", "f16", [x[None]], [x[None]])
    with pytest.raises(qps.QpsError, match="unknown format"):
        qps.PagedKV("f8", "f16", [x], [x])
    with pytest.raises(qps.QpsError, match="CUDA"):
        qps.paged_attn_args(x, None, None, None, scale=1.0)


def test_rope_table_keeps_far_angles():
    import quantized_position_split_gb300 as qps
    t = qps.rope_table(200001, 16, base=5e5, scale=0.5, device="cpu").double().numpy()
    p, j = np.arange(200001)[:, None], np.arange(8)
    a = p * (0.5 * 5e5 ** (-2 * j / 16))
    assert np.abs(t - np.concatenate((np.cos(a), np.sin(a)), 1)).max() <= 2.0 ** -24


# ---- the oracle's definitions -----------------------------------------------------------
def test_oracle_rotation_is_a_rotation_and_relative():
    """Norms of pairs are kept, and the product of a rotated query and key depends on the
    difference of their positions alone."""
    r = np.random.default_rng(0)
    d = 32
    f = 100.0 ** (-np.arange(d // 2) * 2 / d)
    def cs(p):
        a = np.asarray(p)[:, None] * f
        return np.concatenate((np.cos(a), np.sin(a)), 1)
    q, k = r.standard_normal((1, 1, d)), r.standard_normal((1, 1, d))
    for inter in (False, True):
        dots = [float((op.norm_rope(q, cs=cs([m]), interleaved=inter) * op.norm_rope(k, cs=cs([n]), interleaved=inter)).sum())
                for m, n in ((7, 3), (104, 100), (4, 0))]
        assert np.allclose(dots, dots[0], atol=1e-12)
        y = op.norm_rope(q, cs=cs([11]), interleaved=inter)
        ia, ib = op._pairs(d, inter)
        assert np.allclose(y[..., ia] ** 2 + y[..., ib] ** 2, q[..., ia] ** 2 + q[..., ib] ** 2)


def test_oracle_f32_order_is_near_the_definition():
    r = np.random.default_rng(1)
    for d in (32, 128, 512):
        x, w = r.standard_normal((5, 3, d)).astype(np.float32), r.standard_normal(d).astype(np.float32)
        a = r.uniform(0, 6, (5, d // 2))
        cs = np.concatenate((np.cos(a), np.sin(a)), 1).astype(np.float32)
        y, z = (f(x, w, 1.0, 1e-6, True, cs) for f in (op.norm_rope, op.norm_rope_f32))
        assert np.abs(y - z).max() <= 20 * 2.0 ** -24 * 2 * np.abs(op.norm_rope(x, w, 1.0, 1e-6, True)).max()
        rms = op.norm_rope(x, None, 0, 0.0, True)
        assert np.allclose((rms ** 2).mean(-1), 1)


def test_oracle_pages_equal_a_dense_cache():
    from oracle import attention
    r = np.random.default_rng(2)
    page, hkv, d, n = 16, 2, 64, 45
    k, v = (r.standard_normal((n, hkv, d)).astype(np.float16) for _ in range(2))
    table = np.array([[4, 0, 2, -1]])
    slots = [int(table[0, t // page]) * page + t % page for t in range(n)]
    planes = [op.append([np.full((6, hkv, page, d), np.nan, np.float16)], (x,), slots, page) for x in (k, v)]
    q = r.standard_normal((1, 3, 4, d))
    o, lse = op.decode(q, "f16", planes[0], "f16", planes[1], table, [n], 0.2, causal=True)
    wo, wl = attention.multi_query_decode(q[0], k.astype(float), v.astype(float), 0.2, q_pos=n - 3)
    assert np.array_equal(o[0], wo) and np.array_equal(lse[0], wl)
