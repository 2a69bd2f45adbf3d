"""The calls around a paged cache at the edges of what their documentation allows, without a
GPU: lifetimes of argument blocks, overlaps of rows, sizes."""

import ctypes
import gc
import weakref

import pytest
import torch

from quantized_position_split_gb300 import _native as N
from quantized_position_split_gb300 import paged
from tests.test_paged_cpu import INVALID, UNSUPPORTED, _append, _rope, _rows, lib  # noqa: F401


def test_a_dropped_block_frees_its_tensors(lib):  # noqa: F811
    """A block holds its tensors, and nothing but its user holds the block: device memory is
    not left to the cycle collector, which GPU allocations do not start."""
    class Held:
        pass

    was = gc.isenabled()
    gc.disable()
    try:
        for fn, kind in (("qps_qk_norm_rope", N.QkRopeArgs), ("qps_kv_append_paged", N.PagedAppendArgs),
                         ("qps_attn_decode_paged", N.PagedAttnArgs)):
            held = Held()
            alive = weakref.ref(held)
            a = paged._block(kind(), fn, torch.device("cuda", 0), (held,))
            del held
            assert alive() is not None
            del a
            assert alive() is None, fn
    finally:
        if was:
            gc.enable()


# ---- rows that overlap ------------------------------------------------------------------
def _touch(a, b, tokens, d):
    """By every row of both (element addresses; the same row of one set is not compared)."""
    rows_a, rows_b = ([p + t * ts + h * hs for t in range(tokens) for h in range(n)] for p, ts, hs, n in (a, b))
    return any(abs(x - y) < d for i, x in enumerate(rows_a) for j, y in enumerate(rows_b) if a is not b or i != j)


LAYOUTS = [  # (first element, token stride, head stride, heads)
    (0, 256, 128, 2), (0, 128, 512, 2), (0, 128, 128, 2), (0, 128, 256, 3), (0, 384, 128, 2), (0, 136, 544, 2), (0, 256, 640, 3),
    (0, 640, 256, 3), (0, 136, 128, 3), (0, 384, 576, 2), (0, 768, 384, 2), (0, 128, 640, 3),
]


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up: an accepted call must not run")
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("tokens", [1, 2, 4, 5])
def test_rope_output_rows_overlap_one_another(lib, layout, tokens):  # noqa: F811
    """An output whose rows share elements is refused, and only such a one."""
    p, t, h, n = layout
    a = _rope(tokens=tokens, q__heads=n, q__tok_stride=n * 128, q_out=N.Rows(0x300000, 0, n, t, h), k__heads=0, k_out__heads=0)
    refused = lib.qps_qk_norm_rope(ctypes.byref(a), None) == INVALID
    assert refused == _touch(layout, layout, tokens, 128)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are made up: an accepted call must not run")
@pytest.mark.parametrize("off", [0, 8, 64, 120, 128, 136, 192, 256, 384, 512, 640, 1024, 1280, 4096])
@pytest.mark.parametrize("q", LAYOUTS[::2] + [(0, 768, 384, 2)])
@pytest.mark.parametrize("k", [(0, 384, 128, 1), (0, 768, 384, 2), (0, 256, 128, 1), (0, 640, 256, 2)])
def test_rope_outputs_overlap(lib, off, q, k):  # noqa: F811
    """Outputs of both sides in one buffer: side by side, head by head, or over one another
    (tokens the same distance apart, else any meeting of their extents is refused)."""
    tokens, base = 4, 0x800000
    if _touch(q, q, tokens, 128) or _touch(k, k, tokens, 128):
        return
    k = (off,) + k[1:]
    a = _rope(tokens=tokens, q__heads=q[3], q__tok_stride=q[3] * 128, k__heads=k[3], k__tok_stride=k[3] * 128,
              q_out=N.Rows(base, 0, q[3], q[1], q[2]), k_out=N.Rows(base + 2 * off, 0, k[3], k[1], k[2]))
    refused = lib.qps_qk_norm_rope(ctypes.byref(a), None) == INVALID
    meet = off < (tokens - 1) * q[1] + (q[3] - 1) * q[2] + 128
    assert refused == (_touch(q, k, tokens, 128) if q[1] == k[1] else meet)


# ---- sizes ------------------------------------------------------------------------------
@pytest.mark.parametrize("tokens", [1 << 27, 1 << 40, 1 << 62, (1 << 63) - 1])
def test_more_tokens_than_a_launch_holds(lib, tokens):  # noqa: F811
    """Refused before anything is computed from them."""
    assert lib.qps_qk_norm_rope(ctypes.byref(_rope(tokens=tokens)), None) == UNSUPPORTED
    assert lib.qps_kv_append_paged(ctypes.byref(_append(tokens=tokens)), None) == UNSUPPORTED


@pytest.mark.parametrize("stride", [1 << 58, (1 << 62) + 8, (1 << 63) - 8])
def test_strides_behind_any_memory(lib, stride):  # noqa: F811
    for kw in (dict(q__tok_stride=stride), dict(q_out__tok_stride=stride), dict(k__head_stride=stride, k__tok_stride=stride),
               dict(k_out__head_stride=stride)):
        assert lib.qps_qk_norm_rope(ctypes.byref(_rope(tokens=9, **kw)), None) == INVALID, kw
    a = _append(tokens=9, v=_rows(0x20000, tok=stride))
    assert lib.qps_kv_append_paged(ctypes.byref(a), None) == INVALID
