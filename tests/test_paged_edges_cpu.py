"""The calls around a paged cache at the edges of what their documentation allows, without a
GPU: lifetimes of argument blocks, overlaps of rows, sizes."""

import ctypes
import gc
import weakref

import pytest
import torch

from quantized_position_split_gb300 import _native as N
from quantized_position_split_gb300 import paged
from tests.test_paged_cpu import INVALID, _rope, lib  # noqa: F401


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
