"""The calls around a paged cache at the edges of what their documentation allows, without a
GPU: lifetimes of argument blocks, overlaps of rows, sizes."""

import gc
import weakref

import torch

from quantized_position_split_gb300 import _native as N
from quantized_position_split_gb300 import paged
from tests.test_paged_cpu import lib  # noqa: F401


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
