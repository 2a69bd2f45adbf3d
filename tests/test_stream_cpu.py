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
