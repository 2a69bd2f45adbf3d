"""Decode attention behind a sliding window with sinks, on the GPU against the float64 oracle:
every format and kernel, windows and sinks around page and tile borders, pages that were given
back, and what lies in the positions that nothing sees."""

import numpy as np
import pytest
import torch

from oracle import stream as os_
from tests.helpers import assert_parity
from tests.test_gpu_paged import PAIRS, _cache_of, _rotations, _run, qps  # noqa: F401
from tests.test_gpu_paged_edges import _key_plane, _value_plane

pytestmark = pytest.mark.gpu


def _want(cache, q, table, lens, scale, window, sinks, softcap=0.0, ora=None):
    kp, vp = ([p.cpu().numpy() for p in s] for s in (cache.k_planes, cache.v_planes))
    q = q[:, None] if q.dim() == 3 else q
    n_q = q.shape[1]
    starts = [b * n_q for b in range(len(lens) + 1)]
    o, lse = os_.attention(q.flatten(0, 1).cpu().numpy(), starts, cache.k_fmt, kp, cache.v_fmt, vp, table.numpy(), lens, scale,
                           softcap, window, sinks, ora)
    return o.reshape(-1, q.shape[-1]), lse.reshape(-1)


def _bury(cache, table, lens, n_q, window, sinks, poison=True):
    """NaN values and infinite keys in every position that no query token sees; pages that hold
    nothing else are given back (their entries name nothing)."""
    table, page = table.clone(), cache.page_size
    for b, n in enumerate(lens):
        seen = os_.visible(n, min(n_q, n), window, sinks).any(0)
        for j in range(-(-n // page)):
            here = seen[j * page:(j + 1) * page]
            if not here.any():
                table[b, j] = -1 - j
            if not here.any() or not poison:
                continue
            at = torch.from_numpy(np.flatnonzero(~here)).cuda()
            _key_plane(cache)[int(table[b, j])].index_fill_(1, at, float("inf"))
            _value_plane(cache)[int(table[b, j])].index_fill_(1, at, float("nan"))
    return table


LENS = [0, 1, 3, 16, 17, 64, 129, 200, 257, 511, 1000]


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("kf,vf", PAIRS)
def test_window_ragged(qps, d, kf, vf):  # noqa: F811
    """Single tokens, every format; windows of one position, of a page, across pages and longer
    than every sequence; no sinks, a few, a page of them and more."""
    hkv = 2
    for page, group, softcap, window, sinks in ((16, 4, 0.0, 1, 0), (16, 1, 0.0, 16, 1), (64, 5, 30.0, 100, 4), (32, 4, 0.0, 33, 33),
                                                (128, 3, 0.0, 250, 64), (1024, 4, 0.0, 70, 130), (64, 4, 0.0, 5000, 3)):
        rot, ora = _rotations(d, "block" if page == 64 else "whole")
        cache, table = _cache_of(qps, kf, vf, LENS, page, hkv, d, d + page, rot)
        table = _bury(cache, table, LENS, 1, window, sinks)
        q = torch.randn((len(LENS), hkv * group, d), generator=torch.Generator().manual_seed(d + group)).half().cuda()
        ro, rl = _want(cache, q, table, LENS, d ** -0.5, window, sinks, softcap, ora)
        for causal in (False, True):
            o, lse = _run(qps, q, cache, table, LENS, scale=d ** -0.5, softcap=softcap, out_dtype=torch.float32, window=window,
                          sinks=sinks, causal=causal)
            assert_parity(o, lse, ro, rl, (d, kf, vf, page, window, sinks))


@pytest.mark.parametrize("d,kf,vf,n_q,group", [(64, "f16", "f16", 5, 4), (128, "f16", "f16", 2, 3), (128, "f16", "f16", 64, 5),
                                               (128, "q8_0", "tq3", 9, 4), (128, "q8_0", "q8_0", 17, 2), (128, "tq4", "tq4", 5, 4),
                                               (256, "f16", "f16", 5, 4), (256, "q8_0", "q8_0", 3, 3), (512, "q8_0", "tq2", 5, 8),
                                               (512, "f16", "f16", 4, 4), (64, "q8_0", "q8_0", 9, 4)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 3), (128, 16), (300, 129)])
def test_window_multi_query(qps, d, kf, vf, n_q, group, window, sinks):  # noqa: F811
    """Verify batches: every token's own window, through each of the kernels."""
    hkv, page = 2, 32
    rot, ora = _rotations(d, "whole")
    lens = [n_q, 1, 0, n_q + 70, 513, 2000]
    cache, table = _cache_of(qps, kf, vf, lens, page, hkv, d, n_q + group, rot)
    q = torch.randn((len(lens), n_q, hkv * group, d), generator=torch.Generator().manual_seed(n_q)).half().cuda()
    kw = dict(scale=d ** -0.5, causal=True, out_dtype=torch.float32, window=window, sinks=sinks)
    # (a value that some token sees reaches the others as 0 x it; these do not: they are not NaN)
    table = _bury(cache, table, lens, n_q, window, sinks)
    pad = [(n, table[b]) for b, n in enumerate(lens)]
    ro, rl = np.zeros((len(lens), n_q, hkv * group, d)), np.full((len(lens), n_q, hkv * group), -np.inf)
    for b, (n, row) in enumerate(pad):
        m = min(n, n_q)  # (tokens before the first position see nothing)
        if m:
            o, lse = _want(cache, q[b:b + 1, n_q - m:], row[None], [n], d ** -0.5, window, sinks, 0.0, ora)
            ro[b, n_q - m:], rl[b, n_q - m:] = o.reshape(m, -1, d), lse.reshape(m, -1)
    for _ in range(2):
        o, lse = _run(qps, q, cache, table, lens, **kw)
        assert_parity(o, lse, ro.reshape(-1, d), rl.reshape(-1), (d, kf, vf, n_q, group, window, sinks))


@pytest.mark.parametrize("kf,vf,n_q,group", [("f16", "f16", 1, 5), ("q8_0", "tq3", 1, 4), ("f16", "f16", 7, 4), ("q8_0", "q8_0", 7, 4)])
def test_window_of_long_sequences(qps, kf, vf, n_q, group):  # noqa: F811
    """Long windows of long sequences, in many chunks; shared_len changes nothing; the fp16 output
    is the float32 one, rounded once."""
    hkv, page, d, window, sinks = 2, 64, 128, 9000, 70
    rot, ora = _rotations(d, "whole")
    lens = [40007, 12000, 9005, 8000]
    cache, table = _cache_of(qps, kf, vf, lens, page, hkv, d, 7, rot, common=4096)
    q = torch.randn((len(lens), n_q, hkv * group, d), generator=torch.Generator().manual_seed(n_q)).half().cuda()
    table = _bury(cache, table, lens, n_q, window, sinks, poison=False)  # (their pages are others' sinks or window)
    ro, rl = _want(cache, q, table, lens, d ** -0.5, window, sinks, 0.0, ora)
    for shared in (0, 4096):
        kw = dict(scale=d ** -0.5, causal=True, window=window, sinks=sinks, shared_len=shared)
        o, lse = _run(qps, q, cache, table, lens, out_dtype=torch.float32, **kw)
        assert_parity(o, lse, ro, rl, (kf, vf, n_q, group))
        half, _ = _run(qps, q, cache, table, lens, out_dtype=torch.float16, **kw)
        assert np.array_equal(half, torch.from_numpy(o).half().float().numpy())


def test_window_that_nothing_outgrows(qps):  # noqa: F811
    """As long as the tables, or with sinks as long: the plain call, bit for bit."""
    lens, d = [5, 700, 64], 128
    cache, table = _cache_of(qps, "f16", "f16", lens, 64, 2, d, 3)
    q = torch.randn((3, 8, d), generator=torch.Generator().manual_seed(0)).half().cuda()
    plain = _run(qps, q, cache, table, lens, scale=0.1)
    for window, sinks in ((700, 0), (10 ** 9, 5), (3, 10 ** 9), (2 ** 31 - 1, 2 ** 31 - 1)):
        got = _run(qps, q, cache, table, lens, scale=0.1, window=window, sinks=sinks)
        if window == 700:
            assert_parity(got[0], got[1], plain[0].astype(np.float64), plain[1].astype(np.float64))
        else:
            assert all(np.array_equal(a, b) for a, b in zip(got, plain))


def test_window_in_a_captured_graph(qps):  # noqa: F811
    """One graph, lengths that grow past the window: each replay is the eager call."""
    d, hkv, page, width = 128, 2, 32, 40
    cache, _ = _cache_of(qps, "q8_0", "q8_0", [page * width] * 2, page, hkv, d, 1)
    table = torch.arange(2 * width, dtype=torch.int32).view(2, width).cuda()
    for p in cache.k_planes + cache.v_planes:
        if p.dtype == torch.float16:
            p.fill_(0.01)
    q = torch.randn((2, 8, d), generator=torch.Generator().manual_seed(0)).half().cuda()
    lens = torch.tensor([1, 2], dtype=torch.int32).cuda()
    a = qps.paged_attn_args(q, cache, table, lens, scale=0.1, window=100, sinks=5)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        qps.attn_decode_paged(a)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            o, lse = qps.attn_decode_paged(a)
    torch.cuda.synchronize()
    for n in (1, 50, 100, 101, 133, 1000, 1280):
        lens.copy_(torch.tensor([n, max(0, n - 37)], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = o.clone(), lse.clone()
        want = qps.attn_decode_paged(qps.paged_attn_args(q, cache, table, lens, scale=0.1, window=100, sinks=5))
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
