"""Calls for long streams in a paged cache at the edges of what their documentation allows, on the
GPU: scales of any sign, values at the ends of the formats, wide groups, caches past 2^32 bytes,
arrays at any address, threads and first calls under capture."""

import threading

import numpy as np
import pytest
import torch

from oracle import stream as os_
from tests.helpers import assert_parity
from tests.test_gpu_pages import Pair
from tests.test_gpu_paged import _cache_of, _lib_rot, _rotations, qps  # noqa: F401
from tests.test_gpu_paged_edges import _child
from tests.test_gpu_prompt import _args, _q, _run, _starts, _want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,kf,vf", [(64, "q8_0", "q8_0"), (128, "f16", "f16"), (256, "f16", "f16"), (512, "q8_0", "tq3")])
@pytest.mark.parametrize("scale,softcap", [(0.0, 0.0), (-0.07, 0.0), (-0.07, 20.0), (0.05, 0.5), (0.0, 3.0)])
def test_prompt_scales(qps, d, kf, vf, scale, softcap):  # noqa: F811
    """Zero and negative scales, a softcap that saturates; masked tiles among them."""
    rot, ora = _rotations(d, "whole")
    new, lens = [200, 5], [390, 140]
    cache, table = _cache_of(qps, kf, vf, lens, 32, 2, d, 1, rot)
    q = _q(205, 6, d, 2)
    for window, sinks in ((0, 0), (100, 3)):
        kw = dict(scale=scale, softcap=softcap, window=window, sinks=sinks)
        ro, rl = _want(cache, q, _starts(new), table, lens, ora=ora, **kw)
        o, lse = _run(qps, q, cache, table, lens, _starts(new), out_dtype=torch.float32, **kw)
        assert_parity(o, lse, ro, rl, (d, kf, vf, scale, softcap))


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("kf,vf", [("q8_0", "q8_0"), ("q8_0", "f16"), ("f16", "q8_0")])
def test_prompt_at_the_end_of_the_range(qps, d, kf, vf):  # noqa: F811
    """Stored rows as large as fp16 values get: codes of 127 times a scale of 516 pass fp16's largest
    value by a rounding.  Queries are small, so that logits stay finite."""
    lens, new = [150], [150]
    cache, table = _cache_of(qps, kf, vf, lens, 16, 1, d, 3)
    x = torch.randn((150, 2, d), generator=torch.Generator().manual_seed(1)).half()
    x[::7] = 65504.0
    x[3::7] = -65504.0
    slots = torch.tensor([int(table[0, t // 16]) * 16 + t % 16 for t in range(150)])
    qps.kv_append_paged(qps.paged_append_args(cache, x[:, :1].cuda(), x[:, 1:].cuda(), slots.cuda()))
    q = (_q(150, 2, d, 1) * 2.0 ** -13).half()
    ro, rl = _want(cache, q, [0, 150], table, lens, d ** -0.5)
    o, lse = _run(qps, q, cache, table, lens, [0, 150], scale=d ** -0.5, out_dtype=torch.float32)
    # Rows of both signs cancel, so the bar per row does not hold.  Weights are rounded once to fp16,
    # each off by 2^-11 of it at most, and sum to one; values come in two parts, exact to 2^-21; sums of
    # 150 float32 terms are off by 150 x 2^-24: relative to the largest value, 65532.
    assert np.isfinite(o).all()
    assert (np.abs(o - ro) <= (2.0 ** -11 + 2.0 ** -21 + 150 * 2.0 ** -24) * 65532).all()
    assert (np.abs(lse - rl) <= 1e-4).all()


def test_prompt_nan_query(qps):  # noqa: F811
    """A query token of NaN has outputs of NaN, the others theirs."""
    d, lens = 128, [300]
    cache, table = _cache_of(qps, "f16", "f16", lens, 64, 2, d, 1)
    q = _q(300, 6, d, 1)
    q[17] = float("nan")
    o, lse = _run(qps, q, cache, table, lens, [0, 300], scale=0.1, out_dtype=torch.float32)
    o, lse = o.reshape(300, 6, d), lse.reshape(300, 6)
    assert np.isnan(o[17]).all() and np.isnan(lse[17]).all()
    keep = [t for t in range(300) if t != 17]
    q[17] = 0
    ro, rl = _want(cache, q, [0, 300], table, lens, 0.1)
    assert_parity(o[keep].reshape(-1, d), lse[keep].reshape(-1), ro.reshape(300, 6, d)[keep].reshape(-1, d), rl.reshape(300, 6)[keep].reshape(-1))


@pytest.mark.parametrize("d,hq,hkv", [(64, 1, 1), (128, 300, 1), (256, 129, 1), (512, 33, 3), (128, 7, 7)])
def test_prompt_groups(qps, d, hq, hkv):  # noqa: F811
    """One head a group, and groups that are more than a tile of rows."""
    new, lens = [3, 40], [130, 40]
    cache, table = _cache_of(qps, "f16", "f16", lens, 16, hkv, d, 1)
    q = _q(43, hq, d, 2)
    ro, rl = _want(cache, q, _starts(new), table, lens, d ** -0.5, window=50, sinks=2)
    o, lse = _run(qps, q, cache, table, lens, _starts(new), scale=d ** -0.5, out_dtype=torch.float32, window=50, sinks=2)
    assert_parity(o, lse, ro, rl, (d, hq, hkv))


def test_prompt_many_sequences(qps):  # noqa: F811
    """More sequences than a warp's lanes, most of a few tokens, many of none."""
    r = np.random.default_rng(0)
    new = [int(n) for n in r.choice([0, 0, 1, 2, 30], 150)]
    lens = [int(n + p) for n, p in zip(new, r.integers(0, 90, 150))]
    for kf, vf in (("f16", "f16"), ("q8_0", "q8_0")):
        cache, table = _cache_of(qps, kf, vf, lens, 16, 2, 64, 1)
        q = _q(sum(new), 8, 64, 2)
        for window, sinks in ((0, 0), (20, 17)):
            ro, rl = _want(cache, q, _starts(new), table, lens, 0.1, window=window, sinks=sinks)
            o, lse = _run(qps, q, cache, table, lens, _starts(new), scale=0.1, out_dtype=torch.float32, window=window, sinks=sinks)
            assert_parity(o, lse, ro, rl, (kf, vf, window))


@pytest.mark.parametrize("d,kf,vf,pages", [(128, "f16", "f16", 2500), (128, "q8_0", "q8_0", 5000), (512, "q8_0", "tq3", 1400)])
def test_cache_past_32_bits(qps, d, kf, vf, pages):  # noqa: F811
    """Pages whose first byte is past 2^32: attended to, forked and moved at both ends of the pool."""
    hkv, page, n = 8, 1024, 1500
    rot, ora = _rotations(d, "whole")
    cache = qps.PagedKV.empty(kf, vf, pages, page, hkv, d, signs=_lib_rot(qps, rot))
    assert cache.k_planes[0].numel() * cache.k_planes[0].element_size() > 1 << 32
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    table = i32([[pages - 1, 0], [1, pages - 2], [-1, -1]])
    refs = torch.zeros(pages, dtype=torch.int32).cuda()
    refs[[pages - 1, 0, 1, pages - 2]] = 1
    seqs = qps.PagedSeqs(cache, table, i32([n, n, 0]), refs)
    g = torch.Generator().manual_seed(d)
    x = torch.randn((2, n, 2 * hkv, d), generator=g).half().cuda()
    at = torch.arange(n).cuda()
    for b in range(2):
        slots = table[b].long()[at // page] * page + at % page
        qps.kv_append_paged(qps.paged_append_args(cache, x[b, :, :hkv], x[b, :, hkv:], slots))
    q = torch.randn((40, hkv * 2, d), generator=g).half().cuda()
    run = lambda: [t.cpu().numpy() for t in qps.attn_prompt_paged(qps.paged_prompt_args(  # noqa: E731
        q, cache, table, seqs.kv_lens, i32([0, 20, 40, 40]), scale=d ** -0.5, out_dtype=torch.float32))]
    o, lse = run()
    used = [pages - 1, 0, 1, pages - 2]  # (the oracle reads these four alone)
    kp, vp = ([p[used].cpu().numpy() for p in s] for s in (cache.k_planes, cache.v_planes))
    ro, rl = os_.attention(q.cpu().numpy(), [0, 20, 40], kf, kp, vf, vp, np.array([[0, 1], [2, 3]]), [n, n], d ** -0.5, signs=ora)
    assert_parity(o, lse, ro.reshape(-1, d), rl.reshape(-1), (d, kf, vf))
    qps.kv_fork_paged(qps.paged_fork_args(seqs, i32([0]), i32([2])))
    assert table[2].tolist() == [pages - 1, 2] and refs[:4].tolist() == [1, 1, 1, 0]
    ids, live = qps.kv_compact_paged(qps.paged_compact_args(seqs))
    assert live.item() == 5 and table.tolist() == [[4, 0], [1, 3], [4, 2]]
    again = run()
    assert np.array_equal(o, again[0]) and np.array_equal(lse, again[1])
    table[0].copy_(table[2].clone())  # (the copy's rows are the source's)
    assert all(np.array_equal(a, b) for a, b in zip((o, lse), run()))


def test_arrays_at_any_address(qps):  # noqa: F811
    """Counts, lengths and tables that start at any multiple of 4 bytes."""
    page, batch, width, pages = 16, 5, 11, 77
    x = Pair(qps, batch, width, pages, page, seed=1)
    for shift in (1, 2, 3):
        cut = lambda n: torch.zeros(n + 8, dtype=torch.int32).cuda()[shift:shift + n]  # noqa: B023,E731
        table = torch.full((batch, width + 6), -1, dtype=torch.int32).cuda()[:, shift:shift + width]
        y = Pair.__new__(Pair)
        y.__dict__.update(x.__dict__)
        y.seqs = qps.PagedSeqs(x.caches, table, cut(batch), cut(pages))
        y.ora = os_.Pages(page, table.cpu().numpy(), [0] * batch, [0] * pages,
                          [p.view(torch.uint8).cpu().numpy() if p.dtype != torch.uint8 else p.cpu().numpy() for p in x.planes()])
        r = np.random.default_rng(shift)
        for _ in range(6):
            y.extend([int(n) for n in r.integers(-20, 60, batch)], 50, 5)
            y.fork([int(n) for n in r.integers(-1, batch, 2)], r.permutation(batch)[:2].tolist())
        y.compact()


def test_two_threads(qps):  # noqa: F811
    """Calls of two host threads on streams of their own, each on its own sequences."""
    d, lens, errors = 128, [700, 300], []
    cache, table = _cache_of(qps, "q8_0", "q8_0", lens, 64, 2, d, 1)
    want = {}
    jobs = []
    for i in range(2):
        q = _q(400, 8, d, i)
        a = _args(qps, q, cache, table, lens, [0, 250, 400], scale=0.1, out_dtype=torch.float32, window=200 * i, sinks=3)
        c2 = qps.PagedKV.empty("f16", "f16", 500, 16, 1, 64)
        s = qps.PagedSeqs.empty(c2, 4, 60)
        n = torch.tensor([30, 1, 0, 17], dtype=torch.int32).cuda()
        jobs.append((a, qps.paged_extend_args(s, n, max_tokens=50), s, torch.cuda.Stream()))
        want[i] = _want(cache, q, [0, 250, 400], table, lens, 0.1, window=200 * i, sinks=3)
    torch.cuda.synchronize()

    def work(a, e, s, stream):
        try:
            for _ in range(12):
                qps.attn_prompt_paged(a, stream=stream)
                qps.kv_extend_paged(e, stream=stream)
        except Exception as x:  # noqa: BLE001
            errors.append(x)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for i, (a, _, s, _) in enumerate(jobs):
        assert_parity(a._out[0].cpu().numpy(), a._out[1].cpu().numpy(), *want[i], tag=i)
        assert s.kv_lens.tolist() == [360, 12, 0, 204] and int(s.refs.sum()) == 23 + 1 + 13
    qps.device_status()


def test_first_calls_captured(qps):  # noqa: F811
    """The first calls of a process may be captured."""
    _child("""
import torch
import quantized_position_split_gb300 as qps
c = qps.PagedKV.empty("q8_0", "q8_0", 40, 16, 2, 128)
s = qps.PagedSeqs.empty(c, 2, 12)
i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
e = qps.paged_extend_args(s, i32([100, 30]), max_tokens=130, window=64, sinks=4)
kv = torch.ones((130, 2, 128), dtype=torch.float16, device="cuda")
p = qps.paged_append_args(c, kv, kv, e._out[1])
q = torch.randn((130, 4, 128), device="cuda").half()
a = qps.paged_prompt_args(q, c, s.page_table, s.kv_lens, e._out[0], scale=0.1, window=64, sinks=4)
f = qps.paged_fork_args(s, i32([0]), i32([1]))
m = qps.paged_compact_args(s)
torch.cuda.synchronize()
g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.graph(g, stream=side):
    qps.kv_extend_paged(e)
    qps.kv_append_paged(p)
    qps.attn_prompt_paged(a)
    qps.kv_fork_paged(f)
    qps.kv_compact_paged(m)
g.replay()
torch.cuda.synchronize()
assert s.kv_lens.tolist() == [100, 100] and m._out[1].item() == 8, (s.kv_lens, m._out[1])
assert (a._out[0].float() - 1).abs().max() < 1e-3
qps.device_status(reset=True)
print("child ok")
""")
