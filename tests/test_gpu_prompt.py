"""Attention of prompt chunks over a paged cache, on the GPU against the float64 oracle: ragged
chunks of every format, windows, rows that nothing may touch, what lies where nothing looks."""

import numpy as np
import pytest
import torch

from oracle import stream as os_
from tests.helpers import assert_parity
from tests.test_gpu_paged import PAIRS, _cache_of, _rotations, qps  # noqa: F401
from tests.test_gpu_paged_edges import _key_plane, _value_plane

pytestmark = pytest.mark.gpu


def _starts(new, first=0):
    return np.concatenate(([first], first + np.cumsum(new))).tolist()


def _want(cache, q, starts, table, lens, scale, softcap=0.0, window=0, sinks=0, ora=None):
    kp, vp = ([p.cpu().numpy() for p in s] for s in (cache.k_planes, cache.v_planes))
    o, lse = os_.attention(q.cpu().numpy(), starts, cache.k_fmt, kp, cache.v_fmt, vp, table.numpy(), lens, scale, softcap, window,
                           sinks, ora)
    return o.reshape(-1, q.shape[-1]), lse.reshape(-1)


def _values(cache, table, n, ora):
    return os_.rows_of(cache.v_fmt, [p.cpu().numpy() for p in cache.v_planes], table[0].numpy(), n, cache.d, ora)


def _args(qps, q, cache, table, lens, starts, **kw):  # noqa: F811
    return qps.paged_prompt_args(q, cache, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                 torch.tensor(starts, dtype=torch.int32).cuda(), **kw)


def _run(qps, *a, **kw):  # noqa: F811
    o, lse = qps.attn_prompt_paged(_args(qps, *a, **kw))
    return o.float().cpu().numpy(), lse.cpu().numpy()


def _q(tokens, hq, d, seed):
    return torch.randn((tokens, hq, d), generator=torch.Generator().manual_seed(seed)).half().cuda()


def _bury(cache, table, lens, new, window, sinks):
    """NaN values and infinite keys where no query token looks; pages of nothing else are given
    back."""
    table, page = table.clone(), cache.page_size
    for b, (n, m) in enumerate(zip(lens, new)):
        seen = os_.visible(n, min(n, m), window, sinks).any(0) if min(n, m) else np.zeros(n, bool)
        for j in range(-(-n // page)):
            here = seen[j * page:(j + 1) * page]
            pg = int(table[b, j])
            if not here.any():
                table[b, j] = -1 - j
            gone = np.ones(page, bool)
            gone[:len(here)] = ~here
            at = torch.from_numpy(np.flatnonzero(gone)).cuda()
            _key_plane(cache)[pg].index_fill_(1, at, float("inf"))
            _value_plane(cache)[pg].index_fill_(1, at, float("nan"))
    return table


NEW = [1, 0, 5, 17, 64, 130, 3, 300]
LENS = [1, 40, 200, 17, 129, 515, 1000, 300]


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("kf,vf", PAIRS)
def test_prompt_ragged(qps, d, kf, vf):  # noqa: F811
    """Every format: chunks of one token and of hundreds, without past and behind one, sequences
    without tokens, groups of any size, windows and sinks, softcap."""
    hkv = 2
    for page, group, softcap, window, sinks in ((16, 4, 0.0, 0, 0), (64, 1, 30.0, 0, 0), (32, 5, 0.0, 100, 4), (128, 3, 0.0, 1, 0),
                                                (1024, 2, 0.0, 300, 140)):
        rot, ora = _rotations(d, "block" if page == 64 else "whole")
        cache, table = _cache_of(qps, kf, vf, LENS, page, hkv, d, d + page, rot)
        table = _bury(cache, table, LENS, NEW, window, sinks)
        q = _q(sum(NEW), hkv * group, d, d + group)
        kw = dict(scale=d ** -0.5, softcap=softcap, window=window, sinks=sinks)
        ro, rl = _want(cache, q, _starts(NEW), table, LENS, ora=ora, **kw)
        for _ in range(2):
            o, lse = _run(qps, q, cache, table, LENS, _starts(NEW), out_dtype=torch.float32, **kw)
            assert_parity(o, lse, ro, rl, (d, kf, vf, page, window, sinks))


@pytest.mark.parametrize("d,kf,vf,group", [(64, "f16", "f16", 5), (128, "f16", "f16", 5), (128, "q8_0", "tq3", 4), (256, "f16", "f16", 4),
                                           (256, "q8_0", "q8_0", 3), (512, "q8_0", "tq3", 8), (512, "f16", "f16", 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 130)])
def test_prompt_many_tiles(qps, d, kf, vf, group, window, sinks):  # noqa: F811
    """Chunks whose pipelines go round many times; maxima that rise late (keys that grow along the
    sequence) rescale what has been summed."""
    hkv, page = 3, 64
    new, lens = [1500, 700], [1500, 3100]
    rot, ora = _rotations(d, "whole")
    cache, table = _cache_of(qps, kf, vf, lens, page, hkv, d, d, rot)
    if kf == "f16":
        for b, n in enumerate(lens):
            for j in range(-(-n // page)):
                cache.k_planes[0][int(table[b, j])] *= 0.5 + 1.5 * j * page / n
    q = _q(sum(new), hkv * group, d, d)
    kw = dict(scale=d ** -0.5, window=window, sinks=sinks)
    ro, rl = _want(cache, q, _starts(new), table, lens, ora=ora, **kw)
    for _ in range(3):  # (a race does not show every time)
        o, lse = _run(qps, q, cache, table, lens, _starts(new), out_dtype=torch.float32, **kw)
        assert_parity(o, lse, ro, rl, (d, kf, vf, group))


@pytest.mark.parametrize("d,kf,vf", [(128, "f16", "f16"), (512, "q8_0", "tq3"), (64, "f16", "q8_0"), (256, "tq2", "tq2")])
@pytest.mark.parametrize("tokens,past", [(1, 5000), (3, 20000), (40, 9000)])
def test_prompt_split_positions(qps, d, kf, vf, tokens, past):  # noqa: F811
    """Few tokens behind many positions: the positions are shared among CTAs; the fp16 output is the
    float32 one, rounded once, and so is the bf16 one over fp16 values."""
    hkv, group, page = 2, 4, 64
    rot, ora = _rotations(d, "whole")
    lens = [past + tokens]
    cache, table = _cache_of(qps, kf, vf, lens, page, hkv, d, d, rot)
    q = _q(tokens, hkv * group, d, tokens)
    for window, sinks in ((0, 0), (1000, 3)):
        kw = dict(scale=d ** -0.5, window=window, sinks=sinks)
        ro, rl = _want(cache, q, [0, tokens], table, lens, ora=ora, **kw)
        o, lse = _run(qps, q, cache, table, lens, [0, tokens], out_dtype=torch.float32, **kw)
        assert_parity(o, lse, ro, rl, (d, kf, vf, tokens, past))
        for dt in (torch.float16, torch.bfloat16):
            half, l2 = _run(qps, q, cache, table, lens, [0, tokens], out_dtype=dt, **kw)
            assert np.array_equal(l2, lse)
            if dt == torch.float16 or vf == "f16":
                assert np.array_equal(half, torch.from_numpy(o).to(dt).float().numpy())
            else:
                # a compressed V is rounded to fp16 first: each value off by 2^-11 of it at most, and
                # weights that sum to one; then bf16's half step, 2^-8
                big = np.abs(_values(cache, table, lens[0], ora)).max()
                assert (np.abs(half - o) <= 2.0 ** -8 * np.abs(o) + 1.01 * 2.0 ** -11 * big).all()


@pytest.mark.parametrize("d,kf,vf", [(128, "f16", "f16"), (256, "q8_0", "q8_0")])
def test_prompt_rows_of_no_sequence(qps, d, kf, vf):  # noqa: F811
    """Rows before the first and behind the last token stay; tokens before the first position see
    nothing; strided queries and tables."""
    hkv, group, page = 2, 3, 32
    new, lens = [7, 200, 4], [3, 200, 0]
    cache, table = _cache_of(qps, kf, vf, lens, page, hkv, d, d)
    starts = _starts(new, first=5)
    tokens = starts[-1] + 9
    wide = torch.randn((tokens, hkv * group + 4, d), generator=torch.Generator().manual_seed(0)).half().cuda()
    q = wide[:, :hkv * group]
    big = torch.full((len(lens), table.shape[1] + 3), 1 << 30, dtype=torch.int32).cuda()
    big[:, :table.shape[1]] = table.cuda()
    ro, rl = np.zeros((tokens, hkv * group, d)), np.full((tokens, hkv * group), -np.inf)
    for b, (n, m) in enumerate(zip(lens, new)):
        have = min(n, m)
        if have:
            s0 = starts[b] + m - have
            o, lse = _want(cache, q[s0:s0 + have], [0, have], table[b:b + 1], [n], 0.1)
            ro[s0:s0 + have], rl[s0:s0 + have] = o.reshape(have, -1, d), lse.reshape(have, -1)
    rows = tokens * hkv * group
    for few in (False, True):  # (one sequence alone: positions are split)
        o = torch.full((rows, d), 7.0, device="cuda")
        lse = torch.full((rows,), 7.0, device="cuda")
        if few:
            a = qps.paged_prompt_args(q[:12], cache, big[:1, :table.shape[1]], torch.tensor(lens[:1], dtype=torch.int32).cuda(),
                                      torch.tensor([5, 12], dtype=torch.int32).cuda(), scale=0.1, out_dtype=torch.float32,
                                      o=o[:12 * hkv * group], lse=lse[:12 * hkv * group])
        else:
            a = qps.paged_prompt_args(q, cache, big[:, :table.shape[1]], torch.tensor(lens, dtype=torch.int32).cuda(),
                                      torch.tensor(starts, dtype=torch.int32).cuda(), scale=0.1, out_dtype=torch.float32, o=o, lse=lse)
        qps.attn_prompt_paged(a)
        o, lse = o.view(tokens, -1, d), lse.view(tokens, -1)
        s0, s1 = (5, 12) if few else (5, starts[-1])
        assert (o[:s0] == 7).all() and (o[s1:] == 7).all() and (lse[:s0] == 7).all() and (lse[s1:] == 7).all()
        assert_parity(o[s0:s1].reshape(-1, d).cpu().numpy(), lse[s0:s1].reshape(-1).cpu().numpy(), ro[s0:s1].reshape(-1, d), rl[s0:s1].reshape(-1))


def test_prompt_is_the_decode_call_for_single_tokens(qps):  # noqa: F811
    """One token a sequence: what attn_decode_paged gives, within both calls' bounds."""
    lens, d = [1, 33, 700, 64], 128
    cache, table = _cache_of(qps, "q8_0", "q8_0", lens, 64, 2, d, 3)
    q = _q(4, 8, d, 1)
    for window, sinks in ((0, 0), (50, 7)):
        want = qps.attn_decode_paged(qps.paged_attn_args(q, cache, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), scale=0.09,
                                                         out_dtype=torch.float32, window=window, sinks=sinks))
        o, lse = _run(qps, q, cache, table, lens, [0, 1, 2, 3, 4], scale=0.09, out_dtype=torch.float32, window=window, sinks=sinks)
        assert_parity(o, lse, want[0].double().cpu().numpy(), want[1].double().cpu().numpy())


def test_prompt_bad_indexes(qps):  # noqa: F811
    """Lengths, starts and entries out of range: nothing is followed, the others are right, the
    status says so."""
    d, hkv, page = 128, 2, 32
    lens, new = [200, 100, 64], [20, 10, 64]
    cache, table = _cache_of(qps, "f16", "f16", lens, page, hkv, d, 1)
    q = _q(sum(new), 4, d, 1)
    starts = _starts(new)
    ro, rl = _want(cache, q, starts, table, lens, 0.1)
    qps.device_status(reset=True)

    def check(rows, *, t=table, n=lens, s=starts):
        o, lse = _run(qps, q, cache, t, n, s, scale=0.1, out_dtype=torch.float32)
        with pytest.raises(qps.QpsError):
            qps.device_status(reset=True)
        pick = np.concatenate([np.arange(a * 4, b * 4) for a, b in rows])
        assert_parity(o[pick], lse[pick], ro[pick], rl[pick])
        return o, lse

    bad = table.clone()
    bad[1, 0] = cache.n_pages  # its rows read as zeros
    check([(0, 20), (30, 94)], t=bad)
    bad[1, 0] = -5
    check([(0, 20), (30, 94)], t=bad)
    check([(20, 94)], n=[1 << 30, 100, 64])
    check([(20, 94)], n=[-3, 100, 64])
    check([(40, 94)], s=[0, 40, 30, 94])  # (rows that two sequences name hold either one's)
    check([(0, 20)], s=[0, 20, 30, 1 << 30])
    check([(20, 94)], s=[-1, 20, 30, 94])
    qps.device_status(reset=True)


def test_prompt_in_a_captured_graph(qps):  # noqa: F811
    """One graph: lengths, starts and tables of other batches, up to all of its tokens in one."""
    d, hkv, page, width, tokens = 128, 2, 32, 40, 90
    cache, table = _cache_of(qps, "q8_0", "q8_0", [page * width] * 3, page, hkv, d, 1)
    table = table[:, :width].contiguous()  # (the pages that hold rows)
    q = _q(tokens, 8, d, 1)
    lens, starts = (torch.zeros(n, dtype=torch.int32).cuda() for n in (3, 4))
    a = qps.paged_prompt_args(q, cache, table.cuda(), lens, starts, scale=0.1, window=200, sinks=5)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        qps.attn_prompt_paged(a)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            o, lse = qps.attn_prompt_paged(a)
    torch.cuda.synchronize()
    for n, s in (([50, 60, 70], [0, 30, 60, 90]), ([1280, 5, 1], [0, 85, 89, 90]), ([90, 7, 1000], [0, 90, 90, 90]), ([1, 1, 1], [0, 1, 2, 3])):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        starts.copy_(torch.tensor(s, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        ro, rl = _want(cache, q, s, table, n, 0.1, window=200, sinks=5)
        rows = s[-1] * 8
        assert_parity(o[:rows].float().cpu().numpy(), lse[:rows].cpu().numpy(), ro[:rows], rl[:rows], (n, s))


def test_prompt_streams_and_empty_calls(qps):  # noqa: F811
    """Two calls at once on streams of their own; no tokens."""
    d, lens = 128, [3000]
    cache, table = _cache_of(qps, "f16", "f16", lens, 64, 2, d, 1)
    qs = [_q(1000, 8, d, s) for s in (1, 2)]
    args = [_args(qps, q, cache, table, lens, [0, 1000], scale=0.1, out_dtype=torch.float32) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(5):
        for a, s in zip(args, streams):
            qps.attn_prompt_paged(a, stream=s)
    torch.cuda.synchronize()
    for q, a in zip(qs, args):
        ro, rl = _want(cache, q, [0, 1000], table, lens, 0.1)
        assert_parity(a._out[0].cpu().numpy(), a._out[1].cpu().numpy(), ro, rl)
    o, lse = qps.attn_prompt_paged(_args(qps, qs[0][:0], cache, table, lens, [0, 0], scale=0.1))
    assert o.shape == (0, d) and lse.shape == (0,)


@pytest.mark.parametrize("d,kf,vf", [(128, "f16", "f16"), (64, "f16", "f16"), (256, "q8_0", "q8_0"), (512, "q8_0", "tq3")])
@pytest.mark.parametrize("tile", [0, 1, 4])
def test_a_prompt_tile_that_never_comes(qps, d, kf, vf, tile):  # noqa: F811
    """The keys of a tile are withheld: the waits give up, the status says so, the next call is right."""
    rot, ora = _rotations(d, "whole")
    lens, new = [900], [300]
    cache, table = _cache_of(qps, kf, vf, lens, 64, 2, d, 2, rot)
    q = _q(300, 4, d, 1)
    a = _args(qps, q, cache, table, lens, [0, 300], scale=0.1, out_dtype=torch.float32)
    qps.device_status(reset=True)
    qps.paged_inject_fault(tile, 20)
    qps.attn_prompt_paged(a)
    torch.cuda.synchronize()
    if tile == 0:
        with pytest.raises(qps.QpsError, match="TIMEOUT"):
            qps.device_status(reset=True)
    else:  # (a split call's CTAs may hold fewer tiles)
        try:
            qps.device_status(reset=True)
        except qps.QpsError as e:
            assert "TIMEOUT" in str(e)
    o, lse = qps.attn_prompt_paged(a)
    ro, rl = _want(cache, q, [0, 300], table, lens, 0.1, ora=ora)
    assert_parity(o.cpu().numpy(), lse.cpu().numpy(), ro, rl)
