"""The page tables of a paged cache on the GPU against the entry-by-entry oracle: every table,
count, length and byte of every plane after each call; what does not fit; runs of the calls with
the appends and attention that use them."""

import numpy as np
import pytest
import torch

from oracle import stream as os_
from tests.helpers import assert_parity
from tests.test_gpu_paged import _bits, _fill, qps  # noqa: F401
from tests.test_gpu_prompt import _q, _want

pytestmark = pytest.mark.gpu

FORMATS = [("f16", "f16"), ("q8_0", "tq3"), ("tq4", "tq4"), ("q8_0", "q8_0")]


class Pair:
    """The library's state and the oracle's, compared after every call."""

    def __init__(self, qps, batch, width, pages, page, layers=1, hkv=2, d=64, seed=0, wide=0):  # noqa: F811
        self.qps = qps
        signs = torch.arange(d // 32, dtype=torch.int32) + 5
        self.caches = []
        for i in range(layers):
            kf, vf = FORMATS[(seed + i) % len(FORMATS)]
            self.caches.append(qps.PagedKV.empty(kf, vf, pages, page, hkv + i % 2, d, signs=signs))
            _fill(self.caches[-1], seed + i)
        table = torch.full((batch, width + wide), -1, dtype=torch.int32).cuda()[:, :width]
        self.seqs = qps.PagedSeqs(self.caches, table, torch.zeros(batch, dtype=torch.int32).cuda(), torch.zeros(pages, dtype=torch.int32).cuda())
        planes = [p.view(torch.uint8).cpu().numpy() if p.dtype != torch.uint8 else p.cpu().numpy() for p in self.planes()]
        self.ora = os_.Pages(page, table.cpu().numpy(), [0] * batch, [0] * pages, planes)
        qps.device_status(reset=True)

    def planes(self):
        return [p if p.dim() > 3 else p[..., None] for c in self.caches for p in c.k_planes + c.v_planes]

    def check(self, tag=""):
        torch.cuda.synchronize()
        s, o = self.seqs, self.ora
        assert s.kv_lens.tolist() == o.lens, tag
        assert s.refs.tolist() == o.refs, tag
        assert s.page_table.tolist() == o.table, tag
        for a, b in zip(self.planes(), o.planes):
            assert torch.equal(_bits(a), torch.from_numpy(b).reshape(-1)), tag
        if o.bad:
            with pytest.raises(self.qps.QpsError):
                self.qps.device_status(reset=True)
            o.bad = False
        else:
            self.qps.device_status()

    def _t(self, x):
        return torch.tensor(x, dtype=torch.int32).cuda()

    def extend(self, n_new, window=0, sinks=0, max_tokens=None):
        if max_tokens is None:
            max_tokens = sum(max(0, n) for n in n_new) + 3
        got = self.qps.kv_extend_paged(self.qps.paged_extend_args(self.seqs, self._t(n_new), max_tokens=max_tokens, window=window, sinks=sinks))
        want = self.ora.extend(n_new, window, sinks, max_tokens)
        assert [t.tolist() for t in got] == [list(w) for w in want]
        self.check(("extend", n_new, window, sinks))
        return got

    def fork(self, src, dst):
        self.qps.kv_fork_paged(self.qps.paged_fork_args(self.seqs, self._t(src), self._t(dst)))
        self.ora.fork(src, dst)
        self.check(("fork", src, dst))

    def compact(self):
        ids, live = self.qps.kv_compact_paged(self.qps.paged_compact_args(self.seqs))
        want, n = self.ora.compact()
        assert ids.tolist() == want and live.tolist() == [n]
        self.check("compact")


# (batch, width, pages): one CTA and a cluster, by either rule, and odd numbers of pages
SHAPES = [(1, 40, 37, 16), (1, 40, 37, 64), (5, 20, 64, 16), (5, 20, 64, 64), (33, 12, 333, 16), (7, 30, 4099, 16), (3, 9, 9001, 16)]


@pytest.mark.parametrize("batch,width,pages,page", SHAPES)
def test_random_calls(qps, batch, width, pages, page):  # noqa: F811
    """Growing, trimming, forking, giving back and compacting at random, windows that change,
    pools that run out, rows that are full."""
    r = np.random.default_rng(batch + pages)
    large = pages > 1000  # (every byte of every plane is compared after every call)
    x = Pair(qps, batch, width, pages, page, layers=1 if large else 1 + batch % 3, hkv=1 if large else 2, seed=1 if large else batch,
             wide=batch % 2 * 3)
    cap = width * page
    for step in range(16 if large else 24):
        what = r.integers(0, 10)
        if what < 6:
            big = min(cap, max(4, pages * page // batch // 3))
            new = [int(r.choice([0, 1, 1, r.integers(1, big + 1), -int(r.integers(1, big + 1)), page])) for _ in range(batch)]
            window = int(r.choice([0, 0, 1, page, r.integers(1, cap), cap + 5]))
            x.extend(new, window, int(r.choice([0, 1, page, page + 1, 3 * page])) if window else 0)
        elif what < 9:
            n = int(r.integers(1, batch + 1))
            dst = r.permutation(batch)[:n].tolist()
            x.fork([int(r.integers(-1, batch)) for _ in range(n)], dst)
        else:
            x.compact()


def test_shared_last_pages(qps):  # noqa: F811
    """Trimmed into a page that others name too: the next growth copies its rows, for each of the
    sequences that grow; a page with one use is written where it is."""
    x = Pair(qps, 5, 8, 40, 16, layers=3, seed=1)
    x.extend([100, 0, 0, 0, 0])
    x.fork([0, 0, 0], [1, 2, 3])
    x.extend([-30, -30, -25, -100, 0])
    x.extend([1, 30, 0, 5, 16])   # sequences 0 and 1 both leave the page that 2 keeps
    x.extend([0, 0, 1, 0, 0])     # 2 has it alone by now
    x.fork([1, 2], [2, 1])        # trading places
    x.fork([4, 4, -1, 1], [0, 1, 2, 4])
    x.compact()


def test_running_out(qps):  # noqa: F811
    """No free page: a sequence is served whole or not at all, later ones that need none are."""
    x = Pair(qps, 4, 8, 6, 16)
    x.extend([40, 20, 0, 0])      # 5 of 6 pages
    x.extend([3, 2, 20, 1])       # 0 and 1 grow in place, 2 does not fit, nor does 3 behind it
    x.extend([0, 0, 0, 16])
    x.extend([0, 0, 0, 1])
    x.fork([0, 1], [2, 3])        # frees one page, needs two
    x.extend([-100, 0, 0, 0])
    x.extend([200, 1, 0, 0])      # longer than its row
    x.extend([5, 5, 5, 5], max_tokens=12)
    x.extend([2 ** 31 - 1, 2 ** 31 - 1, 1, -2 ** 31], max_tokens=12)
    x.extend([0, 0, 0, 0], max_tokens=0)
    x.extend([-1, -1, 0, 0], max_tokens=0)


def test_indexes_out_of_range(qps):  # noqa: F811
    """Lengths behind the row, sources and destinations out of range, a destination twice, entries
    that name nothing, counts that would fall below 0."""
    x = Pair(qps, 4, 6, 50, 16, layers=2)
    x.extend([30, 40, 50, 60])
    x.fork([0, 9, 1, 1, -5], [7, 1, -1, 3, 2])
    x.fork([0, 1, 2], [3, 3, 3])
    x.fork([0, 3, 0], [0, 0, 1])  # (the first of a pair is a no-op and still the first)
    for t in (x.seqs.kv_lens, x.seqs.page_table[:, 0]):
        t[2] = 10 ** 6
    x.ora.lens[2] = x.ora.table[2][0] = 10 ** 6
    x.extend([1, 1, 1, 1])
    x.fork([2], [0])
    x.seqs.refs.zero_()
    x.ora.refs = [0] * 50
    x.extend([-20, -20, -20, -20])


def test_windows_give_pages_back(qps):  # noqa: F811
    """A long stream in a window holds a constant number of pages."""
    page, window, sinks = 16, 100, 20
    x = Pair(qps, 2, 200, 60, page, layers=1)
    x.extend([300, 150], window, sinks)
    most = 0
    for step in range(60):
        x.extend([7, 40 if step % 9 == 0 else -5], window, sinks)
        most = max(most, sum(r > 0 for r in x.ora.refs))
    assert x.ora.lens[0] == 720 and most <= 2 * (-(-sinks // page) + (window + 40) // page + 2)


@pytest.mark.parametrize("kf,vf", [("f16", "f16"), ("q8_0", "tq3")])
def test_serving_loop(qps, kf, vf):  # noqa: F811
    """Extend, append, prompt attention; fork; window decode; trim; compact; two layers: attention
    gives what the tables say, and the same after the pages have moved."""
    d, hkv, hq, page, batch, width = 128, 2, 6, 32, 5, 30
    g = torch.Generator().manual_seed(1)
    signs = torch.arange(d // 32, dtype=torch.int32) * 77 + 3
    caches = [qps.PagedKV.empty(kf, vf, 90, page, hkv, d, signs=signs) for _ in range(2)]
    seqs = qps.PagedSeqs.empty(caches, batch, width)
    n_new = torch.zeros(batch, dtype=torch.int32).cuda()
    most = 400
    window, sinks = 90, 5
    ext = qps.paged_extend_args(seqs, n_new, max_tokens=most, window=window, sinks=sinks)
    starts, slots, positions = ext._out
    k, v, q = (torch.zeros((most, h, d), dtype=torch.float16, device="cuda") for h in (hkv, hkv, hq))
    appends = [qps.paged_append_args(c, k, v, slots) for c in caches]
    prompts = [qps.paged_prompt_args(q, c, seqs.page_table, seqs.kv_lens, starts, scale=d ** -0.5, window=window, sinks=sinks,
                                     out_dtype=torch.float32) for c in caches]
    qd = torch.randn((batch, hq, d), generator=g).half().cuda()
    decodes = [qps.paged_attn_args(qd, c, seqs.page_table, seqs.kv_lens, scale=d ** -0.5, window=window, sinks=sinks,
                                   out_dtype=torch.float32) for c in caches]
    qps.device_status(reset=True)

    def step(new):
        n_new.copy_(torch.tensor(new, dtype=torch.int32))
        for t in (k, v, q):
            t.copy_(torch.randn(t.shape, generator=g))
        qps.kv_extend_paged(ext)
        out = []
        for a, p in zip(appends, prompts):
            qps.kv_append_paged(a)
            out.append([t.clone() for t in qps.attn_prompt_paged(p)])
        table, lens, s = seqs.page_table.cpu(), seqs.kv_lens.tolist(), starts.tolist()
        for (o, lse), c in zip(out, caches) if s[-1] else ():
            ro, rl = _want(c, q[:s[-1]], s, table, lens, d ** -0.5, 0.0, window, sinks, signs.numpy())
            assert_parity(o[:s[-1] * hq].cpu().numpy(), lse[:s[-1] * hq].cpu().numpy(), ro, rl, new)

    def decode():
        out = []
        for a, c in zip(decodes, caches):
            o, lse = qps.attn_decode_paged(a)
            table, lens = seqs.page_table.cpu(), seqs.kv_lens.tolist()
            ro, rl = np.zeros((batch, hq, d)), np.full((batch, hq), -np.inf)
            for b, n in enumerate(lens):
                if n:
                    o1, l1 = _want(c, qd[b:b + 1], [0, 1], table[b:b + 1], [n], d ** -0.5, 0.0, window, sinks, signs.numpy())
                    ro[b], rl[b] = o1, l1
            assert_parity(o.cpu().numpy(), lse.cpu().numpy(), ro.reshape(-1, d), rl.reshape(-1))
            out.append((o.clone(), lse.clone()))
        return out

    step([200, 31, 0, 64, 1])
    step([1, 1, 33, 150, 0])
    qps.kv_fork_paged(qps.paged_fork_args(seqs, torch.tensor([0, 0, -1], dtype=torch.int32).cuda(),
                                          torch.tensor([2, 4, 1], dtype=torch.int32).cuda()))
    decode()
    step([5, 0, 5, 5, 5])
    step([-3, 0, -1, -5, 0])
    step([1, 7, 1, 1, 1])
    before = decode()
    qps.kv_compact_paged(qps.paged_compact_args(seqs))
    live = int((seqs.refs > 0).sum())
    assert (seqs.refs[:live] > 0).all() and int(seqs.page_table.max()) < live
    for (a, b), (c, e) in zip(before, decode()):
        assert torch.equal(a, c) and torch.equal(b, e)
    step([100, 100, 3, 0, 50])
    qps.device_status()


def test_captured_loop(qps):  # noqa: F811
    """Extend, fork and compact in one graph, replayed with other numbers, against the oracle; two
    graphs on the same sequences, one behind the other."""
    x = Pair(qps, 6, 12, 80, 16, layers=2, seed=2)
    n_new, src, dst = (torch.zeros(n, dtype=torch.int32).cuda() for n in (6, 3, 3))
    ext = qps.paged_extend_args(x.seqs, n_new, max_tokens=60, window=70, sinks=3)
    fork, comp = qps.paged_fork_args(x.seqs, src, dst), qps.paged_compact_args(x.seqs)
    dst.copy_(torch.tensor([0, 1, 2]))
    src.copy_(torch.tensor([0, 1, 2]))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for call, a in ((qps.kv_extend_paged, ext), (qps.kv_fork_paged, fork), (qps.kv_compact_paged, comp)):
            call(a)
        graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = qps.kv_extend_paged(ext)
            qps.kv_fork_paged(fork)
        with torch.cuda.graph(other, stream=side):
            ids, live = qps.kv_compact_paged(comp)
    torch.cuda.synchronize()
    r = np.random.default_rng(5)
    for step in range(12):
        new = [int(n) for n in r.integers(-6, 11, 6)]
        s, t = [int(n) for n in r.integers(-1, 6, 3)], r.permutation(6)[:3].tolist()
        n_new.copy_(torch.tensor(new, dtype=torch.int32))
        src.copy_(torch.tensor(s, dtype=torch.int32))
        dst.copy_(torch.tensor(t, dtype=torch.int32))
        graph.replay()
        want = x.ora.extend(new, 70, 3, 60)
        x.ora.fork(s, t)
        x.check((step, new, s, t))
        assert [u.tolist() for u in out] == [list(w) for w in want]
        if step % 3 == 2:
            other.replay()
            a, n = x.ora.compact()
            x.check(step)
            assert ids.tolist() == a and live.tolist() == [n]


def test_many_planes_and_large_pages(qps):  # noqa: F811
    """More planes than one launch copies; pages of many chunks; part of a page of 1024 rows."""
    x = Pair(qps, 2, 3, 9, 1024, layers=40, hkv=1, d=64, seed=1)
    x.extend([1500, 3])
    x.fork([0], [1])
    x.extend([-477, -476])
    x.extend([3, 3])
    x.extend([-3000, 0])
    x.compact()


def test_large_pool(qps):  # noqa: F811
    """Counts of a million pages; the free ones at the far end."""
    pages, page = 1 << 20, 16
    cache = qps.PagedKV.empty("tq2", "tq2", pages, page, 1, 64, signs=torch.arange(2, dtype=torch.int32))
    seqs = qps.PagedSeqs.empty(cache, 3, 20000)
    seqs.refs.fill_(1)
    at = torch.arange(pages - 30000, pages, 2)
    seqs.refs[at.cuda()] = 0
    n = torch.tensor([5000, 16 * 10000, 1], dtype=torch.int32).cuda()
    qps.device_status(reset=True)
    starts, slots, _ = qps.kv_extend_paged(qps.paged_extend_args(seqs, n, max_tokens=200000))
    qps.device_status()
    assert starts.tolist() == [0, 5000, 165000, 165001]
    need = 313 + 10000 + 1
    assert torch.equal(torch.cat((seqs.page_table[0, :313], seqs.page_table[1, :10000], seqs.page_table[2, :1])).cpu().long(), at[:need])
    assert (slots[165001:] == -1).all() and slots[165000] == int(at[need - 1]) * page
    ids, live = qps.kv_compact_paged(qps.paged_compact_args(seqs))
    used = pages - 15000 + need
    assert live.tolist() == [used] and int((ids >= 0).sum()) == used and torch.equal(ids[ids >= 0].sort().values.cpu(), torch.arange(used, dtype=torch.int32))


def test_as_many_sequences_as_a_call_takes(qps):  # noqa: F811
    """4096 sequences, each of them a fork of another."""
    r = np.random.default_rng(1)
    x = Pair(qps, 4096, 5, 14000, 16, hkv=1, seed=1)
    for _ in range(2):
        x.extend([int(n) for n in r.integers(-20, 40, 4096)], 30, 2)
        x.fork([int(n) for n in r.integers(-1, 4096, 4096)], r.permutation(4096).tolist())
    x.compact()
