"""Long streams in a paged cache (oracle): attention behind a sliding window with a few first
positions that stay visible, prompt chunks, and the page tables' operators, entry by entry.

The pages describe none of these.  Definitions (the library's header states the same):

  * query token i of a sequence of n positions whose n_q newest are the queries' own is its
    position q = n - n_q + i; it sees t <= q with t > q - window (window 0: no such limit) or
    t < sinks;
  * a table row names the page of each page_size positions, -1 none; refs counts the entries
    that name a page.
"""

from __future__ import annotations

import numpy as np

from . import paged


def visible(n: int, n_q: int, window: int = 0, sinks: int = 0) -> np.ndarray:
    """[n_q, n]: what each query token sees."""
    q, t = np.arange(n - n_q, n)[:, None], np.arange(n)
    seen = t <= q
    if window:
        seen &= (t > q - window) | (t < sinks)
    return seen


def attend(q, k, v, seen, scale: float, softcap: float = 0.0):
    """``q[n_q, hq, D]`` over ``k, v[n, hkv, D]`` where ``seen[n_q, n]``, float64; what a query
    does not see is not looked at.  (O [n_q, hq, D], lse [n_q, hq]); nothing seen: 0, -inf."""
    q = np.asarray(q, dtype=np.float64)
    group = q.shape[1] // k.shape[1]
    used = seen.any(0)
    seen, k, v = seen[:, used], k[used], v[used]
    o, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    some = seen.any(1)
    if not some.any():
        return o, lse
    for h in range(q.shape[1]):
        s = scale * (q[:, h] @ k[:, h // group].T)
        if softcap > 0:
            s = softcap * np.tanh(s / softcap)
        s = np.where(seen, s, -np.inf)[some]
        m = s.max(1, keepdims=True)
        p = np.exp(s - m)
        den = p.sum(1, keepdims=True)
        o[some, h] = (p / den) @ v[:, h // group]
        lse[some, h] = (m + np.log(den))[:, 0]
    return o, lse


def rows_of(cache_fmt: str, planes, entries, n: int, d: int, signs=None) -> np.ndarray:
    """The first n positions of a sequence, float64 [n, hkv, D]; positions on no page are NaN."""
    page = planes[0].shape[2]
    entries = np.asarray(entries)[:-(-n // page)]
    own = [np.asarray(p)[np.maximum(entries, 0)] for p in planes]
    own = [np.moveaxis(p, 2, 1).reshape((-1, p.shape[1]) + p.shape[3:])[:n] for p in own]
    with np.errstate(invalid="ignore"):  # (what nothing sees may hold anything)
        x = paged.values(cache_fmt, own, d, signs)
    x[np.repeat(entries < 0, page)[:n]] = np.nan
    return x


def attention(q, starts, k_fmt, k_planes, v_fmt, v_planes, table, lens, scale, softcap=0.0, window=0, sinks=0, signs=None):
    """Attention of the query tokens ``q[tokens, hq, D]``, those of sequence b being
    ``[starts[b], starts[b + 1])`` and its newest positions: (O [tokens, hq, D], lse)."""
    q = np.asarray(q, dtype=np.float64)
    d = q.shape[-1]
    o, lse = np.zeros(q.shape), np.full(q.shape[:2], -np.inf)
    for b, n in enumerate(lens):
        i0, i1 = starts[b], starts[b + 1]
        if i1 > i0 and n > 0:
            k, v = (rows_of(f, p, table[b], n, d, signs) for f, p in ((k_fmt, k_planes), (v_fmt, v_planes)))
            o[i0:i1], lse[i0:i1] = attend(q[i0:i1], k, v, visible(n, i1 - i0, window, sinks), scale, softcap)
    return o, lse


class Pages:
    """The page tables of a paged cache, entry by entry on the host: ``table[batch][width]``,
    ``lens``, ``refs`` and the planes ``[n_pages, ...page offset third...]`` of every cache.
    ``bad`` is set where the library's device status would say so."""

    def __init__(self, page: int, table, lens, refs, planes=()):
        self.page, self.bad = page, False
        self.table = [[int(e) for e in row] for row in np.asarray(table)]
        self.lens, self.refs = [int(n) for n in lens], [int(n) for n in refs]
        self.planes = [np.array(p) for p in planes]

    def _count(self, n: int) -> int:
        return -(-n // self.page)

    def _ok(self, pg: int) -> bool:
        return 0 <= pg < len(self.refs)

    def _drop(self, pg: int):
        if self._ok(pg):
            if self.refs[pg] <= 0:
                self.bad = True
            else:
                self.refs[pg] -= 1

    def _copy(self, a: int, b: int, rows: int):
        for p in self.planes:
            p[b][:, :rows] = p[a][:, :rows]

    def _lens(self):
        most = len(self.table[0]) * self.page
        cut = [min(max(n, 0), most) for n in self.lens]
        self.bad |= cut != self.lens
        return cut

    def extend(self, n_new, window: int = 0, sinks: int = 0, max_tokens: int = 0):
        """(q_starts, slots, positions)"""
        lens, held = self._lens(), len(self.table[0]) * self.page
        if window >= held or sinks >= held:
            window = 0
        ends = [max(0, n + m) for n, m in zip(lens, n_new)]
        for row, n, end, m in zip(self.table, lens, ends, n_new):
            low = (n if m > 0 else end) - window + 1
            for j in range(self._count(n)):
                behind = window > 0 and (j + 1) * self.page <= low and j * self.page >= sinks
                if (j >= self._count(end) or behind) and self._ok(row[j]):
                    self._drop(row[j])
                    row[j] = -1
        starts, wants = [0], []
        for row, n, end, m in zip(self.table, lens, ends, n_new):
            starts.append(starts[-1] + max(0, m))
            want = []  # entries that need a page, the copied one first
            if m > 0:
                if end > held or starts[-1] > max_tokens:
                    want = None
                else:
                    at = n // self.page
                    if n % self.page and self._ok(row[at]) and self.refs[row[at]] > 1:
                        want.append(at)
                    want += range(self._count(n), self._count(end))
            wants.append(want)
        free = [p for p, r in enumerate(self.refs) if r == 0]
        used, copies = 0, []
        for b, want in enumerate(wants):
            if want is None or (want and used + len(want) > len(free)):
                self.bad = True
                used += len(want or ())
                wants[b] = None
                continue
            for j in want:
                old, new = self.table[b][j] if j * self.page < lens[b] else -1, free[used]
                used += 1
                self.table[b][j], self.refs[new] = new, 1
                if old >= 0:
                    copies.append((old, new, lens[b] % self.page))
        for old, new, rows in copies:
            self._copy(old, new, rows)
            self._drop(old)
        slots, positions = [-1] * max_tokens, [0] * max_tokens
        for b, m in enumerate(n_new):
            for to in range(min(starts[b], max_tokens), min(starts[b] + max(0, m), max_tokens)):
                t = lens[b] + to - starts[b]
                pg = -1 if wants[b] is None else self.table[b][t // self.page]
                slots[to] = pg * self.page + t % self.page if self._ok(pg) else -1
                positions[to] = t
            if wants[b] is not None:
                self.lens[b] = ends[b]
        return [min(s, max_tokens) for s in starts], slots, positions

    def fork(self, src, dst):
        lens, width, batch = self._lens(), len(self.table[0]), len(self.table)
        seen, todo = set(), []
        for a, b in zip(src, dst):
            if a >= batch or not 0 <= b < batch or b in seen:
                self.bad = True
                continue
            seen.add(b)
            if a != b:
                n = lens[a] if a >= 0 else 0
                row = [self.table[a][j] if j < self._count(n) and self._ok(self.table[a][j]) else -1 for j in range(width)]
                todo.append((b, n, row))
        for _, _, row in todo:
            for pg in row:
                if pg >= 0:
                    self.refs[pg] += 1
        for b, _, _ in todo:
            for j in range(self._count(lens[b])):
                self._drop(self.table[b][j])
        free = [p for p, r in enumerate(self.refs) if r == 0]
        parts = []
        for b, n, row in todo:
            at = n // self.page
            if n % self.page and row[at] >= 0:
                parts.append(row[at])
                if free:
                    new = free.pop(0)
                    self._copy(row[at], new, n % self.page)
                    self.refs[new], row[at] = 1, new
                else:
                    self.bad = True
                    n, row[at] = at * self.page, -1
            self.table[b], self.lens[b] = row, n
        for pg in parts:
            self._drop(pg)

    def compact(self):
        """(new_ids, live)"""
        lens = self._lens()
        live = sum(r > 0 for r in self.refs)
        ids = [p if r > 0 else -1 for p, r in enumerate(self.refs)]
        holes = [p for p in range(live) if self.refs[p] <= 0]
        far = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        for a, b in zip(far, holes):
            ids[a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
            self._copy(a, b, self.page)
        for row, n in zip(self.table, lens):
            for j in range(self._count(n)):
                if self._ok(row[j]):
                    row[j] = ids[row[j]]
        return ids, live
