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
