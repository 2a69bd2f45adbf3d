"""Rows around a paged cache, and attention over it (oracle).

The pages describe caches that are encoded whole; the paged cache, the per-head norm and
the position rotation have no counterpart there.  Definitions:

  * norm: y = x / sqrt(mean x^2 + eps) * (w + offset);
  * rotation by a table row (cos, sin) of the token's position: (a, b) -> (a c - b s,
    b c + a s) for the pairs (j, j + dim/2) or (2j, 2j + 1) of the first ``dim`` elements;
  * a slot is page * page_size + offset; plane rows are [page, KV head, offset];
  * the attention of a sequence is ``attention.multi_query_decode`` over the rows that
    its page table names, query i of n_q seeing positions < len - n_q + i + 1 if causal.

Float64 throughout, and the norm and rotation once more in the library's float32 order
(squares, folds of each 8 neighbours, folds of their sums by halves, no contraction),
whose rounding to fp16 is what the encoders read.
"""

from __future__ import annotations

import numpy as np

from . import attention, q8_0, turboquant


def _pairs(dim: int, interleaved: bool):
    """Indexes of the first and second members of the rotated pairs."""
    j = np.arange(dim // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + dim // 2)


def norm_rope(x, w=None, offset=0.0, eps=1e-6, norm=False, cs=None, interleaved=False):
    """Rows ``x[tokens, heads, D]`` normed and rotated, float64.  ``cs[tokens, dim]``:
    the tokens' table rows (None: no rotation)."""
    y = np.asarray(x, dtype=np.float64).copy()
    if norm:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps)
        if w is not None:
            y = y * (np.asarray(w, dtype=np.float64) + offset)
    if cs is not None:
        dim = cs.shape[-1]
        ia, ib = _pairs(dim, interleaved)
        c, s = (np.asarray(cs, dtype=np.float64)[:, None, i * dim // 2:(i + 1) * dim // 2] for i in (0, 1))
        a, b = y[..., ia].copy(), y[..., ib].copy()
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def norm_rope_f32(x, w=None, offset=0.0, eps=1e-6, norm=False, cs=None, interleaved=False):
    """The same in the library's float32 order (every operation rounded)."""
    f = np.float32
    y = np.asarray(x).astype(f)
    d = y.shape[-1]
    if norm:
        t = (y * y).reshape(y.shape[:-1] + (d // 8, 8))
        for h in (4, 2, 1):
            t = t[..., :h] + t[..., h:2 * h]
        t = t[..., 0]
        while t.shape[-1] > 1:
            h = t.shape[-1] // 2
            t = t[..., :h] + t[..., h:]
        inv = f(1) / np.sqrt(t * f(1.0 / d) + f(eps))
        y = y * inv
        if w is not None:
            y = y * (np.asarray(w).astype(f) + f(offset))
    if cs is not None:
        dim = cs.shape[-1]
        ia, ib = _pairs(dim, interleaved)
        c, s = (np.asarray(cs).astype(f)[:, None, i * dim // 2:(i + 1) * dim // 2] for i in (0, 1))
        a, b = y[..., ia].copy(), y[..., ib].copy()
        y = y.copy()
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    assert y.dtype == f
    return y


def append(planes, new, slots, page: int):
    """Planes with the encoded rows ``new`` (tuple of [tokens, hkv, ...]) at their slots;
    negative slots are skipped."""
    out = [np.array(p) for p in planes]
    for t, slot in enumerate(np.asarray(slots).tolist()):
        if slot < 0:
            continue
        for p, r in zip(out, new):
            p[slot // page, :, slot % page] = r[t]
    return out


def values(fmt: str, planes, d: int, signs=None):
    """What stored rows decode to, float64 [..., D]."""
    if fmt == "f16":
        return np.asarray(planes[0]).astype(np.float64)
    if fmt == "q8_0":
        return q8_0.decode(np.asarray(planes[0]), np.asarray(planes[1]))
    bits = int(fmt[2])
    return turboquant.decode_tier([np.asarray(p) for p in planes[:-1]], np.asarray(planes[-1]), signs, d, bits)


def decode(q, k_fmt, k_planes, v_fmt, v_planes, table, lens, scale, softcap=0.0, causal=False, signs=None):
    """Attention of ``q[batch, n_q, hq, D]`` over the pages ``table[batch, width]`` of
    sequences of ``lens`` positions: (O [batch, n_q, hq, D], lse [batch, n_q, hq])."""
    q = np.asarray(q, dtype=np.float64)
    batch, n_q, hq, d = q.shape
    page = k_planes[0].shape[2]
    o, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
    for b in range(batch):
        n = int(lens[b])
        if n == 0:
            continue
        at = np.asarray(table)[b, :-(-n // page)]
        rows = []
        for fmt, planes in ((k_fmt, k_planes), (v_fmt, v_planes)):
            own = [np.asarray(p)[at] for p in planes]  # [pages, hkv, page, ...]
            own = [np.moveaxis(p, 2, 1).reshape((-1, p.shape[1]) + p.shape[3:])[:n] for p in own]
            rows.append(values(fmt, own, d, signs))
        o[b], lse[b] = attention.multi_query_decode(q[b], rows[0], rows[1], scale, softcap,
                                                    q_pos=n - n_q if causal else None)
    return o, lse
