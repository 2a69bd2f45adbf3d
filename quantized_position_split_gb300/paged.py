"""Serving calls around a paged KV cache: ``qk_norm_rope``, ``kv_append_paged``,
``attn_decode_paged`` and ``attn_prompt_paged`` of ``include/qps.h``, and those on its pages,
``kv_extend_paged``, ``kv_fork_paged`` and ``kv_compact_paged``, as argument blocks and calls.

Like ``attn_args`` / ``attn_decode_window``, each call takes an argument block that a
decode loop builds once for a layer and keeps: the block holds the addresses of its
tensors (and keeps them alive), so a step writes new rows, positions, slots, lengths or
page tables into the same tensors and calls again, eagerly or in a captured graph.
Calls on one block must not overlap on the GPU.
"""

from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional

import torch

from . import _native as N
from ._native import QpsError

_DTYPES = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}


def _bad(msg: str) -> QpsError:
    return QpsError(N.QPS_ERR_INVALID_ARG, msg)


def _tensor(t, what: str, device=None, dtype=None, shape=None, contiguous=True):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise _bad(f"{what} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise _bad(f"{what} is on {t.device}, the other tensors are on {device}")
    if dtype is not None and t.dtype != dtype:
        raise _bad(f"{what} must be {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise _bad(f"{what} must have shape {tuple(shape)}")
    if contiguous and not t.is_contiguous():
        raise _bad(f"{what} must be contiguous")
    return t


@dataclasses.dataclass(frozen=True)
class Rope:
    """A position rotation: ``table`` [positions, dim] f32 (CUDA), a row holding dim / 2
    cosines and then dim / 2 sines; ``interleaved`` rotates the pairs (2j, 2j + 1)
    instead of (j, j + dim / 2)."""

    table: torch.Tensor
    interleaved: bool = False


def rope_table(positions: int, dim: int, base: float = 10000.0, scale: float = 1.0, device="cuda") -> torch.Tensor:
    """The table of ``Rope`` for the angles p * scale * base^(-2j / dim), computed in 64
    bits (a 32-bit angle of a far position has lost its fraction)."""
    f = torch.arange(dim // 2, dtype=torch.float64, device=device) * (-2.0 / dim)
    a = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * (scale * base ** f)
    return torch.cat((a.cos(), a.sin()), 1).float()


def _rows(t: torch.Tensor, what: str, device=None) -> N.Rows:
    _tensor(t, what, device, contiguous=False)
    if t.dim() != 3 or t.dtype not in _DTYPES:
        raise _bad(f"{what} must be [tokens, heads, D] of float16, bfloat16 or float32")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise _bad(f"{what}: the last dimension must be contiguous")
    return N.Rows(t.data_ptr(), _DTYPES[t.dtype], t.shape[1], t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2],
                  t.stride(1) if t.shape[1] > 1 else t.shape[2])


def _norm(on: bool, w, d: int, eps: float, offset: float, what: str, device) -> N.HeadNorm:
    if w is not None:
        _tensor(w, what, device, shape=(d,))
        if w.dtype not in _DTYPES:
            raise _bad(f"{what} must be float16, bfloat16 or float32")
    return N.HeadNorm(None if w is None else w.data_ptr(), 0 if w is None else _DTYPES[w.dtype],
                      1 if on else 0, eps, offset)


def _rotation(rope: Optional[Rope], positions, tokens: int, device) -> tuple:
    if rope is None:
        return N.RotationArgs(), None
    t = _tensor(rope.table, "rope.table", device, torch.float32)
    if t.dim() != 2:
        raise _bad("rope.table must be [positions, dim]")
    if positions is None:
        raise _bad("positions are needed with a rotation")
    _tensor(positions, "positions", device, torch.int64, (tokens,))
    return N.RotationArgs(t.data_ptr(), t.shape[0], t.shape[1], 1 if rope.interleaved else 0), positions.data_ptr()


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(a, stream):
    """Run a block's call on its device, on ``stream`` (default: that device's current
    stream)."""
    if a._index != torch.cuda.current_device():
        with torch.cuda.device(a._index):
            return _call(a, stream)
    if stream is None:
        stream = _raw_stream(a._index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    st = a._fn(ctypes.byref(a), stream)
    if st:
        N.check(st)


def _block(a, fn, device, keep):
    a._fn = getattr(N.load(), fn)
    a._index = device.index
    a._tensors = keep
    return a


def qk_rope_args(q: torch.Tensor, k: Optional[torch.Tensor] = None, *, positions=None, rope: Optional[Rope] = None,
                 q_norm=None, k_norm=None, norm: Optional[bool] = None, eps: float = 1e-6, norm_offset: float = 0.0,
                 out_dtype=None, q_out=None, k_out=None) -> N.QkRopeArgs:
    """Argument block of ``qk_norm_rope`` for ``q[tokens, hq, D]`` and, optionally,
    ``k[tokens, hkv, D]`` (slices of a fused projection are taken as they lie).

    ``q_norm`` / ``k_norm``: the RMS norms' weights [D]; ``norm`` = True norms without
    them, False not at all (default: norm when a weight is given).  ``norm_offset`` is
    added to the weights (1 for weights stored as w - 1).  ``out_dtype``: float16
    (default) or bfloat16.  ``q_out`` / ``k_out`` (allocated if None) may be the inputs.
    """
    if norm is None:
        on_q, on_k = q_norm is not None, k_norm is not None
    else:
        on_q = on_k = bool(norm)
    a = N.QkRopeArgs()
    a.q = _rows(q, "q")
    dev, (tokens, _, d) = q.device, q.shape
    a.tokens, a.d = tokens, d
    if out_dtype is None:
        out_dtype = q_out.dtype if q_out is not None else torch.float16
    if out_dtype not in (torch.float16, torch.bfloat16):
        raise QpsError(N.QPS_ERR_UNSUPPORTED, "qk_rope_args: out_dtype is float16 or bfloat16")
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=out_dtype, device=dev)
    if tuple(q_out.shape) != tuple(q.shape):
        raise _bad("q_out must have q's shape")
    a.q_out = _rows(q_out, "q_out", dev)
    if k is not None:
        a.k = _rows(k, "k", dev)
        if k.shape[0] != tokens or k.shape[2] != d:
            raise _bad("k must have q's tokens and head_dim")
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=out_dtype, device=dev)
        if tuple(k_out.shape) != tuple(k.shape):
            raise _bad("k_out must have k's shape")
        a.k_out = _rows(k_out, "k_out", dev)
    elif k_out is not None:
        raise _bad("k_out without k")
    a.q_norm = _norm(on_q, q_norm if on_q else None, d, eps, norm_offset, "q_norm", dev)
    a.k_norm = _norm(on_k, k_norm if on_k else None, d, eps, norm_offset, "k_norm", dev)
    a.rot, a.positions = _rotation(rope, positions, tokens, dev)
    a._out = (q_out, k_out)
    return _block(a, "qps_qk_norm_rope", dev, (q, k, q_out, k_out, q_norm, k_norm, rope, positions))


def qk_norm_rope(a: N.QkRopeArgs, stream=None):
    """Norm and rotate the rows of ``qk_rope_args``; returns (q_out, k_out)."""
    _call(a, stream)
    return a._out


_PLANES = {"f16": (torch.float16,), "q8_0": (torch.int8, torch.float16), "tq3": (torch.uint8, torch.uint8, torch.float16),
           "tq2": (torch.uint8, torch.float16), "tq4": (torch.uint8, torch.float16)}


def _plane_tail(fmt: str, i: int, d: int) -> tuple:
    """Trailing shape of plane ``i`` after [n_pages, hkv, page_size]."""
    return {"f16": ((d,),), "q8_0": ((d,), (d // 32,)), "tq3": ((d // 4,), (d // 8,), ()),
            "tq2": ((d // 4,), ()), "tq4": ((d // 2,), ())}[fmt][i]


class PagedKV:
    """A paged cache: the planes of K and of V, each ``[n_pages, hkv, page_size, ...]``
    with the trailing shape of its format's encoder (``kv_quant_*``).  ``signs``: the
    TurboQuant rotation (sign words or ``Rotation``) of such planes."""

    def __init__(self, k_fmt: str, v_fmt: str, k_planes, v_planes, signs=None):
        from . import _rotation as as_rotation
        from . import _sign_array
        for fmt in (k_fmt, v_fmt):
            if fmt not in _PLANES:
                raise _bad(f"unknown format {fmt}")
        self.k_fmt, self.v_fmt = k_fmt, v_fmt
        self.k_planes, self.v_planes = tuple(k_planes), tuple(v_planes)
        first = _tensor(self.k_planes[0], "k_planes[0]") if self.k_planes else None
        if first is None or first.dim() != 4:
            raise _bad("k_planes[0] must be [n_pages, hkv, page_size, bytes or values of a row]")
        self.n_pages, self.hkv, self.page_size = first.shape[:3]
        self.d = first.shape[3] * {"f16": 1, "q8_0": 1, "tq3": 4, "tq2": 4, "tq4": 2}[k_fmt]
        self.device = first.device
        kv = N.PagedKvStruct()
        kv.k_fmt, kv.v_fmt = N.FMT_BY_NAME[k_fmt], N.FMT_BY_NAME[v_fmt]
        kv.hkv, kv.d, kv.page_size, kv.n_pages = self.hkv, self.d, self.page_size, self.n_pages
        for side, fmt, planes in (("k", k_fmt, self.k_planes), ("v", v_fmt, self.v_planes)):
            if len(planes) != len(_PLANES[fmt]):
                raise _bad(f"{side}_planes: {fmt} has {len(_PLANES[fmt])} planes")
            for i, (p, dt, field) in enumerate(zip(planes, _PLANES[fmt], ("data", "aux", "aux2"))):
                _tensor(p, f"{side}_planes[{i}]", self.device, dt,
                        (self.n_pages, self.hkv, self.page_size) + _plane_tail(fmt, i, self.d))
                setattr(kv, f"{side}_{field}", p.data_ptr())
        if v_fmt in ("tq2", "tq3", "tq4") or k_fmt in ("tq2", "tq3", "tq4"):
            if signs is None:
                raise _bad("TurboQuant formats need the sign words")
            rot = as_rotation(signs)
            self._signs = [_sign_array(rot.signs1)] + ([_sign_array(rot.signs2)] if rot.signs2 is not None else [])
            if any(len(s) != self.d // 32 for s in self._signs):
                raise _bad("signs must have D / 32 words")
            kv.signs1 = ctypes.cast(self._signs[0], ctypes.POINTER(ctypes.c_uint32))
            if len(self._signs) > 1:
                kv.signs2 = ctypes.cast(self._signs[1], ctypes.POINTER(ctypes.c_uint32))
            kv.tq_block = int(rot.block)
        self.struct = kv

    @classmethod
    def empty(cls, k_fmt: str, v_fmt: str, n_pages: int, page_size: int, hkv: int, d: int, signs=None, device="cuda"):
        """A cache of zeroed pages."""
        planes = []
        for fmt in (k_fmt, v_fmt):
            if fmt not in _PLANES:
                raise _bad(f"unknown format {fmt}")
            planes.append([torch.zeros((n_pages, hkv, page_size) + _plane_tail(fmt, i, d), dtype=dt, device=device)
                           for i, dt in enumerate(_PLANES[fmt])])
        return cls(k_fmt, v_fmt, planes[0], planes[1], signs)


def paged_append_args(cache: PagedKV, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, *, positions=None,
                      rope: Optional[Rope] = None, k_norm=None, norm: Optional[bool] = None, eps: float = 1e-6,
                      norm_offset: float = 0.0) -> N.PagedAppendArgs:
    """Argument block of ``kv_append_paged`` for new rows ``k, v[tokens, hkv, D]`` and
    their ``slots[tokens]`` (int64: page * page_size + offset; negative: padding).  The
    norm and rotation of K are given as in ``qk_rope_args``."""
    dev, tokens = cache.device, k.shape[0]
    a = N.PagedAppendArgs()
    a.kv = cache.struct
    a.tokens = tokens
    a.k, a.v = _rows(k, "k", dev), _rows(v, "v", dev)
    for t, what in ((k, "k"), (v, "v")):
        if tuple(t.shape) != (tokens, cache.hkv, cache.d):
            raise _bad(f"{what} must be [tokens, {cache.hkv}, {cache.d}]")
    on = k_norm is not None if norm is None else bool(norm)
    a.k_norm = _norm(on, k_norm if on else None, cache.d, eps, norm_offset, "k_norm", dev)
    a.rot, a.positions = _rotation(rope, positions, tokens, dev)
    a.slots = _tensor(slots, "slots", dev, torch.int64, (tokens,)).data_ptr()
    return _block(a, "qps_kv_append_paged", dev, (cache, k, v, slots, positions, rope, k_norm))


def kv_append_paged(a: N.PagedAppendArgs, stream=None) -> None:
    """Encode the rows of ``paged_append_args`` into their slots."""
    _call(a, stream)


def paged_attn_args(q: torch.Tensor, cache: PagedKV, page_table: torch.Tensor, kv_lens: torch.Tensor, *, scale: float,
                    softcap: float = 0.0, causal: bool = False, shared_len: int = 0, out_dtype=torch.float16, o=None,
                    lse=None, workspace=None, window: int = 0, sinks: int = 0) -> N.PagedAttnArgs:
    """Argument block of ``attn_decode_paged`` for float16 ``q[batch, hq, D]`` or
    ``q[batch, n_q, hq, D]``, ``page_table[batch, width]`` and ``kv_lens[batch]`` (int32).

    ``causal``: query token i of a sequence sees its positions < len - n_q + i + 1.
    ``shared_len``: positions whose pages are the same in every sequence's table (a
    shared prefix, a multiple of the page size), read once for the batch.  ``window`` > 0: a
    query token sees the ``window`` positions that end with its own, and the first ``sinks``.  ``o``
    [batch*n_q*hq, D] of ``out_dtype``, ``lse`` [batch*n_q*hq] f32 and ``workspace``
    (uint8) are allocated if None.
    """
    if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dtype != torch.float16 or q.dim() not in (3, 4):
        raise _bad("q must be a CUDA float16 tensor [batch, hq, D] or [batch, n_q, hq, D]")
    batch, n_q, hq, d = (q.shape[0], 1) + tuple(q.shape[1:]) if q.dim() == 3 else tuple(q.shape)
    dev = cache.device
    _tensor(q, "q", dev, contiguous=False)
    if d != cache.d:
        raise _bad(f"q must have the cache's head_dim {cache.d}")
    if batch and not q[0].is_contiguous():
        raise _bad("q must be contiguous per batch entry")
    _tensor(page_table, "page_table", dev, torch.int32, contiguous=False)
    if page_table.dim() != 2 or page_table.shape[0] != batch or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise _bad("page_table must be [batch, width] with contiguous rows")
    _tensor(kv_lens, "kv_lens", dev, torch.int32, (batch,))
    if out_dtype not in _DTYPES:
        raise _bad("out_dtype is float16, bfloat16 or float32")
    rows = batch * n_q * hq
    a = N.PagedAttnArgs()
    a.q, a.q_batch_stride = q.data_ptr(), q.stride(0) if batch > 1 else n_q * hq * d
    a.batch, a.n_q, a.hq, a.causal = batch, n_q, hq, 1 if causal else 0
    a.kv = cache.struct
    a.page_table, a.table_width = page_table.data_ptr(), page_table.shape[1]
    a.table_stride = page_table.stride(0) if batch > 1 else page_table.shape[1]
    a.kv_lens = kv_lens.data_ptr()
    a.shared_len, a.scale, a.softcap, a.o_dtype = int(shared_len), scale, softcap, _DTYPES[out_dtype]
    a.window, a.sinks = int(window), int(sinks)
    need = ctypes.c_size_t()
    with torch.cuda.device(dev):
        N.check(N.load().qps_attn_paged_plan(ctypes.byref(a), ctypes.byref(need)))
    if o is None:
        o = torch.empty((rows, d), dtype=out_dtype, device=dev)
    if lse is None:
        lse = torch.empty((rows,), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty((need.value,), dtype=torch.uint8, device=dev)
    _tensor(o, "o", dev, out_dtype, (rows, d))
    _tensor(lse, "lse", dev, torch.float32, (rows,))
    _tensor(workspace, "workspace", dev, torch.uint8)
    a.o, a.lse, a.workspace, a.workspace_bytes = o.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel()
    a._out = (o, lse)
    return _block(a, "qps_attn_decode_paged", dev, (q, cache, page_table, kv_lens, o, lse, workspace))


def attn_decode_paged(a: N.PagedAttnArgs, stream=None):
    """Decode attention of ``paged_attn_args``; returns (o, lse)."""
    _call(a, stream)
    return a._out


def paged_prompt_args(q: torch.Tensor, cache: PagedKV, page_table: torch.Tensor, kv_lens: torch.Tensor,
                      q_starts: torch.Tensor, *, scale: float, softcap: float = 0.0, window: int = 0, sinks: int = 0,
                      out_dtype=torch.float16, o=None, lse=None, workspace=None) -> N.PagedPromptArgs:
    """Argument block of ``attn_prompt_paged`` for the query tokens float16 ``q[tokens, hq, D]``
    of a ragged batch (a slice of a fused projection is taken as it lies): those of sequence b
    are ``[q_starts[b], q_starts[b + 1])`` (int32 ``q_starts[batch + 1]``) and its newest
    positions, whose rows the cache holds already.  ``page_table`` and ``kv_lens`` as in
    ``paged_attn_args``.

    ``window`` > 0: a token sees the ``window`` positions that end with its own, and the first
    ``sinks``.  ``o`` [tokens*hq, D] of ``out_dtype``, ``lse`` [tokens*hq] f32 and ``workspace``
    (uint8) are allocated if None; rows of no sequence stay as they were.
    """
    dev = cache.device
    _tensor(q, "q", dev, torch.float16, contiguous=False)
    if q.dim() != 3 or q.shape[2] != cache.d:
        raise _bad(f"q must be [tokens, hq, {cache.d}]")
    tokens, hq, d = q.shape
    if tokens and not q[0].is_contiguous():
        raise _bad("q must be contiguous per token")
    _tensor(page_table, "page_table", dev, torch.int32, contiguous=False)
    if page_table.dim() != 2 or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise _bad("page_table must be [batch, width] with contiguous rows")
    batch = page_table.shape[0]
    _tensor(kv_lens, "kv_lens", dev, torch.int32, (batch,))
    _tensor(q_starts, "q_starts", dev, torch.int32, (batch + 1,))
    if out_dtype not in _DTYPES:
        raise _bad("out_dtype is float16, bfloat16 or float32")
    a = N.PagedPromptArgs()
    a.q, a.q_tok_stride, a.tokens = q.data_ptr(), q.stride(0) if tokens > 1 else hq * d, tokens
    a.batch, a.hq = batch, hq
    a.q_starts, a.kv = q_starts.data_ptr(), cache.struct
    a.page_table, a.table_width = page_table.data_ptr(), page_table.shape[1]
    a.table_stride = page_table.stride(0) if batch > 1 else page_table.shape[1]
    a.kv_lens = kv_lens.data_ptr()
    a.scale, a.softcap, a.window, a.sinks, a.o_dtype = scale, softcap, int(window), int(sinks), _DTYPES[out_dtype]
    need = ctypes.c_size_t()
    with torch.cuda.device(dev):
        N.check(N.load().qps_attn_prompt_plan(ctypes.byref(a), ctypes.byref(need)))
    if o is None:
        o = torch.empty((tokens * hq, d), dtype=out_dtype, device=dev)
    if lse is None:
        lse = torch.empty((tokens * hq,), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty((need.value,), dtype=torch.uint8, device=dev)
    _tensor(o, "o", dev, out_dtype, (tokens * hq, d))
    _tensor(lse, "lse", dev, torch.float32, (tokens * hq,))
    _tensor(workspace, "workspace", dev, torch.uint8)
    a.o, a.lse, a.workspace, a.workspace_bytes = o.data_ptr(), lse.data_ptr(), workspace.data_ptr(), workspace.numel()
    a._out = (o, lse)
    return _block(a, "qps_attn_prompt_paged", dev, (q, cache, page_table, kv_lens, q_starts, o, lse, workspace))


def attn_prompt_paged(a: N.PagedPromptArgs, stream=None):
    """Attention of ``paged_prompt_args``; returns (o, lse)."""
    _call(a, stream)
    return a._out


class PagedSeqs:
    """The sequences of one or more paged caches (the layers', of one page size and number of
    pages): ``page_table`` [batch, width], ``kv_lens`` [batch] and ``refs`` [n_pages], int32, all
    on the device.  ``refs`` counts the entries that name a page; 0: the page is free."""

    def __init__(self, caches, page_table: torch.Tensor, kv_lens: torch.Tensor, refs: torch.Tensor):
        self.caches = (caches,) if isinstance(caches, PagedKV) else tuple(caches)
        if not self.caches or not all(isinstance(c, PagedKV) for c in self.caches):
            raise _bad("caches must be a PagedKV or a list of them")
        first = self.caches[0]
        self.device, self.n_pages, self.page_size = first.device, first.n_pages, first.page_size
        for c in self.caches:
            if c.device != self.device or c.n_pages != self.n_pages or c.page_size != self.page_size:
                raise _bad("the caches must share a device, a page size and a number of pages")
        _tensor(page_table, "page_table", self.device, torch.int32, contiguous=False)
        if page_table.dim() != 2 or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
            raise _bad("page_table must be [batch, width] with contiguous rows")
        self.batch = page_table.shape[0]
        _tensor(kv_lens, "kv_lens", self.device, torch.int32, (self.batch,))
        _tensor(refs, "refs", self.device, torch.int32, (self.n_pages,))
        self.page_table, self.kv_lens, self.refs = page_table, kv_lens, refs
        self._array = (N.PagedKvStruct * len(self.caches))(*[c.struct for c in self.caches])
        s = N.PagedSeqsStruct()
        s.caches = ctypes.cast(self._array, ctypes.POINTER(N.PagedKvStruct))
        s.n_caches, s.batch = len(self.caches), self.batch
        s.page_table, s.table_width = page_table.data_ptr(), page_table.shape[1]
        s.table_stride = page_table.stride(0) if self.batch > 1 else page_table.shape[1]
        s.kv_lens, s.refs = kv_lens.data_ptr(), refs.data_ptr()
        self.struct = s

    @classmethod
    def empty(cls, caches, batch: int, width: int):
        """Sequences without positions, over pages that are all free."""
        first = caches if isinstance(caches, PagedKV) else caches[0]
        make = lambda shape, x: torch.full(shape, x, dtype=torch.int32, device=first.device)  # noqa: E731
        return cls(caches, make((batch, width), -1), make((batch,), 0), make((first.n_pages,), 0))


def _workspace(a, plan: str, workspace, dev) -> torch.Tensor:
    need = ctypes.c_size_t()
    N.check(getattr(N.load(), plan)(ctypes.byref(a), ctypes.byref(need)))
    if workspace is None:
        workspace = torch.empty((need.value,), dtype=torch.uint8, device=dev)
    _tensor(workspace, "workspace", dev, torch.uint8)
    a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    return workspace


def _out(t, what: str, shape: tuple, dtype, dev) -> torch.Tensor:
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    return _tensor(t, what, dev, dtype, shape)


def paged_extend_args(seqs: PagedSeqs, n_new: torch.Tensor, *, max_tokens: int, window: int = 0, sinks: int = 0, q_starts=None,
                      slots=None, positions=None, workspace=None) -> N.PagedExtendArgs:
    """Argument block of ``kv_extend_paged``: sequence b grows by ``n_new[b]`` (int32) positions,
    or is cut back by so many where that is negative.  ``max_tokens``: rows of ``slots`` and
    ``positions``, at least the new positions of any call.  ``window`` and ``sinks``: those of the
    attention, so that pages that it no longer reads are given back.  ``q_starts`` [batch + 1]
    int32, ``slots`` and ``positions`` [max_tokens] int64 are allocated if None.
    """
    dev = seqs.device
    if max_tokens < 0:
        raise _bad("max_tokens must be >= 0")
    a = N.PagedExtendArgs()
    a.seqs = seqs.struct
    a.n_new = _tensor(n_new, "n_new", dev, torch.int32, (seqs.batch,)).data_ptr()
    a.window, a.sinks, a.max_tokens = int(window), int(sinks), int(max_tokens)
    q_starts = _out(q_starts, "q_starts", (seqs.batch + 1,), torch.int32, dev)
    slots = _out(slots, "slots", (max_tokens,), torch.int64, dev)
    positions = _out(positions, "positions", (max_tokens,), torch.int64, dev)
    a.q_starts, a.slots, a.positions = q_starts.data_ptr(), slots.data_ptr(), positions.data_ptr()
    workspace = _workspace(a, "qps_kv_extend_plan", workspace, dev)
    a._out = (q_starts, slots, positions)
    return _block(a, "qps_kv_extend_paged", dev, (seqs, n_new, q_starts, slots, positions, workspace))


def kv_extend_paged(a: N.PagedExtendArgs, stream=None):
    """Room for the next positions of ``paged_extend_args``; returns (q_starts, slots,
    positions), as ``attn_prompt_paged`` and ``kv_append_paged`` take them."""
    _call(a, stream)
    return a._out


def paged_fork_args(seqs: PagedSeqs, src: torch.Tensor, dst: torch.Tensor, *, workspace=None) -> N.PagedForkArgs:
    """Argument block of ``kv_fork_paged``: sequence ``dst[i]`` becomes a copy of ``src[i]``
    (int32 [n]), or is given back where that is negative."""
    dev = seqs.device
    _tensor(src, "src", dev, torch.int32)
    if src.dim() != 1:
        raise _bad("src must be [n]")
    _tensor(dst, "dst", dev, torch.int32, tuple(src.shape))
    a = N.PagedForkArgs()
    a.seqs, a.n = seqs.struct, src.shape[0]
    a.src, a.dst = src.data_ptr(), dst.data_ptr()
    workspace = _workspace(a, "qps_kv_fork_plan", workspace, dev)
    return _block(a, "qps_kv_fork_paged", dev, (seqs, src, dst, workspace))


def kv_fork_paged(a: N.PagedForkArgs, stream=None) -> None:
    """Fork and give back the sequences of ``paged_fork_args``."""
    _call(a, stream)


def paged_compact_args(seqs: PagedSeqs, *, new_ids=None, live=None, workspace=None) -> N.PagedCompactArgs:
    """Argument block of ``kv_compact_paged``.  ``new_ids`` [n_pages] and ``live`` [1], int32,
    are allocated if None."""
    dev = seqs.device
    a = N.PagedCompactArgs()
    a.seqs = seqs.struct
    new_ids = _out(new_ids, "new_ids", (seqs.n_pages,), torch.int32, dev)
    live = _out(live, "live", (1,), torch.int32, dev)
    a.new_ids, a.live = new_ids.data_ptr(), live.data_ptr()
    workspace = _workspace(a, "qps_kv_compact_plan", workspace, dev)
    a._out = (new_ids, live)
    return _block(a, "qps_kv_compact_paged", dev, (seqs, new_ids, live, workspace))


def kv_compact_paged(a: N.PagedCompactArgs, stream=None):
    """Move the pages in use of ``paged_compact_args`` to the front; returns (new_ids, live):
    what each page has become (-1: it was free), and how many there are."""
    _call(a, stream)
    return a._out


def paged_inject_fault(tile: int, wait_ms: int = 20) -> None:
    """Withhold the keys of tile ``tile`` of each chunk from the next ``attn_decode_paged`` call
    of many query rows, whose waits then give up after ``wait_ms`` (``qps_paged_inject_fault``;
    -1 disarms)."""
    N.check(N.load().qps_paged_inject_fault(tile, wait_ms))
