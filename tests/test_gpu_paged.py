"""The calls around a paged cache on the GPU against the float64 oracle: norm and
rotation of query / key rows, append (bit for bit), ragged and shared-prefix attention,
and the three of them together in a captured decode step."""

import numpy as np
import pytest
import torch

import synth
from oracle import paged as op
from oracle import pipeline
from oracle import turboquant as otq
from tests.helpers import assert_parity

pytestmark = pytest.mark.gpu

EPS = 1e-6
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half a step, relative
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}  # half a subnormal step


@pytest.fixture(scope="module")
def qps():
    import quantized_position_split_gb300 as q
    from quantized_position_split_gb300 import build
    build.build()
    q.device_status(reset=True)
    yield q
    q.device_status(reset=True)  # no wait gave up and no index was out of range


def _projection(tokens, hq, hkv, d, dtype, seed, wide=0):
    """Query, key and value rows as slices of one projection's output."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((tokens, hq + 2 * hkv + wide, d), generator=g)
    x[:, hq:hq + hkv, :4] *= 20
    x = x.to(dtype).cuda()
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:hq + 2 * hkv]


def _rope_inputs(tokens, d, dim, far, dtype, seed):
    g = torch.Generator().manual_seed(seed + 1)
    pos = torch.randint(0, far, (tokens,), generator=g)
    pos[0] = far - 1
    pos[-1] = 0 if tokens > 1 else far - 1
    w = [(0.3 + torch.randn(d, generator=g)).to(dtype).cuda() for _ in range(2)]
    return pos.cuda(), w


def _f(t):
    return t.detach().float().cpu().numpy()


def _check_rows(got, x, w, offset, norm, cs, inter, out_dtype):
    """Against float64, and bit for bit against the float32 order.  Tolerance: half a step
    of the output type at the value, plus the float32 chain before it: the sum of squares
    (log2(D) + 1 roundings, halved by the root), its mean, root and inverse, the product
    with inv, the weight's sum and product: at most 16 roundings of 2^-24 on each member
    of a pair; then two products and a sum."""
    ref = op.norm_rope(x, w, offset, EPS, norm, cs, inter)
    size = np.abs(op.norm_rope(x, w, offset, EPS, norm, None))
    both = size.copy()
    if cs is not None:
        ia, ib = op._pairs(cs.shape[-1], inter)
        both[..., ia] = both[..., ib] = size[..., ia] + size[..., ib]
    tol = HALF[out_dtype] * np.abs(ref) + 20 * 2.0 ** -24 * both + TINY[out_dtype]
    assert (np.abs(_f(got) - ref) <= tol).all()
    f32 = torch.from_numpy(op.norm_rope_f32(x, w, offset, EPS, norm, cs, inter)).to(out_dtype)
    assert torch.equal(got.cpu(), f32)


@pytest.mark.parametrize("d", [32, 64, 128, 256, 512])
@pytest.mark.parametrize("tokens,hq,hkv", [(1, 8, 2), (1, 1, 1), (7, 5, 1), (613, 10, 3)])
@pytest.mark.parametrize("inter,part", [(False, 1), (True, 1), (False, 2), (True, 2)])
def test_norm_rope(qps, d, tokens, hq, hkv, inter, part):
    for i, (dtype, out) in enumerate([(torch.float16, torch.float16), (torch.bfloat16, torch.float16),
                                      (torch.float32, torch.bfloat16)]):
        dim = d // part
        q, k, _ = _projection(tokens, hq, hkv, d, dtype, d + tokens + i)
        pos, (wq, wk) = _rope_inputs(tokens, d, dim, 9000, dtype, d + i)
        rope = qps.Rope(qps.rope_table(9000, dim), inter)
        offset = float(i == 1)
        a = qps.qk_rope_args(q, k, positions=pos, rope=rope, q_norm=wq, k_norm=wk, eps=EPS, norm_offset=offset,
                             out_dtype=out)
        qo, ko = qps.qk_norm_rope(a)
        cs = _f(rope.table)[pos.cpu().numpy()]
        _check_rows(qo, _f(q), _f(wq), offset, True, cs, inter, out)
        _check_rows(ko, _f(k), _f(wk), offset, True, cs, inter, out)


def test_norm_rope_variants(qps):
    """Norm without weights, no norm, no rotation, one side normed, queries alone, weights
    of another type, a width that is not a power of two, in place, bf16 out of bf16."""
    d, tokens = 128, 37
    q, k, _ = _projection(tokens, 6, 2, d, torch.bfloat16, 5)
    pos, (wq, wk) = _rope_inputs(tokens, d, d, 500, torch.float32, 5)
    rope = qps.Rope(qps.rope_table(500, 48))
    cs = _f(rope.table)[pos.cpu().numpy()]
    qo, ko = qps.qk_norm_rope(qps.qk_rope_args(q, k, positions=pos, rope=rope, norm=True))
    _check_rows(qo, _f(q), None, 0, True, cs, False, torch.float16)
    _check_rows(ko, _f(k), None, 0, True, cs, False, torch.float16)
    qo, ko = qps.qk_norm_rope(qps.qk_rope_args(q, k, positions=pos, rope=rope, norm=False, q_norm=wq))
    _check_rows(qo, _f(q), None, 0, False, cs, False, torch.float16)
    qo, ko = qps.qk_norm_rope(qps.qk_rope_args(q, k, q_norm=wq))
    _check_rows(qo, _f(q), _f(wq), 0, True, None, False, torch.float16)
    _check_rows(ko, _f(k), None, 0, False, None, False, torch.float16)
    qo, none = qps.qk_norm_rope(qps.qk_rope_args(q, positions=pos, rope=rope, q_norm=wq))
    assert none is None
    _check_rows(qo, _f(q), _f(wq), 0, True, cs, False, torch.float16)
    x, y = _f(q), _f(k)
    qps.qk_norm_rope(qps.qk_rope_args(q, k, positions=pos, rope=rope, q_norm=wq, k_norm=wk, out_dtype=torch.bfloat16,
                                      q_out=q, k_out=k))
    _check_rows(q, x, _f(wq), 0, True, cs, False, torch.bfloat16)
    _check_rows(k, y, _f(wk), 0, True, cs, False, torch.bfloat16)


def test_norm_rope_special_rows(qps):
    """A zero row (eps alone under the root), rows of infinities and NaN beside others, and
    values whose rotated result leaves fp16's range."""
    d = 64
    x = torch.randn((5, 2, d), generator=torch.Generator().manual_seed(2)).half()
    x[1] = 0
    x[2, 0, 3] = float("inf")
    x[3, 1, 9] = float("nan")
    x[4] = 60000.0
    pos = torch.arange(5)
    rope = qps.Rope(qps.rope_table(8, d))
    (o, _) = qps.qk_norm_rope(qps.qk_rope_args(x.cuda(), positions=pos.cuda(), rope=rope))
    with np.errstate(all="ignore"):
        want = torch.from_numpy(op.norm_rope_f32(x.float().numpy(), cs=_f(rope.table)[:5])).half()
    assert torch.equal(torch.nan_to_num(o.cpu(), 7.0, 8.0, 9.0), torch.nan_to_num(want, 7.0, 8.0, 9.0))
    assert torch.isinf(o[4]).any() and (o[1] == 0).all()
    o, _ = qps.qk_norm_rope(qps.qk_rope_args(x[1:2].cuda(), norm=True))
    assert (o == 0).all()


def test_norm_rope_position_out_of_range(qps):
    d = 128
    q, _, _ = _projection(6, 4, 1, d, torch.float16, 3)
    rope = qps.Rope(qps.rope_table(100, d))
    pos = torch.tensor([5, 100, -1, 99, 1 << 40, 0]).cuda()
    out = torch.full_like(q, 3.0).contiguous()
    a = qps.qk_rope_args(q, positions=pos, rope=rope, q_out=out)
    qps.qk_norm_rope(a)
    with pytest.raises(qps.QpsError) as e:
        qps.device_status(reset=True)
    assert e.value.status == 1  # INVALID_ARG
    bad = [1, 2, 4]
    assert (out[bad] == 3.0).all()
    good = [0, 3, 5]
    _check_rows(out[good], _f(q[good]), None, 0, False, _f(rope.table)[pos.cpu().numpy()[good]], False, torch.float16)


# ---- append ---------------------------------------------------------------------------
PAIRS = [("f16", "f16"), ("q8_0", "q8_0"), ("q8_0", "tq3"), ("f16", "tq2"), ("q8_0", "tq4"), ("f16", "q8_0"),
         ("tq2", "tq2"), ("tq3", "tq3"), ("tq4", "tq4")]


def _rotations(d, form):
    w1, w2 = synth.sign_bits(d, 42), synth.sign_bits(d, 43)
    if form == "block":
        g = min(d, 64)
        return (w1, w2, g), otq.Rotation(w1.numpy(), w2.numpy(), g)
    return w1, w1.numpy()


def _lib_rot(qps, r):
    return qps.Rotation(*r) if isinstance(r, tuple) else r


def _fill(cache, seed):
    """Arbitrary bytes in every plane (NaN among the fp16 values)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    for p in cache.k_planes + cache.v_planes:
        raw = torch.randint(0, 256, (p.numel() * p.element_size(),), generator=g, device="cuda", dtype=torch.uint8)
        p.view(torch.uint8).view(-1).copy_(raw)


def _bits(p):
    """A plane's bytes (cuda or cpu tensor, or array)."""
    t = p if isinstance(p, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(p))
    return t.cpu().contiguous().view(-1).view(torch.uint8)


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("kf,vf", PAIRS)
def test_append_bit_exact(qps, d, kf, vf):
    for i, (tokens, hkv, page, dtype, form) in enumerate([(1, 1, 16, torch.float16, "whole"),
                                                          (29, 3, 32, torch.bfloat16, "block"),
                                                          (331, 4, 128, torch.float32, "whole")]):
        if hkv * tokens * d > 200000:
            tokens = 97
        seed = d + i
        rot, ora = _rotations(d, form)
        n_pages = tokens // page + 3
        cache = qps.PagedKV.empty(kf, vf, n_pages, page, hkv, d, signs=_lib_rot(qps, rot))
        _fill(cache, seed)
        before = [[p.cpu().numpy() for p in s] for s in (cache.k_planes, cache.v_planes)]
        _, k, v = _projection(tokens, 2, hkv, d, dtype, seed)
        v[0, 0] = 0  # a zero row
        pos, (wk, _) = _rope_inputs(tokens, d, d, 700, dtype, seed)
        g = torch.Generator().manual_seed(seed)
        slots = torch.randperm(n_pages * page, generator=g)[:tokens]
        slots[1:-1:7] = -1 - slots[1:-1:7]  # padding: negative of any size
        rope = qps.Rope(qps.rope_table(700, d), i == 1)
        a = qps.paged_append_args(cache, k, v, slots.cuda(), positions=pos, rope=rope, k_norm=wk, eps=EPS,
                                  norm_offset=float(i == 1))
        qps.kv_append_paged(a)
        k16 = op.norm_rope_f32(_f(k), _f(wk), float(i == 1), EPS, True, _f(rope.table)[pos.cpu().numpy()],
                               i == 1).astype(np.float16)
        v16 = _f(v).astype(np.float16)
        for planes, was, fmt, x in ((cache.k_planes, before[0], kf, k16), (cache.v_planes, before[1], vf, v16)):
            want = op.append(was, pipeline.encode(fmt, x, ora), slots, page)
            for p, w in zip(planes, want):
                assert torch.equal(_bits(p), _bits(w)), (fmt, i)


def test_append_out_of_range_and_no_rotation(qps):
    """Slots behind the cache and positions behind the table leave every plane as it was;
    the others are stored.  Without norm and rotation the rows are encoded as they are."""
    d, page, hkv = 128, 16, 2
    cache = qps.PagedKV.empty("q8_0", "f16", 3, page, hkv, d)
    _fill(cache, 1)
    before = [[p.cpu().numpy() for p in s] for s in (cache.k_planes, cache.v_planes)]
    _, k, v = _projection(5, 1, hkv, d, torch.float16, 9)
    slots = torch.tensor([47, 48, -1, 1 << 40, 3])
    pos = torch.tensor([0, 1, 2, 3, 64])
    rope = qps.Rope(qps.rope_table(64, d))
    qps.kv_append_paged(qps.paged_append_args(cache, k, v, slots.cuda(), positions=pos.cuda(), rope=rope))
    with pytest.raises(qps.QpsError):
        qps.device_status(reset=True)
    k16 = op.norm_rope_f32(_f(k), cs=_f(rope.table)[[0] * 5]).astype(np.float16)
    keep = torch.tensor([47, -1, -1, -1, -1])
    for planes, was, fmt, x in ((cache.k_planes, before[0], "q8_0", k16), (cache.v_planes, before[1], "f16", _f(v).astype(np.float16))):
        for p, w in zip(planes, op.append(was, pipeline.encode(fmt, x), keep, page)):
            assert torch.equal(_bits(p), _bits(w))
    slots = torch.tensor([0, 17, 34, 20, 3]).cuda()
    qps.kv_append_paged(qps.paged_append_args(cache, k, v, slots))
    codes, scales = qps.kv_quant_q8_0(k.contiguous())
    assert torch.equal(cache.k_planes[0][slots // page, :, slots % page], codes)
    assert torch.equal(cache.k_planes[1][slots // page, :, slots % page], scales)
    assert torch.equal(cache.v_planes[0][slots // page, :, slots % page], v)


# ---- attention ------------------------------------------------------------------------
def _cache_of(qps, kf, vf, lens, page, hkv, d, seed, rot=None, common=0):
    """A cache that holds sequences of `lens` positions on scattered pages, everything else
    in it arbitrary bytes, and its table (entries behind a sequence's last page: -7)."""
    g = torch.Generator().manual_seed(seed)
    width = max(1, -(-max(lens) // page)) + 1
    shared = common // page
    need = shared + sum(max(0, -(-n // page) - shared) for n in lens)
    order = torch.randperm(need + 2, generator=g).tolist()
    table = torch.full((len(lens), width), -7, dtype=torch.int32)
    cache = qps.PagedKV.empty(kf, vf, need + 2, page, hkv, d, signs=_lib_rot(qps, rot) if rot is not None else None)
    _fill(cache, seed)
    first = order[:shared]
    del order[:shared]
    for b, n in enumerate(lens):
        own = max(0, -(-n // page) - shared)
        row = first + [order.pop() for _ in range(own)]
        table[b, :len(row)] = torch.tensor(row, dtype=torch.int32)
    slots = []
    for b, n in enumerate(lens):
        for t in range(0 if b == 0 else min(common, n), n):
            slots.append(int(table[b, t // page]) * page + t % page)
    if slots:
        x = torch.randn((len(slots), 2 * hkv, d), generator=g)
        for h in range(hkv):
            x[:, h, torch.randperm(d, generator=g)[:4]] *= 20
        x = x.half().cuda()
        qps.kv_append_paged(qps.paged_append_args(cache, x[:, :hkv], x[:, hkv:], torch.tensor(slots).cuda()))
    return cache, table


def _want(cache, q, table, lens, scale, softcap, causal, ora=None):
    """The oracle over the cache's stored planes (rows no sequence holds are not looked at)."""
    kp, vp = ([p.cpu().numpy() for p in s] for s in (cache.k_planes, cache.v_planes))
    if q.dim() == 3:
        q = q[:, None]
    o, lse = op.decode(q.cpu().numpy(), cache.k_fmt, kp, cache.v_fmt, vp, table.numpy(), lens, scale, softcap, causal, ora)
    return o.reshape(-1, q.shape[-1]), lse.reshape(-1)


def _run(qps, q, cache, table, lens, **kw):
    a = qps.paged_attn_args(q, cache, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), **kw)
    o, lse = qps.attn_decode_paged(a)
    return o.float().cpu().numpy(), lse.cpu().numpy()


RAGGED = [0, 1, 15, 16, 17, 31, 33, 64, 100, 257, 1000]


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("kf,vf", PAIRS)
def test_attention_ragged(qps, d, kf, vf):
    """Every format on small and large pages, lengths of zero, one and around page and tile
    borders, garbage behind each sequence's end."""
    hkv = 2
    for page, group, softcap in ((16, 4, 0.0), (64, 1, 30.0), (256, 5, 0.0)):
        rot, ora = _rotations(d, "block" if page == 64 else "whole")
        lens = RAGGED if page < 256 else [257, 0, 300, 2000]
        cache, table = _cache_of(qps, kf, vf, lens, page, hkv, d, d + page, rot)
        g = torch.Generator().manual_seed(d + group)
        q = torch.randn((len(lens), hkv * group, d), generator=g).half().cuda()
        ro, rl = _want(cache, q, table, lens, d ** -0.5, softcap, False, ora)
        o, lse = _run(qps, q, cache, table, lens, scale=d ** -0.5, softcap=softcap, out_dtype=torch.float32)
        assert_parity(o, lse, ro, rl, (d, kf, vf, page))


@pytest.mark.parametrize("d,kf,vf", [(64, "f16", "f16"), (128, "f16", "f16"), (128, "q8_0", "tq3"), (256, "q8_0", "q8_0"),
                                     (512, "q8_0", "tq3"), (128, "tq4", "tq4")])
@pytest.mark.parametrize("n_q,group", [(1, 1), (2, 5), (5, 4), (17, 2), (64, 5)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_multi_query(qps, d, kf, vf, n_q, group, causal):
    """Verify batches: the causal limit of every query, sequences shorter than the batch of
    queries (rows that see nothing), n-tiles that are not full."""
    hkv, page = 2, 32
    rot, ora = _rotations(d, "whole")
    lens = [n_q, 3, 0, n_q + 70, 513]
    cache, table = _cache_of(qps, kf, vf, lens, page, hkv, d, n_q + group, rot)
    q = torch.randn((len(lens), n_q, hkv * group, d), generator=torch.Generator().manual_seed(n_q)).half().cuda()
    ro, rl = _want(cache, q, table, lens, d ** -0.5, 0.0, causal, ora)
    o, lse = _run(qps, q, cache, table, lens, scale=d ** -0.5, causal=causal, out_dtype=torch.float32)
    assert_parity(o, lse, ro, rl, (d, kf, vf, n_q, group, causal))
    if causal and n_q > 3:
        assert (lse.reshape(len(lens), n_q, -1)[1, :n_q - 3] == -np.inf).all()


@pytest.mark.parametrize("d,kf,vf,page", [(128, "f16", "f16", 16), (64, "f16", "f16", 64), (128, "q8_0", "tq3", 64),
                                          (128, "q8_0", "q8_0", 128), (256, "f16", "q8_0", 32), (512, "q8_0", "tq3", 64)])
@pytest.mark.parametrize("batch,group,n_q", [(2, 1, 1), (15, 4, 1), (9, 4, 3), (40, 8, 1)])
def test_attention_shared_prefix(qps, d, kf, vf, page, batch, group, n_q):
    """A batch behind one prefix (an odd number of pages): the same values as without the
    sharing, sequences that end with the prefix or inside it among them."""
    hkv = 2
    common = 9 * page
    rot, ora = _rotations(d, "whole")
    r = np.random.default_rng(batch)
    lens = [common + int(n) for n in r.integers(1, 130, batch)]
    lens[1] = common
    if batch > 2:
        lens[2] = common - 5
    cache, table = _cache_of(qps, kf, vf, lens, page, hkv, d, batch + d, rot, common)
    q = torch.randn((batch, n_q, hkv * group, d), generator=torch.Generator().manual_seed(d)).half().cuda()
    ro, rl = _want(cache, q, table, lens, d ** -0.5, 0.0, n_q > 1, ora)
    for shared in (common, page, 0):
        o, lse = _run(qps, q, cache, table, lens, scale=d ** -0.5, causal=n_q > 1, shared_len=shared,
                      out_dtype=torch.float32)
        assert_parity(o, lse, ro, rl, (d, kf, vf, batch, group, n_q, shared))


@pytest.mark.parametrize("d,kf,vf,n_q,group", [(512, "q8_0", "tq3", 5, 8), (512, "q8_0", "tq2", 4, 16), (512, "f16", "f16", 5, 4),
                                               (256, "q8_0", "q8_0", 5, 3), (256, "f16", "tq3", 2, 8), (128, "q8_0", "tq3", 9, 4),
                                               (128, "q8_0", "q8_0", 13, 5), (128, "f16", "q8_0", 7, 4), (128, "f16", "f16", 9, 4),
                                               (64, "f16", "f16", 13, 5)])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_attention_many_rows_many_tiles(qps, d, kf, vf, n_q, group, softcap):
    """Chunks of a dozen tiles and more for the kernels that take many query rows: every
    buffer and barrier of their pipelines goes round several times, and maxima that rise
    late (keys that grow along the sequence) rescale what has been summed."""
    hkv, page, batch = 8, 64, 3
    rot, ora = _rotations(d, "whole")
    lens = [7001, 5990, 6400]
    cache, table = _cache_of(qps, kf, vf, lens, page, hkv, d, d + n_q, rot)
    if kf == "f16":  # later positions have larger keys
        for b, n in enumerate(lens):
            for j in range(-(-n // page)):
                cache.k_planes[0][int(table[b, j])] *= 0.5 + 1.5 * j * page / n
    q = torch.randn((batch, n_q, hkv * group, d), generator=torch.Generator().manual_seed(d)).half().cuda()
    ro, rl = _want(cache, q, table, lens, d ** -0.5, softcap, True, ora)
    for _ in range(3):  # (a race does not show every time)
        o, lse = _run(qps, q, cache, table, lens, scale=d ** -0.5, softcap=softcap, causal=True, out_dtype=torch.float32)
        assert_parity(o, lse, ro, rl, (d, kf, vf, n_q, group))


@pytest.mark.parametrize("d,kf,vf", [(128, "f16", "f16"), (64, "f16", "f16"), (128, "q8_0", "tq3"), (512, "q8_0", "tq3")])
def test_attention_long_prefix(qps, d, kf, vf):
    """A shared prefix of many tiles per CTA, more rows than one CTA holds."""
    hkv, page, batch, group, common = 8, 64, 40, 5, 8192
    rot, ora = _rotations(d, "whole")
    lens = [common + 1 + 3 * b for b in range(batch)]
    cache, table = _cache_of(qps, kf, vf, lens, page, hkv, d, d, rot, common)
    q = torch.randn((batch, hkv * group, d), generator=torch.Generator().manual_seed(d)).half().cuda()
    pick = [0, 1, 17, 39]
    ro, rl = _want(cache, q[pick], table[pick], [lens[b] for b in pick], d ** -0.5, 0.0, False, ora)
    for _ in range(3):
        o, lse = _run(qps, q, cache, table, lens, scale=d ** -0.5, shared_len=common, out_dtype=torch.float32)
        o, lse = o.reshape(batch, -1, d)[pick].reshape(-1, d), lse.reshape(batch, -1)[pick].reshape(-1)
        assert_parity(o, lse, ro, rl, (d, kf, vf))


def test_attention_long_and_output_types(qps):
    """One long sequence beside short ones; the fp16 and bf16 outputs are the float32 one,
    rounded once; a table with a row stride and query rows with a batch stride."""
    d, hkv, page = 128, 2, 64
    lens = [20011, 5, 300]
    cache, table = _cache_of(qps, "q8_0", "q8_0", lens, page, hkv, d, 3)
    wide = torch.full((3, table.shape[1] + 5), 1 << 30, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    big = torch.randn((3, 20, d), generator=torch.Generator().manual_seed(1)).half().cuda()
    q = big[:, :10]
    ro, rl = _want(cache, q, table, lens, d ** -0.5, 0.0, False)
    dev_table = wide.cuda()[:, :table.shape[1]]
    lens_t = torch.tensor(lens, dtype=torch.int32).cuda()
    got = {}
    for dt in (torch.float32, torch.float16, torch.bfloat16):
        o, lse = qps.attn_decode_paged(qps.paged_attn_args(q, cache, dev_table, lens_t, scale=d ** -0.5, out_dtype=dt))
        got[dt] = o
        assert_parity(lse.cpu().numpy()[:, None], lse.cpu().numpy(), lse.cpu().numpy()[:, None].astype(np.float64), rl)
    assert_parity(got[torch.float32].cpu().numpy(), lse.cpu().numpy(), ro, rl)
    for dt in (torch.float16, torch.bfloat16):
        assert torch.equal(got[dt], got[torch.float32].to(dt))


MANY = [(64, "f16", "f16", 9, 2), (128, "f16", "f16", 3, 4), (128, "q8_0", "tq3", 9, 4), (256, "q8_0", "q8_0", 5, 3),
        (256, "f16", "f16", 5, 3), (512, "q8_0", "tq2", 3, 8)]


@pytest.mark.parametrize("d,kf,vf,n_q,group", MANY)
def test_attention_many_rows_bad_pages(qps, d, kf, vf, n_q, group):
    """As test_attention_bad_indexes, for the kernels that take many query rows."""
    hkv, page = 2, 32
    lens = [300, 170, 200]
    rot, ora = _rotations(d, "whole")
    cache, table = _cache_of(qps, kf, vf, lens, page, hkv, d, 8, rot)
    q = torch.randn((3, n_q, hkv * group, d), generator=torch.Generator().manual_seed(4)).half().cuda()
    ro, rl = _want(cache, q, table, lens, d ** -0.5, 0.0, True, ora)
    rows = n_q * hkv * group
    keep = np.r_[0:rows, 2 * rows:3 * rows]
    for bad in (cache.n_pages, 1 << 30, -1):
        t = table.clone()
        t[1, 4] = bad
        o, lse = _run(qps, q, cache, t, lens, scale=d ** -0.5, causal=True, out_dtype=torch.float32)
        with pytest.raises(qps.QpsError) as e:
            qps.device_status(reset=True)
        assert e.value.status == 1
        assert_parity(o[keep], lse[keep], ro[keep], rl[keep], bad)
        assert np.isfinite(o).all()


@pytest.mark.parametrize("d,kf,vf,n_q,group", MANY)
def test_attention_many_rows_nan_and_output_types(qps, d, kf, vf, n_q, group):
    """A NaN value or key reaches its own sequence's rows alone; a NaN or infinity behind a
    sequence's end reaches none; fp16 and bf16 outputs are the float32 one rounded once."""
    hkv, page = 2, 64
    lens = [140, 200, 150, 129]
    rot, ora = _rotations(d, "whole")
    cache, table = _cache_of(qps, kf, vf, lens, page, hkv, d, 12, rot)
    q = torch.randn((4, n_q, hkv * group, d), generator=torch.Generator().manual_seed(5)).half().cuda()
    ro, rl = _want(cache, q, table, lens, d ** -0.5, 0.0, False, ora)
    nan = float("nan")
    v_float = cache.v_planes[-1] if vf != "f16" else cache.v_planes[0]
    k_float = cache.k_planes[-1] if kf != "f16" else cache.k_planes[0]
    for t, x in ((v_float, nan), (k_float, float("inf"))):  # behind the ends, in the last pages
        for b, n in enumerate(lens):
            t[int(table[b, n // page]), :, n % page:] = x
    o, lse = _run(qps, q, cache, table, lens, scale=d ** -0.5, out_dtype=torch.float32)
    assert_parity(o, lse, ro, rl, (d, kf, vf))
    for dt in (torch.float16, torch.bfloat16):
        a = qps.paged_attn_args(q, cache, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), scale=d ** -0.5,
                                out_dtype=dt)
        assert torch.equal(qps.attn_decode_paged(a)[0].cpu(), torch.from_numpy(o).to(dt))
    v_float[int(table[0, 1]), :, 7] = nan
    k_float[int(table[2, 0]), :, 9] = nan
    o, lse = _run(qps, q, cache, table, lens, scale=d ** -0.5, out_dtype=torch.float32)
    rows = n_q * hkv * group
    assert np.isnan(o[:rows]).all() and np.isnan(o[2 * rows:3 * rows]).all()
    keep = np.r_[rows:2 * rows, 3 * rows:4 * rows]
    assert_parity(o[keep], lse[keep], ro[keep], rl[keep], (d, kf, vf))


@pytest.mark.parametrize("d,kf,vf,n_q,group", [(128, "f16", "f16", 1, 1), (128, "q8_0", "q8_0", 2, 4), (64, "f16", "f16", 5, 4),
                                               (128, "q8_0", "tq3", 7, 4)])
def test_attention_large_batch(qps, d, kf, vf, n_q, group):
    """More sequences than the lanes' first round of lengths holds, behind a prefix and
    without, empty and short ones among them, on two streams at once."""
    hkv, page, batch = 2, 16, 300
    r = np.random.default_rng(d)
    common = 2 * page
    lens = [common + int(n) for n in r.integers(0, 90, batch)]
    lens[5], lens[140], lens[299] = 0, 3, common
    rot, ora = _rotations(d, "whole")
    cache, table = _cache_of(qps, kf, vf, lens, page, hkv, d, 3, rot, common)
    q = torch.randn((batch, n_q, hkv * group, d), generator=torch.Generator().manual_seed(6)).half().cuda()
    ro, rl = _want(cache, q, table, lens, d ** -0.5, 0.0, n_q > 1, ora)
    lt, tt = torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda()
    blocks = [qps.paged_attn_args(q, cache, tt, lt, scale=d ** -0.5, causal=n_q > 1, shared_len=sh, out_dtype=torch.float32)
              for sh in (0, common)]
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    for _ in range(5):
        for st, a in zip(streams, blocks):
            qps.attn_decode_paged(a, stream=st)
    torch.cuda.synchronize()
    for a in blocks:
        o, lse = a._out
        assert_parity(o.cpu().numpy(), lse.cpu().numpy(), ro, rl, (d, kf, vf))


def test_attention_bad_indexes(qps):
    """A table entry out of range and a length behind the table are reported and change no
    other sequence's result."""
    d, hkv, page = 128, 2, 32
    lens = [100, 70, 200]
    cache, table = _cache_of(qps, "f16", "f16", lens, page, hkv, d, 8)
    q = torch.randn((3, 4, d), generator=torch.Generator().manual_seed(4)).half().cuda()
    ro, rl = _want(cache, q, table, lens, 0.1, 0.0, False)
    for bad in (cache.n_pages, 1 << 30, -1):
        t = table.clone()
        t[1, 1] = bad
        o, lse = _run(qps, q, cache, t, lens, scale=0.1, out_dtype=torch.float32)
        with pytest.raises(qps.QpsError) as e:
            qps.device_status(reset=True)
        assert e.value.status == 1
        keep = np.r_[0:4, 8:12]
        assert_parity(o[keep], lse[keep], ro[keep], rl[keep], bad)
        assert np.isfinite(o).all()
    width = table.shape[1] * page
    for n in (width + 1, -3):
        _, _ = _run(qps, q[:1], cache, table[:1].clamp(min=0), [n], scale=0.1)
        with pytest.raises(qps.QpsError):
            qps.device_status(reset=True)


def test_attention_nan_and_lowest_values(qps):
    """A NaN inside a sequence reaches that sequence's rows alone; keys of fp16's lowest
    value and logits that differ by thousands keep the softmax finite."""
    d, hkv, page = 64, 1, 16
    lens = [40, 40, 40]
    cache, table = _cache_of(qps, "f16", "f16", lens, page, hkv, d, 11)
    cache.v_planes[0][int(table[0, 1]), 0, 3, 5] = float("nan")
    cache.k_planes[0][int(table[1, 0]), 0, 2] = -65504.0
    cache.k_planes[0][int(table[2, 0]), 0, 0] = 2000.0
    q = torch.ones((3, 2, d), dtype=torch.float16).cuda()
    ro, rl = _want(cache, q, table, lens, d ** -0.5, 0.0, False)
    o, lse = _run(qps, q, cache, table, lens, scale=d ** -0.5, out_dtype=torch.float32)
    assert np.isnan(o[:2, 5]).all()
    o[:2, 5] = ro[:2, 5] = 0
    assert_parity(o[:, :], np.zeros(6), ro, np.zeros(6))
    assert (np.abs(lse - rl) <= 2.0 ** -22 * np.abs(rl) + 1e-5).all()


# ---- together -------------------------------------------------------------------------
@pytest.mark.parametrize("kf,vf,n_q", [("f16", "f16", 1), ("q8_0", "tq3", 1), ("q8_0", "q8_0", 3)])
def test_decode_loop_captured(qps, kf, vf, n_q):
    """Steps of a serving loop (norm + rotation, append, attention) captured once on a side
    stream and replayed while sequences grow across page borders, one of them a padding
    row, against the oracle over an fp16 copy of the history."""
    d, hq, hkv, page, batch, start = 128, 8, 2, 16, 3, [14, 40, 0]
    rot, ora = _rotations(d, "whole")
    steps, far = 5, 256
    cache = qps.PagedKV.empty(kf, vf, 16, page, hkv, d, signs=_lib_rot(qps, rot))
    _fill(cache, 5)
    table = torch.randperm(16, generator=torch.Generator().manual_seed(6))[:12].view(3, 4).int()
    g = torch.Generator().manual_seed(7)
    rope = qps.Rope(qps.rope_table(far, d))
    wq, wk = (torch.randn(d, generator=g).cuda() for _ in range(2))
    rows = batch * n_q
    x = torch.zeros((rows, hq + 2 * hkv, d), dtype=torch.bfloat16, device="cuda")
    pos, slots = (torch.zeros(rows, dtype=torch.int64, device="cuda") for _ in range(2))
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    dtable = table.cuda()
    a = qps.qk_rope_args(x[:, :hq], positions=pos, rope=rope, q_norm=wq)
    b = qps.paged_append_args(cache, x[:, hq:hq + hkv], x[:, hq + hkv:], slots, positions=pos, rope=rope, k_norm=wk)
    c = qps.paged_attn_args(a._out[0].view(batch, n_q, hq, d), cache, dtable, lens, scale=d ** -0.5, causal=True,
                            out_dtype=torch.float32)

    def step():
        qps.qk_norm_rope(a)
        qps.kv_append_paged(b)
        qps.attn_decode_paged(c)

    history = [(np.zeros((0, hkv, d), np.float16), np.zeros((0, hkv, d), np.float16)) for _ in range(batch)]

    def feed(counts, q_rows):
        """Rows for `counts[b]` positions of each sequence (padding where it has none)."""
        xs = torch.randn((rows, hq + 2 * hkv, d), generator=g).bfloat16()
        p, s = torch.zeros(rows, dtype=torch.int64), torch.full((rows,), -1)
        for i in range(batch):
            have = history[i][0].shape[0]
            for j in range(counts[i]):
                at = have + j
                p[i * n_q + j] = at
                s[i * n_q + j] = int(table[i, at // page]) * page + at % page
        x.copy_(xs)
        pos.copy_(p)
        slots.copy_(s)
        cs = _f(rope.table)[p.numpy()]
        k16 = op.norm_rope_f32(xs[:, hq:hq + hkv].float().numpy(), _f(wk), 0, EPS, True, cs).astype(np.float16)
        v16 = xs[:, hq + hkv:].float().numpy().astype(np.float16)
        for i in range(batch):
            sl = slice(i * n_q, i * n_q + counts[i])
            history[i] = tuple(np.concatenate((h, r[sl])) for h, r in zip(history[i], (k16, v16)))
        lens.copy_(torch.tensor([h[0].shape[0] for h in history], dtype=torch.int32))
        return op.norm_rope_f32(xs[:, :hq].float().numpy(), _f(wq), 0, EPS, True, cs).astype(np.float16)

    while any(history[i][0].shape[0] < start[i] for i in range(batch)):  # the prompts, eagerly
        feed([min(n_q, start[i] - history[i][0].shape[0]) for i in range(batch)], None)
        qps.kv_append_paged(b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(steps):
        q16 = feed([n_q, n_q, 0], None)
        graph.replay()
        torch.cuda.synchronize()
        o, lse = c._out
        want = [], []
        for i in range(batch):
            n = history[i][0].shape[0]
            qi = q16[i * n_q:(i + 1) * n_q]
            if n == 0:
                want[0].append(np.zeros((n_q, hq, d)))
                want[1].append(np.full((n_q, hq), -np.inf))
                continue
            kd, vd = (pipeline.dequant(f, r, ora) for f, r in ((kf, history[i][0]), (vf, history[i][1])))
            from oracle import attention
            oi, li = attention.multi_query_decode(qi, kd, vd, d ** -0.5, 0.0, q_pos=n - n_q)
            want[0].append(oi)
            want[1].append(li)
        ro, rl = np.concatenate(want[0]).reshape(-1, d), np.concatenate(want[1]).reshape(-1)
        assert_parity(o.cpu().numpy(), lse.cpu().numpy(), ro, rl)
        eager = [t.clone() for t in (o, lse)]
        step()  # the same step again, eagerly: the same rows into the same slots, the same result
        torch.cuda.synchronize()
        assert torch.equal(o, eager[0]) and torch.equal(lse, eager[1])


def test_two_streams_and_empty_calls(qps):
    """Blocks of their own run on two streams at once; calls without tokens do nothing."""
    d, hkv, page = 128, 2, 64
    lens = [700, 90]
    cache, table = _cache_of(qps, "f16", "f16", lens, page, hkv, d, 21)
    lt, tt = torch.tensor(lens, dtype=torch.int32).cuda(), table.cuda()
    streams = [torch.cuda.Stream() for _ in range(2)]
    qs = [torch.randn((2, 8, d), generator=torch.Generator().manual_seed(i)).half().cuda() for i in range(2)]
    blocks = [qps.paged_attn_args(q, cache, tt, lt, scale=0.09, out_dtype=torch.float32) for q in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, a in zip(streams, blocks):
            qps.attn_decode_paged(a, stream=s)
    torch.cuda.synchronize()
    for q, a in zip(qs, blocks):
        ro, rl = _want(cache, q, table, lens, 0.09, 0.0, False)
        assert_parity(a._out[0].cpu().numpy(), a._out[1].cpu().numpy(), ro, rl)
    none = torch.zeros((0, 4, d), dtype=torch.float16, device="cuda")
    qo, _ = qps.qk_norm_rope(qps.qk_rope_args(none))
    assert qo.shape == none.shape
    before = cache.k_planes[0].clone()
    qps.kv_append_paged(qps.paged_append_args(cache, none[:, :hkv], none[:, :hkv], torch.zeros(0, dtype=torch.int64, device="cuda")))
    assert torch.equal(_bits(before), _bits(cache.k_planes[0]))
