"""Calls around a paged cache at the edges of what their documentation allows, on the GPU
against the float64 oracle: what lies behind every sequence's end, padding rows, the
extremes of the stored formats, large pages, first calls under capture."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import paged as op
from tests.helpers import assert_parity
from tests.test_gpu_paged import _cache_of, _f, _lib_rot, _rotations, _run, _want, qps  # noqa: F401

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# one KV head's rows of a whole batch go to attn_mma.cuh (few rows), attn_tm.cuh (many, fp16
# pages of head_dim 64 / 128) or attn_tt.cuh (many, other pages)
PREFIXES = [(128, "f16", "f16", 2, 1), (512, "q8_0", "q8_0", 2, 1), (128, "q8_0", "tq3", 3, 2), (64, "tq2", "tq2", 5, 4),
            (128, "f16", "f16", 5, 4), (64, "f16", "f16", 7, 5),
            (128, "q8_0", "tq3", 9, 4), (256, "f16", "f16", 5, 4), (256, "f16", "q8_0", 5, 4), (512, "q8_0", "tq2", 5, 4)]


def _value_plane(cache):
    """The fp16 plane of V (values, scales or norms)."""
    return cache.v_planes[0] if cache.v_fmt == "f16" else cache.v_planes[-1]


def _key_plane(cache):
    return cache.k_planes[0] if cache.k_fmt == "f16" else cache.k_planes[-1]


@pytest.mark.parametrize("d,kf,vf,batch,group", PREFIXES)
def test_prefix_behind_every_end(qps, d, kf, vf, batch, group):  # noqa: F811
    """Every sequence ends inside the shared pages: NaN values and infinite keys behind the
    longest end, in its last page and in whole chunks, reach no row."""
    hkv, page, common = 2, 64, 64 * 64
    rot, ora = _rotations(d, "whole")
    cache, table = _cache_of(qps, kf, vf, [common] * batch, page, hkv, d, 3 * d, rot, common)
    q = torch.randn((batch, hkv * group, d), generator=torch.Generator().manual_seed(d)).half().cuda()
    for longest in (common - 37, 1203, 37):
        lens = [longest - 3 * (batch - 1 - b) for b in range(batch)]
        lens[0] = 0 if batch > 2 else lens[0]
        ro, rl = _want(cache, q, table, lens, d ** -0.5, 0.0, False, ora)
        k_was, v_was = _key_plane(cache).clone(), _value_plane(cache).clone()
        for plane, x in ((_value_plane(cache), float("nan")), (_key_plane(cache), float("inf"))):
            plane[int(table[0, longest // page]), :, longest % page:] = x
            for j in range(longest // page + 1, common // page):
                plane[int(table[0, j])] = x
        o, lse = _run(qps, q, cache, table, lens, scale=d ** -0.5, shared_len=common, out_dtype=torch.float32)
        assert_parity(o, lse, ro, rl, (d, kf, vf, batch, group, longest))
        _key_plane(cache).copy_(k_was)
        _value_plane(cache).copy_(v_was)


@pytest.mark.parametrize("d,kf,vf,batch,group", PREFIXES)
def test_prefix_behind_a_padding_row(qps, d, kf, vf, batch, group):  # noqa: F811
    """The first row of a padded batch (length zero, or a sequence that ends inside the
    shared pages) names other pages behind its end: the prefix is the others' all the same."""
    hkv, page, common = 2, 32, 16 * 32
    rot, ora = _rotations(d, "whole")
    for first in (0, 70):
        lens = [common + 1 + 9 * b for b in range(batch)]
        cache, table = _cache_of(qps, kf, vf, lens, page, hkv, d, 5 * d, rot, common)
        q = torch.randn((batch, hkv * group, d), generator=torch.Generator().manual_seed(d)).half().cuda()
        lens[0] = first
        ro, rl = _want(cache, q, table, lens, d ** -0.5, 0.0, False, ora)
        own = int(table[1, common // page])  # a page that holds other rows
        for behind in (own, -7):
            t = table.clone()
            t[0, -(-first // page):] = behind
            o, lse = _run(qps, q, cache, t, lens, scale=d ** -0.5, shared_len=common, out_dtype=torch.float32)
            assert_parity(o, lse, ro, rl, (d, kf, vf, batch, group, first, behind))
            qps.device_status(reset=True)


# (n_q, group) on both sides of the rows at which the kernel changes
SIDES = [(128, "q8_0", "f16", 4, 4), (128, "q8_0", "f16", 6, 4), (128, "q8_0", "f16", 5, 5), (128, "q8_0", "tq3", 5, 5),
         (256, "q8_0", "tq3", 2, 4), (256, "q8_0", "f16", 3, 3), (512, "q8_0", "q8_0", 2, 4), (512, "q8_0", "q8_0", 3, 3),
         (512, "q8_0", "tq2", 13, 4)]


@pytest.mark.parametrize("d,kf,vf,n_q,group", SIDES)
@pytest.mark.parametrize("softcap", [0.0, 25.0])
def test_q8_keys_at_the_end_of_the_range(qps, d, kf, vf, n_q, group, softcap):  # noqa: F811
    """q8_0 keys that hold fp16's largest value (the encoder stores scale 516, code 127:
    65532), scales up to fp16's largest and down to its smallest, in rows beside ordinary
    ones, against queries small enough for ordinary logits."""
    hkv, page, n = 2, 64, 700
    rot, ora = _rotations(d, "whole")
    cache, table = _cache_of(qps, kf, vf, [n], page, hkv, d, 7 * d, rot)
    g = torch.Generator().manual_seed(d)
    x = torch.randn((n, hkv, d), generator=g)
    x[5::9, :, ::37] = 65504.0
    x[6::9, 0, 3::41] = -65504.0
    x[7::9] *= 2.0 ** -14
    slots = torch.tensor([int(table[0, t // page]) * page + t % page for t in range(n)]).cuda()
    v = torch.randn((n, hkv, d), generator=g).half().cuda()
    qps.kv_append_paged(qps.paged_append_args(cache, x.half().cuda(), v, slots))
    at = [(int(table[0, t // page]), t % page) for t in range(n)]
    assert float(cache.k_planes[1][at[5][0], 0, at[5][1]].max()) == 516
    for t in range(8, n, 9):  # scales that no encoder of fp16 rows makes, of the largest value's kind
        cache.k_planes[1][at[t][0], :, at[t][1], ::2] = 65504.0 if t % 2 else 2.0 ** -24
    q = torch.randn((1, n_q, hkv * group, d), generator=g)
    q = (q * 2.0 ** -17).half().cuda()  # (subnormal: multiples of 2^-24)
    scale = 40.0 / d ** 0.5
    ro, rl = _want(cache, q, table, [n], scale, softcap, True, ora)
    o, lse = _run(qps, q, cache, table, [n], scale=scale, softcap=softcap, causal=True, out_dtype=torch.float32)
    # float32 logits of size up to |rl|: 2^-24 a step, D terms of a product
    size = float(np.abs(rl).max())
    assert np.isfinite(o).all() and (np.abs(lse - rl) <= d * 2.0 ** -24 * size + 1e-5).all()
    assert_parity(o, np.zeros(rl.shape), ro, np.zeros(rl.shape), (d, kf, vf, n_q, group))


@pytest.mark.parametrize("d,kf,vf,n_q,group", [(64, "f16", "q8_0", 1, 4), (128, "q8_0", "q8_0", 1, 1), (128, "q8_0", "q8_0", 7, 4),
                                               (256, "f16", "q8_0", 1, 4), (256, "q8_0", "q8_0", 5, 4), (512, "q8_0", "q8_0", 1, 8),
                                               (512, "f16", "q8_0", 5, 4)])
def test_q8_values_at_the_end_of_the_range(qps, d, kf, vf, n_q, group):  # noqa: F811
    """q8_0 values that hold fp16's largest value (65532 as stored): finite weights of them
    are finite, and a weight of zero leaves nothing of them."""
    hkv, page, n = 2, 64, 500
    cache, table = _cache_of(qps, kf, vf, [n], page, hkv, d, 9 * d)
    g = torch.Generator().manual_seed(d)
    k = torch.randn((n, hkv, d), generator=g)
    x = torch.randn((n, hkv, d), generator=g) * 20000
    x[3::5, :, ::7] = 65504.0
    x[4::5, :, 1::9] = -65504.0
    k[8::10] *= 40  # (a few keys far above and below the others: weights that underflow)
    slots = torch.tensor([int(table[0, t // page]) * page + t % page for t in range(n)]).cuda()
    qps.kv_append_paged(qps.paged_append_args(cache, k.half().cuda(), x.clamp(-65504, 65504).half().cuda(), slots))
    q = torch.randn((1, n_q, hkv * group, d), generator=g).half().cuda()
    ro, rl = _want(cache, q, table, [n], d ** -0.5, 0.0, False)
    o, lse = _run(qps, q, cache, table, [n], scale=d ** -0.5, out_dtype=torch.float32)
    # a value is off by at most 2^-10 (its block's scale cut to 515.5 of 516) + 2^-11 (its
    # rounding), both relative to the largest value, 65532; P keeps its second part
    assert (np.abs(o - ro) <= (2.0 ** -10 + 2.0 ** -11 + 2.0 ** -17) * 65532).all()
    assert (np.abs(lse - rl) <= 1e-4 + 2.0 ** -20 * np.abs(rl)).all()


@pytest.mark.parametrize("d,kf,vf,n_q,group", [(64, "tq2", "tq2", 1, 4), (128, "q8_0", "tq3", 1, 4), (128, "f16", "tq4", 3, 4),
                                               (128, "q8_0", "tq3", 9, 4), (256, "f16", "tq2", 4, 4), (512, "q8_0", "tq3", 1, 8),
                                               (512, "q8_0", "tq3", 5, 4)])
@pytest.mark.parametrize("size", [2.0 ** -16, 1.0, 2.0 ** 9])
def test_turboquant_values_of_any_size(qps, d, kf, vf, n_q, group, size):  # noqa: F811
    """TurboQuant values far below and far above one, and both in one sequence, keep the
    accuracy of ordinary ones: P times a small norm does not fall below fp16's normal range."""
    hkv, page, n = 2, 64, 3001
    rot, ora = _rotations(d, "whole")
    cache, table = _cache_of(qps, kf, vf, [n, 64], page, hkv, d, 9 * d, rot)
    g = torch.Generator().manual_seed(d)
    k, v = (torch.randn((n, hkv, d), generator=g) for _ in range(2))
    v *= size
    v[100] = 0  # a zero row, and the largest key with it: the reference is not its alone
    k[100] *= 3
    slots = torch.tensor([int(table[0, t // page]) * page + t % page for t in range(n)]).cuda()
    qps.kv_append_paged(qps.paged_append_args(cache, k.half().cuda(), v.half().cuda(), slots))
    q = (torch.randn((2, n_q, hkv * group, d), generator=g) * 1.5).half().cuda()
    if size == 1.0:  # large norms late in the sequence
        _value_plane(cache)[int(table[0, 40])] = 900.0
        _value_plane(cache)[int(table[0, 3])] = 2.0 ** -12
    ro, rl = _want(cache, q, table, [n, 0], d ** -0.5, 0.0, False, ora)
    o, lse = _run(qps, q, cache, table, [n, 0], scale=d ** -0.5, out_dtype=torch.float32)
    assert_parity(o / max(size, 1.0), lse, ro / max(size, 1.0), rl, (d, kf, vf, n_q, group, size))


@pytest.mark.parametrize("d,kf,vf,n_q,group", [(128, "f16", "f16", 1, 4), (512, "q8_0", "q8_0", 1, 8), (128, "q8_0", "tq3", 5, 4),
                                               (64, "f16", "f16", 5, 4), (128, "f16", "f16", 9, 4), (128, "q8_0", "tq3", 9, 4),
                                               (256, "f16", "f16", 5, 4), (512, "f16", "q8_0", 5, 4)])
@pytest.mark.parametrize("above", [9.0, 12.0, 16.0])
def test_one_key_above_all_others(qps, d, kf, vf, n_q, group, above):  # noqa: F811
    """A first position whose logit is far above all others and whose value is zero: the output
    is what the others' small weights make of their values."""
    hkv, page, n = 2, 64, 4001
    rot, ora = _rotations(d, "whole")
    cache, table = _cache_of(qps, kf, vf, [n], page, hkv, d, d, rot)
    g = torch.Generator().manual_seed(d)
    k, v = torch.randn((n, hkv, d), generator=g) * 0.3, 1 + torch.randn((n, hkv, d), generator=g)
    q = 1 + 0.1 * torch.randn((1, n_q, hkv * group, d), generator=g)
    k -= k.mean(-1, keepdim=True)
    k[0] = (above + 1.0) / d ** 0.5
    v[0] = 0
    slots = torch.tensor([int(table[0, t // page]) * page + t % page for t in range(n)]).cuda()
    qps.kv_append_paged(qps.paged_append_args(cache, k.half().cuda(), v.half().cuda(), slots))
    q = q.half().cuda()
    ro, rl = _want(cache, q, table, [n], d ** -0.5, 0.0, False, ora)
    o, lse = _run(qps, q, cache, table, [n], scale=d ** -0.5, out_dtype=torch.float32)
    assert_parity(o, lse, ro, rl, (d, kf, vf, n_q, group, above))


@pytest.mark.parametrize("page", [128, 256, 512, 1024])
@pytest.mark.parametrize("d,kf,vf,n_q,group", [(64, "f16", "f16", 5, 4), (128, "f16", "f16", 9, 4), (128, "q8_0", "tq3", 9, 4),
                                               (256, "f16", "q8_0", 3, 4), (512, "q8_0", "tq2", 5, 4), (128, "q8_0", "q8_0", 1, 4)])
def test_large_pages(qps, page, d, kf, vf, n_q, group):  # noqa: F811
    """Pages as large as a tile and larger: every offset in a page, prefix and own positions."""
    hkv, common = 2, 2 * page
    rot, ora = _rotations(d, "whole")
    lens = [common + 5 * page // 2 + 3, common + page, common + page + 1, common - 30]
    cache, table = _cache_of(qps, kf, vf, lens, page, hkv, d, page + d, rot, common)
    q = torch.randn((len(lens), n_q, hkv * group, d), generator=torch.Generator().manual_seed(d)).half().cuda()
    ro, rl = _want(cache, q, table, lens, d ** -0.5, 0.0, True, ora)
    for shared in (0, common):
        o, lse = _run(qps, q, cache, table, lens, scale=d ** -0.5, causal=True, shared_len=shared, out_dtype=torch.float32)
        assert_parity(o, lse, ro, rl, (d, kf, vf, n_q, group, page, shared))


def _child(code):
    res = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert res.returncode == 0 and "child ok" in res.stdout, (res.stdout + res.stderr)[-3000:]


def test_first_call_captured_on_a_blocking_stream(qps):  # noqa: F811
    """The first call of a process may be captured, also on a stream that synchronises with
    the legacy default stream."""
    _child("""
import ctypes, torch
import quantized_position_split_gb300 as qps
rt = ctypes.CDLL("libcudart.so.13")
x = torch.randn(4, 2, 128, device="cuda").half()
a = qps.qk_rope_args(x, norm=True)
torch.cuda.synchronize()
s = ctypes.c_void_p()
assert rt.cudaStreamCreate(ctypes.byref(s)) == 0  # (a blocking stream)
g, e = ctypes.c_void_p(), ctypes.c_void_p()
assert rt.cudaStreamBeginCapture(s, 0) == 0  # global mode
qps.qk_norm_rope(a, stream=s.value)
assert rt.cudaStreamEndCapture(s, ctypes.byref(g)) == 0
assert rt.cudaGraphInstantiate(ctypes.byref(e), g, ctypes.c_ulonglong(0)) == 0
assert rt.cudaGraphLaunch(e, s) == 0 and rt.cudaStreamSynchronize(s) == 0
o = a._out[0].float()
w = x.float() / (x.float().square().mean(-1, keepdim=True) + 1e-6).sqrt()
assert (o - w).abs().max() < 4e-3, (o - w).abs().max()
qps.device_status(reset=True)
print("child ok")
""")


def test_a_thread_first_call_beside_a_capture(qps):  # noqa: F811
    """A thread whose first CUDA call is the library's, on a stream of its own, while another
    thread captures in the global mode: neither disturbs the other."""
    _child("""
import threading, torch
import quantized_position_split_gb300 as qps
x = torch.randn(4, 2, 128, device="cuda").half()
w = (x.float() / (x.float().square().mean(-1, keepdim=True) + 1e-6).sqrt()).cpu()
a, b = (qps.qk_rope_args(x, norm=True) for _ in range(2))
side, other = torch.cuda.Stream(), torch.cuda.Stream()
qps.qk_norm_rope(a)
torch.cuda.synchronize()
a._out[0].zero_()
torch.cuda.synchronize()
raw, errors = other.cuda_stream, []
def call():
    try:
        qps.qk_norm_rope(b, stream=raw)
    except Exception as e:
        errors.append(e)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g, stream=side, capture_error_mode="global"):
    qps.qk_norm_rope(a)
    t = threading.Thread(target=call)
    t.start()
    t.join()
assert not errors, errors
g.replay()
torch.cuda.synchronize()
for blk in (a, b):
    assert (blk._out[0].float().cpu() - w).abs().max() < 4e-3
print("child ok")
""")


def test_attention_in_a_second_context(qps):  # noqa: F811
    """A second context of a device that has run the same kernels: they are set up there too, and
    what they report goes to a word of that context."""
    _child("""
import ctypes, torch
import quantized_position_split_gb300 as qps
from quantized_position_split_gb300 import _native as N
d, hkv, page = 128, 2, 64
cache = qps.PagedKV.empty("f16", "f16", 8, page, hkv, d)
q = torch.ones(2, 8, d, device="cuda").half()
table = torch.arange(8, device="cuda", dtype=torch.int32).view(2, 4)
lens = torch.tensor([200, 90], device="cuda", dtype=torch.int32)
many = torch.ones(2, 9, 8, d, device="cuda").half()
blocks = [qps.paged_attn_args(q, cache, table, lens, scale=0.1), qps.paged_attn_args(many, cache, table, lens, scale=0.1)]
for a in blocks:
    qps.attn_decode_paged(a)
torch.cuda.synchronize()
cu = ctypes.CDLL("libcuda.so.1")
dev, ctx = ctypes.c_int(), ctypes.c_void_p()
assert cu.cuDeviceGet(ctypes.byref(dev), 0) == 0
assert cu.cuCtxCreate_v2(ctypes.byref(ctx), 0, dev) == 0  # (current in this thread)
def put(n, value=None):
    p = ctypes.c_uint64()
    assert cu.cuMemAlloc_v2(ctypes.byref(p), ctypes.c_size_t(n)) == 0
    if value is None:
        assert cu.cuMemsetD8_v2(p, 0, ctypes.c_size_t(n)) == 0
    else:
        assert cu.cuMemcpyHtoD_v2(p, value, ctypes.c_size_t(n)) == 0
    return p.value
import numpy as np
for a in blocks:
    b = N.PagedAttnArgs()
    ctypes.memmove(ctypes.byref(b), ctypes.byref(a), ctypes.sizeof(b))
    rows = b.batch * b.n_q * b.hq
    b.q = put(rows * d * 2, np.ones(rows * d, np.float16).ctypes.data_as(ctypes.c_void_p))
    b.kv.k_data = put(8 * hkv * page * d * 2)
    b.kv.v_data = put(8 * hkv * page * d * 2, np.ones(8 * hkv * page * d, np.float16).ctypes.data_as(ctypes.c_void_p))
    b.page_table = put(32, np.arange(8, dtype=np.int32).ctypes.data_as(ctypes.c_void_p))
    b.kv_lens = put(8, np.array([200, 90], np.int32).ctypes.data_as(ctypes.c_void_p))
    b.o, b.lse, b.workspace = put(rows * d * 2), put(rows * 4), put(b.workspace_bytes)
    N.check(N.load().qps_attn_decode_paged(ctypes.byref(b), None))
    assert cu.cuCtxSynchronize() == 0
    o = np.empty(rows * d, np.float16)
    assert cu.cuMemcpyDtoH_v2(o.ctypes.data_as(ctypes.c_void_p), ctypes.c_uint64(b.o), ctypes.c_size_t(o.nbytes)) == 0
    assert (o == 1).all()
    b.page_table = put(32, np.full(8, 99, np.int32).ctypes.data_as(ctypes.c_void_p))
    N.check(N.load().qps_attn_decode_paged(ctypes.byref(b), None))  # pages out of range: reported here
    assert N.load().qps_device_status(1) == N.QPS_ERR_INVALID_ARG
    assert N.load().qps_device_status(1) == N.QPS_OK
assert cu.cuCtxPopCurrent_v2(ctypes.byref(ctx)) == 0
torch.cuda.synchronize()
qps.device_status()  # the first context's word is its own
assert float(cache.k_planes[0].abs().max()) == 0
print("child ok")
""")


def test_in_place_over_interleaved_heads(qps):  # noqa: F811
    """Query and key rows that alternate in one projection, normed in place: no row of one
    is a row of the other."""
    d, tokens, heads = 64, 11, 6
    x = torch.randn((tokens, heads, 3, d), generator=torch.Generator().manual_seed(3)).half().cuda()
    was = x.clone()
    q, k = x[:, :, 0], x[:, :, 1]
    qps.qk_norm_rope(qps.qk_rope_args(q, k, norm=True, q_out=q, k_out=k))
    for i in (0, 1):
        want = torch.from_numpy(op.norm_rope_f32(_f(was[:, :, i]), norm=True)).half()
        assert torch.equal(x[:, :, i].cpu(), want)
    assert torch.equal(x[:, :, 2], was[:, :, 2])


def test_prefix_of_nearly_all_positions(qps):  # noqa: F811
    """A shared prefix close to 2^31 positions (its table names few pages over and over): the
    last chunk's end stays in range."""
    d, hkv, page, batch, group = 64, 1, 1024, 3, 8
    width = (1 << 21) - 2
    n = width * page
    cache = qps.PagedKV.empty("f16", "f16", 2, page, hkv, d)
    cache.v_planes[0][1] = 1.0
    table = torch.zeros((1, width), dtype=torch.int32)
    table[0, -(width // 8):] = 1
    q = torch.zeros((batch, group, d), dtype=torch.float16).cuda()
    o, lse = _run(qps, q, cache, table.expand(batch, width).contiguous(), [n] * batch, scale=1.0,
                  shared_len=(width - 1) * page, out_dtype=torch.float32)
    assert np.abs(lse - np.log(float(n))).max() <= 1e-4
    assert np.abs(o - (width // 8) / width).max() <= 1e-4


@pytest.mark.parametrize("d,kf,vf,n_q,group", [(128, "f16", "f16", 9, 4), (64, "f16", "f16", 9, 4), (128, "q8_0", "tq3", 9, 4),
                                               (256, "f16", "f16", 5, 4), (512, "q8_0", "q8_0", 5, 4)])
@pytest.mark.parametrize("tile", [0, 1, 7])
def test_a_tile_that_never_comes(qps, d, kf, vf, n_q, group, tile):  # noqa: F811
    """A tile withheld on the host: the kernel's waits give up after their limit, its roles
    stop, the call ends, the error word and the record say where, and the next call is right."""
    from quantized_position_split_gb300 import _native as N
    hkv, page, n = 1, 64, 150000
    rot, ora = _rotations(d, "whole")
    cache = qps.PagedKV.empty(kf, vf, -(-n // page), page, hkv, d, signs=_lib_rot(qps, rot))
    table = torch.arange(-(-n // page), dtype=torch.int32)[None]
    q = torch.randn((1, n_q, hkv * group, d), generator=torch.Generator().manual_seed(1)).half().cuda()
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    a = qps.paged_attn_args(q, cache, table.cuda(), lens, scale=d ** -0.5, out_dtype=torch.float32)
    qps.attn_decode_paged(a)
    torch.cuda.synchronize()
    qps.device_status(reset=True)
    qps.paged_inject_fault(tile, 20)
    qps.attn_decode_paged(a)
    torch.cuda.synchronize()
    rec = qps.device_wait_record()
    with pytest.raises(N.QpsError) as e:
        qps.device_status(reset=True)
    assert e.value.status == N.QPS_ERR_TIMEOUT
    assert rec[0] == 1 and rec[1] >= 1 and rec[8] > 0 and rec[9] > 0, rec
    assert 15e6 < rec[10] < 200e6 and rec[11] == 0, rec  # the tile's own drain ran its limit too
    lens.fill_(300)
    o, lse = qps.attn_decode_paged(a)
    torch.cuda.synchronize()
    qps.device_status(reset=True)
    ro, rl = _want(cache, q, table, [300], d ** -0.5, 0.0, False, ora)
    assert_parity(o.cpu().numpy(), lse.cpu().numpy(), ro, rl)


def test_fault_arguments(qps):  # noqa: F811
    for tile, ms in ((-2, 20), (0, 0), (0, 1001), (1 << 30, 5)):
        with pytest.raises(qps.QpsError):
            qps.paged_inject_fault(tile, ms)
    qps.paged_inject_fault(3, 5)
    qps.paged_inject_fault(-1)  # disarmed


def test_outputs_lie_apart(qps):  # noqa: F811
    """Outputs over the queries, or over one another, are refused."""
    d, hkv, page, batch, hq = 128, 2, 64, 2, 4
    cache, table = _cache_of(qps, "f16", "f16", [70, 90], page, hkv, d, 3)
    raw = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    q = raw[4096:4096 + batch * hq * d * 2].view(torch.float16).view(batch, hq, d)
    lens, rows = torch.tensor([70, 90], dtype=torch.int32).cuda(), batch * hq
    o = lambda at: raw[at:at + rows * d * 2].view(torch.float16).view(rows, d)  # noqa: E731
    lse = lambda at: raw[at:at + rows * 4].view(torch.float32)  # noqa: E731
    ws = raw[1 << 16:]
    for kw, ok in ((dict(o=o(4096)), False), (dict(o=o(4096 + 16)), False), (dict(o=o(4096 + rows * d * 2), lse=lse(0)), True),
                   (dict(o=o(8192), lse=lse(8192 + rows * d * 2 - 4)), False), (dict(lse=lse(4096)), False),
                   (dict(workspace=ws, o=o(1 << 16)), False), (dict(workspace=ws, lse=lse((1 << 16) + 256)), False),
                   (dict(workspace=ws, o=o(8192), lse=lse(0)), True), (dict(workspace=raw[4096:]), False)):
        a = qps.paged_attn_args(q, cache, table.cuda(), lens, scale=0.1, **kw)
        if "workspace" in kw:
            a.workspace_bytes = min(a.workspace_bytes, 1 << 19)
        if ok:
            qps.attn_decode_paged(a)
            continue
        with pytest.raises(qps.QpsError) as e:
            qps.attn_decode_paged(a)
        assert e.value.status == 1, kw
    torch.cuda.synchronize()


@pytest.mark.parametrize("d,kf,vf,n_q,group,pages", [(512, "f16", "f16", 1, 4, 700), (512, "f16", "q8_0", 5, 4, 700),
                                                     (512, "q8_0", "tq3", 5, 4, 1400), (128, "f16", "f16", 9, 4, 2500),
                                                     (128, "q8_0", "q8_0", 1, 4, 5000), (64, "f16", "f16", 5, 4, 5000)])
def test_cache_past_32_bits(qps, d, kf, vf, n_q, group, pages):  # noqa: F811
    """Pages whose first byte, and for the largest planes first element, is past 2^32: appended
    to and attended at both ends of the cache."""
    hkv, page, n = 8, 1024, 1500
    rot, ora = _rotations(d, "whole")
    cache = qps.PagedKV.empty(kf, vf, pages, page, hkv, d, signs=_lib_rot(qps, rot))
    assert cache.k_planes[0].numel() * cache.k_planes[0].element_size() > 1 << 32
    table = torch.tensor([[pages - 1, 0], [1, pages - 2]], dtype=torch.int32)
    g = torch.Generator().manual_seed(d)
    x = torch.randn((2, n, 2 * hkv, d), generator=g).half().cuda()
    for b in range(2):
        at = torch.arange(n)
        slots = table[b].long()[at // page] * page + at % page
        qps.kv_append_paged(qps.paged_append_args(cache, x[b, :, :hkv], x[b, :, hkv:], slots.cuda()))
    q = torch.randn((2, n_q, hkv * group, d), generator=g).half().cuda()
    o, lse = _run(qps, q, cache, table, [n, n], scale=d ** -0.5, causal=True, out_dtype=torch.float32)
    used = [pages - 1, 0, 1, pages - 2]  # (the oracle reads these four alone)
    small = qps.PagedKV(kf, vf, [p[used].contiguous() for p in cache.k_planes], [p[used].contiguous() for p in cache.v_planes],
                        signs=_lib_rot(qps, rot))
    del cache
    ro, rl = _want(small, q, torch.tensor([[0, 1], [2, 3]], dtype=torch.int32), [n, n], d ** -0.5, 0.0, True, ora)
    assert_parity(o, lse, ro, rl, (d, kf, vf))

