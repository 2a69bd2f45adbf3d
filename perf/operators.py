"""Cases of the serving operators around a paged KV cache, with their plain forms.

Three entry points are measured:

* ``rope``    query / key rows normalised per head (RMS) and rotated by position in one pass
              (``qk_norm_rope``);
* ``append``  new key / value rows encoded into the pages of a KV cache, the key normalised and
              rotated on the way (``kv_append_paged``);
* ``decode``  decode attention of ragged sequences over such a cache (``attn_decode_paged``), with
              ``shared`` > 0 for a batch whose first ``shared`` positions are one common prefix.

Layouts.  A plane of the cache is ``[pages][hkv][page][row]``; a slot is ``page_index * page +
offset``.  A rotation table row is ``rot / 2`` cosines, then ``rot / 2`` sines (float32).  Stored
formats: ``f16`` values; ``q8_0`` int8 codes and one fp16 scale per 32 values; ``tq3`` a 2-bit
magnitude plane, a 1-bit sign plane and an fp16 norm of the rotated row.
"""

import functools
import math
import random

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
LEVELS = (-2.15234375, -1.34375, -0.755859375, -0.2451171875, 0.2451171875, 0.755859375, 1.34375, 2.15234375)
EPS = 1e-6


def listed():
    return [
        # one new token of one sequence: latency
        dict(name="rope_token", op="rope", tokens=1, hq=40, hkv=8, d=128, rot=128, pairs="half", norm=True,
             offset=0.0, inp="f16", out="f16", far=131072),
        # a verify batch (15 agents x 5 tokens) of head_dim-512 layers: neighbouring pairs, half the
        # row rotated, weights stored as w - 1, bf16 activations into the fp16 query of the attention
        dict(name="rope_verify_bf16", op="rope", tokens=75, hq=16, hkv=2, d=512, rot=256, pairs="next", norm=True,
             offset=1.0, inp="bf16", out="f16", far=262144),
        # a prompt chunk: bandwidth
        dict(name="rope_prompt", op="rope", tokens=8192, hq=40, hkv=8, d=128, rot=128, pairs="half", norm=True,
             offset=0.0, inp="f16", out="f16", far=65536),
        # one new token into an uncompressed cache: latency
        dict(name="append_token", op="append", tokens=1, seqs=1, hkv=8, d=128, page=64, k_fmt="f16", v_fmt="f16",
             rot=128, pairs="half", norm=True, offset=0.0, inp="f16", far=131072, pad=0),
        # a decode batch of agents, a few rows of it padding, into 8-bit keys and 3-bit values
        dict(name="append_agents_tq3", op="append", tokens=61, seqs=61, hkv=8, d=128, page=32, k_fmt="q8_0",
             v_fmt="tq3", rot=128, pairs="half", norm=False, offset=0.0, inp="f16", far=4608, pad=3),
        # a prompt chunk of three sequences into an 8-bit cache, from bf16 activations
        dict(name="append_prompt_q8", op="append", tokens=8191, seqs=3, hkv=8, d=128, page=64, k_fmt="q8_0",
             v_fmt="q8_0", rot=128, pairs="half", norm=True, offset=0.0, inp="bf16", far=65536, pad=0),
        # one short sequence: latency
        dict(name="decode_short", op="decode", batch=1, n_q=1, hq=40, hkv=8, d=128, page=64, k_fmt="f16",
             v_fmt="f16", lo=777, hi=777, empty=False, causal=False, cap=0.0, out="f16", shared=0),
        # a ragged batch on small pages, one padding row without positions
        dict(name="decode_ragged", op="decode", batch=33, n_q=1, hq=32, hkv=8, d=128, page=16, k_fmt="f16",
             v_fmt="f16", lo=1, hi=16384, empty=True, causal=False, cap=0.0, out="bf16", shared=0),
        # one long sequence, 8-bit cache
        dict(name="decode_long_q8", op="decode", batch=1, n_q=1, hq=40, hkv=8, d=128, page=64, k_fmt="q8_0",
             v_fmt="q8_0", lo=131072, hi=131072, empty=False, causal=False, cap=0.0, out="f16", shared=0),
        # verify batch of five tokens with softcap, head_dim 512, 8-bit keys and 3-bit values
        dict(name="decode_verify_tq3", op="decode", batch=4, n_q=5, hq=16, hkv=2, d=512, page=128, k_fmt="q8_0",
             v_fmt="tq3", lo=30000, hi=32768, empty=False, causal=True, cap=50.0, out="f16", shared=0),
        # agents that share a compressed prefix of 4096 positions, each with a short suffix
        dict(name="prefix_agents_tq3", op="decode", batch=15, n_q=1, hq=32, hkv=8, d=128, page=64, k_fmt="q8_0",
             v_fmt="tq3", lo=4097, hi=4608, empty=False, causal=False, cap=0.0, out="f16", shared=4096),
        # a large batch behind one long prompt
        dict(name="prefix_batch", op="decode", batch=64, n_q=1, hq=32, hkv=8, d=128, page=64, k_fmt="f16",
             v_fmt="f16", lo=32769, hi=33280, empty=False, causal=False, cap=0.0, out="f16", shared=32768),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "decode"])
    d = rng.choice([64, 128, 128, 256, 512])
    hkv = rng.choice([1, 2, 4, 8])
    if op == "rope":
        heads = hkv * rng.choice([1, 3, 4, 5, 8])
        tokens = _log(rng, 1, 8192 * 48 * 128 // ((heads + hkv) * d) if (heads + hkv) * d > 6144 else 8192)
        return dict(op=op, tokens=tokens, hq=heads, hkv=hkv, d=d, rot=rng.choice([d, d // 2]),
                    pairs=rng.choice(["half", "next"]), norm=rng.random() < 0.7, offset=rng.choice([0.0, 1.0]),
                    inp=rng.choice(["f16", "bf16", "f32"]), out=rng.choice(["f16", "bf16"]),
                    far=rng.choice([4096, 65536, 131072]))
    if op == "append":
        tokens = _log(rng, 1, min(8192, 8192 * 8 * 128 // (hkv * d)))
        k_fmt, v_fmt = rng.choice([("f16", "f16"), ("q8_0", "q8_0"), ("q8_0", "tq3"), ("f16", "tq3")])
        return dict(op=op, tokens=tokens, seqs=rng.randint(1, min(tokens, 64)), hkv=hkv, d=d,
                    page=rng.choice([16, 32, 64, 128, 256]), k_fmt=k_fmt, v_fmt=v_fmt, rot=rng.choice([d, d // 2]),
                    pairs=rng.choice(["half", "next"]), norm=rng.random() < 0.6, offset=rng.choice([0.0, 1.0]),
                    inp=rng.choice(["f16", "bf16", "f32"]), far=rng.choice([4096, 65536]),
                    pad=rng.randint(0, min(3, tokens - 1)))
    batch = _log(rng, 1, 64)
    n_q = rng.choice([1, 1, 1, 2, 5])
    most = min(131072, 64 * 16384 * 8 * 128 // (batch * hkv * d))
    hi = _log(rng, n_q, most)
    page = rng.choice([16, 32, 64, 128, 256])
    shared = 0
    if batch > 1 and hi > 2 * page and rng.random() < 0.4:
        shared = rng.randint(1, (hi - n_q) // page) * page
    lo = rng.randint(shared + n_q, hi)
    k_fmt, v_fmt = rng.choice([("f16", "f16"), ("q8_0", "q8_0"), ("q8_0", "tq3"), ("f16", "q8_0")])
    return dict(op=op, batch=batch, n_q=n_q, hq=hkv * rng.choice([1, 3, 4, 5, 8]), hkv=hkv, d=d, page=page,
                k_fmt=k_fmt, v_fmt=v_fmt, lo=lo, hi=hi, empty=shared == 0 and batch > 2 and rng.random() < 0.5,
                causal=rng.random() < 0.7, cap=rng.choice([0.0, 0.0, 30.0]), out=rng.choice(["f16", "bf16"]),
                shared=shared)


# ---- inputs --------------------------------------------------------------------------
def _lens(c):
    """The lengths of a decode case (of the case alone; the seed permutes them): one of ``hi``, the
    others spread over the logarithm of the range."""
    r = random.Random("%d %d %d" % (c["batch"], c["lo"], c["hi"]))
    v = [c["hi"]] + [_log(r, c["lo"] - c["shared"], c["hi"] - c["shared"]) + c["shared"] for _ in range(c["batch"] - 1)]
    if c["empty"]:
        v[-1] = 0
    return v


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _table(far, rot):
    """Cosines and sines of every position, angles in 64 bits."""
    f = 10000.0 ** (-torch.arange(0, rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)
    a = torch.arange(far, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat((a.cos(), a.sin()), 1).float()


def _signs(d, g):
    """A sign vector of a rotation: +-1 values [d] and the same as 32-bit words."""
    bits = torch.randint(0, 2, (d,), generator=g, device="cuda")
    words = (bits.view(-1, 32) << torch.arange(32, device="cuda")).sum(1)
    return (1 - 2 * bits).float(), [int(w) for w in words.tolist()]


def _row(fmt, d):
    return {"f16": 2 * d, "q8_0": d + d // 16, "tq3": d // 4 + d // 8 + 2}[fmt]


def _pool(fmt, g, pages, hkv, page, d):
    """Planes of a cache that holds rows of N(0, 1) values."""
    shape = (pages, hkv, page)
    if fmt == "f16":
        return (_randn(g, *shape, d).half(),)
    if fmt == "q8_0":
        codes = (_randn(g, *shape, d) * 52).round().clamp(-127, 127).to(torch.int8)
        return (codes, ((2 + 0.6 * torch.rand(shape + (d // 32,), generator=g, device="cuda")) / 127).half())
    lo2 = torch.randint(0, 256, shape + (d // 4,), generator=g, device="cuda", dtype=torch.uint8)
    hi1 = torch.randint(0, 256, shape + (d // 8,), generator=g, device="cuda", dtype=torch.uint8)
    return (lo2, hi1, (math.sqrt(d) * (1 + 0.05 * _randn(g, *shape))).half())


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = dict(c)
    d, hkv = c["d"], c["hkv"]
    if c["op"] in ("rope", "append"):
        # the rows are slices of one projection's output: [tokens][query heads | key heads | value heads]
        hq = c.get("hq", 4 * hkv)
        qkv = _randn(g, c["tokens"], hq + 2 * hkv, d).to(DT[c["inp"]])
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        s["table"] = _table(c["far"], c["rot"])
        weight = lambda: (1 - c["offset"] + 0.2 * _randn(g, d)).to(DT[c["inp"]])  # noqa: E731
        s["wq"], s["wk"] = (weight(), weight()) if c["norm"] else (None, None)
    if c["op"] == "rope":
        s["pos"] = torch.randint(0, c["far"], (c["tokens"],), generator=g, device="cuda")
    elif c["op"] == "append":
        # each sequence continues at a position of its own; its rows go to pages taken in any order
        page, each = c["page"], -(-c["tokens"] // c["seqs"])
        held = (each + page - 1) // page + 1
        order = torch.randperm(c["seqs"] * held, generator=g, device="cuda").view(c["seqs"], held)
        begin = torch.randint(0, c["far"] - each, (c["seqs"],), generator=g, device="cuda")
        t = torch.arange(c["tokens"], device="cuda")
        at = begin[t // each] % page + t % each
        s["pos"] = begin[t // each] + t % each
        s["slots"] = order[t // each, at // page] * page + at % page
        if c["pad"]:
            s["slots"][-c["pad"]:] = -1
        s["sign"], s["words"] = _signs(d, g)
        for side in ("k", "v"):
            s[side + "_planes"] = _pool(c[side + "_fmt"], g, c["seqs"] * held, hkv, page, d)
    else:
        page, lens = c["page"], _lens(c)
        random.Random(seed).shuffle(lens)
        s["lens"] = torch.tensor(lens, device="cuda", dtype=torch.int32)
        wide, common = -(-max(lens) // page), c["shared"] // page
        pages = common + c["batch"] * (wide - common) + 1
        order = torch.randperm(pages, generator=g, device="cuda").int()
        table = order[common:common + c["batch"] * (wide - common)].view(c["batch"], wide - common)
        s["pages"] = torch.cat((order[:common].expand(c["batch"], common), table), 1).contiguous()
        s["sign"], s["words"] = _signs(d, g)
        for side in ("k", "v"):
            s[side + "_planes"] = _pool(c[side + "_fmt"], g, pages, hkv, page, d)
        s["query"] = _randn(g, c["batch"], c["n_q"], c["hq"], d).half()
        s["scale"] = d ** -0.5
    if own:  # the argument blocks that a decode loop builds once for a layer and keeps
        import quantized_position_split_gb300 as qps
        rope = qps.Rope(s["table"], c["pairs"] == "next") if "table" in s else None
        if c["op"] == "rope":
            s["args"] = qps.qk_rope_args(s["q"], s["k"], positions=s["pos"], rope=rope, q_norm=s["wq"], k_norm=s["wk"],
                                         norm=c["norm"], eps=EPS, norm_offset=c["offset"], out_dtype=DT[c["out"]])
        else:
            cache = qps.PagedKV(c["k_fmt"], c["v_fmt"], s["k_planes"], s["v_planes"], signs=s["words"])
            if c["op"] == "append":
                s["args"] = qps.paged_append_args(cache, s["k"], s["v"], s["slots"], positions=s["pos"], rope=rope,
                                                  k_norm=s["wk"], norm=c["norm"], eps=EPS, norm_offset=c["offset"])
            else:
                s["args"] = qps.paged_attn_args(s["query"], cache, s["pages"], s["lens"], scale=s["scale"],
                                                softcap=c["cap"], causal=c["causal"], shared_len=c["shared"],
                                                out_dtype=DT[c["out"]])
    return s


# ---- plain forms ---------------------------------------------------------------------
def _norm_rope(x, w, s):
    """Rows [tokens, heads, d] in 32 bits: RMS norm (sum of squares folded over each 8 neighbours, then
    over the groups by halves), weight, rotation by the table's row."""
    x = x.float()
    d, rot = x.shape[-1], s["rot"]
    if s["norm"]:
        t = (x * x).unflatten(-1, (-1, 8))
        t = t[..., :4] + t[..., 4:]
        t = t[..., :2] + t[..., 2:]
        t = t[..., 0] + t[..., 1]
        t = functools.reduce(lambda u, h: u[..., :h] + u[..., h:], [d >> i for i in range(4, d.bit_length())], t)
        x = x * (1.0 / torch.sqrt(t / d + EPS)) * (w.float() + s["offset"])
    cs = s["table"][s["pos"]][:, None]
    co, si = cs[..., :rot // 2], cs[..., rot // 2:]
    r, rest = x[..., :rot], x[..., rot:]
    if s["pairs"] == "half":
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * co - b * si, b * co + a * si), -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * co - b * si, b * co + a * si), -1).flatten(-2)
    return torch.cat((r, rest), -1)


def _fwht(x):
    """Walsh-Hadamard transform of the last dimension, (a + b, a - b) over spans 1, 2, 4, ..."""
    def stage(u, h):
        a, b = u.unflatten(-1, (-1, 2, h)).unbind(-2)
        return torch.stack((a + b, a - b), -2).flatten(-3)
    return functools.reduce(stage, [1 << i for i in range(x.shape[-1].bit_length() - 1)], x)


def _encode(fmt, x, sign):
    """Stored planes of fp16 rows x [rows, hkv, d], each step rounded to 32 bits."""
    if fmt == "f16":
        return (x,)
    f = x.float()
    d = f.shape[-1]
    if fmt == "q8_0":
        b = f.unflatten(-1, (-1, 32))
        most = b.abs().amax(-1)
        scale = (most / torch.full_like(most, 127.0)).half()
        z = b / scale.float()[..., None]
        t = torch.trunc(z)
        t = t + torch.sign(z) * ((z - t).abs() >= 0.5)  # halves away from zero
        t = torch.where(scale[..., None] == 0, torch.zeros_like(t), t).clamp(-127, 127)
        return (t.flatten(-2).to(torch.int8), scale)
    fold = functools.reduce(lambda u, h: u[..., :h] + u[..., h:], [d >> i for i in range(1, d.bit_length())], f * f)
    n = torch.sqrt(fold)
    z = _fwht(f * sign) / n
    mid = torch.tensor([(a + b) / 2 for a, b in zip(LEVELS, LEVELS[1:])], device=x.device)
    k = torch.where(n == 0, torch.full_like(z, 3), torch.bucketize(z, mid, right=True).float()).int()
    mag = torch.where(k >= 4, k - 4, 3 - k)
    at = torch.arange(8, device=x.device)
    lo2 = (mag.unflatten(-1, (-1, 4)) << (2 * at[:4])).sum(-1)
    hi1 = ((k >= 4).int().unflatten(-1, (-1, 8)) << at).sum(-1)
    return (lo2.to(torch.uint8), hi1.to(torch.uint8), n[..., 0].half())


def _decode(fmt, planes, sign):
    """Values, in 32 bits, of stored rows."""
    if fmt == "f16":
        return planes[0].float()
    if fmt == "q8_0":
        return (planes[0].float().unflatten(-1, (-1, 32)) * planes[1].float()[..., None]).flatten(-2)
    at = torch.arange(8, device=sign.device)
    mag = ((planes[0][..., None].int() >> (2 * at[:4])) & 3).flatten(-2)
    up = ((planes[1][..., None].int() >> at) & 1).flatten(-2)
    c = torch.tensor(LEVELS, device=sign.device)[torch.where(up == 1, 4 + mag, 3 - mag)]
    return _fwht(c) * sign * (planes[2].float()[..., None] / sign.numel())


def _attend(s):
    b, n_q, hkv, d, page = s["batch"], s["n_q"], s["hkv"], s["d"], s["page"]
    wide = s["pages"].shape[1]
    at = s["pages"].long()
    t = torch.arange(wide * page, device="cuda")
    real = t < s["lens"][:, None]
    last = s["lens"][:, None] - (n_q - 1 - torch.arange(n_q, device="cuda") if s["causal"] else torch.zeros(n_q, device="cuda"))
    seen = real[:, None] & (t < last[..., None])  # [b, n_q, t]
    k, v = (_decode(s[x + "_fmt"], [p[at].transpose(1, 2).flatten(2, 3) for p in s[x + "_planes"]], s["sign"])
            for x in ("k", "v"))  # [b, hkv, t, d]
    k, v = (torch.where(real[:, None, :, None], x, torch.zeros_like(x[:1, :1, :1, :1])) for x in (k, v))
    q = s["query"].float().unflatten(2, (hkv, -1)).permute(0, 2, 1, 3, 4)  # [b, hkv, n_q, g, d]
    z = (q.flatten(2, 3) @ k.transpose(2, 3)).unflatten(2, (n_q, -1)) * s["scale"]
    if s["cap"]:
        z = s["cap"] * torch.tanh(z / s["cap"])
    z = torch.where(seen[:, None, :, None], z, torch.full_like(z, -math.inf))
    most = z.amax(-1, keepdim=True)
    most = torch.where(most == -math.inf, torch.zeros_like(most), most)
    p = torch.exp(z - most)
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).unflatten(2, (n_q, -1)) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (most + torch.log(total))[..., 0]
    return o.permute(0, 2, 1, 3, 4).reshape(b * n_q * s["hq"], d).to(DT[s["out"]]), lse.permute(0, 2, 1, 3).reshape(-1)


def run(state):
    s = state
    if own:
        import quantized_position_split_gb300 as qps
        if s["op"] == "rope":
            return qps.qk_norm_rope(s["args"])
        if s["op"] == "append":
            qps.kv_append_paged(s["args"])
            # codes and planes come back as stored: they are held to equality
            return {"k": s["k_planes"], "v": s["v_planes"]}
        return qps.attn_decode_paged(s["args"])
    if s["op"] == "rope":
        return _norm_rope(s["q"], s["wq"], s).to(DT[s["out"]]), _norm_rope(s["k"], s["wk"], s).to(DT[s["out"]])
    if s["op"] == "append":
        keep = s["slots"] >= 0
        slot = s["slots"][keep]
        rows = {"k": _norm_rope(s["k"], s["wk"], s).half(), "v": s["v"].half()}
        for x in ("k", "v"):
            for plane, new in zip(s[x + "_planes"], _encode(s[x + "_fmt"], rows[x][keep], s["sign"])):
                plane[slot // s["page"], :, slot % s["page"]] = new
        return {"k": s["k_planes"], "v": s["v_planes"]}
    return _attend(s)


# ---- what a pass cannot do without ----------------------------------------------------
def work(case):
    c = case
    d, hkv = c["d"], c["hkv"]
    size = {"f16": 2, "bf16": 2, "f32": 4}
    if c["op"] == "rope":
        rows = c["tokens"] * (c["hq"] + hkv)
        table = min(c["tokens"], c["far"]) * c["rot"] * 4
        return {"bytes": rows * d * (size[c["inp"]] + size[c["out"]]) + table + 8 * c["tokens"], "flops": 8 * rows * d}
    if c["op"] == "append":
        kept = c["tokens"] - c["pad"]
        rows = kept * hkv
        out = rows * (_row(c["k_fmt"], d) + _row(c["v_fmt"], d))
        return {"bytes": 2 * rows * d * size[c["inp"]] + out + kept * c["rot"] * 4 + 16 * c["tokens"], "flops": 16 * rows * d}
    lens, common = _lens(c), c["shared"]
    held = common + sum(max(0, n - common) for n in lens)
    rows = c["batch"] * c["n_q"] * c["hq"]
    seen = sum(max(0, n - (c["n_q"] - 1 - i if c["causal"] else 0)) for n in lens for i in range(c["n_q"]))
    return {"bytes": held * hkv * (_row(c["k_fmt"], d) + _row(c["v_fmt"], d)) + rows * (4 * d + 4) + 4 * c["batch"],
            "flops": 4 * seen * c["hq"] * d}


# ---- the definitions in 64 bits -------------------------------------------------------
def _rotated64(x, w, s):
    x = x.double()
    d, rot = x.shape[-1], s["rot"]
    if s["norm"]:
        x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * (w.double() + s["offset"])
    co, si = (s["table"][s["pos"]].double()[:, None, i * rot // 2:(i + 1) * rot // 2] for i in (0, 1))
    first = torch.arange(rot // 2, device="cuda") * (1 if s["pairs"] == "half" else 2)
    second = first + (rot // 2 if s["pairs"] == "half" else 1)
    z = torch.complex(x[..., first], x[..., second]) * torch.complex(co, si)
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _hadamard64(d):
    i = torch.arange(d, device="cuda")
    both = i[:, None] & i[None]
    odd = sum((both >> b) & 1 for b in range(d.bit_length())) % 2
    return 1.0 - 2.0 * odd.double()


def _values64(fmt, planes, sign):
    if fmt == "f16":
        return planes[0].double()
    if fmt == "q8_0":
        return planes[0].double() * planes[1].double().repeat_interleave(32, -1)
    d = sign.numel()
    e = torch.arange(d, device="cuda")
    mag = (planes[0].long()[..., e // 4] >> (2 * (e % 4))) & 3
    up = (planes[1].long()[..., e // 8] >> (e % 8)) & 1
    size = torch.tensor(LEVELS[4:], device="cuda", dtype=torch.float64)[mag]
    c = torch.where(up == 1, size, -size)
    return (c @ _hadamard64(d)) * sign.double() * planes[2].double()[..., None] / d


def exact(case, seed):
    c, s = case, prepare(case, seed)
    d, hkv, page = c["d"], c["hkv"], c.get("page")
    if c["op"] == "rope":
        return _rotated64(s["q"], s["wq"], s), _rotated64(s["k"], s["wk"], s)
    if c["op"] == "append":
        out = {}
        for x, rows in (("k", _rotated64(s["k"], s["wk"], s)), ("v", s["v"].double())):
            new = {"f16": lambda r: [r], "q8_0": lambda r: [None, r.unflatten(-1, (-1, 32)).abs().amax(-1) / 127],
                   "tq3": lambda r: [None, None, r.norm(dim=-1)]}[c[x + "_fmt"]](rows)
            got = []
            for plane, values in zip(s[x + "_planes"], new):
                if values is None:
                    got.append(None)
                    continue
                p = plane.double()
                for h in range(hkv):
                    use = s["slots"] >= 0
                    p[s["slots"][use] // page, h, s["slots"][use] % page] = values[use, h]
                got.append(p)
            out[x] = got
        return out
    o = torch.zeros(c["batch"], c["n_q"], c["hq"], d, device="cuda", dtype=torch.float64)
    lse = torch.full((c["batch"], c["n_q"], c["hq"]), -math.inf, device="cuda", dtype=torch.float64)
    group = c["hq"] // hkv
    for b, n in enumerate(s["lens"].tolist()):
        if not n:
            continue
        at = s["pages"][b, :-(-n // page)].long()
        for h in range(hkv):
            k, v = (_values64(c[x + "_fmt"], [p[at, h].flatten(0, 1)[:n] for p in s[x + "_planes"]], s["sign"])
                    for x in ("k", "v"))
            q = s["query"][b, :, h * group:(h + 1) * group].double()
            z = torch.einsum("igd,td->igt", q, k) * s["scale"]
            if c["cap"]:
                z = c["cap"] * torch.tanh(z / c["cap"])
            if c["causal"]:
                late = torch.arange(n, device="cuda") > n - c["n_q"] + torch.arange(c["n_q"], device="cuda")[:, None]
                z = z.masked_fill(late[:, None], -math.inf)
            lse[b, :, h * group:(h + 1) * group] = torch.logsumexp(z, -1)
            o[b, :, h * group:(h + 1) * group] = torch.softmax(z, -1) @ v
    return o.reshape(-1, d), lse.reshape(-1)
