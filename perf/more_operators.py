"""Cases of the operators for long streams in a paged KV cache, with their plain forms.

Five entry points are measured:

* ``decode``   decode attention over a sliding window and a few first positions that stay visible
               (sinks): ``attn_decode_paged`` with ``window`` / ``sinks``;
* ``prompt``   attention of ragged prompt chunks over such a cache, causal, with or without a window
               (``attn_prompt_paged``);
* ``extend``   pages for the next tokens of each sequence, pages behind the window given back,
               sequences trimmed (``kv_extend_paged``);
* ``fork``     sequences that continue other sequences, their pages shared, the last one copied
               (``kv_fork_paged``);
* ``compact``  a pool's live pages moved to its front (``kv_compact_paged``).

Layouts.  A plane of the cache is ``[pages][hkv][page][row]``; a slot is ``page_index * page +
offset``.  Stored formats: ``f16`` values; ``q8_0`` int8 codes and one fp16 scale per 32 values;
``tq3`` a 2-bit magnitude plane, a 1-bit sign plane and an fp16 norm of the rotated row.  Entry j of
a sequence's row of the page table is the page of its positions ``[j * page, (j + 1) * page)``, or -1;
``refs`` counts the entries that name each page.
"""

import functools
import math
import random

import torch

own = False

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
LEVELS = (-2.15234375, -1.34375, -0.755859375, -0.2451171875, 0.2451171875, 0.755859375, 1.34375, 2.15234375)


def listed():
    return [
        # one token of one long conversation, behind a window of recent positions: latency
        dict(name="window_token", op="decode", batch=1, n_q=1, hq=40, hkv=8, d=128, page=64, k_fmt="f16", v_fmt="f16",
             lo=131072, hi=131072, empty=False, window=4096, sinks=4, cap=0.0, out="f16"),
        # a ragged batch of agents, one row of it padding, 8-bit keys and 3-bit values: bandwidth
        dict(name="window_agents", op="decode", batch=61, n_q=1, hq=32, hkv=8, d=128, page=32, k_fmt="q8_0", v_fmt="tq3",
             lo=1, hi=65536, empty=True, window=8192, sinks=64, cap=0.0, out="bf16"),
        # a few tokens typed behind a conversation: latency
        dict(name="prompt_short", op="prompt", batch=1, tokens=17, past=1000, hq=40, hkv=8, d=128, page=64, k_fmt="f16",
             v_fmt="f16", empty=False, window=0, sinks=0, cap=0.0, out="f16"),
        # one long prompt from its first position: the tensor cores' rate
        dict(name="prompt_long", op="prompt", batch=1, tokens=16384, past=0, hq=40, hkv=8, d=128, page=64, k_fmt="f16",
             v_fmt="f16", empty=False, window=0, sinks=0, cap=0.0, out="f16"),
        # chunks of a ragged batch over an 8-bit cache on small pages, a window and sinks, one sequence without tokens
        dict(name="prompt_ragged_window", op="prompt", batch=13, tokens=8191, past=16384, hq=32, hkv=8, d=128, page=16,
             k_fmt="q8_0", v_fmt="q8_0", empty=True, window=1024, sinks=16, cap=0.0, out="bf16"),
        # a chunk over wide heads with softcap, 8-bit keys and 3-bit values
        dict(name="prompt_wide_tq3", op="prompt", batch=1, tokens=2048, past=8192, hq=16, hkv=2, d=512, page=128,
             k_fmt="q8_0", v_fmt="tq3", empty=False, window=0, sinks=0, cap=50.0, out="f16"),
        # the step of a decode loop: one position for each of 64 sequences, in a window
        dict(name="extend_step", op="extend", batch=64, each=1, trim=False, page=16, far=131072, pages=65536, window=4096,
             sinks=64, layers=2, hkv=2, d=128, k_fmt="q8_0", v_fmt="q8_0", shared=True),
        # prompt chunks are admitted and, their requests cancelled, taken back
        dict(name="extend_prompts", op="extend", batch=33, each=1000, trim=True, page=64, far=16384, pages=16384, window=0,
             sinks=0, layers=4, hkv=2, d=128, k_fmt="f16", v_fmt="f16", shared=True),
        # seven beams continue an eighth one
        dict(name="fork_beams", op="fork", rows=8, parents=1, forks=7, freed=0, page=64, far=1000, pages=512, layers=4, hkv=8,
             d=128, k_fmt="f16", v_fmt="f16"),
        # agents that take up long conversations, some others ended, in a layer stack of wide heads
        dict(name="fork_agents", op="fork", rows=64, parents=4, forks=51, freed=9, page=128, far=32768, pages=2048, layers=4,
             hkv=2, d=512, k_fmt="q8_0", v_fmt="tq3"),
        # a small pool of which a quarter lives
        dict(name="compact_small", op="compact", rows=16, pages=1024, page=16, live=0.25, layers=2, hkv=8, d=64, k_fmt="f16",
             v_fmt="f16"),
        # a large pool, half of it live: bandwidth
        dict(name="compact_pool", op="compact", rows=128, pages=4096, page=64, live=0.5, layers=4, hkv=8, d=128, k_fmt="f16",
             v_fmt="f16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prompt", "prompt", "prompt", "extend", "fork", "compact"])
    page = rng.choice([16, 32, 64, 128, 256])
    k_fmt, v_fmt = rng.choice([("f16", "f16"), ("q8_0", "q8_0"), ("q8_0", "tq3"), ("f16", "q8_0")])
    d = rng.choice([64, 128, 128, 256, 512])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 3, 4, 5, 8])
    out, cap = rng.choice(["f16", "bf16"]), rng.choice([0.0, 0.0, 30.0])
    if op == "decode":
        batch, n_q, window = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 5]), _log(rng, 1, 16384)
        window = min(window, max(1, 61 * 8192 * 8 * 128 // (batch * hkv * d)))
        hi = _log(rng, n_q, min(131072, max(2 * window, 64 * 65536 * 128 // (batch * hkv * d))))
        return dict(op=op, batch=batch, n_q=n_q, hq=hq, hkv=hkv, d=d, page=page, k_fmt=k_fmt, v_fmt=v_fmt,
                    lo=rng.randint(n_q, hi), hi=hi, empty=batch > 2 and rng.random() < 0.5, window=window,
                    sinks=rng.choice([0, 1, 4, 16, 64, 100]), cap=cap, out=out)
    if op == "prompt":
        window = rng.choice([0, _log(rng, 1, 8192)])
        tokens = _log(rng, 1, 8192)
        most = int(2.7e12 / (4 * hq * d * tokens))  # positions a token may see, by the largest case's work
        tokens = min(tokens, most)
        batch = rng.randint(1, min(tokens, 16))
        return dict(op=op, batch=batch, tokens=tokens, past=rng.choice([0, _log(rng, 1, max(1, min(32768, most // 2)))]), hq=hq,
                    hkv=hkv, d=d, page=page, k_fmt=k_fmt, v_fmt=v_fmt, empty=batch > 2 and rng.random() < 0.5, window=window,
                    sinks=rng.choice([0, 1, 4, 16, 64, 100]) if window else 0, cap=cap, out=out)
    # pools of at most 1 GB a layer
    row = _row(k_fmt, d) + _row(v_fmt, d)
    layers = rng.randint(1, 4)
    most = max(64, min(65536, 2 ** 30 // (row * hkv * page)))
    kept = dict(page=page, layers=layers, hkv=hkv, d=d, k_fmt=k_fmt, v_fmt=v_fmt)
    if op == "extend":
        pages = _log(rng, 64, most)
        batch = _log(rng, 1, min(64, pages // 64))
        held = pages * page // (4 * batch)  # positions of a sequence, so that the pool is not filled
        window = rng.choice([0, rng.randint(1, held)])
        return dict(op=op, batch=batch, each=_log(rng, 1, held), trim=True, far=_log(rng, 1, held if not window else 65536),
                    pages=pages, window=window, sinks=rng.choice([0, 1, 64, 100]) if window else 0,
                    shared=rng.random() < 0.5, **kept)
    rows = _log(rng, 2, 64)
    if op == "fork":
        parents = rng.randint(1, rows - 1)
        forks = rng.randint(1, rows - parents)
        pages = _log(rng, max(64, 4 * rows), max(most, 4 * rows))
        return dict(op=op, rows=rows, parents=parents, forks=forks, freed=rng.randint(0, rows - parents - forks),
                    far=_log(rng, 1, (pages - 2 * rows) * page // rows), pages=pages, **kept)
    return dict(op=op, rows=rows, pages=_log(rng, max(64, rows), max(most, rows)), live=rng.uniform(0.05, 0.95), **kept)


# ---- inputs --------------------------------------------------------------------------
def _shares(r, total, n):
    """``total`` in ``n`` parts, sizes spread over their logarithm."""
    w = [math.exp(r.uniform(0.0, 4.0)) for _ in range(n)]
    cut = [0] + [int(round(total * sum(w[:i + 1]) / sum(w))) for i in range(n)]
    cut[-1] = total
    return [b - a for a, b in zip(cut, cut[1:])]


def _of_case(c):
    return random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))


def _lens(c):
    """(new tokens, length) of each sequence of an attention case (of the case alone; the seed
    permutes them)."""
    r = _of_case(c)
    b = c["batch"]
    if c["op"] == "decode":
        v = [(c["n_q"], n) for n in [c["hi"]] + [_log(r, c["lo"], c["hi"]) for _ in range(b - 1)]]
        if c["empty"]:
            v[-1] = (c["n_q"], 0)
        return v
    new = _shares(r, c["tokens"], b - 1) + [0] if c["empty"] else _shares(r, c["tokens"], b)
    past = [c["past"]] + [_log(r, 1, c["past"]) if c["past"] else 0 for _ in range(b - 1)]
    return [(n, n + p) for n, p in zip(new, past)]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


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
        return (torch.randn(shape + (d,), generator=g, device="cuda", dtype=torch.float16),)
    if fmt == "q8_0":
        codes = torch.randint(-127, 128, shape + (d,), generator=g, device="cuda", dtype=torch.int8)
        return (codes, ((1.6 + 0.4 * torch.rand(shape + (d // 32,), generator=g, device="cuda")) / 127).half())
    lo2 = torch.randint(0, 256, shape + (d // 4,), generator=g, device="cuda", dtype=torch.uint8)
    hi1 = torch.randint(0, 256, shape + (d // 8,), generator=g, device="cuda", dtype=torch.uint8)
    return (lo2, hi1, (math.sqrt(d) * (1 + 0.05 * _randn(g, *shape))).half())


def _attention_state(c, seed, g, s):
    page, lens = c["page"], _lens(c)
    random.Random(seed).shuffle(lens)
    s["seqs"] = lens
    total = sum(n for n, _ in lens)
    s["lens"] = torch.tensor([n for _, n in lens], device="cuda", dtype=torch.int32)
    starts = [0]
    for n, _ in lens:
        starts.append(starts[-1] + n)
    s["starts"] = torch.tensor(starts, device="cuda", dtype=torch.int32)
    width = max(1, -(-max(n for _, n in lens) // page))
    # what the window has left behind is no longer held: those entries name no page
    need = []
    for b, (n, length) in enumerate(lens):
        low = max(0, length - n - c["window"] + 1) if c["window"] else 0
        need += [(b, j) for j in range(-(-length // page)) if (j + 1) * page > low or j * page < c["sinks"]]
    pages = len(need) + 1
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((len(lens), width), -1, device="cuda", dtype=torch.int32)
    at = torch.tensor(need, device="cuda", dtype=torch.int64).view(-1, 2)
    table[at[:, 0], at[:, 1]] = order[:len(need)]
    s["table"] = table
    s["sign"], s["words"] = _signs(c["d"], g)
    for side in ("k", "v"):
        s[side + "_planes"] = _pool(c[side + "_fmt"], g, pages, c["hkv"], page, c["d"])
    s["query"] = _randn(g, total, c["hq"], c["d"]).half()
    s["scale"] = c["d"] ** -0.5


def _held(c, seed=0):
    """Lengths (of the case alone) and table rows of a pool's sequences: each holds pages of its own,
    taken in any order."""
    page, pages, r = c["page"], c["pages"], _of_case(c)
    free = list(range(pages))
    random.Random(seed).shuffle(free)
    take = lambda n: [free.pop() for _ in range(n)]  # noqa: E731
    if c["op"] == "extend":
        lens = [_log(r, 1, c["far"]) for _ in range(c["batch"])]
        new = [_log(r, 1, c["each"]) for _ in range(c["batch"])]
        # (a decode loop's sequences grow from call to call)
        width = -(-(c["far"] + (c["each"] if c["trim"] else c["far"])) // page) + 1
        table = []
        for n in lens:
            low = n - c["window"] if c["window"] else 0
            table.append([take(1)[0] if (j + 1) * page > low or j * page < c["sinks"] else -1 for j in range(-(-n // page))])
        if c["shared"]:  # every fourth sequence was forked from the one before it and cut back into the pages they share
            for b in range(3, c["batch"], 4):
                free += [p for p in table[b] if p >= 0]
                lens[b] = max(1, lens[b - 1] - r.randrange(2 * page))
                table[b] = table[b - 1][:-(-lens[b] // page)]
        return lens, table, width, new
    if c["op"] == "fork":
        lens = [_log(r, max(1, c["far"] // 4), c["far"]) if b < c["parents"] else _log(r, 1, c["far"]) for b in range(c["rows"])]
        # (the other rows hold what is left by the pool)
        spare = pages - sum(-(-n // page) for n in lens[:c["parents"]]) - 2 * c["rows"]
        for b in range(c["parents"], c["rows"]):
            lens[b] = min(lens[b], spare * page // c["rows"])
        return lens, [take(-(-n // page)) for n in lens], -(-c["far"] // page) + 1, None
    count = max(c["rows"], int(round(c["live"] * pages)))
    lens = [n * page - r.randrange(page) if n else 0 for n in _shares(r, count, c["rows"])]
    return lens, [take(-(-n // page)) for n in lens], max(1, max(-(-n // page) for n in lens)), None


def _pool_state(c, seed, g, s):
    r = random.Random(seed)
    lens, rows, width, new = _held(c, seed)
    table = torch.full((len(rows), width), -1, dtype=torch.int32)
    refs = [0] * c["pages"]
    for b, row in enumerate(rows):
        table[b, :len(row)] = torch.tensor(row, dtype=torch.int32)
        for p in row:
            if p >= 0:
                refs[p] += 1
    s["table"], s["lens"] = table.cuda(), torch.tensor(lens, device="cuda", dtype=torch.int32)
    s["refs"] = torch.tensor(refs, device="cuda", dtype=torch.int32)
    s["sign"], s["words"] = _signs(c["d"], g)
    s["pool"] = [tuple(_pool(c[x + "_fmt"], g, c["pages"], c["hkv"], c["page"], c["d"]) for x in ("k", "v"))
                 for _ in range(c["layers"])]
    if c["op"] == "extend":
        s["new"] = torch.tensor(new, device="cuda", dtype=torch.int32)
        s["back"] = -s["new"]
        s["most"] = sum(new) + 3  # (the rows of a captured step: a few more than any call fills)
    elif c["op"] == "fork":
        src = [r.randrange(c["parents"]) for _ in range(c["forks"])] + [-1] * c["freed"]
        dst = list(range(c["parents"], c["rows"]))
        r.shuffle(dst)
        s["src"] = torch.tensor(src, device="cuda", dtype=torch.int32)
        s["dst"] = torch.tensor(dst[:len(src)], device="cuda", dtype=torch.int32)
    else:  # the pool as the sequences that ended left it: every pass compacts it again
        s["table0"], s["refs0"] = s["table"].clone(), s["refs"].clone()


def prepare(case, seed):
    c, g, s = case, _gen(seed), dict(case)
    attention = c["op"] in ("decode", "prompt")
    (_attention_state if attention else _pool_state)(c, seed, g, s)
    if own:  # the argument blocks that a serving loop builds once and keeps
        import quantized_position_split_gb300 as qps
        if attention:
            cache = qps.PagedKV(c["k_fmt"], c["v_fmt"], s["k_planes"], s["v_planes"], signs=s["words"])
            more = dict(scale=s["scale"], softcap=c["cap"], window=c["window"], sinks=c["sinks"], out_dtype=DT[c["out"]])
            if c["op"] == "decode":
                q = s["query"].view(c["batch"], c["n_q"], c["hq"], c["d"])
                s["args"] = qps.paged_attn_args(q, cache, s["table"], s["lens"], causal=True, **more)
            else:
                s["args"] = qps.paged_prompt_args(s["query"], cache, s["table"], s["lens"], s["starts"], **more)
            return s
        caches = [qps.PagedKV(c["k_fmt"], c["v_fmt"], k, v, signs=s["words"]) for k, v in s["pool"]]
        seqs = qps.PagedSeqs(caches, s["table"], s["lens"], s["refs"])
        if c["op"] == "extend":
            s["args"] = qps.paged_extend_args(seqs, s["new"], window=c["window"], sinks=c["sinks"], max_tokens=s["most"])
            s["undo"] = qps.paged_extend_args(seqs, s["back"], window=c["window"], sinks=c["sinks"], max_tokens=s["most"])
        elif c["op"] == "fork":
            s["args"] = qps.paged_fork_args(seqs, s["src"], s["dst"])
        else:
            s["args"] = qps.paged_compact_args(seqs)
    return s


# ---- plain forms ---------------------------------------------------------------------
def _fwht(x):
    """Walsh-Hadamard transform of the last dimension, (a + b, a - b) over spans 1, 2, 4, ..."""
    def stage(u, h):
        a, b = u.unflatten(-1, (-1, 2, h)).unbind(-2)
        return torch.stack((a + b, a - b), -2).flatten(-3)
    return functools.reduce(stage, [1 << i for i in range(x.shape[-1].bit_length() - 1)], x)


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


def _visible(q0, q1, window, sinks):
    """The positions that the queries at positions [q0, q1) see: those before the window, the rest."""
    low = max(0, q0 - window + 1) if window else 0
    return min(sinks, low), low, q1


def _attend(s, q, table, length):
    """Queries q [b, n, hq, d], the newest positions of sequences of ``length`` [b], over what they see of
    the cache."""
    (b, n, hq, d), page, hkv = q.shape, s["page"], s["hkv"]
    at = (length[:, None] - n + torch.arange(n, device="cuda"))[..., None]  # [b, n, 1] positions of the queries
    low = (at[:, 0] - s["window"] + 1).clamp(min=0) if s["window"] else torch.zeros_like(at[:, 0])
    few = low.clamp(max=s["sinks"])
    i = torch.arange(s["span"] + n, device="cuda")
    t = torch.where(i < few, i.expand(b, -1), low + i - few)  # [b, t] the positions any of them sees
    seen = (t[:, None] <= at) & (t[:, None] >= 0)
    if s["window"]:
        seen = seen & ((t[:, None] > at - s["window"]) | (t[:, None] < s["sinks"]))
    real = t < length[:, None]
    t = torch.where(real, t, torch.zeros_like(t))
    pages = torch.where(real, table.gather(1, t // page), torch.zeros_like(table[:1, :1])).long()
    k, v = (_decode(s[x + "_fmt"], [p[pages, :, t % page] for p in s[x + "_planes"]], s["sign"]).transpose(1, 2)
            for x in ("k", "v"))  # [b, hkv, t, d]
    q = q.float().unflatten(2, (hkv, -1)).permute(0, 2, 1, 3, 4)  # [b, hkv, n, g, d]
    z = (q.flatten(2, 3) @ k.transpose(2, 3)).unflatten(2, (n, -1)) * s["scale"]
    if s["cap"]:
        z = s["cap"] * torch.tanh(z / s["cap"])
    z = torch.where(seen[:, None, :, None], z, torch.full_like(z[:1, :1, :1, :1], -math.inf))
    most = z.amax(-1, keepdim=True)
    most = torch.where(most == -math.inf, torch.zeros_like(most), most)
    p = torch.exp(z - most)
    total = p.sum(-1, keepdim=True)
    w = (p.flatten(2, 3) @ v).unflatten(2, (n, -1)) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (most + torch.log(total))[..., 0]
    return w.permute(0, 2, 1, 3, 4).reshape(-1, d).to(DT[s["out"]]), lse.permute(0, 2, 1, 3).reshape(-1)


def _attention(s):
    if s["op"] == "decode":
        s["span"] = min(max(n for _, n in s["seqs"]), s["window"] + s["sinks"])
        return _attend(s, s["query"].unflatten(0, (s["batch"], -1)), s["table"], s["lens"].long())
    # one sequence after the other, 1024 queries at a time, so that their logits stay small
    parts, row = [], 0
    for b, (n, length) in enumerate(s["seqs"]):
        for i0 in range(0, n, 1024):
            i1 = min(n, i0 + 1024)
            end = length - n + i1
            s["span"] = min(end, s["window"] + s["sinks"] if s["window"] else end)
            parts.append(_attend(s, s["query"][None, row + i0:row + i1], s["table"][b:b + 1],
                                 torch.full((1,), end, device="cuda")))
        row += n
    return torch.cat([o for o, _ in parts]), torch.cat([e for _, e in parts])


def _planes(s):
    return [p for layer in s["pool"] for side in layer for p in side]


def _count(refs, pages, by):
    refs.index_add_(0, pages.long(), torch.full_like(pages, by, dtype=torch.int32))


def _extend(s, new):
    page, table, refs, lens = s["page"], s["table"], s["refs"], s["lens"]
    width = table.shape[1]
    old = lens.long()
    end = (old + new).clamp(min=0)
    more = new.clamp(min=0).long()
    j = torch.arange(width, device="cuda")
    had, has = (-(-n // page)[:, None] for n in (old, end))
    gone = (j < had) & (j >= has)
    if s["window"]:
        low = (torch.where(new > 0, old, end) - s["window"] + 1)[:, None]
        gone = gone | ((j < had) & ((j + 1) * page <= low) & (j * page >= s["sinks"]))
    gone = gone & (table >= 0)
    _count(refs, table[gone], -1)
    table[gone] = -1
    # a page that is not full and not this sequence's alone is copied before it is written
    part = (old % page > 0) & (new > 0)
    last = (old // page).clamp(max=width - 1)[:, None]
    held = table.gather(1, last)[:, 0].long()
    copied = part & (refs[held.clamp(min=0)] > 1)
    fresh = ((j >= had) & (j < has) & (new > 0)[:, None]) | (copied[:, None] & (j == last))
    order = torch.sort((refs > 0).int(), stable=True).indices.int()
    table[fresh] = order[:int(fresh.sum())]
    _count(refs, table[fresh], 1)
    _count(refs, held[copied].int(), -1)
    t = torch.arange(page, device="cuda")
    keep = t < (old % page)[copied][:, None]
    to = table.gather(1, last)[:, 0].long()[copied]
    for p in _planes(s):
        a, b = p[held[copied]], p[to]
        p[to] = torch.where(keep.view(keep.shape[0], 1, page, *[1] * (p.dim() - 3)), a, b)
    lens.copy_(end)
    # the new tokens' rows, packed; the rows behind them are padding
    starts = torch.cat((torch.zeros(1, device="cuda", dtype=torch.int64), torch.cumsum(more, 0)))
    i = torch.arange(s["most"], device="cuda")
    b = torch.searchsorted(starts, i, right=True) - 1
    real = i < starts[-1]
    b = torch.where(real, b, torch.zeros_like(b))
    pos = torch.where(real, old[b] + i - starts[b], torch.zeros_like(i))
    slots = torch.where(real, table[b, pos // page].long() * page + pos % page, torch.full_like(i, -1))
    return starts.int(), slots, pos


def _fork(s):
    page, table, refs, lens = s["page"], s["table"], s["refs"], s["lens"]
    src, dst = s["src"].long(), s["dst"].long()
    j = torch.arange(table.shape[1], device="cuda")
    n = torch.where(src >= 0, lens[src.clamp(min=0)].long(), torch.zeros_like(src))
    rows = torch.where(j < -(-n // page)[:, None], table[src.clamp(min=0)], torch.full_like(table[:1], -1))
    gone = table[dst]
    gone = gone[(j < -(-lens[dst].long() // page)[:, None]) & (gone >= 0)]
    _count(refs, rows[rows >= 0], 1)
    _count(refs, gone, -1)
    # the last page, where it is not full, becomes a copy
    last = (n // page).clamp(max=table.shape[1] - 1)[:, None]
    held = rows.gather(1, last)[:, 0]
    part = (n % page > 0) & (held >= 0)
    order = torch.sort((refs > 0).int(), stable=True).indices.int()
    to = order[:int(part.sum())]
    rows[part] = rows[part].scatter(1, last[part], to[:, None])
    _count(refs, held[part], -1)
    _count(refs, to, 1)
    keep = torch.arange(page, device="cuda") < (n % page)[part][:, None]
    for p in _planes(s):
        a, b = p[held[part].long()], p[to.long()]
        p[to.long()] = torch.where(keep.view(keep.shape[0], 1, page, *[1] * (p.dim() - 3)), a, b)
    table[dst] = rows
    lens[dst] = n.int()


def _compact(s):
    page, table, refs = s["page"], s["table"], s["refs"]
    live = (refs > 0).sum()
    i = torch.arange(refs.numel(), device="cuda")
    holes, far = i[(refs == 0) & (i < live)], i[(refs > 0) & (i >= live)]
    ids = torch.where(refs > 0, i, torch.full_like(i, -1))
    ids[far] = holes
    for p in _planes(s):
        p[holes] = p[far]
    refs[holes] = refs[far]
    refs[far] = 0
    used = (torch.arange(table.shape[1], device="cuda") < -(-s["lens"].long() // page)[:, None]) & (table >= 0)
    table[used] = ids[table[used].long()].int()
    return ids.int(), live.int().view(1)


def run(state):
    s = state
    if own:
        import quantized_position_split_gb300 as qps
        if s["op"] == "decode":
            return qps.attn_decode_paged(s["args"])
        if s["op"] == "prompt":
            return qps.attn_prompt_paged(s["args"])
    elif s["op"] in ("decode", "prompt"):
        return _attention(s)
    out = {"table": s["table"], "lens": s["lens"], "refs": s["refs"], "planes": _planes(s)}
    if s["op"] == "extend":
        out["new"] = qps.kv_extend_paged(s["args"]) if own else _extend(s, s["new"])
        if s["trim"]:
            qps.kv_extend_paged(s["undo"]) if own else _extend(s, s["back"])
    elif s["op"] == "fork":
        qps.kv_fork_paged(s["args"]) if own else _fork(s)
    else:
        s["table"].copy_(s["table0"])
        s["refs"].copy_(s["refs0"])
        out["moved"] = qps.kv_compact_paged(s["args"]) if own else _compact(s)
    return out


# ---- what a pass cannot do without ----------------------------------------------------
def work(case):
    c = case
    size = {"f16": 2, "bf16": 2, "f32": 4}
    row = c["hkv"] * (_row(c["k_fmt"], c["d"]) + _row(c["v_fmt"], c["d"]))
    if c["op"] in ("decode", "prompt"):
        held = seen = rows = 0
        for n, length in _lens(c):
            few, low, end = _visible(length - n, length, c["window"], c["sinks"])
            held += few + max(0, end - low) if n else 0
            rows += n * c["hq"]
            for p in range(max(0, length - n), length):
                few, low, end = _visible(p, p + 1, c["window"], c["sinks"])
                seen += few + end - low
        return {"bytes": held * row + rows * (c["d"] * (2 + size[c["out"]]) + 4) + 4 * len(_lens(c)),
                "flops": 4 * seen * c["hq"] * c["d"]}
    page = c["page"]
    lens, rows, width, new = _held(c)
    refs = 4 * c["pages"]
    if c["op"] == "extend":
        # lengths, counts and the new rows; the reference counts are searched for free pages
        tokens, fresh = sum(new), sum(-(-(n + m) // page) - -(-n // page) for n, m in zip(lens, new))
        return {"bytes": refs + 16 * tokens + 12 * fresh + 16 * len(lens), "flops": 0}
    if c["op"] == "fork":
        far = (c["far"] + c["far"] // 4) // 2
        return {"bytes": refs + c["forks"] * (8 * (far // page) + c["layers"] * row * page), "flops": 0}
    held = {p for r in rows for p in r}
    moved = sum(1 for p in held if p >= len(held))
    return {"bytes": 2 * moved * c["layers"] * row * page + 2 * refs + 8 * len(held), "flops": 0}


# ---- the definitions in 64 bits -------------------------------------------------------
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


def _exact_attention(c, s):
    page, group = c["page"], c["hq"] // c["hkv"]
    o = torch.zeros(s["query"].shape, device="cuda", dtype=torch.float64)
    lse = torch.full(o.shape[:2], -math.inf, device="cuda", dtype=torch.float64)
    first = 0
    for b, (n, length) in enumerate(s["seqs"]):
        pages = -(-length // page)
        pos = torch.arange(length - n, length, device="cuda")
        t = torch.arange(pages * page, device="cuda")[:length]
        for h in range(c["hkv"] if n and length else 0):
            at = s["table"][b, :pages].clamp(min=0).long()  # (what names no page is hidden from every query)
            k, v = (_values64(c[x + "_fmt"], [p[at, h].flatten(0, 1)[:length] for p in s[x + "_planes"]], s["sign"])
                    for x in ("k", "v"))
            for i0 in range(0, n, 2048):
                i1 = min(n, i0 + 2048)
                end = max(1, length - n + i1)
                low = max(0, length - n + i0 - c["window"]) if c["window"] and c["sinks"] == 0 else 0
                hide = t[low:end] > pos[i0:i1, None]
                if c["window"]:
                    hide |= (t[low:end] <= pos[i0:i1, None] - c["window"]) & (t[low:end] >= c["sinks"])
                for q in range(h * group, (h + 1) * group):
                    z = s["query"][first + i0:first + i1, q].double() @ k[low:end].T * s["scale"]
                    if c["cap"]:
                        z = c["cap"] * torch.tanh(z / c["cap"])
                    z = z.masked_fill(hide, -math.inf)
                    lse[first + i0:first + i1, q] = torch.logsumexp(z, -1)
                    o[first + i0:first + i1, q] = torch.nan_to_num(torch.softmax(z, -1)) @ v[low:end]
        first += n
    return o.view(-1, c["d"]), lse.view(-1)


def _exact_pool(c, s):
    """The page tables' operators, entry by entry, on the host; pages copied one at a time."""
    page = c["page"]
    table, lens, refs = s["table"].tolist(), s["lens"].tolist(), s["refs"].tolist()
    planes = _planes(s)
    out = {}

    def pages_of(b, n=None):
        return range(-(-(lens[b] if n is None else n) // page))

    def drop(b, j):
        if table[b][j] >= 0:
            refs[table[b][j]] -= 1
        table[b][j] = -1

    def copy(a, b, rows):
        for p in planes:
            p[b, :, :rows] = p[a, :, :rows]

    def extend(new):
        wanted, copies = [], []
        for b, n in enumerate(new):
            end = max(0, lens[b] + n)
            low = (lens[b] if n > 0 else end) - c["window"] + 1 if c["window"] else 0
            for j in pages_of(b):
                if j >= -(-end // page) or ((j + 1) * page <= low and j * page >= c["sinks"]):
                    drop(b, j)
        for b, n in enumerate(new):
            if n > 0 and lens[b] % page and refs[table[b][lens[b] // page]] > 1:
                wanted.append((b, lens[b] // page, table[b][lens[b] // page]))
            if n > 0:
                wanted += [(b, j, -1) for j in range(-(-lens[b] // page), -(-(lens[b] + n) // page))]
        free = (p for p in range(len(refs)) if refs[p] == 0)
        given = [(b, j, old, next(free)) for b, j, old in wanted]
        for b, j, old, p in given:
            table[b][j] = p
            refs[p] += 1
            if old >= 0:
                refs[old] -= 1
                copies.append((old, p, lens[b] % page))
        for a, b, rows in copies:
            copy(a, b, rows)
        starts, slots, pos = [0], [], []
        for b, n in enumerate(new):
            for i in range(max(0, n)):
                at = lens[b] + i
                pos.append(at)
                slots.append(table[b][at // page] * page + at % page)
            starts.append(len(pos))
            lens[b] = max(0, lens[b] + n)
        pad = s["most"] - len(pos)
        return starts, slots + [-1] * pad, pos + [0] * pad

    if c["op"] == "extend":
        starts, slots, pos = extend(s["new"].tolist())
        out["new"] = (torch.tensor(starts, dtype=torch.int32), torch.tensor(slots), torch.tensor(pos))
        if c["trim"]:
            extend(s["back"].tolist())
    elif c["op"] == "fork":
        pairs = list(zip(s["src"].tolist(), s["dst"].tolist()))
        rows = [(d, lens[b] if b >= 0 else 0, [table[b][j] for j in pages_of(b)] if b >= 0 else []) for b, d in pairs]
        for _, _, r in rows:
            for p in r:
                refs[p] += 1
        for d, _, _ in rows:
            for j in pages_of(d):
                drop(d, j)
        free = [p for p in range(len(refs)) if refs[p] == 0]
        for d, n, r in rows:
            if n % page:
                p = free.pop(0)
                copy(r[-1], p, n % page)
                refs[r[-1]] -= 1
                refs[p] = 1
                r[-1] = p
            table[d] = r + [-1] * (len(table[d]) - len(r))
            lens[d] = n
    else:
        live = sum(1 for n in refs if n)
        ids = [p if n else -1 for p, n in enumerate(refs)]
        holes = iter([p for p in range(live) if not refs[p]])
        for p in range(live, len(refs)):
            if refs[p]:
                ids[p] = next(holes)
                copy(p, ids[p], page)
                refs[ids[p]], refs[p] = refs[p], 0
        for b in range(len(lens)):
            for j in pages_of(b):
                if table[b][j] >= 0:
                    table[b][j] = ids[table[b][j]]
        out["moved"] = (torch.tensor(ids, dtype=torch.int32), torch.tensor([live], dtype=torch.int32))
    return {"table": torch.tensor(table, dtype=torch.int32), "lens": torch.tensor(lens, dtype=torch.int32),
            "refs": torch.tensor(refs, dtype=torch.int32), "planes": planes, **out}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] not in ("decode", "prompt"):
        return _exact_pool(case, s)
    return _exact_attention(case, s)
