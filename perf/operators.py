"""What the paged key/value cache and the attention over it are measured on.

Four operators, each in its plain form (elementary torch operations in 32 bits) and as
the library's call:

* write      -- the new tokens' keys and values into their pages (kept as bf16, or in 8
                bits with one fp32 scale for each token and head);
* read       -- cached tokens back as bf16 rows ("store" is write, then read: a cache in 8
                bits is looked at through what it stands for);
* attention  -- a chunk of new tokens of each sequence (one token each when decoding)
                over its pages, causal by position, query heads shared by groups;
* window     -- the same with a sliding window and a few first tokens that stay visible.

"step" is write, then attention: what one layer of a serving step does with its cache.

A batch is `starts` [seqs + 1] (the rows of a sequence among the new tokens), `lens`
[seqs] (its length, the new tokens included) and `pages` [seqs, pages per sequence].
New token i of a sequence with `new` of them is at position len - new + i; a row whose
position is negative (a released slot of a fixed batch has length 0) is not stored,
reads back as zeros and attends to nothing: its output is zero.
"""
import functools
import math
import random

import numpy as np
import torch

own = False

#: Largest magnitude of an 8-bit code.
TOP = {"int8": 127.0, "fp8": 448.0}
DTYPE = {"bf16": torch.bfloat16, "int8": torch.int8, "fp8": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "int8": 1, "fp8": 1}


def _case(name, op, **v):
    base = dict(seqs=1, new_lo=1, new_hi=1, len_lo=1, len_hi=1, released=0, heads=32, kv_heads=32, dim=128, page=16,
                format="bf16", layout="split", window=0, sinks=0, salt=1)
    assert not set(v) - set(base)
    return {"name": name, "op": op, **base, **v}


def listed():
    return [
        # one layer's new keys and values of a 64-request decode batch (4096-wide projection)
        _case("write_decode_bf16", "write", seqs=64, len_lo=40, len_hi=200),
        # 16 prefill requests of 1056 tokens stored in 8 bits and handed back (a prefix moved to another place)
        _case("store_prefill_fp8", "store", seqs=16, new_lo=1056, new_hi=1056, len_lo=1056, len_hi=1056, format="fp8", page=32),
        # a long conversation's cache read back whole, to be kept elsewhere
        _case("read_long_int8", "read", seqs=2, new_lo=30011, new_hi=32768, len_lo=30011, len_hi=32768, kv_heads=8, format="int8",
              layout="heads", page=64),
        # the smallest decode: one request, where latency counts
        _case("decode_one", "attention", len_lo=777, len_hi=777),
        # 64 decoding requests of every age, a head of keys for each query head
        _case("decode_mha_bf16", "attention", seqs=64, len_lo=17, len_hi=4095),
        # 256 decode slots, half of them released; shared heads, 8-bit cache in a joint pool
        _case("decode_gqa_int8", "attention", seqs=256, len_lo=500, len_hi=4001, released=128, heads=64, kv_heads=8, format="int8",
              layout="joint", page=64),
        # chunked prefill: ragged chunks over long cached contexts, 8-bit cache
        _case("chunk_fp8", "attention", seqs=4, new_lo=300, new_hi=512, len_lo=5000, len_hi=8705, kv_heads=8, format="fp8", page=32),
        # prefill of 16 requests of 1024 visual and 32 text tokens
        _case("prefill_bf16", "attention", seqs=16, new_lo=1056, new_hi=1056, len_lo=1056, len_hi=1056),
        # one long prompt at once, shared heads, single-token pages in shuffled order
        _case("prefill_long", "attention", new_lo=8191, new_hi=8191, len_lo=8191, len_hi=8191, kv_heads=8, page=1),
        # chunks of long inputs under a window of 4096 with 4 first tokens kept
        _case("window_chunk", "attention", seqs=2, new_lo=1000, new_hi=1024, len_lo=20000, len_hi=32768, kv_heads=8, window=4096, sinks=4,
              page=64),
        # decoding far into long inputs under a window
        _case("window_decode", "attention", seqs=32, len_lo=3000, len_hi=32768, kv_heads=8, window=2048, sinks=16, layout="heads", page=128),
        # a step of a mixed batch (some requests decode, others have a chunk), small heads, stored and attended
        _case("step_mixed_int8", "step", seqs=33, new_lo=1, new_hi=777, len_lo=900, len_hi=3001, released=3, heads=28, kv_heads=4, dim=64,
              format="int8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    while True:
        op = rng.choice(["write", "store", "read", "attention", "attention", "attention", "attention", "step", "step"])
        dim = rng.choice([64, 128, 128])
        kv_heads = rng.choice([1, 2, 3, 4, 8, 8, 16, 32])
        heads = kv_heads * rng.choice([g for g in (1, 1, 2, 3, 4, 5, 7, 8, 16) if g * kv_heads <= 64])
        seqs = _log(rng, 1, 256)
        shape = rng.choice(["decode", "few", "chunk", "ragged"])
        hi = {"decode": 1, "few": rng.randint(2, 8), "chunk": _log(rng, 16, 4096), "ragged": _log(rng, 2, 2048)}[shape]
        lo = 1 if shape == "ragged" else hi
        longest = max(hi, _log(rng, 8, 32768))
        least = max(1, min(longest, int(longest * rng.uniform(0.05, 1.0))))
        if op == "read":
            hi = longest
            lo = least
        window = rng.choice([0, 0, _log(rng, 1, 4096)])
        c = dict(op=op, seqs=seqs, new_lo=lo, new_hi=hi, len_lo=least, len_hi=longest,
                 released=rng.choice([0, 0, rng.randint(0, seqs // 2)]), heads=heads, kv_heads=kv_heads, dim=dim,
                 page=rng.choice([1, 8, 16, 16, 24, 32, 64, 128]), format="bf16" if op == "write" else rng.choice(["bf16", "int8", "fp8"]),
                 layout=rng.choice(["split", "joint", "heads"]), window=window if op in ("attention", "step") else 0,
                 sinks=rng.choice([0, 1, 4, 16]) if window else 0, salt=rng.randrange(1 << 20))
        cells = seqs * longest * kv_heads * dim        # the plain form pads each sequence to the longest
        scores = seqs * hi * heads * longest if op in ("attention", "step") else 0
        w = work(c)
        if cells <= 1 << 30 and scores <= 1 << 31 and w["bytes"] <= 1.0e9 and w["flops"] <= 5.4e11:
            return c


def _lengths(case):
    """(new tokens, length) of each sequence: ragged over the logarithm, by the case alone."""
    rng = random.Random("%(salt)s %(seqs)s %(len_hi)s %(new_hi)s" % case)
    lens = [_log(rng, case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])]
    if case["op"] == "read":
        new = list(lens)
    else:
        new = [_log(rng, case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
        lens = [max(a, b) for a, b in zip(lens, new)]
    for s in rng.sample(range(case["seqs"]), case["released"]):
        lens[s] = 0
        new[s] = min(new[s], 1)
    return new, lens


def work(case):
    new, lens = _lengths(case)
    rows = sum(new)
    kv, dim, size = case["kv_heads"], case["dim"], SIZE[case["format"]]
    cell = kv * (dim * size + (4 if size == 1 else 0))     # a token's keys (or values) in the cache
    given = kv * dim * 2                                   # the same as bf16 rows
    stored = sum(min(n, m) for n, m in zip(new, lens))
    move = 2 * stored * (cell + given)
    tables = 4 * (2 * case["seqs"] + 1 + sum(-(-m // case["page"]) for m in lens))
    if case["op"] in ("write", "read"):
        return {"bytes": move + tables, "flops": 0}
    if case["op"] == "store":
        return {"bytes": 2 * move + tables, "flops": 0}
    pairs = seen = 0
    window, sinks = case["window"], case["sinks"]
    for n, m in zip(new, lens):
        p = np.arange(max(0, m - n), m, dtype=np.int64)
        if not p.size:
            continue
        if window:
            first = np.maximum(0, p - window + 1)
            pairs += int((p + 1 - first + np.minimum(sinks, first)).sum())
            seen += int(m - first[0] + min(sinks, first[0]))
        else:
            pairs += int((p + 1).sum())
            seen += m
    wide = 2 * rows * case["heads"] * dim * 2              # queries in, outputs out
    total = wide + 2 * seen * cell + tables
    if case["op"] == "step":
        total += move                                      # what was just written is read from the cache again
    return {"bytes": total, "flops": 4 * dim * case["heads"] * pairs}


# ------------------------------------------------------------------ inputs


def _quantise(x, fmt):
    """The codes and scales of vectors x [..., dim]: scale = largest magnitude / TOP, code = x / scale to the nearest (ties to even)."""
    x = x.float()
    top = torch.full((), TOP[fmt], device=x.device)
    scale = x.abs().amax(-1) / top
    step = torch.where(scale > 0, scale, torch.ones_like(scale))
    code = (x / step[..., None]).clamp(-TOP[fmt], TOP[fmt])
    return (code.round() if fmt == "int8" else code).to(DTYPE[fmt]), scale


def _blank(n, page, kv, dim, layout, dtype, dev):
    """Key and value pools [pages, page size, heads, dim] in one of three layouts of memory."""
    if layout == "joint":
        pool = torch.zeros((n, 2, page, kv, dim), dtype=dtype, device=dev)
        return pool[:, 0], pool[:, 1]
    if layout == "heads":
        return tuple(torch.zeros((n, kv, page, dim), dtype=dtype, device=dev).transpose(1, 2) for _ in range(2))
    return tuple(torch.zeros((n, page, kv, dim), dtype=dtype, device=dev) for _ in range(2))


def _inputs(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    new, lens = _lengths(case)
    page, kv, dim, fmt = case["page"], case["kv_heads"], case["dim"], case["format"]
    per = [-(-m // page) for m in lens]
    wide, total = max(1, max(per)), sum(per) + 3
    order = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    table = torch.full((case["seqs"], wide), -1, dtype=torch.int32)
    at = torch.cumsum(torch.tensor([0] + per), 0)
    have = torch.arange(wide)[None, :] < torch.tensor(per)[:, None]
    table[have] = order.cpu()[: int(at[-1])]
    rows = sum(new)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)

    lift = 1 + 3 * (torch.rand(kv, dim, generator=gen, device=dev) < 0.03).to(torch.bfloat16)   # a few strong key channels
    s = {"lens": torch.tensor(lens, dtype=torch.int32, device=dev), "pages": table.to(dev),
         "starts": torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32).to(dev)}
    k_pool, v_pool = _blank(total, page, kv, dim, case["layout"], DTYPE[fmt], dev)
    k_scale = v_scale = None
    if fmt != "bf16":   # scales in the order of the pools' heads: [pages, heads, page size] in memory
        k_scale, v_scale = (torch.zeros((total, kv, page), device=dev).transpose(1, 2) for _ in range(2))
    if case["op"] not in ("write", "store"):   # what earlier steps have left in the cache
        for pool, scale, gain in ((k_pool, k_scale, lift), (v_pool, v_scale, None)):
            x = normal(total, page, kv, dim)
            if gain is not None:
                x *= gain
            if fmt == "bf16":
                pool.copy_(x)
            else:
                code, sc = _quantise(x, fmt)
                pool.copy_(code)
                scale.copy_(sc)
            del x
    s.update(k_pool=k_pool, v_pool=v_pool, k_scale=k_scale, v_scale=v_scale)
    if case["op"] in ("write", "store", "step"):
        s["k"], s["v"] = normal(rows, kv, dim) * lift, normal(rows, kv, dim)
    if case["op"] in ("attention", "step"):
        s["q"] = normal(rows, case["heads"], dim)
        s["out"] = torch.empty_like(s["q"])
    if case["op"] in ("read", "store"):
        s["k_back"], s["v_back"] = (torch.empty((rows, kv, dim), dtype=torch.bfloat16, device=dev) for _ in range(2))
    s["case"], s["max_new"] = case, max(new)
    return s


@functools.lru_cache(None)
def _context():
    import adapter_sgmv_bgmv_gb300 as L
    return L, L.Context(0, max_rows=1024)


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        L, ctx = _context()
        s["cache"] = L.KvCache(ctx, s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])
        s["batch"] = L.KvBatch(s["starts"], s["lens"], s["pages"], max_new=s["max_new"])
    return s


# ------------------------------------------------------------------ the passes


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        L, ctx = _context()
        if op in ("write", "store", "step"):
            L.lora_kv_write(ctx, s["cache"], s["batch"], s["k"], s["v"])
        if op in ("read", "store"):
            L.lora_kv_read(ctx, s["cache"], s["batch"], s["k_back"], s["v_back"])
        if op in ("attention", "step"):
            L.lora_attention(ctx, s["cache"], s["batch"], s["q"], s["out"], window=case["window"], sinks=case["sinks"])
    else:
        where = _places(s)
        if op in ("write", "store", "step"):
            _write(s, where)
        if op in ("read", "store"):
            _read(s, where)
        if op in ("attention", "step"):
            _attend(s, where, case["window"], case["sinks"])
    if op == "write":
        return {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    if op in ("read", "store"):
        return {"k": s["k_back"], "v": s["v_back"]}
    return s["out"]


def _places(s):
    """Each new row's sequence, position, page and place in the page."""
    rows = (s["k"] if "k" in s else s["q"] if "q" in s else s["k_back"]).shape[0]
    row = torch.arange(rows, device=s["lens"].device)
    seq = torch.searchsorted(s["starts"][1:], row.to(torch.int32), right=True)
    pos = s["lens"][seq] - s["starts"][seq + 1] + row
    page = s["pages"][seq, (pos.clamp(min=0) // s["k_pool"].shape[1])].long()
    return seq, pos, page, pos % s["k_pool"].shape[1]


def _write(s, where):
    _, pos, page, cell = where
    live = torch.nonzero(pos >= 0)[:, 0]
    for x, pool, scale in ((s["k"], s["k_pool"], s["k_scale"]), (s["v"], s["v_pool"], s["v_scale"])):
        if scale is None:
            pool[page[live], cell[live]] = x[live]
        else:
            code, sc = _quantise(x[live], s["case"]["format"])
            pool.view(torch.int8)[page[live], cell[live]] = code.view(torch.int8)
            scale[page[live], cell[live]] = sc


def _read(s, where):
    _, pos, page, cell = where
    page = page.clamp(min=0)
    for pool, scale, out in ((s["k_pool"], s["k_scale"], s["k_back"]), (s["v_pool"], s["v_scale"], s["v_back"])):
        x = pool.view(torch.int8)[page, cell].view(pool.dtype).float()
        if scale is not None:
            x = x * scale[page, cell][..., None]
        out.copy_(torch.where((pos >= 0)[:, None, None], x, torch.zeros((), device=x.device)))


def _attend(s, where, window, sinks):
    seq, pos, _, _ = where
    q, starts, lens = s["q"], s["starts"].long(), s["lens"].long()
    heads, dim, kv, most = q.shape[1], q.shape[2], s["k_pool"].shape[2], s["max_new"]
    page = s["pages"].clamp(min=0).long()
    seqs = page.shape[0]

    def whole(pool, scale):
        """[seqs, heads, length, dim] of every sequence, padded to the longest."""
        x = pool.view(torch.int8)[page].view(pool.dtype).float()
        if scale is not None:
            x = x * scale[page][..., None]
        return x.flatten(1, 2).transpose(1, 2)

    at = torch.arange(most, device=q.device)
    index = (starts[:-1, None] + at).clamp(max=q.shape[0] - 1)
    x = q[index].float().view(seqs, most, kv, heads // kv, dim).permute(0, 2, 3, 1, 4).reshape(seqs, kv, -1, dim)
    p = x @ whole(s["k_pool"], s["k_scale"]).transpose(2, 3)
    p = p.view(seqs, kv, heads // kv, most, -1).mul_(1 / math.sqrt(dim))
    here = (lens - (starts[1:] - starts[:-1]))[:, None] + at
    j = torch.arange(p.shape[-1], device=q.device)
    seen = j <= here[..., None]
    if window:
        seen &= (j > here[..., None] - window) | (j < sinks)
    seen = seen[:, None, None]
    p = p.masked_fill_(~seen, -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = p.sum(-1, keepdim=True)
    y = p.view(seqs, kv, -1, p.shape[-1]) @ whole(s["v_pool"], s["v_scale"])
    y = y.view(seqs, kv, heads // kv, most, dim) / torch.where(total > 0, total, torch.ones_like(total))
    y = y.permute(0, 3, 1, 2, 4).reshape(seqs, most, heads, dim)
    s["out"].copy_(y[seq, torch.arange(q.shape[0], device=q.device) - starts[seq]])


# ------------------------------------------------------------------ 64 bits


def _wide_codes(x, fmt):
    """What vectors x [n, heads, dim] read back as after being stored in 8 bits, in 64 bits."""
    x = x.double()
    scale = x.abs().amax(-1, keepdim=True) / TOP[fmt]
    z = torch.where(scale > 0, x / scale.clamp(min=1e-300), torch.zeros_like(x))
    if fmt == "int8":
        return z.round() * scale
    # e4m3: three bits after the leading one, exponents from 2^-6 down to multiples of 2^-9
    _, e = torch.frexp(z)
    ulp = torch.ldexp(torch.ones_like(z), (e - 1).clamp(min=-6) - 3)
    return (z / ulp).round() * ulp * scale


def _rows_of(s, a, name, upto):
    """Positions [0, upto) of sequence a from the pool, in 64 bits."""
    p = s["pages"][a].long()
    n = s["k_pool"].shape[1]
    j = torch.arange(upto, device=p.device)
    pool, scale = s[name + "_pool"], s[name + "_scale"]
    x = pool.view(torch.int8)[p[j // n], j % n].view(pool.dtype).float().double()
    return x if scale is None else x * scale[p[j // n], j % n].double()[..., None]


def exact(case, seed):
    s = _inputs(case, seed)
    new, lens = _lengths(case)
    op, fmt, dim = case["op"], case["format"], case["dim"]
    start = np.concatenate([[0], np.cumsum(new)]).tolist()
    if op == "write":
        out = {x: s[x].double() for x in ("k_pool", "v_pool")}
        page = s["pages"].cpu().numpy()
        n = case["page"]
        for name in ("k", "v"):
            x = s[name].double()
            for a in range(case["seqs"]):
                for i in range(new[a]):
                    pos = lens[a] - new[a] + i
                    if pos < 0:
                        continue
                    at = (int(page[a, pos // n]), pos % n)
                    out[name + "_pool"][at] = x[start[a] + i]
        return out
    if op in ("read", "store"):
        out = {}
        for name in ("k", "v"):
            y = torch.zeros(s[name + "_back"].shape, dtype=torch.float64, device="cuda")
            for a in range(case["seqs"]):
                got = min(new[a], lens[a])
                if got:
                    y[start[a + 1] - got:start[a + 1]] = (_rows_of(s, a, name, lens[a])[lens[a] - got:] if op == "read" else
                                                          s[name][start[a + 1] - got:start[a + 1]].double() if fmt == "bf16" else
                                                          _wide_codes(s[name][start[a + 1] - got:start[a + 1]], fmt))
            out[name] = y
        return out
    if work(case)["flops"] > 2e12:
        return None
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = case["heads"] // case["kv_heads"]
    for a in range(case["seqs"]):
        m, got = lens[a], min(new[a], lens[a])
        if not got:
            continue
        k, v = _rows_of(s, a, "k", m), _rows_of(s, a, "v", m)
        rows = slice(start[a + 1] - got, start[a + 1])
        if op == "step":
            for x, name in ((k, "k"), (v, "v")):
                x[m - got:] = s[name][rows].double() if fmt == "bf16" else _wide_codes(s[name][rows], fmt)
        pos = torch.arange(m - got, m, device="cuda")[:, None]
        j = torch.arange(m, device="cuda")[None, :]
        hidden = j > pos
        if case["window"]:
            hidden |= (j <= pos - case["window"]) & (j >= case["sinks"])
        for h in range(case["heads"]):
            z = s["q"][rows, h].double() @ k[:, h // group].T / math.sqrt(dim)
            y[rows, h] = torch.softmax(z.masked_fill_(hidden, -math.inf), -1) @ v[:, h // group]
    return y
