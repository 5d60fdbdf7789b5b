"""What the operators around the paged cache are measured on: those that fill it, those that
manage its pages, and attention that reads a part of it.

Each in its plain form (elementary torch operations in 32 bits) and as the library's calls:

* rope     -- norms of each head's queries and keys, then the rotation by position;
* append   -- the same, with keys and values stored in their cells in the same pass (8-bit
              caches are looked at through what they read back as);
* roll     -- drafted tokens that were refused are taken back and the next ones get their pages;
* beam     -- the beams of the last step end, others fork from their parents, grow by a token,
              and what they would share while writing it is copied in every layer;
* fork     -- many requests start from one long prefix;
* compact  -- requests end, and the pages that are left move to the front of the pool, in
              every layer;
* bounds   -- the smallest and largest keys of the pages that new tokens touched;
* sparse   -- bounds, then a choice of pages for every new token and key head by a cheap
              score, then attention over the chosen pages.

A batch is `starts` [seqs + 1] (the rows of a sequence among the new tokens), `lens` [seqs]
(its length, the new tokens included) and `pages` [seqs, pages per sequence]; `refs` [pages of
the pool] counts the sequences that hold a page.  A row of a released slot (length 0) has no
position: its outputs are zeros.
"""
import functools
import math
import random

import numpy as np
import torch

own = False

TOP = {"int8": 127.0, "fp8": 448.0}
DTYPE = {"bf16": torch.bfloat16, "int8": torch.int8, "fp8": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "int8": 1, "fp8": 1}
EPS = 1e-6

_ROWS = dict(seqs=1, new_lo=1, new_hi=1, len_lo=1, len_hi=1, released=0, heads=32, kv_heads=8, dim=128, page=16, format="bf16", salt=1)
_ROPE = dict(_ROWS, rot=128, interleaved=False, norm=True, theta=10000.0)
_SPARSE = dict(_ROWS, blocks=32, first=1, last=1)
_PAGES = dict(seqs=1, len_lo=1, len_hi=1, page=16, pool=1024, cols=64, layers=1, kv_heads=8, dim=128, grow=1, forks=1, ended=0, salt=1)
_BASE = {"rope": _ROPE, "append": _ROPE, "bounds": _SPARSE, "sparse": _SPARSE, "roll": _PAGES, "beam": _PAGES, "fork": _PAGES, "compact": _PAGES}


def _case(name, op, **v):
    assert not set(v) - set(_BASE[op])
    return {"name": name, "op": op, **_BASE[op], **v}


def listed():
    return [
        # one request decodes: queries and keys of one token, where latency counts
        _case("rope_one", "rope", len_lo=777, len_hi=777),
        # prefill of 16 requests of 1056 tokens, a key head for each query head, no norms
        _case("rope_prefill", "rope", seqs=16, new_lo=1056, new_hi=1056, len_lo=1056, len_hi=1056, kv_heads=32, norm=False),
        # 256 decode slots, half of them released: rotated and stored in 8 bits
        _case("append_decode_int8", "append", seqs=256, len_lo=500, len_hi=4001, released=128, heads=64, kv_heads=8, format="int8", page=64,
              theta=500000.0),
        # one long prompt, shared heads, half of each head rotated in neighbouring pairs, single-token pages
        _case("append_prompt", "append", new_lo=8191, new_hi=8191, len_lo=8191, len_hi=8191, rot=64, interleaved=True, page=1),
        # 64 requests take back up to seven refused drafted tokens and get room for the next ones
        _case("roll_back", "roll", seqs=64, len_lo=17, len_hi=4095, pool=20000, cols=260, grow=8),
        # 16 requests with four beams each: three of them fork anew from the fourth; four layers' pools
        _case("beam_step", "beam", seqs=64, len_lo=40, len_hi=2000, pool=2400, cols=128, layers=4, forks=48),
        # 200 requests that start from one prefix of 30,011 tokens
        _case("fork_prefix", "fork", seqs=201, len_lo=30011, len_hi=30011, pool=65536, cols=2048, forks=200),
        # half of 128 long requests have ended; the rest move to the front of a pool of 24,000 pages in four layers
        _case("compact_pool", "compact", seqs=128, len_lo=500, len_hi=4001, pool=24000, cols=251, layers=4, kv_heads=4, dim=64, ended=64),
        # bounds of 16 prompts' pages
        _case("bounds_prefill", "bounds", seqs=16, new_lo=1056, new_hi=1056, len_lo=1056, len_hi=1056, kv_heads=32, page=32),
        # one request decodes far into a long input, 32 pages of 64 tokens of it at a time
        _case("sparse_one", "sparse", len_lo=32768, len_hi=32768, page=64, blocks=32, last=2),
        # 32 requests decode in inputs of 3000 to 33,000 tokens, 8-bit cache, 64 query heads on 8
        _case("sparse_decode_int8", "sparse", seqs=32, len_lo=3000, len_hi=33000, heads=64, format="int8", page=64, blocks=48),
        # eight requests verify up to eight drafted tokens each, small pages
        _case("sparse_draft", "sparse", seqs=8, new_lo=2, new_hi=8, len_lo=9000, len_hi=30000, heads=28, kv_heads=4, page=16, blocks=128, first=4,
              last=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    while True:
        op = rng.choice(["rope", "append", "append", "roll", "beam", "fork", "compact", "bounds", "sparse", "sparse", "sparse", "sparse"])
        c = {"op": op, **_BASE[op], "salt": rng.randrange(1 << 20), "page": rng.choice([1, 8, 16, 16, 24, 32, 64, 128]), "dim": rng.choice([64, 128, 128])}
        c["kv_heads"] = rng.choice([1, 2, 3, 4, 8, 8, 16, 32])
        if op in ("roll", "beam", "fork", "compact"):
            c["seqs"] = _log(rng, 2, 512)
            c["len_hi"] = _log(rng, 8, 32768)
            c["len_lo"] = max(1, int(c["len_hi"] * rng.uniform(0.05, 1.0)))
            c["grow"] = rng.randint(1, 12)
            c["cols"] = -(-(c["len_hi"] + 12) // c["page"]) + rng.choice([0, 0, 3])
            c["layers"] = rng.choice([1, 1, 2, 3, 8]) if op in ("beam", "compact") else 1
            c["forks"] = rng.randint(1, c["seqs"] - 1)
            c["ended"] = rng.randint(1, max(1, c["seqs"] * 3 // 4))
            pages = sum(-(-(n + 12) // c["page"]) for n in _lengths(c)[1])
            c["pool"] = int(pages * rng.uniform(1.05, 2.0)) + 2 * c["seqs"] + 8
            data = c["pool"] * c["page"] * c["kv_heads"] * c["dim"] * 4 * c["layers"] if op in ("beam", "compact") else 0
            if data <= 3 << 30 and c["pool"] <= 1 << 20 and c["seqs"] * c["cols"] <= 1 << 22 and work(c)["bytes"] <= 5.5e8:
                return c
            continue
        c["heads"] = c["kv_heads"] * rng.choice([g for g in (1, 1, 2, 3, 4, 5, 7, 8, 16) if g * c["kv_heads"] <= 64])
        c["seqs"] = _log(rng, 1, 256)
        longest = _log(rng, 8, 32768)
        hi = {"decode": 1, "few": rng.randint(2, 8), "chunk": _log(rng, 16, 8192)}[rng.choice(["decode", "decode", "few"] + ["chunk"] * (op != "sparse"))]
        c["new_hi"], c["new_lo"] = hi, rng.choice([1, hi])
        c["len_hi"] = max(hi, longest)
        c["len_lo"] = max(1, min(c["len_hi"], int(c["len_hi"] * rng.uniform(0.05, 1.0))))
        c["released"] = rng.choice([0, 0, rng.randint(0, c["seqs"] // 2)])
        c["format"] = rng.choice(["bf16", "bf16", "int8", "fp8"]) if op != "rope" else "bf16"
        if op in ("rope", "append"):
            c["rot"] = rng.choice([c["dim"], c["dim"], c["dim"] // 2, c["dim"] // 4, 0])
            c["interleaved"], c["norm"] = rng.random() < 0.4, rng.random() < 0.6
            c["theta"] = rng.choice([1e4, 5e5, 1e6])
        else:
            c["blocks"] = _log(rng, 2, 256)
            c["first"] = rng.randint(0, min(4, c["blocks"] - 1))
            c["last"] = rng.randint(1, min(4, c["blocks"] - c["first"]))
        new, lens = _lengths(c)
        rows, wide, cols = sum(new), c["kv_heads"] * c["dim"], -(-max(lens) // c["page"])
        pool = sum(-(-n // c["page"]) for n in lens) * c["page"] * wide if op != "rope" else 0
        if op in ("sparse", "bounds") and max(max(lens) * c["seqs"], rows * c["page"], rows * min(cols, c["blocks"]) * c["page"] * (op == "sparse")) * wide > 6e8:
            continue
        if op == "sparse" and max(rows * c["heads"] * cols, c["seqs"] * cols * 2 * wide) > 3e8:
            continue
        if pool <= 1 << 30 and rows * c["heads"] * c["dim"] <= 2 << 27 and work(c)["bytes"] <= 5.5e8:
            return c


def _lengths(case):
    """(new tokens, length) of each sequence: ragged over the logarithm, by the case alone."""
    rng = random.Random("%(salt)s %(seqs)s %(len_hi)s %(op)s" % case)
    lens = [_log(rng, case["len_lo"], case["len_hi"]) for _ in range(case["seqs"])]
    if "new_hi" not in case:
        return None, lens
    new = [_log(rng, case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
    lens = [max(a, b) for a, b in zip(lens, new)]
    for s in rng.sample(range(case["seqs"]), case["released"]):
        lens[s] = 0
        new[s] = min(new[s], 1)
    return new, lens


def work(case):
    op, page = case["op"], case["page"]
    new, lens = _lengths(case)
    used = [-(-n // page) for n in lens]
    if op in ("roll", "beam", "fork", "compact"):
        cell = 2 * case["kv_heads"] * case["dim"] * 2 * case["layers"]
        if op == "roll":       # lengths, what is kept and grown, what was got and is to be copied; the pages that come and go
            return {"bytes": 4 * (10 * case["seqs"] + 6 * case["seqs"] * case["grow"] // (2 * page)), "flops": 0}
        forked = used[0] * case["forks"] if op == "fork" else sum(used) // len(used) * case["forks"]
        if op == "fork":       # the ended ones' pages and the new ones': table and counts
            return {"bytes": 4 * 4 * 2 * forked, "flops": 0}
        if op == "beam":       # also half a page of each fork, in each layer
            return {"bytes": 4 * 4 * 2 * forked + 2 * cell * case["forks"] * page // 2, "flops": 0}
        left = sum(used) * (case["seqs"] - case["ended"]) // case["seqs"]
        moved = left * (case["pool"] - left) // case["pool"]
        return {"bytes": 4 * (2 * case["pool"] + 2 * sum(used)) + 2 * cell * page * moved, "flops": 0}
    rows, kv, dim, size = sum(new), case["kv_heads"], case["dim"], SIZE[case["format"]]
    cell = kv * (dim * size + (4 if size == 1 else 0))     # a token's keys (or values) in the cache
    given = kv * dim * 2                                   # the same as bf16 rows
    wide = rows * case["heads"] * dim * 2                  # the queries
    tables = 4 * (2 * case["seqs"] + 1)
    live = sum(min(n, m) for n, m in zip(new, lens))
    if op == "rope":
        return {"bytes": 2 * (wide + rows * given) + tables, "flops": 10 * rows * (case["heads"] + kv) * dim}
    tables += 4 * sum(-(-m // page) - (m - min(n, m)) // page for n, m in zip(new, lens))
    if op == "append":
        back = 2 * live * (cell + given) if size == 1 else 0
        return {"bytes": 2 * wide + 2 * live * (cell + given) + back + tables, "flops": 10 * rows * (case["heads"] + kv) * dim}
    touched = sum(-(-m // page) - (m - min(n, m)) // page for n, m in zip(new, lens) if m)
    cells = sum(m - (m - min(n, m)) // page * page for n, m in zip(new, lens) if m)
    code = kv * (2 * dim + 4)
    b = cells * cell + touched * code + tables
    if op == "bounds":
        return {"bytes": b, "flops": 0}
    seen = sum(min((min(case["blocks"], u) - 1) * page + (m - 1) % page + 1, m) for u, m in zip(used, lens) if m)
    rowwise = sum(min(n, m) * min(case["blocks"] * page, m) for n, m in zip(new, lens) if m)
    b += sum(used) * (code + 4) + 2 * wide + 2 * seen * cell + rows * kv * case["blocks"] * 4
    flops = 4 * dim * case["heads"] * rowwise + 4 * dim * case["heads"] * sum(n * u for n, u in zip(new, used))
    return {"bytes": b, "flops": flops}


# ------------------------------------------------------------------ inputs


def _codes(x, fmt):
    """The codes and scales of vectors x [..., dim]: scale = largest magnitude / TOP, code = x / scale to the nearest (ties to even)."""
    x = x.float()
    scale = x.abs().amax(-1) / torch.full((), TOP[fmt], device=x.device)
    step = torch.where(scale > 0, scale, torch.ones_like(scale))
    code = (x / step[..., None]).clamp(-TOP[fmt], TOP[fmt])
    return (code.round() if fmt == "int8" else code).to(DTYPE[fmt]), scale


def _batch(case, gen, dev):
    new, lens = _lengths(case)
    per = [-(-m // case["page"]) for m in lens]
    total = sum(per) + 3
    order = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    table = torch.full((case["seqs"], max(1, max(per))), -1, dtype=torch.int32, device=dev)
    have = torch.arange(table.shape[1], device=dev)[None, :] < torch.tensor(per, device=dev)[:, None]
    table[have] = order[: sum(per)]
    return {"lens": torch.tensor(lens, dtype=torch.int32, device=dev), "pages": table, "max_new": max(new), "rows": sum(new),
            "starts": torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32).to(dev)}, total


def _rows_inputs(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    s, total = _batch(case, gen, dev)
    heads, kv, dim, page, fmt, rows = case["heads"], case["kv_heads"], case["dim"], case["page"], case["format"], s["rows"]

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=gen, device=dev, dtype=dtype)

    lift = 1 + 3 * (torch.rand(kv, dim, generator=gen, device=dev) < 0.03).to(torch.bfloat16)   # a few strong key channels
    s["case"] = case
    if case["op"] in ("rope", "append"):
        qkv = normal(rows, heads + 2 * kv, dim)            # one projection's rows
        s["q"], s["k"], s["v"] = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
        s["k"] *= lift
        half = case["rot"] // 2
        s["freqs"] = (1.0 / case["theta"] ** (torch.arange(half, dtype=torch.float64, device=dev) / max(1, half))).float()
        s["q_weight"], s["k_weight"] = ((1 + 0.2 * normal(dim, dtype=torch.float32)) if case["norm"] else None for _ in range(2))
        s["q_out"] = torch.empty((rows, heads, dim), dtype=torch.bfloat16, device=dev)
        s["k_out"], s["v_out"] = (torch.empty((rows, kv, dim), dtype=torch.bfloat16, device=dev) for _ in range(2))
        if case["op"] == "rope":
            return s
    s["k_pool"], s["v_pool"] = (torch.zeros((total, page, kv, dim), dtype=DTYPE[fmt], device=dev) for _ in range(2))
    s["k_scale"] = s["v_scale"] = None
    if fmt != "bf16":
        s["k_scale"], s["v_scale"] = (torch.zeros((total, kv, page), device=dev).transpose(1, 2) for _ in range(2))
    if case["op"] == "append":
        return s
    drift = normal(total, 1, kv, dim)                      # tokens of a page are near one another
    for name, gain in (("k", lift), ("v", None)):
        x = normal(total, page, kv, dim)
        if gain is not None:
            x = (x + drift) * gain
        if fmt == "bf16":
            s[name + "_pool"].copy_(x)
        else:
            code, sc = _codes(x, fmt)
            s[name + "_pool"].copy_(code)
            s[name + "_scale"].copy_(sc)
        del x
    s["q"] = normal(rows, heads, dim)
    s["out"] = torch.empty_like(s["q"])
    s["code"], s["unit"] = torch.zeros((total, kv, 2, dim), dtype=torch.int8, device=dev), torch.zeros((total, kv), device=dev)
    if case["op"] == "sparse":   # what earlier steps have left
        s["code"].copy_(_bound_codes(_page_keys(s, torch.arange(total, device=dev)), torch.full((total,), page, device=dev), s["unit"]))
        s["sel_pages"] = torch.empty((rows, kv, case["blocks"]), dtype=torch.int32, device=dev)
        s["sel_lens"] = torch.empty((rows,), dtype=torch.int32, device=dev)
    return s


def _pages_inputs(case, seed):
    dev = torch.device("cuda")
    rng = np.random.default_rng(seed)
    seqs, cols, pool, page, op = case["seqs"], case["cols"], case["pool"], case["page"], case["op"]
    lens = np.array(_lengths(case)[1])
    children = np.zeros(0, np.int64)
    if op in ("beam", "fork"):
        order = np.arange(seqs) if op == "fork" else rng.permutation(seqs)
        children, left = order[seqs - case["forks"]:], order[:seqs - case["forks"]]
        lens[children] = 0
        parents = left[rng.integers(0, len(left), case["forks"])] if op == "beam" else np.zeros(case["forks"], np.int64)
    used = -(-lens // page)
    free = rng.permutation(pool)
    if op == "roll":
        free = np.sort(free)
    table = np.full((seqs, cols), -1, np.int64)
    have = np.arange(cols)[None, :] < used[:, None]
    table[have] = free[: used.sum()]
    refs = np.zeros(pool, np.int64)
    refs[free[: used.sum()]] = 1
    ints = torch.from_numpy(np.concatenate([lens, table.ravel(), refs]).astype(np.int32)).to(dev)
    s = {"case": case, "start": ints, "ints": ints.clone()}
    s["lens"], s["pages"], s["refs"] = s["ints"][:seqs], s["ints"][seqs:seqs + seqs * cols].view(seqs, cols), s["ints"][seqs + seqs * cols:]
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)  # noqa: E731
    if op in ("beam", "fork"):
        s["parents"], s["children"] = to(parents), to(children)
        s["grow"] = to(np.isin(np.arange(seqs), children))
    if op == "roll":
        s["all"], s["keep"], s["grow"] = to(np.arange(seqs)), to(lens), to(rng.integers(0, case["grow"] + 1, seqs))
    if op == "compact":
        s["ended"] = to(rng.permutation(seqs)[: case["ended"]])
    n = pool // 2 + 1 if op == "compact" else seqs
    s["src"], s["dst"], s["cells"], s["got"] = (torch.empty(m, dtype=torch.int32, device=dev) for m in (n, n, seqs, seqs))
    s["top"] = torch.empty(1, dtype=torch.int32, device=dev)
    if op in ("beam", "compact"):
        gen = torch.Generator(device=dev).manual_seed(seed)
        s["pools"] = torch.randn((case["layers"], 2, pool, page, case["kv_heads"], case["dim"]), generator=gen, device=dev, dtype=torch.bfloat16)
    return s


@functools.lru_cache(None)
def _context():
    import adapter_sgmv_bgmv_gb300 as L
    return L, L.Context(0, max_rows=1024)


def prepare(case, seed):
    s = _pages_inputs(case, seed) if "pool" in case else _rows_inputs(case, seed)
    if own:
        L, ctx = _context()
        if "refs" in s:
            s["table"] = L.PageTable(s["lens"], s["pages"], s["refs"], case["page"])
            if "pools" in s:
                s["caches"] = [L.KvCache(ctx, p[0], p[1]) for p in s["pools"]]
            return s
        s["batch"] = L.KvBatch(s["starts"], s["lens"], s["pages"], max_new=s["max_new"])
        if "k_pool" in s:
            s["cache"] = L.KvCache(ctx, s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"])
        if "freqs" in s:
            s["rope"] = L.HeadRope(s["freqs"], case["dim"], s["q_weight"], s["k_weight"], eps=EPS, interleaved=case["interleaved"])
        if "code" in s:
            s["cache"].attach_bounds(s["code"], s["unit"])
        if "sel_pages" in s:
            s["sel"] = L.BlockSelection(s["sel_lens"], s["sel_pages"])
    return s


# ------------------------------------------------------------------ the passes


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        L, ctx = _context()
        if op == "rope":
            L.lora_head_rope(ctx, s["rope"], s["batch"], s["q"], s["k"], s["q_out"], s["k_out"])
        if op == "append":
            L.lora_kv_write_rope(ctx, s["cache"], s["rope"], s["batch"], s["q"], s["k"], s["v"], s["q_out"])
            if case["format"] != "bf16":
                L.lora_kv_read(ctx, s["cache"], s["batch"], s["k_out"], s["v_out"])
        if op in ("bounds", "sparse"):
            L.lora_kv_bounds(ctx, s["cache"], s["batch"], s["rows"])
        if op == "sparse":
            L.lora_block_select(ctx, s["cache"], s["batch"], s["q"], s["sel"], first=case["first"], last=case["last"])
            L.lora_block_attention(ctx, s["cache"], s["sel"], s["q"], s["out"])
        if op in ("beam", "fork"):
            L.lora_pages_free(ctx, s["table"], s["children"])
            L.lora_pages_fork(ctx, s["table"], s["parents"], s["children"])
        if op == "roll":
            L.lora_pages_free(ctx, s["table"], s["all"], s["keep"])
        if op in ("roll", "beam"):
            L.lora_pages_extend(ctx, s["table"], s["grow"], s["got"], s["src"], s["dst"], s["cells"])
        if op == "beam":
            L.lora_kv_copy(ctx, s["caches"], s["src"], s["dst"], s["cells"])
        if op == "compact":
            s["ints"].copy_(s["start"])
            L.lora_pages_free(ctx, s["table"], s["ended"])
            L.lora_pages_compact(ctx, s["table"], s["src"], s["dst"], s["top"])
            L.lora_kv_copy(ctx, s["caches"], s["src"], s["dst"])
    else:
        if op in ("rope", "append"):
            _rotate(s)
        if op in ("bounds", "sparse"):
            _bounds(s)
        if op == "sparse":
            _select(s)
            _attend(s)
        if op in ("beam", "fork"):
            _free(s, s["children"], torch.zeros_like(s["children"]))
            _fork(s)
        if op == "roll":
            _free(s, s["all"], s["keep"])
        if op in ("roll", "beam"):
            _extend(s)
        if op == "beam":
            _copy(s, s["cells"])
        if op == "compact":
            s["ints"].copy_(s["start"])
            _free(s, s["ended"], torch.zeros_like(s["ended"]))
            _compact(s)
            _copy(s, None)
    if op == "rope":
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "append":
        kept = {"k": s["k_pool"], "v": s["v_pool"]} if case["format"] == "bf16" else {"k": s["k_out"], "v": s["v_out"]}
        return {"q": s["q_out"], **kept}
    if op == "bounds":
        return {"bounds": s["code"].float() * s["unit"][..., None, None]}
    if op == "sparse":
        return {"out": s["out"], "pages": s["sel_pages"], "lens": s["sel_lens"]}
    out = {"lens": s["lens"], "pages": s["pages"], "refs": s["refs"]}
    if op in ("roll", "beam"):
        out.update(got=s["got"], src=s["src"], dst=s["dst"], cells=s["cells"])
    if op == "compact":
        out.update(src=s["src"], dst=s["dst"], top=s["top"])
    if op in ("beam", "compact"):
        out["pools"] = s["pools"]
    return out


def _places(s):
    """Each row's sequence and position."""
    row = torch.arange(s["rows"], device=s["lens"].device)
    seq = torch.searchsorted(s["starts"][1:], row.to(torch.int32), right=True)
    return seq, s["lens"][seq] - s["starts"][seq + 1] + row


def _turn(x, weight, angle, interleaved):
    """One side's heads x [rows, heads, dim] in 32 bits: the norm, then the rotation by angle [rows, rot / 2] in 64 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    half = angle.shape[1]
    c, t = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = x.clone()
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    ya, yb = a * c - b * t, a * t + b * c
    a.copy_(ya)
    b.copy_(yb)
    return x


def _rotate(s):
    case = s["case"]
    seq, pos = _places(s)
    live = (pos >= 0)[:, None, None]
    angle = pos.clamp(min=0).double()[:, None] * s["freqs"].double()
    zero = torch.zeros((), device=pos.device)
    s["q_out"].copy_(torch.where(live, _turn(s["q"], s["q_weight"], angle, case["interleaved"]), zero))
    k = _turn(s["k"], s["k_weight"], angle, case["interleaved"])
    if case["op"] == "rope":
        s["k_out"].copy_(torch.where(live, k, zero))
        return
    page = s["pages"][seq, pos.clamp(min=0) // case["page"]].long()
    at = torch.nonzero(pos >= 0)[:, 0]
    page, cell = page[at], pos[at] % case["page"]
    for name, x in (("k", k), ("v", s["v"])):
        if case["format"] == "bf16":
            s[name + "_pool"][page, cell] = x[at].to(torch.bfloat16)
            continue
        code, sc = _codes(x[at], case["format"])
        s[name + "_pool"].view(torch.int8)[page, cell] = code.view(torch.int8)
        s[name + "_scale"][page, cell] = sc
        back = s[name + "_out"]
        back.zero_()
        back[at] = (code.float() * sc[..., None]).to(torch.bfloat16)


def _page_keys(s, page):
    """The keys [pages, page size, heads, dim] of some pages in 32 bits."""
    x = s["k_pool"].view(torch.int8)[page].view(s["k_pool"].dtype).float() if s["k_scale"] is not None else s["k_pool"][page].float()
    return x if s["k_scale"] is None else x * s["k_scale"][page][..., None]


def _power(top):
    """The power of two that takes numbers up to `top` to codes of up to 127: 2^(e - 6) for 2^e <= top < 2^(e + 1)."""
    e = torch.where(top > 0, torch.frexp(top)[1].clamp(min=-99), -99) - 7
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _bound_codes(x, filled, unit):
    """Codes [pages, heads, 2, dim] of the smallest and largest keys of the first `filled` cells of pages x; their units into `unit`."""
    hidden = (torch.arange(x.shape[1], device=x.device) >= filled[:, None])[..., None, None]
    lo, hi = x.masked_fill(hidden, math.inf).amin(1), x.masked_fill(hidden, -math.inf).amax(1)
    both = torch.stack([lo, hi], 2)
    unit.copy_(_power(both.abs().amax((2, 3))))
    return (both / unit[..., None, None]).round().clamp(-127, 127).to(torch.int8)


def _bounds(s):
    case = s["case"]
    seq, pos = _places(s)
    first = torch.arange(s["rows"], device=pos.device) == s["starts"][seq]
    here = torch.nonzero((pos >= 0) & (first | (pos % case["page"] == 0)))[:, 0]
    # a first row may be ahead of the sequence's positions: those with a position begin at 0
    seq, col = seq[here], pos[here] // case["page"]
    page = s["pages"][seq, col].long()
    unit = torch.empty((page.shape[0], case["kv_heads"]), device=pos.device)
    s["code"][page] = _bound_codes(_page_keys(s, page), s["lens"][seq] - col * case["page"], unit)
    s["unit"][page] = unit


def _select(s):
    case = s["case"]
    blocks, page, kv, dim = case["blocks"], case["page"], case["kv_heads"], case["dim"]
    group, most = case["heads"] // kv, s["max_new"]
    seq, pos = _places(s)
    q = s["q"].float()
    uq = _power(q.abs().amax(-1))
    cq = (q / uq[..., None]).round().clamp(-127, 127)
    table = s["pages"].clamp(min=0).long()
    b = s["code"][table].float().permute(3, 0, 2, 4, 1)                  # [2, seqs, heads, dim, pages]
    starts = s["starts"].long()
    at = (starts[:-1, None] + torch.arange(most, device=q.device)).clamp(max=s["rows"] - 1)
    x = cq[at].view(-1, most, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(-1, kv, group * most, dim)
    z = x.clamp(min=0) @ b[1] + x.clamp(max=0) @ b[0]                    # whole numbers below 2^24: exact
    z = z.view(-1, kv, group, most, table.shape[1])[seq, :, :, torch.arange(s["rows"], device=q.device) - starts[seq]]
    z = z * s["unit"][table][seq].transpose(1, 2)[:, :, None] * uq.view(-1, kv, group)[..., None]
    z = z.amax(2) + 0.0                                                  # [rows, heads, pages]; no zero is negative
    here = (pos // page)[:, None, None]
    col = torch.arange(table.shape[1], device=q.device)
    z = z.masked_fill((col < case["first"]) | (col > here - case["last"]), math.inf).masked_fill(col > here, -math.inf)
    chosen = torch.sort(z, dim=-1, descending=True, stable=True)[1][..., :blocks]
    chosen = torch.where(chosen <= here, chosen, table.shape[1]).sort(-1)[0]
    chosen = torch.nn.functional.pad(chosen, (0, blocks - chosen.shape[-1]), value=table.shape[1])
    there = chosen < table.shape[1]
    ids = s["pages"][seq].gather(1, chosen.clamp(max=table.shape[1] - 1).flatten(1)).view(chosen.shape)
    s["sel_pages"].copy_(torch.where(there, ids, -1))
    s["sel_lens"].copy_(torch.where(pos >= 0, there[:, 0].sum(-1) * page - page + pos % page + 1, 0))


def _attend(s):
    case = s["case"]
    kv, dim, page, blocks = case["kv_heads"], case["dim"], case["page"], case["blocks"]
    rows = s["rows"]
    ids = s["sel_pages"][..., : s["pages"].shape[1]].clamp(min=0).long()
    head = torch.arange(kv, device=ids.device)[None, :, None]

    def chosen(name):
        """[rows, heads, tokens, dim] of the chosen pages."""
        pool, scale = s[name + "_pool"], s[name + "_scale"]
        x = (pool if scale is None else pool.view(torch.int8)).transpose(1, 2)[ids, head]
        x = x.float() if scale is None else x.view(pool.dtype).float() * scale.transpose(1, 2)[ids, head][..., None]
        return x.flatten(2, 3)

    p = s["q"].float().view(rows, kv, -1, dim) @ chosen("k").transpose(2, 3) * (1 / math.sqrt(dim))
    seen = (torch.arange(p.shape[-1], device=ids.device) < s["sel_lens"][:, None])[:, None, None]
    p = p.masked_fill_(~seen, -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = p.sum(-1, keepdim=True)
    y = p @ chosen("v") / torch.where(total > 0, total, torch.ones_like(total))
    s["out"].copy_(y.view(s["out"].shape))


def _free(s, seqs, keep):
    seqs, page = seqs.long(), s["case"]["page"]
    keep = torch.minimum(keep, s["lens"][seqs])
    col = torch.arange(s["pages"].shape[1], device=keep.device)
    held = s["pages"][seqs]
    gone = (col >= ((keep + page - 1) // page)[:, None]) & (col < ((s["lens"][seqs] + page - 1) // page)[:, None])
    s["refs"].index_add_(0, held.clamp(min=0).flatten(), -gone.flatten().to(torch.int32))
    s["pages"][seqs] = torch.where(gone, -1, held)
    s["lens"][seqs] = keep


def _fork(s):
    parents, children, page = s["parents"].long(), s["children"].long(), s["case"]["page"]
    lens = s["lens"][parents]
    col = torch.arange(s["pages"].shape[1], device=lens.device)
    there = col < ((lens + page - 1) // page)[:, None]
    held = s["pages"][parents]
    s["refs"].index_add_(0, held.clamp(min=0).flatten(), there.flatten().to(torch.int32))
    s["pages"][children] = torch.where(there, held, -1)
    s["lens"][children] = lens


def _extend(s):
    lens, grow, refs, pages, page = s["lens"], s["grow"], s["refs"], s["pages"], s["case"]["page"]
    seqs, cols = pages.shape
    n = torch.arange(seqs, device=lens.device)
    ok = (grow > 0) & (lens + grow <= cols * page)
    last = pages[n, (lens // page).clamp(max=cols - 1).long()]
    shared = ok & (lens % page > 0) & (refs[last.clamp(min=0).long()] > 1)
    # writers of one page: all but the last take a copy, all of them where others hold it too
    at = torch.where(shared, last, refs.shape[0]).long()
    count = torch.zeros(refs.shape[0] + 1, dtype=torch.int32, device=lens.device)
    writers = count.index_add(0, at, torch.ones_like(lens))
    final = count.sub(1).scatter_reduce(0, at, n.to(torch.int32), "amax")
    copies = shared & ((final[at] != n) | (writers[at] < refs[last.clamp(min=0).long()]))
    have = (lens + page - 1) // page
    need = torch.where(ok, (lens + grow + page - 1) // page - have + copies, 0)
    upto = need.cumsum(0)
    free = torch.nonzero(refs == 0)[:, 0].to(torch.int32)
    ok &= upto <= free.shape[0]
    copies &= ok
    col = torch.arange(cols, device=lens.device)
    first = have - copies.to(torch.int32)
    k = col - first[:, None]
    new = ok[:, None] & (k >= 0) & (k < need[:, None])
    ids = torch.cat([free, free.new_zeros(1)])[((upto - need)[:, None] + k).clamp(min=0, max=free.shape[0])]
    refs.index_add_(0, at.clamp(max=refs.shape[0] - 1), -copies.to(torch.int32))
    refs.index_add_(0, ids[new].long(), torch.ones_like(ids[new]))
    s["src"].copy_(torch.where(copies, last, -1))
    s["dst"].copy_(torch.where(copies, ids[n, first.clamp(max=cols - 1).long()], -1))
    s["cells"].copy_(torch.where(copies, lens % page, 0))
    s["got"].copy_(torch.where(ok, grow, 0))
    pages.copy_(torch.where(new, ids, pages))
    lens += s["got"]


def _compact(s):
    refs, pages = s["refs"], s["pages"]
    live = refs > 0
    n = int(live.sum())
    holes, movers = torch.nonzero(~live[:n])[:, 0], torch.nonzero(live[n:])[:, 0].flip(0) + n
    to = torch.arange(refs.shape[0], device=refs.device, dtype=torch.int32)
    to[movers] = holes.to(torch.int32)
    refs[holes] = refs[movers]
    refs[movers] = 0
    pages.copy_(torch.where(pages >= 0, to[pages.clamp(min=0).long()], pages))
    m = holes.shape[0]
    for x, y in ((s["src"], movers), (s["dst"], holes)):
        x.fill_(-1)
        x[:m] = y.to(torch.int32)
    s["top"].fill_(n)


def _copy(s, cells):
    live = torch.nonzero(s["src"] >= 0)[:, 0]
    src, dst, pools = s["src"][live].long(), s["dst"][live].long(), s["pools"]
    x = pools[:, :, src]
    if cells is not None:
        fresh = torch.arange(pools.shape[3], device=src.device) < cells[live][:, None]
        x = torch.where(fresh[..., None, None], x, pools[:, :, dst])
    pools[:, :, dst] = x


# ------------------------------------------------------------------ 64 bits


def _wide_rope(x, weight, pos, freqs, interleaved):
    """Heads x [rows, heads, dim] normed and rotated, as products of complex numbers in 64 bits."""
    x = x.double()
    if weight is not None:
        x = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * weight.double()
    half = freqs.shape[0]
    if not half:
        return x
    turn = torch.polar(torch.ones((x.shape[0], half), dtype=torch.float64, device=x.device), pos.double()[:, None] * freqs.double())
    head, tail = x[..., :2 * half], x[..., 2 * half:]
    pair = head.unflatten(-1, (half, 2)) if interleaved else head.unflatten(-1, (2, half)).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn[:, None])
    z = z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, tail], -1)


def _wide_codes(x, fmt):
    """What vectors x [..., dim] read back as after being stored in 8 bits, in 64 bits."""
    scale = x.abs().amax(-1, keepdim=True) / TOP[fmt]
    z = torch.where(scale > 0, x / scale.clamp(min=1e-300), torch.zeros_like(x))
    if fmt == "int8":
        return z.round() * scale
    # e4m3: three bits after the leading one, exponents from 2^-6 down to multiples of 2^-9
    ulp = torch.ldexp(torch.ones_like(z), (torch.frexp(z)[1] - 1).clamp(min=-6) - 3)
    return (z / ulp).round() * ulp * scale


def _wide_units(x):
    """Integer codes and units of vectors x [..., n] in 64 bits, taken together along the last dimension."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100)
    unit = top.view(torch.int64).bitwise_right_shift(52).sub(6).bitwise_left_shift(52).view(torch.float64)
    return torch.clamp(torch.round(x / unit), -127, 127), unit[..., 0]


def exact(case, seed):
    if "pool" in case:
        return None
    s = _rows_inputs(case, seed)
    new, lens = _lengths(case)
    op, fmt, dim, page, kv = case["op"], case["format"], case["dim"], case["page"], case["kv_heads"]
    start = np.concatenate([[0], np.cumsum(new)]).tolist()
    pos = torch.cat([torch.arange(m - n, m) for n, m in zip(new, lens)]).to("cuda")
    if op in ("rope", "append"):
        live = (pos >= 0)[:, None, None].double()
        at = pos.clamp(min=0)
        q = _wide_rope(s["q"], s["q_weight"], at, s["freqs"], case["interleaved"]) * live
        k = _wide_rope(s["k"], s["k_weight"], at, s["freqs"], case["interleaved"]) * live
        if op == "rope":
            return {"q": q, "k": k}
        v = s["v"].double() * live
        if fmt != "bf16":
            return {"q": q, "k": _wide_codes(k, fmt), "v": _wide_codes(v, fmt)}
        out = {"q": q, "k": torch.zeros(s["k_pool"].shape, dtype=torch.float64, device="cuda")}
        out["v"] = out["k"].clone()
        for a in range(case["seqs"]):
            if not lens[a]:
                continue
            p = torch.arange(lens[a] - new[a], lens[a], device="cuda")
            at = (s["pages"][a].long()[p // page], p % page)
            out["k"][at], out["v"][at] = k[start[a]:start[a + 1]], v[start[a]:start[a + 1]]
        return out

    def keys(ids, name, heads=slice(None)):
        x = s[name + "_pool"].view(torch.int8)[ids].view(s["k_pool"].dtype) if fmt != "bf16" else s[name + "_pool"][ids]
        x = x.float().double()
        return (x if fmt == "bf16" else x * s[name + "_scale"][ids].double()[..., None])[:, :, heads]

    if sum(-(-m // page) - max(0, m - n) // page for n, m in zip(new, lens)) > 20000:
        return None
    code, unit = s["code"].double(), s["unit"].double()
    for a in range(case["seqs"]):
        if not lens[a]:
            continue
        for c in range(max(0, lens[a] - new[a]) // page, -(-lens[a] // page)):
            i = int(s["pages"][a, c])
            x = keys(torch.tensor([i], device="cuda"), "k")[0, : min(page, lens[a] - c * page)].float()   # what the cache stands for is in 32 bits
            b = torch.stack([x.amin(0), x.amax(0)], 1)
            y, u = _wide_units(b.flatten(1))
            code[i], unit[i] = y.view(b.shape), u
    if op == "bounds":
        return {"bounds": code * unit[..., None, None]}
    if sum(new) * kv > 4000:
        return None
    y = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = case["heads"] // kv
    for a in range(case["seqs"]):
        for i in range(new[a]):
            p, row = lens[a] - new[a] + i, start[a] + i
            if p < 0:
                continue
            ids = s["pages"][a, : p // page + 1].long()
            cq, uq = _wide_units(s["q"][row].float())
            cq, uq = cq.view(kv, group, 1, dim), uq.view(kv, group, 1)
            b = code[ids].permute(1, 2, 0, 3)                            # [heads, 2, pages, dim]
            z = torch.maximum(cq * b[:, None, 0], cq * b[:, None, 1]).sum(-1) * unit[ids].T[:, None] * uq
            z = z.amax(1)
            z[:, : case["first"]] = math.inf
            z[:, max(0, ids.shape[0] - case["last"]):] = math.inf
            order = torch.argsort(-z, dim=1, stable=True)[:, : case["blocks"]].sort(1)[0]
            for h in range(kv):
                mine = ids[order[h]]
                n = (mine.shape[0] - 1) * page + p % page + 1
                k, v = (keys(mine, name, h).flatten(0, 1)[:n] for name in ("k", "v"))
                w = torch.softmax(s["q"][row, h * group:(h + 1) * group].double() @ k.T / math.sqrt(dim), -1)
                y[row, h * group:(h + 1) * group] = w @ v
    return {"out": y, "pages": None, "lens": None}
