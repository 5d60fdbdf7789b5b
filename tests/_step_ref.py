"""Plain models of the operators around the cache: norms and rotation of heads in 64 bits, page
tables as Python lists, bounds and the choice of pages in integers.  Nothing here calls the
library."""
from __future__ import annotations

import math

import numpy as np
import torch


# ------------------------------------------------------------------ norms and rotation


def rope(x, weight, pos, freqs, eps, interleaved):
    """(y, size) in float64 of heads x [rows, heads, dim] at positions pos: size is the length of
    the pair an element belongs to (its own magnitude where it is not turned)."""
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * weight.double()
    out, size = y.clone(), y.abs().clone()
    half = 0 if freqs is None else freqs.shape[0]
    if half:
        t = pos.double()[:, None] * freqs.double()
        c, s = t.cos()[:, None], t.sin()[:, None]
        ia = torch.arange(0, 2 * half, 2) if interleaved else torch.arange(half)
        ib = ia + (1 if interleaved else half)
        a, b = y[..., ia], y[..., ib]
        out[..., ia], out[..., ib] = a * c - b * s, a * s + b * c
        size[..., ia] = size[..., ib] = torch.sqrt(a * a + b * b)
    return out, size


def rope_bound(y, size):
    """A bf16 result: half a step is at most 2^-8 |y|.  Ahead of it everything is fp32: the norm's sum of
    up to 256 squares (2^-24 each step, 16 + 5 of them in a row), a reciprocal root of 2 ulp, four
    products and a sum, cosines off by 2^-22: below 2^-18 of the pair's length, taken as 2^-16."""
    return 2.0 ** -8 * 1.001 * y.abs() + 2.0 ** -16 * size


# ------------------------------------------------------------------ page tables


class Pages:
    """lens, rows of pages and counts, changed one sequence after another."""

    def __init__(self, n_seqs, n_cols, n_pages, page_size):
        self.lens, self.rows = [0] * n_seqs, [[] for _ in range(n_seqs)]
        self.refs, self.n_cols, self.page = [0] * n_pages, n_cols, page_size

    def arrays(self):
        table = np.full((len(self.lens), self.n_cols), -1, np.int32)
        for s, row in enumerate(self.rows):
            table[s, : len(row)] = row
        return np.array(self.lens, np.int32), table, np.array(self.refs, np.int32)

    def _need(self, n):
        return -(-n // self.page)

    def extend(self, grow):
        n = len(self.lens)
        writes = {}                       # shared page -> the sequences that write into it
        for s in range(n):
            if grow[s] > 0 and self.lens[s] + grow[s] <= self.n_cols * self.page and self.lens[s] % self.page:
                last = self.rows[s][-1]
                if self.refs[last] > 1:
                    writes.setdefault(last, []).append(s)
        held = {p: self.refs[p] for p in writes}
        free = [p for p, r in enumerate(self.refs) if r == 0]
        got, src, dst, cells = [0] * n, [-1] * n, [-1] * n, [0] * n
        out = False
        at = 0
        for s in range(n):
            if grow[s] <= 0 or self.lens[s] + grow[s] > self.n_cols * self.page:
                continue
            copy = None
            for p, who in writes.items():
                if s in who and (s != who[-1] or len(who) < held[p]):
                    copy = p
            need = self._need(self.lens[s] + grow[s]) - self._need(self.lens[s]) + (copy is not None)
            if out or at + need > len(free):
                out = True
                continue
            mine = free[at:at + need]
            at += need
            if copy is not None:
                src[s], dst[s], cells[s] = copy, mine[0], self.lens[s] % self.page
                self.refs[copy] -= 1
                self.rows[s][-1] = mine[0]
                self.rows[s] += mine[1:]
            else:
                self.rows[s] += mine
            for p in mine:
                self.refs[p] = 1
            self.lens[s] += grow[s]
            got[s] = grow[s]
        return got, src, dst, cells

    def fork(self, parents, children):
        for a, c in zip(parents, children):
            self.rows[c], self.lens[c] = list(self.rows[a]), self.lens[a]
            for p in self.rows[c]:
                self.refs[p] += 1

    def free(self, seqs, keep=None):
        for i, s in enumerate(seqs):
            k = 0 if keep is None else keep[i]
            if k >= self.lens[s]:
                continue
            n = self._need(k)
            for p in self.rows[s][n:]:
                self.refs[p] -= 1
            self.rows[s], self.lens[s] = self.rows[s][:n], k

    def compact(self, n):
        held = sum(r > 0 for r in self.refs)
        holes = [p for p in range(held) if not self.refs[p]]
        movers = [p for p in range(len(self.refs) - 1, held - 1, -1) if self.refs[p]]
        moves = list(zip(movers, holes))[:n]
        to = dict(moves)
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.rows = [[to.get(p, p) for p in row] for row in self.rows]
        top = max([p + 1 for p, r in enumerate(self.refs) if r], default=0)
        src, dst = [a for a, _ in moves], [b for _, b in moves]
        pad = [-1] * (n - len(moves))
        return src + pad, dst + pad, top


# ------------------------------------------------------------------ bounds and choice


def _codes(x):
    """Codes and unit of numbers x taken together, in float64 (x finite)."""
    top = float(x.abs().max()) if x.numel() else 0.0
    e = -100 if top == 0 else max(math.frexp(top)[1] - 1, -100)
    unit = 2.0 ** (e - 6)
    return torch.round(x.double() / unit).clamp(-127, 127), unit


def bounds(case, codes, unit):
    """The bounds of the pages that the new tokens of a tests._kv_ref.Case touch, over copies of codes and unit."""
    codes, unit = codes.clone(), unit.clone()
    for s, (n, m) in enumerate(zip(case.new, case.lens)):
        if not min(n, m):
            continue
        # what the cache stands for is in 32 bits: scale * code rounded to fp32
        x = case.get(s, m).float()
        for col in range(max(0, m - n) // case.page, -(-m // case.page)):
            part = x[col * case.page:(col + 1) * case.page]
            page = int(case.table[s, col])
            for h in range(case.kv_heads):
                both = torch.stack([part[:, h].amin(0), part[:, h].amax(0)])
                if not bool(torch.isfinite(part[:, h]).all()):
                    codes[page, h], unit[page, h] = 0, math.nan
                else:
                    c, u = _codes(both)
                    codes[page, h], unit[page, h] = c.to(torch.int8), u
    return codes, unit


def select(case, codes, unit, blocks, first, last):
    """lens [n], pages [n, heads, blocks] of the choice for the rows of a Case."""
    group = case.heads // case.kv_heads
    lens = torch.full((case.n,), -1, dtype=torch.int32)
    pages = torch.full((case.n, case.kv_heads, blocks), -1, dtype=torch.int32)
    for s, (n, m) in enumerate(zip(case.new, case.lens)):
        for i in range(n):
            row, p = int(case.start[s]) + i, m - n + i
            if p < 0:
                lens[row] = 0
                continue
            cols = p // case.page + 1
            ids = [int(v) for v in case.table[s, :cols]]
            lens[row] = (min(cols, blocks) - 1) * case.page + p % case.page + 1
            for h in range(case.kv_heads):
                if cols <= blocks:
                    chosen = range(cols)
                else:
                    lo, hi = codes[ids, h, 0].double(), codes[ids, h, 1].double()
                    u = unit[ids, h].double()
                    best = torch.full((cols,), -math.inf, dtype=torch.float64, device=codes.device)
                    for g in range(group):
                        q = case.q[row, h * group + g]
                        if not bool(torch.isfinite(q).all()):
                            continue
                        c, uq = _codes(q)
                        z = torch.maximum(c * lo, c * hi).sum(-1) * u * uq
                        best = torch.maximum(best, torch.where(torch.isnan(u), -math.inf, z))
                    best = torch.where(torch.isnan(u), math.inf, best).tolist()
                    inner = sorted(range(first, cols - last), key=lambda c: (-best[c], c))[: blocks - first - last]
                    chosen = list(range(first)) + sorted(inner) + list(range(cols - last, cols))
                got = [ids[c] for c in chosen]
                pages[row, h, : len(got)] = torch.tensor(got, dtype=torch.int32)
    return lens, pages


def chosen_attention(case, lens, pages, scale=None):
    """(out, bound) in float64 of the rows over chosen pages; bound as tests._kv_ref has it for few rows."""
    scale = 1 / math.sqrt(case.dim) if scale is None else scale
    out = torch.zeros((case.n, case.heads, case.dim), dtype=torch.float64, device=case.dev)
    mass = torch.zeros_like(out)
    group = case.heads // case.kv_heads

    def cells(ids, h, what, n):
        pool, sc = (case.k_pool, case.k_scale) if what == "k" else (case.v_pool, case.v_scale)
        b = pool if pool.element_size() == 2 else pool.view(torch.int8)
        x = b[ids, :, h].view(pool.dtype).float().double()
        if sc is not None:
            x = x * sc[ids, :, h].double()[..., None]
        return x.flatten(0, 1)[:n]
    for row in range(case.n):
        n = int(lens[row])
        if n <= 0:
            continue
        for h in range(case.kv_heads):
            ids = pages[row, h, : -(-n // case.page)].long().to(case.dev)
            k, v = cells(ids, h, "k", n), cells(ids, h, "v", n)
            heads = slice(h * group, (h + 1) * group)
            w = torch.softmax(case.q[row, heads].double() @ k.T * scale, -1)
            out[row, heads], mass[row, heads] = w @ v, w @ v.abs()
    return out, 2.0 ** -9 * 1.001 * out.abs() + (2.0 ** -9 + 2.0 ** -12) * mass
