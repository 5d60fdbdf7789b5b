"""Plain 64-bit model of the paged key/value cache and of attention over it, and seeded
caches for the tests.  Nothing here calls the library."""
from __future__ import annotations

import math
import random

import numpy as np
import torch

TOP = {"int8": 127.0, "fp8": 448.0}
DTYPE = {"bf16": torch.bfloat16, "int8": torch.int8, "fp8": torch.float8_e4m3fn}


def raw(t):
    """Bytes-level view, for indexing and comparing 8-bit float tensors."""
    return t.view(torch.int8) if t.element_size() == 1 else t.view(torch.int16)


def quantise(x, fmt):
    """Codes and scales of bf16 vectors x [..., dim] by the rule of include/lora.h."""
    x = x.float()
    scale = x.abs().amax(-1) / torch.full((), TOP[fmt], device=x.device)
    d = torch.where(scale > 0, scale, torch.ones_like(scale))
    z = (x / d[..., None]).clamp(-TOP[fmt], TOP[fmt])
    code = (z.round() if fmt == "int8" else z).to(DTYPE[fmt])
    bad = ~torch.isfinite(x).all(-1)
    scale[bad] = math.nan
    code.view(torch.int8)[bad] = 0
    return code, scale


def pools(n, page, heads, dim, fmt, layout, dev):
    """Pools filled with NaN (codes of NaN or with NaN scales): cells nobody wrote."""
    dt = DTYPE[fmt]

    def blank(*shape):
        if fmt == "int8":
            return torch.full(shape, -77, dtype=dt, device=dev)
        return torch.full(shape, math.nan, dtype=torch.float32, device=dev).to(dt)
    if layout == "joint":
        both = blank(n, 2, page, heads, dim)
        k, v = both[:, 0], both[:, 1]
    elif layout == "heads":
        k, v = (blank(n, heads, page, dim).transpose(1, 2) for _ in range(2))
    elif layout == "gaps":        # cells wider than their vectors, heads apart
        k, v = (blank(n, page, heads, dim + 32)[..., 16:16 + dim] for _ in range(2))
    else:
        k, v = (blank(n, page, heads, dim) for _ in range(2))
    ks = vs = None
    if fmt != "bf16":
        if layout == "heads":
            ks, vs = (torch.full((n, heads, page), math.nan, device=dev).transpose(1, 2) for _ in range(2))
        else:
            ks, vs = (torch.full((n, page, heads), math.nan, device=dev) for _ in range(2))
    return k, v, ks, vs


class Case:
    """Sequences with lengths `lens` and `new` new tokens each, in shuffled pages; `fill`
    writes every position of every sequence."""

    def __init__(self, seed, new, lens, heads, kv_heads, dim, page, fmt="bf16", layout="split",
                 fill=True, dev="cuda", extra_pages=2, gain=1.0):
        self.gen = torch.Generator(device=dev).manual_seed(seed)
        self.new, self.lens, self.heads, self.kv_heads = list(new), list(lens), heads, kv_heads
        self.dim, self.page, self.fmt, self.dev = dim, page, fmt, dev
        per = [-(-m // page) for m in self.lens]
        wide = max(1, max(per, default=0))
        total = sum(per) + extra_pages
        order = np.random.default_rng(seed).permutation(total).astype(np.int32)
        table = np.full((len(lens), wide), -1, np.int32)
        at = 0
        for s, n in enumerate(per):
            table[s, :n] = order[at:at + n]
            at += n
        self.table = table
        self.pages = torch.from_numpy(table).to(dev)
        self.start = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.starts = torch.from_numpy(self.start).to(dev)
        self.lens_t = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        self.n = int(self.start[-1])
        self.k_pool, self.v_pool, self.k_scale, self.v_scale = pools(total, page, kv_heads, dim, fmt, layout, dev)
        if fill:
            for s, m in enumerate(self.lens):
                if m:
                    self.put(s, range(m), self.rand(m, kv_heads, dim), self.rand(m, kv_heads, dim))
        self.q = self.rand(self.n, heads, dim) * gain
        self.out = torch.full((self.n, heads, dim), 7.0, dtype=torch.bfloat16, device=dev)

    def rand(self, *shape):
        return torch.randn(shape, generator=self.gen, device=self.dev, dtype=torch.float32).to(torch.bfloat16)

    def cells(self, s, js):
        j = torch.as_tensor(list(js), dtype=torch.int64, device=self.dev)
        return self.pages[s].long()[j // self.page], j % self.page

    def put(self, s, js, k, v):
        p, c = self.cells(s, js)
        for x, pool, scale in ((k, self.k_pool, self.k_scale), (v, self.v_pool, self.v_scale)):
            if self.fmt == "bf16":
                pool[p, c] = x
            else:
                code, sc = quantise(x, self.fmt)
                raw(pool)[p, c] = raw(code)
                scale[p, c] = sc

    def get(self, s, m, what="k"):
        """Positions [0, m) of sequence s in float64 [m, kv_heads, dim]."""
        pool, scale = (self.k_pool, self.k_scale) if what == "k" else (self.v_pool, self.v_scale)
        p, c = self.cells(s, range(m))
        x = raw(pool)[p, c].view(pool.dtype).float().double()
        return x if scale is None else x * scale[p, c].double()[..., None]

    def reference(self, scale=None, window=0, sinks=0):
        """(out, bound) in float64.  Keys a row does not see are left out of its sums, not
        weighted with zero.  bound, per element, with A = sum w |v| >= |out|, for a sequence
        of at most 16 rows (new * query heads per key head): 2^-9 |out| + 2^-9 A, which is
        at least half a bf16 step of the output (2^-8 |out|), and 2^-12 A for everything in
        fp32 and weights of 16 bits (scores of magnitude up to ~64 have absolute errors of
        at most ~2^-13).  For more rows weights are bf16 (each within 2^-8 of itself):
        2^-8 |out| + (2^-8 + 2^-11) A."""
        scale = 1 / math.sqrt(self.dim) if scale is None else scale
        out = torch.zeros((self.n, self.heads, self.dim), dtype=torch.float64, device=self.dev)
        mass, few = torch.zeros_like(out), torch.ones_like(out, dtype=torch.bool)
        group = self.heads // self.kv_heads
        for s, (n, m) in enumerate(zip(self.new, self.lens)):
            got = min(n, m)
            if not got:
                continue
            if n * group > 16:
                few[int(self.start[s]):int(self.start[s + 1])] = False
            k, v = self.get(s, m), self.get(s, m, "v")
            rows = slice(int(self.start[s + 1]) - got, int(self.start[s + 1]))
            pos = torch.arange(m - got, m, device=self.dev)[:, None]
            j = torch.arange(m, device=self.dev)[None, :]
            seen = j <= pos
            if window:
                seen = seen & ((j > pos - window) | (j < sinks))
            clean = bool(torch.isfinite(v).all())
            for h in range(self.heads):
                kh, vh = k[:, h // group], v[:, h // group]
                z = self.q[rows, h].double() @ kh.T * scale
                if not bool(torch.isfinite(kh).all()):   # inf - inf inside one product is its own
                    z = torch.where(seen, z, torch.zeros_like(z))
                z = z.masked_fill(~seen, -math.inf)
                w = torch.exp(z - z.amax(-1, keepdim=True))
                w = torch.where(seen, w, torch.zeros_like(w))
                w = w / w.sum(-1, keepdim=True)
                if clean:
                    out[rows, h], mass[rows, h] = w @ vh, w @ vh.abs()
                else:
                    for i in range(got):
                        on = seen[i]
                        out[rows.start + i, h] = w[i, on] @ vh[on]
                        mass[rows.start + i, h] = w[i, on] @ vh[on].abs()
        fine = 2.0 ** -9 * 1.001 * out.abs() + (2.0 ** -9 + 2.0 ** -12) * mass
        return out, torch.where(few, fine, 2.0 ** -8 * 1.001 * out.abs() + (2.0 ** -8 + 2.0 ** -11) * mass)


def assert_attention(got, want, bound):
    got = got.double()
    same_nan = torch.isnan(got) == torch.isnan(want)
    assert bool(same_nan.all()), f"NaN pattern differs at {int((~same_nan).sum())} elements"
    ok = torch.isnan(want) | ((got - want).abs() <= bound) | (got == want)
    if not bool(ok.all()):
        bad = torch.nonzero(~ok)
        i = tuple(bad[0].tolist())
        raise AssertionError(f"{bad.shape[0]} of {ok.numel()} elements beyond their bound, first {i}: "
                             f"{got[i].item()} for {want[i].item()} (bound {bound[i].item():.3g})")


def random_batch(seed, seqs, new_hi, len_hi, released=0):
    rng = random.Random(seed)
    lens = [rng.randint(1, len_hi) for _ in range(seqs)]
    new = [rng.randint(0 if seqs > 1 else 1, new_hi) for _ in range(seqs)]
    for s in rng.sample(range(seqs), released):
        lens[s] = 0
        new[s] = 1
    if sum(new) == 0:
        new[0] = 1
    return new, lens
