"""A small paged cache on the GPU and the key-value cache operators computed
from their definitions in 64 bits with numpy, one row at a time; shares
nothing with the CUDA path."""

from __future__ import annotations

import math

import numpy as np

NAN8 = 0x7F  # e4m3


def torch_type(name: str):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}[name]


class Cache:
    """Random k, v and weight pools with shuffled pages.  Every slot that no
    sequence holds is NaN, so that a read outside the sequences shows."""

    def __init__(self, lens, heads=2, dim=64, page=16, kind="bf16", seed=0, layout="hnd", spare=3, scales=True,
                 with_weight=True, table_extra=2):
        import torch
        self.lens, self.heads, self.dim, self.page, self.kind = list(lens), heads, dim, page, kind
        gen = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        self.num_pages = sum(need) + spare
        ids = torch.randperm(self.num_pages, generator=gen)[:sum(need)].to(torch.int32)
        self.width = max(need, default=0) + table_extra
        table = torch.full((len(lens), self.width), -1, dtype=torch.int32)  # entries past a length are not read
        held = torch.zeros(self.num_pages, page, dtype=torch.bool)
        at = 0
        for b, m in enumerate(need):
            table[b, :m] = ids[at:at + m]
            for i in range(m):
                held[int(ids[at + i]), :max(0, min(page, lens[b] - i * page))] = True
            at += m
        self.table_host = table.numpy()
        shape = (self.num_pages, heads, page, dim)

        def pool():
            x = torch.randn(shape, generator=gen)
            if kind == "e4m3":
                x = x * 24
            x = x.to(torch_type(kind))
            return x

        k, v = pool(), pool()
        empty = ~held[:, None, :, None].expand(shape)
        for x in (k, v):
            if kind == "e4m3":
                x.view(torch.uint8)[empty] = NAN8
            else:
                x[empty] = math.nan
        w = torch.rand(shape[:3], generator=gen)
        w[~held[:, None].expand(shape[:3])] = math.nan
        self.ks = self.vs = None
        if kind == "e4m3" and scales:
            self.ks = (torch.rand(heads, generator=gen) + 0.5) / 24
            self.vs = (torch.rand(heads, generator=gen) + 0.5) / 24
        self.k_host, self.v_host, self.w_host = k.float().numpy().astype(np.float64), v.float().numpy().astype(np.float64), w.numpy()

        def put(x):
            if layout == "nhd":  # stored [page][slot][head][dim]
                x = x.view(torch.uint8) if kind == "e4m3" else x
                x = x.transpose(1, 2).contiguous().cuda().transpose(1, 2)
                return x.view(torch_type(kind)) if kind == "e4m3" else x
            return x.cuda()

        self.k, self.v = put(k), put(v)
        self.weight = w.cuda() if with_weight else None
        self.table, self.lens_dev = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()

    def ss(self, m):
        c = [None if s is None else s.cuda() for s in (self.ks, self.vs)]
        pages = m.KVPages(self.k, self.v, weight=self.weight, k_scale=c[0], v_scale=c[1])
        return pages, m.KVTable(self.table, self.lens_dev)

    def rows(self, host, b, h):
        """(len, ...) rows of sequence b, head h, of a host pool."""
        p = np.arange(self.lens[b])
        return host[self.table_host[b, p // self.page], h, p % self.page]

    def scale(self, which, h):
        return 1.0 if which is None else float(which[h])


def visible(n, window, sinks):
    p = np.arange(n)
    return np.ones(n, bool) if window <= 0 else (p < sinks) | (p >= n - window)


def attend_reference(c: Cache, q, scale, window=0, sinks=0):
    """out, lse and the weights added to the pool, from q (batch, q_heads, dim) in 64 bits."""
    q = np.asarray(q, np.float64)
    B, QH, D = q.shape
    G = QH // c.heads
    out, lse = np.zeros((B, QH, D)), np.full((B, QH), -np.inf)
    added = np.zeros(c.w_host.shape)
    for b in range(B):
        n = c.lens[b]
        see = visible(n, window, sinks)
        if not see.any():
            continue
        p = np.arange(n)[see]
        for h in range(c.heads):
            k = c.rows(c.k_host, b, h)[see] * c.scale(c.ks, h)
            v = c.rows(c.v_host, b, h)[see] * c.scale(c.vs, h)
            for g in range(G):
                with np.errstate(invalid="ignore", over="ignore"):
                    s = (k @ q[b, h * G + g]) * scale
                    top = s.max()
                    if top == -np.inf:
                        continue
                    e = np.exp(s - top)
                    w = e / e.sum()
                    out[b, h * G + g] = w @ v
                    lse[b, h * G + g] = top + np.log(e.sum())
                added[c.table_host[b, p // c.page], h, p % c.page] += w
    return out, lse, added


def evict_reference(c: Cache, weights, keep, sinks, recent):
    """kept (batch, heads, keep) positions, -1 padded; `weights` is a host pool."""
    kept = np.full((len(c.lens), c.heads, keep), -1, np.int32)
    for b, n in enumerate(c.lens):
        for h in range(c.heads):
            if n <= keep:
                kept[b, h, :n] = np.arange(n)
                continue
            w = c.rows(weights, b, h).astype(np.float64)
            must = [p for p in range(n) if p < sinks or p >= n - recent]
            rest = [p for p in range(n) if sinks <= p < n - recent]
            # best first: NaN last, then by weight, then by position
            rest.sort(key=lambda p: (np.isnan(w[p]), -w[p] if not np.isnan(w[p]) else 0.0, p))
            kept[b, h] = sorted(must + rest[:keep - len(must)])
    return kept


def e4m3_reference(x):
    """Nearest e4m3 value, ties to even, saturating; NaN stays."""
    x = np.asarray(x, np.float64)
    grid = [0.0]
    for e in range(-6, 9):
        for f in range(8):
            grid.append((1 + f / 8) * 2.0 ** e)
    grid += [f / 8 * 2.0 ** -6 for f in range(1, 8)]
    grid = np.array(sorted(v for v in grid if v <= 448))
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(grid, np.nan_to_num(a)), 1, len(grid) - 1)
    lo = hi - 1
    below, above = a - grid[lo], grid[hi] - a
    pick = np.where(below < above, lo, np.where(above < below, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(np.isnan(x), np.nan, np.copysign(grid[pick], x))
