"""One attention layer decoding over a paged key-value cache with a budget.

Prompts enter the cache, then every step appends one token per sequence,
attends over what is cached while gathering the weights, and, whenever the
sequences have outgrown the budget, evicts the least attended positions into
fresh pages and frees the old ones.  The prompts' own tokens do not attend
here, so the first eviction goes by the attention of the first new token.
Random weights and inputs; `--check` recomputes every step in 64 bits from a
plain list of the kept rows.

    python examples/paged_decode.py --batch 8 --prompt 600 --steps 200 --budget 512 --check
"""

from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import stream_compaction_pass_gb300 as ss  # noqa: E402


class Pool:
    """Pages of one layer and a free list on the host."""

    def __init__(self, pages, heads, page, dim, dtype, scale=None):
        shape = (pages, heads, page, dim)
        self.page, self.free = page, list(range(pages))
        k, v = (torch.zeros(shape, dtype=torch.uint8 if dtype == torch.float8_e4m3fn else dtype, device="cuda").view(dtype) for _ in range(2))
        self.scale = None if scale is None else torch.full((heads,), scale, device="cuda")
        self.cache = ss.KVPages(k, v, weight=torch.zeros(shape[:3], device="cuda"), k_scale=self.scale, v_scale=self.scale)

    def take(self, tokens):
        return [self.free.pop() for _ in range(-(-tokens // self.page))]

    def give(self, pages):
        self.free.extend(pages)


def table_of(rows, width):
    return torch.tensor([r + [0] * (width - len(r)) for r in rows], dtype=torch.int32, device="cuda")


class Check:
    """The same layer on plain rows in 64 bits: a list of (k, v, weight) per (sequence, head)."""

    def __init__(self, batch, heads):
        self.rows = [[[] for _ in range(heads)] for _ in range(batch)]

    def append(self, b, k, v):
        for h, rows in enumerate(self.rows[b]):
            rows.append([k[h].double(), v[h].double(), 0.0])

    def attend(self, b, q, group):
        out = []
        for h, rows in enumerate(self.rows[b]):
            k, v = torch.stack([r[0] for r in rows]), torch.stack([r[1] for r in rows])
            w = torch.softmax(q[h * group:(h + 1) * group].double() @ k.t() * k.shape[1] ** -0.5, 1)
            out.append(w @ v)
            for r, x in zip(rows, w.sum(0).tolist()):
                r[2] += x
        return torch.cat(out)

    def keep(self, b, kept):
        self.rows[b] = [[rows[i] for i in kept[h] if i >= 0] for h, rows in enumerate(self.rows[b])]


def run(batch=8, heads=8, group=4, dim=128, page=16, prompt=600, steps=200, budget=512, slack=64, sinks=4, recent=128,
        dtype="bfloat16", check=False, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind, hidden = getattr(torch, dtype), 512
    width = -(-(max(prompt, budget + slack) + 1) // page)
    pool = Pool(3 * batch * width, heads, page, dim, kind, scale=1 / 32 if dtype == "float8_e4m3fn" else None)
    qkv = torch.randn(hidden, (group + 2) * heads * dim, generator=gen, device="cuda", dtype=torch.bfloat16) * hidden ** -0.5

    def project(x):  # tokens x hidden -> q, k, v side by side, used as they lie
        y = (x @ qkv).unflatten(1, ((group + 2) * heads, dim))
        return y[:, :group * heads], y[:, group * heads:(group + 1) * heads], y[:, (group + 1) * heads:]

    # prompts of different lengths, all in one call
    lens = [max(1, prompt - 7 * b) for b in range(batch)]
    rows = [pool.take(width * page) for _ in range(batch)]
    d_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    seqs = ss.KVTable(table_of(rows, width), d_lens, max_len=width * page)
    x = torch.randn(sum(lens), hidden, generator=gen, device="cuda", dtype=torch.bfloat16)
    _, k, v = project(x)
    offsets = torch.tensor([sum(lens[:b]) for b in range(batch + 1)], dtype=torch.int32, device="cuda")
    ss.ss_kv_append(pool.cache, seqs, k, v, offsets=offsets)

    ref = Check(batch, heads) if check else None

    def cached(b, n):  # what the cache holds for position n of sequence b (8-bit caches round)
        at = rows[b][n // page], slice(None), n % page
        s = 1.0 if pool.scale is None else pool.scale[:, None]
        return pool.cache.k[at].float() * s, pool.cache.v[at].float() * s

    if check:
        for b, n in enumerate(lens):
            for i in range(n):
                ref.append(b, *cached(b, i))

    worst, evictions, kept = 0.0, 0, torch.empty(batch, heads, budget, dtype=torch.int32, device="cuda")
    out = torch.empty(batch, group * heads, dim, device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(steps):
        lens = [n + 1 for n in lens]
        d_lens.add_(1)
        q, k, v = project(torch.randn(batch, hidden, generator=gen, device="cuda", dtype=torch.bfloat16))
        ss.ss_kv_append(pool.cache, seqs, k, v)
        ss.ss_kv_attend(pool.cache, seqs, q, out, weight_in=pool.cache.weight, weight_out=pool.cache.weight)
        if check:
            for b in range(batch):
                ref.append(b, *cached(b, lens[b] - 1))
                want = ref.attend(b, q[b], group)
                worst = max(worst, float((out[b].double() - want).abs().max() / want.abs().max()))
        # after the attention: a prompt's weights are zero until a token has attended to it
        if max(lens) >= budget + slack or evictions == 0 and max(lens) > budget:
            fresh = [pool.take(width * page) for _ in range(batch)]
            new_lens = torch.empty(batch, dtype=torch.int32, device="cuda")
            new = ss.KVTable(table_of(fresh, width), new_lens, max_len=width * page)
            ss.ss_kv_evict(pool.cache, seqs, pool.cache, new, budget, sinks=sinks, recent=recent, kept=kept)
            for r in rows:
                pool.give(r)  # the stream runs in order: whoever takes them next writes after the move
            rows, seqs, d_lens, lens, evictions = fresh, new, new_lens, [min(n, budget) for n in lens], evictions + 1
            if check:
                for b in range(batch):
                    ref.keep(b, kept[b].tolist())
    torch.cuda.synchronize()
    seconds = time.perf_counter() - t0
    status, where = ss.ss_stream_status()
    assert status == ss.SS_OK, (status, where, ss.ss_last_error_detail())
    return {"steps": steps, "evictions": evictions, "lens": lens, "us_per_step": seconds / max(steps, 1) * 1e6, "worst": worst}


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("batch", 8), ("heads", 8), ("group", 4), ("dim", 128), ("page", 16), ("prompt", 600), ("steps", 200),
                          ("budget", 512), ("slack", 64), ("sinks", 4), ("recent", 128), ("seed", 0)):
        p.add_argument("--" + name, type=int, default=default)
    p.add_argument("--dtype", default="bfloat16", choices=["bfloat16", "float8_e4m3fn"])
    p.add_argument("--check", action="store_true")
    a = p.parse_args()
    got = run(**vars(a))
    print(f"{got['steps']} steps, {got['evictions']} evictions, {got['us_per_step']:.1f} us a step"
          + (f", largest error {got['worst']:.2e} of the row's largest value" if a.check else ""))


if __name__ == "__main__":
    main()
