"""One attention layer serving requests that come, grow and go: a decode step is
three calls, the same for every length, so that a CUDA graph holds it.

Every step ss_kv_assign hands out pages for the tokens to come (and takes back those
of requests whose place a new one takes over), ss_kv_append_rope norms and rotates
queries and keys and writes keys and values to their slots, and ss_kv_attend attends
with every sequence's last token.  Random weights and inputs; the host decides who
comes and goes and copies each step's counts to the GPU, and nothing else.

    python examples/serve_steps.py --batch 64 --prompt 1000 --steps 300 --cache e2m1
"""

from __future__ import annotations

import argparse
import os
import random
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import stream_compaction_pass_gb300 as ss  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


def make_cache(kind, pages, heads, page, dim):
    shape = (pages, heads, page)
    weight = torch.zeros(shape, device="cuda")
    if kind == "bf16":
        return ss.KVPages(*(torch.zeros(*shape, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)), weight=weight)
    scale = torch.full((heads,), 1 / 32 if kind == "e4m3" else 1.0, device="cuda")
    k, v = (torch.zeros(*shape, dim if kind == "e4m3" else dim // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    if kind == "e4m3":
        return ss.KVPages(k.view(TYPES[kind]), v.view(TYPES[kind]), weight=weight, k_scale=scale, v_scale=scale)
    kb, vb = (torch.zeros(*shape, dim // 16, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    return ss.KVPages(k, v, weight=weight, k_scale=scale, v_scale=scale, k_block=kb, v_block=vb)


def run(batch=64, heads=8, group=4, dim=128, page=16, prompt=1000, steps=300, ends=0.01, cache="e2m1", seed=0):
    gen, rng, hidden = torch.Generator(device="cuda").manual_seed(seed), random.Random(seed), 512
    width = -(-(prompt + 1 + steps) // page)  # a prompt, the step before the capture, the replays
    pages = batch * (width - (-2 // page))  # and the first ones of requests that take places over, whose pages come back a step later
    pool = make_cache(cache, pages, heads, page, dim)
    i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device="cuda")  # noqa: E731
    seqs = ss.KVTable(i32(batch, width), i32(batch))
    free = ss.KVFree(torch.arange(pages, dtype=torch.int32, device="cuda"), torch.tensor([0, pages], dtype=torch.int32, device="cuda"))
    rope = ss.Rope(10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim))
    weights = [torch.ones(dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    project = torch.randn(hidden, (group + 2) * heads * dim, generator=gen, device="cuda", dtype=torch.bfloat16) * hidden ** -0.5
    counts, restart = i32(batch), torch.zeros(batch, dtype=torch.bool, device="cuda")
    # a copy of the counts to the GPU has to leave the host's numbers alone until it is done: one buffer a step
    h_counts, h_restart = torch.zeros(steps, batch, dtype=torch.int32).pin_memory(), torch.zeros(steps, batch, dtype=torch.bool).pin_memory()

    def decode(room, x):
        """A step's calls, for up to `room` tokens."""
        offsets, positions, slots = i32(batch + 1), i32(room), torch.zeros(room, dtype=torch.int64, device="cuda")
        q = torch.empty(room, group * heads, dim, dtype=torch.bfloat16, device="cuda")
        out = torch.empty(batch, group * heads, dim, dtype=torch.bfloat16, device="cuda")

        def step():
            ss.ss_kv_assign(seqs, free, page, counts=counts, restart=restart, offsets=offsets, positions=positions, slots=slots)
            qkv = (x @ project).unflatten(1, ((group + 2) * heads, dim))
            ss.ss_kv_append_rope(pool, slots, qkv[:, :group * heads], qkv[:, group * heads:(group + 1) * heads], qkv[:, (group + 1) * heads:], *weights, rope, positions, q)
            ss.ss_kv_attend(pool, seqs, q[offsets[1:].long() - 1], out)
            return out
        return step

    # prompts enter together, as a chunk that is padded to a fixed size
    first = [rng.randrange(1, prompt + 1) for _ in range(batch)]
    room = max(sum(first), batch * 2)
    x_first = torch.randn(room, hidden, generator=gen, device="cuda", dtype=torch.bfloat16)
    counts.copy_(torch.tensor(first, dtype=torch.int32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        decode(room, x_first)()
        # later steps: one token each, or the two of a short new request in a place that ended
        x = torch.randn(2 * batch, hidden, generator=gen, device="cuda", dtype=torch.bfloat16)
        step = decode(2 * batch, x)
        counts.fill_(1)
        out = step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step()
        side.synchronize()
        lens, served = [n + 1 for n in first], 0
        t0 = time.perf_counter()
        for i in range(steps):
            over = [rng.random() < ends for _ in range(batch)]
            h_counts[i].copy_(torch.tensor([2 if o else 1 for o in over], dtype=torch.int32))
            h_restart[i].copy_(torch.tensor(over))
            counts.copy_(h_counts[i], non_blocking=True)
            restart.copy_(h_restart[i], non_blocking=True)
            x.normal_(generator=gen)
            graph.replay()
            lens = [2 if o else n + 1 for o, n in zip(over, lens)]
            served += sum(over)
        side.synchronize()
        seconds = time.perf_counter() - t0
    status, where = ss.ss_stream_status(side)
    assert status == ss.SS_OK, (status, where, ss.ss_last_error_detail())
    return {"lens": lens, "device_lens": seqs.lens.tolist(), "free": int(free.state[1]), "pages": pages, "page": page, "ended": served,
            "us_per_step": seconds / max(steps, 1) * 1e6, "finite": bool(torch.isfinite(out.float()).all())}


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("batch", 64), ("heads", 8), ("group", 4), ("dim", 128), ("page", 16), ("prompt", 1000), ("steps", 300), ("seed", 0)):
        p.add_argument("--" + name, type=int, default=default)
    p.add_argument("--ends", type=float, default=0.01, help="share of the requests that end in a step")
    p.add_argument("--cache", default="e2m1", choices=["bf16", "e4m3", "e2m1"])
    got = run(**vars(p.parse_args()))
    print(f"{got['us_per_step']:.1f} us a step, {got['ended']} requests ended, {got['free']} of {got['pages']} pages free")


if __name__ == "__main__":
    main()
