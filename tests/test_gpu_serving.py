"""Decode steps as a server runs them: page tables and slots from request
lengths, norms and rotation on the way into the cache, attention over it, and an
eviction, each step against the same sequences kept as plain rows.

Tolerances.  The rows that the attention reads are taken from the cache itself, so
that out is within half a unit of bf16 (2^-8 |out|) and 2^-10 of the largest value of
the formula: the weights' rounding (2^-11, narrow caches) and that of fp32 scores and
sums, below 2^-12 for these sizes.  The cached rows are compared with the formula's: v's
are exact or the nearest code, k's within the error that tests/test_gpu_qk_rope.py
derives and half a step of the cache's type."""

from __future__ import annotations

import random

import numpy as np
import pytest

from kv_helpers import torch_type
from serving_helpers import frequencies, open4, rope_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    import stream_compaction_pass_gb300 as m
    return m


class Server:
    """One attention layer over a paged cache whose pages the GPU hands out."""

    def __init__(self, ss, batch, cache, heads=2, group=4, dim=128, page=16, pages=400, width=40, room=300):
        import torch
        self.ss, self.kind, self.heads, self.group, self.dim, self.page, self.batch = ss, cache, heads, group, dim, page, batch
        shape = (pages, heads, page)
        size = {"e2m1": dim // 2, "e4m3": dim}.get(cache, dim)
        one = torch.uint8 if cache in ("e2m1", "e4m3") else torch_type(cache)
        self.k, self.v = (torch.zeros(*shape, size, dtype=one, device="cuda") for _ in range(2))
        self.scale = torch.full((heads,), 1 / 32 if cache == "e4m3" else 1.0, device="cuda")
        more = {}
        if cache == "e2m1":
            self.kb, self.vb = (torch.zeros(*shape, dim // 16, dtype=torch.uint8, device="cuda") for _ in range(2))
            more = dict(k_block=self.kb.view(torch.float8_e4m3fn), v_block=self.vb.view(torch.float8_e4m3fn))
        view = (lambda x: x.view(torch.float8_e4m3fn)) if cache == "e4m3" else (lambda x: x)
        scales = {} if cache == "bf16" else dict(k_scale=self.scale, v_scale=self.scale)
        self.cache = ss.KVPages(view(self.k), view(self.v), weight=torch.zeros(shape, device="cuda"), **scales, **more)
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.seqs = ss.KVTable(torch.zeros(batch, width, dtype=torch.int32, device="cuda"), self.lens)
        self.free = ss.KVFree(torch.randperm(pages, device="cuda").to(torch.int32), torch.tensor([0, pages], dtype=torch.int32, device="cuda"))
        self.freq = frequencies(dim)
        self.rope = ss.Rope(torch.from_numpy(self.freq).cuda())
        gen = torch.Generator().manual_seed(1)
        self.wq, self.wk = ((torch.rand(dim, generator=gen) + 0.5).to(torch.bfloat16).cuda() for _ in range(2))
        self.room = room
        self.positions, self.slots = torch.empty(room, dtype=torch.int32, device="cuda"), torch.empty(room, dtype=torch.int64, device="cuda")
        self.offsets = torch.empty(batch + 1, dtype=torch.int32, device="cuda")
        self.counts, self.restart = torch.zeros(batch, dtype=torch.int32, device="cuda"), torch.zeros(batch, dtype=torch.bool, device="cuda")
        self.qkv = torch.zeros(room, (group + 2) * heads, dim, dtype=torch.bfloat16, device="cuda")
        self.q = torch.zeros(room, group * heads, dim, dtype=torch.bfloat16, device="cuda")
        self.last, self.out = (torch.zeros(batch, group * heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step(self, stream=None):
        """The GPU's part, the same for every counts, restart and qkv: a graph can hold it."""
        import torch
        ss, hq = self.ss, self.group * self.heads
        ss.ss_kv_assign(self.seqs, self.free, self.page, counts=self.counts, restart=self.restart, offsets=self.offsets, positions=self.positions, slots=self.slots,
                        stream=stream)
        ss.ss_kv_append_rope(self.cache, self.slots, self.qkv[:, :hq], self.qkv[:, hq:hq + self.heads], self.qkv[:, hq + self.heads:], self.wq, self.wk, self.rope,
                             self.positions, self.q, stream=stream)
        torch.index_select(self.q, 0, (self.offsets[1:].long() - 1).clamp(min=0), out=self.last)
        ss.ss_kv_attend(self.cache, self.seqs, self.last, self.out, weight_in=self.cache.weight, weight_out=self.cache.weight, stream=stream)

    def rows(self, b, n):
        """k and v of sequence b as the cache holds them, in 64 bits: (n, heads, dim)."""
        p = np.arange(n)
        at = self.seqs.pages[b].cpu().numpy()[p // self.page], slice(None), p % self.page
        got = []
        for x, blocks in ((self.k, getattr(self, "kb", None)), (self.v, getattr(self, "vb", None))):
            if self.kind == "e2m1":
                y = open4(x.cpu().numpy()[at], blocks.cpu().numpy()[at])
            else:
                import torch
                y = (x.view(torch.float8_e4m3fn) if self.kind == "e4m3" else x).double().cpu().numpy()[at]
            got.append(y * self.scale.cpu().numpy()[:, None])
        return got


def check_step(s, expect, counts, served):
    """out of every sequence that got tokens, from the rows that the cache holds."""
    out, q = s.out.double().cpu().numpy(), s.last.double().cpu().numpy()
    for b in range(s.batch):
        n = len(expect[b])
        assert int(s.lens[b]) == n
        if n == 0 or counts[b] == 0 or not served[b]:
            continue
        k, v = s.rows(b, n)
        want_k, want_v = (np.stack([r[i] for r in expect[b]]) for i in range(2))
        step = {"bf16": 2.0 ** -8, "e4m3": 2.0 ** -4}.get(s.kind)
        if step:
            small = 2.0 ** -10 / 32 if s.kind == "e4m3" else 0.0  # half the smallest e4m3 step
            assert (np.abs(v - want_v) <= step * np.abs(want_v) + small).all()
            assert (np.abs(k - want_k) <= 1.01 * step * np.abs(want_k) + small + 1e-4).all()
        else:  # a block's step is at most its largest element's 1 / 6, and 1 / 16 of that
            for got, want in ((v, want_v), (k, want_k)):
                blocks = np.abs(want).reshape(*want.shape[:2], -1, 16).max(-1)
                assert (np.abs(got - want) <= np.repeat(blocks, 16, -1) * (1 + 1 / 16) / 6 + 2.0 ** -9 + 1e-4).all()
        for j in range(s.group * s.heads):
            h = j // s.group
            x = k[:, h] @ q[b, j] * s.dim ** -0.5
            w = np.exp(x - x.max())
            want = (w / w.sum()) @ v[:, h]
            assert (np.abs(out[b, j] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * np.abs(v[:, h]).max()).all(), (b, j)


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("graph", [False, True])
def test_requests_come_grow_and_go(ss, cache, graph):
    import torch
    batch = 6
    s = Server(ss, batch, cache)
    rng, gen = random.Random(3), torch.Generator().manual_seed(4)
    expect = [[] for _ in range(batch)]
    stream = torch.cuda.Stream()
    g = None
    for step in range(12):
        prompt = [not expect[b] or rng.random() < 0.1 for b in range(batch)]
        restart = [p and bool(expect[b]) for b, p in enumerate(prompt)]
        counts = [rng.choice([1, 7, 16, 45]) if p else rng.choice([0, 1, 1]) for p in prompt]
        s.counts.copy_(torch.tensor(counts, dtype=torch.int32))
        s.restart.copy_(torch.tensor(restart))
        new = torch.randn(s.room, s.qkv.shape[1], s.dim, generator=gen).to(torch.bfloat16)
        s.qkv.copy_(new)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            if not graph:
                s.step(stream)
            elif g is None:
                s.step(stream)
                # scratch is there now, for all lengths that the table can hold; the graph is for the steps to come
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=stream):
                    s.step(stream)
            else:
                g.replay()
        torch.cuda.synchronize()
        st, where = ss.ss_stream_status(stream)
        assert st == ss.SS_OK, (st, where, ss.ss_last_error_detail())
        at, hq = 0, s.group * s.heads
        for b, c in enumerate(counts):
            if restart[b]:
                expect[b] = []
            x = new[at:at + c].double().numpy()
            if c:
                k = rope_reference(x[:, hq:hq + s.heads], s.wk.double().cpu().numpy(), np.arange(len(expect[b]), len(expect[b]) + c), s.freq, False, 1e-6)
                expect[b] += [(k[i], x[i, hq + s.heads:]) for i in range(c)]
            at += c
        check_step(s, expect, counts, [True] * batch)
        # every page is held once or free once
        used = [p for b in range(batch) for p in s.seqs.pages[b, :-(-len(expect[b]) // s.page)].tolist()]
        head, count = s.free.state.tolist()
        ring = s.free.pages.tolist()
        assert sorted(used + [ring[(head + i) % len(ring)] for i in range(count)]) == list(range(len(ring)))


@pytest.mark.parametrize("cache", ["bf16", "e2m1"])
def test_a_pool_that_runs_out_serves_whom_it_can(ss, cache):
    import torch
    s = Server(ss, 4, cache, pages=9, width=12, room=160)
    gen = torch.Generator().manual_seed(5)
    for counts, lens in (([40, 40, 40, 40], [40, 40, 40, 0]), ([1, 8, 9, 3], [41, 48, 40, 0]), ([8, 1, 0, 0], [48 + 1, 48, 40, 0])):
        counts = list(counts)
        s.counts.copy_(torch.tensor(counts, dtype=torch.int32))
        s.qkv.copy_(torch.randn(s.room, s.qkv.shape[1], s.dim, generator=gen).to(torch.bfloat16))
        before = s.lens.tolist()
        s.step()
        st, where = ss.ss_stream_status()
        assert st == ss.SS_OK, (st, where)
        # 9 pages of 16: three prompts of 40 take 3 each; then only what its pages still hold fits
        pages = lambda n: -(-n // 16)  # noqa: E731
        free, want = 9 - sum(map(pages, before)), []
        short = False
        for n, c in zip(before, counts):
            need = pages(n + c) - pages(n)
            short = short or need > free
            if need and short:
                want.append(n)
            else:
                free -= need
                want.append(n + c)
        assert s.lens.tolist() == want
        slots = s.slots.cpu()
        at = 0
        for b, c in enumerate(counts):
            assert bool((slots[at:at + c] >= 0).all()) == (want[b] != before[b] or c == 0)
            at += c
        assert bool((slots[at:] == -1).all())


def test_evict_after_decode_steps_in_4_bits(ss):
    """What eviction moves attends as what stayed."""
    import torch
    s = Server(ss, 3, "e2m1", pages=120, width=30, room=200)
    gen = torch.Generator().manual_seed(6)
    for counts in ([60, 33, 90], [1, 1, 1], [1, 1, 1]):
        s.counts.copy_(torch.tensor(counts, dtype=torch.int32))
        s.qkv.copy_(torch.randn(s.room, s.qkv.shape[1], s.dim, generator=gen).to(torch.bfloat16))
        s.step()
    keep = 40
    lens = s.lens.tolist()
    new = ss.KVTable(torch.arange(9, dtype=torch.int32, device="cuda").view(3, 3), torch.zeros(3, dtype=torch.int32, device="cuda"))
    shape = (9, s.heads, s.page)
    k, v = (torch.zeros(*shape, s.dim // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    kb, vb = (torch.zeros(*shape, s.dim // 16, dtype=torch.uint8, device="cuda") for _ in range(2))
    pool = ss.KVPages(k, v, weight=torch.zeros(shape, device="cuda"), k_scale=s.scale, v_scale=s.scale, k_block=kb.view(torch.float8_e4m3fn),
                      v_block=vb.view(torch.float8_e4m3fn))
    kept = torch.empty(3, s.heads, keep, dtype=torch.int32, device="cuda")
    ss.ss_kv_evict(s.cache, s.seqs, pool, new, keep, sinks=2, recent=8, kept=kept)
    ss.ss_kv_attend(pool, new, s.last, s.out)
    assert ss.ss_stream_status()[0] == ss.SS_OK
    out, q, kept = s.out.double().cpu().numpy(), s.last.double().cpu().numpy(), kept.cpu().numpy()
    for b, n in enumerate(lens):
        m = min(n, keep)
        assert int(new.lens[b]) == m
        k64, v64 = s.rows(b, n)
        for j in range(s.group * s.heads):
            h = j // s.group
            idx = kept[b, h, :m]
            x = k64[idx, h] @ q[b, j] * s.dim ** -0.5
            w = np.exp(x - x.max())
            want = (w / w.sum()) @ v64[idx, h]
            assert (np.abs(out[b, j] - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * np.abs(v64[:, h]).max()).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "e2m1"])
def test_example_serves_requests(cache):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_steps.py")
    spec = importlib.util.spec_from_file_location("serve_steps", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    got = example.run(batch=5, heads=2, group=2, dim=64, prompt=70, steps=40, ends=0.05, cache=cache)
    assert got["device_lens"] == got["lens"] and got["finite"] and got["ended"] > 0
    assert got["free"] == got["pages"] - sum(-(-n // got["page"]) for n in got["lens"])


def load_example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_steps.py")
    spec = importlib.util.spec_from_file_location("serve_steps", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    return example


@pytest.mark.parametrize("prompt,steps", [(1, 14), (1, 15), (1, 16), (2, 30)])
def test_example_has_room_for_its_longest_request(prompt, steps):
    """A prompt, the step before the capture and every replay add a token to a
    request that never ends, and its last page may be full."""
    got = load_example().run(batch=3, heads=2, group=2, dim=64, prompt=prompt, steps=steps, ends=0.0, cache="bf16")
    assert got["device_lens"] == got["lens"] and got["finite"] and max(got["lens"]) <= prompt + 1 + steps
    assert got["free"] == got["pages"] - sum(-(-n // got["page"]) for n in got["lens"])


@pytest.mark.parametrize("page,steps,seed", [(16, 16, 64), (1, 6, 5)])
def test_example_has_pages_for_a_request_that_takes_a_place_over(page, steps, seed):
    """The one request ends at the last step, when it holds all but none or one of
    the pages that its table has places for; they come back after that step."""
    ends = random.Random(seed)
    ends.randrange(1, 2)  # the prompt
    assert [ends.random() < 0.05 for _ in range(steps)] == [False] * (steps - 1) + [True]
    got = load_example().run(batch=1, heads=2, group=2, dim=64, page=page, prompt=1, steps=steps, ends=0.05, cache="bf16", seed=seed)
    assert got["device_lens"] == got["lens"] == [2]
    assert got["free"] == got["pages"] - -(-2 // page)
