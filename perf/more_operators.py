"""The operators around a decode step over the paged key-value cache, as they
are measured: page tables and slot maps from request lengths (`assign`), norms
and position rotation of queries and keys (`rope`, its backward pass `back`,
and `cached`, which writes the rows into the cache), and attention over a cache
held in 4 bits (`attend`).

With ``own = False`` `run` computes an operator in its plain form, elementary
torch operations in 32 bits (angles in 64) rounded once at the end; with ``own =
True`` it makes the calls a user of the library makes.  `exact` computes the
same outputs from the definitions, in 64 bits or in whole numbers.

Definitions:

  assign   sequence b, of length old (0 where it is restarted), gets count
           tokens more: need = ceil((old + count) / page) - ceil(old / page)
           pages, taken from the front of a ring of free pages in the order of
           the sequences.  It is served where it needs none, or where the
           needs up to it do not exceed the ring's count; otherwise its length
           stays at old.  The pages of a restarted sequence go to the ring's
           end, in order.  Token i of sequence b has position old + i and slot
           page * page_size + position % page_size, -1 where it has no place.
  rope     y = R(p) (x / sqrt(mean(x^2) + eps) * w) for every head's row x of
           q and k; R(p) turns the pairs (x_i, x_{i + r/2}), or (x_2i, x_2i+1)
           where interleaved, i < r/2, by the angle p * f_i, and leaves what
           lies behind r.
  back     the gradients of q, k and both weights for given gradients of the
           outputs of rope.
  cached   rope, with k's rows and those of v written to the slots of a cache,
           in an 8-bit one as e4m3(clamp(x / scale[h], -448, 448)); slots of -1
           are passed over.
  attend   over a cache in 4 bits: element d of a row is e2m1(nibble d) *
           e4m3(block d / 16) * scale[h].  s(p) = q . k(p) / sqrt(dim) over the
           visible positions {p < len : p < sinks or p >= len - window} (window
           0: all), w = exp(s - max) / sum, out = sum_p w(p) v(p), lse = log
           sum_p exp(s(p)), and, where weights are kept, weight_out(h, p) =
           weight_in(h, p) + the sum of w(p) over h's query heads.
"""

import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
EPS = 1e-6


def listed():
    return [
        # One decode step of a serving batch: every sequence grows by a token.
        {"name": "assign_tokens", "op": "assign", "batch": 64, "lo": 100, "hi": 8191, "new_lo": 1, "new_hi": 1, "page": 16,
         "restart": 0.0, "pad": 0, "lens": 1},
        # A full machine admits prompts: ragged chunks, some places taken over from requests that ended.
        {"name": "assign_prompts", "op": "assign", "batch": 512, "lo": 1, "hi": 16000, "new_lo": 1, "new_hi": 8191, "page": 32,
         "restart": 0.3, "pad": 1000, "lens": 2},
        # A training step's queries and keys, views of the fused projection.
        {"name": "rope_train", "op": "rope", "tokens": 16384, "q_heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "type": "bf16",
         "interleaved": False, "theta": 1e4, "far": 4096},
        # Narrow heads, part of them rotated in adjacent pairs, at far positions.
        {"name": "rope_odd", "op": "rope", "tokens": 1111, "q_heads": 12, "kv_heads": 12, "dim": 80, "rot": 32, "type": "f16",
         "interleaved": True, "theta": 1e6, "far": 1000000},
        # The training step's gradients.
        {"name": "back_train", "op": "back", "tokens": 16384, "q_heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "type": "bf16",
         "interleaved": False, "theta": 1e4, "far": 4096},
        # The same in 32 bits, a few short sequences.
        {"name": "back_small", "op": "back", "tokens": 777, "q_heads": 12, "kv_heads": 4, "dim": 96, "rot": 96, "type": "f32",
         "interleaved": False, "theta": 5e5, "far": 300},
        # One token of every sequence of a batch on its way into the cache: latency.
        {"name": "cached_tokens", "op": "cached", "tokens": 64, "q_heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "type": "bf16",
         "interleaved": False, "theta": 5e5, "far": 8191, "page": 16, "cache": "bf16", "pad": 0},
        # Prompts on their way into an 8-bit cache, the batch padded to a fixed size.
        {"name": "cached_prompts", "op": "cached", "tokens": 20000, "q_heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "type": "bf16",
         "interleaved": False, "theta": 5e5, "far": 100000, "page": 32, "cache": "e4m3", "pad": 480},
        # One conversation on its own: what a token waits for is latency.
        {"name": "attend_one", "op": "attend", "batch": 1, "lo": 1021, "hi": 1021, "heads": 8, "group": 4, "dim": 128, "page": 16,
         "type": "bf16", "window": 0, "sinks": 0, "weights": False, "lens": 3},
        # An ordinary serving batch of ragged lengths that keeps the weights for a later eviction.
        {"name": "attend_batch", "op": "attend", "batch": 64, "lo": 100, "hi": 16001, "heads": 8, "group": 4, "dim": 128, "page": 16,
         "type": "bf16", "window": 0, "sinks": 0, "weights": True, "lens": 4},
        # Streaming decode: a window and a few first tokens, narrow heads that all have their own keys.
        {"name": "attend_window", "op": "attend", "batch": 96, "lo": 3000, "hi": 30011, "heads": 12, "group": 1, "dim": 64, "page": 16,
         "type": "f16", "window": 4095, "sinks": 4, "weights": False, "lens": 5},
        # A full machine: many long sequences, of which 4 bits let the cache hold more.
        {"name": "attend_large", "op": "attend", "batch": 48, "lo": 20000, "hi": 80000, "heads": 8, "group": 8, "dim": 128, "page": 64,
         "type": "bf16", "window": 0, "sinks": 0, "weights": False, "lens": 6},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _lens(case):
    """The sequences' lengths: spread over the logarithm between lo and hi, the first one hi."""
    rng = random.Random(case["lens"])
    lens = [case["hi"]] + [_log_int(rng, case["lo"], case["hi"]) for _ in range(case["batch"] - 1)]
    rng.shuffle(lens)
    return lens


def _asked(case):
    """assign: each sequence's new tokens, and whether it is restarted."""
    rng = random.Random(case["lens"] + 1)
    counts = [_log_int(rng, case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    return counts, [rng.random() < case["restart"] for _ in range(case["batch"])]


def _draw_assign(rng):
    case = {"op": "assign", "batch": _log_int(rng, 1, 2000), "hi": _log_int(rng, 1, 60000), "page": rng.choice([8, 16, 16, 32, 64, 100, 128]),
            "restart": rng.choice([0.0, 0.05, 0.5]), "pad": rng.choice([0, 0, 1, 777]), "lens": rng.randrange(1 << 30)}
    case["lo"] = max(1, case["hi"] // rng.choice([1, 5, 50]))
    case["new_lo"], case["new_hi"] = rng.choice([(1, 1), (1, 1), (1, _log_int(rng, 2, 8191)), (100, 2000)])
    return case


def _draw_rope(rng):
    op = rng.choice(["rope", "back", "cached"])
    case = {"op": op, "tokens": _log_int(rng, 1, 32768), "kv_heads": rng.choice([1, 2, 4, 8, 12]), "dim": rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256]),
            "type": rng.choice(["bf16", "bf16", "f16", "f32"]), "interleaved": rng.random() < 0.3, "theta": rng.choice([1e4, 5e5, 1e6]),
            "far": _log_int(rng, 100, 1000000)}
    case["q_heads"] = case["kv_heads"] * rng.choice([1, 1, 3, 4, 8])
    case["rot"] = rng.choice([case["dim"], case["dim"], 32, 64])
    if op == "cached":
        case["type"] = rng.choice(["bf16", "bf16", "f16"])
        case["cache"] = rng.choice([case["type"], "e4m3"])
        case["page"], case["pad"] = rng.choice([8, 16, 32, 128]), rng.choice([0, 0, 3, 500])
    return case


def _draw_attend(rng):
    case = {"op": "attend", "batch": _log_int(rng, 1, 96), "heads": rng.choice([1, 2, 4, 8, 12]), "group": rng.choice([1, 2, 4, 5, 8, 16]),
            "dim": rng.choice([64, 128, 128, 128, 256]), "page": rng.choice([8, 16, 16, 32, 64, 128]), "type": rng.choice(["bf16", "bf16", "f16"]),
            "weights": rng.random() < 0.4, "hi": _log_int(rng, 500, 131072), "lens": rng.randrange(1 << 30)}
    case["lo"] = max(1, case["hi"] // rng.choice([1, 2, 5, 20]))
    case["window"], case["sinks"] = rng.choice([(0, 0), (0, 0), (_log_int(rng, 100, 8000), rng.choice([0, 1, 4, 20]))])
    return case


def draw(rng):
    most = {op: max(work(c)["bytes"] for c in listed() if c["op"] == op) for op in ("assign", "rope", "back", "cached", "attend")}
    while True:
        case = rng.choice([_draw_assign, _draw_rope, _draw_rope, _draw_attend, _draw_attend])(rng)
        if case["op"] == "attend" and sum(_lens(case)) * case["heads"] * case["dim"] * 18 // 16 > most["attend"]:
            continue  # what a window hides is held all the same
        if work(case)["bytes"] <= most[case["op"]]:
            return case


def _table(case, lens, gen, spare=1):
    """A page table of the sequences over a shuffled pool, the pool's page count, and the pages that are nobody's."""
    need = [-(-n // case["page"]) for n in lens]
    count = sum(need) + spare
    ids = torch.randperm(count, generator=gen, device="cuda").to(torch.int32).cpu()
    table = torch.zeros(len(lens), max(max(need), 1), dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = ids[at:at + m]
        at += m
    return table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), count, ids[at:].cuda()


def _prepare_assign(case, gen, st):
    lens, (counts, restart), page = _lens(case), _asked(case), case["page"]
    need = [-(-((0 if r else n) + c) // page) - (0 if r else -(-n // page)) for n, c, r in zip(lens, counts, restart)]
    spare = sum(need) + 50 if case["lens"] % 3 else max(1, sum(need) * 3 // 4)  # in a third of the cases the free pages run out
    table, st["lens"], count, free = _table(case, lens, gen, spare)
    st["max_pages"] = max(-(-(n + c) // page) for n, c in zip(lens, counts)) + 1
    st["table"] = torch.zeros(case["batch"], st["max_pages"], dtype=torch.int32, device="cuda")
    st["table"][:, :table.shape[1]] = table
    st["new_table"], st["new_lens"] = torch.zeros_like(st["table"]), torch.zeros_like(st["lens"])
    # a ring in mid-use: the free pages begin near its end and go on at its start
    head = count - spare // 2
    st["ring"] = torch.zeros(count, dtype=torch.int32, device="cuda")
    st["ring"][(torch.arange(spare, device="cuda") + head) % count] = free
    st["state"] = torch.tensor([head, spare], dtype=torch.int32, device="cuda")
    st["new_state"] = torch.zeros_like(st["state"])
    st["counts"] = None if case["new_hi"] == 1 else torch.tensor(counts, dtype=torch.int32, device="cuda")
    st["restart"] = torch.tensor(restart, device="cuda") if case["restart"] else None
    st["tokens"] = sum(counts) + case["pad"]
    st["offsets"] = torch.zeros(case["batch"] + 1, dtype=torch.int32, device="cuda")
    st["positions"] = torch.zeros(st["tokens"], dtype=torch.int32, device="cuda")
    st["slots"] = torch.zeros(st["tokens"], dtype=torch.int64, device="cuda")
    if own:
        import stream_compaction_pass_gb300 as ss
        st["seqs"], st["next"] = ss.KVTable(st["table"], st["lens"]), ss.KVTable(st["new_table"], st["new_lens"])
        st["free"] = ss.KVFree(st["ring"], st["state"])


def _prepare_rope(case, gen, st):
    n, hq, hk, dim, kind = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"], TYPES[case["type"]]

    def packed(heads):  # as a projection leaves them: a token's q, k and v side by side
        return torch.randn(n, heads, dim, generator=gen, dtype=kind, device="cuda")

    qkv = packed(hq + 2 * hk)
    qkv *= torch.rand(n, 1, 1, generator=gen, device="cuda").mul_(3).add_(0.2).to(kind)
    st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    st["qw"], st["kw"] = (torch.rand(dim, generator=gen, device="cuda").add_(0.5).to(kind) for _ in range(2))
    # sequences one after the other, the last one at far
    start = torch.randint(0, max(1, case["far"]), (1,), generator=gen, device="cuda")
    st["positions"] = ((torch.arange(n, device="cuda") + start) % (case["far"] + 1)).to(torch.int32)
    st["freq"] = torch.pow(torch.tensor(case["theta"], dtype=torch.float64, device="cuda"),
                           -torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
    if case["op"] == "back":
        grad = packed(hq + hk)
        st["gq"], st["gk"] = grad[:, :hq], grad[:, hq:]
        st["dq"], st["dk"] = torch.empty_like(st["q"], memory_format=torch.contiguous_format), torch.empty_like(st["k"], memory_format=torch.contiguous_format)
        st["dqw"], st["dkw"] = torch.empty(dim, device="cuda"), torch.empty(dim, device="cuda")
    else:
        st["yq"] = torch.empty(n, hq, dim, dtype=kind, device="cuda")
    if case["op"] == "rope":
        st["yk"] = torch.empty(n, hk, dim, dtype=kind, device="cuda")
    if case["op"] == "cached":
        page, count = case["page"], -(-n // case["page"]) + 3
        shape = (count, hk, page, dim)
        cache = TYPES[case["cache"]]
        st["kc"], st["vc"] = (torch.zeros(shape, dtype=torch.uint8 if case["cache"] == "e4m3" else cache, device="cuda").view(cache) for _ in range(2))
        st["weight"] = torch.ones(shape[:3], device="cuda")
        st["ks"], st["vs"] = (torch.rand(hk, generator=gen, device="cuda").add_(0.5) / 32 for _ in range(2)) if case["cache"] == "e4m3" else (None, None)
        # slots of shuffled pages; the last tokens of the call are padding
        pages = torch.randperm(count - 1, generator=gen, device="cuda")[:-(-n // page)]
        st["slots"] = (pages[:, None] * page + torch.arange(page, device="cuda")).flatten()[:n].contiguous()
        st["slots"][max(1, n - case["pad"]):] = -1
    if own:
        import stream_compaction_pass_gb300 as ss
        st["rope"] = ss.Rope(st["freq"], interleaved=case["interleaved"])
        if case["op"] == "cached":
            st["pages"] = ss.KVPages(st["kc"], st["vc"], weight=st["weight"], k_scale=st["ks"], v_scale=st["vs"])


def _prepare_attend(case, gen, st):
    heads, dim = case["heads"], case["dim"]
    st["table"], st["lens"], count, _ = _table(case, _lens(case), gen)
    shape = (count, heads, case["page"])
    # codes of blocks scaled to their largest element are spread nearly evenly
    st["k"], st["v"] = (torch.randint(0, 256, (*shape, dim // 2), generator=gen, dtype=torch.uint8, device="cuda") for _ in range(2))
    st["kb"], st["vb"] = (torch.rand(*shape, dim // 16, generator=gen, dtype=torch.float16, device="cuda").mul_(0.3).add_(0.2).to(TYPES["e4m3"]) for _ in range(2))
    st["ks"], st["vs"] = (torch.rand(heads, generator=gen, device="cuda").add_(0.5) for _ in range(2))
    kind = TYPES[case["type"]]
    st["q"] = torch.randn(case["batch"], heads * case["group"], dim, generator=gen, dtype=kind, device="cuda") * 2
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty(case["batch"], heads * case["group"], device="cuda")
    st["weight"] = st["weight_out"] = None
    if case["weights"]:
        st["weight"] = torch.randn(shape, generator=gen, device="cuda").mul_(2.5).sub_(8.0).exp_()
        st["weight_out"] = torch.zeros(shape, device="cuda")
    if own:
        import stream_compaction_pass_gb300 as ss
        st["pages"] = ss.KVPages(st["k"], st["v"], weight=st["weight"], k_scale=st["ks"], v_scale=st["vs"], k_block=st["kb"], v_block=st["vb"])
        st["seqs"] = ss.KVTable(st["table"], st["lens"], max_len=max(_lens(case)))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = {"case": case}
    {"assign": _prepare_assign, "attend": _prepare_attend}.get(case["op"], _prepare_rope)(case, gen, st)
    return st


def run(st):
    return (_own if own else _plain)[st["case"]["op"]](st)


# ---- page tables and slot maps ----

def _assign_outputs(st):
    return {"lens": st["new_lens"], "table": st["new_table"], "ring": st["ring"], "state": st["new_state"], "offsets": st["offsets"],
            "positions": st["positions"], "slots": st["slots"]}


def _assign_own(st):
    import stream_compaction_pass_gb300 as ss
    ss.ss_kv_assign(st["seqs"], st["free"], st["case"]["page"], counts=st["counts"], restart=st["restart"], into=st["next"], left=st["new_state"],
                    offsets=st["offsets"], positions=st["positions"], slots=st["slots"])
    return _assign_outputs(st)


def _assign_plain(st):
    page, ring = st["case"]["page"], st["ring"]
    lens = st["lens"].long()
    counts = torch.ones_like(lens) if st["counts"] is None else st["counts"].long()
    again = torch.zeros_like(lens, dtype=torch.bool) if st["restart"] is None else st["restart"]
    old = lens.masked_fill(again, 0)
    had, held = (lens + page - 1) // page, (old + page - 1) // page
    need = (old + counts + page - 1) // page - held
    upto = need.cumsum(0)
    head, free = st["state"][0].long(), st["state"][1].long()
    served = (need == 0) | (upto <= free)
    taken = (need * served).sum()
    new = old + counts * served
    # the new table: what is kept, then pages from the ring
    col = torch.arange(st["max_pages"], device="cuda")
    mine = (col >= held[:, None]) & (col < ((new + page - 1) // page)[:, None])
    fresh = ring[(head + (upto - need - held)[:, None] + col).clamp(min=0) % ring.numel()]
    kept = col < held[:, None]
    st["new_table"].copy_(torch.where(mine, fresh, torch.where(kept, st["table"], st["new_table"])))
    # pages given back
    back = had * again
    upto_back = back.cumsum(0)
    gives = col < back[:, None]
    to = (head + free + (upto_back - back)[:, None] + col) % ring.numel()
    ring[to[gives]] = st["table"][gives]
    st["new_state"].copy_(torch.stack([(head + taken) % ring.numel(), free - taken + upto_back[-1]]))
    st["new_lens"].copy_(new)
    st["offsets"][1:] = counts.cumsum(0)
    # tokens
    token, ends = torch.arange(st["tokens"], device="cuda"), st["offsets"][1:].long()
    real = token < ends[-1]
    seq = torch.searchsorted(ends, token, right=True).clamp(max=ends.numel() - 1)
    pos = (old[seq] + token - (ends - counts)[seq]).masked_fill(~real, 0)
    place = st["new_table"][seq, (pos // page).clamp(max=st["max_pages"] - 1)].long() * page + pos % page
    st["positions"].copy_(pos)
    st["slots"].copy_(place.masked_fill(~real | ~served[seq], -1))
    return _assign_outputs(st)


def _assign_exact(case, st):
    page, lens, (counts, restart) = case["page"], _lens(case), _asked(case)
    table, ring, (head, free) = st["table"].cpu().tolist(), st["ring"].cpu().tolist(), st["state"].cpu().tolist()
    out = [[0] * st["max_pages"] for _ in lens]
    offsets, new, positions, slots, at, tail = [0], [], [], [], 0, head + free
    pages = lambda n: -(-n // page)  # noqa: E731
    gone = []
    short = False
    for b, (n, c, again) in enumerate(zip(lens, counts, restart)):
        if again:
            gone += table[b][:pages(n)]
            n = 0
        need = pages(n + c) - pages(n)
        out[b][:pages(n)] = table[b][:pages(n)]
        short = short or at + need > free
        ok = need == 0 or not short
        if ok:
            out[b][pages(n):pages(n + c)] = [ring[(head + at + i) % len(ring)] for i in range(need)]
            at += need
        new.append(n + c if ok else n)
        offsets.append(offsets[-1] + c)
        positions += range(n, n + c)
        slots += [out[b][p // page] * page + p % page for p in range(n, n + c)] if ok else [-1] * c
    for p in gone:
        ring[tail % len(ring)] = p
        tail += 1
    pad = case["pad"]
    whole = lambda x, kind=torch.int32: torch.tensor(x, dtype=kind, device="cuda")  # noqa: E731
    return {"lens": whole(new), "table": whole(out), "ring": whole(ring), "state": whole([(head + at) % len(ring), free - at + len(gone)]),
            "offsets": whole(offsets), "positions": whole(positions + [0] * pad), "slots": whole(slots + [-1] * pad, torch.int64)}


# ---- norms and rotation ----

def _angles(st):
    a = st["positions"].double()[:, None, None] * st["freq"]
    return a.cos().float(), a.sin().float()


def _halves(st, x):
    """What is turned, as its two parts, and the rest."""
    r = st["case"]["rot"]
    t = x[..., :r]
    if st["case"]["interleaved"]:
        return t[..., 0::2], t[..., 1::2], x[..., r:]
    return t[..., :r // 2], t[..., r // 2:], x[..., r:]


def _whole(st, a, b, rest):
    t = torch.stack([a, b], -1).flatten(-2) if st["case"]["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([t, rest], -1)


def _turned(st, x, back=False):
    cos, sin = _angles(st)
    if back:
        sin = -sin
    a, b, rest = _halves(st, x)
    return _whole(st, a * cos - b * sin, b * cos + a * sin, rest)


def _rope_rows(st, x, w):
    x = x.float()
    return _turned(st, x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w.float())


def _rope_plain(st):
    st["yq"].copy_(_rope_rows(st, st["q"], st["qw"]))
    st["yk"].copy_(_rope_rows(st, st["k"], st["kw"]))
    return {"q": st["yq"], "k": st["yk"]}


def _rope_own(st):
    import stream_compaction_pass_gb300 as ss
    ss.ss_qk_norm_rope(st["q"], st["k"], st["qw"], st["kw"], st["rope"], st["positions"], st["yq"], st["yk"], eps=EPS)
    return {"q": st["yq"], "k": st["yk"]}


def _back_rows(st, x, w, g, dx, dw):
    x, w = x.float(), w.float()
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    g, x = _turned(st, g.float(), back=True), x * r
    dw.copy_((g * x).sum((0, 1)))
    g = g * w
    dx.copy_(r * (g - x * (g * x).mean(-1, keepdim=True)))


def _back_plain(st):
    _back_rows(st, st["q"], st["qw"], st["gq"], st["dq"], st["dqw"])
    _back_rows(st, st["k"], st["kw"], st["gk"], st["dk"], st["dkw"])
    return {"q": st["dq"], "k": st["dk"], "q_weight": st["dqw"], "k_weight": st["dkw"]}


def _back_own(st):
    import stream_compaction_pass_gb300 as ss
    ss.ss_qk_norm_rope_backward(st["gq"], st["gk"], st["q"], st["k"], st["qw"], st["kw"], st["rope"], st["positions"], st["dq"], st["dk"],
                                st["dqw"], st["dkw"], eps=EPS)
    return {"q": st["dq"], "k": st["dk"], "q_weight": st["dqw"], "k_weight": st["dkw"]}


def _cached_outputs(st):
    return {"q": st["yq"], "k": st["kc"], "v": st["vc"], "weight": st["weight"]}


def _cached_plain(st):
    st["yq"].copy_(_rope_rows(st, st["q"], st["qw"]))
    page = st["case"]["page"]
    slots = st["slots"].masked_fill(st["slots"] < 0, (st["kc"].shape[0] - 1) * page)  # the last page is nobody's: it stays zero
    at, slot, there = slots // page, slots % page, (st["slots"] >= 0)[:, None, None]
    for x, pool, scale in ((_rope_rows(st, st["k"], st["kw"]), st["kc"], st["ks"]), (st["v"].float(), st["vc"], st["vs"])):
        if scale is None:
            x = (x * there).to(pool.dtype)
        else:
            x = ((x / scale[:, None]).clamp(-448.0, 448.0) * there).to(pool.dtype).view(torch.uint8)
            pool = pool.view(torch.uint8)
        pool.transpose(1, 2)[at, slot] = x
    st["weight"].transpose(1, 2)[at, slot] = (~there[:, :, 0]).float().expand(-1, st["case"]["kv_heads"])
    return _cached_outputs(st)


def _cached_own(st):
    import stream_compaction_pass_gb300 as ss
    ss.ss_kv_append_rope(st["pages"], st["slots"], st["q"], st["k"], st["v"], st["qw"], st["kw"], st["rope"], st["positions"], st["yq"], eps=EPS)
    return _cached_outputs(st)


def _exact_turn(case, st, x, sign):
    """Rows as complex numbers, turned by exp(sign i p f)."""
    r = case["rot"]
    if case["interleaved"]:
        z = torch.view_as_complex(x[..., :r].reshape(*x.shape[:-1], r // 2, 2).contiguous())
    else:
        z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:r].contiguous())
    z = z * torch.exp(sign * 1j * st["positions"].double()[:, None] * st["freq"])[:, None]
    y = torch.view_as_real(z).flatten(-2) if case["interleaved"] else torch.cat([z.real, z.imag], -1)
    return torch.cat([y, x[..., r:]], -1)


def _exact_rows(case, st, x, w):
    x = x.double()
    norm = torch.sqrt(torch.mean(x ** 2, -1) + EPS)[..., None]
    return _exact_turn(case, st, w.double() * x / norm, 1)


def _rope_exact(case, st):
    return {"q": _exact_rows(case, st, st["q"], st["qw"]), "k": _exact_rows(case, st, st["k"], st["kw"])}


def _back_exact(case, st):
    got = {}
    for name, x, w, g in (("q", st["q"], st["qw"], st["gq"]), ("k", st["k"], st["kw"], st["gk"])):
        x, w = x.double(), w.double()
        norm = torch.sqrt(torch.mean(x ** 2, -1) + EPS)[..., None]
        g = _exact_turn(case, st, g.double(), -1)
        # y = w x / n with n^2 = mean(x^2) + eps: dx = w g / n - x sum(w g x) / (D n^3)
        got[name] = w * g / norm - x * torch.sum(w * g * x, -1, keepdim=True) / (case["dim"] * norm ** 3)
        got[name + "_weight"] = torch.sum(g * x / norm, (0, 1))
    return {n: got[n] for n in ("q", "k", "q_weight", "k_weight")}


def _e4m3(x):
    """The nearest e4m3 value (4 exponent bits of bias 7, 3 of fraction), ties to even, as 64-bit numbers."""
    a = x.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
    return torch.copysign((a / step).round() * step, x)


def _cached_exact(case, st):
    keep = st["slots"] >= 0
    at, slot = st["slots"][keep] // case["page"], st["slots"][keep] % case["page"]
    got = {"q": _exact_rows(case, st, st["q"], st["qw"]), "weight": st["weight"].double()}
    for name, x, scale in (("k", _exact_rows(case, st, st["k"], st["kw"]), st["ks"]), ("v", st["v"].double(), st["vs"])):
        got[name] = torch.zeros(st["kc"].shape, dtype=torch.float64, device="cuda")
        got[name][at, :, slot] = x[keep] if scale is None else _e4m3(x[keep] / scale.double()[:, None])
    got["weight"][at, :, slot] = 0.0
    return {n: got[n] for n in ("q", "k", "v", "weight")}


# ---- attention over 4 bits ----

def _e2m1(codes):
    """The values of packed codes, the low half of a byte first."""
    values = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device="cuda")
    return torch.stack([values[(codes & 15).int()], values[(codes >> 4).int()]], -1).flatten(-2)


def _rows(codes, blocks, scale):
    return (_e2m1(codes).unflatten(-1, (-1, 16)) * blocks.float()[..., None]).flatten(-2) * scale


def _attend_outputs(st):
    got = {"out": st["out"], "lse": st["lse"]}
    if st["weight_out"] is not None:
        got["weight"] = st["weight_out"][:-1]
    return got


def _attend_plain(st):
    c = st["case"]
    page, batch = c["page"], c["batch"]
    pos = torch.arange(st["table"].shape[1] * page, device="cuda").expand(batch, -1)
    real = pos < st["lens"][:, None]
    seen = real if not c["window"] else real & ((pos < c["sinks"]) | (pos >= st["lens"][:, None] - c["window"]))
    table = st["table"].long()

    def rows(codes, blocks, scale):  # batch, head, position, dim
        return _rows(codes[table].transpose(1, 2).flatten(2, 3), blocks.view(torch.uint8)[table].view(blocks.dtype).transpose(1, 2).flatten(2, 3), scale[:, None, None])

    seen = seen[:, None, None]
    q = st["q"].float().unflatten(1, (c["heads"], c["group"]))
    s = (q @ rows(st["k"], st["kb"], st["ks"]).transpose(2, 3)) * (1.0 / math.sqrt(c["dim"]))
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(3, keepdim=True)
    p = (s - top.masked_fill(top == -math.inf, 0.0)).exp()
    total = p.sum(3, keepdim=True)
    p = p / total.masked_fill(total == 0, 1.0)
    st["out"].copy_((p @ rows(st["v"], st["vb"], st["vs"])).flatten(1, 2))
    st["lse"].copy_((total.log() + top).flatten(1))
    if st["weight_out"] is not None:
        at = table.gather(1, pos // page).masked_fill(~real, st["k"].shape[0] - 1)[:, None]
        slot, heads = (pos % page)[:, None], torch.arange(c["heads"], device="cuda")[None, :, None]
        st["weight_out"][at, heads, slot] = st["weight"][at, heads, slot] + p.sum(2)
    return _attend_outputs(st)


def _attend_own(st):
    import stream_compaction_pass_gb300 as ss
    c = st["case"]
    ss.ss_kv_attend(st["pages"], st["seqs"], st["q"], st["out"], window=c["window"], sinks=c["sinks"], lse=st["lse"], weight_in=st["weight"],
                    weight_out=st["weight_out"])
    return _attend_outputs(st)


def _attend_exact(case, st):
    G, H, D = case["group"], case["heads"], case["dim"]
    out = torch.zeros(case["batch"], H * G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"], H * G), -math.inf, dtype=torch.float64, device="cuda")
    weight = None if st["weight_out"] is None else st["weight_out"].double()
    # a code's sign, two bits of exponent and one of fraction; a table of all bytes' two values
    byte = torch.arange(256, device="cuda")

    def value(n):
        e, m = (n >> 1) & 3, n & 1
        return torch.where(n > 7, -1.0, 1.0).double() * torch.where(e > 0, 2.0 ** (e.double() - 1) * (1 + m / 2), m / 2)

    both = torch.stack([value(byte & 15), value(byte >> 4)], 1)

    def rows(codes, blocks, scale, page, h, slot):
        x = both[codes[page, h, slot].long()].reshape(-1, D // 16, 16)
        return (x * blocks.view(torch.uint8)[page, h, slot].view(blocks.dtype).double()[:, :, None]).reshape(-1, D) * scale[h].double()

    for b, n in enumerate(_lens(case)):
        pos = torch.arange(n, device="cuda")
        if case["window"]:
            pos = pos[(pos < case["sinks"]) | (pos >= n - case["window"])]
        page, slot = st["table"][b].long()[pos // case["page"]], pos % case["page"]
        if weight is not None:
            every = torch.arange(n, device="cuda")
            at, to = st["table"][b].long()[every // case["page"]], every % case["page"]
            weight[at, :, to] = st["weight"][at, :, to].double()
        for h in range(H):
            q = st["q"][b, h * G:(h + 1) * G].double()
            s = torch.mm(q, rows(st["k"], st["kb"], st["ks"], page, h, slot).t()) / math.sqrt(D)
            norm = torch.logsumexp(s, 1)
            w = torch.exp(s - norm[:, None])
            out[b, h * G:(h + 1) * G] = torch.mm(w, rows(st["v"], st["vb"], st["vs"], page, h, slot))
            lse[b, h * G:(h + 1) * G] = norm
            if weight is not None:
                weight[page, h, slot] += w.sum(0)
    got = {"out": out, "lse": lse}
    if weight is not None:
        got["weight"] = weight[:-1]
    return got


_plain = {"assign": _assign_plain, "rope": _rope_plain, "back": _back_plain, "cached": _cached_plain, "attend": _attend_plain}
_own = {"assign": _assign_own, "rope": _rope_own, "back": _back_own, "cached": _cached_own, "attend": _attend_own}


def work(case):
    """Bytes that have to move, each once, and the arithmetic on the rows."""
    if case["op"] == "assign":
        page, lens, (counts, restart) = case["page"], _lens(case), _asked(case)
        pages = lambda n: -(-n // page)  # noqa: E731
        entries = sum(2 * pages(n) + 2 * (pages((0 if r else n) + c) - (0 if r else pages(n))) for n, c, r in zip(lens, counts, restart))
        tokens = sum(counts) + case["pad"]
        return {"bytes": 4 * entries + 12 * tokens + 16 * case["batch"], "flops": 0}
    if case["op"] == "attend":
        H, D, lens, W = case["heads"], case["dim"], _lens(case), case["window"]
        seen = [n if not W or n <= W else min(n, W + min(case["sinks"], n - W)) for n in lens]
        rows = case["batch"] * H * case["group"]
        data = sum(seen) * H * (D // 2 + D // 16) * 2 + rows * (D * 2 * 2 + 4) + 4 * sum(1 + -(-n // case["page"]) for n in lens)
        if case["weights"]:
            data += 8 * H * sum(lens)
        return {"bytes": data, "flops": 4 * sum(seen) * H * case["group"] * D}
    n, hq, hk, D, size = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"], SIZE[case["type"]]
    if case["op"] == "rope":
        return {"bytes": n * ((hq + hk) * D * size * 2 + 4) + 2 * D * size, "flops": 8 * n * (hq + hk) * D}
    if case["op"] == "back":
        return {"bytes": n * ((hq + hk) * D * size * 3 + 4) + 2 * D * (size + 4), "flops": 16 * n * (hq + hk) * D}
    there = max(1, n - case["pad"]) if case["pad"] else n
    return {"bytes": n * (hq * D * size * 2 + 12) + there * hk * (2 * D * (size + SIZE[case["cache"]]) + 4) + 2 * D * size, "flops": 8 * n * (hq + hk) * D}


def exact(case, seed):
    st = prepare(case, seed)
    return {"assign": _assign_exact, "rope": _rope_exact, "back": _back_exact, "cached": _cached_exact, "attend": _attend_exact}[case["op"]](case, st)
