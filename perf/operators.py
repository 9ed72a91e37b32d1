"""The paged key-value cache operators, as they are measured: appending new
tokens to the cache (`append`), attention of one new token per sequence over
it (`attend`), and eviction of the least attended tokens into fresh pages
(`evict`).

With ``own = False`` `run` computes an operator in its plain form, elementary
torch operations in 32 bits rounded once at the end; with ``own = True`` it
makes the calls a user of the library makes.  `exact` computes the same
outputs in 64 bits from the definitions, one sequence at a time.

Definitions (b a sequence of len tokens, h a key-value head, g one of the
`group` query heads that share it, position p at slot p % page of page
table[b, p // page]):

  append   a row x of k or v goes to its slot as it is, or, in an 8-bit
           cache, as e4m3(clamp(x / scale[h], -448, 448)), ties to even; the
           slot's weight becomes 0.
  attend   s(p) = softscale * q . k(p) over the visible positions
           {p < len : p < sinks or p >= len - window} (window 0: all),
           w = exp(s - max) / sum, out = sum_p w(p) v(p),
           lse = log(sum_p exp(s(p))), and, where weights are kept,
           weight_out(h, p) = weight_in(h, p) + sum_g w_g(p).
           No visible position: out = 0 and lse = -inf.
  evict    keeps min(len, keep) positions of every (b, h): the first `sinks`,
           the last `recent`, and of the others those of the largest weight,
           ties to the lower position; the kept rows of k, v and weight go to
           the pages of the new table in the order of their positions.
"""

import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f16": 2, "e4m3": 1}


def listed():
    return [
        # One short conversation on its own: what a token waits for is latency.
        {"name": "attend_one_short", "op": "attend", "batch": 1, "lo": 517, "hi": 517, "heads": 8, "group": 4, "dim": 128,
         "page": 16, "cache": "bf16", "q": "bf16", "window": 0, "sinks": 0, "weights": False, "lens": 1},
        # An ordinary serving batch of ragged lengths that keeps the weights for a later eviction.
        {"name": "attend_batch", "op": "attend", "batch": 64, "lo": 100, "hi": 8191, "heads": 8, "group": 4, "dim": 128,
         "page": 16, "cache": "bf16", "q": "bf16", "window": 0, "sinks": 0, "weights": True, "lens": 2},
        # One very long document: few rows, all the parallelism is along the cache.
        {"name": "attend_one_long", "op": "attend", "batch": 1, "lo": 131071, "hi": 131071, "heads": 8, "group": 8, "dim": 128,
         "page": 64, "cache": "f16", "q": "f16", "window": 0, "sinks": 0, "weights": True, "lens": 3},
        # A full machine: many long sequences, several gigabytes of cache read for one token each.
        {"name": "attend_large", "op": "attend", "batch": 32, "lo": 20000, "hi": 50000, "heads": 8, "group": 4, "dim": 128,
         "page": 64, "cache": "bf16", "q": "bf16", "window": 0, "sinks": 0, "weights": True, "lens": 4},
        # The cache held in 8 bits with a scale for each head.
        {"name": "attend_8bit", "op": "attend", "batch": 48, "lo": 900, "hi": 16001, "heads": 8, "group": 8, "dim": 128,
         "page": 32, "cache": "e4m3", "q": "bf16", "window": 0, "sinks": 0, "weights": False, "lens": 5},
        # Streaming decode: a window and a few first tokens of long histories; every query head its own keys, narrow heads.
        {"name": "attend_window", "op": "attend", "batch": 96, "lo": 3000, "hi": 30011, "heads": 12, "group": 1, "dim": 64,
         "page": 16, "cache": "bf16", "q": "bf16", "window": 2047, "sinks": 4, "weights": False, "lens": 6},
        # One conversation over its budget: a small call between two tokens.
        {"name": "evict_one", "op": "evict", "batch": 1, "lo": 2049, "hi": 2049, "heads": 8, "dim": 128, "page": 16,
         "cache": "bf16", "keep": 1024, "sinks": 4, "recent": 256, "lens": 7},
        # A serving batch brought back under its budget, some sequences still below it.
        {"name": "evict_batch", "op": "evict", "batch": 24, "lo": 1000, "hi": 9001, "heads": 8, "dim": 128, "page": 32,
         "cache": "bf16", "keep": 2048, "sinks": 4, "recent": 512, "lens": 8},
        # Long documents after their prompts: a large cut of an 8-bit cache.
        {"name": "evict_large", "op": "evict", "batch": 16, "lo": 60000, "hi": 131072, "heads": 8, "dim": 128, "page": 64,
         "cache": "e4m3", "keep": 32000, "sinks": 16, "recent": 4096, "lens": 9},
        # One token of every sequence of a batch enters the cache before its attention.
        {"name": "append_tokens", "op": "append", "batch": 64, "lo": 100, "hi": 4000, "new_lo": 1, "new_hi": 1, "heads": 8,
         "dim": 128, "page": 16, "cache": "bf16", "src": "bf16", "lens": 10},
        # Whole prompts enter an 8-bit cache, quantised on the way.
        {"name": "append_prompts", "op": "append", "batch": 16, "lo": 1000, "hi": 20000, "new_lo": 1000, "new_hi": 16383, "heads": 8,
         "dim": 128, "page": 32, "cache": "e4m3", "src": "bf16", "lens": 11},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _lens(case):
    """The sequences' lengths: spread over the logarithm between lo and hi, the first one hi."""
    rng = random.Random(case["lens"])
    lens = [case["hi"]] + [_log_int(rng, case["lo"], case["hi"]) for _ in range(case["batch"] - 1)]
    rng.shuffle(lens)
    return lens


def _news(case):
    """append: how many of each sequence's tokens are new (the last ones)."""
    rng = random.Random(case["lens"] + 1)
    return [min(n, _log_int(rng, case["new_lo"], case["new_hi"])) for n in _lens(case)]


def draw(rng):
    most = max(work(c)["bytes"] for c in listed() if c["op"] == "attend")
    while True:
        case = {"op": rng.choice(["attend", "attend", "evict", "append"]), "batch": _log_int(rng, 1, 96),
                "heads": rng.choice([1, 2, 4, 8, 12]), "dim": rng.choice([64, 64, 80, 128, 128, 128, 256]),
                "page": rng.choice([8, 16, 16, 32, 64, 128]), "cache": rng.choice(["bf16", "bf16", "f16", "e4m3"]),
                "lens": rng.randrange(1 << 30)}
        case["hi"] = _log_int(rng, 500, 131072)
        case["lo"] = max(1, case["hi"] // rng.choice([1, 2, 5, 20]))
        if case["op"] == "attend":
            case["q"] = rng.choice(["bf16", "f16"]) if case["cache"] == "e4m3" else case["cache"]
            case["group"] = rng.choice([1, 2, 4, 5, 8, 16])
            case["window"], case["sinks"] = rng.choice([(0, 0), (0, 0), (_log_int(rng, 100, 8000), rng.choice([0, 1, 4, 20]))])
            case["weights"] = rng.random() < 0.5
        elif case["op"] == "evict":
            case["keep"] = max(32, int(case["hi"] * rng.uniform(0.1, 0.7)))
            case["sinks"] = rng.choice([0, 4, 16])
            case["recent"] = int(case["keep"] * rng.uniform(0.0, 0.4))
        else:
            case["src"] = rng.choice(["bf16", "f16"]) if case["cache"] == "e4m3" else case["cache"]
            case["new_lo"], case["new_hi"] = rng.choice([(1, 1), (1, case["hi"]), (max(1, case["hi"] // 4), case["hi"])])
        rows = sum(_lens(case)) * case["heads"] * case["dim"] * SIZE[case["cache"]] * 2
        if rows <= most and 1 << 16 <= work(case)["bytes"] <= most:
            return case


def _pool(case, count, gen, empty=False):
    """k, v and weight pools of `count` pages."""
    shape = (count, case["heads"], case["page"], case["dim"])
    kind = TYPES[case["cache"]]
    if empty:
        k, v = (torch.zeros(shape, dtype=torch.uint8 if case["cache"] == "e4m3" else kind, device="cuda").view(kind) for _ in range(2))
        return k, v, torch.zeros(shape[:3], device="cuda")
    half = torch.bfloat16 if case["cache"] == "e4m3" else kind
    k, v = (torch.randn(shape, generator=gen, dtype=half, device="cuda") for _ in range(2))
    if case["cache"] == "e4m3":  # stored as values / scale, scales near 1 / 32
        k, v = k.mul_(32).to(kind), v.mul_(32).to(kind)
    # what tokens have gathered is spread over orders of magnitude; some have gathered nothing
    weight = torch.randn(shape[:3], generator=gen, device="cuda").mul_(2.5).sub_(8.0).exp_()
    weight[torch.rand(shape[:3], generator=gen, device="cuda") < 0.1] = 0.0
    return k, v, weight


def _table(case, lens, gen, extra=0):
    """A page table of the sequences over a shuffled pool, and the pool's page count."""
    need = [-(-n // case["page"]) for n in lens]
    count = sum(need) + 1 + extra  # the last pages are nobody's
    ids = torch.randperm(count - 1 - extra, generator=gen, device="cuda").to(torch.int32).cpu()
    table = torch.zeros(len(lens), max(need), dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = ids[at:at + m]
        at += m
    return table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), count


def _scales(case, gen):
    if case["cache"] != "e4m3":
        return None, None
    return tuple((torch.rand(case["heads"], generator=gen, device="cuda") + 0.5) / 32 for _ in range(2))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    lens = _lens(case)
    st = {"case": case}
    st["table"], st["lens"], count = _table(case, lens, gen)
    st["ks"], st["vs"] = _scales(case, gen)
    st["k"], st["v"], st["weight"] = _pool(case, count, gen, empty=case["op"] == "append")
    H, D = case["heads"], case["dim"]
    if case["op"] == "attend":
        kind = TYPES[case["q"]]
        st["q"] = torch.randn(case["batch"], H * case["group"], D, generator=gen, dtype=kind, device="cuda") * 2
        st["out"] = torch.empty_like(st["q"])
        st["lse"] = torch.empty(case["batch"], H * case["group"], device="cuda")
        st["weight_out"] = torch.zeros_like(st["weight"]) if case["weights"] else None
    elif case["op"] == "evict":
        kept = [min(n, case["keep"]) for n in lens]
        st["new_table"], st["new_lens"], st["count"] = _table(case, kept, gen)
        st["new_k"], st["new_v"], st["new_weight"] = _pool(case, st["count"], gen, empty=True)
        st["kept"] = torch.empty(case["batch"], H, case["keep"], dtype=torch.int32, device="cuda")
    else:
        news = _news(case)
        offsets = [0]
        for n in news:
            offsets.append(offsets[-1] + n)
        st["offsets"] = None if case["new_hi"] == 1 else torch.tensor(offsets, dtype=torch.int32, device="cuda")
        st["tokens"] = offsets[-1]
        # as a projection leaves them: q, k and v of a token side by side
        qkv = torch.randn(offsets[-1], 3, H, D, generator=gen, dtype=TYPES[case["src"]], device="cuda")
        st["k_new"], st["v_new"] = qkv[:, 1], qkv[:, 2]
    if own:
        import stream_compaction_pass_gb300 as ss
        st["pages"] = ss.KVPages(st["k"], st["v"], weight=st["weight"], k_scale=st["ks"], v_scale=st["vs"])
        st["seqs"] = ss.KVTable(st["table"], st["lens"], max_len=max(lens))
        if case["op"] == "evict":
            st["new_pages"] = ss.KVPages(st["new_k"], st["new_v"], weight=st["new_weight"], k_scale=st["ks"], v_scale=st["vs"])
            st["new_seqs"] = ss.KVTable(st["new_table"], st["new_lens"], max_len=case["keep"])
    return st


def run(st):
    return (_own if own else _plain)[st["case"]["op"]](st)


def _attend_own(st):
    import stream_compaction_pass_gb300 as ss
    c = st["case"]
    w = st["weight_out"]
    ss.ss_kv_attend(st["pages"], st["seqs"], st["q"], st["out"], window=c["window"], sinks=c["sinks"], lse=st["lse"],
                    weight_in=None if w is None else st["weight"], weight_out=w)
    return _attend_outputs(st)


def _attend_outputs(st):
    got = {"out": st["out"], "lse": st["lse"]}
    if st["weight_out"] is not None:
        got["weight"] = st["weight_out"][:-1]
    return got


def _evict_own(st):
    import stream_compaction_pass_gb300 as ss
    c = st["case"]
    ss.ss_kv_evict(st["pages"], st["seqs"], st["new_pages"], st["new_seqs"], c["keep"], sinks=c["sinks"], recent=c["recent"], kept=st["kept"])
    return _evict_outputs(st)


def _evict_outputs(st):
    return {"k": st["new_k"][:-1], "v": st["new_v"][:-1], "weight": st["new_weight"][:-1], "lens": st["new_lens"], "kept": st["kept"]}


def _append_own(st):
    import stream_compaction_pass_gb300 as ss
    ss.ss_kv_append(st["pages"], st["seqs"], st["k_new"], st["v_new"], offsets=st["offsets"])
    return {"k": st["k"][:-1], "v": st["v"][:-1], "weight": st["weight"][:-1]}


def _positions(st):
    """(batch, longest) positions, which of them exist, and their pages and slots (those that do not: the pool's last page)."""
    page = st["case"]["page"]
    pos = torch.arange(st["table"].shape[1] * page, device="cuda").expand(st["table"].shape[0], -1)
    real = pos < st["lens"][:, None]
    at = st["table"].long().gather(1, pos // page).masked_fill(~real, st["k"].shape[0] - 1)
    return pos, real, at, pos % page


def _attend_plain(st):
    c = st["case"]
    pos, real, at, slot = _positions(st)
    seen = real if not c["window"] else real & ((pos < c["sinks"]) | (pos >= st["lens"][:, None] - c["window"]))
    table = st["table"].long()

    def rows(pool, scale):
        x = pool[table].transpose(1, 2).flatten(2, 3).float()  # batch, head, position, dim
        return x if scale is None else x.mul_(scale[:, None, None])

    seen = seen[:, None, None]
    q = st["q"].float().unflatten(1, (c["heads"], c["group"]))
    s = (q @ rows(st["k"], st["ks"]).transpose(2, 3)) * (1.0 / math.sqrt(c["dim"]))
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(3, keepdim=True)
    p = (s - top.masked_fill(top == -math.inf, 0.0)).exp()
    total = p.sum(3, keepdim=True)
    p = p / total.masked_fill(total == 0, 1.0)
    v = rows(st["v"], st["vs"]).mul_(real[:, None, :, None])
    st["out"].copy_((p @ v).flatten(1, 2))
    st["lse"].copy_((total.log() + top).flatten(1))
    if st["weight_out"] is not None:
        at, slot, heads = at[:, None], slot[:, None], torch.arange(c["heads"], device="cuda")[None, :, None]
        st["weight_out"][at, heads, slot] = st["weight"][at, heads, slot] + p.sum(2)
    return _attend_outputs(st)


def _evict_plain(st):
    c = st["case"]
    pos, real, at, slot = _positions(st)
    heads = torch.arange(c["heads"], device="cuda")[None, :, None]
    rank = st["weight"][at[:, None], heads, slot[:, None]]
    forced = real & ((pos < c["sinks"]) | (pos >= st["lens"][:, None] - c["recent"]))
    rank = rank.masked_fill(forced[:, None], math.inf).masked_fill(~real[:, None], -math.inf)
    first = rank.sort(dim=2, descending=True, stable=True)[1][:, :, :c["keep"]]
    lens = st["lens"].clamp(max=c["keep"])
    j = torch.arange(first.shape[2], device="cuda")
    here = (j < lens[:, None])[:, None]
    first = first.masked_fill(~here, pos.shape[1]).sort(2)[0]
    st["kept"].fill_(-1)
    st["kept"][:, :, :first.shape[2]] = first.masked_fill(~here, -1).int()
    first = first.clamp(max=pos.shape[1] - 1)
    seq = torch.arange(c["batch"], device="cuda")[:, None, None]
    src, from_slot = at[seq, first], first % c["page"]
    most = st["new_table"].shape[1] * c["page"]
    dst = st["new_table"].long()[:, (j // c["page"]).clamp(max=st["new_table"].shape[1] - 1)].masked_fill(~here[:, 0], st["count"] - 1)[:, None]
    to_slot = (j % c["page"]).masked_fill(j >= most, 0)
    bits = (lambda x: x.view(torch.uint8)) if c["cache"] == "e4m3" else (lambda x: x)
    for old, new in ((bits(st["k"]), bits(st["new_k"])), (bits(st["v"]), bits(st["new_v"])), (st["weight"], st["new_weight"])):
        new[dst, heads, to_slot] = old[src, heads, from_slot]
    st["new_lens"].copy_(lens)
    return _evict_outputs(st)


def _append_plain(st):
    c = st["case"]
    token = torch.arange(st["tokens"], device="cuda")
    if st["offsets"] is None:
        seq, pos = token, st["lens"].long() - 1
    else:
        ends = st["offsets"][1:].long()
        seq = (token[:, None] >= ends).sum(1)
        pos = st["lens"].long()[seq] - ends[seq] + token
    at, slot = st["table"].long()[seq, pos // c["page"]], pos % c["page"]
    for new, pool, scale in ((st["k_new"], st["k"], st["ks"]), (st["v_new"], st["v"], st["vs"])):
        x = new
        if scale is not None:
            x = (new.float() / scale[:, None]).clamp(-448.0, 448.0).to(pool.dtype).view(torch.uint8)
            pool = pool.view(torch.uint8)
        pool.transpose(1, 2)[at, slot] = x
    st["weight"].transpose(1, 2)[at, slot] = 0.0
    return {"k": st["k"][:-1], "v": st["v"][:-1], "weight": st["weight"][:-1]}


_plain = {"attend": _attend_plain, "evict": _evict_plain, "append": _append_plain}
_own = {"attend": _attend_own, "evict": _evict_own, "append": _append_own}


def work(case):
    """Bytes that have to move, each once, and the multiplies and adds of the two products."""
    H, D, size = case["heads"], case["dim"], SIZE[case["cache"]]
    lens = _lens(case)
    tables = 4 * sum(1 + -(-n // case["page"]) for n in lens)
    if case["op"] == "attend":
        W = case["window"]
        seen = [n if not W or n <= W else min(n, W + min(case["sinks"], n - W)) for n in lens]
        rows = case["batch"] * H * case["group"]
        data = sum(seen) * H * D * size * 2 + rows * (D * 2 * 2 + 4)
        if case["weights"]:
            data += 8 * H * sum(lens)
        return {"bytes": data + tables, "flops": 4 * sum(seen) * H * case["group"] * D}
    if case["op"] == "evict":
        kept = sum(min(n, case["keep"]) for n in lens)
        data = 4 * H * sum(lens) + H * kept * (2 * 2 * D * size + 4) + 4 * case["batch"] * H * case["keep"]
        return {"bytes": data + tables + 4 * sum(1 + -(-min(n, case["keep"]) // case["page"]) for n in lens), "flops": 0}
    new = sum(_news(case))
    return {"bytes": new * H * (2 * D * (2 + size) + 4) + tables, "flops": 0}


def exact(case, seed):
    st = prepare(case, seed)
    return {"attend": _attend_exact, "evict": _evict_exact, "append": _append_exact}[case["op"]](case, st)


def _row_index(case, st, b, n):
    pos = torch.arange(n, device="cuda")
    return pos, st["table"][b].long()[pos // case["page"]], pos % case["page"]


def _attend_exact(case, st):
    G, H, D = case["group"], case["heads"], case["dim"]
    out = torch.zeros(case["batch"], H * G, D, dtype=torch.float64, device="cuda")
    lse = torch.full((case["batch"], H * G), -math.inf, dtype=torch.float64, device="cuda")
    weight = None if st["weight_out"] is None else st["weight_out"].double()
    one = torch.ones(H, dtype=torch.float64, device="cuda")
    ks, vs = (one if s is None else s.double() for s in (st["ks"], st["vs"]))
    for b, n in enumerate(_lens(case)):
        pos, page, slot = _row_index(case, st, b, n)
        keep = torch.ones_like(pos, dtype=torch.bool)
        if case["window"]:
            keep = (pos < case["sinks"]) | (pos >= n - case["window"])
        idx = pos[keep]
        for h in range(H):
            k = st["k"][page[idx], h, slot[idx]].double() * ks[h]
            v = st["v"][page[idx], h, slot[idx]].double() * vs[h]
            q = st["q"][b, h * G:(h + 1) * G].double()
            s = torch.mm(q, k.t()) / math.sqrt(D)
            norm = torch.logsumexp(s, 1)
            w = torch.exp(s - norm[:, None])
            out[b, h * G:(h + 1) * G] = torch.mm(w, v)
            lse[b, h * G:(h + 1) * G] = norm
            if weight is not None:
                weight[page, h, slot] = st["weight"][page, h, slot].double()
                weight[page[idx], h, slot[idx]] += w.sum(0)
    got = {"out": out, "lse": lse}
    if weight is not None:
        got["weight"] = weight[:-1]
    return got


def _evict_exact(case, st):
    keep, H = case["keep"], case["heads"]
    lens = torch.tensor([min(n, keep) for n in _lens(case)], dtype=torch.int32)
    kept = torch.full((case["batch"], H, keep), -1, dtype=torch.int32)
    weight = torch.zeros(st["new_weight"].shape, dtype=torch.float64, device="cuda")
    small = st["new_k"].numel() <= 1 << 28
    k, v = (torch.zeros(st["new_k"].shape, dtype=torch.float64, device="cuda") if small else None for _ in range(2))
    for b, n in enumerate(_lens(case)):
        m = min(n, keep)
        pos, page, slot = _row_index(case, st, b, n)
        held = torch.arange(m, device="cuda")
        to, to_slot = st["new_table"][b].long()[held // case["page"]], held % case["page"]
        for h in range(H):
            w = st["weight"][page, h, slot].double()
            must = (pos < case["sinks"]) | (pos >= n - case["recent"])
            free = pos[~must]
            order = free[torch.argsort(-w[free], stable=True)]
            chosen = torch.cat([pos[must], order])[:m] if n > keep else pos
            chosen = chosen.sort()[0]
            kept[b, h, :m] = chosen.int().cpu()
            weight[to, h, to_slot] = w[chosen]
            if small:
                k[to, h, to_slot] = st["k"][page[chosen], h, slot[chosen]].double()
                v[to, h, to_slot] = st["v"][page[chosen], h, slot[chosen]].double()
    return {"k": k[:-1] if small else None, "v": v[:-1] if small else None, "weight": weight[:-1], "lens": lens, "kept": kept}


def _e4m3(x):
    """The nearest e4m3 value (4 exponent bits of bias 7, 3 of fraction), ties to even, as 64-bit numbers."""
    a = x.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
    return torch.copysign((a / step).round() * step, x)


def _append_exact(case, st):
    if st["k"].numel() > 1 << 29:
        return None
    k, v = (torch.zeros(st["k"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
    weight = torch.zeros(st["weight"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, m) in enumerate(zip(_lens(case), _news(case))):
        pos = torch.arange(n - m, n, device="cuda")
        page, slot = st["table"][b].long()[pos // case["page"]], pos % case["page"]
        for pool, new, scale in ((k, st["k_new"], st["ks"]), (v, st["v_new"], st["vs"])):
            x = new[at:at + m].double()
            pool[page, :, slot] = x if scale is None else _e4m3(x / scale.double()[:, None])
        at += m
    return {"k": k[:-1], "v": v[:-1], "weight": weight[:-1]}
