"""Page tables and slot maps from lengths against the definition, one sequence
after the other (tests/serving_helpers.py).  Everything is exact."""

from __future__ import annotations

import random

import numpy as np
import pytest

from serving_helpers import assign_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    import stream_compaction_pass_gb300 as m
    return m


def ok(ss, stream=None):
    st, where = ss.ss_stream_status(stream=stream)
    assert st == ss.SS_OK, (st, where, ss.ss_last_error_detail())


def build(lens, page, width, spare, seed, wrap=True):
    """Tables of shuffled pages, and a ring of `spare` free ones in mid-use."""
    rng = random.Random(seed)
    need = [-(-n // page) for n in lens]
    count = sum(need) + spare
    ids = list(range(count))
    rng.shuffle(ids)
    table, at = [], 0
    for m in need:
        table.append(ids[at:at + m])
        at += m
    head = (count - spare // 2 if wrap else 0) % max(count, 1)
    ring = [-7] * count
    for i, p in enumerate(ids[at:]):
        ring[(head + i) % count] = p
    return table, ring, head, count


def device_table(table, width, fill=-5):
    import torch
    t = torch.full((len(table), width), fill, dtype=torch.int32)
    for b, row in enumerate(table):
        t[b, :len(row)] = torch.tensor(row, dtype=torch.int32)
    return t.cuda()


def run(ss, lens, page, counts, restart, spare, pad=0, in_place=False, given=("offsets", "positions", "slots"), seed=1, misaligned=False, limit=None, stream=None,
        expect_bad=None):
    import torch
    batch = len(lens)
    width = max([-(-(n + max(1, c)) // page) for n, c in zip(lens, counts or [1] * batch)], default=0) + 2
    table, ring, head, count = build(lens, page, width, spare, seed)
    total = sum(max(c, 0) for c in counts) if counts else batch
    room = total + pad
    max_len = limit or width * page
    want = assign_reference(table, lens, page, counts, restart, ring, head, spare, room, max_len)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    d_table, d_lens, d_ring, d_state = device_table(table, width), i32(lens), i32(ring), i32([head, spare])
    shift = 1 if misaligned else 0
    offsets = torch.full((batch + 1,), -9, dtype=torch.int32, device="cuda") if "offsets" in given else None
    positions = torch.full((room + shift,), -9, dtype=torch.int32, device="cuda")[shift:] if "positions" in given else None
    slots = torch.full((room + shift,), -9, dtype=torch.int64, device="cuda")[shift:] if "slots" in given else None
    seqs = ss.KVTable(d_table, d_lens, max_len=limit)
    free = ss.KVFree(d_ring, d_state, num_pages=count)
    into = left = None
    new_table, new_lens, new_state = d_table, d_lens, d_state
    if not in_place:
        new_table, new_lens, left = torch.full_like(d_table, -6), torch.full_like(d_lens, -6), torch.full_like(d_state, -6)
        into, new_state = ss.KVTable(new_table, new_lens, max_len=limit), left
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    ss.ss_kv_assign(seqs, free, page, counts=None if counts is None else i32(counts), restart=None if restart is None else torch.tensor(restart, dtype=torch.bool, device="cuda"),
                    into=into, left=left, offsets=offsets, positions=positions, slots=slots, stream=stream)
    if want[7]:
        st, where = ss.ss_stream_status(stream=stream)
        assert st == ss.SS_ERR_INVALID_ARG and where in want[7]
    else:
        ok(ss, stream)
    rows, lengths, w_ring, w_state, w_offsets, w_positions, w_slots, _ = want
    assert new_lens.tolist() == lengths
    assert d_ring.tolist() == w_ring and new_state.tolist() == w_state
    got = new_table.tolist()
    for b, row in enumerate(rows):
        assert got[b][:len(row)] == row, b
        if in_place:  # behind, what was there before
            assert got[b][len(row):] == (table[b] + [-5] * width)[len(row):width], b
        else:
            assert got[b][len(row):] == [-6] * (width - len(row)), b
    if not in_place:
        assert d_lens.tolist() == lens and d_state.tolist() == [head, spare]
    if offsets is not None:
        assert offsets.tolist() == w_offsets
    if positions is not None:
        assert positions.tolist() == w_positions
    if slots is not None:
        assert slots.tolist() == w_slots


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("page", [1, 3, 16, 100])
@pytest.mark.parametrize("spare", [0, 5, 500])
def test_decode_steps(ss, in_place, page, spare):
    run(ss, [0, 1, 15, 16, 17, 31, 32, 99, 100, 300], page, None, None, spare, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("page,spare", [(16, 400), (16, 40), (7, 2000), (64, 0)])
@pytest.mark.parametrize("pad", [0, 1, 50])
def test_prompts_with_restarts(ss, in_place, page, spare, pad):
    rng = random.Random(2)
    lens = [rng.choice([0, 1, 16, 33, 200]) for _ in range(40)]
    counts = [rng.choice([0, 0, 1, 5, 16, 100, 333]) for _ in lens]
    restart = [rng.random() < 0.4 for _ in lens]
    run(ss, lens, page, counts, restart, spare, pad, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_one_sequence(ss, in_place):
    run(ss, [0], 16, [1], None, 1, in_place=in_place)
    run(ss, [0], 16, [0], None, 1, in_place=in_place)
    run(ss, [4096], 16, [100000], [True], 7000, in_place=in_place)


@pytest.mark.parametrize("batch", [511, 512, 513, 3000, 8192])
@pytest.mark.parametrize("in_place", [False, True])
def test_many_sequences(ss, batch, in_place):
    rng = random.Random(batch)
    lens = [rng.randrange(0, 90) for _ in range(batch)]
    counts = [rng.choice([0, 1, 1, 2, 40]) for _ in lens]
    restart = [rng.random() < 0.1 for _ in lens]
    run(ss, lens, 16, counts, restart, batch * 2, 3, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_many_tokens(ss, in_place):
    """More than one cluster's CTAs take: a launch of its own writes the lengths."""
    rng = random.Random(3)
    lens = [rng.randrange(0, 3000) for _ in range(64)]
    counts = [rng.randrange(0, 8000) for _ in lens]
    run(ss, lens, 32, counts, [rng.random() < 0.3 for _ in lens], 12000, 100, in_place)
    run(ss, lens, 32, counts, None, 4000, 100, in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_pages_of_one_token(ss, in_place):
    """A page number says nothing about the position that it holds: also page i - 1
    at place i of a row."""
    import torch
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = i32([[9, 0, 1, 2, 3, 4, 5, 6, 7, 8, 10, 11], [12, 13, 14, 15, 16, 17, 18, 19, 20, 21, 22, 23]])
    lens, ring, state = i32([3, 0]), i32([2, 3, 4, 5, 6, 7] + [40 + i for i in range(6)]), i32([0, 12])
    into = None if in_place else ss.KVTable(table.clone(), lens.clone())
    left = None if in_place else state.clone()
    slots, positions = torch.full((9,), -9, dtype=torch.int64, device="cuda"), torch.full((9,), -9, dtype=torch.int32, device="cuda")
    ss.ss_kv_assign(ss.KVTable(table, lens), ss.KVFree(ring, state, num_pages=60), 1, counts=i32([6, 3]), into=into, left=left, positions=positions, slots=slots)
    ok(ss)
    assert slots.tolist() == [2, 3, 4, 5, 6, 7, 40, 41, 42] and positions.tolist() == [3, 4, 5, 6, 7, 8, 0, 1, 2]


@pytest.mark.parametrize("given", [(), ("offsets",), ("positions",), ("slots",), ("positions", "slots")])
def test_optional_outputs(ss, given):
    run(ss, [3, 40, 0], 16, [2, 30, 1], None, 9, given=given)
    run(ss, [3, 40, 0], 16, [2, 30, 1], None, 9, given=given, in_place=True)


def test_outputs_that_are_not_aligned_to_vectors(ss):
    run(ss, [3, 40, 0] * 30, 16, [2, 30, 1] * 30, None, 300, pad=3, misaligned=True)


def test_lengths_past_the_limit_and_negative_counts(ss):
    run(ss, [10, 60, 0], 16, [5, 5, 64], None, 20, limit=64)
    run(ss, [10, 60, 0], 16, [5, 5, 65], None, 20, limit=64)
    run(ss, [10, 60, 0], 16, [5, -1, 3], None, 20, limit=64)
    run(ss, [10, 60, 0], 16, [5, 5, 3], [False, True, False], 20, limit=64, in_place=True)


def test_a_head_beyond_the_ring_is_taken_modulo_its_capacity(ss):
    import torch
    for head in (4, 6, 4 * 1000 + 2):
        ring = torch.tensor([3, 2, 1, 0], dtype=torch.int32, device="cuda")
        state = torch.tensor([head, 2], dtype=torch.int32, device="cuda")
        table, lens = torch.full((1, 3), -1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        ss.ss_kv_assign(ss.KVTable(table, lens), ss.KVFree(ring, state), 4, counts=torch.tensor([7], dtype=torch.int32, device="cuda"))
        ok(ss)
        order = [3, 2, 1, 0]
        assert table.tolist() == [[order[head % 4], order[(head + 1) % 4], -1]] and lens.tolist() == [7] and state.tolist() == [(head + 2) % 4, 0]


def test_bad_pages_states_and_lengths_are_reported(ss):
    import torch
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def call(table, lens, ring, state, counts, num_pages):
        n = len(lens)
        slots = torch.full((8 * n,), -9, dtype=torch.int64, device="cuda")
        d_table, d_lens = i32(table), i32(lens)
        ss.ss_kv_assign(ss.KVTable(d_table, d_lens), ss.KVFree(i32(ring), i32(state), num_pages=num_pages), 4, counts=i32(counts), slots=slots)
        return ss.ss_stream_status(), slots.tolist(), d_lens.tolist()

    good = call([[0, 1, 2], [3, 4, 5]], [3, 8], [6, 7, 8, 9], [0, 4], [1, 2], 10)
    assert good[0] == (ss.SS_OK, -1) and good[1][:3] == [3, 24, 25] and good[2] == [4, 10]
    bad_table = call([[99, 1, 2], [3, 4, 5]], [3, 8], [6, 7, 8, 9], [0, 4], [1, 2], 10)
    assert bad_table[0] == (ss.SS_ERR_INVALID_ARG, 0) and bad_table[1][:3] == [-1, 24, 25]
    bad_ring = call([[0, 1, 2], [3, 4, 5]], [3, 8], [-2, 7, 8, 9], [0, 4], [1, 2], 10)
    assert bad_ring[0] == (ss.SS_ERR_INVALID_ARG, 1) and bad_ring[1][:3] == [3, -1, -1]
    for state in ([-1, 4], [0, 5], [0, -1]):  # an empty ring is assumed
        got = call([[0, 1, 2], [3, 4, 5]], [3, 8], [6, 7, 8, 9], state, [1, 2], 10)
        assert got[0][0] == ss.SS_ERR_INVALID_ARG and got[2] == [4, 8] and got[1][:3] == [3, -1, -1]
    for n in (-3, 13):  # clamped to 0, and to 12 (no room for one more)
        got = call([[0, 1, 2], [3, 4, 5]], [n, 8], [6, 7, 8, 9], [0, 4], [1, 2], 10)
        assert got[0] == (ss.SS_ERR_INVALID_ARG, 0) and got[2][1] == 10 and got[1][1:3] == ([24, 25] if n > 0 else [28, 29])


def test_more_counts_than_room(ss):
    import torch
    slots = torch.full((5,), -9, dtype=torch.int64, device="cuda")
    guard = slots.clone()
    table, lens = torch.zeros(2, 4, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    ring, state = torch.arange(8, dtype=torch.int32, device="cuda"), torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    ss.ss_kv_assign(ss.KVTable(table, lens), ss.KVFree(ring, state), 4, counts=torch.tensor([3, 4], dtype=torch.int32, device="cuda"), slots=slots[:4])
    assert ss.ss_stream_status()[0] == ss.SS_ERR_INVALID_ARG
    assert slots.tolist() == [0, 1, 2, 4, int(guard[4])] and lens.tolist() == [3, 4]


def test_in_a_graph_and_on_another_stream(ss):
    """Replays go on from what the last one left: a loop of decode steps."""
    import torch
    page, batch, steps = 4, 5, 13
    lens0 = [0, 3, 4, 7, 12]
    table, ring, head, count = build(lens0, page, 20, 60, 9)
    d_table, d_lens = device_table(table, 20), torch.tensor(lens0, dtype=torch.int32, device="cuda")
    d_ring, d_state = torch.tensor(ring, dtype=torch.int32, device="cuda"), torch.tensor([head, 60], dtype=torch.int32, device="cuda")
    seqs, free = ss.KVTable(d_table, d_lens), ss.KVFree(d_ring, d_state)
    slots = torch.zeros(batch, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ss.ss_kv_assign(seqs, free, page, slots=slots, stream=side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ss.ss_kv_assign(seqs, free, page, slots=slots, stream=side)
    rows, lens, state = [list(r) for r in table], list(lens0), [head, 60]
    for step in range(steps):
        if step:
            g.replay()
        torch.cuda.synchronize()
        rows, lens, ring, state, _, _, want, _ = assign_reference(rows, lens, page, None, None, ring, state[0], state[1], batch, 80)
        assert slots.tolist() == want and d_lens.tolist() == lens and d_state.tolist() == state
    ok(ss, side)


def test_no_sequences(ss):
    import torch
    table, lens = torch.zeros(0, 4, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    ring, state = torch.arange(8, dtype=torch.int32, device="cuda"), torch.tensor([2, 3], dtype=torch.int32, device="cuda")
    slots, positions = torch.full((6,), 5, dtype=torch.int64, device="cuda"), torch.full((6,), 5, dtype=torch.int32, device="cuda")
    offsets = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    ss.ss_kv_assign(ss.KVTable(table, lens), ss.KVFree(ring, state), 4, slots=slots, positions=positions, offsets=offsets)
    ok(ss)
    assert slots.tolist() == [-1] * 6 and positions.tolist() == [0] * 6 and offsets.tolist() == [0] and state.tolist() == [2, 3]
