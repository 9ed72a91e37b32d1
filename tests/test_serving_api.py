"""The calls around a decode step without a GPU: their arguments' checks, and
the pins of the references that the GPU tests compare with."""

import ctypes
import math

import numpy as np
import pytest

import stream_compaction_pass_gb300 as ss
from kv_helpers import e4m3_reference
from serving_helpers import (E2M1, QuarterTurns, assign_reference, codes_between, e2m1_value, e4m3_between, e4m3_value, frequencies, open4, quantise4,
                             rope_gradients, rope_reference, turn_reference)

INV, UNS = ss.SS_ERR_INVALID_ARG, ss.SS_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from stream_compaction_pass_gb300 import build
    build.build()
    return ss.lib()


# ---- assignment ----

def table(**kw):
    t = ss._KvTable(0x20000, 8, 8, 3, 0x30000, 0)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def assign(lib, t=None, d=None, page=16, num=100, counts=None, restart=None, free=None, left=None, offsets=None, positions=None, slots=None, tokens=0, **f):
    t = t or table()
    free = free or ss._KvFree(f.get("ring", 0x50000), f.get("capacity", 100), f.get("state", 0x60000))
    return lib.ss_kv_assign(ctypes.addressof(t), None if d is None else ctypes.addressof(d), page, num, counts, restart, ctypes.addressof(free), left, offsets,
                            positions, slots, tokens, None)


@pytest.mark.parametrize("bad", [dict(page=0), dict(page=-1), dict(num=0), dict(num=1 << 31), dict(ring=0), dict(state=0), dict(capacity=0),
                                 dict(capacity=1 << 31), dict(ring=0x50002), dict(state=0x60001), dict(counts=0x70002), dict(left=0x80001),
                                 dict(offsets=0x80002), dict(positions=0x80002, tokens=4), dict(slots=0x80004, tokens=4),
                                 dict(slots=0x80000, tokens=1 << 31), dict(offsets=0x30004), dict(positions=0x50010, tokens=4),
                                 dict(slots=0x80000, positions=0x80008, tokens=4), dict(counts=0x50000), dict(left=0x60004), dict(restart=0x60002),
                                 dict(t=table(batch=-1)), dict(t=table(lens=0)), dict(t=table(batch=8193)), dict(t=table(max_pages=1 << 30)),
                                 dict(t=table(row_stride=7)), dict(d=table(batch=2, lens=0x38000)), dict(d=table(max_pages=7, lens=0x38000)),
                                 dict(d=table(max_len=40, lens=0x38000)), dict(d=table(lens=0x30004)), dict(d=table(pages=0x20004, lens=0x38000)),
                                 dict(d=table(row_stride=9, lens=0x38000))], ids=str)
def test_assign_arguments(lib, bad):
    assert assign(lib, **bad) == INV
    assert ss.ss_last_error_detail()


def test_assign_null_descriptions(lib):
    free = ss._KvFree(0x50000, 100, 0x60000)
    held = table()
    assert lib.ss_kv_assign(None, None, 16, 100, None, None, ctypes.addressof(free), None, None, None, None, 0, None) == INV
    assert lib.ss_kv_assign(ctypes.addressof(held), None, 16, 100, None, None, None, None, None, None, None, 0, None) == INV


def test_assign_reference_by_hand():
    # pages of 4: sequence 0 has 6 tokens and gets 3 (a page more), 1 is restarted with 5, 2 finds the ring short
    out = assign_reference([[7, 8], [3], [5]], [6, 4, 4], 4, [3, 5, 9], [0, 1, 0], [0, 1, 2, 9, 9, 9, 9, 9], 0, 3, 18, 100)
    assert out[0] == [[7, 8, 0], [1, 2], [5]] and out[1] == [9, 5, 4]
    assert out[2] == [0, 1, 2, 3, 9, 9, 9, 9] and out[3] == [3, 1]
    assert out[4] == [0, 3, 8, 17]
    assert out[5] == [6, 7, 8, 0, 1, 2, 3, 4, 4, 5, 6, 7, 8, 9, 10, 11, 12, 0]
    assert out[6] == [34, 35, 0, 4, 5, 6, 7, 8] + [-1] * 10


# ---- norms and rotation ----

QK = dict(type=ss.SS_BF16, weight_type=ss.SS_BF16, head_dim=64, q_heads=4, kv_heads=2, eps=1e-6, tokens=3, q=(0x100000, 512, 64), k=(0x200000, 256, 64), q_weight=0x1000,
          k_weight=0x2000, positions=0x3000, turns=0x4000, rotary=64, interleaved=0)


def qk(**kw):
    a = {**QK, **kw}
    return ss._QK.pack(a["type"], a["weight_type"], a["head_dim"], a["q_heads"], a["kv_heads"], a["eps"], a["tokens"], *a["q"], *a["k"], a["q_weight"], a["k_weight"],
                       a["positions"], a["turns"], a["rotary"], a["interleaved"])


def rows(*a):
    return ss._ROWS.pack(*a)


def forward(lib, q_out=(0x300000, 512, 64), k_out=(0x400000, 256, 64), **kw):
    return lib.ss_qk_norm_rope(qk(**kw), rows(*q_out), rows(*k_out), None)


def backward(lib, gq=(0x500000, 512, 64), gk=(0x600000, 256, 64), dq=(0x300000, 512, 64), dk=(0x400000, 256, 64), dqw=None, dkw=None, **kw):
    return lib.ss_qk_norm_rope_backward(qk(**kw), rows(*gq), rows(*gk), rows(*dq), rows(*dk), dqw, dkw, None)


def cached(lib, slots=0x9000, v=(0x700000, 256, 64), q_out=(0x300000, 512, 64), cache=None, **kw):
    p = ss._KvPages(ss.SS_BF16, 2, 64, 16, 100, 0x1000000, 0x2000000, 2048, 1024, 64, None, None, 0x10000)
    for k, x in (cache or {}).items():
        setattr(p, k, x)
    return lib.ss_kv_append_rope(ctypes.addressof(p), slots, qk(**kw), rows(*v), rows(*q_out), None)


BAD_QK = [dict(type=ss.SS_E4M3), dict(type=9), dict(weight_type=ss.SS_E2M1), dict(tokens=-1), dict(tokens=1 << 31), dict(q_heads=-1), dict(q_heads=0, kv_heads=0),
          dict(q_heads=65537), dict(head_dim=60), dict(head_dim=264), dict(head_dim=0), dict(rotary=0), dict(rotary=24), dict(rotary=80), dict(eps=-1e-6),
          dict(eps=math.nan), dict(eps=math.inf), dict(positions=0), dict(positions=0x3002), dict(turns=0), dict(turns=0x4004), dict(q_weight=0x1001),
          dict(weight_type=ss.SS_ELEM_F32, k_weight=0x2002), dict(q=(0, 512, 64)), dict(k=(0x200008, 256, 64)), dict(q=(0x100000, -512, 64)),
          dict(k=(0x200000, 256, 60)), dict(q=(0x100000, 1 << 34, 64))]


@pytest.mark.parametrize("bad", BAD_QK, ids=str)
def test_every_rotation_call_refuses_a_bad_description(lib, bad):
    want = UNS if "type" in bad or bad.get("weight_type") == ss.SS_E2M1 else INV
    assert forward(lib, **bad) == want
    assert backward(lib, **bad) == want
    if "q_heads" not in bad or bad["q_heads"] != 0:
        assert cached(lib, **bad) == want


@pytest.mark.parametrize("bad", [dict(q_out=(0, 512, 64)), dict(q_out=(0x300008, 512, 64)), dict(q_out=(0x300000, 512, 32)), dict(k_out=(0x400000, 32, 64)),
                                 dict(q_out=(0x100000, 1024, 64)), dict(q_out=(0x100080, 512, 64)), dict(k_out=(0x100000, 512, 64)), dict(k_out=(0x300000, 512, 64)),
                                 dict(q_out=(0x200000, 512, 64))], ids=str)
def test_rotation_outputs(lib, bad):
    assert forward(lib, **bad) == INV


@pytest.mark.parametrize("bad", [
    # [token][head][q, k, v] of 2 heads of 64 (192 elements a head): k_out on q, across q and k, and behind the last one's row on the next token's q
    dict(q_heads=2, q=(0x100000, 384, 192), k=(0x100080, 384, 192), q_out=(0x100000, 384, 192), k_out=(0x100000, 384, 192)),
    dict(q_heads=2, q=(0x100000, 384, 192), k=(0x100080, 384, 192), q_out=(0x100000, 384, 192), k_out=(0x1000c0, 384, 192)),
    dict(q_heads=2, q=(0x100000, 384, 192), k=(0x100080, 384, 192), q_out=(0x100000, 384, 192), k_out=(0x100140, 384, 192)),
    dict(q_heads=2, q=(0x100000, 384, 192), k=(0x100080, 384, 192), q_out=(0x100080, 384, 192)),
    # [head][q, k][token] of 3 tokens: k_out on the last token's q
    dict(q_heads=2, q=(0x100000, 64, 384), k=(0x100180, 64, 384), q_out=(0x100000, 64, 384), k_out=(0x100100, 64, 384)),
    # one token: rows of k between, and on, those of q
    dict(tokens=1, q=(0x100000, 0, 128), q_out=(0x100000, 0, 128), k_out=(0x1000c0, 0, 128)),
    # other strides, whose third token meets
    dict(q_heads=1, kv_heads=1, q=(0x100000, 64, 64), q_out=(0x100000, 64, 64), k_out=(0x100100, 128, 64))], ids=str)
def test_rotation_outputs_between_other_rows(lib, bad):
    assert forward(lib, **bad) == INV
    assert "overlaps" in ss.ss_last_error_detail()


@pytest.mark.parametrize("out", [(0x300000, 96, 64), (0x300000, 64, 96), (0x300000, 64, 64), (0x300000, 64, 128), (0x300000, 128, 64), (0x300000, 120, 160)], ids=str)
def test_rotation_outputs_whose_own_rows_meet(lib, out):
    """Each stride reaches past a row, but a token's rows meet another's."""
    shape = dict(q_heads=3, kv_heads=3, q=(0x100000, 192, 64), k=(0x200000, 192, 64), k_out=(0x400000, 192, 64))
    for call in (lambda **kw: forward(lib, q_out=out, **kw), lambda **kw: forward(lib, **{**kw, "q_out": (0x500000, 192, 64), "k_out": out}),
                 lambda **kw: backward(lib, gq=(0x600000, 192, 64), gk=(0x700000, 192, 64), dq=out, dk=(0x800000, 192, 64), **{k: v for k, v in kw.items() if k != "k_out"})):
        assert call(**shape) == INV
        assert "overlap" in ss.ss_last_error_detail()


@pytest.mark.parametrize("bad", [dict(gq=(0, 512, 64)), dict(gk=(0x600004, 256, 64)), dict(dq=(0, 512, 64)), dict(dq=(0x500080, 512, 64)), dict(dk=(0x500000, 512, 64)),
                                 dict(dk=(0x300000, 256, 64)), dict(dqw=0x1002), dict(dqw=0x8000, dkw=0x8010)], ids=str)
def test_rotation_gradients_arguments(lib, bad):
    assert backward(lib, **bad) == INV


@pytest.mark.parametrize("bad", [dict(slots=0), dict(slots=0x9004), dict(v=(0, 256, 64)), dict(v=(0x700000, 250, 64)), dict(q_out=(0x200000, 512, 64)),
                                 dict(q_out=(0x700000, 512, 64)), dict(kv_heads=1), dict(type=ss.SS_F16), dict(cache=dict(slot_stride=32)),
                                 dict(cache=dict(type=ss.SS_E2M1, k_block=0x8000, v_block=0x9000), rotary=48),
                                 dict(cache=dict(type=ss.SS_E2M1))], ids=str)
def test_append_rope_arguments(lib, bad):
    assert cached(lib, **bad) == INV
    assert cached(lib, type=ss.SS_ELEM_F32) == UNS


def test_no_tokens_is_a_noop(lib):
    assert forward(lib, tokens=0) == ss.SS_OK
    assert backward(lib, tokens=0) == ss.SS_OK
    assert cached(lib, tokens=0) == ss.SS_OK


def test_binding_refuses_tensors_before_the_library():
    import torch
    freq = torch.ones(32, dtype=torch.float64)
    rope = ss.Rope(freq)
    q, k, pos = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="not on a GPU"):
        ss.ss_qk_norm_rope(q, k, None, None, rope, pos, q, k)
    with pytest.raises(ValueError, match="both None"):
        ss.ss_qk_norm_rope(None, None, None, None, rope, pos, None, None)
    with pytest.raises(ValueError, match="same tokens"):
        ss.ss_qk_norm_rope(q, torch.zeros(2, 2, 64), None, None, rope, pos, q, k)
    with pytest.raises(ValueError):
        ss.Rope(torch.ones(4, 4))
    ring = torch.zeros(10, dtype=torch.int32)
    free = ss.KVFree(ring, torch.zeros(2, dtype=torch.int32))
    seqs = ss.KVTable(torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="not on a GPU"):
        ss.ss_kv_assign(seqs, free, 16)
    with pytest.raises(ValueError, match="state"):
        ss.KVFree(ring, torch.zeros(3, dtype=torch.int32))


def test_4_bit_pools_of_the_binding():
    import torch
    codes = torch.zeros(5, 2, 16, 32, dtype=torch.uint8)
    blocks = torch.zeros(5, 2, 16, 4, dtype=torch.uint8).view(torch.float8_e4m3fn)
    p = ss.KVPages(codes, codes.clone(), k_block=blocks, v_block=blocks.clone())
    assert p.head_dim == 64 and p._c.type == ss.SS_E2M1 and p._c.page_stride == 2 * 2 * 16 * 32 and p._c.k_block == blocks.data_ptr()
    with pytest.raises(ValueError, match="both"):
        ss.KVPages(codes, codes, k_block=blocks)
    with pytest.raises(ValueError, match="v_block"):
        ss.KVPages(codes, codes, k_block=blocks, v_block=blocks[:, :, :8])
    with pytest.raises(TypeError):
        ss.KVPages(codes.float(), codes.float(), k_block=blocks, v_block=blocks)
    with pytest.raises(TypeError):
        ss.KVPages(codes, codes)


# ---- 4-bit pools ----

def pool4(**kw):
    p = ss._KvPages(ss.SS_E2M1, 2, 64, 16, 100, 0x100000, 0x800000, 2048, 1024, 64, None, None, 0x10000, 0x11000, 0x12000)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("bad", [dict(head_dim=32), dict(head_dim=96), dict(head_dim=192), dict(k_block=0), dict(v_block=0), dict(k_block=0x11008), dict(v_block=0x12001),
                                 dict(slot_stride=48), dict(page_stride=16), dict(k=0x100008), dict(k_scale=0x9002)], ids=str)
def test_4_bit_pool_arguments(lib, bad):
    t = table()
    a = ss._KvAttention(ss.SS_BF16, 8, 0x40000, 512, 64, 0x50000, 512, 64, 0.125, 0, 0, None, None, None)
    p = pool4(**bad)
    assert lib.ss_kv_attend(ctypes.addressof(p), ctypes.addressof(t), ctypes.addressof(a), None) == INV
    assert lib.ss_kv_append(ctypes.addressof(p), ctypes.addressof(t), ss.SS_BF16, 0x40000, 0x50000, 128, 64, None, 3, None) == INV


def test_rows_of_a_4_bit_pool_that_is_written_must_not_overlap(lib):
    t = table()
    for bad in (dict(slot_stride=32), dict(head_stride=32), dict(page_stride=32)):
        p = pool4(**bad)
        assert lib.ss_kv_append(ctypes.addressof(p), ctypes.addressof(t), ss.SS_BF16, 0x40000, 0x50000, 128, 64, None, 3, None) == INV
        assert "overlap" in ss.ss_last_error_detail()


# ---- pins of the references ----

def test_e2m1_codes_and_scales():
    assert e2m1_value(np.arange(16)).tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    assert [float(e4m3_value(c)) for c in (0, 1, 8, 0x38, 0x7e)] == [0.0, 2.0 ** -9, 2.0 ** -6, 1.0, 448.0] and np.isnan(e4m3_value(127))
    for c in range(127):
        assert e4m3_reference(float(e4m3_value(c))) == e4m3_value(c)


def test_quantise4_keeps_what_it_can_hold():
    """Values that are codes times a scale, with a largest element of 6, come back."""
    rng = np.random.default_rng(1)
    code = rng.integers(0, 8, (40, 2, 4, 16))
    code[..., 3] = 7
    for scale in (1.0, 0.25, 2.0 ** -9, 448.0):
        x = (E2M1[code] * scale).reshape(40, 2, 64)
        codes, blocks = quantise4(x, np.ones(2))
        assert np.array_equal(open4(codes, blocks), x)
    codes, blocks = quantise4(np.full((1, 1, 16), np.nan), np.ones(1))
    assert np.isnan(open4(codes, blocks)).all()
    x = np.zeros((1, 1, 16))
    x[0, 0, 5] = np.inf
    assert open4(*quantise4(x, np.ones(1)))[0, 0, 5] == 6 * 448


def test_quantise4_rounds_to_the_nearest():
    """No code is further from y / scale than half the step around it."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((500, 1, 64))
    codes, blocks = quantise4(x, np.ones(1))
    b = np.repeat(e4m3_value(blocks), 16, -1)
    z = np.minimum(np.abs(x / b), 6)
    got = np.abs(open4(codes, blocks)) / b
    gap = np.select([z <= 2, z <= 4], [0.25, 0.5], 1.0)
    assert (np.abs(got - z) <= gap * (1 + 1e-6)).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_reference(interleaved):
    """At position 0 only the norm is left; a rotation keeps lengths and goes back;
    the gradients are those of differences."""
    rng = np.random.default_rng(3)
    x, w, freq = rng.standard_normal((4, 3, 24)), rng.random(24) + 0.5, frequencies(16)
    y = rope_reference(x, w, np.zeros(4), freq, interleaved, 1e-6)
    assert np.allclose(y, x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 1e-6) * w)
    pos = np.array([1, 5, 1000, 77])
    t = turn_reference(x, pos, freq, interleaved, 1)
    assert np.allclose((t ** 2).sum(-1), (x ** 2).sum(-1)) and np.allclose(turn_reference(t, pos, freq, interleaved, -1), x)
    a, b = (0, 1) if interleaved else (0, 8)
    assert np.isclose(t[0, 0, a], x[0, 0, a] * math.cos(1) - x[0, 0, b] * math.sin(1))
    assert np.isclose(t[0, 0, b], x[0, 0, b] * math.cos(1) + x[0, 0, a] * math.sin(1))
    g = rng.standard_normal(x.shape)
    dx, dw = rope_gradients(x, w, g, pos, freq, interleaved, 1e-6)
    f = lambda x, w: (g * rope_reference(x, w, pos, freq, interleaved, 1e-6)).sum()  # noqa: E731
    for i in [(0, 0, 0), (1, 2, 9), (3, 1, 23), (2, 0, 15)]:
        e = np.zeros(x.shape)
        e[i] = 1e-5
        assert abs((f(x + e, w) - f(x - e, w)) / 2e-5 - dx[i]) < 1e-7
        v = np.zeros(24)
        v[i[2]] = 1e-5
        assert abs((f(x, w + v) - f(x, w - v)) / 2e-5 - dw[i[2]]) < 1e-7


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_turned_by_a_quarter_show_angles_of_fp32(dim):
    """What the GPU's caches are held to: the formula's rows pass, also with fp32
    roundings of the cosines; those of angles in fp32, or of cosines off by 2^-21, do not."""
    rows = QuarterTurns(40, 3, dim, 5)
    y = rope_reference(rows.x, rows.weight, rows.positions, rows.freq, False, 0.0)
    assert np.allclose(y, rows.rows(), rtol=1e-9, atol=0)
    s = 2.0 ** -16
    rng = np.random.default_rng(6)
    fine = rows.rows() * (1 + rng.uniform(-1, 1, y.shape) * 2.0 ** -21)
    rounded = rows.rows(lambda x: x.astype(np.float32).astype(np.float64))
    near = rows.rows() + rng.uniform(-1, 1, y.shape) * 2.0 ** -21
    for z, good in ((fine, True), (rounded, False), (near, False)):
        got = e4m3_between(e4m3_reference(np.clip(z / s, -448, 448)), y / s, 2.0 ** -20)
        assert got.all() == good, got.mean()
        codes, blocks = quantise4(z, np.full(3, s, np.float32))
        got = codes_between(codes, blocks, y / s, 2.0 ** -20)
        assert got.all() == good, got.mean()
