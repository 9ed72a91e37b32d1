"""The key-value cache calls without a GPU: their arguments' checks, and the
pins of the 64-bit reference that the GPU tests compare with."""

import ctypes
import math

import numpy as np
import pytest

import stream_compaction_pass_gb300 as ss
from kv_helpers import e4m3_reference, visible

INV, UNS = ss.SS_ERR_INVALID_ARG, ss.SS_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    from stream_compaction_pass_gb300 import build
    build.build()
    return ss.lib()


def pages(**kw):
    p = ss._KvPages(ss.SS_BF16, 2, 64, 16, 100, 0x100000, 0x800000, 2048, 1024, 64, None, None, 0x10000)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def table(**kw):
    t = ss._KvTable(0x20000, 8, 8, 3, 0x30000, 0)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


def attention(**kw):
    a = ss._KvAttention(ss.SS_BF16, 8, 0x40000, 512, 64, 0x50000, 512, 64, 0.125, 0, 0, None, None, None)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def attend(lib, p=None, t=None, a=None):
    p, t, a = p or pages(), t or table(), a or attention()
    return lib.ss_kv_attend(ctypes.addressof(p), ctypes.addressof(t), ctypes.addressof(a), None)


def append(lib, p=None, t=None, type=ss.SS_BF16, k=0x40000, v=0x50000, ts=128, hs=64, offsets=None, tokens=3):
    p, t = p or pages(), t or table()
    return lib.ss_kv_append(ctypes.addressof(p), ctypes.addressof(t), type, k, v, ts, hs, offsets, tokens, None)


def evict(lib, p=None, t=None, d=None, dt=None, keep=64, sinks=4, recent=8, kept=None):
    p, t, d, dt = p or pages(), t or table(), d or pages(), dt or table(lens=0x38000)
    return lib.ss_kv_evict(ctypes.addressof(p), ctypes.addressof(t), ctypes.addressof(d), ctypes.addressof(dt), keep, sinks, recent, kept, None)


BAD_PAGES = [dict(type=7), dict(kv_heads=0), dict(page_size=0), dict(num_pages=0), dict(num_pages=1 << 31), dict(head_dim=0),
             dict(head_dim=264), dict(head_dim=60), dict(k=0), dict(v=0), dict(k=0x100008), dict(v=0x800002), dict(page_stride=-2048),
             dict(slot_stride=63), dict(head_stride=4), dict(k_scale=0x9000), dict(v_scale=0x9000), dict(weight=0x10002),
             dict(type=ss.SS_E4M3, head_dim=72), dict(type=ss.SS_E4M3, k_scale=0x9002)]
BAD_TABLES = [dict(batch=-1), dict(max_pages=-1), dict(max_len=-1), dict(row_stride=-8), dict(pages=0), dict(lens=0), dict(lens=0x30002),
              dict(pages=0x20001), dict(max_pages=1 << 30)]


@pytest.mark.parametrize("bad", BAD_PAGES, ids=str)
def test_every_call_refuses_a_bad_pool(lib, bad):
    want = UNS if bad.get("type") == 7 else INV
    assert attend(lib, p=pages(**bad)) == want
    assert append(lib, p=pages(**bad)) == want
    assert evict(lib, p=pages(**bad)) == want
    assert evict(lib, d=pages(**bad)) == want
    assert ss.ss_last_error_detail().startswith("dst")


@pytest.mark.parametrize("bad", BAD_TABLES, ids=str)
def test_every_call_refuses_a_bad_table(lib, bad):
    assert attend(lib, t=table(**bad)) == INV
    assert append(lib, t=table(**bad)) == INV
    assert evict(lib, t=table(**bad)) == INV
    assert evict(lib, dt=table(**{"lens": 0x38000, **bad})) == INV


def test_null_descriptions(lib):
    held = pages(), table(), attention()
    p, t, a = (ctypes.addressof(x) for x in held)
    assert lib.ss_kv_attend(None, t, a, None) == INV
    assert lib.ss_kv_attend(p, None, a, None) == INV
    assert lib.ss_kv_attend(p, t, None, None) == INV


@pytest.mark.parametrize("bad", [dict(q_heads=0), dict(q_heads=7), dict(q_heads=2 * 129), dict(q=0), dict(out=0), dict(q=0x40008),
                                 dict(out=0x50002), dict(q_seq_stride=-512), dict(out_head_stride=63), dict(sinks=-1),
                                 dict(scale=math.inf), dict(scale=math.nan), dict(lse=0x60001), dict(weight_in=0x70000),
                                 dict(weight_out=0x70002), dict(weight_in=0x70000, weight_out=0x70040), dict(out=0x40040),
                                 dict(type=ss.SS_F16)], ids=str)
def test_attend_arguments(lib, bad):
    assert attend(lib, a=attention(**bad)) == INV


def test_attend_types(lib):
    assert attend(lib, a=attention(type=ss.SS_E4M3)) == UNS
    assert attend(lib, a=attention(type=5)) == UNS
    assert attend(lib, p=pages(type=ss.SS_F16)) == INV


@pytest.mark.parametrize("bad", [dict(k=0), dict(v=0), dict(k=0x40008), dict(ts=-128), dict(hs=60), dict(tokens=4), dict(type=ss.SS_F16),
                                 dict(offsets=0x60002), dict(offsets=0x60000, tokens=1 << 31)], ids=str)
def test_append_arguments(lib, bad):
    assert append(lib, **bad) == INV


def test_append_types(lib):
    assert append(lib, type=ss.SS_E4M3) == UNS


@pytest.mark.parametrize("bad", [dict(keep=0), dict(sinks=-1), dict(recent=-1), dict(sinks=40, recent=25), dict(sinks=2 ** 31 - 1, recent=1),
                                 dict(kept=0x60002), dict(p=pages(weight=0)), dict(d=pages(type=ss.SS_F16)), dict(d=pages(kv_heads=1)),
                                 dict(d=pages(head_dim=128)), dict(dt=table(batch=2, lens=0x38000)), dict(dt=table()),
                                 dict(dt=table(lens=0x38000, max_pages=2)), dict(dt=table(lens=0x30004))], ids=str)
def test_evict_arguments(lib, bad):
    assert evict(lib, **bad) == INV


def test_an_empty_batch_is_a_noop(lib):
    empty = table(batch=0)
    assert attend(lib, t=empty) == ss.SS_OK
    assert append(lib, t=empty, tokens=0) == ss.SS_OK
    assert evict(lib, t=empty, dt=table(batch=0)) == ss.SS_OK


def test_the_binding_checks_shapes():
    torch = pytest.importorskip("torch")
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    ss.KVPages(k, k.clone(), weight=torch.zeros(4, 2, 16))
    for bad in (dict(v=torch.zeros(4, 2, 16, 32, dtype=torch.bfloat16)), dict(v=k.half()), dict(v=k.transpose(0, 1).contiguous().transpose(0, 1)),
                dict(weight=torch.zeros(4, 16, 2)), dict(weight=torch.zeros(4, 2, 16).double()), dict(k_scale=torch.zeros(3))):
        with pytest.raises(ValueError):
            ss.KVPages(**{"k": k, "v": k, **bad})
    with pytest.raises(TypeError):
        ss.KVPages(k.float(), k.float())
    lens = torch.zeros(3, dtype=torch.int32)
    t = ss.KVTable(torch.zeros(3, 5, dtype=torch.int32), lens, max_len=50)
    assert t.max_len == 50
    t.max_len = 20
    assert t._c.max_len == 20
    for bad in (torch.zeros(3, 5), torch.zeros(15, dtype=torch.int32), torch.zeros(5, 3, dtype=torch.int32).t()):
        with pytest.raises(ValueError):
            ss.KVTable(bad, lens)
    with pytest.raises(ValueError):
        ss.KVTable(torch.zeros(2, 5, dtype=torch.int32), lens)
    pool = ss.KVPages(k, k.clone())
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    for bad in (dict(q=q[:2]), dict(out=q[:, :2]), dict(lse=torch.zeros(3, 5)), dict(weight_out=torch.zeros(4, 2, 15)), dict(q=q[0])):
        with pytest.raises(ValueError):
            ss.ss_kv_attend(**{"cache": pool, "seqs": t, "q": q, "out": q.clone(), **bad})
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    for bad in (dict(k_new=x[:, :1]), dict(v_new=x.half()), dict(offsets=torch.zeros(3, dtype=torch.int32)), dict(offsets=torch.zeros(4))):
        with pytest.raises(ValueError):
            ss.ss_kv_append(**{"cache": pool, "seqs": t, "k_new": x, "v_new": x.clone(), **bad})
    with pytest.raises(ValueError):
        ss.ss_kv_evict(pool, t, pool, t, 8, kept=torch.zeros(3, 2, 9, dtype=torch.int32))


def test_reference_pins():
    # e4m3 by hand: 1 + 1/16 lies between 1 and 1.125 and goes to the even 1; 448 is the largest
    x = [0.0, 1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, 460.0, -1e9, 17.0, 19.0]
    assert e4m3_reference(x).tolist() == [0.0, 1.0, 1.25, 0.0, 2.0 ** -8, 448.0, -448.0, 16.0, 20.0]
    assert math.isnan(e4m3_reference([math.nan])[0])
    assert visible(6, 2, 1).tolist() == [True, False, False, False, True, True]
    assert visible(3, 0, 0).all() and visible(3, 9, 0).all() and visible(0, 2, 1).size == 0


def test_e4m3_reference_matches_the_type():
    torch = pytest.importorskip("torch")
    x = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    x = x[torch.isfinite(x)]
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(e4m3_reference(x.numpy()), want)


@pytest.mark.parametrize("bad", [dict(page_stride=1 << 60), dict(slot_stride=1 << 58), dict(head_stride=1 << 60)], ids=str)
def test_strides_past_the_address_space(lib, bad):
    assert attend(lib, p=pages(**bad)) == INV
    assert append(lib, p=pages(**bad)) == INV
    assert evict(lib, d=pages(**bad)) == INV


@pytest.mark.parametrize("bad", [dict(slot_stride=0), dict(head_stride=32), dict(page_stride=0)], ids=str)
def test_rows_that_are_written_do_not_overlap(lib, bad):
    assert append(lib, p=pages(**bad)) == INV
    assert evict(lib, d=pages(**bad)) == INV
    assert "overlap" in ss.ss_last_error_detail()


@pytest.mark.parametrize("bad", [dict(out_seq_stride=0), dict(out_head_stride=0), dict(out_head_stride=56), dict(q_seq_stride=1 << 41),
                                 dict(out_seq_stride=1 << 41)], ids=str)
def test_rows_of_out_do_not_overlap(lib, bad):
    assert attend(lib, a=attention(**bad)) == INV


def test_append_strides_past_the_address_space(lib):
    assert append(lib, ts=1 << 41) == INV
    assert append(lib, hs=1 << 41) == INV


def test_attend_head_counts(lib):
    assert attend(lib, p=pages(kv_heads=1024), a=attention(q_heads=1024 * 65)) == INV
    assert attend(lib, t=table(max_pages=1 << 24), a=attention(q_heads=256)) == INV  # more tiles than a list counts


@pytest.mark.parametrize("n", [1 << 31, (1 << 32) + 8, -(1 << 31) - 1, -(1 << 32)])
def test_the_binding_refuses_integers_that_do_not_fit(n):
    """None is cut to its low 32 bits on the way to the library."""
    torch = pytest.importorskip("torch")
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    pool = ss.KVPages(k, k.clone(), weight=torch.zeros(4, 2, 16))
    lens = torch.zeros(3, dtype=torch.int32)
    seqs, new = (ss.KVTable(torch.zeros(3, 5, dtype=torch.int32), x) for x in (lens, lens.clone()))
    with pytest.raises(ValueError, match="max_len"):
        ss.KVTable(seqs.pages, lens, max_len=n)
    with pytest.raises(ValueError, match="max_len"):
        seqs.max_len = n
    assert seqs.max_len == 0
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    for name in ("window", "sinks"):
        with pytest.raises(ValueError, match=name):
            ss.ss_kv_attend(pool, seqs, q, q.clone(), **{name: n})
    for name in ("keep", "sinks", "recent"):
        with pytest.raises(ValueError, match=name):
            ss.ss_kv_evict(pool, seqs, pool, new, **{"keep": 8, name: n})


def test_the_binding_refuses_tensors_that_are_not_on_the_caches_gpu(monkeypatch):
    """Nothing reaches the library: it would follow their addresses on the GPU."""
    torch = pytest.importorskip("torch")

    class Nothing:
        def __getattr__(self, name):
            raise AssertionError(f"{name} was called")

    monkeypatch.setattr(ss, "lib", lambda: Nothing())
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    pool = ss.KVPages(k, k.clone(), weight=torch.zeros(4, 2, 16))
    seqs, new = (ss.KVTable(torch.zeros(3, 5, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)) for _ in range(2))
    q, x = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    calls = [lambda: ss.ss_kv_attend(pool, seqs, q, q.clone()), lambda: ss.ss_kv_append(pool, seqs, x, x),
             lambda: ss.ss_kv_evict(pool, seqs, pool, new, 8)]
    for call in calls:
        with pytest.raises(ValueError, match="not on a GPU"):
            call()
    # the pool on a GPU, for all that the binding knows, and the tables elsewhere
    pool.device = 0
    for call, name in zip(calls, ("seqs", "seqs", "src_seqs")):
        with pytest.raises(ValueError, match=f"{name} is on cpu"):
            call()
