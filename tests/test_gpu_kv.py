"""The paged key-value cache (append, attend, evict) against the definitions
in 64 bits (tests/kv_helpers.py).

Tolerances.  u = 2^-8 (bf16: 7 fraction bits) or 2^-11 (fp16: 10) is half a
unit in the last place of the output type.  A score is a sum of `dim` products in fp32, so it is off
by at most e = dim * 2^-23 * scale * sum |q k| (+ 1e-6 for the scaling), and a
softmax weight by a factor 1 +- (2 e + 4e-6) with the exponential's and the
sums' rounding.  out is then within u |out| + (2 e + 4e-6 + r) max |v| of the
formula, where r bounds how weights are rounded for the product with v: 2^-16
for 16-bit caches, 2^-11 for 8-bit ones.  Moved rows, kept positions and
quantised values are exact."""

from __future__ import annotations

import math

import numpy as np
import pytest

from kv_helpers import Cache, attend_reference, e4m3_reference, evict_reference, torch_type, visible

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    import stream_compaction_pass_gb300 as m
    return m


def ok(ss, stream=None):
    st, where = ss.ss_stream_status(stream=stream)
    assert st == ss.SS_OK, (st, where, ss.ss_last_error_detail())


def run_attend(ss, c, group, qkind, window=0, sinks=0, weights="add", scale=None, seed=5, strided=False, lse=True,
               qscale=1.5):
    import torch
    gen = torch.Generator().manual_seed(seed)
    B, QH = len(c.lens), c.heads * group
    q_host = (torch.randn(B, QH, c.dim, generator=gen) * qscale).to(torch_type(qkind))
    if strided:  # the query part of a fused projection, out inside a wider buffer
        q = torch.full((B, QH + 5, c.dim + 16), math.nan, dtype=q_host.dtype, device="cuda")[:, :QH, :c.dim]
        q.copy_(q_host)
        wide = torch.full((QH, B, c.dim + 8), 7.0, dtype=q_host.dtype, device="cuda")
        out = wide.transpose(0, 1)[:, :, :c.dim]
    else:
        q = q_host.cuda()
        wide = None
        out = torch.full_like(q, math.nan)
    pages, table = c.ss(ss)
    d_lse = torch.full((B, QH), math.nan, device="cuda") if lse else None
    w_in = w_out = None
    if weights == "add":
        w_in = w_out = c.weight.clone()
    elif weights == "new":
        w_out = torch.full_like(c.weight, -3.0)
    elif weights == "apart":
        w_in, w_out = c.weight, torch.full_like(c.weight, -3.0)
    ss.ss_kv_attend(pages, table, q, out, scale=scale, window=window, sinks=sinks, lse=d_lse, weight_in=w_in, weight_out=w_out)
    ok(ss)
    if wide is not None:
        assert bool((wide[:, :, c.dim:] == 7.0).all()), "a store outside out's rows"
    return q_host.float().numpy(), out.float().cpu().numpy(), None if d_lse is None else d_lse.cpu().numpy(), \
        None if w_out is None else w_out.cpu().numpy()


def check_attend(ss, c, group, qkind, window=0, sinks=0, weights="add", scale=None, **kw):
    q, out, lse, w = run_attend(ss, c, group, qkind, window, sinks, weights, scale, **kw)
    sc = c.dim ** -0.5 if scale is None else scale
    want, want_lse, added = attend_reference(c, q, sc, window, sinks)
    u = 2.0 ** -8 if qkind == "bf16" else 2.0 ** -11
    r = 2.0 ** -11 if c.kind == "e4m3" else 2.0 ** -16
    for b, n in enumerate(c.lens):
        see = visible(n, window, sinks)
        for j in range(out.shape[1]):
            h = j // group
            if not see.any():
                assert (out[b, j] == 0).all() and (lse is None or lse[b, j] == -np.inf)
                continue
            k = np.abs(c.rows(c.k_host, b, h)[see]) * c.scale(c.ks, h)
            v = np.abs(c.rows(c.v_host, b, h)[see]) * c.scale(c.vs, h)
            e = c.dim * 2.0 ** -23 * abs(sc) * float((k @ np.abs(q[b, j]).astype(np.float64)).max()) + 1e-6
            tol = u * np.abs(want[b, j]) + (2 * e + 4e-6 + r) * v.max()
            bad = np.abs(out[b, j] - want[b, j]) > tol
            assert not bad.any(), (b, j, n, float(np.abs(out[b, j] - want[b, j]).max()), float(tol.max()))
            if lse is not None:
                assert abs(lse[b, j] - want_lse[b, j]) <= e + 1e-6 * (1 + abs(want_lse[b, j])), (b, j, lse[b, j], want_lse[b, j])
    if w is not None:
        start = {"add": c.w_host, "apart": c.w_host, "new": np.zeros_like(c.w_host)}[weights]
        kmax = np.nanmax(np.abs(c.k_host)) * (1.0 if c.ks is None else float(c.ks.max()))
        e = c.dim * 2.0 ** -23 * abs(sc) * float(np.abs(q).sum(-1).max()) * kmax + 1e-6
        for b in range(len(c.lens)):
            for h in range(c.heads):
                got, base, add = c.rows(w, b, h), c.rows(start, b, h), c.rows(added, b, h)
                assert (np.abs(got - (base + add)) <= (2 * e + 4e-6) * add + 2.0 ** -22 * (base + add)).all(), (b, h)
        untouched = np.isnan(c.w_host)
        if weights == "add":
            assert np.isnan(w[untouched]).all(), "a weight outside the sequences was written"
        else:
            assert (w[untouched] == -3.0).all(), "a weight outside the sequences was written"


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 100, 257]


@pytest.mark.parametrize("kind,qkind", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("dim", [16, 64, 80, 128, 256])
def test_attend_types_and_dims(ss, kind, qkind, dim):
    check_attend(ss, Cache(LENS, heads=2, dim=dim, page=16, kind=kind, seed=dim), 4, qkind)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("group", [1, 2, 3, 8, 9, 16, 17, 40])
def test_attend_groups(ss, kind, group):
    check_attend(ss, Cache([77, 0, 18, 300], heads=3, dim=64, page=32, kind=kind, seed=group), group, "bf16")


@pytest.mark.parametrize("page", [1, 3, 8, 16, 24, 64, 256])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_attend_pages_and_layouts(ss, page, layout):
    check_attend(ss, Cache([1, 50, 129, 500, 0, 63], heads=2, dim=128, page=page, kind="f16", seed=page, layout=layout), 2, "f16")


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (33, 0), (40, 17), (100, 100), (64, 1000), (5000, 3)])
@pytest.mark.parametrize("weights", ["add", "apart"])
def test_attend_window_and_sinks(ss, window, sinks, weights):
    check_attend(ss, Cache([0, 1, 16, 40, 64, 65, 101, 333, 700], heads=2, dim=64, page=16, seed=3), 2, "bf16", window, sinks, weights)


@pytest.mark.parametrize("weights", ["add", "new", "apart", None])
def test_attend_weights_forms(ss, weights):
    check_attend(ss, Cache([513, 4, 0, 90], heads=2, dim=128, page=32, seed=9), 8, "bf16", weights=weights, lse=weights != "new")


@pytest.mark.parametrize("n,heads,group,dim,kind", [(20011, 1, 8, 128, "bf16"), (9001, 2, 1, 64, "f16"), (30000, 1, 5, 128, "e4m3"),
                                                    (5003, 1, 2, 256, "bf16"), (12345, 1, 33, 64, "bf16")])
def test_attend_one_long_sequence_split_and_joined(ss, n, heads, group, dim, kind):
    check_attend(ss, Cache([n], heads=heads, dim=dim, page=64, kind=kind, seed=n), group, "f16" if kind == "f16" else "bf16")


def test_attend_many_short_sequences(ss):
    rng = np.random.default_rng(4)
    check_attend(ss, Cache(rng.integers(0, 40, 1300).tolist(), heads=2, dim=64, page=8, seed=4), 2, "bf16")


def test_attend_ragged_batch(ss):
    check_attend(ss, Cache([3000, 1, 0, 16, 1500, 47, 0, 2222, 9], heads=4, dim=128, page=16, seed=8), 4, "bf16")


def test_attend_strided_query_and_output(ss):
    check_attend(ss, Cache([5, 90, 200], heads=2, dim=64, page=16, seed=6), 3, "bf16", strided=True)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_attend_scales(ss, scale):
    # 2.0: a nearly one-hot softmax with scores in the hundreds
    check_attend(ss, Cache([64, 301], heads=2, dim=64, page=16, kind="f16", seed=7), 2, "f16", scale=scale)


def test_attend_large_values_in_an_8_bit_cache_with_large_queries(ss):
    # q beyond fp16's range in bf16: the scores are as if it were fp32
    check_attend(ss, Cache([40, 200], heads=2, dim=64, page=16, kind="e4m3", seed=10), 4, "bf16", qscale=3e5, scale=1e-6)


def test_attend_infinities_and_nan_spread_as_in_the_formula(ss):
    import torch
    c = Cache([30, 30, 30, 30], heads=1, dim=64, page=16, seed=11)

    def at(b, p):
        return int(c.table_host[b, p // 16]), 0, p % 16

    c.v[at(0, 7)] = math.nan      # sequence 0: out is NaN
    c.k[at(1, 3)] = math.nan      # sequence 1: everything is NaN
    for p in range(30):           # sequence 2: every score is -inf
        c.k[at(2, p)] = 0.0
        c.k[at(2, p) + (0,)] = -math.inf
    c.k[at(3, 5) + (0,)] = -math.inf  # sequence 3: one position drops out
    q = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    pages, table = c.ss(ss)
    out, lse, w = torch.empty_like(q), torch.empty(4, 2, device="cuda"), torch.zeros_like(c.weight)
    ss.ss_kv_attend(pages, table, q, out, lse=lse, weight_out=w)
    ok(ss)
    assert bool(out[0].isnan().all()) and bool(torch.isfinite(lse[0]).all())
    assert bool(out[1].isnan().all()) and bool(lse[1].isnan().all())
    assert bool((out[2] == 0).all()) and bool((lse[2] == -math.inf).all())
    assert all(float(w[at(2, p)]) == 0 for p in range(30))
    assert bool(torch.isfinite(out[3]).all()) and float(w[at(3, 5)]) == 0.0
    # the same rows where the window hides them change nothing
    out2 = torch.empty_like(q)
    c.v[at(3, 5)] = math.nan
    ss.ss_kv_attend(pages, table, q, out2, window=20)
    ok(ss)
    assert bool(torch.isfinite(out2[[0, 1, 3]]).all())
    # a NaN inside the window spreads to the visible weights only
    c.k[at(1, 25)] = math.nan
    w = torch.zeros_like(c.weight)
    ss.ss_kv_attend(pages, table, q, out2, window=20, weight_out=w)
    ok(ss)
    assert all(math.isnan(float(w[at(1, p)])) == (p >= 10) for p in range(30))
    assert all(float(w[at(1, p)]) == 0.0 for p in range(10))


def test_attend_is_the_same_on_every_run_and_stream(ss):
    import torch
    c = Cache([4001, 17, 900], heads=4, dim=128, page=16, seed=12)
    pages, table = c.ss(ss)
    q = torch.randn(3, 16, 128, device="cuda").to(torch.bfloat16)
    first = None
    torch.cuda.synchronize()
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(stream):
            out, w = torch.empty_like(q), torch.zeros_like(c.weight)
            for _ in range(3):
                ss.ss_kv_attend(pages, table, q, out, weight_out=w, stream=stream)
            stream.synchronize()
            ok(ss, stream)
        first = first or (out, w)
        assert torch.equal(out, first[0]) and torch.equal(w, first[1])


def test_attend_in_a_graph_reads_the_lengths_of_each_replay(ss):
    import torch
    c = Cache([600, 90], heads=2, dim=64, page=16, seed=13)
    pages, table = c.ss(ss)
    q = torch.randn(2, 4, 64, device="cuda").to(torch.bfloat16)
    out, want = torch.empty_like(q), torch.empty_like(q)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        ss.ss_kv_attend(pages, table, q, out, stream=side)
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            ss.ss_kv_attend(pages, table, q, out, stream=torch.cuda.current_stream())
    for lens in ([600, 90], [33, 1], [0, 77]):
        c.lens_dev.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        ss.ss_kv_attend(pages, table, q, want)
        ok(ss)
        assert torch.equal(out, want)


def test_attend_reports_bad_lengths_and_pages_and_keeps_the_other_sequences(ss):
    import torch
    c = Cache([100, 50, 60], heads=2, dim=64, page=16, seed=14)
    pages, table = c.ss(ss)
    q = torch.randn(3, 4, 64, device="cuda").to(torch.bfloat16)
    want, out = torch.empty_like(q), torch.empty_like(q)
    ss.ss_kv_attend(pages, table, q, want)
    ok(ss)
    good = c.table.clone()
    for value in (-1, c.num_pages, 2 ** 31 - 1, -2 ** 31):
        c.table.copy_(good)
        c.table[1, 2] = value
        ss.ss_kv_attend(pages, table, q, out)
        st, where = ss.ss_stream_status()
        assert (st, where) == (ss.SS_ERR_INVALID_ARG, 1)
        assert torch.equal(out[[0, 2]], want[[0, 2]])
    c.table.copy_(good)
    for n in (-5, c.width * 16 + 1, 2 ** 31 - 1):
        c.lens_dev[1] = n
        c.table[1] = good[0, 0]  # every entry names a real page: only the length is wrong
        ss.ss_kv_attend(pages, table, q, out)
        st, where = ss.ss_stream_status()
        assert (st, where) == (ss.SS_ERR_INVALID_ARG, 1)
        assert torch.equal(out[[0, 2]], want[[0, 2]])


def test_pool_past_32_bit_offsets(ss):
    import torch
    heads, dim, page = 8, 128, 64
    pages = (1 << 31) // (heads * dim * page) + 40  # more than 2^31 elements in each of k and v
    k = torch.zeros(pages, heads, page, dim, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    weight = torch.zeros(pages, heads, page, device="cuda")
    n = 10 * page - 7
    near, far = list(range(10)), list(range(pages - 10, pages))
    k[near] = torch.randn(10, heads, page, dim, device="cuda").to(torch.bfloat16)
    v[near] = torch.randn(10, heads, page, dim, device="cuda").to(torch.bfloat16)
    weight[near] = torch.rand(10, heads, page, device="cuda")
    for x in (k, v, weight):
        x[far] = x[near]
    cache = ss.KVPages(k, v, weight=weight)
    seqs = ss.KVTable(torch.tensor([near, far], dtype=torch.int32, device="cuda"), torch.tensor([n, n], dtype=torch.int32, device="cuda"))
    q = torch.randn(1, 16, dim, device="cuda").to(torch.bfloat16).expand(2, -1, -1).contiguous()
    out, lse = torch.empty_like(q), torch.empty(2, 16, device="cuda")
    ss.ss_kv_attend(cache, seqs, q, out, lse=lse)
    ok(ss)
    assert torch.allclose(out[0].float(), out[1].float(), rtol=2 ** -7, atol=1e-4) and float(out.float().abs().max()) > 0
    dst = list(range(pages - 20, pages - 15)), list(range(20, 25))
    new = ss.KVTable(torch.tensor(dst, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"))
    kept = torch.empty(2, heads, 300, dtype=torch.int32, device="cuda")
    ss.ss_kv_evict(cache, seqs, cache, new, 300, sinks=4, recent=30, kept=kept)
    ok(ss)
    assert torch.equal(kept[0], kept[1]) and new.lens.tolist() == [300, 300]
    rows = [x[d].transpose(1, 2).reshape(5 * page, heads, dim)[:300] for x in (k, v) for d in dst]
    assert torch.equal(rows[0], rows[1]) and torch.equal(rows[2], rows[3])
    idx = kept[0].long()
    whole = k[near].transpose(1, 2).reshape(10 * page, heads, dim)
    for h in range(heads):
        assert torch.equal(rows[0][:, h], whole[idx[h], h])
    x = torch.randn(2, heads, dim, device="cuda").to(torch.bfloat16)
    ss.ss_kv_append(cache, seqs, x, x)
    ok(ss)
    for b, last in enumerate((near[9], far[9])):
        assert torch.equal(k[last, :, (n - 1) % page], x[b]) and float(weight[last, :, (n - 1) % page].abs().max()) == 0.0


# ---- eviction ----

def run_evict(ss, c, weights, keep, sinks, recent, dst_page=None, dst_layout="hnd", with_kept=True, dst_weight=True):
    """Evicts c with the given weight pool and compares everything with the reference."""
    import torch
    c.weight.copy_(torch.from_numpy(weights))
    dst_page = dst_page or c.page
    kept_lens = [min(n, keep) for n in c.lens]
    d = Cache(kept_lens, heads=c.heads, dim=c.dim, page=dst_page, kind=c.kind, seed=77, layout=dst_layout, scales=False,
              with_weight=dst_weight)
    d.ks, d.vs = c.ks, c.vs
    before = [x.float().clone() for x in (d.k, d.v)]
    d.lens_dev.fill_(-9)
    pages, table = c.ss(ss)
    new_pages, new_table = d.ss(ss)
    kept = torch.full((len(c.lens), c.heads, keep), 12345, dtype=torch.int32, device="cuda") if with_kept else None
    ss.ss_kv_evict(pages, table, new_pages, new_table, keep, sinks=sinks, recent=recent, kept=kept)
    ok(ss)
    want = evict_reference(c, weights, keep, sinks, recent)
    assert d.lens_dev.tolist() == kept_lens
    if with_kept:
        assert np.array_equal(kept.cpu().numpy(), want)
    got = [x.float().cpu().numpy() for x in (d.k, d.v)]
    new_w = d.weight.cpu().numpy() if dst_weight else None
    touched = np.zeros(got[0].shape[:3], bool)
    for b, m in enumerate(kept_lens):
        j = np.arange(m)
        for h in range(c.heads):
            idx = want[b, h, :m]
            to = d.table_host[b, j // dst_page], h, j % dst_page
            touched[to] = True
            for x, host in zip(got, (c.k_host, c.v_host)):
                assert np.array_equal(x[to], c.rows(host, b, h)[idx])
            if dst_weight:
                assert np.array_equal(new_w[to].view(np.uint32), c.rows(weights, b, h)[idx].view(np.uint32))
    for x, old in zip(got, before):
        assert np.array_equal(x[~touched], old.cpu().numpy()[~touched], equal_nan=True), "a row outside the kept ones was written"


def random_weights(c, seed, zeros=0.2, levels=None):
    rng = np.random.default_rng(seed)
    w = np.exp(2.5 * rng.standard_normal(c.w_host.shape) - 8).astype(np.float32)
    if levels:
        w = rng.integers(0, levels, w.shape).astype(np.float32)
    w[rng.random(w.shape) < zeros] = 0.0
    return w


@pytest.mark.parametrize("kind,dim", [("bf16", 64), ("f16", 80), ("e4m3", 128), ("bf16", 256), ("e4m3", 16)])
@pytest.mark.parametrize("keep,sinks,recent", [(64, 4, 16), (1, 0, 0), (1, 1, 0), (1, 0, 1), (37, 20, 17), (200, 0, 0), (1000, 4, 100)])
def test_evict(ss, kind, dim, keep, sinks, recent):
    c = Cache([0, 1, 63, 64, 65, 300, 999, 1001], heads=2, dim=dim, page=16, kind=kind, seed=keep)
    run_evict(ss, c, random_weights(c, keep + dim), keep, sinks, recent)


@pytest.mark.parametrize("levels,zeros", [(1, 0.0), (2, 0.0), (3, 0.5), (40, 0.0)])
def test_evict_ties_go_to_the_lower_position(ss, levels, zeros):
    c = Cache([1500, 700, 33], heads=3, dim=16, page=16, seed=levels)
    run_evict(ss, c, random_weights(c, levels, zeros, levels), 301, 3, 50)


def test_evict_infinities_nan_and_signed_zeros(ss):
    c = Cache([800, 400], heads=2, dim=16, page=16, seed=2)
    rng = np.random.default_rng(3)
    w = rng.choice(np.array([np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1e-45, 1.0, -1.0, 3.4e38, -3.4e38], np.float32),
                   c.w_host.shape).astype(np.float32)
    for keep in (50, 399, 700):
        run_evict(ss, c, w, keep, 2, 9)


@pytest.mark.parametrize("page,layout,dst_page,dst_layout", [(16, "hnd", 64, "hnd"), (64, "nhd", 8, "hnd"), (7, "hnd", 3, "nhd"), (1, "nhd", 1, "nhd")])
def test_evict_between_page_sizes_and_layouts(ss, page, layout, dst_page, dst_layout):
    c = Cache([130, 257, 64], heads=2, dim=64, page=page, seed=page, layout=layout)
    run_evict(ss, c, random_weights(c, 5), 100, 4, 30, dst_page, dst_layout)


@pytest.mark.parametrize("n", [8191, 8192, 8193, 33000, 70001, 131073])
def test_evict_long(ss, n):
    c = Cache([n, n // 3], heads=2, dim=16, page=64, seed=n, kind="e4m3")
    run_evict(ss, c, random_weights(c, n), n // 4, 4, 1000)


def test_evict_very_long(ss):
    # longer than the keys of one row that shared memory can hold
    c = Cache([500_003], heads=1, dim=16, page=128, seed=1, kind="e4m3")
    run_evict(ss, c, random_weights(c, 1), 123_457, 4, 1000)


def test_evict_many_rows(ss):
    rng = np.random.default_rng(6)
    c = Cache(rng.integers(0, 200, 150).tolist(), heads=8, dim=16, page=16, seed=6)
    run_evict(ss, c, random_weights(c, 6), 48, 2, 8)


def test_evict_without_optional_outputs(ss):
    c = Cache([300, 20], heads=2, dim=64, page=16, seed=15)
    run_evict(ss, c, random_weights(c, 15), 64, 4, 16, with_kept=False, dst_weight=False)
    run_evict(ss, c, random_weights(c, 16), 64, 4, 16, with_kept=False)


def test_evict_reports_bad_pages(ss):
    import torch
    c = Cache([300, 200], heads=2, dim=64, page=16, seed=16)
    pages, table = c.ss(ss)
    d = Cache([64, 64], heads=2, dim=64, page=16, seed=17)
    new_pages, new_table = d.ss(ss)
    c.table[1, 3] = c.num_pages
    ss.ss_kv_evict(pages, table, new_pages, new_table, 64)
    assert ss.ss_stream_status() == (ss.SS_ERR_INVALID_ARG, 1)
    c.table[1, 3] = 0
    d.table[0, 1] = -7
    ss.ss_kv_evict(pages, table, new_pages, new_table, 64)
    assert ss.ss_stream_status() == (ss.SS_ERR_INVALID_ARG, 0)
    torch.cuda.synchronize()


# ---- append ----

def check_append(ss, lens, news, heads, dim, page, kind, src, layout="hnd", strided=False, offsets=True, values=None):
    import torch
    c = Cache(lens, heads=heads, dim=dim, page=page, kind=kind, seed=21, layout=layout)
    before = [x.float().cpu().numpy() for x in (c.k, c.v)] + [c.weight.cpu().numpy()]
    total = sum(news)
    gen = torch.Generator().manual_seed(22)
    if values is None:
        host = (torch.randn(total, 3, heads, dim, generator=gen) * 0.8).to(torch_type(src))
    else:
        host = torch.from_numpy(np.resize(values, (total, 3, heads, dim)).astype(np.float32)).to(torch_type(src))
    dev = host.cuda()
    k_new, v_new = (dev[:, 1], dev[:, 2]) if strided else (dev[:, 1].contiguous(), dev[:, 2].contiguous())
    starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    pages, table = c.ss(ss)
    ss.ss_kv_append(pages, table, k_new, v_new, offsets=torch.from_numpy(starts).cuda() if offsets else None)
    ok(ss)
    after = [x.float().cpu().numpy() for x in (c.k, c.v)] + [c.weight.cpu().numpy()]
    want = [x.copy() for x in before]
    for b, (n, m) in enumerate(zip(lens, news)):
        p = np.arange(n - m, n)
        at = c.table_host[b, p // page], slice(None), p % page
        for i, scale in ((0, c.ks), (1, c.vs)):
            x = host[starts[b]:starts[b + 1], i + 1].float().numpy()
            if kind == "e4m3":
                x = e4m3_reference(x / (np.float32(1) if scale is None else scale.numpy()[:, None]))
            want[i][at] = x
        want[2][at] = 0.0
    for got, ref in zip(after, want):
        assert np.array_equal(got, ref.astype(np.float32), equal_nan=True)


@pytest.mark.parametrize("kind,src", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f16")])
@pytest.mark.parametrize("dim,page", [(16, 16), (64, 1), (80, 7), (128, 16), (256, 64)])
def test_append_prompts(ss, kind, src, dim, page):
    check_append(ss, [100, 1, 0, 300, 64, 17], [100, 1, 0, 299, 5, 0], 3, dim, page, kind, src, strided=dim == 128)


@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_one_token_each(ss, kind, layout):
    check_append(ss, [1, 16, 17, 100, 333], [1] * 5, 8, 128, 16, kind, "bf16", layout, strided=True, offsets=False)


def test_append_rounds_saturates_and_keeps_nan(ss):
    steps = np.arange(-4096, 4096) / 512.0  # every neighbourhood of a tie at the small end
    hard = np.concatenate([steps, [np.inf, -np.inf, np.nan, 447, 449, 464, 465, 480, 1e5, -1e5, 2.0 ** -10, 2.0 ** -9, 3 * 2.0 ** -11, 0.0, -0.0]])
    check_append(ss, [200, 500], [200, 500], 2, 64, 16, "e4m3", "bf16", values=hard)
    check_append(ss, [200, 500], [200, 500], 2, 64, 16, "e4m3", "f16", values=hard[np.abs(np.nan_to_num(hard, posinf=1.0, neginf=1.0)) < 6e4])


def test_append_large_batch_of_prompts(ss):
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 700, 90).tolist()
    check_append(ss, lens, [int(rng.integers(0, n + 1)) for n in lens], 4, 64, 32, "bf16", "bf16")


def test_append_more_tokens_than_the_length_is_reported(ss):
    import torch
    c = Cache([10, 10], heads=1, dim=64, page=16, seed=23)
    pages, table = c.ss(ss)
    x = torch.zeros(16, 1, 64, dtype=torch.bfloat16, device="cuda")
    ss.ss_kv_append(pages, table, x, x, offsets=torch.tensor([0, 4, 16], dtype=torch.int32, device="cuda"))
    assert ss.ss_stream_status() == (ss.SS_ERR_INVALID_ARG, 1)


def test_a_sequence_lives_through_append_attend_and_evict(ss):
    """Weights gathered over steps decide what stays; attention over the
    evicted cache is attention over the kept rows."""
    import torch
    heads, group, dim, page = 2, 4, 64, 16
    c = Cache([120, 90], heads=heads, dim=dim, page=page, seed=31)
    c.weight.zero_()
    pages, table = c.ss(ss)
    gen = torch.Generator().manual_seed(32)
    expect = np.zeros(c.w_host.shape)
    for step in range(4):
        c.lens = [n + 1 for n in c.lens]
        c.lens_dev.add_(1)
        new = torch.randn(2, 2, heads, dim, generator=gen).to(torch.bfloat16)
        ss.ss_kv_append(pages, table, new[:, 0].cuda(), new[:, 1].cuda())
        for b in range(2):
            p = c.lens[b] - 1
            for host, i in ((c.k_host, 0), (c.v_host, 1)):
                host[c.table_host[b, p // page], :, p % page] = new[b, i].float().numpy()
        q = torch.randn(2, heads * group, dim, generator=gen).to(torch.bfloat16)
        out = torch.empty_like(q, device="cuda")
        ss.ss_kv_attend(pages, table, q.cuda(), out, weight_in=c.weight, weight_out=c.weight)
        ok(ss)
        want, _, added = attend_reference(c, q.float().numpy(), dim ** -0.5)
        expect += added
        assert np.abs(out.float().cpu().numpy() - want).max() <= 2.0 ** -8 * np.abs(want).max() + 2e-4
    held = ~np.isnan(c.weight.cpu().numpy())
    for b in range(2):
        for h in range(heads):
            assert np.allclose(c.rows(c.weight.cpu().numpy(), b, h), c.rows(expect, b, h), rtol=1e-4, atol=1e-7)
    assert held.any()
    weights = np.where(held, c.weight.cpu().numpy(), 0).astype(np.float32)
    run_evict(ss, c, weights, 70, 4, 20)


@pytest.mark.parametrize("dtype", ["bfloat16", "float8_e4m3fn"])
def test_example_decodes_within_a_budget(dtype):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_decode.py")
    spec = importlib.util.spec_from_file_location("paged_decode", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    got = example.run(batch=3, heads=2, group=4, dim=64, prompt=90, steps=60, budget=64, slack=16, sinks=2, recent=16, dtype=dtype, check=True)
    assert got["evictions"] >= 3 and max(got["lens"]) <= 80
    # out is rounded to bf16 (2^-8 of the value), weights under an 8-bit cache to fp16 (2^-11)
    assert got["worst"] <= 2.0 ** -8 + 2.0 ** -10


# ---- further sizes ----

@pytest.mark.parametrize("kind,dims", [("bf16", [8, 24, 72, 120, 136, 200, 248]), ("e4m3", [32, 48, 112, 144, 240])])
def test_attend_odd_dims(ss, kind, dims):
    for dim in dims:
        check_attend(ss, Cache([45, 3, 200], heads=2, dim=dim, page=16, kind=kind, seed=dim), 3, "bf16")


@pytest.mark.parametrize("kind,group", [("bf16", 128), ("e4m3", 128), ("f16", 64)])
def test_attend_one_shared_head(ss, kind, group):
    check_attend(ss, Cache([150, 0, 31, 2000], heads=1, dim=64, page=32, kind=kind, seed=group), group, "f16" if kind == "f16" else "bf16")


@pytest.mark.parametrize("dim", [64, 256])
def test_attend_more_sequences_than_one_launch_takes(ss, dim):
    rng = np.random.default_rng(dim)
    n = 600 if dim == 256 else 4200
    check_attend(ss, Cache(rng.integers(0, 20, n).tolist(), heads=1, dim=dim, page=16, seed=dim), 1, "bf16")


def test_attend_scratch_of_larger_calls_does_not_leak(ss):
    """The scratch of a large call does not leak into smaller ones."""
    check_attend(ss, Cache([9000, 5000], heads=2, dim=128, page=16, seed=41), 4, "bf16")
    for n in (1, 17, 400):
        check_attend(ss, Cache([n], heads=1, dim=128, page=16, seed=n), 2, "bf16")
        check_attend(ss, Cache([n, 0, n], heads=1, dim=128, page=16, seed=n), 2, "bf16", window=10, sinks=3, weights="apart")


def test_append_scales_of_every_size(ss):
    """Quotients next to ties and scales outside the reciprocal's range."""
    import torch
    gen = torch.Generator().manual_seed(51)
    heads, dim, n = 64, 128, 64
    for low, high in ((-3.0, 3.0), (-59.0, 59.0), (-120.0, 120.0)):
        c = Cache([n], heads=heads, dim=dim, page=16, kind="e4m3", seed=52)
        c.ks, c.vs = (torch.exp2(torch.rand(heads, generator=gen) * (high - low) + low) for _ in range(2))
        x = torch.randn(n, 2, heads, dim, generator=gen)
        ties = (torch.randint(16, 32, x.shape, generator=gen) * 2 + 1) * torch.exp2(torch.randint(-12, 4, x.shape, generator=gen).float())
        x = torch.where(torch.rand(x.shape, generator=gen) < 0.5, x * 20, ties) * c.ks[None, None, :, None]
        x = x.to(torch.bfloat16).clamp(-3e38, 3e38)
        pages, table = c.ss(ss)
        ss.ss_kv_append(pages, table, x[:, 0].contiguous().cuda(), x[:, 1].contiguous().cuda(),
                        offsets=torch.tensor([0, n], dtype=torch.int32).cuda())
        ok(ss)
        for i, (pool, scale) in enumerate(((c.k, c.ks), (c.v, c.vs))):
            with np.errstate(over="ignore", under="ignore"):
                want = e4m3_reference(x[:, i].float().numpy() / scale.numpy()[:, None])
            p = np.arange(n)
            got = pool.float().cpu().numpy()[c.table_host[0, p // 16], :, p % 16]
            assert np.array_equal(got, want.astype(np.float32))


@pytest.mark.parametrize("n,levels", [(40000, 1), (40000, 2), (70000, 5)])
def test_evict_long_rows_of_equal_weights(ss, n, levels):
    """More candidates than a row can list."""
    c = Cache([n, n - 1], heads=1, dim=16, page=64, seed=n, kind="e4m3")
    run_evict(ss, c, random_weights(c, levels, 0.3, levels), n // 3, 4, 500)


@pytest.mark.parametrize("rows", [1, 3, 80, 200])
def test_evict_rows_alone_and_together(ss, rows):
    """Few rows are split over clusters, many are a CTA each."""
    rng = np.random.default_rng(rows)
    c = Cache(rng.integers(17000, 21000, rows).tolist() if rows <= 3 else rng.integers(3000, 5000, rows).tolist(), heads=1, dim=16, page=32,
              seed=rows, kind="e4m3")
    run_evict(ss, c, random_weights(c, rows), 2500, 4, 700)


def test_back_to_back_calls_read_what_the_calls_before_them_wrote(ss):
    """Kernels of these calls may start before the ones ahead have ended; a run
    that waits between any two of them gives the same bits."""
    import torch

    def chain(wait):
        c = Cache([700, 350, 3000], heads=4, dim=128, page=16, seed=61)
        c.weight.nan_to_num_(0.0)
        d = Cache([256, 256, 256], heads=4, dim=128, page=16, seed=62)
        pages, table = c.ss(ss)
        new_pages, new_table = d.ss(ss)
        q0, x0 = torch.full((3, 16, 128), 0.01, device="cuda"), torch.full((3, 2, 4, 128), 0.5, device="cuda")
        outs = []
        kept = torch.empty(3, 4, 256, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()
        for step in range(30):
            x = (x0 * (step + 1)).sin().to(torch.bfloat16)
            wait()
            ss.ss_kv_append(pages, table, x[:, 0], x[:, 1])
            wait()
            q = (q0 * (step + 3)).cos().to(torch.bfloat16)
            out = torch.empty_like(q)
            wait()
            ss.ss_kv_attend(pages, table, q, out, weight_in=c.weight, weight_out=c.weight)
            wait()
            ss.ss_kv_evict(pages, table, new_pages, new_table, 256, sinks=4, recent=100, kept=kept)
            wait()
            again = torch.empty_like(q)
            ss.ss_kv_attend(new_pages, new_table, out, again)
            wait()
            outs += [out, again, kept.clone(), d.weight.clone()]
        ok(ss)
        return outs

    plain = chain(lambda: None)
    waited = chain(torch.cuda.synchronize)
    for i, (a, b) in enumerate(zip(plain, waited)):
        assert torch.equal(a.nan_to_num(7.0) if a.is_floating_point() else a, b.nan_to_num(7.0) if b.is_floating_point() else b), i


def test_evict_keeping_more_than_there_is(ss):
    """A budget past every length moves whole sequences and needs no scratch of its size."""
    import torch
    c = Cache([40, 0, 300], heads=2, dim=64, page=16, seed=63)
    d = Cache([40, 0, 300], heads=2, dim=64, page=16, seed=64)
    pages, table = c.ss(ss)
    new_pages, new_table = d.ss(ss)
    d.lens_dev.fill_(-1)
    ss.ss_kv_evict(pages, table, new_pages, new_table, 2 ** 31 - 1, sinks=4, recent=16)
    ok(ss)
    assert d.lens_dev.tolist() == [40, 0, 300]
    for new, host in ((d.k, c.k_host), (d.v, c.v_host), (d.weight, c.w_host)):
        got = new.float().cpu().numpy()
        for b in range(3):
            for h in range(2):
                assert np.array_equal(d.rows(got, b, h), c.rows(host, b, h).astype(np.float32))
    torch.cuda.synchronize()


@pytest.mark.parametrize("src", ["bf16", "f16"])
def test_append_keeps_the_sign_of_zeros(ss, src):
    """x / scale in an 8-bit cache, bit for bit: also -0, quotients that round
    to a zero, and negative scales."""
    import torch
    heads, n = 4, 8
    c = Cache([n], heads=heads, dim=16, page=16, kind="e4m3", seed=53)
    c.ks, c.vs = torch.tensor([1.0, 0.37, -0.37, 2.0 ** 70]), torch.tensor([24.0, -1.0, 2.0 ** -70, -3.0])
    x = torch.tensor([0.0, -0.0, 6e-5, -6e-5, 1e-7, -1e-7, 1.0, -1.0]).repeat(n, 2, heads, 2).to(torch_type(src))
    pages, table = c.ss(ss)
    ss.ss_kv_append(pages, table, x[:, 0].contiguous().cuda(), x[:, 1].contiguous().cuda(),
                    offsets=torch.tensor([0, n], dtype=torch.int32).cuda())
    ok(ss)
    for i, (pool, scale) in enumerate(((c.k, c.ks), (c.v, c.vs))):
        q = x[:, i].float().numpy() / scale.numpy()[:, None]
        want = np.copysign(e4m3_reference(q), q)
        p = np.arange(n)
        got = pool.float().cpu().numpy()[c.table_host[0, p // 16], :, p % 16]
        assert np.array_equal(got, want.astype(np.float32)) and np.array_equal(np.signbit(got), np.signbit(want))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("group", [4, 12])
@pytest.mark.parametrize("lens", [[40, 1, 700], [20] * 200, [50000]], ids=["small", "many", "long"])
def test_attend_infinite_visible_values(ss, kind, group, lens):
    """w v(p) is infinite in the dimensions where a visible v is, and the
    others are as if it were not there."""
    c = Cache(lens, heads=1, dim=64, page=16, kind=kind, seed=61)
    for b, n in enumerate(lens):
        for p, d, x in ((n // 2, 3, math.inf), (n - 1, 5, -math.inf), (0, 7, math.inf)):
            at = int(c.table_host[b, p // 16]), 0, p % 16, d
            c.v[at] = x
            c.v_host[at] = x
    q, out, _, _ = run_attend(ss, c, group, kind, weights=None)
    infinite = [3, 5, 7]
    want = np.zeros(out.shape)
    want[..., 3] = want[..., 7] = math.inf
    want[..., 5] = -math.inf
    assert np.array_equal(out[..., infinite], want[..., infinite])
    c.v_host[..., infinite] = 0.0
    want, _, _ = attend_reference(c, q, 64 ** -0.5)
    u = 2.0 ** -8 if kind == "bf16" else 2.0 ** -11
    for b in range(len(lens)):
        k, v = np.abs(c.rows(c.k_host, b, 0)), np.abs(c.rows(c.v_host, b, 0))
        for j in range(group):
            e = 64 * 2.0 ** -23 / 8 * float((k @ np.abs(q[b, j]).astype(np.float64)).max()) + 1e-6
            off = np.abs(np.delete(out[b, j] - want[b, j], infinite))
            assert (off <= np.delete(u * np.abs(want[b, j]), infinite) + (2 * e + 4e-6 + 2.0 ** -16) * v.max()).all()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("group", [4, 12])
@pytest.mark.parametrize("lens", [[40, 1, 700], [20] * 200, [50000]], ids=["small", "many", "long"])
def test_attend_rows_of_minus_infinity_ignore_their_values(ss, kind, group, lens):
    import torch
    c = Cache(lens, heads=1, dim=64, page=16, kind=kind, seed=62)
    c.k[:] = 0.0
    c.k[..., 0] = -math.inf
    c.v[..., 1] = math.inf
    q = torch.ones(len(lens), group, 64, dtype=c.k.dtype, device="cuda")
    pages, table = c.ss(ss)
    out, lse = torch.full_like(q, math.nan), torch.full((len(lens), group), math.nan, device="cuda")
    ss.ss_kv_attend(pages, table, q, out, lse=lse)
    ok(ss)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("lens", [[40, 700], [200] * 200, [50000]], ids=["small", "many", "long"])
def test_attend_values_near_the_largest_number(ss, lens):
    """The mean of values of 3e38 is 3e38, though their sum is not a number of fp32."""
    import torch
    c = Cache(lens, heads=1, dim=64, page=16, kind="bf16", seed=63)
    c.v[:] = 3e38
    q = torch.randn(len(lens), 4, 64, device="cuda").to(torch.bfloat16)
    pages, table = c.ss(ss)
    out = torch.empty_like(q)
    ss.ss_kv_attend(pages, table, q, out)
    ok(ss)
    # u, the exponential's and the sums' 4e-6, 2^-16 of the weights' rounding
    assert bool(((out.double() / c.v[0, 0, 0, 0].double() - 1).abs() <= 2.0 ** -8 + 4e-6 + 2.0 ** -16).all())


def shared(lens, **kw):
    """A cache whose sequences are beginnings of its longest one."""
    import torch
    c = Cache([max(lens)], **kw)
    c.lens, c.table_host = list(lens), np.repeat(c.table_host, len(lens), 0)
    c.table, c.lens_dev = torch.from_numpy(c.table_host).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    return c


@pytest.mark.parametrize("lens", [[100, 60, 1, 0, 100], [777] * 100 + [5000, 4999]])
def test_attend_and_evict_sequences_that_share_pages(ss, lens):
    check_attend(ss, shared(lens, heads=2, dim=64, page=16, seed=71), 4, "bf16", weights=None)
    check_attend(ss, shared(lens, heads=2, dim=64, page=16, kind="e4m3", seed=72), 4, "bf16", window=50, sinks=3, weights=None)
    c = shared(lens, heads=2, dim=64, page=16, seed=73)
    run_evict(ss, c, random_weights(c, 74), 40, 4, 10)


# ---- rows that are long within one warp's share: more of them than the GPU has warps ----

@pytest.mark.parametrize("kind,group,dim", [("f16", 8, 64), ("f16", 8, 256), ("f16", 12, 128), ("e4m3", 4, 128), ("e4m3", 12, 64)])
def test_attend_the_mean_of_ones_is_one(ss, kind, group, dim):
    """4e-6 of the exponential and the sums and 2^-16 of the weights are less
    than 2^-12, so that out rounds to one itself."""
    import torch
    c = shared([131072] * 2600, heads=1, dim=dim, page=128, kind=kind, seed=81, scales=False)
    c.v[:] = 1.0
    q = torch.randn(2600, group, dim, device="cuda").to(torch.float16)
    pages, table = c.ss(ss)
    out = torch.empty_like(q)
    ss.ss_kv_attend(pages, table, q, out)
    ok(ss)
    assert bool((out == 1.0).all()), float((out.float() - 1).abs().max())


@pytest.mark.parametrize("kind,group", [("f16", 5), ("f16", 12), ("bf16", 8), ("e4m3", 8), ("e4m3", 16)])
@pytest.mark.parametrize("slope", [8.0, -8.0])
def test_attend_scores_that_rise_or_fall_along_long_rows(ss, kind, group, slope):
    import torch
    n, B, dim = 9000, 2600, 64
    c = shared([n] * B, heads=1, dim=dim, page=16, kind=kind, seed=82, scales=False)
    p = np.arange(n)
    at = c.table_host[0, p // 16], 0, p % 16, 0
    c.k[at] = torch.linspace(-slope, slope, n, device="cuda").to(c.k.dtype)
    c.k_host[at] = c.k[at].float().cpu().numpy()
    row = torch.randn(1, group, dim, generator=torch.Generator().manual_seed(83)) * (0.05 if kind == "e4m3" else 1.0)
    row[..., 0] = 8.0
    q = row.to(torch_type("bf16" if kind == "bf16" else "f16")).cuda().expand(B, -1, -1).contiguous()
    pages, table = c.ss(ss)
    out, lse = torch.empty_like(q), torch.empty(B, group, device="cuda")
    ss.ss_kv_attend(pages, table, q, out, lse=lse)
    ok(ss)
    c.lens = [n]
    host = q[:1].float().cpu().numpy()
    want, want_lse, _ = attend_reference(c, host, dim ** -0.5)
    e = dim * 2.0 ** -23 * dim ** -0.5 * float((np.abs(c.rows(c.k_host, 0, 0)) @ np.abs(host[0].T.astype(np.float64))).max()) + 1e-6
    u, r = 2.0 ** -8 if kind == "bf16" else 2.0 ** -11, 2.0 ** -11 if kind == "e4m3" else 2.0 ** -16
    tol = u * np.abs(want) + (2 * e + 4e-6 + r) * np.abs(c.rows(c.v_host, 0, 0)).max()
    assert (np.abs(out.float().cpu().numpy() - want) <= tol).all()
    assert (np.abs(lse.cpu().numpy() - want_lse) <= e + 1e-6 * (1 + np.abs(want_lse))).all()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("group", [4, 12])
@pytest.mark.parametrize("lens", [[40, 1, 700], [20, 400] * 100, [50000]], ids=["small", "many", "long"])
def test_attend_infinite_values_of_scores_that_are_far_below_or_minus_infinity(ss, kind, group, lens):
    """The first quarter of a row scores 400 less than its second half and has
    infinite values in dimension 2: inf, as their weights are positive.  The
    second quarter scores -inf, with infinite values in dimension 1: NaN, as 0
    times them is.  Both fill whole tiles, shares and parts of the longer rows."""
    c = Cache(lens, heads=1, dim=64, page=16, kind=kind, seed=84)
    c.k[...] = 0.0
    c.k_host[...] = 0.0
    for b, n in enumerate(lens):
        for lo, hi, score, d in ((0, n // 4, -400.0, 2), (n // 4, n // 2, -math.inf, 1)):
            p = np.arange(lo, hi)
            at = c.table_host[b, p // 16], 0, p % 16
            for pool in (c.k, c.k_host):
                pool[at + (0,)] = score
            c.v[at + (d,)] = math.inf
            c.v_host[at + (d,)] = 0.0
    import torch
    q = torch.zeros(len(lens), group, 64)
    q[..., 0] = 1.0
    pages, table = c.ss(ss)
    dev = q.to(c.k.dtype).cuda()
    out = torch.empty_like(dev)
    ss.ss_kv_attend(pages, table, dev, out, scale=1.0)
    ok(ss)
    out = out.float().cpu().numpy()
    want, _, _ = attend_reference(c, q.numpy(), 1.0)
    u = 2.0 ** -8 if kind == "bf16" else 2.0 ** -11
    for b, n in enumerate(lens):
        assert np.isposinf(out[b, :, 2]).all() if n >= 4 else np.isfinite(out[b, :, 2]).all(), (b, n)
        assert np.isnan(out[b, :, 1]).all() if n // 2 > n // 4 else np.isfinite(out[b, :, 1]).all(), (b, n)
        # the scores are exact
        off, mean = np.delete(out[b] - want[b], [1, 2], 1), np.delete(want[b], [1, 2], 1)
        assert (np.abs(off) <= u * np.abs(mean) + (4e-6 + 2.0 ** -16) * np.abs(c.rows(c.v_host, b, 0)).max()).all()


# ---- scratch and stream capture ----

def captured(stream, work):
    import torch
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        work()
    return g


def test_evict_of_few_long_rows_in_a_graph_after_a_larger_call(ss):
    """Few rows are split and have histograms in scratch, where a larger batch
    is not split and has none; one call of the largest size provides for both."""
    import torch
    n, keep = 60000, 300
    c = shared([n] * 512, heads=1, dim=16, page=64, kind="e4m3", seed=91)
    w = random_weights(c, 92)
    c.weight.copy_(torch.from_numpy(w))
    kept = torch.full((512, 1, keep), -5, dtype=torch.int32, device="cuda")
    dst = Cache([keep] * 512, heads=1, dim=16, page=64, kind="e4m3", seed=93)
    pages, table = c.ss(ss)
    new_pages, new_table = dst.ss(ss)
    few, new_few = ss.KVTable(c.table[:8], c.lens_dev[:8]), ss.KVTable(dst.table[:8], dst.lens_dev[:8])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def evict(src, new):
        ss.ss_kv_evict(pages, src, new_pages, new, keep, sinks=4, recent=50, kept=kept[:src.batch], stream=side)

    evict(table, new_table)
    ok(ss, side)
    c.lens = [n]
    want = torch.from_numpy(evict_reference(c, w, keep, 4, 50)).cuda()
    assert bool((kept == want).all())
    g = captured(side, lambda: evict(few, new_few))
    for _ in range(3):
        kept.fill_(-5)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert bool((kept[:8] == want).all()) and bool((kept[8:] == -5).all())
        kept.fill_(-5)
        torch.cuda.synchronize()
        evict(few, new_few)  # an eager call between replays
        ok(ss, side)
        assert bool((kept[:8] == want).all())


def test_attend_in_a_graph_after_a_larger_call_that_took_more_launches(ss):
    """Scores of more than 2 GB are cut into launches: 8 sequences of up to
    2.2 million positions are eight, 5 of 1.9 million take two at a time."""
    import torch
    c = Cache([300, 40, 0, 700, 1, 90, 33, 16], heads=1, dim=16, page=1024, seed=94)
    q = torch.randn(8, 128, 16, device="cuda").to(torch.bfloat16)
    wide = torch.full((8, 2200), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.width] = c.table
    pages, _ = c.ss(ss)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def attend(batch, out, w, max_len):
        t = ss.KVTable(wide[:batch], c.lens_dev[:batch], max_len=max_len)
        ss.ss_kv_attend(pages, t, q[:batch], out[:batch], weight_out=w, stream=side)

    outs = [torch.zeros_like(q) for _ in range(2)]
    ws = [torch.zeros_like(c.weight) for _ in range(2)]
    torch.cuda.synchronize()
    attend(8, outs[0], ws[0], 2_200_000)
    ok(ss, side)
    g = captured(side, lambda: attend(5, outs[1], ws[1], 1_900_000))
    g.replay()
    torch.cuda.synchronize()
    ok(ss, side)
    # sums in another order, and one rounding more
    assert bool(((outs[1] - outs[0])[:5].float().abs() <= 2.0 ** -7 * outs[0][:5].float().abs() + 1e-4).all())
    for b in range(5):
        assert np.allclose(*(c.rows(w.cpu().numpy(), b, 0) for w in ws), rtol=1e-4, atol=0)


@pytest.mark.filterwarnings("ignore:The CUDA Graph is empty")
def test_nothing_is_allocated_in_a_capture(ss):
    """The call says so and enqueues nothing; one outside the capture, then a
    capture, work as ever, and the graph keeps its scratch when a larger call
    follows."""
    import torch
    c = Cache([5000, 300], heads=2, dim=64, page=16, seed=95)
    d = Cache([64, 64], heads=2, dim=64, page=16, seed=96)
    pages, table = c.ss(ss)
    new_pages, new_table = d.ss(ss)
    q = torch.randn(2, 8, 64, device="cuda").to(torch.bfloat16)
    out, w = torch.zeros_like(q), torch.zeros_like(c.weight)
    x = torch.ones(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    ss.ss_shutdown()  # no stream has a workspace
    attend = lambda: ss.ss_kv_attend(pages, table, q, out, weight_out=w, stream=side)
    evict = lambda: ss.ss_kv_evict(pages, table, new_pages, new_table, 64, stream=side)
    append = lambda: ss.ss_kv_append(pages, table, x, x, stream=side)

    def refused():
        for call in (append, attend, evict):  # the stream's first calls
            with pytest.raises(ss.StreamScanError) as e:
                call()
            assert e.value.status == ss.SS_ERR_NO_MEMORY and "captur" in str(e.value)

    g = captured(side, refused)
    side.synchronize()
    assert float(out.abs().max()) == 0.0
    append()  # makes the workspace, and no scratch

    def refused():
        for call in (attend, evict):
            with pytest.raises(ss.StreamScanError) as e:
                call()
            assert e.value.status == ss.SS_ERR_NO_MEMORY and "captur" in str(e.value)

    captured(side, refused)
    attend()
    ok(ss, side)
    want, want_w = out.clone(), w.clone()
    g = captured(side, attend)
    big = Cache([30000] * 4, heads=2, dim=64, page=16, seed=97)
    big_pages, big_table = big.ss(ss)
    big_q, big_w = torch.randn(4, 8, 64, device="cuda").to(torch.bfloat16), torch.zeros_like(big.weight)
    torch.cuda.synchronize()
    big_out = torch.empty_like(big_q)
    ss.ss_kv_attend(big_pages, big_table, big_q, big_out, weight_out=big_w, stream=side)
    fill = torch.full((1 << 26,), math.nan, device="cuda")  # whoever else allocates
    for _ in range(2):
        out.zero_()
        w.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(w, want_w)
    ok(ss, side)
    del fill


def test_evict_lists_the_kept_positions_of_the_largest_budget(ss):
    """A list of 2^31 - 1 places, past a counter's range with its last step."""
    import torch
    keep = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB")
    c = Cache([100], heads=1, dim=16, page=16, kind="e4m3", seed=98)
    d = Cache([100], heads=1, dim=16, page=16, kind="e4m3", seed=99)
    kept = torch.full((1, 1, keep), -7, dtype=torch.int32, device="cuda")
    pages, table = c.ss(ss)
    new_pages, new_table = d.ss(ss)
    ss.ss_kv_evict(pages, table, new_pages, new_table, keep, kept=kept)
    ok(ss)
    assert kept[0, 0, :100].tolist() == list(range(100)) and d.lens_dev.tolist() == [100]
    assert int(kept[0, 0, 100:].max()) == -1 and int(kept[0, 0, 100:].min()) == -1


def test_tensors_that_are_not_on_the_gpu_are_refused(ss):
    import torch
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    w, lens, pages = torch.zeros(4, 2, 16), torch.zeros(3, dtype=torch.int32), torch.zeros(3, 5, dtype=torch.int32)
    for args in (dict(k=k.cuda(), v=k), dict(k=k, v=k.cuda()), dict(k=k.cuda(), v=k.cuda(), weight=w)):
        with pytest.raises(ValueError, match="is on"):
            ss.KVPages(**args)
    for args in ((pages.cuda(), lens), (pages, lens.cuda())):
        with pytest.raises(ValueError, match="lens is on"):
            ss.KVTable(*args)
    pool, seqs = ss.KVPages(k.cuda(), k.cuda(), weight=w.cuda()), ss.KVTable(pages.cuda(), lens.cuda())
    q, x = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    g, y = q.cuda(), x.cuda()
    for args in (dict(q=q), dict(out=q), dict(lse=torch.zeros(3, 4)), dict(weight_out=w), dict(weight_in=w, weight_out=w.cuda()), dict(seqs=ss.KVTable(pages, lens)),
                 dict(cache=ss.KVPages(k, k))):
        with pytest.raises(ValueError, match="on a GPU" if "cache" in args else "is on cpu"):
            ss.ss_kv_attend(**{"cache": pool, "seqs": seqs, "q": g, "out": g.clone(), **args})
    for args in (dict(k_new=x), dict(v_new=x), dict(offsets=torch.zeros(4, dtype=torch.int32))):
        with pytest.raises(ValueError, match="is on cpu"):
            ss.ss_kv_append(**{"cache": pool, "seqs": seqs, "k_new": y, "v_new": y, **args})
    for args in (dict(dst=ss.KVPages(k, k)), dict(dst_seqs=ss.KVTable(pages, lens)), dict(kept=torch.zeros(3, 2, 8, dtype=torch.int32))):
        with pytest.raises(ValueError, match="is on cpu"):
            ss.ss_kv_evict(**{"src": pool, "src_seqs": seqs, "dst": pool, "dst_seqs": seqs, "keep": 8, **args})
    ok(ss)


@pytest.mark.parametrize("batch", [2, 700])
def test_attend_with_weights_over_tables_without_pages(ss, batch):
    """On a stream that has no scratch yet."""
    import torch
    c = Cache([5], heads=2, dim=64, page=16, seed=100)
    pages, _ = c.ss(ss)
    q = torch.randn(batch, 4, 64, device="cuda").to(torch.bfloat16)
    out, lse, w = torch.full_like(q, 3.0), torch.zeros(batch, 4, device="cuda"), torch.full_like(c.weight, -3.0)
    seqs = ss.KVTable(torch.empty(batch, 0, dtype=torch.int32, device="cuda"), torch.zeros(batch, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    ss.ss_shutdown()
    ss.ss_kv_attend(pages, seqs, q, out, lse=lse, weight_out=w)
    ok(ss)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all()) and bool((w == -3.0).all())


def test_scratch_grows_in_steps_where_the_longest_length_grows(ss):
    """A decode loop that sets max_len to the longest length in use: the
    scratch of the scores grows by half at least, in a few steps."""
    import ctypes

    import torch
    cuda = ctypes.CDLL("libcuda.so.1")
    pool, used = ctypes.c_void_p(), ctypes.c_uint64()
    assert cuda.cuDeviceGetDefaultMemPool(ctypes.byref(pool), torch.cuda.current_device()) == 0

    def held():  # CU_MEMPOOL_ATTR_USED_MEM_CURRENT
        assert cuda.cuMemPoolGetAttribute(pool, 7, ctypes.byref(used)) == 0
        return used.value

    c = Cache([100], heads=4, dim=64, page=64, seed=101)
    pages, _ = c.ss(ss)
    table = torch.full((40, 1200), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(40, dtype=torch.int32, device="cuda")
    q = torch.randn(40, 16, 64, device="cuda").to(torch.bfloat16)
    out, w = torch.empty_like(q), torch.zeros_like(c.weight)
    torch.cuda.synchronize()
    ss.ss_shutdown()
    sizes = []
    for n in range(64, 64 * 1200, 64):
        ss.ss_kv_attend(pages, ss.KVTable(table, lens, max_len=n), q, out, weight_out=w)
        torch.cuda.synchronize()
        sizes.append(held())
    ok(ss)
    steps = [(a, b) for a, b in zip(sizes, sizes[1:]) if a != b]
    # 16 scores of 4 bytes a position and sequence, beside some MB of parts
    assert sizes[-1] - sizes[0] >= 40 * 64 * 1190 * 16 * 4 - (64 << 20)
    assert len(steps) <= 12, steps


# ---- the forms that only larger calls take ----

@pytest.mark.parametrize("page", [64, 7])
@pytest.mark.parametrize("levels", [1, 2, None])
def test_evict_very_long_rows_with_more_candidates_than_they_can_list(ss, page, levels):
    """One row over 8 CTAs, each with more positions than shared memory holds
    keys of, of which (but for spread weights) more share T's digits than a
    CTA lists."""
    c = Cache([300_007], heads=1, dim=16, page=page, seed=111, kind="e4m3")
    run_evict(ss, c, random_weights(c, 112, 0.0 if levels == 1 else 0.3, levels), 100_001, 4, 1000)


@pytest.mark.parametrize("page", [64, 7])
@pytest.mark.parametrize("levels", [1, 3, None])
def test_evict_many_long_rows_of_one_cta_each(ss, page, levels):
    """Rows for more than half the SMs are not split, however long; some are
    below the budget."""
    lens = [17000 + 287 * i for i in range(80)] + [16385, 9000, 12345, 12346, 0, 3]
    c = shared(lens, heads=1, dim=16, page=page, seed=113, kind="e4m3")
    run_evict(ss, c, random_weights(c, 114, 0.2, levels), 12_345, 4, 700)


RAGGED = [int(n) for n in np.random.default_rng(115).integers(0, 400, 60)] + [1500, 777, 0, 1]


@pytest.mark.parametrize("window,sinks", [(1, 0), (33, 5), (200, 0), (256, 40), (900, 4)])
@pytest.mark.parametrize("weights", ["add", "apart", "new"])
@pytest.mark.parametrize("group,page", [(4, 16), (3, 7), (12, 16)])
def test_attend_windows_and_weights_of_batches(ss, window, sinks, weights, group, page):
    """More rows than clusters: the list over all sequences, cut anywhere."""
    check_attend(ss, Cache(RAGGED, heads=3, dim=64, page=page, seed=116), group, "bf16", window, sinks, weights)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,qkind", [(4, "bf16"), (8, "f16"), (12, "bf16"), (16, "f16")])
@pytest.mark.parametrize("window", [0, 100])
def test_attend_8_bit_batches(ss, dim, group, qkind, window):
    check_attend(ss, Cache(RAGGED, heads=3, dim=dim, page=32, kind="e4m3", seed=117), group, qkind, window, 3, "apart")


@pytest.mark.parametrize("kind,dim,group", [("bf16", 128, 4), ("f16", 256, 8), ("bf16", 256, 9), ("f16", 128, 16), ("bf16", 80, 5)])
def test_attend_16_bit_batches(ss, kind, dim, group):
    check_attend(ss, Cache(RAGGED, heads=3, dim=dim, page=16, kind=kind, seed=118), group, kind)


@pytest.mark.parametrize("n,heads,group,dim,kind", [(80011, 2, 1, 64, "f16"), (50021, 1, 5, 128, "e4m3"), (12007, 1, 2, 256, "bf16"), (30011, 1, 12, 128, "f16")])
@pytest.mark.parametrize("weights", ["add", None])
def test_attend_one_sequence_too_long_for_one_launch(ss, n, heads, group, dim, kind, weights):
    check_attend(ss, Cache([n], heads=heads, dim=dim, page=64, kind=kind, seed=n), group, "f16" if kind == "f16" else "bf16", weights=weights)


@pytest.mark.parametrize("lens", [[100, 64, 0, 7], [100, 64, 0, 7] * 60], ids=["small", "many"])
def test_a_tight_bound_on_the_lengths_and_a_length_above_it(ss, lens):
    """max_len is all that a launch provides for; a longer length, though its
    table has the pages, is clamped and reported."""
    import torch
    c = Cache(lens, heads=3, dim=64, page=16, seed=119)
    pages, table = c.ss(ss)
    d = Cache([50] * len(lens), heads=3, dim=64, page=16, seed=120)
    new_pages, new_table = d.ss(ss)
    q = torch.randn(len(lens), 12, 64, device="cuda").to(torch.bfloat16)
    outs, ws, kepts = [], [], []
    for max_len in (None, 100, 80):
        seqs = ss.KVTable(c.table, c.lens_dev, max_len=max_len)
        out, w = torch.empty_like(q), torch.zeros_like(c.weight)
        kept = torch.empty(len(lens), 3, 50, dtype=torch.int32, device="cuda")
        ss.ss_kv_attend(pages, seqs, q, out, weight_out=w)
        late = max_len == 80
        assert ss.ss_stream_status()[0] == (ss.SS_ERR_INVALID_ARG if late else ss.SS_OK)
        ss.ss_kv_evict(pages, seqs, new_pages, new_table, 50, sinks=4, recent=10, kept=kept)
        st, where = ss.ss_stream_status()
        assert st == (ss.SS_ERR_INVALID_ARG if late else ss.SS_OK) and (not late or lens[where] == 100)
        outs.append(out)
        ws.append(w)
        kepts.append(kept)
    short = [b for b, n in enumerate(lens) if n <= 80]
    for i in (1, 2):
        rows = range(len(lens)) if i == 1 else short
        assert bool(((outs[i] - outs[0])[rows].float().abs() <= 2.0 ** -7 * outs[0][rows].float().abs() + 1e-4).all())
        assert torch.equal(kepts[i][rows], kepts[0][rows])
    for b, n in enumerate(lens):
        if n != 100:
            assert np.allclose(c.rows(ws[2].cpu().numpy(), b, 1), c.rows(ws[0].cpu().numpy(), b, 1), rtol=1e-4, atol=0)
    assert np.allclose(ws[1].cpu().numpy(), ws[0].cpu().numpy(), rtol=1e-4, atol=0)


def test_example_evicts_by_weights_that_attention_has_gathered(ss, monkeypatch):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "paged_decode.py")
    spec = importlib.util.spec_from_file_location("paged_decode", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    evict, seen = ss.ss_kv_evict, []

    def check(src, src_seqs, *args, **kw):
        page = src.weight.shape[2]
        for row, n in zip(src_seqs.pages.tolist(), src_seqs.lens.tolist()):
            w = src.weight[row].transpose(1, 2).flatten(0, 1)[:n]
            assert len(row) * page >= n and float(w.sum(0).min()) > 0.0
        seen.append(1)
        evict(src, src_seqs, *args, **kw)

    monkeypatch.setattr(ss, "ss_kv_evict", check)
    got = example.run(batch=3, heads=2, group=4, dim=64, prompt=90, steps=20, budget=64, slack=16, sinks=2, recent=16, check=True)
    assert got["evictions"] == len(seen) == 2 and got["worst"] <= 2.0 ** -8 + 2.0 ** -10


def test_strides_of_extents_of_one_are_not_looked_at(ss):
    """As a slice of one row of a wider buffer leaves them."""
    import torch
    c = Cache([9], heads=1, dim=64, page=16, seed=121)
    pages, table = c.ss(ss)
    q = torch.randn(1, 1, 64, device="cuda").to(torch.bfloat16)
    want, out = torch.empty_like(q), torch.zeros_like(q)

    def odd(x):
        return x.as_strided(x.shape, [n if m > 1 else 13 for n, m in zip(x.stride(), x.shape)])

    ss.ss_kv_attend(pages, table, q, want)
    ss.ss_kv_attend(pages, table, odd(q), odd(out))
    ok(ss)
    assert torch.equal(out, want)
    x = torch.randn(1, 1, 64, device="cuda").to(torch.bfloat16)
    one = ss.KVPages(odd(c.k), odd(c.v), weight=c.weight)  # one head
    assert one._c.head_stride == 13
    ss.ss_kv_append(one, table, odd(x), odd(x))
    ok(ss)
    assert torch.equal(c.k[int(c.table[0, 0]), 0, 8], x[0, 0])
    dst = Cache([4], heads=1, dim=64, page=4, spare=0, seed=122)  # one page
    new = ss.KVPages(odd(dst.k), odd(dst.v), weight=dst.weight)
    assert new._c.page_stride == 13
    c.weight.fill_(1.0)
    ss.ss_kv_evict(one, table, new, ss.KVTable(dst.table, dst.lens_dev), 4, sinks=1, recent=3)
    ok(ss)
    assert torch.equal(dst.k[0, 0], c.k[int(c.table[0, 0]), 0, [0, 6, 7, 8]])


@pytest.mark.parametrize("kind,qkind", [("e4m3", "bf16"), ("e4m3", "f16"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("dim", [128, 256])
@pytest.mark.parametrize("group", [1, 8])
@pytest.mark.parametrize("batch", [10, 600], ids=["small", "many"])
def test_attend_weights_are_finer_than_the_rounding_of_out(ss, kind, qkind, dim, group, batch):
    """Two positions of scores s and 0 and values 1 and -1: out = tanh(s / 2),
    which for small s shows what rounds a weight: 2^-16 of it and 4e-6 of the
    exponential and the sums, beside the rounding of out."""
    c = Cache([2] * batch, heads=1, dim=dim, page=16, kind=kind, seed=123, scales=False)
    c.k[:] = 0.0
    c.k[c.table[:, 0].long(), 0, 0, 0] = 1.0
    c.v[:] = -1.0
    c.v[c.table[:, 0].long(), 0, 0] = 1.0
    import torch
    s = (torch.arange(1, batch * group + 1).view(batch, group) * (0.3 / (batch * group))).to(torch_type(qkind))
    q = torch.zeros(batch, group, dim, dtype=s.dtype)
    q[..., 0] = s
    pages, table = c.ss(ss)
    out = torch.empty_like(q, device="cuda")
    ss.ss_kv_attend(pages, table, q.cuda(), out, scale=1.0)
    ok(ss)
    want = torch.tanh(s.double() / 2)[..., None]
    u = 2.0 ** -8 if qkind == "bf16" else 2.0 ** -11
    assert bool(((out.cpu().double() - want).abs() <= u * want + 4e-6 + 2.0 ** -16).all())


@pytest.mark.parametrize("kind,dim,group", [("bf16", 256, 4), ("f16", 128, 12)])
@pytest.mark.parametrize("weights", [False, True])
def test_attend_in_a_graph_after_a_larger_call_that_took_one_launch(ss, kind, dim, group, weights):
    """Where clusters fill the GPU a call takes one launch, and no scratch for
    parts, which a call of fewer sequences needs."""
    import torch
    n = 1000 if dim == 256 else 2000
    if weights:
        n //= 3
    c = Cache([n] * 32, heads=4, dim=dim, page=16, kind=kind, seed=125)
    pages, _ = c.ss(ss)
    q = torch.randn(32, 4 * group, dim, device="cuda").to(c.k.dtype)
    out, lse = torch.zeros_like(q), torch.zeros(32, 4 * group, device="cuda")
    w = torch.zeros_like(c.weight) if weights else None
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    ss.ss_shutdown()

    def attend(batch):
        t = ss.KVTable(c.table[:batch], c.lens_dev[:batch], max_len=n)
        ss.ss_kv_attend(pages, t, q[:batch], out[:batch], lse=lse[:batch], weight_out=w, stream=side)

    attend(32)
    ok(ss, side)
    want, want_lse = out.clone(), lse.clone()
    for batch in (31, 20, 10, 5, 2, 1):
        g = captured(side, lambda: attend(batch))
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        ok(ss, side)
        assert bool(((out - want)[:batch].float().abs() <= 2.0 ** -7 * want[:batch].float().abs() + 1e-4).all())
        assert torch.allclose(lse[:batch], want_lse[:batch], rtol=1e-5, atol=1e-5)
