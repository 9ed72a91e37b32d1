"""The paged cache in 4 bits (append, attend, evict) against the definitions in
64 bits (tests/serving_helpers.py).

Tolerances.  Codes times their block's scale are exact in fp16, so that what
enters the products is exact but for queries of bf16 that lie 2^-32 below their
row's largest.  A score is a sum of `dim` products in fp32, off by at most e = dim *
2^-23 * scale * sum |q k| (+ 1e-6 for the scaling), and a softmax weight by a factor
1 +- (2 e + 4e-6) with the exponential's and the sums' rounding.  out is then within
u |out| + (2 e + 4e-6 + r) max |v| of the formula, u half a unit in the last place of
its type (bf16 2^-8, fp16 2^-11), where r bounds how a weight is rounded for the
product with v: 2^-11, half a unit of fp16, under bf16 queries, 2^-16 under fp16
ones (two terms).  Quantised codes and scales, moved rows and kept positions are
exact."""

from __future__ import annotations

import math

import numpy as np
import pytest

from kv_helpers import attend_reference, evict_reference, torch_type, visible
from serving_helpers import Cache4, quantise4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    import stream_compaction_pass_gb300 as m
    return m


def ok(ss, stream=None):
    st, where = ss.ss_stream_status(stream=stream)
    assert st == ss.SS_OK, (st, where, ss.ss_last_error_detail())


def queries(c, group, kind, seed=5, scale=1.5):
    import torch
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(len(c.lens), c.heads * group, c.dim, generator=gen) * scale).to(torch_type(kind))


def check_outputs(c, group, kind, q, out, lse, window, sinks, scale=None):
    sc = c.dim ** -0.5 if scale is None else scale
    want, want_lse, added = attend_reference(c, q, sc, window, sinks)
    u, r = (2.0 ** -8, 2.0 ** -11) if kind == "bf16" else (2.0 ** -11, 2.0 ** -16)
    for b, n in enumerate(c.lens):
        see = visible(n, window, sinks)
        for j in range(out.shape[1]):
            h = j // group
            if not see.any():
                assert (out[b, j] == 0).all() and lse[b, j] == -np.inf
                continue
            k = np.abs(c.rows(c.k_host, b, h)[see]) * c.scale(c.ks, h)
            v = np.abs(c.rows(c.v_host, b, h)[see]) * c.scale(c.vs, h)
            e = c.dim * 2.0 ** -23 * abs(sc) * float((k @ np.abs(q[b, j]).astype(np.float64)).max()) + 1e-6
            off = np.abs(out[b, j] - want[b, j])
            tol = u * np.abs(want[b, j]) + (2 * e + 4e-6 + r) * v.max()
            assert (off <= tol).all(), (b, j, n, float((off - tol).max()))
            assert abs(lse[b, j] - want_lse[b, j]) <= e + 1e-6 * (1 + abs(want_lse[b, j])), (b, j, n)
    return added


def check_attend(ss, c, group, kind, window=0, sinks=0, weights="add", scale=None, stream=None):
    import torch
    q_host = queries(c, group, kind)
    q = q_host.cuda()
    out, lse = torch.full_like(q, math.nan), torch.full(q.shape[:2], math.nan, device="cuda")
    pages, table = c.ss(ss)
    w_in = w_out = None
    if weights == "add":
        w_in = w_out = c.weight.clone()
    elif weights == "apart":
        w_in, w_out = c.weight, torch.full_like(c.weight, -3.0)
    ss.ss_kv_attend(pages, table, q, out, scale=scale, window=window, sinks=sinks, lse=lse, weight_in=w_in, weight_out=w_out, stream=stream)
    ok(ss, stream)
    qn = q_host.float().numpy()
    added = check_outputs(c, group, kind, qn, out.float().cpu().numpy(), lse.cpu().numpy(), window, sinks, scale)
    if w_out is not None:
        w = w_out.cpu().numpy()
        sc = c.dim ** -0.5 if scale is None else scale
        e = c.dim * 2.0 ** -23 * abs(sc) * float(np.abs(qn).sum(-1).max()) * np.nanmax(np.abs(c.k_host)) * (1.0 if c.ks is None else float(c.ks.max())) + 1e-6
        for b in range(len(c.lens)):
            for h in range(c.heads):
                got, base, add = c.rows(w, b, h), c.rows(c.w_host, b, h), c.rows(added, b, h)
                assert (np.abs(got - (base + add)) <= (2 * e + 4e-6) * add + 2.0 ** -22 * (base + add)).all(), (b, h)
        untouched = np.isnan(c.w_host)
        assert (np.isnan(w) if weights == "add" else w == -3.0)[untouched].all(), "a weight outside the sequences was written"


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 100, 257]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [3, 12])
def test_attend_types_and_dims(ss, kind, dim, group):
    check_attend(ss, Cache4(LENS, dim=dim, seed=1), group, kind)


@pytest.mark.parametrize("group", [1, 2, 8, 9, 16, 17, 40])
def test_attend_groups(ss, group):
    check_attend(ss, Cache4([70, 200, 5], dim=128, seed=2), group, "bf16")


@pytest.mark.parametrize("page", [1, 2, 3, 8, 16, 24, 32, 48, 64, 100, 128, 192])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("many", [False, True], ids=["small", "many"])
def test_attend_pages_and_layouts(ss, page, layout, many):
    """Whole tiles of pages that hold, divide or straddle them, and of other layouts."""
    lens = [130, 64, 1, 400] + ([90, 300, 65] * 40 if many else [])
    check_attend(ss, Cache4(lens, dim=128, page=page, layout=layout, seed=3), 4, "bf16")


@pytest.mark.parametrize("dim,page", [(64, 16), (64, 32), (64, 64), (64, 8), (256, 8), (256, 4), (256, 32), (256, 16)])
@pytest.mark.parametrize("group", [5, 11])
def test_attend_pages_of_other_dims(ss, dim, page, group):
    check_attend(ss, Cache4([200, 64, 1, 333] + [150, 20] * 60, dim=dim, page=page, seed=4), group, "f16")


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (64, 64), (65, 3), (100, 130), (64, 1000), (5000, 3)])
@pytest.mark.parametrize("weights", ["add", "apart"])
@pytest.mark.parametrize("many", [False, True], ids=["small", "many"])
def test_attend_window_and_sinks(ss, window, sinks, weights, many):
    check_attend(ss, Cache4(LENS + [500] + ([300, 77] * 50 if many else []), dim=128, page=16, seed=6), 2, "bf16", window, sinks, weights)


@pytest.mark.filterwarnings("ignore:All-NaN")
@pytest.mark.parametrize("lens", [[0] * 200, [0] * 150 + [900, 3] + [0] * 100, [900] + [0, 1] * 90 + [1, 2, 3] * 30, [1] * 300], ids=["none", "two", "mixed", "ones"])
@pytest.mark.parametrize("window,weights", [(0, "add"), (40, "apart")])
def test_attend_padded_batches(ss, lens, window, weights):
    """Sequences without a position, and rows that are shorter than a warp's share."""
    check_attend(ss, Cache4(lens, dim=64, page=16, seed=16), 3, "bf16", window, 2, weights)


@pytest.mark.parametrize("n,heads,group,dim", [(30011, 1, 8, 128), (20000, 2, 1, 64), (12007, 1, 5, 256), (15000, 1, 12, 128)])
@pytest.mark.parametrize("weights", ["add", None])
def test_attend_one_long_sequence(ss, n, heads, group, dim, weights):
    check_attend(ss, Cache4([n], heads=heads, dim=dim, page=64, seed=7), group, "bf16", weights=weights)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_attend_scales(ss, scale):
    check_attend(ss, Cache4([40, 300], dim=64, seed=8), 4, "f16", scale=scale, weights=None)


def test_attend_without_head_scales(ss):
    check_attend(ss, Cache4([40, 300], dim=128, scales=False, seed=9), 4, "bf16")


@pytest.mark.parametrize("dim,batch", [(64, 2100), (256, 600)])
def test_attend_more_sequences_than_one_launch_takes(ss, dim, batch):
    rng = np.random.default_rng(10)
    check_attend(ss, Cache4([int(x) for x in rng.integers(0, 40, batch)], heads=1, dim=dim, page=16, seed=10), 2, "bf16")


def test_attend_long_rows_of_one_value(ss):
    """Sums of many products of one sign: the mean of equal values is that value."""
    import torch
    c = Cache4([60000], heads=1, dim=128, page=64, scales=False, seed=11)
    c.v.fill_(0x22)  # 1
    c.vb.view(torch.uint8).fill_(0x38)  # times 1
    pages, table = c.ss(ss)
    for kind in ("bf16", "f16"):
        q = (queries(c, 4, kind) * 0.01).cuda()
        out = torch.empty_like(q)
        ss.ss_kv_attend(pages, table, q, out)
        ok(ss)
        assert float((out.float() - 1).abs().max()) <= (2.0 ** -8 if kind == "bf16" else 2.0 ** -11)


def test_attend_nan_scales_spread_to_their_dimensions_only(ss):
    import torch
    c = Cache4([100, 90], heads=1, dim=128, page=16, seed=12)
    at = int(c.table_host[0, 3]), 0, 5  # position 53 of sequence 0
    c.vb.view(torch.uint8)[at][2] = 127
    c.v_host[at][32:48] = np.nan
    pages, table = c.ss(ss)
    q = queries(c, 2, "bf16")
    out = torch.empty_like(q, device="cuda")
    ss.ss_kv_attend(pages, table, q.cuda(), out)
    ok(ss)
    got = torch.isnan(out).cpu().numpy()
    want = np.zeros(got.shape, bool)
    want[0, :, 32:48] = True
    assert np.array_equal(got, want)


def test_attend_is_the_same_on_every_run_and_stream(ss):
    import torch
    c = Cache4([4000, 17, 900] * 20, dim=128, page=16, seed=13)
    pages, table = c.ss(ss)
    q = queries(c, 4, "bf16").cuda()
    first, w = torch.empty_like(q), torch.zeros_like(c.weight)
    ss.ss_kv_attend(pages, table, q, first, weight_out=w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        out, w2 = torch.empty_like(q), torch.zeros_like(c.weight)
        side.wait_stream(torch.cuda.current_stream())
        ss.ss_kv_attend(pages, table, q, out, weight_out=w2, stream=side)
        side.synchronize()
        assert torch.equal(out, first) and torch.equal(w2, w)
    ok(ss, side)


@pytest.mark.parametrize("lens", [[100, 64, 7], [100, 64, 7] * 60], ids=["small", "many"])
def test_attend_reports_bad_pages_and_keeps_the_other_sequences(ss, lens):
    import torch
    c = Cache4(lens, dim=128, page=16, seed=14)
    pages, table = c.ss(ss)
    q = queries(c, 4, "bf16").cuda()
    want, got = torch.empty_like(q), torch.empty_like(q)
    ss.ss_kv_attend(pages, table, q, want)
    ok(ss)
    for wrong in (-1, c.num_pages, 1 << 30):
        bad = c.table.clone()
        bad[1, 2] = wrong
        ss.ss_kv_attend(pages, ss.KVTable(bad, c.lens_dev), q, got)
        assert ss.ss_stream_status() == (ss.SS_ERR_INVALID_ARG, 1)
        keep = [b for b in range(len(lens)) if b != 1]
        assert torch.equal(got[keep], want[keep])


def test_pool_past_32_bit_offsets(ss):
    """Pages whose codes lie past 2^32 bytes, and their scales past 2^29."""
    import torch
    pages_n, heads, page, dim = 70000, 8, 128, 128
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    codes = [torch.zeros(pages_n, heads, page, dim // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    blocks = [torch.zeros(pages_n, heads, page, dim // 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    small = Cache4([200, 333], heads=heads, dim=dim, page=page, scales=False, seed=15)
    ids = [pages_n - 1 - 7 * i for i in range(small.num_pages)]
    for i, at in enumerate(ids):
        for big, one in ((codes[0], small.k), (codes[1], small.v), (blocks[0], small.kb.view(torch.uint8)), (blocks[1], small.vb.view(torch.uint8))):
            big[at] = one[i]
    cache = ss.KVPages(*codes, k_block=blocks[0].view(torch.float8_e4m3fn), v_block=blocks[1].view(torch.float8_e4m3fn))
    moved = torch.tensor([[ids[x] if x >= 0 else -1 for x in row] for row in small.table.tolist()], dtype=torch.int32, device="cuda")
    for repeat in (1, 100):  # one launch, and three
        q = queries(small, 4, "bf16").repeat(repeat, 1, 1).cuda()
        out, want = torch.empty_like(q), torch.empty_like(q)
        ss.ss_kv_attend(cache, ss.KVTable(moved.repeat(repeat, 1), small.lens_dev.repeat(repeat)), q, out)
        ss.ss_kv_attend(small.ss(ss)[0], ss.KVTable(small.table.repeat(repeat, 1), small.lens_dev.repeat(repeat)), q, want)
        ok(ss)
        assert torch.equal(out, want)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [2, 12])
@pytest.mark.parametrize("many", [False, True], ids=["small", "many"])
def test_attend_is_off_by_the_rounding_of_out_alone(ss, kind, dim, group, many):
    """No weight is rounded to fewer bits than a softmax weight keeps.  Queries have
    one element that is not 0, so that a score's product is exact; X = score * log2 e
    is at most 8 (0.25 * 1.25 * 11.25 * 1.5 * log2 e = 7.7).  X is then off by four
    roundings, 2^-24 each of 8, and its difference to a reference that lies up to 32
    away by 2^-20: 2^-19 + 2^-20, so that a weight is off by ln 2 times that and the
    exponential's 2^-22, below 1.2 * 2^-19 of itself, and a quotient of sums of them by
    twice that.  The products' accumulators cut 2^-23 at each of 14 steps (100
    positions, two terms) and the sums of fp32 weights, the scaling and the quotient
    take less than 16 roundings: 2^-19 + 2^-19.2 more.  Together less than 2^-17 of sum w
    |v|, besides half a unit of out's own last place."""
    import torch
    lens = [2, 3, 100, 17, 64] + ([1, 31, 90, 5] * 60 if many else [])
    c = Cache4(lens, dim=dim, page=16, seed=41)
    rng = np.random.default_rng(42)
    heads = c.heads * group
    q = np.zeros((len(lens), heads, dim), np.float32)
    b, j = np.meshgrid(np.arange(len(lens)), np.arange(heads), indexing="ij")
    q[b, j, rng.integers(0, dim, b.shape)] = rng.uniform(0.5, 1.25, b.shape) * rng.choice([-1, 1], b.shape)
    q = torch.from_numpy(q).to(torch_type(kind))
    assert float(q.float().abs().max()) <= 1.25
    out = torch.full(q.shape, math.nan, dtype=q.dtype, device="cuda")
    pages, table = c.ss(ss)
    ss.ss_kv_attend(pages, table, q.cuda(), out, scale=0.25)
    ok(ss)
    got, q = out.double().cpu().numpy(), q.double().numpy()
    bits = 8 if kind == "bf16" else 11
    for b, n in enumerate(lens):
        for j in range(heads):
            h = j // group
            k, v = c.rows(c.k_host, b, h) * c.scale(c.ks, h), c.rows(c.v_host, b, h) * c.scale(c.vs, h)
            x = 0.25 * (k @ q[b, j])
            w = np.exp(x - x.max())
            w /= w.sum()
            want, tol = w @ v, 2.0 ** -17 * (w @ np.abs(v))
            half = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want) + tol, 2.0 ** -14))) - bits)
            off = np.abs(got[b, j] - want)
            assert (off <= half + tol).all(), (b, j, n, float(((off - half) / np.maximum(tol, 1e-300)).max()))


# ---- append ----

def check_append(ss, lens, news, heads, dim, page, src, layout="hnd", strided=False, offsets=True, values=None, scales=True):
    import torch
    c = Cache4(lens, heads=heads, dim=dim, page=page, seed=21, layout=layout, scales=scales)
    want = c.bytes()
    weight = c.weight.cpu().numpy()
    total = sum(news)
    gen = torch.Generator().manual_seed(22)
    if values is None:
        host = torch.randn(total, 3, heads, dim, generator=gen) * torch.exp(torch.randn(total, 3, heads, 1, generator=gen))
    else:
        host = torch.from_numpy(np.resize(values, (total, 3, heads, dim)).astype(np.float32))
    host = host.to(torch_type(src))
    dev = host.cuda()
    k_new, v_new = (dev[:, 1], dev[:, 2]) if strided else (dev[:, 1].contiguous(), dev[:, 2].contiguous())
    starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    pages, table = c.ss(ss)
    ss.ss_kv_append(pages, table, k_new, v_new, offsets=torch.from_numpy(starts).cuda() if offsets else None)
    ok(ss)
    got = c.bytes()
    one = np.ones(heads, np.float32)
    for b, (n, m) in enumerate(zip(lens, news)):
        p = np.arange(n - m, n)
        at = c.table_host[b, p // page], slice(None), p % page
        for i, scale in ((0, c.ks), (1, c.vs)):
            codes, blocks = quantise4(host[starts[b]:starts[b + 1], i + 1].float().numpy(), one if scale is None else scale.numpy())
            nan = np.repeat(blocks == 127, 8, -1)  # the codes of a block of NaN are not looked at
            codes = np.where(nan, got[2 * i][at], codes)
            want[2 * i][at], want[2 * i + 1][at] = codes, blocks
        weight[at] = 0.0
    for x, y in zip(got, want):
        assert np.array_equal(x, y)
    assert np.array_equal(c.weight.cpu().numpy(), weight, equal_nan=True)


@pytest.mark.parametrize("src", ["bf16", "f16"])
@pytest.mark.parametrize("dim,page", [(64, 1), (64, 16), (128, 7), (128, 16), (256, 64)])
def test_append_prompts(ss, src, dim, page):
    check_append(ss, [40, 3, 0, 129], [40, 1, 0, 100], 3, dim, page, src)


@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_append_one_token_each(ss, layout):
    check_append(ss, [1, 17, 200, 64], [1] * 4, 2, 128, 16, "bf16", layout=layout, strided=True, offsets=False)


def test_append_ties_zeros_infinities_and_nan(ss):
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, -6.0]
    blocks = [ties, [t * 2.0 ** -9 for t in ties], [t * 448 for t in ties], [0.0, -0.0] * 8, [1e-6, -1e-6] * 8, [math.inf] + ties[1:],
              [-math.inf] + ties[1:], [math.nan] + ties[1:], ties[:15] + [math.nan], [6e4] * 16, [0.003] * 15 + [0.1], [1.0] * 16]
    values = np.array(blocks).reshape(-1)
    for src in ("bf16", "f16"):
        check_append(ss, [48], [48], 1, 64, 16, src, values=values, scales=False)
        check_append(ss, [48], [48], 1, 64, 16, src, values=values)


def test_append_of_every_16_bit_value(ss):
    """Every bf16 and fp16 value beside a largest one of its block."""
    import torch
    bits = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    for src in ("bf16", "f16"):
        x = torch.from_numpy(bits.view(np.int16)).view(torch_type(src)).float().numpy()
        x = x[np.isfinite(x)]
        x = x[np.argsort(np.abs(x), kind="stable")]  # neighbours of like size share blocks
        n = len(x) // 64
        check_append(ss, [n], [n], 1, 64, 16, src, values=x[:n * 64], scales=False)


def test_append_large_batch(ss):
    rng = np.random.default_rng(23)
    lens = [int(x) for x in rng.integers(1, 300, 70)]
    check_append(ss, lens, [int(rng.integers(0, n + 1)) for n in lens], 4, 128, 32, "bf16", strided=True)


# ---- eviction ----

@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("keep,dst_page,layout", [(64, 16, "hnd"), (37, 8, "nhd"), (300, 64, "hnd"), (1, 1, "hnd")])
def test_evict_moves_codes_and_scales(ss, dim, keep, dst_page, layout):
    import torch
    lens = [0, 1, 64, 65, 500, 2000]
    c = Cache4(lens, dim=dim, page=16, seed=31)
    rng = np.random.default_rng(32)
    w = rng.random(c.w_host.shape).astype(np.float32)
    c.weight.copy_(torch.from_numpy(w))
    kept_lens = [min(n, keep) for n in lens]
    d = Cache4(kept_lens, dim=dim, page=dst_page, seed=33, layout=layout)
    d.ks, d.vs = c.ks, c.vs
    want_bytes = d.bytes()
    pages, table = c.ss(ss)
    new_pages, new_table = d.ss(ss)
    kept = torch.full((len(lens), c.heads, keep), 12345, dtype=torch.int32, device="cuda")
    ss.ss_kv_evict(pages, table, new_pages, new_table, keep, sinks=min(2, keep - 1), recent=min(10, keep - 1) // 2, kept=kept)
    ok(ss)
    want = evict_reference(c, w, keep, min(2, keep - 1), min(10, keep - 1) // 2)
    assert d.lens_dev.tolist() == kept_lens and np.array_equal(kept.cpu().numpy(), want)
    src = c.bytes()
    for b, m in enumerate(kept_lens):
        j = np.arange(m)
        for h in range(c.heads):
            to = d.table_host[b, j // dst_page], h, j % dst_page
            for x, y in zip(want_bytes, src):
                x[to] = c.rows(y, b, h)[want[b, h, :m]]
    for x, y in zip(d.bytes(), want_bytes):
        assert np.array_equal(x, y)
