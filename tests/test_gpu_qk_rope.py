"""Norms and rotation of query and key rows, their gradients, and the form that
writes to a paged cache, against the definitions in 64 bits
(tests/serving_helpers.py).

Tolerances.  With E = 2^-24: a row's sum of squares is off by a factor 1 +- dim E,
its reciprocal root by half of that and 4 E (2 units in the last place), and the
products around it by 4 E, so that u = r w x is off by a factor 1 +- n, n = (dim / 2
+ 8) E.  A sine or cosine is off by d (serving_helpers.angle_error) and by the
angle's own 2^-52 in either computation, so an element of y = (a cos - b sin, b cos +
a sin) is within (|a| + |b|) (n + d' + 4 E), d' = d + 2^-51 |angle|, and half a unit of
its own type.  Backward, h = R^T g is within t = (|g_a| + |g_b|) (d' + 4 E) of the
formula, and dx = r (w h - x r^2 mean(w h x)) within r (w t + m (|w h| + |x| r^2 mean
|w h x|) + |x| r^2 mean(w t |x|)), m = (3 dim + 32) E.  A weight's gradient adds up N rows'
terms r x h, each off by r |x| t and a factor n; no term meets more than 100 + N / 5000
roundings in the sum (rows of a group, 32 groups, 32 shares of CTAs, 5 of a warp)."""

from __future__ import annotations

import math

import numpy as np
import pytest

from kv_helpers import e4m3_reference, torch_type
from serving_helpers import (Cache4, angle_error, frequencies, half_step, quantise4, rope_gradients, rope_reference, turn_reference)

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
TYPES = {"f32": "float32", "bf16": "bfloat16", "f16": "float16"}


@pytest.fixture(scope="module")
def ss():
    import stream_compaction_pass_gb300 as m
    return m


def kind_of(name):
    import torch
    return getattr(torch, TYPES[name])


def ok(ss, stream=None):
    st, where = ss.ss_stream_status(stream=stream)
    assert st == ss.SS_OK, (st, where, ss.ss_last_error_detail())


def make(tokens, heads, dim, kind, seed, layout="packed"):
    """Rows as a projection leaves them (views of one buffer), or in a layout of their own."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    host = [torch.randn(tokens, h, dim, generator=gen) * torch.exp(torch.randn(tokens, h, 1, generator=gen)) for h in heads]
    host = [x.to(kind_of(kind)) for x in host]
    if layout == "packed":
        both = torch.cat([*host, torch.full((tokens, 1, dim), math.nan, dtype=kind_of(kind))], 1).cuda()
        at = np.cumsum([0, *heads])
        return host, [both[:, at[i]:at[i + 1]] for i in range(len(heads))]
    if layout == "heads":  # [head][token][dim]
        return host, [x.transpose(0, 1).contiguous().cuda().transpose(0, 1) for x in host]
    wide = []
    for x in host:  # rows in wider rows
        w = torch.full((tokens, x.shape[1], dim + 16), math.nan, dtype=kind_of(kind), device="cuda")
        w[:, :, :dim] = x.cuda()
        wide.append(w[:, :, :dim])
    return host, wide


def weights(dim, kind, seed):
    import torch
    gen = torch.Generator().manual_seed(seed)
    return [(torch.rand(dim, generator=gen) + 0.5).to(kind_of(kind)) for _ in range(2)]


def wide(x):
    return None if x is None else x.double().numpy()


def sine_error(kind, positions, freq, dim):
    """d' of every element, (tokens, 1, dim), 0 where nothing is turned."""
    angle = np.abs(np.asarray(positions, np.float64)[:, None] * freq)
    return angle_error(kind) + 2.0 ** -51 * angle.max(1)[:, None, None] * np.ones((1, 1, dim))


def partners(x, rot, interleaved):
    """|a| + |b| of every element's pair."""
    x = np.abs(x)
    y = np.array(x)
    if interleaved:
        s = x[..., 0:rot:2] + x[..., 1:rot:2]
        y[..., 0:rot:2] = y[..., 1:rot:2] = s
    else:
        s = x[..., :rot // 2] + x[..., rot // 2:rot]
        y[..., :rot // 2] = y[..., rot // 2:rot] = s
    return y


def check_rows(got, x, w, positions, freq, inter, eps, kind, extra=0.0):
    want = rope_reference(x, w, positions, freq, inter, eps)
    u = np.abs(x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * (1 if w is None else w))
    dim = x.shape[-1]
    tol = half_step(kind) * np.abs(want) + partners(u, 2 * len(freq), inter) * ((dim / 2 + 12) * E + sine_error(kind, positions, freq, dim)) + extra
    if kind == "f16":
        tol = tol + 2.0 ** -25  # subnormal outputs
    off = np.abs(got - want)
    assert (off <= tol).all(), float((off / np.maximum(tol, 1e-300)).max())


def check_forward(ss, tokens, hq, hk, dim, rot, kind, interleaved=False, theta=1e4, positions=None, wkind=None, layout="packed", eps=1e-6, in_place=False, weighted=True,
                  seed=1):
    import torch
    host, (q, k) = make(tokens, (hq, hk), dim, kind, seed, layout)
    w = weights(dim, wkind or kind, seed + 1) if weighted else [None, None]
    positions = np.arange(tokens) % 5000 if positions is None else np.asarray(positions)
    freq = frequencies(rot, theta)
    rope = ss.Rope(torch.from_numpy(freq).cuda(), interleaved=interleaved)
    pos = torch.from_numpy(positions.astype(np.int32)).cuda()
    if in_place:
        yq, yk = q, k
    else:
        yq, yk = (torch.full((tokens, h, dim), math.nan, dtype=kind_of(kind), device="cuda") for h in (hq, hk))
    dw = [None if x is None else x.cuda() for x in w]
    none = lambda x, h: x if h else None  # noqa: E731
    ss.ss_qk_norm_rope(none(q, hq), none(k, hk), dw[0], dw[1], rope, pos, none(yq, hq), none(yk, hk), eps=eps)
    ok(ss)
    for y, x, wi, h in ((yq, host[0], w[0], hq), (yk, host[1], w[1], hk)):
        if h:
            check_rows(y.double().cpu().numpy(), wide(x), wide(wi), positions, freq, interleaved, eps, kind)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,rot", [(16, 16), (64, 64), (64, 32), (72, 16), (80, 32), (96, 96), (128, 128), (136, 128), (192, 64), (248, 240), (256, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_forward_types_and_dims(ss, kind, dim, rot, interleaved):
    check_forward(ss, 37, 6, 2, dim, rot, kind, interleaved)


@pytest.mark.parametrize("tokens", [1, 2, 3, 63, 64, 65, 257, 1000, 5000])
@pytest.mark.parametrize("hq,hk", [(1, 1), (32, 8), (7, 0), (0, 5), (40, 40)])
def test_forward_sizes(ss, tokens, hq, hk):
    check_forward(ss, tokens, hq, hk, 64, 64, "bf16")


@pytest.mark.parametrize("layout", ["packed", "heads", "wide"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_forward_layouts(ss, layout, in_place, kind):
    check_forward(ss, 130, 5, 3, 80, 48, kind, layout=layout, in_place=in_place)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_forward_weight_types(ss, kind):
    for wkind in ("bf16", "f16", "f32"):
        check_forward(ss, 20, 4, 2, 128, 128, kind, wkind=wkind)
    check_forward(ss, 20, 4, 2, 128, 128, kind, weighted=False)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_forward_far_and_negative_positions(ss, kind):
    """Angles of far positions are exact modulo a turn."""
    p = [0, 1, -1, 100000, -100000, 1 << 20, (1 << 24) + 1, 123456789, (1 << 31) - 1, -(1 << 31)]
    check_forward(ss, len(p), 3, 1, 64, 64, kind, positions=p)
    check_forward(ss, len(p), 3, 1, 128, 64, kind, positions=p, theta=1e6, interleaved=True)


@pytest.mark.parametrize("eps", [0.0, 1e-6, 0.1, 100.0])
def test_forward_eps(ss, eps):
    check_forward(ss, 20, 4, 2, 64, 64, "f32", eps=eps)


def test_rows_of_zeros_infinities_and_nan(ss):
    """A row of zeros stays zero; a NaN or an infinity is its own row's alone."""
    import torch
    x = torch.randn(6, 3, 128, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    x[0, 0] = 0
    x[1, 1, 5] = math.nan
    x[2, 2, 7] = math.inf
    q = x.cuda()
    y = torch.empty_like(q)
    rope = ss.Rope(torch.from_numpy(frequencies(128)).cuda())
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    ss.ss_qk_norm_rope(q, None, None, None, rope, pos, y, None)
    ok(ss)
    y = y.float().cpu().numpy()
    assert (y[0, 0] == 0).all() and np.isnan(y[1, 1]).all()
    bad = np.isnan(y).any(-1)
    assert bad[2, 2] and bad.sum() == 2  # inf / inf, and 0 for its row's others or NaN with it


def interleaved_rows(tokens, heads, dim, kind, seed, layout):
    """q, k and v of as many heads, beside each other in every head of one buffer."""
    import torch
    gen = torch.Generator().manual_seed(seed)
    host = torch.randn(tokens, heads, 3, dim, generator=gen).to(kind_of(kind))
    if layout == "token":  # [token][head][q, k, v]
        dev = host.cuda()
    elif layout == "head":  # [head][q, k, v][token]
        dev = host.permute(1, 2, 0, 3).contiguous().cuda().permute(2, 0, 1, 3)
    else:  # the same in rows that are padded
        dev = torch.full((tokens, heads * 3 * dim + 24), math.nan, dtype=host.dtype, device="cuda")
        dev[:, 8:8 + heads * 3 * dim] = host.flatten(1).cuda()
        dev = dev[:, 8:8 + heads * 3 * dim].unflatten(1, (heads, 3, dim))
    return [host[:, :, i] for i in range(3)], [dev[:, :, i] for i in range(3)]


@pytest.mark.parametrize("tokens", [1, 2, 50])
@pytest.mark.parametrize("layout", ["token", "head", "padded"])
@pytest.mark.parametrize("heads", [1, 5])
def test_rows_beside_each_other_in_every_head(ss, tokens, layout, heads):
    """Rows that share no memory, though their ranges do, are taken in place."""
    import torch
    dim, kind = 64, "bf16"
    host, (q, k, v) = interleaved_rows(tokens, heads, dim, kind, 61, layout)
    w = weights(dim, kind, 62)
    freq = frequencies(dim)
    rope = ss.Rope(torch.from_numpy(freq).cuda())
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    ss.ss_qk_norm_rope(q, k, w[0].cuda(), w[1].cuda(), rope, pos, q, k)
    ok(ss)
    at = np.arange(tokens)
    for x, y, wi in ((q, host[0], w[0]), (k, host[1], w[1])):
        check_rows(x.double().cpu().numpy(), wide(y), wide(wi), at, freq, False, 1e-6, kind)
    assert torch.equal(v.cpu(), host[2])
    # the gradients, in place of the gradients of the outputs, which lie as the inputs do
    _, (gq, gk, _) = interleaved_rows(tokens, heads, dim, kind, 63, layout)
    _, (xq, xk, _) = interleaved_rows(tokens, heads, dim, kind, 61, layout)
    apart = [torch.empty(tokens, heads, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dws = [torch.empty(dim, device="cuda") for _ in range(4)]
    call = lambda dq, dk, dw: ss.ss_qk_norm_rope_backward(gq, gk, xq, xk, w[0].cuda(), w[1].cuda(), rope, pos, dq, dk, *dw)  # noqa: E731
    call(*apart, dws[:2])
    call(gq, gk, dws[2:])
    ok(ss)
    assert torch.equal(gq, apart[0]) and torch.equal(gk, apart[1]) and torch.equal(dws[0], dws[2]) and torch.equal(dws[1], dws[3])
    # queries in place, keys and values into a cache
    _, (q, k, v) = interleaved_rows(tokens, heads, dim, kind, 61, layout)
    pool = [torch.zeros(4, heads, 16, dim, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ss.ss_kv_append_rope(ss.KVPages(*pool), torch.arange(tokens, device="cuda"), q, k, v, w[0].cuda(), w[1].cuda(), rope, pos, q)
    ok(ss)
    check_rows(q.double().cpu().numpy(), wide(host[0]), wide(w[0]), at, freq, False, 1e-6, kind)
    rows = [x.transpose(1, 2).reshape(64, heads, dim)[:tokens] for x in pool]
    check_rows(rows[0].double().cpu().numpy(), wide(host[1]), wide(w[1]), at, freq, False, 1e-6, kind)
    assert torch.equal(rows[1].cpu(), host[2]) and torch.equal(k.cpu(), host[1])


# ---- gradients ----

def check_backward(ss, tokens, hq, hk, dim, rot, kind, interleaved=False, layout="packed", eps=1e-6, weighted=True, in_place=None, seed=11, positions=None, stream=None):
    import torch
    host, (q, k) = make(tokens, (hq, hk), dim, kind, seed, layout)
    ghost, (gq, gk) = make(tokens, (hq, hk), dim, kind, seed + 1, layout)
    w = weights(dim, kind, seed + 2) if weighted else [None, None]
    positions = (np.arange(tokens) * 7) % 3000 if positions is None else np.asarray(positions)
    freq = frequencies(rot)
    rope = ss.Rope(torch.from_numpy(freq).cuda(), interleaved=interleaved)
    pos = torch.from_numpy(positions.astype(np.int32)).cuda()
    dq, dk = {"x": (q, k), "g": (gq, gk)}.get(in_place) or [torch.full((tokens, h, dim), math.nan, dtype=kind_of(kind), device="cuda") for h in (hq, hk)]
    dws = [torch.full((dim,), math.nan, device="cuda") for _ in range(2)]
    none = lambda x, h: x if h else None  # noqa: E731
    dev = [None if x is None else x.cuda() for x in w]
    ss.ss_qk_norm_rope_backward(none(gq, hq), none(gk, hk), none(q, hq), none(k, hk), dev[0], dev[1], rope, pos, none(dq, hq), none(dk, hk), dws[0], dws[1], eps=eps, stream=stream)
    ok(ss, stream)
    n, m = (dim / 2 + 8) * E, (3 * dim + 32) * E
    for x, g, wi, dx, dw, h in ((host[0], ghost[0], w[0], dq, dws[0], hq), (host[1], ghost[1], w[1], dk, dws[1], hk)):
        if h == 0:
            assert (dw == 0).all()
            continue
        x, g, wi = wide(x), wide(g), np.ones(dim) if wi is None else wide(wi)
        want, want_w = rope_gradients(x, wi, g, positions, freq, interleaved, eps)
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        hh = np.abs(turn_reference(g, positions, freq, interleaved, -1))
        t = partners(g, rot, interleaved) * (sine_error(kind, positions, freq, dim) + 4 * E)
        mean = lambda z: z.mean(-1, keepdims=True)  # noqa: E731
        tol = half_step(kind) * np.abs(want) + r * (wi * t + m * (wi * hh + np.abs(x) * r * r * mean(wi * hh * np.abs(x))) + np.abs(x) * r * r * mean(wi * t * np.abs(x)))
        if kind == "f16":
            tol = tol + 2.0 ** -25
        off = np.abs(dx.double().cpu().numpy() - want)
        assert (off <= tol).all(), float((off / tol).max())
        terms = r * np.abs(x) * hh
        tol = (terms * n + r * np.abs(x) * t).sum((0, 1)) + (100 + tokens * h / 5000) * E * terms.sum((0, 1))
        off = np.abs(dw.double().cpu().numpy() - want_w)
        assert (off <= tol).all(), float((off / tol).max())
    return dq, dk, dws


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,rot", [(16, 16), (64, 64), (72, 16), (80, 32), (96, 96), (128, 128), (136, 64), (192, 192), (256, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_backward_types_and_dims(ss, kind, dim, rot, interleaved):
    check_backward(ss, 41, 6, 2, dim, rot, kind, interleaved)


@pytest.mark.parametrize("tokens", [1, 2, 65, 1000, 3000])
@pytest.mark.parametrize("hq,hk", [(1, 1), (32, 8), (7, 0), (0, 5)])
def test_backward_sizes(ss, tokens, hq, hk):
    check_backward(ss, tokens, hq, hk, 64, 64, "bf16")


@pytest.mark.parametrize("layout", ["packed", "heads", "wide"])
@pytest.mark.parametrize("in_place", [None, "x", "g"])
def test_backward_layouts(ss, layout, in_place):
    check_backward(ss, 130, 5, 3, 80, 48, "f16", layout=layout, in_place=in_place)
    check_backward(ss, 130, 5, 3, 80, 48, "f32", layout=layout, in_place=in_place, weighted=False)


def test_backward_is_the_same_on_every_run_and_stream(ss):
    import torch
    first = check_backward(ss, 700, 12, 4, 128, 128, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        torch.cuda.synchronize()
        again = check_backward(ss, 700, 12, 4, 128, 128, "bf16", stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        assert all(torch.equal(a, b) for a, b in zip(first[2], again[2]))


def test_backward_agrees_with_differences(ss):
    """The gradient of a weighted sum of the forward's outputs, by differences."""
    import torch
    tokens, heads, dim = 3, 2, 64
    gen = torch.Generator().manual_seed(5)
    x, g = (torch.randn(tokens, heads, dim, generator=gen).cuda() for _ in range(2))
    w = (torch.rand(dim, generator=gen) + 0.5).cuda()
    rope = ss.Rope(torch.from_numpy(frequencies(dim)).cuda())
    pos = torch.tensor([3, 50, 1000], dtype=torch.int32, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ss.ss_qk_norm_rope_backward(g, None, x, None, w, None, rope, pos, dx, None, dw)

    def f(x, w):
        y = torch.empty_like(x)
        ss.ss_qk_norm_rope(x, None, w, None, rope, pos, y, None)
        return float((y.double() * g.double()).sum())

    step = 2.0 ** -7
    # f is off by about 2^-24 of the sum of |y g| on either side; the rest is the third derivative's step^2 share
    y = torch.empty_like(x)
    ss.ss_qk_norm_rope(x, None, w, None, rope, pos, y, None)
    noise = 16 * E * float((y * g).abs().sum()) / step + 40 * step ** 2
    for i in [(0, 0, 0), (1, 1, 33), (2, 0, 63), (1, 0, 31)]:
        e = torch.zeros_like(x)
        e[i] = step
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * step) - float(dx[i])) <= noise
        v = torch.zeros_like(w)
        v[i[2]] = step
        assert abs((f(x, w + v) - f(x, w - v)) / (2 * step) - float(dw[i[2]])) <= noise
    ok(ss)


def test_backward_in_a_graph(ss):
    import torch
    tokens, hq, hk, dim = 300, 6, 2, 64
    _, (q, k) = make(tokens, (hq, hk), dim, "bf16", 21)
    _, (gq, gk) = make(tokens, (hq, hk), dim, "bf16", 22)
    wq, wk = (x.cuda() for x in weights(dim, "bf16", 23))
    rope = ss.Rope(torch.from_numpy(frequencies(dim)).cuda())
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    out = [torch.empty(tokens, h, dim, dtype=torch.bfloat16, device="cuda") for h in (hq, hk)] + [torch.empty(dim, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call = lambda: ss.ss_qk_norm_rope_backward(gq, gk, q, k, wq, wk, rope, pos, *out, stream=side)  # noqa: E731
    call()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        call()
    for _ in range(2):
        q.mul_(1.5)
        gk.neg_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        replayed = [x.clone() for x in out]
        call()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, out))
    ok(ss, side)


def test_a_first_call_in_a_capture_is_refused(ss):
    """The gradient's scratch is made by a call before the capture."""
    import torch
    _, (q,) = make(40, (2,), 64, "bf16", 31)
    rope = ss.Rope(torch.from_numpy(frequencies(64)).cuda())
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    y, dw = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty(64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        with pytest.raises(ss.StreamScanError) as e:
            ss.ss_qk_norm_rope_backward(q, None, q, None, None, None, rope, pos, y, None, dw, stream=side)
        assert e.value.status == ss.SS_ERR_NO_MEMORY
        y.zero_()


def test_forward_first_in_a_capture(ss):
    """The call needs nothing that a call before the capture would have to make."""
    import torch
    tokens, hq, hk, dim = 90, 6, 2, 64
    host, (q, k) = make(tokens, (hq, hk), dim, "bf16", 33)
    wq, wk = weights(dim, "bf16", 34)
    freq = frequencies(dim)
    rope = ss.Rope(torch.from_numpy(freq).cuda())
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    yq, yk = (torch.full((tokens, h, dim), math.nan, dtype=torch.bfloat16, device="cuda") for h in (hq, hk))
    dev = wq.cuda(), wk.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ss.ss_qk_norm_rope(q, k, *dev, rope, pos, yq, yk, stream=side)
    for shift in (0, 1000):
        pos.copy_(torch.arange(shift, shift + tokens))
        yq.fill_(math.nan)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        at = np.arange(shift, shift + tokens)
        check_rows(yq.double().cpu().numpy(), wide(host[0]), wide(wq), at, freq, False, 1e-6, "bf16")
        check_rows(yk.double().cpu().numpy(), wide(host[1]), wide(wk), at, freq, False, 1e-6, "bf16")


# ---- into the cache ----

def check_append(ss, tokens, hq, hk, dim, rot, kind, cache, page=16, layout="hnd", interleaved=False, skip=(), scales=True, seed=41):
    import torch
    host, (q, k, v) = make(tokens, (hq, hk, hk), dim, kind, seed)
    w = weights(dim, kind, seed + 1)
    rng = np.random.default_rng(seed + 2)
    pages_n = -(-tokens // page) + 3
    slots = rng.permutation(pages_n * page)[:tokens]
    slots[list(skip)] = -1
    positions = rng.integers(0, 40000, tokens)
    freq = frequencies(rot)
    rope = ss.Rope(torch.from_numpy(freq).cuda(), interleaved=interleaved)
    shape = (pages_n, hk, page, dim)
    ks, vs = (torch.rand(hk, generator=torch.Generator().manual_seed(seed + 3 + i)) + 0.5 for i in range(2))
    if cache == "e4m3":
        ks, vs = ks / 16, vs / 16
    has = scales and cache in ("e4m3", "e2m1")
    d_ks, d_vs = (ks.cuda(), vs.cuda()) if has else (None, None)

    def pool(width, fill):
        t = torch.full((pages_n, page, hk, width) if layout == "nhd" else (pages_n, hk, page, width), fill, dtype=torch.uint8, device="cuda")
        return t.transpose(1, 2) if layout == "nhd" else t

    weight = torch.full(shape[:3], 2.5, device="cuda")
    blocks = [None, None]
    if cache == "e2m1":
        kc, vc = pool(dim // 2, 0x5a), pool(dim // 2, 0x5a)
        blocks = [torch.full((*shape[:3], dim // 16), 0x33, dtype=torch.uint8, device="cuda") for _ in range(2)]
        pages = ss.KVPages(kc, vc, weight=weight, k_scale=d_ks, v_scale=d_vs, k_block=blocks[0].view(torch.float8_e4m3fn), v_block=blocks[1].view(torch.float8_e4m3fn))
    else:
        size = 1 if cache == "e4m3" else 2
        kc, vc = pool(dim * size, 0x3a), pool(dim * size, 0x3a)
        pages = ss.KVPages(kc.view(torch_type(cache)), vc.view(torch_type(cache)), weight=weight, k_scale=d_ks, v_scale=d_vs)
    yq = torch.full((tokens, hq, dim), math.nan, dtype=kind_of(kind), device="cuda") if hq else None
    ss.ss_kv_append_rope(pages, torch.from_numpy(slots.astype(np.int64)).cuda(), q if hq else None, k, v, w[0].cuda(), w[1].cuda(), rope,
                         torch.from_numpy(positions.astype(np.int32)).cuda(), yq)
    ok(ss)
    if hq:
        check_rows(yq.double().cpu().numpy(), wide(host[0]), wide(w[0]), positions, freq, interleaved, 1e-6, kind)
    keep = slots >= 0
    at, slot = slots[keep] // page, slots[keep] % page
    want_weight = np.full(shape[:3], 2.5, np.float32)
    want_weight[at, :, slot] = 0
    assert np.array_equal(weight.cpu().numpy(), want_weight)
    kc, vc = kc.cpu().numpy(), vc.cpu().numpy()
    untouched = want_weight > 0
    fill = 0x5a if cache == "e2m1" else 0x3a
    assert (kc[untouched] == fill).all() and (vc[untouched] == fill).all()
    one = np.ones(hk, np.float32)
    sk, sv = (ks.numpy(), vs.numpy()) if has else (one, one)
    y = rope_reference(wide(host[1]), wide(w[1]), positions, freq, interleaved, 1e-6)[keep]
    u = np.abs(wide(host[1])) / np.sqrt((wide(host[1]) ** 2).mean(-1, keepdims=True) + 1e-6) * wide(w[1])
    error = (partners(u, rot, interleaved) * ((dim / 2 + 16) * E + sine_error(kind, positions, freq, dim)))[keep]
    v_host = host[2].float().numpy()[keep]
    if cache == "e2m1":
        kb, vb = (b.cpu().numpy() for b in blocks)
        assert (kb[untouched] == 0x33).all() and (vb[untouched] == 0x33).all()
        codes, scale = quantise4(v_host, sv)
        assert np.array_equal(vc[at, :, slot], codes) and np.array_equal(vb[at, :, slot], scale)
        # a value within `error` of k's: its codes and scales, or their neighbours where a tie lies within that
        from serving_helpers import e2m1_value, e4m3_value
        got, gs = kc[at, :, slot], kb[at, :, slot]
        value = np.stack([e2m1_value(got & 15), e2m1_value(got >> 4)], -1).reshape(y.shape)
        b = e4m3_value(gs)
        z, dz = np.abs(y) / sk[:, None], error / sk[:, None] + 2 * E * np.abs(y) / sk[:, None]
        most, at_most = z.reshape(*b.shape, 16).max(-1), dz.reshape(*b.shape, 16).max(-1)
        low, high = e4m3_reference((most - at_most) / 6 * (1 - 2 * E)), e4m3_reference((most + at_most) / 6 * (1 + 2 * E))
        assert ((low <= b) & (b <= high)).all()
        wide_b = np.repeat(b, 16, -1)
        some = wide_b > 0
        assert (value[~some] == 0).all()
        zb, db = np.where(some, z / np.where(some, wide_b, 1), 0), np.where(some, dz / np.where(some, wide_b, 1), 0) + 4 * E
        gap = np.select([zb <= 2, zb <= 4], [0.25, 0.5], 1.0)
        near = np.abs(np.abs(value) - np.minimum(zb, 6)) <= gap + db * (zb <= 6 + db)
        assert (near | ~some).all()
        assert (np.sign(value) * np.sign(y) >= 0)[np.abs(y) > error].all()
    elif cache == "e4m3":
        from serving_helpers import e4m3_value
        assert np.array_equal(e4m3_value(vc[at, :, slot]), e4m3_reference((v_host / sv[:, None].astype(np.float32)).astype(np.float32)))
        got = e4m3_value(kc[at, :, slot])
        z, dz = y / sk[:, None], error / sk[:, None] + 4 * E * np.abs(y) / sk[:, None]
        assert ((e4m3_reference(z - dz) <= got) & (got <= e4m3_reference(z + dz))).all()
    else:
        import torch as th
        read = lambda c: th.from_numpy(np.ascontiguousarray(c[at, :, slot])).view(torch_type(cache)).double().numpy()  # noqa: E731
        assert np.array_equal(read(vc), v_host.astype(np.float64))
        assert (np.abs(read(kc) - y) <= half_step(kind) * np.abs(y) + error + 2.0 ** -25).all()


@pytest.mark.parametrize("kind,cache", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3"), ("bf16", "e2m1"), ("f16", "e2m1")])
@pytest.mark.parametrize("dim,rot", [(64, 64), (128, 128), (128, 32), (256, 192)])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
def test_append_types_and_dims(ss, kind, cache, dim, rot, layout):
    check_append(ss, 70, 4, 2, dim, rot, kind, cache, layout=layout, skip=(0, 33, 69))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim,rot", [(80, 48), (16, 16), (96, 32)])
def test_append_odd_dims(ss, cache, dim, rot):
    check_append(ss, 40, 3, 3, dim, rot, "bf16", cache, page=5, interleaved=True)


@pytest.mark.parametrize("tokens", [1, 64, 1000, 3000])
@pytest.mark.parametrize("cache", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("hq,hk", [(32, 8), (0, 1)])
def test_append_sizes(ss, tokens, cache, hq, hk):
    check_append(ss, tokens, hq, hk, 128, 128, "bf16", cache, scales=hq > 0)


def test_append_slots_behind_the_pool_are_reported(ss):
    import torch
    _, (q, k, v) = make(4, (2, 1, 1), 64, "bf16", 51)
    pool = [torch.zeros(3, 1, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rope = ss.Rope(torch.from_numpy(frequencies(64)).cuda())
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    for wrong in (48, 1 << 40):
        slots = torch.tensor([0, 5, wrong, 47], device="cuda")
        for x in pool:
            x.zero_()
        ss.ss_kv_append_rope(ss.KVPages(*pool), slots, q, k, v, None, None, rope, pos, torch.empty(4, 2, 64, dtype=torch.bfloat16, device="cuda"))
        assert ss.ss_stream_status() == (ss.SS_ERR_INVALID_ARG, 2)
        assert torch.equal((pool[1] != 0).any(-1).flatten().nonzero().flatten().cpu(), torch.tensor([0, 5, 47]))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("cache", ["e4m3", "e2m1"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_append_of_keys_turned_by_nearly_a_quarter(ss, kind, cache, dim):
    """Narrow caches take sines and cosines of fp32, of angles that are good to more.
    The norm is 1 and the partner 0, so that a key is w cos: off by two units of the
    cosine (2^-22 of it), the angle's remainder in fp32 (2^-24 times 2^-25 / 2^-19 of it,
    and its derivative's 2^-22), the product, the scale's division or inverse and
    product: below 2^-20 of it.  An angle in fp32, 2^-25, is 2^-6 of a cosine of 2^-19."""
    import torch
    from serving_helpers import QuarterTurns, codes_between, e4m3_between, e4m3_value
    tokens, heads, page = 203, 3, 16
    rows = QuarterTurns(tokens, heads, dim, 71)
    k = torch.from_numpy(rows.x).to(kind_of(kind)).cuda()
    w = torch.from_numpy(rows.weight).to(kind_of(kind)).cuda()
    rope = ss.Rope(torch.from_numpy(rows.freq).cuda())
    pos = torch.from_numpy(rows.positions.astype(np.int32)).cuda()
    pages_n = -(-tokens // page)
    scale = torch.full((heads,), 2.0 ** -16, device="cuda")
    size = dim if cache == "e4m3" else dim // 2
    kc, vc = (torch.zeros(pages_n, heads, page, size, dtype=torch.uint8, device="cuda") for _ in range(2))
    if cache == "e4m3":
        pages = ss.KVPages(kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn), k_scale=scale, v_scale=scale)
    else:
        kb, vb = (torch.zeros(pages_n, heads, page, dim // 16, dtype=torch.uint8, device="cuda") for _ in range(2))
        pages = ss.KVPages(kc, vc, k_scale=scale, v_scale=scale, k_block=kb.view(torch.float8_e4m3fn), v_block=vb.view(torch.float8_e4m3fn))
    ss.ss_kv_append_rope(pages, torch.arange(tokens, device="cuda"), None, k, k, None, w, rope, pos, None, eps=0.0)
    ok(ss)
    y = rope_reference(rows.x, rows.weight, rows.positions, rows.freq, False, 0.0) * 2.0 ** 16
    read = lambda x: x.cpu().numpy().swapaxes(1, 2).reshape(pages_n * page, heads, -1)[:tokens]  # noqa: E731
    if cache == "e4m3":
        assert e4m3_between(e4m3_value(read(kc)), y, 2.0 ** -20).all()
    else:
        assert codes_between(read(kc), read(kb), y, 2.0 ** -20).all()


# ---- more rows than a CTA's tables hold ----

# A CTA of 128 threads has 128 / L groups, L = 16 lanes a row of 256, 8 of 128, 4 of 64, and
# every group a row a step.  The tables are filled again after min(32, heads) steps
# (backward min(16, heads)).  No SM holds more than 16 such CTAs, and no call launches more
# than four waves of them, backward one of four an SM.

def least_steps(rows, dim, ctas_per_sm):
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    lanes = {64: 4, 128: 8, 256: 16}[dim]
    return rows / (sms * ctas_per_sm * (128 // lanes))


def large_rows(tokens, heads, dim, kind, seed):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(tokens, h, dim, generator=gen, device="cuda").to(kind_of(kind)) for h in heads]


@pytest.mark.parametrize("tokens,hq,hk,dim,kind", [(170_000, 33, 5, 128, "bf16"), (230_000, 3, 1, 128, "f16"), (120_000, 3, 2, 256, "f32")])
def test_forward_of_more_rows_than_the_tables_hold(ss, tokens, hq, hk, dim, kind):
    """The rows of one large call are those of calls of 999 tokens, which fill the tables
    once, bit by bit; some are compared with the formula."""
    import torch
    assert least_steps(tokens * (hq + hk), dim, 64) > min(32, hq)
    q, k = large_rows(tokens, (hq, hk), dim, kind, 81)
    w = [x.cuda() for x in weights(dim, kind, 82)]
    freq = frequencies(dim)
    rope = ss.Rope(torch.from_numpy(freq).cuda())
    pos = (torch.arange(tokens, device="cuda") * 7919 % 100_003).to(torch.int32)
    yq, yk = torch.full_like(q, math.nan), torch.full_like(k, math.nan)
    ss.ss_qk_norm_rope(q, k, *w, rope, pos, yq, yk)
    pq, pk = torch.full_like(q, math.nan), torch.full_like(k, math.nan)
    for t in range(0, tokens, 999):
        s = slice(t, t + 999)
        ss.ss_qk_norm_rope(q[s], k[s], *w, rope, pos[s], pq[s], pk[s])
    ok(ss)
    assert torch.equal(yq, pq) and torch.equal(yk, pk)
    some = torch.arange(0, tokens, 997, device="cuda")
    at = pos[some].cpu().numpy()
    for x, y, wi in ((q, yq, w[0]), (k, yk, w[1])):
        check_rows(y[some].double().cpu().numpy(), x[some].double().cpu().numpy(), wi.double().cpu().numpy(), at, freq, False, 1e-6, kind)


@pytest.mark.parametrize("tokens,hq,hk,dim,kind", [(20_000, 32, 8, 64, "bf16"), (30_000, 33, 5, 128, "f16"), (60_000, 3, 1, 128, "bf16"), (30_000, 3, 2, 256, "f32")])
def test_backward_of_more_rows_than_the_tables_hold(ss, tokens, hq, hk, dim, kind):
    """The gradients of the rows are those of calls of 99 tokens, bit by bit.  Those of the
    weights are the formula's sums, whose terms meet the rows of a group (below N / 5000 of
    N rows here, 32 groups or fewer), 32 groups, 32 shares of CTAs and 5 of a warp."""
    import torch
    assert least_steps(tokens * (hq + hk), dim, 4) > min(16, hq)
    q, k = large_rows(tokens, (hq, hk), dim, kind, 83)
    gq, gk = large_rows(tokens, (hq, hk), dim, kind, 84)
    w = [x.cuda() for x in weights(dim, kind, 85)]
    freq = frequencies(dim)
    rope = ss.Rope(torch.from_numpy(freq).cuda())
    pos = (torch.arange(tokens, device="cuda") * 7919 % 100_003).to(torch.int32)
    dq, dk = torch.full_like(q, math.nan), torch.full_like(k, math.nan)
    dw = [torch.full((dim,), math.nan, device="cuda") for _ in range(2)]
    ss.ss_qk_norm_rope_backward(gq, gk, q, k, *w, rope, pos, dq, dk, *dw)
    pq, pk = torch.full_like(q, math.nan), torch.full_like(k, math.nan)
    for t in range(0, tokens, 99):
        s = slice(t, t + 99)
        ss.ss_qk_norm_rope_backward(gq[s], gk[s], q[s], k[s], *w, rope, pos[s], pq[s], pk[s])
    ok(ss)
    assert torch.equal(dq, pq) and torch.equal(dk, pk)
    half, n = dim // 2, (dim / 2 + 8) * E
    for x, g, got, h in ((q, gq, dw[0], hq), (k, gk, dw[1], hk)):
        want, terms, off = (torch.zeros(dim, dtype=torch.float64, device="cuda") for _ in range(3))
        for t in range(0, tokens, 4096):
            s = slice(t, t + 4096)
            u = x[s].double()
            u = u / (u.square().mean(-1, keepdim=True) + 1e-6).sqrt()
            angle = (pos[s].double()[:, None] * torch.from_numpy(freq).cuda())[:, None]
            z = torch.complex(g[s][..., :half].double(), g[s][..., half:].double()) * torch.exp(-1j * angle)
            hh = torch.cat([z.real, z.imag], -1)
            want += (u * hh).sum((0, 1))
            terms += (u * hh).abs().sum((0, 1))
            pair = g[s][..., :half].double().abs() + g[s][..., half:].double().abs()
            error = (angle_error(kind) + 2.0 ** -51 * angle.abs().amax(-1, keepdim=True) + 4 * E) * torch.cat([pair, pair], -1)
            off += (u.abs() * error).sum((0, 1))
        tol = off + n * terms + (100 + tokens * h / 5000) * E * terms
        assert bool(((got.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("tokens,hq,hk", [(75_000, 3, 1), (53_000, 1, 3)])
def test_append_of_more_rows_than_the_tables_hold(ss, cache, tokens, hq, hk):
    """The queries and the cache of one large call, some of whose tokens go nowhere, are
    those of calls of 999 tokens, bit by bit."""
    import torch
    dim, page = 128, 16
    assert least_steps(tokens * (hq + 2 * hk), dim, 48) > min(32, max(hq, hk))
    q, k, v = large_rows(tokens, (hq, hk, hk), dim, "bf16", 86)
    w = [x.cuda() for x in weights(dim, "bf16", 87)]
    rope = ss.Rope(torch.from_numpy(frequencies(dim)).cuda())
    pos = (torch.arange(tokens, device="cuda") * 7919 % 100_003).to(torch.int32)
    pages_n = -(-tokens // page) + 3
    gen = torch.Generator(device="cuda").manual_seed(88)
    slots = torch.randperm(pages_n * page, generator=gen, device="cuda")[:tokens]
    slots[::7] = -1
    scale = torch.full((hk,), 1 / 32 if cache == "e4m3" else 1.0, device="cuda")

    def run(step):
        shape = (pages_n, hk, page)
        size = {"bf16": 2 * dim, "e4m3": dim, "e2m1": dim // 2}[cache]
        held = [torch.full((*shape, size), 0x3a, dtype=torch.uint8, device="cuda") for _ in range(2)] + [torch.full(shape, 2.5, device="cuda")]
        if cache == "e2m1":
            held += [torch.full((*shape, dim // 16), 0x33, dtype=torch.uint8, device="cuda") for _ in range(2)]
            pages = ss.KVPages(*held[:2], weight=held[2], k_scale=scale, v_scale=scale, k_block=held[3].view(torch.float8_e4m3fn), v_block=held[4].view(torch.float8_e4m3fn))
        else:
            scales = dict(k_scale=scale, v_scale=scale) if cache == "e4m3" else {}
            pages = ss.KVPages(*(x.view(torch_type(cache)) for x in held[:2]), weight=held[2], **scales)
        y = torch.full_like(q, math.nan)
        for t in range(0, tokens, step):
            s = slice(t, t + step)
            ss.ss_kv_append_rope(pages, slots[s], q[s], k[s], v[s], *w, rope, pos[s], y[s])
        ok(ss)
        return [y, *held]

    for large, small in zip(run(tokens), run(999)):
        assert torch.equal(large, small)
