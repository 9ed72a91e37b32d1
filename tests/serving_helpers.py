"""A paged cache in 4 bits, and the operators around a decode step computed from
their definitions with numpy, in 64 bits or whole numbers; shares nothing with
the CUDA path."""

from __future__ import annotations

import math

import numpy as np

from kv_helpers import Cache, e4m3_reference

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_value(code):
    """e4m3 bytes as 64-bit numbers."""
    code = np.asarray(code, np.int64)
    e, m = code >> 3 & 15, code & 7
    x = np.where(e > 0, 2.0 ** (e - 7.0) * (1 + m / 8), m * 2.0 ** -9)
    x = np.where(code & 127 == 127, np.nan, x)
    return np.where(code & 128, -x, x)


def e2m1_value(code):
    code = np.asarray(code, np.int64)
    return np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]


def open4(codes, blocks):
    """(..., dim / 2) packed codes and (..., dim / 16) e4m3 bytes as values."""
    x = np.stack([e2m1_value(codes & 15), e2m1_value(codes >> 4)], -1).reshape(*codes.shape[:-1], -1)
    return x * np.repeat(e4m3_value(blocks), 16, -1)


def quantise4(x, scale):
    """Rows (..., heads, dim) as (codes, block scales): the definition, whose steps
    are rounded to fp32."""
    inverse = np.float32(1) / np.asarray(scale, np.float32)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        y = (np.asarray(x, np.float32) * inverse[..., None]).astype(np.float32)
        blocks = y.reshape(*y.shape[:-1], y.shape[-1] // 16, 16)
        most = np.abs(blocks).max(-1)
        nan = np.isnan(blocks).any(-1)
        b = e4m3_reference(np.where(nan, 0, np.minimum((most / np.float32(6)).astype(np.float32), np.float32(448))))
        some = (b > 0) & ~nan
        z = np.where(some[..., None], (blocks / np.where(some, b, 1)[..., None].astype(np.float32)).astype(np.float32), 0)
    a = np.minimum(np.abs(np.nan_to_num(z, posinf=6, neginf=-6)), 6.0)
    hi = np.clip(np.searchsorted(E2M1, a), 1, 7)
    below, above = a - E2M1[hi - 1], E2M1[hi] - a
    code = np.where(below < above, hi - 1, np.where(above < below, hi, np.where((hi - 1) % 2 == 0, hi - 1, hi)))
    code = code | np.where(np.signbit(blocks), 8, 0)
    code = code.reshape(y.shape)
    grid = np.array([e4m3_value(i) for i in range(127)])
    scales = np.where(nan, 127, np.searchsorted(grid, b))
    return (code[..., 0::2] | code[..., 1::2] << 4).astype(np.uint8), scales.astype(np.uint8)


class Cache4(Cache):
    """Random codes and scales with shuffled pages.  The blocks' scales of every
    slot that no sequence holds are NaN, so that a read outside shows."""

    def __init__(self, lens, heads=2, dim=64, page=16, seed=0, layout="hnd", spare=3, scales=True, table_extra=2):
        import torch
        super().__init__(lens, heads=heads, dim=16, page=page, kind="bf16", seed=seed, spare=spare, table_extra=table_extra)
        self.dim, self.kind = dim, "e2m1"
        rng = np.random.default_rng(seed + 1000)
        held = ~np.isnan(self.w_host)
        shape = held.shape

        def pool():
            codes = rng.integers(0, 256, (*shape, dim // 2)).astype(np.uint8)
            blocks = rng.integers(0x28, 0x40, (*shape, dim // 16)).astype(np.uint8)  # 0.25 to 1.9
            blocks[rng.random(blocks.shape) < 0.02] = 0  # blocks of zeros
            blocks[~held] = 127
            return codes, blocks

        (kc, kb), (vc, vb) = pool(), pool()
        self.codes, self.blocks = [kc, vc], [kb, vb]
        self.k_host, self.v_host = open4(kc, kb), open4(vc, vb)
        gen = torch.Generator().manual_seed(seed + 1)
        self.ks = self.vs = None
        if scales:
            self.ks, self.vs = (torch.rand(heads, generator=gen) + 0.5 for _ in range(2))

        def put(x):
            x = torch.from_numpy(x)
            return x.transpose(1, 2).contiguous().cuda().transpose(1, 2) if layout == "nhd" else x.cuda()

        self.k, self.v = put(kc), put(vc)
        self.kb, self.vb = (torch.from_numpy(x).cuda().view(torch.float8_e4m3fn) for x in (kb, vb))

    def ss(self, m):
        c = [None if s is None else s.cuda() for s in (self.ks, self.vs)]
        pages = m.KVPages(self.k, self.v, weight=self.weight, k_scale=c[0], v_scale=c[1], k_block=self.kb, v_block=self.vb)
        return pages, m.KVTable(self.table, self.lens_dev)

    def bytes(self):
        """Codes and scales of k, then of v, as they are on the GPU now."""
        import torch
        return [x.cpu().numpy() for x in (self.k, self.kb.view(torch.uint8), self.v, self.vb.view(torch.uint8))]


def rope_reference(x, w, positions, freq, interleaved, eps):
    """Rows (tokens, heads, dim) normed, weighted and turned, in 64 bits."""
    x = np.asarray(x, np.float64)
    u = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if w is not None:
        u = u * np.asarray(w, np.float64)
    return turn_reference(u, positions, freq, interleaved, 1)


def turn_reference(x, positions, freq, interleaved, sign):
    half = len(freq)
    angle = (np.asarray(positions, np.float64)[:, None] * np.asarray(freq, np.float64))[:, None]
    z = x[..., 0:2 * half:2] + 1j * x[..., 1:2 * half:2] if interleaved else x[..., :half] + 1j * x[..., half:2 * half]
    z = z * np.exp(sign * 1j * angle)
    y = np.array(x)
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = z.real, z.imag
    else:
        y[..., :half], y[..., half:2 * half] = z.real, z.imag
    return y


def rope_gradients(x, w, g, positions, freq, interleaved, eps):
    """dx and dw, in 64 bits."""
    x, g = np.asarray(x, np.float64), np.asarray(g, np.float64)
    w = np.ones(x.shape[-1]) if w is None else np.asarray(w, np.float64)
    n = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    h = turn_reference(g, positions, freq, interleaved, -1)
    dx = w * h / n - x * (w * h * x).sum(-1, keepdims=True) / (x.shape[-1] * n ** 3)
    return dx, (h * x / n).sum((0, 1))


def assign_reference(table, lens, page, counts, restart, ring, head, free, room, limit):
    """One sequence after the other.  table: its rows as lists.  Returns new tables
    (rows' pages in use), lengths, ring, state, offsets, positions, slots, and who is at fault."""
    pages = lambda n: -(-n // page)  # noqa: E731
    ring, head = list(ring), head % len(ring)
    out, new, offsets, positions, slots, gone, at, short, bad = [], [], [0], [], [], [], 0, False, []
    for b, n in enumerate(lens):
        c = 1 if counts is None else counts[b]
        rows = list(table[b][:pages(n)])
        if restart is not None and restart[b]:
            gone += rows
            n, rows = 0, []
        fits = c >= 0 and (c == 0 or n + c <= limit)
        c = max(c, 0)
        need = pages(n + c) - pages(n) if fits else 0
        if not fits:
            bad.append(b)
        short = short or at + need > free
        ok = fits and (need == 0 or not short)
        if ok:
            rows += [ring[(head + at + i) % len(ring)] for i in range(need)]
            at += need
        out.append(rows)
        new.append(n + c if ok else n)
        offsets.append(offsets[-1] + c)
        positions += range(n, n + c)
        slots += [rows[p // page] * page + p % page for p in range(n, n + c)] if ok else [-1] * c
    for i, p in enumerate(gone):
        ring[(head + free + i) % len(ring)] = p
    state = [(head + at) % len(ring), free - at + len(gone)]
    positions, slots = positions[:room], slots[:room]
    return out, new, ring, state, offsets, positions + [0] * (room - len(positions)), slots + [-1] * (room - len(slots)), bad


def half_step(kind):
    """Half a unit in the last place, relative to the value."""
    return {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}[kind]


def frequencies(rot, theta=1e4):
    return theta ** (-np.arange(0, rot, 2) / rot)


def largest(x):
    return float(np.max(np.abs(x))) if np.size(x) else 0.0


def angle_error(kind):
    """How far the sine or cosine of an angle may be off: that of 2^-24 of half a
    turn and two units of fp32, or the 2^-20 of the approximations that 16-bit rows take."""
    return math.pi * 2.0 ** -24 + 2.0 ** -22 if kind == "f32" else 2.0 ** -20


class QuarterTurns:
    """Rows of which the first half becomes small: pairs (+-w, 0) turned by nearly a
    quarter, whose cosines, 2^-8 to 2^-19, take angles that are good to far more than
    fp32 holds of them.  Elements are +-1, so that the norm of 2^k of them is 1 in any
    precision, and the weights of the other halves 0."""

    POSITIONS = np.array([1, -1, 3, -3, 5, -7, 9, 1])

    def __init__(self, tokens, heads, dim, seed):
        rng = np.random.default_rng(seed)
        half = dim // 2
        self.x = rng.choice([-1.0, 1.0], (tokens, heads, dim))
        self.weight = np.concatenate([1 + rng.integers(0, 128, half) / 128, np.zeros(half)])
        blocks = np.linspace(-8, -19, half // 16)  # of about one size each, for a block's scale
        self.freq = np.pi / 2 - 2.0 ** np.repeat(blocks, 16) * (1 + np.tile(np.arange(16), half // 16) / 32)
        self.positions = self.POSITIONS[np.arange(tokens) % len(self.POSITIONS)]

    def rows(self, angle=lambda x: x):
        """Rows of k, their angles passed through `angle`."""
        a = angle(self.positions[:, None] * self.freq)[:, None]
        u = (self.x * self.weight)[..., :len(self.freq)]
        return np.concatenate([u * np.cos(a), u * np.sin(a)], -1)


def e4m3_between(got, y, error):
    """Whether every e4m3 value is that of a number within a factor 1 +- error of y."""
    return (e4m3_reference(y - error * np.abs(y)) <= got) & (got <= e4m3_reference(y + error * np.abs(y)))


def codes_between(codes, blocks, y, error):
    """The same of e2m1 codes with their blocks' scales; NaN-free rows of numbers."""
    most = np.abs(y).reshape(*blocks.shape, 16).max(-1)
    b = e4m3_value(blocks)
    cut = lambda x: e4m3_reference(np.minimum(x / 6, 448.0))  # noqa: E731
    good = (cut(most * (1 - error)) <= b) & (b <= cut(most * (1 + error)))
    got = np.abs(np.stack([e2m1_value(codes & 15), e2m1_value(codes >> 4)], -1).reshape(y.shape))
    z = np.abs(y) / np.repeat(b, 16, -1)

    def nearest(a, up):  # of the codes beside it the nearer one; at a tie the higher or lower one
        middle = (E2M1[1:] + E2M1[:-1]) / 2
        return E2M1[np.searchsorted(middle, a, side="right" if up else "left")]

    return (nearest(z * (1 - error), False) <= got) & (got <= nearest(z * (1 + error), True)) & np.repeat(good, 16, -1)
