"""The 8-bit key / value cache on the GPU against its oracle: codes, scales and what is read back bit for bit.

Tolerances of the step follow from the arithmetic: one rounding of the result (half a step of its type), one of the
probabilities before their product (two bfloat16 pieces, 2^-16; float32 three, 2^-22 with the products left out), and
float32 for everything else.  With S = max scale sum |q k|, n positions and D columns a
probability is off by at most
    rel = (D + 8) 2^-24 S + 2^-22 S + 2^-21 + n 2^-24
of itself, in its numerator and in the sum."""

import numpy as np
import pytest
import torch

import selective_state_space_mamba3_amd as m3
from oracle import kv8 as K
from test_gpu_attn import DEV, TYPES, check, f64, half_step, rand, tiny

pytestmark = pytest.mark.gpu

PIECES = {torch.bfloat16: 2.0 ** -16, torch.float16: 2.0 ** -16, torch.float32: 2.0 ** -22}


class Cache:
    """Keys and values on the host and on the GPU; rows' first `lengths` positions written, the rest NaN codes."""

    def __init__(self, G, D, block, lengths, capacity, page, layout="rows", seed=0, spare=2):
        n = len(lengths)
        self.G, self.D, self.block, self.page = G, D, block, page or capacity
        self.per = -(-capacity // self.page)
        pages = n * self.per + spare
        g = np.random.default_rng(seed)
        order = g.permutation(pages)[:n * self.per].reshape(n, self.per) if page else np.arange(n)[:, None]
        self.order, self.table = order, torch.from_numpy(order.astype(np.int32)).to(DEV) if page else None
        self.host = []
        for _ in range(2):
            codes = np.full((pages, self.page, G, D), 127, np.uint8)
            scales = g.integers(0, 255, (pages, G, -(-self.page // block))).astype(np.uint8)
            for b, length in enumerate(lengths):
                if 0 < length <= capacity:
                    K.write(codes, scales, block, g.standard_normal((length, G, D)), 0, list(order[b]))
            self.host.append((codes, scales))
        self.dev = [(self.place(c, layout), torch.from_numpy(s).to(DEV).view(torch.float8_e8m0fnu)) for c, s in self.host]

    def place(self, codes, layout):
        t = torch.from_numpy(codes).to(DEV)
        if layout == "heads":
            t = t.transpose(1, 2).contiguous().transpose(1, 2)
        elif layout == "odd":  # strides and a start that no word divides
            pages, size, g, d = codes.shape
            whole = torch.full((pages, size, g, d + 3), 55, dtype=torch.uint8, device=DEV)
            whole[..., 3:] = t
            t = whole[..., 3:]
        return t.view(torch.float8_e4m3fn) if layout != "odd" else whole.view(torch.float8_e4m3fn)[..., 3:]

    def args(self):
        (kc, ks), (vc, vs) = self.dev
        return kc, ks, vc, vs

    def pages(self, b, bad=()):
        return [None if p in bad else int(x) for p, x in enumerate(self.order[b])]

    def same(self, what):
        """The GPU's caches are the host's, untouched places among them."""
        for (c, s), (dc, ds), name in zip(self.host, self.dev, "kv"):
            got = dc.view(torch.uint8).cpu().numpy()
            wrong = (got != c) & ~((got % 128 == 127) & (c % 128 == 127))
            assert not wrong.any(), f"{what} {name}: {wrong.sum()} codes differ, first at {np.argwhere(wrong)[0]}"
            np.testing.assert_array_equal(ds.view(torch.uint8).cpu().numpy(), s, err_msg=f"{what} {name} scales")


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def view_of(t, how):
    """The same tokens on the GPU: as they are, in packed rows, head by head, or at odd places."""
    n, g, d = t.shape
    if how == "packed":
        row = torch.zeros(n, 3 * g * d, dtype=t.dtype, device=DEV)
        row[:, g * d:2 * g * d] = t.flatten(1).to(DEV)
        return row[:, g * d:2 * g * d].unflatten(1, (g, d))
    if how == "heads":
        return t.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
    if how == "odd":
        row = torch.zeros(n, g * d + 1, dtype=t.dtype, device=DEV)
        row[:, 1:] = t.flatten(1).to(DEV)
        return row[:, 1:].unflatten(1, (g, d))
    return t.to(DEV)


def tokens_of(n, G, D, dtype, seed, spread=0):
    """Tokens whose sizes differ by up to 2^spread from one to the next."""
    t = rand((n, G, D), torch.float32, seed)
    if spread:
        g = torch.Generator().manual_seed(seed + 1)
        t = t * 2.0 ** torch.randint(-spread, spread + 1, (n, G, 1), generator=g).float()
    return t.to(dtype)


# groups, dim, block, lengths before, new tokens, capacity, page (0: dense), cache layout, tokens' layout, spread
WRITES = [
    (1, 1, 16, [0], [1], 1, 0, "rows", "rows", 0),
    (8, 64, 16, [0, 1, 15, 16, 17, 300], [1] * 6, 301, 0, "heads", "packed", 3),
    (8, 64, 64, [0, 0], [200, 137], 256, 64, "heads", "packed", 0),
    (3, 80, 16, [0, 5, 31, 64], [48, 49, 1, 77], 144, 48, "rows", "rows", 9),
    (4, 128, 128, [0, 100, 128], [300, 29, 128], 384, 128, "rows", "heads", 2),
    (2, 40, 32, [7, 250], [130, 3], 253, 0, "heads", "rows", 12),
    (1, 7, 16, [3, 20], [30, 4], 48, 16, "odd", "odd", 4),
    (2, 128, 64, [60], [70], 192, 64, "odd", "rows", 4),
    (5, 100, 128, [130, 0], [140, 17], 512, 256, "rows", "odd", 1),
    (16, 16, 32, [33] * 9, [2] * 9, 96, 96, "rows", "rows", 20),
]


@pytest.mark.parametrize("case", WRITES, ids=str)
@pytest.mark.parametrize("name", list(TYPES))
def test_write(case, name):
    G, D, block, lengths, new, capacity, page, layout, how, spread = case
    dtype, n = TYPES[name], sum(new)
    cache = Cache(G, D, block, lengths, capacity, page, layout)
    k, v = (tokens_of(n, G, D, dtype, s, spread) for s in (1, 11))
    offsets = np.concatenate([[0], np.cumsum(new)])
    cfg = m3.Kv8Config(len(lengths), max(new), capacity, G, G, D, block)
    m3.m3_kv8_write(view_of(k, how), view_of(v, how), *cache.args(), ints(lengths), cfg, offsets=ints(offsets.tolist()),
                    block_table=cache.table)
    torch.cuda.synchronize()
    for x, (codes, scales) in zip((k, v), cache.host):
        for b, length in enumerate(lengths):
            K.write(codes, scales, block, f64(x[offsets[b]:offsets[b + 1]]), length, cache.pages(b))
    cache.same("write")


@pytest.mark.parametrize("name", list(TYPES))
def test_write_extremes(name):
    """Infinities, NaN, the type's largest and smallest values, zeros; blocks that keep, grow and begin a scale."""
    dtype, G, D, block = TYPES[name], 2, 64, 16
    cache = Cache(G, D, block, [8, 8, 8, 0, 16], 48, 16, "heads")
    x = rand((5 * 20, G, D), dtype, 3)
    info = torch.finfo(dtype)
    x[0, 0, 3], x[1, 1, 0], x[2, 0, 1] = float("inf"), float("nan"), -float("inf")
    x[20:40] = 0
    x[40, 0, 0], x[41, 1, 63] = info.max, info.min
    x[60:80] = info.smallest_normal * x[60:80] / 4  # below the normal numbers
    x[80:100, :, ::2] = float("nan")
    x[81, 0] = float("inf")
    cfg = m3.Kv8Config(5, 20, 48, G, G, D, block)
    lengths = [8, 8, 8, 0, 16]
    m3.m3_kv8_write(x.to(DEV), -x.to(DEV), *cache.args(), ints(lengths), cfg, block_table=cache.table)
    torch.cuda.synchronize()
    for sign, (codes, scales) in zip((1, -1), cache.host):
        for b, length in enumerate(lengths):
            K.write(codes, scales, block, sign * f64(x[20 * b:20 * b + 20]), length, cache.pages(b))
    cache.same("extremes")


@pytest.mark.parametrize("name", ["bf16", "f32"])
def test_write_leaves_alone(name):
    """Rows without room or with a negative length, empty rows, tokens of no row, and pages that are none."""
    dtype, G, D, block = TYPES[name], 2, 40, 32
    lengths = [60, -1, 90, 10, 0, 5]
    new = [4, 4, 7, 0, 40, 64]
    cache = Cache(G, D, block, [60, 0, 90, 10, 0, 5], 96, 32)
    table = cache.order.astype(np.int32)
    table[4, 1], table[5, 0], table[5, 2] = -1, 1 << 30, -(1 << 31)
    starts = 3 + np.concatenate([[0], np.cumsum(new)])
    x = tokens_of(int(starts[-1]) + 5, G, D, dtype, 4, 3)
    cfg = m3.Kv8Config(6, 64, 96, G, G, D, block)
    m3.m3_kv8_write(x.to(DEV), x.to(DEV), *cache.args(), ints(lengths), cfg, offsets=ints(starts.tolist()),
                    block_table=ints(table.tolist()))
    torch.cuda.synchronize()
    for codes, scales in cache.host:
        for b in (0, 4, 5):
            pages = cache.pages(b, {4: (1,), 5: (0, 2)}.get(b, ()))
            K.write(codes, scales, block, f64(x[starts[b]:starts[b + 1]]), lengths[b], pages)
    cache.same("left alone")


def test_write_token_by_token_is_one_write_of_like_tokens():
    """Tokens of one size give the same cache whether they come alone or together; the second way twice is the first."""
    G, D, block, n = 2, 64, 32, 70
    x = (torch.sign(rand((n, G, D), torch.float32, 5)) * 1.5).to(torch.bfloat16).to(DEV)
    one, many = (Cache(G, D, block, [0], 96, 32, seed=s) for s in (1, 1))
    for i in range(n):
        m3.m3_kv8_write(x[i:i + 1], x[i:i + 1], *one.args(), ints([i]), m3.Kv8Config(1, 1, 96, G, G, D, block),
                        block_table=one.table)
    for _ in range(2):
        m3.m3_kv8_write(x, x, *many.args(), ints([0]), m3.Kv8Config(1, n, 96, G, G, D, block), block_table=many.table)
    torch.cuda.synchronize()
    for a, b in zip(one.args(), many.args()):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


READS = [
    # groups, dim, block, rows' written positions, capacity, page, layout, starts, tokens, out layout
    (1, 1, 16, [1], 1, 0, "rows", None, [1], "rows"),
    (8, 64, 64, [200, 256], 256, 64, "heads", [0, 13], [200, 243], "rows"),
    (3, 80, 16, [96, 50, 144], 144, 48, "rows", [95, 0, 17], [1, 0, 127], "packed"),
    (4, 128, 128, [300], 300, 0, "heads", [128], [172], "heads"),
    (1, 7, 16, [48, 20], 48, 16, "odd", [15, 1], [18, 19], "odd"),
    (2, 100, 32, [70], 70, 0, "odd", [3], [60], "rows"),
]


@pytest.mark.parametrize("case", READS, ids=str)
@pytest.mark.parametrize("name", list(TYPES))
def test_read(case, name):
    G, D, block, lengths, capacity, page, layout, starts, new, how = case
    dtype, n = TYPES[name], sum(new)
    cache = Cache(G, D, block, lengths, capacity, page, layout)
    offsets = np.concatenate([[0], np.cumsum(new)])
    outs = {x: view_of(torch.full((n, G, D), 7.0, dtype=dtype), how) for x in "kv"}
    cfg = m3.Kv8Config(len(lengths), max(new), capacity, G, G, D, block)
    m3.m3_kv8_read(*cache.args(), cfg, starts=None if starts is None else ints(starts), offsets=ints(offsets.tolist()),
                   block_table=cache.table, outs=outs)
    torch.cuda.synchronize()
    for out, (codes, scales) in zip((outs["k"], outs["v"]), cache.host):
        for b, s in enumerate(starts or [0] * len(lengths)):
            ref = K.read(codes, scales, block, s, s + new[b], cache.pages(b))
            want = torch.from_numpy(ref).to(dtype)
            assert torch.equal(out[offsets[b]:offsets[b + 1]].cpu(), want), b
    cache.same("read")


@pytest.mark.parametrize("name", list(TYPES))
def test_read_outside(name):
    """Positions below zero, past the cache or without a page are zero; tokens of no row are not written; float16
    holds its largest value where the cache stands for more."""
    dtype, G, D, block = TYPES[name], 2, 64, 16
    cache = Cache(G, D, block, [64, 64, 64], 64, 32)
    cache.host[0][1][:] = 127 + 12  # keys up to 448 * 2^12
    cache.dev[0][1].view(torch.uint8).fill_(127 + 12)
    cache.host[1][0][cache.order[0, 0], 5, 0, 3] = 127
    cache.dev[1][0].view(torch.uint8)[int(cache.order[0, 0]), 5, 0, 3] = 255  # NaN stays NaN
    table = cache.order.astype(np.int32)
    table[2, 0] = 1 << 20
    starts, new = [-5, 40, 0], [12, 40, 64]
    offsets = 2 + np.concatenate([[0], np.cumsum(new)])
    outs = {x: torch.full((int(offsets[-1]) + 3, G, D), 7.0, dtype=dtype, device=DEV) for x in "kv"}
    m3.m3_kv8_read(*cache.args(), m3.Kv8Config(3, 64, 64, G, G, D, block), starts=ints(starts),
                   offsets=ints(offsets.tolist()), block_table=ints(table.tolist()), outs=outs)
    torch.cuda.synchronize()
    for out, (codes, scales) in zip((outs["k"], outs["v"]), cache.host):
        assert (out[:2] == 7).all() and (out[offsets[-1]:] == 7).all()
        for b in range(3):
            ref = K.read(codes, scales, block, starts[b], starts[b] + new[b], cache.pages(b, (0,) if b == 2 else ()))
            top = torch.finfo(dtype).max
            want = torch.from_numpy(ref).clamp(-top, top).to(dtype)
            got = out[offsets[b]:offsets[b + 1]].cpu()
            assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(0), want.nan_to_num(0)), b


def bound_of(q, k, v, out, size, scale, dtype, n):
    D = q.shape[-1]
    S = scale * np.abs(q).sum(-1).max() * np.abs(k).max(initial=0.0)
    rel = (D + 8) * 2.0 ** -24 * S + 2.0 ** -22 * S + 2.0 ** -21 + n * 2.0 ** -24
    return (PIECES[dtype] + 2 * rel) * size + half_step(dtype) * np.abs(out) + tiny(dtype)


# heads, groups, dim, block, lengths before, tokens, capacity, page, window, sinks, layout
STEPS = [
    (1, 1, 1, 16, [0], 1, 1, 0, 0, 0, "rows"),
    (2, 1, 16, 16, [0, 1, 15, 16, 17, 63], 1, 64, 0, 0, 0, "heads"),
    (24, 8, 64, 64, [127, 128, 129, 500], 1, 512, 0, 0, 0, "heads"),
    (24, 8, 64, 32, [127, 0, 31, 500], 2, 512, 64, 0, 0, "rows"),
    (8, 1, 128, 128, [700, 3, -1, 895, 896, 1000], 1, 896, 128, 0, 0, "rows"),
    (6, 2, 80, 16, [255, 64, 17, 0], 3, 288, 48, 60, 0, "rows"),
    (6, 2, 80, 16, [255, 64, 17, 140], 3, 288, 48, 60, 5, "heads"),
    (5, 5, 40, 16, [100, 90], 1, 101, 0, 1, 0, "rows"),
    (40, 1, 64, 32, [300, 17], 1, 320, 32, 0, 0, "rows"),
    (32, 4, 128, 64, [900, 130], 7, 960, 192, 129, 4, "heads"),
    (3, 3, 7, 16, [50, 20, 77], 1, 78, 0, 20, 17, "odd"),
    (4, 2, 100, 32, [2000, 5], 4, 2048, 64, 129, 1, "odd"),
    (4, 4, 64, 64, [5000], 1, 5120, 0, 0, 0, "heads"),
    (4, 2, 96, 64, [2900, 200], 1, 2944, 64, 1000, 200, "rows"),
    (2, 2, 32, 16, [700], 64, 800, 16, 33, 3, "rows"),
    (16, 1, 128, 128, [260], 5, 384, 0, 0, 0, "rows"),
]


@pytest.mark.parametrize("case", STEPS, ids=str)
@pytest.mark.parametrize("name", list(TYPES))
def test_step(case, name):
    H, G, D, block, lengths, T, capacity, page, window, sinks, layout = case
    dtype, n = TYPES[name], len(lengths)
    cache = Cache(G, D, block, lengths, capacity, page, layout)
    q = rand((n * T, H, D), dtype, 1)
    k, v = (tokens_of(n * T, G, D, dtype, s, 1) for s in (2, 3))
    cfg = m3.Kv8Config(n, T, capacity, H, G, D, block, window, sinks)
    out = m3.m3_attn_step_kv8(q.to(DEV), k.to(DEV), v.to(DEV), *cache.args(), ints(lengths), cfg, block_table=cache.table)
    again = m3.m3_attn_step_kv8(q.to(DEV), None, None, *cache.args(), ints(lengths), cfg, block_table=cache.table)
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    for b, length in enumerate(lengths):
        rows = slice(b * T, b * T + T)
        if not 0 <= length <= capacity - T:
            assert (out[rows] == 0).all()
            continue
        for x, (codes, scales) in zip((k, v), cache.host):
            K.write(codes, scales, block, f64(x[rows]), length, cache.pages(b))
        kk, vv = (K.read(c, s, block, 0, length + T, cache.pages(b)) for c, s in cache.host)
        seen = K.visible(T, length, window, sinks)
        ref, size = K.step(f64(q[rows]), kk, vv, seen, D ** -0.5)
        bound = bound_of(f64(q[rows]), kk[seen.any(0)], vv, ref, size, D ** -0.5, dtype, length + T)
        check(out[rows], ref, bound, f"row {b} length {length}")
    cache.same("step")


@pytest.mark.parametrize("T,window,sinks", [(1, 0, 0), (3, 40, 2), (9, 40, 2)])
@pytest.mark.parametrize("name", list(TYPES))
def test_step_nan_reaches_those_that_see_it(name, T, window, sinks):
    """NaN codes everywhere a query does not look, and one that only some of the new tokens see."""
    dtype, H, G, D, block, length = TYPES[name], 4, 2, 64, 16, 150
    cache = Cache(G, D, block, [length], 192, 48)
    codes = cache.host[1][0]
    lo = max(0, length + 1 - window) if window else 0
    hide = [j for j in range(192) if j >= length + T or (window and sinks <= j < lo)]
    for c, _ in cache.host:
        for j in hide:
            c[cache.order[0, j // 48], j % 48] = 127
    at = lo + 1  # in the first token's window alone, or in everyone's sight without one
    codes[cache.order[0, at // 48], at % 48, 1, 5] = 255
    cache.dev = [(cache.place(c, "rows"), s) for (c, _), (_, s) in zip(cache.host, cache.dev)]
    q = rand((T, H, D), dtype, 1)
    k, v = (rand((T, G, D), dtype, s) for s in (2, 3))
    cfg = m3.Kv8Config(1, T, 192, H, G, D, block, window, sinks)
    out = m3.m3_attn_step_kv8(q.to(DEV), k.to(DEV), v.to(DEV), *cache.args(), ints([length]), cfg, block_table=cache.table)
    torch.cuda.synchronize()
    for x, (c, s) in zip((k, v), cache.host):
        K.write(c, s, block, f64(x), length, cache.pages(0))
    kk, vv = (K.read(c, s, block, 0, length + T, cache.pages(0)) for c, s in cache.host)
    seen = K.visible(T, length, window, sinks)
    ref, size = K.step(f64(q), kk, vv, seen, D ** -0.5)
    assert np.isnan(ref).any() and np.isnan(ref[:, :, 5][:, 2:]).sum() == np.isnan(ref).sum()
    np.testing.assert_array_equal(np.isnan(f64(out)), np.isnan(ref))
    bound = bound_of(f64(q), kk[seen.any(0)], vv, ref, size, D ** -0.5, dtype, length + T)
    check(torch.from_numpy(np.nan_to_num(f64(out))), np.nan_to_num(ref), np.nan_to_num(bound), "beside the NaN")


@pytest.mark.parametrize("name", list(TYPES))
def test_step_nan_keys_and_queries(name):
    """A NaN key gives NaN to the queries that see it; a query of NaN or infinities spoils its own row alone."""
    dtype, H, G, D, block, T = TYPES[name], 4, 2, 64, 16, 3
    cache = Cache(G, D, block, [40], 64, 0)
    q = rand((T, H, D), dtype, 1)
    k, v = (rand((T, G, D), dtype, s) for s in (2, 3))
    k[2, 0, 7] = float("nan")  # the last token's key, first group
    q[0, 3, 1] = float("inf")
    q[1, 2, 0] = float("nan")
    out = m3.m3_attn_step_kv8(q.to(DEV), k.to(DEV), v.to(DEV), *cache.args(), ints([40]),
                              m3.Kv8Config(1, T, 64, H, G, D, block))
    torch.cuda.synchronize()
    bad = torch.zeros(T, H, dtype=torch.bool)
    bad[2, :2] = bad[0, 3] = bad[1, 2] = True
    assert torch.equal(out.isnan().any(-1).cpu(), bad) and torch.equal(out.isnan().all(-1).cpu(), bad)


@pytest.mark.parametrize("name", list(TYPES))
def test_step_bad_pages(name):
    """Positions whose table entry is no page are not seen; a row of such pages alone is zero."""
    dtype, H, G, D, block, page = TYPES[name], 4, 2, 64, 16, 16
    lengths = [70, 40, 33, 20]
    cache = Cache(G, D, block, lengths, 96, page)
    table = cache.order.astype(np.int32)
    table[0, 1], table[1, 2], table[2, 0], table[3] = -1, 1 << 30, -(1 << 31), -7
    gone = [(1,), (2,), (0,), range(6)]
    q, k, v = rand((4, H, D), dtype, 1), rand((4, G, D), dtype, 2), rand((4, G, D), dtype, 3)
    out = m3.m3_attn_step_kv8(q.to(DEV), k.to(DEV), v.to(DEV), *cache.args(), ints(lengths),
                              m3.Kv8Config(4, 1, 96, H, G, D, block), block_table=ints(table.tolist()))
    torch.cuda.synchronize()
    for b, length in enumerate(lengths):
        for x, (c, s) in zip((k, v), cache.host):
            K.write(c, s, block, f64(x[b:b + 1]), length, cache.pages(b, gone[b]))
        kk, vv = (K.read(c, s, block, 0, length + 1, cache.pages(b)) for c, s in cache.host)
        seen = np.array([[j // page not in gone[b] for j in range(length + 1)]])
        ref, size = K.step(f64(q[b:b + 1]), kk, vv, seen, D ** -0.5)
        if b == 3:
            assert (out[b] == 0).all()
        kk, vv = (np.where(seen[0][:, None, None], x, 0) for x in (kk, vv))
        check(out[b:b + 1], ref, bound_of(f64(q[b:b + 1]), kk, vv, ref, size, D ** -0.5, dtype, length + 1), f"row {b}")
    cache.same("bad pages")


def test_cache_beyond_32_bits():
    """Pages whose codes lie past 2^32: written, read back and attended to."""
    G, D, page, block = 8, 128, 64, 64
    pages = 2 ** 32 // (G * D * page) + 8
    codes = [torch.empty((pages, page, G, D), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2)]
    scales = [torch.empty((pages, G, 1), dtype=torch.uint8, device=DEV).view(torch.float8_e8m0fnu) for _ in range(2)]
    table = ints([[pages - 1, 0, pages - 3]])
    n = 2 * page + 20
    q, k, v = (rand((n + 1, h, D), torch.bfloat16, 20 + h) for h in (16, G, G + 1))
    v = v[:, :G].contiguous()
    args = (codes[0], scales[0], codes[1], scales[1])
    m3.m3_kv8_write(k[:n].to(DEV), v[:n].to(DEV), *args, ints([0]), m3.Kv8Config(1, n, 3 * page, G, G, D, block),
                    block_table=table)
    out = m3.m3_attn_step_kv8(q[n:].to(DEV), k[n:].to(DEV), v[n:].to(DEV), *args, ints([n]),
                              m3.Kv8Config(1, 1, 3 * page, 16, G, D, block), block_table=table)
    got = m3.m3_kv8_read(*args, m3.Kv8Config(1, n + 1, 3 * page, G, G, D, block), block_table=table)
    torch.cuda.synchronize()
    host = [(np.zeros((3, page, G, D), np.uint8), np.zeros((3, G, 1), np.uint8)) for _ in range(2)]
    for x, (c, s), y in zip((k, v), host, (got["k"], got["v"])):
        K.write(c, s, block, f64(x[:n]), 0, [0, 1, 2])
        K.write(c, s, block, f64(x[n:]), n, [0, 1, 2])
        np.testing.assert_array_equal(f64(y), K.read(c, s, block, 0, n + 1, [0, 1, 2]))
    kk, vv = (K.read(c, s, block, 0, n + 1, [0, 1, 2]) for c, s in host)
    ref, size = K.step(f64(q[n:]), kk, vv, K.visible(1, n, 0, 0), D ** -0.5)
    check(out, ref, bound_of(f64(q[n:]), kk, vv, ref, size, D ** -0.5, torch.bfloat16, n + 1), "far pages")
