"""The 8-bit key / value cache at the limits of its numbers: the largest values of the types, bits that are no finite
number, scales and codes that m3_kv8_write never leaves, queries and scores near the ends of float32.  Codes, scales
and what is read back are the oracle's bit for bit; tolerances of the step are those of test_gpu_kv8."""

import numpy as np
import pytest
import torch

import selective_state_space_mamba3_amd as m3
from oracle import kv8 as K
from test_gpu_attn import DEV, TYPES, check, f64, half_step, rand, tiny
from test_gpu_kv8 import PIECES, Cache, bound_of, ints

pytestmark = pytest.mark.gpu

WIDE = ["f32", "bf16"]  # the types that reach float32's largest values


def place(cache):
    """The host's caches on the GPU, after a test changed them there."""
    cache.dev = [(cache.place(c, "rows"), torch.from_numpy(s).to(DEV).view(torch.float8_e8m0fnu)) for c, s in cache.host]


def read_back(cache, dtype, n, capacity):
    got = m3.m3_kv8_read(*cache.args(), m3.Kv8Config(1, n, capacity, cache.G, cache.G, cache.D, cache.block),
                         block_table=cache.table, dtype=dtype)
    torch.cuda.synchronize()
    return got["k"], got["v"]


@pytest.mark.parametrize("grown", [False, True])
@pytest.mark.parametrize("name", list(TYPES))
def test_largest_values_are_held(name, grown):
    """Values up to the type's largest come back finite and within e4m3's half step of themselves, from blocks that begin
    with them and from blocks that grow to hold them."""
    dtype, G, D, block, n = TYPES[name], 2, 64, 16, 9
    cache, before = Cache(G, D, block, [5 if grown else 0], 48, 16), 5 if grown else 0
    top = torch.finfo(dtype).max
    x = rand((n, G, D), torch.float32, 1)
    sizes = torch.tensor([1.0, 0.998, 0.98, 0.97, 0.969, 0.96875, 0.95, 0.9, 0.5])
    x = torch.where(torch.arange(D) % 2 == 0, sizes[:, None, None] * torch.sign(x), x).double() * top
    x = x.clamp(-top, top).to(dtype)
    assert x.isfinite().all() and x.max() == top
    m3.m3_kv8_write(x.to(DEV), -x.to(DEV), *cache.args(), ints([before]), m3.Kv8Config(1, n, 48, G, G, D, block),
                    block_table=cache.table)
    got = read_back(cache, dtype, before + n, 48)
    for sign, out, (codes, scales) in zip((1, -1), got, cache.host):
        K.write(codes, scales, block, sign * f64(x), before, cache.pages(0))
        ref = K.read(codes, scales, block, 0, before + n, cache.pages(0))
        want = torch.from_numpy(ref).clamp(-top, top).to(dtype)
        assert out.isfinite().all() and torch.equal(out.cpu(), want)
        exact = sign * f64(x)
        # half a step of e4m3 relative to the value, half its least step (2^-10 2^e) for the small ones, and none of the
        # type's own for what float16 does not hold
        e = scales[cache.order[0, 0], :, 0].astype(np.int64) - K.BIAS
        bound = np.maximum(2.0 ** -4 * np.abs(exact), 2.0 ** (e[None, :, None] - 10.0))
        assert (np.abs(f64(out[before:]) - exact) <= bound).all()
    cache.same("largest")


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("name", WIDE)
def test_largest_values_stay_hidden(name, T):
    """The type's largest value in the last of the new tokens, and in the position before the window: it reaches no query
    that does not see it."""
    dtype, H, G, D, block, window = TYPES[name], 4, 2, 64, 16, 50
    lengths = [70, 61]
    top = torch.finfo(dtype).max
    cache = Cache(G, D, block, lengths, 128, 64)
    for b, length in enumerate(lengths):  # the first of these twelve stands just outside the first token's window
        x, y = rand((12, G, D), dtype, 9), (rand((12, G, D), torch.float32, 10) * 2.0 ** 113).to(dtype)
        x[0, :, 3::7], y[0, :, ::4] = top, top if b else -top
        at = ints([-1, -1])
        at[b] = length - window
        m3.m3_kv8_write(torch.cat([x, x]).to(DEV), torch.cat([y, y]).to(DEV), *cache.args(), at,
                        m3.Kv8Config(2, 12, 128, G, G, D, block), block_table=cache.table)
        for t, (codes, scales) in zip((x, y), cache.host):
            K.write(codes, scales, block, f64(t), length - window, cache.pages(b))
    q = rand((2 * T, H, D), dtype, 1)
    k, v = (rand((2 * T, G, D), dtype, s) for s in (2, 3))
    for b in range(2):
        v[b * T + T - 1, :, ::5] = top
    out = m3.m3_attn_step_kv8(q.to(DEV), k.to(DEV), v.to(DEV), *cache.args(), ints(lengths),
                              m3.Kv8Config(2, T, 128, H, G, D, block, window), block_table=cache.table)
    torch.cuda.synchronize()
    for b, length in enumerate(lengths):
        rows = slice(b * T, b * T + T)
        for x, (c, s) in zip((k, v), cache.host):
            K.write(c, s, block, f64(x[rows]), length, cache.pages(b))
        kk, vv = (K.read(c, s, block, 0, length + T, cache.pages(b)) for c, s in cache.host)
        seen = K.visible(T, length, window, 0)
        seen[-1] = False  # (the last query sums what passes float32; the others see none of it)
        ref, size = K.step(f64(q[rows]), kk, vv, seen, D ** -0.5)
        bound = bound_of(f64(q[rows]), kk[seen.any(0)], vv, ref, size, D ** -0.5, dtype, length + T)
        check(out[rows][:-1], ref[:-1], bound[:-1], f"row {b}")
    cache.same("hidden")


@pytest.mark.parametrize("name", list(TYPES))
def test_hidden_bits_of_any_kind(name):
    """Codes and scales that stand for more than float32 holds, as memory that was never written has them: outside the
    window they reach nobody, inside only the queries that see them."""
    dtype, H, G, D, block, T, window = TYPES[name], 4, 2, 64, 64, 3, 20
    for byte, big in ((247, 0x78), (247, 0x7e), (254, 0x40), (250, 0x7e)):
        length = 50
        cache = Cache(G, D, block, [length], 64, 64)
        lo, page = length + 1 - window, cache.order[0, 0]
        codes, scales = cache.host[1]
        # visible values so small that their sums stay in float32 (none in float16, whose results end before them)
        codes[page, lo:length] = 0
        codes[page, lo + 1] = 0 if name == "f16" else np.random.default_rng(1).integers(0, 2, (G, D))
        codes[page, :lo] = big
        codes[page, lo, 1, 5] = big  # the first token's query sees it, and no other
        scales[page] = byte
        cache.host[0][0][page, :lo] = 0x7e
        place(cache)
        q = rand((T, H, D), dtype, 1)
        k, v = (rand((T, G, D), dtype, s) for s in (2, 3))
        out = m3.m3_attn_step_kv8(q.to(DEV), k.to(DEV), v.to(DEV), *cache.args(), ints([length]),
                                  m3.Kv8Config(1, T, 64, H, G, D, block, window), block_table=cache.table)
        torch.cuda.synchronize()
        bad = torch.zeros(T, H, D, dtype=torch.bool)
        bad[0, 2:, 5] = True
        assert torch.equal(~out.isfinite().cpu(), bad), (byte, big, (~out.isfinite()).sum().item())
        for x, (c, s) in zip((k, v), cache.host):
            K.write(c, s, block, f64(x), length, cache.pages(0))
        kk, vv = (K.read(c, s, block, 0, length + T, cache.pages(0)) for c, s in cache.host)
        seen = K.visible(T, length, window, 0)
        ref, size = K.step(f64(q), kk, vv, seen, D ** -0.5)
        bound = bound_of(f64(q), kk[seen.any(0)], vv, ref, size, D ** -0.5, dtype, length + T)
        keep = ~bad.numpy()
        check(out.cpu()[~bad], ref[keep], bound[keep], f"byte {byte} code {big}")


@pytest.mark.parametrize("name", WIDE)
def test_signalling_nan_hides_no_larger_neighbour(name):
    """A NaN of either kind, at each place of a piece, leaves the scale to the finite elements beside it."""
    dtype, G, D, block = TYPES[name], 1, 64, 16
    quiet, signalling = {"bf16": (0x7fc1, 0x7f81), "f32": (0x7fc00001, 0x7f800001)}[name]
    ints_of = {"bf16": torch.int16, "f32": torch.int32}[name]
    cases = [(bits, at, big) for bits in (quiet, signalling) for at in range(8) for big in range(8) if big != at]
    n = len(cases)
    x = rand((n, G, D), dtype, 3)
    for i, (bits, at, big) in enumerate(cases):
        x[i, 0, 8 + big] = 100.0 + i
        x.view(ints_of)[i, 0, 8 + at] = bits
    for T in (1, 2):  # written alone, and by the decode step
        cache = Cache(G, D, block, [0] * n, 16, 0)
        if T == 1:
            m3.m3_kv8_write(x.to(DEV), x.to(DEV), *cache.args(), ints([0] * n), m3.Kv8Config(n, 1, 16, G, G, D, block))
        else:
            m3.m3_attn_step_kv8(rand((n, G, D), dtype, 4).to(DEV), x.to(DEV), x.to(DEV), *cache.args(), ints([0] * n),
                                m3.Kv8Config(n, 1, 16, G, G, D, block))
        torch.cuda.synchronize()
        for codes, scales in cache.host:
            for b in range(n):
                K.write(codes, scales, block, f64(x[b:b + 1]), 0, cache.pages(b))
        cache.same(f"way {T}")


@pytest.mark.parametrize("name", list(TYPES))
def test_scale_bytes_of_any_value(name):
    """New tokens beside older ones whose scale byte is any of 256: 255 counts as 254, and what is written stands for the
    tokens at the scale that results."""
    dtype, G, D, block = TYPES[name], 1, 64, 16
    x = rand((256, G, D), torch.float32, 3)
    x = (x * torch.finfo(dtype).max / 64).to(dtype)
    for step in (False, True):
        cache = Cache(G, D, block, [4] * 256, 16, 0)
        for codes, scales in cache.host:
            scales[:256, 0, 0] = np.arange(256)
        place(cache)
        if step:
            m3.m3_attn_step_kv8(rand((256, G, D), dtype, 4).to(DEV), x.to(DEV), x.to(DEV), *cache.args(), ints([4] * 256),
                                m3.Kv8Config(256, 1, 16, G, G, D, block))
        else:
            m3.m3_kv8_write(x.to(DEV), x.to(DEV), *cache.args(), ints([4] * 256), m3.Kv8Config(256, 1, 16, G, G, D, block))
        torch.cuda.synchronize()
        for codes, scales in cache.host:
            scales[255] = 254
            for b in range(256):
                K.write(codes, scales, block, f64(x[b:b + 1]), 4, cache.pages(b))
        cache.same(f"step {step}")


@pytest.mark.parametrize("size", [1e20, 1e36, 1e38])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("name", WIDE)
def test_large_queries_at_a_small_scale(name, window, size):
    """Scores are right wherever they themselves are in float32, though queries times codes pass it; and a query's bits
    do not depend on the size of the one beside it."""
    dtype, H, G, D, block, T, length = TYPES[name], 4, 2, 64, 16, 2, 150
    cache = Cache(G, D, block, [length], 192, 48)
    q = rand((T, H, D), torch.float32, 1).clamp(-3, 3)
    q[:, ::2] *= size
    q = q.to(dtype)
    k, v = (rand((T, G, D), dtype, s) for s in (2, 3))
    cfg = m3.Kv8Config(1, T, 192, H, G, D, block, window, scale=1 / size)
    out = m3.m3_attn_step_kv8(q.to(DEV), k.to(DEV), v.to(DEV), *cache.args(), ints([length]), cfg, block_table=cache.table)
    other = q.clone()
    other[:, ::2] = 0
    beside = m3.m3_attn_step_kv8(other.to(DEV), None, None, *cache.args(), ints([length]), cfg, block_table=cache.table)
    torch.cuda.synchronize()
    for x, (c, s) in zip((k, v), cache.host):
        K.write(c, s, block, f64(x), length, cache.pages(0))
    kk, vv = (K.read(c, s, block, 0, length + T, cache.pages(0)) for c, s in cache.host)
    seen = K.visible(T, length, window, 0)
    scale = float(np.float32(1 / size))
    ref, out_size = K.step(f64(q), kk, vv, seen, scale)
    check(out, ref, bound_of(f64(q), kk[seen.any(0)], vv, ref, out_size, scale, dtype, length + T), f"size {size}")
    assert torch.equal(out[:, 1::2], beside[:, 1::2])
    cache.same("queries")


@pytest.mark.parametrize("power", [10, 26, 40, 120])
@pytest.mark.parametrize("capacity", [704, 8192])
@pytest.mark.parametrize("name", list(TYPES))
def test_scores_far_from_zero(name, capacity, power):
    """Scores of some 2^power, exact in float32: the largest takes all, and equal ones share alike."""
    dtype, H, G, D, block, T, length = TYPES[name], 4, 2, 64, 16, 2, 700
    cache = Cache(G, D, block, [0], capacity, 64)
    g = np.random.default_rng(4)
    keys, values = (g.standard_normal((length + T, G, D)) for _ in range(2))
    keys[:, :, 0] = g.integers(1, 12, (length + T, G))
    keys[:, :, 0] *= np.where(np.arange(length + T) % 300 == 150, 2, 1)[:, None]
    values = torch.from_numpy(values).to(dtype)
    keys = torch.from_numpy(keys).to(dtype)
    q = torch.zeros(T, H, D, dtype=dtype)
    q[:, :, 0] = torch.tensor([3.0, -3.0, 1.0, -1.0])
    m3.m3_kv8_write(keys[:length].to(DEV), values[:length].to(DEV), *cache.args(), ints([0]),
                    m3.Kv8Config(1, length, capacity, G, G, D, block), block_table=cache.table)
    scale = 1.25 * 2.0 ** (power - 4)
    out = m3.m3_attn_step_kv8(q.to(DEV), keys[length:].to(DEV), values[length:].to(DEV), *cache.args(), ints([length]),
                              m3.Kv8Config(1, T, capacity, H, G, D, block, scale=scale), block_table=cache.table)
    torch.cuda.synchronize()
    for x, (c, s) in zip((keys, values), cache.host):
        K.write(c, s, block, f64(x[:length]), 0, cache.pages(0))
        K.write(c, s, block, f64(x[length:]), length, cache.pages(0))
    kk, vv = (K.read(c, s, block, 0, length + T, cache.pages(0)) for c, s in cache.host)
    ref, size = K.step(f64(q), kk, vv, K.visible(T, length, 0, 0), scale)
    # equal scores are equal products, and others lie too far apart to count (2^10 / 16 at the least): probabilities are
    # one or nothing before they are rounded to their pieces; 2^-21 for the exponentials and the sum
    assert np.abs(ref).max() > 0.1
    check(out, ref, (PIECES[dtype] + 2.0 ** -20) * size + half_step(dtype) * np.abs(ref) + tiny(dtype), f"2^{power}")


@pytest.mark.parametrize("capacity", [64, 4096, 16384])
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("name", list(TYPES))
def test_scores_of_minus_infinity(name, T, capacity):
    """A query that holds an infinity has no finite scores: its row is NaN, also where all of them are minus infinity,
    at the first position, in a window and in one stretch of many; a row without positions stays zero."""
    dtype, H, G, D, block = TYPES[name], 4, 2, 64, 16
    lengths = [0, 1, 33, capacity - T, -1]
    caches = Cache(G, D, block, [0, 1, 33, min(capacity - T, 700), 0], capacity, 64)
    if capacity > 700:
        lengths[3] = 700
    for c, s in caches.host:
        c &= 0x7f  # no value below zero
        c[c < 8] = 8
        c[c == 127] = 9
        s[:] = 120
    place(caches)
    q = torch.zeros(5 * T, H, D)
    q[:, 1, 7], q[:, 2] = -float("inf"), rand((5 * T, D), torch.float32, 1)
    k, v = (rand((5 * T, G, D), torch.float32, s).abs() + 0.5 for s in (2, 3))
    for window in (0, 20):
        out = m3.m3_attn_step_kv8(q.to(dtype).to(DEV), k.to(dtype).to(DEV), v.to(dtype).to(DEV), *caches.args(),
                                  ints(lengths), m3.Kv8Config(5, T, capacity, H, G, D, block, window),
                                  block_table=caches.table)
        torch.cuda.synchronize()
        assert (out[4 * T:] == 0).all()
        bad = torch.zeros(4 * T, H, D, dtype=torch.bool)
        bad[:, 1] = True
        assert torch.equal(out[:4 * T].isnan().cpu(), bad) and out[:4 * T, 2:].isfinite().all(), window
