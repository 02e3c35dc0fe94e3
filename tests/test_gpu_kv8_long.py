"""The decode step over the 8-bit cache along whole rows: many tiles to a workgroup of four and of eight waves, table
entries stepped from page to page, new tokens in a late tile, running maxima that move often; then reads and steps on two
streams at once, and a layer's rows decoded from such a cache.  Tolerances are those of test_gpu_kv8."""

import os
import sys

import numpy as np
import pytest
import torch

import selective_state_space_mamba3_amd as m3
from oracle import kv8 as K
from test_gpu_attn import DEV, TYPES, check, f64, half_step, rand
from test_gpu_kv8 import Cache, bound_of, ints

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

# heads, groups, dim, block, rows, longest row before the new tokens, tokens, page, window, sinks, layout.
# 1024 (row, group) pairs and more take workgroups of four waves (tiles of 128 positions), half the places and more eight
# (256 positions), both without a split.
LONG = [
    (16, 8, 64, 16, 130, 2291, 1, 144, 0, 0, "heads"),
    (8, 8, 32, 64, 130, 2047, 1, 0, 0, 0, "rows"),
    (32, 8, 32, 32, 130, 1500, 5, 96, 0, 0, "heads"),
    (16, 8, 64, 32, 130, 2291, 2, 96, 1500, 300, "rows"),
    (16, 8, 128, 32, 40, 4341, 1, 0, 0, 0, "heads"),
    (32, 4, 128, 128, 40, 4090, 4, 128, 0, 0, "rows"),
    (8, 4, 96, 16, 40, 4200, 3, 48, 2900, 700, "rows"),
    (4, 4, 20, 16, 80, 3000, 1, 80, 0, 0, "odd"),
]


@pytest.mark.parametrize("case", LONG, ids=str)
@pytest.mark.parametrize("name", list(TYPES))
def test_whole_rows(case, name):
    H, G, D, block, rows, longest, T, page, window, sinks, layout = case
    dtype, g = TYPES[name], np.random.default_rng(8)
    page, capacity = page or longest + T, longest + T
    per = -(-capacity // page)
    cache = Cache(G, D, block, [], capacity, page, layout, spare=rows * per)
    # any codes but NaN, at scales that make keys of size one and let the running maxima move along a row
    for i, (codes, scales) in enumerate(cache.host):
        codes[:] = g.integers(0, 0x70, codes.shape) + 128 * g.integers(0, 2, codes.shape)
        scales[:] = 127 - 8 + (g.integers(-3, 2, scales.shape) if i == 0 else g.integers(-2, 3, scales.shape))
    order = g.permutation(rows * per).reshape(rows, per)
    cache.dev = [(cache.place(c, layout), torch.from_numpy(s).to(DEV).view(torch.float8_e8m0fnu)) for c, s in cache.host]
    lengths = g.integers(longest // 3, longest + 1, rows)
    look = [0, 1, rows // 2, rows - 1]
    lengths[look[:2]], lengths[look[3]] = longest, longest - 257
    lengths[3] = -1
    q = rand((rows * T, H, D), dtype, 1)
    k, v = (rand((rows * T, G, D), dtype, s) for s in (2, 3))
    out = m3.m3_attn_step_kv8(q.to(DEV), k.to(DEV), v.to(DEV), *cache.args(), ints(lengths.tolist()),
                              m3.Kv8Config(rows, T, capacity, H, G, D, block, window, sinks),
                              block_table=ints(order.tolist()))
    torch.cuda.synchronize()
    assert (out[3 * T:4 * T] == 0).all() and out.isfinite().all()
    for b in range(rows):
        if b != 3:
            at, pages = int(lengths[b]), [int(p) for p in order[b]]
            for x, (codes, scales) in zip((k, v), cache.host):
                K.write(codes, scales, block, f64(x[b * T:b * T + T]), at, pages)
    cache.same("whole rows")
    for b in look:
        at, pages, mine = int(lengths[b]), [int(p) for p in order[b]], slice(b * T, b * T + T)
        kk, vv = (K.read(c, s, block, 0, at + T, pages) for c, s in cache.host)
        ref, size = K.step(f64(q[mine]), kk, vv, K.visible(T, at, window, sinks), D ** -0.5)
        check(out[mine], ref, bound_of(f64(q[mine]), kk, vv, ref, size, D ** -0.5, dtype, at + T), f"row {b}")


def test_reads_and_steps_at_once():
    """Reads and steps of one cache on a stream, of another on another, at the same time: each as if alone."""
    H, G, D, block, dtype, n = 8, 4, 128, 64, torch.bfloat16, 3000
    runs = []
    for s in range(2):
        g = np.random.default_rng(s)
        cache = Cache(G, D, block, [], 4096, 256, seed=s, spare=48)
        for codes, scales in cache.host:
            codes[:] = g.integers(0, 0x7f, codes.shape)
            scales[:] = 119
        cache.dev = [(cache.place(c, "rows"), torch.from_numpy(x).to(DEV).view(torch.float8_e8m0fnu)) for c, x in cache.host]
        q = rand((3, H, D), dtype, 7 * s).to(DEV)
        runs.append((cache, q, ints([n, 60, 1200]), ints(g.permutation(48).reshape(3, 16).tolist())))
    step, read = m3.Kv8Config(3, 1, 4096, H, G, D, block), m3.Kv8Config(3, n, 4096, H, G, D, block)

    def go(run, stream=None):
        cache, q, at, table = run
        out = m3.m3_attn_step_kv8(q, None, None, *cache.args(), at, step, block_table=table, stream=stream)
        got = m3.m3_kv8_read(*cache.args(), read, block_table=table, stream=stream)
        return out, got["k"], got["v"]

    want = [go(run) for run in runs]
    torch.cuda.synchronize()
    for x in want:
        assert x[0].isfinite().all() and x[1].abs().max() > 1
    streams = [torch.cuda.Stream() for _ in runs]
    got = [go(run, stream) for _ in range(4) for run, stream in zip(runs, streams)]
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        for a, b in zip(outs, want[i % 2]):
            assert torch.equal(a, b), i


def test_layer_decodes_what_its_cache_holds():
    """The example layer's rows from an 8-bit cache against float64 attention over the same cache: half a step of bfloat16
    for the layer's inner result and for its output, two pieces of the probabilities, float32 for the sums."""
    import attention_layer as example

    H, G, D, W, block, page, T = example.HEADS, example.GROUPS, example.DIM, example.WIDTH, 16, 32, 4
    layer = example.AttentionLayer(7)
    cache = Cache(G, D, block, [0, 0], 96, page, "heads")
    x = rand((2, 60, W), torch.bfloat16, 5).to(DEV)
    weight = f64(layer.weights["out"].to(torch.bfloat16))
    u, at = half_step(torch.bfloat16), [0, 13]
    prompt = x[:, :40].flatten(0, 1)
    positions = torch.cat([torch.arange(a, a + 40) for a in at]).to(torch.int32).to(DEV)
    q, k, v = layer.project(prompt)
    _, kn = layer.normed(q, k, positions)
    # (row 1 begins at 13: what is before it is written first, with the same tokens)
    first = ints([0, 0])
    m3.m3_kv8_write(kn, v, *cache.args(), first, m3.Kv8Config(2, 40, 96, G, G, D, block), block_table=cache.table)
    m3.m3_kv8_write(kn, v, *cache.args(), ints(at), m3.Kv8Config(2, 40, 96, G, G, D, block), block_table=cache.table)
    for t, (c, s) in zip((kn, v), cache.host):
        for b in range(2):
            K.write(c, s, block, f64(t[40 * b:40 * b + 40]), 0, cache.pages(b))
            K.write(c, s, block, f64(t[40 * b:40 * b + 40]), at[b], cache.pages(b))
    at = [a + 40 for a in at]
    for turn in range(5):
        new = x[:, 40 + 4 * turn:44 + 4 * turn].flatten(0, 1)
        got = layer.decode_8bit(new, cache.args(), ints(at), cache.table, T, block)
        q, k, v = layer.project(new)
        qn, kn = layer.normed(q, k, torch.cat([torch.arange(a, a + T) for a in at]).to(torch.int32).to(DEV))
        torch.cuda.synchronize()
        for b in range(2):
            mine = slice(b * T, b * T + T)
            for t, (c, s) in zip((kn, v), cache.host):
                K.write(c, s, block, f64(t[mine]), at[b], cache.pages(b))
            kk, vv = (K.read(c, s, block, 0, at[b] + T, cache.pages(b)) for c, s in cache.host)
            o, size = K.step(f64(qn[mine]), kk, vv, K.visible(T, at[b], 0, 0), D ** -0.5)
            off = bound_of(f64(qn[mine]), kk, vv, o, size, D ** -0.5, torch.bfloat16, at[b] + T)
            ref = o.reshape(T, -1) @ weight
            # the product's float32 sum of H D terms, and its rounding
            bound = off.reshape(T, -1) @ np.abs(weight) + H * D * 2.0 ** -24 * (np.abs(o).reshape(T, -1) @ np.abs(weight))
            bound = bound * (1 + u) + u * np.abs(ref)
            assert np.sqrt((bound ** 2).mean()) < 0.1 * np.sqrt((ref ** 2).mean())  # (rows of zeros would not pass)
            check(got[mine], ref, bound, f"turn {turn} row {b}")
        at = [a + T for a in at]
    cache.same("layer")
