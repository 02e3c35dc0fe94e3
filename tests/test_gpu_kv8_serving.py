"""The 8-bit cache's calls together, as a serving program makes them: prompts written, tokens decoded one and a few at a
time, drafts taken back, contexts read back for a prompt that goes on; from graphs, from other streams, over calls
that are alike.  Tolerances are those of test_gpu_kv8."""

import os
import sys

import numpy as np
import pytest
import torch

import selective_state_space_mamba3_amd as m3
from oracle import kv8 as K
from test_gpu_attn import DEV, TYPES, check, f64, half_step, rand
from test_gpu_kv8 import PIECES, Cache, bound_of, ints

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("name", list(TYPES))
def test_prompt_decode_and_a_prompt_that_goes_on(name):
    """Write, step token by token, take drafts back, read, attend: every result against the oracle's cache."""
    dtype, H, G, D, block, page = TYPES[name], 6, 2, 64, 32, 32
    lengths, total = [45, 0], 128
    cache = Cache(G, D, block, [0, 0], total, page, "heads")
    n = sum(lengths)
    k, v = rand((n, G, D), dtype, 1), rand((n, G, D), dtype, 2)
    m3.m3_kv8_write(k.to(DEV), v.to(DEV), *cache.args(), ints([0, 0]), m3.Kv8Config(2, 45, total, G, G, D, block),
                    offsets=ints([0, 45, 45]), block_table=cache.table)
    for x, (c, s) in zip((k, v), cache.host):
        K.write(c, s, block, f64(x), 0, cache.pages(0))
    at = list(lengths)
    for turn, (T, kept) in enumerate([(1, 1), (1, 1), (5, 2), (3, 3), (7, 0), (1, 1)]):
        q = rand((2 * T, H, D), dtype, 10 + turn)
        k, v = (rand((2 * T, G, D), dtype, 30 + turn + i) * 2 ** turn for i in (0, 50))
        out = m3.m3_attn_step_kv8(q.to(DEV), k.to(DEV), v.to(DEV), *cache.args(), ints(at),
                                  m3.Kv8Config(2, T, total, H, G, D, block), block_table=cache.table)
        torch.cuda.synchronize()
        for b in range(2):
            rows = slice(b * T, b * T + T)
            for x, (c, s) in zip((k, v), cache.host):
                K.write(c, s, block, f64(x[rows]), at[b], cache.pages(b))
            kk, vv = (K.read(c, s, block, 0, at[b] + T, cache.pages(b)) for c, s in cache.host)
            ref, size = K.step(f64(q[rows]), kk, vv, K.visible(T, at[b], 0, 0), D ** -0.5)
            check(out[rows], ref, bound_of(f64(q[rows]), kk, vv, ref, size, D ** -0.5, dtype, at[b] + T), f"{turn} {b}")
        cache.same(f"turn {turn}")
        at = [x + kept for x in at]  # the rest of the drafts is taken back
    # a prompt goes on behind what the cache holds
    offsets = [0, at[0], at[0] + at[1]]
    held = m3.m3_kv8_read(*cache.args(), m3.Kv8Config(2, max(at), total, G, G, D, block), offsets=ints(offsets),
                          total=offsets[2], block_table=cache.table, dtype=dtype)
    q = rand((offsets[2], H, D), dtype, 90)
    o, _ = m3.m3_attn_fwd(q.to(DEV), held["k"], held["v"], m3.AttnConfig(2, max(at), max(at), H, G, D),
                          q_offsets=ints(offsets), kv_offsets=ints(offsets))
    torch.cuda.synchronize()
    for b in range(2):
        rows = slice(offsets[b], offsets[b + 1])
        kk, vv = (K.read(c, s, block, 0, at[b], cache.pages(b)) for c, s in cache.host)
        np.testing.assert_array_equal(f64(held["k"][rows]), kk)
        ref, size = K.step(f64(q[rows]), kk, vv, K.visible(at[b], 0, 0, 0), D ** -0.5)
        bound = bound_of(f64(q[rows]), kk, vv, ref, size, D ** -0.5, dtype, at[b])
        # m3_attn_fwd rounds its probabilities to the operands' type
        check(o[rows], ref, bound + half_step(dtype) * size, f"goes on {b}")


@pytest.mark.parametrize("name", ["bf16", "f32"])
def test_replayed_steps(name):
    """Steps from one graph, with the program's own work and synchronizations between the replays, against eager ones."""
    dtype, H, G, D, block, T = TYPES[name], 8, 2, 64, 16, 2
    caches = [Cache(G, D, block, [0, 30], 1024, 64, seed=3) for _ in range(2)]
    cfg = m3.Kv8Config(2, T, 1024, H, G, D, block, 700, 3)
    q, k, v = (torch.empty(2 * T, h, D, dtype=dtype, device=DEV) for h in (H, G, G))
    length, out = ints([0, 30]), torch.empty(2 * T, H, D, dtype=dtype, device=DEV)
    need = m3.attn_step_kv8_workspace_bytes(cfg, dtype)
    assert need > 0  # stretches and their join are part of the graph
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    for x in (q, k, v):
        x.normal_()
    m3.m3_attn_step_kv8(q, k, v, *Cache(G, D, block, [0, 30], 1024, 64, seed=3).args(), length, cfg,
                        block_table=caches[0].table)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m3.m3_attn_step_kv8(q, k, v, *caches[0].args(), length, cfg, block_table=caches[0].table, out=out, workspace=ws)
    for i in range(20):
        gen = torch.Generator(device=DEV).manual_seed(i)
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=gen, device=DEV) * 2 ** (i % 5))
        length.copy_(ints([T * i, 30 + T * i]))
        graph.replay()
        if i % 3 == 0:
            torch.cuda.synchronize()
        want = m3.m3_attn_step_kv8(q, k, v, *caches[1].args(), length, cfg, block_table=caches[1].table)
        ws.fill_(255 if i % 2 else 0)  # nothing is kept in the workspace
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        for a, b in zip(caches[0].args(), caches[1].args()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i


def test_other_streams_and_calls_at_once():
    """Calls on two streams of their own, each with its own cache, at the same time: as one after the other."""
    H, G, D, block, dtype = 8, 4, 128, 64, torch.bfloat16
    cfg = m3.Kv8Config(3, 1, 4096, H, G, D, block)
    runs = []
    for s in range(2):
        cache = Cache(G, D, block, [100, 60, 20], 4096, 256, seed=s)
        q, k, v = (rand((3, h, D), dtype, 7 * s + h).to(DEV) for h in (H, G, G))
        runs.append((cache, q, k, v, ints([100, 60, 20])))
    want = [m3.m3_attn_step_kv8(q, k, v, *(t.clone() for t in c.args()), at, cfg, block_table=c.table)
            for c, q, k, v, at in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = []
    for _ in range(3):
        for stream, (c, q, k, v, at) in zip(streams, runs):
            got.append(m3.m3_attn_step_kv8(q, k, v, *c.args(), at, cfg, block_table=c.table, stream=stream))
            m3.m3_kv8_read(*c.args(), m3.Kv8Config(3, 64, 4096, H, G, D, block), block_table=c.table, stream=stream)
    torch.cuda.synchronize()
    for i, x in enumerate(got):
        assert torch.equal(x, want[i % 2]), i


@pytest.mark.parametrize("name", list(TYPES))
def test_rows_do_not_depend_on_each_other(name):
    """A row's result and cache are the same bits with other rows, other tokens' queries and NaN beside it."""
    dtype, H, G, D, block = TYPES[name], 8, 2, 64, 16
    cache = Cache(G, D, block, [200, 333], 512, 64)
    cfg = m3.Kv8Config(2, 3, 512, H, G, D, block)
    q, k, v = (rand((6, h, D), dtype, h) for h in (H, G, G))
    first = m3.m3_attn_step_kv8(q.to(DEV), k.to(DEV), v.to(DEV), *(t.clone() for t in cache.args()), ints([200, 333]), cfg,
                                block_table=cache.table)
    other = [x.clone() for x in (q, k, v)]
    for x in other:
        x[3:] = float("nan")
    other[0][0] *= 100  # another query of the same row
    args = tuple(t.clone() for t in cache.args())
    second = m3.m3_attn_step_kv8(*(x.to(DEV) for x in other), *args, ints([200, 400]), cfg, block_table=cache.table)
    torch.cuda.synchronize()
    assert torch.equal(first[1:3], second[1:3]) and second[3:].isnan().all()
    for x, (c, s), (dc, ds) in zip((k, v), cache.host, (args[:2], args[2:])):
        K.write(c, s, block, f64(x[:3]), 200, cache.pages(0))
        for p in cache.pages(0):
            assert np.array_equal(dc[p].view(torch.uint8).cpu().numpy() % 128 == 127, c[p] % 128 == 127)
            assert np.array_equal(ds[p].view(torch.uint8).cpu().numpy(), s[p])


@pytest.mark.parametrize("name", list(TYPES))
def test_strided_views_of_a_step(name):
    """Queries, keys and values in one packed row, results into a wider buffer, bits as for rows of their own."""
    dtype, H, G, D, block, T = TYPES[name], 6, 3, 80, 32, 4
    row = rand((2 * T, (H + 2 * G) * D + 8), dtype, 5).to(DEV)
    q, k, v = (row[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, H), (H, H + G), (H + G, H + 2 * G)))
    caches = [Cache(G, D, block, [77, 3], 160, 32, how) for how in ("rows", "heads", "odd")]
    cfg = m3.Kv8Config(2, T, 160, H, G, D, block)
    want = m3.m3_attn_step_kv8(q.contiguous(), k.contiguous(), v.contiguous(), *caches[0].args(), ints([77, 3]), cfg,
                               block_table=caches[0].table)
    for wide, cache in ((8, caches[1]), (3, caches[2])):
        out = torch.full((2 * T, H, D + wide), 9.0, dtype=dtype, device=DEV)
        m3.m3_attn_step_kv8(q, k, v, *cache.args(), ints([77, 3]), cfg, block_table=cache.table, out=out[..., :D])
        torch.cuda.synchronize()
        assert torch.equal(out[..., :D], want) and (out[..., D:] == 9).all()
        for a, b in zip(cache.args(), caches[0].args()):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("name", list(TYPES))
def test_scale_and_extremes_of_a_step(name):
    """A scale of its own, down to one that leaves nothing of the scores; keys of all sizes; scores far apart."""
    dtype, H, G, D, block, n = TYPES[name], 2, 1, 64, 16, 150
    cache = Cache(G, D, block, [n - 1], 160, 0)
    sizes = 2.0 ** np.random.default_rng(1).integers(-12, 5, (n - 1, 1, 1))
    for c, s in cache.host:
        K.write(c, s, block, np.random.default_rng(2).standard_normal((n - 1, G, D)) * sizes, 0, [0])
    cache.dev = [(cache.place(c, "rows"), torch.from_numpy(s).to(DEV).view(torch.float8_e8m0fnu)) for c, s in cache.host]
    q, k, v = rand((1, H, D), dtype, 1), rand((1, G, D), dtype, 2), rand((1, G, D), dtype, 3)
    for x, (c, s) in zip((k, v), cache.host):
        K.write(c, s, block, f64(x), n - 1, [0])
    kk, vv = (K.read(c, s, block, 0, n, [0]) for c, s in cache.host)
    for scale in (1.0, 0.03, 1e-30, 1e-38):
        out = m3.m3_attn_step_kv8(q.to(DEV), k.to(DEV), v.to(DEV), *cache.args(), ints([n - 1]),
                                  m3.Kv8Config(1, 1, 160, H, G, D, block, scale=scale))
        torch.cuda.synchronize()
        ref, size = K.step(f64(q), kk, vv, np.ones((1, n), bool), np.float32(scale))
        S = scale * np.einsum("ihd,jgd->hij", np.abs(f64(q)), np.abs(kk)).max()
        rel = (D + 8) * 2.0 ** -24 * S + 2.0 ** -22 * S + 2.0 ** -21 + n * 2.0 ** -24
        bound = (PIECES[dtype] + 2 * rel) * size + half_step(dtype) * np.abs(ref) + (2.0 ** -25 if name == "f16" else 0)
        check(out, ref, bound, f"scale {scale}")


@pytest.mark.parametrize("name", list(TYPES))
def test_zero_scores_at_a_scale_that_passes_float32(name):
    """A zero query has equal scores, though the scale of the scores times a block's is beyond float32."""
    dtype, H, G, D, block, n = TYPES[name], 2, 1, 64, 16, 150
    cache = Cache(G, D, block, [n - 1], 160, 0)
    k = rand((1, G, D), dtype, 2) * 2 ** 14
    for c, s in cache.host:
        K.write(c, s, block, np.random.default_rng(2).standard_normal((n - 1, G, D)) * 2 ** 14, 0, [0])
    cache.dev = [(cache.place(c, "rows"), torch.from_numpy(s).to(DEV).view(torch.float8_e8m0fnu)) for c, s in cache.host]
    q, v = torch.zeros((1, H, D), dtype=dtype), rand((1, G, D), dtype, 3)
    for x, (c, s) in zip((k, v), cache.host):
        K.write(c, s, block, f64(x), n - 1, [0])
    kk, vv = (K.read(c, s, block, 0, n, [0]) for c, s in cache.host)
    for window in (0, 70):
        out = m3.m3_attn_step_kv8(q.to(DEV), k.to(DEV), v.to(DEV), *cache.args(), ints([n - 1]),
                                  m3.Kv8Config(1, 1, 160, H, G, D, block, window, scale=1e38))
        torch.cuda.synchronize()
        ref, size = K.step(f64(q), kk, vv, K.visible(1, n - 1, window, 0), 1e38)
        check(out, ref, bound_of(f64(q), kk, vv, ref, size, 1e38, dtype, n), f"window {window}")


def test_example_serves_from_8_bits():
    import attention_layer as example

    layer = example.AttentionLayer(7)
    held, diff, size = example.serve_8bit(layer)
    # bfloat16 rows: half a step for the roundings of P, of the layer's inner result and of its output, on both sides; and
    # the blocks that the last tokens made coarser after earlier ones had read them: e4m3's half step, at most
    assert held <= (2 * 3 * 2.0 ** -8 + 2.0 ** -4) * size
    assert diff < size
