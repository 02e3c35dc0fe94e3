"""The single-token step over dense and paged caches against the float64 oracle (bounds as in test_gpu_attn)."""

import numpy as np
import pytest
import torch

import selective_state_space_mamba3_amd as m3
from oracle import attention as A
from test_gpu_attn import DEV, TYPES, check, f64, half_step, rand, tiny, unit

pytestmark = pytest.mark.gpu

# heads, groups, dim, cached lengths, capacity, page (0: dense), window
CASES = [
    (1, 1, 1, [0], 1, 0, 0),
    (2, 1, 16, [0, 1, 31, 32, 33], 40, 0, 0),
    (24, 8, 64, [127, 128, 129, 500], 512, 0, 0),
    (8, 1, 128, [700, 3, -1, 899, 900, 1000], 900, 48, 0),
    (6, 2, 80, [255, 64, 17], 256, 64, 60),
    (5, 5, 40, [100, 90], 101, 1, 1),
    (40, 1, 64, [300, 17], 320, 16, 0),
    (3, 3, 7, [50, 20, 77], 78, 3, 20),
    (32, 4, 128, [9000], 9216, 256, 0),
    (4, 2, 100, [2000, 5], 2048, 0, 129),
    (4, 4, 64, [5000], 5120, 0, 0),
]


class Cache:
    def __init__(self, G, D, lengths, capacity, page, dtype, seed=0, combined=False):
        n = len(lengths)
        self.page = page or capacity
        self.per = -(-capacity // self.page)
        pages = n * self.per + 2
        both = torch.full((pages, 2, self.page, G, D), float("nan"), dtype=dtype)
        g = torch.Generator().manual_seed(seed)
        self.table = torch.randperm(pages, generator=g)[:n * self.per].to(torch.int32).view(n, self.per)
        if not page:
            self.table = torch.arange(n, dtype=torch.int32)[:, None]
        for b, length in enumerate(lengths):
            for j in range(max(0, min(length, capacity))):  # what lies past the length stays NaN
                both[self.table[b, j // self.page], :, j % self.page] = torch.randn(2, G, D, generator=g).to(dtype)
        dev = both.to(DEV)
        self.k, self.v = dev[:, 0], dev[:, 1]  # strided: keys and values share pages
        if not combined:
            self.k, self.v = self.k.contiguous(), self.v.contiguous()

    def rows(self, t, b, n):
        t = t.cpu()
        return torch.stack([t[self.table[b, j // self.page], j % self.page] for j in range(n)])


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("name", list(TYPES))
def test_step(case, name):
    H, G, D, lengths, capacity, page, window = case
    dtype, n, share = TYPES[name], len(lengths), H // G
    cache = Cache(G, D, lengths, capacity, page, dtype, combined=H == 8)
    before = cache.k.cpu(), cache.v.cpu()
    q, k, v = rand((n, H, D), dtype, 1), rand((n, G, D), dtype, 2), rand((n, G, D), dtype, 3)
    cfg = m3.AttnConfig(n, 1, capacity, H, G, D, window=window)
    out = m3.m3_attn_step(q.to(DEV), k.to(DEV), v.to(DEV), cache.k, cache.v,
                          torch.tensor(lengths, dtype=torch.int32, device=DEV), cfg,
                          block_table=cache.table.to(DEV) if page else None)
    torch.cuda.synchronize()
    u, w, scale = unit(dtype), half_step(dtype), D ** -0.5
    changed = torch.zeros(before[0].shape[:2], dtype=torch.bool)
    for b, length in enumerate(lengths):
        if not 0 <= length < capacity:
            assert (out[b] == 0).all()
            continue
        at = int(cache.table[b, length // cache.page]), length % cache.page
        assert torch.equal(cache.k[at].cpu(), k[b]) and torch.equal(cache.v[at].cpu(), v[b])
        changed[at] = True
        kk, vv = (f64(cache.rows(t, b, length + 1)) for t in (cache.k, cache.v))
        ref, _ = A.attention(f64(q[b:b + 1]), kk, vv, True, window)
        p, _ = A.probabilities(f64(q[b:b + 1]), kk, True, window, scale)
        av = np.einsum("hij,jhd->ihd", p, np.abs(np.repeat(vv, share, 1)))
        big = scale * np.einsum("ihd,jhd->hij", np.abs(f64(q[b:b + 1])), np.abs(np.repeat(kk, share, 1))).max()
        rel = (D + 8) * 2.0 ** -24 * big + 2.0 ** -22 * big + 2.0 ** -21 + (length + 1) * 2.0 ** -24
        bound = (u + 2 * rel) * av + w * np.abs(ref) + tiny(dtype) * (np.abs(vv).sum(0).repeat(share, 0)[None] + 1)
        check(out[b:b + 1], ref, bound, f"row {b} length {length}")
    for now, old in zip((cache.k.cpu(), cache.v.cpu()), before):  # nothing else was written
        bits = torch.int32 if dtype == torch.float32 else torch.int16
        assert torch.equal(now.view(bits)[~changed], old.view(bits)[~changed])


@pytest.mark.parametrize("name", list(TYPES))
def test_bad_pages_are_left_alone(name):
    """Entries outside the pages hide their positions; the token of such a page is attended to, not stored."""
    dtype, G, D, page = TYPES[name], 2, 64, 16
    lengths = [70, 40, 33]
    cache = Cache(G, D, lengths, 96, page, dtype)
    table = cache.table.clone()
    table[0, 1], table[1, 2], table[2, 0] = -1, 1 << 30, -(1 << 31)
    q, k, v = rand((3, 4, D), dtype, 1), rand((3, G, D), dtype, 2), rand((3, G, D), dtype, 3)
    cfg = m3.AttnConfig(3, 1, 96, 4, G, D)
    out = m3.m3_attn_step(q.to(DEV), k.to(DEV), v.to(DEV), cache.k, cache.v,
                          torch.tensor(lengths, dtype=torch.int32, device=DEV), cfg, block_table=table.to(DEV))
    torch.cuda.synchronize()
    for b, length in enumerate(lengths):
        keep = [j for j in range(length) if 0 <= table[b, j // page] < cache.k.shape[0]]
        old = [torch.stack([t[cache.table[b, j // page], j % page] for j in keep]) for t in (cache.k.cpu(), cache.v.cpu())]
        kk, vv = (f64(torch.cat([o, t[b:b + 1]])) for o, t in zip(old, (k, v)))
        ref, _ = A.attention(f64(q[b:b + 1]), kk, vv, True)
        bound = (2 * unit(dtype) + 2.0 ** -17) * np.abs(vv).max() + half_step(dtype) * np.abs(ref)
        check(out[b:b + 1], ref, bound, f"row {b}")


def test_cache_beyond_32_bits():
    """Pages whose elements lie past 2^32."""
    G, D, page = 8, 128, 64
    pages = 2 ** 32 // (G * D * page) + 8
    kc = torch.empty((pages, page, G, D), dtype=torch.bfloat16, device=DEV)
    vc = torch.empty_like(kc)
    use = [pages - 1, 0, pages - 3]
    for i, p in enumerate(use):
        kc[p] = rand((page, G, D), torch.bfloat16, i).to(DEV)
        vc[p] = rand((page, G, D), torch.bfloat16, 7 + i).to(DEV)
    q, k, v = (rand((1, h, D), torch.bfloat16, 20 + h) for h in (16, G, G + 8))
    v = v[:, :G].contiguous()
    cfg = m3.AttnConfig(1, 1, 3 * page, 16, G, D)
    out = m3.m3_attn_step(q.to(DEV), k.to(DEV), v.to(DEV), kc, vc, torch.tensor([2 * page + 20], dtype=torch.int32,
                          device=DEV), cfg, block_table=torch.tensor([use], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    n = 2 * page + 21
    kk, vv = (f64(torch.cat([t[p].cpu() for p in use])[:n]) for t in (kc, vc))
    assert torch.equal(kc[use[2], 20].cpu(), k[0]) and torch.equal(vc[use[2], 20].cpu(), v[0])
    ref, _ = A.attention(f64(q), kk, vv, True)
    check(out, ref, 2.0 ** -8 * (np.abs(vv).max() + np.abs(ref)), "far pages")


@pytest.mark.parametrize("name", ["bf16", "f32"])
def test_replayed_decode_matches_the_prompt_pass(name):
    """Decoding token by token from a graph gives the rows of one causal pass over the whole sequence."""
    dtype, H, G, D, n = TYPES[name], 6, 2, 64, 37
    q, k, v = rand((n, H, D), dtype, 1).to(DEV), rand((n, G, D), dtype, 2).to(DEV), rand((n, G, D), dtype, 3).to(DEV)
    whole, _ = m3.m3_attn_fwd(q, k, v, m3.AttnConfig(1, n, n, H, G, D))
    cfg = m3.AttnConfig(1, 1, 48, H, G, D)
    kc, vc = (torch.full((3, 16, G, D), float("nan"), dtype=dtype, device=DEV) for _ in range(2))
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    length = torch.zeros(1, dtype=torch.int32, device=DEV)
    tq, tk, tv = torch.empty_like(q[:1]), torch.empty_like(k[:1]), torch.empty_like(v[:1])
    out = torch.empty_like(tq)
    ws = torch.empty(max(1, m3.attn_step_workspace_bytes(cfg, dtype)), dtype=torch.uint8, device=DEV)
    # made before the graph: loading a kernel's code is not part of a capture
    m3.m3_attn_step(k[:1].repeat(1, H // G, 1), k[:1], v[:1], kc.clone(), vc.clone(), length, cfg, block_table=table)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m3.m3_attn_step(tq, tk, tv, kc, vc, length, cfg, block_table=table, out=out, workspace=ws)
    size = float(v.abs().max())
    for i in range(n):
        tq.copy_(q[i:i + 1])
        tk.copy_(k[i:i + 1])
        tv.copy_(v[i:i + 1])
        length.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        # both sides carry the rounding of P and of the result
        worst = float((out.double() - whole[i:i + 1].double()).abs().max())
        assert worst <= (4 * unit(dtype) + 2.0 ** -17) * size, (i, worst)
