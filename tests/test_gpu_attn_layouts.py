"""Outputs and caches in every order of their axes that leaves rows, heads and pages apart: the same bits as contiguous ones."""

import pytest
import torch

import selective_state_space_mamba3_amd as m3
import test_gpu_attn as base

pytestmark = pytest.mark.gpu


def ordered(t, order, pad=0):
    """The values of t with its axes but the last in this order in memory, `pad` elements behind each run of the last."""
    shape = [t.shape[i] for i in order] + [t.shape[-1] + pad]
    inverse = [order.index(i) for i in range(len(order))]
    view = torch.full(shape, 7.0, dtype=t.dtype, device=t.device)[..., :t.shape[-1]].permute(*inverse, len(order))
    view.copy_(t)
    return view


@pytest.mark.parametrize("order", [(0, 1, 2), (0, 2, 1), (1, 0, 2), (2, 0, 1), (1, 2, 0), (2, 1, 0)], ids=str)
@pytest.mark.parametrize("pad", [0, 8, 3])
@pytest.mark.parametrize("page", [0, 16])
def test_caches(order, pad, page):
    G, D, capacity, n = 2, 64, 96, 3
    dtype = torch.bfloat16
    size = page or capacity
    pages = n * (capacity // size)
    kc, vc = (base.rand((pages * size, G, D), dtype, i).view(pages, size, G, D).to(base.DEV) for i in (1, 2))
    q, k, v = (base.rand((n, h, D), dtype, 3 + h).to(base.DEV) for h in (4, G, G + 1))
    v = v[:, :G].contiguous()
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(0)).to(torch.int32).view(n, -1).to(base.DEV)
    lengths = torch.tensor([95, 40, 0], dtype=torch.int32, device=base.DEV)
    cfg = m3.AttnConfig(n, 1, capacity, 4, G, D)
    results = []
    for layout in (lambda t: t.clone(), lambda t: ordered(t, order, pad)):
        a, b = layout(kc), layout(vc)
        out = m3.m3_attn_step(q, k, v, a, b, lengths, cfg, block_table=table if page else None)
        results.append((out, a, b))
    torch.cuda.synchronize()
    for x, y in zip(*results):
        assert torch.equal(x, y)


def test_interleaved_outputs():
    """Heads two places apart and rows five: rows 0 and 1 pass between one another."""
    q, k, v, g = (base.rand((n, h, 64), torch.float16, i).to(base.DEV) for i, (n, h) in enumerate(
        [(2, 6), (9, 1), (9, 1), (2, 6)]))
    cfg = m3.AttnConfig(1, 2, 9, 6, 1, 64)
    want, lse = m3.m3_attn_fwd(q, k, v, cfg)
    grads = m3.m3_attn_bwd(g, q, k, v, want, lse, cfg)
    outs = [torch.full((20 * 64,), 7.0, dtype=q.dtype, device=base.DEV) for _ in range(2)]
    out, dq = (o.as_strided((2, 6, 64), (5 * 64, 2 * 64, 1)) for o in outs)
    m3.m3_attn_fwd(q, k, v, cfg, out=out)
    m3.m3_attn_bwd(g, q, k, v, want, lse, cfg, grads={"q": dq})
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(dq, grads["q"])
    used = {5 * r + 2 * h for r in range(2) for h in range(6)}
    for o in outs:
        assert all((o.view(20, 64)[i] == 7).all() for i in range(20) if i not in used)
