"""Queries that hold an infinity: no score of theirs is finite, and where all are minus infinity they are not those of
hidden keys.  Their rows are NaN wherever they see a key, zero where they see none, and no other row changes."""

import pytest
import torch

import selective_state_space_mamba3_amd as m3
from test_gpu_attn import DEV, TYPES, rand

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("lengths", [([40, 1, 300], [40, 1, 300]), ([70], [2900]), ([9, 33], [5, 400])], ids=str)
@pytest.mark.parametrize("dim", [64, 80, 128])
@pytest.mark.parametrize("name", list(TYPES))
def test_forward(name, dim, lengths):
    """Whole sequences, keys shared by several workgroups, and queries before the first key."""
    dtype, H, G = TYPES[name], 4, 2
    lq, lk = lengths
    at = [[sum(x[:i]) for i in range(len(x) + 1)] for x in lengths]
    k, v = (rand((sum(lk), G, dim), torch.float32, s).abs().add(0.5).to(dtype).to(DEV) for s in (1, 2))
    q = rand((sum(lq), H, dim), dtype, 3)
    cfg = m3.AttnConfig(len(lq), max(lq), max(lk), H, G, dim)
    cut = dict(q_offsets=ints(at[0]), kv_offsets=ints(at[1]))
    want, want_lse = m3.m3_attn_fwd(q.to(DEV), k, v, cfg, **cut)
    bad = q.clone()
    bad[:, 1] = 0
    bad[:, 1, 7] = -float("inf")
    bad[::3, 2, dim - 1] = float("inf")
    out, lse = m3.m3_attn_fwd(bad.to(DEV), k, v, cfg, **cut)
    torch.cuda.synchronize()
    sees = torch.cat([torch.arange(a) >= a - b for a, b in zip(lq, lk)])
    spoilt = torch.zeros(q.shape[:2], dtype=torch.bool)
    spoilt[:, 1] = sees
    spoilt[::3, 2] = sees[::3]
    assert torch.equal(out.isnan().all(-1).cpu(), spoilt) and torch.equal(out.isnan().any(-1).cpu(), spoilt)
    same = ~spoilt
    same[:, 1] = same[::3, 2] = False
    assert torch.equal(out.cpu()[same], want.cpu()[same]) and torch.equal(lse.cpu()[same], want_lse.cpu()[same])
    assert (out.cpu()[~sees] == 0).all() and (lse.cpu()[~sees] == -float("inf")).all()
    assert lse.cpu()[spoilt].isnan().all()


@pytest.mark.parametrize("capacity", [64, 8192])
@pytest.mark.parametrize("name", list(TYPES))
def test_step(name, capacity):
    dtype, H, G, dim = TYPES[name], 4, 2, 64
    lengths = [0, 1, 33, capacity - 1, -1]
    kc, vc = (rand((5, capacity, G, dim), torch.float32, s).abs().add(0.5).to(dtype).to(DEV) for s in (1, 2))
    k, v = (rand((5, G, dim), torch.float32, s).abs().add(0.5).to(dtype).to(DEV) for s in (4, 5))
    q = rand((5, H, dim), dtype, 3)
    cfg = m3.AttnConfig(5, 1, capacity, H, G, dim)
    want = m3.m3_attn_step(q.to(DEV), k, v, kc, vc, ints(lengths), cfg)
    q[:, 1] = 0
    q[:, 1, 7] = -float("inf")
    out = m3.m3_attn_step(q.to(DEV), k, v, kc, vc, ints(lengths), cfg)
    torch.cuda.synchronize()
    assert out[:4, 1].isnan().all() and (out[4] == 0).all()
    for h in (0, 2, 3):
        assert torch.equal(out[:, h], want[:, h])
