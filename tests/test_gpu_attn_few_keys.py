"""Gradients of queries that see few keys, where dS = P (dP - delta) is small beside P dP, so that the rounding of
the out that delta is made of weighs more than dS's own.  Up to 32 keys a query's delta is made in float32, whatever
the lengths of the other sequences, the window or the tile that the query stands in.

The bounds are those of test_gpu_attn without the rounding of out in delta: with pe = 2 rel + 2^-22 (|lse| + 1)
for a probability made from the scores and lse, delta is off by at most
    pe sum_j p |dp| + (D + 8 + n) 2^-24 sum_j p (|do| . |v|)."""

import numpy as np
import pytest
import torch

import selective_state_space_mamba3_amd as m3
import test_gpu_attn as base
from oracle import attention as A

pytestmark = pytest.mark.gpu

FEW = 32
# sequences as (queries, keys), heads, groups, dim, causal, window, layout
CASES = [
    ([(700, 700)], 3, 1, 64, True, 0, "plain"),
    ([(600, 900)], 2, 2, 64, True, 1, "packed"),
    ([(300, 1100), (1, 1), (2, 2), (33, 33), (20, 7)], 4, 2, 40, True, 0, "odd"),
    ([(200, 600), (140, 140)], 2, 1, 128, True, 9, "plain"),
    ([(150, 800), (64, 64)], 2, 1, 16, True, 32, "heads first"),
    ([(90, 1)], 2, 1, 64, False, 0, "plain"),
    ([(40, 32), (530, 3), (5, 1)], 2, 1, 96, False, 0, "plain"),
    ([(513, 520)], 8, 2, 80, True, 0, "plain"),
]


@pytest.mark.parametrize("case", CASES, ids=base.case_id)
@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_queries_of_few_keys(case, name):
    dtype = base.TYPES[name]
    pr = base.Problem(case, dtype)
    q, k, v, g = pr.dev
    out, lse = m3.m3_attn_fwd(q, k, v, pr.cfg, **pr.offsets)
    grads = m3.m3_attn_bwd(g, q, k, v, out, lse, pr.cfg, **pr.offsets)
    torch.cuda.synchronize()
    D, share = q.shape[2], q.shape[1] // k.shape[1]
    scale, u, w, t0 = D ** -0.5, base.unit(dtype), base.half_step(dtype), base.tiny(dtype)
    rows = 0
    for s, t, q64, k64, v64, g64 in pr.sequences():
        seen = A.allowed(len(q64), len(k64), pr.causal, pr.window).sum(-1)
        few = (seen > 0) & (seen <= FEW)
        rows += few.sum()
        dq, dk, _ = A.attention_backward(g64, q64, k64, v64, pr.causal, pr.window)
        p, lse64 = A.probabilities(q64, k64, pr.causal, pr.window, scale)
        kk, vv = np.repeat(k64, share, 1), np.repeat(v64, share, 1)
        big = scale * np.einsum("ihd,jhd->hij", np.abs(q64), np.abs(kk)).max()
        rel = (D + 8) * 2.0 ** -24 * big + 2.0 ** -22 * big + 2.0 ** -21 + FEW * 2.0 ** -24
        pe = (2 * rel + 2.0 ** -22 * (np.abs(np.where(np.isfinite(lse64), lse64, 0)) + 1)).T[..., None]
        dp = np.einsum("ihd,jhd->hij", g64, vv)
        adp = np.einsum("ihd,jhd->hij", np.abs(g64), np.abs(vv))
        ds = np.abs(p * (dp - (p * dp).sum(-1, keepdims=True)))
        d_err = pe * (p * np.abs(dp)).sum(-1, keepdims=True) + (D + 8 + FEW) * 2.0 ** -24 * (p * adp).sum(-1, keepdims=True)
        ds_err = (u + pe) * ds + p * (d_err + (D + 8) * 2.0 ** -24 * adp) + t0 * (p > 0)
        bound = scale * np.einsum("hij,jhd->ihd", ds_err + FEW * 2.0 ** -24 * ds, np.abs(kk)) + w * np.abs(dq) + t0
        base.check(grads["q"][s][torch.from_numpy(few)], dq[few], bound[few], "dq")
        if few[seen > 0].all():
            n_sum = len(q64) * share * 2.0 ** -24
            each = np.einsum("hij,ihd->jhd", ds_err + n_sum * ds, np.abs(q64))
            bound = scale * each.reshape(len(k64), -1, share, D).sum(2) + w * np.abs(dk) + t0
            base.check(grads["k"][t], dk, bound, "dk")
    assert rows


@pytest.mark.parametrize("name", list(base.TYPES))
@pytest.mark.parametrize("length", [5, 33, 100, 512])
def test_other_sequences_do_not_matter(name, length):
    """A sequence's gradients are the same bits alone and beside a longer one (24 heads: no key is shared by workgroups)."""
    dtype, H, G, D, other = base.TYPES[name], 24, 24, 64, 700
    n = length + other
    q, k, v, g = (base.rand((n, H, D), dtype, i).to(base.DEV) for i in range(4))
    both = torch.tensor([0, length, n], dtype=torch.int32, device=base.DEV)
    cfg = m3.AttnConfig(2, other, other, H, G, D)
    out, lse = m3.m3_attn_fwd(q, k, v, cfg, q_offsets=both, kv_offsets=both)
    # the sequence many times over, so that this launch shares no keys either
    many = 16
    reps = [x[:length].repeat(many, 1, 1) for x in (g, q, k, v, out)]
    alone = m3.m3_attn_bwd(*reps, lse[:length].repeat(many, 1), m3.AttnConfig(many, length, length, H, G, D))
    beside = m3.m3_attn_bwd(g, q, k, v, out, lse, cfg, q_offsets=both, kv_offsets=both)
    torch.cuda.synchronize()
    assert torch.equal(alone["q"][:length], beside["q"][:length])
    if length <= 128:  # one workgroup makes a block's key gradients in both
        for n_ in "kv":
            assert torch.equal(alone[n_][:length], beside[n_][:length])
