"""Attention where a few blocks of queries are shared by several workgroups along the keys: the joined
results against the float64 oracle with the bounds of the unsplit ones (a join is one more rescaling of
the running sums, which the bounds count for every key)."""

import pytest
import torch

import selective_state_space_mamba3_amd as m3
import test_gpu_attn as base

pytestmark = pytest.mark.gpu

# sequences as (queries, keys), heads, groups, dim, causal, window, layout
CASES = [
    ([(300, 2000), (40, 900), (0, 5), (7, 0), (129, 129)], 2, 1, 64, True, 700, "plain"),
    ([(257, 1500)], 2, 2, 128, True, 0, "packed"),
    ([(5, 1200)], 3, 1, 40, False, 0, "odd"),
    ([(1, 4096)], 4, 1, 128, True, 0, "heads first"),
    ([(130, 700), (260, 700)], 1, 1, 80, True, 0, "plain"),
    ([(900, 513)], 2, 1, 32, True, 0, "plain"),
]


@pytest.mark.parametrize("case", CASES, ids=base.case_id)
@pytest.mark.parametrize("name", list(base.TYPES))
def test_forward_and_backward(case, name):
    pr = base.Problem(case, base.TYPES[name])
    assert m3.attn_fwd_workspace_bytes(pr.cfg, pr.dtype) > 0  # the keys are shared
    base.test_forward_and_backward(case, name)


@pytest.mark.parametrize("name", list(base.TYPES))
def test_rows_of_no_sequence_are_left_alone(name):
    """Rows before, between and behind the sequences keep what they held, in every output."""
    dtype, H, G, D = base.TYPES[name], 2, 1, 64
    q, k, v, g = (base.rand((n, h, D), dtype, i).to(base.DEV) for i, (n, h) in enumerate(
        [(220, H), (1700, G), (1700, G), (220, H)]))
    cq, ck = torch.tensor([20, 20, 190], dtype=torch.int32), torch.tensor([30, 30, 1600], dtype=torch.int32)
    cfg = m3.AttnConfig(2, 170, 1570, H, G, D)
    offsets = dict(q_offsets=cq.to(base.DEV), kv_offsets=ck.to(base.DEV))
    out, lse = torch.full_like(q, 7), torch.full((220, H), 7.0, device=base.DEV)
    m3.m3_attn_fwd(q, k, v, cfg, **offsets, out=out, lse=lse)
    grads = {"q": torch.full_like(q, 7), "k": torch.full_like(k, 7), "v": torch.full_like(v, 7)}
    m3.m3_attn_bwd(g, q, k, v, out, lse, cfg, **offsets, grads=grads)
    alone, alone_lse = m3.m3_attn_fwd(q[20:190], k[30:1600], v[30:1600], m3.AttnConfig(1, 170, 1570, H, G, D))
    torch.cuda.synchronize()
    for t, lo, hi in ((out, 20, 190), (lse, 20, 190), (grads["q"], 20, 190), (grads["k"], 30, 1600),
                      (grads["v"], 30, 1600)):
        assert (t[:lo] == 7).all() and (t[hi:] == 7).all() and not (t[lo:hi] == 7).all()
    # another number of workgroups may share the keys: both sides carry the bounds' rounding of P and of the result
    size = float(v.abs().max())
    assert float((out[20:190].double() - alone.double()).abs().max()) <= (4 * base.unit(dtype) + 2.0 ** -17) * size
    assert float((lse[20:190] - alone_lse).abs().max()) <= 2.0 ** -17 * float(alone_lse.abs().max())


@pytest.mark.parametrize("name", list(base.TYPES))
def test_hidden_infinities_stay_hidden(name):
    dtype = base.TYPES[name]
    pr = base.Problem(([(200, 1400)], 2, 1, 64, True, 0, "plain"), dtype)
    assert m3.attn_fwd_workspace_bytes(pr.cfg, dtype) > 0
    q, k, v, _ = pr.dev
    out, lse = m3.m3_attn_fwd(q, k, v, pr.cfg)
    k2, v2 = k.clone(), v.clone()
    v2[1300, 0, 5] = float("nan")
    v2[1301, 0, 6] = float("inf")
    k2[1302] = float("nan")
    out2, lse2 = m3.m3_attn_fwd(q, k2, v2, pr.cfg)
    torch.cuda.synchronize()
    assert torch.equal(out2[:100], out[:100]) and torch.equal(lse2[:100], lse[:100])
    assert out2[100, :, 5].isnan().all() and not out2[101, :, 6].isfinite().any() and out2[102:].isnan().all()
    assert out2[100, :, :5].isfinite().all() and out2[100, :, 6:].isfinite().all()


def test_workspace_is_asked_for():
    cfg = m3.AttnConfig(1, 64, 4096, 2, 1, 64)
    q, k = torch.zeros(64, 2, 64, device=base.DEV), torch.zeros(4096, 1, 64, device=base.DEV)
    small = torch.empty(m3.attn_fwd_workspace_bytes(cfg, q.dtype) - 16, dtype=torch.uint8, device=base.DEV)
    with pytest.raises(m3.M3Error, match="workspace of"):
        m3.m3_attn_fwd(q, k, k, cfg, workspace=small)
