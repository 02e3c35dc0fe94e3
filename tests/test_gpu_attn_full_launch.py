"""Attention where the blocks of queries alone fill the compute units, as at training sizes: two blocks of
queries to a wave (16-bit heads up to 64), each workgroup with all keys of its queries and each gradient stored
directly.  Oracle and bounds are those of test_gpu_attn."""

import pytest
import torch

import selective_state_space_mamba3_amd as m3
import test_gpu_attn as base

pytestmark = pytest.mark.gpu

# sequences as (queries, keys), heads, groups, dim, causal, window, layout
CASES = [
    ([(n, n) for n in (256, 129, 1, 64, 65, 33, 31, 128, 3, 96, 17)], 24, 8, 64, True, 0, "plain"),
    ([(257, 300), (130, 120), (1, 9), (90, 60), (64, 0), (33, 40)], 24, 8, 40, True, 65, "odd"),
    ([(n, n + 60) for n in (256, 70, 1, 130, 97, 31)] + [(5, 5)] * 16, 12, 4, 64, True, 33, "packed"),
    ([(100, 170)] * 16, 16, 16, 32, False, 0, "packed"),
    ([(700, 700), (300, 900), (260, 100)] + [(3, 7)] * 19, 4, 1, 64, True, 0, "heads first"),
    ([(290, 520), (300, 290)] + [(9, 33)] * 14, 8, 2, 56, False, 0, "odd"),
    ([(129, 400), (256, 256), (140, 530)] + [(20, 40)] * 21, 4, 1, 128, True, 0, "plain"),
    ([(129, 290), (256, 200), (140, 140)] + [(11, 9)] * 21, 4, 4, 80, True, 65, "odd"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: base.case_id((c[0][:3], *c[1:])) + f"-{len(c[0])}")
@pytest.mark.parametrize("name", list(base.TYPES))
def test_forward_and_backward(case, name):
    pr = base.Problem(case, base.TYPES[name])
    assert m3.attn_fwd_workspace_bytes(pr.cfg, pr.dtype) == 0  # no keys are shared
    pairs = len(case[0]) * case[1]
    longest = max(s[0] for s in case[0])
    assert -(-longest // 128) * pairs >= 192 and (case[3] > 64 or -(-longest // 256) * pairs >= 256)
    base.test_forward_and_backward(case, name)


@pytest.mark.parametrize("name", list(base.TYPES))
@pytest.mark.parametrize("window", [0, 50])
def test_hidden_infinities_stay_hidden(name, window):
    pr = base.Problem(([(150, 150), (90, 90)] * 6, 24, 8, 64, True, window, "plain"), base.TYPES[name])
    q, k, v, _ = pr.dev
    out, lse = m3.m3_attn_fwd(q, k, v, pr.cfg, **pr.offsets)
    k2, v2 = k.clone(), v.clone()
    v2[100, 0, 5] = float("nan")
    v2[101, 0, 6] = float("inf")
    k2[102] = float("nan")
    v2[150 + 40] = float("inf")
    out2, lse2 = m3.m3_attn_fwd(q, k2, v2, pr.cfg, **pr.offsets)
    torch.cuda.synchronize()
    row = torch.arange(q.shape[0], device=base.DEV)
    at = torch.where(row < 150, row, row - 150)
    reach = window or 1000
    touched = torch.where(row < 150, (at >= 100) & (at < 102 + reach), (at >= 40) & (at < 40 + reach)) & (row < 240)
    assert torch.equal(out2[~touched], out[~touched]) and torch.equal(lse2[~touched], lse[~touched])
    assert out2[100, :3, 5].isnan().all() and out2[101, :3, 6].isfinite().logical_not().all()
    assert out2[102:min(102 + reach, 150)].isnan().all()
    assert out2[100, :, :5].isfinite().all() and out2[100, :, 6:].isfinite().all() and out2[100, 3:].isfinite().all()
    assert not out2[150 + 40].isfinite().any()


@pytest.mark.parametrize("case", [([(70, 130)], 4, 2, 64, True, 0, "plain"), CASES[0]], ids=["few", "full"])
@pytest.mark.parametrize("name", list(base.TYPES))
def test_scale(case, name):
    """A scale of its own: the same as queries 2.4 times as long."""
    pr = base.Problem(case, base.TYPES[name])
    factor = 2.4
    scale = factor * pr.q.shape[2] ** -0.5
    q, k, v, g = pr.dev
    cfg = m3.AttnConfig(**{f: getattr(pr.cfg, f) for f in pr.cfg.__dataclass_fields__} | {"scale": scale})
    out, lse = m3.m3_attn_fwd(q, k, v, cfg, **pr.offsets)
    grads = m3.m3_attn_bwd(g, q, k, v, out, lse, cfg, **pr.offsets)
    torch.cuda.synchronize()
    pr.q = pr.q.double() * factor
    ref, bound = pr.reference()
    base.check(out, ref[0], bound[0], "out")
    base.check(lse, ref[1], bound[1] + 2.0 ** -23 * abs(ref[1]), "lse")
    base.check(grads["q"], ref[2] * factor, bound[2] * factor, "dq")
    base.check(grads["k"], ref[3], bound[3], "dk")
    base.check(grads["v"], ref[4], bound[4], "dv")


@pytest.mark.parametrize("name", list(base.TYPES))
def test_scale_of_a_step(name):
    """Twice the scale and half the query: the same bits."""
    dtype = base.TYPES[name]
    q, k, v = (base.rand((3, h, 64), dtype, h).to(base.DEV) for h in (8, 2, 2))
    kc, vc = (base.rand((3 * 700, 2, 64), dtype, i).view(3, 700, 2, 64).to(base.DEV) for i in (5, 6))
    lengths = torch.tensor([699, 300, 0], dtype=torch.int32, device=base.DEV)
    want = m3.m3_attn_step(q, k, v, kc.clone(), vc.clone(), lengths, m3.AttnConfig(3, 1, 700, 8, 2, 64))
    got = m3.m3_attn_step(q / 2, k, v, kc, vc, lengths, m3.AttnConfig(3, 1, 700, 8, 2, 64, scale=0.25))
    torch.cuda.synchronize()
    assert torch.equal(got, want)
