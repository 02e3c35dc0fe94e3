"""Per-head norm and rotation, forward and backward, against the float64 oracle.

One rounding of each result (half a step of its type) and float32 in between: a mean of D squares, a root
and a reciprocal, the turn's two products, so (D + 16) 2^-24 of the magnitudes that enter a result."""

import numpy as np
import pytest
import torch

import selective_state_space_mamba3_amd as m3
from oracle import attention as A
from test_gpu_attn import DEV, TYPES, check, f64, half_step, layout, rand, tiny

pytestmark = pytest.mark.gpu

# rows, heads, groups, dim, angles, layout
CASES = [
    (1, 1, 1, 1, 0, "plain"), (1, 2, 1, 2, 1, "odd"), (3, 4, 2, 64, 32, "plain"), (130, 24, 8, 64, 32, "packed"),
    (65, 6, 3, 80, 24, "heads first"), (17, 32, 4, 128, 64, "packed"), (9, 5, 5, 7, 3, "odd"), (33, 3, 1, 100, 10, "plain"),
    (40, 2, 2, 128, 0, "plain"), (21, 3, 1, 40, 8, "odd"), (1300, 2, 1, 16, 8, "plain"), (12, 70, 70, 96, 48, "plain"),
]


def inputs(case, dtype):
    rows, H, G, D, a, how = case
    q, k, gq, gk = (rand((rows, h, D), dtype, i) for i, h in enumerate((H, G, H, G)))
    at = (torch.arange(rows) * 977 % 65536).to(torch.int32)
    freq = 10000.0 ** (-torch.arange(a, dtype=torch.float32) / max(a, 1))
    qw, kw = 1 + 0.1 * rand((D,), torch.float32, 8), 1 + 0.1 * rand((D,), torch.float32, 9)
    cfg = m3.QkNormRopeConfig(H, G, D, a, 1e-5)
    dev = [layout(t, how) for t in (q, k, gq, gk)]
    return (q, k, gq, gk), dev, at, freq, (qw, kw), cfg


def swap(x, a):
    """Each column plus its partner: the magnitudes that a turned result is made of."""
    y = np.abs(x)
    z = y.copy()
    z[..., :a] = z[..., a:2 * a] = y[..., :a] + y[..., a:2 * a]
    return z


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("name", list(TYPES))
def test_forward_and_backward(case, name):
    dtype = TYPES[name]
    host, dev, at, freq, w, cfg = inputs(case, dtype)
    D, a = cfg.head_dim, cfg.num_rope_angles
    e, h, t = (D + 16) * 2.0 ** -24, half_step(dtype), tiny(dtype)
    common = (at.to(DEV), freq.to(DEV), w[0].to(DEV), w[1].to(DEV), cfg)
    y = m3.m3_qk_norm_rope(dev[0], dev[1], *common)
    g = m3.m3_qk_norm_rope_bwd(dev[2], dev[3], dev[0], dev[1], *common)
    torch.cuda.synchronize()
    for i, n in enumerate("qk"):
        x, gr, wt = f64(host[i]), f64(host[2 + i]), f64(w[i])
        ref = A.norm_rope(x, wt, at.numpy(), freq.numpy(), 1e-5)
        plain = A.norm_rope(x, wt, at.numpy() * 0, freq.numpy(), 1e-5)
        check(y[n], ref, h * np.abs(ref) + e * swap(plain, a) + t, n)
        dx, dw = A.norm_rope_backward(gr, x, wt, at.numpy(), freq.numpy(), 1e-5)
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
        ug = swap(gr, a)
        size = r * ug * np.abs(wt) + np.abs(x) * r ** 3 * (ug * np.abs(wt * x)).mean(-1, keepdims=True)
        check(g[n], dx, h * np.abs(dx) + 2 * e * size + t, "d" + n)
        terms = (ug * np.abs(x) * r).sum((0, 1))
        # a lane adds up to its share of the rows and heads in float32
        many = e + min(x.shape[0] * x.shape[1], 4096) * 2.0 ** -24
        check(g[n + "_weight"], dw, h * 0 + 2.0 ** -24 * np.abs(dw) + many * terms, f"d{n} weight")


def test_in_place_and_far_positions():
    host, dev, at, freq, w, cfg = inputs((50, 4, 2, 64, 32, "plain"), torch.float32)
    at = at * 0 + 2 ** 31 - 1 - torch.arange(50, dtype=torch.int32)
    common = (at.to(DEV), freq.to(DEV), w[0].to(DEV), w[1].to(DEV), cfg)
    y = m3.m3_qk_norm_rope(dev[0], dev[1], *common)
    ref = A.norm_rope(f64(host[0]), f64(w[0]), at.numpy(), freq.numpy(), 1e-5)
    plain = A.norm_rope(f64(host[0]), f64(w[0]), at.numpy() * 0, freq.numpy(), 1e-5)
    # the float64 angle of a position of 2^31 has 2^-22 of absolute accuracy left
    check(y["q"], ref, 2.0 ** -24 * np.abs(ref) + (80 * 2.0 ** -24 + 2.0 ** -22) * swap(plain, 32), "far")
    m3.m3_qk_norm_rope(dev[0], dev[1], *common, outs={"q": dev[0], "k": dev[1]})
    torch.cuda.synchronize()
    assert torch.equal(dev[0], y["q"]) and torch.equal(dev[1], y["k"])


def test_repeats_bitwise_and_replays():
    _, dev, at, freq, w, cfg = inputs((2500, 6, 2, 64, 32, "plain"), torch.bfloat16)
    common = (at.to(DEV), freq.to(DEV), w[0].to(DEV), w[1].to(DEV), cfg)
    first = m3.m3_qk_norm_rope_bwd(dev[2], dev[3], dev[0], dev[1], *common)
    grads = {n: torch.empty_like(t) for n, t in first.items()}
    ws = torch.empty(m3.qk_norm_rope_bwd_workspace_bytes(cfg, 2500), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m3.m3_qk_norm_rope_bwd(dev[2], dev[3], dev[0], dev[1], *common, grads=grads, workspace=ws)
    for turn in range(3):
        for t in (*grads.values(), ws):
            t.fill_(turn)
        graph.replay()
        torch.cuda.synchronize()
        again = m3.m3_qk_norm_rope_bwd(dev[2], dev[3], dev[0], dev[1], *common)
        assert all(torch.equal(grads[n], first[n]) and torch.equal(again[n], first[n]) for n in first)
