"""float16 gradients of attention from upstream gradients of many sizes, over many keys: P and dS lie far outside
float16's normal range there (below 2^-14, or above 65504) while the gradients themselves do not.

The measure is the error that rounding the exact gradients to float16 makes by itself.  A gradient carries that
rounding, the one of each dS (for dv: of each P) of the same relative size, and the one of out in delta, which is
smaller where a query sees many keys; independent errors add in squares, to sqrt(3) at most of the first,
and float32 adds nothing to speak of.  So each gradient has to stand within twice of it, in the Euclidean norm."""

import pytest
import torch

import selective_state_space_mamba3_amd as m3

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def rand(shape, seed, size=1.0):
    return (size * torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)).half()


def reference(q, k, v, g, causal):
    """(dq, dk, dv) of one sequence in float64."""
    share = q.shape[1] // k.shape[1]
    q, k, v, g = (x.double().transpose(0, 1).contiguous() for x in (q, k, v, g))
    n, m, scale = q.shape[1], k.shape[1], q.shape[2] ** -0.5
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    hidden = torch.ones(n, m, dtype=torch.bool).triu(1 + m - n) if causal else None
    for h in range(q.shape[0]):
        i = h // share
        z = q[h] @ k[i].T.contiguous() * scale
        p = torch.softmax(z.masked_fill(hidden, -torch.inf) if causal else z, -1)
        dp = g[h] @ v[i].T.contiguous()
        ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
        dq[h] = ds @ k[i]
        dk[i] += ds.T.contiguous() @ q[h]
        dv[i] += p.T.contiguous() @ g[h]
    return [x.transpose(0, 1) for x in (dq, dk, dv)]


def within_rounding(got, ref, what):
    err = float((got.cpu().double() - ref).norm())
    rounding = float((ref.half().double() - ref).norm())
    print(f"[attn] {what}: {err / rounding:.3f} of the result's rounding", flush=True)
    assert err <= 2 * rounding, f"{what}: {err / rounding} times the result's rounding"


def gradients(q, k, v, g, cfg):
    q, k, v, g = (x.to(DEV) for x in (q, k, v, g))
    out, lse = m3.m3_attn_fwd(q, k, v, cfg)
    return m3.m3_attn_bwd(g, q, k, v, out, lse, cfg)


# sequences, queries, keys, heads, groups, dim, causal, size of dout
CASES = [
    (1, 256, 2048, 2, 1, 64, False, 1e-3),
    (1, 256, 2048, 2, 1, 64, False, 1e-4),
    (1, 64, 8192, 2, 1, 64, False, 1e-2),
    (1, 64, 8192, 2, 2, 128, False, 1e-3),
    (1, 130, 8192, 1, 1, 40, True, 1e-4),
    (1, 64, 40000, 1, 1, 64, False, 1.0),
    (1, 64, 40000, 1, 1, 128, False, 1e-2),
    (2, 1024, 1024, 12, 4, 64, True, 1e-3),   # neither queries' nor keys' blocks shared
    (2, 1024, 1024, 12, 4, 96, False, 1e-4),
    (4, 512, 512, 2, 1, 64, True, 1e-4),
    (3, 100, 100, 2, 2, 7, False, 1e-3),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_small_upstream_gradients(case):
    n, lq, lk, H, G, D, causal, size = case
    q, k, v = rand((n * lq, H, D), 1), rand((n * lk, G, D), 2), rand((n * lk, G, D), 3)
    g = rand((n * lq, H, D), 4, size)
    got = gradients(q, k, v, g, m3.AttnConfig(n, lq, lk, H, G, D, causal))
    ref = [torch.cat(x) for x in zip(*(reference(q[b * lq:(b + 1) * lq], k[b * lk:(b + 1) * lk], v[b * lk:(b + 1) * lk],
                                                 g[b * lq:(b + 1) * lq], causal) for b in range(n)))]
    for i, name in enumerate("qkv"):
        within_rounding(got[name], ref[i], f"d{name} {case}")


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("rising", [False, True])
def test_queries_of_unlike_sizes(causal, rising):
    """Upstream gradients whose size changes by 2^24 from query to query and along the sequence; each size is looked at alone."""
    n, m, D = 384, 1500, 64
    q, k, v, g = rand((n, 2, D), 1), rand((m, 1, D), 2), rand((m, 1, D), 3), rand((n, 2, D), 4)
    step = torch.arange(n) * 13 // n if rising else 12 - torch.arange(n) * 13 // n
    step = torch.where(torch.arange(n) % 5 == 0, 12 - step, step)
    g = (g.double() * 4.0 ** (step - 8.0)[:, None, None]).half()
    got = gradients(q, k, v, g, m3.AttnConfig(1, n, m, 2, 1, D, causal))
    ref = reference(q, k, v, g, causal)
    for s in range(13):
        within_rounding(got["q"][step == s], ref[0][step == s], f"dq, size 4^{s - 8}")
    within_rounding(got["k"], ref[1], "dk")
    within_rounding(got["v"], ref[2], "dv")


def test_keys_of_unlike_sizes():
    """Values whose size changes by 2^10 from key to key: dS of one query spans them, dk of a key has its own."""
    n, m, D = 300, 700, 64
    q, k, v, g = rand((n, 2, D), 1), rand((m, 1, D), 2), rand((m, 1, D), 3), rand((n, 2, D), 4, 1e-3)
    size = 2.0 ** (torch.arange(m) * 11 // m - 5.0)
    v = (v.double() * size[:, None, None]).half()
    got = gradients(q, k, v, g, m3.AttnConfig(1, n, m, 2, 1, D, False))
    ref = reference(q, k, v, g, False)
    for i, name in enumerate("qkv"):
        within_rounding(got[name], ref[i], "d" + name)


def test_large_upstream_gradients():
    """dS above float16's largest value, gradients well inside."""
    q, k, v, g = rand((9, 1, 64), 1, 0.1), rand((9, 1, 64), 2, 0.05), rand((9, 1, 64), 3, 8.0), rand((9, 1, 64), 4, 1.5e4)
    got = gradients(q, k, v, g, m3.AttnConfig(1, 9, 9, 1, 1, 64, False))
    ref = reference(q, k, v, g, False)
    assert max(float(x.abs().max()) for x in ref) < 4e4
    for i, name in enumerate("qkv"):
        within_rounding(got[name], ref[i], "d" + name)


def test_zero_and_one_hot_gradients():
    """No upstream gradient at all gives zeros; one query's alone reaches the keys it sees."""
    q, k, v = rand((200, 2, 64), 1), rand((200, 1, 64), 2), rand((200, 1, 64), 3)
    g = torch.zeros(200, 2, 64, dtype=torch.float16)
    cfg = m3.AttnConfig(1, 200, 200, 2, 1, 64)
    got = gradients(q, k, v, g, cfg)
    assert all((got[n] == 0).all() for n in "qkv")
    g[150, 1] = rand((64,), 4, 1e-4)
    got, ref = gradients(q, k, v, g, cfg), reference(q, k, v, g, True)
    assert (got["q"][:150] == 0).all() and (got["k"][151:] == 0).all() and (got["v"][151:] == 0).all()
    for i, name in enumerate("qkv"):
        within_rounding(got[name], ref[i], "d" + name)
