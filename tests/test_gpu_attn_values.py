"""Infinities, NaN and each type's largest values in keys and values, seen and hidden."""

import pytest
import torch

import selective_state_space_mamba3_amd as m3
import test_gpu_attn as base

pytestmark = pytest.mark.gpu

# sequences, heads, groups, dim, causal, window, layout: one block of queries to a wave, two, and shared keys
GEOMETRIES = [
    ([(150, 150)], 2, 1, 64, True, 0, "plain"),
    ([(150, 150)], 2, 1, 64, True, 50, "odd"),
    ([(130, 300)], 2, 2, 128, True, 70, "plain"),
    ([(520, 520)] * 4, 24, 8, 64, True, 0, "plain"),
    ([(200, 1400)], 2, 1, 40, True, 0, "plain"),
]


def seen_by(pr, key):
    """[queries] which queries of the first sequence see a key."""
    nq, nk = pr.lens[0]
    at = torch.arange(nq, device=base.DEV) + nk - nq
    return (at >= key) & (at < key + (pr.window or nk))


@pytest.mark.parametrize("case", GEOMETRIES, ids=base.case_id)
@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_seen_infinities_come_out(case, name):
    """A query that sees an infinity gets it, with its sign; one that sees both gets NaN."""
    pr = base.Problem(case, base.TYPES[name])
    q, k, v, _ = pr.dev
    nq, nk = pr.lens[0]
    inf = float("inf")
    for key in (0, 5, nk - nq + 3, nk - 30):
        v2 = v.clone()
        v2[key, 0, 1], v2[key, 0, 2], v2[key, 0, 3] = inf, -inf, inf
        v2[key + 1, 0, 3] = -inf
        out, lse = m3.m3_attn_fwd(q, k, v2, pr.cfg, **pr.offsets)
        clean, clean_lse = m3.m3_attn_fwd(q, k, v, pr.cfg, **pr.offsets)
        torch.cuda.synchronize()
        assert torch.equal(lse, clean_lse)
        first, second = seen_by(pr, key), seen_by(pr, key + 1)
        heads = slice(0, q.shape[1] // k.shape[1])
        one = out[:nq, heads]
        assert (one[first][..., 1] == inf).all() and (one[first][..., 2] == -inf).all()
        assert one[first & second][..., 3].isnan().all()
        assert (one[first & ~second][..., 3] == inf).all() and (one[second & ~first][..., 3] == -inf).all()
        assert torch.equal(one[~first & ~second], clean[:nq, heads][~first & ~second])
        rest = [0, *range(4, q.shape[2])]
        assert torch.equal(one[..., rest], clean[:nq, heads][..., rest])


@pytest.mark.parametrize("case", GEOMETRIES, ids=base.case_id)
@pytest.mark.parametrize("name", list(base.TYPES))
def test_hidden_keys_change_no_bit(case, name):
    """Large scores of the queries beside it leave a query's result as it is, bit for bit."""
    pr = base.Problem(case, base.TYPES[name])
    q, k, v, _ = pr.dev
    nq, nk = pr.lens[0]
    clean, clean_lse = m3.m3_attn_fwd(q, k, v, pr.cfg, **pr.offsets)
    for key in (nk - nq + 3, nk - 60):
        k2 = k.clone()
        k2[key:key + 4] *= 30
        out, lse = m3.m3_attn_fwd(q, k2, v, pr.cfg, **pr.offsets)
        torch.cuda.synchronize()
        touched = sum(seen_by(pr, key + i) for i in range(4)) > 0
        assert torch.equal(out[:nq][~touched], clean[:nq][~touched])
        assert torch.equal(lse[:nq][~touched], clean_lse[:nq][~touched])
        assert not torch.equal(lse[:nq][touched], clean_lse[:nq][touched])


@pytest.mark.parametrize("case", GEOMETRIES, ids=base.case_id)
@pytest.mark.parametrize("name", list(base.TYPES))
def test_hidden_largest_values_stay_hidden(case, name):
    """Finite values, the lowest and the largest of the type, where a mask would put them."""
    dtype = base.TYPES[name]
    pr = base.Problem(case, dtype)
    q, k, v, _ = pr.dev
    nq, nk = pr.lens[0]
    clean, clean_lse = m3.m3_attn_fwd(q, k, v, pr.cfg, **pr.offsets)
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    for key in (nk - nq + 3, nk - 60):
        k2, v2 = k.clone(), v.clone()
        v2[key], v2[key + 1] = low, high
        k2[key + 2], k2[key + 3] = low, high
        out, lse = m3.m3_attn_fwd(q, k2, v2, pr.cfg, **pr.offsets)
        torch.cuda.synchronize()
        touched = sum(seen_by(pr, key + i) for i in range(4)) > 0
        assert torch.equal(out[:nq][~touched], clean[:nq][~touched])
        assert torch.equal(lse[:nq][~touched], clean_lse[:nq][~touched])


@pytest.mark.parametrize("case", [
    ([(64, 200)], 2, 1, 64, True, 10, "plain"), ([(70, 300)], 4, 2, 128, True, 33, "packed"),
    ([(40, 333), (33, 150)], 3, 3, 80, True, 65, "odd")], ids=base.case_id)
@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_gradients_beside_largest_values(case, name):
    """Keys and values that no query sees hold the type's largest values: no gradient, and nobody else's changes."""
    dtype = base.TYPES[name]
    pr = base.Problem(case, dtype)
    q, k, v, g = pr.dev
    nq, nk = pr.lens[0]
    out, lse = m3.m3_attn_fwd(q, k, v, pr.cfg, **pr.offsets)
    clean = m3.m3_attn_bwd(g, q, k, v, out, lse, pr.cfg, **pr.offsets)
    first = nk - nq + 1 - pr.window  # the first key that any query sees
    k2, v2 = k.clone(), v.clone()
    for i, value in enumerate((torch.finfo(dtype).min, torch.finfo(dtype).max)):
        k2[first - 1 - i], v2[first - 3 - i], v2[first - 5 - i, :, ::2] = value, value, value
        k2[first - 7 - i], v2[first - 7 - i] = value, value
    grads = m3.m3_attn_bwd(g, q, k2, v2, out, lse, pr.cfg, **pr.offsets)
    torch.cuda.synchronize()
    for n in "qkv":
        assert torch.equal(grads[n], clean[n]), n
    assert (grads["k"][:first] == 0).all() and (grads["v"][:first] == 0).all()
