"""Attention layer on the GPU against the float64 oracle.

Tolerances follow from the arithmetic, element by element: one rounding of the result (half a step of
its type), one of P and of dS before the products they enter, and float32 for everything else.  With
u = eps / 2 of the type (2^-22 for the split float32 products), S = max scale sum |q k|, n keys and D
columns, a probability is off by at most
    rel = (D + 8) 2^-24 S + 2^-22 max|z| + 2^-21 + n 2^-24
of itself (float32 dot product; argument, exponential and sum), and every bound below is that and u over
the sums of magnitudes that the errors enter; float16 adds half its smallest step for values below its
normal range."""

import numpy as np
import pytest
import torch

import selective_state_space_mamba3_amd as m3
from oracle import attention as A

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def unit(dtype):
    return 2.0 ** -22 if dtype == torch.float32 else half_step(dtype)


def tiny(dtype):
    return 2.0 ** -25 if dtype == torch.float16 else 0.0


def rand(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def check(got, ref, bound, what):
    got = f64(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), f"{what}: not finite"
    worst = (np.abs(got - ref) / (bound + 1e-300)).max() if got.size else 0.0
    print(f"[attn] {what}: {worst:.3f} of the bound", flush=True)
    assert worst <= 1.0, f"{what}: {worst} times the bound"


def split(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)


def layout(t, how):
    """The same values on the GPU under another layout."""
    t = t.to(DEV)
    rows, heads, dim = t.shape
    if how == "plain":
        return t.contiguous()
    if how == "packed":  # columns of wider rows, aligned
        wide = torch.full((rows, heads * dim + 3 * 16), 7.0, dtype=t.dtype, device=DEV)
        view = wide[:, 16:16 + heads * dim].view(rows, heads, dim)
    elif how == "odd":  # starts at an odd element, rows an odd distance apart
        wide = torch.full((rows, heads * dim + 5), 7.0, dtype=t.dtype, device=DEV)
        view = wide[:, 3:3 + heads * dim].view(rows, heads, dim)
    else:  # heads first
        view = torch.empty((heads, rows, dim), dtype=t.dtype, device=DEV).transpose(0, 1)
    view.copy_(t)
    return view


# sequences' (queries, keys), heads, groups, dim, causal, window, layout
CASES = [
    ([(1, 1)], 1, 1, 1, True, 0, "plain"),
    ([(1, 1), (1, 5)], 2, 1, 7, True, 0, "odd"),
    ([(64, 64)], 2, 1, 16, True, 0, "plain"),
    ([(65, 65), (63, 63), (1, 1)], 4, 2, 40, True, 0, "packed"),
    ([(129, 200), (31, 102)], 6, 2, 64, True, 0, "heads first"),
    ([(70, 130)], 3, 3, 64, False, 0, "plain"),
    ([(200, 90), (10, 0), (0, 12), (33, 32)], 4, 1, 64, True, 0, "plain"),
    ([(150, 150)], 2, 2, 80, True, 1, "plain"),
    ([(140, 333), (257, 257)], 8, 1, 128, True, 65, "packed"),
    ([(97, 161)], 5, 5, 100, True, 40, "odd"),
    ([(300, 300)], 2, 1, 128, False, 0, "heads first"),
    ([(1, 700), (2, 650)], 8, 2, 128, True, 0, "plain"),
    ([(385, 385)], 3, 1, 96, True, 0, "plain"),
    ([(3, 5000)], 2, 1, 64, False, 0, "plain"),
]


class Problem:
    def __init__(self, case, dtype, seed=0):
        seqs, H, G, D, self.causal, self.window, how = case
        self.dtype = dtype
        self.lens = seqs
        nq, nk = sum(s[0] for s in seqs), sum(s[1] for s in seqs)
        self.cq, self.ck = split([s[0] for s in seqs]), split([s[1] for s in seqs])
        # float32 rows keep bits that a 16-bit path would lose
        self.q, self.k, self.v, self.g = (rand((n, h, D), dtype, 10 * seed + i) for i, (n, h) in enumerate(
            [(nq, H), (nk, G), (nk, G), (nq, H)]))
        self.cfg = m3.AttnConfig(len(seqs), max(s[0] for s in seqs), max(s[1] for s in seqs), H, G, D, self.causal,
                                 self.window)
        self.dev = [layout(t, how) for t in (self.q, self.k, self.v, self.g)]
        equal = len(set(seqs)) == 1
        self.offsets = dict(q_offsets=None, kv_offsets=None) if equal else dict(
            q_offsets=torch.from_numpy(self.cq).to(DEV), kv_offsets=torch.from_numpy(self.ck).to(DEV))

    def sequences(self):
        for b, (nq, nk) in enumerate(self.lens):
            s, t = slice(self.cq[b], self.cq[b] + nq), slice(self.ck[b], self.ck[b] + nk)
            yield s, t, f64(self.q[s]), f64(self.k[t]), f64(self.v[t]), f64(self.g[s])

    def reference(self):
        """out, lse, dq, dk, dv and the bounds of their errors."""
        D, share = self.q.shape[2], self.q.shape[1] // self.k.shape[1]
        scale, u, w, t0 = D ** -0.5, unit(self.dtype), half_step(self.dtype), tiny(self.dtype)
        ref = [np.zeros(x.shape) for x in (self.q, self.q[..., 0], self.q, self.k, self.v)]
        bound = [np.zeros(x.shape) for x in ref]
        for s, t, q, k, v, g in self.sequences():
            if not len(q) or not len(k):
                ref[1][s] = -np.inf
                continue
            out, lse = A.attention(q, k, v, self.causal, self.window)
            dq, dk, dv = A.attention_backward(g, q, k, v, self.causal, self.window)
            p, _ = A.probabilities(q, k, self.causal, self.window, scale)
            kk, vv = np.repeat(k, share, 1), np.repeat(v, share, 1)
            big = scale * np.einsum("ihd,jhd->hij", np.abs(q), np.abs(kk)).max()
            rel = (D + 8) * 2.0 ** -24 * big + 2.0 ** -22 * big + 2.0 ** -21 + len(k) * 2.0 ** -24
            av = np.einsum("hij,jhd->ihd", p, np.abs(vv))
            dp = np.einsum("ihd,jhd->hij", g, vv)
            adp = np.einsum("ihd,jhd->hij", np.abs(g), np.abs(vv))
            delta = np.einsum("ihd,ihd->hi", g, out)
            # delta comes from the rounded out; dp and delta are float32 sums of magnitude adp
            out_err = (u + 2 * rel) * av + w * np.abs(out) + t0 * np.abs(vv).sum(0)[None] * 2
            d_err = np.einsum("ihd,ihd->hi", np.abs(g), out_err)[..., None] + (D + 8) * 2.0 ** -24 * 2 * adp
            ds = np.abs(p * (dp - delta[..., None]))
            ds_err = (u + 2 * rel) * ds + p * d_err + t0
            shared = lambda x: x.reshape(x.shape[0], -1, share, D).sum(2)
            n_sum = len(q) * share * 2.0 ** -24
            values = [out, lse, dq, dk, dv]
            errors = [
                out_err, rel + 2.0 ** -22 * (np.abs(np.where(np.isfinite(lse), lse, 0)) + 1),
                scale * np.einsum("hij,jhd->ihd", ds_err + len(k) * 2.0 ** -24 * ds, np.abs(kk)) + w * np.abs(dq) + t0,
                scale * shared(np.einsum("hij,ihd->jhd", ds_err + n_sum * ds, np.abs(q))) + w * np.abs(dk) + t0,
                shared(np.einsum("hij,ihd->jhd", (u + 2 * rel + n_sum) * p + t0, np.abs(g))) + w * np.abs(dv) + t0]
            for i, at in enumerate((s, s, s, t, t)):
                ref[i][at], bound[i][at] = values[i], errors[i]
        return ref, bound


def case_id(c):
    return "-".join(f"{a}x{b}" for a, b in c[0]) + f"-h{c[1]}g{c[2]}d{c[3]}" + ("c" if c[4] else "") + f"w{c[5]}-{c[6]}"


@pytest.mark.parametrize("case", CASES, ids=case_id)
@pytest.mark.parametrize("name", list(TYPES))
def test_forward_and_backward(case, name):
    dtype = TYPES[name]
    pr = Problem(case, dtype)
    q, k, v, g = pr.dev
    ref, bound = pr.reference()
    out, lse = m3.m3_attn_fwd(q, k, v, pr.cfg, **pr.offsets)
    grads = m3.m3_attn_bwd(g, q, k, v, out, lse, pr.cfg, **pr.offsets)
    torch.cuda.synchronize()
    check(out, ref[0], bound[0], "out")
    got = f64(lse)
    empty = np.isinf(ref[1])
    assert (got[empty] == -np.inf).all()
    check(torch.from_numpy(got[~empty]), ref[1][~empty], bound[1][~empty], "lse")
    for i, n in enumerate("qkv"):
        check(grads[n], ref[2 + i], bound[2 + i], "d" + n)
    # the same buffers again: the same bits
    again = m3.m3_attn_bwd(g, q, k, v, out, lse, pr.cfg, **pr.offsets)
    for n in "qkv":
        assert torch.equal(again[n], grads[n])


@pytest.mark.parametrize("name", list(TYPES))
def test_outputs_take_strides_and_leave_the_rest(name):
    dtype = TYPES[name]
    pr = Problem(([(77, 77)], 4, 2, 64, True, 0, "plain"), dtype)
    q, k, v, g = pr.dev
    plain, lse = m3.m3_attn_fwd(q, k, v, pr.cfg)
    plain_grads = m3.m3_attn_bwd(g, q, k, v, plain, lse, pr.cfg)
    for how in ("packed", "odd", "heads first"):
        out = layout(torch.zeros_like(plain), how)
        m3.m3_attn_fwd(q, k, v, pr.cfg, out=out)
        grads = {n: layout(torch.zeros_like(plain_grads[n]), how) for n in "qkv"}
        m3.m3_attn_bwd(g, q, k, v, out, lse, pr.cfg, grads=grads)
        assert torch.equal(out, plain)
        for n in "qkv":
            assert torch.equal(grads[n], plain_grads[n])
        if how != "heads first":
            start = {"packed": 16, "odd": 3}[how]
            base = out._base
            assert (base[:, :start] == 7).all() and (base[:, start + 4 * 64:] == 7).all()


@pytest.mark.parametrize("name", list(TYPES))
def test_hidden_infinities_stay_hidden(name):
    """Keys and values behind the diagonal, outside the window or in the next sequence."""
    dtype = TYPES[name]
    for window in (0, 50):
        pr = Problem(([(150, 150), (90, 90)], 2, 1, 64, True, window, "plain"), dtype)
        q, k, v, _ = pr.dev
        out, lse = m3.m3_attn_fwd(q, k, v, pr.cfg, **pr.offsets)
        k2, v2 = k.clone(), v.clone()
        v2[100, 0, 5] = float("nan")
        v2[101, 0, 6] = float("inf")
        k2[102] = float("nan")
        v2[150 + 40] = float("inf")
        out2, lse2 = m3.m3_attn_fwd(q, k2, v2, pr.cfg, **pr.offsets)
        torch.cuda.synchronize()
        row = torch.arange(240, device=DEV)
        in_first, at = row < 150, torch.where(row < 150, row, row - 150)
        reach = window or 1000
        touched = torch.where(in_first, (at >= 100) & (at < 102 + reach), (at >= 40) & (at < 40 + reach))
        assert torch.equal(out2[~touched], out[~touched]) and torch.equal(lse2[~touched], lse[~touched])
        assert out2[100, :, 5].isnan().all() and out2[101, :, 6].isfinite().logical_not().all()
        assert out2[102:min(102 + reach, 150)].isnan().all()
        assert out2[100, :, :5].isfinite().all() and out2[100, :, 6:].isfinite().all()
        assert not out2[150 + 40].isfinite().any()


@pytest.mark.parametrize("name", list(TYPES))
def test_large_scores_and_one_hot_rows(name):
    """Scores in the thousands: each query picks its largest key; nothing overflows."""
    dtype = TYPES[name]
    n, D = 192, 64
    q = torch.zeros(n, 1, D, dtype=dtype)
    k = torch.zeros(n, 1, D, dtype=dtype)
    q[:, 0, 0] = 200
    k[:, 0, 0] = torch.arange(n).to(dtype)  # rising: the running maximum moves in every tile
    v = rand((n, 1, D), dtype, 3)
    cfg = m3.AttnConfig(1, n, n, 1, 1, D)
    out, _ = m3.m3_attn_fwd(q.to(DEV), k.to(DEV), v.to(DEV), cfg)
    torch.cuda.synchronize()
    # next key: exp(-25) of the largest
    check(out, f64(v), half_step(dtype) * np.abs(f64(v)) + 2.0 ** -33 + unit(dtype) * np.abs(f64(v)), "one-hot")


def test_gradient_against_differences():
    pr = Problem(([(40, 61)], 4, 2, 40, True, 0, "plain"), torch.float32, seed=5)
    q, k, v, g = pr.dev
    out, lse = m3.m3_attn_fwd(q, k, v, pr.cfg)
    grads = m3.m3_attn_bwd(g, q, k, v, out, lse, pr.cfg)
    _, bound = pr.reference()
    host = [f64(x) for x in (pr.q, pr.k, pr.v)]
    r = np.random.default_rng(0)
    for i, n in enumerate("qkv"):
        way = r.normal(size=host[i].shape)
        vals = []
        for h in (1e-4, -1e-4):
            args = list(host)
            args[i] = args[i] + h * way
            vals.append((f64(pr.g) * A.attention(*args)[0]).sum())
        quotient = (vals[0] - vals[1]) / 2e-4
        # the quotient's own error: third derivatives of order one times h^2, cancellation 1e-12
        assert abs(quotient - (f64(grads[n]) * way).sum()) <= (bound[2 + i] * np.abs(way)).sum() + 1e-4


@pytest.mark.parametrize("name", ["bf16", "f32"])
def test_streams_workspaces_and_graphs(name):
    dtype = TYPES[name]
    pr = Problem(([(130, 130), (97, 97)], 4, 2, 64, True, 0, "plain"), dtype)
    q, k, v, g = pr.dev
    out, lse = m3.m3_attn_fwd(q, k, v, pr.cfg, **pr.offsets)
    grads = m3.m3_attn_bwd(g, q, k, v, out, lse, pr.cfg, **pr.offsets)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out2, lse2 = m3.m3_attn_fwd(q, k, v, pr.cfg, **pr.offsets, stream=side)
    grads2 = m3.m3_attn_bwd(g, q, k, v, out2, lse2, pr.cfg, **pr.offsets, stream=side)
    side.synchronize()
    assert torch.equal(out, out2) and all(torch.equal(grads[n], grads2[n]) for n in "qkv")

    bufs = dict(out=torch.empty_like(out), lse=torch.empty_like(lse))
    gb = {n: torch.empty_like(grads[n]) for n in "qkv"}
    ws = torch.empty(max(1, m3.attn_bwd_workspace_bytes(pr.cfg, dtype, q.shape[0], k.shape[0]),
                         m3.attn_fwd_workspace_bytes(pr.cfg, dtype)), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m3.m3_attn_fwd(q, k, v, pr.cfg, **pr.offsets, **bufs, workspace=ws)
        m3.m3_attn_bwd(g, q, k, v, bufs["out"], bufs["lse"], pr.cfg, **pr.offsets, grads=gb, workspace=ws)
    for turn in range(4):
        for t in (*bufs.values(), *gb.values(), ws):
            t.fill_(turn)
        q.copy_(rand(q.shape, dtype, 50 + turn))
        graph.replay()
        torch.cuda.synchronize()
        want, want_lse = m3.m3_attn_fwd(q, k, v, pr.cfg, **pr.offsets)
        want_g = m3.m3_attn_bwd(g, q, k, v, want, want_lse, pr.cfg, **pr.offsets)
        assert torch.equal(want, bufs["out"]) and torch.equal(want_lse, bufs["lse"])
        assert all(torch.equal(want_g[n], gb[n]) for n in "qkv")


def test_bad_offsets_stay_inside():
    """Offsets outside the rows are clamped: rows of whole sequences keep their results."""
    pr = Problem(([(40, 40), (50, 50)], 2, 2, 64, True, 0, "plain"), torch.bfloat16)
    q, k, v, _ = pr.dev
    good, _ = m3.m3_attn_fwd(q, k, v, pr.cfg, **pr.offsets)
    bad = torch.tensor([0, 40, 1 << 30], dtype=torch.int32, device=DEV)
    out, _ = m3.m3_attn_fwd(q, k, v, pr.cfg, q_offsets=bad, kv_offsets=bad)
    torch.cuda.synchronize()
    assert torch.equal(out, good)
    back = torch.tensor([50, -7, 20], dtype=torch.int32, device=DEV)
    m3.m3_attn_fwd(q, k, v, pr.cfg, q_offsets=back, kv_offsets=back)
    torch.cuda.synchronize()
