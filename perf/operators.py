"""Timed cases of the attention layer's operators: the per-head norm with rotation, softmax attention
forward and backward, and the single-token step over a key / value cache.

``run`` computes each operator in plain torch (``own`` false) or through the library (``own`` true) on the
inputs that ``prepare`` made; ``exact`` is the same in float64 straight from the definition.

Geometries are those of the scan workloads (24 or 32 heads of 64, states of 128, 4 x 2048 tokens for
training, 256 rows for decoding, 65536 tokens for long contexts), with shared key / value heads.
"""

from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5


# ---------------------------------------------------------------- cases


def listed():
    return [
        # queries and keys of 4 x 2048 training tokens, read in place from the packed projection rows
        dict(name="norm_rope_train", op="norm_rope", dtype="bf16", rows=8192, heads=24, groups=8, dim=64,
             angles=32, packed=True, far=2048),
        # one decode token for each of 256 rows, far positions
        dict(name="norm_rope_decode", op="norm_rope", dtype="bf16", rows=256, heads=32, groups=4, dim=128,
             angles=64, packed=True, far=65536),
        # its gradient over the training tokens
        dict(name="norm_rope_bwd_train", op="norm_rope_bwd", dtype="bf16", rows=8192, heads=24, groups=8, dim=64,
             angles=32, packed=True, far=2048),
        # float32, an odd number of rows, a head dimension that is no power of two, part of it rotated
        dict(name="norm_rope_bwd_odd", op="norm_rope_bwd", dtype="f32", rows=1537, heads=6, groups=3, dim=80,
             angles=24, packed=False, far=4096),
        # the tiny scan's geometry: a call that is all latency
        dict(name="attn_fwd_tiny", op="attn_fwd", dtype="f32", heads=2, groups=1, dim=16, causal=True, window=0,
             seqs=1, q_len=64, k_len=64, ragged=0, packed=False),
        # the training layer: 4 x 2048 tokens
        dict(name="attn_fwd_train", op="attn_fwd", dtype="bf16", heads=24, groups=8, dim=64, causal=True, window=0,
             seqs=4, q_len=2048, k_len=2048, ragged=0, packed=True),
        # prompts of odd lengths packed behind one another, each with a cached prefix, over a sliding window
        dict(name="attn_fwd_ragged", op="attn_fwd", dtype="f16", heads=32, groups=4, dim=128, causal=True, window=513,
             seqs=9, q_len=1023, k_len=2047, ragged=7, packed=False),
        # one long prompt
        dict(name="attn_fwd_long", op="attn_fwd", dtype="bf16", heads=16, groups=2, dim=128, causal=True, window=0,
             seqs=1, q_len=16384, k_len=16384, ragged=0, packed=False),
        # the training layer's gradient
        dict(name="attn_bwd_train", op="attn_bwd", dtype="bf16", heads=24, groups=8, dim=64, causal=True, window=0,
             seqs=4, q_len=2048, k_len=2048, ragged=0, packed=True),
        # gradient over packed sequences of odd lengths, heads of 128
        dict(name="attn_bwd_ragged", op="attn_bwd", dtype="f16", heads=16, groups=2, dim=128, causal=True, window=0,
             seqs=6, q_len=1999, k_len=1999, ragged=5, packed=False),
        # 256 rows decode one token each, contexts up to 2048, a dense cache
        dict(name="attn_step_batch", op="attn_step", dtype="bf16", heads=24, groups=8, dim=64, window=0,
             seqs=256, k_len=2048, ragged=3, page=0),
        # one row decodes at the end of a 65536-token context, a cache of 64-token pages
        dict(name="attn_step_long", op="attn_step", dtype="bf16", heads=32, groups=4, dim=128, window=0,
             seqs=1, k_len=65536, ragged=0, page=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    """Heads, shared heads and their width: one head to 32, all of their own to one for all."""
    groups = rng.choice([1, 2, 4, 8])
    heads = groups * rng.choice([1, 2, 4, 8] if groups < 8 else [1, 3])
    return heads, groups, rng.choice([16, 40, 64, 64, 80, 128, 128] if heads <= 16 else [16, 40, 64, 80])


def draw(rng):
    """One more case: any operator, type and head layout, lengths spread over their logarithm."""
    op = rng.choice(["norm_rope", "norm_rope_bwd", "attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "attn_step",
                     "attn_step"])
    heads, groups, dim = _heads(rng)
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), heads=heads, groups=groups, dim=dim)
    if op.startswith("norm_rope"):
        case.update(rows=_log_int(rng, 1, 8000), angles=rng.choice([dim // 2, dim // 4]),
                    packed=groups < 4 and rng.random() < 0.6, far=rng.choice([2048, 65536]))
        return case
    if op == "attn_step":
        seqs = _log_int(rng, 1, 256)
        case.update(seqs=seqs, k_len=_log_int(rng, 2, min(65000, 260000 // seqs)),
                    window=rng.choice([0, 0, 129, 1000]), ragged=rng.randrange(1, 1000),
                    page=rng.choice([0, 16, 48, 64, 256]))
        return case
    top = 4000 if case["dtype"] != "f32" else 1500
    q_len = _log_int(rng, 1, top)
    seqs = rng.randrange(1, max(2, min(8, 12000 // max(q_len, 256))))
    k_len = q_len if op == "attn_bwd" or rng.random() < 0.7 else min(top, q_len + _log_int(rng, 1, 2000))
    case.update(seqs=seqs, q_len=q_len, k_len=k_len, causal=rng.random() < 0.7,
                window=rng.choice([0, 0, 0, 65, 300]) if case["dtype"] != "f32" else 0,
                ragged=rng.choice([0, rng.randrange(1, 1000)]), packed=False)
    if not case["causal"]:
        case["window"] = 0
    return case


def _lengths(case):
    """Query and key lengths of a case's sequences; ragged ones are spread below the largest."""
    n, lq, lk = case["seqs"], case.get("q_len", 1), case["k_len"]
    if not case["ragged"]:
        return [lq] * n, [lk] * n
    r = random.Random(case["ragged"])
    if case["op"] == "attn_step":
        return [1] * n, [lk if i == 0 else r.randint(max(1, lk // 4), lk) for i in range(n)]
    q = [lq if i == 0 else r.randint(max(1, lq // 8), lq) for i in range(n)]
    return q, [x + (lk - lq) for x in q]


def _pairs(case):
    """How many (query, allowed key) pairs a head has."""
    total = 0
    for lq, lk in zip(*_lengths(case)):
        if not case["causal"]:
            total += lq * lk
            continue
        c, w = lk - lq, case["window"] or lk
        full = min(max(w - c - 1, 0), lq)  # rows whose window is not full yet: i + c + 1 keys
        total += full * (full + 1) // 2 + full * c + (lq - full) * min(w, lk)
    return total


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    heads, groups, dim = case["heads"], case["groups"], case["dim"]
    if case["op"] == "norm_rope":
        rows = case["rows"] * (heads + groups)
        return {"bytes": 2 * rows * dim * size + 4 * case["rows"], "flops": 8 * rows * dim}
    if case["op"] == "norm_rope_bwd":
        rows = case["rows"] * (heads + groups)
        return {"bytes": 3 * rows * dim * size + 4 * case["rows"], "flops": 16 * rows * dim}
    lq, lk = _lengths(case)
    if case["op"] == "attn_step":
        seen = sum(min(n, case["window"] or n) for n in lk)
        return {"bytes": 2 * seen * groups * dim * size + 2 * len(lk) * (heads + groups) * dim * size,
                "flops": 4 * seen * heads * dim}
    q, k = sum(lq) * heads * dim * size, sum(lk) * groups * dim * size
    lse = 4 * sum(lq) * heads
    if case["op"] == "attn_fwd":
        return {"bytes": 2 * q + 2 * k + lse, "flops": 4 * _pairs(case) * heads * dim}
    return {"bytes": 4 * q + 4 * k + lse, "flops": 10 * _pairs(case) * heads * dim}


# ---------------------------------------------------------------- inputs


def _unit(shape, dtype, gen):
    """Rows as the norm leaves them: unit RMS over the last axis."""
    x = torch.randn(shape, generator=gen, device="cuda")
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)).to(dtype)


def _offsets(lengths):
    return torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    heads, groups, dim = case["heads"], case["groups"], case["dim"]
    state = dict(case=case)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    if case["op"].startswith("norm_rope"):
        rows, angles = case["rows"], case["angles"]
        if case["packed"]:  # q | k | v of one projection row
            row = randn(rows, (heads + 2 * groups) * dim).to(dtype)
            q = row[:, :heads * dim].view(rows, heads, dim)
            k = row[:, heads * dim:(heads + groups) * dim].view(rows, groups, dim)
        else:
            q, k = randn(rows, heads, dim).to(dtype), randn(rows, groups, dim).to(dtype)
        start = torch.randint(0, case["far"], (1,), generator=gen, device="cuda")
        state.update(q=q, k=k, positions=((start + torch.arange(rows, device="cuda")) % case["far"]).to(torch.int32),
                     inv_freq=10000.0 ** (-torch.arange(angles, device="cuda", dtype=torch.float32) / angles),
                     q_weight=1 + 0.02 * randn(dim), k_weight=1 + 0.02 * randn(dim))
        if case["op"] == "norm_rope":
            state.update(out_q=torch.empty(rows, heads, dim, dtype=dtype, device="cuda"),
                         out_k=torch.empty(rows, groups, dim, dtype=dtype, device="cuda"))
        else:
            state.update(g_q=randn(rows, heads, dim).to(dtype), g_k=randn(rows, groups, dim).to(dtype),
                         d_q=torch.empty(rows, heads, dim, dtype=dtype, device="cuda"),
                         d_k=torch.empty(rows, groups, dim, dtype=dtype, device="cuda"),
                         d_qw=torch.empty(dim, device="cuda"), d_kw=torch.empty(dim, device="cuda"))
        return state

    lq, lk = _lengths(case)
    if case["op"] == "attn_step":
        n, page = case["seqs"], case["page"] or case["k_len"]
        per = -(-case["k_len"] // page)
        state.update(q=_unit((n, heads, dim), dtype, gen), k=_unit((n, groups, dim), dtype, gen),
                     v=randn(n, groups, dim).to(dtype),
                     k_cache=_unit((n * per, page, groups, dim), dtype, gen),
                     v_cache=torch.randn((n * per, page, groups, dim), generator=gen, device="cuda", dtype=dtype),
                     lengths=torch.tensor([x - 1 for x in lk], dtype=torch.int32, device="cuda"),
                     out=torch.empty(n, heads, dim, dtype=dtype, device="cuda"), table=None)
        if case["page"]:  # pages handed out in no order
            state["table"] = torch.randperm(n * per, generator=gen, device="cuda").to(torch.int32).view(n, per)
        return state

    tq, tk = sum(lq), sum(lk)
    if case["packed"]:  # v stays in its packed projection row, q and k come from the norm
        row = randn(tk, (heads + 2 * groups) * dim).to(dtype)
        v = row[:, (heads + groups) * dim:].view(tk, groups, dim)
    else:
        v = randn(tk, groups, dim).to(dtype)
    state.update(q=_unit((tq, heads, dim), dtype, gen), k=_unit((tk, groups, dim), dtype, gen), v=v,
                 q_offsets=_offsets(lq) if case["ragged"] else None,
                 k_offsets=_offsets(lk) if case["ragged"] else None,
                 out=torch.empty(tq, heads, dim, dtype=dtype, device="cuda"),
                 lse=torch.empty(tq, heads, device="cuda"))
    if case["op"] == "attn_bwd":
        state["dout"] = randn(tq, heads, dim).to(dtype)
        out, lse = _attn_fwd(state)  # what the forward pass left
        state.update(out=out, lse=lse, d_q=torch.empty_like(state["q"]), d_k=torch.empty_like(state["k"]),
                     d_v=torch.empty(tk, groups, dim, dtype=dtype, device="cuda"))
    return state


# ---------------------------------------------------------------- plain forms


def _rotate(x, positions, inv_freq, sign):
    """Turn the pairs (a, a + A) of each head by sign * position * inv_freq[a]."""
    a = inv_freq.numel()
    theta = positions.double()[:, None, None] * inv_freq.double()
    cos, sin = theta.cos().float(), sign * theta.sin().float()
    lo, hi = x[..., :a], x[..., a:2 * a]
    return torch.cat([lo * cos - hi * sin, lo * sin + hi * cos, x[..., 2 * a:]], -1)


def _norm_rope(x, weight, s):
    n = x.float()
    n = n * torch.rsqrt(n.square().mean(-1, keepdim=True) + EPS) * weight
    return _rotate(n, s["positions"], s["inv_freq"], 1).to(x.dtype)


def _norm_rope_bwd(x, weight, g, s):
    x32, g = x.float(), _rotate(g.float(), s["positions"], s["inv_freq"], -1)
    r = torch.rsqrt(x32.square().mean(-1, keepdim=True) + EPS)
    dw = (g * x32 * r).sum((0, 1), dtype=torch.float64).float()
    g = g * weight
    dx = r * g - x32 * r ** 3 * (g * x32).mean(-1, keepdim=True)
    return dx.to(x.dtype), dw


def _pad(x, offsets, case, length):
    """Rows of packed sequences as [seqs, heads, length, dim] in float32 (zeros behind each end), and which are real."""
    n = case["seqs"]
    if offsets is None:
        return x.float().reshape(n, length, *x.shape[1:]).transpose(1, 2), None
    at = offsets[:-1, None] + torch.arange(length, device="cuda")
    real = at < offsets[1:, None]
    at = at.clamp(max=x.shape[0] - 1).long()
    return (x[at].float() * real[..., None, None]).transpose(1, 2), real


def _unpad(x, real, dtype):
    x = x.transpose(1, 2)
    return (x.reshape(-1, *x.shape[2:]) if real is None else x[real]).to(dtype)


def _probabilities(s):
    """Scores' softmax over the allowed keys: q, k, v, p as [seqs, groups, heads per group, length, .]."""
    c = s["case"]
    lq, lk = (max(x) for x in _lengths(c))
    q, q_real = _pad(s["q"], s["q_offsets"], c, lq)
    k, k_real = _pad(s["k"], s["k_offsets"], c, lk)
    v, _ = _pad(s["v"], s["k_offsets"], c, lk)
    q = q.reshape(c["seqs"], c["groups"], -1, lq, c["dim"])
    k, v = k[:, :, None], v[:, :, None]
    i = torch.arange(lq, device="cuda")[:, None]
    j = torch.arange(lk, device="cuda")
    allowed = torch.ones(1, lq, lk, dtype=torch.bool, device="cuda")
    if c["causal"]:  # the last query of a sequence stands on its last key
        allowed = allowed & (j <= i + (c["k_len"] - c["q_len"]))
        if c["window"]:
            allowed = allowed & (j > i + (c["k_len"] - c["q_len"]) - c["window"])
    if k_real is not None:
        allowed = allowed & k_real[:, None, :]
    p = torch.matmul(q, k.transpose(-1, -2)).mul_(c["dim"] ** -0.5)
    p.masked_fill_(~allowed[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)
    return q, k, v, p.div_(torch.where(total == 0, torch.ones_like(total), total)), lse, q_real, k_real


def _attn_fwd(s):
    q, _, v, p, lse, q_real, _ = _probabilities(s)
    o = torch.matmul(p, v).flatten(1, 2)
    lse = lse.flatten(1, 2).transpose(1, 2)
    lse = lse.reshape(-1, lse.shape[-1]) if q_real is None else lse[q_real]
    return _unpad(o, q_real, s["q"].dtype), lse.contiguous()


def _attn_bwd(s):
    c, dtype = s["case"], s["q"].dtype
    q, k, v, p, _, q_real, k_real = _probabilities(s)
    do, _ = _pad(s["dout"], s["q_offsets"], c, q.shape[-2])
    do = do.reshape(q.shape)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    ds = torch.matmul(do, v.transpose(-1, -2))
    ds = p.mul_(ds.sub_((p * ds).sum(-1, keepdim=True))).mul_(c["dim"] ** -0.5)
    dq = torch.matmul(ds, k).flatten(1, 2)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2)
    return _unpad(dq, q_real, dtype), _unpad(dk, k_real, dtype), _unpad(dv, k_real, dtype)


def _attn_step(s):
    c, at = s["case"], s["lengths"].long()
    n, page = c["seqs"], s["k_cache"].shape[1]
    row = torch.arange(n, device="cuda")
    table = row[:, None] if s["table"] is None else s["table"].long()
    slot = table[row, at // page]
    s["k_cache"][slot, at % page] = s["k"]
    s["v_cache"][slot, at % page] = s["v"]
    k = s["k_cache"][table].flatten(1, 2).float().transpose(1, 2)  # [rows, groups, capacity, dim]
    v = s["v_cache"][table].flatten(1, 2).float().transpose(1, 2)
    q = s["q"].float().view(n, c["groups"], -1, c["dim"])
    j = torch.arange(k.shape[2], device="cuda")
    allowed = j <= at[:, None]
    if c["window"]:
        allowed = allowed & (j > at[:, None] - c["window"])
    p = torch.matmul(q, k.transpose(-1, -2)) * c["dim"] ** -0.5
    p = p.masked_fill(~allowed[:, None, None], -math.inf)
    p = (p - p.amax(-1, keepdim=True)).exp()
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    return o.view(n, c["heads"], c["dim"]).to(s["q"].dtype), s["k_cache"], s["v_cache"]


# ---------------------------------------------------------------- one pass


def _library(s):
    """The configuration and the workspace that a user's program makes once for its geometry."""
    import selective_state_space_mamba3_amd as m3
    c = s["case"]
    if c["op"].startswith("norm_rope"):
        s["cfg"] = m3.QkNormRopeConfig(num_heads=c["heads"], num_groups=c["groups"], head_dim=c["dim"],
                                       num_rope_angles=c["angles"], epsilon=EPS)
        need = m3.qk_norm_rope_bwd_workspace_bytes(s["cfg"], c["rows"]) if c["op"] == "norm_rope_bwd" else 0
    elif c["op"] == "attn_step":
        s["cfg"] = m3.AttnConfig(batch_size=c["seqs"], q_length=1, kv_length=s["k_cache"].shape[1] * (
            1 if s["table"] is None else s["table"].shape[1]), num_heads=c["heads"], num_groups=c["groups"],
            head_dim=c["dim"], causal=True, window=c["window"])
        need = m3.attn_step_workspace_bytes(s["cfg"], s["q"].dtype)
    else:
        lq, lk = _lengths(c)
        s["cfg"] = m3.AttnConfig(batch_size=c["seqs"], q_length=max(lq), kv_length=max(lk), num_heads=c["heads"],
                                 num_groups=c["groups"], head_dim=c["dim"], causal=c["causal"], window=c["window"])
        need = (m3.attn_fwd_workspace_bytes(s["cfg"], s["q"].dtype) if c["op"] == "attn_fwd"
                else m3.attn_bwd_workspace_bytes(s["cfg"], s["q"].dtype, s["q"].shape[0], s["k"].shape[0]))
    s["workspace"] = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    s["m3"] = m3


def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "norm_rope":
            return _norm_rope(s["q"], s["q_weight"], s), _norm_rope(s["k"], s["k_weight"], s)
        if op == "norm_rope_bwd":
            dq, dqw = _norm_rope_bwd(s["q"], s["q_weight"], s["g_q"], s)
            dk, dkw = _norm_rope_bwd(s["k"], s["k_weight"], s["g_k"], s)
            return dq, dk, dqw, dkw
        return {"attn_fwd": _attn_fwd, "attn_bwd": _attn_bwd, "attn_step": _attn_step}[op](s)
    if "cfg" not in s:
        _library(s)
    m3, cfg, ws = s["m3"], s["cfg"], s["workspace"]
    if op == "norm_rope":
        o = m3.m3_qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_weight"], s["k_weight"], cfg,
                               outs={"q": s["out_q"], "k": s["out_k"]})
        return o["q"], o["k"]
    if op == "norm_rope_bwd":
        g = m3.m3_qk_norm_rope_bwd(s["g_q"], s["g_k"], s["q"], s["k"], s["positions"], s["inv_freq"], s["q_weight"],
                                   s["k_weight"], cfg, grads={"q": s["d_q"], "k": s["d_k"], "q_weight": s["d_qw"],
                                                              "k_weight": s["d_kw"]}, workspace=ws)
        return g["q"], g["k"], g["q_weight"], g["k_weight"]
    if op == "attn_fwd":
        return m3.m3_attn_fwd(s["q"], s["k"], s["v"], cfg, q_offsets=s["q_offsets"], kv_offsets=s["k_offsets"],
                              out=s["out"], lse=s["lse"], workspace=ws)
    if op == "attn_bwd":
        g = m3.m3_attn_bwd(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], cfg, q_offsets=s["q_offsets"],
                           kv_offsets=s["k_offsets"], grads={"q": s["d_q"], "k": s["d_k"], "v": s["d_v"]},
                           workspace=ws)
        return g["q"], g["k"], g["v"]
    out = m3.m3_attn_step(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["lengths"], cfg,
                          block_table=s["table"], out=s["out"], workspace=ws)
    return out, s["k_cache"], s["v_cache"]


# ---------------------------------------------------------------- the definition in float64


def _exact_head(x, w, s):
    """y = R(theta) diag(w) x / rms as one complex rotation, on whole rows."""
    x, a = x.double(), s["inv_freq"].numel()
    n = w.double() * x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["positions"].double()[:, None, None] * s["inv_freq"].double())
    z = torch.complex(n[..., :a].contiguous(), n[..., a:2 * a].contiguous()) * turn
    return torch.cat([z.real, z.imag, n[..., 2 * a:]], -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return _exact_head(s["q"], s["q_weight"], s), _exact_head(s["k"], s["k_weight"], s)
    if case["op"] == "norm_rope_bwd":  # the gradient of sum(g y), by differentiating the definition
        leaves = [s[n].double().clone().requires_grad_() for n in ("q", "k", "q_weight", "k_weight")]
        y = (_exact_head(leaves[0], leaves[2], s) * s["g_q"].double()).sum() + (
            _exact_head(leaves[1], leaves[3], s) * s["g_k"].double()).sum()
        return torch.autograd.grad(y, leaves)
    lq, lk = _lengths(case)
    heads, groups, dim = case["heads"], case["groups"], case["dim"]
    share = heads // groups
    if case["op"] == "attn_step":
        page = s["k_cache"].shape[1]
        out = torch.zeros(case["seqs"], heads, dim, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lk):
            pages = [b] if s["table"] is None else s["table"][b].tolist()
            s["k_cache"][pages[(n - 1) // page], (n - 1) % page] = s["k"][b]
            s["v_cache"][pages[(n - 1) // page], (n - 1) % page] = s["v"][b]
            lo = max(0, n - case["window"]) if case["window"] else 0
            k, v = (s[x][pages].reshape(-1, groups, dim)[lo:n].double() for x in ("k_cache", "v_cache"))
            q = s["q"][b].double().view(groups, share, dim)
            p = torch.softmax(q @ k.permute(1, 2, 0) / dim ** 0.5, -1)
            out[b] = (p @ v.transpose(0, 1)).reshape(heads, dim)
        return out, s["k_cache"], s["v_cache"]
    grads = case["op"] == "attn_bwd"
    outs = [torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"),
            torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")]
    d = [torch.zeros(s[x].shape, dtype=torch.float64, device="cuda") for x in "qkv"]
    q0 = k0 = 0
    for nq, nk in zip(lq, lk):
        i, j = torch.arange(nq, device="cuda")[:, None] + (nk - nq), torch.arange(nk, device="cuda")
        hidden = torch.zeros(nq, nk, dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden = (j > i) | ((j <= i - case["window"]) if case["window"] else hidden)
        for h in range(heads):
            g = h // share
            q, k, v = (s["q"][q0:q0 + nq, h].double(), s["k"][k0:k0 + nk, g].double(), s["v"][k0:k0 + nk, g].double())
            z = (q @ k.T / dim ** 0.5).masked_fill(hidden, -math.inf)
            if not grads:
                outs[0][q0:q0 + nq, h] = torch.softmax(z, -1) @ v
                outs[1][q0:q0 + nq, h] = torch.logsumexp(z, -1)
                continue
            do, p = s["dout"][q0:q0 + nq, h].double(), torch.softmax(z, -1)
            d[2][k0:k0 + nk, g] += p.T @ do
            dp = do @ v.T
            z = p * (dp - (p * dp).sum(-1, keepdim=True)) / dim ** 0.5
            d[0][q0:q0 + nq, h] = z @ k
            d[1][k0:k0 + nk, g] += z.T @ q
        q0, k0 = q0 + nq, k0 + nk
    return tuple(d) if grads else tuple(outs)
