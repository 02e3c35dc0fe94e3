"""Host-side refusals of the attention layer's entry points: each broken rule is named, before any HIP
call (these run on a CPU-only host), and the binding's own checks of tensors."""

import pytest
import torch

import selective_state_space_mamba3_amd as m3
from selective_state_space_mamba3_amd import _binding as bd

INVALID, UNSUPPORTED = bd.M3_ERR_INVALID_ARGUMENT, bd.M3_ERR_UNSUPPORTED
FAKE = 0x1000  # never dereferenced: every call below is rejected by validation
ROPE = dict(num_heads=4, num_groups=2, head_dim=64, num_rope_angles=32)
ATTN = dict(batch_size=2, q_length=8, kv_length=16, num_heads=4, num_groups=2, head_dim=64)
STEP = dict(batch_size=2, q_length=1, kv_length=64, num_heads=4, num_groups=2, head_dim=64)


def view(data=FAKE, row=256, head=64):
    return bd._CView(data, row, head)


def rope(views=None, vectors=None, rows=3, ws_bytes=1 << 40, dtype=torch.bfloat16, bwd=False, **kw):
    c = bd.c_rope(m3.QkNormRopeConfig(**{**ROPE, **kw}), dtype)
    names = ("g_q", "g_k", "q", "k", "out_q", "out_k")
    v = {n: view() for n in names} | (views or {})
    p = dict(positions=FAKE, inv_freq=FAKE, q_weight=FAKE, k_weight=FAKE, dqw=FAKE, dkw=FAKE, ws=FAKE) | (vectors or {})
    vec = [p[n] for n in ("positions", "inv_freq", "q_weight", "k_weight")]
    if not bwd:
        return m3.lib().m3_qk_norm_rope(v["q"], v["k"], *vec, rows, c, v["out_q"], v["out_k"], None)
    return m3.lib().m3_qk_norm_rope_bwd(v["g_q"], v["g_k"], v["q"], v["k"], *vec, rows, c, v["out_q"], v["out_k"],
                                        p["dqw"], p["dkw"], p["ws"], ws_bytes, None)


def fwd(views=None, lse=FAKE, offsets=(None, None), totals=(16, 32), c=None, **kw):
    c = c or bd.c_attn(m3.AttnConfig(**{**ATTN, **kw}), torch.bfloat16)
    v = {n: view() for n in ("q", "k", "v", "out")} | (views or {})
    return m3.lib().m3_attn_fwd(v["q"], v["k"], v["v"], *offsets, *totals, c, v["out"], lse, FAKE, 1 << 40, None)


def bwd(views=None, lse=FAKE, offsets=(None, None), totals=(16, 32), ws=FAKE, ws_bytes=1 << 40, **kw):
    c = bd.c_attn(m3.AttnConfig(**{**ATTN, **kw}), torch.bfloat16)
    v = {n: view() for n in ("dout", "q", "k", "v", "out", "d_q", "d_k", "d_v")} | (views or {})
    return m3.lib().m3_attn_bwd(v["dout"], v["q"], v["k"], v["v"], v["out"], lse, *offsets, *totals, c, v["d_q"],
                                v["d_k"], v["d_v"], ws, ws_bytes, None)


def cache(data=FAKE, page=64 * 128, row=128, head=64):
    return bd._CCache(data, page, row, head)


def step(views=None, caches=None, lengths=FAKE, table=None, pages=2, size=64, most=1, ws=FAKE, ws_bytes=1 << 40, **kw):
    c = bd.c_attn(m3.AttnConfig(**{**STEP, **kw}), torch.bfloat16)
    v = {n: view() for n in ("q", "k", "v", "out")} | (views or {})
    kc = {n: cache() for n in ("k_cache", "v_cache")} | (caches or {})
    return m3.lib().m3_attn_step(v["q"], v["k"], v["v"], kc["k_cache"], kc["v_cache"], lengths, table, pages, size,
                                 most, c, v["out"], ws, ws_bytes, None)


def refused(status, op, rule, code=INVALID):
    assert status == code
    assert m3.last_error().startswith(op + ": ") and rule in m3.last_error(), m3.last_error()


HEADS_BAD = [
    (dict(num_heads=0), "num_heads is 0"), (dict(num_groups=3), "num_groups 3 does not divide num_heads 4"),
    (dict(num_groups=8), "num_groups 8 does not divide num_heads 4"), (dict(head_dim=0), "head_dim is 0"),
    (dict(head_dim=129, num_rope_angles=0), "head_dim 129 is above the limit of 128"),
]


@pytest.mark.parametrize("bad,rule", HEADS_BAD + [
    (dict(num_rope_angles=33), "2 * num_rope_angles = 66"), (dict(epsilon=0.0), "epsilon is 0"),
    (dict(epsilon=float("nan")), "epsilon is not a finite"), (dict(rows=0), "rows is 0")])
@pytest.mark.parametrize("back", [False, True])
def test_norm_rope_geometry(bad, rule, back):
    refused(rope(bwd=back, **bad), "m3_qk_norm_rope" + "_bwd" * back, rule)


@pytest.mark.parametrize("back", [False, True])
def test_norm_rope_operands(back):
    op = "m3_qk_norm_rope" + "_bwd" * back
    names = dict(q="q", k="k", out_q="d_q" if back else "out_q", out_k="d_k" if back else "out_k")
    if back:
        names |= dict(g_q="g_q", g_k="g_k")
    for n, shown in names.items():
        refused(rope({n: view(None)}, bwd=back), op, f"operand {shown} is NULL")
        refused(rope({n: view(FAKE + 1)}, bwd=back), op, f"operand {shown} is not aligned")
        refused(rope({n: view(row=63)}, bwd=back), op, f"operand {shown} has row_stride 63")
        refused(rope({n: view(head=-1)}, bwd=back), op, f"operand {shown} has head_stride -1")
        refused(rope({n: view(row=1 << 23)}, bwd=back), op, f"operand {shown} has row_stride", UNSUPPORTED)
    refused(rope({"out_q": view(head=63)}, bwd=back), op, "heads must not overlap")
    for n in ("positions", "inv_freq", "q_weight", "k_weight"):
        refused(rope(vectors={n: None}, bwd=back), op, f"operand {n} is NULL")
    if back:
        refused(rope(vectors=dict(ws=None), bwd=True), op, "workspace of")
        refused(rope(vectors=dict(ws=FAKE + 4), bwd=True), op, "aligned to 16 bytes")
        refused(rope(ws_bytes=8, bwd=True), op, "workspace of")


ATTN_BAD = [(b, r) for b, r in HEADS_BAD if "num_rope_angles" not in b] + [
    (dict(head_dim=129), "head_dim 129 is above"), (dict(batch_size=0), "batch_size is 0"),
    (dict(q_length=0), "q_length is 0"), (dict(kv_length=0), "kv_length is 0"),
    (dict(causal=False, window=4), "window 4 needs causal"), (dict(scale=-1.0), "scale is -1"),
    (dict(scale=float("inf")), "scale is inf"), (dict(causal=2), "flag causal is 2")]


@pytest.mark.parametrize("bad,rule", ATTN_BAD)
def test_attention_geometry(bad, rule):
    refused(fwd(**bad), "m3_attn_fwd", rule)
    refused(bwd(**bad), "m3_attn_bwd", rule)
    cfg = m3.AttnConfig(**{**ATTN, **bad})
    assert m3.attn_bwd_workspace_bytes(cfg, torch.bfloat16, 16, 32) == 0 and rule in m3.last_error()


def test_attention_rows_and_operands():
    for call, op, names in ((fwd, "m3_attn_fwd", ("q", "k", "v", "out")),
                            (bwd, "m3_attn_bwd", ("dout", "q", "k", "v", "out", "d_q", "d_k", "d_v"))):
        refused(call(totals=(15, 32)), op, "total_q is 15; without offsets it is batch_size * q_length = 16")
        refused(call(totals=(16, 33)), op, "total_kv is 33")
        refused(call(totals=(16, 1 << 31), offsets=(None, FAKE)), op, "total_kv is above", UNSUPPORTED)
        refused(call(lse=None), op, "operand lse is NULL")
        for n in names:
            refused(call({n: view(None)}), op, f"operand {n} is NULL")
            refused(call({n: view(FAKE + 1)}), op, f"operand {n} is not aligned")
            refused(call({n: view(row=60)}), op, f"operand {n} has row_stride 60")
        refused(call(q_length=1 << 30, batch_size=64, offsets=(FAKE, FAKE)), op, "more than one launch", UNSUPPORTED)
    refused(bwd(ws=None), "m3_attn_bwd", "workspace of")
    refused(bwd(ws_bytes=16), "m3_attn_bwd", "workspace of")
    refused(bwd(ws=FAKE + 8), "m3_attn_bwd", "aligned to 16 bytes")
    c = bd.c_attn(m3.AttnConfig(**ATTN), torch.bfloat16)
    bad = bd._CAttn(*[getattr(c, n) for n, _ in bd._CAttn._fields_])
    bad.dtype = 3
    refused(fwd(c=bad), "m3_attn_fwd", "dtype 3 is not one of")


@pytest.mark.parametrize("bad,rule", [(b, r) for b, r in ATTN_BAD if b not in (dict(causal=2),)] + [
    (dict(q_length=2), "q_length is 2; a decode step takes exactly one token"),
    (dict(causal=False), "a decode step is causal"), (dict(pages=0), "num_pages is 0"), (dict(size=0), "page_size is 0"),
    (dict(most=0, table=FAKE), "max_pages is 0"), (dict(size=31), "kv_length 64 is above max_pages * page_size = 31"),
    (dict(pages=1), "without a block_table"), (dict(most=2, size=32), "without a block_table"),
    (dict(lengths=None), "operand lengths is NULL"), (dict(ws=None), "workspace of"), (dict(ws_bytes=4), "workspace of")])
def test_step_refusals(bad, rule):
    if "ws" in bad or "ws_bytes" in bad:  # only a long cache is split and needs a workspace
        bad = {**bad, "kv_length": 65536, "size": 65536}
    refused(step(**bad), "m3_attn_step", rule)


def test_step_operands():
    for n in ("q", "k", "v", "out"):
        refused(step({n: view(None)}), "m3_attn_step", f"operand {n} is NULL")
        refused(step({n: view(row=1)}), "m3_attn_step", f"operand {n} has row_stride 1")
    for n in ("k_cache", "v_cache"):
        refused(step(caches={n: cache(None)}), "m3_attn_step", f"operand {n} is NULL")
        refused(step(caches={n: cache(FAKE + 1)}), "m3_attn_step", f"operand {n} is not aligned")
        for s in ("page", "row", "head"):
            refused(step(caches={n: cache(**{s: 63})}), "m3_attn_step", f"operand {n} has a stride below head_dim 64")


def test_binding_checks_tensors():
    cfg = m3.AttnConfig(**ATTN)
    q, k = torch.zeros(16, 4, 64), torch.zeros(32, 2, 64)
    with pytest.raises(ValueError, match="expected a GPU"):
        m3.m3_attn_fwd(q, k, k, cfg)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        m3.m3_attn_fwd(q.double(), k, k, cfg)
    with pytest.raises(ValueError, match=r"expected \(rows, heads, head_dim\)"):
        m3.m3_attn_fwd(q[0], k, k, cfg)
    with pytest.raises(TypeError, match="torch.Tensor"):
        m3.m3_attn_bwd(None, None, k, k, q, q, cfg)
    with pytest.raises(ValueError, match="expected a GPU"):
        m3.m3_qk_norm_rope(q, k, None, None, None, None, m3.QkNormRopeConfig(**ROPE))
    cfg = m3.AttnConfig(**STEP)
    q, k, kc = torch.zeros(2, 4, 64), torch.zeros(2, 2, 64), torch.zeros(2, 64, 2, 64)
    with pytest.raises(ValueError, match="v_cache has shape"):
        m3.m3_attn_step(q, k, k, kc, kc[:1], torch.zeros(2, dtype=torch.int32), cfg)
    with pytest.raises(ValueError, match="k_cache has shape"):
        m3.m3_attn_step(q, k, k, kc[:, :, :1], kc, torch.zeros(2, dtype=torch.int32), cfg)
    with pytest.raises(ValueError, match="block_table must be"):
        m3.m3_attn_step(q, k, k, kc, kc, torch.zeros(2, dtype=torch.int32), cfg, block_table=torch.zeros(2))
    with pytest.raises(ValueError, match="contiguous along its last axis"):
        bd._view("q", torch.zeros(3, 64, 4).transpose(1, 2), (3, 4, 64), torch.float32, torch.device("cpu"))
