"""Host-side refusals of the 8-bit cache's entry points: each broken rule is named, before any HIP call (these run on
a CPU-only host), and the binding's own checks of tensors."""

import ctypes

import pytest
import torch

import selective_state_space_mamba3_amd as m3
from selective_state_space_mamba3_amd import _binding as bd
from test_abi_attn import refused, view

INVALID, UNSUPPORTED = bd.M3_ERR_INVALID_ARGUMENT, bd.M3_ERR_UNSUPPORTED
FAKE = 0x1000  # never dereferenced: every call below is rejected by validation
CFG = dict(batch_size=2, q_length=3, kv_length=128, num_heads=4, num_groups=2, head_dim=64, block_size=16)


def cache(codes=FAKE, scales=FAKE, page=64 * 128, row=128, head=64):
    return bd._CKv8Cache(codes, scales, page, row, head)


def config(dtype=torch.bfloat16, **kw):
    return bd.c_kv8(m3.Kv8Config(**{**CFG, **kw}), dtype)


def parts(caches, pages, size, most, table):
    c = {"k_cache": cache(), "v_cache": cache()} | (caches or {})
    return c["k_cache"], c["v_cache"], table, pages, size, most


def write(views=None, caches=None, offsets=None, total=6, lengths=FAKE, pages=8, size=64, most=2, table=FAKE, c=None, **kw):
    v = {n: view() for n in "kv"} | (views or {})
    kc, vc, *rest = parts(caches, pages, size, most, table)
    return m3.lib().m3_kv8_write(v["k"], v["v"], offsets, total, lengths, kc, vc, *rest, c or config(**kw), None)


def read(views=None, caches=None, offsets=None, total=6, starts=None, pages=8, size=64, most=2, table=FAKE, c=None, **kw):
    v = {n: view() for n in "kv"} | (views or {})
    kc, vc, *rest = parts(caches, pages, size, most, table)
    return m3.lib().m3_kv8_read(kc, vc, starts, offsets, total, *rest, c or config(**kw), v["k"], v["v"], None)


def step(views=None, caches=None, lengths=FAKE, pages=8, size=64, most=2, table=FAKE, ws=FAKE, ws_bytes=1 << 40, c=None,
         **kw):
    v = {n: view() for n in ("q", "k", "v", "out")} | (views or {})
    kc, vc, *rest = parts(caches, pages, size, most, table)
    return m3.lib().m3_attn_step_kv8(v["q"], v["k"], v["v"], kc, vc, lengths, *rest, c or config(**kw), v["out"], ws,
                                     ws_bytes, None)


CALLS = [(write, "m3_kv8_write"), (read, "m3_kv8_read"), (step, "m3_attn_step_kv8")]
SHARED = [
    (dict(batch_size=0), "batch_size is 0"), (dict(q_length=0), "q_length is 0"), (dict(kv_length=0), "kv_length is 0"),
    (dict(num_heads=0), "num_heads is 0"), (dict(head_dim=0), "head_dim is 0"),
    (dict(num_groups=3), "num_groups 3 does not divide num_heads 4"), (dict(head_dim=129), "head_dim 129 is above"),
    (dict(block_size=0), "block_size 0 is not one of 16, 32, 64, 128"), (dict(block_size=8), "block_size 8 is not one"),
    (dict(block_size=48), "block_size 48 is not one"), (dict(block_size=256), "block_size 256 is not one"),
    (dict(scale=-1.0), "scale is -1"), (dict(scale=float("nan")), "scale is"),
    (dict(pages=0), "num_pages is 0"), (dict(size=0), "page_size is 0"), (dict(most=0), "max_pages is 0"),
    (dict(most=1), "kv_length 128 is above max_pages * page_size = 64"),
    (dict(table=None), "without a block_table each of the 2 rows has one page of its own"),
    (dict(table=None, pages=1, size=128, most=1), "num_pages is 1"),
    (dict(size=72), "page_size 72 is not a multiple of block_size 16"),
    (dict(caches={"k_cache": cache(codes=None)}), "operand k_cache is NULL"),
    (dict(caches={"v_cache": cache(scales=None)}), "the scales of operand v_cache are NULL"),
    (dict(caches={"v_cache": cache(row=63)}), "operand v_cache has a stride below head_dim 64"),
    (dict(caches={"k_cache": cache(head=0)}), "operand k_cache has a stride below head_dim 64"),
    (dict(caches={"k_cache": cache(row=64)}), "rows and heads must not overlap"),
    (dict(caches={"v_cache": cache(page=128 * 63)}), "rows and heads must not overlap"),
]


@pytest.mark.parametrize("bad,rule", SHARED, ids=lambda x: x if isinstance(x, str) else "")
@pytest.mark.parametrize("call,op", CALLS, ids=[op for _, op in CALLS])
def test_shared_rules(call, op, bad, rule):
    refused(call(**bad), op, rule)


@pytest.mark.parametrize("call,op", CALLS, ids=[op for _, op in CALLS])
def test_sizes_beyond_a_launch(call, op):
    for bad, rule in ((dict(batch_size=1 << 31), "more than one launch can cover"),
                      (dict(kv_length=1 << 31, most=1 << 26), "more than one launch can cover"),
                      (dict(num_heads=1 << 17, num_groups=1), "more than one launch can cover"),
                      (dict(pages=1 << 31), "num_pages is above 2^31 - 1"),
                      (dict(caches={"k_cache": cache(row=(1 << 26) + 8, page=1 << 40)}), "at most 67108864 codes apart")):
        refused(call(**bad), op, rule, UNSUPPORTED)
    many = dict(batch_size=1 << 24, pages=1 << 24, table=FAKE)
    if call is not step:
        many["total"] = 3 << 24
    refused(call(**many), op, "more than one launch can cover", UNSUPPORTED)


@pytest.mark.parametrize("call,op", CALLS[:2], ids=[op for _, op in CALLS[:2]])
def test_token_rules(call, op):
    refused(call(total=7), op, "total is 7; without offsets it is batch_size * q_length = 6")
    refused(call(offsets=FAKE, total=1 << 31), op, "total is above 2^31 - 1", UNSUPPORTED)
    refused(call(window=4), op, "window 4 and sinks 0 belong to m3_attn_step_kv8")
    refused(call(window=4, sinks=2), op, "window 4 and sinks 2 belong to m3_attn_step_kv8")
    for n in "kv":
        refused(call({n: view(data=None)}), op, f"operand {n} is NULL")
        refused(call({n: view(row=63)}), op, f"operand {n} has row_stride 63 below head_dim 64")
        refused(call({n: view(data=FAKE + 1)}), op, f"operand {n} is not aligned to its 2-byte elements")
    if call is read:
        refused(call({"k": view(row=64, head=64)}), op, "must not overlap")
        refused(call({"v": view(head=0)}), op, "heads must not overlap")
    else:
        refused(call(lengths=None), op, "lengths is NULL")


def test_no_tokens_are_no_work():
    """A call that cuts no tokens ends on the host, whatever its views point to."""
    none = {n: view(data=None) for n in "kv"}
    assert write(none, offsets=FAKE, total=0) == bd.M3_OK
    assert read(none, offsets=FAKE, total=0) == bd.M3_OK


def test_step_rules():
    op = "m3_attn_step_kv8"
    refused(step(sinks=2), op, "sinks 2 need a window")
    refused(step(q_length=65), op, "a step takes at most 64 tokens", UNSUPPORTED)
    for n in ("q", "k", "v", "out"):
        refused(step({n: view(data=None)}), op, f"operand {n} is NULL")
    refused(step({"out": view(row=64, head=64)}), op, "must not overlap")
    refused(step({"q": view(row=1 << 23)}), op, "rows may stand at most", UNSUPPORTED)
    refused(step(lengths=None), op, "lengths is NULL")
    # no keys and values at all is a call; the next rule speaks
    refused(step({n: view(data=None) for n in "kv"}, lengths=None), op, "lengths is NULL")
    long = dict(batch_size=1, kv_length=1 << 16, most=1 << 10, pages=1 << 10)
    need = m3.lib().m3_attn_step_kv8_workspace_bytes(config(**{k: v for k, v in long.items() if k in CFG}))
    assert need > 0
    refused(step(ws_bytes=need - 1, **long), op, f"workspace of {need} bytes required, {need - 1} given")
    refused(step(ws=None, **long), op, "workspace of")
    refused(step(ws=FAKE + 8, **long), op, "the workspace is not aligned to 16 bytes")


def test_bad_types_are_refused():
    c = config()
    c.dtype = 3
    bad = bd._CKv8.from_buffer_copy(bytes(c))
    for call, op in CALLS:
        refused(call(c=bad), op, "dtype 3 is not one of")
    assert ctypes.sizeof(bd._CKv8) == 44 and ctypes.sizeof(bd._CKv8Cache) == 40


def test_workspace_queries_of_broken_configs_are_zero():
    for bad in (dict(block_size=3), dict(num_groups=3), dict(q_length=65), dict(sinks=1)):
        assert m3.lib().m3_attn_step_kv8_workspace_bytes(config(**bad)) == 0


# ---- the binding's own checks (any device: they come before the launch) ----


def tensors(G=2, D=64, pages=4, size=32, block=16, rows=2):
    codes = torch.zeros(pages, size, G, D, dtype=torch.uint8).view(torch.float8_e4m3fn)
    scales = torch.zeros(pages, G, size // block, dtype=torch.uint8).view(torch.float8_e8m0fnu)
    return dict(k=torch.zeros(rows, G, D), v=torch.zeros(rows, G, D), k_cache=codes, k_scales=scales,
                v_cache=codes.clone(), v_scales=scales.clone(), lengths=torch.zeros(rows, dtype=torch.int32))


def cfg(**kw):
    return m3.Kv8Config(**{**dict(batch_size=2, q_length=1, kv_length=32, num_heads=4, num_groups=2, head_dim=64,
                                  block_size=16), **kw})


BAD = [
    (dict(k_cache=torch.zeros(4, 32, 2, 64)), TypeError, "k_cache must be torch.float8_e4m3fn"),
    (dict(v_cache=torch.zeros(4, 32, 2, 32, dtype=torch.uint8).view(torch.float8_e4m3fn)), ValueError, "v_cache has shape"),
    (dict(v_cache=torch.zeros(5, 32, 2, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)), ValueError, "v_cache has shape"),
    (dict(k_cache=torch.zeros(4, 32, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)), ValueError, "k_cache has shape"),
    (dict(k_cache=torch.zeros(4, 32, 64, 2, dtype=torch.uint8).view(torch.float8_e4m3fn).transpose(2, 3)), ValueError,
     "k_cache must be contiguous along its last axis"),
    (dict(k_cache=None), TypeError, "k_cache must be a torch.Tensor"),
    (dict(k_scales=torch.zeros(4, 2, 2, dtype=torch.uint8)), TypeError, "k_scales must be torch.float8_e8m0fnu"),
    (dict(v_scales=torch.zeros(4, 2, 3, dtype=torch.uint8).view(torch.float8_e8m0fnu)), ValueError, "v_scales has shape"),
    (dict(k_scales=torch.zeros(4, 2, 4, dtype=torch.uint8).view(torch.float8_e8m0fnu)[..., ::2]), ValueError,
     "k_scales must be contiguous"),
]


@pytest.mark.parametrize("bad,error,text", BAD, ids=[t for _, _, t in BAD])
def test_caches_of_other_kinds(bad, error, text):
    t = tensors() | bad
    caches = [t[n] for n in ("k_cache", "k_scales", "v_cache", "v_scales")]
    with pytest.raises(error, match=text):
        m3.m3_kv8_write(t["k"], t["v"], *caches, t["lengths"], cfg())
    with pytest.raises(error, match=text):
        m3.m3_attn_step_kv8(torch.zeros(2, 4, 64), t["k"], t["v"], *caches, t["lengths"], cfg())
    if t["k_cache"] is not None:
        with pytest.raises(error, match=text):
            m3.m3_kv8_read(*caches, cfg())


def test_other_arguments_of_the_binding():
    t = tensors()
    caches = [t[n] for n in ("k_cache", "k_scales", "v_cache", "v_scales")]
    with pytest.raises(ValueError, match="expected a GPU"):
        m3.m3_kv8_write(t["k"], t["v"], *caches, t["lengths"], cfg())
    with pytest.raises(ValueError, match="given together"):
        m3.m3_attn_step_kv8(torch.zeros(2, 4, 64), t["k"], None, *caches, t["lengths"], cfg())
    with pytest.raises(ValueError, match="total"):
        m3.m3_kv8_read(*caches, cfg(), offsets=t["lengths"])
    with pytest.raises(ValueError, match="block_table must be a tensor"):
        m3.m3_kv8_write(t["k"], t["v"], *caches, t["lengths"], cfg(), block_table=t["lengths"])
    with pytest.raises(TypeError, match="must be float32, bfloat16 or float16"):
        m3.m3_kv8_write(t["k"].double(), t["v"].double(), *caches, t["lengths"], cfg())
    with pytest.raises(TypeError, match="must be float32, bfloat16 or float16"):
        m3.m3_kv8_read(*caches, cfg(), dtype=torch.int32)
    with pytest.raises(ValueError, match="k has shape"):
        m3.m3_kv8_write(t["k"][0], t["v"], *caches, t["lengths"], cfg())
