"""Host-side refusals of outputs and caches whose rows, heads or pages lie over one another, before any HIP
call; and layouts that look like it and are none."""

import pytest

from test_abi_attn import bwd, cache, fwd, refused, rope, step, view

OVER = "must not overlap"

# rows 16, heads 4 (or 2) of 64: row stride, head stride
CROSSED = [(64, 64), (128, 64), (64, 128), (192, 128), (100, 300), (64, 16 * 64 - 64 - 1)]
APART = [(256, 64), (64, 16 * 64), (1000, 70), (64, 5000), (64, 16 * 64 + 3)]


@pytest.mark.parametrize("row,head", CROSSED)
def test_crossed_outputs_are_refused(row, head):
    for back in (False, True):
        op = "m3_qk_norm_rope" + "_bwd" * back
        refused(rope({"out_q": view(row=row, head=head)}, rows=16, bwd=back), op, OVER)
    refused(fwd({"out": view(row=row, head=head)}), "m3_attn_fwd", OVER)
    refused(bwd({"d_q": view(row=row, head=head)}), "m3_attn_bwd", OVER)
    refused(step({"out": view(row=row, head=head)}, batch_size=16, pages=16), "m3_attn_step", OVER)


@pytest.mark.parametrize("n", ["d_k", "d_v"])
def test_crossed_key_gradients_are_refused(n):
    refused(bwd({n: view(row=64, head=64)}), "m3_attn_bwd", f"operand {n} has row_stride 64 and head_stride 64")


@pytest.mark.parametrize("row,head", CROSSED)
def test_crossed_inputs_are_taken(row, head):
    """Inputs may share elements: the next rule is the one that speaks."""
    refused(fwd({n: view(row=row, head=head) for n in "qkv"}, lse=None), "m3_attn_fwd", "operand lse is NULL")


@pytest.mark.parametrize("row,head", APART)
def test_layouts_apart_are_taken(row, head):
    refused(fwd({"out": view(row=row, head=head)}, lse=None), "m3_attn_fwd", "operand lse is NULL")
    refused(bwd({"d_q": view(row=row, head=head)}, lse=None), "m3_attn_bwd", "operand lse is NULL")


def test_interleaved_layouts_are_told_from_crossed_ones():
    """Heads two places apart, rows five: rows 0 and 1 pass between one another, row 2 meets row 0's sixth head."""
    def out(rows, heads):
        return fwd({"out": view(row=5 * 64, head=2 * 64)}, totals=(rows, 32), batch_size=1, q_length=rows, kv_length=32,
                   num_heads=heads, num_groups=1, lse=None)
    for rows, heads in ((2, 4), (2, 6), (3, 5), (100, 2)):
        refused(out(rows, heads), "m3_attn_fwd", "operand lse is NULL")
    for rows, heads in ((3, 6), (100, 8)):
        refused(out(rows, heads), "m3_attn_fwd", OVER)


@pytest.mark.parametrize("bad", [dict(row=64), dict(head=64, row=64, page=64), dict(page=64), dict(page=128 * 63),
                                 dict(row=100, head=64), dict(row=64, head=64 * 63, page=64 * 126)])
@pytest.mark.parametrize("n", ["k_cache", "v_cache"])
def test_crossed_caches_are_refused(n, bad):
    refused(step(caches={n: cache(**bad)}), "m3_attn_step", OVER)


def test_rows_without_extent_have_any_stride():
    """One row cannot cross."""
    refused(fwd({"out": view(row=64, head=64)}, totals=(1, 32), batch_size=1, q_length=1, kv_length=32, lse=None), "m3_attn_fwd",
            "operand lse is NULL")


def test_many_pages_and_rows_are_checked_at_once():
    """2^20 pages of 2^20 positions: the answer does not take a walk over them."""
    big = dict(pages=1 << 20, size=1 << 20, batch_size=1, kv_length=1 << 20, num_groups=1, num_heads=1)
    refused(step(caches={"k_cache": cache(row=64 * 3, page=64 * 2)}, **big), "m3_attn_step", OVER)
    refused(step(caches={"k_cache": cache(row=(1 << 26) + 64, page=(1 << 26) + 129)}, **big), "m3_attn_step", OVER)
