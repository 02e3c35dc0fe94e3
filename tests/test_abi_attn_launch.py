"""Host-side refusals of calls that take more workgroups than one launch can hold (fewer than 2^32 threads), before any
HIP call, whichever of a call's kernels it is."""

import torch

import selective_state_space_mamba3_amd as m3
from test_abi_attn import FAKE, UNSUPPORTED, bwd, cache, fwd, refused, rope, step, view

RULE = "16777216 workgroups are more than one launch can cover (16777215)"


def rows(*names, heads, dim=64):
    """Contiguous operands of so many heads."""
    return {n: view(row=heads * dim, head=dim) for n in names}


def test_norm_rope_rows():
    refused(rope(rows=1 << 28, num_heads=1, num_groups=1, head_dim=2, num_rope_angles=1), "m3_qk_norm_rope", RULE, UNSUPPORTED)


def test_forward_sequences():
    n = 1 << 19
    refused(fwd(rows("q", "out", heads=32), batch_size=n, q_length=1, kv_length=1, num_heads=32, num_groups=1, totals=(n, n)),
            "m3_attn_fwd", RULE, UNSUPPORTED)


def test_backward_sequences():
    n = 1 << 19
    refused(bwd(rows("q", "out", "dout", "d_q", heads=32), batch_size=n, q_length=1, kv_length=1, num_heads=32, num_groups=1,
                totals=(n, n)), "m3_attn_bwd", RULE, UNSUPPORTED)


def test_backward_key_blocks():
    """The queries' launch is small, the keys' is not: refused before either runs."""
    refused(bwd(batch_size=64, q_length=1, kv_length=1 << 25, num_heads=1, num_groups=1, totals=(64, 1 << 30),
                offsets=(FAKE, FAKE)), "m3_attn_bwd", RULE, UNSUPPORTED)


def test_backward_joins():
    """Rows of no sequence count for the pass that adds the parts."""
    kw = dict(batch_size=1, q_length=64, kv_length=8192, num_heads=128, num_groups=128, head_dim=128, causal=False)
    small = m3.attn_bwd_workspace_bytes(m3.AttnConfig(**kw), torch.bfloat16, 64, 8192)
    assert small > 2 * 4 * 64 * 128  # the queries' sums are shared
    views = rows("q", "k", "v", "out", "dout", "d_q", "d_k", "d_v", heads=128, dim=128)
    refused(bwd(views, totals=(1 << 20, 8192), offsets=(FAKE, FAKE), ws_bytes=1 << 60, **kw), "m3_attn_bwd", RULE, UNSUPPORTED)


def test_step_rows():
    caches = {n: cache(page=64 * 1024, row=1024) for n in ("k_cache", "v_cache")}
    refused(step(rows("q", "k", "v", "out", heads=16), caches, batch_size=1 << 20, num_heads=16, num_groups=16, pages=1 << 20),
            "m3_attn_step", RULE, UNSUPPORTED)
