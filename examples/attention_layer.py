"""A softmax-attention layer that stands between scan layers, trained and then served with the library.

    python examples/attention_layer.py

One layer of 6 heads of 64 that share 2 key / value heads: projection rows [q | k | v] from the token's
features, per-head norm with rotation, causal attention, output projection.  The layer learns to follow
a teacher of the same shape by plain gradient descent through m3_attn_bwd and m3_qk_norm_rope_bwd; then
it reads a prompt into a cache of pages and decodes token by token with m3_attn_step, and the decoded rows
are compared with those of one pass over the whole sequence.  Last, the same with a cache of 8 bits (m3_kv8_write,
m3_attn_step_kv8, a few tokens at a time), compared with attention over what m3_kv8_read says the cache holds.
"""

from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import selective_state_space_mamba3_amd as m3  # noqa: E402

HEADS, GROUPS, DIM, WIDTH = 6, 2, 64, 384
ROPE = m3.QkNormRopeConfig(num_heads=HEADS, num_groups=GROUPS, head_dim=DIM, num_rope_angles=DIM // 2)


class AttentionLayer:
    def __init__(self, seed: int, dtype=torch.bfloat16):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.dtype = dtype
        self.weights = {
            "in": torch.randn(WIDTH, (HEADS + 2 * GROUPS) * DIM, generator=gen, device="cuda") * WIDTH ** -0.5,
            "out": torch.randn(HEADS * DIM, WIDTH, generator=gen, device="cuda") * (HEADS * DIM) ** -0.5,
            "q": torch.ones(DIM, device="cuda"), "k": torch.ones(DIM, device="cuda")}
        self.inv_freq = 10000.0 ** (-torch.arange(DIM // 2, device="cuda", dtype=torch.float32) / (DIM // 2))

    def project(self, x):
        """q, k and v as views of the packed projection rows."""
        row = x @ self.weights["in"].to(self.dtype)
        cut = HEADS * DIM, (HEADS + GROUPS) * DIM
        return (row[:, :cut[0]].unflatten(1, (HEADS, DIM)), row[:, cut[0]:cut[1]].unflatten(1, (GROUPS, DIM)),
                row[:, cut[1]:].unflatten(1, (GROUPS, DIM)))

    def normed(self, q, k, positions):
        y = m3.m3_qk_norm_rope(q, k, positions, self.inv_freq, self.weights["q"], self.weights["k"], ROPE)
        return y["q"], y["k"]

    def forward(self, x, offsets, longest):
        """x [tokens, WIDTH], sequences of any lengths behind one another; keeps what the backward pass reads."""
        positions = token_positions(offsets, x.shape[0])
        q, k, v = self.project(x)
        qn, kn = self.normed(q, k, positions)
        cfg = m3.AttnConfig(batch_size=offsets.numel() - 1, q_length=longest, kv_length=longest, num_heads=HEADS,
                            num_groups=GROUPS, head_dim=DIM)
        o, lse = m3.m3_attn_fwd(qn, kn, v, cfg, q_offsets=offsets, kv_offsets=offsets)
        self.kept = x, positions, q, k, v, qn, kn, o, lse, cfg, offsets
        return o.flatten(1) @ self.weights["out"].to(self.dtype)

    def backward(self, dy):
        """Gradients of the weights from the gradient of the last forward pass's result."""
        x, positions, q, k, v, qn, kn, o, lse, cfg, offsets = self.kept
        do = (dy @ self.weights["out"].to(self.dtype).T).unflatten(1, (HEADS, DIM))
        rows = torch.empty(x.shape[0], self.weights["in"].shape[1], dtype=self.dtype, device="cuda")
        cut = HEADS * DIM, (HEADS + GROUPS) * DIM
        dq, dk = rows[:, :cut[0]].unflatten(1, (HEADS, DIM)), rows[:, cut[0]:cut[1]].unflatten(1, (GROUPS, DIM))
        dv = rows[:, cut[1]:].unflatten(1, (GROUPS, DIM))
        # the gradients go straight into the projection rows; the norm's replace the attention's in place
        m3.m3_attn_bwd(do, qn, kn, v, o, lse, cfg, q_offsets=offsets, kv_offsets=offsets,
                       grads={"q": dq, "k": dk, "v": dv})
        w = m3.m3_qk_norm_rope_bwd(dq, dk, q, k, positions, self.inv_freq, self.weights["q"], self.weights["k"], ROPE,
                                   grads={"q": dq, "k": dk})
        return {"in": x.T.float() @ rows.float(), "out": o.flatten(1).T.float() @ dy.float(), "q": w["q_weight"],
                "k": w["k_weight"]}

    def decode(self, x, k_cache, v_cache, lengths, table):
        """One token for each row of x [rows, WIDTH], lengths[b] positions already in the caches."""
        q, k, v = self.project(x)
        qn, kn = self.normed(q, k, lengths)
        cfg = m3.AttnConfig(batch_size=x.shape[0], q_length=1, kv_length=table.shape[1] * k_cache.shape[1],
                            num_heads=HEADS, num_groups=GROUPS, head_dim=DIM)
        o = m3.m3_attn_step(qn, kn, v, k_cache, v_cache, lengths, cfg, block_table=table)
        return o.flatten(1) @ self.weights["out"].to(self.dtype)

    def decode_8bit(self, x, caches, lengths, table, tokens, block):
        """`tokens` tokens of each row, x [rows * tokens, WIDTH], into and against an 8-bit cache."""
        rows, page = lengths.numel(), caches[0].shape[1]
        q, k, v = self.project(x)
        positions = (lengths[:, None] + torch.arange(tokens, device="cuda", dtype=torch.int32)).flatten()
        qn, kn = self.normed(q, k, positions)
        cfg = m3.Kv8Config(batch_size=rows, q_length=tokens, kv_length=table.shape[1] * page, num_heads=HEADS,
                           num_groups=GROUPS, head_dim=DIM, block_size=block)
        o = m3.m3_attn_step_kv8(qn, kn, v, *caches, lengths, cfg, block_table=table)
        return o.flatten(1) @ self.weights["out"].to(self.dtype)


def token_positions(offsets, tokens):
    """Position of each token in its sequence."""
    at = torch.arange(tokens, device="cuda", dtype=torch.int32)
    return at - offsets[torch.searchsorted(offsets, at, right=True) - 1]


def train(steps=40, lengths=(129, 64, 200, 1), rate=0.02):
    """The student's loss against the teacher before and after `steps` of gradient descent."""
    teacher, student = AttentionLayer(1), AttentionLayer(2)
    offsets = torch.tensor([0, *torch.tensor(lengths).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    x = torch.randn(sum(lengths), WIDTH, generator=gen, device="cuda").to(student.dtype)
    want = teacher.forward(x, offsets, max(lengths)).float()
    losses = []
    for _ in range(steps):
        err = student.forward(x, offsets, max(lengths)).float() - want
        losses.append(err.square().mean().item())
        dy = (2 * err / err.shape[0]).to(student.dtype)
        for name, g in student.backward(dy).items():
            student.weights[name] -= rate * g
    return student, losses


def serve(layer, rows=3, prompt=70, tokens=60, page=16):
    """The largest difference between rows decoded from a paged cache and those of one whole pass, and the rows' size."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    total, per = prompt + tokens, -(-(prompt + tokens) // page)
    x = torch.randn(rows, total, WIDTH, generator=gen, device="cuda").to(layer.dtype)
    offsets = torch.arange(rows + 1, device="cuda", dtype=torch.int32) * total
    whole = layer.forward(x.flatten(0, 1), offsets, total).view(rows, total, WIDTH)
    _, _, _, _, v, _, kn, *_ = layer.kept
    table = torch.randperm(rows * per, generator=gen, device="cuda").to(torch.int32).view(rows, per)
    k_cache = torch.zeros(rows * per, page, GROUPS, DIM, dtype=layer.dtype, device="cuda")
    v_cache = torch.zeros_like(k_cache)
    at = torch.arange(prompt, device="cuda")  # the prompt's keys and values, page by page
    for c, src in ((k_cache, kn), (v_cache, v)):
        c[table[:, at // page].long(), at % page] = src.view(rows, total, GROUPS, DIM)[:, :prompt]
    lengths = torch.full((rows,), prompt, dtype=torch.int32, device="cuda")
    out = []
    for t in range(tokens):
        out.append(layer.decode(x[:, prompt + t], k_cache, v_cache, lengths, table))
        lengths += 1
    diff = (torch.stack(out, 1).float() - whole[:, prompt:].float()).abs().max()
    return diff.item(), whole.float().abs().max().item()


def serve_8bit(layer, rows=3, prompt=70, tokens=60, at_once=4, page=32, block=16):
    """Rows decoded a few at a time from an 8-bit cache: their largest difference from attention over the values that the
    cache stands for, from one pass over the whole sequence, and that pass's size."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    total, per = prompt + tokens, -(-(prompt + tokens) // page)
    x = torch.randn(rows, total, WIDTH, generator=gen, device="cuda").to(layer.dtype)
    offsets = torch.arange(rows + 1, device="cuda", dtype=torch.int32) * total
    whole = layer.forward(x.flatten(0, 1), offsets, total).view(rows, total, WIDTH)
    _, _, _, _, v, qn, kn, *_ = layer.kept
    table = torch.randperm(rows * per, generator=gen, device="cuda").to(torch.int32).view(rows, per)
    codes = [torch.zeros(rows * per, GROUPS, page, DIM, dtype=torch.uint8, device="cuda").transpose(1, 2) for _ in "kv"]
    scales = [torch.zeros(rows * per, GROUPS, page // block, dtype=torch.uint8, device="cuda") for _ in "kv"]
    caches = [t for c, s in zip(codes, scales) for t in (c.view(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu))]

    def config(n):
        return m3.Kv8Config(batch_size=rows, q_length=n, kv_length=per * page, num_heads=HEADS, num_groups=GROUPS,
                            head_dim=DIM, block_size=block)

    lengths = torch.zeros(rows, dtype=torch.int32, device="cuda")
    first = [t.view(rows, total, GROUPS, DIM)[:, :prompt].flatten(0, 1) for t in (kn, v)]
    m3.m3_kv8_write(*first, *caches, lengths, config(prompt), block_table=table)
    lengths += prompt
    out = []
    for t in range(0, tokens, at_once):
        n = min(at_once, tokens - t)
        new = x[:, prompt + t:prompt + t + n].flatten(0, 1)
        out.append(layer.decode_8bit(new, caches, lengths, table, n, block).view(rows, n, WIDTH))
        lengths += n
    # the same rows in one pass over what the cache holds now
    held = m3.m3_kv8_read(*caches, config(total), block_table=table, dtype=layer.dtype)
    ends = torch.arange(rows + 1, device="cuda", dtype=torch.int32) * tokens
    last = qn.view(rows, total, HEADS, DIM)[:, prompt:].flatten(0, 1)
    cfg = m3.AttnConfig(batch_size=rows, q_length=tokens, kv_length=total, num_heads=HEADS, num_groups=GROUPS, head_dim=DIM)
    o, _ = m3.m3_attn_fwd(last, held["k"], held["v"], cfg, q_offsets=ends, kv_offsets=offsets)
    same = (o.flatten(1) @ layer.weights["out"].to(layer.dtype)).view(rows, tokens, WIDTH).float()
    got = torch.cat(out, 1).float()
    return ((got - same).abs().max().item(), (got - whole[:, prompt:].float()).abs().max().item(),
            whole.float().abs().max().item())


if __name__ == "__main__":
    layer, losses = train()
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    diff, size = serve(layer)
    print(f"decoded rows against one whole pass: {diff:.4f} of {size:.2f}")
    held, diff, size = serve_8bit(layer)
    print(f"decoded from 8 bits: {held:.4f} from what the cache holds, {diff:.4f} from the whole pass, of {size:.2f}")
