"""Prompts and single tokens of a hybrid model: a state space layer and an attention layer over a paged cache, with the
norms, the short convolution and the rotation around them.

    r = embed                     h = norm(r)                       add_rms_norm
    z, xBC, dt = h W_in           x, B, C = silu(conv(xBC))         short_conv (its history moves on)
    y = scan(x, dt, B, C) silu(z) W_out                             ssm_prefill_chunked, or ssm_decode_step for single tokens
    r += y                        h = norm(r)                       add_rms_norm
    q, k, v = h W_qkv             turned; k and v into the cache    attn_cache_append
    a = attention(q, cache) W_o                                     attn_paged
    r += a                        logits = norm(r) W_head           add_rms_norm

Prompts of several sequences are packed; one may come in pieces, and single tokens go on from there.  Weights are random: the
example shows the calls, not a language.  Run: python examples/hybrid_prompt.py
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import gated_deltanet_delta_gb300 as gdn

B16 = torch.bfloat16


class HybridModel:
    """N sequences with all that is kept of them between calls."""

    def __init__(self, N=3, vocab=500, hidden=512, heads=8, head_dim=64, groups=2, state=128, q_heads=8, kv_heads=2, attn_dim=128, page_size=16,
                 max_tokens=2048, e4m3=False, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(*shape, scale=None):
            return (torch.randn(shape, generator=g, device="cuda") * (shape[0] ** -0.5 if scale is None else scale)).to(B16)

        def f(*shape, low=0.0, high=1.0):
            return low + (high - low) * torch.rand(shape, generator=g, device="cuda")
        self.N, self.vocab, self.page_size, self.q_heads, self.kv_heads, self.attn_dim = N, vocab, page_size, q_heads, kv_heads, attn_dim
        self.heads, self.head_dim, self.groups, self.state_dim = heads, head_dim, groups, state
        inner, bc = heads * head_dim, groups * state
        self.splits = (inner, bc, bc)
        self.embed = w(vocab, hidden, scale=1.0)
        self.norms = [f(hidden, low=0.5, high=1.5) for _ in range(3)]
        self.w_in = w(hidden, 2 * inner + 2 * bc + heads)  # the gate, the convolution's channels, dt
        self.conv, self.conv_bias = f(sum(self.splits), 4, low=-0.5, high=0.5), f(sum(self.splits), low=-0.1, high=0.1)
        self.A_log, self.D, self.dt_bias = f(heads, high=2.0), f(heads, low=0.5, high=1.5), f(heads, low=-4.0, high=-1.0)
        self.w_out = w(inner, hidden)
        self.w_qkv = w(hidden, (q_heads + 2 * kv_heads) * attn_dim)
        self.w_o = w(q_heads * attn_dim, hidden)
        self.w_head = w(hidden, vocab)
        angle = torch.arange(max_tokens, device="cuda")[:, None] * 10000.0 ** (-torch.arange(attn_dim // 2, device="cuda") / (attn_dim // 2))
        self.rotation = torch.cat([angle.cos(), angle.sin()], 1)
        # what is kept: the convolution's history, the scan's state, the paged cache, the lengths
        self.hist = torch.zeros((N, sum(self.splits), 3), device="cuda")
        self.state = torch.zeros((N, heads, head_dim, state), device="cuda")
        self.slots = torch.arange(N, device="cuda")
        per_seq = -(-max_tokens // page_size)
        self.table = torch.randperm(N * per_seq, generator=g, device="cuda").reshape(N, per_seq)
        shape = (N * per_seq, kv_heads, page_size, attn_dim)
        self.cache = [torch.zeros(shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) if e4m3 else
                      torch.zeros(shape, dtype=B16, device="cuda") for _ in range(2)]
        self.scales = [torch.ones(shape[:3], device="cuda") if e4m3 else None for _ in range(2)]
        self.lens = torch.zeros(N, dtype=torch.int64, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.workspace = torch.empty(gdn.attn_paged_workspace_size(attn_dim), dtype=torch.uint8, device="cuda")

    def _norm(self, i, x, residual=None):
        return gdn.add_rms_norm(x, self.norms[i], residual, 1e-6)

    def _scan_layer(self, h, cu, longest):
        inner = self.splits[0]
        rows = h @ self.w_in
        z, xbc, dt = rows.split([inner, sum(self.splits), self.heads], 1)
        x, B, C = gdn.short_conv(xbc, self.conv, self.hist, self.slots, cu, bias=self.conv_bias, splits=self.splits, dev_status=self.status)
        x, z = x.unflatten(1, (self.heads, self.head_dim)), z.unflatten(1, (self.heads, self.head_dim))
        B, C = B.unflatten(1, (self.groups, self.state_dim)), C.unflatten(1, (self.groups, self.state_dim))
        args = (x, dt, B, C, self.A_log, self.dt_bias, self.state, self.slots)
        if cu is None:
            y = gdn.ssm_decode_step(*args, D=self.D, z=z, dev_status=self.status)
        else:
            y = gdn.ssm_prefill_chunked(*args, cu, longest, D=self.D, z=z, dev_status=self.status)
        return y.flatten(1) @ self.w_out

    def _attention(self, h, seq, positions, cu, longest):
        qkv = (h @ self.w_qkv).unflatten(1, (-1, self.attn_dim))
        q, k, v = qkv.split([self.q_heads, self.kv_heads, self.kv_heads], 1)  # slices of one row per token
        slots = self.table[seq, positions // self.page_size] * self.page_size + positions % self.page_size
        q = gdn.attn_cache_append(q, k, v, self.rotation, positions, slots, *self.cache, *self.scales, dev_status=self.status)
        out = gdn.attn_paged(q, *self.cache, self.table, self.lens, cu, longest, k_scale=self.scales[0], v_scale=self.scales[1],
                             workspace=self.workspace, dev_status=self.status)
        return out.flatten(1) @ self.w_o

    def _run(self, tokens, seq, positions, cu_scan, cu, longest):
        r = self.embed[tokens]  # the residual stream: the norms add to it in place
        h = self._norm(0, r)
        h = self._norm(1, self._scan_layer(h, cu_scan, longest), r)
        h = self._norm(2, self._attention(h, seq, positions, cu, longest), r)
        return h, h @ self.w_head

    def prompt(self, tokens, counts):
        """The next counts[n] tokens of each sequence, packed in `tokens` [T]; returns the last norm's rows and the logits."""
        n = torch.tensor(counts, device="cuda")
        cu = torch.nn.functional.pad(n.cumsum(0), (1, 0))
        seq = torch.repeat_interleave(self.slots, n)
        positions = self.lens[seq] + torch.arange(len(tokens), device="cuda") - cu[seq]
        self.lens += n
        return self._run(tokens, seq, positions, cu, cu, max(counts))

    def step(self, tokens):
        """One token of every sequence [N].  Nothing of it depends on the host: it can be captured in a CUDA graph."""
        positions = self.lens.clone()
        self.lens += 1
        return self._run(tokens, self.slots, positions, None, torch.arange(self.N + 1, device="cuda"), 1)


def main(steps=8):
    model = HybridModel(e4m3=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    counts = [300, 17, 131]
    _, logits = model.prompt(torch.randint(model.vocab, (sum(counts),), generator=g, device="cuda"), counts)
    last = logits[torch.tensor(counts, device="cuda").cumsum(0) - 1].argmax(-1)
    for i in range(steps):
        _, logits = model.step(last)
        last = logits.argmax(-1)
        print(f"step {i}: tokens {last.tolist()}, lengths {model.lens.tolist()}")
    assert int(model.status.item()) == 0


if __name__ == "__main__":
    main()
