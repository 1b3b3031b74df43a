"""Drafted decoding of a hybrid model: a recurrent layer (fused decode window) and an attention layer over
a paged, quantised cache, with the drafted tokens verified against the model's own probabilities.

One step of N sequences works on a window of T + 1 tokens each: the token sampled last, whose effects are
in neither the state nor the cache yet, and T drafted ones.
  1. gdn_window_fused in verify mode: the recurrent layer's outputs; its state is not written.
  2. attn_cache_write: the window's keys and values enter the cache behind the committed tokens.
  3. attn_paged: the window's tokens attend to the cache, each up to its own position.
  4. draft_verify: how many drafts stand, and the token that follows them.
  5. gdn_window_fused with the commit code of the accepted prefix; the cache needs no such thing: its
     length moves on by the accepted tokens, and what lies behind it is never read.

Weights are random: the example shows the calls, not a language.  Run: python examples/hybrid_decode.py
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import gated_deltanet_delta_gb300 as gdn

HEAD = 128  # head width of both layers


class HybridModel:
    """Embedding, one recurrent layer, one attention layer, output head; N sequences with their state."""

    def __init__(self, N=4, vocab=500, hidden=256, h_k=2, h_v=4, q_heads=8, kv_heads=2, page_size=16, max_tokens=512, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(*shape, scale=None):
            return torch.randn(shape, generator=g, device="cuda") * (shape[0] ** -0.5 if scale is None else scale)
        self.N, self.vocab, self.h_k, self.h_v, self.q_heads, self.kv_heads, self.page_size = N, vocab, h_k, h_v, q_heads, kv_heads, page_size
        self.embed = w(vocab, hidden, scale=1.0)
        C = (2 * h_k + h_v) * HEAD
        # the recurrent layer is the first: its projections depend on the token alone, so they are laid out by token
        self.qkv_of, self.alpha_of, self.beta_of, self.z_of = (self.embed @ w(hidden, n) for n in (C, h_v, h_v, h_v * HEAD))
        self.conv = w(C, 4, scale=0.5)
        self.dt, self.ssm_a, self.gamma = w(h_v, scale=0.5), -torch.rand(h_v, generator=g, device="cuda") - 0.5, torch.ones(HEAD, device="cuda")
        self.w_rec = w(h_v * HEAD, hidden)
        self.w_attn = w(hidden, (q_heads + 2 * kv_heads) * HEAD)
        self.w_out = w(q_heads * HEAD, hidden)
        self.head = w(hidden, vocab, scale=4 * hidden ** -0.5)
        # what is kept from step to step: the recurrent state, the convolution's history, the paged cache
        self.state = torch.zeros((N, HEAD, h_v, HEAD), device="cuda")
        self.hist = torch.zeros((N, C, 3), device="cuda")
        per_seq = -(-max_tokens // page_size)
        pages = N * per_seq
        self.table = torch.randperm(pages, generator=g, device="cuda").reshape(N, per_seq)
        shape = (pages, kv_heads, page_size, HEAD)
        self.k_cache, self.v_cache = (torch.zeros(shape, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
        self.k_scale, self.v_scale = (torch.ones(shape[:3], device="cuda") for _ in range(2))
        self.lens = torch.zeros(N, dtype=torch.int64, device="cuda")  # committed tokens
        self.workspace = torch.empty(gdn.attn_paged_workspace_size(HEAD), dtype=torch.uint8, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def _recurrent(self, tokens, commit, rows=slice(None)):
        """The recurrent layer on the window tokens [n, W] of the sequences `rows` (a slice)."""
        state, hist = self.state[rows], self.hist[rows]
        n, W = tokens.shape
        hist_out = torch.empty_like(hist)
        y = gdn.gdn_window_fused(state, hist, hist_out, self.qkv_of[tokens], self.alpha_of[tokens], self.beta_of[tokens],
                                 self.z_of[tokens].reshape(n, W, self.h_v, HEAD), self.conv, self.dt, self.ssm_a, self.gamma, self.h_k,
                                 commit)
        if commit:
            hist.copy_(hist_out)
        return y.reshape(n, W, -1) @ self.w_rec

    def _attention(self, x):
        N, W, _ = x.shape
        qkv = (x @ self.w_attn).to(torch.bfloat16).reshape(N * W, -1, HEAD)
        q, k, v = qkv.split([self.q_heads, self.kv_heads, self.kv_heads], 1)  # slices of one row per token
        pos = self.lens[:, None] + torch.arange(W, device="cuda")
        slots = self.table.gather(1, pos // self.page_size) * self.page_size + pos % self.page_size
        gdn.attn_cache_write(k, v, slots.reshape(-1), self.k_cache, self.v_cache, self.k_scale, self.v_scale, dev_status=self.status)
        cu = torch.arange(0, N * W + 1, W, device="cuda")
        out = gdn.attn_paged(q, self.k_cache, self.v_cache, self.table, self.lens + W, cu, W, k_scale=self.k_scale,
                             v_scale=self.v_scale, workspace=self.workspace, dev_status=self.status)
        return out.float().reshape(N, W, -1) @ self.w_out

    def probabilities(self, tokens):
        """The next-token distributions [N, W, vocab] of the windows `tokens` [N, W]; nothing is committed."""
        h = self.embed[tokens] + self._recurrent(tokens, 0)
        h = h + self._attention(h)
        return torch.softmax(h @ self.head / h.norm(dim=-1, keepdim=True), -1)

    def commit(self, tokens, counts):
        """Sequence n moves on by the first counts[n] tokens of its window."""
        for n, c in enumerate(counts):
            self._recurrent(tokens[n:n + 1], 0x100 | c, slice(n, n + 1))
        self.lens += torch.tensor(counts, device="cuda")

    def step(self, last, drafts, draft_p, u_accept, u_sample):
        """One drafted step.  last [N]: the tokens sampled before; drafts [N, T] with the distributions they
        were drawn from.  Returns (accepted [N], tokens [N, T + 1]), the new tokens of each sequence."""
        window = torch.cat([last[:, None], drafts], 1)
        accepted, tokens = gdn.draft_verify(self.probabilities(window), draft_p, drafts, u_accept, u_sample, dev_status=self.status)
        self.commit(window, [c + 1 for c in accepted.tolist()])  # the last sampled token, and the drafts that stand
        return accepted, tokens


def main(steps=6, T=4):
    model = HybridModel()
    g = torch.Generator(device="cuda").manual_seed(1)
    last = torch.randint(model.vocab, (model.N,), generator=g, device="cuda")
    for i in range(steps):
        # a stand-in for a draft model: the target's own distribution one token ahead, flattened
        p = model.probabilities(last[:, None])
        draft_p = (0.7 * p + 0.3 / model.vocab).expand(-1, T, -1).contiguous()
        drafts = torch.multinomial(draft_p.reshape(-1, model.vocab), 1, generator=g).reshape(model.N, T)
        accepted, tokens = model.step(last, drafts, draft_p, torch.rand((model.N, T), generator=g, device="cuda"),
                                      torch.rand(model.N, generator=g, device="cuda"))
        last = tokens.gather(1, accepted[:, None]).squeeze(1)
        print(f"step {i}: accepted {accepted.tolist()}, lengths {model.lens.tolist()}")
    assert int(model.status.item()) == 0


if __name__ == "__main__":
    main()
