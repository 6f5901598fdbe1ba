"""One step of speculative decoding around the masked head, with every operator that stands next to it:

    hidden -> 4-bit projection -> append to the 8-bit cache -> attention over it -> 4-bit projection
           -> masked head: draft tokens
           -> 4-bit head over the whole vocabulary: the verifier's logits -> log probabilities of the drafts
    and, for training the draft model, the gradient of those log probabilities.

Random weights and prompts; `python examples/speculative_step.py` prints the drafts and what the verifier
thinks of them.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import centroid_masked_sparse_gb300 as mtp  # noqa: E402


class Model:
    """A draft layer (4-bit projections, an 8-bit cache) and the two heads over one vocabulary."""

    def __init__(self, hidden=256, heads=8, kv_heads=2, dim=64, vocab=8192, clusters=64, top_k=8, batch=4, page=32,
                 longest=256, device="cuda", seed=0):
        self.gen = torch.Generator(device).manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.batch, self.hidden = heads, kv_heads, dim, batch, hidden

        def weight(rows, cols):
            return (torch.randn(rows, cols, device=device, generator=self.gen) * cols ** -0.5).to(torch.bfloat16)

        self.qkv = mtp.Q4Weight.quantize(weight((heads + 2 * kv_heads) * dim, hidden), group=64)
        self.output = mtp.Q4Weight.quantize(weight(hidden, heads * dim), group=64)
        embed = weight(vocab, hidden)
        self.verifier = mtp.Q4Weight.quantize(embed, group=64, zeros=True)
        order = torch.randperm(vocab, device=device, generator=self.gen).to(torch.int32)
        self.head = mtp.MaskedHead(weight(clusters, hidden), embed, order, top_k)
        width = -(-longest // page)
        self.cache = mtp.KvCache.allocate(batch * width, page, kv_heads, dim, "e4m3", device)
        self.table = torch.arange(batch * width, dtype=torch.int32, device=device).view(batch, width)
        self.lengths = torch.zeros(batch, dtype=torch.int32, device=device)

    def states(self, tokens):
        return torch.randn(tokens, self.hidden, device=self.table.device, generator=self.gen).to(torch.bfloat16)

    def attend(self, hidden, new):
        """`new` tokens of every sequence through the draft layer: into the cache, attention, back to hidden states."""
        fused = mtp.mtp_q4_matvec(self.qkv, hidden, out_dtype=torch.bfloat16).view(hidden.shape[0], -1, self.dim)
        q, k, v = fused.split([self.heads, self.kv_heads, self.kv_heads], dim=1)
        mtp.mtp_kv_append(self.cache, self.table, self.lengths, k, v)
        self.lengths += new
        out, _ = mtp.mtp_kv_attention(self.cache, self.table, self.lengths, q)
        return hidden + mtp.mtp_q4_matvec(self.output, out.flatten(1), out_dtype=torch.bfloat16)


def speculative_step(model, hidden):
    """(draft tokens [B], the verifier's logits [B, V], TokenLogprobs of the drafts with five alternatives)."""
    state = model.attend(hidden, 1)
    drafts, _ = mtp.mtp_masked_topk_tokens(model.head, state)
    logits = mtp.mtp_q4_matvec(model.verifier, state, softcap=30.0)
    return drafts, logits, mtp.mtp_token_logprobs(logits, drafts, top=5)


def main():
    model = Model()
    model.attend(model.states(model.batch * 21), 21)   # prompts of 21 tokens
    for step in range(3):
        drafts, logits, scored = speculative_step(model, model.states(model.batch))
        for b in range(model.batch):
            print(f"step {step} sequence {b}: draft {int(drafts[b])} logprob {float(scored.logprob[b]):.3f} rank "
                  f"{int(scored.rank[b])} entropy {float(scored.entropy[b]):.3f} instead of {scored.top_ids[b].tolist()}")
    assert model.cache.read_errors() == 0
    # training the draft model on the same tokens: the loss's gradient with respect to the logits
    leaf = logits.requires_grad_()
    loss = -mtp.token_logprobs(leaf, drafts)[0].mean()
    loss.backward()
    print(f"loss {float(loss.detach()):.4f}, |gradient| {float(leaf.grad.norm()):.4f}")


if __name__ == "__main__":
    main()
