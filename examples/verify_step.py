"""Speculative decoding steps of a small random decoder over the paged 8-bit KV cache.

The target model is a stack of attention layers with random weights (the library's part of a real one).
Prompts of uneven lengths are appended; then each step drafts a random candidate tree, scores all of its
nodes in one pass (append, attention over the cache and the node's ancestors, LM head), verifies it
greedily and keeps the accepted path in every layer's cache. Half of the drafted tokens are what the
target itself prefers, so that paths of some length are accepted.

    python examples/verify_step.py [--steps 4] [--batch 4] [--nodes 16] [--layers 2]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_78_gb300 as sv   # noqa: E402


class Target:
    """Random decoder: embedding, `layers` of pre-norm attention, LM head; bf16."""

    def __init__(self, vocab, layers, q_heads, kv_heads, head_dim, max_len, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        hidden = q_heads * head_dim
        rand = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5).bfloat16()
        self.shape = (q_heads, kv_heads, head_dim)
        self.embed = (torch.randn(vocab, hidden, generator=g, device="cuda")).bfloat16()
        self.qkv = [rand((q_heads + 2 * kv_heads) * head_dim, hidden) for _ in range(layers)]
        self.proj = [rand(hidden, hidden) for _ in range(layers)]
        self.head = rand(vocab, hidden)
        inv = 10000.0 ** (-torch.arange(0, head_dim, 2, device="cuda", dtype=torch.float64) / head_dim)
        angle = torch.arange(max_len, device="cuda", dtype=torch.float64)[:, None] * inv
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float()

    def logits(self, tokens, cache, table, lens, status, mask=None, new_lens=None):
        """Scores tokens [B, N], which are appended to the cache at slots lens[b] ..: [B, N, vocab]."""
        B, N = tokens.shape
        Hq, Hkv, D = self.shape
        x = self.embed[tokens.long()]
        for i, (qkv, proj) in enumerate(zip(self.qkv, self.proj)):
            h = torch.nn.functional.rms_norm(x, x.shape[-1:]) @ qkv.T
            q, k, v = h.view(B, N, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], 2)
            q, _ = sv.kv_append(cache, table, lens, k, v, q=q, rope=self.rope, layer=i, mask=mask,
                                new_lens=new_lens, status=status)
            a, _, _ = sv.kv_attention(cache, table, lens, q, layer=i, mask=mask, new_lens=new_lens,
                                      status=status)
            x = x + a.view(B, N, -1) @ proj.T
        return (torch.nn.functional.rms_norm(x, x.shape[-1:]) @ self.head.T).float()


def run(steps=4, batch=4, nodes=16, layers=2, vocab=512, q_heads=8, kv_heads=2, head_dim=64,
        page=16, seed=0):
    """Returns (tokens emitted per sequence, lengths of the caches, status)."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    prompt = 40
    pages_per_seq = -(-(prompt + (steps + 1) * nodes) // page)
    cache = sv.new_kv_cache(batch * pages_per_seq, kv_heads, head_dim, page, layers)
    table = torch.randperm(batch * pages_per_seq, generator=g, device="cuda").int()
    table = table.view(batch, pages_per_seq)
    model = Target(vocab, layers, q_heads, kv_heads, head_dim, pages_per_seq * page, seed)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    # the prompts: one chain of up to `prompt` tokens a sequence
    sizes = torch.randint(prompt // 2, prompt + 1, (batch,), generator=g, device="cuda").int()
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    text = torch.randint(0, vocab, (batch, prompt), generator=g, device="cuda").int()
    logits = model.logits(text, cache, table, lens, status, new_lens=sizes)
    root = logits[torch.arange(batch, device="cuda"), sizes.long() - 1].argmax(-1).int()
    lens = sizes.clone()
    emitted = [[int(t)] for t in root]

    for _ in range(steps):
        # a random tree below the last emitted token; node i's parent is one of the few before it
        parents = torch.full((batch, nodes), -1, dtype=torch.int32, device="cuda")
        for i in range(1, nodes):
            parents[:, i] = torch.randint(max(0, i - 4), i, (batch,), generator=g, device="cuda").int()
        mask, _ = sv.tree_mask(parents)
        drafts = torch.randint(0, vocab, (batch, nodes), generator=g, device="cuda").int()
        drafts[:, 0] = root
        # a stand-in for a good drafter: every other node takes the target's own choice at its parent
        for i in range(1, nodes, 2):
            peek = model.logits(drafts, cache, table, lens, status, mask=mask).argmax(-1).int()
            drafts[:, i] = peek.gather(1, parents[:, i:i + 1].long())[:, 0]
        scores = model.logits(drafts, cache, table, lens, status, mask=mask)
        accepted, path, out, _ = sv.verify_tree(scores, parents, drafts)
        lens, _ = sv.kv_commit(cache, table, lens, path, accepted, status=status)
        for b in range(batch):
            new = out[b, :int(accepted[b]) + 1].tolist()
            emitted[b] += new
            root[b] = new[-1]
    return emitted, lens, status


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("steps", 4), ("batch", 4), ("nodes", 16), ("layers", 2)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    emitted, lens, status = run(a.steps, a.batch, a.nodes, a.layers)
    sv.check(int(status.item()), "the steps")
    for b, tokens in enumerate(emitted):
        print(f"sequence {b}: {len(tokens)} tokens in {a.steps} steps, cache length {int(lens[b])}")
