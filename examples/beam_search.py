"""Beam search with a small random decoder over the paged 8-bit KV cache, with a sliding window.

The decoder is the one of verify_step.py, its attention over the last `window` tokens and the first `sinks`.
Prompts are appended once; their first step makes `beams` hypotheses of each, and from there on every step
gives the new tokens' places pages, scores them, selects the best continuations, forks the caches by their
parents, reorders the histories and gives back the pages behind the window. Now and then the pool is
compacted. A hypothesis that emits the end token stays as it is.

    python examples/beam_search.py [--steps 24] [--batch 4] [--beams 4] [--window 48]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_78_gb300 as sv   # noqa: E402
from verify_step import Target   # noqa: E402


class WindowedTarget(Target):
    """The decoder with a sliding window and sinks in every layer."""

    def __init__(self, window, sinks, *args, **kw):
        super().__init__(*args, **kw)
        self.window, self.sinks = window, sinks

    def logits(self, tokens, cache, table, lens, status, new_lens=None):
        B, N = tokens.shape
        Hq, Hkv, D = self.shape
        x = self.embed[tokens.long()]
        for i, (qkv, proj) in enumerate(zip(self.qkv, self.proj)):
            h = torch.nn.functional.rms_norm(x, x.shape[-1:]) @ qkv.T
            q, k, v = h.view(B, N, Hq + 2 * Hkv, D).split([Hq, Hkv, Hkv], 2)
            q, _ = sv.kv_append(cache, table, lens, k, v, q=q, rope=self.rope, layer=i, new_lens=new_lens,
                                status=status)
            a, _, _ = sv.kv_attention(cache, table, lens, q, layer=i, new_lens=new_lens, status=status,
                                      window=self.window, sinks=self.sinks)
            x = x + a.view(B, N, -1) @ proj.T
        return (torch.nn.functional.rms_norm(x, x.shape[-1:]) @ self.head.T).float()


def run(steps=24, batch=4, beams=4, window=48, sinks=4, layers=2, vocab=512, q_heads=8, kv_heads=2,
        head_dim=64, page=16, end=1, compact_every=8, seed=0, trace=None):
    """Returns (histories [batch, beams, steps], scores [batch, beams], (cache, refs, table, lens), status).
    `trace` gets (logits, scores, done, tokens, parents, best) of every selection."""
    dev, C = "cuda", batch * beams
    g = torch.Generator(device=dev).manual_seed(seed + 1)
    prompt = 40
    span = -(-(prompt + steps) // page)
    held = -(-(window + sinks) // page) + 3   # pages that a hypothesis holds at most, once some are behind it
    cache = sv.new_kv_cache(batch * span + C * held, kv_heads, head_dim, page, layers)
    refs = sv.new_page_refs(cache)
    model = WindowedTarget(window, sinks, vocab, layers, q_heads, kv_heads, head_dim, prompt + steps, seed)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    text = torch.randint(2, vocab, (batch, prompt), generator=g, device=dev).int()
    table = torch.full((batch, span), -1, dtype=torch.int32, device=dev)
    lens = torch.zeros(batch, dtype=torch.int32, device=dev)

    # the prompts, uneven; each is one beam until its first selection
    sizes = torch.randint(prompt // 2, prompt + 1, (batch,), generator=g, device=dev).int()
    new, _ = sv.kv_reserve(cache, refs, table, lens, prompt, new_lens=sizes, status=status)
    x = model.logits(text, cache, table, lens, status, new_lens=new)
    lens += new
    logits = x[torch.arange(batch, device=dev), lens.long() - 1].view(batch, 1, vocab)
    scores = torch.zeros(batch, 1, device=dev)
    done = torch.zeros(batch, 1, dtype=torch.int32, device=dev)
    history = torch.zeros(batch, steps, dtype=torch.int32, device=dev)
    for step in range(steps):
        tokens, parents, best, _ = sv.beam_select(logits, scores, beams, done=done, pad_token=end, status=status)
        if trace is not None:
            trace.append((logits, scores, done, tokens, parents, best))
        table, lens, _ = sv.kv_fork(cache, refs, table, lens, parents.view(-1), release=True, status=status)
        history, was_done, _ = sv.beam_reorder([history, done.view(-1, 1)], parents.view(-1), status=status)
        history[:, step] = tokens.view(-1)
        scores = best
        done = (was_done.view(batch, beams) | (tokens == end)).int()
        if step % compact_every == compact_every - 1:
            sv.kv_compact(cache, refs, table, status=status)
        if step + 1 == steps:
            break
        sv.kv_trim(cache, refs, table, lens, window=window, sinks=sinks, status=status)
        new, _ = sv.kv_reserve(cache, refs, table, lens, 1, new_lens=(1 - done).view(-1), status=status)
        logits = model.logits(tokens.view(C, 1), cache, table, lens, status, new_lens=new).view(batch, beams, vocab)
        lens += new
    return history.view(batch, beams, steps), scores, (cache, refs, table, lens), status


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, default in (("steps", 24), ("batch", 4), ("beams", 4), ("window", 48)):
        p.add_argument("--" + name, type=int, default=default)
    a = p.parse_args()
    texts, scores, (_, refs, _, _), status = run(a.steps, a.batch, a.beams, a.window)
    sv.check(int(status.item()), "the search")
    for b in range(a.batch):
        print(f"sequence {b}: best score {float(scores[b, 0]):.2f}, tokens {texts[b, 0].tolist()[:8]} ...")
    print(f"{int((refs > 0).sum())} of {refs.numel()} pages in use")
