"""The beam search example: the operators together, as they are used."""

import os
import sys

import numpy as np
import pytest
import torch

from test_gpu_beam import as64, select

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import beam_search
    return beam_search


@pytest.mark.parametrize("kw", [dict(), dict(batch=1, beams=3, window=5, sinks=0, steps=40),
                                dict(batch=3, beams=8, window=500, page=32, compact_every=3),
                                dict(batch=2, beams=4, q_heads=16, window=17, sinks=20, head_dim=128)])
def test_beam_search(example, kw):
    """Every selection is the plain form's of the same logits; histories and scores are what the selections say; and
    at the end the counts of the pages are those of the table's entries."""
    trace = []
    history, scores, (cache, refs, table, lens), status = example.run(trace=trace, **kw)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    batch, beams, steps = history.shape
    want = np.zeros((batch * beams, 0), np.int64)
    for logits, before, done, tokens, parents, best in trace:
        t, p, s = select(as64(logits), as64(before), beams, done.cpu().numpy(), 1)
        np.testing.assert_array_equal(tokens.cpu().numpy(), t)
        np.testing.assert_array_equal(parents.cpu().numpy(), p)
        assert (np.abs(as64(best) - s) <= 2.0 ** -24 * np.abs(s) + 4e-6).all()
        if want.shape[1] == 0:
            want = np.zeros((batch, 0), np.int64)
        want = np.concatenate([want[p.ravel()], t.reshape(-1, 1)], 1)
    np.testing.assert_array_equal(history.cpu().numpy().reshape(batch * beams, steps), want)
    held = np.zeros(refs.numel(), np.int64)
    entries = table.cpu().numpy()
    np.add.at(held, entries[entries >= 0], 1)
    np.testing.assert_array_equal(refs.cpu().numpy(), held)
    kw = dict(window=48, sinks=4, page=16) | kw
    if kw["window"] < 100:   # what is behind the window has gone back
        assert held.astype(bool).sum() <= batch * beams * (-(-(kw["window"] + kw["sinks"]) // kw["page"]) + 3)


def test_one_beam_is_greedy_decoding(example):
    """One beam takes the largest logit every time, as plain decoding of the same model with the library's top-1
    does."""
    import speculative_decoding_verification_78_gb300 as sv
    trace = []
    history, _, _, status = example.run(steps=20, batch=3, beams=1, end=0, trace=trace)
    assert int(status.item()) == 0
    for step, (logits, _, done, tokens, _, _) in enumerate(trace):
        top, _ = sv.topk(logits.view(3, -1).contiguous(), 1)
        live = done.view(-1) == 0
        assert torch.equal(tokens.view(-1)[live], top.view(-1)[live])
        assert torch.equal(history[:, 0, step], tokens.view(-1)) or not bool(live.all())
