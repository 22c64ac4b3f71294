"""GPU tests of beam selection and reordering against plain fp64 forms.

Tokens and parents have to be equal (the order is that of exact scores; inputs here have no two scores of
different beams nearer than 1e-9 but equal ones). A returned score is within half a step of fp32 (2^-24 of it)
and the bound of the fp32 sum's relative error (4e-6) of the exact one."""

import numpy as np
import pytest
import torch

from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_78_gb300 as sv
    sv.load_library()
    return sv


def select(logits, scores, n, done=None, pad=0):
    """(tokens, parents, scores) by the definition: logits [B, K, V] and scores [B, K] in fp64."""
    B, K, V = logits.shape
    tok, par = np.full((B, n), -1, np.int32), np.full((B, n), -1, np.int32)
    best = np.full((B, n), -np.inf)
    for b in range(B):
        s = np.full((K, V), -np.inf)
        bad = False
        for k in range(K):
            x = scores[b, k]
            if x == -np.inf:
                continue
            if not x < np.inf:
                bad = True
            elif done is not None and done[b, k]:
                s[k, pad] = x
            else:
                l = logits[b, k]
                m = l.max()
                if not np.isfinite(m):
                    bad = True
                    continue
                s[k] = x + ((l - m) - np.log(np.exp(l - m).sum()))
        if bad:
            best[b] = np.nan
            continue
        # (equal in fp64: by beam; within a beam by logit, which decides in exact arithmetic, then by token)
        l = np.where(np.isfinite(s), logits[b], 0.0).ravel() if done is None else np.where(done[b][:, None] != 0, 0.0, logits[b]).ravel()
        order = np.lexsort((np.arange(K * V), -np.nan_to_num(l), np.repeat(np.arange(K), V), -s.ravel()))[:n]
        order = order[s.ravel()[order] > -np.inf]
        tok[b, :len(order)], par[b, :len(order)] = order % V, b * K + order // V
        best[b, :len(order)] = s.ravel()[order]
    return tok, par, best


def as64(t):
    return t.double().cpu().numpy()


def check(sv, logits, scores, n, done=None, pad=0, **kw):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tok, par, best, _ = sv.beam_select(logits, scores, n, done=done, pad_token=pad, status=st, **kw)
    torch.cuda.synchronize()
    wt, wp, wb = select(as64(logits), as64(scores), n, None if done is None else done.cpu().numpy(), pad)
    np.testing.assert_array_equal(par.cpu().numpy(), wp)
    np.testing.assert_array_equal(tok.cpu().numpy(), wt)
    got = as64(best)
    fin = np.isfinite(wb)
    np.testing.assert_array_equal(got[~fin], wb[~fin])
    assert (np.abs(got[fin] - wb[fin]) <= 2.0 ** -24 * np.abs(wb[fin]) + 4e-6).all()
    assert int(st.item()) == (sv.SPEC_ERR_NONFINITE if np.isnan(wb).any() else 0)
    return tok, par, best


def some(rng, B, K, V, dtype, sd=3.0, off=0):
    x = rng.standard_normal((B, 1, V)) * sd + rng.standard_normal((B, K, V)) * 0.5
    t = torch.from_numpy(x.astype(np.float32)).to(dtype)
    big = torch.empty(t.numel() + off, dtype=dtype, device="cuda")
    big[off:] = t.reshape(-1).cuda()
    s = -np.cumsum(rng.random((B, K)), 1)
    return big[off:].view(B, K, V), torch.from_numpy(s.astype(np.float32)).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,K,V,n", [(1, 1, 1, 1), (1, 1, 1, 5), (2, 3, 7, 4), (2, 3, 7, 40), (3, 4, 1000, 4),
                                     (1, 4, 32000, 8), (5, 8, 4099, 16), (2, 16, 2049, 64), (2, 64, 1023, 64),
                                     (4, 5, 50257, 10), (2, 8, 152064, 16), (1, 3, 1 << 20, 6)])
def test_select(sv, dtype, B, K, V, n):
    rng = np.random.default_rng(V + n)
    logits, scores = some(rng, B, K, V, dtype)
    check(sv, logits, scores, n)


@pytest.mark.parametrize("dtype,off", [(torch.float32, 1), (torch.float32, 3), (torch.bfloat16, 1),
                                       (torch.bfloat16, 3), (torch.bfloat16, 6)])
@pytest.mark.parametrize("V", [9, 2047, 5000, 16384])
def test_select_unaligned(sv, dtype, off, V):
    rng = np.random.default_rng(V * 8 + off)
    logits, scores = some(rng, 3, 4, V, dtype, off=off)
    check(sv, logits, scores, 8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_beams_not_in_use_and_at_their_end(sv, dtype):
    """The first step has one beam; ended beams keep their score; their logits may hold anything."""
    rng = np.random.default_rng(3)
    logits, scores = some(rng, 6, 4, 3001, dtype)
    scores[0, 1:] = -np.inf
    logits[0, 1:] = np.nan
    done = torch.zeros(6, 4, dtype=torch.int32, device="cuda")
    done[1] = 1
    done[2, 1] = -7
    done[3, 0] = 1
    scores[3, 0] = -30.0   # ended, and far behind
    scores[4] = -np.inf    # none in use
    done[5, 2] = 1
    scores[5, 2] = -np.inf
    logits[1] = np.inf
    logits[2, 1] = np.nan
    tok, par, best = check(sv, logits, scores, 9, done=done, pad=17)
    assert tok[4].eq(-1).all() and best[4].eq(-np.inf).all()
    assert tok[1, :4].eq(17).all() and par[1].tolist()[4:] == [-1] * 5


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_tokens(sv, dtype):
    rng = np.random.default_rng(4)
    logits, scores = some(rng, 4, 3, 5003, dtype)
    logits[0, :, 100:] = -np.inf
    logits[1, 0, :5002] = -np.inf          # one token left in a beam, in its last unit
    logits[2, :, torch.from_numpy(rng.permutation(5003)[:5000]).cuda()] = -np.inf
    logits[3] = torch.finfo(dtype).min     # masked by the lowest value: equal everywhere
    check(sv, logits, scores, 12)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", ["nan", "inf", "masked", "score_nan", "score_inf"])
def test_bad_rows(sv, dtype, bad):
    rng = np.random.default_rng(5)
    logits, scores = some(rng, 3, 4, 4100, dtype)
    if bad == "nan":
        logits[1, 2, 4099] = np.nan
    elif bad == "inf":
        logits[1, 0, 0] = np.inf
    elif bad == "masked":
        logits[1, 3] = -np.inf
    else:
        scores[1, 1] = np.nan if bad == "score_nan" else np.inf
    tok, par, best = check(sv, logits, scores, 6)
    assert tok[1].eq(-1).all() and best[1].isnan().all() and tok[0].ge(0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1000, 5001, 40000])
def test_equal_scores(sv, dtype, V):
    """Equal logits everywhere; a few values only; beams that are copies of each other, at rows of different
    alignment: equal scores go by beam, then by token."""
    rng = np.random.default_rng(6)
    logits, scores = some(rng, 4, 5, V, dtype)
    logits[0] = 1.25
    scores[0] = -1.0
    logits[1] = torch.from_numpy(rng.integers(0, 3, (5, V)).astype(np.float32)).to(dtype).cuda()
    scores[1] = -2.0
    logits[1, 1:] = logits[1, :1]
    logits[2, 1:] = logits[2, :1]
    scores[2] = -0.5
    logits[3, 2] = logits[3, 0]
    scores[3, 2] = scores[3, 0]
    check(sv, logits, scores, 40)


def near_ties(rng, V, gap):
    """Two beams whose best tokens' scores differ by `gap`: row 1 is row 0 permuted but for one token, whose
    logit makes up for the scores."""
    a = (rng.standard_normal(V) * 3).astype(np.float32)
    b = a[rng.permutation(V)].copy()
    b[rng.integers(0, V)] += np.float32(0.37)
    la, lb = (np.log(np.exp(x.astype(np.float64)).sum()) for x in (a, b))
    best_a, best_b = a.max() - la, b.max() - lb
    sa = np.float32(-1.0)
    sb = np.float32(sa + best_a - best_b + gap)   # exact scores then differ by about gap
    return np.stack([a, b]), np.array([sa, sb])


@pytest.mark.parametrize("V", [700, 33000])
def test_scores_nearer_than_fp32_tells(sv, V):
    """Beams whose best candidates are closer than the fp32 sums' errors: the order is the exact one."""
    rng = np.random.default_rng(7)
    rows = [near_ties(rng, V, g) for g in rng.uniform(-3e-7, 3e-7, 48)]
    logits = torch.from_numpy(np.stack([r[0] for r in rows])).cuda()
    scores = torch.from_numpy(np.stack([r[1] for r in rows])).cuda()
    for n in (1, 2, 5):
        check(sv, logits, scores, n)


@pytest.mark.parametrize("V", [500, 29270])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_rows_that_one_token_fills(sv, V, dtype):
    """Beams with equal scores and largest logits, whose sums differ by less than fp32 holds beside that token: by 3e-9
    and more, which is told apart, or not at all."""
    x = np.full((3, 4, V), -60.0)              # all of these together: below 1e-21 of the sum
    x[:, :, V // 3] = 0.0
    x[0, :, V - 2] = -18.0, -18.5, -19.0, -20.0      # exp: 15.2e-9, 9.2e-9, 5.6e-9, 2.1e-9; 1 in fp32 with the 1
    x[1, :, V - 2] = -18.5, -20.0, -18.5, -20.0
    x[2, :, V - 2] = -18.0
    logits = torch.from_numpy(x).to(dtype).cuda()
    scores = torch.full((3, 4), -1.5, device="cuda")
    for n in (1, 3, 4, 8, 10):
        check(sv, logits, scores, n)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_equal_beams_with_a_little_elsewhere(sv, dtype):
    """Equal beams, part of whose sums (1e-13 to 1e-11 of them) is too little for the finest sums asked for, but not 0."""
    V = 9000
    x = np.full((40, 3, V), -60.0)
    x[:, :, 10] = 0.0
    x[:, :, 11] = np.linspace(-1.5, 0.0, 8).repeat(5)[:, None]
    x[:, :, V - 3] = np.tile(np.linspace(-29.0, -25.0, 20), 2)[:, None]
    x[20:, 2, V - 3] += 0.25
    logits = torch.from_numpy(x).to(dtype).cuda()
    scores = torch.full((40, 3), -1.5, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tok, par, best, _ = sv.beam_select(logits, scores, 6, status=st)
    wt, wp, wb = select(as64(logits), as64(scores), 6)
    # the third beam differs from the others by less than 1e-9: the first 20 batch rows have one order, the others' scores
    np.testing.assert_array_equal(par.cpu().numpy()[:20], wp[:20])
    np.testing.assert_array_equal(tok.cpu().numpy()[:20], wt[:20])
    assert (np.abs(as64(best) - wb) <= 2.0 ** -24 * np.abs(wb) + 4e-6).all() and int(st.item()) == 0


def test_extreme_logits(sv):
    """Magnitudes at which fp32 has no fractions left, up to its largest."""
    rng = np.random.default_rng(8)
    logits, scores = some(rng, 6, 3, 3000, torch.float32)
    logits[0] *= 1e5
    logits[1] = logits[1] * 100 + 2.0 ** 20
    logits[2] = 3e38 + logits[2] * 1e36
    logits[3] = -3e38 + logits[3] * 1e36
    logits[4] *= 1e-30
    logits[5, 1] += 2.0 ** 20 - 3
    check(sv, logits, scores, 7)


def test_units_of_both_kinds(sv):
    """Rows whose units' maxima lie on both sides of the magnitude from which fractions are lost (2^20)."""
    rng = np.random.default_rng(11)
    logits, scores = some(rng, 8, 2, 5000, torch.float32)
    step = torch.linspace(-1, 1, 5000, device="cuda")
    for b, (mid, spread) in enumerate([(-2.0 ** 20, 1), (-2.0 ** 20, 30), (-2.0 ** 20, 70), (-2.0 ** 20, 200),
                                       (2.0 ** 20, 1), (2.0 ** 20, 30), (2.0 ** 20, 200), (0, 2.0 ** 20)]):
        logits[b] = mid + spread * step + logits[b] * 0.1
    check(sv, logits, scores, 5)


def test_deterministic_and_workspace_contents(sv):
    rng = np.random.default_rng(9)
    logits, scores = some(rng, 4, 8, 20011, torch.bfloat16)
    ws = sv.new_beam_workspace(4, 8, 20011, torch.bfloat16)
    first = check(sv, logits, scores, 16, workspace=ws)
    for fill in (0, 255, 127):
        ws.fill_(fill)
        again = sv.beam_select(logits, scores, 16, workspace=ws)
        for x, y in zip(first, again):
            assert torch.equal(x, y)


def test_select_in_a_graph_and_on_a_stream(sv):
    rng = np.random.default_rng(10)
    logits, scores = some(rng, 3, 4, 9000, torch.float32)
    others = [some(rng, 3, 4, 9000, torch.float32) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want = sv.beam_select(logits, scores, 8)
    got = sv.beam_select(logits, scores, 8, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = sv.beam_select(logits, scores, 8)
    for l, s in others:
        logits.copy_(l)
        scores.copy_(s)
        graph.replay()
        want = sv.beam_select(l, s, 8)
        torch.cuda.synchronize()
        for x, y in zip(out, want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("shapes", [[(5, 1)], [(4, 33), (4, 7, 3)], [(6, 4096), (6, 1000), (6, 3), (6, 2, 8)],
                                    [(128, 20000)]])
@pytest.mark.parametrize("dtype", [torch.int32, torch.bfloat16, torch.uint8, torch.float64])
def test_reorder(sv, shapes, dtype):
    g = torch.Generator(device="cuda").manual_seed(1)
    states = [torch.randint(0, 100, s, generator=g, device="cuda").to(dtype) for s in shapes]
    R = shapes[0][0]
    for C in (1, R, 2 * R + 1):
        parents = torch.randint(-1, R, (C,), generator=g, device="cuda").int()
        *outs, st = sv.beam_reorder(states, parents)
        assert int(st.item()) == 0
        for x, y in zip(states, outs):
            want = x[parents.long().clamp(min=0)] * (parents >= 0).view(-1, *[1] * (x.dim() - 1)).to(dtype)
            assert torch.equal(y, want)


def test_reorder_bad_parent(sv):
    x = torch.arange(12, device="cuda").view(3, 4)
    parents = torch.tensor([2, 3, -2, 0], dtype=torch.int32, device="cuda")
    y, st = sv.beam_reorder([x], parents)
    assert int(st.item()) == sv.SPEC_ERR_PARENT
    assert y.tolist() == [x[2].tolist(), [0] * 4, [0] * 4, x[0].tolist()]


def test_reorder_odd_addresses(sv):
    flat = torch.arange(1000, device="cuda", dtype=torch.int32).to(torch.uint8)
    for off, width in ((1, 7), (2, 10), (4, 12), (8, 24), (16, 32)):
        x = flat[off:off + 5 * width].view(5, width)
        y, _ = sv.beam_reorder([x], torch.tensor([4, 0, 4], dtype=torch.int32, device="cuda"))
        assert torch.equal(y, x[[4, 0, 4]])
