"""GPU tests of beam selection where candidates of different beams lie near each other: scores of any magnitude, rows
that hold the same logits in another order, sums of many small units.

The order has to be that of exact scores: the scores, logits and their differences as fractions, and the logarithm of a
row's sum in fp64 over its sorted logits (off by at most 2^-52 of itself and 2^-53 a term of its sorted sum, below 1e-13
here, where the nearest two scores that are not equal differ by 1e-9 at least). A returned score is within half a step
of fp32 and 4e-6 of the exact one."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_78_gb300 as sv
    sv.load_library()
    return sv


def log_sum(l):
    """log sum e^(l - max l), the same for the same logits in any order."""
    x = np.sort(l[np.isfinite(l)].astype(np.float64))
    return math.log(math.fsum(np.exp(x - x[-1])))


def exact(logits, scores, n, done=None, pad=0):
    """[(score, beam, token)] of the n best of one batch row: logits [K, V], scores [K] in fp64."""
    all_ = []
    for k, (l, s) in enumerate(zip(logits, scores)):
        if done is not None and done[k]:
            all_.append((-Fraction(float(s)), k, pad))
            continue
        best = np.argsort(-l, kind="stable")[:n]   # a beam has at most n of them
        base = Fraction(float(s)) - Fraction(float(l.max())) - Fraction(log_sum(l))
        all_ += [(-(base + Fraction(float(l[v]))), k, int(v)) for v in best if l[v] > -np.inf]
    return sorted(all_)[:n]


def check(sv, logits, scores, n, done=None, pad=0):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tok, par, best, _ = sv.beam_select(logits, scores, n, done=done, pad_token=pad, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    B, K, V = logits.shape
    l, s = logits.double().cpu().numpy(), scores.double().cpu().numpy()
    d = None if done is None else done.cpu().numpy()
    for b in range(B):
        want = exact(l[b], s[b], n, None if d is None else d[b], pad)
        assert par[b].tolist() == [b * K + k for _, k, _ in want], b
        assert tok[b].tolist() == [v for _, _, v in want], b
        for got, (x, _, _) in zip(best[b].double().tolist(), want):
            assert abs(Fraction(got) + x) <= abs(x) / 2 ** 24 + Fraction(4e-6), b


LARGE = [-1e3, -1e5, -1e6, -2.0 ** 24, -1e9, -3e12, -1e20, -3e38, 1e9]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("V", [300, 9000])
def test_large_scores(sv, V, dtype):
    """Beams with one large score and much the same rows, whose sums differ by 1e-8 to 1e-4: every token of the one with
    the smaller sum comes before the others' same token."""
    rng = np.random.default_rng(V)
    x = np.repeat(rng.standard_normal((1, 1, V)), 3 * len(LARGE), 0).repeat(3, 1) * 3
    for i in range(3 * len(LARGE)):
        for k, far in ((0, 9.0), (2, 11.0)):   # a token less: the sum's share of it is about e^-(4 (i % 3) + far)
            x[i, k, V // 2] = x[i, 1].max() - far - 4 * (i % 3)
        x[i, 1, V // 2] = -np.inf
    logits = torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()
    scores = torch.tensor(LARGE, dtype=torch.float32).repeat_interleave(3)[:, None].repeat(1, 3).cuda()
    for n in (1, 5, 24):
        check(sv, logits, scores, n)


def test_large_and_small_scores(sv):
    """An ended beam, or one not far from 0, beside beams that are far behind; scores a step of fp32 apart."""
    rng = np.random.default_rng(1)
    logits = torch.from_numpy((rng.standard_normal((6, 4, 12)) * 2).astype(np.float32)).cuda()
    logits[:, 2] = logits[:, 1]
    logits[:, 2, 5] -= 1e-4
    scores = torch.tensor([[0.0, -1e9, -1e9, -1e9], [0.0, -1e6, -1e6, -1e9], [-1e9, -1e9 + 64, -1e9 + 64, -1e9],
                           [-2.0 ** 30, -2.0 ** 20, -2.0 ** 20, 3.0], [-1.0, -1e30, -1e30, -1e25],
                           [-3.4e38, -3.4e38, -3.4e38, 3.4e38]], dtype=torch.float32).cuda()
    done = torch.tensor([[1, 0, 0, 0]] * 6, dtype=torch.int32).cuda()
    for n in (3, 20, 37):
        check(sv, logits, scores, n)
        check(sv, logits, scores, n, done=done, pad=3)


def test_equal_scores_of_unlike_beams(sv):
    """Scores and logits that make up for each other exactly, in beams with the same rows: by beam, then by token."""
    rng = np.random.default_rng(2)
    row = torch.from_numpy(rng.integers(-64, 64, (8, 1, 700)).astype(np.float32) / 16).cuda()
    logits = row.repeat(1, 4, 1).contiguous()
    scores = torch.tensor([[-2.0, -2.5, -1.75, -3.0]]).repeat(8, 1).cuda()
    scores[4:] -= 1e6
    for n in (4, 17, 60):
        check(sv, logits, scores, n)

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("V", [50, 2100, 33000])
def test_rows_in_another_order(sv, V, dtype):
    """Beams with equal scores whose rows hold the same logits in another order: their scores are equal."""
    rng = np.random.default_rng(V + 1)
    x = rng.standard_normal((12, 1, V)).repeat(4, 1) * np.linspace(0.5, 6, 12)[:, None, None]
    for b in range(12):
        for k in range(4):
            x[b, k] = x[b, k, rng.permutation(V)]
    logits = torch.from_numpy(x.astype(np.float32)).to(dtype).cuda()
    scores = torch.from_numpy(rng.random((12, 1)).astype(np.float32)).cuda().repeat(1, 4).contiguous()
    for n in (1, 4, 15):
        check(sv, logits, scores, n)

def test_many_units_with_little_each(sv):
    """1023 units, each just below 2^-40 of the sum's power of two: 1.86e-9 of the sum together. The scores bring its
    beam 0.81e-9 nearer, so that it is 1.05e-9 behind."""
    V = 1 << 20
    x = np.full((2, 2, V), -np.inf)
    x[:, :, 0] = 1e-3
    x[0, 0, 1024::1024] = x[1, 1, 1024::1024] = -39 * math.log(2) - 1e-3
    logits = torch.from_numpy(x.astype(np.float32)).cuda()
    scores = torch.tensor([[0.81e-9, 0.0], [0.0, 0.81e-9]]).cuda()
    for n in (1, 2):
        check(sv, logits, scores, n)
