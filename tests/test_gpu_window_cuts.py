"""GPU tests of windowed attention on both sides of the rule that cuts its work: whole items, or even shares whose parts
are joined; one sequence, few, and as many items as there are CTAs or a few more."""

import numpy as np
import pytest
import torch

from test_gpu_kv import Case, rand16, tree_words
from test_gpu_window import check, forget, sv   # noqa: F401

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("B", [1, 2, 5])
@pytest.mark.parametrize("window", [500, 1100, 2040])
@pytest.mark.parametrize("N,G,D,dtype", [(64, 4, 64, BF16), (24, 4, 128, F16)])   # 256 and 128 rows
def test_few_trees(sv, N, G, D, dtype, window, B):   # noqa: F811
    Hkv = 5
    c = Case(window + B, [2300 - 37 * b for b in range(B)], N, Hkv, D, 64)
    words = tree_words(c.rng, B, N, sv)
    forget(c, window, 64)
    check(sv, c, rand16(c.rng, (B, N, Hkv * G, D), dtype), window, 64, words=words)


@pytest.mark.parametrize("B", [1, 2, 4])
@pytest.mark.parametrize("window", [700, 1500])
@pytest.mark.parametrize("N,dtype", [(1, BF16), (6, F16)])   # 16 and 32 columns
def test_few_chains(sv, N, dtype, window, B):   # noqa: F811
    Hkv = 8
    c = Case(window + B, [3000 - 101 * b for b in range(B)], N, Hkv, 128, 32)
    forget(c, window, 4)
    check(sv, c, rand16(c.rng, (B, N, Hkv * 4, 128), dtype), window, 4)


@pytest.mark.parametrize("B", [17, 19, 20, 39])
def test_about_as_many_items_as_ctas(sv, B):   # noqa: F811
    c = Case(B, [400 + 29 * (b % 7) for b in range(B)], 2, 8, 64, 16)
    forget(c, 300, 5)
    check(sv, c, rand16(c.rng, (B, 2, 16, 64), BF16), 300, 5)


def test_a_short_piece_of_a_prompt(sv):   # noqa: F811
    c = Case(9, [1200], 100, 2, 64, 16)
    forget(c, 1000, 16)
    check(sv, c, rand16(c.rng, (1, 100, 16, 64), F16), 1000, 16)


def test_the_cut_does_not_depend_on_padding(sv):   # noqa: F811
    """Sequences without tokens among those with some, one of them long."""
    c = Case(11, [2300, 0, 5, 0], 64, 2, 64, 64)
    new = [64, 0, 3, 0]
    forget(c, 2040, 64)
    out, lse = check(sv, c, rand16(c.rng, (4, 64, 8, 64), BF16), 2040, 64, new_lens=new)
    for b, n in enumerate(new):
        assert out[b, n:].eq(0).all() and lse[b, n:].eq(-np.inf).all()
