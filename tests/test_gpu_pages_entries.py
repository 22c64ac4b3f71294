"""GPU tests of reservations over page tables with entries past the pool: they count as none."""

import numpy as np
import pytest
import torch

import pages_ref as ref
from test_gpu_pages import World, sv   # noqa: F401

pytestmark = pytest.mark.gpu


def reserve(w, table, lens, N):
    """The plain form, where an entry past the pool that new tokens need is a place without a page."""
    P = len(w.refs)
    for b, n in enumerate(lens):
        if not (ref.length_ok(n, table, w.page) and ref.length_ok(int(n) + N, table, w.page)):
            continue
        for j in range(n // w.page, (n + N - 1) // w.page + 1):
            if table[b, j] >= P:
                w.codes.append(ref.PAGE)
                table[b, j] = -1
    return ref.reserve(w.refs, table, lens, None, N, w.page, w.codes)


@pytest.mark.parametrize("bad", [30, 31, 2 ** 31 - 1])
def test_entries_past_the_pool(sv, bad):
    w = World(sv, 3, 30)
    table, lens = w.sequences([20, 40, 5, 64], 8)
    table[0, 2] = bad           # among the places of the new tokens
    table[1, 3] = table[1, 4] = bad
    table[2, 0] = bad           # the last page, which is not full
    table[3, 7] = bad           # not needed: left alone
    w.refs[:] = 0
    for p in table[(table >= 0) & (table < 30)]:
        w.refs[p] += 1
    d_refs, d_table, d_lens = w.up(w.refs, table, lens)
    granted, _ = sv.kv_reserve(w.cache, d_refs, d_table, d_lens, 40, status=w.status)
    want = reserve(w, table, lens, 40)
    assert set(w.codes) == {ref.PAGE} and (want == 40).all() and table[3, 7] == bad
    w.check(d_refs, (d_table, table), (granted, want), (d_lens, lens))


def test_entries_past_the_pool_when_pages_run_out(sv):
    """A sequence that is not served keeps its table; the code is one of the two."""
    w = World(sv, 4, 30)
    table, lens = w.sequences([16, 16], 6)
    table[0, 1] = table[1, 1] = 30
    w.refs[w.refs == 0] = 7
    w.refs[np.flatnonzero(w.refs == 7)[:2]] = 0
    d_refs, d_table, d_lens = w.up(w.refs, table, lens)
    granted, _ = sv.kv_reserve(w.cache, d_refs, d_table, d_lens, 32, status=w.status)
    second = table[1].copy()
    want = reserve(w, table, lens, 32)
    table[1] = second
    assert want.tolist() == [32, 0] and set(w.codes) == {ref.PAGE, ref.NO_PAGE}
    w.check(d_refs, (d_table, table), (granted, want))
