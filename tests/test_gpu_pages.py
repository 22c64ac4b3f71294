"""GPU tests of the calls that deal with a cache's pages against their plain forms (pages_ref): every table,
count, length and byte has to be equal."""

import numpy as np
import pytest
import torch

import pages_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_78_gb300 as sv
    sv.load_library()
    return sv


class World:
    """A cache, counts and sequences, on the GPU and as numpy arrays that the plain forms change."""

    def __init__(self, sv, seed, P, page=16, Hkv=2, D=64, layers=1):
        self.sv, self.page, self.rng = sv, page, np.random.default_rng(seed)
        shape = (layers, P, Hkv, page, D)
        self.pools = [self.rng.integers(0, 126, shape, dtype=np.uint8) for _ in range(2)]
        self.scales = [self.rng.random(shape[:3], dtype=np.float32) for _ in range(2)]
        d = [torch.from_numpy(x.copy()).cuda() for x in (*self.pools, *self.scales)]
        self.cache = sv.KVCache(*d)
        self.refs = np.zeros(P, np.int32)
        self.codes = []
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def sequences(self, lens, S, share=0):
        """Tables with pages for `lens` tokens, the first `share` places of all sequences the same pages."""
        lens = np.array(lens, np.int32)
        table = np.full((len(lens), S), -1, np.int32)
        order = list(self.rng.permutation(np.flatnonzero(self.refs == 0)))
        common = [order.pop() for _ in range(share)]
        for b, n in enumerate(lens):
            for j in range(-(-int(n) // self.page)):
                table[b, j] = common[j] if j < min(share, n // self.page) else order.pop()
                self.refs[table[b, j]] += 1
        return table, lens

    def up(self, *arrays):
        return [None if x is None else torch.from_numpy(np.array(x)).cuda() for x in arrays]

    def check(self, refs, *pairs):
        torch.cuda.synchronize()
        for got, want in ((refs, self.refs), *pairs):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
        for got, want in zip((self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale),
                             (*self.pools, *self.scales)):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
        code = int(self.status.item())
        assert (code in self.codes) if self.codes else code == 0, (code, set(self.codes))


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("lens,N,S,P", [
    ([0], 1, 1, 1), ([16], 1, 2, 40), ([15, 16, 17, 31, 0], 1, 4, 60), ([3, 100, 48], 70, 40, 5000),
    ([128] * 9, 129, 30, 9000), (list(range(0, 1300, 13)), 33, 90, 9999)])
def test_reserve(sv, page, lens, N, S, P):
    w = World(sv, N, P, page, Hkv=1)
    table, lens = w.sequences([min(n, S * page - N) if page == 16 else n for n in lens], S)
    news = w.rng.integers(0, N + 1, len(lens)).astype(np.int32)
    for new in (None, news):   # the second call finds the pages of the first
        d_refs, d_table, d_lens, d_new = w.up(w.refs, table, lens, new)
        granted, _ = sv.kv_reserve(w.cache, d_refs, d_table, d_lens, N, new_lens=d_new, status=w.status)
        want = ref.reserve(w.refs, table, lens, new, N, page, w.codes)
        w.check(d_refs, (d_table, table), (granted, want), (d_lens, lens))


def test_reserve_fills_gaps(sv):
    """Places without a page between places that have one; table entries that are any negative number."""
    w = World(sv, 5, 30)
    table, lens = w.sequences([20, 40], 8)
    table[0, 4] = w.refs.argmin()
    w.refs[table[0, 4]] = 1
    table[1, 5:] = -77
    d_refs, d_table, d_lens = w.up(w.refs, table, lens)
    granted, _ = sv.kv_reserve(w.cache, d_refs, d_table, d_lens, 88, status=w.status)
    want = ref.reserve(w.refs, table, lens, None, 88, 16, w.codes)
    w.check(d_refs, (d_table, table), (granted, want))


@pytest.mark.parametrize("free", [0, 1, 3, 7])
def test_reserve_when_pages_run_out(sv, free):
    """Served are the sequences up to the first that does not fit, and those after it that need nothing."""
    w = World(sv, free, 40)
    table, lens = w.sequences([16, 20, 30, 0, 16, 90, 47, 10], 8)
    spare = np.flatnonzero(w.refs == 0)
    w.refs[spare[free:]] = 3   # held by others
    new = np.array([17, 4, 20, 16, 0, 1, 40, 1], np.int32)
    d_refs, d_table, d_lens, d_new = w.up(w.refs, table, lens, new)
    granted, _ = sv.kv_reserve(w.cache, d_refs, d_table, d_lens, 40, new_lens=d_new, status=w.status)
    want = ref.reserve(w.refs, table, lens, new, 40, 16, w.codes)
    assert ref.NO_PAGE in w.codes or free == 7
    w.check(d_refs, (d_table, table), (granted, want))


def test_reserve_bad_lengths(sv):
    w = World(sv, 6, 30)
    table, lens = w.sequences([5, 5, 5, 5, 5], 3)
    lens[1], lens[2] = -1, 2 ** 31 - 1
    new = np.array([1, 1, 1, 44, -3], np.int32)
    d_refs, d_table, d_lens, d_new = w.up(w.refs, table, lens, new)
    granted, _ = sv.kv_reserve(w.cache, d_refs, d_table, d_lens, 50, new_lens=d_new, status=w.status)
    want = ref.reserve(w.refs, table, lens, new, 50, 16, w.codes)
    assert set(w.codes) == {ref.LENGTH} and list(want) == [1, 0, 0, 0, 0]
    w.check(d_refs, (d_table, table), (granted, want))


@pytest.mark.parametrize("window,sinks", [(None, 0), (1, 0), (1, 1), (16, 0), (17, 16), (33, 17), (100, 4),
                                          (1000, 0), (50, 1000)])
def test_trim(sv, window, sinks):
    w = World(sv, 7, 900)
    table, lens = w.sequences([0, 1, 15, 16, 17, 31, 32, 33, 64, 100, 333, 480], 32)
    d_refs, d_table, d_lens = w.up(w.refs, table, lens)
    sv.kv_reserve(w.cache, d_refs, d_table, d_lens, 32, status=w.status)   # a tail that is not used
    ref.reserve(w.refs, table, lens, None, 32, 16, w.codes)
    for _ in range(2):   # the second call finds nothing more
        sv.kv_trim(w.cache, d_refs, d_table, d_lens, window=window, sinks=sinks, status=w.status)
        ref.trim(w.refs, table, lens, window or 1 << 30, sinks, 16, w.codes)
        w.check(d_refs, (d_table, table), (d_lens, lens))


def test_trim_keeps_what_the_next_token_sees(sv):
    """By the definition, slot by slot."""
    w = World(sv, 8, 400)
    table, lens = w.sequences(list(range(60, 110)), 7)
    d_refs, d_table, d_lens = w.up(w.refs, table, lens)
    sv.kv_trim(w.cache, d_refs, d_table, d_lens, window=21, sinks=5, status=w.status)
    got = d_table.cpu().numpy()
    for b, n in enumerate(lens):
        need = {t // 16 for t in range(n) if t < 5 or t > n - 21}
        assert {j for j in range(7) if got[b, j] >= 0} == need


@pytest.mark.parametrize("ended", [None, [0, 1, 0, 5, 1], [0, 0, 0, 0, 0]])
def test_free(sv, ended):
    w = World(sv, 9, 60)
    table, lens = w.sequences([40, 33, 100, 16, 1], 8, share=2)
    d_refs, d_table, d_lens, d_ended = w.up(w.refs, table, lens, None if ended is None else np.array(ended, np.int32))
    sv.kv_free(w.cache, d_refs, d_table, d_lens, ended=d_ended, status=w.status)
    ref.free(w.refs, table, lens, ended, w.codes)
    w.check(d_refs, (d_table, table), (d_lens, lens))


def test_free_reports_what_cannot_be(sv):
    """The same page more often than it is held; entries past the pool."""
    w = World(sv, 10, 20)
    table, lens = w.sequences([40, 33], 5)
    table[1, 0] = table[0, 0]
    lens[1] = -5   # lengths are not read
    d_refs, d_table, d_lens = w.up(w.refs, table, lens)
    sv.kv_free(w.cache, d_refs, d_table, d_lens, status=w.status)
    ref.free(w.refs, table, lens, None, w.codes)
    assert w.codes == [ref.REFS]
    w.check(d_refs, (d_table, table), (d_lens, lens))
    w.status.zero_()
    w.codes = []
    table[0, 3] = 20
    d_refs, d_table, d_lens = w.up(w.refs, table, lens)
    sv.kv_free(w.cache, d_refs, d_table, d_lens, status=w.status)
    ref.free(w.refs, table, lens, None, w.codes)
    assert w.codes == [ref.PAGE]
    w.check(d_refs, (d_table, table), (d_lens, lens))


FORKS = {
    "one": ([37], [0]),
    "beams": ([37, 32, 5, 48], [0, 0, 2, 2]),
    "all_of_one": ([37, 33, 17, 31], [1, 1, 1, 1]),
    "swapped": ([20, 21, 22], [2, 1, 0]),
    "more": ([64, 3], [0, 1, 1, 0, 0, 1, 0]),
    "fewer": ([64, 3, 18], [2]),
    "empty_parents": ([0, 16, 0], [0, 0, 1, 2]),
    "none": ([20, 30], [-1, 0, -1]),
    "bad": ([20, 30, 40], [0, 3, -2, 1, 7]),
    "nobody": ([20, 30], []),
}


@pytest.mark.parametrize("release", [False, True])
@pytest.mark.parametrize("case", list(FORKS))
def test_fork(sv, case, release):
    lens, parents = FORKS[case]
    w = World(sv, 11, 50, layers=2)
    table, lens = w.sequences(lens, 6, share=1)
    for b, n in enumerate(lens):   # pages reserved past the last token do not go to the children
        if -(-int(n) // 16) < 6:
            table[b, 5] = np.flatnonzero(w.refs == 0)[-1]
            w.refs[table[b, 5]] = 1
    parents = np.array(parents, np.int32)
    d_refs, d_table, d_lens, d_par = w.up(w.refs, table, lens, parents)
    before = table.copy(), lens.copy()
    got_t, got_n, _ = sv.kv_fork(w.cache, d_refs, d_table, d_lens, d_par, release=release, status=w.status)
    want = ref.fork(w.refs, table, lens, parents, release, 16, w.pools, w.scales, w.codes)
    w.check(d_refs, (got_t, want[0]), (got_n, want[1]), (d_table, before[0]), (d_lens, before[1]))


@pytest.mark.parametrize("page,Hkv,D,layers", [(16, 1, 64, 1), (32, 3, 128, 5), (64, 8, 128, 2), (128, 1, 128, 3)])
def test_fork_copies_rows(sv, page, Hkv, D, layers):
    """Partial pages of every length; only their tokens' rows are written."""
    w = World(sv, 12, 3 * page + 8, page, Hkv, D, layers)
    lens = list(range(1, page + 1, max(1, page // 16)))
    table, lens = w.sequences(lens, 3)
    parents = np.repeat(np.arange(len(lens), dtype=np.int32), 2)
    d_refs, d_table, d_lens, d_par = w.up(w.refs, table, lens, parents)
    got_t, got_n, _ = sv.kv_fork(w.cache, d_refs, d_table, d_lens, d_par, status=w.status)
    want = ref.fork(w.refs, table, lens, parents, False, page, w.pools, w.scales, w.codes)
    w.check(d_refs, (got_t, want[0]), (got_n, want[1]))


@pytest.mark.parametrize("release", [False, True])
@pytest.mark.parametrize("free", [0, 2])
def test_fork_when_pages_run_out(sv, free, release):
    w = World(sv, 13, 60, layers=2)
    table, lens = w.sequences([37, 32, 5, 48, 19], 6, share=1)
    spare = np.flatnonzero(w.refs == 0)
    w.refs[spare[free:]] = 2
    parents = np.array([0, 2, 0, 0, 2, 1, 0, 3, 2], np.int32)
    d_refs, d_table, d_lens, d_par = w.up(w.refs, table, lens, parents)
    got_t, got_n, _ = sv.kv_fork(w.cache, d_refs, d_table, d_lens, d_par, release=release, status=w.status)
    want = ref.fork(w.refs, table, lens, parents, release, 16, w.pools, w.scales, w.codes)
    assert w.codes and set(w.codes) == {ref.NO_PAGE} and (want[1] == -1).any()
    w.check(d_refs, (got_t, want[0]), (got_n, want[1]))


@pytest.mark.parametrize("release", [False, True])
def test_fork_bad_tables(sv, release):
    """Bad lengths and entries past the pool; places without a page among the full ones (behind a window)."""
    w = World(sv, 14, 50)
    table, lens = w.sequences([37, 40, 50, 60], 6)
    w.refs[table[0, 1]] -= 1
    table[0, 1] = -1
    w.refs[table[1, 0]] -= 1
    table[1, 0] = 50
    w.refs[table[2, 3]] -= 1
    table[2, 3] = 99
    lens[3] = 97
    parents = np.array([0, 1, 1, 2, 2, 3], np.int32)
    d_refs, d_table, d_lens, d_par = w.up(w.refs, table, lens, parents)
    got_t, got_n, _ = sv.kv_fork(w.cache, d_refs, d_table, d_lens, d_par, release=release, status=w.status)
    want = ref.fork(w.refs, table, lens, parents, release, 16, w.pools, w.scales, w.codes)
    w.check(d_refs, (got_t, want[0]), (got_n, want[1]))


def test_fork_leaves_others_alone(sv):
    """A parent with a bad length that no child continues from is nobody's error, unless it ends."""
    w = World(sv, 20, 50)
    table, lens = w.sequences([37, 40], 6)
    lens[1] = -1
    parents = np.array([0, 0], np.int32)
    d_refs, d_table, d_lens, d_par = w.up(w.refs, table, lens, parents)
    got_t, got_n, _ = sv.kv_fork(w.cache, d_refs, d_table, d_lens, d_par, status=w.status)
    want = ref.fork(w.refs, table, lens, parents, False, 16, w.pools, w.scales, w.codes)
    assert not w.codes
    w.check(d_refs, (got_t, want[0]), (got_n, want[1]))
    sv.kv_fork(w.cache, d_refs, d_table, d_lens, d_par, release=True, status=w.status)
    ref.fork(w.refs, table, lens, parents, True, 16, w.pools, w.scales, w.codes)
    assert set(w.codes) == {ref.LENGTH}
    w.check(d_refs)


@pytest.mark.parametrize("P,B,page,Hkv,D,layers", [(1, 1, 16, 1, 64, 1), (40, 3, 16, 2, 64, 2), (3000, 60, 16, 1, 64, 1),
                                                   (70, 4, 128, 8, 128, 3), (33, 2, 64, 3, 128, 1)])
@pytest.mark.parametrize("share", [0.0, 0.3, 1.0])
def test_compact(sv, P, B, page, Hkv, D, layers, share):
    w = World(sv, 15, P, page, Hkv, D, layers)
    w.refs[w.rng.random(P) < share] = 2   # pages that other tables hold
    places = int((w.refs == 0).sum()) * 2 // 3 // B
    table, lens = w.sequences([places * page] * B, max(1, places))
    for b in range(B):   # any of them may go
        ref.drop(w.refs, table[b], [j for j in range(places) if w.rng.random() < 0.4], w.codes)
    d_refs, d_table = w.up(w.refs, table)
    page_map, live, _ = sv.kv_compact(w.cache, d_refs, d_table, status=w.status)
    want_map, want_live = ref.compact(w.refs, table, [*w.pools, *w.scales], w.codes)
    w.check(d_refs, (d_table, table), (page_map, want_map), (live, np.array([want_live], np.int32)))


def test_compact_bad_entry_and_empty_table(sv):
    w = World(sv, 16, 20)
    table, lens = w.sequences([40, 33], 5)
    w.refs[0:3] = 0
    table[table < 3] = -1
    table[1, 4] = 20
    d_refs, d_table = w.up(w.refs, table)
    page_map, live, _ = sv.kv_compact(w.cache, d_refs, d_table, status=w.status)
    want_map, want_live = ref.compact(w.refs, table, [*w.pools, *w.scales], w.codes)
    w.check(d_refs, (d_table, table), (page_map, want_map), (live, np.array([want_live], np.int32)))
    empty = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    page_map, live, _ = sv.kv_compact(w.cache, d_refs, empty)
    want_map, want_live = ref.compact(w.refs, table, [*w.pools, *w.scales], w.codes)
    w.check(d_refs, (page_map, want_map))


def test_a_life_of_calls(sv):
    """Sequences start, grow, fork, fall behind a window, end, and the pool is compacted, many times over: after
    every call counts, tables, lengths and contents are the plain forms', and no page is lost."""
    w = World(sv, 17, 120, layers=2)
    B, S, page = 6, 9, 16
    table, lens = np.full((B, S), -1, np.int32), np.zeros(B, np.int32)
    d_refs, d_table, d_lens = w.up(w.refs, table, lens)
    ws = sv.new_pages_workspace(w.cache, B)
    for step in range(40):
        new = w.rng.integers(0, 24, B).astype(np.int32)
        new = np.minimum(new, S * page - lens)
        d_new, = w.up(new)
        granted, _ = sv.kv_reserve(w.cache, d_refs, d_table, d_lens, 24, new_lens=d_new, workspace=ws, status=w.status)
        want = ref.reserve(w.refs, table, lens, new, 24, page, w.codes)
        d_lens += granted
        lens += want
        w.check(d_refs, (d_table, table), (d_lens, lens))
        parents = w.rng.integers(0, B, B).astype(np.int32)
        d_par, = w.up(parents)
        d_table, d_lens, _ = sv.kv_fork(w.cache, d_refs, d_table, d_lens, d_par, release=True, workspace=ws, status=w.status)
        table, lens = ref.fork(w.refs, table, lens, parents, True, page, w.pools, w.scales, w.codes)
        w.check(d_refs, (d_table, table), (d_lens, lens))
        sv.kv_trim(w.cache, d_refs, d_table, d_lens, window=70, sinks=3, status=w.status)
        ref.trim(w.refs, table, lens, 70, 3, page, w.codes)
        ended = ((lens > 110) | (w.rng.random(B) < 0.05)).astype(np.int32)
        d_ended, = w.up(ended)
        sv.kv_free(w.cache, d_refs, d_table, d_lens, ended=d_ended, status=w.status)
        ref.free(w.refs, table, lens, ended, w.codes)
        w.check(d_refs, (d_table, table), (d_lens, lens))
        if step % 3 == 0:
            _, live, _ = sv.kv_compact(w.cache, d_refs, d_table, workspace=ws, status=w.status)
            ref.compact(w.refs, table, [*w.pools, *w.scales], w.codes)
            w.check(d_refs, (d_table, table))
            assert int(live.item()) == len(set(table[table >= 0].tolist()))
        assert not w.codes
        held = np.zeros_like(w.refs)
        np.add.at(held, table[table >= 0], 1)
        np.testing.assert_array_equal(held, w.refs)


def test_pages_in_a_graph_and_on_a_stream(sv):
    """A step's calls captured once and replayed: each replay works on what the one before left."""
    w = World(sv, 18, 80)
    table, lens = w.sequences([30, 47, 16], 12)
    parents, new = np.array([0, 0, 2], np.int32), np.array([9, 9, 9], np.int32)
    d_refs, d_table, d_lens, d_par, d_new = w.up(w.refs, table, lens, parents, new)
    other_t, other_n = torch.empty_like(d_table), torch.empty_like(d_lens)
    granted = torch.empty_like(d_lens)
    ws = sv.new_pages_workspace(w.cache, 3)

    def step(stream=None):
        kw = dict(status=w.status, stream=stream)
        sv.kv_reserve(w.cache, d_refs, d_table, d_lens, 9, new_lens=d_new, granted=granted, workspace=ws, **kw)
        d_lens.add_(granted)
        sv.kv_fork(w.cache, d_refs, d_table, d_lens, d_par, release=True, page_table_out=other_t,
                   lens_out=other_n, workspace=ws, **kw)
        d_table.copy_(other_t)
        d_lens.copy_(other_n)
        sv.kv_trim(w.cache, d_refs, d_table, d_lens, window=40, **kw)

    def plain():
        nonlocal table, lens
        lens += ref.reserve(w.refs, table, lens, new, 9, 16, w.codes)
        table, lens = ref.fork(w.refs, table, lens, parents, True, 16, w.pools, w.scales, w.codes)
        ref.trim(w.refs, table, lens, 40, 0, 16, w.codes)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    plain()
    torch.cuda.current_stream().wait_stream(side)
    w.check(d_refs, (d_table, table), (d_lens, lens))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(5):
        graph.replay()
        plain()
        w.check(d_refs, (d_table, table), (d_lens, lens))


def test_large_tables(sv):
    """As many sequences as a call takes, a pool whose free pages lie far apart and at its end."""
    B, S = sv.SPEC_MAX_SEQS, 4
    w = World(sv, 19, 70001, Hkv=1)
    w.refs[:] = 1
    w.refs[w.rng.integers(0, 70001, 500)] = 0
    w.refs[-40000:] = 0
    table, lens = w.sequences(w.rng.integers(0, 33, B), S)
    new = w.rng.integers(0, 32, B).astype(np.int32)
    d_refs, d_table, d_lens, d_new = w.up(w.refs, table, lens, new)
    granted, _ = sv.kv_reserve(w.cache, d_refs, d_table, d_lens, 31, new_lens=d_new, status=w.status)
    want = ref.reserve(w.refs, table, lens, new, 31, 16, w.codes)
    w.check(d_refs, (d_table, table), (granted, want))
    parents = w.rng.integers(0, B, B).astype(np.int32)
    d_par, = w.up(parents)
    got_t, got_n, _ = sv.kv_fork(w.cache, d_refs, d_table, d_lens, d_par, release=True, status=w.status)
    table, lens = ref.fork(w.refs, table, lens, parents, True, 16, w.pools, w.scales, w.codes)
    w.check(d_refs, (got_t, table), (got_n, lens))
    _, live, _ = sv.kv_compact(w.cache, d_refs, got_t, status=w.status)
    _, want_live = ref.compact(w.refs, table, [*w.pools, *w.scales], w.codes)
    w.check(d_refs, (got_t, table), (live, np.array([want_live], np.int32)))
