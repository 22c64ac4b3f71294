"""GPU parity of the KV-cache operators against their plain fp64 forms (kv_ref), at the sizes and
masks where they can go wrong.

Tolerances, from the roundings the operators make. Append: a stored value is within half an e4m3
step of the rotated value (fp32 rotation: 2^-22 of the two products more), a rotated query within
half a step of its type of it. Attention: half a step of the output type; half a step of fp16
(2^-11) for each weight, so at most 2^-11 of the weighted average of |v|; an error d of a score
moves a normalised weight by at most 2 d: d is D + 8 fp32 roundings of the sum's magnitude plus the
representation of the query by e4m3 terms, at most 2^-17 of its largest element for each
element (bf16; fp16 queries have one term more), and 2^-20 for exponentials and sums in fp32."""

import numpy as np
import pytest
import torch

import kv_ref as ref

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
E4 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_78_gb300 as sv
    sv.load_library()


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_78_gb300 as sv
    return sv


class Case:
    """Random cache, page table and lengths; unused page rows and table entries hold garbage."""

    def __init__(self, seed, lens, N, Hkv, D, page, layers=1, junk=True):
        rng = self.rng = np.random.default_rng(seed)
        self.B, self.N, self.Hkv, self.D, self.page = len(lens), N, Hkv, D, page
        self.lens = np.array(lens, np.int32)
        self.pps = max(lens) // page + (N + page - 1) // page + 1
        pages = self.B * self.pps + 2
        self.table = rng.permutation(pages)[:self.B * self.pps].reshape(self.B, -1).astype(np.int32)
        shape = (layers, pages, Hkv, page, D)
        self.pool = [self.codes(shape), self.codes(shape)]
        self.scale = [np.exp2(rng.integers(-8, -4, shape[:3])).astype(np.float32) for _ in range(2)]
        if junk:   # entries past the last page a sequence needs are not read
            for b in range(self.B):
                self.table[b, (lens[b] + N + page - 1) // page:] = -12345

    def codes(self, shape):
        x = np.clip(self.rng.standard_normal(shape) * 90, -448, 448)
        return torch.from_numpy(x).float().to(E4).view(torch.uint8).numpy()

    def cache(self, sv):
        d = [torch.from_numpy(x.copy()).cuda() for x in (*self.pool, *self.scale)]
        return sv.KVCache(d[0].view(E4), d[1].view(E4), d[2], d[3])

    def dev(self, *names):
        return [torch.from_numpy(np.ascontiguousarray(getattr(self, n))).cuda() for n in names]


def tree_words(rng, B, N, sv):
    par = np.full((B, N), -1, np.int32)
    for i in range(1, N):
        par[:, i] = rng.integers(max(0, i // 4 - 1), i, B)
    words, st = sv.tree_mask(torch.from_numpy(par).cuda())
    assert int(st.item()) == 0
    return words


def rand16(rng, shape, dtype, sd=1.0):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * sd).to(dtype).cuda()


def f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------ attention

def check_attention(sv, c, q, words=None, new_lens=None, scale=None, cache=None, stream=None,
                    workspace=None):
    cache = cache or c.cache(sv)
    table, lens = c.dev("table", "lens")
    nl = None if new_lens is None else torch.tensor(new_lens, dtype=torch.int32).cuda()
    out, lse, st = sv.kv_attention(cache, table, lens, q, scale=scale, mask=words, new_lens=nl,
                                   return_lse=True, stream=stream, workspace=workspace)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    scale = scale if scale is not None else c.D ** -0.5
    pool = [x.view(torch.uint8).cpu().numpy()[0] for x in (cache.k, cache.v)]
    scales = [x.cpu().numpy()[0] for x in (cache.k_scale, cache.v_scale)]
    qd, o, l = f64(q), f64(out), f64(lse)
    for b in range(c.B):
        n = c.N if new_lens is None else new_lens[b]
        total = int(c.lens[b]) + n
        see = np.ones((c.N, total), bool)
        if words is None:
            see[:, c.lens[b]:] = np.arange(n)[None] <= np.arange(c.N)[:, None]
        else:
            see[:, c.lens[b]:] = ref.mask_bits(words[b].cpu().numpy(), c.N)[:, :n]
        see[n:] = False
        k, v = (ref.cached(p, s, c.table[b], total, c.page) for p, s in zip(pool, scales))
        want, wl, avg, big, spread = ref.attention(qd[b], k, v, see, scale)
        d = big * (c.D + 8) * 2.0 ** -24 + spread * 2.0 ** -17 + 2.0 ** -20
        tol = HALF[q.dtype] * np.abs(want) + (2.0 ** -11 + 2 * d[..., None]) * avg + 1e-30
        err = np.abs(o[b] - want)
        assert (err <= tol).all(), (b, float((err / tol).max()), np.argwhere(~(err <= tol))[:4])
        fin = np.isfinite(wl)
        assert (np.isneginf(l[b]) == ~fin).all()
        le = np.abs(l[b][fin] - wl[fin])
        lt = d[fin] + 2.0 ** -22 * np.abs(wl[fin]) + 2.0 ** -20
        assert (le <= lt).all(), (b, float((le / lt).max()))
    return out, lse


LENS = [0, 1, 15, 16, 17, 127, 128, 129, 300, 1000]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,Hq,Hkv,D,page", [
    (1, 4, 4, 128, 16), (1, 8, 2, 64, 32), (1, 12, 1, 128, 64), (2, 8, 1, 128, 128),
    (5, 6, 2, 64, 16), (6, 16, 4, 128, 64), (17, 2, 2, 128, 16), (9, 56, 8, 64, 128),
    (33, 8, 4, 128, 32), (70, 4, 1, 64, 64)])
def test_attention_chain(sv, dtype, N, Hq, Hkv, D, page):
    c = Case(N * 7 + D, LENS, N, Hkv, D, page)
    check_attention(sv, c, rand16(c.rng, (c.B, N, Hq, D), dtype))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,Hq,Hkv,D,page", [(2, 2, 2, 128, 16), (13, 8, 2, 128, 32),
                                             (64, 4, 4, 128, 64), (64, 8, 2, 64, 16),
                                             (65, 4, 1, 128, 128)])
def test_attention_tree(sv, dtype, N, Hq, Hkv, D, page):
    c = Case(N * 3 + D, [0, 1, 63, 64, 129, 500], N, Hkv, D, page)
    check_attention(sv, c, rand16(c.rng, (c.B, N, Hq, D), dtype, 1.5),
                    tree_words(c.rng, c.B, N, sv))


def test_attention_prompt(sv):
    """A long piece of a prompt: many row tiles, the diagonal inside tiles."""
    c = Case(5, [0, 130], 300, 1, 128, 32)
    check_attention(sv, c, rand16(c.rng, (2, 300, 3, 128), torch.bfloat16))


def test_attention_large_nodes(sv):
    c = Case(6, [77], 1024, 1, 64, 64)
    check_attention(sv, c, rand16(c.rng, (1, 1024, 1, 64), torch.bfloat16),
                    tree_words(c.rng, 1, 1024, sv))


def test_attention_long_context_is_split(sv):
    """Few rows and a long cache: the tokens are shared out and the parts joined."""
    c = Case(8, [20000, 3], 1, 2, 128, 64)
    check_attention(sv, c, rand16(c.rng, (2, 1, 8, 128), torch.bfloat16, 2.0))


def test_attention_growing_scores(sv):
    """Scores that rise along the sequence (the running maximum moves in every tile), and a first
    token far above all others."""
    c = Case(9, [2000, 2000, 700], 3, 2, 128, 64)
    for b in range(c.B):
        for p in range(c.lens[b] // 64 + 1):
            c.scale[0][0, c.table[b, p]] = 2.0 ** -9 * (1 + p) if b == 0 else 2.0 ** -6
    c.scale[0][0, c.table[1, 0]] = 2.0 ** -3
    check_attention(sv, c, rand16(c.rng, (3, 3, 8, 128), torch.bfloat16, 2.0))


def test_attention_unlike_value_scales(sv):
    """Pages whose value scales differ by many powers of two, and any positive scale."""
    c = Case(10, [900, 100], 4, 2, 128, 16)
    c.scale[1] = np.exp2(c.rng.uniform(-30, 10, c.scale[1].shape)).astype(np.float32)
    c.scale[0] *= c.rng.uniform(0.5, 1.5, c.scale[0].shape).astype(np.float32)
    check_attention(sv, c, rand16(c.rng, (2, 4, 4, 128), torch.bfloat16))


def test_attention_rows_that_see_nothing(sv):
    c = Case(11, [0, 0, 40], 40, 2, 128, 16)
    words = tree_words(c.rng, 3, 40, sv)
    words[0, 7] = 0
    words[1] = 0
    words[2, 39] = 0
    out, lse = check_attention(sv, c, rand16(c.rng, (3, 40, 4, 128), torch.bfloat16), words)
    assert float(out[1].abs().max()) == 0 and bool(torch.isneginf(lse[1]).all())


@pytest.mark.parametrize("tree", [False, True])
def test_attention_padding(sv, tree):
    c = Case(12, [0, 5, 200, 64], 20, 2, 64, 32)
    words = tree_words(c.rng, 4, 20, sv) if tree else None
    check_attention(sv, c, rand16(c.rng, (4, 20, 8, 64), torch.float16), words, [0, 20, 7, 1])


def test_attention_nan_in_unseen_slots(sv):
    """NaN codes after a sequence's last token, in pages of others, and in nodes a query does not
    see change nothing for it; queries that see one are NaN throughout."""
    N = 8
    c = Case(13, [50, 128], N, 2, 128, 64)
    par = torch.tensor([[-1, 0, 0, 1, 1, 2, 2, 0]] * 2, dtype=torch.int32).cuda()
    words, _ = sv.tree_mask(par)
    for side in range(2):
        for b in range(2):
            n = int(c.lens[b]) + N
            pg = c.table[b, (n - 1) // 64]
            c.pool[side][0, pg, :, (n - 1) % 64 + 1:] = 0x7f
    q = rand16(c.rng, (2, N, 4, 128), torch.bfloat16)
    out, lse = check_attention(sv, c, q, words)
    for side in range(2):   # node 7 becomes NaN: only itself sees it
        slot = int(c.lens[0]) + 7
        c.pool[side][0, c.table[0, slot // 64], :, slot % 64] = 0xff
        table, lens = c.dev("table", "lens")
        o2, l2, st = sv.kv_attention(c.cache(sv), table, lens, q, mask=words, return_lse=True)
        assert int(st.item()) == 0
        assert bool(o2[0, 7].isnan().all())
        assert torch.equal(o2[0, :7], out[0, :7]) and torch.equal(o2[1], out[1])
        assert torch.equal(l2[0, :7], lse[0, :7])


@pytest.mark.parametrize("N,Hq", [(40, 4), (40, 8), (70, 8)])
@pytest.mark.parametrize("side", [0, 1])
def test_attention_nan_node_of_many_rows(sv, N, Hq, side):
    """A node whose key or value is NaN: the queries that see it are NaN, the others as before."""
    c = Case(N + Hq, [50, 300], N, 2, 128, 64)
    words = tree_words(c.rng, 2, N, sv)
    q = rand16(c.rng, (2, N, Hq, 128), torch.bfloat16)
    out, lse = check_attention(sv, c, q, words)
    node = 5
    sees = torch.from_numpy(ref.mask_bits(words.cpu().numpy(), N)[1, :, node]).cuda()
    assert bool(sees.any()) and not bool(sees.all())
    slot = int(c.lens[1]) + node
    c.pool[side][0, c.table[1, slot // 64], :, slot % 64] = 0x7f
    table, lens = c.dev("table", "lens")
    o2, l2, st = sv.kv_attention(c.cache(sv), table, lens, q, mask=words, return_lse=True)
    assert int(st.item()) == 0
    assert bool(o2[1, sees].isnan().all())
    assert torch.equal(o2[1, ~sees], out[1, ~sees]) and torch.equal(o2[0], out[0])
    assert torch.equal(l2[1, ~sees], lse[1, ~sees]) and torch.equal(l2[0], lse[0])


@pytest.mark.parametrize("N,Hq,D", [(300, 4, 128), (520, 8, 64)])
def test_attention_nan_value_in_a_prompt(sv, N, Hq, D):
    """A prompt's token whose value has one NaN: that dim of the queries from it on is NaN (all of their
    dims may be), the queries before it are as before."""
    c = Case(N + D, [70, 5], N, 1, D, 64)
    q = rand16(c.rng, (2, N, Hq, D), torch.bfloat16)
    table, lens = c.dev("table", "lens")
    out, lse, _ = sv.kv_attention(c.cache(sv), table, lens, q, return_lse=True)
    for token in (0, 10, 200):
        slot = int(c.lens[0]) + token
        at = (0, c.table[0, slot // 64], 0, slot % 64, 3)
        keep = c.pool[1][at]
        c.pool[1][at] = 0x7f
        o2, l2, st = sv.kv_attention(c.cache(sv), table, lens, q, return_lse=True)
        c.pool[1][at] = keep
        assert int(st.item()) == 0
        assert bool(o2[0, token:, :, 3].isnan().all())
        assert torch.equal(o2[0, :token], out[0, :token]) and torch.equal(o2[1], out[1])
        assert torch.equal(l2[0, :token], lse[0, :token]) and torch.equal(l2[1], lse[1])


def test_attention_nan_query_stays_in_its_row(sv):
    c = Case(14, [100, 30], 3, 2, 128, 16)
    q = rand16(c.rng, (2, 3, 4, 128), torch.bfloat16)
    out, _ = check_attention(sv, c, q)
    for bad in (float("nan"), float("inf")):
        q2 = q.clone()
        q2[0, 1, 2, 5] = bad
        table, lens = c.dev("table", "lens")
        o2, _, _ = sv.kv_attention(c.cache(sv), table, lens, q2)
        assert bool(o2[0, 1, 2].isnan().all())
        o2[0, 1, 2] = out[0, 1, 2]
        assert torch.equal(o2, out)


def test_attention_extreme_queries(sv):
    """Rows of very different magnitude share a tile: each keeps its own precision."""
    c = Case(15, [333], 6, 1, 128, 64)
    q = rand16(c.rng, (1, 6, 4, 128), torch.bfloat16)
    q = (q.float() * torch.exp2(torch.linspace(-100, 3, 24)).view(1, 6, 4, 1).cuda()).bfloat16()
    q[0, 0, 0] = 0
    check_attention(sv, c, q)


def test_attention_strided_queries_streams_and_shared_pages(sv):
    c = Case(16, [200, 200, 190], 5, 2, 128, 64)
    c.table[1, :3] = c.table[0, :3]   # a shared prefix
    qkv = rand16(c.rng, (3, 5, 8 + 4, 128), torch.bfloat16)
    q = qkv[:, :, :8]
    want, _ = check_attention(sv, c, q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = check_attention(sv, c, q.contiguous(), stream=s)
    assert torch.equal(want, got)


def test_attention_repeats_bit_for_bit(sv):
    c = Case(17, [5000, 3000, 1, 0], 6, 2, 128, 64)
    q = rand16(c.rng, (4, 6, 16, 128), torch.bfloat16)
    table, lens = c.dev("table", "lens")
    cache = c.cache(sv)
    ws = sv.new_attention_workspace(4, 6, 16, 2, 128)
    runs = []
    for fill in (0, 255, 85):   # the workspace's contents do not matter
        ws.fill_(fill)
        runs.append(sv.kv_attention(cache, table, lens, q, return_lse=True, workspace=ws)[:2])
    torch.cuda.synchronize()
    for o, l in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(l, runs[0][1])


def test_attention_in_a_graph(sv):
    """Captured once, replayed with longer sequences."""
    c = Case(18, [40, 700], 4, 2, 128, 32, junk=False)
    q = rand16(c.rng, (2, 4, 4, 128), torch.bfloat16)
    table, lens = c.dev("table", "lens")
    cache, ws = c.cache(sv), sv.new_attention_workspace(2, 4, 4, 2, 128)
    out, st = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda: sv.kv_attention(cache, table, lens, q, out=out, workspace=ws, status=st)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for now in ([40, 700], [57, 13], [0, 703]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        c.lens = np.array(now, np.int32)
        want, _ = check_attention(sv, c, q, cache=cache)
        assert torch.equal(out, want)


def test_attention_bad_data(sv):
    """Lengths and page numbers out of range: that sequence is NaN and reported, the others are
    what they were."""
    c = Case(19, [100, 200, 300], 3, 2, 128, 64)
    q = rand16(c.rng, (3, 3, 4, 128), torch.bfloat16)
    good, _ = check_attention(sv, c, q)
    for kind, code in (("neg", -25), ("long", -25), ("count", -25), ("page", -26), ("page-", -26)):
        table, lens = c.dev("table", "lens")
        nl = torch.full((3,), 3, dtype=torch.int32, device="cuda")
        if kind == "neg":
            lens[1] = -5
        elif kind == "long":
            lens[1] = 2 ** 31 - 2
        elif kind == "count":
            nl[1] = 4
        else:
            table[1, 1] = 10 ** 6 if kind == "page" else -1
        out, lse, st = sv.kv_attention(c.cache(sv), table, lens, q, new_lens=nl, return_lse=True)
        torch.cuda.synchronize()
        assert int(st.item()) == code, kind
        assert bool(out[1].isnan().all()) and bool(lse[1].isnan().all()), kind
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])


# ------------------------------------------------------------------ append

def rope_table(rows, R):
    a = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(0, R, 2) / R)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def check_append(sv, c, Hq, dtype, R, pairs, words=None, positions=None, new_lens=None,
                 packed=True, x=None, code=0):
    cache = c.cache(sv)
    table, lens = c.dev("table", "lens")
    if x is None:
        x = rand16(c.rng, (c.B, c.N, Hq + 2 * c.Hkv, c.D), dtype)
    q, k, v = x.split([Hq, c.Hkv, c.Hkv], 2)
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    rope = rope_table(int(c.lens.max()) + c.N + 1, R) if R else None
    nl = None if new_lens is None else torch.tensor(new_lens, dtype=torch.int32).cuda()
    pos = None if positions is None else torch.from_numpy(positions).cuda()
    qo, st = sv.kv_append(cache, table, lens, k, v, q=q if Hq else None,
                          rope=None if rope is None else torch.from_numpy(rope).cuda(),
                          interleaved=pairs, mask=words, positions=pos, new_lens=nl)
    torch.cuda.synchronize()
    assert int(st.item()) == code
    got = [t.view(torch.uint8).cpu().numpy()[0] for t in (cache.k, cache.v)]
    gots = [t.cpu().numpy()[0] for t in (cache.k_scale, cache.v_scale)]
    want = [p[0].copy() for p in c.pool]
    wants = [s[0].copy() for s in c.scale]
    touched = [np.zeros(p.shape[:3], bool) for p in want]   # rows checked by value
    bits = None if words is None else ref.mask_bits(words.cpu().numpy(), c.N)
    for b in range(c.B):
        n = c.N if new_lens is None else new_lens[b]
        L = int(c.lens[b])
        where = lambda i: positions[b, i] if positions is not None else \
            L + (i if bits is None else int(bits[b, i].sum()) - 1)
        rows = []
        for side, t in ((0, k), (1, v)):
            y = f64(t[b])
            e = np.zeros_like(y)
            if side == 0 and R:
                e = e + np.abs(y).max() * 2 * 2.0 ** -22   # two products in fp32
                y = np.stack([ref.rotated(y[i], rope, where(i), pairs) for i in range(c.N)])
            rows.append((y, e))
        if Hq:
            y = f64(q[b])
            if R:
                y = np.stack([ref.rotated(y[i], rope, where(i), pairs) for i in range(c.N)])
            g = f64(qo[b])[:n]
            tol = HALF[dtype] * np.abs(y[:n]) + np.abs(y).max(initial=0) * 2 * 2.0 ** -22 + 2.0 ** -25
            assert (np.abs(g - y[:n]) <= tol).all()
        for p in range(L // c.page, (L + n - 1) // c.page + 1 if n else 0):
            pg, p0 = c.table[b, p], p * c.page
            lo, hi = max(L, p0), min(L + n, p0 + c.page)
            for side in range(2):
                y, e = rows[side]
                for h in range(c.Hkv):
                    new = y[lo - L:hi - L, h]
                    s = ref.scale_for(np.abs(new).max())
                    if lo > p0:
                        s = max(s, wants[side][pg, h])
                    assert gots[side][pg, h] == np.float32(s), (b, p, side, h)
                    have = ref.E4M3[got[side][pg, h]]
                    z = new / s
                    tol = ref.half_step(z) * (1 + 2.0 ** -10) + e[lo - L:hi - L, h] / s
                    assert (np.abs(have[lo - p0:hi - p0] - z) <= tol).all()
                    if lo > p0:
                        old = ref.E4M3[want[side][pg, h, :lo - p0]] * (wants[side][pg, h] / s)
                        assert (np.abs(have[:lo - p0] - old) <=
                                (0 if s == wants[side][pg, h] else ref.half_step(old))).all()
                    wants[side][pg, h] = s
                touched[side][pg, :, :hi - p0] = True
    for side in range(2):   # nothing else changed
        np.testing.assert_array_equal(got[side][~touched[side]], want[side][~touched[side]])
        np.testing.assert_array_equal(gots[side], wants[side])
    return cache, qo


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,Hq,Hkv,D,page,R,pairs", [
    (1, 8, 2, 128, 64, 128, False), (1, 1, 1, 64, 16, 0, False), (3, 4, 4, 64, 16, 32, True),
    (17, 8, 1, 128, 16, 64, False), (40, 6, 3, 64, 32, 64, True), (130, 2, 2, 128, 128, 128, True),
    (200, 4, 1, 128, 64, 16, False), (7, 0, 2, 128, 128, 128, False)])
def test_append(sv, dtype, N, Hq, Hkv, D, page, R, pairs):
    c = Case(N + D + R, [0, 1, 15, 16, 63, 64, 65, 200], N, Hkv, D, page)
    check_append(sv, c, Hq, dtype, R, pairs, packed=N % 2 == 1)


@pytest.mark.parametrize("pairs", [False, True])
def test_append_keys_are_the_exact_rotation_rounded_once(sv, pairs):
    """Four million keys: every byte is the e4m3 value nearest to the exact rotation (ties to even)."""
    B, N, Hkv, D, page = 4, 512, 16, 128, 64
    rng = np.random.default_rng(17 + pairs)
    cache = sv.new_kv_cache(B * N // page, Hkv, D, page)
    table = torch.arange(B * N // page, dtype=torch.int32).view(B, -1).cuda()
    k = rand16(rng, (B, N, Hkv, D), torch.bfloat16)
    rope = rope_table(N, D)
    sv.kv_append(cache, table, torch.zeros(B, dtype=torch.int32, device="cuda"), k, k,
                 rope=torch.from_numpy(rope).cuda(), interleaved=pairs)
    codes, scales = cache.k.view(torch.uint8).cpu().numpy()[0], cache.k_scale.cpu().numpy()[0]
    x = f64(k)
    for b in range(B):
        y = np.stack([ref.rotated(x[b, i], rope, i, pairs) for i in range(N)])
        y = y.reshape(N // page, page, Hkv, D).transpose(0, 2, 1, 3)   # as the pages lie
        at = slice(b * N // page, (b + 1) * N // page)
        z = y / scales[at][:, :, None, None]
        step = 2 * ref.half_step(z)
        np.testing.assert_array_equal(ref.E4M3[codes[at]], np.rint(z / step) * step)


@pytest.mark.parametrize("N", [2, 33, 64])
def test_append_tree_positions(sv, N):
    c = Case(N, [0, 10, 64, 100], N, 2, 128, 64)
    check_append(sv, c, 4, torch.bfloat16, 128, False, words=tree_words(c.rng, 4, N, sv))


def test_append_given_positions_and_padding(sv):
    c = Case(31, [50, 0, 16, 7], 20, 2, 64, 16)
    pos = c.rng.integers(0, 60, (4, 20)).astype(np.int32)
    check_append(sv, c, 2, torch.float16, 64, True, positions=pos, new_lens=[20, 0, 3, 16])


def test_append_zeros_and_large_values(sv):
    """An all-zero page gets the smallest scale, bf16 values far outside fp16's range their own."""
    c = Case(32, [5, 64, 64], 4, 1, 64, 64)
    x = rand16(c.rng, (3, 4, 3, 64), torch.bfloat16)
    x[1] = 0
    x[2] *= 1e30
    cache, _ = check_append(sv, c, 1, torch.bfloat16, 0, False, x=x)
    assert float(cache.k_scale[0, int(c.table[1, 1]), 0]) == 2.0 ** -64


def test_append_nonfinite_values_are_reported(sv):
    c = Case(33, [0, 0], 4, 1, 64, 16)
    x = rand16(c.rng, (2, 4, 3, 64), torch.bfloat16)
    x[0, 1, 2, 3] = float("nan")
    x[0, 2, 2, 4] = float("-inf")
    cache = c.cache(sv)
    table, lens = c.dev("table", "lens")
    _, st = sv.kv_append(cache, table, lens, x[:, :, 1:2], x[:, :, 2:])
    assert int(st.item()) == sv.SPEC_ERR_NONFINITE
    row = ref.E4M3[cache.v.view(torch.uint8).cpu().numpy()[0, c.table[0, 0], 0]]
    assert np.isnan(row[1, 3]) and row[2, 4] == -448
    fin = f64(x[0, :, 2])
    s = ref.scale_for(np.abs(fin[np.isfinite(fin)]).max())
    assert float(cache.v_scale[0, int(c.table[0, 0]), 0]) == s


def test_append_bad_data(sv):
    """Bad lengths, pages and positions are reported; what they do not concern is written."""
    for kind, code in (("neg", -25), ("long", -25), ("count", -25), ("page", -26), ("pos", -27)):
        c = Case(34, [10, 20, 30], 3, 1, 64, 16)
        x = rand16(c.rng, (3, 3, 1, 64), torch.bfloat16)
        cache = c.cache(sv)
        table, lens = c.dev("table", "lens")
        nl = torch.full((3,), 3, dtype=torch.int32, device="cuda")
        pos = torch.zeros((3, 3), dtype=torch.int32, device="cuda")
        if kind == "neg":
            lens[1] = -1
        elif kind == "long":
            lens[1] = 2 ** 31 - 2
        elif kind == "count":
            nl[1] = -1
        elif kind == "page":
            table[1, 1] = cache.num_pages
        else:
            pos[1, 2] = 99
        rope = torch.from_numpy(rope_table(50, 64)).cuda()
        q, st = sv.kv_append(cache, table, lens, x, x, q=x, rope=rope, new_lens=nl, positions=pos)
        torch.cuda.synchronize()
        assert int(st.item()) == code, kind
        before = c.pool[1][0]
        after = cache.v.view(torch.uint8).cpu().numpy()[0]
        changed = {int(p) for p in np.argwhere((before != after).any((1, 2, 3)))[:, 0]}
        mine = {int(c.table[0, 0]), int(c.table[2, 1]), int(c.table[2, 2])}
        assert changed == (mine | {int(c.table[1, 1])} if kind == "pos" else mine), kind


def test_append_in_place_queries(sv):
    c = Case(35, [3, 77], 9, 2, 128, 32)
    x = rand16(c.rng, (2, 9, 4, 128), torch.bfloat16)
    k = rand16(c.rng, (2, 9, 2, 128), torch.bfloat16)
    rope = torch.from_numpy(rope_table(100, 128)).cuda()
    table, lens = c.dev("table", "lens")
    for pairs in (False, True):
        want, _ = sv.kv_append(c.cache(sv), table, lens, k, k, q=x, rope=rope, interleaved=pairs)
        y = x.clone()
        got, _ = sv.kv_append(c.cache(sv), table, lens, k, k, q=y, q_out=y, rope=rope,
                              interleaved=pairs)
        assert got.data_ptr() == y.data_ptr() and torch.equal(want, got)


# ------------------------------------------------------------------ commit

def check_commit(sv, c, paths, code=0, layers=1):
    """paths: the accepted nodes of each sequence (root first), or None for accept_len -1."""
    cache = c.cache(sv)
    table, lens = c.dev("table", "lens")
    pn = np.full((c.B, c.N), -1, np.int32)
    for b, p in enumerate(paths):
        if p:
            pn[b, :len(p)] = p
    acc = np.array([len(p) - 1 if p else -1 for p in paths], np.int32)
    out, st = sv.kv_commit(cache, table, lens, torch.from_numpy(pn).cuda(),
                           torch.from_numpy(acc).cuda())
    torch.cuda.synchronize()
    assert int(st.item()) == code
    np.testing.assert_array_equal(out.cpu().numpy(), c.lens + acc + 1)
    got = [t.view(torch.uint8).cpu().numpy() for t in (cache.k, cache.v)]
    gots = [t.cpu().numpy() for t in (cache.k_scale, cache.v_scale)]
    for side in range(2):
        for lay in range(layers):
            was, ws = ref.E4M3[c.pool[side][lay]], c.scale[side][lay].astype(np.float64)
            want, s = was * ws[:, :, None, None], ws.copy()
            dest = np.zeros(want.shape[:3], bool)
            for b, p in enumerate(paths):
                L = int(c.lens[b])
                for k, node in enumerate(p or []):
                    if node != k:
                        f, t = L + node, L + k
                        pf, pt = c.table[b, f // c.page], c.table[b, t // c.page]
                        row = was[pf, :, f % c.page] * ws[pf][:, None]
                        want[pt, :, t % c.page] = row
                        dest[pt, :, t % c.page] = True
                        for h in range(c.Hkv):
                            s[pt, h] = max(s[pt, h], ref.scale_for(np.abs(row[h]).max()))
            np.testing.assert_array_equal(gots[side][lay], s.astype(np.float32))
            have = ref.E4M3[got[side][lay]]
            z = want / s[:, :, None, None]
            same = (s == ws)[:, :, None] & ~dest
            # a row may be stored twice on its way (its page's scale grew, then it moved)
            tol = np.where(same[..., None], 0, 2 * ref.half_step(z))
            exact = np.abs(z) >= 2.0 ** -6   # between powers of two only subnormals round
            assert (np.abs(have - z) <= np.where(exact, 0, tol)).all()
            np.testing.assert_array_equal(got[side][lay][same], c.pool[side][lay][same])


@pytest.mark.parametrize("D,page,Hkv", [(128, 16, 2), (64, 64, 1), (128, 128, 3), (64, 16, 4)])
def test_commit(sv, D, page, Hkv):
    N = 40
    c = Case(D + page, [0, 1, 13, 15, 63, 64, 100, 250], N, Hkv, D, page, layers=2)
    paths = [[0], [0, 1, 2], None, [0, 3, 9, 30], [0, 2, 3, 4, 39], list(range(40)), [0, 39],
             [0] + list(range(5, 40))]
    check_commit(sv, c, paths, layers=2)


def test_commit_many_layers_and_one_node(sv):
    c = Case(41, [10, 17], 1, 2, 64, 16, layers=5)
    check_commit(sv, c, [[0], None], layers=5)


def test_commit_bad_data(sv):
    c = Case(42, [10, 20, 30], 8, 1, 64, 16)
    for kind, code in (("acc", -28), ("order", -28), ("root", -28), ("range", -28), ("neg", -25),
                       ("page", -26)):
        cache = c.cache(sv)
        table, lens = c.dev("table", "lens")
        pn = torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
        pn[:, :3] = torch.tensor([0, 4, 7], dtype=torch.int32)
        acc = torch.full((3,), 2, dtype=torch.int32, device="cuda")
        want = [13, 20, 33]
        if kind == "acc":
            acc[1] = 8
        elif kind == "order":
            pn[1, 2] = 4
        elif kind == "root":
            pn[1, 0] = 1
        elif kind == "range":
            pn[1, 2] = 8
        elif kind == "neg":
            lens[1] = want[1] = -3
        else:
            table[1, 1] = -1
            want[1] = 23
        out, st = sv.kv_commit(cache, table, lens, pn, acc)
        torch.cuda.synchronize()
        assert int(st.item()) == code, kind
        assert out.cpu().tolist() == want
        same = cache.k.view(torch.uint8).cpu().numpy()[0, c.table[1, :2]] == c.pool[0][0, c.table[1, :2]]
        assert same.all(), kind


# ------------------------------------------------------------------ together

def test_verify_step(sv):
    """Draft tree -> append -> attention -> verify -> commit, against the same tokens appended in
    order: the kept path's keys and values are what a plain decode would have stored."""
    N, Hq, Hkv, D, page, V = 12, 4, 2, 64, 16, 50
    c = Case(51, [33, 5], N, Hkv, D, page)
    cache = c.cache(sv)
    table, lens = c.dev("table", "lens")
    rng = c.rng
    par = torch.tensor([[-1, 0, 0, 1, 1, 2, 3, 3, 5, 6, 6, 8]] * 2, dtype=torch.int32).cuda()
    mask, _ = sv.tree_mask(par)
    x = rand16(rng, (2, N, Hq + 2 * Hkv, D), torch.bfloat16)
    q, k, v = x.split([Hq, Hkv, Hkv], 2)
    rope = torch.from_numpy(rope_table(80, D)).cuda()
    qr, st = sv.kv_append(cache, table, lens, k, v, q=q, rope=rope, mask=mask)
    out, _, st = sv.kv_attention(cache, table, lens, qr, mask=mask, status=st)
    logits = torch.zeros(2, N, V, device="cuda")
    tok = torch.arange(N, dtype=torch.int32).repeat(2, 1).cuda()
    for node, child in ((0, 2), (2, 5), (5, 8), (8, 40)):   # the target's choices: 2, 5, 8, 40
        logits[:, node, child] = 5.0
    acc, path, toks, _ = sv.verify_tree(logits, par, tok)
    new, st = sv.kv_commit(cache, table, lens, path, acc, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and acc.tolist() == [3, 3] and new.tolist() == [37, 9]
    plain = c.cache(sv)
    keep = torch.tensor([0, 2, 5, 8]).cuda()
    qp, _ = sv.kv_append(plain, table, lens, k[:, keep].contiguous(), v[:, keep].contiguous(),
                         q=q[:, keep].contiguous(), rope=rope)
    assert torch.equal(qp, qr[:, keep])
    got = [t.view(torch.uint8).cpu().numpy()[0] for t in (cache.k, cache.v, plain.k, plain.v)]
    sc = [t.cpu().numpy()[0] for t in (cache.k_scale, cache.v_scale, plain.k_scale, plain.v_scale)]
    for b in range(2):
        n = int(new[b])
        for side in range(2):
            a = ref.cached(got[side], sc[side], c.table[b], n, page)
            w = ref.cached(got[2 + side], sc[2 + side], c.table[b], n, page)
            # the tree's other nodes may have raised a page's scale: subnormals then round anew
            step = sc[side][c.table[b][np.arange(n) // page]][:, :, None] * 2.0 ** -9
            assert (np.abs(a - w) <= 1.5 * step).all()
    # and the deepest node's attention is a plain decode's over the committed cache
    last = lens + 3
    o1, _, _ = sv.kv_attention(plain, table, last, qp[:, 3:].contiguous())
    err = (out[:, 8].float() - o1[:, 0].float()).abs().max()
    assert float(err) < 2.0 ** -4


def test_example():
    """The example's steps run, accept some drafts, and repeat themselves token for token."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "verify_step.py")
    spec = importlib.util.spec_from_file_location("verify_step", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    emitted, lens, status = ex.run(steps=2, batch=2, nodes=8, layers=2)
    assert int(status.item()) == 0
    assert all(len(e) >= 3 for e in emitted) and any(len(e) > 3 for e in emitted)
    again, lens2, _ = ex.run(steps=2, batch=2, nodes=8, layers=2)
    assert again == emitted and torch.equal(lens, lens2)


# ------------------------------------------------------------------ large offsets, streams, checks

def test_offsets_past_32_bits(sv):
    """A pool of more than 4 GiB a side: pages at its far end."""
    Hkv, D, page, pages = 8, 128, 128, 33000
    assert pages * Hkv * page * D > 1 << 32
    cache = sv.new_kv_cache(pages, Hkv, D, page)
    small = sv.new_kv_cache(8, Hkv, D, page)
    rng = np.random.default_rng(71)
    lens = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    far = torch.tensor([[32999, 32768], [16384, 32991]], dtype=torch.int32, device="cuda")
    near = torch.tensor([[0, 3], [5, 1]], dtype=torch.int32, device="cuda")
    x = rand16(rng, (2, 200, 16 + 2 * Hkv, D), torch.bfloat16)
    q, k, v = x.split([16, Hkv, Hkv], 2)
    out = []
    for c, t in ((cache, far), (small, near)):
        qo, st = sv.kv_append(c, t, lens, k, v, q=q)
        o, lse, st = sv.kv_attention(c, t, lens, qo, return_lse=True, status=st)
        now = lens + 150
        path = torch.full((2, 50), -1, dtype=torch.int32, device="cuda")
        path[:, :3] = torch.tensor([0, 20, 49], dtype=torch.int32)
        new, st = sv.kv_commit(c, t, now, path, torch.full((2,), 2, dtype=torch.int32, device="cuda"),
                               status=st)
        o1, _, st = sv.kv_attention(c, t, new - 1, q[:, :1].contiguous(), status=st)
        assert int(st.item()) == 0
        out.append((o, lse, new, o1))
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_two_streams_at_once(sv):
    """Calls in flight on two streams, each with its own workspace."""
    cs = [Case(72 + i, [3000 + 500 * i, 700, 90], 5, 2, 128, 64) for i in range(2)]
    qs = [rand16(c.rng, (3, 5, 8 * (i + 1), 128), torch.bfloat16) for i, c in enumerate(cs)]
    want = [check_attention(sv, c, q)[0] for c, q in zip(cs, qs)]
    args = [(c.cache(sv), *c.dev("table", "lens"), q) for c, q in zip(cs, qs)]
    streams = [torch.cuda.Stream() for _ in cs]
    ws = [sv.new_attention_workspace(3, 5, q.shape[2], 2, 128) for q in qs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(sv.kv_attention(*args[i], workspace=ws[i])[0])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for o in g:
            assert torch.equal(o, w)


def test_checked_build(sv):
    """The checked build (indices range-checked) reports nothing and gives the same results."""
    import speculative_decoding_verification_78_gb300._binding as bnd
    plain, checked = bnd.load_library(), bnd.load_library(checked=True)
    saved = bnd.load_library
    results = []
    for lib in (plain, checked):
        bnd.load_library = lambda checked=False, lib=lib: lib
        try:
            out = []
            for N, Hq, dtype, tree in ((1, 8, torch.bfloat16, False), (9, 8, torch.float16, True),
                                       (40, 16, torch.bfloat16, True), (70, 4, torch.bfloat16, False)):
                c = Case(81 + N, [0, 77, 600], N, 2, 128, 32)
                cache = c.cache(sv)
                table, lens = c.dev("table", "lens")
                words = tree_words(c.rng, 3, N, sv) if tree else None
                x = rand16(c.rng, (3, N, Hq + 4, 128), dtype)
                q, k, v = x.split([Hq, 2, 2], 2)
                rope = torch.from_numpy(rope_table(800, 128)).cuda()
                qo, st = sv.kv_append(cache, table, lens, k, v, q=q, rope=rope, mask=words)
                o, lse, st = sv.kv_attention(cache, table, lens, qo, mask=words, return_lse=True,
                                             status=st)
                path = torch.full((3, N), -1, dtype=torch.int32, device="cuda")
                acc = min(N - 1, 1)
                path[:, 0] = 0
                if acc:
                    path[:, 1] = N - 1
                new, st = sv.kv_commit(cache, table, lens, path,
                                       torch.full((3,), acc, dtype=torch.int32, device="cuda"),
                                       status=st)
                torch.cuda.synchronize()
                assert int(st.item()) == 0
                out += [qo, o, lse, new, cache.k.view(torch.uint8), cache.k_scale]
            results.append(out)
        finally:
            bnd.load_library = saved
    for a, b in zip(*results):
        assert torch.equal(a, b)
