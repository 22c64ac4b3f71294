"""GPU parity of the KV-cache operators in every form of their kernels: the row counts, head dims and types
that choose one, and the paths inside that random data seldom takes."""

import numpy as np
import pytest
import torch

import kv_ref as ref
import test_gpu_kv as kv
from test_gpu_kv import Case, check_attention, f64, rand16, rope_table, tree_words

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import speculative_decoding_verification_78_gb300 as sv
    sv.load_library()
    return sv


# ------------------------------------------------------------------ scratch on the stream of the call

@pytest.mark.parametrize("raw", [False, True])
def test_scratch_of_a_call_on_another_stream(sv, raw):
    """The workspace that kv_attention makes for itself stays its own until the call has ended, whatever
    the current stream allocates meanwhile; and a reported status is not zeroed afterwards."""
    c = Case(91, [6000, 2500], 1, 2, 128, 64)
    q = rand16(c.rng, (2, 1, 8, 128), torch.bfloat16)
    want, wlse = check_attention(sv, c, q)
    table, lens = c.dev("table", "lens")
    cache = c.cache(sv)
    bad = table.clone()
    bad[0, 1] = -1
    size = sv.spec_kv_attention_workspace_bytes(2, 1, 8, 2, 128)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for pages, code in ((table, 0), (bad, sv.SPEC_ERR_PAGE)):
        with torch.cuda.stream(s):
            torch.cuda._sleep(100_000_000)   # about 50 ms: the call waits behind it
        out, lse, st = sv.kv_attention(cache, pages, lens, q, return_lse=True,
                                       stream=s.cuda_stream if raw else s)
        junk = [torch.full((n,), 0x3f, dtype=torch.uint8, device="cuda")
                for n in (size, size, out.numel() * 2, lse.numel() * 4, 4, 4) for _ in range(2)]
        torch.cuda.synchronize()
        assert int(st.item()) == code
        assert torch.equal(out[1], want[1]) and torch.equal(lse[1], wlse[1])
        if code == 0:
            assert torch.equal(out, want) and torch.equal(lse, wlse)
        assert all(bool((j == 0x3f).all()) for j in junk)


# ------------------------------------------------------------------ references that rise

@pytest.mark.parametrize("G", [16, 32])
def test_a_row_whose_reference_rises_leaves_the_others_sums(sv, G):
    """Rows share tiles with one whose scores rise by more than 2^7 a tile, so that every tile is weighed
    twice. What the first time added to the others' sums is taken off again to half a unit of the sum: of
    6 tiles a group at most 3.5 x 2^-24, 2^-21.7 of a base-2 logarithm, which is held in steps of 2^-18 (the
    values' scale is 2^70): at most one row in 13 may show it, and one in 8 is let pass."""
    B, Hkv, D, page, tiles = 19, 8, 64, 64, 12
    n = 128 * tiles
    rng = np.random.default_rng(G)
    k = np.zeros((B, n, Hkv, D), np.float32)
    k[..., 1:] = rng.integers(-8, 9, (B, 1, Hkv, D - 1))   # every token the same but for dim 0
    k[..., 0] = (np.arange(n) // 128)[None, :, None]
    pages = B * n // page

    def pool(x):   # [B, n, Hkv, D] -> pages in order
        x = x.reshape(pages, page, Hkv, D).transpose(0, 2, 1, 3)
        return torch.from_numpy(np.ascontiguousarray(x)).cuda().to(kv.E4)

    v = pool(rng.integers(-8, 9, k.shape).astype(np.float32))
    one = torch.ones(pages, Hkv, device="cuda")
    cache = sv.KVCache(pool(k), v, one, one * 2.0 ** 70)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(B, -1)
    lens = torch.full((B,), n - 1, dtype=torch.int32, device="cuda")
    q = rand16(rng, (B, 1, Hkv * G, D), torch.bfloat16, 0.05)
    q[..., 0] = 0
    lses = []
    for rising in (0.0, 16.0):
        r = q.clone()
        r[:, :, ::G] = 0
        r[:, :, ::G, 0] = rising
        _, lse, st = sv.kv_attention(cache, table, lens, r, scale=1.0, return_lse=True)
        assert int(st.item()) == 0
        lses.append(lse.view(-1, G)[:, 1:])
    assert bool(torch.isfinite(lses[0]).all())
    differ = float((lses[0] != lses[1]).float().mean())
    assert differ <= 1 / 8, differ


def test_an_empty_batch(sv):
    cache = sv.new_kv_cache(4, 2, 64, 16)
    before = cache.k.view(torch.uint8).clone()
    table = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    lens = torch.empty(0, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 3, 8, 64, dtype=torch.bfloat16, device="cuda")
    q, st = sv.kv_append(cache, table, lens, x[:, :, :2], x[:, :, :2], q=x)
    out, lse, st = sv.kv_attention(cache, table, lens, q, return_lse=True, status=st)
    new, st = sv.kv_commit(cache, table, lens, torch.empty(0, 3, dtype=torch.int32, device="cuda"), lens, status=st)
    assert int(st.item()) == 0
    assert (q.shape, out.shape, lse.shape, new.shape) == (x.shape, x.shape, x.shape[:3], lens.shape)
    assert torch.equal(cache.k.view(torch.uint8), before)


# ------------------------------------------------------------------ attention, every form

# new tokens and query heads over 2 key heads: 12 and 24 rows a key head (tokens along the MMA's rows, 16 and
# 32 columns), 80 rows (one tile of 128), 200 and 300 rows (one and two tiles of 256)
FORMS = [(3, 8), (6, 8), (20, 8), (50, 8), (75, 8)]
TYPES = [torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,Hq", FORMS)
def test_attention_scores_that_rise_in_every_tile(sv, N, Hq, D, dtype):
    """One dim carries a score that rises by about 9 (base 2) from tile to tile, so the reference of every row
    moves in each of a group's tiles; falls; or is highest at the first token. The other dims are random."""
    c = Case(200 + N + D, [1792 - N, 1500, 900], N, 2, D, 64)
    c.scale[0][:] = 2.0 ** -5
    codes = c.pool[0].view(np.uint8)
    for b in range(3):
        t = np.arange(c.lens[b] + N)
        tile = t // 128
        top = np.where(b == 2, np.where(t == 0, 14, 0), tile if b == 0 else tile.max() - tile)
        value = torch.from_numpy(32.0 * top).float().to(kv.E4).view(torch.uint8).numpy()
        codes[0, c.table[b][t // 64], :, t % 64, 0] = value[:, None]
    q = rand16(c.rng, (3, N, Hq, D), dtype)
    q[..., 0] = 6.2 * D ** 0.5
    check_attention(sv, c, q)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,Hq", FORMS)
def test_attention_value_scales_apart(sv, N, Hq, D, dtype):
    c = Case(300 + N + D, [900, 100], N, 2, D, 16)
    c.scale[1] = np.exp2(c.rng.uniform(-30, 5, c.scale[1].shape)).astype(np.float32)
    c.scale[0] *= c.rng.uniform(0.5, 1.5, c.scale[0].shape).astype(np.float32)
    check_attention(sv, c, rand16(c.rng, (2, N, Hq, D), dtype))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,Hq", FORMS)
def test_attention_queries_of_unlike_size(sv, N, Hq, D):
    c = Case(400 + N + D, [333], N, 2, D, 64)
    q = rand16(c.rng, (1, N, Hq, D), torch.bfloat16)
    up = torch.linspace(-100, 3, N * Hq)[torch.from_numpy(c.rng.permutation(N * Hq))]
    q = (q.float() * torch.exp2(up).view(1, N, Hq, 1).cuda()).bfloat16()
    q[0, 0, 0] = 0
    check_attention(sv, c, q)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,Hq", FORMS)
@pytest.mark.parametrize("tree", [False, True])
def test_attention_padding_in_every_form(sv, N, Hq, D, dtype, tree):
    c = Case(500 + N + D, [0, 5, 200, 64], N, 2, D, 32)
    words = tree_words(c.rng, 4, N, sv) if tree else None
    check_attention(sv, c, rand16(c.rng, (4, N, Hq, D), dtype), words, [0, N, N // 2, 1])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
def test_attention_first_token_seen_in_a_late_tile(sv, D, dtype):
    """Nodes that see nothing but themselves, over no cache: rows whose first token lies in the second or
    third tile, some that see none."""
    N = 300
    c = Case(600 + D, [0, 0], N, 2, D, 64)
    words = torch.zeros(2, N, 10, dtype=torch.int64)
    for i in range(N):
        words[:, i, i // 32] = 1 << (i % 32)
    words[1, ::7] = 0
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32).cuda()
    check_attention(sv, c, rand16(c.rng, (2, N, 4, D), dtype), words)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,Hq", FORMS)
def test_attention_refused_sequences_in_every_form(sv, N, Hq, D):
    """Lengths and counts out of range: that sequence is NaN and reported, the others are what they were."""
    c = Case(700 + N + D, [100, 200, 300], N, 2, D, 64)
    q = rand16(c.rng, (3, N, Hq, D), torch.bfloat16)
    good, glse = check_attention(sv, c, q)
    for kind in ("neg", "long", "count", "none"):
        table, lens = c.dev("table", "lens")
        nl = torch.full((3,), N, dtype=torch.int32, device="cuda")
        if kind == "neg":
            lens[1] = -5
        elif kind == "long":
            lens[1] = 2 ** 31 - 2
        else:
            nl[1] = N + 1 if kind == "count" else -1
        out, lse, st = sv.kv_attention(c.cache(sv), table, lens, q, new_lens=nl, return_lse=True)
        assert int(st.item()) == sv.SPEC_ERR_LENGTH, kind
        assert bool(out[1].isnan().all()) and bool(lse[1].isnan().all()), kind
        for b in (0, 2):
            assert torch.equal(out[b], good[b]) and torch.equal(lse[b], glse[b]), kind


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,Hq", FORMS)
@pytest.mark.parametrize("page", [16, 64])
def test_attention_bad_pages_in_every_form(sv, N, Hq, D, dtype, page):
    """A bad page that every query sees makes them all NaN; one that holds new tokens only, the queries from
    the first of them on. The others are what they were, bit for bit."""
    c = Case(800 + N + D, [300, 14 * page - 1], N, 2, D, page)
    q = rand16(c.rng, (2, N, Hq, D), dtype)
    good, glse = check_attention(sv, c, q)
    last = (int(c.lens[1]) + N - 1) // page
    for at in sorted({0, 7, 13, 14, last}):
        for number in (-1, int(c.table.max()) + 10 ** 6):
            table, lens = c.dev("table", "lens")
            table[1, at] = number
            out, lse, st = sv.kv_attention(c.cache(sv), table, lens, q, return_lse=True)
            assert int(st.item()) == sv.SPEC_ERR_PAGE
            first = max(0, at * page - int(c.lens[1]))   # query from which on the page is seen
            assert bool(out[1, first:].isnan().all()) and bool(lse[1, first:].isnan().all()), at
            assert torch.equal(out[1, :first], good[1, :first]), at
            assert torch.equal(lse[1, :first], glse[1, :first]), at
            assert torch.equal(out[0], good[0]) and torch.equal(lse[0], glse[0])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,Hq", FORMS)
def test_attention_rows_do_not_depend_on_others(sv, N, Hq, D):
    """A NaN query and NaN in slots past the end change nothing for the other rows."""
    c = Case(900 + N + D, [500, 77], N, 2, D, 64)
    q = rand16(c.rng, (2, N, Hq, D), torch.bfloat16)
    out, lse = check_attention(sv, c, q)
    for side in range(2):
        for b in range(2):
            n = int(c.lens[b]) + N
            c.pool[side][0, c.table[b, (n - 1) // 64], :, (n - 1) % 64 + 1:] = 0x7f
    q[0, N // 2, 1, 5] = float("nan")
    table, lens = c.dev("table", "lens")
    o2, l2, st = sv.kv_attention(c.cache(sv), table, lens, q, return_lse=True)
    assert int(st.item()) == 0
    assert bool(o2[0, N // 2, 1].isnan().all()) and bool(l2[0, N // 2, 1].isnan())
    o2[0, N // 2, 1] = out[0, N // 2, 1]
    l2[0, N // 2, 1] = lse[0, N // 2, 1]
    assert torch.equal(o2, out) and torch.equal(l2, lse)


@pytest.mark.parametrize("dtype", TYPES)
def test_attention_prompt_over_many_tiles(sv, dtype):
    c = Case(95, [0, 700], 400, 2, 128, 128)
    check_attention(sv, c, rand16(c.rng, (2, 400, 6, 128), dtype))


# ------------------------------------------------------------------ append

def check_exact_keys(sv, c, dtype, R, pairs, positions=None, words=None):
    """Every byte of a page that received keys, and its scale: the exact rotation (and what the page held)
    over the scale, rounded once to nearest, ties to even."""
    cache = c.cache(sv)
    table, lens = c.dev("table", "lens")
    k = rand16(c.rng, (c.B, c.N, c.Hkv, c.D), dtype)
    rope = rope_table(int(c.lens.max()) + c.N + 60, R) if R else None
    _, st = sv.kv_append(cache, table, lens, k, k, rope=None if rope is None else torch.from_numpy(rope).cuda(),
                         interleaved=pairs, mask=words,
                         positions=None if positions is None else torch.from_numpy(positions).cuda())
    assert int(st.item()) == 0
    codes, scales = cache.k.view(torch.uint8).cpu().numpy()[0], cache.k_scale.cpu().numpy()[0]
    bits = None if words is None else ref.mask_bits(words.cpu().numpy(), c.N)
    x = f64(k)

    def nearest(z):
        step = 2 * ref.half_step(z)
        return np.rint(z / step) * step

    for b in range(c.B):
        L = int(c.lens[b])
        if R:
            at = positions[b] if positions is not None else \
                L + (np.arange(c.N) if bits is None else bits[b].sum(-1) - 1)
            y = np.stack([ref.rotated(x[b, i], rope, int(at[i]), pairs) for i in range(c.N)])
        else:
            y = x[b]
        for p in range(L // c.page, (L + c.N - 1) // c.page + 1):
            pg, p0 = c.table[b, p], p * c.page
            lo, hi = max(L, p0), min(L + c.N, p0 + c.page)
            for h in range(c.Hkv):
                was = c.scale[0][0, pg, h]
                s = ref.scale_for(np.abs(y[lo - L:hi - L, h]).max())
                if lo > p0:
                    s = max(s, float(was))
                assert scales[pg, h] == np.float32(s)
                have = ref.E4M3[codes[pg, h]]
                np.testing.assert_array_equal(have[lo - p0:hi - p0], nearest(y[lo - L:hi - L, h] / s))
                np.testing.assert_array_equal(have[:lo - p0],
                                              nearest(ref.E4M3[c.pool[0][0, pg, h, :lo - p0]] * (float(was) / s)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,page,R,pairs", [(128, 64, 128, False), (128, 16, 64, True), (64, 32, 64, False),
                                            (64, 16, 32, True), (128, 128, 16, False), (64, 128, 0, False)])
def test_append_keys_byte_for_byte(sv, dtype, D, page, R, pairs):
    """Pages that held tokens (at scales that have to grow, and that need not) and fresh ones."""
    c = Case(D + page + R, [0, 1, page - 1, page, 5 * page // 2, 200], 150, 4, D, page)
    check_exact_keys(sv, c, dtype, R, pairs)


@pytest.mark.parametrize("dtype", TYPES)
def test_append_keys_byte_for_byte_at_given_and_tree_positions(sv, dtype):
    c = Case(77, [3, 40, 0], 60, 2, 128, 32)
    check_exact_keys(sv, c, dtype, 128, False, positions=c.rng.integers(0, 150, (3, 60)).astype(np.int32))
    check_exact_keys(sv, c, dtype, 128, True, words=tree_words(c.rng, 3, 60, sv))


@pytest.mark.parametrize("Hkv", [6, 5, 16])
def test_append_several_heads_of_a_page_a_cta(sv, Hkv):
    """Calls with so many pages that a CTA takes several heads of one in turn: heads that do not divide evenly,
    pages that held tokens."""
    c = Case(60 + Hkv, [5, 21, 0, 47], 376, Hkv, 64, 16)
    kv.check_append(sv, c, 3, torch.bfloat16, 64, False)
    check_exact_keys(sv, c, torch.float16, 32, True)


@pytest.mark.parametrize("D,Hq", [(128, 40), (128, 71), (64, 70), (64, 131)])
@pytest.mark.parametrize("pairs", [False, True])
def test_append_more_query_heads_than_a_task_takes(sv, D, Hq, pairs):
    c = Case(D + Hq, [5, 130], 7, 1, D, 32)
    kv.check_append(sv, c, Hq, torch.bfloat16, D, pairs)
    x = rand16(c.rng, (2, 7, Hq, D), torch.bfloat16)
    k = rand16(c.rng, (2, 7, 1, D), torch.bfloat16)
    rope = torch.from_numpy(rope_table(200, D)).cuda()
    table, lens = c.dev("table", "lens")
    want, _ = sv.kv_append(c.cache(sv), table, lens, k, k, q=x, rope=rope, interleaved=pairs)
    got, _ = sv.kv_append(c.cache(sv), table, lens, k, k, q=x, q_out=x, rope=rope, interleaved=pairs)
    assert got.data_ptr() == x.data_ptr() and torch.equal(want, got)


@pytest.mark.parametrize("shift", [1, 2, 3])
def test_append_rotation_table_off_16_bytes(sv, shift):
    c = Case(88, [5, 64], 40, 2, 128, 64)
    x = rand16(c.rng, (2, 40, 8, 128), torch.bfloat16)
    rope = torch.from_numpy(rope_table(120, 128)).cuda()
    off = torch.empty(rope.numel() + shift, device="cuda")[shift:].view(rope.shape)
    off.copy_(rope)
    assert off.data_ptr() % 16 == 4 * shift and off.is_contiguous()
    table, lens = c.dev("table", "lens")
    out = []
    for r in (rope, off):
        cache = c.cache(sv)
        q, st = sv.kv_append(cache, table, lens, x[:, :, 4:6], x[:, :, 6:], q=x[:, :, :4], rope=r)
        assert int(st.item()) == 0
        out.append((q, cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scale, cache.v_scale))
    for a, b in zip(*out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("sizes", [(-64, 16), (-70, 8), (0, 80)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N,Hq", FORMS)
def test_attention_value_scales_as_far_apart_as_allowed(sv, N, Hq, D, sizes):
    """Pages of two value scales 2^78 to 2^80 apart, in runs of random lengths: the small ones' values vanish
    beside the others', but their weights count. (bf16, whose range holds the outputs of either.)"""
    c = Case(1000 + N + D, [1100, 300, 128], N, 2, D, 16)
    for b in range(3):
        at = 0
        while at < c.pps:
            run = int(c.rng.integers(1, 40))
            pick = c.rng.integers(0, 2, 2)
            for h in range(2):
                c.scale[1][0, np.maximum(c.table[b, at:at + run], 0), h] = 2.0 ** sizes[pick[h]]
            at += run
    check_attention(sv, c, rand16(c.rng, (3, N, Hq, D), torch.bfloat16))
