"""Long texts and several hypotheses on the paged KV cache, as cases to measure.

attend   attention of the new tokens (one token, a candidate tree, a piece of a prompt) over the last `window` tokens
         of a paged 8-bit cache and its first few (sinks), which stay visible
select   the best continuations of a set of beams: every beam's score plus the log-probability of every token
fork     the chosen beams' caches, token histories and hidden states from those of their parents
roll     a decoding step's pages: those behind the window go back, the new tokens' places get free ones
compact  some sequences end, the pool's live pages move to its front, and new sequences take the places

`run` computes each in plain torch operations, or with the library's calls where `own` is true.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token of one sequence: the smallest call, where latency counts
        dict(name="attend_one", op="attend", dtype="bf16", B=1, N=1, Hq=32, Hkv=8, D=128, page=64, L=1000, window=512, sinks=4, tree=False),
        # one token for each sequence of a serving batch, long texts of uneven lengths
        dict(name="attend_decode", op="attend", dtype="bf16", B=64, N=1, Hq=32, Hkv=8, D=128, page=64, L=16000, window=4096, sinks=4, tree=False),
        # candidate trees of 64 nodes, four query heads to a key head
        dict(name="attend_tree", op="attend", dtype="bf16", B=32, N=64, Hq=32, Hkv=8, D=128, page=64, L=8192, window=2048, sinks=64, tree=True),
        # pieces of two prompts, longer than the window, small pages and heads
        dict(name="attend_prompt", op="attend", dtype="fp16", B=2, N=1500, Hq=16, Hkv=2, D=64, page=16, L=5003, window=1000, sinks=16, tree=False),
        # four beams of one sequence: the smallest call
        dict(name="select_one", op="select", dtype="fp32", B=1, K=4, V=32000, n=4, done=False),
        # eight beams of 64 sequences, twice as many candidates as beams, some beams at their end
        dict(name="select_batch", op="select", dtype="bf16", B=64, K=8, V=152064, n=16, done=True),
        # four beams in one layer
        dict(name="fork_one", op="fork", B=1, K=4, Hkv=2, D=64, page=16, L=1000, layers=1, hidden=512, ends=True),
        # eight beams of 16 sequences in 32 layers
        dict(name="fork_beams", op="fork", B=16, K=8, Hkv=8, D=128, page=64, L=500, layers=32, hidden=4096, ends=True),
        # a batch of single tokens that crosses a page now and then
        dict(name="roll_decode", op="roll", B=16, N=1, page=16, L=3000, window=1024, sinks=4),
        # candidate trees of 64 nodes for each sequence of a large batch
        dict(name="roll_tree", op="roll", B=256, N=64, page=16, L=9000, window=4096, sinks=4),
        # a small pool
        dict(name="compact_small", op="compact", B=8, Hkv=2, D=64, page=16, L=300, layers=1),
        # 16 layers of a pool that half of its sequences leave
        dict(name="compact_pool", op="compact", B=32, Hkv=8, D=128, page=64, L=2000, layers=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "select", "select", "fork", "fork", "roll", "compact"])
    if op == "select":
        B, K = _log(rng, 1, 64), rng.choice([1, 2, 3, 4, 5, 8, 12, 16])
        dtype = rng.choice(["bf16", "fp32"])
        V = _log(rng, 1000, min(152064, 70_000_000 // (B * K * (2 if dtype == "fp32" else 1))))
        return dict(op=op, dtype=dtype, B=B, K=K, V=V, n=rng.choice([K, 2 * K, rng.randint(1, 32)]), done=rng.random() < 0.5)
    page = rng.choice([16, 32, 64, 128])
    if op == "roll":
        B = _log(rng, 1, 256)
        L = _log(rng, 1, min(9000, 9000 * 256 // B, 144 * page))
        return dict(op=op, B=B, N=_log(rng, 1, 64), page=page, L=L, window=_log(rng, 1, 8000), sinks=rng.choice([0, 1, 4, page, 100]))
    D, Hkv = rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 8])
    if op == "fork":
        K, layers = rng.choice([1, 2, 3, 4, 8]), _log(rng, 1, 32)
        B = _log(rng, 1, 128 // K)
        L = _log(rng, 1, min(8000, max(2, 8 * 64 * 32 * 16 * 8 // (layers * B * Hkv))))
        return dict(op=op, B=B, K=K, Hkv=Hkv, D=D, page=page, L=L, layers=layers, hidden=8 * rng.randint(1, 512), ends=rng.random() < 0.6)
    if op == "compact":
        B, layers = rng.randint(2, 32), _log(rng, 1, 16)
        return dict(op=op, B=B, Hkv=Hkv, D=D, page=page, L=_log(rng, 1, 2000), layers=layers)
    G = rng.choice([1, 2, 4, 8])
    tree = rng.random() < 0.4
    B = _log(rng, 1, 64)
    N = rng.randint(2, 96) if tree else _log(rng, 1, 600)
    # keys seen by the batch, and products, no more than the largest listed cases have
    most = max(2, min(2_000_000 // (B * Hkv), int(1.1e8 / (B * N * Hkv * G)), 4500))
    window = max(_log(rng, 1, most), N if tree else 1)
    return dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16"]), B=B, N=N, Hq=Hkv * G, Hkv=Hkv, D=D, page=page, L=_log(rng, 1, max(2, min(16000, 8_000_000 // (B * Hkv)))),
                window=window, sinks=rng.choice([0, 1, 4, page, 130]), tree=tree)


def _uneven(c, n):
    """Lengths between half of L and L, the first one L."""
    return [c["L"] - (b * 37) % (c["L"] // 2 + 1) for b in range(n)]


def _parents(c):
    """The parent of each beam, some of them more than once; or of the samples of each prompt."""
    B, K = c["B"], c["K"]
    if not c["ends"]:
        return [b for b in range(B) for _ in range(K)]
    return [b * K + (j * 2 // 3 + b) % K for b in range(B) for j in range(K)]


def work(case):
    c = case
    if c["op"] == "attend":
        B, N, Hkv, D = c["B"], c["N"], c["Hkv"], c["D"]
        keys = pairs = 0
        for n in _uneven(c, B):
            start = max(0, n - c["window"] + 1)
            early = min(c["sinks"], start)
            keys += early + n + N - start
            if c["tree"]:
                pairs += N * (early + n - start + min(N, 6))
            else:
                pairs += sum(min(c["sinks"], max(0, n + i + 1 - c["window"])) + min(c["window"], n + i + 1) for i in range(N))
        return {"bytes": keys * Hkv * (2 * D + 8 / c["page"]) + B * N * c["Hq"] * (4 * D + 4), "flops": 4 * pairs * c["Hq"] * D}
    if c["op"] == "select":
        n = c["B"] * c["K"] * c["V"]
        return {"bytes": n * (2 if c["dtype"] == "bf16" else 4) + c["B"] * (c["n"] * 12 + c["K"] * 8), "flops": 4 * n}
    if c["op"] == "fork":
        C, par = c["B"] * c["K"], _parents(c)
        lens = [n for n in _uneven(c, c["B"]) for _ in range(c["K"] if c["ends"] else 1)]
        rows, seen = 0, set()
        for p in par:
            rows += lens[p] % c["page"] if p in seen or not c["ends"] else 0
            seen.add(p)
        copied = rows * c["layers"] * c["Hkv"] * 2 * c["D"]
        return {"bytes": 2 * (copied + C * (2 * c["hidden"] + 4 * c["L"])) + 8 * sum(-(-lens[p] // c["page"]) for p in par), "flops": copied}
    if c["op"] == "roll":
        lens = _uneven(c, c["B"])
        gone = sum(max(0, (n - c["window"] + 1) // c["page"] - -(-c["sinks"] // c["page"])) for n in lens)
        new = sum(-(-(n + c["N"]) // c["page"]) - -(-n // c["page"]) for n in lens)
        return {"bytes": 4 * (4 * gone + 4 * new + 2 * c["B"]), "flops": gone + new}
    lens = _uneven(c, c["B"])
    moved = sum(-(-n // c["page"]) for n in lens[1::2])
    places = sum(-(-n // c["page"]) for n in lens)
    return {"bytes": 2 * moved * c["layers"] * c["Hkv"] * (2 * c["page"] * c["D"] + 8) + 12 * places, "flops": places}


def _pages(g, shape):
    """A pool of random finite e4m3 values, [layers, pages, heads, page, dims], with a scale for each page and head."""
    x = torch.empty(shape, dtype=torch.uint8, device=DEV)
    x.random_(0, 256, generator=g)
    x = torch.where((x & 127) >= 104, x & 0xB7, x)  # below 64, no NaN
    scale = torch.exp2(torch.randint(-6, -3, shape[:3], generator=g, device=DEV).float())
    return x.view(E4M3), scale


def _tree_masks(g, B, N):
    """Random candidate trees: ancestor-or-self bits [B, N, ceil(N / 32)] as int32 words."""
    u = torch.rand(B, N, generator=g, device=DEV).cpu()
    anc = torch.zeros(B, N, N, dtype=torch.bool)
    anc[:, 0, 0] = True
    rows = torch.arange(B)
    for i in range(1, N):
        lo = max(0, (i - 1) // 4)
        parent = (lo + (u[:, i] * (min(i, lo + 3) - lo)).long()).clamp(max=i - 1)
        anc[:, i] = anc[rows, parent]
        anc[:, i, i] = True
    W = -(-N // 32)
    bits = torch.zeros(B, N, W * 32, dtype=torch.int64)
    bits[:, :, :N] = anc.long()
    words = (bits.view(B, N, W, 32) << torch.arange(32)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32).to(DEV)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 31)
    s = dict(case=c)
    if c["op"] == "select":
        B, K, V = c["B"], c["K"], c["V"]
        # beams of one sequence continue much the same text: the same logits but for some noise, a few tokens likely
        base = torch.randn(B, 1, V, generator=g, device=DEV) * 2.0
        base += torch.where(torch.rand(B, 1, V, generator=g, device=DEV) < 30.0 / V, 9.0, 0.0)
        s["logits"] = (base + torch.randn(B, K, V, generator=g, device=DEV) * 0.7).to(TYPES[c["dtype"]])
        s["scores"] = -torch.rand(B, K, generator=g, device=DEV).cumsum(1) * 2.0
        s["done"] = (torch.rand(B, K, generator=g, device=DEV) < 0.15).to(torch.int32) if c["done"] else None
        return s
    page = c["page"]
    if c["op"] == "attend":
        B, N = c["B"], c["N"]
        lens = _uneven(c, B)
        span = -(-(c["L"] + N) // page)
        table = torch.randperm(B * span + 3, generator=g, device=DEV)[:B * span].view(B, span).to(torch.int32)
        s["lens"] = _ints(lens)
        # what lies behind the window of the next token has gone back to the pool
        place = torch.arange(span, device=DEV)
        start = (s["lens"] - c["window"] + 1).clamp(min=0)[:, None]
        s["table"] = torch.where((place * page < c["sinks"]) | ((place + 1) * page > start), table, -1)
        s["k"], s["k_scale"] = _pages(g, (1, B * span + 3, c["Hkv"], page, c["D"]))
        s["v"], s["v_scale"] = _pages(g, (1, B * span + 3, c["Hkv"], page, c["D"]))
        s["q"] = torch.randn(B, N, c["Hq"], c["D"], generator=g, device=DEV).to(TYPES[c["dtype"]])
        s["scale"] = 1.0 / math.sqrt(c["D"])
        s["mask"] = _tree_masks(g, B, N) if c["tree"] else None
        return s
    if c["op"] == "roll":
        B = c["B"]
        lens = _uneven(c, B)
        span = -(-(c["L"] + c["N"]) // page)
        pool = B * span + 7
        # decoding sequences take pages in turn: a random permutation; all of them held, none reserved
        table = torch.randperm(pool, generator=g, device=DEV)[:B * span].view(B, span).to(torch.int32)
        s["lens"] = _ints(lens)
        held = torch.arange(span, device=DEV) * page < s["lens"][:, None]
        s["table"] = torch.where(held, table, -1)
        s["refs"] = torch.zeros(pool, dtype=torch.int32, device=DEV)
        s["refs"][s["table"][held].long()] = 1
        s["k"], s["k_scale"] = _pages(g, (1, pool, 1, page, 64))
        s["v"], s["v_scale"] = _pages(g, (1, pool, 1, page, 64))
        return s
    B, layers = c["B"], c["layers"]
    heads, D = c["Hkv"], c["D"]
    if c["op"] == "fork":
        K = c["K"]
        lens = _uneven(c, B)
        par = _parents(c)
        seqs = B * K if c["ends"] else B
        own_lens = [n for n in lens for _ in range(seqs // B)]
        span = -(-c["L"] // page) + 1
        # the beams of a sequence share its full pages and have the last one, not full, for themselves
        pool = sum(n // page for n in lens) + seqs + B * K + 3
        order = torch.randperm(pool, generator=g, device=DEV).tolist()
        rows, at, refs = [], 0, [0] * pool
        for b, n in enumerate(lens):
            shared = order[at:at + n // page]
            at += n // page
            for _ in range(seqs // B):
                row = shared + (order[at:at + 1] if n % page else [])
                at += 1 if n % page else 0
                rows.append(row + [-1] * (span - len(row)))
                for p in row:
                    refs[p] += 1
        s["table"], s["lens"], s["refs"], s["parents"] = _ints(rows), _ints(own_lens), _ints(refs), _ints(par)
        s["next_table"] = torch.full((B * K, span), -1, dtype=torch.int32, device=DEV)
        s["next_lens"] = torch.zeros(B * K, dtype=torch.int32, device=DEV)
        s["tokens"] = torch.randint(0, 32000, (seqs, c["L"]), generator=g, device=DEV, dtype=torch.int32)
        s["hidden"] = torch.randn(seqs, c["hidden"], generator=g, device=DEV).to(torch.bfloat16)
    else:
        lens = _uneven(c, B)
        counts = [-(-n // page) for n in lens]
        span = max(counts)
        # every other sequence ends in the first pass, the others in the second, and so on: those that end hold the pool's front
        n_first = sum(counts[0::2])
        pool = sum(counts) + 5
        first = torch.randperm(n_first, generator=g, device=DEV).tolist()
        rest = (torch.randperm(sum(counts) - n_first, generator=g, device=DEV) + n_first).tolist()
        rows, refs = [], [0] * pool
        for b, n in enumerate(counts):
            take = first if b % 2 == 0 else rest
            row = [take.pop() for _ in range(n)]
            rows.append(row + [-1] * (span - n))
            for p in row:
                refs[p] = 1
        s["table"], s["lens"], s["refs"] = _ints(rows), _ints(lens), _ints(refs)
        even = _ints([1 - b % 2 for b in range(B)])
        s["ended"], s["turn"] = [even, 1 - even], 0
        s["fresh"] = [s["lens"] * e for e in s["ended"]]  # the new sequences' lengths
    s["k"], s["k_scale"] = _pages(g, (layers, pool, heads, page, D))
    s["v"], s["v_scale"] = _pages(g, (layers, pool, heads, page, D))
    return s


# ------------------------------------------------------------------------------------------------ the calls of a user

def _call(s):
    import speculative_decoding_verification_78_gb300 as sv

    c = s["case"]
    if "status" not in s:  # what a program keeps between calls: the cache, workspaces and a status word
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        if c["op"] == "select":
            s["ws"] = sv.new_beam_workspace(c["B"], c["K"], c["V"], s["logits"].dtype)
        else:
            s["cache"] = sv.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
            if c["op"] == "attend":
                s["ws"] = sv.new_attention_workspace(c["B"], c["N"], c["Hq"], c["Hkv"], c["D"])
            else:
                s["ws"] = sv.new_pages_workspace(s["cache"], s["table"].shape[0] if c["op"] != "fork" else c["B"] * c["K"])
    st = s["status"]
    if c["op"] == "select":
        tokens, parents, scores, _ = sv.beam_select(s["logits"], s["scores"], c["n"], done=s["done"], pad_token=2, workspace=s["ws"], status=st)
        return {"tokens": tokens, "parents": parents, "scores": scores}
    if c["op"] == "attend":
        out, lse, _ = sv.kv_attention(s["cache"], s["table"], s["lens"], s["q"], scale=s["scale"], mask=s["mask"], window=c["window"], sinks=c["sinks"],
                                      workspace=s["ws"], status=st, return_lse=True)
        return {"out": out, "lse": lse}
    kv = {"k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if c["op"] == "roll":
        sv.kv_trim(s["cache"], s["refs"], s["table"], s["lens"], window=c["window"], sinks=c["sinks"], status=st)
        granted, _ = sv.kv_reserve(s["cache"], s["refs"], s["table"], s["lens"], c["N"], workspace=s["ws"], status=st)
        return {"granted": granted, "table": s["table"], "refs": s["refs"]}
    if c["op"] == "fork":
        if not c["ends"]:  # the samples of the pass before have ended
            sv.kv_free(s["cache"], s["refs"], s["next_table"], s["next_lens"], status=st)
        sv.kv_fork(s["cache"], s["refs"], s["table"], s["lens"], s["parents"], release=c["ends"], page_table_out=s["next_table"], lens_out=s["next_lens"],
                   workspace=s["ws"], status=st)
        tokens, hidden, _ = sv.beam_reorder([s["tokens"], s["hidden"]], s["parents"], status=st)
        table, lens = s["next_table"], s["next_lens"]
        if c["ends"]:
            s["table"], s["next_table"], s["lens"], s["next_lens"] = table, s["table"], lens, s["lens"]
        return {"table": table, "lens": lens, "refs": s["refs"], "tokens": tokens, "hidden": hidden, **kv}
    turn = s["turn"]
    s["turn"] = 1 - turn
    sv.kv_free(s["cache"], s["refs"], s["table"], s["lens"], ended=s["ended"][turn], status=st)
    page_map, live, _ = sv.kv_compact(s["cache"], s["refs"], s["table"], workspace=s["ws"], status=st)
    granted, _ = sv.kv_reserve(s["cache"], s["refs"], s["table"], s["lens"], c["L"], new_lens=s["fresh"][turn], workspace=s["ws"], status=st)
    s["lens"] += granted
    return {"table": s["table"], "lens": s["lens"], "refs": s["refs"], "map": page_map, "live": live, **kv}


# ------------------------------------------------------------------------------------------------ the plain forms

def _bits(mask, n):
    """Mask words [..., W] -> truth values [..., n]."""
    return (((mask[..., None] >> torch.arange(32, device=mask.device, dtype=torch.int32)) & 1) != 0).flatten(-2)[..., :n]


def _attend(s):
    c = s["case"]
    B, N, Hq, Hkv, D, page, window = c["B"], c["N"], c["Hq"], c["Hkv"], c["D"], c["page"], c["window"]
    G = Hq // Hkv
    lens = s["lens"].long()[:, None]
    start = (lens - window + 1).clamp(min=0)  # the first slot in the first new token's window
    early = torch.arange(min(c["sinks"], c["L"] + N), device=DEV).expand(B, -1)
    late = start + torch.arange(min(window - 1, c["L"]) + N, device=DEV)
    slot = torch.cat([early, late], 1)  # [B, T]
    there = torch.cat([early < start, late < lens + N], 1)
    page_of = s["table"].long().gather(1, (slot // page).clamp(max=s["table"].shape[1] - 1)).clamp(min=0)

    def rows(pool, scales):  # [B, Hkv, T, D] in 32 bits
        x = pool.view(torch.uint8)[page_of, :, slot % page].view(E4M3).float() * scales[page_of][..., None]
        return x.transpose(1, 2)

    rel = (slot - lens)[:, None]  # [B, 1, T]
    node = torch.arange(N, device=DEV)[:, None]
    if s["mask"] is None:
        seen = rel <= node
        depth = node
    else:
        bits = _bits(s["mask"], N)
        seen = (rel < 0) | bits.gather(2, rel.clamp(0, N - 1).expand(B, N, -1))
        depth = bits.sum(-1, keepdim=True) - 1
    seen = seen & there[:, None] & ((slot[:, None] < c["sinks"]) | (rel > depth - window) | ((rel >= 0) if s["mask"] is not None else False))
    seen = seen[:, None, :, None, :]  # [B, 1, N, 1, T]
    q = s["q"].float().view(B, N, Hkv, G, D).transpose(1, 2)
    x = (q.reshape(B, Hkv, N * G, D) @ rows(s["k"][0], s["k_scale"][0]).transpose(-1, -2)).view(B, Hkv, N, G, -1) * s["scale"]
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = (x - m.clamp(min=-3e38)).exp()
    total = p.sum(-1, keepdim=True)
    out = (p.view(B, Hkv, N * G, -1) @ rows(s["v"][0], s["v_scale"][0])).view(B, Hkv, N, G, D) / total.clamp(min=1e-38)
    lse = (m + total.log())[..., 0]
    return {"out": out.transpose(1, 2).reshape(B, N, Hq, D).to(s["q"].dtype), "lse": lse.transpose(1, 2).reshape(B, N, Hq)}


def _select(s):
    c = s["case"]
    B, K, V, n = c["B"], c["K"], c["V"], c["n"]
    x = s["logits"].double()  # two beams' candidates may lie closer than 32 bits tell apart
    top = x.amax(-1, keepdim=True)
    total = (x - top).exp().sum(-1, keepdim=True).log() + top
    score = s["scores"].double()[..., None] + (x - total)
    if s["done"] is not None:  # a beam at its end goes on as it is
        stays = torch.full_like(score, -math.inf)
        stays[..., 2] = s["scores"].double()
        score = torch.where((s["done"] != 0)[..., None], stays, score)
    flat = score.view(B, K * V)
    least = flat.topk(n).values[:, -1:]
    more = flat > least
    ties = flat == least
    chosen = more | (ties & (ties.cumsum(1) <= n - more.sum(1, keepdim=True)))
    idx = chosen.nonzero()[:, 1].view(B, n)  # by increasing index
    best, order = flat.gather(1, idx).sort(dim=1, descending=True, stable=True)
    idx = idx.gather(1, order)
    return {"tokens": (idx % V).int(), "parents": (idx // V + torch.arange(B, device=DEV)[:, None] * K).int(), "scores": best.float()}


def _add(refs, pages, by):
    """refs[p] += by for every p in `pages` that is a page."""
    refs.index_add_(0, pages.clamp(min=0).long().flatten(), (by * (pages >= 0)).to(torch.int32).flatten())


def _take(refs, wanted):
    """The lowest free pages for the places that want one, in their order: page numbers where wanted."""
    free = refs == 0
    numbers = torch.arange(refs.numel(), device=DEV)
    lowest = torch.zeros_like(numbers).scatter_(0, torch.where(free, free.cumsum(0) - 1, free.sum() + (~free).cumsum(0) - 1), numbers)
    pages = lowest[(wanted.flatten().cumsum(0) - 1).clamp(min=0)].view(wanted.shape)
    _add(refs, torch.where(wanted, pages, -1), 1)
    return pages.int()


def _free(s, table, lens, ended):
    goes = ended[:, None] != 0
    _add(s["refs"], torch.where(goes, table, -1), -1)
    table.copy_(torch.where(goes, -1, table))
    lens.copy_(torch.where(ended != 0, 0, lens))


def _reserve(s, table, lens, n):
    page = s["case"]["page"]
    place = torch.arange(table.shape[1], device=DEV)
    wants = (table < 0) & (place >= (lens // page)[:, None]) & (place * page < (lens + n)[:, None]) & (n > 0)[:, None]
    table.copy_(torch.where(wants, _take(s["refs"], wants), table))
    return n


def _roll(s):
    c = s["case"]
    page, table, lens = c["page"], s["table"], s["lens"]
    place = torch.arange(table.shape[1], device=DEV)
    behind = (place * page >= c["sinks"]) & ((place + 1) * page <= (lens - c["window"] + 1)[:, None])
    goes = behind | (place * page >= lens[:, None])
    _add(s["refs"], torch.where(goes, table, -1), -1)
    table.copy_(torch.where(goes, -1, table))
    granted = _reserve(s, table, lens, torch.full_like(lens, c["N"]))
    return {"granted": granted, "table": table, "refs": s["refs"]}


def _fork(s):
    c = s["case"]
    page, refs, par, lens = c["page"], s["refs"], s["parents"].long(), s["lens"]
    if not c["ends"]:
        _free(s, s["next_table"], s["next_lens"], torch.ones_like(s["next_lens"]))
    C = par.numel()
    child = torch.arange(C, device=DEV)
    row, n = s["table"][par], lens[par]
    place = torch.arange(row.shape[1], device=DEV)
    full, rest = (n // page)[:, None], n % page
    first = torch.full((lens.numel(),), C, device=DEV).scatter_reduce_(0, par, child, "amin")
    keeps = (first[par] == child) & c["ends"]
    takes = (place < full) | ((place == full) & (rest > 0)[:, None] & keeps[:, None])
    out = torch.where(takes, row, -1)
    _add(refs, out, 1)
    if c["ends"]:
        _add(refs, s["table"], -1)
    copies = (rest > 0) & ~keeps
    new = _take(refs, copies)
    out = torch.where((place == full) & copies[:, None], new[:, None], out)
    src = row.gather(1, full.long().clamp(max=row.shape[1] - 1))[:, 0]
    which = copies.nonzero()[:, 0]
    src, dst = src[which].long(), new[which].long()
    rows = (torch.arange(page, device=DEV) < rest[which][:, None])[None, :, None, :, None]
    for pool, scales in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
        raw = pool.view(torch.uint8)
        raw[:, dst] = torch.where(rows, raw[:, src], raw[:, dst])
        scales[:, dst] = scales[:, src]
    s["next_table"].copy_(out)
    s["next_lens"].copy_(n)
    table, next_lens = s["next_table"], s["next_lens"]
    if c["ends"]:
        s["table"], s["next_table"], s["lens"], s["next_lens"] = table, s["table"], next_lens, s["lens"]
    return {"table": table, "lens": next_lens, "refs": refs, "tokens": s["tokens"][par], "hidden": s["hidden"][par],
            "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _compact(s):
    turn, table, refs = s["turn"], s["table"], s["refs"]
    s["turn"] = 1 - turn
    _free(s, table, s["lens"], s["ended"][turn])
    held = refs > 0
    live = held.sum(dtype=torch.int32).view(1)
    numbers = torch.arange(refs.numel(), device=DEV)
    hole, mover = ~held & (numbers < live), held & (numbers >= live)
    src, dst = mover.nonzero()[:, 0], hole.nonzero()[:, 0]
    page_map = torch.where(held, numbers, -1).int()
    page_map[src] = dst.int()
    for x in (s["k"].view(torch.uint8), s["v"].view(torch.uint8), s["k_scale"], s["v_scale"]):
        x[:, dst] = x[:, src]
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, page_map[table.clamp(min=0).long()], -1))
    s["lens"] += _reserve(s, table, s["lens"], s["fresh"][turn])
    return {"table": table, "lens": s["lens"], "refs": refs, "map": page_map, "live": live,
            "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def run(state):
    if own:
        return _call(state)
    return {"attend": _attend, "select": _select, "fork": _fork, "roll": _roll, "compact": _compact}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    c = case
    if c["op"] not in ("attend", "select"):
        return None  # pages, tables and counts are moved, not computed
    s = prepare(case, seed)
    if c["op"] == "select":
        tokens, parents, scores = [], [], []
        for b in range(c["B"]):
            logp = torch.log_softmax(s["logits"][b].double(), -1) + s["scores"][b].double()[:, None]
            if s["done"] is not None:
                ends = s["done"][b] != 0
                logp[ends] = -math.inf
                logp[ends, 2] = s["scores"][b][ends].double()
            best, idx = logp.flatten().sort(descending=True, stable=True)
            tokens.append(idx[:c["n"]] % c["V"])
            parents.append(b * c["K"] + idx[:c["n"]] // c["V"])
            scores.append(best[:c["n"]])
        return {"tokens": torch.stack(tokens).int(), "parents": torch.stack(parents).int(), "scores": torch.stack(scores)}
    B, N, Hkv, page, window, sinks = c["B"], c["N"], c["Hkv"], c["page"], c["window"], c["sinks"]
    G = c["Hq"] // Hkv
    mask = None
    if s["mask"] is not None:
        words = s["mask"].cpu().tolist()
        mask = torch.tensor([[[(w[j // 32] >> (j % 32)) & 1 for j in range(N)] for w in rows] for rows in words], dtype=torch.bool, device=DEV)
    outs, lses = [], []
    for b, n in enumerate(_uneven(c, B)):
        slots = torch.tensor([t for t in range(n + N) if t < sinks or t > n - window], device=DEV)
        at = s["table"][b].long()[slots // page]
        k, v = ((x[0].view(torch.uint8)[at, :, slots % page].view(E4M3).double() * f[0][at].double()[..., None]).transpose(0, 1)
                for x, f in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])))
        if mask is None:
            pos = n + torch.arange(N, device=DEV)[:, None]
            see = (slots <= pos) & ((slots < sinks) | (slots > pos - window))
        else:
            pos = n + mask[b].sum(1, keepdim=True) - 1
            old = slots < n
            see = (old & ((slots < sinks) | (slots > pos - window))) | (~old & mask[b][:, (slots - n).clamp(min=0)])
        o, l = [], []
        for h in range(c["Hq"]):
            z = (s["q"][b, :, h].double() @ k[h // G].T * s["scale"]).masked_fill(~see, -math.inf)
            l.append(torch.logsumexp(z, -1))
            o.append(torch.exp(z - l[-1][:, None]) @ v[h // G])
        outs.append(torch.stack(o, 1))
        lses.append(torch.stack(l, 1))
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
