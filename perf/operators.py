"""The KV-cache operators of a verification step, as cases to measure.

kv_append     rotates the new tokens' queries and keys and writes keys and values into a paged cache held in
              8 bits (e4m3) with one power-of-two scale for each page and head
kv_attention  attention of the new tokens (a chain, a candidate tree, one token, a piece of a prompt) over that cache
kv_commit     keeps the accepted path of a verified tree: its rows move to the front of the new tokens' slots

`run` computes each in plain torch operations, or with the library's calls where `own` is true.
"""
import math

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # a single sequence decoding token by token: the smallest call, where latency counts
        dict(name="append_one", op="append", dtype="bf16", B=1, N=1, Hq=32, Hkv=8, D=128, page=64, L=1000, rope=128, pairs=False, tree=False),
        # the drafts of a chain-verification batch, rotated by interleaved pairs over part of the head
        dict(name="append_chain", op="append", dtype="fp16", B=64, N=6, Hq=16, Hkv=2, D=64, page=16, L=700, rope=32, pairs=True, tree=False),
        # the nodes of 32 candidate trees of 64 nodes, positions by depth
        dict(name="append_tree", op="append", dtype="bf16", B=32, N=64, Hq=32, Hkv=8, D=128, page=64, L=2000, rope=128, pairs=False, tree=True),
        # a batch of prompts, a few thousand tokens each
        dict(name="append_prompt", op="append", dtype="bf16", B=8, N=4096, Hq=32, Hkv=8, D=128, page=64, L=500, rope=128, pairs=False, tree=False),
        # one token of one sequence: the smallest call
        dict(name="attend_one", op="attend", dtype="bf16", B=1, N=1, Hq=32, Hkv=8, D=128, page=64, L=1000, tree=False),
        # one token for each sequence of a serving batch, long contexts of uneven lengths
        dict(name="attend_decode", op="attend", dtype="bf16", B=64, N=1, Hq=32, Hkv=8, D=128, page=64, L=16000, tree=False),
        # chain verification, gamma = 5, 64 steps, small pages and heads
        dict(name="attend_chain", op="attend", dtype="fp16", B=64, N=6, Hq=16, Hkv=2, D=64, page=16, L=5003, tree=False),
        # a candidate tree of 64 nodes with as many key heads as query heads
        dict(name="attend_tree", op="attend", dtype="bf16", B=32, N=64, Hq=32, Hkv=32, D=128, page=32, L=2000, tree=True),
        # the same tree with four query heads to a key head, over long contexts
        dict(name="attend_tree_long", op="attend", dtype="bf16", B=32, N=64, Hq=32, Hkv=8, D=128, page=64, L=8192, tree=True),
        # a piece of a prompt against what is already cached
        dict(name="attend_prompt", op="attend", dtype="bf16", B=2, N=1500, Hq=32, Hkv=8, D=128, page=128, L=4099, tree=False),
        # the accepted paths of one tree in one layer, and of 32 trees in all of 32 layers
        dict(name="commit_one", op="commit", dtype="bf16", B=1, N=64, Hkv=8, D=128, page=64, L=1000, layers=1),
        dict(name="commit_layers", op="commit", dtype="bf16", B=32, N=64, Hkv=8, D=128, page=64, L=1000, layers=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "commit"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16"]), Hkv=Hkv, D=D, page=rng.choice([16, 32, 64, 128]))
    tree = rng.random() < 0.4
    if op == "commit":
        return c | dict(B=_log(rng, 1, 32), N=rng.randint(13, 64), L=_log(rng, 1, 1200), layers=_log(rng, 1, 32))
    G = rng.choice([1, 2, 4, 8])
    c |= dict(Hq=Hkv * G, tree=tree)
    if op == "append":
        B = _log(rng, 1, 64)
        N = rng.randint(2, 96) if tree else _log(rng, 1, 32768 // B)
        return c | dict(B=B, N=N, L=_log(rng, 1, 2000), rope=rng.choice([D, D // 2]), pairs=rng.random() < 0.3)
    B = _log(rng, 1, 64)
    N = rng.randint(2, 96) if tree else _log(rng, 1, 600)
    # keys of the batch, and products, no more than the largest listed case has
    most = min(7_500_000 // (B * Hkv), int(5e8 / (B * N * Hkv * G)), 20000)
    return c | dict(B=B, N=N, L=_log(rng, 1, max(2, most)))


def _lens(c):
    """Cached tokens of each sequence: uneven, between half of L and L, the first one L."""
    return [c["L"] - (b * 37) % (c["L"] // 2 + 1) for b in range(c["B"])]


def _span(c):
    """Pages of a sequence's table."""
    return -(-(c["L"] + c["N"]) // c["page"])


def work(case):
    c = case
    B, N, Hkv, D = c["B"], c["N"], c["Hkv"], c["D"]
    lens = _lens(c)
    if c["op"] == "append":
        row = D * (c["Hq"] + 2 * Hkv)
        table = 4 * c["rope"] * (max(lens) - min(lens) + min(N, 64) if c["tree"] else N + max(lens) - min(lens))
        return {"bytes": B * N * (2 * row + 2 * D * c["Hq"] + 2 * D * Hkv) + min(table, 4 * c["rope"] * B * N),
                "flops": 3 * B * N * c["rope"] * (c["Hq"] + Hkv)}
    if c["op"] == "attend":
        keys = sum(lens) + B * N
        pairs = sum(N * n for n in lens) + (B * N * min(N, 6) if c["tree"] else B * N * (N + 1) // 2)
        return {"bytes": keys * Hkv * (2 * D + 8 / c["page"]) + B * N * c["Hq"] * (4 * D + 4), "flops": 4 * pairs * c["Hq"] * D}
    moved = c["layers"] * sum(_accepted(c)) * 2 * Hkv * D
    return {"bytes": 2 * moved, "flops": moved}


def _accepted(c):
    """Accepted nodes below the root, 0 to 6 a tree."""
    return [(b * 5 + 3) % 7 for b in range(c["B"])]


def _e4m3_pages(g, shape, spread):
    """Pages of random values with a power-of-two scale for each page and head: (bytes as e4m3, scales)."""
    out = torch.empty(shape, dtype=E4M3, device=DEV)
    scale = torch.empty(shape[:-2], dtype=torch.float32, device=DEV)
    flat, fs = out.view(-1, *shape[-3:]), scale.view(-1, shape[-3])
    step = max(1, (1 << 26) // (shape[-3] * shape[-2] * shape[-1]))
    for i in range(0, flat.shape[0], step):
        x = torch.randn(flat[i:i + step].shape, generator=g, device=DEV) * spread
        s = _scale_of(x.abs().amax((-2, -1)))
        flat[i:i + step] = (x / s[..., None, None]).to(E4M3)
        fs[i:i + step] = s
    return out, scale


def _scale_of(amax):
    """The smallest power of two s with amax <= 448 s, at least 2^-64."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1)
    e = e - 9 + (m > 0.875)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e.clamp(-64, 127)), torch.full_like(amax, 2.0 ** -64))


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


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 13)
    B, N, Hkv, D, page = c["B"], c["N"], c["Hkv"], c["D"], c["page"]
    T = TYPES[c["dtype"]]
    span = _span(c)
    pages = B * span + 3
    s = dict(case=c, lens=torch.tensor(_lens(c), dtype=torch.int32, device=DEV))
    s["table"] = torch.randperm(pages, generator=g, device=DEV)[:B * span].view(B, span).to(torch.int32)
    layers = c.get("layers", 1)
    s["k"], s["k_scale"] = _e4m3_pages(g, (layers, pages, Hkv, page, D), 1.5)
    s["v"], s["v_scale"] = _e4m3_pages(g, (layers, pages, Hkv, page, D), 1.0)
    if c["op"] == "commit":
        acc = torch.tensor(_accepted(c), dtype=torch.int32, device=DEV)
        # root, then increasing node numbers past the longest path, as in a breadth-first tree that is wider than deep
        path = torch.rand(B, N - 7, generator=g, device=DEV).argsort(1)[:, :6].sort(1).values + 7
        path = torch.nn.functional.pad(path, (1, N - 7), value=0)
        s["path"] = torch.where(torch.arange(N, device=DEV)[None] <= acc[:, None], path, -1).to(torch.int32)
        s["acc"] = acc
        return s
    s["mask"] = _tree_masks(g, B, N) if c["tree"] else None
    if c["op"] == "append":
        # one projection's output, queries, keys and values side by side, as a layer hands them on
        qkv = torch.randn(B, N, c["Hq"] + 2 * Hkv, D, generator=g, device=DEV).to(T)
        s["q"], s["new_k"], s["new_v"] = qkv.split([c["Hq"], Hkv, Hkv], 2)
        R = c["rope"]
        inv = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device=DEV) / R)
        angle = torch.arange(c["L"] + N + 1, dtype=torch.float64, device=DEV)[:, None] * inv
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    else:
        s["q"] = torch.randn(B, N, c["Hq"], D, generator=g, device=DEV).to(T)
        s["scale"] = 1.0 / math.sqrt(D)
    return s


# ------------------------------------------------------------------------------------------------ the calls of a user

def _call(s):
    import speculative_decoding_verification_78_gb300 as sv

    c = s["case"]
    if "cache" not in s:  # what a program keeps between calls: the cache, a workspace and a status word
        s["cache"] = sv.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        if c["op"] == "attend":
            s["ws"] = sv.new_attention_workspace(c["B"], c["N"], c["Hq"], c["Hkv"], c["D"])
    cache = s["cache"]
    if c["op"] == "append":
        q, _ = sv.kv_append(cache, s["table"], s["lens"], s["new_k"], s["new_v"], q=s["q"], rope=s["rope"], interleaved=c["pairs"],
                            mask=s["mask"], status=s["status"])
        return {"q": q, "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if c["op"] == "attend":
        out, lse, _ = sv.kv_attention(cache, s["table"], s["lens"], s["q"], scale=s["scale"], mask=s["mask"], workspace=s["ws"],
                                      status=s["status"], return_lse=True)
        return {"out": out, "lse": lse}
    lens, _ = sv.kv_commit(cache, s["table"], s["lens"], s["path"], s["acc"], status=s["status"])
    return {"lens": lens, "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


# ------------------------------------------------------------------------------------------------ the plain forms

def _bits(mask, n):
    """Mask words [..., W] -> truth values [..., n]."""
    return (((mask[..., None] >> torch.arange(32, device=mask.device, dtype=torch.int32)) & 1) != 0).flatten(-2)[..., :n]


def _rotate(x, cos, sin, R, pairs):
    """x [B, N, H, D] in 32 bits; cos, sin [B, N, 1, R / 2]."""
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if pairs else (x[..., :R // 2], x[..., R // 2:R])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if pairs else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _append(s):
    c = s["case"]
    B, N, Hkv, D, page, R = c["B"], c["N"], c["Hkv"], c["D"], c["page"], c["rope"]
    lens = s["lens"].long()
    node = torch.arange(N, device=DEV)
    slot = lens[:, None] + node
    pos = slot if s["mask"] is None else lens[:, None] + _bits(s["mask"], N).sum(-1) - 1
    cos, sin = s["rope"][pos][:, :, None].split(R // 2, -1)
    q = _rotate(s["q"].float(), cos, sin, R, c["pairs"]).to(s["q"].dtype)
    k = _rotate(s["new_k"].float(), cos, sin, R, c["pairs"])
    v = s["new_v"].float()
    first = lens // page
    local = slot // page - first[:, None]  # [B, N], the page of each token among those touched
    P = (N + page - 2) // page + 1
    where = s["table"].long().gather(1, (first[:, None] + torch.arange(P, device=DEV)).clamp(max=s["table"].shape[1] - 1))  # [B, P]
    touched = torch.arange(P, device=DEV) <= local[:, -1:]  # [B, P]
    kept = lens % page  # rows of the first page that were there
    for x, pool, scales in ((k, s["k"][0], s["k_scale"][0]), (v, s["v"][0], s["v_scale"][0])):
        amax = torch.zeros(B, P, Hkv, device=DEV).scatter_reduce_(1, local[:, :, None].expand(B, N, Hkv), x.abs().amax(-1), "amax")
        new = _scale_of(amax)  # [B, P, Hkv]
        old = scales[where[:, 0]]  # [B, Hkv]
        new[:, 0] = torch.where((kept > 0)[:, None], torch.maximum(new[:, 0], old), new[:, 0])
        raw = pool.view(torch.uint8)
        head = raw[where[:, 0]]  # [B, Hkv, page, D]
        again = (head.view(E4M3).float() * (old / new[:, 0])[..., None, None]).to(E4M3).view(torch.uint8)
        raw[where[:, 0]] = torch.where((torch.arange(page, device=DEV) < kept[:, None])[:, None, :, None], again, head)
        by_token = new.gather(1, local[:, :, None].expand(B, N, Hkv))
        raw[where.gather(1, local), :, slot % page] = (x / by_token[..., None]).to(E4M3).view(torch.uint8)
        scales[where[touched]] = new[touched]
    return {"q": q, "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _attend(s):
    c = s["case"]
    B, N, Hq, Hkv, D, page = c["B"], c["N"], c["Hq"], c["Hkv"], c["D"], c["page"]
    G = Hq // Hkv
    table = s["table"].long()
    L = table.shape[1] * page

    def pages(pool, scales):  # [B, Hkv, L, D] in 32 bits; tokens past a sequence's end may hold anything
        x = pool.view(torch.uint8)[table].view(E4M3).float() * scales[table][..., None, None]
        return x.transpose(1, 2).reshape(B, Hkv, L, D)

    slot = torch.arange(L, device=DEV)
    lens = s["lens"].long()[:, None, None]
    rel = slot - lens  # [B, 1, L]
    node = torch.arange(N, device=DEV)[:, None]
    if s["mask"] is None:
        seen = rel <= node
    else:
        bits = _bits(s["mask"], N)  # [B, N, N]
        seen = (rel < 0) | ((rel >= 0) & (rel < N) & bits.gather(2, rel.clamp(0, N - 1).expand(B, N, L)))
    seen = seen[:, None, :, None, :]  # [B, 1, N, 1, L]
    q = s["q"].float().view(B, N, Hkv, G, D).transpose(1, 2)  # [B, Hkv, N, G, D]
    x = (q.reshape(B, Hkv, N * G, D) @ pages(s["k"][0], s["k_scale"][0]).transpose(-1, -2)).view(B, Hkv, N, G, L) * s["scale"]
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = (x - m.clamp(min=-3e38)).exp()
    total = p.sum(-1, keepdim=True)
    out = (p.view(B, Hkv, N * G, L) @ pages(s["v"][0], s["v_scale"][0])).view(B, Hkv, N, G, D) / total.clamp(min=1e-38)
    lse = (m + total.log())[..., 0]
    return {"out": out.transpose(1, 2).reshape(B, N, Hq, D).to(s["q"].dtype), "lse": lse.transpose(1, 2).reshape(B, N, Hq)}


def _commit(s):
    c = s["case"]
    B, N, Hkv, D, page, layers = c["B"], c["N"], c["Hkv"], c["D"], c["page"], c["layers"]
    lens, acc = s["lens"].long(), s["acc"].long()
    K = min(N, 7)
    k = torch.arange(K, device=DEV)
    path = s["path"].long()[:, :K].clamp(min=0)
    to = lens[:, None] + k
    frm = torch.where(k <= acc[:, None], lens[:, None] + path, to)  # what is not accepted stays
    moves = frm != to  # [B, K]
    first = lens // page
    P = (K + page - 2) // page + 1
    idx = (first[:, None] + torch.arange(P, device=DEV)).clamp(max=s["table"].shape[1] - 1)
    where = s["table"].long().gather(1, idx)  # [B, P]
    local = to // page - first[:, None]
    table = s["table"].long()
    src = table.gather(1, frm // page)  # [B, K]
    dst = table.gather(1, to // page)
    for pool, scales in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
        raw = pool.view(torch.uint8)
        x = raw[:, src, :, frm % page].view(E4M3).float()  # [B, K, layers, Hkv, D]: indices apart from each other come first
        x = x * scales[:, src].permute(1, 2, 0, 3)[..., None]
        need = torch.where(moves[..., None, None], _scale_of(x.abs().amax(-1)), torch.zeros((), device=DEV))  # [B, K, layers, Hkv]
        new = torch.zeros(B, P, layers, Hkv, device=DEV).scatter_reduce_(1, local[:, :, None, None].expand_as(need), need, "amax")
        old = scales[:, where].permute(1, 2, 0, 3)  # [B, P, layers, Hkv]
        new = torch.maximum(new, old)
        there = (torch.arange(P, device=DEV) <= local[:, -1:])  # pages that hold a place of the path
        # the rows of those pages at their new scale, then the moved rows
        held = raw[:, where[there]].view(E4M3).float()  # [layers, n, Hkv, page, D]
        ratio = (old / new)[there].permute(1, 0, 2)  # [layers, n, Hkv]
        raw[:, where[there]] = (held * ratio[..., None, None]).to(E4M3).view(torch.uint8)
        by_row = new.gather(1, local[:, :, None, None].expand_as(need))
        y = (x / by_row[..., None]).to(E4M3).view(torch.uint8)
        row = to % page
        raw[:, dst[moves], :, row[moves]] = y[moves]
        scales[:, where[there]] = new[there].permute(1, 0, 2)
    return {"lens": (lens + acc + 1).to(torch.int32), "k": s["k"], "v": s["v"], "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def run(state):
    if own:
        return _call(state)
    return {"append": _append, "attend": _attend, "commit": _commit}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------ in 64 bits

def _pow2(a):
    """The scale of a page by its largest magnitude a (a Python number)."""
    return max(2.0 ** -64, 2.0 ** math.ceil(math.log2(a / 448.0))) if a > 0 else 2.0 ** -64


_GRID = sorted({m * 2.0 ** e / 8 for e in range(-6, 9) for m in range(8, 16)} - {480.0} | {m * 2.0 ** -9 for m in range(8)})


def _near(x):
    """The e4m3 value nearest to each x, ties to the even code."""
    grid = torch.tensor(_GRID, dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    lo = torch.bucketize(x.abs(), mid)  # ties: mid[i - 1] < |x| <= mid[i] -> i
    tie = (lo < len(mid)) & (x.abs() == mid[lo.clamp(max=len(mid) - 1)]) & (lo % 2 == 1)
    return torch.where(x < 0, -1.0, 1.0) * grid[lo + tie]


def exact(case, seed):
    c = case
    if c["op"] == "attend" and work(c)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    B, N, Hkv, D, page = c["B"], c["N"], c["Hkv"], c["D"], c["page"]
    lens, table = _lens(c), s["table"].tolist()
    mask = None
    if s.get("mask") is not None:
        words = s["mask"].cpu().tolist()
        mask = torch.tensor([[[(w[j // 32] >> (j % 32)) & 1 for j in range(N)] for w in rows] for rows in words], dtype=torch.bool, device=DEV)
    if c["op"] == "attend":
        G = c["Hq"] // Hkv
        outs, lses = [], []
        for b in range(B):
            n = lens[b] + N
            t = torch.tensor(table[b], device=DEV)
            val = [(x[0].view(torch.uint8)[t].view(E4M3).double() * f[0][t].double()[..., None, None]).transpose(0, 1).reshape(Hkv, -1, D)[:, :n]
                   for x, f in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"]))]
            new = torch.ones(N, N, dtype=torch.bool, device=DEV).tril() if mask is None else mask[b]
            see = torch.cat([torch.ones(N, lens[b], dtype=torch.bool, device=DEV), new], 1)
            q = s["q"][b].double()
            o, l = [], []
            for h in range(c["Hq"]):
                z = (q[:, h] @ val[0][h // G].T * s["scale"]).masked_fill(~see, -math.inf)
                l.append(torch.logsumexp(z, -1))
                o.append(torch.exp(z - l[-1][:, None]) @ val[1][h // G])
            outs.append(torch.stack(o, 1))
            lses.append(torch.stack(l, 1))
        return {"out": torch.stack(outs), "lse": torch.stack(lses)}
    vals = {}
    for name in ("k", "v"):
        vals[name] = s[name].double()
        vals[name + "_scale"] = s[name + "_scale"].double()
    if c["op"] == "append":
        R, half = c["rope"], c["rope"] // 2
        first, second = (list(range(0, R, 2)), list(range(1, R, 2))) if c["pairs"] else (list(range(half)), list(range(half, R)))
        depth = torch.arange(N, device=DEV).expand(B, N) if mask is None else mask.sum(-1) - 1
        pos = torch.tensor(lens, device=DEV)[:, None] + depth
        cos, sin = s["rope"].double()[pos][:, :, None, :half], s["rope"].double()[pos][:, :, None, half:]

        def turn(x):
            y = x.double()
            z = y.clone()
            z[..., first] = y[..., first] * cos - y[..., second] * sin
            z[..., second] = y[..., second] * cos + y[..., first] * sin
            return z

        if B * N * Hkv > 400_000:  # the loop over pages below would take too long
            return {"q": turn(s["q"]), "k": None, "v": None, "k_scale": None, "v_scale": None}
        for name, x in (("k", turn(s["new_k"])), ("v", s["new_v"].double())):
            for b in range(B):
                at = lens[b]
                while at < lens[b] + N:
                    end = min((at // page + 1) * page, lens[b] + N)
                    pg, r = table[b][at // page], at % page
                    rows = x[b, at - lens[b]:end - lens[b]].transpose(0, 1)  # [Hkv, n, D]
                    amax = rows.abs().amax((1, 2)).tolist()
                    for h in range(Hkv):
                        new = _pow2(amax[h])
                        if r > 0:
                            was = float(vals[name + "_scale"][0, pg, h])
                            new = max(new, was)
                            if new != was:
                                vals[name][0, pg, h, :r] = _near(vals[name][0, pg, h, :r] * was / new)
                        vals[name][0, pg, h, r:r + end - at] = _near(rows[h] / new)
                        vals[name + "_scale"][0, pg, h] = new
                    at = end
        return {"q": turn(s["q"]), **vals}
    acc = s["acc"].tolist()
    path = s["path"].tolist()
    for name in ("k", "v"):
        x, f = vals[name], vals[name + "_scale"]
        for b in range(B):
            rows = []
            for k in range(acc[b] + 1):
                if path[b][k] != k:
                    at = lens[b] + path[b][k]
                    rows.append((lens[b] + k, x[:, table[b][at // page], :, at % page] * f[:, table[b][at // page], :, None]))
            for pi in sorted({at // page for at, _ in rows}):
                pg = table[b][pi]
                mine = [(at % page, y) for at, y in rows if at // page == pi]
                amax = torch.stack([y for _, y in mine]).abs().amax((0, -1)).clamp(min=2.0 ** -60)  # [layers, Hkv]
                was = f[:, pg].clone()
                m, e = torch.frexp(amax / 448.0)  # an exact logarithm: the largest value is often 448 times a power of two
                new = torch.maximum(was, torch.ldexp(torch.ones_like(amax), e - (m == 0.5).to(e.dtype)))
                if bool((new != was).any()):
                    x[:, pg] = _near(x[:, pg] * (was / new)[..., None, None])
                for r, y in mine:
                    x[:, pg, :, r] = _near(y / new[..., None])
                f[:, pg] = new
    return {"lens": torch.tensor([lens[b] + acc[b] + 1 for b in range(B)], dtype=torch.int32, device=DEV), **vals}
