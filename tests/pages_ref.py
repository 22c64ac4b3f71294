"""Plain forms of the calls that deal with a cache's pages, for the GPU tests: numpy, one sequence and one
place at a time."""

import numpy as np

NO_PAGE, REFS, PAGE, LENGTH, PARENT = -29, -30, -26, -25, -22


def free_pages(refs):
    return [int(p) for p in np.flatnonzero(refs == 0)]


def drop(refs, row, places, codes):
    for j in places:
        p = row[j]
        if p < 0:
            continue
        row[j] = -1
        if p >= len(refs):
            codes.append(PAGE)
        elif refs[p] <= 0:
            codes.append(REFS)
        else:
            refs[p] -= 1


def length_ok(n, table, page):
    return 0 <= n <= table.shape[1] * page


def reserve(refs, table, lens, news, N, page, codes):
    granted = np.zeros(len(lens), np.int32)
    left, needed = free_pages(refs), 0
    for b, n0 in enumerate(lens):
        n = N if news is None else int(news[b])
        if not (0 <= n <= N and length_ok(n0, table, page) and length_ok(int(n0) + n, table, page)):
            codes.append(LENGTH)
            continue
        want = [j for j in range(n0 // page, (n0 + n - 1) // page + 1) if table[b, j] < 0] if n else []
        needed += len(want)
        if want and needed > len(left):
            codes.append(NO_PAGE)
            continue
        granted[b] = n
        for j in want:
            p = left[needed - len(want) + want.index(j)]
            table[b, j] = p
            refs[p] = 1
    return granted


def trim(refs, table, lens, window, sinks, page, codes):
    for b, n in enumerate(lens):
        if not length_ok(n, table, page):
            codes.append(LENGTH)
            continue
        gone = [j for j in range(table.shape[1])
                if j * page >= n or (j * page >= sinks and (j + 1) * page - 1 <= int(n) - window)]
        drop(refs, table[b], gone, codes)


def free(refs, table, lens, ended, codes):
    for b in range(len(lens)):
        if ended is None or ended[b]:
            drop(refs, table[b], range(table.shape[1]), codes)
            lens[b] = 0


def fork(refs, table, lens, parents, release, page, pools, scales, codes):
    """pools, scales: arrays [layers, pages, ...] that copies are made in. Returns (table_out, lens_out)."""
    B, S = table.shape
    C = len(parents)
    out, n_out = np.full((C, S), -1, np.int32), np.zeros(C, np.int32)
    copies, seen = [], set()
    for c, p in enumerate(parents):
        if p == -1:
            continue
        if not 0 <= p < B:
            codes.append(PARENT)
            n_out[c] = -1
            continue
        n = int(lens[p])
        if not length_ok(n, table, page):
            codes.append(LENGTH)
            n_out[c] = -1
            continue
        n_out[c] = n
        for j in range(-(-n // page)):
            q = int(table[p, j])
            if q >= len(refs):
                codes.append(PAGE)
                continue
            if q < 0:
                continue
            if j < n // page or (release and p not in seen):
                out[c, j] = q
                refs[q] += 1
            else:
                copies.append((c, j, q, n % page))
        seen.add(p)
    if release:
        for p in range(B):
            if not length_ok(lens[p], table, page):
                codes.append(LENGTH)
            drop(refs, table[p].copy(), range(S), codes)
    left = free_pages(refs)
    for i, (c, j, q, rows) in enumerate(copies):
        if i >= len(left):
            codes.append(NO_PAGE)
            n_out[c] = -1
            drop(refs, out[c], range(S), codes)
            continue
        out[c, j] = left[i]
        refs[left[i]] = 1
        for x in pools:
            x[:, left[i], :, :rows] = x[:, q, :, :rows]
        for x in scales:
            x[:, left[i]] = x[:, q]
    return out, n_out


def compact(refs, table, pools, codes):
    live = int((refs > 0).sum())
    holes = [p for p in range(live) if refs[p] == 0]
    movers = [p for p in range(live, len(refs)) if refs[p] > 0]
    page_map = np.where(refs > 0, np.arange(len(refs)), -1).astype(np.int32)
    for to, frm in zip(holes, movers):
        page_map[frm] = to
        for x in pools:
            x[:, to] = x[:, frm]
        refs[to], refs[frm] = refs[frm], 0
    for b, j in np.argwhere(table >= 0):
        if table[b, j] >= len(refs):
            codes.append(PAGE)
        else:
            table[b, j] = page_map[table[b, j]]
    return page_map, live
