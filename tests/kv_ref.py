"""Plain fp64 forms of the KV-cache operators, for the GPU tests: numpy, loops over sequences and
heads, one token at a time where that is clearest."""

import numpy as np

E4M3 = np.array([(-1.0 if c & 128 else 1.0) *
                 (np.nan if c & 127 == 127 else (c & 7) * 2.0 ** -9 if not c & 120 else
                  (1 + (c & 7) / 8) * 2.0 ** ((c >> 3 & 15) - 7)) for c in range(256)])


def half_step(y):
    """Half the distance between e4m3 values around |y| (saturating above 448)."""
    e = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -6)))
    return 2.0 ** (e - 4)


def scale_for(amax):
    if not amax > 0:
        return 2.0 ** -64
    s = 2.0 ** -64
    m, e = np.frexp(amax / 448.0)
    return max(s, 2.0 ** (e - 1 if m == 0.5 else e))


def rotated(x, rope, pos, pairs):
    """x [heads, D] fp64 by table row `pos`."""
    R = rope.shape[1]
    c, s = rope[pos, :R // 2].astype(np.float64), rope[pos, R // 2:].astype(np.float64)
    y = x.copy()
    i, j = (slice(0, R, 2), slice(1, R, 2)) if pairs else (slice(0, R // 2), slice(R // 2, R))
    y[:, i] = x[:, i] * c - x[:, j] * s
    y[:, j] = x[:, j] * c + x[:, i] * s
    return y


def mask_bits(words, N):
    w = words.astype(np.int64) & 0xffffffff
    return ((w[..., None] >> np.arange(32)) & 1).reshape(*words.shape[:-1], -1)[..., :N].astype(bool)


def cached(pool, scale, table, n, page):
    """The first n tokens of a sequence: values [n, Hkv, D] fp64."""
    t = np.arange(n)
    pg = table[t // page]
    return E4M3[pool[pg, :, t % page]] * scale[pg][:, :, None].astype(np.float64)


def attention(q, k, v, see, scale):
    """q [N, Hq, D], k, v [n, Hkv, D], see [N, n]: (out, lse, average |v| under the weights, and
    for each (i, h) the largest scale * sum_d |q_d k_d| and scale * max |q| * sum_d |k_d|)."""
    N, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, avg = np.zeros((N, Hq, D)), np.zeros((N, Hq, D))
    lse = np.full((N, Hq), -np.inf)
    big, spread = np.zeros((N, Hq)), np.zeros((N, Hq))
    for h in range(Hq):
        kk, vv = k[:, h // G], v[:, h // G]
        for i in range(N):
            w = see[i]
            if not w.any():
                continue
            x = kk[w] @ q[i, h] * scale
            m = x.max()
            p = np.exp(x - m)
            lse[i, h] = m + np.log(p.sum())
            out[i, h] = p @ vv[w] / p.sum()
            avg[i, h] = p @ np.abs(vv[w]) / p.sum()
            big[i, h] = (np.abs(kk[w]) @ np.abs(q[i, h])).max() * abs(scale)
            spread[i, h] = np.abs(kk[w]).sum(1).max() * np.abs(q[i, h]).max() * abs(scale)
    return out, lse, avg, big, spread
