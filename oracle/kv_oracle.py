"""CPU oracle of the 8-bit paged KV cache -- TEST INFRASTRUCTURE ONLY.

Append, attention and eviction as plain definitions (numpy, float64), sequence
by sequence.  It shares no code with the CUDA path.  Pools are dicts of numpy
arrays: k, v uint8 [pages, Hkv, P, D], ks, vs float32 [pages, Hkv].
"""
from __future__ import annotations

import numpy as np

# the value of each e4m3 code; the NaN codes 0x7f and 0xff, which the cache never holds, as V's conversion and the
# rescaling of codes read them, +-480
VALUE = np.array([(-1.0 if c & 0x80 else 1.0) *
                  ((c & 7) * 2.0 ** -9 if not c & 0x78 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3 & 15) - 7))
                  for c in range(256)])


def nearest_code(x: np.ndarray) -> np.ndarray:
    """The e4m3 code nearest to each x (ties to the even code, magnitudes above 448 to 448)."""
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(VALUE[:127], a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = VALUE[hi] - a, a - VALUE[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def least_scale(amax: float) -> float:
    """The least power of two s >= 2^-126 with amax <= 448 s."""
    e = -126
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def rescaled(codes: np.ndarray, ratio: np.float32) -> np.ndarray:
    """Codes of the values times a ratio (the product in fp32)."""
    return nearest_code((VALUE[codes].astype(np.float32) * np.float32(ratio)).astype(np.float64))


def append(pool, table, lens, cu, k, v):
    """Stores rows k, v (float64 [T, Hkv, D]) in the pool, in place."""
    P = pool["k"].shape[2]
    for b, L in enumerate(lens):
        n = int(cu[b + 1] - cu[b])
        for p in range((L - n) // P, -(-L // P)) if n else ():
            page, lo, hi = table[b][p], max(L - n, p * P), min(L, p * P + P)
            for name, new in (("k", k), ("v", v)):
                rows = new[cu[b] + lo - (L - n):cu[b] + hi - (L - n)]
                for h in range(rows.shape[1]):
                    x = rows[:, h]
                    finite = np.abs(x[np.isfinite(x)])
                    s = least_scale(finite.max() if finite.size else 0.0)
                    codes, was = pool[name][page, h], float(pool[name + "s"][page, h])
                    if lo > p * P:
                        s = max(s, was)
                        if s != was:
                            ratio = np.float32(was) / np.float32(s)
                            codes[:lo - p * P] = rescaled(codes[:lo - p * P], ratio)
                    x = np.where(np.isnan(x), 0.0, x).astype(np.float32) / np.float32(s)
                    codes[lo - p * P:hi - p * P] = nearest_code(x.astype(np.float64))
                    pool[name + "s"][page, h] = s


def rows(pool, name, table_row, n, h):
    """The values of the first n tokens of a sequence for head h: [n, D]."""
    P = pool[name].shape[2]
    ids = np.asarray(table_row[:-(-n // P)], dtype=np.int64)
    x = VALUE[pool[name][ids, h]] * pool[name + "s"][ids, h].astype(np.float64)[:, None, None]
    return x.reshape(-1, x.shape[-1])[:n]


def attention(pool, table, lens, cu, q, scale, weights=None):
    """(out, lse, sum_t p_t |V|, max_t scale sum_d |q K|), of q float64 [T, Hq,
    D]; weights float64 [B, Hkv, W] gains the softmax weights in place.  The last
    two say how large the terms were that the results add up."""
    T, Hq, D = q.shape
    Hkv = pool["k"].shape[1]
    g = Hq // Hkv
    out, mass = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, size = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for b, L in enumerate(lens):
        n = int(cu[b + 1] - cu[b])
        for h in range(Hkv if n else 0):
            k, v = rows(pool, "k", table[b], L, h), rows(pool, "v", table[b], L, h)
            for i in range(n):
                seen = L - n + i + 1
                if seen <= 0:
                    continue
                r = cu[b] + i
                for head in range(h * g, h * g + g):
                    s = scale * (k[:seen] @ q[r, head])
                    m = s.max()
                    p = np.exp(s - m)
                    l = p.sum()
                    p = p / l
                    out[r, head], lse[r, head] = p @ v[:seen], m + np.log(l)
                    mass[r, head] = p @ np.abs(v[:seen])
                    size[r, head] = scale * (np.abs(k[:seen]) @ np.abs(q[r, head])).max()
                    if weights is not None:
                        weights[b, h, :seen] += p
    return out, lse, mass, size


def evict(pool, table, lens, weights, budget, sink, recent, dst, dst_table):
    """Copies the tokens that stay into dst (in place).  Returns (lens, weights, kept)."""
    P, D = pool["k"].shape[2:]
    B, Hkv = len(lens), pool["k"].shape[1]
    kept = np.full((B, Hkv, budget), -1, np.int32)
    w = np.zeros((B, Hkv, budget), np.float32)
    for b, L in enumerate(lens):
        for h in range(Hkv):
            stay = list(range(L))
            if L > budget:
                key = np.where(np.isnan(weights[b, h, :L]), np.inf, weights[b, h, :L])
                nan = np.isnan(weights[b, h, :L])
                mid = sorted(range(sink, L - recent), key=lambda t: (not nan[t], -key[t], t))
                stay = sorted([*range(sink), *mid[:budget - sink - recent], *range(L - recent, L)])
            kept[b, h, :len(stay)], w[b, h, :len(stay)] = stay, weights[b, h, stay]
            for p in range(-(-len(stay) // P)):
                here, to = stay[p * P:p * P + P], dst_table[b][p]
                for name in ("k", "v"):
                    src = [(table[b][t // P], t % P) for t in here]
                    s = np.array([pool[name + "s"][i, h] for i, _ in src], np.float32)
                    big = s.max()
                    dst[name + "s"][to, h] = big
                    for j, (i, slot) in enumerate(src):
                        c = pool[name][i, h, slot]
                        dst[name][to, h, j] = c if s[j] == big else rescaled(c[None], s[j] / big)[0]
    return np.minimum(lens, budget).astype(np.int32), w, kept
