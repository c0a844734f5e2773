"""Plain statements, in 64 bits, of the operators of a cache that is short of room:
4-bit pages, attention weights per token, selection within a budget, compaction."""
from __future__ import annotations

import numpy as np

BS = 16
LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def e4m3_round(x):
    """x >= 0 (64 bits) to the nearest e4m3 number, half to even, at most 448."""
    x = np.asarray(x, dtype=np.float64)
    step = np.exp2(np.maximum(np.frexp(x)[1] - 1, -6) - 3.0)
    with np.errstate(invalid="ignore"):
        return np.minimum(np.round(x / step) * step, 448.0)


def e4m3_code(v):
    """The byte of a number that e4m3 has (NaN: 0x7f)."""
    table = e4m3_values()
    order = np.argsort(table[:127])
    code = order[np.searchsorted(table[:127][order], np.where(np.isnan(v), 0, v))]
    return np.where(np.isnan(v), 0x7f, code).astype(np.uint8)


def e4m3_values():
    """The 256 values."""
    c = np.arange(256)
    e, m = c >> 3 & 15, c & 7
    v = np.where(e > 0, (1 + m / 8) * np.exp2(e - 7.0), m / 8 * np.exp2(-6.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


def quantise4(x, g):
    """Codes [..., d / 2] and scales [..., d / 16] (bytes) of rows x [..., d]; g: fp32."""
    g = float(np.float32(g))
    d = x.shape[-1]
    b = np.asarray(x, dtype=np.float64).reshape(x.shape[:-1] + (d // 16, 16))
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        top = np.abs(b).max(-1)
        s = np.where(np.isnan(top), np.nan, np.where(np.isinf(top), 448.0, e4m3_round(np.where(np.isfinite(top), top, 0) / (6 * g))))
        # |x| against half-way points t s g: at most 31 significant bits, exact
        a, unit = np.abs(b), (s * g)[..., None]
        code = np.zeros(b.shape, dtype=np.uint8)
        for t, up in ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5, 0)):
            code += (a >= t * unit) if up else (a > t * unit)
    code |= np.signbit(b).astype(np.uint8) << 3
    code[(s == 0) | np.isnan(s)] = 0
    code = code.reshape(x.shape[:-1] + (d // 2, 2))
    return code[..., 0] | code[..., 1] << 4, e4m3_code(s)


def pages4(blocks, heads, d, byte=0):
    return np.full((blocks, heads, 9 * d), byte, dtype=np.uint8)


def store4(cache, x, slots, g):
    """cache with row t of x [tokens, heads, d] at slots[t] (skipped outside the cache)."""
    cache, d = cache.copy(), x.shape[-1]
    codes, scales = quantise4(x, g)
    for t, s in enumerate(slots):
        if 0 <= s < cache.shape[0] * BS:
            b, o = s // BS, s % BS
            cache[b, :, o * (d // 2):(o + 1) * (d // 2)] = codes[t]
            cache[b, :, 8 * d + o * (d // 16):8 * d + (o + 1) * (d // 16)] = scales[t]
    return cache


def values4(cache, g):
    """What the pages stand for: [blocks, heads, 16, d]."""
    blocks, heads, d = cache.shape[0], cache.shape[1], cache.shape[2] // 9
    c = cache[:, :, :8 * d].reshape(blocks, heads, BS, d // 2)
    c = np.stack([c & 15, c >> 4], -1).reshape(blocks, heads, BS, d)
    v = np.where(c >= 8, -1.0, 1.0) * LEVELS[c & 7]
    f = e4m3_values()[cache[:, :, 8 * d:].reshape(blocks, heads, BS, d // 16)]
    return v * np.repeat(f, 16, -1) * float(np.float32(g))


def row_weights(q, keys, scale, lo, pos, cap=0.0, slope=0.0):
    """softmax weights of one query over keys [lo, pos] of `keys` [tokens, d]."""
    z = scale * keys[lo:pos + 1] @ q
    if cap > 0:
        z = cap * np.tanh(z / cap)
    z = z + slope * np.arange(lo, pos + 1)
    w = np.exp(z - z.max())
    return w / w.sum()


def attention(q, k, v, lens, start, group, scale, cap=0.0, slopes=None, window=-1):
    """out [rows, heads, d] for k, v: lists of [tokens, kv heads, d] per sequence."""
    out = np.zeros(q.shape)
    for s, n in enumerate(lens):
        for r in range(start[s], start[s + 1]):
            pos = n - (start[s + 1] - r)
            if pos < 0:
                continue
            lo = max(0, pos - window) if window >= 0 else 0
            for h in range(q.shape[1]):
                w = row_weights(q[r, h], k[s][:, h // group], scale, lo, pos, cap, 0.0 if slopes is None else slopes[h])
                out[r, h] = w @ v[s][lo:pos + 1, h // group]
    return out


def sequences(values, table, lens):
    """Per sequence the rows [tokens, heads, d] of `values` [blocks, heads, 16, d]."""
    out = []
    for s, n in enumerate(lens):
        p = values[table[s, :-(-n // BS)]]
        out.append(p.transpose(0, 2, 1, 3).reshape(-1, p.shape[1], p.shape[3])[:n])
    return out


def select_ref(scores, table, lens, budgets, sink, recent, width, fill):
    """(kept [sequences, heads, width], new lengths)."""
    heads = scores.shape[1]
    kept, new = np.full((len(lens), heads, width), fill, dtype=np.int64), np.zeros(len(lens), dtype=np.int64)
    for s, (n, budget) in enumerate(zip(lens, budgets)):
        new[s] = min(n, budget)
        last = min(recent, budget)
        first = min(sink, budget - last)
        for h in range(heads):
            if n <= budget:
                kept[s, h, :n] = np.arange(n)
                continue
            t = np.arange(first, n - last)
            x = scores[table[s, t // BS], h, t % BS].astype(np.float64)
            x = np.where(np.isnan(x), -np.inf, x)
            number = ~np.isnan(scores[table[s, t // BS], h, t % BS])
            order = np.lexsort((t, -x, ~number))  # numbers first, the largest first, the lowest position first
            chosen = t[order[:budget - first - last]]
            kept[s, h, :budget] = np.sort(np.concatenate([np.arange(first), chosen, np.arange(n - last, n)]))
    return kept, new


def compact_ref(caches, scores, table, kept, new, layout, kv_heads, four_bits):
    """caches (key, value: numpy bits) and scores after the tokens have moved."""
    out = []
    for i, c in enumerate(list(caches) + ([] if scores is None else [scores])):
        c = c.copy()
        if i == 2:
            parts = [(c, 1)]
        elif four_bits:
            d = c.shape[2] // 9
            parts = [(c[:, :, :8 * d].reshape(c.shape[0], c.shape[1], BS, d // 2), 1), (c[:, :, 8 * d:].reshape(c.shape[0], c.shape[1], BS, d // 16), 1)]
        else:
            parts = [(c, 1 if layout == "nhd" else (2 if i == 0 else 3))]
        done = []
        for x, kind in parts:
            # tokens in front of what a token holds: [blocks, heads, 16, ...]
            y = x if kind == 1 else (x.transpose(0, 1, 3, 2, 4) if kind == 2 else x.transpose(0, 1, 3, 2))
            was, now = y.copy(), y.copy()
            ratio = y.shape[1] // kv_heads
            for s in range(len(new)):
                for h in range(kv_heads):
                    to, src = np.arange(new[s]), kept[s, h, :new[s]]
                    for k in range(ratio):
                        now[table[s, to // BS], h * ratio + k, to % BS] = was[table[s, src // BS], h * ratio + k, src % BS]
            done.append(now if kind == 1 else (now.transpose(0, 1, 3, 2, 4) if kind == 2 else now.transpose(0, 1, 3, 2)))
        if four_bits and i < 2:
            out.append(np.ascontiguousarray(np.concatenate([p.reshape(p.shape[0], p.shape[1], -1) for p in done], 2)))
        else:
            out.append(np.ascontiguousarray(done[0]))
    return out
