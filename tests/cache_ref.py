"""Plain statements of the cache operators, for the tests: pages handed out one by
one in Python, rows stored one by one."""
from __future__ import annotations

import numpy as np

BS = 16


def pages(n):
    return -(-int(n) // BS)


def tables_ref(table, lens, ring, state, rows, keep=None, start=None):
    """(table, ring, slots, positions, new lens, new state) after a step; inputs unchanged."""
    table, ring = table.copy(), ring.copy()
    n, blocks = len(lens), len(ring)
    keep = lens if keep is None else keep
    start = np.arange(n + 1) if start is None else start
    head, count = int(state[0]), int(state[1])
    taken = back = 0
    slots, positions = np.full(rows, -1), np.zeros(rows, dtype=np.int64)
    new = np.zeros(n, dtype=np.int64)
    for s in range(n):
        own, new[s] = pages(lens[s]), int(keep[s]) + int(start[s + 1] - start[s])
        want = pages(new[s])
        for page in range(own, want):
            table[s, page] = ring[(head + taken) % blocks]
            taken += 1
        for page in range(want, own):
            ring[(head + count + back) % blocks] = table[s, page]
            back += 1
        for i, t in enumerate(range(start[s], start[s + 1])):
            pos = int(keep[s]) + i
            positions[t] = pos
            slots[t] = table[s, pos // BS] * BS + pos % BS
    return table, ring, slots, positions, new, np.array([(head + taken) % blocks, count - taken + back])


def make_batch(seed, n, longest, tokens, cut=False, spare=40, single=False, fresh=False):
    """A consistent state: lengths, tables and a ring that holds every other page."""
    rng = np.random.default_rng(seed)
    lens = np.zeros(n, dtype=np.int64) if fresh else rng.integers(0, longest + 1, n)
    keep = None
    new = np.ones(n, dtype=np.int64) if single else rng.integers(0, tokens + 1, n)
    if cut:
        keep = np.maximum(lens - rng.integers(0, 40, n), 0)
        keep[rng.random(n) < 0.2] = 0
    start = None if single else np.concatenate([[0], np.cumsum(new)])
    width = pages(longest + tokens) + 1
    own = np.array([pages(x) for x in lens], dtype=np.int64)
    blocks = int(own.sum()) + n * (pages(tokens) + 1) + spare
    ids = rng.permutation(blocks)
    table = np.full((n, width), -7, dtype=np.int64)
    at = 0
    for s in range(n):
        table[s, :own[s]] = ids[at:at + own[s]]
        at += own[s]
    free = blocks - at
    head = int(rng.integers(0, blocks))
    ring = np.full(blocks, -9, dtype=np.int64)
    ring[(head + np.arange(free)) % blocks] = ids[at:]
    return dict(table=table, lens=lens, keep=keep, start=start, ring=ring, state=np.array([head, free]),
                max_len=longest + tokens, tokens=int(new.sum()))


def cache_shapes(blocks, k_heads, k_size, v_heads, v_size, layout, elem):
    if layout == "nhd":
        return (blocks, k_heads, BS, k_size), (blocks, v_heads, BS, v_size)
    x = 16 // elem
    return (blocks, k_heads, k_size // x, BS, x), (blocks, v_heads, v_size, BS)


def store_ref(cache, rows, slots, layout, is_key):
    """cache (numpy, element bits) with row t stored at slots[t] (skipped outside the cache)."""
    cache = cache.copy()
    for t, s in enumerate(slots):
        if s < 0 or s >= cache.shape[0] * BS:
            continue
        b, o = s // BS, s % BS
        if layout == "nhd":
            cache[b, :, o] = rows[t]
        elif is_key:
            cache[b, :, :, o] = rows[t].reshape(cache.shape[1], cache.shape[2], cache.shape[4])
        else:
            cache[b, :, :, o] = rows[t]
    return cache
