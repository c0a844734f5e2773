"""The operators of a serving step around the paged cache, as cases to be measured.

  tables  block tables, slot map and positions of a step, and the pool of free pages, from the sequences' lengths
  append  the step's keys and values stored into the paged cache through the slot map
  diff    differential attention of the new tokens over the paged cache, with the per-head RMS norm of its output

`run` computes the plain form of an operator, in elementary torch operations, or with `own` calls the framework's.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16,
          "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FP8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
DEVICE = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of the 32 x 4096 batch: the smallest call, all latency
        dict(name="tables decode 32", op="tables", seqs=32, longest=4096, equal=True, tokens=1, cut=False, fresh=False),
        # a ragged batch after speculative decoding: drafts dropped, sequences finished, up to four new tokens each
        dict(name="tables drafts 256", op="tables", seqs=256, longest=32768, equal=False, tokens=4, cut=True, fresh=False),
        # the prompts of a large batch: every page of 128 x 16384 handed out at once
        dict(name="tables prompts 128", op="tables", seqs=128, longest=16384, equal=True, tokens=16384, cut=False, fresh=True),
        # the new token of the 32 x 4096 batch, fp16, both caches in the split layout
        dict(name="append decode 32 f16", op="append", tokens=32, run=1, k_heads=4, k_size=128, v_heads=4, v_size=128,
             dtype="f16", kv="same", layout="split", fused=True),
        # an odd chunk of a prompt into an fp8 cache of differential heads
        dict(name="append chunk bf16 e4m3", op="append", tokens=5003, run=700, k_heads=16, k_size=64, v_heads=8, v_size=128,
             dtype="bf16", kv="e4m3", layout="nhd", fused=True),
        # drafted tokens of many sequences into an e5m2 cache, few per page
        dict(name="append drafts f16 e5m2", op="append", tokens=1021, run=4, k_heads=8, k_size=128, v_heads=8, v_size=128,
             dtype="f16", kv="e5m2", layout="split", fused=False),
        # a whole prompt, bf16, split layout: bandwidth
        dict(name="append prompt bf16", op="append", tokens=32768, run=32768, k_heads=8, k_size=128, v_heads=8, v_size=128,
             dtype="bf16", kv="same", layout="split", fused=True),
        # two short sequences in fp32: latency
        dict(name="diff tiny f32", op="diff", seqs=2, longest=600, equal=False, heads=4, kv_heads=2, size=64, dtype="f32",
             kv="same", layout="nhd", tokens=1, norm=True, softcap=0.0, alibi=False, window=-1),
        # the 32 x 4096 decode batch with differential heads
        dict(name="diff decode 32x4096 f16", op="diff", seqs=32, longest=4096, equal=True, heads=16, kv_heads=4, size=64,
             dtype="f16", kv="same", layout="split", tokens=1, norm=True, softcap=0.0, alibi=False, window=-1),
        # long contexts: 4 x 100000, groups of seven heads
        dict(name="diff long 4x100000 bf16", op="diff", seqs=4, longest=100000, equal=True, heads=28, kv_heads=4, size=64,
             dtype="bf16", kv="same", layout="nhd", tokens=1, norm=True, softcap=0.0, alibi=False, window=-1),
        # four drafted tokens verified at once over an fp8 cache
        dict(name="diff drafts 32x4096 e4m3", op="diff", seqs=32, longest=4096, equal=True, heads=16, kv_heads=8, size=64,
             dtype="bf16", kv="e4m3", layout="split", tokens=4, norm=True, softcap=30.0, alibi=False, window=-1),
        # a ragged batch of wide heads (keys of 128, values of 256) with ALiBi
        dict(name="diff ragged wide bf16", op="diff", seqs=64, longest=16384, equal=False, heads=16, kv_heads=8, size=128,
             dtype="bf16", kv="same", layout="split", tokens=1, norm=True, softcap=0.0, alibi=True, window=-1),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "diff", "diff"])
    if op == "tables":
        if rng.random() < 0.3:
            longest = _spread(rng, 17, 16384)
            return dict(op=op, seqs=_spread(rng, 1, min(1024, 2097152 // longest)), longest=longest,
                        equal=rng.random() < 0.5, tokens=longest, cut=False, fresh=True)
        return dict(op=op, seqs=_spread(rng, 1, 4096), longest=_spread(rng, 64, 32768), equal=rng.random() < 0.3,
                    tokens=rng.choice([1, 1, 2, 4, 7, 16]), cut=rng.random() < 0.5, fresh=False)
    if op == "append":
        dtype = rng.choice(["f32", "f16", "bf16"])
        kv = "same" if dtype == "f32" else rng.choice(["same", "e4m3", "e5m2"])
        heads = rng.choice([1, 2, 4, 8])
        wide = rng.random() < 0.4
        size = rng.choice([64, 128])
        tokens = _spread(rng, 1, 32768 // (2 if dtype == "f32" else 1) // (2 if wide and size == 128 else 1))
        return dict(op=op, tokens=tokens, run=_spread(rng, 1, tokens), k_heads=heads * (2 if wide else 1), k_size=size,
                    v_heads=heads, v_size=size * (2 if wide else 1), dtype=dtype, kv=kv,
                    layout=rng.choice(["split", "nhd"]), fused=rng.random() < 0.5)
    dtype = rng.choice(["f32", "f16", "bf16", "f16", "bf16"])
    kv = "same" if dtype == "f32" else rng.choice(["same", "same", "e4m3", "e5m2"])
    size = rng.choice([64, 64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8])
    longest = _spread(rng, 1, 65536)
    per = kv_heads * 4 * size * (4 if dtype == "f32" else 2)
    seqs = _spread(rng, 1, max(1, min(128, 819200000 // (longest * per))))
    return dict(op=op, seqs=seqs, longest=longest, equal=rng.random() < 0.5, heads=group * kv_heads, kv_heads=kv_heads,
                size=size, dtype=dtype, kv=kv, layout=rng.choice(["split", "nhd"]),
                tokens=rng.choice([1, 1, 1, 2, 4]) if group <= 2 else 1, norm=rng.random() < 0.8,
                softcap=rng.choice([0.0, 0.0, 30.0]), alibi=rng.random() < 0.3,
                window=rng.choice([-1, -1, -1, 1000]))


def _lengths(case):
    """The batch's lengths but for their order: all the longest, or spread over their logarithm."""
    n, top = case["seqs"], case["longest"]
    if case["equal"]:
        return np.full(n, top, dtype=np.int64)
    return np.clip(np.round(top ** ((np.arange(n) + 1) / n)), 1, top).astype(np.int64)


def _pages(n):
    return (n + BLOCK - 1) // BLOCK


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    torch.cuda.set_device(0)
    rng = np.random.default_rng([seed, 11])
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed * 7 + 3)
    return {"tables": _prepare_tables, "append": _prepare_append, "diff": _prepare_diff}[case["op"]](case, rng, gen)


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEVICE)


def _prepare_tables(case, rng, gen):
    n, top = case["seqs"], case["longest"]
    lens = rng.permutation(_lengths(case))
    if case["fresh"]:  # prompts: nothing stored yet, every token of the length is new
        new, lens, keep = lens, np.zeros(n, dtype=np.int64), None
    else:
        if case["equal"]:
            lens = lens - rng.integers(0, 2 * BLOCK, n).clip(max=top - 1)
        new = np.ones(n, dtype=np.int64) if case["tokens"] == 1 else rng.integers(1, case["tokens"] + 1, n)
        keep = None
        if case["cut"]:  # drafted tokens turned down, and one sequence in eight at its end
            keep = lens - rng.integers(0, case["tokens"] + 1, n).clip(max=lens)
            done = rng.random(n) < 0.125
            keep[done] = 0
            new[done] = 0
    start = None
    if case["fresh"] or case["tokens"] > 1 or case["cut"]:
        start = np.concatenate([[0], np.cumsum(new)])
    rows = int(new.sum()) if case["fresh"] else n * case["tokens"]  # rows behind the last token: a padded batch
    max_len = top + 64  # the sizes of pool and table go by the case alone
    width = _pages(max_len)
    owned = _pages(lens)
    blocks = int(_pages(_lengths(case)).sum()) + 64 + (0 if case["fresh"] else n * (1 + _pages(case["tokens"])))
    ids = rng.permutation(blocks)
    table = np.full((n, width), -1, dtype=np.int64)
    table[np.arange(width)[None, :] < owned[:, None]] = ids[:owned.sum()]
    free = blocks - int(owned.sum())
    head = int(rng.integers(0, blocks))
    ring = np.full(blocks, -1, dtype=np.int64)
    ring[(head + np.arange(free)) % blocks] = ids[owned.sum():]
    return dict(op="tables", block_tables=_int(table), seq_lens=_int(lens), free_ring=_int(ring),
                pool_state=_int([head, free]), keep_lens=None if keep is None else _int(keep),
                query_start=None if start is None else _int(start), max_seq_len=max_len,
                slots=torch.empty(rows, dtype=torch.int32, device=DEVICE),
                positions=torch.empty(rows, dtype=torch.int32, device=DEVICE),
                new_seq_lens=torch.empty(n, dtype=torch.int32, device=DEVICE),
                new_pool_state=torch.empty(2, dtype=torch.int32, device=DEVICE),
                done_counter=torch.zeros(1, dtype=torch.int32, device=DEVICE))


def _cache_shapes(blocks, k_heads, k_size, v_heads, v_size, layout, width):
    if layout == "nhd":
        return (blocks, k_heads, BLOCK, k_size), (blocks, v_heads, BLOCK, v_size)
    x = 16 // width
    return (blocks, k_heads, k_size // x, BLOCK, x), (blocks, v_heads, v_size, BLOCK)


def _normal(shape, dtype, gen, scale=1.0):
    t = torch.empty(shape, dtype=dtype if dtype.itemsize > 1 else torch.float16, device=DEVICE)
    t.normal_(generator=gen)
    if scale != 1.0:
        t.mul_(1.0 / scale)
    return t if t.dtype == dtype else t.to(dtype)


def _prepare_append(case, rng, gen):
    tokens, dtype = case["tokens"], DTYPES[case["dtype"]]
    kv = case["dtype"] if case["kv"] == "same" else case["kv"]
    # runs of `run` tokens at successive positions, each from an odd place inside a page
    runs = [min(case["run"], tokens - a) for a in range(0, tokens, case["run"])]
    first = rng.integers(0, BLOCK, len(runs))
    need = _pages(first + np.array(runs))
    blocks = int((_pages(np.array(runs)) + 1).sum()) + 8
    ids = rng.permutation(blocks)
    page0 = np.repeat(np.cumsum(need) - need, runs)
    pos = np.arange(tokens) - np.repeat(np.cumsum(runs) - runs, runs) + np.repeat(first, runs)
    slots = ids[page0 + pos // BLOCK] * BLOCK + pos % BLOCK
    if tokens > 40:
        slots[-int(rng.integers(1, 9)):] = -1  # rows behind the last token: a padded batch
    hk, dk, hv, dv = case["k_heads"], case["k_size"], case["v_heads"], case["v_size"]
    if case["fused"]:  # keys and values as the projection leaves them, beside the queries
        row = _normal((tokens, 2 * hk * dk + hk * dk + hv * dv), dtype, gen)
        key = row[:, 2 * hk * dk:3 * hk * dk].unflatten(1, (hk, dk))
        value = row[:, 3 * hk * dk:].unflatten(1, (hv, dv))
    else:
        key, value = _normal((tokens, hk, dk), dtype, gen), _normal((tokens, hv, dv), dtype, gen)
    ks, vs = _cache_shapes(blocks, hk, dk, hv, dv, case["layout"], DTYPES[kv].itemsize)
    scale = 1.0 if case["kv"] == "same" else 0.0173
    return dict(op="append", key=key, value=value, slots=_int(slots), key_cache=_normal(ks, DTYPES[kv], gen),
                value_cache=_normal(vs, DTYPES[kv], gen), layout=case["layout"],
                kv_dtype=None if case["kv"] == "same" else case["kv"], k_scale=scale, v_scale=1.25 * scale)


def _prepare_diff(case, rng, gen):
    n, h, hk, d = case["seqs"], case["heads"], case["kv_heads"], case["size"]
    dtype, kv = DTYPES[case["dtype"]], case["dtype"] if case["kv"] == "same" else case["kv"]
    lens = _lengths(case)
    new = np.minimum(1 + np.arange(n) % case["tokens"], lens)
    order = rng.permutation(n)
    lens, new = lens[order], new[order]
    width = _pages(case["longest"])
    owned = _pages(lens)
    blocks = int(owned.sum()) + 3
    ids = rng.permutation(blocks)
    table = np.zeros((n, width), dtype=np.int64)
    table[np.arange(width)[None, :] < owned[:, None]] = ids[:owned.sum()]
    rows = int(new.sum())
    scale = 1.0 if case["kv"] == "same" else 2.0 ** -6
    ks, vs = _cache_shapes(blocks, 2 * hk, d, hk, 2 * d, case["layout"], DTYPES[kv].itemsize)
    parts = max(1, -(-case["longest"] // 512))
    real = lambda *shape: torch.empty(shape, dtype=torch.float32, device=DEVICE)  # noqa: E731
    return dict(
        op="diff", query=_normal((rows, h, 2, d), dtype, gen), out=torch.empty((rows, h, 2 * d), dtype=dtype, device=DEVICE),
        key_cache=_normal(ks, DTYPES[kv], gen, scale), value_cache=_normal(vs, DTYPES[kv], gen, scale),
        block_tables=_int(table), seq_lens=_int(lens), seq_lens_host=lens.astype(np.int32),
        query_start=_int(np.concatenate([[0], np.cumsum(new)])) if case["tokens"] > 1 else None,
        max_query_len=case["tokens"], num_kv_heads=hk, scale=1.0 / math.sqrt(d), max_seq_len=case["longest"],
        lambdas=torch.rand((h,), generator=gen, device=DEVICE) * 0.7 + 0.1,
        norm=case["norm"], norm_weight=1.0 + 0.1 * torch.randn((2 * d,), generator=gen, device=DEVICE) if case["norm"] else None,
        norm_eps=1e-5, out_scale=0.2, softcap=case["softcap"], window_left=case["window"],
        alibi_slopes=torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device=DEVICE) if case["alibi"] else None,
        layout=case["layout"], kv_dtype=None if case["kv"] == "same" else case["kv"], k_scale=scale, v_scale=scale,
        exp_sums=real(rows, 2 * h, parts), max_logits=real(rows, 2 * h, parts), tmp_out=real(rows, 2 * h, parts, 2 * d),
        partition_counters=torch.zeros((n, hk), dtype=torch.int32, device=DEVICE),
        tile_counters=torch.zeros(2, dtype=torch.int32, device=DEVICE))


# ------------------------------------------------------------------ passes

def run(state):
    if own:
        return {"tables": _own_tables, "append": _own_append, "diff": _own_diff}[state["op"]](state)
    return {"tables": _plain_tables, "append": _plain_append, "diff": _plain_diff}[state["op"]](state)


def _tables_outputs(s):
    return {k: s[k] for k in ("slots", "positions", "new_seq_lens", "new_pool_state", "block_tables", "free_ring")}


def _own_tables(s):
    import paged_kv_attention_v2_gb300 as pa
    pa.pa_build_tables(s["block_tables"], s["seq_lens"], s["free_ring"], s["pool_state"], s["slots"],
                       max_seq_len=s["max_seq_len"], keep_lens=s["keep_lens"], query_start=s["query_start"],
                       positions=s["positions"], new_seq_lens=s["new_seq_lens"], new_pool_state=s["new_pool_state"],
                       done_counter=s["done_counter"])
    return _tables_outputs(s)


def _own_append(s):
    import paged_kv_attention_v2_gb300 as pa
    pa.pa_append_kv(s["key"], s["value"], s["key_cache"], s["value_cache"], s["slots"], layout=s["layout"],
                    kv_dtype=s["kv_dtype"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return {"key_cache": s["key_cache"], "value_cache": s["value_cache"]}


def _own_diff(s):
    import paged_kv_attention_v2_gb300 as pa
    several = dict(query_start=s["query_start"], max_query_len=s["max_query_len"]) if s["query_start"] is not None else {}
    pa.pa_diff_decode(s["out"], s["query"], s["key_cache"], s["value_cache"], s["block_tables"], s["seq_lens"],
                      lambdas=s["lambdas"], num_kv_heads=s["num_kv_heads"], scale=s["scale"], max_seq_len=s["max_seq_len"],
                      norm=s["norm"], norm_weight=s["norm_weight"], norm_eps=s["norm_eps"], out_scale=s["out_scale"],
                      softcap=s["softcap"], window_left=s["window_left"], alibi_slopes=s["alibi_slopes"],
                      layout=s["layout"], kv_dtype=s["kv_dtype"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                      seq_lens_host=s["seq_lens_host"], exp_sums=s["exp_sums"], max_logits=s["max_logits"],
                      tmp_out=s["tmp_out"], partition_counters=s["partition_counters"],
                      tile_counters=s["tile_counters"], **several)
    return s["out"]


def _plain_tables(s):
    table, ring, lens = s["block_tables"], s["free_ring"], s["seq_lens"].long()
    n, width, blocks, rows = table.shape[0], table.shape[1], ring.shape[0], s["slots"].shape[0]
    keep = lens if s["keep_lens"] is None else s["keep_lens"].long()
    seq = torch.arange(n, device=DEVICE)
    start = torch.arange(n + 1, device=DEVICE) if s["query_start"] is None else s["query_start"].long()
    after = keep + start[1:] - start[:-1]
    owned, wanted = (lens + BLOCK - 1) // BLOCK, (after + BLOCK - 1) // BLOCK
    pops, pushes = (wanted - owned).clamp(min=0), (owned - wanted).clamp(min=0)
    pop0, push0 = pops.cumsum(0) - pops, pushes.cumsum(0) - pushes
    head, count = s["pool_state"][0].long(), s["pool_state"][1].long()
    # freed pages go behind the last free one (the ring's last place but one takes what is no push)
    page = torch.arange(width, device=DEVICE)[None, :]
    freed = (page >= wanted[:, None]) & (page < owned[:, None])
    to = torch.where(freed, (head + count + push0[:, None] + page - wanted[:, None]) % blocks, blocks)
    ring.copy_(torch.cat([ring, ring[:1]]).scatter(0, to.reshape(-1), table.reshape(-1))[:blocks])
    # new pages come from the front
    taken = (page >= owned[:, None]) & (page < wanted[:, None])
    at = (head + pop0[:, None] + page - owned[:, None]) % blocks
    table.copy_(torch.where(taken, ring[at], table))
    # the new tokens
    row = torch.arange(rows, device=DEVICE)
    owner = torch.searchsorted(start[1:], row, right=True).clamp(max=n - 1)
    pos = keep[owner] + row - start[owner]
    there = row < start[n]
    pos = torch.where(there, pos, 0)
    slot = table[seq[owner], pos // BLOCK] * BLOCK + pos % BLOCK
    s["slots"].copy_(torch.where(there, slot, -1))
    s["positions"].copy_(pos)
    s["new_seq_lens"].copy_(after)
    popped, pushed = pops.sum(), pushes.sum()
    s["new_pool_state"].copy_(torch.stack([(head + popped) % blocks, count - popped + pushed]))
    return _tables_outputs(s)


def _plain_store(x, cache, slots, layout, scale, kv, is_key):
    x = x.float()
    if kv is not None:
        x = (x / scale).clamp(-FP8_MAX[kv], FP8_MAX[kv])
    x = x.to(cache.dtype)
    # a row without a slot stores the first row that has one again
    there = slots >= 0
    row = torch.where(there, torch.arange(slots.shape[0], device=DEVICE), there.int().argmax())
    blk, off = slots[row].long() // BLOCK, slots[row].long() % BLOCK
    # an all-bits view of the elements: index operations are plain copies
    bits = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[cache.element_size()]
    c, x = cache.view(bits), x.contiguous().view(bits)[row]
    if layout == "nhd":
        c[blk, :, off] = x
    elif is_key:
        c[blk, :, :, off] = x.unflatten(2, (cache.shape[2], cache.shape[4]))
    else:
        c[blk, :, :, off] = x
    return cache


def _plain_append(s):
    return {"key_cache": _plain_store(s["key"], s["key_cache"], s["slots"], s["layout"], s["k_scale"], s["kv_dtype"], True),
            "value_cache": _plain_store(s["value"], s["value_cache"], s["slots"], s["layout"], s["v_scale"], s["kv_dtype"],
                                        False)}


def _gathered(cache, table, layout, scale, is_key, tokens):
    """The cache's rows of each sequence in order: [sequences, heads, tokens, size], 32 bits."""
    p = cache.view(torch.uint8)[table].view(cache.dtype) if cache.element_size() == 1 else cache[table]
    p = p.float()
    if scale != 1.0:
        p = p * scale
    if layout == "nhd":      # [s, page, head, off, d]
        p = p.transpose(1, 2)
    elif is_key:             # [s, page, head, d/x, off, x]
        p = p.permute(0, 2, 1, 4, 3, 5).flatten(4)
    else:                    # [s, page, head, d, off]
        p = p.permute(0, 2, 1, 4, 3)
    return p.reshape(p.shape[0], p.shape[1], -1, p.shape[-1])[:, :, :tokens]


def _plain_diff(s):
    q, table, lens = s["query"].float(), s["block_tables"].long(), s["seq_lens"].long()
    n, hk, longest, device = table.shape[0], s["num_kv_heads"], s["max_seq_len"], q.device
    rows, h, d = q.shape[0], q.shape[1], q.shape[3]
    g, most = h // hk, s["max_query_len"]
    # the queries of a sequence side by side, padded to the most that one has
    if s["query_start"] is None:
        owner, index, count = torch.arange(n, device=device), torch.zeros(n, dtype=torch.long, device=device), 1
    else:
        start = s["query_start"].long()
        owner = torch.searchsorted(start[1:], torch.arange(rows, device=device), right=True)
        index = torch.arange(rows, device=device) - start[owner]
        count = start[1:] - start[:-1]
    many = torch.zeros((n, most, h, 2, d), device=device)
    many[owner, index] = q
    at = lens - count  # position of the first query
    pos = at[:, None] + torch.arange(most, device=device)[None, :]
    keys = _gathered(s["key_cache"], table, s["layout"], s["k_scale"], True, longest)      # [n, 2 hk, t, d]
    z = torch.einsum("nmkgcd,nkctd->nmkgct", many.unflatten(2, (hk, g)), keys.unflatten(1, (hk, 2))) * s["scale"]
    if s["softcap"] > 0:
        z = s["softcap"] * torch.tanh(z / s["softcap"])
    t = torch.arange(longest, device=device)
    if s["alibi_slopes"] is not None:  # a shift by the last position leaves the softmax as it is, and its values small
        z = z + s["alibi_slopes"].view(hk, g)[None, None, :, :, None, None] * (t[None, :] - lens[:, None] + 1)[:, None, None, None, None, :]
    seen = (t <= pos[:, :, None]) & (t < lens[:, None, None])
    if s["window_left"] >= 0:
        seen = seen & (t >= pos[:, :, None] - s["window_left"])
    z = z.masked_fill(~seen[:, :, None, None, None, :], float("-inf"))
    z = torch.exp(z - z.amax(-1, keepdim=True))
    z = z / z.sum(-1, keepdim=True)
    z = z[:, :, :, :, 0] - s["lambdas"].view(hk, g)[None, None, :, :, None] * z[:, :, :, :, 1]
    z = z.masked_fill(~seen[:, :, None, None, :], 0.0)
    values = _gathered(s["value_cache"], table, s["layout"], s["v_scale"], False, longest)  # [n, hk, t, 2 d]
    o = torch.einsum("nmkgt,nkte->nmkge", z, values).flatten(2, 3)[owner, index]
    if s["norm"]:
        o = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + s["norm_eps"]) * s["norm_weight"]
    s["out"].copy_(o * s["out_scale"])
    return s["out"]


# ------------------------------------------------------------------ bytes and operations

def work(case):
    if case["op"] == "tables":
        n = case["seqs"]
        new = int(_lengths(case).sum()) if case["fresh"] else n * (1 + case["tokens"]) // 2
        pages = new // BLOCK + (n if case["fresh"] else 0)
        # lengths in and out, offsets, the pages that new tokens share with old ones; each new page is read and written
        return {"bytes": n * (16 + (4 if case["cut"] else 0)) + pages * 8 + new * 8, "flops": 0}
    if case["op"] == "append":
        values = case["tokens"] * (case["k_heads"] * case["k_size"] + case["v_heads"] * case["v_size"])
        size = DTYPES[case["dtype"]].itemsize
        return {"bytes": values * (size + (size if case["kv"] == "same" else 1)) + 4 * case["tokens"],
                "flops": 0 if case["kv"] == "same" else values}
    lens, d = _lengths(case), case["size"]
    if case["window"] >= 0:
        lens = np.minimum(lens, case["window"] + (1 + case["tokens"]) // 2)
    seen, rows = int(lens.sum()), int(np.minimum(1 + np.arange(case["seqs"]) % case["tokens"], _lengths(case)).sum())
    wide = DTYPES[case["dtype"] if case["kv"] == "same" else case["kv"]].itemsize
    return {"bytes": int(seen * case["kv_heads"] * 4 * d * wide + rows * case["heads"] * 4 * d * DTYPES[case["dtype"]].itemsize
                         + 4 * (_pages(lens).sum() + case["seqs"])),
            "flops": int(seen * case["heads"] * 12 * d * rows / case["seqs"])}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_diff(s)


def _exact_append(s):
    """Each stored value: the quotient in 64 bits, rounded once to the cache's type (half to even)."""
    done = {}
    for name, x, cache, scale in (("key_cache", s["key"], s["key_cache"], s["k_scale"]),
                                  ("value_cache", s["value"], s["value_cache"], s["v_scale"])):
        c = cache.double()
        x = x.double() / (scale if s["kv_dtype"] else 1.0)
        if s["kv_dtype"]:
            bits, least = {"e4m3": (3, -6), "e5m2": (2, -14)}[s["kv_dtype"]]
            step = torch.exp2(((torch.frexp(x).exponent - 1).clamp(min=least) - bits).double())
            x = (torch.round(x / step) * step).clamp(-FP8_MAX[s["kv_dtype"]], FP8_MAX[s["kv_dtype"]])
        rows = torch.nonzero(s["slots"] >= 0).flatten()
        slot = s["slots"][rows].long()
        if name == "value_cache" and s["layout"] == "split":
            tokens_first = c.permute(0, 3, 1, 2)                    # [block, off, head, d]
        elif s["layout"] == "split":
            tokens_first = c.permute(0, 3, 1, 2, 4)                 # [block, off, head, d/x, x]
        else:
            tokens_first = c.permute(0, 2, 1, 3)
        tokens_first[slot // BLOCK, slot % BLOCK] = x[rows].reshape((len(rows),) + tuple(tokens_first.shape[2:]))
        done[name] = c
    return done


def _exact_diff(s):
    """Sequence by sequence and map by map, in 64 bits."""
    lens = s["seq_lens"].tolist()
    start = list(range(len(lens) + 1)) if s["query_start"] is None else s["query_start"].tolist()
    h, d, hk = s["query"].shape[1], s["query"].shape[3], s["num_kv_heads"]
    answer = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["out"].device)
    for i, length in enumerate(lens):
        pages = s["block_tables"][i, :_pages(length)].long()
        k8, v8 = s["key_cache"], s["value_cache"]
        if s["kv_dtype"]:
            k = k8.view(torch.uint8)[pages].view(k8.dtype).double() * s["k_scale"]
            v = v8.view(torch.uint8)[pages].view(v8.dtype).double() * s["v_scale"]
        else:
            k, v = k8[pages].double(), v8[pages].double()
        if s["layout"] == "split":
            k = k.permute(0, 3, 1, 2, 4).reshape(len(pages) * BLOCK, 2 * hk, d)[:length]
            v = v.permute(0, 3, 1, 2).reshape(len(pages) * BLOCK, hk, 2 * d)[:length]
        else:
            k = k.permute(0, 2, 1, 3).reshape(len(pages) * BLOCK, 2 * hk, d)[:length]
            v = v.permute(0, 2, 1, 3).reshape(len(pages) * BLOCK, hk, 2 * d)[:length]
        for r in range(start[i], start[i + 1]):
            last = length - (start[i + 1] - r)
            low = max(0, last - s["window_left"]) if s["window_left"] >= 0 else 0
            t = torch.arange(low, last + 1, device=k.device)
            maps = []
            for c in (0, 1):
                q = s["query"][r, :, c].double().reshape(hk, h // hk, d)
                z = torch.matmul(q, k[low:last + 1, c::2].permute(1, 2, 0)) * s["scale"]   # [hk, g, t]
                if s["softcap"] > 0:
                    z = s["softcap"] * torch.tanh(z / s["softcap"])
                if s["alibi_slopes"] is not None:
                    z = z + s["alibi_slopes"].double().reshape(hk, h // hk, 1) * t
                maps.append(torch.matmul(torch.softmax(z, -1), v[low:last + 1].permute(1, 0, 2)))
            o = (maps[0] - s["lambdas"].double().reshape(hk, h // hk, 1) * maps[1]).reshape(h, 2 * d)
            if s["norm"]:
                o = o / torch.sqrt(o.square().mean(-1, keepdim=True) + s["norm_eps"]) * s["norm_weight"].double()
            answer[r] = o * s["out_scale"]
    return answer
