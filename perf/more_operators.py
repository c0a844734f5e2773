"""The operators of a cache that is short of room, as cases to be measured: fewer bits per token, fewer tokens.

  append   the step's keys and values into a 4-bit cache (e2m1 codes, an e4m3 scale for every 16 of them)
  decode   paged decode attention over a 4-bit cache
  weights  the attention weights of a step added to the score of every cached token
  select   the tokens that stay within a budget: the first, the last, and those with the largest scores
  compact  the keys, values and scores of those tokens moved to the front of their sequence's pages

`run` computes the plain form of an operator, in elementary torch operations, or with `own` calls the framework's.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16,
          "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "e2m1": torch.uint8}
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
DEVICE = "cuda"
# scales of 4-bit caches of values about 1: their largest over 6 * 448, as numbers of 32 bits
K_SCALE, V_SCALE = float(np.float32(0.0019)), float(np.float32(0.0023))


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the new token of a 32-sequence decode batch, both caches: latency
        dict(name="append decode 32 f16", op="append", tokens=32, run=1, heads=4, size=128, dtype="f16", fused=True),
        # a whole prompt: bandwidth
        dict(name="append prompt bf16", op="append", tokens=32768, run=32768, heads=8, size=128, dtype="bf16", fused=True),
        # two short sequences: latency
        dict(name="decode tiny f16", op="decode", seqs=2, longest=600, equal=False, heads=4, kv_heads=2, size=64,
             dtype="f16", tokens=1, softcap=0.0, alibi=False, window=-1),
        # the 32 x 4096 decode batch, groups of seven heads
        dict(name="decode 32x4096 f16", op="decode", seqs=32, longest=4096, equal=True, heads=28, kv_heads=4, size=128,
             dtype="f16", tokens=1, softcap=0.0, alibi=False, window=-1),
        # long contexts: 4 x 100000
        dict(name="decode long 4x100000 bf16", op="decode", seqs=4, longest=100000, equal=True, heads=28, kv_heads=4,
             size=128, dtype="bf16", tokens=1, softcap=0.0, alibi=False, window=-1),
        # two short sequences in fp32: latency
        dict(name="weights tiny f32", op="weights", seqs=2, longest=600, equal=False, heads=4, kv_heads=2, size=64,
             dtype="f32", kv="same", layout="nhd", tokens=1, softcap=0.0, alibi=False, window=-1, decay=1.0),
        # a decode step's weights, fp16, split layout
        dict(name="weights 32x4096 f16", op="weights", seqs=32, longest=4096, equal=True, heads=28, kv_heads=4, size=128,
             dtype="f16", kv="same", layout="split", tokens=1, softcap=0.0, alibi=False, window=-1, decay=1.0),
        # long contexts over a 4-bit cache, scores that fade
        dict(name="weights long 4x100000 e2m1", op="weights", seqs=4, longest=100000, equal=True, heads=28, kv_heads=4,
             size=128, dtype="bf16", kv="e2m1", layout="nhd", tokens=1, softcap=0.0, alibi=False, window=-1, decay=0.98),
        # a batch that has grown past its budget by four pages
        dict(name="select 32x4096", op="select", seqs=32, longest=4096, equal=True, kv_heads=4, budget=4032, sink=4,
             recent=256),
        # long contexts cut to a twelfth
        dict(name="select long 4x100000", op="select", seqs=4, longest=100000, equal=True, kv_heads=4, budget=8192,
             sink=16, recent=1024),
        # the same growth, fp16 in the split layout: nearly every token moves by some places
        dict(name="compact 32x4096 f16", op="compact", seqs=32, longest=4096, equal=True, k_heads=4, k_size=128,
             v_heads=4, v_size=128, dtype="f16", layout="split", budget=4032, sink=4, recent=256),
        # prompts cut to 2048 tokens each: one in eight stays
        dict(name="compact prompts 32x16384 bf16", op="compact", seqs=32, longest=16384, equal=True, k_heads=8, k_size=128,
             v_heads=8, v_size=128, dtype="bf16", layout="nhd", budget=2048, sink=4, recent=64),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "weights", "weights", "select", "compact"])
    heads = rng.choice([1, 2, 4, 8])
    size = rng.choice([64, 128, 128])
    if op == "append":
        tokens = _spread(rng, 1, 32768)
        return dict(op=op, tokens=tokens, run=_spread(rng, 1, tokens), heads=heads, size=size,
                    dtype=rng.choice(["f16", "bf16"]), fused=rng.random() < 0.5)
    if op in ("select", "compact"):
        longest = _spread(rng, 20, 65536)
        budget = max(1, int(longest * rng.choice([0.05, 0.25, 0.5, 0.9, 0.99])))
        both = dict(longest=longest, equal=rng.random() < 0.5, budget=budget, sink=rng.choice([0, 4, 16]),
                    recent=rng.choice([0, 16, 1 + budget // 8]))
        if op == "select":
            return dict(op=op, seqs=_spread(rng, 1, max(1, min(256, 3200000 // (longest * heads)))), kv_heads=heads, **both)
        dtype = rng.choice(["f32", "f16", "bf16", "e4m3", "e5m2", "e2m1"])
        twin = dtype != "e2m1" and size == 64 and rng.random() < 0.3  # differential heads: two key heads to a value head
        per = heads * 2 * size * DTYPES[dtype].itemsize * (2 if twin else 1)
        return dict(op=op, seqs=_spread(rng, 1, max(1, min(64, 250000000 // (longest * per)))),
                    k_heads=heads * (2 if twin else 1), k_size=size, v_heads=heads, v_size=size * (2 if twin else 1),
                    dtype=dtype, layout="nhd" if dtype == "e2m1" else rng.choice(["split", "nhd"]), **both)
    tokens = rng.choice([1, 1, 1, 2, 4])
    group = rng.choice([1, 2, 3, 4, 7, 8, 16]) if tokens == 1 else rng.choice([1, 2, 4])
    longest = _spread(rng, 1, 65536)
    seqs = _spread(rng, 1, max(1, min(128, 1600000 // (longest * heads))))
    case = dict(op=op, seqs=seqs, longest=longest, equal=rng.random() < 0.5, heads=group * heads, kv_heads=heads,
                size=size, dtype=rng.choice(["f16", "bf16"]), tokens=tokens, softcap=rng.choice([0.0, 0.0, 30.0]),
                alibi=rng.random() < 0.3, window=rng.choice([-1, -1, -1, 1000]))
    if op == "decode":
        return case
    kv = rng.choice(["same", "same", "e4m3", "e5m2", "e2m1"])
    if kv == "same":
        case["dtype"] = rng.choice(["f32", "f16", "bf16"])
        case["seqs"] = max(1, seqs // 2) if case["dtype"] == "f32" else seqs
    return dict(case, kv=kv, layout="nhd" if kv == "e2m1" else rng.choice(["split", "nhd"]),
                decay=rng.choice([1.0, 1.0, 0.9, 0.0]))


def _lengths(case):
    """The batch's lengths but for their order: all the longest, or spread over their logarithm."""
    n, top = case["seqs"], case["longest"]
    if case["equal"]:
        return np.full(n, top, dtype=np.int64)
    return np.clip(np.round(top ** ((np.arange(n) + 1) / n)), 1, top).astype(np.int64)


def _pages(n):
    return (n + BLOCK - 1) // BLOCK


def _tokens_of(case, lens):
    """New tokens of each sequence: between one and the most that one has."""
    return np.minimum(1 + np.arange(case["seqs"]) % case["tokens"], lens)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    torch.cuda.set_device(0)
    rng = np.random.default_rng([seed, 17])
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed * 13 + 5)
    make = {"append": _prepare_append, "decode": _prepare_attention, "weights": _prepare_attention,
            "select": _prepare_select, "compact": _prepare_compact}
    return make[case["op"]](case, rng, gen)


def _int(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEVICE)


def _normal(shape, dtype, gen, scale=1.0):
    t = torch.empty(shape, dtype=dtype if dtype.itemsize > 1 else torch.float16, device=DEVICE)
    t.normal_(generator=gen)
    if scale != 1.0:
        t.mul_(1.0 / scale)
    return t if t.dtype == dtype else t.to(dtype)


def _codes(shape, gen, scale):
    """A 4-bit cache of normal values, [blocks, heads, 9 * size] bytes (codes near enough to the nearest)."""
    blocks, heads, size = shape
    cache = torch.empty((blocks, heads, 9 * size), dtype=torch.uint8, device=DEVICE)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEVICE)
    step = max(1, (1 << 24) // (heads * BLOCK * size))
    for a in range(0, blocks, step):
        c = cache[a:a + step]
        x = torch.randn((c.shape[0], heads, BLOCK, size // 16, 16), generator=gen, device=DEVICE)
        s = (x.abs().amax(-1) / (6.0 * scale)).clamp(max=448.0).to(torch.float8_e4m3fn)
        code = torch.bucketize(x.abs() / (s.float().unsqueeze(-1) * scale), edges, out_int32=True).to(torch.uint8)
        code |= (x < 0).to(torch.uint8) << 3
        code = code.flatten(3).unflatten(3, (size // 2, 2))
        c[:, :, :8 * size] = (code[..., 0] | code[..., 1] << 4).flatten(2)
        c[:, :, 8 * size:] = s.view(torch.uint8).flatten(2)
    return cache


def _cache_shapes(blocks, k_heads, k_size, v_heads, v_size, layout, width):
    if layout == "nhd":
        return (blocks, k_heads, BLOCK, k_size), (blocks, v_heads, BLOCK, v_size)
    x = 16 // width
    return (blocks, k_heads, k_size // x, BLOCK, x), (blocks, v_heads, v_size, BLOCK)


def _table(lens, width, rng):
    """Block table of sequences of these lengths and the number of pages of the cache, three of them spare."""
    owned = _pages(lens)
    blocks = int(owned.sum()) + 3
    ids = rng.permutation(blocks)
    table = np.zeros((len(lens), width), dtype=np.int64)
    table[np.arange(width)[None, :] < owned[:, None]] = ids[:owned.sum()]
    return _int(table), blocks


def _prepare_append(case, rng, gen):
    tokens, h, d, dtype = case["tokens"], case["heads"], case["size"], DTYPES[case["dtype"]]
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
    if case["fused"]:  # keys and values as the projection leaves them, beside the queries
        row = _normal((tokens, 4 * h * d), dtype, gen)
        key = row[:, 2 * h * d:3 * h * d].unflatten(1, (h, d))
        value = row[:, 3 * h * d:].unflatten(1, (h, d))
    else:
        key, value = _normal((tokens, h, d), dtype, gen), _normal((tokens, h, d), dtype, gen)
    old = lambda: torch.randint(0, 256, (blocks, h, 9 * d), generator=gen, device=DEVICE, dtype=torch.uint8)  # noqa: E731
    return dict(op="append", key=key, value=value, slots=_int(slots), key_cache=old(), value_cache=old(),
                k_scale=K_SCALE, v_scale=V_SCALE)


def _prepare_attention(case, rng, gen):
    n, h, hk, d = case["seqs"], case["heads"], case["kv_heads"], case["size"]
    weights = case["op"] == "weights"
    dtype, kv = DTYPES[case["dtype"]], case["kv"] if weights else "e2m1"
    order = rng.permutation(n)
    lens = _lengths(case)
    new = _tokens_of(case, lens)[order]
    lens = lens[order]
    table, blocks = _table(lens, _pages(case["longest"]), rng)
    rows = int(new.sum())
    layout = case["layout"] if weights else "nhd"
    scale = {"same": 1.0, "e2m1": K_SCALE}.get(kv, 2.0 ** -6)
    ks, vs = _cache_shapes(blocks, hk, d, hk, d, layout, DTYPES[case["dtype"] if kv == "same" else kv].itemsize)
    fill = lambda shape: (_codes((blocks, hk, d), gen, scale) if kv == "e2m1" else  # noqa: E731
                          _normal(shape, dtype if kv == "same" else DTYPES[kv], gen, scale))
    parts = max(1, -(-case["longest"] // 512))
    real = lambda *shape: torch.empty(shape, dtype=torch.float32, device=DEVICE)  # noqa: E731
    s = dict(
        op=case["op"], query=_normal((rows, h, d), dtype, gen), key_cache=fill(ks), block_tables=table, seq_lens=_int(lens),
        query_start=_int(np.concatenate([[0], np.cumsum(new)])) if case["tokens"] > 1 else None,
        max_query_len=case["tokens"], num_kv_heads=hk, scale=1.0 / math.sqrt(d), max_seq_len=case["longest"],
        softcap=case["softcap"], window_left=case["window"],
        alibi_slopes=torch.tensor([2.0 ** (-8.0 * (i + 1) / h) for i in range(h)], device=DEVICE) if case["alibi"] else None,
        layout=layout, kv_dtype=None if kv == "same" else kv, k_scale=scale)
    if not weights:
        s.update(out=torch.empty((rows, h, d), dtype=dtype, device=DEVICE), value_cache=fill(vs), v_scale=scale,
                 seq_lens_host=lens.astype(np.int32), exp_sums=real(rows, h, parts), max_logits=real(rows, h, parts),
                 tmp_out=real(rows, h, parts, d),
                 partition_counters=torch.zeros((n, hk), dtype=torch.int32, device=DEVICE),
                 tile_counters=torch.zeros(2, dtype=torch.int32, device=DEVICE))
        return s
    # what the decode call before has left: its statistics; and the scores of the steps before
    z, seen, owner, index = _logits(s)
    room = parts * 512 - z.shape[-1]
    z = torch.nn.functional.pad(z.masked_fill(~seen[:, :, None, None, :], float("-inf")), (0, room), value=float("-inf"))
    z = z.unflatten(-1, (parts, 512))
    most = z.amax(-1)
    sums = torch.exp(z - most.masked_fill(most == float("-inf"), 0.0).unsqueeze(-1)).sum(-1)
    del z
    s.update(max_logits=most.flatten(2, 3)[owner, index].float().contiguous(),
             exp_sums=sums.flatten(2, 3)[owner, index].float().contiguous(), decay=case["decay"],
             # what eight such steps would leave
             scores=torch.rand((blocks, hk, BLOCK), generator=gen, device=DEVICE).mul_(16.0 * h / hk / case["longest"]))
    return s


def _prepare_select(case, rng, gen):
    n, hk = case["seqs"], case["kv_heads"]
    lens = rng.permutation(_lengths(case))
    table, blocks = _table(lens, _pages(case["longest"]), rng)
    # sums of weights: few tokens hold most of them, many are nearly the same; some ties
    scores = torch.rand((blocks, hk, BLOCK), generator=gen, device=DEVICE).pow_(4)
    tie = torch.rand((blocks, hk, BLOCK), generator=gen, device=DEVICE) < 0.02
    scores.masked_fill_(tie, 0.015625)
    return dict(op="select", scores=scores, block_tables=table, seq_lens=_int(lens), max_seq_len=case["longest"],
                budgets=torch.full((n,), case["budget"], dtype=torch.int32, device=DEVICE), sink=case["sink"],
                recent=case["recent"], new_seq_lens=torch.empty(n, dtype=torch.int32, device=DEVICE),
                kept=torch.full((n, hk, case["budget"]), -1, dtype=torch.int32, device=DEVICE))


def _prepare_compact(case, rng, gen):
    n, hk, top, budget = case["seqs"], case["v_heads"], case["longest"], case["budget"]
    lens = rng.permutation(_lengths(case))
    table, blocks = _table(lens, _pages(top), rng)
    dtype, layout = DTYPES[case["dtype"]], case["layout"]
    ks, vs = _cache_shapes(blocks, case["k_heads"], case["k_size"], hk, case["v_size"], layout, dtype.itemsize)
    fill = lambda shape, size: (_codes((blocks, hk, size), gen, K_SCALE) if case["dtype"] == "e2m1" else  # noqa: E731
                                _normal(shape, dtype, gen))
    # a choice as the selection makes it: the first and the last tokens, and some of those between
    live = torch.from_numpy(lens).to(DEVICE)[:, None, None]
    t = torch.arange(top, device=DEVICE)
    rank = torch.rand((n, hk, top), generator=gen, device=DEVICE)
    rank = torch.where((t < case["sink"]) | (t >= live - case["recent"]), 2.0, rank)
    rank = torch.where(t >= live, -1.0, rank)
    kept = torch.topk(rank, budget, dim=-1).indices
    kept = torch.where(torch.arange(budget, device=DEVICE) < live, kept, top).sort(-1).values
    kept = torch.where(kept < top, kept, -1).int()
    return dict(op="compact", key_cache=fill(ks, case["k_size"]), value_cache=fill(vs, case["v_size"]),
                scores=torch.rand((blocks, hk, BLOCK), generator=gen, device=DEVICE), block_tables=table, kept=kept,
                new_seq_lens=_int(np.minimum(lens, budget)), layout=layout,
                kv_dtype=case["dtype"] if case["dtype"] in ("e4m3", "e5m2", "e2m1") else None)


# ------------------------------------------------------------------ passes

def run(state):
    if own:
        return {"append": _own_append, "decode": _own_decode, "weights": _own_weights, "select": _own_select,
                "compact": _own_compact}[state["op"]](state)
    return {"append": _plain_append, "decode": _plain_decode, "weights": _plain_weights, "select": _plain_select,
            "compact": _plain_compact}[state["op"]](state)


def _own_append(s):
    import paged_kv_attention_v2_gb300 as pa
    pa.pa_append_kv(s["key"], s["value"], s["key_cache"], s["value_cache"], s["slots"], layout="nhd", kv_dtype="e2m1",
                    k_scale=s["k_scale"], v_scale=s["v_scale"])
    return {"key_cache": s["key_cache"], "value_cache": s["value_cache"]}


def _several(s):
    return dict(query_start=s["query_start"], max_query_len=s["max_query_len"]) if s["query_start"] is not None else {}


def _own_decode(s):
    import paged_kv_attention_v2_gb300 as pa
    pa.pa_decode(s["out"], s["query"], s["key_cache"], s["value_cache"], s["block_tables"], s["seq_lens"],
                 num_kv_heads=s["num_kv_heads"], scale=s["scale"], max_seq_len=s["max_seq_len"], softcap=s["softcap"],
                 alibi_slopes=s["alibi_slopes"], window_left=s["window_left"], layout="nhd", kv_dtype="e2m1",
                 k_scale=s["k_scale"], v_scale=s["v_scale"], seq_lens_host=s["seq_lens_host"], exp_sums=s["exp_sums"],
                 max_logits=s["max_logits"], tmp_out=s["tmp_out"], partition_counters=s["partition_counters"],
                 tile_counters=s["tile_counters"], **_several(s))
    return s["out"]


def _own_weights(s):
    import paged_kv_attention_v2_gb300 as pa
    pa.pa_add_weights(s["scores"], s["query"], s["key_cache"], s["block_tables"], s["seq_lens"], s["exp_sums"],
                      s["max_logits"], num_kv_heads=s["num_kv_heads"], scale=s["scale"], max_seq_len=s["max_seq_len"],
                      decay=s["decay"], softcap=s["softcap"], alibi_slopes=s["alibi_slopes"],
                      window_left=s["window_left"], layout=s["layout"], kv_dtype=s["kv_dtype"], k_scale=s["k_scale"],
                      **_several(s))
    return s["scores"]


def _own_select(s):
    import paged_kv_attention_v2_gb300 as pa
    pa.pa_select_tokens(s["kept"], s["new_seq_lens"], s["scores"], s["block_tables"], s["seq_lens"], s["budgets"],
                        max_seq_len=s["max_seq_len"], sink=s["sink"], recent=s["recent"])
    return {"kept": s["kept"], "new_seq_lens": s["new_seq_lens"]}


def _own_compact(s):
    import paged_kv_attention_v2_gb300 as pa
    pa.pa_compact_kv(s["key_cache"], s["value_cache"], s["block_tables"], s["kept"], s["new_seq_lens"], scores=s["scores"],
                     layout=s["layout"], kv_dtype=s["kv_dtype"])
    return {"key_cache": s["key_cache"], "value_cache": s["value_cache"], "scores": s["scores"]}


def _e4m3(x):
    """Numbers of 64 bits, none negative, rounded once to e4m3 (half to even), still in 64 bits."""
    step = torch.exp2(((torch.frexp(x).exponent - 1).clamp(min=-6) - 3).double())
    return (torch.round(x / step) * step).clamp(max=448.0)


def _plain_store4(x, cache, slots, scale):
    """Codes and scales are compared as they are stored, so both quotients are taken in 64 bits: next to the border
    between two codes 32 lose which side a value is on."""
    d = x.shape[-1]
    x = x.unflatten(-1, (d // 16, 16)).double()
    s = _e4m3(x.abs().amax(-1) / (6.0 * scale))
    y = x.abs() / (s * scale).unsqueeze(-1)
    code = torch.zeros(y.shape, dtype=torch.uint8, device=y.device)
    code += y > 0.25
    code += y >= 0.75
    code += y > 1.25
    code += y >= 1.75
    code += y > 2.5
    code += y >= 3.5
    code += y > 5.0
    code |= torch.signbit(x).to(torch.uint8) << 3
    code = torch.where(s.unsqueeze(-1) == 0, 0, code).to(torch.uint8).flatten(-2).unflatten(-1, (d // 2, 2))
    # a row without a slot stores the first row that has one again
    there = slots >= 0
    row = torch.where(there, torch.arange(slots.shape[0], device=DEVICE), there.int().argmax())
    blk, off = slots[row].long() // BLOCK, slots[row].long() % BLOCK
    cache[:, :, :8 * d].unflatten(2, (BLOCK, d // 2))[blk, :, off] = (code[..., 0] | code[..., 1] << 4)[row]
    cache[:, :, 8 * d:].unflatten(2, (BLOCK, d // 16))[blk, :, off] = s.float().to(torch.float8_e4m3fn).view(torch.uint8)[row]
    return cache


def _plain_append(s):
    return {"key_cache": _plain_store4(s["key"], s["key_cache"], s["slots"], s["k_scale"]),
            "value_cache": _plain_store4(s["value"], s["value_cache"], s["slots"], s["v_scale"])}


def _gathered(cache, table, layout, kv, scale, is_key, tokens):
    """The cache's rows of each sequence in order: [sequences, heads, tokens, size], 32 bits."""
    if kv == "e2m1":
        p = cache[table]                                                  # [s, page, head, 9 d]
        d = p.shape[-1] // 9
        c, f = p[..., :8 * d].unflatten(-1, (BLOCK, d // 2)), p[..., 8 * d:].contiguous().view(torch.float8_e4m3fn).float()
        level = torch.tensor(LEVELS + [-v for v in LEVELS], device=p.device)
        p = torch.stack([level[(c & 15).int()], level[(c >> 4).int()]], -1).flatten(-2)
        p = p.unflatten(-1, (d // 16, 16)) * (f * scale).unflatten(-1, (BLOCK, d // 16)).unsqueeze(-1)
        p = p.flatten(-2).transpose(1, 2)
        return p.reshape(p.shape[0], p.shape[1], -1, d)[:, :, :tokens]
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


def _logits(s):
    """Logits [sequences, queries, kv heads, group, tokens], which of them count, and where each query row is. Those with
    ALiBi in 64 bits: far positions."""
    q, table, lens = s["query"].float(), s["block_tables"].long(), s["seq_lens"].long()
    n, hk, longest, device = table.shape[0], s["num_kv_heads"], s["max_seq_len"], q.device
    rows, h, d = q.shape
    g, most = h // hk, s["max_query_len"]
    # the queries of a sequence side by side, padded to the most that one has
    if s["query_start"] is None:
        owner, index, count = torch.arange(n, device=device), torch.zeros(n, dtype=torch.long, device=device), torch.ones_like(lens)
    else:
        start = s["query_start"].long()
        owner = torch.searchsorted(start[1:], torch.arange(rows, device=device), right=True)
        index = torch.arange(rows, device=device) - start[owner]
        count = start[1:] - start[:-1]
    many = torch.zeros((n, most, h, d), device=device)
    many[owner, index] = q
    pos = (lens - count)[:, None] + torch.arange(most, device=device)[None, :]
    keys = _gathered(s["key_cache"], table, s["layout"], s["kv_dtype"], s["k_scale"], True, longest)
    z = torch.einsum("nmkgd,nktd->nmkgt", many.unflatten(2, (hk, g)), keys) * s["scale"]
    if s["softcap"] > 0:
        z = s["softcap"] * torch.tanh(z / s["softcap"])
    t = torch.arange(longest, device=device)
    if s["alibi_slopes"] is not None:
        z = z.double() + s["alibi_slopes"].double().view(hk, g)[:, :, None] * t
    seen = (t <= pos[:, :, None]) & (t < lens[:, None, None]) & \
        (torch.arange(most, device=device)[:, None] < count[:, None, None])
    if s["window_left"] >= 0:
        seen = seen & (t >= pos[:, :, None] - s["window_left"])
    return z, seen, owner, index


def _plain_decode(s):
    z, seen, owner, index = _logits(s)
    seen = seen[:, :, None, None, :]
    z = z.masked_fill(~seen, float("-inf"))
    z = torch.exp(z - z.amax(-1, keepdim=True)).masked_fill(~seen, 0.0).float()
    z = z / z.sum(-1, keepdim=True)
    values = _gathered(s["value_cache"], s["block_tables"].long(), "nhd", "e2m1", s["v_scale"], False, s["max_seq_len"])
    s["out"].copy_(torch.einsum("nmkgt,nktd->nmkgd", z, values).flatten(2, 3)[owner, index])
    return s["out"]


def _plain_weights(s):
    z, seen, owner, index = _logits(s)
    hk, lens, t = s["num_kv_heads"], s["seq_lens"].long(), torch.arange(s["max_seq_len"], device=DEVICE)
    # each row's maximum and sum, from those of its partitions
    part = s["max_logits"].double()
    most = part.amax(-1)
    total = (s["exp_sums"].double() * torch.exp(part - most.unsqueeze(-1))).sum(-1)
    level = torch.zeros(z.shape[:4], dtype=torch.float64, device=DEVICE)
    level[owner, index] = (most + total.log()).unflatten(-1, (hk, -1))
    w = torch.exp(z - (level if z.dtype == torch.float64 else level.float()).unsqueeze(-1))
    w = w.masked_fill(~seen[:, :, None, None, :], 0.0).sum((1, 3)).float()           # [sequences, kv heads, tokens]
    blk = s["block_tables"].long()[:, t // BLOCK]
    at = lambda: (blk[:, None, :], torch.arange(hk, device=DEVICE)[None, :, None], (t % BLOCK)[None, None, :])  # noqa: E731
    old = s["scores"][at()]
    count = 1 if s["query_start"] is None else (s["query_start"][1:] - s["query_start"][:-1]).long()
    fresh = (t >= (lens - count)[:, None])[:, None, :] if s["decay"] != 0 else torch.ones_like(w, dtype=torch.bool)
    w = torch.where(fresh, w, s["decay"] * old + w)
    # places behind a sequence's end go to the first token again
    live = (t < lens[:, None])[:, None, :]
    b, h, o = (x.expand(w.shape) for x in at())
    first = lambda x: torch.where(live, x, x[:, :, :1])  # noqa: E731
    s["scores"][first(b), first(h), first(o)] = first(w)
    return s["scores"]


def _plain_select(s):
    hk, lens, longest = s["kept"].shape[1], s["seq_lens"].long(), s["max_seq_len"]
    t = torch.arange(longest, device=DEVICE)
    score = s["scores"][s["block_tables"].long()[:, None, t // BLOCK], torch.arange(hk, device=DEVICE)[None, :, None],
                        t % BLOCK]
    budget = s["budgets"].long()
    recent = budget.clamp(max=s["recent"])
    sink = (budget - recent).clamp(max=s["sink"])
    live, new = lens[:, None, None], torch.minimum(lens, budget)
    always = (t < sink[:, None, None]) | (t >= live - recent[:, None, None]) | (lens <= budget)[:, None, None]
    score = score.masked_fill(always, float("inf")).masked_fill(t >= live, float("-inf"))
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[:, :, :s["kept"].shape[2]]
    i = torch.arange(order.shape[2], device=DEVICE)
    order = torch.where(i < new[:, None, None], order, longest).sort(-1).values
    s["kept"][:, :, :order.shape[2]] = torch.where(order < longest, order, s["kept"][:, :, :order.shape[2]]).int()
    s["new_seq_lens"].copy_(new)
    return {"kept": s["kept"], "new_seq_lens": s["new_seq_lens"]}


def _moved(cache, src, dst, ratio, layout, kv):
    """Rows of the cache from the places `src` (page, head, slot) to `dst`, all read before any is written."""
    if kv == "e2m1":
        d = cache.shape[-1] // 9
        views = [cache[:, :, :8 * d].unflatten(2, (BLOCK, d // 2)), cache[:, :, 8 * d:].unflatten(2, (BLOCK, d // 16))]
    else:
        views = [cache.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[cache.element_size()])]
    heads = torch.arange(ratio, device=DEVICE)
    for c in views:
        (sb, sh, so), (db, dh, do) = (tuple((x[0][..., None], x[1][..., None] * ratio + heads, x[2][..., None])) for x in (src, dst))
        if layout == "nhd":
            c[db, dh, do] = c[sb, sh, so]
        else:
            c[db, dh, :, do] = c[sb, sh, :, so]
    return cache


def _plain_compact(s):
    kept, table, new = s["kept"].long(), s["block_tables"].long(), s["new_seq_lens"].long()
    n, hk, most = kept.shape
    to = torch.arange(most, device=DEVICE)
    live = (to < new[:, None])[:, None, :]
    to = torch.where(live, to, 0).expand(kept.shape)
    kept = torch.where(live, kept, kept[:, :, :1])  # places behind the last token: the first one again
    seq, head = torch.arange(n, device=DEVICE)[:, None, None], torch.arange(hk, device=DEVICE)[None, :, None].expand(kept.shape)
    src, dst = ((table[seq, x // BLOCK], head, x % BLOCK) for x in (kept, to))
    _moved(s["key_cache"], src, dst, s["key_cache"].shape[1] // hk, s["layout"], s["kv_dtype"])
    _moved(s["value_cache"], src, dst, 1, s["layout"], s["kv_dtype"])
    s["scores"][dst] = s["scores"][src]
    return {"key_cache": s["key_cache"], "value_cache": s["value_cache"], "scores": s["scores"]}


# ------------------------------------------------------------------ bytes and operations

def work(case):
    op = case["op"]
    if op == "append":
        values = 2 * case["tokens"] * case["heads"] * case["size"]
        return {"bytes": int(values * (2 + 9 / 16) + 4 * case["tokens"]), "flops": values}
    lens = _lengths(case)
    if op in ("select", "compact"):
        hk = case["kv_heads"] if op == "select" else case["v_heads"]
        kept = np.minimum(lens, case["budget"])
        if op == "select":
            return {"bytes": int((lens.sum() + kept.sum()) * hk * 4), "flops": int(lens.sum() * hk)}
        # tokens in front of the first one that goes stay where they are: about one in (tokens that may go) / (those that do)
        gone = lens - kept
        stay = np.where(gone > 0, np.minimum(kept, case["sink"] + (lens - case["sink"]) / (gone + 1)), kept)
        wide = 2 * 9 / 16 * case["k_size"] if case["dtype"] == "e2m1" else \
            (case["k_heads"] // hk * case["k_size"] + case["v_size"]) * DTYPES[case["dtype"]].itemsize
        return {"bytes": int((kept - stay).sum() * hk * (2 * (wide + 4)) + kept.sum() * hk * 4), "flops": 0}
    new = _tokens_of(case, lens)
    rows, d, h, hk = int(new.sum()), case["size"], case["heads"], case["kv_heads"]
    size = DTYPES[case["dtype"]].itemsize
    seen = np.minimum(lens, case["window"] + new) if case["window"] >= 0 else lens
    seen, pages = int(seen.sum()), int(_pages(seen).sum())
    kv = case.get("kv", "e2m1")
    wide = 9 / 16 if kv == "e2m1" else DTYPES[case["dtype"] if kv == "same" else kv].itemsize
    if op == "decode":
        return {"bytes": int(2 * seen * hk * d * wide + 2 * rows * h * d * size + 4 * pages),
                "flops": int(4 * seen * h * d * rows / case["seqs"])}
    parts = -(-case["longest"] // 512)
    return {"bytes": int(seen * hk * d * wide + 8 * lens.sum() * hk + rows * h * (d * size + 8 * parts) + 4 * pages),
            "flops": int(2 * seen * h * d * rows / case["seqs"])}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """Codes, positions and moved bytes are whole or copied: nothing to compute. The others sequence by sequence."""
    if case["op"] not in ("decode", "weights"):
        return None
    s = prepare(case, seed)
    lens = s["seq_lens"].tolist()
    start = list(range(len(lens) + 1)) if s["query_start"] is None else s["query_start"].tolist()
    hk, (rows, h, d) = s["num_kv_heads"], s["query"].shape
    answer = torch.zeros((rows, h, d), dtype=torch.float64, device=DEVICE) if case["op"] == "decode" else s["scores"].double()
    for i, length in enumerate(lens):
        pages = s["block_tables"][i, :_pages(length)].long()
        k = _exact_rows(s["key_cache"], pages, s, s["k_scale"], length)
        added = torch.zeros((length, hk), dtype=torch.float64, device=DEVICE)
        for r in range(start[i], start[i + 1]):
            last = length - (start[i + 1] - r)
            low = max(0, last - s["window_left"]) if s["window_left"] >= 0 else 0
            q = s["query"][r].double().reshape(hk, h // hk, d)
            z = torch.matmul(q, k[low:last + 1].permute(1, 2, 0)) * s["scale"]                    # [hk, g, t]
            if s["softcap"] > 0:
                z = s["softcap"] * torch.tanh(z / s["softcap"])
            if s["alibi_slopes"] is not None:
                z = z + s["alibi_slopes"].double().reshape(hk, h // hk, 1) * torch.arange(low, last + 1, device=DEVICE)
            if case["op"] == "decode":
                v = _exact_rows(s["value_cache"], pages, s, s["v_scale"], length)[low:last + 1]
                answer[r] = torch.matmul(torch.softmax(z, -1), v.permute(1, 0, 2)).reshape(h, d)
            else:
                level = torch.logsumexp(s["max_logits"][r].double() + s["exp_sums"][r].double().log(), -1)
                added[low:last + 1] += torch.exp(z - level.reshape(hk, h // hk, 1)).sum(1).t()
        if case["op"] == "weights":
            t = torch.arange(length, device=DEVICE)
            old = answer[pages[t // BLOCK], :, t % BLOCK]
            faded = torch.where((t < length - (start[i + 1] - start[i]))[:, None], s["decay"] * old, 0.0) if s["decay"] != 0 else 0.0
            answer[pages[t // BLOCK], :, t % BLOCK] = faded + added
    return answer


def _exact_rows(cache, pages, s, scale, length):
    """Keys or values of one sequence, [tokens, heads, size], 64 bits."""
    if s["kv_dtype"] == "e2m1":
        p = cache[pages]
        n, hk, d = p.shape[0], p.shape[1], p.shape[2] // 9
        byte = p[:, :, :8 * d].reshape(n, hk, BLOCK, d // 2)
        x = torch.zeros((n, hk, BLOCK, d), dtype=torch.float64, device=DEVICE)
        for half in (0, 1):
            c = (byte >> (4 * half)) & 15
            e, m = ((c >> 1) & 3).double(), (c & 1).double()
            v = torch.where(e > 0, (1 + m / 2) * torch.exp2(e - 1), m / 2)
            x[..., half::2] = torch.where(c >= 8, -v, v)
        f = p[:, :, 8 * d:].contiguous().view(torch.float8_e4m3fn).double() * scale
        x = x * f.reshape(n, hk, BLOCK, d // 16).repeat_interleave(16, -1)
        return x.permute(0, 2, 1, 3).reshape(n * BLOCK, hk, d)[:length]
    p = cache.view(torch.uint8)[pages].view(cache.dtype) if cache.element_size() == 1 else cache[pages]
    p = p.double() * scale
    if s["layout"] == "nhd":
        return p.permute(0, 2, 1, 3).flatten(0, 1)[:length]
    return p.permute(0, 3, 1, 2, 4).flatten(0, 1).flatten(2)[:length]
