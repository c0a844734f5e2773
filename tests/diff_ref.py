"""Differential attention in 64 bits from the formula, and how far the kernel may
be from it, for the tests.

With a_t the softmax weights of one map and v_t the value rows, the kernel's o of
that map is off by at most
    E_j = sum_t a_t dz_t |v_tj| + A_j sum_t a_t dz_t + A_j (u_p + u_s),   A_j = sum_t a_t |v_tj|
where
  dz_t  is the error of a logit: products of the inputs are exact (16-bit, fp8) or
        good to 2^-21 (fp32 in three tf32 terms); the tensor core sums them in groups
        of at most 16 and the d / 8 group sums (at most) are added, with a step 2^-23
        of sum |q k| lost each; softcap, scale and ALiBi take a few roundings of their
        own results:  2^-23 ((d / 8 + 24) S_t + 4 cap + 4 |bias_t|), S_t = scale sum |q k|,
        and a bf16 query against fp8 keys goes through fp16 (2^-25 below its normal range)
  u_p   is half a step of a softmax weight as the P.V operand: 2^-21 (fp16 in two
        terms; and an absolute 2^-25 where it is subnormal, against a sum of at least
        one), 2^-11 (a bf16 query over an fp8 cache: fp16 in one), 2^-17 (bf16 in two
        terms), 2^-21 (fp32 in three tf32 terms)
  u_s   is the summation over n tokens, in pages of 16 and one merge per partition,
        with a step 2^-23 for each: 2^-23 (n / 16 + 64)
and y = s w o / r, r = sqrt(mean o^2 + eps), by
    |dy_j| <= s |w_j| / r (E_j + |o_j| / r rms(E)) + half a step of the output,
of which the second-order terms are covered by a factor 1.1.
"""
from __future__ import annotations

import numpy as np
import torch

BS, PART = 16, 512
U_P = {"f16": 2.0 ** -21, "bf16": 2.0 ** -17, "f32": 2.0 ** -21, "bf16 over fp8": 2.0 ** -11}
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def logical(cache, table, length, layout, is_key, kv):
    """[tokens, heads, size] in 64 bits of one sequence (torch cache on the CPU)."""
    pages = torch.as_tensor(np.asarray(table[:-(-length // BS)], dtype=np.int64))
    if kv is not None:
        cache = cache.view(torch.uint8)[pages].view(FP8[kv])
    else:
        cache = cache[pages]
    c = cache.double()
    if layout == "nhd":
        c = c.permute(0, 2, 1, 3)
    elif is_key:
        c = c.permute(0, 3, 1, 2, 4).flatten(3)
    else:
        c = c.permute(0, 3, 1, 2)
    return c.reshape(-1, c.shape[2], c.shape[3])[:length].numpy()


def diff_ref(case, part=PART):
    """out, tol [rows, heads, 2d]; max_logits, exp_sums [rows, heads, 2, P] in 64 bits."""
    q = case["query"].double().numpy()
    rows, heads, _, d = q.shape
    g = heads // case["kv_heads"]
    parts = max(1, -(-case["max_seq_len"] // part))
    out, tol = np.zeros((rows, heads, 2 * d)), np.zeros((rows, heads, 2 * d))
    ml = np.full((rows, heads, 2, parts), -np.inf)
    es = np.zeros((rows, heads, 2, parts))
    start = case["start"] if case["start"] is not None else np.arange(len(case["lens"]) + 1)
    lam = case["lambdas"].double().numpy()
    w = np.ones(2 * d) if case["norm_weight"] is None else case["norm_weight"].double().numpy()
    dtype, kv = case["dtype"], case["kv"]
    pdt = "bf16 over fp8" if kv and dtype == "bf16" else dtype
    cap, scale = case["softcap"], float(np.float32(case["scale"]))
    for s, length in enumerate(case["lens"]):
        length = int(min(max(length, 0), case["max_seq_len"]))
        if not length:
            continue
        k = logical(case["key_cache"], case["table"][s], length, case["layout"], True, kv) * np.float32(case["k_scale"])
        v = logical(case["value_cache"], case["table"][s], length, case["layout"], False, kv) * np.float32(case["v_scale"])
        n_q = int(start[s + 1] - start[s])
        for i in range(n_q):
            r, pos = int(start[s]) + i, length - n_q + i
            lo = max(0, pos - case["window"]) if case["window"] >= 0 else 0
            if pos < 0:
                continue
            t = np.arange(lo, pos + 1)
            for h in range(heads):
                o, err = [], []
                vv = v[lo:pos + 1, h // g]
                for m in (0, 1):
                    kk = k[lo:pos + 1, 2 * (h // g) + m]
                    z = scale * (kk @ q[r, h, m])
                    big = abs(scale) * (np.abs(kk) @ np.abs(q[r, h, m]))
                    dz = 2.0 ** -23 * ((d / 8 + 24) * big + 4 * cap)
                    if kv and dtype == "bf16":
                        dz += 2.0 ** -25 * abs(scale) * np.abs(kk).sum(1)
                    if cap > 0:
                        z = cap * np.tanh(z / cap)
                    if case["alibi"] is not None:
                        bias = float(case["alibi"][h]) * t
                        z = z + bias
                        dz = dz + 2.0 ** -21 * np.abs(bias - bias[-1])
                    zmax = z.max()
                    a = np.exp(z - zmax)
                    total = a.sum()
                    a /= total
                    for p in range(lo // part, pos // part + 1):
                        zp = z[(t // part) == p]
                        ml[r, h, m, p], es[r, h, m, p] = zp.max(), np.exp(zp - zp.max()).sum()
                    av = a @ np.abs(vv)
                    o.append(a @ vv)
                    e = (a * dz) @ np.abs(vv) + av * (a * dz).sum() + av * (U_P[pdt] + 2.0 ** -23 * (len(t) / 16 + 64))
                    if kv or dtype == "f16":
                        e = e + 2.0 ** -25 * np.abs(vv).sum(0)
                    err.append(e)
                f = lam[r, h] if lam.ndim == 2 else lam[h]
                x, e = o[0] - f * o[1], err[0] + abs(f) * err[1] + 2.0 ** -23 * (np.abs(o[0]) + abs(f) * np.abs(o[1]))
                if case["norm"]:
                    rms = np.sqrt((x * x).mean() + case["eps"])
                    y = case["out_scale"] * w * x / rms
                    dy = abs(case["out_scale"]) * np.abs(w) / rms * (e + np.abs(x) / rms * np.sqrt((e * e).mean()))
                else:
                    y, dy = case["out_scale"] * x, abs(case["out_scale"]) * e
                out[r, h] = y
                tol[r, h] = 1.1 * dy + (HALF[dtype] + 2.0 ** -21) * np.abs(y) + (2.0 ** -25 if dtype == "f16" else 1e-30)
    return out, tol, ml, es


def make_case(seed, dtype, kv, size, layout, kv_heads, group, lens, *, q_len=None, softcap=0.0, alibi=False, window=-1,
              norm=True, weight=True, per_row=False, max_seq_len=None, spare=3, mult=1.0):
    """Inputs on the CPU.  Slots that no token owns, and spare pages, are NaN."""
    gen = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, dtype=np.int64)
    n, heads = len(lens), kv_heads * group
    own = [-(-int(x) // BS) for x in lens]
    blocks = sum(own) + spare
    ids = rng.permutation(blocks)
    max_len = int(max(lens.max(), 1)) if max_seq_len is None else max_seq_len
    table = np.full((n, -(-max_len // BS)), int(ids[-1]), dtype=np.int64)
    used, at = np.zeros((blocks, BS), dtype=bool), 0
    for s in range(n):
        table[s, :own[s]] = ids[at:at + own[s]]
        at += own[s]
        for p in range(own[s]):
            used[table[s, p], :min(BS, int(lens[s]) - p * BS)] = True
    start = None if q_len is None else np.concatenate([[0], np.cumsum(q_len)]).astype(np.int64)
    rows = n if q_len is None else int(start[-1])
    ct = FP8[kv] if kv else TORCH[dtype]
    x = 16 // ct.itemsize
    scale = 0.02 if kv else 1.0

    def cache(h, d, is_key):
        c = torch.randn((blocks, h, BS, d), generator=gen) * mult / scale
        if kv:  # as a cache is filled: beyond the largest value, that value
            c = c.clamp(-torch.finfo(ct).max, torch.finfo(ct).max)
        c = c.masked_fill(~torch.from_numpy(used)[:, None, :, None], float("nan")).to(ct)
        if layout == "split":
            c = c.unflatten(3, (d // x, x)).permute(0, 1, 3, 2, 4) if is_key else c.transpose(2, 3)
        return c.contiguous()

    query = (torch.randn((rows, heads, 2, size), generator=gen) * mult).to(TORCH[dtype])
    lam = torch.rand((rows, heads) if per_row else (heads,), generator=gen) * 0.8 + 0.1
    return dict(query=query, key_cache=cache(2 * kv_heads, size, True), value_cache=cache(kv_heads, 2 * size, False),
                table=table, lens=lens, start=start, q_len=q_len, lambdas=lam, kv_heads=kv_heads, dtype=dtype, kv=kv,
                layout=layout, scale=size ** -0.5, softcap=softcap, window=window, norm=norm, eps=1e-5, out_scale=0.4,
                norm_weight=1 + 0.2 * torch.randn(2 * size, generator=gen) if weight and norm else None,
                alibi=torch.tensor([2.0 ** (-8.0 * (i + 1) / heads) for i in range(heads)]) if alibi else None,
                k_scale=scale, v_scale=scale, max_seq_len=max_len)
