"""How far pa_diff_decode may be from the formula, closer than diff_ref.py says it:
from what each kernel computes, and with the softcap's error relative to the logit.

Per row, head and map, with a_t the softmax weights, v_t the value rows, m the
reference that the weights are taken against and u = 2^-24 (half a step of fp32):

  logit     16-bit and fp8 keys: exact products on the tensor cores, summed in groups
            of at most 16, and the d / 8 group sums (at most) added, a step 2^-23 of
            S_t = scale sum |q k| lost each, and as diff_ref.py some roundings of the
            result:  2^-23 (d / 8 + 24) S_t.  Over fp8 keys a bf16 query goes through
            fp16: |q - fp16(q)| |k| more.  fp32 keys: a chain of d / 4 fused
            multiply-adds, two exchange additions, the scale and one more rounding:
            u (d / 4 + 4) S_t.
  softcap   tanhf path (fp32): the reciprocal of the cap, its product, tanhf (two steps)
            and the product with the cap:  8 u |z|.  Quick form (16-bit queries): four
            steps of 1 times the cap, 4 2^-23 cap; above QUICK_CAP that only from a
            quarter of the cap on (where |z| >= 0.24 cap: 2^-18 |z|), below it a series
            of five terms, whose rounding is within that of tanhf.
  alibi     slope x distance and its addition, relative to the sequence's last token:
            2 u |bias_t| + u |z_t|
  weight    exp2((z - m) log2 e): 4 u |z_t - m| in the exponent, and exp2f's own two
            steps; the same again when the warps and the partitions are merged:
            a relative 3 x 2^-22.  m may lag behind the maximum (by 8 at most).
  P.V       the weight as an operand: 2^-21 (fp16 in two terms; and an absolute 2^-25
            where it is subnormal, against a sum of exp(z - m) >= exp(z - max z)), 2^-17 (bf16 in two
            terms), none (fp32).  Sums over n tokens, in pages of 16:  2^-23 (n / 16 + 64)
            on the tensor cores; fp32 a chain of 16 per page, one addition per page and
            one per merge:  u (n / 16 + 64).

A relative error r_t of the weights moves an output of the map by at most
sum a_t r_t |v_tj| + A_j sum a_t r_t, A_j = sum a_t |v_tj|; the norm's part is as in
diff_ref.py, with the same factor 1.1 for second-order terms.
"""
from __future__ import annotations

import numpy as np
import torch

from diff_ref import HALF, logical

QUICK_CAP = 64.0


def tight_ref(case):
    """out, tol [rows, heads, 2d] in 64 bits."""
    q = case["query"].double().numpy()
    q16 = case["query"].half().double().numpy()  # what meets fp8 keys
    rows, heads, _, d = q.shape
    g, dtype, kv = heads // case["kv_heads"], case["dtype"], case["kv"]
    u, f32 = 2.0 ** -24, dtype == "f32"
    out, tol = np.zeros((rows, heads, 2 * d)), np.zeros((rows, heads, 2 * d))
    start = case["start"] if case["start"] is not None else np.arange(len(case["lens"]) + 1)
    lam = case["lambdas"].double().numpy()
    w = np.ones(2 * d) if case["norm_weight"] is None else case["norm_weight"].double().numpy()
    cap, scale = case["softcap"], float(np.float32(case["scale"]))
    for s, length in enumerate(case["lens"]):
        length = int(length)
        n_q = int(start[s + 1] - start[s])
        if not length or not n_q:
            continue
        k = logical(case["key_cache"], case["table"][s], length, case["layout"], True, kv) * np.float32(case["k_scale"])
        v = logical(case["value_cache"], case["table"][s], length, case["layout"], False, kv) * np.float32(case["v_scale"])
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
                    dz = u * (d / 4 + 4) * big if f32 else 2.0 ** -23 * (d / 8 + 24) * big
                    if kv and dtype == "bf16":
                        dz = dz + abs(scale) * (np.abs(kk) @ np.abs(q[r, h, m] - q16[r, h, m]))
                    if cap > 0:
                        quarter = np.abs(z) >= 0.25 * cap
                        z = cap * np.tanh(z / cap)
                        quick = 4 * 2.0 ** -23 * cap if cap <= QUICK_CAP else np.where(quarter, 2.0 ** -18, 8 * u) * np.abs(z)
                        dz = dz + (8 * u * np.abs(z) if f32 else quick)
                    if case["alibi"] is not None:
                        bias = float(case["alibi"][h]) * (t - pos)
                        z = z + bias
                        dz = dz + 2 * u * np.abs(bias) + u * np.abs(z)
                    rel = dz + 4 * u * (np.abs(z - z.max()) + 8) + 3 * 2.0 ** -22
                    a = np.exp(z - z.max())
                    a /= a.sum()
                    av = a @ np.abs(vv)
                    u_p = 0.0 if f32 else 2.0 ** -17 if dtype == "bf16" and not kv else 2.0 ** -21
                    u_s = (u if f32 else 2.0 ** -23) * (len(t) / 16 + 64)
                    e = (a * rel) @ np.abs(vv) + av * (a * rel).sum() + av * (u_p + u_s)
                    if not f32 and (kv or dtype == "f16"):
                        e = e + 2.0 ** -25 / np.exp(z - z.max()).sum() * np.abs(vv).sum(0)
                    o.append(a @ vv)
                    err.append(e)
                f = lam[r, h] if lam.ndim == 2 else lam[h]
                x, e = o[0] - f * o[1], err[0] + abs(f) * err[1] + u * (np.abs(o[0]) + abs(f) * np.abs(o[1]))
                if case["norm"]:
                    rms = np.sqrt((x * x).mean() + case["eps"])
                    y = case["out_scale"] * w * x / rms
                    dy = abs(case["out_scale"]) * np.abs(w) / rms * (e + np.abs(x) / rms * np.sqrt((e * e).mean()))
                else:
                    y, dy = case["out_scale"] * x, abs(case["out_scale"]) * e
                out[r, h] = y
                # a few roundings of the result in fp32, then the output's own
                tol[r, h] = 1.1 * dy + (HALF[dtype] + 2.0 ** -21) * np.abs(y) + (2.0 ** -25 if dtype == "f16" else 1e-30)
    return out, tol


def nearly_equal_maps(case, noise=0.02, lam=1.0, seed=0):
    """The case with the second map almost the first, so that their difference cancels,
    and small logits, whose own error leaves that of the weights to be seen."""
    gen = torch.Generator().manual_seed(seed)
    q = 0.25 * case["query"].float()
    q[:, :, 1] = q[:, :, 0] + noise * torch.randn(q[:, :, 0].shape, generator=gen)
    case["query"] = q.to(case["query"].dtype)
    k = case["key_cache"].view(torch.uint8) if case["kv"] else case["key_cache"]
    k[:, 1::2] = k[:, 0::2]
    case["lambdas"].fill_(lam)
    return case
