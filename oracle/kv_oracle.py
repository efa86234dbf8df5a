"""Plain fp64 definitions of the key-value cache's operations and of the
scores read from logits: what kv_append stores, what kv_attend and kv_evict
compute of one sequence's slots, log probabilities with entropy and
alternatives. Loops and numpy only; no paging (the tests place the slots)."""

from __future__ import annotations

import numpy as np

EPS = 2.0 ** -24  # half a step of fp32, relative


def round_bf16(x):
    """fp32 values rounded to bfloat16 (nearest even), as fp32."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32)


def kv_store(x, kind: str):
    """What a cache holds of fp32 rows x [..., head_dim]: (codes or values,
    scales or None). int8: s = max|x| / 127 rounded once to fp32 (1 for zeros),
    code = rint(x / s) in fp64."""
    x = np.asarray(x, dtype=np.float32)
    if kind == "float32":
        return x, None
    if kind == "float16":
        with np.errstate(over="ignore"):
            return x.astype(np.float16), None
    if kind == "bfloat16":
        return round_bf16(x), None
    top = np.abs(x).max(axis=-1)
    s = np.where(top > 0, (top.astype(np.float64) / 127.0).astype(np.float32), np.float32(1))
    q = np.clip(np.rint(x.astype(np.float64) / s.astype(np.float64)[..., None]), -127, 127)
    return q.astype(np.int8), s


def kv_values(codes, scales):
    """fp64 values that stored rows stand for."""
    v = np.asarray(codes).astype(np.float64)
    return v if scales is None else v * np.asarray(scales).astype(np.float64)[..., None]


def kv_attend_ref(q, k, v, scale: float, window: int = 0):
    """One sequence: q [q_heads, dim], k / v [slots, kv_heads, dim] (fp64
    values). Returns out, lse, the weights [q_heads, slots], and the bounds
    (out, lse, weights) that the fp32 kernels are held to.

    The bounds count roundings (EPS each, relative). A score is a dot product
    of dim terms, a multiplication by the scale and one by an int8 scale: at
    most (dim + 4) EPS of sum |q k| scale. Matrix instructions take q and the
    weights as two fp16 pieces of what lies at or below 2^15: the first one's
    rest is at most 2^-11 of it and exact in fp32, the second one (that rest
    times 2^11) is off by at most 2^-11 of the rest, or by half of fp16's
    smallest step, 2^-25, which is 2^-36 of what is stored. So 2^-22 of each
    term is left out, or 2^-36, where the largest q is at least 2^14 and the
    largest weight at least 2^7: 2^-50 of the largest q, 2^-43 of the largest
    weight (int8: of the largest weight times scale, so less than the 2^-42 of
    the largest value that is counted here). A weight is the exponential
    of a difference of two scores (the exponential itself is good to 2^-22),
    and sums of n weights, in any order, rescaled at most once a slot, lose at
    most 2 n roundings."""
    q, k, v = (np.asarray(a, dtype=np.float64) for a in (q, k, v))
    Hq, D = q.shape
    n, H, _ = k.shape
    G = Hq // H
    out, lse, w = np.zeros((Hq, D)), np.full(Hq, -np.inf), np.zeros((Hq, n))
    t_out, t_lse, t_w = np.zeros((Hq, D)), np.zeros(Hq), np.zeros((Hq, n))
    lo = max(0, n - window) if window > 0 else 0
    if n == 0:
        return out, lse, w, (t_out, t_lse, t_w)
    for i in range(Hq):
        kk, vv = k[lo:, i // G], v[lo:, i // G]
        s = scale * (kk @ q[i])
        m = s.max()
        e = np.exp(s - m)
        w[i, lo:] = e / e.sum()
        lse[i] = m + np.log(e.sum())
        out[i] = w[i, lo:] @ vv
        ds = ((D + 4) * EPS + 2.0 ** -21) * abs(scale) * (np.abs(kk) @ np.abs(q[i])).max() + 4 * EPS * np.abs(s).max()
        ds += 2.0 ** -50 * abs(scale) * np.abs(q[i]).max() * np.abs(kk).sum(1).max()
        rel = 2 * ds + (2 * (n - lo) + 64) * EPS
        t_out[i] = rel * (w[i, lo:] @ np.abs(vv)) + 2.0 ** -42 * 127 * (n - lo) * np.abs(vv).max() + 1e-37
        t_lse[i] = rel + 4 * EPS * abs(lse[i])
        t_w[i, lo:] = rel * w[i, lo:] + 1e-37
    return out, lse, w, (t_out, t_lse, t_w)


def kv_evict_ref(acc, n: int, keep: int, recent: int):
    """The slots of one sequence that stay, ascending: the last
    min(recent, keep), and of the others those with the largest acc, ties to
    the lower slot, NaN below everything."""
    if n <= keep:
        return list(range(n))
    last = min(recent, keep)
    m = n - last
    w = [float(a) for a in acc[:m]]
    order = sorted(range(m), key=lambda j: (w[j] != w[j], -w[j] if w[j] == w[j] else 0.0, j))
    return sorted(order[:keep - last]) + list(range(m, n))


def logprobs_ref(logits, tokens=None, top: int = 0):
    """(logp, entropy, top_logp, top_ids) of rows of logits in fp64."""
    x = np.asarray(logits, dtype=np.float64)
    M, V = x.shape
    logp, entropy = np.zeros(M), np.full(M, np.nan)
    top_logp, top_ids = np.full((M, top), np.nan), np.zeros((M, top), np.int64)
    for m in range(M):
        r = x[m]
        nan = np.isnan(r)
        order = sorted(range(V), key=lambda j: (nan[j], -r[j] if not nan[j] else 0.0, j))[:top]
        top_ids[m] = order
        lp = np.full(V, np.nan)  # about the maximum: a large one would drown the logarithm
        if not nan.any() and np.max(r) < np.inf and np.max(r) > -np.inf:
            top_x = np.max(r)
            lp = (r - top_x) - np.log(np.exp(r - top_x).sum())
            p = np.exp(lp)
            entropy[m] = -(p[p > 0] * lp[p > 0]).sum()
        top_logp[m] = lp[order]
        if tokens is not None:
            t = int(tokens[m])
            logp[m] = 0.0 if t == -1 else (lp[t] if 0 <= t < V else np.nan)
    return logp, entropy, top_logp, top_ids
