"""Helpers of the key-value cache's GPU tests: a paged cache built from
per-sequence rows, with NaN (or codes whose scales are NaN) wherever no
sequence holds a slot, so that a kernel that lets such a slot in shows it."""

from __future__ import annotations

import numpy as np

import oracle

KINDS = ["float32", "float16", "bfloat16", "int8"]


def torch():
    import torch as T
    return T


def w4():
    import int8_weight_quantized_w4_b200 as w
    return w


def build(rng, kind, lengths, heads, dim, page, max_pages=None, spare=2, gap=0, shared=False, amp=1.0):
    """(cache, [k rows of each sequence], [v rows]) with fp64 values
    [len, heads, dim]; pages in random order, `gap` pages between two of them
    in memory; `shared`: one row of pages for all sequences."""
    T = torch()
    dt = getattr(T, kind)
    need = [-(-n // page) for n in lengths]
    if shared:
        need = [max(need)] + [0] * (len(need) - 1)
    mp = max_pages or max(1, max(need))
    total = sum(need) + spare
    ids = rng.permutation(total)
    table = np.full((len(lengths), mp), -1, np.int32)  # entries behind the last page name none
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    if shared:
        table[:] = table[0]
    shape = (total, heads, page, dim)
    store, scales, rows = {}, {}, {}
    for name in ("k", "v"):
        x = (rng.standard_normal(shape) * amp).astype(np.float32)
        codes, sc = oracle.kv_store(x, kind)
        held = np.zeros((total, page), bool)
        per_seq = []
        for b, n in enumerate(lengths):
            j = np.arange(n)
            p = table[b, j // page]
            held[p, j % page] = True
            per_seq.append(oracle.kv_values(codes[p, :, j % page], None if sc is None else sc[p, :, j % page]))
        t = T.from_numpy(np.ascontiguousarray(codes)).to(dt)
        free = T.from_numpy(~held)
        if sc is None:
            t.masked_fill_(free[:, None, :, None], float("nan"))
        else:
            s = T.from_numpy(sc.copy())
            s.masked_fill_(free[:, None, :], float("nan"))
            scales[name] = s.cuda()
        big = T.zeros((total * (gap + 1),) + shape[1:], dtype=dt, device="cuda")
        view = big[::gap + 1]
        view.copy_(t)
        store[name], rows[name] = view, per_seq
    tb = T.from_numpy(table).cuda()
    if shared:
        tb = tb[:1].expand(len(lengths), mp)
    ln = T.tensor(lengths, dtype=T.int32, device="cuda")
    cache = w4().KvCache(store["k"], store["v"], tb, ln, k_scales=scales.get("k"), v_scales=scales.get("v"))
    return cache, rows["k"], rows["v"]


def read_rows(cache, b, n):
    """fp64 values [n, heads, dim] of k and v that sequence b holds."""
    S = cache.page_size
    j = np.arange(n)
    p = cache.page_table[b].cpu().numpy()[j // S]
    out = []
    for t, s in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
        x = t.cpu().double().numpy()[p, :, j % S]
        out.append(x if s is None else x * s.cpu().double().numpy()[p, :, j % S][..., None])
    return out


def clear_error():
    w4().device_error(clear=True)


def error_status():
    torch().cuda.synchronize()
    return w4().device_error(clear=True)[0]
