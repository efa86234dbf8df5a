"""What is measured of the decode step's operators around the matmuls: the
paged key-value cache (append, attention of one new token, eviction) and the
log probabilities read from the head's logits.

`listed()` and `draw()` give cases, `prepare()` the inputs of one, `run()` one
pass: in plain torch operations (own = False) or through the library's entry
points (own = True). `exact()` is the definition in 64 bits.
"""

import math
import random

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16, "int8": torch.int8}
SIZES = {"fp32": 4, "fp16": 2, "bf16": 2, "int8": 1}
LN2 = math.log(2.0)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a small batch: a token's keys and values of the 12 x 64 heads each, into 16-slot pages
        dict(name="append step", op="append", type="fp32", seqs=8, heads=12, dim=64, page=16, most=1, past=900, lens=1),
        # a batch of prompts of unequal length enters the cache at once (32 heads of 96: a 9216-wide qkv row)
        dict(name="append prompts", op="append", type="bf16", seqs=24, heads=32, dim=96, page=32, most=600, past=40,
             lens=2),
        # the decode step of one GPT-2-shaped sequence near its 1024-token limit
        dict(name="attend one 12x64", op="attend", type="fp32", seqs=1, heads=12, group=1, dim=64, page=16, most=1021,
             full=True, window=0, acc=False, lens=3),
        # a serving batch of the same shape at unequal lengths (an empty slot of the batch among them)
        dict(name="attend batch 12x64", op="attend", type="bf16", seqs=48, heads=12, group=1, dim=64, page=16,
             most=1024, full=False, window=0, acc=False, lens=4),
        # the 3.8B shape's attention (32 heads of 96), mid-sized batch, attention weights gathered for eviction
        dict(name="attend 32x96 weights", op="attend", type="fp16", seqs=8, heads=32, group=1, dim=96, page=32,
             most=4000, full=False, window=0, acc=True, lens=5),
        # grouped queries over a quantised cache, unequal lengths, a sliding window
        dict(name="attend grouped int8", op="attend", type="int8", seqs=32, heads=8, group=8, dim=128, page=16,
             most=6000, full=False, window=4096, acc=False, lens=6),
        # one very long sequence, grouped queries: the split over the length is all there is to share out
        dict(name="attend long grouped", op="attend", type="bf16", seqs=1, heads=8, group=4, dim=128, page=64,
             most=131072, full=True, window=0, acc=False, lens=7),
        # one GPT-2-shaped sequence halved once it reaches its limit
        dict(name="evict one 12x64", op="evict", type="fp32", seqs=1, heads=12, dim=64, page=16, most=1024, full=True,
             keep=512, recent=128, lens=8),
        # a batch of long sequences cut to a budget (odd sizes, some already within it)
        dict(name="evict batch", op="evict", type="bf16", seqs=16, heads=8, dim=128, page=64, most=16000, full=False,
             keep=2045, recent=301, lens=9),
        # the decode step's answer: one row of GPT-2's vocabulary, five alternatives
        dict(name="logprobs one row", op="logprobs", rows=1, vocab=50257, top=5),
        # a prompt of 58 tokens scored, twenty alternatives each
        dict(name="logprobs prompt", op="logprobs", rows=58, vocab=50257, top=20),
        # a long text scored: no alternatives
        dict(name="logprobs text", op="logprobs", rows=2048, vocab=50257, top=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "evict", "logprobs"])
    if op == "logprobs":
        rows = _log(rng, 1, 2048)
        vocab = min(_log(rng, 300, 200000), 100_000_000 // rows)
        return dict(op=op, rows=rows, vocab=vocab, top=rng.choice([0, 1, rng.randint(2, 20), 32]))
    kind = rng.choice(["fp32", "fp16", "bf16", "int8"])
    heads, dim = _log(rng, 1, 40), 16 * rng.choice([1, 2, 3, 4, 4, 4, 5, 6, 6, 7, 8, 8, 8, 10, 12, 16])
    page, lens = rng.choice([16, 32, 64, 128, _log(rng, 1, 200)]), rng.randrange(1 << 30)
    room = 60_000_000 // (heads * dim)  # slots of all sequences together
    if op == "append":
        seqs = _log(rng, 1, 256)
        most = _log(rng, 1, max(1, min(4000, room // (4 * seqs))))
        return dict(op=op, type=kind, seqs=seqs, heads=heads, dim=dim, page=page, most=most, past=rng.randint(0, 300),
                    lens=lens)
    seqs = _log(rng, 1, 200)
    most = _log(rng, 1, max(1, min(131072, room // seqs)))
    full = rng.random() < 0.3
    if op == "evict":
        keep = rng.randint(1, most)
        return dict(op=op, type=kind, seqs=seqs, heads=heads, dim=dim, page=page, most=most, full=full, keep=keep,
                    recent=rng.randint(0, keep), lens=lens)
    group = rng.choice([1, 1, 2, 3, 4, 5, 8, 16])
    return dict(op=op, type=kind, seqs=seqs, heads=heads, group=group, dim=dim, page=page, most=most, full=full,
                window=rng.choice([0, 0, rng.randint(1, most)]), acc=rng.random() < 0.3, lens=lens)


def _counts(case):
    """A number from 0 to `most` for each sequence, the case's own: lengths, or tokens to append. Of unequal ones, one
    is `most` and, of more than two, one is 0: an unused place of the batch."""
    r, most, n = random.Random(case["lens"]), case["most"], case["seqs"]
    if case.get("full") or most == 1:
        return [most] * n
    got = [r.randint(0, most) for _ in range(n)]
    first = r.randrange(n)
    got[first] = most
    if n > 2:
        got[(first + r.randrange(1, n)) % n] = 0
    return got


def _past(case):
    r = random.Random(case["lens"] + 1)
    return [r.randint(0, case["past"]) for _ in range(case["seqs"])]


def work(case):
    if case["op"] == "logprobs":
        n = case["rows"] * case["vocab"]
        return {"bytes": 4 * n + case["rows"] * (12 + 8 * case["top"]), "flops": 5 * n}
    n = _counts(case)
    es, wide = SIZES[case["type"]], case["heads"] * case["dim"]
    slot = 2 * wide * es + (8 * case["heads"] if case["type"] == "int8" else 0)
    if case["op"] == "append":
        return {"bytes": sum(n) * (8 * wide + slot) + 16 * case["seqs"], "flops": 2 * sum(n) * wide}
    if case["op"] == "evict":
        kept = sum(min(x, case["keep"]) for x in n)
        return {"bytes": 4 * sum(n) + kept * (2 * slot + 8), "flops": sum(n)}
    used = sum(min(x, case["window"]) if case["window"] else x for x in n)
    return {"bytes": used * (slot + (8 if case["acc"] else 0)) + case["seqs"] * case["group"] * (8 * wide + 4 * case["heads"]),
            "flops": 4 * used * wide * case["group"]}


# ---------------------------------------------------------------- inputs

def _pages(case, counts, g, order):
    """Page table rows of `counts` slots each over shuffled pages, and the number of pages."""
    page = case["page"]
    need = [-(-c // page) for c in counts]
    width = max(1, max(need))
    total = sum(need) + 3
    ids = list(range(1, total))  # page 0 is nobody's: the table's unused entries name it
    order.shuffle(ids)
    rows, at = [], 0
    for n in need:
        rows.append(ids[at:at + n] + [0] * (width - n))
        at += n
    return torch.tensor(rows, dtype=torch.int32, device="cuda"), total


def _values(case, pages, g):
    """Keys or values of all pages as a cache holds them, and their scales."""
    shape = (pages, case["heads"], case["page"], case["dim"])
    if case["type"] == "int8":
        codes = torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)
        return codes, torch.rand(shape[:3], generator=g, device="cuda") * 0.02 + 0.008
    return torch.randn(shape, generator=g, device="cuda").to(DTYPES[case["type"]]), None


def _blank(case, pages):
    shape = (pages, case["heads"], case["page"], case["dim"])
    scales = torch.zeros(shape[:3], device="cuda") if case["type"] == "int8" else None
    return torch.zeros(shape, dtype=DTYPES[case["type"]], device="cuda"), scales


def _cache(k, ks, v, vs, table, lengths):
    """What a program holds of one layer's cache; with the library, its handle too."""
    c = {"k": k, "ks": ks, "v": v, "vs": vs, "table": table, "lengths": lengths}
    if own:
        import int8_weight_quantized_w4_b200 as w4
        c["handle"] = w4.KvCache(k, v, table, lengths, k_scales=ks, v_scales=vs)
    return c


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "logprobs":
        m, n = case["rows"], case["vocab"]
        s["logits"] = torch.randn((m, n), generator=g, device="cuda") * 3.0
        s["tokens"] = torch.randint(0, n, (m,), generator=g, device="cuda", dtype=torch.int32)
        return s
    order = random.Random(seed)
    counts = _counts(case)
    ints = dict(dtype=torch.int32, device="cuda")
    if case["op"] == "append":
        past = _past(case)
        table, pages = _pages(case, [a + b for a, b in zip(past, counts)], g, order)
        (k, ks), (v, vs) = _blank(case, pages), _blank(case, pages)
        s["cache"] = _cache(k, ks, v, vs, table, torch.tensor(past, **ints))
        # the new tokens' keys and values are columns of their qkv rows
        wide, tokens = case["heads"] * case["dim"], sum(counts)
        qkv = torch.randn((tokens, 3 * wide), generator=g, device="cuda")
        s["new_k"] = qkv[:, wide:2 * wide].view(tokens, case["heads"], case["dim"])
        s["new_v"] = qkv[:, 2 * wide:].view(tokens, case["heads"], case["dim"])
        s["cu"] = torch.tensor([0] + counts, **ints).cumsum(0, dtype=torch.int32)
        s["lengths"] = torch.empty(case["seqs"], **ints)
        return s
    table, pages = _pages(case, counts, g, order)
    (k, ks), (v, vs) = _values(case, pages, g), _values(case, pages, g)
    s["cache"] = _cache(k, ks, v, vs, table, torch.tensor(counts, **ints))
    slots = table.shape[1] * case["page"]
    held = torch.arange(slots, device="cuda") < s["cache"]["lengths"][:, None]
    if case["op"] == "evict":
        # weights gathered over many steps: a few slots hold most of them
        s["acc"] = torch.where(held, torch.rand((case["seqs"], slots), generator=g, device="cuda") ** 8 * 40.0, 0.0)
        to, pages = _pages(case, [min(c, case["keep"]) for c in counts], g, order)
        (k, ks), (v, vs) = _blank(case, pages), _blank(case, pages)
        s["to"] = _cache(k, ks, v, vs, to, torch.zeros(case["seqs"], **ints))
        s["acc_to"] = torch.zeros((case["seqs"], slots), device="cuda")
        s["kept"] = torch.empty((case["seqs"], case["keep"]), **ints)
        return s
    # queries are the first columns of their rows; a few keys stand out, as in a trained model
    hq = case["heads"] * case["group"]
    rows = torch.randn((case["seqs"], (hq + 2 * case["heads"]) * case["dim"]), generator=g, device="cuda")
    s["q"] = rows[:, :hq * case["dim"]].view(case["seqs"], hq, case["dim"]) * 1.5
    s["scale"] = 1.0 / math.sqrt(case["dim"])
    s["out"] = torch.empty((case["seqs"], hq, case["dim"]), device="cuda")
    s["lse"] = torch.empty((case["seqs"], hq), device="cuda")
    if case["acc"]:
        s["acc"] = torch.where(held, torch.rand((case["seqs"], slots), generator=g, device="cuda"), 0.0)
    return s


# ---------------------------------------------------------------- plain forms

def _stored(x, kind):
    """x [tokens, heads, dim] as the cache holds it: (elements, scales)."""
    if kind != "int8":
        return x.to(DTYPES[kind]), None
    top = x.abs().amax(-1)
    scale = torch.where(top > 0, (top.double() / 127.0).float(), 1.0)
    return torch.round(x.double() / scale.double()[..., None]).clamp(-127, 127).to(torch.int8), scale


def _held(pages, scales):
    """The values that stored elements stand for, in 32 bits."""
    return pages.float() if scales is None else pages.float() * scales[..., None]


def _plain_append(s):
    c, cu, kind = s["cache"], s["cu"].long(), s["case"]["type"]
    page = c["k"].shape[2]
    t = torch.arange(s["new_k"].shape[0], device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    at = c["lengths"].long()[seq] + t - cu[seq]
    where = c["table"].long()[seq, at // page], slice(None), at % page
    for name, new in (("k", s["new_k"]), ("v", s["new_v"])):
        x, scale = _stored(new, kind)
        c[name][where] = x
        if scale is not None:
            c[name + "s"][where] = scale
    return torch.add(c["lengths"], torch.diff(s["cu"]), out=s["lengths"])


def _gather(pages, scales, table):
    """[seqs, heads, slots, dim] in 32 bits of the pages that the table names."""
    t = table.long()
    x = _held(pages[t], None if scales is None else scales[t])
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attend(s):
    case, c = s["case"], s["cache"]
    k, v = _gather(c["k"], c["ks"], c["table"]), _gather(c["v"], c["vs"], c["table"])
    b, h, n, d = k.shape
    at, length = torch.arange(n, device="cuda"), c["lengths"].long()[:, None]
    seen = at < length
    if case["window"]:
        seen &= at >= length - case["window"]
    q = s["q"].reshape(b, h, case["group"], d)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"])
    x.masked_fill_(~seen[:, None, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    v = v.masked_fill(~seen[:, None, :, None], 0.0)
    p = p / torch.where(total > 0, total, 1.0)
    s["out"].copy_(torch.matmul(p, v).reshape(b, h * case["group"], d))
    s["lse"].copy_((torch.log(total) + top).reshape(b, h * case["group"]))
    if case["acc"]:
        s["acc"] += p.sum((1, 2))
        return s["out"], s["lse"], s["acc"]
    return s["out"], s["lse"]


def _plain_evict(s):
    case, c, to, acc = s["case"], s["cache"], s["to"], s["acc"]
    n, keep, page = acc.shape[1], case["keep"], case["page"]
    at, length = torch.arange(n, device="cuda"), c["lengths"].long()[:, None]
    held = at < length
    rank = torch.where(held, acc, -math.inf)
    rank = torch.where(held & (at >= length - case["recent"]), math.inf, rank)
    best = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :keep]
    fresh = length.clamp(max=keep)
    i = torch.arange(best.shape[1], device="cuda")
    kept = torch.where(i < fresh, best, n).sort(1).values  # ascending, `n` behind the last
    s["kept"].fill_(-1)
    s["kept"][:, :best.shape[1]] = torch.where(i < fresh, kept, -1).int()
    j = torch.arange(to["table"].shape[1] * page, device="cuda")
    live = j < fresh
    src = torch.nn.functional.pad(kept, (0, max(0, j.numel() - kept.shape[1])))[:, :j.numel()].clamp(max=n - 1)
    a = torch.gather(c["table"].long(), 1, src // page), slice(None), src % page
    z = to["table"].long()[:, j // page], slice(None), (j % page).expand_as(src)
    z = tuple(x if isinstance(x, slice) else torch.where(live, x, 0) for x in z)
    for name in ("k", "v", "ks", "vs"):
        if c[name] is not None:
            # what lies past a sequence's new end goes to page 0, which stays as it is
            old = to[name][0, :, 0]
            to[name][z] = torch.where(live.reshape(live.shape + (1,) * old.dim()), c[name][a], old)
    to["lengths"].copy_(fresh[:, 0])
    m = min(n, kept.shape[1])
    s["acc_to"].masked_fill_(held, 0.0)
    s["acc_to"][:, :m] = torch.where(i[:m] < fresh, torch.gather(acc, 1, kept.clamp(max=n - 1))[:, :m], s["acc_to"][:, :m])


def _plain_logprobs(s):
    x, top = s["logits"], s["case"]["top"]
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(1, keepdim=True)
    lse = m + torch.log(total)
    logp = torch.gather(x, 1, s["tokens"].long()[:, None]) - lse
    entropy = torch.log(total) - (e * (x - m)).sum(1, keepdim=True) / total
    if not top:
        return logp[:, 0], entropy[:, 0]
    # keys in the logits' order, the lower id first among equals
    bits = x.view(torch.int32).long()
    bits = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    ids = torch.arange(x.shape[1], device="cuda")
    got = torch.topk((bits << 32) - ids, top, dim=1).values
    ids = (-got) & 0xFFFFFFFF
    return logp[:, 0], entropy[:, 0], torch.gather(x, 1, ids) - lse, ids.int()


# ---------------------------------------------------------------- a pass

def run(s):
    op, case = s["case"]["op"], s["case"]
    if op == "logprobs":
        if own:
            import int8_weight_quantized_w4_b200 as w4
            got = w4.token_logprobs(s["logits"], s["tokens"], top=case["top"])
            return got if case["top"] else got[:2]
        return _plain_logprobs(s)
    if op == "attend":
        if own:
            import int8_weight_quantized_w4_b200 as w4
            out = w4.kv_attend(s["q"], s["cache"]["handle"], scale=s["scale"], window=case["window"], out=s["out"],
                               lse=s["lse"], acc=s.get("acc"))
            return (out, s["lse"], s["acc"]) if case["acc"] else (out, s["lse"])
        return _plain_attend(s)
    if op == "append":
        c = s["cache"]
        if own:
            import int8_weight_quantized_w4_b200 as w4
            w4.kv_append(c["handle"], s["new_k"], s["new_v"], cu_tokens=s["cu"], lengths_out=s["lengths"])
        else:
            _plain_append(s)
        return _values_of(c) + (s["lengths"],)
    if own:
        import int8_weight_quantized_w4_b200 as w4
        w4.kv_evict(s["cache"]["handle"], s["acc"], case["keep"], recent=case["recent"], dst=s["to"]["handle"],
                    acc_out=s["acc_to"], kept=s["kept"])
    else:
        _plain_evict(s)
    return _values_of(s["to"]) + (s["to"]["lengths"], s["acc_to"], s["kept"])


def _values_of(c):
    """The cache's content; where it is held in 8 bits, the values that it stands for."""
    if c["ks"] is None:
        return c["k"], c["v"]
    return _held(c["k"], c["ks"]), _held(c["v"], c["vs"])


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_logprobs(s):
    top, out = s["case"]["top"], []
    for x, t in zip(s["logits"], s["tokens"].tolist()):
        x64 = x.double()
        lp = x64 - torch.logsumexp(x64, 0)
        p = lp.exp()
        row = [lp[t], -(p * lp).sum()]
        if top:
            order = torch.sort(x, descending=True, stable=True).indices[:top]
            row += [lp[order], order.int()]
        out.append(row)
    return tuple(torch.stack(col) for col in zip(*out))


def _row64(c, name, b, j):
    """Slot j of sequence b, all heads, in 64 bits."""
    page = c[name].shape[2]
    p = c["table"][b].long()[j // page]
    x = c[name][p, :, j % page].double()
    return x if c[name + "s"] is None else x * c[name + "s"][p, :, j % page].double()[..., None]


def _exact_attend(s):
    case, c, g = s["case"], s["cache"], s["case"]["group"]
    out, lse = torch.zeros_like(s["out"], dtype=torch.float64), torch.full_like(s["lse"], -math.inf, dtype=torch.float64)
    acc = s["acc"].double() if case["acc"] else None
    for b, n in enumerate(c["lengths"].tolist()):
        lo = max(0, n - case["window"]) if case["window"] else 0
        if n == lo:
            continue
        j = torch.arange(lo, n, device="cuda")
        k, v = _row64(c, "k", b, j), _row64(c, "v", b, j)  # [slots, heads, dim]
        for h in range(case["heads"]):
            x = s["q"][b, h * g:(h + 1) * g].double() @ k[:, h].T * float(s["scale"])
            z = torch.logsumexp(x, 1)
            p = torch.exp(x - z[:, None])
            out[b, h * g:(h + 1) * g] = p @ v[:, h]
            lse[b, h * g:(h + 1) * g] = z
            if acc is not None:
                acc[b, lo:n] += p.sum(0)
    return (out, lse) if acc is None else (out, lse, acc)


def _exact_append(s):
    c, kind = s["cache"], s["case"]["type"]
    page, cu, past = s["case"]["page"], s["cu"].tolist(), c["lengths"].tolist()
    out = []
    for name, new in (("k", s["new_k"]), ("v", s["new_v"])):
        values = torch.zeros(c[name].shape, dtype=torch.float64, device="cuda")
        for b in range(len(past)):
            x = new[cu[b]:cu[b + 1]]
            if kind == "int8":  # codes of a scale that is held in 32 bits
                scale = (x.double().abs().amax(-1, keepdim=True) / 127).float().double()
                scale[scale == 0] = 1
                x = (x.double() / scale).round().clamp(-127, 127) * scale
            else:
                x = x.to(DTYPES[kind])
            j = torch.arange(past[b], past[b] + cu[b + 1] - cu[b], device="cuda")
            values[c["table"][b].long()[j // page], :, j % page] = x.double()
        out.append(values)
    return out[0], out[1], torch.tensor([n + cu[b + 1] - cu[b] for b, n in enumerate(past)], dtype=torch.int32)


def _exact_evict(s):
    case, c, to, page = s["case"], s["cache"], s["to"], s["case"]["page"]
    values = [torch.zeros(to["k"].shape, dtype=torch.float64, device="cuda") for _ in range(2)]
    acc, kept, lengths = torch.zeros_like(s["acc"], dtype=torch.float64), torch.full_like(s["kept"], -1), []
    for b, n in enumerate(c["lengths"].tolist()):
        m = min(n, case["keep"])
        lengths.append(m)
        if not m:
            continue
        w = s["acc"][b, :n].clone()
        if case["recent"]:
            w[max(0, n - case["recent"]):] = math.inf
        order = torch.sort(-w, stable=True).indices[:m]
        j = order.sort().values
        i = torch.arange(m, device="cuda")
        for x, name in zip(values, ("k", "v")):
            x[to["table"][b].long()[i // page], :, i % page] = _row64(c, name, b, j)
        acc[b, :m] = s["acc"][b, j].double()
        kept[b, :m] = j.int()
    return values[0], values[1], torch.tensor(lengths, dtype=torch.int32), acc, kept


def exact(case, seed):
    s = prepare(case, seed)
    return {"logprobs": _exact_logprobs, "attend": _exact_attend, "append": _exact_append, "evict": _exact_evict}[case["op"]](s)
