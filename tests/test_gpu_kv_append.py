"""GPU tests of kv_append: stored values bit for bit, places, lengths."""

import numpy as np
import pytest

import oracle
from kv_util import KINDS, build, clear_error, error_status, read_rows, torch, w4

pytestmark = pytest.mark.gpu


def as_stored(x, kind):
    return oracle.kv_values(*oracle.kv_store(x, kind))


def fresh(rng, kind, past, counts, heads, dim, page):
    """An appended-to cache with room for past + counts, holding `past` slots."""
    T = torch()
    cache, k, v = build(rng, kind, [a + b for a, b in zip(past, counts)], heads, dim, page)
    cache.lengths.copy_(T.tensor(past, dtype=T.int32))
    return cache, k, v


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,dim,page,strided", [(12, 64, 16, True), (3, 96, 7, False), (2, 256, 1, True),
                                                    (1, 16, 33, False), (40, 80, 16, True)])
def test_append_prompts(kind, heads, dim, page, strided):
    T = torch()
    rng = np.random.default_rng(heads + dim)
    past, counts = [0, 5, 16, 3, 0, 100], [7, 0, 1, 40, 0, 9]
    cache, k, v = fresh(rng, kind, past, counts, heads, dim, page)
    n = sum(counts)
    extra = 3  # rows behind the last sequence: not read
    x = (rng.standard_normal((2, n + extra, heads, dim)) * rng.uniform(0.1, 9, (2, n + extra, heads, 1))).astype(np.float32)
    x[:, 2, 0] = 0.0
    x[:, n:] = np.nan
    if strided:  # odd row strides: no 16-byte loads
        d = T.zeros((2, n + extra, heads * dim + 5), device="cuda")
        d[:, :, 1:1 + heads * dim] = T.from_numpy(x.reshape(2, n + extra, -1)).cuda()
        kd, vd = (d[i, :, 1:1 + heads * dim].view(n + extra, heads, dim) for i in range(2))
    else:
        kd, vd = T.from_numpy(x[0]).cuda(), T.from_numpy(x[1]).cuda()
    cu = T.tensor(np.r_[0, np.cumsum(counts)], dtype=T.int32, device="cuda")
    before = cache.k.clone()
    clear_error()
    out = T.full((len(counts),), -7, dtype=T.int32, device="cuda")
    w4().kv_append(cache, kd, vd, cu_tokens=cu, lengths_out=out)
    assert error_status() == 0
    assert out.tolist() == [a + b for a, b in zip(past, counts)]
    assert cache.lengths.tolist() == past  # elsewhere: the cache's own stay
    at = 0
    for b, c in enumerate(counts):
        gk, gv = read_rows(cache, b, past[b] + c)
        assert np.array_equal(gk[:past[b]], k[b][:past[b]]) and np.array_equal(gv[:past[b]], v[b][:past[b]])
        assert np.array_equal(gk[past[b]:], as_stored(x[0, at:at + c], kind))
        assert np.array_equal(gv[past[b]:], as_stored(x[1, at:at + c], kind))
        at += c
    # pages that no sequence holds are as they were
    used = set(cache.page_table.cpu().numpy().ravel().tolist())
    for p in set(range(cache.k.shape[0])) - used:
        assert T.equal(cache.k[p].view(T.uint8), before[p].view(T.uint8))
    # the same in place
    w4().kv_append(cache, kd, vd, cu_tokens=cu)
    assert error_status() == 0 and cache.lengths.tolist() == out.tolist()


@pytest.mark.parametrize("kind", KINDS)
def test_append_one_token_each(kind):
    T = torch()
    rng = np.random.default_rng(4)
    past = [0, 15, 16, 33]
    cache, k, v = fresh(rng, kind, past, [3] * 4, 12, 64, 16)
    qkv = rng.standard_normal((3, 4, 3 * 768)).astype(np.float32)
    d = T.from_numpy(qkv).cuda()
    for t in range(3):
        got = w4().kv_append(cache, d[t, :, 768:1536].view(4, 12, 64), d[t, :, 1536:].view(4, 12, 64))
        assert got is cache.lengths
    assert cache.lengths.tolist() == [n + 3 for n in past]
    for b in range(4):
        gk, gv = read_rows(cache, b, past[b] + 3)
        assert np.array_equal(gk[past[b]:], as_stored(qkv[:, b, 768:1536].reshape(3, 12, 64), kind))
        assert np.array_equal(gv[past[b]:], as_stored(qkv[:, b, 1536:].reshape(3, 12, 64), kind))
        assert np.array_equal(gk[:past[b]], k[b][:past[b]])


def test_append_many_sequences():
    """Enough sequences for more than one step of the row search."""
    T = torch()
    rng = np.random.default_rng(9)
    counts = [int(c) for c in rng.integers(0, 4, 1500)]
    past = [int(c) for c in rng.integers(0, 5, 1500)]
    cache, _, _ = fresh(rng, "float32", past, counts, 1, 16, 4)
    x = rng.standard_normal((sum(counts), 1, 16)).astype(np.float32)
    d = T.from_numpy(x).cuda()
    cu = T.tensor(np.r_[0, np.cumsum(counts)], dtype=T.int32, device="cuda")
    clear_error()
    w4().kv_append(cache, d, d, cu_tokens=cu)
    assert error_status() == 0
    assert cache.lengths.tolist() == [a + b for a, b in zip(past, counts)]
    kc, tb = cache.k.cpu().numpy(), cache.page_table.cpu().numpy()
    at = 0
    for b, c in enumerate(counts):
        j = np.arange(past[b], past[b] + c)
        assert np.array_equal(kc[tb[b, j // 4], 0, j % 4], x[at:at + c, 0])
        at += c


def test_append_int8_rounding_and_non_finite_rows():
    """Codes at halves (ties to even in the fp64 quotient), the largest and
    the smallest magnitudes; a row with Inf or NaN reads back as NaN."""
    T = torch()
    rng = np.random.default_rng(14)
    D = 64
    x = np.zeros((9, 1, D), np.float32)
    x[0, 0, :5] = [127, 0.5, 1.5, 2.5, -3.5]
    x[1] = rng.standard_normal((1, D)) * 1e30
    x[2] = rng.standard_normal((1, D)) * 1e-30
    x[3] = 1e-44  # the scale underflows
    x[4, 0, 3] = np.nan
    x[5, 0, 60] = np.inf
    x[6, 0, 0] = -np.inf
    x[7] = np.float32(1) / 3
    cache, _, _ = fresh(rng, "int8", [0], [9], 1, D, 4)
    d = T.from_numpy(x).cuda()
    w4().kv_append(cache, d, d, cu_tokens=T.tensor([0, 9], dtype=T.int32, device="cuda"))
    gk, _ = read_rows(cache, 0, 9)
    for t in (0, 1, 2, 7, 8):
        assert np.array_equal(gk[t], as_stored(x[t], "int8")), t
    assert np.all(np.abs(gk[3]) <= 127 * 1e-44)
    for t in (4, 5, 6):
        assert np.all(np.isnan(gk[t])), t


@pytest.mark.parametrize("kind", ["float16", "bfloat16"])
def test_append_16_bit_edges(kind):
    T = torch()
    rng = np.random.default_rng(15)
    v = np.array([0.0, -0.0, 65504.0, 65519.0, 65520.0, -1e30, 3e-8, 6e-8, 1 + 2.0 ** -9, 1 + 3 * 2.0 ** -9, 3.4e38,
                  np.inf, -np.inf, 1 + 2.0 ** -11, 1 + 3 * 2.0 ** -11, 1e-40], np.float32)
    cache, _, _ = fresh(rng, kind, [0], [1], 1, 16, 4)
    d = T.from_numpy(v.reshape(1, 1, 16)).cuda()
    w4().kv_append(cache, d, d)
    gk, _ = read_rows(cache, 0, 1)
    assert np.array_equal(gk.ravel(), as_stored(v, kind).ravel())


def test_append_beyond_the_capacity_and_broken_pages():
    T = torch()
    rng = np.random.default_rng(16)
    cache, k, _ = build(rng, "float32", [30, 32], 2, 16, 16)
    x = rng.standard_normal((8, 2, 16)).astype(np.float32)
    d = T.from_numpy(x).cuda()
    cu = T.tensor([0, 5, 8], dtype=T.int32, device="cuda")
    clear_error()
    w4().kv_append(cache, d, d, cu_tokens=cu)
    assert error_status() == 8  # 30 + 5 > 32, 32 + 3 > 32
    assert cache.lengths.tolist() == [32, 32]
    gk, _ = read_rows(cache, 0, 32)
    assert np.array_equal(gk[:30], k[0]) and np.array_equal(gk[30:], x[:2].astype(np.float64))
    gk, _ = read_rows(cache, 1, 32)
    assert np.array_equal(gk, k[1])
    # no page: nothing is written, the error word says so
    cache.page_table[0, 1] = 1000
    cache.lengths.copy_(T.tensor([20, 5], dtype=T.int32))
    before = cache.k.clone()
    w4().kv_append(cache, d[:1].expand(2, 2, 16).contiguous(), d[:2], lengths_out=T.empty(2, dtype=T.int32, device="cuda"))
    assert error_status() == 8
    # sequence 1 was written at slot 5, the rest is untouched
    p = int(cache.page_table[1, 0])
    assert np.array_equal(cache.k[p, :, 5].cpu().numpy(), x[0])
    cache.k[p, :, 5] = before[p, :, 5]
    assert T.equal(cache.k.view(T.int32), before.view(T.int32))
    # a descending cu_tokens gives no rows to its sequence
    cache.lengths.copy_(T.tensor([3, 5], dtype=T.int32))
    w4().kv_append(cache, d, d, cu_tokens=T.tensor([4, 2, 2], dtype=T.int32, device="cuda"))
    assert error_status() == 8 and cache.lengths.tolist() == [3, 5]


def test_append_counts_only_rows_that_are_there():
    T = torch()
    rng = np.random.default_rng(17)
    cache, k, _ = build(rng, "float32", [30, 32], 2, 16, 16)
    x = rng.standard_normal((4, 2, 16)).astype(np.float32)
    d = T.from_numpy(x).cuda()
    cache.lengths.copy_(T.tensor([3, 5], dtype=T.int32))
    clear_error()
    w4().kv_append(cache, d, d, cu_tokens=T.tensor([-2, 2, 100], dtype=T.int32, device="cuda"))
    assert error_status() == 8 and cache.lengths.tolist() == [5, 7]
    for b, n in enumerate((3, 5)):
        gk, _ = read_rows(cache, b, n + 2)
        assert np.array_equal(gk[:n], k[b][:n]) and np.array_equal(gk[n:], x[2 * b:2 * b + 2].astype(np.float64))


def test_append_nothing():
    T = torch()
    rng = np.random.default_rng(18)
    cache, _, _ = build(rng, "bfloat16", [3, 4], 2, 16, 16)
    d = T.zeros((0, 2, 16), device="cuda")
    out = T.full((2,), -1, dtype=T.int32, device="cuda")
    clear_error()
    w4().kv_append(cache, d, d, cu_tokens=T.zeros(3, dtype=T.int32, device="cuda"), lengths_out=out)
    assert out.tolist() == [3, 4] and error_status() == 0


def test_append_in_a_graph():
    """A captured step is replayed: each replay appends at the new end."""
    T = torch()
    rng = np.random.default_rng(19)
    cache, _, _ = fresh(rng, "float16", [2, 0], [6, 6], 2, 32, 4)
    x = T.zeros((2, 2, 32), device="cuda")
    cu = T.tensor([0, 1, 2], dtype=T.int32, device="cuda")
    g = T.cuda.CUDAGraph()
    with T.cuda.graph(g):
        w4().kv_append(cache, x, x)
        w4().kv_append(cache, x, x, cu_tokens=cu)
    vals = []
    for _ in range(3):
        r = rng.standard_normal((2, 2, 32)).astype(np.float32)
        x.copy_(T.from_numpy(r))
        vals += [r, r]
        g.replay()
        T.cuda.synchronize()
    assert cache.lengths.tolist() == [8, 6]
    for b, past in enumerate((2, 0)):
        gk, gv = read_rows(cache, b, past + 6)
        want = np.stack([as_stored(r[b], "float16") for r in vals])
        assert np.array_equal(gk[past:], want) and np.array_equal(gv[past:], want)


def test_append_refusals():
    T = torch()
    rng = np.random.default_rng(20)
    cache, _, _ = build(rng, "float32", [3, 4], 2, 16, 16)
    x = T.zeros((2, 2, 16), device="cuda")
    for k, v in ((x.half(), x), (x, x[:1]), (x[:, :1], x), (x.cpu(), x), (x[..., :8], x)):
        with pytest.raises(ValueError):
            w4().kv_append(cache, k, v)
    with pytest.raises(w4().W4Error):
        w4().kv_append(cache, x[:1], x[:1])  # one row for two sequences
    with pytest.raises(ValueError):
        w4().kv_append(cache, x, x, cu_tokens=T.zeros(2, dtype=T.int32, device="cuda"))
    with pytest.raises(ValueError):
        w4().kv_append(cache, x, x, lengths_out=T.zeros(2, dtype=T.int64, device="cuda"))
    lengths = T.zeros(3, dtype=T.int32, device="cuda")
    c2 = w4().KvCache(cache.k, cache.v, cache.page_table, lengths[:2])
    with pytest.raises(w4().W4Error):
        w4().kv_append(c2, x, x, lengths_out=lengths[1:])  # overlaps the lengths in part
    shared = w4().KvCache(cache.k, cache.v, cache.page_table[:1].expand(2, 1), cache.lengths)
    with pytest.raises(w4().W4Error):
        w4().kv_append(shared, x, x)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("form", ["one each", "one each, elsewhere", "prompts", "prompts, elsewhere"])
def test_append_to_a_negative_length_writes_nothing(kind, form):
    """A length below 0 is no place: its sequence's rows are not written, the
    length stays as it is, the error word says so; others advance."""
    T = torch()
    rng = np.random.default_rng(21)
    cache, _, _ = build(rng, kind, [20, 20, 20], 2, 32, 16)
    start = [-1, 4, -2 ** 31]
    cache.lengths.copy_(T.tensor(start, dtype=T.int32))
    x = rng.standard_normal((3, 2, 32)).astype(np.float32)
    d = T.from_numpy(x).cuda()
    stores = [t for t in (cache.k, cache.v, cache.k_scales, cache.v_scales) if t is not None]
    before = [t.clone() for t in stores]
    cu = T.tensor([0, 1, 2, 3], dtype=T.int32, device="cuda") if "prompts" in form else None
    out = T.full((3,), 77, dtype=T.int32, device="cuda") if "elsewhere" in form else None
    clear_error()
    got = w4().kv_append(cache, d, d, cu_tokens=cu, lengths_out=out)
    assert error_status() == 8
    assert got.tolist() == [-1, 5, -2 ** 31]
    assert cache.lengths.tolist() == (start if out is not None else got.tolist())
    p = int(cache.page_table[1, 0])
    s = None if cache.k_scales is None else cache.k_scales[p, :, 4].cpu().numpy()
    assert np.array_equal(oracle.kv_values(cache.k[p, :, 4].float().cpu().numpy(), s), as_stored(x[1], kind))
    for t, b in zip(stores, before):
        t[p, :, 4] = b[p, :, 4]
        assert T.equal(t.view(T.uint8), b.view(T.uint8))
