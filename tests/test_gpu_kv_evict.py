"""GPU tests of kv_evict: the kept slots exactly, rows and weights moved bit
for bit, in place and into other pages."""

import numpy as np
import pytest

import oracle
from kv_util import KINDS, build, clear_error, error_status, read_rows, torch, w4

pytestmark = pytest.mark.gpu


def weights(rng, lengths, width, ties=False):
    acc = np.zeros((len(lengths), width), np.float32)
    for b, n in enumerate(lengths):
        acc[b, :n] = rng.random(n) ** 6 * 30
        if ties:
            acc[b, :n] = np.floor(acc[b, :n])
    return acc


def run(kind, lengths, keep, recent, heads=2, dim=64, page=16, in_place=False, ties=False, seed=0, acc=None):
    T = torch()
    rng = np.random.default_rng(seed)
    cache, k, v = build(rng, kind, lengths, heads, dim, page)
    if acc is None:
        acc = weights(rng, lengths, cache.capacity, ties)
    accd = T.from_numpy(acc).cuda()
    B = len(lengths)
    kept = T.full((B, keep + 2), 77, dtype=T.int32, device="cuda")
    dst, acc_out = None, accd
    if not in_place:
        dst, _, _ = build(rng, kind, [min(n, keep) for n in lengths], heads, dim, page)
        dst.lengths.fill_(-1)
        acc_out = T.full((B, cache.capacity), 5.0, device="cuda")
    clear_error()
    got = w4().kv_evict(cache, accd, keep, recent=recent, dst=dst, acc_out=None if in_place else acc_out, kept=kept)
    assert error_status() == 0
    to = dst if dst is not None else cache
    want = [oracle.kv_evict_ref(acc[b], n, keep, recent) for b, n in enumerate(lengths)]
    assert got.tolist() == [len(j) for j in want]
    kc, ao = kept.cpu().numpy(), acc_out.cpu().numpy()
    for b, j in enumerate(want):
        n, m = lengths[b], len(j)
        assert kc[b, :m].tolist() == j, (b, n)
        assert np.all(kc[b, m:keep] == -1) and np.all(kc[b, keep:] == 77)
        gk, gv = read_rows(to, b, m)
        assert np.array_equal(gk, k[b][j]) and np.array_equal(gv, v[b][j]), (b, n)
        assert np.array_equal(ao[b, :m], acc[b, j], equal_nan=True)
        assert np.all(ao[b, m:n] == 0)
        assert np.all(ao[b, n:] == (0 if in_place else 5.0))
    if not in_place:  # the source is as it was
        assert cache.lengths.tolist() == lengths
        for b, n in enumerate(lengths):
            gk, gv = read_rows(cache, b, n)
            assert np.array_equal(gk, k[b]) and np.array_equal(gv, v[b])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("keep,recent", [(50, 10), (1, 0), (1, 1), (64, 64), (128, 200), (33, 0)])
def test_evict(kind, in_place, keep, recent):
    run(kind, [0, 1, 32, 33, 50, 51, 64, 65, 129, 500], keep, recent, in_place=in_place, seed=keep)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("heads,dim,page,kind", [(12, 64, 16, "float32"), (3, 96, 7, "float16"), (1, 256, 33, "float32"),
                                                 (2, 16, 1, "int8"), (1, 80, 16, "int8"), (5, 112, 3, "bfloat16")])
def test_evict_layouts(in_place, heads, dim, page, kind):
    run(kind, [300, 77, 140], 100, 20, heads, dim, page, in_place, seed=dim)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_ties_go_to_the_lower_slot(in_place):
    run("float32", [200, 900, 40], 37, 5, ties=True, in_place=in_place, seed=3)
    run("float32", [200, 900, 40], 37, 5, in_place=in_place, acc=np.zeros((3, 912), np.float32))


def test_evict_negative_infinite_and_nan_weights():
    rng = np.random.default_rng(5)
    acc = rng.standard_normal((4, 304)).astype(np.float32)
    acc[0, 5::7] = np.nan
    acc[1, ::3] = -np.inf
    acc[1, 1::3] = np.inf
    acc[2, :] = np.nan
    acc[3, ::2] = 0.0
    acc[3, 1::2] = -0.0
    for keep, recent in ((40, 3), (290, 0), (299, 1)):
        run("float32", [300, 300, 300, 300], keep, recent, acc=acc)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n,keep", [(20000, 5000), (70001, 69000), (9000, 1), (150003, 40001)])
def test_evict_one_long_sequence(in_place, n, keep):
    """Lengths that a cluster of CTAs shares."""
    run("bfloat16", [n], keep, keep // 10, heads=1, dim=32, in_place=in_place, seed=n)


def test_evict_everything():
    T = torch()
    rng = np.random.default_rng(6)
    cache, _, _ = build(rng, "float32", [30, 5], 2, 16, 16)
    acc = T.ones((2, 32), device="cuda")
    clear_error()
    assert w4().kv_evict(cache, acc, 0, recent=4).tolist() == [0, 0]
    assert error_status() == 0
    assert T.count_nonzero(acc[0, :30]) == 0 and T.count_nonzero(acc[1, :5]) == 0


def test_evict_into_too_few_pages_is_recorded():
    T = torch()
    rng = np.random.default_rng(7)
    cache, k, _ = build(rng, "float32", [100, 20], 2, 16, 16)
    dst, _, _ = build(rng, "float32", [32, 32], 2, 16, 16)
    acc = T.from_numpy(weights(rng, [100, 20], 112)).cuda()
    clear_error()
    got = w4().kv_evict(cache, acc, 50, dst=dst, acc_out=T.zeros((2, 112), device="cuda"))
    assert error_status() == 8 and got.tolist() == [32, 20]
    j = oracle.kv_evict_ref(acc[0].cpu().numpy(), 100, 50, 0)[:32]
    assert np.array_equal(read_rows(dst, 0, 32)[0], k[0][j])
    assert np.array_equal(read_rows(dst, 1, 20)[0], k[1])


def test_evict_in_a_graph_and_twice():
    """Replayed eviction: the second replay finds nothing left to evict."""
    T = torch()
    rng = np.random.default_rng(8)
    lengths = [200, 90, 64]
    cache, k, _ = build(rng, "float16", lengths, 2, 32, 16)
    acc = weights(rng, lengths, cache.capacity)
    accd = T.from_numpy(acc).cuda()
    g = T.cuda.CUDAGraph()
    with T.cuda.graph(g):
        w4().kv_evict(cache, accd, 64, recent=16)
    for _ in range(2):
        g.replay()
        T.cuda.synchronize()
        assert cache.lengths.tolist() == [64, 64, 64]
        for b, n in enumerate(lengths):
            j = oracle.kv_evict_ref(acc[b], n, 64, 16)
            assert np.array_equal(read_rows(cache, b, 64)[0], k[b][j])


def test_evict_refusals():
    T = torch()
    rng = np.random.default_rng(9)
    cache, _, _ = build(rng, "float32", [30, 5], 2, 16, 16)
    acc = T.ones((2, 32), device="cuda")
    W = w4()
    for kw in (dict(keep=-1), dict(keep=3, recent=-1)):
        with pytest.raises(W.W4Error):
            W.kv_evict(cache, acc, **kw)
    with pytest.raises(ValueError):
        W.kv_evict(cache, T.ones((2, 31), device="cuda"), 3)
    with pytest.raises(ValueError):
        W.kv_evict(cache, acc, 3, kept=T.zeros((2, 2), dtype=T.int32, device="cuda"))
    other, _, _ = build(rng, "float32", [30, 5], 2, 32, 16)
    with pytest.raises(W.W4Error):
        W.kv_evict(cache, acc, 3, dst=other)
    half = W.KvCache(cache.k, cache.v, cache.page_table.clone(), cache.lengths.clone())
    with pytest.raises(W.W4Error):  # the same pages by another table
        W.kv_evict(cache, acc, 3, dst=half)
    free, _, _ = build(rng, "float32", [30, 5], 2, 16, 16)
    with pytest.raises(W.W4Error):  # the same lengths
        W.kv_evict(cache, acc, 3, dst=W.KvCache(free.k, free.v, free.page_table, cache.lengths))
    shared = W.KvCache(free.k, free.v, free.page_table[:1].expand(2, 2), free.lengths)
    with pytest.raises(W.W4Error):
        W.kv_evict(cache, acc, 3, dst=shared, acc_out=T.zeros((2, 32), device="cuda"))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lengths,keep,recent", [([100, 40, 64], 50, 10), ([100, 40, 64], 300, 0), ([100, 40, 64], 20, 20),
                                                 ([9000, 40, 70], 3000, 200), ([150003], 20011, 5000)])
def test_evict_drops_kept_slots_of_broken_pages(kind, in_place, lengths, keep, recent):
    """Slots whose page id names no page count as empty: none is kept, what is
    kept closes up, and the length counts that alone."""
    T = torch()
    if len(lengths) == 1 and kind in ("float32", "float16"):
        pytest.skip("the long sequence once for 16 bits, once with scales")
    rng = np.random.default_rng(len(lengths) * 10 + keep)
    page, heads, dim = 16, 1 if max(lengths) > 1000 else 2, 16
    cache, k, v = build(rng, kind, lengths, heads, dim, page)
    acc = weights(rng, lengths, cache.capacity)
    B, table = len(lengths), cache.page_table.cpu().numpy()
    bad = {0: [3, 5, lengths[0] // page], 1: [0]}  # of sequence 0 the last one too; sequence 2 is whole
    if B == 1:
        bad = {0: [1, 700, 9000, lengths[0] // page]}
    for b, pages in bad.items():
        for i, p in enumerate(pages):
            cache.page_table[b, p] = (-1, cache.k.shape[0], 2 ** 31 - 1, -2 ** 31)[i]
    accd = T.from_numpy(acc).cuda()
    kept = T.full((B, keep + 1), 77, dtype=T.int32, device="cuda")
    dst = None
    if not in_place:
        dst, _, _ = build(rng, kind, [min(n, keep) for n in lengths], heads, dim, page)
    for with_kept in (True, False):
        if not with_kept and in_place:
            break  # the cache has been cut
        acc_out = accd if in_place else T.full((B, cache.capacity), 5.0, device="cuda")
        clear_error()
        got = w4().kv_evict(cache, accd, keep, recent=recent, dst=dst, acc_out=acc_out, kept=kept if with_kept else None)
        assert error_status() == 8
        want = []
        for b, n in enumerate(lengths):
            j = np.array(oracle.kv_evict_ref(acc[b], n, keep, recent))
            want.append(j[~np.isin(j // page, bad.get(b, []))])
        assert got.tolist() == [len(j) for j in want]
        to = dst if dst is not None else cache
        to_table = to.page_table.cpu().numpy()
        kc, ao = kept.cpu().numpy(), acc_out.cpu().numpy()
        for b, j in enumerate(want):
            n, m = lengths[b], len(j)
            if with_kept:
                assert np.array_equal(kc[b, :m], j) and np.all(kc[b, m:keep] == -1) and np.all(kc[b, keep:] == 77)
            assert np.array_equal(ao[b, :m], acc[b, j]) and np.all(ao[b, m:n] == 0)
            assert np.all(ao[b, n:] == (0 if in_place else 5.0))
            r = np.arange(m)
            there = r if not in_place else r[~np.isin(r // page, bad.get(b, []))]  # in place the broken pages hold nothing
            p = to_table[b, there // page]
            for t, sc, rows in ((to.k, to.k_scales, k), (to.v, to.v_scales, v)):
                x = t.cpu().double().numpy()[p, :, there % page]
                s = None if sc is None else sc.cpu().numpy()[p, :, there % page]
                assert np.array_equal(oracle.kv_values(x, s), rows[b][j[there]]), b


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n", [9000, 40000, 150003])
@pytest.mark.parametrize("steps", [1, 4, 0])
def test_evict_ties_over_a_cluster(in_place, n, steps):
    """A threshold that many slots of several CTAs share, of which only part
    stay: few different weights, and all alike."""
    rng = np.random.default_rng(n + steps)
    cap = -(-n // 16) * 16
    acc = np.zeros((1, cap), np.float32)
    if steps:
        acc[0, :n] = np.floor(rng.random(n) * (steps + 1))
    for keep, recent in ((n // 3, 100), (n - 5, 0), (n // 2, n // 2)):
        run("bfloat16", [n], keep, recent, heads=1, dim=16, in_place=in_place, acc=acc, seed=n)


@pytest.mark.parametrize("kind,heads", [("int8", 3), ("float32", 4), ("bfloat16", 5)])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("recent", [0, 1200, 5000])
def test_evict_many_rows_of_several_heads(kind, heads, in_place, recent):
    """More rows than a batch, of several heads and with scales; recent >= keep
    asks nothing of the weights."""
    run(kind, [5000, 9000, 1100, 1201], 1200, recent, heads, 64, 16, in_place, seed=recent + heads)
