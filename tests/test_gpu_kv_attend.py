"""GPU parity of kv_attend against the fp64 definition: element types, head
layouts, page sizes, lengths from none to several splits, windows, strides,
gathered weights, graphs, streams and broken descriptors."""

import numpy as np
import pytest

import oracle
from kv_util import KINDS, build, clear_error, error_status, torch, w4

pytestmark = pytest.mark.gpu


def check(cache, rows_k, rows_v, q, window=0, scale=None, with_acc=False, strided=False, what=""):
    T = torch()
    B, Hq, D = q.shape
    clear_error()
    scale = D ** -0.5 if scale is None else scale
    if strided:  # q and out as columns of wider rows, the columns around out untouched
        wide = T.full((B, Hq * D + 40), float("nan"), device="cuda")
        wide[:, 8:8 + Hq * D] = T.from_numpy(q.reshape(B, -1)).cuda()
        qd = wide[:, 8:8 + Hq * D].view(B, Hq, D)
        obuf = T.full((B, Hq * D + 12), 7.0, device="cuda")
        out = obuf[:, 4:4 + Hq * D].view(B, Hq, D)
    else:
        qd, out = T.from_numpy(q).cuda(), T.full((B, Hq, D), float("nan"), device="cuda")
    lse = T.full((B, Hq), float("nan"), device="cuda")
    acc = acc0 = None
    if with_acc:
        acc0 = np.random.default_rng(5).random((B, cache.capacity + 3)).astype(np.float32)
        acc = T.from_numpy(acc0).cuda()
    w4().kv_attend(qd, cache, scale=scale, window=window, out=out, lse=lse, acc=acc)
    assert error_status() == 0, what
    got, gl = out.cpu().double().numpy(), lse.cpu().double().numpy()
    for b in range(B):
        ro, rl, rw, (to, tl, tw) = oracle.kv_attend_ref(q[b], rows_k[b], rows_v[b], scale, window)
        off = np.abs(got[b] - ro)
        assert np.all(off <= to), f"{what} seq {b}: out off by {np.nanmax(off / np.maximum(to, 1e-300)):.3g} bounds"
        if len(rows_k[b]) == 0:
            assert np.all(gl[b] == -np.inf)
        else:
            assert np.all(np.abs(gl[b] - rl) <= tl), (what, b, np.abs(gl[b] - rl).max(), tl.max())
        if with_acc:
            ga, n = acc[b].cpu().double().numpy(), rw.shape[1]
            want = acc0[b].astype(np.float64)
            assert np.array_equal(ga[n:], want[n:]), f"{what} seq {b}: weights behind the last slot changed"
            full = want[:n] + rw.sum(0)
            tol = tw.sum(0) + (Hq + 1) * oracle.EPS * full
            assert np.all(np.abs(ga[:n] - full) <= tol), (what, b)
    if strided:
        o = obuf.cpu().numpy()
        assert np.all(o[:, :4] == 7.0) and np.all(o[:, 4 + Hq * D:] == 7.0)
    return out


# Slots that a sequence may grow to: few (an item is a cluster of CTAs) and many
# (runs of units, joined behind them).
ROOMS = [0, 20000]


def room_for(slots, page):
    return -(-slots // page) if slots else None


@pytest.mark.parametrize("room", ROOMS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,group,dim,page", [
    (12, 1, 64, 16), (3, 1, 96, 7), (2, 2, 128, 32), (2, 3, 48, 5), (1, 4, 128, 64), (2, 8, 64, 16), (1, 5, 80, 1),
    (1, 16, 32, 3), (2, 7, 112, 33), (1, 1, 256, 16), (1, 9, 256, 20), (2, 1, 16, 4), (1, 4, 192, 8), (1, 6, 96, 16),
    (1, 2, 160, 16), (1, 12, 128, 16), (2, 3, 256, 16), (1, 8, 192, 7), (1, 5, 160, 16), (1, 4, 224, 16), (2, 8, 256, 5),
])
def test_attend_matches_the_definition(kind, heads, group, dim, page, room):
    rng = np.random.default_rng(heads * 1000 + group * 100 + dim + page)
    lengths = [0, 1, 2, 15, 16, 17, 63, 64, 65, 130, 301]
    cache, k, v = build(rng, kind, lengths, heads, dim, page, max_pages=room_for(room, page))
    q = rng.standard_normal((len(lengths), heads * group, dim)).astype(np.float32)
    check(cache, k, v, q, with_acc=True, strided=True, what=f"{kind} {heads}x{group}x{dim}")


@pytest.mark.parametrize("room", ROOMS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 5, 64, 100, 5000])
def test_attend_window(kind, window, room):
    rng = np.random.default_rng(window)
    lengths = [0, 1, 99, 100, 101, 333, 700]
    cache, k, v = build(rng, kind, lengths, 2, 64, 16, max_pages=room_for(room, 16))
    q = rng.standard_normal((len(lengths), 4, 64)).astype(np.float32)
    check(cache, k, v, q, window=window, with_acc=True, what=f"window {window}")


@pytest.mark.parametrize("kind,heads,group,dim,n", [
    ("float32", 1, 1, 64, 20011), ("bfloat16", 2, 4, 128, 30000), ("int8", 1, 8, 128, 40003), ("float16", 1, 1, 96, 9001),
    ("float16", 1, 8, 256, 1900), ("bfloat16", 1, 8, 256, 900), ("int8", 1, 4, 192, 3000), ("float32", 1, 8, 256, 800),
    ("bfloat16", 1, 4, 128, 1000), ("int8", 2, 8, 64, 1024), ("float32", 1, 1, 256, 700),
])
def test_attend_one_long_sequence_is_split_and_joined(kind, heads, group, dim, n):
    """Of one sequence: 16 CTAs and more share an item."""
    rng = np.random.default_rng(n)
    cache, k, v = build(rng, kind, [n], heads, dim, 64)
    q = (rng.standard_normal((1, heads * group, dim)) * 2).astype(np.float32)
    check(cache, k, v, q, with_acc=True, what=f"{kind} {n}")


@pytest.mark.parametrize("room", ROOMS)
@pytest.mark.parametrize("kind", ["float32", "int8"])
def test_attend_many_sequences(kind, room):
    """More sequences than one pass of the run search takes, some empty."""
    rng = np.random.default_rng(17)
    lengths = [int(x) for x in rng.integers(0, 90, 300)]
    lengths[0] = lengths[127] = lengths[128] = lengths[299] = 0
    cache, k, v = build(rng, kind, lengths, 2, 64, 16, max_pages=room_for(room, 16))
    q = rng.standard_normal((300, 4, 64)).astype(np.float32)
    check(cache, k, v, q, what="300 sequences")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group,dim", [(1, 64), (3, 64), (8, 128), (5, 256), (13, 16)])
def test_attend_few_slots(kind, group, dim):
    """Sequences of at most one tile, in a small and in a large batch, and a
    small batch of a few tiles: the plain lanes for any group."""
    rng = np.random.default_rng(group + dim)
    for n, most, heads in ((3, 16, 2), (500, 16, 3), (2, 250, 2)):
        lengths = [int(x) for x in rng.integers(0, most + 1, n)]
        lengths[-1] = most
        cache, k, v = build(rng, kind, lengths, heads, dim, 16)
        q = rng.standard_normal((n, heads * group, dim)).astype(np.float32)
        check(cache, k, v, q, with_acc=n < 10, what=f"few slots {kind} {group}x{dim} {n}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("group,dim", [(1, 64), (2, 32), (3, 96), (8, 128), (16, 48), (5, 192)])
def test_attend_many_short_items(kind, group, dim):
    """More items than CTAs at once, all of them short: a warp for each."""
    rng = np.random.default_rng(group * 100 + dim)
    heads, n = 3, 400
    lengths = [int(x) for x in rng.integers(0, 50, n)]
    lengths[0] = lengths[1] = lengths[-1] = 0
    cache, k, v = build(rng, kind, lengths, heads, dim, 16, max_pages=4)
    q = rng.standard_normal((n, heads * group, dim)).astype(np.float32)
    check(cache, k, v, q, with_acc=True, strided=True, what=f"short {kind} {group}x{dim}")
    check(cache, k, v, q, window=9, what=f"short {kind} {group}x{dim} window")


@pytest.mark.parametrize("room", ROOMS)
@pytest.mark.parametrize("kind", KINDS)
def test_attend_large_scores_and_values(kind, room):
    """Scores of +-100 and more, values of very different magnitude: the
    running maximum rescales, and each rescaling keeps its precision."""
    rng = np.random.default_rng(3)
    for heads, group in ((2, 1), (1, 8)):
        cache, k, v = build(rng, kind, [257, 64, 1000], heads, 64, 16, amp=6.0, max_pages=room_for(room, 16))
        q = (rng.standard_normal((3, heads * group, 64)) * 5).astype(np.float32)
        check(cache, k, v, q, scale=0.3, with_acc=True, what="large scores")
        check(cache, k, v, q, scale=-0.3, what="negative scale")
        check(cache, k, v, q, scale=0.0, what="zero scale: the mean of the values")
        check(cache, k, v, (q * 1e-30).astype(np.float32), what="tiny queries")
        check(cache, k, v, (q * 0).astype(np.float32), what="zero queries")


def test_attend_int8_scales_of_any_size():
    """int8 rows whose scales span 1e-6 .. 1e5, zero scales among them."""
    T = torch()
    rng = np.random.default_rng(8)
    for group in (1, 8):
        lengths = [100, 700]
        cache, k, v = build(rng, "int8", lengths, 2, 64, 16)
        for t in (cache.k_scales, cache.v_scales):
            f = T.from_numpy((10.0 ** rng.uniform(-6, 5, tuple(t.shape))).astype(np.float32)).cuda()
            t.mul_(f if t is cache.v_scales else f.clamp(max=10.0))
            t[:, :, 0] *= 0.0
        # slot 0 of a page that no sequence holds is NaN * 0 and stays NaN
        from kv_util import read_rows
        rows = [read_rows(cache, b, n) for b, n in enumerate(lengths)]
        q = rng.standard_normal((2, 2 * group, 64)).astype(np.float32)
        check(cache, [r[0] for r in rows], [r[1] for r in rows], q, with_acc=True, what="scales")


@pytest.mark.parametrize("kind", KINDS)
def test_attend_pages_far_apart_and_shared(kind):
    """Pages with others between them, and one row of pages that "sequences"
    of lengths 1 .. T share: a prompt attended causally."""
    rng = np.random.default_rng(23)
    cache, k, v = build(rng, kind, [77, 130], 2, 64, 16, gap=2)
    q = rng.standard_normal((2, 2, 64)).astype(np.float32)
    check(cache, k, v, q, what="gaps")
    T_len = 58
    cache, k, v = build(rng, kind, list(range(1, T_len + 1)), 2, 64, 16, shared=True)
    assert cache.page_table.stride(0) == 0
    q = rng.standard_normal((T_len, 4, 64)).astype(np.float32)
    check(cache, k, v, q, with_acc=True, what="causal prompt")


def test_attend_offsets_beyond_32_bits():
    """Pages whose elements lie more than 2^32 elements (and bytes) in."""
    T = torch()
    rng = np.random.default_rng(31)
    H, S, D = 2, 16, 64
    page = H * S * D
    far = (1 << 32) // page + 5
    k = T.empty((far + 1, H, S, D), dtype=T.float16, device="cuda")
    v = T.empty((far + 1, H, S, D), dtype=T.float16, device="cuda")
    x = rng.standard_normal((2, S, H, D)).astype(np.float16)
    ids = [far, 1]
    for i, p in enumerate(ids):
        k[p].copy_(T.from_numpy(np.ascontiguousarray(x[i].transpose(1, 0, 2))).cuda())
        v[p].copy_(T.from_numpy(np.ascontiguousarray(x[1 - i].transpose(1, 0, 2))).cuda())
    cache = w4().KvCache(k, v, T.tensor([ids], dtype=T.int32, device="cuda"), T.tensor([30], dtype=T.int32, device="cuda"))
    rows_k = x.reshape(32, H, D)[:30].astype(np.float64)
    rows_v = x[::-1].reshape(32, H, D)[:30].astype(np.float64)
    for group in (1, 8):
        q = rng.standard_normal((1, H * group, D)).astype(np.float32)
        check(cache, [rows_k], [rows_v], q, with_acc=True, what="far pages")


@pytest.mark.parametrize("room", ROOMS)
@pytest.mark.parametrize("kind,group", [("float32", 1), ("bfloat16", 4), ("int8", 8), ("float16", 8)])
def test_attend_nan_reaches_only_its_own_rows(kind, group, room):
    """A NaN in q, or Inf and NaN in an attended slot, makes the rows that it
    reaches non-finite and leaves every other row's bits as they were."""
    T = torch()
    rng = np.random.default_rng(41)
    cache, k, v = build(rng, kind, [150, 90, 33], 2, 64, 16, max_pages=room_for(room, 16))
    q = rng.standard_normal((3, 2 * group, 64)).astype(np.float32)
    base = check(cache, k, v, q, what="clean").cpu().numpy()
    bad = q.copy()
    bad[1, 0, 5] = np.nan
    out = w4().kv_attend(T.from_numpy(bad).cuda(), cache).cpu().numpy()
    assert np.all(np.isnan(out[1, 0]))
    keep = np.ones((3, 2 * group), bool)
    keep[1, 0] = False
    assert np.array_equal(out[keep], base[keep])
    p = int(cache.page_table[0, 2])
    if kind == "int8":
        cache.v_scales[p, 1, 3] = float("nan")
    else:
        cache.v[p, 1, 3, :] = float("inf")
    out = w4().kv_attend(T.from_numpy(q).cuda(), cache).cpu().numpy()
    assert not np.any(np.isfinite(out[0, group:]))
    assert np.array_equal(out[0, :group], base[0, :group]) and np.array_equal(out[1:], base[1:])


@pytest.mark.parametrize("room", ROOMS)
def test_attend_broken_pages_and_lengths_are_recorded(room):
    """A page id that names no page, and lengths outside the capacity: the
    error word says so, the slots concerned count as empty."""
    T = torch()
    rng = np.random.default_rng(51)
    for kind, group in (("float32", 1), ("bfloat16", 4), ("int8", 8)):
        cache, k, v = build(rng, kind, [40, 48], 2, 64, 16, max_pages=room_for(room, 16))
        q = rng.standard_normal((2, 2 * group, 64)).astype(np.float32)
        qd = T.from_numpy(q).cuda()
        clear_error()
        good = int(cache.page_table[0, 1])
        for broken in (-1, cache.k.shape[0], 2 ** 31 - 1):
            cache.page_table[0, 1] = broken
            out = w4().kv_attend(qd, cache).cpu().double().numpy()
            assert error_status() == 8
            j = np.r_[0:16, 32:40]
            ro, _, _, (to, _, _) = oracle.kv_attend_ref(q[0], k[0][j], v[0][j], 0.125)
            assert np.all(np.abs(out[0] - ro) <= to)
        cache.page_table[0, 1] = good
        # entries behind the last page name none: a length beyond the capacity ends there
        cache.lengths.copy_(T.tensor([-5, cache.capacity + 1], dtype=T.int32))
        out = w4().kv_attend(qd, cache).cpu().double().numpy()
        assert error_status() == 8
        assert np.all(out[0] == 0)
        ro, _, _, (to, _, _) = oracle.kv_attend_ref(q[1], k[1], v[1], 0.125)
        assert np.all(np.abs(out[1] - ro) <= to)


@pytest.mark.parametrize("room", ROOMS)
@pytest.mark.parametrize("kind,group", [("float32", 1), ("float16", 4)])
def test_attend_in_a_graph_follows_the_lengths(kind, group, room):
    """A captured call is replayed while the lengths change, two captured
    calls are replayed on two streams at once, and every result is bit for bit
    what an eager call gives."""
    T = torch()
    rng = np.random.default_rng(61)
    cache, k, v = build(rng, kind, [500, 3, 260], 2, 64, 16, max_pages=room_for(room, 16))
    q = T.from_numpy(rng.standard_normal((3, 2 * group, 64)).astype(np.float32)).cuda()
    q2 = T.from_numpy(rng.standard_normal((3, 2 * group, 64)).astype(np.float32)).cuda()
    w4().kv_attend(q, cache)
    T.cuda.synchronize()
    graphs = []
    for x in (q, q2):
        g = T.cuda.CUDAGraph()
        with T.cuda.graph(g):
            out = w4().kv_attend(x, cache)
        graphs.append((g, out))
    streams = [T.cuda.Stream(), T.cuda.Stream()]
    for lengths in ([500, 3, 260], [1, 0, 0], [0, 0, 0], [499, 2, 17]):
        cache.lengths.copy_(T.tensor(lengths, dtype=T.int32))
        T.cuda.synchronize()
        for _ in range(20):
            for (g, _), s in zip(graphs, streams):
                with T.cuda.stream(s):
                    g.replay()
        T.cuda.synchronize()
        for (g, out), x in zip(graphs, (q, q2)):
            assert T.equal(out, w4().kv_attend(x, cache))


def test_attend_on_a_stream_of_its_own():
    T = torch()
    rng = np.random.default_rng(71)
    cache, k, v = build(rng, "bfloat16", [300, 200], 2, 64, 16)
    q = T.from_numpy(rng.standard_normal((2, 2, 64)).astype(np.float32)).cuda()
    want = w4().kv_attend(q, cache)
    T.cuda.synchronize()
    s = T.cuda.Stream()
    outs = [w4().kv_attend(q, cache, stream=s) for _ in range(50)]
    mine = [w4().kv_attend(q, cache) for _ in range(50)]
    T.cuda.synchronize()
    assert all(T.equal(o, want) for o in outs + mine)


def test_attend_no_sequences_and_no_capacity():
    T = torch()
    k = T.zeros((1, 2, 16, 64), device="cuda")
    none = w4().KvCache(k, k.clone(), T.zeros((0, 3), dtype=T.int32, device="cuda"),
                        T.zeros(0, dtype=T.int32, device="cuda"))
    assert w4().kv_attend(T.zeros((0, 4, 64), device="cuda"), none).shape == (0, 4, 64)
    flat = w4().KvCache(k, k.clone(), T.zeros((2, 0), dtype=T.int32, device="cuda"),
                        T.zeros(2, dtype=T.int32, device="cuda"))
    out = w4().kv_attend(T.ones((2, 4, 64), device="cuda"), flat, acc=T.zeros((2, 0), device="cuda"))
    assert T.count_nonzero(out) == 0 and error_status() == 0


def test_attend_refusals():
    T = torch()
    rng = np.random.default_rng(81)
    cache, _, _ = build(rng, "float32", [40, 48], 2, 64, 16)
    q = T.zeros((2, 4, 64), device="cuda")
    for bad in (q[:1], q.half(), q[:, :, :32], q.cpu(), T.zeros((2, 4, 128), device="cuda")[:, :, ::2]):
        with pytest.raises(ValueError):
            w4().kv_attend(bad, cache)
    with pytest.raises(w4().W4Error):
        w4().kv_attend(T.zeros((2, 3, 64), device="cuda"), cache)  # 3 query heads over 2
    with pytest.raises(w4().W4Error):
        w4().kv_attend(q, cache, window=-1)
    with pytest.raises(w4().W4Error):
        w4().kv_attend(q, cache, scale=float("nan"))
    with pytest.raises(w4().W4Error) as e:
        w4().kv_attend(q, cache, acc=T.zeros((2, 48), device="cuda"), ws=T.empty(16, dtype=T.uint8, device="cuda"))
    assert e.value.status == 7
    with pytest.raises(ValueError):
        w4().kv_attend(q, cache, lse=T.zeros((2, 2), device="cuda"))
    with pytest.raises(ValueError):
        w4().kv_attend(q, cache, acc=T.zeros((2, 47), device="cuda"))
    with pytest.raises(ValueError):
        w4().kv_attend(q, cache, out=T.zeros((2, 4, 64), device="cuda").half())


def test_attend_workspace_refusals():
    T = torch()
    rng = np.random.default_rng(82)
    cache, _, _ = build(rng, "float32", [40, 48], 2, 64, 16)
    q, acc = T.zeros((2, 4, 64), device="cuda"), T.zeros((2, 48), device="cuda")
    room = 1 << 20
    for bad in (T.zeros(room, dtype=T.uint8), T.zeros(1, dtype=T.uint8, device="cuda").expand(room),
                T.zeros(2 * room, dtype=T.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            w4().kv_attend(q, cache, acc=acc, ws=bad)
        with pytest.raises(ValueError):
            w4().kv_evict(cache, acc, 8, ws=bad)
    own = T.full((room // 4,), float("nan"), device="cuda")
    want = w4().kv_attend(q, cache, acc=T.zeros_like(acc))
    assert T.equal(want, w4().kv_attend(q, cache, acc=acc, ws=own))


@pytest.mark.parametrize("kind,group", [("float32", 1), ("bfloat16", 1), ("bfloat16", 4), ("float32", 8), ("int8", 8)])
def test_attend_large_values(kind, group):
    """Values of 2^96 are averaged without overflow, whatever the scores do."""
    T = torch()
    rng = np.random.default_rng(83)
    n, heads, dim = 600, 2, 64
    cache, _, _ = build(rng, kind, [n], heads, dim, 16)
    k = T.randn((n, heads, dim), device="cuda", generator=T.Generator("cuda").manual_seed(5))
    k *= T.linspace(0.1, 3.0, n, device="cuda")[:, None, None]  # maxima that keep rising
    v = T.full((n, heads, dim), 2.0 ** 96, device="cuda")
    cache.lengths.zero_()
    w4().kv_append(cache, k, v, cu_tokens=T.tensor([0, n], dtype=T.int32, device="cuda"))
    q = T.randn((1, heads * group, dim), device="cuda", generator=T.Generator("cuda").manual_seed(6))
    out = w4().kv_attend(q, cache)
    # all values are alike: what differs is the rounding of two sums of 600 terms of one sign (each
    # term at most 600 x 2^-24 off in its sum), the pieces' 2^-21 and, for int8, one rounding of the scale
    bound = 2 * n * 2.0 ** -24 + 2.0 ** -20
    assert float((out / 2.0 ** 96 - 1).abs().max()) <= bound


@pytest.mark.parametrize("window", [0, 77])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,group,dim,page", [
    (2, 3, 48, 5), (1, 4, 128, 64), (2, 8, 64, 16), (1, 5, 80, 1), (1, 9, 256, 20), (1, 2, 160, 16), (2, 2, 256, 7),
    (1, 16, 96, 3), (1, 7, 192, 16),
])
def test_attend_short_sequences_in_long_rooms(kind, heads, group, dim, page, window):
    """Room for more slots than the plain lanes are taken for, few items: the
    matrices (where there are heads enough), an item a cluster."""
    rng = np.random.default_rng(heads * 1000 + group * 100 + dim + page + window)
    lengths = [0, 1, 2, 15, 16, 17, 33, 64, 65, 130, 301, 1100]
    cache, k, v = build(rng, kind, lengths, heads, dim, page, max_pages=room_for(1500, page))
    q = rng.standard_normal((len(lengths), heads * group, dim)).astype(np.float32)
    check(cache, k, v, q, window=window, with_acc=True, strided=True, what=f"{kind} {heads}x{group}x{dim}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [7, 160])
@pytest.mark.parametrize("window", [1, 20, 200, 1300])
def test_attend_window_decides_the_body(kind, n, window):
    """A window far below the room: another body and launch than without one,
    in the workspace that fits every window."""
    rng = np.random.default_rng(n + window)
    lengths = [int(x) for x in rng.integers(0, 1500, n)]
    lengths[0], lengths[-1] = 0, 1400
    cache, k, v = build(rng, kind, lengths, 2, 32, 16, max_pages=room_for(20000, 16))
    q = rng.standard_normal((n, 8, 32)).astype(np.float32)
    check(cache, k, v, q, window=window, with_acc=n < 10, what=f"window {window} of {n}")


def test_attend_most_sequences():
    """65535 of them, over one row of pages."""
    T = torch()
    B, cap, dim = 65535, 40, 16
    rng = np.random.default_rng(91)
    rows = rng.standard_normal((2, cap // 8, 1, 8, dim)).astype(np.float32)
    k, v = (T.from_numpy(x).cuda() for x in rows)
    table = T.arange(cap // 8, dtype=T.int32, device="cuda").view(1, -1).expand(B, -1)
    lengths = (T.arange(B, device="cuda") % (cap + 1)).to(T.int32)
    cache = w4().KvCache(k, v, table, lengths)
    q = T.from_numpy(rng.standard_normal((B, 2, dim)).astype(np.float32)).cuda()
    clear_error()
    out = w4().kv_attend(q, cache)
    assert error_status() == 0
    flat = rows.astype(np.float64).reshape(2, cap, 1, dim)
    for b in [*range(0, B, 1009), B - 1]:
        n = int(lengths[b])
        ro, _, _, (to, _, _) = oracle.kv_attend_ref(q[b].cpu().numpy(), flat[0, :n], flat[1, :n], dim ** -0.5)
        assert np.all(np.abs(out[b].cpu().double().numpy() - ro) <= to), b


@pytest.mark.parametrize("room", ROOMS)
@pytest.mark.parametrize("group,dim", [(1, 64), (4, 64), (8, 128), (5, 192), (8, 256)])
@pytest.mark.parametrize("where", ["zeros", "zeros first", "negligible", "outweighed"])
def test_attend_int8_scales_of_slots_that_add_nothing(where, group, dim, room):
    """Values of 1e-8 to 1e-11 beside slots whose large scale adds nothing:
    rows of zeros (stored with scale 1), one slot of negligible weight, and one
    that weighed everything until later slots outweighed it.

    Bound: the definition's (score errors, roundings of the sums) relative to
    sum w |v|; and what the weights' two fp16 pieces leave out, 2^-36 for each
    code (127 at most) while the largest product of a weight and a scale, rows
    of zeros aside, lies at 2^8 or above: 127 n 2^-44 of that product."""
    T = torch()
    rng = np.random.default_rng(group * dim)
    n, heads = 700, 2
    cache, _, _ = build(rng, "int8", [n], heads, dim, 16, max_pages=room_for(room, 16))
    k = rng.standard_normal((n, heads, dim)).astype(np.float32)
    v = (rng.standard_normal((n, heads, dim)) * 10.0 ** -rng.uniform(8, 11)).astype(np.float32)
    k[:, :, 0] = 0.0  # the queries' first element is such that this one is added to the score
    if where == "zeros":
        v[rng.integers(0, n, 60)] = 0.0
    elif where == "zeros first":
        v[:65] = 0.0
    elif where == "negligible":
        k[5, :, 0], v[5] = -40.0, v[5] * 1e13
    else:
        k[:n // 2, :, 0], v[5] = -40.0, v[5] * 1e10
    q = rng.standard_normal((1, heads * group, dim)).astype(np.float32)
    q[:, :, 0] = dim ** 0.5
    j = np.arange(n)
    page = T.from_numpy(cache.page_table[0].cpu().numpy()[j // 16].astype(np.int64)).cuda()
    inner = T.from_numpy(j % 16).cuda()
    rows = []
    for x, codes, scales in ((k, cache.k, cache.k_scales), (v, cache.v, cache.v_scales)):
        c, s = oracle.kv_store(x, "int8")
        codes[page, :, inner], scales[page, :, inner] = T.from_numpy(c).cuda(), T.from_numpy(s).cuda()
        rows.append((oracle.kv_values(c, s), np.where(c.any(-1), s, 0.0)))
    (k, _), (v, s) = rows
    out = w4().kv_attend(T.from_numpy(q).cuda(), cache).cpu().double().numpy()[0]
    ro, _, w, (_, _, tw) = oracle.kv_attend_ref(q[0], k, v, dim ** -0.5)
    for i in range(heads * group):
        h = i // group
        bound = tw[i] @ np.abs(v[:, h]) + 127 * n * 2.0 ** -44 * (w[i] * s[:, h]).max()
        off = np.abs(out[i] - ro[i])
        assert np.all(off <= bound), f"head {i}: off by {np.max(off / bound):.3g} bounds, {np.max(off) / np.abs(ro[i]).max():.3g} of the result"


@pytest.mark.parametrize("kind,group", [("bfloat16", 1), ("bfloat16", 4), ("bfloat16", 8), ("float16", 8), ("int8", 8),
                                        ("float32", 8)])
def test_attend_long_sums_of_one_sign_have_no_bias(kind, group):
    """Values of one sign over 65536 slots, about 2400 of them to a warp.

    Sums rounded to nearest are off to either side: a row's by a walk of at most
    1200 steps (a lane's weights; its values' tiles are fewer) of 2^-24, so by
    2.1e-6 in a row's standard deviation at most, and 9.2e-8 in the mean over the
    512 query heads here; ten of those are the bound, 2^-20. Cut off instead of
    rounded, each step would lose 2^-25 and more of the sum to one side."""
    T = torch()
    rng = T.Generator("cuda").manual_seed(3)
    B, H, n, D, page = 8, 8, 65536, 64, 64
    P, dt = n // page, getattr(T, kind)
    scales = (None, None)
    if kind == "int8":
        k, v = (T.randint(lo, 128, (P, H, page, D), generator=rng, device="cuda", dtype=T.int8) for lo in (-127, 40))
        scales = [T.rand((P, H, page), generator=rng, device="cuda") * 0.01 + 0.01 for _ in range(2)]
    else:
        k = T.randn((P, H, page, D), generator=rng, device="cuda").to(dt)
        v = (T.rand((P, H, page, D), generator=rng, device="cuda") + 0.5).to(dt)
    table = T.randperm(P, generator=rng, device="cuda").to(T.int32)
    cache = w4().KvCache(k, v, table.view(1, P).expand(B, P), T.full((B,), n, dtype=T.int32, device="cuda"), *scales)
    q = T.randn((B, H * group, D), generator=rng, device="cuda")
    out = w4().kv_attend(q, cache).double().view(B, H, group, D)
    off = []
    for h in range(H):
        kk, vv = (x[table.long(), h].double() * (1 if s is None else s[table.long(), h].double()[..., None])
                  for x, s in zip((k, v), scales))
        kk, vv = kk.reshape(n, D), vv.reshape(n, D)
        p = T.softmax(q.view(B, H, group, D)[:, h].double() @ kk.T * D ** -0.5, -1)
        off.append(out[:, h] / (p @ vv) - 1)
    off = T.stack(off)
    assert abs(float(off.mean())) <= 2.0 ** -20, float(off.mean())
    assert float(off.abs().max()) <= 2.0 ** -16


@pytest.mark.parametrize("room", ROOMS)
@pytest.mark.parametrize("kind", ["float32", "float16", "bfloat16"])
@pytest.mark.parametrize("group,dim", [(1, 64), (2, 64), (4, 128), (8, 64), (5, 192)])
def test_attend_infinite_keys_reach_their_rows(kind, group, dim, room):
    """An Inf in an attended key makes every row of its key-value head
    non-finite, with weights and log sums, whichever sign the score has and
    whichever body the sizes choose; every other row keeps its bits."""
    T = torch()
    rng = np.random.default_rng(43)
    for n, most in (([700, 90, 33], 0), ([20, 90, 33], 8)):  # the second: few slots, the plain lanes for any group
        cache, k, v = build(rng, kind, n, 2, dim, 16, max_pages=room_for(room, 16) or most or None)
        q = rng.standard_normal((3, 2 * group, dim)).astype(np.float32)
        q[0, :, 7] = np.where(np.arange(2 * group) % 2, 0.5, -0.5)  # scores of both signs
        qd = T.from_numpy(q).cuda()
        lse0, acc0 = T.empty((3, 2 * group), device="cuda"), T.zeros((3, cache.capacity), device="cuda")
        base = w4().kv_attend(qd, cache, lse=lse0, acc=acc0)
        for at in (0, 13, n[0] - 1):
            p = int(cache.page_table[0, at // 16])
            was = float(cache.k[p, 1, at % 16, 7])
            cache.k[p, 1, at % 16, 7] = float("inf")
            lse, acc = T.empty_like(lse0), T.zeros_like(acc0)
            out = w4().kv_attend(qd, cache, lse=lse, acc=acc)
            cache.k[p, 1, at % 16, 7] = was
            assert not T.isfinite(out[0, group:]).any() and not T.isfinite(lse[0, group:]).any()
            assert not T.isfinite(acc[0, :n[0]]).any()
            assert T.equal(out[0, :group], base[0, :group]) and T.equal(out[1:], base[1:])
            assert T.equal(lse[0, :group], lse0[0, :group]) and T.equal(lse[1:], lse0[1:]) and T.equal(acc[1:], acc0[1:])


@pytest.mark.parametrize("room", ROOMS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,group,dim", [(3, 1, 64), (2, 2, 96), (2, 5, 128), (1, 8, 64), (1, 4, 256)])
def test_attend_queries_at_any_address(kind, heads, group, dim, room):
    """Rows of queries that begin at 4-byte addresses, an odd distance apart:
    runs, clusters and warps' items."""
    T = torch()
    rng = np.random.default_rng(heads * 7 + group + dim)
    for lengths, pages in (([0, 1, 17, 130, 700], room_for(room, 16)), ([int(x) for x in rng.integers(0, 50, 900)], 4)):
        cache, k, v = build(rng, kind, lengths, heads, dim, 16, max_pages=pages)
        B, W = len(lengths), heads * group * dim
        q = rng.standard_normal((B, heads * group, dim)).astype(np.float32)
        wide = T.full((B, W + 41), float("nan"), device="cuda")
        wide[:, 9:9 + W] = T.from_numpy(q.reshape(B, W)).cuda()
        odd = wide[:, 9:9 + W].view(B, heads * group, dim)
        assert odd.data_ptr() % 16 and odd.stride(0) % 4
        out = w4().kv_attend(odd, cache)
        assert T.equal(out, check(cache, k, v, q, what=f"{kind} {heads}x{group}x{dim}"))
