"""GPU parity of token_logprobs against fp64.

Bounds: logits are exact inputs; lse sums V exponentials (2^-22 each) in fp32
partial sums (at most V / 256 + 64 roundings, each of half a step, in one
thread's sum and the joins) and takes a logarithm; logp adds one subtraction.
The entropy is log l - t / l: the same relative errors, times t / l <= the
largest |x - m| that still weighs in."""

import numpy as np
import pytest

import oracle
from kv_util import clear_error, error_status, torch, w4

pytestmark = pytest.mark.gpu


def check(x, tokens, top, ld=None, offset=0):
    T = torch()
    M, V = x.shape
    ld = ld or V
    buf = T.full((offset + M * ld + 8,), float("nan"), device="cuda")
    rows = buf[offset:offset + M * ld].view(M, ld)[:, :V]
    rows.copy_(T.from_numpy(x))
    tok = None if tokens is None else T.from_numpy(np.asarray(tokens, np.int32)).cuda()
    logp, ent, tl, ti = w4().token_logprobs(rows, tok, top=top)
    with np.errstate(all="ignore"):
        rp, re, rtl, rti = oracle.logprobs_ref(x, tokens, top)
    rel = (V / 256 + 64) * oracle.EPS + 2.0 ** -20
    spread = np.nan_to_num(np.abs(re), nan=0.0) + 20.0  # |x - m| of the logits that weigh in

    def near(got, want, tol):
        got = got.cpu().double().numpy()
        tol = np.broadcast_to(tol, want.shape)
        same = (got == want) | (np.isnan(got) & np.isnan(want))
        with np.errstate(invalid="ignore"):
            off = np.where(same, 0.0, np.abs(got - want))
        assert np.all(off <= tol), (np.nanmax(off), tol.max())

    # logp = (x - m) - log l: two roundings of values no larger than itself, and those of log l
    tol = rel + 2.0 ** -20
    if tokens is not None:
        near(logp, rp, tol + 4 * oracle.EPS * np.nan_to_num(np.abs(rp), posinf=0, neginf=0))
    near(ent, re, rel * spread)
    if top:
        assert ti.dtype == T.int32 and np.array_equal(ti.cpu().numpy(), rti)
        near(tl, rtl, tol + 4 * oracle.EPS * np.nan_to_num(np.abs(rtl), posinf=0, neginf=0))
    else:
        assert tl is None and ti is None


@pytest.mark.parametrize("M,V,top,ld,offset", [
    (1, 50257, 5, None, 0), (1, 50257, 32, 50304, 1), (3, 50257, 1, None, 3), (58, 1001, 20, 1003, 2), (1, 1, 1, None, 0),
    (2, 2, 2, None, 1), (5, 3, 0, None, 0), (4, 31, 31, None, 2), (4, 33, 32, 37, 1), (200, 777, 7, None, 0),
    (1, 16384, 10, None, 0), (2, 4099, 32, None, 1), (1, 200001, 3, None, 3), (150, 4097, 2, None, 0), (6, 256, 16, None, 0),
])
def test_logprobs(M, V, top, ld, offset):
    rng = np.random.default_rng(M * 7 + V)
    x = (rng.standard_normal((M, V)) * 3).astype(np.float32)
    check(x, rng.integers(0, V, M), top, ld, offset)


def test_logprobs_ties_zeros_and_infinities():
    rng = np.random.default_rng(2)
    V = 5000
    x = np.round(rng.standard_normal((8, V)) * 2).astype(np.float32)  # many equal logits
    x[1] = 0.0
    x[1, ::2] = -0.0
    x[2, 100:] = -np.inf
    x[3] = -np.inf
    x[3, 4321] = 1.5
    x[4] = -np.inf
    x[5] = np.finfo(np.float32).min  # a mask of the type's lowest value
    x[5, 77] = 12.0
    x[6] = np.finfo(np.float32).min
    x[7, :] = np.linspace(-3e38, 3e38, V, dtype=np.float32)
    check(x, [3, 5, 4000, 4321, 9, 77, 2, V - 1], 32)


def test_logprobs_nan_and_positive_infinity():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 3000)).astype(np.float32)
    x[0, 5] = np.nan
    x[1, 2999] = np.inf
    x[2, :] = np.nan
    x[3, ::2] = -np.nan
    check(x, [1, 2, 3, 4], 9)


def test_logprobs_ascending_logits_insert_every_time():
    """Each logit beats all before it: the list takes an insertion each."""
    V = 20000
    x = np.stack([np.linspace(-10, 10, V), np.linspace(10, -10, V)]).astype(np.float32)
    check(x, [0, V - 1], 32)


def test_logprobs_ids_that_score_nothing_or_are_wrong():
    T = torch()
    rng = np.random.default_rng(4)
    x = rng.standard_normal((4, 100)).astype(np.float32)
    clear_error()
    check(x[:2], [-1, 7], 0)
    assert error_status() == 0
    lp, _, _, _ = w4().token_logprobs(T.from_numpy(x).cuda(), T.tensor([100, -2, 5, -1], dtype=T.int32, device="cuda"))
    assert error_status() == 8
    lp = lp.cpu().numpy()
    assert np.isnan(lp[0]) and np.isnan(lp[1]) and np.isfinite(lp[2]) and lp[3] == 0
    check(x, None, 3)


def test_logprobs_on_the_heads_logits_in_a_graph():
    """Head and scores captured together, replayed with other hidden rows:
    the best alternative is the head's greedy token."""
    T = torch()
    from int8_weight_quantized_w4_b200 import synth
    K, V = 256, 5003
    H = synth.i8_head(K, V, seed=3)
    table, scales = T.from_numpy(H["table"]).cuda(), T.from_numpy(H["scales"]).cuda()
    tiles = w4().i8t_head_repack(table, scales, K, V)
    h = T.zeros((3, K), device="cuda")
    tok = T.tensor([1, 2, 3], dtype=T.int32, device="cuda")
    logits = T.empty((3, V), device="cuda")
    w4().i8t_head_logits(h, tiles, K, V, logits=logits)
    w4().token_logprobs(logits, tok, top=4)
    T.cuda.synchronize()
    g = T.cuda.CUDAGraph()
    with T.cuda.graph(g):
        w4().i8t_head_logits(h, tiles, K, V, logits=logits)
        got = w4().token_logprobs(logits, tok, top=4)
    for seed in (1, 2):
        x = synth.activations(3, K, 9, seed=seed)
        h.copy_(T.from_numpy(x))
        g.replay()
        T.cuda.synchronize()
        best, _ = w4().i8t_head_argmax(h, tiles, K, V)
        assert T.equal(got[3][:, 0], best)
        rp, re, rtl, _ = oracle.logprobs_ref(logits.cpu().numpy(), [1, 2, 3], 4)
        tol = 2e-5 + 1e-6 * np.abs(logits.cpu().numpy()).max()
        assert np.all(np.abs(got[0].cpu().numpy() - rp) <= tol)
        assert np.all(np.abs(got[2].cpu().numpy() - rtl) <= tol)


def test_logprobs_refusals():
    T = torch()
    W = w4()
    x = T.zeros((2, 10), device="cuda")
    for top in (-1, 33, 11):
        with pytest.raises((W.W4Error, RuntimeError)):
            W.token_logprobs(x, top=top)
    for bad in (x.half(), x.cpu(), x.t(), x.view(2, 2, 5)):
        with pytest.raises(ValueError):
            W.token_logprobs(bad)
    with pytest.raises(ValueError):
        W.token_logprobs(x, T.zeros(3, dtype=T.int32, device="cuda"))
    with pytest.raises(ValueError):
        W.token_logprobs(x, T.zeros(2, dtype=T.int64, device="cuda"))
    got = W.token_logprobs(T.zeros((0, 10), device="cuda"), top=3)
    assert got[1].shape == (0,) and got[2].shape == (0, 3)
