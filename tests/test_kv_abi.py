"""Host-side refusals of the cache and scoring entry points (no device is
touched), the descriptor's layout, and the oracle's own pins."""

import ctypes as C
import os
import subprocess

import numpy as np
import pytest

import oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _lib():
    from int8_weight_quantized_w4_b200 import _lib as L
    if not os.path.exists(L.LIB_PATH):
        from int8_weight_quantized_w4_b200 import build
        build.build(quiet=True)
    return L.load()


def desc(**kw):
    from int8_weight_quantized_w4_b200._lib import KvCacheDesc
    a = dict(k=0x10000, v=0x20000, k_scales=0, v_scales=0, page_table=0x30000, lengths=0x40000, page_stride=2 * 16 * 64,
             num_pages=10, ldp=4, max_pages=4, seqs=2, kv_heads=2, page_size=16, head_dim=64, type=0)
    a.update(kw)
    return KvCacheDesc(**a)


BROKEN = [
    (dict(type=4), 8), (dict(type=-1), 8), (dict(head_dim=0), 2), (dict(head_dim=24), 2), (dict(head_dim=272), 2),
    (dict(page_size=0), 2), (dict(page_size=65537), 2), (dict(kv_heads=0), 2), (dict(kv_heads=5000), 2),
    (dict(seqs=-1), 2), (dict(seqs=70000), 2), (dict(num_pages=-1), 2), (dict(num_pages=1 << 31), 2),
    (dict(max_pages=-1), 2), (dict(max_pages=1 << 27), 2), (dict(ldp=3), 2), (dict(page_stride=2047), 2),
    (dict(page_stride=2049), 2), (dict(page_stride=1 << 41), 2), (dict(k=0), 1), (dict(v=0), 1), (dict(page_table=0), 1),
    (dict(lengths=0), 1), (dict(k=0x10008), 3), (dict(v=0x20004), 3), (dict(page_table=0x30002), 3),
    (dict(lengths=0x40001), 3), (dict(k_scales=0x50000), 8), (dict(type=3), 1),
    (dict(type=3, k_scales=0x50002, v_scales=0x60000), 3),
]


def append(lib, d, k=0x70000, ldk=128, v=0x80000, ldv=128, cu=0x90000, tokens=5, out=0xA0000):
    return lib.kv_append(C.byref(d) if d else None, k, ldk, v, ldv, cu, tokens, out, None)


def attend(lib, d, q=0x70000, ldq=256, heads=4, scale=0.125, window=0, out=0x80000, ldo=256, lse=0, acc=0, ldacc=0, ws=0,
           wsb=0):
    return lib.kv_attend(C.byref(d) if d else None, q, ldq, heads, scale, window, out, ldo, lse, acc, ldacc, ws, wsb, None)


def evict(lib, s, d, acc=0x70000, ldacc=64, keep=8, recent=2, acc_out=0x71000, ldo=64, kept=0, ldkept=0):
    return lib.kv_evict(C.byref(s) if s else None, acc, ldacc, keep, recent, C.byref(d) if d else None, acc_out, ldo, kept,
                        ldkept, None, 0, None)


@pytest.mark.parametrize("kw,status", BROKEN)
def test_broken_descriptors_are_refused_before_any_launch(kw, status):
    lib = _lib()
    d = desc(**kw)
    other = desc(k=0x110000, v=0x120000, page_table=0x130000, lengths=0x140000)
    for st in (append(lib, d), attend(lib, d), evict(lib, d, other), evict(lib, other, d)):
        assert st == status
        assert lib.w4_last_error()
    assert lib.kv_attend_workspace_size(C.byref(d), 4, 0) == 0
    assert lib.kv_evict_workspace_size(C.byref(d), 4, 0) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(k=0), 1), (dict(v=0), 1), (dict(out=0), 1), (dict(tokens=-1), 2), (dict(tokens=1 << 31), 2),
    (dict(ldk=127), 2), (dict(ldv=100), 2), (dict(k=0x70002), 3), (dict(out=0xA0001), 3), (dict(cu=0x90002), 3),
    (dict(cu=0), 2), (dict(out=0x40004), 8),
])
def test_append_argument_errors(kw, status):
    assert append(_lib(), desc(), **kw) == status


def test_append_more_refusals_and_noops():
    lib = _lib()
    assert append(lib, None) == 1
    assert append(lib, desc(ldp=0)) == 8
    assert append(lib, desc(seqs=0), k=0, v=0, cu=0, tokens=0, out=0) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), 1), (dict(out=0), 1), (dict(heads=3), 2), (dict(heads=0), 2), (dict(heads=-2), 2), (dict(ldq=255), 2),
    (dict(ldo=255), 2), (dict(window=-1), 8), (dict(scale=float("inf")), 8), (dict(scale=float("nan")), 8), (dict(scale=3e38), 8),
    (dict(q=0x70002), 3), (dict(out=0x80001), 3), (dict(lse=0x90002), 3), (dict(acc=0x90002, ldacc=64), 3),
    (dict(acc=0x90000, ldacc=63), 2),
])
def test_attend_argument_errors(kw, status):
    assert attend(_lib(), desc(), **kw) == status


def test_attend_noops_need_no_device():
    lib = _lib()
    assert attend(lib, None) == 1
    assert attend(lib, desc(seqs=0), q=0, out=0) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(acc=0), 1), (dict(acc_out=0), 1), (dict(keep=-1), 8), (dict(recent=-1), 8), (dict(keep=1 << 31), 8),
    (dict(ldacc=63), 2), (dict(ldo=63), 2), (dict(acc=0x70002), 3), (dict(kept=0x90002, ldkept=8), 3),
    (dict(kept=0x90000, ldkept=7), 2), (dict(acc_out=0x70000, ldo=65), 2), (dict(acc_out=0x70010), 8),
    (dict(ldacc=127, ldo=127, acc_out=0x70000 + 64 * 4), 8),
])
def test_evict_argument_errors(kw, status):
    d = desc(k=0x110000, v=0x120000, page_table=0x130000, lengths=0x140000)
    assert evict(_lib(), desc(), d, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(kv_heads=1), 2), (dict(head_dim=32), 2), (dict(page_size=8), 2), (dict(seqs=3), 2), (dict(type=1), 2),
    (dict(k=0x10000), 8), (dict(v=0x20000), 8), (dict(lengths=0x40000), 8), (dict(lengths=0x40004), 8), (dict(ldp=0), 8),
])
def test_evict_refuses_a_destination_that_does_not_fit(kw, status):
    a = dict(k=0x110000, v=0x120000, page_table=0x130000, lengths=0x140000)
    a.update(kw)
    assert evict(_lib(), desc(), desc(**a)) == status
    assert evict(_lib(), desc(seqs=0), desc(seqs=0)) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), 2), (dict(V=-1), 2), (dict(V=0), 2), (dict(ldl=9), 2), (dict(top=-1), 8), (dict(top=33, V=100, ldl=100), 8),
    (dict(top=11), 8), (dict(logits=0), 1), (dict(tokens=0), 1), (dict(logits=0x1002), 3), (dict(tokens=0x2001), 3),
    (dict(entropy=0x4002), 3), (dict(V=1 << 31, ldl=1 << 31), 2),
])
def test_logprobs_argument_errors(kw, status):
    lib = _lib()
    a = dict(logits=0x1000, ldl=10, tokens=0x2000, M=2, V=10, top=3, logp=0x3000, entropy=0x4000, tl=0x5000, ti=0x6000)
    a.update(kw)
    call = lambda **k: lib.token_logprobs(*{**a, **k}.values(), None)  # noqa: E731
    assert call() == status
    assert lib.token_logprobs(0, 0, 0, 0, 10, 0, 0, 0, 0, 0, None) == 0  # M = 0


def test_cache_descriptor_layout_matches_the_c_struct(tmp_path):
    from int8_weight_quantized_w4_b200._lib import KvCacheDesc as D
    fields = ["lengths", "page_stride", "num_pages", "ldp", "max_pages", "seqs", "kv_heads", "type"]
    src = tmp_path / "kv.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "w4.h"\nint main(void) { printf("%zu", '
                   'sizeof(kv_cache));\n' + "".join(f'printf(" %zu", offsetof(kv_cache, {f}));\n' for f in fields) +
                   "return 0; }\n")
    exe = tmp_path / "kv"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [C.sizeof(D)] + [getattr(D, f).offset for f in fields]


def test_python_cache_refuses_what_it_cannot_hold():
    import torch as T

    from int8_weight_quantized_w4_b200 import KvCache, token_logprobs
    k = T.zeros((3, 2, 16, 64))
    tb, ln = T.zeros((2, 1), dtype=T.int32), T.zeros(2, dtype=T.int32)
    s = T.zeros((3, 2, 16))
    for args, kw in [((k.double(), k.double(), tb, ln), {}), ((k, k.half(), tb, ln), {}), ((k, k[:2], tb, ln), {}),
                     ((k[0], k[0], tb, ln), {}), ((k.transpose(1, 2), k.transpose(1, 2), tb, ln), {}),
                     ((k, k, tb.long(), ln), {}), ((k, k, tb, ln.long()), {}), ((k, k, tb, ln[:1]), {}),
                     ((k, k, tb[0], ln), {}), ((k, k, tb, ln), dict(k_scales=s, v_scales=s)),
                     ((k.to(T.int8), k.to(T.int8), tb, ln), {}), ((k.to(T.int8), k.to(T.int8), tb, ln), dict(k_scales=s)),
                     ((k.to(T.int8), k.to(T.int8), tb, ln), dict(k_scales=s, v_scales=s[:2])),
                     ((k, k, tb, ln), {})]:  # the last: host tensors
        with pytest.raises(ValueError):
            KvCache(*args, **kw)
    with pytest.raises(ValueError):
        token_logprobs(T.zeros((2, 10)))


# ---------------------------------------------------------------- oracle pins

def test_oracle_attend_by_hand():
    """Two slots, two heads by hand: weights 1/(1+e^-1) and its complement."""
    k = np.zeros((2, 1, 2))
    k[0, 0], k[1, 0] = [1, 0], [0, 3]
    v = np.array([[[1.0, 2.0]], [[5.0, -2.0]]])
    out, lse, w, tol = oracle.kv_attend_ref([[2.0, 0.0], [0.0, 0.0]], k, v, 0.5)
    a = 1 / (1 + np.exp(-1.0))
    assert np.allclose(w[0], [a, 1 - a], atol=1e-15) and np.allclose(w[1], [0.5, 0.5], atol=1e-15)
    assert np.allclose(out[0], [a + 5 * (1 - a), 2 * a - 2 * (1 - a)], atol=1e-14)
    assert np.allclose(out[1], [3, 0], atol=1e-15)
    assert np.allclose(lse, [np.log(np.e + 1), np.log(2)], atol=1e-15)
    out, _, w, _ = oracle.kv_attend_ref([[2.0, 0.0]], k, v, 0.5, window=1)
    assert np.array_equal(out[0], [5, -2]) and np.array_equal(w[0], [0, 1])
    out, lse, _, _ = oracle.kv_attend_ref([[2.0, 0.0]], k[:0], v[:0], 0.5)
    assert np.array_equal(out, [[0, 0]]) and lse[0] == -np.inf


def test_oracle_store_by_hand():
    codes, s = oracle.kv_store(np.array([[127, 63.5, -0.5, 0.5, 1.5]], np.float32), "int8")
    assert s[0] == 1 and codes.tolist() == [[127, 64, 0, 0, 2]]
    codes, s = oracle.kv_store(np.zeros((1, 4), np.float32), "int8")
    assert s[0] == 1 and not codes.any()
    b, _ = oracle.kv_store(np.array([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, -1e-40], np.float32), "bfloat16")
    import torch as T
    x = np.random.default_rng(0).standard_normal(1000).astype(np.float32)
    assert b[0] == 1 and b[1] == 1 + 2.0 ** -6
    assert np.array_equal(oracle.round_bf16(x), T.from_numpy(x).bfloat16().float().numpy())


def test_oracle_evict_by_hand():
    acc = [3, 1, 3, np.nan, 2, 0, 9]
    assert oracle.kv_evict_ref(acc, 7, 3, 1) == [0, 2, 6]
    assert oracle.kv_evict_ref(acc, 7, 2, 0) == [0, 6]
    assert oracle.kv_evict_ref(acc, 7, 2, 5) == [5, 6]
    assert oracle.kv_evict_ref(acc, 7, 6, 0) == [0, 1, 2, 4, 5, 6]
    assert oracle.kv_evict_ref(acc, 4, 4, 0) == [0, 1, 2, 3]


def test_oracle_logprobs_by_hand():
    x = np.log(np.array([[1.0, 2.0, 1.0]]))
    lp, ent, tl, ti = oracle.logprobs_ref(x, [1], 3)
    assert np.allclose(lp, np.log(0.5)) and np.allclose(ent, 1.5 * np.log(2))
    assert ti.tolist() == [[1, 0, 2]] and np.allclose(tl, np.log([[0.5, 0.25, 0.25]]))
