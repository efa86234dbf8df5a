"""B200 quantised-weight matmul library: Python binding of libw4b200.so.

Argument marshalling only: every step of the computation runs in the
library's CUDA kernels (sm_100a). PyTorch provides device memory and
streams. If the library is missing or the GPU is not a B200 the calls raise;
nothing falls back to another implementation.

Operations (see include/w4.h for layouts and error behaviour):
  w4_matmul(x, qw, scales, zp, K, N)        y = x . W, W 4-bit blocked
      (..., bias=, residual=, act=)         y = act(x . W + bias) + residual, fused
  w4_matmul_grouped([...])                  many independent ones, one launch
  w4_repack(qw, scales, zp, K, N)           the weight in the streaming layout (once, at load)
  w4r_matmul(x, wr, K, N) / _grouped        decode (M = 1) on repacked weights
  i8_head_logits(h, table, scales, K, V)    last-position logits, int8 head
  i8_head_repack(table, scales, K, V)       the head in the streaming layout (once, at load)
  i8r_head_logits(h, tr, K, V) / _argmax    M = 1 head on the repacked table
  w4i_matmul(x, wt, K, N)                   M = 1 on the tile layout: integer tensor-core MMAs
  i8t_head_repack(table, scales, K, V)      the head in the tensor cores' tile layout (once, at load)
  i8t_head_logits(h, tiles, K, V) / _argmax M <= 8 rows on the tensor-core head
  KvCache(k, v, page_table, lengths)        one layer's paged key-value cache
  kv_append(cache, k, v)                    new tokens' keys and values into it
  kv_attend(q, cache)                       attention of each sequence's newest token over it
  kv_evict(cache, acc, keep)                the slots that the attention has used least leave it
  token_logprobs(logits, tokens, top)       log probabilities, entropy, alternatives from logits
  w4_quantize(w, block, scale_type)         the dq4 quantiser (GPU)
  i8_quantize_head(w)                       the embedding_int8 quantiser (GPU)
  pack_nibbles / unpack_nibbles             host-side UINT4 packing
"""

from __future__ import annotations

import ctypes as C
from typing import Sequence

import numpy as np

from . import _lib
from ._lib import (ACTS, GROUP_MAX, KV_TYPES, PATHS, STATUS, TOP_MAX, KvCacheDesc, W4Desc,  # noqa: F401
                   W4LibraryMissing, W4RDesc)


class W4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = ""
        try:
            detail = (_lib.load().w4_last_error() or b"").decode()
        except Exception:
            pass
        super().__init__(f"{where}: {STATUS.get(status, status)}: {detail}")


def _check(status: int, where: str) -> None:
    if status != 0:
        raise W4Error(status, where)


def lib():
    return _lib.load()


def abi_version() -> int:
    return lib().w4_abi_version()


# ---------------------------------------------------------------- torch helpers

def _torch():
    import torch
    return torch


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _stream_handle(stream) -> int:
    if stream is None:
        torch = _torch()
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return int(stream.cuda_stream)


_WS = {}  # device index -> zero-filled uint8 workspace tensor


def workspace(nbytes: int, device=None):
    """A zero-filled device workspace of at least nbytes (cached per device).

    The kernels leave it zero-filled, so it is zeroed only when allocated.
    Calls that may overlap on the GPU must not share one: pass your own.
    """
    torch = _torch()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    cur = _WS.get(idx)
    if nbytes == 0:
        return None
    if cur is None or cur.numel() < nbytes:
        cur = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=dev)
        _WS[idx] = cur
    return cur


def _ld(t, inner: int) -> int:
    """Row stride in elements; a single row has no stride of its own."""
    if t.dim() == 1 or t.shape[0] <= 1:
        return max(inner, 1)
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError("innermost dimension must be contiguous")
    return int(t.stride(0))


# ---------------------------------------------------------------- body

def w4_matmul_workspace_size(M: int, K: int, N: int) -> int:
    return int(lib().w4_matmul_workspace_size(M, K, N))


def _epilogue(it: dict, N: int):
    """(bias ptr, residual ptr, ldr, act code) of an item's optional epilogue."""
    bias, res, act = it.get("bias"), it.get("residual"), it.get("act", "none")
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    return _ptr(bias), _ptr(res), (0 if res is None else _ld(res, N)), ACTS[act]


def w4_matmul(x, qw, scales, zp, K: int, N: int, y=None, path: str = "auto", ws=None, stream=None, bias=None,
              residual=None, act: str = "none"):
    """y[M, N] = x[M, K] . W[K, N] (fp32) with W given as packed nibbles,
    fp32 scales [K/32, N] and packed zero points; returns y.

    With bias ([N]), residual ([M, N], may be y itself) or act ("gelu_tanh",
    "gelu_erf") the kernel's final store computes act(x . W + bias) + residual."""
    torch = _torch()
    M = x.shape[0] if x.dim() == 2 else 1
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=x.device)
    need = w4_matmul_workspace_size(M, K, N)
    if ws is None:
        ws = workspace(need, x.device)
    if bias is not None or residual is not None or act != "none":
        b, r, ldr, a = _epilogue({"bias": bias, "residual": residual, "act": act}, N)
        d = W4Desc(_ptr(x), _ld(x, K), _ptr(qw), _ptr(scales), _ptr(zp), _ptr(y), _ld(y, N), M, K, N, b, r, ldr, a, 0)
        st = lib().w4_matmul_desc(C.byref(d), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                  PATHS[path], _stream_handle(stream))
        _check(st, "w4_matmul")
        return y
    st = lib().w4_matmul_path(_ptr(x), _ld(x, K), _ptr(qw), _ptr(scales), _ptr(zp), _ptr(y), _ld(y, N), M, K, N,
                              _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), PATHS[path],
                              _stream_handle(stream))
    _check(st, "w4_matmul")
    return y


def make_descs(items: Sequence[dict]):
    """ctypes descriptor array for w4_matmul_grouped; each item holds the
    tensors x, qw, scales, zp, y and the ints K, N (M from x), and optionally
    the fused epilogue "bias", "residual" and "act" (as in w4_matmul)."""
    arr = (W4Desc * len(items))()
    for i, it in enumerate(items):
        x, y = it["x"], it["y"]
        K, N = int(it["K"]), int(it["N"])
        M = x.shape[0] if x.dim() == 2 else 1
        b, r, ldr, a = _epilogue(it, N)
        arr[i] = W4Desc(_ptr(x), _ld(x, K), _ptr(it["qw"]), _ptr(it["scales"]), _ptr(it["zp"]), _ptr(y),
                        _ld(y, N), M, K, N, b, r, ldr, a, 0)
    return arr


def w4_matmul_grouped_workspace_size(descs) -> int:
    return int(lib().w4_matmul_grouped_workspace_size(descs, len(descs)))


def w4_matmul_grouped(items: Sequence[dict] | None = None, descs=None, ws=None, stream=None):
    """All matmuls of `items` (or a prepared descriptor array) in grouped launches."""
    if descs is None:
        descs = make_descs(items)
    need = w4_matmul_grouped_workspace_size(descs)
    if ws is None:
        ws = workspace(need)
    st = lib().w4_matmul_grouped(descs, len(descs), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                 _stream_handle(stream))
    _check(st, "w4_matmul_grouped")


# ---------------------------------------------------------------- streaming layout (decode)

def w4_repacked_bytes(K: int, N: int) -> int:
    return int(lib().w4_repacked_bytes(K, N))


def w4_repack(qw, scales, zp, K: int, N: int, out=None, stream=None):
    """The weight (page format: packed nibbles, fp32 scales, packed zero
    points) in the streaming layout the decode GEMV reads: a uint8 device
    tensor of w4_repacked_bytes(K, N) bytes holding the same words, reordered."""
    torch = _torch()
    nbytes = w4_repacked_bytes(K, N)
    if nbytes == 0:
        raise ValueError(f"the streaming layout does not take K={K}, N={N} (K % 32 == 0, N % 8 == 0)")
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=qw.device)
    st = lib().w4_repack(_ptr(qw), _ptr(scales), _ptr(zp), K, N, _ptr(out), _stream_handle(stream))
    _check(st, "w4_repack")
    return out


def w4_repack_restore(wr, K: int, N: int, stream=None):
    """The page-format buffers (qw, scales, zp) of a repacked weight."""
    torch = _torch()
    nb = K // 32
    qw = torch.empty(K * N // 2, dtype=torch.uint8, device=wr.device)
    sc = torch.empty((nb, N), dtype=torch.float32, device=wr.device)
    zp = torch.empty(nb * N // 2, dtype=torch.uint8, device=wr.device)
    st = lib().w4_repack_restore(_ptr(wr), K, N, _ptr(qw), _ptr(sc), _ptr(zp), _stream_handle(stream))
    _check(st, "w4_repack_restore")
    return qw, sc, zp


def make_rdescs(items: Sequence[dict]):
    """ctypes w4r_desc array for w4r_matmul_grouped; each item holds the
    tensors x ([1, K] or [K]), wr (repacked), y and the ints K, N, and
    optionally "bias", "residual" and "act"."""
    arr = (W4RDesc * len(items))()
    for i, it in enumerate(items):
        x, y = it["x"], it["y"]
        K, N = int(it["K"]), int(it["N"])
        M = x.shape[0] if x.dim() == 2 else 1
        b, r, ldr, a = _epilogue(it, N)
        arr[i] = W4RDesc(_ptr(x), _ld(x, K), _ptr(it["wr"]), _ptr(y), _ld(y, N), M, K, N, b, r, ldr, a, 0)
    return arr


def w4r_matmul_grouped(items: Sequence[dict] | None = None, descs=None, stream=None):
    """All decode matmuls of `items` (or a prepared w4r_desc array)."""
    if descs is None:
        descs = make_rdescs(items)
    st = lib().w4r_matmul_grouped(descs, len(descs), _stream_handle(stream))
    _check(st, "w4r_matmul_grouped")


def w4r_matmul(x, wr, K: int, N: int, y=None, stream=None, bias=None, residual=None, act: str = "none"):
    """y[1, N] = act(x[1, K] . W + bias) + residual with W repacked (w4_repack)."""
    torch = _torch()
    if y is None:
        y = torch.empty((1, N), dtype=torch.float32, device=x.device)
    item = {"x": x, "wr": wr, "y": y, "K": K, "N": N, "bias": bias, "residual": residual, "act": act}
    w4r_matmul_grouped(descs=make_rdescs([item]), stream=stream)
    return y


# ---------------------------------------------------------------- tile layout (prefill)

_TWS: dict = {}


def tile_workspace(nbytes: int, device=None):
    """A device scratch of at least nbytes for w4t_matmul_grouped (cached per
    device; no zeroing needed). Calls that may overlap on the GPU must not
    share one: pass your own."""
    torch = _torch()
    if nbytes == 0:
        return None
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    cur = _TWS.get(idx)
    if cur is None or cur.numel() < nbytes:
        cur = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=dev)
        _TWS[idx] = cur
    return cur


def w4t_repacked_bytes(K: int, N: int) -> int:
    return int(lib().w4t_repacked_bytes(K, N))


def w4t_repack(qw, scales, zp, K: int, N: int, out=None, stream=None):
    """The weight (page format) in the tile layout the tensor-core tile GEMM
    reads: a uint8 device tensor of w4t_repacked_bytes(K, N) bytes."""
    torch = _torch()
    nbytes = w4t_repacked_bytes(K, N)
    if nbytes == 0:
        raise ValueError(f"the tile layout does not take K={K}, N={N} (K % 32 == 0, N % 8 == 0)")
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=qw.device)
    _check(lib().w4t_repack(_ptr(qw), _ptr(scales), _ptr(zp), K, N, _ptr(out), _stream_handle(stream)), "w4t_repack")
    return out


def w4t_repack_restore(wt, K: int, N: int, stream=None):
    """The page-format buffers (qw, scales, zp) of a weight in the tile layout."""
    torch = _torch()
    nb = K // 32
    qw = torch.empty(K * N // 2, dtype=torch.uint8, device=wt.device)
    sc = torch.empty((nb, N), dtype=torch.float32, device=wt.device)
    zp = torch.empty(nb * N // 2, dtype=torch.uint8, device=wt.device)
    _check(lib().w4t_repack_restore(_ptr(wt), K, N, _ptr(qw), _ptr(sc), _ptr(zp), _stream_handle(stream)),
           "w4t_repack_restore")
    return qw, sc, zp


def w4t_workspace_size(descs) -> int:
    return int(lib().w4t_workspace_size(descs, len(descs)))


def w4t_matmul_grouped(items: Sequence[dict] | None = None, descs=None, ws=None, stream=None):
    """Matmuls of any M on tile-layout weights ("wr" = w4t_repack output) on
    the tensor cores; items as for make_rdescs (x [M, K])."""
    if descs is None:
        descs = make_rdescs(items)
    need = w4t_workspace_size(descs)
    if ws is None:
        ws = tile_workspace(need)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().w4t_matmul_grouped(descs, len(descs), _ptr(ws), nbytes, _stream_handle(stream)),
           "w4t_matmul_grouped")


def w4t_matmul(x, wt, K: int, N: int, y=None, ws=None, stream=None, bias=None, residual=None, act: str = "none"):
    """y[M, N] = act(x[M, K] . W + bias) + residual with W in the tile layout
    (w4t_repack); returns y."""
    torch = _torch()
    if x.dim() == 1:
        x = x.view(1, -1)
    if y is None:
        y = torch.empty((x.shape[0], N), dtype=torch.float32, device=x.device)
    item = {"x": x, "wr": wt, "y": y, "K": K, "N": N, "bias": bias, "residual": residual, "act": act}
    w4t_matmul_grouped(descs=make_rdescs([item]), ws=ws, stream=stream)
    return y


def w4i_workspace_size(descs) -> int:
    return int(lib().w4i_workspace_size(descs, len(descs)))


def w4i_matmul_grouped(items: Sequence[dict] | None = None, descs=None, ws=None, stream=None):
    """Decode matmuls (M = 1) on tile-layout weights ("wr" = w4t_repack output)
    with integer tensor-core MMAs; items as for make_rdescs (x [1, K])."""
    if descs is None:
        descs = make_rdescs(items)
    need = w4i_workspace_size(descs)
    if ws is None:
        ws = tile_workspace(need)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib().w4i_matmul_grouped(descs, len(descs), _ptr(ws), nbytes, _stream_handle(stream)),
           "w4i_matmul_grouped")


def w4i_matmul(x, wt, K: int, N: int, y=None, ws=None, stream=None, bias=None, residual=None, act: str = "none"):
    """y[1, N] = act(x[1, K] . W + bias) + residual with W in the tile layout
    (w4t_repack), on the integer tensor-core GEMV; returns y."""
    torch = _torch()
    if x.dim() == 1:
        x = x.view(1, -1)
    if y is None:
        y = torch.empty((x.shape[0], N), dtype=torch.float32, device=x.device)
    item = {"x": x, "wr": wt, "y": y, "K": K, "N": N, "bias": bias, "residual": residual, "act": act}
    w4i_matmul_grouped(descs=make_rdescs([item]), ws=ws, stream=stream)
    return y


# ---------------------------------------------------------------- head

def i8_head_workspace_size(M: int, K: int, V: int) -> int:
    return int(lib().i8_head_workspace_size(M, K, V))


def i8_head_logits(h, table, scales, K: int, V: int, ldt: int | None = None, logits=None, path: str = "auto",
                   ws=None, stream=None):
    """logits[M, V] = h[M, K] . (T[K, V] * s[V]) for the int8 tied head; h holds
    the last-position rows."""
    torch = _torch()
    M = h.shape[0] if h.dim() == 2 else 1
    ldt = V if ldt is None else ldt
    if logits is None:
        logits = torch.empty((M, V), dtype=torch.float32, device=h.device)
    if ws is None:
        ws = workspace(i8_head_workspace_size(M, K, V), h.device)
    st = lib().i8_head_logits_path(_ptr(h), _ld(h, K), _ptr(table), ldt, _ptr(scales), _ptr(logits),
                                   _ld(logits, V), M, K, V, _ptr(ws),
                                   0 if ws is None else ws.numel() * ws.element_size(), PATHS[path],
                                   _stream_handle(stream))
    _check(st, "i8_head_logits")
    return logits


def i8_head_argmax(h, table, scales, K: int, V: int, ldt: int | None = None, stream=None):
    """Greedy next tokens of the last-position rows h: (tokens int32 [M],
    best logits fp32 [M]), the argmax of the logits i8_head_logits gives
    (ties to the lowest token id)."""
    torch = _torch()
    M = h.shape[0] if h.dim() == 2 else 1
    ldt = V if ldt is None else ldt
    tokens = torch.empty(M, dtype=torch.int32, device=h.device)
    best = torch.empty(M, dtype=torch.float32, device=h.device)
    ws = workspace(int(lib().i8_head_argmax_workspace_size(M, K, V)), h.device)
    st = lib().i8_head_argmax(_ptr(h), _ld(h, K), _ptr(table), ldt, _ptr(scales), M, K, V, _ptr(tokens), _ptr(best),
                              _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), _stream_handle(stream))
    _check(st, "i8_head_argmax")
    return tokens, best


def i8_head_repacked_bytes(K: int, V: int) -> int:
    return int(lib().i8_head_repacked_bytes(K, V))


def i8_head_repack(table, scales, K: int, V: int, ldt: int | None = None, stream=None):
    """The int8 head (page format) in the streaming layout the M = 1 head
    GEMV reads: a uint8 device tensor of i8_head_repacked_bytes(K, V) bytes."""
    torch = _torch()
    ldt = V if ldt is None else ldt
    n = i8_head_repacked_bytes(K, V)
    if n == 0:
        raise ValueError(f"the streaming head does not take K={K}, V={V}")
    out = torch.empty(n, dtype=torch.uint8, device=table.device)
    _check(lib().i8_head_repack(_ptr(table), ldt, _ptr(scales), K, V, _ptr(out), _stream_handle(stream)),
           "i8_head_repack")
    return out


def i8_head_repack_restore(tr, K: int, V: int, stream=None):
    """(table [K, V] int8, scales [V] fp32) of a repacked head."""
    torch = _torch()
    table = torch.empty((K, V), dtype=torch.int8, device=tr.device)
    sc = torch.empty(V, dtype=torch.float32, device=tr.device)
    _check(lib().i8_head_repack_restore(_ptr(tr), K, V, _ptr(table), V, _ptr(sc), _stream_handle(stream)),
           "i8_head_repack_restore")
    return table, sc


def i8r_head_logits(h, tr, K: int, V: int, logits=None, stream=None):
    """logits [1, V] of one last-position row h on a repacked head."""
    torch = _torch()
    if logits is None:
        logits = torch.empty((1, V), dtype=torch.float32, device=h.device)
    _check(lib().i8r_head_logits(_ptr(h), _ptr(tr), K, V, _ptr(logits), _stream_handle(stream)), "i8r_head_logits")
    return logits


def w4r_decode_step(items: Sequence[dict] | None, h, tr, K: int, V: int, logits=None, descs=None, stream=None):
    """One decode step in one launch: the matmuls of `items` (or a prepared
    w4r_desc array) and the head's logits [1, V] of h on the repacked head."""
    torch = _torch()
    if descs is None:
        descs = make_rdescs(items or [])
    if logits is None:
        logits = torch.empty((1, V), dtype=torch.float32, device=h.device)
    _check(lib().w4r_decode_step(descs, len(descs), _ptr(h), _ptr(tr), K, V, _ptr(logits), _stream_handle(stream)),
           "w4r_decode_step")
    return logits


def w4r_decode_step_argmax(items: Sequence[dict] | None, h, tr, K: int, V: int, descs=None, stream=None):
    """One decode step in one launch with greedy decoding: the matmuls of
    `items` and (token int32 [1], best logit fp32 [1]) of h on the head."""
    torch = _torch()
    if descs is None:
        descs = make_rdescs(items or [])
    tok = torch.empty(1, dtype=torch.int32, device=h.device)
    best = torch.empty(1, dtype=torch.float32, device=h.device)
    keys = torch.empty(1, dtype=torch.int64, device=h.device)
    _check(lib().w4r_decode_step_argmax(descs, len(descs), _ptr(h), _ptr(tr), K, V, _ptr(tok), _ptr(best), _ptr(keys),
                                        _stream_handle(stream)), "w4r_decode_step_argmax")
    return tok, best


def i8r_head_argmax(h, tr, K: int, V: int, stream=None):
    """(token int32 [1], best logit fp32 [1]) of one row h on a repacked head."""
    torch = _torch()
    tok = torch.empty(1, dtype=torch.int32, device=h.device)
    best = torch.empty(1, dtype=torch.float32, device=h.device)
    keys = torch.empty(1, dtype=torch.int64, device=h.device)
    _check(lib().i8r_head_argmax(_ptr(h), _ptr(tr), K, V, _ptr(tok), _ptr(best), _ptr(keys), _stream_handle(stream)),
           "i8r_head_argmax")
    return tok, best


def i8t_head_repacked_bytes(K: int, V: int) -> int:
    return int(lib().i8t_head_repacked_bytes(K, V))


def i8t_head_repack(table, scales, K: int, V: int, ldt: int | None = None, stream=None):
    """The int8 head (page format) in the tile layout the tensor-core head
    reads: a uint8 device tensor of i8t_head_repacked_bytes(K, V) bytes."""
    torch = _torch()
    ldt = V if ldt is None else ldt
    n = i8t_head_repacked_bytes(K, V)
    if n == 0:
        raise ValueError(f"the head tile layout does not take K={K}, V={V}")
    out = torch.empty(n, dtype=torch.uint8, device=table.device)
    _check(lib().i8t_head_repack(_ptr(table), ldt, _ptr(scales), K, V, _ptr(out), _stream_handle(stream)),
           "i8t_head_repack")
    return out


def i8t_head_repack_restore(tiles, K: int, V: int, stream=None):
    """(table [K, V] int8, scales [V] fp32) of a head in the tile layout."""
    torch = _torch()
    table = torch.empty((K, V), dtype=torch.int8, device=tiles.device)
    sc = torch.empty(V, dtype=torch.float32, device=tiles.device)
    _check(lib().i8t_head_repack_restore(_ptr(tiles), K, V, _ptr(table), V, _ptr(sc), _stream_handle(stream)),
           "i8t_head_repack_restore")
    return table, sc


def i8t_head_logits(h, tiles, K: int, V: int, logits=None, stream=None):
    """logits [M, V] of M <= 8 last-position rows h [M, K] on the tensor-core
    head (tile layout)."""
    torch = _torch()
    M = h.shape[0] if h.dim() == 2 else 1
    if logits is None:
        logits = torch.empty((M, V), dtype=torch.float32, device=h.device)
    _check(lib().i8t_head_logits(_ptr(h), _ld(h, K), _ptr(tiles), K, V, M, _ptr(logits), _ld(logits, V),
                                 _stream_handle(stream)), "i8t_head_logits")
    return logits


def i8t_head_argmax(h, tiles, K: int, V: int, stream=None):
    """(tokens int32 [M], best logits fp32 [M]) of M <= 8 rows h on the
    tensor-core head."""
    torch = _torch()
    M = h.shape[0] if h.dim() == 2 else 1
    tok = torch.empty(M, dtype=torch.int32, device=h.device)
    best = torch.empty(M, dtype=torch.float32, device=h.device)
    keys = torch.empty(max(M, 1), dtype=torch.int64, device=h.device)
    _check(lib().i8t_head_argmax(_ptr(h), _ld(h, K), _ptr(tiles), K, V, M, _ptr(tok), _ptr(best), _ptr(keys),
                                 _stream_handle(stream)), "i8t_head_argmax")
    return tok, best


def i8_embed_lookup(table, scales, tokens, K: int, V: int, ldt: int | None = None, out=None, stream=None):
    """out[i, k] = T[k, tokens[i]] * s[tokens[i]]: the token lookup on the tied
    int8 [K, V] table; tokens is a device int32 tensor."""
    torch = _torch()
    ldt = V if ldt is None else ldt
    n = int(tokens.numel())
    if tokens.dtype != torch.int32 or not tokens.is_contiguous():
        raise ValueError("tokens must be a contiguous int32 tensor")
    if out is None:
        out = torch.empty((n, K), dtype=torch.float32, device=table.device)
    st = lib().i8_embed_lookup(_ptr(table), ldt, _ptr(scales), _ptr(tokens), n, _ptr(out), _ld(out, K), K, V,
                               _stream_handle(stream))
    _check(st, "i8_embed_lookup")
    return out


# ---------------------------------------------------------------- key-value cache

class KvCache:
    """One layer's paged key-value cache: the caller's tensors, checked once.

    k, v: [pages, kv_heads, page_size, head_dim] of float32, float16, bfloat16
    or int8 (k_scales / v_scales: fp32 [pages, kv_heads, page_size]); a page is
    contiguous, pages may lie further apart (a slice of all layers' pages).
    page_table: int32 [seqs, max_pages], rows of page ids (`expand` of one row
    shares it); lengths: int32 [seqs], the slots held. All on one CUDA device.
    """

    def __init__(self, k, v, page_table, lengths, k_scales=None, v_scales=None):
        torch = _torch()
        kind = KV_TYPES.get(str(k.dtype).replace("torch.", ""))
        if kind is None or v.dtype != k.dtype:
            raise ValueError(f"k and v must both be one of {sorted(KV_TYPES)}")
        if k.dim() != 4 or v.shape != k.shape:
            raise ValueError("k and v must be [pages, kv_heads, page_size, head_dim], of one shape")
        P, H, S, D = k.shape
        for name, t in (("k", k), ("v", v)):
            if P > 0 and t[0].numel() > 0 and not t[0].is_contiguous():
                raise ValueError(f"a page of {name} must be contiguous")
        if P > 1 and k.stride(0) != v.stride(0):
            raise ValueError("the pages of k and v must lie equally far apart")
        if (kind == KV_TYPES["int8"]) != (k_scales is not None and v_scales is not None) or \
                (k_scales is None) != (v_scales is None):
            raise ValueError("an int8 cache needs k_scales and v_scales, another has none")
        for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
            if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != (P, H, S) or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous fp32 [pages, kv_heads, page_size]")
        if page_table.dtype != torch.int32 or page_table.dim() != 2:
            raise ValueError("page_table must be int32 [seqs, max_pages]")
        B, MP = page_table.shape
        if MP > 1 and page_table.stride(1) != 1:
            raise ValueError("the rows of page_table must be contiguous")
        if lengths.dtype != torch.int32 or tuple(lengths.shape) != (B,) or not lengths.is_contiguous():
            raise ValueError("lengths must be a contiguous int32 [seqs]")
        for t in (v, page_table, lengths, k_scales, v_scales):
            if t is not None and t.device != k.device:
                raise ValueError("all tensors of a cache must be on one device")
        if not k.is_cuda:
            raise ValueError("a cache lies in device memory: its tensors must be CUDA tensors")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.page_table, self.lengths = page_table, lengths
        self.device, self.seqs, self.kv_heads, self.page_size, self.head_dim = k.device, B, H, S, D
        self.capacity = MP * S
        self.desc = KvCacheDesc(_ptr(k), _ptr(v), _ptr(k_scales), _ptr(v_scales), _ptr(page_table), _ptr(lengths),
                                k.stride(0) if P > 1 else H * S * D, P, page_table.stride(0) if B > 1 else MP, MP, B,
                                H, S, D, kind)
        self._ref = C.byref(self.desc)
        self._need = {}  # (operation, sizes) -> workspace bytes

    @classmethod
    def empty(cls, pages: int, kv_heads: int, page_size: int, head_dim: int, page_table, dtype):
        """A cache of fresh pages; every sequence of page_table is empty."""
        torch = _torch()
        shape, dev = (pages, kv_heads, page_size, head_dim), page_table.device
        scales = [torch.zeros(shape[:3], device=dev) for _ in range(2)] if dtype == torch.int8 else [None, None]
        return cls(torch.zeros(shape, dtype=dtype, device=dev), torch.zeros(shape, dtype=dtype, device=dev), page_table,
                   torch.zeros(page_table.shape[0], dtype=torch.int32, device=dev), *scales)


def _rows3(t, name: str, rows: int | None, heads: int | None, dim: int, device) -> int:
    """Row stride of an fp32 [rows, heads, dim] tensor whose rows are contiguous."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or t.dtype is not _torch().float32 or t.device != device:
        raise ValueError(f"{name} must be an fp32 [rows, heads, head_dim] tensor on {device}")
    n, h, d = shape
    if (rows is not None and n != rows) or (heads is not None and h != heads) or d != dim:
        raise ValueError(f"{name} is {tuple(shape)}, expected [{rows}, {heads}, {dim}]")
    if (d > 1 and stride[2] != 1) or (h > 1 and stride[1] != d):
        raise ValueError(f"a row of {name} must be contiguous")
    return stride[0] if n > 1 else h * d


def _vector(t, name: str, dtype, n: int, device) -> int:
    shape = t.shape
    if len(shape) != 1 or shape[0] != n or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} [{n}] tensor on {device}")
    return t.data_ptr()


def _matrix(t, name: str, dtype, n: int, width: int, device) -> int:
    """Row stride of an [n, >= width] tensor with contiguous rows."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[0] != n or shape[1] < width or t.dtype is not dtype or t.device != device or \
            (shape[1] > 1 and stride[1] != 1):
        raise ValueError(f"{name} must be a {dtype} [{n}, {width}] tensor with contiguous rows on {device}")
    return stride[0] if n > 1 else max(width, 1)


def _room(ws, device) -> int:
    """Bytes of a workspace."""
    if ws is None:
        return 0
    if ws.device != device or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on {device}")
    return ws.numel() * ws.element_size()


class _On:
    """Makes a tensor's device current, and `stream` if one is given: what is
    allocated inside belongs to the stream that the call runs on."""

    def __init__(self, device, stream):
        if stream is not None and stream.device != device:
            raise ValueError(f"the stream belongs to {stream.device}, the tensors to {device}")
        self.cuda = _torch().cuda
        self.index, self.was = device.index, self.cuda.current_device()
        self.stream = None if stream is None else self.cuda.stream(stream)

    def __enter__(self):
        self.cuda.set_device(self.index)
        if self.stream is not None:
            self.stream.__enter__()

    def __exit__(self, *exc):
        if self.stream is not None:
            self.stream.__exit__(*exc)
        self.cuda.set_device(self.was)


def _elsewhere(device, stream) -> bool:
    """Whether a call has to be made inside _On: another stream than the
    current one is asked for, or the tensors' device is not the current one."""
    return stream is not None or _torch()._C._cuda_getDevice() != device.index


def kv_append(cache: KvCache, k, v, cu_tokens=None, lengths_out=None, stream=None):
    """New tokens' keys and values (fp32 [tokens, kv_heads, head_dim], columns
    of qkv rows for instance) to the ends of their sequences: rows
    cu_tokens[b] .. cu_tokens[b + 1] - 1 (int32 [seqs + 1]) to sequence b, or
    one row each without cu_tokens. The lengths advance in place, or go to
    lengths_out (int32 [seqs]); returns them."""
    torch, dev = _torch(), cache.device
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return kv_append(cache, k, v, cu_tokens, lengths_out)
    n = k.shape[0]
    ldk = _rows3(k, "k", None, cache.kv_heads, cache.head_dim, dev)
    ldv = _rows3(v, "v", n, cache.kv_heads, cache.head_dim, dev)
    cu = 0 if cu_tokens is None else _vector(cu_tokens, "cu_tokens", torch.int32, cache.seqs + 1, dev)
    if lengths_out is None:
        lengths_out = cache.lengths
    out = _vector(lengths_out, "lengths_out", torch.int32, cache.seqs, dev)
    st = lib().kv_append(cache._ref, k.data_ptr(), ldk, v.data_ptr(), ldv, cu, n, out,
                         torch._C._cuda_getCurrentRawStream(dev.index))
    if st != 0:
        _check(st, "kv_append")
    return lengths_out


def kv_attend(q, cache: KvCache, scale: float | None = None, window: int = 0, out=None, lse=None, acc=None, ws=None,
              stream=None):
    """out [seqs, q_heads, head_dim]: attention of the queries q (fp32, one
    token per sequence, row stride free) over each sequence's slots, the last
    `window` of them when it is positive; scale defaults to head_dim ** -0.5.
    lse: fp32 [seqs, q_heads], filled. acc: fp32 [seqs, >= capacity], each
    slot's weight summed over the query heads is added."""
    torch, dev, B, D = _torch(), cache.device, cache.seqs, cache.head_dim
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return kv_attend(q, cache, scale, window, out, lse, acc, ws)
    ldq = _rows3(q, "q", B, None, D, dev)
    Hq = q.shape[1]
    ldo = Hq * D if out is None else _rows3(out, "out", B, Hq, D, dev)
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (B, Hq) or not lse.is_contiguous() or
                            lse.device != dev):
        raise ValueError(f"lse must be a contiguous fp32 [{B}, {Hq}] tensor on {dev}")
    ldacc = 0 if acc is None else _matrix(acc, "acc", torch.float32, B, cache.capacity, dev)
    key = (Hq, acc is not None)
    need = cache._need.get(key)
    if need is None:
        need = cache._need[key] = int(lib().kv_attend_workspace_size(cache._ref, Hq, int(acc is not None)))
    if out is None:
        out = torch.empty(B, Hq, D, dtype=torch.float32, device=dev)
    # torch hands the workspace out again only behind this call on its stream,
    # and a captured call's belongs to its graph
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    st = lib().kv_attend(cache._ref, q.data_ptr(), ldq, Hq, D ** -0.5 if scale is None else scale, window,
                         out.data_ptr(), ldo, _ptr(lse), _ptr(acc), ldacc, _ptr(ws), _room(ws, dev),
                         torch._C._cuda_getCurrentRawStream(dev.index))
    if st != 0:
        _check(st, "kv_attend")
    return out


def kv_evict(cache: KvCache, acc, keep: int, recent: int = 0, dst: KvCache | None = None, acc_out=None, kept=None,
             ws=None, stream=None):
    """Cuts every sequence to `keep` slots: its last `recent` ones and those
    with the largest acc (fp32 [seqs, >= capacity], as kv_attend gathers it;
    ties to the lower slot). The kept slots move to the front in their order,
    in place or into dst (a cache of other pages); acc moves along, in place
    or into acc_out. kept: int32 [seqs, >= keep], filled with the kept slots'
    old places and -1. Returns the new lengths."""
    torch, dev, B = _torch(), cache.device, cache.seqs
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return kv_evict(cache, acc, keep, recent, dst, acc_out, kept, ws)
    if dst is None:
        dst = cache
    elif dst.device != dev:
        raise ValueError("dst must be on the cache's device")
    if acc_out is None:
        acc_out = acc
    ld = _matrix(acc, "acc", torch.float32, B, cache.capacity, dev)
    ldo = _matrix(acc_out, "acc_out", torch.float32, B, cache.capacity, dev)
    ldk = 0 if kept is None else _matrix(kept, "kept", torch.int32, B, keep, dev)
    key = (keep, kept is None, "evict")
    need = cache._need.get(key)
    if need is None:
        need = cache._need[key] = int(lib().kv_evict_workspace_size(cache._ref, keep, int(kept is not None)))
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    st = lib().kv_evict(cache._ref, acc.data_ptr(), ld, keep, recent, dst._ref, acc_out.data_ptr(), ldo, _ptr(kept),
                        ldk, _ptr(ws), _room(ws, dev), torch._C._cuda_getCurrentRawStream(dev.index))
    if st != 0:
        _check(st, "kv_evict")
    return dst.lengths


# ---------------------------------------------------------------- scoring

def token_logprobs(logits, tokens=None, top: int = 0, stream=None):
    """Per row of logits (fp32 [M, V], as the head writes them): (logp [M] of
    tokens (int32 [M], -1 scores nothing), entropy [M], the `top` best tokens'
    top_logp [M, top] and top_ids int32 [M, top], best first). logp is None
    without tokens, the last two without top."""
    torch, dev = _torch(), logits.device
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    if _elsewhere(dev, stream):
        with _On(dev, stream):
            return token_logprobs(logits, tokens, top)
    shape, f32 = logits.shape, torch.float32
    if len(shape) != 2:
        if len(shape) != 1:
            raise ValueError("logits must be [M, V]")
        logits = logits.view(1, -1)
        shape = logits.shape
    M, V = shape
    ld = _matrix(logits, "logits", f32, M, V, dev)
    t = lp = tl = ti = 0
    logp = top_logp = top_ids = None
    new = logits.new_empty
    if tokens is not None:
        t = _vector(tokens, "tokens", torch.int32, M, dev)
        logp = new(M)
        lp = logp.data_ptr()
    entropy = new(M)
    if top > 0:
        top_logp = new(M, top)
        top_ids = new(M, top, dtype=torch.int32)
        tl, ti = top_logp.data_ptr(), top_ids.data_ptr()
    st = lib().token_logprobs(logits.data_ptr(), ld, t, M, V, top, lp, entropy.data_ptr(), tl, ti,
                              torch._C._cuda_getCurrentRawStream(dev.index))
    if st != 0:
        _check(st, "token_logprobs")
    return logp, entropy, top_logp, top_ids


# ---------------------------------------------------------------- quantisers

SCALE_TYPES = {"fp32": 0, "fp16": 1}


def w4_quantize(w, block: int = 32, scale_type: str = "fp32", stream=None):
    """The export's dq4 step on the GPU: fp32 w [K, N] -> (qw [K*N/2] uint8,
    scales [K/block, N] fp32 or fp16, zp [(K/block)*N/2] uint8)."""
    torch = _torch()
    if w.dim() != 2 or w.dtype != torch.float32:
        raise ValueError("w must be a 2-D fp32 tensor")
    if scale_type not in SCALE_TYPES:
        raise ValueError(f"scale_type must be one of {sorted(SCALE_TYPES)}")
    K, N = w.shape
    nb = K // block if block > 0 else 0
    qw = torch.empty(K * N // 2, dtype=torch.uint8, device=w.device)
    sc = torch.empty((nb, N), dtype=torch.float32 if scale_type == "fp32" else torch.float16, device=w.device)
    zp = torch.empty(nb * N // 2, dtype=torch.uint8, device=w.device)
    st = lib().w4_quantize(_ptr(w), _ld(w, N), K, N, block, SCALE_TYPES[scale_type], _ptr(qw), _ptr(sc), _ptr(zp),
                           _stream_handle(stream))
    _check(st, "w4_quantize")
    return qw, sc, zp


def i8_quantize_head(w, stream=None):
    """The export's embedding_int8 step on the GPU: fp32 w [K, V] ->
    (table [K, V] int8, scales [V] fp32)."""
    torch = _torch()
    if w.dim() != 2 or w.dtype != torch.float32:
        raise ValueError("w must be a 2-D fp32 tensor")
    K, V = w.shape
    table = torch.empty((K, V), dtype=torch.int8, device=w.device)
    sc = torch.empty(V, dtype=torch.float32, device=w.device)
    st = lib().i8_quantize_head(_ptr(w), _ld(w, V), K, V, _ptr(table), V, _ptr(sc), _stream_handle(stream))
    _check(st, "i8_quantize_head")
    return table, sc


# ---------------------------------------------------------------- host packing

def pack_nibbles(q) -> np.ndarray:
    q = np.ascontiguousarray(q, dtype=np.uint8).reshape(-1)
    out = np.zeros((q.size + 1) // 2, dtype=np.uint8)
    _check(lib().w4_pack_nibbles(q.ctypes.data, q.size, out.ctypes.data), "w4_pack_nibbles")
    return out


def unpack_nibbles(packed, n: int) -> np.ndarray:
    p = np.ascontiguousarray(packed, dtype=np.uint8).reshape(-1)
    if 2 * p.size < n:
        raise ValueError("buffer too small")
    out = np.zeros(n, dtype=np.uint8)
    _check(lib().w4_unpack_nibbles(p.ctypes.data, n, out.ctypes.data), "w4_unpack_nibbles")
    return out


# ---------------------------------------------------------------- diagnostics

def device_error(clear: bool = True):
    """(status, [status, kernel, block, detail]) of the current device's error word."""
    info = (C.c_int32 * 4)()
    st = lib().w4_device_error(info, 1 if clear else 0)
    return st, list(info)


def set_wait_timeout_ns(ns: int) -> None:
    _check(lib().w4_set_wait_timeout_ns(ns), "w4_set_wait_timeout_ns")


def debug_wait_timeout(ns: int, stream=None) -> None:
    _check(lib().w4_debug_wait_timeout(ns, _stream_handle(stream)), "w4_debug_wait_timeout")
