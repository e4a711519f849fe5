"""Binding of the cache held in 4 bits (include/swab.h): the write with norms and
rotary positions, rows read back, and decode over it.

K and V are codes [n_blocks, hk, page, head_dim / 2] (uint8, an even channel in
the low half of a byte) and scales [n_blocks, hk, page, head_dim / 32] of the
tensors' type; a code c stands for scale * (c - 8).

Marshalling and checks like serve.py, whose compiled module takes the usual
call; what that finds unusual is checked and made here.
"""
from __future__ import annotations

import ctypes

import torch

from . import _binding as _b
from . import norm as _n
from . import serve as _s


def signatures():
    """Argument types of the entry points below, by name (used by load())."""
    P, i32 = ctypes.c_void_p, ctypes.c_int32
    R, N, C, D = (ctypes.POINTER(t) for t in (_s._RotaryDesc, _n._NormDesc, _s._CacheDesc, _s._DecodeDesc))
    return {
        "rotary_append4": [R, N, C] + [P] * 14,
        "cache_read4": [C, i32, i32, i32, i32] + [P] * 8,
        "band_decode4": [D, ctypes.c_float] + [P] * 12,
    }


def cache4_shapes(cache: _s.CacheDesc, hk, head_dim):
    """(shape of the codes, shape of the scales) of K, and of V, in 4 bits."""
    return (cache.n_blocks, hk, cache.page, head_dim // 2), (cache.n_blocks, hk, cache.page, head_dim // 32)


def _cells(cache, hk, hd, dtype, Kc, Ks, Vc, Vs, dev):
    codes, scales = cache4_shapes(cache, hk, hd)
    return [_s._cache("Kc", Kc, codes, torch.uint8, dev), _s._cache("Ks", Ks, scales, dtype, dev),
            _s._cache("Vc", Vc, codes, torch.uint8, dev), _s._cache("Vs", Vs, scales, dtype, dev)]


def rotary_append4(desc: _s.RotaryDesc, cache: _s.CacheDesc, turns, Q, K, V, pos, slots, Qo, Kc, Ks, Vc, Vs, norm=None, wq=None,
                   wk=None, stream=None):
    """rotary_append into a cache in 4 bits: Q -> Qo rotated, K rotated and V as it
    is quantised into the rows slots[t] of codes and scales.  With ``norm`` (a
    NormDesc; weights wq, wk, None: 1) Q and K are normed first."""
    if stream is None and _s._done("rotary_append4", _n._calls().rotary_append4(
            desc._addr, 0 if norm is None else norm._addr, cache._addr, turns, pos, slots, Q, K, V, wq, wk, Qo, Kc, Ks, Vc, Vs)):
        return
    if norm is None and (wq is not None or wk is not None):
        raise ValueError("wq, wk: weights without a norm")
    dev, struct, t, args = _n._append(desc, turns, Q, K, V, pos, slots, Qo, wq, wk)
    _s._run("rotary_append4", dev, stream, struct, None if norm is None else norm._ref, cache._ref, t, *args,
            *_cells(cache, desc.hk, desc.head_dim, desc.dtype, Kc, Ks, Vc, Vs, dev))


def cache_read4(cache: _s.CacheDesc, slots, Kc, Ks, Vc, Vs, K, V, stream=None):
    """The values of the rows slots[t] of a cache in 4 bits -> K, V [tokens, hk,
    hd] (contiguous, of the scales' type).  Rows with slot -1 stay as they are."""
    if stream is None and _s._done("cache_read4", _n._calls().cache_read4(cache._addr, slots, Kc, Ks, Vc, Vs, K, V)):
        return
    dev = _s._device("K", K)
    if K.dim() != 3 or K.dtype not in _b._DTYPES:
        raise ValueError(f"K: expected [tokens, hk, head_dim], float16, bfloat16 or float32, got {list(K.shape)} {K.dtype}")
    T, hk, hd = K.shape
    k, v = _s._cache("K", K, K.shape, K.dtype, dev), _s._cache("V", V, K.shape, K.dtype, dev)
    args = _cells(cache, hk, hd, K.dtype, Kc, Ks, Vc, Vs, dev)
    _s._run("cache_read4", dev, stream, cache._ref, *(_s._number(n, x) for n, x in (("tokens", T), ("hk", hk), ("head_dim", hd))),
            _b._DTYPES[K.dtype], _s._ints("slots", slots, T, dev), *args, k, v)


def band_decode4_workspace(desc: _s.DecodeDesc) -> int:
    """Bytes of device workspace band_decode4 needs (0: none)."""
    if desc._workspace4 is None:
        desc._workspace4 = int(_b.load().band_decode4_workspace(desc._ref))
    return desc._workspace4


def band_decode4(desc: _s.DecodeDesc, scale, Q, Kc, Ks, Vc, Vs, table, lens, q_start, O, lse=None, workspace=None, stream=None):
    """band_decode over a cache in 4 bits (no shared prefix): O [tokens, h, hd]
    (and lse [tokens, h] fp32) of queries Q whose rows q_start[r]:q_start[r + 1]
    are the last positions of request r's lens[r]."""
    need = desc._workspace4
    if need is None:
        need = band_decode4_workspace(desc)
    if stream is None and _s._done("band_decode4", _n._calls().band_decode4(desc._addr, need, scale, Q, Kc, Ks, Vc, Vs, table, lens,
                                                                           q_start, O, lse, workspace)):
        return
    d, dev = desc, _s._device("Q", Q)
    q, o = _s._heads("Q", Q, d, d.q_row_stride, dev), _s._heads("O", O, d, d.out_row_stride, dev)
    cells = _cells(d.cache, d.hk, d.head_dim, d.dtype, Kc, Ks, Vc, Vs, dev)
    ints = [_s._ints(n, t, k, dev) for n, t, k in (("table", table, d._table), ("lens", lens, d._batch), ("q_start", q_start, d._batch + 1))]
    lp = ws = None
    if lse is not None:
        if lse.get_device() != dev:
            raise _s._place("lse", lse, dev)
        if lse.dtype is not torch.float32 or lse.shape != d._shape[:2] or not lse.is_contiguous():
            raise ValueError(f"lse: expected a contiguous float32 tensor [{d.tokens}, {d.h}]")
        lp = lse.data_ptr()
    if need:
        if workspace is None:
            raise ValueError("workspace: needed (band_decode4_workspace)")
        if workspace.get_device() != dev:
            raise _s._place("workspace", workspace, dev)
        if workspace.numel() * workspace.element_size() < need or not workspace.is_contiguous():
            raise ValueError(f"workspace: expected at least {need} contiguous bytes")
        ws = workspace.data_ptr()
    _s._run("band_decode4", dev, stream, d._ref, scale, q, *cells, *ints, o, lp, ws)


def check_step4(cache: _s.CacheDesc, rotary: _s.RotaryDesc, decode: _s.DecodeDesc, bits):
    """Raises the error with which rotary_append4 or band_decode4 would refuse these
    descriptors (with ``bits`` 4), stopped by a pointer off its alignment as in
    check_step: nothing is launched, no GPU is needed."""
    if bits != 4:
        return
    if rotary.head_dim % 32 or rotary.head_dim > 256:
        raise ValueError(f"head_dim: a multiple of 32, at most 256, in 4 bits, got {rotary.head_dim}")
    rc = _b.load().band_decode4(decode._ref, 1.0, *[2] * 11, None)
    if rc != _b.STATUS_NAMES.index("SWAB_ERR_MISALIGNED"):
        raise _b.SwabError("band_decode4", rc)
