"""Binding of the norms of queries and keys with rotary positions in the same
pass (include/swab.h): forward, gradient, and fused with the cache write.

Marshalling and checks like serve.py, whose compiled module takes the usual
call; what that finds unusual is checked and made here.
"""
from __future__ import annotations

import ctypes

import torch

from . import _binding as _b
from . import serve as _s


class _NormDesc(ctypes.Structure):
    _fields_ = [("eps", ctypes.c_float), ("offset", ctypes.c_float), ("q_stride", _s._S3), ("k_stride", _s._S3)]


def signatures():
    """Argument types of the entry points below, by name (used by load())."""
    P = ctypes.c_void_p
    R, N, C = (ctypes.POINTER(t) for t in (_s._RotaryDesc, _NormDesc, _s._CacheDesc))
    return {
        "norm_rotary": [R, N] + [P] * 9,
        "norm_rotary_bwd": [R, N] + [P] * 14,
        "norm_rotary_append": [R, N, C] + [P] * 12,
    }


class NormDesc:
    """RMS norm of a head (swab_norm_desc): x_c / sqrt(mean(x^2) + eps) * (w_c +
    offset); ``offset`` 1 where a model stores its weights less 1."""

    def __init__(self, eps=1e-6, offset=0.0):
        self.eps, self.offset = float(eps), float(offset)
        self.c = _NormDesc(self.eps, self.offset)
        self._ref, self._addr = ctypes.byref(self.c), ctypes.addressof(self.c)

    def struct(self, d, q, k):
        """The C struct with Q's and K's strides (norm_rotary_bwd)."""
        zero = (0, 0, 0)
        return ctypes.byref(_NormDesc(self.eps, self.offset, _s._S3(*(_s._row_strides("Q", q, d, d.h) if q else zero)),
                                      _s._S3(*(_s._row_strides("K", k, d, d.hk) if k else zero))))


def _vector(name, t, n, dtype, dev):
    """Pointer of a contiguous tensor [n], None for None."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise _s._place(name, t, dev)
    if t.dtype is not dtype or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor [{n}], got {list(t.shape)} {t.dtype}")
    return t.data_ptr()


def _pos(desc, pos, dev):
    return None if pos is None else _s._ints("pos", pos, desc.tokens, dev)


def _heads(desc, names, tensors, shapes, dev):
    return [_s._rows(n, t, desc, shapes, dev) for n, t in zip(names, tensors)]


def _calls():
    return _s._calls or _s._load_calls()


def norm_rotary(desc: _s.RotaryDesc, norm: NormDesc, turns, Q, Qo, K=None, Ko=None, wq=None, wk=None, pos=None, stream=None):
    """Norms of Q [b, n, h, hd] -> Qo and K [b, n, hk, hd] -> Ko, a head at a time,
    and rotary positions, in one pass (any strides with adjacent channels; an
    output may be its own input).  Weights wq, wk [hd] of the same type, None:
    1.  turns, pos as for rotary."""
    if stream is None and _s._done("norm_rotary", _calls().norm_rotary(desc._addr, norm._addr, turns, pos, Q, K, wq, wk, Qo, Ko)):
        return
    dev = _s._device("Q", Q)
    q, qo = _heads(desc, ("Q", "Qo"), (Q, Qo), desc._q, dev)
    k = ko = sk = sko = None
    if desc.hk > 0:
        if K is None or Ko is None:
            raise ValueError("K, Ko: needed when hk > 0")
        (k, ko), sk, sko = _heads(desc, ("K", "Ko"), (K, Ko), desc._k, dev), K.stride(), Ko.stride()
    w = [_vector(n, t, desc.head_dim, desc.dtype, dev) for n, t in (("wq", wq), ("wk", wk))]
    _s._run("norm_rotary", dev, stream, desc.struct(Q.stride(), sk, Qo.stride(), sko), norm._ref, _s._turns(desc, turns, dev),
            _pos(desc, pos, dev), q, k, *w, qo, ko)


def norm_rotary_bwd_workspace(desc: _s.RotaryDesc) -> int:
    """Bytes of device workspace norm_rotary_bwd needs for the weights' gradients."""
    return int(_b.load().norm_rotary_bwd_workspace(ctypes.byref(desc._plain)))


def norm_rotary_bwd(desc: _s.RotaryDesc, norm: NormDesc, turns, dQo, Q, dQ, dKo=None, K=None, dK=None, wq=None, wk=None, dwq=None,
                    dwk=None, workspace=None, pos=None, stream=None):
    """Gradient of norm_rotary: dQo and the call's Q -> dQ, dKo and K -> dK (dQ may
    be dQo or Q), and the weights' gradients dwq, dwk [hd] float32, summed over
    all rows (without keys dwk is 0; None: left out; they need workspace)."""
    if stream is None and _s._done("norm_rotary_bwd", _calls().norm_rotary_bwd(desc._addr, norm._addr, turns, pos, dQo, dKo, Q, K, wq, wk,
                                                                               dQ, dK, dwq, dwk, workspace)):
        return
    d, dev = desc, _s._device("dQo", dQo)
    go, q, dq = _heads(d, ("dQo", "Q", "dQ"), (dQo, Q, dQ), d._q, dev)
    gk = k = dk = sg = sk = sd = None
    if d.hk > 0:
        if dKo is None or K is None or dK is None:
            raise ValueError("dKo, K, dK: needed when hk > 0")
        gk, k, dk = _heads(d, ("dKo", "K", "dK"), (dKo, K, dK), d._k, dev)
        sg, sk, sd = dKo.stride(), K.stride(), dK.stride()
    w = [_vector(n, t, d.head_dim, d.dtype, dev) for n, t in (("wq", wq), ("wk", wk))]
    dw = [_vector(n, t, d.head_dim, torch.float32, dev) for n, t in (("dwq", dwq), ("dwk", dwk))]
    if workspace is not None:
        if workspace.get_device() != dev:
            raise _s._place("workspace", workspace, dev)
        if workspace.numel() * workspace.element_size() < norm_rotary_bwd_workspace(d) or not workspace.is_contiguous():
            raise ValueError(f"workspace: expected at least {norm_rotary_bwd_workspace(d)} contiguous bytes")
    elif dwq is not None or dwk is not None:
        raise ValueError("workspace: needed for dwq, dwk (norm_rotary_bwd_workspace)")
    _s._run("norm_rotary_bwd", dev, stream, d.struct(dQo.stride(), sg, dQ.stride(), sd), norm.struct(d, Q.stride(), sk),
            _s._turns(d, turns, dev), _pos(d, pos, dev), go, gk, q, k, *w, dq, dk, *dw,
            None if workspace is None else workspace.data_ptr())


def _append(desc, turns, Q, K, V, pos, slots, Qo, wq, wk):
    """What the appending calls share: (device, struct, turns, [pos, slots, Q, K, V, wq, wk, Qo])."""
    if (Q is None) != (Qo is None):
        raise ValueError("Q, Qo: both or neither")
    if slots is None:
        raise ValueError("slots: needed")
    dev = _s._device("K", K)
    k, v = _heads(desc, ("K", "V"), (K, V), desc._k, dev)
    at = _s._ints("slots", slots, desc.tokens, dev)
    q = qo = sq = sqo = None
    if Q is not None:
        (q, qo), sq, sqo = _heads(desc, ("Q", "Qo"), (Q, Qo), desc._q, dev), Q.stride(), Qo.stride()
    w = [_vector(n, t, desc.head_dim, desc.dtype, dev) for n, t in (("wq", wq), ("wk", wk))]
    return dev, desc.struct(sq, K.stride(), sqo, None, V.stride()), _s._turns(desc, turns, dev), [_pos(desc, pos, dev), at, q, k, v, *w, qo]


def norm_rotary_append(desc: _s.RotaryDesc, norm: NormDesc, cache: _s.CacheDesc, turns, Q, K, V, pos, slots, Qo, Kc, Vc, wq=None,
                       wk=None, stream=None):
    """rotary_append with Q and K normed first: norms and rotary positions on Q ->
    Qo, the same on K, and V as it is, into the rows slots[t] of the cache
    tensors Kc, Vc [n_blocks, hk, page, hd]."""
    if stream is None and _s._done("norm_rotary_append", _calls().norm_rotary_append(
            desc._addr, norm._addr, cache._addr, turns, pos, slots, Q, K, V, wq, wk, Qo, Kc, Vc)):
        return
    dev, struct, t, args = _append(desc, turns, Q, K, V, pos, slots, Qo, wq, wk)
    kv = (cache.n_blocks, desc.hk, cache.page, desc.head_dim)
    _s._run("norm_rotary_append", dev, stream, struct, norm._ref, cache._ref, t, *args, _s._cache("Kc", Kc, kv, desc.dtype, dev),
            _s._cache("Vc", Vc, kv, desc.dtype, dev))


def check_norm(rotary: _s.RotaryDesc, norm):
    """Raises the error with which the calls would refuse this norm (None: no norm),
    stopped by a pointer off its alignment as in check_step."""
    if norm is None:
        return
    ok, odd = 16, 2
    rc = _b.load().norm_rotary(ctypes.byref(rotary._plain), norm._ref, ok, ok, odd, odd, ok, ok, odd, odd, None)
    if rc != _b.STATUS_NAMES.index("SWAB_ERR_MISALIGNED"):
        raise _b.SwabError("norm_rotary", rc)
