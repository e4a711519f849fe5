"""Binding of the entry points for answering with the banded attention
(include/swab.h): rotary positions, block tables and slot maps, the cache
write, and decode over the paged cache.

Argument marshalling and checks only, like the rest of the binding.  Every
tensor of a call lies on one CUDA device; the call runs on that device's
current stream (or the stream given), whichever device is current.

The usual call goes through a compiled module (csrc/serve_call.cpp).  Where
that finds anything unusual, or is not there, the call is checked and made
here.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import warnings

import torch

from . import _binding as _b
from . import build as _build

_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}
_S3 = ctypes.c_int64 * 3


class _CacheDesc(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int32) for k in ("batch", "page", "n_blocks", "cols", "ring", "pinned", "max_new")]


class _RotaryDesc(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int32) for k in ("b", "n", "h", "hk", "head_dim", "rot_dim", "interleaved", "dtype")] + \
        [("scale", ctypes.c_float), ("pos0", ctypes.c_int32)] + \
        [(k, _S3) for k in ("q_stride", "k_stride", "qo_stride", "ko_stride", "v_stride")]


class _DecodeDesc(ctypes.Structure):
    _fields_ = [("cache", _CacheDesc)] + \
        [(k, ctypes.c_int32) for k in ("tokens", "h", "hk", "head_dim", "w", "dilation", "n_sink", "max_q", "max_len",
                                       "prefix_len", "dtype")] + \
        [("q_row_stride", ctypes.c_int64), ("out_row_stride", ctypes.c_int64)]


def signatures():
    """Argument types of the entry points below, by name (used by load())."""
    P, i32, f64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_double
    R, C, D = (ctypes.POINTER(t) for t in (_RotaryDesc, _CacheDesc, _DecodeDesc))
    return {
        "rotary_frequencies": [i32, f64, i32, f64, f64, f64, f64, P, ctypes.POINTER(ctypes.c_float)],
        "rotary": [R, P, P, P, P, P, P, P],
        "rotary_bwd": [R, P, P, P, P, P, P, P],
        "cache_slots": [C, i32, i32, P, P, P, P, i32, P, P, P, P, P, P, P],
        "rotary_append": [R, C, P, P, P, P, P, P, P, P, P, P],
        "band_decode": [D, ctypes.c_float, P, P, P, P, P, P, P, P, P, P, P],
    }


def _number(name, value, bits=32):
    """value as an int; ctypes would cut it down to the field's bits without a word."""
    value = int(value)
    if not -(1 << (bits - 1)) <= value < 1 << (bits - 1):
        raise ValueError(f"{name}: {value} does not fit {bits} bits")
    return value


def _take_numbers(self, bits=32, **values):
    for name, value in values.items():
        setattr(self, name, _number(name, value, bits))


class CacheDesc:
    """A paged cache (swab_cache_desc): K and V as [n_blocks, hk, page, head_dim]
    and a block table [batch, cols]; with ``ring`` the columns from ``pinned``
    on are recycled once a window has left their blocks.  With ``max_new``
    cache_slots serves no request that adds more tokens than that, or more than
    it has rows for (0: no such limits)."""

    def __init__(self, batch, page, n_blocks, cols, ring=False, pinned=0, max_new=0):
        _take_numbers(self, batch=batch, page=page, n_blocks=n_blocks, cols=cols, pinned=pinned, max_new=max_new)
        self.ring = bool(ring)
        self.c = _CacheDesc(self.batch, self.page, self.n_blocks, self.cols, int(self.ring), self.pinned, self.max_new)
        self._ref, self._addr = ctypes.byref(self.c), ctypes.addressof(self.c)


class RotaryDesc:
    """Rotary positions (swab_rotary_desc) over tokens [b, n] with h query and hk
    key heads; ``scale`` multiplies cos and sin, ``pos0`` is added to every
    position.  The strides come from the tensors of each call."""

    def __init__(self, b, n, h, hk, head_dim, rot_dim, interleaved=False, scale=1.0, pos0=0, dtype=torch.float16):
        if dtype not in _b._DTYPES:
            raise ValueError(f"unsupported dtype {dtype}")
        _take_numbers(self, b=b, n=n, h=h, hk=hk, head_dim=head_dim, rot_dim=rot_dim, pos0=pos0)
        self.interleaved, self.scale, self.dtype = bool(interleaved), float(scale), dtype
        self.tokens = self.b * self.n
        # the shapes a tensor of h or hk heads may have: tokens as [b, n] or flat
        self._q = ((self.b, self.n, self.h, self.head_dim), (self.tokens, self.h, self.head_dim))
        self._k = ((self.b, self.n, self.hk, self.head_dim), (self.tokens, self.hk, self.head_dim))
        self._plain = _RotaryDesc(self.b, self.n, self.h, self.hk, self.head_dim, self.rot_dim, int(self.interleaved),
                                  _b._DTYPES[dtype], self.scale, self.pos0)
        self._addr = ctypes.addressof(self._plain)
        self._structs = {}      # the C struct by the strides of a call's tensors

    def struct(self, q=None, k=None, qo=None, ko=None, v=None):
        """The C struct for tensors of these strides, each a tensor's own
        stride() (3 or 4 numbers), or None."""
        key = (q, k, qo, ko, v)
        c = self._structs.get(key)
        if c is None:
            names = (("Q", q, self.h), ("K", k, self.hk), ("Qo", qo, self.h), ("Ko", ko, self.hk), ("V", v, self.hk))
            strides = [_S3(*(_row_strides(n, s, self, heads) if s else (0, 0, 0))) for n, s, heads in names]
            c = _RotaryDesc(self.b, self.n, self.h, self.hk, self.head_dim, self.rot_dim, int(self.interleaved),
                            _b._DTYPES[self.dtype], self.scale, self.pos0, *strides)
            if len(self._structs) < 64:
                self._structs[key] = c
        return ctypes.byref(c)


class DecodeDesc:
    """Decode over a paged cache (swab_decode_desc).  ``w`` keys on the left
    (None: all of them), ``dilation``, ``n_sink`` leading positions every later
    query attends to, ``max_q`` most new tokens of a request, ``max_len`` the
    longest context (it divides the work), ``prefix_len`` positions shared by
    the batch."""

    def __init__(self, cache, tokens, h, hk, head_dim, w=None, dilation=0, n_sink=0, max_q=1, max_len=None, prefix_len=0,
                 dtype=torch.float16, q_row_stride=0, out_row_stride=0):
        if dtype not in _b._DTYPES:
            raise ValueError(f"unsupported dtype {dtype}")
        _take_numbers(self, tokens=tokens, h=h, hk=hk, head_dim=head_dim, w=1 << 30 if w is None else w, dilation=dilation,
                      n_sink=n_sink, max_q=max_q, prefix_len=prefix_len,
                      max_len=min(cache.cols * cache.page, 0x7fffffff) if max_len is None else max_len)
        _take_numbers(self, 64, q_row_stride=q_row_stride, out_row_stride=out_row_stride)
        self.cache, self.dtype = cache, dtype
        self.c = _DecodeDesc(cache.c, self.tokens, self.h, self.hk, self.head_dim, self.w, self.dilation, self.n_sink,
                             self.max_q, self.max_len, self.prefix_len, _b._DTYPES[dtype], self.q_row_stride,
                             self.out_row_stride)
        self._shape = (self.tokens, self.h, self.head_dim)
        self._kv = (cache.n_blocks, self.hk, cache.page, self.head_dim)
        self._batch, self._table = cache.batch, cache.batch * cache.cols
        self._ref, self._addr = ctypes.byref(self.c), ctypes.addressof(self.c)
        self._workspace = None


# ---------------------------------------------------------------------------
# marshalling helpers.  A call of a few microseconds must not wait for its
# checks: the compiled module asks all its tensors; where it returns -1, each
# entry point asks them in one expression, and only when that fails looks again,
# one by one, for the one to name in the error.
# ---------------------------------------------------------------------------
_I32, _F32, _I64 = torch.int32, torch.float32, torch.int64
_fns = {}
_calls = None


class _NoCalls:
    """In place of the compiled module where it has not been built."""

    rotary = rotary_bwd = cache_slots = rotary_append = band_decode = staticmethod(lambda *args: -1)


def _load_calls():
    global _calls
    lib = _b.load()
    calls = _NoCalls
    if os.path.exists(_build.CALLS):
        spec = importlib.util.spec_from_file_location("_serve_call", _build.CALLS)
        try:
            calls = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(calls)
            calls.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
                         for name in ("rotary", "rotary_bwd", "cache_slots", "rotary_append", "band_decode")))
        except ImportError as e:
            warnings.warn(f"the compiled serving calls do not load, they take some microseconds more: {e}")
            calls = _NoCalls
    _calls = calls
    return calls


def _done(name, rc):
    """True when the compiled module has made the call, False when it has to be looked at again."""
    if rc > 0:
        raise _b.SwabError(name, rc)
    return rc == 0


def _run(name, dev, stream, *args):
    """Call `name` with the stream appended, on CUDA device number dev."""
    fn = _fns.get(name)
    if fn is None:
        fn = _fns[name] = getattr(_b.load(), name)
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(dev)
    else:
        s = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)
    if torch._C._cuda_getDevice() == dev:
        rc = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, s)
    if rc:
        raise _b.SwabError(name, rc)


def _unnamed():
    return ValueError("the call's tensors changed while they were checked")


def _place(name, t, dev):
    """The error for a tensor that is not on CUDA device dev (-1: on none)."""
    if not t.is_cuda:
        return ValueError(f"{name}: expected a CUDA tensor")
    return ValueError(f"{name}: on {t.device}, the call's other tensors are on cuda:{dev}")


def _device(name, t):
    dev = t.get_device()
    if dev < 0:
        raise _place(name, t, dev)
    return dev


def _ints(name, t, n, dev):
    """Pointer of a contiguous int32 tensor of n elements."""
    if t.get_device() != dev:
        raise _place(name, t, dev)
    if t.dtype is not _I32 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous int32 tensor of {n} elements, got {tuple(t.shape)} {t.dtype}")
    return t.data_ptr()


def _turns(d, t, dev):
    if d.rot_dim == 0:
        return None
    if t is None:
        raise ValueError("turns: needed when rot_dim > 0")
    if t.get_device() != dev:
        raise _place("turns", t, dev)
    if t.dtype is not _I64 or t.numel() != d.rot_dim // 2 or not t.is_contiguous():
        raise ValueError(f"turns: expected {d.rot_dim // 2} contiguous int64 values (rotary_frequencies), got "
                         f"{tuple(t.shape)} {t.dtype}")
    return t.data_ptr()


def _rows(name, t, d, shapes, dev):
    """Pointer of a tensor of heads; its strides go through d.struct()."""
    if t.get_device() != dev:
        raise _place(name, t, dev)
    if t.dtype is not d.dtype:
        raise ValueError(f"{name}: expected dtype {d.dtype}, got {t.dtype}")
    shape = t.shape
    if shape != shapes[0] and shape != shapes[1]:
        raise ValueError(f"{name}: expected {list(shapes[0])} (or the tokens flat), got {list(shape)}")
    return t.data_ptr()


def _row_strides(name, st, d, heads):
    """Element strides over (b, n, head) from those of a [b, n, heads, hd] or,
    the tokens flat, [b * n, heads, hd] tensor with adjacent channels."""
    sizes, strides = (d.b, d.n, heads), st[:3] if len(st) == 4 else (d.n * st[0], st[0], st[1])
    if st[-1] != 1 and d.head_dim > 1:
        raise ValueError(f"{name}: the channels must be adjacent")
    strides = tuple(0 if k == 1 else s for k, s in zip(sizes, strides))   # a single element's stride says nothing
    if not any(strides) and max(sizes) > 1:
        raise ValueError(f"{name}: the same row for every token and head")
    return strides


# ---------------------------------------------------------------------------
# the entry points (same names as the C ABI)
# ---------------------------------------------------------------------------
def rotary_frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, original=0, low_turns=1.0, high_turns=None):
    """(turns, scale): the int64 CPU tensor of rot_dim / 2 frequencies that the
    rotary calls take (move it to the GPU) and the factor for RotaryDesc(scale=).
    ``scaling``: "none", "linear", "ntk", "yarn" or "bands", to contexts ``factor``
    times the ``original`` length; pairs turning less than ``low_turns`` times
    within it are slowed down by the factor, more than ``high_turns`` (32 for
    "yarn", 4 for "bands") kept."""
    if scaling not in _SCALING:
        raise ValueError(f"scaling: expected one of {sorted(_SCALING)}, got {scaling!r}")
    if high_turns is None:
        high_turns = 32.0 if scaling == "yarn" else 4.0
    rot_dim = _number("rot_dim", rot_dim)
    turns = torch.empty(max(rot_dim, 0) // 2, dtype=torch.int64)
    scale = ctypes.c_float(1.0)
    rc = _b.load().rotary_frequencies(rot_dim, float(base), _SCALING[scaling], float(factor), float(original),
                                      float(low_turns), float(high_turns), turns.data_ptr(), ctypes.byref(scale))
    if rc != _b.SWAB_OK:
        raise _b.SwabError("rotary_frequencies", rc)
    return turns, float(scale.value)


def _rotary(fn, d, turns, Q, Qo, K, Ko, pos, stream):
    dev = _device("Q", Q)
    q, qo = _rows("Q", Q, d, d._q, dev), _rows("Qo", Qo, d, d._q, dev)
    k = ko = sk = sko = None
    if d.hk > 0:
        if K is None or Ko is None:
            raise ValueError("K, Ko: needed when hk > 0")
        k, ko, sk, sko = _rows("K", K, d, d._k, dev), _rows("Ko", Ko, d, d._k, dev), K.stride(), Ko.stride()
    _run(fn, dev, stream, d.struct(Q.stride(), sk, Qo.stride(), sko), _turns(d, turns, dev),
         None if pos is None else _ints("pos", pos, d.tokens, dev), q, k, qo, ko)


def rotary(desc: RotaryDesc, turns, Q, Qo, K=None, Ko=None, pos=None, stream=None):
    """Rotary positions: Q [b, n, h, hd] -> Qo and K [b, n, hk, hd] -> Ko (any
    strides with adjacent channels; an output may be its own input).  pos
    [b, n] int32, None for 0, 1, ... in every sequence."""
    if stream is None and _done("rotary", (_calls or _load_calls()).rotary(desc._addr, turns, pos, Q, K, Qo, Ko)):
        return
    _rotary("rotary", desc, turns, Q, Qo, K, Ko, pos, stream)


def rotary_bwd(desc: RotaryDesc, turns, dQo, dQ, dKo=None, dK=None, pos=None, stream=None):
    """Gradient of rotary: dQo -> dQ and dKo -> dK."""
    if stream is None and _done("rotary_bwd", (_calls or _load_calls()).rotary_bwd(desc._addr, turns, pos, dQo, dKo, dQ, dK)):
        return
    _rotary("rotary_bwd", desc, turns, dQo, dQ, dKo, dK, pos, stream)


def cache_slots(cache: CacheDesc, lens, n_new, table, free_list, used, lens_out, used_out, q_start, slots, pos, pos0=0,
                stream=None):
    """Block tables and slot maps for a step that adds n_new[r] tokens to request
    r's lens[r]: new blocks from free_list[used[0]:] into `table` [batch, cols],
    q_start [batch + 1], and for every new token its slot and position (rows
    past the last token: -1 and 0).  lens_out [batch] (may be lens) and
    used_out [2] (may be used): lengths and blocks taken after the step, and
    how many blocks were missing (such requests get slots of -1)."""
    if stream is None and _done("cache_slots", (_calls or _load_calls()).cache_slots(
            cache._addr, pos0, lens, n_new, table, free_list, used, lens_out, used_out, q_start, slots, pos)):
        return
    B, n_free, tokens, dev = cache.batch, free_list.numel(), slots.numel(), lens.get_device()
    if max(n_free, tokens) > 0x7fffffff:
        raise ValueError(f"free_list, slots: at most 2^31 - 1 elements, got {n_free} and {tokens}")
    pos0 = _number("pos0", pos0)
    if not (dev >= 0 and lens.dtype is _I32 and n_new.dtype is _I32 and table.dtype is _I32 and free_list.dtype is _I32
            and used.dtype is _I32 and lens_out.dtype is _I32 and used_out.dtype is _I32 and q_start.dtype is _I32
            and slots.dtype is _I32 and pos.dtype is _I32 and lens.numel() == B and n_new.numel() == B
            and table.numel() == B * cache.cols and used.numel() >= 1 and lens_out.numel() == B and used_out.numel() == 2
            and q_start.numel() == B + 1 and pos.numel() == tokens and lens.is_contiguous() and n_new.is_contiguous()
            and table.is_contiguous() and free_list.is_contiguous() and used.is_contiguous() and lens_out.is_contiguous()
            and used_out.is_contiguous() and q_start.is_contiguous() and slots.is_contiguous() and pos.is_contiguous()
            and n_new.get_device() == dev and table.get_device() == dev and free_list.get_device() == dev
            and used.get_device() == dev and lens_out.get_device() == dev and used_out.get_device() == dev
            and q_start.get_device() == dev and slots.get_device() == dev and pos.get_device() == dev):
        _device("lens", lens)
        for name, t, n in (("lens", lens, B), ("n_new", n_new, B), ("table", table, B * cache.cols),
                           ("free_list", free_list, n_free), ("used", used, max(1, used.numel())), ("lens_out", lens_out, B),
                           ("used_out", used_out, 2), ("q_start", q_start, B + 1), ("slots", slots, tokens), ("pos", pos, tokens)):
            _ints(name, t, n, dev)
        raise _unnamed()
    _run("cache_slots", dev, stream, cache._ref, tokens, pos0, lens.data_ptr(), n_new.data_ptr(), table.data_ptr(),
         free_list.data_ptr(), n_free, used.data_ptr(), lens_out.data_ptr(), used_out.data_ptr(), q_start.data_ptr(),
         slots.data_ptr(), pos.data_ptr())


def _cache(name, t, shape, dtype, dev):
    if t.get_device() != dev:
        raise _place(name, t, dev)
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor {list(shape)}, got {list(t.shape)} {t.dtype}")
    return t.data_ptr()


def rotary_append(desc: RotaryDesc, cache: CacheDesc, turns, Q, K, V, pos, slots, Qo, Kc, Vc, stream=None):
    """rotary on Q -> Qo, and K (rotated) and V into the rows slots[t] of the
    cache tensors Kc, Vc [n_blocks, hk, page, hd]; slot -1 is not written.  Q
    and Qo may both be None."""
    if stream is None and _done("rotary_append", (_calls or _load_calls()).rotary_append(
            desc._addr, cache._addr, turns, Q, K, V, pos, slots, Qo, Kc, Vc)):
        return
    if (Q is None) != (Qo is None):
        raise ValueError("Q, Qo: both or neither")
    d, dev, dt, n = desc, K.get_device(), desc.dtype, desc.tokens
    kv, ks = (cache.n_blocks, d.hk, cache.page, d.head_dim), d._k
    if not (dev >= 0 and K.dtype is dt and V.dtype is dt and Kc.dtype is dt and Vc.dtype is dt and slots.dtype is _I32
            and (K.shape == ks[1] or K.shape == ks[0]) and (V.shape == ks[1] or V.shape == ks[0]) and Kc.shape == kv
            and Vc.shape == kv and slots.numel() == n and Kc.is_contiguous() and Vc.is_contiguous() and slots.is_contiguous()
            and V.get_device() == dev and Kc.get_device() == dev and Vc.get_device() == dev and slots.get_device() == dev):
        if slots is None:
            raise ValueError("slots: needed")
        _device("K", K)
        _rows("K", K, d, ks, dev)
        _rows("V", V, d, ks, dev)
        _ints("slots", slots, n, dev)
        _cache("Kc", Kc, kv, dt, dev)
        _cache("Vc", Vc, kv, dt, dev)
        raise _unnamed()
    q = qo = sq = sqo = None
    if Q is not None:
        q, qo, sq, sqo = _rows("Q", Q, d, d._q, dev), _rows("Qo", Qo, d, d._q, dev), Q.stride(), Qo.stride()
    _run("rotary_append", dev, stream, d.struct(sq, K.stride(), sqo, None, V.stride()), cache._ref, _turns(d, turns, dev),
         None if pos is None else _ints("pos", pos, n, dev), slots.data_ptr(), q, K.data_ptr(), V.data_ptr(), qo, Kc.data_ptr(),
         Vc.data_ptr())


def band_decode_workspace(desc: DecodeDesc) -> int:
    """Bytes of device workspace band_decode needs (0: none)."""
    if desc._workspace is None:
        desc._workspace = int(_b.load().band_decode_workspace(desc._ref))
    return desc._workspace


def _heads(name, t, d, row_stride, dev):
    if t.get_device() != dev:
        raise _place(name, t, dev)
    if t.dtype is not d.dtype or t.shape != d._shape:
        raise ValueError(f"{name}: expected {list(d._shape)} {d.dtype}, got {list(t.shape)} {t.dtype}")
    if row_stride == 0 and t.is_contiguous():
        return t.data_ptr()
    s, st = t.stride(), row_stride or d.h * d.head_dim
    if (s[0] != st and d.tokens > 1) or (s[1] != d.head_dim and d.h > 1) or (s[2] != 1 and d.head_dim > 1):
        raise ValueError(f"{name}: expected strides ({st}, {d.head_dim}, 1), got {s}")
    return t.data_ptr()


def band_decode(desc: DecodeDesc, scale, Q, Kc, Vc, table, lens, q_start, O, lse=None, workspace=None, prefix_table=None,
                stream=None):
    """Banded attention of the new tokens over the paged cache: O [tokens, h, hd]
    (and lse [tokens, h] fp32) of queries Q whose rows q_start[r]:q_start[r + 1]
    are the last positions of request r's lens[r].  With ``prefix_len`` the
    shared prefix lies in the blocks prefix_table of the same cache."""
    need = desc._workspace
    if need is None:
        need = band_decode_workspace(desc)
    if stream is None and _done("band_decode", (_calls or _load_calls()).band_decode(
            desc._addr, need, scale, Q, Kc, Vc, table, lens, q_start, prefix_table, O, lse, workspace)):
        return
    d, dev, dt, kv = desc, Q.get_device(), desc.dtype, desc._kv
    if not (dev >= 0 and Q.dtype is dt and O.dtype is dt and Kc.dtype is dt and Vc.dtype is dt and table.dtype is _I32
            and lens.dtype is _I32 and q_start.dtype is _I32 and Q.shape == d._shape and O.shape == d._shape and Kc.shape == kv
            and Vc.shape == kv and table.numel() == d._table and lens.numel() == d._batch and q_start.numel() == d._batch + 1
            and Kc.is_contiguous() and Vc.is_contiguous() and table.is_contiguous() and lens.is_contiguous()
            and q_start.is_contiguous() and O.get_device() == dev and Kc.get_device() == dev and Vc.get_device() == dev
            and table.get_device() == dev and lens.get_device() == dev and q_start.get_device() == dev):
        _device("Q", Q)
        _heads("Q", Q, d, d.q_row_stride, dev)
        _heads("O", O, d, d.out_row_stride, dev)
        _cache("Kc", Kc, kv, dt, dev)
        _cache("Vc", Vc, kv, dt, dev)
        _ints("table", table, d._table, dev)
        _ints("lens", lens, d._batch, dev)
        _ints("q_start", q_start, d._batch + 1, dev)
        raise _unnamed()
    if d.q_row_stride or not Q.is_contiguous():
        _heads("Q", Q, d, d.q_row_stride, dev)
    if d.out_row_stride or not O.is_contiguous():
        _heads("O", O, d, d.out_row_stride, dev)
    pt = lp = ws = None
    if d.prefix_len > 0:
        if prefix_table is None:
            raise ValueError("prefix_table: needed when prefix_len > 0")
        pt = _ints("prefix_table", prefix_table, -(-d.prefix_len // d.cache.page), dev)
    if lse is not None:
        if lse.get_device() != dev:
            raise _place("lse", lse, dev)
        if lse.dtype is not _F32 or lse.shape != d._shape[:2] or not lse.is_contiguous():
            raise ValueError(f"lse: expected a contiguous float32 tensor [{d.tokens}, {d.h}]")
        lp = lse.data_ptr()
    if need:
        if workspace is None:
            raise ValueError("workspace: needed (band_decode_workspace)")
        if workspace.get_device() != dev:
            raise _place("workspace", workspace, dev)
        if workspace.numel() * workspace.element_size() < need or not workspace.is_contiguous():
            raise ValueError(f"workspace: expected at least {need} contiguous bytes")
        ws = workspace.data_ptr()
    _run("band_decode", dev, stream, d._ref, scale, Q.data_ptr(), Kc.data_ptr(), Vc.data_ptr(), table.data_ptr(), lens.data_ptr(),
         q_start.data_ptr(), pt, O.data_ptr(), lp, ws)


def check_step(cache: CacheDesc, rotary: RotaryDesc, decode: DecodeDesc):
    """Raises the error with which cache_slots, rotary_append or band_decode would
    refuse these descriptors.  The library looks at them before it looks at
    pointers, so a call with good ones is stopped by a pointer off its alignment:
    nothing is launched, no GPU is needed."""
    ok, odd = 16, 2
    calls = {"cache_slots": (cache._ref, 0, 0, odd, odd, odd, odd, 0, odd, odd, odd, odd, odd, odd, None),
             "rotary_append": (ctypes.byref(rotary._plain), cache._ref, ok, ok, ok, odd, odd, odd, odd, odd, odd, None),
             "band_decode": (decode._ref, 1.0, odd, odd, odd, odd, odd, odd, odd, odd, odd, odd, None)}
    for name, args in calls.items():
        rc = getattr(_b.load(), name)(*args)
        if rc != _b.STATUS_NAMES.index("SWAB_ERR_MISALIGNED"):
            raise _b.SwabError(name, rc)
