"""Binding of the entry points for answering with the banded attention
(include/swab.h): rotary positions, block tables and slot maps, the cache
write, and decode over the paged cache.

Argument marshalling and checks only, like the rest of the binding.  Every
tensor of a call lies on one CUDA device; the call runs on that device's
current stream (or the stream given), whichever device is current.
"""
from __future__ import annotations

import ctypes

import torch

from . import _binding as _b

_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}
_S3 = ctypes.c_int64 * 3


class _CacheDesc(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int32) for k in ("batch", "page", "n_blocks", "cols", "ring", "pinned")]


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


class CacheDesc:
    """A paged cache (swab_cache_desc): K and V as [n_blocks, hk, page, head_dim]
    and a block table [batch, cols]; with ``ring`` the columns from ``pinned``
    on are recycled once a window has left their blocks."""

    def __init__(self, batch, page, n_blocks, cols, ring=False, pinned=0):
        self.batch, self.page, self.n_blocks, self.cols = int(batch), int(page), int(n_blocks), int(cols)
        self.ring, self.pinned = bool(ring), int(pinned)
        self.c = _CacheDesc(self.batch, self.page, self.n_blocks, self.cols, int(self.ring), self.pinned)


class RotaryDesc:
    """Rotary positions (swab_rotary_desc) over tokens [b, n] with h query and hk
    key heads; ``scale`` multiplies cos and sin, ``pos0`` is added to every
    position.  The strides come from the tensors of each call."""

    def __init__(self, b, n, h, hk, head_dim, rot_dim, interleaved=False, scale=1.0, pos0=0, dtype=torch.float16):
        if dtype not in _b._DTYPES:
            raise ValueError(f"unsupported dtype {dtype}")
        self.b, self.n, self.h, self.hk = int(b), int(n), int(h), int(hk)
        self.head_dim, self.rot_dim, self.interleaved = int(head_dim), int(rot_dim), bool(interleaved)
        self.scale, self.pos0, self.dtype = float(scale), int(pos0), dtype
        self._structs = {}      # the C struct by the strides of a call

    def struct(self, q=None, k=None, qo=None, ko=None, v=None):
        key = (q, k, qo, ko, v)
        c = self._structs.get(key)
        if c is None:
            zero = (0, 0, 0)
            c = _RotaryDesc(self.b, self.n, self.h, self.hk, self.head_dim, self.rot_dim, int(self.interleaved),
                            _b._DTYPES[self.dtype], self.scale, self.pos0, *(_S3(*(s or zero)) for s in key))
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
        self.cache, self.tokens, self.h, self.hk, self.head_dim = cache, int(tokens), int(h), int(hk), int(head_dim)
        self.w = 1 << 30 if w is None else int(w)
        self.dilation, self.n_sink, self.max_q = int(dilation), int(n_sink), int(max_q)
        self.max_len = cache.cols * cache.page if max_len is None else int(max_len)
        self.prefix_len, self.dtype = int(prefix_len), dtype
        self.q_row_stride, self.out_row_stride = int(q_row_stride), int(out_row_stride)
        self.c = _DecodeDesc(cache.c, self.tokens, self.h, self.hk, self.head_dim, self.w, self.dilation, self.n_sink,
                             self.max_q, self.max_len, self.prefix_len, _b._DTYPES[dtype], self.q_row_stride,
                             self.out_row_stride)
        self.workspace_bytes = None


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------
def _run(name, like, stream, *args):
    """Call `name` with the stream appended, on the device of the tensor `like`."""
    dev = like.device
    if stream is None:
        s = torch.cuda.current_stream(dev).cuda_stream
    else:
        s = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)
    fn = getattr(_b.load(), name)
    if torch.cuda.current_device() == dev.index:
        rc = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, s)
    if rc != _b.SWAB_OK:
        raise _b.SwabError(name, rc)


def _on(name, t, like):
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if like is not None and t.device != like.device:
        raise ValueError(f"{name}: on {t.device}, the call's other tensors are on {like.device}")


def _ints(name, t, n, like):
    """Pointer of a contiguous int32 tensor of n elements (None: None)."""
    if t is None:
        return None
    _on(name, t, like)
    if t.dtype != torch.int32 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous int32 tensor of {n} elements, got {tuple(t.shape)} {t.dtype}")
    return t.data_ptr()


def _turns(d, t, like):
    if d.rot_dim == 0:
        return None
    if t is None:
        raise ValueError("turns: needed when rot_dim > 0")
    _on("turns", t, like)
    if t.dtype != torch.int64 or t.numel() != d.rot_dim // 2 or not t.is_contiguous():
        raise ValueError(f"turns: expected {d.rot_dim // 2} contiguous int64 values (rotary_frequencies), got "
                         f"{tuple(t.shape)} {t.dtype}")
    return t.data_ptr()


def _rows(name, t, d, heads, like):
    """(pointer, element strides over (b, n, head)) of a [b, n, heads, hd] or, the
    tokens flat, [b * n, heads, hd] tensor with adjacent channels."""
    _on(name, t, like)
    if t.dtype != d.dtype:
        raise ValueError(f"{name}: expected dtype {d.dtype}, got {t.dtype}")
    shape, st = t.shape, t.stride()
    if len(shape) == 3 and tuple(shape) == (d.b * d.n, heads, d.head_dim):
        sizes, strides = (d.b, d.n, heads), (d.n * st[0], st[0], st[1])
    elif len(shape) == 4 and tuple(shape) == (d.b, d.n, heads, d.head_dim):
        sizes, strides = (d.b, d.n, heads), st[:3]
    else:
        raise ValueError(f"{name}: expected [{d.b}, {d.n}, {heads}, {d.head_dim}] (or the tokens flat), got {tuple(shape)}")
    if st[-1] != 1 and d.head_dim > 1:
        raise ValueError(f"{name}: the channels must be adjacent")
    strides = tuple(0 if k == 1 else s for k, s in zip(sizes, strides))   # a single element's stride says nothing
    if not any(strides) and max(sizes) > 1:
        raise ValueError(f"{name}: the same row for every token and head")
    return t.data_ptr(), strides


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
    turns = torch.empty(max(int(rot_dim), 0) // 2, dtype=torch.int64)
    scale = ctypes.c_float(1.0)
    rc = _b.load().rotary_frequencies(int(rot_dim), float(base), _SCALING[scaling], float(factor), float(original),
                                      float(low_turns), float(high_turns), turns.data_ptr(), ctypes.byref(scale))
    if rc != _b.SWAB_OK:
        raise _b.SwabError("rotary_frequencies", rc)
    return turns, float(scale.value)


def _rotary(fn, d, turns, Q, Qo, K, Ko, pos, stream):
    q, sq = _rows("Q", Q, d, d.h, None)
    qo, sqo = _rows("Qo", Qo, d, d.h, Q)
    k = ko = sk = sko = None
    if d.hk > 0:
        if K is None or Ko is None:
            raise ValueError("K, Ko: needed when hk > 0")
        k, sk = _rows("K", K, d, d.hk, Q)
        ko, sko = _rows("Ko", Ko, d, d.hk, Q)
    _run(fn, Q, stream, d.struct(sq, sk, sqo, sko), _turns(d, turns, Q), _ints("pos", pos, d.b * d.n, Q), q, k, qo, ko)


def rotary(desc: RotaryDesc, turns, Q, Qo, K=None, Ko=None, pos=None, stream=None):
    """Rotary positions: Q [b, n, h, hd] -> Qo and K [b, n, hk, hd] -> Ko (any
    strides with adjacent channels; an output may be its own input).  pos
    [b, n] int32, None for 0, 1, ... in every sequence."""
    _rotary("rotary", desc, turns, Q, Qo, K, Ko, pos, stream)


def rotary_bwd(desc: RotaryDesc, turns, dQo, dQ, dKo=None, dK=None, pos=None, stream=None):
    """Gradient of rotary: dQo -> dQ and dKo -> dK."""
    _rotary("rotary_bwd", desc, turns, dQo, dQ, dKo, dK, pos, stream)


def cache_slots(cache: CacheDesc, lens, n_new, table, free_list, used, lens_out, used_out, q_start, slots, pos, pos0=0,
                stream=None):
    """Block tables and slot maps for a step that adds n_new[r] tokens to request
    r's lens[r]: new blocks from free_list[used[0]:] into `table` [batch, cols],
    q_start [batch + 1], and for every new token its slot and position (rows
    past the last token: -1 and 0).  lens_out [batch] (may be lens) and
    used_out [2] (may be used): lengths and blocks taken after the step, and
    how many blocks were missing (such requests get slots of -1)."""
    B = cache.batch
    n_free = free_list.numel()
    tokens = slots.numel()
    args = [_ints("lens", lens, B, None), _ints("n_new", n_new, B, lens), _ints("table", table, B * cache.cols, lens),
            _ints("free_list", free_list, n_free, lens)]
    _on("used", used, lens)
    if used.dtype != torch.int32 or used.numel() < 1 or not used.is_contiguous():
        raise ValueError("used: expected a contiguous int32 tensor")
    outs = [_ints("lens_out", lens_out, B, lens), _ints("used_out", used_out, 2, lens), _ints("q_start", q_start, B + 1, lens),
            _ints("slots", slots, tokens, lens), _ints("pos", pos, tokens, lens)]
    _run("cache_slots", lens, stream, ctypes.byref(cache.c), tokens, int(pos0), *args, n_free, used.data_ptr(), *outs)


def _cache(name, t, c, d, like):
    _on(name, t, like)
    if t.dtype != d.dtype or tuple(t.shape) != (c.n_blocks, d.hk, c.page, d.head_dim) or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {d.dtype} tensor [{c.n_blocks}, {d.hk}, {c.page}, {d.head_dim}], got "
                         f"{tuple(t.shape)} {t.dtype}")
    return t.data_ptr()


def rotary_append(desc: RotaryDesc, cache: CacheDesc, turns, Q, K, V, pos, slots, Qo, Kc, Vc, stream=None):
    """rotary on Q -> Qo, and K (rotated) and V into the rows slots[t] of the
    cache tensors Kc, Vc [n_blocks, hk, page, hd]; slot -1 is not written.  Q
    and Qo may both be None."""
    q = qo = sq = sqo = None
    if (Q is None) != (Qo is None):
        raise ValueError("Q, Qo: both or neither")
    if Q is not None:
        q, sq = _rows("Q", Q, desc, desc.h, K)
        qo, sqo = _rows("Qo", Qo, desc, desc.h, K)
    k, sk = _rows("K", K, desc, desc.hk, None)
    v, sv = _rows("V", V, desc, desc.hk, K)
    n = desc.b * desc.n
    if slots is None:
        raise ValueError("slots: needed")
    _run("rotary_append", K, stream, desc.struct(sq, sk, sqo, None, sv), ctypes.byref(cache.c), _turns(desc, turns, K),
         _ints("pos", pos, n, K), _ints("slots", slots, n, K), q, k, v, qo, _cache("Kc", Kc, cache, desc, K),
         _cache("Vc", Vc, cache, desc, K))


def band_decode_workspace(desc: DecodeDesc) -> int:
    """Bytes of device workspace band_decode needs (0: none)."""
    if desc.workspace_bytes is None:
        desc.workspace_bytes = int(_b.load().band_decode_workspace(ctypes.byref(desc.c)))
    return desc.workspace_bytes


def _heads(name, t, d, row_stride, like):
    _on(name, t, like)
    st = row_stride or d.h * d.head_dim
    if t.dtype != d.dtype or tuple(t.shape) != (d.tokens, d.h, d.head_dim):
        raise ValueError(f"{name}: expected [{d.tokens}, {d.h}, {d.head_dim}] {d.dtype}, got {tuple(t.shape)} {t.dtype}")
    s = t.stride()
    if (s[0] != st and d.tokens > 1) or (s[1] != d.head_dim and d.h > 1) or (s[2] != 1 and d.head_dim > 1):
        raise ValueError(f"{name}: expected strides ({st}, {d.head_dim}, 1), got {s}")
    return t.data_ptr()


def band_decode(desc: DecodeDesc, scale, Q, Kc, Vc, table, lens, q_start, O, lse=None, workspace=None, prefix_table=None,
                stream=None):
    """Banded attention of the new tokens over the paged cache: O [tokens, h, hd]
    (and lse [tokens, h] fp32) of queries Q whose rows q_start[r]:q_start[r + 1]
    are the last positions of request r's lens[r].  With ``prefix_len`` the
    shared prefix lies in the blocks prefix_table of the same cache."""
    c = desc.cache
    args = [_heads("Q", Q, desc, desc.q_row_stride, None), _cache("Kc", Kc, c, desc, Q), _cache("Vc", Vc, c, desc, Q),
            _ints("table", table, c.batch * c.cols, Q), _ints("lens", lens, c.batch, Q),
            _ints("q_start", q_start, c.batch + 1, Q)]
    pt = None
    if desc.prefix_len > 0:
        if prefix_table is None:
            raise ValueError("prefix_table: needed when prefix_len > 0")
        pt = _ints("prefix_table", prefix_table, -(-desc.prefix_len // c.page), Q)
    o = _heads("O", O, desc, desc.out_row_stride, Q)
    if lse is not None:
        _on("lse", lse, Q)
        if lse.dtype != torch.float32 or tuple(lse.shape) != (desc.tokens, desc.h) or not lse.is_contiguous():
            raise ValueError(f"lse: expected a contiguous float32 tensor [{desc.tokens}, {desc.h}]")
    need = band_decode_workspace(desc)
    if need:
        if workspace is None:
            raise ValueError("workspace: needed (band_decode_workspace)")
        _on("workspace", workspace, Q)
        if workspace.numel() * workspace.element_size() < need or not workspace.is_contiguous():
            raise ValueError(f"workspace: expected at least {need} contiguous bytes")
    _run("band_decode", Q, stream, ctypes.byref(desc.c), float(scale), *args, pt, o,
         lse.data_ptr() if lse is not None else None, workspace.data_ptr() if need else None)
