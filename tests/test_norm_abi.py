"""Refusals of the norms of queries and keys, the cache in 4 bits and the decode
over it, checked on the host before any CUDA call (fake pointers, never
dereferenced), and the binding's checks."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

import sliding_window_attention_band_gb300 as swab
from sliding_window_attention_band_gb300 import _binding as B
from sliding_window_attention_band_gb300 import build as swab_build
from sliding_window_attention_band_gb300 import norm as nm
from sliding_window_attention_band_gb300 import serve
from test_serve_abi import (CUDA, FAKE, INVALID, MISALIGNED, UNSUPPORTED, FakeCuda, FakeInts, cache_desc, decode_desc,
                            needs_no_gpu, rotary_desc)

REF = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    swab_build.build()
    return B.load()


def norm_desc(eps=1e-6, offset=0.0, q=(0, 0, 0), k=(0, 0, 0)):
    return nm._NormDesc(eps, offset, serve._S3(*q), serve._S3(*k))


def ref(d):
    return REF(d) if d is not None else None


def forward(lib, d, n, turns=FAKE, pos=FAKE, q=FAKE, k=FAKE, wq=FAKE, wk=FAKE, qo=FAKE, ko=FAKE):
    return lib.norm_rotary(ref(d), ref(n), turns, pos, q, k, wq, wk, qo, ko, None)


def backward(lib, d, n, turns=FAKE, pos=FAKE, gq=FAKE, gk=FAKE, q=FAKE, k=FAKE, wq=FAKE, wk=FAKE, dq=FAKE, dk=FAKE, dwq=FAKE,
             dwk=2 * FAKE, ws=FAKE):
    return lib.norm_rotary_bwd(ref(d), ref(n), turns, pos, gq, gk, q, k, wq, wk, dq, dk, dwq, dwk, ws, None)


def append(lib, d, n, c, turns=FAKE, pos=FAKE, slots=FAKE, q=FAKE, k=FAKE, v=FAKE, wq=FAKE, wk=FAKE, qo=FAKE, kc=FAKE, vc=2 * FAKE):
    return lib.norm_rotary_append(ref(d), ref(n), ref(c), turns, pos, slots, q, k, v, wq, wk, qo, kc, vc, None)


def append4(lib, d, n, c, turns=FAKE, pos=FAKE, slots=FAKE, q=FAKE, k=FAKE, v=FAKE, wq=FAKE, wk=FAKE, qo=FAKE, kc=FAKE, ks=3 * FAKE,
            vc=2 * FAKE, vs=4 * FAKE):
    return lib.rotary_append4(ref(d), ref(n), ref(c), turns, pos, slots, q, k, v, wq, wk, qo, kc, ks, vc, vs, None)


def read4(lib, c, tokens=5, hk=2, hd=64, dtype=1, slots=FAKE, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, k=FAKE, v=2 * FAKE):
    return lib.cache_read4(ref(c), tokens, hk, hd, dtype, slots, kc, ks, vc, vs, k, v, None)


def decode4(lib, d, scale=0.125, q=FAKE, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, table=FAKE, lens=FAKE, start=FAKE, o=FAKE, lse=None,
            ws=FAKE):
    return lib.band_decode4(ref(d), scale, q, kc, ks, vc, vs, table, lens, start, o, lse, ws, None)


@pytest.mark.parametrize("bad,want", [
    (dict(b=0), INVALID), (dict(n=0), INVALID), (dict(h=0), INVALID), (dict(hk=-1), INVALID), (dict(rot_dim=66), INVALID),
    (dict(dtype=3), INVALID), (dict(scale=math.nan), INVALID), (dict(pos0=-1), INVALID), (dict(head_dim=68), UNSUPPORTED),
    (dict(head_dim=1024), UNSUPPORTED), (dict(b=1 << 16, n=1 << 16), UNSUPPORTED)])
def test_rows_descriptor(lib, bad, want):
    d, n, c = rotary_desc(**bad), norm_desc(), cache_desc()
    assert forward(lib, d, n) == backward(lib, d, n) == append(lib, d, n, c) == append4(lib, d, n, c) == want
    assert lib.norm_rotary_bwd_workspace(REF(d)) == 0
    assert forward(lib, None, n) == backward(lib, None, n) == append(lib, None, n, c) == append4(lib, None, n, c) == INVALID
    assert lib.norm_rotary_bwd_workspace(None) == 0


@pytest.mark.parametrize("bad", [dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(offset=math.nan),
                                 dict(offset=math.inf)])
def test_norm_descriptor(lib, bad):
    d, n, c = rotary_desc(), norm_desc(**bad), cache_desc()
    assert forward(lib, d, n) == backward(lib, d, n) == append(lib, d, n, c) == append4(lib, d, n, c) == INVALID
    assert forward(lib, d, None) == backward(lib, d, None) == append(lib, d, None, c) == INVALID


def test_pointers_and_strides(lib):
    d, n, c = rotary_desc(), norm_desc(), cache_desc()
    for fn, need, free in ((lambda **kw: forward(lib, d, n, **kw), ("turns", "q", "k", "qo", "ko"), ("wq", "wk")),
                           (lambda **kw: backward(lib, d, n, **kw), ("turns", "gq", "gk", "q", "k", "dq", "dk", "ws"), ("dwq", "dwk")),
                           (lambda **kw: append(lib, d, n, c, **kw), ("turns", "pos", "slots", "q", "k", "v", "qo", "kc", "vc"), ("wq", "wk")),
                           (lambda **kw: append4(lib, d, n, c, **kw),
                            ("turns", "pos", "slots", "q", "k", "v", "qo", "kc", "ks", "vc", "vs"), ("wq", "wk"))):
        for name in need:
            assert fn(**{name: None}) == INVALID, name
            assert fn(**{name: 9 * FAKE + (2 if name in ("pos", "slots") else 4 if name == "turns" else 8)}) == MISALIGNED, name
        for name in free:
            assert fn(**{name: 9 * FAKE + 8}) == MISALIGNED, name
    for name in ("wq", "wk"):
        assert backward(lib, d, n, **{name: None}) == INVALID                     # a gradient of no weight
    assert backward(lib, d, n, dwq=2 * FAKE) == INVALID                           # both gradients in one place
    assert append(lib, d, n, c, vc=FAKE) == append4(lib, d, n, c, vc=FAKE) == INVALID
    for name, other in (("ks", FAKE), ("ks", 2 * FAKE), ("vs", FAKE), ("vs", 2 * FAKE), ("vs", 3 * FAKE)):
        assert append4(lib, d, n, c, **{name: other}) == INVALID
    assert forward(lib, rotary_desc({"q": (2048, 256, 68)}), n) == MISALIGNED
    assert forward(lib, rotary_desc({"qo": (2048, 128, 64)}), n) == INVALID
    assert backward(lib, d, norm_desc(q=(2048, 256, 68))) == MISALIGNED
    assert backward(lib, d, norm_desc(k=(2048, -256, 64))) == INVALID
    assert backward(lib, d, norm_desc(q=(1 << 36, 256, 64))) == UNSUPPORTED
    assert append(lib, rotary_desc(hk=0), n, c) == append4(lib, rotary_desc(hk=0), n, c) == INVALID


@pytest.mark.parametrize("bad,want", [
    (dict(batch=0), INVALID), (dict(n_blocks=0), INVALID), (dict(cols=0), INVALID), (dict(ring=2), INVALID),
    (dict(pinned=1), INVALID), (dict(page=8), UNSUPPORTED), (dict(n_blocks=1 << 27, page=16), UNSUPPORTED)])
def test_cache_descriptor(lib, bad, want):
    c = cache_desc(**bad)
    assert append(lib, rotary_desc(), norm_desc(), c) == append4(lib, rotary_desc(), norm_desc(), c) == read4(lib, c) == want
    assert decode4(lib, decode_desc(c)) == want
    assert lib.band_decode4_workspace(REF(decode_desc(c))) == 0


def test_head_sizes_in_4_bits(lib):
    for hd in (16, 80, 288):
        assert append4(lib, rotary_desc(head_dim=hd, rot_dim=16), norm_desc(), cache_desc()) == UNSUPPORTED
        assert read4(lib, cache_desc(), hd=hd) == UNSUPPORTED
        assert decode4(lib, decode_desc(head_dim=hd)) == UNSUPPORTED
        assert lib.band_decode4_workspace(REF(decode_desc(head_dim=hd))) == 0


def test_read_arguments(lib):
    c = cache_desc()
    for bad in (dict(tokens=0), dict(hk=0), dict(hd=0), dict(dtype=3), dict(v=FAKE)):
        assert read4(lib, c, **bad) == INVALID
    assert read4(lib, None) == INVALID
    assert read4(lib, c, hk=70000) == UNSUPPORTED
    assert read4(lib, cache_desc(n_blocks=1 << 26, page=16), hk=4) == UNSUPPORTED       # 2^32 lines
    for name in ("slots", "kc", "ks", "vc", "vs", "k", "v"):
        assert read4(lib, c, **{name: None}) == INVALID, name
        assert read4(lib, c, **{name: 9 * FAKE + 2}) == MISALIGNED, name


@pytest.mark.parametrize("bad,want", [
    (dict(tokens=0), INVALID), (dict(h=0), INVALID), (dict(hk=3), INVALID), (dict(max_q=0), INVALID), (dict(max_len=0), INVALID),
    (dict(w=-1), INVALID), (dict(dilation=-1), INVALID), (dict(n_sink=-1), INVALID), (dict(dtype=5), INVALID),
    (dict(q_row_stride=64), INVALID), (dict(prefix_len=16), UNSUPPORTED), (dict(h=258, hk=2), UNSUPPORTED),
    (dict(dilation=100), UNSUPPORTED), (dict(q_row_stride=516), MISALIGNED)])
def test_decode_descriptor(lib, bad, want):
    assert decode4(lib, decode_desc(**bad)) == want
    assert lib.band_decode4_workspace(REF(decode_desc(**bad))) == 0
    assert decode4(lib, None) == INVALID


def test_decode_pointers(lib):
    d = decode_desc()
    for name in ("q", "kc", "ks", "vc", "vs", "table", "lens", "start", "o"):
        assert decode4(lib, d, **{name: None}) == INVALID, name
        assert decode4(lib, d, **{name: FAKE + 2}) == MISALIGNED, name
    assert decode4(lib, d, lse=FAKE + 4) == MISALIGNED
    for scale in (math.nan, math.inf):
        assert decode4(lib, d, scale=scale) == INVALID
    cut = decode_desc(cache_desc(cols=4000, n_blocks=9000), max_len=60000, w=1 << 30)
    assert lib.band_decode4_workspace(REF(cut)) > 0
    assert decode4(lib, cut, ws=None) == INVALID and decode4(lib, cut, ws=FAKE + 8) == MISALIGNED


def test_workspace_does_not_overflow(lib):
    """The longest lists, the most rows: sizes stay positive and divide the work."""
    for dtype in (0, 1, 2):
        for hd in (32, 64, 128, 256):
            c = cache_desc(batch=65535, n_blocks=1 << 24, cols=1 << 24)
            d = decode_desc(c, tokens=65535, h=256, hk=2, head_dim=hd, w=1 << 30, max_len=0x7fffffff, max_q=65535, dtype=dtype)
            assert lib.band_decode4_workspace(REF(d)) < 1 << 50


@needs_no_gpu
def test_valid_calls_reach_the_launch(lib):
    d, n, c = rotary_desc(), norm_desc(), cache_desc()
    assert forward(lib, d, n) == forward(lib, d, n, pos=None, wq=None, wk=None) == CUDA
    assert forward(lib, rotary_desc(rot_dim=0), n, turns=None) == forward(lib, rotary_desc(hk=0), n, k=None, ko=None, wk=None) == CUDA
    assert backward(lib, d, n) == backward(lib, d, n, wq=None, wk=None, dwq=None, dwk=None, ws=None) == CUDA
    assert backward(lib, rotary_desc(hk=0), n, gk=None, k=None, wk=None, dk=None, dwk=None) == CUDA
    assert append(lib, d, n, c) == append(lib, d, n, c, q=None, qo=None) == CUDA
    assert append4(lib, d, n, c) == append4(lib, d, None, c, wq=None, wk=None) == append4(lib, d, n, c, q=None, qo=None) == CUDA
    assert append4(lib, rotary_desc(rot_dim=0), n, c, turns=None, pos=None) == read4(lib, c) == CUDA
    assert decode4(lib, decode_desc()) == decode4(lib, decode_desc(head_dim=96)) == CUDA


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
class FakeTensor(FakeCuda):
    def __init__(self, shape, dtype=torch.float16, device=0):
        strides = [1]
        for n in reversed(shape[1:]):
            strides.append(strides[-1] * n)
        super().__init__(torch.Size(shape), tuple(reversed(strides)), dtype, device)

    def numel(self):
        return int(np.prod(self.shape))

    def element_size(self):
        return torch.empty((), dtype=self.dtype).element_size()

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)


def test_binding_names_what_is_wrong(lib):
    T, h, hk, hd, page = 3, 4, 2, 64, 16
    d, n, c = swab.RotaryDesc(1, T, h, hk, hd, hd), swab.NormDesc(), swab.CacheDesc(2, page, 8, 4)
    q, k, w = FakeTensor((T, h, hd)), FakeTensor((T, hk, hd)), FakeTensor((hd,))
    turns, ints, dw = FakeTensor((hd // 2,), torch.int64), FakeInts(T), FakeTensor((hd,), torch.float32)
    codes, scales = (FakeTensor(s, t) for s, t in zip(swab.cache4_shapes(c, hk, hd), (torch.uint8, torch.float16)))
    kv = FakeTensor((8, hk, page, hd))
    assert codes.shape == (8, hk, page, hd // 2) and scales.shape == (8, hk, page, hd // 32)

    def check(fn, args, wrong, match):
        with pytest.raises(ValueError, match=match):
            fn(**{**args, **wrong})

    fwd = dict(desc=d, norm=n, turns=turns, Q=q, Qo=q, K=k, Ko=k, wq=w, wk=w)
    other = FakeTensor((hd,), device=1)
    for wrong, match in ((dict(wq=FakeTensor((hd - 1,))), "wq"), (dict(wk=FakeTensor((hd,), torch.float32)), "wk"), (dict(wq=other), "wq"),
                         (dict(Q=k), "Q"), (dict(Ko=None), "Ko"), (dict(pos=FakeInts(2)), "pos"), (dict(turns=None), "turns")):
        check(swab.norm_rotary, fwd, wrong, match)
    bwd = dict(desc=d, norm=n, turns=turns, dQo=q, Q=q, dQ=q, dKo=k, K=k, dK=k, wq=w, wk=w, dwq=dw, dwk=dw,
               workspace=FakeTensor((swab.norm_rotary_bwd_workspace(d),), torch.uint8))
    for wrong, match in ((dict(dwq=w), "dwq"), (dict(workspace=None), "workspace"), (dict(workspace=FakeTensor((64,), torch.uint8)), "workspace"),
                         (dict(dK=None), "dK"), (dict(Q=FakeTensor((T, h, hd), torch.float32)), "Q")):
        check(swab.norm_rotary_bwd, bwd, wrong, match)
    app = dict(desc=d, norm=n, cache=c, turns=turns, Q=q, K=k, V=k, pos=ints, slots=ints, Qo=q, Kc=kv, Vc=kv, wq=w, wk=w)
    for wrong, match in ((dict(Qo=None), "Qo"), (dict(slots=None), "slots"), (dict(Kc=codes), "Kc"), (dict(V=q), "V"), (dict(wk=other), "wk")):
        check(swab.norm_rotary_append, app, wrong, match)
    app4 = {**{k_: v for k_, v in app.items() if k_ not in ("Kc", "Vc")}, "Kc": codes, "Ks": scales, "Vc": codes, "Vs": scales}
    for wrong, match in ((dict(norm=None), "norm"), (dict(Kc=kv), "Kc"), (dict(Vs=codes), "Vs"), (dict(slots=FakeInts(2)), "slots")):
        check(swab.rotary_append4, app4, wrong, match)
    read = dict(cache=c, slots=ints, Kc=codes, Ks=scales, Vc=codes, Vs=scales, K=k, V=k)
    for wrong, match in ((dict(V=q), "V"), (dict(K=FakeTensor((T, hk, hd), torch.int32)), "K"), (dict(K=w), "K"), (dict(slots=FakeInts(4)), "slots"),
                         (dict(Ks=FakeTensor(scales.shape, torch.float32)), "Ks")):
        check(swab.cache_read4, read, wrong, match)
    dd = swab.DecodeDesc(c, T, h, hk, hd)
    dec = dict(desc=dd, scale=0.1, Q=q, Kc=codes, Ks=scales, Vc=codes, Vs=scales, table=FakeInts(8), lens=FakeInts(2), q_start=FakeInts(3), O=q)
    for wrong, match in ((dict(Kc=kv), "Kc"), (dict(Vs=FakeTensor((8, hk, page, 4))), "Vs"), (dict(lens=FakeInts(3)), "lens"), (dict(O=k), "O"),
                         (dict(lse=dw), "lse")):
        check(swab.band_decode4, dec, wrong, match)
    cut = swab.DecodeDesc(swab.CacheDesc(1, page, 8, 4000), T, h, hk, hd, max_len=60000)
    dec.update(desc=cut, table=FakeInts(4000), lens=FakeInts(1), q_start=FakeInts(2))
    assert swab.band_decode4_workspace(cut) > 0
    check(swab.band_decode4, dec, {}, "workspace")


def test_compiled_calls_leave_what_is_unusual(lib):
    call = serve._calls or serve._load_calls()
    assert call is not serve._NoCalls
    c, r, n = swab.CacheDesc(2, 16, 8, 4), swab.RotaryDesc(1, 2, 4, 2, 64, 64), swab.NormDesc()
    d = swab.DecodeDesc(c, 2, 4, 2, 64)
    f16, i32 = torch.zeros(2, 4, 64, dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    codes = torch.zeros(8, 2, 16, 32, dtype=torch.uint8)
    odd = [None, 3, -1, "x", 1.5, f16, i32, codes, codes.to("meta"), f16.to_sparse(), torch.nn.Parameter(f16), object()]
    rng = np.random.default_rng(0)
    for name, lead, k in (("norm_rotary", (r._addr, n._addr), 10), ("norm_rotary_bwd", (r._addr, n._addr), 15),
                          ("norm_rotary_append", (r._addr, n._addr, c._addr), 14), ("rotary_append4", (r._addr, 0, c._addr), 16),
                          ("rotary_append4", (r._addr, n._addr, c._addr), 16), ("cache_read4", (c._addr,), 8),
                          ("band_decode4", (d._addr, 0, 0.125), 14)):
        fn = getattr(call, name)
        assert fn() == -1 and fn(*lead) == -1 and fn(0, *[None] * (k - 1)) == -1
        for _ in range(60):
            assert fn(*lead, *(odd[i] for i in rng.integers(0, len(odd), k - len(lead)))) == -1
        assert fn("descriptor", *[f16] * (k - 1)) == -1
    for bad in ((), (1, 2)):
        with pytest.raises(TypeError):
            call.bind_more(*bad)
    with pytest.raises(ValueError):
        call.bind_more(*[0] * 7)


def test_structs_follow_the_header():
    n = swab.NormDesc(1e-5, 1.0)
    a = nm._NormDesc.from_address(n._addr)
    assert a.offset == 1.0 and abs(a.eps - 1e-5) < 1e-12 and not any(a.q_stride) and not any(a.k_stride)
    assert ctypes.sizeof(nm._NormDesc) == 8 + 6 * 8


def test_loop_takes_weights_wherever_they_start(lib):
    w = torch.arange(65, dtype=torch.bfloat16)
    loop = swab.DecodeLoop(2, 4, 2, 64, 16, device="cpu", norm=swab.NormDesc(), wq=w[1:], wk=w[:64])
    assert w[1:].data_ptr() % 16 and loop.wq.data_ptr() % 16 == loop.wk.data_ptr() % 16 == 0
    assert torch.equal(loop.wq, w[1:]) and torch.equal(loop.wk, w[:64])


def test_loop_refuses_what_its_calls_would(lib):
    for kw, error in ((dict(bits=8), ValueError), (dict(bits=4, head_dim=80), ValueError), (dict(bits=4, head_dim=288), swab.SwabError),
                      (dict(norm=swab.NormDesc(0.0)), swab.SwabError), (dict(wq=torch.ones(64)), ValueError),
                      (dict(norm=swab.NormDesc(), wq=torch.ones(64)), ValueError),
                      (dict(norm=swab.NormDesc(), wk=torch.ones(32, dtype=torch.bfloat16)), ValueError)):
        with pytest.raises(error):
            swab.DecodeLoop(**{**dict(batch=2, h=4, hk=2, head_dim=64, w=16, device="cpu"), **kw})
    loop = swab.DecodeLoop(2, 4, 2, 64, 16, device="cpu", bits=4, norm=swab.NormDesc(), wq=torch.ones(64, dtype=torch.bfloat16))
    assert loop.Kc.shape == (loop.cache.n_blocks, 2, 64, 32) and loop.Ks.shape[-1] == 2 and loop.Ks.dtype is torch.bfloat16
