"""Refusals of the serving entry points, checked on the host before any CUDA
call (the pointers are fake and never dereferenced), and the binding's checks."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

import sliding_window_attention_band_gb300 as swab
from oracle import serve as orc
from sliding_window_attention_band_gb300 import _binding as B
from sliding_window_attention_band_gb300 import build as swab_build
from sliding_window_attention_band_gb300 import serve

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA = 0, 1, 2, 3, 4
FAKE = 0x10000
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    swab_build.build()
    return B.load()


def rotary_desc(strides=None, **kw):
    base = dict(b=2, n=8, h=4, hk=2, head_dim=64, rot_dim=64, interleaved=0, dtype=1, scale=1.0, pos0=0)
    base.update(kw)
    zero = (0, 0, 0)
    s = dict(q=zero, k=zero, qo=zero, ko=zero, v=zero)
    s.update(strides or {})
    return serve._RotaryDesc(*(base[k] for k in ("b", "n", "h", "hk", "head_dim", "rot_dim", "interleaved", "dtype", "scale",
                                                 "pos0")), *(serve._S3(*s[k]) for k in ("q", "k", "qo", "ko", "v")))


def cache_desc(**kw):
    base = dict(batch=3, page=16, n_blocks=40, cols=8, ring=0, pinned=0)
    base.update(kw)
    return serve._CacheDesc(*(base[k] for k in ("batch", "page", "n_blocks", "cols", "ring", "pinned")))


def decode_desc(cache=None, **kw):
    base = dict(tokens=5, h=8, hk=2, head_dim=64, w=32, dilation=0, n_sink=0, max_q=2, max_len=128, prefix_len=0, dtype=1,
                q_row_stride=0, out_row_stride=0)
    base.update(kw)
    return serve._DecodeDesc(cache or cache_desc(), *(base[k] for k in (
        "tokens", "h", "hk", "head_dim", "w", "dilation", "n_sink", "max_q", "max_len", "prefix_len", "dtype", "q_row_stride",
        "out_row_stride")))


def rotary(lib, d, turns=FAKE, pos=FAKE, q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, fn="rotary"):
    return getattr(lib, fn)(ctypes.byref(d) if d is not None else None, turns, pos, q, k, qo, ko, None)


def append(lib, d, c, turns=FAKE, pos=FAKE, slots=FAKE, q=FAKE, k=FAKE, v=FAKE, qo=FAKE, kc=FAKE, vc=2 * FAKE):
    return lib.rotary_append(ctypes.byref(d), ctypes.byref(c) if c is not None else None, turns, pos, slots, q, k, v, qo, kc, vc,
                             None)


def slots(lib, c, tokens=10, pos0=0, lens=FAKE, new=2 * FAKE, table=FAKE, free=FAKE, n_free=5, used=FAKE, lens_out=FAKE,
          used_out=FAKE, start=3 * FAKE, sl=4 * FAKE, pos=5 * FAKE):
    return lib.cache_slots(ctypes.byref(c) if c is not None else None, tokens, pos0, lens, new, table, free, n_free, used,
                           lens_out, used_out, start, sl, pos, None)


def decode(lib, d, scale=0.125, q=FAKE, kc=FAKE, vc=FAKE, table=FAKE, lens=FAKE, start=FAKE, prefix=FAKE, o=FAKE, lse=None,
           ws=FAKE):
    return lib.band_decode(ctypes.byref(d) if d is not None else None, scale, q, kc, vc, table, lens, start, prefix, o, lse, ws,
                           None)


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="a valid call with fake pointers")


@pytest.mark.parametrize("fn", ["rotary", "rotary_bwd"])
@pytest.mark.parametrize("bad,want", [
    (dict(b=0), INVALID), (dict(n=0), INVALID), (dict(h=0), INVALID), (dict(hk=-1), INVALID), (dict(head_dim=0), INVALID),
    (dict(rot_dim=-2), INVALID), (dict(rot_dim=66), INVALID), (dict(rot_dim=31), INVALID), (dict(interleaved=2), INVALID),
    (dict(dtype=3), INVALID), (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID), (dict(pos0=-1), INVALID),
    (dict(head_dim=68), UNSUPPORTED), (dict(head_dim=1024), UNSUPPORTED), (dict(h=70000), UNSUPPORTED),
    (dict(b=1 << 16, n=1 << 16), UNSUPPORTED)])
def test_rotary_descriptor(lib, fn, bad, want):
    assert rotary(lib, rotary_desc(**bad), fn=fn) == want
    assert rotary(lib, None, fn=fn) == INVALID


def test_rotary_pointers_and_strides(lib):
    d = rotary_desc()
    for name in ("turns", "q", "k", "qo", "ko"):
        assert rotary(lib, d, **{name: None}) == INVALID
    for name in ("q", "k", "qo", "ko"):
        assert rotary(lib, d, **{name: FAKE + 8}) == MISALIGNED
    assert rotary(lib, d, turns=FAKE + 4) == MISALIGNED
    assert rotary(lib, d, pos=FAKE + 2) == MISALIGNED
    assert rotary(lib, rotary_desc({"q": (2048, -256, 64)})) == INVALID
    assert rotary(lib, rotary_desc({"k": (2048, 256, 68)})) == MISALIGNED
    assert rotary(lib, rotary_desc({"qo": (2048, 128, 64)})) == INVALID       # 4 heads of 64 in rows of 128
    assert rotary(lib, rotary_desc({"qo": (0, 256, 64)})) == INVALID          # both sequences in one place
    assert rotary(lib, rotary_desc({"ko": (1024, 64, 56)})) == INVALID
    assert rotary(lib, rotary_desc({"q": (1 << 36, 256, 64)})) == UNSUPPORTED  # over 64 GB
    assert rotary(lib, rotary_desc({"qo": (1 << 41, 256, 64)})) == UNSUPPORTED


@needs_no_gpu
def test_valid_rotary_calls_reach_the_launch(lib):
    assert rotary(lib, rotary_desc()) == CUDA
    assert rotary(lib, rotary_desc(), pos=None) == CUDA
    assert rotary(lib, rotary_desc(rot_dim=0), turns=None) == CUDA
    assert rotary(lib, rotary_desc(hk=0), k=None, ko=None) == CUDA
    assert rotary(lib, rotary_desc({"qo": (64, 128, 1024)}), fn="rotary_bwd") == CUDA   # head-major, interleaved sequences
    assert rotary(lib, rotary_desc({"q": (0, 256, 64)})) == CUDA              # one sequence read for both


@pytest.mark.parametrize("bad,want", [
    (dict(batch=0), INVALID), (dict(n_blocks=0), INVALID), (dict(cols=0), INVALID), (dict(ring=2), INVALID),
    (dict(pinned=1), INVALID), (dict(ring=1, pinned=8), INVALID), (dict(ring=1, pinned=-1), INVALID),
    (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(batch=70000), UNSUPPORTED),
    (dict(n_blocks=1 << 27, page=16), UNSUPPORTED)])
def test_cache_descriptor(lib, bad, want):
    c = cache_desc(**bad)
    assert slots(lib, c) == want
    assert append(lib, rotary_desc(), c) == want
    assert decode(lib, decode_desc(c)) == want
    assert lib.band_decode_workspace(ctypes.byref(decode_desc(c))) == 0


def test_cache_slots_arguments(lib):
    c = cache_desc()
    assert slots(lib, None) == INVALID
    for bad in (dict(tokens=-1), dict(pos0=-1), dict(n_free=-1)):
        assert slots(lib, c, **bad) == INVALID
    for name in ("lens", "new", "table", "free", "used", "lens_out", "used_out", "start", "sl", "pos"):
        assert slots(lib, c, **{name: None}) == INVALID, name
        assert slots(lib, c, **{name: 9 * FAKE + 2}) == MISALIGNED, name
    assert slots(lib, c, lens_out=2 * FAKE) == INVALID                        # lens_out over n_new
    assert slots(lib, c, sl=5 * FAKE) == INVALID
    assert slots(lib, c, start=FAKE) == INVALID


def test_cache_max_new(lib):
    c = cache_desc()
    c.max_new = -1
    assert slots(lib, c) == INVALID and append(lib, rotary_desc(), c) == INVALID and decode(lib, decode_desc(c)) == INVALID
    if not torch.cuda.is_available():
        c.max_new = 2 ** 31 - 1
        assert slots(lib, c) == CUDA


@needs_no_gpu
def test_valid_cache_calls_reach_the_launch(lib):
    assert slots(lib, cache_desc()) == CUDA
    assert slots(lib, cache_desc(ring=1, pinned=7), tokens=0, sl=None, pos=None, free=None, n_free=0) == CUDA
    assert append(lib, rotary_desc(), cache_desc()) == CUDA
    assert append(lib, rotary_desc(rot_dim=0), cache_desc(), turns=None, pos=None, q=None, qo=None) == CUDA


def test_append_arguments(lib):
    d, c = rotary_desc(), cache_desc()
    assert append(lib, d, None) == INVALID
    for name in ("turns", "pos", "slots", "q", "k", "v", "qo", "kc", "vc"):
        assert append(lib, d, c, **{name: None}) == INVALID, name
    for name in ("q", "k", "v", "qo", "kc", "vc"):
        assert append(lib, d, c, **{name: FAKE + 4}) == MISALIGNED, name
    assert append(lib, d, c, slots=FAKE + 1) == MISALIGNED
    assert append(lib, d, c, vc=FAKE) == INVALID                              # both caches in one place
    assert append(lib, rotary_desc(hk=0), c) == INVALID
    assert append(lib, rotary_desc({"v": (1024, 128, 60)}), c) == MISALIGNED
    assert append(lib, rotary_desc(hk=5000), cache_desc(n_blocks=1 << 20)) == UNSUPPORTED     # 2^32 lines and more
    assert decode(lib, decode_desc(cache_desc(n_blocks=1 << 26), h=512, hk=256)) == UNSUPPORTED


@pytest.mark.parametrize("bad,want", [
    (dict(tokens=0), INVALID), (dict(h=0), INVALID), (dict(hk=0), INVALID), (dict(hk=3), INVALID), (dict(head_dim=0), INVALID),
    (dict(max_q=0), INVALID), (dict(max_len=0), INVALID), (dict(w=-1), INVALID), (dict(w=(1 << 30) + 1), INVALID),
    (dict(dilation=-1), INVALID), (dict(n_sink=-1), INVALID), (dict(prefix_len=-1), INVALID), (dict(prefix_len=641), INVALID), (dict(dtype=9), INVALID),
    (dict(q_row_stride=64), INVALID), (dict(out_row_stride=-512), INVALID), (dict(head_dim=68), UNSUPPORTED),
    (dict(head_dim=264), UNSUPPORTED), (dict(dilation=16), UNSUPPORTED), (dict(h=258, hk=2), UNSUPPORTED),
    (dict(tokens=1 << 29), UNSUPPORTED), (dict(q_row_stride=1 << 37), UNSUPPORTED), (dict(q_row_stride=516), MISALIGNED), (dict(out_row_stride=516), MISALIGNED)])
def test_decode_descriptor(lib, bad, want):
    d = decode_desc(**bad)
    assert decode(lib, d) == want
    assert lib.band_decode_workspace(ctypes.byref(d)) == 0


def test_decode_ring_has_to_hold_the_window(lib):
    ring = cache_desc(ring=1, pinned=1)            # 7 recycled columns of 16: 97 positions reach back
    assert decode(lib, decode_desc(ring, w=96, max_q=2)) == INVALID
    assert decode(lib, decode_desc(ring, w=48, dilation=1, max_q=2)) == INVALID
    assert decode(lib, decode_desc(ring, w=32, n_sink=17)) == INVALID
    if not torch.cuda.is_available():
        assert decode(lib, decode_desc(ring, w=95, max_q=2, n_sink=16)) == CUDA


def test_decode_pointers(lib):
    d = decode_desc()
    assert decode(lib, None) == INVALID
    assert lib.band_decode_workspace(None) == 0
    for name in ("q", "kc", "vc", "table", "lens", "start", "o"):
        assert decode(lib, d, **{name: None}) == INVALID, name
        assert decode(lib, d, **{name: FAKE + 2}) == MISALIGNED, name
    assert decode(lib, decode_desc(prefix_len=3), prefix=None) == INVALID
    assert decode(lib, d, lse=FAKE + 4) == MISALIGNED
    assert decode(lib, d, scale=math.nan) == INVALID
    long = decode_desc(cache_desc(cols=4000, n_blocks=5000), w=1 << 30, max_len=64000)
    assert lib.band_decode_workspace(ctypes.byref(long)) > 0
    assert decode(lib, long, ws=None) == INVALID
    assert decode(lib, long, ws=FAKE + 8) == MISALIGNED


@needs_no_gpu
@pytest.mark.parametrize("kw", [dict(), dict(dtype=0), dict(dtype=2, head_dim=128, prefix_len=100), dict(head_dim=80),
                                dict(w=1 << 30, max_len=64000)])
def test_valid_decode_calls_reach_the_launch(lib, kw):
    assert decode(lib, decode_desc(cache_desc(cols=4000, n_blocks=5000), **kw)) == CUDA


def test_frequency_arguments(lib):
    def f(rot=8, base=1e4, scaling=0, factor=1.0, original=4096.0, low=1.0, high=32.0, turns=True, scale=True):
        t, s = torch.zeros(64, dtype=torch.int64), ctypes.c_float()
        return lib.rotary_frequencies(rot, base, scaling, factor, original, low, high, t.data_ptr() if turns else None,
                                      ctypes.byref(s) if scale else None)
    assert f() == OK and f(scaling=3, factor=4.0) == OK
    for bad in (dict(rot=0), dict(rot=7), dict(base=1.0), dict(base=math.inf), dict(base=math.nan), dict(factor=0.5),
                dict(factor=math.inf), dict(scaling=5), dict(scaling=-1), dict(scaling=3, original=0.0),
                dict(scaling=4, low=4.0, high=4.0), dict(scaling=3, low=0.0), dict(scaling=3, high=math.inf),
                dict(turns=False), dict(scale=False)):
        assert f(**bad) == INVALID, bad
    with pytest.raises(ValueError):
        swab.rotary_frequencies(8, scaling="other")
    with pytest.raises(B.SwabError):
        swab.rotary_frequencies(9)


@pytest.mark.parametrize("rot", [2, 20, 64, 128])
@pytest.mark.parametrize("scaling,factor,original", [("none", 1, 0), ("linear", 4, 0), ("ntk", 8, 0), ("yarn", 16, 8192),
                                                     ("bands", 8, 8192)])
def test_frequencies_match_the_oracle(lib, rot, scaling, factor, original):
    """Turns to 1e-13 relative: pow against exp(log), both within a few 2^-52 times the exponent's size (below 30)."""
    turns, scale = swab.rotary_frequencies(rot, 10000.0, scaling, factor, original)
    f, want = orc.frequencies(rot, 10000.0, scaling, factor, original, 1.0, 32.0 if scaling == "yarn" else 4.0)
    got = turns.numpy().astype(np.uint64).astype(np.float64) * 2.0 ** -64 * 2 * math.pi
    assert np.abs(got / f - 1).max() < 1e-13
    assert abs(scale - want) <= want * 2.0 ** -24


def test_binding_checks():
    """Shapes, types, places: refused before the library is called."""
    d = swab.RotaryDesc(1, 4, 2, 1, 64, 64)
    x = torch.zeros(4, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        swab.rotary(d, None, x, x)
    with pytest.raises(ValueError):
        swab.RotaryDesc(1, 4, 2, 1, 64, 64, dtype=torch.int32)
    c = swab.CacheDesc(1, 16, 2, 2)
    with pytest.raises(ValueError):
        swab.DecodeDesc(c, 1, 2, 1, 64, dtype=torch.int8)
    with pytest.raises(ValueError, match="CUDA"):
        z = torch.zeros(1, dtype=torch.int32)
        swab.cache_slots(c, z, z, z, z, z, z, z, z, z, z)
    with pytest.raises(ValueError, match="CUDA"):
        swab.band_decode(swab.DecodeDesc(c, 4, 2, 1, 64), 0.1, x, x, x, x, x, x, x)
    with pytest.raises(ValueError, match="both or neither"):
        swab.rotary_append(d, c, None, x, x, x, None, None, None, x, x)


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32, 2 ** 32 + 16, -2 ** 31 - 1, 2 ** 64 + 16])
def test_numbers_past_32_bits_are_refused_not_wrapped(big):
    """A window of 2^32 + 16 is no window of 16."""
    c = swab.CacheDesc(1, 16, 2, 2)
    for k in ("batch", "page", "n_blocks", "cols", "pinned", "max_new"):
        with pytest.raises(ValueError, match=k):
            swab.CacheDesc(**{**dict(batch=1, page=16, n_blocks=2, cols=2), k: big})
    for k in ("b", "n", "h", "hk", "head_dim", "rot_dim", "pos0"):
        with pytest.raises(ValueError, match=k):
            swab.RotaryDesc(**{**dict(b=1, n=4, h=2, hk=1, head_dim=64, rot_dim=64), k: big})
    for k in ("tokens", "h", "hk", "head_dim", "w", "dilation", "n_sink", "max_q", "max_len", "prefix_len"):
        with pytest.raises(ValueError, match=k):
            swab.DecodeDesc(c, **{**dict(tokens=1, h=2, hk=1, head_dim=64), k: big})
    for k in ("q_row_stride", "out_row_stride"):
        with pytest.raises(ValueError, match=k):
            swab.DecodeDesc(c, 1, 2, 1, 64, **{k: big << 33})
    with pytest.raises(ValueError, match="rot_dim"):
        swab.rotary_frequencies(big)
    names = ("lens", "n_new", "table", "free_list", "used", "lens_out", "used_out", "q_start", "slots", "pos")
    sizes = dict(table=2, used_out=2, q_start=2)
    with pytest.raises(ValueError, match="pos0"):
        swab.cache_slots(c, *[FakeInts(sizes.get(k, 1)) for k in names], pos0=big)
    for name in ("free_list", "slots"):
        with pytest.raises(ValueError, match=name):
            swab.cache_slots(c, *[FakeInts(2 ** 32 + 1 if k == name or (k, name) == ("pos", "slots") else sizes.get(k, 1))
                                  for k in names])


class FakeCuda:
    """Enough of a CUDA tensor for the binding's checks."""

    def __init__(self, shape, strides, dtype=torch.float16, device=0):
        self.shape, self._s, self.dtype, self._d, self.is_cuda, self.device = shape, strides, dtype, device, True, f"cuda:{device}"

    def get_device(self):
        return self._d

    def stride(self):
        return self._s

    def data_ptr(self):
        return FAKE


def test_an_odd_rot_dim_is_the_librarys_error_on_either_way(lib, monkeypatch):
    """The binding's own check of turns lets through what the compiled module lets through."""
    d = swab.RotaryDesc(1, 1, 2, 1, 64, 31)
    t = FakeInts(15)
    t.dtype = torch.int64
    assert serve._turns(d, t, 0) == FAKE
    t.shape = (16,)
    with pytest.raises(ValueError, match="turns"):
        serve._turns(d, t, 0)
    assert rotary(lib, d._plain) == INVALID


class FakeInts(FakeCuda):
    def __init__(self, n):
        super().__init__((n,), (1,), torch.int32)

    def numel(self):
        return self.shape[0]

    def is_contiguous(self):
        return True


def test_binding_rows_and_strides():
    d = swab.RotaryDesc(2, 3, 4, 2, 64, 64)
    strides = lambda st: serve._row_strides("Q", st, d, 4)  # noqa: E731
    assert strides((768, 256, 64, 1)) == (768, 256, 64)
    assert strides((512, 64, 1)) == (1536, 512, 64)
    assert strides((0, 256, 64, 1)) == (0, 256, 64)
    for bad in ((768, 256, 64, 2), (0, 0, 0, 1)):
        with pytest.raises(ValueError):
            strides(bad)
    one = swab.RotaryDesc(1, 1, 1, 0, 64, 64)
    assert serve._row_strides("Q", (7, 9, 3, 1), one, 1) == (0, 0, 0)
    rows = lambda t: serve._rows("Q", t, d, d._q, 0)  # noqa: E731
    assert rows(FakeCuda((2, 3, 4, 64), (768, 256, 64, 1))) == FAKE
    assert rows(FakeCuda((6, 4, 64), (256, 64, 1))) == FAKE
    for bad in (FakeCuda((2, 3, 5, 64), (960, 320, 64, 1)), FakeCuda((6, 4, 64), (256, 64, 1), torch.bfloat16)):
        with pytest.raises(ValueError):
            rows(bad)
    with pytest.raises(ValueError, match="other tensors"):
        rows(FakeCuda((6, 4, 64), (256, 64, 1), device=1))


def test_decode_loop_refuses_a_prompt_before_its_lengths_move(lib, monkeypatch):
    loop = swab.DecodeLoop(2, 4, 2, 64, w=16, page=16, dtype=torch.float16, device="cpu")
    called = []
    monkeypatch.setattr(loop, "_place", lambda *a: called.append(a))
    n_new = torch.tensor([3, 2], dtype=torch.int32)
    wide = torch.zeros(5, 8, 72, dtype=torch.float16)
    for qkv in (torch.zeros(5, 8, 64), torch.zeros(5, 7, 64, dtype=torch.float16), torch.zeros(0, 8, 64, dtype=torch.float16),
                torch.zeros(5, 8, 64, dtype=torch.float16, device="meta"), torch.zeros(5, 512, dtype=torch.float16),
                torch.zeros(5, 64, 8, dtype=torch.float16).transpose(1, 2), wide[:, :, 1:65],
                torch.zeros(5, 8, 68, dtype=torch.float16)[:, :, :64]):
        with pytest.raises(ValueError):
            loop.fill(qkv, n_new)
    assert not called
    with pytest.raises(ValueError, match="CUDA"):     # heads side by side in a wider row: right but for the device
        loop.fill(wide[:, :, :64], n_new)
    assert len(called) == 1


@pytest.mark.parametrize("bad", [
    dict(head_dim=68), dict(head_dim=264), dict(h=3), dict(h=256, hk=1), dict(dilation=16), dict(dilation=-1), dict(page=48),
    dict(max_new=0), dict(w=-1), dict(w=(1 << 30) + 1), dict(n_sink=-1), dict(batch=0), dict(batch=70000), dict(hk=0), dict(rot_dim=31),
    dict(rot_dim=66), dict(rot_dim=-2), dict(turns=torch.zeros(31, dtype=torch.int64)),
    dict(turns=torch.zeros(32)), dict(dtype=torch.int8)])
def test_decode_loop_refuses_when_it_is_made_what_its_calls_would(lib, bad):
    """Not at its first step, when the lengths have moved on."""
    with pytest.raises((ValueError, B.SwabError)):
        swab.DecodeLoop(**{**dict(batch=2, h=4, hk=2, head_dim=64, w=16, page=16, dtype=torch.float16, device="cpu"), **bad})


def test_decode_loop_keeps_the_rotary_scale_it_is_given(lib):
    make = lambda **kw: swab.DecodeLoop(2, 4, 2, 64, w=16, page=16, dtype=torch.float16, device="cpu", **kw)  # noqa: E731
    turns, scale = swab.rotary_frequencies(64, scaling="yarn", factor=4.0, original=4096)
    for loop, want in ((make(), 1.0), (make(rotary_scale=1.25), 1.25), (make(turns=turns, rotary_scale=scale), scale)):
        assert loop.rotary_scale == want and loop._rotary.scale == want and abs(loop._rotary._plain.scale - want) < 1e-7
    assert torch.equal(make(turns=turns).turns, turns) and not torch.equal(make().turns, turns)
    with pytest.raises(B.SwabError):
        make(rotary_scale=math.inf)


def test_decode_loop_of_a_workload_takes_leading_global_tokens_only(lib):
    wl = lambda idx: swab.Workload(9, "w", 2, 2, 64, 64, 8, 8, 0, torch.float16, idx)  # noqa: E731
    for idx, sinks in (((), 0), ((0,), 1), ((0, 1, 2), 3), ((2, 0, 1), 3)):
        assert swab.DecodeLoop.from_workload(wl(idx), device="cpu")._decode.n_sink == sinks
    for idx in ((1,), (0, 2), (0, 1, 63), (5, 6)):
        with pytest.raises(ValueError, match="leading"):
            swab.DecodeLoop.from_workload(wl(idx), device="cpu")


def test_decode_loop_refuses_prompts_longer_than_their_rows(lib, monkeypatch):
    """n_new may not add up to more than the rows of qkv (their positions would never be written); fewer is padding."""
    loop = swab.DecodeLoop(3, 4, 2, 64, w=16, page=16, dtype=torch.float16, device="cpu")
    called = []
    monkeypatch.setattr(loop, "_place", lambda *a: called.append(a))
    qkv = torch.zeros(5, 8, 64, dtype=torch.float16)
    for n_new in ([3, 2, 1], [6, 0, 0], [6, -2, 0], [2 ** 31 - 1, 2 ** 31 - 1, 4]):
        with pytest.raises(ValueError, match="n_new"):
            loop.fill(qkv, torch.tensor(n_new, dtype=torch.int32))
    assert not called
    for n_new in ([3, 2, 0], [1, -7, 2], [5, -1, 0]):
        with pytest.raises(ValueError, match="CUDA"):          # right but for the device
            loop.fill(qkv, torch.tensor(n_new, dtype=torch.int32))
    assert len(called) == 3


def test_decode_loop_restart_takes_each_row_once_and_no_other(lib):
    """A row outside the batch (a negative one too) is refused with nothing changed; one named twice is emptied once."""
    loop = swab.DecodeLoop(2, 4, 2, 64, w=16, page=16, dtype=torch.float16, device="cpu")
    loop.table[:] = torch.arange(loop.cache.n_blocks, dtype=torch.int32).view(2, -1)
    loop.lens[:], loop.used[0] = 40, loop.cache.n_blocks
    held = lambda: [t.clone() for t in (loop.table, loop.lens, loop.used, loop.free_list)]  # noqa: E731
    before = held()
    for bad in ([2], [-1], [0, 2], [-1, 1], [1.5], ["1"], [None]):
        with pytest.raises((ValueError, TypeError)):
            loop.restart(bad)
        assert all(torch.equal(a, b) for a, b in zip(before, held()))
    loop.restart([])
    assert int(loop.used[0]) == loop.cache.n_blocks and torch.equal(loop.table, before[0])
    for one in ([1, 1], [np.int64(1), 1], torch.tensor([1, 1])):
        loop.table[1], loop.lens[1], loop.used[0] = before[0][1], 40, loop.cache.n_blocks
        loop.restart(one)
        assert sorted(loop.free_list[int(loop.used[0]):].tolist()) == before[0][1].tolist()
        assert loop.table[0].tolist() == before[0][0].tolist() and loop.table[1].tolist() == [-1] * loop.cache.cols
        assert loop.lens.tolist() == [40, 0]


def test_compiled_calls_leave_what_is_unusual_to_the_binding(lib):
    """Anything but the expected tensors gives -1 and no exception; the binding then names what is wrong."""
    call = serve._calls or serve._load_calls()
    assert call is not serve._NoCalls
    c = swab.CacheDesc(2, 16, 8, 4)
    r = swab.RotaryDesc(1, 2, 4, 2, 64, 64)
    d = swab.DecodeDesc(c, 2, 4, 2, 64)
    f16, i32 = torch.zeros(2, 4, 64, dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    kv = torch.zeros(8, 2, 16, 64, dtype=torch.float16)
    odd = [None, 3, -1, "x", 1.5, f16, i32, kv, kv.to("meta"), f16.to_sparse(), torch.nn.Parameter(f16), object()]
    rng = np.random.default_rng(0)
    for name, lead, n in (("rotary", (r._addr,), 7), ("rotary_bwd", (r._addr,), 7), ("cache_slots", (c._addr, 0), 12),
                          ("rotary_append", (r._addr, c._addr), 11), ("band_decode", (d._addr, 0, 0.125), 13)):
        fn = getattr(call, name)
        assert fn() == -1 and fn(*lead) == -1 and fn(0, *[None] * (n - 1)) == -1
        for _ in range(60):
            assert fn(*lead, *(odd[k] for k in rng.integers(0, len(odd), n - len(lead)))) == -1
        assert fn("descriptor", *[f16] * (n - 1)) == -1
    for scale in ("x", None, torch.zeros(())):
        assert call.band_decode(d._addr, 0, scale, *[f16] * 10) == -1
    with pytest.raises(TypeError):
        call.bind(1, 2)
    with pytest.raises(ValueError):
        call.bind(0, 0, 0, 0, 0)
    with pytest.raises(ValueError, match="CUDA"):
        swab.rotary(r, torch.zeros(32, dtype=torch.int64), f16, f16, f16[:, :2], f16[:, :2])


def test_library_is_built_and_called_without_the_compiled_calls(lib, monkeypatch, tmp_path):
    """A compiler that cannot make the module, or a module that does not load: a warning, and the calls go through Python."""
    linked = []
    monkeypatch.setattr(swab_build, "CALLS", str(tmp_path / "_serve_call.so"))
    (tmp_path / "_serve_call.so").write_bytes(b"of another machine")
    monkeypatch.setattr(serve, "_calls", None)
    with pytest.warns(UserWarning, match="compiled"):
        assert serve._load_calls() is serve._NoCalls
    with pytest.raises(ValueError, match="CUDA"):
        z = torch.zeros(1, dtype=torch.int32)
        swab.cache_slots(swab.CacheDesc(1, 16, 2, 2), z, z, z, z, z, z, z, z, z, z)

    def no_compiler():
        raise RuntimeError("g++ failed")
    monkeypatch.setattr(swab_build, "_build_calls", no_compiler)
    monkeypatch.setattr(swab_build, "calls_up_to_date", lambda: False)
    monkeypatch.setattr(swab_build, "up_to_date", lambda v: False)
    monkeypatch.setattr(swab_build, "_compile_jobs", lambda *a: [("x.cu", lambda src: "x.o")])
    monkeypatch.setattr(swab_build, "_link", lambda v, objs: linked.append((v, objs)))
    with pytest.warns(UserWarning, match="compiled"):
        assert swab_build.build_variants(("regular",)) == [swab_build.LIB]
    assert linked == [("regular", ["x.o"])]
    assert not (tmp_path / "_serve_call.so").exists()          # one of older sources must not be loaded


def test_descriptors_of_the_compiled_calls_follow_the_header(lib):
    """The C structs the compiled calls read by address are those the binding passes by reference."""
    r = swab.RotaryDesc(2, 3, 4, 2, 64, 32, interleaved=True, scale=1.25, pos0=7, dtype=torch.bfloat16)
    a = serve._RotaryDesc.from_address(r._addr)
    assert [getattr(a, k) for k in ("b", "n", "h", "hk", "head_dim", "rot_dim", "interleaved", "dtype", "scale", "pos0")] == [
        2, 3, 4, 2, 64, 32, 1, 2, 1.25, 7]
    assert not any(x for k in ("q", "k", "qo", "ko", "v") for x in getattr(a, k + "_stride"))
    c = swab.CacheDesc(2, 16, 8, 4, ring=True, pinned=1)
    d = swab.DecodeDesc(c, 5, 4, 2, 64, w=3, q_row_stride=512)
    assert ctypes.addressof(d.c) == d._addr and ctypes.addressof(c.c) == c._addr
    assert d.c.q_row_stride == 512 and d.c.cache.cols == 4 and d.c.cache.pinned == 1
