"""The cache in 4 bits -- the write with norms and rotary positions, rows read back,
decode over it -- against the fp64 oracle, on the GPU.

Codes and scales of values that are not computed (V; K without norm and rotary
positions) have to be the oracle's, bit for bit.  A computed K is quantised from its
value in the tensors' type, which norm_rotary_append writes by the same arithmetic:
its codes have to be the oracle's codes of that.  Decode is held to the bounds of
tests/test_gpu_serve.py (same arithmetic over exact values): its docstring derives
them.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import sliding_window_attention_band_gb300 as swab
from oracle import quant
from oracle import serve as orc
from test_gpu_serve import (BF16, F16, F32, INVALID_BIT, LENGTHS, ROOT, Decode, check_some, f64, frequencies, i32, randn, same_bits)

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("device_status_guard")]
NAMES = {F16: "f16", BF16: "bf16", F32: "f32"}


def cells(x, dtype):
    """(codes uint8, scales) on the GPU of rows x [..., hd] by the oracle."""
    codes, scales = quant.quantise(f64(x), NAMES[dtype])
    return torch.tensor(quant.pack(codes)).cuda(), torch.tensor(scales).to(dtype).cuda()


def empty_cells(cache, hk, hd, dtype, fill=0xa5):
    codes, scales = swab.cache4_shapes(cache, hk, hd)
    c = [torch.full(codes, fill, dtype=torch.uint8, device="cuda") for _ in range(2)]
    s = [torch.full(scales, 0.25, dtype=dtype, device="cuda") for _ in range(2)]
    return c[0], s[0], c[1], s[1]


# ---------------------------------------------------------------------------
# the write
# ---------------------------------------------------------------------------
APPEND = [  # h, hk, hd, rot, interleaved, page
    (4, 2, 64, 64, False, 16), (4, 2, 64, 32, True, 64), (4, 2, 64, 32, False, 64), (3, 1, 128, 128, False, 32), (3, 3, 128, 64, False, 16),
    (2, 2, 128, 128, True, 128), (6, 2, 96, 96, False, 32), (2, 1, 96, 48, True, 16), (2, 2, 32, 32, False, 16), (1, 1, 256, 256, False, 16),
    (2, 1, 64, 0, False, 16), (2, 2, 160, 64, False, 16), (40, 8, 128, 128, False, 64), (2, 2, 128, 32, False, 16), (6, 3, 96, 0, False, 16),
    (3, 1, 96, 48, False, 32), (3, 2, 96, 96, True, 16), (2, 1, 64, 16, False, 16)]


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("case", APPEND)
def test_append4_writes_the_oracles_codes(case, normed, dtype):
    h, hk, hd, rot, inter, page = case
    T, blocks = 37, 6
    turns, freq, scale = frequencies(rot, "none")
    q, k, v = randn((T, h + 2 * hk, hd), dtype, 1).split([h, hk, hk], dim=1)
    v[3, 0, :32] = 0.0                                            # a group of zeros
    v[4, 0, 5], v[4, 0, 6] = 3.0, -3.0                            # two of a magnitude
    v[5] = v[5] * 1e-3
    w = [randn((hd,), dtype, 2 + s) for s in range(2)] if normed else [None, None]
    nd = swab.NormDesc(1e-5, 0.5) if normed else None
    pos = np.random.default_rng(4).integers(0, 9000, T)
    slots = np.random.default_rng(5).permutation(blocks * page)[:T]
    slots[[2, 11]] = -1
    d, cache = swab.RotaryDesc(1, T, h, hk, hd, rot, inter, dtype=dtype), swab.CacheDesc(1, page, blocks, blocks)
    kc, vc = (torch.zeros(blocks, hk, page, hd, dtype=dtype, device="cuda") for _ in range(2))
    want_q, qo = (torch.empty(T, h, hd, dtype=dtype, device="cuda") for _ in range(2))
    if normed:
        swab.norm_rotary_append(d, nd, cache, turns, q, k, v, i32(pos), i32(slots), want_q, kc, vc, *w)
    else:
        swab.rotary_append(d, cache, turns, q, k, v, i32(pos), i32(slots), want_q, kc, vc)
    got = empty_cells(cache, hk, hd, dtype)
    before = [x.clone() for x in got]
    swab.rotary_append4(d, cache, turns, q, k, v, i32(pos), i32(slots), qo, *got, nd, *w)
    same_bits(qo, want_q)
    live = np.flatnonzero(slots >= 0)
    blk, off = torch.tensor(slots[live] // page).cuda(), torch.tensor(slots[live] % page).cuda()
    want = [*cells(kc[blk, :, off], dtype), *cells(v[live], dtype)]
    for now, then, ref in zip(got, before, want):
        same_bits(now[blk, :, off], ref)
        then[blk, :, off] = ref
        same_bits(now, then)                                      # the other rows stay
    # rows read back: what the codes stand for, other rows left alone
    ko, vo = (torch.full((T, hk, hd), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    swab.cache_read4(cache, i32(slots), *got, ko, vo)
    for x, c, s in ((ko, *want[:2]), (vo, *want[2:])):
        ref = quant.values(quant.unpack(c.cpu().numpy()), f64(s))
        assert np.array_equal(f64(x)[live], ref)
        assert (x[[2, 11]] == 7.0).all()
    # no queries: the same cells
    again = empty_cells(cache, hk, hd, dtype)
    swab.rotary_append4(d, cache, turns, None, k, v, i32(pos), i32(slots), None, *again, nd, None, w[1])
    for a, b in zip(got, again):
        same_bits(a, b)
    # slots outside the cache are flagged, not written and not read
    slots[7], slots[9] = blocks * page, -2
    swab.rotary_append4(d, cache, turns, q, k, v, i32(pos), i32(slots), qo, *again, nd, *w)
    assert swab.device_status(reset=True) == INVALID_BIT
    for a, b in zip(got, again):
        same_bits(a, b)
    ko.fill_(5.0)
    swab.cache_read4(cache, i32(slots), *again, ko, vo)
    assert swab.device_status(reset=True) == INVALID_BIT and (ko[[2, 7, 9, 11]] == 5.0).all()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("hd", [64, 96])
def test_groups_at_the_ends_of_the_format(hd, dtype):
    """Every tie, the smallest and largest values, zeros, NaN and infinities: the oracle's cells."""
    page, blocks = 16, 40
    rng = np.random.default_rng(6)
    tiny = 2.0 ** -24 if dtype is F16 else 2.0 ** -126
    top = float(torch.finfo(dtype).max)
    rows = [np.zeros(32), np.full(32, tiny), np.full(32, -tiny), np.full(32, top), np.full(32, -top)]
    for k in range(1, 40):
        rows.append(rng.integers(-k, k + 1, 32) * tiny)                          # a few steps of the smallest
        rows.append(np.where(rng.random(32) < 0.2, top, rng.standard_normal(32)))
        s = float(2.0 ** rng.integers(-10, 8)) * rng.integers(16, 32)            # s a scale: x / s on every tie
        rows.append(np.append(rng.permutation(np.arange(-15, 16)) / 2.0, 8.0) * s * rng.choice([-1, 1]))
        rows.append(rng.standard_normal(32) * 10.0 ** rng.uniform(-6, 4))
    for bad in (np.nan, np.inf, -np.inf):
        rows.append(np.where(np.arange(32) == 17, bad, 1.0))
    while len(rows) % (hd // 32):
        rows.append(np.ones(32))
    x = torch.tensor(np.array(rows)).to(dtype).view(-1, 1, hd).cuda()
    T = len(x)
    assert T <= page * blocks
    d, cache = swab.RotaryDesc(1, T, 1, 1, hd, 0, dtype=dtype), swab.CacheDesc(1, page, blocks, blocks)
    got = empty_cells(cache, 1, hd, dtype)
    swab.rotary_append4(d, cache, None, None, x, x, None, i32(np.arange(T)), None, *got)
    codes, scales = cells(x, dtype)
    for c, s in (got[:2], got[2:]):
        c, s = c.view(blocks * page, 1, -1)[:T], s.view(blocks * page, 1, -1)[:T]
        assert torch.equal(c, codes)
        assert torch.equal(s.isnan(), scales.isnan()) and torch.equal(s.nan_to_num(), scales.nan_to_num())
    ko, vo = torch.zeros_like(x), torch.zeros_like(x)
    swab.cache_read4(cache, i32(np.arange(T)), *got, ko, vo)
    ref = quant.values(quant.unpack(codes.cpu().numpy()), f64(scales))
    assert np.array_equal(f64(ko), ref, equal_nan=True) and np.array_equal(f64(vo), ref, equal_nan=True)


def test_many_tokens_and_heads():
    """More rows than the grid holds at once, more heads than a block lists."""
    for T, h, hk, hd, dtype in ((3000, 8, 2, 128, BF16), (5, 600, 300, 64, F16), (2000, 1, 1, 64, F16)):
        turns, freq, scale = frequencies(hd, "none")
        page, blocks = 64, -(-T // 64) + 1
        q, k, v = randn((T, h + 2 * hk, hd), dtype, 11).split([h, hk, hk], dim=1)
        d, cache = swab.RotaryDesc(1, T, h, hk, hd, hd, dtype=dtype), swab.CacheDesc(1, page, blocks, blocks)
        kc, vc = (torch.zeros(blocks, hk, page, hd, dtype=dtype, device="cuda") for _ in range(2))
        qo, q2 = (torch.empty(T, h, hd, dtype=dtype, device="cuda") for _ in range(2))
        at, pos = i32(np.random.default_rng(7).permutation(blocks * page)[:T]), i32(np.arange(T))
        swab.rotary_append(d, cache, turns, q, k, v, pos, at, qo, kc, vc)
        got = empty_cells(cache, hk, hd, dtype)
        swab.rotary_append4(d, cache, turns, q, k, v, pos, at, q2, *got)
        same_bits(qo, q2)
        some = torch.tensor(np.random.default_rng(8).choice(T, min(T, 40), replace=False)).cuda()
        blk, off = at[some].long() // page, at[some].long() % page
        for (c, s), x in ((got[:2], kc[blk, :, off]), (got[2:], v[some])):
            codes, scales = cells(x, dtype)
            same_bits(c[blk, :, off], codes)
            same_bits(s[blk, :, off], scales)


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
class Decode4(Decode):
    """Decode over the same cache in 4 bits: what is not attended to has NaN scales and any codes."""

    def __init__(self, dtype, *args, **kw):
        super().__init__(dtype, *args, **kw)
        self.quantise()

    def quantise(self):
        shape = self.kc.shape
        g = torch.Generator().manual_seed(5)
        self.cells = []
        for name in ("kc", "vc"):
            x = getattr(self, name)
            rows = x.reshape(-1, shape[-1])
            there = ~rows.isnan().any(1)
            codes = torch.randint(0, 256, (len(rows), shape[-1] // 2), generator=g, dtype=torch.uint8).cuda()
            scales = torch.full((len(rows), shape[-1] // 32), float("nan"), dtype=self.dtype, device="cuda")
            if there.any():
                codes[there], scales[there] = cells(rows[there], self.dtype)
            values = quant.values(quant.unpack(codes.cpu().numpy()), f64(scales))
            self.cells += [codes.view(*shape[:-1], -1), scales.view(*shape[:-1], -1)]
            setattr(self, name, torch.tensor(values).view(shape).to(self.dtype).cuda())

    def run(self, stream=None, lse=True):
        o = torch.full_like(self.q, 7.0)
        l = torch.full(self.q.shape[:2], 7.0, dtype=F32, device="cuda") if lse else None
        ws = torch.empty(swab.band_decode4_workspace(self.desc) + 16, dtype=torch.uint8, device="cuda")[16:]
        ints = i32(self.table), i32(self.lens), i32(self.q_start)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
            self.held = ws, *ints                # in use behind this call: not for the next tensor made here
        swab.band_decode4(self.desc, self.scale, self.q, *self.cells, *ints, o, l, ws, stream=stream)
        return o, l


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("heads", [(4, 4, 64), (8, 2, 128), (6, 1, 64), (5, 5, 96), (2, 2, 256), (3, 1, 128), (16, 1, 128), (12, 1, 64), (2, 1, 32)])
def test_decode_matches_the_oracle(heads, dtype):
    for k, (lens, new) in enumerate(LENGTHS):
        Decode4(dtype, lens, new, *heads, seed=30 + k, pad=k % 3).check()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("case", [
    dict(w=0), dict(w=7), dict(w=16, n_sink=3), dict(w=31, n_sink=16, page=32), dict(w=5, dilation=1), dict(w=70),
    dict(w=9, dilation=3, n_sink=5), dict(w=20, ring=True), dict(w=20, ring=True, n_sink=20, page=16),
    dict(w=6, dilation=2, ring=True, n_sink=1), dict(w=100, n_sink=90), dict(w=3, n_sink=400), dict(w=40, dilation=15)])
def test_decode_windows_and_sinks(case, dtype):
    for heads in ((4, 2, 64), (2, 1, 128), (12, 1, 64)):
        for k, (lens, new) in enumerate(LENGTHS[1:]):
            Decode4(dtype, lens, new, *heads, seed=50 + k, **case).check()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("case", [
    dict(lens=[5000], new=[1], h=4, hk=1, hd=128, page=64), dict(lens=[3000, 17, 4100], new=[1, 1, 1], h=4, hk=2, hd=64, page=128),
    dict(lens=[2500, 900], new=[4, 7], h=16, hk=2, hd=128, page=32), dict(lens=[1500], new=[1], h=128, hk=1, hd=64, page=16),
    dict(lens=[2600, 2601], new=[1, 2], h=4, hk=4, hd=64, w=2048, page=64, ring=True), dict(lens=[700], new=[40], h=2, hk=1, hd=64),
    dict(lens=[900, 1200], new=[3, 2], h=24, hk=2, hd=128, w=100, dilation=3), dict(lens=[2000, 130], new=[1, 1], h=3, hk=1, hd=96),
    dict(lens=[3000], new=[2], h=4, hk=4, hd=128, w=2500, n_sink=7, page=64)])
def test_decode_long_and_wide(case, dtype):
    Decode4(dtype, seed=90, **case).check()


@pytest.mark.parametrize("dtype,hd", [(F16, 64), (BF16, 128), (F16, 128), (BF16, 64), (F32, 64)])
@pytest.mark.parametrize("case", [dict(n=60, keys=600, h=16, hk=8), dict(n=100, keys=500, h=8, hk=8), dict(n=32, keys=2600, h=8, hk=8),
                                  dict(n=45, keys=2600, h=8, hk=4, m=2), dict(n=20, keys=900, h=12, hk=1, m=2), dict(n=130, keys=400, h=8, hk=8)])
def test_decode_of_many_requests(case, dtype, hd):
    n, keys, m = case["n"], case["keys"], case.get("m", 1)
    rng = np.random.default_rng(113)
    lens, new = rng.integers(m, keys + 1, n), rng.integers(0, m + 1, n)
    lens[rng.random(n) < 0.8] //= 16                                 # (few of the long ones: the oracle quantises them)
    lens = np.maximum(lens, m)
    lens[n // 2], new[n // 2], new[0], new[n - 1] = keys, m, m, 1
    c = Decode4(dtype, lens.tolist(), new.tolist(), case["h"], case["hk"], hd, page=64, pad=2, seed=114)
    o, lse = c.run()
    assert (o[int(c.q_start[-1]):] == 7.0).all() and not o.isnan().any()
    check_some(c, o, lse, sorted({0, 1, n // 3, n // 2, n - 2, n - 1}))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("case", [
    dict(lens=[700, 33, 1, 260], new=[1, 1, 1, 1], h=4, hk=2), dict(lens=[500, 90, 64], new=[4, 0, 3], h=12, hk=3),
    dict(lens=[1500], new=[2], h=40, hk=2, page=64), dict(lens=[400, 17], new=[2, 1], h=6, hk=2, w=50, n_sink=19),
    dict(lens=[300, 120], new=[2, 2], h=8, hk=2, w=40, ring=True, n_sink=16), dict(lens=[300, 80], new=[3, 1], h=4, hk=2, w=30, dilation=2)])
def test_decode_with_three_groups_a_head(case, dtype):
    Decode4(dtype, hd=96, seed=116, pad=1, **case).check()


@pytest.mark.parametrize("heads,m", [((4, 1, 64), 1), ((8, 1, 128), 2)])
def test_decode_of_requests_of_very_different_lengths(heads, m):
    """More lists than the GPU holds at once, a few of them long: several pieces a list, empty for the others."""
    lens = [10300, 2, 5121, 5120] + [2 + 7 * r % 40 for r in range(396)]
    new = [m if r % 3 else 1 for r in range(400)]
    c = Decode4(BF16, lens, new, *heads, page=64, pad=2, seed=115)
    o, lse = c.run()
    assert (o[int(c.q_start[-1]):] == 7.0).all() and not o.isnan().any()
    check_some(c, o, lse, [0, 1, 2, 3, 4, 200, 399])


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_decode_scores_scales_and_announced_lengths(dtype):
    Decode4(dtype, [200, 31], [1, 2], 4, 2, 64, qscale=40.0, seed=97).check()
    for max_len in (1, 300):                                         # max_len divides the work only
        Decode4(dtype, [900, 40], [1, 1], 4, 2, 64, max_len=max_len, seed=95).check()
    for scale in (-0.3, 0.0, 1e-8):
        c = Decode4(dtype, [90, 5], [1, 1], 4, 2, 64, seed=98)
        c.scale = scale
        c.check()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 2, 128)])
def test_decode_with_scores_that_keep_growing(heads, dtype):
    """The reference is raised again and again, and what was summed so far scaled."""
    c = Decode(dtype, [700, 300], [1, 2], *heads, page=64, qscale=2.0, seed=108)
    for r in range(2):
        for j in range(c.lens[r]):
            b = int(c.table[r][j // 64])
            c.kc[b, :, j % 64] *= 1.0 + j / 40.0
    c.__class__ = Decode4
    c.quantise()
    c.check()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("hd", [64, 96, 128])
def test_decode_with_blocks_that_are_not_there(hd, dtype):
    """Absent columns, blocks outside the cache (flagged), empty requests, lengths past the table: no key, no fault."""
    c = Decode4(dtype, [64, 33, 16, 50], [2, 1, 1, 1], 4, 2, hd, seed=120)
    o, lse = c.run()
    c.table[1, :] = -1                                               # nothing left of request 1
    c.table[0, 1] = -1                                               # a hole in request 0
    o, lse = c.run()
    c.check(o, lse)
    assert (o[2] == 0).all() and torch.isneginf(lse[2]).all()
    assert swab.device_status(reset=True) == 0
    c.table[3, 0], c.table[2, 0] = c.cells[0].shape[0], -7
    o, lse = c.run()
    assert swab.device_status(reset=True) == INVALID_BIT
    c.check(o, lse)
    assert (o[3] == 0).all() and torch.isneginf(lse[3]).all()
    # longer than the table: flagged, the keys past it absent
    c = Decode4(dtype, [40, 20], [1, 1], 4, 2, hd, seed=121)
    c.lens[0] = c.table.shape[1] * 16 + 30
    o, lse = c.run()
    assert swab.device_status(reset=True) == INVALID_BIT
    for lens, start in (([0, 0], [0, 1, 2]), ([-5, 2 ** 31 - 1], [0, 1, 2]), ([40, 20], [2, 1, 0]), ([40, 20], [-2 ** 31, 2 ** 31 - 1, 0]),
                        ([40, 20], [5, 9, 2 ** 31 - 1])):
        c.lens, c.q_start = lens, np.array(start)
        c.run()
        torch.cuda.synchronize()
    swab.device_status(reset=True)


@pytest.mark.parametrize("hd,dtype", [(64, F16), (96, BF16), (128, F16), (128, BF16)])
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("case", [dict(), dict(w=150), dict(w=130, n_sink=20), dict(w=90, n_sink=33, dilation=1)])
def test_decode_with_present_keys_behind_absent_ones(case, page, hd, dtype):
    """Tiles of 16 rows, and of 8 with a tail behind them.  Request r has holes where the bits of r are set in four
    adjacent columns: every choice of the four halves of a group of 64 keys where page is 16 and lists start at 0, else
    holes anywhere in a group, as windows and sinks start lists off multiples of 64."""
    lens = [200 + 13 * r for r in range(16)]
    for h, hk, m in ((16, 1, 1), (8, 2, 4), (12, 2, 3), (4, 2, 2)):
        c = Decode4(dtype, lens, [m] * 16, h, hk, hd, page=page, pad=1, seed=122, **case)
        for r in range(16):
            first = (lens[r] - 120 if "w" in case else 64) // page
            for k in range(4):
                if r >> k & 1 and first + k < c.table.shape[1]:
                    c.table[r, first + k] = -1
        o, lse = c.run()
        c.check(o, lse)
        assert swab.device_status(reset=True) == 0
        outside = np.where(np.arange(c.table.shape[1]) % 2 == 0, c.cells[0].shape[0] + 3, -2)
        for r in range(16):                                          # ids outside the cache: the same keys, flagged
            holes = (c.table[r] == -1) & (np.arange(c.table.shape[1]) < lens[r] // page)
            c.table[r, holes] = outside[holes]
        again = c.run()
        assert swab.device_status(reset=True) == INVALID_BIT
        same_bits(again[0], o)
        same_bits(again[1], lse)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_not_finite_show(dtype, bad):
    """A group with a NaN or infinity has a NaN scale: attended to, its request's heads are NaN; the other requests' are not."""
    page, hd, hk, h = 16, 64, 2, 4
    lens = [40, 40]
    cache, d = swab.CacheDesc(2, page, 6, 3), swab.RotaryDesc(1, 80, h, hk, hd, 0, dtype=dtype)
    x = randn((80, h + 2 * hk, hd), dtype, 130)
    q, k, v = x.split([h, hk, hk], dim=1)
    k[60, 0, 7] = bad                                                # request 1, key head 0
    v[10, 1, 40] = bad                                               # request 0, key head 1, channels 32..63
    table = i32([[0, 1, 2], [3, 4, 5]])
    slots = i32([r * 48 + j for r in range(2) for j in range(40)])
    got = empty_cells(cache, hk, hd, dtype)
    swab.rotary_append4(d, cache, None, None, k, v, None, slots, None, *got)
    dec = swab.DecodeDesc(cache, 2, h, hk, hd, max_len=48, dtype=dtype)
    o, lse = torch.zeros(2, h, hd, dtype=dtype, device="cuda"), torch.zeros(2, h, device="cuda")
    ws = torch.empty(max(1, swab.band_decode4_workspace(dec)), dtype=torch.uint8, device="cuda")
    swab.band_decode4(dec, 0.125, q[[0, 1]].contiguous(), *got, table, i32(lens), i32([0, 1, 2]), o, lse, ws)
    nan = o.isnan()
    assert nan[1, :2].all() and lse[1, :2].isnan().all() and nan[0, 2:, 32:].all()
    assert not nan[1, 2:].any() and not nan[0, :2].any() and not nan[0, 2:, :32].any() and not lse[0].isnan().any()


def test_decode_row_strides_streams_and_repeats():
    c = Decode4(BF16, [300, 1200, 47], [1, 2, 1], 4, 2, 128, page=32, seed=140)
    want = c.run()
    c.check(*want)
    qkv = randn((4, 8, 128), BF16, 141)
    qkv[:, :4] = c.q
    out = torch.full((4, 6, 128), 5.0, dtype=BF16, device="cuda")
    c.desc = swab.DecodeDesc(c.cache, 4, 4, 2, 128, max_q=2, max_len=1200, dtype=BF16, q_row_stride=8 * 128, out_row_stride=6 * 128)
    ws = torch.empty(max(1, swab.band_decode4_workspace(c.desc)), dtype=torch.uint8, device="cuda")
    swab.band_decode4(c.desc, c.scale, qkv[:, :4], *c.cells, i32(c.table), i32(c.lens), i32(c.q_start), out[:, :4], None, ws)
    same_bits(out[:, :4], want[0])
    assert (out[:, 4:] == 5.0).all()
    # two at once on streams of their own, workspaces of their own; then from graphs
    other = Decode4(BF16, [500, 900], [1, 1], 8, 2, 64, page=64, seed=142)
    ref = other.run()
    first = Decode4(BF16, [300, 1200, 47], [1, 2, 1], 4, 2, 128, page=32, seed=140)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        got = [x.run(stream=s) for x, s in zip((first, other), streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, (want, ref)):
            same_bits(a[0], b[0])
            same_bits(a[1], b[1])


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("graph", [False, True])
def test_steps_over_a_cache_in_4_bits(dtype, graph):
    """cache_slots, rotary_append4 with norms, band_decode4: prompts, then steps of up to two tokens under a window with
    recycled blocks, against attention in fp64 over the values that the cells stand for."""
    B, h, hk, hd, w, page, sinks = 3, 4, 2, 64, 40, 16, 5
    loop = swab.DecodeLoop(B, h, hk, hd, w, n_sink=sinks, max_new=2, page=page, dtype=dtype, bits=4, norm=swab.NormDesc(1e-5),
                           wq=randn((hd,), dtype, 150), wk=randn((hd,), dtype, 151))
    turns, freq, _ = frequencies(hd, "none")
    x = randn((B, 200, h + 2 * hk, hd), dtype, 152)
    n = [37, 5, 64]
    rows = torch.cat([x[r, :n[r]] for r in range(B)])
    q0 = loop.fill(rows, i32(n))
    # what the cells will stand for: keys and queries as the 16-bit calls compute them, quantised by the oracle
    d = swab.RotaryDesc(B, 200, h, hk, hd, hd, dtype=dtype)
    qn, kn = torch.empty(B, 200, h, hd, dtype=dtype, device="cuda"), torch.empty(B, 200, hk, hd, dtype=dtype, device="cuda")
    swab.norm_rotary(d, loop.norm, loop.turns, x[:, :, :h], qn, x[:, :, h:h + hk], kn, loop.wq, loop.wk)
    same_bits(q0, torch.cat([qn[r, :n[r]] for r in range(B)]))
    kv = []
    for y in (kn, x[:, :, h + hk:]):
        codes, scales = quant.quantise(f64(y), NAMES[dtype])
        kv.append(quant.values(codes, scales))
    step = loop.step
    if graph:
        loop.n_new.copy_(i32([1, 1, 1]))
        loop.qkv[:3] = torch.stack([x[r, n[r]] for r in range(B)])
        loop.step()                                                  # warm
        n = [m + 1 for m in n]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            loop.step()
        step = g.replay
    for s in range(30):
        new = [(1 + (r + s) % 2) if s % 5 else 1 for r in range(B)]
        loop.n_new.copy_(i32(new))
        loop.qkv[:sum(new)] = torch.cat([x[r, n[r]:n[r] + new[r]] for r in range(B)])
        step()
        if s % 6 == 5:
            c = Decode.__new__(Decode)
            c.q = torch.cat([qn[r, n[r]:n[r] + new[r]] for r in range(B)])
            # one block a position, so the oracle's table is the identity
            L = [m + k for m, k in zip(n, new)]
            c.kc, c.vc = (torch.tensor(np.concatenate([t[r, :L[r]] for r in range(B)])[:, :, None]).to(dtype).cuda() for t in kv)
            at = np.cumsum([0] + L)
            c.table = np.full((B, max(L)), -1)
            for r in range(B):
                c.table[r, :L[r]] = np.arange(at[r], at[r + 1])
            c.lens, c.q_start, c.scale, c.w, c.dilation, c.n_sink, c.ring, c.pinned = L, np.cumsum([0] + new), hd ** -0.5, w, 0, sinks, False, 0
            c.ptable, c.prefix, c.dtype, c.tokens = np.zeros(0, int), 0, dtype, sum(new)
            c.check(loop.out[:sum(new)].clone(), loop.lse[:sum(new)].clone())
        n = [m + k for m, k in zip(n, new)]
    assert loop.lens.tolist() == n and loop.used.tolist()[1] == 0


@pytest.mark.parametrize("bits", [4, None])
def test_loop_with_norms_and_in_16_bits(bits):
    """Norms without 4 bits and 4 bits without norms: the loop's results are those of its calls made by hand."""
    B, h, hk, hd, w, page = 2, 4, 2, 64, 30, 16
    kw = dict(bits=4) if bits else dict(norm=swab.NormDesc(), wq=randn((hd,), F16, 160), wk=randn((hd,), F16, 161))
    loop = swab.DecodeLoop(B, h, hk, hd, w, page=page, dtype=F16, **kw)
    x = randn((B, 60, h + 2 * hk, hd), F16, 162)
    loop.fill(x[:, :50].reshape(-1, h + 2 * hk, hd), i32([50, 50]))
    loop.n_new.fill_(1)
    loop.qkv.copy_(x[:, 50])
    loop.step()
    assert loop.lens.tolist() == [51, 51] and swab.device_status() == 0
    q, k, v = loop.qkv.split([h, hk, hk], dim=1)
    d = swab.RotaryDesc(1, B, h, hk, hd, hd, dtype=F16)
    qo, out, lse = torch.empty(B, h, hd, dtype=F16, device="cuda"), torch.empty(B, h, hd, dtype=F16, device="cuda"), torch.empty(B, h, device="cuda")
    dec = swab.DecodeDesc(loop.cache, B, h, hk, hd, w=w, max_len=1 << 30, dtype=F16)
    if bits:
        swab.rotary_append4(d, loop.cache, loop.turns, q, k, v, loop.pos, loop.slots, qo, loop.Kc, loop.Ks, loop.Vc, loop.Vs)
        ws = torch.empty(max(1, swab.band_decode4_workspace(dec)), dtype=torch.uint8, device="cuda")
        swab.band_decode4(dec, hd ** -0.5, qo, loop.Kc, loop.Ks, loop.Vc, loop.Vs, loop.table, loop.lens, loop.q_start, out, lse, ws)
    else:
        swab.norm_rotary_append(d, loop.norm, loop.cache, loop.turns, q, k, v, loop.pos, loop.slots, qo, loop.Kc, loop.Vc, loop.wq, loop.wk)
        ws = torch.empty(max(1, swab.band_decode_workspace(dec)), dtype=torch.uint8, device="cuda")
        swab.band_decode(dec, hd ** -0.5, qo, loop.Kc, loop.Vc, loop.table, loop.lens, loop.q_start, out, lse, ws)
    same_bits(out, loop.out)
    same_bits(lse, loop.lse)
    loop.restart([1])
    assert loop.lens.tolist() == [51, 0]


@pytest.mark.parametrize("name", ["tiny_fp32_n512_w32", "longformer_base_fp16_n4096_w256_d3", "train_bf16_b12_n4096_w256_g16"])
def test_run_workload_decodes_in_4_bits(name):
    res = subprocess.run([sys.executable, "-m", "sliding_window_attention_band_gb300.run_workload", "--workload", name, "--call",
                          "decode", "--bits", "4", "--repeat", "3"], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr[-2000:]


@pytest.mark.parametrize("dtype", [F16, F32])
def test_compiled_calls_and_the_binding_agree(dtype, monkeypatch):
    B, h, hk, hd, page = 2, 4, 2, 64, 16
    turns = swab.rotary_frequencies(hd)[0].cuda()
    cache, d, nd = swab.CacheDesc(B, page, 8, 4), swab.RotaryDesc(1, 10, h, hk, hd, hd, dtype=dtype), swab.NormDesc(1e-5)
    q, k, v = randn((10, h + 2 * hk, hd), dtype, 170).split([h, hk, hk], dim=1)
    w, pos = [randn((hd,), dtype, 171 + s) for s in range(2)], i32(np.arange(10) * 7)
    dec = swab.DecodeDesc(cache, 10, h, hk, hd, max_q=5, dtype=dtype)
    slots = i32([*range(5), *range(64, 69)])

    def all_calls():
        qo, o, lse = torch.zeros(10, h, hd, dtype=dtype, device="cuda"), torch.zeros(10, h, hd, dtype=dtype, device="cuda"), torch.zeros(10, h, device="cuda")
        got = empty_cells(cache, hk, hd, dtype)
        swab.rotary_append4(d, cache, turns, q, k, v, pos, slots, qo, *got)
        plain = [x.clone() for x in got]
        swab.rotary_append4(d, cache, turns, q, k, v, pos, slots, qo, *got, nd, *w)
        ko, vo = (torch.zeros(10, hk, hd, dtype=dtype, device="cuda") for _ in range(2))
        swab.cache_read4(cache, slots, *got, ko, vo)
        ws = torch.empty(max(16, swab.band_decode4_workspace(dec)), dtype=torch.uint8, device="cuda")
        swab.band_decode4(dec, 0.125, qo, *got, i32(np.arange(8).reshape(2, 4)), i32([5, 5]), i32([0, 5, 10]), o, lse, ws)
        with pytest.raises(swab.SwabError, match="INVALID"):
            swab.rotary_append4(d, cache, turns, q, k, v, pos, slots, qo, *got, swab.NormDesc(-1.0), *w)
        with pytest.raises(ValueError, match="lse"):
            swab.band_decode4(dec, 0.125, qo, *got, i32(np.arange(8).reshape(2, 4)), i32([5, 5]), i32([0, 5, 10]), o, lse.flatten(), ws)
        return [*plain, *got, qo, ko, vo, o, lse]

    got = all_calls()
    monkeypatch.setattr(swab.serve, "_calls", swab.serve._NoCalls)
    for a, b in zip(got, all_calls()):
        assert a.abs().sum() > 0
        same_bits(a, b)


@pytest.mark.parametrize("hd", [64, 32])
def test_offsets_past_32_bits(hd):
    """A cache whose codes and scales lie past 2^32 bytes: blocks at its end are written, read and attended to."""
    page, hk, dtype = 128, 64, F16
    blocks = (1 << 32) // (page * hk * hd // 2) + 9
    cache = swab.CacheDesc(1, page, blocks, 3)
    codes, scales = swab.cache4_shapes(cache, hk, hd)
    got = [torch.zeros(codes, dtype=torch.uint8, device="cuda"), torch.zeros(scales, dtype=dtype, device="cuda"),
           torch.zeros(codes, dtype=torch.uint8, device="cuda"), torch.zeros(scales, dtype=dtype, device="cuda")]
    assert got[0].numel() > 1 << 32
    T = 300
    k, v, q = randn((T, hk, hd), dtype, 180), randn((T, hk, hd), dtype, 181), randn((1, hk, hd), dtype, 182)
    ids = [blocks - 1, blocks - 5, blocks - 2]
    slots = np.array([ids[j // page] * page + j % page for j in range(T)])
    swab.rotary_append4(swab.RotaryDesc(1, T, hk, hk, hd, 0, dtype=dtype), cache, None, None, k, v, None, i32(slots), None, *got)
    for cs, x in ((got[:2], k), (got[2:], v)):
        c, s = cells(x[-20:], dtype)
        blk, off = torch.tensor(slots[-20:] // page).cuda(), torch.tensor(slots[-20:] % page).cuda()
        same_bits(cs[0][blk, :, off], c)
        same_bits(cs[1][blk, :, off], s)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    swab.cache_read4(cache, i32(slots), *got, ko, vo)
    dec = swab.DecodeDesc(cache, 1, hk, hk, hd, dtype=dtype, max_len=T)
    o, lse = torch.zeros_like(q), torch.zeros(1, hk, device="cuda")
    ws = torch.empty(max(16, swab.band_decode4_workspace(dec)), dtype=torch.uint8, device="cuda")
    swab.band_decode4(dec, hd ** -0.5, q, *got, i32([ids]), i32([T]), i32([0, 1]), o, lse, ws)
    K, V, Q = f64(ko), f64(vo), f64(q)[0]
    x = np.einsum("jhd,hd->hj", K, Q) * hd ** -0.5
    p = np.exp(x - x.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    ref = np.einsum("hj,jhd->hd", p, V)
    # (weights and the result rounded to fp16, sums of 300 terms of size 1)
    assert np.abs(f64(o)[0] - ref).max() < 4e-3


@pytest.mark.skipif(os.environ.get("SWAB_BOUNDS_CHECK") == "1", reason="is that run")
def test_bounds_checked_build_records_nothing():
    res = subprocess.run([sys.executable, "-m", "pytest", os.path.abspath(__file__), "-m", "gpu", "-x", "-q"], cwd=ROOT,
                         env=dict(os.environ, SWAB_BOUNDS_CHECK="1"), capture_output=True, text=True, timeout=1500)
    assert res.returncode == 0, res.stdout[-3000:] + res.stderr[-2000:]
