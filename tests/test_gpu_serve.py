"""Rotary positions, block tables, the cache write and decode against the fp64
oracle (oracle/serve.py), on the GPU.

Tolerances, set before the first run.  A stored value is off by at most half a
step of its type (u = eps / 2 relative).  Rotary: cos and sin come from an
argument within 2^-25 pi rad, sincospi within 2 ulp, the factor, the products
and the sum round once each: together below 2^-21 (|x_a| + |x_b|).  Decode: a
score of hd products in fp32 is within X (hd + 8) 2^-24 (X = the largest sum of
|q| |k| times the scale), times log2 e, and 2^x within 2^-21, so a weight is
within `delta` relatively; a sum of N weights adds N 2^-24; the tensor-core
kernels round a weight to 16 bits once more (u, and for fp16 at most 2^-25 of
the reference weight below its normal range).  O is a quotient of two such sums,
its numerator bounded by A = sum p |v|.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import sliding_window_attention_band_gb300 as swab
from oracle import serve as orc

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("device_status_guard")]

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
INVALID_BIT = 1 << 1
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def f64(t):
    return t.double().cpu().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def smallest_half_step(dtype):
    """Half the spacing below the normal range (fp16: its values reach it)."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32, 8: torch.int64}[t.element_size()])


def same_bits(a, b):
    assert torch.equal(bits(a), bits(b))


# ---------------------------------------------------------------------------
# rotary
# ---------------------------------------------------------------------------
def rotary_bound(x, ref, rot, interleaved, scale, dtype):
    """Per element: half a step of the result plus 2^-21 (|x_a| + |x_b|) scale."""
    a = np.abs(x)
    pair = np.zeros_like(a)
    if rot:
        k = np.arange(rot // 2)
        one, two = (2 * k, 2 * k + 1) if interleaved else (k, k + rot // 2)
        s = a[..., one] + a[..., two]
        pair[..., one] = pair[..., two] = s * abs(scale) * 2.0 ** -21
    return pair + (np.abs(ref) + pair) * half_step(dtype) + smallest_half_step(dtype)


def check_rotary(got, x, pos, freq, scale, interleaved, dtype, backward=False):
    ref = orc.rotary(f64(x), pos, freq, scale, interleaved, backward)
    err = np.abs(f64(got) - ref)
    bound = rotary_bound(f64(x), ref, 2 * len(freq), interleaved, scale, dtype)
    assert (err <= bound).all(), float((err - bound).max())
    same_bits(got[..., 2 * len(freq):], x[..., 2 * len(freq):])      # the rest is copied


ROTARY = [  # b, n, h, hk, hd, rot, interleaved, scaling
    (1, 1, 1, 0, 64, 64, False, "none"),
    (1, 1, 4, 2, 64, 64, True, "linear"),
    (2, 33, 5, 1, 80, 20, False, "yarn"),
    (2, 33, 5, 1, 80, 20, True, "bands"),
    (3, 70, 12, 4, 128, 128, False, "yarn"),
    (3, 70, 12, 4, 128, 64, True, "ntk"),
    (1, 257, 3, 3, 96, 96, False, "none"),
    (1, 9, 2, 2, 512, 510, False, "none"),
    (1, 5000, 2, 1, 64, 32, False, "none"),
    (2, 7, 3, 1, 64, 0, False, "none"),
    (1, 12, 3, 1, 64, 2, True, "none"),
    (1, 3, 700, 300, 64, 64, False, "none"),      # more heads than a block lists
    (1, 13000, 1, 0, 512, 512, True, "none"),     # the widest table
]


def frequencies(rot, scaling):
    factor, original = {"none": (1, 0), "linear": (4, 0), "ntk": (8, 0), "yarn": (16, 8192), "bands": (8, 8192)}[scaling]
    if rot == 0:
        return None, np.zeros(0), 1.0
    turns, scale = swab.rotary_frequencies(rot, 10000.0, scaling, factor, original)
    freq, _ = orc.frequencies(rot, 10000.0, scaling, factor, original, 1.0, 32.0 if scaling == "yarn" else 4.0)
    return turns.cuda(), freq, scale


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("case", ROTARY)
def test_rotary_matches_the_oracle(case, dtype):
    b, n, h, hk, hd, rot, inter, scaling = case
    turns, freq, scale = frequencies(rot, scaling)
    q, k = randn((b, n, h, hd), dtype, 1), randn((b, n, max(hk, 1), hd), dtype, 2)
    rng = np.random.default_rng(3)
    pos = rng.integers(0, 1_000_000, (b, n))
    d = swab.RotaryDesc(b, n, h, hk, hd, rot, inter, scale, dtype=dtype)
    for fn, back in ((swab.rotary, False), (swab.rotary_bwd, True)):
        qo, ko = torch.empty_like(q), torch.full_like(k, 3.0)
        fn(d, turns, q, qo, k if hk else None, ko if hk else None, pos=i32(pos))
        check_rotary(qo, q, pos, freq, scale, inter, dtype, back)
        if hk:
            check_rotary(ko, k, pos, freq, scale, inter, dtype, back)


@pytest.mark.parametrize("dtype", [F16, F32])
def test_rotary_positions_at_the_ends_of_their_range(dtype):
    """Negative positions, 0 and the last int32; pos None counts from pos0 in every sequence."""
    turns, freq, scale = frequencies(64, "none")
    pos = np.array([[-1, 0, 1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1]])
    x = randn((1, 6, 2, 64), dtype, 4)
    y = torch.empty_like(x)
    swab.rotary(swab.RotaryDesc(1, 6, 2, 0, 64, 64, dtype=dtype), turns, x, y, pos=i32(pos))
    check_rotary(y, x, pos, freq, 1.0, False, dtype)
    x = randn((3, 5, 2, 64), dtype, 5)
    y = torch.empty_like(x)
    swab.rotary(swab.RotaryDesc(3, 5, 2, 0, 64, 64, pos0=1000, dtype=dtype), turns, x, y)
    check_rotary(y, x, np.tile(1000 + np.arange(5), (3, 1)), freq, 1.0, False, dtype)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
def test_rotary_angles_next_to_quarter_turns(inter, sign):
    """x = (1, 0) gives (cos t, sin t) themselves.  The turns are cut to 2^-32 (2 pi 2^-32 rad); what is left of the
    quarter turn is then rounded relatively (2^-24) and its sine and cosine are within 2 ulp (2^-22), so a small value
    keeps its bits: nothing of the size of the whole angle's rounding (2^-25 pi) may show."""
    N = 256
    rng = np.random.default_rng(40)
    quarter, off = rng.integers(0, 4, N), (2.0 ** rng.uniform(33, 61, N)).astype(np.int64) * rng.choice([-1, 1], N)
    turns = ((quarter.astype(object) << 62) + off.astype(object)) % (1 << 64)
    t64 = torch.tensor([int(t) - (1 << 64) if t >= 1 << 63 else int(t) for t in turns], dtype=torch.int64).cuda()
    x = torch.zeros(1, 1, 1, 2 * N, dtype=F32, device="cuda")
    (x[..., 0::2] if inter else x[..., :N]).fill_(1.0)
    y = torch.empty_like(x)
    swab.rotary(swab.RotaryDesc(1, 1, 1, 0, 2 * N, 2 * N, inter, dtype=F32), t64, x, y, pos=i32([[sign]]))
    a = off.astype(np.float64) * 2 * np.pi * 2.0 ** -64          # the part past the quarter turns
    c, s = np.cos(a), np.sin(a)
    cos = np.choose(quarter, [c, -s, -c, s])
    sin = np.choose(quarter, [s, c, -s, -c]) * sign
    got = f64(y).reshape(-1)
    got_c, got_s = (got[0::2], got[1::2]) if inter else (got[:N], got[N:])
    for g, w in ((got_c, cos), (got_s, sin)):
        assert (np.abs(g - w) <= 2 * np.pi * 2.0 ** -32 + np.abs(w) * (2.0 ** -24 + 2.0 ** -22)).all(), np.abs(g - w).max()


@pytest.mark.parametrize("inter", [False, True])
def test_rotary_on_strided_views_and_in_place(inter):
    """Q, K inside a merged projection, outputs head-major; then in place, which gives the same bits."""
    b, n, h, hk, hd, rot = 2, 37, 4, 2, 64, 32
    turns, freq, scale = frequencies(rot, "none")
    qkv = randn((b, n, h + 2 * hk, hd), BF16, 6)
    q, k = qkv[:, :, :h], qkv[:, :, h:h + hk]
    pos = np.tile(np.arange(n) + 7, (b, 1))
    d = swab.RotaryDesc(b, n, h, hk, hd, rot, inter, dtype=BF16)
    qo = torch.empty(b, h, n, hd, dtype=BF16, device="cuda").transpose(1, 2)
    ko = torch.empty(b, hk, n, hd, dtype=BF16, device="cuda").transpose(1, 2)
    swab.rotary(d, turns, q, qo, k, ko, pos=i32(pos))
    check_rotary(qo, q, pos, freq, scale, inter, BF16)
    check_rotary(ko, k, pos, freq, scale, inter, BF16)
    v = qkv[:, :, h + hk:].clone()
    swab.rotary(d, turns, q, q, k, k, pos=i32(pos))
    same_bits(q, qo)
    same_bits(k, ko)
    same_bits(qkv[:, :, h + hk:], v)
    # one row of positions and heads read for every batch entry
    one = randn((1, n, h, hd), BF16, 8).expand(b, n, h, hd)
    out = torch.empty(b, n, h, hd, dtype=BF16, device="cuda")
    swab.rotary(swab.RotaryDesc(b, n, h, 0, hd, rot, inter, dtype=BF16), turns, one, out, pos=i32(pos))
    check_rotary(out, one, pos, freq, scale, inter, BF16)


def test_rotary_gradient_against_differences():
    """The map is linear, so a difference over any step is its derivative: (f(x + e) - f(x - e)) / 2 along unit
    steps, f = sum(g * y).  Both sides carry fp32 roundings only: y and g below 8 in magnitude, two values each."""
    b, n, h, hd, rot = 1, 3, 1, 16, 12
    turns, _, scale = frequencies(rot, "yarn")
    d = swab.RotaryDesc(b, n, h, 0, hd, rot, False, scale, dtype=F32)
    x, g = randn((b, n, h, hd), F32, 9), randn((b, n, h, hd), F32, 10)
    pos = i32([[5, 1000, 70000]])
    dx = torch.empty_like(x)
    swab.rotary_bwd(d, turns, g, dx, pos=pos)

    def f(v):
        y = torch.empty_like(v)
        swab.rotary(d, turns, v, y, pos=pos)
        return (y.double() * g.double()).sum().item()

    for at in range(0, x.numel(), 5):
        e = torch.zeros(x.numel(), device="cuda").view_as(x)
        e.view(-1)[at] = 1.0
        assert abs((f(x + e) - f(x - e)) / 2 - dx.view(-1)[at].item()) <= 8 * 8 * 2.0 ** -21


# ---------------------------------------------------------------------------
# block tables and slots
# ---------------------------------------------------------------------------
def run_slots(cache, lens, new, table, free, used, tokens, pos0=0, in_place=False):
    t, L = i32(table), i32(lens)
    U = torch.tensor([used, -7], dtype=torch.int32).cuda()
    lo, uo = (L, U) if in_place else (torch.full_like(L, -9), torch.full_like(U, -9))
    e = lambda k: torch.full((k,), -9, dtype=torch.int32, device="cuda")  # noqa: E731
    start, slots, pos = e(len(lens) + 1), e(tokens), e(tokens)
    swab.cache_slots(cache, L, i32(new), t, i32(free) if len(free) else e(0), U if in_place else U[:1].contiguous(), lo, uo,
                     start, slots, pos, pos0=pos0)
    return [x.cpu().numpy() for x in (t, lo, uo, start, slots, pos)]


def slots_case(batch, page, cols, ring, pinned, len_hi, new_hi, seed, short=0):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, len_hi + 1, batch)
    new = rng.integers(0, new_hi + 1, batch)
    have = np.minimum(-(-lens // page), cols)
    want = np.minimum(-(-(lens + new) // page), cols)
    n_blocks = int(want.sum()) + 7
    perm = rng.permutation(n_blocks)
    table, at = np.full((batch, cols), -1), 0
    for r in range(batch):
        table[r, :have[r]] = perm[at:at + have[r]]
        at += have[r]
    free = np.concatenate([[n_blocks - 1] * 2, perm[at:]])[:max(2, 2 + int((want - have).sum()) - short)]
    return swab.CacheDesc(batch, page, n_blocks, cols, ring, pinned), lens, new, table, free


SLOTS = [  # batch, page, cols, ring, pinned, len_hi, new_hi, missing blocks
    (1, 16, 4, False, 0, 0, 1, 0),
    (1, 16, 40, False, 0, 300, 300, 0),
    (7, 64, 6, True, 0, 2000, 1, 0),
    (7, 64, 6, True, 2, 2000, 700, 0),
    (64, 32, 300, False, 0, 5000, 3, 0),
    (1500, 128, 90, False, 0, 9000, 5, 0),
    (300, 16, 5, True, 1, 100, 60, 0),
    (40, 16, 600, False, 0, 4000, 900, 0),
    (40, 16, 600, False, 0, 4000, 900, 25),
    (40, 16, 120, False, 0, 1500, 900, 0),       # some requests pass the table
    (2, 16, 2, True, 1, 4, 200, 0),              # a step longer than the recycled table
    (3, 16, 8, False, 0, 100, 0, 0),             # nothing new
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", SLOTS)
def test_cache_slots_matches_the_oracle(case, in_place):
    batch, page, cols, ring, pinned, len_hi, new_hi, short = case
    cache, lens, new, table, free = slots_case(batch, page, cols, ring, pinned, len_hi, new_hi, 11, short)
    tokens = int(new.sum()) + 5
    got = run_slots(cache, lens, new, table, free, 2, tokens, pos0=13, in_place=in_place)
    want = orc.cache_slots(lens, new, table, free, 2, page, cols, ring, pinned, tokens, 13)
    for name, g, w in zip(("table", "lens", "used", "start", "slots", "pos"), got, want):
        np.testing.assert_array_equal(g, w, err_msg=name)
    live = got[4][got[4] >= 0]
    assert len(np.unique(live)) == len(live)       # no two tokens share a slot


def test_cache_slots_writes_no_token_past_its_rows_and_takes_negative_counts_as_none():
    cache, _, _, table, free = slots_case(4, 16, 10, False, 0, 0, 0, 12)
    free = np.arange(cache.n_blocks)
    lens, new = [-5, 3, 0, 16], [4, -2, 100, 1]
    got = run_slots(cache, lens, new, table, free[:7], 0, 50)
    want = orc.cache_slots(lens, new, table, free[:7], 0, 16, 10, tokens=50)
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g, w)
    assert swab.device_status(reset=True) == 0


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", [(7, 16, 5, True, 1, 100, 6, 4, 0), (40, 16, 600, False, 0, 4000, 90, 60, 300),
                                  (1500, 128, 90, False, 0, 9000, 5, 5, 1000), (40, 16, 600, False, 0, 4000, 900, 2 ** 31 - 1, 5000)])
def test_cache_slots_serves_no_request_past_its_limits(case, in_place):
    """More tokens than max_new, or than there are rows for: slots of -1, the length kept, no block lost, the status raised."""
    batch, page, cols, ring, pinned, len_hi, new_hi, max_new, cut = case
    cache, lens, new, table, free = slots_case(batch, page, cols, ring, pinned, len_hi, new_hi, 13)
    cache = swab.CacheDesc(batch, page, cache.n_blocks, cols, ring, pinned, max_new=max_new)
    tokens = int(new.sum()) - cut
    got = run_slots(cache, lens, new, table, free, 2, tokens, pos0=13, in_place=in_place)
    want = orc.cache_slots(lens, new, table, free, 2, page, cols, ring, pinned, tokens, 13, max_new=max_new)
    for name, g, w in zip(("table", "lens", "used", "start", "slots", "pos"), got, want):
        np.testing.assert_array_equal(g, w, err_msg=name)
    assert got[2][1] > 0 and swab.device_status(reset=True) == INVALID_BIT
    # the same within the limits raises nothing
    within = np.minimum(new, max_new)
    run_slots(cache, lens, within, table, free, 2, int(within.sum()), pos0=13, in_place=in_place)
    assert swab.device_status(reset=True) == 0


def test_cache_slots_flags_blocks_outside_the_cache():
    cache = swab.CacheDesc(2, 16, 4, 3)
    table = [[4, -1, -1], [1, -1, -1]]              # block 4 of a cache of 4
    got = run_slots(cache, [3, 3], [2, 2], table, [2, 3], 0, 4)
    np.testing.assert_array_equal(got[4], [-1, -1, 19, 20])
    assert swab.device_status(reset=True) == INVALID_BIT


# ---------------------------------------------------------------------------
# the cache write
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("case", [(1, 4, 2, 64, 64, False, 16), (23, 5, 1, 80, 20, True, 16), (200, 12, 4, 128, 64, False, 64),
                                  (9, 2, 2, 64, 0, False, 128), (6000, 2, 1, 64, 64, True, 32)])
def test_rotary_append_matches_the_oracle(case, dtype):
    T, h, hk, hd, rot, inter, page = case
    turns, freq, scale = frequencies(rot, "bands")
    rng = np.random.default_rng(20)
    n_blocks = T // page + 3
    slots = rng.permutation(n_blocks * page)[:T]
    slots[rng.random(T) < 0.2] = -1
    pos = rng.integers(0, 100000, T)
    qkv = randn((T, h + 2 * hk, hd), dtype, 21)
    q, k, v = qkv.split([h, hk, hk], dim=1)
    kc, vc = randn((n_blocks, hk, page, hd), dtype, 22), randn((n_blocks, hk, page, hd), dtype, 23)
    k0, v0 = kc.clone(), vc.clone()
    qo = torch.empty(T, h, hd, dtype=dtype, device="cuda")
    d = swab.RotaryDesc(1, T, h, hk, hd, rot, inter, scale, dtype=dtype)
    cache = swab.CacheDesc(1, page, n_blocks, 1)
    swab.rotary_append(d, cache, turns, q, k, v, i32(pos), i32(slots), qo, kc, vc)
    check_rotary(qo, q, pos, freq, scale, inter, dtype)
    keep = slots >= 0
    b, o = torch.tensor(slots[keep] // page).cuda(), torch.tensor(slots[keep] % page).cuda()
    rows = torch.tensor(np.nonzero(keep)[0]).cuda()
    check_rotary(kc[b, :, o], k[rows], pos[keep], freq, scale, inter, dtype)
    same_bits(vc[b, :, o], v[rows])
    untouched = torch.ones(n_blocks, page, dtype=torch.bool, device="cuda")
    untouched[b, o] = False
    same_bits(kc.transpose(1, 2)[untouched], k0.transpose(1, 2)[untouched])
    same_bits(vc.transpose(1, 2)[untouched], v0.transpose(1, 2)[untouched])
    # without Q: the same cache
    k1, v1 = k0.clone(), v0.clone()
    swab.rotary_append(d, cache, turns, None, k, v, i32(pos), i32(slots), None, k1, v1)
    same_bits(k1, kc)
    same_bits(v1, vc)


def test_rotary_append_skips_and_flags_slots_outside_the_cache():
    cache = swab.CacheDesc(1, 16, 2, 1)
    d = swab.RotaryDesc(1, 4, 1, 1, 64, 0, dtype=F16)
    q, k, v = (randn((4, 1, 64), F16, s) for s in (1, 2, 3))
    kc, vc = torch.zeros(2, 1, 16, 64, dtype=F16, device="cuda"), torch.zeros(2, 1, 16, 64, dtype=F16, device="cuda")
    swab.rotary_append(d, cache, None, q, k, v, None, i32([32, -2, 31, -1]), torch.empty_like(q), kc, vc)
    assert swab.device_status(reset=True) == INVALID_BIT
    same_bits(kc[1, 0, 15], k[2, 0])
    same_bits(vc[1, 0, 15], v[2, 0])
    assert int((kc != 0).any(-1).sum()) == 1


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
class Decode:
    """A batch over a cache that holds NaN wherever no query of a request looks."""

    def __init__(self, dtype, lens, new, h, hk, hd, page=16, w=None, dilation=0, n_sink=0, ring=False, prefix=0, pad=0, seed=0,
                 max_len=None, qscale=1.0):
        rng = np.random.default_rng(seed)
        self.dtype, self.lens, self.new = dtype, list(lens), list(new)
        self.w = 1 << 30 if w is None else w
        self.dilation, self.n_sink, self.ring, self.prefix = dilation, n_sink, ring, prefix
        B, s = len(lens), dilation + 1
        max_q = max(1, max(new))
        self.pinned = -(-n_sink // page) if ring else 0
        cols = self.pinned + -(-(self.w * s + max_q - 1) // page) + 1 if ring else max(1, -(-max(lens) // page))
        used = [min(-(-x // page), cols) for x in lens]
        pre = -(-prefix // page)
        n_blocks = sum(used) + pre + 2
        perm = rng.permutation(n_blocks)
        table, at = np.full((B, cols), -1), 0
        for r in range(B):
            table[r, :used[r]] = perm[at:at + used[r]]
            at += used[r]
        self.table, self.ptable = table, perm[at:at + pre]
        self.q_start = np.concatenate([[0], np.cumsum(new)])
        self.tokens = int(self.q_start[-1]) + pad
        self.q = randn((max(1, self.tokens), h, hd), dtype, seed + 1, qscale)
        self.kc = torch.full((n_blocks, hk, page, hd), float("nan"), dtype=dtype, device="cuda")
        self.vc = torch.full_like(self.kc, float("nan"))
        rows = [(self.ptable[p // page], p % page) for p in range(prefix)]
        for r in range(B):
            seen = set()
            for i in range(lens[r] - new[r], lens[r]):
                seen |= set(orc.keys_of(i, self.w, dilation, n_sink))
            rows += [(table[r, orc.column(j // page, cols, ring, self.pinned)], j % page) for j in sorted(seen)]
        if rows:
            b, o = (torch.tensor([int(x[k]) for x in rows]).cuda() for k in (0, 1))
            self.kc[b, :, o] = randn((len(rows), hk, hd), dtype, seed + 2)
            self.vc[b, :, o] = randn((len(rows), hk, hd), dtype, seed + 3)
        self.cache = swab.CacheDesc(B, page, n_blocks, cols, ring, self.pinned)
        self.desc = swab.DecodeDesc(self.cache, max(1, self.tokens), h, hk, hd, self.w, dilation, n_sink, max_q,
                                    max_len or max(1, max(lens)), prefix, dtype)
        self.scale = hd ** -0.5

    def run(self, stream=None, lse=True):
        o = torch.full_like(self.q, 7.0)
        l = torch.full(self.q.shape[:2], 7.0, dtype=F32, device="cuda") if lse else None
        ws = torch.empty(swab.band_decode_workspace(self.desc) + 16, dtype=torch.uint8, device="cuda")[16:]   # 16-byte aligned, no more
        swab.band_decode(self.desc, self.scale, self.q, self.kc, self.vc, i32(self.table), i32(self.lens), i32(self.q_start),
                         o, l, ws, i32(self.ptable) if self.prefix else None, stream=stream)
        return o, l

    def oracle(self):
        return orc.decode(f64(self.q), f64(self.kc), f64(self.vc), self.table, self.lens, self.q_start, self.scale, self.w,
                          self.dilation, self.n_sink, self.ring, self.pinned, self.ptable, self.prefix)

    def check(self, o=None, lse=None):
        if o is None:
            o, lse = self.run()
        O, L, A, X = self.oracle()
        u, hd, n = half_step(self.dtype), self.q.shape[2], self.prefix + max(self.lens) + 4
        delta = (X * (hd + 8) * 2.0 ** -24 * 1.5 + 2.0 ** -21)[..., None]
        weight = 0.0 if self.dtype == F32 else u
        tiny = n * 2.0 ** -25 * 6.0 if self.dtype == F16 else 0.0        # |v| below 6
        bound = A * (2 * delta + 2 * n * 2.0 ** -24 + weight) + tiny
        bound = bound + (np.abs(O) + bound) * u + smallest_half_step(self.dtype)
        live = int(self.q_start[-1])
        live = min(live, self.tokens)
        err = np.abs(f64(o)[:live] - O[:live])
        assert (err <= bound[:live]).all(), float(np.nanmax(err / np.maximum(bound[:live], 1e-30)))
        if lse is not None:
            got = f64(lse)[:live]
            empty = np.isneginf(L[:live])
            assert (np.isneginf(got) == empty).all()
            lb = (delta[..., 0] + n * 2.0 ** -24 + (np.abs(L) + 1) * 2.0 ** -22)[:live]
            diff = np.abs(np.where(empty, 0.0, got) - np.where(empty, 0.0, L[:live]))
            assert (diff <= np.where(empty, 0.0, lb)).all(), float(diff.max())
            assert (f64(lse)[live:] == 7.0).all()
        assert (f64(o)[live:] == 7.0).all()              # rows of no request stay as they were


LENGTHS = [([1], [1]), ([5], [1]), ([16, 17, 1, 33], [1, 1, 1, 1]), ([300, 1, 47], [1, 1, 1]),
           ([40, 0, 9, 64], [3, 0, 1, 4]), ([2, 70], [2, 0])]


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("heads", [(4, 4, 64), (8, 2, 128), (6, 1, 64), (5, 5, 80), (2, 2, 256), (3, 1, 128)])
def test_decode_matches_the_oracle(heads, dtype):
    for k, (lens, new) in enumerate(LENGTHS):
        Decode(dtype, lens, new, *heads, seed=30 + k, pad=k % 3).check()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("case", [
    dict(w=0), dict(w=7), dict(w=16, n_sink=3), dict(w=31, n_sink=16, page=32), dict(w=5, dilation=1),
    dict(w=9, dilation=3, n_sink=5), dict(w=20, ring=True), dict(w=20, ring=True, n_sink=20, page=16),
    dict(w=6, dilation=2, ring=True, n_sink=1), dict(w=100, n_sink=90), dict(w=3, n_sink=400), dict(w=40, dilation=15)])
def test_decode_windows_and_sinks(case, dtype):
    for heads in ((4, 2, 64), (2, 1, 128)):
        for k, (lens, new) in enumerate(LENGTHS[1:]):
            Decode(dtype, lens, new, *heads, seed=50 + k, **case).check()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("prefix", [1, 15, 16, 100, 129, 700])
@pytest.mark.parametrize("heads", [(4, 2, 64), (7, 1, 128), (3, 3, 64), (2, 2, 80)])
def test_decode_behind_a_shared_prefix(heads, prefix, dtype):
    for k, (lens, new) in enumerate(LENGTHS[1:]):
        Decode(dtype, lens, new, *heads, prefix=prefix, seed=70 + k, pad=k % 2).check()
    Decode(dtype, [80, 3], [2, 1], *heads, prefix=prefix, w=11, n_sink=2, page=32, seed=80).check()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("case", [
    dict(lens=[5000], new=[1], h=4, hk=1, hd=128, page=64), dict(lens=[3000, 17, 4100], new=[1, 1, 1], h=4, hk=2, hd=64, page=128),
    dict(lens=[2500, 900], new=[4, 7], h=16, hk=2, hd=128, page=32),          # more rows than a tile
    dict(lens=[1500], new=[1], h=128, hk=1, hd=64, page=16),                  # one key head for 128
    dict(lens=[2600, 2601], new=[1, 2], h=4, hk=4, hd=64, w=2048, page=64, ring=True),
    dict(lens=[100] * 70, new=[1] * 70, h=8, hk=2, hd=64, prefix=1000),       # more prefix rows than a tile
    dict(lens=[30] * 9, new=[3] * 9, h=20, hk=4, hd=128, prefix=600, page=64),
    dict(lens=[700], new=[40], h=2, hk=1, hd=64)])
def test_decode_long_and_wide(case, dtype):
    Decode(dtype, seed=90, **case).check()


def check_some(c, o, lse, requests):
    """Decode.check for the named requests of a large batch: each against the oracle over its own blocks."""
    for r in requests:
        pre = len(c.ptable) if c.prefix else 0
        used = c.table[r][c.table[r] >= 0]
        blocks = torch.tensor(np.concatenate([c.ptable[:pre], used]).astype(np.int64), device="cuda")
        one = Decode.__new__(Decode)
        one.__dict__.update(c.__dict__)
        rows = slice(int(c.q_start[r]), int(c.q_start[r + 1]))
        one.q, one.kc, one.vc, one.tokens = c.q[rows], c.kc[blocks], c.vc[blocks], rows.stop - rows.start
        one.table, one.ptable = np.full((1, c.table.shape[1]), -1), np.arange(pre)
        one.table[0, :len(used)] = pre + np.arange(len(used))
        one.lens, one.q_start = [c.lens[r]], np.array([0, one.tokens])
        one.check(o[rows], lse[rows])


# 12 warps an SM come as blocks of four, three or two by how many blocks there are (152 SMs: 456 of four, 608 of
# three, 912 of two fit at once) and, for lists of 2048 keys and more, by how well the pieces fill them
BLOCKS = [  # requests, most keys, and: how the rows kernel runs
    dict(n=60, keys=600, h=16, hk=8),                        # 480 blocks: three warps, lists whole
    dict(n=60, keys=600, h=16, hk=8, prefix=260),            # three warps, the prefix's parts folded in
    dict(n=60, keys=600, h=8, hk=8, m=2, w=300, n_sink=5),   # three warps under a window
    dict(n=100, keys=500, h=8, hk=8),                        # 800 blocks: two warps
    dict(n=100, keys=500, h=16, hk=8, prefix=300),           # two warps, the prefix's parts folded in
    dict(n=32, keys=2600, h=8, hk=8),                        # 256 long lists: three warps, two pieces
    dict(n=32, keys=2600, h=8, hk=8, prefix=700),            # three warps, two pieces and the prefix's parts joined
    dict(n=45, keys=2600, h=8, hk=4, m=2),                   # 180 long lists: two warps, five pieces
    dict(n=45, keys=2600, h=8, hk=4, m=2, prefix=300),       # two warps, five pieces and the prefix's parts joined
    dict(n=130, keys=400, h=8, hk=8),                        # 1040 blocks: four warps, more than fit at once
    dict(n=130, keys=400, h=8, hk=8, prefix=300)]


@pytest.mark.parametrize("dtype,hd", [(F16, 64), (BF16, 128), (F16, 128), (BF16, 64)])
@pytest.mark.parametrize("case", BLOCKS)
def test_decode_in_blocks_of_four_three_and_two_warps(case, dtype, hd):
    n, keys, m = case["n"], case["keys"], case.get("m", 1)
    rng = np.random.default_rng(113)
    lens, new = rng.integers(m, keys + 1, n), rng.integers(0, m + 1, n)
    lens[n // 2], new[n // 2], new[0], new[n - 1] = keys, m, m, 1
    if keys > 2000:
        lens[rng.random(n) < 0.7] //= 16             # (few of the long ones are filled in)
        lens, lens[n // 2] = np.maximum(lens, m), keys
    c = Decode(dtype, lens.tolist(), new.tolist(), case["h"], case["hk"], hd, page=64, w=case.get("w"),
               n_sink=case.get("n_sink", 0), prefix=case.get("prefix", 0), pad=2, seed=114)
    o, lse = c.run()
    assert (o[int(c.q_start[-1]):] == 7.0).all() and not o.isnan().any()
    check_some(c, o, lse, sorted({0, 1, n // 3, n // 2, n - 2, n - 1}))


def test_decode_of_contexts_longer_than_announced():
    """max_len divides the work only."""
    for dtype in (F16, F32):
        Decode(dtype, [900, 40], [1, 1], 4, 2, 64, max_len=1, seed=95).check()
        Decode(dtype, [900, 40], [2, 1], 4, 2, 64, max_len=300, prefix=40, seed=96).check()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_decode_with_large_scores(dtype):
    """Scores of a few hundred: the running maximum keeps the weights finite."""
    Decode(dtype, [200, 31], [1, 2], 4, 2, 64, qscale=40.0, prefix=50, seed=97).check()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 2, 128)])
def test_decode_with_scores_that_keep_growing(heads, dtype):
    """Keys that grow along the prefix and along the own context: the reference is raised again and again, and what was
    summed so far scaled."""
    c = Decode(dtype, [700, 300], [1, 2], *heads, page=64, prefix=900, qscale=2.0, seed=108)
    for p in range(900):
        c.kc[int(c.ptable[p // 64]), :, p % 64] *= 0.2 + p / 300
    for r in range(2):
        for j in range(c.lens[r]):
            c.kc[int(c.table[r, j // 64]), :, j % 64] *= 0.2 + j / 100
    c.check()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("case", [dict(h=128, hk=1, hd=64, page=16), dict(h=100, hk=1, hd=128, page=64),
                                  dict(h=12, hk=4, hd=64, page=128), dict(h=24, hk=8, hd=128, page=32)])
def test_prefix_row_tiles(case, dtype):
    """Groups that leave rows of a tile over, one row tile and several, every page size."""
    for lens, new in (([20, 5], [1, 1]), ([9] * 50, [1] * 50)):
        Decode(dtype, lens, new, prefix=300, seed=109, **case).check()


def test_prefix_with_absent_blocks():
    """Columns of the prefix that are -1 are skipped without an error; all of them: the own keys alone."""
    for dtype in (F16, F32):
        for gone in ([1], [0, 2, 3], list(range(13))):
            c = Decode(dtype, [20, 5, 3], [1, 1, 2], 4, 2, 64, prefix=200, seed=110)
            c.ptable = c.ptable.copy()
            c.ptable[gone] = -1
            c.check()
    assert swab.device_status(reset=True) == 0


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("scale", [0.0, -0.125, 1e-4, 3.0])
def test_decode_scales(dtype, scale):
    """Negative scales turn the order of the scores round, zero makes the weights equal."""
    for prefix in (0, 70):
        c = Decode(dtype, [90, 21], [2, 1], 4, 2, 64, w=60, prefix=prefix, seed=106)
        c.scale = scale
        c.check()


def test_decode_without_keys():
    """Contexts shorter than their new tokens, empty columns: rows without a key give 0 and -inf."""
    for dtype in (F16, F32):
        c = Decode(dtype, [4, 20], [2, 1], 4, 2, 64, seed=98)
        c.lens[0] = 1                                  # two new tokens, one position held
        c.check()
        c.lens[0] = 0
        c.check()
        c = Decode(dtype, [4, 20], [2, 1], 4, 2, 64, seed=99)
        c.table[0, :] = -1                             # nothing allocated: absent, not an error
        c.check()
    assert swab.device_status(reset=True) == 0


NOT_FINITE = [  # how the lists are cut: whole, pieces joined by a launch of their own, behind a prefix (folded, joined)
    dict(lens=[40, 20, 9], new=[1, 2, 1], h=4, hk=2, hd=64),
    dict(lens=[3000, 50], new=[1, 1], h=8, hk=2, hd=128, page=64),
    dict(lens=[40, 20, 9], new=[1, 2, 1], h=4, hk=2, hd=64, prefix=70),
    dict(lens=[30] * 40, new=[1] * 40, h=8, hk=4, hd=128, page=64, prefix=260),
    dict(lens=[20] * 16, new=[1] * 16, h=32, hk=8, hd=128, page=64, prefix=4096),
    dict(lens=[40, 20, 9], new=[1, 2, 1], h=6, hk=2, hd=80),
    dict(lens=[2000], new=[2], h=2, hk=2, hd=80)]


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("case", NOT_FINITE)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_decode_of_queries_that_are_not_finite(case, dtype, bad):
    """softmax of NaN is NaN: a query with a NaN, or with both infinities, gives NaN in O and lse, however its list is
    cut, and leaves the other heads and tokens as they are."""
    c = Decode(dtype, seed=111, **case)
    want, wlse = c.run()
    rows, heads, q = [0, c.tokens - 1], [0, c.q.shape[1] - 1], c.q.clone()
    for t, h in zip(rows, heads):
        c.q[t, h, 5], c.q[t, h, 6] = bad, -bad
    o, lse = c.run()
    hit = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    hit[rows, heads] = True
    assert o[hit].isnan().all() and lse[hit].isnan().all()
    # (not the same bits: an infinite score makes its warp raise the references of the rows beside it as well)
    o[hit], lse[hit], c.q = want[hit], wlse[hit], q
    c.check(o, lse)


def test_decode_skips_and_flags_blocks_outside_the_cache():
    for dtype in (F16, F32):
        for prefix in (0, 40):
            c = Decode(dtype, [40, 20], [1, 1], 4, 2, 64, prefix=prefix, seed=100)
            c.table[0, 1] = c.cache.n_blocks
            c.table[1, 0] = -5
            if prefix:
                c.ptable = c.ptable.copy()
                c.ptable[1] = 1 << 30
            c.check()
            assert swab.device_status(reset=True) == INVALID_BIT
        c = Decode(dtype, [40, 20], [1, 1], 4, 2, 64, seed=101)
        c.kc.nan_to_num_(0.5)
        c.vc.nan_to_num_(0.5)
        c.lens[0] = 200                                # longer than its table
        c.check()
        assert swab.device_status(reset=True) == INVALID_BIT


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("case", [dict(), dict(w=30), dict(w=3, dilation=2, n_sink=2), dict(w=20, ring=True)])
def test_decode_of_lengths_that_make_no_sense(dtype, case):
    """A length up to the last int32, row starts that go backwards or below zero: the call ends, the other requests are
    right, and a length past its table is flagged."""
    c = Decode(dtype, [40, 20, 30], [1, 2, 1], 4, 2, 64, seed=107, **case)
    want, lse = c.run()
    for bad in (2 ** 31 - 1, 2 ** 31 - 17, 49):
        c.lens[0] = bad
        o, l = c.run()
        same_bits(o[1:], want[1:])
        same_bits(l[1:], lse[1:])
        assert swab.device_status(reset=True) == (0 if c.ring else INVALID_BIT)
    c.lens[0] = 40
    for starts in ([-5, 1, 3, 4], [-2 ** 31, 1, 3, 4], [7, 1, 3, 4]):
        c.q_start = np.array(starts)
        o, l = c.run()
        same_bits(o[1:], want[1:])
        same_bits(l[1:], lse[1:])
    c.q_start = np.array([0, 1, 3, 2 ** 31 - 1])
    same_bits(c.run()[0][:3], want[:3])
    assert swab.device_status(reset=True) == 0


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("prefix", [0, 40])
def test_decode_of_row_starts_that_fall_from_above_zero_to_the_lowest_integer(dtype, prefix):
    """Their difference does not fit 32 bits: no row belongs to the first request, the last one is right."""
    c = Decode(dtype, [40, 20, 30], [1, 2, 1], 4, 2, 64, prefix=prefix, seed=107)
    want, lse = c.run()
    for starts in ([3, -2 ** 31, 3, 4], [2, -2 ** 31 + 1, 3, 4], [2 ** 31 - 1, -2 ** 31, 3, 4]):
        c.q_start = np.array(starts)
        o, l = c.run()
        same_bits(o[3:], want[3:])
        same_bits(l[3:], lse[3:])
    assert swab.device_status(reset=True) == 0


@pytest.mark.parametrize("case", [
    dict(n=16, own=20, h=32, hk=8, hd=128, prefix=4096),       # the own keys end long before the prefix, a launch of its own joins
    dict(n=300, own=9, h=8, hk=8, hd=64, prefix=700),          # more blocks than the GPU holds at once
    dict(n=40, own=30, h=8, hk=4, hd=128, prefix=260),         # few parts, joined by the rows kernel
    dict(n=4, own=900, h=8, hk=2, hd=64, prefix=2000)])        # own keys cut into pieces as well
def test_prefix_parts_of_the_call_before_are_never_joined(case):
    """Two inputs through one workspace in turn, back to back and in a graph: each keeps its own result."""
    n = case["n"]
    a, b = (Decode(BF16, [case["own"] + k % 3 for k in range(n)], [1] * n, case["h"], case["hk"], case["hd"], page=64,
                   prefix=case["prefix"], seed=seed) for seed in (120, 130))
    ws = torch.full((swab.band_decode_workspace(a.desc) // 4,), float("nan"), device="cuda")
    args = [(c, i32(c.table), i32(c.lens), i32(c.q_start), i32(c.ptable)) for c in (a, b)]
    out = [[torch.empty_like(a.q) for _ in range(8)], [torch.empty(a.q.shape[:2], device="cuda") for _ in range(8)]]

    def run():
        for k in range(8):
            c, table, lens, q_start, ptable = args[k % 2]
            swab.band_decode(c.desc, c.scale, c.q, c.kc, c.vc, table, lens, q_start, out[0][k], out[1][k], ws, ptable)

    run()
    torch.cuda.synchronize()
    a.check(out[0][0], out[1][0])
    b.check(out[0][1], out[1][1])
    first = [[t.clone() for t in x[:2]] for x in out]
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=stream):
        run()
    for again in range(3):
        for k in range(8):
            same_bits(out[0][k], first[0][k % 2])
            same_bits(out[1][k], first[1][k % 2])
        graph.replay()
        torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("case", [dict(lens=[40, 20], new=[2, 1]), dict(lens=[3000, 50], new=[1, 1], page=64),
                                  dict(lens=[40, 20], new=[2, 1], prefix=70),
                                  dict(lens=[20] * 16, new=[1] * 16, page=64, prefix=4096)])
def test_rows_before_the_first_request_stay_as_they_were(case, dtype):
    """The first three rows of Q and O belong to no request (q_start[0] = 3), however the lists are cut."""
    c = Decode(dtype, h=8, hk=2, hd=128, pad=3, seed=112, **case)
    want, lse = c.run()
    c.q = torch.cat((c.q[-3:], c.q[:-3])).contiguous()
    c.q_start = c.q_start + 3
    o, l = c.run()
    assert (o[:3] == 7.0).all() and (l[:3] == 7.0).all()
    n = int(c.q_start[-1])
    same_bits(o[3:n], want[:n - 3])
    same_bits(l[3:n], lse[:n - 3])


def test_decode_row_strides_and_optional_lse():
    c = Decode(BF16, [70, 9], [2, 1], 4, 2, 64, seed=102)
    want, lse = c.run()
    c.check(want, lse)
    qkv = torch.zeros(c.tokens, 8, 64, dtype=BF16, device="cuda")
    qkv[:, :4] = c.q
    out = torch.full((c.tokens, 6, 64), 5.0, dtype=BF16, device="cuda")
    d = swab.DecodeDesc(c.cache, c.tokens, 4, 2, 64, c.w, max_q=2, max_len=70, dtype=BF16, q_row_stride=512, out_row_stride=384)
    ws = torch.empty(swab.band_decode_workspace(d), dtype=torch.uint8, device="cuda")
    swab.band_decode(d, c.scale, qkv[:, :4], c.kc, c.vc, i32(c.table), i32(c.lens), i32(c.q_start), out[:, :4], None, ws)
    same_bits(out[:, :4], want)
    assert (out[:, 4:] == 5.0).all()
    same_bits(c.run(lse=False)[0], want)


@pytest.mark.parametrize("dtype", [F16, F32])
def test_compiled_calls_and_the_binding_agree(dtype, monkeypatch):
    """Every call through the compiled module and marshalled in Python: the same bits, on strided views as well."""
    B, h, hk, hd, page = 5, 4, 2, 64, 16
    turns = swab.rotary_frequencies(hd)[0].cuda()
    cache = swab.CacheDesc(B, page, 40, 6)
    x = randn((2 * B, h + 2 * hk, hd), dtype, 140)
    q, k, v = x.split([h, hk, hk], dim=1)
    desc = swab.RotaryDesc(2, B, h, hk, hd, hd, dtype=dtype)
    dec = swab.DecodeDesc(cache, 2 * B, h, hk, hd, max_q=3, dtype=dtype, q_row_stride=(h + 1) * hd)
    seen = []

    def all_calls():
        out = [torch.zeros(2 * B, n, hd, dtype=dtype, device="cuda") for n in (h, hk, h, hk, h)]
        swab.rotary(desc, turns, q, out[0], k, out[1])
        swab.rotary_bwd(desc, turns, q, out[2], k, out[3])
        lens, new = i32([17, 3, 0, 60, 9]), i32([2, 3, 1, 1, 3])
        lens_out, used, table = i32([0] * B), i32([0, 0]), torch.full((B, 6), -1, dtype=torch.int32, device="cuda")
        table[:, :4] = i32(np.arange(20).reshape(B, 4))
        slots, pos, start = i32([0] * (2 * B)), i32([0] * (2 * B)), i32([0] * (B + 1))
        swab.cache_slots(cache, lens, new, table, i32(np.arange(20, 40)), used, lens_out, used, start, slots, pos, pos0=2)
        kc, vc = randn((40, hk, page, hd), dtype, 141), randn((40, hk, page, hd), dtype, 142)
        qo = torch.zeros(2 * B, h + 1, hd, dtype=dtype, device="cuda")[:, :h]
        swab.rotary_append(swab.RotaryDesc(1, 2 * B, h, hk, hd, hd, dtype=dtype), cache, turns, q, k, v, pos, slots, qo, kc, vc)
        lse = torch.zeros(2 * B, h, device="cuda")
        need = swab.band_decode_workspace(dec)
        swab.band_decode(dec, 0.125, qo, kc, vc, table, lens_out, start, out[4], lse, torch.empty(max(need, 16), dtype=torch.uint8, device="cuda"))
        with pytest.raises(swab.SwabError, match="MISALIGNED"):
            swab.rotary(desc, turns, x.flatten()[1:1 + 2 * B * h * hd].view(2 * B, h, hd), out[0], k, out[1])
        with pytest.raises(ValueError, match="lse"):
            swab.band_decode(dec, 0.125, qo, kc, vc, table, lens_out, start, out[4], lse.flatten(), None)
        return [*out, lens_out, used, table, slots, pos, start, kc, vc, qo.contiguous(), lse]

    calls = swab.serve._load_calls()
    assert calls is not swab.serve._NoCalls
    for name in ("rotary", "rotary_bwd", "cache_slots", "rotary_append", "band_decode"):
        fn = getattr(calls, name)
        monkeypatch.setattr(calls, name, lambda *a, _f=fn, _n=name: (seen.append((_n, rc := _f(*a))), rc)[1])
    fast = all_calls()
    assert [rc for _, rc in seen] == [0, 0, 0, 0, 0, 3, -1]
    monkeypatch.setattr(swab.serve, "_calls", swab.serve._NoCalls)
    slow = all_calls()
    for a, b in zip(fast, slow):
        same_bits(a.float(), b.float())


def test_decode_fewer_rows_than_tokens():
    """Rows past `tokens` are neither read nor written."""
    c = Decode(F16, [30, 20], [3, 2], 4, 2, 64, seed=103)
    want, _ = c.run()
    c.tokens, full = 4, c.q
    c.q = full[:4].contiguous()
    c.desc = swab.DecodeDesc(c.cache, 4, 4, 2, 64, c.w, max_q=3, max_len=30, dtype=F16)
    same_bits(c.run()[0], want[:4])


def test_decode_repeats_bitwise_on_other_streams_and_two_at_once():
    a = Decode(BF16, [3000, 40], [1, 1], 8, 2, 128, prefix=500, seed=104)
    b = Decode(F16, [900] * 5, [2] * 5, 4, 4, 64, w=300, seed=105)
    wa, wb = a.run(), b.run()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(4):
        with torch.cuda.stream(s1):
            got.append((a.run(), wa))
        with torch.cuda.stream(s2):
            got.append((b.run(stream=s2), wb))
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in got:
        same_bits(o, wo)
        same_bits(l, wl)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
class Server:
    """A small serving loop: a window of 24, 4 leading global tokens, recycled blocks, everything on the GPU."""

    H, HK, HD, W, PAGE, SINK = 4, 4, 64, 24, 16, 4

    def __init__(self, batch, max_q, dtype, prefix=0, w=None, ring=True):
        self.w, self.dtype, self.batch, self.max_q = self.W if w is None else w, dtype, batch, max_q
        pinned = 1 if ring else 0
        cols = pinned + -(-(self.w + max_q - 1) // self.PAGE) + 1 if ring else 20
        pre = -(-prefix // self.PAGE)
        n_blocks = batch * cols + pre + 1
        self.cache = swab.CacheDesc(batch, self.PAGE, n_blocks, cols, ring, pinned)
        self.free = torch.randperm(n_blocks - pre, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
        self.prefix, self.ptable = prefix, torch.arange(n_blocks - pre, n_blocks, dtype=torch.int32, device="cuda")
        z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.lens, self.used, self.start = z(batch), z(2), z(batch + 1)
        self.table = z(batch, cols) - 1
        self.kc = torch.full((n_blocks, self.HK, self.PAGE, self.HD), float("nan"), dtype=dtype, device="cuda")
        self.vc = torch.full_like(self.kc, float("nan"))
        self.turns = swab.rotary_frequencies(self.HD)[0].cuda()

    def buffers(self, tokens):
        z = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
        self.rot = swab.RotaryDesc(1, tokens, self.H, self.HK, self.HD, self.HD, dtype=self.dtype)
        self.dec = swab.DecodeDesc(self.cache, tokens, self.H, self.HK, self.HD, self.w, n_sink=self.SINK, max_q=self.max_q,
                                   max_len=2000, prefix_len=self.prefix, dtype=self.dtype)
        self.n_new, self.slots, self.pos = z(self.batch), z(tokens), z(tokens)
        self.qkv = z(tokens, self.H + 2 * self.HK, self.HD, t=self.dtype)
        self.q, self.k, self.v = self.qkv.split([self.H, self.HK, self.HK], dim=1)
        self.qo, self.o = z(tokens, self.H, self.HD, t=self.dtype), z(tokens, self.H, self.HD, t=self.dtype)
        self.lse = z(tokens, self.H, t=F32)
        self.ws = torch.empty(max(1, swab.band_decode_workspace(self.dec)), dtype=torch.uint8, device="cuda")

    def step(self):
        swab.cache_slots(self.cache, self.lens, self.n_new, self.table, self.free, self.used, self.lens, self.used,
                         self.start, self.slots, self.pos, pos0=self.prefix)
        swab.rotary_append(self.rot, self.cache, self.turns, self.q, self.k, self.v, self.pos, self.slots, self.qo, self.kc,
                           self.vc)
        swab.band_decode(self.dec, self.HD ** -0.5, self.qo, self.kc, self.vc, self.table, self.lens, self.start, self.o,
                         self.lse, self.ws, self.ptable if self.prefix else None)


def full_attention(x, w, n_sink, dtype, prefix=None):
    """fp64 attention of a whole sequence x [n, heads of Q, K, V, hd], q and k rotated and rounded to the type,
    and how far a step-by-step result may be off.  The rounded q and k of the kernel and of this function may
    differ by one step (2 u) where the two sums round apart, which moves a score by at most 4 u X, X = the largest
    sum of |q| |k| times the scale, and a weighted mean by 2 (e^(4 u X) - 1) A; the weights and the result round
    to u each, the fp32 sums are far below u."""
    n, H, HK = x.shape[0], Server.H, Server.HK
    freq, _ = orc.frequencies(Server.HD)
    p0 = 0 if prefix is None else len(prefix)
    pos = p0 + np.arange(n)
    rnd = lambda y: f64(torch.tensor(y).to(dtype))  # noqa: E731
    q, k, v = rnd(orc.rotary(x[:, :H], pos, freq)), rnd(orc.rotary(x[:, H:H + HK], pos, freq)), x[:, H + HK:]
    if prefix is not None:
        pk, pv = rnd(orc.rotary(prefix[:, H:H + HK], np.arange(p0), freq)), prefix[:, H + HK:]
    out, bound, u = np.zeros((n, H, Server.HD)), np.zeros((n, H, Server.HD)), half_step(dtype)
    for i in range(n):
        keys = orc.keys_of(i, w, 0, n_sink)
        for h in range(H):
            kk, vv = k[keys, h], v[keys, h]
            if prefix is not None:
                kk, vv = np.concatenate([pk[:, h], kk]), np.concatenate([pv[:, h], vv])
            s = kk @ q[i, h] * Server.HD ** -0.5
            e = np.exp(s - s.max())
            A, X = e @ np.abs(vv) / e.sum(), (np.abs(kk) @ np.abs(q[i, h])).max() * Server.HD ** -0.5
            out[i, h] = e @ vv / e.sum()
            bound[i, h] = A * (2 * np.expm1(4 * u * X) + 2 * u) + np.abs(out[i, h]) * u + 2.0 ** -18
    return out, bound


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("graph", [False, True])
def test_steps_give_the_attention_of_the_whole_sequence(dtype, graph):
    """Requests that grow by 1 to 4 tokens a step, eager or as replays of one captured graph, against fp64
    attention over each finished sequence."""
    torch.manual_seed(5)
    B, steps = 3, 30
    s = Server(B, 4, dtype)
    s.buffers(B * 4)
    rng = np.random.default_rng(6)
    data = [randn((steps * 4, s.H + 2 * s.HK, s.HD), dtype, 200 + r) for r in range(B)]
    news = rng.integers(0, 5, (steps, B))
    s.n_new.zero_()
    s.step()                                           # warm up: no tokens
    torch.cuda.synchronize()
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.step()
    got, at = [[] for _ in range(B)], [0] * B
    for t in range(steps):
        s.n_new.copy_(i32(news[t]))
        rows = torch.cat([data[r][at[r]:at[r] + news[t][r]] for r in range(B)])
        s.qkv[:len(rows)] = rows
        g.replay() if graph else s.step()
        first = 0
        for r in range(B):
            got[r].append(s.o[first:first + news[t][r]].clone())
            first += news[t][r]
            at[r] += int(news[t][r])
    assert int(s.used[1]) == 0
    for r in range(B):
        want, bound = full_attention(f64(data[r])[:at[r]], s.w, s.SINK, dtype)
        assert (np.abs(f64(torch.cat(got[r])) - want) <= bound).all()


def test_prompt_then_steps_behind_a_shared_prefix():
    """The prefix is appended once through its own table, then three requests decode behind it."""
    dtype, P, B, n = F16, 50, 3, 9
    s = Server(B, 1, dtype, prefix=P, w=100, ring=False)
    pre = randn((P, s.H + 2 * s.HK, s.HD), dtype, 300)
    slots = i32([int(s.ptable[p // s.PAGE]) * s.PAGE + p % s.PAGE for p in range(P)])
    q, k, v = pre.split([s.H, s.HK, s.HK], dim=1)
    swab.rotary_append(swab.RotaryDesc(1, P, s.H, s.HK, s.HD, s.HD, dtype=dtype), s.cache, s.turns, None, k, v,
                       i32(np.arange(P)), slots, None, s.kc, s.vc)
    s.buffers(B)
    data = [randn((n, s.H + 2 * s.HK, s.HD), dtype, 310 + r) for r in range(B)]
    got = []
    for t in range(n):
        s.n_new.fill_(1)
        s.qkv.copy_(torch.stack([data[r][t] for r in range(B)]))
        s.step()
        got.append(s.o.clone())
    for r in range(B):
        want, bound = full_attention(f64(data[r]), 100, s.SINK, dtype, f64(pre))
        assert (np.abs(f64(torch.stack([x[r] for x in got])) - want) <= bound).all()


@pytest.mark.parametrize("batch,prefix,steps", [(3, 50, 12), (40, 300, 6)])
def test_replayed_steps_behind_a_shared_prefix(batch, prefix, steps):
    """Whole steps of one captured graph, their inputs rewritten in place and the workspace filled with noise between
    replays: the rows kernel, which starts beside the prefix kernel, sees what the calls before it have just written."""
    s = Server(batch, 4, BF16, prefix=prefix)
    pre = randn((prefix, s.H + 2 * s.HK, s.HD), BF16, 320)
    slots = i32([int(s.ptable[p // s.PAGE]) * s.PAGE + p % s.PAGE for p in range(prefix)])
    _, k, v = pre.split([s.H, s.HK, s.HK], dim=1)
    swab.rotary_append(swab.RotaryDesc(1, prefix, s.H, s.HK, s.HD, s.HD, dtype=BF16), s.cache, s.turns, None, k, v,
                       i32(np.arange(prefix)), slots, None, s.kc, s.vc)
    s.buffers(batch * 4)
    news = np.random.default_rng(7).integers(0, 5, (steps, batch))
    data = [randn((max(1, int(news[:, r].sum())), s.H + 2 * s.HK, s.HD), BF16, 330 + r) for r in range(batch)]
    s.step()                                           # warm up: no tokens
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    got, at = [[] for _ in range(batch)], [0] * batch
    for t in range(steps):
        s.n_new.copy_(i32(news[t]))
        rows = torch.cat([data[r][at[r]:at[r] + news[t][r]] for r in range(batch)])
        s.qkv[:len(rows)] = rows
        s.ws.copy_(torch.randint(0, 256, s.ws.shape, dtype=torch.uint8, device="cuda"))
        graph.replay()
        first = 0
        for r in range(batch):
            got[r].append(s.o[first:first + news[t][r]].clone())
            first += news[t][r]
            at[r] += int(news[t][r])
    assert int(s.used[1]) == 0
    for r in range(batch):
        want, bound = full_attention(f64(data[r])[:at[r]], s.w, s.SINK, BF16, f64(pre))
        assert (np.abs(f64(torch.cat(got[r])) - want) <= bound).all()


def test_last_rows_agree_with_the_banded_forward():
    """rotary, then band_attention over the sequence; the cache write and band_decode give its last rows."""
    n, h, hd, w = 200, 4, 64, 40
    x = randn((n, 3 * h, hd), F16, 400)
    q, k, v = x.split([h, h, h], dim=1)
    turns = swab.rotary_frequencies(hd)[0].cuda()
    d = swab.RotaryDesc(1, n, h, h, hd, hd, dtype=F16)
    qo, ko = torch.empty(1, h, n, hd, dtype=F16, device="cuda"), torch.empty(1, h, n, hd, dtype=F16, device="cuda")
    swab.rotary(d, turns, q, qo.transpose(1, 2), k, ko.transpose(1, 2))
    O = torch.empty(h, n, hd, dtype=F16, device="cuda")
    swab.band_attention(swab.Desc(1, h, n, hd, w, 0, dtype=F16), hd ** -0.5, qo[0], ko[0],
                        v.transpose(0, 1).contiguous(), O, torch.empty(h, n, dtype=F32, device="cuda"))
    cache = swab.CacheDesc(1, 16, 13, 13)
    kc, vc = (torch.full((13, h, 16, hd), float("nan"), dtype=F16, device="cuda") for _ in range(2))
    table = i32([np.random.default_rng(1).permutation(13)])
    slots = i32([int(table[0, j // 16]) * 16 + j % 16 for j in range(n)])
    flat = torch.empty(n, h, hd, dtype=F16, device="cuda")
    swab.rotary_append(d, cache, turns, q, k, v, i32(np.arange(n)), slots, flat, kc, vc)
    same_bits(flat, qo[0].transpose(0, 1))
    m = 5
    dd = swab.DecodeDesc(cache, m, h, h, hd, w, max_q=m, dtype=F16)
    o = torch.empty(m, h, hd, dtype=F16, device="cuda")
    ws = torch.empty(max(1, swab.band_decode_workspace(dd)), dtype=torch.uint8, device="cuda")
    swab.band_decode(dd, hd ** -0.5, flat[-m:], kc, vc, table, i32([n]), i32([0, m]), o, None, ws)
    # each side is within A (2^-11 weights + sums) + half a step of the exact value, A <= 4.5
    bound = 2 * (4.5 * (2.0 ** -11 + 2.0 ** -13) + 4.5 * 2.0 ** -11)
    assert (o.float() - O[:, -m:].transpose(0, 1).float()).abs().max().item() <= bound


@pytest.mark.parametrize("dtype", [F16, F32])
def test_decode_loop_matches_attention_over_the_sequences(dtype):
    """DecodeLoop: prompts of different lengths, then steps of 0 to 2 tokens a request, dilation and sinks."""
    B, h, hd, w, dil, sink, steps = 3, 2, 64, 9, 1, 2, 12
    loop = swab.DecodeLoop(B, h, h, hd, w, dil, sink, max_new=2, page=16, rot_dim=0, dtype=dtype)
    rng = np.random.default_rng(12)
    first, news = np.array([40, 1, 17]), rng.integers(0, 3, (steps, B))
    data = [randn((int(first[r] + news[:, r].sum()), 3 * h, hd), dtype, 500 + r) for r in range(B)]
    loop.fill(torch.cat([data[r][:first[r]] for r in range(B)]), i32(first))
    at, got = list(first), [[] for _ in range(B)]
    for t in range(steps):
        loop.n_new.copy_(i32(news[t]))
        rows = torch.cat([data[r][at[r]:at[r] + news[t][r]] for r in range(B)])
        loop.qkv[:len(rows)] = rows
        loop.step()
        pos = 0
        for r in range(B):
            got[r].append(loop.out[pos:pos + news[t][r]].clone())
            pos += news[t][r]
            at[r] += int(news[t][r])
    assert loop.lens.tolist() == [len(x) for x in data] and loop.used.tolist()[1] == 0
    for r in range(B):
        x, out = f64(data[r]), f64(torch.cat(got[r]))
        for i in range(int(first[r]), len(data[r])):
            keys = orc.keys_of(i, w, dil, sink)
            for hh in range(h):
                k, v = x[keys, h + hh], x[keys, 2 * h + hh]
                s = k @ x[i, hh] * hd ** -0.5
                p = np.exp(s - s.max())
                A = p @ np.abs(v) / p.sum()
                # weights and result rounded to the type once each, fp32 sums of at most 64 products and 12 keys
                bound = A * ((half_step(dtype) if dtype != F32 else 0) + 2.0 ** -17) + (A + 1) * half_step(dtype)
                assert (np.abs(out[i - first[r], hh] - p @ v / p.sum()) <= bound).all()


@pytest.mark.parametrize("hd", [64, 80])
def test_offsets_past_32_bits(hd):
    """A cache of more than 2^32 elements a tensor, the blocks in use at its end: the write, decode and the prefix."""
    page, hk, h, n = 128, 1, 2, 300
    n_blocks = (1 << 32) // (page * hd) + 4000
    if torch.cuda.mem_get_info()[0] < 3 * n_blocks * page * hd * 2:
        pytest.skip("not enough memory")
    kc, vc = (torch.empty(n_blocks, hk, page, hd, dtype=F16, device="cuda") for _ in range(2))
    blocks = [n_blocks - 1, n_blocks - 3900, n_blocks - 7, n_blocks - 2, n_blocks - 5]
    table, ptable = [blocks[:3]], blocks[3:]
    x = randn((n + 200, h + 2 * hk, hd), F16, 700)
    q, k, v = x.split([h, hk, hk], dim=1)
    slots = [blocks[j // page] * page + j % page for j in range(n)] + [ptable[j // page] * page + j % page for j in range(200)]
    cache = swab.CacheDesc(1, page, n_blocks, 3)
    d = swab.RotaryDesc(1, n + 200, h, hk, hd, 0, dtype=F16)
    swab.rotary_append(d, cache, None, None, k, v, None, i32(slots), None, kc, vc)
    b, o = (torch.tensor(y, device="cuda") for y in ([s // page for s in slots], [s % page for s in slots]))
    same_bits(kc[b, :, o], k)
    same_bits(vc[b, :, o], v)
    dd = swab.DecodeDesc(cache, 1, h, hk, hd, max_len=n, prefix_len=200, dtype=F16)
    out, lse = torch.empty(1, h, hd, dtype=F16, device="cuda"), torch.empty(1, h, dtype=F32, device="cuda")
    ws = torch.empty(max(1, swab.band_decode_workspace(dd)), dtype=torch.uint8, device="cuda")
    swab.band_decode(dd, hd ** -0.5, q[n - 1:n].contiguous(), kc, vc, i32(table), i32([n]), i32([0, 1]), out, lse, ws, i32(ptable))
    # the same over a small cache
    small = [c[blocks].contiguous() for c in (kc, vc)]
    del kc, vc
    sc = swab.CacheDesc(1, page, 5, 3)
    sd = swab.DecodeDesc(sc, 1, h, hk, hd, max_len=n, prefix_len=200, dtype=F16)
    want, wlse = torch.empty_like(out), torch.empty_like(lse)
    swab.band_decode(sd, hd ** -0.5, q[n - 1:n].contiguous(), *small, i32([[0, 1, 2]]), i32([n]), i32([0, 1]), want, wlse, ws, i32([3, 4]))
    same_bits(out, want)
    same_bits(lse, wlse)


def test_decode_loop_leaves_out_requests_that_add_too_much():
    """A step with more tokens than max_new for one request: its length stays, the others go on, the status is raised."""
    h, hd, w = 2, 64, 20
    loops = [swab.DecodeLoop(3, h, h, hd, w, max_new=2, page=16, rot_dim=0, dtype=F16) for _ in range(2)]
    x = randn((3, 40, 3 * h, hd), F16, 610)
    for loop in loops:
        loop.fill(x[:, :30].reshape(90, 3 * h, hd), i32([30] * 3))
        loop.n_new.copy_(i32([1, 3, 2] if loop is loops[0] else [1, 0, 2]))
        rows = torch.cat((x[0, 30:31], x[1, 30:33 if loop is loops[0] else 30], x[2, 30:32]))
        loop.qkv[:len(rows)] = rows
        loop.step()
    assert loops[0].lens.tolist() == loops[1].lens.tolist() == [31, 30, 32]
    assert loops[0].used.tolist()[1] > 0 and loops[1].used.tolist()[1] == 0
    assert swab.device_status(reset=True) == INVALID_BIT
    same_bits(loops[0].out[[0, 4, 5]], loops[1].out[[0, 1, 2]])
    # and the left-out request goes on as if nothing had been asked of it
    for loop in loops:
        loop.n_new.copy_(i32([0, 2, 1]))
        loop.qkv[:3] = torch.cat((x[1, 30:32], x[2, 32:33]))
        loop.step()
    same_bits(loops[0].out[:3], loops[1].out[:3])
    assert loops[0].lens.tolist() == [31, 32, 33] and swab.device_status(reset=True) == 0


def test_decode_loop_restarts_requests():
    """A request emptied and filled again answers as a fresh one, in the same captured step."""
    h, hd, w = 2, 64, 20
    loop = swab.DecodeLoop(2, h, h, hd, w, page=16, rot_dim=0, dtype=F16)
    x = randn((2, 60, 3 * h, hd), F16, 600)
    loop.fill(x[:, :50].reshape(100, 3 * h, hd), i32([50, 50]))
    loop.n_new.fill_(1)
    loop.qkv.copy_(x[:, 50])
    loop.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loop.step()
    for round_ in range(3):
        loop.restart([1])
        loop.fill(x[1, :8 + round_], i32([0, 8 + round_]))
        loop.qkv[1] = x[1, 8 + round_]
        graph.replay()
        assert loop.used.tolist()[1] == 0 and int(loop.lens[1]) == 9 + round_
        fresh = swab.DecodeLoop(1, h, h, hd, w, page=16, rot_dim=0, dtype=F16)
        fresh.fill(x[1, :8 + round_], i32([8 + round_]))
        fresh.n_new.fill_(1)
        fresh.qkv[0] = x[1, 8 + round_]
        fresh.step()
        same_bits(loop.out[1], fresh.out[0])
        live = loop.table[loop.table >= 0].tolist()
        assert len(set(live)) == len(live)


@pytest.mark.parametrize("name", ["tiny_fp32_n512_w32", "longformer_base_fp16_n4096_w256_d3", "train_bf16_b12_n4096_w256_g16"])
def test_run_workload_decodes(name):
    res = subprocess.run([sys.executable, "-m", "sliding_window_attention_band_gb300.run_workload", "--workload", name, "--call",
                          "decode", "--repeat", "3"], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr[-2000:]


@pytest.mark.skipif(os.environ.get("SWAB_BOUNDS_CHECK") == "1", reason="is that run")
def test_bounds_checked_build_records_nothing():
    """This file on the bounds-checked build: an access outside the call's buffers fails a status check."""
    res = subprocess.run([sys.executable, "-m", "pytest", os.path.abspath(__file__), "-m", "gpu", "-x", "-q"], cwd=ROOT,
                         env=dict(os.environ, SWAB_BOUNDS_CHECK="1"), capture_output=True, text=True, timeout=1500)
    assert res.returncode == 0, res.stdout[-3000:] + res.stderr[-2000:]
