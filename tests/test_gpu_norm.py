"""Norms of queries and keys with rotary positions, their gradient and the fused
cache write against the fp64 oracle, on the GPU.

Tolerances, set before the first run.  A stored value is off by at most half a
step of its type.  A sum of squares is made of at most 16 sums in a row in a lane
and 5 exchanges, of positive terms: within 2^-19 relatively (32 roundings), its
root's inverse within half of that; weight, factor and rotation round a few times
more (2^-21 of |x_a| + |x_b|, as for rotary): together below E = 2^-18 (|y_a| +
|y_b|), y the normed values of a pair.  Backward: g within 2^-21 of its pair, a
product sum of hd terms within 2^-18 of the sum of its magnitudes, so
    |dx - dx'| <= 2^-17 r (|g v| + |x| r^2 mean |g v x|),  |g| the pair's sum,
and a weight's gradient, of R rows, is summed in at least 8 strands (of R / 8 + 1
terms, then at most 64 + 32 + 32 of these): (R / 8 + 136) 2^-24 + 2^-18 of the sum
of magnitudes.
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import sliding_window_attention_band_gb300 as swab
from oracle import quant, serve as orc
from test_gpu_serve import BF16, F16, F32, INVALID_BIT, ROOT, f64, frequencies, half_step, i32, randn, same_bits, smallest_half_step

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("device_status_guard")]


def pair_sums(a, rot, inter):
    """|value| of a channel plus that of its pair's other one."""
    a = np.abs(a)
    out = a.copy()
    k = np.arange(rot // 2)
    one, two = (2 * k, 2 * k + 1) if inter else (k, k + rot // 2)
    out[..., one] = out[..., two] = a[..., one] + a[..., two]
    return out


def assert_within(got, ref, bound, what=""):
    bound = np.broadcast_to(bound, ref.shape)
    err = np.abs(f64(got) - ref)
    worst = np.unravel_index(np.argmax(err - bound), err.shape)
    assert (err <= bound).all(), (what, worst, float(err[worst]), float(bound[worst]))


def stored(ref, bound, dtype):
    return bound + (np.abs(ref) + bound) * half_step(dtype) + smallest_half_step(dtype)


def check_forward(got, x, w, pos, freq, scale, inter, dtype, eps, offset):
    ref = quant.norm_rotary(f64(x), w, pos, freq, scale, inter, eps, offset)
    y = quant.norm(f64(x), w, eps, offset)
    assert_within(got, ref, stored(ref, 2.0 ** -18 * max(1.0, abs(scale)) * pair_sums(y, 2 * len(freq), inter), dtype))


def check_gradient(dx, g, x, w, pos, freq, scale, inter, dtype, eps, offset):
    x64, g64, hd = f64(x), f64(g), x.shape[-1]
    ref, _ = quant.norm_rotary_bwd(g64, x64, w, pos, freq, scale, inter, eps, offset)
    r = 1 / np.sqrt((x64 ** 2).mean(-1, keepdims=True) + eps)
    gv = pair_sums(g64, 2 * len(freq), inter) * max(1.0, abs(scale)) * (1.0 if w is None else np.abs(w + offset))
    mag = r * (gv + np.abs(x64) * r ** 2 * (gv * np.abs(x64)).sum(-1, keepdims=True) / hd)
    assert_within(dx, ref, stored(ref, 2.0 ** -17 * mag, dtype))


def check_weight(dw, g, x, w, pos, freq, scale, inter, eps, offset):
    x64, g64, hd = f64(x), f64(g), x.shape[-1]
    _, ref = quant.norm_rotary_bwd(g64, x64, w, pos, freq, scale, inter, eps, offset)
    r = 1 / np.sqrt((x64 ** 2).mean(-1, keepdims=True) + eps)
    mag = (pair_sums(g64, 2 * len(freq), inter) * max(1.0, abs(scale)) * np.abs(x64) * r).reshape(-1, hd)
    assert_within(dw, ref, ((len(mag) / 8 + 136) * 2.0 ** -24 + 2.0 ** -18) * mag.sum(0), "weight")


CASES = [  # b, n, h, hk, hd, rot, interleaved, scaling, offset, weighted
    (1, 1, 1, 0, 64, 64, False, "none", 0.0, True),
    (1, 1, 4, 2, 64, 64, True, "linear", 1.0, True),
    (2, 33, 5, 1, 80, 20, False, "yarn", 0.0, True),
    (2, 33, 5, 1, 80, 20, True, "bands", 1.0, True),
    (3, 70, 12, 4, 128, 128, False, "yarn", 0.0, True),
    (3, 70, 12, 4, 128, 64, True, "ntk", 0.0, False),
    (3, 70, 12, 4, 128, 64, False, "none", 0.0, True),
    (1, 257, 3, 3, 96, 96, False, "none", 0.0, True),
    (1, 57, 3, 3, 96, 48, False, "none", 0.0, True),
    (1, 9, 2, 2, 512, 510, False, "none", 0.0, True),
    (1, 9, 2, 2, 512, 512, True, "none", 0.0, True),
    (1, 9, 2, 2, 256, 256, False, "none", 0.0, True),
    (1, 700, 2, 1, 64, 32, False, "none", 0.0, True),
    (2, 7, 3, 1, 64, 0, False, "none", 0.0, True),
    (1, 12, 3, 1, 64, 2, True, "none", 0.0, False),
    (1, 5, 3, 1, 8, 8, False, "none", 0.0, True),
    (1, 5, 3, 1, 24, 16, False, "none", 0.0, True),
    (1, 3, 700, 300, 64, 64, False, "none", 0.0, True),      # more heads than a block lists
    (1, 1300, 1, 0, 512, 512, True, "none", 0.0, True),      # the widest table
]


def build(case, dtype, seed=1):
    b, n, h, hk, hd, rot, inter, scaling, offset, weighted = case
    turns, freq, scale = frequencies(rot, scaling)
    q, k = randn((b, n, h, hd), dtype, seed), randn((b, n, max(hk, 1), hd), dtype, seed + 1, 3.0)
    q[0, 0, 0] = 0.0                                             # a row of zeros
    if n > 2:
        k[0, 1, 0] = randn((hd,), dtype, seed + 2, 1e-3)         # eps counts
        q[0, 2, 0] = randn((hd,), dtype, seed + 3, 200.0)
    wq, wk = ((randn((hd,), dtype, seed + s, 0.3) + (0.0 if offset else 1.0)).to(dtype) if weighted else None for s in (4, 5))
    pos = np.random.default_rng(3).integers(0, 1_000_000, (b, n))
    return turns, freq, scale, q, k, wq, wk, pos


def w64(w):
    return None if w is None else f64(w)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("case", CASES)
def test_norm_rotary_matches_the_oracle(case, dtype):
    b, n, h, hk, hd, rot, inter, scaling, offset, weighted = case
    turns, freq, scale, q, k, wq, wk, pos = build(case, dtype)
    d, eps = swab.RotaryDesc(b, n, h, hk, hd, rot, inter, scale, dtype=dtype), 1e-5
    qo, ko = torch.empty_like(q), torch.full_like(k, 3.0)
    swab.norm_rotary(d, swab.NormDesc(eps, offset), turns, q, qo, k if hk else None, ko if hk else None, wq, wk if hk else None, pos=i32(pos))
    check_forward(qo, q, w64(wq), pos, freq, scale, inter, dtype, eps, offset)
    if hk:
        check_forward(ko, k, w64(wk), pos, freq, scale, inter, dtype, eps, offset)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("case", CASES)
def test_gradient_matches_the_oracle(case, dtype):
    b, n, h, hk, hd, rot, inter, scaling, offset, weighted = case
    turns, freq, scale, q, k, wq, wk, pos = build(case, dtype, 11)
    gq, gk = randn(q.shape, dtype, 21), randn(k.shape, dtype, 22)
    d, eps = swab.RotaryDesc(b, n, h, hk, hd, rot, inter, scale, dtype=dtype), 1e-2
    dq, dk = torch.empty_like(q), torch.full_like(k, 3.0)
    dwq, dwk = (torch.full((hd,), 7.0, device="cuda") if weighted else None for _ in range(2))
    ws = torch.full((swab.norm_rotary_bwd_workspace(d),), 0xff, dtype=torch.uint8, device="cuda")     # NaN before the call
    keys = (gk, k, dk) if hk else (None, None, None)
    swab.norm_rotary_bwd(d, swab.NormDesc(eps, offset), turns, gq, q, dq, *keys, wq, wk if hk else None, dwq, dwk if hk else None, ws,
                         pos=i32(pos))
    check_gradient(dq, gq, q, w64(wq), pos, freq, scale, inter, dtype, eps, offset)
    if hk:
        check_gradient(dk, gk, k, w64(wk), pos, freq, scale, inter, dtype, eps, offset)
    if weighted:
        check_weight(dwq, gq, q, w64(wq), pos, freq, scale, inter, eps, offset)
        if hk:
            check_weight(dwk, gk, k, w64(wk), pos, freq, scale, inter, eps, offset)
        else:
            assert (dwk == 7.0).all()


def test_long_weight_sums():
    """Many rows: every block of the grid has a share."""
    case = (1, 3001, 16, 2, 64, 64, False, "none", 0.0, True)
    b, n, h, hk, hd, rot, inter, *_ = case
    turns, freq, scale, q, k, wq, wk, pos = build(case, BF16, 31)
    gq, gk = randn(q.shape, BF16, 33), randn(k.shape, BF16, 34)
    d = swab.RotaryDesc(b, n, h, hk, hd, rot, dtype=BF16)
    runs = []
    for _ in range(2):
        dq, dk, dwq, dwk = torch.empty_like(q), torch.empty_like(k), *(torch.empty(hd, device="cuda") for _ in range(2))
        ws = torch.empty(swab.norm_rotary_bwd_workspace(d), dtype=torch.uint8, device="cuda")
        swab.norm_rotary_bwd(d, swab.NormDesc(), turns, gq, q, dq, gk, k, dk, wq, wk, dwq, dwk, ws, pos=i32(pos))
        runs.append((dq, dk, dwq, dwk))
    check_weight(runs[0][2], gq, q, f64(wq), pos, freq, scale, inter, 1e-6, 0.0)
    check_weight(runs[0][3], gk, k, f64(wk), pos, freq, scale, inter, 1e-6, 0.0)
    check_gradient(runs[0][0], gq, q, f64(wq), pos, freq, scale, inter, BF16, 1e-6, 0.0)
    for a, b_ in zip(*runs):
        same_bits(a, b_)                                          # the sums' order is fixed


def test_gradient_against_differences():
    """fp32: (f(x + h e) - f(x - h e)) / 2 h of sum(g y) against dx and dw, some channels."""
    n, h, hd = 3, 2, 64
    turns, _, _ = frequencies(hd, "none")
    d, nd = swab.RotaryDesc(1, n, h, 0, hd, hd, dtype=F32), swab.NormDesc(1e-3)
    q, g, w = randn((1, n, h, hd), F32, 41), randn((1, n, h, hd), F32, 42), randn((hd,), F32, 43) + 1.0
    dq, dw = torch.empty_like(q), torch.empty(hd, device="cuda")
    ws = torch.empty(swab.norm_rotary_bwd_workspace(d), dtype=torch.uint8, device="cuda")
    swab.norm_rotary_bwd(d, nd, turns, g, q, dq, wq=w, dwq=dw, workspace=ws)

    def f(x, w_):
        y = torch.empty_like(x)
        swab.norm_rotary(d, nd, turns, x, y, wq=w_)
        return float((y.double() * g.double()).sum())

    step = 2.0 ** -6
    # (f's fp32 rounding, 2^-22 of each of 384 terms of size about 1, over 2 h = 2^-5: below 4e-3; curvature h^2)
    for i, head, c in ((0, 0, 0), (1, 1, 33), (2, 0, 63), (0, 1, 31)):
        e = torch.zeros_like(q)
        e[0, i, head, c] = step
        assert abs((f(q + e, w) - f(q - e, w)) / (2 * step) - float(dq[0, i, head, c])) < 1e-2
    for c in (0, 31, 32, 63):
        e = torch.zeros_like(w)
        e[c] = step
        assert abs((f(q, w + e) - f(q, w - e)) / (2 * step) - float(dw[c])) < 1e-2


@pytest.mark.parametrize("inter", [False, True])
def test_strided_views_and_in_place(inter):
    """Heads out of a merged projection, head-major outputs, an output over its input: the same bits as contiguous calls."""
    b, n, h, hk, hd = 2, 19, 4, 2, 64
    turns, freq, scale = frequencies(hd, "none")
    x, gx = randn((b, n, h + 2 * hk, hd), BF16, 51), randn((b, n, h + 2 * hk, hd), BF16, 52)
    q, k, _ = x.split([h, hk, hk], dim=2)
    gq, gk, _ = gx.split([h, hk, hk], dim=2)
    w = [randn((hd,), BF16, 53 + s) for s in range(2)]
    d, nd = swab.RotaryDesc(b, n, h, hk, hd, hd, inter, dtype=BF16), swab.NormDesc()
    qc, kc = q.contiguous(), k.contiguous()
    want = [torch.empty_like(qc), torch.empty_like(kc), torch.empty_like(qc), torch.empty_like(kc)]
    swab.norm_rotary(d, nd, turns, qc, want[0], kc, want[1], *w)
    ws = torch.empty(swab.norm_rotary_bwd_workspace(d), dtype=torch.uint8, device="cuda")
    dw = [torch.empty(hd, device="cuda") for _ in range(4)]
    swab.norm_rotary_bwd(d, nd, turns, gq.contiguous(), qc, want[2], gk.contiguous(), kc, want[3], *w, dw[0], dw[1], ws)
    # head-major outputs
    qo, ko = (torch.empty(b, m, n, hd, dtype=BF16, device="cuda").transpose(1, 2) for m in (h, hk))
    swab.norm_rotary(d, nd, turns, q, qo, k, ko, *w)
    same_bits(qo, want[0])
    same_bits(ko, want[1])
    swab.norm_rotary_bwd(d, nd, turns, gq, q, qo, gk, k, ko, *w, dw[2], dw[3], ws)
    same_bits(qo, want[2])
    same_bits(ko, want[3])
    same_bits(dw[0], dw[2])
    same_bits(dw[1], dw[3])
    # in place: dQ over dQo, dK over K, then the forward over its own input
    g2, x2 = gx.clone(), x.clone()
    swab.norm_rotary_bwd(d, nd, turns, g2[:, :, :h], q, g2[:, :, :h], gk, x2[:, :, h:h + hk], x2[:, :, h:h + hk], *w, dw[2], dw[3], ws)
    same_bits(g2[:, :, :h], want[2])
    same_bits(x2[:, :, h:h + hk], want[3])
    same_bits(dw[0], dw[2])
    same_bits(g2[:, :, h:], gx[:, :, h:])
    x3 = x.clone()
    swab.norm_rotary(d, nd, turns, x3[:, :, :h], x3[:, :, :h], x3[:, :, h:h + hk], x3[:, :, h:h + hk], *w)
    same_bits(x3[:, :, :h], want[0])
    same_bits(x3[:, :, h:h + hk], want[1])
    same_bits(x3[:, :, h + hk:], x[:, :, h + hk:])
    # a gradient broadcast over the sequences (stride 0) is read as it is
    one = gq[:1].expand(b, -1, -1, -1)
    a, b_ = torch.empty_like(qc), torch.empty_like(qc)
    swab.norm_rotary_bwd(d, nd, turns, one, q, a, gk, k, ko, *w, dw[0], dw[1], ws)
    swab.norm_rotary_bwd(d, nd, turns, one.contiguous(), q, b_, gk, k, ko, *w, dw[2], dw[3], ws)
    same_bits(a, b_)
    same_bits(dw[0], dw[2])


def test_one_of_the_weights_gradients_and_none():
    b, n, h, hk, hd = 1, 40, 3, 2, 64
    turns, *_ = frequencies(hd, "none")
    q, k, gq, gk = randn((b, n, h, hd), F16, 61), randn((b, n, hk, hd), F16, 62), randn((b, n, h, hd), F16, 63), randn((b, n, hk, hd), F16, 64)
    w = [randn((hd,), F16, 65 + s) for s in range(2)]
    d, nd = swab.RotaryDesc(b, n, h, hk, hd, hd, dtype=F16), swab.NormDesc()
    out = []
    for have in ((1, 1), (1, 0), (0, 1), (0, 0)):
        dq, dk = torch.empty_like(q), torch.empty_like(k)
        dw = [torch.full((hd,), 7.0, device="cuda") for _ in range(2)]
        ws = torch.empty(swab.norm_rotary_bwd_workspace(d), dtype=torch.uint8, device="cuda") if any(have) else None
        swab.norm_rotary_bwd(d, nd, turns, gq, q, dq, gk, k, dk, *w, *(x if y else None for x, y in zip(dw, have)), ws)
        out.append((dq, dk, *dw))
    for got, have in zip(out[1:], ((1, 0), (0, 1), (0, 0))):
        same_bits(got[0], out[0][0])
        same_bits(got[1], out[0][1])
        for s in range(2):
            if have[s]:
                same_bits(got[2 + s], out[0][2 + s])
            else:
                assert (got[2 + s] == 7.0).all()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_rows_that_are_not_finite(dtype):
    """A NaN or infinity stays in its row; a row whose squares pass fp32's range gives 0."""
    n, hd = 12, 64
    turns, freq, scale = frequencies(hd, "none")
    q = randn((1, n, 2, hd), dtype, 71)
    clean = torch.empty_like(q)
    d, nd = swab.RotaryDesc(1, n, 2, 0, hd, hd, dtype=dtype), swab.NormDesc()
    swab.norm_rotary(d, nd, turns, q, clean)
    q[0, 3, 1, 5], q[0, 7, 0, 60] = float("nan"), float("inf")
    if dtype is not F16:
        q[0, 9, 0] = 1e30
    y = torch.empty_like(q)
    swab.norm_rotary(d, nd, turns, q, y)
    assert y[0, 3, 1].isnan().all() and y[0, 7, 0, [60, 28]].isnan().all()
    rest = torch.ones(n, 2, dtype=torch.bool)
    rest[3, 1] = rest[7, 0] = False
    if dtype is not F16:
        assert (y[0, 9, 0] == 0).all()
        rest[9, 0] = False
    same_bits(y[0][rest], clean[0][rest])


@pytest.mark.parametrize("hd,rot", [(64, 64), (80, 20)])                 # rows on lane groups, a warp a row
@pytest.mark.parametrize("with_q", [False, True])
def test_gradient_of_a_key_weight_without_keys(hd, rot, with_q):
    """A sum over no rows is 0, not what the buffer held."""
    turns, *_ = frequencies(rot, "none")
    d, q, g, w = swab.RotaryDesc(1, 9, 3, 0, hd, rot, dtype=F16), *(randn(s, F16, 75) for s in ((1, 9, 3, hd), (1, 9, 3, hd), (hd,)))
    ws = torch.empty(swab.norm_rotary_bwd_workspace(d), dtype=torch.uint8, device="cuda")
    dwq, ref = (torch.full((hd,), 7.0, device="cuda") for _ in range(2))
    swab.norm_rotary_bwd(d, swab.NormDesc(), turns, g, q, torch.empty_like(q), wq=w, dwq=ref, workspace=ws)
    for wk in (w, None):
        dwk = torch.full((hd,), 7.0, device="cuda")
        swab.norm_rotary_bwd(d, swab.NormDesc(), turns, g, q, torch.empty_like(q), wq=w, wk=wk, dwq=dwq if with_q else None, dwk=dwk,
                             workspace=ws)
        assert (dwk == 0.0).all()
    if with_q:
        same_bits(dwq, ref)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("hd,rot", [(64, 64), (80, 20)])                 # rows on lane groups, a warp a row
def test_gradient_of_rows_past_the_range(hd, rot, dtype):
    """A row whose squares pass fp32's range has the output 0 and the gradient 0, also where the products with it pass the
    range, and adds nothing to the weights'; a NaN stays in its row."""
    turns, *_ = frequencies(rot, "none")
    q, g, w = randn((1, 8, 2, hd), dtype, 76), randn((1, 8, 2, hd), dtype, 77), randn((hd,), dtype, 78).abs() + 1.0
    g[0, 3] = 1.0
    d, nd = swab.RotaryDesc(1, 8, 2, 0, hd, rot, dtype=dtype), swab.NormDesc()
    ws = torch.empty(swab.norm_rotary_bwd_workspace(d), dtype=torch.uint8, device="cuda")
    out = []
    for far in (0.0, 1e30, 1e38):
        x = q.clone()
        x[0, 3] = far
        dq, dw = torch.full_like(q, 7.0), torch.full((hd,), 7.0, device="cuda")
        swab.norm_rotary_bwd(d, nd, turns, g, x, dq, wq=w, dwq=dw, workspace=ws)
        out.append((dq, dw))
    for dq, dw in out[1:]:
        assert (dq[0, 3] == 0.0).all()
        dq[0, 3] = out[0][0][0, 3]
        same_bits(dq, out[0][0])
        same_bits(dw, out[0][1])
    x[0, 3], x[0, 5, 1, 7] = 0.0, float("nan")
    swab.norm_rotary_bwd(d, nd, turns, g, x, dq, wq=w, dwq=dw, workspace=ws)
    assert dq[0, 5, 1].isnan().all() and dw.isnan().all()
    dq[0, 5, 1] = out[0][0][0, 5, 1]
    same_bits(dq, out[0][0])


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("case", [(4, 2, 64, 64, False, 16), (3, 1, 128, 64, True, 64), (6, 6, 96, 96, False, 32), (2, 2, 80, 20, False, 16),
                                  (1, 1, 64, 0, False, 128)])
def test_append_writes_normed_keys(case, dtype):
    """Rows of the cache: K as norm_rotary gives it, V as it is; slots of -1 and the other rows stay."""
    h, hk, hd, rot, inter, page = case
    T, blocks = 23, 5
    turns, freq, scale = frequencies(rot, "none")
    q, k, v = randn((T, h + 2 * hk, hd), dtype, 81).split([h, hk, hk], dim=1)
    w = [randn((hd,), dtype, 82 + s) for s in range(2)]
    pos = np.random.default_rng(4).integers(0, 9000, T)
    slots = np.random.default_rng(5).permutation(blocks * page)[:T]
    slots[[2, 11]] = -1
    d, nd = swab.RotaryDesc(1, T, h, hk, hd, rot, inter, dtype=dtype), swab.NormDesc(1e-5, 0.5)
    cache = swab.CacheDesc(1, page, blocks, blocks)
    kc, vc = randn((blocks, hk, page, hd), dtype, 84), randn((blocks, hk, page, hd), dtype, 85)
    before = kc.clone(), vc.clone()
    qo = torch.empty(T, h, hd, dtype=dtype, device="cuda")
    swab.norm_rotary_append(d, nd, cache, turns, q, k, v, i32(pos), i32(slots), qo, kc, vc, *w)
    check_forward(qo[None], q[None], f64(w[0]), pos[None], freq, scale, inter, dtype, 1e-5, 0.5)
    live = np.flatnonzero(slots >= 0)
    blk, off = torch.tensor(slots[live] // page).cuda(), torch.tensor(slots[live] % page).cuda()
    check_forward(kc[blk, :, off][None], k[live][None], f64(w[1]), pos[live][None], freq, scale, inter, dtype, 1e-5, 0.5)
    same_bits(vc[blk, :, off], v[live])
    for now, then in zip((kc, vc), before):
        then[blk, :, off] = now[blk, :, off]
        same_bits(now, then)
    # without queries: the same rows
    k2, v2 = before[0].clone(), before[1].clone()
    swab.norm_rotary_append(d, nd, cache, turns, None, k, v, i32(pos), i32(slots), None, k2, v2, None, w[1])
    same_bits(k2, kc)
    same_bits(v2, vc)
    # a slot outside the cache is flagged, its row not written
    slots[5] = blocks * page
    swab.norm_rotary_append(d, nd, cache, turns, q, k, v, i32(pos), i32(slots), qo, kc, vc, *w)
    assert swab.device_status(reset=True) == INVALID_BIT
    same_bits(kc, k2)


def test_streams_graphs_and_two_at_once():
    """The same bits on a stream of its own, replayed from a graph, and with another call of other inputs beside it."""
    b, n, h, hk, hd = 2, 300, 8, 2, 128
    turns, *_ = frequencies(hd, "none")
    d, nd = swab.RotaryDesc(b, n, h, hk, hd, hd, dtype=BF16), swab.NormDesc()

    def state(seed):
        q, k, gq, gk = randn((b, n, h, hd), BF16, seed), randn((b, n, hk, hd), BF16, seed + 1), randn((b, n, h, hd), BF16, seed + 2), randn((b, n, hk, hd), BF16, seed + 3)
        w = [randn((hd,), BF16, seed + 4 + s) for s in range(2)]
        out = [torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(q), torch.zeros_like(k), torch.zeros(hd, device="cuda"), torch.zeros(hd, device="cuda")]
        ws = torch.empty(swab.norm_rotary_bwd_workspace(d), dtype=torch.uint8, device="cuda")

        def call(stream=None):
            swab.norm_rotary(d, nd, turns, q, out[0], k, out[1], *w, stream=stream)
            swab.norm_rotary_bwd(d, nd, turns, gq, q, out[2], gk, k, out[3], *w, out[4], out[5], ws, stream=stream)
        return call, out

    calls = [state(s) for s in (91, 101)]
    want = []
    for call, out in calls:
        call()
        want.append([x.clone() for x in out])
        [x.zero_() for x in out]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        for (call, _), s in zip(calls, streams):
            call(s)
    torch.cuda.synchronize()
    for (_, out), ref in zip(calls, want):
        for x, y in zip(out, ref):
            same_bits(x, y)
            x.zero_()
    graphs = []
    for call, _ in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for s, g in zip(streams, graphs):
        with torch.cuda.stream(s):
            for _ in range(3):
                g.replay()
    torch.cuda.synchronize()
    for (_, out), ref in zip(calls, want):
        for x, y in zip(out, ref):
            same_bits(x, y)


@pytest.mark.parametrize("dtype", [F16, F32])
def test_compiled_calls_and_the_binding_agree(dtype, monkeypatch):
    T, h, hk, hd, page = 10, 4, 2, 64, 16
    turns = swab.rotary_frequencies(hd)[0].cuda()
    cache, d, nd = swab.CacheDesc(1, page, 4, 4), swab.RotaryDesc(2, T // 2, h, hk, hd, hd, dtype=dtype), swab.NormDesc(1e-5, 1.0)
    x, g = randn((T, h + 2 * hk, hd), dtype, 111), randn((T, h + 2 * hk, hd), dtype, 112)
    (q, k, v), (gq, gk, _) = x.split([h, hk, hk], dim=1), g.split([h, hk, hk], dim=1)
    w, pos = [randn((hd,), dtype, 113 + s) for s in range(2)], i32(np.arange(T) * 7)
    ws = torch.empty(swab.norm_rotary_bwd_workspace(d), dtype=torch.uint8, device="cuda")

    def all_calls():
        out = [torch.zeros(T, m, hd, dtype=dtype, device="cuda") for m in (h, hk, h, hk, h)]
        dw, kv = [torch.zeros(hd, device="cuda") for _ in range(2)], [torch.zeros(4, hk, page, hd, dtype=dtype, device="cuda") for _ in range(2)]
        swab.norm_rotary(d, nd, turns, q, out[0], k, out[1], *w, pos=pos)
        swab.norm_rotary_bwd(d, nd, turns, gq, q, out[2], gk, k, out[3], *w, *dw, ws, pos=pos)
        swab.norm_rotary_append(d, nd, cache, turns, q, k, v, pos, pos % 64, out[4], *kv, *w)
        with pytest.raises(swab.SwabError, match="INVALID"):
            swab.norm_rotary(d, swab.NormDesc(0.0), turns, q, out[0], k, out[1], *w)
        return [*out, *dw, *kv]

    got = all_calls()
    monkeypatch.setattr(swab.serve, "_calls", swab.serve._NoCalls)
    for a, b in zip(got, all_calls()):
        assert a.abs().sum() > 0
        same_bits(a, b)


@pytest.mark.skipif(os.environ.get("SWAB_BOUNDS_CHECK") == "1", reason="is that run")
def test_bounds_checked_build_records_nothing():
    res = subprocess.run([sys.executable, "-m", "pytest", os.path.abspath(__file__), "-m", "gpu", "-x", "-q"], cwd=ROOT,
                         env=dict(os.environ, SWAB_BOUNDS_CHECK="1"), capture_output=True, text=True, timeout=1500)
    assert res.returncode == 0, res.stdout[-3000:] + res.stderr[-2000:]
