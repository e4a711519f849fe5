"""Pins of the serving oracle (oracle/serve.py) against independent
computations: rotation matrices and torch autograd, hand-worked tables, and the
banded-attention oracle on whole sequences; planted mistakes fail."""
import numpy as np
import pytest
import torch

import oracle
from oracle import serve as orc


def rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("inter", [False, True])
def test_rotary_is_a_block_rotation(inter):
    r = rng(1)
    x, pos, f = r.standard_normal((3, 2, 10)), np.array([0, 5, -3]), np.array([1.0, 0.3, 0.01])
    y = orc.rotary(x, pos, f, 1.5, inter)
    for t in range(3):
        for k in range(3):
            a, b = (2 * k, 2 * k + 1) if inter else (k, k + 3)
            c, s = np.cos(pos[t] * f[k]), np.sin(pos[t] * f[k])
            R = 1.5 * np.array([[c, -s], [s, c]])
            np.testing.assert_allclose(y[t][:, [a, b]], x[t][:, [a, b]] @ R.T, rtol=0, atol=1e-14)
    np.testing.assert_array_equal(y[..., 6:], x[..., 6:])
    # only differences of positions enter a score
    q, k = x[:1], x[1:2]
    score = lambda p: (orc.rotary(q, [p + 9], f, 1.0, inter)[..., :6] * orc.rotary(k, [p], f, 1.0, inter)[..., :6]).sum()  # noqa: E731
    assert abs(score(0) - score(1000)) < 1e-11


@pytest.mark.parametrize("inter", [False, True])
def test_rotary_gradient_is_autograd(inter):
    x = torch.randn(4, 2, 8, dtype=torch.float64, requires_grad=True)
    g = torch.randn(4, 2, 8, dtype=torch.float64)
    f, pos = np.array([1.0, 0.1, 0.02]), np.array([3, 10, 0, 7])
    ang = torch.tensor(pos[:, None, None] * f)
    a, b = (x[..., 0:6:2], x[..., 1:6:2]) if inter else (x[..., :3], x[..., 3:6])
    one, two = 2 * (a * ang.cos() - b * ang.sin()), 2 * (b * ang.cos() + a * ang.sin())
    y = torch.cat([torch.stack([one, two], -1).flatten(-2) if inter else torch.cat([one, two], -1), x[..., 6:]], -1)
    np.testing.assert_allclose(orc.rotary(x.detach().numpy(), pos, f, 2.0, inter), y.detach().numpy(), atol=1e-14)
    (y * g).sum().backward()
    np.testing.assert_allclose(orc.rotary(g.numpy(), pos, f, 2.0, inter, backward=True), x.grad.numpy(), atol=1e-14)
    wrong = orc.rotary(g.numpy(), pos, f, 2.0, inter)                  # planted: the forward rotation
    assert np.abs(wrong - x.grad.numpy()).max() > 0.1


def test_cache_slots_by_hand():
    # pages of 16; request 0 holds 15 + 3, request 1 nothing, request 2 holds 32 + 1
    table = [[5, -1, -1], [-1, -1, -1], [7, 1, -1]]
    t, lens, used, start, slots, pos = orc.cache_slots([15, 0, 32], [3, 0, 1], table, [9, 4, 2], 1, 16, 3, tokens=6, pos0=100)
    assert t.tolist() == [[5, 4, -1], [-1, -1, -1], [7, 1, 2]]
    assert lens.tolist() == [18, 0, 33] and used.tolist() == [3, 0] and start.tolist() == [0, 3, 3, 4]
    assert slots.tolist() == [5 * 16 + 15, 4 * 16, 4 * 16 + 1, 2 * 16, -1, -1]
    assert pos.tolist() == [115, 116, 117, 132, 0, 0]
    # a list with one block: request 0 is served, request 2 is not
    t, lens, used, _, slots, _ = orc.cache_slots([15, 0, 32], [3, 0, 1], table, [9, 4], 1, 16, 3, tokens=4)
    assert lens.tolist() == [18, 0, 32] and used.tolist() == [2, 1] and slots[3] == -1 and t[2].tolist() == [7, 1, -1]
    # recycled: two columns behind one pinned, positions 48.. go back to column 1
    t, lens, used, _, slots, _ = orc.cache_slots([47], [3], [[3, 8, 6]], [], 0, 16, 3, ring=True, pinned=1, tokens=3)
    assert slots.tolist() == [6 * 16 + 15, 8 * 16, 8 * 16 + 1] and used.tolist() == [0, 0]
    # not recycled: position 48 passes the table
    _, lens, used, _, slots, _ = orc.cache_slots([47], [3], [[3, 8, 6]], [9], 0, 16, 3, tokens=3)
    assert lens.tolist() == [47] and used.tolist() == [0, 1] and slots.tolist() == [-1] * 3


def test_cache_slots_limits_by_hand():
    # at most 2 tokens a request, 4 rows: request 1 adds 3, request 3 ends at row 6; request 2 is served
    t, lens, used, start, slots, _ = orc.cache_slots([15, 0, 0, 16], [1, 3, 0, 2], [[5, -1]] * 4, [9, 4, 2], 0, 16, 2, tokens=4,
                                                     max_new=2)
    assert lens.tolist() == [16, 0, 0, 16] and used.tolist() == [0, 2] and start.tolist() == [0, 1, 4, 4, 6]
    assert slots.tolist() == [5 * 16 + 15, -1, -1, -1] and t.tolist() == [[5, -1]] * 4
    # no limits: request 1 takes block 9, request 3 block 4, rows or not
    _, lens, used, _, slots, _ = orc.cache_slots([15, 0, 0, 16], [1, 3, 0, 2], [[5, -1]] * 4, [9, 4, 2], 0, 16, 2, tokens=4)
    assert lens.tolist() == [16, 3, 0, 18] and used.tolist() == [2, 0] and slots.tolist() == [95, 144, 145, 146]


def paged(x, page, perm):
    """[n, hk, hd] -> cache blocks in the order perm."""
    n, hk, hd = x.shape
    c = np.full((len(perm), hk, page, hd), np.nan)
    for j in range(n):
        c[perm[j // page], :, j % page] = x[j]
    return c


@pytest.mark.parametrize("w,dilation", [(5, 0), (3, 2), (40, 0), (0, 0)])
def test_decode_is_the_last_rows_of_the_banded_attention(w, dilation):
    r = rng(3)
    n, h, hd, page = 37, 2, 8, 16
    q, k, v = (r.standard_normal((h, n, hd)) for _ in range(3))
    O, lse = oracle.attention_fwd(q, k, v, w, 0, dilation, 0.3)
    perm = [2, 0, 1]
    kc, vc = paged(k.transpose(1, 0, 2), page, perm), paged(v.transpose(1, 0, 2), page, perm)
    o, l, A, X = orc.decode(q[:, -4:].transpose(1, 0, 2), kc, vc, [perm], [n], [0, 4], 0.3, w, dilation)
    np.testing.assert_allclose(o.transpose(1, 0, 2), O[:, -4:], atol=1e-13)
    np.testing.assert_allclose(l.T, lse[:, -4:], atol=1e-13)
    assert (A >= np.abs(o) - 1e-15).all() and (X > 0).all()
    if w < n - 1:                                                       # planted: a window one key wider
        wrong, *_ = orc.decode(q[:, -4:].transpose(1, 0, 2), kc, vc, [perm], [n], [0, 4], 0.3, w + 1, dilation)
        assert np.abs(wrong.transpose(1, 0, 2) - O[:, -4:]).max() > 1e-4


def test_decode_sinks_and_prefix_are_a_dense_mask():
    r = rng(4)
    n, P, hd, page, w, sink = 30, 21, 8, 16, 4, 3
    k, v = r.standard_normal((P + n, 1, hd)), r.standard_normal((P + n, 1, hd))
    q = r.standard_normal((n, 2, hd))
    blocks = -(-P // page)
    kc = np.concatenate([paged(k[:P], page, [1, 0]), paged(k[P:], page, [0, 1])])
    vc = np.concatenate([paged(v[:P], page, [1, 0]), paged(v[P:], page, [0, 1])])
    o, l, _, _ = orc.decode(q, kc, vc, [[blocks, blocks + 1]], [n], [0, n], 0.5, w, 0, sink, prefix=[1, 0], prefix_len=P)
    i, j = np.arange(n)[:, None], np.arange(-P, n)[None]
    seen = (j < 0) | ((j <= i) & ((j < sink) | (i - j <= w)))
    x = torch.einsum("ihd,jd->hij", torch.tensor(q), torch.tensor(k[:, 0])) * 0.5
    x = x.masked_fill(~torch.tensor(seen), float("-inf"))
    want = torch.einsum("hij,jd->ihd", x.softmax(-1), torch.tensor(v[:, 0]))
    np.testing.assert_allclose(o, want.numpy(), atol=1e-13)
    np.testing.assert_allclose(l, x.logsumexp(-1).T.numpy(), atol=1e-13)
    # shared heads: both query heads read key head 0; a recycled table shows the same window
    ring_k, ring_v = np.full((4, 1, page, hd), np.nan), np.full((4, 1, page, hd), np.nan)
    long_k, long_v = r.standard_normal((70, 1, hd)), r.standard_normal((70, 1, hd))
    for jj in range(70):
        c = orc.column(jj // page, 3, True, 1)
        ring_k[c, :, jj % page], ring_v[c, :, jj % page] = long_k[jj], long_v[jj]
    a, la, _, _ = orc.decode(q[:2], ring_k, ring_v, [[0, 1, 2]], [70], [0, 2], 0.5, 9, 0, sink, ring=True, pinned=1)
    full = list(range(5))
    b, lb, _, _ = orc.decode(q[:2], paged(long_k, page, full), paged(long_v, page, full), [full], [70], [0, 2], 0.5, 9, 0, sink)
    np.testing.assert_array_equal(a, b)
    np.testing.assert_array_equal(la, lb)


def test_decode_rows_without_keys_and_rows_of_no_request():
    q, kc = np.ones((4, 1, 8)), np.ones((1, 1, 16, 8))
    o, l, _, _ = orc.decode(q, kc, kc, [[0]], [1], [0, 2], 1.0, 5)
    assert (o[0] == 0).all() and l[0, 0] == -np.inf and (o[1] == 1).all() and np.isnan(o[2:]).all()
