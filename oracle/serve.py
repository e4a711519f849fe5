"""fp64 oracle of the operators that answer with the banded attention: rotary
positions, block tables and slot maps, the cache write and decode over the
paged cache.  TEST INFRASTRUCTURE, like the rest of this package: numpy and
plain loops from the definitions, no code shared with the library.
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original=0, low=1.0, high=32.0):
    """(rot / 2 frequencies in radians a position, factor on cos and sin)."""
    k = np.arange(rot // 2)
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = np.exp(-2.0 * k / rot * math.log(base))
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        def pair(turns):
            return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        first, last = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
        slow = np.clip((k - first) / max(last - first, 1e-3), 0, 1)
        return f * (slow / factor + (1 - slow)), 0.1 * math.log(factor) + 1
    if scaling == "bands":
        keep = np.clip((original * f / (2 * math.pi) - low) / (high - low), 0, 1)
        return f * (keep + (1 - keep) / factor), 1.0
    return f, 1.0


def rotary(x, pos, freq, scale=1.0, interleaved=False, backward=False):
    """x [..., heads, hd] at positions pos [...]: the pairs turned as complex numbers."""
    y = np.array(x, dtype=np.float64)
    rot = 2 * len(freq)
    if rot == 0:
        return y
    a = np.arange(rot // 2)
    one, two = (2 * a, 2 * a + 1) if interleaved else (a, a + rot // 2)
    turn = scale * np.exp((-1j if backward else 1j) * np.asarray(pos, np.float64)[..., None] * freq)
    z = (y[..., one] + 1j * y[..., two]) * turn[..., None, :]
    y[..., one], y[..., two] = z.real, z.imag
    return y


def column(block, cols, ring, pinned):
    """Table column of block number `block` of a request; None past a table that is not recycled."""
    if block < cols:
        return block
    return pinned + (block - pinned) % (cols - pinned) if ring else None


def cache_slots(lens, new, table, free, used, page, cols, ring=False, pinned=0, tokens=0, pos0=0, n_blocks=1 << 30,
                max_new=0):
    """One token at a time: (table, lens_out, used_out, q_start, slots, pos)."""
    table = np.array(table)
    lens = [max(int(x), 0) for x in lens]
    new = [max(int(x), 0) for x in new]
    used = max(int(used), 0)
    start, lens_out, slots, pos = [0], [], [], []
    asked, taken, missing = used, used, 0
    for r, (a, m) in enumerate(zip(lens, new)):
        start.append(start[-1] + m)
        have, want = min(-(-a // page), cols), -(-(a + m) // page)
        too_many = 0 < max_new < m
        too_long = too_many or (not ring and want > cols)
        need = 0 if too_long else min(want, cols) - have
        asked += need
        no_rows = max_new > 0 and m > 0 and start[-1] > tokens
        ok = not too_long and not no_rows and (need == 0 or asked <= len(free))
        if not ok:
            missing += max(want - cols if too_long else need, 1)
            lens_out.append(a)
            slots += [-1] * m
            pos += [a + k + pos0 for k in range(m)]
            continue
        for k in range(need):
            table[r, have + k] = free[asked - need + k]
        if need:
            taken = asked
        lens_out.append(a + m)
        # a block is recycled as a whole: its column belongs to the last block number that maps to it
        newest = {column(b, cols, ring, pinned): b for b in range(-(-(a + m) // page))}
        for j in range(a, a + m):
            c = column(j // page, cols, ring, pinned)
            latest = newest.get(c, j // page)
            slots.append(int(table[r, c]) * page + j % page if latest == j // page else -1)
            pos.append(j + pos0)
    slots = (slots + [-1] * max(0, tokens - len(slots)))[:tokens]
    pos = (pos + [0] * max(0, tokens - len(pos)))[:tokens]
    return table, np.array(lens_out), np.array([taken, missing]), np.array(start), np.array(slots), np.array(pos)


def keys_of(i, w, dilation, n_sink):
    """Positions the query at position i attends to."""
    s = dilation + 1
    band = [j for j in range(i, max(i - w * s, 0) - 1, -s) if j >= n_sink] if i >= 0 else []
    return list(range(0, min(n_sink, i + 1))) + band[::-1]


def decode(q, kc, vc, table, lens, q_start, scale, w, dilation=0, n_sink=0, ring=False, pinned=0, prefix=None,
           prefix_len=0):
    """q [T, h, hd], kc / vc [n_blocks, hk, page, hd].  Returns O [T, h, hd] (rows of no request NaN), lse
    [T, h], and for tolerances: A = sum p |v| [T, h, hd] and X = the largest sum |q| |k| * |scale| [T, h]."""
    q, kc, vc = (np.asarray(x, np.float64) for x in (q, kc, vc))
    T, h, hd = q.shape
    n_blocks, hk, page, _ = kc.shape
    group, cols = h // hk, np.asarray(table).shape[1]
    O, A = np.full((T, h, hd), np.nan), np.full((T, h, hd), np.nan)
    lse, X = np.full((T, h), np.nan), np.zeros((T, h))

    def line(block, off):
        return (int(block), off) if 0 <= block < n_blocks else None

    shared = [line(prefix[p // page], p % page) for p in range(prefix_len)]
    for r in range(len(lens)):
        L, m = max(int(lens[r]), 0), int(q_start[r + 1]) - int(q_start[r])
        for a in range(m):
            t = int(q_start[r]) + a
            if t >= T:
                continue
            lines = list(shared)
            last = (L - 1) // page
            for j in keys_of(L - m + a, w, dilation, n_sink):
                c = column(j // page, cols, ring, pinned)
                if c is None or (ring and j // page >= pinned and j // page <= last - (cols - pinned)):
                    continue
                lines.append(line(table[r][c], j % page))
            lines = [x for x in lines if x is not None]
            if not lines:
                O[t], A[t], lse[t] = 0.0, 0.0, -np.inf
                continue
            b, o = np.array([x[0] for x in lines]), np.array([x[1] for x in lines])
            for hh in range(h):
                k, v = kc[b, hh // group, o], vc[b, hh // group, o]
                x = k @ q[t, hh] * scale
                mx = x.max()
                p = np.exp(x - mx)
                z = p.sum()
                O[t, hh], A[t, hh] = p @ v / z, p @ np.abs(v) / z
                lse[t, hh] = mx + math.log(z)
                X[t, hh] = (np.abs(k) @ np.abs(q[t, hh])).max() * abs(scale)
    return O, lse, A, X
