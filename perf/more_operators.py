"""More serving and training operators, measured one call at a time.

What a model with normed queries and keys, and a server with a cache in 4 bits,
need around the banded attention:

* ``norm``    -- RMS norms of queries and keys, a head at a time, and rotary
                 positions in the same pass (and the gradient);
* ``append``  -- the same fused with the write into the paged cache;
* ``append4`` -- the same with the cache held in 4 bits, and its rows read back;
* ``decode4`` -- banded attention of a few new tokens a request over that cache.

4 bits: 32 adjacent channels of a head share a scale s, a code c stands for
s (c - 8).  The values are rounded to the tensors' type first; s is their value
of largest magnitude over -8, in 5 significant bits, so that s (c - 8) has no
more than 8 and is exact in every type.

Where ``own`` is false ``run`` computes them from elementary torch operations,
where it is true with the package's entry points.
"""
import math

import torch

own = False

_DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"f16": 2, "bf16": 2, "f32": 4}
_FULL = 1 << 28      # a window wider than any sequence: plain causal attention
_BASE = 10000.0
_EPS = 1e-6
_GROUP = 32          # channels that share a scale
_FLOOR = {"f16": -24, "bf16": -120, "f32": -120}                  # a scale is a multiple of 2 to this ...
_MOST = {"f16": 1.25 * 2.0 ** 11, "bf16": 1.25 * 2.0 ** 123, "f32": 1.25 * 2.0 ** 123}    # ... and at most that


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def _norm(name, dtype, b, n, h, hk, hd, rot, interleaved, pos_hi, offset, backward):
    return {"name": name, "op": "norm", "dtype": dtype, "b": b, "n": n, "h": h, "hk": hk, "hd": hd, "rot": rot,
            "interleaved": interleaved, "pos_hi": pos_hi, "offset": offset, "backward": backward}


def _append(name, bits, norm, dtype, batch, new_lo, new_hi, pad, h, hk, hd, rot, interleaved, page):
    return {"name": name, "op": "append4" if bits == 4 else "append", "norm": norm, "dtype": dtype, "batch": batch,
            "new_lo": new_lo, "new_hi": new_hi, "pad": pad, "h": h, "hk": hk, "hd": hd, "rot": rot,
            "interleaved": interleaved, "page": page}


def _decode(name, dtype, batch, q_max, len_lo, len_hi, h, hk, hd, w, dilation, sinks, page, ring):
    return {"name": name, "op": "decode4", "dtype": dtype, "batch": batch, "q_max": q_max, "len_lo": len_lo, "len_hi": len_hi,
            "h": h, "hk": hk, "hd": hd, "w": w, "dilation": dilation, "sinks": sinks, "page": page, "ring": ring}


def listed():
    return [
        # the queries and keys of one long prompt between the projection and the attention
        _norm("norm_prompt", "bf16", 1, 8192, 32, 8, 128, 128, False, 131072, 0.0, False),
        # a training step's gradient: the padded batch of the repository's training workload, a third of its length
        _norm("norm_gradient", "f16", 12, 1365, 12, 12, 64, 64, False, 1365, 0.0, True),
        # the gradient check of a model in full precision: odd sizes, part of the head turned in adjacent pairs,
        # weights stored less 1
        _norm("norm_odd_f32", "f32", 3, 257, 5, 1, 80, 20, True, 4096, 1.0, True),
        # one step of a running batch into a cache in 16 bits
        _append("append_step", 16, True, "bf16", 64, 1, 1, 0, 32, 8, 128, 128, False, 64),
        # prompts of several requests in one flat, padded batch, the repository's heads
        _append("append_prompts", 16, True, "f16", 16, 100, 1000, 91, 12, 12, 64, 64, False, 64),
        # one step of a running batch into a cache in 4 bits
        _append("append4_step", 4, True, "bf16", 64, 1, 1, 0, 32, 8, 128, 128, False, 64),
        # prompts into a cache in 4 bits
        _append("append4_prompts", 4, True, "bf16", 16, 100, 1000, 91, 32, 8, 128, 128, False, 64),
        # a model without norms, up to four tokens a request, half of the head turned in adjacent pairs
        _append("append4_drafts", 4, False, "f16", 48, 1, 4, 7, 12, 4, 64, 32, True, 32),
        # the smallest call: one request, a window of 256, the repository's heads
        _decode("decode4_latency", "f16", 1, 1, 200, 200, 12, 12, 64, 256, 0, 0, 64, False),
        # one request with a long context and shared key heads
        _decode("decode4_long", "bf16", 1, 1, 131072, 131072, 32, 8, 128, _FULL, 0, 0, 64, False),
        # a batch under the window of the repository's causal workload (4096), 16 leading global tokens, up to
        # four tokens a request (drafts being checked), recycled blocks
        _decode("decode4_window", "bf16", 48, 4, 4, 20000, 32, 8, 128, 4096, 0, 16, 32, True),
        # ragged contexts under the repository's dilated window, 3 heads a key head
        _decode("decode4_dilated", "f16", 32, 1, 1000, 8000, 12, 4, 64, 1024, 3, 0, 64, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "append", "append4", "append4", "decode4", "decode4", "decode4"])
    heads = rng.choice([(12, 12), (12, 4), (32, 8), (16, 16), (24, 8), (8, 1), (14, 2)])
    dtype = rng.choice(["f16", "bf16"])
    page = rng.choice([16, 32, 64, 128])
    if op == "norm":
        hd = rng.choice([64, 80, 96, 128])
        b, total = rng.choice([1, 1, 2, 5]), _log(rng, 8, 8192)
        c = _norm("", rng.choice(["f16", "bf16", "bf16", "f32"]), b, max(1, total // b), *heads, hd,
                  rng.choice([hd, hd // 2, hd // 4]) // 2 * 2, rng.random() < 0.4, rng.choice([8192, 131072, 1000000]),
                  rng.choice([0.0, 0.0, 1.0]), rng.random() < 0.5)
        if c["dtype"] == "f32":
            c["n"] = max(1, c["n"] // 2)
        if c["backward"]:
            c["n"] = max(1, c["n"] * 2 // 3)
    elif op != "decode4":
        hd, batch = rng.choice([64, 64, 128, 128, 96]), _log(rng, 1, 128)
        new_hi = rng.choice([1, 1, 4, max(1, 8000 // batch)])
        c = _append("", 4 if op == "append4" else 16, op == "append" or rng.random() < 0.6, dtype, batch, 1, new_hi,
                    rng.choice([0, 0, 7]), *heads, hd, rng.choice([hd, hd // 2, 0]), rng.random() < 0.4, page)
    else:
        q_max, batch, hd = rng.choice([1, 1, 1, 2, 4]), _log(rng, 1, 64), rng.choice([64, 64, 128, 128, 128, 96])
        hi = _log(rng, 16, max(64, min(131072, 400000 // batch)))
        w = rng.choice([256, 1024, 4096, _FULL])
        dilation = rng.choice([0, 0, 0, 1, 3]) if w < _FULL else 0
        c = _decode("", rng.choice([dtype] * 7 + ["f32"]), batch, q_max, rng.choice([q_max, max(q_max, hi // 2)]), max(hi, q_max),
                    *heads, hd, w, dilation, rng.choice([0, 0, 4, 16]), page, w < _FULL and rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# lengths and sizes that follow from a case alone
# ---------------------------------------------------------------------------
def _spread(count, lo, hi, shift=0.31):
    """`count` whole numbers spread over [lo, hi] (one of them: hi)."""
    if count == 1:
        return [hi]
    return [lo + int(((0.6180339887498949 * r + shift) % 1.0) * (hi - lo + 1)) for r in range(count)]


def _lengths(c):
    """Tokens held after the call and new tokens of each request."""
    if c["op"] != "decode4":
        new = _spread(c["batch"], c["new_lo"], c["new_hi"])
        return [m + k for m, k in zip(new, _spread(c["batch"], 0, 3000, 0.5))], new
    new = _spread(c["batch"], 1, c["q_max"], 0.77)
    return [max(a, b) for a, b in zip(_spread(c["batch"], c["len_lo"], c["len_hi"]), new)], new


def _columns(c, lens):
    """(columns of the block table, leading columns that are never recycled)"""
    page = c["page"]
    if c.get("ring"):
        pinned = -(-c["sinks"] // page)
        return pinned + -(-(c["w"] * (c["dilation"] + 1) + c["q_max"] - 1) // page) + 1, pinned
    return max(1, -(-max(lens) // page)), 0


def _visible(c, i):
    """How many keys the query at position i attends to."""
    sinks = min(c["sinks"], i + 1)
    band = 0 if i < c["sinks"] else min(c["w"], (i - c["sinks"]) // (c["dilation"] + 1)) + 1
    return sinks + band


def _union(c, lo, hi):
    """How many keys at least one of the queries at positions lo..hi attends to."""
    if c["dilation"]:
        return min(hi + 1, sum(_visible(c, i) for i in range(lo, hi + 1)))
    return min(hi + 1, _visible(c, lo) + hi - lo)


def _row4(c):
    """Bytes of a row of K or V in 4 bits: codes and scales (of the tensors' type)."""
    return c["hd"] // 2 + c["hd"] // _GROUP * _SIZE[c["dtype"]]


def work(case):
    c = case
    es, hd = _SIZE[c["dtype"]], c["hd"]
    if c["op"] == "norm":
        rows = c["b"] * c["n"] * (c["h"] + c["hk"])
        return {"bytes": (3.0 if c["backward"] else 2.0) * rows * hd * es + 4.0 * c["b"] * c["n"] + 2.0 * hd * es,
                "flops": rows * (3.0 * c["rot"] + (10.0 if c["backward"] else 4.0) * hd)}
    lens, new = _lengths(c)
    if c["op"] != "decode4":
        t, heads = sum(new), c["h"] + 2 * c["hk"]
        if c["op"] == "append":
            moved = 2.0 * t * heads * hd * es
        else:                        # queries and rows read, queries and codes written; codes read, rows written
            moved = t * ((c["h"] + heads) * hd * es + 2.0 * c["hk"] * (2 * _row4(c) + hd * es))
        return {"bytes": moved + 8.0 * t,
                "flops": t * (c["h"] + c["hk"]) * (3.0 * c["rot"] + 4.0 * hd * c["norm"]) + (c["op"] == "append4") * 8.0 * t * c["hk"] * hd}
    keys = sum(_union(c, a - m, a - 1) for a, m in zip(lens, new))
    pairs = sum(_visible(c, i) for a, m in zip(lens, new) for i in range(a - m, a))
    return {"bytes": 2.0 * keys * c["hk"] * _row4(c) + sum(new) * c["h"] * (2.0 * hd * es + 4.0),
            "flops": 4.0 * pairs * c["h"] * hd}


# ---------------------------------------------------------------------------
# the cache in 4 bits, in torch
# ---------------------------------------------------------------------------
def _quantise(x, dtype):
    """(codes [..., hd / 2] uint8, low half the even channel; scales [..., hd / 32]) of values x [..., hd]."""
    g = x.to(_DTYPES[dtype]).float().unflatten(-1, (-1, _GROUP))
    top, low = g.amax(-1), g.amin(-1)
    s = torch.where(top >= -low, top, low) / -8.0
    step = torch.exp2((torch.frexp(s)[1].float() - 5.0).clamp(min=_FLOOR[dtype]))
    s = (torch.round(s / step) * step).clamp(-_MOST[dtype], _MOST[dtype])
    code = torch.round(g / s.unsqueeze(-1)).nan_to_num(0.0).clamp(-8, 7)
    code = (torch.where(s.unsqueeze(-1) == 0, 0.0, code) + 8).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (s + 0.0).to(_DTYPES[dtype])


def _values(codes, scales):
    """The values that codes and scales stand for, in fp32."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8.0
    return (c.unflatten(-1, (-1, _GROUP)) * scales.float().unsqueeze(-1)).flatten(-2)


# ---------------------------------------------------------------------------
# states
# ---------------------------------------------------------------------------
def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _keys(g, shape, dtype):
    """Keys or values: some channels are several times larger than the others."""
    width = 1.0 + 3.0 * (torch.rand(shape[-1], generator=g, device="cuda") < 0.06)
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * width).to(dtype)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _starts(new):
    at, out = 0, [0]
    for m in new:
        at += m
        out.append(at)
    return out


def _column(block, cols, pinned, ring):
    return pinned + (block - pinned) % (cols - pinned) if ring and block >= cols else block


def _table(used, cols, blocks, seed):
    """A block table with `used` blocks in each row, at random places of the cache, and -1 behind them."""
    perm = torch.randperm(blocks, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table, at = torch.full((len(used), cols), -1, dtype=torch.int32), 0
    for r, k in enumerate(used):
        table[r, :k] = perm[at:at + k]
        at += k
    return table


def _weights(c, s, g, dt):
    for name in ("wq", "wk"):
        w = torch.randn(c["hd"], generator=g, device="cuda") * 0.2
        s[name] = (w if c.get("offset") else w + 1.0).to(dt)


def _rotary_state(c, s, b, n):
    f = [_BASE ** (-2.0 * k / c["rot"]) for k in range(c["rot"] // 2)]
    s["freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
    if own:
        import sliding_window_attention_band_gb300 as swab

        s["turns"] = swab.rotary_frequencies(c["rot"], _BASE)[0].cuda() if c["rot"] else None
        s["d"] = swab.RotaryDesc(b, n, c["h"], c["hk"], c["hd"], c["rot"], interleaved=c["interleaved"], dtype=_DTYPES[c["dtype"]])
        s["nd"] = swab.NormDesc(_EPS, c.get("offset", 0.0)) if c.get("norm", True) else None


def prepare(case, seed):
    c = dict(case)
    s = {"c": c}
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = _DTYPES[c["dtype"]]
    if c["op"] == "norm":
        first = torch.randint(0, max(1, c["pos_hi"] - c["n"] + 1), (c["b"], 1), generator=g, device="cuda")
        s["pos"] = (first + torch.arange(c["n"], device="cuda")).to(torch.int32)
        s["q"] = _randn(g, (c["b"], c["n"], c["h"], c["hd"]), dt)
        s["k"] = _keys(g, (c["b"], c["n"], c["hk"], c["hd"]), dt)
        _weights(c, s, g, dt)
        if c["backward"]:
            s["gq"], s["gk"] = _randn(g, s["q"].shape, dt), _randn(g, s["k"].shape, dt)
        _rotary_state(c, s, c["b"], c["n"])
        if own:
            import sliding_window_attention_band_gb300 as swab

            s["qo"], s["ko"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
            if c["backward"]:
                s["dwq"], s["dwk"] = (torch.empty(c["hd"], dtype=torch.float32, device="cuda") for _ in range(2))
                s["ws"] = torch.empty(max(1, swab.norm_rotary_bwd_workspace(s["d"])), dtype=torch.uint8, device="cuda")
        return s
    lens, new = _lengths(c)
    cols, pinned = _columns(c, lens)
    page, ring, hk, hd = c["page"], bool(c.get("ring")), c["hk"], c["hd"]
    used = [min(-(-a // page), cols) for a in lens]
    blocks = sum(used) + 3
    table = _table(used, cols, blocks, int(seed))
    if c["op"] == "append":
        s["kc"], s["vc"] = _randn(g, (blocks, hk, page, hd), dt), _randn(g, (blocks, hk, page, hd), dt)
    else:
        s["kc"], s["ks"] = _quantise(_keys(g, (blocks, hk, page, hd), dt), c["dtype"])
        s["vc"], s["vs"] = _quantise(_randn(g, (blocks, hk, page, hd), dt), c["dtype"])
    if c["op"] != "decode4":
        pos, slots = [], []
        host = table.tolist()
        for r, (a, m) in enumerate(zip(lens, new)):
            pos += range(a - m, a)
            slots += [host[r][j // page] * page + j % page for j in range(a - m, a)]
        s["pos"] = _i32(pos + [0] * c["pad"])
        s["slots"] = _i32(slots + [-1] * c["pad"])
        t = len(pos) + c["pad"]
        qkv = _randn(g, (t, c["h"] + 2 * hk, hd), dt)                          # one merged projection
        s["q"], s["k"], s["v"] = qkv.split([c["h"], hk, hk], dim=1)
        _weights(c, s, g, dt)
        _rotary_state(c, s, 1, t)
        if own:
            import sliding_window_attention_band_gb300 as swab

            s["qo"] = torch.empty(t, c["h"], hd, dtype=dt, device="cuda")
            s["cache"] = swab.CacheDesc(c["batch"], page, blocks, cols)
            if c["op"] == "append4":
                s["ko"], s["vo"] = (torch.zeros(t, hk, hd, dtype=dt, device="cuda") for _ in range(2))
        return s
    s["q"] = _randn(g, (sum(new), c["h"], hd), dt)
    s["lens"], s["start"], s["table"] = _i32(lens), _i32(_starts(new)), table.cuda()
    s["new"] = new
    s["host"] = (lens, new, cols, pinned, max(new), max(min(a, m + c["w"] * (c["dilation"] + 1)) for a, m in zip(lens, new)))
    if own:
        import sliding_window_attention_band_gb300 as swab

        cache = swab.CacheDesc(c["batch"], page, blocks, cols, ring=ring, pinned=pinned)
        s["d"] = swab.DecodeDesc(cache, sum(new), c["h"], hk, hd, w=c["w"], dilation=c["dilation"], n_sink=c["sinks"],
                                 max_q=c["q_max"], max_len=max(lens), dtype=dt)
        s["ws"] = torch.empty(max(1, swab.band_decode4_workspace(s["d"])), dtype=torch.uint8, device="cuda")
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(sum(new), c["h"], dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    c = s["c"]
    if own:
        return _run_own(c, s)
    if c["op"] == "norm":
        return _plain_gradient(c, s) if c["backward"] else {"q": _plain_norm(s["q"], s["wq"], s, c), "k": _plain_norm(s["k"], s["wk"], s, c)}
    if c["op"] == "decode4":
        return _plain_decode(c, s)
    q, k = (_plain_norm(s[x], s["w" + x], s, c) for x in ("q", "k"))
    keep = s["slots"] >= 0
    slot = s["slots"][keep].long()
    block, off = slot // c["page"], slot % c["page"]
    if c["op"] == "append":
        s["kc"][block, :, off] = k[keep]
        s["vc"][block, :, off] = s["v"][keep]
        return {"q": q, "kc": s["kc"], "vc": s["vc"]}
    out = {"q": q}
    k = _plain_norm(s["k"], s["wk"], s, c, torch.float64)                  # values next to a border of two codes
    for name, x in (("k", k), ("v", s["v"])):
        codes, scales = s[name + "c"], s[name + "s"]
        codes[block, :, off], scales[block, :, off] = _quantise(x[keep], c["dtype"])
        rows = torch.zeros_like(s[name])
        rows[keep] = _values(codes[block, :, off], scales[block, :, off]).to(rows.dtype)
        out[name] = rows
    return out


def _run_own(c, s):
    import sliding_window_attention_band_gb300 as swab

    if c["op"] == "norm":
        if not c["backward"]:
            swab.norm_rotary(s["d"], s["nd"], s["turns"], s["q"], s["qo"], s["k"], s["ko"], s["wq"], s["wk"], pos=s["pos"])
            return {"q": s["qo"], "k": s["ko"]}
        swab.norm_rotary_bwd(s["d"], s["nd"], s["turns"], s["gq"], s["q"], s["qo"], s["gk"], s["k"], s["ko"], s["wq"], s["wk"],
                             s["dwq"], s["dwk"], s["ws"], pos=s["pos"])
        return {"q": s["qo"], "k": s["ko"], "wq": s["dwq"], "wk": s["dwk"]}
    if c["op"] == "append":
        swab.norm_rotary_append(s["d"], s["nd"], s["cache"], s["turns"], s["q"], s["k"], s["v"], s["pos"], s["slots"], s["qo"],
                                s["kc"], s["vc"], s["wq"], s["wk"])
        return {"q": s["qo"], "kc": s["kc"], "vc": s["vc"]}
    if c["op"] == "append4":
        w = (s["wq"], s["wk"]) if c["norm"] else (None, None)
        swab.rotary_append4(s["d"], s["cache"], s["turns"], s["q"], s["k"], s["v"], s["pos"], s["slots"], s["qo"], s["kc"], s["ks"],
                            s["vc"], s["vs"], s["nd"], *w)
        swab.cache_read4(s["cache"], s["slots"], s["kc"], s["ks"], s["vc"], s["vs"], s["ko"], s["vo"])
        return {"q": s["qo"], "k": s["ko"], "v": s["vo"]}
    swab.band_decode4(s["d"], c["hd"] ** -0.5, s["q"], s["kc"], s["ks"], s["vc"], s["vs"], s["table"], s["lens"], s["start"],
                      s["o"], s["lse"], s["ws"])
    return {"o": s["o"], "lse": s["lse"]}


def _angles(s, dtype=torch.float32):
    a = s["pos"].double().unsqueeze(-1) * s["freq"]                         # far positions need 64 bits
    return a.cos().to(dtype).unsqueeze(-2), a.sin().to(dtype).unsqueeze(-2)


def _turn(v, cos, sin, c):
    r = c["rot"]
    a, b = (v[..., 0:r:2], v[..., 1:r:2]) if c["interleaved"] else (v[..., :r // 2], v[..., r // 2:r])
    p, q = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((p, q), -1).flatten(-2) if c["interleaved"] else torch.cat((p, q), -1)
    return torch.cat((y, v[..., r:]), -1)


def _plain_norm(x, w, s, c, dtype=torch.float32):
    v = x.to(dtype)
    if c.get("norm", True):
        v = v * torch.rsqrt(v.square().mean(-1, keepdim=True) + _EPS) * (w.to(dtype) + c.get("offset", 0.0))
    if c["rot"]:
        v = _turn(v, *_angles(s, dtype), c)
    return v.to(x.dtype)


def _plain_gradient(c, s):
    cos, sin = _angles(s)
    out = {}
    for name in ("q", "k"):
        x, w = s[name].float(), s["w" + name].float() + c["offset"]
        g = _turn(s["g" + name].float(), cos, -sin, c)
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + _EPS)
        n, gw = x * r, g * w
        out[name] = (r * (gw - n * (gw * n).mean(-1, keepdim=True))).to(s[name].dtype)
        out["w" + name] = (g * n).sum((0, 1, 2), dtype=torch.float64).float()      # a long sum
    return out


def _plain_decode(c, s):
    lens, new, cols, pinned, m, span = s["host"]
    page, stride, w, sinks, hk, hd = c["page"], c["dilation"] + 1, c["w"], c["sinks"], c["hk"], c["hd"]
    held, start = s["lens"].long()[:, None], s["start"].long()
    count = (start[1:] - start[:-1])[:, None]
    j = torch.arange(span, device="cuda") + (held - span).clamp(min=0)
    j = torch.cat((torch.arange(sinks, device="cuda").expand(c["batch"], -1), j), 1)
    band = torch.arange(j.shape[1], device="cuda") >= sinks
    block = j // page
    column = torch.where(block >= cols, pinned + (block - pinned) % max(1, cols - pinned), block)
    ids = s["table"].long().gather(1, column).clamp(min=0)
    k = _values(s["kc"][ids, :, j % page], s["ks"][ids, :, j % page])          # [requests, keys, hk, hd]
    v = _values(s["vc"][ids, :, j % page], s["vs"][ids, :, j % page])
    a = torch.arange(m, device="cuda")
    i, jj = (held - count + a)[:, :, None], j[:, None, :]                       # positions of the queries and keys
    seen = torch.where(band, (jj >= sinks) & (i - jj <= w * stride) & ((i - jj) % stride == 0), True) & (jj <= i)
    rows = (start[:-1, None] + a).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float().view(-1, hk, c["h"] // hk, hd)[rows]                     # [requests, m, hk, group, hd]
    x = torch.einsum("rmkgd,rjkd->rkgmj", q, k) * hd ** -0.5
    x = x.masked_fill(~seen[:, None, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    p = (x - top).exp()
    z = p.sum(-1, keepdim=True)
    y = (torch.einsum("rkgmj,rjkd->rkgmd", p, v) / z).permute(0, 3, 1, 2, 4).flatten(2, 3)
    l = (top + z.log())[..., 0].permute(0, 3, 1, 2).flatten(2, 3)
    live = a < count
    return {"o": y[live].to(s["q"].dtype), "lse": l[live]}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_norm(x, w, s, c):
    """Rows of x [..., heads, hd], normed and turned as complex numbers."""
    if c.get("norm", True):
        x = x / (x.pow(2).sum(-1, keepdim=True) / c["hd"] + _EPS).sqrt() * (w + c.get("offset", 0.0))
    if not c["rot"]:
        return x
    half = c["rot"] // 2
    pairs = torch.arange(half, device="cuda")
    one, two = (2 * pairs, 2 * pairs + 1) if c["interleaved"] else (pairs, pairs + half)
    t = s["pos"].double()[..., None] * s["freq"]
    z = torch.complex(x[..., one], x[..., two]) * torch.polar(torch.ones_like(t), t)[..., None, :]
    y = x.clone()
    y[..., one], y[..., two] = z.real, z.imag
    return y


def _exact_cells(x, dtype):
    """The values that rows x [..., hd] become in 4 bits, from the definition."""
    g = x.to(_DTYPES[dtype]).double().reshape(-1, _GROUP)
    at = torch.where(g.amax(1) >= -g.amin(1), g.argmax(1), g.argmin(1))
    s = g.gather(1, at[:, None]) / -8
    _, e = torch.frexp(s)
    step = torch.ldexp(torch.ones_like(s), torch.clamp(e - 5, min=_FLOOR[dtype]))
    s = torch.clamp(torch.round(s / step) * step, -_MOST[dtype], _MOST[dtype])
    n = torch.clamp(torch.round(g / torch.where(s == 0, 1.0, s)), -8, 7)
    return (n * s).reshape(x.shape)


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    if c["op"] == "decode4":
        return _exact_decode(c, s)
    out = {}
    for name in ("q", "k"):
        x, w = s[name].double().requires_grad_(), s["w" + name].double().requires_grad_()
        y = _exact_norm(x, w, s, c)
        if c.get("backward"):
            out[name], out["w" + name] = torch.autograd.grad(y, (x, w), s["g" + name].double())
        else:
            out[name] = y.detach()
    if c["op"] == "norm":
        return out
    live = [t for t, x in enumerate(s["slots"].tolist()) if x >= 0]
    if c["op"] == "append4":
        # (a code is a step function of its value: where 32 bits and 64 fall on two sides of a border, here once in
        # some millions, they are a whole step apart.  So a key that has been computed has no value to be held to.)
        for name, x in (("k", out["k"]), ("v", s["v"].double())):
            rows = torch.zeros_like(x)
            rows[live] = _exact_cells(x[live], c["dtype"])
            out[name] = None if name == "k" and (c["norm"] or c["rot"]) else rows
        return out
    at = torch.tensor([s["slots"].tolist()[t] for t in live], device="cuda")
    kept = {"q": out["q"]}
    for name, x in (("kc", out["k"]), ("vc", s["v"].double())):
        flat = s[name].double().transpose(1, 2).reshape(-1, c["hk"], c["hd"])
        flat.index_copy_(0, at, x[live])
        kept[name] = flat.view(-1, c["page"], c["hk"], c["hd"]).transpose(1, 2)
    return kept


def _exact_decode(c, s):
    lens, new, cols, pinned = s["host"][:4]
    table, page, hk, hd = s["table"].tolist(), c["page"], c["hk"], c["hd"]
    stride, group = c["dilation"] + 1, c["h"] // c["hk"]

    def rows(codes, scales, slots):
        slots = torch.tensor(slots, device="cuda")
        byte = codes[slots // page, :, slots % page].int()                      # [keys, hk, hd / 2]
        n = torch.empty(*byte.shape[:-1], hd, dtype=torch.float64, device="cuda")
        n[..., 0::2], n[..., 1::2] = (byte % 16).double(), (byte // 16).double()
        return ((n - 8) * scales[slots // page, :, slots % page].double().repeat_interleave(_GROUP, -1)).transpose(0, 1)

    out, lses, t = [], [], 0
    for r, (a, m) in enumerate(zip(lens, new)):
        for i in range(a - m, a):
            keys = list(range(min(c["sinks"], i + 1)))
            keys += [j for j in range(i, max(c["sinks"], i - c["w"] * stride) - 1, -stride)]
            slot = [table[r][_column(j // page, cols, pinned, c["ring"])] * page + j % page for j in keys]
            k, v = rows(s["kc"], s["ks"], slot), rows(s["vc"], s["vs"], slot)    # [hk, keys, hd]
            x = s["q"][t].double().view(hk, group, hd) @ k.transpose(1, 2) / math.sqrt(hd)
            l = x.logsumexp(-1)
            out.append(((x - l[..., None]).exp() @ v).reshape(c["h"], hd))
            lses.append(l.reshape(-1))
            t += 1
    return {"o": torch.stack(out), "lse": torch.stack(lses)}
