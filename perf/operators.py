"""The serving operators, measured one call at a time.

Five operators that a program around the banded attention needs to answer with
it, one token or a few at a time:

* ``rotary``  -- rotary positions on queries and keys (and the gradient);
* ``slots``   -- block tables and slot maps from request lengths;
* ``append``  -- rotary positions fused with the write into the paged cache;
* ``decode``  -- banded attention of a few new tokens a request over that cache;
* ``prefix``  -- the same where the batch shares a long prefix, read once for all.

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


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def _rotary(name, dtype, b, n, h, hk, hd, rot, interleaved, scaling, pos_hi, backward):
    return {"name": name, "op": "rotary", "dtype": dtype, "b": b, "n": n, "h": h, "hk": hk, "hd": hd, "rot": rot,
            "interleaved": interleaved, "scaling": scaling, "pos_hi": pos_hi, "backward": backward}


def _slots(name, batch, len_lo, len_hi, new_lo, new_hi, page, ring):
    """ring: columns of a recycled table (0: the table holds the whole sequence)."""
    return {"name": name, "op": "slots", "batch": batch, "len_lo": len_lo, "len_hi": len_hi, "new_lo": new_lo,
            "new_hi": new_hi, "page": page, "ring": ring}


def _append(name, dtype, batch, new_lo, new_hi, pad, h, hk, hd, rot, interleaved, scaling, page):
    return {"name": name, "op": "append", "dtype": dtype, "batch": batch, "new_lo": new_lo, "new_hi": new_hi, "pad": pad,
            "h": h, "hk": hk, "hd": hd, "rot": rot, "interleaved": interleaved, "scaling": scaling, "page": page}


def _decode(name, dtype, batch, q_max, len_lo, len_hi, h, hk, hd, w, dilation, sinks, page, ring, prefix=0):
    return {"name": name, "op": "prefix" if prefix else "decode", "dtype": dtype, "batch": batch, "q_max": q_max,
            "len_lo": len_lo, "len_hi": len_hi, "h": h, "hk": hk, "hd": hd, "w": w, "dilation": dilation, "sinks": sinks,
            "page": page, "ring": ring, "prefix": prefix}


def listed():
    return [
        # the queries and keys of one long prompt before the attention, positions scaled for a long context
        _rotary("rotary_prompt", "bf16", 1, 8192, 32, 8, 128, 128, False, "yarn", 131072, False),
        # a training step's gradient: the padded batch of the repository's training workload, a third of its
        # length, adjacent pairs in half of the head
        _rotary("rotary_gradient", "f16", 12, 1365, 12, 12, 64, 32, True, "none", 1365, True),
        # the check of a model in full precision: odd sizes, part of a head that is no power of two
        _rotary("rotary_odd_f32", "f32", 3, 257, 5, 1, 80, 20, False, "linear", 4096, False),
        # one step of a running batch: a token for each request, most of them inside their last block
        _slots("slots_step", 64, 1, 8192, 1, 1, 64, 0),
        # a scheduler that admits prompts beside running requests, in the recycled table of a window of 4096
        _slots("slots_prompts", 256, 0, 20000, 0, 500, 64, 66),
        # one step of a running batch: 64 tokens into the cache
        _append("append_step", "bf16", 64, 1, 1, 0, 32, 8, 128, 128, False, "bands", 64),
        # prompts of several requests in one flat, padded batch
        _append("append_prompts", "f16", 16, 100, 1000, 91, 12, 12, 64, 64, True, "none", 64),
        # the smallest call: one request, a window of 256, the repository's heads
        _decode("decode_latency", "f16", 1, 1, 200, 200, 12, 12, 64, 256, 0, 0, 64, False),
        # one request with a long context and shared key heads
        _decode("decode_long", "bf16", 1, 1, 131072, 131072, 32, 8, 128, _FULL, 0, 0, 64, False),
        # a batch under the window of the repository's causal workload (4096), 16 leading global tokens, up to
        # four tokens a request (drafts being checked), recycled blocks
        _decode("decode_window", "bf16", 48, 4, 4, 20000, 32, 8, 128, 4096, 0, 16, 32, True),
        # a small batch behind a short shared prefix that ends inside a block
        _decode("prefix_small", "f16", 16, 1, 1, 200, 12, 4, 64, _FULL, 0, 0, 16, False, 1000),
        # a large batch behind one long shared prompt
        _decode("prefix_large", "bf16", 128, 1, 1, 512, 32, 8, 128, _FULL, 0, 0, 64, False, 16384),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "slots", "append", "decode", "decode", "prefix"])
    heads = rng.choice([(12, 12), (12, 4), (32, 8), (16, 16), (24, 8), (8, 1), (14, 2)])
    dtype = rng.choice(["f16", "bf16"])
    hd = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    if op == "rotary":
        hd = rng.choice([64, 80, 96, 128])
        b, total = rng.choice([1, 1, 2, 5]), _log(rng, 8, 8192)
        c = _rotary("", rng.choice(["f16", "bf16", "bf16", "f32"]), b, max(1, total // b), *heads, hd,
                    rng.choice([hd, hd // 2, hd // 4]) // 2 * 2, rng.random() < 0.5,
                    rng.choice(["none", "linear", "ntk", "yarn", "bands"]), rng.choice([8192, 131072, 1000000]),
                    rng.random() < 0.4)
        if c["dtype"] == "f32":
            c["n"] = max(1, c["n"] // 2)
    elif op == "slots":
        batch, ring = _log(rng, 1, 1024), rng.random() < 0.5
        w = rng.choice([256, 1024, 4096])
        new_hi = rng.choice([1, 1, 4, max(1, 60000 // batch)])
        c = _slots("", batch, 0, _log(rng, 100, 40000), rng.choice([0, 1]), min(new_hi, 20000), page,
                   (w + 3) // page + 2 if ring else 0)
    elif op == "append":
        batch = _log(rng, 1, 128)
        new_hi = rng.choice([1, 1, 4, max(1, 8000 // batch)])
        c = _append("", dtype, batch, 1, new_hi, rng.choice([0, 0, 7]), *heads, hd, rng.choice([hd, hd // 2, 0]),
                    rng.random() < 0.5, rng.choice(["none", "yarn", "bands"]), page)
    else:
        q_max, prefix = rng.choice([1, 1, 1, 2, 4]), 0
        if op == "prefix":
            prefix, batch, hi = _log(rng, 100, 16384), _log(rng, 2, 128), _log(rng, 4, 512)
            if q_max * batch > 128:
                q_max = 1
        else:
            batch = _log(rng, 1, 64)
            hi = _log(rng, 16, max(64, min(131072, 400000 // batch)))
        w = rng.choice([256, 1024, 4096, _FULL])
        dilation = rng.choice([0, 0, 0, 1, 3]) if w < _FULL else 0
        c = _decode("", dtype, batch, q_max, rng.choice([q_max, max(q_max, hi // 2)]), max(hi, q_max), *heads, hd, w, dilation,
                    rng.choice([0, 0, 4, 16]), page, w < _FULL and rng.random() < 0.5, prefix)
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
    if c["op"] == "slots":
        return _spread(c["batch"], c["len_lo"], c["len_hi"]), _spread(c["batch"], c["new_lo"], c["new_hi"], 0.77)
    if c["op"] == "append":
        new = _spread(c["batch"], c["new_lo"], c["new_hi"])
        return [m + k for m, k in zip(new, _spread(c["batch"], 0, 3000, 0.5))], new
    new = _spread(c["batch"], 1, c["q_max"], 0.77)
    return [max(a, b) for a, b in zip(_spread(c["batch"], c["len_lo"], c["len_hi"]), new)], new


def _columns(c, lens):
    """(columns of the block table, leading columns that are never recycled)"""
    page = c["page"]
    if c["op"] == "slots":
        return (c["ring"], 0) if c["ring"] else (max(1, -(-max(a + b for a, b in zip(*_lengths(c))) // page)), 0)
    if c.get("ring"):
        pinned = -(-c["sinks"] // page)
        return pinned + -(-(c["w"] * (c["dilation"] + 1) + c["q_max"] - 1) // page) + 1, pinned
    return max(1, -(-max(lens) // page)), 0


def _visible(c, i):
    """How many of its own keys the query at position i attends to."""
    s = c["dilation"] + 1
    sinks = min(c["sinks"], i + 1)
    band = 0 if i < c["sinks"] else min(c["w"], (i - c["sinks"]) // s) + 1
    return sinks + band


def _union(c, lo, hi):
    """How many own keys at least one of the queries at positions lo..hi attends to."""
    if c["dilation"]:
        return min(hi + 1, sum(_visible(c, i) for i in range(lo, hi + 1)))
    return min(hi + 1, _visible(c, lo) + hi - lo)


def work(case):
    c = case
    if c["op"] == "slots":
        lens, new = _lengths(c)
        fresh = sum(-(-(a + b) // c["page"]) - -(-a // c["page"]) for a, b in zip(lens, new))
        return {"bytes": 4.0 * (4 * c["batch"] + 2 * sum(new) + 2 * fresh), "flops": float(sum(new))}
    es = _SIZE[c["dtype"]]
    if c["op"] == "rotary":
        rows = c["b"] * c["n"] * (c["h"] + c["hk"])
        return {"bytes": 2.0 * rows * c["hd"] * es + 4.0 * c["b"] * c["n"], "flops": 3.0 * rows * c["rot"]}
    lens, new = _lengths(c)
    if c["op"] == "append":
        t = sum(new)
        return {"bytes": 2.0 * t * (c["h"] + 2 * c["hk"]) * c["hd"] * es + 8.0 * t,
                "flops": 3.0 * t * (c["h"] + c["hk"]) * c["rot"]}
    keys = sum(_union(c, a - m, a - 1) for a, m in zip(lens, new)) + c["prefix"]
    pairs = sum(_visible(c, i) + c["prefix"] for a, m in zip(lens, new) for i in range(a - m, a))
    return {"bytes": 2.0 * keys * c["hk"] * c["hd"] * es + sum(new) * c["h"] * (2.0 * c["hd"] * es + 4.0),
            "flops": 4.0 * pairs * c["h"] * c["hd"]}


# ---------------------------------------------------------------------------
# rotary frequencies, in radians a position
# ---------------------------------------------------------------------------
_SCALING = {"none": (1.0, 0), "linear": (4.0, 4096), "ntk": (8.0, 4096), "yarn": (16.0, 8192), "bands": (8.0, 8192)}


def _frequencies(rot, kind):
    """(rot / 2 frequencies, factor on cos and sin) for one way of scaling to long contexts: positions divided
    (linear), a larger base (ntk), divided only where a pair turns seldom within the original length (yarn, which
    also scales cos and sin), or by bands of wavelengths (bands)."""
    factor, original = _SCALING[kind]
    f = [_BASE ** (-2.0 * k / rot) for k in range(rot // 2)]
    if kind == "linear":
        return [x / factor for x in f], 1.0
    if kind == "ntk":
        base = _BASE * factor ** (rot / (rot - 2.0)) if rot > 2 else _BASE
        return [base ** (-2.0 * k / rot) for k in range(rot // 2)], 1.0
    if kind == "yarn":
        pair = lambda turns: rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(_BASE))  # noqa: E731
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        ramp = [min(max((k - lo) / max(hi - lo, 0.001), 0.0), 1.0) for k in range(rot // 2)]
        return [x / factor * r + x * (1 - r) for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0
    if kind == "bands":
        out = []
        for x in f:
            turns = original * x / (2 * math.pi)
            smooth = min(max((turns - 1.0) / (4.0 - 1.0), 0.0), 1.0)
            out.append((1 - smooth) * x / factor + smooth * x)
        return out, 1.0
    return f, 1.0


def _own_frequencies(rot, kind):
    import sliding_window_attention_band_gb300 as swab

    factor, original = _SCALING[kind]
    extra = {"low_turns": 1.0, "high_turns": 4.0} if kind == "bands" else {}
    return swab.rotary_frequencies(rot, _BASE, kind, factor, original, **extra)


# ---------------------------------------------------------------------------
# states
# ---------------------------------------------------------------------------
def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


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
    return table.cuda(), perm[at:].contiguous().cuda()


def prepare(case, seed):
    c = dict(case)
    s = {"c": c}
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    if c["op"] == "slots":
        return _prepare_slots(c, s, seed)
    dt = _DTYPES[c["dtype"]]
    if c["op"] == "rotary":
        first = torch.randint(0, max(1, c["pos_hi"] - c["n"] + 1), (c["b"], 1), generator=g, device="cuda")
        s["pos"] = (first + torch.arange(c["n"], device="cuda")).to(torch.int32)
        s["q"] = _randn(g, (c["b"], c["n"], c["h"], c["hd"]), dt)
        s["k"] = _randn(g, (c["b"], c["n"], c["hk"], c["hd"]), dt)
        _rotary_state(c, s, c["b"], c["n"])
        if own:
            s["qo"], s["ko"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        return s
    lens, new = _lengths(c)
    cols, pinned = _columns(c, lens)
    page, ring = c["page"], bool(c.get("ring"))
    used = [min(-(-a // page), cols) for a in lens]
    pre = -(-c.get("prefix", 0) // page)
    blocks = sum(used) + pre + 3
    table, spare = _table(used, cols, blocks, int(seed))
    tokens = sum(new)
    s["kc"] = _randn(g, (blocks, c["hk"], page, c["hd"]), dt)
    s["vc"] = _randn(g, (blocks, c["hk"], page, c["hd"]), dt)
    if c["op"] == "append":
        pos, slots = [], []
        host = table.tolist()
        for r, (a, m) in enumerate(zip(lens, new)):
            pos += range(a - m, a)
            slots += [host[r][j // page] * page + j % page for j in range(a - m, a)]
        s["pos"] = _i32(pos + [0] * c["pad"])
        s["slots"] = _i32(slots + [-1] * c["pad"])
        t = tokens + c["pad"]
        qkv = _randn(g, (t, c["h"] + 2 * c["hk"], c["hd"]), dt)      # one merged projection
        s["q"], s["k"], s["v"] = qkv.split([c["h"], c["hk"], c["hk"]], dim=1)
        _rotary_state(c, s, 1, t)
        if own:
            import sliding_window_attention_band_gb300 as swab

            s["qo"] = torch.empty(t, c["h"], c["hd"], dtype=dt, device="cuda")
            s["cache"] = swab.CacheDesc(c["batch"], page, blocks, cols)
        return s
    s["q"] = _randn(g, (tokens, c["h"], c["hd"]), dt)
    s["lens"], s["new"], s["start"] = _i32(lens), new, _i32(_starts(new))
    s["host"] = (lens, new, cols, pinned)
    s["table"] = table
    s["ptable"] = spare[:pre].contiguous() if pre else None
    if own:
        import sliding_window_attention_band_gb300 as swab

        cache = swab.CacheDesc(c["batch"], page, blocks, cols, ring=ring, pinned=pinned)
        s["d"] = swab.DecodeDesc(cache, tokens, c["h"], c["hk"], c["hd"], w=c["w"], dilation=c["dilation"],
                                 n_sink=c["sinks"], max_q=c["q_max"], max_len=max(lens), prefix_len=c["prefix"], dtype=dt)
        s["ws"] = torch.empty(max(1, swab.band_decode_workspace(s["d"])), dtype=torch.uint8, device="cuda")
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(tokens, c["h"], dtype=torch.float32, device="cuda")
    return s


def _rotary_state(c, s, b, n):
    if not c["rot"]:
        s["freq"], s["mscale"] = None, 1.0
    else:
        f, s["mscale"] = _frequencies(c["rot"], c["scaling"])
        s["freq"] = torch.tensor(f, dtype=torch.float64, device="cuda")
    if own:
        import sliding_window_attention_band_gb300 as swab

        scale = 1.0
        if c["rot"]:
            s["turns"], scale = _own_frequencies(c["rot"], c["scaling"])
            s["turns"] = s["turns"].cuda()
        else:
            s["turns"] = None
        s["d"] = swab.RotaryDesc(b, n, c["h"], c["hk"], c["hd"], c["rot"], interleaved=c["interleaved"], scale=scale,
                                 dtype=_DTYPES[c["dtype"]])


def _prepare_slots(c, s, seed):
    lens, new = _lengths(c)
    cols, _ = _columns(c, lens)
    order = torch.randperm(c["batch"], generator=torch.Generator().manual_seed(int(seed) + 1)).tolist()
    lens, new = [lens[r] for r in order], [new[r] for r in order]
    used = [min(-(-a // c["page"]), cols) for a in lens]
    want = sum(min(-(-(a + m) // c["page"]), cols) - u for a, m, u in zip(lens, new, used))
    blocks = sum(used) + want + 5
    s["table"], s["free"] = _table(used, cols, blocks, int(seed))
    s["lens"], s["new"], s["used"] = _i32(lens), _i32(new), _i32([2])     # two blocks of the list are gone already
    s["tokens"] = sum(new) + 3                                            # a flat batch with three rows of padding
    s["cols"] = cols
    if own:
        import sliding_window_attention_band_gb300 as swab

        s["d"] = swab.CacheDesc(c["batch"], c["page"], blocks, cols, ring=bool(c["ring"]))
        e = lambda *n: torch.empty(*n, dtype=torch.int32, device="cuda")  # noqa: E731
        s["lens_out"], s["used_out"], s["start"] = e(c["batch"]), e(2), e(c["batch"] + 1)
        s["slots"], s["pos"] = e(s["tokens"]), e(s["tokens"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    c = s["c"]
    if own:
        return _run_own(c, s)
    if c["op"] == "rotary":
        cos, sin = _angles(s["pos"], s["freq"], s["mscale"])
        if c["backward"]:
            sin = -sin
        return {"q": _turn(s["q"], cos, sin, c), "k": _turn(s["k"], cos, sin, c)}
    if c["op"] == "slots":
        return _plain_slots(c, s)
    if c["op"] == "append":
        q, k = s["q"], s["k"]
        if c["rot"]:
            cos, sin = _angles(s["pos"], s["freq"], s["mscale"])
            q, k = _turn(q, cos, sin, c), _turn(k, cos, sin, c)
        keep = s["slots"] >= 0
        slot = s["slots"][keep].long()
        block, off = slot // c["page"], slot % c["page"]
        s["kc"][block, :, off] = k[keep]
        s["vc"][block, :, off] = s["v"][keep]
        return {"q": q.clone() if q is s["q"] else q, "kc": s["kc"], "vc": s["vc"]}
    return _plain_decode(c, s)


def _run_own(c, s):
    import sliding_window_attention_band_gb300 as swab

    if c["op"] == "rotary":
        (swab.rotary_bwd if c["backward"] else swab.rotary)(s["d"], s["turns"], s["q"], s["qo"], s["k"], s["ko"], pos=s["pos"])
        return {"q": s["qo"], "k": s["ko"]}
    if c["op"] == "slots":
        swab.cache_slots(s["d"], s["lens"], s["new"], s["table"], s["free"], s["used"], s["lens_out"], s["used_out"],
                         s["start"], s["slots"], s["pos"])
        return {"table": s["table"], "lens": s["lens_out"], "used": s["used_out"], "start": s["start"], "slots": s["slots"],
                "pos": s["pos"]}
    if c["op"] == "append":
        swab.rotary_append(s["d"], s["cache"], s["turns"], s["q"], s["k"], s["v"], s["pos"], s["slots"], s["qo"], s["kc"],
                           s["vc"])
        return {"q": s["qo"], "kc": s["kc"], "vc": s["vc"]}
    swab.band_decode(s["d"], c["hd"] ** -0.5, s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["start"], s["o"], s["lse"],
                     s["ws"], prefix_table=s["ptable"])
    return {"o": s["o"], "lse": s["lse"]}


def _angles(pos, freq, mscale):
    a = pos.double().unsqueeze(-1) * freq                                  # far positions need 64 bits
    return (a.cos() * mscale).float().unsqueeze(-2), (a.sin() * mscale).float().unsqueeze(-2)


def _turn(x, cos, sin, c):
    r, v = c["rot"], x.float()
    a, b = (v[..., 0:r:2], v[..., 1:r:2]) if c["interleaved"] else (v[..., :r // 2], v[..., r // 2:r])
    p, q = a * cos - b * sin, b * cos + a * sin
    y = torch.stack((p, q), -1).flatten(-2) if c["interleaved"] else torch.cat((p, q), -1)
    return torch.cat((y, v[..., r:]), -1).to(x.dtype)


def _plain_slots(c, s):
    page, cols, batch = c["page"], s["cols"], c["batch"]
    lens, new, used = s["lens"].long(), s["new"].long(), s["used"].long()
    total = lens + new
    start = torch.cat((new.new_zeros(1), new.cumsum(0)))
    have = ((lens + page - 1) // page).clamp(max=cols)
    want = ((total + page - 1) // page).clamp(max=cols)
    before = torch.cat((new.new_zeros(1), (want - have).cumsum(0)))
    col = torch.arange(cols, device="cuda")
    fresh = (col >= have[:, None]) & (col < want[:, None])
    at = (used + before[:-1, None] + col - have[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][at], s["table"])
    t = torch.arange(s["tokens"], device="cuda")
    r = torch.searchsorted(start[1:], t, right=True).clamp(max=batch - 1)
    live = t < start[-1]
    pos = lens[r] + t - start[r]
    block = pos // page
    if c["ring"]:
        live_slot = live & (block > (total[r] - 1) // page - cols)
    else:
        live_slot = live
    slots = torch.where(live_slot, table[r, (block % cols).clamp(0, cols - 1)].long() * page + pos % page, -1)
    i = lambda x: x.to(torch.int32)  # noqa: E731
    return {"table": table, "lens": i(total), "used": i(torch.cat((used + before[-1:], used.new_zeros(1)))), "start": i(start),
            "slots": i(slots), "pos": i(torch.where(live, pos, 0))}


def _plain_decode(c, s):
    lens, new, cols, pinned = s["host"]
    page, stride, w, sinks, hk, hd = c["page"], c["dilation"] + 1, c["w"], c["sinks"], c["hk"], c["hd"]
    group, scale = c["h"] // hk, c["hd"] ** -0.5
    q_all = s["q"].float().view(-1, hk, group, hd)
    o, lse = torch.empty_like(s["q"]), torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    extra = extra_v = None
    if c["prefix"]:
        extra = s["kc"][s["ptable"].long()].transpose(1, 2).reshape(-1, hk, hd)[:c["prefix"]].float()
        extra_v = s["vc"][s["ptable"].long()].transpose(1, 2).reshape(-1, hk, hd)[:c["prefix"]].float()
    starts, m = _starts(new), max(new)
    first = [max(0, a - k - w * stride) for a, k in zip(lens, new)]
    longest = max(a - f for a, f in zip(lens, first)) + sinks
    at_once = max(1, int(6e8 / (longest * hk * hd * 4)))                   # requests gathered at a time
    for r0 in range(0, len(lens), at_once):
        rs = range(r0, min(len(lens), r0 + at_once))
        span = max(lens[r] - first[r] for r in rs)
        held = s["lens"][rs.start:rs.stop].long()[:, None]
        lo = _i32([first[r] for r in rs]).long()[:, None]
        j = torch.cat((torch.arange(sinks, device="cuda").expand(len(rs), -1), lo + torch.arange(span, device="cuda")), 1)
        band = torch.arange(j.shape[1], device="cuda") >= sinks
        block = j // page
        column = torch.where(block >= cols, pinned + (block - pinned) % max(1, cols - pinned), block)
        ids = s["table"][rs.start:rs.stop].long().gather(1, column).clamp(min=0)
        k = s["kc"][ids, :, j % page].float()                              # [requests, keys, hk, hd]
        v = s["vc"][ids, :, j % page].float()
        a = torch.arange(m, device="cuda")
        count = _i32([new[r] for r in rs]).long()[:, None]
        i = (held - count + a)[:, :, None]                                  # positions of the queries
        jj = j[:, None, :]
        seen = torch.where(band, (jj >= sinks) & (i - jj <= w * stride) & ((i - jj) % stride == 0), True) & (jj <= i)
        rows = (s["start"][rs.start:rs.stop].long()[:, None] + a).clamp(max=starts[-1] - 1)
        q = q_all[rows]                                                    # [requests, m, hk, group, hd]
        x = torch.einsum("rmkgd,rjkd->rkgmj", q, k) * scale
        x = x.masked_fill(~seen[:, None, None], float("-inf"))
        v = v.transpose(1, 2)[:, :, None]                                  # [requests, hk, 1, keys, hd]
        if extra is not None:
            x = torch.cat((torch.einsum("rmkgd,jkd->rkgmj", q, extra) * scale, x), -1)
        top = x.amax(-1, keepdim=True)
        p = (x - top).exp()
        z = p.sum(-1, keepdim=True)
        y = torch.matmul(p[..., c["prefix"]:], v)
        if extra is not None:
            y = y + torch.einsum("rkgmj,jkd->rkgmd", p[..., :c["prefix"]], extra_v)
        y = (y / z).permute(0, 3, 1, 2, 4).reshape(len(rs), m, c["h"], hd)
        l = (top + z.log())[..., 0].permute(0, 3, 1, 2).reshape(len(rs), m, c["h"])
        live = a < count
        o[rows[live]] = y[live].to(o.dtype)
        lse[rows[live]] = l[live]
    return {"o": o, "lse": lse}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    if c["op"] == "slots":
        return _exact_slots(c, s)
    if c["op"] in ("rotary", "append"):
        out = {}
        for name in ("q", "k"):
            x = s[name].double().contiguous()
            if c["rot"]:
                pairs = torch.arange(c["rot"] // 2, device="cuda")
                one, two = (2 * pairs, 2 * pairs + 1) if c["interleaved"] else (pairs, pairs + c["rot"] // 2)
                z = torch.polar(torch.full_like(s["freq"], s["mscale"]).expand(*s["pos"].shape, -1).contiguous(),
                                s["pos"].double()[..., None] * s["freq"] * (-1.0 if c.get("backward") else 1.0))
                turned = torch.complex(x[..., one], x[..., two]) * z[..., None, :]
                x[..., one], x[..., two] = turned.real.contiguous(), turned.imag.contiguous()
            out[name] = x
        if c["op"] == "rotary":
            return out
        kc, vc = s["kc"].double(), s["vc"].double()
        flat_k, flat_v = kc.transpose(1, 2).reshape(-1, c["hk"], c["hd"]), vc.transpose(1, 2).reshape(-1, c["hk"], c["hd"])
        at = torch.tensor([x for x in s["slots"].tolist() if x >= 0], device="cuda")
        rows = torch.tensor([t for t, x in enumerate(s["slots"].tolist()) if x >= 0], device="cuda")
        flat_k.index_copy_(0, at, out["k"][rows])
        flat_v.index_copy_(0, at, s["v"].double()[rows])
        back = lambda f: f.view(-1, c["page"], c["hk"], c["hd"]).transpose(1, 2)  # noqa: E731
        return {"q": out["q"], "kc": back(flat_k), "vc": back(flat_v)}
    return _exact_decode(c, s)


def _exact_slots(c, s):
    page, cols = c["page"], s["cols"]
    table, free, at = s["table"].tolist(), s["free"].tolist(), int(s["used"][0])
    lens, new = s["lens"].tolist(), s["new"].tolist()
    slots, pos = [], []
    for r, (a, m) in enumerate(zip(lens, new)):
        held = min(-(-a // page), cols)
        last = (a + m - 1) // page
        while held < min(last + 1, cols):
            table[r][held] = free[at]
            at, held = at + 1, held + 1
        for j in range(a, a + m):
            pos.append(j)
            gone = c["ring"] and j // page <= last - cols                 # overwritten within this very call
            slots.append(-1 if gone else table[r][j // page % cols] * page + j % page)
    pad = s["tokens"] - len(slots)
    return {"table": _i32(table), "lens": _i32([a + m for a, m in zip(lens, new)]), "used": _i32([at, 0]),
            "start": _i32(_starts(new)), "slots": _i32(slots + [-1] * pad), "pos": _i32(pos + [0] * pad)}


def _exact_decode(c, s):
    lens, new, cols, pinned = s["host"]
    table, page, hk, hd = s["table"].tolist(), c["page"], c["hk"], c["hd"]
    stride, group = c["dilation"] + 1, c["h"] // c["hk"]
    kc, vc = s["kc"].transpose(1, 2).flatten(0, 1), s["vc"].transpose(1, 2).flatten(0, 1)    # rows by slot

    def rows(cache, slots):
        return cache[torch.tensor(slots, device="cuda")].double().transpose(0, 1)            # [hk, keys, hd]

    shared = [int(b) * page + o for b in (s["ptable"].tolist() if c["prefix"] else []) for o in range(page)][:c["prefix"]]
    pk, pv = (rows(kc, shared), rows(vc, shared)) if shared else (None, None)
    out, lses, t = [], [], 0
    for r, (a, m) in enumerate(zip(lens, new)):
        for i in range(a - m, a):
            keys = list(range(min(c["sinks"], i + 1)))
            keys += [j for j in range(i, max(c["sinks"], i - c["w"] * stride) - 1, -stride)]
            slot = [table[r][_column(j // page, cols, pinned, c["ring"])] * page + j % page for j in keys]
            k, v = rows(kc, slot), rows(vc, slot)
            q = s["q"][t].double().view(hk, group, hd)
            x = q @ k.transpose(1, 2) / math.sqrt(hd)
            y = None
            if shared:
                x2 = q @ pk.transpose(1, 2) / math.sqrt(hd)
                l = torch.logaddexp(x.logsumexp(-1), x2.logsumexp(-1))
                y = (x2 - l[..., None]).exp() @ pv
            else:
                l = x.logsumexp(-1)
            o = (x - l[..., None]).exp() @ v
            out.append((o if y is None else o + y).reshape(c["h"], hd))
            lses.append(l.reshape(-1))
            t += 1
    return {"o": torch.stack(out), "lse": torch.stack(lses)}
