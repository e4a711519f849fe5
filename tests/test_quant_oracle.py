"""Pins of oracle/quant.py: norms against dense torch and autograd, the 4-bit
format against worked groups, with planted mistakes."""
import numpy as np
import pytest
import torch

from oracle import quant, serve


def rows(shape, seed, scale=1.0):
    return np.random.default_rng(seed).standard_normal(shape) * scale


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("offset,weighted", [(0.0, True), (1.0, True), (0.0, False)])
def test_norm_and_gradient_against_autograd(inter, offset, weighted):
    x, g, w = rows((2, 5, 3, 24), 0), rows((2, 5, 3, 24), 1), rows(24, 2)
    pos, (freq, _) = np.random.default_rng(3).integers(0, 5000, (2, 5)), serve.frequencies(16)
    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    n = torch.nn.functional.rms_norm(tx, (24,), eps=1e-3) * (tw + offset if weighted else 1.0)
    t = torch.tensor(pos)[..., None, None] * torch.tensor(freq)
    one, two = (slice(0, 16, 2), slice(1, 16, 2)) if inter else (slice(0, 8), slice(8, 16))
    a, b = n[..., one], n[..., two]
    y = n.clone()
    y[..., one], y[..., two] = 1.5 * (a * t.cos() - b * t.sin()), 1.5 * (b * t.cos() + a * t.sin())
    got = quant.norm_rotary(x, w if weighted else None, pos, freq, 1.5, inter, 1e-3, offset)
    np.testing.assert_allclose(got, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    dx, dw = quant.norm_rotary_bwd(g, x, w if weighted else None, pos, freq, 1.5, inter, 1e-3, offset)
    grads = torch.autograd.grad(y, (tx, tw) if weighted else (tx,), torch.tensor(g))
    np.testing.assert_allclose(dx, grads[0].numpy(), rtol=1e-11, atol=1e-12)
    if weighted:
        np.testing.assert_allclose(dw, grads[1].numpy(), rtol=1e-11, atol=1e-12)
        assert np.abs(dw - (serve.rotary(g, pos, freq, 1.5, inter, True) * x).reshape(-1, 24).sum(0)).max() > 0.1   # without r


def group(*head):
    return np.array(list(head) + [0.0] * (32 - len(head)))


def test_worked_groups():
    codes, scales = quant.quantise(group(8.0, -8.0, 1.0, -1.0, 0.5, 1.5, -2.5), "bf16")
    assert scales[0] == -1.0                                     # the positive one of two: its code is 0
    assert codes[:8].tolist() == [0, 15, 7, 9, 8, 6, 10, 8]      # -8 / -1 = 8 has no code; ties to even
    assert quant.values(codes, scales)[:7].tolist() == [8.0, -7.0, 1.0, -1.0, 0.0, 2.0, -2.0]
    codes, scales = quant.quantise(group(-8.0, 7.0, 4.0), "f16")
    assert scales[0] == 1.0 and codes[:3].tolist() == [0, 15, 12]
    assert quant.quantise(group(8.25), "f16")[1][0] == -1.0      # 33 / 32: a tie to the even one
    assert quant.quantise(group(8.26), "f16")[1][0] == -1.0625
    assert quant.quantise(group(8.75), "f16")[1][0] == -1.125
    codes, scales = quant.quantise(group(), "f16")
    assert scales[0] == 0.0 and (codes == 8).all()
    for bad in (np.nan, np.inf, -np.inf):
        codes, scales = quant.quantise(group(1.0, bad), "f16")
        assert np.isnan(scales[0]) and (codes == 8).all()
    assert quant.quantise(group(2.0 ** -21), "f16")[1][0] == -2.0 ** -24
    assert quant.quantise(group(2.0 ** -22), "f16")[1][0] == 0.0
    assert quant.quantise(group(65504.0), "f16")[1][0] == -2560.0
    assert quant.quantise(group(3e38), "bf16")[1][0] == -1.25 * 2.0 ** 123


@pytest.mark.parametrize("dtype,torch_dtype", [("f16", torch.float16), ("bf16", torch.bfloat16)])
def test_values_are_exact_in_their_type_and_near(dtype, torch_dtype):
    x = torch.tensor(rows((400, 64), 5) * 10.0 ** rows((400, 1), 6)).to(torch_dtype).double().numpy()
    codes, scales = quant.quantise(x, dtype)
    v = quant.values(codes, scales)
    assert np.array_equal(torch.tensor(v).to(torch_dtype).double().numpy(), v)
    assert np.array_equal(quant.unpack(quant.pack(codes)), codes)
    s = np.repeat(np.abs(scales), 32, -1)
    err, clipped = np.abs(v - x), codes == 15
    big = s > 2.0 ** -18
    assert (err <= s * np.where(clipped, 1.25, 0.5))[big].all()
    m = np.abs(x.reshape(400, -1, 32)).max(-1)
    # (m itself: its scale is within 2^-5, its code 0)
    assert (np.abs(8 * np.abs(scales) - m) <= m / 32)[np.abs(scales) > 2.0 ** -18].all()


@pytest.mark.parametrize("dtype,torch_dtype", [("f16", torch.float16), ("bf16", torch.bfloat16), ("f32", torch.float32)])
def test_errors_by_the_size_of_the_largest_value(dtype, torch_dtype):
    """What the header says of a group: near between two sizes, saturated above, within half a step of the smallest scale
    below."""
    low, high, least = (2.0 ** -17, 20480.0, 2.0 ** -22) if dtype == "f16" else (2.0 ** -113, 1.25 * 2.0 ** 126, 2.0 ** -118)
    top = float(torch.finfo(torch_dtype).max)
    rng = np.random.default_rng(9)
    sizes = np.concatenate([np.exp2(rng.uniform(np.log2(low) - 8, np.log2(low) + 2, 300)), np.exp2(rng.uniform(np.log2(high) - 3, np.log2(top), 300)),
                            [low, high, least, top]])
    g = rng.uniform(-1, 1, (len(sizes), 32))
    g[:, 3], g[::2, 5] = rng.choice([-1, 1], len(sizes)), -g[::2, 3]                   # one of the size, or both signs
    x = torch.tensor(np.clip(g * sizes[:, None], -top, top)).to(torch_dtype).double().numpy()
    codes, scales = quant.quantise(x, dtype)
    v, s, m = quant.values(codes, scales), np.abs(scales), np.abs(x).max(1, keepdims=True)
    first = np.where(x.max(1) == m[:, 0], x.argmax(1), x.argmin(1))[:, None]            # m: of two, the positive one
    v_m = np.abs(np.take_along_axis(v, first, 1))
    mine = np.sign(x) == np.sign(np.take_along_axis(x, first, 1))                      # on m's side of 0
    assert np.isfinite(v).all()
    mid, above, below = ((m >= low) & (m <= high))[:, 0], (m > high)[:, 0], (m < low)[:, 0]
    assert min(mid.sum(), above.sum(), below.sum()) > 60
    assert (np.abs(v_m - m) <= m / 32)[mid].all() and (np.take_along_axis(codes, first, 1) == 0)[mid].all()
    assert (np.abs(v - x) <= s * np.where(codes == 15, 1.25, 0.5))[mid].all()
    assert (np.abs(v) <= np.where(mine, high, 7 / 8 * high))[above].all() and (v_m == high)[above & (m[:, 0] > 33 / 32 * high)].all()
    assert (np.abs(v_m - m) <= least)[below].all()
    zeros = (m <= least)[:, 0]
    assert zeros.any() and (v[zeros] == 0).all() and (s[~zeros] > 0).all()


def test_planted_mistakes_show():
    x = torch.tensor(rows((50, 64), 7)).half().double().numpy()
    codes, scales = quant.quantise(x, "f16")
    assert np.abs(quant.values(codes, scales) - x).max() < 0.35
    assert np.abs(quant.values(codes, -scales) - x).max() > 1.0                        # the scale's sign lost
    assert np.abs(quant.values(quant.unpack(quant.pack(codes)[..., ::-1]), scales) - x).max() > 1.0
    swapped = codes.reshape(50, 32, 2)[..., ::-1].reshape(50, 64)                      # halves of a byte swapped
    assert np.abs(quant.values(swapped, scales) - x).max() > 1.0
