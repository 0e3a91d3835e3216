"""Pins of the 64-bit oracle of the paged operators (CPU): the plan against its own invariants, the
rotation against complex products and its inverse, the gradient against differences, the decode against
the SSA oracle's window and torch's attention."""
import math

import numpy as np
import pytest

from oracle import paged


def test_plan_invariants():
    g = np.random.default_rng(1)
    ctx, new, P = g.integers(0, 50, 40), g.integers(0, 60, 40), 8
    cols = int(((ctx + new + P - 1) // P).max())
    order = g.permutation(1000)
    have = (ctx + P - 1) // P
    table = np.full((40, cols), -1)
    used = 0
    for r in range(40):
        table[r, :have[r]] = order[used:used + have[r]]
        used += have[r]
    total = int(new.sum())
    t, cu, lens, pos, slots, counts = paged.plan(ctx, new, order[used:], table, P, total + 5)
    assert counts[0] == total and counts[2] == 0 and (lens == ctx + new).all()
    assert (slots[total:] == -1).all() and (pos[total:] == 0).all()
    assert len(set(slots[:total])) == total                 # every token its own slot
    held = t[t >= 0]
    assert len(set(held)) == len(held) == have.sum() + counts[1]
    for r in range(40):                                     # a token's slot is its position's row of its page
        for j in range(new[r]):
            p = ctx[r] + j
            assert pos[cu[r] + j] == p and slots[cu[r] + j] == t[r, p // P] * P + p % P


def test_plan_short_requests():
    t, cu, lens, pos, slots, counts = paged.plan([3, 4, 0, 8], [1, 1, 0, 4], [7], np.array([[5, -1, -1]] * 4), 4, 8)
    # request 0 fits its page; 1 takes page 7; 2 is idle; 3 would need page number 2 of a list of one
    assert list(lens) == [4, 5, 0, 8] and list(counts) == [6, 2, 1]
    assert list(slots) == [23, 28, -1, -1, -1, -1, -1, -1] and t[1, 1] == 7 and t[3, 2] == -1


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    g = np.random.default_rng(2)
    x, pos = g.standard_normal((5, 3, 20)), np.array([0, 1, 7, -3, 100000])
    freq, _ = paged.frequencies(12)
    y, _ = paged.rotate(x, pos, freq, 4, interleaved, 1.5)
    part, turned = x[..., 4:16], y[..., 4:16]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :6], part[..., 6:])
    c, d = (turned[..., 0::2], turned[..., 1::2]) if interleaved else (turned[..., :6], turned[..., 6:])
    want = (a + 1j * b) * 1.5 * np.exp(1j * pos[:, None, None] * freq)
    assert np.allclose(c + 1j * d, want, rtol=0, atol=1e-9)
    assert (y[..., :4] == x[..., :4]).all() and (y[..., 16:] == x[..., 16:]).all()
    back, _ = paged.rotate(y, pos, freq, 4, interleaved, 1 / 1.5, transposed=True)
    assert np.allclose(back, x, rtol=0, atol=1e-9)


def test_frequencies():
    f, s = paged.frequencies(64)
    assert s == 1.0 and f[0] == 1.0 and np.allclose(f[1:] / f[:-1], 10000 ** (-1 / 32))
    lin, _ = paged.frequencies(64, scaling="linear", factor=8)
    assert np.allclose(lin, f / 8)
    ntk, _ = paged.frequencies(64, scaling="ntk", factor=8)
    assert ntk[0] == 1.0 and np.isclose(ntk[-1], f[-1] / 8)  # the slowest pair is stretched by the whole factor
    yarn, s = paged.frequencies(64, scaling="yarn", factor=8)
    turns = 4096 * f / (2 * math.pi)
    assert np.allclose(yarn[turns > 40], f[turns > 40]) and np.allclose(yarn[turns < 0.8], f[turns < 0.8] / 8)
    assert (yarn <= f).all() and (yarn >= f / 8).all() and s == 0.1 * math.log(8) + 1


@pytest.mark.parametrize("norm_dim,weight", [(10, True), (6, True), (10, False)])
def test_gradient_against_differences(norm_dim, weight):
    g = np.random.default_rng(3)
    x, dy, pos = g.standard_normal((3, 2, 10)), g.standard_normal((3, 2, 10)), np.array([0, 5, 900])
    w = g.standard_normal(norm_dim) if weight else None
    freq, _ = paged.frequencies(4)
    args = (norm_dim, 1e-3, pos, freq, 3, False, 1.2)
    dx, _, dw, _ = paged.norm_rope_backward(x, dy, w, *args)
    h = 1e-5
    f = lambda x_, w_: float((paged.norm_rope(x_, w_, *args)[0] * dy).sum())
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[at]) < 1e-8
    if weight:
        for c in range(norm_dim):
            e = np.zeros_like(w)
            e[c] = h
            assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[c]) < 1e-8


@pytest.mark.parametrize("length", [1, 5, 128, 129, 1000, 1500])
def test_window_keys_match_the_kernels_form(length):
    for b, s, l in [(128, 1, 7), (1, 16, 1024), (64, 2, 5), (16, 0, 3)]:
        i = length - 1
        lo = max(0, (i // b - l + 1) * b)
        assert paged.window_keys(length, b, s, l) == [t for t in range(length) if t < s * b or t >= lo]


def test_decode_is_attention():
    import torch
    g = np.random.default_rng(4)
    B, H, Hk, d, P = 3, 6, 2, 8, 4
    lens = np.array([9, 0, 13])
    table = g.permutation(12).reshape(3, 4)
    k, v, q = g.standard_normal((12, P, Hk, d)), g.standard_normal((12, P, Hk, d)), g.standard_normal((B, H, d))
    out, lse, _, _ = paged.decode(q, k, v, table, lens, 128, 0, -1, 0.3)
    assert (out[1] == 0).all() and np.isneginf(lse[1]).all()
    for n in (0, 2):
        rows = [(table[n][t // P], t % P) for t in range(lens[n])]
        kk = np.stack([k[r] for r in rows]).repeat(H // Hk, axis=1)
        vv = np.stack([v[r] for r in rows]).repeat(H // Hk, axis=1)
        want = torch.nn.functional.scaled_dot_product_attention(
            torch.tensor(q[n])[:, None], torch.tensor(kk).transpose(0, 1), torch.tensor(vv).transpose(0, 1),
            scale=0.3)[:, 0]
        assert np.allclose(out[n], want.numpy(), atol=1e-12)
