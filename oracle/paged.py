"""64-bit oracle of the operators around a paged cache: the page plan, the position rotation, norms of
query and key heads with their gradient, and decode over paged K and V. Plain numpy, row by row from the
definitions; it shares no code with the CUDA library. Where a comparison needs it, the functions also
return the magnitudes that rounding errors are proportional to."""
from __future__ import annotations

import math

import numpy as np


def plan(ctx, new, free, table, page, capacity):
    """(table, cu, seqlens, positions, slots, counts), request by request."""
    table = np.array(table, dtype=np.int64)
    cols = table.shape[1]
    cu, seqlens = [0], []
    positions, slots = np.zeros(capacity, np.int64), np.full(capacity, -1, np.int64)
    dealt = short = 0
    for r, (c, n) in enumerate(zip(ctx, new)):
        c, n = int(c), int(n)
        have = -(-c // page)
        need = -(-(c + n) // page) - have
        lacks = have + need > cols or (need > 0 and dealt + need > len(free))
        if not lacks:
            for k in range(need):
                table[r, have + k] = free[dealt + k]
        for j in range(n):
            at = cu[-1] + j
            if at >= capacity:
                break
            positions[at] = c + j
            if not lacks and table[r, (c + j) // page] >= 0:
                slots[at] = table[r, (c + j) // page] * page + (c + j) % page
        dealt += need
        short += lacks
        cu.append(cu[-1] + n)
        seqlens.append(c if lacks else c + n)
    return table, np.array(cu), np.array(seqlens), positions, slots, np.array([cu[-1], dealt, short])


def frequencies(dim, theta=10000.0, scaling=None, factor=1.0, original_max=4096, beta_fast=32.0, beta_slow=1.0):
    """Angles per position of dim / 2 pairs, and the scale of cos and sin."""
    half = dim // 2
    if scaling == "ntk":
        theta = theta * factor ** (dim / (dim - 2))
    out, scale = [], 1.0
    for i in range(half):
        f = theta ** (-2.0 * i / dim)
        if scaling == "linear":
            f = f / factor
        elif scaling == "yarn":
            # the pair whose frequency makes a given number of turns over the original length
            edge = [half * math.log(original_max / (2 * math.pi * b)) / math.log(theta) for b in (beta_fast, beta_slow)]
            lo, hi = max(0.0, math.floor(edge[0])), min(dim - 1.0, math.ceil(edge[1]))
            stretched = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f = f * (1 - stretched) + f / factor * stretched
            scale = 0.1 * math.log(factor) + 1.0
        out.append(f)
    return np.array(out), scale


def rotate(x, pos, freq, rope_off, interleaved, scale, transposed=False):
    """(rotated x, |terms| of each output): x [T, H, d] float64."""
    x = np.asarray(x, np.float64)
    y, size = x.copy(), np.abs(x)
    half = len(freq)
    for i in range(half):
        a = rope_off + (2 * i if interleaved else i)
        b = a + 1 if interleaved else a + half
        angle = np.asarray(pos, np.float64) * freq[i]
        c, s = np.cos(angle)[:, None] * scale, np.sin(angle)[:, None] * scale
        if transposed:
            s = -s
        y[:, :, a] = x[:, :, a] * c - x[:, :, b] * s
        y[:, :, b] = x[:, :, a] * s + x[:, :, b] * c
        size[:, :, a] = size[:, :, b] = (np.abs(x[:, :, a]) + np.abs(x[:, :, b])) * abs(scale)
    return y, size


def norm(x, w, norm_dim, eps):
    x = np.asarray(x, np.float64)
    y = x.copy()
    if w is not None:
        part = x[:, :, :norm_dim]
        y[:, :, :norm_dim] = part * w / np.sqrt(np.mean(part * part, axis=-1, keepdims=True) + eps)
    return y


def norm_rope(x, w, norm_dim, eps, pos, freq, rope_off, interleaved, scale):
    return rotate(norm(x, w, norm_dim, eps), pos, freq, rope_off, interleaved, scale)


def norm_rope_backward(x, dy, w, norm_dim, eps, pos, freq, rope_off, interleaved, scale):
    """(dx, |terms| of dx, dw, sum of |terms| of dw); dw is None without weight."""
    dn, dn_size = rotate(dy, pos, freq, rope_off, interleaved, scale, transposed=True)
    if w is None:
        return dn, dn_size, None, None
    x = np.asarray(x, np.float64)[:, :, :norm_dim]
    inv = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    u = x * inv
    g, gs = dn[:, :, :norm_dim] * w, dn_size[:, :, :norm_dim] * np.abs(w)
    dx, size = dn.copy(), dn_size.copy()
    dx[:, :, :norm_dim] = inv * (g - u * np.mean(g * u, axis=-1, keepdims=True))
    size[:, :, :norm_dim] = inv * (gs + np.abs(u) * np.mean(gs * np.abs(u), axis=-1, keepdims=True))
    return (dx, size, np.sum(dn[:, :, :norm_dim] * u, axis=(0, 1)),
            np.sum(dn_size[:, :, :norm_dim] * np.abs(u), axis=(0, 1)))


def window_keys(length, block, n_sink, n_local):
    """Visible keys of the last position of a sequence, by the block definition."""
    i = length - 1
    if n_local < 0:
        return list(range(length))
    j = i // block
    return [t for t in range(length) if t // block < n_sink or t // block > j - n_local]


def decode(q, k_pool, v_pool, table, lens, block, n_sink, n_local, scale):
    """(out, lse, |terms| of out, largest sum |q||k| scale of each head): q [B, H, d], pools [pages, rows, Hk, d],
    pages outside the pool hold no keys."""
    B, H, _ = q.shape
    pages, P, Hk, d_v = v_pool.shape
    out, size = np.zeros((B, H, d_v)), np.zeros((B, H, d_v))
    lse, dots = np.full((B, H), -np.inf), np.zeros((B, H))
    for n in range(B):
        keys = [t for t in window_keys(int(lens[n]), block, n_sink, n_local) if 0 <= table[n][t // P] < pages]
        if not keys:
            continue
        at = [int(table[n][t // P]) for t in keys]
        row = [t % P for t in keys]
        k, v = np.asarray(k_pool[at, row], np.float64), np.asarray(v_pool[at, row], np.float64)
        for h in range(H):
            kh = h // (H // Hk)
            z = k[:, kh] @ np.asarray(q[n, h], np.float64) * scale
            dots[n, h] = np.max(np.abs(k[:, kh]) @ np.abs(np.asarray(q[n, h], np.float64)) * abs(scale))
            top = z.max()
            p = np.exp(z - top)
            lse[n, h] = top + math.log(p.sum())
            p /= p.sum()
            out[n, h] = p @ v[:, kh]
            size[n, h] = p @ np.abs(v[:, kh])
    return out, lse, size, dots
