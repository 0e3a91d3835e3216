"""GPU parity of the paged operators with the 64-bit oracle on the same bits, at the sizes, layouts and
masks where they can go wrong. Bounds are derived, not measured: a rounding to the output's type is half
a step (finfo.eps / 2 of the value), and the 32-bit arithmetic before it is bounded by a count of 2^-24
steps times the magnitude of the terms, which the oracle returns beside each value."""
import ctypes
import math

import numpy as np
import pytest
import torch

from helpers import record
from oracle import paged

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
STEP = 2.0 ** -24


@pytest.fixture(scope="module")
def bss():
    import block_sparse_streaming_b200 as m
    m.build()
    return m


def f64(t):
    return t.detach().cpu().double().numpy()


def normal(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def close(got, want, slack, what):
    """|got - want| <= slack (32-bit arithmetic) + the rounding to got's type."""
    eps = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).smallest_normal * eps * 2  # half a step among the subnormals
    err, rounding = np.abs(f64(got) - want), eps * (np.abs(want) + slack) + tiny
    assert np.isfinite(f64(got)).all(), what
    if err.size:  # what the arithmetic took of its share (the rounding always takes nearly all of its own)
        record(what, "arithmetic", float(((err - rounding).clip(0) / np.maximum(slack, tiny)).max()), 1.0)
    assert (err <= slack + rounding).all(), f"{what}: {float((err / (slack + rounding)).max()):.3g} of the bound"


# ---------------------------------------------------------------------------
# Page plan
# ---------------------------------------------------------------------------
def plan_case(seed, B, page, ctx_hi, new_hi, extra_cols=0, zeros=0.0, holes=False):
    g = np.random.default_rng(seed)
    ctx, new = g.integers(0, ctx_hi + 1, B), g.integers(0, new_hi + 1, B)
    new[g.random(B) < zeros] = 0
    have, total = -(-ctx // page), -(-(ctx + new) // page)
    table = np.full((B, max(1, int(total.max())) + extra_cols), -7)
    order = g.permutation(int(total.sum()) + 3)
    used = 0
    for r in range(B):
        table[r, :have[r]] = order[used:used + have[r]]
        used += have[r]
        if holes and have[r] > 1:
            table[r, 0] = -1  # handed back
    return ctx, new, order[used:], table


def run_plan(bss, ctx, new, free, table, page, capacity, strided=False):
    dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    t = dev(table)
    if strided:  # rows of a wider table: what lies beside them stays as it was
        wide = torch.full((t.shape[0], t.shape[1] + 5), 99, dtype=torch.int32, device="cuda")
        wide[:, :t.shape[1]] = t
        t = wide[:, :table.shape[1]]
    got = bss.loza_page_plan(dev(ctx), dev(new), dev(free), t, page, capacity)
    torch.cuda.synchronize()
    if strided:
        assert (wide[:, table.shape[1]:] == 99).all()
    return t, got


@pytest.mark.parametrize("B,page,ctx_hi,new_hi,zeros,strided", [
    (1, 16, 0, 1, 0.0, False), (1, 1, 5, 9, 0.0, False), (7, 16, 40, 33, 0.5, True), (255, 128, 2000, 1, 0.3, False),
    (256, 32, 70, 64, 0.0, True), (257, 16, 100, 17, 0.2, False), (1000, 64, 300, 5, 0.9, False),
    (3, 65536, 70000, 131073, 0.0, False), (5, 16, 0, 0, 1.0, False)])
def test_plan(bss, B, page, ctx_hi, new_hi, zeros, strided):
    ctx, new, free, table = plan_case(B + page, B, page, ctx_hi, new_hi, 2, zeros, holes=B > 4)
    for capacity in {int(new.sum()), int(new.sum()) + 13, max(0, int(new.sum()) - 3)}:
        want = paged.plan(ctx, new, free, table, page, capacity)
        t, got = run_plan(bss, ctx, new, free, table, page, capacity, strided)
        for g, w, name in zip((t,) + got, want, ("table", "cu", "seqlens", "positions", "slots", "counts")):
            assert np.array_equal(g.cpu().numpy(), w), name


def test_plan_of_many_requests(bss):
    ctx, new, free, table = plan_case(9, 16384, 16, 40, 3)
    want = paged.plan(ctx, new, free, table, 16, int(new.sum()))
    t, got = run_plan(bss, ctx, new, free, table, 16, int(new.sum()))
    for g, w in zip((t,) + got, want):
        assert np.array_equal(g.cpu().numpy(), w)


def test_plan_short_of_pages(bss):
    """Requests that the free list or the table cannot hold get nothing; nothing outside their rows changes."""
    for cut, cols in ((10, 0), (0, 0), (10**6, 3)):
        ctx, new, free, table = plan_case(11, 60, 16, 90, 70)
        free = free[:cut] if cut < len(free) else free
        if cols:
            table = table[:, :cols]
        want = paged.plan(ctx, new, free, table, 16, int(new.sum()) + 1)
        assert want[5][2] > 0
        t, got = run_plan(bss, ctx, new, free, table, 16, int(new.sum()) + 1, strided=True)
        for g, w in zip((t,) + got, want):
            assert np.array_equal(g.cpu().numpy(), w)


def test_plan_bad_lengths_count_as_zero(bss):
    ctx, new = np.array([5, -1, 1 << 30, 7]), np.array([3, 4, 2, -(1 << 31)])
    table, free = np.full((4, 6), -1), np.arange(20, 40)
    table[0, 0] = table[3, 0] = 3
    want = paged.plan([5, 0, 0, 7], [3, 4, 2, 0], free, table, 8, 12)
    t, got = run_plan(bss, ctx, new, free, table, 8, 12)
    for g, w in zip((t,) + got, want):
        assert np.array_equal(g.cpu().numpy(), w)
    # sums past 31 bits are saturated and reported as short, nothing is written out of place
    big = np.full(8, (1 << 30) - 1)
    t, got = run_plan(bss, big, big, free, np.full((8, 6), -1), 8, 12)
    assert (t.cpu().numpy() == -1).all() and (got[3].cpu().numpy() == -1).all()
    assert got[4].cpu().tolist()[0] == 2**31 - 1 and got[4].cpu().tolist()[2] == 8


# ---------------------------------------------------------------------------
# Rotation and norm
# ---------------------------------------------------------------------------
ROPES = [  # d, rope_dim, rope_off, norm_dim
    (64, 64, 0, 64), (128, 128, 0, 128), (192, 64, 128, 192), (576, 64, 512, 512), (128, 64, 32, 128), (80, 20, 60, 60),
    (100, 24, 75, 75), (256, 2, 1, 3), (1024, 1024, 0, 1024), (1023, 1022, 1, 1023), (7, 6, 0, 7), (2, 2, 0, 2),
    (1, 0, 0, 1), (96, 0, 0, 96)]


def rope_inputs(bss, seed, T, dim, far=True):
    g = np.random.default_rng(seed)
    pos = g.integers(0, 1 << 20, T)
    pos[:3] = [0, 1, (1 << 20) + 1][:min(3, T)]
    if T > 4:
        pos[3], pos[4] = -5, 2**31 - 1
    freq = paged.frequencies(dim, scaling="yarn", factor=4.0)[0] if dim else np.zeros(0)
    return pos, freq, torch.tensor(pos, dtype=torch.int32, device="cuda"), torch.tensor(freq, device="cuda")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", ROPES, ids=str)
@pytest.mark.parametrize("T,H,interleaved", [(5, 3, False), (13, 8, True), (0, 2, False), (1, 1, True)])
def test_rope(bss, dtype, shape, T, H, interleaved):
    d, dim, off, _ = shape
    pos, freq, pos_d, freq_d = rope_inputs(bss, d + T, T, dim)
    x = normal(d + H, T, H, d, dtype=DTYPES[dtype])
    rope = bss.RopeParams(dim, off, interleaved, 1.25)
    for transposed in (False, True):
        want, size = paged.rotate(f64(x), pos, freq, off, interleaved, float(np.float32(1.25)), transposed)
        y = bss.loza_rope(x, pos_d, freq_d, rope, transposed=transposed)
        # per term: the angle's rounding 2 pi 2^-26, two steps each of sin and cos and of scaling, product and sum: < 12
        close(y, want, 12 * STEP * size, f"rope {dtype} {shape}")
    z = x.clone()
    assert bss.loza_rope(z, pos_d, freq_d, rope, out=z) is z
    assert torch.equal(z, bss.loza_rope(x, pos_d, freq_d, rope))  # in place: the same bits


def test_rope_strided_rows(bss):
    """Slices of a wider row, aligned and not; what lies between the rows stays as it was."""
    for lead in (0, 8, 3):
        rows = normal(5, 9, 1000 + lead, dtype=torch.bfloat16)
        x = rows[:, lead:lead + 4 * 128].view(9, 4, 128)
        pos, freq, pos_d, freq_d = rope_inputs(bss, 6, 9, 64)
        rope = bss.RopeParams(64, 64, False)
        want, size = paged.rotate(f64(x), pos, freq, 64, False, 1.0)
        close(bss.loza_rope(x, pos_d, freq_d, rope), want, 12 * STEP * size, "rope strided")
        before = rows.clone()
        bss.loza_rope(x, pos_d, freq_d, rope, out=x)
        close(x, want, 12 * STEP * size, "rope strided in place")
        rows[:, lead:lead + 512] = before[:, lead:lead + 512]
        assert torch.equal(rows, before)


def norm_slack(w, n, size, d):
    """40 steps of the terms: the sum of squares (at most 32 + 5 additions, halved by the root), rsqrt (4), two
    products, and the rotation's 12."""
    return 40 * STEP * size


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", ROPES, ids=str)
@pytest.mark.parametrize("T,H,Hk,interleaved", [(6, 5, 2, False), (11, 8, 8, True), (1, 1, 1, False), (3, 64, 1, True)])
def test_norm_rope(bss, dtype, shape, T, H, Hk, interleaved):
    d, dim, off, nd = shape
    dt = DTYPES[dtype]
    pos, freq, pos_d, freq_d = rope_inputs(bss, d + T, T, dim)
    rows = normal(T + d, T, (H + Hk) * d, dtype=dt, scale=3.0)
    q, k = rows[:, :H * d].view(T, H, d), rows[:, H * d:].view(T, Hk, d)
    qw, kw = normal(1, nd, dtype=dt) + 1, normal(2, nd, dtype=dt) + 1
    rope, eps = bss.RopeParams(dim, off, interleaved, 0.75), 1e-5
    for a, b in ((qw, kw), (None, kw), (qw, None), (None, None)):
        qo, ko = bss.loza_qk_norm_rope(q, k, pos_d, freq_d, rope, a, b, eps)
        for x, w, y, s in ((q, a, qo, "q"), (k, b, ko, "k")):
            want, size = paged.norm_rope(f64(x), None if w is None else f64(w), nd, float(np.float32(eps)), pos, freq,
                                         off, interleaved, 0.75)
            close(y, want, norm_slack(w, nd, size, d), f"norm_rope {s} {dtype} {shape}")
    # each side alone, and in place: the same bits
    both = bss.loza_qk_norm_rope(q, k, pos_d, freq_d, rope, qw, None, eps)
    assert torch.equal(bss.loza_qk_norm_rope(q, None, pos_d, freq_d, rope, qw, None, eps)[0], both[0])
    assert torch.equal(bss.loza_qk_norm_rope(None, k, pos_d, freq_d, rope, None, None, eps, norm_dim=nd)[1], both[1])
    bss.loza_qk_norm_rope(q, k, pos_d, freq_d, rope, qw, None, eps, q_out=q, k_out=k)
    assert torch.equal(q, both[0]) and torch.equal(k, both[1])


def test_norm_of_zero_and_huge_rows(bss):
    """A row of zeros gives zeros (eps keeps the root away from 0); rows near the 16-bit limits stay right."""
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    x[1] = 2.0 ** 50
    x[2] = 2.0 ** -60
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    pos, freq, pos_d, freq_d = rope_inputs(bss, 1, 3, 0)
    y, _ = bss.loza_qk_norm_rope(x, None, pos_d, freq_d, bss.RopeParams(0), w, None, 1e-6)
    assert (y[0] == 0).all() and (y[1] == 1).all()
    close(y[2:], np.full((1, 2, 64), 2.0 ** -60 / 1e-3), 1e-6 * 2.0 ** -60 / 1e-3, "tiny row")
    x[0, 0, 3] = float("nan")  # a bad row stays bad, its neighbours are untouched
    y, _ = bss.loza_qk_norm_rope(x, None, pos_d, freq_d, bss.RopeParams(0), w, None, 1e-6)
    assert torch.isnan(y[0, 0]).all() and (y[0, 1] == 0).all() and (y[1] == 1).all()


def pool_layouts(pages, P, Hk, d, dtype, fill):
    """The same pool as [pages, rows, heads, d], heads before rows, and beside another one."""
    nhd = torch.full((pages, P, Hk, d), fill, dtype=dtype, device="cuda")
    hnd = torch.full((pages, Hk, P, d), fill, dtype=dtype, device="cuda").transpose(1, 2)
    both = torch.full((pages, 2, P, Hk, d), fill, dtype=dtype, device="cuda")[:, 1]
    return {"nhd": nhd, "hnd": hnd, "pair": both}


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("d,d_v,nd,dim,off,P", [(128, 128, 128, 128, 0, 16), (192, 128, 192, 64, 128, 64),
                                                (576, 0, 512, 64, 512, 128), (100, 60, 75, 24, 75, 1),
                                                (64, 64, 64, 32, 0, 256)])
def test_norm_rope_into_pool(bss, dtype, d, d_v, nd, dim, off, P):
    dt, T, H, Hk = DTYPES[dtype], 21, 4, 1 if d == 576 else 3
    pages = 40 // P + 3
    pos, freq, pos_d, freq_d = rope_inputs(bss, d, T, dim)
    q, k = normal(1, T, H, d, dtype=dt), normal(2, T, Hk, d, dtype=dt)
    v = normal(3, T, Hk, d_v, dtype=dt) if d_v else None
    kw = normal(4, nd, dtype=dt) + 1
    g = np.random.default_rng(d)
    slots = g.permutation(pages * P)[:T]
    slots[4], slots[9], slots[10] = -1, pages * P, 2**40  # padded rows, and rows that are not there
    slots_d = torch.tensor(slots, device="cuda")
    rope = bss.RopeParams(dim, off, True)
    _, k_ref = bss.loza_qk_norm_rope(q, k, pos_d, freq_d, rope, None, kw, 1e-6)
    keep = [t for t in range(T) if 0 <= slots[t] < pages * P]
    for name, kp in pool_layouts(pages, P, Hk, d, dt, 7.0).items():
        vp = pool_layouts(pages, P, Hk, d_v, dt, 9.0)[name] if d_v else None
        qo, ko = bss.loza_qk_norm_rope(q, k, pos_d, freq_d, rope, None, kw, 1e-6, v=v, k_pool=kp, v_pool=vp,
                                       slots=slots_d, k_out=torch.empty_like(k) if name == "hnd" else None)
        assert ko is None or torch.equal(ko, k_ref)
        want = torch.full((pages * P, Hk, d), 7.0, dtype=dt, device="cuda")
        want[slots_d[keep]] = k_ref[keep]
        assert torch.equal(kp.reshape(pages * P, Hk, d), want), name
        if d_v:
            want = torch.full((pages * P, Hk, d_v), 9.0, dtype=dt, device="cuda")
            want[slots_d[keep]] = v[keep]
            assert torch.equal(vp.reshape(pages * P, Hk, d_v), want), name


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", ROPES, ids=str)
@pytest.mark.parametrize("T,H,Hk,interleaved", [(6, 5, 2, True), (1, 1, 1, False), (700, 4, 4, False)])
def test_norm_rope_backward(bss, dtype, shape, T, H, Hk, interleaved):
    d, dim, off, nd = shape
    if T > 100 and d > 200:
        T = 90
    dt = DTYPES[dtype]
    pos, freq, pos_d, freq_d = rope_inputs(bss, d + T, T, dim)
    q, k = normal(1, T, H, d, dtype=dt, scale=2.0), normal(2, T, Hk, d, dtype=dt)
    gq, gk = normal(3, T, H, d, dtype=dt), normal(4, T, Hk, d, dtype=dt)
    qw, kw = normal(5, nd, dtype=dt) + 1, normal(6, nd, dtype=dt) + 1
    rope, eps = bss.RopeParams(dim, off, interleaved, 1.5), 1e-5
    for a, b in ((qw, kw), (qw, None), (None, None)):
        dq, dk, dqw, dkw = bss.loza_qk_norm_rope_backward(gq, gk, q, k, pos_d, freq_d, rope, a, b, eps)
        for x, dy, w, dx, dw, s in ((q, gq, a, dq, dqw, "q"), (k, gk, b, dk, dkw, "k")):
            want, size, want_w, size_w = paged.norm_rope_backward(
                f64(x), f64(dy), None if w is None else f64(w), nd, float(np.float32(eps)), pos, freq, off,
                interleaved, 1.5)
            # the rotation (12), the root (25), products and the mean's sum (37 + 6): < 96 steps of the terms
            close(dx, want, 96 * STEP * size, f"bwd {s} {dtype} {shape}")
            assert (dw is None) == (w is None)
            if w is not None:
                # each term 48 steps, and one step per addition: at most one per row
                close(dw, want_w, (48 + x.shape[0] * x.shape[1]) * STEP * size_w, f"bwd {s}_weight {dtype} {shape}")
    again = bss.loza_qk_norm_rope_backward(gq, gk, q, k, pos_d, freq_d, rope, qw, kw, eps)
    once = bss.loza_qk_norm_rope_backward(gq, gk, q, k, pos_d, freq_d, rope, qw, kw, eps)
    assert all(torch.equal(x, y) for x, y in zip(again, once))
    alone = bss.loza_qk_norm_rope_backward(None, gk, None, k, pos_d, freq_d, rope, None, kw, eps)
    assert alone[0] is None and alone[2] is None and torch.equal(alone[1], once[1])
    place = gq.clone(), k.clone()  # gradients in the place of their inputs
    bss.loza_qk_norm_rope_backward(place[0], gk, q, place[1], pos_d, freq_d, rope, qw, kw, eps, dq=place[0], dk=place[1])
    assert torch.equal(place[0], once[0]) and torch.equal(place[1], once[1])


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,dim,off,nd", [(8, 4, 2, 6), (66, 60, 4, 66), (128, 128, 0, 128), (514, 260, 10, 500),
                                          (1022, 1020, 2, 1022)])
def test_rows_of_four_byte_alignment(bss, dtype, interleaved, d, dim, off, nd):
    """Head slices that begin two elements into their rows, and head dims that 16-byte vectors do not fit: rotation,
    norm, cache write and gradient, all in place of slices of one buffer, whose other columns stay as they were."""
    dt, T, H, Hk = DTYPES[dtype], 19, 3, 2
    pos, freq, pos_d, freq_d = rope_inputs(bss, d, T, dim)
    rope, eps = bss.RopeParams(dim, off, interleaved, 0.5), 1e-5
    wide = (H + 2 * Hk) * d + 6
    rows = normal(d, T, wide, dtype=dt)
    cut = lambda r: (r[:, 2:2 + H * d].view(T, H, d), r[:, 4 + H * d:4 + (H + Hk) * d].view(T, Hk, d),
                     r[:, 4 + (H + Hk) * d:4 + (H + 2 * Hk) * d].view(T, Hk, d))
    q, k, v = cut(rows)
    qw, kw = normal(1, nd + 2, dtype=dt)[2:] + 1, normal(2, nd, dtype=dt) + 1
    want_r, size_r = paged.rotate(f64(q), pos, freq, off, interleaved, 0.5)
    close(bss.loza_rope(q, pos_d, freq_d, rope), want_r, 12 * STEP * size_r, "rope 4-byte")
    want = [paged.norm_rope(f64(x), f64(w), nd, float(np.float32(eps)), pos, freq, off, interleaved, 0.5)
            for x, w in ((q, qw), (k, kw))]
    back = [paged.norm_rope_backward(f64(x), f64(x), f64(w), nd, float(np.float32(eps)), pos, freq, off, interleaved,
                                     0.5) for x, w in ((q, qw), (k, kw))]
    grads = rows.clone()
    gq, gk, _ = cut(grads)
    _, _, dqw, dkw = bss.loza_qk_norm_rope_backward(gq, gk, q, k, pos_d, freq_d, rope, qw, kw, eps, dq=gq, dk=gk)
    for dx, dw, (wx, sx, ww, sw), x in ((gq, dqw, back[0], q), (gk, dkw, back[1], k)):
        close(dx, wx, 96 * STEP * sx, "bwd 4-byte")
        close(dw, ww, (48 + T * x.shape[1]) * STEP * sw, "bwd weight 4-byte")
    place = rows.clone()
    pq, pk, pv = cut(place)
    pool = torch.full((2, 2, 16, Hk, d), 5.0, dtype=dt, device="cuda")
    slots = torch.arange(T, device="cuda") + 7
    bss.loza_qk_norm_rope(pq, pk, pos_d, freq_d, rope, qw, kw, eps, v=pv, k_pool=pool[:, 0], v_pool=pool[:, 1],
                          slots=slots, q_out=pq, k_out=pk)
    for x, (wx, sx) in ((pq, want[0]), (pk, want[1])):
        close(x, wx, norm_slack(None, nd, sx, d), "norm_rope 4-byte")
    flat = [pool[:, i].reshape(32, Hk, d) for i in range(2)]
    assert torch.equal(flat[0][slots], pk) and torch.equal(flat[1][slots], v)
    rest = [i for i in range(32) if not 7 <= i < 7 + T]
    assert (flat[0][rest] == 5).all() and (flat[1][rest] == 5).all()
    for buf in (grads, place):  # between and beside the slices
        for x, y in zip(cut(buf)[:2], (q, k)):
            x.copy_(y)
        assert torch.equal(buf, rows)


def test_rows_far_apart(bss):
    """Rows whose offsets pass 2^31 elements and 2^32 bytes, forward and backward."""
    T, H, d, stride = 1100, 2, 64, 1 << 21
    buf = torch.empty(T * stride, dtype=torch.bfloat16, device="cuda").view(T, stride)
    pos, freq, pos_d, freq_d = rope_inputs(bss, 4, T, d)
    rope = bss.RopeParams(d)
    x, dy = normal(1, T, H, d, dtype=torch.bfloat16), normal(2, T, H, d, dtype=torch.bfloat16)
    w = normal(3, d, dtype=torch.bfloat16) + 1
    cut = lambda i: buf[:, i * H * d:(i + 1) * H * d].view(T, H, d)
    cut(0).copy_(x)
    cut(1).copy_(dy)
    bss.loza_rope(cut(0), pos_d, freq_d, rope, out=cut(2))
    bss.loza_qk_norm_rope(cut(0), None, pos_d, freq_d, rope, w, q_out=cut(3))
    far = bss.loza_qk_norm_rope_backward(cut(1), None, cut(0), None, pos_d, freq_d, rope, w, dq=cut(4))
    near = bss.loza_qk_norm_rope_backward(dy, None, x, None, pos_d, freq_d, rope, w)
    assert torch.equal(cut(2), bss.loza_rope(x, pos_d, freq_d, rope))
    assert torch.equal(cut(3), bss.loza_qk_norm_rope(x, None, pos_d, freq_d, rope, w)[0])
    assert torch.equal(cut(4), near[0]) and torch.equal(far[2], near[2])


@pytest.mark.parametrize("dtype,H,Hk,d,weights,T", [
    ("bf16", 32, 0, 128, False, 7201), ("bf16", 32, 8, 128, False, 3601), ("fp32", 32, 8, 128, True, 3555),
    ("bf16", 64, 8, 128, True, 7150), ("fp16", 24, 1, 576, True, 3003), ("bf16", 8, 8, 64, True, 5003)])
def test_tokens_are_dealt_in_any_way(bss, dtype, H, Hk, d, weights, T):
    """Many tokens (equal shares, or short walks dealt out one after another) give the bits of the same tokens a few
    at a time, which the tests above compare with the oracle; rows behind the last token stay as they were."""
    dt = DTYPES[dtype]
    pos, freq, pos_d, freq_d = rope_inputs(bss, 9, T, 64)
    rope = bss.RopeParams(64, d - 64, True)
    q = normal(1, T, H, d, dtype=dt)
    k, v = (normal(s, T, Hk, d, dtype=dt) for s in (2, 3)) if Hk else (None, None)
    w = normal(4, d, dtype=dt) + 1 if weights else None
    slots = torch.randperm(T + 20, generator=torch.Generator().manual_seed(5)).cuda()[:T]

    def run(a, b, q_out, k_pool, v_pool):
        if not Hk:
            return bss.loza_rope(q[a:b], pos_d[a:b], freq_d, rope, out=q_out[a:b])
        bss.loza_qk_norm_rope(q[a:b], k[a:b], pos_d[a:b], freq_d, rope, w, w, v=v[a:b], k_pool=k_pool, v_pool=v_pool,
                              slots=slots[a:b], q_out=q_out[a:b])

    def fresh():
        pages = -(-(T + 20) // 16)
        return (torch.full((T + 8, H, d), 3.0, dtype=dt, device="cuda"),
                *(torch.full((pages, 16, max(Hk, 1), d), 4.0, dtype=dt, device="cuda") for _ in range(2)))

    once, parts = fresh(), fresh()
    run(0, T, *once)
    for a in range(0, T, 400):
        run(a, min(a + 400, T), *parts)
    assert all(torch.equal(x, y) for x, y in zip(once, parts))
    assert (once[0][T:] == 3).all()


def test_captured_rotation_and_gradient_on_two_streams(bss):
    """Rotation, norm and gradient captured on two streams with buffers of their own (the gradient's workspace, made
    inside the capture, among them), replayed at the same time over new inputs: the bits of calls made one by one."""
    T, H, Hk, d = 900, 8, 2, 128
    pos, freq, pos_d, freq_d = rope_inputs(bss, 8, T, d)
    rope = bss.RopeParams(d)
    w = normal(1, d, dtype=torch.bfloat16) + 1
    make = lambda s: [normal(s + i, T, n, d, dtype=torch.bfloat16) for i, n in enumerate((H, Hk, H, Hk))]

    def run(q, k, gq, gk):
        return (bss.loza_rope(q, pos_d, freq_d, rope, transposed=True), *bss.loza_qk_norm_rope(
            q, k, pos_d, freq_d, rope, w, w), *bss.loza_qk_norm_rope_backward(gq, gk, q, k, pos_d, freq_d, rope, w, w))

    runs = []
    for i in range(2):
        st, x = torch.cuda.Stream(), make(10 * i)
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            run(*x)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            out = run(*x)
        runs.append((st, g, x, out))
    for seed in (100, 200):
        for i, (_, _, x, _) in enumerate(runs):
            for a, b in zip(x, make(seed + 10 * i)):
                a.copy_(b)
        torch.cuda.synchronize()
        for _ in range(20):
            for st, g, *_rest in runs:
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for _, _, x, out in runs:
            assert all(torch.equal(a, b) for a, b in zip(out, run(*x)))


def test_norm_rope_backward_of_no_tokens(bss):
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")
    pos, freq, pos_d, freq_d = rope_inputs(bss, 1, 0, 64)
    out = bss.loza_qk_norm_rope_backward(e(0, 4, 64), e(0, 2, 64), e(0, 4, 64), e(0, 2, 64), pos_d, freq_d,
                                         bss.RopeParams(64), torch.ones(64, dtype=torch.bfloat16, device="cuda"), None)
    assert out[0].shape == (0, 4, 64) and (out[2] == 0).all() and out[3] is None


def test_gradient_against_differences_of_the_kernel(bss):
    """<dy, F(x + h e) - F(x - h e)> / 2h of the 32-bit forward kernel against the backward kernel's <dx, e>. Their
    distance is at most the forward's rounding over h (40 steps of each output), the curvature (the oracle's
    difference at the same h against its gradient) and the gradient's own bound."""
    T, H, d, dim, off = 9, 3, 64, 32, 16
    pos, freq, pos_d, freq_d = rope_inputs(bss, 3, T, dim)
    x, dy, ex = (normal(s, T, H, d) for s in (1, 2, 3))
    w, ew = normal(4, d) + 1, normal(5, d)
    rope, eps, h = bss.RopeParams(dim, off), float(np.float32(1e-5)), 2.0 ** -8
    dx, _, dw, _ = bss.loza_qk_norm_rope_backward(dy, None, x, None, pos_d, freq_d, rope, w, None, eps)
    args = (d, eps, pos, freq, off, False, 1.0)
    dx64, dx_size, dw64, dw_size = paged.norm_rope_backward(f64(x), f64(dy), f64(w), *args)
    steps = ((dx, dx64, 96 * STEP * dx_size, ex, (x + h * ex, w), (x - h * ex, w)),
             (dw, dw64, (48 + T * H) * STEP * dw_size, ew, (x, w + h * ew), (x, w - h * ew)))
    for got, want, slack, e, plus, minus in steps:
        kernel = [f64(bss.loza_qk_norm_rope(a, None, pos_d, freq_d, rope, b, None, eps)[0]) for a, b in (plus, minus)]
        truth = [paged.norm_rope(f64(a), f64(b), *args) for a, b in (plus, minus)]
        # the steps x +- h e are themselves rounded: the oracle takes the rounded ones
        diff = (f64(dy) * (kernel[0] - kernel[1])).sum() / (2 * h)
        exact = (f64(dy) * (truth[0][0] - truth[1][0])).sum() / (2 * h)
        rounding = 40 * STEP * (np.abs(f64(dy)) * (truth[0][1] + truth[1][1])).sum() / (2 * h)
        curvature = abs(exact - (want * f64(e)).sum())
        assert abs(diff - (f64(got) * f64(e)).sum()) <= rounding + curvature + (slack * np.abs(f64(e))).sum()


# ---------------------------------------------------------------------------
# Decode over paged K and V
# ---------------------------------------------------------------------------
WINDOWS = {"full": (128, 0, -1), "blocks": (128, 1, 7), "tokens": (1, 16, 1024), "small": (16, 2, 3), "one": (1, 0, 1)}


def decode_case(seed, lens, H, Hk, d, d_v, P, dtype, spare=2):
    g = np.random.default_rng(seed)
    need = [-(-L // P) for L in lens]
    pages = sum(need) + spare
    order = g.permutation(pages)
    cols = max(1, max(need))
    table = np.full((len(lens), cols), -1)
    used = 0
    for n, c in enumerate(need):
        table[n, :c] = order[used:used + c]
        used += c
    dt = DTYPES[dtype]
    return (normal(seed, len(lens), H, d, dtype=dt), normal(seed + 1, pages, P, Hk, d, dtype=dt),
            normal(seed + 2, pages, P, Hk, d_v, dtype=dt), table)


def check_decode(got, q, k, v, table, lens, window, scale, what):
    out, lse = got
    b, s, l = window
    want, want_lse, size, dots = paged.decode(f64(q), f64(k), f64(v), table, lens, b, s, l, scale)
    empty = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(f64(lse)), empty), what
    assert (f64(out)[empty] == 0).all(), what
    # logits: products and sums of the matrix unit, two truncated 2^-23 steps per 16 columns, and scaling; a logit's
    # error is a weight's relative error. Weights: ex2 2^-22, P as two 16-bit parts 2^-16 of it squared away, the
    # sums one step per step of 64 keys and a few dozen joins
    keys = max([1] + list(lens))
    dz = (q.shape[2] / 8 + 8) * 2.0 ** -23 * dots
    rel = 2 * dz + (keys / 64 + 64) * 2.0 ** -23 + 2.0 ** -16
    close(out, want, rel[..., None] * size, what)
    slack = dz + (keys / 64 + 64) * 2.0 ** -23 + 2.0 ** -22 * np.abs(np.where(empty, 0, want_lse))
    err = np.abs(f64(lse)[~empty] - want_lse[~empty])
    assert (err <= slack[~empty]).all(), what
    if err.size:
        record(what, "lse err/bound", float((err / slack[~empty]).max()), 1.0)


HEADS = [(8, 8), (32, 8), (28, 4), (16, 1), (9, 1), (71, 1), (40, 40)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,d_v", [(64, 64), (128, 128), (192, 128)])
@pytest.mark.parametrize("H,Hk", HEADS)
def test_decode_shapes(bss, dtype, d, d_v, H, Hk):
    lens = [300, 1, 0, 64, 65, 777]
    q, k, v, table = decode_case(d + H, lens, H, Hk, d, d_v, 16, dtype)
    got = bss.loza_ssa_decode_paged_kv(q, k, v, torch.tensor(table, dtype=torch.int32, device="cuda"),
                                       torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens),
                                       bss.Params(d ** -0.5, 128, 0, -1))
    check_decode(got, q, k, v, table, lens, (128, 0, -1), float(np.float32(d ** -0.5)), f"decode {d} {H}/{Hk} {dtype}")


@pytest.mark.parametrize("window", list(WINDOWS))
@pytest.mark.parametrize("P", [16, 64, 128, 1024])
@pytest.mark.parametrize("lens", [[1], [2300], [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 1023, 1024, 1025, 1153],
                                  [0, 0, 0], [40] * 33], ids=lambda v: f"{len(v)}x{max(v)}")
def test_decode_windows_and_lengths(bss, window, P, lens):
    b, s, l = WINDOWS[window]
    H, Hk, d = (8, 2, 128) if len(lens) < 20 else (4, 4, 64)
    d_v = d
    q, k, v, table = decode_case(P + len(lens), lens, H, Hk, d, d_v, P, "bf16")
    got = bss.loza_ssa_decode_paged_kv(q, k, v, torch.tensor(table, dtype=torch.int32, device="cuda"),
                                       torch.tensor(lens, dtype=torch.int32, device="cuda"), max(1, max(lens)),
                                       bss.Params(0.1, b, s, l))
    check_decode(got, q, k, v, table, lens, (b, s, l), float(np.float32(0.1)), f"decode {window} P={P}")


def test_decode_reads_nothing_that_is_masked(bss):
    """Rows past the length, outside the window, and whole pages of nobody hold NaN and infinities; freed pages are
    -1 or out of range. The result is bit for bit that of a clean pool."""
    lens, P = [1500, 77, 2047, 1, 0], 16
    for window in WINDOWS.values():
        b, s, l = window
        q, k, v, table = decode_case(3, lens, 8, 2, 128, 128, P, "bf16", spare=5)
        bad = torch.ones(k.shape[0] * P, dtype=torch.bool)
        for n, L in enumerate(lens):
            keys = paged.window_keys(L, b, s, l) if L else []
            for t in keys:
                bad[table[n][t // P] * P + t % P] = False
            for c in range(table.shape[1]):  # hand back the pages without a visible key
                if not any(t // P == c for t in keys):
                    table[n, c] = (-1, -2**31, k.shape[0], 2**31 - 1)[c % 4]
        t_d, l_d = torch.tensor(table, dtype=torch.int32, device="cuda"), torch.tensor(lens, dtype=torch.int32).cuda()
        p = bss.Params(0.08, b, s, l)
        clean = bss.loza_ssa_decode_paged_kv(q, k, v, t_d, l_d, 2047, p)
        kb, vb = k.clone(), v.clone()
        kb.view(-1, 2, 128)[bad.cuda()] = float("nan")
        vb.view(-1, 2, 128)[bad.cuda()] = float("inf")
        dirty = bss.loza_ssa_decode_paged_kv(q, kb, vb, t_d, l_d, 2047, p)
        assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])
        check_decode(dirty, q, k, v, table, lens, window, float(np.float32(0.08)), "decode masked")


def test_decode_with_missing_pages(bss):
    """A visible page that is not there holds no keys; a sequence with none gives out 0 and lse -inf."""
    lens, P = [200, 130, 64], 16
    q, k, v, table = decode_case(4, lens, 4, 2, 64, 64, P, "fp16")
    table[0, [0, 3, 12]] = -1
    table[1, :] = k.shape[0] + 5
    got = bss.loza_ssa_decode_paged_kv(q, k, v, torch.tensor(table, dtype=torch.int32, device="cuda"),
                                       torch.tensor(lens, dtype=torch.int32, device="cuda"), 200,
                                       bss.Params(0.2, 128, 0, -1))
    check_decode(got, q, k, v, table, lens, (128, 0, -1), float(np.float32(0.2)), "decode missing pages")
    assert torch.isneginf(got[1][1]).all()


def test_decode_extreme_scores(bss):
    """Scores of thousands either way, equal keys, a scale of 0, and weights far below the largest."""
    lens, P = [333, 64, 2000], 32
    for dtype in ("bf16", "fp16"):
        for scale in (0.0, 30.0, -30.0):
            q, k, v, table = decode_case(6, lens, 8, 4, 64, 64, P, dtype)
            got = bss.loza_ssa_decode_paged_kv(q, k, v, torch.tensor(table, dtype=torch.int32, device="cuda"),
                                               torch.tensor(lens, dtype=torch.int32, device="cuda"), 2000,
                                               bss.Params(scale, 128, 0, -1))
            check_decode(got, q, k, v, table, lens, (128, 0, -1), scale, f"decode scale {scale}")
        # one key far above 60,000 equal ones: together they weigh as much as it does
        L = 60001
        q, k, v, table = decode_case(7, [L], 4, 1, 64, 64, 64, dtype)
        k.zero_()
        q.zero_()
        q[..., 0], k[table[0, 0], 0, 0, 0] = 1.0, math.log(60000.0)
        got = bss.loza_ssa_decode_paged_kv(q, k, v, torch.tensor(table, dtype=torch.int32, device="cuda"),
                                           torch.tensor([L], dtype=torch.int32, device="cuda"), L,
                                           bss.Params(1.0, 128, 0, -1))
        check_decode(got, q, k, v, table, [L], (128, 0, -1), 1.0, f"decode many small {dtype}")


@pytest.mark.parametrize("B", [32, 33, 700, 5000])
def test_decode_of_many_sequences(bss, B):
    """More sequences than CTAs, and than one pass of a warp over the lengths; many of them empty."""
    g = np.random.default_rng(B)
    lens = [int(x) for x in np.where(g.random(B) < 0.3, 0, g.integers(0, 90, B))]
    lens[-1] = 70
    q, k, v, table = decode_case(B, lens, 2, 1, 64, 64, 16, "bf16")
    got = bss.loza_ssa_decode_paged_kv(q, k, v, torch.tensor(table, dtype=torch.int32, device="cuda"),
                                       torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens),
                                       bss.Params(0.125, 128, 0, -1))
    check_decode(got, q, k, v, table, lens, (128, 0, -1), 0.125, f"decode of {B}")


@pytest.mark.parametrize("layout", ["nhd", "hnd", "pair"])
def test_decode_pool_layouts_and_strided_queries(bss, layout):
    lens, P, Hk = [513, 90, 0], 32, 3
    q, k, v, table = decode_case(8, lens, 12, Hk, 192, 128, P, "bf16")
    wide = normal(9, 3, 12 * 192 + 64, dtype=torch.bfloat16)
    wide[:, :12 * 192] = q.view(3, -1)
    kp, vp = (pool_layouts(t.shape[0], P, Hk, t.shape[3], torch.bfloat16, float("nan"))[layout] for t in (k, v))
    kp.copy_(k)
    vp.copy_(v)
    tab = torch.full((3, table.shape[1] + 3), -1, dtype=torch.int32, device="cuda")
    tab[:, :table.shape[1]] = torch.tensor(table, dtype=torch.int32)
    args = (tab[:, :table.shape[1]], torch.tensor(lens, dtype=torch.int32, device="cuda"), 513,
            bss.Params(0.07, 128, 0, -1))
    got = bss.loza_ssa_decode_paged_kv(wide[:, :12 * 192].view(3, 12, 192), kp, vp, *args)
    check_decode(got, q, k, v, table, lens, (128, 0, -1), float(np.float32(0.07)), f"decode {layout}")


def test_decode_lengths_outside_their_range(bss):
    """Device lengths beyond max_seqlen, or negative, are taken to be in [0, max_seqlen]: nothing is read outside."""
    q, k, v, table = decode_case(10, [256, 256, 256], 4, 4, 64, 64, 16, "bf16")
    t_d = torch.tensor(table, dtype=torch.int32, device="cuda")
    lens = torch.tensor([1 << 30, -3, 256], dtype=torch.int32, device="cuda")
    got = bss.loza_ssa_decode_paged_kv(q, k, v, t_d, lens, 256, bss.Params(0.1, 128, 0, -1))
    check_decode(got, q, k, v, table, [256, 0, 256], (128, 0, -1), float(np.float32(0.1)), "decode bad lengths")


def test_decode_far_pages(bss):
    """A pool of more than 2^32 bytes and 2^31 elements: the last pages are read from where they are."""
    P, Hk, d = 64, 8, 128
    pages = 2 ** 31 // (P * Hk * d) + 300  # 5.0 GB each for K and V
    k = torch.empty(pages, P, Hk, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty(pages, P, Hk, d, dtype=torch.bfloat16, device="cuda")
    lens = [300, 190]
    table = np.array([[pages - 1, 3, pages - 7, 0, pages - 2], [pages - 3, pages - 200, 5, -1, -1]])
    for n, pg in enumerate([x for x in table.reshape(-1) if x >= 0]):
        k[pg], v[pg] = normal(n, P, Hk, d, dtype=torch.bfloat16), normal(n + 50, P, Hk, d, dtype=torch.bfloat16)
    q = normal(99, 2, 16, d, dtype=torch.bfloat16)
    got = bss.loza_ssa_decode_paged_kv(q, k, v, torch.tensor(table, dtype=torch.int32, device="cuda"),
                                       torch.tensor(lens, dtype=torch.int32, device="cuda"), 300,
                                       bss.Params(0.09, 128, 0, -1))
    used = sorted({int(x) for x in table.reshape(-1) if x >= 0})
    small = np.vectorize(lambda x: used.index(x) if x >= 0 else -1)(table)
    idx = torch.tensor(used, device="cuda")
    check_decode(got, q, k[idx], v[idx], small, lens, (128, 0, -1), float(np.float32(0.09)), "decode far pages")
    # the write side of the same pool
    slots = torch.tensor([(pages - 1) * P + 63, (pages - 9) * P, 1], device="cuda")
    x = normal(5, 3, Hk, d, dtype=torch.bfloat16)
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    none = torch.zeros(0, dtype=torch.float64, device="cuda")
    bss.loza_qk_norm_rope(None, x, pos, none, bss.RopeParams(0), v=x, k_pool=k, v_pool=v, slots=slots)
    assert torch.equal(k.view(-1, Hk, d)[slots], x) and torch.equal(v.view(-1, Hk, d)[slots], x)


def test_decode_is_deterministic_and_captures(bss):
    """The same bits every call, from a workspace full of NaN, and in a replayed graph over new inputs; two graphs on
    two streams with a workspace each, replayed at the same time."""
    lens = [900, 33, 2500, 0, 64]
    q, k, v, table = decode_case(12, lens, 16, 4, 128, 128, 16, "bf16")
    t_d, l_d = torch.tensor(table, dtype=torch.int32, device="cuda"), torch.tensor(lens, dtype=torch.int32).cuda()
    p = bss.Params(0.09, 128, 0, -1)
    n = bss.lib().loza_decode_paged_kv_workspace_size(16, 4, 128, 128)
    runs = []
    for k_ in range(2):
        st = torch.cuda.Stream()
        ws = torch.full((n // 4,), float("nan"), device="cuda")
        out, lse = torch.empty(5, 16, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(5, 16, device="cuda")
        st.wait_stream(torch.cuda.current_stream())
        qs = q.clone()
        bss.loza_ssa_decode_paged_kv(qs, k, v, t_d, l_d, 2500, p, out=out, lse=lse, workspace=ws, stream=st)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            bss.loza_ssa_decode_paged_kv(qs, k, v, t_d, l_d, 2500, p, out=out, lse=lse, workspace=ws, stream=st)
        runs.append((st, g, qs, out, lse))
    eager = bss.loza_ssa_decode_paged_kv(q, k, v, t_d, l_d, 2500, p)
    q2 = normal(77, 5, 16, 128, dtype=torch.bfloat16)
    eager2 = bss.loza_ssa_decode_paged_kv(q2, k, v, t_d, l_d, 2500, p)
    torch.cuda.synchronize()
    for st, g, qs, out, lse in runs:
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
        qs.copy_(q2)
    torch.cuda.synchronize()
    for _ in range(20):
        for st, g, *_rest in runs:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for st, g, qs, out, lse in runs:
        assert torch.equal(out, eager2[0]) and torch.equal(lse, eager2[1])


def test_captured_step_at_a_fixed_capacity(bss):
    """A whole step - plan, norm + rotation into the pool (keys in place as well), decode - captured once at a fixed
    capacity and replayed with other lengths, against the same calls made one by one. The padded rows write nothing."""
    B, P, H, Hk, d, cap = 6, 16, 8, 2, 128, 40
    dt = torch.bfloat16
    rope, params = bss.RopeParams(d), bss.Params(d ** -0.5, 128, 0, -1)
    freq, _ = bss.rope_frequencies(d, device="cuda")
    kw = normal(1, d, dtype=dt) + 1
    free = torch.randperm(200, generator=torch.Generator().manual_seed(3)).int().cuda()
    ctx, new = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2))

    def state():
        return dict(table=torch.full((B, 30), -1, dtype=torch.int32, device="cuda"),
                    k_pool=torch.zeros(200, P, Hk, d, dtype=dt, device="cuda"),
                    v_pool=torch.zeros(200, P, Hk, d, dtype=dt, device="cuda"))

    q, k, v = normal(2, cap, H, d, dtype=dt), normal(3, cap, Hk, d, dtype=dt), normal(4, cap, Hk, d, dtype=dt)

    def step(s, k_rows):
        cu, lens, pos, slots, counts = bss.loza_page_plan(ctx, new, free, s["table"], P, cap)
        q_out, k_out = bss.loza_qk_norm_rope(q, k_rows, pos, freq, rope, None, kw, 1e-6, v=v, k_pool=s["k_pool"],
                                             v_pool=s["v_pool"], slots=slots, k_out=k_rows)
        rows = q_out[(cu[1:].long() - 1).clamp(min=0)]
        out, lse = bss.loza_ssa_decode_paged_kv(rows, s["k_pool"], s["v_pool"], s["table"], lens, 480, params)
        return cu, lens, pos, slots, counts, q_out, k_out, out, lse

    a, b, kb = state(), state(), k.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(state(), k.clone())
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step(b, kb)
    for seed, lengths in enumerate(([5, 0, 17, 3, 1, 9], [0, 0, 0, 0, 0, 0], [40, 0, 0, 0, 0, 0], [1, 1, 1, 1, 1, 1])):
        new.copy_(torch.tensor(lengths, dtype=torch.int32))
        k.copy_(normal(50 + seed, cap, Hk, d, dtype=dt))
        kb.copy_(k)
        ka = k.clone()
        eager = step(a, ka)
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(eager, captured):
            assert torch.equal(x, y)
        assert all(torch.equal(a[n], b[n]) for n in a) and torch.equal(ka, kb)
        n = sum(lengths)
        assert (eager[3][n:] == -1).all() and (a["k_pool"].view(-1, Hk, d)[eager[3][:n]] == ka[:n]).all()
        ctx.copy_(eager[1])
        free.copy_(torch.roll(free, -int(eager[4][1])))  # what was taken goes to the end


def test_norm_rope_on_another_stream(bss):
    """`stream` runs the whole call there, buffers made inside included."""
    T, H, d = 500, 8, 128
    pos, freq, pos_d, freq_d = rope_inputs(bss, 1, T, d)
    q, gq = normal(1, T, H, d, dtype=torch.bfloat16), normal(2, T, H, d, dtype=torch.bfloat16)
    w = normal(3, d, dtype=torch.bfloat16)
    rope = bss.RopeParams(d)
    want = bss.loza_qk_norm_rope_backward(gq, None, q, None, pos_d, freq_d, rope, w, None)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for _ in range(5):
        got = bss.loza_qk_norm_rope_backward(gq, None, q, None, pos_d, freq_d, rope, w, None, stream=st)
        junk = torch.full((1 << 20,), 3.0, device="cuda")  # on the current stream meanwhile
        st.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    del junk
    assert torch.cuda.current_stream() != st


def test_binding_refuses(bss):
    q, k = normal(1, 4, 8, 128, dtype=torch.bfloat16), normal(2, 4, 2, 128, dtype=torch.bfloat16)
    pos, freq, pos_d, freq_d = rope_inputs(bss, 1, 4, 128)
    rope, w = bss.RopeParams(128), torch.ones(128, dtype=torch.bfloat16, device="cuda")
    bad = [
        lambda: bss.loza_rope(q, pos_d.long(), freq_d, rope), lambda: bss.loza_rope(q, pos_d, freq_d.float(), rope),
        lambda: bss.loza_rope(q, pos_d, freq_d[:5], rope), lambda: bss.loza_rope(q, pos_d[:3], freq_d, rope),
        lambda: bss.loza_rope(q.double(), pos_d, freq_d, rope), lambda: bss.loza_rope(q, pos_d.cpu(), freq_d, rope),
        lambda: bss.loza_rope(q.transpose(1, 2), pos_d, freq_d, rope), lambda: bss.loza_rope(q, pos_d, freq_d, rope, out=k),
        lambda: bss.loza_qk_norm_rope(q, k.half(), pos_d, freq_d, rope, w, w),
        lambda: bss.loza_qk_norm_rope(q, k, pos_d, freq_d, rope, w.float(), w),
        lambda: bss.loza_qk_norm_rope(q, k, pos_d, freq_d, rope, w, w[:64]),
        lambda: bss.loza_qk_norm_rope(q, k, pos_d, freq_d, rope, w, w, v=k),
        lambda: bss.loza_qk_norm_rope(q, k[:3], pos_d, freq_d, rope, w, w),
        lambda: bss.loza_qk_norm_rope(q, None, pos_d, freq_d, rope, w, w),
        lambda: bss.loza_qk_norm_rope_backward(q, k, None, k, pos_d, freq_d, rope, w, w),
        lambda: bss.loza_qk_norm_rope_backward(q, k, q, k, pos_d, freq_d, rope, w, w,
                                               workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
        lambda: bss.loza_ssa_decode_paged_kv(q, k.view(1, 4, 2, 128), k.view(1, 4, 2, 128), pos_d.view(4, 1), pos_d, 4,
                                             bss.Params(1.0)),  # pages of 4 rows
        lambda: bss.loza_page_plan(pos_d, pos_d, pos_d, pos_d.view(4, 1), 3, 8),
        lambda: bss.loza_page_plan(pos_d, pos_d, pos_d, pos_d.view(2, 2), 16, 8),
    ]
    before = bss.launch_count()
    for i, call in enumerate(bad):
        with pytest.raises((TypeError, ValueError, bss.LozaError)):
            call()
            raise AssertionError(f"call {i} went through")
    assert bss.launch_count() == before
