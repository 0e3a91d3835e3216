"""The loops that carry large calls of the norm and rotation kernels: several batches of angles, several tokens a
warp, sums of the weights' gradients over all of them. A few tokens at a time (which test_gpu_paged.py compares with
the oracle) never enter them. Both sides of these comparisons are derived, not measured."""
import numpy as np
import pytest
import torch

from oracle import paged
from test_gpu_paged import DTYPES, STEP, close, f64, norm_slack, normal, rope_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bss():
    import block_sparse_streaming_b200 as m
    m.build()
    return m


def additions(T, H):
    """Additions that one value goes through at most on its way into a weight's gradient, on a GPU of 148 SMs or more:
    a lane's rows (at least one CTA of 8 warps per SM, equal shares of the tokens, one row per head), 5 over the
    warp, 8 over the CTA's warps, at most 5 rows of sums a thread (2 CTAs per SM, every 64th row), 16 + 2 at the end."""
    return (-(-T // 148) // 8 + 1) * H + 5 + 8 + max(5, -(-2 * torch.cuda.get_device_properties(0).multi_processor_count // 64)) + 18


@pytest.mark.parametrize("dtype,T,H,Hk,d,dim,off,nd,interleaved", [
    ("bf16", 20011, 4, 2, 64, 64, 0, 64, False), ("bf16", 20011, 4, 2, 64, 32, 32, 64, True),
    ("fp16", 20000, 3, 1, 128, 64, 0, 128, True), ("fp32", 20011, 4, 2, 64, 64, 0, 64, False),
    ("fp32", 20011, 2, 2, 64, 32, 16, 48, True), ("bf16", 9001, 2, 1, 576, 64, 512, 512, True),
    ("bf16", 12007, 3, 2, 100, 24, 76, 100, False), ("fp16", 12007, 3, 2, 66, 60, 4, 66, True),
    ("fp32", 9001, 1, 1, 1024, 1024, 0, 1024, False), ("bf16", 9001, 2, 1, 7, 6, 0, 7, False)])
def test_gradient_of_many_tokens(bss, dtype, T, H, Hk, d, dim, off, nd, interleaved):
    """dx: the bits of the same tokens in slices of 1,000; the weights' gradients: the 64-bit sum over all of them."""
    dt = DTYPES[dtype]
    pos, freq, pos_d, freq_d = rope_inputs(bss, d + T, T, dim)
    q, k = normal(1, T, H, d, dtype=dt, scale=2.0), normal(2, T, Hk, d, dtype=dt)
    gq, gk = normal(3, T, H, d, dtype=dt), normal(4, T, Hk, d, dtype=dt)
    qw, kw = normal(5, nd, dtype=dt) + 1, normal(6, nd, dtype=dt) + 1
    rope, eps = bss.RopeParams(dim, off, interleaved, 1.5), 1e-5
    dq, dk, dqw, dkw = bss.loza_qk_norm_rope_backward(gq, gk, q, k, pos_d, freq_d, rope, qw, kw, eps)
    for a in range(0, T, 1000):
        s = slice(a, min(a + 1000, T))
        part = bss.loza_qk_norm_rope_backward(gq[s], gk[s], q[s], k[s], pos_d[s], freq_d, rope, qw, kw, eps)
        assert torch.equal(dq[s], part[0]) and torch.equal(dk[s], part[1]), f"tokens {a}.."
    for x, dy, w, dx, dw, heads in ((q, gq, qw, dq, dqw, H), (k, gk, kw, dk, dkw, Hk)):
        want, size, want_w, size_w = paged.norm_rope_backward(f64(x), f64(dy), f64(w), nd, float(np.float32(eps)), pos,
                                                              freq, off, interleaved, 1.5)
        close(dx, want, 96 * STEP * size, f"long bwd {dtype} {d}")
        # each term 48 steps, and a step of the sum so far (at most all terms' magnitudes) per addition
        close(dw, want_w, (48 + additions(T, heads)) * STEP * size_w, f"long bwd weight {dtype} {d}")


@pytest.mark.parametrize("dtype,T,H,Hk,d,dim,off,weights,interleaved", [
    ("bf16", 13003, 8, 0, 64, 64, 0, False, False), ("bf16", 30011, 4, 2, 64, 32, 0, True, True),
    ("fp16", 30011, 2, 1, 128, 128, 0, True, False), ("fp32", 21001, 3, 2, 64, 64, 0, True, False),
    ("bf16", 15013, 1, 1, 576, 64, 512, True, True), ("bf16", 17011, 3, 1, 100, 24, 76, True, False),
    ("fp16", 17011, 3, 1, 66, 60, 4, False, True), ("bf16", 11003, 2, 1, 7, 6, 0, True, False),
    ("bf16", 50021, 1, 0, 64, 64, 0, False, True)])
def test_forward_of_many_tokens_a_walk(bss, dtype, T, H, Hk, d, dim, off, weights, interleaved):
    """Few heads: every warp walks more tokens than one batch of angles holds. The bits of the same tokens 400 at a
    time, and the oracle's values; rows that no token writes stay as they were."""
    dt = DTYPES[dtype]
    pos, freq, pos_d, freq_d = rope_inputs(bss, 9, T, dim)
    rope = bss.RopeParams(dim, off, interleaved)
    q = normal(1, T, H, d, dtype=dt)
    k, v = (normal(s, T, Hk, d, dtype=dt) for s in (2, 3)) if Hk else (None, None)
    w = normal(4, d, dtype=dt) + 1 if weights else None
    pages = -(-(T + 20) // 16)
    slots = torch.randperm(pages * 16, generator=torch.Generator().manual_seed(5)).cuda()[:T]
    runs = []
    for step in (T, 400):
        out = torch.full((T + 8, H, d), 3.0, dtype=dt, device="cuda")
        pools = [torch.full((pages, 16, max(Hk, 1), d), 4.0, dtype=dt, device="cuda") for _ in range(2)]
        for a in range(0, T, step):
            s = slice(a, min(a + step, T))
            if Hk:
                bss.loza_qk_norm_rope(q[s], k[s], pos_d[s], freq_d, rope, w, w, 1e-6, v=v[s], k_pool=pools[0],
                                      v_pool=pools[1], slots=slots[s], q_out=out[s])
            else:
                bss.loza_rope(q[s], pos_d[s], freq_d, rope, out=out[s])
        runs.append((out, *pools))
    assert all(torch.equal(x, y) for x, y in zip(*runs))
    out, k_pool, v_pool = runs[0]
    assert (out[T:] == 3).all()
    args = (d, float(np.float32(1e-6)), pos, freq, off, interleaved, 1.0)
    want, size = paged.norm_rope(f64(q), None if w is None else f64(w), *args)
    close(out[:T], want, norm_slack(w, d, size, d), f"long forward {dtype} {d}")
    if Hk:
        want, size = paged.norm_rope(f64(k), None if w is None else f64(w), *args)
        close(k_pool.view(-1, Hk, d)[slots], want, norm_slack(w, d, size, d), f"long forward keys {dtype} {d}")
        assert torch.equal(v_pool.view(-1, Hk, d)[slots], v)
        rest = torch.ones(pages * 16, dtype=torch.bool, device="cuda")
        rest[slots] = False
        assert (k_pool.view(-1, Hk, d)[rest] == 4).all() and (v_pool.view(-1, Hk, d)[rest] == 4).all()
