"""The paged operators run together, as a serving loop uses them: plan the step, norm and rotate the new
queries and keys and write the cache, attend, for a prompt step and several decode steps; for grouped heads
over K and V pools and for the latent cache that the absorbed paged decode reads. Each stage is compared with
the oracle on what the stage before it gave."""
import numpy as np
import pytest
import torch

import oracle
from helpers import assert_close_lse, assert_close_o
from oracle import paged
from test_gpu_paged import check_decode, close, f64, norm_slack, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bss():
    import block_sparse_streaming_b200 as m
    m.build()
    return m


class Cache:
    """Host bookkeeping of a server: lengths, free pages, the table on the device."""

    def __init__(self, B, pages, cols, P, seed):
        self.P, self.lens = P, np.zeros(B, np.int64)
        self.free = np.random.default_rng(seed).permutation(pages)
        self.host = np.full((B, cols), -1)
        self.table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")

    def step(self, bss, new, capacity):
        i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
        want = paged.plan(self.lens, new, self.free, self.host, self.P, capacity)
        got = bss.loza_page_plan(i32(self.lens), i32(new), i32(self.free), self.table, self.P, capacity)
        for g, w in zip((self.table,) + got, want):
            assert np.array_equal(g.cpu().numpy(), w)
        assert want[5][2] == 0
        self.host, self.lens, self.free = want[0], want[2], self.free[want[5][1]:]
        return got


@pytest.mark.parametrize("window", [(128, 0, -1), (128, 1, 7), (1, 16, 64)])
def test_grouped_heads(bss, window):
    B, H, Hk, d, P, dtype = 5, 16, 4, 128, 16, torch.bfloat16
    cache = Cache(B, 500, 100, P, 1)
    k_pool = torch.full((500, P, Hk, d), float("nan"), dtype=dtype, device="cuda")
    v_pool = torch.full_like(k_pool, float("nan"))
    qw, kw = normal(1, d, dtype=dtype) + 1, normal(2, d, dtype=dtype) + 1
    freq, scale = bss.rope_frequencies(64, scaling="yarn", factor=4.0, device="cuda")
    rope, params = bss.RopeParams(64, 0, False, scale), bss.Params(d ** -0.5, *window)
    for step, new in enumerate([[700, 1, 0, 1290, 65], [1, 1, 1, 0, 1], [1, 1, 0, 1, 1], [0, 30, 2, 1, 1]]):
        capacity = sum(new) + 3
        cu, lens, pos, slots, _ = cache.step(bss, np.array(new), capacity)
        rows = normal(10 + step, capacity, (H + 2 * Hk) * d, dtype=dtype)
        q, k, v = (rows[:, a * d:b * d].view(capacity, b - a, d) for a, b in ((0, H), (H, H + Hk), (H + Hk, H + 2 * Hk)))
        q_out, _ = bss.loza_qk_norm_rope(q, k, pos, freq, rope, qw, kw, 1e-6, v=v, k_pool=k_pool, v_pool=v_pool,
                                         slots=slots)
        n = sum(new)
        args = (d, float(np.float32(1e-6)), pos.cpu().numpy(), freq.cpu().numpy(), 0, False, float(np.float32(scale)))
        want, size = paged.norm_rope(f64(q), f64(qw), *args)
        close(q_out, want, norm_slack(qw, d, size, d), "step q")
        want, size = paged.norm_rope(f64(k), f64(kw), *args)
        close(k_pool.view(-1, Hk, d)[slots[:n]], want[:n], norm_slack(kw, d, size, d)[:n], "step k")
        assert torch.equal(v_pool.view(-1, Hk, d)[slots[:n]], v[:n])
        # the last new token of each request attends (idle requests: their padded row)
        last = (cu[1:].long() - 1).clamp(min=0)
        got = bss.loza_ssa_decode_paged_kv(q_out[last], k_pool, v_pool, cache.table, lens, int(cache.lens.max()), params)
        check_decode(got, q_out[last], k_pool.nan_to_num(), v_pool.nan_to_num(), cache.host, cache.lens, window,
                     float(np.float32(d ** -0.5)), f"step {step} {window}")


def test_latent_cache(bss):
    """The absorbed path: the latent normed over its first 512 columns, the last 64 rotated and all 576 written to a
    page of the pool that loza_ssa_decode_paged reads; compared with the contiguous oracle decode."""
    B, H, d, P, dtype = 3, 64, 576, 128, torch.bfloat16
    oracle.build()
    cache = Cache(B, 60, 16, P, 2)
    pool = torch.zeros(60, P, 1, d, dtype=dtype, device="cuda")
    kw = normal(2, 512, dtype=dtype) * 0.1 + 1
    freq, scale = bss.rope_frequencies(64, device="cuda")
    rope, params = bss.RopeParams(64, 512, True, scale), bss.Params(192 ** -0.5)
    for step, new in enumerate([[1300, 1, 200], [1, 1, 1], [1, 1, 1]]):
        cu, lens, pos, slots, _ = cache.step(bss, np.array(new), sum(new) + 1)
        T = sum(new) + 1
        q, lat = normal(20 + step, T, H, d, dtype=dtype), normal(30 + step, T, 1, d, dtype=dtype)
        q_out, _ = bss.loza_qk_norm_rope(q, lat, pos, freq, rope, None, kw, 1e-6, k_pool=pool, slots=slots)
        want, size = paged.norm_rope(f64(lat), f64(kw), 512, float(np.float32(1e-6)), pos.cpu().numpy(),
                                     freq.cpu().numpy(), 512, True, 1.0)
        close(pool.view(-1, 1, d)[slots[:-1]], want[:-1], norm_slack(kw, 512, size, d)[:-1], "latent")
        assert torch.equal(q_out, bss.loza_rope(q, pos, freq, rope))
        last = cu[1:].long() - 1
        out, lse = bss.loza_ssa_decode_paged(q_out[last], pool.view(60, P, d), cache.table, lens,
                                             int(cache.lens.max()), params)
        rows = max(cache.lens)
        cont = torch.zeros(B, rows, d, dtype=dtype, device="cuda")
        for n in range(B):
            pages = torch.tensor(cache.host[n][: -(-cache.lens[n] // P)], device="cuda")
            cont[n, :cache.lens[n]] = pool[pages].view(-1, d)[:cache.lens[n]]
        want_o, want_l, _, _ = paged.decode(f64(q_out[last]), f64(cont)[:, :, None, :], f64(cont)[:, :, None, :512],
                                            np.arange(B)[:, None], cache.lens, 128, 1, 7, float(np.float32(192 ** -0.5)))
        assert_close_o(f64(out), want_o, "latent step O")
        assert_close_lse(f64(lse), want_l, "latent step LSE")
