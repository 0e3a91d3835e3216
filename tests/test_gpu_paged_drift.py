"""Sums of the paged decode over long contexts: their error must not grow one way with the number of keys."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bss():
    import block_sparse_streaming_b200 as m
    m.build()
    return m


@pytest.mark.parametrize("d,heads", [(64, 1), (64, 16), (128, 2)])
def test_long_sums_do_not_drift(bss, d, heads):
    """Equal weights (queries of zero) over 131,072 keys that one CTA adds up: each output is the mean of its keys'
    values, and the mean of all outputs' relative errors is that of their roundings to 16 bits. A rounding is at most
    2^-11 of the value and as often up as down, over values spread over many steps: its mean over N outputs has a
    deviation of 2^-11 / sqrt(3 N); five of them are allowed. The 32-bit sums' own roundings, 2^-24 each and to either
    side, add up to 2^-24 sqrt(2,048) = 2^-18.5 an output and vanish in that mean. (Sums cut off toward zero instead
    of rounded lose half a step of 2^-23 at most additions: 2^-24 x 2,048 / 2 = 6e-5 here, every one the same way.)"""
    B, L, P = 2 * torch.cuda.get_device_properties(0).multi_processor_count, 131072, 64
    pages = 2 * L // P
    g = torch.Generator(device="cuda").manual_seed(d + heads)
    v = (torch.rand(pages, P, 1, d, device="cuda", generator=g) * 0.5 + 0.25 +
         torch.arange(d, device="cuda") / d).half()
    k = torch.randn(pages, P, 1, d, device="cuda", generator=g).half()
    q = torch.zeros(B, heads, d, dtype=torch.float16, device="cuda")
    table = torch.stack([torch.randperm(pages, device="cuda", generator=g)[:L // P] for _ in range(B)]).int()
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    out, lse = bss.loza_ssa_decode_paged_kv(q, k, v, table, lens, L, bss.Params(0.125, 128, 0, -1))
    means = v.double().sum(dim=(1, 2))[table.long()].sum(1) / L
    assert torch.equal(out, out[:, :1].expand_as(out))
    rel = ((out[:, 0].double() - means) / means).cpu().numpy()
    assert np.abs(rel).max() <= 2.0 ** -11 + 2048 * 2.0 ** -24
    drift, allowed = float(rel.mean()), 5 * 2.0 ** -11 / (3 * rel.size) ** 0.5
    print(f"drift {drift:.2e}, allowed {allowed:.2e}")
    assert abs(drift) <= allowed, f"mean relative error {drift:.2e}, at most {allowed:.2e}"
    assert (lse - np.log(L)).abs().max() <= 12 * 2.0 ** -22
