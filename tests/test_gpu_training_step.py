"""A training step over the library's calls: norm + rotation, attention, and both gradients behind torch.autograd.
The outputs and the gradients of q, k and v against the same step in 64 bits by torch's own differentiation (the bars
of the attention's tests); the weights' gradients, sums over all rows of what the attention's backward rounded to
bf16, against the 64-bit oracle on what it gave."""
import math

import numpy as np
import pytest
import torch

from helpers import assert_close_grad, assert_close_o
from oracle import paged
from test_gpu_paged import STEP, close, f64, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bss():
    import block_sparse_streaming_b200 as m
    m.build()
    return m


def attention(bss, positions, inv_freq, rope, cu, max_len, params, eps, seen):
    class Attention(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, q_weight, k_weight):
            qr, kr = bss.loza_qk_norm_rope(q, k, positions, inv_freq, rope, q_weight, k_weight, eps)
            out, lse = bss.loza_ssa_prefill(qr, kr, v, cu, max_len, params)
            ctx.save_for_backward(q, k, v, q_weight, k_weight, qr, kr, out, lse)
            return out

        @staticmethod
        def backward(ctx, dout):
            q, k, v, q_weight, k_weight, qr, kr, out, lse = ctx.saved_tensors
            dqr, dkr, dv = bss.loza_ssa_backward(qr, kr, v, out, dout.contiguous(), lse, cu, max_len, params)
            seen.update(dq=dqr, dk=dkr)
            dq, dk, dqw, dkw = bss.loza_qk_norm_rope_backward(dqr, dkr, q, k, positions, inv_freq, rope, q_weight,
                                                              k_weight, eps)
            return dq, dk, dv, dqw.to(q_weight.dtype), dkw.to(k_weight.dtype)

    return Attention.apply


def reference(q, k, v, qw, kw, pos, freq, lens, scale, eps):
    def norm_rope(x, w):
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w
        a, b = x.chunk(2, -1)
        angle = (pos.double()[:, None] * freq)[:, None]
        return torch.cat([a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()], -1)

    qr, kr, outs, at = norm_rope(q, qw), norm_rope(k, kw), [], 0
    for n in lens:
        z = torch.einsum("qhd,khd->hqk", qr[at:at + n], kr[at:at + n]) * scale
        z = z.masked_fill(torch.ones(n, n, dtype=torch.bool, device=z.device).triu(1), -math.inf)
        outs.append(torch.einsum("hqk,khd->qhd", z.softmax(-1), v[at:at + n]))
        at += n
    return torch.cat(outs)


@pytest.mark.parametrize("lens", [[300, 200], [1, 129, 640]])
def test_gradients_of_a_step(bss, lens):
    T, H, d, eps, scale = sum(lens), 2, 64, 1e-6, 64 ** -0.5
    dt = torch.bfloat16
    freq, _ = bss.rope_frequencies(d, device="cuda")
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).cuda()
    cu = torch.tensor([0, *torch.tensor(lens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    leaves = [normal(s, T, H, d, dtype=dt).requires_grad_() for s in (1, 2, 3)]
    leaves += [(normal(s, d, dtype=dt) * 0.2 + 1).detach().requires_grad_() for s in (4, 5)]
    dout = normal(6, T, H, d, dtype=dt)
    seen = {}
    out = attention(bss, pos, freq, bss.RopeParams(d), cu, max(lens), bss.Params(scale), eps, seen)(*leaves)
    out.backward(dout)
    wide = [t.detach().double().requires_grad_() for t in leaves]
    want = reference(*wide, pos, freq, lens, scale, eps)
    want.backward(dout.double())
    assert bss.device_status() == 0
    assert_close_o(f64(out), f64(want), "training step O")
    for name, a, b in zip(("dq", "dk", "dv"), leaves, wide):
        assert_close_grad(f64(a.grad), f64(b.grad), f"training step {name}")
    for x, w, dy in ((leaves[0], leaves[3], seen["dq"]), (leaves[1], leaves[4], seen["dk"])):
        _, _, want_w, size_w = paged.norm_rope_backward(f64(x), f64(dy), f64(w), d, float(np.float32(eps)),
                                                        pos.cpu().numpy(), freq.cpu().numpy(), 0, False, 1.0)
        # each term 48 steps and one per addition, at most one per row; then one rounding to bf16
        close(w.grad, want_w, (48 + T * H) * STEP * size_w, "training step weight")
