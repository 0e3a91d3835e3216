"""The entry points as the first CUDA call of a host thread, as torch.autograd's thread makes them in a backward pass:
such a thread has no current context until a call binds the device's."""
import threading

import pytest
import torch

from test_gpu_paged import normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bss():
    import block_sparse_streaming_b200 as m
    m.build()
    return m


def in_new_thread(call):
    got = []

    def body():
        try:
            got.append(call())
        except Exception as e:  # handed to the test's thread
            got.append(e)

    t = threading.Thread(target=body)
    t.start()
    t.join()
    torch.cuda.synchronize()
    if isinstance(got[0], Exception):
        raise got[0]
    return got[0]


def calls(bss):
    bf16 = torch.bfloat16
    T, H, L = 300, 2, 256
    q, k, v, dout = (normal(s, T, H, 64, dtype=bf16) for s in range(4))
    cu, p = torch.tensor([0, T], dtype=torch.int32, device="cuda"), bss.Params(0.125)
    out, lse = bss.loza_ssa_prefill(q, k, v, cu, T, p)
    q5, lat = normal(5, T, 4, 576, dtype=bf16), normal(6, T, 1, 576, dtype=bf16)
    qd, cache = normal(7, 2, 64, 576, dtype=bf16), normal(8, 2, L, 1, 576, dtype=bf16)
    lens = torch.tensor([200, 7], dtype=torch.int32, device="cuda")
    pool, table = cache.view(4, 128, 576), torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    kp, vp = normal(9, 4, 64, 2, 64, dtype=bf16), normal(10, 4, 64, 2, 64, dtype=bf16)
    pos, freq = torch.arange(T, dtype=torch.int32, device="cuda"), bss.rope_frequencies(64, device="cuda")[0]
    w, rope, st = normal(11, 64, dtype=bf16), bss.RopeParams(64), torch.cuda.current_stream()
    return {
        "prefill": lambda: bss.loza_ssa_prefill(q, k, v, cu, T, p, stream=st),
        "absorbed prefill": lambda: bss.loza_ssa_prefill(q5, lat, lat[:, :, :512], cu, T, p, stream=st),
        "backward": lambda: bss.loza_ssa_backward(q, k, v, out, dout, lse, cu, T, p, stream=st),
        "decode": lambda: bss.loza_ssa_decode(qd, cache, None, lens, L, p, stream=st),
        "paged decode": lambda: bss.loza_ssa_decode_paged(qd, pool, table, lens, L, p, stream=st),
        "paged K/V decode": lambda: bss.loza_ssa_decode_paged_kv(qd[:, :4, :64].contiguous(), kp, vp, table, lens, 128, p),
        "norm + rotation": lambda: bss.loza_qk_norm_rope(q, k, pos, freq, rope, w, w),
        "its gradient": lambda: bss.loza_qk_norm_rope_backward(q, k, q, k, pos, freq, rope, w, w),
    }


@pytest.mark.parametrize("name", ["prefill", "absorbed prefill", "backward", "decode", "paged decode",
                                  "paged K/V decode", "norm + rotation", "its gradient"])
def test_first_call_of_a_thread(bss, name):
    call = calls(bss)[name]
    want = call()
    torch.cuda.synchronize()
    got = in_new_thread(call)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bss.device_status() == 0
