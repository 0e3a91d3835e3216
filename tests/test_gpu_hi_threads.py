"""The hierarchical selection from several threads at once: calls whose cache lengths differ keep bitmaps of different
sizes in shared memory."""
import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bss():
    import block_sparse_streaming_b200 as m
    m.build()
    return m


def test_selections_of_different_lengths_in_threads(bss):
    L, d, top_pages, top_k = bss.lib(), 64, 4, 64
    p = bss.Params(0.1, 1, 16, 1024)
    start = threading.Barrier(3)
    errors = []

    def work(cap):
        g = torch.Generator().manual_seed(cap)
        q = torch.randn(1, d, generator=g).bfloat16().cuda()
        k = torch.zeros(1, cap, d, dtype=torch.bfloat16, device="cuda")
        k[:, :2048] = torch.randn(1, 2048, d, generator=g).bfloat16().cuda()
        seq = torch.tensor([2000], dtype=torch.int32, device="cuda")
        keys = bss.loza_hi_page_keys(k, seq, cap)
        want = bss.loza_hi_select(q, k, keys, seq, cap, p, top_pages, top_k)
        got, st = torch.empty_like(want), torch.cuda.Stream()
        ws = torch.empty(bss.hi_workspace_size(1, cap, top_pages, top_k, p), dtype=torch.uint8, device="cuda")
        ptr = lambda t: ctypes.c_void_p(t.data_ptr())
        args = (ptr(q), ptr(k), k.stride(0), k.stride(1), ptr(keys), ptr(seq), 1, cap, d, p, top_pages, top_k, ptr(got),
                ptr(ws), ws.numel(), ctypes.c_void_p(st.cuda_stream))

        def body(keep=(q, k, seq, keys, ws)):
            codes = set()
            start.wait()
            for i in range(3000):
                codes.add(L.loza_hi_select(*args))
                if i % 100 == 99:
                    st.synchronize()
            if codes != {0} or not torch.equal(got, want):
                errors.append((cap, codes))

        return body

    threads = [threading.Thread(target=work(cap)) for cap in (2048, 65536, 262144)]
    torch.cuda.synchronize()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert errors == []
