"""How a server's or trainer's program meets the paged operators: calls from several threads at once,
with arguments mixed up, short of memory, beside autograd, and with a pool of one page."""
import threading

import numpy as np
import pytest
import torch

from oracle import paged
from test_abi_paged import NORM_ROPE_BACKWARD_ARGS, PLAN_ARGS, pack
from test_gpu_paged import normal, plan_case, rope_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bss():
    import block_sparse_streaming_b200 as m
    m.build()
    return m


def in_threads(*bodies):
    """The bodies at the same time; the first error of each."""
    errors, start = [], threading.Barrier(len(bodies))

    def run(body):
        try:
            start.wait()
            body()
        except Exception as e:  # handed to the test's thread
            errors.append(e)

    threads = [threading.Thread(target=run, args=(b,)) for b in bodies]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return errors


def test_gradients_of_different_sizes_in_threads(bss):
    """One kernel instance with more or less shared memory, launched by several threads at once through the C ABI
    (ctypes lets go of the interpreter's lock, so the calls really meet)."""
    L, T, d = bss.lib(), 1300, 128
    w = normal(1, d, dtype=torch.bfloat16) + 1
    x, dy = normal(2, T, 1, d, dtype=torch.bfloat16), normal(3, T, 1, d, dtype=torch.bfloat16)

    def work(dim):
        pos, freq, pos_d, freq_d = rope_inputs(bss, 4, T, dim)
        want = bss.loza_qk_norm_rope_backward(dy, None, x, None, pos_d, freq_d, bss.RopeParams(dim), w)
        st, dx, dw = torch.cuda.Stream(), torch.empty_like(x), torch.empty(d, device="cuda")
        ws = torch.empty(L.loza_qk_norm_rope_workspace_size(d), dtype=torch.uint8, device="cuda")
        args = pack(NORM_ROPE_BACKWARD_ARGS, dq_out=dy.data_ptr(), q=x.data_ptr(), positions=pos_d.data_ptr(),
                    inv_freq=freq_d.data_ptr(), q_weight=w.data_ptr(), dq=dx.data_ptr(), dq_weight=dw.data_ptr(),
                    workspace=ws.data_ptr(), workspace_bytes=ws.numel(), tokens=T, dq_out_row_stride=d, q_row_stride=d,
                    dq_row_stride=d, n_heads=1, d=d, norm_dim=d, eps=1e-6, rope_dim=dim, rope_scale=1.0, dtype=0)

        def body(keep=(pos_d, freq_d, ws)):
            codes = set()
            for i in range(8000):
                codes.add(L.loza_qk_norm_rope_backward(args, st.cuda_stream))
                if i % 100 == 99:
                    st.synchronize()
            assert codes == {0}, codes
            assert torch.equal(dx, want[0]) and torch.equal(dw, want[2])

        return body

    bodies = [work(dim) for dim in (128, 64, 32, 2)]
    torch.cuda.synchronize()
    assert in_threads(*bodies) == []


def test_plans_of_different_sizes_in_threads(bss):
    """Plans of thousands of requests keep their sums in more or less shared memory."""
    L = bss.lib()

    def work(B):
        ctx, new, free, table = plan_case(B, B, 16, 40, 3)
        dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
        ctx_d, new_d, free_d, table_d = dev(ctx), dev(new), dev(free), dev(table)
        capacity, st = int(new.sum()), torch.cuda.Stream()
        want = paged.plan(ctx, new, free, table, 16, capacity)
        cu, lens, counts = dev(np.zeros(B + 1)), dev(np.zeros(B)), dev(np.zeros(3))
        pos, slots = dev(np.zeros(capacity)), torch.zeros(capacity, dtype=torch.int64, device="cuda")
        args = pack(PLAN_ARGS, ctx_lens=ctx_d.data_ptr(), new_lens=new_d.data_ptr(), free_pages=free_d.data_ptr(),
                    block_table=table_d.data_ptr(), cu_seqlens=cu.data_ptr(), seqlens=lens.data_ptr(),
                    positions=pos.data_ptr(), slots=slots.data_ptr(), counts=counts.data_ptr(),
                    bt_stride=table_d.stride(0), capacity=capacity, batch=B, n_free=len(free), page_size=16,
                    max_pages=table_d.shape[1])

        def body(keep=(ctx_d, new_d, free_d)):
            codes = set()
            for i in range(3000):
                codes.add(L.loza_page_plan(args, st.cuda_stream))
                if i % 100 == 99:
                    st.synchronize()
            assert codes == {0}, codes
            for g, w in zip((table_d, cu, lens, pos, slots, counts), want):
                assert (g.cpu().numpy() == w).all()

        return body

    bodies = [work(B) for B in (16384, 7000, 9001)]
    torch.cuda.synchronize()
    assert in_threads(*bodies) == []


def test_exchanged_structures_are_refused(bss):
    """Params and RopeParams have the same size: each is taken only where it belongs, and nothing else is."""
    q = normal(1, 2, 8, 64, dtype=torch.bfloat16)
    pool = normal(2, 4, 16, 8, 64, dtype=torch.bfloat16)
    pos, freq, pos_d, freq_d = rope_inputs(bss, 1, 2, 64)
    table = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    window, rope = bss.Params(1.0, 64, 0, 1), bss.RopeParams(64, 0, True)
    decode = lambda p: bss.loza_ssa_decode_paged_kv(q, pool, pool, table, pos_d.clamp(0, 9), 9, p)
    rotate = lambda r: bss.loza_rope(q, pos_d, freq_d, r)
    norm = lambda r: bss.loza_qk_norm_rope(q, None, pos_d, freq_d, r)
    grad = lambda r: bss.loza_qk_norm_rope_backward(q, None, None, None, pos_d, freq_d, r)
    decode(window), rotate(rope), norm(rope), grad(rope)
    before = bss.launch_count()
    for bad in (rope, bytes(rope), bytearray(bytes(window)), torch.zeros(4).numpy(), None):
        with pytest.raises(TypeError):
            decode(bad)
    for call in (rotate, norm, grad):
        for bad in (window, bytes(rope), torch.zeros(4).numpy(), None):
            with pytest.raises(TypeError):
                call(bad)
    assert bss.launch_count() == before


def test_out_of_memory_is_torchs_error(bss):
    """An output or workspace that does not fit raises what torch.empty raises (the allocator's own limit, set low)."""
    x = normal(1, 4000, 8, 128, dtype=torch.bfloat16)
    pos, freq, pos_d, freq_d = rope_inputs(bss, 1, 4000, 128)
    i32 = torch.zeros(1, dtype=torch.int32, device="cuda")
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (1 << 22)) / total)
    held = []
    try:
        for size in (1 << 25, 1 << 22, 1 << 21):  # what the allocator kept of earlier tests
            with pytest.raises(torch.OutOfMemoryError):
                while True:
                    held.append(torch.empty(size, dtype=torch.uint8, device="cuda"))
        with pytest.raises(torch.OutOfMemoryError):
            bss.loza_page_plan(i32, i32, i32, i32.view(1, 1), 16, 1 << 24)
        with pytest.raises(torch.OutOfMemoryError):
            y = [bss.loza_rope(x, pos_d, freq_d, bss.RopeParams(128)) for _ in range(4)]
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    y = bss.loza_rope(x, pos_d, freq_d, bss.RopeParams(128))
    assert y.shape == x.shape


def test_written_tensors_count_their_versions(bss):
    """What a call writes in place counts as changed, so that autograd notices a saved tensor that was overwritten;
    what it reads does not, and tensors of inference mode, which keep no count, are taken."""
    T, H, Hk, d, P = 6, 4, 2, 64, 16
    dt = torch.bfloat16
    pos, freq, pos_d, freq_d = rope_inputs(bss, 1, T, d)
    rope, w = bss.RopeParams(d), normal(9, d, dtype=dt) + 1
    q, k, v, gq, gk = (normal(s, T, h, d, dtype=dt) for s, h in enumerate((H, Hk, Hk, H, Hk)))
    kp, vp = (normal(7, 4, P, Hk, d, dtype=dt) for _ in range(2))
    slots, lens = torch.arange(T, device="cuda"), torch.full((T,), 3, dtype=torch.int32, device="cuda")
    table = torch.zeros(T, 2, dtype=torch.int32, device="cuda")
    free = torch.arange(3, 40, dtype=torch.int32, device="cuda")
    out, lse = torch.empty(T, H, d, dtype=dt, device="cuda"), torch.empty(T, H, device="cuda")
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    q2 = q.clone()
    p = bss.Params(0.1, 128, 0, -1)
    calls = [
        (lambda: bss.loza_rope(q, pos_d, freq_d, rope, out=q), [q], [pos_d, freq_d]),
        (lambda: bss.loza_rope(q, pos_d, freq_d, rope), [], [q]),
        (lambda: bss.loza_qk_norm_rope(q, k, pos_d, freq_d, rope, w, w, v=v, k_pool=kp, v_pool=vp, slots=slots, q_out=q,
                                       k_out=k), [q, k, kp, vp], [v, w, slots]),
        (lambda: bss.loza_qk_norm_rope_backward(gq, gk, q, k, pos_d, freq_d, rope, w, w, dq=dq, dk=dk), [dq, dk],
         [gq, gk, q, k, w]),
        (lambda: bss.loza_ssa_decode_paged_kv(q2, kp, vp, table, lens, 3, p, out=out, lse=lse), [out, lse],
         [q2, kp, vp, table, lens]),
        (lambda: bss.loza_page_plan(lens, lens, free, table, P, 40), [table], [lens, free])]
    for call, written, read in calls:
        before = [t._version for t in written], [t._version for t in read]
        call()
        assert all(t._version > n for t, n in zip(written, before[0]))
        assert [t._version for t in read] == before[1]
    x = normal(11, T, H, d).requires_grad_()
    y = x * 2
    z = (y * y).sum()  # keeps y
    bss.loza_rope(y.detach(), pos_d, freq_d, rope, out=y.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        z.backward()
    with torch.inference_mode():
        a = q.clone()
        assert bss.loza_rope(a, pos_d, freq_d, rope, out=a) is a


def test_pool_of_one_page_has_any_page_stride(bss):
    """The stride of a dimension of size one is never used, whatever the tensor says it is."""
    T, Hk, d, P = 5, 2, 64, 16
    dt = torch.bfloat16
    pos, freq, pos_d, freq_d = rope_inputs(bss, 1, T, d)
    k = normal(1, T, Hk, d, dtype=dt)
    slots = torch.arange(T, device="cuda")
    pools = [torch.zeros(1, P, Hk, d, dtype=dt, device="cuda") for _ in range(2)]
    odd = [t.as_strided(t.shape, (3, *t.stride()[1:])) for t in pools]
    bss.loza_qk_norm_rope(None, k, pos_d, freq_d, bss.RopeParams(d), v=k, k_pool=odd[0], v_pool=odd[1], slots=slots)
    q = normal(2, 1, 4, d, dtype=dt)
    table, lens = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.full((1,), T, dtype=torch.int32).cuda()
    p = bss.Params(0.1, 128, 0, -1)
    want = bss.loza_ssa_decode_paged_kv(q, *pools, table, lens, T, p)
    got = bss.loza_ssa_decode_paged_kv(q, *odd, table, lens, T, p)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(pools[1][0, :T], k)


def test_infinite_values_stay_in_their_column(bss):
    """An infinity in a visible value row spoils that column of its key head's queries and nothing else."""
    B, H, Hk, d, P, L = 2, 8, 2, 64, 16, 100
    dt = torch.bfloat16
    q, k, v = normal(1, B, H, d, dtype=dt), normal(2, 16, P, Hk, d, dtype=dt), normal(3, 16, P, Hk, d, dtype=dt)
    table = torch.arange(14, device="cuda", dtype=torch.int32).view(2, 7)
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")
    p = bss.Params(0.1, 128, 0, -1)
    clean = bss.loza_ssa_decode_paged_kv(q, k, v, table, lens, L, p)
    v[3, 5, 1, 17], v[8, 0, 0, 2] = float("inf"), float("nan")  # sequence 0, key head 1; sequence 1, key head 0
    out, lse = bss.loza_ssa_decode_paged_kv(q, k, v, table, lens, L, p)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[0, 4:, 17], bad[1, :4, 2] = True, True
    assert torch.equal(lse, clean[1]) and torch.equal(out[~bad], clean[0][~bad])
    assert not torch.isfinite(out[bad]).any()
