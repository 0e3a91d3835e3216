"""Host-side checks of the paged operators' entry points: what they refuse before any launch, workspace
sizes, and the frequencies, which are host arithmetic. No GPU: every call here is refused on the host or
launches nothing."""
import math
import struct

import numpy as np
import pytest
import torch

import block_sparse_streaming_b200 as bss
from oracle import paged


class Args:
    """The layout of an entry point's argument struct: names and their struct codes, in order."""

    def __init__(self, *fields):
        self.names = [n for names, _ in fields for n in names.split()]
        self.struct = struct.Struct("@" + "".join(c * len(n.split()) for n, c in fields) + "0P")  # in whole pointers


_POOL = (("k_pool v_pool", "P"), ("num_pages page_size", "i"), ("k_page k_row k_head v_page v_row v_head", "q"))
_ROPE = (("rope_dim rope_offset interleaved", "i"), ("rope_scale", "f"))
PLAN_ARGS = Args(("ctx_lens new_lens free_pages block_table cu_seqlens seqlens positions slots counts", "P"),
                 ("bt_stride capacity", "q"), ("batch n_free page_size max_pages", "i"))
ROPE_ARGS = Args(("x positions inv_freq out", "P"), ("tokens x_row_stride out_row_stride", "q"), ("n_heads d", "i"),
                 *_ROPE, ("transposed dtype", "i"))
NORM_ROPE_ARGS = Args(("q k v positions inv_freq q_weight k_weight q_out k_out slots", "P"), *_POOL,
                      ("tokens q_row_stride k_row_stride v_row_stride q_out_row_stride k_out_row_stride", "q"),
                      ("n_heads n_kv_heads d d_v norm_dim", "i"), ("eps", "f"), *_ROPE, ("dtype", "i"))
NORM_ROPE_BACKWARD_ARGS = Args(
    ("dq_out dk_out q k positions inv_freq q_weight k_weight dq dk dq_weight dk_weight workspace", "P"),
    ("workspace_bytes", "N"),
    ("tokens dq_out_row_stride dk_out_row_stride q_row_stride k_row_stride dq_row_stride dk_row_stride", "q"),
    ("n_heads n_kv_heads d norm_dim", "i"), ("eps", "f"), *_ROPE, ("dtype", "i"))
DECODE_ARGS = Args(("q", "P"), *_POOL, ("block_table seqlens out lse workspace", "P"), ("workspace_bytes", "N"),
                   ("q_row_stride bt_stride", "q"), ("batch max_seqlen n_heads n_kv_heads d_qk d_v", "i"),
                   ("block_size n_sink n_local", "i"), ("scale", "f"), ("dtype", "i"))


def pack(args, **values):
    """An argument struct from its fields by name; those not given are 0."""
    assert not set(values) - set(args.names)
    return args.struct.pack(*[values.get(n) or 0 for n in args.names])


INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def L():
    bss.build()
    return bss.lib()


def _plan(L, **over):
    a = dict(ctx=1 << 20, new=1 << 21, batch=4, free=1 << 22, n_free=9, page=16, table=1 << 23, stride=8, cols=8,
             capacity=32, cu=1 << 24, lens=1 << 25, pos=1 << 26, slots=1 << 27, counts=1 << 28)
    a.update(over)
    return L.loza_page_plan(pack(PLAN_ARGS, ctx_lens=a["ctx"], new_lens=a["new"], batch=a["batch"],
                                 free_pages=a["free"], n_free=a["n_free"], page_size=a["page"],
                                 block_table=a["table"], bt_stride=a["stride"], max_pages=a["cols"],
                                 capacity=a["capacity"], cu_seqlens=a["cu"], seqlens=a["lens"], positions=a["pos"],
                                 slots=a["slots"], counts=a["counts"]), None)


@pytest.mark.parametrize("over,code", [
    (dict(batch=0), INVALID), (dict(batch=16385), UNSUPPORTED), (dict(page=24), INVALID), (dict(page=0), INVALID),
    (dict(page=1 << 17), INVALID), (dict(n_free=-1), INVALID), (dict(free=0), INVALID), (dict(table=0), INVALID),
    (dict(stride=7), INVALID), (dict(cols=-1), INVALID), (dict(capacity=-1), INVALID),
    (dict(capacity=1 << 31), INVALID),
    (dict(ctx=0), INVALID), (dict(new=0), INVALID), (dict(cu=0), INVALID), (dict(lens=0), INVALID),
    (dict(counts=0), INVALID), (dict(pos=0), INVALID), (dict(slots=0), INVALID), (dict(pos=(1 << 26) + 4), INVALID),
    (dict(slots=(1 << 27) + 8), INVALID),
])
def test_plan_refuses(L, over, code):
    count = L.loza_launch_count()
    assert _plan(L, **over) == code and L.loza_launch_count() == count


def _rope(L, rope=(64, 128, 0), **over):
    a = dict(x=1 << 20, pos=1 << 21, freq=1 << 22, T=4, H=8, d=192, xs=8 * 192, tr=0, dt=0, out=1 << 23, os=8 * 192)
    a.update(over)
    return L.loza_rope(pack(ROPE_ARGS, x=a["x"], positions=a["pos"], inv_freq=a["freq"], tokens=a["T"],
                            n_heads=a["H"], d=a["d"], x_row_stride=a["xs"], rope_dim=rope[0], rope_offset=rope[1],
                            interleaved=rope[2], rope_scale=1.0, transposed=a["tr"], dtype=a["dt"], out=a["out"],
                            out_row_stride=a["os"]), None)


@pytest.mark.parametrize("rope,over,code", [
    ((64, 128, 0), dict(x=0), INVALID), ((64, 128, 0), dict(out=0), INVALID), ((64, 128, 0), dict(pos=0), INVALID),
    ((64, 128, 0), dict(freq=0), INVALID), ((64, 128, 0), dict(x=(1 << 20) + 1), INVALID),
    ((64, 128, 0), dict(pos=(1 << 21) + 2), INVALID), ((64, 128, 0), dict(freq=(1 << 22) + 4), INVALID),
    ((63, 128, 0), {}, INVALID), ((66, 128, 0), {}, INVALID), ((64, -2, 0), {}, INVALID), ((-2, 0, 0), {}, INVALID),
    ((64, 128, 0), dict(T=-1), INVALID), ((64, 128, 0), dict(T=1 << 31), INVALID), ((64, 128, 0), dict(H=0), INVALID),
    ((64, 128, 0), dict(H=65536, xs=65536 * 192, os=65536 * 192), INVALID),
    ((64, 0, 0), dict(d=1032, xs=8 * 1032, os=8 * 1032), UNSUPPORTED), ((64, 128, 0), dict(xs=8 * 192 - 1), INVALID),
    ((64, 128, 0), dict(os=8 * 192 - 8), INVALID), ((64, 128, 0), dict(tr=2), INVALID),
    ((64, 128, 0), dict(dt=3), INVALID), ((64, 128, 0), dict(out=1 << 20, os=8 * 192 + 8), INVALID),
])
def test_rope_refuses(L, rope, over, code):
    count = L.loza_launch_count()
    assert _rope(L, rope, **over) == code and L.loza_launch_count() == count


def test_rope_of_no_tokens_launches_nothing(L):
    count = L.loza_launch_count()
    assert _rope(L, T=0, x=0, out=0, pos=0) == 0 and L.loza_launch_count() == count
    assert _rope(L, (64, 128, 2)) == INVALID and L.loza_rope(None, None) == INVALID


def _pool(**over):
    a = dict(k_pool=1 << 30, v_pool=1 << 31, num_pages=10, page_size=16, k_page=16 * 256, k_row=256, k_head=128,
             v_page=16 * 256, v_row=256, v_head=128)
    a.update(over)
    return a


def _fwd(L, pool=None, rope=(128, 0, 0), **over):
    a = dict(q=1 << 20, k=1 << 21, v=0, pos=1 << 22, freq=1 << 23, T=4, H=8, Hk=2, d=128, dv=128, qs=1024, ks=256,
             vs=256, qw=1 << 24, kw=1 << 25, nd=128, eps=1e-6, dt=0, qo=1 << 26, qos=1024, ko=1 << 27, kos=256,
             slots=0)
    a.update(over)
    return L.loza_qk_norm_rope(pack(
        NORM_ROPE_ARGS, q=a["q"], k=a["k"], v=a["v"], positions=a["pos"], inv_freq=a["freq"], tokens=a["T"],
        n_heads=a["H"], n_kv_heads=a["Hk"], d=a["d"], d_v=a["dv"], q_row_stride=a["qs"], k_row_stride=a["ks"],
        v_row_stride=a["vs"], q_weight=a["qw"], k_weight=a["kw"], norm_dim=a["nd"], eps=a["eps"], rope_dim=rope[0],
        rope_offset=rope[1], interleaved=rope[2], rope_scale=1.0, dtype=a["dt"], q_out=a["qo"],
        q_out_row_stride=a["qos"], k_out=a["ko"], k_out_row_stride=a["kos"], slots=a["slots"], **(pool or {})), None)


@pytest.mark.parametrize("pool,over,code", [
    (None, dict(q=0), INVALID), (None, dict(k=0), INVALID), (None, dict(qo=0), INVALID), (None, dict(ko=0), INVALID),
    (None, dict(H=0, Hk=0), INVALID), (None, dict(H=-1), INVALID), (None, dict(nd=0), INVALID),
    (None, dict(nd=129), INVALID), (None, dict(eps=-1e-6), INVALID), (None, dict(eps=float("nan")), INVALID),
    (None, dict(qw=(1 << 24) + 1), INVALID), (None, dict(dt=7), INVALID), (None, dict(ks=255), INVALID),
    (None, dict(v=1 << 28), INVALID), (None, dict(slots=1 << 28), INVALID),           # without a pool
    (None, dict(qo=1 << 20, qos=2048), INVALID),                                      # in place, other rows
    ({}, dict(slots=1 << 28), INVALID),                                               # a value pool without values
    (dict(v_pool=None), dict(v=1 << 29, slots=1 << 28), INVALID),                          # values without a pool
    (dict(v_pool=None), dict(), INVALID),                                                  # no slots
    (dict(v_pool=None), dict(slots=(1 << 28) + 4), INVALID),
    (dict(v_pool=None, k_pool=None), dict(slots=1 << 28), INVALID),
    (dict(v_pool=None, page_size=20), dict(slots=1 << 28), INVALID),
    (dict(v_pool=None, num_pages=0), dict(slots=1 << 28), INVALID),
    (dict(v_pool=None, num_pages=1 << 28), dict(slots=1 << 28), INVALID),                  # more rows than 31 bits
    (dict(v_pool=None, k_row=-256), dict(slots=1 << 28), INVALID),
    (dict(v_pool=None), dict(slots=1 << 28, H=8, Hk=0, k=0, kw=0), INVALID),
    ({}, dict(v=1 << 29, slots=1 << 28, dv=0), INVALID), ({}, dict(v=1 << 29, slots=1 << 28, vs=255), INVALID),
])
def test_norm_rope_refuses(L, pool, over, code):
    count = L.loza_launch_count()
    assert _fwd(L, _pool(**pool) if pool is not None else None, **over) == code
    assert L.loza_launch_count() == count


def _bwd(L, rope=(128, 0, 0), **over):
    a = dict(gq=1 << 20, gk=1 << 21, q=1 << 22, k=1 << 23, pos=1 << 24, freq=1 << 25, T=4, H=8, Hk=2, d=128, gqs=1024,
             gks=256, qs=1024, ks=256, qw=1 << 26, kw=1 << 27, nd=128, eps=1e-6, dt=0, dq=1 << 28, dqs=1024,
             dk=1 << 29, dks=256, dqw=1 << 30, dkw=(1 << 30) + 4096, ws=1 << 31, wsb=1 << 22)
    a.update(over)
    return L.loza_qk_norm_rope_backward(pack(
        NORM_ROPE_BACKWARD_ARGS, dq_out=a["gq"], dk_out=a["gk"], q=a["q"], k=a["k"], positions=a["pos"],
        inv_freq=a["freq"], tokens=a["T"], n_heads=a["H"], n_kv_heads=a["Hk"], d=a["d"], dq_out_row_stride=a["gqs"],
        dk_out_row_stride=a["gks"], q_row_stride=a["qs"], k_row_stride=a["ks"], q_weight=a["qw"], k_weight=a["kw"],
        norm_dim=a["nd"], eps=a["eps"], rope_dim=rope[0], rope_offset=rope[1], interleaved=rope[2], rope_scale=1.0,
        dtype=a["dt"], dq=a["dq"], dq_row_stride=a["dqs"], dk=a["dk"], dk_row_stride=a["dks"], dq_weight=a["dqw"],
        dk_weight=a["dkw"], workspace=a["ws"], workspace_bytes=a["wsb"]), None)


@pytest.mark.parametrize("over,code", [
    (dict(gq=0), INVALID), (dict(gk=0), INVALID), (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(dq=0), INVALID),
    (dict(dk=0), INVALID), (dict(dqw=0), INVALID), (dict(qw=0), INVALID), (dict(dkw=0), INVALID),
    (dict(H=0), INVALID), (dict(ws=0), INVALID), (dict(ws=(1 << 31) + 8), INVALID), (dict(wsb=1024), WORKSPACE),
    (dict(nd=0), INVALID), (dict(dqs=1023), INVALID), (dict(dq=1 << 20, dqs=2048), INVALID),
    (dict(dk=1 << 23, dks=512), INVALID), (dict(dqw=(1 << 30) + 2), INVALID), (dict(dt=-1), INVALID),
])
def test_norm_rope_backward_refuses(L, over, code):
    count = L.loza_launch_count()
    assert _bwd(L, **over) == code and L.loza_launch_count() == count


def _decode(L, pool={}, params=None, **over):
    a = dict(q=1 << 20, qs=1024, bt=1 << 21, bts=8, lens=1 << 22, batch=3, max_len=128, H=8, Hk=2, d=128, dv=128,
             dt=0, out=1 << 23, lse=1 << 24, ws=1 << 25, wsb=1 << 30)
    a.update(over)
    w = params or bss.Params(0.1, 128, 0, -1)
    return L.loza_ssa_decode_paged_kv(pack(
        DECODE_ARGS, q=a["q"], q_row_stride=a["qs"], block_table=a["bt"], bt_stride=a["bts"],
        seqlens=a["lens"], batch=a["batch"], max_seqlen=a["max_len"], n_heads=a["H"], n_kv_heads=a["Hk"],
        d_qk=a["d"], d_v=a["dv"], block_size=w.block_size, n_sink=w.n_sink, n_local=w.n_local, scale=w.scale,
        dtype=a["dt"], out=a["out"], lse=a["lse"], workspace=a["ws"], workspace_bytes=a["wsb"], **_pool(**pool)),
        None)


@pytest.mark.parametrize("pool,over,code", [
    ({}, dict(q=0), INVALID), ({}, dict(q=(1 << 20) + 8), INVALID), (dict(v_pool=None), {}, INVALID),
    (dict(k_pool=None), {}, INVALID), (dict(k_pool=(1 << 30) + 8), {}, INVALID), ({}, dict(bt=0), INVALID),
    ({}, dict(lens=0), INVALID), ({}, dict(out=0), INVALID), ({}, dict(lse=0), INVALID), ({}, dict(batch=0), INVALID),
    ({}, dict(batch=65536), INVALID), ({}, dict(max_len=0), INVALID),
    ({}, dict(max_len=(1 << 30) + 1, bts=1 << 30), INVALID), ({}, dict(max_len=129), INVALID),
    ({}, dict(bts=7), INVALID), ({}, dict(H=7), INVALID), ({}, dict(qs=1016), INVALID), ({}, dict(qs=1028), INVALID),
    (dict(k_row=260), {}, INVALID), (dict(v_head=132), {}, INVALID),
    (dict(k_page=-4096), {}, INVALID), (dict(page_size=48), {}, INVALID), ({}, dict(dt=3), INVALID),
    (dict(page_size=8), dict(bts=16), UNSUPPORTED), ({}, dict(dt=2), UNSUPPORTED),
    ({}, dict(d=96, qs=768), UNSUPPORTED), ({}, dict(d=576, dv=512, qs=8 * 576), UNSUPPORTED),
    ({}, dict(ws=0), INVALID), ({}, dict(ws=(1 << 25) + 4), INVALID), ({}, dict(wsb=4096), WORKSPACE),
])
def test_decode_refuses(L, pool, over, code):
    count = L.loza_launch_count()
    assert _decode(L, pool, **over) == code and L.loza_launch_count() == count


def test_decode_refuses_windows(L):
    count = L.loza_launch_count()
    for p in (bss.Params(0.1, 96), bss.Params(0.1, 128, 1, 0), bss.Params(0.1, 128, -1, 7)):
        assert _decode(L, params=p) == UNSUPPORTED
    assert L.loza_launch_count() == count


def test_workspace_sizes(L):
    assert L.loza_qk_norm_rope_workspace_size(128) == 2 * L.loza_qk_norm_rope_workspace_size(64) > 0
    assert L.loza_qk_norm_rope_workspace_size(0) == L.loza_qk_norm_rope_workspace_size(1025) == 0
    size = L.loza_decode_paged_kv_workspace_size
    assert size(32, 8, 128, 128) == size(64, 64, 192, 128) > size(8, 8, 64, 64) > 0
    assert size(32, 8, 128, 64) == size(30, 8, 128, 128) == size(0, 1, 64, 64) == 0


@pytest.mark.parametrize("dim", [2, 24, 64, 576])
@pytest.mark.parametrize("scaling,factor", [(None, 1.0), ("linear", 4.0), ("ntk", 8.0), ("yarn", 1.0), ("yarn", 32.0)])
def test_frequencies(L, dim, scaling, factor):
    if scaling == "ntk" and dim == 2:
        with pytest.raises(bss.LozaError):
            bss.rope_frequencies(dim, scaling=scaling, factor=factor)
        return
    got, scale = bss.rope_frequencies(dim, 1e6, scaling, factor, 8192)
    want, want_scale = paged.frequencies(dim, 1e6, scaling, factor, 8192)
    # a few roundings of pow in 64 bits, and one to 32 bits for the scale
    assert np.allclose(got.numpy(), want, rtol=1e-14, atol=0) and abs(scale - want_scale) <= 2 ** -24 * want_scale


def test_frequencies_refuse(L):
    for kw in (dict(rope_dim=3), dict(rope_dim=0), dict(rope_dim=1026), dict(theta=1.0), dict(theta=math.inf),
               dict(factor=0.5), dict(factor=math.nan), dict(scaling="yarn", original_max=0),
               dict(scaling="yarn", beta_fast=1.0, beta_slow=2.0)):
        with pytest.raises(bss.LozaError):
            bss.rope_frequencies(**{"rope_dim": 64, **kw})
    with pytest.raises(ValueError):
        bss.rope_frequencies(64, scaling="other")


def test_binding_refuses_host_tensors(L):
    q, k, pos = torch.zeros(2, 8, 64), torch.zeros(2, 2, 64), torch.zeros(2, dtype=torch.int32)
    freq, rope = torch.zeros(32, dtype=torch.float64), bss.RopeParams(64)
    for call in (lambda: bss.loza_rope(q, pos, freq, rope), lambda: bss.loza_qk_norm_rope(q, k, pos, freq, rope),
                 lambda: bss.loza_qk_norm_rope_backward(q, k, q, k, pos, freq, rope),
                 lambda: bss.loza_page_plan(pos, pos, pos, pos.view(2, 1), 16, 4),
                 lambda: bss.loza_ssa_decode_paged_kv(q, q, q, pos.view(2, 1), pos, 1, bss.Params(1.0))):
        with pytest.raises(TypeError):
            call()
