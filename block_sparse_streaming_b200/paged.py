"""Serving and training operators around the attention: page plan, position rotation, norms of query and key
heads with their gradient, decode over paged K and V pools.

Marshalling only, like the rest of the package (which re-exports these names). The calls are short, so this
layer is too: a call's arguments travel as one packed struct, checks that hold cost one comparison each, and
what went wrong is worked out only after one of them failed. Every tensor of a call lives on one GPU, which
need not be the current one; with `stream` the whole call runs there, its buffers included. Nothing is read back
to the host, and every call can be captured into a graph."""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import LozaError, Params, lib

LOZA_BF16, LOZA_FP16, LOZA_FP32 = 0, 1, 2
_DTYPES = {torch.bfloat16: LOZA_BF16, torch.float16: LOZA_FP16, torch.float32: LOZA_FP32}
_SCALING = {None: 0, "none": 0, "linear": 1, "ntk": 2, "yarn": 3}  # LOZA_ROPE_*
_i32, _i64, _f32, _f64, _u8 = torch.int32, torch.int64, torch.float32, torch.float64, torch.uint8
_Tensor, _empty, _empty_like = torch.Tensor, torch.empty, torch.empty_like
_current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


class RopeParams(ctypes.Structure):
    """loza_rope_params {rope_dim, rope_offset, interleaved, scale}."""
    _fields_ = [("rope_dim", ctypes.c_int32), ("rope_offset", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("scale", ctypes.c_float)]

    def __init__(self, rope_dim: int, rope_offset: int = 0, interleaved: bool = False, scale: float = 1.0):
        super().__init__(rope_dim, rope_offset, int(bool(interleaved)), scale)


class Args:
    """The layout of an entry point's argument struct: names and their struct codes, in order."""

    def __init__(self, *fields):
        self.names = [n for names, _ in fields for n in names.split()]
        self.codes = "@" + "".join(code * len(names.split()) for names, code in fields)
        self.pack = struct.Struct(self.codes + "0P").pack  # the struct's size is a multiple of 8


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
_plan_pack, _rope_pack, _fwd_pack, _bwd_pack, _decode_pack = (
    a.pack for a in (PLAN_ARGS, ROPE_ARGS, NORM_ROPE_ARGS, NORM_ROPE_BACKWARD_ARGS, DECODE_ARGS))


def _on_its_device(fn):
    """Run `fn` with the device of its first tensor current and, if `stream` is given, that stream current too:
    buffers made inside belong to the stream that uses them."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        first = args[0] if args and args[0] is not None else args[1] if len(args) > 1 else None
        if not isinstance(first, _Tensor) or not first.is_cuda:
            raise TypeError(f"{fn.__name__}: the tensors must be CUDA tensors, the first ones given by position")
        if stream is None:
            if first.get_device() == _current_device():
                return fn(*args, **kw)
        elif stream.device != first.device:
            raise ValueError(f"{fn.__name__}: stream and tensors are on different devices")
        with torch.cuda.device(first.device), torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _bad(t, name, device, dtype, ndim, shape=None):
    """Why `t` is not what a call takes."""
    if not isinstance(t, _Tensor):
        return TypeError(f"{name} must be a tensor")
    if t.get_device() != device:
        return (ValueError if t.is_cuda else TypeError)(f"{name} must be on cuda:{device}")
    if t.dtype is not dtype:
        return TypeError(f"{name} must be {dtype}")
    if shape is not None and t.shape != shape:
        return ValueError(f"{name} must have shape {shape}")
    if t.dim() != ndim:
        return ValueError(f"{name} must have {ndim} dimensions")
    return ValueError(f"{name} must be contiguous" if ndim != 3 else
                      f"{name}: heads and head dim must be contiguous within a row")


def _plain(t, name, device, dtype, shape):
    """Address of a contiguous tensor of exactly this dtype and shape."""
    if not isinstance(t, _Tensor) or t.get_device() != device or t.dtype is not dtype or t.shape != shape \
            or not t.is_contiguous():
        raise _bad(t, name, device, dtype, len(shape), shape)
    return t.data_ptr()


def _rows(t, name, device, dtype, shape):
    """(address, row stride) of [rows, heads, dim] with heads and dim contiguous (of one row: any stride that fits)."""
    if not isinstance(t, _Tensor) or t.get_device() != device or t.dtype is not dtype or t.shape != shape:
        raise _bad(t, name, device, dtype, 3, shape)
    row, head, one = t.stride()
    if (one != 1 and shape[2] > 1) or (head != shape[2] and shape[1] > 1):
        raise _bad(t, name, device, dtype, 3)
    return t.data_ptr(), row if shape[0] > 1 else shape[1] * shape[2]


def _shape3(t, name, device, dtype):
    if not isinstance(t, _Tensor) or t.dim() != 3 or t.get_device() != device or t.dtype is not dtype:
        raise _bad(t, name, device, dtype, 3)
    return t.shape


def _first(t, name):
    """(device, dtype, its code) of a call's first tensor."""
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32")
    return t.get_device(), t.dtype, code


def _table(t, device, batch):
    """(address, row stride, columns) of a block table [batch, columns]."""
    if not isinstance(t, _Tensor) or t.get_device() != device or t.dtype is not _i32 or t.dim() != 2:
        raise _bad(t, "block_table", device, _i32, 2)
    (rows, cols), (row, one) = t.shape, t.stride()
    if rows != batch or (one != 1 and cols > 1):
        raise ValueError("block_table must be [batch, columns] with contiguous rows")
    return t.data_ptr(), row if batch > 1 else cols, cols


def _pool(t, name, device, dtype, heads, dim):
    """(address, pages, rows, page stride, row stride, head stride) of a pool [pages, rows, heads, dim]."""
    if not isinstance(t, _Tensor) or t.get_device() != device or t.dtype is not dtype or t.dim() != 4:
        raise _bad(t, name, device, dtype, 4)
    (pages, rows, h, d), (page, row, head, one) = t.shape, t.stride()
    if h != heads or d != dim or (one != 1 and d > 1):
        raise ValueError(f"{name} must be [pages, rows, {heads}, {dim}] with contiguous columns")
    return t.data_ptr(), pages, rows, page, row, head if heads > 1 else 0


def _failed(status, name):
    raise LozaError(status, name)


@_on_its_device
def loza_page_plan(ctx_lens, new_lens, free_pages, block_table, page_size: int, capacity: int):
    """Block table, slots and offsets of a step of a paged cache. ctx_lens, new_lens [B] int32: tokens cached and
    tokens appended; free_pages [F] int32: pages to hand out, in order; block_table [B, columns] int32 (rows may be
    strided), updated in place; capacity: packed rows of the step. Returns (cu_seqlens [B+1] int32, seqlens [B]
    int32, positions [capacity] int32, slots [capacity] int64, counts [3] int32: tokens, pages taken, requests short
    of pages)."""
    i = ctx_lens.get_device()
    if not isinstance(free_pages, _Tensor):
        raise TypeError("free_pages must be a tensor")
    B, F = ctx_lens.numel(), free_pages.numel()
    ctx, new = _plain(ctx_lens, "ctx_lens", i, _i32, (B,)), _plain(new_lens, "new_lens", i, _i32, (B,))
    free = _plain(free_pages, "free_pages", i, _i32, (F,))
    table, bt_stride, cols = _table(block_table, i, B)
    if B < 1 or capacity < 0:
        _failed(-1, "loza_page_plan")
    dev = ctx_lens.device
    cu, lens = _empty(B + 1, dtype=_i32, device=dev), _empty_like(ctx_lens)
    positions, slots = _empty(capacity, dtype=_i32, device=dev), _empty(capacity, dtype=_i64, device=dev)
    counts = _empty(3, dtype=_i32, device=dev)
    rc = lib().loza_page_plan(_plan_pack(ctx, new, free, table, cu.data_ptr(), lens.data_ptr(), positions.data_ptr(),
                                         slots.data_ptr(), counts.data_ptr(), bt_stride, capacity, B, F, page_size,
                                         cols), _raw_stream(i))
    if rc:
        _failed(rc, "loza_page_plan")
    return cu, lens, positions, slots, counts


def rope_frequencies(rope_dim: int, theta: float = 10000.0, scaling=None, factor: float = 1.0,
                     original_max: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """Angles per position (float64 [rope_dim / 2], on `device`) and the scale of RopeParams; scaling: None, "linear",
    "ntk" or "yarn" (for contexts `factor` times longer than original_max)."""
    if scaling not in _SCALING:
        raise ValueError(f"scaling must be one of {[k for k in _SCALING if k]} or None")
    freq = _empty(max(0, int(rope_dim)) // 2, dtype=_f64)
    scale = ctypes.c_float()
    rc = lib().loza_rope_frequencies(float(theta), int(rope_dim), _SCALING[scaling], float(factor),
                                     float(original_max), float(beta_fast), float(beta_slow), freq.data_ptr(),
                                     ctypes.addressof(scale))
    if rc:
        _failed(rc, "loza_rope_frequencies")
    return (freq.to(device) if device is not None else freq), scale.value


@_on_its_device
def loza_rope(x, positions, inv_freq, rope: RopeParams, out=None, transposed: bool = False):
    """Position rotation of x [T, H, d] (bf16, fp16 or fp32; rows may be strided) by positions [T] int32 and inv_freq
    [rope_dim / 2] float64. out may be x (in place). transposed: the gradient (dx from dout). Returns out."""
    i, dtype, code = _first(x, "x")
    shape = T, H, d = _shape3(x, "x", i, dtype)
    n = rope.rope_dim
    pos = _plain(positions, "positions", i, _i32, (T,))
    freq = _plain(inv_freq, "inv_freq", i, _f64, (n // 2,))
    xp, x_row = _rows(x, "x", i, dtype, shape)
    if out is None:
        out = _empty(shape, dtype=dtype, device=x.device)
        op, o_row = out.data_ptr(), H * d
    else:
        op, o_row = _rows(out, "out", i, dtype, shape)
    rc = lib().loza_rope(_rope_pack(xp, pos, freq, op, T, x_row, o_row, H, d, n, rope.rope_offset, rope.interleaved,
                                    rope.scale, 1 if transposed else 0, code), _raw_stream(i))
    if rc:
        _failed(rc, "loza_rope")
    return out


def _weight(w, rows, name, norm_dim, device, dtype):
    """(address, norm_dim) of a side's weight; norm_dim is its length unless given."""
    if w is None:
        return 0, norm_dim
    if rows is None:
        raise ValueError(f"{name} without its rows")
    if norm_dim is None:
        norm_dim = w.numel() if isinstance(w, _Tensor) else 0
    return _plain(w, name, device, dtype, (norm_dim,)), norm_dim


_NO_POOL = (0, 0, 0, 0, 0, 0)


@_on_its_device
def loza_qk_norm_rope(q, k, positions, inv_freq, rope: RopeParams, q_weight=None, k_weight=None, eps: float = 1e-6,
                      v=None, k_pool=None, v_pool=None, slots=None, q_out=None, k_out=None, norm_dim=None):
    """RMS norm of each head of q [T, H, d] and k [T, Hkv, d] over its first norm_dim columns (default: the weights'
    length; a side without weight is not normed), then the rotation, and - with k_pool [pages, rows, Hkv, d] and slots
    [T] int64 - the keys (and v [T, Hkv, d_v] into v_pool) written to the paged cache. q or k may be None. Returns
    (q_out, k_out); k_out is None when there is a pool and none was given."""
    i, dtype, code = _first(q if q is not None else k, "q or k")
    H = Hk = d_v = 0
    qp = kp = vp = q_row = k_row = v_row = qo = ko = qo_row = ko_row = sp = 0
    if q is not None:
        shape = T, H, d = _shape3(q, "q", i, dtype)
        qp, q_row = _rows(q, "q", i, dtype, shape)
        if q_out is None:
            q_out = _empty(shape, dtype=dtype, device=q.device)
            qo, qo_row = q_out.data_ptr(), H * d
        else:
            qo, qo_row = _rows(q_out, "q_out", i, dtype, shape)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if k is not None:
        shape = _shape3(k, "k", i, dtype)
        if q is not None and (shape[0] != T or shape[2] != d):
            raise ValueError("q and k must agree in tokens and head dim")
        T, Hk, d = shape
        kp, k_row = _rows(k, "k", i, dtype, shape)
        if k_out is None and k_pool is None:
            k_out = _empty(shape, dtype=dtype, device=k.device)
        if k_out is not None:
            ko, ko_row = _rows(k_out, "k_out", i, dtype, shape)
    elif k_out is not None or k_pool is not None:
        raise ValueError("k_out and k_pool need k")
    pool_k = pool_v = _NO_POOL
    if k_pool is not None:
        if (v is None) != (v_pool is None):
            raise ValueError("v and v_pool come together")
        pool_k = _pool(k_pool, "k_pool", i, dtype, Hk, d)
        sp = _plain(slots, "slots", i, _i64, (T,))
        if v is not None:
            shape = _shape3(v, "v", i, dtype)
            d_v = shape[2]
            if shape[0] != T or shape[1] != Hk:
                raise ValueError("v and k must agree in tokens and heads")
            vp, v_row = _rows(v, "v", i, dtype, shape)
            pool_v = _pool(v_pool, "v_pool", i, dtype, Hk, d_v)
            if pool_v[1:3] != pool_k[1:3]:
                raise ValueError("k_pool and v_pool must have the same pages")
    elif v is not None or v_pool is not None or slots is not None:
        raise ValueError("v, v_pool and slots need k_pool")
    n = rope.rope_dim
    pos = _plain(positions, "positions", i, _i32, (T,))
    freq = _plain(inv_freq, "inv_freq", i, _f64, (n // 2,))
    qw, norm_dim = _weight(q_weight, q, "q_weight", norm_dim, i, dtype)
    kw, norm_dim = _weight(k_weight, k, "k_weight", norm_dim, i, dtype)
    rc = lib().loza_qk_norm_rope(
        _fwd_pack(qp, kp, vp, pos, freq, qw, kw, qo, ko, sp, pool_k[0], pool_v[0], pool_k[1], pool_k[2], pool_k[3],
                  pool_k[4], pool_k[5], pool_v[3], pool_v[4], pool_v[5], T, q_row, k_row, v_row, qo_row, ko_row, H, Hk,
                  d, d_v, norm_dim or 0, eps, n, rope.rope_offset, rope.interleaved, rope.scale, code),
        _raw_stream(i))
    if rc:
        _failed(rc, "loza_qk_norm_rope")
    return q_out, k_out


@_on_its_device
def loza_qk_norm_rope_backward(dq_out, dk_out, q, k, positions, inv_freq, rope: RopeParams, q_weight=None,
                               k_weight=None, eps: float = 1e-6, dq=None, dk=None, norm_dim=None, workspace=None):
    """Gradient of loza_qk_norm_rope: (dq, dk, dq_weight, dk_weight) from dq_out and dk_out and the forward's inputs;
    the weights' gradients are fp32 [norm_dim], None for a side without weight. A side is given (dq_out, or dk_out) or
    None; q and k are only read where there is a weight."""
    first = dq_out if dq_out is not None else dk_out
    i, dtype, code = _first(first, "dq_out or dk_out")
    H = Hk = 0
    gq = gk = qp = kp = dqp = dkp = gq_row = gk_row = q_row = k_row = dq_row = dk_row = dqw_p = dkw_p = wp = 0
    dqw = dkw = None
    ws_bytes = 0
    qw, norm_dim = _weight(q_weight, dq_out, "q_weight", norm_dim, i, dtype)
    kw, norm_dim = _weight(k_weight, dk_out, "k_weight", norm_dim, i, dtype)
    dev = first.device
    if dq_out is not None:
        shape = T, H, d = _shape3(dq_out, "dq_out", i, dtype)
        gq, gq_row = _rows(dq_out, "dq_out", i, dtype, shape)
        if qw:
            qp, q_row = _rows(q, "q", i, dtype, shape)
            dqw = _empty(norm_dim, dtype=_f32, device=dev)
            dqw_p = dqw.data_ptr()
        if dq is None:
            dq = _empty(shape, dtype=dtype, device=dev)
            dqp, dq_row = dq.data_ptr(), H * d
        else:
            dqp, dq_row = _rows(dq, "dq", i, dtype, shape)
    elif dq is not None:
        raise ValueError("dq without dq_out")
    if dk_out is not None:
        shape = _shape3(dk_out, "dk_out", i, dtype)
        if dq_out is not None and (shape[0] != T or shape[2] != d):
            raise ValueError("dq_out and dk_out must agree in tokens and head dim")
        T, Hk, d = shape
        gk, gk_row = _rows(dk_out, "dk_out", i, dtype, shape)
        if kw:
            kp, k_row = _rows(k, "k", i, dtype, shape)
            dkw = _empty(norm_dim, dtype=_f32, device=dev)
            dkw_p = dkw.data_ptr()
        if dk is None:
            dk = _empty(shape, dtype=dtype, device=dev)
            dkp, dk_row = dk.data_ptr(), Hk * d
        else:
            dkp, dk_row = _rows(dk, "dk", i, dtype, shape)
    elif dk is not None:
        raise ValueError("dk without dk_out")
    n = rope.rope_dim
    pos = _plain(positions, "positions", i, _i32, (T,))
    freq = _plain(inv_freq, "inv_freq", i, _f64, (n // 2,))
    L = lib()
    if qw or kw:
        if workspace is None:
            workspace = _empty(L.loza_qk_norm_rope_workspace_size(norm_dim), dtype=_u8, device=dev)
        wp, ws_bytes = _workspace(workspace, i)
    rc = L.loza_qk_norm_rope_backward(
        _bwd_pack(gq, gk, qp, kp, pos, freq, qw, kw, dqp, dkp, dqw_p, dkw_p, wp, ws_bytes, T, gq_row, gk_row, q_row,
                  k_row, dq_row, dk_row, H, Hk, d, norm_dim or 0, eps, n, rope.rope_offset, rope.interleaved,
                  rope.scale, code), _raw_stream(i))
    if rc:
        _failed(rc, "loza_qk_norm_rope_backward")
    return dq, dk, dqw, dkw


def _workspace(t, device):
    """(address, bytes) of a workspace of any dtype."""
    if not isinstance(t, _Tensor) or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{device}")
    return t.data_ptr(), t.numel() * t.element_size()


@_on_its_device
def loza_ssa_decode_paged_kv(q, k_pool, v_pool, block_table, seqlens, max_seqlen: int, params: Params, out=None,
                             lse=None, workspace=None):
    """Decode over paged K and V pools, heads of their own or shared by groups. q [B, H, d_qk] bf16 or fp16 (rows may
    be strided); k_pool [pages, rows, Hkv, d_qk] and v_pool [pages, rows, Hkv, d_v] (any strides that are multiples of
    16 bytes, columns contiguous); block_table [B, columns] int32; seqlens [B] int32, 0 for an idle row (out 0, lse
    -inf). Returns (out [B, H, d_v], lse [B, H])."""
    i, dtype, code = _first(q, "q")
    shape = B, H, d = _shape3(q, "q", i, dtype)
    qp, q_row = _rows(q, "q", i, dtype, shape)
    lens = _plain(seqlens, "seqlens", i, _i32, (B,))
    table, bt_stride, cols = _table(block_table, i, B)
    if not isinstance(k_pool, _Tensor) or not isinstance(v_pool, _Tensor) or k_pool.dim() != 4 or v_pool.dim() != 4:
        raise TypeError("k_pool and v_pool must be tensors of 4 dimensions")
    Hk, d_v = k_pool.size(2), v_pool.size(3)
    kp, pages, rows, k_page, k_row, k_head = _pool(k_pool, "k_pool", i, dtype, Hk, d)
    vp, v_pages, v_rows, v_page, v_row, v_head = _pool(v_pool, "v_pool", i, dtype, Hk, d_v)
    if v_pages != pages or v_rows != rows:
        raise ValueError("k_pool and v_pool must have the same pages")
    if cols * rows < max_seqlen:
        raise ValueError("block_table has too few columns for max_seqlen")
    dev = q.device
    if out is None:
        out = _empty((B, H, d_v), dtype=dtype, device=dev)
        op = out.data_ptr()
    else:
        op = _plain(out, "out", i, dtype, (B, H, d_v))
    if lse is None:
        lse = _empty((B, H), dtype=_f32, device=dev)
        lp = lse.data_ptr()
    else:
        lp = _plain(lse, "lse", i, _f32, (B, H))
    L = lib()
    if workspace is None:
        workspace = _empty(max(16, L.loza_decode_paged_kv_workspace_size(H, Hk, d, d_v)), dtype=_u8, device=dev)
    wp, ws_bytes = _workspace(workspace, i)
    rc = L.loza_ssa_decode_paged_kv(
        _decode_pack(qp, kp, vp, pages, rows, k_page, k_row, k_head, v_page, v_row, v_head, table, lens, op, lp, wp,
                     ws_bytes, q_row, bt_stride, B, max_seqlen, H, Hk, d, d_v, params.block_size, params.n_sink,
                     params.n_local, params.scale, code), _raw_stream(i))
    if rc:
        _failed(rc, "loza_ssa_decode_paged_kv")
    return out, lse
