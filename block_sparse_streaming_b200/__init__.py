"""B200 (sm_100a) streaming sparse attention of LongCat ZigZag Attention.

Python binding of the C ABI in ``include/loza_ssa.h``: argument marshalling
only. Every step of the computation runs in the CUDA kernels of
``libloza_ssa.so``; there is no CPU path. If the library is missing or cannot
be loaded, every call raises.

Tensors are torch CUDA tensors (PyTorch provides device memory and streams):
  q [T, H, d_qk], k [T, Hkv, d_qk], v [T, Hkv, d_v] bf16 (rows may be strided,
  heads and head dims contiguous); for the absorbed MLA layout pass the latent
  [T, 1, 576] as k and its first 512 columns (a view of the same storage) as v.
"""
from __future__ import annotations

import ctypes
import functools
import os

from ._build import LIB_PATH, build  # noqa: F401  (build is re-exported)

LOZA_UNBOUNDED = -1
LOZA_OP_PREFILL, LOZA_OP_DECODE, LOZA_OP_BACKWARD, LOZA_OP_PREFILL_HOST = 0, 1, 2, 3

_STATUS = {
    0: "LOZA_OK",
    -1: "LOZA_ERR_INVALID_ARG",
    -2: "LOZA_ERR_UNSUPPORTED",
    -3: "LOZA_ERR_WORKSPACE",
    -4: "LOZA_ERR_CUDA",
    -5: "LOZA_ERR_TIMEOUT",
}

# Every symbol include/loza_ssa.h declares.
EXPORTED = [
    "loza_ssa_workspace_size",
    "loza_ssa_prefill",
    "loza_ssa_prefill_host",
    "loza_ssa_decode",
    "loza_ssa_decode_noalloc",
    "loza_ssa_decode_paged",
    "loza_ssa_merge",
    "loza_ssa_mix",
    "loza_ssa_backward",
    "loza_status_string",
    "loza_device_status",
    "loza_launch_count",
    "loza_hi_page_keys",
    "loza_hi_workspace_size",
    "loza_hi_select",
    "loza_ssa_decode_selected",
    "loza_hi_decode",
    "loza_page_plan",
    "loza_rope_frequencies",
    "loza_rope",
    "loza_qk_norm_rope",
    "loza_qk_norm_rope_workspace_size",
    "loza_qk_norm_rope_backward",
    "loza_decode_paged_kv_workspace_size",
    "loza_ssa_decode_paged_kv",
    "loza_wait_selftest",
]


class LozaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {_STATUS.get(status, status)}")
        self.status = status


class Params(ctypes.Structure):
    """loza_ssa_params {block_size, n_sink, n_local, scale}."""
    _fields_ = [("block_size", ctypes.c_int32), ("n_sink", ctypes.c_int32),
                ("n_local", ctypes.c_int32), ("scale", ctypes.c_float)]

    def __init__(self, scale: float, block_size: int = 128, n_sink: int = 1, n_local: int = 7):
        super().__init__(block_size, n_sink, n_local, scale)


class RopeParams(ctypes.Structure):
    """loza_rope_params {rope_dim, rope_offset, interleaved, scale}."""
    _fields_ = [("rope_dim", ctypes.c_int32), ("rope_offset", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("scale", ctypes.c_float)]

    def __init__(self, rope_dim: int, rope_offset: int = 0, interleaved: bool = False, scale: float = 1.0):
        super().__init__(rope_dim, rope_offset, int(bool(interleaved)), scale)


class KvPool(ctypes.Structure):
    """loza_kv_pool: base pointers, pages and strides of a paged cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32)] + \
               [(f"{s}_{n}_stride", ctypes.c_int64) for s in "kv" for n in ("page", "row", "head")]


_lib = None
_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


def lib() -> ctypes.CDLL:
    """The loaded libloza_ssa.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run block_sparse_streaming_b200.build() "
                               "(nvcc, sm_100a); there is no fallback path")
        L = ctypes.CDLL(LIB_PATH)
        L.loza_ssa_workspace_size.restype = _sz
        L.loza_ssa_workspace_size.argtypes = [ctypes.c_int, _i32, _i64, _i32, _i32, _i32, _i32, _i32, Params]
        L.loza_ssa_prefill.restype = ctypes.c_int
        L.loza_ssa_prefill.argtypes = [_vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32, _i32, _i32,
                                       _i64, _i64, _i64, Params, _vp, _vp, _vp, _sz, _vp]
        L.loza_ssa_prefill_host.restype = ctypes.c_int
        L.loza_ssa_prefill_host.argtypes = [_vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32, _i32, _i32, Params,
                                            _vp, _vp, _vp, _sz, _vp]
        L.loza_ssa_decode.restype = ctypes.c_int
        L.loza_ssa_decode.argtypes = [_vp, _vp, _vp, _vp, _i32, _i32, _i64, _i64, _i32, _i32, _i32, _i32,
                                      Params, _vp, _vp, _vp, _sz, _vp]
        L.loza_ssa_decode_noalloc.restype = ctypes.c_int
        L.loza_ssa_decode_noalloc.argtypes = [_vp, _vp, _vp, _vp, _i32, _i32, _i64, _i64, _i32, _i32, _i32, _i32,
                                              Params, _vp, _vp, _vp]
        L.loza_ssa_backward.restype = ctypes.c_int
        L.loza_ssa_backward.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i32, _i32,
                                        _i32, _i32, Params, _vp, _vp, _vp, _vp, _sz, _vp]
        L.loza_ssa_decode_paged.restype = ctypes.c_int
        L.loza_ssa_decode_paged.argtypes = [_vp, _vp, _i32, _i64, _vp, _i32, _vp, _i32, _i32, _i32, Params, _vp, _vp,
                                            _vp, _sz, _vp]
        L.loza_ssa_merge.restype = ctypes.c_int
        L.loza_ssa_merge.argtypes = [_vp, _vp, _vp, _vp, _i64, _i32, _vp, _vp, _vp]
        L.loza_ssa_mix.restype = ctypes.c_int
        L.loza_ssa_mix.argtypes = [_vp, _vp, _i64, ctypes.c_float, _vp, _vp]
        L.loza_status_string.restype = ctypes.c_char_p
        L.loza_status_string.argtypes = [ctypes.c_int]
        L.loza_device_status.restype = ctypes.c_int
        L.loza_device_status.argtypes = [_vp]
        L.loza_launch_count.restype = ctypes.c_uint64
        L.loza_launch_count.argtypes = []
        L.loza_wait_selftest.restype = ctypes.c_int
        L.loza_wait_selftest.argtypes = [ctypes.c_uint32, _vp]
        L.loza_hi_page_keys.restype = ctypes.c_int
        L.loza_hi_page_keys.argtypes = [_vp, _i64, _i64, _vp, _i32, _i32, _i32, _vp, _vp]
        L.loza_hi_workspace_size.restype = _sz
        L.loza_hi_workspace_size.argtypes = [_i32, _i32, _i32, _i32, Params]
        L.loza_hi_select.restype = ctypes.c_int
        L.loza_hi_select.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _i32, _i32, _i32, Params, _i32, _i32, _vp, _vp,
                                     _sz, _vp]
        L.loza_ssa_decode_selected.restype = ctypes.c_int
        L.loza_ssa_decode_selected.argtypes = [_vp, _vp, _i64, _i64, _vp, _i32, _i32, Params, _vp, _i32, _vp, _vp,
                                               _vp, _sz, _vp]
        L.loza_hi_decode.restype = ctypes.c_int
        L.loza_hi_decode.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _i32, _i32, _i32, Params,
                                     _i32, _i32, _vp, _vp, _vp, _sz, _vp]
        _f32, _f64, _pool = ctypes.c_float, ctypes.c_double, ctypes.POINTER(KvPool)
        L.loza_page_plan.restype = ctypes.c_int
        L.loza_page_plan.argtypes = [_vp, _vp, _i32, _vp, _i32, _i32, _vp, _i64, _i32, _i64, _vp, _vp, _vp, _vp, _vp,
                                     _vp]
        L.loza_rope_frequencies.restype = ctypes.c_int
        L.loza_rope_frequencies.argtypes = [_f64, _i32, _i32, _f64, _f64, _f64, _f64, _vp, _vp]
        L.loza_rope.restype = ctypes.c_int
        L.loza_rope.argtypes = [_vp, _vp, _vp, _i64, _i32, _i32, _i64, RopeParams, _i32, _i32, _vp, _i64, _vp]
        L.loza_qk_norm_rope.restype = ctypes.c_int
        L.loza_qk_norm_rope.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i32, _i64, _i64, _i64, _vp,
                                        _vp, _i32, _f32, RopeParams, _i32, _vp, _i64, _vp, _i64, _pool, _vp, _vp]
        L.loza_qk_norm_rope_workspace_size.restype = _sz
        L.loza_qk_norm_rope_workspace_size.argtypes = [_i32]
        L.loza_qk_norm_rope_backward.restype = ctypes.c_int
        L.loza_qk_norm_rope_backward.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i32, _i32, _i32, _i64, _i64,
                                                 _i64, _i64, _vp, _vp, _i32, _f32, RopeParams, _i32, _vp, _i64, _vp,
                                                 _i64, _vp, _vp, _vp, _sz, _vp]
        L.loza_decode_paged_kv_workspace_size.restype = _sz
        L.loza_decode_paged_kv_workspace_size.argtypes = [_i32, _i32, _i32, _i32]
        L.loza_ssa_decode_paged_kv.restype = ctypes.c_int
        L.loza_ssa_decode_paged_kv.argtypes = [_vp, _i64, _pool, _vp, _i64, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                               Params, _i32, _vp, _vp, _vp, _sz, _vp]
        _lib = L
    return _lib


def _check(rc: int, what: str):
    if rc != 0:
        raise LozaError(rc, what)


def _stream_ptr(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _require(t, name, dtype=None, ndim=None):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")


def _row_tensor(t, name):
    """[rows, heads, dim] with heads/dim contiguous; returns its row stride."""
    if t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
        raise ValueError(f"{name}: heads and head dim must be contiguous within a row")
    return t.stride(0)


def workspace_size(op, batch, total_tokens, max_seqlen, n_heads, n_kv_heads, d_qk, d_v, params: Params) -> int:
    return int(lib().loza_ssa_workspace_size(op, batch, total_tokens, max_seqlen, n_heads, n_kv_heads,
                                             d_qk, d_v, params))


def loza_ssa_prefill(q, k, v, cu_seqlens, max_seqlen: int, params: Params, out=None, lse=None,
                     workspace=None, stream=None):
    """SSA forward over a packed batch. Returns (out [T,H,d_v] bf16, lse [T,H] fp32)."""
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _require(t, n, torch.bfloat16, 3)
    _require(cu_seqlens, "cu_seqlens", torch.int32, 1)
    T, H, d_qk = q.shape
    Hkv, d_v = k.shape[1], v.shape[2]
    if out is None:
        out = torch.empty((T, H, d_v), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    if workspace is None:
        n = workspace_size(LOZA_OP_PREFILL, cu_seqlens.numel() - 1, T, int(max_seqlen), H, Hkv, d_qk, d_v, params)
        if n:
            workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = lib().loza_ssa_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), cu_seqlens.numel() - 1, T,
                                int(max_seqlen), H, Hkv, d_qk, d_v, _row_tensor(q, "q"), _row_tensor(k, "k"),
                                _row_tensor(v, "v"), params, _ptr(out), _ptr(lse), _ptr(workspace), ws_bytes,
                                _stream_ptr(stream))
    _check(rc, "loza_ssa_prefill")
    return out, lse


def loza_ssa_prefill_host(q, k, v, params: Params, cu_seqlens=None, max_seqlen=None, out=None, lse=None,
                          workspace=None, stream=None):
    """Prefill of a packed batch from and to host memory (copies inside the call,
    overlapped with the kernels). q [T, H, d_qk], k [T, Hkv, d_qk], v [T, Hkv, d_v]:
    contiguous bf16 CPU tensors (pinned for overlap); absorbed MLA: pass the
    latent [T, 1, 576] as k and v (the same tensor, or its first 512 columns).
    cu_seqlens: host sequence offsets [0, ..., T] (a list, numpy array or CPU
    tensor; None = one sequence of T tokens). Returns (out [T, H, d_v] bf16,
    lse [T, H] fp32) as CPU tensors; they hold the results once `stream`
    (default: the current CUDA stream) has passed the call. The workspace is a
    CUDA uint8 tensor (allocated if None)."""
    import numpy as np
    import torch
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or t.dim() != 3:
            raise TypeError(f"{n} must be a 3-D bf16 tensor")
    T, H, d_qk = q.shape
    Hkv, d_v = k.shape[1], v.shape[2]
    latent = v.data_ptr() == k.data_ptr()
    for t, n in ((q, "q"), (k, "k")) + (() if latent else ((v, "v"),)):
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    if latent and v.stride(0) != k.stride(0):
        raise ValueError("a latent v must be a column slice of k")
    if cu_seqlens is None:
        cu_seqlens = [0, T]
    if isinstance(cu_seqlens, torch.Tensor):
        cu_seqlens = cu_seqlens.cpu().numpy()
    cu = np.ascontiguousarray(cu_seqlens, dtype=np.int32)
    if cu.ndim != 1 or cu.size < 2:
        raise ValueError("cu_seqlens needs at least two offsets")
    batch = cu.size - 1
    if max_seqlen is None:
        max_seqlen = max(1, int(np.max(np.diff(cu))))
    pin = q.device.type == "cpu" and q.is_pinned()
    if out is None:
        out = torch.empty((T, H, d_v), dtype=torch.bfloat16, device=q.device, pin_memory=pin)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device, pin_memory=pin)
    if not out.is_contiguous() or not lse.is_contiguous():
        raise ValueError("out and lse must be contiguous")
    if workspace is None:
        n = workspace_size(LOZA_OP_PREFILL_HOST, batch, T, int(max_seqlen), H, Hkv, d_qk, d_v, params)
        if n == 0:
            raise LozaError(-2, "loza_ssa_prefill_host")
        workspace = torch.empty(n, dtype=torch.uint8, device="cuda")
    _require(workspace, "workspace", torch.uint8)
    rc = lib().loza_ssa_prefill_host(_ptr(q), _ptr(k), _ptr(k if latent else v),
                                     cu.ctypes.data_as(ctypes.c_void_p), batch, T, int(max_seqlen), H, Hkv, d_qk,
                                     d_v, params, _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
                                     _stream_ptr(stream))
    _check(rc, "loza_ssa_prefill_host")
    return out, lse


def loza_ssa_decode(q, k_cache, v_cache, seqlens, max_seqlen: int, params: Params, out=None, lse=None,
                    workspace=None, stream=None):
    """SSA decode. q [B,H,d_qk]; k_cache [B,Lcap,Hkv,d_qk] (row/batch strides taken from the
    tensor); v_cache None for the absorbed latent cache. Returns (out [B,H,d_v], lse [B,H])."""
    import torch
    _require(q, "q", torch.bfloat16, 3)
    _require(k_cache, "k_cache", torch.bfloat16, 4)
    _require(seqlens, "seqlens", torch.int32, 1)
    B, H, d_qk = q.shape
    Hkv = k_cache.shape[2]
    d_v = v_cache.shape[3] if v_cache is not None else 512
    if k_cache.stride(3) != 1 or (Hkv > 1 and k_cache.stride(2) != d_qk):
        raise ValueError("k_cache: heads and head dim must be contiguous within a row")
    if out is None:
        out = torch.empty((B, H, d_v), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    if workspace is None:
        n = workspace_size(LOZA_OP_DECODE, B, 0, int(max_seqlen), H, Hkv, d_qk, d_v, params)
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = lib().loza_ssa_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seqlens), B, int(max_seqlen),
                               k_cache.stride(0), k_cache.stride(1), H, Hkv, d_qk, d_v, params, _ptr(out),
                               _ptr(lse), _ptr(workspace), ws_bytes, _stream_ptr(stream))
    _check(rc, "loza_ssa_decode")
    return out, lse


def loza_ssa_decode_noalloc(q, k_cache, v_cache, seqlens, max_seqlen: int, params: Params, out, lse,
                            stream=None):
    """Decode for callers that cannot allocate device memory: like loza_ssa_decode,
    but the split-KV partials live in a fixed 16 MiB array inside the library, so
    nothing is allocated here either (out and lse must be given). Calls that can
    overlap on the GPU share that array and must not run concurrently."""
    import torch
    _require(q, "q", torch.bfloat16, 3)
    _require(k_cache, "k_cache", torch.bfloat16, 4)
    _require(seqlens, "seqlens", torch.int32, 1)
    _require(out, "out", torch.bfloat16, 3)
    _require(lse, "lse", torch.float32, 2)
    B, H, d_qk = q.shape
    Hkv = k_cache.shape[2]
    d_v = v_cache.shape[3] if v_cache is not None else 512
    rc = lib().loza_ssa_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seqlens), B, int(max_seqlen),
                                       k_cache.stride(0), k_cache.stride(1), H, Hkv, d_qk, d_v, params, _ptr(out),
                                       _ptr(lse), _stream_ptr(stream))
    _check(rc, "loza_ssa_decode_noalloc")
    return out, lse


def loza_ssa_backward(q, k, v, out, dout, lse, cu_seqlens, max_seqlen: int, params: Params, dq=None, dk=None,
                      dv=None, workspace=None, stream=None):
    """SSA backward. All of q, k, v, out, dout contiguous [T, heads, dim]. Returns (dq, dk, dv)."""
    import torch
    T, H, d_qk = q.shape
    Hkv, d_v = k.shape[1], v.shape[2]
    B = cu_seqlens.numel() - 1
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        n = workspace_size(LOZA_OP_BACKWARD, B, T, int(max_seqlen), H, Hkv, d_qk, d_v, params)
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = lib().loza_ssa_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse), _ptr(cu_seqlens),
                                 B, T, int(max_seqlen), H, Hkv, d_qk, d_v, params, _ptr(dq), _ptr(dk), _ptr(dv),
                                 _ptr(workspace), ws_bytes, _stream_ptr(stream))
    _check(rc, "loza_ssa_backward")
    return dq, dk, dv


def device_status(stream=None) -> int:
    """Synchronise and return the kernels' device status (0, or -5 after a timed-out wait)."""
    return int(lib().loza_device_status(_stream_ptr(stream)))


def launch_count() -> int:
    return int(lib().loza_launch_count())


def loza_ssa_merge(o_a, lse_a, o_b, lse_b, out=None, lse_out=None, stream=None):
    """Attention over the union of two disjoint key sets from two branches:
    o_* [..., d_v] bf16 contiguous, lse_* of shape o_*.shape[:-1] fp32 (natural
    log, -inf for a branch without keys). Returns (out, lse_out)."""
    import torch
    _require(o_a, "o_a", torch.bfloat16)
    _require(o_b, "o_b", torch.bfloat16)
    _require(lse_a, "lse_a", torch.float32)
    _require(lse_b, "lse_b", torch.float32)
    if o_a.shape != o_b.shape or lse_a.shape != o_a.shape[:-1] or lse_b.shape != o_a.shape[:-1]:
        raise ValueError("merge: branch shapes differ")
    for t, n in ((o_a, "o_a"), (o_b, "o_b"), (lse_a, "lse_a"), (lse_b, "lse_b")):
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")
    d_v = o_a.shape[-1]
    rows = o_a.numel() // d_v
    if out is None:
        out = torch.empty_like(o_a)
    if lse_out is None:
        lse_out = torch.empty_like(lse_a)
    rc = lib().loza_ssa_merge(_ptr(o_a), _ptr(lse_a), _ptr(o_b), _ptr(lse_b), rows, d_v, _ptr(out), _ptr(lse_out),
                              _stream_ptr(stream))
    _check(rc, "loza_ssa_merge")
    return out, lse_out


def loza_ssa_mix(o_full, o_ssa, alpha: float, out=None, stream=None):
    """alpha * o_full + (1 - alpha) * o_ssa (bf16, contiguous, same shape)."""
    import torch
    _require(o_full, "o_full", torch.bfloat16)
    _require(o_ssa, "o_ssa", torch.bfloat16)
    if o_full.shape != o_ssa.shape or not o_full.is_contiguous() or not o_ssa.is_contiguous():
        raise ValueError("mix: inputs must be contiguous and of one shape")
    if out is None:
        out = torch.empty_like(o_full)
    rc = lib().loza_ssa_mix(_ptr(o_full), _ptr(o_ssa), o_full.numel(), float(alpha), _ptr(out), _stream_ptr(stream))
    _check(rc, "loza_ssa_mix")
    return out


def loza_ssa_decode_paged(q, kv_pool, block_table, seqlens, max_seqlen: int, params: Params, out=None, lse=None,
                          workspace=None, stream=None):
    """Absorbed SSA decode from a paged latent cache. q [B,64,576]; kv_pool
    [num_pages, 128, 576] (or [num_pages * 128, 576]) bf16 with contiguous rows;
    block_table [B, pages per sequence] int32: the pool page of each logical
    128-token block. Returns (out [B,64,512], lse [B,64])."""
    import torch
    _require(q, "q", torch.bfloat16, 3)
    _require(kv_pool, "kv_pool", torch.bfloat16)
    _require(block_table, "block_table", torch.int32, 2)
    _require(seqlens, "seqlens", torch.int32, 1)
    if kv_pool.shape[-1] != 576 or kv_pool.stride(-1) != 1:
        raise ValueError("kv_pool rows must be 576 contiguous latent columns")
    pool2 = kv_pool.reshape(-1, 576) if kv_pool.dim() == 3 else kv_pool
    if pool2.dim() != 2 or pool2.shape[0] % 128 != 0:
        raise ValueError("kv_pool must hold whole pages of 128 rows")
    if not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous")
    B, H, d_qk = q.shape
    if out is None:
        out = torch.empty((B, H, 512), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    if workspace is None:
        n = workspace_size(LOZA_OP_DECODE, B, 0, int(max_seqlen), H, 1, d_qk, 512, params)
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = lib().loza_ssa_decode_paged(_ptr(q), _ptr(pool2), pool2.shape[0] // 128, pool2.stride(0), _ptr(block_table),
                                     block_table.shape[1], _ptr(seqlens), B, int(max_seqlen), H, params, _ptr(out),
                                     _ptr(lse), _ptr(workspace), ws_bytes, _stream_ptr(stream))
    _check(rc, "loza_ssa_decode_paged")
    return out, lse


# ---------------------------------------------------------------------------
# Hierarchical index decode (page 4's streaming-aware and hierarchical index)
# ---------------------------------------------------------------------------
def _contiguous(t, name):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _latent_cache(kv_cache):
    import torch
    _require(kv_cache, "kv_cache", torch.bfloat16, 4)
    if kv_cache.shape[2] != 1 or kv_cache.shape[3] < 576 or kv_cache.stride(3) != 1:
        raise ValueError("kv_cache must be [batch, rows, 1, 576] with contiguous latent rows")


def _index_keys(k_index):
    import torch
    _require(k_index, "k_index", torch.bfloat16, 3)
    if k_index.stride(2) != 1:
        raise ValueError("k_index: the index dimension must be contiguous")
    return k_index.shape[2], k_index.stride(0), k_index.stride(1)


def loza_hi_page_keys(k_index, seqlens, max_seqlen: int, page_keys=None, stream=None):
    """Mean index key of every whole 128-token page: k_index [B, Lcap, d] bf16 ->
    page_keys [B, d, max_seqlen // 128] float32 (pages innermost)."""
    import torch
    d, bs, rs = _index_keys(k_index)
    _require(seqlens, "seqlens", torch.int32, 1)
    B = k_index.shape[0]
    if page_keys is None:
        page_keys = torch.zeros((B, d, int(max_seqlen) // 128), dtype=torch.float32, device=k_index.device)
    _contiguous(page_keys, "page_keys")
    rc = lib().loza_hi_page_keys(_ptr(k_index), bs, rs, _ptr(seqlens), B, int(max_seqlen), d, _ptr(page_keys),
                                 _stream_ptr(stream))
    _check(rc, "loza_hi_page_keys")
    return page_keys


def hi_workspace_size(batch, max_seqlen, top_pages, top_k, params: Params) -> int:
    return int(lib().loza_hi_workspace_size(batch, max_seqlen, top_pages, top_k, params))


def loza_hi_select(q_index, k_index, page_keys, seqlens, max_seqlen: int, params: Params, top_pages: int, top_k: int,
                   selected=None, workspace=None, stream=None):
    """Tokens the hierarchical index selects: int32 [B, top_k], ascending, -1 padded."""
    import torch
    d, bs, rs = _index_keys(k_index)
    _require(q_index, "q_index", torch.bfloat16, 2)
    _require(page_keys, "page_keys", torch.float32, 3)
    _contiguous(q_index, "q_index")
    _contiguous(page_keys, "page_keys")
    B = k_index.shape[0]
    if selected is None:
        selected = torch.empty((B, top_k), dtype=torch.int32, device=k_index.device)
    if workspace is None:
        workspace = torch.empty(max(16, hi_workspace_size(B, int(max_seqlen), top_pages, top_k, params)),
                                dtype=torch.uint8, device=k_index.device)
    rc = lib().loza_hi_select(_ptr(q_index), _ptr(k_index), bs, rs, _ptr(page_keys), _ptr(seqlens), B,
                              int(max_seqlen), d, params, top_pages, top_k, _ptr(selected), _ptr(workspace),
                              workspace.numel(), _stream_ptr(stream))
    _check(rc, "loza_hi_select")
    return selected


def loza_ssa_decode_selected(q, kv_cache, seqlens, max_seqlen: int, params: Params, selected, out=None, lse=None,
                             workspace=None, stream=None):
    """Attention of each decode query over its window `params` and the tokens of
    `selected` (int32 [B, top_k]; entries that are negative, past the query or
    inside the window are ignored). Absorbed latent cache [B, Lcap, 1, 576];
    returns (out [B, 64, 512], lse [B, 64])."""
    import torch
    _require(q, "q", torch.bfloat16, 3)
    _latent_cache(kv_cache)
    _require(selected, "selected", torch.int32, 2)
    _require(seqlens, "seqlens", torch.int32, 1)
    _contiguous(q, "q")
    _contiguous(selected, "selected")
    B, H, _ = q.shape
    top_k = selected.shape[1]
    if out is None:
        out = torch.empty((B, H, 512), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(max(16, hi_workspace_size(B, int(max_seqlen), 1, top_k, params)),
                                dtype=torch.uint8, device=q.device)
    rc = lib().loza_ssa_decode_selected(_ptr(q), _ptr(kv_cache), kv_cache.stride(0), kv_cache.stride(1),
                                        _ptr(seqlens), B, int(max_seqlen), params, _ptr(selected), top_k, _ptr(out),
                                        _ptr(lse), _ptr(workspace), workspace.numel(), _stream_ptr(stream))
    _check(rc, "loza_ssa_decode_selected")
    return out, lse


def loza_hi_decode(q, kv_cache, q_index, k_index, page_keys, seqlens, max_seqlen: int, params: Params,
                   top_pages: int, top_k: int, out=None, lse=None, workspace=None, stream=None):
    """Decode over the window `params` and the tokens the hierarchical index
    selects, merged; returns (out [B, 64, 512], lse [B, 64])."""
    import torch
    _require(q, "q", torch.bfloat16, 3)
    _latent_cache(kv_cache)
    d, bs, rs = _index_keys(k_index)
    _require(q_index, "q_index", torch.bfloat16, 2)
    _require(page_keys, "page_keys", torch.float32, 3)
    for t, name in ((q, "q"), (q_index, "q_index"), (page_keys, "page_keys")):
        _contiguous(t, name)
    B, H, _ = q.shape
    if out is None:
        out = torch.empty((B, H, 512), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = torch.empty(max(16, hi_workspace_size(B, int(max_seqlen), top_pages, top_k, params)),
                                dtype=torch.uint8, device=q.device)
    rc = lib().loza_hi_decode(_ptr(q), _ptr(kv_cache), kv_cache.stride(0), kv_cache.stride(1), _ptr(q_index),
                              _ptr(k_index), bs, rs, _ptr(page_keys), _ptr(seqlens), B, int(max_seqlen), d, params,
                              top_pages, top_k, _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
                              _stream_ptr(stream))
    _check(rc, "loza_hi_decode")
    return out, lse


# ---------------------------------------------------------------------------
# Serving and training around the attention: page plan, rotation, norms of
# query and key heads, decode over paged K and V pools
# ---------------------------------------------------------------------------
LOZA_BF16, LOZA_FP16, LOZA_FP32 = 0, 1, 2
LOZA_ROPE_NONE, LOZA_ROPE_LINEAR, LOZA_ROPE_NTK, LOZA_ROPE_YARN = 0, 1, 2, 3
_ROPE_SCALING = {None: LOZA_ROPE_NONE, "none": LOZA_ROPE_NONE, "linear": LOZA_ROPE_LINEAR, "ntk": LOZA_ROPE_NTK,
                 "yarn": LOZA_ROPE_YARN}
_dtype_codes = {}


def _dtype_code(t, name):
    if not _dtype_codes:
        import torch
        _dtype_codes.update({torch.bfloat16: LOZA_BF16, torch.float16: LOZA_FP16, torch.float32: LOZA_FP32})
    code = _dtype_codes.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32")
    return code


def _on_its_device(fn):
    """Run `fn` with the device of its first tensor current and, if `stream` is
    given, that stream current too: buffers made inside belong to the stream
    that uses them."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        import torch
        first = next((a for a in args if isinstance(a, torch.Tensor)), None)
        if first is None or not first.is_cuda:
            raise TypeError(f"{fn.__name__}: the first tensor must be a CUDA tensor, given by position")
        if stream is None and first.device.index == torch.cuda.current_device():
            return fn(*args, **kw)
        if stream is not None and stream.device != first.device:
            raise ValueError(f"{fn.__name__}: stream and tensors are on different devices")
        with torch.cuda.device(first.device), torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _tensor(t, name, device, dtype, ndim):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")
    return t


def _plain(t, name, device, dtype, shape):
    """A contiguous tensor of exactly this dtype and shape."""
    _tensor(t, name, device, dtype, len(shape))
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _head_rows(t, name):
    """[rows, heads, dim] with heads and dim contiguous; its row stride (of one row: any that fits)."""
    if (t.shape[2] > 1 and t.stride(2) != 1) or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
        raise ValueError(f"{name}: heads and head dim must be contiguous within a row")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * t.shape[2]


def _current_stream():
    import torch
    return torch.cuda.current_stream().cuda_stream


def _data(t):
    return t.data_ptr() if t is not None else None


def _kv_pool(k_pool, v_pool, device, dtype, n_kv, d, d_v):
    """loza_kv_pool of [pages, rows, heads, dim] tensors (any strides, columns contiguous)."""
    _tensor(k_pool, "k_pool", device, dtype, 4)
    pages, rows = k_pool.shape[0], k_pool.shape[1]
    if k_pool.shape[2] != n_kv or k_pool.shape[3] != d or (d > 1 and k_pool.stride(3) != 1):
        raise ValueError(f"k_pool must be [pages, rows, {n_kv}, {d}] with contiguous columns")
    pool = KvPool(k=k_pool.data_ptr(), num_pages=pages, page_size=rows, k_page_stride=k_pool.stride(0),
                  k_row_stride=k_pool.stride(1), k_head_stride=k_pool.stride(2) if n_kv > 1 else 0)
    if v_pool is not None:
        _tensor(v_pool, "v_pool", device, dtype, 4)
        if v_pool.shape != (pages, rows, n_kv, d_v) or (d_v > 1 and v_pool.stride(3) != 1):
            raise ValueError(f"v_pool must be [{pages}, {rows}, {n_kv}, {d_v}] with contiguous columns")
        pool.v = v_pool.data_ptr()
        pool.v_page_stride, pool.v_row_stride = v_pool.stride(0), v_pool.stride(1)
        pool.v_head_stride = v_pool.stride(2) if n_kv > 1 else 0
    return pool


@_on_its_device
def loza_page_plan(ctx_lens, new_lens, free_pages, block_table, page_size: int, capacity: int):
    """Block table, slots and offsets of a step of a paged cache. ctx_lens,
    new_lens [B] int32: tokens cached and tokens appended; free_pages [F] int32:
    pages to hand out, in order; block_table [B, columns] int32 (rows may be
    strided), updated in place; capacity: packed rows of the step. Returns
    (cu_seqlens [B+1] int32, seqlens [B] int32, positions [capacity] int32,
    slots [capacity] int64, counts [3] int32: tokens, pages taken, requests
    short of pages). Nothing is read back to the host."""
    import torch
    dev, i32 = ctx_lens.device, torch.int32
    _tensor(ctx_lens, "ctx_lens", dev, i32, 1)
    B = ctx_lens.shape[0]
    _plain(ctx_lens, "ctx_lens", dev, i32, (B,))
    _plain(new_lens, "new_lens", dev, i32, (B,))
    _tensor(free_pages, "free_pages", dev, i32, 1)
    if free_pages.shape[0] > 1 and free_pages.stride(0) != 1:
        raise ValueError("free_pages must be contiguous")
    _tensor(block_table, "block_table", dev, i32, 2)
    cols = block_table.shape[1]
    if block_table.shape[0] != B or (cols > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be [batch, columns] with contiguous rows")
    if B < 1 or capacity < 0:
        raise LozaError(-1, "loza_page_plan")
    small = torch.empty(2 * B + 4, dtype=i32, device=dev)  # cu_seqlens, seqlens and counts: one buffer
    cu, lens, counts = small[:B + 1], small[B + 1:2 * B + 1], small[2 * B + 1:]
    positions = torch.empty(capacity, dtype=i32, device=dev)
    slots = torch.empty(capacity, dtype=torch.int64, device=dev)
    rc = lib().loza_page_plan(ctx_lens.data_ptr(), new_lens.data_ptr(), B, free_pages.data_ptr(),
                              free_pages.shape[0], page_size, block_table.data_ptr(),
                              block_table.stride(0) if B > 1 else cols, cols, capacity, cu.data_ptr(),
                              lens.data_ptr(), positions.data_ptr(), slots.data_ptr(), counts.data_ptr(),
                              _current_stream())
    _check(rc, "loza_page_plan")
    return cu, lens, positions, slots, counts


def rope_frequencies(rope_dim: int, theta: float = 10000.0, scaling=None, factor: float = 1.0,
                     original_max: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """Angles per position (float64 [rope_dim / 2], on `device`) and the scale of
    RopeParams; scaling: None, "linear", "ntk" or "yarn" (for contexts `factor`
    times longer than original_max)."""
    import torch
    if scaling not in _ROPE_SCALING:
        raise ValueError(f"scaling must be one of {[k for k in _ROPE_SCALING if k]} or None")
    freq = torch.empty(max(0, int(rope_dim)) // 2, dtype=torch.float64)
    scale = ctypes.c_float()
    _check(lib().loza_rope_frequencies(float(theta), int(rope_dim), _ROPE_SCALING[scaling], float(factor),
                                       float(original_max), float(beta_fast), float(beta_slow), freq.data_ptr(),
                                       ctypes.addressof(scale)), "loza_rope_frequencies")
    return (freq.to(device) if device is not None else freq), scale.value


def _rope_tables(positions, inv_freq, rope, dev, tokens):
    import torch
    _plain(positions, "positions", dev, torch.int32, (tokens,))
    _plain(inv_freq, "inv_freq", dev, torch.float64, (rope.rope_dim // 2,))


@_on_its_device
def loza_rope(x, positions, inv_freq, rope: RopeParams, out=None, transposed: bool = False):
    """Position rotation of x [T, H, d] (bf16, fp16 or fp32; rows may be strided)
    by positions [T] int32 and inv_freq [rope_dim / 2] float64. out may be x (in
    place). transposed: the gradient (dx from dout). Returns out."""
    import torch
    dev, code = x.device, _dtype_code(x, "x")
    _tensor(x, "x", dev, x.dtype, 3)
    T, H, d = x.shape
    _rope_tables(positions, inv_freq, rope, dev, T)
    if out is None:
        out = torch.empty((T, H, d), dtype=x.dtype, device=dev)
    else:
        _tensor(out, "out", dev, x.dtype, 3)
        if out.shape != x.shape:
            raise ValueError("out must have the shape of x")
    _check(lib().loza_rope(x.data_ptr(), positions.data_ptr(), inv_freq.data_ptr(), T, H, d, _head_rows(x, "x"), rope,
                           int(bool(transposed)), code, out.data_ptr(), _head_rows(out, "out"), _current_stream()),
           "loza_rope")
    return out


def _sides(q, k, q_weight, k_weight, norm_dim):
    """Shapes common to the norm-and-rotation calls: (device, dtype, code, T, H, Hk, d, norm_dim)."""
    first = q if q is not None else k
    dev, dtype, code = first.device, first.dtype, _dtype_code(first, "q or k")
    _tensor(first, "q or k", dev, dtype, 3)
    T, _, d = first.shape
    for t, name in ((q, "q"), (k, "k")):
        if t is not None:
            _tensor(t, name, dev, dtype, 3)
            if t.shape[0] != T or t.shape[2] != d:
                raise ValueError("q and k must agree in tokens and head dim")
    for w in (q_weight, k_weight):
        if w is not None and norm_dim is None:
            norm_dim = w.shape[0] if w.dim() == 1 else -1
    norm_dim = 0 if norm_dim is None else int(norm_dim)
    for w, t, name in ((q_weight, q, "q_weight"), (k_weight, k, "k_weight")):
        if w is not None:
            if t is None:
                raise ValueError(f"{name} without its rows")
            _plain(w, name, dev, dtype, (norm_dim,))
    return dev, dtype, code, T, 0 if q is None else q.shape[1], 0 if k is None else k.shape[1], d, norm_dim


def _like_rows(t, ref, name):
    """`t`, or new rows like `ref`: shape and dtype checked."""
    import torch
    if t is None:
        return torch.empty(ref.shape, dtype=ref.dtype, device=ref.device)
    _tensor(t, name, ref.device, ref.dtype, 3)
    if t.shape != ref.shape:
        raise ValueError(f"{name} must have the shape of its input")
    return t


@_on_its_device
def loza_qk_norm_rope(q, k, positions, inv_freq, rope: RopeParams, q_weight=None, k_weight=None, eps: float = 1e-6,
                      v=None, k_pool=None, v_pool=None, slots=None, q_out=None, k_out=None, norm_dim=None):
    """RMS norm of each head of q [T, H, d] and k [T, Hkv, d] over its first
    norm_dim columns (default: the weights' length; a side without weight is not
    normed), then the rotation, and - with k_pool [pages, rows, Hkv, d] and slots
    [T] int64 - the keys (and v [T, Hkv, d_v] into v_pool) written to the paged
    cache. q or k may be None. Returns (q_out, k_out); k_out is None when there
    is a pool and none was given."""
    import torch
    dev, dtype, code, T, H, Hk, d, norm_dim = _sides(q, k, q_weight, k_weight, norm_dim)
    _rope_tables(positions, inv_freq, rope, dev, T)
    if q is not None:
        q_out = _like_rows(q_out, q, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q")
    pool, d_v = None, 0
    if k_pool is not None:
        if k is None:
            raise ValueError("k_pool without k")
        if (v is None) != (v_pool is None):
            raise ValueError("v and v_pool come together")
        if v is not None:
            _tensor(v, "v", dev, dtype, 3)
            d_v = v.shape[2]
            if v.shape[:2] != k.shape[:2]:
                raise ValueError("v and k must agree in tokens and heads")
        _plain(slots, "slots", dev, torch.int64, (T,))
        pool = _kv_pool(k_pool, v_pool, dev, dtype, Hk, d, d_v)
    elif v is not None or v_pool is not None or slots is not None:
        raise ValueError("v, v_pool and slots need k_pool")
    if k is not None and (k_pool is None or k_out is not None):
        k_out = _like_rows(k_out, k, "k_out")
    elif k is None and k_out is not None:
        raise ValueError("k_out without k")
    row = lambda t, name: 0 if t is None else _head_rows(t, name)
    rc = lib().loza_qk_norm_rope(
        _data(q), _data(k), _data(v), positions.data_ptr(), inv_freq.data_ptr(), T, H, Hk, d, d_v, row(q, "q"),
        row(k, "k"), row(v, "v"), _data(q_weight), _data(k_weight), norm_dim, eps, rope, code, _data(q_out),
        row(q_out, "q_out"), _data(k_out), row(k_out, "k_out"), ctypes.byref(pool) if pool is not None else None,
        _data(slots), _current_stream())
    _check(rc, "loza_qk_norm_rope")
    return q_out, k_out


@_on_its_device
def loza_qk_norm_rope_backward(dq_out, dk_out, q, k, positions, inv_freq, rope: RopeParams, q_weight=None,
                               k_weight=None, eps: float = 1e-6, dq=None, dk=None, norm_dim=None, workspace=None):
    """Gradient of loza_qk_norm_rope: (dq, dk, dq_weight, dk_weight) from dq_out
    and dk_out and the forward's inputs; the weights' gradients are fp32
    [norm_dim], None for a side without weight. A side is given (dq_out, or
    dk_out) or None; q and k are only read where there is a weight."""
    import torch
    dev, dtype, code, T, H, Hk, d, norm_dim = _sides(dq_out, dk_out, q_weight, k_weight, norm_dim)
    _rope_tables(positions, inv_freq, rope, dev, T)
    grads = []
    for dy, x, w, g, s in ((dq_out, q, q_weight, dq, "q"), (dk_out, k, k_weight, dk, "k")):
        if dy is None and g is not None:
            raise ValueError(f"d{s} without d{s}_out")
        if w is not None:
            if x is None:
                raise ValueError(f"{s} is needed where there is {s}_weight")
            _tensor(x, s, dev, dtype, 3)
            if x.shape != dy.shape:
                raise ValueError(f"{s} and d{s}_out must have one shape")
        grads.append(_like_rows(g, dy, f"d{s}") if dy is not None else None)
    dq, dk = grads
    sums = [torch.empty(norm_dim, dtype=torch.float32, device=dev) if w is not None else None
            for w in (q_weight, k_weight)]
    if workspace is None and (q_weight is not None or k_weight is not None):
        workspace = torch.empty(lib().loza_qk_norm_rope_workspace_size(norm_dim), dtype=torch.uint8, device=dev)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    row = lambda t, name: 0 if t is None else _head_rows(t, name)
    qx, kx = q if q_weight is not None else None, k if k_weight is not None else None
    rc = lib().loza_qk_norm_rope_backward(
        _data(dq_out), _data(dk_out), _data(qx), _data(kx), positions.data_ptr(), inv_freq.data_ptr(), T, H, Hk, d,
        row(dq_out, "dq_out"), row(dk_out, "dk_out"), row(qx, "q"), row(kx, "k"), _data(q_weight), _data(k_weight),
        norm_dim, eps, rope, code, _data(dq), row(dq, "dq"), _data(dk), row(dk, "dk"), _data(sums[0]),
        _data(sums[1]), _data(workspace), ws_bytes, _current_stream())
    _check(rc, "loza_qk_norm_rope_backward")
    return dq, dk, sums[0], sums[1]


@_on_its_device
def loza_ssa_decode_paged_kv(q, k_pool, v_pool, block_table, seqlens, max_seqlen: int, params: Params, out=None,
                             lse=None, workspace=None):
    """Decode over paged K and V pools, heads of their own or shared by groups.
    q [B, H, d_qk] bf16 or fp16 (rows may be strided); k_pool [pages, rows, Hkv,
    d_qk] and v_pool [pages, rows, Hkv, d_v] (any strides that are multiples of
    16 bytes, columns contiguous); block_table [B, columns] int32; seqlens [B]
    int32, 0 for an idle row (out 0, lse -inf). Returns (out [B, H, d_v],
    lse [B, H])."""
    import torch
    dev, code = q.device, _dtype_code(q, "q")
    _tensor(q, "q", dev, q.dtype, 3)
    B, H, d = q.shape
    _plain(seqlens, "seqlens", dev, torch.int32, (B,))
    _tensor(block_table, "block_table", dev, torch.int32, 2)
    cols = block_table.shape[1]
    if block_table.shape[0] != B or (cols > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be [batch, columns] with contiguous rows")
    bt_stride = block_table.stride(0) if B > 1 else cols
    page = max(1, k_pool.shape[1]) if isinstance(k_pool, torch.Tensor) and k_pool.dim() == 4 else 1
    if cols * page < max_seqlen:
        raise ValueError("block_table has too few columns for max_seqlen")
    if v_pool is None:
        raise TypeError("v_pool must be a tensor")
    Hk, d_v = (k_pool.shape[2], v_pool.shape[3]) if k_pool.dim() == 4 and v_pool.dim() == 4 else (0, 0)
    pool = _kv_pool(k_pool, v_pool, dev, q.dtype, Hk, d, d_v)
    out = torch.empty((B, H, d_v), dtype=q.dtype, device=dev) if out is None else \
        _plain(out, "out", dev, q.dtype, (B, H, d_v))
    lse = torch.empty((B, H), dtype=torch.float32, device=dev) if lse is None else \
        _plain(lse, "lse", dev, torch.float32, (B, H))
    if workspace is None:
        workspace = torch.empty(max(16, lib().loza_decode_paged_kv_workspace_size(H, Hk, d, d_v)), dtype=torch.uint8,
                                device=dev)
    rc = lib().loza_ssa_decode_paged_kv(
        q.data_ptr(), _head_rows(q, "q"), ctypes.byref(pool), block_table.data_ptr(), bt_stride, seqlens.data_ptr(),
        B, max_seqlen, H, Hk, d, d_v, params, code, out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _current_stream())
    _check(rc, "loza_ssa_decode_paged_kv")
    return out, lse


def wait_selftest(limit_us: int, stream=None) -> int:
    """Launch the bounded-wait self-test (a wait that nothing completes gives
    up after limit_us); returns the status of the following device-status
    read, LOZA_ERR_TIMEOUT (-5) when the bound works."""
    _check(lib().loza_wait_selftest(int(limit_us), _stream_ptr(stream)), "loza_wait_selftest")
    return device_status(stream)
