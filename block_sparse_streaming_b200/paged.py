"""Serving and training operators around the attention: page plan, position rotation, norms of query and key
heads with their gradient, decode over paged K and V pools.

The package re-exports these names. Marshalling only, like the rest of the binding; checks, outputs and the call of
the C ABI are in the compiled part (csrc/paged_binding.cpp), because the calls are a few microseconds long. Every
tensor of a call lives on one GPU, which need not be the current one; with `stream` the whole call runs there, its
buffers included. Nothing is read back to the host, and every call can be captured into a graph.

The calls record no autograd graph, whether their inputs require gradients or not: a training step calls the gradient
(loza_qk_norm_rope_backward; loza_rope with transposed) itself. What a call writes in place (out, pools, the block
table) counts as modified, so autograd refuses a backward that had saved it."""
from __future__ import annotations

import ctypes
import os

import torch

from . import LozaError, Params, lib
from ._build import BINDING_PATH

if not os.path.exists(BINDING_PATH):
    raise RuntimeError(f"{BINDING_PATH} is missing: run block_sparse_streaming_b200.build() (a warning says why it "
                       "cannot be built); there is no fallback path")
from . import _paged_binding as _c  # noqa: E402

if _c.torch_version != torch.__version__:
    raise RuntimeError(f"{BINDING_PATH} was built for torch {_c.torch_version}, not {torch.__version__}: remove it and "
                       "run block_sparse_streaming_b200.build()")

LOZA_BF16, LOZA_FP16, LOZA_FP32 = 0, 1, 2
_SCALING = {None: 0, "none": 0, "linear": 1, "ntk": 2, "yarn": 3}  # LOZA_ROPE_*
_page_plan, _rope, _qk_norm_rope, _qk_norm_rope_backward, _decode_paged_kv = (
    _c.page_plan, _c.rope, _c.qk_norm_rope, _c.qk_norm_rope_backward, _c.decode_paged_kv)


class RopeParams(ctypes.Structure):
    """loza_rope_params {rope_dim, rope_offset, interleaved, scale}."""
    _fields_ = [("rope_dim", ctypes.c_int32), ("rope_offset", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("scale", ctypes.c_float)]

    def __init__(self, rope_dim: int, rope_offset: int = 0, interleaved: bool = False, scale: float = 1.0):
        super().__init__(rope_dim, rope_offset, int(bool(interleaved)), scale)


_c.bind({name: ctypes.cast(getattr(lib(), name), ctypes.c_void_p).value for name in (
    "loza_page_plan", "loza_rope", "loza_qk_norm_rope", "loza_qk_norm_rope_backward",
    "loza_qk_norm_rope_workspace_size", "loza_ssa_decode_paged_kv", "loza_decode_paged_kv_workspace_size")},
    LozaError, RopeParams, Params, torch.OutOfMemoryError)


def _on(stream, call, *args):
    """The call with `stream` current: the kernels run there, and buffers made inside belong to it."""
    first = args[0] if args[0] is not None else args[1]
    if isinstance(first, torch.Tensor) and stream.device != first.device:
        raise ValueError("stream and tensors are on different devices")
    with torch.cuda.stream(stream):
        return call(*args)


def loza_page_plan(ctx_lens, new_lens, free_pages, block_table, page_size: int, capacity: int, stream=None):
    """Block table, slots and offsets of a step of a paged cache. ctx_lens, new_lens [B] int32: tokens cached and
    tokens appended; free_pages [F] int32: pages to hand out, in order; block_table [B, columns] int32 (rows may be
    strided), updated in place; capacity: packed rows of the step. Returns (cu_seqlens [B+1] int32, seqlens [B]
    int32, positions [capacity] int32, slots [capacity] int64, counts [3] int32: tokens, pages taken, requests short
    of pages)."""
    if stream is not None:
        return _on(stream, _page_plan, ctx_lens, new_lens, free_pages, block_table, page_size, capacity)
    return _page_plan(ctx_lens, new_lens, free_pages, block_table, page_size, capacity)


def rope_frequencies(rope_dim: int, theta: float = 10000.0, scaling=None, factor: float = 1.0,
                     original_max: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """Angles per position (float64 [rope_dim / 2], on `device`) and the scale of RopeParams; scaling: None, "linear",
    "ntk" or "yarn" (for contexts `factor` times longer than original_max)."""
    if scaling not in _SCALING:
        raise ValueError(f"scaling must be one of {[k for k in _SCALING if k]} or None")
    freq = torch.empty(max(0, int(rope_dim)) // 2, dtype=torch.float64)
    scale = ctypes.c_float()
    rc = lib().loza_rope_frequencies(float(theta), int(rope_dim), _SCALING[scaling], float(factor),
                                     float(original_max), float(beta_fast), float(beta_slow), freq.data_ptr(),
                                     ctypes.addressof(scale))
    if rc:
        raise LozaError(rc, "loza_rope_frequencies")
    return (freq.to(device) if device is not None else freq), scale.value


def loza_rope(x, positions, inv_freq, rope: RopeParams, out=None, transposed: bool = False, stream=None):
    """Position rotation of x [T, H, d] (bf16, fp16 or fp32; rows may be strided) by positions [T] int32 and inv_freq
    [rope_dim / 2] float64. out may be x (in place). transposed: the gradient (dx from dout). Returns out."""
    if stream is not None:
        return _on(stream, _rope, x, positions, inv_freq, rope, out, transposed)
    return _rope(x, positions, inv_freq, rope, out, transposed)


def loza_qk_norm_rope(q, k, positions, inv_freq, rope: RopeParams, q_weight=None, k_weight=None, eps: float = 1e-6,
                      v=None, k_pool=None, v_pool=None, slots=None, q_out=None, k_out=None, norm_dim=None,
                      stream=None):
    """RMS norm of each head of q [T, H, d] and k [T, Hkv, d] over its first norm_dim columns (default: the weights'
    length; a side without weight is not normed), then the rotation, and - with k_pool [pages, rows, Hkv, d] and slots
    [T] int64 - the keys (and v [T, Hkv, d_v] into v_pool) written to the paged cache. q or k may be None. Returns
    (q_out, k_out); k_out is None when there is a pool and none was given."""
    if stream is not None:
        return _on(stream, _qk_norm_rope, q, k, positions, inv_freq, rope, q_weight, k_weight, eps, v, k_pool, v_pool,
                   slots, q_out, k_out, norm_dim)
    return _qk_norm_rope(q, k, positions, inv_freq, rope, q_weight, k_weight, eps, v, k_pool, v_pool, slots, q_out,
                         k_out, norm_dim)


def loza_qk_norm_rope_backward(dq_out, dk_out, q, k, positions, inv_freq, rope: RopeParams, q_weight=None,
                               k_weight=None, eps: float = 1e-6, dq=None, dk=None, norm_dim=None, workspace=None,
                               stream=None):
    """Gradient of loza_qk_norm_rope: (dq, dk, dq_weight, dk_weight) from dq_out and dk_out and the forward's inputs;
    the weights' gradients are fp32 [norm_dim], None for a side without weight. A side is given (dq_out, or dk_out) or
    None; q and k are only read where there is a weight."""
    if stream is not None:
        return _on(stream, _qk_norm_rope_backward, dq_out, dk_out, q, k, positions, inv_freq, rope, q_weight, k_weight,
                   eps, dq, dk, norm_dim, workspace)
    return _qk_norm_rope_backward(dq_out, dk_out, q, k, positions, inv_freq, rope, q_weight, k_weight, eps, dq, dk,
                                  norm_dim, workspace)


def loza_ssa_decode_paged_kv(q, k_pool, v_pool, block_table, seqlens, max_seqlen: int, params: Params, out=None,
                             lse=None, workspace=None, stream=None):
    """Decode over paged K and V pools, heads of their own or shared by groups. q [B, H, d_qk] bf16 or fp16 (rows may
    be strided); k_pool [pages, rows, Hkv, d_qk] and v_pool [pages, rows, Hkv, d_v] (any strides that are multiples of
    16 bytes, columns contiguous); block_table [B, columns] int32; seqlens [B] int32, 0 for an idle row (out 0, lse
    -inf). Returns (out [B, H, d_v], lse [B, H])."""
    if stream is not None:
        return _on(stream, _decode_paged_kv, q, k_pool, v_pool, block_table, seqlens, max_seqlen, params, out, lse,
                   workspace)
    return _decode_paged_kv(q, k_pool, v_pool, block_table, seqlens, max_seqlen, params, out, lse, workspace)
