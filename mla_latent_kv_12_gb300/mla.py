"""Thin binding of libmla (the C ABI declared in ``include/mla.h``): ctypes, and for the paged cache the extension
module ``_native`` (``csrc/binding.cpp``).

Argument marshalling only: every step runs in the library's CUDA kernels.
PyTorch supplies device memory and the current stream.  Importing this module
fails loudly if the built library is missing; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmla.so")

F32, BF16 = 0, 1
DEVICE_BAD_SELECTION_COUNT = 1 << 1
DEVICE_INDEX_OUT_OF_RANGE = 1 << 4
DEVICE_TIMEOUT = 1 << 5
DEVICE_LAYOUT = 1 << 6
DEVICE_SCORE_RANGE = 1 << 7
DEVICE_VALUE_RANGE = 1 << 8
DEVICE_BAD_BLOCK_START = 1 << 9
FP16_SCORE_LIMIT = 256.0

_DT = {torch.float32: F32, torch.bfloat16: BF16}

EXPORTS = (
    "mla_status_string", "mla_last_error_detail", "mla_version", "mla_default_softmax_scale",
    "mla_rope_partial_interleaved", "mla_absorb_q", "mla_decode_attend",
    "mla_decode_workspace_size", "mla_decode_kernel_kind", "mla_project_v",
    "mla_gather_selected", "mla_decode_attend_no_alloc", "mla_decode_step",
    "mla_decode_step_workspace_size", "mla_append_compressed", "mla_select_topk",
    "mla_selftest_bounded_wait", "mla_plan_rollback", "mla_plan_filter", "mla_plan_merge",
    "mla_cache_shift_rows", "mla_rollback_lengths", "mla_reconstruct_kv", "mla_prefill_attend",
    "mla_append_compressed_q8", "mla_quantize_cache", "mla_dequantize_cache", "mla_decode_attend_q8",
    "mla_key_weights", "mla_key_weights_q8", "mla_evict_plan", "mla_cache_compact",
    "mla_append_paged", "mla_tree_plan", "mla_decode_paged_workspace_size", "mla_decode_attend_paged", "mla_commit_paged",
)


class MLAError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"mla status {status}: {detail}")
        self.status = status
        self.detail = detail


class StateArray(ctypes.Structure):
    """``mla_state_array``: one state array of a cache, sizes in bytes."""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride_bytes", ctypes.c_int64),
                ("batch_stride_bytes", ctypes.c_int64), ("row_bytes", ctypes.c_int32)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libmla.so is not built ({LIB_PATH}); run __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    i64, i32, vp, f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float
    sz = ctypes.c_size_t
    i64p = ctypes.POINTER(ctypes.c_int64)
    lib.mla_status_string.restype = ctypes.c_char_p
    lib.mla_status_string.argtypes = [ctypes.c_int]
    lib.mla_last_error_detail.restype = ctypes.c_char_p
    lib.mla_last_error_detail.argtypes = []
    lib.mla_version.restype = ctypes.c_int
    lib.mla_default_softmax_scale.restype = f32
    lib.mla_default_softmax_scale.argtypes = [i32, i32]
    lib.mla_rope_partial_interleaved.restype = ctypes.c_int
    lib.mla_rope_partial_interleaved.argtypes = [vp, vp, ctypes.c_int, i64, i64, i64, i64, i64p, i64p,
                                                 i32, f32, vp, i64, vp]
    lib.mla_absorb_q.restype = ctypes.c_int
    lib.mla_absorb_q.argtypes = [vp, i64, i64, vp, vp, i64, i64, ctypes.c_int, i32, i32, i32, i32, i32, vp]
    lib.mla_decode_attend.restype = ctypes.c_int
    lib.mla_decode_attend.argtypes = [vp, i64, i64, vp, i64, i64, vp, i64, i64, ctypes.c_int, vp, vp,
                                      i32, i32, i32, i32, i32, i64, vp, vp, i32, f32, vp, i64, i64,
                                      ctypes.c_int, vp, vp, sz, vp, vp]
    lib.mla_decode_workspace_size.restype = sz
    lib.mla_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32, i64, i32, ctypes.c_int, ctypes.c_int]
    lib.mla_decode_paged_workspace_size.restype = sz
    lib.mla_decode_paged_workspace_size.argtypes = lib.mla_decode_workspace_size.argtypes
    lib.mla_decode_kernel_kind.restype = ctypes.c_int
    lib.mla_decode_kernel_kind.argtypes = [i32, i32, i32, ctypes.c_int, ctypes.c_int]
    lib.mla_project_v.restype = ctypes.c_int
    lib.mla_project_v.argtypes = [vp, i64, i64, vp, ctypes.c_int, vp, i64, ctypes.c_int, i32, i32, i32,
                                  i32, i32, vp]
    lib.mla_decode_attend_no_alloc.restype = ctypes.c_int
    lib.mla_decode_attend_no_alloc.argtypes = [vp, i64, i64, vp, i64, i64, vp, i64, i64, ctypes.c_int, vp,
                                               vp, i32, i32, i32, i32, i32, i64, vp, vp, i32, f32, vp, i64,
                                               i64, ctypes.c_int, vp, vp, vp]
    lib.mla_decode_step.restype = ctypes.c_int
    lib.mla_decode_step.argtypes = [vp, i64, i64, vp, i64, i64, vp, i64, f32, vp, vp, i64, i64, vp, i64, i64,
                                    ctypes.c_int, vp, vp, i32, i32, i32, i32, i32, i32, i32, i64, vp, vp, i32,
                                    f32, vp, i64, ctypes.c_int, vp, vp, sz, vp, vp]
    lib.mla_decode_step_workspace_size.restype = sz
    lib.mla_decode_step_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32, i64, i32, ctypes.c_int,
                                                   ctypes.c_int]
    lib.mla_append_compressed.restype = ctypes.c_int
    lib.mla_append_compressed.argtypes = [vp, i64, i64, vp, i64, i64, ctypes.c_int, vp, f32, f32, vp, vp, i64,
                                          i64, vp, i64, i64, ctypes.c_int, vp, vp, vp, i32, i32, i32, i32, i64,
                                          vp, vp]
    lib.mla_select_topk.restype = ctypes.c_int
    lib.mla_select_topk.argtypes = [vp, i64, vp, i32, i32, vp, i64, vp, vp, vp]
    lib.mla_selftest_bounded_wait.restype = ctypes.c_int
    lib.mla_selftest_bounded_wait.argtypes = [i64, vp, vp, vp]
    for name, args in (("mla_plan_rollback", [i32, i32, vp, vp, vp, vp, vp, vp, vp, vp]),
                       ("mla_plan_filter", [i32, i32, vp, vp, vp, i32, vp, vp, vp, vp]),
                       ("mla_plan_merge", [i32, vp, vp, vp, vp, vp, vp, vp]),
                       ("mla_cache_shift_rows", [vp, i64, i64, i32, i32, vp, i64, i64, i32, i32,
                                                 ctypes.c_int, vp, vp, vp, i32, vp, vp]),
                       ("mla_rollback_lengths", [vp, vp, vp, vp, i32, vp, vp]),
                       ("mla_reconstruct_kv", [vp, i64, i64, vp, i32, i32, i32, i32, vp, i64, i64, vp, i64, i64,
                                               ctypes.c_int, vp, vp]),
                       ("mla_prefill_attend", [vp, i64, i64, vp, i64, i64, vp, i64, i64, vp, i64, i64, vp, i64,
                                               ctypes.c_int, ctypes.c_int, vp, vp, i32, i32, i32, i32, i32, i32,
                                               i64, f32, vp, i64, ctypes.c_int, vp, vp, vp]),
                       ("mla_append_compressed_q8", [vp, i64, i64, vp, i64, i64, ctypes.c_int, vp, f32, f32, vp, vp,
                                                     i64, i64, vp, i64, i32, vp, i64, i64, ctypes.c_int, vp, vp, vp,
                                                     i32, i32, i32, i32, i64, vp, vp]),
                       ("mla_quantize_cache", [vp, i64, i64, ctypes.c_int, vp, i64, i64, vp, i64, i32, vp, vp, i32,
                                               i32, i64, vp, vp]),
                       ("mla_dequantize_cache", [vp, i64, i64, vp, i64, i32, vp, i64, i64, ctypes.c_int, vp, vp, i32,
                                                 i32, i64, vp, vp]),
                       ("mla_decode_attend_q8", [vp, i64, i64, vp, i64, i64, vp, i64, i32, vp, i64, i64, ctypes.c_int,
                                                 vp, vp, i32, i32, i32, i32, i32, i64, vp, vp, i32, f32, vp, i64, i64,
                                                 ctypes.c_int, vp, vp, sz, vp, vp]),
                       ("mla_key_weights", [vp, i64, i64, vp, i64, i64, vp, i64, i64, ctypes.c_int, vp, vp, i32, i32,
                                            i32, i32, i32, i64, vp, f32, f32, i32, vp, i64, vp, vp]),
                       ("mla_key_weights_q8", [vp, i64, i64, vp, i64, i64, vp, i64, i32, vp, i64, i64, ctypes.c_int,
                                               vp, vp, i32, i32, i32, i32, i32, i64, vp, f32, f32, i32, vp, i64, vp,
                                               vp]),
                       ("mla_evict_plan", [vp, i64, vp, vp, i32, i64, i32, i32, i32, vp, i64, vp, vp, vp, vp]),
                       ("mla_cache_compact", [ctypes.POINTER(StateArray), i32, vp, vp, i64, vp, i32, i32, i64, vp,
                                              vp]),
                       ("mla_append_paged", [vp, i64, i64, vp, i64, i64, ctypes.c_int, vp, f32, f32, vp, vp, i64, i64, vp,
                                             i64, i64, ctypes.c_int, vp, i64, i32, i32, i32, vp, vp, vp, i32, i32, i32,
                                             i32, vp, vp]),
                       ("mla_tree_plan", [vp, i64, vp, vp, i32, i32, vp, vp, vp, vp]),
                       ("mla_decode_attend_paged", [vp, i64, i64, vp, i64, i64, vp, i64, i64, ctypes.c_int, vp, i64, i32,
                                                    i32, i32, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp, i32, f32, vp,
                                                    i64, i64, ctypes.c_int, vp, vp, sz, vp, vp]),
                       ("mla_commit_paged", [ctypes.POINTER(StateArray), i32, vp, i64, i32, i32, i32, vp, vp, i64, i32,
                                             vp, vp, i32, vp, vp])):
        getattr(lib, name).restype = ctypes.c_int
        getattr(lib, name).argtypes = args
    lib.mla_gather_selected.restype = ctypes.c_int
    lib.mla_gather_selected.argtypes = [vp, i64, i64, vp, i64, i64, ctypes.c_int, vp, vp, i32, i32, i32,
                                        i32, i64, vp, vp, i32, vp, vp, vp]
    return lib


lib = _load()
from . import _native  # noqa: E402  (the binding of the paged cache; it is linked with the library)


def _check(status: int) -> None:
    if status != 0:
        raise MLAError(status, lib.mla_last_error_detail().decode())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _dt(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return _DT[t.dtype]


def status_string(status: int) -> str:
    return lib.mla_status_string(status).decode()


def _scratch(nbytes: int, device, stream) -> torch.Tensor:
    """A workspace of one call.  The allocator hands memory freed on the current stream to that stream's next call: on
    another stream it is told to wait for the kernels that use it."""
    t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if stream is not None:
        t.record_stream(stream)
    return t


# ---------------------------------------------------------------- entry points

def rope_partial_interleaved(x: torch.Tensor, out: torch.Tensor, rotary_dims: int, theta: float,
                             position_offset: int = 0, row_offsets: Optional[torch.Tensor] = None,
                             stream=None) -> torch.Tensor:
    """``x`` / ``out``: 4-D ``[rows, tokens, inner, width]`` views (last dim contiguous)."""
    assert x.dim() == 4 and out.shape == x.shape and x.dtype == out.dtype
    assert x.stride(3) == 1 and out.stride(3) == 1
    ins = (ctypes.c_int64 * 3)(*x.stride()[:3])
    outs = (ctypes.c_int64 * 3)(*out.stride()[:3])
    _check(lib.mla_rope_partial_interleaved(
        _ptr(x), _ptr(out), _dt(x), x.shape[0], x.shape[1], x.shape[2], x.shape[3], ins, outs,
        rotary_dims, float(theta), _ptr(row_offsets), int(position_offset), _stream(stream)))
    return out


def absorb_q(q_nope: torch.Tensor, kv_b_proj: torch.Tensor, q_out: torch.Tensor, heads: int,
             nope: int, v_dim: int, rank: int, stream=None) -> torch.Tensor:
    """``q_nope`` ``[n_q, H, >=nope]`` view; writes ``q_out[:, :, :rank]``."""
    assert q_nope.dim() == 3 and q_out.dim() == 3 and q_nope.stride(2) == 1 and q_out.stride(2) == 1
    assert kv_b_proj.is_contiguous()
    _check(lib.mla_absorb_q(_ptr(q_nope), q_nope.stride(0), q_nope.stride(1), _ptr(kv_b_proj),
                            _ptr(q_out), q_out.stride(0), q_out.stride(1), _dt(q_nope),
                            q_nope.shape[0], heads, nope, v_dim, rank, _stream(stream)))
    return q_out


def decode_workspace_size(batch, s_q, heads, rank, rope_dim, t_max, k_max=0, selected=False,
                          dtype=torch.bfloat16) -> int:
    return lib.mla_decode_workspace_size(batch, s_q, heads, rank, rope_dim, t_max, k_max,
                                         1 if selected else 0, _DT[dtype])


def decode_kernel_kind(heads, rank, rope_dim, dtype=torch.bfloat16, out_dtype=torch.bfloat16) -> int:
    return lib.mla_decode_kernel_kind(heads, rank, rope_dim, _DT[dtype], _DT[out_dtype])


def decode_attend(q: torch.Tensor, latent: torch.Tensor, rope: torch.Tensor, kv_start, kv_len,
                  batch: int, s_q: int, softmax_scale: float, ctx_out: torch.Tensor,
                  lse_out: Optional[torch.Tensor] = None, sel: Optional[torch.Tensor] = None,
                  sel_count: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  device_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``q`` ``[n_q, H, rank+rope]``; ``latent`` ``[B_buf, T_max, rank]`` and ``rope``
    ``[B_buf, T_max, rope]`` views (a batch stride of 0 for the packed-flat layout is
    expressed by passing ``B_buf == 1``); ``ctx_out`` ``[n_q, H, rank]``."""
    n_q, heads, _ = q.shape
    rank, rope_dim = latent.shape[-1], rope.shape[-1]
    t_max = latent.shape[1]
    lat_bs = latent.stride(0) if latent.shape[0] > 1 else 0
    rope_bs = rope.stride(0) if rope.shape[0] > 1 else 0
    k_max = sel.shape[1] if sel is not None else 0
    if workspace is None:
        nbytes = decode_workspace_size(batch, s_q, heads, rank, rope_dim, t_max, k_max,
                                       sel is not None, latent.dtype)
        workspace = _scratch(max(nbytes, 1), q.device, stream)
    _check(lib.mla_decode_attend(
        _ptr(q), q.stride(0), q.stride(1), _ptr(latent), latent.stride(1), lat_bs,
        _ptr(rope), rope.stride(1), rope_bs, _dt(latent), _ptr(kv_start), _ptr(kv_len),
        batch, s_q, heads, rank, rope_dim, t_max, _ptr(sel), _ptr(sel_count), k_max,
        float(softmax_scale), _ptr(ctx_out), ctx_out.stride(0), ctx_out.stride(1), _dt(ctx_out),
        _ptr(lse_out), _ptr(workspace), workspace.numel(), _ptr(device_status), _stream(stream)))
    return ctx_out


def project_v(ctx: torch.Tensor, kv_b_proj: torch.Tensor, out: torch.Tensor, heads: int, nope: int,
              v_dim: int, stream=None) -> torch.Tensor:
    """``ctx`` ``[n_q, H, rank]`` view; ``out`` ``[n_q, H*v]`` (row stride free)."""
    n_q, _, rank = ctx.shape
    assert ctx.stride(2) == 1 and out.stride(1) == 1 and kv_b_proj.is_contiguous()
    _check(lib.mla_project_v(_ptr(ctx), ctx.stride(0), ctx.stride(1), _ptr(kv_b_proj), _dt(ctx),
                             _ptr(out), out.stride(0), _dt(out), n_q, heads, nope, v_dim, rank,
                             _stream(stream)))
    return out


def decode_step_workspace_size(batch, s_q, heads, nope, v_dim, rank, rope_dim, t_max, k_max=0,
                               selected=False, dtype=torch.bfloat16) -> int:
    return lib.mla_decode_step_workspace_size(batch, s_q, heads, nope, v_dim, rank, rope_dim, t_max, k_max,
                                              1 if selected else 0, _DT[dtype])


def decode_step(q_nope: torch.Tensor, q_rope: torch.Tensor, theta: float, kv_b_proj: torch.Tensor,
                latent: torch.Tensor, rope: torch.Tensor, kv_start, kv_len, batch: int, s_q: int, nope: int,
                v_dim: int, softmax_scale: float, out: torch.Tensor, lse_out: Optional[torch.Tensor] = None,
                row_offsets: Optional[torch.Tensor] = None, position_offset: int = 0,
                sel: Optional[torch.Tensor] = None, sel_count: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, device_status: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """Fused decode step.  ``q_nope`` ``[n_q, H, >=nope]`` and ``q_rope`` ``[n_q, H, >=rope]`` views
    (raw, pair-interleaved); cache views as for ``decode_attend``; ``out`` ``[n_q, H*v]``."""
    n_q, heads, _ = q_nope.shape
    rank, rope_dim = latent.shape[-1], rope.shape[-1]
    t_max = latent.shape[1]
    lat_bs = latent.stride(0) if latent.shape[0] > 1 else 0
    rope_bs = rope.stride(0) if rope.shape[0] > 1 else 0
    k_max = sel.shape[1] if sel is not None else 0
    if workspace is None:
        nbytes = decode_step_workspace_size(batch, s_q, heads, nope, v_dim, rank, rope_dim, t_max, k_max,
                                            sel is not None, latent.dtype)
        workspace = _scratch(max(nbytes, 256), latent.device, stream)
    _check(lib.mla_decode_step(
        _ptr(q_nope), q_nope.stride(0), q_nope.stride(1), _ptr(q_rope), q_rope.stride(0), q_rope.stride(1),
        _ptr(row_offsets), int(position_offset), float(theta), _ptr(kv_b_proj),
        _ptr(latent), latent.stride(1), lat_bs, _ptr(rope), rope.stride(1), rope_bs, _dt(latent),
        _ptr(kv_start), _ptr(kv_len), batch, s_q, heads, nope, v_dim, rank, rope_dim, t_max,
        _ptr(sel), _ptr(sel_count), k_max, float(softmax_scale), _ptr(out), out.stride(0), _dt(out),
        _ptr(lse_out), _ptr(workspace), workspace.numel(), _ptr(device_status), _stream(stream)))
    return out


def append_compressed(latent_raw: torch.Tensor, rope_raw: torch.Tensor, norm_weight: torch.Tensor, eps: float,
                      theta: float, latent: torch.Tensor, rope: torch.Tensor, kv_start, kv_len,
                      kv_len_out: Optional[torch.Tensor] = None, row_offsets: Optional[torch.Tensor] = None,
                      device_status: Optional[torch.Tensor] = None, stream=None):
    """``latent_raw`` ``[B, S, rank]`` / ``rope_raw`` ``[B, S, rope]`` views (last dim contiguous); cache
    views ``[B_buf, T_max, .]`` as for ``decode_attend`` (``B_buf == 1``: packed rows)."""
    B, S, rank = latent_raw.shape
    rope_dim = rope.shape[-1]
    lat_bs = latent.stride(0) if latent.shape[0] > 1 else 0
    rope_bs = rope.stride(0) if rope.shape[0] > 1 else 0
    _check(lib.mla_append_compressed(
        _ptr(latent_raw), latent_raw.stride(0), latent_raw.stride(1), _ptr(rope_raw), rope_raw.stride(0),
        rope_raw.stride(1), _dt(latent_raw), _ptr(norm_weight), float(eps), float(theta), _ptr(row_offsets),
        _ptr(latent), latent.stride(1), lat_bs, _ptr(rope), rope.stride(1), rope_bs, _dt(latent),
        _ptr(kv_start), _ptr(kv_len), _ptr(kv_len_out), B, S, rank, rope_dim, latent.shape[1],
        _ptr(device_status), _stream(stream)))


def select_topk(scores: torch.Tensor, lengths: torch.Tensor, top_k: int, selected: torch.Tensor,
                counts: torch.Tensor, device_status=None, stream=None):
    """``scores`` ``[n_rows, >=max length]`` f32 (last dim contiguous); ``selected`` ``[n_rows, >=top_k]``
    int32; ``counts`` ``[n_rows]`` int32."""
    assert scores.dtype == torch.float32 and scores.stride(1) == 1 and selected.stride(1) == 1
    _check(lib.mla_select_topk(_ptr(scores), scores.stride(0), _ptr(lengths), scores.shape[0], top_k,
                               _ptr(selected), selected.stride(0), _ptr(counts), _ptr(device_status),
                               _stream(stream)))


def selftest_bounded_wait(limit_cycles: int, device_status: torch.Tensor,
                          waited: Optional[torch.Tensor] = None, stream=None) -> None:
    _check(lib.mla_selftest_bounded_wait(int(limit_cycles), _ptr(device_status), _ptr(waited), _stream(stream)))


def gather_selected(latent: torch.Tensor, rope: torch.Tensor, kv_start, kv_len, batch: int, s_q: int,
                    sel: Optional[torch.Tensor], sel_count: torch.Tensor, k_max: int,
                    out: torch.Tensor, device_status=None, stream=None) -> torch.Tensor:
    lat_bs = latent.stride(0) if latent.shape[0] > 1 else 0
    rope_bs = rope.stride(0) if rope.shape[0] > 1 else 0
    _check(lib.mla_gather_selected(
        _ptr(latent), latent.stride(1), lat_bs, _ptr(rope), rope.stride(1), rope_bs, _dt(latent),
        _ptr(kv_start), _ptr(kv_len), batch, s_q, latent.shape[-1], rope.shape[-1], latent.shape[1],
        _ptr(sel), _ptr(sel_count), k_max, _ptr(out), _ptr(device_status), _stream(stream)))
    return out


# ---------------------------------------------------------------- cache row operations

def _host_i32(values) -> torch.Tensor:
    t = torch.as_tensor(values, dtype=torch.int32, device="cpu").contiguous()
    return t


def plan_rollback(left_pad, row_offsets, before_offsets, keep, width: int):
    """Host plan of a speculative-round rollback of a right-aligned cache.
    Returns ``(shift, new_left_pad, new_row_offsets, new_width)`` (CPU int32 tensors, int)."""
    lp, ro, bo, kp = (_host_i32(x) for x in (left_pad, row_offsets, before_offsets, keep))
    B = lp.numel()
    shift, pad, off = (torch.empty(B, dtype=torch.int32) for _ in range(3))
    w = ctypes.c_int32(0)
    _check(lib.mla_plan_rollback(B, int(width), _ptr(lp), _ptr(ro), _ptr(bo), _ptr(kp), _ptr(shift), _ptr(pad),
                                 _ptr(off), ctypes.addressof(w)))
    return shift, pad, off, w.value


def plan_filter(left_pad, row_offsets, keep_rows, width: int):
    """Host plan of a row filter. Returns ``(shift, new_left_pad, new_row_offsets, new_width)``."""
    lp, ro, kr = (_host_i32(x) for x in (left_pad, row_offsets, keep_rows))
    n = kr.numel()
    shift, pad, off = (torch.empty(n, dtype=torch.int32) for _ in range(3))
    w = ctypes.c_int32(0)
    _check(lib.mla_plan_filter(lp.numel(), int(width), _ptr(lp), _ptr(ro), _ptr(kr), n, _ptr(shift), _ptr(pad),
                               _ptr(off), ctypes.addressof(w)))
    return shift, pad, off, w.value


def plan_merge(source_width, left_pad, row_offsets):
    """Host plan of a merge of rows listed in merge order (each with its source's width).
    Returns ``(shift, zero_below, new_left_pad, new_width)``."""
    sw, lp, ro = (_host_i32(x) for x in (source_width, left_pad, row_offsets))
    n = lp.numel()
    shift, zero, pad = (torch.empty(n, dtype=torch.int32) for _ in range(3))
    w = ctypes.c_int32(0)
    _check(lib.mla_plan_merge(n, _ptr(sw), _ptr(lp), _ptr(ro), _ptr(shift), _ptr(zero), _ptr(pad),
                              ctypes.addressof(w)))
    return shift, zero, pad, w.value


def cache_shift_rows(src: torch.Tensor, dst: torch.Tensor, shift: Optional[torch.Tensor] = None,
                     src_row: Optional[torch.Tensor] = None, zero_below: Optional[torch.Tensor] = None,
                     device_status=None, stream=None) -> torch.Tensor:
    """``dst[i, c] = c < zero_below[i] ? 0 : src[src_row[i], (c + shift[i]) mod width]`` on views
    ``[B, width, F]`` (last dim contiguous); the index arrays are device int32 ``[dst rows]``."""
    assert src.dtype == dst.dtype and src.stride(-1) == 1 and dst.stride(-1) == 1
    _check(lib.mla_cache_shift_rows(_ptr(src), src.stride(1), src.stride(0), src.shape[0], src.shape[1],
                                    _ptr(dst), dst.stride(1), dst.stride(0), dst.shape[1], src.shape[2],
                                    _dt(src), _ptr(src_row), _ptr(shift), _ptr(zero_below), dst.shape[0],
                                    _ptr(device_status), _stream(stream)))
    return dst


def rollback_lengths(kv_len_before: torch.Tensor, keep: torch.Tensor, kv_len: torch.Tensor,
                     kv_len_out: Optional[torch.Tensor] = None, device_status=None, stream=None) -> torch.Tensor:
    """Per-row window layout: ``kv_len_out = kv_len_before + keep`` (in place when ``kv_len_out`` is None)."""
    out = kv_len if kv_len_out is None else kv_len_out
    _check(lib.mla_rollback_lengths(_ptr(kv_len_before), _ptr(keep), _ptr(kv_len), _ptr(out), kv_len.numel(),
                                    _ptr(device_status), _stream(stream)))
    return out


# ---------------------------------------------------------------- reconstructed prefill

def reconstruct_kv(latent: torch.Tensor, kv_b_proj: torch.Tensor, k_nope: torch.Tensor, v: torch.Tensor,
                   heads: int, nope: int, v_dim: int, device_status=None, stream=None):
    """``latent`` ``[rows, rank]`` view; ``k_nope`` ``[rows, H, nope]`` and ``v`` ``[rows, H, v]`` views."""
    assert latent.stride(-1) == 1 and k_nope.stride(-1) == 1 and v.stride(-1) == 1
    assert kv_b_proj.is_contiguous()
    _check(lib.mla_reconstruct_kv(_ptr(latent), latent.stride(0), latent.shape[0], _ptr(kv_b_proj), heads, nope,
                                  v_dim, latent.shape[1], _ptr(k_nope), k_nope.stride(0), k_nope.stride(1), _ptr(v),
                                  v.stride(0), v.stride(1), _dt(latent), _ptr(device_status), _stream(stream)))


def prefill_attend(q_nope: torch.Tensor, q_rope: torch.Tensor, k_nope: torch.Tensor, v: torch.Tensor,
                   rope: torch.Tensor, kv_start, kv_len, batch: int, s_q: int, t_max: int, packed: bool,
                   softmax_scale: float, out: torch.Tensor, lse_out: Optional[torch.Tensor] = None,
                   device_status=None, stream=None) -> torch.Tensor:
    """``q_nope`` ``[n_q, H, nope]`` / ``q_rope`` ``[n_q, H, rope]`` (rotated) views; ``k_nope`` / ``v``
    ``[buffer rows, H, .]``; ``rope`` ``[buffer rows, rope]``; ``out`` ``[n_q, H*v]``."""
    _, heads, nope = q_nope.shape
    _check(lib.mla_prefill_attend(
        _ptr(q_nope), q_nope.stride(0), q_nope.stride(1), _ptr(q_rope), q_rope.stride(0), q_rope.stride(1),
        _ptr(k_nope), k_nope.stride(0), k_nope.stride(1), _ptr(v), v.stride(0), v.stride(1), _ptr(rope),
        rope.stride(0), 1 if packed else 0, _dt(q_nope), _ptr(kv_start), _ptr(kv_len), batch, s_q, heads, nope,
        q_rope.shape[-1], v.shape[-1], int(t_max), float(softmax_scale), _ptr(out), out.stride(0), _dt(out),
        _ptr(lse_out), _ptr(device_status), _stream(stream)))
    return out


def default_scale(nope: int, rope_dim: int) -> float:
    """The page's softmax scale ``1/sqrt(qk_nope + qk_rope)``, as the library computes it."""
    return float(lib.mla_default_softmax_scale(nope, rope_dim))


# ---------------------------------------------------------------- 8-bit cache
#
# These calls run once per layer and token, so their checks are written to be
# cheap: each tensor's shape and strides are taken once.

_raw_stream = torch._C._cuda_getCurrentRawStream


def _launch_stream(stream, *tensors: Optional[torch.Tensor]) -> int:
    """The stream's handle, after a check that every tensor lives on the current CUDA device."""
    device = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"a tensor on {t.device} in a call on cuda:{device}")
    return _raw_stream(device) if stream is None else stream.cuda_stream


def _check_int32(count: int, *tensors: Optional[torch.Tensor]) -> None:
    """Lengths, starts, offsets and counts that the kernels read or write ``count`` of."""
    for t in tensors:
        assert t is None or (t.dtype is torch.int32 and t.is_contiguous() and t.numel() >= count), \
            f"lengths, starts and counts: contiguous int32, at least {count}"


def _check_status(status: Optional[torch.Tensor]) -> None:
    assert status is None or status.numel() * status.element_size() >= 4, "device_status: one int32"


def _cache_strides(t: torch.Tensor):
    """``(row stride, batch stride)`` of a ``[B_buf, T_max, F]`` view, rows contiguous; the batch stride is 0 for
    the packed-flat layout (``B_buf == 1``)."""
    batch, row, last = t.stride()
    assert last == 1, "the last axis must be contiguous"
    return row, (batch if t.shape[0] > 1 else 0)


def _q8_strides(codes: torch.Tensor, scales: torch.Tensor, scale_block: int):
    """``(T_max, rank, codes row stride, codes batch stride, scales batch stride)`` of ``codes`` ``[B_buf, T_max,
    rank]`` and ``scales`` ``[B_buf, >= ceil(T_max / scale_block)]``, one byte each."""
    rows, t_max, rank = codes.shape
    n, blocks = scales.shape
    batch, last = scales.stride()
    assert codes.element_size() == 1 and scales.element_size() == 1, "codes and scales hold one byte each"
    assert n == rows and last == 1 and blocks * scale_block >= t_max, "scales: [B_buf, >= ceil(T_max / scale_block)]"
    row, batch_c = _cache_strides(codes)
    return t_max, rank, row, batch_c, (batch if rows > 1 else 0)


def append_compressed_q8(latent_raw: torch.Tensor, rope_raw: torch.Tensor, norm_weight: torch.Tensor, eps: float,
                         theta: float, codes: torch.Tensor, scales: torch.Tensor, scale_block: int,
                         rope: torch.Tensor, kv_start, kv_len, kv_len_out: Optional[torch.Tensor] = None,
                         row_offsets: Optional[torch.Tensor] = None, device_status=None, stream=None):
    """``append_compressed`` into an 8-bit cache: ``codes`` ``[B_buf, T_max, rank]`` and ``scales`` ``[B_buf,
    blocks]`` of one byte each (uint8, or float8_e4m3fn / float8_e8m0fnu), one exponent per ``scale_block``
    buffer rows; ``rope`` ``[B_buf, T_max, rope]`` in f32 or bf16."""
    B, S, rank = latent_raw.shape
    l_batch, l_token, l_last = latent_raw.stride()
    r_batch, r_token, r_last = rope_raw.stride()
    t_max, width, c_row, c_batch, s_batch = _q8_strides(codes, scales, scale_block)
    k_row, k_batch = _cache_strides(rope)
    rows, t_rope, rope_dim = rope.shape
    dtype = latent_raw.dtype
    assert l_last == 1 and r_last == 1 and norm_weight.is_contiguous() and width == rank == norm_weight.numel()
    assert rope_raw.dtype is dtype and norm_weight.dtype is dtype and rope_raw.shape == (B, S, rope_dim)
    assert rows == codes.shape[0] and t_rope == t_max and kv_len.numel() == B and (rows == 1 or rows == B)
    _check_int32(B, kv_start, kv_len, kv_len_out, row_offsets)
    _check_status(device_status)
    handle = _launch_stream(stream, latent_raw, rope_raw, norm_weight, codes, scales, rope, kv_start, kv_len, kv_len_out,
                            row_offsets, device_status)
    _check(lib.mla_append_compressed_q8(
        latent_raw.data_ptr(), l_batch, l_token, rope_raw.data_ptr(), r_batch, r_token, _dt(latent_raw),
        norm_weight.data_ptr(), eps, theta, _ptr(row_offsets), codes.data_ptr(), c_row, c_batch, scales.data_ptr(),
        s_batch, scale_block, rope.data_ptr(), k_row, k_batch, _dt(rope), _ptr(kv_start), kv_len.data_ptr(),
        _ptr(kv_len_out), B, S, rank, rope_dim, t_max, _ptr(device_status), handle))


def quantize_cache(latent: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, scale_block: int, kv_start, kv_len,
                   device_status=None, stream=None) -> torch.Tensor:
    """The windows of ``latent`` ``[B_buf, T_max, rank]`` (f32 or bf16) into ``codes`` / ``scales``."""
    t_max, rank, c_row, c_batch, s_batch = _q8_strides(codes, scales, scale_block)
    l_row, l_batch = _cache_strides(latent)
    batch = kv_len.numel()
    assert latent.shape == codes.shape and latent.shape[0] in (1, batch)
    _check_int32(batch, kv_start, kv_len)
    _check_status(device_status)
    handle = _launch_stream(stream, latent, codes, scales, kv_start, kv_len, device_status)
    _check(lib.mla_quantize_cache(latent.data_ptr(), l_row, l_batch, _dt(latent), codes.data_ptr(), c_row, c_batch,
                                  scales.data_ptr(), s_batch, scale_block, _ptr(kv_start), kv_len.data_ptr(), batch, rank,
                                  t_max, _ptr(device_status), handle))
    return codes


def dequantize_cache(codes: torch.Tensor, scales: torch.Tensor, scale_block: int, latent: torch.Tensor, kv_start,
                     kv_len, device_status=None, stream=None) -> torch.Tensor:
    """The windows of an 8-bit cache back into ``latent`` ``[B_buf, T_max, rank]`` (f32 or bf16), exact."""
    t_max, rank, c_row, c_batch, s_batch = _q8_strides(codes, scales, scale_block)
    l_row, l_batch = _cache_strides(latent)
    batch = kv_len.numel()
    assert latent.shape == codes.shape and latent.shape[0] in (1, batch)
    _check_int32(batch, kv_start, kv_len)
    _check_status(device_status)
    handle = _launch_stream(stream, latent, codes, scales, kv_start, kv_len, device_status)
    _check(lib.mla_dequantize_cache(codes.data_ptr(), c_row, c_batch, scales.data_ptr(), s_batch, scale_block,
                                    latent.data_ptr(), l_row, l_batch, _dt(latent), _ptr(kv_start), kv_len.data_ptr(),
                                    batch, rank, t_max, _ptr(device_status), handle))
    return latent


def decode_attend_q8(q: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, scale_block: int, rope: torch.Tensor,
                     kv_start, kv_len, batch: int, s_q: int, softmax_scale: float, ctx_out: torch.Tensor,
                     lse_out: Optional[torch.Tensor] = None, sel: Optional[torch.Tensor] = None,
                     sel_count: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                     device_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``decode_attend`` over an 8-bit cache (views as in ``append_compressed_q8``; ``rope`` in the query's type).
    The workspace is that of ``decode_workspace_size`` for the query's type."""
    n_q, heads, width = q.shape
    q_row, q_head, q_last = q.stride()
    x_row, x_head, x_last = ctx_out.stride()
    t_max, rank, c_row, c_batch, s_batch = _q8_strides(codes, scales, scale_block)
    k_row, k_batch = _cache_strides(rope)
    rows, t_rope, rope_dim = rope.shape
    assert q_last == 1 and x_last == 1 and width == rank + rope_dim and n_q == batch * s_q
    assert ctx_out.shape == (n_q, heads, rank) and rope.dtype is q.dtype and t_rope == t_max
    assert rows == codes.shape[0] and (rows == 1 or rows == batch) and kv_len.numel() == batch
    _check_int32(batch, kv_start, kv_len)
    _check_status(device_status)
    if lse_out is not None:
        assert lse_out.dtype is torch.float32 and lse_out.is_contiguous() and lse_out.numel() == n_q * heads
    k_max = 0
    if sel is not None:
        k_max = sel.shape[1]
        assert sel.shape[0] == n_q and sel_count is not None and sel_count.numel() == n_q
        _check_int32(n_q, sel, sel_count)
    if workspace is None:
        nbytes = decode_workspace_size(batch, s_q, heads, rank, rope_dim, t_max, k_max, sel is not None, q.dtype)
        workspace = _scratch(max(nbytes, 1), q.device, stream)
    assert workspace.element_size() == 1 and workspace.is_contiguous()
    handle = _launch_stream(stream, q, codes, scales, rope, kv_start, kv_len, ctx_out, lse_out, sel, sel_count, workspace,
                            device_status)
    _check(lib.mla_decode_attend_q8(
        q.data_ptr(), q_row, q_head, codes.data_ptr(), c_row, c_batch, scales.data_ptr(), s_batch, scale_block,
        rope.data_ptr(), k_row, k_batch, _dt(q), _ptr(kv_start), kv_len.data_ptr(), batch, s_q, heads, rank, rope_dim,
        t_max, _ptr(sel), _ptr(sel_count), k_max, softmax_scale, ctx_out.data_ptr(), x_row, x_head, _dt(ctx_out),
        _ptr(lse_out), workspace.data_ptr(), workspace.numel(), _ptr(device_status), handle))
    return ctx_out


# ---------------------------------------------------------------- attention weights and eviction

def _weight_strides(q: torch.Tensor, lse: torch.Tensor, weights: torch.Tensor, rope: torch.Tensor, kv_start, kv_len,
                    batch: int, s_q: int, rows: int, t_max: int, rank: int, device_status):
    """Checks shared by both forms; ``(heads, q row stride, q head stride, rope_dim, rope strides, weights batch
    stride)``."""
    n_q, heads, width = q.shape
    q_row, q_head, q_last = q.stride()
    k_rows, t_rope, rope_dim = rope.shape
    k_row, k_batch = _cache_strides(rope)
    w_batch, w_last = weights.stride()
    w_rows, w_cols = weights.shape
    assert q_last == 1 and n_q == batch * s_q and width == rank + rope_dim and rope.dtype is q.dtype
    assert k_rows == rows and t_rope == t_max and (rows == 1 or rows == batch) and kv_len.numel() == batch
    assert lse.dtype is torch.float32 and lse.is_contiguous() and lse.numel() == n_q * heads
    assert weights.dtype is torch.float32 and w_last == 1 and w_rows == rows and w_cols >= t_max
    _check_int32(batch, kv_start, kv_len)
    _check_status(device_status)
    return heads, q_row, q_head, rope_dim, k_row, k_batch, (w_batch if rows > 1 else 0)


def key_weights(q: torch.Tensor, latent: torch.Tensor, rope: torch.Tensor, lse: torch.Tensor, kv_start, kv_len,
                batch: int, s_q: int, softmax_scale: float, weights: torch.Tensor, decay: float = 1.0, n_new: int = 0,
                device_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Adds the attention weight that each cached key received from ``q`` (all heads and tokens) to ``weights``
    ``[B_buf, T_max]`` f32, decayed first; the ``n_new`` newest keys start from zero.  ``q`` and the cache as for
    ``decode_attend``, ``lse`` its ``lse_out``."""
    rows, t_max, rank = latent.shape
    l_row, l_batch = _cache_strides(latent)
    assert latent.dtype is q.dtype
    heads, q_row, q_head, rope_dim, k_row, k_batch, w_batch = _weight_strides(q, lse, weights, rope, kv_start, kv_len,
                                                                              batch, s_q, rows, t_max, rank,
                                                                              device_status)
    handle = _launch_stream(stream, q, latent, rope, lse, kv_start, kv_len, weights, device_status)
    _check(lib.mla_key_weights(
        q.data_ptr(), q_row, q_head, latent.data_ptr(), l_row, l_batch, rope.data_ptr(), k_row, k_batch, _dt(q),
        _ptr(kv_start), kv_len.data_ptr(), batch, s_q, heads, rank, rope_dim, t_max, lse.data_ptr(), softmax_scale, decay,
        n_new, weights.data_ptr(), w_batch, _ptr(device_status), handle))
    return weights


def key_weights_q8(q: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, scale_block: int, rope: torch.Tensor,
                   lse: torch.Tensor, kv_start, kv_len, batch: int, s_q: int, softmax_scale: float,
                   weights: torch.Tensor, decay: float = 1.0, n_new: int = 0,
                   device_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``key_weights`` over an 8-bit cache."""
    t_max, rank, c_row, c_batch, s_batch = _q8_strides(codes, scales, scale_block)
    heads, q_row, q_head, rope_dim, k_row, k_batch, w_batch = _weight_strides(q, lse, weights, rope, kv_start, kv_len,
                                                                              batch, s_q, codes.shape[0], t_max, rank,
                                                                              device_status)
    handle = _launch_stream(stream, q, codes, scales, rope, lse, kv_start, kv_len, weights, device_status)
    _check(lib.mla_key_weights_q8(
        q.data_ptr(), q_row, q_head, codes.data_ptr(), c_row, c_batch, scales.data_ptr(), s_batch, scale_block,
        rope.data_ptr(), k_row, k_batch, _dt(q), _ptr(kv_start), kv_len.data_ptr(), batch, s_q, heads, rank, rope_dim,
        t_max, lse.data_ptr(), softmax_scale, decay, n_new, weights.data_ptr(), w_batch, _ptr(device_status), handle))
    return weights


def evict_plan(weights: torch.Tensor, kv_start, kv_len, n_keep: int, n_sink: int, n_recent: int, kept: torch.Tensor,
               counts: torch.Tensor, kv_len_out: Optional[torch.Tensor] = None, device_status=None,
               stream=None) -> torch.Tensor:
    """Window positions that stay, ascending: ``kept`` ``[B, >= n_keep]`` int32, ``counts`` ``[B]`` (``n_keep``, or
    -1 for a row within its budget).  ``weights`` ``[B_buf, T_max]`` f32."""
    rows, t_max = weights.shape
    w_batch, w_last = weights.stride()
    n, width = kept.shape
    k_row, k_last = kept.stride()
    batch = kv_len.numel()
    assert weights.dtype is torch.float32 and w_last == 1 and (rows == 1 or rows == batch)
    assert kept.dtype is torch.int32 and k_last == 1 and width >= n_keep and n == batch == counts.numel()
    _check_int32(batch, kv_start, kv_len, counts, kv_len_out)
    _check_status(device_status)
    handle = _launch_stream(stream, weights, kv_start, kv_len, kept, counts, kv_len_out, device_status)
    _check(lib.mla_evict_plan(weights.data_ptr(), w_batch if rows > 1 else 0, _ptr(kv_start), kv_len.data_ptr(), batch,
                              t_max, n_keep, n_sink, n_recent, kept.data_ptr(), k_row, counts.data_ptr(), _ptr(kv_len_out),
                              _ptr(device_status), handle))
    return kept


def cache_compact(arrays, kv_start, kept: torch.Tensor, counts: torch.Tensor, device_status=None, stream=None) -> None:
    """Moves each row's kept tokens to the front of its window in every array of ``arrays`` (``[B_buf, T_max, F]``
    views of any dtype, last dim contiguous; one launch), in place and in order."""
    n, width = kept.shape
    k_row, k_last = kept.stride()
    batch = counts.numel()
    rows, t_max, _ = arrays[0].shape
    assert kept.dtype is torch.int32 and k_last == 1 and n == batch and (rows == 1 or rows == batch)
    _check_int32(batch, kv_start, counts)
    _check_status(device_status)
    states = []
    for a in arrays:
        a_rows, a_len, features = a.shape
        a_row, a_batch = _cache_strides(a)
        size = a.element_size()
        assert a_rows == rows and a_len == t_max
        states.append((a.data_ptr(), a_row * size, a_batch * size, features * size))
    states = (StateArray * len(states))(*states)
    handle = _launch_stream(stream, kv_start, kept, counts, device_status, *arrays)
    _check(lib.mla_cache_compact(states, len(arrays), _ptr(kv_start), kept.data_ptr(), k_row, counts.data_ptr(), width,
                                 batch, t_max, _ptr(device_status), handle))


# ---------------------------------------------------------------- paged cache
#
# The tensors are checked and their sizes and strides taken in ``_native``.

_native.setup(MLAError, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)


def append_paged(latent_raw: torch.Tensor, rope_raw: torch.Tensor, norm_weight: torch.Tensor, eps: float, theta: float,
                 latent: torch.Tensor, rope: torch.Tensor, page_table: torch.Tensor, kv_len: torch.Tensor,
                 kv_len_out: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                 counts: Optional[torch.Tensor] = None, device_status: Optional[torch.Tensor] = None,
                 stream=None) -> None:
    """``append_compressed`` into pages.  ``latent_raw`` ``[B, S, rank]`` / ``rope_raw`` ``[B, S, rope]`` views; pools
    ``latent`` ``[num_pages, page_size, rank]`` / ``rope`` ``[num_pages, page_size, rope]``; ``page_table``
    ``[B, width]`` int32.  ``counts`` ``[B]``: how many of the S tokens each row has (all); ``positions`` ``[B, S]``:
    where they are rotated (at their key index)."""
    _native.append_paged(latent_raw, rope_raw, norm_weight, eps, theta, latent, rope, page_table, kv_len, kv_len_out,
                         positions, counts, device_status, stream)


def tree_plan(parents: torch.Tensor, kv_len: Optional[torch.Tensor], positions: torch.Tensor, tree_mask: torch.Tensor,
              counts: Optional[torch.Tensor] = None, device_status: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """Positions ``[B, n]`` int32 and ancestor masks ``[B * n, ceil(n / 64)]`` int64 (bits) of drafted trees, from
    ``parents`` ``[B, n]`` int32 (a node's parent before it, -1: a root); ``kv_len``: the rows' lengths before the
    trees are appended."""
    _native.tree_plan(parents, kv_len, positions, tree_mask, counts, device_status, stream)
    return tree_mask


def decode_paged_workspace_size(batch, s_q, heads, rank, rope_dim, t_max, k_max=0, selected=False,
                                dtype=torch.bfloat16) -> int:
    """Bytes of ``decode_attend_paged``'s workspace; ``t_max``: keys of a row's whole table."""
    return lib.mla_decode_paged_workspace_size(batch, s_q, heads, rank, rope_dim, t_max, k_max, 1 if selected else 0,
                                               _DT[dtype])


def decode_attend_paged(q: torch.Tensor, latent: torch.Tensor, rope: torch.Tensor, page_table: torch.Tensor,
                        kv_len: torch.Tensor, batch: int, s_q: int, softmax_scale: float, ctx_out: torch.Tensor,
                        lse_out: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                        tree_mask: Optional[torch.Tensor] = None, sel: Optional[torch.Tensor] = None,
                        sel_count: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                        device_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``decode_attend`` over pages: ``q`` ``[batch * s_q, H, rank+rope]``, pools and table as for ``append_paged``,
    ``kv_len`` with the new tokens; ``tree_mask`` as ``tree_plan`` writes it (none: the tokens follow one another)."""
    if workspace is None:
        nbytes = decode_paged_workspace_size(batch, s_q, q.shape[1], latent.shape[2], rope.shape[2],
                                             page_table.shape[1] * latent.shape[1], 0 if sel is None else sel.shape[1],
                                             sel is not None, q.dtype)
        workspace = _scratch(max(nbytes, 1), q.device, stream)
    _native.decode_attend_paged(q, latent, rope, page_table, kv_len, batch, s_q, softmax_scale, ctx_out, lse_out, counts,
                                tree_mask, sel, sel_count, workspace, device_status, stream)
    return ctx_out


class PagedArrays:
    """Pools ``[num_pages, page_size, F]`` that ``commit_paged`` moves together (every layer's latent and rope keys,
    say), checked once and kept: their memory must stay where it is (no ``resize_`` or ``set_``)."""

    def __init__(self, arrays) -> None:
        self.tensors = list(arrays)
        first = self.tensors[0]
        self.pages, self.page_size, _ = first.shape
        self.device = first.get_device()
        states = []
        for a in self.tensors:
            pages, rows, features = a.shape
            page, row, last = a.stride()
            size = a.element_size()
            assert last == 1, "the last axis must be contiguous"
            assert pages == self.pages and rows == self.page_size and a.device == first.device
            states.append((a.data_ptr(), row * size, page * size, features * size))
        self.states = (StateArray * len(states))(*states)
        self.address = ctypes.addressof(self.states)


def commit_paged(arrays, page_table: torch.Tensor, kv_len: torch.Tensor, path: torch.Tensor, counts: torch.Tensor,
                 kv_len_out: Optional[torch.Tensor] = None, device_status: Optional[torch.Tensor] = None,
                 stream=None) -> None:
    """Moves the accepted path of each row's tree to the end of its sequence in every pool of ``arrays`` (a
    ``PagedArrays``, or the pools, which are then looked through at every call: for 48 pools 55 us of host time instead
    of 3): ``path`` ``[B, width]`` int32 node numbers, ascending, ``counts`` ``[B]`` of them;
    ``kv_len``: the lengths before the trees were appended."""
    if not isinstance(arrays, PagedArrays):
        arrays = PagedArrays(arrays)
    _native.commit_paged(arrays.address, len(arrays.states), arrays.pages, arrays.page_size, arrays.device, page_table,
                         kv_len, path, counts, kv_len_out, device_status, stream)
