"""Python binding of libkrea2.so: argument marshalling from torch tensors to the C ABI.

Every function here has the name of a C entry point in ``include/krea2.h`` (without the
``krea2_`` prefix) and does no arithmetic of its own: it checks devices, dtypes and
contiguity, passes raw pointers and the current CUDA stream, and raises ``Krea2Error``
with the library's message when a call fails. Weight containers build the library's
device layout (fused [q|k|v|gate] rows, gate/up rows interleaved in 64-row groups).
"""
from __future__ import annotations

import ctypes
from typing import Dict, List, Optional, Sequence

import numpy as np
import torch

from . import _lib
from ._lib import KREA2_BF16, KREA2_F32, KREA2_EPI_RESID, KREA2_EPI_STORE, KREA2_EPI_SWIGLU  # noqa: F401

__all__ = [
    "Krea2Error", "lib", "dims_struct", "dtype_code", "workspace_size", "attention_workspace_size",
    "rope_tables", "gqa_attention", "gqa_attention_noalloc", "block_causal_key_end", "gqa_attention_block_causal",
    "kv_cache_append", "kv_cache_attention_workspace_size", "gqa_attention_kv_cache", "modulated_rmsnorm", "linear", "time_embed", "final_layer_workspace_size", "final_layer",
    "text_dims_struct", "TextWeights", "text_fusion_workspace_size", "text_fusion",
    "shift_mu", "sigma_schedule", "euler_cfg_step", "sample_workspace_size", "sample",
    "block_forward", "block_forward_traced", "BLOCK_STEPS", "launch_count", "backbone_forward", "check_device_error", "BlockWeights", "ModelWeights",
    "PagedBatch", "paged_batch_check", "paged_kv_append", "paged_attention_workspace_size", "gqa_attention_paged",
    "LoraAdapters", "lora_workspace_size", "lora_linear",
    "interleave_gate_up", "KREA2_BF16", "KREA2_F32", "KREA2_EPI_STORE", "KREA2_EPI_SWIGLU", "KREA2_EPI_RESID",
]

_LIB = None


class Krea2Error(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"krea2 error {code}: {msg}")
        self.code = code


def lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        _LIB = _lib.load()
    return _LIB


def _check(rc: int) -> None:
    if rc != 0:
        raise Krea2Error(rc, lib().krea2_last_error_string().decode())


def dims_struct(d) -> _lib.Krea2Dims:
    """Krea2Dims from any object with C, H, Hkv, D, F, axes, theta, eps, n_layers, in_ch, t_dim.

    A Krea2Dims is returned as it is, so a caller of many short calls can build it once."""
    if isinstance(d, _lib.Krea2Dims):
        return d
    s = _lib.Krea2Dims()
    s.C, s.H, s.Hkv, s.D, s.F = d.C, d.H, d.Hkv, d.D, d.F
    s.axes[0], s.axes[1], s.axes[2] = tuple(d.axes)
    s.theta, s.eps = float(d.theta), float(d.eps)
    s.n_layers, s.in_ch, s.t_dim = d.n_layers, d.in_ch, d.t_dim
    return s


def dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return KREA2_BF16
    if dt == torch.float32:
        return KREA2_F32
    raise TypeError(f"unsupported dtype {dt}")


def _p(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _s(stream: Optional[torch.cuda.Stream]) -> int:
    return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream


def _want(t: torch.Tensor, dt: torch.dtype, name: str) -> None:
    if t.dtype != dt:
        raise TypeError(f"{name} must be {dt}, got {t.dtype}")


def workspace_size(dims, B: int, T: int, N: int, dtype: torch.dtype) -> int:
    return int(lib().krea2_workspace_size(ctypes.byref(dims_struct(dims)), B, T, N, dtype_code(dtype)))


def attention_workspace_size(dims, B: int, T: int, N: int, dtype: torch.dtype) -> int:
    return int(lib().krea2_attention_workspace_size(ctypes.byref(dims_struct(dims)), B, T, N, dtype_code(dtype)))


def check_device_error(stream=None) -> None:
    _check(lib().krea2_check_device_error(_s(stream)))


def rope_tables(dims, position_ids: torch.Tensor, cos_out: torch.Tensor, sin_out: torch.Tensor, stream=None) -> None:
    for t, n in ((position_ids, "position_ids"), (cos_out, "cos_out"), (sin_out, "sin_out")):
        _want(t, torch.float32, n)
    if position_ids.dim() != 2 or position_ids.shape[1] != 3:
        raise ValueError("position_ids must have shape (T+N, 3)")
    S = position_ids.shape[0]
    _check(lib().krea2_rope_tables(ctypes.byref(dims_struct(dims)), _p(position_ids), S, _p(cos_out), _p(sin_out),
                                   _s(stream)))


def gqa_attention(dims, B: int, T: int, N: int, qkvg: torch.Tensor, q_norm_w: torch.Tensor, k_norm_w: torch.Tensor,
                  cos: torch.Tensor, sin: torch.Tensor, text_mask: Optional[torch.Tensor], out: torch.Tensor,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    dt = dtype_code(qkvg.dtype)
    _want(out, qkvg.dtype, "out")
    if text_mask is not None:
        _want(text_mask, torch.uint8, "text_mask")
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().krea2_gqa_attention(ctypes.byref(dims_struct(dims)), B, T, N, dt, _p(qkvg), _p(q_norm_w),
                                     _p(k_norm_w), _p(cos), _p(sin), _p(text_mask), _p(out), _p(workspace), ws,
                                     _s(stream)))


def gqa_attention_noalloc(dims, B: int, T: int, N: int, qkvg: torch.Tensor, q_norm_w: torch.Tensor,
                          k_norm_w: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor,
                          text_mask: Optional[torch.Tensor], out: torch.Tensor, stream=None) -> None:
    """gqa_attention for callers that cannot allocate: the library's static scratch replaces the workspace."""
    _want(out, qkvg.dtype, "out")
    if text_mask is not None:
        _want(text_mask, torch.uint8, "text_mask")
    _check(lib().krea2_gqa_attention_noalloc(ctypes.byref(dims_struct(dims)), B, T, N, dtype_code(qkvg.dtype),
                                             _p(qkvg), _p(q_norm_w), _p(k_norm_w), _p(cos), _p(sin),
                                             _p(text_mask), _p(out), _s(stream)))


def block_causal_key_end(image_ids: np.ndarray) -> np.ndarray:
    """Per-query key prefix of the block-causal pattern (host computation in the library)."""
    ids = np.ascontiguousarray(image_ids, dtype=np.int32)
    out = np.zeros(len(ids), dtype=np.int32)
    _check(lib().krea2_block_causal_key_end(ids.ctypes.data, len(ids), out.ctypes.data))
    return out


def gqa_attention_block_causal(dims, B: int, T: int, N: int, qkvg: torch.Tensor, q_norm_w: torch.Tensor,
                               k_norm_w: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor,
                               text_mask: Optional[torch.Tensor], key_end: torch.Tensor, out: torch.Tensor,
                               workspace: torch.Tensor, stream=None) -> None:
    _want(key_end, torch.int32, "key_end")
    _want(out, qkvg.dtype, "out")
    _check(lib().krea2_gqa_attention_block_causal(
        ctypes.byref(dims_struct(dims)), B, T, N, dtype_code(qkvg.dtype), _p(qkvg), _p(q_norm_w), _p(k_norm_w),
        _p(cos), _p(sin), _p(text_mask), _p(key_end), _p(out), _p(workspace),
        workspace.numel() * workspace.element_size(), _s(stream)))


def kv_cache_append(dims, B: int, n: int, row0: int, qkvg: torch.Tensor, k_norm_w: torch.Tensor, cos: torch.Tensor,
                    sin: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, stream=None) -> None:
    """Keys and values of n tokens into rows [row0, row0 + n) of a (B, capacity, Hkv*D) cache."""
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _want(t, qkvg.dtype, name)
    if k_cache.shape != v_cache.shape or k_cache.dim() != 3 or k_cache.shape[0] != B:
        raise ValueError("k_cache and v_cache must both be (B, capacity, Hkv*D)")
    _check(lib().krea2_kv_cache_append(ctypes.byref(dims_struct(dims)), B, n, row0, k_cache.shape[1],
                                       dtype_code(qkvg.dtype), _p(qkvg), _p(k_norm_w), _p(cos), _p(sin),
                                       _p(k_cache), _p(v_cache), _s(stream)))


def kv_cache_attention_workspace_size(dims, B: int, Nq: int, dtype: torch.dtype) -> int:
    return int(lib().krea2_kv_cache_attention_workspace_size(ctypes.byref(dims_struct(dims)), B, Nq,
                                                             dtype_code(dtype)))


def gqa_attention_kv_cache(dims, B: int, T: int, L: int, Nq: int, qkvg: torch.Tensor, q_norm_w: torch.Tensor,
                           cos: torch.Tensor, sin: torch.Tensor, text_mask: Optional[torch.Tensor],
                           k_cache: torch.Tensor, v_cache: torch.Tensor, key_end: Optional[torch.Tensor],
                           out: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    """Attention of the Nq tokens at key positions [L - Nq, L) over the first L cached keys."""
    if key_end is not None:
        _want(key_end, torch.int32, "key_end")
    _want(out, qkvg.dtype, "out")
    _check(lib().krea2_gqa_attention_kv_cache(
        ctypes.byref(dims_struct(dims)), B, T, L, Nq, dtype_code(qkvg.dtype), _p(qkvg), _p(q_norm_w), _p(cos),
        _p(sin), _p(text_mask), _p(k_cache), _p(v_cache), k_cache.shape[1], _p(key_end), _p(out), _p(workspace),
        workspace.numel() * workspace.element_size(), _s(stream)))


def modulated_rmsnorm(dims, B: int, S: int, h: torch.Tensor, norm_w: torch.Tensor, temb: torch.Tensor,
                      table: torch.Tensor, chunk: int, out: torch.Tensor, stream=None) -> None:
    _check(lib().krea2_modulated_rmsnorm(ctypes.byref(dims_struct(dims)), B, S, dtype_code(out.dtype), _p(h),
                                         _p(norm_w), _p(temb), _p(table), chunk, _p(out), _s(stream)))


def linear(epilogue: int, A: torch.Tensor, W: torch.Tensor, out: torch.Tensor, gate: Optional[torch.Tensor] = None,
           rows_per_batch: int = 1, gate_stride: int = 0, stream=None) -> None:
    M, K = A.shape
    Nw = W.shape[0]
    if W.shape[1] != K:
        raise ValueError("A and W disagree on K")
    _want(W, A.dtype, "W")
    _check(lib().krea2_linear(dtype_code(A.dtype), epilogue, M, Nw, K, _p(A), _p(W), _p(out), _p(gate),
                              rows_per_batch, gate_stride, _s(stream)))


def time_embed(dims, timestep: torch.Tensor, mw: "ModelWeights", temb_out: torch.Tensor, e_out: torch.Tensor,
               scratch: torch.Tensor, stream=None) -> None:
    _check(lib().krea2_time_embed(ctypes.byref(dims_struct(dims)), timestep.shape[0], mw.dtype_code, _p(timestep),
                                  ctypes.byref(mw.struct), _p(temb_out), _p(e_out), _p(scratch), _s(stream)))


def final_layer_workspace_size(dims, B: int, N: int, dtype: torch.dtype) -> int:
    return int(lib().krea2_final_layer_workspace_size(ctypes.byref(dims_struct(dims)), B, N, dtype_code(dtype)))


def final_layer(dims, B: int, T: int, N: int, h: torch.Tensor, e: torch.Tensor, mw: "ModelWeights",
                velocity: torch.Tensor, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    ws = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().krea2_final_layer(ctypes.byref(dims_struct(dims)), B, T, N, mw.dtype_code, _p(h), _p(e),
                                   ctypes.byref(mw.struct), _p(velocity), _p(workspace), ws, _s(stream)))


def block_forward(dims, B: int, T: int, N: int, h: torch.Tensor, temb: torch.Tensor, bw: "BlockWeights",
                  cos: torch.Tensor, sin: torch.Tensor, text_mask: Optional[torch.Tensor], workspace: torch.Tensor,
                  stream=None) -> None:
    _want(h, torch.float32, "h")
    _check(lib().krea2_block_forward(ctypes.byref(dims_struct(dims)), B, T, N, bw.dtype_code, _p(h), _p(temb),
                                     ctypes.byref(bw.struct), _p(cos), _p(sin), _p(text_mask), _p(workspace),
                                     workspace.numel() * workspace.element_size(), _s(stream)))


def text_dims_struct(td) -> _lib.Krea2TextDims:
    s = _lib.Krea2TextDims()
    for f in ("Dt", "L", "H", "Hkv", "D", "F", "n_layerwise", "n_refiner", "C"):
        setattr(s, f, getattr(td, f))
    s.eps = float(td.eps)
    return s


def text_fusion_workspace_size(td, B: int, T: int, dtype: torch.dtype) -> int:
    return int(lib().krea2_text_fusion_workspace_size(ctypes.byref(text_dims_struct(td)), B, T, dtype_code(dtype)))


def text_fusion(td, B: int, T: int, ehs: torch.Tensor, text_mask: Optional[torch.Tensor], tw: "TextWeights",
                text_out: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    _want(ehs, tw.dtype, "ehs")
    _want(text_out, tw.dtype, "text_out")
    _check(lib().krea2_text_fusion(ctypes.byref(text_dims_struct(td)), B, T, tw.dtype_code, _p(ehs), _p(text_mask),
                                   ctypes.byref(tw.struct), _p(text_out), _p(workspace),
                                   workspace.numel() * workspace.element_size(), _s(stream)))


def shift_mu(image_seq_len: int) -> float:
    return float(lib().krea2_shift_mu(image_seq_len))


def sigma_schedule(n_steps: int, mu: float) -> np.ndarray:
    out = np.zeros(n_steps + 1, dtype=np.float32)
    _check(lib().krea2_sigma_schedule(n_steps, mu, out.ctypes.data))
    return out


def euler_cfg_step(x: torch.Tensor, v_cond: torch.Tensor, v_uncond: Optional[torch.Tensor], guidance: float,
                   sigma: float, sigma_next: float, x_model: Optional[torch.Tensor] = None, copies: int = 1,
                   timestep_out: Optional[torch.Tensor] = None, stream=None) -> None:
    _want(x, torch.float32, "x")
    _check(lib().krea2_euler_cfg_step(dtype_code(v_cond.dtype), x.numel(), _p(x), _p(v_cond), _p(v_uncond),
                                      guidance, sigma, sigma_next, _p(x_model), copies, _p(timestep_out),
                                      _s(stream)))


def sample_workspace_size(dims, T: int, N: int, dtype: torch.dtype, cfg: bool) -> int:
    return int(lib().krea2_sample_workspace_size(ctypes.byref(dims_struct(dims)), T, N, dtype_code(dtype), int(cfg)))


def sample(dims, T: int, N: int, latents: torch.Tensor, text_cond: torch.Tensor, text_uncond: Optional[torch.Tensor],
           mask_cond: Optional[torch.Tensor], mask_uncond: Optional[torch.Tensor], position_ids: torch.Tensor,
           sigmas: np.ndarray, guidance: float, mw: "ModelWeights", workspace: torch.Tensor, stream=None) -> None:
    """The device sampling loop (krea2_sample); `sigmas` is a host array of n_steps + 1 values."""
    _want(latents, torch.float32, "latents")
    sg = np.ascontiguousarray(sigmas, dtype=np.float32)
    _check(lib().krea2_sample(ctypes.byref(dims_struct(dims)), T, N, mw.dtype_code, _p(latents), _p(text_cond),
                              _p(text_uncond), _p(mask_cond), _p(mask_uncond), _p(position_ids), sg.ctypes.data,
                              len(sg) - 1, guidance, ctypes.byref(mw.struct), _p(workspace),
                              workspace.numel() * workspace.element_size(), _s(stream)))


BLOCK_STEPS = ("modulation", "norm1", "qkv_proj", "attention", "out_proj_resid", "norm2", "gate_up_swiglu",
               "down_proj_resid")


def block_forward_traced(dims, B: int, T: int, N: int, h: torch.Tensor, temb: torch.Tensor, bw: "BlockWeights",
                         cos: torch.Tensor, sin: torch.Tensor, text_mask: Optional[torch.Tensor],
                         workspace: torch.Tensor, events: Sequence[torch.cuda.Event], stream=None) -> None:
    """block_forward recording events[i] before launch i (BLOCK_STEPS order) and events[8] after."""
    if len(events) != 9:
        raise ValueError("need 9 events")
    st = stream if stream is not None else torch.cuda.current_stream()
    for e in events:
        if not e.cuda_event:
            e.record(st)  # torch creates the CUDA event lazily, on its first record
    arr = (ctypes.c_void_p * 9)(*[e.cuda_event for e in events])
    _want(h, torch.float32, "h")
    _check(lib().krea2_block_forward_traced(ctypes.byref(dims_struct(dims)), B, T, N, bw.dtype_code, _p(h), _p(temb),
                                            ctypes.byref(bw.struct), _p(cos), _p(sin), _p(text_mask),
                                            _p(workspace), workspace.numel() * workspace.element_size(), arr,
                                            _s(stream)))


def launch_count() -> int:
    return int(lib().krea2_launch_count())


def backbone_forward(dims, B: int, T: int, N: int, hidden_states: torch.Tensor, text_states: torch.Tensor,
                     position_ids: torch.Tensor, text_mask: Optional[torch.Tensor], timestep: torch.Tensor,
                     mw: "ModelWeights", velocity: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    _check(lib().krea2_backbone_forward(ctypes.byref(dims_struct(dims)), B, T, N, mw.dtype_code, _p(hidden_states),
                                        _p(text_states), _p(position_ids), _p(text_mask), _p(timestep),
                                        ctypes.byref(mw.struct), _p(velocity), _p(workspace),
                                        workspace.numel() * workspace.element_size(), _s(stream)))


# ----------------------------------------------------------------------------- ragged batches

# These calls are short next to what a checked argument costs in Python, so each tensor is checked by one
# function that looks at nothing twice and words its complaint only when there is one.

def _int32(v: int, name: str) -> int:
    # ctypes would pass on the low 32 bits of a larger number
    if not -2 ** 31 <= v < 2 ** 31:
        raise ValueError(f"{name} = {v} does not fit 32 bits")
    return v


def _complain(t: Optional[torch.Tensor], dev: int, dtype: torch.dtype, shape: tuple, name: str) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: expected a contiguous tensor")


def _arg(t: torch.Tensor, dev: int, dtype: torch.dtype, shape: tuple, name: str) -> int:
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _complain(t, dev, dtype, shape, name)


def _ws(t: Optional[torch.Tensor], dev: int) -> tuple:
    if t is None:
        return None, 0
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on cuda:{dev}")
    return t.data_ptr(), t.nbytes


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_on(dev: int, stream) -> int:
    """The stream to launch on, once it and the tensors are known to belong to the current device."""
    if dev != torch.cuda.current_device():
        raise ValueError(f"tensors are on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    if stream is None:
        return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream().cuda_stream
    if stream.device.index != dev:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to cuda:{dev}")
    return stream.cuda_stream


def _shape(t: torch.Tensor, shape: tuple, name: str) -> None:
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")


class PagedBatch:
    """A ragged batch over a paged key/value cache: device tensors plus the Krea2PagedBatch struct.

    q_start (R + 1), kv_len (R), page_table (R, max_pages): int32; k_pages, v_pages (num_pages, page_size,
    Hkv*D); rows: the packed rows that qkvg and out have (at least q_start[R]). The lengths and page
    numbers stay on the device and may change between calls, under a captured graph too."""

    def __init__(self, q_start: torch.Tensor, kv_len: torch.Tensor, page_table: torch.Tensor, k_pages: torch.Tensor,
                 v_pages: torch.Tensor, rows: int):
        for t, n in ((q_start, "q_start"), (kv_len, "kv_len"), (page_table, "page_table")):
            _want(t, torch.int32, n)
        if kv_len.dim() != 1 or page_table.dim() != 2:
            raise ValueError("kv_len must be (R), page_table (R, max_pages)")
        R = kv_len.shape[0]
        _shape(q_start, (R + 1,), "q_start")
        _shape(page_table, (R, page_table.shape[1]), "page_table")
        if k_pages.dim() != 3 or k_pages.shape != v_pages.shape or k_pages.dtype != v_pages.dtype:
            raise ValueError("k_pages and v_pages must both be (num_pages, page_size, Hkv*D) of one dtype")
        for v, n in ((R, "R"), (rows, "rows"), (page_table.shape[1], "max_pages"), (k_pages.shape[0], "num_pages"),
                     (k_pages.shape[1], "page_size")):
            _int32(v, n)
        self.dtype, self.device = k_pages.dtype, k_pages.device
        self.tensors = (q_start, kv_len, page_table, k_pages, v_pages)
        s = _lib.Krea2PagedBatch()
        s.R, s.M, s.max_pages = R, rows, page_table.shape[1]
        s.num_pages, s.page_size = k_pages.shape[0], k_pages.shape[1]
        s.q_start, s.kv_len, s.page_table, s.k_pages, s.v_pages = (_p(t) for t in self.tensors)
        if any(t.device != self.device for t in self.tensors):
            raise ValueError("the batch's tensors must be on one device")
        self.dev, self.R, self.rows, self.kv_cols = k_pages.get_device(), R, rows, k_pages.shape[2]
        self.struct = s
        self.ref = ctypes.byref(s)


def _host_int32(a, name: str) -> np.ndarray:
    a = np.asarray(a)
    if a.size and a.dtype.kind not in "iu":
        raise TypeError(f"{name} must hold integers, got {a.dtype}")
    if a.size:
        _int32(int(a.min()), name), _int32(int(a.max()), name)
    return np.ascontiguousarray(a, dtype=np.int32)


def paged_batch_check(q_start, kv_len, page_table, num_pages: int, page_size: int, rows: int) -> None:
    """Checks a batch's lengths and page numbers on the host (integer arrays, lists or CPU tensors)."""
    host = [_host_int32(a, n) for a, n in ((q_start, "q_start"), (kv_len, "kv_len"), (page_table, "page_table"))]
    for v, n in ((num_pages, "num_pages"), (page_size, "page_size"), (rows, "rows")):
        _int32(v, n)
    R = host[1].shape[0]
    if host[0].shape != (R + 1,) or host[2].ndim != 2 or host[2].shape[0] != R:
        raise ValueError("need q_start (R + 1), kv_len (R) and page_table (R, max_pages)")
    s = _lib.Krea2PagedBatch()
    s.R, s.M, s.max_pages, s.page_size, s.num_pages = R, rows, host[2].shape[1], page_size, num_pages
    s.q_start, s.kv_len, s.page_table = (a.ctypes.data for a in host)
    _check(lib().krea2_paged_batch_check(ctypes.byref(s)))


def _paged_cols(d: _lib.Krea2Dims, batch: PagedBatch) -> None:
    if batch.kv_cols != d.Hkv * d.D:
        raise ValueError(f"the pages have {batch.kv_cols} columns, the model has Hkv*D = {d.Hkv * d.D}")


def paged_kv_append(dims, batch: PagedBatch, qkvg: torch.Tensor, k_norm_w: torch.Tensor, cos: torch.Tensor,
                    sin: torch.Tensor, stream=None) -> None:
    """Keys and values of a ragged batch's new tokens into its pages."""
    d = dims if isinstance(dims, _lib.Krea2Dims) else dims_struct(dims)
    dev, rows, D = batch.dev, batch.rows, d.D
    _paged_cols(d, batch)
    table = (rows, D // 2)
    rc = lib().krea2_paged_kv_append(
        ctypes.byref(d), batch.ref, dtype_code(batch.dtype),
        _arg(qkvg, dev, batch.dtype, (rows, 2 * (d.H + d.Hkv) * D), "qkvg"),
        _arg(k_norm_w, dev, torch.float32, (D,), "k_norm_w"), _arg(cos, dev, torch.float32, table, "cos"),
        _arg(sin, dev, torch.float32, table, "sin"), _stream_on(dev, stream))
    if rc:
        _check(rc)


def paged_attention_workspace_size(dims, batch: PagedBatch, dtype: torch.dtype) -> int:
    return int(lib().krea2_paged_attention_workspace_size(ctypes.byref(dims_struct(dims)), ctypes.byref(batch.struct),
                                                          dtype_code(dtype)))


def gqa_attention_paged(dims, batch: PagedBatch, qkvg: torch.Tensor, q_norm_w: torch.Tensor, cos: torch.Tensor,
                        sin: torch.Tensor, text_mask: Optional[torch.Tensor], key_end: Optional[torch.Tensor],
                        out: torch.Tensor, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Attention of a ragged batch's new tokens over its pages; text_mask (R, T) uint8, key_end (rows) int32."""
    d = dims if isinstance(dims, _lib.Krea2Dims) else dims_struct(dims)
    dev, rows, D = batch.dev, batch.rows, d.D
    _paged_cols(d, batch)
    table = (rows, D // 2)
    T, mask, end = 0, None, None
    if text_mask is not None:
        T = _int32(text_mask.shape[-1], "text_mask's length")
        mask = _arg(text_mask, dev, torch.uint8, (batch.R, T), "text_mask")
    if key_end is not None:
        end = _arg(key_end, dev, torch.int32, (rows,), "key_end")
    ws, ws_bytes = _ws(workspace, dev)
    rc = lib().krea2_gqa_attention_paged(
        ctypes.byref(d), batch.ref, T, dtype_code(batch.dtype),
        _arg(qkvg, dev, batch.dtype, (rows, 2 * (d.H + d.Hkv) * D), "qkvg"),
        _arg(q_norm_w, dev, torch.float32, (D,), "q_norm_w"), _arg(cos, dev, torch.float32, table, "cos"),
        _arg(sin, dev, torch.float32, table, "sin"), mask, end,
        _arg(out, dev, batch.dtype, (rows, d.H * D), "out"), ws, ws_bytes, _stream_on(dev, stream))
    if rc:
        _check(rc)


class LoraAdapters:
    """Low-rank adapters of one projection: down (n, rank, K), up (n, Nw, rank) in the projection's dtype, scale
    (n) fp32. `up` has the order of the projection's weight rows (interleave_gate_up for SwiGLU)."""

    def __init__(self, down: torch.Tensor, up: torch.Tensor, scale: torch.Tensor):
        if down.dim() != 3 or up.dim() != 3 or up.dtype != down.dtype:
            raise ValueError("need down (n, rank, K) and up (n, Nw, rank) of one dtype")
        n, self.rank, self.K = down.shape
        self.Nw = up.shape[1]
        _shape(up, (n, self.Nw, self.rank), "up")
        _want(scale, torch.float32, "scale")
        _shape(scale, (n,), "scale")
        for v, m in ((n, "n_adapters"), (self.rank, "rank"), (self.K, "K"), (self.Nw, "Nw")):
            _int32(v, m)
        self.down, self.up, self.scale = down, up, scale
        self.dtype, self.device = down.dtype, down.device
        if up.device != self.device or scale.device != self.device:
            raise ValueError("the adapters' tensors must be on one device")
        self.struct = _lib.Krea2Lora()
        self.struct.n_adapters, self.struct.rank = n, self.rank
        self.struct.down, self.struct.up, self.struct.scale = _p(down), _p(up), _p(scale)
        self.dev = down.get_device()

    @staticmethod
    def fused(parts: Sequence[Sequence[tuple]], scale: torch.Tensor) -> "LoraAdapters":
        """Adapters of stacked projections (to_q, to_k, to_v, to_gate of w_qkvg) from those of each one.

        parts[a] lists adapter a's (down (r, K), up (N_i, r)) per projection, in the order of the stacked
        rows. Ranks add up (padded to a multiple of 8), and `up` is block diagonal."""
        rank = max(sum(d.shape[0] for d, _ in p) for p in parts)
        rank = max(8, (rank + 7) // 8 * 8)
        d0 = parts[0][0][0]
        down = d0.new_zeros(len(parts), rank, d0.shape[1])
        up = d0.new_zeros(len(parts), sum(u.shape[0] for _, u in parts[0]), rank)
        for a, p in enumerate(parts):
            j = c = 0
            for d, u in p:
                down[a, j:j + d.shape[0]] = d
                up[a, c:c + u.shape[0], j:j + d.shape[0]] = u
                j, c = j + d.shape[0], c + u.shape[0]
        return LoraAdapters(down, up, scale)


def lora_workspace_size(dtype: torch.dtype, epilogue: int, M: int, Nw: int, K: int, R: int, rank: int) -> int:
    for v, n in ((epilogue, "epilogue"), (M, "M"), (Nw, "Nw"), (K, "K"), (R, "R"), (rank, "rank")):
        _int32(v, n)
    return int(lib().krea2_lora_workspace_size(dtype_code(dtype), epilogue, M, Nw, K, R, rank))


def lora_linear(epilogue: int, A: torch.Tensor, W: torch.Tensor, adapters: LoraAdapters, row_start: torch.Tensor,
                adapter: torch.Tensor, out: torch.Tensor, workspace: torch.Tensor, gate: Optional[torch.Tensor] = None,
                rows_per_batch: int = 0, gate_stride: Optional[int] = None, stream=None) -> None:
    """linear() with the adapter of each row's request; row_start (R + 1) and adapter (R) int32 device tensors.

    rows_per_batch = 0 gates a residual with the gate row of the row's request; gate_stride None is the
    gate's row length."""
    dev, dt, K, Nw, R = adapters.dev, adapters.dtype, adapters.K, adapters.Nw, _int32(adapter.shape[0], "R")
    M = _int32(A.shape[0], "M")
    _int32(epilogue, "epilogue")
    resid = epilogue == KREA2_EPI_RESID
    gate_p = None
    if resid:
        if gate is None:
            raise ValueError("a residual epilogue needs a gate")
        if gate_stride is None:
            gate_stride = gate.shape[-1]
        _int32(rows_per_batch, "rows_per_batch")
        rows = R if rows_per_batch == 0 else (M + rows_per_batch - 1) // max(rows_per_batch, 1)
        if gate.numel() < (rows - 1) * gate_stride + Nw:
            raise ValueError(f"the gate has {gate.numel()} values, {rows} rows of stride {gate_stride} are read")
        gate_p = _arg(gate, dev, torch.float32, gate.shape, "gate")
    ws, ws_bytes = _ws(workspace, dev)
    s = _lib.Krea2Lora.from_buffer_copy(adapters.struct)
    s.R = R
    s.row_start = _arg(row_start, dev, torch.int32, (R + 1,), "row_start")
    s.adapter = _arg(adapter, dev, torch.int32, (R,), "adapter")
    rc = lib().krea2_lora_linear(
        dtype_code(dt), epilogue, M, Nw, K, _arg(A, dev, dt, (M, K), "A"), _arg(W, dev, dt, (Nw, K), "W"),
        ctypes.byref(s),
        _arg(out, dev, torch.float32 if resid else dt, (M, Nw // 2 if epilogue == KREA2_EPI_SWIGLU else Nw), "out"),
        gate_p, rows_per_batch, gate_stride or 0, ws, ws_bytes, _stream_on(dev, stream))
    if rc:
        _check(rc)


# ----------------------------------------------------------------------------- weights

def interleave_gate_up(w_gate: torch.Tensor, w_up: torch.Tensor) -> torch.Tensor:
    """(F, C) gate and up rows -> (2F, C) in 64-row groups [gate 64 | up 64 | gate 64 | ...]."""
    F, C = w_gate.shape
    if F % 64:
        raise ValueError("intermediate size must be a multiple of 64")
    return torch.stack([w_gate.reshape(F // 64, 64, C), w_up.reshape(F // 64, 64, C)], dim=1).reshape(2 * F, C)


def _dev(a, dtype, device) -> torch.Tensor:
    t = a if isinstance(a, torch.Tensor) else torch.from_numpy(np.ascontiguousarray(a))
    return t.to(device=device, dtype=dtype).contiguous()


class BlockWeights:
    """One block's device tensors in the library layout plus the Krea2BlockWeights struct."""

    def __init__(self, w: Dict[str, object], dtype: torch.dtype, device):
        self.dtype = dtype
        self.dtype_code = dtype_code(dtype)
        f32 = torch.float32
        self.w_qkvg = _dev(torch.cat([_dev(w[k], dtype, device) for k in ("wq", "wk", "wv", "wg")], 0), dtype, device)
        self.w_out = _dev(w["wo"], dtype, device)
        self.w_gu = interleave_gate_up(_dev(w["w_gate"], dtype, device), _dev(w["w_up"], dtype, device)).contiguous()
        self.w_down = _dev(w["w_down"], dtype, device)
        self.norm1_w = _dev(w["norm1_w"], f32, device)
        self.norm2_w = _dev(w["norm2_w"], f32, device)
        self.q_norm_w = _dev(w["q_norm_w"], f32, device)
        self.k_norm_w = _dev(w["k_norm_w"], f32, device)
        self.table = _dev(w["table"], f32, device)
        self.struct = _lib.Krea2BlockWeights()
        self.fill(self.struct)

    def fill(self, s: _lib.Krea2BlockWeights) -> None:
        s.w_qkvg, s.w_out, s.w_gu, s.w_down = (_p(self.w_qkvg), _p(self.w_out), _p(self.w_gu), _p(self.w_down))
        s.norm1_w, s.norm2_w = _p(self.norm1_w), _p(self.norm2_w)
        s.q_norm_w, s.k_norm_w = _p(self.q_norm_w), _p(self.k_norm_w)
        s.scale_shift_table = _p(self.table)

    @staticmethod
    def random(dims, dtype: torch.dtype, device, generator: torch.Generator) -> "BlockWeights":
        """Seeded random weights drawn on the device (N(0,1)/sqrt(fan_in) linears, N(0, 0.1^2) rest)."""
        C, HD, KVD, F, D = dims.C, dims.H * dims.D, dims.Hkv * dims.D, dims.F, dims.D

        def n(shape, std):
            return (torch.randn(shape, device=device, generator=generator, dtype=torch.float32) * std).to(dtype)

        w = {"wq": n((HD, C), C ** -0.5), "wk": n((KVD, C), C ** -0.5), "wv": n((KVD, C), C ** -0.5),
             "wg": n((HD, C), C ** -0.5), "wo": n((C, HD), HD ** -0.5), "w_gate": n((F, C), C ** -0.5),
             "w_up": n((F, C), C ** -0.5), "w_down": n((C, F), F ** -0.5),
             "norm1_w": n((C,), 0.1).float(), "norm2_w": n((C,), 0.1).float(), "q_norm_w": n((D,), 0.1).float(),
             "k_norm_w": n((D,), 0.1).float(), "table": n((6, C), 0.1).float()}
        return BlockWeights(w, dtype, device)


class TextWeights:
    """Text-fusion device tensors: layerwise / refiner blocks (no modulation table), the layer-axis
    projection and txt_in."""

    def __init__(self, tw: Dict[str, object], dtype: torch.dtype, device):
        self.dtype = dtype
        self.dtype_code = dtype_code(dtype)
        self.layerwise = [BlockWeights(dict(w, table=np.zeros((6, 1), np.float32)), dtype, device)
                          for w in tw["layerwise"]]
        self.refiner = [BlockWeights(dict(w, table=np.zeros((6, 1), np.float32)), dtype, device)
                        for w in tw["refiner"]]
        self.layer_w = _dev(tw["layer_w"], torch.float32, device)
        self.txt_in_w = _dev(tw["txt_in_w"], dtype, device)
        self.txt_in_b = _dev(tw["txt_in_b"], torch.float32, device)
        self._lw = (_lib.Krea2BlockWeights * max(1, len(self.layerwise)))()
        self._rf = (_lib.Krea2BlockWeights * max(1, len(self.refiner)))()
        for arr, blocks in ((self._lw, self.layerwise), (self._rf, self.refiner)):
            for i, b in enumerate(blocks):
                b.fill(arr[i])
                arr[i].scale_shift_table = None   # fusion blocks carry no time modulation
        s = _lib.Krea2TextWeights()
        s.layerwise = ctypes.cast(self._lw, ctypes.POINTER(_lib.Krea2BlockWeights))
        s.refiner = ctypes.cast(self._rf, ctypes.POINTER(_lib.Krea2BlockWeights))
        s.layer_w, s.txt_in_w, s.txt_in_b = _p(self.layer_w), _p(self.txt_in_w), _p(self.txt_in_b)
        self.struct = s


class ModelWeights:
    """Backbone device tensors (img_in, time path, final layer) plus the block list."""

    def __init__(self, mw: Dict[str, object], blocks: Sequence[BlockWeights], dtype: torch.dtype, device):
        self.dtype = dtype
        self.dtype_code = dtype_code(dtype)
        f32 = torch.float32
        self.tensors = {}
        for k in ("img_in_w", "t1_w", "t2_w", "mod_w", "final_w"):
            self.tensors[k] = _dev(mw[k], dtype, device)
        for k in ("img_in_b", "t1_b", "t2_b", "mod_b", "final_norm_w", "final_table", "final_b"):
            self.tensors[k] = _dev(mw[k], f32, device)
        self.blocks: List[BlockWeights] = list(blocks)
        self._block_array = (_lib.Krea2BlockWeights * max(1, len(self.blocks)))()
        for i, b in enumerate(self.blocks):
            b.fill(self._block_array[i])
        s = _lib.Krea2ModelWeights()
        t = self.tensors
        s.img_in_w, s.img_in_b = _p(t["img_in_w"]), _p(t["img_in_b"])
        s.t1_w, s.t1_b, s.t2_w, s.t2_b = _p(t["t1_w"]), _p(t["t1_b"]), _p(t["t2_w"]), _p(t["t2_b"])
        s.mod_w, s.mod_b = _p(t["mod_w"]), _p(t["mod_b"])
        s.final_norm_w, s.final_table = _p(t["final_norm_w"]), _p(t["final_table"])
        s.final_w, s.final_b = _p(t["final_w"]), _p(t["final_b"])
        s.blocks = ctypes.cast(self._block_array, ctypes.POINTER(_lib.Krea2BlockWeights))
        self.struct = s
