"""Exact softmax attention for NVIDIA B200 (sm_100a).

Causal / sliding-window / full grouped-query prefill (contiguous, or the
newest positions against a paged context) and paged single-token decode (whole
cache, or a sliding window with sink positions and learned sink logits), with
the block tables, slot maps and query/key norms and rotations around them,
computed by hand-written CUDA kernels behind the C ABI of
``include/attn.h``. This module is the thin Python binding: it checks tensor
dtypes, shapes and devices, allocates outputs with PyTorch (device memory
plumbing only) and passes raw pointers and the current CUDA stream to the
library. Every step of the computation runs in the library's kernels; there
is no CPU or PyTorch fallback, and calls raise if the library is not built.
"""

from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import _lib
from ._lib import AttnError, STATUS_BIT_DEVICE_CHECK, STATUS_BIT_TIMEOUT  # noqa: F401

MASKS = {"full": 0, "causal": 1, "window": 2, "sliding_window": 2}

__all__ = ["prefill", "prefill_paged", "decode_paged", "decode_paged_window", "paged_gather", "decode_plan",
           "decode_workspace_bytes", "decode_window_workspace_bytes", "mla_decode_paged", "mla_decode_workspace_bytes",
           "prefill_backward", "prefill_backward_workspace_bytes", "prefill_paged_varlen",
           "prefill_paged_varlen_workspace_bytes", "paged_extend", "paged_release", "qk_norm_rope",
           "qk_norm_rope_paged", "qk_norm_rope_backward", "qk_norm_rope_backward_workspace_bytes",
           "AttnError", "version"]


def version() -> int:
    return int(_lib.lib().attn_version())


def _stream_handle(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _need(t: torch.Tensor, name: str, dtype, ndim: int) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {t.dim()}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_out(t, name: str, dtype, shape) -> None:
    """A caller-provided output must be a contiguous CUDA tensor of the exact
    dtype and shape: the library writes shape-many elements at its address."""
    _need(t, name, dtype, len(shape))
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _need_buf(t, name: str) -> None:
    """Workspace / status buffers: contiguous CUDA memory (any dtype)."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if name == "status" and (t.dtype != torch.int32 or t.numel() < 1):
        raise TypeError("status must be an int32 CUDA tensor with at least one element")


def prefill(q, k, v, mask: str = "causal", window: int = 0, scale: float | None = None, out=None, lse=None,
            status=None, stream=None, return_lse: bool = True):
    """O = softmax(scale * Q K^T + M) V for every query row; returns (O, LSE).

    q [B, Hq, N, d], k/v [B, Hkv, N, d], bf16 CUDA tensors; O bf16 like q,
    LSE fp32 [B, Hq, N] (natural log). mask: "full", "causal" or "window"
    (keys i - window < j <= i).
    """
    _need(q, "q", torch.bfloat16, 4)
    _need(k, "k", torch.bfloat16, 4)
    _need(v, "v", torch.bfloat16, 4)
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    if k.shape != (B, Hkv, N, d) or v.shape != k.shape:
        raise ValueError("k and v must be [B, Hkv, N, d] matching q")
    if mask not in MASKS:
        raise ValueError(f"mask must be one of {sorted(MASKS)}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    _need_out(out, "out", torch.bfloat16, q.shape)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need_out(lse, "lse", torch.float32, (B, Hq, N))
    _need_buf(status, "status")
    rc = _lib.lib().attn_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, N, d, MASKS[mask],
                                 int(window), float(scale), _ptr(status), _stream_handle(stream))
    _lib.check(rc, "attn_prefill")
    return out, lse


def prefill_backward_workspace_bytes(B: int, Hq: int, N: int) -> int:
    n = int(_lib.lib().attn_prefill_backward_workspace_bytes(B, Hq, N))
    if n == 0:
        raise AttnError(_lib.ATTN_ERR_INVALID_ARG, "attn_prefill_backward_workspace_bytes")
    return n


def prefill_backward(q, k, v, o, lse, d_o, mask: str = "causal", window: int = 0, scale: float | None = None,
                     dq=None, dk=None, dv=None, workspace=None, status=None, stream=None):
    """Gradients (dQ, dK, dV) of prefill() for the output gradient d_o, from the
    forward's inputs, output O and LSE. Shapes as in prefill(); bf16 results."""
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (d_o, "d_o")):
        _need(t, name, torch.bfloat16, 4)
    _need(lse, "lse", torch.float32, 3)
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    if k.shape != (B, Hkv, N, d) or v.shape != k.shape or o.shape != q.shape or d_o.shape != q.shape:
        raise ValueError("k, v must be [B, Hkv, N, d]; o and d_o like q")
    if lse.shape != (B, Hq, N):
        raise ValueError("lse must be [B, Hq, N]")
    if mask not in MASKS:
        raise ValueError(f"mask must be one of {sorted(MASKS)}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _need_out(dq, "dq", torch.bfloat16, q.shape)
    _need_out(dk, "dk", torch.bfloat16, k.shape)
    _need_out(dv, "dv", torch.bfloat16, v.shape)
    if workspace is None:
        workspace = torch.empty(prefill_backward_workspace_bytes(B, Hq, N), dtype=torch.uint8, device=q.device)
    _need_buf(workspace, "workspace")
    _need_buf(status, "status")
    rc = _lib.lib().attn_prefill_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(d_o), _ptr(lse), _ptr(dq), _ptr(dk),
                                          _ptr(dv), B, Hq, Hkv, N, d, MASKS[mask], int(window), float(scale),
                                          _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(status),
                                          _stream_handle(stream))
    _lib.check(rc, "attn_prefill_backward")
    return dq, dk, dv


def prefill_paged(q, k_cache, v_cache, block_table, seq_lens, max_seq_len: int, mask: str = "causal",
                  window: int = 0, scale: float | None = None, out=None, lse=None, status=None, stream=None,
                  return_lse: bool = True):
    """Prefix (chunked) prefill: the newest Nq positions of every sequence attend
    to its seq_lens[b] cached tokens through the block table; returns (O, LSE).

    q [B, Hq, Nq, d] bf16; caches [num_blocks, block_size, Hkv, d] bf16;
    block_table [B, max_blocks] int32; seq_lens [B] int32 (each >= Nq).
    Query row i of sequence b sits at position seq_lens[b] - Nq + i.
    """
    _need(q, "q", torch.bfloat16, 4)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(block_table, "block_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    B, Hq, Nq, d = q.shape
    num_blocks, block_size, Hkv, d2 = k_cache.shape
    if d2 != d or v_cache.shape != k_cache.shape:
        raise ValueError("caches must be [num_blocks, block_size, Hkv, d] matching q")
    if block_table.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("block_table and seq_lens need one row per sequence")
    if mask not in MASKS:
        raise ValueError(f"mask must be one of {sorted(MASKS)}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    _need_out(out, "out", torch.bfloat16, q.shape)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq, Nq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need_out(lse, "lse", torch.float32, (B, Hq, Nq))
    _need_buf(status, "status")
    rc = _lib.lib().attn_prefill_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seq_lens),
                                       _ptr(out), _ptr(lse), B, Hq, Hkv, Nq, d, num_blocks, block_size,
                                       block_table.shape[1], int(max_seq_len), MASKS[mask], int(window),
                                       float(scale), _ptr(status), _stream_handle(stream))
    _lib.check(rc, "attn_prefill_paged")
    return out, lse


def decode_plan(B: int, Hq: int, Hkv: int, max_seq_len: int, num_sms: int):
    """(chunk_tokens, num_splits) of the split-KV decode plan; host only."""
    chunk, splits = ctypes.c_int(0), ctypes.c_int(0)
    rc = _lib.lib().attn_decode_plan(B, Hq, Hkv, max_seq_len, num_sms, ctypes.byref(chunk), ctypes.byref(splits))
    _lib.check(rc, "attn_decode_plan")
    return chunk.value, splits.value


def decode_workspace_bytes(B: int, Hq: int, Hkv: int, d: int, max_seq_len: int, block_size: int) -> int:
    n = int(_lib.lib().attn_decode_workspace_bytes(B, Hq, Hkv, d, max_seq_len, block_size))
    if n == 0:
        raise AttnError(_lib.ATTN_ERR_INVALID_ARG, "attn_decode_workspace_bytes")
    return n


def decode_paged(q, k_cache, v_cache, block_table, seq_lens, max_seq_len: int, scale: float | None = None,
                 out=None, lse=None, workspace=None, status=None, stream=None, return_lse: bool = True):
    """One query token per sequence against its paged cache; returns (O, LSE).

    q [B, Hq, d] bf16; caches [num_blocks, block_size, Hkv, d] bf16;
    block_table [B, max_blocks] int32; seq_lens [B] int32.
    """
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(block_table, "block_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    B, Hq, d = q.shape
    num_blocks, block_size, Hkv, d2 = k_cache.shape
    if d2 != d or v_cache.shape != k_cache.shape:
        raise ValueError("caches must be [num_blocks, block_size, Hkv, d] matching q")
    if block_table.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("block_table and seq_lens need one row per sequence")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if workspace is None:
        nbytes = decode_workspace_bytes(B, Hq, Hkv, d, max_seq_len, block_size)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    _need_buf(workspace, "workspace")
    if out is None:
        out = torch.empty_like(q)
    _need_out(out, "out", torch.bfloat16, q.shape)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need_out(lse, "lse", torch.float32, (B, Hq))
    _need_buf(status, "status")
    rc = _lib.lib().attn_decode_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seq_lens),
                                      _ptr(out), _ptr(lse), B, Hq, Hkv, d, num_blocks, block_size,
                                      block_table.shape[1], int(max_seq_len), float(scale), _ptr(workspace),
                                      workspace.numel() * workspace.element_size(), _ptr(status),
                                      _stream_handle(stream))
    _lib.check(rc, "attn_decode_paged")
    return out, lse


def decode_window_workspace_bytes(B: int, Hq: int, Hkv: int, d: int, max_seq_len: int, block_size: int, window: int,
                                  n_sink: int) -> int:
    n = int(_lib.lib().attn_decode_window_workspace_bytes(B, Hq, Hkv, d, max_seq_len, block_size, window, n_sink))
    if n == 0:
        raise AttnError(_lib.ATTN_ERR_INVALID_ARG, "attn_decode_window_workspace_bytes")
    return n


def decode_paged_window(q, k_cache, v_cache, block_table, seq_lens, max_seq_len: int, window: int = 0,
                        n_sink: int = 0, sinks=None, scale: float | None = None, out=None, lse=None, workspace=None,
                        status=None, stream=None, return_lse: bool = True):
    """Paged decode with a sliding window of `window` positions (0: none), the
    first `n_sink` positions kept visible, and optional learned per-head sink
    logits `sinks` (fp32 [Hq], appended to the scaled scores with no value).
    Returns (O [B, Hq, d] bf16, LSE [B, Hq] fp32, including the sink column).
    """
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(block_table, "block_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    B, Hq, d = q.shape
    num_blocks, block_size, Hkv, d2 = k_cache.shape
    if d2 != d or v_cache.shape != k_cache.shape:
        raise ValueError("caches must be [num_blocks, block_size, Hkv, d] matching q")
    if block_table.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("block_table and seq_lens need one row per sequence")
    if sinks is not None:
        _need(sinks, "sinks", torch.float32, 1)
        if sinks.shape[0] != Hq:
            raise ValueError("sinks needs one logit per query head")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if workspace is None:
        nbytes = decode_window_workspace_bytes(B, Hq, Hkv, d, max_seq_len, block_size, int(window), int(n_sink))
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    _need_buf(workspace, "workspace")
    if out is None:
        out = torch.empty_like(q)
    _need_out(out, "out", torch.bfloat16, q.shape)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need_out(lse, "lse", torch.float32, (B, Hq))
    _need_buf(status, "status")
    rc = _lib.lib().attn_decode_paged_window(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                             _ptr(seq_lens), _ptr(sinks), _ptr(out), _ptr(lse), B, Hq, Hkv, d,
                                             num_blocks, block_size, block_table.shape[1], int(max_seq_len),
                                             int(window), int(n_sink), float(scale), _ptr(workspace),
                                             workspace.numel() * workspace.element_size(), _ptr(status),
                                             _stream_handle(stream))
    _lib.check(rc, "attn_decode_paged_window")
    return out, lse


def mla_decode_workspace_bytes(B: int, H: int, max_seq_len: int, d_latent: int = 512, d_rope: int = 64) -> int:
    n = int(_lib.lib().attn_mla_decode_workspace_bytes(B, H, d_latent, d_rope, max_seq_len))
    if n == 0:
        raise AttnError(_lib.ATTN_ERR_INVALID_ARG, "attn_mla_decode_workspace_bytes")
    return n


def mla_decode_paged(q, cache, block_table, seq_lens, max_seq_len: int, scale: float, d_latent: int = 512, out=None,
                     lse=None, workspace=None, status=None, stream=None, return_lse: bool = True):
    """Absorbed MLA decode: q [B, H, d_latent + d_rope] (absorbed content query,
    then positional query), cache [num_blocks, block_size, d_latent + d_rope]
    (latent, then positional key), both bf16. Returns the latent output
    O [B, H, d_latent] bf16 (apply the value up-projection afterwards) and
    LSE [B, H] fp32. `scale` is 1 / sqrt(d_head + d_rope).
    """
    _need(q, "q", torch.bfloat16, 3)
    _need(cache, "cache", torch.bfloat16, 3)
    _need(block_table, "block_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    B, H, width = q.shape
    num_blocks, block_size, width2 = cache.shape
    if width2 != width or width <= d_latent:
        raise ValueError("q and cache rows must both be d_latent + d_rope wide")
    if block_table.shape[0] != B or seq_lens.shape[0] != B:
        raise ValueError("block_table and seq_lens need one row per sequence")
    d_rope = width - d_latent
    if workspace is None:
        workspace = torch.empty(mla_decode_workspace_bytes(B, H, max_seq_len, d_latent, d_rope), dtype=torch.uint8,
                                device=q.device)
    _need_buf(workspace, "workspace")
    if out is None:
        out = torch.empty((B, H, d_latent), dtype=torch.bfloat16, device=q.device)
    _need_out(out, "out", torch.bfloat16, (B, H, d_latent))
    if lse is None and return_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need_out(lse, "lse", torch.float32, (B, H))
    _need_buf(status, "status")
    rc = _lib.lib().attn_mla_decode_paged(_ptr(q), _ptr(cache), _ptr(block_table), _ptr(seq_lens), _ptr(out), _ptr(lse),
                                          B, H, d_latent, d_rope, num_blocks, block_size, block_table.shape[1],
                                          int(max_seq_len), float(scale), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(), _ptr(status),
                                          _stream_handle(stream))
    _lib.check(rc, "attn_mla_decode_paged")
    return out, lse


def paged_gather(cache, block_table, seq_lens, max_seq_len: int, out=None, status=None, stream=None):
    """Contiguous [B, Hkv, max_seq_len, d] copy of a paged cache (zeros past seq_len)."""
    _need(cache, "cache", torch.bfloat16, 4)
    _need(block_table, "block_table", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    num_blocks, block_size, Hkv, d = cache.shape
    B = block_table.shape[0]
    if out is None:
        out = torch.empty((B, Hkv, max_seq_len, d), dtype=cache.dtype, device=cache.device)
    _need_out(out, "out", torch.bfloat16, (B, Hkv, max_seq_len, d))
    _need_buf(status, "status")
    rc = _lib.lib().attn_paged_gather(_ptr(cache), _ptr(block_table), _ptr(seq_lens), _ptr(out), B, Hkv, d,
                                      num_blocks, block_size, block_table.shape[1], int(max_seq_len), _ptr(status),
                                      _stream_handle(stream))
    _lib.check(rc, "attn_paged_gather")
    return out


def _here(first, stream) -> bool:
    """Whether a call can run as it stands: no stream named and the device of its first argument current."""
    if not isinstance(first, torch.Tensor) or not first.is_cuda:
        raise ValueError("the inputs must be CUDA tensors")
    return stream is None and first.get_device() == torch._C._cuda_getDevice()


def _elsewhere(fn, first, args: dict):
    """fn again with the device of its first argument current and, when the
    caller names a stream, with that stream current: outputs and workspaces
    then come from that stream's memory, so nothing else can still be using
    them when the kernels run."""
    stream = args.pop("stream")
    if stream is None:
        with torch.cuda.device(first.device):
            return fn(**args)
    if stream.device != first.device:
        raise ValueError(f"stream is on {stream.device}, the inputs on {first.device}")
    with torch.cuda.stream(stream):
        return fn(**args)


def _need_on(t, name: str, dtype, shape, dev, strided: bool = False) -> None:
    """One input or output: dtype, exact shape, device, and contiguous unless strided."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is dtype and t.get_device() == dev.index and t.shape == shape and (strided or t.is_contiguous()):
        return  # most of a small call's time is the host's: the reasons are looked for only when there is one
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} must be a CUDA tensor on {dev}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _need_dims(t, name: str, ndim: int, layout: str) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != ndim:
        raise ValueError(f"{name} must be {layout}")


def _need_status(t, dev) -> None:
    if t is not None:
        _need_buf(t, "status")
        if t.device != dev:
            raise ValueError(f"status must be on {dev}")


def _need_workspace(t, dev) -> None:
    if t is not None:
        _need_buf(t, "workspace")
        if t.device != dev:
            raise ValueError(f"workspace must be on {dev}")


def _out_on(t, name: str, dtype, shape, dev, like=None):
    """The caller's output, checked, or a new one (like: a tensor of its dtype and device, the quicker way to one)."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev) if like is None else like.new_empty(shape)
    _need_on(t, name, dtype, shape, dev)
    return t


def _current(dev) -> int:
    """The raw handle of the device's current stream."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _addr(t) -> int:
    return 0 if t is None else t.data_ptr()


def prefill_paged_varlen_workspace_bytes(d: int) -> int:
    n = int(_lib.lib().attn_prefill_paged_varlen_workspace_bytes(d))
    if n == 0:
        raise AttnError(_lib.ATTN_ERR_INVALID_ARG, "attn_prefill_paged_varlen_workspace_bytes")
    return n


def prefill_paged_varlen(q, k_cache, v_cache, block_table, cu_q, seq_lens, max_seq_len: int, mask: str = "causal",
                         window: int = 0, n_sink: int = 0, sinks=None, scale: float | None = None, out=None, lse=None,
                         workspace=None, status=None, return_lse: bool = True, stream=None):
    """prefill_paged() with each sequence's own number of query rows, packed;
    returns (O [T, Hq, d], LSE [T, Hq]).

    q [T, Hq, d] bf16; caches [num_blocks, block_size, Hkv, d] bf16;
    block_table [B, max_blocks] int32; cu_q [B + 1] int32: sequence b has rows
    [cu_q[b], cu_q[b + 1]), its newest positions; seq_lens [B] int32 counts its
    cached tokens, the new ones included. window, n_sink and sinks as in
    decode_paged_window(), with mask="window". Rows outside [cu_q[0], cu_q[B])
    of a given out and lse stay as they were (else they are undefined). For single
    tokens alone with up to 8 query heads per K/V head decode_paged() and
    decode_paged_window() are quicker, for equal chunks of 512 rows and more
    prefill_paged().
    """
    if not _here(q, stream):
        return _elsewhere(prefill_paged_varlen, q, locals())
    _need_dims(q, "q", 3, "[T, Hq, d]")
    _need_dims(k_cache, "k_cache", 4, "[num_blocks, block_size, Hkv, d]")
    _need_dims(block_table, "block_table", 2, "[B, max_blocks]")
    dev, bf16, (T, Hq, d), B = q.device, torch.bfloat16, q.shape, block_table.shape[0]
    num_blocks, block_size, Hkv, _ = pool = k_cache.shape
    _need_on(q, "q", bf16, (T, Hq, d), dev)
    _need_on(k_cache, "k_cache", bf16, (num_blocks, block_size, Hkv, d), dev)
    _need_on(v_cache, "v_cache", bf16, pool, dev)
    _need_on(block_table, "block_table", torch.int32, block_table.shape, dev)
    _need_on(cu_q, "cu_q", torch.int32, (B + 1,), dev)
    _need_on(seq_lens, "seq_lens", torch.int32, (B,), dev)
    if sinks is not None:
        _need_on(sinks, "sinks", torch.float32, (Hq,), dev)
    if mask not in MASKS:
        raise ValueError(f"mask must be one of {sorted(MASKS)}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out = _out_on(out, "out", bf16, (T, Hq, d), dev, q)
    if lse is not None or return_lse:
        lse = _out_on(lse, "lse", torch.float32, (T, Hq), dev)
    _need_status(status, dev)
    if T == 0:
        return out, lse
    if workspace is None:
        workspace = torch.empty(prefill_paged_varlen_workspace_bytes(d), dtype=torch.uint8, device=dev)
    _need_workspace(workspace, dev)
    rc = _lib.lib().attn_prefill_paged_varlen(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                              block_table.data_ptr(), cu_q.data_ptr(), seq_lens.data_ptr(),
                                              _addr(sinks), out.data_ptr(), _addr(lse), B, T, Hq, Hkv, d, num_blocks,
                                              block_size, block_table.shape[1], int(max_seq_len), MASKS[mask],
                                              int(window), int(n_sink), float(scale), workspace.data_ptr(),
                                              workspace.numel() * workspace.element_size(), _addr(status),
                                              _current(dev))
    _lib.check(rc, "attn_prefill_paged_varlen")
    return out, lse


def _table_args(seq_lens, second, second_name, block_table, free_blocks, num_free, status):
    _need_dims(seq_lens, "seq_lens", 1, "[B]")
    _need_dims(block_table, "block_table", 2, "[B, max_blocks]")
    _need_dims(free_blocks, "free_blocks", 1, "[capacity]")
    dev, B, i32 = seq_lens.device, seq_lens.shape[0], torch.int32
    _need_on(seq_lens, "seq_lens", i32, (B,), dev)
    _need_on(second, second_name, i32, (B,), dev)
    _need_on(block_table, "block_table", i32, (B, block_table.shape[1]), dev)
    _need_on(free_blocks, "free_blocks", i32, (free_blocks.shape[0],), dev)
    _need_on(num_free, "num_free", i32, (1,), dev)
    _need_status(status, dev)
    return dev, B


def _int32_outs(given, dev):
    """Outputs [n] int32: those of (tensor or None, name, n) that the caller gave, the others out of one allocation."""
    sizes = [n for t, _, n in given if t is None]
    fresh = iter(torch.empty(sum(sizes), dtype=torch.int32, device=dev).unsafe_split_with_sizes(sizes) if sizes else ())
    outs = []
    for t, name, n in given:
        if t is None:
            t = next(fresh)
        else:
            _need_on(t, name, torch.int32, (n,), dev)
        outs.append(t)
    return outs


def paged_extend(seq_lens, new_lens, block_table, free_blocks, num_free, block_size: int, num_blocks: int,
                 max_tokens: int, seq_lens_out=None, num_free_out=None, cu_q=None, positions=None, slots=None,
                 status=None, stream=None):
    """The block table, positions and slot map of one serving step, from the
    requests' lengths; returns (seq_lens_out, num_free_out, cu_q, positions,
    slots) and writes the new entries of block_table.

    seq_lens, new_lens [B] int32: cached and new tokens of each sequence;
    free_blocks int32, a stack of num_free [1] free blocks; max_tokens rows of
    positions and slots are written, those past the new tokens as 0 and -1.
    cu_q [B + 1]: sequence b's new tokens are rows [cu_q[b], cu_q[b + 1]).
    seq_lens_out and num_free_out may be seq_lens and num_free themselves. A
    sequence that cannot be served gets the length -1 - seq_lens[b] (negative)
    and slots of -1, and sets the status bit.
    """
    if not _here(seq_lens, stream):
        return _elsewhere(paged_extend, seq_lens, locals())
    dev, B = _table_args(seq_lens, new_lens, "new_lens", block_table, free_blocks, num_free, status)
    n = max(0, int(max_tokens))
    positions, slots, cu_q, seq_lens_out, num_free_out = _int32_outs(
        ((positions, "positions", n), (slots, "slots", n), (cu_q, "cu_q", B + 1), (seq_lens_out, "seq_lens_out", B),
         (num_free_out, "num_free_out", 1)), dev)
    rc = _lib.lib().attn_paged_extend(seq_lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(),
                                      free_blocks.data_ptr(), num_free.data_ptr(), seq_lens_out.data_ptr(),
                                      num_free_out.data_ptr(), cu_q.data_ptr(), positions.data_ptr(),
                                      slots.data_ptr(), B, int(num_blocks), int(block_size), block_table.shape[1],
                                      free_blocks.shape[0], int(max_tokens), _addr(status), _current(dev))
    _lib.check(rc, "attn_paged_extend")
    return seq_lens_out, num_free_out, cu_q, positions, slots


def paged_release(seq_lens, finished, block_table, free_blocks, num_free, block_size: int, num_blocks: int,
                  seq_lens_out=None, num_free_out=None, status=None, stream=None):
    """Puts the blocks of the sequences with finished[b] != 0 (int32) back on
    the free list; returns (seq_lens_out, num_free_out), the finished lengths 0.
    A length -1 - L that paged_extend left counts as L. free_blocks is written
    from num_free on; in place as paged_extend."""
    if not _here(seq_lens, stream):
        return _elsewhere(paged_release, seq_lens, locals())
    dev, B = _table_args(seq_lens, finished, "finished", block_table, free_blocks, num_free, status)
    seq_lens_out, num_free_out = _int32_outs(((seq_lens_out, "seq_lens_out", B), (num_free_out, "num_free_out", 1)),
                                             dev)
    rc = _lib.lib().attn_paged_release(seq_lens.data_ptr(), finished.data_ptr(), block_table.data_ptr(),
                                       free_blocks.data_ptr(), num_free.data_ptr(), seq_lens_out.data_ptr(),
                                       num_free_out.data_ptr(), B, int(num_blocks), int(block_size),
                                       block_table.shape[1], free_blocks.shape[0], _addr(status), _current(dev))
    _lib.check(rc, "attn_paged_release")
    return seq_lens_out, num_free_out


@functools.lru_cache(maxsize=256)
def _strides(*values):
    """The host array of element strides that the library reads (made once for each set of values)."""
    return (ctypes.c_int64 * len(values))(*values)


def _need_heads(t, name: str, shape, dev) -> None:
    """A [.., heads, d] view whose head rows are contiguous (a view of a fused projection is one)."""
    _need_on(t, name, torch.bfloat16, shape, dev, strided=True)
    if t.stride(-1) != 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")


def _need_heads_out(t, name: str, shape, dev) -> None:
    _need_heads(t, name, shape, dev)
    if any(s == 0 and n > 1 for s, n in zip(t.stride(), shape)):
        raise ValueError(f"{name}: an output's rows may not share memory")


def _angles(q_weight, k_weight, cos, sin, positions, pos_shape, d, dev):
    """Checks weights, angle tables and positions; returns (weights are bf16, rotary_dim, max_pos)."""
    w_bf16 = 0
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight come together")
    if q_weight is not None:
        _need_dims(q_weight, "q_weight", 1, "[d]")
        dtype = q_weight.dtype
        if dtype is torch.bfloat16:
            w_bf16 = 1
        elif dtype is not torch.float32:
            raise TypeError(f"q_weight must be float32 or bfloat16, got {dtype}")
        _need_on(q_weight, "q_weight", dtype, (d,), dev)
        _need_on(k_weight, "k_weight", dtype, (d,), dev)
    _need_dims(cos, "cos", 2, "[max_pos, rotary_dim / 2]")
    shape = max_pos, half = cos.shape
    _need_on(cos, "cos", torch.float32, shape, dev)
    _need_on(sin, "sin", torch.float32, shape, dev)
    if positions is not None:
        _need_on(positions, "positions", torch.int32, pos_shape, dev)
    return w_bf16, 2 * half, max_pos


def qk_norm_rope(q, k, v, q_weight, k_weight, cos, sin, positions=None, eps: float = 1e-6, interleaved: bool = False,
                 q_out=None, k_out=None, v_out=None, status=None, stream=None):
    """RMS norm of each query and key head and the position rotation in one
    pass, into the layout of prefill(); returns (q, k, v) as [B, H, N, d].

    q [B, N, Hq, d], k and v [B, N, Hkv, d] bf16 (views of a fused projection
    are fine: only a head's elements must be contiguous); q_weight, k_weight
    [d] fp32 or bf16, both None for no norm; cos, sin [max_pos, rotary_dim / 2]
    fp32; positions [B, N] int32 (default 0 .. N - 1). The first rotary_dim
    elements turn in pairs (f, f + rotary_dim / 2), or (2 f, 2 f + 1) when
    interleaved.
    """
    if not _here(q, stream):
        return _elsewhere(qk_norm_rope, q, locals())
    _need_dims(q, "q", 4, "[B, N, Hq, d]")
    _need_dims(k, "k", 4, "[B, N, Hkv, d]")
    dev, (B, N, Hq, d), Hkv = q.device, q.shape, k.shape[2]
    _need_heads(q, "q", (B, N, Hq, d), dev)
    _need_heads(k, "k", (B, N, Hkv, d), dev)
    _need_heads(v, "v", (B, N, Hkv, d), dev)
    w_bf16, rd, max_pos = _angles(q_weight, k_weight, cos, sin, positions, (B, N), d, dev)
    _need_status(status, dev)
    q_out = _out_on(q_out, "q_out", torch.bfloat16, (B, Hq, N, d), dev, q)
    k_out = _out_on(k_out, "k_out", torch.bfloat16, (B, Hkv, N, d), dev, q)
    v_out = _out_on(v_out, "v_out", torch.bfloat16, (B, Hkv, N, d), dev, q)
    rc = _lib.lib().attn_qk_norm_rope(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                      _strides(*q.stride()[:3], *k.stride()[:3], *v.stride()[:3]),
                                      _addr(q_weight), _addr(k_weight), w_bf16, cos.data_ptr(), sin.data_ptr(),
                                      _addr(positions), q_out.data_ptr(), k_out.data_ptr(), v_out.data_ptr(), B, N,
                                      Hq, Hkv, d, rd, max_pos, float(eps), int(interleaved), _addr(status),
                                      _current(dev))
    _lib.check(rc, "attn_qk_norm_rope")
    return q_out, k_out, v_out


def qk_norm_rope_paged(q, k, v, q_weight, k_weight, cos, sin, positions, slots, k_cache, v_cache, eps: float = 1e-6,
                       interleaved: bool = False, q_out=None, status=None, stream=None):
    """The serving form of qk_norm_rope: packed tokens q [T, Hq, d], k and v
    [T, Hkv, d]; returns q [T, Hq, d] and writes the keys and values into the
    caches [num_blocks, block_size, Hkv, d] at slots [T] (int32, -1: nowhere;
    no slot twice). positions and slots are paged_extend's."""
    if not _here(q, stream):
        return _elsewhere(qk_norm_rope_paged, q, locals())
    _need_dims(q, "q", 3, "[T, Hq, d]")
    _need_dims(k, "k", 3, "[T, Hkv, d]")
    dev, (T, Hq, d), Hkv = q.device, q.shape, k.shape[1]
    _need_heads(q, "q", (T, Hq, d), dev)
    _need_heads(k, "k", (T, Hkv, d), dev)
    _need_heads(v, "v", (T, Hkv, d), dev)
    if positions is None or slots is None:
        raise TypeError("positions and slots must be int32 tensors")
    w_bf16, rd, max_pos = _angles(q_weight, k_weight, cos, sin, positions, (T,), d, dev)
    _need_on(slots, "slots", torch.int32, (T,), dev)
    _need_dims(k_cache, "k_cache", 4, "[num_blocks, block_size, Hkv, d]")
    num_blocks, block_size = k_cache.shape[:2]
    _need_on(k_cache, "k_cache", torch.bfloat16, (num_blocks, block_size, Hkv, d), dev)
    _need_on(v_cache, "v_cache", torch.bfloat16, (num_blocks, block_size, Hkv, d), dev)
    _need_status(status, dev)
    q_out = _out_on(q_out, "q_out", torch.bfloat16, (T, Hq, d), dev, q)
    if T == 0:
        return q_out
    rc = _lib.lib().attn_qk_norm_rope_paged(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                            _strides(*q.stride()[:2], *k.stride()[:2], *v.stride()[:2]),
                                            _addr(q_weight), _addr(k_weight), w_bf16, cos.data_ptr(), sin.data_ptr(),
                                            positions.data_ptr(), slots.data_ptr(), q_out.data_ptr(),
                                            k_cache.data_ptr(), v_cache.data_ptr(), T, Hq, Hkv, d, num_blocks,
                                            block_size, rd, max_pos, float(eps), int(interleaved), _addr(status),
                                            _current(dev))
    _lib.check(rc, "attn_qk_norm_rope_paged")
    return q_out


def qk_norm_rope_backward_workspace_bytes(B: int, N: int, Hq: int, Hkv: int, d: int) -> int:
    n = int(_lib.lib().attn_qk_norm_rope_backward_workspace_bytes(B, N, Hq, Hkv, d))
    if n == 0:
        raise AttnError(_lib.ATTN_ERR_INVALID_ARG, "attn_qk_norm_rope_backward_workspace_bytes")
    return n


def qk_norm_rope_backward(q, k, q_weight, k_weight, cos, sin, d_q, d_k, d_v, positions=None, eps: float = 1e-6,
                          interleaved: bool = False, dq=None, dk=None, dv=None, workspace=None, status=None,
                          stream=None):
    """Gradients of qk_norm_rope() from those of its outputs, d_q [B, Hq, N, d],
    d_k and d_v [B, Hkv, N, d] (what prefill_backward returns): (dq, dk, dv,
    dq_weight, dk_weight), the weights' in fp32, or None without weights.

    dq [B, N, Hq, d], dk and dv [B, N, Hkv, d] come as views of one fused
    [B, N, Hq + 2 Hkv, d] gradient unless given (any strides with contiguous
    head rows). q, k: the forward's inputs.
    """
    if not _here(q, stream):
        return _elsewhere(qk_norm_rope_backward, q, locals())
    _need_dims(q, "q", 4, "[B, N, Hq, d]")
    _need_dims(k, "k", 4, "[B, N, Hkv, d]")
    dev, (B, N, Hq, d), Hkv, bf16 = q.device, q.shape, k.shape[2], torch.bfloat16
    _need_heads(q, "q", (B, N, Hq, d), dev)
    _need_heads(k, "k", (B, N, Hkv, d), dev)
    _need_on(d_q, "d_q", bf16, (B, Hq, N, d), dev)
    _need_on(d_k, "d_k", bf16, (B, Hkv, N, d), dev)
    _need_on(d_v, "d_v", bf16, (B, Hkv, N, d), dev)
    w_bf16, rd, max_pos = _angles(q_weight, k_weight, cos, sin, positions, (B, N), d, dev)
    _need_status(status, dev)
    if dq is None and dk is None and dv is None:
        heads = Hq + 2 * Hkv
        dq, dk, dv = torch.empty((B, N, heads, d), dtype=bf16, device=dev).split_with_sizes((Hq, Hkv, Hkv), 2)
        grad_strides = _strides(*(N * heads * d, heads * d, d) * 3)
    else:
        dq = torch.empty((B, N, Hq, d), dtype=bf16, device=dev) if dq is None else dq
        dk = torch.empty((B, N, Hkv, d), dtype=bf16, device=dev) if dk is None else dk
        dv = torch.empty((B, N, Hkv, d), dtype=bf16, device=dev) if dv is None else dv
        _need_heads_out(dq, "dq", (B, N, Hq, d), dev)
        _need_heads_out(dk, "dk", (B, N, Hkv, d), dev)
        _need_heads_out(dv, "dv", (B, N, Hkv, d), dev)
        grad_strides = _strides(*dq.stride()[:3], *dk.stride()[:3], *dv.stride()[:3])
    dwq = dwk = None
    if q_weight is not None:
        dwq, dwk = torch.empty(2 * d, dtype=torch.float32, device=dev).unsafe_split_with_sizes((d, d))
        if workspace is None:
            workspace = torch.empty(qk_norm_rope_backward_workspace_bytes(B, N, Hq, Hkv, d), dtype=torch.uint8,
                                    device=dev)
    _need_workspace(workspace, dev)
    rc = _lib.lib().attn_qk_norm_rope_backward(
        q.data_ptr(), k.data_ptr(), _strides(*q.stride()[:3], *k.stride()[:3]), _addr(q_weight), _addr(k_weight),
        w_bf16, cos.data_ptr(), sin.data_ptr(), _addr(positions), d_q.data_ptr(), d_k.data_ptr(), d_v.data_ptr(),
        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), grad_strides,
        _addr(dwq), _addr(dwk), B, N, Hq, Hkv, d, rd, max_pos, float(eps), int(interleaved), _addr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(), _addr(status), _current(dev))
    _lib.check(rc, "attn_qk_norm_rope_backward")
    return dq, dk, dv, dwq, dwk
