"""Torch-side calls of the layers beside the gated delta rule.

Head norms with the position rotation, linear attention with a decay for each
head, and a paged KV cache held in 4 bits with the attention that reads it.
Every computation runs in libpace.so (include/pace.h documents the formulas);
this module checks tensors, allocates outputs and workspaces with torch, and
passes pointers.  ``stream`` is a ``torch.cuda.Stream`` or None for the
current stream of the tensors' device; outputs and workspaces that a call
allocates belong to that stream.  Nothing here waits, and every call can be
captured into a graph.  The calls are for inference: autograd does not see them.
"""
from __future__ import annotations

import functools
from typing import Optional, Tuple

import torch

from . import pace

_DTYPES = {torch.bfloat16: pace.PACE_DTYPE_BF16, torch.float32: pace.PACE_DTYPE_F32}
_NORMS = {"none": pace.PACE_NORM_NONE, "l2": pace.PACE_NORM_L2, "rms": pace.PACE_NORM_RMS}

# A decode step's kernels are shorter than a call's Python unless that is little:
# tensors are compared by device number, a check's details are worked out only
# for its message, and pointers go to the C entry points directly (norms of a
# small batch: 8.3 us a call, of which 2.6 are the launch and 2.3 the outputs'
# allocation; 9.4 us through the binding's general wrappers).
_LIB = pace.LIB


def _ptr(x: Optional[torch.Tensor]) -> Optional[int]:
    return None if x is None else x.data_ptr()


def _dtype(x: torch.Tensor, name: str) -> int:
    code = _DTYPES.get(x.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32, not {x.dtype}")
    return code


def _refuse(x, name: str, dtype, shape, device: int) -> None:
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not x.is_cuda:
        raise ValueError(f"{name} must be on a GPU, not on {x.device}")
    if x.get_device() != device:
        raise ValueError(f"{name} is on {x.device}, the first tensor on cuda:{device}")
    if x.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {x.dtype}")
    if x.shape != shape:
        raise ValueError(f"{name} must have shape {shape}, not {tuple(x.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _check(x, name: str, dtype, shape: tuple, device: int, dense: bool = True) -> None:
    """x is a tensor of this type, shape and device, without gaps."""
    try:
        if (x.get_device() == device and x.dtype is dtype and x.shape == shape
                and (not dense or x.is_contiguous())):
            return
    except AttributeError:
        pass
    _refuse(x, name, dtype, shape, device)


def _first(x, name: str, dims: int) -> int:
    """Number of the device that x, a tensor of so many dimensions, is on."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    device = x.get_device()
    if device < 0:
        raise ValueError(f"{name} must be on a GPU, not on {x.device}")
    if x.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, not {x.dim()}")
    return device


def _elsewhere(device: int, stream):
    """Context that makes `device` current, and `stream` its current stream;
    None where that is so already."""
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            raise TypeError("stream must be a torch.cuda.Stream or None")
        if stream.device.index != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{device}")
        return torch.cuda.stream(stream)
    if _current_device() != device:
        return torch.cuda.device(device)
    return None


# the current device's number, and a device's current stream's handle without
# the Stream object around it (tensors on the device exist: it is initialised)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)


def _workspace(given, need: int, like: torch.Tensor) -> Tuple[torch.Tensor, int]:
    if given is None:
        return like.new_empty(need, dtype=torch.uint8), need
    if not isinstance(given, torch.Tensor) or given.dtype != torch.uint8 or not given.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 tensor")
    if given.get_device() != like.get_device():
        raise ValueError(f"workspace is on {given.device}, the tensors on {like.device}")
    return given, given.numel()


# ---- head norms with rotation ----------------------------------------------

def _heads(x, name: str, heads: int, d: int) -> int:
    """Row stride of x [tokens, heads, d], whose heads are dense."""
    if x.is_contiguous():
        return heads * d
    row, head, channel = x.stride()
    if (d > 1 and channel != 1) or (heads > 1 and head != d):
        raise ValueError(f"{name}: the heads of a row must be dense")
    if x.shape[0] <= 1:
        return heads * d
    if row < heads * d:
        raise ValueError(f"{name}: rows overlap")
    return row


def qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor] = None, norm: str = "l2",
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, q_scale: float = 1.0, pos: Optional[torch.Tensor] = None,
                 inv_freq: Optional[torch.Tensor] = None, adjacent: bool = False,
                 q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Normalise (and rotate) the heads of q [tokens, heads_q, d] and k [tokens,
    heads_k, d]; rows may be parts of wider ones (a packed projection).  The
    first 2 * len(inv_freq) channels are rotated by pos[t] * inv_freq[i], in
    halves, or in adjacent pairs.  Returns dense (q_out, k_out); an output may
    be its dense input.  See pace_qk_norm_rope."""
    device = _first(q, "q", 3)
    code = _dtype(q, "q")
    tokens, hq, d = q.shape
    q_stride = _heads(q, "q", hq, d)
    hk = k_stride = 0
    if k is not None:
        _first(k, "k", 3)
        hk = k.shape[1]
        _check(k, "k", q.dtype, (tokens, hk, d), device, dense=False)
        k_stride = _heads(k, "k", hk, d)
    if norm not in _NORMS:
        raise ValueError(f"norm must be one of {sorted(_NORMS)}")
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _check(w, name, torch.float32, (d,), device)
    rot = 0
    if inv_freq is not None:
        _check(inv_freq, "inv_freq", torch.float32, (inv_freq.numel(),), device)
        rot = 2 * inv_freq.numel()
        if rot:
            _check(pos, "pos", torch.int32, (tokens,), device)
    cfg = pace.pace_norm_config(tokens, hq, hk, d, code, _NORMS[norm], eps, q_scale, rot,
                                pace.PACE_ROT_ADJACENT if adjacent else pace.PACE_ROT_HALVES,
                                q_stride, k_stride)
    if q_out is not None:
        _check(q_out, "q_out", q.dtype, (tokens, hq, d), device)
    if k_out is not None:
        if k is None:
            raise ValueError("k_out needs k")
        _check(k_out, "k_out", q.dtype, (tokens, hk, d), device)

    context = _elsewhere(device, stream)
    if context is not None:
        with context:
            return qk_norm_rope(q, k, norm, q_weight, k_weight, eps, q_scale, pos, inv_freq, adjacent,
                                q_out, k_out)
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
    if k is not None and k_out is None:
        k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
    if tokens:
        pace._check(_LIB.pace_qk_norm_rope(
            cfg, q.data_ptr(), _ptr(k), _ptr(q_weight), _ptr(k_weight), _ptr(pos) if rot else None,
            _ptr(inv_freq) if rot else None, q_out.data_ptr(), _ptr(k_out), _raw_stream(device)))
    return q_out, k_out


# ---- linear attention with a decay for each head ---------------------------

# bytes by sizes alone
_linear_need = functools.lru_cache(maxsize=256)(pace.pace_linear_attn_workspace)


def linear_attention_workspace(q: torch.Tensor, v: torch.Tensor) -> Optional[torch.Tensor]:
    """A workspace for linear_attention calls of these shapes (None if none is needed)."""
    t, b, h, dk = q.shape
    need = pace.pace_linear_attn_workspace(b, h, dk, v.shape[-1], t, _dtype(q, "q"))
    return torch.empty(need, dtype=torch.uint8, device=q.device) if need else None


def linear_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, decay: torch.Tensor,
                     state: Optional[torch.Tensor] = None, lens: Optional[torch.Tensor] = None,
                     scale: float = 1.0, out: Optional[torch.Tensor] = None,
                     state_out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None,
                     stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """o_t = scale * M_t^T q_t with M_t = decay_h M_{t-1} + k_t v_t^T over the
    tokens of q, k [T, B, H, d_k] and v [T, B, H, d_v], from the float32 state
    [B, H, d_k, d_v] (None: zeros).  lens int32 [B] gives sequences of different
    lengths; rows of `out` behind them are not written (undefined in an `out`
    that the call allocates).  Returns (out, state_out), float32; state_out may
    be state.  See pace_linear_attn."""
    device = _first(q, "q", 4)
    code = _dtype(q, "q")
    t, b, h, dk = q.shape
    _first(v, "v", 4)
    dv = v.shape[3]
    _check(q, "q", q.dtype, (t, b, h, dk), device)
    _check(k, "k", q.dtype, (t, b, h, dk), device)
    _check(v, "v", q.dtype, (t, b, h, dv), device)
    _check(decay, "decay", torch.float32, (h,), device)
    if state is not None:
        _check(state, "state", torch.float32, (b, h, dk, dv), device)
    if lens is not None:
        _check(lens, "lens", torch.int32, (b,), device)
    if out is not None:
        _check(out, "out", torch.float32, (t, b, h, dv), device)
    if state_out is not None:
        _check(state_out, "state_out", torch.float32, (b, h, dk, dv), device)
    need = _linear_need(b, h, dk, dv, t, code)

    context = _elsewhere(device, stream)
    if context is not None:
        with context:
            return linear_attention(q, k, v, decay, state, lens, scale, out, state_out, workspace)
    if out is None:
        out = v.new_empty((t, b, h, dv), dtype=torch.float32)
    if state_out is None:
        state_out = q.new_empty((b, h, dk, dv), dtype=torch.float32) if state is None else torch.empty_like(state)
    ws, n = _workspace(workspace, need, q) if need else (None, 0)
    pace._check(_LIB.pace_linear_attn(
        b, h, dk, dv, t, code, q.data_ptr(), k.data_ptr(), v.data_ptr(), decay.data_ptr(), _ptr(lens), scale,
        _ptr(state), state_out.data_ptr(), out.data_ptr(), _ptr(ws), n, _raw_stream(device)))
    return out, state_out


# ---- 4-bit paged KV cache --------------------------------------------------

@functools.lru_cache(maxsize=256)
def _attention_need(batch, heads_q, heads_kv, d, page_tokens, pages, columns, code, t) -> int:
    """Bytes by sizes alone."""
    return pace.pace_kv4_attention_workspace(
        pace.pace_kv4_config(batch, heads_q, heads_kv, d, page_tokens, pages, columns, code), t)


class Kv4Cache:
    """The pool of a paged KV cache in 4 bits: `pages` pages of `page_tokens`
    tokens for `heads_kv` heads of d channels.  Page tables (int32 [B, columns],
    page numbers, anything outside 0..pages - 1 for none) belong to the caller
    and are given to each call."""

    def __init__(self, pages: int, heads_kv: int, d: int, page_tokens: int = 64, device="cuda"):
        self.pages, self.heads_kv, self.d, self.page_tokens = pages, heads_kv, d, page_tokens
        cfg = pace.pace_kv4_config(0, 0, heads_kv, d, page_tokens, pages, 0, 0)
        self.pool = torch.empty(pace.pace_kv4_pool_bytes(cfg), dtype=torch.uint8, device=device)

    @property
    def nbytes(self) -> int:
        return self.pool.numel()

    def _config(self, table, batch: int, heads_q: int, code: int) -> Tuple[pace.pace_kv4_config, int]:
        device = _first(table, "table", 2)
        if device != self.pool.get_device():
            raise ValueError(f"table is on {table.device}, the cache on {self.pool.device}")
        columns = table.shape[1]
        _check(table, "table", torch.int32, (batch, columns), device)
        return pace.pace_kv4_config(batch, heads_q, self.heads_kv, self.d, self.page_tokens,
                                    self.pages, columns, code), device

    def append(self, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, start: torch.Tensor,
               count: Optional[torch.Tensor] = None, stream=None) -> None:
        """Quantize k, v [T, B, heads_kv, d] into positions start[b] + t of the
        cache, for t < count[b] (None: all T).  See pace_kv4_append."""
        _first(k, "k", 4)
        t, b = k.shape[0], k.shape[1]
        cfg, device = self._config(table, b, 0, _dtype(k, "k"))
        shape = (t, b, self.heads_kv, self.d)
        _check(k, "k", k.dtype, shape, device)
        _check(v, "v", k.dtype, shape, device)
        _check(start, "start", torch.int32, (b,), device)
        if count is not None:
            _check(count, "count", torch.int32, (b,), device)

        context = _elsewhere(device, stream)
        if context is not None:
            with context:
                return self.append(k, v, table, start, count)
        pace._check(_LIB.pace_kv4_append(
            cfg, self.pool.data_ptr(), table.data_ptr(), start.data_ptr(), _ptr(count), t, k.data_ptr(),
            v.data_ptr(), _raw_stream(device)))

    def read(self, table: torch.Tensor, start: torch.Tensor, n_tok: int,
             count: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """float32 (k, v) [n_tok, B, heads_kv, d]: what the cache holds at
        positions start[b] + t (zeros for t >= count[b] and without a page)."""
        _first(table, "table", 2)
        b = table.shape[0]
        cfg, device = self._config(table, b, 0, pace.PACE_DTYPE_F32)
        _check(start, "start", torch.int32, (b,), device)
        if count is not None:
            _check(count, "count", torch.int32, (b,), device)
        if n_tok < 1:
            raise ValueError("n_tok must be >= 1")

        context = _elsewhere(device, stream)
        if context is not None:
            with context:
                return self.read(table, start, n_tok, count)
        k = self.pool.new_empty((n_tok, b, self.heads_kv, self.d), dtype=torch.float32)
        v = torch.empty_like(k)
        pace._check(_LIB.pace_kv4_read(
            cfg, self.pool.data_ptr(), table.data_ptr(), start.data_ptr(), _ptr(count), n_tok, k.data_ptr(),
            v.data_ptr(), _raw_stream(device)))
        return k, v

    def attention_workspace(self, q: torch.Tensor, table: torch.Tensor) -> Optional[torch.Tensor]:
        """A workspace for attention calls with queries and tables of these shapes."""
        cfg, _ = self._config(table, q.shape[1], q.shape[2], _dtype(q, "q"))
        need = pace.pace_kv4_attention_workspace(cfg, q.shape[0])
        return torch.empty(need, dtype=torch.uint8, device=q.device) if need else None

    def attention(self, q: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
                  count: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                  window: int = 0, sinks: int = 0, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Causal softmax attention of q [T, B, heads_q, d] over the lens[b]
        cached tokens of each sequence, the last count[b] (None: T) of which
        are the queries' own; window and sinks as in pace_kv4_attention.
        scale defaults to d ** -0.5.  Returns out, of q's type (rows
        t >= count[b] are not written)."""
        _first(q, "q", 4)
        t, b, hq, d = q.shape
        cfg, device = self._config(table, b, hq, _dtype(q, "q"))
        _check(q, "q", q.dtype, (t, b, hq, self.d), device)
        _check(lens, "lens", torch.int32, (b,), device)
        if count is not None:
            _check(count, "count", torch.int32, (b,), device)
        if out is not None:
            _check(out, "out", q.dtype, (t, b, hq, d), device)
        context = _elsewhere(device, stream)
        if context is not None:
            with context:
                return self.attention(q, table, lens, count, scale, window, sinks, out, workspace)
        need = _attention_need(b, hq, self.heads_kv, self.d, self.page_tokens, self.pages, table.shape[1],
                               cfg.in_dtype, t)
        if out is None:
            out = torch.empty_like(q)
        ws, n = _workspace(workspace, need, q) if need else (None, 0)
        pace._check(_LIB.pace_kv4_attention(
            cfg, self.pool.data_ptr(), table.data_ptr(), lens.data_ptr(), _ptr(count), t, q.data_ptr(),
            d ** -0.5 if scale is None else scale, window, sinks, out.data_ptr(), _ptr(ws), n,
            _raw_stream(device)))
        return out
