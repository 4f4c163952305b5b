"""The 8-bit shared KV cache over the libshkv C ABI.

``QuantizedKVPool`` is ``SharedKVPool`` with every (token, KV head) row of K
and V held as e4m3 codes and one power-of-two scale: about half the bytes a
decode step reads, and twice the tokens in the same memory.  Tokens are
quantised as they are appended, read back as bf16, and attended by the stacked
decode and by ragged causal chunks.
"""
from __future__ import annotations

from typing import Dict, Optional

import numpy as np
import torch

from . import _native as N

_BF16, _F32, _U8 = torch.bfloat16, torch.float32, torch.uint8


def _host_i32(x, name: str) -> np.ndarray:
    a = np.asarray(x)
    if a.ndim != 1 or (a.size and a.dtype.kind not in "iu"):
        raise ValueError(f"{name} must be a one-dimensional list of integers")
    if a.size and (a.min() < 0 or a.max() > 2 ** 31 - 1):
        raise ValueError(f"{name} must lie in [0, 2**31)")
    return np.ascontiguousarray(a, dtype=np.int32)


class QuantizedKVPool:
    """One paged 8-bit KV cache shared by N decoders.

    k_pages / v_pages: uint8 (e4m3 codes) [num_pages, num_kv_heads, page_size, head_dim]
    scales: uint8 (e8m0) [num_pages, num_kv_heads, 2, page_size], K's then V's
    block_table: int32 [max_batch, max_pages_per_seq], filled by the caller
    seq_lens: int32 [max_batch], owned by the pool after creation

    A row stands for ``code * 2**(scale - 127)``; the scale is the least power
    of two that brings the row's largest magnitude to at most 448.

    Every call runs on ``stream`` (the pool device's current stream if None),
    which must be ordered after the work that made its inputs.  The workspace
    of the attentions is one per stream; a call that is being captured into a
    CUDA graph takes one of its own from the graph's memory, so graphs share
    none.  ``workspace=`` names another (zeroed before its first use, see
    ``workspace_bytes``).
    """

    def __init__(self, num_pages: int, page_size: int, num_kv_heads: int, head_dim: int, max_batch: int,
                 max_pages_per_seq: int, device=None, k_pages: Optional[torch.Tensor] = None,
                 v_pages: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                 initial_seq_lens=None):
        N.load()
        if device is None:
            device = k_pages.device if k_pages is not None else "cuda"
        device = torch.device(device)
        if device.type != "cuda":
            raise ValueError("the pool lives on a CUDA device")
        if device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        self.device = device
        self.num_pages, self.page_size = num_pages, page_size
        self.num_kv_heads, self.head_dim = num_kv_heads, head_dim
        self.max_batch, self.max_pages_per_seq = max_batch, max_pages_per_seq
        shape = (num_pages, num_kv_heads, page_size, head_dim)
        with torch.cuda.device(device):
            self.k_pages = self._pages(k_pages, shape, "k_pages")
            self.v_pages = self._pages(v_pages, shape, "v_pages")
            self.scales = self._pages(scales, (num_pages, num_kv_heads, 2, page_size), "scales")
            self.block_table = torch.full((max_batch, max_pages_per_seq), -1, dtype=torch.int32, device=device)
            self.seq_lens = torch.zeros(max_batch, dtype=torch.int32, device=device)
            self.error_word = torch.zeros(1, dtype=torch.int32, device=device)
            init = None
            if initial_seq_lens is not None:
                given = _host_i32(initial_seq_lens, "initial_seq_lens")
                if len(given) > max_batch:
                    raise ValueError("initial_seq_lens is longer than max_batch")
                init = np.zeros(max_batch, dtype=np.int32)
                init[: len(given)] = given
            cfg = N.shkv_q8_pool_config(
                num_pages=num_pages, page_size=page_size, num_kv_heads=num_kv_heads, head_dim=head_dim,
                max_batch=max_batch, max_pages_per_seq=max_pages_per_seq, k_pages=self.k_pages.data_ptr(),
                v_pages=self.v_pages.data_ptr(), scales=self.scales.data_ptr(),
                block_table=self.block_table.data_ptr(), seq_lens=self.seq_lens.data_ptr(),
                error_word=self.error_word.data_ptr(), initial_seq_lens=init.ctypes.data if init is not None else None)
            torch.cuda.synchronize(device)
            self.handle = N.shkv_q8_pool_create(cfg)
        self.workspace_bytes = N.shkv_q8_workspace_size(self.handle)
        self._workspaces: Dict[int, torch.Tensor] = {}

    def _pages(self, t: Optional[torch.Tensor], shape, name: str) -> torch.Tensor:
        if t is None:
            return torch.zeros(shape, dtype=_U8, device=self.device)
        if t.device != self.device or t.dtype != _U8 or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous uint8 tensor {list(shape)} on {self.device}")
        return t

    # -- lifecycle ----------------------------------------------------------
    def close(self):
        if getattr(self, "handle", None):
            N.shkv_q8_pool_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- arguments ------------------------------------------------------------
    def _stream(self, stream: Optional[torch.cuda.Stream]) -> torch.cuda.Stream:
        s = stream if stream is not None else torch.cuda.current_stream(self.device)
        if s.device != self.device:
            raise ValueError(f"stream must be one of {self.device}")
        return s

    def _rows(self, t: torch.Tensor, heads: Optional[int], name: str) -> int:
        """Checks a [tokens, heads, head_dim] bf16 operand whose tokens may be strided; its stride in elements."""
        if t.device != self.device or t.dtype != _BF16:
            raise ValueError(f"{name} must be bfloat16 on {self.device}")
        if t.dim() != 3 or t.shape[2] != self.head_dim or (heads is not None and t.shape[1] != heads):
            raise ValueError(f"{name} must be [tokens, {'heads' if heads is None else heads}, {self.head_dim}]")
        row = t.shape[1] * self.head_dim
        if t.shape[0] <= 1 and t.is_contiguous():
            return row
        if t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != self.head_dim) or t.stride(0) < row or t.stride(0) % 8:
            raise ValueError(f"{name}: a token's rows must be contiguous and tokens a multiple of 8 elements apart")
        return t.stride(0)

    def _out(self, t: Optional[torch.Tensor], shape, dtype, name: str) -> torch.Tensor:
        if t is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        if t.device != self.device or t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on {self.device}")
        return t

    def _workspace(self, given: Optional[torch.Tensor], stream: torch.cuda.Stream) -> torch.Tensor:
        if given is not None:
            if given.device != self.device or given.dtype != _U8 or not given.is_contiguous():
                raise ValueError(f"workspace must be a contiguous uint8 tensor on {self.device}")
            return given
        if torch.cuda.is_current_stream_capturing():
            return torch.zeros(self.workspace_bytes, dtype=_U8, device=self.device)
        ws = self._workspaces.get(stream.cuda_stream)
        if ws is None:
            ws = self._workspaces[stream.cuda_stream] = torch.zeros(self.workspace_bytes, dtype=_U8,
                                                                    device=self.device)
        return ws

    # -- lengths --------------------------------------------------------------
    def set_seq_lens(self, lens, stream=None):
        """Set the cached lengths of the first len(lens) requests (synchronises the stream)."""
        arr = _host_i32(lens, "lens")
        s = self._stream(stream)
        with torch.cuda.stream(s):
            N.shkv_q8_pool_set_seq_lens(self.handle, len(arr), arr.ctypes.data, s.cuda_stream)

    def host_seq_lens(self, batch: Optional[int] = None) -> np.ndarray:
        out = np.zeros(self.max_batch if batch is None else batch, dtype=np.int32)
        N.shkv_q8_pool_get_seq_lens(self.handle, len(out), out.ctypes.data)
        return out

    # -- the path -------------------------------------------------------------
    def append_kv(self, k_new: torch.Tensor, v_new: torch.Tensor, new_lens, start=None, stream=None) -> None:
        """Quantise and append: request b takes the next new_lens[b] tokens of
        k_new / v_new (bf16 [sum(new_lens), num_kv_heads, head_dim], tokens may
        be strided).  ``start`` writes from given positions on instead of the
        current lengths (dropping what lies behind them)."""
        new = _host_i32(new_lens, "new_lens")
        first = _host_i32(start, "start") if start is not None else None
        if first is not None and len(first) != len(new):
            raise ValueError("start and new_lens must have the same length")
        ks, vs = self._rows(k_new, self.num_kv_heads, "k_new"), self._rows(v_new, self.num_kv_heads, "v_new")
        total = int(new.sum(dtype=np.int64))
        if k_new.shape[0] != total or v_new.shape[0] != total:
            raise ValueError("k_new and v_new must hold sum(new_lens) tokens")
        s = self._stream(stream)
        with torch.cuda.stream(s):
            N.shkv_q8_append_kv(self.handle, len(new), first.ctypes.data if first is not None else None,
                                new.ctypes.data, k_new.data_ptr(), ks, v_new.data_ptr(), vs, s.cuda_stream)

    def read_kv(self, start, lens, k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                stream=None):
        """Tokens start[b] .. start[b] + lens[b] - 1 of every request as bf16
        (K, V), each [sum(lens), num_kv_heads, head_dim]."""
        first, n = _host_i32(start, "start"), _host_i32(lens, "lens")
        if len(first) != len(n):
            raise ValueError("start and lens must have the same length")
        shape = (int(n.sum(dtype=np.int64)), self.num_kv_heads, self.head_dim)
        s = self._stream(stream)
        with torch.cuda.stream(s):
            k, v = self._out(k_out, shape, _BF16, "k_out"), self._out(v_out, shape, _BF16, "v_out")
            row = self.num_kv_heads * self.head_dim
            N.shkv_q8_read_kv(self.handle, len(n), first.ctypes.data, n.ctypes.data, k.data_ptr(), row, v.data_ptr(),
                              row, s.cuda_stream)
        return k, v

    def decode_attention(self, q: torch.Tensor, n_models: int, scale: Optional[float] = None,
                         out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                         return_lse: bool = False, workspace: Optional[torch.Tensor] = None, stream=None):
        """Stacked decode attention, as ``SharedKVPool.decode_attention``:
        q bf16 [B, n_models * hq, head_dim], model-major.  A request of length
        0 gives zeros and an lse of -inf."""
        if q.device != self.device or q.dtype != _BF16 or q.dim() != 3 or not q.is_contiguous():
            raise ValueError(f"q must be a contiguous bfloat16 tensor [B, n_models * hq, head_dim] on {self.device}")
        B, rows, D = q.shape
        if n_models < 1 or rows % n_models or D != self.head_dim:
            raise ValueError("q must be [B, n_models * hq, head_dim]")
        s = self._stream(stream)
        with torch.cuda.stream(s):
            o = self._out(out, q.shape, _BF16, "out")
            e = self._out(lse, (B, rows), _F32, "lse") if return_lse or lse is not None else None
            ws = self._workspace(workspace, s)
            N.shkv_q8_decode_attention(self.handle, B, n_models, rows // n_models, q.data_ptr(),
                                       D ** -0.5 if scale is None else float(scale), o.data_ptr(),
                                       e.data_ptr() if e is not None else None, ws.data_ptr(), ws.numel(),
                                       s.cuda_stream)
        return (o, e) if e is not None else o

    def chunk_attention(self, q: torch.Tensor, new_lens, scale: Optional[float] = None,
                        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        return_lse: bool = False, workspace: Optional[torch.Tensor] = None, stream=None):
        """Causal attention of the new_lens[b] last tokens of every request,
        already appended: q bf16 [sum(new_lens), hq, head_dim], requests packed
        one after another (tokens may be strided).  New token i attends the
        cached prefix and the new tokens up to itself."""
        new = _host_i32(new_lens, "new_lens")
        qs = self._rows(q, None, "q")
        T, hq, D = q.shape
        if T != int(new.sum(dtype=np.int64)):
            raise ValueError("q must hold sum(new_lens) tokens")
        s = self._stream(stream)
        with torch.cuda.stream(s):
            o = self._out(out, (T, hq, D), _BF16, "out")
            e = self._out(lse, (T, hq), _F32, "lse") if return_lse or lse is not None else None
            if T:
                ws = self._workspace(workspace, s)
                N.shkv_q8_chunk_attention(self.handle, len(new), new.ctypes.data, hq, q.data_ptr(), qs,
                                          D ** -0.5 if scale is None else float(scale), o.data_ptr(),
                                          e.data_ptr() if e is not None else None, ws.data_ptr(), ws.numel(),
                                          s.cuda_stream)
        return (o, e) if e is not None else o

    def check_errors(self, stream=None) -> int:
        """Synchronize and return (then clear) the device error bits."""
        s = self._stream(stream)
        with torch.cuda.stream(s):
            return N.shkv_q8_check_errors(self.handle, s.cuda_stream)
