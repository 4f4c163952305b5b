"""The 8-bit shared KV cache over the libshkv C ABI.

``QuantizedKVPool`` is ``SharedKVPool`` with every (token, KV head) row of K
and V held as e4m3 codes and one power-of-two scale: about half the bytes a
decode step reads, and twice the tokens in the same memory.  Tokens are
quantised as they are appended, read back as bf16, and attended by the stacked
decode and by ragged causal chunks.
"""
from __future__ import annotations

import array
import contextlib
from typing import Dict, Optional

import numpy as np
import torch

from . import _native as N

_BF16, _F32, _U8 = torch.bfloat16, torch.float32, torch.uint8
_HERE = contextlib.nullcontext()
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


class _HostInts:
    """Host int32 array of a C call (a list, a numpy array or a CPU tensor of
    non-negative integers).  A decode step makes several of these per layer:
    no numpy on the way."""
    __slots__ = ("n", "total", "ptr", "_keep")

    def __init__(self, x, name: str):
        if not isinstance(x, (list, tuple)):
            if getattr(x, "ndim", 1) != 1:
                raise ValueError(f"{name} must be a one-dimensional list of integers")
            x = x.tolist() if hasattr(x, "tolist") else x
        try:
            x = list(x)
            a = array.array("i", x)
        except TypeError:
            raise ValueError(f"{name} must be a one-dimensional list of integers") from None
        except OverflowError:
            raise ValueError(f"{name} must lie in [0, 2**31)") from None
        if x and min(x) < 0:
            raise ValueError(f"{name} must lie in [0, 2**31)")
        self.n, self.total, self._keep = len(a), sum(x), a
        self.ptr = a.buffer_info()[0] if a else None


class QuantizedKVPool:
    """One paged 8-bit KV cache shared by N decoders.

    k_pages / v_pages: uint8 (e4m3 codes) [num_pages, num_kv_heads, page_size, head_dim]
    scales: uint8 (e8m0) [num_pages, num_kv_heads, 2, page_size], K's then V's
    block_table: int32 [max_batch, max_pages_per_seq], filled by the caller
    seq_lens: int32 [max_batch], owned by the pool after creation

    A row stands for ``code * 2**(scale - 127)``; the scale is the least power
    of two that brings the row's largest magnitude to at most 448.

    Every call runs on ``stream`` (the pool device's current stream if None),
    which must be ordered after the work that made its inputs.  A call on a
    named stream, or where a side stream is current, holds its tensors back:
    they may be dropped once it has returned, whichever stream they are of.  On
    the default stream, unnamed, tensors of other streams are the caller's to
    keep or record, as with torch's own operations.  The pool may be dropped at
    any time.  A captured call's tensors, and the pool, have to live as long as
    the graph.  The workspace of the attentions is one per stream; a call that is being captured into a
    CUDA graph takes one of its own from the graph's memory, so graphs share
    none.  ``workspace=`` names another, of ``workspace_bytes`` bytes (40 MB at
    head_dim 128) whose first ``workspace_zero_bytes`` are zero before its first
    use; pools of one shape, as the layers of a model have, can share one where
    their calls follow one another on a stream.
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
                given = _HostInts(initial_seq_lens, "initial_seq_lens")
                if given.n > max_batch:
                    raise ValueError("initial_seq_lens is longer than max_batch")
                init = np.zeros(max_batch, dtype=np.int32)
                init[: given.n] = given._keep
            cfg = N.shkv_q8_pool_config(
                num_pages=num_pages, page_size=page_size, num_kv_heads=num_kv_heads, head_dim=head_dim,
                max_batch=max_batch, max_pages_per_seq=max_pages_per_seq, k_pages=self.k_pages.data_ptr(),
                v_pages=self.v_pages.data_ptr(), scales=self.scales.data_ptr(),
                block_table=self.block_table.data_ptr(), seq_lens=self.seq_lens.data_ptr(),
                error_word=self.error_word.data_ptr(), initial_seq_lens=init.ctypes.data if init is not None else None)
            torch.cuda.synchronize(device)
            self.handle = N.shkv_q8_pool_create(cfg)
        self.workspace_bytes, self.workspace_zero_bytes = N.shkv_q8_workspace_size(self.handle)
        self._workspaces: Dict[int, torch.Tensor] = {}
        self._streams: Dict[int, torch.cuda.Stream] = {}

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
    def _on(self, stream: Optional[torch.cuda.Stream]):
        """(context that makes the stream and the pool's device current, raw stream)."""
        if stream is None:
            index = self.device.index
            if _raw_stream is not None and _current_device() == index:
                return _HERE, _raw_stream(index)
            stream = torch.cuda.current_stream(self.device)
        elif stream.device != self.device:
            raise ValueError(f"stream must be one of {self.device}")
        return torch.cuda.stream(stream), stream.cuda_stream

    def _used_on(self, raw: int, named: Optional[torch.cuda.Stream], *tensors: Optional[torch.Tensor]) -> None:
        """Keeps the memory of the pool, and of the tensors of a call whose
        stream is named or a side stream, from being handed out again before
        the current stream, ``raw``, is through with it: called before the
        kernels are enqueued, so that a call that fails half-way is covered.
        (Recording the tensors of a short call costs 2 to 4 us of 20.)"""
        stream = self._streams.get(raw)
        mine = raw == 0 and named is None
        if mine and stream is not None or torch.cuda.is_current_stream_capturing():
            return
        if stream is None:
            # the pool's own memory, once: from here on until it is freed
            stream = torch.cuda.current_stream(self.device)
            for t in (self.k_pages, self.v_pages, self.scales, self.block_table, self.seq_lens, self.error_word):
                t.record_stream(stream)
            self._streams[raw] = stream
        for t in () if mine else tensors:
            if t is not None:
                t.record_stream(stream)

    def _rows(self, t: torch.Tensor, heads: Optional[int], name: str) -> int:
        """Checks a [tokens, heads, head_dim] bf16 operand whose tokens may be strided; its stride in elements."""
        if t.dtype is not _BF16 or t.device != self.device:
            raise ValueError(f"{name} must be bfloat16 on {self.device}")
        shape = t.shape
        if len(shape) != 3 or shape[2] != self.head_dim or (heads is not None and shape[1] != heads):
            raise ValueError(f"{name} must be [tokens, {'heads' if heads is None else heads}, {self.head_dim}]")
        row = shape[1] * self.head_dim
        if t.is_contiguous():
            return row
        token, head, one = t.stride()
        if one != 1 or (shape[1] > 1 and head != self.head_dim) or token < row or token % 8:
            raise ValueError(f"{name}: a token's rows must be contiguous and tokens a multiple of 8 elements apart")
        return token

    def _out(self, t: Optional[torch.Tensor], shape, dtype, name: str) -> torch.Tensor:
        if t is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        if t.device != self.device or t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on {self.device}")
        return t

    def _workspace(self, given: Optional[torch.Tensor], stream: int) -> torch.Tensor:
        if given is not None:
            if given.device != self.device or given.dtype != _U8 or not given.is_contiguous():
                raise ValueError(f"workspace must be a contiguous uint8 tensor on {self.device}")
            return given
        if torch.cuda.is_current_stream_capturing():
            return self._new_workspace()
        ws = self._workspaces.get(stream)
        if ws is None:
            ws = self._workspaces[stream] = self._new_workspace()
        return ws

    def _new_workspace(self) -> torch.Tensor:
        ws = torch.empty(self.workspace_bytes, dtype=_U8, device=self.device)
        ws[: self.workspace_zero_bytes].zero_()
        return ws

    # -- lengths --------------------------------------------------------------
    def set_seq_lens(self, lens, stream=None):
        """Set the cached lengths of the first len(lens) requests (synchronises the stream)."""
        n = _HostInts(lens, "lens")
        ctx, s = self._on(stream)
        with ctx:
            N.shkv_q8_pool_set_seq_lens(self.handle, n.n, n.ptr, s)

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
        new = _HostInts(new_lens, "new_lens")
        first = _HostInts(start, "start") if start is not None else None
        if first is not None and first.n != new.n:
            raise ValueError("start and new_lens must have the same length")
        ks, vs = self._rows(k_new, self.num_kv_heads, "k_new"), self._rows(v_new, self.num_kv_heads, "v_new")
        if k_new.shape[0] != new.total or v_new.shape[0] != new.total:
            raise ValueError("k_new and v_new must hold sum(new_lens) tokens")
        ctx, s = self._on(stream)
        with ctx:
            self._used_on(s, stream, k_new, v_new)
            N.shkv_q8_append_kv(self.handle, new.n, first.ptr if first is not None else None, new.ptr,
                                k_new.data_ptr(), ks, v_new.data_ptr(), vs, s)

    def read_kv(self, start, lens, k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                stream=None):
        """Tokens start[b] .. start[b] + lens[b] - 1 of every request as bf16
        (K, V), each [sum(lens), num_kv_heads, head_dim]."""
        first, n = _HostInts(start, "start"), _HostInts(lens, "lens")
        if first.n != n.n:
            raise ValueError("start and lens must have the same length")
        shape = (n.total, self.num_kv_heads, self.head_dim)
        row = self.num_kv_heads * self.head_dim
        ctx, s = self._on(stream)
        with ctx:
            k, v = self._out(k_out, shape, _BF16, "k_out"), self._out(v_out, shape, _BF16, "v_out")
            self._used_on(s, stream, k_out, v_out)
            N.shkv_q8_read_kv(self.handle, n.n, first.ptr, n.ptr, k.data_ptr(), row, v.data_ptr(), row, s)
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
        ctx, s = self._on(stream)
        with ctx:
            o = self._out(out, q.shape, _BF16, "out")
            e = self._out(lse, (B, rows), _F32, "lse") if return_lse or lse is not None else None
            ws = self._workspace(workspace, s)
            self._used_on(s, stream, q, out, lse, workspace)
            N.shkv_q8_decode_attention(self.handle, B, n_models, rows // n_models, q.data_ptr(),
                                       D ** -0.5 if scale is None else float(scale), o.data_ptr(),
                                       e.data_ptr() if e is not None else None, ws.data_ptr(), ws.numel(), s)
        return (o, e) if e is not None else o

    def chunk_attention(self, q: torch.Tensor, new_lens, scale: Optional[float] = None,
                        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        return_lse: bool = False, workspace: Optional[torch.Tensor] = None, stream=None):
        """Causal attention of the new_lens[b] last tokens of every request,
        already appended: q bf16 [sum(new_lens), hq, head_dim], requests packed
        one after another (tokens may be strided).  New token i attends the
        cached prefix and the new tokens up to itself."""
        new = _HostInts(new_lens, "new_lens")
        qs = self._rows(q, None, "q")
        T, hq, D = q.shape
        if T != new.total:
            raise ValueError("q must hold sum(new_lens) tokens")
        ctx, s = self._on(stream)
        with ctx:
            o = self._out(out, (T, hq, D), _BF16, "out")
            e = self._out(lse, (T, hq), _F32, "lse") if return_lse or lse is not None else None
            if T:
                ws = self._workspace(workspace, s)
                self._used_on(s, stream, q, out, lse, workspace)
                N.shkv_q8_chunk_attention(self.handle, new.n, new.ptr, hq, q.data_ptr(), qs,
                                          D ** -0.5 if scale is None else float(scale), o.data_ptr(),
                                          e.data_ptr() if e is not None else None, ws.data_ptr(), ws.numel(), s)
        return (o, e) if e is not None else o

    def check_errors(self, stream=None) -> int:
        """Wait for the stream and return (then clear) the device error bits;
        those of calls on other streams are reported by this check or a later one."""
        ctx, s = self._on(stream)
        with ctx:
            return N.shkv_q8_check_errors(self.handle, s)
