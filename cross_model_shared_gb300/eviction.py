"""Eviction from the shared KV cache by accumulated attention weight.

``SharedKVPool`` has these calls.  ``decode_mass`` and ``prefill_mass`` add the
softmax weights that a decode step's or a chunk's rows gave every cached token
to the token's mass, ``select_tokens`` names every KV head's tokens of most
mass, and ``evict_tokens`` moves them into new pages.
"""
from __future__ import annotations

import contextlib
from typing import Dict, Optional

import torch

from . import _native as N
from .q8 import _HostInts, _current_device, _raw_stream

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_HERE = contextlib.nullcontext()


class EvictionCalls:
    """Masses are fp32 [B, num_kv_heads, T], T at least the longest request's
    length, the last dimension contiguous and the others of any stride.  A
    request's new tokens start from the masses that the tensor holds at their
    positions: zeros, as a rule.

    Every call runs on ``stream`` (the pool device's current stream if None),
    which must be ordered after the work that made its inputs.  A call on a
    named stream, or where a side stream is current, holds its tensors back:
    they may be dropped once it has returned.  A captured call's tensors, and
    the pool, have to live as long as the graph, which replays with the lengths
    of the capture.  Scratch memory is the pool's, one per stream; a captured call
    takes its own from the graph's memory.
    """

    # -- arguments ------------------------------------------------------------
    def _enter(self, stream: Optional[torch.cuda.Stream]):
        """(context that makes the stream and the pool's device current, raw stream)."""
        if stream is None:
            index = self.k_pages.device.index
            if _raw_stream is not None and _current_device() == index:
                return _HERE, _raw_stream(index)
            stream = torch.cuda.current_stream(self.k_pages.device)
        elif stream.device != self.k_pages.device:
            raise ValueError(f"stream must be one of {self.k_pages.device}")
        return torch.cuda.stream(stream), int(stream.cuda_stream)

    def _hold(self, raw: int, named: Optional[torch.cuda.Stream], *tensors: Optional[torch.Tensor]) -> None:
        """Keeps the memory of the pool, and of the tensors of a call whose
        stream is named or a side stream, from being handed out again before
        the current stream, ``raw``, is through with it: before the kernels are
        enqueued."""
        held: Dict[int, torch.cuda.Stream] = self.__dict__.setdefault("_held_for", {})
        stream = held.get(raw)
        mine = raw == 0 and named is None
        if mine and stream is not None or torch.cuda.is_current_stream_capturing():
            return
        if stream is None:
            # the pool's own memory, once: from here on until it is freed
            stream = torch.cuda.current_stream(self.k_pages.device)
            for t in (self.k_pages, self.v_pages, self.block_table, self.seq_lens, self.error_word):
                t.record_stream(stream)
            held[raw] = stream
        for t in () if mine else tensors:
            if t is not None:
                t.record_stream(stream)

    def _mass_of(self, t: torch.Tensor, batch: int, name: str) -> N.shkv_mass:
        if t.dtype is not _F32 or t.device != self.k_pages.device:
            raise ValueError(f"{name} must be float32 on {self.k_pages.device}")
        shape = t.shape
        if len(shape) != 3 or shape[0] < batch or shape[1] != self.num_kv_heads:
            raise ValueError(f"{name} must be [B, {self.num_kv_heads}, T] of at least {batch} requests")
        request, head, token = t.stride()
        if token != 1 and shape[2] > 1:
            raise ValueError(f"{name}: a row's masses must be contiguous")
        return N.shkv_mass(t.data_ptr(), request, head, shape[2])

    def _mass_workspace(self, raw: int) -> torch.Tensor:
        """Scratch of the calls on a stream, or of a captured call alone (from
        the graph's memory, so graphs share none)."""
        ws: Dict[int, torch.Tensor] = self.__dict__.setdefault("_mass_workspaces", {})
        t = ws.get(raw)
        capturing = torch.cuda.is_current_stream_capturing()
        if t is None or capturing:
            t = torch.empty(N.shkv_prefill_mass_workspace_size(self.handle), dtype=torch.uint8,
                            device=self.k_pages.device)
            if not capturing:
                ws[raw] = t
        return t

    def _masses(self, mass: Optional[torch.Tensor], out: Optional[torch.Tensor], batch: int):
        """Masses read (or None) and written, for the C call, and the tensor written."""
        m = self._mass_of(mass, batch, "mass") if mass is not None else None
        if out is not None:
            return m, self._mass_of(out, batch, "out"), out
        if mass is None:
            if batch > self.max_batch:
                raise ValueError(f"at most {self.max_batch} requests")
            longest = int(self.host_seq_lens(batch).max(initial=0))
            mass = torch.zeros((batch, self.num_kv_heads, longest), dtype=_F32, device=self.k_pages.device)
            return None, self._mass_of(mass, batch, "out"), mass
        return m, m, mass

    # -- the path -------------------------------------------------------------
    def decode_mass(self, q: torch.Tensor, lse: torch.Tensor, n_models: int, mass: Optional[torch.Tensor],
                    decay: float = 1.0, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
        """``out[b, g, t] = decay * mass[b, g, t] +`` the sum of the softmax
        weights that the stacked rows of KV head g gave cached token t.

        q: bf16 [B, n_models * hq, head_dim] and lse: fp32 [B, n_models * hq],
        of the same ``decode_attention`` (also ``DecoderTails``').  ``out`` is
        ``mass`` itself if None; with ``mass`` None it holds the sums alone.
        Positions behind a request's last token are left as they are."""
        if q.dtype is not _BF16 or q.device != self.k_pages.device or q.dim() != 3 or not q.is_contiguous():
            raise ValueError(f"q must be a contiguous bfloat16 tensor [B, n_models * hq, head_dim] on {self.k_pages.device}")
        B, rows, D = q.shape
        if n_models < 1 or rows % n_models or D != self.head_dim:
            raise ValueError("q must be [B, n_models * hq, head_dim]")
        if lse.dtype is not _F32 or lse.device != q.device or tuple(lse.shape) != (B, rows) or not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous float32 tensor {[B, rows]} on {q.device}")
        ctx, s = self._enter(stream)
        with ctx:
            m, o, result = self._masses(mass, out, B)
            self._hold(s, stream, q, lse, mass, out)
            N.shkv_decode_mass(self.handle, B, n_models, rows // n_models, q.data_ptr(),
                               D ** -0.5 if scale is None else float(scale), lse.data_ptr(), float(decay), m, o, s)
        return result

    def prefill_mass(self, q: torch.Tensor, lse: torch.Tensor, mass: Optional[torch.Tensor], decay: float = 1.0,
                     scale: Optional[float] = None, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """The same for the last n_new tokens of every request, of which new
        token i weighs the tokens up to itself: q bf16 [B, n_new, hq, head_dim]
        and lse fp32 [B, n_new, hq] of the same ``prefill_attention``.  Slices
        of both (``q[:, -64:]``) make the chunk's last tokens a window of
        voters: a token's own rows have to be contiguous, tokens a multiple of
        head_dim elements apart and requests a multiple of the tokens' stride
        (of head_dim, for one token each)."""
        shape, stride = q.shape, q.stride()
        if q.dtype is not _BF16 or q.device != self.k_pages.device or len(shape) != 4 or shape[3] != self.head_dim:
            raise ValueError(f"q must be bfloat16 [B, n_new, hq, head_dim] on {self.k_pages.device}")
        B, T, H, D = shape
        if stride[3] != 1 or (stride[2] != D and H > 1):
            raise ValueError("q: a token's rows must be contiguous")
        if lse.dtype is not _F32 or lse.device != q.device or lse.shape != shape[:3]:
            raise ValueError(f"lse must be float32 {[B, T, H]} on {q.device}")
        ls = lse.stride()
        if ls[2] != 1 and H > 1:
            raise ValueError("lse: a token's values must be contiguous")
        ctx, s = self._enter(stream)
        with ctx:
            m, o, result = self._masses(mass, out, B)
            ws = self._mass_workspace(s)
            self._hold(s, stream, q, lse, mass, out)
            N.shkv_prefill_mass(self.handle, B, T, H, q.data_ptr(), stride[0], stride[1],
                                D ** -0.5 if scale is None else float(scale), lse.data_ptr(), ls[0], ls[1], float(decay),
                                m, o, ws.data_ptr(), ws.numel(), s)
        return result

    def select_tokens(self, mass: torch.Tensor, keep, sink: int = 0, recent: int = 0,
                      out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Positions of the ``keep[b]`` tokens that stay, for every request and
        KV head: the first ``sink``, the last ``recent``, and of the others
        those of largest mass (of equals the lower position; a NaN above all).
        int32 [B, num_kv_heads, most kept], ascending, -1 behind a request's
        kept tokens; a request of at most ``keep[b]`` tokens keeps them all."""
        k = _HostInts(keep, "keep")
        sink, recent = int(sink), int(recent)
        if not (0 <= sink < 2 ** 31 and 0 <= recent < 2 ** 31):
            raise ValueError("sink and recent must lie in [0, 2**31)")
        ctx, s = self._enter(stream)
        with ctx:
            m = self._mass_of(mass, k.n, "mass")
            index = out
            if out is None:
                if k.n > self.max_batch:
                    raise ValueError(f"at most {self.max_batch} requests")
                most = N.shkv_select_width(self.handle, k.n, k.ptr)
                index = torch.empty((k.n, self.num_kv_heads, max(most, 1)), dtype=_I32, device=self.k_pages.device)
            elif out.dtype is not _I32 or out.device != self.k_pages.device or out.dim() != 3 or \
                    not out.is_contiguous() or out.shape[0] != k.n or out.shape[1] != self.num_kv_heads:
                raise ValueError(f"out must be a contiguous int32 tensor [{k.n}, {self.num_kv_heads}, K]")
            if k.n:
                self._hold(s, stream, mass, out)
                N.shkv_select_tokens(self.handle, k.n, m, k.ptr, sink, recent, index.data_ptr(), index.shape[2], s)
        return index

    def evict_tokens(self, index: torch.Tensor, keep, new_table: torch.Tensor, mass: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, source=None, stream=None) -> None:
        """Moves the kept tokens of every request longer than ``keep[b]`` to
        the pages ``new_table[b]`` names, KV head by KV head; its row of
        ``block_table`` and its length follow, its old pages are free once the
        call has run.  Other requests are left alone.

        index: int32 [B, num_kv_heads, K], as ``select_tokens`` returns it
        new_table: int32 [B, W], W * page_size >= keep[b], of pages that no
        request of the call reads; its row becomes the request's, with the pages
        it names for tokens to come
        mass: masses that move along: to the front of the request's row, zeros
        behind them up to the old length, into ``out`` (``mass`` itself if None:
        the index must ascend then; another ``out`` must not overlap ``mass``)
        source: (table, lens) that say where the tokens are, instead of the
        pool's own: int32 [B, W'] on the device, and a host list.  A table that
        is no part of the pool's saves the call its second launch."""
        k = _HostInts(keep, "keep")
        device = self.k_pages.device
        if index.dtype is not _I32 or index.device != device or index.dim() != 3 or not index.is_contiguous() or \
                index.shape[0] < k.n or index.shape[1] != self.num_kv_heads:
            raise ValueError(f"index must be a contiguous int32 tensor [{k.n}, {self.num_kv_heads}, K] on {device}")
        if out is not None and mass is None:
            raise ValueError("out without mass")
        tables = [(new_table, "new_table")]
        table = lens = None
        if source is not None:
            table, lens = source[0], _HostInts(source[1], "source lengths")
            if lens.n != k.n:
                raise ValueError("source lengths and keep must have the same length")
            tables.append((table, "source table"))
        for t, name in tables:
            if t.dtype is not _I32 or t.device != device or t.dim() != 2 or not t.is_contiguous() or t.shape[0] < k.n:
                raise ValueError(f"{name} must be a contiguous int32 tensor [{k.n}, pages] on {device}")
        ctx, s = self._enter(stream)
        with ctx:
            m, o, _ = self._masses(mass, out, k.n) if mass is not None else (None, None, None)
            if k.n:
                self._hold(s, stream, index, new_table, table, mass, out)
                N.shkv_evict_tokens(self.handle, k.n, k.ptr, index.data_ptr(), index.shape[2], new_table.data_ptr(),
                                    new_table.shape[1], table.data_ptr() if table is not None else None,
                                    table.shape[1] if table is not None else 0, lens.ptr if lens is not None else None,
                                    m, o, s)
