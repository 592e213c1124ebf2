"""Serving: a key/value cache in pages and the attention of one new token per
sequence over it.

A prompt runs through ``UlyssesAttention``; its keys and values in head layout
go into the cache (``PagedCache.append``), document by document of a packed
batch.  From there on each step has one new token per sequence:
``DecodeAttention.step`` turns its query and key (``Rotary``), appends key and
value and attends over the sequence's pages.  Tensors have the head layout of
one token per sequence, ``[P][sequences][H/P][D]``: every rank holds every
sequence for its heads, so nothing is exchanged.

Everything that grows or changes between steps (lengths, block tables) is read
from device memory, so a captured step replays for longer sequences.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import binding as B_
from .pipeline import layer_positions

_BF, _F8, _I32, _F32, _U8 = torch.bfloat16, torch.float8_e4m3fn, torch.int32, torch.float32, torch.uint8


def _where(t, name, dtype, n, index):
    """The address of `t`, which has to be contiguous, of `n` elements of `dtype`, on device `index`."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.numel() == n and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    if B_._dev(t, name, dtype) is None:
        raise TypeError(f"{name} must be a CUDA tensor")
    raise ValueError(f"{name} must have {n} elements on cuda:{index}, got {tuple(t.shape)} on {t.device}")


class PagedCache:
    """The pool of pages of one layer: ``k_pages``, ``v_pages``
    ``[P][n_pages][heads of a rank][page_size][D]`` in bf16, or in e4m3
    (``dtype=torch.float8_e4m3fn``) with ``k_scales``, ``v_scales`` bytes
    ``[P][n_pages][heads of a rank][page_size]``.  ``block_table`` is int32
    ``[sequences][max_pages]``, ``lens`` int32 ``[sequences]`` counts each
    sequence's tokens, appended ones included."""

    def __init__(self, n_pages: int, page_size: int, Hkv: int, D: int, P: int = 1, dtype=torch.bfloat16,
                 device="cuda"):
        if dtype not in (_BF, _F8):
            raise TypeError(f"a cache holds torch.bfloat16 or torch.float8_e4m3fn, not {dtype}")
        if (Hkv % P if Hkv >= P else P % Hkv) != 0:
            raise ValueError(f"{P} ranks and {Hkv} key/value heads: neither divides the other")
        self.n_pages, self.page_size, self.Hkv, self.D, self.P, self.dtype = n_pages, page_size, Hkv, D, P, dtype
        self.hk = Hkv // P if Hkv >= P else 1
        dev = torch.device(device)
        shape = (P, n_pages, self.hk, page_size, D)
        self.k_pages, self.v_pages = (torch.zeros(shape, dtype=_U8 if dtype is _F8 else _BF, device=dev).view(dtype)
                                      for _ in range(2))
        eight = dtype is _F8
        self.k_scales, self.v_scales = (torch.ones(shape[:-1], dtype=_U8, device=dev) if eight else None
                                        for _ in range(2))
        self.status = torch.zeros((1,), dtype=_I32, device=dev)
        self.device = self.status.device
        self._index = self.status.get_device()
        self._fixed = B_.PagedCacheStruct(P, Hkv, D, n_pages, page_size, 0, 0,
                                          B_.USP_CACHE_E4M3 if eight else B_.USP_CACHE_BF16)
        lib = B_.load()
        self._append, self._read = lib.usp_cache_append, lib.usp_cache_read
        self._find()
        B_.settle(self._index)

    def _find(self):
        """The addresses of the pool's tensors, which have to be of their sizes and types, for the calls to come (which
        see when a tensor or its storage was exchanged; references keep others from getting the same places meanwhile)."""
        c, index, n = self._fixed, self._index, self.P * self.n_pages * self.hk * self.page_size
        held = self.k_pages, self.v_pages, self.k_scales, self.v_scales, self.status
        ks = vs = None
        k = _where(held[0], "k_pages", self.dtype, n * self.D, index)
        v = _where(held[1], "v_pages", self.dtype, n * self.D, index)
        if self.dtype is _F8:
            ks = _where(held[2], "k_scales", _U8, n, index)
            vs = _where(held[3], "v_scales", _U8, n, index)
        status = _where(held[4], "status", _I32, 1, index)
        # (all of them are in order)
        c.k_pages, c.v_pages, c.k_scales, c.v_scales, self._status = k, v, ks, vs, status
        self._held, self._found = held, (k, v, ks, vs, status)

    def _struct(self, block_table, lens) -> B_.PagedCacheStruct:
        """This call's own structure (threads may use one cache at once), with the addresses that the tensors have now."""
        k, v, ks, vs, status = self._found
        hk, hv, hks, hvs, hstatus = self._held
        if (self.k_pages is not hk or self.v_pages is not hv or self.status is not hstatus or self.k_scales is not hks
                or self.v_scales is not hvs or hk.data_ptr() != k or hv.data_ptr() != v or hstatus.data_ptr() != status
                or (ks is not None and (hks.data_ptr() != ks or hvs.data_ptr() != vs))):
            self._find()
        c = B_.PagedCacheStruct.from_buffer_copy(self._fixed)
        index = self._index
        if (block_table.dtype is _I32 and lens.dtype is _I32 and block_table.get_device() == index
                and lens.get_device() == index and block_table.is_contiguous() and lens.is_contiguous()
                and block_table.dim() == 2 and lens.dim() == 1 and block_table.size(0) == lens.size(0)):
            c.n_seqs, c.max_pages = lens.size(0), block_table.size(1)
            c.block_table, c.lens = block_table.data_ptr(), lens.data_ptr()
            return c
        if block_table.dim() != 2 or lens.dim() != 1:
            raise ValueError("block_table must be [sequences][max_pages], lens [sequences]")
        _where(lens, "lens", _I32, lens.numel(), index)
        _where(block_table, "block_table", _I32, lens.numel() * block_table.shape[1], index)
        raise ValueError(f"block_table has {block_table.shape[0]} rows, lens {lens.shape[0]} sequences")

    def _move(self, fn, where, k, v, block_table, lens, cu_seqlens, stream):
        c = self._struct(block_table, lens)
        per, index = self.P * self.hk * self.D, self._index
        n = k.numel()
        if n == 0 or n % per != 0:
            raise ValueError(f"k must be [{self.P}][tokens][{self.hk}][{self.D}], got {tuple(k.shape)}")
        kp, vp = _where(k, "k", _BF, n, index), _where(v, "v", _BF, n, index)
        cu = None
        if cu_seqlens is not None:  # (the boundaries of a packed batch have room for more documents)
            if cu_seqlens.numel() <= c.n_seqs:
                raise ValueError(f"cu_seqlens must have at least {c.n_seqs + 1} elements, got {cu_seqlens.numel()}")
            cu = _where(cu_seqlens, "cu_seqlens", _I32, cu_seqlens.numel(), index)
        B_.run_on(index, stream, fn, where, ctypes.byref(c), kp, vp, n // per, cu, self._status)

    def append(self, k, v, block_table, lens, cu_seqlens=None, stream=None):
        """Write the last tokens of each sequence: k, v bf16 ``[P][tokens][heads of a rank][D]`` (head layout), tokens
        ``[cu_seqlens[s], cu_seqlens[s+1])`` of sequence s, or one of each sequence without ``cu_seqlens``.
        A layer that ran a packed batch has these in ``head_kv()`` and ``cu_seqlens``; ``block_table`` and ``lens`` have a
        row for each of its first documents then, but none beyond its last (where its ``cu_seqlens`` hold nothing)."""
        self._move(self._append, "usp_cache_append", k, v, block_table, lens, cu_seqlens, stream)

    def read(self, block_table, lens, cu_seqlens=None, out=None, tokens: Optional[int] = None, stream=None):
        """The way back: (k, v) of the last tokens of each sequence, into ``out``, or into new tensors of ``tokens``
        tokens (places without a token are zero there, and left alone in ``out``); the new ones are memory of ``stream``."""
        if out is None:
            if tokens is None:
                if cu_seqlens is not None:
                    raise ValueError("read needs out or tokens beside cu_seqlens (their sum is on the device)")
                tokens = lens.shape[0]
            with B_.memory_of(self._index, stream):
                out = tuple(torch.zeros((self.P, tokens, self.hk, self.D), dtype=_BF, device=self.device) for _ in range(2))
        self._move(self._read, "usp_cache_read", out[0], out[1], block_table, lens, cu_seqlens, stream)
        return out

    def read_status(self) -> int:
        return int(self.status.item())


class DecodeAttention:
    """Attention of one new token per sequence over a ``PagedCache``, with the
    window, scale and sinks of the layer; ``rope``: the layer's ``Rotary``,
    for ``step``.  Outputs are views of the layer's own buffers, which hold up
    to ``max_seqs`` sequences; the workspace is the layer's too, so calls that
    may overlap (other streams, captured graphs) need a layer each."""

    def __init__(self, cache: PagedCache, Hq: int, max_seqs: int, window_left: int = -1, softmax_scale: float = 0.0,
                 rope=None):
        self.cache, self.Hq, self.max_seqs = cache, Hq, max_seqs
        self.window_left, self.softmax_scale, self.rope = int(window_left), float(softmax_scale), rope
        if Hq % cache.P != 0 or Hq % cache.Hkv != 0:
            raise ValueError(f"{Hq} query heads over {cache.P} ranks and {cache.Hkv} key/value heads")
        dev = cache.device
        self.hq = Hq // cache.P
        rows = max_seqs * Hq
        self._o = torch.empty((rows * cache.D,), dtype=_BF, device=dev)
        self._lse = torch.empty((rows,), dtype=_F32, device=dev)
        self._turned = None if rope is None else (
            torch.empty((rows * cache.D,), dtype=_BF, device=dev),
            torch.empty((cache.P * max_seqs * cache.hk * cache.D,), dtype=_BF, device=dev))
        one = torch.zeros((1, 1), dtype=_I32, device=dev)
        with torch.cuda.device(dev):
            n = B_.usp_attn_decode_workspace_bytes(cache._struct(one, one[0]), Hq)
        if n == 0:
            raise ValueError("the library has no such attention: D 64 or 128, page_size a multiple of 16, Hq <= 1024")
        self._ws = torch.zeros((n,), dtype=_U8, device=dev)
        self._ws_bytes = n
        self._decode = B_.load().usp_attn_decode
        self._views = {}
        self.lse = None
        B_.settle(cache._index)

    def _out(self, n):
        v = self._views.get(n)
        if v is None:
            c = self.cache
            if not 0 < n <= self.max_seqs:
                raise ValueError(f"{n} sequences, the layer has room for 1 to {self.max_seqs}")
            v = self._views[n] = (self._o[:n * self.Hq * c.D].view(c.P, n, self.hq, c.D),
                                  self._lse[:n * self.Hq].view(c.P, n, self.hq))
        return v

    def forward(self, q, block_table, lens, sinks=None, stream=None):
        """q bf16 ``[P][sequences][Hq/P][D]``, already turned -> O of the same shape (and ``self.lse``)."""
        c = self.cache
        index = c._index
        prm = c._struct(block_table, lens)
        n = prm.n_seqs
        o, lse = self._out(n)
        B_.run_on(index, stream, self._decode, "usp_attn_decode", ctypes.byref(prm), self.Hq, self.window_left,
                  self.softmax_scale, None if sinks is None else _where(sinks, "sinks", _F32, self.Hq, index),
                  _where(q, "q", _BF, n * self.Hq * c.D, index), o.data_ptr(), lse.data_ptr(), self._ws.data_ptr(),
                  self._ws_bytes, c._status)
        self.lse = lse
        return o

    def _check_attend(self, prm, q, sinks, o, lse):
        """What the library refuses of the attention, by addresses, before the step's tokens are in the pool."""
        if q % 16 != 0:
            raise B_.UspError(B_.USP_ERR_ALIGNMENT, "usp_attn_decode")
        if self.window_left < -1:
            raise B_.UspError(B_.USP_ERR_UNSUPPORTED, "usp_attn_decode")
        n, D = prm.n_seqs, prm.D
        o0, l0 = o.data_ptr(), lse.data_ptr()
        o1, l1 = o0 + 2 * n * self.Hq * D, l0 + 4 * n * self.Hq
        bad = not 0.0 <= self.softmax_scale < float("inf")
        for at, size in ((q, o1 - o0), (sinks, 4 * self.Hq), (prm.block_table, 4 * n * prm.max_pages), (prm.lens, 4 * n)):
            bad |= at is not None and (at < o1 and o0 < at + size or at < l1 and l0 < at + size)
        if bad:
            raise B_.UspError(B_.USP_ERR_INVALID_ARG, "usp_attn_decode")

    def step(self, q, k, v, block_table, lens, sinks=None, positions=None, stream=None):
        """One token of each sequence through the layer: turn q and k (``rope``; positions int32
        ``[n_axes][sequences]``), append k and v (bf16 ``[P][sequences][heads of a rank][D]``), attend.  ``lens`` counts the
        new token.  A step that is refused leaves the cache as it was."""
        c = self.cache
        index = c._index
        prm = c._struct(block_table, lens)
        n = prm.n_seqs
        o, lse = self._out(n)
        rows = n * c.P * c.hk * c.D
        qp = _where(q, "q", _BF, n * self.Hq * c.D, index)
        sp = None if sinks is None else _where(sinks, "sinks", _F32, self.Hq, index)
        kp, vp = _where(k, "k", _BF, rows, index), _where(v, "v", _BF, rows, index)
        if self.rope is None:
            self._check_attend(prm, qp, sp, o, lse)
        else:
            layer_positions(self.rope, positions, None, n)
            out = (self._turned[0][:n * self.Hq * c.D].view(c.P, n, self.hq, c.D),
                   self._turned[1][:rows].view(c.P, n, c.hk, c.D))
            qp, kp = out[0].data_ptr(), out[1].data_ptr()
            self._check_attend(prm, qp, sp, o, lse)
            self.rope.forward(q, k, positions, out=out, stream=stream)
        B_.run_on(index, stream, c._append, "usp_cache_append", ctypes.byref(prm), kp, vp, n, None, c._status)
        B_.run_on(index, stream, self._decode, "usp_attn_decode", ctypes.byref(prm), self.Hq, self.window_left,
                  self.softmax_scale, sp, qp, o.data_ptr(), lse.data_ptr(), self._ws.data_ptr(), self._ws_bytes, c._status)
        self.lse = lse
        return o

    def read_status(self) -> int:
        return self.cache.read_status() or (0 if self.rope is None else self.rope.read_status())
