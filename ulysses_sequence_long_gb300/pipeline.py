"""One attention layer of emulated Ulysses, composed from the C entry points.

``UlyssesAttention`` owns the device buffers of one problem shape and calls
the library in the order of the attention wrapper of huggingface/accelerate
PR #4209: the q/k/v exchange (gather sequence, scatter heads), document
boundaries from the gathered position_ids, attention over the gathered
sequence, and the output exchange back; the backward swaps the exchanges.

Two ways to run the exchanges:

* fused (default when S/P is a multiple of 128): the attention kernels read
  q/dO (and, in the backward, k/v) straight from the sequence shards and
  write O/dQ/dK/dV straight back (``io_layout = USP_IO_SEQ``); the
  permutation happens in their TMA loads and stores.  Only k and v are
  exchanged explicitly for the forward (``USP_IO_SEQ_KV_HEAD``), which
  re-reads every k/v tile many times and runs faster from head-layout rows;
* explicit: ``usp_relayout_*`` kernels move the tensors between the shard
  layout and the head layout around head-layout attention.

With fewer key/value heads than ranks (P a multiple of Hkv) every key/value
head is replicated on P/Hkv ranks; the exchange back of dK/dV sums the
replicas (explicit mode), or the dK/dV kernel sums the whole query group
directly (fused mode).

The backward stores dS for the dQ pass when the workspace fits in half the
free memory; for long sequences whose whole dS does not, the dK/dV and dQ
passes run one group of key/value heads at a time over one workspace
(``plan_backward``).

torch only allocates the buffers and supplies the stream; every step runs in
the library's kernels.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import binding as B_


# Layers with modified scores: up to this many tokens the forward reads k and v from their shards instead of
# moving them to head layout first.  Two launches fewer, but the rows of a key tile lie a whole token's
# key/value heads apart and are read again by every query tile.  Forward on 8 ranks, microseconds in place /
# moved: 32 heads over 8, D 128: 31.3 / 34.9 at 1024 tokens, 55.4 / 59.4 at 2048, 157.9 / 158.2 at 4096,
# 508 / 506 at 8192, 1838 / 1806 at 16384; 64 heads over 8, D 64: 248 / 256 at 4096.
KV_IN_PLACE_TOKENS = 4096


@dataclass
class Shape:
    B: int
    S: int
    Hq: int
    Hkv: int
    D: int
    P: int
    causal: bool = True
    window_left: int = -1
    softmax_scale: float = 0.0

    @property
    def hq(self):
        return self.Hq // self.P

    @property
    def hk(self):
        """Key/value heads per rank; with fewer of them than ranks each rank
        holds one replicated head."""
        return self.Hkv // self.P if self.Hkv >= self.P else 1

    @property
    def can_fuse(self) -> bool:
        return (self.S // self.P) % 128 == 0


@dataclass
class ScoreMods:
    """What modifies the scores of a layer (``usp_score_mods``): a tanh cap, a
    linear bias by distance (slopes fp32 ``[Hq]``), a learned bias by distance
    bucket (rel_bias fp32 ``[Hq][n_buckets]``, buckets int32
    ``[2*max_distance + 1]``, e.g. ``rel_buckets_log``), and a prefix mask
    (prefix_lens int32, one per document).  Heads are the layer's global ones.
    The layer reads the tensors at every call, so a table updated in place is
    the one the next call uses."""
    softcap: float = 0.0
    slopes: Optional[torch.Tensor] = None
    rel_bias: Optional[torch.Tensor] = None
    buckets: Optional[torch.Tensor] = None
    prefix_lens: Optional[torch.Tensor] = None
    rel_bias_grad: bool = True   # the backward gives the table's gradient

    def struct(self, Hq: int, with_backward: bool = True) -> B_.ScoreModsStruct:
        return B_.score_mods(Hq, self.softcap, self.slopes, self.rel_bias, self.buckets,
                             with_backward and self.rel_bias is not None and self.rel_bias_grad, self.prefix_lens)


def rel_buckets_log(n_buckets: int, max_distance: int, bidirectional: bool, device="cuda") -> torch.Tensor:
    """A bucket map for ``ScoreMods.buckets`` on ``device`` (``usp_rel_buckets_log``)."""
    return B_.usp_rel_buckets_log(n_buckets, max_distance, bidirectional).to(device)


class Rotary:
    """Rotary positions of a model (``usp_rope_fwd``): ``freqs`` fp32
    ``[pairs]`` in radians per position, ``axes`` int32 ``[pairs]`` the axis of
    each pair (``n_axes`` of them; None: one axis).  Pair i is elements i and
    i + pairs of a head, or 2i and 2i + 1 (``interleaved``); elements behind
    the pairs pass through."""

    def __init__(self, freqs: torch.Tensor, axes: Optional[torch.Tensor] = None, n_axes: int = 1,
                 interleaved: bool = False):
        if B_._dev(freqs, "freqs", torch.float32) is None:
            raise TypeError("freqs must be a CUDA tensor")
        B_._dev(axes, "axes", torch.int32)
        if axes is None and n_axes != 1:
            raise ValueError("several axes need the axis of each pair")
        if axes is not None and (axes.numel() != freqs.numel() or axes.device != freqs.device):
            raise ValueError(f"axes must have an entry for each of the {freqs.numel()} frequencies, on their device")
        self.freqs, self.axes, self.n_axes, self.interleaved = freqs, axes, int(n_axes), bool(interleaved)
        self.status = torch.zeros((1,), dtype=torch.int32, device=freqs.device)
        self.device, self._index = freqs.device, freqs.get_device()
        lib = B_.load()
        self._fwd, self._bwd = lib.usp_rope_fwd, lib.usp_rope_bwd
        self._n_pairs = freqs.numel()
        self._find()
        B_.settle(self._index)

    def _find(self):
        """The addresses of the rotation's tensors, for the calls to come (which see when a tensor or its storage was
        exchanged; references keep others from getting the same places meanwhile)."""
        at, n = self._at, self._n_pairs
        held = self.freqs, self.axes, self.status
        self._found = (at(held[0], "freqs", torch.float32, n),
                       None if held[1] is None else at(held[1], "axes", torch.int32, n),
                       at(held[2], "status", torch.int32, 1))
        self._held, self._seen = held, {}

    def _plan(self, q, k, positions):
        """Sizes of a call, by the shapes."""
        if q.dim() < 2 or (k is not None and (k.dim() < 2 or k.shape[-1] != q.shape[-1])):
            raise ValueError("q and k must be [..., heads, D]")
        Hq, D = q.shape[-2:]
        tokens, Hkv = q.numel() // max(1, Hq * D), 0 if k is None else k.shape[-2]
        if k is not None and k.numel() != tokens * Hkv * D:
            raise ValueError(f"q has {tokens} tokens, k {k.numel() // max(1, Hkv * D)}")
        n = positions.numel()
        if n == 0 or n % self.n_axes or tokens % (n // self.n_axes):
            raise ValueError(f"positions must be [{self.n_axes}][n] with n tokens or a divisor of their {tokens}, "
                             f"got {n} elements")
        return B_.RopeParams(tokens, Hq, Hkv, D, self.n_axes, n // self.n_axes, self._n_pairs, int(self.interleaved),
                             None, self._found[0], self._found[1])

    def _at(self, t, name, dtype, n):
        if isinstance(t, torch.Tensor) and t.dtype is dtype and t.numel() == n and t.get_device() == self._index and t.is_contiguous():
            return t.data_ptr()
        if B_._dev(t, name, dtype) is None:
            raise TypeError(f"{name} must be a CUDA tensor")
        raise ValueError(f"{name} must have {n} elements on {self.device}, got {tuple(t.shape)} on {t.device}")

    def _turn(self, fn, where, q, k, positions, out, stream):
        freqs, axes, status = self._found
        mine, mine_axes, mine_status = self._held
        if (self.freqs is not mine or self.axes is not mine_axes or self.status is not mine_status
                or mine.data_ptr() != freqs or mine_status.data_ptr() != status
                or (axes is not None and mine_axes.data_ptr() != axes)):
            self._find()
            status = self._found[2]
        n_pos = positions.numel()
        shapes = (q.shape, None if k is None else k.shape, n_pos, self.n_axes, self.interleaved)
        p = self._seen.get(shapes)
        if p is None:
            p = self._plan(q, k, positions)
            if len(self._seen) < 1024:
                self._seen[shapes] = p
        p = B_.RopeParams.from_buffer_copy(p)   # this call's own (threads may share a Rotary)
        bf, index, at = torch.bfloat16, self._index, self._at
        p.positions = at(positions, "positions", torch.int32, n_pos)
        if out is None:
            with B_.memory_of(index, stream):
                out = (torch.empty_like(q, memory_format=torch.contiguous_format),
                       None if k is None else torch.empty_like(k, memory_format=torch.contiguous_format))
        y, yk = out
        if (k is not None and q.dtype is bf and k.dtype is bf and y.dtype is bf and yk.dtype is bf
                and q.get_device() == index and k.get_device() == index and y.get_device() == index
                and yk.get_device() == index and q.is_contiguous() and k.is_contiguous() and y.is_contiguous()
                and yk.is_contiguous() and y.numel() == q.numel() and yk.numel() == k.numel()):
            x, xk, y, yk = q.data_ptr(), k.data_ptr(), y.data_ptr(), yk.data_ptr()
        else:
            x, y = at(q, "q", bf, q.numel()), at(y, "the output of q", bf, q.numel())
            xk, yk = (None, None) if k is None else (at(k, "k", bf, k.numel()), at(yk, "the output of k", bf, k.numel()))
        B_.run_on(index, stream, fn, where, ctypes.byref(p), x, xk, y, yk, status)
        return out

    def forward(self, q, k, positions, out=None, stream=None):
        """(q, k) turned: bf16 ``[..., H, D]`` each (k may be None), positions int32 ``[n_axes][tokens]``, or of a
        divisor of the tokens, over which they repeat.  ``out``: the tensors to write, which may be q and k (new ones are
        memory of ``stream``)."""
        return self._turn(self._fwd, "usp_rope_fwd", q, k, positions, out, stream)

    def backward(self, dq, dk, positions, out=None, stream=None):
        """The gradients of ``forward``'s outputs to those of its inputs (``out`` may be dq and dk)."""
        return self._turn(self._bwd, "usp_rope_bwd", dq, dk, positions, out, stream)

    def read_status(self) -> int:
        return int(self.status.item())


def layer_positions(rope, given, ids, tokens: int):
    """The positions by which a layer turns its `tokens` tokens: `given`, or the position ids of a ``rope`` of one axis.  A
    layer takes one for each of its tokens and axes (``Rotary`` itself repeats those of a divisor of the tokens: fewer
    would be taken for another axis' or another rank's)."""
    if given is None:
        if ids is None or rope.n_axes != 1:
            raise ValueError(f"a layer whose rope has {rope.n_axes} axes needs its tokens' positions")
        given = ids
    if given.numel() != rope.n_axes * tokens:
        raise ValueError(f"positions must be [{rope.n_axes}] axes of {tokens} tokens, got {tuple(given.shape)}")
    return given


class _Turned:
    """A layer's rotary positions: buffers for the turned shards, and the positions of the forward for the backward."""

    def _init_rope(self, rope, dev, seq_q, seq_kv):
        self.rope = rope
        if rope is None:
            return
        self.q_rot = torch.empty(seq_q, dtype=torch.bfloat16, device=dev)
        self.k_rot = torch.empty(seq_kv, dtype=torch.bfloat16, device=dev)
        if rope.device != self.q_rot.device:
            raise ValueError(f"the rotary frequencies are on {rope.device}, the layer on {self.q_rot.device}")
        self._rope_positions = None

    def _check_turned(self, v_seq, pos_shards, sinks):
        """A forward that is refused leaves the turned shards, which the backward reads: what else it takes is looked at
        before they are written."""
        B_._sized(v_seq, "v", torch.bfloat16, self.k_rot.numel(), self.k_rot)
        B_._sized(pos_shards, "position ids", torch.int32, self.shape.B * self.shape.S, self.k_rot)
        if sinks is not None:
            B_._sized(sinks, "sinks", torch.float32, self.shape.Hq, self.k_rot)

    def rotate(self, q_seq, k_seq, positions, stream=None):
        """The layer's first step: q and k shards turned (as they are without ``rope``), for ``exchange_qkv``."""
        if self.rope is None:
            return q_seq, k_seq
        layer_positions(self.rope, positions, None, self.shape.B * self.shape.S)
        self.rope.forward(q_seq, k_seq, positions, out=(self.q_rot, self.k_rot), stream=stream)
        self._rope_positions = positions
        return self.q_rot, self.k_rot

    def _rotate_back(self, stream):
        """dQ and dK shards to the gradients of q and k before they were turned, in place."""
        if self.rope is not None:
            self.rope.backward(self.dq_seq, self.dk_seq, self._rope_positions, out=(self.dq_seq, self.dk_seq),
                               stream=stream)


def plan_backward(prm: B_.AttnParams, free_bytes: int, stored_ds: Optional[bool] = None, Hkv: int = 0,
                  groups_ok: bool = False, group_size: Optional[int] = None,
                  mods: Optional[B_.ScoreModsStruct] = None):
    """(workspace bytes, stored dS?, key/value head groups) of the backward
    calls for ``free_bytes`` of free device memory (host arithmetic only).

    With stored dS the dK/dV pass writes dS blocks and the dQ pass reads them
    instead of recomputing S and dP.  None picks it when its workspace takes
    at most half of the free memory, for all heads at once or, when
    ``groups_ok`` (fused layout), for the largest group of key/value heads
    that fits (the passes then run group by group over the same workspace);
    True insists on it (ValueError if the shape has none).  ``group_size``
    forces groups of that many key/value heads.  A group is (first key/value
    head, count); [(0, 0)] means all heads in one pass.  ``mods``: the layer's
    modified scores, if any."""
    def fast_bytes(prm):
        if mods is not None:
            return B_.usp_attn_mod_bwd_fast_workspace_bytes(prm, mods)
        return B_.usp_attn_bwd_fast_workspace_bytes(prm)

    def with_group(c):
        prm_c = B_.AttnParams(*[getattr(prm, f) for f, _ in prm._fields_])
        prm_c.head_first, prm_c.head_count = 0, c
        return fast_bytes(prm_c)

    fast = fast_bytes(prm)
    groups = [(0, 0)]
    if group_size is not None:
        if not groups_ok or stored_ds is False:
            raise ValueError("head groups need the fused layout and the stored-dS backward")
        if not 0 < group_size <= Hkv:
            raise ValueError(f"group_size must be in [1, {Hkv}]")
        fast, stored_ds = with_group(group_size), True
        groups = [(h, min(group_size, Hkv - h)) for h in range(0, Hkv, group_size)]
    elif stored_ds is None:
        stored_ds = 0 < fast <= free_bytes // 2
        if not stored_ds and fast > 0 and groups_ok:
            for c in range(Hkv - 1, 0, -1):
                need = with_group(c)
                if 0 < need <= free_bytes // 2:
                    fast, stored_ds = need, True
                    groups = [(h, min(c, Hkv - h)) for h in range(0, Hkv, c)]
                    break
    if stored_ds and fast == 0:
        raise ValueError("this shape has no stored-dS backward (it needs a causal mask and S % 128 == 0)")
    if stored_ds:
        n = fast
    elif mods is not None:
        n = B_.usp_attn_mod_bwd_workspace_bytes(prm, mods)
    else:
        n = B_.usp_attn_bwd_workspace_bytes(prm)
    return n, bool(stored_ds), groups


def backward_workspace(prm: B_.AttnParams, device, stored_ds: Optional[bool] = None, Hkv: int = 0,
                       groups_ok: bool = False, group_size: Optional[int] = None,
                       mods: Optional[B_.ScoreModsStruct] = None):
    """The workspace tensor of the backward calls on ``device``, with the
    choices of ``plan_backward`` for the device's free memory."""
    free = torch.cuda.mem_get_info(device)[0] if stored_ds is None and group_size is None else 0
    n, stored_ds, groups = plan_backward(prm, free, stored_ds, Hkv, groups_ok, group_size, mods)
    return torch.empty((max(n, 256),), dtype=torch.uint8, device=device), stored_ds, groups


class UlyssesAttention(_Turned):
    """Buffers and calls for one shape on one device.  With ``mods`` the scores
    are modified (``ScoreMods``): the same calls, and ``drel_bias`` after a
    backward.  With ``rope`` (``Rotary``) q and k are turned before the
    exchange, and the gradients turned back."""

    def __init__(self, shape: Shape, device="cuda", with_backward: bool = True, fused: Optional[bool] = None,
                 stored_ds: Optional[bool] = None, ds_group_size: Optional[int] = None,
                 mods: Optional[ScoreMods] = None, rope: Optional[Rotary] = None):
        s = self.shape = shape
        self._mods = None if mods is None else mods.struct(s.Hq, with_backward)
        self.stored_ds = stored_ds
        self.ds_group_size = ds_group_size
        self.fused = shape.can_fuse if fused is None else bool(fused)
        if self.fused and not shape.can_fuse:
            raise ValueError("fused exchanges need S/P to be a multiple of 128")
        dev = torch.device(device)
        bf = torch.bfloat16
        P, Bb, S, D = s.P, s.B, s.S, s.D
        seq_q = (P, Bb, S // P, s.Hq, D)
        seq_kv = (P, Bb, S // P, s.Hkv, D)
        self.k_head = torch.empty((P, Bb, S, s.hk, D), dtype=bf, device=dev)
        self.v_head = torch.empty((P, Bb, S, s.hk, D), dtype=bf, device=dev)
        if not self.fused:
            self.q_head = torch.empty((P, Bb, S, s.hq, D), dtype=bf, device=dev)
            self.o_head = torch.empty((P, Bb, S, s.hq, D), dtype=bf, device=dev)
        self.lse = torch.empty((P, Bb, s.hq, S), dtype=torch.float32, device=dev)
        self.o_seq = torch.empty(seq_q, dtype=bf, device=dev)
        self.cu_seqlens = torch.empty((Bb * S + 1,), dtype=torch.int32, device=dev)
        self.n_docs = torch.zeros((1,), dtype=torch.int32, device=dev)
        self.max_len = torch.zeros((1,), dtype=torch.int32, device=dev)
        self.status = torch.zeros((1,), dtype=torch.int32, device=dev)
        ws = B_.usp_cu_seqlens_workspace_bytes(Bb, S)
        self.scan_ws = torch.empty((ws,), dtype=torch.uint8, device=dev)
        self.with_backward = with_backward
        if with_backward:
            if not self.fused:
                self.do_head = torch.empty((P, Bb, S, s.hq, D), dtype=bf, device=dev)
                self.dq_head = torch.empty((P, Bb, S, s.hq, D), dtype=bf, device=dev)
                self.dk_head = torch.empty((P, Bb, S, s.hk, D), dtype=bf, device=dev)
                self.dv_head = torch.empty((P, Bb, S, s.hk, D), dtype=bf, device=dev)
            self.dq_seq = torch.empty(seq_q, dtype=bf, device=dev)
            self.dk_seq = torch.empty(seq_kv, dtype=bf, device=dev)
            self.dv_seq = torch.empty(seq_kv, dtype=bf, device=dev)
            self.dsinks = torch.zeros((s.Hq,), dtype=torch.float32, device=dev)
            if self._mods is not None and self._mods.rel_bias_grad:
                self.drel_bias = torch.zeros((s.Hq, self._mods.n_buckets), dtype=torch.float32, device=dev)
        self._init_rope(rope, dev, seq_q, seq_kv)
        self._bwd_ws = None
        self.ds_groups = [(0, 0)]
        # the forward's q/k/v: as the attention kernels read them, with modified scores the caller's tensors, whose
        # addresses are taken at each call
        self._inputs = None
        if self._mods is not None:
            if self._mods.device not in (None, self.lse.device):
                raise ValueError(f"the score modifications are on {self._mods.device}, the layer on {self.lse.device}")
            # One rank's shards are its head layout, byte for byte: nothing to exchange.
            self._one_rank = P == 1
            self._in_place = self.fused or self._one_rank   # the attention kernels read and write the shards
            # Few tokens: the forward reads k and v from the shards too.
            self._kv_in_place = self.fused and Bb * S <= KV_IN_PLACE_TOKENS
            self._index = self.lse.get_device()
            self._seen = {}
            for n in [n for n, t in vars(self).items() if isinstance(t, torch.Tensor)]:
                self._remember(n)
            self._n_q, self._n_kv = Bb * S * s.Hq * D, Bb * S * s.Hkv * D
            self._prm = {}

    def params(self, sinks: Optional[torch.Tensor], io: Optional[int] = None, group=(0, 0)) -> B_.AttnParams:
        s = self.shape
        if io is None:
            io = B_.USP_IO_SEQ if self.fused else B_.USP_IO_HEAD
        return B_.attn_params(s.B, s.S, s.Hq, s.Hkv, s.D, s.P, self.cu_seqlens, self.n_docs, s.causal,
                              s.window_left, s.softmax_scale, sinks, io, head_first=group[0], head_count=group[1])

    def _ws(self, prm):
        if self._bwd_ws is None:
            self._bwd_ws, self.stored_ds, self.ds_groups = backward_workspace(
                prm, self.lse.device, self.stored_ds, self.shape.Hkv, groups_ok=self.fused,
                group_size=self.ds_group_size, mods=self._mods)
            if self._mods is not None:
                self._remember("_bwd_ws")
        return self._bwd_ws

    # -- a layer with modified scores: its calls take the addresses of their tensors, and check them, each time ----
    def _remember(self, name):
        t = getattr(self, name)
        self._seen[name] = (t.data_ptr(), t.dtype, t.numel())   # (no reference: a dropped buffer is freed)

    def _at(self, t, name, dtype, n):
        """The address that ``t`` has now."""
        if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.numel() == n and t.get_device() == self._index
                and t.is_contiguous()):
            return t.data_ptr()
        if B_._dev(t, name, dtype) is None:
            raise TypeError(f"{name} must be a CUDA tensor")
        raise ValueError(f"{name} must have {n} elements on {self.lse.device}, got {t.numel()} on {t.device}")

    def _own(self, *names):
        """The addresses of the layer's own buffers: the caller may have put another tensor, or another storage under
        it, in a buffer's place.  It has to have the buffer's type and size and lie on the layer's device."""
        mine, seen, out = self.__dict__, self._seen, []
        for name in names:
            t = mine[name]
            at, dtype, n = seen[name]
            if not (t.data_ptr() == at and t.dtype is dtype and t.numel() == n and t.is_contiguous()):
                at = self._at(t, name, dtype, n)
                seen[name] = (at, dtype, n)
            out.append(at)
        return out

    def _shards(self, t, name, H):
        return self._at(t, name, torch.bfloat16, self._n_q if H == self.shape.Hq else self._n_kv)

    def _handle(self, stream):
        """The CUDA stream of a whole pass, looked up once."""
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self._index)
        return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)

    def _on_device(self, step, *args, stream=None):
        """step(*args, stream's handle) with the layer's device current."""
        if torch._C._cuda_getDevice() == self._index:
            return step(*args, self._handle(stream))
        with torch.cuda.device(self._index):
            return step(*args, self._handle(stream))

    @staticmethod
    def _launch(where, *args):
        rc = getattr(B_.load(), where)(*args)
        if rc != B_.USP_OK:
            raise B_.UspError(rc, where)

    def _mod_call(self, where, io, group, docs, sinks, *args):
        """``where(params, mods, *args)``; ``docs``: the addresses of cu_seqlens and n_docs.  The structures of a
        layout and group are built once, of which the addresses change; a call has read them when it returns."""
        prm = self._prm.get((io, group))
        if prm is None:
            prm = self._prm[io, group] = self.params(None, io, group)
        prm.cu_seqlens, prm.n_docs = docs
        prm.sinks = None if sinks is None else self._at(sinks, "sinks", torch.float32, self.shape.Hq)
        self._mods.point()
        self._launch(where, ctypes.byref(prm), ctypes.byref(self._mods), *args)

    def _input_shards(self, q_seq, k_seq, v_seq):
        s = self.shape
        return self._shards(q_seq, "q", s.Hq), self._shards(k_seq, "k", s.Hkv), self._shards(v_seq, "v", s.Hkv)

    def _attention_inputs(self):
        """The forward's q, k and v as the attention kernels read them."""
        return self._input_shards(*self._inputs) if self._in_place else self._own("q_head", "k_head", "v_head")

    def _mod_exchange(self, q_seq, k_seq, v_seq, stream):
        s = self.shape
        q, k, v = inputs = self._input_shards(q_seq, k_seq, v_seq)
        if self._in_place:
            self._inputs = (q_seq, k_seq, v_seq)
        if self._one_rank or self._kv_in_place:
            return inputs
        if self.fused:
            for x, y in zip((k, v), self._own("k_head", "v_head")):
                self._launch("usp_relayout_fwd", x, y, s.B, s.S, s.Hkv, s.D, s.P, 2, stream)
            return inputs
        inputs = self._own("q_head", "k_head", "v_head")
        self._launch("usp_relayout_fwd_qkv", q, k, v, *inputs, s.B, s.S, s.Hq, s.Hkv, s.D, s.P, 2, stream)
        return inputs

    def _mod_boundaries(self, pos_shards, stream):
        s = self.shape
        pos = self._at(pos_shards, "position ids", torch.int32, s.B * s.S)
        cu, n_docs, max_len, ws, status = self._own("cu_seqlens", "n_docs", "max_len", "scan_ws", "status")
        self._launch("usp_cu_seqlens_from_position_ids", pos, s.B, s.S, s.P, cu, n_docs, max_len, ws,
                     self.scan_ws.numel(), status, stream)
        return cu, n_docs, status

    def _mod_attention(self, inputs, docs, sinks, stream):
        q, k, v = inputs
        cu, n_docs, status = docs
        o, lse = self._own("o_seq" if self._in_place else "o_head", "lse")
        if self._one_rank or not self.fused:
            io = B_.USP_IO_HEAD
        elif self._kv_in_place:
            io = B_.USP_IO_SEQ
        else:
            io = B_.USP_IO_SEQ_KV_HEAD
            k, v = self._own("k_head", "v_head")
        self._mod_call("usp_attn_mod_fwd", io, (0, 0), (cu, n_docs), sinks, q, k, v, o, lse, status, stream)
        return o

    def _mod_exchange_out(self, o, stream):
        s = self.shape
        self._launch("usp_relayout_bwd", o, *self._own("o_seq"), s.B, s.S, s.Hq, s.D, s.P, 2, stream)

    def _mod_forward(self, q_seq, k_seq, v_seq, pos_shards, sinks, stream):
        inputs = self._mod_exchange(q_seq, k_seq, v_seq, stream)
        docs = self._mod_boundaries(pos_shards, stream)
        o = self._mod_attention(inputs, docs, sinks, stream)
        if not self._in_place:
            self._mod_exchange_out(o, stream)
        return self.o_seq

    def _mod_backward(self, do_seq, sinks, marks, group_marks, stream):
        """``backward_phases`` with modified scores: one library call where no one asks for its phases and
        the stored dS holds every head."""
        s, rel = self.shape, self._mods.rel_bias_grad
        io = B_.USP_IO_SEQ if self.fused else B_.USP_IO_HEAD
        self._ws(self.params(None, io) if self._bwd_ws is None else None)
        mark = marks or (lambda i: None)
        lay = "_seq" if self._in_place else "_head"
        q, k, v = self._attention_inputs()
        o, dq, dk, dv, lse, status, ws, *docs = self._own("o" + lay, "dq" + lay, "dk" + lay, "dv" + lay, "lse", "status",
                                                          "_bwd_ws", "cu_seqlens", "n_docs")
        ws = (ws, self._bwd_ws.numel())
        dsinks = self._own("dsinks")[0] if sinks is not None else None
        drel = self._own("drel_bias")[0] if rel else None
        do = self._shards(do_seq, "do", s.Hq)
        call = lambda where, grp, snk, *args: self._mod_call(where, io, grp, docs, snk, *args)
        mark(0)
        if not self._in_place:
            moved, = self._own("do_head")
            self._launch("usp_relayout_fwd", do, moved, s.B, s.S, s.Hq, s.D, s.P, 2, stream)
            do = moved
        mark(1)
        if marks is None and len(self.ds_groups) == 1:
            call("usp_attn_mod_bwd", (0, 0), sinks, q, k, v, o, lse, do, dq, dk, dv, dsinks, drel, *ws, status, stream)
        else:
            gmark = group_marks or (lambda g, i: None)
            call("usp_attn_mod_bwd_preprocess", (0, 0), sinks, q, k, v, o, lse, do, dsinks, *ws, status, stream)
            mark(2)
            one = len(self.ds_groups) == 1
            for gi, grp in enumerate(self.ds_groups):
                call("usp_attn_mod_bwd_dkdv", grp, sinks if one else None, q, k, v, do, dk, dv, *ws, status, stream)
                mark(3) if one else gmark(gi, 0)
                call("usp_attn_mod_bwd_dq", grp, sinks if one else None, q, k, v, do, dq, *ws, status, stream)
                if not one:
                    gmark(gi, 1)
            if not one:
                mark(3)
            if rel:
                call("usp_attn_mod_bwd_rel_bias", (0, 0), sinks, drel, *ws, stream)
        mark(4)
        if not self._in_place:
            for grad, name, H in ((dq, "dq_seq", s.Hq), (dk, "dk_seq", s.Hkv), (dv, "dv_seq", s.Hkv)):
                self._launch("usp_relayout_bwd", grad, *self._own(name), s.B, s.S, H, s.D, s.P, 2, stream)
        mark(5)
        return self.dq_seq, self.dk_seq, self.dv_seq

    # -- steps ---------------------------------------------------------------
    def exchange_qkv(self, q_seq, k_seq, v_seq, stream=None):
        s = self.shape
        if self._mods is not None:
            self._on_device(self._mod_exchange, q_seq, k_seq, v_seq, stream=stream)
            return
        if self.fused:
            # q stays in its shards; k and v go to head layout for the forward
            B_.usp_relayout_fwd(k_seq, self.k_head, s.B, s.S, s.Hkv, s.D, s.P, stream)
            B_.usp_relayout_fwd(v_seq, self.v_head, s.B, s.S, s.Hkv, s.D, s.P, stream)
            self._inputs = (q_seq, k_seq, v_seq)
            return
        B_.usp_relayout_fwd_qkv(q_seq, k_seq, v_seq, self.q_head, self.k_head, self.v_head,
                                s.B, s.S, s.Hq, s.Hkv, s.D, s.P, stream)
        self._inputs = (self.q_head, self.k_head, self.v_head)

    def boundaries(self, pos_shards, stream=None):
        s = self.shape
        if self._mods is not None:
            self._on_device(self._mod_boundaries, pos_shards, stream=stream)
            return
        B_.usp_cu_seqlens_from_position_ids(pos_shards, s.B, s.S, s.P, self.cu_seqlens, self.n_docs,
                                            self.max_len, self.scan_ws, self.status, stream)

    def attention(self, sinks=None, stream=None):
        if self._mods is not None:
            self._on_device(self._mod_attention, self._attention_inputs(), self._own("cu_seqlens", "n_docs", "status"),
                            sinks, stream=stream)
            return
        q, k, v = self._inputs
        if self.fused:
            B_.usp_attn_fwd(self.params(sinks, B_.USP_IO_SEQ_KV_HEAD), q, self.k_head, self.v_head, self.o_seq,
                            self.lse, self.status, stream)
        else:
            B_.usp_attn_fwd(self.params(sinks), q, k, v, self.o_head, self.lse, self.status, stream)

    def exchange_out(self, stream=None):
        s = self.shape
        if self._mods is not None:
            if not self._in_place:
                self._on_device(self._mod_exchange_out, *self._own("o_head"), stream=stream)
        elif not self.fused:
            B_.usp_relayout_bwd(self.o_head, self.o_seq, s.B, s.S, s.Hq, s.D, s.P, stream)

    def forward(self, q_seq, k_seq, v_seq, pos_shards, sinks=None, stream=None, rope_positions=None):
        """Sequence shards in, sequence shards out (``self.o_seq``).  ``rope_positions``: int32
        ``[n_axes][P][B][S/P]`` for the layer's ``rope`` (default, for one axis: the position ids)."""
        if self.rope is not None:
            self._check_turned(v_seq, pos_shards, sinks)
            rope_positions = layer_positions(self.rope, rope_positions, pos_shards, self.shape.B * self.shape.S)
            q_seq, k_seq = self.rotate(q_seq, k_seq, rope_positions, stream)
        if self._mods is not None:
            return self._on_device(self._mod_forward, q_seq, k_seq, v_seq, pos_shards, sinks, stream=stream)
        self.exchange_qkv(q_seq, k_seq, v_seq, stream)
        self.boundaries(pos_shards, stream)
        self.attention(sinks, stream)
        self.exchange_out(stream)
        return self.o_seq

    def head_kv(self, stream=None):
        """The last forward's keys (turned, with ``rope``) and values in head layout ``[P][B][S][heads of a rank][D]``:
        what ``serving.PagedCache.append`` takes, with ``cu_seqlens``.  The forward has left them there but for a layer with
        modified scores that read them from their shards."""
        if self._mods is None or not (self._one_rank or self._kv_in_place):
            return self.k_head, self.v_head
        k, v = self._inputs[1:]
        if self._one_rank:   # its shards are its head layout
            return k.view(self.k_head.shape), v.view(self.v_head.shape)
        self._on_device(self._mod_exchange_kv, k, v, stream=stream)
        return self.k_head, self.v_head

    def _mod_exchange_kv(self, k, v, stream):
        s = self.shape
        for t, name, y in zip((k, v), ("k", "v"), self._own("k_head", "v_head")):
            self._launch("usp_relayout_fwd", self._shards(t, name, s.Hkv), y, s.B, s.S, s.Hkv, s.D, s.P, 2, stream)

    def backward_phases(self, do_seq, sinks=None, stream=None, marks=None, group_marks=None):
        """The backward as its separate library calls; `marks(i)` is called
        between them (for timing): 0 before, 1 after the dO exchange, 2 after
        the preprocess, 3 after dK/dV, 4 after dQ, 5 after the output exchanges
        (with ``rope`` the gradients are turned back after that).
        When the passes run in key/value head groups, marks 3 and 4 both come
        after the last group and `group_marks(g, 0)` / `group_marks(g, 1)`
        after group g's dK/dV and dQ passes."""
        self._backward_phases(do_seq, sinks, stream, marks, group_marks)
        self._rotate_back(stream)
        return self.dq_seq, self.dk_seq, self.dv_seq

    def _backward_phases(self, do_seq, sinks, stream, marks, group_marks):
        s = self.shape
        if self._mods is not None:
            return self._on_device(self._mod_backward, do_seq, sinks, marks, group_marks, stream=stream)
        prm = self.params(sinks)
        ws = self._ws(prm)
        mark = marks or (lambda i: None)
        q, k, v = self._inputs
        mark(0)
        if self.fused:
            do, o, dq, dk, dv = do_seq, self.o_seq, self.dq_seq, self.dk_seq, self.dv_seq
        else:
            B_.usp_relayout_fwd(do_seq, self.do_head, s.B, s.S, s.Hq, s.D, s.P, stream)
            do, o, dq, dk, dv = self.do_head, self.o_head, self.dq_head, self.dk_head, self.dv_head
        mark(1)
        B_.usp_attn_bwd_preprocess(prm, o, self.lse, do, self.dsinks if sinks is not None else None, ws,
                                   self.status, stream)
        mark(2)
        if len(self.ds_groups) == 1:
            B_.usp_attn_bwd_dkdv(prm, q, k, v, self.lse, do, dk, dv, ws, self.status, stream)
            mark(3)
            B_.usp_attn_bwd_dq(prm, q, k, v, self.lse, do, dq, ws, self.status, stream)
        else:  # stored dS a key/value head group at a time (both passes per group)
            gmark = group_marks or (lambda g, i: None)
            for gi, grp in enumerate(self.ds_groups):
                prm_g = self.params(None, group=grp)
                B_.usp_attn_bwd_dkdv(prm_g, q, k, v, self.lse, do, dk, dv, ws, self.status, stream)
                gmark(gi, 0)
                B_.usp_attn_bwd_dq(prm_g, q, k, v, self.lse, do, dq, ws, self.status, stream)
                gmark(gi, 1)
            mark(3)
        mark(4)
        if not self.fused:
            B_.usp_relayout_bwd(self.dq_head, self.dq_seq, s.B, s.S, s.Hq, s.D, s.P, stream)
            B_.usp_relayout_bwd(self.dk_head, self.dk_seq, s.B, s.S, s.Hkv, s.D, s.P, stream)
            B_.usp_relayout_bwd(self.dv_head, self.dv_seq, s.B, s.S, s.Hkv, s.D, s.P, stream)
        mark(5)
        return self.dq_seq, self.dk_seq, self.dv_seq

    def backward(self, do_seq, sinks=None, stream=None):
        """dO shards in; dQ/dK/dV shards out (``self.dq_seq`` ...), dsinks.
        In explicit mode this is the single ``usp_attn_bwd`` (or
        ``usp_attn_mod_bwd``) call."""
        if self.fused or self._mods is not None:
            return self.backward_phases(do_seq, sinks, stream)
        s = self.shape
        prm = self.params(sinks)
        ws = self._ws(prm)
        q, k, v = self._inputs
        B_.usp_relayout_fwd(do_seq, self.do_head, s.B, s.S, s.Hq, s.D, s.P, stream)
        B_.usp_attn_bwd(prm, q, k, v, self.o_head, self.lse, self.do_head, self.dq_head, self.dk_head,
                        self.dv_head, self.dsinks if sinks is not None else None, ws, self.status, stream)
        B_.usp_relayout_bwd(self.dq_head, self.dq_seq, s.B, s.S, s.Hq, s.D, s.P, stream)
        B_.usp_relayout_bwd(self.dk_head, self.dk_seq, s.B, s.S, s.Hkv, s.D, s.P, stream)
        B_.usp_relayout_bwd(self.dv_head, self.dv_seq, s.B, s.S, s.Hkv, s.D, s.P, stream)
        self._rotate_back(stream)
        return self.dq_seq, self.dk_seq, self.dv_seq

    def read_status(self) -> int:
        return int(self.status.item()) or (0 if self.rope is None else self.rope.read_status())


class HybridAttention(_Turned):
    """Ring x Ulysses (USP) over P = ring * ulysses emulated ranks.

    The Ulysses exchange runs inside each ring group; then ``ring`` steps
    each run the attention kernels restricted to the key/value super-chunk a
    ring rank holds at that step (``params.ring``/``ring_step``).  The forward
    merges each step's (O, LSE) into the running result
    (``usp_ring_fwd_merge``, sink folded in at the last step); the backward
    sums each step's bf16 block gradients in fp32
    (``usp_ring_grad_accumulate``) with the final LSE and D statistics
    computed once.

    Fused (default when each sequence shard is a multiple of 128 tokens): the
    kernels read and write the sequence shards directly and every
    intermediate is in that layout, so no exchange kernel runs.  Explicit:
    ``usp_hybrid_relayout_*`` move tensors to and from the hybrid head layout
    [U][B][S][H/U][D].

    With ``rope`` (``Rotary``) q and k are turned before the exchange, and the
    gradients turned back.
    """

    def __init__(self, shape: Shape, ring: int, device="cuda", with_backward: bool = True,
                 stored_ds: Optional[bool] = None, fused: Optional[bool] = None, ds_group_size: Optional[int] = None,
                 rope: Optional[Rotary] = None):
        s = self.shape = shape
        self.stored_ds = stored_ds
        self.ds_group_size = ds_group_size
        if ring < 1 or s.P % ring != 0:
            raise ValueError("the ring degree must divide the ranks")
        self.ring = R = ring
        self.U = U = s.P // ring
        can_fuse = (s.S // s.P) % 128 == 0
        self.fused = can_fuse if fused is None else bool(fused)
        if self.fused and not can_fuse:
            raise ValueError("fused exchanges need each sequence shard to be a multiple of 128 tokens")
        dev = torch.device(device)
        bf, f32 = torch.bfloat16, torch.float32
        Bb, S, D = s.B, s.S, s.D
        self.hq = hq = s.Hq // U
        self.hk = hk = s.Hkv // U if s.Hkv >= U else 1
        seq_q, seq_kv = (s.P, Bb, S // s.P, s.Hq, D), (s.P, Bb, S // s.P, s.Hkv, D)
        head_q, head_kv = (U, Bb, S, hq, D), (U, Bb, S, hk, D)
        lay_q, lay_kv = (seq_q, seq_kv) if self.fused else (head_q, head_kv)
        stat = (U, Bb, hq, S)
        self.k_head = torch.empty(head_kv, dtype=bf, device=dev)
        self.v_head = torch.empty(head_kv, dtype=bf, device=dev)
        if not self.fused:
            self.q_head = torch.empty(head_q, dtype=bf, device=dev)
            self.o_head = torch.empty(head_q, dtype=bf, device=dev)
        self.o_step = torch.empty(lay_q, dtype=bf, device=dev)
        self.lse_step = torch.empty(stat, dtype=f32, device=dev)
        self.o_acc = torch.empty(lay_q, dtype=f32, device=dev) if R > 1 else None
        self.lse_acc = torch.empty(stat, dtype=f32, device=dev) if R > 1 else None
        self.lse = torch.empty(stat, dtype=f32, device=dev)
        self.o_seq = torch.empty(seq_q, dtype=bf, device=dev)
        self.cu_seqlens = torch.empty((Bb * S + 1,), dtype=torch.int32, device=dev)
        self.n_docs = torch.zeros((1,), dtype=torch.int32, device=dev)
        self.max_len = torch.zeros((1,), dtype=torch.int32, device=dev)
        self.status = torch.zeros((1,), dtype=torch.int32, device=dev)
        self.scan_ws = torch.empty((B_.usp_cu_seqlens_workspace_bytes(Bb, S),), dtype=torch.uint8, device=dev)
        self.with_backward = with_backward
        if with_backward:
            if not self.fused:
                self.do_head = torch.empty(head_q, dtype=bf, device=dev)
                self.dq_head = torch.empty(head_q, dtype=bf, device=dev)
                self.dk_head = torch.empty(head_kv, dtype=bf, device=dev)
                self.dv_head = torch.empty(head_kv, dtype=bf, device=dev)
            self.dq_step = torch.empty(lay_q, dtype=bf, device=dev)
            self.dk_step = torch.empty(lay_kv, dtype=bf, device=dev)
            self.dv_step = torch.empty(lay_kv, dtype=bf, device=dev)
            self.dq_acc = torch.empty(lay_q, dtype=f32, device=dev) if R > 1 else None
            self.dk_acc = torch.empty(lay_kv, dtype=f32, device=dev) if R > 1 else None
            self.dv_acc = torch.empty(lay_kv, dtype=f32, device=dev) if R > 1 else None
            self.dq_seq = torch.empty(seq_q, dtype=bf, device=dev)
            self.dk_seq = torch.empty(seq_kv, dtype=bf, device=dev)
            self.dv_seq = torch.empty(seq_kv, dtype=bf, device=dev)
            self.dsinks = torch.zeros((s.Hq,), dtype=torch.float32, device=dev)
        self._init_rope(rope, dev, seq_q, seq_kv)
        self._bwd_ws = None
        self.ds_groups = [(0, 0)]
        self._inputs = None

    def params(self, sinks=None, step: int = 0, io: Optional[int] = None, group=(0, 0)) -> B_.AttnParams:
        s = self.shape
        if io is None:
            io = B_.USP_IO_SEQ if self.fused else B_.USP_IO_HEAD
        return B_.attn_params(s.B, s.S, s.Hq, s.Hkv, s.D, self.U, self.cu_seqlens, self.n_docs, s.causal,
                              s.window_left, s.softmax_scale, sinks, io, self.ring, step, group[0], group[1])

    def _flags(self, step: int) -> int:
        return (B_.USP_RING_FIRST if step == 0 else 0) | (B_.USP_RING_LAST if step == self.ring - 1 else 0)

    def forward_phases(self, q_seq, k_seq, v_seq, pos_shards, sinks=None, stream=None, marks=None,
                       rope_positions=None):
        """marks(i): 0 before (with ``rope``, after q and k are turned), 1 after the q/k/v exchange, 2 after the document
        boundaries, 3 after the ring steps and merges, 4 after the O exchange.  ``rope_positions``: int32
        ``[n_axes][P][B][S/P]`` for ``rope`` (default, for one axis: the position ids)."""
        s = self.shape
        mark = marks or (lambda i: None)
        if self.rope is not None:
            self._check_turned(v_seq, pos_shards, sinks)
            rope_positions = layer_positions(self.rope, rope_positions, pos_shards, s.B * s.S)
            q_seq, k_seq = self.rotate(q_seq, k_seq, rope_positions, stream)
        mark(0)
        if self.fused:
            # q stays in its shards; k and v go to the hybrid head layout for the forward
            B_.usp_hybrid_relayout_fwd(k_seq, self.k_head, s.B, s.S, s.Hkv, s.D, self.ring, self.U, stream)
            B_.usp_hybrid_relayout_fwd(v_seq, self.v_head, s.B, s.S, s.Hkv, s.D, self.ring, self.U, stream)
            self._inputs = (q_seq, k_seq, v_seq)
            o_out = self.o_seq
        else:
            B_.usp_hybrid_relayout_fwd_qkv(q_seq, k_seq, v_seq, self.q_head, self.k_head, self.v_head,
                                           s.B, s.S, s.Hq, s.Hkv, s.D, self.ring, self.U, stream)
            self._inputs = (self.q_head, self.k_head, self.v_head)
            o_out = self.o_head
        mark(1)
        B_.usp_cu_seqlens_from_position_ids(pos_shards, s.B, s.S, s.P, self.cu_seqlens, self.n_docs,
                                            self.max_len, self.scan_ws, self.status, stream)
        mark(2)
        q, k, v = self._inputs
        io_fwd = B_.USP_IO_SEQ_KV_HEAD if self.fused else B_.USP_IO_HEAD
        for st in range(self.ring):
            B_.usp_attn_fwd(self.params(None, st, io_fwd), q, self.k_head, self.v_head, self.o_step, self.lse_step,
                            self.status, stream)
            B_.usp_ring_fwd_merge(self.params(sinks, st), self.o_step, self.lse_step, self.o_acc, self.lse_acc,
                                  o_out, self.lse, self._flags(st), stream)
        mark(3)
        if not self.fused:
            B_.usp_hybrid_relayout_bwd(self.o_head, self.o_seq, s.B, s.S, s.Hq, s.D, self.ring, self.U, stream)
        mark(4)
        return self.o_seq

    def forward(self, q_seq, k_seq, v_seq, pos_shards, sinks=None, stream=None, rope_positions=None):
        return self.forward_phases(q_seq, k_seq, v_seq, pos_shards, sinks, stream, rope_positions=rope_positions)

    def backward_phases(self, do_seq, sinks=None, stream=None, marks=None):
        """marks(i): 0 before, 1 after the dO exchange, 2 after the
        statistics, 3 after the dK/dV ring steps, 4 after the dQ ring steps,
        5 after the dQ/dK/dV exchanges (with ``rope`` the gradients are
        turned back after that)."""
        s = self.shape
        mark = marks or (lambda i: None)
        prm = self.params(sinks, 0)
        if self._bwd_ws is None:
            self._bwd_ws, self.stored_ds, self.ds_groups = backward_workspace(
                prm, self.lse.device, self.stored_ds, s.Hkv, groups_ok=self.fused, group_size=self.ds_group_size)
        ws = self._bwd_ws
        q, k, v = self._inputs
        mark(0)
        if self.fused:
            do, o = do_seq, self.o_seq
            dq_out, dk_out, dv_out = self.dq_seq, self.dk_seq, self.dv_seq
        else:
            B_.usp_hybrid_relayout_fwd(do_seq, self.do_head, s.B, s.S, s.Hq, s.D, self.ring, self.U, stream)
            do, o = self.do_head, self.o_head
            dq_out, dk_out, dv_out = self.dq_head, self.dk_head, self.dv_head
        mark(1)
        B_.usp_attn_bwd_preprocess(prm, o, self.lse, do, self.dsinks if sinks is not None else None, ws,
                                   self.status, stream)
        mark(2)
        if len(self.ds_groups) == 1:
            for st in range(self.ring):
                B_.usp_attn_bwd_dkdv(self.params(None, st), q, k, v, self.lse, do, self.dk_step, self.dv_step, ws,
                                     self.status, stream)
                B_.usp_ring_grad_accumulate(self.dk_step, self.dk_acc, dk_out, self._flags(st), stream)
                B_.usp_ring_grad_accumulate(self.dv_step, self.dv_acc, dv_out, self._flags(st), stream)
            mark(3)
            for st in range(self.ring):
                B_.usp_attn_bwd_dq(self.params(None, st), q, k, v, self.lse, do, self.dq_step, ws, self.status,
                                   stream)
                B_.usp_ring_grad_accumulate(self.dq_step, self.dq_acc, dq_out, self._flags(st), stream)
        else:  # stored dS a key/value head group at a time (both passes per group)
            for st in range(self.ring):
                for grp in self.ds_groups:
                    prm_g = self.params(None, st, group=grp)
                    B_.usp_attn_bwd_dkdv(prm_g, q, k, v, self.lse, do, self.dk_step, self.dv_step, ws, self.status,
                                         stream)
                    B_.usp_attn_bwd_dq(prm_g, q, k, v, self.lse, do, self.dq_step, ws, self.status, stream)
                B_.usp_ring_grad_accumulate(self.dk_step, self.dk_acc, dk_out, self._flags(st), stream)
                B_.usp_ring_grad_accumulate(self.dv_step, self.dv_acc, dv_out, self._flags(st), stream)
                B_.usp_ring_grad_accumulate(self.dq_step, self.dq_acc, dq_out, self._flags(st), stream)
            mark(3)
        mark(4)
        if not self.fused:
            B_.usp_hybrid_relayout_bwd(self.dq_head, self.dq_seq, s.B, s.S, s.Hq, s.D, self.ring, self.U, stream)
            B_.usp_hybrid_relayout_bwd(self.dk_head, self.dk_seq, s.B, s.S, s.Hkv, s.D, self.ring, self.U, stream)
            B_.usp_hybrid_relayout_bwd(self.dv_head, self.dv_seq, s.B, s.S, s.Hkv, s.D, self.ring, self.U, stream)
        mark(5)
        self._rotate_back(stream)
        return self.dq_seq, self.dk_seq, self.dv_seq

    def backward(self, do_seq, sinks=None, stream=None):
        return self.backward_phases(do_seq, sinks, stream)

    def read_status(self) -> int:
        return int(self.status.item()) or (0 if self.rope is None else self.rope.read_status())
