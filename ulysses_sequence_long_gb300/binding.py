"""ctypes binding of libusp.so: the C entry points of include/usp.h, same names.

Argument marshalling only: tensors become device pointers, the stream becomes
torch's current CUDA stream unless one is given, and a non-zero status raises
``UspError``.  Every step of the path runs in the library's CUDA kernels; there
is no CPU fallback, and a missing library or a CPU tensor is an error.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libusp.so")
_lib = None

# status codes (include/usp.h)
USP_OK = 0
USP_ERR_INVALID_ARG = 1
USP_ERR_INDIVISIBLE = 2
USP_ERR_UNSUPPORTED = 3
USP_ERR_ALIGNMENT = 4
USP_ERR_BAD_SEQLENS = 5
USP_ERR_BAD_POSITIONS = 6
USP_ERR_TIMEOUT = 7
USP_ERR_CUDA = 8
USP_ERR_WORKSPACE = 9
USP_ERR_BAD_MODS = 10

EXPORTED = [
    "usp_status_string", "usp_version",
    "usp_relayout_fwd", "usp_relayout_bwd", "usp_relayout_fwd_qkv",
    "usp_cu_seqlens_workspace_bytes", "usp_cu_seqlens_from_position_ids",
    "usp_cu_seqlens_from_position_ids_noalloc",
    "usp_attn_fwd", "usp_attn_bwd_workspace_bytes", "usp_attn_bwd",
    "usp_attn_bwd_preprocess", "usp_attn_bwd_dkdv", "usp_attn_bwd_dq",
    "usp_hybrid_relayout_fwd", "usp_hybrid_relayout_bwd", "usp_hybrid_relayout_fwd_qkv",
    "usp_ring_fwd_merge", "usp_ring_grad_accumulate", "usp_attn_bwd_fast_workspace_bytes",
    "usp_a2a_pack_seq_to_head", "usp_a2a_unpack_seq_to_head", "usp_a2a_pack_head_to_seq",
    "usp_a2a_unpack_head_to_seq",
    "usp_rel_buckets_log", "usp_attn_mod_fwd", "usp_attn_mod_bwd_workspace_bytes",
    "usp_attn_mod_bwd_fast_workspace_bytes", "usp_attn_mod_bwd", "usp_attn_mod_bwd_preprocess",
    "usp_attn_mod_bwd_dkdv", "usp_attn_mod_bwd_dq", "usp_attn_mod_bwd_rel_bias",
]

USP_RING_FIRST = 1
USP_RING_LAST = 2


class UspError(RuntimeError):
    def __init__(self, code: int, where: str = ""):
        self.code = int(code)
        super().__init__(f"{where}: {status_string(code)}" if where else status_string(code))


class AttnParams(ctypes.Structure):
    """usp_attn_params (include/usp.h)."""
    _fields_ = [
        ("B", ctypes.c_int), ("S", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
        ("D", ctypes.c_int), ("P", ctypes.c_int), ("causal", ctypes.c_int),
        ("window_left", ctypes.c_int), ("softmax_scale", ctypes.c_float),
        ("cu_seqlens", ctypes.c_void_p), ("n_docs", ctypes.c_void_p), ("sinks", ctypes.c_void_p),
        ("io_layout", ctypes.c_int), ("ring", ctypes.c_int), ("ring_step", ctypes.c_int),
        ("head_first", ctypes.c_int), ("head_count", ctypes.c_int),
    ]


class ScoreModsStruct(ctypes.Structure):
    """usp_score_mods (include/usp.h).  ``tensors`` keeps what its pointers point at, as (field, tensor, type, shape),
    all on ``device`` (None when there is no tensor)."""
    _fields_ = [
        ("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p), ("rel_bias", ctypes.c_void_p),
        ("buckets", ctypes.c_void_p), ("n_buckets", ctypes.c_int), ("max_distance", ctypes.c_int),
        ("rel_bias_grad", ctypes.c_int), ("prefix_lens", ctypes.c_void_p), ("n_prefix", ctypes.c_int),
    ]
    tensors = ()
    device = None

    def point(self):
        """The tensors' addresses of now: a parameter's storage may have been exchanged since the last call (a module
        that is moved to another type keeps its parameters' objects)."""
        for field, t, dtype, shape in self.tensors:
            if t.dtype is not dtype:
                raise TypeError(f"{field} must be {dtype}, it has become {t.dtype}")
            if t.shape != shape or t.device != self.device or not t.is_contiguous():
                raise ValueError(f"{field} has changed its size, strides or device")
            setattr(self, field, t.data_ptr())


USP_IO_HEAD = 0
USP_IO_SEQ = 1
USP_IO_SEQ_KV_HEAD = 2


def lib_path() -> str:
    return _LIB_PATH


def load() -> ctypes.CDLL:
    """Load libusp.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is missing: build it with ulysses_sequence_long_gb300._build.build()")
    L = ctypes.CDLL(_LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.usp_status_string.restype = ctypes.c_char_p
    L.usp_status_string.argtypes = [i32]
    L.usp_version.restype = i32
    L.usp_relayout_fwd.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, vp]
    L.usp_relayout_bwd.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, vp]
    L.usp_relayout_fwd_qkv.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, vp]
    L.usp_cu_seqlens_workspace_bytes.restype = sz
    L.usp_cu_seqlens_workspace_bytes.argtypes = [i32, i32]
    L.usp_cu_seqlens_from_position_ids.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, sz, vp, vp]
    L.usp_cu_seqlens_from_position_ids_noalloc.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, vp]
    L.usp_attn_fwd.argtypes = [ctypes.POINTER(AttnParams), vp, vp, vp, vp, vp, vp, vp]
    L.usp_attn_bwd_workspace_bytes.restype = sz
    L.usp_attn_bwd_workspace_bytes.argtypes = [ctypes.POINTER(AttnParams)]
    L.usp_attn_bwd_fast_workspace_bytes.restype = sz
    L.usp_attn_bwd_fast_workspace_bytes.argtypes = [ctypes.POINTER(AttnParams)]
    L.usp_attn_bwd.argtypes = [ctypes.POINTER(AttnParams), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    L.usp_attn_bwd_preprocess.argtypes = [ctypes.POINTER(AttnParams), vp, vp, vp, vp, vp, sz, vp, vp]
    L.usp_attn_bwd_dkdv.argtypes = [ctypes.POINTER(AttnParams), vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    L.usp_attn_bwd_dq.argtypes = [ctypes.POINTER(AttnParams), vp, vp, vp, vp, vp, vp, vp, sz, vp, vp]
    L.usp_hybrid_relayout_fwd.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, i32, vp]
    L.usp_hybrid_relayout_bwd.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, i32, vp]
    L.usp_hybrid_relayout_fwd_qkv.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32, vp]
    L.usp_ring_fwd_merge.argtypes = [ctypes.POINTER(AttnParams), vp, vp, vp, vp, vp, vp, i32, vp]
    L.usp_ring_grad_accumulate.argtypes = [vp, vp, vp, sz, i32, vp]
    for name in ("usp_a2a_pack_seq_to_head", "usp_a2a_unpack_seq_to_head", "usp_a2a_pack_head_to_seq",
                 "usp_a2a_unpack_head_to_seq"):
        getattr(L, name).argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, vp]
    prm, mods = ctypes.POINTER(AttnParams), ctypes.POINTER(ScoreModsStruct)
    L.usp_rel_buckets_log.argtypes = [i32, i32, i32, vp]
    L.usp_attn_mod_fwd.argtypes = [prm, mods] + [vp] * 7
    for name in ("usp_attn_mod_bwd_workspace_bytes", "usp_attn_mod_bwd_fast_workspace_bytes"):
        getattr(L, name).restype = sz
        getattr(L, name).argtypes = [prm, mods]
    L.usp_attn_mod_bwd.argtypes = [prm, mods] + [vp] * 12 + [sz, vp, vp]
    L.usp_attn_mod_bwd_preprocess.argtypes = [prm, mods] + [vp] * 8 + [sz, vp, vp]
    L.usp_attn_mod_bwd_dkdv.argtypes = [prm, mods] + [vp] * 7 + [sz, vp, vp]
    L.usp_attn_mod_bwd_dq.argtypes = [prm, mods] + [vp] * 6 + [sz, vp, vp]
    L.usp_attn_mod_bwd_rel_bias.argtypes = [prm, mods, vp, vp, sz, vp]
    for name in ("usp_rel_buckets_log", "usp_attn_mod_fwd", "usp_attn_mod_bwd", "usp_attn_mod_bwd_preprocess",
                 "usp_attn_mod_bwd_dkdv", "usp_attn_mod_bwd_dq", "usp_attn_mod_bwd_rel_bias"):
        getattr(L, name).restype = i32
    for name in ("usp_relayout_fwd", "usp_relayout_bwd", "usp_relayout_fwd_qkv",
                 "usp_cu_seqlens_from_position_ids", "usp_cu_seqlens_from_position_ids_noalloc",
                 "usp_attn_fwd", "usp_attn_bwd",
                 "usp_attn_bwd_preprocess", "usp_attn_bwd_dkdv", "usp_attn_bwd_dq",
                 "usp_hybrid_relayout_fwd", "usp_hybrid_relayout_bwd", "usp_hybrid_relayout_fwd_qkv",
                 "usp_ring_fwd_merge", "usp_ring_grad_accumulate", "usp_a2a_pack_seq_to_head",
                 "usp_a2a_unpack_seq_to_head", "usp_a2a_pack_head_to_seq", "usp_a2a_unpack_head_to_seq"):
        getattr(L, name).restype = i32
    _lib = L
    return L


def status_string(code: int) -> str:
    return load().usp_status_string(int(code)).decode()


def _check(rc: int, where: str) -> None:
    if rc != USP_OK:
        raise UspError(rc, where)


def _dev(t: Optional[torch.Tensor], name: str, dtype=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def usp_relayout_fwd(x_seq, x_head, B, S, H, D, P, stream=None):
    _check(load().usp_relayout_fwd(_dev(x_seq, "x_seq"), _dev(x_head, "x_head"), B, S, H, D, P,
                                   x_seq.element_size(), _stream(stream)), "usp_relayout_fwd")


def usp_relayout_bwd(x_head, x_seq, B, S, H, D, P, stream=None):
    _check(load().usp_relayout_bwd(_dev(x_head, "x_head"), _dev(x_seq, "x_seq"), B, S, H, D, P,
                                   x_head.element_size(), _stream(stream)), "usp_relayout_bwd")


def usp_relayout_fwd_qkv(q_seq, k_seq, v_seq, q_head, k_head, v_head, B, S, Hq, Hkv, D, P, stream=None):
    _check(load().usp_relayout_fwd_qkv(_dev(q_seq, "q_seq"), _dev(k_seq, "k_seq"), _dev(v_seq, "v_seq"),
                                       _dev(q_head, "q_head"), _dev(k_head, "k_head"), _dev(v_head, "v_head"),
                                       B, S, Hq, Hkv, D, P, q_seq.element_size(), _stream(stream)),
           "usp_relayout_fwd_qkv")


def usp_cu_seqlens_workspace_bytes(B, S) -> int:
    return int(load().usp_cu_seqlens_workspace_bytes(B, S))


def usp_cu_seqlens_from_position_ids(pos, B, S, P, cu_seqlens, n_docs, max_len, ws, dev_status=None,
                                     stream=None):
    _check(load().usp_cu_seqlens_from_position_ids(
        _dev(pos, "pos", torch.int32), B, S, P, _dev(cu_seqlens, "cu_seqlens", torch.int32),
        _dev(n_docs, "n_docs", torch.int32), _dev(max_len, "max_len", torch.int32), _dev(ws, "ws"),
        ws.numel() * ws.element_size(), _dev(dev_status, "dev_status", torch.int32), _stream(stream)),
        "usp_cu_seqlens_from_position_ids")


def usp_cu_seqlens_from_position_ids_noalloc(pos, B, S, P, cu_seqlens, n_docs, max_len, dev_status=None,
                                             stream=None):
    """The scan without a workspace: its scratch is a fixed array inside the library (B*S <= 2^24)."""
    _check(load().usp_cu_seqlens_from_position_ids_noalloc(
        _dev(pos, "pos", torch.int32), B, S, P, _dev(cu_seqlens, "cu_seqlens", torch.int32),
        _dev(n_docs, "n_docs", torch.int32), _dev(max_len, "max_len", torch.int32),
        _dev(dev_status, "dev_status", torch.int32), _stream(stream)),
        "usp_cu_seqlens_from_position_ids_noalloc")


def attn_params(B, S, Hq, Hkv, D, P, cu_seqlens, n_docs, causal=True, window_left=-1, softmax_scale=0.0,
                sinks=None, io_layout=USP_IO_HEAD, ring=1, ring_step=0, head_first=0, head_count=0) -> AttnParams:
    return AttnParams(B, S, Hq, Hkv, D, P, 1 if causal else 0, window_left, softmax_scale,
                      _dev(cu_seqlens, "cu_seqlens", torch.int32), _dev(n_docs, "n_docs", torch.int32),
                      _dev(sinks, "sinks", torch.float32), int(io_layout), int(ring), int(ring_step),
                      int(head_first), int(head_count))


def usp_attn_fwd(params: AttnParams, q, k, v, o, lse, dev_status=None, stream=None):
    _check(load().usp_attn_fwd(ctypes.byref(params), _dev(q, "q", torch.bfloat16), _dev(k, "k", torch.bfloat16),
                               _dev(v, "v", torch.bfloat16), _dev(o, "o", torch.bfloat16),
                               _dev(lse, "lse", torch.float32), _dev(dev_status, "dev_status", torch.int32),
                               _stream(stream)), "usp_attn_fwd")


def usp_attn_bwd_workspace_bytes(params: AttnParams) -> int:
    return int(load().usp_attn_bwd_workspace_bytes(ctypes.byref(params)))


def usp_attn_bwd_fast_workspace_bytes(params: AttnParams) -> int:
    return int(load().usp_attn_bwd_fast_workspace_bytes(ctypes.byref(params)))


def usp_attn_bwd(params: AttnParams, q, k, v, o, lse, dO, dq, dk, dv, dsinks, ws, dev_status=None, stream=None):
    _check(load().usp_attn_bwd(
        ctypes.byref(params), _dev(q, "q", torch.bfloat16), _dev(k, "k", torch.bfloat16),
        _dev(v, "v", torch.bfloat16), _dev(o, "o", torch.bfloat16), _dev(lse, "lse", torch.float32),
        _dev(dO, "dO", torch.bfloat16), _dev(dq, "dq", torch.bfloat16), _dev(dk, "dk", torch.bfloat16),
        _dev(dv, "dv", torch.bfloat16), _dev(dsinks, "dsinks", torch.float32), _dev(ws, "ws"),
        ws.numel() * ws.element_size(), _dev(dev_status, "dev_status", torch.int32), _stream(stream)),
        "usp_attn_bwd")


def usp_attn_bwd_preprocess(params: AttnParams, o, lse, dO, dsinks, ws, dev_status=None, stream=None):
    _check(load().usp_attn_bwd_preprocess(
        ctypes.byref(params), _dev(o, "o", torch.bfloat16), _dev(lse, "lse", torch.float32),
        _dev(dO, "dO", torch.bfloat16), _dev(dsinks, "dsinks", torch.float32), _dev(ws, "ws"),
        ws.numel() * ws.element_size(), _dev(dev_status, "dev_status", torch.int32), _stream(stream)),
        "usp_attn_bwd_preprocess")


def usp_attn_bwd_dkdv(params: AttnParams, q, k, v, lse, dO, dk, dv, ws, dev_status=None, stream=None):
    _check(load().usp_attn_bwd_dkdv(
        ctypes.byref(params), _dev(q, "q", torch.bfloat16), _dev(k, "k", torch.bfloat16),
        _dev(v, "v", torch.bfloat16), _dev(lse, "lse", torch.float32), _dev(dO, "dO", torch.bfloat16),
        _dev(dk, "dk", torch.bfloat16), _dev(dv, "dv", torch.bfloat16), _dev(ws, "ws"),
        ws.numel() * ws.element_size(), _dev(dev_status, "dev_status", torch.int32), _stream(stream)),
        "usp_attn_bwd_dkdv")


def usp_attn_bwd_dq(params: AttnParams, q, k, v, lse, dO, dq, ws, dev_status=None, stream=None):
    _check(load().usp_attn_bwd_dq(
        ctypes.byref(params), _dev(q, "q", torch.bfloat16), _dev(k, "k", torch.bfloat16),
        _dev(v, "v", torch.bfloat16), _dev(lse, "lse", torch.float32), _dev(dO, "dO", torch.bfloat16),
        _dev(dq, "dq", torch.bfloat16), _dev(ws, "ws"), ws.numel() * ws.element_size(),
        _dev(dev_status, "dev_status", torch.int32), _stream(stream)),
        "usp_attn_bwd_dq")


def usp_hybrid_relayout_fwd(x_seq, x_head, B, S, H, D, ring, ulysses, stream=None):
    _check(load().usp_hybrid_relayout_fwd(_dev(x_seq, "x_seq"), _dev(x_head, "x_head"), B, S, H, D, ring, ulysses,
                                          x_seq.element_size(), _stream(stream)), "usp_hybrid_relayout_fwd")


def usp_hybrid_relayout_bwd(x_head, x_seq, B, S, H, D, ring, ulysses, stream=None):
    _check(load().usp_hybrid_relayout_bwd(_dev(x_head, "x_head"), _dev(x_seq, "x_seq"), B, S, H, D, ring, ulysses,
                                          x_head.element_size(), _stream(stream)), "usp_hybrid_relayout_bwd")


def usp_hybrid_relayout_fwd_qkv(q_seq, k_seq, v_seq, q_head, k_head, v_head, B, S, Hq, Hkv, D, ring, ulysses,
                                stream=None):
    _check(load().usp_hybrid_relayout_fwd_qkv(
        _dev(q_seq, "q_seq"), _dev(k_seq, "k_seq"), _dev(v_seq, "v_seq"), _dev(q_head, "q_head"),
        _dev(k_head, "k_head"), _dev(v_head, "v_head"), B, S, Hq, Hkv, D, ring, ulysses, q_seq.element_size(),
        _stream(stream)), "usp_hybrid_relayout_fwd_qkv")


def usp_ring_fwd_merge(params: AttnParams, o_step, lse_step, o_acc, lse_acc, o, lse, flags, stream=None):
    _check(load().usp_ring_fwd_merge(
        ctypes.byref(params), _dev(o_step, "o_step", torch.bfloat16), _dev(lse_step, "lse_step", torch.float32),
        _dev(o_acc, "o_acc", torch.float32), _dev(lse_acc, "lse_acc", torch.float32), _dev(o, "o", torch.bfloat16),
        _dev(lse, "lse", torch.float32), int(flags), _stream(stream)), "usp_ring_fwd_merge")


def usp_ring_grad_accumulate(g_step, g_acc, g_out, flags, stream=None):
    _check(load().usp_ring_grad_accumulate(
        _dev(g_step, "g_step", torch.bfloat16), _dev(g_acc, "g_acc", torch.float32),
        _dev(g_out, "g_out", torch.bfloat16), g_step.numel(), int(flags), _stream(stream)),
        "usp_ring_grad_accumulate")


def _a2a(name, src, dst, B, S_local, H, D, P, stream):
    _check(getattr(load(), name)(_dev(src, "src"), _dev(dst, "dst"), B, S_local, H, D, P, src.element_size(),
                                 _stream(stream)), name)


def usp_a2a_pack_seq_to_head(x_local, send, B, S_local, H, D, P, stream=None):
    _a2a("usp_a2a_pack_seq_to_head", x_local, send, B, S_local, H, D, P, stream)


def usp_a2a_unpack_seq_to_head(recv, x_head, B, S_local, H, D, P, stream=None):
    _a2a("usp_a2a_unpack_seq_to_head", recv, x_head, B, S_local, H, D, P, stream)


def usp_a2a_pack_head_to_seq(x_head, send, B, S_local, H, D, P, stream=None):
    _a2a("usp_a2a_pack_head_to_seq", x_head, send, B, S_local, H, D, P, stream)


def usp_a2a_unpack_head_to_seq(recv, x_local, B, S_local, H, D, P, stream=None):
    _a2a("usp_a2a_unpack_head_to_seq", recv, x_local, B, S_local, H, D, P, stream)


# -- attention with modified scores ------------------------------------------
def usp_rel_buckets_log(n_buckets: int, max_distance: int, bidirectional: bool) -> torch.Tensor:
    """The bucket of every distance -max_distance..max_distance (int32 host tensor, for ``score_mods``): near
    distances one bucket each, farther ones in buckets of geometrically growing width."""
    out = torch.empty((2 * int(max_distance) + 1 if max_distance > 0 else 1,), dtype=torch.int32)
    _check(load().usp_rel_buckets_log(int(n_buckets), int(max_distance), 1 if bidirectional else 0,
                                      ctypes.c_void_p(out.data_ptr())), "usp_rel_buckets_log")
    return out


def score_mods(Hq, softcap=0.0, slopes=None, rel_bias=None, buckets=None, rel_bias_grad=False,
               prefix_lens=None) -> ScoreModsStruct:
    """usp_score_mods from tensors: slopes fp32 [Hq], rel_bias fp32 [Hq][n_buckets] with buckets int32
    [2*max_distance + 1], prefix_lens int32 [documents]."""
    sl, rb = _dev(slopes, "slopes", torch.float32), _dev(rel_bias, "rel_bias", torch.float32)
    bk, pl = _dev(buckets, "buckets", torch.int32), _dev(prefix_lens, "prefix_lens", torch.int32)
    if slopes is not None and slopes.numel() != Hq:
        raise ValueError(f"slopes must hold one value per query head ({Hq}), got {slopes.numel()}")
    if (rel_bias is None) != (buckets is None):
        raise ValueError("rel_bias and buckets come together")
    if rel_bias is not None:
        if rel_bias.dim() != 2 or rel_bias.shape[0] != Hq or rel_bias.shape[1] < 1:
            raise ValueError(f"rel_bias must be [{Hq}][n_buckets], got {tuple(rel_bias.shape)}")
        if buckets.dim() != 1 or buckets.numel() < 3 or buckets.numel() % 2 != 1:
            raise ValueError("buckets must be [2*max_distance + 1] with max_distance >= 1")
    elif rel_bias_grad:
        raise ValueError("rel_bias_grad needs a rel_bias")
    if prefix_lens is not None and (prefix_lens.dim() != 1 or prefix_lens.numel() < 1):
        raise ValueError("prefix_lens must be [documents]")
    m = ScoreModsStruct(float(softcap), sl, rb, bk, 0 if rel_bias is None else rel_bias.shape[1],
                        0 if buckets is None else (buckets.numel() - 1) // 2, 1 if rel_bias_grad else 0, pl,
                        0 if prefix_lens is None else prefix_lens.numel())
    m.tensors = tuple((f, t, t.dtype, t.shape) for f, t in (("slopes", slopes), ("rel_bias", rel_bias),
                                                            ("buckets", buckets), ("prefix_lens", prefix_lens))
                      if t is not None)
    for _, t, _, _ in m.tensors:
        if m.device is None:
            m.device = t.device
        elif t.device != m.device:
            raise ValueError(f"the tensors of the score modifications are on {m.device} and {t.device}")
    return m


def _mod_sizes(prm: AttnParams, mods: ScoreModsStruct) -> dict:
    """Elements that the parameters ask of each tensor."""
    P, tok = max(prm.P, 1), prm.B * prm.S
    hk = prm.Hkv // P if prm.Hkv >= P else 1
    kv = (prm.Hkv if prm.io_layout == USP_IO_SEQ else P * hk) * tok * prm.D
    return {"q": tok * prm.Hq * prm.D, "kv": kv, "lse": tok * prm.Hq, "heads": prm.Hq, "rel": prm.Hq * mods.n_buckets,
            None: None}


class _Call:
    """The tensors of one call: their sizes against the parameters, one device, that device's stream."""

    __slots__ = ("prm", "mods", "stream", "device", "sizes")

    def __init__(self, prm: AttnParams, mods: ScoreModsStruct, stream):
        self.prm, self.mods, self.stream, self.device, self.sizes = prm, mods, stream, mods.device, None
        mods.point()

    def __call__(self, t, name, dtype, size):
        if t is None:
            return None
        ptr = _dev(t, name, dtype)
        if self.device is None:
            self.device = t.device
        elif t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, other tensors of the call on {self.device}")
        if size is not None:
            if self.sizes is None:
                self.sizes = _mod_sizes(self.prm, self.mods)
            if t.numel() != self.sizes[size]:
                raise ValueError(f"{name} has {t.numel()} elements, the parameters need {self.sizes[size]}")
        return ptr

    def run(self, where, *args):
        stream = _stream(torch.cuda.current_stream(self.device) if self.stream is None else self.stream)
        if torch.cuda.current_device() == self.device.index:
            rc = getattr(load(), where)(ctypes.byref(self.prm), ctypes.byref(self.mods), *args, stream)
        else:
            with torch.cuda.device(self.device):
                rc = getattr(load(), where)(ctypes.byref(self.prm), ctypes.byref(self.mods), *args, stream)
        if rc != USP_OK:
            raise UspError(rc, where)


_BF, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def usp_attn_mod_fwd(params: AttnParams, mods: ScoreModsStruct, q, k, v, o, lse, dev_status=None, stream=None):
    c = _Call(params, mods, stream)
    c.run("usp_attn_mod_fwd", c(q, "q", _BF, "q"), c(k, "k", _BF, "kv"), c(v, "v", _BF, "kv"), c(o, "o", _BF, "q"),
          c(lse, "lse", _F32, "lse"), c(dev_status, "dev_status", _I32, None))


def usp_attn_mod_bwd_workspace_bytes(params: AttnParams, mods: ScoreModsStruct) -> int:
    return int(load().usp_attn_mod_bwd_workspace_bytes(ctypes.byref(params), ctypes.byref(mods)))


def usp_attn_mod_bwd_fast_workspace_bytes(params: AttnParams, mods: ScoreModsStruct) -> int:
    return int(load().usp_attn_mod_bwd_fast_workspace_bytes(ctypes.byref(params), ctypes.byref(mods)))


def usp_attn_mod_bwd(params: AttnParams, mods: ScoreModsStruct, q, k, v, o, lse, dO, dq, dk, dv, dsinks, drel_bias,
                     ws, dev_status=None, stream=None):
    c = _Call(params, mods, stream)
    c.run("usp_attn_mod_bwd", c(q, "q", _BF, "q"), c(k, "k", _BF, "kv"), c(v, "v", _BF, "kv"), c(o, "o", _BF, "q"),
          c(lse, "lse", _F32, "lse"), c(dO, "dO", _BF, "q"), c(dq, "dq", _BF, "q"),
          c(dk, "dk", _BF, "kv"), c(dv, "dv", _BF, "kv"), c(dsinks, "dsinks", _F32, "heads"),
          c(drel_bias, "drel_bias", _F32, "rel"), c(ws, "ws", None, None), ws.numel() * ws.element_size(),
          c(dev_status, "dev_status", _I32, None))


def usp_attn_mod_bwd_preprocess(params: AttnParams, mods: ScoreModsStruct, q, k, v, o, lse, dO, dsinks, ws,
                                dev_status=None, stream=None):
    c = _Call(params, mods, stream)
    c.run("usp_attn_mod_bwd_preprocess", c(q, "q", _BF, "q"), c(k, "k", _BF, "kv"), c(v, "v", _BF, "kv"),
          c(o, "o", _BF, "q"), c(lse, "lse", _F32, "lse"), c(dO, "dO", _BF, "q"), c(dsinks, "dsinks", _F32, "heads"), c(ws, "ws", None, None),
          ws.numel() * ws.element_size(), c(dev_status, "dev_status", _I32, None))


def usp_attn_mod_bwd_dkdv(params: AttnParams, mods: ScoreModsStruct, q, k, v, dO, dk, dv, ws, dev_status=None,
                          stream=None):
    c = _Call(params, mods, stream)
    c.run("usp_attn_mod_bwd_dkdv", c(q, "q", _BF, "q"), c(k, "k", _BF, "kv"), c(v, "v", _BF, "kv"),
          c(dO, "dO", _BF, "q"), c(dk, "dk", _BF, "kv"), c(dv, "dv", _BF, "kv"), c(ws, "ws", None, None),
          ws.numel() * ws.element_size(), c(dev_status, "dev_status", _I32, None))


def usp_attn_mod_bwd_dq(params: AttnParams, mods: ScoreModsStruct, q, k, v, dO, dq, ws, dev_status=None, stream=None):
    c = _Call(params, mods, stream)
    c.run("usp_attn_mod_bwd_dq", c(q, "q", _BF, "q"), c(k, "k", _BF, "kv"), c(v, "v", _BF, "kv"),
          c(dO, "dO", _BF, "q"), c(dq, "dq", _BF, "q"), c(ws, "ws", None, None), ws.numel() * ws.element_size(),
          c(dev_status, "dev_status", _I32, None))


def usp_attn_mod_bwd_rel_bias(params: AttnParams, mods: ScoreModsStruct, drel_bias, ws, stream=None):
    c = _Call(params, mods, stream)
    c.run("usp_attn_mod_bwd_rel_bias", c(drel_bias, "drel_bias", _F32, "rel"), c(ws, "ws", None, None),
          ws.numel() * ws.element_size())
