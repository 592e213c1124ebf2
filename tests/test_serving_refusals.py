"""Rotary positions, the paged cache and the attention of single tokens: what the
library and the Python layers refuse before anything runs on a device, and the oracle they are compared with."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import serving as OS

P = ctypes.c_void_p
A, Bq, Cq, Dq = P(1 << 20), P(1 << 30), P(1 << 40), P(1 << 41)


@pytest.fixture(scope="module")
def lib():
    from ulysses_sequence_long_gb300 import _build, binding
    _build.build()
    return binding.load()


def _rope(**kw):
    from ulysses_sequence_long_gb300 import binding as B
    d = dict(tokens=10, Hq=4, Hkv=2, D=64, n_axes=1, n_pos=10, n_pairs=32, interleaved=0, positions=16, freqs=16, axes=None)
    d.update(kw)
    return B.RopeParams(*d.values())


def test_rope_refusals(lib):
    from ulysses_sequence_long_gb300 import binding as B

    def rc(q=A, k=Bq, qo=Cq, ko=Dq, **kw):
        codes = {f(ctypes.byref(_rope(**kw)), q, k, qo, ko, None, None) for f in (lib.usp_rope_fwd, lib.usp_rope_bwd)}
        assert len(codes) == 1
        return codes.pop()
    bad = B.USP_ERR_INVALID_ARG
    assert lib.usp_rope_fwd(None, A, Bq, Cq, Dq, None, None) == bad
    for kw in (dict(tokens=0), dict(Hq=0), dict(Hkv=-1), dict(n_axes=0), dict(n_pos=0), dict(n_pairs=0), dict(positions=None),
               dict(freqs=None), dict(interleaved=2), dict(q=None), dict(qo=None), dict(k=None), dict(ko=None),
               dict(Hkv=0), dict(qo=P((1 << 20) + 16)), dict(qo=Bq), dict(ko=A), dict(ko=Cq), dict(tokens=-5, n_pos=-5)):
        assert rc(**kw) == bad, kw
    assert rc(n_pos=3) == B.USP_ERR_INDIVISIBLE
    for kw in (dict(D=96), dict(D=256), dict(n_pairs=12), dict(n_pairs=40), dict(n_axes=9), dict(Hq=4095),
               dict(tokens=1 << 30, n_pos=1)):
        assert rc(**kw) == B.USP_ERR_UNSUPPORTED, kw
    for kw in (dict(q=P((1 << 20) + 8)), dict(ko=P((1 << 41) + 2)), dict(positions=18), dict(freqs=17), dict(axes=2)):
        assert rc(**kw) == B.USP_ERR_ALIGNMENT, kw


def _cache(**kw):
    from ulysses_sequence_long_gb300 import binding as B
    d = dict(P=2, Hkv=4, D=64, n_pages=10, page_size=16, n_seqs=3, max_pages=4, dtype=B.USP_CACHE_BF16, k_pages=1 << 30,
             v_pages=1 << 31, k_scales=None, v_scales=None, block_table=16, lens=16)
    d.update(kw)
    return B.PagedCacheStruct(*d.values())


def test_cache_refusals(lib):
    from ulysses_sequence_long_gb300 import binding as B
    e = dict(dtype=B.USP_CACHE_E4M3, k_scales=1 << 20, v_scales=1 << 21)

    def rc(k=A, v=Dq, tokens=3, cu=None, Hq=8, ws=Cq, ws_bytes=None, **kw):
        c = _cache(**kw)
        codes = [f(ctypes.byref(c), k, v, tokens, cu, None, None) for f in (lib.usp_cache_append, lib.usp_cache_read)]
        n = lib.usp_attn_decode_workspace_bytes(ctypes.byref(c), Hq)
        codes.append(lib.usp_attn_decode(ctypes.byref(c), Hq, -1, 0.0, None, A, Cq, Dq, ws, n - 1, None, None))
        assert (n == 0) == (codes[2] != B.USP_ERR_WORKSPACE)
        return codes
    for f in (lib.usp_cache_append, lib.usp_cache_read):
        assert f(None, A, Bq, 3, None, None, None) == B.USP_ERR_INVALID_ARG
        for args in ((None, None, 3, None), (A, Dq, 0, None), (A, Dq, -1, P(16)), (A, Dq, 4, None)):
            assert f(ctypes.byref(_cache()), *args, None, None) == B.USP_ERR_INVALID_ARG, args
        assert f(ctypes.byref(_cache()), P(8), Bq, 3, None, None, None) == B.USP_ERR_ALIGNMENT
        assert f(ctypes.byref(_cache()), A, Bq, 3, P(6), None, None) == B.USP_ERR_ALIGNMENT
        assert f(ctypes.byref(_cache()), A, Bq, 1 << 30, P(16), None, None) == B.USP_ERR_UNSUPPORTED
        inside = P((1 << 31) + 2 * 4 * 64 * 10 * 16 - 16)         # the last bytes of the values' pool
        assert f(ctypes.byref(_cache()), inside, Bq, 3, None, None, None) == B.USP_ERR_INVALID_ARG
        assert f(ctypes.byref(_cache()), A, inside, 3, None, None, None) == B.USP_ERR_INVALID_ARG
    assert lib.usp_cache_read(ctypes.byref(_cache()), A, P((1 << 20) + 16), 3, None, None, None) == B.USP_ERR_INVALID_ARG
    eight = _cache(**e)
    for f in (lib.usp_cache_append, lib.usp_cache_read):          # 640 scales each; table and lengths
        for p in ((1 << 20) + 624, 1 << 21, 16):
            assert f(ctypes.byref(eight), P(p), None, 3, None, None, None) == B.USP_ERR_INVALID_ARG
    assert lib.usp_cache_read(ctypes.byref(_cache()), Dq, None, 3, P((1 << 41) + 4), None, None) == B.USP_ERR_INVALID_ARG
    for kw in (dict(P=0), dict(Hkv=0), dict(D=0), dict(n_pages=0), dict(page_size=0), dict(n_seqs=0), dict(max_pages=0),
               dict(dtype=2), dict(k_pages=None), dict(v_pages=None), dict(block_table=None), dict(lens=None),
               dict(k_scales=1 << 20), dict(dtype=B.USP_CACHE_E4M3), dict(e, v_scales=None)):
        assert set(rc(**kw)) == {B.USP_ERR_INVALID_ARG}, kw
    for kw in (dict(P=3), dict(P=8, Hkv=3), dict(Hkv=3)):
        assert set(rc(**kw)) == {B.USP_ERR_INDIVISIBLE}, kw
    for kw in (dict(D=96), dict(page_size=24), dict(page_size=8), dict(n_pages=1 << 30), dict(max_pages=1 << 26),
               dict(n_seqs=1 << 20)):
        assert set(rc(**kw)) == {B.USP_ERR_UNSUPPORTED}, kw
    for kw in (dict(k_pages=(1 << 30) + 8), dict(e, k_scales=(1 << 20) + 1), dict(block_table=18), dict(lens=17)):
        assert set(rc(**kw)) == {B.USP_ERR_ALIGNMENT}, kw


def test_decode_refusals(lib):
    from ulysses_sequence_long_gb300 import binding as B
    c = _cache()
    n = lib.usp_attn_decode_workspace_bytes(ctypes.byref(c), 8)
    assert n > 0

    def rc(Hq=8, window=-1, scale=0.0, sinks=None, q=A, o=Bq, lse=Dq, ws=Cq, n=n):
        return lib.usp_attn_decode(ctypes.byref(c), Hq, window, scale, sinks, q, o, lse, ws, n, None, None)
    for kw in (dict(Hq=0), dict(q=None), dict(o=None), dict(lse=None), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(o=A), dict(o=P((1 << 20) + 64)), dict(lse=A), dict(lse=Bq)):
        assert rc(**kw) == B.USP_ERR_INVALID_ARG, kw
    for h in (6, 7, 2):
        assert rc(Hq=h) == B.USP_ERR_INDIVISIBLE and lib.usp_attn_decode_workspace_bytes(ctypes.byref(c), h) == 0
    assert rc(Hq=1028) == B.USP_ERR_UNSUPPORTED and rc(window=-2) == B.USP_ERR_UNSUPPORTED
    assert rc(q=P((1 << 20) + 2)) == B.USP_ERR_ALIGNMENT and rc(sinks=P(2)) == B.USP_ERR_ALIGNMENT
    assert rc(lse=P((1 << 41) + 2)) == B.USP_ERR_ALIGNMENT
    # what is written lies on nothing else (rows: 24 of 64)
    table, lens, sinks = c.block_table, c.lens, P(1 << 22)
    c.block_table, c.lens = 1 << 23, 1 << 24
    far = dict(q=P(1 << 42), o=P(1 << 43), lse=P(1 << 44), ws=P(1 << 45), sinks=sinks)
    for name, at in (("o", 24 * 64 * 2), ("lse", 24 * 4), ("ws", n)):
        ends_in = [p - (at + 15) // 16 * 16 + 16 for p in (c.k_pages, c.v_pages, c.block_table, c.lens, 1 << 22, 1 << 42)]
        begins_in = [c.v_pages + 2 * 4 * 64 * 10 * 16 - 16, c.block_table + 32, (1 << 42) + 24 * 64 * 2 - 16]
        if name == "ws":
            ends_in, begins_in = [(p + 255) // 256 * 256 for p in ends_in], [p // 256 * 256 for p in begins_in]
        for p in ends_in + begins_in:
            assert rc(**dict(far, **{name: P(p)})) == B.USP_ERR_INVALID_ARG, (name, hex(p))
    assert rc(**dict(far, ws=P((1 << 43) - n // 512 * 256))) == rc(**dict(far, ws=P((1 << 44) - n // 512 * 256))) == B.USP_ERR_INVALID_ARG
    c.block_table, c.lens = table, lens
    assert rc(ws=None) == rc(ws=P((1 << 40) + 16)) == rc(n=n - 1) == B.USP_ERR_WORKSPACE


def test_status_names(lib):
    from ulysses_sequence_long_gb300 import binding as B
    assert "ROPE" in B.status_string(B.USP_ERR_BAD_ROPE) and "PAGES" in B.status_string(B.USP_ERR_BAD_PAGES)


def test_cpu_tensors_are_refused(lib):
    from ulysses_sequence_long_gb300.pipeline import Rotary
    from ulysses_sequence_long_gb300.serving import PagedCache
    with pytest.raises(TypeError):
        Rotary(torch.ones(32))
    with pytest.raises(TypeError):
        PagedCache(4, 16, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        PagedCache(4, 16, 3, 64, P=2)


# ---- the oracle
def test_oracle_rounding_to_e4m3_is_torchs():
    rng = np.random.default_rng(0)
    x = torch.from_numpy(rng.standard_normal((50, 64)) * 10.0 ** rng.integers(-30, 30, (50, 1))).to(torch.bfloat16)
    y, e = OS.to_e4m3(x.double().numpy())
    assert (np.abs(x.double().numpy()).max(-1) <= 448 * np.exp2(e.astype(float))).all()
    assert (np.abs(x.double().numpy()).max(-1) > 224 * np.exp2(e.astype(float)))[e > -126].all()
    want = (x.double() / torch.from_numpy(np.exp2(e.astype(float)))[:, None]).float().to(torch.float8_e4m3fn)
    assert np.array_equal(want.double().numpy(), y)
    y, e = OS.to_e4m3(np.array([[np.inf, np.nan, 1.0, -np.inf], [448.0, 0, 0, 0], [450.0, 0, 0, 0], [0, 0, 0, 0.0]]))
    assert e.tolist() == [120, 0, 1, -126] and y[0, 0] == 448 and np.isnan(y[0, 1]) and y[0, 3] == -448


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_gradient_of_the_rotation_is_that_of_differences(interleaved):
    """sum(dy . y(x)) for one element of x at a time: the rotation is linear, so a difference of any width is exact."""
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((2, 3, 2, 64))
    pos, f, ax = rng.integers(-50, 5000, (2, 3)), rng.uniform(0, 1, 24), rng.integers(0, 2, 24)
    dx, _ = OS.rope(dy, pos, f, ax, interleaved, back=True)
    for _ in range(200):
        i = tuple(rng.integers(0, n) for n in x.shape)
        up = x.copy()
        up[i] += 1.0
        diff = ((OS.rope(up, pos, f, ax, interleaved)[0] - OS.rope(x, pos, f, ax, interleaved)[0]) * dy).sum()
        assert abs(diff - dx[i]) < 1e-12


def test_kernels_that_are_launched_early_wait_first():
    """As the library's other chained kernels: grid_wait before any load (of global memory), no read-only loads."""
    import os
    import re
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ulysses_sequence_long_gb300", "csrc")
    for name, kernel in (("usp_rope.cu", "rope_kernel"), ("usp_cache.cu", "cache_kernel"), ("usp_decode.cu", "decode_kernel")):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(csrc, name)).read())
        bodies = text.split("__global__")[1:]
        assert len(bodies) == 1 and kernel in bodies[0] and "launch_chained(" in text
        before, wait, _ = bodies[0].partition("grid_wait()")
        assert wait and "gld(" not in before and "atom" not in before
        assert "__ldg(" not in text and not re.search(r"const\s+\w+\s*\*\s*__restrict__", text)
