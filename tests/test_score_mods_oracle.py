"""Pins of the fp64 restatement of attention with modified scores, and the
refusals of the C entry points (no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest

import oracle
import usp_workloads as W
from oracle import score_mods as SM
from ulysses_sequence_long_gb300 import binding as B


@pytest.fixture(scope="module")
def lib():
    from ulysses_sequence_long_gb300 import _build
    _build.build()
    return B.load()


def _inputs(T, Hq, Hkv, D, seed):
    r = np.random.default_rng(seed)
    return [r.standard_normal((T, h, D)) for h in (Hq, Hkv, Hkv, Hq)]


def test_without_mods_it_is_the_plain_attention():
    w = W.Workload("plain", B=2, S=96, Hq=4, Hkv=2, D=8, P=2, window_left=20, sinks=True, doc_mode="geometric",
                   doc_mean=30, seed=4)
    t = {n: W.bf16_to_f64(x) for n, x in W.qkv_do_shards(w).items()}
    pos, snk = W.position_ids_shards(w), W.sinks(w).double().numpy()
    f = oracle.ulysses_fwd(t["q"], t["k"], t["v"], pos, True, 20, None, snk)
    g = oracle.ulysses_bwd(f, t["do"], True, 20, None, snk)
    r = SM.mod_layer(t["q"], t["k"], t["v"], pos, t["do"], window_left=20, sinks=snk)
    for got, want in ((r["o"], f["o_seq"]), (r["lse"], f["lse"]), (r["dq"], g["dq_seq"]), (r["dk"], g["dk_seq"]),
                      (r["dv"], g["dv_seq"]), (r["dsinks"], g["dsinks"])):
        assert np.max(np.abs(got - want)) <= 1e-12 * max(1.0, np.max(np.abs(want)))


MODS = [
    dict(softcap=2.0),
    dict(slopes=True, causal=False),
    dict(rel=(6, 5), window_left=9, sinks=True),
    dict(softcap=1.5, slopes=True, rel=(8, 12), prefix=True, sinks=True),
]


def _kwargs(spec, Hq, n_docs, seed):
    r = np.random.default_rng(seed + 1)
    kw = {k: spec[k] for k in ("softcap", "causal", "window_left") if k in spec}
    if spec.get("slopes"):
        kw["slopes"] = 2.0 ** -np.arange(1, Hq + 1)
    if spec.get("rel"):
        nb, R = spec["rel"]
        kw["rel_bias"] = r.standard_normal((Hq, nb))
        kw["buckets"] = SM.rel_buckets_log(nb, R, True)
    if spec.get("prefix"):
        kw["prefix_lens"] = r.integers(0, 12, n_docs)
    if spec.get("sinks"):
        kw["sinks"] = r.standard_normal(Hq)
    return kw


@pytest.mark.parametrize("spec", MODS, ids=[str(i) for i in range(len(MODS))])
def test_gradients_against_differences(spec):
    T, Hq, Hkv, D = 23, 4, 2, 8
    cu = np.array([0, 1, 9, 23])
    q, k, v, do = _inputs(T, Hq, Hkv, D, 3)
    kw = _kwargs(spec, Hq, 3, 3)
    r = SM.mod_attention(q, k, v, cu, do=do, **kw)

    def loss():
        return (SM.mod_attention(q, k, v, cu, **kw)["o"] * do).sum()

    pick = np.random.default_rng(5)
    pairs = [(q, r["dq"]), (k, r["dk"]), (v, r["dv"])]
    pairs += [(kw["rel_bias"], r["drel_bias"])] if "rel_bias" in kw else []
    pairs += [(kw["sinks"], r["dsinks"])] if "sinks" in kw else []
    for x, g in pairs:
        for _ in range(12):
            at = tuple(pick.integers(0, n) for n in x.shape)
            old, h = x[at], 1e-5
            x[at] = old + h
            up = loss()
            x[at] = old - h
            down = loss()
            x[at] = old
            # central difference: O(h^2) truncation and 1e-16/h rounding
            assert abs((up - down) / (2 * h) - g[at]) <= 1e-7 * max(1.0, abs(g[at]))


def test_visible_keys_of_a_prefix():
    m = SM.visible_mask(6, True, -1, 3)
    assert np.array_equal(m, np.tril(np.ones((6, 6), bool)) | (np.arange(6) < 3)[None, :])
    assert np.array_equal(SM.visible_mask(6, True, 2, 3)[5], [False, False, False, True, True, True])
    assert SM.visible_mask(6, True, -1, 99).all()


@pytest.mark.parametrize("nb,R,both", [(32, 128, False), (32, 128, True), (32, 64, True), (8, 2048, False),
                                       (2, 5, False), (4, 2, True), (33, 400, False), (64, 1024, True)])
def test_bucket_map(lib, nb, R, both):
    got = B.usp_rel_buckets_log(nb, R, both).numpy()
    assert np.array_equal(got, SM.rel_buckets_log(nb, R, both))
    K = nb // 2 if both else nb
    up = got[R:]
    assert up[0] == 0 and up[-1] == K - 1 and np.all(np.diff(up) >= 0) and np.all(np.diff(up[:K // 2]) == 1)
    assert np.array_equal(got[:R][::-1], up[1:] + K if both else np.zeros(R))


def test_bucket_map_refusals(lib):
    buf = (ctypes.c_int32 * 64)()
    f = lib.usp_rel_buckets_log
    assert f(8, 16, 0, None) == B.USP_ERR_INVALID_ARG
    assert f(8, 16, 2, buf) == B.USP_ERR_INVALID_ARG
    assert f(9, 16, 1, buf) == B.USP_ERR_INVALID_ARG       # odd, both ways
    assert f(1, 16, 0, buf) == B.USP_ERR_INVALID_ARG
    assert f(2, 16, 1, buf) == B.USP_ERR_INVALID_ARG       # one bucket a side
    assert f(32, 16, 0, buf) == B.USP_ERR_INVALID_ARG      # no room past the single ones
    assert f(32, 4096, 0, buf) == B.USP_ERR_UNSUPPORTED


def _params(S=256, causal=1, w=-1, io=0, ring=1, hc=0, D=64):
    return B.AttnParams(1, S, 4, 2, D, 2, causal, w, 0.0, 16, 16, None, io, ring, 0, 0, hc)


def _mods(cap=0.0, slopes=None, rel=None, buckets=None, nb=0, R=0, grad=0, prefix=None, np_=0):
    return B.ScoreModsStruct(cap, slopes, rel, buckets, nb, R, grad, prefix, np_)


def test_refusals_of_the_entry_points(lib):
    """Every check returns before the device is touched (the pointers are made up)."""
    p, ws = ctypes.c_void_p(16), ctypes.c_void_p(1 << 20)
    ref = ctypes.byref

    def fwd(prm=None, mods=None, q=p, o=p):
        return lib.usp_attn_mod_fwd(ref(prm or _params()), ref(mods or _mods()), q, p, p, o, p, None, None)

    def bwd(prm=None, mods=None, drel=None, ws=ws, n=1 << 30, dq=p):
        return lib.usp_attn_mod_bwd(ref(prm or _params()), ref(mods or _mods()), p, p, p, p, p, p, dq, p, p, None, drel,
                                     ws, n, None, None)

    INV, UNS, ALI, WSP = B.USP_ERR_INVALID_ARG, B.USP_ERR_UNSUPPORTED, B.USP_ERR_ALIGNMENT, B.USP_ERR_WORKSPACE
    rel = dict(rel=16, buckets=16, nb=8, R=16)
    bad = [
        (INV, dict(cap=-1.0)), (INV, dict(cap=math.nan)), (INV, dict(cap=math.inf)),
        (UNS, dict(cap=1e-6)), (UNS, dict(cap=2000.0)),
        (INV, dict(rel, buckets=None)), (INV, dict(rel, nb=0)), (INV, dict(rel, R=0)), (INV, dict(rel, grad=2)),
        (UNS, dict(rel, R=2049)), (UNS, dict(rel, nb=5000)),
        (INV, dict(buckets=16)), (INV, dict(nb=3)), (INV, dict(R=3)), (INV, dict(grad=1)),
        (INV, dict(prefix=16, np_=0)), (INV, dict(np_=2)),
        (ALI, dict(slopes=18)), (ALI, dict(rel, rel=18)), (ALI, dict(rel, buckets=18)), (ALI, dict(prefix=18, np_=1)),
    ]
    for code, spec in bad:
        m = _mods(**spec)
        assert fwd(mods=m) == code, spec
        assert bwd(mods=m) == code, spec
        assert lib.usp_attn_mod_bwd_workspace_bytes(ref(_params()), ref(m)) == 0
    pre = _mods(prefix=16, np_=4)
    assert fwd(_params(causal=0), pre) == INV                       # a prefix without causal order
    assert fwd(_params(S=512, ring=2)) == UNS and bwd(_params(S=512, ring=2)) == UNS
    assert fwd(_params(D=96)) == UNS
    assert lib.usp_attn_mod_fwd(ref(_params()), None, p, p, p, p, p, None, None) == INV
    assert fwd(q=None) == INV and fwd(q=ctypes.c_void_p(18)) == ALI and fwd(o=ctypes.c_void_p(18)) == ALI
    assert fwd(_params(io=1, hc=1)) == INV and bwd(_params(io=1, hc=1)) == INV
    assert bwd(_params(io=2)) == UNS
    # the table's gradient is asked for exactly when it has a place
    assert bwd(mods=_mods(**rel, grad=1)) == INV and bwd(mods=_mods(**rel), drel=p) == INV
    assert bwd(ws=None) == WSP and bwd(n=16) == WSP and bwd(ws=ctypes.c_void_p(1 << 20 | 16)) == WSP
    assert bwd(dq=None) == INV
    f = lib.usp_attn_mod_bwd_rel_bias
    assert f(ref(_params()), ref(_mods(**rel)), p, ws, 1 << 30, None) == INV
    assert f(ref(_params()), ref(_mods(**rel, grad=1)), None, ws, 1 << 30, None) == INV


def test_workspace_sizes(lib):
    """Statistics, then rows by distance, then partial sums, then the stored dS blocks of the mask."""
    ref = ctypes.byref
    stats = lib.usp_attn_bwd_workspace_bytes(ref(_params()))
    n = lambda prm, m: (lib.usp_attn_mod_bwd_workspace_bytes(ref(prm), ref(m)),
                        lib.usp_attn_mod_bwd_fast_workspace_bytes(ref(prm), ref(m)))
    cap = _mods(cap=30.0)
    blk = 128 * 64 * 2
    assert n(_params(), cap) == (stats, stats + 4 * (4 + 2) * blk)        # 2 key tiles meet 4 and 2 slices, 4 heads
    assert n(_params(causal=0), cap) == (stats, stats + 4 * 8 * blk)      # every pair
    assert n(_params(), _mods(prefix=16, np_=1)) == (stats, stats + 4 * 8 * blk)
    assert n(_params(S=250), cap)[1] == 0
    # a window that spans the row is none
    assert n(_params(w=10 ** 9), cap) == n(_params(), cap)
    up = lambda x: -(-x // 256) * 256
    rel = dict(rel=16, buckets=16, nb=8, R=16)
    rows = up(4 * 4 * (2 * (16 + 160) + 1))
    assert n(_params(), _mods(**rel))[0] == stats + rows
    part = up(4 * 4 * 32 * 33) + up(4 * 4 * 1 * 33)                       # 8 blocks of 32 keys, 4 quarters; 1 split
    assert n(_params(), _mods(**rel, grad=1))[0] == stats + rows + part
