"""Attention with modified scores at the ends of its parameters' ranges, forward
and backward, against the fp64 restatement of ``oracle.score_mods``.  Tolerances
as in ``test_gpu_score_mods``, with the roundings of P, dX and O to bf16 left out
element by element (`*_slack`): gradients scale with the softmax scale."""
import numpy as np
import pytest
import torch

import usp_workloads as W
from gpu_util import assert_close, built_lib
from oracle import score_mods as SM
from test_gpu_score_mods import _device_mods, _f32_close, _np, _w

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    built_lib()


def _layer(w, kw, scale=0.0, **more):
    from ulysses_sequence_long_gb300.pipeline import Shape, UlyssesAttention
    return UlyssesAttention(Shape(w.B, w.S, w.Hq, w.Hkv, w.D, w.P, w.causal, w.window_left, scale),
                            mods=_device_mods(kw), **more)


def _step(ua, t, pos, sinks=None):
    d = {n: x.cuda() for n, x in t.items()}
    ua.forward(d["q"], d["k"], d["v"], torch.from_numpy(pos).cuda(), sinks)
    ua.backward(d["do"], sinks)
    torch.cuda.synchronize()
    assert ua.read_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("softcap,scale", [(2.0 ** -10, 2.0), (2.0 ** -10, 0.5), (0.25, 1024.0), (4.0, 0.25),
                                           (2.0 ** 10, 2.0 ** -4), (2.0 ** 10, 8.0), (1.0, 2.0 ** 40),
                                           (2.0 ** -10, 2.0 ** 100)])
def test_any_ratio_of_scale_and_cap(D, softcap, scale):
    """Whatever the cap and the softmax scale are: scores whose deviation is a quarter of the cap (a block's largest
    lies between half the cap and a little beyond it), or 1 where the cap is far above that."""
    w = _w("ratio", S=256, Hq=4, Hkv=2, D=D, P=2, doc_mode="explicit", doc_lens=(100, 156))
    t = W.qkv_do_shards(w)
    pos = W.position_ids_shards(w)
    t["q"] = (t["q"].double() * (min(0.25 * softcap, 1.0) / scale / D ** 0.5)).to(torch.bfloat16)
    t["do"] = (t["do"].double() * min(1.0, 1.0 / scale)).to(torch.bfloat16)   # keeps dQ's values in fp32
    kw = dict(softcap=softcap)
    ua = _layer(w, kw, scale)
    _step(ua, t, pos)
    host = {n: W.bf16_to_f64(x) for n, x in t.items()}
    ref = SM.mod_layer(host["q"], host["k"], host["v"], pos, host["do"], scale=scale, **kw)
    assert_close("o", _np(ua.o_seq), ref["o"])
    assert_close("lse", _np(ua.lse), ref["lse"], bf16_out=False)
    # (dq and dk carry the scale and the queries' size: bounds in units of their largest value)
    for n, x in (("dq", ua.dq_seq), ("dk", ua.dk_seq), ("dv", ua.dv_seq)):
        top = np.abs(ref[n]).max()
        if n != "dv" and top / scale < 2.0 ** -126:
            # sum dX q (or k) before the scale: below the smallest normal fp32 number, as dX (here 2^-100) times q
            # (2^-115) is under a scale of 2^100.  It may be lost; it adds at most itself.
            assert np.abs(_np(x)).max() <= 2.0 * top
            continue
        assert_close(n, _np(x) / top, ref[n] / top, slack=ref[n + "_slack"] / top)


@pytest.mark.parametrize("low", [-np.inf, float(np.finfo(np.float32).min)])
def test_a_sink_of_no_weight_where_a_row_sees_nothing(low):
    """Head 0 has a sink of no weight and a table that hides every key of some rows: those rows' weights are all
    zero, and so is what they add to the sink's gradient."""
    w = _w("no_sink", S=384, Hq=2, Hkv=1, D=64, P=1, sinks=True, doc_mode="explicit", doc_lens=(150, 234))
    t = W.qkv_do_shards(w)
    pos = W.position_ids_shards(w)
    rb = np.random.default_rng(0).standard_normal((2, 8)).astype(np.float32).astype(np.float64)
    rb[0, 0] = rb[0, -1] = -np.inf
    kw = dict(rel_bias=rb, buckets=SM.rel_buckets_log(8, 20, False))
    sinks = np.array([low, 0.5])
    ua = _layer(w, kw)
    _step(ua, t, pos, torch.tensor(sinks, dtype=torch.float32).cuda())
    host = {n: W.bf16_to_f64(x) for n, x in t.items()}
    # (-1e30 is a sink without weight too, and keeps the restatement's logarithms finite)
    ref = SM.mod_layer(host["q"], host["k"], host["v"], pos, host["do"], sinks=np.array([-1e30, 0.5]), **kw)
    none = ref["lse"] == -1e30
    assert none.any() and np.array_equal(np.isneginf(_np(ua.lse)), none)
    assert float(ua.dsinks[0]) == 0.0
    _f32_close("dsinks", ua.dsinks, ref["dsinks"])
    _f32_close("drel_bias", ua.drel_bias, ref["drel_bias"])
    for n, x in (("o", ua.o_seq), ("dq", ua.dq_seq), ("dk", ua.dk_seq), ("dv", ua.dv_seq)):
        assert_close(n, _np(x), ref[n])


def test_threads_with_tables_of_different_reach():
    """Two host threads, each with its own layer, tensors and stream: a table that reaches 5 tokens and one that reaches
    2048 take the same kernel with different amounts of shared memory.  Neither thread's calls may fail."""
    import threading
    w = _w("threads", S=128, Hq=2, Hkv=1, D=64, P=1)
    t = W.qkv_do_shards(w)
    pos = torch.from_numpy(W.position_ids_shards(w)).cuda()
    d = {n: x.cuda() for n, x in t.items()}
    rng = np.random.default_rng(0)
    layers = [_layer(w, dict(rel_bias=rng.standard_normal((2, 8)), buckets=SM.rel_buckets_log(8, R, False)))
              for R in (5, 2048)]
    torch.cuda.synchronize()
    failed = []

    def work(ua):
        try:
            stream = torch.cuda.Stream()
            for i in range(4000):
                ua.forward(d["q"], d["k"], d["v"], pos, stream=stream)
                if i % 100 == 99:
                    stream.synchronize()
        except Exception as e:  # noqa: BLE001 (reported below, in the test's thread)
            failed.append(e)

    threads = [threading.Thread(target=work, args=(ua,)) for ua in layers]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    torch.cuda.synchronize()
    assert not failed, failed
    assert all(ua.read_status() == 0 for ua in layers)


@pytest.mark.parametrize("D,causal", [(64, True), (128, True), (64, False)])
def test_slopes_below_zero(D, causal):
    """Slopes below 0 put the weights on the farthest keys, where the bias is largest.  An exponent carries, in units of
    2^-24 |slope| d: the rounding of slope log2e, of its product with the distance, of their sum with the score's part,
    and of the LSE and its product with log2e: 5 half steps, and 1.2e-5 of the rest (see test_gpu_score_mods).  With
    P' = P (1 + e), |e| <= eps: |dX' - dX| <= eps P (|dP| + |D| + sum_u P |dP|)."""
    w = _w("below_zero", S=1536, Hq=4, Hkv=2, D=D, P=2, causal=causal, doc_mode="explicit", doc_lens=(1400, 136))
    t = W.qkv_do_shards(w)
    pos = W.position_ids_shards(w)
    slopes = np.array([-0.5, -2.0 ** -5, 2.0 ** -3, -0.125])
    table = np.random.default_rng(2).standard_normal((4, 32)).astype(np.float32).astype(np.float64)
    kw = dict(slopes=slopes, rel_bias=table, buckets=SM.rel_buckets_log(32, 128, not causal))
    ua = _layer(w, kw)
    _step(ua, t, pos)
    host = {n: W.bf16_to_f64(x) for n, x in t.items()}
    ref = SM.mod_layer(host["q"], host["k"], host["v"], pos, host["do"], causal=causal, **kw)
    assert_close("o", _np(ua.o_seq), ref["o"])
    assert_close("lse", _np(ua.lse), ref["lse"], bf16_out=False)
    for n, x in (("dq", ua.dq_seq), ("dk", ua.dk_seq), ("dv", ua.dv_seq)):
        assert_close(n, _np(x), ref[n], slack=ref[n + "_slack"])
    flat = {n: np.moveaxis(x, 0, 1).reshape(w.S, -1, D) for n, x in host.items()}
    lse = np.moveaxis(ref["lse"], 0, 1).reshape(4, w.S)
    bound = np.zeros_like(table)
    for h in range(4):
        for a, b in ((0, 1400), (1400, 1536)):
            at = np.arange(b - a)
            dist = at[:, None] - at[None, :]
            bucket = kw["buckets"][np.clip(dist, -128, 128) + 128]
            x = flat["q"][a:b, h] @ flat["k"][a:b, h // 2].T / D ** 0.5 - slopes[h] * np.abs(dist) + table[h][bucket]
            p = np.where((dist >= 0) | (not causal), np.exp(np.minimum(x - lse[h, a:b, None], 0.0)), 0.0)
            dp = flat["do"][a:b, h] @ flat["v"][a:b, h // 2].T
            eps = 5 * 2.0 ** -24 * abs(slopes[h]) * (b - a + 128) + 1.2e-5
            some = p * (np.abs(dp) + np.abs((p * dp).sum(1))[:, None] + (p * np.abs(dp)).sum(1)[:, None])
            bound[h] += eps * np.bincount(bucket.reshape(-1), some.reshape(-1), 32)
    err = np.abs(_np(ua.drel_bias) - ref["drel_bias"])
    print(f"[parity] drel_bias: worst error / bound {np.max(err / np.maximum(bound, 1e-30)):.3f}")
    assert np.all(err <= bound)
