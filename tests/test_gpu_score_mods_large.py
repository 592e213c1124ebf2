"""Attention with modified scores where many tiles and heads meet: the kernels as
long sequences run them (two query tiles per CTA, several query heads per CTA of
dK/dV and clusters that share them, several units per CTA of the pass for D),
against the fp64 restatement.  Documents of a few hundred tokens keep that cheap.
Tolerances as in ``test_gpu_score_mods``."""
import dataclasses
import functools
import json

import numpy as np
import pytest
import torch

import usp_workloads as W
from gpu_util import assert_close, built_lib
from oracle import score_mods as SM
from test_gpu_score_mods import Case, _f32_close, _inputs, _layer, _np, _run, _w

pytestmark = pytest.mark.gpu

DOCS = (700, 1, 300, 129, 640, 256, 511, 3, 900, 912)            # 4352 tokens: 34 tiles of 128
PREFIX = (350, 1, 0, 129, 500, 7, 300, 1, 450, 10 ** 6)


@dataclasses.dataclass(frozen=True)
class Large:
    case: Case
    tiles: int          # query tiles per CTA of the forward
    halves: int         # threads that share a row
    split: int          # CTAs of a cluster that share a key tile's query heads (exchanges fused)
    heads: int          # query heads of a CTA of dK/dV


def _l(name, tiles, halves, split, heads, S=4352, Hq=16, Hkv=4, D=128, P=2, docs=DOCS, **kw):
    keys = ("sinks", "causal", "window_left", "B")
    w = _w(name, S=S, Hq=Hq, Hkv=Hkv, D=D, P=P, **({"doc_lens": docs} if docs else {}), **{k: kw.pop(k) for k in keys if k in kw})
    return Large(Case(w, **kw), tiles, halves, split, heads)


LARGE = [
    _l("cap", 2, 2, 2, 2, softcap=30.0, gain=3.0, sinks=True),
    _l("cap_d64", 2, 2, 1, 2, D=64, Hkv=8, softcap=20.0, gain=3.0, sinks=True),
    _l("cap_wide_window", 2, 2, 2, 2, softcap=80.0, gain=3.0, window_left=600),
    _l("cap_saturated_d64", 2, 2, 2, 2, D=64, softcap=1.5, gain=3.0, window_left=520),
    _l("slopes", 2, 1, 2, 2, slopes=True, sinks=True),
    _l("slopes_bidir_d64", 2, 1, 2, 2, D=64, slopes=True, causal=False),
    _l("rel", 2, 1, 1, 2, Hkv=8, rel=(32, 128), sinks=True),
    _l("rel_bidir_d64", 2, 1, 1, 4, Hq=32, Hkv=8, D=64, rel=(32, 400), causal=False),
    _l("rel_rows", 2, 1, 2, 2, B=3, S=1280, docs=(500, 1, 779), P=1, rel=(16, 40), sinks=True),
    _l("prefix", 2, 1, 2, 2, prefix=PREFIX),
    _l("all", 2, 2, 2, 2, gain=3.0, softcap=30.0, slopes=True, rel=(32, 128), prefix=PREFIX, sinks=True),
    _l("all_d64", 2, 2, 1, 4, Hq=32, Hkv=8, D=64, gain=3.0, softcap=50.0, slopes=True, rel=(32, 64), prefix=PREFIX,
       sinks=True),
    # one key/value head: clusters of 8, with one query head each and with two
    _l("group8", 1, 2, 8, 1, S=1024, Hq=8, Hkv=1, P=2, docs=(400, 624), gain=3.0, softcap=30.0, slopes=True, rel=(32, 128),
       sinks=True),
    _l("group16_d64", 1, 2, 8, 2, S=1024, Hq=16, Hkv=1, D=64, P=4, docs=(700, 324), rel=(32, 128), sinks=True),
]


@functools.lru_cache(maxsize=2)
def _reference(i):
    c = LARGE[i].case
    t, pos, kw = _inputs(c)
    host = {n: W.bf16_to_f64(x) for n, x in t.items()}
    return SM.mod_layer(host["q"], host["k"], host["v"], pos, host["do"], causal=c.w.causal, window_left=c.w.window_left,
                        **kw)


@pytest.mark.parametrize("i,fused,stored_ds", [(i, f, d) for i in range(len(LARGE))
                                               for f, d in ((True, True), (True, False), (False, True))],
                         ids=[f"{x.case.w.name}-{n}" for x in LARGE for n in ("fused", "recompute", "explicit")])
def test_parity_of_many_tiles(i, fused, stored_ds):
    c = LARGE[i].case
    t, pos, kw = _inputs(c)
    ua = _layer(c, kw, fused=fused, stored_ds=stored_ds)
    _run(c, ua, t, pos, kw)
    ref = _reference(i)
    assert_close("o", _np(ua.o_seq), ref["o"])
    assert_close("lse", _np(ua.lse), ref["lse"], bf16_out=False)
    slack = {n: ref[n + "_slack"] for n in ("dq", "dk", "dv")}
    if not fused and c.w.Hkv < c.w.P:
        # partial dK/dV of a replicated head: half a step of each, the sum of magnitudes at most 4 x the largest
        for n in ("dk", "dv"):
            slack[n] = slack[n] + c.w.P // c.w.Hkv * 2.0 ** -9 * 2.0 * np.abs(ref[n]).max()
    for n, x in (("dq", ua.dq_seq), ("dk", ua.dk_seq), ("dv", ua.dv_seq)):
        assert_close(n, _np(x), ref[n], slack=slack[n])
    if "sinks" in kw:
        _f32_close("dsinks", ua.dsinks, ref["dsinks"])
    if "rel_bias" in kw:
        _f32_close("drel_bias", ua.drel_bias, ref["drel_bias"])


def _launches(run, path):
    """(kernel, blocks) of the launches of ``run``."""
    from torch.profiler import ProfilerActivity, profile
    for _ in range(2):      # (a process's first recording may come back empty)
        with profile(activities=[ProfilerActivity.CUDA]) as p:
            run()
            torch.cuda.synchronize()
        p.export_chrome_trace(str(path))
        events = json.load(open(path))["traceEvents"]
        got = [(e["name"], e["args"]["grid"][0]) for e in events if e.get("cat") == "kernel"]
        if got:
            break
    return got


@pytest.mark.parametrize("i", range(len(LARGE)), ids=[x.case.w.name for x in LARGE])
def test_the_variants_these_cases_are_for(i, tmp_path):
    """A rule that sends a case to another variant is to bring another case for this one.  (152 SMs.)"""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if sms != 152:
        pytest.skip("the cases are made for 152 SMs")
    x = LARGE[i]
    w = x.case.w
    t, pos, kw = _inputs(x.case)
    ua = _layer(x.case, kw, fused=True, stored_ds=True)
    _run(x.case, ua, t, pos, kw)
    got = _launches(lambda: _run(x.case, ua, t, pos, kw), tmp_path / "trace.json")
    if not got:
        pytest.skip("no records of the launches here")
    one = lambda part: next((n, g) for n, g in got if part in n)
    assert f"attn_fwd_kernel<{w.D}, {x.tiles}, {x.halves}," in one("attn_fwd_kernel")[0]
    name, blocks = one("dkdv_kernel")
    n_tiles = -(-w.B * w.S // 128)
    assert blocks == n_tiles * w.Hkv * x.split and f", {'true' if x.split > 1 else 'false'}>(" in name
    assert x.split * x.heads == w.Hq // w.Hkv
    if "sinks" in kw or "rel_bias" in kw:
        assert one("delta_kernel")[1] == min(sms, n_tiles * w.Hq)
