"""GPU parity of attention with modified scores (tanh cap, linear and learned
bias by distance, prefix mask), forward and backward, against the fp64
restatement of ``oracle.score_mods``.

Tolerances.  bf16 outputs: the bar of the plain attention (max-abs 2e-2 without
the output's own rounding, relative L2 5e-3).  That max-abs is set for scores of
unit size; where the queries are scaled up (`gain`), so are the gradients, and the
roundings of P, dX and O to bf16 that the kernels take are left out element by
element (`*_slack` of the restatement, where the bound is derived); the relative
L2 stays.  dsinks and drel_bias (fp32): the
weights P carry the error of the exponent, |z2| 2^-23 for |z2| <= 64 plus tanh's
1.3e-7 c log2e, times ln 2: under 1.2e-5 for c <= 80, and D, a sum of P dP, no more;
both are random over a sum's terms: relative L2 2e-5 over the table or the sinks.
"""
import dataclasses

import numpy as np
import pytest
import torch

import oracle
import usp_workloads as W
from gpu_util import assert_close, built_lib
from oracle import score_mods as SM

pytestmark = pytest.mark.gpu

F32_REL = 2e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    built_lib()


@dataclasses.dataclass(frozen=True)
class Case:
    w: W.Workload
    gain: float = 1.0            # factor of the queries
    softcap: float = 0.0
    slopes: bool = False
    rel: tuple = ()              # (n_buckets, max_distance)
    rel_inf: bool = False        # -inf in the table: buckets that hide their keys
    prefix: tuple = ()           # prefix lengths
    sink_shift: float = 0.0
    train: bool = True


def _w(name, **kw):
    kw.setdefault("doc_mode", "explicit" if "doc_lens" in kw else "single")
    kw.setdefault("B", 1)
    return W.Workload(name, **kw)


CASES = [
    # one token, documents of one token, odd lengths; D = 64 and 128
    Case(_w("cap_one_token", S=1, Hq=2, Hkv=1, D=64, P=1), softcap=5.0, train=False),
    Case(_w("cap_odd_docs", S=333, Hq=4, Hkv=2, D=64, P=1, doc_lens=(1, 100, 231, 1)), softcap=30.0, gain=3.0),
    # scores far beyond the cap: tanh leaves the polynomial
    Case(_w("cap_saturated", S=256, Hq=4, Hkv=2, D=128, P=2), softcap=1.5, gain=3.0),
    # a cap too wide for the fixed reference, and a sink above every capped score
    Case(_w("cap_wide", S=512, Hq=4, Hkv=4, D=128, P=2, sinks=True), softcap=80.0, gain=3.0),
    Case(_w("cap_high_sink", S=256, Hq=4, Hkv=2, D=64, P=1, sinks=True), softcap=10.0, sink_shift=14.0),
    Case(_w("cap_window", S=1024, Hq=8, Hkv=2, D=64, P=2, window_left=127, sinks=True, doc_lens=(300, 1, 723)),
         softcap=20.0, gain=3.0),
    Case(_w("cap_window_d128", S=640, B=2, Hq=4, Hkv=2, D=128, P=1, window_left=0), softcap=20.0, train=False),
    Case(_w("cap_bidir", S=300, Hq=2, Hkv=1, D=128, P=1, causal=False, doc_lens=(120, 180)), softcap=20.0, gain=3.0),
    Case(_w("cap_many_ranks", S=1024, Hq=8, Hkv=2, D=64, P=4, doc_lens=(500, 524)), softcap=30.0),
    Case(_w("slope_rows", S=258, B=3, Hq=4, Hkv=4, D=64, P=2, doc_mode="geometric", doc_mean=90, seed=6), slopes=True),
    Case(_w("slope_bidir", S=512, Hq=4, Hkv=2, D=128, P=1, causal=False, doc_lens=(200, 312)), slopes=True),
    Case(_w("slope_window_sinks", S=768, Hq=4, Hkv=2, D=128, P=2, window_left=200, sinks=True), slopes=True),
    # a table that ends inside a tile, one that ends past the row, one that never reaches its end
    Case(_w("rel_short", S=512, Hq=4, Hkv=2, D=64, P=2, doc_lens=(40, 300, 172)), rel=(6, 5)),
    Case(_w("rel_odd", S=333, Hq=2, Hkv=2, D=128, P=1, sinks=True), rel=(32, 77)),
    Case(_w("rel_long", S=512, Hq=2, Hkv=1, D=128, P=1), rel=(64, 2048)),
    Case(_w("rel_window", S=512, Hq=4, Hkv=2, D=64, P=1, window_left=130), rel=(32, 128)),
    Case(_w("rel_bidir", S=640, B=2, Hq=4, Hkv=2, D=64, P=1, causal=False, doc_mode="geometric", doc_mean=200, seed=2),
         rel=(32, 128)),
    Case(_w("rel_bidir_window", S=512, Hq=2, Hkv=2, D=128, P=2, causal=False, window_left=90), rel=(16, 40)),
    Case(_w("rel_many_ranks", S=1024, Hq=8, Hkv=2, D=128, P=4, doc_lens=(700, 324)), rel=(32, 128)),
    Case(_w("rel_hides", S=384, Hq=2, Hkv=1, D=64, P=1, doc_lens=(150, 234)), rel=(8, 20), rel_inf=True),
    # prefixes of nothing, of a part, of all and of more than the document; documents of one token
    Case(_w("prefix", S=640, Hq=4, Hkv=2, D=64, P=1, doc_lens=(1, 200, 139, 299, 1)), prefix=(1, 0, 77, 1000, 0)),
    Case(_w("prefix_d128", S=768, Hq=4, Hkv=2, D=128, P=2, doc_lens=(500, 268)), prefix=(350, 268)),
    Case(_w("prefix_window", S=512, Hq=4, Hkv=4, D=128, P=1, window_left=60, sinks=True, doc_lens=(300, 212)),
         prefix=(250, 130)),
    Case(_w("prefix_odd_rows", S=333, B=2, Hq=4, Hkv=2, D=64, P=1, doc_mode="single"), prefix=(200, 17)),
    Case(_w("all", S=768, Hq=8, Hkv=2, D=128, P=2, sinks=True, doc_lens=(1, 400, 367)), gain=3.0, softcap=30.0,
         slopes=True, rel=(32, 128), prefix=(1, 150, 60)),
    Case(_w("all_d64", S=501, Hq=4, Hkv=2, D=64, P=1, sinks=True, doc_lens=(250, 251)), gain=3.0, softcap=50.0,
         slopes=True, rel=(32, 64), prefix=(30, 251)),
    Case(_w("none", S=512, Hq=4, Hkv=2, D=128, P=2, sinks=True, doc_lens=(130, 382))),
]
MODES = [(c, f, d) for c in CASES for f in ([False, True] if (c.w.S // c.w.P) % 128 == 0 else [False])
         for d in (([True, False] if c.w.S % 128 == 0 else [False]) if c.train else [None])]


def _inputs(c: Case):
    w = c.w
    t = W.qkv_do_shards(w)
    t["q"] = (t["q"].float() * c.gain).to(torch.bfloat16)
    pos = W.position_ids_shards(w)
    rng = np.random.default_rng(w.S + w.Hq)
    kw = {}
    if w.sinks:
        kw["sinks"] = (W.sinks(w) + c.sink_shift).double().numpy()
    if c.softcap:
        kw["softcap"] = c.softcap
    if c.slopes:
        kw["slopes"] = (2.0 ** (-8.0 * np.arange(1, w.Hq + 1) / w.Hq)).astype(np.float32).astype(np.float64)
    if c.rel:
        both = not w.causal or bool(c.prefix)
        kw["buckets"] = SM.rel_buckets_log(c.rel[0], c.rel[1], both)
        rb = rng.standard_normal((w.Hq, c.rel[0])).astype(np.float32)
        if c.rel_inf:
            rb[0, 0] = rb[0, -1] = -np.inf    # a row that sees only itself or only far keys sees nothing
            rb[1, 2] = -np.inf
        kw["rel_bias"] = rb.astype(np.float64)
    if c.prefix:
        kw["prefix_lens"] = np.array(c.prefix, dtype=np.int32)
    return t, pos, kw


def _device_mods(kw, **more):
    from ulysses_sequence_long_gb300.pipeline import ScoreMods
    dev = lambda n, dt: torch.tensor(kw[n], dtype=dt).cuda() if n in kw else None
    return ScoreMods(softcap=kw.get("softcap", 0.0), slopes=dev("slopes", torch.float32),
                     rel_bias=dev("rel_bias", torch.float32), buckets=dev("buckets", torch.int32),
                     prefix_lens=dev("prefix_lens", torch.int32), **more)


def _layer(c: Case, kw, **more):
    from ulysses_sequence_long_gb300.pipeline import Shape, UlyssesAttention
    w = c.w
    return UlyssesAttention(Shape(w.B, w.S, w.Hq, w.Hkv, w.D, w.P, w.causal, w.window_left), with_backward=c.train,
                            mods=_device_mods(kw), **more)


def _run(c: Case, ua, t, pos, kw):
    d = {n: x.cuda() for n, x in t.items()}
    sinks = torch.tensor(kw["sinks"], dtype=torch.float32).cuda() if "sinks" in kw else None
    ua.forward(d["q"], d["k"], d["v"], torch.from_numpy(pos).cuda(), sinks)
    if c.train:
        ua.backward(d["do"], sinks)
    torch.cuda.synchronize()
    assert ua.read_status() == 0
    return d, sinks


def _np(x):
    return x.double().cpu().numpy()


def _f32_close(name, got, want):
    rel = np.linalg.norm(_np(got) - want) / np.linalg.norm(want)
    print(f"[parity] {name}: rel_l2={rel:.3e}")
    assert rel <= F32_REL, (name, rel)


@pytest.mark.parametrize("c,fused,stored_ds", MODES, ids=[
    f"{c.w.name}-{'fused' if f else 'explicit'}" + {True: "-stored", False: "-recompute", None: ""}[d]
    for c, f, d in MODES])
def test_parity(c, fused, stored_ds):
    t, pos, kw = _inputs(c)
    ua = _layer(c, kw, fused=fused, stored_ds=stored_ds)
    _run(c, ua, t, pos, kw)
    host = {n: W.bf16_to_f64(x) for n, x in t.items()}
    ref = SM.mod_layer(host["q"], host["k"], host["v"], pos, host["do"] if c.train else None, causal=c.w.causal,
                       window_left=c.w.window_left, **kw)
    assert_close("o", _np(ua.o_seq), ref["o"])
    lse = _np(ua.lse)
    empty = np.isneginf(ref["lse"])
    assert np.array_equal(np.isneginf(lse), empty) and empty.any() == c.rel_inf
    assert_close("lse", lse[~empty], ref["lse"][~empty], bf16_out=False)
    if not c.train:
        return
    sq = sk = sv = None
    if c.gain > 1.0:
        sq, sk, sv = (ref[n + "_slack"] for n in ("dq", "dk", "dv"))
    if not fused and c.w.Hkv < c.w.P:
        # each rank's partial dK/dV of a replicated head is rounded to bf16 before the exchange sums them: half
        # a step of |partial| each, of which the sum of magnitudes is at most 4 x the largest value here
        assert c.gain == 1.0
        reps = c.w.P // c.w.Hkv
        sk, sv = (np.full(ref[n].shape, reps * 2.0 ** -9 * 2.0 * np.abs(ref[n]).max()) for n in ("dk", "dv"))
    assert_close("dq", _np(ua.dq_seq), ref["dq"], slack=sq)
    assert_close("dk", _np(ua.dk_seq), ref["dk"], slack=sk)
    assert_close("dv", _np(ua.dv_seq), ref["dv"], slack=sv)
    if "sinks" in kw:
        _f32_close("dsinks", ua.dsinks, ref["dsinks"])
    if "rel_bias" in kw:
        _f32_close("drel_bias", ua.drel_bias, ref["drel_bias"])
        # buckets that no visible pair has get exactly nothing
        none = ref["drel_bias"] == 0
        assert np.all(_np(ua.drel_bias)[none] == 0)


def test_without_mods_equals_the_plain_attention():
    """No cap, bias or prefix: the plain attention.  The row sums join in another order (half a row at a time):
    the LSE differs by the roundings of at most 512 positive terms added in chains of at most 128, under 128 half
    steps of the sum, 128 2^-24 = 7.6e-6 of its logarithm, and a rounding of the result (below 8: 2.4e-7)."""
    from ulysses_sequence_long_gb300.pipeline import Shape, UlyssesAttention
    c = next(x for x in CASES if x.w.name == "none")
    t, pos, kw = _inputs(c)
    ua = _layer(c, kw, fused=False)
    d, sinks = _run(c, ua, t, pos, kw)
    w = c.w
    plain = UlyssesAttention(Shape(w.B, w.S, w.Hq, w.Hkv, w.D, w.P), fused=False)
    plain.forward(d["q"], d["k"], d["v"], torch.from_numpy(pos).cuda(), sinks)
    torch.cuda.synchronize()
    assert (plain.lse - ua.lse).abs().max().item() <= 8e-6
    assert_close("o", _np(ua.o_seq), _np(plain.o_seq))


def test_head_groups_and_repeats_give_the_same_bits():
    """Stored dS a key/value head at a time, and a second run on the same buffers: nothing is left over from
    one pass to the next, and no sum depends on the schedule."""
    c = next(x for x in CASES if x.w.name == "all")
    t, pos, kw = _inputs(c)
    one = _layer(c, kw, fused=True, stored_ds=True)
    _run(c, one, t, pos, kw)
    grads = lambda ua: [x.clone() for x in (ua.o_seq, ua.lse, ua.dq_seq, ua.dk_seq, ua.dv_seq, ua.dsinks, ua.drel_bias)]
    first = grads(one)
    one._bwd_ws.fill_(0xFF)
    _run(c, one, t, pos, kw)
    parts = _layer(c, kw, fused=True, ds_group_size=1)
    _run(c, parts, t, pos, kw)
    assert len(parts.ds_groups) == c.w.Hkv
    for a, b, g in zip(first, grads(one), grads(parts)):
        assert torch.equal(a, b) and torch.equal(a, g)


def test_table_updates_and_a_frozen_table():
    """The layer reads the table at every call; without its gradient the other gradients stay the same."""
    c = next(x for x in CASES if x.w.name == "rel_short")
    t, pos, kw = _inputs(c)
    mods = _device_mods(kw)
    from ulysses_sequence_long_gb300.pipeline import ScoreMods, Shape, UlyssesAttention
    w = c.w
    shape = Shape(w.B, w.S, w.Hq, w.Hkv, w.D, w.P)
    ua = UlyssesAttention(shape, mods=mods)
    _run(c, ua, t, pos, kw)
    mods.rel_bias.mul_(-2.0)
    _run(c, ua, t, pos, kw)
    host = {n: W.bf16_to_f64(x) for n, x in t.items()}
    kw2 = dict(kw, rel_bias=-2.0 * kw["rel_bias"])
    ref = SM.mod_layer(host["q"], host["k"], host["v"], pos, host["do"], **kw2)
    assert_close("o", _np(ua.o_seq), ref["o"])
    _f32_close("drel_bias", ua.drel_bias, ref["drel_bias"])
    frozen = UlyssesAttention(shape, mods=dataclasses.replace(mods, rel_bias_grad=False))
    _run(c, frozen, t, pos, kw2)
    assert not hasattr(frozen, "drel_bias")
    assert_close("dq", _np(frozen.dq_seq), ref["dq"])
    assert_close("dk", _np(frozen.dk_seq), ref["dk"])


def test_exchanged_storage_of_a_table():
    """A parameter whose storage is exchanged between calls is read where it is now; another size is refused."""
    c = next(x for x in CASES if x.w.name == "rel_short")
    t, pos, kw = _inputs(c)
    from ulysses_sequence_long_gb300.pipeline import Shape, UlyssesAttention
    w = c.w
    mods = _device_mods(kw)
    mods.rel_bias = torch.nn.Parameter(mods.rel_bias)
    ua = UlyssesAttention(Shape(w.B, w.S, w.Hq, w.Hkv, w.D, w.P), mods=mods)
    _run(c, ua, t, pos, kw)
    old = mods.rel_bias.data
    mods.rel_bias.data = old * -2.0
    old.fill_(5.0)
    d, _ = _run(c, ua, t, pos, kw)
    host = {n: W.bf16_to_f64(x) for n, x in t.items()}
    ref = SM.mod_layer(host["q"], host["k"], host["v"], pos, host["do"], **dict(kw, rel_bias=-2.0 * kw["rel_bias"]))
    assert_close("o", _np(ua.o_seq), ref["o"])
    _f32_close("drel_bias", ua.drel_bias, ref["drel_bias"])
    mods.rel_bias.data = old[:, :-1].contiguous()
    with pytest.raises(ValueError):
        ua.forward(d["q"], d["k"], d["v"], torch.from_numpy(pos).cuda())


def test_captured_and_replayed_on_another_stream():
    """A captured training step replays on new inputs and gives what the eager calls give."""
    c = next(x for x in CASES if x.w.name == "all")
    t, pos, kw = _inputs(c)
    ua = _layer(c, kw)
    d, sinks = _run(c, ua, t, pos, kw)     # warm-up: allocations and first launches
    dpos = torch.from_numpy(pos).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ua.forward(d["q"], d["k"], d["v"], dpos, sinks)
        ua.backward(d["do"], sinks)
    for x in d.values():
        x.copy_(x.flip(0).neg())           # other inputs, in place
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in (ua.o_seq, ua.lse, ua.dq_seq, ua.dk_seq, ua.dv_seq, ua.dsinks, ua.drel_bias)]
    other = _layer(c, kw)
    with torch.cuda.stream(side):
        other.forward(d["q"], d["k"], d["v"], dpos, sinks)
        other.backward(d["do"], sinks)
    torch.cuda.synchronize()
    want = (other.o_seq, other.lse, other.dq_seq, other.dk_seq, other.dv_seq, other.dsinks, other.drel_bias)
    assert ua.read_status() == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_two_layers_together():
    """A capped window layer whose output feeds a layer with a learned bias and a prefix, forward and backward:
    the gradients of the first layer's inputs through both."""
    wa = _w("stack", S=512, Hq=4, Hkv=2, D=64, P=2, window_left=150, sinks=True, doc_lens=(200, 312))
    a = Case(wa, softcap=20.0, gain=3.0)
    b = Case(dataclasses.replace(wa, window_left=-1, sinks=False, seed=1), rel=(32, 128), prefix=(50, 312))
    ta, pos, ka = _inputs(a)
    tb, _, kb = _inputs(b)
    la, lb = _layer(a, ka), _layer(b, kb)
    dev = {n: x.cuda() for n, x in ta.items()}
    devb = {n: x.cuda() for n, x in tb.items()}
    dpos, sinks = torch.from_numpy(pos).cuda(), torch.tensor(ka["sinks"], dtype=torch.float32).cuda()
    mid = la.forward(dev["q"], dev["k"], dev["v"], dpos, sinks)
    lb.forward(mid, devb["k"], devb["v"], dpos)               # the queries of the second layer
    dmid, dkb, _ = lb.backward(devb["do"])
    dq, dk, dv = la.backward(dmid, sinks)
    torch.cuda.synchronize()
    assert la.read_status() == 0 and lb.read_status() == 0
    h, hb = ({n: W.bf16_to_f64(x) for n, x in y.items()} for y in (ta, tb))
    ra = SM.mod_layer(h["q"], h["k"], h["v"], pos, None, window_left=150, **ka)
    # what passes between the layers is bf16: the reference takes the values that passed
    rb = SM.mod_layer(_np(mid), hb["k"], hb["v"], pos, hb["do"], **kb)
    ra2 = SM.mod_layer(h["q"], h["k"], h["v"], pos, _np(dmid), window_left=150, **ka)
    assert_close("mid", _np(mid), ra["o"])
    assert_close("o", _np(lb.o_seq), rb["o"])
    assert_close("dmid", _np(dmid), rb["dq"])
    assert_close("dkb", _np(dkb), rb["dk"])
    _f32_close("drel_bias", lb.drel_bias, rb["drel_bias"])
    for n, x in (("dq", dq), ("dk", dk), ("dv", dv)):
        assert_close(n, _np(x), ra2[n], slack=ra2[n + "_slack"])
    _f32_close("dsinks", la.dsinks, ra2["dsinks"])


def test_masks_of_the_lowest_value_hide_as_infinities_do():
    """A table's entries far below any score: the same bits whatever their value, rows without a key among them."""
    c = next(x for x in CASES if x.w.name == "rel_hides")
    t, pos, kw = _inputs(c)
    got = []
    for low in (-np.inf, np.finfo(np.float32).min, -2.0 ** 20 - 1):
        kx = dict(kw, rel_bias=np.where(np.isneginf(kw["rel_bias"]), low, kw["rel_bias"]))
        ua = _layer(c, kx)
        _run(c, ua, t, pos, kx)
        got.append([x.clone() for x in (ua.o_seq, ua.lse, ua.dq_seq, ua.dk_seq, ua.dv_seq, ua.drel_bias)])
    assert torch.isneginf(got[0][1]).any()
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b)


@pytest.mark.parametrize("n_buckets,R", [(1, 1), (3, 1), (4097, 2048), (5, 160)])
@pytest.mark.parametrize("S,D", [(1, 64), (1, 128), (129, 128), (257, 64)])
def test_any_bucket_map(n_buckets, R, S, D):
    """Bucket maps without order, from one bucket to one for every distance, sequences from one token; with
    slopes and a prefix of the whole sequence, so that every distance of both signs is met."""
    rng = np.random.default_rng(R + S)
    c = Case(_w("map", S=S, Hq=4, Hkv=2, D=D, P=1, sinks=True), slopes=True, rel=(2, 2), prefix=(S,))
    t, pos, kw = _inputs(c)
    kw["buckets"] = rng.integers(0, n_buckets, 2 * R + 1).astype(np.int32)
    kw["rel_bias"] = rng.standard_normal((4, n_buckets)).astype(np.float32).astype(np.float64)
    ua = _layer(c, kw)
    _run(c, ua, t, pos, kw)
    host = {n: W.bf16_to_f64(x) for n, x in t.items()}
    ref = SM.mod_layer(host["q"], host["k"], host["v"], pos, host["do"], **kw)
    for n, x in (("o", ua.o_seq), ("dq", ua.dq_seq), ("dk", ua.dk_seq), ("dv", ua.dv_seq)):
        if S > 1 or n in ("o", "dv"):
            assert_close(n, _np(x), ref[n])
        else:
            # one key and the sink: dX = P (1 - P) dO.v, and D from O's rounding has no part in it here (fp32 pass)
            assert_close(n, _np(x), ref[n], slack=ref[n + "_slack"])
    assert_close("lse", _np(ua.lse), ref["lse"], bf16_out=False)
    _f32_close("dsinks", ua.dsinks, ref["dsinks"])
    _f32_close("drel_bias", ua.drel_bias, ref["drel_bias"])
    assert np.all(_np(ua.drel_bias)[ref["drel_bias"] == 0] == 0)


@pytest.mark.parametrize("D,P,causal", [(64, 1, True), (128, 2, True), (128, 1, False)])
@pytest.mark.parametrize("mod", ["cap", "slopes", "none"])
def test_one_visible_key_has_no_score_gradient(D, P, causal, mod):
    """A window of 0: every row sees itself alone, so O = v and dQ = dK = 0.  P is exactly 1 in the forward, O = v in
    bf16, and D = dO.v differs from dP by the orders of two fp32 sums over D terms, each within D 2^-24 sum |dO v| <
    128 6e-8 200 = 1.6e-3 of the value; P of the backward is 1 to 1e-5.  Times scale |k| < 0.125 * 5, and for dK twice
    (two query heads)."""
    c = Case(_w("alone", S=512, Hq=4, Hkv=2, D=D, P=P, causal=causal, window_left=0),
             softcap=20.0 if mod == "cap" else 0.0, slopes=mod == "slopes")
    t, pos, kw = _inputs(c)
    ua = _layer(c, kw)
    _run(c, ua, t, pos, kw)
    v = t["v"].repeat_interleave(2, dim=3)
    assert torch.equal(ua.o_seq.cpu(), v)
    assert ua.dq_seq.abs().max().item() <= 2e-3 * 0.625 and ua.dk_seq.abs().max().item() <= 4e-3 * 0.625


@pytest.mark.parametrize("name", ["cap_window", "slope_window_sinks", "rel_many_ranks", "all"])
def test_keys_and_values_moved_first(name):
    """What a sequence beyond KV_IN_PLACE_TOKENS takes: k and v in head layout for the forward."""
    c = next(x for x in CASES if x.w.name == name)
    t, pos, kw = _inputs(c)
    ua = _layer(c, kw, fused=True)
    assert ua._kv_in_place
    ua._kv_in_place = False
    _run(c, ua, t, pos, kw)
    host = {n: W.bf16_to_f64(x) for n, x in t.items()}
    ref = SM.mod_layer(host["q"], host["k"], host["v"], pos, host["do"], window_left=c.w.window_left, **kw)
    assert_close("o", _np(ua.o_seq), ref["o"])
    assert_close("lse", _np(ua.lse), ref["lse"], bf16_out=False)
    for n, x in (("dq", ua.dq_seq), ("dk", ua.dk_seq), ("dv", ua.dv_seq)):
        assert_close(n, _np(x), ref[n], slack=ref[n + "_slack"])


def test_back_to_back_steps_see_the_step_before():
    """Steps queued without a wait between them, each on the outputs of the one before and with a table that the
    step before updates: the same bits as with a wait after every call (the launches overlap their set-up only)."""
    c = next(x for x in CASES if x.w.name == "all")
    t, pos, kw = _inputs(c)
    dpos, sinks = torch.from_numpy(pos).cuda(), torch.tensor(kw["sinks"], dtype=torch.float32).cuda()

    def steps(wait):
        mods = _device_mods(kw)
        from ulysses_sequence_long_gb300.pipeline import Shape, UlyssesAttention
        w = c.w
        ua = UlyssesAttention(Shape(w.B, w.S, w.Hq, w.Hkv, w.D, w.P, w.causal, w.window_left), mods=mods)
        d = {n: x.cuda() for n, x in t.items()}
        for _ in range(8):
            ua.forward(d["q"], d["k"], d["v"], dpos, sinks)
            wait()
            ua.backward(d["do"], sinks)
            wait()
            d["q"].copy_(ua.o_seq).add_(ua.dq_seq)
            d["k"].add_(ua.dk_seq)
            d["do"].copy_(ua.o_seq)
            mods.rel_bias.sub_(ua.drel_bias, alpha=1e-3)
            wait()
        torch.cuda.synchronize()
        assert ua.read_status() == 0
        return [x.clone() for x in (ua.o_seq, ua.lse, d["q"], d["k"], ua.dv_seq, ua.dsinks, mods.rel_bias)]

    for a, b in zip(steps(torch.cuda.synchronize), steps(lambda: None)):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)


def test_values_beyond_the_limits_are_reported():
    """Biases and slopes that are too large or NaN: a status, no fault."""
    from ulysses_sequence_long_gb300 import binding as Bd
    for name, key, values in (("rel_short", "rel_bias", (np.nan, np.inf, 2.0 ** 21)),
                              ("slope_rows", "slopes", (np.nan, np.inf, -2.0 ** 11))):
        c = next(x for x in CASES if x.w.name == name)
        t, pos, kw = _inputs(c)
        for v in values:
            bad = kw[key].copy()
            bad.reshape(-1)[0] = v
            ua = _layer(c, dict(kw, **{key: bad}))
            d = {n: x.cuda() for n, x in t.items()}
            ua.forward(d["q"], d["k"], d["v"], torch.from_numpy(pos).cuda())
            torch.cuda.synchronize()
            assert ua.read_status() == Bd.USP_ERR_BAD_MODS


def test_bad_data_is_reported():
    """A bucket id outside the table, a negative prefix length, too few prefix lengths: a status, no fault."""
    from ulysses_sequence_long_gb300 import binding as Bd
    c = next(x for x in CASES if x.w.name == "rel_short")
    t, pos, kw = _inputs(c)
    for bad in (dict(kw, buckets=np.where(np.arange(11) == 7, 6, kw["buckets"])),
                dict(kw, buckets=np.where(np.arange(11) == 7, -1, kw["buckets"])),
                dict(kw, prefix_lens=np.array([3, -1, 4])), dict(kw, prefix_lens=np.array([3, 1]))):
        ua = _layer(c, bad)
        d = {n: x.cuda() for n, x in t.items()}
        ua.forward(d["q"], d["k"], d["v"], torch.from_numpy(pos).cuda())
        ua.backward(d["do"])
        torch.cuda.synchronize()
        assert ua.read_status() == Bd.USP_ERR_BAD_MODS


def test_refusals_of_the_binding():
    from ulysses_sequence_long_gb300 import binding as Bd
    from ulysses_sequence_long_gb300.pipeline import ScoreMods, Shape, UlyssesAttention
    f = lambda *s: torch.zeros(s, device="cuda")
    i = lambda n: torch.zeros((n,), dtype=torch.int32, device="cuda")
    shape = Shape(1, 256, 4, 2, 64, 2)
    for bad in (ScoreMods(slopes=f(3)), ScoreMods(rel_bias=f(4, 2)), ScoreMods(buckets=i(3)),
                ScoreMods(rel_bias=f(3, 2), buckets=i(3)), ScoreMods(rel_bias=f(4, 2), buckets=i(4)),
                ScoreMods(rel_bias=f(4, 2), buckets=i(1)), ScoreMods(prefix_lens=i(0))):
        with pytest.raises(ValueError):
            UlyssesAttention(shape, mods=bad)
    for bad in (ScoreMods(slopes=f(4).double()), ScoreMods(slopes=torch.zeros(4)), ScoreMods(prefix_lens=f(2))):
        with pytest.raises(TypeError):
            UlyssesAttention(shape, mods=bad)
    two = UlyssesAttention(shape, mods=ScoreMods(softcap=5.0))
    q2, kv2 = (torch.zeros((2, 1, 128, h, 64), dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    for args in ((kv2, kv2, kv2, i(256)), (q2, q2, kv2, i(256)), (q2, kv2, kv2, i(255)), (q2, kv2, kv2, i(256), f(3))):
        with pytest.raises(ValueError):
            two.forward(*args)
    two.forward(q2, kv2, kv2, i(256))
    with pytest.raises(ValueError):
        two.backward(kv2)
    cu, n = i(257), i(1)
    x = torch.zeros((2, 1, 128, 4, 64), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros((2, 1, 128, 2, 64), dtype=torch.bfloat16, device="cuda")
    lse = f(2, 1, 2, 256)
    prm = Bd.attn_params(1, 256, 4, 2, 64, 2, cu, n, io_layout=Bd.USP_IO_SEQ)
    m = Bd.score_mods(4, softcap=10.0)
    with pytest.raises(ValueError):                # k as large as q
        Bd.usp_attn_mod_fwd(prm, m, x, x, kv, x.clone(), lse)
    with pytest.raises(ValueError):                # an lse of half the heads
        Bd.usp_attn_mod_fwd(prm, m, x, kv, kv, x.clone(), lse[:1].clone())
    with pytest.raises(Bd.UspError) as e:
        Bd.usp_attn_mod_fwd(prm, Bd.score_mods(4, softcap=-1.0), x, kv, kv, x.clone(), lse)
    assert e.value.code == Bd.USP_ERR_INVALID_ARG
