"""Rotary positions on the GPU against the fp64 oracle, and the layers that call them."""
import numpy as np
import pytest
import torch

import usp_workloads as W
from gpu_util import built_lib, device_inputs, shape_of
from oracle import serving as OS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    built_lib()


def _rotary(pairs, n_axes=1, interleaved=False, seed=0, freqs=None):
    from ulysses_sequence_long_gb300.pipeline import Rotary
    rng = np.random.default_rng(seed)
    f = np.asarray(10000.0 ** -rng.uniform(0, 1, pairs) if freqs is None else freqs, np.float32)
    ax = rng.integers(0, n_axes, pairs).astype(np.int32)
    return Rotary(torch.from_numpy(f).cuda(), torch.from_numpy(ax).cuda(), n_axes, interleaved), f, ax


def _assert_turned(got, x, pos, f, ax, interleaved, back=False):
    """The angle is within 5e-7 and sin, cos a few units of 2^-24 (8e-7 of |x1| + |x2| with the fp32 products and
    sum, 3 2^-24); the result is rounded once to bf16, half a step: 2^-8 of it."""
    want, size = OS.rope(x.reshape(-1, *x.shape[-2:]).double().cpu().numpy(), pos, f, ax, interleaved, back)
    tol = 2.0 ** -8 * (np.abs(want) + 1e-6 * size) + 1e-6 * size
    off = np.abs(got.reshape(want.shape).double().cpu().numpy() - want)
    assert (off <= tol).all(), float((off / np.maximum(tol, 1e-300)).max())


CASES = [  # tokens, Hq, Hkv, D, pairs, axes, interleaved
    (1, 1, 0, 64, 32, 1, False), (1, 32, 8, 128, 64, 1, False), (3, 3, 1, 64, 8, 2, True), (257, 5, 5, 128, 24, 3, False),
    (64, 28, 4, 128, 64, 3, True), (33, 64, 8, 64, 24, 8, False), (5, 7, 1, 128, 40, 4, True), (1000, 12, 12, 64, 16, 2, True),
    (2, 200, 56, 128, 56, 1, False), (4099, 2, 1, 64, 32, 3, False),
]


@pytest.mark.parametrize("T,Hq,Hkv,D,pairs,axes,interleaved", CASES)
@pytest.mark.parametrize("back", [False, True])
def test_against_the_formula(T, Hq, Hkv, D, pairs, axes, interleaved, back):
    rope, f, ax = _rotary(pairs, axes, interleaved, seed=T)
    rng = np.random.default_rng(T + 1)
    pos = rng.integers(-1000, 100000, (axes, T)).astype(np.int32)
    g = torch.Generator().manual_seed(T)
    q = torch.randn((T, Hq, D), generator=g).to(torch.bfloat16).cuda()
    k = torch.randn((T, Hkv, D), generator=g).to(torch.bfloat16).cuda() if Hkv else None
    dev = torch.from_numpy(pos).cuda()
    qo, ko = (rope.backward if back else rope.forward)(q, k, dev)
    _assert_turned(qo, q, pos, f, ax, interleaved, back)
    if Hkv:
        _assert_turned(ko, k, pos, f, ax, interleaved, back)
        assert torch.equal(ko[..., 2 * pairs:], k[..., 2 * pairs:])
    assert torch.equal(qo[..., 2 * pairs:], q[..., 2 * pairs:])
    a, b = q.clone(), None if k is None else k.clone()
    (rope.backward if back else rope.forward)(a, b, dev, out=(a, b))      # in place: the same bits
    assert torch.equal(a, qo) and (k is None or torch.equal(b, ko))
    assert rope.read_status() == 0


def test_far_positions_and_frequencies_of_all_sizes():
    """Any int32 position; frequencies from none over the smallest to the largest that are taken."""
    f = np.array([0.0, 1e-45, 1e-38, 1e-20, 2.0 ** -41, 1e-10, 1e-7, 1e-4, 0.1, 0.99999994, 1.0, -1.0, 3.1415927, 17.3, -511.7, 1024.0],
                 np.float32)
    rope, f, ax = _rotary(16, 1, False, freqs=f)
    pos = np.array([[0, 1, -1, 2, 1000003, -1000003, 2 ** 30 + 7, 2 ** 31 - 1, -2 ** 31, 123456789]], np.int32)
    x = torch.randn((10, 2, 64), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    # in 64 bits the angle itself loses digits here: reduced before the sine, by exact integers
    from fractions import Fraction
    two_pi = Fraction(884279719003555, 140737488355328) + Fraction(2.4492935982947064e-16)   # 2 pi in two doubles
    w = [[float((Fraction(int(p)) * Fraction(float(v))) % two_pi) for v in f] for p in pos[0]]
    want, size = OS.rope(x.double().cpu().numpy(), np.zeros((1, 10)), f)
    c, s, xa = np.cos(w)[:, None], np.sin(w)[:, None], x.double().cpu().numpy()
    want[..., :16], want[..., 16:32] = xa[..., :16] * c - xa[..., 16:32] * s, xa[..., :16] * s + xa[..., 16:32] * c
    got, _ = rope.forward(x, None, torch.from_numpy(pos).cuda())
    tol = 2.0 ** -8 * (np.abs(want) + 1e-6 * size) + 1e-6 * size
    assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()


def test_there_and_back_is_near_and_norms_are_kept():
    rope, _, _ = _rotary(64)
    x = torch.randn((50, 4, 128), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    pos = torch.arange(50, dtype=torch.int32).cuda() * 977
    y, _ = rope.forward(x, None, pos)
    z, _ = rope.backward(y, None, pos)
    # two roundings of half a step (2^-8 of each element of a pair, so 2^-8 of the pair's length), each
    pair = torch.hypot(x[..., :64].double(), x[..., 64:].double()).repeat(1, 1, 2)
    assert ((z.double() - x.double()).abs() <= 2.05 * 2.0 ** -8 * pair).all()


def test_positions_repeat_over_ranks_and_values_that_are_not_finite_stay_in_their_pair():
    rope, f, ax = _rotary(8, 2)
    x = torch.randn((4, 6, 3, 64), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    pos = torch.randint(0, 99, (2, 6), generator=torch.Generator().manual_seed(5), dtype=torch.int32).cuda()
    y, _ = rope.forward(x, None, pos)
    z, _ = rope.forward(x, None, pos.repeat(1, 4))
    assert torch.equal(y, z)
    x[0, 0, 0, 3] = float("nan")
    x[0, 0, 0, 40] = float("inf")       # an element that passes through
    w, _ = rope.forward(x, None, pos)
    bad = w.isnan().nonzero()
    assert {tuple(i) for i in bad.tolist()} == {(0, 0, 0, 3), (0, 0, 0, 11)} and w[0, 0, 0, 40] == float("inf")


def test_bad_axes_and_frequencies_are_reported():
    from ulysses_sequence_long_gb300 import binding as B
    from ulysses_sequence_long_gb300.pipeline import Rotary
    x = torch.randn((2, 2, 64), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).cuda()
    pos = torch.ones((2, 2), dtype=torch.int32).cuda()
    for fr, ax in ((1.0, 2), (1.0, -1), (float("nan"), 0), (float("inf"), 0), (1025.0, 1)):
        freqs, axes = torch.zeros(8).cuda(), torch.zeros(8, dtype=torch.int32).cuda()
        freqs[5], axes[5] = fr, ax
        rope = Rotary(freqs, axes, 2)
        y, _ = rope.forward(x, None, pos)
        assert rope.read_status() == B.USP_ERR_BAD_ROPE and torch.equal(x, y)


def test_refused_tensors():
    rope, _, _ = _rotary(16, 2)
    q, k = torch.zeros((4, 2, 64), dtype=torch.bfloat16).cuda(), torch.zeros((4, 1, 64), dtype=torch.bfloat16).cuda()
    pos = torch.zeros((2, 4), dtype=torch.int32).cuda()
    from ulysses_sequence_long_gb300.binding import UspError
    rope.forward(q, k, pos)
    for bad in (lambda: rope.forward(q.float(), k, pos), lambda: rope.forward(q, k.cpu(), pos),
                lambda: rope.forward(q, k, pos.long()), lambda: rope.forward(q, k[:2], pos),
                lambda: rope.forward(q, k, pos[:, :3].contiguous()), lambda: rope.forward(q, k, pos.t()),
                lambda: rope.forward(q[:, :, ::2], k, pos), lambda: rope.forward(q, k, pos, out=(q[:2], k)),
                lambda: rope.forward(q, k, pos, out=(k, q)), lambda: rope.forward(q[:0], k[:0], pos)):
        with pytest.raises((TypeError, ValueError, UspError)):
            bad()
    with pytest.raises(UspError):       # overlapping, but not in place
        buf = torch.zeros((5, 2, 64), dtype=torch.bfloat16).cuda()
        rope.forward(buf[:4], k, pos, out=(buf[1:], k))


def test_streams_graphs_and_exchanged_storage():
    rope, f, ax = _rotary(64)
    x = torch.randn((300, 8, 128), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).cuda()
    pos = torch.arange(300, dtype=torch.int32).cuda()
    want, _ = rope.forward(x, None, pos)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.zeros_like(x)
    rope.forward(x, None, pos, out=(out, None), stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    # new outputs are memory of the stream, given as an object or as its handle: what the current stream has just let go
    # of and still writes is not theirs
    for stream in (s, s.cuda_stream):
        for _ in range(20):
            y = torch.empty_like(x)
            torch.cuda._sleep(200_000)
            y.zero_()
            del y
            got, _ = rope.forward(x, None, pos, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rope.forward(x, None, pos, out=(out, None))
    pos += 5
    g.replay()
    want, _ = rope.forward(x, None, pos)
    assert torch.equal(out, want)
    old, rope.freqs.data = rope.freqs.data, rope.freqs.data.clone() * 0.5
    half, _ = rope.forward(x, None, pos * 2)
    rope.freqs.data = old
    assert torch.equal(half, want)
    for name in ("freqs", "axes"):   # at the same place, but fewer
        t = getattr(rope, name)
        setattr(rope, name, t[:8])
        for _ in range(2):
            with pytest.raises(ValueError):
                rope.forward(x, None, pos)
        setattr(rope, name, t)
    rope.interleaved = True
    other = rope.forward(x, None, pos)[0]
    rope.interleaved = False
    assert torch.equal(rope.forward(x, None, pos)[0], want) and not torch.equal(other, want)
    for name in ("freqs", "axes", "status"):
        t = getattr(rope, name)
        setattr(rope, name, t.clone())
        assert torch.equal(rope.forward(x, None, pos)[0], want)
        for bad in (t.double(), t[:-1].clone() if name != "status" else t.cpu()):
            setattr(rope, name, bad)
            with pytest.raises((TypeError, ValueError)):
                rope.forward(x, None, pos)
        setattr(rope, name, t)
    assert torch.equal(rope.forward(x, None, pos)[0], want) and rope.read_status() == 0


def test_the_binding_itself():
    from ulysses_sequence_long_gb300 import binding as B
    rope, f, ax = _rotary(64)
    x = torch.randn((300, 8, 128), generator=torch.Generator().manual_seed(7)).to(torch.bfloat16).cuda()
    k = x[:, :2].contiguous()
    pos = torch.arange(150 * rope.n_axes, dtype=torch.int32).cuda()
    prm = B.rope_params(8, 2, 128, pos.clone(), rope.freqs.clone(), 300, rope.n_axes, rope.axes.clone())
    torch.full((150 * rope.n_axes,), 9, dtype=torch.int32, device="cuda")   # (the parameters keep their tensors)
    for fn, turn in ((B.usp_rope_fwd, rope.forward), (B.usp_rope_bwd, rope.backward)):
        y, yk = torch.empty_like(x), torch.empty_like(k)
        fn(prm, x, k, y, yk, rope.status)
        want = turn(x, k, pos)
        assert torch.equal(y, want[0]) and torch.equal(yk, want[1])
        for args in ((x, k, y, yk[:1], rope.status), (x, k, y, yk, rope.status.cpu()), (x.float(), k, y, yk),
                     (x.cpu(), k, y, yk), (x, k, y, None)):
            with pytest.raises((TypeError, ValueError, B.UspError)):
                fn(prm, *args)


def _layer(w, rope, **kw):
    from ulysses_sequence_long_gb300.pipeline import UlyssesAttention
    return UlyssesAttention(shape_of(w), rope=rope, **kw)


@pytest.mark.parametrize("kind", ["fused", "explicit", "one rank", "mods", "mods in shards"])
def test_the_layer_turns_q_and_k_and_their_gradients(kind):
    """Bits: the layer with rope is the rotation, the layer without, and the rotation back of its gradients."""
    from ulysses_sequence_long_gb300.pipeline import ScoreMods
    P = 1 if kind == "one rank" else 2
    w = W.Workload("rope", B=2 if kind == "explicit" else 1, S=512, Hq=4, Hkv=2, D=64, P=P, sinks=True,
                   doc_mode="explicit", doc_lens=(200, 1, 311), window_left=150)
    kw = dict(fused=kind in ("fused", "mods in shards"))
    if kind.startswith("mods"):
        kw["mods"] = ScoreMods(softcap=20.0)
    dev, _ = device_inputs(w)
    rope, f, ax = _rotary(24, 3, True)
    pos = torch.randint(0, 5000, (3, w.P, w.B, w.S // w.P), generator=torch.Generator().manual_seed(7), dtype=torch.int32).cuda()
    a, b = _layer(w, rope, **kw), _layer(w, None, **kw)
    o = a.forward(dev["q"], dev["k"], dev["v"], dev["pos"], dev["sinks"], rope_positions=pos)
    dq, dk, dv = a.backward(dev["do"], dev["sinks"])
    q, k = rope.forward(dev["q"], dev["k"], pos)
    o2 = b.forward(q, k, dev["v"], dev["pos"], dev["sinks"])
    dq2, dk2, dv2 = b.backward(dev["do"], dev["sinks"])
    dq2, dk2 = rope.backward(dq2, dk2, pos)
    assert a.read_status() == b.read_status() == 0
    for x, y in ((o, o2), (a.lse, b.lse), (dq, dq2), (dk, dk2), (dv, dv2), (a.dsinks, b.dsinks)):
        assert torch.equal(x, y)
    assert not torch.equal(q, dev["q"])
    # one axis: the position ids, when no others are given
    text, _, _ = _rotary(32)
    c = _layer(w, text, **kw)
    o = c.forward(dev["q"], dev["k"], dev["v"], dev["pos"], dev["sinks"]).clone()
    q, k = text.forward(dev["q"], dev["k"], dev["pos"])
    assert torch.equal(o, b.forward(q, k, dev["v"], dev["pos"], dev["sinks"]))
    # step by step
    c.exchange_qkv(*c.rotate(dev["q"], dev["k"], dev["pos"]), dev["v"])
    c.boundaries(dev["pos"])
    c.attention(dev["sinks"])
    c.exchange_out()
    assert torch.equal(o, c.o_seq)


@pytest.mark.parametrize("kind", ["fused", "explicit", "one rank", "mods", "mods in shards", "mods on one rank", "mods moved"])
def test_keys_and_values_in_head_layout(kind):
    """What a cache takes from a layer: the exchange of the turned keys and of the values."""
    from ulysses_sequence_long_gb300 import binding as B
    from ulysses_sequence_long_gb300.pipeline import ScoreMods
    P = 1 if "one rank" in kind else 2
    w = W.Workload("rope", B=2, S=512, Hq=4, Hkv=2, D=64, P=P, doc_mode="explicit", doc_lens=(200, 1, 311))
    dev, _ = device_inputs(w)
    rope, _, _ = _rotary(32)
    kw = dict(fused=kind in ("fused", "mods in shards", "mods moved"))
    if kind.startswith("mods"):
        kw["mods"] = ScoreMods(softcap=20.0)
    a = _layer(w, rope, **kw)
    if kind == "mods moved":
        a._kv_in_place = False
    a.forward(dev["q"], dev["k"], dev["v"], dev["pos"])
    k, v = a.head_kv()
    for got, x in ((k, rope.forward(dev["k"], None, dev["pos"])[0]), (v, dev["v"])):
        want = torch.empty_like(a.k_head)
        B.usp_relayout_fwd(x, want, w.B, w.S, w.Hkv, w.D, w.P)
        assert got.shape == want.shape and torch.equal(got, want)


def test_the_hybrid_layer():
    from ulysses_sequence_long_gb300.pipeline import HybridAttention, Shape
    w = W.Workload("rope", B=1, S=1024, Hq=4, Hkv=2, D=64, P=4, sinks=True, doc_mode="explicit", doc_lens=(600, 424))
    dev, _ = device_inputs(w)
    rope, _, _ = _rotary(32)
    sh = Shape(w.B, w.S, w.Hq, w.Hkv, w.D, w.P)
    a, b = HybridAttention(sh, 2, rope=rope), HybridAttention(sh, 2)
    o = a.forward(dev["q"], dev["k"], dev["v"], dev["pos"], dev["sinks"])
    grads = a.backward(dev["do"], dev["sinks"])
    q, k = rope.forward(dev["q"], dev["k"], dev["pos"])
    assert torch.equal(o, b.forward(q, k, dev["v"], dev["pos"], dev["sinks"]))
    dq, dk, dv = b.backward(dev["do"], dev["sinks"])
    dq, dk = rope.backward(dq, dk, dev["pos"])
    for x, y in zip(grads, (dq, dk, dv)):
        assert torch.equal(x, y)
    assert a.read_status() == 0


@pytest.mark.parametrize("kind", ["layer", "capped", "hybrid"])
def test_a_refused_forward_leaves_the_turned_shards(kind):
    from ulysses_sequence_long_gb300.pipeline import HybridAttention, ScoreMods
    S, P = (1024, 4) if kind == "hybrid" else (256, 2)   # (a ring step has S/ring keys, a multiple of 256)
    w = W.Workload("rope", B=1, S=S, Hq=4, Hkv=2, D=64, P=P, doc_mode="explicit", doc_lens=(S,))
    dev, _ = device_inputs(w)
    rope, _, _ = _rotary(32)
    if kind == "hybrid":
        a = HybridAttention(shape_of(w), 2, rope=rope)
    else:
        a = _layer(w, rope, mods=ScoreMods(softcap=20.0) if kind == "capped" else None)
    a.forward(dev["q"], dev["k"], dev["v"], dev["pos"])
    kept = [x.clone() for x in a.backward(dev["do"])]
    for bad in (dict(v=dev["q"]), dict(pos=dev["pos"].long()), dict(q=dev["k"])):
        d = dict(dev, **bad)
        with pytest.raises((TypeError, ValueError)):
            a.forward(d["q"], d["k"], d["v"], d["pos"])
    for x, y in zip(kept, a.backward(dev["do"])):
        assert torch.equal(x, y)


def test_gradient_through_the_layer_against_differences():
    """sum(O dO) of the oracle's attention over the oracle's rotation, differentiated by a central difference along a
    random direction of q and of k, against the layer's gradients along it."""
    import oracle
    w = W.Workload("rope", B=1, S=128, Hq=2, Hkv=1, D=64, P=1, doc_mode="explicit", doc_lens=(50, 78))
    dev, host = device_inputs(w)
    rope, f, ax = _rotary(32, 2)
    pos = np.random.default_rng(8).integers(0, 300, (2, w.S)).astype(np.int32)
    a = _layer(w, rope)
    a.forward(dev["q"], dev["k"], dev["v"], dev["pos"], rope_positions=torch.from_numpy(pos).cuda())
    dq, dk, _ = a.backward(dev["do"])
    assert a.read_status() == 0

    def loss(q, k):
        turn = lambda x: OS.rope(x.reshape(w.S, -1, w.D), pos, f, ax)[0].reshape(x.shape)
        o = oracle.ulysses_fwd(turn(q), turn(k), host["v"], host["pos"], True, -1, None, None)["o_seq"]
        return float((np.asarray(o) * host["do"]).sum())
    rng = np.random.default_rng(9)
    for grad, which in ((dq, "q"), (dk, "k")):
        u = rng.standard_normal(host[which].shape)
        step = 1e-5
        up, dn = dict(q=host["q"], k=host["k"]), dict(q=host["q"], k=host["k"])
        up[which], dn[which] = host[which] + step * u, host[which] - step * u
        diff = (loss(**up) - loss(**dn)) / (2 * step)
        g = grad.double().cpu().numpy()
        # the parity bar of the gradients (relative L2 5e-3), taken along a random direction: 6 standard deviations
        assert abs(float((g * u).sum()) - diff) <= 6 * 5e-3 * np.linalg.norm(g)


def test_a_rank_of_the_distributed_layer(tmp_path):
    import torch.distributed as dist
    from ulysses_sequence_long_gb300.distributed import RankShape, UlyssesRankAttention
    w = W.Workload("rope", B=1, S=256, Hq=4, Hkv=2, D=64, P=1, doc_mode="explicit", doc_lens=(100, 156))
    dev, _ = device_inputs(w)
    x = {n: dev[n][0] for n in ("q", "k", "v", "do", "pos")}
    rope, _, _ = _rotary(32)
    dist.init_process_group("gloo", init_method=f"file://{tmp_path}/store", rank=0, world_size=1)
    try:
        a = UlyssesRankAttention(RankShape(1, 256, 4, 2, 64, 1), rope=rope)
        b = UlyssesRankAttention(RankShape(1, 256, 4, 2, 64, 1))
        o = a.forward(x["q"], x["k"], x["v"], x["pos"])
        grads = a.backward(x["do"])
        q, k = rope.forward(x["q"], x["k"], x["pos"])
        assert torch.equal(o, b.forward(q, k, x["v"], x["pos"]))
        dq, dk, dv, _ = b.backward(x["do"])
        dq, dk = rope.backward(dq.contiguous(), dk.contiguous(), x["pos"])
        for p, r in zip(grads, (dq, dk, dv)):
            assert torch.equal(p, r)
    finally:
        dist.destroy_process_group()
