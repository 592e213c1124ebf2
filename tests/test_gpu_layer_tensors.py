"""Tensors that change their storage between a layer's calls, and a layer's own
buffers exchanged for the caller's: every call reads and writes where they are
now.  Bits are compared with an undisturbed layer's."""
import pytest
import torch

import usp_workloads as W
from gpu_util import built_lib
from test_gpu_score_mods import _device_mods, _w

pytestmark = pytest.mark.gpu

# exchanges in place (one rank), fused with k and v read in place, fused with k and v moved first, explicit
LAYOUTS = [(1, None, True), (2, True, True), (2, True, False), (2, False, True)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    built_lib()


def _make(P, fused, in_place, **kw):
    from ulysses_sequence_long_gb300.pipeline import Shape, UlyssesAttention
    import numpy as np
    from oracle import score_mods as SM
    w = _w("exchange", S=256, Hq=4, Hkv=2, D=64, P=P, sinks=True, doc_lens=(100, 156))
    rng = np.random.default_rng(1)
    mods = dict(softcap=20.0, rel_bias=rng.standard_normal((4, 8)), buckets=SM.rel_buckets_log(8, 20, False))
    ua = UlyssesAttention(Shape(w.B, w.S, w.Hq, w.Hkv, w.D, w.P), fused=fused, mods=_device_mods(mods), **kw)
    ua._kv_in_place = ua._kv_in_place and in_place
    d = {n: x.cuda() for n, x in W.qkv_do_shards(w).items()}
    d["pos"] = torch.from_numpy(W.position_ids_shards(w)).cuda()
    d["sinks"] = W.sinks(w).cuda()
    return ua, d


OUT = ("o_seq", "lse", "dq_seq", "dk_seq", "dv_seq", "dsinks", "drel_bias")


def _forward(ua, d):
    return ua.forward(d["q"], d["k"], d["v"], d["pos"], d["sinks"])


def _results(ua):
    torch.cuda.synchronize()
    assert ua.read_status() == 0
    return [getattr(ua, n).clone() for n in OUT]


def _expected(P, fused, in_place):
    ua, d = _make(P, fused, in_place)
    _forward(ua, d)
    ua.backward(d["do"], d["sinks"])
    return _results(ua)


@pytest.mark.parametrize("P,fused,in_place", LAYOUTS)
def test_inputs_whose_storage_is_exchanged_before_the_backward(P, fused, in_place):
    """What moving a saved tensor out and in again does: the backward reads it where it is."""
    ua, d = _make(P, fused, in_place)
    _forward(ua, d)
    old = []
    for n in ("q", "k", "v"):
        old.append(d[n].data)
        d[n].data = d[n].data.clone()
        old[-1].fill_(7.0)           # kept alive: nothing else gets this memory
    ua.backward(d["do"], d["sinks"])
    for a, b in zip(_results(ua), _expected(P, fused, in_place)):
        assert torch.equal(a, b)


def test_a_refused_forward_changes_nothing_for_the_backward():
    ua, d = _make(2, True, True)
    _forward(ua, d)
    with pytest.raises(ValueError):
        ua.forward(d["q"], d["q"], d["v"], d["pos"], d["sinks"])
    ua.backward(d["do"], d["sinks"])
    for a, b in zip(_results(ua), _expected(2, True, True)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("P,fused,in_place", LAYOUTS)
def test_the_steps_called_one_by_one(P, fused, in_place):
    ua, d = _make(P, fused, in_place)
    ua.exchange_qkv(d["q"], d["k"], d["v"])
    ua.boundaries(d["pos"])
    ua.attention(d["sinks"])
    ua.exchange_out()
    ua.backward_phases(d["do"], d["sinks"], marks=lambda i: None)
    for a, b in zip(_results(ua), _expected(P, fused, in_place)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("P,fused,in_place", LAYOUTS)
def test_own_buffers_that_were_exchanged(P, fused, in_place):
    """A buffer put in place of a layer's own, or another storage under it, is the one that the calls use."""
    ua, d = _make(P, fused, in_place)
    _forward(ua, d)
    ua.backward(d["do"], d["sinks"])     # (the workspace exists from here on)
    torch.cuda.synchronize()
    names = [n for n, x in vars(ua).items() if isinstance(x, torch.Tensor)]
    assert set(OUT) <= set(names) and "_bwd_ws" in names and "cu_seqlens" in names
    old = {}
    for i, n in enumerate(names):
        x = getattr(ua, n)
        fresh = torch.zeros_like(x)
        if i % 2:
            setattr(ua, n, fresh)
            old[n] = x
        else:
            old[n], x.data = x.data, fresh
        old[n].view(-1).view(torch.uint8).fill_(0x5A)
    o = _forward(ua, d)
    assert o is ua.o_seq
    ua.backward(d["do"], d["sinks"])
    for a, b in zip(_results(ua), _expected(P, fused, in_place)):
        assert torch.equal(a, b)
    for n, x in old.items():
        assert (x.view(-1).view(torch.uint8) == 0x5A).all(), n


def test_exchanged_tensors_of_another_size_or_type_are_refused():
    ua, d = _make(2, True, True)
    _forward(ua, d)
    before = ua.o_seq.clone()
    for n in ("q", "k", "v"):
        keep = d[n].data
        d[n].data = keep[:1].clone()
        with pytest.raises(ValueError):
            ua.backward(d["do"], d["sinks"])
        d[n].data = keep.float()
        with pytest.raises(TypeError):
            ua.backward(d["do"], d["sinks"])
        d[n].data = keep
    for n in ("o_seq", "lse", "status", "cu_seqlens", "n_docs"):
        keep = getattr(ua, n)
        setattr(ua, n, torch.cat([keep.view(-1)] * 2))
        with pytest.raises(ValueError):
            _forward(ua, d)
        setattr(ua, n, keep.double())
        with pytest.raises(TypeError):
            _forward(ua, d)
        setattr(ua, n, keep)
    ua.backward(d["do"], d["sinks"])
    for a, b in zip(_results(ua), _expected(2, True, True)):
        assert torch.equal(a, b)
    assert torch.equal(before, ua.o_seq)


def test_parameters_of_a_call_belong_to_the_caller():
    """What params() gives is not changed by later calls and holds the buffers' addresses of now."""
    ua, d = _make(2, True, True)
    a = ua.params(d["sinks"])
    b = ua.params(None)
    assert a.sinks == d["sinks"].data_ptr() and b.sinks is None
    _forward(ua, d)
    assert b.sinks is None and a.cu_seqlens == ua.cu_seqlens.data_ptr()
    ua.cu_seqlens = ua.cu_seqlens.clone()
    assert ua.params(None).cu_seqlens == ua.cu_seqlens.data_ptr() != a.cu_seqlens


def test_a_layer_frees_its_buffers_when_it_is_dropped():
    import gc
    import weakref
    ua, d = _make(2, True, True)
    _forward(ua, d)
    ua.backward(d["do"], d["sinks"])
    torch.cuda.synchronize()
    gc.disable()
    try:
        gone = weakref.ref(ua.dv_seq)
        ua.dv_seq = torch.empty_like(ua.dv_seq)     # the replaced one is not kept
        assert gone() is None
        gone = weakref.ref(ua.o_seq)
        del ua
        assert gone() is None
    finally:
        gc.enable()


def test_two_layers_at_once_on_two_streams():
    """Steps of two layers queued in turn on two streams, nothing waiting for anything: each gives what it gives alone."""
    one, d1 = _make(2, True, True)
    two, d2 = _make(1, None, True)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        for ua, d, st in ((one, d1, streams[0]), (two, d2, streams[1])):
            ua.forward(d["q"], d["k"], d["v"], d["pos"], d["sinks"], stream=st)
            ua.backward(d["do"], d["sinks"], stream=st)
    for ua, want in ((one, _expected(2, True, True)), (two, _expected(1, None, True))):
        for a, b in zip(_results(ua), want):
            assert torch.equal(a, b)
