"""The positions that layers with rotary positions take: one for each of their tokens and axes, no other number."""
from types import SimpleNamespace

import pytest
import torch

import usp_workloads as W
from gpu_util import built_lib, device_inputs, shape_of


def test_one_for_each_token_and_axis():
    from ulysses_sequence_long_gb300.pipeline import layer_positions
    ids = torch.zeros((4, 1, 8), dtype=torch.int32)
    one, two = SimpleNamespace(n_axes=1), SimpleNamespace(n_axes=2)
    assert layer_positions(one, None, ids, 32) is ids
    given = torch.zeros((2, 4, 1, 8), dtype=torch.int32)
    assert layer_positions(two, given, ids, 32) is given
    assert layer_positions(one, given[1], ids, 32) is not ids
    for rope, pos in ((two, None), (two, ids), (two, given[:, 0]), (one, given), (one, ids[0]), (one, ids[:0])):
        with pytest.raises(ValueError):
            layer_positions(rope, pos, ids, 32)
    with pytest.raises(ValueError):
        layer_positions(one, None, None, 32)


def _rotary(n_axes):
    from ulysses_sequence_long_gb300.pipeline import Rotary
    return Rotary(torch.ones(32).cuda(), (torch.arange(32) % n_axes).to(torch.int32).cuda(), n_axes)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["layer", "capped", "hybrid", "rank"])
@pytest.mark.parametrize("n_axes", [1, 2, 4])
def test_layers_refuse_other_numbers(kind, n_axes, tmp_path):
    built_lib()
    import torch.distributed as dist
    from ulysses_sequence_long_gb300.distributed import RankShape, UlyssesRankAttention
    from ulysses_sequence_long_gb300.pipeline import HybridAttention, ScoreMods, UlyssesAttention
    S, P = (1024, 4) if kind == "hybrid" else (256, 1 if kind == "rank" else 2)
    w = W.Workload("rope", B=1, S=S, Hq=4, Hkv=2, D=64, P=P, doc_mode="explicit", doc_lens=(S,))
    dev, _ = device_inputs(w)
    rope = _rotary(n_axes)
    x = {n: dev[n][0] if kind == "rank" else dev[n] for n in ("q", "k", "v", "do", "pos")}
    if kind == "rank":
        dist.init_process_group("gloo", init_method=f"file://{tmp_path}/store", rank=0, world_size=1)
    try:
        if kind == "rank":
            a = UlyssesRankAttention(RankShape(1, S, 4, 2, 64, 1), rope=rope)
        elif kind == "hybrid":
            a = HybridAttention(shape_of(w), 2, rope=rope)
        else:
            a = UlyssesAttention(shape_of(w), rope=rope, mods=ScoreMods(softcap=20.0) if kind == "capped" else None)
        whole = torch.stack([x["pos"]] * n_axes).contiguous()
        a.forward(x["q"], x["k"], x["v"], x["pos"], rope_positions=whole)
        if n_axes == 1:
            a.forward(x["q"], x["k"], x["v"], x["pos"])
        kept = [t.clone() for t in a.backward(x["do"])[:3]]
        half = whole.reshape(-1)
        bad = [half[:half.numel() // 2].contiguous(), half[:n_axes].contiguous(), torch.cat([half, half])]
        if n_axes > 1:
            bad += [None, x["pos"]]
        for pos in bad:
            with pytest.raises(ValueError):
                a.forward(x["q"], x["k"], x["v"], x["pos"], rope_positions=pos)
            if kind != "rank":
                with pytest.raises(ValueError):
                    a.rotate(x["q"], x["k"], pos)
        if kind != "rank":
            for t, u in zip(kept, a.backward(x["do"])):
                assert torch.equal(t, u)
    finally:
        if kind == "rank":
            dist.destroy_process_group()


@pytest.mark.gpu
@pytest.mark.parametrize("n_axes", [1, 2])
def test_a_step_refuses_other_numbers(n_axes):
    built_lib()
    from ulysses_sequence_long_gb300.serving import DecodeAttention, PagedCache
    n = 4
    c = PagedCache(8, 16, 2, 64, 2)
    att = DecodeAttention(c, 4, n, rope=_rotary(n_axes))
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn((2, n, h, 64), generator=g).to(torch.bfloat16).cuda() for h in (2, 1, 1))
    table, lens = torch.arange(8, dtype=torch.int32).view(4, 2).cuda(), torch.ones(n, dtype=torch.int32).cuda()
    att.step(q, k, v, table, lens, positions=torch.zeros((n_axes, n), dtype=torch.int32).cuda())
    pool = c.k_pages.clone(), c.v_pages.clone()
    for bad in (None, *(torch.zeros(m, dtype=torch.int32).cuda() for m in (n_axes, n_axes * n // 2, n_axes * n * 2))):
        with pytest.raises(ValueError):
            att.step(q * 2, k * 2, v * 2, table, lens, positions=bad)
    assert torch.equal(pool[0], c.k_pages) and torch.equal(pool[1], c.v_pages) and att.read_status() == 0
