"""A decoding step: the same bits as its three parts, and steps that are refused before they change anything."""
import pytest
import torch

from gpu_util import built_lib
from test_gpu_paged import BF, F8, _decode_case, _rotary, _tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    built_lib()


def _case(dtype, rope, lens=(40, 3, 0, 17), P=2):
    from ulysses_sequence_long_gb300.serving import DecodeAttention
    c, table, ln, k, v, q, z, att = _decode_case(list(lens), 2, 2, 64, P, 16, dtype, sinks=True)
    if rope:
        att = DecodeAttention(c, 4, len(lens), rope=_rotary())
    new = [_tokens((P, len(lens), h, 64), i) for i, h in enumerate((q.shape[2], c.hk, c.hk))]
    return c, table, ln, new, z, att


def _pool(c):
    return [t.view(torch.uint8).clone() for t in (c.k_pages, c.v_pages, c.k_scales, c.v_scales) if t is not None]


@pytest.mark.parametrize("dtype", [BF, F8], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("rope", [False, True])
def test_a_step_is_its_parts(dtype, rope):
    c, table, ln, (q, k, v), z, att = _case(dtype, rope)
    pos = torch.arange(4, dtype=torch.int32).cuda() if rope else None
    before = _pool(c)
    o = att.step(q, k, v, table, ln, z, positions=pos).clone()
    lse, after = att.lse.clone(), _pool(c)
    for t, old in zip((c.k_pages, c.v_pages, c.k_scales, c.v_scales), before):
        t.view(torch.uint8).copy_(old)
    if rope:
        q, k = att.rope.forward(q, k, pos)
    c.append(k, v, table, ln)
    assert torch.equal(att.forward(q, table, ln, z), o) and torch.equal(att.lse, lse)
    assert all(torch.equal(x, y) for x, y in zip(after, _pool(c))) and att.read_status() == 0


@pytest.mark.parametrize("rope", [False, True])
def test_a_refused_step_leaves_the_cache(rope):
    from ulysses_sequence_long_gb300.binding import UspError
    c, table, ln, (q, k, v), z, att = _case(BF, rope)
    pos = torch.arange(4, dtype=torch.int32).cuda() if rope else None
    att.step(q, k, v, table, ln, z, positions=pos)
    before, o = _pool(c), att._out(4)[0].clone()
    shifted = torch.zeros(q.numel() + 1, dtype=BF).cuda()[1:].view(q.shape)        # not on 16 bytes
    mine = att._out(4)
    bad = [(q, k[:, :1].contiguous(), v[:, :1].contiguous(), table, ln, z), (q, k[:, :3].contiguous(), v, table, ln, z),
           (q, k, v[:, :3].contiguous(), table, ln, z), (q, k.float(), v, table, ln, z), (q, k, v.cpu(), table, ln, z),
           (q[:, :3].contiguous(), k, v, table, ln, z), (q.float(), k, v, table, ln, z), (q.cpu(), k, v, table, ln, z),
           (q, k, v, table, ln, z[:2]), (q, k, v, table, ln, z.double()), (q, k, v, table, ln, z.cpu()),
           (q, k, v, table, ln.long(), z), (q, k, v, table[:2], ln, z), (q, k, v, table, ln, mine[1].view(-1)[:4]),
           (shifted, k, v, table, ln, z)]
    if not rope:
        bad.append((mine[0], k, v, table, ln, z))        # (the queries that a rotation has read may lie there)
    for args in bad:
        for x in args[1:3]:
            x.mul_(2) if x.is_cuda else None             # other tokens than those there
        with pytest.raises((TypeError, ValueError, UspError)):
            att.step(*args, positions=pos)
    for name, value in (("window_left", -2), ("softmax_scale", -1.0), ("softmax_scale", float("inf")),
                        ("softmax_scale", float("nan"))):
        old = getattr(att, name)
        setattr(att, name, value)
        with pytest.raises(UspError):
            att.step(q, k, v, table, ln, z, positions=pos)
        setattr(att, name, old)
    assert all(torch.equal(x, y) for x, y in zip(before, _pool(c)))
    assert torch.equal(o, att._out(4)[0]) and att.read_status() == 0
