"""A cache, a layer and a rotation made on one stream and used at once on another: what they were filled with is there."""
import pytest
import torch

from gpu_util import built_lib
from test_gpu_paged import BF, F8, _cu, _rotary, _tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    built_lib()


@pytest.mark.parametrize("dtype", [BF, F8], ids=["bf16", "e4m3"])
def test_used_on_another_stream_at_once(dtype):
    from ulysses_sequence_long_gb300.serving import DecodeAttention, PagedCache
    lens = [3000, 40]
    table = torch.randperm(100).to(torch.int32).view(2, 50).cuda()
    ln, cu = torch.tensor(lens, dtype=torch.int32).cuda(), _cu(lens)
    k, v = _tokens((1, sum(lens), 2, 64), 1), _tokens((1, sum(lens), 2, 64), 2)
    q, new = _tokens((1, 2, 8, 64), 3), [_tokens((1, 2, 2, 64), 4 + i) for i in range(2)]
    pos = ln - 1

    def all_of_it(stream):
        c = PagedCache(100, 64, 2, 64, 1, dtype=dtype)
        c.append(k, v, table, ln, cu, stream=stream)
        att = DecodeAttention(c, 8, 2, rope=_rotary())
        o = att.step(q, *new, table, ln, positions=pos, stream=stream)
        torch.cuda.synchronize()
        assert att.read_status() == 0
        return [o.clone(), att.lse.clone(), c.k_pages.view(torch.uint8).clone(), c.v_pages.view(torch.uint8).clone()]
    want = all_of_it(None)
    s = torch.cuda.Stream()
    for _ in range(5):
        # the current stream is behind, and what the allocator has was somebody else's
        for size in (1 << 12, 1 << 20, 100 * 2 * 64 * 64, 1 << 22):
            torch.empty((size,), dtype=torch.uint8, device="cuda").fill_(0x7B)
        torch.cuda._sleep(20_000_000)
        for x, y in zip(all_of_it(s), want):
            assert torch.equal(x, y)


def test_made_within_a_capture():
    """Nothing waits within a capture; the zeros are part of it."""
    from ulysses_sequence_long_gb300.serving import DecodeAttention, PagedCache
    table, ln = torch.arange(4, dtype=torch.int32).view(2, 2).cuda(), torch.ones(2, dtype=torch.int32).cuda()
    q, k, v = _tokens((1, 2, 4, 64), 1), _tokens((1, 2, 2, 64), 2), _tokens((1, 2, 2, 64), 3)
    warm = PagedCache(4, 16, 2, 64, 1)
    want = DecodeAttention(warm, 4, 2).step(q, k, v, table, ln).clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = PagedCache(4, 16, 2, 64, 1)
        o = DecodeAttention(c, 4, 2).step(q, k, v, table, ln)
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
