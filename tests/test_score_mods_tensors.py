"""The tensors of a layer's score modifications after their storage was
exchanged: another type, shape or strides are refused before anything is
launched (no GPU needed: only addresses are taken)."""
import pytest
import torch

from ulysses_sequence_long_gb300 import binding as B


@pytest.fixture
def mods(monkeypatch):
    # the checks of a tensor without the one for its device
    monkeypatch.setattr(B, "_dev", lambda t, name, dtype=None: None if t is None else t.data_ptr())

    class Table(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.rel_bias = torch.nn.Parameter(torch.zeros(4, 8))
            self.slopes = torch.nn.Parameter(torch.zeros(4))
            self.register_buffer("buckets", torch.zeros(41, dtype=torch.int32))
            self.register_buffer("prefix_lens", torch.zeros(3, dtype=torch.int32))

    t = Table()
    return t, B.score_mods(4, slopes=t.slopes, rel_bias=t.rel_bias, buckets=t.buckets, rel_bias_grad=True,
                           prefix_lens=t.prefix_lens)


def test_another_storage_of_the_same_kind_is_read_where_it_is(mods):
    t, m = mods
    keep = t.rel_bias.data
    t.rel_bias.data = keep.clone()
    m.point()
    assert m.rel_bias == t.rel_bias.data_ptr() != keep.data_ptr()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float64])
def test_a_module_moved_to_another_type_is_refused(mods, dtype):
    """`.to(bfloat16)` leaves the parameter the same object of the same size: read as fp32, its end would lie past
    the allocation."""
    t, m = mods
    t.to(dtype)
    assert t.rel_bias.numel() == 32
    with pytest.raises(TypeError):
        m.point()
    t.to(torch.float32)
    m.point()


@pytest.mark.parametrize("name", ["buckets", "prefix_lens"])
def test_integers_of_another_size_are_refused(mods, name):
    t, m = mods
    x = getattr(t, name)
    x.data = x.long()
    with pytest.raises(TypeError):
        m.point()


@pytest.mark.parametrize("name", ["rel_bias", "slopes", "buckets", "prefix_lens"])
def test_another_shape_or_strides_are_refused(mods, name):
    t, m = mods
    x = getattr(t, name)
    keep = x.data
    wide = torch.zeros(*keep.shape[:-1], 2 * keep.shape[-1], dtype=keep.dtype)
    for other in (keep[..., :-1].contiguous(), wide[..., ::2], keep.view(*reversed(keep.shape), 1)):
        x.data = other
        with pytest.raises(ValueError):
            m.point()
    x.data = keep
    m.point()
