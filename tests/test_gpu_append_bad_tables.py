"""Appends with tables, lengths and boundaries that do not fit: what may be written is, nothing else in the pool changes."""
import numpy as np
import pytest
import torch

from gpu_util import built_lib
from test_gpu_paged import BF, F8, _cu, _pool, _stored, _tokens

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    built_lib()


def _places(table, lens, cu, tokens, n_pages, page):
    """{token: (page, token in it)} of those with a place: the last sequence that begins at or before a token (halving, as
    boundaries that go down have none) has it if it ends behind it, at the position that its length says."""
    out, n, capacity = {}, len(lens), table.shape[1] * page
    for i in range(tokens):
        lo, hi = 0, n
        while hi - lo > 1:
            mid = (lo + hi) // 2
            lo, hi = (mid, hi) if cu[mid] <= i else (lo, mid)
        pos = int(lens[lo]) - (int(cu[lo + 1]) - i)
        if cu[lo] <= i < cu[lo + 1] and 0 <= pos < capacity and 0 <= table[lo, pos // page] < n_pages:
            out[i] = int(table[lo, pos // page]), pos % page
    return out


@pytest.mark.parametrize("dtype", [BF, F8], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("P,Hkv,D", [(1, 2, 64), (2, 4, 128)])
@pytest.mark.parametrize("what,written", [("page", 112), ("negative page", 104), ("long", 103), ("negative", 80),
                                          ("boundary", 80), ("down", 80), ("short", 119)])
def test_only_valid_places_are_written(what, written, dtype, P, Hkv, D):
    from ulysses_sequence_long_gb300 import binding as B
    page, n = 16, 120
    c, table, ln = _pool([40, 40, 40], page, Hkv, D, P, dtype)
    cu = _cu([40, 40, 40])
    new = lambda seed: (_tokens((P, n, c.hk, D), seed), _tokens((P, n, c.hk, D), seed + 1))
    c.append(*new(1), table, ln, cu)
    assert c.read_status() == 0
    names = ("k_pages", "v_pages") + (("k_scales", "v_scales") if dtype is F8 else ())
    before = {name: getattr(c, name).view(torch.uint8).clone() for name in names}
    t2, l2, c2 = table.clone(), ln.clone(), cu.clone()
    if what == "page":
        t2[1, 2] = c.n_pages
    if what == "negative page":
        t2[1, 0] = -1
    if what == "long":            # one more than the table's row holds: the last token and the page that is none
        l2[1] = table.shape[1] * page + 1
    if what == "negative":
        l2[1] = -3
    if what == "boundary":
        c2[3] = 2 ** 31 - 1
    if what == "down":
        c2[2] = 20
    if what == "short":
        l2[1] = 39
    k, v = new(5)                 # others than those there
    c.append(k, v, t2, l2, c2)
    assert c.read_status() == B.USP_ERR_BAD_PAGES
    places = _places(t2.cpu().numpy(), l2.cpu().numpy(), c2.cpu().numpy().astype(np.int64), n, c.n_pages, page)
    assert len(places) == written
    touched = torch.zeros((c.n_pages, page), dtype=torch.bool)
    for p, r in places.values():
        assert not touched[p, r]
        touched[p, r] = True
    for name in names:            # bytes of all other rows are as they were
        rows = (getattr(c, name).view(torch.uint8).view(P, c.n_pages, c.hk, page, -1) ==
                before[name].view(P, c.n_pages, c.hk, page, -1)).all(-1).transpose(2, 3).cpu()
        assert rows[:, ~touched].all(), name
    at = torch.tensor([places[i] for i in sorted(places)])
    tok = sorted(places)
    for pages, scales, x in ((c.k_pages, c.k_scales, k), (c.v_pages, c.v_scales, v)):
        got = pages[:, at[:, 0].cuda(), :, at[:, 1].cuda()].transpose(0, 1).double().cpu().numpy() if dtype is BF else (
            pages.view(torch.uint8)[:, at[:, 0].cuda(), :, at[:, 1].cuda()].view(F8).float().double().cpu().numpy() *
            np.exp2(scales[:, at[:, 0].cuda(), :, at[:, 1].cuda()].double().cpu().numpy() - 127)[..., None]).swapaxes(0, 1)
        assert np.array_equal(got, _stored(c, x)[:, tok])
