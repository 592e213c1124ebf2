"""The attention of single tokens where scores are infinite: keys of -inf, or so large that a product overflows, in the
places where a warp, a team of warps or a whole sequence begins."""
import numpy as np
import pytest
import torch

from gpu_util import built_lib
from oracle import serving as OS
from test_gpu_paged import BF, F8, _cu, _decode_case, _stored

pytestmark = pytest.mark.gpu
LOW = -3e38     # times a query's 64 and the scale it is below fp32's range; times its 0 it is 0


@pytest.fixture(scope="module", autouse=True)
def _lib():
    built_lib()


def _case(lens, G, Hkv, D, dtype, hidden, value=LOW, signs=(64.0,), **kw):
    """A case whose tokens `hidden` (over all sequences) have `value` as their keys' first element, the others 0 (so that
    their scores are ordinary ones); a head's query has one of `signs` there, in turn."""
    c, table, ln, k, v, q, z, att = _decode_case(lens, G, Hkv, D, 1, 64, dtype, **kw)
    k[..., 0] = 0
    k[:, torch.from_numpy(hidden).cuda(), :, 0] = value
    c.append(k, v, table, ln, _cu(lens))
    q[..., 0] = torch.tensor(signs, dtype=BF).cuda().repeat(-(-G * Hkv // len(signs)))[:G * Hkv]
    return c, table, ln, k, v, q, z, att


def _check(c, lens, k, v, q, z, att, hidden, seen=lambda h: False, heads=1, only=None):
    """Where the score is -inf a token has no weight: the oracle over the others (over all of them for heads h with
    seen(h)).  Bounds as for finite scores: a score's fp32 sum of D products, twice that for a weight, the weight's own
    rounding (bf16 in two parts: 2^-16; f16: 2^-11), n 2^-23 for a sum of n, 2^-8 for the output's rounding."""
    D, G = q.shape[-1], q.shape[2] // c.hk
    scale = 1 / np.sqrt(D)
    ks, vs, qs = _stored(c, k)[0], _stored(c, v)[0], q.double().cpu().numpy()[0]
    zz = None if z is None else z.double().cpu().numpy()
    o, lse = att._out(len(lens))
    o, lse = o.double().cpu().numpy()[0], lse.double().cpu().numpy()[0]
    begin = np.cumsum([0] + list(lens))
    for s, m in enumerate(lens):
        if only is not None and s not in only:
            continue
        a = begin[s] + (0 if att.window_left < 0 else max(0, m - 1 - att.window_left))
        for h in range(0, qs.shape[1], heads):
            use = np.ones(begin[s + 1] - a, bool) if seen(h) else ~hidden[a:begin[s + 1]]
            kk, vv = ks[a:begin[s + 1], h // G][use], vs[a:begin[s + 1], h // G][use]
            want, wl, size, qk = OS.decode(qs[s, h], kk, vv, scale, None if zz is None else zz[h])
            ds = 2 * D * 2.0 ** -24 * qk + 2.0 ** -20 * (1 + qk)
            rel = 2 * ds + (2.0 ** -16 if c.dtype is BF else 2.0 ** -11) + len(kk) * 2.0 ** -23 + 2.0 ** -20
            tol = 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * rel * size
            assert (np.abs(o[s, h] - want) <= tol).all(), (s, h, np.abs(o[s, h] - want).max(), tol.min())
            if np.isinf(wl):
                assert lse[s, h] == wl
            else:
                assert abs(lse[s, h] - wl) <= ds + 2.0 ** -21 * (1 + abs(wl)) + len(kk) * 2.0 ** -23


def _tiles(lens, which):
    """Whole tiles of 16 positions of each sequence: which(sequence, tile)."""
    return np.array([bool(which(s, t // 16)) for s, n in enumerate(lens) for t in range(n)])


@pytest.mark.parametrize("dtype", [BF, F8], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("value", [LOW, -np.inf], ids=["overflow", "infinite"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sinks", [False, True])
def test_first_tiles_without_weight(dtype, value, D, sinks):
    """The first tile, the first ones of many warps, every second one, most, a whole sequence: in a batch large enough
    that a warp has several tiles."""
    lens = [64, 100, 1600, 1601, 33, 40, 16, 1] * 16
    off = np.random.default_rng(1).random(101) < 0.7
    hidden = _tiles(lens, lambda s, t: (t == 0, t < 5, t % 2 == 0, off[t], t < 2, True, True, True)[s % 8])
    c, table, ln, k, v, q, z, att = _case(lens, 3, 2, D, dtype, hidden, value, sinks=sinks, seed=2)
    att.forward(q, table, ln, z)
    assert att.read_status() == 0
    _check(c, lens, k, v, q, z, att, hidden, only=[*range(8), *range(27, 128, 5)])


@pytest.mark.parametrize("dtype", [BF, F8], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("G", [2, 8, 12])
def test_one_column_of_two(dtype, G):
    """Neighbouring heads of a warp: one for which the first tiles have no weight, one that sees them."""
    lens = [200, 16, 50] * 300
    hidden = _tiles(lens, lambda s, t: t < (4, 1, 2)[s % 3])
    c, table, ln, k, v, q, z, att = _case(lens, G, 1, 64, dtype, hidden, signs=(64.0, 0.0), seed=3)
    att.forward(q, table, ln, z)
    assert att.read_status() == 0
    _check(c, lens, k, v, q, z, att, hidden, seen=lambda h: h % 2 == 1, only=range(0, 900, 7))


@pytest.mark.parametrize("dtype", [BF, F8], ids=["bf16", "e4m3"])
def test_the_begin_of_a_window(dtype):
    lens = [150, 90, 31] * 200
    hidden = np.array([t < n - 10 for n in lens for t in range(n)])
    c, table, ln, k, v, q, z, att = _case(lens, 4, 2, 64, dtype, hidden, seed=4)
    att.window_left = 40
    att.forward(q, table, ln, z)
    assert att.read_status() == 0
    _check(c, lens, k, v, q, z, att, hidden, only=range(0, 600, 7))


@pytest.mark.parametrize("dtype", [BF, F8], ids=["bf16", "e4m3"])
def test_teams_of_warps(dtype):
    """A line long enough for two warps to share a ring; about half of the stretches begin with tiles without weight."""
    lens = [160001, 300]
    rng = np.random.default_rng(5)
    off = rng.random((2, 10001)) < 0.5
    hidden = _tiles(lens, lambda s, t: off[s, t])
    c, table, ln, k, v, q, z, att = _case(lens, 16, 4, 64, dtype, hidden, seed=6)
    o = att.forward(q, table, ln, z).clone()
    lse = att.lse.clone()
    assert att.read_status() == 0
    _check(c, lens, k, v, q, z, att, hidden, heads=7)
    assert torch.equal(att.forward(q, table, ln, z), o) and torch.equal(att.lse, lse)


@pytest.mark.parametrize("dtype", [BF, F8], ids=["bf16", "e4m3"])
def test_scores_above_all_others_stay_in_their_head(dtype):
    """+inf leaves no softmax (NaN) for the heads that see it; for those whose query is negative there it is -inf."""
    lens = [100, 40]
    hidden = _tiles(lens, lambda s, t: s == 0 and t < 2)
    c, table, ln, k, v, q, z, att = _case(lens, 4, 1, 64, dtype, hidden, value=-LOW, signs=(64.0, -64.0), seed=7)
    o = att.forward(q, table, ln, z)
    assert o[0, 0, ::2].isnan().all() and not att.lse[0, 0, ::2].isfinite().any()
    o, lse = o.double().cpu(), att.lse.double().cpu()
    ks, vs, qs = _stored(c, k)[0, :, 0], _stored(c, v)[0, :, 0], q.double().cpu().numpy()[0]
    for s, h in ((0, 1), (0, 3), (1, 0), (1, 1), (1, 2), (1, 3)):
        use = ~hidden[:100] if s == 0 else slice(None)
        kk, vv = ks[:100][use] if s == 0 else ks[100:], vs[:100][use] if s == 0 else vs[100:]
        want, wl, size, qk = OS.decode(qs[s, h], kk, vv, 1 / 8)
        ds = 2 * 64 * 2.0 ** -24 * qk + 2.0 ** -20 * (1 + qk)
        rel = 2 * ds + (2.0 ** -16 if dtype is BF else 2.0 ** -11) + 100 * 2.0 ** -23 + 2.0 ** -20
        assert (np.abs(o[0, s, h].numpy() - want) <= 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * rel * size).all()
        assert abs(float(lse[0, s, h]) - wl) <= ds + 2.0 ** -21 * (1 + abs(wl)) + 100 * 2.0 ** -23


def test_teams_of_warps_of_8_bit_rows():
    lens = [120001, 300]
    off = np.random.default_rng(5).random((2, 7501)) < 0.5
    hidden = _tiles(lens, lambda s, t: off[s, t])
    c, table, ln, k, v, q, z, att = _case(lens, 16, 4, 128, F8, hidden, seed=6)
    att.forward(q, table, ln, z)
    assert att.read_status() == 0
    _check(c, lens, k, v, q, z, att, hidden, heads=9)


def test_an_infinite_value_stays_in_its_element():
    lens = [300, 40]
    c, table, ln, k, v, q, z, att = _decode_case(lens, 4, 1, 64, 1, 64, BF, seed=8)
    want, lse = att.forward(q, table, ln, z).clone(), att.lse.clone()
    v[0, 5, 0, 9], v[0, 320, 0, 33] = float("inf"), float("-inf")
    c.append(k, v, table, ln, _cu(lens))
    o = att.forward(q, table, ln, z)
    odd = torch.zeros_like(o, dtype=torch.bool)
    odd[:, 0, :, 9] = odd[:, 1, :, 33] = True
    assert not o[odd].isfinite().any() and torch.equal(o[~odd], want[~odd]) and torch.equal(att.lse, lse)
