"""The attention of single tokens over an 8-bit cache whose values are near the ends of bf16's range, where a value's power
of two is far from its token's weight: neither the sum of the weights nor that of the values may lose what counts."""
import numpy as np
import pytest
import torch

from gpu_util import built_lib
from oracle import serving as OS
from test_gpu_paged import BF, F8, _cu, _decode_case, _stored

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    built_lib()


def _check(c, lens, k, v, q, z, att, heads=1, only=None):
    """Bounds as for values around 1: a score's fp32 sum of D products (2 D 2^-24 of their sizes' sum) and 2^-20, twice that
    for a weight, 2^-11 for its rounding to f16, n 2^-23 for a sum of n, 2^-8 for the output's rounding.  Beside them the
    references' difference, up to 2^8, which scales the values' sum with an error of a few 2^-17 (four roundings of half a
    step of 2^-16 and 2^-22 of each power); half a step of bf16's subnormals, 2^-134."""
    D, G = q.shape[-1], q.shape[2] // c.hk
    ks, vs, qs = _stored(c, k)[0], _stored(c, v)[0], q.double().cpu().numpy()[0]
    zz = None if z is None else z.double().cpu().numpy()
    o, lse = att._out(len(lens))
    o, lse = o.double().cpu().numpy()[0], lse.double().cpu().numpy()[0]
    begin = np.cumsum([0] + list(lens))
    for s in range(len(lens)) if only is None else only:
        for h in range(0, qs.shape[1], heads):
            kk, vv = ks[begin[s]:begin[s + 1], h // G], vs[begin[s]:begin[s + 1], h // G]
            want, wl, size, qk = OS.decode(qs[s, h], kk, vv, 1 / np.sqrt(D), None if zz is None else zz[h])
            ds = 2 * D * 2.0 ** -24 * qk + 2.0 ** -20 * (1 + qk)
            rel = 2 * ds + 2.0 ** -11 + len(kk) * 2.0 ** -23 + 2.0 ** -15
            tol = 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * rel * size + 2.0 ** -134
            assert (np.abs(o[s, h] - want) <= tol).all(), (s, h, (np.abs(o[s, h] - want) / tol).max())
            if np.isinf(wl):
                assert lse[s, h] == wl
            else:
                assert abs(lse[s, h] - wl) <= ds + 2.0 ** -21 * (1 + abs(wl)) + len(kk) * 2.0 ** -23, (s, h)


def _case(lens, G, Hkv, D, exponents, seed=0, **kw):
    """Values of 2^exponents[token] times ordinary ones."""
    c, table, ln, k, v, q, z, att = _decode_case(lens, G, Hkv, D, 1, 64, F8, seed=seed, **kw)
    v = (v.double() * torch.exp2(torch.from_numpy(np.asarray(exponents, float)).cuda())[None, :, None, None]).to(BF)
    assert v.isfinite().all()
    c.append(k, v, table, ln, _cu(lens))
    return c, table, ln, k, v, q, z, att


LENS = [333, 0, 5000, 16, 1]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("e", [-120, -100, -70, -50, 50, 70, 100, 120])
@pytest.mark.parametrize("gain", [1.0, 6.0])
def test_all_values_far_from_one(D, e, gain):
    c, table, ln, k, v, q, z, att = _case(LENS, 3, 2, D, [e] * sum(LENS), seed=D + e + 200, sinks=gain == 1.0, gain=gain)
    att.forward(q, table, ln, z)
    assert att.read_status() == 0
    _check(c, LENS, k, v, q, z, att)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["any", "first far above", "one far above", "most far below", "last far above", "halves"])
def test_values_far_from_one_another(D, kind):
    """The tokens that make up the sum of the weights are others than those that make up the output's."""
    n = sum(LENS)
    e = np.random.default_rng(D).integers(-120, 121, n) if kind == "any" else np.zeros(n)
    if kind == "first far above":
        e[:16] = e[333:349] = 120
    if kind == "one far above":
        e[100] = e[333 + 2500] = 110
    if kind == "last far above":
        e[325:333] = e[5300:5333] = 118
    if kind == "halves":
        e[333:2833], e[2833:5333] = 40, -45
    if kind == "most far below":
        e[:] = -118
        e[50] = e[4000] = 3
    c, table, ln, k, v, q, z, att = _case(LENS, 3, 2, D, e, seed=D, sinks=True)
    att.forward(q, table, ln, z)
    assert att.read_status() == 0
    _check(c, LENS, k, v, q, z, att)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("e", [-120, 100, 120, 124])
def test_many_tokens_of_little_weight(D, e):
    """One token 2^16 above 4999 others, which together have 7% of the sum."""
    lens = [5000, 300]
    c, table, ln, k, v, q, z, att = _case(lens, 2, 1, D, [0] * 5300, seed=7)
    v = (v.double().clamp(-1, 1) * 2.0 ** e).to(BF)      # (2^128 is no bf16)
    k.zero_()
    k[0, 2000, 0, 0] = k[0, 5100, 0, 0] = 1.0
    q[..., 0] = 16 * np.log(2) * np.sqrt(D)
    c.append(k, v, table, ln, _cu(lens))
    att.forward(q, table, ln, z)
    assert att.read_status() == 0
    _check(c, lens, k, v, q, z, att)


@pytest.mark.parametrize("e", ["any", 120, -120])
def test_teams_of_warps(e):
    """A line long enough for two warps to share a ring, joined over all CTAs."""
    lens = [160001, 300]
    exps = np.random.default_rng(1).integers(-120, 121, sum(lens)) if e == "any" else [e] * sum(lens)
    c, table, ln, k, v, q, z, att = _case(lens, 16, 4, 64, exps, seed=3)
    att.forward(q, table, ln, z)
    assert att.read_status() == 0 and not att._ws[:12 * 1024].any()
    _check(c, lens, k, v, q, z, att, heads=9)


def test_scores_and_values_that_make_up_for_one_another():
    """Each tile's scores rise by 20 or fall by 20 where its values' exponents do the opposite: both references move."""
    lens = [640, 640]
    c, table, ln, k, v, q, z, att = _decode_case(lens, 2, 1, 64, 1, 64, F8, seed=5)
    rise = torch.arange(640).double() // 16 - 20
    steps = torch.cat([rise, -rise]).cuda()
    k[0, :, 0, 0] = steps.to(BF)
    q[..., 0] = 16.0                        # 16 x 1/8: scores rise by 2 a tile, 40 tiles
    v = (v.double() * torch.exp2(-4 * steps)[None, :, None, None]).to(BF)
    c.append(k, v, table, ln, _cu(lens))
    att.forward(q, table, ln, z)
    _check(c, lens, k, v, q, z, att)


@pytest.mark.parametrize("e", ["any", 120, -120, 0])
def test_teams_of_warps_of_long_rows(e):
    """Rows of 128 bytes: two warps share a ring, and go through a unit once more together (e = 0: they do not)."""
    lens = [120001, 300]
    exps = np.random.default_rng(1).integers(-120, 121, sum(lens)) if e == "any" else [e] * sum(lens)
    c, table, ln, k, v, q, z, att = _case(lens, 16, 4, 128, exps, seed=3, sinks=True)
    assert sum(-(-n // 16) for n in lens) * 4 >= 32 * 152 * 6       # (tiles of a team)
    o = att.forward(q, table, ln, z).clone()
    lse = att.lse.clone()
    assert att.read_status() == 0 and not att._ws[:12 * 1024].any()
    _check(c, lens, k, v, q, z, att, heads=9)
    assert torch.equal(att.forward(q, table, ln, z), o) and torch.equal(att.lse, lse)


def test_one_warp_of_a_team_finds_values_that_are_far():
    """Heads 0 to 7 of a group see only ordinary values, heads 8 to 15 large ones: both of its warps go once more."""
    lens = [120001]
    e = np.zeros(lens[0])
    e[::2] = 100
    c, table, ln, k, v, q, z, att = _case(lens, 16, 4, 128, e, seed=4)
    k[0, ::2, :, 0], k[0, 1::2, :, 0] = -60.0, 0.0
    q[..., 0] = torch.tensor([64.0] * 8 + [0.0] * 8, dtype=BF).repeat(4).cuda()   # 2^-490 for every second token
    c.append(k, v, table, ln, _cu(lens))
    att.forward(q, table, ln, z)
    assert att.read_status() == 0
    _check(c, lens, k, v, q, z, att, heads=5)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,G", [([40, 0, 90, 17, 1] * 120, 3), ([300] * 100, 2), ([1000, 30] * 30, 5),
                                    ([310, 33, 0, 2001] * 40, 16)], ids=["short", "middle", "ragged", "groups"])
def test_some_sequences_of_a_warp(lens, G, D):
    """Sequences with values far from 1 between others: a warp, or team, that goes through one once more has others before
    and behind it, on every way to deal them out.  The others are what they are among sequences of ordinary values."""
    kind = np.arange(len(lens)) % 4
    e = np.concatenate([np.full(n, (0, 115, 0, -115)[k]) for n, k in zip(lens, kind)])
    hkv = 4 if G == 16 else 2
    c, table, ln, k, v, q, z, att = _decode_case(lens, G, hkv, D, 1, 64, F8, seed=9, sinks=True)
    o, lse = att.forward(q, table, ln, z).clone(), att.lse.clone()
    v = (v.double() * torch.exp2(torch.from_numpy(e.astype(float)).cuda())[None, :, None, None]).to(BF)
    c.append(k, v, table, ln, _cu(lens))
    att.forward(q, table, ln, z)
    assert att.read_status() == 0
    same = torch.from_numpy(kind % 2 == 0).cuda()
    assert torch.equal(att._out(len(lens))[0][:, same], o[:, same]) and torch.equal(att.lse[:, same], lse[:, same])
    only = [s for s in range(len(lens)) if s % 4 != 0][::1 + len(lens) // 40]
    _check(c, lens, k, v, q, z, att, only=only)


@pytest.mark.parametrize("window", [0, 20, 300])
@pytest.mark.parametrize("e", [-118, 110])
def test_windows(window, e):
    """What a window hides and what lies behind a sequence's end (scales of 2^128 among them) moves no reference."""
    lens = [400, 16, 0, 33, 1, 700] * 20
    exps = np.where(np.arange(sum(lens)) % 3 == 0, 0, e)
    c, table, ln, k, v, q, z, att = _case(lens, 3, 2, 64, exps, seed=11, window=window, sinks=True)
    for s, m in enumerate(lens):        # (again: the values were appended anew)
        for t in range(0, max(0, m - 1 - window)):
            pg = int(table[s, t // 64])
            for x in (c.k_pages, c.v_pages):
                x.view(torch.uint8)[:, pg, :, t % 64] = 255
            c.k_scales[:, pg, :, t % 64] = c.v_scales[:, pg, :, t % 64] = 255
        if s == 5:
            break
    att.forward(q, table, ln, z)
    assert att.read_status() == 0
    begin = np.cumsum([0] + lens)
    seen = [np.arange(max(0, m - 1 - window), m) for m in lens[:6]]
    kk = torch.cat([k[:, begin[s] + torch.from_numpy(t).cuda()] for s, t in enumerate(seen)], 1)
    vv = torch.cat([v[:, begin[s] + torch.from_numpy(t).cuda()] for s, t in enumerate(seen)], 1)
    _check(c, [len(t) for t in seen], kk, vv, q[:, :6], z, att)
