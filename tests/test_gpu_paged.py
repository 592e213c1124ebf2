"""The paged key/value cache and the attention of single tokens over it, on the GPU, against the fp64 oracle."""
import numpy as np
import pytest
import torch

import usp_workloads as W
from gpu_util import assert_close, built_lib, device_inputs, shape_of
from oracle import serving as OS

pytestmark = pytest.mark.gpu
BF, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    built_lib()


def _pool(lens, page, Hkv, D, P, dtype, seed=0, extra=3, nan=True):
    """A cache whose every byte is NaN (what no token has may hold anything), a table in random order whose entries
    behind a sequence's end are far outside."""
    from ulysses_sequence_long_gb300.serving import PagedCache
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    c = PagedCache(sum(need) + extra, page, Hkv, D, P, dtype=dtype)
    if nan:
        for t in (c.k_pages, c.v_pages):
            t.view(torch.uint8).fill_(255)
        if dtype is F8:
            c.k_scales.fill_(255)
            c.v_scales.fill_(254)
    order, table, at = rng.permutation(c.n_pages), np.full((len(lens), max(need + [1]) + 1), 2 ** 31 - 1, np.int32), 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return c, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()


def _tokens(shape, seed=0, spread=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g, dtype=torch.float64)
    if spread:   # rows of very different sizes
        x = x * torch.exp2(torch.randint(-spread, spread + 1, shape[:-1] + (1,), generator=g).double())
    return x.to(BF).cuda()


def _cu(counts):
    return torch.tensor([0] + list(counts), dtype=torch.int32).cumsum(0).to(torch.int32).cuda()


def _stored(c, x):
    """What the cache holds for tokens x, as fp64."""
    x = x.double().cpu().numpy()
    if c.dtype is BF:
        return x
    y, e = OS.to_e4m3(x)
    return y * np.exp2(e.astype(float))[..., None]


LENS = [[1], [16], [17, 0, 1, 64], [65, 130, 15, 1], [300, 2, 0, 0, 47, 128]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("dtype", [BF, F8], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D,Hkv,P,page", [(64, 2, 1, 16), (128, 4, 2, 64), (64, 1, 4, 48), (128, 12, 1, 256)])
def test_append_and_read(lens, dtype, D, Hkv, P, page):
    c, table, ln = _pool(lens, page, Hkv, D, P, dtype)
    rng = np.random.default_rng(1)
    past = [int(rng.integers(0, n + 1)) if i % 2 else 0 for i, n in enumerate(lens)]
    total = np.zeros((2, P, sum(lens), c.hk, D))
    begin = np.cumsum([0] + lens)
    # in two calls: what was there, then more of each sequence (of some none)
    for turn, (upto, counts) in enumerate(((past, past), (lens, [n - p for n, p in zip(lens, past)]))):
        if sum(counts) == 0:
            continue
        behind = 5   # tokens behind the last sequence are not written
        k, v = (_tokens((P, sum(counts) + behind, c.hk, D), seed=10 * turn + i, spread=6) for i in range(2))
        cu = _cu(counts)
        before = [t.view(torch.uint8).clone() for t in (c.k_pages, c.v_pages)]
        c.append(k, v, table, torch.tensor(upto, dtype=torch.int32).cuda(), cu)
        assert c.read_status() == 0
        for i, x in enumerate((k, v)):
            y, a = _stored(c, x), 0
            for s, n in enumerate(counts):
                total[i][:, begin[s] + upto[s] - n:begin[s] + upto[s]] = y[:, a:a + n]
                a += n
        # nothing else in the pool has changed
        rows = torch.zeros((c.n_pages, page), dtype=torch.bool)
        for s, n in enumerate(counts):
            for t in range(upto[s] - n, upto[s]):
                rows[int(table[s, t // page]), t % page] = True
        for t, b in zip((c.k_pages, c.v_pages), before):
            same = (t.view(torch.uint8) == b).all(-1).cpu()
            assert same[:, ~rows.any(1)].all()
            assert same.transpose(2, 3)[:, ~rows].all()
    k, v = c.read(table, ln, _cu(lens), tokens=sum(lens) + 2) if sum(lens) else (None, None)
    assert c.read_status() == 0
    for got, want in zip((k, v), total):
        if got is not None:
            # e4m3 values times their powers of two are bf16 values here: no rounding
            assert np.array_equal(got[:, :sum(lens)].double().cpu().numpy(), want) and not got[:, sum(lens):].any()


@pytest.mark.parametrize("D", [64, 128])
def test_codes_scales_and_their_ties(D):
    """Bits of the 8-bit cache: rows of all sizes, ties, zeros, subnormals, infinities, NaN."""
    rows = 4096
    x = torch.randint(-2 ** 15, 2 ** 15, (rows, D), generator=torch.Generator().manual_seed(2), dtype=torch.int16).view(BF)
    x[0], x[1], x[2] = 0, 1e-40, torch.tensor(float("inf"))
    x[3:1000] = (torch.randint(0, 64, (997, D), generator=torch.Generator().manual_seed(3)) * 8 - 256).to(BF)   # many ties
    x[1000:2000] = torch.randn((1000, D), generator=torch.Generator().manual_seed(4)).to(BF)
    x[2000] = 448.0
    x[2001, :2] = torch.tensor([450.0, -1.0]).to(BF)
    c, table, ln = _pool([rows], 64, 1, D, 1, F8)
    k = x.view(1, rows, 1, D).cuda()
    c.append(k, k.flip(1).contiguous(), table, ln, _cu([rows]))
    want, e = OS.to_e4m3(x.double().numpy())
    use = table[0, :rows // 64].long()
    for pages, scales, flip in ((c.k_pages, c.k_scales, False), (c.v_pages, c.v_scales, True)):
        got = pages.view(torch.uint8)[0, use, 0].reshape(rows, D).view(F8).float().double().cpu().numpy()
        se = scales[0, use, 0].reshape(rows).cpu().numpy().astype(int) - 127
        w, we = (want[::-1], e[::-1]) if flip else (want, e)
        assert np.array_equal(se, we)
        assert np.array_equal(np.isnan(got), np.isnan(w)) and np.array_equal(np.nan_to_num(got), np.nan_to_num(w))
    # e4m3 values below bf16's normal range are rounded on their way back, no others
    back, _ = c.read(table, ln, _cu([rows]), tokens=rows)
    exact = torch.from_numpy(want * np.exp2(e.astype(float))[:, None]).float().to(BF)
    assert torch.equal(back[0, :, 0].cpu().view(torch.int16)[~exact.isnan()], exact.view(torch.int16)[~exact.isnan()])
    assert back[0, :, 0].cpu()[exact.isnan()].isnan().all()


def test_one_token_each_and_empty_places():
    c, table, ln = _pool([5, 0, 33, 1], 16, 2, 64, 2, F8)
    k, v = _tokens((2, 4, 1, 64), 1), _tokens((2, 4, 1, 64), 2)
    c.append(k, v, table, ln)
    a = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    c.read(table, ln, out=a)
    assert c.read_status() == 0
    for got, x in zip(a, (k, v)):
        want = _stored(c, x)
        want[:, 1] = 7.0
        assert np.array_equal(got.double().cpu().numpy(), want)


def test_bad_tables_lengths_and_boundaries_are_reported_and_passed_over():
    from ulysses_sequence_long_gb300 import binding as B
    for what in ("page", "negative page", "long", "negative", "boundary", "down", "short"):
        c, table, ln = _pool([40, 40, 40], 16, 2, 64, 1, BF)
        cu = _cu([40, 40, 40])
        k, v = _tokens((1, 120, 2, 64), 1), _tokens((1, 120, 2, 64), 2)
        c.append(k, v, table, ln, cu)
        good = [t.clone() for t in c.read(table, ln, cu, tokens=120)]
        assert c.read_status() == 0
        t2, l2, c2 = table.clone(), ln.clone(), cu.clone()
        if what == "page":
            t2[1, 2] = c.n_pages
        if what == "negative page":
            t2[1, 0] = -1
        if what == "long":
            l2[1] = table.shape[1] * 16 + 1
        if what == "negative":
            l2[1] = -3
        if what == "boundary":
            c2[3] = 2 ** 31 - 1
        if what == "down":
            c2[2] = 20
        if what == "short":
            l2[1] = 39
        out = torch.zeros_like(k), torch.zeros_like(v)
        c.read(t2, l2, c2, out=out)
        assert c.read_status() == B.USP_ERR_BAD_PAGES, what
        c.status.zero_()
        for got, want in zip(out, good):
            assert torch.equal(got[:, :40], want[:, :40])                       # the first sequence
            assert what in ("boundary", "down") or torch.equal(got[:, 80:], want[:, 80:])
        before = c.k_pages.clone()
        c.append(k, v, t2, l2, c2)
        assert c.read_status() == B.USP_ERR_BAD_PAGES, what
        c.status.zero_()
        if what in ("long", "negative", "page"):      # the others' tokens are the same as before
            c.read(table, ln, cu, out=out)
            assert torch.equal(out[0][:, :40], good[0][:, :40]) and torch.equal(out[1][:, 80:], good[1][:, 80:])
        assert c.k_pages.shape == before.shape


# ---------------------------------------------------------------- attention
def _decode_case(lens, G, Hkv, D, P, page, dtype, window=-1, sinks=False, seed=0, gain=1.0, spread=0, scale=0.0):
    from ulysses_sequence_long_gb300.serving import DecodeAttention
    c, table, ln = _pool(lens, page, Hkv, D, P, dtype, seed)
    n, hk = len(lens), c.hk
    Hq = G * hk * P
    k, v = _tokens((P, max(1, sum(lens)), hk, D), seed + 1, 0), _tokens((P, max(1, sum(lens)), hk, D), seed + 2, spread)
    c.append(k, v, table, ln, _cu(lens))
    q = (_tokens((P, n, G * hk, D), seed + 3) * gain).to(BF)
    z = torch.randn((Hq,), generator=torch.Generator().manual_seed(seed + 4)).cuda() if sinks else None
    if window >= 0:  # what the window hides may hold anything
        for s, m in enumerate(lens):
            for t in range(0, max(0, m - 1 - window)):
                pg = int(table[s, t // page])
                for x in (c.k_pages, c.v_pages):
                    x.view(torch.uint8)[:, pg, :, t % page] = 255
    att = DecodeAttention(c, Hq, n, window_left=window, softmax_scale=scale)
    return c, table, ln, k, v, q, z, att


def _check_decode(c, lens, k, v, q, z, att, o, lse, scale=0.0, only=None):
    """Against the oracle over the values that the cache holds.  Bounds, per output, with n visible keys:
    a score's fp32 sum of D products (2 D 2^-24 of their sizes' sum; tensor cores cut, so a whole step each) and the
    arithmetic behind it (2^-20); a weight's relative error is twice that, and its own rounding (bf16 in two parts:
    2^-16; f16: 2^-11); the sum of n weighted values n 2^-23; the output's rounding 2^-8."""
    P, n, hq, D = q.shape
    hk = c.hk
    G = hq // hk
    scale = scale or 1 / np.sqrt(D)
    ks, vs = _stored(c, k), _stored(c, v)
    qs = q.double().cpu().numpy()
    zz = None if z is None else z.double().cpu().numpy()
    got, gl = o.double().cpu().numpy(), lse.double().cpu().numpy()
    begin = np.cumsum([0] + list(lens))
    for s, m in enumerate(lens):
        if only is not None and s not in only:
            continue
        a = begin[s] + (0 if att.window_left < 0 else max(0, m - 1 - att.window_left))
        for r in range(P):
            for h in range(hq):
                kk, vv = ks[r, a:begin[s + 1], h // G], vs[r, a:begin[s + 1], h // G]
                want, wl, size, qk = OS.decode(qs[r, s, h], kk, vv, scale, None if zz is None else zz[r * hq + h])
                ds = 2 * D * 2.0 ** -24 * qk + 2.0 ** -20 * (1 + qk)
                rel = 2 * ds + (2.0 ** -16 if c.dtype is BF else 2.0 ** -11) + len(kk) * 2.0 ** -23 + 2.0 ** -20
                tol = 2.0 ** -8 * np.abs(want) + (1 + 2.0 ** -8) * rel * size
                assert (np.abs(got[r, s, h] - want) <= tol).all(), (s, r, h, np.abs(got[r, s, h] - want).max(), tol.min())
                if np.isinf(wl):
                    assert gl[r, s, h] == wl
                else:
                    assert abs(gl[r, s, h] - wl) <= ds + 2.0 ** -21 * (1 + abs(wl)) + len(kk) * 2.0 ** -23


DECODE_LENS = [[1], [2, 16, 0, 17], [64, 65, 63, 1, 0, 200], [1000, 3], [0, 0], [5000]]


@pytest.mark.parametrize("lens", DECODE_LENS, ids=str)
@pytest.mark.parametrize("dtype", [BF, F8], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D,Hkv,P,page,G", [(64, 2, 1, 16, 1), (128, 4, 2, 64, 4), (64, 1, 4, 48, 8), (128, 1, 1, 256, 7),
                                            (64, 2, 2, 32, 12), (128, 1, 1, 64, 17), (64, 1, 1, 16, 130)])
def test_decode(lens, dtype, D, Hkv, P, page, G):
    c, table, ln, k, v, q, z, att = _decode_case(lens, G, Hkv, D, P, page, dtype, seed=G, sinks=G % 4 == 0, gain=1.5)
    o = att.forward(q, table, ln, z)
    assert att.read_status() == 0
    _check_decode(c, lens, k, v, q, z, att, o, att.lse)


@pytest.mark.parametrize("window", [0, 1, 15, 16, 127, 128, 400])
@pytest.mark.parametrize("dtype", [BF, F8], ids=["bf16", "e4m3"])
def test_decode_with_a_window(window, dtype):
    lens = [1, 2, 17, 129, 128, 0, 700, 401]
    c, table, ln, k, v, q, z, att = _decode_case(lens, 4, 2, 64, 2, 32, dtype, window=window, sinks=True, seed=window)
    o = att.forward(q, table, ln, z)
    assert att.read_status() == 0
    _check_decode(c, lens, k, v, q, z, att, o, att.lse)


@pytest.mark.parametrize("dtype", [BF, F8], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("gain,spread,scale", [(30.0, 0, 0.0), (1e-3, 0, 0.0), (1.0, 20, 0.0), (1.0, 0, 3.0), (1e18, 0, 1e-19),
                                               (1e-30, 3, 1e29)])
def test_decode_of_sharp_flat_and_scaled_scores(dtype, gain, spread, scale):
    """Scores far apart, equal ones, values of very different sizes, queries far from 1."""
    lens = [333, 64]
    c, table, ln, k, v, q, z, att = _decode_case(lens, 3, 2, 128, 1, 64, dtype, gain=gain, spread=spread, scale=scale, seed=5)
    o = att.forward(q, table, ln, z)
    assert att.read_status() == 0
    _check_decode(c, lens, k, v, q, z, att, o, att.lse, scale)


@pytest.mark.parametrize("sink", [-1e30, 80.0, 1e4])
def test_decode_sinks_far_above_and_below(sink):
    lens = [0, 5, 900]
    c, table, ln, k, v, q, _, att = _decode_case(lens, 2, 1, 64, 1, 16, BF)
    z = torch.full((2,), sink).cuda()
    o = att.forward(q, table, ln, z)
    _check_decode(c, lens, k, v, q, z, att, o, att.lse)


def test_decode_many_sequences_more_than_threads():
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 90, 700)]
    c, table, ln, k, v, q, z, att = _decode_case(lens, 2, 1, 64, 1, 16, F8, seed=11)
    o = att.forward(q, table, ln, z)
    assert att.read_status() == 0
    _check_decode(c, lens, k, v, q, z, att, o, att.lse)


@pytest.mark.parametrize("D,dtype", [(64, BF), (128, F8)], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("n,most", [(40, 1500), (120, 1500), (300, 40), (150, 300)])
def test_decode_ragged_batches(D, dtype, n, most):
    """Units that lie in a warp, in a CTA, across warps and across CTAs, some sequences empty."""
    rng = np.random.default_rng(n + most)
    lens = [0 if i % 7 == 3 else int(x) for i, x in enumerate(rng.integers(1, most + 1, n))]
    c, table, ln, k, v, q, z, att = _decode_case(lens, 2, 4, D, 2, 16, dtype, seed=n, sinks=True)
    o = att.forward(q, table, ln, z)
    assert att.read_status() == 0
    _check_decode(c, lens, k, v, q, z, att, o, att.lse)


@pytest.mark.parametrize("D,dtype", [(64, BF), (128, BF), (64, F8), (128, F8)], ids=str)
@pytest.mark.parametrize("G", [9, 16, 24, 40])
@pytest.mark.parametrize("lens,Hkv", [([9000, 3, 0, 17], 1), ([20001], 1), ([300] * 12 + [0, 1], 3), ([40, 0, 7] * 60, 2)],
                         ids=["long", "one", "middle", "short"])
def test_decode_groups_of_several_warps(lens, Hkv, G, D, dtype):
    """More query heads of a key/value head than a warp has: teams of warps, some of them without heads."""
    c, table, ln, k, v, q, z, att = _decode_case(lens, G, Hkv, D, 1, 48, dtype, seed=G, sinks=G == 24, gain=1.5,
                                                 window=-1 if G < 40 else 1000)
    o = att.forward(q, table, ln, z).clone()
    lse = att.lse.clone()
    assert att.read_status() == 0 and not att._ws[:12 * 1024].any()
    _check_decode(c, lens, k, v, q, z, att, o, lse)
    assert torch.equal(att.forward(q, table, ln, z), o) and torch.equal(att.lse, lse)


@pytest.mark.parametrize("D,dtype", [(64, BF), (128, BF), (64, F8), (128, F8)], ids=str)
@pytest.mark.parametrize("lens,Hkv,G,window", [([160001, 0, 5, 300], 2, 24, -1), ([150000], 1, 40, 147003),
                                               ([1297] * 38 + [0, 0], 8, 16, -1), ([310] * 150 + [0, 309], 5, 33, -1),
                                               ([310, 33, 0, 2001] * 40, 4, 9, -1)],
                         ids=["long", "one", "units to CTAs", "units to teams", "ragged"])
def test_decode_long_lines_of_large_groups(lens, Hkv, G, window, D, dtype):
    """Lines long enough (in most of the cases) for two warps to share a ring, on every way to deal them out."""
    c, table, ln, k, v, q, z, att = _decode_case(lens, G, Hkv, D, 1, 64, dtype, seed=G, sinks=G % 2 == 0)
    att.window_left = window
    o = att.forward(q, table, ln, z).clone()
    lse = att.lse.clone()
    assert att.read_status() == 0 and not att._ws[:12 * 1024].any()
    _check_decode(c, lens, k, v, q, z, att, o, lse, only=range(0, len(lens), 1 + len(lens) // 7))
    for _ in range(3):
        assert torch.equal(att.forward(q, table, ln, z), o) and torch.equal(att.lse, lse)


@pytest.mark.parametrize("dtype", [BF, F8], ids=["bf16", "e4m3"])
def test_decode_one_long_sequence(dtype):
    """Split over all SMs and joined; every head of one rank against fp64 on the device."""
    lens = [70001]
    c, table, ln, k, v, q, z, att = _decode_case(lens, 7, 2, 128, 2, 128, dtype, seed=2, gain=2.0)
    o = att.forward(q, table, ln, z).clone()
    lse = att.lse.clone()
    assert att.read_status() == 0
    _check_decode(c, lens, k, v, q, z, att, o, lse)
    for _ in range(3):   # the join's order is that of the positions
        assert torch.equal(att.forward(q, table, ln, z), o) and torch.equal(att.lse, lse)


def test_decode_bad_pages_and_lengths_are_reported_and_others_are_right():
    from ulysses_sequence_long_gb300 import binding as B
    lens = [100, 200, 0, 50]
    c, table, ln, k, v, q, z, att = _decode_case(lens, 2, 2, 64, 1, 32, F8)
    att.forward(q, table, ln, z)
    assert att.read_status() == 0
    for what in ("page", "negative page", "long", "negative"):
        t2, l2 = table.clone(), ln.clone()
        if what == "page":
            t2[1, 3] = c.n_pages
        if what == "negative page":
            t2[1, 0] = -5
        if what == "long":
            l2[1] = 2 ** 31 - 1
        if what == "negative":
            l2[1] = -2 ** 31
        got = att.forward(q, t2, l2, z)
        assert att.read_status() == B.USP_ERR_BAD_PAGES, what
        c.status.zero_()
        # Another length deals the work out in other pieces, with other references, against which the weights round
        # to f16 (2^-11 of each): two right results are apart by more than their own roundings (2 2^-8 of them, a
        # first form of this test), by up to 2 2^-11 sum p |v|.  Each is within the oracle's bound.
        _check_decode(c, lens, k, v, q, z, att, got, att.lse, only=(0, 2, 3))


def test_tokens_behind_the_last_sequence_and_pages_of_others_do_not_matter():
    lens = [70, 33]
    c, table, ln, k, v, q, z, att = _decode_case(lens, 4, 2, 128, 1, 64, BF)
    o = att.forward(q, table, ln, z).clone()
    mine = {int(p) for s, n in enumerate(lens) for p in table[s, :-(-n // 64)]}
    for p in range(c.n_pages):
        if p not in mine:
            c.k_pages[:, p] = float("inf")
            c.v_pages[:, p] = float("nan")
    table[table == 2 ** 31 - 1] = -7
    assert torch.equal(o, att.forward(q, table, ln, z)) and att.read_status() == 0


def test_sequences_that_share_a_prefix_and_places_of_the_table():
    """Pages that several sequences read: each is what it is alone."""
    c, table, ln, k, v, q, z, att = _decode_case([200, 0, 0], 4, 2, 64, 1, 64, F8, seed=3)
    table[1] = table[0]
    table[2] = table[0]
    ln[1:] = torch.tensor([130, 200])
    q[:, 2] = q[:, 0]
    o = att.forward(q, table, ln, z)
    assert att.read_status() == 0
    _check_decode(c, [200], k, v, q[:, :1].contiguous(), z, att, o[:, :1], att.lse[:, :1])
    _check_decode(c, [200], k, v, q[:, 2:].contiguous(), z, att, o[:, 2:], att.lse[:, 2:])
    _check_decode(c, [130], k[:, :130].contiguous(), v[:, :130].contiguous(), q[:, 1:2].contiguous(), z, att, o[:, 1:2], att.lse[:, 1:2])


def test_more_work_than_the_line_holds_is_reported():
    """64 sequences of 2^30 positions, all of them in the same page: refused on the device before anything is read."""
    from ulysses_sequence_long_gb300 import binding as B
    from ulysses_sequence_long_gb300.serving import DecodeAttention, PagedCache
    c = PagedCache(1, 2 ** 20, 1, 64, 1, dtype=F8)
    table = torch.zeros((64, 1000), dtype=torch.int32).cuda()
    att = DecodeAttention(c, 1, 64)
    att.forward(_tokens((1, 64, 1, 64)), table, torch.full((64,), 1000 * 2 ** 20, dtype=torch.int32).cuda())
    assert att.read_status() == B.USP_ERR_UNSUPPORTED
    c.status.zero_()
    o = att.forward(_tokens((1, 64, 1, 64)), table, torch.full((64,), 3, dtype=torch.int32).cuda())
    assert att.read_status() == 0 and not o.any()       # (zeros in the pool)


def test_scores_and_sums_that_are_not_finite_stay_in_their_sequence():
    lens = [40, 40, 40]
    c, table, ln, k, v, q, z, att = _decode_case(lens, 2, 1, 64, 1, 16, BF, sinks=True)
    want = att.forward(q, table, ln, z).clone()
    c.v_pages[0, table[1, 1].item(), 0, 3, 5] = float("nan")      # one value of one token
    c.k_pages[0, table[2, 0].item(), 0, 0] = float("nan")         # a key
    o = att.forward(q, table, ln, z)
    assert torch.equal(o[:, 0], want[:, 0])
    assert o[:, 1, :, 5].isnan().all() and torch.equal(o[:, 1, :, :5], want[:, 1, :, :5]) and torch.equal(o[:, 1, :, 6:], want[:, 1, :, 6:])
    assert o[:, 2].isnan().all() and att.lse[:, 2].isnan().all()


def test_a_workspace_is_as_it_was_found_and_serves_caches_of_all_kinds():
    """What has to be zero is zero after every call, whatever the split; so calls of different caches may follow one
    another in one workspace."""
    from ulysses_sequence_long_gb300 import binding as B
    ws = torch.zeros((8 << 20,), dtype=torch.uint8).cuda()
    for i, (lens, D, dt, P, Hkv) in enumerate([([5000], 128, BF, 1, 1), ([300] * 40, 64, F8, 2, 4), ([20001, 7], 64, BF, 1, 1),
                                               ([30000, 0, 9], 128, F8, 1, 2), ([100] * 200, 128, BF, 1, 8)]):
        c, table, ln, k, v, q, z, att = _decode_case(lens, 2, Hkv, D, P, 64, dt, seed=i)
        want, lse = att.forward(q, table, ln).clone(), att.lse.clone()
        o, l2 = torch.empty_like(want), torch.empty_like(lse)
        prm = B.paged_cache(Hkv, D, P, c.k_pages, c.v_pages, table, ln, c.k_scales, c.v_scales)
        assert B.usp_attn_decode_workspace_bytes(prm, 2 * Hkv) <= ws.numel()
        B.usp_attn_decode(prm, 2 * Hkv, q, o, l2, ws, dev_status=c.status)
        assert c.read_status() == 0 and torch.equal(o, want) and torch.equal(l2, lse)
        assert not ws[:1024 * 12].any()


def test_a_pool_beyond_32_bits():
    """Pages on both sides of 2^32 elements (and bytes) of a pool."""
    from ulysses_sequence_long_gb300.serving import DecodeAttention, PagedCache
    page, hk, D = 64, 8, 128
    n_pages = 2 ** 32 // (page * hk * D) + 40
    c = PagedCache(n_pages, page, hk, D, 1, dtype=F8)
    lens = [130, 70, 64]
    table = torch.tensor([[n_pages - 1, 0, n_pages - 20], [2 ** 32 // (page * hk * D) - 1, 2 ** 32 // (page * hk * D), 5],
                          [2 ** 31 // (page * hk * D), 7, 8]], dtype=torch.int32).cuda()
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    k, v = _tokens((1, sum(lens), hk, D), 1), _tokens((1, sum(lens), hk, D), 2)
    c.append(k, v, table, ln, _cu(lens))
    kk, vv = c.read(table, ln, _cu(lens), tokens=sum(lens))
    assert np.array_equal(kk.double().cpu().numpy(), _stored(c, k)) and np.array_equal(vv.double().cpu().numpy(), _stored(c, v))
    q = _tokens((1, 3, 16, D), 3)
    att = DecodeAttention(c, 16, 3)
    o = att.forward(q, table, ln)
    assert att.read_status() == 0
    _check_decode(c, lens, k, v, q, None, att, o, att.lse)


# ---------------------------------------------------------------- as they are used
def _rotary(pairs=32):
    from ulysses_sequence_long_gb300.pipeline import Rotary
    return Rotary(10000.0 ** -(torch.arange(pairs).float() / pairs).cuda())


@pytest.mark.parametrize("dtype", [BF, F8], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("P,Hkv", [(1, 2), (2, 2), (4, 2)])
@pytest.mark.parametrize("window", [-1, 100])
def test_prompts_then_tokens(dtype, P, Hkv, window):
    """A packed batch of prompts through the layer, its keys and values into the cache, then tokens one by one; in the
    end the steps' outputs are those of the layer over the whole sequences (bf16), or the oracle's over the cache."""
    from ulysses_sequence_long_gb300.pipeline import UlyssesAttention
    from ulysses_sequence_long_gb300.serving import DecodeAttention
    docs, more, D, Hq, page = (200, 1, 55), 5, 64, 4, 16
    rope = _rotary()
    whole = tuple(n + more for n in docs)
    S = sum(whole)
    S += -S % P
    w = W.Workload("serve", B=1, S=S, Hq=Hq, Hkv=Hkv, D=D, P=P, sinks=True, window_left=window, doc_mode="explicit",
                   doc_lens=whole + ((S - sum(whole),) if S > sum(whole) else ()))
    dev, _ = device_inputs(w)
    full = UlyssesAttention(shape_of(w), rope=rope)
    full.forward(dev["q"], dev["k"], dev["v"], dev["pos"], dev["sinks"])
    flat = lambda x: x.transpose(0, 1).reshape(S, *x.shape[3:])
    q, k, v, want = flat(dev["q"]), flat(dev["k"]), flat(dev["v"]), flat(full.o_seq)
    at = np.cumsum((0,) + whole)
    # the prompts alone
    prompt = np.concatenate([np.arange(at[i], at[i] + n) for i, n in enumerate(docs)])
    Sp = len(prompt) + (-len(prompt)) % P
    prompt = torch.from_numpy(np.concatenate([prompt, prompt[:Sp - len(prompt)]])).cuda()
    pos = torch.cat([torch.arange(n) for n in docs + ((Sp - sum(docs),) if Sp > sum(docs) else ())]).to(torch.int32).cuda()
    shards = lambda x: x[prompt].view(P, 1, Sp // P, *x.shape[1:]).contiguous()
    from ulysses_sequence_long_gb300.pipeline import Shape
    ua = UlyssesAttention(Shape(1, Sp, Hq, Hkv, D, P, window_left=window), with_backward=False, rope=rope)
    ua.forward(shards(q), shards(k), shards(v), pos.view(P, 1, Sp // P), dev["sinks"])
    c, table, ln = _pool([n for n in whole], page, Hkv, D, P, dtype)
    lens = torch.tensor(docs, dtype=torch.int32).cuda()
    c.append(*ua.head_kv(), table, lens, ua.cu_seqlens)
    att = DecodeAttention(c, Hq, len(docs), window_left=window, rope=rope)
    hq, hk = Hq // P, c.hk
    rank_kv = [list(range(r * hk, (r + 1) * hk)) if Hkv >= P else [r * Hkv // P] for r in range(P)]
    for t in range(more):
        rows = torch.tensor([at[i] + n + t for i, n in enumerate(docs)]).cuda()
        positions = lens.clone()
        lens += 1
        head = lambda x, sel: torch.stack([x[rows][:, sel(r)] for r in range(P)]).contiguous()
        o = att.step(head(q, lambda r: slice(r * hq, (r + 1) * hq)), head(k, lambda r: rank_kv[r]), head(v, lambda r: rank_kv[r]),
                     table, lens, dev["sinks"], positions=positions)
        assert att.read_status() == 0 and full.read_status() == 0
        got = o.transpose(0, 1).reshape(len(docs), Hq, D).double().cpu().numpy()
        if dtype is BF:
            assert_close(f"step {t}", got, want[rows].double().cpu().numpy(), slack=0.0)
        else:
            kk, vv = c.read(table, lens, _cu(lens.tolist()), tokens=int(lens.sum()))
            qt, _ = rope.forward(q[rows].contiguous(), None, positions)
            b = np.cumsum([0] + lens.tolist())
            for i in range(len(docs)):
                a = b[i] if window < 0 else max(b[i], b[i + 1] - 1 - window)
                for h in range(Hq):
                    r, g = h // hq, (h % hq) // (hq // hk)
                    ref, _, _, _ = OS.decode(qt[i, h].double().cpu().numpy(), kk[r, a:b[i + 1], g].double().cpu().numpy(),
                                             vv[r, a:b[i + 1], g].double().cpu().numpy(), 1 / 8.0, float(dev["sinks"][h]))
                    assert_close(f"step {t} {i} {h}", got[i, h], ref, rel_l2=1e-2)


def test_a_captured_step_replays_as_the_sequences_grow():
    lens = [40, 0, 17]
    c, table, ln, k, v, q, z, att = _decode_case(lens, 2, 2, 64, 1, 16, F8)
    from ulysses_sequence_long_gb300.serving import DecodeAttention
    table = torch.randperm(24).to(torch.int32).view(3, 8).cuda()
    c2, _, _ = _pool([100] * 4, 16, 2, 64, 1, F8)
    c2.k_pages.view(torch.uint8).zero_()
    c2.v_pages.view(torch.uint8).zero_()
    rope = _rotary()
    mk = lambda: DecodeAttention(c2, 4, 3, rope=rope)
    a, b = mk(), mk()
    ln = torch.tensor([1, 1, 1], dtype=torch.int32).cuda()
    pos = torch.zeros((1, 3), dtype=torch.int32).cuda()
    x = {n: _tokens((1, 3, h, 64), i) for i, (n, h) in enumerate((("q", 4), ("k", 2), ("v", 2)))}
    a.step(x["q"], x["k"], x["v"], table, ln, positions=pos)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = a.step(x["q"], x["k"], x["v"], table, ln, positions=pos)
    for t in range(70):
        for i, n in enumerate(("q", "k", "v")):
            x[n].copy_(_tokens(tuple(x[n].shape), 3 * t + i))
        ln.fill_(t + 1)
        ln[1] = 1 + t // 2     # one that grows more slowly (its last place is written again)
        pos.fill_(t)
        g.replay()
        got, lse = o.clone(), a.lse.clone()
        assert torch.equal(got, b.step(x["q"], x["k"], x["v"], table, ln, positions=pos)) and torch.equal(lse, b.lse)
    assert a.read_status() == 0


def test_two_streams_and_two_layers_at_once():
    cases = [_decode_case([3000, 5], 4, 2, 128, 1, 64, dt, seed=i) for i, dt in enumerate((BF, F8))]
    want = [(att.forward(q, table, ln, z).clone(), att.lse.clone()) for c, table, ln, k, v, q, z, att in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for s, (c, table, ln, k, v, q, z, att) in zip(streams, cases):
            att.forward(q, table, ln, z, stream=s)
    torch.cuda.synchronize()
    for (o, lse), (c, table, ln, k, v, q, z, att) in zip(want, cases):
        assert torch.equal(att._out(2)[0], o) and torch.equal(att.lse, lse)


def test_tokens_read_on_another_stream_into_new_tensors():
    lens = [70, 33]
    c, table, ln, k, v, q, z, att = _decode_case(lens, 4, 2, 64, 1, 16, BF)
    cu = _cu(lens)
    want = c.read(table, ln, cu, tokens=sum(lens) + 5)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        for _ in range(20):
            y = torch.empty_like(want[0]), torch.empty_like(want[1])
            torch.cuda._sleep(200_000)   # the current stream is behind: its zeros would come after the tokens
            for t in y:
                t.fill_(7)
            del y, t
            got = c.read(table, ln, cu, tokens=sum(lens) + 5, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_pool_whose_tensors_were_exchanged():
    """Every call reads and writes the tensors where they are then; one of another size or type is refused."""
    lens = [70, 33]
    c, table, ln, k, v, q, z, att = _decode_case(lens, 4, 2, 64, 1, 16, F8)
    want = att.forward(q, table, ln, z).clone()
    for name in ("k_pages", "v_pages", "k_scales", "v_scales", "status"):
        old = getattr(c, name)
        setattr(c, name, old.clone())                      # another tensor
        old.view(torch.uint8).fill_(0x5A)
        assert torch.equal(att.forward(q, table, ln, z), want), name
        t = getattr(c, name)
        keep = t.data
        t.data = keep.clone()                              # another storage under it
        keep.view(torch.uint8).fill_(0x5A)
        assert torch.equal(att.forward(q, table, ln, z), want), name
        t = getattr(c, name)
        for bad in (torch.cat([t.view(torch.uint8).view(-1)] * 2), t[:0],
                    t.view(torch.int16 if name == "status" else torch.int8), t.view(torch.uint8).double(), t.cpu()):
            setattr(c, name, bad)
            for _ in range(2):
                with pytest.raises((TypeError, ValueError)):
                    att.forward(q, table, ln, z)
            setattr(c, name, t)
    t, other, s = c.k_pages, c.k_pages.clone(), c.status   # one that is good beside one that is not: neither is taken
    other.view(torch.uint8).fill_(0x5A)
    c.k_pages, c.status = other, s.cpu()
    with pytest.raises(TypeError):
        att.forward(q, table, ln, z)
    c.k_pages, c.status = t, s
    assert torch.equal(att.forward(q, table, ln, z), want) and att.read_status() == 0


@pytest.mark.parametrize("dtype", [BF, F8])
def test_the_binding_itself(dtype):
    from ulysses_sequence_long_gb300 import binding as B
    lens = [40, 3]
    c, table, ln, k, v, q, z, att = _decode_case(lens, 2, 2, 64, 1, 16, dtype, sinks=True)
    cu = _cu(lens)
    pools = [None if t is None else torch.zeros_like(t) for t in (c.k_pages, c.v_pages, c.k_scales, c.v_scales)]
    prm = B.paged_cache(2, 64, 1, *pools[:2], table, ln, *pools[2:])
    B.usp_cache_append(prm, k, None, 43, cu, c.status)
    B.usp_cache_append(prm, None, v, 43, cu, c.status)
    got, want = (torch.empty_like(k), torch.empty_like(v)), c.read(table, ln, cu, tokens=43)
    B.usp_cache_read(prm, got[0], got[1], 43, cu)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ws = torch.zeros((B.usp_attn_decode_workspace_bytes(prm, 4),), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty((2, 4), device="cuda")
    B.usp_attn_decode(prm, 4, q, o, lse, ws, sinks=z, dev_status=c.status)
    assert torch.equal(o, att.forward(q, table, ln, z)) and torch.equal(lse.view(-1), att.lse.view(-1))
    bad = [lambda: B.usp_cache_append(prm, None, None, 43, cu), lambda: B.usp_cache_append(prm, k, v, 43, cu, c.status.cpu()),
           lambda: B.usp_cache_read(prm, got[0], got[1][:, :5], 43, cu), lambda: B.usp_cache_read(prm, got[0], got[0], 43, cu),
           lambda: B.usp_attn_decode(prm, 4, q, o, lse, ws[:256]), lambda: B.usp_attn_decode(prm, 4, q, q, lse, ws),
           lambda: B.usp_attn_decode(prm, 4, q, o, lse, ws.cpu()), lambda: B.usp_attn_decode(prm, 4, q, o, lse[:1], ws),
           lambda: B.paged_cache(2, 64, 1, *pools[:2], table, ln.cpu(), *pools[2:]),
           lambda: B.paged_cache(2, 64, 1, pools[0], pools[1][:, :1], table, ln, *pools[2:])]
    for f in bad:
        with pytest.raises((TypeError, ValueError, B.UspError)):
            f()
    assert c.read_status() == 0 and not ws[:12288].any()


def test_refused_tensors():
    from ulysses_sequence_long_gb300.binding import UspError
    lens = [40, 3]
    c, table, ln, k, v, q, z, att = _decode_case(lens, 2, 2, 64, 1, 16, BF, sinks=True)
    bad = [lambda: att.forward(q[:, :1], table, ln, z), lambda: att.forward(q.float(), table, ln, z),
           lambda: att.forward(q, table.long(), ln, z), lambda: att.forward(q, table, ln.cpu(), z),
           lambda: att.forward(q, table[0], ln, z), lambda: att.forward(q, table, ln, z[:2]),
           lambda: att.forward(q, table[:, ::2], ln, z), lambda: att.forward(q, table[:1], ln, z),
           lambda: att.step(q, k[:, :1], v[:, :2], table, ln, z), lambda: c.append(k, v[:, :3], table, ln, _cu(lens)),
           lambda: c.append(k, v, table, ln), lambda: c.append(k, v, table, ln, _cu([1])), lambda: c.read(table, ln, _cu(lens)),
           lambda: c.read(table, ln, _cu(lens).long(), tokens=4), lambda: c.append(k[:, :0], v[:, :0], table, ln, _cu(lens)),
           lambda: att.forward(torch.cat([q, q], 1), torch.cat([table, table]), torch.cat([ln, ln]), z)]
    for f in bad:
        with pytest.raises((TypeError, ValueError, UspError)):
            f()
    att.forward(q, table, ln, z)
    _check_decode(c, lens, k, v, q, z, att, att._out(2)[0], att.lse)
