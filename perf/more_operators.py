"""Rotary positions, a paged key/value cache and the attention of one new token
over it, as cases to measure.

Rotary positions of several axes (text: one; images: height, width; video: time,
height, width).  Pair i of a head's elements turns by the angle of its axis,
w = positions[axes[i]] freqs[i]:

    y1 = x1 cos w - x2 sin w,   y2 = x1 sin w + x2 cos w

with (x1, x2) = elements (i, i + n) or (2i, 2i + 1), n pairs in all; elements
behind the pairs pass through.  The gradient turns back by the same angles.

The cache holds tokens in pages of `page` tokens, [rank][page][head][token][D];
position t of sequence s is token t % page of page block_table[s][t // page].
In 8 bits (e4m3) each token and head has a power of two, 2^e with the smallest
e >= -126 for which every |x| <= 448 2^e, and holds x / 2^e.  Appending writes the
last tokens of each sequence, reading gives them back.

One new token per sequence, query head h over key/value head h / (Hq / Hkv),
positions u < lens[s] (and u >= lens[s] - 1 - window with a window):

    s_u = q.k_u / sqrt(D),  LSE = ln(sum_u exp(s_u) + exp(sink_h)),  O = sum_u exp(s_u - LSE) v_u

(O = 0 and LSE = -inf, or the sink, where nothing is visible).
"""
import math
import random

import torch

own = False

BASE = 10000.0   # the rotation's slowest pair turns once in about 2 pi BASE positions


def _rope(name, B, S, Hq, Hkv, D, P, train, n_axes=1, pairs=0, interleaved=False, first=0):
    c = dict(op="rope", B=B, S=S, Hq=Hq, Hkv=Hkv, D=D, P=P, train=train, n_axes=n_axes, pairs=pairs or D // 2,
             interleaved=interleaved, first=first)
    return dict(c, name=name) if name else c


def _cache(name, op, seqs, new, past, Hkv, D, P, page, eight, ragged=True):
    c = dict(op=op, seqs=seqs, new=new, past=past, Hkv=Hkv, D=D, P=P, page=page, eight=eight, ragged=ragged)
    return dict(c, name=name) if name else c


def _decode(name, seqs, len_, Hq, Hkv, D, P, page, eight, ragged=True, window=-1, sinks=False, empty=False):
    c = dict(op="decode", seqs=seqs, len=len_, Hq=Hq, Hkv=Hkv, D=D, P=P, page=page, eight=eight, ragged=ragged,
             window=window, sinks=sinks, empty=empty)
    return dict(c, name=name) if name else c


def listed():
    return [
        # queries and keys of one new token for four sequences, far in a text: the latency of the smallest call
        _rope("rope_fwd_one_token_b4", 4, 1, 32, 8, 128, 1, False, first=100000),
        # a training step of an image model: odd rows, height and width, neighbouring pairs, half of each head turned
        _rope("rope_train_image_rows3_s1000", 3, 1000, 12, 12, 64, 4, True, n_axes=2, pairs=16, interleaved=True),
        # a training step of a video model at the default benchmark's size: time, height and width
        _rope("rope_train_video_s32768", 1, 32768, 32, 8, 128, 8, True, n_axes=3),
        # one new token for each of 64 sequences goes into the 8-bit cache: mostly latency
        _cache("append_e4m3_one_token_b64", "append", 64, 1, 3000, 8, 128, 8, 64, True),
        # packed prompts go into the 8-bit cache after their exchange
        _cache("append_e4m3_packed_prompts", "append", 8, 6300, 0, 8, 128, 8, 64, True),
        # prompts continued over a 16-bit cache with small pages
        _cache("append_bf16_continued_prompts", "append", 5, 2400, 1000, 8, 64, 2, 16, False),
        # an 8-bit cache read back as keys and values of the attention kernels
        _cache("read_e4m3_packed_prompts", "read", 8, 6300, 0, 8, 128, 8, 64, True),
        # the last tokens of a few sequences read back
        _cache("read_bf16_few_tokens", "read", 3, 100, 700, 2, 128, 2, 32, False),
        # the smallest step: one sequence of a short conversation
        _decode("decode_bf16_b1_len500", 1, 500, 32, 8, 128, 1, 64, False, ragged=False),
        # a batch of long conversations: the cache is most of the card's traffic
        _decode("decode_bf16_b32_len8192", 32, 8192, 32, 8, 128, 8, 64, False),
        # one very long document in 8 bits: few rows, split over its length
        _decode("decode_e4m3_b1_len131072", 1, 131072, 28, 4, 128, 4, 128, True, ragged=False),
        # many sequences in a layer with a window and sinks; some places of the batch are empty
        _decode("decode_bf16_window128_b256", 256, 2000, 64, 8, 64, 8, 16, False, window=127, sinks=True, empty=True),
    ]


def _between(rng, lo, hi):
    """A whole number spread evenly over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["rope", "rope", "append", "read", "decode", "decode", "decode"])
        D = rng.choice([64, 128])
        P = rng.choice([1, 2, 4, 8])
        Hkv = rng.choice([1, 2, 4, 8, 12])
        Hq = Hkv * rng.choice([1, 2, 4, 7, 8])
        if Hq % P or (Hkv % P if Hkv >= P else P % Hkv):
            continue
        if op == "rope":
            B, S = rng.choice([1, 1, 2, 3]), P * _between(rng, 1, 4096)
            if B * S * (Hq + Hkv) * D > 32768 * 40 * 128:
                continue
            return _rope(None, B, S, Hq, Hkv, D, P, rng.random() < 0.7, n_axes=rng.choice([1, 2, 3, 3, 4]),
                         pairs=rng.choice([D // 2, D // 2, D // 4, 24]), interleaved=rng.random() < 0.5,
                         first=rng.choice([0, 0, 1000, 1000000]))
        page, eight, ragged = rng.choice([16, 32, 64, 128, 256]), rng.random() < 0.5, rng.random() < 0.7
        seqs = _between(rng, 1, 256)
        if op == "decode":
            n = _between(rng, 1, 131072)
            if seqs * n * Hkv * D > 32 * 8192 * 8 * 128:
                continue
            return _decode(None, seqs, n, Hq, Hkv, D, P, page, eight, ragged, window=rng.choice([-1, -1, 127, 1000]),
                           sinks=rng.random() < 0.3, empty=rng.random() < 0.3)
        new, past = rng.choice([1, _between(rng, 1, 16384)]), rng.choice([0, _between(rng, 1, 4096)])
        if seqs * (new + past) * Hkv * D > 32768 * 8 * 128:
            continue
        return _cache(None, op, seqs, new, past, Hkv, D, P, page, eight, ragged)


# ------------------------------------------------------------------ inputs
def _heads(case):
    """Key/value heads of a rank: one, on several ranks, where there are fewer of them than ranks."""
    return max(1, case["Hkv"] // case["P"])


def _counts(case):
    """(length of each sequence, tokens of it that are appended or read), by the case alone, as its work is."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    some = lambda n: max(1, int(n * rng.uniform(0.3, 1.0))) if case["ragged"] else n
    if case["op"] == "decode":
        return [0 if case["empty"] and i % 5 == 3 else some(case["len"]) for i in range(case["seqs"])], [1] * case["seqs"]
    new = [1 if case["new"] == 1 else some(case["new"]) for _ in range(case["seqs"])]
    return [n + (some(case["past"]) if case["past"] else 0) for n in new], new


def _frequencies(case):
    """Each axis has a ladder of its own, from one radian a position down to nearly 1 / BASE."""
    n, a = case["pairs"], case["n_axes"]
    sizes = [n // a + (1 if i < n % a else 0) for i in range(a)]
    return [BASE ** (-j / m) for m in sizes for j in range(m)], [i for i, m in enumerate(sizes) for _ in range(m)]


def _power(e):
    """2^e in 32 bits, exactly (a power function may be a step off, which moves ties of a rounding)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _to_8_bits(x):
    """(e4m3 values, exponents) of x [..., D]."""
    amax = x.float().abs().amax(-1)
    m, e = torch.frexp(amax)                         # amax = m 2^e with m in [0.5, 1);  448 = 0.875 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, -126).clamp(min=-126)
    return (x.float() * _power(-e)[..., None]).to(torch.float8_e4m3fn), e


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    randn = lambda *shape: torch.randn(shape, generator=g, device=dev).to(torch.bfloat16)
    s = dict(case=case)
    P, D = case["P"], case["D"]
    if case["op"] == "rope":
        B, Sl, n_axes = case["B"], case["S"] // P, case["n_axes"]
        for name, H in (("q", case["Hq"]), ("k", case["Hkv"])):
            s[name] = randn(P, B, Sl, H, D)
            if case["train"]:
                s["d" + name] = randn(P, B, Sl, H, D)
            for out in ("_out", "_in")[:1 + case["train"]]:
                s[name + out] = torch.empty_like(s[name])
        at = case["first"] + torch.arange(case["S"], device=dev, dtype=torch.int32)
        if n_axes == 1:
            axes = [at]
        else:  # frames of side x side patches, in raster order
            side = max(1, round(math.sqrt(case["S"] / 8)))
            t, h, w = at // (side * side), at // side % side, at % side
            axes = ([h, w] if n_axes == 2 else [t, h, w, at])[:n_axes]
        grid = torch.stack(axes).view(n_axes, P, 1, Sl).expand(n_axes, P, B, Sl)
        s["pos"] = (grid + torch.randint(0, 16, (n_axes, 1, B, 1), generator=g, device=dev)).to(torch.int32).contiguous()
        freqs, axes = _frequencies(case)
        s["freqs"] = torch.tensor(freqs, dtype=torch.float32, device=dev)
        s["axes"] = torch.tensor(axes, dtype=torch.int32, device=dev)
        if own:
            from ulysses_sequence_long_gb300.pipeline import Rotary
            s["rope"] = Rotary(s["freqs"], s["axes"], n_axes, interleaved=case["interleaved"])
        return s
    page, hk, seqs = case["page"], _heads(case), case["seqs"]
    lens, new = _counts(case)
    pages = [-(-n // page) for n in lens]
    n_pages = sum(pages) + 3
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    rows = torch.cat([torch.full((n,), i) for i, n in enumerate(pages)]).to(dev)
    cols = torch.cat([torch.arange(n) for n in pages]).to(dev)
    s["table"] = torch.full((seqs, max(pages + [1])), -1, dtype=torch.int32, device=dev)
    s["table"][rows, cols] = order[:sum(pages)]
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    for name in ("k", "v"):  # what earlier tokens and earlier sequences left in the pool
        x = torch.empty((P, n_pages, hk, page, D), dtype=torch.bfloat16, device=dev)
        for r in range(P):
            x[r] = randn(n_pages, hk, page, D)
        if case["eight"]:
            vals, exps = zip(*[_to_8_bits(x[r]) for r in range(P)])
            x, s[name + "_scales"] = torch.stack(vals), (torch.stack(exps) + 127).to(torch.uint8)
        s[name + "_pages"] = x
    if case["op"] == "decode":
        s["q"] = (randn(P, seqs, case["Hq"] // P, D) * 1.5).to(torch.bfloat16)
        s["sinks"] = torch.randn((case["Hq"],), generator=g, device=dev) if case["sinks"] else None
    else:
        s["cu"] = None if max(new) == 1 else torch.tensor([0] + new, dtype=torch.int32, device=dev).cumsum(0).to(torch.int32)
        for name in ("k", "v"):
            s[name] = randn(P, sum(new), hk, D) * 2 if case["op"] == "append" else torch.empty(
                (P, sum(new), hk, D), dtype=torch.bfloat16, device=dev)
    if own:
        from ulysses_sequence_long_gb300.serving import DecodeAttention, PagedCache
        cache = s["cache"] = PagedCache(n_pages, page, case["Hkv"], D, P,
                                        dtype=torch.float8_e4m3fn if case["eight"] else torch.bfloat16)
        for name in ("k_pages", "v_pages") + (("k_scales", "v_scales") if case["eight"] else ()):
            getattr(cache, name).copy_(s.pop(name))
        if case["op"] == "decode":
            s["layer"] = DecodeAttention(cache, case["Hq"], seqs, window_left=case["window"])
    return s


# ------------------------------------------------------------------ the pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    op = s["case"]["op"]
    if op == "rope":
        q, k = s["rope"].forward(s["q"], s["k"], s["pos"], out=(s["q_out"], s["k_out"]))
        out = {"q": q, "k": k}
        if s["case"]["train"]:
            out["dq"], out["dk"] = s["rope"].backward(s["dq"], s["dk"], s["pos"], out=(s["q_in"], s["k_in"]))
        return out
    cache = s["cache"]
    if op == "append":
        cache.append(s["k"], s["v"], s["table"], s["lens"], s["cu"])
        return _pools(cache.k_pages, cache.v_pages, cache.k_scales, cache.v_scales)
    if op == "read":
        k, v = cache.read(s["table"], s["lens"], s["cu"], out=(s["k"], s["v"]))
        return {"k": k, "v": v}
    o = s["layer"].forward(s["q"], s["table"], s["lens"], s["sinks"])
    return {"o": o, "lse": s["layer"].lse}


def _pools(k, v, k_scales, v_scales):
    """The cache's tensors; in 8 bits the values that the codes are, and the exponents (by 127 larger), whole numbers."""
    out = {"k": k, "v": v}
    if k_scales is not None:
        out["k_scales"], out["v_scales"] = k_scales, v_scales
    return out


def _turn(x, cos, sin, pairs, interleaved):
    """x [..., H, D] turned; cos, sin [..., 1, pairs]."""
    x = x.float()
    y = x.clone()
    if interleaved:
        a, b = slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)
    else:
        a, b = slice(0, pairs), slice(pairs, 2 * pairs)
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y.to(torch.bfloat16)


def _places(s):
    """(page, token in it) of each token that is appended or read."""
    page = s["case"]["page"]
    lens = s["lens"].long()
    if s["cu"] is None:
        seq, pos = torch.arange(lens.numel(), device=lens.device), lens - 1
    else:
        cu = s["cu"].long()
        at = torch.arange(s["k"].shape[1], device=lens.device)
        seq = torch.searchsorted(cu, at, right=True) - 1
        pos = lens[seq] - (cu[seq + 1] - at)
    return s["table"][seq, pos // page].long(), pos % page


def _run_plain(s):
    case = s["case"]
    if case["op"] == "rope":
        # 64 bits: a far position's angle has no digits behind the point in 32
        w = s["pos"].double()[s["axes"].long()].movedim(0, -1) * s["freqs"].double()
        cos, sin = torch.cos(w).float().unsqueeze(-2), torch.sin(w).float().unsqueeze(-2)
        how = case["pairs"], case["interleaved"]
        out = {"q": _turn(s["q"], cos, sin, *how), "k": _turn(s["k"], cos, sin, *how)}
        if case["train"]:
            out["dq"], out["dk"] = _turn(s["dq"], cos, -sin, *how), _turn(s["dk"], cos, -sin, *how)
        return out
    if case["op"] == "append":
        page, at = _places(s)
        scales = None, None
        if case["eight"]:
            (k, ke), (v, ve) = _to_8_bits(s["k"]), _to_8_bits(s["v"])
            s["k_scales"][:, page, :, at] = (ke + 127).to(torch.uint8).transpose(0, 1)
            s["v_scales"][:, page, :, at] = (ve + 127).to(torch.uint8).transpose(0, 1)
            scales = s["k_scales"], s["v_scales"]
        else:
            k, v = s["k"], s["v"]
        as_bits = torch.uint8 if case["eight"] else torch.bfloat16
        for pool, x in ((s["k_pages"], k), (s["v_pages"], v)):
            pool.view(as_bits)[:, page, :, at] = x.view(as_bits).transpose(0, 1)
        return _pools(s["k_pages"], s["v_pages"], *scales)
    if case["op"] == "read":
        page, at = _places(s)
        out = {}
        for name in ("k", "v"):
            if case["eight"]:
                x = s[name + "_pages"].view(torch.uint8)[:, page, :, at].view(torch.float8_e4m3fn).float()
                x = x * _power(s[name + "_scales"][:, page, :, at].int() - 127)[..., None]
            else:
                x = s[name + "_pages"][:, page, :, at]
            out[name] = x.transpose(0, 1).to(torch.bfloat16).contiguous()
        return out
    return _decode_plain(s)


def _gathered(s, name, table):
    """fp32 [P][seqs][hk][places][D] of the table's pages."""
    P, _, hk, page, D = s[name + "_pages"].shape
    if s["case"]["eight"]:
        x = s[name + "_pages"].view(torch.uint8)[:, table].view(torch.float8_e4m3fn).float()
        x = x * _power(s[name + "_scales"][:, table].int() - 127)[..., None]
    else:
        x = s[name + "_pages"][:, table].float()
    return x.permute(0, 1, 3, 2, 4, 5).reshape(P, table.shape[0], hk, -1, D)


def _decode_plain(s):
    case = s["case"]
    P, seqs, hq, D = s["q"].shape
    hk = _heads(case)
    table = s["table"].long().clamp(min=0)
    at = torch.arange(table.shape[1] * case["page"], device=table.device)
    lens = s["lens"][:, None]
    seen = at < lens
    if case["window"] >= 0:
        seen = seen & (at >= lens - 1 - case["window"])
    hidden = ~seen[None, :, None, None, :]
    q = s["q"].float().view(P, seqs, hk, hq // hk, D)
    x = torch.matmul(q, _gathered(s, "k", table).transpose(-1, -2)) / math.sqrt(D)
    x.masked_fill_(hidden, -math.inf)
    m = x.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        z = s["sinks"].view(P, 1, hk, hq // hk, 1)
        m = torch.maximum(m, z)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    del x
    total = p.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        total = total + torch.exp(z - m)
    lse = m + torch.log(total)
    p /= torch.where(total == 0, 1.0, total)
    v = _gathered(s, "v", table).masked_fill_(hidden.squeeze(3)[..., None], 0.0)
    return {"o": torch.matmul(p, v).view(P, seqs, hq, D).to(torch.bfloat16), "lse": lse.view(P, seqs, hq)}


# ------------------------------------------------------------------ work
def work(case):
    P, D = case["P"], case["D"]
    if case["op"] == "rope":
        tok, H = case["B"] * case["S"], case["Hq"] + case["Hkv"]
        passes = 2 if case["train"] else 1
        return {"bytes": passes * 4 * tok * H * D + 4 * case["n_axes"] * tok, "flops": passes * 6 * tok * H * case["pairs"]}
    hk = _heads(case)
    lens, new = _counts(case)
    held = 2 * P * hk * (D + 1 if case["eight"] else 2 * D)     # bytes of a token's keys and values in the cache
    if case["op"] != "decode":
        return {"bytes": sum(new) * (held + 2 * P * hk * 2 * D) + sum(4 * (2 + -(-n // case["page"])) for n in new),
                "flops": sum(new) * 2 * P * hk * D}
    seen = [n if case["window"] < 0 else min(n, case["window"] + 1) for n in lens]
    return {"bytes": sum(seen) * held + case["seqs"] * case["Hq"] * (4 * D + 4) + sum(4 * (1 + -(-n // case["page"])) for n in seen),
            "flops": 4 * D * case["Hq"] * sum(seen)}


# ------------------------------------------------------------------ 64 bits
def _two_to(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _as_8_bits(x):
    """The e4m3 value next to each x (ties to even) and its exponent, by arithmetic on doubles."""
    big = x.abs().amax(-1, keepdim=True)
    m, up = torch.frexp(big / 448)
    e = torch.where(big > 0, up - (m == 0.5).to(up.dtype), -126).clamp(min=-126)
    y = x * _two_to(-e)
    step = _two_to((torch.frexp(y)[1] - 1).clamp(min=-6) - 3)
    return torch.round(y / step) * step, (e.squeeze(-1) + 127).to(torch.uint8)


def exact(case, seed):
    """Rotations as products of complex numbers; the cache and the attention one sequence at a time."""
    s = prepare(case, seed)
    P, D = case["P"], case["D"]
    if case["op"] == "rope":
        n = case["pairs"]
        w = torch.stack([s["pos"][a].double() * f for a, f in zip(s["axes"].tolist(), s["freqs"].tolist())], -1)
        out = {}
        for name in ("q", "k") + (("dq", "dk") if case["train"] else ()):
            x = s[name].double()
            turn = torch.polar(torch.ones_like(w), -w if name[0] == "d" else w)[..., None, :]
            if case["interleaved"]:
                z = torch.view_as_complex(x[..., :2 * n].reshape(*x.shape[:-1], n, 2).contiguous()) * turn
                x[..., :2 * n] = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(x[..., :n].contiguous(), x[..., n:2 * n].contiguous()) * turn
                x[..., :n], x[..., n:2 * n] = z.real, z.imag
            out[name] = x
        return out
    page, hk = case["page"], _heads(case)
    lens, new = _counts(case)
    table = s["table"].cpu()

    def sequence(name, i, a, b):
        """Positions a..b of sequence i, [P][hk][b - a][D]."""
        if a >= b:
            return torch.zeros((P, hk, 0, D), dtype=torch.float64, device="cuda")
        use = table[i, a // page:-(-b // page)].long().cuda()
        x = (s[name + "_pages"].view(torch.uint8)[:, use].view(torch.float8_e4m3fn) if case["eight"] else s[name + "_pages"][:, use]).double()
        if case["eight"]:
            x = x * _two_to(s[name + "_scales"][:, use].int() - 127)[..., None]
        x = x.transpose(1, 2).reshape(P, hk, -1, D)
        return x[:, :, a - a // page * page:][:, :, :b - a]

    if case["op"] == "read":
        return {name: torch.cat([sequence(name, i, lens[i] - new[i], lens[i]).transpose(1, 2) for i in range(case["seqs"])], 1)
                for name in ("k", "v")}
    if case["op"] == "append":
        where = [int(table[i, t // page]) * page + t % page for i in range(case["seqs"]) for t in range(lens[i] - new[i], lens[i])]
        where = torch.tensor(where, device="cuda")
        out = {}
        for name in ("k", "v"):
            x, pool = s[name].double(), s[name + "_pages"].double().transpose(2, 3).reshape(P, -1, hk, D)
            if case["eight"]:
                x, e = _as_8_bits(x)
                exps = s[name + "_scales"].transpose(2, 3).reshape(P, -1, hk)
                exps[:, where] = e
                out[name + "_scales"] = exps.view(P, -1, page, hk).transpose(2, 3)
            pool[:, where] = x
            out[name] = pool.view(P, -1, page, hk, D).transpose(2, 3)
        return out
    G = case["Hq"] // P // hk
    o, lse = [], []
    for i, n in enumerate(lens):
        a = 0 if case["window"] < 0 else max(0, n - 1 - case["window"])
        k, v = sequence("k", i, a, n), sequence("v", i, a, n)
        x = s["q"][:, i].double().view(P, hk, G, D) @ k.transpose(-1, -2) / math.sqrt(D)
        if s["sinks"] is not None:
            x = torch.cat([x, s["sinks"].double().view(P, hk, G, 1)], -1)
        total = torch.logsumexp(x, -1)
        p = torch.exp(x - total[..., None])[..., :n - a] if x.shape[-1] else x
        o.append((p @ v).reshape(P, case["Hq"] // P, D))
        lse.append(total.reshape(P, case["Hq"] // P))
    return {"o": torch.stack(o, 1), "lse": torch.stack(lse, 1)}
