"""Attention with modified scores, as cases to measure: scores capped by a tanh,
scores with a bias that grows with distance, a learned bias by distance buckets
(with its gradient), and the prefix mask of packed documents.

Per document [a, b) of the gathered sequence, query t, key u, head h:

    x = scale q_t.k_u - slopes[h] |t - u| + rel_bias[h][buckets[clamp(t - u, -R, R) + R]]
    z = softcap tanh(x / softcap)            (x itself without a cap)
    visible: u <= t, or u in the document's prefix (causal); any u (not causal);
             t - u <= window_left with a window
    LSE_t = ln(sum_u exp(z) + exp(sink_h)),  O_t = sum_u exp(z - LSE_t) v_u

and the gradients of sum(O * dO).  `run` is one forward, or one forward and
backward (a training step of the layer) where the case says "train".
"""
import math
import random

import torch

own = False

LOG_BASE = 8.0  # ALiBi's slopes: 2^(-8 (h + 1) / H)


def _case(name, mod, B, S, Hq, Hkv, D, P, train, doc_mean=0, causal=True, window=-1, sinks=False, softcap=0.0,
          n_buckets=0, max_distance=0, prefix=0.0):
    c = dict(mod=mod, B=B, S=S, Hq=Hq, Hkv=Hkv, D=D, P=P, train=train, doc_mean=doc_mean, causal=causal,
             window=window, sinks=sinks, softcap=softcap, n_buckets=n_buckets, max_distance=max_distance,
             prefix=prefix)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one forward over 256 packed tokens: launch and set-up latency of the smallest call
        _case("cap_fwd_s256", "cap", 1, 256, 4, 2, 64, 2, False, doc_mean=90, softcap=50.0),
        # a training step of a capped layer, one document, plain multi-head attention
        _case("cap_train_s4096_h12", "cap", 1, 4096, 12, 12, 128, 4, True, softcap=50.0),
        # packed documents and grouped heads at the size of the default benchmark's quarter: the largest work
        _case("cap_train_packed_s8192", "cap", 1, 8192, 32, 8, 128, 8, True, doc_mean=4096, softcap=30.0),
        # capped sliding-window layer with a sink logit per head
        _case("cap_train_window128_sinks", "cap", 1, 4096, 64, 8, 64, 8, True, window=127, sinks=True, softcap=20.0),
        # rows of odd length, several in a batch, forward alone (evaluation)
        _case("slope_fwd_rows3_s1000", "slope", 3, 1000, 8, 8, 64, 2, False, doc_mean=300),
        # a training step with a distance bias over packed documents
        _case("slope_train_packed_s8192", "slope", 1, 8192, 32, 8, 128, 8, True, doc_mean=4096),
        # the smallest training step of the learned bias: every gradient, mostly latency
        _case("rel_train_s256", "rel", 1, 256, 4, 2, 64, 2, True, doc_mean=90, n_buckets=32, max_distance=128),
        # the learned bias in a causal model, packed documents, its table's gradient over all tokens
        _case("rel_train_packed_s8192", "rel", 1, 8192, 32, 8, 128, 8, True, doc_mean=4096, n_buckets=32,
              max_distance=128),
        # the learned bias in a bidirectional encoder: buckets for both signs, a batch of rows
        _case("rel_train_bidir_rows4_s2048", "rel", 4, 2048, 12, 12, 64, 4, True, doc_mean=700, causal=False,
              n_buckets=32, max_distance=128),
        # prompts seen in both directions, answers causally, packed into one row
        _case("prefix_train_packed_s4096", "prefix", 1, 4096, 32, 8, 128, 8, True, doc_mean=1024, prefix=0.5),
        # the same for odd rows, forward alone
        _case("prefix_fwd_rows2_s1500", "prefix", 2, 1500, 8, 2, 64, 2, False, doc_mean=400, prefix=0.4),
        # a cap over a learned bias with prompts seen in both directions
        _case("cap_rel_prefix_train_s2048", "all", 1, 2048, 16, 4, 128, 4, True, doc_mean=600, softcap=30.0,
              sinks=True, n_buckets=32, max_distance=128, prefix=0.3),
    ]


def _between(rng, lo, hi):
    """A whole number spread evenly over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        mod = rng.choice(["cap", "slope", "rel", "prefix", "all"])
        D = rng.choice([64, 128])
        P = rng.choice([1, 2, 4, 8])
        Hkv = rng.choice([2, 4, 8, 12])
        Hq = Hkv * rng.choice([1, 2, 4])
        if Hq % P or (Hkv % P if Hkv >= P else P % Hkv):
            continue
        B = rng.choice([1, 1, 1, 2, 3])
        # whole shards of 128 tokens (exchanges fused into the kernels), or any multiple of the ranks
        S = _between(rng, 96, 8192)
        S = max(128 * P, S // (128 * P) * 128 * P) if rng.random() < 0.5 else max(P, S // P * P)
        if B * S > 8192 or B * S * S * Hq > 8192 * 8192 * 32:
            continue
        causal = mod in ("cap", "slope", "prefix", "all") or rng.random() < 0.5
        return _case(None, mod, B, S, Hq, Hkv, D, P, rng.random() < 0.7,
                     doc_mean=rng.choice([0, max(48, S // 7), max(64, S // 2)]), causal=causal,
                     window=rng.choice([-1, -1, 127, 500]) if mod in ("cap", "slope", "rel") else -1,
                     sinks=rng.random() < 0.3, softcap=rng.choice([15.0, 30.0, 50.0, 80.0]) if mod in ("cap", "all") else 0.0,
                     n_buckets=32 if mod in ("rel", "all") else 0,
                     max_distance=rng.choice([64, 128, 400]) if mod in ("rel", "all") else 0,
                     prefix=round(rng.uniform(0.1, 0.9), 2) if mod in ("prefix", "all") else 0.0)


# ------------------------------------------------------------------ inputs
def _doc_lengths(case):
    """Lengths of the packed documents, row by row (they go by the case alone, as its work does)."""
    rng = random.Random("%(B)d %(S)d %(doc_mean)d" % case)
    rows = []
    for _ in range(case["B"]):
        lens, left = [], case["S"]
        while left:
            n = left if not case["doc_mean"] else min(left, 1 + int(rng.expovariate(1.0 / case["doc_mean"])))
            lens.append(n)
            left -= n
        rows.append(lens)
    return rows


def _prefix_lengths(case):
    rng = random.Random("prefix %(B)d %(S)d" % case)
    return [[int(n * min(1.0, case["prefix"] * rng.uniform(0.0, 2.0))) for n in lens] for lens in _doc_lengths(case)]


def _bucket_map(case):
    """Bucket of every distance -R..R: near ones have a bucket each, farther ones share buckets whose widths
    grow geometrically; half of them for keys after the query when the model looks both ways."""
    nb, R = case["n_buckets"], case["max_distance"]
    both = not case["causal"] or case["prefix"] > 0
    half = nb // 2 if both else nb
    exact_ = half // 2

    def one(n):
        if n < exact_:
            return n
        return min(half - 1, exact_ + int(math.log(n / exact_) / math.log(R / exact_) * (half - exact_)))

    return [one(abs(d)) + (half if both and d < 0 else 0) if both or d >= 0 else 0 for d in range(-R, R + 1)]


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    B, S, Hq, Hkv, D, P = (case[k] for k in ("B", "S", "Hq", "Hkv", "D", "P"))
    # capped models' scores reach the cap: queries three times the size that 1/sqrt(D) makes of unit scores
    gain = 3.0 if case["softcap"] else 1.0
    s = dict(case=case)
    for name, H, mul in (("q", Hq, gain), ("k", Hkv, 1.0), ("v", Hkv, 1.0), ("do", Hq, 1.0)):
        if name != "do" or case["train"]:
            s[name] = (torch.randn((P, B, S // P, H, D), generator=g, device=dev) * mul).to(torch.bfloat16)
    lens = _doc_lengths(case)
    pos = torch.tensor([[i for n in row for i in range(n)] for row in lens], dtype=torch.int32)
    s["pos"] = pos.view(B, P, S // P).transpose(0, 1).contiguous().to(dev)
    s["sinks"] = torch.randn((Hq,), generator=g, device=dev) if case["sinks"] else None
    s["slopes"] = torch.tensor([2.0 ** (-LOG_BASE * (h + 1) / Hq) for h in range(Hq)],
                               device=dev) if case["mod"] == "slope" else None
    s["rel_bias"] = torch.randn((Hq, case["n_buckets"]), generator=g, device=dev) if case["n_buckets"] else None
    s["buckets"] = torch.tensor(_bucket_map(case), dtype=torch.int32, device=dev) if case["n_buckets"] else None
    s["prefix_lens"] = torch.tensor([n for row in _prefix_lengths(case) for n in row], dtype=torch.int32,
                                    device=dev) if case["prefix"] else None
    if own:  # the layer object that a program keeps: buffers of its shape
        from ulysses_sequence_long_gb300.pipeline import ScoreMods, Shape, UlyssesAttention
        mods = ScoreMods(softcap=case["softcap"], slopes=s["slopes"], rel_bias=s["rel_bias"], buckets=s["buckets"],
                         prefix_lens=s["prefix_lens"])
        s["layer"] = UlyssesAttention(Shape(B, S, Hq, Hkv, D, P, case["causal"], case["window"]),
                                      with_backward=case["train"], mods=mods)
    return s


# ------------------------------------------------------------------ the pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    layer = s["layer"]
    out = {"o": layer.forward(s["q"], s["k"], s["v"], s["pos"], s["sinks"]), "lse": layer.lse}
    if s["case"]["train"]:
        out["dq"], out["dk"], out["dv"] = layer.backward(s["do"], s["sinks"])
        if s["sinks"] is not None:
            out["dsinks"] = layer.dsinks
        if s["rel_bias"] is not None:
            out["drel_bias"] = layer.drel_bias
    return out


def _rows(x, Hkv):
    """Shards [P][B][S/P][H][D] as fp32 [B][Hkv][H/Hkv][S][D]."""
    P, B, Sl, H, D = x.shape
    return x.permute(1, 3, 0, 2, 4).reshape(B, Hkv, H // Hkv, P * Sl, D).float()


def _shards(x, P):
    """fp32 [B][Hkv][G][S][D] as bf16 shards [P][B][S/P][H][D]."""
    B, Hkv, G, S, D = x.shape
    return x.reshape(B, Hkv * G, P, S // P, D).permute(2, 0, 3, 1, 4).to(torch.bfloat16)


def _per_head(x, Hkv):
    return x.view(1, Hkv, -1, 1, 1)


def _run_plain(s):
    """The whole score matrix in 32 bits; rounded to the outputs' types at the end."""
    case = s["case"]
    P, B, Sl, Hq, D = s["q"].shape
    S, Hkv = P * Sl, case["Hkv"]
    q, k, v = _rows(s["q"], Hkv), _rows(s["k"], Hkv), _rows(s["v"], Hkv)
    scale = 1.0 / math.sqrt(D)
    pos = s["pos"].transpose(0, 1).reshape(B, S)
    starts = pos == 0
    starts[:, 0] = True
    doc = starts.long().cumsum(1)                       # document of each token, from 1
    at = torch.arange(S, device=q.device)
    dist = at[:, None] - at[None, :]                    # t - u
    seen = doc[:, :, None] == doc[:, None, :]
    if case["causal"]:
        order = dist >= 0
        if s["prefix_lens"] is not None:                # keys of a document's first tokens are seen by all of it
            number = starts.reshape(-1).long().cumsum(0).reshape(B, S) - 1
            order = order | (pos < s["prefix_lens"][number])[:, None, :]
        seen = seen & order
    if case["window"] >= 0:
        seen = seen & ((dist <= case["window"]) if case["causal"] else (dist.abs() <= case["window"]))
    hidden = ~seen[:, None, None]
    x = torch.matmul(q * scale, k.transpose(-1, -2))
    if s["slopes"] is not None:
        x -= _per_head(s["slopes"], Hkv) * dist.abs()
    if s["rel_bias"] is not None:
        R = case["max_distance"]
        bucket = s["buckets"].long()[dist.clamp(-R, R) + R]
        x += s["rel_bias"].view(Hkv, Hq // Hkv, -1)[:, :, bucket]
    th = None
    if case["softcap"]:
        th = torch.tanh(x / case["softcap"])
        x = th * case["softcap"]
    x.masked_fill_(hidden, -math.inf)
    m = x.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        m = torch.maximum(m, _per_head(s["sinks"], Hkv))
    p = torch.exp(x - m)
    del x
    total = p.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        total = total + torch.exp(_per_head(s["sinks"], Hkv) - m)
    p /= total
    o = torch.matmul(p, v)
    lse = (m + torch.log(total)).view(B, P, Hq // P, S).transpose(0, 1)
    out = {"o": _shards(o, P), "lse": lse.contiguous()}
    if not case["train"]:
        return out
    do = _rows(s["do"], Hkv)
    delta = (do * o).sum(-1, keepdim=True)
    out["dv"] = _shards(torch.matmul(p.transpose(-1, -2), do).sum(2, keepdim=True), P)
    dx = torch.matmul(do, v.transpose(-1, -2)).sub_(delta).mul_(p)
    if th is not None:
        dx *= 1.0 - th * th
    del p, th
    out["dq"] = _shards(torch.matmul(dx, k) * scale, P)
    out["dk"] = _shards(torch.matmul(dx.transpose(-1, -2), q).sum(2, keepdim=True) * scale, P)
    if s["sinks"] is not None:
        out["dsinks"] = -(torch.exp(_per_head(s["sinks"], Hkv) - (m + torch.log(total))) * delta).sum((0, 3, 4)).reshape(Hq)
    if s["rel_bias"] is not None:
        # sums along the diagonals first (64 bits: a diagonal has thousands of values, a bucket millions): with the keys
        # reversed and a row of zeros behind each row, the values of one distance stand in one column of rows of 2S - 1
        skew = torch.nn.functional.pad(dx.sum(0).view(Hq, S, S).flip(-1), (0, S)).view(Hq, 2 * S * S)
        by_dist = skew[:, :S * (2 * S - 1)].view(Hq, S, 2 * S - 1).sum(1, dtype=torch.float64)   # t - u = column - (S - 1)
        column = s["buckets"].long()[torch.arange(1 - S, S, device=q.device).clamp(-R, R) + R]
        table = torch.zeros((Hq, case["n_buckets"]), dtype=torch.float64, device=q.device)
        out["drel_bias"] = table.index_add_(1, column, by_dist).float()
    return out


# ------------------------------------------------------------------ work
def _pairs(case):
    """Visible (query, key) pairs of all documents, one head."""
    n = 0
    w = case["window"]
    for lens, pls in zip(_doc_lengths(case), _prefix_lengths(case) if case["prefix"] else [[0] * len(r) for r in _doc_lengths(case)]):
        for L, pl in zip(lens, pls):
            if not case["causal"]:
                n += L * L if w < 0 or w >= L else sum(min(t, w) + 1 + min(L - 1 - t, w) for t in range(L))
            elif w >= 0:
                n += sum(min(t, w) + 1 for t in range(L))
            else:
                n += L * (L + 1) // 2 + pl * (pl - 1) // 2
    return n


def work(case):
    B, S, Hq, Hkv, D = (case[k] for k in ("B", "S", "Hq", "Hkv", "D"))
    qb, kb, st = 2 * B * S * Hq * D, 2 * B * S * Hkv * D, 4 * B * S * Hq
    small = 4 * Hq * ((2 if case["train"] else 1) * case["n_buckets"] + 2) + 4 * B * S
    fwd = qb + 2 * kb + qb + st + small
    if not case["train"]:
        return {"bytes": fwd, "flops": 4 * D * _pairs(case) * Hq}
    return {"bytes": fwd + 2 * qb + 2 * kb, "flops": 14 * D * _pairs(case) * Hq}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """One key/value head at a time, from the definition, gradients by differentiation."""
    s = prepare(case, seed)
    P, B, S, Hq, Hkv, D = (case[k] for k in ("P", "B", "S", "Hq", "Hkv", "D"))
    G = Hq // Hkv
    f8 = dict(dtype=torch.float64, device="cuda")
    whole = {n: s[n].double().transpose(0, 1).reshape(B, S, -1, D) for n in ("q", "k", "v", "do") if n in s}
    mask = torch.zeros((B, S, S), dtype=torch.bool, device="cuda")
    for b, lens in enumerate(_doc_lengths(case)):
        a = 0
        for i, L in enumerate(lens):
            sub = mask[b, a:a + L, a:a + L]
            sub.fill_(True)
            if case["causal"]:
                sub.tril_()
                if case["prefix"]:
                    sub[:, :_prefix_lengths(case)[b][i]] = True
            if case["window"] >= 0:
                sub.triu_(-case["window"])
                if not case["causal"]:
                    sub.tril_(case["window"])
            a += L
    line = torch.arange(S, device="cuda")
    gap = line[:, None] - line[None, :]
    o, lse = torch.empty((B, S, Hq, D), **f8), torch.empty((B, Hq, S), **f8)
    grad = {n: torch.empty_like(whole[n]) for n in ("q", "k", "v")} if case["train"] else {}
    dsinks, drel = torch.zeros((Hq,), **f8), torch.zeros((Hq, max(1, case["n_buckets"])), **f8)
    for b in range(B):
        for h in range(Hkv):
            heads = slice(h * G, (h + 1) * G)
            q = whole["q"][b, :, heads].transpose(0, 1).clone().requires_grad_(case["train"])
            k = whole["k"][b, :, h].clone().requires_grad_(case["train"])
            v = whole["v"][b, :, h].clone().requires_grad_(case["train"])
            leaves = [q, k, v]
            x = q @ k.T / math.sqrt(D)
            if s["slopes"] is not None:
                x = x - s["slopes"][heads].double()[:, None, None] * gap.abs()
            if s["rel_bias"] is not None:
                rel = s["rel_bias"][heads].double().requires_grad_(case["train"])
                leaves.append(rel)
                R = case["max_distance"]
                by_gap = rel[:, s["buckets"].long()]
                x = x + by_gap.gather(1, (gap.clamp(-R, R) + R).reshape(1, -1).expand(G, -1)).view(G, S, S)
            if case["softcap"]:
                x = case["softcap"] * torch.tanh(x / case["softcap"])
            x = x.masked_fill(~mask[b], -math.inf)
            total = torch.logsumexp(x, -1)
            if s["sinks"] is not None:
                sink = s["sinks"][heads].double().requires_grad_(case["train"])
                leaves.append(sink)
                total = torch.logaddexp(total, sink[:, None].expand(G, S))
            y = torch.exp(x - total[..., None]) @ v
            o[b, :, heads] = y.detach().transpose(0, 1)
            lse[b, heads] = total.detach()
            if case["train"]:
                got = list(torch.autograd.grad((y * whole["do"][b, :, heads].transpose(0, 1)).sum(), leaves))
                grad["q"][b, :, heads] = got.pop(0).transpose(0, 1)
                grad["k"][b, :, h], grad["v"][b, :, h] = got.pop(0), got.pop(0)
                if s["rel_bias"] is not None:
                    drel[heads] += got.pop(0)
                if s["sinks"] is not None:
                    dsinks[heads] += got.pop(0)
            del x, total, y

    def shards(t):
        return t.reshape(B, P, S // P, *t.shape[2:]).transpose(0, 1).contiguous()

    out = {"o": shards(o), "lse": lse.view(B, P, Hq // P, S).transpose(0, 1).contiguous()}
    for n in grad:
        out["d" + n] = shards(grad[n])
    if case["train"] and case["sinks"]:
        out["dsinks"] = dsinks
    if case["train"] and case["n_buckets"]:
        out["drel_bias"] = drel
    return out
