"""fp64 restatement of attention with modified scores (TEST INFRASTRUCTURE ONLY,
as the rest of this package): a tanh cap, a linear bias by distance, a learned
bias by distance bucket, a prefix mask, on top of documents, causal order,
windows, grouped heads and sink logits.  Dense per document: small sizes.

For head h, token t and key u of the same document [a, b):

    x = scale q_t.k_u - slopes[h] |t - u| + rel_bias[h][buckets[clamp(t - u, -R, R) + R]]
    z = softcap tanh(x / softcap)
    LSE_t = ln(sum_u e^z + e^sink),  O_t = sum_u e^(z - LSE_t) v_u

Rows that see nothing have O = 0 and LSE = -inf (or the sink's logit).
"""
from __future__ import annotations

import math

import numpy as np

from .usp_oracle import cu_seqlens_from_position_ids, gather_position_ids  # noqa: F401

__all__ = ["rel_buckets_log", "visible_mask", "mod_attention", "mod_layer"]


def rel_buckets_log(n_buckets: int, max_distance: int, bidirectional: bool) -> np.ndarray:
    """Bucket of every distance t - u in -max_distance..max_distance, in exact
    integer arithmetic: past K/2 the bucket is K/2 + the largest j with
    (n / (K/2))^(K - K/2) >= (max_distance / (K/2))^j."""
    K = n_buckets // 2 if bidirectional else n_buckets
    e = K // 2
    m = K - e
    out = np.zeros(2 * max_distance + 1, dtype=np.int32)
    for d in range(-max_distance, max_distance + 1):
        n = abs(d)
        if n < e:
            b = n
        else:
            j = 0
            while j + 1 <= m and n ** m * e ** (j + 1) >= max_distance ** (j + 1) * e ** m:
                j += 1
            b = min(K - 1, e + j)
        out[d + max_distance] = b if d >= 0 else (b + K if bidirectional else 0)
    return out


def visible_mask(n: int, causal: bool, window_left: int, prefix: int) -> np.ndarray:
    """[n][n] (query, key) of one document of n tokens."""
    t, u = np.arange(n)[:, None], np.arange(n)[None, :]
    v = np.ones((n, n), dtype=bool)
    if causal:
        v &= (u <= t) | (u < prefix)
    if window_left >= 0:
        v &= t - u <= window_left
        if not causal:
            v &= u - t <= window_left
    return v


def mod_attention(q, k, v, cu, causal=True, window_left=-1, scale=None, sinks=None, softcap=0.0, slopes=None,
                  rel_bias=None, buckets=None, prefix_lens=None, do=None):
    """q [T][Hq][D], k/v [T][Hkv][D] float64 over documents cu -> dict with o
    [T][Hq][D], lse [Hq][T], and with do also dq, dk, dv, dsinks, drel_bias.

    ``*_slack`` (with do): to first order, how far an element can be off when P,
    dX and O are rounded once to bf16 (half a step: u = 2^-9 of the value) on
    the way and everything else is exact:
        |dO_td|  u sum_u P |v|                       |dV|  u sum_t P |dO|
        |dD_t|   u sum_d |dO_d| (|O_d| + sum_u P |v_d|)
        |dQ|     scale sum_u (u |dX| + P g |dD_t|) |k|,  dK alike with |q|
    with g = 1 - tanh^2."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out = {"o": np.zeros((T, Hq, D)), "lse": np.full((Hq, T), -np.inf)}
    if do is not None:
        out.update(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v))
        out.update(o_slack=np.zeros_like(q), dq_slack=np.zeros_like(q), dk_slack=np.zeros_like(k),
                   dv_slack=np.zeros_like(v))
        if sinks is not None:
            out["dsinks"] = np.zeros(Hq)
        if rel_bias is not None:
            out["drel_bias"] = np.zeros(np.shape(rel_bias))
    for i in range(len(cu) - 1):
        a, b = int(cu[i]), int(cu[i + 1])
        n = b - a
        mask = visible_mask(n, causal, window_left, 0 if prefix_lens is None else int(prefix_lens[i]))
        dist = np.arange(n)[:, None] - np.arange(n)[None, :]
        bucket = None
        if rel_bias is not None:
            R = (len(buckets) - 1) // 2
            bucket = np.asarray(buckets)[np.clip(dist, -R, R) + R]
        for h in range(Hq):
            qd, kd, vd = q[a:b, h], k[a:b, h // G], v[a:b, h // G]
            x = scale * (qd @ kd.T)
            if slopes is not None:
                x = x - float(slopes[h]) * np.abs(dist)
            if rel_bias is not None:
                row = np.asarray(rel_bias, dtype=np.float64)[h]
                x = x + np.where(row < -2.0 ** 20, -np.inf, row)[bucket]
            th = None
            if softcap:
                th = np.tanh(x / softcap)
                x = softcap * th
            x = np.where(mask, x, -np.inf)
            m = x.max(axis=1)
            if sinks is not None:
                m = np.maximum(m, float(sinks[h]))
            m0 = np.where(np.isneginf(m), 0.0, m)
            e = np.exp(x - m0[:, None])
            s = e.sum(axis=1) + (np.exp(float(sinks[h]) - m0) if sinks is not None else 0.0)
            with np.errstate(divide="ignore"):
                lse = m0 + np.log(s)
            p = e / np.where(s > 0, s, 1.0)[:, None]
            o = p @ vd
            out["o"][a:b, h] = o
            out["lse"][h, a:b] = lse
            if do is None:
                continue
            g = do[a:b, h]
            delta = (g * o).sum(axis=1)
            dx = p * (g @ vd.T - delta[:, None])
            out["dv"][a:b, h // G] += p.T @ g
            if sinks is not None:
                out["dsinks"][h] -= (np.exp(float(sinks[h]) - lse) * delta).sum()
            pv = p @ np.abs(vd)
            slip = p * (2.0 ** -9 * (np.abs(g) * (np.abs(o) + pv)).sum(axis=1))[:, None]
            if th is not None:
                dx = dx * (1.0 - th * th)
                slip = slip * (1.0 - th * th)
            slip += 2.0 ** -9 * np.abs(dx)
            out["o_slack"][a:b, h] = 2.0 ** -9 * pv
            out["dv_slack"][a:b, h // G] += 2.0 ** -9 * (p.T @ np.abs(g))
            out["dq_slack"][a:b, h] = scale * (slip @ np.abs(kd))
            out["dk_slack"][a:b, h // G] += scale * (slip.T @ np.abs(qd))
            out["dq"][a:b, h] = scale * (dx @ kd)
            out["dk"][a:b, h // G] += scale * (dx.T @ qd)
            if rel_bias is not None:
                out["drel_bias"][h] += np.bincount(bucket.reshape(-1), dx.reshape(-1), rel_bias.shape[1])
    return out


def mod_layer(q_seq, k_seq, v_seq, pos_shards, do_seq=None, **kw):
    """The layer over sequence shards [P][B][S/P][H][D]: every head sees the
    gathered sequence, so the exchange is only a reordering.  Returns o/dq/dk/dv
    as shards and lse as [P][B][Hq/P][S]."""
    P, B, Sl, Hq, D = q_seq.shape
    S = P * Sl
    flat = lambda x: np.moveaxis(x, 0, 1).reshape(B * S, x.shape[3], D)
    shards = lambda x: np.ascontiguousarray(np.moveaxis(x.reshape(B, P, Sl, x.shape[1], D), 1, 0))
    cu, _, _ = cu_seqlens_from_position_ids(pos_shards)
    r = mod_attention(flat(q_seq), flat(k_seq), flat(v_seq), cu, do=None if do_seq is None else flat(do_seq), **kw)
    r["lse"] = np.ascontiguousarray(r["lse"].reshape(P, Hq // P, B, S).transpose(0, 2, 1, 3))
    for n in ("o", "dq", "dk", "dv"):
        for m in (n, n + "_slack"):
            if m in r:
                r[m] = shards(r[m])
    return r
