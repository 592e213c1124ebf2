// usp_attn_mods.cuh — what the attention kernels do between the scores and the
// softmax when the scores are modified (usp_attn_mod_* of include/usp.h): the
// kernel parameters, the prefix mask, and the arithmetic of the cap and the
// biases.  The kernels take the parameters as a template type: `NoMods` leaves
// the plain kernels as they are, `Mods` compiles the modified ones.
//
// A raw score s (a dot product) of query t and key u becomes, in the log2
// domain (x2 = x log2 e),
//     x2 = s scale log2e - slope log2e |t-u| + table[t-u] log2e
//     z2 = c2 tanh(x / c),  c2 = c log2e           (with a cap c)
// so that the softmax weight is 2^(z2 - LSE2) as in the plain kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "usp_attn_common.cuh"

namespace usp {

constexpr int kMaxBiasDistance = 2048;  // largest R of a bias table (its rows live in shared memory in the forward)
constexpr float kLog2E = 1.4426950408889634f;

// A bias row by distance covers -R-kTabPad .. R+kTabPad, the entries beyond
// +-R holding the end values: a block of scores whose distances reach inside
// (-R, R) anywhere then indexes the row without clamping, since a block spans
// at most 32 rows x 128 keys.
constexpr int kTabPad = 160;
__host__ __device__ constexpr int tab_len(int R) { return 2 * (R + kTabPad) + 1; }

struct NoMods {
  static constexpr bool on = false;
};

struct ModArgs {
  float cap;               // softcap, 0: none
  const float* slopes;     // global [Hq] or null
  const float* rel_bias;   // global [Hq][n_buckets] or null
  const int32_t* buckets;  // [2R+1]
  int n_buckets, R;
  bool later_hidden;       // causal without a prefix: no row sees a key after it
  const int32_t* prefix;   // [n_prefix] or null
  int n_prefix;
  // backward: the expanded rows [Hq][tab_len(R)] (log2 domain), and the partial
  // sums of dX by distance [Hq][n_kb][4][2R+1] (null: the table's gradient is not asked for)
  const float* table;
  float* partial;
  int n_kb;  // 32-key blocks of the rank-local tokens
};

// The compiled combinations: a kernel that tests for the cap and the biases at
// run time keeps their registers alive, and the ones at the 168-register limit
// then spill (prefixes cost a few instructions per tile and are tested for).
template <bool CAP, bool BIAS>
struct Mods : ModArgs {
  static constexpr bool on = true;
};

template <class M>
constexpr bool bias_on = false;
template <bool CAP, bool BIAS>
constexpr bool bias_on<Mods<CAP, BIAS>> = BIAS;
template <class M>
constexpr bool cap_on = false;
template <bool CAP, bool BIAS>
constexpr bool cap_on<Mods<CAP, BIAS>> = CAP;

// f(M{}) with the combination that `m` needs.
template <class F>
auto with_mods(const ModArgs& m, F f) {
  const bool bias = m.slopes != nullptr || m.rel_bias != nullptr;
  if (m.cap > 0.f) return bias ? f(Mods<true, true>{m}) : f(Mods<true, false>{m});
  return bias ? f(Mods<false, true>{m}) : f(Mods<false, false>{m});
}

// The partial sums (distance -R at 0) of head hg over the 32 keys from `uw` and
// query group `grp` of the dK/dV pass.
constexpr int kModGroups = 4;
__device__ __forceinline__ float* rel_row(const ModArgs& m, int hg, int uw, int grp) {
  return m.partial + ((static_cast<size_t>(hg) * m.n_kb + (uw >> 5)) * kModGroups + grp) * (2 * m.R + 1);
}

// Bucket of distance index i, clamped into the table; an id outside it is reported.
__device__ __forceinline__ int checked_bucket(const ModArgs& m, int i, int32_t* status) {
  const int b = gld(m.buckets + i);
  if (b < 0 || b >= m.n_buckets) set_status(status, USP_ERR_BAD_MODS);
  return min(max(b, 0), m.n_buckets - 1);
}

// Entry e (of tab_len(R)) of head h's row by distance, in the log2 domain.  Beyond
// 2^20 a bias leaves nothing of a score in fp32: below it hides the key as -inf does
// (a mask of the type's lowest value among them), above it is reported.
constexpr float kMaxBias = 0x1p20f, kMaxSlope = 0x1p10f;
__device__ __forceinline__ float table_entry(const ModArgs& m, int h, int e, int32_t* status) {
  const int d = min(max(e - (m.R + kTabPad), -m.R), m.R);
  const float v = gld(m.rel_bias + static_cast<size_t>(h) * m.n_buckets + checked_bucket(m, d + m.R, status));
  if (!(v <= kMaxBias)) set_status(status, USP_ERR_BAD_MODS);
  return v < -kMaxBias ? -INFINITY : v * kLog2E;
}

__device__ __forceinline__ float checked_slope(const ModArgs& m, int h, int32_t* status) {
  const float v = gld(m.slopes + h);
  if (!(fabsf(v) <= kMaxSlope)) set_status(status, USP_ERR_BAD_MODS);
  return v;
}

// One past the last prefix token of document d = [a, b).
__device__ __forceinline__ int prefix_end(const ModArgs& m, int d, int a, int b, int32_t* status) {
  if (m.prefix == nullptr) return a;
  if (d >= m.n_prefix) {
    set_status(status, USP_ERR_BAD_MODS);
    return a;
  }
  const int len = gld(m.prefix + d);
  if (len < 0) set_status(status, USP_ERR_BAD_MODS);
  return a + min(max(len, 0), b - a);
}

// doc_bounds with the end of the document's prefix (pe = a without one).
__device__ __forceinline__ void doc_bounds(const AttnArgs& p, const NoMods&, int n, int t, int& a, int& b, int& pe) {
  doc_bounds(p.cu, n, p.BS, t, a, b);
  pe = a;
}
__device__ __forceinline__ void doc_bounds(const AttnArgs& p, const ModArgs& m, int n, int t, int& a, int& b, int& pe) {
  const int d = find_doc(p.cu, n, t);
  a = max(0, min(gld(p.cu + d), t));
  b = min(p.BS, max(gld(p.cu + d + 1), t + 1));
  pe = prefix_end(m, d, a, b, p.status);
}

// visible_keys with a prefix: the keys of a causal row are [a, max(t, pe - 1)],
// still one interval; the window bounds t - u only, so it never hides a later key.
template <class M>
__device__ __forceinline__ void visible_keys(const M&, int t, int a, int b, int pe, int causal, int wl, bool ok,
                                             int& vlo, int& vhi) {
  visible_keys(t, a, b, causal, wl, ok, vlo, vhi);
  if constexpr (M::on) {
    if (ok && causal) vhi = max(vhi, min(pe, b) - 1);
  }
}

// visible_rows with a prefix: a prefix key is seen by every row of its document.
template <class M>
__device__ __forceinline__ void visible_rows(const M&, int u, int a, int b, int pe, int causal, int wl, bool ok,
                                             int& vlo, int& vhi) {
  visible_rows(u, a, b, causal, wl, ok, vlo, vhi);
  if constexpr (M::on) {
    if (ok && causal && u < pe) vlo = a;
  }
}

// key_range / query_range with a prefix.  Rows before the last row's document
// end before it starts, so only that document's prefix can reach past t_last;
// keys after the first key's document start after it, so only that document's
// prefix rows can lie before u_first.
template <class M>
__device__ __forceinline__ void key_range(const AttnArgs& p, const M& m, int n, int t_first, int t_last, int& lo,
                                          int& hi) {
  key_range(p, n, t_first, t_last, lo, hi);
  if constexpr (M::on) {
    if (p.causal && m.prefix != nullptr) {
      int a, b, pe;
      doc_bounds(p, m, n, t_last, a, b, pe);
      hi = max(hi, pe);
    }
  }
}
template <class M>
__device__ __forceinline__ void query_range(const AttnArgs& p, const M& m, int n, int u_first, int u_last, int& lo,
                                            int& hi) {
  query_range(p, n, u_first, u_last, lo, hi);
  if constexpr (M::on) {
    if (p.causal && m.prefix != nullptr) {
      int a, b, pe;
      doc_bounds(p, m, n, u_first, a, b, pe);
      if (u_first < pe) lo = a;
    }
  }
}

// find_doc by a whole warp, for one token: 32 boundaries are looked at at once
// instead of one after the other.
__device__ __forceinline__ int find_doc_warp(const int32_t* cu, int n, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const unsigned at_or_before = __ballot_sync(0xffffffffu, at < hi && gld(cu + at) <= t) | 1u;  // (cu[lo] <= t)
    lo += (31 - __clz(at_or_before)) * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// The documents of a tile's first and last token, found by a whole warp.
struct TileDocs {
  int d0, a0, b0, pe0, d1, a1, b1, pe1;
};
template <class M>
__device__ __forceinline__ TileDocs tile_docs(const AttnArgs& p, const M& m, int n, int first, int last) {
  TileDocs w;
  w.d0 = find_doc_warp(p.cu, n, first);
  w.a0 = max(0, min(gld(p.cu + w.d0), first));
  w.b0 = min(p.BS, max(gld(p.cu + w.d0 + 1), first + 1));
  w.pe0 = prefix_end(m, w.d0, w.a0, w.b0, p.status);
  w.d1 = w.d0;
  w.a1 = w.a0;
  w.b1 = w.b0;
  w.pe1 = w.pe0;
  if (last >= w.b0) {
    w.d1 = find_doc_warp(p.cu, n, last);
    w.a1 = max(0, min(gld(p.cu + w.d1), last));
    w.b1 = min(p.BS, max(gld(p.cu + w.d1 + 1), last + 1));
    w.pe1 = prefix_end(m, w.d1, w.a1, w.b1, p.status);
  }
  return w;
}

// checked_docs and tile_docs together, their loads in flight at the same time:
// false (the status recorded) when cu_seqlens cannot describe the sequence.  The
// lookups stay inside cu_seqlens whatever it holds, since 1 <= n <= B*S.
template <class M>
__device__ __forceinline__ bool checked_tile_docs(const AttnArgs& p, const M& m, int first, int last, int& n,
                                                  TileDocs& w) {
  n = gld(p.n_docs);
  bool ok = n >= 1 && n <= p.BS;
  if (ok) {
    const int c0 = gld(p.cu), cn = gld(p.cu + n);
    w = tile_docs(p, m, n, first, last);
    ok = c0 == 0 && cn == p.BS;
  }
  if (!ok) {
    if (threadIdx.x == 0) set_status(p.status, USP_ERR_BAD_SEQLENS);
    return false;
  }
  if (blockIdx.x == 0) {
    for (int d = threadIdx.x; d < n; d += blockDim.x)
      if (gld(p.cu + d + 1) <= gld(p.cu + d)) set_status(p.status, USP_ERR_BAD_SEQLENS);
  }
  return true;
}

// doc_bounds of a token of the tile.
template <class M>
__device__ __forceinline__ void doc_bounds(const AttnArgs& p, const M& m, const TileDocs& w, int t, int& a, int& b,
                                           int& pe) {
  a = w.a0;
  b = w.b0;
  pe = w.pe0;
  if (t >= w.a1) {
    a = w.a1;
    b = w.b1;
    pe = w.pe1;
  } else if (t >= w.b0) {  // a document inside the tile
    int lo = w.d0 + 1, hi = w.d1;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (gld(p.cu + mid) <= t) lo = mid; else hi = mid;
    }
    a = max(0, min(gld(p.cu + lo), t));
    b = min(p.BS, max(gld(p.cu + lo + 1), t + 1));
    pe = prefix_end(m, lo, a, b, p.status);
  }
}

// key_range / query_range of the tile.
template <class M>
__device__ __forceinline__ void key_range(const AttnArgs& p, const M&, const TileDocs& w, int first, int last, int& lo,
                                          int& hi) {
  lo = w.a0;
  hi = p.causal ? max(last + 1, w.pe1) : w.b1;
  if (p.window_left >= 0) {
    lo = max(lo, first - p.window_left);
    if (!p.causal) hi = min(hi, last + p.window_left + 1);
  }
}
template <class M>
__device__ __forceinline__ void query_range(const AttnArgs& p, const M&, const TileDocs& w, int first, int last,
                                            int& lo, int& hi) {
  lo = !p.causal || first < w.pe0 ? w.a0 : first;
  hi = w.b1;
  if (p.window_left >= 0) {
    hi = min(hi, last + p.window_left + 1);
    if (!p.causal) lo = max(lo, first - p.window_left);
  }
}

// What a block of scores still has to go through: x2 = x * sc + off.
struct Affine {
  float sc, off;
};

// Adds the biases to N raw scores of one row: column c is the key at distance
// d0 - c.  [dmin, dmax] are the distances that the whole warp meets in the block
// (warp-uniform).  `row` points at distance 0 of the head's table (null: none).
// Distances all beyond R cost nothing per element: their bias is one value and
// goes into `off`.  `later_hidden`: keys after the query are masked anyway, so
// their slope may have either sign.  `ramp`: slope2 * c for every column in shared
// memory, or null (computed here).  A slope's part is split at the block's first column,
// -slope d0 + slope c, so it is rounded at the size of slope d0: for slopes >= 0 far keys, which
// have no weight, carry that; for slopes below 0 the keys that have the weight do.
template <int N>
__device__ __forceinline__ Affine add_bias(float (&x)[N], const float* row, int R, float slope2, const float* ramp,
                                           int d0, int dmin, int dmax, bool later_hidden, float scale_log2) {
  Affine f{scale_log2, 0.f};
  if (row != nullptr) {
    if (dmin >= R || dmax <= -R) {
      f.off = row[dmin >= R ? R : -R];
    } else {
      const float* at = row + d0;
#pragma unroll
      for (int c = 0; c < N; ++c) x[c] = fmaf(x[c], f.sc, at[-c]);
      f.sc = 1.f;
    }
  }
  if (slope2 != 0.f) {
    const float d0f = static_cast<float>(d0);
    if (dmin >= 0 || later_hidden) {
      // -slope (d0 - c) = -slope d0 + slope c
      const uint64_t sc2 = f2_pack(f.sc, f.sc), k2 = f2_pack(slope2, slope2);
#pragma unroll
      for (int c = 0; c < N; c += 4) {
        uint64_t a2, b2;
        if (ramp != nullptr) {
          const float4 r4 = *reinterpret_cast<const float4*>(ramp + c);
          a2 = f2_pack(r4.x, r4.y);
          b2 = f2_pack(r4.z, r4.w);
        } else {
          a2 = f2_mul(f2_pack(static_cast<float>(c), static_cast<float>(c + 1)), k2);
          b2 = f2_mul(f2_pack(static_cast<float>(c + 2), static_cast<float>(c + 3)), k2);
        }
        const float2 y = f2_unpack(f2_fma(f2_pack(x[c], x[c + 1]), sc2, a2));
        const float2 z = f2_unpack(f2_fma(f2_pack(x[c + 2], x[c + 3]), sc2, b2));
        x[c] = y.x;
        x[c + 1] = y.y;
        x[c + 2] = z.x;
        x[c + 3] = z.y;
      }
      f.off -= slope2 * d0f;
    } else {
#pragma unroll
      for (int c = 0; c < N; ++c) x[c] = fmaf(x[c], f.sc, -slope2 * fabsf(d0f - static_cast<float>(c)));
    }
    f.sc = 1.f;
  }
  return f;
}

// The dK/dV pass reads a row's -LSE log2e for 32 queries at a time, the same for
// every key: without a cap (which takes the biased score) a row's part of the
// slope's bias goes there, slope2 (t & 31), so that a key adds one value per block
// of 32 queries (which start at multiples of 32).  Within 32 queries the values stay
// small enough for fp32 not to lose the LSE.
template <class M>
__device__ __forceinline__ float slope_of_row(const M& m, float slope2, int t) {
  if constexpr (bias_on<M>) {
    if constexpr (!cap_on<M>) return slope2 * static_cast<float>(t & 31);
  }
  return 0.f;
}

// The biases of 32 raw scores of one key: column c is the query at distance d0 + c;
// `in_stats`: its -slope2 c comes with its statistics (above).  As add_bias otherwise.
__device__ __forceinline__ Affine add_bias_of_key(float (&x)[32], const float* row, int R, float slope2, bool in_stats,
                                                  int d0, int dmin, int dmax, bool later_hidden, float scale_log2) {
  Affine f{scale_log2, 0.f};
  if (row != nullptr) {
    if (dmin >= R || dmax <= -R) {
      f.off = row[dmin >= R ? R : -R];
    } else {
      const float* at = row + d0;
#pragma unroll
      for (int c = 0; c < 32; ++c) x[c] = fmaf(x[c], f.sc, at[c]);
      f.sc = 1.f;
    }
  }
  if (slope2 != 0.f) {
    const float d0f = static_cast<float>(d0);
    if (in_stats) {
      f.off -= slope2 * d0f;  // -slope (d0 + c) = -slope d0 - slope c
      if (dmin < 0 && !later_hidden) {
        // queries before the key: -slope |d| = -slope d + 2 slope min(d, 0)
#pragma unroll
        for (int c = 0; c < 32; ++c)
          x[c] = fmaf(x[c], f.sc, 2.f * slope2 * fminf(d0f + static_cast<float>(c), 0.f));
        f.sc = 1.f;
      }
    } else {
#pragma unroll
      for (int c = 0; c < 32; ++c) x[c] = fmaf(x[c], f.sc, -slope2 * fabsf(d0f + static_cast<float>(c)));
      f.sc = 1.f;
    }
  }
  return f;
}

// tanh(y) / y as a polynomial q in t = y^2 (own fits by interpolation at Chebyshev
// nodes): degree 2 for |y| <= 1/4, 4 for |y| <= 1/2, 6 for |y| <= 1.  The absolute
// error of y q(y^2) evaluated in fp32 is at most 1.2e-7 in each range; c times that
// is below what fp32 leaves of a score of that size, which the fp32 gradients of
// rel_bias and the sinks need.  (One exponential and a reciprocal per score, tanh =
// 1 - 2 / (1 + e^(2y)), costs an absolute 2e-7 at y = 0 already.)
template <int DEG>
__host__ __device__ constexpr float tanh_q(int i) {
  static_assert(DEG == 2 || DEG == 4 || DEG == 6, "");
  if (DEG == 2) return i == 0 ? 0.999999583f : i == 1 ? -0.333218962f : 0.128414333f;
  if (DEG == 4)
    return i == 0   ? 1.f
           : i == 1 ? -0.333330691f
           : i == 2 ? 0.13324751f
           : i == 3 ? -0.0529842377f
                    : 0.0171313453f;
  return i == 0   ? 0.99999994f
         : i == 1 ? -0.333328277f
         : i == 2 ? 0.133250758f
         : i == 3 ? -0.0534516461f
         : i == 4 ? 0.0202797074f
         : i == 5 ? -0.0061943247f
                  : 0.00103802513f;
}

// tanh of any y: the polynomial inside |y| <= 1, outside 1 - 2 e / (1 + e) with
// e = e^(-2|y|) <= 0.14, whose absolute error is under 1e-7.  Keeps NaN.
__device__ __forceinline__ float tanh_any(float y) {
  const float t = y * y;
  float q = tanh_q<6>(6);
#pragma unroll
  for (int i = 5; i >= 0; --i) q = fmaf(q, t, tanh_q<6>(i));
  const float e = ex2(-2.f * kLog2E * fabsf(y));
  const float big = fmaf(-2.f * e, rcp(1.f + e), 1.f);
  return fabsf(y) <= 1.f ? y * q : copysignf(big, y);
}

// x -> tanh(k x) for scores of which some lie beyond the cap.  Rare, and unrolled
// over a block several times the size of the code that does run, so a loop over the
// block: through TMEM, whose columns [tmem, tmem + N) are this warp's to write.
template <int N>
__device__ __forceinline__ void tanh_rare(float (&x)[N], float k, uint32_t tmem) {
#pragma unroll
  for (int c = 0; c < N; c += 32) {
    uint32_t v[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(x[c + e]);
    tmem_st32(tmem + c, v);
  }
  tmem_wait_st();
#pragma unroll 1
  for (int c = 0; c < N; c += 4) {
    uint32_t v[4];
    tmem_ld4(tmem + c, v);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __float_as_uint(tanh_any(__uint_as_float(v[e]) * k));
    tmem_st4(tmem + c, v);
    tmem_wait_st();
  }
#pragma unroll
  for (int c = 0; c < N; c += 32) {
    uint32_t v[32];
    tmem_ld32(tmem + c, v);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) x[c + e] = __uint_as_float(v[e]);
  }
}

// x -> tanh(k x) / k by the polynomial of degree DEG in (k x)^2: the powers of k
// go into its coefficients, so k costs no multiplication per score.
template <int DEG, int N>
__device__ __forceinline__ void tanh_poly(float (&x)[N], float k) {
  uint64_t q2[DEG + 1];
  float kp = 1.f;
#pragma unroll
  for (int i = 0; i <= DEG; ++i) {
    q2[i] = f2_pack(tanh_q<DEG>(i) * kp, tanh_q<DEG>(i) * kp);
    kp *= k * k;
  }
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const uint64_t y = f2_pack(x[c], x[c + 1]), t = f2_mul(y, y);
    uint64_t q = f2_fma(q2[DEG], t, q2[DEG - 1]);
#pragma unroll
    for (int i = DEG - 2; i >= 0; --i) q = f2_fma(q, t, q2[i]);
    const float2 z = f2_unpack(f2_mul(y, q));
    x[c] = z.x;
    x[c + 1] = z.y;
  }
}

// x -> w = tanh(y) / k in place, y = x2 ln2 / cap, x2 = x f.sc + f.off, and returns
// k: the capped score in the log2 domain is then w k cap log2e, and tanh is w k.
// SHORT (the forward): a warp takes the shortest polynomial that its largest |y|
// allows.  Causal rows of 4096, 8192 tokens, 32 heads of 128, scores' deviation / the
// cap of 0.06, 0.1, 0.15, 0.5: 294, 316, 341, 563 us, and 322, 322, 322, 568 with
// degree 6 alone; the same order at D = 64 and in windows.  (0.5 and more: every
// block has scores beyond the cap, tanh_rare.)  The backward takes degree 6 alone.
// `tmem`: N columns of this warp's lanes, free to write.
template <bool SHORT, int N>
__device__ __forceinline__ float cap_scores(float (&x)[N], Affine f, float cap, bool biased, uint32_t tmem) {
  float k = fminf(f.sc * (0.6931471805599453f / cap), FLT_MAX);
  if (!SHORT || biased || k < 0x1p-9f || k > 0x1p9f) {
    // to y itself: the offset of a bias, or a k whose powers (up to k^12) would leave fp32
    const float ko = f.off * (0.6931471805599453f / cap);
    const uint64_t k2 = f2_pack(k, k), o2 = f2_pack(ko, ko);
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const float2 y = f2_unpack(f2_fma(f2_pack(x[c], x[c + 1]), k2, o2));
      x[c] = y.x;
      x[c + 1] = y.y;
    }
    k = 1.f;
  }
  float top4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < N; c += 2) top4[(c >> 1) & 3] = fmax3(top4[(c >> 1) & 3], fabsf(x[c]), fabsf(x[c + 1]));
  // (the max skips a NaN, which every path keeps)
  const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3])) * k;
  if (SHORT && !__any_sync(0xffffffffu, top > 0.25f)) {
    tanh_poly<2>(x, k);
  } else if (SHORT && !__any_sync(0xffffffffu, top > 0.5f)) {
    tanh_poly<4>(x, k);
  } else if (!__any_sync(0xffffffffu, top > 1.f)) {
    tanh_poly<6>(x, k);
  } else {
    tanh_rare(x, k, tmem);
    k = 1.f;
  }
  return k;
}

// g = 1 - tanh^2, the cap's derivative, from the tanh.
template <int N>
__device__ __forceinline__ void cap_slope(const float (&th)[N], float (&g)[N]) {
  const uint64_t minus = f2_pack(-1.f, -1.f), one = f2_pack(1.f, 1.f);
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const uint64_t y = f2_pack(th[c], th[c + 1]);
    const float2 z = f2_unpack(f2_fma(f2_mul(y, minus), y, one));
    g[c] = z.x;
    g[c + 1] = z.y;
  }
}

// p *= g
template <int N>
__device__ __forceinline__ void f2_scale(float (&p)[N], const float (&g)[N]) {
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const float2 z = f2_unpack(f2_mul(f2_pack(p[c], p[c + 1]), f2_pack(g[c], g[c + 1])));
    p[c] = z.x;
    p[c + 1] = z.y;
  }
}

// A capped score lies in [-c2, c2].  Up to this c2 the softmax's reference does not
// follow the running maximum past a row's first keys, as long as it lies no more
// than this below c2: 2^(z2 - reference) and sums of up to 2^31 of them stay in fp32
// (and bf16, which has its range), with room for O's products.
constexpr float kFixedRefCap2 = 80.f;

}  // namespace usp
