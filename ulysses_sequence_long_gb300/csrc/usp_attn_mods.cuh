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
  static constexpr bool cap_on = CAP;
  static constexpr bool bias_on = BIAS;
};

template <class M>
constexpr bool bias_on = false;
template <bool CAP, bool BIAS>
constexpr bool bias_on<Mods<CAP, BIAS>> = BIAS;

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
  const int b = __ldg(m.buckets + i);
  if (b < 0 || b >= m.n_buckets) set_status(status, USP_ERR_BAD_MODS);
  return min(max(b, 0), m.n_buckets - 1);
}

// Entry e (of tab_len(R)) of head h's row by distance, in the log2 domain.
__device__ __forceinline__ float table_entry(const ModArgs& m, int h, int e, int32_t* status) {
  const int d = min(max(e - (m.R + kTabPad), -m.R), m.R);
  return __ldg(m.rel_bias + static_cast<size_t>(h) * m.n_buckets + checked_bucket(m, d + m.R, status)) * kLog2E;
}

// One past the last prefix token of document d = [a, b).
__device__ __forceinline__ int prefix_end(const ModArgs& m, int d, int a, int b, int32_t* status) {
  if (m.prefix == nullptr) return a;
  if (d >= m.n_prefix) {
    set_status(status, USP_ERR_BAD_MODS);
    return a;
  }
  const int len = __ldg(m.prefix + d);
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
  a = max(0, min(__ldg(p.cu + d), t));
  b = min(p.BS, max(__ldg(p.cu + d + 1), t + 1));
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

// What a block of scores still has to go through: x2 = x * sc + off.
struct Affine {
  float sc, off;
};

// Adds the biases to N raw scores of one row (STEP = -1: column c is the key
// at distance d0 - c) or one key (STEP = +1: column c is the query at distance
// d0 + c), d0 = t - u of column 0.  [dmin, dmax] are the distances that the
// whole warp meets in the block (warp-uniform).  `row` points at distance 0 of
// the head's table (null: none).  Distances all beyond R cost nothing per
// element: their bias is one value and goes into `off`.
template <int N, int STEP>
__device__ __forceinline__ Affine add_bias(float (&x)[N], const float* row, int R, float slope2, int d0, int dmin,
                                           int dmax, float scale_log2) {
  Affine f{scale_log2, 0.f};
  if (row != nullptr) {
    if (dmin >= R || dmax <= -R) {
      f.off = row[dmin >= R ? R : -R];
    } else {
      const float* at = row + d0;
#pragma unroll
      for (int c = 0; c < N; ++c) x[c] = fmaf(x[c], f.sc, at[STEP * c]);
      f.sc = 1.f;
    }
  }
  if (slope2 != 0.f) {
    const float d0f = static_cast<float>(d0);
    if (dmin >= 0 || dmax <= 0) {
      // one side of the diagonal: -slope |d0 + STEP c| = -slope |d0| + k c
      const float k = dmin >= 0 ? -STEP * slope2 : STEP * slope2;
      const uint64_t sc2 = f2_pack(f.sc, f.sc), k2 = f2_pack(k, k);
#pragma unroll
      for (int c = 0; c < N; c += 2) {
        const float2 y = f2_unpack(f2_fma(f2_pack(x[c], x[c + 1]), sc2,
                                          f2_mul(f2_pack(static_cast<float>(c), static_cast<float>(c + 1)), k2)));
        x[c] = y.x;
        x[c + 1] = y.y;
      }
      f.off -= slope2 * fabsf(d0f);
    } else {
#pragma unroll
      for (int c = 0; c < N; ++c) x[c] = fmaf(x[c], f.sc, -slope2 * fabsf(d0f + static_cast<float>(STEP * c)));
    }
    f.sc = 1.f;
  }
  return f;
}

// tanh(y) / y on |y| <= 1 as a polynomial in t = y^2, degree 6, fitted by
// interpolation at Chebyshev nodes: the absolute error of y q(y^2) evaluated in
// fp32 is at most 1.3e-7 (the fit's own is 3.7e-8).  An absolute error of c
// times that in the score is below what fp32 leaves of a score of that size,
// which the fp32 gradients of rel_bias and the sinks need.  (One exponential and a
// reciprocal per score, tanh = 1 - 2 / (1 + e^(2y)), costs an absolute 2e-7 at
// y = 0 already.)
__host__ __device__ constexpr float tanh_q(int i) {
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
  float q = tanh_q(6);
#pragma unroll
  for (int i = 5; i >= 0; --i) q = fmaf(q, t, tanh_q(i));
  const float e = ex2(-2.f * kLog2E * fabsf(y));
  const float big = fmaf(-2.f * e, rcp(1.f + e), 1.f);
  return fabsf(y) <= 1.f ? y * q : copysignf(big, y);
}

// x -> tanh(x2 ln2 / cap) in place, where x2 = x f.sc + f.off: the capped score
// is then cap log2e times that.  The warp takes the polynomial alone, two scores
// per instruction, unless one of its scores is beyond |y| = 1.
template <int N>
__device__ __forceinline__ void cap_scores(float (&x)[N], Affine f, float cap) {
  const float k = 0.6931471805599453f / cap;
  const uint64_t k2 = f2_pack(f.sc * k, f.sc * k), o2 = f2_pack(f.off * k, f.off * k);
  float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const float2 y = f2_unpack(f2_fma(f2_pack(x[c], x[c + 1]), k2, o2));
    x[c] = y.x;
    x[c + 1] = y.y;
    top[(c >> 1) & 3] = fmax3(top[(c >> 1) & 3], fabsf(y.x), fabsf(y.y));
  }
  // (the max skips a NaN, which the polynomial keeps)
  if (!__any_sync(0xffffffffu, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) > 1.f)) {
    uint64_t q2[7];
#pragma unroll
    for (int i = 0; i < 7; ++i) q2[i] = f2_pack(tanh_q(i), tanh_q(i));
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const uint64_t y = f2_pack(x[c], x[c + 1]), t = f2_mul(y, y);
      uint64_t q = f2_fma(q2[6], t, q2[5]);
#pragma unroll
      for (int i = 4; i >= 0; --i) q = f2_fma(q, t, q2[i]);
      const float2 z = f2_unpack(f2_mul(y, q));
      x[c] = z.x;
      x[c + 1] = z.y;
    }
  } else {
#pragma unroll
    for (int c = 0; c < N; ++c) x[c] = tanh_any(x[c]);
  }
}

// g = 1 - tanh^2, the cap's derivative, from the tanh.
template <int N>
__device__ __forceinline__ void cap_slope(const float (&th)[N], float (&g)[N]) {
#pragma unroll
  for (int c = 0; c < N; c += 2) {
    const uint64_t y = f2_pack(th[c], th[c + 1]);
    const float2 z = f2_unpack(f2_fma(f2_mul(y, f2_pack(-1.f, -1.f)), y, f2_pack(1.f, 1.f)));
    g[c] = z.x;
    g[c + 1] = z.y;
  }
}

// A capped score lies in [-c2, c2].  Up to this c2 the softmax takes a fixed
// reference instead of a running maximum: 2^z2 and sums of up to 2^31 of them
// stay in fp32 (and bf16, which has its range), with room for O's products.
constexpr float kFixedRefCap2 = 80.f;

}  // namespace usp
