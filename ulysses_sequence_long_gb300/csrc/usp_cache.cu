// usp_cache.cu — tokens into the pages of a key/value cache and out of them: a copy
// for bf16, for e4m3 a power of two per token and head found on the way.
//
// Both directions are bound by HBM: 2 bytes of each element on the token side, 2 or 1 on
// the pages' side.  One group of D/16 lanes has one token's head, keys and values
// together (64 bytes a lane in flight); the token's place (its sequence, its position, its page:
// a chain of dependent loads) is looked up while the rows are on their way.
// A power of two as the scale: x / 2^e and its way back are exact, so the one rounding
// is that to e4m3, and the attention moves the scale from the elements to the scores.
//
// Measured (one GB300, several states in turn, larger than L2 together): 31153 tokens of 8 heads, D 128, into e4m3 pages
// 30.1 us (floor at 6.69 TB/s 28.7); 25478 of them back 26.2 us (23.5); 7400 tokens of 8 heads, D 64, bf16 6.6 us (4.5); one
// token of 64 sequences 1.8 us.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "usp_internal.h"
#include "usp_paged.cuh"
#include "usp_ptx.cuh"

namespace usp {
namespace cache {

constexpr int kWarps = 4;

struct Geom {
  paged::Pool pool;
  int tokens;
  uint32_t chunks;         // groups of 32 / (D/16) tokens
  uint32_t items;          // P * chunks * hk
  FastDiv by_hk, by_chunks;
  const int32_t* cu;       // nullptr: token i is sequence i's last
};

// The row of token i's head j of rank r in the pages; < 0: none.
__device__ __forceinline__ int64_t page_row(const Geom& g, int i, int r, int j, int32_t* status) {
  int seq, pos;
  bool bad = false;
  int64_t row = -1;
  if (g.pool.place(g.cu, i, seq, pos, bad)) row = g.pool.row(seq, pos, r, j, bad);
  if (bad) set_status(status, USP_ERR_BAD_PAGES);
  return row;
}

// boundaries that go down, begin after token 0 or end behind the last one (each block of the grid's first ones looks at
// a part)
__device__ __forceinline__ void check_boundaries(const Geom& g, int32_t* status) {
  if (g.cu == nullptr || status == nullptr) return;
  for (int s = blockIdx.x * blockDim.x + threadIdx.x; s < g.pool.n_seqs; s += gridDim.x * blockDim.x) {
    const int a = gld(g.cu + s), b = gld(g.cu + s + 1);
    if ((s == 0 && a != 0) || b < a || b > g.tokens) set_status(status, USP_ERR_BAD_PAGES);
  }
}

// Exponent e of a row whose largest finite |x| is amax: the smallest e >= -126 with amax <= 448 2^e.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  return max(static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0), -126);  // 448 = 1.75 2^8
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return lo | static_cast<uint32_t>(hi) << 16;
}

// 16 elements of a row as e4m3, eight of each half of the row; the row's scale byte
template <int LPR>
__device__ __forceinline__ uint4 quantise(const uint4& x0, const uint4& x1, int& byte) {
  const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  float amax = 0.f;  // (fmaxf passes NaN over)
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16lo(w[i])), fabsf(bf16hi(w[i]))));
#pragma unroll
  for (int m = 1; m < LPR; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  const int e = scale_exponent(fminf(amax, __uint_as_float(0x7F7F0000u)));
  byte = e + 127;
  const float inv = pow2(-e);
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = e4m3x4(bf16lo(w[2 * i]) * inv, bf16hi(w[2 * i]) * inv, bf16lo(w[2 * i + 1]) * inv, bf16hi(w[2 * i + 1]) * inv);
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ void dequantise(const uint4& x, int byte, uint4& y0, uint4& y1) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  const float s = byte ? pow2(byte - 127) : 0x1p-127f;
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t two = paged::e4m3x2_to_f16x2(static_cast<uint16_t>(w[i] >> (16 * h)));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two));
      o[2 * i + h] = pack_bf16x2(f.x * s, f.y * s);
    }
  y0 = make_uint4(o[0], o[1], o[2], o[3]);
  y1 = make_uint4(o[4], o[5], o[6], o[7]);
}

// One warp: 32 / (D/16) consecutive tokens of one head, so that it writes consecutive rows of a page.  A lane has eight
// elements of each half of a row: what an instruction reads or writes lies side by side (two neighbouring pieces
// a lane would write half a 32-byte sector at a time).  Warps that looped over more tokens, with
// the next ones' look-ups under way, were slower (29 -> 37 us), as were two tokens at once (28 -> 30 us).
template <int D, bool kE4m3, bool kAppend>
__global__ void __launch_bounds__(32 * kWarps) cache_kernel(Geom g, uint4* k, uint4* v, int32_t* status) {
  constexpr int LPR = D / 16, TPW = 32 / LPR, V = D / 8;  // lanes a row, tokens a warp, vectors of a bf16 row
  const int lane = threadIdx.x & 31, t = lane % LPR;
  grid_wait();
  check_boundaries(g, status);
  const uint32_t item = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (item >= g.items) return;
  const uint32_t rc = g.by_hk.div(item), j = item - rc * g.pool.hk, r = g.by_chunks.div(rc), c = rc - r * g.chunks;
  const int i = static_cast<int>(c) * TPW + lane / LPR;
  const bool have = i < g.tokens;
  const int64_t tok = ((static_cast<int64_t>(r) * g.tokens + i) * g.pool.hk + j) * V + t;
  uint4 x[4] = {};
  if (kAppend && have) {
    if (k != nullptr) {
      x[0] = gld(k + tok);
      x[1] = gld(k + tok + LPR);
    }
    if (v != nullptr) {
      x[2] = gld(v + tok);
      x[3] = gld(v + tok + LPR);
    }
  }
  const int64_t row = have ? page_row(g, i, r, j, status) : -1;
  if constexpr (kE4m3) {
    uint2* kp = static_cast<uint2*>(g.pool.k) + row * V + t;
    uint2* vp = static_cast<uint2*>(g.pool.v) + row * V + t;
    if constexpr (kAppend) {
      int kb, vb;
      const uint4 kq = quantise<LPR>(x[0], x[1], kb), vq = quantise<LPR>(x[2], x[3], vb);
      if (row < 0) return;
      if (k != nullptr) {
        kp[0] = make_uint2(kq.x, kq.y);
        kp[LPR] = make_uint2(kq.z, kq.w);
        if (t == 0) g.pool.k_scales[row] = static_cast<uint8_t>(kb);
      }
      if (v != nullptr) {
        vp[0] = make_uint2(vq.x, vq.y);
        vp[LPR] = make_uint2(vq.z, vq.w);
        if (t == 1) g.pool.v_scales[row] = static_cast<uint8_t>(vb);
      }
    } else {
      if (row < 0) return;
      uint2 a[2] = {}, b[2] = {};
      int kb = 0, vb = 0;
      if (k != nullptr) {
        a[0] = gld(kp);
        a[1] = gld(kp + LPR);
        kb = gld(g.pool.k_scales + row);
      }
      if (v != nullptr) {
        b[0] = gld(vp);
        b[1] = gld(vp + LPR);
        vb = gld(g.pool.v_scales + row);
      }
      dequantise(make_uint4(a[0].x, a[0].y, a[1].x, a[1].y), kb, x[0], x[1]);
      dequantise(make_uint4(b[0].x, b[0].y, b[1].x, b[1].y), vb, x[2], x[3]);
    }
  } else {
    if (row < 0) return;
    uint4* kp = static_cast<uint4*>(g.pool.k) + row * V + t;
    uint4* vp = static_cast<uint4*>(g.pool.v) + row * V + t;
    if constexpr (kAppend) {
      if (k != nullptr) {
        kp[0] = x[0];
        kp[LPR] = x[1];
      }
      if (v != nullptr) {
        vp[0] = x[2];
        vp[LPR] = x[3];
      }
    } else {
      if (k != nullptr) {
        x[0] = gld(kp);
        x[1] = gld(kp + LPR);
      }
      if (v != nullptr) {
        x[2] = gld(vp);
        x[3] = gld(vp + LPR);
      }
    }
  }
  if constexpr (!kAppend) {
    if (k != nullptr) {
      __stcs(k + tok, x[0]);
      __stcs(k + tok + LPR, x[1]);
    }
    if (v != nullptr) {
      __stcs(v + tok, x[2]);
      __stcs(v + tok + LPR, x[3]);
    }
  }
}

}  // namespace cache

int launch_cache_move(const usp_paged_cache& c, void* k, void* v, int tokens, const int32_t* cu, bool append,
                      int32_t* status, cudaStream_t st) {
  cache::Geom g{};
  g.pool = paged::Pool(c);
  g.tokens = tokens;
  g.cu = cu;
  const int per_warp = 32 / (c.D / 16);
  g.chunks = static_cast<uint32_t>((static_cast<int64_t>(tokens) + per_warp - 1) / per_warp);
  g.items = static_cast<uint32_t>(c.P) * g.chunks * static_cast<uint32_t>(g.pool.hk);
  g.by_hk = FastDiv(static_cast<uint32_t>(g.pool.hk));
  g.by_chunks = FastDiv(g.chunks);
  const unsigned ctas = (g.items + cache::kWarps - 1) / cache::kWarps;
  void (*kern)(cache::Geom, uint4*, uint4*, int32_t*) = nullptr;
  const bool e = c.dtype == USP_CACHE_E4M3;
  if (c.D == 64)
    kern = append ? (e ? cache::cache_kernel<64, true, true> : cache::cache_kernel<64, false, true>)
                  : (e ? cache::cache_kernel<64, true, false> : cache::cache_kernel<64, false, false>);
  else
    kern = append ? (e ? cache::cache_kernel<128, true, true> : cache::cache_kernel<128, false, true>)
                  : (e ? cache::cache_kernel<128, true, false> : cache::cache_kernel<128, false, false>);
  return launch_chained(kern, dim3(ctas), 32 * cache::kWarps, 0, 1, st, g, static_cast<uint4*>(k),
                        static_cast<uint4*>(v), status);
}

}  // namespace usp
