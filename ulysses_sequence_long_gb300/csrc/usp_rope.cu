// usp_rope.cu — rotary positions of several axes, q and k in one pass: a pair
// (x1, x2) of a head turns by w = position[axis] * freq.
//
// The pass is bound by HBM (2 bytes in and 2 out per element), so cos and sin have
// to be cheap: they are the same for every head of a token, and a warp makes each
// of a token's values once for all the rows it turns.
//
// The angle in turns is position * (freq / 2 pi), of which only the fraction counts.
// freq / 2 pi is held as a 64-bit fraction F of a turn (an fp32 mantissa times 1 / 2 pi
// to 64 bits, by integers); position * F modulo 2^64 then drops the whole turns exactly,
// where an fp32 product has no digits behind the point left for far positions.
//
// Measured (one GB300, several states in turn, larger than L2 together): 32768 tokens, 32 + 8 heads, D 128, forward and
// backward 197 us (6.8 TB/s); 3000 tokens, 12 + 12 heads, D 64, half of each head turned: 5.2 us a pass (floor 2.8; 3.5
// where L2 has them); one token of four sequences: 2.3 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "usp_internal.h"
#include "usp_ptx.cuh"

namespace usp {
namespace rope {

constexpr int kWarps = 4;
constexpr int kUnroll = 4;                                   // rows in flight per group of lanes
constexpr unsigned long long kTurn = 0x28BE60DB9391054Aull;  // 2^64 / (2 pi)
constexpr float kMaxFreq = 1024.f;

struct Geom {
  int tokens, Hq, H, n_axes, n_pos, n_pairs;  // H = Hq + Hkv
  int slices;                                 // items of a token: its heads in groups of rows
  uint32_t items;
  const int32_t* pos;
  const float* freqs;
  const int32_t* axes;
};

// freq / (2 pi) modulo 1 as a 64-bit fraction; |freq| <= 1024.
__device__ __forceinline__ unsigned long long turn_fraction(float f) {
  const uint32_t u = __float_as_uint(f);
  const int e = static_cast<int>((u >> 23) & 255);
  const unsigned long long m = e ? (u & 0x7FFFFFu) | 0x800000u : u & 0x7FFFFFu;  // |f| = m 2^(max(e, 1) - 150)
  const int s = 150 - max(e, 1);                                                  // 13 <= s <= 149
  const unsigned long long lo = m * kTurn, hi = __umul64hi(m, kTurn);
  // (hi : lo) >> s, rounded
  unsigned long long r;
  if (s < 64)
    r = ((hi << (64 - s)) | (lo >> s)) + ((lo >> (s - 1)) & 1);
  else if (s < 128)
    r = s == 64 ? hi + (lo >> 63) : (hi >> (s - 64)) + ((hi >> (s - 65)) & 1);
  else
    r = 0;
  return u >> 31 ? 0ull - r : r;
}

// A row is one head's D elements, turned by D/16 lanes of 16 elements each: the lanes below n_pairs/8 hold
// eight pairs (in two 16-byte vectors), the others elements that pass through.
template <int D, bool kInterleaved, bool kBack>
__global__ void __launch_bounds__(32 * kWarps) rope_kernel(Geom g, const uint4* q, const uint4* k, uint4* q_out,
                                                           uint4* k_out, int32_t* status) {
  constexpr int LPR = D / 16, RPW = 32 / LPR, PPL = 8 / RPW;  // lanes per row, rows at once, pairs a lane prepares
  __shared__ __align__(16) float2 turns[kWarps][LPR * 8];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, t = lane % LPR, rg = lane / LPR;
  const int rot_lanes = g.n_pairs / 8;
  const bool rot = t < rot_lanes;
  // the lane's two vectors within a row: neighbouring lanes have neighbouring ones (half a row's vectors apart, so that a
  // pair's two elements meet, and pairs of neighbours do anyway)
  const int va = rot ? t : rot_lanes + t, vb = rot ? t + rot_lanes : LPR + t;
  grid_wait();
  // the pairs whose angles this lane prepares: rg * PPL .. of its row position t
  unsigned long long frac[PPL];
  int axis[PPL];
#pragma unroll
  for (int i = 0; i < PPL; ++i) {
    frac[i] = 0;
    axis[i] = 0;
    if (rot) {
      const int p = t * 8 + rg * PPL + i;
      const float f = gld(g.freqs + p);
      axis[i] = g.axes != nullptr ? gld(g.axes + p) : 0;
      if (!(fabsf(f) <= kMaxFreq) || axis[i] < 0 || axis[i] >= g.n_axes) {
        set_status(status, USP_ERR_BAD_ROPE);
        axis[i] = 0;
      } else {
        frac[i] = turn_fraction(f);
      }
    }
  }
  for (uint32_t item = blockIdx.x * kWarps + w; item < g.items; item += gridDim.x * kWarps) {
    const uint32_t tok = item / g.slices;
    const int h0 = static_cast<int>(item - tok * g.slices) * (RPW * kUnroll) + rg;
    const uint32_t at = tok % static_cast<uint32_t>(g.n_pos);
    int32_t pos[PPL];
#pragma unroll
    for (int i = 0; i < PPL; ++i) pos[i] = gld(g.pos + static_cast<size_t>(axis[i]) * g.n_pos + at);
    uint4 a[kUnroll], b[kUnroll];
    size_t row[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * RPW;
      const bool is_q = h < g.Hq;
      row[u] = (is_q ? static_cast<size_t>(tok) * g.Hq + h : static_cast<size_t>(tok) * (g.H - g.Hq) + (h - g.Hq)) *
               (D / 8);
      if (h < g.H) {
        const uint4* src = (is_q ? q : k) + row[u];
        a[u] = gld(src + va);
        b[u] = gld(src + vb);
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PPL; ++i) {
      const unsigned long long turn = static_cast<unsigned long long>(static_cast<long long>(pos[i])) * frac[i];
      // the fraction of a turn, -1/2 .. 1/2, as half turns
      const float half = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
      float s, c;
      sincospif(half, &s, &c);
      turns[w][t * 8 + rg * PPL + i] = make_float2(c, kBack ? -s : s);
    }
    __syncwarp();
    float2 cs[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = kInterleaved ? 4 * (i < 2 ? va : vb) + 2 * (i & 1) : 8 * t + 2 * i;
      const float4 x = *reinterpret_cast<const float4*>(&turns[w][p]);
      cs[2 * i] = make_float2(x.x, x.y);
      cs[2 * i + 1] = make_float2(x.z, x.w);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * RPW;
      if (h >= g.H) continue;
      if (rot) {
        uint32_t xa[4] = {a[u].x, a[u].y, a[u].z, a[u].w}, xb[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (kInterleaved) {  // a pair is a word
            const float a1 = bf16lo(xa[e]), a2 = bf16hi(xa[e]), b1 = bf16lo(xb[e]), b2 = bf16hi(xb[e]);
            const float2 ca = cs[e], cb = cs[4 + e];
            xa[e] = pack_bf16x2(a1 * ca.x - a2 * ca.y, a1 * ca.y + a2 * ca.x);
            xb[e] = pack_bf16x2(b1 * cb.x - b2 * cb.y, b1 * cb.y + b2 * cb.x);
          } else {
            const float a1 = bf16lo(xa[e]), b1 = bf16hi(xa[e]), a2 = bf16lo(xb[e]), b2 = bf16hi(xb[e]);
            const float2 ca = cs[2 * e], cb = cs[2 * e + 1];
            xa[e] = pack_bf16x2(a1 * ca.x - a2 * ca.y, b1 * cb.x - b2 * cb.y);
            xb[e] = pack_bf16x2(a1 * ca.y + a2 * ca.x, b1 * cb.y + b2 * cb.x);
          }
        }
        a[u] = make_uint4(xa[0], xa[1], xa[2], xa[3]);
        b[u] = make_uint4(xb[0], xb[1], xb[2], xb[3]);
      }
      uint4* dst = (h < g.Hq ? q_out : k_out) + row[u];
      dst[va] = a[u];
      dst[vb] = b[u];
    }
  }
}

template <int D>
int launch(const Geom& g, const void* q, const void* k, void* q_out, void* k_out, bool interleaved, bool back,
           int32_t* status, cudaStream_t st) {
  // (64 CTAs per SM in turn: 198 us for the 32768 tokens above; 16 of them 211, 32 201, one per item 212)
  const int ctas = static_cast<int>(std::min<int64_t>((static_cast<int64_t>(g.items) + kWarps - 1) / kWarps,
                                                      static_cast<int64_t>(device_sm_count()) * 64));
  auto* kern = interleaved ? (back ? rope_kernel<D, true, true> : rope_kernel<D, true, false>)
                           : (back ? rope_kernel<D, false, true> : rope_kernel<D, false, false>);
  return launch_chained(kern, dim3(ctas), 32 * kWarps, 0, 1, st, g, static_cast<const uint4*>(q),
                        static_cast<const uint4*>(k), static_cast<uint4*>(q_out), static_cast<uint4*>(k_out), status);
}

}  // namespace rope

int launch_rope(const usp_rope_params& p, const void* q, const void* k, void* q_out, void* k_out, bool back,
                int32_t* status, cudaStream_t st) {
  rope::Geom g{};
  g.tokens = p.tokens;
  g.Hq = p.Hq;
  g.H = p.Hq + p.Hkv;
  g.n_axes = p.n_axes;
  g.n_pos = p.n_pos;
  g.n_pairs = p.n_pairs;
  g.pos = p.positions;
  g.freqs = p.freqs;
  g.axes = p.axes;
  const int rows = 32 / (p.D / 16) * rope::kUnroll;
  g.slices = (g.H + rows - 1) / rows;
  g.items = static_cast<uint32_t>(p.tokens) * static_cast<uint32_t>(g.slices);
  return p.D == 64 ? rope::launch<64>(g, q, k, q_out, k_out, p.interleaved != 0, back, status, st)
                   : rope::launch<128>(g, q, k, q_out, k_out, p.interleaved != 0, back, status, st);
}

}  // namespace usp
