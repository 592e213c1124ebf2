// usp_decode.cu — attention of one new token per sequence over a paged cache.
//
//   s_u = scale q.k_u,  O = sum_u exp(s_u - LSE) v_u,  LSE = ln(sum_u exp(s_u) + exp(sink))
//
// Bound by HBM: every visible token's key and value are read once and take part in 4 D flop
// for each of the G query heads of their group, G a few: far below the card's ratio.  So
// what counts is that loads never pause and that all SMs have the same share of them.
//
// Shares.  The work of all sequences is one line of tiles of 64 positions (of a sequence, a rank
// and a key/value head: a "unit"); each CTA takes an equal stretch of the line, found from the
// lengths on the device, whatever they are.  A unit that lies in one CTA is finished there.  One
// that several CTAs share leaves partial results (O, maximum, sum in fp32) which a second
// kernel joins in the order of the positions.
//
// Loads.  A warp has 16 positions of each tile.  The products are arranged so that the
// positions are the rows of the matrix instruction and the query heads its 8 columns
// (S^T = K q^T, O^T = V^T P^T): rows of 16 query heads would be half empty for groups up to 8.
// Sums over d may take d in any order, so a thread's operands are whole 16-byte pieces of its rows:
// each thread copies its own pieces into shared memory (cp.async, several tiles ahead)
// and takes them from there itself.  No barrier, no swizzle, no other thread's data; only the pairs of
// positions that V^T's operands want next to each other are interleaved, by byte permutations.  (Matrix
// instructions with operands from shared memory and results in tensor memory want 64 rows of queries; here there are
// G.)
//
// e4m3: an element is exactly an f16, so products run in f16; a token's scales are powers of two
// and act on its score (keys) and on its weight (values).  The running reference M is the maximum of
// log2 weight + value exponent, so that the weights of the products, 2^(s + e - M + 15), stay below 2^15 and
// lose nothing down to 2^-29 of the largest.  q is scaled by a power of two into f16's range.
// bf16: the weights are rounded to bf16 in two parts (high and the rest), 16 bits of them in all: one part alone would make the
// output's error 1.4 times that of its own rounding.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "usp_internal.h"
#include "usp_paged.cuh"
#include "usp_ptx.cuh"

namespace usp {
namespace decode {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
using paged::Cursor;
using paged::kTile;
static_assert(kTile == 16 * kWarps, "a warp has 16 positions of a tile");
constexpr int kHeads = 8;           // query heads of a unit (more of them in a group: more units)
constexpr int kMaxCtas = 1024;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// What fits into an SM's shared memory with the stages below (64 to 96 KB of loads in flight).
constexpr int ctas_per_sm(int row_bytes) { return row_bytes == 256 ? 2 : row_bytes == 128 ? 3 : 5; }

template <int D, bool kE4m3>
struct Cfg {
  static constexpr int kRow = D * (kE4m3 ? 1 : 2);               // bytes of a token's head
  static constexpr int kKPieces = kRow / 64;                     // 16-byte pieces of a K row per thread (4 threads a row)
  static constexpr int kVBytes = kRow / 8 >= 16 ? 16 : 8;        // a thread's piece of a V row (8 threads a row)
  static constexpr int kVPieces = kRow / 8 / kVBytes;
  static constexpr int kScaleBytes = kE4m3 ? 32 : 0;             // 16 tokens' key and value scales
  static constexpr int kStage = 2 * 16 * kRow + kScaleBytes;     // one warp's share of a tile
  static constexpr int kCtas = ctas_per_sm(kRow);
  static constexpr int kStages = kRow == 64 ? 4 : 3;
  static constexpr int kMerge = kWarps * kHeads * D * 4;         // the warps' O
  static constexpr int kSmem = kStages * kStage * kWarps + kMerge;
};

struct Args {
  paged::Pool pool;
  int n_seqs, P, hq, G, chunks, units;  // chunks of 8 heads in a group of G; units = P * hk * chunks per sequence
  int window;                           // -1: none
  float scale;                          // softmax scale
  const float* sinks;
  const uint16_t* q;
  uint16_t* o;
  float* lse;
  float* parts;                         // [2 * ctas][kHeads][D] then [2 * ctas][kHeads][2]
  float* stats;
  int32_t* desc;                        // [ctas][2]: the unit that begins in this CTA and ends in another (or -1), its parts
  int32_t* status;
};

__device__ __forceinline__ int tiles_of(const Args& a, int seq, bool& bad) {
  return paged::Span(a.pool, a.window, seq, bad).tiles();
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(ok ? 8 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ int lds1(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return static_cast<int>(v);
}

// c += A B, A 16 x 16 (rows g, g + 8; columns by the thread's place in its four), B 16 x 8
template <bool kF16>
__device__ __forceinline__ void mma(float c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (kF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the transposed 8 x 8 matrix of 16-bit values, a row in each four threads
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The matrix row pair mt of V^T that thread group g has: elements d, d + 1 with
// d = value_column(mt, g) (its 16-byte pieces, two elements a row pair).
template <int D, bool kE4m3>
__device__ __forceinline__ int value_column(int mt, int g) {
  if constexpr (!kE4m3) return 64 * (mt >> 2) + 8 * g + 2 * (mt & 3);
  return (D / 8) * g + 2 * mt;
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads, Cfg<D, kE4m3>::kCtas) decode_kernel(Args a) {
  using C = Cfg<D, kE4m3>;
  constexpr int MT = D / 16, KS = D / 16;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long scan[kWarps];
  __shared__ int at_seq;
  __shared__ long long at_rest;
  __shared__ float wm[kWarps][kHeads], wl[kWarps][kHeads];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, qd = lane & 3;
  grid_wait();

  // ---- the CTA's stretch of the line
  const int per = (a.n_seqs + kThreads - 1) / kThreads, s0 = tid * per, s1 = min(a.n_seqs, s0 + per);
  long long mine = 0;
  bool bad = false;
  for (int s = s0; s < s1; ++s) mine += tiles_of(a, s, bad);
  if (bad) set_status(a.status, USP_ERR_BAD_PAGES);
  long long before = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += x;
  }
  if (lane == 31) scan[w] = before;
  __syncthreads();
  long long all = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < w) before += scan[i];
    all += scan[i];
  }
  before = (before - mine) * a.units;
  const long long W = all * a.units;
  const long long n_ctas = min(static_cast<long long>(gridDim.x), W);
  const int cta = blockIdx.x;
  if (tid == 0) {
    a.desc[2 * cta] = -1;
    a.desc[2 * cta + 1] = 0;
  }
  // sequences without a visible token have no tile: their outputs are written here
  for (int s = cta; s < a.n_seqs; s += gridDim.x)
    if (tiles_of(a, s, bad) == 0) {
      for (int i = tid; i < a.P * a.hq; i += kThreads) {
        const int r = i / a.hq, h = i - r * a.hq;
        a.lse[(static_cast<int64_t>(r) * a.n_seqs + s) * a.hq + h] = a.sinks ? gld(a.sinks + r * a.hq + h) : -INFINITY;
      }
      for (int i = tid; i < a.P * a.hq * (D / 8); i += kThreads) {
        const int r = i / (a.hq * (D / 8)), x = i - r * (a.hq * (D / 8));
        reinterpret_cast<uint4*>(a.o)[(static_cast<int64_t>(r) * a.n_seqs + s) * a.hq * (D / 8) + x] = make_uint4(0, 0, 0, 0);
      }
    }
  if (cta >= n_ctas) return;
  const long long begin = paged::stretch(W, n_ctas, cta), finish = paged::stretch(W, n_ctas, cta + 1);
  if (begin >= before && begin < before + mine * a.units) {
    long long rest = begin - before;
    int s = s0;
    for (;; ++s) {
      const long long n = static_cast<long long>(tiles_of(a, s, bad)) * a.units;
      if (rest < n) break;
      rest -= n;
    }
    at_seq = s;
    at_rest = rest;
  }
  __syncthreads();
  Cursor cur;
  cur.seek(a.pool, a.window, at_seq, at_rest, bad);
  const int count = static_cast<int>(finish - begin);
  const int start_tile = cur.tile, start_first = cur.first;

  // ---- loads, kStages - 1 tiles ahead
  const uint32_t ring = smem_u32(smem) + w * (C::kStages * C::kStage);
  float* merge = reinterpret_cast<float*>(smem + C::kStages * C::kStage * kWarps);
  Cursor ld = cur;
  int left = count;     // tiles not asked for yet
  int page = 0;         // of the tile at ld
  auto find_page = [&]() {
    const int t0 = ld.tile * kTile + 16 * w;
    page = 0;
    if (left > 0 && t0 < ld.len && t0 + 16 > ld.lo)
      page = gld(a.pool.table + static_cast<int64_t>(ld.b) * a.pool.max_pages + a.pool.by_page.div(t0));
  };
  find_page();
  int slot = 0;
  auto load = [&]() {
    if (left > 0) {
      const int t0 = ld.tile * kTile + 16 * w;
      if (t0 < ld.len && t0 + 16 > ld.lo) {
        const bool ok = page >= 0 && page < a.pool.n_pages;
        if (!ok) {
          set_status(a.status, USP_ERR_BAD_PAGES);
          page = 0;
        }
        const int rj = ld.u / a.chunks, r = rj / a.pool.hk, j = rj - r * a.pool.hk;
        const int64_t row = a.pool.row_of(page, t0, a.pool.by_page.div(t0), r, j);
        const unsigned char* kp = static_cast<const unsigned char*>(a.pool.k) + row * C::kRow;
        const unsigned char* vp = static_cast<const unsigned char*>(a.pool.v) + row * C::kRow;
        const uint32_t dst = ring + slot * C::kStage;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int rr = g + 8 * i;
          const bool in = ok && t0 + rr < ld.len && t0 + rr >= ld.lo;
#pragma unroll
          for (int p = 0; p < C::kKPieces; ++p)
            cp_async16(dst + ((i * C::kKPieces + p) * 32 + lane) * 16, kp + rr * C::kRow + (qd + 4 * p) * 16, in);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = 2 * qd + (i & 1) + 8 * (i >> 1);
          const bool in = ok && t0 + rr < ld.len && t0 + rr >= ld.lo;
#pragma unroll
          for (int p = 0; p < C::kVPieces; ++p) {
            const uint32_t to = dst + 16 * C::kRow + ((i * C::kVPieces + p) * 32 + lane) * C::kVBytes;
            const unsigned char* from = vp + rr * C::kRow + (g + 8 * p) * C::kVBytes;
            if constexpr (C::kVBytes == 16)
              cp_async16(to, from, in);
            else
              cp_async8(to, from, in);
          }
        }
        if constexpr (kE4m3) {
          if (lane < 2)
            cp_async16(dst + 32 * C::kRow + 16 * lane, (lane == 0 ? a.pool.k_scales : a.pool.v_scales) + row, ok);
        }
      }
      --left;
      ld.next(a.pool, a.window, a.units, bad);
      find_page();
    }
    slot = slot + 1 == C::kStages ? 0 : slot + 1;
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) load();

  // ---- the tiles
  uint32_t qf[KS][2];
  float qs[2];          // log2(e) scale / q's power of two, of the thread's two columns
  float m[2], l[2], acc[MT][4];
  bool fresh = true;    // a unit begins (in this CTA)
  int read = 0;
  int part = start_tile == start_first;  // 0: of a unit that began in an earlier CTA; 1: of one that begins here
  for (int it = 0; it < count; ++it) {
    const int rj = cur.u / a.chunks, chunk = cur.u - rj * a.chunks;
    const int r = rj / a.pool.hk, j = rj - r * a.pool.hk;
    const int heads = min(kHeads, a.G - chunk * kHeads);
    // the unit's first query head among [P][n_seqs][hq]
    const int64_t head0 = (static_cast<int64_t>(r) * a.n_seqs + cur.b) * a.hq + j * a.G + chunk * kHeads;
    if (fresh) {
      fresh = false;
      const uint4* qrow = reinterpret_cast<const uint4*>(a.q + (head0 + min(g, heads - 1)) * D);
      const bool have = g < heads;
      if constexpr (!kE4m3) {
#pragma unroll
        for (int p = 0; p < C::kKPieces; ++p) {
          const uint4 x = have ? gld(qrow + qd + 4 * p) : make_uint4(0, 0, 0, 0);
          qf[2 * p][0] = x.x;
          qf[2 * p][1] = x.y;
          qf[2 * p + 1][0] = x.z;
          qf[2 * p + 1][1] = x.w;
        }
        qs[0] = qs[1] = a.scale * kLog2e;
      } else {
        uint32_t x[KS * 2];
        float amax = 0.f;
#pragma unroll
        for (int p = 0; p < C::kKPieces; ++p)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 y = have ? gld(qrow + 2 * (qd + 4 * p) + h) : make_uint4(0, 0, 0, 0);
            const uint32_t z[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[8 * p + 4 * h + e] = z[e];
              amax = fmaxf(amax, fmaxf(fabsf(bf16lo(z[e])), fabsf(bf16hi(z[e]))));
            }
          }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // 2^e with max |q| 2^-e in [2^14, 2^15): f16's range, and 2^-29 of the largest is still normal
        const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14, -126), 112);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < KS * 2; ++i) qf[i >> 1][i & 1] = pack_f16x2(bf16lo(x[i]) * down, bf16hi(x[i]) * down);
        const float up = a.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        qs[0] = __shfl_sync(0xffffffffu, up, 8 * qd);
        qs[1] = __shfl_sync(0xffffffffu, up, 8 * qd + 4);
      }
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    }
    cp_async_wait<C::kStages - 2>();
    __syncwarp();  // (the scales are another lane's copies)
    load();
    const uint32_t src = ring + read * C::kStage;
    read = read + 1 == C::kStages ? 0 : read + 1;
    const int t0 = cur.tile * kTile + 16 * w;
    if (t0 < cur.len && t0 + 16 > cur.lo) {
      // S^T: rows g and g + 8 are positions, columns 2 qd and 2 qd + 1 query heads
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int p = 0; p < C::kKPieces; ++p) {
        const uint4 x = lds16(src + (p * 32 + lane) * 16), y = lds16(src + ((C::kKPieces + p) * 32 + lane) * 16);
        if constexpr (!kE4m3) {
          mma<false>(s, x.x, y.x, x.y, y.y, qf[2 * p][0], qf[2 * p][1]);
          mma<false>(s, x.z, y.z, x.w, y.w, qf[2 * p + 1][0], qf[2 * p + 1][1]);
        } else {
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mma<true>(s, paged::e4m3x2_to_f16x2(xw[e] & 0xffff), paged::e4m3x2_to_f16x2(yw[e] & 0xffff),
                      paged::e4m3x2_to_f16x2(xw[e] >> 16), paged::e4m3x2_to_f16x2(yw[e] >> 16), qf[4 * p + e][0],
                      qf[4 * p + e][1]);
        }
      }
      float ve[2] = {0.f, 0.f};  // exponents of the two positions' values
      float ks[2] = {1.f, 1.f};
      if constexpr (kE4m3) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int kb = lds1(src + 32 * C::kRow + g + 8 * i), vb = lds1(src + 32 * C::kRow + 16 + g + 8 * i);
          ks[i] = kb ? __uint_as_float(static_cast<uint32_t>(kb) << 23) : 0x1p-127f;
          ve[i] = static_cast<float>(vb - 127);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = s[i] * qs[i & 1] * ks[i >> 1];
      if (t0 + 16 > cur.len || t0 < cur.lo) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (t0 + g + 8 * i >= cur.len || t0 + g + 8 * i < cur.lo) s[2 * i] = s[2 * i + 1] = -INFINITY;
      }
      // the running reference of each column (for e4m3 with the values' exponents, from -60 up)
      float top[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        top[c] = kE4m3 ? fmaxf(s[c] + fmaxf(ve[0], -60.f), s[2 + c] + fmaxf(ve[1], -60.f)) : fmaxf(s[c], s[2 + c]);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) top[c] = fmaxf(top[c], __shfl_xor_sync(0xffffffffu, top[c], d));
      }
      if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float mn = fmaxf(m[c], top[c]);
          const float f = m[c] == -INFINITY ? 0.f : ex2(m[c] - mn);
          m[c] = mn;
          l[c] *= f;
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            acc[i][c] *= f;
            acc[i][2 + c] *= f;
          }
        }
      }
      float p[4], pv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float mm = m[i & 1] == -INFINITY ? 0.f : m[i & 1];
        p[i] = ex2(s[i] - mm);
        if constexpr (kE4m3) pv[i] = ex2(s[i] + ve[i >> 1] - mm + 15.f);
      }
      l[0] += p[0] + p[2];
      l[1] += p[1] + p[3];
      // P^T as the operand whose rows are positions
      uint32_t b0, b1, c0 = 0, c1 = 0;
      if constexpr (kE4m3) {
        b0 = transpose8(pack_f16x2(pv[0], pv[1]));
        b1 = transpose8(pack_f16x2(pv[2], pv[3]));
      } else {
        const uint32_t h0 = pack_bf16x2(p[0], p[1]), h1 = pack_bf16x2(p[2], p[3]);
        b0 = transpose8(h0);
        b1 = transpose8(h1);
        c0 = transpose8(pack_bf16x2(p[0] - bf16lo(h0), p[1] - bf16hi(h0)));
        c1 = transpose8(pack_bf16x2(p[2] - bf16lo(h1), p[3] - bf16hi(h1)));
      }
      // O^T += V^T P^T
      const uint32_t vsrc = src + 16 * C::kRow;
      constexpr int W = C::kVBytes / 4;  // words of a piece
#pragma unroll
      for (int pc = 0; pc < C::kVPieces; ++pc) {
        uint32_t x[4][W];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t at = vsrc + ((i * C::kVPieces + pc) * 32 + lane) * C::kVBytes;
          if constexpr (W == 4) {
            const uint4 y = lds16(at);
            x[i][0] = y.x;
            x[i][1] = y.y;
            x[i][2] = y.z;
            x[i][3] = y.w;
          } else {
            const uint2 y = lds8(at);
            x[i][0] = y.x;
            x[i][1] = y.y;
          }
        }
#pragma unroll
        for (int e = 0; e < W; ++e) {
          if constexpr (!kE4m3) {
            const uint32_t a0 = __byte_perm(x[0][e], x[1][e], 0x5410), a1 = __byte_perm(x[0][e], x[1][e], 0x7632);
            const uint32_t a2 = __byte_perm(x[2][e], x[3][e], 0x5410), a3 = __byte_perm(x[2][e], x[3][e], 0x7632);
            mma<false>(acc[pc * 4 + e], a0, a1, a2, a3, b0, b1);
            mma<false>(acc[pc * 4 + e], a0, a1, a2, a3, c0, c1);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // two elements of the two positions each: (x, y, x', y')
              const uint32_t lo = __byte_perm(x[0][e], x[1][e], h ? 0x7362 : 0x5140);
              const uint32_t hi = __byte_perm(x[2][e], x[3][e], h ? 0x7362 : 0x5140);
              mma<true>(acc[2 * e + h], paged::e4m3x2_to_f16x2(lo & 0xffff), paged::e4m3x2_to_f16x2(lo >> 16),
                        paged::e4m3x2_to_f16x2(hi & 0xffff), paged::e4m3x2_to_f16x2(hi >> 16), b0, b1);
            }
          }
        }
      }
    }
    // ---- the unit (or its part in this CTA) ends
    const bool ends = cur.tile + 1 == cur.end;
    if (ends || it + 1 == count) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], d);
      if (g == 0) {
        wm[w][2 * qd] = m[0];
        wm[w][2 * qd + 1] = m[1];
        wl[w][2 * qd] = l[0];
        wl[w][2 * qd + 1] = l[1];
      }
      // [warp][head][d], d with bits 1 and 2 turned over by the head's place so that the stores meet all banks
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int d = value_column<D, kE4m3>(i, g) ^ (2 * qd);
        float* to = merge + (w * kHeads + 2 * qd) * D + d;
        *reinterpret_cast<float2*>(to) = make_float2(acc[i][0], acc[i][2]);
        *reinterpret_cast<float2*>(to + D) = make_float2(acc[i][1], acc[i][3]);
      }
      __syncthreads();
      // 16 threads a head, D/16 elements each
      constexpr int E = D / 16;
      const int h = tid >> 4, d0 = (tid & 15) * E;
      float M = -INFINITY;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) M = fmaxf(M, wm[i][h]);
      const float base = M == -INFINITY ? 0.f : M;
      float L = 0.f, o[E] = {};
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const float f = ex2(wm[i][h] - base);
        L += wl[i][h] * f;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 x = *reinterpret_cast<const float2*>(merge + (i * kHeads + h) * D + ((d0 + e) ^ (2 * (h >> 1))));
          o[e] += x.x * f;
          o[e + 1] += x.y * f;
        }
      }
      if constexpr (kE4m3) {
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= 0x1p-15f;
      }
      if (ends && part == 1) {
        if (h < heads) {
          if (a.sinks != nullptr) {
            const float z = gld(a.sinks + r * a.hq + j * a.G + chunk * kHeads + h) * kLog2e;
            const float mz = fmaxf(M, z), b2 = mz == -INFINITY ? 0.f : mz, f = ex2(base - b2);
            L = L * f + ex2(z - b2);
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] *= f;
            M = b2;
          } else {
            M = base;
          }
          const float inv = L > 0.f ? 1.f / L : 0.f;
          uint32_t out[E / 2];
#pragma unroll
          for (int e = 0; e < E; e += 2) out[e / 2] = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
          uint16_t* to = a.o + (head0 + h) * D + d0;
          if constexpr (E == 8)
            *reinterpret_cast<uint4*>(to) = make_uint4(out[0], out[1], out[2], out[3]);
          else
            *reinterpret_cast<uint2*>(to) = make_uint2(out[0], out[1]);
          if ((tid & 15) == 0) a.lse[head0 + h] = (M + log2f(L)) * kLn2;
        }
      } else {
        const int64_t at = (static_cast<int64_t>(2 * cta + part) * kHeads + h);
        float* to = a.parts + at * D + d0;
#pragma unroll
        for (int e = 0; e < E; e += 4) *reinterpret_cast<float4*>(to + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        if ((tid & 15) == 0) *reinterpret_cast<float2*>(a.stats + at * 2) = make_float2(M, L);
        if (!ends && part == 1 && tid == 0) {
          const long long stop = begin + it + (cur.end - cur.tile);
          a.desc[2 * cta] = cur.b * a.units + cur.u;
          a.desc[2 * cta + 1] = static_cast<int>(paged::cta_of_last(W, n_ctas, stop)) - cta + 1;
        }
      }
      __syncthreads();
      part = 1;
      fresh = true;
    }
    cur.next(a.pool, a.window, a.units, bad);
  }
}

// The parts of the unit that begins in CTA blockIdx.x and ends in a later one, head blockIdx.y of the unit.
template <int D>
__global__ void __launch_bounds__(kThreads) join_kernel(Args a) {
  __shared__ float so[kWarps][D], sl[kWarps];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, h = blockIdx.y;
  constexpr int E = D / 32;
  grid_wait();
  const int cta = blockIdx.x, unit = gld(a.desc + 2 * cta), n = gld(a.desc + 2 * cta + 1);
  if (unit < 0) return;
  const int b = unit / a.units, u = unit - b * a.units, rj = u / a.chunks, chunk = u - rj * a.chunks;
  const int r = rj / a.pool.hk, j = rj - r * a.pool.hk, heads = min(kHeads, a.G - chunk * kHeads);
  if (h >= heads) return;
  // part 0 is the second of the first CTA's two places, the others the first of theirs
  auto place = [&](int i) { return static_cast<int64_t>(2 * (cta + i) + (i == 0)) * kHeads + h; };
  float M = -INFINITY;
  for (int i = lane; i < n; i += 32) M = fmaxf(M, gld(a.stats + 2 * place(i)));
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  const float z = a.sinks != nullptr ? gld(a.sinks + r * a.hq + j * a.G + chunk * kHeads + h) * kLog2e : -INFINITY;
  M = fmaxf(M, z);
  if (M == -INFINITY) M = 0.f;
  float L = 0.f, o[E] = {};
#pragma unroll 4
  for (int i = w; i < n; i += kWarps) {
    const int64_t at = place(i);
    const float2 ml = *reinterpret_cast<const float2*>(a.stats + 2 * at);
    const float f = ex2(ml.x - M);
    L += ml.y * f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] += gld(a.parts + at * D + e * 32 + lane) * f;
  }
  if (lane == 0) sl[w] = L;
#pragma unroll
  for (int e = 0; e < E; ++e) so[w][e * 32 + lane] = o[e];
  __syncthreads();
  float total = ex2(z - M);
#pragma unroll
  for (int i = 0; i < kWarps; ++i) total += sl[i];
  const int64_t head = (static_cast<int64_t>(r) * a.n_seqs + b) * a.hq + j * a.G + chunk * kHeads + h;
  const float inv = total > 0.f ? 1.f / total : 0.f;
  if (tid < D / 2) {
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      x += so[i][2 * tid];
      y += so[i][2 * tid + 1];
    }
    reinterpret_cast<uint32_t*>(a.o)[head * (D / 2) + tid] = pack_bf16x2(x * inv, y * inv);
  }
  if (tid == 0) a.lse[head] = (M + log2f(total)) * kLn2;
}

template <int D, bool kE4m3>
int launch(const Args& a, int ctas, cudaStream_t st) {
  auto* kern = decode_kernel<D, kE4m3>;
  constexpr int smem = Cfg<D, kE4m3>::kSmem;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
    cudaGetLastError();
    return USP_ERR_CUDA;
  }
  const int rc = launch_chained(kern, dim3(ctas), kThreads, smem, 1, st, a);
  if (rc != USP_OK) return rc;
  return launch_chained(join_kernel<D>, dim3(ctas, std::min(kHeads, a.G)), kThreads, 0, 1, st, a);
}

int grid_of(const usp_paged_cache& c) {
  const int row = c.D * (c.dtype == USP_CACHE_E4M3 ? 1 : 2);
  return std::min(kMaxCtas, device_sm_count() * ctas_per_sm(row));
}

}  // namespace decode

// parts, then statistics, then descriptors
size_t attn_decode_ws_bytes(const usp_paged_cache& c) {
  const size_t ctas = decode::grid_of(c), rows = 2 * ctas * decode::kHeads;
  return rows * c.D * 4 + rows * 8 + ctas * 8;
}

int launch_attn_decode(const usp_paged_cache& c, int Hq, int window_left, float scale, const float* sinks,
                       const void* q, void* o, float* lse, void* ws, int32_t* status, cudaStream_t st) {
  decode::Args a{};
  a.pool = paged::Pool(c);
  a.n_seqs = c.n_seqs;
  a.P = c.P;
  a.hq = Hq / c.P;
  a.G = a.hq / a.pool.hk;
  a.chunks = (a.G + decode::kHeads - 1) / decode::kHeads;
  a.units = c.P * a.pool.hk * a.chunks;
  a.window = window_left;
  a.scale = scale;
  a.sinks = sinks;
  a.q = static_cast<const uint16_t*>(q);
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  a.status = status;
  const int ctas = decode::grid_of(c);
  const size_t rows = 2 * static_cast<size_t>(ctas) * decode::kHeads;
  a.parts = static_cast<float*>(ws);
  a.stats = a.parts + rows * c.D;
  a.desc = reinterpret_cast<int32_t*>(a.stats + rows * 2);
  const bool e = c.dtype == USP_CACHE_E4M3;
  if (c.D == 64) return e ? decode::launch<64, true>(a, ctas, st) : decode::launch<64, false>(a, ctas, st);
  return e ? decode::launch<128, true>(a, ctas, st) : decode::launch<128, false>(a, ctas, st);
}

}  // namespace usp
