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
// Sums over d may take d in any order, so a thread's operands are whole 16-byte pieces of its rows.  A warp copies
// its own 16 rows into shared memory (cp.async, 512 consecutive bytes an instruction, tiles ahead) and no barrier but
// the warp's own is needed; only the pairs of positions that V^T's operands want next to each other are
// interleaved, by byte permutations.  Copying each thread's own pieces, in segments of 64 bytes of a
// K row, kept loads at 5.2 TB/s, consecutive rows at 7.0.  (Matrix instructions with operands from shared memory and
// results in tensor memory want 64 rows of queries; here there are G.)
//
// e4m3: an element is exactly an f16, so products run in f16; a token's scales are powers of two
// and act on its score (keys) and on its weight (values).  The reference M of a column is near the maximum of
// score + value exponent (log2), so that the weights of the products, 2^(s + e - M + 7), stay within f16: below
// 2^15, and whole down to 2^-21 of the largest (less than 2^-31 of it is lost).  q is scaled by a power of two into
// f16's range.  The reference moves only when a weight would pass 2^8: no reduction over the warp in most tiles.
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
// A column's reference may stay this far (log2) below a weight; e4m3: weights go into f16 kUp higher (2^15 at most), and
// a token's value exponent counts from kLeast up in the reference.
constexpr float kAbove = 8.f, kUp = 7.f, kDown = 0x1p-7f, kLeast = -60.f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// What fits into an SM's shared memory with the stages below (64 to 96 KB of loads in flight).
constexpr int ctas_per_sm(int row_bytes) { return row_bytes == 256 ? 2 : row_bytes == 128 ? 3 : 4; }

template <int D, bool kE4m3>
struct Cfg {
  static constexpr int kRow = D * (kE4m3 ? 1 : 2);               // bytes of a token's head
  static constexpr int kCopies = kRow / 32;                      // 16-byte copies of a thread for 16 rows
  static constexpr int kKPieces = kRow / 64;                     // 16-byte pieces of a K row that a thread takes (4 threads a row)
  static constexpr int kVBytes = kRow / 8 >= 16 ? 16 : 8;        // a thread's piece of a V row (8 threads a row)
  static constexpr int kVPieces = kRow / 8 / kVBytes;
  static constexpr int kScaleBytes = kE4m3 ? 128 : 0;            // 16 tokens' key and value scales (and up to whole lines)
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

// 16 bytes from global memory to shared memory, past L1
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_or_zero(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
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

// A stretch's place with the unit's parts spelt out.
struct Place : Cursor {
  int r, j, chunk;  // rank, its key/value head, chunk of 8 query heads
  __device__ __forceinline__ void split(const Args& a) {
    const int rj = u / a.chunks;
    chunk = u - rj * a.chunks;
    r = rj / a.pool.hk;
    j = rj - r * a.pool.hk;
  }
  __device__ __forceinline__ void next_unit(const Args& a, bool& bad) {
    tile = end - 1;
    next(a.pool, a.window, a.units, bad);
    split(a);
  }
};

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads, Cfg<D, kE4m3>::kCtas) decode_kernel(Args a) {
  using C = Cfg<D, kE4m3>;
  constexpr int MT = D / 16, KS = D / 16, QV = D / 32;  // QV: 16-byte pieces of a query head that a thread has
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
  Place cur;
  cur.seek(a.pool, a.window, at_seq, at_rest, bad);
  cur.split(a);
  int count = static_cast<int>(finish - begin);
  long long at = begin;                 // the tile of the line that is next
  int part = cur.tile == cur.first;     // 0: of a unit that began in an earlier CTA; 1: of one that begins here

  // ---- loads, kStages - 1 tiles ahead
  const uint32_t ring = smem_u32(smem) + w * (C::kStages * C::kStage);
  float* merge = reinterpret_cast<float*>(smem + C::kStages * C::kStage * kWarps);
  Place ld = cur;
  int left = count;                     // tiles not asked for yet
  int page = 0;                         // of the tile at ld; looked up a tile ahead
  uint32_t col = 0;
  uint32_t slot = 0;                    // where it goes in the ring
  const int64_t page_rows = static_cast<int64_t>(a.pool.hk) * a.pool.page_size;
  const int32_t* table;                 // the sequence's row of the table
  int64_t unit_row;                     // the unit's first row in a page 0
  auto enter_unit = [&]() {
    table = a.pool.table + static_cast<int64_t>(ld.b) * a.pool.max_pages;
    unit_row = static_cast<int64_t>(ld.r) * a.pool.n_pages * page_rows + ld.j * a.pool.page_size;
  };
  auto find_page = [&]() {
    const int t0 = ld.tile * kTile + 16 * w;
    if (t0 < ld.len && t0 + 16 > ld.lo) {
      col = a.pool.by_page.div(t0);
      page = gld(table + col);
    }
  };
  enter_unit();
  find_page();
  // Shared memory holds rows as they are, 16-byte pieces turned over within 128 bytes so that both the copies (512 bytes
  // of consecutive rows an instruction) and the reads below meet all banks: a K row's by 4 where it is odd, a V row's by
  // twice its pair's number mod 4 (rows of 64 bytes: K not at all, V by 2 where the pair is odd).
  constexpr int R = C::kRow;
  const int kput = (lane ^ (R == 256 ? lane >> 4 << 2 : R == 128 ? (lane >> 3 & 1) << 2 : 0)) * 16;
  const int vput = (lane ^ (R == 256 ? 0 : R == 128 ? lane >> 4 << 1 : (lane >> 3 & 1) << 1)) * 16;
  const int kget = g * R + qd * 16 + (R == 64 ? 0 : (g & 1) * 64);
  const int vget = 2 * qd * R + (R == 64 ? ((g >> 1) ^ ((qd & 1) << 1)) * 16 + (g & 1) * 8 : (g ^ (2 * qd)) * 16);
  auto load = [&]() {
    if (left > 0) {
      const int t0 = ld.tile * kTile + 16 * w;
      if (t0 < ld.len && t0 + 16 > ld.lo) {
        const bool ok = page >= 0 && page < a.pool.n_pages;
        const int64_t row = unit_row + (ok ? page : 0) * page_rows + (t0 - static_cast<int>(col) * a.pool.page_size);
        const unsigned char* kp = static_cast<const unsigned char*>(a.pool.k) + row * R + lane * 16;
        const unsigned char* vp = static_cast<const unsigned char*>(a.pool.v) + row * R + lane * 16;
        const uint32_t kdst = ring + slot + kput, vdst = ring + slot + 16 * R + vput;
        const auto vturn = [](int i) { return R == 256 ? (i & 3) << 5 : R == 128 ? (i & 1) << 6 : 0; };
        if (ok && t0 >= ld.lo && t0 + 16 <= ld.len) {
#pragma unroll
          for (int i = 0; i < C::kCopies; ++i) cp_async(kdst + i * 512, kp + i * 512);
#pragma unroll
          for (int i = 0; i < C::kCopies; ++i) cp_async((vdst ^ vturn(i)) + i * 512, vp + i * 512);
        } else {  // zeros for what is not seen: a weight of 0 does not undo a value that is not finite
          if (!ok) set_status(a.status, USP_ERR_BAD_PAGES);
#pragma unroll
          for (int i = 0; i < C::kCopies; ++i) {
            const int t = t0 + (i * 512 + lane * 16) / R;
            const bool in = ok && t < ld.len && t >= ld.lo;
            cp_async_or_zero(kdst + i * 512, kp + i * 512, in);
            cp_async_or_zero((vdst ^ vturn(i)) + i * 512, vp + i * 512, in);
          }
        }
        if constexpr (kE4m3) {
          if (lane < 2)
            cp_async(ring + slot + 32 * R + 16 * lane, (lane == 0 ? a.pool.k_scales : a.pool.v_scales) + row);
        }
      }
      if (--left > 0) {
        if (++ld.tile == ld.end) {
          ld.next_unit(a, bad);
          enter_unit();
        }
        find_page();
      }
    }
    slot = slot == (C::kStages - 1) * C::kStage ? 0 : slot + C::kStage;
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) load();

  // ---- the tiles, unit by unit
  uint4 qx[QV];                        // the thread's pieces of its query head, of the unit that comes
  auto fetch_q = [&]() {
    const int64_t head0 = (static_cast<int64_t>(cur.r) * a.n_seqs + cur.b) * a.hq + cur.j * a.G + cur.chunk * kHeads;
    const uint4* qrow = reinterpret_cast<const uint4*>(a.q + (head0 + g) * D);
    const bool have = cur.chunk * kHeads + g < a.G;
#pragma unroll
    for (int p = 0; p < QV; ++p) {
      // the elements d that meet the thread's pieces of K
      const int at = kE4m3 ? 2 * (qd + 4 * (p >> 1)) + (p & 1) : qd + 4 * p;
      qx[p] = have ? gld(qrow + at) : make_uint4(0, 0, 0, 0);
    }
  };
  fetch_q();
  uint32_t read = 0;
  while (true) {
    uint32_t qf[KS][2];
    float qs[2];  // log2(e) scale q's power of two, of the thread's two columns
    {
      uint32_t x[KS * 2];
#pragma unroll
      for (int p = 0; p < QV; ++p) {
        x[4 * p] = qx[p].x;
        x[4 * p + 1] = qx[p].y;
        x[4 * p + 2] = qx[p].z;
        x[4 * p + 3] = qx[p].w;
      }
      if constexpr (!kE4m3) {
#pragma unroll
        for (int i = 0; i < KS * 2; ++i) qf[i >> 1][i & 1] = x[i];
        qs[0] = qs[1] = a.scale * kLog2e;
      } else {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < KS * 2; ++i) amax = fmaxf(amax, fmaxf(fabsf(bf16lo(x[i])), fabsf(bf16hi(x[i]))));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // 2^e with max |q| 2^-e in [2^14, 2^15): f16's range, and 2^-28 of the largest is still normal
        const int e = min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14, -126), 112);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < KS * 2; ++i) qf[i >> 1][i & 1] = pack_f16x2(bf16lo(x[i]) * down, bf16hi(x[i]) * down);
        const float up = a.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
        qs[0] = __shfl_sync(0xffffffffu, up, 8 * qd);
        qs[1] = __shfl_sync(0xffffffffu, up, 8 * qd + 4);
      }
    }
    float m[2] = {-INFINITY, -INFINITY}, ref[2] = {0.f, 0.f};  // the columns' references (ref: finite)
    float l[2] = {0.f, 0.f}, acc[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
    bool none = true;  // no visible position yet
    const int tiles = min(count, cur.end - cur.tile);
    int t0 = cur.tile * kTile + 16 * w;
    for (int it = 0; it < tiles; ++it, t0 += kTile) {
      cp_async_wait<C::kStages - 2>();
      __syncwarp();  // every lane's copies are here, and its reads of the place that is filled next are done
      load();
      const uint32_t src = ring + read;
      read = read == (C::kStages - 1) * C::kStage ? 0 : read + C::kStage;
      if (t0 >= cur.len || t0 + 16 <= cur.lo) continue;
      // S^T: rows g and g + 8 are positions, columns 2 qd and 2 qd + 1 query heads
      float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int p = 0; p < C::kKPieces; ++p) {
        const uint32_t from = ((src + kget) ^ (p & 1) * 64) + (p >> 1) * 128;
        const uint4 x = lds16(from), y = lds16(from + 8 * R);
        if constexpr (!kE4m3) {
          mma<false>(s, x.x, y.x, x.y, y.y, qf[2 * p][0], qf[2 * p][1]);
          mma<false>(s2, x.z, y.z, x.w, y.w, qf[2 * p + 1][0], qf[2 * p + 1][1]);
        } else {
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mma<true>(e & 1 ? s2 : s, paged::e4m3x2_to_f16x2(xw[e] & 0xffff), paged::e4m3x2_to_f16x2(yw[e] & 0xffff),
                      paged::e4m3x2_to_f16x2(xw[e] >> 16), paged::e4m3x2_to_f16x2(yw[e] >> 16), qf[4 * p + e][0],
                      qf[4 * p + e][1]);
        }
      }
      float ve[2] = {0.f, 0.f};  // exponents of the two positions' values
      float ks[2] = {1.f, 1.f};
      if constexpr (kE4m3) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int kb = lds1(src + 32 * R + g + 8 * i), vb = lds1(src + 32 * R + 16 + g + 8 * i);
          ks[i] = kb ? __uint_as_float(static_cast<uint32_t>(kb) << 23) : 0x1p-127f;
          ve[i] = static_cast<float>(vb - 127);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[i] = (s[i] + s2[i]) * qs[i & 1];
        if constexpr (kE4m3) s[i] *= ks[i >> 1];
      }
      if (t0 + 16 > cur.len || t0 < cur.lo) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (t0 + g + 8 * i >= cur.len || t0 + g + 8 * i < cur.lo) s[2 * i] = s[2 * i + 1] = -INFINITY;
      }
      // The reference of a column follows its scores only when one is 2^8 above it.
      float x[4];
      bool above = none;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = s[i] - ref[i & 1];
        above |= (kE4m3 ? x[i] + fmaxf(ve[i >> 1], kLeast) : x[i]) > kAbove;
      }
      if (__any_sync(0xffffffffu, above)) {
        none = false;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float top = kE4m3 ? fmaxf(s[c] + fmaxf(ve[0], kLeast), s[2 + c] + fmaxf(ve[1], kLeast)) : fmaxf(s[c], s[2 + c]);
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          const float mn = fmaxf(m[c], top);
          const float f = m[c] == -INFINITY ? 0.f : ex2(m[c] - mn);
          m[c] = mn;
          ref[c] = mn == -INFINITY ? 0.f : mn;
          l[c] *= f;
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            acc[i][c] *= f;
            acc[i][2 + c] *= f;
          }
          x[c] = s[c] - ref[c];
          x[2 + c] = s[2 + c] - ref[c];
        }
      }
      float p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = ex2(x[i]);
      l[0] += p[0] + p[2];
      l[1] += p[1] + p[3];
      // P^T as the operand whose rows are positions
      uint32_t b0, b1, c0 = 0, c1 = 0;
      if constexpr (kE4m3) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = ex2(x[i] + (ve[i >> 1] + kUp));
        b0 = transpose8(pack_f16x2(p[0], p[1]));
        b1 = transpose8(pack_f16x2(p[2], p[3]));
      } else {
        const uint32_t h0 = pack_bf16x2(p[0], p[1]), h1 = pack_bf16x2(p[2], p[3]);
        b0 = transpose8(h0);
        b1 = transpose8(h1);
        c0 = transpose8(pack_bf16x2(p[0] - bf16lo(h0), p[1] - bf16hi(h0)));
        c1 = transpose8(pack_bf16x2(p[2] - bf16lo(h1), p[3] - bf16hi(h1)));
      }
      // O^T += V^T P^T
      const uint32_t vsrc = src + 16 * R + vget;
      constexpr int W4 = C::kVBytes / 4;  // words of a piece
#pragma unroll
      for (int pc = 0; pc < C::kVPieces; ++pc) {
        uint32_t v[4][W4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t from = vsrc + ((i & 1) + 8 * (i >> 1)) * R + pc * 128;
          if constexpr (W4 == 4) {
            const uint4 y = lds16(from);
            v[i][0] = y.x;
            v[i][1] = y.y;
            v[i][2] = y.z;
            v[i][3] = y.w;
          } else {
            const uint2 y = lds8(from);
            v[i][0] = y.x;
            v[i][1] = y.y;
          }
        }
#pragma unroll
        for (int e = 0; e < W4; ++e) {
          if constexpr (!kE4m3) {
            const uint32_t a0 = __byte_perm(v[0][e], v[1][e], 0x5410), a1 = __byte_perm(v[0][e], v[1][e], 0x7632);
            const uint32_t a2 = __byte_perm(v[2][e], v[3][e], 0x5410), a3 = __byte_perm(v[2][e], v[3][e], 0x7632);
            mma<false>(acc[pc * 4 + e], a0, a1, a2, a3, b0, b1);
            mma<false>(acc[pc * 4 + e], a0, a1, a2, a3, c0, c1);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // two elements of the two positions each: (x, y, x', y')
              const uint32_t lo = __byte_perm(v[0][e], v[1][e], h ? 0x7362 : 0x5140);
              const uint32_t hi = __byte_perm(v[2][e], v[3][e], h ? 0x7362 : 0x5140);
              mma<true>(acc[2 * e + h], paged::e4m3x2_to_f16x2(lo & 0xffff), paged::e4m3x2_to_f16x2(lo >> 16),
                        paged::e4m3x2_to_f16x2(hi & 0xffff), paged::e4m3x2_to_f16x2(hi >> 16), b0, b1);
            }
          }
        }
      }
    }

    // ---- the unit (or its part in this CTA) ends
    const bool ends = cur.tile + tiles == cur.end;
    const int unit = cur.b * a.units + cur.u, heads = min(kHeads, a.G - cur.chunk * kHeads);
    const int64_t head0 = (static_cast<int64_t>(cur.r) * a.n_seqs + cur.b) * a.hq + cur.j * a.G + cur.chunk * kHeads;
    const int sink0 = cur.r * a.hq + cur.j * a.G + cur.chunk * kHeads;
    const long long stop = at + (cur.end - cur.tile);  // where the unit ends on the line
    count -= tiles;
    at += tiles;
    if (count > 0) {  // the next unit's query is on its way while the warps' results are put together
      cur.next_unit(a, bad);
      fetch_q();
    }
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
        const float2 y = *reinterpret_cast<const float2*>(merge + (i * kHeads + h) * D + ((d0 + e) ^ (2 * (h >> 1))));
        o[e] += y.x * f;
        o[e + 1] += y.y * f;
      }
    }
    if constexpr (kE4m3) {
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= kDown;
    }
    if (ends && part == 1) {
      if (h < heads) {
        M = base;
        if (a.sinks != nullptr) {
          const float z = gld(a.sinks + sink0 + h) * kLog2e;
          M = fmaxf(base, z);
          const float f = ex2(base - M);
          L = L * f + ex2(z - M);
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] *= f;
        }
        const float inv = L > 0.f ? 1.f / L : L;  // (0 stays 0, NaN NaN)
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
      const int64_t place = static_cast<int64_t>(2 * cta + part) * kHeads + h;
      float* to = a.parts + place * D + d0;
#pragma unroll
      for (int e = 0; e < E; e += 4) *reinterpret_cast<float4*>(to + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
      if ((tid & 15) == 0) *reinterpret_cast<float2*>(a.stats + place * 2) = make_float2(M, L);
      if (!ends && part == 1 && tid == 0) {
        a.desc[2 * cta] = unit;
        a.desc[2 * cta + 1] = static_cast<int>(paged::cta_of_last(W, n_ctas, stop)) - cta + 1;
      }
    }
    if (count == 0) return;
    part = 1;
    __syncthreads();
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
  const float inv = total > 0.f ? 1.f / total : total;  // (0 stays 0, NaN NaN)
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
