// usp_decode.cu — attention of one new token per sequence over a paged cache.
//
//   s_u = scale q.k_u,  O = sum_u exp(s_u - LSE) v_u,  LSE = ln(sum_u exp(s_u) + exp(sink))
//
// Bound by HBM: every visible token's key and value are read once and take part in 4 D flop
// for each of the G query heads of their group, G a few: far below the card's ratio.  So
// what counts is that loads never pause and that all SMs have the same share of them.
//
// Shares.  The work of all sequences is one line of tiles of 16 positions (of a sequence, a rank
// and a key/value head: a "unit"); each CTA takes an equal stretch of the line and each of its warps
// a part of that, found from the lengths on the device, whatever they are.  A warp runs through its tiles
// without waiting for the others.  A unit that lies in one warp is finished there.  Of one that several share
// each leaves a partial result (O, maximum, sum in fp32): the CTA puts its warps' together once,
// when all are done, and what crosses CTAs goes through the workspace.  Parts are joined in the order of the
// positions.  A warp has 8 query heads.  Where a group has more and the line is long, two warps make a team: they go through
// the same tiles, which one ring of twice the size holds, each for 8 heads, so that tiles are read once for 16 of them.
//
// Loads.  The products are arranged so that the positions are the rows of the matrix
// instruction and the query heads its 8 columns (S^T = K q^T, O^T = V^T P^T): rows of 16 query heads would be
// half empty for groups up to 8.  Sums over d may take d in any order, so a thread's operands are whole 16-byte
// pieces of its rows.  A warp copies its own 16 rows into shared memory (cp.async, 512 consecutive bytes an
// instruction, tiles ahead) and no barrier but the warp's own is needed; only the pairs of positions that V^T's
// operands want next to each other are interleaved, by byte permutations.  Copying each thread's own pieces, in
// segments of 64 bytes of a K row, kept loads at 5.2 TB/s, consecutive rows at 7.0.
// (The matrix instruction with operands in shared memory and results in tensor memory takes this arrangement too,
// positions as its 64 or 128 rows and 8 heads or more as columns.  Up to 8 heads a group it has nothing to give: HBM
// bounds them, with the tensor pipe 12% busy.  Larger groups are bound by instructions here; it is not tried for them:
// weights would go through shared or tensor memory, and e4m3 codes be made f16 first, or weights and queries 8 bits.)
//
// e4m3: an element is exactly an f16, so products run in f16; a token's scales are powers of two
// and act on its score (keys) and on its weight (values).  The reference M of a column is near the maximum of
// score + value exponent (log2), so that the weights of the products, 2^(s + e - M + 7), stay within f16: below
// 2^15, and whole down to 2^-21 of the largest (less than 2^-31 of it is lost).  q is scaled by a power of two into
// f16's range.  The reference moves only when a weight would pass 2^8: no reduction over the warp in most tiles.
// The same reference would flush the sum of the weights 2^(s - M) where values are near the largest bf16, and the
// products' weights where they are near the smallest: a unit whose sum shows that goes through the warp once more, its
// references near the scores' maximum and those of the products' weights kept beside them.  (That look at the sums costs
// groups of 16 heads 1.9%, up to 6% of them over one sequence, 0.4 us of the smallest calls and 1% of others; finding such
// values on the way, in one pass for all, 4 to 8% of 16 heads.)
// bf16: the weights are rounded to bf16 in two parts (high and the rest), 16 bits of them in all: one part alone would
// make the output's error 1.4 times that of its own rounding.
//
// Measured (one GB300, the GPU's time in a captured graph of calls on several states in turn, larger than L2 together; the
// floor is the cache's visible bytes at the measured copy rate of 6.69 TB/s): 32 sequences of up to 8192, 32/8 heads, D
// 128, bf16: 109 us, floor 104; one of 131072, 28/4 heads, e4m3: 32 to 33 us, floor 20; windows of 128 over 256 sequences,
// 64/8 heads, D 64, bf16: 15.1 us, floor 8.7; one of 500: 7.3 us.  What is above the floor is the begin (lengths, table
// and first rows: a chain of loads, 2 us) and the end (a sum over the warps, a ticket, the parts of other CTAs: round trips
// that wait behind the loads of the SMs that still work, 3 to 6 us).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>
#include <utility>

#include "usp_internal.h"
#include "usp_paged.cuh"
#include "usp_ptx.cuh"

namespace usp {
namespace decode {

using paged::Cursor;
using paged::Deal;
using paged::kTile;
static_assert(kTile == 16, "the rows of a matrix instruction");
constexpr int kFan = 48;            // parts that a CTA puts together at once
// Tiles that a warp works through in the time that putting a CTA's parts together takes, and joining those of CTAs too.
// (us, of one state, which L2 holds; 8 heads, D 128, bf16 unless stated: the rule counts tiles, whatever their bytes.  64
// sequences of up to 100 tokens: tiles to the warps 10.5, units to the warps 8.2; 8 of up to 200: tiles 8.4, units to the
// CTAs 5.8, to the warps 11.5; 16 of 1000: 12.7, 10.1; 200 of up to 500, D 64, e4m3: 22.9, units to the CTAs 23.4, to the
// warps 26.8.)
constexpr int kWarpsTiles = 3, kCtasTiles = 8;
constexpr int kHeads = 8;           // query heads of a warp
// Groups of more than 8 query heads: teams of two warps where each team of the grid would have this many tiles and a
// token's row has 128 bytes or more, else a unit for each 8 heads.  (us, as teams / as units of 8; groups of 16 heads.
// bf16, D 128: 32 sequences of 8000, 8 groups 172 / 305; of 2000, 53 tiles a team, 56 / 86; 8 of 4000, 26 tiles, 36 / 27; one of
// 131072, 4 groups, 54 tiles, 61 / 82.  D 64: 32 of 2000, 35 tiles, 35 / 46; 16 of 4000, 35 tiles, 35.3 / 33.6; 8 of 4000, 18
// tiles, 26 / 18.  e4m3, D 128: 32 of 8000 121 / 165; of 2000, 35 tiles, 45 / 50; one of 131072, 36 tiles, 54 / 49; of 262144,
// 72 tiles, 80 / 88.  e4m3, D 64, whose codes are converted once a warp and bound it: 32 of 2000, 26 tiles, 33 / 31; of 4000,
// 53 tiles, 54 / 48; of 16000, 211 tiles, 163 / 167; 4 of 262144, 431 tiles, 317 / 289: no teams.  Teams of four for 32
// heads a group were slower than two of two.)
constexpr int kTeamTiles = 32;
constexpr int kMaxCtas = 1024, kTicketBytes = kMaxCtas * 12;
// A column's reference may stay this far (log2) below a weight; e4m3: weights of the products go into f16 kUp higher
// (2^15 at most), and a token's value exponent counts from kLeast up in the reference.
constexpr float kAbove = 8.f, kUp = 7.f, kDown = 0x1p-7f, kLeast = -60.f;
// e4m3: a sum of weights within these has its reference at most 2^44 below the scores' maximum (kLeast has had no effect)
// and 2^30 a position above it, so that nothing that counts is flushed here or beside other parts (values from about
// 2^-20 to 2^30 are within them, however many); scores up to kHuge have roundings that are small beside an exponent.
// Else the unit goes once more, its references within kFar of the maximum.
constexpr float kSumLeast = 0x1p-30f, kSumMost = 0x1p44f, kHuge = 0x1p22f, kFar = 20.f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int D, bool kE4m3>
struct Cfg {
  static constexpr int kRow = D * (kE4m3 ? 1 : 2);               // bytes of a token's head
  static constexpr int kCopies = kRow / 32;                      // 16-byte copies of a thread for 16 rows
  static constexpr int kKPieces = kRow / 64;                     // 16-byte pieces of a K row that a thread takes (4 threads a row)
  static constexpr int kVBytes = kRow / 8 >= 16 ? 16 : 8;        // a thread's piece of a V row (8 threads a row)
  static constexpr int kVPieces = kRow / 8 / kVBytes;
  static constexpr int kScaleBytes = kE4m3 ? 128 : 0;            // 16 tokens' key and value scales (and up to whole lines)
  static constexpr int kStage = 2 * 16 * kRow + kScaleBytes;     // one warp's share of a tile
  // One CTA per SM, of as many warps as its registers and shared memory hold: few CTAs leave few parts to join.
  static constexpr int kWarps = kRow == 256 ? 8 : kRow == 128 ? 12 : 16, kThreads = 32 * kWarps;
  // Tiles ahead: 100 to 130 KB of loads in flight per SM.  (Two stages: the same at D 128 bf16, 2% slower at e4m3; ten
  // warps of two stages: 2 to 4% faster on a gigabyte, 8% slower on the smallest calls.)
  static constexpr int kStages = kRow == 64 ? 4 : 3;
  static constexpr int kRing = kStages * kStage;
  static constexpr int kKept = kHeads * D * 4;                   // a partial O of a warp
  // Of a partial result: reference and sum of its weights; e4m3: how far above that reference the values' one is, too.
  using Stat = std::conditional_t<kE4m3, float4, float2>;
  static constexpr int kRings = kWarps * (kRing + kKept), kJoin = kFan * (kKept + kHeads * static_cast<int>(sizeof(Stat)));
  static constexpr int kSmem = kRings > kJoin ? kRings : kJoin;  // (the join takes shared memory that is done with)
  static_assert(kRing >= kKept, "a partial O fits into a ring that is done with");
};

// The units of a sequence: P * hk * chunks, chunks of the G query heads of a group.
struct Units {
  int chunks, all;
  FastDiv by_all, by_chunks;
};

struct Args {
  paged::Pool pool;
  int n_seqs, P, hq, G;
  Units one, team;                      // with chunks of a warp's heads, of a team's
  int window;                           // -1: none
  float scale;                          // softmax scale
  FastDiv by_hk;
  const float* sinks;
  const uint16_t* q;
  uint16_t* o;
  float* lse;
  float* parts;                         // [2 * ctas][team's warps][kHeads][D], then [2 * ctas][team's warps][kHeads] Stats
  void* stats;
  int32_t* tickets;                     // [ctas][3], zero between calls
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

// The matrix row pair mt of V^T has elements d, d + 1 of thread group g's pieces, in order: row pairs 4 x .. 4 x + 3 are
// the eight elements from first_column(x, g) on.
template <int D, bool kE4m3>
__device__ __forceinline__ int first_column(int x, int g) {
  return kE4m3 ? (D / 8) * g + 8 * x : 64 * x + 8 * g;
}

// O and LSE of the sequences first, first + step, ... that see nothing, in a warp.
template <int D>
__device__ __noinline__ void write_empty(const Args& a, int first, int step) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  for (int s = first; s < a.n_seqs; s += step) {
    if (tiles_of(a, s, bad) != 0) continue;
    for (int r = 0; r < a.P; ++r) {
      uint4* o = reinterpret_cast<uint4*>(a.o + (static_cast<int64_t>(r) * a.n_seqs + s) * a.hq * D);
      for (int i = lane; i < a.hq * (D / 8); i += 32) o[i] = make_uint4(0, 0, 0, 0);
    }
    for (int i = lane; i < a.P * a.hq; i += 32) {
      const int r = i / a.hq;
      a.lse[(static_cast<int64_t>(r) * a.n_seqs + s) * a.hq + (i - r * a.hq)] = a.sinks ? gld(a.sinks + i) : -INFINITY;
    }
  }
}

// A warp's part of a unit that its team shares with others.
struct Part {
  int unit;           // (sequence * units + unit) * the team's warps + which of them, -1: none
  int begins, ends;   // the unit begins, ends in it
  int tiles;          // of the whole unit
  uint32_t stop;      // where the unit ends on the line
};

// The query heads of a warp in a unit: row of the first among [P][n_seqs][hq], how many (none: <= 0), its sink.
struct Heads {
  int64_t row;
  int n, sink;
  __device__ __forceinline__ Heads(const Args& a, int b, int r, int j, int chunk) {
    const int h0 = j * a.G + chunk * kHeads;
    row = (static_cast<int64_t>(r) * a.n_seqs + b) * a.hq + h0;
    n = min(kHeads, a.G - chunk * kHeads);
    sink = r * a.hq + h0;
  }
};

// From a head's reference M (log2; -inf: no weight), how far V the values' one is above it (e4m3) and the sum: its LSE,
// and what makes outputs of its weighted values, x half scale (e4m3: 2^(M + V) in two halves, either of which is in
// fp32's range) or x scale.
template <bool kE4m3>
struct Finish {
  float half, scale, lse;
  __device__ __forceinline__ Finish(const Args& a, const Heads& hd, int h, float M, float V, float sum) {
    // the sink joins the sum once, with no value
    const float z = a.sinks != nullptr ? gld(a.sinks + hd.sink + h) * kLog2e : -INFINITY, top = fmaxf(M, z);
    const float ref = top == -INFINITY ? 0.f : top, f = ex2(M - ref);
    sum = sum * f + ex2(z - ref);
    half = kE4m3 ? ex2(0.5f * (M - ref + V)) : 1.f;
    scale = sum > 0.f ? (kE4m3 ? half : f) / sum : sum;  // (0 stays 0, NaN NaN)
    lse = (ref + log2f(sum)) * kLn2;
  }
  __device__ __forceinline__ float operator()(float x) const { return (kE4m3 ? x * half : x) * scale; }
};

// How the work is dealt out: the line's tiles to the teams, whole units to the CTAs, whose teams share them, or to the
// teams.
enum class Split { kTiles, kUnitsToCtas, kUnitsToTeams };

// A stretch's place with the unit's parts spelt out.
struct Place : Cursor {
  int r, j, chunk;  // rank, its key/value head, chunk of a team's query heads
  __device__ __forceinline__ void split(const Args& a, const Units& un) {
    const int rj = un.by_chunks.div(u);
    chunk = u - rj * un.chunks;
    r = a.by_hk.div(rj);
    j = rj - r * a.pool.hk;
  }
  __device__ __forceinline__ void next_unit(const Args& a, const Units& un, bool& bad) {
    Cursor::next_unit(a.pool, a.window, un.all, bad);
    split(a, un);
  }
};

// The largest value of a column (in the lanes of the same place in their four).
__device__ __forceinline__ float column_max(float v) {
#pragma unroll
  for (int d = 4; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}

// The reference of a column whose value exponents are far from 0 moves: to m, within kFar of the scores' maximum, with
// the products' weights raised beside it; (log2) drop is what their earlier ones have less.  kept: the scores' maximum and
// the raise; was, m: the reference so far (-inf: none), and at least; z, e: the lane's scores and their values' exponents.
struct Moved {
  float m, drop, raise;
};
__device__ __noinline__ Moved far_reference(float4* kept, float was, float m, float z0, float z1, float e0,
                                            float e1) {
  const bool first = was == -INFINITY;
  const float raised = first ? 0.f : kept->y;
  const float most = fmaxf(first ? -INFINITY : kept->x, column_max(fmaxf(z0, z1)));
  m = fminf(fmaxf(m, most - kFar), most + kFar);
  const float ref = m == -INFINITY ? 0.f : m;
  // above the reference, that of the values: near 0 unless the one is at an end or scores are huge
  float over = column_max(fmaxf(z0 - ref + e0, z1 - ref + e1));
  if (!first) over = fmaxf(over, was - m - raised);
  const float raise = fabsf(over) > 1.f && over != -INFINITY ? -over : 0.f;
  __syncwarp();
  if ((threadIdx.x & 31) < 4) *kept = make_float4(most, raise, 0.f, 0.f);
  return Moved{m, was - m - raised + raise, raise};
}

// The barrier of a team of T warps.
template <int T>
__device__ __forceinline__ void team_sync(int team) {
  if constexpr (T == 1)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * T) : "memory");
}

// Whether p holds in one of a team's lanes; a barrier.
template <int T>
__device__ __forceinline__ bool team_any(int team, bool p) {
  if constexpr (T == 1) return __any_sync(0xffffffffu, p);
  int any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %3, 0;\n\tbar.red.or.pred q, %1, %2, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(1 + team), "n"(32 * T), "r"(static_cast<int>(p))
      : "memory");
  return any != 0;
}

// (Whatever the lengths have become since, each of a team's warps comes to its barrier once a tile and once behind the
// last one, e4m3 at each end of a unit too, of as many tiles as its first warp found: what decides on that has been read
// once, in the CTA or the team.)
//
// A team's stretch: `count` tiles from `at` of the line, `count` whole units, or its share of the CTA's `count` units; it
// (for a share, they) begins start.y tiles, or units, into sequence start.x.
template <int D, bool kE4m3, int T>
__device__ __forceinline__ void run_stretch(const Args& a, unsigned char* smem, Part* parts,
                                            typename Cfg<D, kE4m3>::Stat (*stats)[kHeads],
                                            volatile uint32_t* shared, int2 start, Split split, uint32_t at,
                                            int count) {
  using C = Cfg<D, kE4m3>;
  constexpr int MT = D / 16, KS = D / 16, QV = D / 32;  // QV: 16-byte pieces of a query head that a thread has
  const Units& un = T > 1 ? a.team : a.one;
  constexpr int kTeams = C::kWarps / T, kSlots = T * C::kStages;  // (of the CTA; tiles that the team's ring holds)
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, qd = lane & 3;
  const int team = w / T, mem = w % T;
  float* kept = reinterpret_cast<float*>(smem + C::kWarps * C::kRing + w * C::kKept);
  bool bad = false;  // (reported when the lengths were added up)
  Place cur;
  if (split != Split::kTiles) {
    cur.sequence(a.pool, a.window, start.x, bad);
    cur.u = static_cast<int>(min(static_cast<uint32_t>(start.y), static_cast<uint32_t>(un.all - 1)));
    Cursor c = cur;
    uint32_t tiles = 0;
    const int units = count;
    for (int i = 0; i < units; ++i) {
      tiles += c.tiles();
      c.next_unit(a.pool, a.window, un.all, bad);
    }
    if constexpr (T > 1) {
      if (mem == 0 && lane == 0) shared[0] = tiles;
      team_sync<T>(team);
      tiles = shared[0];
    }
    count = tiles;
    if (split == Split::kUnitsToCtas) {
      const Deal own(tiles, kTeams);
      at = own.begin(team);
      count = own.begin(team + 1) - at;
      if (count == 0) return;
      int skip = at;
      for (int i = 1; i < units && skip >= cur.tiles(); ++i) {
        skip -= cur.tiles();
        cur.Cursor::next_unit(a.pool, a.window, un.all, bad);
      }
      cur.tile = cur.first + skip;
    }
  } else {
    cur.seek(a.pool, a.window, un.all, start.x, start.y, bad);
  }
  cur.split(a, un);
  bool begins = cur.tile == cur.first;  // the unit at hand begins in this team

  // ---- loads, kSlots - 1 tiles ahead
  const uint32_t ring = smem_u32(smem) + team * T * C::kRing;
  Place ld = cur;
  int left = count;                     // tiles not asked for yet
  uint32_t slot = 0;                    // where the next one goes in the ring
  const int64_t page_rows = a.pool.page_rows();
  const int32_t* table;                 // the entry of the page at hand
  int64_t unit_row;                     // the unit's first row in a page 0
  int page, off;                        // the page at hand (looked up a tile ahead), where in it the next tile begins
  bool new_page = true, ok = false;     // it has not been entered yet; it is one of the pool's
  int full, full_end;                   // tiles of which every position is visible
  const unsigned char *kp, *vp;         // the lane's first pieces of the next tile (in a team kp: keys' or values')
  const uint8_t* sp;                    // its scales, keys' in lane 0, values' in lane 1
  auto enter_unit = [&]() {
    const int t0 = ld.tile * kTile;
    const uint32_t col = min(a.pool.by_page.div(t0), static_cast<uint32_t>(a.pool.max_pages - 1));
    table = a.pool.table + static_cast<int64_t>(ld.b) * a.pool.max_pages + col;
    page = gld(table);
    off = min(t0 - static_cast<int>(col) * a.pool.page_size, a.pool.page_size - kTile);
    unit_row = a.pool.unit_row(ld.r, ld.j);
    full = (ld.lo + kTile - 1) / kTile;
    full_end = ld.len / kTile;
    new_page = true;
  };
  enter_unit();
  // Shared memory holds rows as they are, 16-byte pieces turned over within 128 bytes so that both the copies (512 bytes
  // of consecutive rows an instruction) and the reads below meet all banks: a K row's by 4 where it is odd, a V row's by
  // twice its pair's number mod 4 (rows of 64 bytes: K not at all, V by 2 where the pair is odd).
  constexpr int R = C::kRow;
  const int kput = (lane ^ (R == 256 ? lane >> 4 << 2 : R == 128 ? (lane >> 3 & 1) << 2 : 0)) * 16;
  const int vput = (lane ^ (R == 256 ? 0 : R == 128 ? lane >> 4 << 1 : (lane >> 3 & 1) << 1)) * 16;
  const int kget = g * R + qd * 16 + (R == 64 ? 0 : (g & 1) * 64);
  const int vget = 2 * qd * R + (R == 64 ? ((g >> 1) ^ ((qd & 1) << 1)) * 16 + (g & 1) * 8 : (g ^ (2 * qd)) * 16);
  // In a team one warp copies the keys, the other the values.
  const bool values = mem != 0;
  const int put = values ? 16 * R + vput : kput, turned = values ? -1 : 0;
  auto load = [&]() {
    if (left > 0) {
      if (new_page) {
        new_page = false;
        ok = page >= 0 && page < a.pool.n_pages;
        if (!ok) set_status(a.status, USP_ERR_BAD_PAGES);
        const int64_t row = unit_row + (ok ? page : 0) * page_rows + off;
        kp = static_cast<const unsigned char*>(values ? a.pool.v : a.pool.k) + row * R + lane * 16;
        if constexpr (T == 1) vp = static_cast<const unsigned char*>(a.pool.v) + row * R + lane * 16;
        if constexpr (kE4m3) sp = (lane == 0 ? a.pool.k_scales : a.pool.v_scales) + row;
      }
      const uint32_t kdst = ring + slot + kput, vdst = ring + slot + 16 * R + vput;
      const auto vturn = [](int i) { return R == 256 ? (i & 3) << 5 : R == 128 ? (i & 1) << 6 : 0; };
      if constexpr (T > 1) {
        const uint32_t dst = ring + slot + put;
        if (ok && ld.tile >= full && ld.tile < full_end) {
#pragma unroll
          for (int i = 0; i < C::kCopies; ++i) cp_async((dst ^ (vturn(i) & turned)) + i * 512, kp + i * 512);
        } else {
#pragma unroll
          for (int i = 0; i < C::kCopies; ++i) {
            const int t = ld.tile * kTile + (i * 512 + lane * 16) / R;
            cp_async_or_zero((dst ^ (vturn(i) & turned)) + i * 512, kp + i * 512, ok && t < ld.len && t >= ld.lo);
          }
        }
      } else if (ok && ld.tile >= full && ld.tile < full_end) {
#pragma unroll
        for (int i = 0; i < C::kCopies; ++i) cp_async(kdst + i * 512, kp + i * 512);
#pragma unroll
        for (int i = 0; i < C::kCopies; ++i) cp_async((vdst ^ vturn(i)) + i * 512, vp + i * 512);
      } else {  // zeros for what is not seen: a weight of 0 does not undo a value that is not finite
#pragma unroll
        for (int i = 0; i < C::kCopies; ++i) {
          const int t = ld.tile * kTile + (i * 512 + lane * 16) / R;
          const bool in = ok && t < ld.len && t >= ld.lo;
          cp_async_or_zero(kdst + i * 512, kp + i * 512, in);
          cp_async_or_zero((vdst ^ vturn(i)) + i * 512, vp + i * 512, in);
        }
      }
      if constexpr (kE4m3) {
        if (lane < 2 && mem == 0) cp_async(ring + slot + 32 * R + 16 * lane, sp);
        sp += kTile;
      }
      kp += kTile * R;
      if constexpr (T == 1) vp += kTile * R;
      off += kTile;
      if (--left > 0) {
        if (++ld.tile >= ld.end) {
          ld.next_unit(a, un, bad);
          enter_unit();
        } else if (off == a.pool.page_size) {
          off = 0;
          page = gld(++table);
          new_page = true;
        }
      }
    }
    slot = slot == (kSlots - 1) * C::kStage ? 0 : slot + C::kStage;
    cp_async_commit();
  };
#pragma unroll(T == 1 ? C::kStages - 1 : 1)
  for (int i = 0; i < kSlots - 1; ++i) load();

  // ---- the tiles, unit by unit
  uint4 qx[QV];                        // the thread's pieces of its query head, of the unit that comes
  auto fetch_q = [&]() {
    const Heads hd(a, cur.b, cur.r, cur.j, cur.chunk * T + mem);
    const uint4* qrow = reinterpret_cast<const uint4*>(a.q + (hd.row + g) * D);
    const bool have = g < hd.n;
#pragma unroll
    for (int p = 0; p < QV; ++p) {
      // the elements d that meet the thread's pieces of K
      const int at = kE4m3 ? 2 * (qd + 4 * (p >> 1)) + (p & 1) : qd + 4 * p;
      qx[p] = have ? gld(qrow + at) : make_uint4(0, 0, 0, 0);
    }
  };
  fetch_q();
  uint32_t read = 0;
  bool far = false;  // e4m3: the unit goes through once more, with references for value exponents far from 0
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
    // a column has no weight yet (every score so far hidden or -inf): its reference is to be set; or far
    bool none = true;
    const int kept_at = 2 * w + begins;
    int tiles = min(count, cur.left());
    if constexpr (T > 1 && kE4m3) {
      if (mem == 0 && lane == 0) shared[1] = tiles;
      team_sync<T>(team);
      tiles = shared[1];
    }
    int t0 = cur.tile * kTile;
    for (int it = 0; it < tiles; ++it, t0 += kTile) {
      cp_async_wait<kSlots - 2>();
      team_sync<T>(team);  // every lane's copies are here, and its reads of the place that is filled next are done
      load();
      const uint32_t src = ring + read;
      read = read == (kSlots - 1) * C::kStage ? 0 : read + C::kStage;
      // S^T: rows g and g + 8 are positions, columns 2 qd and 2 qd + 1 query heads
      constexpr bool kTwo = C::kWarps <= 8;  // two chains of products where few warps hide one's latency
      float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int p = 0; p < C::kKPieces; ++p) {
        const uint32_t from = ((src + kget) ^ (p & 1) * 64) + (p >> 1) * 128;
        const uint4 x = lds16(from), y = lds16(from + 8 * R);
        if constexpr (!kE4m3) {
          mma<false>(s, x.x, y.x, x.y, y.y, qf[2 * p][0], qf[2 * p][1]);
          mma<false>(kTwo ? s2 : s, x.z, y.z, x.w, y.w, qf[2 * p + 1][0], qf[2 * p + 1][1]);
        } else {
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mma<true>(s, paged::e4m3x2_to_f16x2(xw[e] & 0xffff), paged::e4m3x2_to_f16x2(yw[e] & 0xffff),
                      paged::e4m3x2_to_f16x2(xw[e] >> 16), paged::e4m3x2_to_f16x2(yw[e] >> 16), qf[4 * p + e][0],
                      qf[4 * p + e][1]);
        }
      }
      float f[4] = {qs[0], qs[1], qs[0], qs[1]};  // what makes scores of log2 of the products
      float ve[2] = {0.f, 0.f};                  // exponents of the two positions' values, and kUp
      if constexpr (kE4m3) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int kb = lds1(src + 32 * R + g + 8 * i), vb = lds1(src + 32 * R + 16 + g + 8 * i);
          const float by = __uint_as_float(static_cast<uint32_t>(kb) << 23);
          f[2 * i] *= by;
          f[2 * i + 1] *= by;
          ve[i] = static_cast<float>(vb) + (kUp - 127.f);
        }
      }
      const bool edge = t0 + 16 > cur.len || t0 < cur.lo;
      auto hide = [&](float (&y)[4]) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (t0 + g + 8 * i >= cur.len || t0 + g + 8 * i < cur.lo) y[2 * i] = y[2 * i + 1] = -INFINITY;
      };
      // x: weights over the column's reference; y: those of the products, with the values' exponents.  The reference
      // follows its scores only when one is 2^kAbove above it.
      float x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (kTwo) s[i] += s2[i];
        x[i] = fmaf(s[i], f[i], -ref[i & 1]);
      }
      if (edge) hide(x);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = x[i] + ve[i >> 1];
      bool above = none || fmaxf(fmax3(y[0], y[1], y[2]), y[3]) > kAbove + (kE4m3 ? kUp : 0.f);
      if constexpr (kE4m3) above |= fmaxf(fmax3(x[0], x[1], x[2]), x[3]) > kAbove - kLeast;
      if (__any_sync(0xffffffffu, above)) {
        float z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = s[i] * f[i];
        if (edge) hide(z);
        float raise[2] = {0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const bool first = m[c] == -INFINITY;  // (what there is has no weight)
          const float top = kE4m3 ? fmaxf(z[c] + fmaxf(ve[0] - kUp, kLeast), z[2 + c] + fmaxf(ve[1] - kUp, kLeast)) : fmaxf(z[c], z[2 + c]);
          float mn = fmaxf(m[c], column_max(top)), drop = m[c] - mn;  // (log2) what the values' sum is lowered by
          if constexpr (kE4m3) {
            if (__builtin_expect(far, 0)) {
              const Moved to = far_reference(&stats[kept_at][2 * qd + c], m[c], mn, z[c], z[2 + c], ve[0] - kUp, ve[1] - kUp);
              mn = to.m;
              drop = to.drop;
              raise[c] = to.raise;
            }
          }
          const float by = first ? 0.f : ex2(drop);
          l[c] *= first ? 0.f : ex2(m[c] - mn);
          m[c] = mn;
          ref[c] = mn == -INFINITY ? 0.f : mn;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            x[2 * i + c] = z[2 * i + c] - ref[c];
            y[2 * i + c] = x[2 * i + c] + ve[i];
            if (kE4m3) y[2 * i + c] += raise[c];
          }
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            acc[i][c] *= by;
            acc[i][2 + c] *= by;
          }
        }
        none = far || m[0] == -INFINITY || m[1] == -INFINITY;
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
        for (int i = 0; i < 4; ++i) p[i] = ex2(y[i]);
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

#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], d);
    float over[2] = {0.f, 0.f};  // how far the values' references are above the columns'
    if constexpr (kE4m3) {
      const auto lost = [&](int c) {
        return m[c] > -INFINITY && (l[c] < kSumLeast || l[c] > kSumMost || fabsf(m[c]) > kHuge);
      };
      if (__builtin_expect(far, 0)) {
        __syncwarp();
        over[0] = -stats[kept_at][2 * qd].y;
        over[1] = -stats[kept_at][2 * qd + 1].y;
        far = false;
      } else if (__builtin_expect(team_any<T>(team, lost(0) || lost(1)), 0)) {
        cp_async_wait<0>();
        team_sync<T>(team);
        ld = cur;
        left = count;
        slot = read;
        enter_unit();
#pragma unroll 1
        for (int i = 0; i < kSlots - 1; ++i) load();
        far = true;
        continue;
      }
    }

    // ---- the unit, or its part in this team, ends
    const bool ends = cur.tile + tiles >= cur.end, own = begins;
    const int unit = (cur.b * un.all + cur.u) * T + mem;
    const Heads hd(a, cur.b, cur.r, cur.j, cur.chunk * T + mem);
    const int unit_tiles = cur.tiles();
    const uint32_t stop = at + cur.left();  // where the unit ends on the line
    count -= tiles;
    at += tiles;
    if (T > 1 && count == 0) team_sync<T>(team);
    if (count > 0) {  // the next unit's query is on its way meanwhile
      cur.next_unit(a, un, bad);
      begins = true;
      fetch_q();
    }
    // a thread has the elements d .. d + 7 of two heads, d = first_column(x, g)
    if (own && ends) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int h = 2 * qd + c;
        if (h < hd.n) {
          Finish<kE4m3> f(a, hd, h, m[c], over[c], l[c]);
          if constexpr (kE4m3) f.scale *= kDown;
#pragma unroll
          for (int x = 0; x < D / 64; ++x)
            *reinterpret_cast<uint4*>(a.o + (hd.row + h) * D + first_column<D, kE4m3>(x, g)) =
                make_uint4(pack_bf16x2(f(acc[4 * x][c]), f(acc[4 * x][2 + c])),
                           pack_bf16x2(f(acc[4 * x + 1][c]), f(acc[4 * x + 1][2 + c])),
                           pack_bf16x2(f(acc[4 * x + 2][c]), f(acc[4 * x + 2][2 + c])),
                           pack_bf16x2(f(acc[4 * x + 3][c]), f(acc[4 * x + 3][2 + c])));
          if (g == 0) a.lse[hd.row + h] = f.lse;
        }
      }
    } else {
      // [head][d] in shared memory: of a unit that began earlier in the place kept for it, of one that goes on in the
      // warp's part of the ring, whose last tile has been read
      __syncwarp();
      const int k = 2 * w + own;
      float* to = own ? reinterpret_cast<float*>(smem + w * C::kRing) : kept;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
          float* at8 = to + (2 * qd + c) * D + first_column<D, kE4m3>(x, g);
          reinterpret_cast<float4*>(at8)[0] = make_float4(acc[4 * x][c], acc[4 * x][2 + c], acc[4 * x + 1][c], acc[4 * x + 1][2 + c]);
          reinterpret_cast<float4*>(at8)[1] =
              make_float4(acc[4 * x + 2][c], acc[4 * x + 2][2 + c], acc[4 * x + 3][c], acc[4 * x + 3][2 + c]);
        }
        if (g == 0) {
          if constexpr (kE4m3)
            stats[k][2 * qd + c] = make_float4(m[c], l[c], over[c], 0.f);
          else
            stats[k][2 * qd + c] = make_float2(m[c], l[c]);
        }
      }
      if (lane == 0 && hd.n > 0) parts[k] = Part{unit, own, ends, unit_tiles, stop};
    }
    if (count == 0) break;
  }
}

// A head's partial result in a warp: reference and sum, how far the values' reference is above it (e4m3), and D/32
// elements of each lane.
template <int D, bool kE4m3>
struct Partial {
  static constexpr int E = D / 32;
  using Stat = typename Cfg<D, kE4m3>::Stat;
  float M = -INFINITY, L = 0.f, V = 0.f, o[E] = {};
  __device__ __forceinline__ void add(Stat st, const float* from) {
    const float top = fmaxf(M, st.x), ref = top == -INFINITY ? 0.f : top;
    float f = ex2(M - ref), by = ex2(st.x - ref);
    L = L * f + st.y * by;
    if constexpr (kE4m3) {
      const float mine = M - ref + V, its = st.x - ref + st.z, over = fmaxf(mine, its);
      V = over == -INFINITY ? 0.f : over;
      f = ex2(mine - V);
      by = ex2(its - V);
    }
    M = top;
    float y[E];
    load(from, y);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + y[e] * by;
  }
  __device__ __forceinline__ Stat stat() const {
    if constexpr (kE4m3)
      return make_float4(M, L, V, 0.f);
    else
      return make_float2(M, L);
  }
  static __device__ __forceinline__ void load(const float* from, float (&y)[E]) {
    if constexpr (E == 4) {
      const float4 x = *reinterpret_cast<const float4*>(from);
      y[0] = x.x, y[1] = x.y, y[2] = x.z, y[3] = x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(from);
      y[0] = x.x, y[1] = x.y;
    }
  }
};

template <int D, bool kE4m3, int TM>
__device__ __forceinline__ void write_out(const Args& a, const Units& un, bool teams, int unit, int h,
                                          const Partial<D, kE4m3>& p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, bu = teams ? unit / TM : unit, b = un.by_all.div(bu), u = bu - b * un.all;
  const int rj = un.by_chunks.div(u), r = a.by_hk.div(rj), chunk = u - rj * un.chunks;
  const Heads hd(a, b, r, rj - r * a.pool.hk, teams ? chunk * TM + unit % TM : chunk);
  if (h >= hd.n) return;
  const Finish<kE4m3> f(a, hd, h, p.M, p.V, p.L);
  uint32_t* to = reinterpret_cast<uint32_t*>(a.o + (hd.row + h) * D) + lane * (E / 2);
  if constexpr (E == 4)
    *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(f(p.o[0]), f(p.o[1])), pack_bf16x2(f(p.o[2]), f(p.o[3])));
  else
    *to = pack_bf16x2(f(p.o[0]), f(p.o[1]));
  if (lane == 0) a.lse[hd.row + h] = f.lse;
}

// A ticket: what this CTA's threads wrote before (a barrier lies between) is visible to whoever takes a later one.
__device__ __forceinline__ int take(int32_t* ticket) {
  int t;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(t) : "l"(ticket) : "memory");
  return t;
}

// A CTA's part of a unit that crosses CTAs: it is part i of the n in CTAs first .. first + n - 1.
struct Crossing {
  int unit, first, n, i;  // unit: as a Part's of the team's first warp, -1: none
};

// Part x of a unit that begins in CTA `first`: its place in the workspace.  A CTA has two: the first for a unit that began
// in an earlier CTA, the second for one that begins in it.
__device__ __forceinline__ int64_t place_of(int first, int x) { return 2 * (first + x) + (x == 0); }

template <int D, bool kE4m3>
__device__ __forceinline__ void leave(const Args& a, int T, int first, int x, int mem, int h, const Partial<D, kE4m3>& p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t row = (place_of(first, x) * T + mem) * kHeads + h;
  float* to = a.parts + row * D + lane * E;
  if constexpr (E == 4)
    __stcg(reinterpret_cast<float4*>(to), make_float4(p.o[0], p.o[1], p.o[2], p.o[3]));
  else
    __stcg(reinterpret_cast<float2*>(to), make_float2(p.o[0], p.o[1]));
  if (lane == 0) __stcg(static_cast<typename Cfg<D, kE4m3>::Stat*>(a.stats) + row, p.stat());
}

// The units that cross CTAs, in the CTAs that come last: every CTA leaves its part in the workspace and takes a ticket; of
// kFan parts in a row the last CTA puts them together, and of these sums again the last one.  The
// order of the additions goes by the positions, whoever is last.  (All of this runs once: it is kept
// short, for its instructions come from L2.)
template <int D, bool kE4m3, int TM>
__device__ __forceinline__ void join(const Args& a, const Units& un, bool teams, unsigned char* smem, const Crossing* crossing) {
  using C = Cfg<D, kE4m3>;
  __shared__ int last[2];
  using Stat = typename C::Stat;
  Stat* stats = reinterpret_cast<Stat*>(smem + kFan * C::kKept);  // [part][head], behind the parts
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, T = teams ? TM : 1;
  __syncthreads();  // the CTA's parts are written
  if (tid < 2) {
    int is_last = 0;
    if (crossing[tid].unit >= 0) {
      const int x0 = crossing[tid].i / kFan * kFan, x1 = min(crossing[tid].n, x0 + kFan);
      // tickets of the CTA that has a group's first part: [0] of a unit that began earlier, [1] of one that begins there,
      // [2] of the groups of that one.  The last to come leaves 0.
      int32_t* ticket = a.tickets + 3 * (crossing[tid].first + x0) + (x0 == 0);
      is_last = take(ticket) == x1 - x0 - 1;
      if (is_last) *ticket = 0;
    }
    last[tid] = is_last;
  }
  __syncthreads();
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    const int n = crossing[c].n, first = crossing[c].first, groups = (n + kFan - 1) / kFan;
    int x0 = crossing[c].i / kFan * kFan, step = 1, parts = min(n - x0, kFan);
    while (last[c]) {
      const bool done = step > 1 || groups == 1;
#pragma unroll 1
      for (int m = 0; m < T; ++m) {  // the team's warps
        // parts x0, x0 + step, ... into shared memory, past L1 (other CTAs wrote them)
        constexpr int kPieces = kHeads * D / 4;
        for (int i = tid; i < parts * kPieces; i += C::kThreads) {
          const int p = i / kPieces;
          cp_async(smem_u32(smem) + i * 16,
                   a.parts + ((place_of(first, x0 + p * step) * T + m) * kPieces + (i - p * kPieces)) * 4);
        }
        cp_async_commit();
        for (int i = tid; i < parts * kHeads; i += C::kThreads)
          stats[i] = __ldcg(static_cast<const Stat*>(a.stats) +
                            (place_of(first, x0 + i / kHeads * step) * T + m) * kHeads + i % kHeads);
        cp_async_wait<0>();
        __syncthreads();
        if (w < kHeads) {
          Partial<D, kE4m3> sum;
          for (int p = 0; p < parts; ++p)
            sum.add(stats[p * kHeads + w], reinterpret_cast<const float*>(smem) + (p * kHeads + w) * D + lane * (D / 32));
          if (done)
            write_out<D, kE4m3, TM>(a, un, teams, crossing[c].unit + m, w, sum);
          else
            leave<D, kE4m3>(a, T, first, x0, m, w, sum);
        }
        __syncthreads();
      }
      if (done) break;
      if (tid == 0) {
        int32_t* ticket = a.tickets + 3 * first + 2;
        last[c] = take(ticket) == groups - 1;
        if (last[c]) *ticket = 0;
      }
      __syncthreads();
      x0 = 0;
      step = kFan;
      parts = groups;
    }
  }
}

template <int D, bool kE4m3, int TM>
__global__ void __launch_bounds__(Cfg<D, kE4m3>::kThreads, 1) decode_kernel(Args a) {
  using C = Cfg<D, kE4m3>;
  constexpr int kWarps = C::kWarps;
  static_assert(TM <= 2 && kWarps % TM == 0, "one warp of a team copies the keys, the other the values");
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Part parts[2 * kWarps];
  __shared__ uint32_t team_tiles[kWarps / TM][2];  // what a team goes by: of its units, of the one at hand
  __shared__ typename C::Stat stats[2 * kWarps][kHeads];
  __shared__ Crossing crossing[2];              // of a unit that began in an earlier CTA, of one that begins here
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  if (lane < 2) parts[2 * w + lane].unit = -1;
  if (tid < 2) crossing[tid].unit = -1;
  grid_wait();

  // ---- the line, in each warp: a lane adds up n_seqs / 32 sequences' tiles, and how many have any
  constexpr uint32_t kMost = 1u << 26;  // of a lane (a table's row has less)
  const int per = (a.n_seqs + 31) / 32, s0 = min(a.n_seqs, lane * per), s1 = min(a.n_seqs, s0 + per);
  uint32_t mine = 0, mine_any = 0, most = 0;
  bool bad = false;
#pragma unroll 4
  for (int s = s0; s < s1; ++s) {
    const uint32_t n = tiles_of(a, s, bad);
    mine = min(mine + n, kMost + 1);
    mine_any += n > 0;
    most = max(most, n);
  }
  if (bad) set_status(a.status, USP_ERR_BAD_PAGES);
  uint32_t before = mine, before_any = mine_any;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, before, d), y = __shfl_up_sync(0xffffffffu, before_any, d);
    if (lane >= d) {
      before += x;
      before_any += y;
    }
  }
  uint32_t all = __shfl_sync(0xffffffffu, before, 31), any = __shfl_sync(0xffffffffu, before_any, 31);
  most = __reduce_max_sync(0xffffffffu, most);
  bool over = __any_sync(0xffffffffu, mine > kMost);
  if constexpr (TM > 1) {  // warps that wait for each other go by one reading of the lengths
    __shared__ uint4 line_of;
    if (tid == 0) line_of = make_uint4(all, any, most, over);
    __syncthreads();
    all = line_of.x, any = line_of.y, most = line_of.z, over = line_of.w;
  }
  const bool teams =
      TM > 1 && static_cast<uint64_t>(all) * a.team.all >= static_cast<uint64_t>(kTeamTiles) * gridDim.x * (kWarps / TM);
  const Units& un = teams ? a.team : a.one;
  const int T = teams ? TM : 1;
  const uint32_t n_teams = teams ? kWarps / TM : kWarps;  // of a CTA
  const uint64_t tiles = static_cast<uint64_t>(all) * un.all;
  if (over || tiles >= (1ull << 31)) {
    set_status(a.status, USP_ERR_UNSUPPORTED);
    return;
  }
  // The longest share of a team, in tiles: of whole units dealt out to the teams (nothing is to be joined then), to
  // the CTAs (nothing across them), of tiles.
  const uint32_t W = static_cast<uint32_t>(tiles), U = any * un.all, grid_teams = gridDim.x * n_teams;
  const uint32_t even = (W + grid_teams - 1) / grid_teams;
  const uint64_t to_team = static_cast<uint64_t>((U + grid_teams - 1) / grid_teams) * most;
  const uint64_t to_cta = (static_cast<uint64_t>((U + gridDim.x - 1) / gridDim.x) * most + n_teams - 1) / n_teams;
  const Split split = to_team <= min(to_cta + kWarpsTiles, static_cast<uint64_t>(even) + kCtasTiles) ? Split::kUnitsToTeams
                      : to_cta + kWarpsTiles <= even + kCtasTiles                                     ? Split::kUnitsToCtas
                                                                                                      : Split::kTiles;
  const bool by_unit = split != Split::kTiles;
  const uint32_t things = by_unit ? U : W, takers = split == Split::kUnitsToCtas ? 1 : n_teams;  // of a CTA
  const uint32_t n_ctas = min(gridDim.x, (things + takers - 1) / takers);
  // sequences that see nothing have no tile: CTAs without work write their outputs, or all when they are done
  if (cta >= n_ctas) {
    if (any < a.n_seqs) write_empty<D>(a, (cta - n_ctas) * kWarps + w, (gridDim.x - n_ctas) * kWarps);
    return;
  }
  const Deal line(things, n_ctas * takers);
  const uint32_t taker = cta * takers + (takers > 1 ? (teams ? w / TM : w) : 0);
  const uint32_t at = line.begin(taker), count = line.begin(taker + 1) - at;
  if (count > 0) {
    const uint32_t hi = (by_unit ? before_any : before) * un.all, lo = hi - (by_unit ? mine_any : mine) * un.all;
    const bool here = at >= lo && at < hi;
    int s = s0;
    uint32_t rest = at - lo;
    while (here && s + 1 < s1) {
      const uint32_t n = tiles_of(a, s, bad), things_of = (by_unit ? n > 0 : n) * un.all;
      if (rest < things_of) break;
      rest -= things_of;
      ++s;
    }
    const int from = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    const int2 start = make_int2(min(__shfl_sync(0xffffffffu, s, from & 31), a.n_seqs - 1),
                                 __shfl_sync(0xffffffffu, rest, from & 31));
    if (teams)
      run_stretch<D, kE4m3, TM>(a, smem, parts, stats, team_tiles[w / TM], start, split, at, count);
    else
      run_stretch<D, kE4m3, 1>(a, smem, parts, stats, nullptr, start, split, at, count);
  }
  if (any < a.n_seqs && n_ctas == gridDim.x) write_empty<D>(a, cta * kWarps + w, gridDim.x * kWarps);
  if (split == Split::kUnitsToTeams) return;

  // ---- the warps' parts, in order: those of one unit next to each other, a team's first warps' before its second ones'
  __syncthreads();
  const auto part_of = [&](int i) {
    constexpr int n = kWarps / TM;
    return teams ? 2 * ((i >> 1) % n * TM + i / (2 * n)) + (i & 1) : i;
  };
  // a lane's part: which there are, and which begin another unit than the one before
  const int unit_k = lane < 2 * kWarps ? parts[part_of(lane)].unit : -1;
  const uint32_t there = __ballot_sync(0xffffffffu, unit_k >= 0), below = there & ((1u << lane) - 1);
  const int unit_before = __shfl_sync(0xffffffffu, unit_k, below ? 31 - __clz(below) : 0);
  uint32_t starters = __ballot_sync(0xffffffffu, unit_k >= 0 && (below == 0 || unit_before != unit_k));
  // a warp for each head of a unit, the warps in turn
  for (int h = w; starters != 0; h += h < kHeads ? kWarps - kHeads : -kHeads) {
    const int i = __ffs(starters) - 1;
    starters &= starters - 1;
    uint32_t members = there & ~((1u << i) - 1) & (starters ? (starters & -starters) - 1 : 0xffffffffu);
    if (h >= kHeads) continue;
    const int unit = parts[part_of(i)].unit;
    Partial<D, kE4m3> sum;
    int last = part_of(i);
    for (; members != 0; members &= members - 1) {
      last = part_of(__ffs(members) - 1);
      sum.add(stats[last][h],
              reinterpret_cast<const float*>(smem + (last & 1 ? last / 2 * C::kRing : kWarps * C::kRing + last / 2 * C::kKept)) +
                  h * D + lane * (D / 32));
    }
    if constexpr (kE4m3) {
#pragma unroll
      for (int e = 0; e < D / 32; ++e) sum.o[e] *= kDown;
    }
    const bool begins = parts[part_of(i)].begins;
    if (begins && parts[last].ends) {
      write_out<D, kE4m3, TM>(a, un, teams, unit, h, sum);
    } else {
      const uint32_t stop = parts[last].stop;
      // (n_ctas and the bounds hold whatever the lengths have become meanwhile)
      const uint32_t me = cta, first_of = line.owner(stop - parts[last].tiles) / n_teams, last_of = line.owner(stop - 1) / n_teams;
      const int first = begins ? cta : static_cast<int>(min(first_of, me));
      const int end = static_cast<int>(min(max(last_of, me), n_ctas - 1)) + 1;
      const int mem = teams ? unit % TM : 0;
      leave<D, kE4m3>(a, T, first, cta - first, mem, h, sum);
      if (h == 0 && lane == 0 && mem == 0) crossing[begins] = Crossing{unit, first, end - first, cta - first};
    }
  }
  if (split == Split::kTiles) join<D, kE4m3, TM>(a, un, teams, smem, crossing);
}

template <int D, bool kE4m3, int TM>
int launch(const Args& a, int ctas, cudaStream_t st) {
  auto* kern = decode_kernel<D, kE4m3, TM>;
  constexpr int smem = Cfg<D, kE4m3>::kSmem;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
    cudaGetLastError();
    return USP_ERR_CUDA;
  }
  return launch_chained(kern, dim3(ctas), Cfg<D, kE4m3>::kThreads, smem, 1, st, a);
}

template <int D, bool kE4m3>
int launch_team(const Args& a, int warps, int ctas, cudaStream_t st) {
  if constexpr (Cfg<D, kE4m3>::kRow >= 128) {
    if (warps == 2) return launch<D, kE4m3, 2>(a, ctas, st);
  }
  return launch<D, kE4m3, 1>(a, ctas, st);
}

int grid_of() { return std::min(kMaxCtas, device_sm_count()); }

// Warps of a team, 8 query heads each (see kTeamTiles).
int team_of(const usp_paged_cache& c, int Hq) {
  const int G = Hq / std::max(c.P, c.Hkv), row = c.D * (c.dtype == USP_CACHE_E4M3 ? 1 : 2);
  return G <= kHeads || row < 128 ? 1 : 2;
}

}  // namespace decode

// Tickets (of kMaxCtas, so that they lie at the same place for every cache), then parts, then statistics.
size_t attn_decode_ws_bytes(const usp_paged_cache& c, int Hq) {
  const size_t ctas = decode::grid_of(), rows = 2 * ctas * decode::team_of(c, Hq) * decode::kHeads;
  return decode::kTicketBytes + rows * c.D * 4 + rows * (c.dtype == USP_CACHE_E4M3 ? sizeof(float4) : sizeof(float2));
}

int launch_attn_decode(const usp_paged_cache& c, int Hq, int window_left, float scale, const float* sinks,
                       const void* q, void* o, float* lse, void* ws, int32_t* status, cudaStream_t st) {
  decode::Args a{};
  a.pool = paged::Pool(c);
  a.n_seqs = c.n_seqs;
  a.P = c.P;
  a.hq = Hq / c.P;
  a.G = a.hq / a.pool.hk;
  const int team = decode::team_of(c, Hq);
  for (auto [un, heads] : {std::pair(&a.one, decode::kHeads), std::pair(&a.team, team * decode::kHeads)}) {
    un->chunks = (a.G + heads - 1) / heads;
    un->all = c.P * a.pool.hk * un->chunks;
    un->by_all = FastDiv(static_cast<uint32_t>(un->all));
    un->by_chunks = FastDiv(static_cast<uint32_t>(un->chunks));
  }
  a.by_hk = FastDiv(static_cast<uint32_t>(a.pool.hk));
  a.window = window_left;
  a.scale = scale;
  a.sinks = sinks;
  a.q = static_cast<const uint16_t*>(q);
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  a.status = status;
  const int ctas = decode::grid_of();
  const size_t rows = 2 * static_cast<size_t>(ctas) * team * decode::kHeads;
  a.tickets = static_cast<int32_t*>(ws);
  a.parts = reinterpret_cast<float*>(static_cast<char*>(ws) + decode::kTicketBytes);
  a.stats = a.parts + rows * c.D;
  const bool e = c.dtype == USP_CACHE_E4M3;
  if (c.D == 64) return e ? decode::launch_team<64, true>(a, team, ctas, st) : decode::launch_team<64, false>(a, team, ctas, st);
  return e ? decode::launch_team<128, true>(a, team, ctas, st) : decode::launch_team<128, false>(a, team, ctas, st);
}

}  // namespace usp
