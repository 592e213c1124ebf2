// usp_attn_fwd.cuh — varlen causal GQA attention forward on the 5th-generation
// tensor core (tcgen05), one launch for all P emulated ranks.
//
// What it computes (huggingface/accelerate PR #4209: attention runs on the
// gathered sequence of the rank's heads; each head has a single sink logit,
// taken from the slice of the rank's heads; sliding windows and packing keep
// working): for every
// rank r, local query head j, token t,
//     LSE_t = ln( sum_{u visible} exp(scale q_t.k_u) + exp(z_{r*hq+j}) )
//     O_t   = sum_{u visible} exp(scale q_t.k_u - LSE_t) v_u
//
// CTA = one (rank, query head, block of 128*NQT query rows) = NQT 128-row Q
// tiles that share every K/V tile.  Warp roles (NQT = 2: 320 threads):
//   warps 0-3   softmax for Q tile 0 (thread = query row = TMEM lane)
//   warps 4-7   softmax for Q tile 1 (NQT = 2)
//   warp  4NQT  TMA producer: Q tiles once, then a ring of K/V stages
//   warp  4NQT+1 MMA issuer (one thread): S_q = Q_q K^T into TMEM, then
//               O_q += P_q V with P_q read from TMEM (bf16, written over S_q)
// TMEM: S_q [128q, 128q+128), O_q [128NQT + qD, 128NQT + (q+1)D) (512 columns
// for NQT = 2).  With two tiles the MMA thread alternates them (PV_0, S_0
// next, PV_1, S_1 next), so the tensor core works on one tile while the other
// tile's softmax runs; with one tile (short windows at D = 64; with modified
// scores where there are few tiles) at D = 64 two CTAs share an SM and overlap
// instead.
//
// Online softmax in the log2 domain with a lazy rescale: the running max only
// moves when a row's new max exceeds it by more than 8 (a factor 256), and the
// O row in TMEM is rescaled then.  Because S_q[n] is committed after
// PV_q[n-1], waiting for S_q[n] also guarantees PV_q[n-1] has finished, so the
// softmax threads may rescale O without another barrier.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "usp_attn_common.cuh"
#include "usp_attn_mods.cuh"
#include "usp_internal.h"

namespace usp {

namespace fwd {

constexpr int kAtomBytes = kBM * 128;  // one 64-column (128-byte) swizzle column of a 128-row tile
// Stage-release barriers in flight: more than the K/V stages, so that the
// producer's waits (at most ST - 1 releases behind the MMA thread) never see
// a barrier two phases ahead.
constexpr int kRel = 8;

// NQT Q tiles per CTA: 2 (two softmax warpgroups that alternate on the tensor
// core, 512 TMEM columns, one CTA per SM) or 1 (one softmax warpgroup; at
// D = 64 its 192 TMEM columns and 82 KB of shared memory let two CTAs share
// an SM, which then overlap each other's latencies).
// NH softmax warpgroups per Q tile: 1 (a thread takes a whole row) or, with
// modified scores, 2 (a thread takes half of a row's keys; the halves meet in the
// row's maximum and sum through shared memory).
template <int D, int NQT, int NH = 1>
struct Cfg {
  static constexpr int THREADS = 128 * NQT * NH + 64;  // softmax warpgroups, producer warp, MMA warp
  static constexpr int WP = 4 * NQT * NH;              // producer warp (the MMA warp is WP + 1)
  static constexpr int CTAS = (NQT == 1 && D == 64) ? 2 : 1;  // CTAs per SM
  static constexpr uint32_t TCOLS = NQT == 2 ? 512 : 256;     // TMEM columns allocated
  static constexpr int NCH = D / 64;                  // 64-wide column atoms per row
  static constexpr int ST = (D == 128 || NQT == 1) ? 2 : 4;  // K/V pipeline stages
  static constexpr bool KV_ONE = ST >= 4;             // one barrier for a stage's K and V
  static constexpr int TILE = NCH * kAtomBytes;       // bytes of one 128-row tile
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + NQT * TILE;
  static constexpr int OFF_V = OFF_K + ST * TILE;
  static constexpr int OFF_BAR = OFF_V + ST * TILE;
  static constexpr int XBYTES = NH == 2 ? 2 * NQT * 2 * kBM * 4 : 0;  // [2 buffers][tile][half][row] floats
  static constexpr int OFF_RAMP = OFF_BAR + 512;      // Mods: slope times column (128 floats)
  static constexpr int OFF_X = OFF_BAR + 1024;        // NH = 2: what the halves of a row exchange
  static constexpr int OFF_TAB = OFF_X + XBYTES;      // Mods: the head's bias row by distance (SMEM grows by it)
  static constexpr int SMEM = OFF_BAR + 1024 + XBYTES + 1024;  // barriers, exchange, alignment slack
  static constexpr uint32_t T_O = 128 * NQT;          // first O column (S_q at 128q)
};

struct Bars {
  uint64_t q_full[2];
  uint64_t s_full[2];
  uint64_t p_full[2];
  uint64_t o_final[2];
  uint64_t mma_done;
  uint64_t x_full[2][4];  // NH = 2: both halves of 32 rows of the tile have written their exchange values
  // Four stages (KV_ONE): kv_full[s] = K and V of the tile in stage s
  // landed (V has time to land before S, so PV needs no wait of its own).
  // Two stages: K_0 signals k_first, and kv_full[m % 2] = V_m and K_{m+1}
  // landed (both are loaded once release m-1 completes, and one wait before
  // PV_m covers them).
  uint64_t kv_full[4], k_first;
  // rel[j % kRel] completes once the MMAs issued up to S_j are done: K_j's
  // stage and V_{j-1}'s (its PV was issued before S_j) are free
  uint64_t rel[8];
  uint32_t tmem;
  int abort;
};

static_assert(sizeof(Bars) <= 512, "barrier block");

struct Out {
  __nv_bfloat16* o;
  float* lse;
  int nqb;  // query blocks (NQT tiles of 128 rows) per (rank, head)
};

// Halves of a row's keys (see Cfg) where there are tiles enough for CTAs of two.  A cap lengthens a row's chain from S to P, and 8
// softmax warps do not hide it (8192 packed tokens, D = 128: 214 us with whole rows,
// 192 with halves).  Without one the exchange of the row's maximum costs more than
// the shorter chain gains (prefix 123 and 127 us, slopes 211 and 219).
template <class M>
constexpr int kHalves = 1;
template <bool BIAS>
constexpr int kHalves<Mods<true, BIAS>> = 2;

template <int D, int NQT, int NH, class M>
__global__ void __launch_bounds__(Cfg<D, NQT, NH>::THREADS, Cfg<D, NQT>::CTAS)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                    const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap to, AttnArgs p, Out out,
                    M mods) {
  constexpr int NC = kBN / NH;  // columns of a thread
  using C = Cfg<D, NQT, NH>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + C::OFF_BAR);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // ---- work unit: late query blocks first (they see the most keys); the
  // query heads of one key/value head are adjacent, so they share K/V in L2.
  const int per_blk = p.P * p.hq;
  const int qb = out.nqb - 1 - static_cast<int>(blockIdx.x) / per_blk;
  const int rem = static_cast<int>(blockIdx.x) % per_blk;
  const int r = rem / p.hq, j = rem % p.hq;
  const HeadRef qh = q_head_ref(p, r, j), kvh = kv_head_ref(p, r, j / p.G);
  const int t0 = qb * NQT * kBM;

  bool tile_ok[NQT];
  for (int q = 0; q < NQT; ++q) tile_ok[q] = t0 + q * kBM < p.BS;
  volatile int* abort = &bars->abort;
  auto init_bars = [&] {
    for (int q = 0; q < NQT; ++q) {
      mbar_init(&bars->q_full[q], 1);
      mbar_init(&bars->s_full[q], 1);
      mbar_init(&bars->p_full[q], 4 * NH);
      for (int w = 0; w < 4; ++w) mbar_init(&bars->x_full[q][w], NH);
      mbar_init(&bars->o_final[q], 1);
    }
    mbar_init(&bars->mma_done, 1);
    for (int j = 0; j < kRel; ++j) mbar_init(&bars->rel[j], 1);
    mbar_init(&bars->k_first, 1);
    for (int s = 0; s < C::ST; ++s) mbar_init(&bars->kv_full[s], 1);
    bars->abort = 0;
    fence_barrier_init();
  };
  auto load_q = [&] {
    prefetch_tmap(&tq);
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
    for (int q = 0; q < NQT; ++q) {
      if (!tile_ok[q]) continue;
      mbar_arrive_expect_tx(&bars->q_full[q], C::TILE);
      for (int c = 0; c < C::NCH; ++c)
        tma_load_rows(smem + C::OFF_Q + q * C::TILE + c * kAtomBytes, &tq, &bars->q_full[q], p, c, qh, t0 + q * kBM);
    }
  };
  // Mods: Q, which waits for nothing, is on its way before the documents are looked
  // up, and the first K before the CTA has its TMEM; by the producer itself.
  const bool is_producer = warp == C::WP && lane == 0;
  if constexpr (M::on) {
    if (is_producer) init_bars();
    grid_wait();
    if (is_producer) {
      load_q();
    }
  }
  auto leave_early = [&] {  // never with copies still landing
    if constexpr (M::on) {
      if (is_producer)
        for (int q = 0; q < NQT; ++q)
          if (tile_ok[q]) mbar_wait(&bars->q_full[q], 0, abort, p.status);
    }
  };

  int n_docs, lo = 0x7FFFFFFF, hi = 0;
  [[maybe_unused]] TileDocs docs;
  if constexpr (M::on) {
    const int last = min(t0 + NQT * kBM, p.BS) - 1;
    if (!checked_tile_docs(p, mods, t0, last, n_docs, docs)) {
      leave_early();
      return;
    }
    key_range(p, mods, docs, t0, last, lo, hi);
  } else {
    n_docs = checked_docs(p);
    if (n_docs == 0) return;
    for (int q = 0; q < NQT; ++q) {
      int first = t0 + q * kBM;
      if (tile_ok[q]) {
        int last = min(first + kBM, p.BS) - 1, l0, h0;
        key_range(p, n_docs, first, last, l0, h0);
        lo = min(lo, l0);
        hi = max(hi, h0);
      }
    }
  }
  // Ring x Ulysses step: only the key/value super-chunk held at this step (the
  // CTA's rows lie in one super-chunk).
  int rk0 = 0, rk1 = 0x7FFFFFFF;
  if (p.ring > 1) {
    ring_key_window(p, t0, rk0, rk1);
    lo = max(lo, rk0);
    hi = min(hi, rk1);
  }
  // With k/v read from the sequence shards, key tiles are aligned to 128
  // tokens so that a tile never straddles a shard (keys before the document
  // are masked).
  if (p.kv_seq_io) lo &= ~(kBN - 1);
  const int n_kv = hi > lo ? (hi - lo + kBN - 1) / kBN : 0;
  if (n_kv == 0) {
    // no key to see (a ring step whose block lies after these rows): O = 0 and
    // LSE = the sink logit alone, or -inf
    if (warp < C::WP) {
      const int q = (warp >> 2) / NH, t = t0 + q * kBM + (tid & 127);
      if (tile_ok[q] && t < p.BS && (warp >> 2) % NH == 0) {
        uint4* dst = reinterpret_cast<uint4*>(out.o + row_offset(p, qh, p.hq, p.Hq, t, D));
        for (int e = 0; e < D / 8; ++e) dst[e] = make_uint4(0, 0, 0, 0);
        const int bb = t / p.S, ss = t - bb * p.S;
        out.lse[(static_cast<size_t>(r * p.B + bb) * p.hq + j) * p.S + ss] =
            p.sinks != nullptr ? gld(p.sinks + r * p.hq + j) : -INFINITY;
      }
    }
    leave_early();
    return;
  }

  auto load = [&](int kv, int n, uint64_t* full) {  // K (kv 0) or V tile n into its stage
    uint8_t* dst = smem + (kv == 0 ? C::OFF_K : C::OFF_V) + (n % C::ST) * C::TILE;
    for (int c = 0; c < C::NCH; ++c)
      tma_load_rows(dst + c * kAtomBytes, kv == 0 ? &tk : &tv, full, p, c, kvh, lo + n * kBN, p.kv_seq_io != 0);
  };
  auto load_first = [&] {
    if constexpr (C::KV_ONE) {
      mbar_arrive_expect_tx(&bars->kv_full[0], 2 * C::TILE);
      load(0, 0, &bars->kv_full[0]);
      load(1, 0, &bars->kv_full[0]);
    } else {
      mbar_arrive_expect_tx(&bars->k_first, C::TILE);
      load(0, 0, &bars->k_first);
    }
  };
  if constexpr (M::on) {
    if (is_producer) load_first();
  } else if (tid == 0) {
    init_bars();
  }
  if constexpr (M::on) {
    if (bias_on<M> && mods.slopes != nullptr && tid < kBN)
      reinterpret_cast<float*>(smem + C::OFF_RAMP)[tid] =
          checked_slope(mods, r * p.hq + j, p.status) * kLog2E * static_cast<float>(tid);
    if (bias_on<M> && mods.rel_bias != nullptr)
      for (int e = tid; e < tab_len(mods.R); e += C::THREADS)
        reinterpret_cast<float*>(smem + C::OFF_TAB)[e] = table_entry(mods, r * p.hq + j, e, p.status);
  }
  if (warp == 0) {
    tmem_alloc(&bars->tmem, C::TCOLS);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  const uint32_t sbase = smem_u32(smem);

  if (warp == C::WP) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      if constexpr (!M::on) {
        load_q();
        load_first();
      }
      int issued = 0;  // KV_ONE: tiles whose K and V loads were issued; else V_m (with K_{m+1}) groups
      if constexpr (C::KV_ONE) {
        // K_n and V_n once their stage is free: K_n replaces K_{n-ST} (free
        // after release n-ST), V_n replaces V_{n-ST} (release n-ST+1)
        issued = 1;
        for (int n = 1; n < n_kv; ++n) {
          const int st = n % C::ST;
          bool ok_n = true;
          for (int kv = 0; kv < 2 && ok_n; ++kv) {
            const int j = n - C::ST + kv;  // the release this load waits for
            if (n >= C::ST && !(ok_n = mbar_wait(&bars->rel[j % kRel], (j / kRel) & 1, abort, p.status))) break;
            if (kv == 0) mbar_arrive_expect_tx(&bars->kv_full[st], 2 * C::TILE);
            load(kv, n, &bars->kv_full[st]);
          }
          if (!ok_n) break;
          issued = n + 1;
        }
        for (int n = max(0, issued - C::ST); n < issued; ++n)
          mbar_wait(&bars->kv_full[n % C::ST], (n / C::ST) & 1, abort, p.status);
      } else {
        // K_0 alone; then V_m with K_{m+1}: V_m replaces V_{m-2} (free after
        // PV_{m-2}), K_{m+1} replaces K_{m-1} (free after S_{m-1}), both by
        // release m-1
        for (int m = 0; m < n_kv; ++m) {
          if (m >= 1 && !mbar_wait(&bars->rel[(m - 1) % kRel], ((m - 1) / kRel) & 1, abort, p.status)) break;
          const bool k_next = m + 1 < n_kv;
          uint64_t* full = &bars->kv_full[m & 1];
          mbar_arrive_expect_tx(full, (k_next ? 2 : 1) * C::TILE);
          load(1, m, full);
          if (k_next) load(0, m + 1, full);
          issued = m + 1;
        }
        mbar_wait(&bars->k_first, 0, abort, p.status);
        for (int m = max(0, issued - 2); m < issued; ++m)
          mbar_wait(&bars->kv_full[m & 1], (m >> 1) & 1, abort, p.status);
      }
      // Never leave the CTA with copies still landing in its shared memory (above).
      for (int q = 0; q < NQT; ++q)
        if (tile_ok[q]) mbar_wait(&bars->q_full[q], 0, abort, p.status);
    }
  } else if (warp == C::WP + 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_s = idesc_bf16(kBM, kBN, false, false);
      constexpr uint32_t idesc_o = idesc_bf16(kBM, D, false, true);
      bool ok = true;
      for (int q = 0; q < NQT && ok; ++q)
        if (tile_ok[q]) ok = mbar_wait(&bars->q_full[q], 0, abort, p.status);
      // descriptors are built once per tile and moved by a constant per MMA step
      auto issue_s = [&](int q, int st) {
        const uint64_t qd = sdesc_sw128(sbase + C::OFF_Q + q * C::TILE, 16, 1024);
        const uint64_t kd = sdesc_sw128(sbase + C::OFF_K + st * C::TILE, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * kAtomBytes + (kk & 3) * 32;
          mma_ss(tmem + q * kBN, sdesc_add(qd, off), sdesc_add(kd, off), idesc_s, kk > 0);
        }
      };
      // Release j (after S_j): one commit frees K_j and V_{j-1}; only the
      // releases a later load waits for are committed (j - 1 + ST < n_kv).
      auto release = [&](int j) {
        if (j - 1 + C::ST < n_kv) mma_commit(&bars->rel[j % kRel]);
      };
      auto issue_pv = [&](int q, int st, bool acc) {
        const uint64_t vd = sdesc_sw128(sbase + C::OFF_V + st * C::TILE, kAtomBytes, 1024);
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk)  // P of half h sits in columns NC h .. NC h + NC / 2
          mma_ts(tmem + C::T_O + q * D, tmem + q * kBN + kk / (8 / NH) * NC + kk % (8 / NH) * 8,
                 sdesc_add(vd, kk * 16 * 128), idesc_o,
                 (acc || kk > 0) ? 1u : 0u);
      };
      if (ok) ok = C::KV_ONE ? mbar_wait(&bars->kv_full[0], 0, abort, p.status)
                             : mbar_wait(&bars->k_first, 0, abort, p.status);
      if (ok) {
        tc_fence_after();
        for (int q = 0; q < NQT; ++q)
          if (tile_ok[q]) {
            issue_s(q, 0);
            mma_commit(&bars->s_full[q]);
          }
        release(0);
      }
      for (int n = 0; n < n_kv && ok; ++n) {
        const int st = n % C::ST;
        // two stages: V_n and K_{n+1} in one wait; KV_ONE: V_n landed with K_n
        if (!C::KV_ONE && !(ok = mbar_wait(&bars->kv_full[n & 1], (n >> 1) & 1, abort, p.status))) break;
        bool next_k_ready = !C::KV_ONE;
        for (int q = 0; q < NQT && ok; ++q) {
          if (!tile_ok[q]) continue;
          if (!(ok = mbar_wait(&bars->p_full[q], n & 1, abort, p.status))) break;
          tc_fence_after();
          issue_pv(q, st, n > 0);
          if (n + 1 < n_kv) {
            if (!next_k_ready) {
              const int st1 = (n + 1) % C::ST;
              if (!(ok = mbar_wait(&bars->kv_full[st1], ((n + 1) / C::ST) & 1, abort, p.status))) break;
              tc_fence_after();
              next_k_ready = true;
            }
            issue_s(q, (n + 1) % C::ST);
            mma_commit(&bars->s_full[q]);
          } else {
            mma_commit(&bars->o_final[q]);
          }
        }
        if (ok && n + 1 < n_kv) release(n + 1);
      }
      // Every MMA issued above has finished before TMEM can be released.
      mma_commit(&bars->mma_done);
      mbar_wait(&bars->mma_done, 0, abort, p.status);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int q = (warp >> 2) / NH;     // which Q tile
    const int half = (warp >> 2) % NH;  // which half of a row's keys
    const int row = tid & 127;          // TMEM lane = row of the tile
    const int t = t0 + q * kBM + row;   // rank-local token
    const bool row_ok = t < p.BS;
    const uint32_t lane_base = tmem + ((static_cast<uint32_t>(warp & 3) * 32) << 16);
    const uint32_t s_tm = lane_base + q * kBN;
    const uint32_t o_tm = lane_base + C::T_O + q * D;
    int a = 0, b = 0, pe = 0;
    if constexpr (M::on) {
      if (row_ok) doc_bounds(p, mods, docs, t, a, b, pe);
    } else {
      if (row_ok) doc_bounds(p, mods, n_docs, t, a, b, pe);
    }
    a = max(a, rk0);  // a ring step sees one key/value super-chunk
    b = min(b, rk1);
    const int gh = r * p.hq + j;  // global query head: the sink slice of this rank
    float m = -INFINITY, l = 0.f;
    if (p.sinks != nullptr) {
      m = gld(p.sinks + gh) * 1.4426950408889634f;
      l = half == 0 ? 1.f : 0.f;  // the sink counts once
    }
    // Mods: the row's visible keys, its bias row and slope, and whether the cap bounds
    // the scores tightly enough to leave the softmax's reference where the row's first
    // tile with keys (`starts`) put it: at that tile's maximum, so that P is exact where
    // one key is all that a row sees (any other reference leaves P's rounding to bf16 in
    // O alone, and with it in D against dP), and at most kFixedRefCap2 below the cap.
    [[maybe_unused]] int mvlo = 1, mvhi = 0;
    [[maybe_unused]] bool fixed_ref = false;
    [[maybe_unused]] auto starts = [&](int n) {
      return static_cast<uint32_t>(mvlo - (lo + n * kBN)) < static_cast<uint32_t>(kBN);
    };
    [[maybe_unused]] auto floored = [&](float ref) {
      if constexpr (M::on) ref = fmaxf(ref, mods.cap * kLog2E - kFixedRefCap2);
      return ref;
    };
    [[maybe_unused]] float slope2 = 0.f;
    [[maybe_unused]] const float* tab = nullptr;
    [[maybe_unused]] const float* ramp = reinterpret_cast<const float*>(smem + C::OFF_RAMP);
    if constexpr (M::on) {
      visible_keys(mods, t, a, b, pe, p.causal, p.window_left, row_ok, mvlo, mvhi);
      if (bias_on<M> && mods.slopes != nullptr) slope2 = gld(mods.slopes + gh) * kLog2E;
      if (bias_on<M> && mods.rel_bias != nullptr) tab = reinterpret_cast<const float*>(smem + C::OFF_TAB) + mods.R + kTabPad;
      fixed_ref = cap_on<M> && mods.cap * kLog2E <= kFixedRefCap2;
    }
    // NH = 2: hands this half's value of the row to the other half and gets the other's,
    // between the two warps of 32 rows.  Two buffers in turn: a thread writes a buffer again only after the
    // next exchange, to which the other half comes after reading it.
    [[maybe_unused]] uint32_t xn = 0;
    [[maybe_unused]] auto exchange = [&](float mine, float& other) -> bool {
      float* x = reinterpret_cast<float*>(smem + C::OFF_X) + ((xn & 1) * NQT + q) * 2 * kBM;
      x[half * kBM + row] = mine;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->x_full[q][warp & 3]);
      if (!mbar_wait(&bars->x_full[q][warp & 3], xn & 1, abort, p.status)) return false;
      other = x[(half ^ 1) * kBM + row];
      ++xn;
      return true;
    };
    // Moves the running maximum to the tile's; true when some row of the warp moved,
    // and then alpha is the row's factor.
    auto move_max = [&](float m_tile, float& alpha) -> bool {
      const float m_new = fmaxf(m, m_tile);
      const bool need = m_new > m + 8.f;
      const bool any = __any_sync(0xffffffffu, need);
      alpha = need ? ex2(m - m_new) : 1.f;
      if (need) {
        l *= alpha;
        m = m_new;
      }
      return any;
    };
    // The O rows times alpha.  PV of the previous tile has finished (S of this tile was
    // committed after it), and PV of this tile waits for this warp's arrival on p_full.
    auto scale_o = [&](float alpha) {
#pragma unroll 1
      for (int c = half * (D / 32 / NH); c < (half + 1) * (D / 32 / NH); ++c) {
        uint32_t ov[32];
        tmem_ld32(o_tm + c * 32, ov);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
        tmem_st32(o_tm + c * 32, ov);
      }
    };
    bool ok = tile_ok[q];
    for (int n = 0; n < n_kv && ok; ++n) {
      if (!(ok = mbar_wait(&bars->s_full[q], n & 1, abort, p.status))) break;
      tc_fence_after();
      // whether the reference may move at this tile (for both halves of a row alike)
      const bool track = !fixed_ref || __any_sync(0xffffffffu, starts(n));
      if constexpr (NH == 2) {
        // A half that none of the warp's rows sees (past the diagonal, before a window)
        // has P = 0: it only follows the other half's maximum.
        const int k0 = lo + n * kBN + half * NC;
        if (!__any_sync(0xffffffffu, mvlo <= mvhi && mvlo < k0 + NC && mvhi >= k0)) {
          if (track) {
            float other, alpha;
            if (!(ok = exchange(-INFINITY, other))) break;
            if (cap_on<M> && fixed_ref && starts(n)) other = floored(other);
            if (move_max(other, alpha) && n > 0) scale_o(alpha);
          }
          uint32_t zero[NC / 2];
#pragma unroll
          for (int c = 0; c < NC / 2; ++c) zero[c] = 0u;
          tmem_st(s_tm + half * NC, zero);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->p_full[q]);
          continue;
        }
      }
      uint32_t sr[NC / 32][32];
#pragma unroll
      for (int c = 0; c < NC / 32; ++c) tmem_ld32(s_tm + half * NC + c * 32, sr[c]);
      tmem_wait_ld();
      float s[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) s[c] = __uint_as_float(sr[c >> 5][c & 31]);
      const int kv0 = lo + n * kBN + half * NC;  // the thread's first key
      float sc = p.scale_log2;  // a score's factor into the log2 domain
      [[maybe_unused]] float off = 0.f;
      if constexpr (M::on) {
        const int d0 = t - kv0, dw = d0 - lane;  // distance of column 0; the warp's first row's
        Affine f{sc, 0.f};
        if constexpr (bias_on<M>)
          f = add_bias(s, tab, mods.R, slope2, ramp, d0, dw - (NC - 1), dw + 31, mods.later_hidden, sc);
        if constexpr (cap_on<M>) {
          const float k = cap_scores<true>(s, f, mods.cap, bias_on<M>, s_tm + half * NC);
          f = {k * mods.cap * kLog2E, 0.f};
        }
        sc = f.sc;
        off = f.off;
        const int c_lo = mvlo - kv0, c_hi = mvhi - kv0;
        if (!(c_lo <= 0 && c_hi >= NC - 1)) {
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (c < c_lo || c > c_hi) s[c] = -INFINITY;
        }
      } else {
        // rows whose keys in this tile are all visible skip the per-element mask
        bool full = row_ok && kv0 >= a && kv0 + kBN <= b && (!p.causal || kv0 + kBN - 1 <= t);
        if (p.window_left >= 0) full = full && (t - kv0 <= p.window_left) && (p.causal || kv0 + kBN - 1 - t <= p.window_left);
        if (!full) {
          int vlo, vhi;  // the row's visible keys, as one interval: two compares per element
          visible_keys(t, a, b, p.causal, p.window_left, row_ok, vlo, vhi);
          const int c_lo = vlo - kv0, c_hi = vhi - kv0;
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (c < c_lo || c > c_hi) s[c] = -INFINITY;
        }
      }
      float alpha = 1.f;
      bool rescale = false;
      if (track) {
        // row max as 8 independent chains
        float mx8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) mx8[e] = s[e];
#pragma unroll
        for (int c = 8; c < NC; c += 8)
#pragma unroll
          for (int e = 0; e < 8; ++e) mx8[e] = fmaxf(mx8[e], s[c + e]);
        const float mx = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                               fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
        float m_tile = M::on ? fmaf(mx, sc, off) : mx * sc;  // -inf stays -inf
        if constexpr (NH == 2) {
          float other;
          if (!(ok = exchange(m_tile, other))) break;
          m_tile = fmaxf(m_tile, other);
        }
        if (cap_on<M> && fixed_ref && starts(n)) m_tile = floored(m_tile);
        rescale = move_max(m_tile, alpha);
      }
      const float m_use = (m == -INFINITY) ? 0.f : m;
      uint64_t rs2[4] = {0, 0, 0, 0};  // 8 independent partial sums, two per register
      const float nm = M::on ? off - m_use : -m_use;
      const uint64_t sc2 = f2_pack(sc, sc), nm2 = f2_pack(nm, nm);
      constexpr int PC = NC == kBN ? 64 : 32;  // columns packed and stored as soon as they are done
#pragma unroll
      for (int h = 0; h < NC / PC; ++h) {
        uint32_t pk[PC / 2];
#pragma unroll
        for (int c = 0; c < PC / 2; ++c) {
          const float2 e = f2_unpack(f2_fma(f2_pack(s[PC * h + 2 * c], s[PC * h + 2 * c + 1]), sc2, nm2));
          const float p0 = ex2(e.x), p1 = ex2(e.y);
          rs2[c & 3] = f2_add(rs2[c & 3], f2_pack(p0, p1));
          pk[c] = pack_bf16x2(p0, p1);
        }
        tmem_st(s_tm + half * NC + PC / 2 * h, pk);
      }
      const float2 r01 = f2_unpack(f2_add(rs2[0], rs2[1])), r23 = f2_unpack(f2_add(rs2[2], rs2[3]));
      l += (r01.x + r01.y) + (r23.x + r23.y);
      if (rescale && n > 0) scale_o(alpha);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->p_full[q]);
    }
    if constexpr (NH == 2) {
      float other = 0.f;
      if (ok && (ok = exchange(l, other))) l = half == 0 ? l + other : other + l;
    }
    [[maybe_unused]] bool stored = false;
    // ---- epilogue: O /= l, bf16 out; LSE = ln(sum) including the sink
    if (ok && (ok = mbar_wait(&bars->o_final[q], 0, abort, p.status))) {
      tc_fence_after();
      const float inv_l = l > 0.f ? 1.f / l : 0.f;
      if constexpr (M::on) {
        // The warp's 32 rows go through its part of the Q tile (every S has read it),
        // 64 columns at a time in the swizzle of the tensor map (16-byte chunk e of row
        // r at r*128 + (e ^ r%8)*16), and out by TMA: stores of whole rows by their
        // threads touch a sector per 16 bytes and kept a CTA 2 us longer on its SM.
        // Halves: of a 128-wide row one atom each, of a 64-wide one the first has it all.
        constexpr int ATOMS = D / 64;
        const int c0 = NH == 2 && ATOMS == 2 ? half : 0, c1 = NH == 2 ? (ATOMS == 2 ? half + 1 : 1 - half) : ATOMS;
        if (c0 < c1) {
#pragma unroll 1
          for (int c = c0; c < c1; ++c) {
            uint8_t* stage = smem + C::OFF_Q + q * C::TILE + c * kAtomBytes + (row & ~31) * 128;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t ov[32];
              tmem_ld32(o_tm + c * 64 + h * 32, ov);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint4 pk;
                pk.x = pack_bf16x2(__uint_as_float(ov[8 * e]) * inv_l, __uint_as_float(ov[8 * e + 1]) * inv_l);
                pk.y = pack_bf16x2(__uint_as_float(ov[8 * e + 2]) * inv_l, __uint_as_float(ov[8 * e + 3]) * inv_l);
                pk.z = pack_bf16x2(__uint_as_float(ov[8 * e + 4]) * inv_l, __uint_as_float(ov[8 * e + 5]) * inv_l);
                pk.w = pack_bf16x2(__uint_as_float(ov[8 * e + 6]) * inv_l, __uint_as_float(ov[8 * e + 7]) * inv_l);
                *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * h + e) ^ (lane & 7)) << 4)) = pk;
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          const int tw = t - lane;  // the warp's first row; rows past the tensor's end are dropped by the copy
          if (lane == 0 && tw < p.BS) {
            for (int c = c0; c < c1; ++c)
              tma_store_rows(&to, smem + C::OFF_Q + q * C::TILE + c * kAtomBytes + (row & ~31) * 128, p, c, qh, tw);
            bulk_commit_group();
            stored = true;
          }
        }
      } else {
        __nv_bfloat16* orow = out.o + row_offset(p, qh, p.hq, p.Hq, row_ok ? t : 0, D);
#pragma unroll 1
        for (int c = half * (D / 32 / NH); c < (half + 1) * (D / 32 / NH); ++c) {
          uint32_t ov[32];
          tmem_ld32(o_tm + c * 32, ov);
          tmem_wait_ld();
          uint32_t pkd[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            pkd[e] = pack_bf16x2(__uint_as_float(ov[2 * e]) * inv_l, __uint_as_float(ov[2 * e + 1]) * inv_l);
          if (row_ok) {
            uint4* dst = reinterpret_cast<uint4*>(orow + c * 32);
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[e] = make_uint4(pkd[4 * e], pkd[4 * e + 1], pkd[4 * e + 2], pkd[4 * e + 3]);
          }
        }
      }
      if (row_ok && half == 0) {
        const int bb = t / p.S, ss = t - bb * p.S;
        out.lse[(static_cast<size_t>(r * p.B + bb) * p.hq + j) * p.S + ss] =
            l > 0.f || (M::on && l != l) ? (m + __log2f(l)) * 0.6931471805599453f : -INFINITY;
      }
    }
    if (stored) bulk_wait_group_all();  // the O stores are complete before the CTA ends
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TCOLS);
  }
}

}  // namespace fwd

// `tab_bytes`: shared memory of the bias row (Mods with a table, else 0).
template <int D, int NQT, int NH, class M>
static int run_fwd(const AttnArgs& a, const M& mods, int tab_bytes, const CUtensorMap& tq, const CUtensorMap& tk,
                   const CUtensorMap& tv, void* o, float* lse, cudaStream_t st) {
  using C = fwd::Cfg<D, NQT, NH>;
  fwd::Out out{static_cast<__nv_bfloat16*>(o), lse, (a.BS + NQT * kBM - 1) / (NQT * kBM)};
  auto kern = fwd::attn_fwd_kernel<D, NQT, NH, M>;
  const int smem = C::SMEM + tab_bytes;
  // the limit is one value per kernel, so one that fits every call: a call of another thread must not lower it
  // between this call's two steps
  constexpr int limit = C::SMEM + (bias_on<M> ? tab_len(kMaxBiasDistance) * static_cast<int>(sizeof(float)) : 0);
  static_assert(limit <= kMaxDynSmem, "forward shared memory");
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, limit) != cudaSuccess)
    return USP_ERR_CUDA;
  const unsigned grid = static_cast<unsigned>(out.nqb) * a.P * a.hq;
  CUtensorMap to;
  memset(&to, 0, sizeof(to));  // used with modified scores alone
  if constexpr (M::on) {
    const int rc = make_rows_tmap(&to, o, a, a.hq, a.Hq, D, 32);
    if (rc != USP_OK) return rc;
    return launch_chained(kern, grid, C::THREADS, smem, 1, st, tq, tk, tv, to, a, out, mods);
  }
  kern<<<grid, C::THREADS, smem, st>>>(tq, tk, tv, to, a, out, mods);
  return check_launch();
}

template <int D, class M>
static int run_fwd(const AttnArgs& a, const M& mods, int tab_bytes, const void* q, const void* k, const void* v,
                   void* o, float* lse, cudaStream_t st) {
  CUtensorMap tq, tk, tv;
  int rc;
  if ((rc = make_rows_tmap(&tq, q, a, a.hq, a.Hq, D, kBM)) != USP_OK) return rc;
  if ((rc = make_rows_tmap(&tk, k, a, a.hk, a.Hkv, D, kBN, a.kv_seq_io != 0)) != USP_OK) return rc;
  if ((rc = make_rows_tmap(&tv, v, a, a.hk, a.Hkv, D, kBN, a.kv_seq_io != 0)) != USP_OK) return rc;
  // Short causal windows at D = 64: the persistent schedule over the heads of
  // a key/value group.  Other short windows at D = 64: one Q tile per CTA (the
  // two tiles of a CTA would share little, and two small CTAs per SM overlap
  // each other's set-up and latencies instead).
  if (!M::on && fwd_window_fits(a, D)) return run_fwd_window(a, tq, tk, tv, o, lse, st);
  if constexpr (D == 64) {
    if (a.window_left >= 0 && a.window_left < 4 * kBN)
      return run_fwd<D, 1, fwd::kHalves<M>, M>(a, mods, tab_bytes, tq, tk, tv, o, lse, st);
  }
  // Few tiles: a CTA of two would leave SMs empty, and one tile in two halves has the shorter chain from S to P.
  // Two tiles / one, slopes, D = 128: 256 tokens of 8 heads (8 CTAs of two tiles) 12.9 /
  // 10.5 us, 2048 of 16 (128) 47.4 / 37.2; two rows of 1500 of 12 (144) 45.3 / 43.3 and at D = 64 39.6 / 41.2; 2048
  // of 32 (256) 53.6 / 70.0.  Half of the gain is that CTAs of unequal length spread better: where rows see later
  // keys too, D = 128 (one CTA per SM) keeps two tiles (2048 of 16 with a cap, a table and a prefix: 50 / 59).
  if constexpr (M::on) {
    const long long ctas = static_cast<long long>((a.BS + 2 * kBM - 1) / (2 * kBM)) * a.P * a.hq;
    if (ctas * 8 <= device_sm_count() * (D == 64 || mods.later_hidden ? 7 : 4)) return run_fwd<D, 1, 2, M>(a, mods, tab_bytes, tq, tk, tv, o, lse, st);
  }
  return run_fwd<D, 2, fwd::kHalves<M>, M>(a, mods, tab_bytes, tq, tk, tv, o, lse, st);
}

static inline AttnArgs make_fwd_args(const usp_attn_params& prm, int32_t* status) {
  AttnArgs a;
  a.B = prm.B;
  a.S = prm.S;
  a.BS = prm.B * prm.S;
  a.P = prm.P;
  a.hq = prm.Hq / prm.P;
  a.hk = prm.Hkv >= prm.P ? prm.Hkv / prm.P : 1;
  a.G = a.hq / a.hk;
  a.Hq = prm.Hq;
  a.Hkv = prm.Hkv;
  a.causal = prm.causal ? 1 : 0;
  a.window_left = prm.window_left;
  a.scale = prm.softmax_scale > 0.f ? prm.softmax_scale : 1.0f / sqrtf(static_cast<float>(prm.D));
  a.scale_log2 = a.scale * 1.4426950408889634f;
  a.cu = prm.cu_seqlens;
  a.n_docs = prm.n_docs;
  a.sinks = prm.sinks;
  a.status = status;
  a.seq_io = prm.io_layout != USP_IO_HEAD ? 1 : 0;
  a.kv_seq_io = prm.io_layout == USP_IO_SEQ ? 1 : 0;
  a.ring = prm.ring > 1 ? prm.ring : 1;
  a.ring_step = a.ring > 1 ? prm.ring_step : 0;
  a.C = prm.S / a.ring;
  a.Sl = prm.S / (prm.P * a.ring);  // sequence shard: P Ulysses ranks in each of `ring` groups
  a.kvh0 = 0;
  a.n_kvh = prm.Hkv;
  a.hq0 = 0;
  a.n_qh = prm.Hq;
  return a;
}

}  // namespace usp
