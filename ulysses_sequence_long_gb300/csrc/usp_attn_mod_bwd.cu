// usp_attn_mod_bwd.cu — the backward with modified scores: the kernels of
// usp_attn_bwd.cuh with the steps of usp_attn_mods.cuh compiled in, the rows of
// the bias by distance, and the reduction of the table's gradient.
//
// Workspace: the statistics of the plain backward | the bias rows by distance
// [Hq][tab_len(R)] | partial sums of dX by distance [Hq][n_kb][4][2R+1] (one row
// for each head, 32-key block and quarter of a query slice; the dK/dV pass writes
// them) | their sums over key blocks [Hq][splits][2R+1] | the stored dS blocks.
#include "usp_attn_bwd.cuh"

namespace usp {

ModArgs make_mods(const usp_attn_params& p, const usp_score_mods& m);

namespace bwd {

// --------------------------------------------------------------- delta
// The row statistics with D_t = sum_u P_tu (dO_t . v_u) summed in fp32 over the
// scores themselves (D_t = dO_t . O_t by the definition of O).  O reaches the
// backward as bf16 and from P rounded to bf16, each good to 2^-9: invisible in
// bf16 gradients, but the fp32 gradients of the sinks and of the bias table sum
// over all tokens and would carry it (relative error 1e-3 measured; with this
// pass under 1e-5).  It costs two of the five products of the backward.
//
// Persistent: one CTA per SM walks units (query head, 128 rows), late rows first,
// u = blockIdx.x, + gridDim.x, ...  A CTA per unit spent as long on its set-up
// (barriers, TMEM, first loads) and tear-down as on its tiles (capped windows of 128,
// D = 64: 102 us, and 76 so; learned bias, 8192 packed tokens, D = 128: 200 and 186).
// Q and dO tiles and a ring of 128-key tiles of K and V come by TMA and run on from
// unit to unit; S has two TMEM buffers, so S_{n+1} is issued while the compute warps
// turn S_n into P_n, behind dP_n, which takes dP's one buffer once they have read
// dP_{n-1}.  The tile counter n runs over all of the CTA's units.
// TMEM: S [0,128) and [128,256), dP [256,384), scratch [384,512) (tanh_rare).
// Column groups of four warps; a thread takes a row's 128 / kDeltaGroups keys of a tile.
// A cap's longer chain wants more warps (capped windows of 128, D = 64: 76 us with two
// groups, 66 with four; cap and table, 2048 tokens, D = 128: 52.5 and 50), a bias alone
// does not (8192 packed tokens, D = 128: 186 and 198).
template <class M>
constexpr int kDeltaGroups = cap_on<M> ? 4 : 2;

template <int D, int NG>
struct CfgD {
  static constexpr int THREADS = 128 * NG + 64;
  static constexpr int NCH = D / 64;
  static constexpr int TILE = NCH * kBN * 128;       // 128-row bf16 tile
  static constexpr int QST = D == 128 ? 1 : 2;       // buffers of (Q, dO)
  static constexpr int KST = D == 64 ? 5 : NG == 4 ? 2 : 3;  // buffers of K; S runs a tile ahead of dP
  static constexpr int VST = D == 128 ? 2 : 4;       // buffers of V
  static constexpr int OFF_Q = 0;                    // per buffer: Q, then dO
  static constexpr int OFF_K = OFF_Q + QST * 2 * TILE;
  static constexpr int OFF_V = OFF_K + KST * TILE;
  static constexpr int OFF_BAR = OFF_V + VST * TILE;
  static constexpr int OFF_RED = OFF_BAR + 512;      // [2][groups - 1][128] floats
  static constexpr int SMEM = OFF_RED + 2 * (NG - 1) * kBM * 4 + 1024;
};
static_assert(CfgD<128, 2>::SMEM <= kMaxDynSmem && CfgD<128, 4>::SMEM <= kMaxDynSmem &&
                  CfgD<64, 2>::SMEM <= kMaxDynSmem && CfgD<64, 4>::SMEM <= kMaxDynSmem,
              "delta shared memory");

struct BarsD {
  uint64_t qd_full[2], qd_free[2];
  uint64_t k_full[5], k_free[5], v_full[4], v_free[4];
  uint64_t s_full[2], s_free[2], dp_full, dp_free;
  uint64_t red_full[2];  // the other groups' row sums of a unit (two in turn) are in shared memory
  uint64_t mma_done;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(BarsD) <= 512, "delta barrier block");

struct DeltaUnit {
  int r, j, hg, t0, lo, n_kv;
  TileDocs docs;
};

// (by a whole warp)
template <class M>
__device__ __forceinline__ DeltaUnit delta_unit(const AttnArgs& p, const M& mods, int n_docs, int n_tiles, int u) {
  DeltaUnit w;
  w.hg = u % p.Hq;
  w.r = w.hg / p.hq;
  w.j = w.hg % p.hq;
  w.t0 = (n_tiles - 1 - u / p.Hq) * kBM;
  const int last = min(w.t0 + kBM, p.BS) - 1;
  int hi;
  w.docs = tile_docs(p, mods, n_docs, w.t0, last);
  key_range(p, mods, w.docs, w.t0, last, w.lo, hi);
  if (p.seq_io) w.lo &= ~(kBN - 1);  // key tiles inside one rank's shard
  w.n_kv = hi > w.lo ? (hi - w.lo + kBN - 1) / kBN : 0;
  return w;
}

template <int D, class M>
__global__ void __launch_bounds__(CfgD<D, kDeltaGroups<M>>::THREADS, 1)
    delta_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tdo,
                 const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, AttnArgs p,
                 const float* lse, float* __restrict__ stats, int bsp, int n_tiles, M mods) {
  constexpr int NG = kDeltaGroups<M>;
  using C = CfgD<D, NG>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  BarsD* bars = reinterpret_cast<BarsD*>(smem + C::OFF_BAR);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  grid_wait();
  const int n_docs = checked_docs(p);
  if (n_docs == 0) return;
  const int n_units = n_tiles * p.Hq;

  if (tid == 0) {
    for (int s = 0; s < C::QST; ++s) {
      mbar_init(&bars->qd_full[s], 1);
      mbar_init(&bars->qd_free[s], 1);
    }
    for (int s = 0; s < C::KST; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_free[s], 1);
    }
    for (int s = 0; s < C::VST; ++s) {
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_free[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->s_full[b], 1);
      mbar_init(&bars->s_free[b], 4 * NG);
      mbar_init(&bars->red_full[b], 4 * (NG - 1));
    }
    mbar_init(&bars->dp_full, 1);
    mbar_init(&bars->dp_free, 4 * NG);
    mbar_init(&bars->mma_done, 1);
    bars->abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(&bars->tmem, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  volatile int* abort = &bars->abort;
  const uint32_t sbase = smem_u32(smem);
  constexpr uint32_t T_DP = 256, T_SCRATCH = 384;

  // The producer's and the MMA issuer's warps walk the units as a whole (delta_unit);
  // their first lanes act.
  if (warp == 4 * NG) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      prefetch_tmap(&tq);
      prefetch_tmap(&tdo);
      prefetch_tmap(&tk);
      prefetch_tmap(&tv);
    }
    int n = 0, k = 0;  // tiles and units whose loads were issued
    int vn = 0;        // (a K without its V, where a wait gave up between them)
    bool ok = true;
    for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
      const DeltaUnit w = delta_unit(p, mods, n_docs, n_tiles, u);
      if (w.n_kv == 0) continue;
      if (lane == 0) {
        const HeadRef qh = q_head_ref(p, w.r, w.j), kvh = kv_head_ref(p, w.r, w.j / p.G);
        for (int i = 0; i < w.n_kv && ok; ++i) {
          const int s = n % C::KST;
          if (n >= C::KST && !(ok = mbar_wait(&bars->k_free[s], ((n / C::KST) - 1) & 1, abort, p.status))) break;
          mbar_arrive_expect_tx(&bars->k_full[s], C::TILE);
          for (int c = 0; c < C::NCH; ++c)
            tma_load_rows(smem + C::OFF_K + s * C::TILE + c * kAtomBytes, &tk, &bars->k_full[s], p, c, kvh,
                          w.lo + i * kBN);
          ++n;
          if (i == 0) {  // the unit's Q and dO, after its first keys: their buffer may still be read
            const int b = k % C::QST;
            if (k >= C::QST && !(ok = mbar_wait(&bars->qd_free[b], ((k / C::QST) - 1) & 1, abort, p.status))) break;
            uint8_t* qd = smem + C::OFF_Q + b * 2 * C::TILE;
            mbar_arrive_expect_tx(&bars->qd_full[b], 2 * C::TILE);
            for (int c = 0; c < C::NCH; ++c) {
              tma_load_rows(qd + c * kAtomBytes, &tq, &bars->qd_full[b], p, c, qh, w.t0);
              tma_load_rows(qd + C::TILE + c * kAtomBytes, &tdo, &bars->qd_full[b], p, c, qh, w.t0);
            }
            ++k;
          }
          const int v = vn % C::VST;
          if (vn >= C::VST && !(ok = mbar_wait(&bars->v_free[v], ((vn / C::VST) - 1) & 1, abort, p.status))) break;
          mbar_arrive_expect_tx(&bars->v_full[v], C::TILE);
          for (int c = 0; c < C::NCH; ++c)
            tma_load_rows(smem + C::OFF_V + v * C::TILE + c * kAtomBytes, &tv, &bars->v_full[v], p, c, kvh,
                          w.lo + i * kBN);
          ++vn;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (lane == 0) {
      // never leave the CTA with copies still landing in its shared memory
      for (int i = max(0, n - C::KST); i < n; ++i)
        mbar_wait(&bars->k_full[i % C::KST], (i / C::KST) & 1, abort, p.status);
      for (int i = max(0, vn - C::VST); i < vn; ++i)
        mbar_wait(&bars->v_full[i % C::VST], (i / C::VST) & 1, abort, p.status);
      for (int i = max(0, k - C::QST); i < k; ++i)
        mbar_wait(&bars->qd_full[i % C::QST], (i / C::QST) & 1, abort, p.status);
    }
  } else if (warp == 4 * NG + 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc = idesc_bf16(kBM, kBN, false, false);  // [128 rows x 128 keys], K = D
    auto issue = [&](uint32_t t_out, uint32_t a, uint32_t b) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_ss(tmem + t_out, kmajor_desc(a, kAtomBytes, kk), kmajor_desc(b, kAtomBytes, kk), idesc, kk > 0);
    };
    auto issue_s = [&](int n, uint32_t q_at) -> bool {
      const int s = n % C::KST, b = n & 1;
      if (!mbar_wait(&bars->k_full[s], (n / C::KST) & 1, abort, p.status)) return false;
      if (n >= 2 && !mbar_wait(&bars->s_free[b], ((n >> 1) - 1) & 1, abort, p.status)) return false;
      tc_fence_after();
      issue(b * kBN, q_at, sbase + C::OFF_K + s * C::TILE);
      mma_commit(&bars->s_full[b]);
      mma_commit(&bars->k_free[s]);
      return true;
    };
    auto issue_dp = [&](int n, uint32_t do_at) -> bool {
      const int s = n % C::VST;
      if (!mbar_wait(&bars->v_full[s], (n / C::VST) & 1, abort, p.status)) return false;
      if (n >= 1 && !mbar_wait(&bars->dp_free, (n - 1) & 1, abort, p.status)) return false;
      tc_fence_after();
      issue(T_DP, do_at, sbase + C::OFF_V + s * C::TILE);
      mma_commit(&bars->dp_full);
      mma_commit(&bars->v_free[s]);
      return true;
    };
    int n = 0, k = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
      const DeltaUnit w = delta_unit(p, mods, n_docs, n_tiles, u);
      if (w.n_kv == 0) continue;
      const int b = k % C::QST;
      if (lane == 0 && (ok = mbar_wait(&bars->qd_full[b], (k / C::QST) & 1, abort, p.status))) {
        const uint32_t q_at = sbase + C::OFF_Q + b * 2 * C::TILE, do_at = q_at + C::TILE;
        ok = issue_s(n, q_at);
        // dP_n before S_{n+1}: the compute warps come to dP_n first
        for (int i = 0; i < w.n_kv && ok; ++i, ++n) {
          ok = issue_dp(n, do_at);
          if (ok && i + 1 < w.n_kv) ok = issue_s(n + 1, q_at);
        }
        if (ok) mma_commit(&bars->qd_free[b]);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      ++k;
    }
    if (lane == 0) {
      mma_commit(&bars->mma_done);
      mbar_wait(&bars->mma_done, 0, abort, p.status);
    }
  } else {
    // ------------------------------------------------------------ compute
    constexpr int NC = kBN / NG;
    const int grp = warp >> 2;  // key columns [NC*grp, NC*grp + NC) of every tile
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lb = tmem + ((static_cast<uint32_t>(warp & 3) * 32) << 16);
    float* red = reinterpret_cast<float*>(smem + C::OFF_RED);
    // What a unit needs of its geometry; the next unit's is looked up under the first
    // tile of the current one, whose dP is not there yet.
    struct Row {
      int lo, n_kv, vlo, vhi;
      float lse;
    };
    auto row_of = [&](int u) -> Row {
      Row x{0, 0, 1, 0, 0.f};
      if (u >= n_units) return x;
      const DeltaUnit w = delta_unit(p, mods, n_docs, n_tiles, u);
      const int t = w.t0 + row;
      const bool row_ok = t < p.BS;
      if (row_ok) x.lse = gld(lse + stat_index(p, w.r, w.j, t));
      int a = 0, b = 0, pe = 0;
      if (row_ok) doc_bounds(p, mods, w.docs, t, a, b, pe);
      visible_keys(mods, t, a, b, pe, p.causal, p.window_left, row_ok, x.vlo, x.vhi);
      x.lo = w.lo;
      x.n_kv = w.n_kv;
      return x;
    };
    Row next = row_of(blockIdx.x);
    int n = 0, k = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
      const Row w = next;
      const int hg = u % p.Hq, t = (n_tiles - 1 - u / p.Hq) * kBM + row;
      const float nlse2 = w.lse == -INFINITY || t >= p.BS ? -INFINITY : w.lse * -kLog2e;  // (as in preprocess_kernel)
      const float* tab =
          mods.table != nullptr ? mods.table + static_cast<size_t>(hg) * tab_len(mods.R) + mods.R + kTabPad : nullptr;
      const float slope2 = mods.slopes != nullptr ? gld(mods.slopes + hg) * kLog2E : 0.f;
      if (w.n_kv == 0) {
        next = row_of(u + static_cast<int>(gridDim.x));
        continue;
      }
      uint64_t acc2[4] = {0, 0, 0, 0};  // 8 independent partial sums, two per register
      for (int i = 0; i < w.n_kv && ok; ++i, ++n) {
        const int k0 = w.lo + i * kBN + grp * NC;  // first key of this group's columns
        if (!(ok = mbar_wait(&bars->s_full[n & 1], (n >> 1) & 1, abort, p.status))) break;
        tc_fence_after();
        float x[NC];
        tmem_ld_cols<NC>(lb + (n & 1) * kBN + grp * NC, x);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->s_free[n & 1]);
        const int d0 = t - k0, dw = d0 - lane;
        Affine f{p.scale_log2, 0.f};
        if constexpr (bias_on<M>)
          f = add_bias(x, tab, mods.R, slope2, nullptr, d0, dw - (NC - 1), dw + 31, mods.later_hidden, p.scale_log2);
        if constexpr (cap_on<M>) {
          cap_scores<false>(x, f, mods.cap, true, lb + T_SCRATCH + grp * NC);
          f = {mods.cap * kLog2E, 0.f};
        }
        const int c_lo = w.vlo - k0, c_hi = w.vhi - k0;
        if (!(c_lo <= 0 && c_hi >= NC - 1)) {
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (c < c_lo || c > c_hi) x[c] = -INFINITY;
        }
        const uint64_t sc2 = f2_pack(f.sc, f.sc), nl2 = f2_pack(nlse2 + f.off, nlse2 + f.off);
#pragma unroll
        for (int c = 0; c < NC; c += 2) {
          const float2 e = f2_unpack(f2_fma(f2_pack(x[c], x[c + 1]), sc2, nl2));
          x[c] = ex2(e.x);
          x[c + 1] = ex2(e.y);
        }
        if (i == 0) next = row_of(u + static_cast<int>(gridDim.x));
        if (!(ok = mbar_wait(&bars->dp_full, n & 1, abort, p.status))) break;
        tc_fence_after();
        float dp[NC];
        tmem_ld_cols<NC>(lb + T_DP + grp * NC, dp);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->dp_free);
#pragma unroll
        for (int c = 0; c < NC; c += 2)
          acc2[(c >> 1) & 3] = f2_fma(f2_pack(x[c], x[c + 1]), f2_pack(dp[c], dp[c + 1]), acc2[(c >> 1) & 3]);
      }
      if (!ok) break;
      const float2 s01 = f2_unpack(f2_add(acc2[0], acc2[1])), s23 = f2_unpack(f2_add(acc2[2], acc2[3]));
      const float sum = (s01.x + s01.y) + (s23.x + s23.y);
      // The parts of a row meet.  The other groups write a buffer again two units
      // later, for which they have waited for a dP that the first group's reading of
      // the unit between released: the first group has read this one by then.
      float* part = red + (k & 1) * (NG - 1) * kBM + row;
      if (grp > 0) {
        part[(grp - 1) * kBM] = sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->red_full[k & 1]);
      } else {
        if (!(ok = mbar_wait(&bars->red_full[k & 1], (k >> 1) & 1, abort, p.status))) break;
        if (t < p.BS) {
          float* plane = stats + plane_index(bsp, p.hq, hg / p.hq, hg % p.hq, 0, t);
          plane[0] = nlse2 - slope_of_row(mods, slope2, t);
          float all = sum;
#pragma unroll
          for (int e = 0; e < NG - 1; ++e) all += part[e * kBM];
          plane[bsp] = all;
        }
      }
      ++k;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace bwd

namespace {

template <int D, class M>
int run_delta(const AttnArgs& a, const M& m, const void* q, const void* k, const void* v, const void* dO,
              const float* lse, float* stats, cudaStream_t st) {
  using C = bwd::CfgD<D, bwd::kDeltaGroups<M>>;
  CUtensorMap tq, tdo, tk, tv;
  int rc;
  if ((rc = make_rows_tmap(&tq, q, a, a.hq, a.Hq, D, kBM)) != USP_OK) return rc;
  if ((rc = make_rows_tmap(&tdo, dO, a, a.hq, a.Hq, D, kBM)) != USP_OK) return rc;
  if ((rc = make_rows_tmap(&tk, k, a, a.hk, a.Hkv, D, kBN)) != USP_OK) return rc;
  if ((rc = make_rows_tmap(&tv, v, a, a.hk, a.Hkv, D, kBN)) != USP_OK) return rc;
  auto kern = bwd::delta_kernel<D, M>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return USP_ERR_CUDA;
  const int n_tiles = (a.BS + kBM - 1) / kBM;
  const long long units = static_cast<long long>(n_tiles) * a.Hq;
  const int grid = units < device_sm_count() ? static_cast<int>(units) : device_sm_count();
  return launch_chained(kern, grid, C::THREADS, C::SMEM, 1, st, tq, tdo, tk, tv, a, lse, stats,
                        stats_row_pitch(a.BS), n_tiles, m);
}

constexpr int kRelThreads = 256;
constexpr int kRelRows = 32;    // partial rows that one block of the first reduction sums
constexpr int kRelSplits = 64;  // most blocks per head
constexpr int kRelDirect = 96;  // rows that the second reduction takes by itself: 32 rows of 257 in 4.7 us, 8.5 with the
                                // first before it (8192 tokens: 16 us both; blocks that join by a ticket: 26)
constexpr int kRelAhead = 16;   // rows whose loads a thread has in flight

// Threads of a block for each distance of a row, and how many such teams 1024 hold.
__host__ __device__ constexpr int rel_width(int row) { return row < 1024 ? (row + 31) / 32 * 32 : 1024; }
__host__ __device__ constexpr int rel_teams(int row) { return 1024 / rel_width(row); }

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

struct Layout {
  size_t table, partial, sums, ds, total;  // byte offsets; total without the stored dS
  int n_kb, n_rows, splits;
};

Layout mod_layout(const usp_attn_params& p, const usp_score_mods& m) {
  Layout L{};
  L.table = L.partial = L.sums = attn_bwd_ws_bytes(p);
  L.n_kb = (p.B * p.S + 31) / 32;
  L.n_rows = kModGroups * L.n_kb;
  L.splits = L.n_rows <= kRelDirect ? 1 : (L.n_rows + kRelRows - 1) / kRelRows;
  if (L.splits > kRelSplits) L.splits = kRelSplits;
  size_t end = L.table;
  if (m.rel_bias != nullptr) {
    const size_t row = 2 * static_cast<size_t>(m.max_distance) + 1;
    end = L.partial = end + up256(sizeof(float) * p.Hq * tab_len(m.max_distance));
    if (m.rel_bias_grad) {
      end = L.sums = end + up256(sizeof(float) * p.Hq * static_cast<size_t>(L.n_rows) * row);
      end += up256(sizeof(float) * p.Hq * static_cast<size_t>(L.splits) * row);
    }
  }
  L.ds = L.total = end;
  return L;
}

// A prefix, or no causal order, lets a key be seen by earlier rows: the stored
// dS then takes every (key tile, query slice) pair.
bool every_slice(const usp_attn_params& p, const usp_score_mods& m) { return !p.causal || m.prefix_lens != nullptr; }

size_t mod_ds_bytes(const usp_attn_params& p, const usp_score_mods& m) {
  bwd::DsGeom g;
  long long n;
  return ds_geom(p, g, n, every_slice(p, m)) ? static_cast<size_t>(n) * kBN * bwd::kSL * 2 : 0;
}

// Rows by distance in the log2 domain (the first block of a head), and cleared
// partial sums (every block).
__global__ void __launch_bounds__(kRelThreads)
    rel_expand_kernel(ModArgs m, float* __restrict__ table, float4* __restrict__ clear, size_t n_clear, int32_t* status) {
  const int n = tab_len(m.R), h = blockIdx.x;
  grid_wait();
  if (blockIdx.y == 0)
    for (int e = threadIdx.x; e < n; e += kRelThreads)
      table[static_cast<size_t>(h) * n + e] = table_entry(m, h, e, status);
  // the partial sums: distances that no chunk reaches stay at zero
  const size_t step = static_cast<size_t>(gridDim.x) * gridDim.y * kRelThreads;
  for (size_t i = (static_cast<size_t>(blockIdx.y) * gridDim.x + h) * kRelThreads + threadIdx.x; i < n_clear; i += step)
    clear[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

// One column of rows [r0, r1), kRelAhead of them in flight (the last again past the
// end: a load behind a branch would wait for the one before), joined in a fixed order.
__device__ __forceinline__ float rel_column(const float* src, int r0, int r1, int step, int row) {
  float acc = 0.f;
  for (int r = r0; r < r1; r += step) {
    float x[kRelAhead];
#pragma unroll
    for (int e = 0; e < kRelAhead; ++e) x[e] = gld(src + static_cast<size_t>(min(r + e, r1 - 1)) * row);
#pragma unroll
    for (int e = 0; e < kRelAhead; ++e) x[e] = r + e < r1 ? x[e] : 0.f;
#pragma unroll
    for (int o = kRelAhead / 2; o > 0; o >>= 1)
#pragma unroll
      for (int e = 0; e < o; ++e) x[e] += x[e + o];
    acc += x[0];
  }
  return acc;
}

// Many rows: a split's partial rows of a head become one, thread = distance.
__global__ void __launch_bounds__(1024, 1)
    rel_sum_kernel(const float* partial, float* __restrict__ sums, int n_rows, int per, int row) {
  const int h = blockIdx.x, s = blockIdx.y;
  grid_wait();
  const float* src = partial + static_cast<size_t>(h) * n_rows * row;
  for (int c = threadIdx.x; c < row; c += blockDim.x)
    sums[(static_cast<size_t>(h) * gridDim.y + s) * row + c] =
        rel_column(src + c, s * per, min(n_rows, (s + 1) * per), kRelAhead, row);
}

// A head's rows, teams of threads in turn over them, then its buckets: a warp takes a
// bucket at a time, its lanes the distances, joined by a fixed tree (no atomics: the
// result does not depend on the schedule).
__global__ void __launch_bounds__(1024, 1)
    rel_grad_kernel(ModArgs m, const float* rows, float* __restrict__ drel, int n_rows, int row) {
  extern __shared__ float by_dist[];  // [teams][row]
  const int teams = rel_teams(row), width = blockDim.x / teams, team = threadIdx.x / width;
  int* bucket = reinterpret_cast<int*>(by_dist + teams * row);
  const int h = blockIdx.x, lane = threadIdx.x & 31;
  grid_wait();
  const float* src = rows + static_cast<size_t>(h) * n_rows * row;
  for (int c = threadIdx.x - team * width; c < row; c += width)
    by_dist[team * row + c] = rel_column(src + c, team * kRelAhead, n_rows, teams * kRelAhead, row);
  for (int c = threadIdx.x; c < row; c += blockDim.x) bucket[c] = min(max(gld(m.buckets + c), 0), m.n_buckets - 1);
  __syncthreads();
  for (int b = threadIdx.x >> 5; b < m.n_buckets; b += blockDim.x / 32) {
    float acc = 0.f;
    for (int c = lane; c < row; c += 32)
      if (bucket[c] == b)
        for (int e = 0; e < teams; ++e) acc += by_dist[e * row + c];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0) drel[static_cast<size_t>(h) * m.n_buckets + b] = acc;
  }
}

// dsink_h = -sum_t exp(sink_h - LSE_t) D_t: one block per head, fixed-order tree.
constexpr int kSinkThreads = 512;
__global__ void __launch_bounds__(kSinkThreads)
    mod_dsink_kernel(const float* stats, const float* lse, float* __restrict__ dsinks,
                     AttnArgs p, int bsp) {
  __shared__ float red[kSinkThreads];
  const int r = blockIdx.x / p.hq, j = blockIdx.x % p.hq;
  grid_wait();
  const float z2 = gld(p.sinks + blockIdx.x) * kLog2E;
  const float* dd = stats + bwd::plane_index(bsp, p.hq, r, j, 1, 0);
  float acc = 0.f;
  for (int b = 0; b < p.B; ++b) {
    const float* l = lse + (static_cast<size_t>(r * p.B + b) * p.hq + j) * p.S;
#pragma unroll 4
    for (int s = threadIdx.x; s < p.S; s += kSinkThreads) {
      // a row that sees nothing, beside a sink of no weight (-inf): its weights are zero
      const float lse_s = gld(l + s), w = lse_s == -INFINITY ? 0.f : ex2(fmaf(-kLog2E, lse_s, z2));
      acc -= w * gld(dd + b * p.S + s);
    }
  }
  red[threadIdx.x] = acc;
  __syncthreads();
  for (int s = kSinkThreads / 2; s > 0; s >>= 1) {
    if (threadIdx.x < s) red[threadIdx.x] += red[threadIdx.x + s];
    __syncthreads();
  }
  if (threadIdx.x == 0) dsinks[blockIdx.x] = red[0];
}

ModArgs bwd_mods(const usp_attn_params& p, const usp_score_mods& sm, const void* ws) {
  ModArgs m = make_mods(p, sm);
  const Layout L = mod_layout(p, sm);
  uint8_t* base = static_cast<uint8_t*>(const_cast<void*>(ws));
  m.n_kb = L.n_kb;
  if (sm.rel_bias != nullptr) {
    m.table = reinterpret_cast<const float*>(base + L.table);
    if (sm.rel_bias_grad) m.partial = reinterpret_cast<float*>(base + L.partial);
  }
  return m;
}

// The stored-dS region of the workspace, or null when it does not hold one.
void* mod_ds_region(const usp_attn_params& p, const usp_score_mods& m, const void* ws, size_t ws_bytes,
                    bwd::DsGeom& g, long long& n) {
  const size_t need = mod_ds_bytes(p, m), at = mod_layout(p, m).ds;
  if (need == 0 || ws_bytes < at + need || !ds_geom(p, g, n, every_slice(p, m))) return nullptr;
  return static_cast<uint8_t*>(const_cast<void*>(ws)) + at;
}

}  // namespace

size_t attn_mod_bwd_ws_bytes(const usp_attn_params& p, const usp_score_mods& m) { return mod_layout(p, m).total; }

size_t attn_mod_bwd_fast_ws_bytes(const usp_attn_params& p, const usp_score_mods& m) {
  const size_t ds = mod_ds_bytes(p, m);
  return ds == 0 ? 0 : mod_layout(p, m).total + ds;
}

int launch_attn_mod_bwd_preprocess(const usp_attn_params& p, const usp_score_mods& sm, const void* q, const void* k,
                                   const void* v, const void* o, const float* lse, const void* dO, float* dsinks,
                                   void* ws, int32_t* status, cudaStream_t st) {
  const ModArgs m = bwd_mods(p, sm, ws);
  if (sm.rel_bias != nullptr) {
    const Layout L = mod_layout(p, sm);
    uint8_t* base = static_cast<uint8_t*>(ws);
    const size_t n_clear = sm.rel_bias_grad ? (L.sums - L.partial) / sizeof(float4) : 0;
    const int per_head = n_clear > 0 ? (4 * device_sm_count() + p.Hq - 1) / p.Hq : 1;
    const int rc = launch_chained(rel_expand_kernel, dim3(p.Hq, per_head), kRelThreads, 0, 1, st, m,
                                  reinterpret_cast<float*>(base + L.table),
                                  reinterpret_cast<float4*>(base + L.partial), n_clear, status);
    if (rc != USP_OK) return rc;
  }
  const bool exact_delta = dsinks != nullptr || m.partial != nullptr;  // a gradient in fp32 hangs on D
  if (!exact_delta)
    return with_mods(m, [&](const auto& mods) { return run_preprocess(p, mods, o, lse, dO, nullptr, ws, status, st); });
  const AttnArgs a = make_args(p, status);
  float* stats = static_cast<float*>(ws);
  const int rc = with_mods(m, [&](const auto& mods) {
    return p.D == 128 ? run_delta<128>(a, mods, q, k, v, dO, lse, stats, st)
                      : run_delta<64>(a, mods, q, k, v, dO, lse, stats, st);
  });
  if (rc != USP_OK || dsinks == nullptr) return rc;
  return launch_chained(mod_dsink_kernel, a.Hq, kSinkThreads, 0, 1, st, stats, lse, dsinks, a, stats_row_pitch(a.BS));
}

int launch_attn_mod_bwd_dkdv(const usp_attn_params& p, const usp_score_mods& sm, const void* q, const void* k,
                             const void* v, const void* dO, void* dk, void* dv, const void* ws, size_t ws_bytes,
                             int32_t* status, cudaStream_t st) {
  const AttnArgs a = make_args(p, status);
  const ModArgs m = bwd_mods(p, sm, ws);
  const float* stats = static_cast<const float*>(ws);
  bwd::DsGeom g{};
  long long nb = 0;
  void* ds = mod_ds_region(p, sm, ws, ws_bytes, g, nb);
  return with_mods(m, [&](const auto& mods) {
    return p.D == 128 ? run_grad_pass<128>(false, a, mods, q, k, v, dO, nullptr, dk, dv, stats, ds, g, nb, st)
                      : run_grad_pass<64>(false, a, mods, q, k, v, dO, nullptr, dk, dv, stats, ds, g, nb, st);
  });
}

int launch_attn_mod_bwd_dq(const usp_attn_params& p, const usp_score_mods& sm, const void* q, const void* k,
                           const void* v, const void* dO, void* dq, const void* ws, size_t ws_bytes, int32_t* status,
                           cudaStream_t st) {
  const AttnArgs a = make_args(p, status);
  const ModArgs m = bwd_mods(p, sm, ws);
  const float* stats = static_cast<const float*>(ws);
  bwd::DsGeom g{};
  long long nb = 0;
  void* ds = mod_ds_region(p, sm, ws, ws_bytes, g, nb);
  return with_mods(m, [&](const auto& mods) {
    return p.D == 128 ? run_grad_pass<128>(true, a, mods, q, k, v, dO, dq, nullptr, nullptr, stats, ds, g, nb, st)
                      : run_grad_pass<64>(true, a, mods, q, k, v, dO, dq, nullptr, nullptr, stats, ds, g, nb, st);
  });
}

int launch_attn_mod_bwd_rel_bias(const usp_attn_params& p, const usp_score_mods& sm, float* drel_bias, void* ws,
                                 cudaStream_t st) {
  const Layout L = mod_layout(p, sm);
  uint8_t* base = static_cast<uint8_t*>(ws);
  const int row = 2 * sm.max_distance + 1, width = rel_width(row), teams = rel_teams(row);
  const float* rows = reinterpret_cast<const float*>(base + L.partial);
  int n_rows = L.n_rows;
  if (L.splits > 1) {
    float* sums = reinterpret_cast<float*>(base + L.sums);
    const int per = (L.n_rows + L.splits - 1) / L.splits;
    const int rc = launch_chained(rel_sum_kernel, dim3(p.Hq, L.splits), width, 0, 1, st, rows, sums, n_rows, per, row);
    if (rc != USP_OK) return rc;
    rows = sums;
    n_rows = L.splits;
  }
  const int smem = row * (teams * static_cast<int>(sizeof(float)) + static_cast<int>(sizeof(int)));
  return launch_chained(rel_grad_kernel, p.Hq, teams * width, smem, 1, st, make_mods(p, sm), rows, drel_bias, n_rows,
                        row);
}

}  // namespace usp
