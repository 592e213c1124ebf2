// usp_attn_bwd.cu — the launches of the plain attention backward (the kernels
// are in usp_attn_bwd.cuh, the backward with modified scores in usp_attn_mod_bwd.cu).
#include "usp_attn_bwd.cuh"

namespace usp {

size_t attn_bwd_ws_bytes(const usp_attn_params& p) {
  // planar {-LSE*log2e, D} per (rank, query head), rows padded to 4 tokens
  size_t n = static_cast<size_t>(p.Hq) * 2 * stats_row_pitch(p.B * p.S);
  return (n * sizeof(float) + 255) / 256 * 256;
}

size_t attn_bwd_ds_bytes(const usp_attn_params& p) {
  bwd::DsGeom g;
  long long n_blocks;
  if (!ds_geom(p, g, n_blocks)) return 0;
  return static_cast<size_t>(n_blocks) * kBN * bwd::kSL * 2;
}

// 1. D = rowsum(dO * O) and -LSE*log2e into the workspace, then the sink gradients.
int launch_attn_bwd_preprocess(const usp_attn_params& prm, const void* o, const float* lse, const void* dO,
                               float* dsinks, void* ws, int32_t* status, cudaStream_t st) {
  return run_preprocess(prm, NoMods{}, o, lse, dO, dsinks, ws, status, st);
}

// The stored-dS region of the workspace (after the statistics), or null when
// the workspace is too small for it or the shape has no such path.
static void* ds_region(const usp_attn_params& prm, const void* ws, size_t ws_bytes, bwd::DsGeom& g,
                       long long& n_blocks) {
  const size_t need = attn_bwd_ds_bytes(prm);
  if (need == 0 || ws_bytes < attn_bwd_ws_bytes(prm) + need || !ds_geom(prm, g, n_blocks)) return nullptr;
  return static_cast<uint8_t*>(const_cast<void*>(ws)) + attn_bwd_ws_bytes(prm);
}

// 2. dK, dV (and the dS blocks, when the workspace holds them)
int launch_attn_bwd_dkdv(const usp_attn_params& prm, const void* q, const void* k, const void* v, const float* lse,
                         const void* dO, void* dk, void* dv, const void* ws, size_t ws_bytes, int32_t* status,
                         cudaStream_t st) {
  const AttnArgs a = make_args(prm, status);
  const float* stats = static_cast<const float*>(ws);
  (void)lse;  // read through the preprocess's statistics
  bwd::DsGeom g{};
  long long nb = 0;
  void* ds = ds_region(prm, ws, ws_bytes, g, nb);
  if (prm.D == 128) return run_grad_pass<128>(false, a, NoMods{}, q, k, v, dO, nullptr, dk, dv, stats, ds, g, nb, st);
  return run_grad_pass<64>(false, a, NoMods{}, q, k, v, dO, nullptr, dk, dv, stats, ds, g, nb, st);
}

// 3. dQ (from the stored dS blocks when the workspace holds them, else by
// recomputing S and dP)
int launch_attn_bwd_dq(const usp_attn_params& prm, const void* q, const void* k, const void* v, const float* lse,
                       const void* dO, void* dq, const void* ws, size_t ws_bytes, int32_t* status, cudaStream_t st) {
  const AttnArgs a = make_args(prm, status);
  const float* stats = static_cast<const float*>(ws);
  (void)lse;
  bwd::DsGeom g{};
  long long nb = 0;
  void* ds = ds_region(prm, ws, ws_bytes, g, nb);
  if (prm.D == 128) return run_grad_pass<128>(true, a, NoMods{}, q, k, v, dO, dq, nullptr, nullptr, stats, ds, g, nb, st);
  return run_grad_pass<64>(true, a, NoMods{}, q, k, v, dO, dq, nullptr, nullptr, stats, ds, g, nb, st);
}

int launch_attn_bwd(const usp_attn_params& prm, const void* q, const void* k, const void* v, const void* o,
                    const float* lse, const void* dO, void* dq, void* dk, void* dv, float* dsinks, void* ws,
                    size_t ws_bytes, int32_t* status, cudaStream_t st) {
  int rc;
  if ((rc = launch_attn_bwd_preprocess(prm, o, lse, dO, dsinks, ws, status, st)) != USP_OK) return rc;
  if ((rc = launch_attn_bwd_dkdv(prm, q, k, v, lse, dO, dk, dv, ws, ws_bytes, status, st)) != USP_OK) return rc;
  return launch_attn_bwd_dq(prm, q, k, v, lse, dO, dq, ws, ws_bytes, status, st);
}

}  // namespace usp
