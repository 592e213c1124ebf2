// usp_attn_mod_fwd.cu — the launch of the attention forward with modified
// scores (the kernel of usp_attn_fwd.cuh with the steps of usp_attn_mods.cuh
// compiled in).
#include "usp_attn_fwd.cuh"

namespace usp {

ModArgs make_mods(const usp_attn_params& p, const usp_score_mods& m) {
  ModArgs x{};
  x.later_hidden = p.causal && m.prefix_lens == nullptr;
  x.cap = m.softcap;
  x.slopes = m.slopes;
  x.rel_bias = m.rel_bias;
  x.buckets = m.buckets;
  x.n_buckets = m.n_buckets;
  x.R = m.rel_bias != nullptr ? m.max_distance : 0;
  x.prefix = m.prefix_lens;
  x.n_prefix = m.n_prefix;
  return x;
}

int launch_attn_mod_fwd(const usp_attn_params& prm, const usp_score_mods& sm, const void* q, const void* k,
                        const void* v, void* o, float* lse, int32_t* status, cudaStream_t st) {
  const AttnArgs a = make_fwd_args(prm, status);
  const ModArgs m = make_mods(prm, sm);
  const int tab_bytes = m.rel_bias != nullptr ? tab_len(m.R) * static_cast<int>(sizeof(float)) : 0;
  return with_mods(m, [&](const auto& mods) {
    return prm.D == 128 ? run_fwd<128>(a, mods, tab_bytes, q, k, v, o, lse, st)
                        : run_fwd<64>(a, mods, tab_bytes, q, k, v, o, lse, st);
  });
}

}  // namespace usp
