// usp_attn_fwd.cu — the launch of the plain attention forward (the kernel is in
// usp_attn_fwd.cuh, the forward with modified scores in usp_attn_mod_fwd.cu).
#include "usp_attn_fwd.cuh"

namespace usp {

int launch_attn_fwd(const usp_attn_params& prm, const void* q, const void* k, const void* v, void* o, float* lse,
                    int32_t* status, cudaStream_t st) {
  const AttnArgs a = make_fwd_args(prm, status);
  if (prm.D == 128) return run_fwd<128>(a, NoMods{}, 0, q, k, v, o, lse, st);
  return run_fwd<64>(a, NoMods{}, 0, q, k, v, o, lse, st);
}

}  // namespace usp
