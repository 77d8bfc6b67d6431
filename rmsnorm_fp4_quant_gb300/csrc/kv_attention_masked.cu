// kv_attention_masked.cu - attention over the paged NVFP4 key/value cache with a window, a
// prefix and a bias that grows with distance.
#include "kv_attention_launch.cuh"

namespace fp4q {

// (kv_attention_capped.cu)
cudaError_t launch_kv_attention_capped(int dtype, const KvAttentionParams& p, int pdl, cudaStream_t stream);

cudaError_t launch_kv_attention_masked(int dtype, const KvAttentionParams& p, int pdl, cudaStream_t stream) {
  if (p.softcap > 0.0f) return launch_kv_attention_capped(dtype, p, pdl, stream);
  return p.slopes ? launch_attention<kBiased, kBiased>(dtype, p, pdl, stream)
                  : launch_attention<kMasked, kBiased>(dtype, p, pdl, stream);
}

}  // namespace fp4q
