// kv_attention_capped.cu - attention over the paged NVFP4 key/value cache with capped
// logits (and a window, a prefix or a bias besides).
#include "kv_attention_launch.cuh"

namespace fp4q {

// (kv_attention_wide_cap.cu)
cudaError_t launch_kv_attention_wide_cap(int dtype, const KvAttentionParams& p, int pdl, cudaStream_t stream);

cudaError_t launch_kv_attention_capped(int dtype, const KvAttentionParams& p, int pdl, cudaStream_t stream) {
  if (p.softcap > kWideCap) return launch_kv_attention_wide_cap(dtype, p, pdl, stream);
  return p.slopes ? launch_attention<kCappedBiased, kCappedBiased>(dtype, p, pdl, stream)
                  : launch_attention<kCapped, kCappedBiased>(dtype, p, pdl, stream);
}

}  // namespace fp4q
