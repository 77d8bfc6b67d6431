// kv_attention_wide_cap.cu - attention over the paged NVFP4 key/value cache with logits capped
// far above most of them (and a window, a prefix or a bias besides).
#include "kv_attention_launch.cuh"

namespace fp4q {

cudaError_t launch_kv_attention_wide_cap(int dtype, const KvAttentionParams& p, int pdl, cudaStream_t stream) {
  return launch_attention<kWideCapBiased, kWideCapBiased>(dtype, p, pdl, stream);
}

}  // namespace fp4q
