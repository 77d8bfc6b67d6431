// kv_attention.cu - attention over the paged NVFP4 key/value cache: choice of
// kernel and launch.

#include "fp4q_launch.h"
#include "kv_decode.cuh"

namespace fp4q {
namespace {

// Query rows of a key/value head that one item covers: 8 where a sequence
// has no more of them, else 16.
int decode_tiles(int64_t B, int64_t T, int group) { return T * group <= 8 * B ? 1 : 2; }

template <typename T, int D, int NT>
cudaError_t launch_decode(const KvAttentionParams& p, int pdl, cudaStream_t stream) {
  using S = DecodeShape<D, NT>;
  static_assert(S::kSmem <= 48 * 1024, "needs no raised shared-memory limit");
  const int ctas = sm_count_current_device() * S::kCtas;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kDecThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_decode_kernel<T, D, NT>, p);
  if (e != cudaSuccess) return e;
  const int64_t slots = decode_row_slots(p.B, p.T, p.group, S::kRows) * p.c.heads;
  cfg.gridDim = dim3(static_cast<unsigned>(slots), S::kRows);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;                              // its launch overlaps the first kernel
  return cudaLaunchKernelEx(&cfg, kv_decode_join_kernel<T, D, NT>, p, ctas);
}

template <typename T>
cudaError_t launch_type(const KvAttentionParams& p, int pdl, cudaStream_t stream) {
  const int nt = decode_tiles(p.B, p.T, p.group);
  if (p.c.D == 128)
    return nt == 1 ? launch_decode<T, 128, 1>(p, pdl, stream) : launch_decode<T, 128, 2>(p, pdl, stream);
  return nt == 1 ? launch_decode<T, 64, 1>(p, pdl, stream) : launch_decode<T, 64, 2>(p, pdl, stream);
}

template <int D, int NT>
int64_t decode_workspace(int sms, int64_t B, int64_t T, int group, int heads) {
  using S = DecodeShape<D, NT>;
  return 4LL * (2LL * sms * S::kCtas * S::kPart) + 8LL * decode_row_slots(B, T, group, S::kRows) * heads;
}

}  // namespace

int64_t kv_attention_workspace(int sms, int64_t B, int64_t T, int Hq, int heads, int D) {
  const int group = Hq / heads;
  if (B == 0 || T == 0) return 0;
  const int nt = decode_tiles(B, T, group);
  if (D == 128)
    return nt == 1 ? decode_workspace<128, 1>(sms, B, T, group, heads)
                   : decode_workspace<128, 2>(sms, B, T, group, heads);
  return nt == 1 ? decode_workspace<64, 1>(sms, B, T, group, heads)
                 : decode_workspace<64, 2>(sms, B, T, group, heads);
}

cudaError_t launch_kv_attention(int dtype, const KvAttentionParams& p, int pdl,
                                cudaStream_t stream) {
  return dtype == 0 ? launch_type<__nv_bfloat16>(p, pdl, stream) : launch_type<__half>(p, pdl, stream);
}

}  // namespace fp4q
