// beam_api.cu - the C entry points of the beam selection (declared in
// include/fp4q.h): argument checks; the kernels are in beam_select.cu.
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/fp4q.h"
#include "beam_launch.h"
#include "fp4q_launch.h"

using namespace fp4q;

namespace {

int beam_dtype(fp4_dtype_t d) {
  return d == FP4_DT_BF16 ? 0 : d == FP4_DT_FP16 ? 1 : d == FP4_DT_FP32 ? 2 : -1;
}

fp4_status_t check_sizes(int64_t B, int64_t K, int64_t V, int64_t n) {
  if (B < 0 || K <= 0 || V <= 0 || n <= 0) return FP4_ERR_INVALID_ARG;
  if (K > kBeamMostBeams || n > kBeamMostTake || V > kBeamMostVocab || B > INT32_MAX / (2 * K) ||
      B * K > INT32_MAX / (V / 512 + 2))
    return FP4_ERR_UNSUPPORTED_SHAPE;   // the kernels number rows and their parts in 32 bits
  return FP4_OK;
}

struct Extent {
  const void* p;
  int64_t bytes;
};

}  // namespace

extern "C" {

int64_t fp4_beam_select_workspace_bytes(int64_t B, int64_t K, int64_t V, int64_t n, fp4_dtype_t dtype) {
  const int dt = beam_dtype(dtype);
  if (dt < 0 || check_sizes(B, K, V, n) != FP4_OK) return -1;
  return beam_workspace(sm_count_current_device(), B, K, V);
}

fp4_status_t fp4_beam_select(const void* logits, int64_t row_stride, fp4_dtype_t dtype, const float* scores,
                             const uint8_t* finished, int64_t end_token, int64_t B, int64_t K, int64_t V,
                             int64_t n, float* out_scores, int32_t* out_parents, int32_t* out_tokens,
                             uint8_t* out_finished, void* workspace, int64_t workspace_bytes, int pdl,
                             fp4q_stream_t stream) {
  const int dt = beam_dtype(dtype);
  if (dt < 0 || workspace_bytes < 0) return FP4_ERR_INVALID_ARG;
  const fp4_status_t cs = check_sizes(B, K, V, n);
  if (cs != FP4_OK) return cs;
  const int64_t size = dt == 2 ? 4 : 2;
  if (row_stride == 0) row_stride = V;
  if (row_stride < V || end_token < 0 || end_token >= V) return FP4_ERR_INVALID_ARG;
  if ((finished == nullptr) != (out_finished == nullptr)) return FP4_ERR_INVALID_ARG;
  if (row_stride > INT64_MAX / 8 / (B * K + 1)) return FP4_ERR_UNSUPPORTED_SHAPE;   // extents that 64 bits number
  if (B == 0) return FP4_OK;
  const int64_t need = beam_workspace(sm_count_current_device(), B, K, V);
  if (!logits || !scores || !out_scores || !out_parents || !out_tokens || !workspace || workspace_bytes < need)
    return FP4_ERR_INVALID_ARG;
  if (!abi_aligned(logits, static_cast<uintptr_t>(size)) || !abi_aligned(scores, 4) || !abi_aligned(out_scores, 4) ||
      !abi_aligned(out_parents, 4) || !abi_aligned(out_tokens, 4) || !abi_aligned(workspace, 16))
    return FP4_ERR_MISALIGNED;
  const Extent writes[] = {{out_scores, B * n * 4}, {out_parents, B * n * 4}, {out_tokens, B * n * 4},
                           {out_finished, B * n}, {workspace, need}};
  const Extent reads[] = {{logits, ((B * K - 1) * row_stride + V) * size}, {scores, B * K * 4}, {finished, B * K}};
  for (int i = 0; i < 5; ++i) {
    if (!writes[i].p) continue;
    for (int j = i + 1; j < 5; ++j)
      if (writes[j].p && abi_overlap(writes[i].p, writes[i].bytes, writes[j].p, writes[j].bytes))
        return FP4_ERR_INVALID_ARG;
    for (const Extent& r : reads)
      if (r.p && abi_overlap(writes[i].p, writes[i].bytes, r.p, r.bytes)) return FP4_ERR_INVALID_ARG;
  }
  BeamParams p{};
  p.logits = logits;
  p.stride = row_stride;
  p.scores = scores;
  p.finished = finished;
  p.end_token = static_cast<int>(end_token);
  p.B = static_cast<int>(B);
  p.K = static_cast<int>(K);
  p.V = static_cast<int>(V);
  p.n = static_cast<int>(n);
  p.out_scores = out_scores;
  p.out_parents = out_parents;
  p.out_tokens = out_tokens;
  p.out_finished = out_finished;
  beam_shape(sm_count_current_device(), &p);
  p.stats = static_cast<float2*>(workspace);
  p.tops = reinterpret_cast<float*>(static_cast<char*>(workspace) + beam_stats_bytes(p));
  FP4Q_SET_DEBUG(p);
  return static_cast<fp4_status_t>(
      record_cuda_error(launch_beam_select(dt, p, pdl, reinterpret_cast<cudaStream_t>(stream))));
}

}  // extern "C"
