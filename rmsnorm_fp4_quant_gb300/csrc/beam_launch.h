// beam_launch.h - parameter block and launch entry of the beam selection
// (beam_select.cu), used by the C entry point in beam_api.cu.  Internal.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "debug_checks.h"

namespace fp4q {

constexpr int kBeamMostTake = 64;            // candidates of a batch entry
constexpr int kBeamMostBeams = 256;
constexpr int64_t kBeamMostVocab = 1 << 24;

struct BeamParams {
  const void* logits;
  int64_t stride;            // elements between rows
  const float* scores;
  const uint8_t* finished;   // or null
  int end_token;
  int B, K, V, n;
  float* out_scores;
  int32_t* out_parents;
  int32_t* out_tokens;
  uint8_t* out_finished;     // or null
  float2* stats;             // workspace: of every part of every row {M, sum of 2^(logit log2(e) - M)},
  float* tops;               // and the largest logit of every group of every row
  int parts;                 // pieces that a row is cut into
  int groups;                // of a row
  FP4Q_DEBUG_FIELD
};

__host__ __device__ inline long long beam_logits_extent(const BeamParams& p, int size) {
  return ((static_cast<long long>(p.B) * p.K - 1) * p.stride + p.V) * size;
}

// The parts and groups that the call's other sizes lead to.
void beam_shape(int sms, BeamParams* p);
int64_t beam_stats_bytes(const BeamParams& p);
// An upper bound that grows with each size.
int64_t beam_workspace(int sms, int64_t B, int64_t K, int64_t V);
// dtype 0 = bf16, 1 = fp16, 2 = fp32; sizes and alignment checked by the caller.
cudaError_t launch_beam_select(int dtype, const BeamParams& p, int pdl, cudaStream_t stream);

}  // namespace fp4q
