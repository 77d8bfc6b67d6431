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
  uint64_t* keys;            // workspace: n keys of every part of every row,
  float2* stats;             // and its {largest logit, sum of exp(logit - largest)}
  int parts;                 // pieces that a row is cut into
  int part_len;              // elements of one, a multiple of the vector
  FP4Q_DEBUG_FIELD
};

__host__ __device__ inline long long beam_logits_extent(const BeamParams& p, int size) {
  return ((static_cast<long long>(p.B) * p.K - 1) * p.stride + p.V) * size;
}

// parts and part_len of the call's other sizes.  dtype 0 = bf16, 1 = fp16, 2 = fp32.
void beam_shape(int dtype, BeamParams* p);
int64_t beam_workspace(int dtype, int64_t B, int64_t K, int64_t V, int64_t n);
cudaError_t launch_beam_select(int dtype, const BeamParams& p, int pdl, cudaStream_t stream);

}  // namespace fp4q
