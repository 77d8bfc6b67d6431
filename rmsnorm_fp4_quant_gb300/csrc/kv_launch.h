// kv_launch.h - parameter blocks and launch entries of the NVFP4 key/value
// cache kernels (kv_cache.cu, kv_attention.cu), used by the C entry points in
// kv_api.cu.  Internal.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "debug_checks.h"

namespace fp4q {

// The cache's buffers and sizes (include/fp4q.h, fp4_kv_cache_t).
struct KvCache {
  uint8_t* k_packed;
  uint8_t* k_sf;
  uint8_t* v_packed;
  uint8_t* v_sf;
  const float* k_gs;
  const float* v_gs;
  int64_t num_pages;
  int page_size;
  int heads;           // key/value heads
  int D;               // channels of a head
};
__host__ __device__ inline long long kv_packed_extent(const KvCache& c) {
  return c.num_pages * c.heads * c.page_size * static_cast<long long>(c.D / 2);
}
__host__ __device__ inline long long kv_sf_extent(const KvCache& c) {
  return c.num_pages * c.heads * c.page_size * static_cast<long long>(c.D / 16);
}

struct KvAppendParams {
  const void* q;
  void* out_q;
  const void* k;
  const void* v;
  int64_t q_stride, out_q_stride, k_stride, v_stride;   // elements between tokens
  const int64_t* positions;
  const float* cos_sin;
  const int64_t* slots;
  int64_t max_position;
  int64_t T;
  int Hq;
  int rot;             // rotated channels, 0 = none
  int interleaved;
  KvCache c;
  FP4Q_DEBUG_FIELD
};

struct KvGatherParams {
  const int64_t* slots;
  void* out_k;
  void* out_v;
  int64_t T;
  KvCache c;
  FP4Q_DEBUG_FIELD
};

struct KvAttentionParams {
  const void* q;
  int64_t q_stride;
  KvCache c;
  const int32_t* tables;
  int64_t max_pages;
  const int32_t* seq_lens;
  const int32_t* cu;   // or null: one row per sequence
  int B;
  int64_t T;
  int Hq;
  int group;           // Hq / heads
  float sm_scale;
  int causal;
  void* out;
  float* lse;
  float* ws;
  int64_t ws_bytes;    // what the kernels need of it
  int* status;
  FP4Q_DEBUG_FIELD
};

// dtype 0 = bf16, 1 = fp16; sizes and alignment checked by the caller.
cudaError_t launch_kv_append(int dtype, const KvAppendParams& p, int pdl, cudaStream_t stream);
cudaError_t launch_kv_gather(int dtype, const KvGatherParams& p, int pdl, cudaStream_t stream);
cudaError_t launch_kv_attention(int dtype, const KvAttentionParams& p, int pdl, cudaStream_t stream);
// Bytes for sequences of at most `keys` keys.
int64_t kv_attention_workspace(int sms, int64_t B, int64_t T, int Hq, int heads, int D, int64_t keys);
// Bytes for every call of at most B sequences, T rows and `keys` keys.
int64_t kv_attention_workspace_bound(int sms, int64_t B, int64_t T, int Hq, int heads, int D, int64_t keys);
// fp4_attention_launch_shape (B and T not zero).
void kv_attention_shape(int sms, int64_t B, int64_t T, int Hq, int heads, int D, int64_t keys, int64_t out[2]);

}  // namespace fp4q
