// kv_attention.cu - attention over the paged NVFP4 key/value cache.
//
//   out = softmax(sm_scale / gs_k * q k^T) v / gs_v,  k, v = code * block scale
#include "async_copy.cuh"
#include "fused_common.cuh"
#include "kv_launch.h"

namespace fp4q {
namespace {

__device__ __forceinline__ float e2m1_decode(uint32_t code) {
  const uint32_t e = (code >> 1) & 3u, m = code & 1u;
  const float mag = e ? (1.0f + 0.5f * static_cast<float>(m)) * static_cast<float>(1u << (e - 1))
                      : 0.5f * static_cast<float>(m);
  return (code & 8u) ? -mag : mag;
}

template <typename T> __device__ __forceinline__ float to_f32(T x);
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f32(float x) { return __float2half_rn(x); }

// One warp per query row and head: 32 keys at a time, one per lane, then the
// weighted values with D / 32 channels per lane.
template <typename T>
__global__ void __launch_bounds__(128) kv_attention_simple_kernel(const KvAttentionParams p) {
  __shared__ float qs[4][128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + warp;
  if (item >= p.T * p.Hq) return;
  griddep_wait();
  const int64_t t = item / p.Hq;
  const int h = static_cast<int>(item - t * p.Hq), kvh = h / p.group;
  const int D = p.c.D;
  int b = 0;
  int64_t q0 = t, n_q = 1;
  if (p.cu) {
    int lo = 0, hi = p.B - 1;                    // last b with cu[b] <= t
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (p.cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    b = lo;
    q0 = p.cu[b];
    n_q = p.cu[b + 1] - q0;
    if (t < q0 || t >= q0 + n_q) return;         // a row of no sequence
  } else {
    b = static_cast<int>(t);
  }
  const int64_t limit = p.max_pages * p.c.page_size;
  int64_t len = p.seq_lens[b];
  len = len < 0 ? 0 : len > limit ? limit : len;
  const int64_t seen = p.causal ? (len - n_q + (t - q0) + 1) : len;
  const T* qrow = static_cast<const T*>(p.q) + t * p.q_stride + static_cast<int64_t>(h) * D;
  for (int i = lane; i < D; i += 32) qs[warp][i] = to_f32<T>(qrow[i]);
  __syncwarp();
  const float scale = p.c.k_gs ? p.sm_scale / __ldg(p.c.k_gs) : p.sm_scale;
  float m = -INFINITY, l = 0.0f, acc[4] = {};
  const int per = D / 32;
  for (int64_t j0 = 0; j0 < seen; j0 += 32) {
    const int64_t j = j0 + lane;
    int64_t page = -1, row = 0;
    if (j < seen) {
      page = p.tables[b * p.max_pages + j / p.c.page_size];
      if (page >= p.c.num_pages) page = -1;
      row = (page * p.c.heads + kvh) * p.c.page_size + j % p.c.page_size;
    }
    float s = -INFINITY;
    if (page >= 0) {
      s = 0.0f;
      for (int blk = 0; blk < D / 16; ++blk) {
        float part = 0.0f;
        const uint8_t* kp = p.c.k_packed + row * (D / 2) + blk * 8;
        for (int i = 0; i < 8; ++i) {
          part += e2m1_decode(kp[i] & 15u) * qs[warp][blk * 16 + 2 * i];
          part += e2m1_decode(kp[i] >> 4) * qs[warp][blk * 16 + 2 * i + 1];
        }
        s += part * e4m3_decode(p.c.k_sf[row * (D / 16) + blk]);
      }
      s *= scale;
    }
    float top = s;
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
    if (!__any_sync(kFullMask, page >= 0)) continue;
    const float m_new = fmaxf(m, top);
    const float f = expf(m - m_new);
    const float w = page >= 0 ? expf(s - m_new) : 0.0f;
    l = l * f + w;
    for (int i = 0; i < per; ++i) acc[i] *= f;
    for (int k = 0; k < 32; ++k) {
      const float wk = __shfl_sync(kFullMask, w, k);
      const int64_t pk = __shfl_sync(kFullMask, page, k);
      const int64_t rk = __shfl_sync(kFullMask, row, k);
      if (pk < 0) continue;
      const int d = lane * per;
      const int64_t in_page = rk % p.c.page_size;
      const int64_t ph = rk / p.c.page_size;
      const float sv = e4m3_decode(p.c.v_sf[(ph * (D / 16) + d / 16) * p.c.page_size + in_page]);
      for (int i = 0; i < per; ++i) {
        const uint32_t byte = p.c.v_packed[rk * (D / 2) + (d + i) / 2];
        acc[i] += wk * sv * e2m1_decode(((d + i) & 1) ? byte >> 4 : byte & 15u);
      }
    }
    m = m_new;
  }
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(kFullMask, l, o);
  const float inv = l > 0.0f ? 1.0f / (l * (p.c.v_gs ? __ldg(p.c.v_gs) : 1.0f)) : 0.0f;
  T* orow = static_cast<T*>(p.out) + item * D;
  for (int i = 0; i < per; ++i) orow[lane * per + i] = from_f32<T>(acc[i] * inv);
  if (p.lse && lane == 0) p.lse[item] = m == -INFINITY ? -INFINITY : m + logf(l);
}

}  // namespace

int64_t kv_attention_workspace(int sms, int64_t B, int64_t T, int Hq, int heads, int D) { return 0; }

cudaError_t launch_kv_attention(int dtype, const KvAttentionParams& p, int pdl,
                                cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((p.T * p.Hq + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return dtype == 0 ? cudaLaunchKernelEx(&cfg, kv_attention_simple_kernel<__nv_bfloat16>, p)
                    : cudaLaunchKernelEx(&cfg, kv_attention_simple_kernel<__half>, p);
}

}  // namespace fp4q
