// kv_attention.cu - attention over the paged NVFP4 key/value cache: choice of
// kernel and launch.

#include <mutex>

#include "fp4q_launch.h"
#include "kv_decode.cuh"
#include "kv_prefill.cuh"

namespace fp4q {
namespace {

// Query rows of a key/value head that one item of the decode kernel covers: 8 where a
// sequence has no more of them, else 16 (32 sequences of 4096 tokens, 8 heads of 128:
// 8 rows 46 us, 16 rows 63 us; two tiles of 8 for 16 rows would read every key twice).
int decode_tiles(int64_t B, int64_t T, int group) { return T * group <= 8 * B ? 1 : 2; }

// CTAs of the cluster that takes one item each, 0 where the keys are to be split evenly
// over all CTAs instead (by the table's width: the lengths are on the device).  A CTA
// has at most 16 units of keys then; an item gets more CTAs than that asks for as long
// as all run at once and have a unit each, and where even the fewest do not run at
// once it has to be one each (short sequences, which the hardware then deals out).
// One sequence of 1000 tokens, 2 key/value heads: 5.8 us on the device and one launch,
// against 8.6 us and two.
constexpr int kClusterKeys = kDecUnit * 16;
template <int D, int NT>
int cluster_of(int sms, int64_t B, int64_t T, int group, int heads, int64_t keys) {
  const int64_t items = decode_row_slots(B, T, group, 8 * NT) * heads;
  const int64_t at_once = static_cast<int64_t>(sms) * DecodeShape<D, NT>::kCtas;
  int64_t c = 1;
  while (c < kDecCluster && keys > c * kClusterKeys) c *= 2;
  if (keys > c * kClusterKeys || (c > 1 && items * c > at_once) || items * c > INT32_MAX) return 0;
  while (c < kDecCluster && items * c * 2 <= at_once && keys >= c * 2 * kDecUnit) c *= 2;
  return static_cast<int>(c);
}

template <typename T, int D, int NT>
cudaError_t launch_decode(const KvAttentionParams& p, int pdl, cudaStream_t stream) {
  using S = DecodeShape<D, NT>;
  static_assert(S::kSmemCluster <= 48 * 1024, "needs no raised shared-memory limit");
  const int sms = sm_count_current_device(), ctas = sms * S::kCtas;
  const int64_t slots = decode_row_slots(p.B, p.T, p.group, S::kRows) * p.c.heads;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  const int cluster = cluster_of<D, NT>(sms, p.B, p.T, p.group, p.c.heads, p.max_pages * p.c.page_size);
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kDecThreads);
  cfg.stream = stream;
  if (cluster) {
    cfg.gridDim = dim3(static_cast<unsigned>(slots * cluster));
    cfg.dynamicSmemBytes = S::kSmemCluster;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kv_decode_kernel<T, D, NT, true>, p);
  }
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.attrs = attr + 1;
  cfg.numAttrs = pdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_decode_kernel<T, D, NT, false>, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(slots), S::kRows);
  // few items, many parts each: more threads per row take them side by side
  cfg.blockDim = dim3(slots * 8 <= ctas ? kJoinMost : 128);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;                              // its launch overlaps the first kernel
  return cudaLaunchKernelEx(&cfg, kv_decode_join_kernel<T, D, NT>, p, ctas);
}

// Rows of a key/value head per sequence (on average: the lengths are on the device)
// from which on the 256-row items are used.  32 sequences of 4096 tokens, 8 heads of
// 128, 256-row items against 16-row items: 32 rows 164 / 104 us, 48 rows 141 / 143 us,
// 64 rows 141 / 183 us, 128 rows 145 / 340 us; heads of 64: 111 / 101 us at 48 rows,
// 112 / 126 us at 64.
constexpr int kPrefillRows = 64;
bool use_prefill(int64_t B, int64_t T, int group) { return T * group >= kPrefillRows * B; }

// Ranges of keys that an item is cut into: so many that every SM gets two CTAs, each
// range being four steps at least (by the table's width).
int prefill_splits(int sms, int64_t B, int64_t T, int group, int heads, int64_t keys) {
  const int64_t items = prefill_row_slots(B, T, group) * heads;
  int64_t s = (2 * sms + items - 1) / items;
  s = s < 8 ? s : 8;
  while (s > 1 && keys < 4 * kPreKeys * s) --s;
  return static_cast<int>(s);
}

template <typename T, int D>
cudaError_t launch_prefill(const KvAttentionParams& p, int pdl, cudaStream_t stream) {
  using S = PrefillShape<D>;
  {
    // a per-device function attribute, set once
    static bool done[64] = {};
    static std::mutex mu;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (!done[dev]) {
      // the warpgroups' register budgets must be covered by the launch's registers
      cudaFuncAttributes fa;
      e = cudaFuncGetAttributes(&fa, kv_prefill_kernel<T, D>);
      if (e != cudaSuccess) return e;
      if (fa.numRegs * kPreThreads < kPreRegs) return cudaErrorInvalidConfiguration;
      e = cudaFuncSetAttribute(kv_prefill_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  const int splits = prefill_splits(sm_count_current_device(), p.B, p.T, p.group, p.c.heads,
                                    p.max_pages * p.c.page_size);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(prefill_row_slots(p.B, p.T, p.group) * p.c.heads),
                     static_cast<unsigned>(splits));
  cfg.blockDim = dim3(kPreThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_prefill_kernel<T, D>, p, splits);
  if (e != cudaSuccess || splits == 1) return e;
  cfg.gridDim = dim3(static_cast<unsigned>((p.T * p.Hq * (D / 4) + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_prefill_join_kernel<T, D>, p, splits);
}

template <typename T>
cudaError_t launch_type(const KvAttentionParams& p, int pdl, cudaStream_t stream) {
  if (use_prefill(p.B, p.T, p.group))
    return p.c.D == 128 ? launch_prefill<T, 128>(p, pdl, stream) : launch_prefill<T, 64>(p, pdl, stream);
  const int nt = decode_tiles(p.B, p.T, p.group);
  if (p.c.D == 128)
    return nt == 1 ? launch_decode<T, 128, 1>(p, pdl, stream) : launch_decode<T, 128, 2>(p, pdl, stream);
  return nt == 1 ? launch_decode<T, 64, 1>(p, pdl, stream) : launch_decode<T, 64, 2>(p, pdl, stream);
}

template <int D, int NT>
int64_t decode_workspace(int sms, int64_t B, int64_t T, int group, int heads, int64_t keys) {
  using S = DecodeShape<D, NT>;
  if (cluster_of<D, NT>(sms, B, T, group, heads, keys)) return 0;
  return 4LL * (2LL * sms * S::kCtas * S::kPart) + 8LL * decode_row_slots(B, T, group, S::kRows) * heads;
}

}  // namespace

int64_t kv_attention_workspace(int sms, int64_t B, int64_t T, int Hq, int heads, int D, int64_t keys) {
  const int group = Hq / heads;
  if (B == 0 || T == 0) return 0;
  if (use_prefill(B, T, group)) {
    const int64_t splits = prefill_splits(sms, B, T, group, heads, keys);
    return splits > 1 ? splits * T * Hq * (D + 2) * 4 : 0;
  }
  const int nt = decode_tiles(B, T, group);
  if (D == 128)
    return nt == 1 ? decode_workspace<128, 1>(sms, B, T, group, heads, keys)
                   : decode_workspace<128, 2>(sms, B, T, group, heads, keys);
  return nt == 1 ? decode_workspace<64, 1>(sms, B, T, group, heads, keys)
                 : decode_workspace<64, 2>(sms, B, T, group, heads, keys);
}

cudaError_t launch_kv_attention(int dtype, const KvAttentionParams& p, int pdl,
                                cudaStream_t stream) {
  return dtype == 0 ? launch_type<__nv_bfloat16>(p, pdl, stream) : launch_type<__half>(p, pdl, stream);
}

}  // namespace fp4q
