// kv_attention_launch.cuh - attention over the paged NVFP4 key/value cache: choice of
// kernel and launch.
#pragma once

#include <algorithm>
#include <cmath>
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

// The choices below compare times in microseconds, estimated from the sizes (the lengths
// are on the device: every sequence counts with the average number of rows and the
// table's width).  Their constants are fits to timed calls whose tables were as wide as
// their longest sequence and whose sequences had the same number of rows; what is said of
// them holds for such calls.  Elsewhere the choice can be far off.  Wider tables than the
// lengths: 64 sequences of 200 keys, 8 heads of 128, 13.1 us with a table of 200 keys, 21.1
// of 8192; one of 80 rows and keys 7.0 and 18.4.  Rows that differ: one sequence of 1000
// rows and 60 of one, 4000 keys each, 278 us in one call, 62 + 64 in two.
int64_t row_tiles(int64_t B, int64_t T, int group, int rows) {
  const int64_t each = (T * group + B - 1) / B;
  return B * ((each + rows - 1) / rows);
}

// A 16-key tile in a CTA that has an SM to itself, and per CTA where several share one;
// an item's setup, and its join in a cluster; the even split's two kernels, an item's
// share of them, and the second one's time per part of an item; how many of an SM's places
// clusters find.
struct DecodeTimes {
  double alone, shared, item, peers, split, split_item, part, places;
};
template <int D, int NT>
constexpr DecodeTimes kDecTimes =
    D == 64 ? (NT == 1 ? DecodeTimes{0.076, 0.033, 4.0, 1.8, 6.5, 2.0, 0.09, 0.95}
                       : DecodeTimes{0.101, 0.044, 4.0, 4.3, 8.8, 3.1, 0.12, 0.95})
            : (NT == 1 ? DecodeTimes{0.084, 0.063, 4.7, 1.9, 8.4, 3.0, 0.03, 0.95}
                       : DecodeTimes{0.099, 0.065, 5.7, 4.3, 10.9, 4.4, 0.04, 0.88});

constexpr double kEvenSplit = 0.95;

// CTAs that share an item (more than one as a cluster, joined in shared memory; the
// hardware deals the items out), or 0 where the keys are split evenly over all CTAs and
// joined by a second kernel.  1055 calls of 1 to 128 sequences with 100 to 16000 keys (all
// of them, or from 0.3 of the longest up), each timed with every choice: the one made is
// 2.2 % slower than the best on average and 30 % at most.  The even split's estimate is
// taken at kEvenSplit of itself, as it gains where lengths differ: that costs those calls
// nothing, and 100 sequences of 400 to 10000 keys, 8 heads of 128, take 124 us instead of
// 155.  One CTA an item against the even split: 128 sequences of 2000 keys, 24 heads of 64,
// 112 / 144 us, 16 of 8000 with 4 rows each 74 / 59; 8 CTAs: one sequence of 1000 keys, 2
// heads of 128, 6.1 / 8.9 us, 4 of 16000 with 8 heads 26.2 / 22.5.
template <int D, int NT>
int cluster_of(int sms, int64_t B, int64_t T, int group, int heads, int64_t keys, double* cost = nullptr) {
  constexpr DecodeTimes t = kDecTimes<D, NT>;
  constexpr int kCtas = DecodeShape<D, NT>::kCtas;
  const double items = static_cast<double>(row_tiles(B, T, group, 8 * NT)) * heads;
  const int64_t units = (keys + kDecUnit - 1) / kDecUnit;
  int best = 0;
  // the even split follows the lengths, where a cluster takes as long as its own: the more
  // they differ the better for it
  double least = kEvenSplit * (t.split + items * (t.split_item + keys / 16.0 * t.shared) / sms +
                               t.part * std::fmin(sms * kCtas / items, static_cast<double>(units)));
  for (const int c : {1, 2, 3, 4, 6, 8}) {
    if (decode_row_slots(B, T, group, 8 * NT) * heads > INT32_MAX / c) break;
    const double per_sm = items * c / sms;
    const double side = std::fmin(std::ceil(per_sm), kCtas);
    const double waves = std::fmax(1.0, per_sm / (kCtas * (c > 1 ? t.places : 1.0)));
    const double tiles = static_cast<double>((units + c - 1) / c * (kDecUnit / 16));
    const double x = 0.5 * (waves + std::ceil(waves)) *
                     (t.item + (c > 1 ? t.peers : 0.0) + tiles * std::fmax(t.alone, side * t.shared));
    if (x < least) least = x, best = c;
  }
  if (cost) *cost = least;
  return best;
}

// Keys that the choices count a call's sequences with.
inline int64_t keys_of(const KvAttentionParams& p) {
  return kv_attention_keys(p.B, p.T, p.max_pages * p.c.page_size, p.window);
}

template <typename T, int D, int NT, int MODE>
cudaError_t launch_decode(const KvAttentionParams& p, int pdl, cudaStream_t stream) {
  using S = DecodeShape<D, NT>;
  static_assert(S::kSmemCluster <= 48 * 1024, "needs no raised shared-memory limit");
  const int sms = sm_count_current_device(), ctas = sms * S::kCtas;
  const int64_t slots = decode_row_slots(p.B, p.T, p.group, S::kRows) * p.c.heads;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  const int cluster = cluster_of<D, NT>(sms, p.B, p.T, p.group, p.c.heads, keys_of(p));
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
    return cudaLaunchKernelEx(&cfg, kv_decode_kernel<T, D, NT, true, MODE>, p);
  }
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.attrs = attr + 1;
  cfg.numAttrs = pdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_decode_kernel<T, D, NT, false, MODE>, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(slots), S::kRows);
  // few items, many parts each: more threads per row take them side by side
  cfg.blockDim = dim3(slots * 8 <= ctas ? kJoinMost : 128);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;                              // its launch overlaps the first kernel
  return cudaLaunchKernelEx(&cfg, kv_decode_join_kernel<T, D, NT>, p, ctas);
}

// Constants as above, from calls timed with both kernels and with 1 to 8 ranges of keys
// (heads of 64 and 128, 1 to 100 sequences of 1 to 4000 rows and 48 to 60000 keys).  Over
// 831 of them the choice of kernel is 0.7 % slower than the faster one on average and 30 %
// at most (a fixed limit of 64 rows: 6.5 % and a factor of 2.1); over 214 the ranges are
// 11 % slower than the best of 1 to 8 at most.  8 heads of 128, 4 query heads each, 16-row
// items against 256-row items: one sequence of 80 rows and keys 6.7 / 11.8 us, of 320 over
// 1320 keys 43 / 26; one range against two: 2048 rows and keys 43 / 100 us, 500 over 4000
// keys 62 / 46.
constexpr double kPreItem = 8.0, kPreJoin = 4.0, kPreJoinBytes = 5e6;   // per CTA; per join, bytes per us
constexpr int kPreMostSplits = 32;

// A wave is one CTA per SM: its setup and its steps.
double prefill_cost(int sms, int64_t items, int64_t rows, int D, int64_t keys, int splits) {
  const int64_t steps = ((keys + splits - 1) / splits + kPreKeys - 1) / kPreKeys;
  const int64_t waves = (items * splits + sms - 1) / sms;
  return waves * (kPreItem + steps * (D == 128 ? 1.7 : 1.3)) +
         (splits > 1 ? kPreJoin + rows * D * 8.0 * splits / kPreJoinBytes : 0.0);
}

// Ranges of keys that an item is cut into: the fewest of the best.
int prefill_splits(int sms, int64_t B, int64_t T, int Hq, int heads, int D, int64_t keys, double* cost) {
  const int64_t items = row_tiles(B, T, Hq / heads, kPreRows) * heads;
  int best = 1;
  double least = prefill_cost(sms, items, T * Hq, D, keys, 1);
  // more waves than four only add CTAs to set up
  for (int s = 2; s <= kPreMostSplits && (s - 1) * kPreKeys < keys && items * s <= 4LL * sms; ++s) {
    const double c = prefill_cost(sms, items, T * Hq, D, keys, s);
    if (c < least) least = c, best = s;
  }
  if (cost) *cost = least;
  return best;
}

// Up to 16 rows of a key/value head per sequence are one item of the decode kernel.
bool use_prefill(int sms, int64_t B, int64_t T, int Hq, int heads, int D, int64_t keys) {
  const int group = Hq / heads;
  if (T * group <= 16 * B) return false;
  double prefill = 0.0, decode = 0.0;
  prefill_splits(sms, B, T, Hq, heads, D, keys, &prefill);
  if (D == 128) cluster_of<128, 2>(sms, B, T, group, heads, keys, &decode);
  else cluster_of<64, 2>(sms, B, T, group, heads, keys, &decode);
  return prefill < decode;
}

template <typename T, int D, int MODE>
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
      e = cudaFuncGetAttributes(&fa, kv_prefill_kernel<T, D, MODE>);
      if (e != cudaSuccess) return e;
      if (fa.numRegs * kPreThreads < kPreRegs) return cudaErrorInvalidConfiguration;
      e = cudaFuncSetAttribute(kv_prefill_kernel<T, D, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
      if (e != cudaSuccess) return e;
      done[dev] = true;
    }
  }
  const int splits = prefill_splits(sm_count_current_device(), p.B, p.T, p.Hq, p.c.heads, D, keys_of(p), nullptr);
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_prefill_kernel<T, D, MODE>, p, splits);
  if (e != cudaSuccess || splits == 1) return e;
  cfg.gridDim = dim3(static_cast<unsigned>((p.T * p.Hq * (D / 4) + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_prefill_join_kernel<T, D>, p, splits);
}

// PRE, DEC: the kinds of logits of the two kernels (KvLogits).
template <typename T, int PRE, int DEC>
cudaError_t launch_type(const KvAttentionParams& p, int pdl, cudaStream_t stream) {
  if (use_prefill(sm_count_current_device(), p.B, p.T, p.Hq, p.c.heads, p.c.D, keys_of(p)))
    return p.c.D == 128 ? launch_prefill<T, 128, PRE>(p, pdl, stream) : launch_prefill<T, 64, PRE>(p, pdl, stream);
  const int nt = decode_tiles(p.B, p.T, p.group);
  if (p.c.D == 128)
    return nt == 1 ? launch_decode<T, 128, 1, DEC>(p, pdl, stream) : launch_decode<T, 128, 2, DEC>(p, pdl, stream);
  return nt == 1 ? launch_decode<T, 64, 1, DEC>(p, pdl, stream) : launch_decode<T, 64, 2, DEC>(p, pdl, stream);
}
// dtype 0 = bf16, 1 = fp16.
template <int PRE, int DEC>
cudaError_t launch_attention(int dtype, const KvAttentionParams& p, int pdl, cudaStream_t stream) {
  return dtype == 0 ? launch_type<__nv_bfloat16, PRE, DEC>(p, pdl, stream) : launch_type<__half, PRE, DEC>(p, pdl, stream);
}

}  // namespace
}  // namespace fp4q
