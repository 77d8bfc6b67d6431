// beam_select.cu - the best continuations of every beam search of a batch: over
// beams k and tokens v, the n largest of
//     s_k + x_kv - log(sum_v exp(x_kv)).
//
// The logits are read once and bound the time.  Two kernels:
//   scan  a warp takes a part of one row, 512 logits (a group) at a time with the next ones on
//         their way, and leaves the largest of every group and the part's sum of exponentials;
//   join  a CTA per batch entry: every row's log-sum from its parts; the n groups whose
//         largest scores are the best; these groups' logits once more, n * 512 of them, and
//         of those the n best.
// A candidate outside the n best groups has the largest of each of these before it, so it is
// not among the n.  That holds with equal scores too, as groups and candidates are
// ordered alike: a score, then the lower beam, then the lower token.  The order is total, so
// results do not depend on what runs when.  (Keeping the n largest of every part
// while scanning costs more than the scan: 97 us with parts of 8192 logits, 273 us with
// longer ones, where a warp meets a new one of 16 in most of its first 30 steps.)
//
// The sum.  Exponentials are 2^(x log2(e) - M) against a whole number M of the lane, near
// the first logit above -infinity that it met, moved up where one lies 2^kSlack above it.  Sums of
// different lanes and parts differ by powers of two then, whose products are exact.
// log2(e) is taken as a sum of two floats: its rounding times x would be in every term of a
// row alike, and with it in comparisons between beams.
//
// The join's scores are sums of two floats (48 bits; the 64-bit units of this device do two
// operations a clock and took 350 us here), as is the logarithm.
#include <algorithm>

#include "async_copy.cuh"
#include "beam_launch.h"
#include "fp4q_launch.h"
#include "fused_common.cuh"

namespace fp4q {
namespace {

constexpr int kScanThreads = 128;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kScanCtas = 5;              // per SM
constexpr int kGroup = 512;               // logits of a warp's step, 16 a lane
constexpr int kJoinThreads = 512;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinList = 1024;
constexpr float kLog2eHi = 1.44269502f, kLog2eLo = 1.925963e-08f;
constexpr float kLn2Hi = 0.693147182f, kLn2Lo = -1.9046542e-09f;
constexpr float kSlack = 64.0f;
constexpr float kNoRef = -1.0e38f;        // M of a lane that has met no logit above -2^125
// Logits up to here count as -infinity (a mask of a type's lowest value; times log2(e) such
// a one leaves fp32's numbers).
constexpr float kLowest = -4.2535296e37f;

// A total order on floats as unsigned numbers; both zeros are one, and what is not
// a number must not come here.  0 is below -infinity's.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float(o ^ (o & 0x80000000u ? 0x80000000u : 0xffffffffu));
}
// A logit and its token: larger is earlier.
__device__ __forceinline__ uint64_t beam_key(float x, int token) {
  return static_cast<uint64_t>(ordered(x)) << 32 | static_cast<uint32_t>(~token);
}
__device__ __forceinline__ float key_high(uint64_t k) { return from_ordered(static_cast<uint32_t>(k >> 32)); }
__device__ __forceinline__ int key_token(uint64_t k) { return static_cast<int>(~static_cast<uint32_t>(k)); }

// Whether the row has candidates of its own logits.
__device__ __forceinline__ bool beam_live(const BeamParams& p, int row) {
  const bool here = FP4Q_IN_RANGE(p, p.scores + row, 4, p.scores, 4LL * p.B * p.K);
  if (!here || !isfinite(__ldg(p.scores + row))) return false;
  if (!p.finished || !FP4Q_IN_RANGE(p, p.finished + row, 1, p.finished, 1LL * p.B * p.K)) return true;
  return __ldg(p.finished + row) == 0;
}

// The 16 logits of a lane's step: one vector of a 16-bit type, two of fp32 (256 logits apart).
template <typename T> struct Logits {
  static constexpr int kVec = 16;
  static constexpr int kVectors = 1;
  __device__ static float2 pair(const Chunk (&c)[1], int i) { return Pair<T>::to_f32(c[0].u[i]); }
  __device__ static void set(Chunk& c, int i, const void* src) {
    const uint32_t v = __ldg(static_cast<const unsigned short*>(src));
    c.u[i / 2] = i & 1 ? (c.u[i / 2] & 0xffffu) | v << 16 : (c.u[i / 2] & 0xffff0000u) | v;
  }
  __device__ static uint32_t none() { return Pair<T>::from_f32(-INFINITY, -INFINITY); }
};
template <> struct Logits<float> {
  static constexpr int kVec = 8;
  static constexpr int kVectors = 2;
  __device__ static float2 pair(const Chunk (&c)[2], int i) {
    return make_float2(__uint_as_float(c[i / 4].u[2 * (i & 3)]), __uint_as_float(c[i / 4].u[2 * (i & 3) + 1]));
  }
  __device__ static void set(Chunk& c, int i, const void* src) { c.u[i] = __ldg(static_cast<const unsigned int*>(src)); }
  __device__ static uint32_t none() { return 0xff800000u; }
};

__device__ __forceinline__ float ex2_beam(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3_beam(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// 2^d for a whole number d <= 0 (0 below the normal numbers).
__device__ __forceinline__ float pow2_whole(float d) {
  return d < -126.0f ? 0.0f : __uint_as_float(static_cast<uint32_t>(static_cast<int>(d) + 127) << 23);
}

// Group `group` of row `row`: the lane's 16 logits, -infinity outside the row.  Elements are
// numbered from the 32-byte boundary at or before the row: number e is token e - lead, and
// whole vectors are aligned loads whatever the row's address is.
template <typename T>
__device__ __forceinline__ void load_group(const BeamParams& p, const T* base, int lead, int group, int lane,
                                           Chunk (&c)[Logits<T>::kVectors]) {
  using L = Logits<T>;
  constexpr int VEC = L::kVec, SIZE = sizeof(T);
  const int end = lead + p.V;
#pragma unroll
  for (int j = 0; j < L::kVectors; ++j) {
    const int e = group * kGroup + (j * 32 + lane) * VEC;
    const T* src = base + (e - lead);
    if (e >= lead && e + VEC <= end && FP4Q_IN_RANGE(p, src, 32, p.logits, beam_logits_extent(p, SIZE))) {
      c[j] = ld_stream_ro(src);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) c[j].u[i] = L::none();
      if (e < end && e + VEC > lead) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (e + i >= lead && e + i < end && FP4Q_IN_RANGE(p, src + i, SIZE, p.logits, beam_logits_extent(p, SIZE)))
            L::set(c[j], i, src + i);
      }
    }
  }
}
template <typename T> __device__ __forceinline__ const T* beam_row(const BeamParams& p, int row, int& lead) {
  const T* base = static_cast<const T*>(p.logits) + static_cast<int64_t>(row) * p.stride;
  lead = static_cast<int>(reinterpret_cast<uintptr_t>(base) & 31u) / static_cast<int>(sizeof(T));
  return base;
}

template <typename T>
__global__ void __launch_bounds__(kScanThreads, kScanCtas) beam_scan_kernel(const BeamParams p) {
  using L = Logits<T>;
  constexpr int NV = L::kVectors;
  constexpr int kAhead = 4 - NV;             // groups on their way

  const int lane = threadIdx.x & 31;
  const int64_t slot = static_cast<int64_t>(blockIdx.x) * kScanWarps + (threadIdx.x >> 5);
  griddep_wait();
  griddep_launch_dependents();
  if (slot >= static_cast<int64_t>(p.B) * p.K * p.parts) return;
  const int row = static_cast<int>(slot / p.parts), part = static_cast<int>(slot - static_cast<int64_t>(row) * p.parts);
  if (!beam_live(p, row)) return;
  int lead;
  const T* base = beam_row<T>(p, row, lead);
  const int g0 = static_cast<int>(static_cast<int64_t>(p.groups) * part / p.parts);
  const int g1 = static_cast<int>(static_cast<int64_t>(p.groups) * (part + 1) / p.parts);

  float ref = kNoRef, sum = 0.0f;
  auto work = [&](int group, const Chunk (&c)[NV]) {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = L::pair(c, i);
      top = max3_beam(top, x.x, x.y);                      // skips NaN
    }
    const uint32_t most = __reduce_max_sync(kFullMask, ordered(top));
    float* out = p.tops + static_cast<int64_t>(row) * p.groups + group;
    if (lane == 0 && FP4Q_IN_RANGE(p, out, 4, p.tops, 4LL * p.B * p.K * p.groups)) *out = from_ordered(most);
    // the reference moves where a term would pass 2^kSlack
    if (fmaf(top, kLog2eHi, -ref) > kSlack) {
      const float to = rintf(top * kLog2eHi);
      sum *= pow2_whole(ref - to);
      ref = to;
    }
    const float2 hi = make_float2(kLog2eHi, kLog2eHi), lo = make_float2(kLog2eLo, kLog2eLo);
    const float2 neg = make_float2(-ref, -ref);
    float2 part_sum = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = L::pair(c, i);
      float2 y = __ffma2_rn(x, lo, __ffma2_rn(x, hi, neg));
      y.x = ex2_beam(y.x);
      y.y = ex2_beam(y.y);
      part_sum = __fadd2_rn(part_sum, y);
    }
    sum += part_sum.x + part_sum.y;
  };
  Chunk c[kAhead + 1][NV];
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (g0 + i < g1) load_group<T>(p, base, lead, g0 + i, lane, c[i]);
  for (int g = g0; g < g1; g += kAhead + 1) {
#pragma unroll
    for (int i = 0; i <= kAhead; ++i) {
      if (g + i >= g1) break;
      if (g + i + kAhead < g1) load_group<T>(p, base, lead, g + i + kAhead, lane, c[(i + kAhead) % (kAhead + 1)]);
      work(g + i, c[i]);
    }
  }
  float m = ref;
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
  sum *= pow2_whole(fmaxf(ref - m, -200.0f));              // (a lane without a reference has 0, or NaN)
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
  if (lane == 0 && FP4Q_IN_RANGE(p, p.stats + slot, 8, p.stats, 8LL * p.B * p.K * p.parts))
    p.stats[slot] = make_float2(m, sum);
}

// --- sums of two floats: hi = rn(hi + lo) -------------------------------------
__device__ __forceinline__ float2 two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return make_float2(s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t)));
}
__device__ __forceinline__ float2 add_pairs(float2 a, float2 b) {
  const float2 s = two_sum(a.x, b.x);
  return two_sum(s.x, __fadd_rn(s.y, __fadd_rn(a.y, b.y)));
}
// m ln(2) + log(s) for a whole number m and s > 0: s = f 2^e with f in [0.707, 1.414], and
// log(f) = 2 artanh(z), z = (f - 1) / (f + 1), by its series, of which only the first term needs
// both floats.  Off by less than 2^-28 for |m| < 1000.
__device__ __forceinline__ float2 log_pair(float m, float2 s) {
  int e;
  float f = frexpf(s.x, &e) * 2.0f;
  --e;
  if (f > 1.4140625f) {
    f *= 0.5f;
    ++e;
  }
  const float lo = ldexpf(s.y, -e);
  const float num = __fsub_rn(f, 1.0f), den = __fadd_rn(f, 1.0f);
  const float den_lo = __fsub_rn(num, __fsub_rn(den, 2.0f));
  const float z = __fdiv_rn(num, den);
  const float z_lo = fmaf(-z, den_lo, fmaf(-z, den, num)) / den;
  const float zz = z * z;
  const float series = fmaf(zz, fmaf(zz, fmaf(zz, fmaf(zz, 2.0f / 11, 2.0f / 9), 2.0f / 7), 2.0f / 5), 2.0f / 3);
  const float rest = z * zz * series + 2.0f * z_lo + lo / f;
  const float E = m + static_cast<float>(e);
  const float a = __fmul_rn(E, kLn2Hi);
  const float2 t = two_sum(a, 2.0f * z);
  return two_sum(t.x, t.y + (rest + (fmaf(E, kLn2Hi, -a) + E * kLn2Lo)));
}

// A candidate of the join, or a group by its largest: a score of two floats in order, then
// the lower beam, then within the beam the larger key (logit and token, or logit and group).
struct Candidate {
  uint64_t score;
  uint64_t key;
  int k;
};
__device__ __forceinline__ bool before(const Candidate& a, const Candidate& b) {
  if (a.score != b.score) return a.score > b.score;
  return a.k != b.k ? a.k < b.k : a.key > b.key;
}

// What the CTA keeps of a set of candidates, and the n best of them.
struct CandidateList {
  uint64_t score[kJoinList], key[kJoinList];
  uint8_t k[kJoinList];
  int count;
  Candidate round_best[kJoinWarps];

  __device__ void add(const Candidate& x) {
    const int at = atomicAdd(&count, 1);
    if (at < kJoinList) {
      score[at] = x.score;
      key[at] = x.key;
      k[at] = static_cast<uint8_t>(x.k);
    }
  }
  // After a barrier: calls out(rank, some, candidate) once for every rank below n, by one
  // thread each.  All threads call it; `each` calls its argument for every candidate of the thread,
  // for where the list was too short for them: n rounds of a maximum then.
  template <typename Each, typename Out>
  __device__ void best(int n, int tid, Each each, Out out) {
    const int found = count;
    if (found <= kJoinList) {
      for (int i = tid; i < max(found, n); i += kJoinThreads) {
        Candidate x{};
        int rank = i;
        if (i < found) {
          x = Candidate{score[i], key[i], k[i]};
          rank = 0;
#pragma unroll 4
          for (int j = 0; j < found; ++j) {
            const uint64_t other = score[j];
            if (other == x.score && j != i)                // rare: the rest of the order counts
              rank += before(Candidate{other, key[j], k[j]}, x);
            else
              rank += other > x.score;
          }
        }
        if (rank < n) out(rank, i < found, x);
      }
      return;
    }
    Candidate last{~0ull, 0, -1};
    for (int r = 0; r < n; ++r) {
      Candidate top{0, 0, kBeamMostBeams};
      each([&](const Candidate& x) {
        if (before(last, x) && before(x, top)) top = x;
      });
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const Candidate y{__shfl_xor_sync(kFullMask, top.score, o), __shfl_xor_sync(kFullMask, top.key, o),
                          __shfl_xor_sync(kFullMask, top.k, o)};
        if (before(y, top)) top = y;
      }
      if ((tid & 31) == 0) round_best[tid >> 5] = top;
      __syncthreads();
      for (int w = 0; w < kJoinWarps; ++w)
        if (before(round_best[w], top)) top = round_best[w];
      if (tid == 0) out(r, top.k < kBeamMostBeams, top);
      if (top.k < kBeamMostBeams) last = top;
      __syncthreads();
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(kJoinThreads) beam_join_kernel(const BeamParams p) {
  using L = Logits<T>;
  __shared__ float2 lse[kBeamMostBeams];                   // NaN: the row has no candidates of its own
  __shared__ float score[kBeamMostBeams];
  __shared__ bool ended[kBeamMostBeams];
  __shared__ CandidateList groups, list;
  __shared__ uint32_t warp_top[kJoinWarps];
  __shared__ Candidate chosen[kBeamMostTake];
  __shared__ int n_chosen;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  if (tid == 0) groups.count = list.count = n_chosen = 0;
  // --- log-sums of the rows, a warp each
  for (int k = warp; k < p.K; k += kJoinWarps) {
    const int row = b * p.K + k;
    float s = __uint_as_float(0x7fc00000u);
    if (FP4Q_IN_RANGE(p, p.scores + row, 4, p.scores, 4LL * p.B * p.K)) s = __ldg(p.scores + row);
    bool over = false;
    if (p.finished && FP4Q_IN_RANGE(p, p.finished + row, 1, p.finished, 1LL * p.B * p.K))
      over = __ldg(p.finished + row) != 0;
    float2 total = make_float2(__uint_as_float(0x7fc00000u), 0.0f);
    if (isfinite(s) && !over) {
      const float2* st = p.stats + static_cast<int64_t>(row) * p.parts;
      const long long stat_bytes = 8LL * p.B * p.K * p.parts;
      float m = kNoRef;
      for (int i = lane; i < p.parts; i += 32)
        if (FP4Q_IN_RANGE(p, st + i, 8, p.stats, stat_bytes)) m = fmaxf(m, st[i].x);
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
      float2 sum = make_float2(0.0f, 0.0f);
      for (int i = lane; i < p.parts; i += 32)
        if (FP4Q_IN_RANGE(p, st + i, 8, p.stats, stat_bytes))
          sum = add_pairs(sum, make_float2(st[i].y * pow2_whole(fmaxf(st[i].x - m, -200.0f)), 0.0f));
#pragma unroll
      for (int o = 16; o; o >>= 1)
        sum = add_pairs(sum, make_float2(__shfl_xor_sync(kFullMask, sum.x, o), __shfl_xor_sync(kFullMask, sum.y, o)));
      if (sum.x > 0.0f && isfinite(sum.x) && isfinite(m)) total = log_pair(m, sum);
    }
    if (lane == 0) {
      lse[k] = total;
      score[k] = s;
      ended[k] = over && isfinite(s);
    }
  }
  __syncthreads();
  auto scored = [&](int k, float x) {
    const float2 l = lse[k];
    float2 v = two_sum(x, -l.x);
    v.y -= l.y;
    v = add_pairs(v, make_float2(score[k], 0.0f));
    return static_cast<uint64_t>(ordered(v.x)) << 32 | ordered(v.y);
  };

  // --- the n best groups; an ended beam counts as its first group, with its score as it is
  const int total = p.K * p.groups;
  const float* tops = p.tops + static_cast<int64_t>(b) * total;
  auto group = [&](int e, Candidate& x) {
    x.k = e / p.groups;
    const int g = e - x.k * p.groups;
    if (ended[x.k]) {
      x.key = beam_key(0.0f, 0);
      x.score = static_cast<uint64_t>(ordered(score[x.k])) << 32 | ordered(0.0f);
      return g == 0;
    }
    if (isnan(lse[x.k].x) || !FP4Q_IN_RANGE(p, tops + e, 4, p.tops, 4LL * p.B * p.K * p.groups)) return false;
    const float t = tops[e];
    if (!(t > kLowest)) return false;
    x.key = beam_key(t, g);
    x.score = scored(x.k, t);
    return true;
  };
  auto each_group = [&](auto f) {
    for (int e = tid; e < total; e += kJoinThreads) {
      Candidate x;
      if (group(e, x)) f(x);
    }
  };
  uint32_t mine = 0;
  each_group([&](const Candidate& x) { mine = max(mine, static_cast<uint32_t>(x.score >> 32)); });
  // A bound that n groups are not below and not many more than n: of the threads' largest, by
  // halving what lies between 0 and the largest of all until n to 2 n of them are left.
  uint32_t low = 0;
  if (__syncthreads_count(mine != 0) > p.n) {
    const uint32_t top = __reduce_max_sync(kFullMask, mine);
    if (lane == 0) warp_top[warp] = top;
    __syncthreads();
    uint32_t high = 0;                                     // fewer than n are above it
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) high = max(high, warp_top[w]);
    while (high - low > 1) {
      const uint32_t mid = low + (high - low) / 2;
      const int above = __syncthreads_count(mine >= mid);
      if (above >= p.n) low = mid; else high = mid;
      if (above >= p.n && above <= 2 * p.n) break;
    }
  }
  if (mine != 0 && mine >= low)
    each_group([&](const Candidate& x) {
      if (static_cast<uint32_t>(x.score >> 32) >= low) groups.add(x);
    });
  __syncthreads();
  groups.best(p.n, tid, each_group, [&](int rank, bool some, const Candidate& x) {
    if (!some) return;
    chosen[rank] = x;
    atomicAdd(&n_chosen, 1);
  });
  __syncthreads();

  // --- their logits: those that are not behind the n-th group's largest
  const int n_groups = n_chosen;
  const uint64_t least = n_groups == p.n ? chosen[p.n - 1].score : 0;
  auto each_logit = [&](auto f) {
    for (int i = warp; i < n_groups; i += kJoinWarps) {
      const int k = chosen[i].k;
      if (ended[k]) {
        if (lane == 0) f(Candidate{chosen[i].score, beam_key(0.0f, p.end_token), k});
        continue;
      }
      const int g = key_token(chosen[i].key);
      int lead;
      const T* base = beam_row<T>(p, b * p.K + k, lead);
      // most logits are far below: their scores need not be computed
      const float far_from = key_high(least), s0 = score[k], l0 = lse[k].x;
      const float far = least ? far_from - s0 + l0 - 1e-6f * (fabsf(far_from) + fabsf(s0) + fabsf(l0)) : kLowest;
      Chunk c[L::kVectors];
      load_group<T>(p, base, lead, g, lane, c);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float2 pr = L::pair(c, j / 2);
        const float x = j & 1 ? pr.y : pr.x;
        if (!(x > kLowest) || x < far) continue;
        const uint64_t s = scored(k, x);
        if (s < least) continue;
        f(Candidate{s, beam_key(x, g * kGroup + ((j / L::kVec) * 32 + lane) * L::kVec + j % L::kVec - lead), k});
      }
    }
  };
  each_logit([&](const Candidate& x) { list.add(x); });
  __syncthreads();
  const long long outs = static_cast<long long>(p.B) * p.n;
  list.best(p.n, tid, each_logit, [&](int rank, bool some, const Candidate& x) {
    const int64_t at = static_cast<int64_t>(b) * p.n + rank;
    const int token = some ? key_token(x.key) : -1;
    if (FP4Q_IN_RANGE(p, p.out_scores + at, 4, p.out_scores, 4 * outs))
      p.out_scores[at] = some ? key_high(x.score) : -INFINITY;
    if (FP4Q_IN_RANGE(p, p.out_parents + at, 4, p.out_parents, 4 * outs))
      p.out_parents[at] = some ? b * p.K + x.k : -1;
    if (FP4Q_IN_RANGE(p, p.out_tokens + at, 4, p.out_tokens, 4 * outs)) p.out_tokens[at] = token;
    if (p.out_finished && FP4Q_IN_RANGE(p, p.out_finished + at, 1, p.out_finished, outs))
      p.out_finished[at] = some && (ended[x.k] || token == p.end_token);
  });
}

}  // namespace

// Parts of a row: four times as many warps as the device holds at a time, of whole groups.
constexpr int kScanWarpsPerSm = 4 * kScanCtas * kScanWarps;

static int64_t groups_of(int64_t V) { return (V + 15 + kGroup - 1) / kGroup; }   // of a row of any alignment
static int64_t part_slots(int sms, int64_t rows) { return std::max<int64_t>(rows, static_cast<int64_t>(sms) * kScanWarpsPerSm); }

void beam_shape(int sms, BeamParams* p) {
  const int64_t rows = static_cast<int64_t>(p->B) * p->K;
  p->groups = static_cast<int>(groups_of(p->V));
  p->parts = static_cast<int>(std::min<int64_t>(p->groups, part_slots(sms, rows) / rows));
}

int64_t beam_stats_bytes(const BeamParams& p) { return 8LL * p.B * p.K * p.parts; }

// The parts' statistics, of which rows * parts <= part_slots, then the groups' largest.
int64_t beam_workspace(int sms, int64_t B, int64_t K, int64_t V) {
  const int64_t rows = B * K;
  return std::min(rows * groups_of(V), part_slots(sms, rows)) * 8 + (rows * groups_of(V) * 4 + 15) / 16 * 16;
}

template <typename T>
static cudaError_t launch_type(const BeamParams& p, int pdl, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(p.B) * p.K * p.parts + kScanWarps - 1) / kScanWarps));
  cfg.blockDim = dim3(kScanThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, beam_scan_kernel<T>, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(p.B));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.numAttrs = 1;                              // its launch overlaps the first kernel
  return cudaLaunchKernelEx(&cfg, beam_join_kernel<T>, p);
}

cudaError_t launch_beam_select(int dtype, const BeamParams& p, int pdl, cudaStream_t stream) {
  return dtype == 0   ? launch_type<__nv_bfloat16>(p, pdl, stream)
         : dtype == 1 ? launch_type<__half>(p, pdl, stream)
                      : launch_type<float>(p, pdl, stream);
}

}  // namespace fp4q
