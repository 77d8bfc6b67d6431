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
// Beyond 2^30 (masks of -1e10 or -1e30) floats are 128 or more apart, and M's own steps pass what
// an exponent may be.  There M is 2 x and the terms 2^(2 x - M): 1 for the logit that set it,
// 0 for every smaller one, as e^-128 is, too, next to 1; and a larger one moves M.  Both kinds of
// M are ordered alike (|x log2(e)| < 2^31 below, 2 |x| > 2^31 above) and differ by more than
// 2^28, so that sums with different ones are still joined by the same powers of two, then 0.
// (64 x 8 beams of 131072 logits take 0.7 us more for it, 35.5.)
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
constexpr int kScanCtas = 8;              // per SM
constexpr int kGroup = 512;               // logits of a warp's step, 16 a lane
constexpr int kJoinThreads = 512;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinList = 1024;
constexpr int kJoinPerWarp = kBeamMostTake / kJoinWarps + 1;
constexpr int kJoinGroups = 160;          // groups that are looked through without choosing among them
constexpr int kJoinEarly = 2560;          // groups whose largest is read at once
constexpr float kLog2eHi = 1.44269502f, kLog2eLo = 1.925963e-08f;
constexpr float kLn2Hi = 0.693147182f, kLn2Lo = -1.9046542e-09f;
constexpr float kSlack = 64.0f;
constexpr float kNoRef = -1.0e38f;        // M of a lane that has met no logit above -2^125
constexpr float kFar = 1073741824.0f;     // 2^30: logits beyond it (of either sign) are far
constexpr float kFarRef = 2147483648.0f;  // 2^31: so are M beyond it
constexpr float kFarBy = 2.0f, kFarByLo = 7.1746481e-43f;   // in log2(e)'s place (2^-140, as 0 would make NaN of infinities)
// Logits up to here count as -infinity (a mask of a type's lowest value; times log2(e) such
// a one leaves fp32's numbers).
constexpr float kLowest = -4.2535296e37f;
constexpr float kHighestRef = -2.0f * kLowest;   // M of the largest logit that a row may have

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

// What makes exponents of logits next to M.
__device__ __forceinline__ float scale_of(float M) { return fabsf(M) > kFarRef ? kFarBy : kLog2eHi; }

// The largest of the lanes' values, none of which is NaN.
__device__ __forceinline__ float warp_max(float x) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}

// Group `group` of row `row`: the lane's 16 logits, -infinity outside the row.  Elements are
// numbered from the 32-byte boundary at or before the row: number e is token e - lead, and
// whole vectors are aligned loads whatever the row's address is.
template <typename T>
__device__ __forceinline__ void load_group(const BeamParams& p, const T* base, int lead, int group, int lane,
                                           Chunk (&c)[Logits<T>::kVectors]) {
  using L = Logits<T>;
  constexpr int VEC = L::kVec;
  const int end = lead + p.V;
#pragma unroll
  for (int j = 0; j < L::kVectors; ++j) {
    const int e = group * kGroup + (j * 32 + lane) * VEC;
    const T* src = base + (e - lead);
    if (e >= lead && e + VEC <= end && FP4Q_IN_RANGE(p, src, 32, p.logits, beam_logits_extent(p, sizeof(T)))) {
      c[j] = ld_stream_ro(src);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) c[j].u[i] = L::none();
      if (e < end && e + VEC > lead) {
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          if (e + i >= lead && e + i < end && FP4Q_IN_RANGE(p, src + i, sizeof(T), p.logits, beam_logits_extent(p, sizeof(T))))
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
  constexpr int kAhead = 3 - NV;             // groups on their way

  const int lane = threadIdx.x & 31;
  const int64_t slot = static_cast<int64_t>(blockIdx.x) * kScanWarps + (threadIdx.x >> 5);
  griddep_wait();
  griddep_launch_dependents();
  if (slot >= static_cast<int64_t>(p.B) * p.K * p.parts) return;
  const int row = static_cast<int>(slot / p.parts), part = static_cast<int>(slot - static_cast<int64_t>(row) * p.parts);
  int lead;
  const T* base = beam_row<T>(p, row, lead);
  const int g0 = static_cast<int>(static_cast<int64_t>(p.groups) * part / p.parts);
  const int g1 = static_cast<int>(static_cast<int64_t>(p.groups) * (part + 1) / p.parts);

  // groups that lie in the row as a whole
  const int whole0 = lead ? 1 : 0, whole1 = (lead + p.V) / kGroup;
  const T* mine = base - lead + lane * L::kVec;
  auto load = [&](int g, Chunk (&c)[NV]) {
    if (g >= whole0 && g < whole1) {
      const T* src = mine + static_cast<int64_t>(g) * kGroup;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (FP4Q_IN_RANGE(p, src + 32 * j * L::kVec, 32, p.logits, beam_logits_extent(p, sizeof(T))))
          c[j] = ld_stream_ro(src + 32 * j * L::kVec);
    } else if (g < g1) {
      load_group<T>(p, base, lead, g, lane, c);
    }
  };
  float ref = kNoRef, sum = 0.0f, keep = 0.0f;
  float by = kLog2eHi;                                     // scale_of(ref), once there is one
  auto flush = [&](int first, int n) {                     // lane i: the largest of group first + i
    float* out = p.tops + static_cast<int64_t>(row) * p.groups + first + lane;
    if (lane < n && FP4Q_IN_RANGE(p, out, 4, p.tops, 4LL * p.B * p.K * p.groups)) *out = keep;
  };
  auto work = [&](int g, const Chunk (&c)[NV]) {
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = L::pair(c, i);
      top = max3_beam(top, x.x, x.y);                      // skips NaN
    }
    const float most = warp_max(top);
    const int at = (g - g0) & 31;
    if (lane == at) keep = most;
    if (at == 31) flush(g - 31, 32);
    // the reference moves where a term would pass 2^kSlack
    if (fmaf(top, by, -ref) > kSlack) {
      const float to = fabsf(top) > kFar ? kFarBy * top : rintf(top * kLog2eHi);
      sum *= pow2_whole(ref - to);
      ref = to;
      by = scale_of(to);
    }
    const float by_lo = by == kFarBy ? kFarByLo : kLog2eLo;
    const float2 hi = make_float2(by, by), lo = make_float2(by_lo, by_lo);
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
  for (int i = 0; i < kAhead; ++i) load(g0 + i, c[i]);
  if (!beam_live(p, row)) return;                          // (looked up beside the first logits)
  for (int g = g0; g < g1; g += kAhead + 1) {
#pragma unroll
    for (int i = 0; i <= kAhead; ++i) {
      if (g + i >= g1) break;
      load(g + i + kAhead, c[(i + kAhead) % (kAhead + 1)]);
      work(g + i, c[i]);
    }
  }
  const int left = (g1 - g0) & 31;
  flush(g1 - left, left);
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
// m ln(2) + log(s) for a whole number m and a normal s > 0: s = f 2^e with f in [0.707, 1.414],
// and log(f) = 2 artanh(z), z = (f - 1) / (f + 1), by its series, of which only the first term
// needs both floats (z itself may be off: z_lo is what is left of the division).  Off by less than
// 2^-28 for |m| < 1000.
__device__ __forceinline__ float2 log_pair(float m, float2 s) {
  const uint32_t bits = __float_as_uint(s.x);
  int e = static_cast<int>(bits >> 23) - 127;
  float f = __uint_as_float((bits & 0x007fffffu) | 0x3f800000u);
  if (f > 1.4140625f) {
    f *= 0.5f;
    ++e;
  }
  const float lo = s.y * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  const float num = __fsub_rn(f, 1.0f), den = __fadd_rn(f, 1.0f);
  const float den_lo = __fsub_rn(num, __fsub_rn(den, 2.0f));
  const float z = __fdividef(num, den);
  const float z_lo = __fdividef(fmaf(-z, den_lo, fmaf(-z, den, num)), den);
  const float zz = z * z;
  const float series = fmaf(zz, fmaf(zz, fmaf(zz, fmaf(zz, 2.0f / 11, 2.0f / 9), 2.0f / 7), 2.0f / 5), 2.0f / 3);
  const float rest = z * zz * series + 2.0f * z_lo + __fdividef(lo, f);
  const float E = m + static_cast<float>(e);
  const float a = __fmul_rn(E, kLn2Hi);
  const float2 t = two_sum(a, 2.0f * z);
  return two_sum(t.x, t.y + (rest + (fmaf(E, kLn2Hi, -a) + E * kLn2Lo)));
}
// The same of a row's sum: beyond 2^23 M apart from the logarithm, which its rounding would
// swallow, and far from 0 as the logit that it is.
__device__ __forceinline__ float2 log_sum(float m, float2 s) {
  const bool apart = fabsf(m) >= 8388608.0f;
  float2 l = log_pair(apart ? 0.0f : m, s);
  if (apart) {
    const bool far = fabsf(m) > kFarRef;
    const float a = __fmul_rn(m, far ? 1.0f / kFarBy : kLn2Hi);
    l = add_pairs(two_sum(a, far ? 0.0f : fmaf(m, kLn2Hi, -a) + m * kLn2Lo), l);
  }
  return l;
}

// s + (x - l) in order, to the 53 bits of a 64-bit number: two floats can hold a large one and
// what is left of a small one far below, by which tokens filled with -1e30 would be ordered by
// their beams' scores where they are as far behind in all of them.
__device__ __forceinline__ uint64_t pair_score(float x, float2 l, float s) {
  float2 v = two_sum(x, -l.x);
  v.y -= l.y;
  v = add_pairs(v, make_float2(s, 0.0f));
  const float top = __uint_as_float(__float_as_uint(v.x) & 0x7f800000u);   // the power of two in it
  const float step = top * 2.7939677e-9f;                                 // 1.5 * 2^-29: steps of 2^-52 of that
  if (fabsf(v.y) < top * 9.3132257e-10f) v.y = __fsub_rn(__fadd_rn(v.y, step), step);
  return static_cast<uint64_t>(ordered(v.x)) << 32 | ordered(v.y);
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
  __device__ Candidate at(int i) const { return Candidate{score[i], key[i], k[i]}; }
  // Calls out(rank, some, candidate) once for every rank below n, by one thread each; after
  // a barrier, with at most kJoinList candidates.
  template <typename Out> __device__ void best(int n, int tid, Out out) {
    const int found = count;
    for (int i = tid; i < max(found, n); i += kJoinThreads) {
      Candidate x{};
      int rank = i;
      if (i < found) {
        x = at(i);
        rank = 0;
        int same = 0;
#pragma unroll 4
        for (int j = 0; j < found; ++j) {
          const uint64_t other = score[j];
          rank += other > x.score;
          same += other == x.score;
        }
        if (same > 1) {                                    // rare: the rest of the order counts
          rank = 0;
#pragma unroll 1
          for (int j = 0; j < found; ++j) rank += before(at(j), x);
        }
      }
      if (rank < n) out(rank, i < found, x);
    }
  }
  // The same of any number of candidates, which `each` calls its argument for, thread by
  // thread: n rounds of a maximum.  All threads call it.
  template <typename Each, typename Out> __device__ void best_in_rounds(int n, int tid, Each each, Out out) {
    Candidate last{~0ull, 0, -1};
    for (int r = 0; r < n; ++r) {
      Candidate top{0, 0, kBeamMostBeams};
      each([&](const Candidate& x) {
        if (before(last, x) && before(x, top)) top = x;
      });
#pragma unroll 1
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
  __shared__ CandidateList list;
  __shared__ float early[kJoinEarly];                      // groups' largest,
  __shared__ uint32_t early_score[kJoinEarly];             // and the first floats of their scores in order
  __shared__ uint32_t tops_of_warps[kJoinWarps * kJoinPerWarp];
  __shared__ Candidate chosen[kJoinGroups];
  __shared__ int n_chosen;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  // everything that the log-sums do not change is on its way before they are computed
  auto row_score = [&](int k) {
    const float* s = p.scores + static_cast<int64_t>(b) * p.K + k;
    return k < p.K && FP4Q_IN_RANGE(p, s, 4, p.scores, 4LL * p.B * p.K) ? __ldg(s) : __uint_as_float(0x7fc00000u);
  };
  auto row_ended = [&](int k) {
    const uint8_t* f = p.finished + static_cast<int64_t>(b) * p.K + k;
    return p.finished && k < p.K && FP4Q_IN_RANGE(p, f, 1, p.finished, 1LL * p.B * p.K) && __ldg(f) != 0;
  };
  auto stat = [&](int k, int i) {
    const float2* st = p.stats + (static_cast<int64_t>(b) * p.K + k) * p.parts + i;
    const bool here = k < p.K && i < p.parts && FP4Q_IN_RANGE(p, st, 8, p.stats, 8LL * p.B * p.K * p.parts);
    return here ? *st : make_float2(kNoRef, 0.0f);
  };
  const float s_first = row_score(warp);
  const bool over_first = row_ended(warp);
  const float2 stat_first = stat(warp, lane);
  const int total = p.K * p.groups;
  const float* tops = p.tops + static_cast<int64_t>(b) * total;
  auto group_top = [&](int e) {                            // (of rows without candidates: any bytes)
    return FP4Q_IN_RANGE(p, tops + e, 4, p.tops, 4LL * p.B * p.K * p.groups) ? tops[e] : -INFINITY;
  };
  {
    constexpr int kEach = kJoinEarly / kJoinThreads;
    float t[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) t[i] = tid + i * kJoinThreads < total ? group_top(tid + i * kJoinThreads) : 0.0f;
#pragma unroll
    for (int i = 0; i < kEach; ++i) early[tid + i * kJoinThreads] = t[i];
  }
  if (tid == 0) list.count = n_chosen = 0;
  // --- log-sums of the rows, a warp each
  for (int k = warp; k < p.K; k += kJoinWarps) {
    const float s = k == warp ? s_first : row_score(k);
    const bool over = k == warp ? over_first : row_ended(k);
    const float2 x0 = k == warp ? stat_first : stat(k, lane);
    float m = x0.x;
    for (int i = lane + 32; i < p.parts; i += 32) m = fmaxf(m, stat(k, i).x);
    m = warp_max(m);
    auto scaled = [&](float2 x) { return make_float2(x.y * pow2_whole(fmaxf(x.x - m, -200.0f)), 0.0f); };
    float2 sum = scaled(x0);
#pragma unroll 1
    for (int i = lane + 32; i < p.parts; i += 32) sum = add_pairs(sum, scaled(stat(k, i)));
#pragma unroll 1
    for (int o = 16; o; o >>= 1)
      sum = add_pairs(sum, make_float2(__shfl_xor_sync(kFullMask, sum.x, o), __shfl_xor_sync(kFullMask, sum.y, o)));
    if (lane == 0) {
      const bool has = isfinite(s) && !over && sum.x > 0.0f && isfinite(sum.x) && m <= kHighestRef;
      lse[k] = has ? log_sum(m, sum) : make_float2(__uint_as_float(0x7fc00000u), 0.0f);
      score[k] = s;
      ended[k] = over && isfinite(s);
    }
  }
  __syncthreads();

  // --- the best groups; an ended beam counts as its first group, with its score as it is
  auto group_score = [&](int k, int g, float t) -> uint64_t {   // 0: no candidate
    if (ended[k]) return g ? 0 : static_cast<uint64_t>(ordered(score[k])) << 32 | ordered(0.0f);
    return isnan(lse[k].x) || !(t > kLowest) ? 0 : pair_score(t, lse[k], score[k]);
  };
  // calls f(e, k, g) for the thread's groups, numbered through the rows
  auto each_group = [&](auto f) {
    int k = tid / p.groups, g = tid - k * p.groups;
#pragma unroll 1
    for (int e = tid; e < total; e += kJoinThreads) {
      f(e, k, g);
      for (g += kJoinThreads; g >= p.groups; g -= p.groups) ++k;
    }
  };
  auto top_of = [&](int e) { return e < kJoinEarly ? early[e] : group_top(e); };
  uint32_t mine = 0;
  each_group([&](int e, int k, int g) {
    const uint32_t o = static_cast<uint32_t>(group_score(k, g, top_of(e)) >> 32);
    if (e < kJoinEarly) early_score[e] = o;
    mine = max(mine, o);
  });
  // A bound that n groups are not below and not many more than n: the n-th largest of what the
  // warps' lanes have, ceil(n / warps) + 1 of each warp's.
  const int per_warp = (p.n + kJoinWarps - 1) / kJoinWarps + 1;
  for (int i = 0; i < per_warp; ++i) {
    const uint32_t top = __reduce_max_sync(kFullMask, mine);
    const uint32_t who = __ballot_sync(kFullMask, mine == top);
    if (lane == 0) tops_of_warps[warp * per_warp + i] = top;
    if (lane == __ffs(who) - 1) mine = 0;
  }
  __syncthreads();
  uint32_t low = 0;
  const int n_tops = kJoinWarps * per_warp;
  for (int i = lane; i - lane < n_tops; i += 32) {         // the one with n - 1 before it
    const uint32_t x = i < n_tops ? tops_of_warps[i] : 0;
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n_tops; ++j) {
      const uint32_t other = tops_of_warps[j];
      rank += other > x || (other == x && j < i);
    }
    const uint32_t who = __ballot_sync(kFullMask, i < n_tops && rank == p.n - 1);
    if (who) low = __shfl_sync(kFullMask, x, __ffs(who) - 1);
  }
  const uint64_t bound = static_cast<uint64_t>(low) << 32 | 1u;   // (1: what scores 0 is no candidate)
  auto group = [&](int e, int k, int g) {
    const float t = top_of(e);
    return Candidate{group_score(k, g, t), beam_key(ended[k] ? 0.0f : t, g), k};
  };
  each_group([&](int e, int k, int g) {
    if (e < kJoinEarly && early_score[e] < max(low, 1u)) return;
    const Candidate x = group(e, k, g);
    if (x.score < bound) return;
    const int at = atomicAdd(&n_chosen, 1);
    if (at < kJoinGroups) chosen[at] = x;
  });
  __syncthreads();
  // few enough to look through all of them; else the n best alone
  uint64_t least = bound;
  int n_groups = n_chosen;
  if (n_groups > kJoinGroups) {
    list.best_in_rounds(p.n, tid, [&](auto f) {
      each_group([&](int e, int k, int g) {
        const Candidate x = group(e, k, g);
        if (x.score) f(x);
      });
    }, [&](int rank, bool, const Candidate& x) { chosen[rank] = x; });
    n_groups = p.n;                                        // (there are more than that)
    least = chosen[p.n - 1].score;
  }

  // --- their logits, as far as they may be among the n
  auto each_logit = [&](auto f) {
#pragma unroll 1
    for (int i = warp; i < n_groups; i += kJoinWarps) {
      const Candidate from = chosen[i];
      if (ended[from.k]) {
        if (lane == 0) f(Candidate{from.score, beam_key(0.0f, p.end_token), from.k});
        continue;
      }
      const int g = key_token(from.key);
      int lead;
      const T* base = beam_row<T>(p, b * p.K + from.k, lead);
      Chunk c[L::kVectors];
      load_group<T>(p, base, lead, g, lane, c);
      // most logits are far below: their scores need not be computed
      const float far_from = key_high(least), s0 = score[from.k];
      const float2 l = lse[from.k];
      const float far = far_from > -INFINITY
                            ? far_from - s0 + l.x - 1e-6f * (fabsf(far_from) + fabsf(s0) + fabsf(l.x))
                            : kLowest;                     // (a bound below every number)
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float2 pr = L::pair(c, j / 2);
        const float x = j & 1 ? pr.y : pr.x;
        if (x > kLowest && x >= far)
          f(Candidate{pair_score(x, l, s0),
                      beam_key(x, g * kGroup + ((j / L::kVec) * 32 + lane) * L::kVec + j % L::kVec - lead), from.k});
      }
    }
  };
  each_logit([&](const Candidate& x) { list.add(x); });
  __syncthreads();
  const long long outs = static_cast<long long>(p.B) * p.n;
  auto out = [&](int rank, bool some, const Candidate& x) {
    const int64_t at = static_cast<int64_t>(b) * p.n + rank;
    const int token = some ? key_token(x.key) : -1;
    if (FP4Q_IN_RANGE(p, p.out_scores + at, 4, p.out_scores, 4 * outs))
      p.out_scores[at] = some ? key_high(x.score) : -INFINITY;
    if (FP4Q_IN_RANGE(p, p.out_parents + at, 4, p.out_parents, 4 * outs))
      p.out_parents[at] = some ? b * p.K + x.k : -1;
    if (FP4Q_IN_RANGE(p, p.out_tokens + at, 4, p.out_tokens, 4 * outs)) p.out_tokens[at] = token;
    if (p.out_finished && FP4Q_IN_RANGE(p, p.out_finished + at, 1, p.out_finished, outs))
      p.out_finished[at] = some && (ended[x.k] || token == p.end_token);
  };
  if (list.count <= kJoinList)
    list.best(p.n, tid, out);
  else
    list.best_in_rounds(p.n, tid, each_logit, out);
}

}  // namespace

// Parts of a row: twice as many warps as the device holds at a time, of whole groups (when it was
// chosen, 64 x 8 beams of 131072 logits took 35.7 us so, 36.6 with as many, 37.9 with four times).
constexpr int kScanWarpsPerSm = 2 * kScanCtas * kScanWarps;

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
