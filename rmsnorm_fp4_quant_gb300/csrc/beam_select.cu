// beam_select.cu - the best continuations of every beam search of a batch: over
// beams k and tokens v, the n largest of
//     s_k + x_kv - log(sum_v exp(x_kv)).
//
// The logits are read once and bound the time.  Two kernels:
//   scan  a CTA takes a part of one row (up to 8192 logits, held in registers): its
//         largest logit m, the sum of exp(x - m), and its n largest logits in order;
//   join  a CTA per batch entry: every row's log-sum from its parts (64 bits), the
//         scores of the parts' candidates in 64 bits, the n best of them.
// A row's own order is that of its logits, so that no score is computed before the
// candidates are few.  The order is total (a logit's bits, then the lower token; a
// score, then the lower beam), so results do not depend on what runs when.
//
// The n largest of a part, without sorting it: every warp finds the q-th largest of
// its lanes' maxima, q = ceil(n / warps).  At least q * warps >= n logits are not below
// the smallest of these, T, and of random ones hardly twice as many (8192 logits, n = 16: 30 to 50).
// Those go to shared memory, where each counts how many are before it.  Where more than
// kBeamList do (equal logits), n rounds of a maximum over the CTA find them instead.
//
// x - m is taken before the factor log2(e): x * log2(e) - m * log2(e) would carry
// the constant's rounding times m into the sum, and with it into comparisons between beams.
#include <algorithm>

#include "async_copy.cuh"
#include "beam_launch.h"
#include "fp4q_launch.h"
#include "fused_common.cuh"

namespace fp4q {
namespace {

constexpr int kScanThreads = 256;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kJoinThreads = 512;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kBeamList = 1024;
constexpr float kLog2eBeam = 1.4426950408889634f;

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
__device__ __forceinline__ float key_logit(uint64_t k) { return from_ordered(static_cast<uint32_t>(k >> 32)); }
__device__ __forceinline__ int key_token(uint64_t k) { return static_cast<int>(~static_cast<uint32_t>(k)); }

// Whether the row has candidates of its own logits.
__device__ __forceinline__ bool beam_live(const BeamParams& p, int row) {
  const bool here = FP4Q_IN_RANGE(p, p.scores + row, 4, p.scores, 4LL * p.B * p.K);
  if (!here || !isfinite(__ldg(p.scores + row))) return false;
  if (!p.finished || !FP4Q_IN_RANGE(p, p.finished + row, 1, p.finished, 1LL * p.B * p.K)) return true;
  return __ldg(p.finished + row) == 0;
}

template <typename T> struct Logits {                      // 16-bit types
  static constexpr int kVec = 16;
  static constexpr int kSize = 2;
  __device__ static float2 pair(const Chunk& c, int i) { return Pair<T>::to_f32(c.u[i]); }
  __device__ static void set(Chunk& c, int i, const void* src) {
    const uint32_t v = __ldg(static_cast<const unsigned short*>(src));
    c.u[i / 2] = i & 1 ? (c.u[i / 2] & 0xffffu) | v << 16 : (c.u[i / 2] & 0xffff0000u) | v;
  }
  __device__ static Chunk none() {
    Chunk c;
    const uint32_t w = Pair<T>::from_f32(-INFINITY, -INFINITY);
#pragma unroll
    for (int i = 0; i < 8; ++i) c.u[i] = w;
    return c;
  }
};
template <> struct Logits<float> {
  static constexpr int kVec = 8;
  static constexpr int kSize = 4;
  __device__ static float2 pair(const Chunk& c, int i) {
    return make_float2(__uint_as_float(c.u[2 * i]), __uint_as_float(c.u[2 * i + 1]));
  }
  __device__ static void set(Chunk& c, int i, const void* src) {
    c.u[i] = __ldg(static_cast<const unsigned int*>(src));
  }
  __device__ static Chunk none() {
    Chunk c;
#pragma unroll
    for (int i = 0; i < 8; ++i) c.u[i] = 0xff800000u;
    return c;
  }
};

__device__ __forceinline__ float ex2_beam(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The q-th largest of the lanes' values (0 where a lane has none; 0 if there are fewer).
__device__ __forceinline__ uint32_t warp_qth(uint32_t mine, int q, int lane) {
  uint32_t best = 0;
  for (int i = 0; i < q; ++i) {
    best = __reduce_max_sync(kFullMask, mine);
    if (best == 0) return 0;
    const uint32_t who = __ballot_sync(kFullMask, mine == best);
    if (lane == __ffs(who) - 1) mine = 0;
  }
  return best;
}

template <typename T, int NV>
__global__ void __launch_bounds__(kScanThreads) beam_scan_kernel(const BeamParams p) {
  using L = Logits<T>;
  constexpr int VEC = L::kVec;
  __shared__ uint64_t list[kBeamList];
  __shared__ uint32_t warp_top[kScanWarps], warp_low[kScanWarps];
  __shared__ float warp_sum[kScanWarps];
  __shared__ int count;
  __shared__ uint64_t round_best[kScanWarps];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x / p.parts, part = blockIdx.x - row * p.parts;
  griddep_wait();
  if (!beam_live(p, row)) {
    griddep_launch_dependents();
    return;
  }
  // Elements are numbered from the 32-byte boundary at or before the row: number e is
  // token e - lead, and whole vectors are aligned loads whatever the row's address is.
  const T* base = static_cast<const T*>(p.logits) + static_cast<int64_t>(row) * p.stride;
  const int lead = static_cast<int>(reinterpret_cast<uintptr_t>(base) & 31u) / L::kSize;
  const int e0 = part * p.part_len;
  const int e1 = min(e0 + p.part_len, lead + p.V);
  Chunk c[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = e0 + (j * kScanThreads + tid) * VEC;
    c[j] = L::none();
    if (e >= e1 || e + VEC <= lead) continue;
    const T* src = base + (e - lead);
    if (e >= lead && e + VEC <= e1) {
      if (FP4Q_IN_RANGE(p, src, 32, p.logits, beam_logits_extent(p, L::kSize))) c[j] = ld_stream_ro(src);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (e + i >= lead && e + i < e1 &&
            FP4Q_IN_RANGE(p, src + i, L::kSize, p.logits, beam_logits_extent(p, L::kSize)))
          L::set(c[j], i, src + i);
    }
  }
  if (tid == 0) count = 0;
  griddep_launch_dependents();

  // --- the largest, and a bound that n logits are not below
  float top = -INFINITY;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      const float2 x = L::pair(c[j], i);
      top = fmaxf(top, fmaxf(x.x, x.y));                   // skips NaN
    }
  const uint32_t mine = top > -INFINITY ? ordered(top) : 0u;
  // warps that have a logit at all, each of which gives q
  const int vectors = max(0, e1 - e0 + VEC - 1) / VEC;
  const int warps = min(kScanWarps, (vectors + 31) / 32);
  const int q = (p.n + warps - 1) / max(warps, 1);
  {
    const uint32_t m = __reduce_max_sync(kFullMask, mine);
    const uint32_t low = q <= 32 ? warp_qth(mine, q, lane) : 0u;
    if (lane == 0) {
      warp_top[warp] = m;
      warp_low[warp] = low;
    }
  }
  __syncthreads();
  uint32_t o_top = 0, o_low = 0xffffffffu;
#pragma unroll
  for (int w = 0; w < kScanWarps; ++w) {
    o_top = max(o_top, warp_top[w]);
    if (w < warps) o_low = min(o_low, warp_low[w]);
  }
  const float m = o_top ? from_ordered(o_top) : 0.0f;      // no logit above -infinity: every term is 0
  const bool some = mine != 0 && mine >= o_low;

  // --- the sum, and the logits that may be among the n
  float2 sum2 = make_float2(0.0f, 0.0f);
  const float2 neg = make_float2(-m, -m), scale = make_float2(kLog2eBeam, kLog2eBeam);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      float2 y = __fmul2_rn(__fadd2_rn(L::pair(c[j], i), neg), scale);
      y.x = ex2_beam(y.x);
      y.y = ex2_beam(y.y);
      sum2 = __fadd2_rn(sum2, y);
    }
  float sum = sum2.x + sum2.y;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
  if (lane == 0) warp_sum[warp] = sum;
  if (some) {
    const float low = o_low ? from_ordered(o_low) : -INFINITY;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {
        const float2 x = L::pair(c[j], i);
        const int token = e0 + (j * kScanThreads + tid) * VEC + 2 * i - lead;
        if (x.x >= low && x.x > -INFINITY) {
          const int at = atomicAdd(&count, 1);
          if (at < kBeamList) list[at] = beam_key(x.x, token);
        }
        if (x.y >= low && x.y > -INFINITY) {
          const int at = atomicAdd(&count, 1);
          if (at < kBeamList) list[at] = beam_key(x.y, token + 1);
        }
      }
  }
  __syncthreads();
  const int64_t slot = blockIdx.x;
  const long long key_bytes = 8LL * p.B * p.K * p.parts * p.n;
  uint64_t* out = p.keys + slot * p.n;
  const int found = count;
  if (found <= kBeamList) {
    for (int i = tid; i < max(found, p.n); i += kScanThreads) {
      uint64_t key = 0;
      int rank = i;                                        // places behind the last: nothing
      if (i < found) {
        key = list[i];
        rank = 0;
        for (int k = 0; k < found; ++k) rank += list[k] > key;
      }
      if (rank < p.n && FP4Q_IN_RANGE(p, out + rank, 8, p.keys, key_bytes)) out[rank] = key;
    }
  } else {
    uint64_t last = ~0ull;
    for (int r = 0; r < p.n; ++r) {
      uint64_t best = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
          const float2 x = L::pair(c[j], i);
          const int token = e0 + (j * kScanThreads + tid) * VEC + 2 * i - lead;
          if (x.x > -INFINITY) {
            const uint64_t k = beam_key(x.x, token);
            if (k < last && k > best) best = k;
          }
          if (x.y > -INFINITY) {
            const uint64_t k = beam_key(x.y, token + 1);
            if (k < last && k > best) best = k;
          }
        }
#pragma unroll
      for (int o = 16; o; o >>= 1) best = max(best, __shfl_xor_sync(kFullMask, best, o));
      if (lane == 0) round_best[warp] = best;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kScanWarps; ++w) best = max(best, round_best[w]);
      if (tid == 0 && FP4Q_IN_RANGE(p, out + r, 8, p.keys, key_bytes)) out[r] = best;
      last = best ? best : 1;
      __syncthreads();
    }
  }
  if (tid == 0) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kScanWarps; ++w) s += warp_sum[w];
    // a part without a logit above -infinity has no part in the row's sum
    if (FP4Q_IN_RANGE(p, p.stats + slot, 8, p.stats, 8LL * p.B * p.K * p.parts))
      p.stats[slot] = make_float2(o_top ? m : -INFINITY, s);
  }
}

// A candidate of the join: score, then lower row, then the row's own order.
struct Candidate {
  double score;
  uint64_t key;
  int k;
};
__device__ __forceinline__ bool before(const Candidate& a, const Candidate& b) {
  if (a.score != b.score) return a.score > b.score;
  return a.k != b.k ? a.k < b.k : a.key > b.key;
}

__global__ void __launch_bounds__(kJoinThreads) beam_join_kernel(const BeamParams p) {
  __shared__ double lse[kBeamMostBeams];                   // NaN: the row has no candidates
  __shared__ double score[kBeamMostBeams];
  __shared__ bool ended[kBeamMostBeams];
  __shared__ double list_score[kBeamList];
  __shared__ uint64_t list_key[kBeamList];
  __shared__ int list_k[kBeamList];
  __shared__ uint32_t warp_low[kJoinWarps];
  __shared__ Candidate round_best[kJoinWarps];
  __shared__ int count;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  if (tid == 0) count = 0;
  // --- log-sums of the rows, a warp each
  for (int k = warp; k < p.K; k += kJoinWarps) {
    const int row = b * p.K + k;
    float s = __uint_as_float(0x7fc00000u);
    if (FP4Q_IN_RANGE(p, p.scores + row, 4, p.scores, 4LL * p.B * p.K)) s = __ldg(p.scores + row);
    bool over = false;
    if (p.finished && FP4Q_IN_RANGE(p, p.finished + row, 1, p.finished, 1LL * p.B * p.K))
      over = __ldg(p.finished + row) != 0;
    double total = __longlong_as_double(0x7ff8000000000000LL);
    if (isfinite(s) && !over) {
      const float2* st = p.stats + static_cast<int64_t>(row) * p.parts;
      float m = -INFINITY;
      for (int i = lane; i < p.parts; i += 32)
        if (FP4Q_IN_RANGE(p, st + i, 8, p.stats, 8LL * p.B * p.K * p.parts)) m = fmaxf(m, st[i].x);
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, o));
      double sum = 0.0;
      for (int i = lane; i < p.parts; i += 32) {
        if (!FP4Q_IN_RANGE(p, st + i, 8, p.stats, 8LL * p.B * p.K * p.parts)) continue;
        const float2 x = st[i];
        // (a part of -infinities adds 0; one with a NaN or +infinity makes the sum NaN)
        sum += x.x == -INFINITY ? static_cast<double>(x.y)
                                : static_cast<double>(x.y) * exp(static_cast<double>(x.x) - static_cast<double>(m));
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
      total = static_cast<double>(m) + log(sum);
    }
    if (lane == 0) {
      lse[k] = isfinite(total) ? total : __longlong_as_double(0x7ff8000000000000LL);
      score[k] = static_cast<double>(s);
      ended[k] = over && isfinite(s);
    }
  }
  __syncthreads();

  // --- candidate e: element e % n of part e / n of the entry's rows; of an ended row the
  // first element alone, its score as it is
  const int per_row = p.parts * p.n, total = p.K * per_row;
  const uint64_t* keys = p.keys + static_cast<int64_t>(b) * total;
  const long long key_bytes = 8LL * p.B * p.K * p.parts * p.n;
  auto candidate = [&](int e, Candidate& x) {
    x.k = e / per_row;
    if (ended[x.k]) {
      x.key = beam_key(0.0f, p.end_token);
      x.score = score[x.k];
      return e == x.k * per_row;
    }
    if (isnan(lse[x.k]) || !FP4Q_IN_RANGE(p, keys + e, 8, p.keys, key_bytes)) return false;
    x.key = keys[e];
    if (x.key == 0) return false;
    x.score = score[x.k] + (static_cast<double>(key_logit(x.key)) - lse[x.k]);
    return true;
  };
  uint32_t mine = 0;
  for (int e = tid; e < total; e += kJoinThreads) {
    Candidate x;
    if (candidate(e, x)) mine = max(mine, ordered(__double2float_rd(x.score)));
  }
  const int q = (p.n + kJoinWarps - 1) / kJoinWarps;
  const uint32_t low = warp_qth(mine, q, lane);
  if (lane == 0) warp_low[warp] = low;
  __syncthreads();
  uint32_t o_low = 0xffffffffu;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) o_low = min(o_low, warp_low[w]);
  if (mine != 0 && mine >= o_low) {
    for (int e = tid; e < total; e += kJoinThreads) {
      Candidate x;
      if (!candidate(e, x) || ordered(__double2float_rd(x.score)) < o_low) continue;
      const int at = atomicAdd(&count, 1);
      if (at < kBeamList) {
        list_score[at] = x.score;
        list_key[at] = x.key;
        list_k[at] = x.k;
      }
    }
  }
  __syncthreads();
  const int found = count;
  const long long outs = static_cast<long long>(p.B) * p.n;
  auto write = [&](int rank, bool some, const Candidate& x) {
    const int64_t at = static_cast<int64_t>(b) * p.n + rank;
    const int token = some ? key_token(x.key) : -1;
    if (FP4Q_IN_RANGE(p, p.out_scores + at, 4, p.out_scores, 4 * outs))
      p.out_scores[at] = some ? static_cast<float>(x.score) : -INFINITY;
    if (FP4Q_IN_RANGE(p, p.out_parents + at, 4, p.out_parents, 4 * outs))
      p.out_parents[at] = some ? b * p.K + x.k : -1;
    if (FP4Q_IN_RANGE(p, p.out_tokens + at, 4, p.out_tokens, 4 * outs)) p.out_tokens[at] = token;
    if (p.out_finished && FP4Q_IN_RANGE(p, p.out_finished + at, 1, p.out_finished, outs))
      p.out_finished[at] = some && (ended[x.k] || token == p.end_token);
  };
  if (found <= kBeamList) {
    for (int i = tid; i < max(found, p.n); i += kJoinThreads) {
      Candidate x{};
      int rank = i;
      if (i < found) {
        x = Candidate{list_score[i], list_key[i], list_k[i]};
        rank = 0;
        for (int k = 0; k < found; ++k) rank += before(Candidate{list_score[k], list_key[k], list_k[k]}, x);
      }
      if (rank < p.n) write(rank, i < found, x);
    }
    return;
  }
  Candidate last{INFINITY, 0, -1};
  for (int r = 0; r < p.n; ++r) {
    Candidate best{-INFINITY, 0, p.K};
    for (int e = tid; e < total; e += kJoinThreads) {
      Candidate x;
      if (candidate(e, x) && before(last, x) && before(x, best)) best = x;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const Candidate y{__shfl_xor_sync(kFullMask, best.score, o), __shfl_xor_sync(kFullMask, best.key, o),
                        __shfl_xor_sync(kFullMask, best.k, o)};
      if (before(y, best)) best = y;
    }
    if (lane == 0) round_best[warp] = best;
    __syncthreads();
    for (int w = 0; w < kJoinWarps; ++w)
      if (before(round_best[w], best)) best = round_best[w];
    if (tid == 0) write(r, best.k < p.K, best);
    if (best.k < p.K) last = best;
    __syncthreads();
  }
}

int vec_of(int dtype) { return dtype == 2 ? 8 : 16; }

}  // namespace

void beam_shape(int dtype, BeamParams* p) {
  const int vec = vec_of(dtype);
  // elements from the boundary before the row: an upper bound for rows of any alignment
  const int64_t len = static_cast<int64_t>(p->V) + vec - 1;
  const int64_t most = 32LL * kScanThreads;
  p->parts = static_cast<int>((len + most - 1) / most);
  p->part_len = static_cast<int>(((len + p->parts - 1) / p->parts + vec - 1) / vec * vec);
}

int64_t beam_workspace(int dtype, int64_t B, int64_t K, int64_t V, int64_t n) {
  BeamParams p{};
  p.B = static_cast<int>(B);
  p.K = static_cast<int>(K);
  p.V = static_cast<int>(V);
  p.n = static_cast<int>(n);
  beam_shape(dtype, &p);
  return B * K * p.parts * (n + 1) * 8;
}

template <typename T>
cudaError_t launch_scan(const BeamParams& p, const cudaLaunchConfig_t& cfg) {
  return cudaLaunchKernelEx(&cfg, beam_scan_kernel<T, 32 / Logits<T>::kVec>, p);
}

cudaError_t launch_beam_select(int dtype, const BeamParams& p, int pdl, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<int64_t>(p.B) * p.K * p.parts));
  cfg.blockDim = dim3(kScanThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  const cudaError_t e = dtype == 0   ? launch_scan<__nv_bfloat16>(p, cfg)
                        : dtype == 1 ? launch_scan<__half>(p, cfg)
                                     : launch_scan<float>(p, cfg);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3(static_cast<unsigned>(p.B));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.numAttrs = 1;                              // its launch overlaps the first kernel
  return cudaLaunchKernelEx(&cfg, beam_join_kernel, p);
}

}  // namespace fp4q
