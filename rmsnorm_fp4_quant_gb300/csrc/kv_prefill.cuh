// kv_prefill.cuh - attention of many query rows per sequence over the paged
// NVFP4 cache, on the 5th-generation tensor cores: the products bound the time.
//
// A CTA has one (sequence, key/value head, 256 query rows, range of keys); the
// rows are the sequence's query tokens times the heads that share the key/value
// head, as two tiles of 128.  Keys are taken 128 at a time:
//     S [128 x 128] = Q K^T        (A, B from shared memory, D / 16 steps)
//     O [128 x D]  += P V          (A = P from tensor memory, B = V^T from shared memory)
// per tile, all operands fp16 (exact for K and V, see kv_attention_common.cuh),
// accumulators fp32 in tensor memory: S of both tiles (256 columns; the fp16 P
// takes the place of its S) and O of both (2 D columns).
//
//   warps 0-3, 4-7   softmax of tile 0, 1: one row per thread, so a row's sum never
//                    leaves the thread.  S is read once (in an item's first step
//                    twice), P written back over it.
//                    O is rescaled in place, by the same threads, in the rare step
//                    in which a row's reference moves; when S of a step is there the
//                    product before it has ended, so nothing else touches O then.
//   warps 8-11       key and value tiles: codes and scales from the cache to
//                    registers one tile ahead, to fp16 in registers, to shared
//                    memory in the 128-byte-swizzled K-major form (V transposed: a
//                    thread takes 8 keys' codes of D / 8 channels, whose nibbles
//                    interleave to pairs of keys), two stages of each.  One
//                    conversion serves 256 rows.
//   warps 12, 13     one thread each issues one tile's products: P V, then Q K' of the
//                    next keys into the S that P has left (products of one thread run
//                    in order).  The two take turns, so that one tile's softmax runs
//                    beside the other's products; while one issues, the other has its
//                    waits and commits behind it (one thread for both tiles spends 800
//                    of 3900 clocks a step on them; two without turns fall into step).
//
// Why these sizes: 128 x 128 tiles read 128 bytes of shared memory per clock at
// the tensor cores' full rate, no less would; two tiles per CTA fill tensor
// memory (512 columns at D = 128) and share every conversion.
//
// Every wait is bounded.  A role whose wait runs out stops and the others' waits
// run out after it; the rows not finished by then are written as NaN, the status
// word (if any) set, and tensor memory freed once the products issued so far have
// ended.
#pragma once

#include "kv_attention_common.cuh"
#include "kv_tcgen05.cuh"

namespace fp4q {

constexpr int kPreRows = 256;            // query rows of an item, two tiles of 128
constexpr int kPreKeys = 128;            // keys of a step
constexpr int kPreThreads = 16 * 32;
// Registers per thread of the three kinds of warpgroups: 2 x 128 x 160 + 128 x 128 +
// 128 x 64 = 65536.  Together they may not pass what the CTA is launched with (512
// threads of 128), or the increase would wait forever: the launch checks that.
constexpr int kPreSoftmaxRegs = 160, kPreTileRegs = 128, kPreIssueRegs = 64;
constexpr int kPreRegs = 256 * kPreSoftmaxRegs + 128 * kPreTileRegs + 128 * kPreIssueRegs;
// A row's weights of one step are taken against the reference of the steps before;
// only if their sum passes this is the maximum looked for and the reference moved to
// kRefBelow below it (which leaves the sum at 128 * 2^6 at most).  Weights then stay
// below 2^14, far from fp16's end, and the usual step needs no maximum at all.
constexpr float kPreMostSum = 16384.0f;
constexpr uint32_t kPreTmemCols = 512;

template <int D>
struct PrefillShape {
  static constexpr int kTile = 128 * D * 2;                // bytes of one fp16 tile
  static constexpr int kQ = 0, kK = 2 * kTile, kV = 4 * kTile;
  static constexpr int kBars = 6 * kTile;                  // after two tiles of Q, two stages of K, of V
  static constexpr int kSmem = 1024 + 6 * kTile + 256;     // 1 KiB of alignment slack
};

__host__ __device__ inline int64_t prefill_row_slots(int64_t B, int64_t T, int group) {
  return T * group / kPreRows + B;
}

enum PrefillBar { kBarQ = 0, kBarKFull = 1, kBarKEmpty = 3, kBarVFull = 5, kBarVEmpty = 7, kBarS = 9,
                  kBarP = 11, kBarO = 13, kBarDrain = 15, kBarTurn = 17 };

// The warp's arrival, once all its lanes have come here.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" :: "r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Row numbers (and places in the page) of the eight 16-key groups of the tile
// that begins at key0, one per lane 0-7; kNoRow without a page.
constexpr uint32_t kPreNoRow = 0xffffffffu;
__device__ __forceinline__ int prefill_page(const KvAttentionParams& p, int b, int idx) {
  const int32_t* entry = p.tables + static_cast<int64_t>(b) * p.max_pages + idx;
  return FP4Q_IN_RANGE(p, entry, 4, p.tables, 4LL * p.B * p.max_pages) ? __ldg(entry) : -1;
}
__device__ __forceinline__ uint32_t prefill_row(const KvAttentionParams& p, int kvh, int page, int at) {
  return page >= 0 && page < p.c.num_pages ? (static_cast<uint32_t>(page) * p.c.heads + kvh) * p.c.page_size + at
                                           : kPreNoRow;
}
__device__ __forceinline__ void prefill_rows(const KvAttentionParams& p, int b, int kvh, int key0, int len,
                                             int lane, uint32_t& row, uint32_t& at) {
  const int key = key0 + 16 * lane;
  row = kPreNoRow;
  at = 0;
  if (lane < 8 && key < len) {
    const int idx = key / p.c.page_size;
    at = key - idx * p.c.page_size;
    row = prefill_row(p, kvh, prefill_page(p, b, idx), at);
  }
}

// The codes and scales that a thread of warps 8-11 takes of one key tile.
template <int D>
struct PrefillRaw {
  static constexpr int KP = D / 32;      // 16-byte pieces of a key's codes
  static constexpr int VW = D / 64;      // words of a key's codes that a thread takes for V
  uint4 k[KP];
  uint32_t ks[KP];                       // scale bytes of a piece's two blocks
  uint32_t v[8][VW];
  uint2 vs;
};

template <int D>
__device__ __forceinline__ void prefill_load(const KvAttentionParams& p, uint32_t row_of, uint32_t at_of,
                                             int pw, int lane, PrefillRaw<D>& r) {
  constexpr int KP = PrefillRaw<D>::KP, VW = PrefillRaw<D>::VW;
  // K: piece lane / KEYS of key i * 4 KEYS + pw * KEYS + lane % KEYS; eight neighbouring
  // lanes hold eight keys, whose swizzled places lie in different banks
  constexpr int KEYS = 32 / KP;
#pragma unroll
  for (int i = 0; i < KP; ++i) {
    const int key = i * 4 * KEYS + pw * KEYS + lane % KEYS, piece = lane / KEYS;
    const uint32_t base = __shfl_sync(kFullMask, row_of, key >> 4);
    r.k[i] = make_uint4(0, 0, 0, 0);
    r.ks[i] = 0;
    if (base != kPreNoRow) {
      const uint64_t row = static_cast<uint64_t>(base) + (key & 15);
      const uint8_t* src = p.c.k_packed + row * (D / 2) + piece * 16;
      const uint8_t* sf = p.c.k_sf + row * (D / 16) + piece * 2;
      if (FP4Q_IN_RANGE(p, src, 16, p.c.k_packed, kv_packed_extent(p.c)))
        r.k[i] = __ldg(reinterpret_cast<const uint4*>(src));
      if (FP4Q_IN_RANGE(p, sf, 2, p.c.k_sf, kv_sf_extent(p.c)))
        r.ks[i] = __ldg(reinterpret_cast<const unsigned short*>(sf));
    }
  }
  // V: the 8 keys of group lane % 8 of half pw % 2, channels D/8 * (4 (pw / 2) + lane / 8) ...
  const int first = (pw & 1) * 64 + (lane & 7) * 8, dw = (pw >> 1) * 4 + (lane >> 3);
  const uint32_t base = __shfl_sync(kFullMask, row_of, first >> 4);
  const uint32_t at = __shfl_sync(kFullMask, at_of, first >> 4);
  r.vs = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int w = 0; w < VW; ++w) r.v[i][w] = 0;
  if (base != kPreNoRow) {
    const uint64_t row = static_cast<uint64_t>(base) + (first & 15);
    const uint8_t* src = p.c.v_packed + row * (D / 2) + dw * (4 * VW);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!FP4Q_IN_RANGE(p, src + i * (D / 2), 4 * VW, p.c.v_packed, kv_packed_extent(p.c))) continue;
      if constexpr (VW == 2) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(src + i * (D / 2)));
        r.v[i][0] = x.x;
        r.v[i][1] = x.y;
      } else {
        r.v[i][0] = __ldg(reinterpret_cast<const uint32_t*>(src + i * (D / 2)));
      }
    }
    const uint64_t in_page = at + (first & 15);
    const uint8_t* sf = p.c.v_sf + (row - in_page) * (D / 16) +
                        static_cast<uint64_t>(dw * VW / 2) * p.c.page_size + in_page;
    if (FP4Q_IN_RANGE(p, sf, 8, p.c.v_sf, kv_sf_extent(p.c))) r.vs = __ldg(reinterpret_cast<const uint2*>(sf));
  }
}

template <int D>
__device__ __forceinline__ void prefill_store_k(const PrefillRaw<D>& r, uint32_t dst, int pw, int lane) {
  constexpr int KP = PrefillRaw<D>::KP, KEYS = 32 / KP;
#pragma unroll
  for (int i = 0; i < KP; ++i) {
    const int key = i * 4 * KEYS + pw * KEYS + lane % KEYS, piece = lane / KEYS;
    const uint32_t sf = e4m3x2_to_f16x2(r.ks[i]);
    const uint32_t s0 = __byte_perm(sf, 0, 0x1010), s1 = __byte_perm(sf, 0, 0x3232);
    const uint32_t row = dst + (piece >> 1) * 16384 + key * 128;
    const uint32_t words[4] = {r.k[i].x, r.k[i].y, r.k[i].z, r.k[i].w};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t h[4];
      e2m1x8_to_f16x2(words[w], h);
      const uint32_t s = w < 2 ? s0 : s1;
      sts128(row + ((((piece & 1) * 4 + w) ^ (key & 7)) << 4), mul_f16x2(h[0], s), mul_f16x2(h[1], s),
             mul_f16x2(h[2], s), mul_f16x2(h[3], s));
    }
  }
}

template <int D>
__device__ __forceinline__ void prefill_store_v(const PrefillRaw<D>& r, uint32_t dst, int keys_left, int pw,
                                                int lane) {
  constexpr int VW = PrefillRaw<D>::VW;
  const int kg = lane & 7, dw = (pw >> 1) * 4 + (lane >> 3);
  const uint32_t base = dst + (pw & 1) * (D * 128);
  // slots behind the sequence's end may hold no numbers: their scales count as 0 (here
  // and not with the load, which nothing is to wait for)
  uint2 vs = r.vs;
  const int left = keys_left - (pw & 1) * 64 - kg * 8;
  if (left < 8) {
    vs.x = left <= 0 ? 0u : left >= 4 ? vs.x : vs.x & (0xffffffffu >> (32 - 8 * left));
    vs.y = left <= 4 ? 0u : vs.y & (0xffffffffu >> (64 - 8 * left));
  }
  uint32_t sc[4];
  sc[0] = e4m3x2_to_f16x2(vs.x);
  sc[1] = e4m3x2_to_f16x2(vs.x >> 16);
  sc[2] = e4m3x2_to_f16x2(vs.y);
  sc[3] = e4m3x2_to_f16x2(vs.y >> 16);
#pragma unroll
  for (int w = 0; w < VW; ++w) {
    uint32_t lo[4][4], hi[4][4];                      // [pair of keys][channel pair]
#pragma unroll
    for (int kp = 0; kp < 4; ++kp) {
      e2m1x8_to_f16x2(low_nibbles_of(r.v[2 * kp][w], r.v[2 * kp + 1][w] << 4), lo[kp]);
      e2m1x8_to_f16x2(low_nibbles_of(r.v[2 * kp][w] >> 4, r.v[2 * kp + 1][w]), hi[kp]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int d = dw * (8 * VW) + 8 * w + 2 * c;
      sts128(base + d * 128 + ((kg ^ (d & 7)) << 4), mul_f16x2(lo[0][c], sc[0]), mul_f16x2(lo[1][c], sc[1]),
             mul_f16x2(lo[2][c], sc[2]), mul_f16x2(lo[3][c], sc[3]));
      sts128(base + (d + 1) * 128 + ((kg ^ ((d + 1) & 7)) << 4), mul_f16x2(hi[0][c], sc[0]),
             mul_f16x2(hi[1][c], sc[1]), mul_f16x2(hi[2][c], sc[2]), mul_f16x2(hi[3][c], sc[3]));
    }
  }
}

// One row's weights of a step: S from tensor memory, 16 columns being read while 16
// are worked on, p = 2^(fac s - ref) in fp32 summed and in fp16 packed.  Keys that the
// row does not see, and keys of 16-key groups without a page (bits of `have`), get 0.
template <bool EDGE>
__device__ __forceinline__ float2 prefill_weights_16(const uint32_t (&x)[16], int c, int key0, int lim,
                                                     uint32_t have, float2 fac2, float2 ref2, float2 sum2,
                                                     uint32_t (&h)[64]) {
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    float2 y = __ffma2_rn(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), fac2, ref2);
    if (EDGE) {
      const bool page = have >> c & 1u;
      if (!page || key0 + 16 * c + i >= lim) y.x = -INFINITY;
      if (!page || key0 + 16 * c + i + 1 >= lim) y.y = -INFINITY;
    }
    y.x = ex2(y.x);
    y.y = ex2(y.y);
    sum2 = __fadd2_rn(sum2, y);
    h[8 * c + i / 2] = pack_f16x2(y.x, y.y);
  }
  return sum2;
}
template <bool EDGE>
__device__ __forceinline__ float prefill_weights(uint32_t ts, int key0, int lim, uint32_t have, float fac,
                                                 float ref, uint32_t (&h)[64]) {
  const float2 fac2 = make_float2(fac, fac), ref2 = make_float2(-ref, -ref);
  float2 sum2 = make_float2(0.0f, 0.0f);
  uint32_t a[16], b[16];
  tmem_load_16cols_async(ts, a);
  tmem_load_wait(a);
#pragma unroll
  for (int c = 0; c < 8; c += 2) {
    tmem_load_16cols_async(ts + 16 * c + 16, b);
    sum2 = prefill_weights_16<EDGE>(a, c, key0, lim, have, fac2, ref2, sum2, h);
    tmem_load_wait(b);
    if (c < 6) tmem_load_16cols_async(ts + 16 * c + 32, a);
    sum2 = prefill_weights_16<EDGE>(b, c + 1, key0, lim, have, fac2, ref2, sum2, h);
    if (c < 6) tmem_load_wait(a);
  }
  return sum2.x + sum2.y;
}
// The largest product of a row with a key that it sees.
template <bool EDGE>
__device__ __forceinline__ float prefill_maximum(uint32_t ts, int key0, int lim, uint32_t have) {
  float m = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t x[32];
    tmem_load_32cols(ts + 32 * c, x);
    float y[2] = {-INFINITY, -INFINITY};           // two chains
#pragma unroll
    for (int i = 0; i < 32; i += 4)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float u = __uint_as_float(x[i + 2 * k]), v = __uint_as_float(x[i + 2 * k + 1]);
        if (EDGE) {
          const bool page = have >> (2 * c + i / 16) & 1u;
          if (!page || key0 + 32 * c + i + 2 * k >= lim) u = -INFINITY;
          if (!page || key0 + 32 * c + i + 2 * k + 1 >= lim) v = -INFINITY;
        }
        y[k] = max3(y[k], u, v);
      }
    m = max3(m, y[0], y[1]);
  }
  return m;
}

// Multiplies 32 n columns of tensor memory, this thread's lane of them, by f.
__device__ __forceinline__ void prefill_scale(uint32_t taddr, int n, float f) {
#pragma unroll 1
  for (int c = 0; c < n; ++c) {
    uint32_t x[32];
    tmem_load_32cols(taddr + 32 * c, x);
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__fmul_rn(__uint_as_float(x[i]), f));
    tmem_store_32cols(taddr + 32 * c, x);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kPreThreads, 1) kv_prefill_kernel(const KvAttentionParams p, int splits) {
  using S = PrefillShape<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t tmem_slot;
  const uint32_t smem0 = (smem_addr(smem_raw) + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (smem0 - smem_addr(smem_raw));
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + S::kBars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  griddep_wait();
  // the item: row slots are counted from the last, which sees the most keys
  const int kvh = static_cast<int>(blockIdx.x % p.c.heads);
  const int64_t rs = prefill_row_slots(p.B, p.T, p.group) - 1 - blockIdx.x / p.c.heads;
  auto slots_from = [&](int b) {
    const int64_t q0 = p.cu ? min(max(kv_cu(p, b), 0), static_cast<int>(p.T)) : b;
    return q0 * p.group / kPreRows + b;
  };
  int b = 0, b_hi = p.B - 1;
  while (b < b_hi) {
    const int mid = (b + b_hi + 1) / 2;
    if (slots_from(mid) <= rs) b = mid; else b_hi = mid - 1;
  }
  const int64_t rt = rs - slots_from(b);
  const KvSeq seq = kv_sequence(p, b);
  const int rows = seq.n_q * p.group;
  if (rt < 0 || rt * kPreRows >= rows) return;
  const int r0 = static_cast<int>(rt) * kPreRows;
  const int off = seq.len - seq.n_q;
  // steps of 128 keys: this split's share of what the last row sees, and how many of
  // them each tile's last row sees
  auto limit_of = [&](int r) { return p.causal ? min(seq.len, off + r / p.group + 1) : seq.len; };
  const int last0 = min(r0 + 128, rows) - 1, last1 = min(r0 + 256, rows) - 1;
  const int all = (max(0, limit_of(last1)) + kPreKeys - 1) / kPreKeys;
  const int per = (all + splits - 1) / splits;
  const int t0 = min(all, static_cast<int>(blockIdx.y) * per), t1 = min(all, t0 + per);
  const int all0 = (max(0, limit_of(last0)) + kPreKeys - 1) / kPreKeys;
  const int n[2] = {max(0, min(t1, all0) - t0), r0 + 128 < rows ? t1 - t0 : 0};
  const int steps = max(n[0], n[1]);

  if (warp == 12) tmem_alloc(&tmem_slot, kPreTmemCols);
  if (tid == 0) {
    // one arrival per warp of the writers, one commit of each tile's products
    mbar_init(&bars[kBarQ], 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars[kBarKFull + i], 4);
      mbar_init(&bars[kBarKEmpty + i], 2);
      mbar_init(&bars[kBarVFull + i], 4);
      mbar_init(&bars[kBarVEmpty + i], 2);
      mbar_init(&bars[kBarS + i], 1);
      mbar_init(&bars[kBarP + i], 4);
      mbar_init(&bars[kBarO + i], 1);
      mbar_init(&bars[kBarDrain + i], 1);
      mbar_init(&bars[kBarTurn + i], 1);
    }
    mbar_init_fence();
  }
  // whether a page of these keys is outside the cache: only then are the steps' pages
  // looked at by the softmax too
  bool bad = false;
  {
    const int32_t* table = p.tables + static_cast<int64_t>(b) * p.max_pages;
    const int end = min(t1 * kPreKeys, seq.len);
    for (int i = t0 * kPreKeys / p.c.page_size + tid; static_cast<int64_t>(i) * p.c.page_size < end; i += kPreThreads) {
      if (!FP4Q_IN_RANGE(p, table + i, 4, p.tables, 4LL * p.B * p.max_pages)) continue;
      const int page = __ldg(table + i);
      bad |= page < 0 || page >= p.c.num_pages;
    }
  }
  tc_fence_before_sync();
  const bool bad_pages = __syncthreads_or(bad);
  tc_fence_after_sync();
  griddep_launch_dependents();
  const uint32_t tmem = tmem_slot;
  const long long wait_limit = FP4Q_WAIT_LIMIT(p);

  if (warp < 8) {
    // --- softmax: one row per thread
    registers_up<kPreSoftmaxRegs>();
    const int tile = warp >> 2, r_in = (warp & 3) * 32 + lane;
    const int r = r0 + tile * 128 + r_in;
    const bool ok = r < rows;
    const int tok = r / p.group, hq = kvh * p.group + r - tok * p.group;
    const int64_t at = static_cast<int64_t>(seq.q0 + tok) * p.Hq + hq;     // row of out and lse
    float fac;
    {
      const T* src = static_cast<const T*>(p.q) + static_cast<int64_t>(seq.q0 + (ok ? tok : 0)) * p.q_stride +
                     static_cast<int64_t>(ok ? hq : 0) * D;
      Chunk c[D / 16];
      float top = 0.0f;
      bool nan = false;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        c[i] = Chunk{};
        if (ok && FP4Q_IN_RANGE(p, src + 16 * i, 32, p.q, 2LL * ((p.T - 1) * p.q_stride + p.Hq * D)))
          c[i] = ld_cached_ro(src + 16 * i);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 x = Pair<T>::to_f32(c[i].u[j]);
          top = max_abs3(top, x.x, x.y);
          nan |= x.x != x.x || x.y != x.y;
        }
      }
      if (nan) top = INFINITY;
      const int k = q_exponent(top);
      // a row with an infinity or NaN is NaN, and its products with every key are
      const float up = top < INFINITY ? pow2(k) : __uint_as_float(0x7fc00000u);
      const uint32_t dst = smem0 + S::kQ + tile * S::kTile + r_in * 128;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {          // 16 bytes: 8 channels
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = Pair<T>::to_f32(c[i / 2].u[(i & 1) * 4 + j]);
          h[j] = pack_f16x2(x.x * up, x.y * up);
        }
        sts128(dst + (i >> 3) * 16384 + (((i & 7) ^ (r_in & 7)) << 4), h[0], h[1], h[2], h[3]);
      }
      fence_proxy_async_smem();
      warp_arrive(&bars[kBarQ], lane);
      const float kgs = p.c.k_gs ? __ldg(p.c.k_gs) : 1.0f;
      fac = p.sm_scale * kLog2e / kgs * pow2(-k);
    }
    const uint32_t ts = tmem + tile * 128 + ((warp & 3) * 32 << 16);
    const uint32_t to = tmem + 256 + tile * D + ((warp & 3) * 32 << 16);
    const int lim = ok ? limit_of(r) : 0;
    int lim_lo = ok ? lim : INT32_MAX;           // smallest of the warp's rows
    lim_lo = __reduce_min_sync(kFullMask, lim_lo);
    constexpr int kCoarseRows = INT32_MIN;       // in lim_lo's place: a row's reference is_coarse, or was
    float ref = kRefStart, sum = 0.0f;
    bool alive = true;
    for (int j = 0; j < n[tile]; ++j) {
      const int key0 = (t0 + j) * kPreKeys;
      uint32_t have = 0xffu;                       // 16-key groups that have a page
      if (bad_pages) {
        uint32_t row_of, at_of;
        prefill_rows(p, b, kvh, key0, seq.len, lane, row_of, at_of);
        have = __ballot_sync(kFullMask, row_of != kPreNoRow);
      }
      if (!__all_sync(kFullMask, mbar_wait_bounded(&bars[kBarS + tile], j & 1, wait_limit))) {
        alive = false;
        break;
      }
      tc_fence_after_sync();
      const bool edge = key0 + kPreKeys > lim_lo || have != 0xffu;
      // the weights against the reference there is; where a row's sum passes the limit
      // (rare after the first step, which begins with its maximum), once more.  A warp that
      // had a coarse reference begins every step so, and rounds S times the factor in place
      // after it: the exponents' code is the usual one, with a factor of 1 (other code for
      // such rows, or two roundings in the masked steps', made every call 1 to 2 % slower)
      uint32_t h[64];
      float step_sum;
      bool moved = j == 0 || lim_lo == kCoarseRows, last = moved;
#pragma unroll 1
      for (;;) {
        if (last) {
          const float m = edge ? prefill_maximum<true>(ts, key0, lim, have)
                               : prefill_maximum<false>(ts, key0, lim, have);
          float f = 1.0f;
          if (moved && m > -INFINITY) {
            const float to_ref = ref_for(ref, m, fac);
            f = ex2(ref - to_ref);
            ref = to_ref;
            sum *= f;
          }
          if (j > 0) prefill_scale(to, D / 32, f);
          if (lim_lo == kCoarseRows || __any_sync(kFullMask, is_coarse(ref))) {
            lim_lo = kCoarseRows;
            prefill_scale(ts, kPreKeys / 32, fac);
            tmem_store_wait();
          }
        }
        const float f = lim_lo == kCoarseRows ? 1.0f : fac;
        step_sum = edge ? prefill_weights<true>(ts, key0, lim, have, f, ref, h)
                        : prefill_weights<false>(ts, key0, lim, have, f, ref, h);
        if (last) break;
        moved = !(step_sum <= kPreMostSum);
        if (!__any_sync(kFullMask, moved)) break;
        last = true;
      }
      sum += step_sum;
#pragma unroll
      for (int c = 0; c < 2; ++c) {                // P over S, all of which has been read
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = h[32 * c + i];
        tmem_store_32cols(ts + 32 * c, w);
      }
      tmem_store_wait();
      tc_fence_before_sync();
      warp_arrive(&bars[kBarP + tile], lane);
    }
    // --- the row's result
    if (alive && n[tile] > 0) {
      alive = __all_sync(kFullMask, mbar_wait_bounded(&bars[kBarO + tile], 0, wait_limit));
      tc_fence_after_sync();
    }
    if (!alive) {
      sum = __uint_as_float(0x7fc00000u);
      if (p.status) atomicExch(p.status, kStatusTimeout);
    }
    const float vgs = p.c.v_gs ? __ldg(p.c.v_gs) : 1.0f;
    const bool parts = splits > 1;
    const float scale = parts ? 1.0f : sum > 0.0f ? 1.0f / (sum * vgs) : sum == 0.0f ? 0.0f : sum;
    const int64_t total = p.T * p.Hq;
    const int64_t pr = blockIdx.y * total + at;  // row of the partial results
    if (alive && n[tile] == 0) {                 // no key for any row of the tile
      if (ok && !parts) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          T* dst = static_cast<T*>(p.out) + at * D + 16 * i;
          if (FP4Q_IN_RANGE(p, dst, 32, p.out, 2LL * total * D)) st_stream(dst, Chunk{});
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t x[32];
        if (alive) {
          tmem_load_32cols(to + 32 * c, x);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = 0x7fc00000u;
        }
        if (ok && parts) {
          float* dst = p.ws + pr * D + 32 * c;
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            if (FP4Q_IN_RANGE(p, dst + i, 16, p.ws, p.ws_bytes))
              *reinterpret_cast<uint4*>(dst + i) = make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]);
        } else if (ok) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            Chunk o;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              o.u[k] = Pair<T>::from_f32(__uint_as_float(x[16 * i + 2 * k]) * scale,
                                         __uint_as_float(x[16 * i + 2 * k + 1]) * scale);
            T* dst = static_cast<T*>(p.out) + at * D + 32 * c + 16 * i;
            if (FP4Q_IN_RANGE(p, dst, 32, p.out, 2LL * total * D)) st_stream(dst, o);
          }
        }
        __syncwarp();
      }
    }
    if (ok) {
      float* rl = p.ws + splits * total * D + 2 * pr;
      if (parts && FP4Q_IN_RANGE(p, rl, 8, p.ws, p.ws_bytes))
        *reinterpret_cast<float2*>(rl) = make_float2(ref, sum);
      else if (!parts && p.lse && FP4Q_IN_RANGE(p, p.lse + at, 4, p.lse, 4LL * total))
        p.lse[at] = sum == 0.0f ? -INFINITY : kLn2 * (ref + log2f(sum));
    }
    tc_fence_before_sync();
  } else if (warp < 12) {
    // --- key and value tiles
    const int pw = warp - 8;
    // group `lane` (of 8) of the step after the one whose page is in page_of: page idx, place at;
    // a step of 128 keys is page_q pages and page_r places
    const int page_q = kPreKeys / p.c.page_size, page_r = kPreKeys - page_q * p.c.page_size;
    int key = t0 * kPreKeys + 16 * (lane & 7);
    int idx = key / p.c.page_size, at = key - idx * p.c.page_size;
    int page_of, at_of;                            // the page's number is looked at a step later
    auto next_page = [&]() {
      at_of = at;
      page_of = key < seq.len ? prefill_page(p, b, idx) : -1;
      key += kPreKeys;
      idx += page_q;
      at += page_r;
      if (at >= p.c.page_size) {
        at -= p.c.page_size;
        ++idx;
      }
    };
    PrefillRaw<D> raw[2];                          // loaded one step before it is converted
    next_page();
    if (steps > 0) prefill_load<D>(p, prefill_row(p, kvh, page_of, at_of), at_of, pw, lane, raw[0]);
    next_page();
    bool alive = true;
    for (int j0 = 0; j0 < steps && alive; j0 += 2) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int j = j0 + s;
        if (j >= steps || !alive) break;
        if (j + 1 < steps) {
          prefill_load<D>(p, prefill_row(p, kvh, page_of, at_of), at_of, pw, lane, raw[s ^ 1]);
          next_page();
        }
        const uint32_t parity = ((j >> 1) & 1) ^ 1;    // of the use before
        alive = j < 2 || __all_sync(kFullMask, mbar_wait_bounded(&bars[kBarKEmpty + s], parity, wait_limit));
        if (!alive) break;
        prefill_store_k<D>(raw[s], smem0 + S::kK + s * S::kTile, pw, lane);
        fence_proxy_async_smem();
        warp_arrive(&bars[kBarKFull + s], lane);
        alive = j < 2 || __all_sync(kFullMask, mbar_wait_bounded(&bars[kBarVEmpty + s], parity, wait_limit));
        if (!alive) break;
        prefill_store_v<D>(raw[s], smem0 + S::kV + s * S::kTile, seq.len - (t0 + j) * kPreKeys, pw, lane);
        fence_proxy_async_smem();
        warp_arrive(&bars[kBarVFull + s], lane);
      }
    }
  } else {
    registers_down<kPreIssueRegs>();
  }
  if ((warp == 12 || warp == 13) && lane == 0 && steps > 0) {
    // --- products of one tile
    const int tile = warp - 12, mine = n[tile];
    constexpr uint32_t kIdescS = idesc_f16(128, 128), kIdescO = idesc_f16(128, D);
    // the descriptors differ in their address field, the low word's 14 bits of 16-byte
    // units: a step of 16 adds 32 bytes, one of 64 a sub-tile, without a carry out
    const uint32_t first = static_cast<uint32_t>(smem_desc(smem0, 0, 1024, kSwizzle128B));
    const uint32_t high = static_cast<uint32_t>(smem_desc(smem0, 0, 1024, kSwizzle128B) >> 32);
    auto desc = [&](uint32_t low) { return static_cast<uint64_t>(high) << 32 | low; };
    const uint32_t ts = tmem + tile * 128, to = tmem + 256 + tile * D;
    const uint32_t qa = first + ((S::kQ + tile * S::kTile) >> 4);
    auto q_k = [&](int s, bool hand_over) {
      const uint32_t ka = first + ((S::kK + s * S::kTile) >> 4);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t o = ((k >> 2) * 16384 + (k & 3) * 32) >> 4;
        if (k == D / 16 - 2 && hand_over) mbar_arrive(&bars[kBarTurn + (tile ^ 1)]);
        mma_f16_ss(ts, desc(qa + o), desc(ka + o), kIdescS, k > 0);
      }
      tc_commit(&bars[kBarS + tile]);
    };
    auto p_v = [&](int s, bool begins) {
      const uint32_t va = first + ((S::kV + s * S::kTile) >> 4);
#pragma unroll
      for (int k = 0; k < kPreKeys / 16; ++k) {
        const uint32_t o = ((k >> 2) * (D * 128) + (k & 3) * 32) >> 4;
        mma_f16_ts(to, ts + 8 * k, desc(va + o), kIdescO, !(begins && k == 0));
      }
    };
    // the release of a stage: with the tile's last product of it, or, behind the tile's
    // last step, plainly, once the stage was filled (so no phase gets an arrival too many)
    bool alive = mbar_wait_bounded(&bars[kBarQ], 0, wait_limit) &&
                 mbar_wait_bounded(&bars[kBarKFull], 0, wait_limit);
    if (alive) {
      tc_fence_after_sync();
      if (mine > 0) q_k(0, false);
      tc_commit(&bars[kBarKEmpty]);
    }
    for (int j = 0; j < steps && alive; ++j) {
      const int s = j & 1;
      const bool more = j + 1 < steps;
      alive = mbar_wait_bounded(&bars[kBarVFull + s], (j >> 1) & 1, wait_limit) &&
              (!more || mbar_wait_bounded(&bars[kBarKFull + (s ^ 1)], ((j + 1) >> 1) & 1, wait_limit)) &&
              (j >= mine || mbar_wait_bounded(&bars[kBarP + tile], j & 1, wait_limit)) &&
              // the turns: tile 0 of step 0 has the first
              (j + tile == 0 || mbar_wait_bounded(&bars[kBarTurn + tile], (j + tile + 1) & 1, wait_limit));
      if (!alive) break;
      tc_fence_after_sync();
      if (j < mine) p_v(s, j == 0);
      if (j + 1 < mine) {
        q_k(s ^ 1, true);
      } else {
        mbar_arrive(&bars[kBarTurn + (tile ^ 1)]);
        if (j + 1 == mine) tc_commit(&bars[kBarO + tile]);
      }
      tc_commit(&bars[kBarVEmpty + s]);
      if (more) tc_commit(&bars[kBarKEmpty + (s ^ 1)]);
    }
    tc_commit(&bars[kBarDrain + tile]);          // nothing may run when tensor memory is freed
    mbar_wait_bounded(&bars[kBarDrain + tile], 0);
  }
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 12) tmem_dealloc(tmem, kPreTmemCols);
}

// Joins the splits of every row: one group of D / 4 lanes per row.
template <typename T, int D>
__global__ void __launch_bounds__(256) kv_prefill_join_kernel(const KvAttentionParams p, int splits) {
  constexpr int LANES = D / 4;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t total = p.T * p.Hq;
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / LANES;
  const int ln = threadIdx.x % LANES;
  if (at >= total) return;
  // rows of no sequence are left as they were
  const int64_t t = at / p.Hq;
  bool mine = true;
  if (p.cu) {
    int b = 0, hi = p.B - 1;
    while (b < hi) {
      const int mid = (b + hi + 1) / 2;
      if (kv_cu(p, mid) <= t) b = mid; else hi = mid - 1;
    }
    // of several sequences that begin at one row all but the last are empty
    const KvSeq s = kv_sequence(p, b);
    mine = t >= s.q0 && t < s.q0 + s.n_q;
  }
  if (!mine) return;
  float top = kRefStart;
  const float* stats = p.ws + splits * total * D;
  for (int i = 0; i < splits; ++i) {
    const float* ref = stats + 2 * (i * total + at);
    if (FP4Q_IN_RANGE(p, ref, 4, p.ws, p.ws_bytes)) top = fmaxf(top, *ref);
  }
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float l = 0.0f;
  for (int i = 0; i < splits; ++i) {
    if (!FP4Q_IN_RANGE(p, stats + 2 * (i * total + at), 8, p.ws, p.ws_bytes) ||
        !FP4Q_IN_RANGE(p, p.ws + (i * total + at) * D + 4 * ln, 16, p.ws, p.ws_bytes))
      continue;
    const float2 rl = *reinterpret_cast<const float2*>(stats + 2 * (i * total + at));
    if (rl.y == 0.0f) continue;                  // saw no key: its O was not written
    const float4 x = *reinterpret_cast<const float4*>(p.ws + (i * total + at) * D + 4 * ln);
    const float f = ex2(rl.x - top);
    o.x += x.x * f;
    o.y += x.y * f;
    o.z += x.z * f;
    o.w += x.w * f;
    l += rl.y * f;
  }
  const float vgs = p.c.v_gs ? __ldg(p.c.v_gs) : 1.0f;
  const float inv = l > 0.0f ? 1.0f / (l * vgs) : l == 0.0f ? 0.0f : l;
  T* dst = static_cast<T*>(p.out) + at * D + 4 * ln;
  if (FP4Q_IN_RANGE(p, dst, 8, p.out, 2LL * total * D))
    *reinterpret_cast<uint2*>(dst) = make_uint2(Pair<T>::from_f32(o.x * inv, o.y * inv),
                                                Pair<T>::from_f32(o.z * inv, o.w * inv));
  if (ln == 0 && p.lse && FP4Q_IN_RANGE(p, p.lse + at, 4, p.lse, 4LL * total))
    p.lse[at] = l == 0.0f ? -INFINITY : kLn2 * (top + log2f(l));
}

}  // namespace fp4q
