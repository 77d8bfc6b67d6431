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
// Windows, prefixes, biases and caps (MODE, KvLogits).  A row sees a run of keys, [first, limit),
// and an item takes the steps that one of its rows has keys in.  A window or a prefix alone only
// changes the masks.  A bias is a straight line on either side of a row's own place: one
// more multiply-add a pair of keys (a prompt of 4096, 32 heads of 128, logits of deviation 2: 163 us,
// 126 without), and the keys are taken from the last to the first.  A cap is three special
// functions instead of one, two reciprocals in one of them (with logits of deviation 9 230 us): 13.2
// instructions a logit (114 million warp instructions, all roles', over 8.65 million warps of
// logits) where there are 7.7 without, at the same share of the issue slots (43 and 44 %).  No unit is
// near its limit (tensor pipe 25 %, special functions 32 %): two softmax warps per scheduler wait for
// one result after the other.  An exponential in polynomials instead of the special function made
// the calls 12 % slower and more.
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
// FROM: and keys before `from`.
template <bool EDGE, bool FROM>
__device__ __forceinline__ float2 prefill_weights_16(const uint32_t (&x)[16], int c, int key0, int lim, int from,
                                                     uint32_t have, float2 fac2, float2 ref2, float2 sum2,
                                                     uint32_t (&h)[64]) {
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    float2 y = __ffma2_rn(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), fac2, ref2);
    if (EDGE) {
      const bool page = have >> c & 1u;
      const int key = key0 + 16 * c + i;
      if (!page || key >= lim || (FROM && key < from)) y.x = -INFINITY;
      if (!page || key + 1 >= lim || (FROM && key + 1 < from)) y.y = -INFINITY;
    }
    y.x = ex2(y.x);
    y.y = ex2(y.y);
    sum2 = __fadd2_rn(sum2, y);
    h[8 * c + i / 2] = pack_f16x2(y.x, y.y);
  }
  return sum2;
}
template <bool EDGE, bool FROM>
__device__ __forceinline__ float prefill_weights(uint32_t ts, int key0, int lim, int from, uint32_t have, float fac,
                                                 float ref, uint32_t (&h)[64]) {
  const float2 fac2 = make_float2(fac, fac), ref2 = make_float2(-ref, -ref);
  float2 sum2 = make_float2(0.0f, 0.0f);
  uint32_t a[16], b[16];
  tmem_load_16cols_async(ts, a);
  tmem_load_wait(a);
#pragma unroll
  for (int c = 0; c < 8; c += 2) {
    tmem_load_16cols_async(ts + 16 * c + 16, b);
    sum2 = prefill_weights_16<EDGE, FROM>(a, c, key0, lim, from, have, fac2, ref2, sum2, h);
    tmem_load_wait(b);
    if (c < 6) tmem_load_16cols_async(ts + 16 * c + 32, a);
    sum2 = prefill_weights_16<EDGE, FROM>(b, c + 1, key0, lim, from, have, fac2, ref2, sum2, h);
    if (c < 6) tmem_load_wait(a);
  }
  return sum2.x + sum2.y;
}
// The largest product of a row with a key that it sees (of keys `from` on: FROM).
template <bool EDGE, bool FROM>
__device__ __forceinline__ float prefill_maximum(uint32_t ts, int key0, int lim, int from, uint32_t have) {
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
          const int key = key0 + 32 * c + i + 2 * k;
          if (!page || key >= lim || (FROM && key < from)) u = -INFINITY;
          if (!page || key + 1 >= lim || (FROM && key + 1 < from)) v = -INFINITY;
        }
        y[k] = max3(y[k], u, v);
      }
    m = max3(m, y[0], y[1]);
  }
  return m;
}

// What a row needs to turn products into logits (has_bias, has_cap): kv_logit's arguments,
// its own place, and the keys [from, lim) that it sees.
struct PrefillLogits {
  float fac, cap, slope;
  int own, from, lim;
  __device__ __forceinline__ bool sees(int key, bool page) const { return page && key < lim && key >= from; }
};
// (away: the distance of key0, `key` of these behind it)
template <int MODE>
__device__ __forceinline__ float prefill_logit(uint32_t s, int key0, int key, float away, bool page, const PrefillLogits& l) {
  const float z = kv_logit<MODE>(__uint_as_float(s), l.fac, l.cap, l.slope, away + static_cast<float>(key));
  return l.sees(key0 + key, page) ? z : -INFINITY;
}
// As prefill_weights above, logit by logit, each rounded before the reference is taken from it:
// for steps on both sides of a row's own place, for coarse references, and for wide caps.
template <int MODE>
__device__ __forceinline__ float prefill_weights_by_logit(uint32_t ts, int key0, uint32_t have, const PrefillLogits& l,
                                                          float ref, uint32_t (&h)[64]) {
  float2 sum2 = make_float2(0.0f, 0.0f);
  const float away = static_cast<float>(key0 - l.own);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint32_t x[16];
    tmem_load_16cols_async(ts + 16 * c, x);
    tmem_load_wait(x);
    const bool page = have >> c & 1u;
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      float2 y;
      y.x = ex2(__fsub_rn(prefill_logit<MODE>(x[i], key0, 16 * c + i, away, page, l), ref));
      y.y = ex2(__fsub_rn(prefill_logit<MODE>(x[i + 1], key0, 16 * c + i + 1, away, page, l), ref));
      sum2 = __fadd2_rn(sum2, y);
      h[8 * c + i / 2] = pack_f16x2(y.x, y.y);
    }
  }
  return sum2.x + sum2.y;
}
// The largest logit of a row's step, by logit, too.
template <int MODE>
__device__ __forceinline__ float prefill_maximum_by_logit(uint32_t ts, int key0, uint32_t have, const PrefillLogits& l) {
  float m = -INFINITY;
  const float away = static_cast<float>(key0 - l.own);
#pragma unroll 1
  for (int c = 0; c < 8; ++c) {
    uint32_t x[16];
    tmem_load_16cols_async(ts + 16 * c, x);
    tmem_load_wait(x);
    const bool page = have >> c & 1u;
    const float at = away + static_cast<float>(16 * c);
#pragma unroll
    for (int i = 0; i < 16; i += 2)
      m = max3(m, prefill_logit<MODE>(x[i], key0 + 16 * c, i, at, page, l),
               prefill_logit<MODE>(x[i + 1], key0 + 16 * c, i + 1, at, page, l));
  }
  return m;
}
// The same where the step lies on one side of the row's own place, so that the bias is a
// straight line: `base` is its value at the row's own place (with the reference, and the cap,
// taken in), `grow` what it grows by from key to key.  Pairs of floats.  The cap's reciprocals
// come two at a time from one, of their product, whose factors are held to 2^60, where tanh is
// long 1 to the last bit (when it was chosen, a prompt of 4096, 32 heads of 128, took 221 us so, 235
// with one for each and 239 with one for four, whose chains are longer).
// Logits i .. i + 3 of x, the keys from `key` on; t and tb are the line at the two pairs.  EDGE:
// keys that the row does not see (by prefill_bits where there is a bias, 5 % faster, by
// comparisons where there is only a cap, 5 % faster again: registers) are -infinity.
template <int MODE, bool EDGE>
__device__ __forceinline__ void prefill_line_4(const uint32_t (&x)[16], int i, int key, bool page, uint32_t bits,
                                               const PrefillLogits& l, float2 t, float2 tb, float2& y, float2& z) {
  const float2 fac2 = make_float2(l.fac, l.fac);
  const float2 cap2 = make_float2(-2.0f * l.cap, -2.0f * l.cap), one2 = make_float2(1.0f, 1.0f);
  float2 a = make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1]));
  float2 b = make_float2(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
  bool seen[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) seen[k] = !EDGE || (has_bias(MODE) ? (bits >> (i + k) & 1u) != 0 : l.sees(key + i + k, page));
  if (EDGE) {
    if (has_cap(MODE)) {                           // what is in the other keys' place must not meet theirs
      a = make_float2(seen[0] ? a.x : 0.0f, seen[1] ? a.y : 0.0f);
      b = make_float2(seen[2] ? b.x : 0.0f, seen[3] ? b.y : 0.0f);
    }
  }
  if constexpr (has_cap(MODE)) {
    const float2 u = __fmul2_rn(a, fac2), v = __fmul2_rn(b, fac2);
    const float2 d = __fadd2_rn(make_float2(ex2(min_nan(u.x, 60.0f)), ex2(min_nan(u.y, 60.0f))), one2);
    const float2 e = __fadd2_rn(make_float2(ex2(min_nan(v.x, 60.0f)), ex2(min_nan(v.y, 60.0f))), one2);
    const float2 w = make_float2(rcp(d.x * d.y), rcp(e.x * e.y));
    y = __ffma2_rn(__fmul2_rn(make_float2(w.x, w.x), make_float2(d.y, d.x)), cap2, t);
    z = __ffma2_rn(__fmul2_rn(make_float2(w.y, w.y), make_float2(e.y, e.x)), cap2, tb);
  } else {
    y = __ffma2_rn(a, fac2, t);
    z = __ffma2_rn(b, fac2, tb);
  }
  if (EDGE) {
    y = make_float2(seen[0] ? y.x : -INFINITY, seen[1] ? y.y : -INFINITY);
    z = make_float2(seen[2] ? z.x : -INFINITY, seen[3] ? z.y : -INFINITY);
  }
}
// Bit i: the row sees key `key` + i, i < 16.
__device__ __forceinline__ uint32_t prefill_bits(const PrefillLogits& l, int key, bool page) {
  const int lo = min(max(l.from - key, 0), 16), hi = min(max(l.lim - key, lo), 16);
  return page ? (1u << hi) - (1u << lo) : 0u;
}
// The line at keys i and i + 1 of 16, from its value `start` at the first of these (begun anew for
// every 16 keys, so that its roundings are of the size of these keys' biases).
template <int MODE>
__device__ __forceinline__ float2 prefill_line_at(float start, float grow, int i) {
  return has_bias(MODE) ? make_float2(fmaf(grow, static_cast<float>(i), start), fmaf(grow, static_cast<float>(i + 1), start))
                        : make_float2(start, start);
}
template <int MODE, bool EDGE>
__device__ __forceinline__ float2 prefill_line_16(const uint32_t (&x)[16], int c, int key0, uint32_t have,
                                                  const PrefillLogits& l, float base, float away, float grow,
                                                  float2 sum2,
                                                  uint32_t (&h)[64]) {
  const float start = has_bias(MODE) ? fmaf(grow, away + 16.0f * c, base) : base;
  const uint32_t bits = EDGE ? prefill_bits(l, key0 + 16 * c, have >> c & 1u) : 0u;
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    float2 y, z;
    prefill_line_4<MODE, EDGE>(x, i, key0 + 16 * c, have >> c & 1u, bits, l, prefill_line_at<MODE>(start, grow, i),
                               prefill_line_at<MODE>(start, grow, i + 2), y, z);
    y.x = ex2(y.x);
    y.y = ex2(y.y);
    z.x = ex2(z.x);
    z.y = ex2(z.y);
    sum2 = __fadd2_rn(sum2, __fadd2_rn(y, z));
    h[8 * c + i / 2] = pack_f16x2(y.x, y.y);
    h[8 * c + i / 2 + 1] = pack_f16x2(z.x, z.y);
  }
  return sum2;
}
// The largest logit of a row's step (base without the reference).
template <int MODE>
__device__ __forceinline__ float prefill_maximum_line(uint32_t ts, int key0, uint32_t have, const PrefillLogits& l,
                                                      float base, float away, float grow) {
  float m = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 8; ++c) {
    uint32_t x[16];
    tmem_load_16cols_async(ts + 16 * c, x);
    tmem_load_wait(x);
    const float start = fmaf(grow, away + 16.0f * c, base);
    const uint32_t bits = prefill_bits(l, key0 + 16 * c, have >> c & 1u);
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      float2 y, z;
      prefill_line_4<MODE, true>(x, i, key0 + 16 * c, have >> c & 1u, bits, l, prefill_line_at<MODE>(start, grow, i),
                                 prefill_line_at<MODE>(start, grow, i + 2), y, z);
      m = max3(max3(m, y.x, y.y), z.x, z.y);
    }
  }
  return m;
}
template <int MODE, bool EDGE>
__device__ __forceinline__ float prefill_weights_line(uint32_t ts, int key0, uint32_t have, const PrefillLogits& l,
                                                      float base, float away, float grow, uint32_t (&h)[64]) {
  float2 sum2 = make_float2(0.0f, 0.0f);
  uint32_t a[16], b[16];
  tmem_load_16cols_async(ts, a);
  tmem_load_wait(a);
#pragma unroll
  for (int c = 0; c < 8; c += 2) {
    tmem_load_16cols_async(ts + 16 * c + 16, b);
    sum2 = prefill_line_16<MODE, EDGE>(a, c, key0, have, l, base, away, grow, sum2, h);
    tmem_load_wait(b);
    if (c < 6) tmem_load_16cols_async(ts + 16 * c + 32, a);
    sum2 = prefill_line_16<MODE, EDGE>(b, c + 1, key0, have, l, base, away, grow, sum2, h);
    if (c < 6) tmem_load_wait(a);
  }
  return sum2.x + sum2.y;
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

template <typename T, int D, int MODE = kPlain>
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
  const KvSeen<MODE> seen(p, seq, b);
  // steps of 128 keys: this split's share of what the last row sees, and how many of
  // them each tile's last row sees
  auto limit_of = [&](int r) { return seen.limit(r / p.group); };
  const int from_key = seen.first(r0 / p.group), skip = from_key / kPreKeys;   // (0 of kPlain)
  const int last0 = min(r0 + 128, rows) - 1, last1 = min(r0 + 256, rows) - 1;
  const int all = (max(0, limit_of(last1)) + kPreKeys - 1) / kPreKeys;
  const int per = (max(0, all - skip) + splits - 1) / splits;
  const int t0 = min(all, skip + static_cast<int>(blockIdx.y) * per), t1 = min(all, t0 + per);
  const int all0 = (max(0, limit_of(last0)) + kPreKeys - 1) / kPreKeys;
  // with a bias from the last keys to the first, as it makes logits grow towards a row's own
  // place and every step would move its reference; tile 0 then begins with keys that it may
  // not see
  constexpr bool backwards = has_bias(MODE);
  const int n[2] = {backwards ? t1 - t0 : max(0, min(t1, all0) - t0), r0 + 128 < rows ? t1 - t0 : 0};
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
    for (int i = max(from_key, t0 * kPreKeys) / p.c.page_size + tid; static_cast<int64_t>(i) * p.c.page_size < end; i += kPreThreads) {
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
      fac = kv_factor<MODE>(p, p.sm_scale * kLog2e / kgs * pow2(-k));
    }
    const uint32_t ts = tmem + tile * 128 + ((warp & 3) * 32 << 16);
    const uint32_t to = tmem + 256 + tile * D + ((warp & 3) * 32 << 16);
    const int lim = ok ? limit_of(r) : 0;
    int lim_lo = ok ? lim : INT32_MAX;           // smallest of the warp's rows
    lim_lo = __reduce_min_sync(kFullMask, lim_lo);
    [[maybe_unused]] int from_hi = 0;            // largest first key of the warp's rows
    [[maybe_unused]] int own_lo = 0, own_hi = 0; // the rows' own places
    [[maybe_unused]] PrefillLogits logits;
    const int from = ok ? seen.first(tok) : 0;   // (0 of kPlain)
    if constexpr (MODE != kPlain) from_hi = __reduce_max_sync(kFullMask, from);
    if constexpr (has_bias(MODE) || has_cap(MODE))
      logits = PrefillLogits{fac, has_cap(MODE) ? kLog2e * p.softcap : 0.0f,
                             has_bias(MODE) && ok ? kv_slope(p, hq) : 0.0f, seen.off + tok, from, lim};
    if constexpr (has_bias(MODE)) {
      own_lo = __reduce_min_sync(kFullMask, ok ? seen.off + tok : INT32_MAX);
      own_hi = __reduce_max_sync(kFullMask, ok ? seen.off + tok : INT32_MIN);
    }
    // a straight line of logits (prefill_weights_line) rather than products times a factor; a
    // first key that is not 0
    constexpr bool kLines = has_bias(MODE) || has_cap(MODE), kFrom = MODE != kPlain;
    constexpr int kCoarseRows = INT32_MIN;       // in lim_lo's place: a row's reference is_coarse, or was
    // (places behind the last row take part in steps without an edge: they need a reference,
    // which they would not find in the masked steps)
    float ref = MODE == kPlain || ok ? kRefStart : 0.0f, sum = 0.0f;
    bool alive = true;
    for (int j = 0; j < n[tile]; ++j) {
      const int key0 = (backwards ? t1 - 1 - j : t0 + j) * kPreKeys;
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
      const bool edge = key0 + kPreKeys > lim_lo || have != 0xffu || (MODE != kPlain && key0 < from_hi);
      // the weights against the reference there is; where a row's sum passes the limit
      // (rare after the first step, which begins with its maximum), once more.  A warp that
      // had a coarse reference begins every step so, and rounds S times the factor in place
      // after it: the exponents' code is the usual one, with a factor of 1 (other code for
      // such rows, or two roundings in the masked steps', made every call 1 to 2 % slower)
      // the side of the rows' own places that the step lies on (keys behind them that no row sees
      // do not count)
      [[maybe_unused]] bool line = true;
      [[maybe_unused]] float grow = 0.0f, away = 0.0f;
      if constexpr (has_bias(MODE)) {
        const bool left = key0 + kPreKeys - 1 <= own_lo || (seen.causal && key0 >= seen.prefix);
        line = !has_wide_cap(MODE) && (left || key0 >= own_hi);
        grow = left ? logits.slope : -logits.slope;
        away = static_cast<float>(key0 - logits.own);
      }
      uint32_t h[64];
      float step_sum;
      bool moved = j == 0 || lim_lo == kCoarseRows;
      if constexpr (MODE != kPlain)                // a row's first keys may come later
        moved = lim_lo == kCoarseRows || __any_sync(kFullMask, ref == kRefStart && key0 < lim && key0 + kPreKeys > from);
      bool last = moved;
      const bool blind = kFrom && !__any_sync(kFullMask, key0 < lim && key0 + kPreKeys > from);
      if (blind) {                                 // no row of the warp sees a key of the step
        step_sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 64; ++i) h[i] = 0;
      }
#pragma unroll 1
      while (!blind) {
        if (last) {
          float m;
          if constexpr (has_bias(MODE)) {
            m = line ? prefill_maximum_line<MODE>(ts, key0, have, logits, logits.cap, away, grow)
                     : prefill_maximum_by_logit<MODE>(ts, key0, have, logits);
          } else {
            m = edge ? prefill_maximum<true, kFrom>(ts, key0, lim, from, have)
                     : prefill_maximum<false, kFrom>(ts, key0, lim, from, have);
            if (has_cap(MODE) && m > -INFINITY) m = kv_logit<MODE>(m, fac, logits.cap, 0.0f, 0.0f);
          }
          float f = 1.0f;
          if (moved && m > -INFINITY) {
            const float to_ref = kLines ? fmaxf(ref, m) : ref_for(ref, m, fac);
            f = ex2(ref - to_ref);
            ref = to_ref;
            sum *= f;
          }
          if (j > 0) prefill_scale(to, D / 32, f);
          if (!kLines && (lim_lo == kCoarseRows || __any_sync(kFullMask, is_coarse(ref)))) {
            lim_lo = kCoarseRows;
            prefill_scale(ts, kPreKeys / 32, fac);
            tmem_store_wait();
          }
        }
        if constexpr (!kLines) {
          const float f = lim_lo == kCoarseRows ? 1.0f : fac;
          step_sum = edge ? prefill_weights<true, kFrom>(ts, key0, lim, from, have, f, ref, h)
                          : prefill_weights<false, kFrom>(ts, key0, lim, from, have, f, ref, h);
        } else {
          if (has_wide_cap(MODE) || (has_bias(MODE) && (!line || __any_sync(kFullMask, is_coarse(ref))))) {
            step_sum = prefill_weights_by_logit<MODE>(ts, key0, have, logits, ref, h);
          } else {
            const float base = logits.cap - ref;
            step_sum = edge ? prefill_weights_line<MODE, true>(ts, key0, have, logits, base, away, grow, h)
                            : prefill_weights_line<MODE, false>(ts, key0, have, logits, base, away, grow, h);
          }
        }
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
    int key = (backwards ? t1 - 1 : t0) * kPreKeys + 16 * (lane & 7);
    int idx = key / p.c.page_size, at = key - idx * p.c.page_size;
    int page_of, at_of;                            // the page's number is looked at a step later
    auto next_page = [&]() {
      at_of = at;
      // (16 keys before a window may be in a page that has been given up: zeros stand for them)
      page_of = key < seq.len && (MODE == kPlain || key + 16 > from_key) ? prefill_page(p, b, idx) : -1;
      if (backwards) {
        key -= kPreKeys;
        idx -= page_q;
        at -= page_r;
        if (at < 0) {
          at += p.c.page_size;
          --idx;
        }
      } else {
        key += kPreKeys;
        idx += page_q;
        at += page_r;
        if (at >= p.c.page_size) {
          at -= p.c.page_size;
          ++idx;
        }
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
        prefill_store_v<D>(raw[s], smem0 + S::kV + s * S::kTile, seq.len - (backwards ? t1 - 1 - j : t0 + j) * kPreKeys, pw, lane);
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
