// kv_decode.cuh - attention of few query rows per sequence over the paged NVFP4
// cache: the cache's bytes are read once and bound the time.
//
// An item is (sequence, key/value head, tile of 8 * NT query rows), the rows
// being the sequence's query tokens times the heads that share the key/value
// head.  Products are taken transposed, keys and channels in the 16 rows of
// mma.m16n8k16 and query rows in its 8 columns, so 4 to 8 heads of a group fill
// the tile that 16 rows would leave half empty:
//     S^T [16 keys x 8 rows]      = K [16 x D] * Q^T      (D / 16 steps)
//     O^T [D channels x 8 rows]  += V^T [D x 16 keys] * P^T
// Both contractions may run over their index in any order, so a lane takes
// its operands where they lie: of K, D/4 consecutive channels of two keys (one
// load each), and of V, D/8 consecutive channels of four consecutive keys;
// codes become fp16 pairs byte by byte in registers (for V the nibbles of two
// keys are first interleaved), and one multiplication by the block scales
// makes them exact values.  P^T comes from S^T by an 8x8 transposition.
//
// Work split.  Every item is cut into units of 64 keys, the units of all items
// are numbered in order, and CTA c of G takes units [c W / G, (c+1) W / G): the
// CTAs get the same number of keys whatever the lengths are, and each item is
// shared by consecutive CTAs.  Lengths are read on the device.  An item that
// one CTA has whole is finished there; else each CTA leaves its part (O, the
// reference r and the sum l, fp32) in the workspace and a second, small
// kernel joins the parts in order.
//
// With a window, an item's units begin with the first that one of its sequence's rows sees.  A
// cap and a bias are taken in place of the product (MODE, KvLogits): 16 sequences of 12-16 K tokens,
// 40 query and 8 key/value heads of 128, 58.4 us without, 59.3 with a bias, 61.0 with a cap, 64.7 with
// one above kWideCap.
//
// A CTA is 4 warps, each with its own 16 keys of a unit, its own r, l and O, and
// its own ring of tiles in shared memory that cp.async fills ahead (a tile: 16
// keys' codes and scales, 18 D bytes); no barrier in the loop.
// At the end of an item's segment the four are joined in shared memory.
#pragma once

#include "kv_attention_common.cuh"

namespace fp4q {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kDecUnit = 16 * kDecWarps;       // keys of a unit
constexpr int kDecStages = 4;
constexpr int kDecCluster = 8;                 // CTAs of a cluster that share an item, at most
constexpr int kDecMinUnits = 2;                // a CTA's share is at least this long
// What an item costs besides its keys (its queries, the ring's first tiles, the
// join), in units: the CTAs' shares are even in these too.  Without it the one CTA
// that has all the shortest sequences works on long after the others.
constexpr int kDecItemCost = 6;

template <int D, int NT>
struct DecodeShape {
  static constexpr int kRows = 8 * NT;
  static constexpr int kTile = 18 * D;         // bytes of 16 keys: K codes, V codes, K scales, V scales
  static constexpr int kV = 8 * D, kKs = 16 * D, kVs = 17 * D;
  static constexpr int kMergeStride = D + 8;   // floats per row in the merge buffer
  static constexpr int kRing = kDecWarps * kDecStages * kTile;
  static constexpr int kMerge = kDecWarps * kRows * kMergeStride * 4;
  static constexpr int kResult = (kRows * D + 4 * kRows) * 4;   // what a cluster's CTAs read of each other
  static constexpr int kSmem = kRing > kMerge ? kRing : kMerge;
  static constexpr int kSmemCluster = kRing > kMerge + kResult ? kRing : kMerge + kResult;
  // CTAs per SM, and with them registers per thread (128, 168 or 255), and tiles a warp
  // takes per step.  Two tiles share the loop's, the addresses' and the maximum's
  // instructions and fill each other's waits.  Registers count for more than warps
  // with 128 channels: 128 sequences of 12-16 K tokens, 8 rows, 382 us with four CTAs,
  // 358 with three, 405 with two; 16 rows 63 us with three, 58 with two.  With 64
  // channels it is the other way: 8 rows 68 us with four, 74 with three, 76 with five.
  static constexpr int kCtas = D == 128 ? (NT == 1 ? 3 : 2) : (NT == 1 ? 4 : 3);
  static constexpr int kStep = NT == 1 || D == 128 ? 2 : 1;
  static constexpr int kPart = kRows * (D + 2);   // floats of one part in the workspace
};

// Workspace: 2 G parts, then one {first CTA, parts} pair per item.
__host__ __device__ inline int64_t decode_row_slots(int64_t B, int64_t T, int group, int rows) {
  return T * group / rows + B;
}

template <int OFF> __device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0+%2], [%1], 16;" :: "r"(dst), "l"(src), "n"(OFF) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}
// Shared-memory loads at a register address and a constant offset.
template <int OFF> __device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1+%2];" : "=r"(v) : "r"(a), "n"(OFF) : "memory");
  return v;
}
template <int OFF> __device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u16 %0, [%1+%2];" : "=r"(v) : "r"(a), "n"(OFF) : "memory");
  return v;
}
template <int OFF> __device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1+%2];" : "=r"(v) : "r"(a), "n"(OFF) : "memory");
  return v;
}
template <int W, int OFF> __device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&w)[W]) {
  if constexpr (W == 4)
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4+%5];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(a), "n"(OFF) : "memory");
  else if constexpr (W == 2)
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2+%3];" : "=r"(w[0]), "=r"(w[1]) : "r"(a), "n"(OFF) : "memory");
  else
    w[0] = lds32<OFF>(a);
}
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Places of the 16-byte pieces of a tile's K and V codes: rows (keys) are D/2
// bytes.  Chosen so that the lanes of one load (K: keys {0,1,4,5,...}, four
// pieces each; V: keys {i, 4+i, 8+i, 12+i}, every piece) fall on different banks.
template <int D> __device__ __forceinline__ int k_place(int row, int piece) {
  if (D == 128) return row * 64 + piece * 16;
  const int slot = (row & 9) | ((row & 2) << 1) | ((row & 4) >> 1);
  return slot * 32 + piece * 16;
}
template <int D> __device__ __forceinline__ int v_place(int row, int piece) {
  if (D == 128) return (row ^ ((row >> 2) & 1)) * 64 + ((piece ^ (row >> 2)) & 3) * 16;
  return ((row >> 2) | ((row & 3) << 2)) * 32 + piece * 16;
}

template <int V> struct Const { static constexpr int value = V; };

__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// One row's result in 8 channels: o relative to 2^ref, l the sum of weights.
template <typename T, int D>
__device__ __forceinline__ void decode_write(const KvAttentionParams& p, const KvSeq& s, int kvh, int row, int d0,
                                             const float (&o)[8], float ref, float l, float vgs) {
  const int tok = row / p.group;
  const int64_t at = static_cast<int64_t>(s.q0 + tok) * p.Hq + kvh * p.group + row - tok * p.group;
  const float inv = l > 0.0f ? 1.0f / (l * vgs) : l == 0.0f ? 0.0f : l;   // NaN stays
  T* dst = static_cast<T*>(p.out) + at * D + d0;
  if (FP4Q_IN_RANGE(p, dst, 16, p.out, 2LL * p.T * p.Hq * D))
    *reinterpret_cast<uint4*>(dst) = make_uint4(
        Pair<T>::from_f32(o[0] * inv, o[1] * inv), Pair<T>::from_f32(o[2] * inv, o[3] * inv),
        Pair<T>::from_f32(o[4] * inv, o[5] * inv), Pair<T>::from_f32(o[6] * inv, o[7] * inv));
  if (d0 == 0 && p.lse && FP4Q_IN_RANGE(p, p.lse + at, 4, p.lse, 4LL * p.T * p.Hq))
    p.lse[at] = l == 0.0f ? -INFINITY : kLn2 * (ref + log2f(l));
}

// The sequence of row slot rs, and which of its row tiles that is: the last sequence
// whose slots begin at or before rs (the tile may lie behind the sequence's last).
template <int ROWS>
__device__ __forceinline__ int decode_sequence(const KvAttentionParams& p, int64_t rs, int64_t& tile) {
  auto slots_from = [&](int b) {
    const int64_t q0 = p.cu ? min(max(kv_cu(p, b), 0), static_cast<int>(p.T)) : b;
    return q0 * p.group / ROWS + b;
  };
  int b = 0, hi = p.B - 1;
  while (b < hi) {
    const int mid = (b + hi + 1) / 2;
    if (slots_from(mid) <= rs) b = mid; else hi = mid - 1;
  }
  tile = rs - slots_from(b);
  return b;
}

// What one CTA's walk over the units needs to know of the sequence it is in.
struct DecodeWalk {
  int b;             // sequence
  int64_t base;      // its first unit
  int skip;          // units of keys before the first that a row sees
  int tiles;         // units of keys per item
  int cost;          // kDecItemCost + tiles: places per item in the numbering
  int row_tiles;     // row tiles
  KvSeq s;
};
template <int ROWS, int MODE>
__device__ __forceinline__ int64_t decode_units(const KvAttentionParams& p, int b, DecodeWalk& w) {
  w.s = kv_sequence(p, b);
  w.b = b;
  w.skip = MODE != kPlain && p.window ? max(0, w.s.len - w.s.n_q + 1 - p.window) / kDecUnit : 0;
  // a sequence without keys still has a unit: its rows are written as 0
  w.tiles = max(1, (w.s.len + kDecUnit - 1) / kDecUnit - w.skip);
  w.cost = w.tiles + kDecItemCost;
  w.row_tiles = (w.s.n_q * p.group + ROWS - 1) / ROWS;
  return static_cast<int64_t>(w.cost) * w.row_tiles * p.c.heads;
}

// CLUSTER: instead, an item's keys go to one CTA or to the 2 to 8 of a cluster, which
// read each other's results from shared memory: no workspace and no second kernel, for
// short sequences and for few of moderate length (kv_attention.cu chooses).
template <typename T, int D, int NT, bool CLUSTER, int MODE = kPlain>
__global__ void __launch_bounds__(kDecThreads, DecodeShape<D, NT>::kCtas)
kv_decode_kernel(const KvAttentionParams p) {
  using S = DecodeShape<D, NT>;
  constexpr int ROWS = S::kRows;
  constexpr int KW = D / 32;          // words of K a lane takes of one key
  constexpr int VW = D / 64;          // words of V a lane takes of one key
  constexpr int TP = S::kStep;
  constexpr int AHEAD = kDecStages / TP - 1;     // steps whose tiles are on their way
  constexpr int kNoKey = INT32_MAX - 64;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t scan_tot[kDecThreads / 32];
  __shared__ int64_t start_base;
  __shared__ int start_b;
  __shared__ float merge_r[kDecWarps][ROWS], merge_l[kDecWarps][ROWS];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  griddep_wait();
  griddep_launch_dependents();

  const int64_t cta = blockIdx.x;
  DecodeWalk w;
  int64_t total = 0, G = 0, units = 0, u = 0, u_end = 1;
  int kvh = 0, rt = 0;                           // key/value head, tile of rows
  const int rank = CLUSTER ? static_cast<int>(cluster_ctarank()) : 0;
  const int peers = CLUSTER ? static_cast<int>(cluster_nctarank()) : 1;
  if constexpr (CLUSTER) {
    const int64_t slot = cta / peers;
    kvh = static_cast<int>(slot % p.c.heads);
    int64_t tile;
    const int b = decode_sequence<ROWS>(p, slot / p.c.heads, tile);
    decode_units<ROWS, MODE>(p, b, w);
    if (tile < 0 || tile >= w.row_tiles) return;   // the whole cluster
    rt = static_cast<int>(tile);
  } else {
    // total units, and the sequence that holds this CTA's first one: each thread
    // sums a run of consecutive sequences
    const int run = (p.B + kDecThreads - 1) / kDecThreads;
    const int b_lo = min(tid * run, p.B), b_hi = min(b_lo + run, p.B);
    int64_t mine = 0;
    for (int b = b_lo; b < b_hi; ++b) mine += decode_units<ROWS, MODE>(p, b, w);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(kFullMask, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) scan_tot[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine;
#pragma unroll
    for (int i = 0; i < kDecThreads / 32; ++i) {
      if (i < warp) before += scan_tot[i];
      total += scan_tot[i];
    }
    G = (total + kDecMinUnits - 1) / kDecMinUnits;
    if (G > static_cast<int64_t>(gridDim.x)) G = gridDim.x;
    if (cta >= G) return;
    u = cta * total / G;
    u_end = (cta + 1) * total / G;
    if (u >= before && u < before + mine) {       // exactly one thread
      int64_t base = before;
      int b = b_lo;
      for (;;) {
        const int64_t n = decode_units<ROWS, MODE>(p, b, w);
        if (u < base + n) break;
        base += n;
        ++b;
      }
      start_b = b;
      start_base = base;
    }
    __syncthreads();
    units = decode_units<ROWS, MODE>(p, start_b, w);
    w.base = start_base;
  }

  const uint32_t ring = smem_addr(smem) + warp * kDecStages * S::kTile;   // this warp's
  const float kgs = p.c.k_gs ? __ldg(p.c.k_gs) : 1.0f;
  const float vgs = p.c.v_gs ? __ldg(p.c.v_gs) : 1.0f;
  const int row_k = 4 * (g >> 1) + (g & 1);     // key of tile row g; row g + 8 is key row_k + 2
  // what a lane copies of a tile: 16-byte pieces of K and V codes, 32 pieces (512
  // bytes of the source) apart, and one piece of the scales (D/16 lanes K, D/16 V:
  // a block's 16 scales, which lie page_size apart per block and not per key)
  constexpr int kPieces = D / 32;               // per key
  const uint8_t* const k_lane = p.c.k_packed + lane * 16;
  const uint8_t* const v_lane = p.c.v_packed + lane * 16;
  const uint32_t k_dst = ring + k_place<D>(lane / kPieces, lane % kPieces);
  const uint32_t v_dst = ring + S::kV + v_place<D>(lane / kPieces, lane % kPieces);
  const uint32_t s_dst = ring + S::kKs + lane * 16;
  constexpr int kRows1 = 32 / kPieces;          // keys between a lane's two pieces (D = 128)
  const uint32_t k_dst1 = D == 128 ? ring + k_place<D>(lane / kPieces + kRows1, lane % kPieces) - k_dst : 0;
  const uint32_t v_dst1 = D == 128 ? ring + S::kV + v_place<D>(lane / kPieces + kRows1, lane % kPieces) - v_dst : 0;
  const uint8_t* const s_lane = lane < D / 16 ? p.c.k_sf + lane * 16
                                              : p.c.v_sf + static_cast<int64_t>(lane - D / 16) * p.c.page_size;
  const int s_back = lane < D / 16 ? 0 : D / 16 - 1;
  // what it reads of a tile for the products
  const uint32_t k_src = ring + k_place<D>(row_k, KW * t / 4) + (KW * t % 4) * 4;
  const uint32_t k_src2 = ring + k_place<D>(row_k + 2, KW * t / 4) + (KW * t % 4) * 4;
  const uint32_t ks_src = ring + S::kKs + row_k * (D / 16) + t * (D / 64);
  const uint32_t vs_src = ring + S::kVs + (D == 128 ? g : g / 2) * 16 + 4 * t;
  uint32_t v_src[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v_src[i] = ring + S::kV + v_place<D>(4 * t + i, VW * g / 4) + (VW * g % 4) * 4;

  while (u < u_end) {
    int64_t item_base = 0;
    int tile0, n_units;
    if constexpr (CLUSTER) {
      tile0 = w.tiles * rank / peers;
      n_units = w.tiles * (rank + 1) / peers - tile0;
      u = u_end;                                // one item
    } else {
      while (u >= w.base + units) {             // the next sequence that has units
        w.base += units;
        units = decode_units<ROWS, MODE>(p, w.b + 1, w);
      }
      const int item = static_cast<int>((u - w.base) / w.cost);
      item_base = w.base + static_cast<int64_t>(item) * w.cost;
      kvh = item / w.row_tiles;
      rt = item - kvh * w.row_tiles;
      tile0 = max(0, static_cast<int>(u - item_base) - kDecItemCost);
      n_units = static_cast<int>(min(static_cast<int64_t>(w.cost), u_end - item_base)) - kDecItemCost - tile0;
      u = item_base + w.cost;                   // the next item, or beyond this share
      if (n_units <= 0) continue;               // the share ends in the item's own cost
    }
    const int rows = w.s.n_q * p.group;         // of the whole sequence
    const int r0 = rt * ROWS;

    // --- the rows' limits: keys that columns 2t, 2t + 1 see, smallest and largest of the tile
    const int off = w.s.len - w.s.n_q;          // last visible key of token i: off + i
    const KvSeen<MODE> seen(p, w.s, w.b);
    int lim[NT][2];
    [[maybe_unused]] int from[NT][2];            // first visible keys
    [[maybe_unused]] float slope[NT][2];         // of the distance to the token's own place
    [[maybe_unused]] int own[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rc = r0 + 8 * n + 2 * t + e;
        const int tok = rc / p.group;
        lim[n][e] = rc < rows ? seen.limit(tok) : w.s.len;
        if constexpr (MODE != kPlain) {
          from[n][e] = rc < rows ? seen.first(tok) : 0;
          own[n][e] = off + tok;
          slope[n][e] = rc < rows ? kv_slope(p, kvh * p.group + rc - tok * p.group) : 0.0f;
        }
      }
    const int last = min(r0 + ROWS, rows) - 1;
    const int lim_lo = MODE != kPlain ? seen.limit(r0 / p.group) : p.causal ? off + r0 / p.group + 1 : w.s.len;
    const int lim_hi = MODE != kPlain ? seen.limit(last / p.group) : p.causal ? off + last / p.group + 1 : w.s.len;
    const int from_lo = MODE != kPlain ? seen.first(r0 / p.group) : 0;
    const int from_hi = MODE != kPlain ? seen.first(last / p.group) : 0;

    // --- the ring: tile x of this warp is keys key0(x) ... + 15
    const int first_key = (w.skip + tile0) * kDecUnit + warp * 16;
    const int32_t* table = p.tables + static_cast<int64_t>(w.b) * p.max_pages;
    // with a bias from the last tile to the first, as it makes logits grow towards a row's own place
    // and every step would move its reference
    const bool backwards = MODE != kPlain && p.slopes;
    auto key_of = [&](int x) { return first_key + (backwards ? n_units - 1 - x : x) * kDecUnit; };
    // a row number counts slots of all pages and heads and fits 32 bits
    constexpr uint32_t kNoRow = 0xffffffffu;
    uint32_t row_of = kNoRow, row_next = kNoRow;
    int at_of = 0, at_next = 0;
    auto look_up = [&](int x, uint32_t& row, int& at) {      // tile x + lane
      const int key = key_of(x + lane);
      row = kNoRow;
      // (keys before a window may be in pages that have been given up: they have no row here,
      // and their values are zeros)
      if (x + lane < n_units && key < lim_hi && (MODE == kPlain || key + 16 > from_lo)) {
        const int idx = key / p.c.page_size;
        int page = -1;
        if (FP4Q_IN_RANGE(p, table + idx, 4, p.tables, 4LL * p.B * p.max_pages)) page = __ldg(table + idx);
        if (page >= 0 && page < p.c.num_pages) {
          at = key - idx * p.c.page_size;
          row = (static_cast<uint32_t>(page) * p.c.heads + kvh) * p.c.page_size + at;
        }
      }
    };
    look_up(0, row_of, at_of);
    look_up(32, row_next, at_next);
    // --- the item's queries, as the B operand: lane (g, t) holds channels
    // D/4 * t ... of row g of each 8-row tile; loaded while the pages are looked up
    Chunk qc[NT][D / 64];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = r0 + 8 * n + g;
      const bool ok = r < rows;
      const int tok = r / p.group, hq = kvh * p.group + r - tok * p.group;
      const T* src = static_cast<const T*>(p.q) +
                     static_cast<int64_t>(w.s.q0 + (ok ? tok : 0)) * p.q_stride +
                     static_cast<int64_t>(ok ? hq : 0) * D + t * (D / 4);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        qc[n][i] = Chunk{};
        if (ok && FP4Q_IN_RANGE(p, src + 16 * i, 32, p.q, 2LL * ((p.T - 1) * p.q_stride + p.Hq * D)))
          qc[n][i] = ld_cached_ro(src + 16 * i);
      }
    }
    uint32_t valid = 0;                          // bit i: the tile issued i tiles ago holds keys
    auto issue = [&](int x, auto slot) {
      constexpr int kSlot = decltype(slot)::value * S::kTile;
      if ((x & 31) == 0 && x) {
        row_of = row_next;
        at_of = at_next;
        look_up(x + 32, row_next, at_next);
      }
      const uint32_t row = __shfl_sync(kFullMask, row_of, x & 31);
      const uint32_t at = __shfl_sync(kFullMask, at_of, x & 31);
      valid <<= 1;
      if (row != kNoRow) {
        valid |= 1;
        const uint8_t* kc = k_lane + static_cast<uint64_t>(row) * (D / 2);
        const uint8_t* vc = v_lane + static_cast<uint64_t>(row) * (D / 2);
        const uint8_t* sc = s_lane + static_cast<uint64_t>(row) * (D / 16) - static_cast<uint64_t>(at) * s_back;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          if (FP4Q_IN_RANGE(p, kc + 512 * i, 16, p.c.k_packed, kv_packed_extent(p.c)))
            cp_async16<kSlot>(k_dst + (i ? k_dst1 : 0), kc + 512 * i);
          if (FP4Q_IN_RANGE(p, vc + 512 * i, 16, p.c.v_packed, kv_packed_extent(p.c)))
            cp_async16<kSlot>(v_dst + (i ? v_dst1 : 0), vc + 512 * i);
        }
        if (lane < D / 8 && FP4Q_IN_RANGE(p, sc, 16, lane < D / 16 ? p.c.k_sf : p.c.v_sf, kv_sf_extent(p.c)))
          cp_async16<kSlot>(s_dst, sc);
      }
    };
    auto issue_step = [&](int step, auto phase) {
      issue(step * TP, Const<decltype(phase)::value * TP>{});
      if constexpr (TP == 2) issue(step * TP + 1, Const<decltype(phase)::value * TP + 1>{});
      cp_async_commit();
    };
    constexpr int PHASES = kDecStages / TP;      // steps until the ring's slots come again
    issue_step(0, Const<0>{});
    if constexpr (AHEAD > 1) issue_step(1, Const<1>{});
    if constexpr (AHEAD > 2) issue_step(2, Const<2>{});

    uint32_t qf[NT][D / 16][2];
    float fac[NT][2], ref[NT][2], sum[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float top = 0.0f;
      bool nan = false;
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 x = Pair<T>::to_f32(qc[n][i].u[j]);
          top = max_abs3(top, x.x, x.y);
          nan |= x.x != x.x || x.y != x.y;
        }
      if (nan) top = INFINITY;                  // no scaling: the row is NaN whatever is done
      top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
      const int k = q_exponent(top);
      // a row with an infinity or NaN is NaN, and its products with every key are
      const float up = top < INFINITY ? pow2(k) : __uint_as_float(0x7fc00000u);
#pragma unroll
      for (int i = 0; i < D / 64; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 x = Pair<T>::to_f32(qc[n][i].u[j]);
          qf[n][4 * i + j / 2][j & 1] = pack_f16x2(x.x * up, x.y * up);
        }
      const float f = kv_factor<MODE>(p, p.sm_scale * kLog2e / kgs * pow2(-k));
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        fac[n][e] = __shfl_sync(kFullMask, f, (2 * t + e) * 4);
        ref[n][e] = kRefStart;
        sum[n][e] = 0.0f;
      }
    }

    float acc[NT][D / 16][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][i][e] = 0.0f;

    // a reference of the warp's rows is_coarse: its steps take the masked steps' code, where
    // the product is rounded before the reference is taken from it
    bool coarse = false;
    [[maybe_unused]] const float cap = has_cap(MODE) ? kLog2e * p.softcap : 0.0f;
    // one step, whose slots of the ring are constants
    auto work = [&](int step, auto phase) {
      constexpr int kPhase = decltype(phase)::value;
      cp_async_wait<AHEAD - 1>();
      __syncwarp();                              // the step's tiles are here for every lane, the last one's read
      const uint32_t here = valid >> (TP * (AHEAD - 1)) & ((1u << TP) - 1);   // bit TP - 1: the first tile
      issue_step(step + AHEAD, Const<(kPhase + AHEAD) % PHASES>{});
      if (!here) return;
      constexpr int kAt[2] = {kPhase * TP * S::kTile, (kPhase * TP + TP - 1) * S::kTile};
      int key0[TP];                              // a tile without keys lies behind every limit
#pragma unroll
      for (int j = 0; j < TP; ++j)
        key0[j] = here >> (TP - 1 - j) & 1u ? key_of(step * TP + j) : kNoKey;

      // S^T = K Q^T
      float s[TP][NT][4];
      auto products = [&](auto tile) {
        constexpr int j = decltype(tile)::value, at = kAt[j];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[j][n][e] = 0.0f;
        uint32_t ka[KW], kb[KW], sa[2], sb[2];
        lds_words<KW, at>(k_src, ka);
        lds_words<KW, at>(k_src2, kb);
        if constexpr (D == 128) {                // two blocks per lane
          const uint32_t fa = e4m3x2_to_f16x2(lds16<at>(ks_src));
          const uint32_t fb = e4m3x2_to_f16x2(lds16<at + 16>(ks_src));
          sa[0] = __byte_perm(fa, 0, 0x1010);
          sa[1] = __byte_perm(fa, 0, 0x3232);
          sb[0] = __byte_perm(fb, 0, 0x1010);
          sb[1] = __byte_perm(fb, 0, 0x3232);
        } else {
          const uint32_t ba = lds8<at>(ks_src), bb = lds8<at + 8>(ks_src);
          sa[0] = sa[1] = e4m3x2_to_f16x2(ba | ba << 8);
          sb[0] = sb[1] = e4m3x2_to_f16x2(bb | bb << 8);
        }
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          uint32_t ha[4], hb[4];
          e2m1x8_to_f16x2(ka[i], ha);
          e2m1x8_to_f16x2(kb[i], hb);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            ha[e] = mul_f16x2(ha[e], sa[i / 2]);
            hb[e] = mul_f16x2(hb[e], sb[i / 2]);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_16816(s[j][n], ha[0], hb[0], ha[1], hb[1], qf[n][2 * i][0], qf[n][2 * i][1]);
            mma_16816(s[j][n], ha[2], hb[2], ha[3], hb[3], qf[n][2 * i + 1][0], qf[n][2 * i + 1][1]);
          }
        }
      };
      products(Const<0>{});
      if constexpr (TP == 2) products(Const<1>{});

      // exponents of 2 against the reference; keys that a row does not see get -inf
      float y[TP][NT][4];
      bool over = false, edge = coarse;
#pragma unroll
      for (int j = 0; j < TP; ++j) {
        edge |= key0[j] > lim_lo - 16;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (MODE == kPlain) {
              y[j][n][e] = fmaf(s[j][n][e], fac[n][e & 1], -ref[n][e & 1]);
            } else {                             // the logit itself in the product's place, rounded once
              const float away = static_cast<float>(key0[j] - own[n][e & 1]) + static_cast<float>(row_k + (e & 2));
              s[j][n][e] = kv_logit<MODE>(s[j][n][e], fac[n][e & 1], cap, slope[n][e & 1], away);
              y[j][n][e] = __fsub_rn(s[j][n][e], ref[n][e & 1]);
            }
          }
      }
      if constexpr (MODE != kPlain) {
#pragma unroll
        for (int j = 0; j < TP; ++j) edge |= key0[j] < from_hi;
        if (edge) {
#pragma unroll
          for (int j = 0; j < TP; ++j)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int key = key0[j] + row_k + (e & 2);
                if (key >= lim[n][e & 1] || key < from[n][e & 1]) y[j][n][e] = s[j][n][e] = -INFINITY;
              }
        }
      } else if (edge) {
#pragma unroll
        for (int j = 0; j < TP; ++j)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              y[j][n][e] = coarse_exponent(s[j][n][e], fac[n][e & 1], ref[n][e & 1]);
              if (key0[j] + row_k + (e & 2) >= lim[n][e & 1]) y[j][n][e] = s[j][n][e] = -INFINITY;
            }
      }
#pragma unroll
      for (int j = 0; j < TP; ++j)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) over |= y[j][n][e] > kRefSlack;
      if (__any_sync(kFullMask, over)) {         // rare after the first tiles
        bool far = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = fmaxf(s[0][n][e], s[0][n][e + 2]);
            if (TP == 2) m = fmaxf(m, fmaxf(s[TP - 1][n][e], s[TP - 1][n][e + 2]));
            m = fmaxf(m, __shfl_xor_sync(kFullMask, m, 4));
            m = fmaxf(m, __shfl_xor_sync(kFullMask, m, 8));
            m = fmaxf(m, __shfl_xor_sync(kFullMask, m, 16));
            // (a logit that is rounded already stands for its product, with a factor of 1)
            const float r = ref_for(ref[n][e], m, MODE == kPlain ? fac[n][e] : 1.0f);
            const float f = ex2(ref[n][e] - r);
            ref[n][e] = r;
            far |= MODE == kPlain && is_coarse(r);   // (a logit that is rounded needs no other code)
            sum[n][e] *= f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              acc[n][i][e] *= f;
              acc[n][i][e + 2] *= f;
            }
          }
        coarse = __any_sync(kFullMask, far);
#pragma unroll
        for (int j = 0; j < TP; ++j)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              y[j][n][e] = s[j][n][e] == -INFINITY ? -INFINITY
                                                   : coarse_exponent(s[j][n][e], MODE == kPlain ? fac[n][e & 1] : 1.0f,
                                                                     ref[n][e & 1]);
      }
      uint32_t pb[TP][NT][2];
#pragma unroll
      for (int j = 0; j < TP; ++j)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[j][n][e] = ex2(y[j][n][e]);
            sum[n][e & 1] += y[j][n][e];
          }
          pb[j][n][0] = transpose8x8(pack_f16x2(y[j][n][0], y[j][n][1]));
          pb[j][n][1] = transpose8x8(pack_f16x2(y[j][n][2], y[j][n][3]));
        }

      // O^T += V^T P^T: keys 4t .. 4t + 3 of each tile
      auto values = [&](auto tile) {
        constexpr int j = decltype(tile)::value, at = kAt[j];
        uint32_t sv = lds32<at>(vs_src);
        if (edge && key0[j] > w.s.len - 16) {    // slots behind the end may hold no numbers
          const int left = w.s.len - key0[j] - 4 * t;
          sv = left <= 0 ? 0u : left >= 4 ? sv : sv & (0xffffffffu >> (32 - 8 * left));
        }
        const uint32_t s01 = e4m3x2_to_f16x2(sv), s23 = e4m3x2_to_f16x2(sv >> 16);
        uint32_t v[4][VW];
#pragma unroll
        for (int i = 0; i < 4; ++i) lds_words<VW, at>(v_src[i], v[i]);
#pragma unroll
        for (int i = 0; i < VW; ++i) {
          uint32_t e01[4], o01[4], e23[4], o23[4];
          e2m1x8_to_f16x2(low_nibbles_of(v[0][i], v[1][i] << 4), e01);
          e2m1x8_to_f16x2(low_nibbles_of(v[0][i] >> 4, v[1][i]), o01);
          e2m1x8_to_f16x2(low_nibbles_of(v[2][i], v[3][i] << 4), e23);
          e2m1x8_to_f16x2(low_nibbles_of(v[2][i] >> 4, v[3][i]), o23);
#pragma unroll
          for (int c = 0; c < 4; ++c) {          // channels D/8 g + 8 i + 2 c and the next
            const uint32_t a0 = mul_f16x2(e01[c], s01), a1 = mul_f16x2(o01[c], s01);
            const uint32_t a2 = mul_f16x2(e23[c], s23), a3 = mul_f16x2(o23[c], s23);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma_16816(acc[n][4 * i + c], a0, a1, a2, a3, pb[j][n][0], pb[j][n][1]);
          }
        }
      };
      values(Const<0>{});
      if constexpr (TP == 2) values(Const<1>{});
    };
    const int steps = (n_units + TP - 1) / TP;
    for (int step = 0; step < steps; step += PHASES) {
      work(step, Const<0>{});
      if (step + 1 < steps) work(step + 1, Const<1>{});
      if constexpr (PHASES > 2) {
        if (step + 2 < steps) work(step + 2, Const<2>{});
        if (step + 3 < steps) work(step + 3, Const<3>{});
      }
    }
    cp_async_wait<0>();

    // --- join the four warps
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        sum[n][e] += __shfl_xor_sync(kFullMask, sum[n][e], 4);
        sum[n][e] += __shfl_xor_sync(kFullMask, sum[n][e], 8);
        sum[n][e] += __shfl_xor_sync(kFullMask, sum[n][e], 16);
        if (g == 0) {
          merge_r[warp][8 * n + 2 * t + e] = ref[n][e];
          merge_l[warp][8 * n + 2 * t + e] = sum[n][e];
        }
      }
    __syncthreads();                             // every warp is done with its ring
    float* mo = reinterpret_cast<float*>(smem) + warp * ROWS * S::kMergeStride;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * n + 2 * t + e;
        float top = merge_r[0][r];
#pragma unroll
        for (int i = 1; i < kDecWarps; ++i) top = fmaxf(top, merge_r[i][r]);
        const float f = ex2(ref[n][e] - top);
#pragma unroll
        for (int i = 0; i < D / 16; ++i)         // channels D/8 g + 2 i, + 1 at 16 i + 2 g, + 1
          *reinterpret_cast<float2*>(mo + r * S::kMergeStride + 16 * i + 2 * g) =
              make_float2(acc[n][i][e] * f, acc[n][i][e + 2] * f);
      }
    __syncthreads();
    const bool whole_item = n_units == w.tiles;
    // a part that begins the item is this CTA's last, one that does not its first
    float* part = p.ws + (2 * cta + (tile0 == 0 ? 1 : 0)) * S::kPart;
    const float* m0 = reinterpret_cast<const float*>(smem);
    float* c_out = reinterpret_cast<float*>(smem + S::kMerge);   // CLUSTER: this CTA's results
    for (int x = tid; x < ROWS * (D / 8); x += kDecThreads) {
      const int r = x / (D / 8), d0 = (x % (D / 8)) * 8;
      float top = merge_r[0][r];
#pragma unroll
      for (int i = 1; i < kDecWarps; ++i) top = fmaxf(top, merge_r[i][r]);
      float l = 0.0f;
#pragma unroll
      for (int i = 0; i < kDecWarps; ++i) l += merge_l[i][r] * ex2(merge_r[i][r] - top);
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const int d = d0 + j, gg = d / (D / 8), i = (d % (D / 8)) / 2;
        float2 a = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kDecWarps; ++k) {
          const float2 y = *reinterpret_cast<const float2*>(m0 + (k * ROWS + r) * S::kMergeStride +
                                                            16 * i + 2 * gg);
          a.x += y.x;
          a.y += y.y;
        }
        o[j] = a.x;
        o[j + 1] = a.y;
      }
      const int row = r0 + r;
      if (row >= rows) continue;
      if (CLUSTER && peers > 1) {
        float* co = c_out + r * D + d0;
        *reinterpret_cast<float4*>(co) = make_float4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<float4*>(co + 4) = make_float4(o[4], o[5], o[6], o[7]);
        if (d0 == 0) *reinterpret_cast<float4*>(c_out + ROWS * D + 4 * r) = make_float4(top, l, 0.0f, 0.0f);
      } else if (CLUSTER || whole_item) {
        decode_write<T, D>(p, w.s, kvh, row, d0, o, top, l, vgs);
      } else {
        float4* po = reinterpret_cast<float4*>(part + r * D + d0);
        if (FP4Q_IN_RANGE(p, po, 32, p.ws, p.ws_bytes)) {
          po[0] = make_float4(o[0], o[1], o[2], o[3]);
          po[1] = make_float4(o[4], o[5], o[6], o[7]);
        }
        float* rl = part + ROWS * D + 2 * r;
        if (d0 == 0 && FP4Q_IN_RANGE(p, rl, 8, p.ws, p.ws_bytes))
          *reinterpret_cast<float2*>(rl) = make_float2(top, l);
      }
    }
    if constexpr (CLUSTER) {
      if (peers == 1) return;
      cluster_arrive_release();
      cluster_wait_acquire();                    // every CTA's results are there
      const uint32_t mine = smem_addr(c_out);
      for (int x = tid * peers + rank; x < ROWS * (D / 8); x += kDecThreads * peers) {
        const int r = x / (D / 8), d0 = (x % (D / 8)) * 8;
        if (r0 + r >= rows) continue;
        float4 rl[kDecCluster];
        float top = kRefStart, l = 0.0f;
        float o[8] = {};
#pragma unroll
        for (int i = 0; i < kDecCluster; ++i) {
          // (a smaller cluster's last CTA again: the loads stay side by side)
          rl[i] = ld_peer_f32x4(peer_smem_addr(mine + (ROWS * D + 4 * r) * 4, min(i, peers - 1)));
          top = fmaxf(top, rl[i].x);
        }
#pragma unroll
        for (int i = 0; i < kDecCluster; ++i) {
          const uint32_t peer = peer_smem_addr(mine + (r * D + d0) * 4, min(i, peers - 1));
          const float4 y = ld_peer_f32x4(peer), z = ld_peer_f32x4(peer + 16);
          if (i >= peers) continue;
          const float f = ex2(rl[i].x - top);
          l += rl[i].y * f;
          o[0] += y.x * f;
          o[1] += y.y * f;
          o[2] += y.z * f;
          o[3] += y.w * f;
          o[4] += z.x * f;
          o[5] += z.y * f;
          o[6] += z.z * f;
          o[7] += z.w * f;
        }
        decode_write<T, D>(p, w.s, kvh, r0 + r, d0, o, top, l, vgs);
      }
      cluster_arrive_release();
      cluster_wait_acquire();                    // no CTA leaves while another reads from it
      return;
    }
    if (tid == 0 && tile0 == 0) {
      // where the joining kernel finds the item's parts
      const int64_t slot = (static_cast<int64_t>(w.s.q0) * p.group / ROWS + w.b + rt) * p.c.heads + kvh;
      const int64_t last = item_base + w.cost - 1;
      const int n = static_cast<int>(((last + 1) * G - 1) / total - cta) + 1;
      int* desc = reinterpret_cast<int*>(p.ws + 2 * static_cast<int64_t>(gridDim.x) * S::kPart) + 2 * slot;
      if (FP4Q_IN_RANGE(p, desc, 8, p.ws, p.ws_bytes)) {
        desc[0] = static_cast<int>(cta);
        desc[1] = n;
      }
    }
    __syncthreads();                             // the merge buffer becomes the ring again
  }
}

// Joins the parts of the items that several CTAs shared: block = (item, row),
// D / 4 lanes per part, parts taken in turn by the block's groups of lanes and
// summed in order.
constexpr int kJoinMost = 512;                 // threads of a block at most
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kJoinMost) kv_decode_join_kernel(const KvAttentionParams p, int ctas) {
  using S = DecodeShape<D, NT>;
  constexpr int ROWS = S::kRows;
  constexpr int LANES = D / 4;
  const int groups = blockDim.x / LANES;
  __shared__ float red[kJoinMost / 32];
  __shared__ float4 o_part[kJoinMost / LANES][LANES];
  __shared__ float l_part[kJoinMost / LANES];
  const int tid = threadIdx.x;
  const int64_t slot = blockIdx.x;
  const int kvh = static_cast<int>(slot % p.c.heads), r = blockIdx.y;
  const int64_t rs = slot / p.c.heads;
  griddep_wait();
  griddep_launch_dependents();
  int64_t rt;
  const int b = decode_sequence<ROWS>(p, rs, rt);
  const KvSeq s = kv_sequence(p, b);
  const int rows = s.n_q * p.group;
  if (rt < 0 || rt * ROWS + r >= rows) return;
  const int row = static_cast<int>(rt) * ROWS + r;
  const int* desc = reinterpret_cast<const int*>(p.ws + 2 * static_cast<int64_t>(ctas) * S::kPart) + 2 * slot;
  if (!FP4Q_IN_RANGE(p, desc, 8, p.ws, p.ws_bytes)) return;
  const int c0 = desc[0], n = desc[1];
  if (n <= 1 || c0 < 0 || n > ctas - c0) return;
  // part i: the last of CTA c0 for i = 0, the first of CTA c0 + i else
  auto part = [&](int i) { return p.ws + (2 * static_cast<int64_t>(c0 + i) + (i == 0 ? 1 : 0)) * S::kPart; };
  float top = kRefStart;
  for (int i = tid; i < n; i += blockDim.x) {
    const float* ref = part(i) + ROWS * D + 2 * r;
    if (FP4Q_IN_RANGE(p, ref, 4, p.ws, p.ws_bytes)) top = fmaxf(top, *ref);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
  if ((tid & 31) == 0) red[tid >> 5] = top;
  __syncthreads();
  for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) top = fmaxf(top, red[i]);
  const int grp = tid / LANES, ln = tid % LANES;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float l = 0.0f;
#pragma unroll 4
  for (int i = grp; i < n; i += groups) {
    const float* q = part(i);
    if (!FP4Q_IN_RANGE(p, q + ROWS * D + 2 * r, 8, p.ws, p.ws_bytes) ||
        !FP4Q_IN_RANGE(p, q + r * D + 4 * ln, 16, p.ws, p.ws_bytes))
      continue;
    const float2 rl = *reinterpret_cast<const float2*>(q + ROWS * D + 2 * r);
    const float4 x = *reinterpret_cast<const float4*>(q + r * D + 4 * ln);
    const float f = ex2(rl.x - top);
    o.x += x.x * f;
    o.y += x.y * f;
    o.z += x.z * f;
    o.w += x.w * f;
    l += rl.y * f;
  }
  o_part[grp][ln] = o;
  if (ln == 0) l_part[grp] = l;
  __syncthreads();
  if (grp) return;
  l = l_part[0];
  for (int i = 1; i < groups; ++i) {
    const float4 x = o_part[i][ln];
    o.x += x.x;
    o.y += x.y;
    o.z += x.z;
    o.w += x.w;
    l += l_part[i];
  }
  const float vgs = p.c.v_gs ? __ldg(p.c.v_gs) : 1.0f;
  const float inv = l > 0.0f ? 1.0f / (l * vgs) : l == 0.0f ? 0.0f : l;
  const int tok = row / p.group;
  const int64_t at = static_cast<int64_t>(s.q0 + tok) * p.Hq + kvh * p.group + row - tok * p.group;
  T* dst = static_cast<T*>(p.out) + at * D + 4 * ln;
  if (FP4Q_IN_RANGE(p, dst, 8, p.out, 2LL * p.T * p.Hq * D))
    *reinterpret_cast<uint2*>(dst) = make_uint2(Pair<T>::from_f32(o.x * inv, o.y * inv),
                                                Pair<T>::from_f32(o.z * inv, o.w * inv));
  if (ln == 0 && p.lse && FP4Q_IN_RANGE(p, p.lse + at, 4, p.lse, 4LL * p.T * p.Hq))
    p.lse[at] = l == 0.0f ? -INFINITY : kLn2 * (top + log2f(l));
}

}  // namespace fp4q
