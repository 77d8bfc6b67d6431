// kv_cache.cu - what writes and reads back the paged NVFP4 key/value cache:
// append (rotation of queries and keys by their positions, NVFP4 quantization
// of keys and values, the store into the tokens' slots) and gather (slots back
// to 16 bits).
//
// Both only move bytes: append reads 2 bytes per channel of q, k and v and
// writes 2 per channel of q and 9/16 per channel of k and v; gather the
// reverse for k and v.  No value depends on anything outside its own pair of
// 16-channel blocks, so there is no reduction and no shared memory.
//
// Append's work unit is a pair of blocks of one head: for paired channels i and
// i + rot/2 the two blocks that hold the partners, else two neighbours, so a
// rotation never leaves the thread, both blocks are whole, and the 16 cosines
// and sines of a unit are the same for every head of the token.  A warp takes
// one token and 32 / (D/32) heads at a time; a thread keeps its unit's cosines
// and sines in registers over the heads it walks.
#include <algorithm>
#include <type_traits>

#include "async_copy.cuh"
#include "fp4q_launch.h"
#include "fused_common.cuh"
#include "kv_attention_common.cuh"
#include "kv_launch.h"

namespace fp4q {
namespace {

// NVFP4 of 16 values: 8 bytes of codes, and the scale byte (the rule of
// fp4_quantize: quantize.cu).
__device__ __forceinline__ uint64_t quantize_block(const float (&y)[16], float gs, uint32_t& sf) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; i += 2) amax = max_abs3(amax, y[i], y[i + 1]);
  float inv_s;
  sf = e4m3_block_scale(amax, gs, inv_s);
  float v[16];
  const float2 inv2 = make_float2(inv_s, inv_s);
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const float2 vv = __fmul2_rn(make_float2(y[i], y[i + 1]), inv2);
    v[i] = vv.x;
    v[i + 1] = vv.y;
  }
  const uint64_t codes = static_cast<uint64_t>(e2m1_pack8(v)) |
                         (static_cast<uint64_t>(e2m1_pack8(v + 8)) << 32);
  return inv_s > 0.0f ? codes : 0;                  // a zero scale gives +0 codes
}

template <typename T>
__device__ __forceinline__ void unpack(const Chunk& c, float (&y)[16]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 f = Pair<T>::to_f32(c.u[j]);
    y[2 * j] = f.x;
    y[2 * j + 1] = f.y;
  }
}

// The two products and the sum are rounded one by one: the same bits whatever
// the compiler would contract, and the sum of two equal and opposite products
// is 0.
__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

// Where a head of the list q heads, k heads, v heads lies in token t.
struct HeadRow {
  int kind;            // 0 q, 1 k, 2 v
  int head;
};
__device__ __forceinline__ HeadRow head_of(const KvAppendParams& p, int h) {
  const int kind = h < p.Hq ? 0 : h < p.Hq + p.c.heads ? 1 : 2;
  return {kind, kind == 0 ? h : kind == 1 ? h - p.Hq : h - p.Hq - p.c.heads};
}

// One warp: token t, the heads h0 + lane / units, + step, ... of its run of the list
// q heads, k heads, v heads; D / 32 units per head.  The next heads' channels are
// loaded before the present ones are worked on, the first ones before the token's
// position and slot are known.
template <typename T, bool ROT>
__global__ void __launch_bounds__(128, ROT ? 5 : 7) kv_append_kernel(const KvAppendParams p, int heads_per_warp) {
  const int units = p.c.D / 32;
  const int lane = threadIdx.x & 31;
  const int u = lane % units;
  const int step = 32 / units;                      // heads a warp takes at a time
  const int all = p.Hq + 2 * p.c.heads;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (t >= p.T) return;
  int h = blockIdx.y * heads_per_warp + lane / units;
  const int h_end = min(all, static_cast<int>(blockIdx.y + 1) * heads_per_warp);
  const bool rotated = ROT && u < p.rot / 32;
  const int b0 = rotated && !p.interleaved ? u : 2 * u;              // blocks of the unit in q and k;
  const int b1 = rotated && !p.interleaved ? u + p.rot / 32 : 2 * u + 1;   // in v they are neighbours

  griddep_wait();                                   // inputs may come from the kernel before (PDL)
  Chunk x0 = {}, x1 = {};
  auto load = [&](int head) {
    if (head >= h_end) return;
    const HeadRow r = head_of(p, head);
    const void* base = r.kind == 0 ? p.q : r.kind == 1 ? p.k : p.v;
    const int64_t stride = r.kind == 0 ? p.q_stride : r.kind == 1 ? p.k_stride : p.v_stride;
    const T* src = static_cast<const T*>(base) + t * stride + static_cast<int64_t>(r.head) * p.c.D;
    const int heads = r.kind == 0 ? p.Hq : p.c.heads;
    [[maybe_unused]] const long long extent = 2LL * ((p.T - 1) * stride + static_cast<int64_t>(heads) * p.c.D);
    const int c0 = r.kind == 2 ? 2 * u : b0, c1 = r.kind == 2 ? 2 * u + 1 : b1;
    if (FP4Q_IN_RANGE(p, src + c0 * 16, 32, base, extent)) x0 = ld_stream_rw(src + c0 * 16);
    if (FP4Q_IN_RANGE(p, src + c1 * 16, 32, base, extent)) x1 = ld_stream_rw(src + c1 * 16);
  };
  load(h);
  const int64_t slot = FP4Q_IN_RANGE(p, p.slots + t, 8, p.slots, 8LL * p.T) ? p.slots[t] : -1;
  float cs[16], sn[16];
  if (ROT) {
    const int64_t pos = FP4Q_IN_RANGE(p, p.positions + t, 8, p.positions, 8LL * p.T) ? p.positions[t] : -1;
    if (pos < 0 || pos >= p.max_position) return;   // the whole token is left out
    if (rotated) {
      const float* row = p.cos_sin + pos * p.rot + u * 16;
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        if (FP4Q_IN_RANGE(p, row + i, 16, p.cos_sin, p.max_position * p.rot * 4LL))
          *reinterpret_cast<float4*>(cs + i) = __ldg(reinterpret_cast<const float4*>(row + i));
        if (FP4Q_IN_RANGE(p, row + p.rot / 2 + i, 16, p.cos_sin, p.max_position * p.rot * 4LL))
          *reinterpret_cast<float4*>(sn + i) =
              __ldg(reinterpret_cast<const float4*>(row + p.rot / 2 + i));
      }
    }
  }
  // slots times heads are numbered in 32 bits (checked by the caller)
  const bool store_kv = slot >= 0 && slot < p.c.num_pages * p.c.page_size;
  const uint32_t page = static_cast<uint32_t>(store_kv ? slot : 0) / p.c.page_size;
  const uint32_t in_page = static_cast<uint32_t>(store_kv ? slot : 0) - page * p.c.page_size;

  for (; h < h_end; h += step) {
    const HeadRow r = head_of(p, h);
    float y0[16], y1[16];
    unpack<T>(x0, y0);
    unpack<T>(x1, y1);
    load(h + step);
    if (rotated && r.kind != 2) {
      if (p.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          rotate_pair(y0[2 * i], y0[2 * i + 1], cs[i], sn[i]);
          rotate_pair(y1[2 * i], y1[2 * i + 1], cs[8 + i], sn[8 + i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) rotate_pair(y0[i], y1[i], cs[i], sn[i]);
      }
    }
    const int c0 = r.kind == 2 ? 2 * u : b0, c1 = r.kind == 2 ? 2 * u + 1 : b1;
    if (r.kind == 0) {
      T* dst = static_cast<T*>(p.out_q) + t * p.out_q_stride + static_cast<int64_t>(r.head) * p.c.D;
      [[maybe_unused]] const long long qext = 2LL * ((p.T - 1) * p.out_q_stride + static_cast<int64_t>(p.Hq) * p.c.D);
      Chunk o0, o1;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o0.u[j] = Pair<T>::from_f32(y0[2 * j], y0[2 * j + 1]);
        o1.u[j] = Pair<T>::from_f32(y1[2 * j], y1[2 * j + 1]);
      }
      if (FP4Q_IN_RANGE(p, dst + c0 * 16, 32, p.out_q, qext)) st_stream(dst + c0 * 16, o0);
      if (FP4Q_IN_RANGE(p, dst + c1 * 16, 32, p.out_q, qext)) st_stream(dst + c1 * 16, o1);
    } else if (store_kv) {
      const float gs = load_global_scale(r.kind == 1 ? p.c.k_gs : p.c.v_gs);
      uint32_t s0, s1;
      const uint64_t w0 = quantize_block(y0, gs, s0), w1 = quantize_block(y1, gs, s1);
      const uint32_t ph = page * p.c.heads + r.head;
      const uint64_t row = ph * p.c.page_size + in_page;
      uint8_t* pk_base = r.kind == 1 ? p.c.k_packed : p.c.v_packed;
      uint8_t* pk = pk_base + row * (p.c.D / 2);
      if (c1 == c0 + 1) {                           // neighbours: one store
        if (FP4Q_IN_RANGE(p, pk + c0 * 8, 16, pk_base, kv_packed_extent(p.c)))
          *reinterpret_cast<ulonglong2*>(pk + c0 * 8) = make_ulonglong2(w0, w1);
      } else {
        if (FP4Q_IN_RANGE(p, pk + c0 * 8, 8, pk_base, kv_packed_extent(p.c))) st_u64(pk + c0 * 8, w0);
        if (FP4Q_IN_RANGE(p, pk + c1 * 8, 8, pk_base, kv_packed_extent(p.c))) st_u64(pk + c1 * 8, w1);
      }
      uint8_t* sf_base = r.kind == 1 ? p.c.k_sf : p.c.v_sf;
      uint8_t* sf0 = r.kind == 1 ? sf_base + row * (p.c.D / 16) + c0
                                 : sf_base + (row - in_page) * (p.c.D / 16) + c0 * p.c.page_size + in_page;
      uint8_t* sf1 = r.kind == 1 ? sf_base + row * (p.c.D / 16) + c1
                                 : sf_base + (row - in_page) * (p.c.D / 16) + c1 * p.c.page_size + in_page;
      if (r.kind == 1 && c1 == c0 + 1) {
        if (FP4Q_IN_RANGE(p, sf0, 2, sf_base, kv_sf_extent(p.c)))
          *reinterpret_cast<uint16_t*>(sf0) = static_cast<uint16_t>(s0 | s1 << 8);
      } else {
        if (FP4Q_IN_RANGE(p, sf0, 1, sf_base, kv_sf_extent(p.c))) st_u8(sf0, s0);
        if (FP4Q_IN_RANGE(p, sf1, 1, sf_base, kv_sf_extent(p.c))) st_u8(sf1, s1);
      }
    }
  }
  griddep_launch_dependents();
}

// One warp: token t, heads of its run of the list k heads, v heads; a thread two
// neighbouring blocks (32 channels).
template <typename T>
__global__ void __launch_bounds__(128) kv_gather_kernel(const KvGatherParams p, int heads_per_warp) {
  const int units = p.c.D / 32;
  const int lane = threadIdx.x & 31;
  const int u = lane % units;
  const int step = 32 / units;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (t >= p.T) return;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t slot = FP4Q_IN_RANGE(p, p.slots + t, 8, p.slots, 8LL * p.T) ? p.slots[t] : -1;
  if (slot < 0 || slot >= p.c.num_pages * p.c.page_size) return;
  const uint32_t page = static_cast<uint32_t>(slot) / p.c.page_size;
  const uint32_t in_page = static_cast<uint32_t>(slot) - page * p.c.page_size;
  const int h_end = min(2 * p.c.heads, static_cast<int>(blockIdx.y + 1) * heads_per_warp);
#pragma unroll 2
  for (int h = blockIdx.y * heads_per_warp + lane / units; h < h_end; h += step) {
    const bool is_v = h >= p.c.heads;
    const int head = is_v ? h - p.c.heads : h;
    void* out = is_v ? p.out_v : p.out_k;
    if (!out) continue;
    const uint64_t row = (page * p.c.heads + head) * p.c.page_size + in_page;
    const uint8_t* pk_base = is_v ? p.c.v_packed : p.c.k_packed;
    const uint8_t* sf_base = is_v ? p.c.v_sf : p.c.k_sf;
    const uint8_t* pk = pk_base + row * (p.c.D / 2) + u * 16;
    const uint8_t* sf0 = is_v ? sf_base + (row - in_page) * (p.c.D / 16) + 2 * u * p.c.page_size + in_page
                              : sf_base + row * (p.c.D / 16) + 2 * u;
    const uint8_t* sf1 = sf0 + (is_v ? p.c.page_size : 1);
    uint4 w = {};
    uint32_t s[2] = {};
    if (FP4Q_IN_RANGE(p, pk, 16, pk_base, kv_packed_extent(p.c)))
      w = *reinterpret_cast<const uint4*>(pk);
    if (FP4Q_IN_RANGE(p, sf0, 1, sf_base, kv_sf_extent(p.c))) s[0] = *sf0;
    if (FP4Q_IN_RANGE(p, sf1, 1, sf_base, kv_sf_extent(p.c))) s[1] = *sf1;
    const float* gsp = is_v ? p.c.v_gs : p.c.k_gs;
    const float gs = load_global_scale(gsp);
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
    T* dst = static_cast<T*>(out) + (t * p.c.heads + head) * static_cast<int64_t>(p.c.D) + u * 32;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint32_t sc = e4m3x2_to_f16x2(s[b] | s[b] << 8);
      Chunk o;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t x[4];
        e2m1x8_to_f16x2(words[2 * b + j], x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = mul_f16x2(x[i], sc);               // exact: at most 6 significant bits
          if (gsp || !std::is_same<T, __half>::value) {
            float2 f = __half22float2(*reinterpret_cast<__half2*>(&x[i]));
            if (gsp) f = make_float2(__fdiv_rn(f.x, gs), __fdiv_rn(f.y, gs));
            x[i] = Pair<T>::from_f32(f.x, f.y);
          }
          o.u[4 * j + i] = x[i];
        }
      }
      if (FP4Q_IN_RANGE(p, dst + b * 16, 32, out, 2LL * p.T * p.c.heads * p.c.D))
        st_stream(dst + b * 16, o);
    }
  }
}

cudaLaunchConfig_t config(dim3 grid, int threads, cudaStream_t stream, cudaLaunchAttribute* attr,
                          int pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cfg;
}

// Heads of a token that one warp walks: as many as leave every SM 32 warps.
int heads_per_warp(int all, int D, int64_t T) {
  const int per = 32 / (D / 32);                    // at a time
  const int64_t want = all * T / (32 * sm_count_current_device());
  return per * static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((want + per - 1) / per, (all + per - 1) / per)));
}

}  // namespace

cudaError_t launch_kv_append(int dtype, const KvAppendParams& p, int pdl, cudaStream_t stream) {
  const int all = p.Hq + 2 * p.c.heads;
  const int run = heads_per_warp(all, p.c.D, p.T);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      config(dim3(static_cast<unsigned>((p.T + 3) / 4), static_cast<unsigned>((all + run - 1) / run)),
             128, stream, attr, pdl);
  if (p.rot)
    return dtype == 0 ? cudaLaunchKernelEx(&cfg, kv_append_kernel<__nv_bfloat16, true>, p, run)
                      : cudaLaunchKernelEx(&cfg, kv_append_kernel<__half, true>, p, run);
  return dtype == 0 ? cudaLaunchKernelEx(&cfg, kv_append_kernel<__nv_bfloat16, false>, p, run)
                    : cudaLaunchKernelEx(&cfg, kv_append_kernel<__half, false>, p, run);
}

cudaError_t launch_kv_gather(int dtype, const KvGatherParams& p, int pdl, cudaStream_t stream) {
  const int all = 2 * p.c.heads;
  const int run = heads_per_warp(all, p.c.D, p.T);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      config(dim3(static_cast<unsigned>((p.T + 3) / 4), static_cast<unsigned>((all + run - 1) / run)),
             128, stream, attr, pdl);
  return dtype == 0 ? cudaLaunchKernelEx(&cfg, kv_gather_kernel<__nv_bfloat16>, p, run)
                    : cudaLaunchKernelEx(&cfg, kv_gather_kernel<__half>, p, run);
}

}  // namespace fp4q
