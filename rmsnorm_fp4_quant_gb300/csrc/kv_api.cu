// kv_api.cu - the C entry points of the NVFP4 key/value cache (declared in
// include/fp4q.h): argument checks; the kernels are in kv_cache.cu,
// kv_attention.cu and kv_pages.cu.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/fp4q.h"
#include "fp4q_launch.h"
#include "kv_launch.h"

using namespace fp4q;

namespace {

constexpr int64_t kMaxHeads = 4096;

// Rows of `width` bytes, `stride` bytes apart (n of them, n > 0).
struct Rows {
  const void* p;
  int64_t n, stride, width;
};
Rows flat(const void* p, int64_t bytes) { return Rows{p, 1, bytes, bytes}; }

// True if two strided buffers share a byte.  Column slices of one buffer (the
// same stride) are compared column by column; other strides by their extents.
bool rows_overlap(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || a.n <= 0 || b.n <= 0 || a.width <= 0 || b.width <= 0) return false;
  if (!abi_overlap(a.p, (a.n - 1) * a.stride + a.width, b.p, (b.n - 1) * b.stride + b.width))
    return false;
  if (a.stride != b.stride || a.n == 1 || b.n == 1) return true;
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.p) -
                                         reinterpret_cast<uintptr_t>(a.p));
  const int64_t off = ((d % a.stride) + a.stride) % a.stride;   // b's column within a's rows
  return off < a.width || off + b.width > a.stride;
}

// Whether n rows, `stride` 16-bit elements apart, span bytes that 64 bits number: the
// overlaps above could not be seen otherwise.
bool spans_64_bits(int64_t n, int64_t stride) { return n <= 1 || stride <= INT64_MAX / 4 / n; }

struct CacheBuffers {
  Rows rows[4];
};
CacheBuffers buffers(const fp4_kv_cache_t& c) {
  const int64_t slots = c.num_pages * c.page_size * c.num_kv_heads;
  return CacheBuffers{{flat(c.k_packed, slots * (c.head_dim / 2)), flat(c.k_sf, slots * (c.head_dim / 16)),
                       flat(c.v_packed, slots * (c.head_dim / 2)),
                       flat(c.v_sf, slots * (c.head_dim / 16))}};
}

// Sizes, then pointers and alignment of the cache itself.
fp4_status_t check_cache_sizes(const fp4_kv_cache_t* c) {
  if (!c) return FP4_ERR_INVALID_ARG;
  if (c->num_pages < 0 || c->page_size <= 0 || c->num_kv_heads <= 0 || c->head_dim <= 0)
    return FP4_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return FP4_ERR_UNSUPPORTED_SHAPE;
  if (c->page_size % 16 || c->page_size > (1 << 20) || c->num_kv_heads > kMaxHeads ||
      c->num_pages > INT32_MAX ||
      c->num_pages * c->page_size > (int64_t{UINT32_MAX} - 1) / c->num_kv_heads)
    return FP4_ERR_UNSUPPORTED_SHAPE;   // the kernels number slots times heads in 32 bits
  return FP4_OK;
}
fp4_status_t check_cache_buffers(const fp4_kv_cache_t* c) {
  if (!c->k_packed || !c->k_sf || !c->v_packed || !c->v_sf) return FP4_ERR_INVALID_ARG;
  if (!abi_aligned(c->k_packed, 16) || !abi_aligned(c->k_sf, 16) || !abi_aligned(c->v_packed, 16) ||
      !abi_aligned(c->v_sf, 16) || !abi_aligned(c->k_global_scale, 4) ||
      !abi_aligned(c->v_global_scale, 4))
    return FP4_ERR_MISALIGNED;
  return FP4_OK;
}
KvCache device_cache(const fp4_kv_cache_t& c) {
  return KvCache{c.k_packed, c.k_sf, c.v_packed, c.v_sf, c.k_global_scale, c.v_global_scale,
                 c.num_pages, static_cast<int>(c.page_size), static_cast<int>(c.num_kv_heads),
                 static_cast<int>(c.head_dim)};
}

// Keys of a sequence and rows of a key/value head are 32-bit numbers in the kernels, and
// so are the grids over rows and sequences times heads.
bool numbered_in_32_bits(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t max_keys) {
  return Hq <= kMaxHeads && B <= INT32_MAX / 2 && T <= INT32_MAX / 2 && B * Hkv <= INT32_MAX / 2 &&
         T * Hq <= INT32_MAX && max_keys <= INT32_MAX / 2;
}
bool valid_attention_sizes(int64_t B, int64_t T, int64_t Hq, int64_t num_kv_heads, int64_t head_dim,
                           int64_t max_keys) {
  return B >= 0 && T >= 0 && max_keys >= 0 && Hq > 0 && num_kv_heads > 0 && Hq % num_kv_heads == 0 &&
         (head_dim == 64 || head_dim == 128) && numbered_in_32_bits(B, T, Hq, num_kv_heads, max_keys);
}

// Page tables, lengths and counts of fork, trim and compact: sizes that the kernels number
// in 32 bits (tokens of a sequence, slots of children, entries of the plan's grid).
bool pages_in_32_bits(const fp4_kv_cache_t& c, int64_t rows, int64_t max_pages) {
  return max_pages <= INT32_MAX / 2 / c.page_size && rows <= INT32_MAX / 4 &&
         (max_pages == 0 || rows <= INT32_MAX / 2 / max_pages);
}
// What is written overlaps nothing else that is written or read.
template <int W, int R>
bool apart(const Rows (&writes)[W], const Rows (&reads)[R]) {
  for (int i = 0; i < W; ++i) {
    for (int j = i + 1; j < W; ++j)
      if (rows_overlap(writes[i], writes[j])) return false;
    for (const Rows& r : reads)
      if (rows_overlap(writes[i], r)) return false;
  }
  return true;
}

bool valid_dtype(fp4_dtype_t d) { return d == FP4_DT_BF16 || d == FP4_DT_FP16; }

}  // namespace

extern "C" {

fp4_status_t fp4_kv_append_nvfp4(const void* q, int64_t q_stride, void* out_q,
                                 int64_t out_q_stride, const void* k, int64_t k_stride,
                                 const void* v, int64_t v_stride, const int64_t* positions,
                                 const float* cos_sin, int64_t max_position, int64_t rot_dim,
                                 int interleaved, const int64_t* slots, int64_t T, int64_t Hq,
                                 fp4_dtype_t dtype, const fp4_kv_cache_t* cache, int pdl,
                                 fp4q_stream_t stream) {
  if (!valid_dtype(dtype) || T < 0 || Hq < 0 || rot_dim < 0 || max_position < 0 ||
      interleaved < 0 || interleaved > 1)
    return FP4_ERR_INVALID_ARG;
  const fp4_status_t cs = check_cache_sizes(cache);
  if (cs != FP4_OK) return cs;
  const int64_t D = cache->head_dim, Hkv = cache->num_kv_heads;
  if (Hq > kMaxHeads || rot_dim % 32 || rot_dim > D || T > INT32_MAX) return FP4_ERR_UNSUPPORTED_SHAPE;
  if ((q == nullptr) != (out_q == nullptr) || (q == nullptr) != (Hq == 0)) return FP4_ERR_INVALID_ARG;
  if (q_stride == 0) q_stride = Hq * D;
  if (out_q_stride == 0) out_q_stride = Hq * D;
  if (k_stride == 0) k_stride = Hkv * D;
  if (v_stride == 0) v_stride = Hkv * D;
  if ((q && (q_stride < Hq * D || out_q_stride < Hq * D)) || k_stride < Hkv * D ||
      v_stride < Hkv * D)
    return FP4_ERR_INVALID_ARG;
  if (!spans_64_bits(T, k_stride) || !spans_64_bits(T, v_stride) ||
      (q && (!spans_64_bits(T, q_stride) || !spans_64_bits(T, out_q_stride))) ||
      (rot_dim && max_position > INT64_MAX / 8 / rot_dim))
    return FP4_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return FP4_OK;
  if (!k || !v || !slots || (rot_dim && (!positions || !cos_sin))) return FP4_ERR_INVALID_ARG;
  const fp4_status_t cb = check_cache_buffers(cache);
  if (cb != FP4_OK) return cb;
  if (!abi_aligned(q, 32) || !abi_aligned(out_q, 32) || !abi_aligned(k, 32) || !abi_aligned(v, 32) ||
      (q && (q_stride % 16 || out_q_stride % 16)) || k_stride % 16 || v_stride % 16 ||
      !abi_aligned(slots, 8) || (rot_dim && (!abi_aligned(positions, 8) || !abi_aligned(cos_sin, 16))))
    return FP4_ERR_MISALIGNED;
  // what is written against what is written, and against what is read
  const Rows oq{out_q, q ? T : 0, out_q_stride * 2, Hq * D * 2};
  const Rows iq{q, q ? T : 0, q_stride * 2, Hq * D * 2};
  const Rows ik{k, T, k_stride * 2, Hkv * D * 2}, iv{v, T, v_stride * 2, Hkv * D * 2};
  const CacheBuffers cbuf = buffers(*cache);
  const Rows writes[] = {oq, cbuf.rows[0], cbuf.rows[1], cbuf.rows[2], cbuf.rows[3]};
  const Rows reads[] = {iq, ik, iv, flat(slots, T * 8), flat(rot_dim ? positions : nullptr, T * 8),
                        flat(rot_dim ? cos_sin : nullptr, max_position * rot_dim * 4),
                        flat(cache->k_global_scale, 4), flat(cache->v_global_scale, 4)};
  for (int i = 0; i < 5; ++i) {
    for (int j = i + 1; j < 5; ++j)
      if (rows_overlap(writes[i], writes[j])) return FP4_ERR_INVALID_ARG;
    for (const Rows& r : reads) {
      const bool in_place = i == 0 && r.p == q && q == out_q && r.width == iq.width &&
                            r.stride == iq.stride && q_stride == out_q_stride && &r == &reads[0];
      if (!in_place && rows_overlap(writes[i], r)) return FP4_ERR_INVALID_ARG;
    }
  }
  KvAppendParams p{};
  p.q = q;
  p.out_q = out_q;
  p.k = k;
  p.v = v;
  p.q_stride = q_stride;
  p.out_q_stride = out_q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.slots = slots;
  p.max_position = max_position;
  p.T = T;
  p.Hq = static_cast<int>(Hq);
  p.rot = static_cast<int>(rot_dim);
  p.interleaved = interleaved;
  p.c = device_cache(*cache);
  FP4Q_SET_DEBUG(p);
  return static_cast<fp4_status_t>(record_cuda_error(launch_kv_append(
      dtype == FP4_DT_BF16 ? 0 : 1, p, pdl, reinterpret_cast<cudaStream_t>(stream))));
}

fp4_status_t fp4_kv_gather_nvfp4(const fp4_kv_cache_t* cache, const int64_t* slots, int64_t T,
                                 fp4_dtype_t dtype, void* out_k, void* out_v, int pdl,
                                 fp4q_stream_t stream) {
  if (!valid_dtype(dtype) || T < 0) return FP4_ERR_INVALID_ARG;
  const fp4_status_t cs = check_cache_sizes(cache);
  if (cs != FP4_OK) return cs;
  const int64_t width = cache->num_kv_heads * cache->head_dim * 2;
  if (T > INT32_MAX) return FP4_ERR_UNSUPPORTED_SHAPE;
  if (T == 0 || (!out_k && !out_v)) return FP4_OK;
  if (!slots) return FP4_ERR_INVALID_ARG;
  const fp4_status_t cb = check_cache_buffers(cache);
  if (cb != FP4_OK) return cb;
  if (!abi_aligned(slots, 8) || !abi_aligned(out_k, 32) || !abi_aligned(out_v, 32))
    return FP4_ERR_MISALIGNED;
  const CacheBuffers cbuf = buffers(*cache);
  const Rows outs[2] = {flat(out_k, T * width), flat(out_v, T * width)};
  if (rows_overlap(outs[0], outs[1])) return FP4_ERR_INVALID_ARG;
  const Rows reads[] = {cbuf.rows[0], cbuf.rows[1], cbuf.rows[2], cbuf.rows[3], flat(slots, T * 8),
                        flat(cache->k_global_scale, 4), flat(cache->v_global_scale, 4)};
  for (const Rows& o : outs)
    for (const Rows& r : reads)
      if (rows_overlap(o, r)) return FP4_ERR_INVALID_ARG;
  KvGatherParams p{};
  p.slots = slots;
  p.out_k = out_k;
  p.out_v = out_v;
  p.T = T;
  p.c = device_cache(*cache);
  FP4Q_SET_DEBUG(p);
  return static_cast<fp4_status_t>(record_cuda_error(launch_kv_gather(
      dtype == FP4_DT_BF16 ? 0 : 1, p, pdl, reinterpret_cast<cudaStream_t>(stream))));
}

int64_t fp4_attention_workspace_bytes(int64_t B, int64_t T, int64_t Hq, int64_t num_kv_heads,
                                      int64_t head_dim, int64_t max_keys) {
  if (!valid_attention_sizes(B, T, Hq, num_kv_heads, head_dim, max_keys)) return -1;
  return kv_attention_workspace(sm_count_current_device(), B, T, static_cast<int>(Hq),
                                static_cast<int>(num_kv_heads), static_cast<int>(head_dim), max_keys);
}

int64_t fp4_attention_workspace_bound(int64_t B, int64_t T, int64_t Hq, int64_t num_kv_heads,
                                      int64_t head_dim, int64_t max_keys) {
  if (!valid_attention_sizes(B, T, Hq, num_kv_heads, head_dim, max_keys)) return -1;
  return kv_attention_workspace_bound(sm_count_current_device(), B, T, static_cast<int>(Hq),
                                      static_cast<int>(num_kv_heads), static_cast<int>(head_dim), max_keys);
}

fp4_status_t fp4_attention_launch_shape(int64_t B, int64_t T, int64_t Hq, int64_t num_kv_heads,
                                        int64_t head_dim, int64_t max_keys, int64_t out[2]) {
  if (!valid_attention_sizes(B, T, Hq, num_kv_heads, head_dim, max_keys) || !B || !T || !out)
    return FP4_ERR_INVALID_ARG;
  kv_attention_shape(sm_count_current_device(), B, T, static_cast<int>(Hq),
                     static_cast<int>(num_kv_heads), static_cast<int>(head_dim), max_keys, out);
  return FP4_OK;
}

fp4_status_t fp4_attention_nvfp4_ex(const void* q, int64_t q_stride, const fp4_kv_cache_t* cache,
                                    const int32_t* block_tables, int64_t max_pages,
                                    const int32_t* seq_lens, const int32_t* cu_seqlens_q, int64_t B,
                                    int64_t T, int64_t Hq, fp4_dtype_t dtype, float sm_scale,
                                    int causal, float softcap, const float* alibi_slopes, int64_t window,
                                    const int32_t* prefix_lens, void* out, float* lse, void* workspace,
                                    int64_t workspace_bytes, int32_t* status, int pdl,
                                    fp4q_stream_t stream) {
  if (!valid_dtype(dtype) || B < 0 || T < 0 || Hq <= 0 || max_pages < 0 || workspace_bytes < 0)
    return FP4_ERR_INVALID_ARG;
  if (!(sm_scale > 0.0f) || !std::isfinite(sm_scale)) return FP4_ERR_INVALID_ARG;
  if (!(softcap >= 0.0f) || softcap > 1048576.0f || window < 0 || (!causal && (window || prefix_lens)))
    return FP4_ERR_INVALID_ARG;
  const fp4_status_t cs = check_cache_sizes(cache);
  if (cs != FP4_OK) return cs;
  const int64_t D = cache->head_dim, Hkv = cache->num_kv_heads;
  if (Hq % Hkv) return FP4_ERR_INVALID_ARG;
  if (q_stride == 0) q_stride = Hq * D;
  if (q_stride < Hq * D) return FP4_ERR_INVALID_ARG;
  if (!cu_seqlens_q && B != T) return FP4_ERR_INVALID_ARG;
  if (max_pages > INT32_MAX / 2 / cache->page_size || !spans_64_bits(T, q_stride) ||
      !numbered_in_32_bits(B, T, Hq, Hkv, max_pages * cache->page_size))
    return FP4_ERR_UNSUPPORTED_SHAPE;
  if (B == 0 || T == 0) return FP4_OK;
  if (!q || !out || !seq_lens || (max_pages && !block_tables)) return FP4_ERR_INVALID_ARG;
  const fp4_status_t cb = check_cache_buffers(cache);
  if (cb != FP4_OK) return cb;
  if (!abi_aligned(q, 32) || q_stride % 16 || !abi_aligned(out, 32) || !abi_aligned(lse, 4) ||
      !abi_aligned(block_tables, 4) || !abi_aligned(seq_lens, 4) || !abi_aligned(cu_seqlens_q, 4) ||
      !abi_aligned(workspace, 16) || !abi_aligned(status, 4) || !abi_aligned(alibi_slopes, 4) ||
      !abi_aligned(prefix_lens, 4))
    return FP4_ERR_MISALIGNED;
  if (window > INT32_MAX / 2) window = 0;             // longer than any sequence
  const int64_t keys = kv_attention_keys(B, T, max_pages * cache->page_size, window);
  const int64_t need = fp4_attention_workspace_bytes(B, T, Hq, Hkv, D, keys);
  if (workspace_bytes < need || (need && !workspace)) return FP4_ERR_INVALID_ARG;
  const CacheBuffers cbuf = buffers(*cache);
  const Rows writes[] = {flat(out, T * Hq * D * 2), flat(lse, T * Hq * 4),
                         flat(need ? workspace : nullptr, need), flat(status, 4)};
  const Rows reads[] = {Rows{q, T, q_stride * 2, Hq * D * 2},
                        cbuf.rows[0], cbuf.rows[1], cbuf.rows[2], cbuf.rows[3],
                        flat(block_tables, B * max_pages * 4), flat(seq_lens, B * 4),
                        flat(cu_seqlens_q, (B + 1) * 4), flat(alibi_slopes, Hq * 4), flat(prefix_lens, B * 4),
                        flat(cache->k_global_scale, 4), flat(cache->v_global_scale, 4)};
  for (int i = 0; i < 4; ++i) {
    for (int j = i + 1; j < 4; ++j)
      if (rows_overlap(writes[i], writes[j])) return FP4_ERR_INVALID_ARG;
    for (const Rows& r : reads)
      if (rows_overlap(writes[i], r)) return FP4_ERR_INVALID_ARG;
  }
  KvAttentionParams p{};
  p.q = q;
  p.q_stride = q_stride;
  p.c = device_cache(*cache);
  p.tables = block_tables;
  p.max_pages = max_pages;
  p.seq_lens = seq_lens;
  p.cu = cu_seqlens_q;
  p.B = static_cast<int>(B);
  p.T = T;
  p.Hq = static_cast<int>(Hq);
  p.group = static_cast<int>(Hq / Hkv);
  p.sm_scale = sm_scale;
  p.causal = causal ? 1 : 0;
  p.softcap = softcap;
  p.slopes = alibi_slopes;
  p.window = static_cast<int>(window);
  p.prefix = prefix_lens;
  p.out = out;
  p.lse = lse;
  p.ws = static_cast<float*>(workspace);
  p.ws_bytes = need;
  p.status = status;
  FP4Q_SET_DEBUG(p);
  const bool plain = softcap == 0.0f && !alibi_slopes && !window && !prefix_lens;
  return static_cast<fp4_status_t>(record_cuda_error((plain ? launch_kv_attention : launch_kv_attention_masked)(
      dtype == FP4_DT_BF16 ? 0 : 1, p, pdl, reinterpret_cast<cudaStream_t>(stream))));
}

fp4_status_t fp4_attention_nvfp4(const void* q, int64_t q_stride, const fp4_kv_cache_t* cache,
                                 const int32_t* block_tables, int64_t max_pages,
                                 const int32_t* seq_lens, const int32_t* cu_seqlens_q, int64_t B,
                                 int64_t T, int64_t Hq, fp4_dtype_t dtype, float sm_scale,
                                 int causal, void* out, float* lse, void* workspace,
                                 int64_t workspace_bytes, int32_t* status, int pdl,
                                 fp4q_stream_t stream) {
  return fp4_attention_nvfp4_ex(q, q_stride, cache, block_tables, max_pages, seq_lens, cu_seqlens_q, B, T, Hq,
                                dtype, sm_scale, causal, 0.0f, nullptr, 0, nullptr, out, lse, workspace,
                                workspace_bytes, status, pdl, stream);
}

const char* fp4_kv_status_string(fp4_status_t s) { return fp4_status_string(s); }

fp4_status_t fp4_kv_read_status(const int32_t* status, fp4q_stream_t stream) {
  return fp4_read_device_status(status, stream);
}

int64_t fp4_kv_pages_workspace_bytes(int64_t num_pages, int64_t N) {
  if (num_pages < 0 || num_pages > INT32_MAX || N < 0 || N > INT32_MAX / 4) return -1;
  return 4 * kv_pages_workspace(num_pages, N);
}

fp4_status_t fp4_kv_fork_nvfp4(const fp4_kv_cache_t* cache, const int32_t* refs, const int32_t* tables,
                               int64_t max_pages, const int32_t* seq_lens, int64_t B, const int32_t* parents,
                               const int32_t* new_lens, int64_t N, int64_t new_tokens, int32_t* out_tables,
                               int32_t* out_seq_lens, int32_t* out_refs, int64_t* out_slots, void* workspace,
                               int64_t workspace_bytes, int32_t* status, int pdl, fp4q_stream_t stream) {
  if (B < 0 || N < 0 || max_pages < 0 || new_tokens < 0 || workspace_bytes < 0) return FP4_ERR_INVALID_ARG;
  const fp4_status_t cs = check_cache_sizes(cache);
  if (cs != FP4_OK) return cs;
  if (!parents && N && N != B) return FP4_ERR_INVALID_ARG;
  if (!pages_in_32_bits(*cache, B, max_pages) || !pages_in_32_bits(*cache, N, max_pages) ||
      new_tokens > INT32_MAX / 4 || (new_tokens && N > INT32_MAX / new_tokens))
    return FP4_ERR_UNSUPPORTED_SHAPE;
  const int64_t pages = cache->num_pages, need = fp4_kv_pages_workspace_bytes(pages, N);
  if (pages == 0 && B == 0 && N == 0) return FP4_OK;
  if ((pages && (!refs || !out_refs)) || (B && !seq_lens) || (B && max_pages && !tables) ||
      (N && (!out_seq_lens || (max_pages && !out_tables) || (new_tokens && !out_slots))) || !workspace ||
      workspace_bytes < need)
    return FP4_ERR_INVALID_ARG;
  const fp4_status_t cb = check_cache_buffers(cache);
  if (cb != FP4_OK) return cb;
  if (!abi_aligned(refs, 4) || !abi_aligned(tables, 4) || !abi_aligned(seq_lens, 4) || !abi_aligned(parents, 4) ||
      !abi_aligned(new_lens, 4) || !abi_aligned(out_tables, 4) || !abi_aligned(out_seq_lens, 4) ||
      !abi_aligned(out_refs, 4) || !abi_aligned(out_slots, 8) || !abi_aligned(workspace, 16) || !abi_aligned(status, 4))
    return FP4_ERR_MISALIGNED;
  const CacheBuffers cbuf = buffers(*cache);
  const Rows writes[] = {flat(out_tables, N * max_pages * 4), flat(out_seq_lens, N * 4), flat(out_refs, pages * 4),
                         flat(out_slots, N * new_tokens * 8), flat(workspace, need), flat(status, 4),
                         cbuf.rows[0], cbuf.rows[1], cbuf.rows[2], cbuf.rows[3]};
  const Rows reads[] = {flat(refs, pages * 4), flat(tables, B * max_pages * 4), flat(seq_lens, B * 4),
                        flat(parents, N * 4), flat(new_lens, N * 4)};
  if (!apart(writes, reads)) return FP4_ERR_INVALID_ARG;
  KvPagesParams p{};
  p.c = device_cache(*cache);
  p.refs = refs;
  p.tables = tables;
  p.max_pages = max_pages;
  p.seq_lens = seq_lens;
  p.B = static_cast<int>(B);
  p.out_tables = out_tables;
  p.out_lens = out_seq_lens;
  p.out_refs = out_refs;
  p.parents = parents;
  p.new_lens = new_lens;
  p.N = static_cast<int>(N);
  p.new_tokens = static_cast<int>(new_tokens);
  p.out_slots = out_slots;
  p.status = status;
  p.ws = static_cast<int*>(workspace);
  p.ws_ints = need / 4;
  FP4Q_SET_DEBUG(p);
  return static_cast<fp4_status_t>(
      record_cuda_error(launch_kv_fork(p, pdl, reinterpret_cast<cudaStream_t>(stream))));
}

fp4_status_t fp4_kv_trim_nvfp4(const fp4_kv_cache_t* cache, const int32_t* refs, const int32_t* tables,
                               int64_t max_pages, const int32_t* seq_lens, int64_t B, const int32_t* first,
                               const int32_t* end, int32_t* out_tables, int32_t* out_seq_lens, int32_t* out_refs,
                               int pdl, fp4q_stream_t stream) {
  if (B < 0 || max_pages < 0) return FP4_ERR_INVALID_ARG;
  const fp4_status_t cs = check_cache_sizes(cache);
  if (cs != FP4_OK) return cs;
  if (!pages_in_32_bits(*cache, B, max_pages)) return FP4_ERR_UNSUPPORTED_SHAPE;
  const int64_t pages = cache->num_pages;
  if (pages == 0 && B == 0) return FP4_OK;
  if ((pages && (!refs || !out_refs)) || (B && (!seq_lens || !out_seq_lens || (max_pages && (!tables || !out_tables)))))
    return FP4_ERR_INVALID_ARG;
  if (!abi_aligned(refs, 4) || !abi_aligned(tables, 4) || !abi_aligned(seq_lens, 4) || !abi_aligned(first, 4) ||
      !abi_aligned(end, 4) || !abi_aligned(out_tables, 4) || !abi_aligned(out_seq_lens, 4) || !abi_aligned(out_refs, 4))
    return FP4_ERR_MISALIGNED;
  const Rows writes[] = {flat(out_tables, B * max_pages * 4), flat(out_seq_lens, B * 4), flat(out_refs, pages * 4)};
  const Rows reads[] = {flat(refs, pages * 4), flat(tables, B * max_pages * 4), flat(seq_lens, B * 4),
                        flat(first, B * 4), flat(end, B * 4)};
  if (!apart(writes, reads)) return FP4_ERR_INVALID_ARG;
  KvPagesParams p{};
  p.c = device_cache(*cache);
  p.refs = refs;
  p.tables = tables;
  p.max_pages = max_pages;
  p.seq_lens = seq_lens;
  p.B = static_cast<int>(B);
  p.out_tables = out_tables;
  p.out_lens = out_seq_lens;
  p.out_refs = out_refs;
  p.first = first;
  p.end = end;
  FP4Q_SET_DEBUG(p);
  return static_cast<fp4_status_t>(
      record_cuda_error(launch_kv_trim(p, pdl, reinterpret_cast<cudaStream_t>(stream))));
}

fp4_status_t fp4_kv_compact_nvfp4(const fp4_kv_cache_t* cache, const int32_t* refs, const int32_t* tables,
                                  int64_t max_pages, const int32_t* seq_lens, int64_t B, int32_t* out_tables,
                                  int32_t* out_refs, int32_t* out_map, int32_t* out_live, void* workspace,
                                  int64_t workspace_bytes, int pdl, fp4q_stream_t stream) {
  if (B < 0 || max_pages < 0 || workspace_bytes < 0) return FP4_ERR_INVALID_ARG;
  const fp4_status_t cs = check_cache_sizes(cache);
  if (cs != FP4_OK) return cs;
  if (!pages_in_32_bits(*cache, B, max_pages)) return FP4_ERR_UNSUPPORTED_SHAPE;
  const int64_t pages = cache->num_pages, need = fp4_kv_pages_workspace_bytes(pages, 0);
  if ((pages && (!refs || !out_refs || !out_map)) || !out_live ||
      (B && (!seq_lens || (max_pages && (!tables || !out_tables)))) || !workspace || workspace_bytes < need)
    return FP4_ERR_INVALID_ARG;
  const fp4_status_t cb = check_cache_buffers(cache);
  if (cb != FP4_OK) return cb;
  if (!abi_aligned(refs, 4) || !abi_aligned(tables, 4) || !abi_aligned(seq_lens, 4) || !abi_aligned(out_tables, 4) ||
      !abi_aligned(out_refs, 4) || !abi_aligned(out_map, 4) || !abi_aligned(out_live, 4) || !abi_aligned(workspace, 16))
    return FP4_ERR_MISALIGNED;
  const CacheBuffers cbuf = buffers(*cache);
  const Rows writes[] = {flat(out_tables, B * max_pages * 4), flat(out_refs, pages * 4), flat(out_map, pages * 4),
                         flat(out_live, 4), flat(workspace, need), cbuf.rows[0], cbuf.rows[1], cbuf.rows[2], cbuf.rows[3]};
  const Rows reads[] = {flat(refs, pages * 4), flat(tables, B * max_pages * 4), flat(seq_lens, B * 4)};
  if (!apart(writes, reads)) return FP4_ERR_INVALID_ARG;
  KvPagesParams p{};
  p.c = device_cache(*cache);
  p.refs = refs;
  p.tables = tables;
  p.max_pages = max_pages;
  p.seq_lens = seq_lens;
  p.B = static_cast<int>(B);
  p.out_tables = out_tables;
  p.out_refs = out_refs;
  p.out_map = out_map;
  p.out_live = out_live;
  p.ws = static_cast<int*>(workspace);
  p.ws_ints = need / 4;
  FP4Q_SET_DEBUG(p);
  return static_cast<fp4_status_t>(
      record_cuda_error(launch_kv_compact(p, pdl, reinterpret_cast<cudaStream_t>(stream))));
}

}  // extern "C"
