// kv_pages.cu - the pages of the NVFP4 key/value cache between two tokens: sequences
// continued by their children (fork), tokens given up (trim), live pages moved together
// (compact).
//
// Each is a plan over tables and reference counts, small next to the cache, and (fork and
// compact) a copy of pages that follows it.  The plan is one cluster of up to 8 CTAs: its phases
// pass results through L2 and are kept apart by the cluster's barrier, which costs less
// than a launch each.  Counts change by atomic additions of whole numbers, which give the
// same results in any order; what has to be chosen (which child keeps a page, which free
// page a child takes) goes by the lowest number.
//
// Nothing is written that the call reads, but pages that no sequence holds: a call that is
// repeated on the same tables does the same again.
#include <algorithm>

#include "async_copy.cuh"
#include "fp4q_launch.h"
#include "kv_launch.h"

namespace fp4q {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanMostCtas = 8;
constexpr int kPlanMostWarps = kPlanWarps * kPlanMostCtas;
constexpr int kNoChild = INT32_MAX;
constexpr int kStatusNoPages = 6;             // FP4_ERR_NO_PAGES of the C ABI

// --- workspace, in ints ---------------------------------------------------------
// Per warp of the plan a count of free (or live) pages and one of pages wanted, then a
// header; per page two lists; per child its state and its copy.
enum : int { kWsFree = 0, kWsWanted = kPlanMostWarps, kWsHeader = 2 * kPlanMostWarps, kWsPages = kWsHeader + 32 };
enum : int { kHeadMoves = 0 };
// Per child four ints: its parent (-1: none), tokens before and after, pages to take, with kCopies
// on top if the first of these is a copy of its last page; and four of that copy: from, to (< 0:
// none), groups of 16 tokens.
constexpr int kCopies = 1 << 30;
__host__ __device__ inline int64_t ws_children(int64_t pages) { return kWsPages + (2 * pages + 3) / 4 * 4; }
__host__ __device__ inline int64_t ws_copies(int64_t pages, int64_t N) { return ws_children(pages) + 4 * N; }

// --- checked accesses (the debug build's checks; plain ones else) --------------------
__device__ __forceinline__ int page_ref(const KvPagesParams& p, int64_t i) {
  return FP4Q_IN_RANGE(p, p.refs + i, 4, p.refs, 4LL * p.c.num_pages) ? __ldg(p.refs + i) : 0;
}
__device__ __forceinline__ void set_out_ref(const KvPagesParams& p, int64_t i, int v) {
  if (FP4Q_IN_RANGE(p, p.out_refs + i, 4, p.out_refs, 4LL * p.c.num_pages)) __stcg(p.out_refs + i, v);
}
__device__ __forceinline__ int out_ref(const KvPagesParams& p, int64_t i) {
  return FP4Q_IN_RANGE(p, p.out_refs + i, 4, p.out_refs, 4LL * p.c.num_pages) ? __ldcg(p.out_refs + i) : 0;
}
__device__ __forceinline__ void add_out_ref(const KvPagesParams& p, int page, int v) {
  if (FP4Q_IN_RANGE(p, p.out_refs + page, 4, p.out_refs, 4LL * p.c.num_pages)) atomicAdd(p.out_refs + page, v);
}
__device__ __forceinline__ int old_entry(const KvPagesParams& p, int b, int64_t i) {
  const int32_t* e = p.tables + b * p.max_pages + i;
  return FP4Q_IN_RANGE(p, e, 4, p.tables, 4LL * p.B * p.max_pages) ? __ldg(e) : -1;
}
__device__ __forceinline__ void set_entry(const KvPagesParams& p, int64_t rows, int64_t at, int v) {
  if (FP4Q_IN_RANGE(p, p.out_tables + at, 4, p.out_tables, 4LL * rows * p.max_pages)) __stcg(p.out_tables + at, v);
}
__device__ __forceinline__ int ws_load(const KvPagesParams& p, int64_t i) {
  return FP4Q_IN_RANGE(p, p.ws + i, 4, p.ws, 4LL * p.ws_ints) ? __ldcg(p.ws + i) : 0;
}
__device__ __forceinline__ void ws_store(const KvPagesParams& p, int64_t i, int v) {
  if (FP4Q_IN_RANGE(p, p.ws + i, 4, p.ws, 4LL * p.ws_ints)) __stcg(p.ws + i, v);
}
__device__ __forceinline__ int4 ws_load4(const KvPagesParams& p, int64_t i) {
  return FP4Q_IN_RANGE(p, p.ws + i, 16, p.ws, 4LL * p.ws_ints) ? __ldcg(reinterpret_cast<const int4*>(p.ws + i))
                                                              : make_int4(-1, 0, 0, 0);
}
__device__ __forceinline__ void ws_store4(const KvPagesParams& p, int64_t i, int4 v) {
  if (FP4Q_IN_RANGE(p, p.ws + i, 16, p.ws, 4LL * p.ws_ints)) __stcg(reinterpret_cast<int4*>(p.ws + i), v);
}
// Cached tokens of sequence b, held to what its table has room for.
__device__ __forceinline__ int tokens_of(const KvPagesParams& p, int b) {
  const int n = FP4Q_IN_RANGE(p, p.seq_lens + b, 4, p.seq_lens, 4LL * p.B) ? __ldg(p.seq_lens + b) : 0;
  return min(max(n, 0), static_cast<int>(p.max_pages) * p.c.page_size);
}
__device__ __forceinline__ int pages_of(const KvPagesParams& p, int tokens) {
  return (tokens + p.c.page_size - 1) / p.c.page_size;
}
__device__ __forceinline__ bool is_page(const KvPagesParams& p, int page) { return page >= 0 && page < p.c.num_pages; }

// Every thread's writes before it are seen by the cluster's threads behind it.
__device__ __forceinline__ void plan_sync() {
  cluster_arrive_release();
  cluster_wait_acquire();
}

// The plan's place: thread and warp of the cluster, and the run of pages (a multiple of 32)
// that the warp counts.
struct PlanPlace {
  int thread, threads, warp, warps, lane;
  int64_t page0, page1;
};
__device__ __forceinline__ PlanPlace plan_place(int64_t pages) {
  PlanPlace w;
  w.thread = blockIdx.x * kPlanThreads + threadIdx.x;      // the grid is the cluster
  w.threads = gridDim.x * kPlanThreads;
  w.warp = w.thread >> 5;
  w.warps = w.threads >> 5;
  w.lane = threadIdx.x & 31;
  const int64_t run = ((pages + w.warps - 1) / w.warps + 31) / 32 * 32;
  w.page0 = min(pages, w.warp * run);
  w.page1 = min(pages, w.page0 + run);
  return w;
}
// Sum of the counts that the warps before this one left in the workspace, and of all.
__device__ __forceinline__ int counts_before(const KvPagesParams& p, const PlanPlace& w, int at, int& all) {
  int before = 0;
  all = 0;
  for (int i = w.lane; i < w.warps; i += 32) {
    const int x = ws_load(p, at + i);
    all += x;
    if (i < w.warp) before += x;
  }
  all = __reduce_add_sync(kAll, all);
  return __reduce_add_sync(kAll, before);
}

// --- fork -----------------------------------------------------------------------
__device__ __forceinline__ void copy16(const KvPagesParams& p, uint8_t* base, int64_t src, int64_t dst, long long extent) {
  if (FP4Q_IN_RANGE(p, base + src, 16, base, extent) && FP4Q_IN_RANGE(p, base + dst, 16, base, extent))
    *reinterpret_cast<uint4*>(base + dst) = *reinterpret_cast<const uint4*>(base + src);
}
// The tokens of a last page that a child has copied, one head: by threads tid, tid + threads ...
__device__ __forceinline__ void fork_copy(const KvPagesParams& p, const int4& m, int head, int tid, int threads) {
  const int src = m.x, dst = m.y, groups = m.z;
  if (dst < 0) return;
  const int D = p.c.D, page = p.c.page_size;
  const long long codes = kv_packed_extent(p.c), scales = kv_sf_extent(p.c);
  const int64_t a = static_cast<int64_t>(src) * p.c.heads + head, b = static_cast<int64_t>(dst) * p.c.heads + head;
  const int64_t page_codes = static_cast<int64_t>(page) * (D / 2), page_sf = static_cast<int64_t>(page) * (D / 16);
  for (int x = tid; x < groups * (D / 2); x += threads) {            // 16 bytes of 16 tokens' D / 2 each
    copy16(p, p.c.k_packed, a * page_codes + 16 * x, b * page_codes + 16 * x, codes);
    copy16(p, p.c.v_packed, a * page_codes + 16 * x, b * page_codes + 16 * x, codes);
  }
  for (int x = tid; x < groups * (D / 16); x += threads) {
    copy16(p, p.c.k_sf, a * page_sf + 16 * x, b * page_sf + 16 * x, scales);
    const int block = x / groups, g = x - block * groups;            // the values' scales: tokens side by side
    const int64_t o = static_cast<int64_t>(block) * page + 16 * g;
    copy16(p, p.c.v_sf, a * page_sf + o, b * page_sf + o, scales);
  }
}
// The slots of a child's new tokens.
__device__ __forceinline__ void fork_slots(const KvPagesParams& p, int i, int had, int grown, int tid, int threads) {
  for (int x = tid; x < p.new_tokens; x += threads) {
    const int64_t pos = static_cast<int64_t>(had) + x;
    int64_t slot = -1;
    if (pos < grown) {
      const int32_t* e = p.out_tables + i * p.max_pages + pos / p.c.page_size;
      const int page = FP4Q_IN_RANGE(p, e, 4, p.out_tables, 4LL * p.N * p.max_pages) ? __ldcg(e) : -1;
      if (is_page(p, page)) slot = static_cast<int64_t>(page) * p.c.page_size + pos % p.c.page_size;
    }
    int64_t* out = p.out_slots + static_cast<int64_t>(i) * p.new_tokens + x;
    if (FP4Q_IN_RANGE(p, out, 8, p.out_slots, 8LL * p.N * p.new_tokens)) *out = slot;
  }
}

// Phases: (1) counts copied, children's lengths; (2) the old sequences' references dropped,
// the children's to pages that they share added, the first child of every last page that is to be
// written noted; (3) such a page stays with its first child if nobody else holds it; pages
// wanted and free counted; (4) free pages listed, lowest first; (5) taken, child by child.
// What a phase reads comes from L2, a microsecond's part at a time, so a thread asks for several
// table entries at once, children are kept in every CTA's shared memory and what a warp has found
// out stays in its registers (512 children of 65 pages each: the plan takes 16.5 us, 21
// with an entry a thread at a time and all counts by atomics).
constexpr int kPlanChildren = 2048;             // children in shared memory; further ones in the workspace
constexpr int kPlanMasks = 8;                   // times 32 pages of a warp whose free ones it remembers
// COPY: the plan's CTAs make the copies and slots themselves.
template <bool COPY>
__global__ void __launch_bounds__(kPlanThreads) kv_fork_plan_kernel(const KvPagesParams p) {
  __shared__ int4 near_children[kPlanChildren];
  __shared__ int kids[kPlanChildren];            // of an old sequence: children, and 2^16 times those that grow
  const bool counted = p.N <= kPlanChildren && p.B <= kPlanChildren;
  const PlanPlace w = plan_place(p.c.num_pages);
  const int64_t heirs = kWsPages, free_list = kWsPages + p.c.num_pages;
  const int64_t children = ws_children(p.c.num_pages), copies = ws_copies(p.c.num_pages, p.N);
  const int most = static_cast<int>(p.max_pages);
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t i = w.thread; i < p.c.num_pages; i += w.threads) {
    set_out_ref(p, i, page_ref(p, i));
    ws_store(p, heirs + i, kNoChild);
  }
  const int room = most * p.c.page_size;
  bool short_of = false;
  auto look_up = [&](int i) {
    int parent = i;
    if (p.parents) parent = FP4Q_IN_RANGE(p, p.parents + i, 4, p.parents, 4LL * p.N) ? __ldg(p.parents + i) : -1;
    int4 c = make_int4(-1, 0, 0, 0);                         // parent, tokens before and after, (pages wanted)
    if (parent >= 0 && parent < p.B) {
      c.x = parent;
      c.y = tokens_of(p, parent);
      int more = p.new_tokens;
      if (p.new_lens)
        more = FP4Q_IN_RANGE(p, p.new_lens + i, 4, p.new_lens, 4LL * p.N) ? min(max(__ldg(p.new_lens + i), 0), more) : 0;
      c.z = static_cast<int>(min(static_cast<int64_t>(c.y) + more, static_cast<int64_t>(room)));
      short_of |= c.z < static_cast<int64_t>(c.y) + more;
    }
    return c;
  };
  if (counted) {
    for (int b = threadIdx.x; b < p.B; b += kPlanThreads) kids[b] = 0;
    __syncthreads();
  }
  for (int i = threadIdx.x; i < min(p.N, kPlanChildren); i += kPlanThreads) {
    const int4 c = look_up(i);
    near_children[i] = c;
    if (counted && c.x >= 0) atomicAdd(&kids[c.x], c.z > c.y ? 65537 : 1);
  }
  for (int i = kPlanChildren + w.thread; i < p.N; i += w.threads) ws_store4(p, children + 4LL * i, look_up(i));
  plan_sync();

  auto child = [&](int i) { return i < kPlanChildren ? near_children[i] : ws_load4(p, children + 4LL * i); };
  // a warp takes 128 entries of a row: what the row decides is looked up once for them
  const int pages = static_cast<int>(p.c.num_pages);
  const int segs = (most + 127) / 128;
  for (int u = w.warp; u < p.B * segs; u += w.warps) {
    const int b = u / segs, from = (u - b * segs) * 128 + w.lane;
    const int len = tokens_of(p, b), used = pages_of(p, len);
    // what the sequence gives up, and, where they were counted, what its children take on; a last
    // page that is not full is taken on by those that do not write it
    const int all = counted ? (kids[b] & 0xffff) - 1 : -1, last = counted ? all - (kids[b] >> 16) : -1;
    int page[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) page[k] = from + 32 * k < used ? old_entry(p, b, from + 32 * k) : -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int by = from + 32 * k == used - 1 && len % p.c.page_size ? last : all;
      if (by && page[k] >= 0 && page[k] < pages) add_out_ref(p, page[k], by);
    }
  }
  for (int u = w.warp; u < p.N * segs; u += w.warps) {
    const int i = u / segs, from = (u - i * segs) * 128 + w.lane;
    const int4 c = child(i);
    const int used = pages_of(p, c.y);
    // a page that is to be written goes to one child
    const int written = c.z > c.y && c.y % p.c.page_size ? used - 1 : -1;
    int page[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) page[k] = from + 32 * k < used ? old_entry(p, c.x, from + 32 * k) : -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int idx = from + 32 * k;
      if (idx >= most) continue;
      set_entry(p, p.N, static_cast<int64_t>(i) * most + idx, page[k]);
      if (page[k] < 0 || page[k] >= pages) continue;
      if (idx != written) {
        if (!counted) add_out_ref(p, page[k], 1);
      } else if (FP4Q_IN_RANGE(p, p.ws + heirs + page[k], 4, p.ws, 4LL * p.ws_ints)) {
        atomicMin(p.ws + heirs + page[k], i);
      }
    }
  }
  plan_sync();

  // free: held by nobody, and not about to stay with its first child
  auto is_free = [&](int64_t page) { return out_ref(p, page) <= 0 && ws_load(p, heirs + page) == kNoChild; };
  uint32_t masks[kPlanMasks];                              // free pages of the warp's first ones
  int free = 0;
  {
    bool here[kPlanMasks];
#pragma unroll
    for (int k = 0; k < kPlanMasks; ++k) here[k] = w.page0 + 32 * k + w.lane < w.page1 && is_free(w.page0 + 32 * k + w.lane);
#pragma unroll
    for (int k = 0; k < kPlanMasks; ++k) {
      masks[k] = __ballot_sync(kAll, here[k]);
      free += __popc(masks[k]);
    }
  }
  for (int64_t i = w.page0 + 32 * kPlanMasks; i < w.page1; i += 32)
    free += __popc(__ballot_sync(kAll, i + w.lane < w.page1 && is_free(i + w.lane)));
  const int run = (p.N + w.warps - 1) / w.warps;           // children of a warp
  const int child0 = static_cast<int>(min(static_cast<int64_t>(p.N), static_cast<int64_t>(w.warp) * run));
  const int child1 = min(p.N, child0 + run);
  int wanted = 0;
  int4 first_child = make_int4(-1, 0, 0, 0);               // the lane's, with what it wants
  for (int i = child0 + w.lane; i < child1; i += 32) {
    int4 c = child(i);
    const int used = pages_of(p, c.y);
    int wants = pages_of(p, c.z) - used;
    const bool part = c.y % p.c.page_size != 0 && c.z > c.y;
    const int last = part ? old_entry(p, c.x, used - 1) : -1;
    if (is_page(p, last)) {
      const int heir = ws_load(p, heirs + last), held = out_ref(p, last);
      if (heir != i || held > 0)
        wants = (wants + 1) | kCopies;
      else
        set_out_ref(p, last, 1);                           // no other child reads or writes it
    }
    c.w = wants;
    ws_store4(p, children + 4LL * i, c);
    if (FP4Q_IN_RANGE(p, p.out_lens + i, 4, p.out_lens, 4LL * p.N)) p.out_lens[i] = c.z;
    if (i - child0 < 32) first_child = c;
    wanted += wants & ~kCopies;
  }
  wanted = __reduce_add_sync(kAll, wanted);
  if (w.lane == 0) {
    ws_store(p, kWsFree + w.warp, free);
    ws_store(p, kWsWanted + w.warp, wanted);
  }
  plan_sync();

  int all_free, all_wanted;
  int rank = counts_before(p, w, kWsFree, all_free);
  const int first_wanted = counts_before(p, w, kWsWanted, all_wanted);
  auto list = [&](int64_t page, uint32_t who) {            // 32 pages from `page` on
    const int r = rank + __popc(who & ((1u << w.lane) - 1));
    if (who >> w.lane & 1u) {
      if (r < all_wanted) ws_store(p, free_list + r, static_cast<int>(page) + w.lane);
      set_out_ref(p, page + w.lane, 0);
    }
    rank += __popc(who);
  };
#pragma unroll
  for (int k = 0; k < kPlanMasks; ++k)
    if (masks[k]) list(w.page0 + 32 * k, masks[k]);
  for (int64_t i = w.page0 + 32 * kPlanMasks; i < w.page1; i += 32)
    list(i, __ballot_sync(kAll, i + w.lane < w.page1 && is_free(i + w.lane)));
  short_of |= all_wanted > all_free;
  plan_sync();

  int at = first_wanted;
  for (int i0 = child0; i0 < child1; i0 += 32) {
    // 32 children: where each one's pages begin in the list
    const int4 none = make_int4(-1, 0, 0, 0);
    const int4 mine = i0 == child0 ? first_child : i0 + w.lane < child1 ? ws_load4(p, children + 4LL * (i0 + w.lane)) : none;
    int incl = mine.w & ~kCopies;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(kAll, incl, o);
      if (w.lane >= o) incl += up;
    }
    for (int j = 0; j < min(32, child1 - i0); ++j) {
      const int parent = __shfl_sync(kAll, mine.x, j), had = __shfl_sync(kAll, mine.y, j);
      const int wants = __shfl_sync(kAll, mine.w, j), n = wants & ~kCopies;
      const int from = at + __shfl_sync(kAll, incl, j) - n;
      const int first = pages_of(p, had) - (wants & kCopies ? 1 : 0);
      int4 copy = make_int4(-1, -1, 0, 0);
      for (int x = w.lane; x < n; x += 32) {
        const int page = from + x < all_free ? ws_load(p, free_list + from + x) : -1;
        if (x == 0 && (wants & kCopies)) copy = make_int4(old_entry(p, parent, first), page, (had % p.c.page_size + 15) / 16, 0);
        set_entry(p, p.N, static_cast<int64_t>(i0 + j) * most + first + x, page);
        if (page >= 0) set_out_ref(p, page, 1);
      }
      if (w.lane == 0) ws_store4(p, copies + 4LL * (i0 + j), copy);
    }
    at += __shfl_sync(kAll, incl, 31);
  }
  if (p.status && __any_sync(kAll, short_of) && w.lane == 0) atomicExch(p.status, kStatusNoPages);
  if constexpr (COPY) {
    plan_sync();
    for (int x = w.warp; x < p.N * p.c.heads; x += w.warps) {
      const int i = x / p.c.heads, head = x - i * p.c.heads;
      const int4 m = ws_load4(p, copies + 4LL * i);
      if (head == 0) {
        const int4 c = ws_load4(p, children + 4LL * i);
        fork_slots(p, i, c.y, c.z, w.lane, 32);
      }
      fork_copy(p, m, head, w.lane, 32);
    }
  }
}

// The rest of a larger fork: pages, a head per CTA, and slots.
constexpr int kForkThreads = 128;
__global__ void __launch_bounds__(kForkThreads) kv_fork_copy_kernel(const KvPagesParams p) {
  const int i = blockIdx.x, head = blockIdx.y, tid = threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  const int4 m = ws_load4(p, ws_copies(p.c.num_pages, p.N) + 4LL * i);
  if (head == 0 && p.new_tokens > 0) {
    const int4 c = ws_load4(p, ws_children(p.c.num_pages) + 4LL * i);
    fork_slots(p, i, c.y, c.z, tid, kForkThreads);
  }
  fork_copy(p, m, head, tid, kForkThreads);
}

// --- trim -----------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads) kv_trim_kernel(const KvPagesParams p) {
  const PlanPlace w = plan_place(p.c.num_pages);
  griddep_wait();
  griddep_launch_dependents();
  for (int64_t i = w.thread; i < p.c.num_pages; i += w.threads) set_out_ref(p, i, page_ref(p, i));
  plan_sync();
  auto range = [&](int b, int& first, int& end) {
    const int n = tokens_of(p, b);
    first = 0;
    end = n;
    if (p.first && FP4Q_IN_RANGE(p, p.first + b, 4, p.first, 4LL * p.B)) first = max(__ldg(p.first + b), 0);
    if (p.end && FP4Q_IN_RANGE(p, p.end + b, 4, p.end, 4LL * p.B)) end = min(max(__ldg(p.end + b), 0), n);
    return n;
  };
  for (int b = w.thread; b < p.B; b += w.threads) {
    int first, end;
    range(b, first, end);
    if (FP4Q_IN_RANGE(p, p.out_lens + b, 4, p.out_lens, 4LL * p.B)) p.out_lens[b] = end;
  }
  const int most = static_cast<int>(p.max_pages), segs = (most + 127) / 128;
  for (int u = w.warp; u < p.B * segs; u += w.warps) {     // a warp takes 128 entries of a row
    const int b = u / segs, from = (u - b * segs) * 128 + w.lane;
    int first, end;
    const int used = pages_of(p, range(b, first, end));
    const int keep0 = first / p.c.page_size, keep1 = pages_of(p, end);
    int page[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) page[k] = from + 32 * k < used ? old_entry(p, b, from + 32 * k) : -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int idx = from + 32 * k;
      if (idx >= most) continue;
      if (!is_page(p, page[k])) page[k] = -1;
      if (page[k] >= 0 && (idx < keep0 || idx >= keep1)) {
        add_out_ref(p, page[k], -1);
        page[k] = -1;
      }
      set_entry(p, p.B, static_cast<int64_t>(b) * most + idx, page[k]);
    }
  }
}

// --- compact --------------------------------------------------------------------
// With n live pages, the live ones from n on go to the holes before n, both in
// ascending order.  Phases: (1) live pages counted; (2) holes listed by the holes before
// them, pages to move by the live ones behind them; (3) pairs, map, counts; (4) tables.
__global__ void __launch_bounds__(kPlanThreads) kv_compact_plan_kernel(const KvPagesParams p) {
  const PlanPlace w = plan_place(p.c.num_pages);
  const int64_t holes = kWsPages, movers = kWsPages + p.c.num_pages;
  griddep_wait();
  griddep_launch_dependents();
  int live = 0;
  for (int64_t i = w.page0; i < w.page1; i += 32)
    live += __popc(__ballot_sync(kAll, i + w.lane < w.page1 && page_ref(p, i + w.lane) > 0));
  if (w.lane == 0) ws_store(p, kWsFree + w.warp, live);
  plan_sync();

  int n;
  int rank = counts_before(p, w, kWsFree, n);              // live pages before the warp's
  int n_holes = 0;
  for (int64_t i0 = w.page0; i0 < w.page1; i0 += 32) {
    const int64_t i = i0 + w.lane;
    const int refs = i < w.page1 ? page_ref(p, i) : 0;
    const bool here = refs > 0;
    const uint32_t who = __ballot_sync(kAll, here);
    const int before = rank + __popc(who & ((1u << w.lane) - 1));
    const bool hole = i < w.page1 && !here && i < n;
    if (hole) ws_store(p, holes + i - before, static_cast<int>(i));
    if (here && i >= n) ws_store(p, movers + n - 1 - before, static_cast<int>(i));
    if (i < w.page1) {
      if (FP4Q_IN_RANGE(p, p.out_map + i, 4, p.out_map, 4LL * p.c.num_pages))
        __stcg(p.out_map + i, here ? static_cast<int>(i) : -1);
      set_out_ref(p, i, here && i < n ? refs : 0);
    }
    n_holes += __popc(__ballot_sync(kAll, hole));
    rank += __popc(who);
  }
  if (w.lane == 0) ws_store(p, kWsWanted + w.warp, n_holes);
  plan_sync();

  int moves;
  counts_before(p, w, kWsWanted, moves);
  for (int r = w.thread; r < moves; r += w.threads) {
    const int src = ws_load(p, movers + moves - 1 - r), dst = ws_load(p, holes + r);
    if (FP4Q_IN_RANGE(p, p.out_map + src, 4, p.out_map, 4LL * p.c.num_pages)) __stcg(p.out_map + src, dst);
    set_out_ref(p, dst, page_ref(p, src));
  }
  if (w.thread == 0) {
    ws_store(p, kWsHeader + kHeadMoves, moves);
    if (FP4Q_IN_RANGE(p, p.out_live, 4, p.out_live, 4)) *p.out_live = n;
  }
  plan_sync();

  const int most = static_cast<int>(p.max_pages), segs = (most + 127) / 128;
  for (int u = w.warp; u < p.B * segs; u += w.warps) {     // a warp takes 128 entries of a row
    const int b = u / segs, from = (u - b * segs) * 128 + w.lane;
    const int used = pages_of(p, tokens_of(p, b));
    int page[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) page[k] = from + 32 * k < used ? old_entry(p, b, from + 32 * k) : -1;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool here = is_page(p, page[k]) && FP4Q_IN_RANGE(p, p.out_map + page[k], 4, p.out_map, 4LL * p.c.num_pages);
      page[k] = here ? __ldcg(p.out_map + page[k]) : -1;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (from + 32 * k < most) set_entry(p, p.B, static_cast<int64_t>(b) * most + from + 32 * k, page[k]);
  }
}

// The moved pages, 16 bytes a thread and eight of them in flight: HBM bounds the time.
constexpr int kMoveThreads = 256, kMoveEach = 8;
__global__ void __launch_bounds__(kMoveThreads) kv_compact_copy_kernel(const KvPagesParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int moves = ws_load(p, kWsHeader + kHeadMoves);
  const int64_t holes = kWsPages, movers = kWsPages + p.c.num_pages;
  // 16-byte pieces of a page: codes of keys and values, then scales of keys and values
  const int64_t slots = static_cast<int64_t>(p.c.heads) * p.c.page_size;
  const int64_t codes = slots * p.c.D / 32, scales = slots * p.c.D / 256, all = 2 * (codes + scales);
  constexpr int kSlab = kMoveThreads * kMoveEach;
  const int64_t slabs = (all + kSlab - 1) / kSlab;
  for (int64_t s = blockIdx.x; s < moves * slabs; s += gridDim.x) {
    const int64_t r = s / slabs;
    const int64_t src = ws_load(p, movers + moves - 1 - r), dst = ws_load(p, holes + r);
    const int64_t x0 = (s - r * slabs) * kSlab + threadIdx.x;
    uint4 v[kMoveEach];
    uint4* to[kMoveEach];
#pragma unroll
    for (int j = 0; j < kMoveEach; ++j) {
      const int64_t x = x0 + j * kMoveThreads;
      to[j] = nullptr;
      if (x >= all) continue;
      const bool code = x < 2 * codes;
      const int64_t y = code ? x : x - 2 * codes, each = code ? codes : scales;
      const bool value = y >= each;
      uint8_t* base = code ? (value ? p.c.v_packed : p.c.k_packed) : (value ? p.c.v_sf : p.c.k_sf);
      const int64_t at = value ? y - each : y;
      const long long extent = code ? kv_packed_extent(p.c) : kv_sf_extent(p.c);
      const uint4* from = reinterpret_cast<const uint4*>(base) + src * each + at;
      uint4* out = reinterpret_cast<uint4*>(base) + dst * each + at;
      if (!FP4Q_IN_RANGE(p, from, 16, base, extent) || !FP4Q_IN_RANGE(p, out, 16, base, extent)) continue;
      v[j] = __ldcs(from);
      to[j] = out;
    }
#pragma unroll
    for (int j = 0; j < kMoveEach; ++j)
      if (to[j]) __stcs(to[j], v[j]);
  }
}

// CTAs of a plan over that many pages and table entries: one where that does it (no barrier between
// CTAs), else as many as are portable.
unsigned plan_ctas(int64_t work) { return work <= 4 * kPlanThreads ? 1 : work <= 16 * kPlanThreads ? 4 : kPlanMostCtas; }

cudaError_t launch_plan(void (*kernel)(KvPagesParams), unsigned ctas, const KvPagesParams& p, int pdl,
                        cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = stream;
  // (a CTA alone is a cluster of its own without being told so)
  cfg.attrs = ctas > 1 || pdl ? attr : nullptr;
  cfg.numAttrs = ctas > 1 ? 2 : pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}
cudaError_t launch_after(void (*kernel)(KvPagesParams), dim3 grid, int threads, const KvPagesParams& p,
                         cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;                              // its launch overlaps the plan
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

int64_t kv_pages_workspace(int64_t num_pages, int64_t N) { return ws_copies(num_pages, N) + 4 * N; }

// A fork whose plan is one CTA and whose copies (a page a child at most) are no more than this
// makes them there: 4 children of 16-token pages 18.2 -> 14.4 us; with 0.7 MB one CTA takes 20 us
// for what 140 do in 4.
constexpr int64_t kForkOwnCopies = 64 << 10;

cudaError_t launch_kv_fork(const KvPagesParams& p, int pdl, cudaStream_t stream) {
  const unsigned ctas = plan_ctas(p.c.num_pages + (p.B + static_cast<int64_t>(p.N)) * p.max_pages);
  const int64_t page_bytes = 18LL * p.c.heads * p.c.page_size * p.c.D / 16;
  if (ctas == 1 && p.N * page_bytes <= kForkOwnCopies && static_cast<int64_t>(p.N) * p.new_tokens <= 4096)
    return launch_plan(kv_fork_plan_kernel<true>, ctas, p, pdl, stream);
  const cudaError_t e = launch_plan(kv_fork_plan_kernel<false>, ctas, p, pdl, stream);
  if (e != cudaSuccess || p.N == 0) return e;
  return launch_after(kv_fork_copy_kernel, dim3(static_cast<unsigned>(p.N), static_cast<unsigned>(p.c.heads)),
                      kForkThreads, p, stream);
}

cudaError_t launch_kv_trim(const KvPagesParams& p, int pdl, cudaStream_t stream) {
  return launch_plan(kv_trim_kernel, plan_ctas(p.c.num_pages + p.B * p.max_pages), p, pdl, stream);
}

cudaError_t launch_kv_compact(const KvPagesParams& p, int pdl, cudaStream_t stream) {
  const cudaError_t e = launch_plan(kv_compact_plan_kernel, plan_ctas(2 * p.c.num_pages + p.B * p.max_pages), p, pdl, stream);
  if (e != cudaSuccess) return e;
  const int64_t page_bytes = 18LL * p.c.heads * p.c.page_size * p.c.D / 16;
  const int64_t slabs = (p.c.num_pages / 2) * ((page_bytes + 16 * kMoveThreads * kMoveEach - 1) / (16 * kMoveThreads * kMoveEach));
  const int64_t ctas = std::max<int64_t>(1, std::min<int64_t>(slabs, 4LL * sm_count_current_device()));
  return launch_after(kv_compact_copy_kernel, dim3(static_cast<unsigned>(ctas)), kMoveThreads, p, stream);
}

}  // namespace fp4q
