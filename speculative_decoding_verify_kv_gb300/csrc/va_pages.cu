// Pages of a paged cache: forking and growing sequences, giving pages back,
// pulling the live pages of a pool together, and copying pages.
//
// The state is the block table (-1: no page) and one reference count per
// page; a page is free when its count is 0.  Fresh pages are the free ones
// of lowest index, in command order, and moved pages fill the holes in
// ascending order, so every result is a function of the inputs alone: the
// ranks come from prefix sums, the atomics only add.
//
// The planning kernels (fork, free, compact) touch a few hundred kilobytes
// of integers and are bound by latency.  Each is one launch of one cluster
// of eight CTAs: the counts are split over its 256 warps, whose partial
// sums meet through distributed shared memory, and the cluster's barriers
// order the steps (check everything, then change anything) without a
// second launch.  The copy kernel is bound by the bytes it moves.
#include <cooperative_groups.h>
#include <string.h>

#include "va_common.cuh"
#include "va_host.h"

namespace va {
namespace cg = cooperative_groups;

constexpr int kPlanThreads = 1024;
constexpr int kPlanCtas = 8;
constexpr int kPlanWarps = kPlanCtas * kPlanThreads / 32;

struct PageParams {
  int num_seqs, max_blocks, num_blocks;
  int* table;
  int* ref;
  int count;          // commands
  const int* a;       // fork: src; free: sequence
  const int* b;       // fork: dst; free: first entry
  const int* c;       // fork: tokens; free: one past the last entry
  const int* d;       // fork: entries
  int* copies;        // [..][2]
  int* num_copies;
  int* live;
  int* ws;
  unsigned* status;
};

struct PlanShared {
  unsigned seg[kPlanWarps];  // each warp's count
  unsigned err;
  unsigned scan[32];
  int below;
};

// One warp's share of n items, in whole groups of 32.
__device__ __forceinline__ void warp_share(int n, int warp, int* lo, int* hi) {
  const int per = ((n + kPlanWarps - 1) / kPlanWarps + 31) / 32 * 32;
  *lo = (int)min((long long)warp * per, (long long)n);
  *hi = min(*lo + per, n);
}

__device__ __forceinline__ unsigned warp_add(unsigned v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Each warp's count v (the same in every lane) into every CTA's table.
__device__ __forceinline__ void share_count(cg::cluster_group& cluster, PlanShared& sh, int gwarp, int lane,
                                            unsigned v) {
  if (lane < kPlanCtas) *cluster.map_shared_rank(&sh.seg[gwarp], lane) = v;
}

__device__ __forceinline__ unsigned sum_before(const PlanShared& sh, int gwarp, int lane) {
  unsigned t = 0;
  for (int g = lane; g < gwarp; g += 32) t += sh.seg[g];
  return warp_add(t);
}

// An error anywhere reaches the first CTA; read_error after a cluster barrier.
__device__ __forceinline__ void note_error(cg::cluster_group& cluster, PlanShared& sh, unsigned bits) {
  atomicOr(cluster.map_shared_rank(&sh.err, 0), bits);
}
__device__ __forceinline__ unsigned read_error(cg::cluster_group& cluster, PlanShared& sh) {
  return *cluster.map_shared_rank(&sh.err, 0);
}

// What the caller's status word holds on entry: after an earlier step of
// it failed, a planning call changes nothing.  One thread of the cluster
// reads it, so that every CTA decides alike.
__device__ __forceinline__ unsigned status_before(const PageParams& p) {
  return p.status ? *reinterpret_cast<volatile unsigned*>(p.status) : 0u;
}

// A table entry that holds a page in use.
__device__ __forceinline__ bool page_in_use(const PageParams& p, int e) {
  return e >= 0 && e < p.num_blocks && p.ref[e] > 0;
}

// Does command i of a fork take this entry (col) from the free pages?
__device__ __forceinline__ bool takes_fresh(bool grow, int full, int keep, int pages, int col, int old) {
  return grow ? col >= keep && col < pages && old < 0 : col >= full && col < pages;
}

// Fork and grow.  Workspace: mark[num_seqs], need[count], tail[count],
// free pages found [num_blocks].
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
    pages_fork_kernel(const PageParams p) {
  __shared__ PlanShared sh;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, gwarp = rank * (kPlanThreads / 32) + tid / 32;
  const int gtid = rank * kPlanThreads + tid;
  int* mark = p.ws;
  int* need = mark + p.num_seqs;
  int* tail = need + p.count;
  int* found = tail + p.count;
  if (tid == 0) sh.err = rank == 0 ? status_before(p) : 0u;
  for (int s = gtid; s < p.num_seqs; s += kPlanCtas * kPlanThreads) mark[s] = 0;
  cluster.sync();

  // Check every command and count what it needs, one warp each; count the
  // free pages, one part of the pool per warp.
  for (int i = gwarp; i < p.count; i += kPlanWarps) {
    const int src = p.a[i], dst = p.b[i], len = p.c[i], pages = p.d[i];
    unsigned err = 0u;
    int fresh = 0, tails = 0;
    if (src < 0 || src >= p.num_seqs || dst < 0 || dst >= p.num_seqs) {
      err = VA_DEV_BAD_ROWS;
    } else if (len < 0 || pages < 0 || pages > p.max_blocks || len > pages * kPage) {
      err = VA_DEV_CTX_OVERFLOW;
    } else {
      const bool grow = src == dst;
      const int full = len / kPage, keep = (len + kPage - 1) / kPage;
      const int* row = p.table + (long long)src * p.max_blocks;
      const int end = grow ? pages : keep;
      for (int c = lane; c < end; c += 32) {
        const int e = row[c];
        if (e != -1 && !page_in_use(p, e)) err = VA_DEV_BAD_BLOCK;
        if (!grow && c == full && e < 0) err = VA_DEV_BAD_BLOCK;  // the page to copy
        if (grow && takes_fresh(true, full, keep, pages, c, e)) ++fresh;
      }
      fresh = (int)warp_add((unsigned)fresh);
      if (!grow) {
        fresh = pages - full;
        tails = keep - full;
      }
      if (lane == 0 && atomicAdd(&mark[dst], 1) != 0) err = VA_DEV_BAD_ROWS;  // named twice
    }
    if (lane == 0) {
      need[i] = fresh;
      tail[i] = tails;
    }
    if (err) note_error(cluster, sh, err);
  }
  int lo, hi;
  warp_share(p.num_blocks, gwarp, &lo, &hi);
  unsigned freec = 0;
#pragma unroll 4
  for (int i = lo + lane; i < hi; i += 32) {
    const int r = p.ref[i];
    if (r < 0) note_error(cluster, sh, VA_DEV_BAD_BLOCK);
    freec += r == 0;
  }
  freec = warp_add(freec);
  share_count(cluster, sh, gwarp, lane, freec);
  cluster.sync();
  // A source that this call rewrites has no defined contents.
  for (int i = gtid; i < p.count; i += kPlanCtas * kPlanThreads) {
    const int src = p.a[i], dst = p.b[i];
    if (src >= 0 && src < p.num_seqs && src != dst && mark[src] != 0) note_error(cluster, sh, VA_DEV_BAD_ROWS);
  }
  // The first CTA turns the needs into running totals.
  if (rank == 0) {
    __shared__ unsigned base_need, base_tail;
    if (tid == 0) base_need = base_tail = 0u;
    __syncthreads();
    for (int i0 = 0; i0 < p.count; i0 += kPlanThreads) {
      const int i = i0 + tid;
      unsigned a = i < p.count ? (unsigned)need[i] : 0u, b = i < p.count ? (unsigned)tail[i] : 0u;
      unsigned long long v = ((unsigned long long)b << 32) | a;
      unsigned long long inc = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
      }
      __shared__ unsigned long long part[32];
      if (lane == 31) part[tid / 32] = inc;
      __syncthreads();
      unsigned long long off = 0ull;
      for (int w = 0; w < tid / 32; ++w) off += part[w];
      const unsigned long long ex = off + inc - v;
      const unsigned bn = base_need, bt = base_tail;
      if (i < p.count) {
        need[i] = (int)(bn + (unsigned)ex);
        tail[i] = (int)(bt + (unsigned)(ex >> 32));
      }
      __syncthreads();
      if (tid == kPlanThreads - 1) {
        base_need = bn + (unsigned)(off + inc);
        base_tail = bt + (unsigned)((off + inc) >> 32);
      }
      __syncthreads();
    }
    if (tid == 0) {
      sh.below = (int)base_need;
      sh.scan[0] = base_tail;
    }
  }
  cluster.sync();
  const unsigned wanted = (unsigned)*cluster.map_shared_rank(&sh.below, 0);
  const unsigned tails_all = *cluster.map_shared_rank(&sh.scan[0], 0);
  unsigned err = read_error(cluster, sh);
  const unsigned total = sum_before(sh, kPlanWarps, lane);
  if (!err && total < wanted) err = VA_DEV_NO_PAGES;
  const unsigned ahead = sum_before(sh, gwarp, lane);
  if (err) {
    if (rank == 0 && tid == 0) {
      flag(p.status, err);
      *p.num_copies = 0;
    }
    cluster.sync();  // the first CTA's memory is read until here
    return;
  }
  // The wanted free pages, ascending, and their first reference.
  unsigned at = ahead;
  for (int i0 = lo; i0 < hi && at < wanted; i0 += 32) {
    const int i = i0 + lane;
    const bool is_free = i < hi && p.ref[i] == 0;
    const unsigned m = __ballot_sync(0xffffffffu, is_free);
    const unsigned r = at + __popc(m & ((1u << lane) - 1u));
    if (is_free && r < wanted) found[r] = i;
    at += __popc(m);
  }
  cluster.sync();
  // Apply, one warp per command.
  for (int i = gwarp; i < p.count; i += kPlanWarps) {
    const int src = p.a[i], dst = p.b[i], len = p.c[i], pages = p.d[i];
    const bool grow = src == dst;
    const int full = len / kPage, keep = (len + kPage - 1) / kPage;
    const int* from = p.table + (long long)src * p.max_blocks;
    int* to = p.table + (long long)dst * p.max_blocks;
    int next = need[i];
    const int end = grow ? pages : p.max_blocks;
    for (int c0 = grow ? keep : 0; c0 < end; c0 += 32) {
      const int c = c0 + lane;
      const bool in = c < end;
      const int old = in && (grow || c < keep) ? from[c] : -1;
      const bool fresh = in && takes_fresh(grow, full, keep, pages, c, old);
      const unsigned m = __ballot_sync(0xffffffffu, fresh);
      int e = grow || c < full ? old : -1;
      if (fresh) {
        e = found[next + __popc(m & ((1u << lane) - 1u))];
        p.ref[e] = 1;
        if (!grow && c == full && keep > full) {  // the partial page is copied
          p.copies[2 * tail[i]] = old;
          p.copies[2 * tail[i] + 1] = e;
        }
      } else if (in && !grow && e >= 0) {
        atomicAdd(&p.ref[e], 1);
      }
      next += __popc(m);
      if (in && (!grow || fresh)) to[c] = e;
    }
  }
  if (rank == 0 && tid == 0) *p.num_copies = (int)tails_all;
}

// Give back the table entries [first, last) of the listed sequences.
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
    pages_free_kernel(const PageParams p) {
  __shared__ PlanShared sh;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, gwarp = rank * (kPlanThreads / 32) + tid / 32;
  if (tid == 0) sh.err = rank == 0 ? status_before(p) : 0u;
  cluster.sync();
  for (int i = gwarp; i < p.count; i += kPlanWarps) {
    const int s = p.a[i], first = p.b[i], last = p.c[i];
    unsigned err = 0u;
    if (s < 0 || s >= p.num_seqs) {
      err = VA_DEV_BAD_ROWS;
    } else if (first < 0 || last < first || last > p.max_blocks) {
      err = VA_DEV_CTX_OVERFLOW;
    } else {
      for (int c = first + lane; c < last; c += 32) {
        const int e = p.table[(long long)s * p.max_blocks + c];
        if (e != -1 && !page_in_use(p, e)) err = VA_DEV_BAD_BLOCK;
      }
    }
    if (err) note_error(cluster, sh, err);
  }
  cluster.sync();
  const unsigned err = read_error(cluster, sh);
  cluster.sync();  // the first CTA's memory is read until here
  if (err) {
    if (rank == 0 && tid == 0) flag(p.status, err);
    return;
  }
  for (int i = gwarp; i < p.count; i += kPlanWarps) {
    const int s = p.a[i], first = p.b[i], last = p.c[i];
    for (int c = first + lane; c < last; c += 32) {
      // Ranges may overlap: the exchange gives each entry to one of them.
      const int e = atomicExch(&p.table[(long long)s * p.max_blocks + c], -1);
      if (e < 0) continue;
      if (atomicSub(&p.ref[e], 1) <= 0) {  // more entries than references
        atomicAdd(&p.ref[e], 1);
        flag(p.status, VA_DEV_BAD_BLOCK);
      }
    }
  }
}

// Pull the live pages together: with N pages in use, the k-th page in use
// at or above N moves to the k-th hole below N.  Workspace: new place of
// each page [num_blocks].
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanThreads)
    pages_compact_kernel(const PageParams p) {
  __shared__ PlanShared sh;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, gwarp = rank * (kPlanThreads / 32) + tid / 32;
  const int gtid = rank * kPlanThreads + tid;
  if (tid == 0) sh.err = rank == 0 ? status_before(p) : 0u;
  cluster.sync();
  int lo, hi;
  warp_share(p.num_blocks, gwarp, &lo, &hi);
  unsigned livec = 0;
#pragma unroll 4
  for (int i = lo + lane; i < hi; i += 32) {
    const int r = p.ref[i];
    if (r < 0) note_error(cluster, sh, VA_DEV_BAD_BLOCK);
    livec += r > 0;
  }
  livec = warp_add(livec);
  const long long entries = (long long)p.num_seqs * p.max_blocks;
#pragma unroll 4
  for (long long i = gtid; i < entries; i += kPlanCtas * kPlanThreads) {
    const int e = p.table[i];
    if (e != -1 && !page_in_use(p, e)) note_error(cluster, sh, VA_DEV_BAD_BLOCK);
  }
  share_count(cluster, sh, gwarp, lane, livec);
  cluster.sync();
  const unsigned err = read_error(cluster, sh);
  const int live = (int)sum_before(sh, kPlanWarps, lane);
  const unsigned ahead = sum_before(sh, gwarp, lane);
  // The warp whose part holds page N counts the pages in use below N.
  if (!err && (live < p.num_blocks ? lo <= live && live < hi : gwarp == 0)) {
    unsigned c = 0;
    if (live < p.num_blocks) {
      for (int i = lo + lane; i < live; i += 32) c += p.ref[i] > 0;
      c = warp_add(c) + ahead;
    } else {
      c = (unsigned)live;
    }
    if (lane < kPlanCtas) *cluster.map_shared_rank(&sh.below, lane) = (int)c;
  }
  cluster.sync();
  if (err) {
    if (rank == 0 && tid == 0) {
      flag(p.status, err);
      *p.num_copies = 0;
      if (p.live) *p.live = 0;
    }
    return;
  }
  const int below = sh.below;
  // Holes below N, then the pages that fill them.
  unsigned at = ahead;
  for (int i0 = lo; i0 < hi && i0 < live; i0 += 32) {
    const int i = i0 + lane;
    const bool used = i < hi && p.ref[i] > 0;
    const unsigned m = __ballot_sync(0xffffffffu, used);
    const int rank_live = (int)(at + __popc(m & ((1u << lane) - 1u)));
    if (i < hi && i < live && !used) p.copies[2 * (i - rank_live) + 1] = i;
    at += __popc(m);
  }
  cluster.sync();
  at = ahead;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    // Counts below N change under other warps' hands here; those at or
    // above N are this warp's own, and `below` pages in use precede them.
    const int r = i < hi && i >= live ? p.ref[i] : 0;
    const unsigned m = __ballot_sync(0xffffffffu, r > 0);
    if (i0 <= live) at = (unsigned)below;
    if (r > 0) {
      const int k = (int)(at + __popc(m & ((1u << lane) - 1u))) - below;
      const int to = p.copies[2 * k + 1];
      p.copies[2 * k] = i;
      p.ws[i] = to;
      p.ref[to] = r;
      p.ref[i] = 0;
    }
    at += __popc(m);
  }
  cluster.sync();
#pragma unroll 4
  for (long long i = gtid; i < entries; i += kPlanCtas * kPlanThreads) {
    const int e = p.table[i];
    if (e >= live) p.table[i] = p.ws[e];
  }
  if (rank == 0 && tid == 0) {
    *p.num_copies = live - below;
    if (p.live) *p.live = live;
  }
}

// ---------------------------------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kCopyPools = 64;  // pools of one launch

struct CopyParams {
  uint4* pool[kCopyPools];
  int num_blocks, max_copies;
  int vecs;  // 16-byte pieces of a page
  const int* copies;
  const int* num_copies;
  unsigned* status;
};

// grid = (CTAs per pool, pools): page pairs in turn, 16 bytes per thread.
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const CopyParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // After a failed plan nothing is copied.  This kernel's own finding does
  // not count: whether other pairs are copied must not depend on its timing.
  if (p.status && (*reinterpret_cast<volatile unsigned*>(p.status) & ~VA_DEV_BAD_COPY) != 0u) return;
  const int n = min(*p.num_copies, p.max_copies);
  if (*p.num_copies > p.max_copies && threadIdx.x == 0) flag(p.status, VA_DEV_BAD_COPY);
  uint4* pool = p.pool[blockIdx.y];
  for (int c = blockIdx.x; c < n; c += gridDim.x) {
    const int src = p.copies[2 * c], dst = p.copies[2 * c + 1];
    if (src < 0 || src >= p.num_blocks || dst < 0 || dst >= p.num_blocks) {
      if (threadIdx.x == 0) flag(p.status, VA_DEV_BAD_COPY);
      continue;
    }
    const uint4* from = pool + (long long)src * p.vecs;
    uint4* to = pool + (long long)dst * p.vecs;
#pragma unroll 4
    for (int i = threadIdx.x; i < p.vecs; i += kCopyThreads) to[i] = from[i];
  }
}

static va_status check_pool(const va_page_pool* g) {
  if (!g || !g->block_table || !g->ref_count) return VA_ERR_INVALID_ARG;
  if (g->num_seqs < 1 || g->max_blocks_per_seq < 1 || g->num_blocks < 1) return VA_ERR_INVALID_ARG;
  // Totals of fresh pages and token counts stay within 32 bits.
  if (g->max_blocks_per_seq > (1 << 26)) return VA_ERR_UNSUPPORTED;
  if ((uintptr_t)g->block_table % 4 || (uintptr_t)g->ref_count % 4) return VA_ERR_ALIGNMENT;
  return VA_OK;
}

static PageParams page_params(const va_page_pool* g, uint32_t* status) {
  PageParams q;
  memset(&q, 0, sizeof(q));
  q.num_seqs = g->num_seqs;
  q.max_blocks = g->max_blocks_per_seq;
  q.num_blocks = g->num_blocks;
  q.table = g->block_table;
  q.ref = g->ref_count;
  q.status = (unsigned*)status;
  return q;
}

template <typename P>
static cudaError_t launch_pages(void (*kernel)(const P), dim3 grid, int threads, cudaStream_t st, const P& q) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, q);
  return e != cudaSuccess ? e : cudaGetLastError();
}

static size_t pages_ws_bytes(const va_page_pool* g, int32_t num_forks) {
  const size_t ints = (size_t)g->num_seqs + 2 * (size_t)num_forks + (size_t)g->num_blocks;
  return (ints * 4 + 255) / 256 * 256;
}

// Workspace and stream of a planning call.
static va_status check_plan(size_t need, void* ws, size_t ws_bytes, cudaStream_t cs) {
  if (!ws || ws_bytes < need) return VA_ERR_WORKSPACE_TOO_SMALL;
  if (((uintptr_t)ws & 255u) != 0) return VA_ERR_ALIGNMENT;
  return check_stream_device(cs);
}

}  // namespace va

using namespace va;

extern "C" {

size_t verify_attn_pages_workspace_size(const va_page_pool* pool, int32_t num_forks) {
  if (check_pool(pool) != VA_OK || num_forks < 0) return 0;
  return pages_ws_bytes(pool, num_forks);
}

va_status verify_attn_pages_fork(const va_page_pool* pool, int32_t num_forks, const int32_t* src,
                                 const int32_t* dst, const int32_t* len, const int32_t* pages, int32_t* copies,
                                 int32_t* num_copies, void* ws, size_t ws_bytes, uint32_t* status, void* stream) {
  va_status st = check_pool(pool);
  if (st != VA_OK) return st;
  if (num_forks < 0 || !num_copies) return VA_ERR_INVALID_ARG;
  if (num_forks > 0 && (!src || !dst || !len || !pages || !copies)) return VA_ERR_INVALID_ARG;
  if ((long long)num_forks * pool->max_blocks_per_seq > 0x7fffffffLL) return VA_ERR_UNSUPPORTED;
  cudaStream_t cs = (cudaStream_t)stream;
  st = check_plan(pages_ws_bytes(pool, num_forks), ws, ws_bytes, cs);
  if (st != VA_OK) return st;
  PageParams q = page_params(pool, status);
  q.count = num_forks;
  q.a = src;
  q.b = dst;
  q.c = len;
  q.d = pages;
  q.copies = copies;
  q.num_copies = num_copies;
  q.ws = (int*)ws;
  cudaError_t e = launch_pages(pages_fork_kernel, dim3(kPlanCtas), kPlanThreads, cs, q);
  return e == cudaSuccess ? VA_OK : note_cuda(e);
}

va_status verify_attn_pages_free(const va_page_pool* pool, int32_t num_ranges, const int32_t* seq,
                                 const int32_t* first, const int32_t* last, uint32_t* status, void* stream) {
  va_status st = check_pool(pool);
  if (st != VA_OK) return st;
  if (num_ranges < 0 || (num_ranges > 0 && (!seq || !first || !last))) return VA_ERR_INVALID_ARG;
  if (num_ranges == 0) return VA_OK;
  cudaStream_t cs = (cudaStream_t)stream;
  st = check_stream_device(cs);
  if (st != VA_OK) return st;
  PageParams q = page_params(pool, status);
  q.count = num_ranges;
  q.a = seq;
  q.b = first;
  q.c = last;
  cudaError_t e = launch_pages(pages_free_kernel, dim3(kPlanCtas), kPlanThreads, cs, q);
  return e == cudaSuccess ? VA_OK : note_cuda(e);
}

va_status verify_attn_pages_compact(const va_page_pool* pool, int32_t* copies, int32_t* num_copies,
                                    int32_t* live_blocks, void* ws, size_t ws_bytes, uint32_t* status,
                                    void* stream) {
  va_status st = check_pool(pool);
  if (st != VA_OK) return st;
  if (!num_copies || (pool->num_blocks > 1 && !copies)) return VA_ERR_INVALID_ARG;
  cudaStream_t cs = (cudaStream_t)stream;
  st = check_plan(pages_ws_bytes(pool, 0), ws, ws_bytes, cs);
  if (st != VA_OK) return st;
  PageParams q = page_params(pool, status);
  q.copies = copies;
  q.num_copies = num_copies;
  q.live = live_blocks;
  q.ws = (int*)ws;
  cudaError_t e = launch_pages(pages_compact_kernel, dim3(kPlanCtas), kPlanThreads, cs, q);
  return e == cudaSuccess ? VA_OK : note_cuda(e);
}

va_status verify_attn_pages_copy(void* const* pools, int32_t num_pools, int64_t page_bytes, int32_t num_blocks,
                                 const int32_t* copies, const int32_t* num_copies, int32_t max_copies,
                                 uint32_t* status, void* stream) {
  if (num_pools < 0 || page_bytes < 1 || num_blocks < 1 || max_copies < 0 || !num_copies)
    return VA_ERR_INVALID_ARG;
  if ((num_pools > 0 && !pools) || (max_copies > 0 && !copies)) return VA_ERR_INVALID_ARG;
  if (page_bytes % 16 || page_bytes > (1LL << 30)) return VA_ERR_UNSUPPORTED;
  for (int32_t i = 0; i < num_pools; ++i) {
    if (!pools[i]) return VA_ERR_INVALID_ARG;
    if (((uintptr_t)pools[i] & 15u) != 0) return VA_ERR_ALIGNMENT;
  }
  if (num_pools == 0 || max_copies == 0) return VA_OK;
  cudaStream_t cs = (cudaStream_t)stream;
  va_status st = check_stream_device(cs);
  if (st != VA_OK) return st;
  for (int32_t i0 = 0; i0 < num_pools; i0 += kCopyPools) {
    const int32_t m = num_pools - i0 < kCopyPools ? num_pools - i0 : kCopyPools;
    CopyParams q;
    memset(&q, 0, sizeof(q));
    for (int32_t i = 0; i < m; ++i) q.pool[i] = (uint4*)pools[i0 + i];
    q.num_blocks = num_blocks;
    q.max_copies = max_copies;
    q.vecs = (int)(page_bytes / 16);
    q.copies = copies;
    q.num_copies = num_copies;
    q.status = (unsigned*)status;
    int per = (152 * 8 + m - 1) / m;
    if (per > max_copies) per = max_copies;
    cudaError_t e = launch_pages(pages_copy_kernel, dim3((unsigned)per, (unsigned)m), kCopyThreads, cs, q);
    if (e != cudaSuccess) return note_cuda(e);
  }
  return VA_OK;
}

}  // extern "C"
