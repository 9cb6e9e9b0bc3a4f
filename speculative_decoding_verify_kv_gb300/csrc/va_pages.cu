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
// of integers and are bound by latency: each is one launch of one CTA, or
// for large pools of one cluster of eight, so that barriers order the steps
// (check everything, then change anything) without a second launch.  The
// counts are split over the warps, whose partial sums meet in (distributed)
// shared memory.  The copy kernel is bound by the bytes it moves.
#include <cooperative_groups.h>
#include <string.h>

#include "va_common.cuh"
#include "va_host.h"

namespace va {
namespace cg = cooperative_groups;

constexpr int kPlanThreads = 1024;
constexpr int kCtaWarps = kPlanThreads / 32;
constexpr int kPart = 128;  // table entries that a warp goes through at once
constexpr int kWideCtas = 8;
// Largest plan of one CTA.  Three forks over 2,048 pages (2,300 integers):
// 8.5 us against 10.5 with a cluster; a compaction of 27,000: 16.3 against
// 13.0; 60 forks of rows of 514 entries over 32,768 pages: 41 against 18.
constexpr long long kOneCtaInts = 8192;

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
  // extend: a is tokens held, b new rows
  int mode, max_rows;
  const int* parent;
  const unsigned char* kind;
  int* cu;
  int* row_first;  // first fresh page of each sequence (many sequences)
  int* row_seq;
  int* position;
  long long* slot;
};

struct PlanShared {
  unsigned seg[kWideCtas * kCtaWarps];  // each warp's count
  unsigned err;
  unsigned total_need, total_tail;
  int below;
};

// The CTAs of a planning kernel: one, or a cluster of NC.
template <int NC>
struct Team {
  cg::cluster_group cluster;
  __device__ __forceinline__ Team() : cluster(cg::this_cluster()) {}
  __device__ __forceinline__ int rank() const { return NC > 1 ? (int)cluster.block_rank() : 0; }
  __device__ __forceinline__ void sync() {
    if (NC > 1) cluster.sync();
    else __syncthreads();
  }
  template <typename V>
  __device__ __forceinline__ V* at(V* p, int r) {
    return NC > 1 ? cluster.map_shared_rank(p, r) : p;
  }
};

// One warp's share of n items, in whole groups of 32.
template <int NC>
__device__ __forceinline__ void warp_share(int n, int warp, int* lo, int* hi) {
  constexpr int W = NC * kCtaWarps;
  const int per = ((n + W - 1) / W + 31) / 32 * 32;
  *lo = (int)min((long long)warp * per, (long long)n);
  *hi = min(*lo + per, n);
}

__device__ __forceinline__ unsigned warp_add(unsigned v) { return __reduce_add_sync(0xffffffffu, v); }

// Each warp's count v (the same in every lane) into every CTA's table.
template <int NC>
__device__ __forceinline__ void share_count(Team<NC>& team, PlanShared& sh, int gwarp, int lane, unsigned v) {
  if (lane < NC) *team.at(&sh.seg[gwarp], lane) = v;
}

__device__ __forceinline__ unsigned sum_before(const PlanShared& sh, int gwarp, int lane) {
  unsigned t = 0;
  for (int g = lane; g < gwarp; g += 32) t += sh.seg[g];
  return warp_add(t);
}

// An error anywhere reaches the first CTA; read_error after a barrier.
template <int NC>
__device__ __forceinline__ void note_error(Team<NC>& team, PlanShared& sh, unsigned bits) {
  atomicOr(team.at(&sh.err, 0), bits);
}
template <int NC>
__device__ __forceinline__ unsigned read_error(Team<NC>& team, PlanShared& sh) {
  return *team.at(&sh.err, 0);
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
template <int NC>
__global__ void __launch_bounds__(kPlanThreads) pages_fork_kernel(const PageParams p) {
  __shared__ PlanShared sh;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Team<NC> team;
  const int rank = team.rank();
  const int tid = threadIdx.x, lane = tid & 31, gwarp = rank * (kPlanThreads / 32) + tid / 32;
  const int gtid = rank * kPlanThreads + tid;
  int* mark = p.ws;
  int* need = mark + p.num_seqs;
  int* tail = need + p.count;
  int* found = tail + p.count;
  if (tid == 0) sh.err = rank == 0 ? status_before(p) : 0u;
  for (int s = gtid; s < p.num_seqs; s += NC * kPlanThreads) mark[s] = 0;
  for (int i = gtid; i < p.count; i += NC * kPlanThreads) need[i] = 0;
  team.sync();

  // Check every command and count what it needs, a warp per 128 entries;
  // count the free pages, one part of the pool per warp.
  const int parts = (p.max_blocks + kPart - 1) / kPart;
  for (long long job = gwarp; job < (long long)p.count * parts; job += NC * kCtaWarps) {
    const int i = (int)(job / parts), part = (int)(job % parts);
    const int src = p.a[i], dst = p.b[i], len = p.c[i], pages = p.d[i];
    unsigned err = 0u;
    if (src < 0 || src >= p.num_seqs || dst < 0 || dst >= p.num_seqs) {
      err = VA_DEV_BAD_ROWS;
    } else if (len < 0 || pages < 0 || pages > p.max_blocks || len > pages * kPage) {
      err = VA_DEV_CTX_OVERFLOW;
    } else {
      const bool grow = src == dst;
      const int full = len / kPage, keep = (len + kPage - 1) / kPage;
      const int* row = p.table + (long long)src * p.max_blocks;
      const int end = grow ? pages : keep;
      int e[4], r[4], fresh = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = part * kPart + 32 * k + lane;
        e[k] = c < end ? row[c] : -1;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) r[k] = e[k] >= 0 && e[k] < p.num_blocks ? p.ref[e[k]] : 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = part * kPart + 32 * k + lane;
        if (c >= end) continue;
        if (e[k] != -1 && r[k] <= 0) err = VA_DEV_BAD_BLOCK;
        if (!grow && c == full && e[k] < 0) err = VA_DEV_BAD_BLOCK;  // the page to copy
        if (grow && takes_fresh(true, full, keep, pages, c, e[k])) ++fresh;
      }
      fresh = (int)warp_add((unsigned)fresh);
      if (lane == 0) {
        if (grow && fresh) atomicAdd(&need[i], fresh);
        if (part == 0) {
          if (!grow) need[i] = pages - full;
          tail[i] = grow ? 0 : keep - full;
          if (atomicAdd(&mark[dst], 1) != 0) err = VA_DEV_BAD_ROWS;  // named twice
        }
      }
    }
    if (err) note_error(team, sh, err);
  }
  int lo, hi;
  warp_share<NC>(p.num_blocks, gwarp, &lo, &hi);
  unsigned freec = 0;
#pragma unroll 4
  for (int i = lo + lane; i < hi; i += 32) {
    const int r = p.ref[i];
    if (r < 0) note_error(team, sh, VA_DEV_BAD_BLOCK);
    freec += r == 0;
  }
  freec = warp_add(freec);
  share_count(team, sh, gwarp, lane, freec);
  team.sync();
  // A source that this call rewrites has no defined contents.
  for (int i = gtid; i < p.count; i += NC * kPlanThreads) {
    const int src = p.a[i], dst = p.b[i];
    if (src >= 0 && src < p.num_seqs && src != dst && mark[src] != 0) note_error(team, sh, VA_DEV_BAD_ROWS);
  }
  // One warp turns the needs into running totals.
  if (gwarp == 0) {
    unsigned base_need = 0u, base_tail = 0u;
    for (int i0 = 0; i0 < p.count; i0 += 32) {
      const int i = i0 + lane;
      const unsigned a = i < p.count ? (unsigned)need[i] : 0u, b = i < p.count ? (unsigned)tail[i] : 0u;
      unsigned ia = a, ib = b;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned ua = __shfl_up_sync(0xffffffffu, ia, o), ub = __shfl_up_sync(0xffffffffu, ib, o);
        if (lane >= o) {
          ia += ua;
          ib += ub;
        }
      }
      if (i < p.count) {
        need[i] = (int)(base_need + ia - a);
        tail[i] = (int)(base_tail + ib - b);
      }
      base_need += __shfl_sync(0xffffffffu, ia, 31);
      base_tail += __shfl_sync(0xffffffffu, ib, 31);
    }
    if (lane == 0) {
      sh.total_need = base_need;
      sh.total_tail = base_tail;
    }
  }
  team.sync();
  const unsigned wanted = *team.at(&sh.total_need, 0);
  const unsigned tails_all = *team.at(&sh.total_tail, 0);
  unsigned err = read_error(team, sh);
  const unsigned total = sum_before(sh, (NC * kCtaWarps), lane);
  if (!err && total < wanted) err = VA_DEV_NO_PAGES;
  const unsigned ahead = sum_before(sh, gwarp, lane);
  if (err) {
    if (rank == 0 && tid == 0) {
      flag(p.status, err);
      *p.num_copies = 0;
    }
    team.sync();  // the first CTA's memory is read until here
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
  team.sync();
  // Apply: a warp per 128 entries of a fork, one for a sequence that grows.
  for (long long job = gwarp; job < (long long)p.count * parts; job += NC * kCtaWarps) {
    const int i = (int)(job / parts), part = (int)(job % parts);
    const int src = p.a[i], dst = p.b[i], len = p.c[i], pages = p.d[i];
    const int full = len / kPage, keep = (len + kPage - 1) / kPage;
    const int* from = p.table + (long long)src * p.max_blocks;
    int* to = p.table + (long long)dst * p.max_blocks;
    if (src != dst) {
      const int* mine = found + need[i] - full;  // of entry c in [full, pages)
#pragma unroll 4
      for (int k = 0; k < kPart; k += 32) {
        const int c = part * kPart + k + lane;
        if (c >= p.max_blocks) continue;
        const int old = c < keep ? from[c] : -1;
        int e = c < full ? old : -1;
        if (c >= full && c < pages) {
          e = mine[c];
          p.ref[e] = 1;
          if (c < keep) {  // the partial page is copied
            p.copies[2 * tail[i]] = old;
            p.copies[2 * tail[i] + 1] = e;
          }
        } else if (e >= 0) {
          atomicAdd(&p.ref[e], 1);
        }
        to[c] = e;
      }
    } else if (part == 0) {
      int next = need[i];
      for (int c0 = keep; c0 < pages; c0 += 32) {
        const int c = c0 + lane;
        const bool fresh = c < pages && from[c] < 0;
        const unsigned m = __ballot_sync(0xffffffffu, fresh);
        if (fresh) {
          const int e = found[next + __popc(m & ((1u << lane) - 1u))];
          p.ref[e] = 1;
          to[c] = e;
        }
        next += __popc(m);
      }
    }
  }
  if (rank == 0 && tid == 0) *p.num_copies = (int)tails_all;
}

// Give back the table entries [first, last) of the listed sequences.
template <int NC>
__global__ void __launch_bounds__(kPlanThreads) pages_free_kernel(const PageParams p) {
  __shared__ PlanShared sh;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Team<NC> team;
  const int rank = team.rank();
  const int tid = threadIdx.x, lane = tid & 31, gwarp = rank * (kPlanThreads / 32) + tid / 32;
  if (tid == 0) sh.err = rank == 0 ? status_before(p) : 0u;
  team.sync();
  const int parts = (p.max_blocks + kPart - 1) / kPart;
  for (long long job = gwarp; job < (long long)p.count * parts; job += NC * kCtaWarps) {
    const int i = (int)(job / parts), c0 = (int)(job % parts) * kPart;
    const int s = p.a[i], first = p.b[i], last = p.c[i];
    unsigned err = 0u;
    if (s < 0 || s >= p.num_seqs) {
      err = VA_DEV_BAD_ROWS;
    } else if (first < 0 || last < first || last > p.max_blocks) {
      err = VA_DEV_CTX_OVERFLOW;
    } else {
#pragma unroll
      for (int k = 0; k < kPart; k += 32) {
        const int c = c0 + k + lane;
        if (c < first || c >= last) continue;
        const int e = p.table[(long long)s * p.max_blocks + c];
        if (e != -1 && !page_in_use(p, e)) err = VA_DEV_BAD_BLOCK;
      }
    }
    if (err) note_error(team, sh, err);
  }
  team.sync();
  const unsigned err = read_error(team, sh);
  team.sync();  // the first CTA's memory is read until here
  if (err) {
    if (rank == 0 && tid == 0) flag(p.status, err);
    return;
  }
  for (long long job = gwarp; job < (long long)p.count * parts; job += NC * kCtaWarps) {
    const int i = (int)(job / parts), c0 = (int)(job % parts) * kPart;
    const int s = p.a[i], first = p.b[i], last = p.c[i];
#pragma unroll
    for (int k = 0; k < kPart; k += 32) {
      const int c = c0 + k + lane;
      if (c < first || c >= last) continue;
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

// Block tables and slot maps from request lengths.  Sequence s holds a[s]
// tokens and gets b[s] rows: entries ceil(a / 16) to ceil((a + b) / 16) - 1
// that hold no page take the lowest free ones, and every row learns its
// sequence, position and slot.  Workspace: need[num_seqs], free pages found
// [num_blocks], first fresh page [num_seqs].
//
// Bound by the latency of its dependent steps, so there are few: check and
// count; each CTA then has every sequence's rows and needs in its own shared
// memory and sums them up itself; the free pages wanted; then tables and rows
// together, since a row can tell its page from the list as well as from the
// table.  Two barriers of the CTAs (three with trees), against six where one CTA
// sums and the rows wait for the tables: 40 sequences of one row, 8,192 pages, 6.2
// us against 14; 256 of up to 8 over 131,072, 12.2 against 23.
// Integers of a step that one CTA plans.  One row a sequence, us by one CTA and by a
// cluster: 40 sequences over 8,192 pages 4.9 and 6.7, 8 over 16,000 5.1 and 6.6, over
// 32,768 6.0 and 7.0, over 65,536 7.7 and 6.8, 1,000 over 8,192 12.9 and 8.4; 256 of 8
// rows over 4,096 7.5 and 7.7, over 131,072 13.9 and 8.3.
constexpr long long kOneCtaExtend = 16384;
constexpr int kSeqLanes = 8;     // go through a sequence's entries
constexpr int kSeqShared = 2048; // sequences whose sums stand in shared memory
constexpr unsigned kSomeHeld = 0x80000000u;  // beside the findings: an entry that would be fresh holds a page
static_assert(kSeqLanes >= kWideCtas, "each lane of a sequence tells one CTA");

struct ExtendShared {
  unsigned count[kWideCtas * kCtaWarps];  // free pages of each warp's part
  unsigned found[kWideCtas * kCtaWarps];  // findings
  unsigned parents;
  unsigned long long part[2][kCtaWarps];
  int cu[kSeqShared + 1];                 // rows, then offsets
  int first[kSeqShared];                  // needs, then each sequence's first fresh page
};

// The largest s with cu[s] <= r: of sequences that start at r, the one with rows.
__device__ __forceinline__ int seq_of_row(const int* cu, int n, int r) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= r) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ bool extend_is_tree(const PageParams& p, int s) {
  return p.mode == VA_MODE_TREE || (p.mode == VA_MODE_MIXED && p.kind[s] != 0);
}

template <int NC>
__global__ void __launch_bounds__(kPlanThreads) pages_extend_kernel(const PageParams p) {
  __shared__ ExtendShared sh;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Team<NC> team;
  if (NC > 1) cluster_started();  // waited for before the first write into another CTA
  const int rank = team.rank();
  const int tid = threadIdx.x, lane = tid & 31, gwarp = rank * kCtaWarps + tid / 32;
  const int gtid = rank * kPlanThreads + tid;
  const bool shared = p.num_seqs <= kSeqShared;
  int* const need_g = p.ws;
  int* const found = p.ws + p.num_seqs;
  if (tid == 0) sh.parents = 0u;

  // Free pages of this warp's part, as bits while it is 1,024 pages or less.
  int lo, hi;
  warp_share<NC>(p.num_blocks, gwarp, &lo, &hi);
  const bool kept = hi - lo <= 1024;
  unsigned err = rank == 0 && tid == 0 ? status_before(p) : 0u;
  unsigned freec = 0, bits = 0;
  {
    int k = 0;
#pragma unroll 8
    for (int i = lo + lane; i < hi; i += 32, ++k) {
      const int r = p.ref[i];
      if (r < 0) err |= VA_DEV_BAD_BLOCK;
      freec += r == 0;
      if (r == 0 && k < 32) bits |= 1u << k;
    }
  }
  if (NC > 1) cluster_met();
  // Check every sequence and count the pages it takes.
  const int sub = lane & (kSeqLanes - 1);
  const unsigned peers = 0xffu << (lane & ~(kSeqLanes - 1));
  const long long groups = (long long)NC * kPlanThreads / kSeqLanes;
  for (long long s0 = gtid / kSeqLanes; s0 < p.num_seqs; s0 += groups) {
    const int s = (int)s0;
    const int held = p.a[s], n = p.b[s];
    int fresh = 0;
    if (n < 0 || (n > kMaxTreeRows && extend_is_tree(p, s))) {
      err |= VA_DEV_BAD_ROWS;
    } else if (held < 0 || ((long long)held + n + kPage - 1) / kPage > p.max_blocks) {
      err |= VA_DEV_CTX_OVERFLOW;
    } else if (n > 0) {
      const int keep = (held + kPage - 1) / kPage, end = (held + n + kPage - 1) / kPage;
      const int* row = p.table + (long long)s * p.max_blocks;
      for (int c = held / kPage + sub; c < end; c += kSeqLanes) {
        const int e = row[c];
        // A page that rows are written to belongs to this sequence alone.
        if (e != -1 && !(e >= 0 && e < p.num_blocks && p.ref[e] == 1)) err |= VA_DEV_BAD_BLOCK;
        if (e == -1 && c < keep) err |= VA_DEV_BAD_BLOCK;  // the page that the held tokens end in
        if (e != -1 && c >= keep) err |= kSomeHeld;
        fresh += e == -1;
      }
    }
    fresh += __shfl_xor_sync(peers, fresh, 1);
    fresh += __shfl_xor_sync(peers, fresh, 2);
    fresh += __shfl_xor_sync(peers, fresh, 4);
    if (!shared) {
      if (sub == 0) need_g[s] = fresh;
    } else if (sub < NC) {
      ExtendShared* to = team.at(&sh, sub);
      to->cu[s] = n;
      to->first[s] = fresh;
    }
  }
  __syncwarp();
  freec = warp_add(freec);
  err = __reduce_or_sync(0xffffffffu, err);
  if (lane < NC) {
    ExtendShared* to = team.at(&sh, lane);
    to->count[gwarp] = freec;
    to->found[gwarp] = err;
  }
  team.sync();

  // Every CTA: findings, free pages in all and before this warp's part.
  unsigned all_free = 0, before = 0;
  err = 0u;
  for (int g = lane; g < NC * kCtaWarps; g += 32) {
    err |= sh.found[g];
    all_free += sh.count[g];
    before += g < gwarp ? sh.count[g] : 0u;
  }
  err = __reduce_or_sync(0xffffffffu, err);
  all_free = warp_add(all_free);
  before = warp_add(before);
  const bool some_held = (err & kSomeHeld) != 0u;
  err &= ~kSomeHeld;
  // Rows and needs to running totals, 1,024 sequences at a time (64-bit sums:
  // past the limits the call fails below).
  unsigned long long total_rows = 0, total_need = 0;
  for (int s0 = 0; s0 < p.num_seqs && !err; s0 += kPlanThreads) {
    const int s = s0 + tid;
    const unsigned long long a = s < p.num_seqs ? (unsigned long long)(shared ? sh.cu[s] : p.b[s]) : 0ull;
    const unsigned long long b = s < p.num_seqs ? (unsigned long long)(shared ? sh.first[s] : need_g[s]) : 0ull;
    unsigned long long ia = a, ib = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long ua = __shfl_up_sync(0xffffffffu, ia, o), ub = __shfl_up_sync(0xffffffffu, ib, o);
      if (lane >= o) {
        ia += ua;
        ib += ub;
      }
    }
    if (lane == 31) {
      sh.part[0][tid / 32] = ia;
      sh.part[1][tid / 32] = ib;
    }
    __syncthreads();
    unsigned long long wa = sh.part[0][lane], wb = sh.part[1][lane];
    const unsigned long long own_a = __shfl_sync(0xffffffffu, wa, tid / 32), own_b = __shfl_sync(0xffffffffu, wb, tid / 32);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long ua = __shfl_up_sync(0xffffffffu, wa, o), ub = __shfl_up_sync(0xffffffffu, wb, o);
      if (lane >= o) {
        wa += ua;
        wb += ub;
      }
    }
    const unsigned long long pa = total_rows + __shfl_sync(0xffffffffu, wa, tid / 32) - own_a + ia - a;
    const unsigned long long pb = total_need + __shfl_sync(0xffffffffu, wb, tid / 32) - own_b + ib - b;
    total_rows += __shfl_sync(0xffffffffu, wa, 31);
    total_need += __shfl_sync(0xffffffffu, wb, 31);
    if (s < p.num_seqs) {
      const int cu = (int)min(pa, 0x7fffffffull), first = (int)min(pb, 0x7fffffffull);
      if (rank == 0) p.cu[s] = cu;
      if (shared) {
        sh.cu[s] = cu;
        sh.first[s] = first;
      }
    }
    __syncthreads();  // part
    if (!shared && rank == 0 && s < p.num_seqs) p.row_first[s] = (int)min(pb, 0x7fffffffull);
  }
  if (!err && total_rows > (unsigned long long)p.max_rows) err = VA_DEV_BAD_ROWS;
  const int rows = err ? 0 : (int)total_rows;
  if (!err) {
    if (rank == 0 && tid == 0) p.cu[p.num_seqs] = rows;
    if (shared && tid == 0) sh.cu[p.num_seqs] = rows;
  }
  if (!shared || p.mode != VA_MODE_CHAIN) {
    if (!shared) team.sync();  // offsets in global memory
    else __syncthreads();
    const int* cu = shared ? sh.cu : p.cu;
    unsigned bad = 0u;
    if (!err && p.mode != VA_MODE_CHAIN) {
      for (int r = gtid; r < rows; r += NC * kPlanThreads) {
        const int s = seq_of_row(cu, p.num_seqs, r);
        const int j = r - cu[s], up = p.parent[r];
        if (extend_is_tree(p, s) && (up < -1 || up >= j)) bad = VA_DEV_BAD_PARENT;
      }
      if (bad)
        for (int c = 0; c < NC; ++c) atomicOr(team.at(&sh.parents, c), bad);
    }
    team.sync();
    err |= sh.parents;
  }
  if (!err && all_free < total_need) err = VA_DEV_NO_PAGES;
  if (err) {
    __syncthreads();  // the first CTA has written offsets
    if (gtid == 0) flag(p.status, err);
    if (rank == 0)
      for (int i = tid; i <= p.num_seqs; i += kPlanThreads) p.cu[i] = 0;
    for (int r = gtid; r < p.max_rows; r += NC * kPlanThreads) {
      p.row_seq[r] = p.position[r] = -1;
      p.slot[r] = -1;
    }
    return;
  }
  // The wanted free pages, ascending, and their first reference.
  const unsigned wanted = (unsigned)total_need;
  unsigned at = before;
  for (int i0 = lo, k = 0; i0 < hi && at < wanted; i0 += 32, ++k) {
    const int i = i0 + lane;
    const bool is_free = kept ? ((bits >> k) & 1u) != 0u : i < hi && p.ref[i] == 0;
    const unsigned m = __ballot_sync(0xffffffffu, is_free);
    const unsigned r = at + __popc(m & ((1u << lane) - 1u));
    if (is_free && r < wanted) {
      found[r] = i;
      p.ref[i] = 1;
    }
    at += __popc(m);
  }
  team.sync();
  const int* cu = shared ? sh.cu : p.cu;
  const int* first = shared ? sh.first : p.row_first;
  for (long long s0 = gtid / kSeqLanes; s0 < p.num_seqs; s0 += groups) {
    const int s = (int)s0;
    const int held = p.a[s], n = p.b[s];
    if (n == 0) continue;  // the same in all lanes of a sequence
    const int end = (held + n + kPage - 1) / kPage;
    int* row = p.table + (long long)s * p.max_blocks;
    int next = first[s];
    for (int c0 = (held + kPage - 1) / kPage; c0 < end; c0 += kSeqLanes) {
      const int c = c0 + sub;
      const bool fresh = c < end && (!some_held || row[c] == -1);
      const unsigned m = __ballot_sync(peers, fresh) & peers;
      if (fresh) row[c] = found[next + __popc(m & ((1u << lane) - 1u))];
      next += __popc(m);
    }
  }
  if (some_held) team.sync();  // rows then have to see the tables
  for (int r = gtid; r < p.max_rows; r += NC * kPlanThreads) {
    int seq = -1, pos = -1;
    long long slot = -1;
    if (r < rows) {
      seq = seq_of_row(cu, p.num_seqs, r);
      const int start = cu[seq], j = r - start, held = p.a[seq], tok = held + j;
      int depth = j;
      if (p.mode != VA_MODE_CHAIN && extend_is_tree(p, seq)) {
        depth = 0;
        for (int u = p.parent[r]; u >= 0; u = p.parent[start + u]) ++depth;
      }
      pos = held + depth;
      const int c = tok / kPage, keep = (held + kPage - 1) / kPage;
      const int page = c >= keep && !some_held ? found[first[seq] + c - keep] : p.table[(long long)seq * p.max_blocks + c];
      slot = (long long)page * kPage + tok % kPage;
    }
    p.row_seq[r] = seq;
    p.position[r] = pos;
    p.slot[r] = slot;
  }
}

// Pull the live pages together: with N pages in use, the k-th page in use
// at or above N moves to the k-th hole below N.  Workspace: new place of
// each page [num_blocks].
template <int NC>
__global__ void __launch_bounds__(kPlanThreads) pages_compact_kernel(const PageParams p) {
  __shared__ PlanShared sh;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Team<NC> team;
  const int rank = team.rank();
  const int tid = threadIdx.x, lane = tid & 31, gwarp = rank * (kPlanThreads / 32) + tid / 32;
  const int gtid = rank * kPlanThreads + tid;
  if (tid == 0) sh.err = rank == 0 ? status_before(p) : 0u;
  team.sync();
  int lo, hi;
  warp_share<NC>(p.num_blocks, gwarp, &lo, &hi);
  unsigned livec = 0;
#pragma unroll 4
  for (int i = lo + lane; i < hi; i += 32) {
    const int r = p.ref[i];
    if (r < 0) note_error(team, sh, VA_DEV_BAD_BLOCK);
    livec += r > 0;
  }
  livec = warp_add(livec);
  const long long entries = (long long)p.num_seqs * p.max_blocks;
#pragma unroll 4
  for (long long i = gtid; i < entries; i += NC * kPlanThreads) {
    const int e = p.table[i];
    if (e != -1 && !page_in_use(p, e)) note_error(team, sh, VA_DEV_BAD_BLOCK);
  }
  share_count(team, sh, gwarp, lane, livec);
  team.sync();
  const unsigned err = read_error(team, sh);
  const int live = (int)sum_before(sh, (NC * kCtaWarps), lane);
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
    if (lane < NC) *team.at(&sh.below, lane) = (int)c;
  }
  team.sync();
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
  team.sync();
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
  team.sync();
#pragma unroll 4
  for (long long i = gtid; i < entries; i += NC * kPlanThreads) {
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

// grid = (CTAs per pool, pools): page pairs in turn, 16 bytes per thread, four
// loads in flight.  60 pages of 32 KB in 32 pools: 20 us, 6.2 TB/s read and
// written; 6,900 of 17 KB in 8 pools: 178 us, 6.1 TB/s.
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
  // Totals of fresh pages, token counts and loop counters stay within 32 bits.
  if (g->max_blocks_per_seq > (1 << 26)) return VA_ERR_UNSUPPORTED;
  if (g->num_blocks > (1 << 30) || g->num_seqs > (1 << 30)) return VA_ERR_UNSUPPORTED;
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
static cudaError_t launch_pages(void (*kernel)(const P), dim3 grid, int threads, int cluster, cudaStream_t st,
                                const P& q) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, q);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// One CTA or a cluster of eight, by the integers a plan goes through.
template <typename K>
static cudaError_t launch_plan(K one, K wide, long long ints, cudaStream_t st, const PageParams& q,
                               long long most = kOneCtaInts) {
  if (ints <= most) return launch_pages(one, dim3(1), kPlanThreads, 1, st, q);
  return launch_pages(wide, dim3(kWideCtas), kPlanThreads, kWideCtas, st, q);
}

// An extension's workspace: need and first page of each sequence, pages found.
static size_t extend_ws_bytes(const va_page_pool* g) {
  return (((size_t)g->num_seqs * 2 + (size_t)g->num_blocks) * 4 + 255) / 256 * 256;
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
  if (num_forks > (1 << 30)) return VA_ERR_UNSUPPORTED;
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
  cudaError_t e = launch_plan(pages_fork_kernel<1>, pages_fork_kernel<kWideCtas>,
                              pool->num_blocks + (long long)num_forks * pool->max_blocks_per_seq, cs, q);
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
  cudaError_t e = launch_plan(pages_free_kernel<1>, pages_free_kernel<kWideCtas>,
                              (long long)num_ranges * pool->max_blocks_per_seq, cs, q);
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
  cudaError_t e = launch_plan(pages_compact_kernel<1>, pages_compact_kernel<kWideCtas>,
                              pool->num_blocks + (long long)pool->num_seqs * pool->max_blocks_per_seq, cs, q);
  return e == cudaSuccess ? VA_OK : note_cuda(e);
}

size_t verify_attn_pages_extend_workspace_size(const va_page_pool* pool) {
  if (check_pool(pool) != VA_OK) return 0;
  return extend_ws_bytes(pool);
}

va_status verify_attn_pages_extend(const va_page_pool* pool, const va_extend* x, int32_t mode, int32_t* cu_rows,
                                   int32_t* row_seq, int32_t* position, int64_t* slot, void* ws, size_t ws_bytes,
                                   uint32_t* status, void* stream) {
  va_status st = check_pool(pool);
  if (st != VA_OK) return st;
  if (!x || mode < VA_MODE_CHAIN || mode > VA_MODE_MIXED) return VA_ERR_INVALID_ARG;
  if (!x->ctx_len || !x->rows || x->max_rows < 0 || !cu_rows) return VA_ERR_INVALID_ARG;
  if (x->max_rows > (1 << 30)) return VA_ERR_UNSUPPORTED;
  if (x->max_rows > 0 && (!row_seq || !position || !slot)) return VA_ERR_INVALID_ARG;
  if (mode != VA_MODE_CHAIN && x->max_rows > 0 && !x->parent) return VA_ERR_INVALID_ARG;
  if (mode == VA_MODE_MIXED && !x->seq_kind) return VA_ERR_INVALID_ARG;
  if ((uintptr_t)slot % 8) return VA_ERR_ALIGNMENT;
  cudaStream_t cs = (cudaStream_t)stream;
  st = check_plan(extend_ws_bytes(pool), ws, ws_bytes, cs);
  if (st != VA_OK) return st;
  PageParams q = page_params(pool, status);
  q.a = x->ctx_len;
  q.b = x->rows;
  q.ws = (int*)ws;
  q.mode = mode;
  q.max_rows = x->max_rows;
  q.parent = x->parent;
  q.kind = x->seq_kind;
  q.row_first = (int*)ws + pool->num_seqs + (size_t)pool->num_blocks;
  q.cu = cu_rows;
  q.row_seq = row_seq;
  q.position = position;
  q.slot = (long long*)slot;
  cudaError_t e = launch_plan(pages_extend_kernel<1>, pages_extend_kernel<kWideCtas>,
                              pool->num_blocks + 8LL * pool->num_seqs + 4LL * x->max_rows, cs, q, kOneCtaExtend);
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
    int per = (152 * 8 + m - 1) / m;  // eight CTAs to each of the GB300's 152 SMs
    if (per > max_copies) per = max_copies;
    cudaError_t e = launch_pages(pages_copy_kernel, dim3((unsigned)per, (unsigned)m), kCopyThreads, 1, cs, q);
    if (e != cudaSuccess) return note_cuda(e);
  }
  return VA_OK;
}

}  // extern "C"
