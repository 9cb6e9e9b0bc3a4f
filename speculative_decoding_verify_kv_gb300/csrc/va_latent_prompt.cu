// Tensor-core attention over expanded prompt keys, bf16: tcgen05 + TMEM + TMA, 128
// query rows of a head to a block.
//
// Per tile of 128 keys:
//   S = Q K^T     tcgen05.mma into one of two S buffers in TMEM
//   softmax       eight warps, one TMEM lane (query row) per thread and half of the
//                 tile's columns per warp; online (m, l) in log2 units, O rescaled
//                 only when the maximum grows by more than 2^8; P in bf16
//   O += P V      tcgen05.mma, A = P (TMEM), B = V tile (MN-major)
// so that S of the next tile runs under this tile's softmax.
//
// A CTA takes one block after the other: the one it was launched for, then blocks
// whose launch it takes over (clusterlaunchcontrol), asked for one ahead.  The
// warp that loads the keys finds out what a block is and tells the others, which
// go through the blocks by themselves: loads and S of the next run under the last
// softmax, P V and store of this one.
//
// Shared memory holds two rings of 64-column blocks of a tile: V stages of VBLK
// blocks, freed by P V, and single key blocks, freed as soon as S has read them.
// The first 128 query columns pass through the key ring to TMEM, the others stay in
// shared memory.
//
// Every wait is bounded (VA_DEV_TIMEOUT); on a timeout the CTA still goes through
// its blocks, writes NaN, drains its own copies and MMAs and frees TMEM.
#include <string.h>

#include "va_latent_mma.cuh"

namespace va {
using namespace sm100;

constexpr int kLqM = 128;
constexpr int kLqTile = 128;
constexpr int kLqThreads = 384;
constexpr int kLqWarps = kLqThreads / 32;

// One block of rows over one chunk of keys.  work: its tiles; 0: none of its rows
// sees a key; kLqSkip: no rows; kLqBad: offsets that make no sense; kLqEnd: no more.
enum { kLqSkip = -1, kLqBad = -2, kLqEnd = -3 };
struct LqItem {
  int row0, rbase, nrows, head;
  int live, ctx, lo;
  int hi, all_see, work, key0;
  int s;
  long long part;  // of the chunk's partials, see latent_part
};

template <int DK_, int DV_>
struct LqCfg {
  static constexpr int DK = DK_;                     // key width
  static constexpr int DV = DV_;                     // value width
  static constexpr int NT = kLqTile;                 // tokens per tile
  static constexpr int BLK = NT * 128;               // bytes of a 64-column block
  static constexpr int VBLK = DV / 64;               // blocks of a V stage
  static constexpr int KBLK = DK / 64;               // blocks of a key tile
  static constexpr int QT = 128;                     // query columns in TMEM
  static constexpr int QBLK = QT / 64;               // their blocks in the key ring
  static constexpr int QS = DK - QT;                 // query columns in shared memory
  static constexpr int NV = DV == 128 ? 2 : 4;       // V stages
  static constexpr int NK = DV == 128 ? 9 : 8;       // key blocks
  // P has columns of its own, so that S(i + 2) waits for S(i) to be read only, not
  // for P(i) V (in S's place: 750 us against 714 for 2 x 2,048 rows of 128 heads
  // over 4,096 keys).  Values of 64 columns take less time for P V than for the
  // wait before P is written: 668 us with, 633 without.
  static constexpr bool SEP = DV == 128;
  static constexpr int COL_O = 0;
  static constexpr int COL_S = DV;
  static constexpr int COL_P = COL_S + 2 * NT;
  static constexpr int COL_Q = COL_P + (SEP ? NT / 2 : 0);
  static constexpr int OFF_V = 0;
  static constexpr int OFF_K = NV * VBLK * BLK;
  static constexpr int OFF_Q = OFF_K + NK * BLK;
  static constexpr int OFF_RED = OFF_Q + QS / 64 * BLK;  // float [2][2][kLqM]
  static constexpr int OFF_NEXT = OFF_RED + 2 * 2 * kLqM * 4;
  static constexpr int OFF_ITEM = OFF_NEXT + 16;     // the block at work and the next
  static constexpr int NB = 19 + 2 * NV + 2 * NK;    // barriers
  static constexpr int OFF_MINE = OFF_ITEM + 2 * (int)sizeof(LqItem);  // of each softmax warp
  static constexpr int OFF_BAR = OFF_MINE + 8 * (int)sizeof(LqItem);
  static constexpr int SMEM = OFF_BAR + NB * 8 + 16;
  static_assert(BLK == kLqM * 128, "a query block in a key block's place");
  static_assert(COL_Q + QT / 2 <= 512, "TMEM columns");
  static_assert(SMEM <= 232448, "shared memory");
};

enum { QB_SFULL = 0, QB_PFULL = 2, QB_SFREE = 4, QB_QLAND = 6, QB_QREADY = 7, QB_QFREE = 8, QB_OFINAL = 9, QB_FIX = 10, QB_PFREE = 11,
       QB_SDRAIN = 12, QB_ODRAIN = 13, QB_NEXT = 14, QB_TOLD = 15, QB_TAKEN = 17, QB_RING = 19 };

struct LqMaps {
  CUtensorMap q, k, r;  // queries; expanded keys and values; rope part of the keys
};

__device__ __forceinline__ void bar_arrive(int id, int count) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// Asks for a block that has not been launched yet: 16 bytes, which the barrier counts.
__device__ __forceinline__ void ask_next(uint32_t dst, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(dst), "r"(bar)
               : "memory");
}
// The answer: false if there is none left.
__device__ __forceinline__ bool read_next(uint32_t src, int* x, int* y) {
  uint32_t ok, a = 0u, b = 0u;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\t.reg .b32 z;\n\t"
      "ld.shared.b128 h, [%3];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, %2, z, _}, h;\n\t}"
      : "=&r"(ok), "+r"(a), "+r"(b)
      : "r"(src)
      : "memory");
  *x = (int)a, *y = (int)b;
  return ok != 0u;
}

// Four pieces of four words in each of four lanes: lane i gets piece i of each.
__device__ __forceinline__ void deal4(uint32_t (&w)[16], int lane) {
#pragma unroll
  for (int d = 1; d < 4; d *= 2) {
    const bool high = lane & d;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      if (a & d) continue;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t &x = w[4 * a + k], &y = w[4 * (a | d) + k];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? x : y, d);
        if (high) x = got;
        else y = got;
      }
    }
  }
}

// What block x of a head is, found by a warp that goes through the sequences 32 at a
// time; false behind the last.  The grid has as many blocks as the rows can have at
// most, not as many a sequence as the longest may have, since one that is nothing
// costs 0.8 us (15 sequences of 256 rows, 128 heads, where 4,096 rows a sequence are
// allowed: 449 us by sequence, 142 so).  base, start: where the search stands, and
// the blocks before it.
__device__ __forceinline__ bool find_item(const LatentParams& p, int x, int* base, int* start, int lane, LqItem* it) {
  it->work = kLqSkip;
  if (x < *start) *base = *start = 0;
  for (; *base < p.num_seqs; *base += 32) {
    LatentSeq q;
    int b = 0;  // blocks of the lane's sequence; a bad one has one, that says so
    q.err = 0u, q.row0 = q.n = q.ctx = q.len = 0, q.key0 = 0;
    if (*base + lane < p.num_seqs) {
      q = latent_seq(p, *base + lane);
      b = q.err ? 1 : (q.n + kLqM - 1) / kLqM * latent_chunks(p, q.n);
    }
    int upto = b;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += v;
    }
    const int all = __shfl_sync(0xffffffffu, upto, 31);
    if (x - *start >= all) {
      *start += all;
      continue;
    }
    const int at = __ffs(__ballot_sync(0xffffffffu, upto > x - *start)) - 1;
    auto its = [&](int v) { return __shfl_sync(0xffffffffu, v, at); };
    const int place = x - *start - its(upto - b);
    q.err = (unsigned)its((int)q.err);
    q.row0 = its(q.row0), q.n = its(q.n), q.ctx = its(q.ctx), q.len = its(q.len), q.kind = 0;
    it->s = *base + at, it->key0 = its((int)q.key0);
    if (q.err) {
      it->work = kLqBad;
      return true;
    }
    const int blocks = (q.n + kLqM - 1) / kLqM, nchunk = latent_chunks(p, q.n);
    // A head's longest row blocks first: a few short ones end the launch (2 x 2,048
    // rows, 128 heads: 721 us in order, 714 so).
    const int rb = blocks - 1 - place % blocks, chunk = place / blocks;
    it->live = latent_live(p, q.len, nchunk);
    if (chunk >= it->live) return true;
    it->part = latent_part(p, *base + at, q.row0, q.n, chunk);
    it->row0 = q.row0, it->rbase = rb * kLqM, it->nrows = min(kLqM, q.n - it->rbase);
    it->ctx = q.ctx;
    int lo, hi;
    latent_range(p, q.len, nchunk, chunk, &lo, &hi);
    hi = max(lo, min(hi, latent_end(p, q, it->rbase + it->nrows - 1)));
    it->lo = lo, it->hi = hi;
    it->work = (hi - lo + kLqTile - 1) / kLqTile;
    // Keys below it are seen by every row of the block.
    it->all_see = p.causal ? min(hi, q.ctx + it->rbase + 1) : hi;
    return true;
  }
  return false;
}

// What a block without work has of outputs, by thread t of 256.  (Not inlined: it
// is rare, and its divisions cost the loop over the tiles registers.)
template <int DV>
__device__ __noinline__ void no_work(const LatentParams& p, const LqItem& it, int t) {
  if (it.work == kLqBad) {
    if (t == 0) flag(p.status, VA_DEV_BAD_ROWS);
    latent_nan_rows(p, it.s, it.head, 1, t, 256);  // its one block
  } else if (it.work == 0) {
    // A chunk that the block's rows see nothing of, or no keys.
    for (int u = t; u < it.nrows * DV; u += 256) {
      const long long i = latent_item(p, it.row0, it.rbase + u / DV, it.head);
      const int d = u % DV;
      if (it.live > 1) {
        if (d == 0) {
          const long long si = it.part + i;
          p.ws_ml[2 * si] = -INFINITY;
          p.ws_ml[2 * si + 1] = 0.f;
        }
      } else {
        reinterpret_cast<unsigned short*>(p.o)[i * DV + d] = 0u;
        if (d == 0) p.lse[i] = -INFINITY;
      }
    }
  }
}

// A finished block's rows: row r (TMEM lane), half of O's columns.
//
// O: fp32 sums for the merge, or the finished bf16 row.  Four lanes exchange their
// rows' 16-byte pieces, so that a store writes 64 bytes of a row, not 16.
template <int DV>
__device__ __forceinline__ void store_rows(const LatentParams& p, const LqItem& was, uint32_t col, int r, int half, float m_use, float l, bool bad) {
  const int lane = threadIdx.x & 31;
  const float inv = bad ? NAN : l != 0.f ? 1.f / l : 0.f;
  const long long at = latent_item(p, was.row0, was.rbase + r, was.head);
  const long long slot = was.part + at;
  if (r < was.nrows && half == 0) {
    if (was.live > 1) {
      p.ws_ml[2 * slot] = bad ? NAN : m_use;
      p.ws_ml[2 * slot + 1] = bad ? NAN : l;
    } else {
      p.lse[at] = bad ? NAN : l != 0.f ? (m_use + log2f(l)) * kLn2 : -INFINITY;
    }
  }
  const long long at4 = __shfl_sync(0xffffffffu, was.live > 1 ? slot : at, lane & 28), step4 = p.H;
  const int left4 = was.nrows - (r & ~3);  // rows of the four lanes
  if (r - lane >= was.nrows) return;
#pragma unroll 1
  for (int c0 = half * (DV / 2); c0 < (half + 1) * (DV / 2); c0 += 32) {
    uint32_t o[32];
    tmem_ld32(col + c0, o);
    tmem_wait_ld();
    if (was.live > 1) {
      float* to = p.ws_acc + at4 * DV + c0 + (lane & 3) * 4;
#pragma unroll
      for (int c = 0; c < 32; c += 16) {
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) w[k] = bad ? 0x7fffffffu : o[c + k];
        deal4(w, lane);
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (t < left4) *reinterpret_cast<uint4*>(to + t * step4 * DV + c) = make_uint4(w[4 * t], w[4 * t + 1], w[4 * t + 2], w[4 * t + 3]);
      }
    } else {
      uint32_t w[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        // A row that sees nothing has no sum (its lanes of O may hold anything).
        const __nv_bfloat162 h = l != 0.f || bad ? __floats2bfloat162_rn(__uint_as_float(o[2 * c]) * inv, __uint_as_float(o[2 * c + 1]) * inv)
                                                : __floats2bfloat162_rn(0.f, 0.f);
        w[c] = *reinterpret_cast<const uint32_t*>(&h);
      }
      deal4(w, lane);
      unsigned short* to = reinterpret_cast<unsigned short*>(p.o) + at4 * DV + c0 + (lane & 3) * 8;
#pragma unroll
      for (int t = 0; t < 4; ++t)
        if (t < left4) *reinterpret_cast<uint4*>(to + t * step4 * DV) = make_uint4(w[4 * t], w[4 * t + 1], w[4 * t + 2], w[4 * t + 3]);
    }
  }
}

template <class C>
__global__ void __launch_bounds__(kLqThreads, 1) latent_prompt_kernel(const __grid_constant__ LatentParams p,
                                                                      const __grid_constant__ LqMaps maps) {
  constexpr int NT = C::NT, NC = NT / 2, DV = C::DV;
  extern __shared__ __align__(1024) unsigned char sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  float* red = reinterpret_cast<float*>(sm + C::OFF_RED);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(sm + C::OFF_BAR + C::NB * 8);
  volatile int* abort_p = reinterpret_cast<volatile int*>(tmem_at + 1);

  asm volatile("griddepcontrol.launch_dependents;");
  // Broadcasts: what a warp has in common is known to be so.
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  if (warp == 0) {
    if (lane == 0) {
      *abort_p = 0;
      prefetch_map(&maps.q);
      prefetch_map(&maps.k);
      prefetch_map(&maps.r);
    }
    for (int i = lane; i < C::NB; i += 32)
      mbar_init(bar(i), (i >= QB_TAKEN && i < QB_RING) ? kLqWarps - 1
                        : (i >= QB_PFULL && i < QB_SFREE) || (C::SEP && i >= QB_SFREE && i < QB_QLAND) || i == QB_QREADY ? 8 : 1);
    fence_barrier_init();
    __syncwarp();
  }
  // Nothing but this CTA's own shared memory is touched before the work ahead
  // on the stream has completed.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_at), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  // The barriers' and TMEM's set-up.  Warp 0 needs nothing of it but its own.
  if (warp == 0) bar_arrive(2, kLqThreads);
  else bar_sync(2, kLqThreads);
  tc_fence_after();
  const uint32_t tm = warp == 0 ? 0u : __shfl_sync(0xffffffffu, *tmem_at, 0);

  auto vfull = [&](int i) { return bar(QB_RING + i); };
  auto vfree = [&](int i) { return bar(QB_RING + C::NV + i); };
  auto kfull = [&](int i) { return bar(QB_RING + 2 * C::NV + i); };
  auto kfree = [&](int i) { return bar(QB_RING + 2 * C::NV + C::NK + i); };
  const uint32_t base = smem_u32(sm);
  auto fail = [&]() {
    *abort_p = 1;
    flag(p.status, VA_DEV_TIMEOUT);
  };
  auto drain = [&](uint32_t b, uint32_t parity) {
    int dummy = 0;
    return mbar_wait(b, parity, &dummy, kLatentWaitNs);
  };

  // A warp's way through the CTA's blocks: the next that the first warp tells of.
  // Those without work are the outputs' (empty) matter.
  LqItem* items_s = reinterpret_cast<LqItem*>(sm + C::OFF_ITEM);
  int told = 0;
  auto next_item = [&](LqItem* it, auto empty) {
    for (;;) {
      const int n = told & 1;
      if (!__all_sync(0xffffffffu, drain(bar(QB_TOLD + n), (told >> 1) & 1))) {
        if (lane == 0) fail();
        return false;
      }
      const int work = __shfl_sync(0xffffffffu, items_s[n].work, 0);
      if (work > 0) *it = items_s[n];
      else empty(items_s[n]);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(QB_TAKEN + n));
      ++told;
      if (work == kLqEnd) return false;
      if (work > 0) break;
    }
    // What a warp has in common is known to be so.
    auto same = [&](int& v) { v = __shfl_sync(0xffffffffu, v, 0); };
    same(it->row0), same(it->rbase), same(it->nrows), same(it->head), same(it->live);
    same(it->ctx), same(it->lo), same(it->hi), same(it->all_see), same(it->work), same(it->key0);
    return true;
  };
  auto nothing = [](const LqItem&) {};

  if (warp == 0) {
    // ---------------------------------------------------------------- keys, queries
    const uint32_t one = elected();
    bool ok = true;
    int issued = 0, items = 0;  // blocks of the ring; row blocks with work
    int st = 0, x = blockIdx.x, head = blockIdx.y, base_s = 0, start = 0, asks = 0;
    uint32_t par = 1;
    for (bool more = true; more; ++told) {
      LqItem it;
      const int n = told & 1;
      const bool there = find_item(p, x, &base_s, &start, lane, &it);
      // Sequences of bad offsets may leave more blocks than the grid has: the last
      // block goes on with those.
      const bool on = __shfl_sync(0xffffffffu, there && x >= (int)gridDim.x - 1 ? 1 : 0, 0) != 0;
      it.head = head;
      it.work = __shfl_sync(0xffffffffu, it.work, 0), it.lo = __shfl_sync(0xffffffffu, it.lo, 0), it.key0 = __shfl_sync(0xffffffffu, it.key0, 0);
      it.row0 = __shfl_sync(0xffffffffu, it.row0, 0), it.rbase = __shfl_sync(0xffffffffu, it.rbase, 0);
      if (told >= 2 && !__all_sync(0xffffffffu, drain(bar(QB_TAKEN + n), ((told >> 1) - 1) & 1)) && lane == 0) fail();
      if (lane == 0) {
        items_s[n] = it;
        mbar_arrive(bar(QB_TOLD + n));
        if (!on) {
          mbar_arrive_expect_tx(bar(QB_NEXT), 16);
          ask_next(base + C::OFF_NEXT, bar(QB_NEXT));
        }
      }
      __syncwarp();
      if (it.work > 0 && ok) {
        if (C::QS > 0) {
          ok = __all_sync(0xffffffffu, items == 0 || mbar_wait(bar(QB_QFREE), (items - 1) & 1, abort_p, kLatentWaitNs));
          if (ok) {
            expect_by(one, bar(QB_QLAND), C::QS / 64 * C::BLK);
#pragma unroll
            for (int c = C::QBLK; c < C::KBLK; ++c)
              tma_3d_by(one, base + C::OFF_Q + (c - C::QBLK) * C::BLK, &maps.q, c * 64, head, it.row0 + it.rbase, bar(QB_QLAND));
          }
        }
        if (ok) ++items;
        for (int i = -1; i < it.work && ok; ++i) {
          const int key = it.key0 + it.lo + i * NT;
#pragma unroll
          for (int c = 0; c < C::KBLK; ++c) {
            if (i < 0 && c >= C::QBLK) break;
            ok = __all_sync(0xffffffffu, ok && mbar_wait(kfree(st), par, abort_p, kLatentWaitNs));
            if (!ok) break;
            const uint32_t dst = base + C::OFF_K + st * C::BLK, b = kfull(st);
            expect_by(one, b, C::BLK);
            if (i < 0) tma_3d_by(one, dst, &maps.q, c * 64, head, it.row0 + it.rbase, b);
            else if (c == C::KBLK - 1) tma_2d_by(one, dst, &maps.r, 0, key, b);
            else tma_3d_by(one, dst, &maps.k, c * 64, head, key, b);
            ++issued;
            if (++st == C::NK) st = 0, par ^= 1;
          }
        }
        if (!ok && lane == 0) fail();
      }
      if (on) {
        ++x;
        continue;
      }
      more = __all_sync(0xffffffffu, drain(bar(QB_NEXT), asks & 1));
      ++asks;
      if (!more && lane == 0) fail();
      if (more) {
        more = read_next(base + C::OFF_NEXT, &x, &head);
        fence_proxy_async_smem();  // the place will be written again
        __syncwarp();
        more = __shfl_sync(0xffffffffu, more ? 1 : 0, 0) != 0;
        x = __shfl_sync(0xffffffffu, x, 0), head = __shfl_sync(0xffffffffu, head, 0);
      }
    }
    const int n = told & 1;
    if (told >= 2 && !__all_sync(0xffffffffu, drain(bar(QB_TAKEN + n), ((told >> 1) - 1) & 1)) && lane == 0) fail();
    if (lane == 0) {
      items_s[n].work = kLqEnd;
      mbar_arrive(bar(QB_TOLD + n));
    }
    // No copy may still be landing when the CTA goes away.
    if (*abort_p && lane == 0) {
      if (C::QS > 0 && items > 0) drain(bar(QB_QLAND), (items - 1) & 1);
      for (int i = max(0, issued - C::NK); i < issued; ++i) drain(kfull(i % C::NK), (i / C::NK) & 1);
    }
  } else if (warp == 10) {
    // ---------------------------------------------------------------- values
    const uint32_t one = elected();
    bool ok = true;
    int issued = 0, st = 0, fixed = -1;  // stages; the last one cleared
    uint32_t par = 1;
    for (LqItem it; next_item(&it, nothing);) {
      if (ok) {
        for (int i = 0; i < it.work; ++i) {
          ok = __all_sync(0xffffffffu, mbar_wait(vfree(st), par, abort_p, kLatentWaitNs));
          if (!ok) break;
          const uint32_t dst = base + C::OFF_V + st * C::VBLK * C::BLK, b = vfull(st);
          expect_by(one, b, C::VBLK * C::BLK);
#pragma unroll
          for (int c = 0; c < C::VBLK; ++c)
            tma_3d_by(one, dst + c * C::BLK, &maps.k, C::DK - kLatentRope + c * 64, it.head, it.key0 + it.lo + i * NT, b);
          ++issued;
          if (++st == C::NV) st = 0, par ^= 1;
        }
        const int valid = it.hi - it.lo - (it.work - 1) * NT;
        if (ok && valid < NT) {
          // Keys behind the range may hold anything: their V is cleared (their
          // scores are masked).
          const int last = (issued - 1) % C::NV;
          ok = mbar_wait(vfull(last), ((issued - 1) / C::NV) & 1, abort_p, kLatentWaitNs);
          // One clearing is told at a time: the last one's stage has been used (if
          // its place was loaded again, that was waited for).
          if (fixed >= 0 && issued - fixed <= C::NV)
            ok = ok && mbar_wait(vfree(fixed % C::NV), (fixed / C::NV) & 1, abort_p, kLatentWaitNs);
          fixed = issued - 1;
          ok = __all_sync(0xffffffffu, ok);
          if (ok) {
            for (int c = 0; c < C::VBLK; ++c) clear_rows(sm + C::OFF_V + (last * C::VBLK + c) * C::BLK, valid, NT, lane);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(QB_FIX));
          }
        }
        if (!ok && lane == 0) fail();
      }
    }
    if (*abort_p && lane == 0)
      for (int i = max(0, issued - C::NV); i < issued; ++i) drain(vfull(i % C::NV), (i / C::NV) & 1);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- S issuer
    constexpr uint32_t ID = idesc_f16(kLqM, NT, true, false);
    const uint32_t one = elected();
    bool ok = true, any = false;
    int sk = 0, items = 0, g = 0;  // key block, blocks with work, tiles
    uint32_t pk = 0;               // its parity
    const uint64_t kd0 = sdesc_sw128(base + C::OFF_K, 16, 1024), qd0 = sdesc_sw128(base + C::OFF_Q, 16, 1024);
    for (LqItem it; next_item(&it, nothing);) {
      if (ok) {
        ok = (C::QS == 0 || mbar_wait(bar(QB_QLAND), items & 1, abort_p, kLatentWaitNs)) &&
             mbar_wait(bar(QB_QREADY), items & 1, abort_p, kLatentWaitNs);
        ok = __all_sync(0xffffffffu, ok);
        ++items;
        if (ok) {
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < C::QBLK; ++c) {
            if (lane == 0) mbar_arrive(kfree(sk));
            if (++sk == C::NK) sk = 0, pk ^= 1;
          }
        }
        bool there = false;
        for (int i = 0; i < it.work && ok; ++i, ++g) {
          const int b = g & 1;
          const uint32_t scol = tm + C::COL_S + b * NT;
          ok = there || ((g < 2 || mbar_wait(bar(QB_SFREE + b), ((g - 2) >> 1) & 1, abort_p, kLatentWaitNs)) &&
                         mbar_wait(kfull(sk), pk, abort_p, kLatentWaitNs));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < C::KBLK; ++c) {
            if (c > 0) {
              ok = __all_sync(0xffffffffu, there || mbar_wait(kfull(sk), pk, abort_p, kLatentWaitNs));
              if (!ok) break;
              tc_fence_after();
            }
            const uint64_t kd = kd0 + (uint64_t)((sk * C::BLK) >> 4);
            const uint32_t free = kfree(sk);
            if (++sk == C::NK) sk = 0, pk ^= 1;
            // What the next tile starts with: its S buffer free and its first block there.
            there = c + 1 < C::KBLK ? mbar_peek(kfull(sk), pk)
                                    : i + 1 < it.work && (g < 1 || mbar_peek(bar(QB_SFREE + (b ^ 1)), ((g - 1) >> 1) & 1)) &&
                                          mbar_peek(kfull(sk), pk);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (c < C::QBLK) mma_ts_by(one, scol, tm + C::COL_Q + (c * 4 + kk) * 8, kd + kk * 2, ID, c > 0 || kk > 0 ? 1u : 0u);
              else mma_ss_by(one, scol, qd0 + (uint64_t)(((c - C::QBLK) * C::BLK) >> 4) + kk * 2, kd + kk * 2, ID, 1u);
            }
            any = true;
            commit_by(one, free);
          }
          if (!ok) break;
          commit_by(one, bar(QB_SFULL + b));
        }
        if (ok) commit_by(one, bar(QB_QFREE));
        else if (lane == 0) fail();
      }
    }
    // What was issued completes before TMEM and shared memory go.
    if (any) {
      commit_by(one, bar(QB_SDRAIN));
      drain(bar(QB_SDRAIN), 0);
    }
  } else if (warp == 11) {
    // ---------------------------------------------------------------- P.V issuer
    constexpr uint32_t ID = idesc_f16(kLqM, DV, true, true);
    const uint32_t one = elected();
    bool ok = true, any = false;
    int st = 0, g = 0, fixes = 0;  // V stage, tiles, ragged blocks
    uint32_t pv = 0;
    const uint64_t vd0 = sdesc_sw128(base + C::OFF_V, C::BLK, 1024);
    for (LqItem it; next_item(&it, nothing);) {
      if (ok) {
        const bool ragged = (it.hi - it.lo) % NT != 0;  // of the last tile
        for (int i = 0; i < it.work; ++i, ++g) {
          const int b = g & 1;
          ok = mbar_wait(bar(QB_PFULL + b), (g >> 1) & 1, abort_p, kLatentWaitNs) && mbar_wait(vfull(st), pv, abort_p, kLatentWaitNs) &&
               (i < it.work - 1 || !ragged || mbar_wait(bar(QB_FIX), fixes & 1, abort_p, kLatentWaitNs));
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = vd0 + (uint64_t)((st * C::VBLK * C::BLK) >> 4);
#pragma unroll
          for (int kk = 0; kk < NT / 16; ++kk)
            mma_ts_by(one, tm + C::COL_O, tm + (C::SEP ? C::COL_P : C::COL_S + b * NT) + kk * 8, vd + (uint64_t)((kk * 2048) >> 4), ID,
                      i > 0 || kk > 0 ? 1u : 0u);
          any = true;
          commit_by(one, bar(C::SEP ? QB_PFREE : QB_SFREE + b));
          commit_by(one, vfree(st));
          if (++st == C::NV) st = 0, pv ^= 1;
        }
        fixes += ragged ? 1 : 0;
        if (ok) commit_by(one, bar(QB_OFINAL));
        else if (lane == 0) fail();
      }
    }
    if (any) {
      commit_by(one, bar(QB_ODRAIN));
      drain(bar(QB_ODRAIN), 0);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const int r = quad * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const float c_r = p.scale_log2;
    bool ok = true;
    int sk = 0, g = 0, items = 0;  // key block, tiles, blocks with work
    uint32_t pk = 0;
    // The next block with work, its queries on the way to TMEM.
    auto advance = [&](LqItem* it) {
      if (!next_item(it, [&](const LqItem& e) { no_work<DV>(p, e, tid - 64); })) return false;
      // Both halves: 16-byte pieces of a swizzled block each.  (Rows behind the
      // block's last hold other rows, or zeros: no one reads what comes of them.)
      static_assert(C::QBLK == 2, "a block to a half");
      const int at = sk + half < C::NK ? sk + half : sk + half - C::NK;
      const uint32_t par = sk + half < C::NK ? pk : pk ^ 1;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(kfull(at), par, abort_p, kLatentWaitNs));
      if (ok) {
#pragma unroll 1
        for (int c0 = 0; c0 < 8; c0 += 4) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 v = *reinterpret_cast<const uint4*>(sm + C::OFF_K + at * C::BLK + r * 128 + (((c0 + k) ^ (r & 7)) << 4));
            w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
          }
          tmem_st16(tm + lanes + C::COL_Q + half * 32 + c0 * 4, w);
        }
        tmem_wait_st();
        // Copies will write where these reads were.
        fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(QB_QREADY));
      sk += C::QBLK + it->work * C::KBLK;
      pk ^= (uint32_t)(sk / C::NK) & 1u;
      sk %= C::NK;
      return true;
    };

    LqItem it;
    bool have = advance(&it);
    // What a block's rows are is kept in shared memory while the tiles are at work.
    LqItem* mine = reinterpret_cast<LqItem*>(sm + C::OFF_MINE) + (warp - 2);
    auto keep = [&]() {
      __syncwarp();
      if (lane == 0) mine->row0 = it.row0, mine->rbase = it.rbase, mine->nrows = it.nrows, mine->head = it.head, mine->part = it.part, mine->live = it.live;
      __syncwarp();
    };
    keep();
    while (have) {
      const bool rvalid = r < it.nrows, warp_live = quad * 32 < it.nrows;
      // Keys below it are seen by this row.
      const int see = !rvalid ? 0 : p.causal ? min(it.hi, it.ctx + it.rbase + r + 1) : it.hi;
      float m_use = -INFINITY, l_run = 0.f;
      bool there = false;  // S of the tile, seen ahead
      // A failed wait does not leave the loop: every iteration has one named
      // barrier shared with the partner warp.
      for (int i = 0; i < it.work; ++i, ++g) {
        const int b = g & 1;
        if (ok && !__all_sync(0xffffffffu, there || mbar_wait(bar(QB_SFULL + b), (g >> 1) & 1, abort_p, kLatentWaitNs))) ok = false;
        tc_fence_after();
        const uint32_t scol = tm + lanes + C::COL_S + b * NT;
        float sv[NC];
        float mx = -INFINITY;
        if (ok && warp_live) {
          uint32_t sr[NC];
          tmem_ld32_into<0>(scol + NC * half, sr);
          tmem_ld32_into<32>(scol + NC * half + 32, sr);
          tmem_wait_ld();
          if (it.lo + (i + 1) * NT <= it.all_see) {
            float m2 = -INFINITY;
#pragma unroll
            for (int c = 0; c < NC; c += 4) {
              mx = max3(mx, __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
              m2 = max3(m2, __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
            }
            mx = fmaxf(mx, m2);
#pragma unroll
            for (int c = 0; c < NC; ++c) sv[c] = __uint_as_float(sr[c]);
          } else {
            const int left = see - (it.lo + i * NT + NC * half);
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              sv[c] = c < left ? __uint_as_float(sr[c]) : -INFINITY;
              mx = fmaxf(mx, sv[c]);
            }
          }
        }
        if (C::SEP) {
          // S(i) is in registers: its buffer may be written again.
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(QB_SFREE + b));
        }
        // The previous P.V: it has to be done before O is rescaled, or (SEP) P
        // written; warps without rows wait for it too, or they would tell of tile
        // i + 2's P before the others do of tile i's.
        auto pv_done = [&]() {
          return i < 1 || (C::SEP ? mbar_wait(bar(QB_PFREE), (g - 1) & 1, abort_p, kLatentWaitNs)
                                  : mbar_wait(bar(QB_SFREE + (b ^ 1)), ((g - 1) >> 1) & 1, abort_p, kLatentWaitNs));
        };
        // The row's maximum over both halves (raw scores; c_r > 0).
        red[(b * 2 + half) * kLqM + r] = mx;
        bar_sync(5 + quad, 64);
        mx = fmaxf(mx, red[(b * 2 + (half ^ 1)) * kLqM + r]);
        const float mt = mx * c_r;
        const bool need = rvalid && m_use != -INFINITY && mt > m_use + 8.f;
        const float m_new = m_use == -INFINITY || need ? mt : m_use;
        if (ok && __any_sync(0xffffffffu, need)) {
          // Rescale this half of the warp's O rows once the previous P.V landed.
          if (!__all_sync(0xffffffffu, pv_done())) ok = false;
          if (ok) {
            tc_fence_after();
            const float f = need ? exp2f(m_use - m_new) : 1.f;
#pragma unroll 1
            for (int c0 = half * (DV / 2); c0 < (half + 1) * (DV / 2); c0 += 16) {
              uint32_t o[16];
              tmem_ld16(tm + lanes + C::COL_O + c0, o);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f);
              tmem_st16(tm + lanes + C::COL_O + c0, o);
            }
            tmem_wait_st();
            l_run *= f;
          }
        }
        m_use = m_new;
        there = i + 1 < it.work && mbar_peek(bar(QB_SFULL + (b ^ 1)), ((g + 1) >> 1) & 1);
        if (ok && warp_live) {
          uint32_t ph[NC / 2];
          uint64_t l2 = pack2(0.f, 0.f);
          // A masked score (-inf) gives 0; while nothing of the row was visible
          // every score is masked, and the 0 offset keeps them at -inf.
          const float mneg = m_use == -INFINITY ? 0.f : -m_use;
          const uint64_t c2 = pack2(c_r, c_r), m2 = pack2(mneg, mneg);
#pragma unroll
          for (int c = 0; c < NC / 2; ++c) {
            float a, d;
            unpack2(fma2(pack2(sv[2 * c], sv[2 * c + 1]), c2, m2), a, d);
            a = lu_ex2(a);
            d = lu_ex2(d);
            l2 = add2(l2, pack2(a, d));
            // Rounded to bf16 (2^-8 at most): the matrix unit takes 16 bits, and
            // a second part for the rest would cost P.V again, for an o that is
            // rounded alike.
            const __nv_bfloat162 h = __floats2bfloat162_rn(a, d);
            ph[c] = *reinterpret_cast<const uint32_t*>(&h);
          }
          float l0, l1;
          unpack2(l2, l0, l1);
          l_run += l0 + l1;
          if (C::SEP && !__all_sync(0xffffffffu, pv_done())) ok = false;
          if (C::SEP) tc_fence_after();
          tmem_st32_from<0>((C::SEP ? tm + lanes + C::COL_P : scol) + 32 * half, ph);
          tmem_wait_st();
        } else if (C::SEP && ok) {
          if (!__all_sync(0xffffffffu, pv_done())) ok = false;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(QB_PFULL + b));
      }

      // S has read this block's queries: the next one's, before this one's store.
      // (Every S of the block was waited for.)
      have = advance(&it);
      if (ok && !__all_sync(0xffffffffu, mbar_wait(bar(QB_OFINAL), items & 1, abort_p, kLatentWaitNs))) ok = false;
      ++items;
      if (!ok && lane == 0) fail();
      tc_fence_after();
      float* lsum = red + (g & 1) * 2 * kLqM;
      lsum[half * kLqM + r] = l_run;
      bar_sync(5 + quad, 64);
      const float l = lsum[r] + lsum[kLqM + r];
      bar_sync(5 + quad, 64);  // the next block's first tile writes there
      const bool bad = __any_sync(0xffffffffu, !ok || *abort_p != 0);
      store_rows<DV>(p, *mine, tm + lanes + C::COL_O, r, half, m_use, l, bad);
      keep();
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*abort_p) settle();
  if (warp == 1) tmem_dealloc(tm, 512);
}

// ---------------------------------------------------------------------------
static bool lq_maps(LqMaps* m, const LatentParams& p, int tile) {
  memset(m, 0, sizeof(*m));
  const cuuint64_t dk = (cuuint64_t)p.DK, H = (cuuint64_t)p.H;
  const cuuint64_t qd[3] = {dk, H, (cuuint64_t)p.total_rows}, qs[2] = {dk * 2, H * dk * 2};
  const cuuint32_t qb[3] = {64, 1, kLqM}, kb[3] = {64, 1, (cuuint32_t)tile}, rb[2] = {64, (cuuint32_t)tile};
  if (!latent_map(&m->q, p.q, 3, qd, qs, qb)) return false;
  if (p.total_kv == 0) return true;  // no tile, no load
  const cuuint64_t w = dk - kLatentRope + (cuuint64_t)p.DV, T = (cuuint64_t)p.total_kv;
  const cuuint64_t kd[3] = {w, H, T}, ks[2] = {w * 2, H * w * 2};
  const cuuint64_t rd[2] = {kLatentRope, T}, rs[1] = {(cuuint64_t)(T > 1 ? p.kr_stride : kLatentRope) * 2};
  return latent_map(&m->k, p.kv, 3, kd, ks, kb) && latent_map(&m->r, p.k_rope, 2, rd, rs, rb);
}

template <class C>
static cudaError_t launch_prompt_of(const LatentParams& p, dim3 grid, cudaStream_t st) {
  static std::atomic<unsigned long long> ready{0ull};
  cudaError_t e = allow_smem(latent_prompt_kernel<C>, C::SMEM, ready);
  if (e != cudaSuccess) return e;
  LqMaps m;
  if (!lq_maps(&m, p, C::NT)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kLqThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, latent_prompt_kernel<C>, p, m);
  return e != cudaSuccess ? e : cudaGetLastError();
}

int latent_prompt_rows() { return kLqM; }

cudaError_t launch_latent_prompt(const LatentParams& p, dim3 grid, cudaStream_t st) {
  return p.DV == 128 ? launch_prompt_of<LqCfg<192, 128>>(p, grid, st) : launch_prompt_of<LqCfg<128, 64>>(p, grid, st);
}

}  // namespace va
