// Tensor-core attention over latent caches of 512 columns, bf16, more than 32
// query rows: 128 rows to a pair of CTAs (cta_group::2), 64 in each.
//
// O of 128 rows x 512 columns is all of one SM's TMEM, so the rows are dealt to
// two.  A product over both (M = 128, issued by the first CTA) has each CTA's own
// 64 rows of A and D and half of B's columns, and D's columns folded: lanes 0 to
// 63 hold a row's first half, lanes 64 to 127 its second.  So S of 64 rows x 128
// tokens takes 64 TMEM columns, O 256, and each product is done once (with O's
// columns dealt to two CTAs instead, as in the 128-row kernel, both compute S:
// 832 multiply-adds to a row and token of each where 544 do).
//
// Per tile of 128 tokens:
//   S = Q C^T    A = Q (shared memory), B = the key's nine column blocks, each CTA
//                holding its 64 tokens
//   softmax      eight warps: a row has four threads, by half of the tile and half
//                of that; online (m, l) in log2 units, O rescaled only when the
//                maximum grows by more than 2^8; P (bf16) to shared memory
//   O += P V     A = P, B = the value columns, each CTA holding half of them for
//                all 128 tokens: two products of 256 columns
//
// Shared memory: queries, P, and a tile: three groups of key blocks and four units
// of V, each loaded again as soon as it has been read, key groups while the
// softmax and P.V are at work, V during S.
//
// Waits are bounded (VA_DEV_TIMEOUT); on a timeout the pair ends and writes NaN.
#include <string.h>

#include "va_latent_mma.cuh"

namespace va {

constexpr int kLpThreads = 448;  // 8 softmax warps, 2 + 2 producers, 2 issuers
constexpr int kLpRows = 64;    // of a CTA
constexpr int kLpTile = 128;

struct LpCfg {
  static constexpr int DV = 512, DK = DV + kLatentRope;
  static constexpr int KB = kLpTile / 2 * 128;      // a 64-column key block: this CTA's 64 tokens
  static constexpr int KG = 3;                      // blocks to a barrier
  static constexpr int KU = DK / 64 / KG;           // groups of a tile, and of the ring
  static constexpr int VB = kLpTile / 2 * 128;      // a 64-column value block: half of the tokens
  static constexpr int VG = 2;                      // blocks of this CTA's half of 256 columns
  static constexpr int VU = DV / 256 * 2;           // such units of a tile, and of the ring: (columns, tokens)
  static constexpr int QB = kLpRows * 128;
  static constexpr int PB = kLpRows * 128;          // P of 64 tokens
  static constexpr int OFF_V = 0;
  static constexpr int OFF_K = VU * VG * VB;
  static constexpr int OFF_Q = OFF_K + KU * KG * KB;
  static constexpr int OFF_P = OFF_Q + DK / 64 * QB;
  static constexpr int OFF_END = OFF_P + 2 * PB;
  static constexpr int OROW = DV * 4 + 16;          // O staging at the end, padded rows
  static constexpr int OFF_RED = OFF_END;           // float [2][4][64]
  static constexpr int NB = 16 + 2 * VU + 2 * KU;
  static constexpr int OFF_BAR = OFF_RED + 2 * 4 * kLpRows * 4;
  static constexpr int SMEM = OFF_BAR + NB * 8 + 16;
  static constexpr int COL_O = 0, COL_S = 256;      // two S buffers of 64 columns
  static_assert(kLpRows * OROW <= OFF_END, "O staging");
  static_assert(SMEM <= 232448, "shared memory");
};

enum { PB_SFULL = 0, PB_SREAD = 2, PB_PFULL = 4, PB_PFREE = 5, PB_QLAND = 6, PB_QALL = 7, PB_OFINAL = 8, PB_FIX = 9,
       PB_SDRAIN = 10, PB_VLAST = 11, PB_RING = 16 };

struct LpMaps {
  CUtensorMap q, k;
};

__global__ void __launch_bounds__(kLpThreads, 1) latent_pair_kernel(const LatentParams p, const __grid_constant__ LpMaps maps) {
  using C = LpCfg;
  extern __shared__ __align__(1024) unsigned char sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  float* red = reinterpret_cast<float*>(sm + C::OFF_RED);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(sm + C::OFF_BAR + C::NB * 8);
  volatile int* abort_p = reinterpret_cast<volatile int*>(tmem_at + 1);
  int* err_s = reinterpret_cast<int*>(tmem_at + 2);

  asm volatile("griddepcontrol.launch_dependents;");
  // Broadcasts: what a warp has in common is known to be so.
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rank = blockIdx.x & 1;  // in the pair
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  if (warp == 0) {
    if (lane == 0) {
      *err_s = 0;
      *abort_p = 0;
      prefetch_map(&maps.q);
      prefetch_map(&maps.k);
    }
    for (int i = lane; i < C::NB; i += 32)
      mbar_init(bar(i), (i >= PB_SREAD && i <= PB_PFULL) ? 16 : i == PB_FIX ? 4 : i == PB_QALL ? 2 : 1);
    fence_barrier_init();
    __syncwarp();
  }
  // Nothing but this CTA's own shared memory is touched before the work ahead
  // on the stream has completed.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int s = blockIdx.z;
  const LatentSeq q = latent_seq(p, s);
  if (q.err & VA_DEV_BAD_ROWS) {
    if (tid == 0) flag(p.status, q.err);
    if (blockIdx.x == 0) latent_nan_rows(p, s, 0, p.H, threadIdx.x, blockDim.x);
    return;
  }
  const int R = latent_rows(p, q.n);
  const int blocks = (R + 2 * kLpRows - 1) / (2 * kLpRows);
  if (blocks == 0) return;
  const int nchunk = latent_chunks(p, q.n);
  const int pair = blockIdx.x >> 1, rb = pair % blocks, chunk = pair / blocks;
  const int live = latent_live(p, q.err ? 0 : q.len, nchunk);
  if (chunk >= live) return;
  // (The second CTA may have no rows; it then holds its half of keys and values
  // all the same.)
  const int rpair = rb * 2 * kLpRows, rbase = rpair + rank * kLpRows, nrows = max(0, min(kLpRows, R - rbase));
  const int jfirst = rpair / p.H, jlast = (min(R, rpair + 2 * kLpRows) - 1) / p.H;
  int lo, hi;
  latent_range(p, q.len, nchunk, chunk, &lo, &hi);
  hi = max(lo, min(hi, latent_end(p, q, jlast)));
  const int ntiles = q.err ? 0 : (hi - lo + kLpTile - 1) / kLpTile;
  // Tokens below it are seen by every row of the pair.
  const int all_see = q.kind == 1 ? min(hi, q.ctx) : min(hi, q.ctx + jfirst + 1);

  auto vfull = [&](int i) { return bar(PB_RING + i); };
  auto vfree = [&](int i) { return bar(PB_RING + C::VU + i); };
  auto kfull = [&](int i) { return bar(PB_RING + 2 * C::VU + i); };
  auto kfree = [&](int i) { return bar(PB_RING + 2 * C::VU + C::KU + i); };
  const uint32_t base = smem_u32(sm);

  // A producer's lane l < 8: (row, plane) of page l of the tile at t0, in the
  // cache's map.
  unsigned late = 0u;
  auto look_up = [&](int t0) {
    const int pg = t0 / kPage + lane;
    return lane < 8 && pg * kPage < hi && p.page_size ? p.block_table[(long long)s * p.max_blocks + pg] : 0;
  };
  auto page_at = [&](int t0, int blk) {
    if (p.page_size == 0) return make_int2(t0 + lane * kPage, s);
    if (blk < 0 || blk >= p.num_blocks) {
      late = VA_DEV_BAD_BLOCK;
      blk = 0;
    }
    return make_int2(0, blk);
  };
  // Looked up a tile ahead; the first beside the rest of the prologue.
  int blk0 = 0, blk1 = 0;
  const bool keys = warp == 0 || warp == 13, values = warp == 10 || warp == 12;
  if ((keys || values) && ntiles > 0) {
    blk0 = look_up(lo);
    blk1 = look_up(lo + kLpTile);
  }
  if (warp == 0 && ntiles > 0) {
    // The queries, at once: their barrier was set up by this warp.
    const uint32_t one = elected();
    const int qrow = __shfl_sync(0xffffffffu, q.row0 * p.H + rbase, 0);
    expect_by(one, bar(PB_QLAND), C::DK / 64 * C::QB);
#pragma unroll
    for (int c = 0; c < C::DK / 64; ++c) tma_2d_by(one, base + C::OFF_Q + c * C::QB, &maps.q, c * 64, qrow, bar(PB_QLAND));
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(tmem_at), 512);
  tc_fence_before();
  cluster_sync_all();  // the barriers of both CTAs are set up
  tc_fence_after();
  const uint32_t tm = __shfl_sync(0xffffffffu, *tmem_at, 0);
  const int work = __shfl_sync(0xffffffffu, ntiles, 0);
  const bool ragged = __shfl_sync(0xffffffffu, (hi - lo) % kLpTile, 0) != 0;  // of the last tile
  if (q.err && tid == 0) flag(p.status, q.err);
  // A finding on the way (a bad parent or page) does not stop the pipeline: what
  // it computes then is replaced by NaN at the end.
  auto found = [&](unsigned bits) {
    atomicOr(err_s, (int)bits);
    flag(p.status, bits);
  };
  // Both CTAs give up, and know it behind the closing barrier.
  auto fail = [&]() {
    *abort_p = 1;
    store_at(smem_u32(const_cast<int*>(abort_p)), rank ^ 1, 1);
    flag(p.status, VA_DEV_TIMEOUT);
  };
  auto drain = [&](uint32_t b, uint32_t parity) {
    int dummy = 0;
    mbar_wait(b, parity, &dummy, kLatentWaitNs);
  };
  // Barriers that the issuers wait for are the first CTA's.
  auto arrive_first = [&](int i) { arrive_cluster(at_first(bar(i))); };

  if (work == 0) {
    // nothing to read: straight to the outputs
  } else if (keys || values) {
    // ---------------------------------------------------------------- producers
    // Warps 0 and 13: the key groups, of this CTA's half of the tokens, two pages
    // each.  Warps 10 and 12: its half of V's columns, half of the tokens each.
    // (What is freed has to be back within a tile, and a page's block is a copy of
    // its own: issued by one warp each they took as long again.)
    const int who = warp >= 12 ? 1 : 0;
    const uint32_t one = elected();
    const int lo_u = __shfl_sync(0xffffffffu, lo, 0), hi_u = __shfl_sync(0xffffffffu, hi, 0);
    bool ok = true;
    if (warp == 0) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar(PB_QLAND), 0, abort_p, kLatentWaitNs));
      if (ok && lane == 0) arrive_first(PB_QALL);
    }
    int issued = 0;  // groups; or units of this warp, every second one
    uint32_t par = 1;
    for (int i = 0; i < work && ok; ++i) {
      const int t0 = lo_u + i * kLpTile;
      const int pages = (min(kLpTile, hi_u - t0) + kPage - 1) / kPage;
      const int2 a = page_at(t0, blk0);
      if (late) found(late);  // before anything of the tile is loaded
      __syncwarp();
      blk0 = blk1;
      blk1 = look_up(t0 + 2 * kLpTile);
      if (keys) {
        // The next tile's pages into L2: what is freed has to be back soon (32
        // sequences of 5,100 tokens, 128 heads: 65 us without, 59 with, 61.5 two
        // tiles ahead).
        if (lane >= 4 * rank + 2 * who && lane < 4 * rank + 2 * who + 2) {
          const int t = t0 + kLpTile + lane * kPage;
          const long long row = p.page_size ? (long long)blk0 * kPage : (long long)s * p.capacity + t;
          if (t < hi && blk0 >= 0 && (p.page_size == 0 || blk0 < p.num_blocks))
            bulk_prefetch_l2(reinterpret_cast<const unsigned short*>(p.cache) + row * C::DK, kPage * C::DK * 2);
        }
        int2 at[2];
#pragma unroll
        for (int g = 0; g < 2; ++g)
          at[g] = make_int2(__shfl_sync(0xffffffffu, a.x, 4 * rank + 2 * who + g), __shfl_sync(0xffffffffu, a.y, 4 * rank + 2 * who + g));
#pragma unroll
        for (int u = 0; u < C::KU; ++u) {
          ok = __all_sync(0xffffffffu, ok && mbar_wait(kfree(u), par, abort_p, kLatentWaitNs));
          if (!ok) break;
          if (rank == 0 && who == 0) expect_by(one, kfull(u), (uint32_t)(C::KG * pages * kPage * 128));
          const uint32_t b = at_first(kfull(u));
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (4 * rank + 2 * who + g >= pages) break;
#pragma unroll
            for (int k = 0; k < C::KG; ++k)
              tma_3d_by<true>(one, base + C::OFF_K + (u * C::KG + k) * C::KB + (2 * who + g) * kPage * 128, &maps.k, (u * C::KG + k) * 64, at[g].x,
                              at[g].y, b);
          }
          issued = i * C::KU + u + 1;
        }
      } else {
        int2 at[4];
#pragma unroll
        for (int g = 0; g < 4; ++g)
          at[g] = make_int2(__shfl_sync(0xffffffffu, a.x, 4 * who + g), __shfl_sync(0xffffffffu, a.y, 4 * who + g));
        const int mine = max(0, min(4, pages - 4 * who));
        // The last, ragged tile lands on barriers of each CTA's own, which then
        // clears what is behind the range.
        const bool alone = ragged && i == work - 1;
#pragma unroll
        for (int u = who; u < C::VU; u += 2) {
          ok = __all_sync(0xffffffffu, ok && mbar_wait(vfree(u), par, abort_p, kLatentWaitNs));
          if (!ok) break;
          const uint32_t bytes = (uint32_t)(C::VG * mine * kPage * 128);
          if (alone) expect_by(one, bar(PB_VLAST + u), bytes);
          else if (rank == 0) expect_by(one, vfull(u), 2 * bytes);
          const uint32_t b = alone ? bar(PB_VLAST + u) : at_first(vfull(u));
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            if (g >= mine) break;
#pragma unroll
            for (int k = 0; k < C::VG; ++k)
              tma_3d_by<true>(one, base + C::OFF_V + (u * C::VG + k) * C::VB + g * kPage * 128, &maps.k, u / 2 * 256 + rank * 128 + k * 64, at[g].x,
                              at[g].y, b);
          }
          issued = i * (C::VU / 2) + u / 2 + 1;
        }
      }
      par ^= 1;
    }
    if (!ok && lane == 0) fail();
    if (values && ok && ragged) {
      // Tokens behind the range may hold anything: their V is cleared (their
      // scores are masked).
      const int valid = max(0, min(kLpTile / 2, hi - lo - (work - 1) * kLpTile - who * (kLpTile / 2)));
      bool there = true;
      for (int u = who; u < C::VU; u += 2) there = there && mbar_wait(bar(PB_VLAST + u), 0, abort_p, kLatentWaitNs);
      if (__all_sync(0xffffffffu, there)) {
        for (int u = who; u < C::VU; u += 2)
          for (int k = 0; k < C::VG; ++k) clear_rows(sm + C::OFF_V + (u * C::VG + k) * C::VB, valid, kLpTile / 2, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive_first(PB_FIX);
      } else if (lane == 0) {
        fail();
      }
    }
    // No copy may still be landing when the pair goes away: the last of each group
    // and unit, those before have been read.  Keys, and values of whole tiles, are
    // counted in the first CTA, a ragged last tile's values in each.
    if (*abort_p && lane == 0) {
      const int n = keys ? C::KU : C::VU / 2;
      for (int k = max(0, issued - n); k < issued; ++k) {
        const int i = k / n, u = keys ? k % n : who + 2 * (k % n);
        if (values && ragged && i == work - 1) drain(bar(PB_VLAST + u), 0);
        else if (rank == 0) drain(keys ? kfull(u) : vfull(u), i & 1);
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ---------------------------------------------------------------- S issuer
    constexpr uint32_t ID = idesc_f16(2 * kLpRows, kLpTile, true, false);
    const uint32_t one = elected();
    bool ok = __all_sync(0xffffffffu, mbar_wait(bar(PB_QALL), 0, abort_p, kLatentWaitNs));
    bool any = false, there = false;
    const uint64_t kd0 = sdesc_sw128(base + C::OFF_K, 16, 1024), qd0 = sdesc_sw128(base + C::OFF_Q, 16, 1024);
    for (int i = 0; i < work && ok; ++i) {
      const int b = i & 1;
      const uint32_t scol = tm + C::COL_S + b * 64;
      ok = i < 2 || mbar_wait(bar(PB_SREAD + b), ((i - 2) >> 1) & 1, abort_p, kLatentWaitNs);
#pragma unroll
      for (int u = 0; u < C::KU; ++u) {
        ok = __all_sync(0xffffffffu, ok && (there || mbar_wait(kfull(u), i & 1, abort_p, kLatentWaitNs)));
        if (!ok) break;
        tc_fence_after();
        there = u + 1 < C::KU ? mbar_peek(kfull(u + 1), i & 1) : false;
#pragma unroll
        for (int kk = 0; kk < 4 * C::KG; ++kk) {
          const int c = u * C::KG + kk / 4;
          mma_ss_by<true>(one, scol, qd0 + (uint64_t)((c * C::QB) >> 4) + (kk & 3) * 2, kd0 + (uint64_t)((c * C::KB) >> 4) + (kk & 3) * 2, ID,
                          c > 0 || kk > 0 ? 1u : 0u);
        }
        any = true;
        commit_by<true>(one, kfree(u));
      }
      if (!ok) break;
      commit_by<true>(one, bar(PB_SFULL + b));
    }
    if (!ok && lane == 0) fail();
    if (!ok && any) {
      // What was issued completes before TMEM and shared memory go.  (A commit is
      // for what its own thread has issued.)
      commit_by<true>(one, bar(PB_SDRAIN));
      drain(bar(PB_SDRAIN), 0);
    }
  } else if (warp == 11 && rank == 0) {
    // ---------------------------------------------------------------- P.V issuer
    constexpr uint32_t ID = idesc_f16(2 * kLpRows, 256, true, true);
    const uint32_t one = elected();
    bool ok = true, any = false, there = false;
    const uint64_t vd0 = sdesc_sw128(base + C::OFF_V, C::VB, 1024), pd0 = sdesc_sw128(base + C::OFF_P, 16, 1024);
    for (int i = 0; i < work && ok; ++i) {
      const bool fixed = ragged && i == work - 1;
      ok = mbar_wait(bar(PB_PFULL), i & 1, abort_p, kLatentWaitNs) && (!fixed || mbar_wait(bar(PB_FIX), 0, abort_p, kLatentWaitNs));
#pragma unroll
      for (int u = 0; u < C::VU; ++u) {  // 256 columns, 64 tokens
        ok = __all_sync(0xffffffffu, ok && (fixed || there || mbar_wait(vfull(u), i & 1, abort_p, kLatentWaitNs)));
        if (!ok) break;
        tc_fence_after();
        there = u + 1 < C::VU && mbar_peek(vfull(u + 1), i & 1);
#pragma unroll
        for (int kk = 0; kk < kLpTile / 2 / 16; ++kk)
          mma_ss_by<true>(one, tm + C::COL_O + u / 2 * 128, pd0 + (uint64_t)(((u & 1) * C::PB + kk * 32) >> 4),
                          vd0 + (uint64_t)((u * C::VG * C::VB + kk * 2048) >> 4), ID, i > 0 || (u & 1) || kk > 0 ? 1u : 0u);
        any = true;
        commit_by<true>(one, vfree(u));
      }
      if (ok) commit_by<true>(one, bar(PB_PFREE));
    }
    if (!ok && lane == 0) fail();
    if (any) {
      // After every P.V, in a failed run too.
      commit_by<true>(one, bar(PB_OFINAL));
      drain(bar(PB_OFINAL), 0);
    }
  } else if (warp >= 2 && warp < 10) {
    // ---------------------------------------------------------------- softmax
    // TMEM lane 64 t + r: row r, half t of the tile's tokens (and of each 256 of
    // O's columns); of its 64 columns of S a warp takes half.
    const int quad = warp & 3, part = (warp - 2) >> 2;
    const int r = (quad & 1) * 32 + lane, th = quad >> 1;
    const int who = th * 2 + part;             // of the row's four threads
    const int id = 5 + (quad & 1);             // barrier of the rows' four warps
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const bool rvalid = r < nrows;
    const bool warp_live = __any_sync(0xffffffffu, rvalid);
    const int j = rvalid ? (rbase + r) / p.H : 0;
    unsigned anc = 0u;
    if (rvalid && q.kind == 1) {
      bool bad_parent = false;
      anc = row_mask(1, p.parent + q.row0, j, &bad_parent);
      if (bad_parent) found(VA_DEV_BAD_PARENT);
    }
    bool ok = true;
    float m_use = -INFINITY, l_run = 0.f;
    bool there = false;  // S of the tile, seen ahead
    const float c_r = p.scale_log2;
    // A failed wait does not leave the loop: its barriers are shared.
    for (int i = 0; i < work; ++i) {
      const int b = i & 1;
      if (ok && !__all_sync(0xffffffffu, there || mbar_wait(bar(PB_SFULL + b), (i >> 1) & 1, abort_p, kLatentWaitNs))) ok = false;
      tc_fence_after();
      const int t0 = lo + i * kLpTile + th * 64 + part * 32;
      float sv[32];
      float mx = -INFINITY;
      if (ok && warp_live) {
        uint32_t sr[32];
        tmem_ld32(tm + lanes + C::COL_S + b * 64 + part * 32, sr);
        tmem_wait_ld();
        if (lo + (i + 1) * kLpTile <= all_see) {
          float m2 = -INFINITY;
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            mx = max3(mx, __uint_as_float(sr[c]), __uint_as_float(sr[c + 1]));
            m2 = max3(m2, __uint_as_float(sr[c + 2]), __uint_as_float(sr[c + 3]));
          }
          mx = fmaxf(mx, m2);
#pragma unroll
          for (int c = 0; c < 32; ++c) sv[c] = __uint_as_float(sr[c]);
        } else {
          const unsigned vis = rvalid ? latent_bits(p, q, anc, j, hi, t0) : 0u;
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            sv[c] = (vis >> c) & 1u ? __uint_as_float(sr[c]) : -INFINITY;
            mx = fmaxf(mx, sv[c]);
          }
        }
      }
      // S(i) is in registers: its buffer may be written again.
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_first(PB_SREAD + b);
      // The row's maximum over its four threads (raw scores; c_r > 0).
      red[(b * 4 + who) * kLpRows + r] = mx;
      bar_sync(id, 128);
#pragma unroll
      for (int o = 0; o < 4; ++o) mx = fmaxf(mx, red[(b * 4 + o) * kLpRows + r]);
      const float mt = mx * c_r;
      const bool need = rvalid && m_use != -INFINITY && mt > m_use + 8.f;
      const float m_new = m_use == -INFINITY || need ? mt : m_use;
      // The previous P.V has to be done before O is rescaled or P written.
      if (i > 0 && ok && !__all_sync(0xffffffffu, mbar_wait(bar(PB_PFREE), (i - 1) & 1, abort_p, kLatentWaitNs))) ok = false;
      if (ok && __any_sync(0xffffffffu, need)) {
        tc_fence_after();
        const float f = need ? exp2f(m_use - m_new) : 1.f;
#pragma unroll 1
        for (int c0 = part * 128; c0 < (part + 1) * 128; c0 += 16) {
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
      m_use = m_new;
      there = i + 1 < work && mbar_peek(bar(PB_SFULL + (b ^ 1)), ((i + 1) >> 1) & 1);
      if (ok && warp_live) {
        uint32_t ph[16];
        uint64_t l2 = pack2(0.f, 0.f);
        // A masked score (-inf) gives 0; while nothing of the row was visible
        // every score is masked, and the 0 offset keeps them at -inf.
        const float mneg = m_use == -INFINITY ? 0.f : -m_use;
        const uint64_t c2 = pack2(c_r, c_r), m2 = pack2(mneg, mneg);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          float a, d;
          unpack2(fma2(pack2(sv[2 * c], sv[2 * c + 1]), c2, m2), a, d);
          a = lu_ex2(a);
          d = lu_ex2(d);
          l2 = add2(l2, pack2(a, d));
          // bf16, as the matrix unit takes it (2^-8 at most, see the 128-row kernel).
          const __nv_bfloat162 h = __floats2bfloat162_rn(a, d);
          ph[c] = *reinterpret_cast<const uint32_t*>(&h);
        }
        float l0, l1;
        unpack2(l2, l0, l1);
        l_run += l0 + l1;
        unsigned char* prow = sm + C::OFF_P + th * C::PB + r * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4*>(prow + (((part * 4 + c) ^ (r & 7)) << 4)) = make_uint4(ph[4 * c], ph[4 * c + 1], ph[4 * c + 2], ph[4 * c + 3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_first(PB_PFULL);
    }
    if (ok && !__all_sync(0xffffffffu, mbar_wait(bar(PB_OFINAL), 0, abort_p, kLatentWaitNs))) ok = false;
    if (!ok && lane == 0) fail();
    tc_fence_after();
    red[who * kLpRows + r] = l_run;
    bar_sync(1, 256);
    const float l = (red[r] + red[kLpRows + r]) + (red[2 * kLpRows + r] + red[3 * kLpRows + r]);
    const bool bad = __any_sync(0xffffffffu, *abort_p != 0 || *reinterpret_cast<volatile int*>(err_s) != 0);
    const float inv = bad ? NAN : l != 0.f ? 1.f / l : 0.f;
    const long long first = (long long)q.row0 * p.H + rbase, partials = latent_part(p, s, q.row0, q.n, chunk);
    if (rvalid && who == 0) {
      if (live > 1) {
        const long long si = partials + first + r;
        p.ws_ml[2 * si] = bad ? NAN : m_use;
        p.ws_ml[2 * si + 1] = bad ? NAN : l;
      } else {
        p.lse[first + r] = bad ? NAN : l != 0.f ? (m_use + log2f(l)) * kLn2 : -INFINITY;
      }
    }
    // O rows through shared memory (keys, values and queries are done with) to
    // coalesced stores; fp32 sums for the merge, or the finished bf16 row.
    if (warp_live) {
      unsigned char* row = sm + r * C::OROW;
#pragma unroll 1
      for (int c0 = part * 128; c0 < (part + 1) * 128; c0 += 32) {
        uint32_t o[32];
        tmem_ld32(tm + lanes + C::COL_O + c0, o);
        tmem_wait_ld();
        const int d0 = (c0 >> 7) * 256 + th * 128 + (c0 & 127);
        if (live > 1) {
          if (bad) {
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = 0x7fffffffu;
          }
#pragma unroll
          for (int c = 0; c < 32; c += 4) *reinterpret_cast<uint4*>(row + (d0 + c) * 4) = make_uint4(o[c], o[c + 1], o[c + 2], o[c + 3]);
        } else {
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const __nv_bfloat162 h = l != 0.f || bad ? __floats2bfloat162_rn(__uint_as_float(o[2 * c]) * inv, __uint_as_float(o[2 * c + 1]) * inv)
                                                    : __floats2bfloat162_rn(0.f, 0.f);
            w[c] = *reinterpret_cast<const uint32_t*>(&h);
          }
#pragma unroll
          for (int c = 0; c < 16; c += 4) *reinterpret_cast<uint4*>(row + d0 * 2 + c * 4) = make_uint4(w[c], w[c + 1], w[c + 2], w[c + 3]);
        }
      }
    }
    bar_sync(1, 256);
    if (live > 1) {
      constexpr int PIECES = C::DV / 4;  // of 16 bytes
      float* to = p.ws_acc + (partials + first) * C::DV;
      for (int u = tid - 64; u < nrows * PIECES; u += 256)
        *reinterpret_cast<uint4*>(to + (long long)u * 4) = *reinterpret_cast<const uint4*>(sm + u / PIECES * C::OROW + u % PIECES * 16);
    } else {
      constexpr int PIECES = C::DV / 8;
      unsigned short* to = reinterpret_cast<unsigned short*>(p.o) + first * C::DV;
      for (int u = tid - 64; u < nrows * PIECES; u += 256)
        *reinterpret_cast<uint4*>(to + (long long)u * 8) = *reinterpret_cast<const uint4*>(sm + u / PIECES * C::OROW + u % PIECES * 16);
    }
  }

  if (work == 0) {
    // An error, or a chunk that the block's rows see nothing of.
    for (int u = tid; u < nrows * C::DV; u += kLpThreads) {
      const long long item = (long long)q.row0 * p.H + rbase + u / C::DV;
      const int d = u % C::DV;
      if (live > 1) {
        if (d == 0) {
          const long long si = latent_part(p, s, q.row0, q.n, chunk) + item;
          p.ws_ml[2 * si] = q.err ? NAN : -INFINITY;
          p.ws_ml[2 * si + 1] = q.err ? NAN : 0.f;
        }
      } else {
        reinterpret_cast<unsigned short*>(p.o)[item * C::DV + d] = q.err ? 0x7fffu : 0u;
        if (d == 0) p.lse[item] = q.err ? NAN : -INFINITY;
      }
    }
  }
  tc_fence_before();
  cluster_sync_all();  // the other CTA's products and arrivals reach into this one
  tc_fence_after();
  if (*abort_p) {  // in both or in none
    settle();
    cluster_sync_all();
  }
  if (warp == 1) tmem_dealloc_pair(tm, 512);
}

int latent_pair_rows() { return 2 * kLpRows; }

cudaError_t launch_latent_pair(const LatentParams& p, dim3 grid, cudaStream_t st) {
  static std::atomic<unsigned long long> ready{0ull};
  cudaError_t e = allow_smem(latent_pair_kernel, LpCfg::SMEM, ready);
  if (e != cudaSuccess) return e;
  LpMaps m;
  memset(&m, 0, sizeof(m));
  if (!latent_query_map(&m.q, p, kLpRows) || !latent_cache_map(&m.k, p)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(grid.x * 2, grid.y, grid.z);
  cfg.blockDim = dim3(kLpThreads);
  cfg.dynamicSmemBytes = LpCfg::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, latent_pair_kernel, p, m);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace va
