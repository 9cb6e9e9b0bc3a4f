// Tensor-core attention over latent caches of 256 columns, bf16, more than 32 query
// rows: tcgen05 + TMEM + TMA, 128 query rows to a CTA.
//
// Per tile of 64 tokens:
//   S = Q C^T     tcgen05.mma into one of two S buffers in TMEM
//   softmax       eight warps, one TMEM lane (query row) per thread and half
//                 of the tile's columns per warp; online (m, l) in log2 units,
//                 O rescaled only when the maximum grows by more than 2^8; P
//                 in bf16 over S's place
//   O += P V      tcgen05.mma, A = P (TMEM), B = V tile (MN-major)
// so that S of the next tile runs under this tile's softmax.
//
// A token has one row of 320 values and V is the first 256 of them, so the column
// blocks of V are loaded once and read by both products (as K they are K-major, as
// V MN-major: the same bytes).  The queries of the V columns go to TMEM, those of
// the rope part stay in shared memory.
//
// Shared memory holds two rings of 64-column blocks of a tile: V stages of
// VBLK blocks, freed by P.V, and single blocks of the key's other columns,
// freed as soon as S has read them.
//
// Every wait is bounded (VA_DEV_TIMEOUT); on a timeout the CTA drains its own
// copies and MMAs, frees TMEM and writes NaN.
#include <string.h>

#include "va_latent_mma.cuh"

namespace va {
using namespace sm100;

constexpr int kLuM = 128;
constexpr int kLuThreads = 384;

struct LuCfg {
  static constexpr int DV = 256, DK = DV + kLatentRope;
  static constexpr int NT = 64;                      // tokens per tile
  static constexpr int BLK = NT * 128;               // bytes of a 64-column block
  static constexpr int VBLK = DV / 64;               // blocks of a V stage
  static constexpr int KBLK = DK / 64 - VBLK;        // other blocks of the key
  static constexpr int QT = DV;                      // query columns in TMEM
  static constexpr int QS = DK - QT;                 // query columns in shared memory
  static constexpr int NV = 5;                       // V stages
  static constexpr int NK = 5;                       // key blocks
  static constexpr int COL_O = 0;
  static constexpr int COL_S = DV;
  static constexpr int COL_Q = COL_S + 2 * NT;
  static constexpr int OFF_V = 0;
  static constexpr int OFF_K = NV * VBLK * BLK;
  static constexpr int OFF_Q = OFF_K + NK * BLK;
  static constexpr int OFF_END = OFF_Q + QS / 64 * kLuM * 128;
  // The queries on their way to TMEM: in the last V stages.
  static constexpr int QSTAGE = OFF_K - QT / 64 * kLuM * 128;
  static constexpr int QV_FIRST = QSTAGE / (VBLK * BLK);  // the first tile whose place they have
  static constexpr int OROW = DV * 4 + 16;           // O staging at the end, padded rows
  static constexpr int NB = 11 + 2 * NV + 2 * NK;    // barriers
  static constexpr int OFF_RED = OFF_END > kLuM * OROW ? OFF_END : kLuM * OROW;
  static constexpr int OFF_BAR = OFF_RED + 2 * 2 * kLuM * 4;
  static constexpr int SMEM = OFF_BAR + NB * 8 + 16;
  static_assert(COL_Q + QT / 2 <= 512, "TMEM columns");
  static_assert(QSTAGE >= VBLK * BLK, "tile 0 beside the queries");
  static_assert(SMEM <= 232448, "shared memory");
};

enum { LB_SFULL = 0, LB_PFULL = 2, LB_SFREE = 4, LB_QLAND = 6, LB_QREADY = 7, LB_OFINAL = 8, LB_FIX = 9, LB_SDRAIN = 10, LB_RING = 11 };

struct LuMaps {
  CUtensorMap q, k;  // queries; cache
};

__global__ void __launch_bounds__(kLuThreads, 1) latent_umma_kernel(const LatentParams p, const __grid_constant__ LuMaps maps) {
  using C = LuCfg;
  constexpr int NT = C::NT, NC = NT / 2, DV = C::DV;
  extern __shared__ __align__(1024) unsigned char sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  float* red = reinterpret_cast<float*>(sm + C::OFF_RED);  // [2][2][kLuM]
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(sm + C::OFF_BAR + C::NB * 8);
  volatile int* abort_p = reinterpret_cast<volatile int*>(tmem_at + 1);
  int* err_s = reinterpret_cast<int*>(tmem_at + 2);

  asm volatile("griddepcontrol.launch_dependents;");
  // Broadcasts: what a warp has in common is known to be so.
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  if (warp == 0) {
    if (lane == 0) {
      *err_s = 0;
      *abort_p = 0;
      prefetch_map(&maps.q);
      prefetch_map(&maps.k);
    }
    for (int i = lane; i < C::NB; i += 32)
      mbar_init(bar(i), (i >= LB_PFULL && i < LB_SFREE) || i == LB_QREADY ? 8 : 1);
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
    if (blockIdx.x == 0) latent_nan_rows(p, s, 0, p.H, tid, kLuThreads);
    return;
  }
  const int R = latent_rows(p, q.n);
  const int blocks = (R + kLuM - 1) / kLuM;
  if (blocks == 0) return;
  const int nchunk = latent_chunks(p, q.n);
  const int rb = blockIdx.x % blocks, chunk = blockIdx.x / blocks;
  const int live = latent_live(p, q.err ? 0 : q.len, nchunk);
  if (chunk >= live) return;
  const int rbase = rb * kLuM, nrows = min(kLuM, R - rbase);
  const int jfirst = rbase / p.H, jlast = (rbase + nrows - 1) / p.H;
  int lo, hi;
  latent_range(p, q.len, nchunk, chunk, &lo, &hi);
  hi = max(lo, min(hi, latent_end(p, q, jlast)));
  const int ntiles = q.err ? 0 : (hi - lo + NT - 1) / NT;
  // Tokens below it are seen by every row of the block.
  const int all_see = q.kind == 1 ? min(hi, q.ctx) : min(hi, q.ctx + jfirst + 1);

  auto vfull = [&](int i) { return bar(LB_RING + i); };
  auto vfree = [&](int i) { return bar(LB_RING + C::NV + i); };
  auto kfull = [&](int i) { return bar(LB_RING + 2 * C::NV + i); };
  auto kfree = [&](int i) { return bar(LB_RING + 2 * C::NV + C::NK + i); };
  const uint32_t base = smem_u32(sm);

  // A producer's lane l < 4: (row, plane) of page l of the tile at t0, in the
  // cache's map.
  unsigned late = 0u;
  auto look_up = [&](int t0) {
    const int pg = t0 / kPage + lane;
    return lane < 4 && pg * kPage < hi && p.page_size ? p.block_table[(long long)s * p.max_blocks + pg] : 0;
  };
  auto page_at = [&](int t0, int blk) {
    if (p.page_size == 0) return make_int2(t0 + lane * kPage, s);
    if (blk < 0 || blk >= p.num_blocks) {
      late = VA_DEV_BAD_BLOCK;
      blk = 0;
    }
    return make_int2(0, blk);
  };
  // The first tile's are looked up beside the rest of the prologue.
  int blk0 = 0;
  if ((warp == 0 || warp == 10) && ntiles > 0) blk0 = look_up(lo);
  if (warp == 0 && ntiles > 0) {
    // The queries, at once: their barrier was set up by this warp.
    const uint32_t one = elected();
    const int qrow = __shfl_sync(0xffffffffu, q.row0 * p.H + rbase, 0);
    expect_by(one, bar(LB_QLAND), C::DK / 64 * kLuM * 128);
#pragma unroll
    for (int c = 0; c < C::DK / 64; ++c) {
      const uint32_t dst = base + (c < C::QT / 64 ? C::QSTAGE + c * kLuM * 128 : C::OFF_Q + (c - C::QT / 64) * kLuM * 128);
      tma_2d_by(one, dst, &maps.q, c * 64, qrow, bar(LB_QLAND));
    }
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_at), 512);
    tmem_relinquish();
  }
  const int quad = warp & 3;
  const int r = quad * 32 + lane;
  const bool is_sm = warp >= 2 && warp < 10;
  const bool rvalid = is_sm && r < nrows;
  const int j = rvalid ? (rbase + r) / p.H : 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = __shfl_sync(0xffffffffu, *tmem_at, 0);
  const int work = __shfl_sync(0xffffffffu, ntiles, 0);
  const bool ragged = __shfl_sync(0xffffffffu, (hi - lo) % NT, 0) != 0;  // of the last tile
  if (q.err && tid == 0) flag(p.status, q.err);
  // A finding on the way (a bad parent or page) does not stop the pipeline: what
  // it computes then is replaced by NaN at the end.
  auto found = [&](unsigned bits) {
    atomicOr(err_s, (int)bits);
    flag(p.status, bits);
  };
  auto fail = [&]() {
    *abort_p = 1;
    flag(p.status, VA_DEV_TIMEOUT);
  };
  auto drain = [&](uint32_t b, uint32_t parity) {
    int dummy = 0;
    mbar_wait(b, parity, &dummy, kLatentWaitNs);
  };

  if (work == 0) {
    // nothing to read: straight to the outputs
  } else if (warp == 0 || warp == 10) {
    // ---------------------------------------------------------------- producers
    // Warp 10: the V stages.  Warp 0: the key's other blocks.
    // Lane l < 4 looks the tile's page l up.
    const bool keys = warp == 0;
    const uint32_t one = elected();
    const int lo_u = __shfl_sync(0xffffffffu, lo, 0), hi_u = __shfl_sync(0xffffffffu, hi, 0);
    bool ok = true;
    int issued = 0;  // tiles (V) or blocks (keys)
    int st = 0;
    uint32_t par = 1;
    for (int i = 0; i < work && ok; ++i) {
      const int t0 = lo_u + i * NT;
      const int pages = (min(NT, hi_u - t0) + kPage - 1) / kPage;
      int2 at[4];
      const int2 a = page_at(t0, i == 0 ? blk0 : look_up(t0));
      if (late) found(late);  // before anything of the tile is loaded
      __syncwarp();
#pragma unroll
      for (int g = 0; g < 4; ++g) at[g] = make_int2(__shfl_sync(0xffffffffu, a.x, g), __shfl_sync(0xffffffffu, a.y, g));
      if (!keys) {
        ok = (i != C::QV_FIRST || mbar_wait(bar(LB_QREADY), 0, abort_p, kLatentWaitNs)) && mbar_wait(vfree(st), par, abort_p, kLatentWaitNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t dst = base + C::OFF_V + st * C::VBLK * C::BLK, b = vfull(st);
        expect_by(one, b, (uint32_t)(C::VBLK * pages * kPage * 128));
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (g >= pages) break;
#pragma unroll
          for (int c = 0; c < C::VBLK; ++c)
            tma_3d_by(one, dst + c * C::BLK + g * kPage * 128, &maps.k, c * 64, at[g].x, at[g].y, b);
        }
        issued = i + 1;
        if (++st == C::NV) st = 0, par ^= 1;
      } else {
#pragma unroll
        for (int c = 0; c < C::KBLK; ++c) {
          const int n = i * C::KBLK + c;
          ok = __all_sync(0xffffffffu, ok && mbar_wait(kfree(st), par, abort_p, kLatentWaitNs));
          if (!ok) break;
          const uint32_t dst = base + C::OFF_K + st * C::BLK, b = kfull(st);
          const int col = (c + C::VBLK) * 64;
          expect_by(one, b, (uint32_t)(pages * kPage * 128));
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            if (g >= pages) break;
            tma_3d_by(one, dst + g * kPage * 128, &maps.k, col, at[g].x, at[g].y, b);
          }
          issued = n + 1;
          if (++st == C::NK) st = 0, par ^= 1;
        }
      }
    }
    if (!ok && lane == 0) fail();
    if (!keys && ok && ragged) {
      // Tokens behind the range may hold anything: their V is cleared (their
      // scores are masked).
      const int i = work - 1, st = i % C::NV, valid = hi - lo - i * NT;
      if (__all_sync(0xffffffffu, mbar_wait(vfull(st), (i / C::NV) & 1, abort_p, kLatentWaitNs))) {
        for (int c = 0; c < C::VBLK; ++c) clear_rows(sm + C::OFF_V + (st * C::VBLK + c) * C::BLK, valid, NT, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(LB_FIX));
      } else if (lane == 0) {
        fail();
      }
    }
    // No copy may still be landing when the CTA goes away.
    if (*abort_p && lane == 0) {
      if (keys) drain(bar(LB_QLAND), 0);
      const int n = keys ? C::NK : C::NV;
      for (int i = max(0, issued - n); i < issued; ++i) drain(keys ? kfull(i % n) : vfull(i % n), (i / n) & 1);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- S issuer
    constexpr uint32_t ID = idesc_f16(kLuM, NT, true, false);
    const uint32_t one = elected();
    bool ok = mbar_wait(bar(LB_QLAND), 0, abort_p, kLatentWaitNs) && mbar_wait(bar(LB_QREADY), 0, abort_p, kLatentWaitNs);
    ok = __all_sync(0xffffffffu, ok);
    bool any = false;
    int st = 0, sk = 0;                     // V stage, key block
    uint32_t pv = 0, pk = 0;                // their parities
    const uint64_t vd0 = sdesc_sw128(base + C::OFF_V, 16, 1024), kd0 = sdesc_sw128(base + C::OFF_K, 16, 1024);
    const uint64_t qd0 = sdesc_sw128(base + C::OFF_Q, 16, 1024);
    // What a tile starts with: its S buffer free, and its V stage there.
    auto peek_tile = [&](int i) {
      return (i < 2 || mbar_peek(bar(LB_SFREE + (i & 1)), ((i - 2) >> 1) & 1)) &&
             mbar_peek(vfull(st), pv);
    };
    auto wait_tile = [&](int i) {
      return (i < 2 || mbar_wait(bar(LB_SFREE + (i & 1)), ((i - 2) >> 1) & 1, abort_p, kLatentWaitNs)) &&
             mbar_wait(vfull(st), pv, abort_p, kLatentWaitNs);
    };
    bool there = false;
    for (int i = 0; i < work && ok; ++i) {
      const int b = i & 1;
      const uint32_t scol = tm + C::COL_S + b * NT;
      ok = __all_sync(0xffffffffu, there || wait_tile(i));
      if (!ok) break;
      tc_fence_after();
      there = mbar_peek(kfull(sk), pk);
      const uint64_t kv = vd0 + (uint64_t)((st * C::VBLK * C::BLK) >> 4);
#pragma unroll
      for (int kk = 0; kk < C::VBLK * 4; ++kk)
        mma_ts_by(one, scol, tm + C::COL_Q + kk * 8, kv + (uint64_t)(((kk >> 2) * C::BLK + (kk & 3) * 32) >> 4), ID,
                  kk > 0 ? 1u : 0u);
      any = true;
      if (++st == C::NV) st = 0, pv ^= 1;
#pragma unroll
      for (int c = 0; c < C::KBLK; ++c) {
        ok = __all_sync(0xffffffffu, there || mbar_wait(kfull(sk), pk, abort_p, kLatentWaitNs));
        if (!ok) break;
        tc_fence_after();
        const uint64_t kd = kd0 + (uint64_t)((sk * C::BLK) >> 4);
        const uint32_t free = kfree(sk);
        if (++sk == C::NK) sk = 0, pk ^= 1;
        there = c + 1 < C::KBLK ? mbar_peek(kfull(sk), pk) : i + 1 < work && peek_tile(i + 1);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ss_by(one, scol, qd0 + (uint64_t)((c * kLuM * 128) >> 4) + kk * 2, kd + kk * 2, ID, 1u);
        commit_by(one, free);
      }
      if (!ok) break;
      commit_by(one, bar(LB_SFULL + b));
    }
    if (!ok && lane == 0) fail();
    if (!ok && any) {
      // What was issued completes before TMEM and shared memory go.  (A commit is
      // for what its own thread has issued.)
      commit_by(one, bar(LB_SDRAIN));
      drain(bar(LB_SDRAIN), 0);
    }
  } else if (warp == 11) {
    // ---------------------------------------------------------------- P.V issuer
    constexpr uint32_t ID = idesc_f16(kLuM, DV, true, true);
    const uint32_t one = elected();
    bool ok = true, any = false;
    int st = 0;
    uint32_t pv = 0;
    const uint64_t vd0 = sdesc_sw128(base + C::OFF_V, C::BLK, 1024);
    for (int i = 0; i < work; ++i) {
      const int b = i & 1;
      ok = mbar_wait(bar(LB_PFULL + b), (i >> 1) & 1, abort_p, kLatentWaitNs) &&
           mbar_wait(vfull(st), pv, abort_p, kLatentWaitNs) &&
           (i < work - 1 || !ragged || mbar_wait(bar(LB_FIX), 0, abort_p, kLatentWaitNs));
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint64_t vd = vd0 + (uint64_t)((st * C::VBLK * C::BLK) >> 4);
#pragma unroll
      for (int kk = 0; kk < NT / 16; ++kk)
        mma_ts_by(one, tm + C::COL_O, tm + C::COL_S + b * NT + kk * 8, vd + (uint64_t)((kk * 2048) >> 4), ID,
                  i > 0 || kk > 0 ? 1u : 0u);
      any = true;
      commit_by(one, bar(LB_SFREE + b));
      commit_by(one, vfree(st));
      if (++st == C::NV) st = 0, pv ^= 1;
    }
    if (!ok && lane == 0) fail();
    if (any) {
      // After every P.V, in a failed run too.
      commit_by(one, bar(LB_OFINAL));
      drain(bar(LB_OFINAL), 0);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int half = (warp - 2) >> 2;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const bool warp_live = __any_sync(0xffffffffu, rvalid);
    bool ok = __all_sync(0xffffffffu, mbar_wait(bar(LB_QLAND), 0, abort_p, kLatentWaitNs));
    if (ok) {
      // Query row -> TMEM: this half's 16-byte pieces of the swizzled blocks.
      // (Rows behind the block's last hold other rows, or zeros: no one reads
      // what comes of them.)
      constexpr int PIECES = C::QT / 16;  // per half
#pragma unroll 1
      for (int c0 = half * PIECES; c0 < (half + 1) * PIECES; c0 += 4) {
        uint32_t w[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = c0 + k;
          const uint4 v = *reinterpret_cast<const uint4*>(sm + C::QSTAGE + c / 8 * kLuM * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
          w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
        }
        tmem_st16(tm + lanes + C::COL_Q + c0 * 4, w);
      }
      tmem_wait_st();
      // Copies will write where these reads were.
      fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(LB_QREADY));

    unsigned anc = 0u;
    if (rvalid && q.kind == 1) {
      bool bad_parent = false;
      anc = row_mask(1, p.parent + q.row0, j, &bad_parent);
      if (bad_parent) found(VA_DEV_BAD_PARENT);
    }
    float m_use = -INFINITY, l_run = 0.f;
    bool there = false;  // S of the tile, seen ahead
    const float c_r = p.scale_log2;
    // A failed wait does not leave the loop: every iteration has one named
    // barrier shared with the partner warp.
    for (int i = 0; i < work; ++i) {
      const int b = i & 1;
      if (ok && !__all_sync(0xffffffffu, there || mbar_wait(bar(LB_SFULL + b), (i >> 1) & 1, abort_p, kLatentWaitNs))) ok = false;
      tc_fence_after();
      const uint32_t scol = tm + lanes + C::COL_S + b * NT;
      const int t0 = lo + i * NT + NC * half;
      float sv[NC];
      float mx = -INFINITY;
      if (ok && warp_live) {
        uint32_t sr[NC];
        tmem_ld32_into<0>(scol + NC * half, sr);
        tmem_wait_ld();
        if (lo + (i + 1) * NT <= all_see) {
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
          static_assert(NC == 32, "a word of bits");
          const unsigned vis = rvalid ? latent_bits(p, q, anc, j, hi, t0) : 0u;
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            sv[c] = (vis >> c) & 1u ? __uint_as_float(sr[c]) : -INFINITY;
            mx = fmaxf(mx, sv[c]);
          }
        }
      }
      // The row's maximum over both halves (raw scores; c_r > 0).
      red[(b * 2 + half) * kLuM + r] = mx;
      bar_sync(5 + quad, 64);
      mx = fmaxf(mx, red[(b * 2 + (half ^ 1)) * kLuM + r]);
      const float mt = mx * c_r;
      const bool need = rvalid && m_use != -INFINITY && mt > m_use + 8.f;
      const float m_new = m_use == -INFINITY || need ? mt : m_use;
      if (ok && __any_sync(0xffffffffu, need)) {
        // Rescale this half of the warp's O rows once the previous P.V landed.
        if (i > 0 && !__all_sync(0xffffffffu, mbar_wait(bar(LB_SFREE + (b ^ 1)), ((i - 1) >> 1) & 1, abort_p, kLatentWaitNs))) ok = false;
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
      there = i + 1 < work && mbar_peek(bar(LB_SFULL + (b ^ 1)), ((i + 1) >> 1) & 1);
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
        tmem_st16(scol + 16 * half, ph);
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(LB_PFULL + b));
    }
    if (ok && !__all_sync(0xffffffffu, mbar_wait(bar(LB_OFINAL), 0, abort_p, kLatentWaitNs))) ok = false;
    if (!ok && lane == 0) fail();
    tc_fence_after();
    red[half * kLuM + r] = l_run;
    bar_sync(1, 256);
    const float l = red[r] + red[kLuM + r];
    const bool bad = __any_sync(0xffffffffu, *abort_p != 0 || *reinterpret_cast<volatile int*>(err_s) != 0);
    const float inv = bad ? NAN : l != 0.f ? 1.f / l : 0.f;
    const long long part = latent_part(p, s, q.row0, q.n, chunk);
    if (rvalid && half == 0) {
      const long long item = latent_item(p, q.row0, rbase + r, 0);
      if (live > 1) {
        const long long si = part + item;
        p.ws_ml[2 * si] = bad ? NAN : m_use;
        p.ws_ml[2 * si + 1] = bad ? NAN : l;
      } else {
        p.lse[item] = bad ? NAN : l != 0.f ? (m_use + log2f(l)) * kLn2 : -INFINITY;
      }
    }
    // O rows through shared memory (its rings are idle now) to coalesced
    // stores; fp32 sums for the merge, or the finished bf16 row.
    if (warp_live) {
#pragma unroll 1
      for (int c0 = half * (DV / 2); c0 < (half + 1) * (DV / 2); c0 += 32) {
        uint32_t o[32];
        tmem_ld32(tm + lanes + C::COL_O + c0, o);
        tmem_wait_ld();
        unsigned char* row = sm + r * C::OROW;
        if (live > 1) {
          if (bad) {
#pragma unroll
            for (int c = 0; c < 32; ++c) o[c] = 0x7fffffffu;
          }
#pragma unroll
          for (int c = 0; c < 32; c += 4)
            *reinterpret_cast<uint4*>(row + (c0 + c) * 4) = make_uint4(o[c], o[c + 1], o[c + 2], o[c + 3]);
        } else {
          uint32_t w[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            // A row that sees nothing has no sum (its lanes of O may hold anything).
            const __nv_bfloat162 h = l != 0.f || bad ? __floats2bfloat162_rn(__uint_as_float(o[2 * c]) * inv, __uint_as_float(o[2 * c + 1]) * inv)
                                                    : __floats2bfloat162_rn(0.f, 0.f);
            w[c] = *reinterpret_cast<const uint32_t*>(&h);
          }
#pragma unroll
          for (int c = 0; c < 16; c += 4)
            *reinterpret_cast<uint4*>(row + c0 * 2 + c * 4) = make_uint4(w[c], w[c + 1], w[c + 2], w[c + 3]);
        }
      }
    }
    bar_sync(1, 256);
    const long long first = latent_item(p, q.row0, rbase, 0);
    if (live > 1) {
      constexpr int PIECES = DV / 4;  // of 16 bytes
      float* to = p.ws_acc + (part + first) * DV;
      for (int u = tid - 64; u < nrows * PIECES; u += 256) {
        const int row = u / PIECES, c = u % PIECES;
        *reinterpret_cast<uint4*>(to + row * DV + c * 4) = *reinterpret_cast<const uint4*>(sm + row * C::OROW + c * 16);
      }
    } else {
      constexpr int PIECES = DV / 8;
      unsigned short* to = reinterpret_cast<unsigned short*>(p.o) + first * DV;
      for (int u = tid - 64; u < nrows * PIECES; u += 256) {
        const int row = u / PIECES, c = u % PIECES;
        *reinterpret_cast<uint4*>(to + row * DV + c * 8) = *reinterpret_cast<const uint4*>(sm + row * C::OROW + c * 16);
      }
    }
  }

  if (work == 0) {
    // An error, a chunk that the block's rows see nothing of, or no keys.
    for (int u = tid; u < nrows * DV; u += kLuThreads) {
      const int row = u / DV, d = u % DV;
      const long long item = latent_item(p, q.row0, rbase + row, 0);
      if (live > 1) {
        if (d == 0) {
          const long long si = latent_part(p, s, q.row0, q.n, chunk) + item;
          p.ws_ml[2 * si] = q.err ? NAN : -INFINITY;
          p.ws_ml[2 * si + 1] = q.err ? NAN : 0.f;
        }
      } else {
        reinterpret_cast<unsigned short*>(p.o)[item * DV + d] = q.err ? 0x7fffu : 0u;
        if (d == 0) p.lse[item] = q.err ? NAN : -INFINITY;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*abort_p) settle();
  if (warp == 1) tmem_dealloc(tm, 512);
}

// ---------------------------------------------------------------------------
cudaError_t launch_latent_umma(const LatentParams& p, dim3 grid, cudaStream_t st) {
  static std::atomic<unsigned long long> ready{0ull};
  cudaError_t e = allow_smem(latent_umma_kernel, LuCfg::SMEM, ready);
  if (e != cudaSuccess) return e;
  LuMaps m;
  memset(&m, 0, sizeof(m));
  if (!latent_query_map(&m.q, p, kLuM) || !latent_cache_map(&m.k, p)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kLuThreads);
  cfg.dynamicSmemBytes = LuCfg::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, latent_umma_kernel, p, m);
  return e != cudaSuccess ? e : cudaGetLastError();
}

int latent_umma_rows() { return kLuM; }

}  // namespace va
