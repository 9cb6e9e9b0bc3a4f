// Tensor-core attention over latent caches for few query rows (n rows x H heads
// of a sequence at most 32): bf16, tokens on the MMA's M axis.
//
// Per tile of 64 tokens, with N = 16 or 32 query rows (padded):
//   S^T = C Q^T      M = 64 tokens, A = the tile's column blocks (K-major)
//   softmax          a token per thread, its N scores in registers
//   O^T += V^T P^T   M = 128 value columns, A = the same column blocks, read
//                    transposed (MN-major), B = P^T from shared memory
// so a CTA holds all of O (DV / 128 times N columns of TMEM) and reads each byte
// of the cache once, where the 128-row kernel would load it twice and multiply
// rows that are not there.  Bound by the bytes of the cache: tiles are small so
// that three of them fit, one worked through while two are on their way (tiles of
// 128 tokens and M = 128: 64 sequences of 4,096 tokens, 16 heads, 82 us).
//
// Rows are columns here, so a running maximum over tokens would be a reduction
// over lanes in every tile.  The reference m of a row's exponents instead stays
// until some score exceeds it by 2^8 (or the row sees its first token): a test
// within each thread and one barrier per tile; the reduction, and the rescaling
// of O, only then.  Row sums stay spread over the threads until the end.
//
// Rings in shared memory: the key's rope blocks, and pairs of value blocks (128
// columns, the M of the second product), freed as O^T's blocks are done.
//
// Waits are bounded, as in the 128-row kernel.
#include <string.h>

#include "va_latent_mma.cuh"

namespace va {

constexpr int kLrTile = 64;
constexpr int kLrThreads = 256;  // two producers, two issuers, four softmax warps

template <int DV_, int N_>
struct LrCfg {
  static constexpr int DV = DV_, DK = DV + kLatentRope, N = N_;
  static constexpr int BLK = kLrTile * 128;        // a 64-column block of a tile
  static constexpr int MB = DV / 128;              // pairs of value blocks
  static constexpr int NV = N == 16 ? 11 : 10;     // pairs in the ring
  static constexpr int NK = N == 16 ? 3 : 2;       // rope blocks in the ring
  static constexpr int QBLK = N * 128;
  static constexpr int OFF_V = 0;
  static constexpr int OFF_K = NV * 2 * BLK;
  static constexpr int OFF_Q = OFF_K + NK * BLK;
  static constexpr int OFF_P = OFF_Q + DK / 64 * QBLK;  // [2][N][64 tokens]
  static constexpr int OFF_F = OFF_P + 2 * QBLK;        // float: m[N], factor[N], per-warp[4][N]; int: see[N]
  static constexpr int OFF_BAR = OFF_F + 7 * N * 4;
  static constexpr int NB = 11 + 2 * NV + 2 * NK;
  static constexpr int SMEM = OFF_BAR + NB * 8 + 16;
  static constexpr int COL_S = MB * N;
  static constexpr int COLS = MB * N + 2 * N <= 128 ? 128 : 256;
  static_assert(SMEM <= 232448, "shared memory");
  static_assert(NV >= MB + 1 && MB % 2 == 0, "a pair to load beside the tile's");
};

enum { RB_QLAND = 0, RB_SFULL = 1, RB_SREAD = 3, RB_PFULL = 5, RB_PFREE = 7, RB_OFINAL = 9, RB_SDRAIN = 10, RB_RING = 11 };

struct LrMaps {
  CUtensorMap q, k;
};

// Whether any of the 128 threads says so.
__device__ __forceinline__ bool any_of_four_warps(int id, bool mine) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)mine), "r"(id)
      : "memory");
  return r != 0;
}

template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t at, uint32_t (&r)[N]) {
  if constexpr (N == 16) tmem_ld16(at, r);
  else tmem_ld32(at, r);
}
template <int N>
__device__ __forceinline__ void tmem_st_n(uint32_t at, const uint32_t (&r)[N]) {
  if constexpr (N == 16) tmem_st16(at, r);
  else tmem_st32(at, r);
}

// The lanes' N values v[n] combined over the warp (op: sum or maximum), by halves:
// each step keeps half of the values, so N shuffles at most instead of 5 N (code
// that runs once is paid for by its size).  Lane l returns value l (N = 32) or
// l / 2 (N = 16).
template <int N, int BIT, class Op>
__device__ __forceinline__ float combine_lanes(const float (&v)[N], int lane, Op op) {
  if constexpr (N == 1) {
    float x = v[0];
#pragma unroll
    for (int o = BIT; o > 0; o >>= 1) x = op(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
  } else {
    float half[N / 2];
    const bool up = (lane & BIT) != 0;
#pragma unroll
    for (int n = 0; n < N / 2; ++n) {
      const float other = __shfl_xor_sync(0xffffffffu, up ? v[n] : v[n + N / 2], BIT);
      half[n] = op(up ? v[n + N / 2] : v[n], other);
    }
    return combine_lanes<N / 2, BIT / 2>(half, lane, op);
  }
}

template <class C>
__global__ void __launch_bounds__(kLrThreads, 1) latent_rows_kernel(const LatentParams p, const __grid_constant__ LrMaps maps) {
  constexpr int N = C::N, MB = C::MB;
  extern __shared__ __align__(1024) unsigned char sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::OFF_BAR);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(sm + C::OFF_BAR + C::NB * 8);
  volatile int* abort_p = reinterpret_cast<volatile int*>(tmem_at + 1);
  int* err_s = reinterpret_cast<int*>(tmem_at + 2);
  float* m_s = reinterpret_cast<float*>(sm + C::OFF_F);
  float* f_s = m_s + N;
  float* w_s = f_s + N;  // [4][N]
  int* see_s = reinterpret_cast<int*>(w_s + 4 * N);  // chain: drafts that a row sees; tree: its ancestors, as bits

  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  if (warp == 0) {
    if (lane == 0) {
      *err_s = 0;
      *abort_p = 0;
      prefetch_map(&maps.q);
      prefetch_map(&maps.k);
    }
    for (int i = lane; i < C::NB; i += 32) mbar_init(bar(i), i >= RB_SREAD && i < RB_PFREE ? 4 : 1);
    fence_barrier_init();
    __syncwarp();
  }
  // Nothing but this CTA's own shared memory is touched before the work ahead
  // on the stream has completed.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int s = blockIdx.z, chunk = blockIdx.x;
  const LatentSeq q = latent_seq(p, s);
  if (q.err & VA_DEV_BAD_ROWS) {
    if (tid == 0) flag(p.status, q.err);
    if (chunk == 0) latent_nan_rows(p, s, 0, p.H, threadIdx.x, blockDim.x);
    return;
  }
  const int R = q.n * p.H;
  const int live = latent_live(p, q.err ? 0 : q.len, latent_chunks(p, q.n));
  if (R == 0 || chunk >= live) return;
  // Columns behind the sequence's rows hold what stands there in memory (other
  // sequences' queries): a reference that no score exceeds, so that they move none.
  if (tid < N) m_s[tid] = tid < R ? -INFINITY : INFINITY;
  int lo, hi;
  latent_range(p, q.len, latent_chunks(p, q.n), chunk, &lo, &hi);
  const int ntiles = q.err ? 0 : (hi - lo + kLrTile - 1) / kLrTile;
  const int all_see = q.kind == 1 ? min(hi, q.ctx) : min(hi, q.ctx + 1);

  auto vfull = [&](int i) { return bar(RB_RING + i); };
  auto vfree = [&](int i) { return bar(RB_RING + C::NV + i); };
  auto kfull = [&](int i) { return bar(RB_RING + 2 * C::NV + i); };
  auto kfree = [&](int i) { return bar(RB_RING + 2 * C::NV + C::NK + i); };
  const uint32_t base = smem_u32(sm);

  // A producer's lane l: (row, plane) of page l of the tile at t0, in the cache's map.
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
  if ((warp == 0 || warp == 7) && ntiles > 0) blk0 = look_up(lo);
  if (warp == 0 && ntiles > 0) {
    // The queries, at once: their barrier was set up by this warp.
    const uint32_t one = elected();
    const int qrow = __shfl_sync(0xffffffffu, q.row0 * p.H, 0);
    expect_by(one, bar(RB_QLAND), C::DK / 64 * C::QBLK);
#pragma unroll
    for (int c = 0; c < C::DK / 64; ++c) tma_2d_by(one, base + C::OFF_Q + c * C::QBLK, &maps.q, c * 64, qrow, bar(RB_QLAND));
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_at), C::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = __shfl_sync(0xffffffffu, *tmem_at, 0);
  const int work = __shfl_sync(0xffffffffu, ntiles, 0);
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
    // nothing to read
  } else if (warp == 0 || warp == 7) {
    // ---------------------------------------------------------------- producers
    // Warp 0: the rope blocks and even pairs.  Warp 7: odd pairs.
    // (A copy is one block of one page, 36 to a tile: issued by one warp, they
    // were what the call waited for.)
    const int who = warp == 0 ? 0 : 1;
    const uint32_t one = elected();
    const int lo_u = __shfl_sync(0xffffffffu, lo, 0), hi_u = __shfl_sync(0xffffffffu, hi, 0);
    bool ok = true;
    int nk = 0, nv = who;  // rope blocks issued; the next pair
    int sk = 0, sv = who;
    uint32_t pk = 1, pv = 1;
    for (int i = 0; i < work && ok; ++i) {
      const int t0 = lo_u + i * kLrTile;
      const int pages = (min(kLrTile, hi_u - t0) + kPage - 1) / kPage;
      const int2 mine = page_at(t0, i == 0 ? blk0 : look_up(t0));
      if (late) found(late);  // before anything of the tile is loaded
      __syncwarp();
      int2 at[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) at[g] = make_int2(__shfl_sync(0xffffffffu, mine.x, g), __shfl_sync(0xffffffffu, mine.y, g));
      if (who == 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(kfree(sk), pk, abort_p, kLatentWaitNs));
        if (!ok) break;
        expect_by(one, kfull(sk), (uint32_t)(pages * kPage * 128));
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (g >= pages) break;
          tma_3d_by(one, base + C::OFF_K + sk * C::BLK + g * kPage * 128, &maps.k, C::DV, at[g].x, at[g].y, kfull(sk));
        }
        ++nk;
        if (++sk == C::NK) sk = 0, pk ^= 1;
      }
#pragma unroll
      for (int h = 0; h < MB / 2; ++h) {
        ok = __all_sync(0xffffffffu, ok && mbar_wait(vfree(sv), pv, abort_p, kLatentWaitNs));
        if (!ok) break;
        const uint32_t b = vfull(sv), dst = base + C::OFF_V + sv * 2 * C::BLK;
        const int col = (2 * h + who) * 128;
        expect_by(one, b, (uint32_t)(2 * pages * kPage * 128));
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (g >= pages) break;
          tma_3d_by(one, dst + g * kPage * 128, &maps.k, col, at[g].x, at[g].y, b);
          tma_3d_by(one, dst + C::BLK + g * kPage * 128, &maps.k, col + 64, at[g].x, at[g].y, b);
        }
        nv += 2;
        sv += 2;
        if (sv >= C::NV) sv -= C::NV, pv ^= 1;
      }
    }
    if (!ok && lane == 0) fail();
    // No copy may still be landing when the CTA goes away.
    if (*abort_p && lane == 0) {
      if (who == 0) {
        drain(bar(RB_QLAND), 0);
        for (int i = max(0, nk - C::NK); i < nk; ++i) drain(kfull(i % C::NK), (i / C::NK) & 1);
      }
      for (int i = nv - 2; i >= max(0, nv - 1 - C::NV); i -= 2) drain(vfull(i % C::NV), (i / C::NV) & 1);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- S issuer
    constexpr uint32_t ID = idesc_f16(kLrTile, N, true, false);
    const uint32_t one = elected();
    bool ok = __all_sync(0xffffffffu, mbar_wait(bar(RB_QLAND), 0, abort_p, kLatentWaitNs));
    bool any = false;
    int sk = 0, sv = 0;
    uint32_t pk = 0, pv = 0;
    const uint64_t qd = sdesc_sw128(base + C::OFF_Q, 16, 1024);
    const uint64_t kd0 = sdesc_sw128(base + C::OFF_K, 16, 1024), vd0 = sdesc_sw128(base + C::OFF_V, 16, 1024);
    for (int i = 0; i < work && ok; ++i) {
      const int b = i & 1;
      const uint32_t scol = tm + C::COL_S + b * N;
      ok = (i < 2 || mbar_wait(bar(RB_SREAD + b), ((i - 2) >> 1) & 1, abort_p, kLatentWaitNs)) &&
           mbar_wait(kfull(sk), pk, abort_p, kLatentWaitNs);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint64_t kd = kd0 + (uint64_t)((sk * C::BLK) >> 4);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_ss_by(one, scol, kd + kk * 2, qd + (uint64_t)((MB * 2 * C::QBLK) >> 4) + kk * 2, ID, kk > 0 ? 1u : 0u);
      any = true;
      commit_by(one, kfree(sk));
      if (++sk == C::NK) sk = 0, pk ^= 1;
#pragma unroll
      for (int c = 0; c < MB; ++c) {
        ok = __all_sync(0xffffffffu, mbar_wait(vfull(sv), pv, abort_p, kLatentWaitNs));
        if (!ok) break;
        tc_fence_after();
        const uint64_t vd = vd0 + (uint64_t)((sv * 2 * C::BLK) >> 4);
        if (++sv == C::NV) sv = 0, pv ^= 1;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ss_by(one, scol, vd + (uint64_t)(((kk >> 2) * C::BLK + (kk & 3) * 32) >> 4),
                    qd + (uint64_t)(((c * 2 + (kk >> 2)) * C::QBLK + (kk & 3) * 32) >> 4), ID, 1u);
      }
      if (!ok) break;
      commit_by(one, bar(RB_SFULL + b));
    }
    if (!ok && lane == 0) fail();
    if (!ok && any) {
      // What was issued completes before TMEM and shared memory go.  (A commit is
      // for what its own thread has issued.)
      commit_by(one, bar(RB_SDRAIN));
      drain(bar(RB_SDRAIN), 0);
    }
  } else if (warp == 6) {
    // ---------------------------------------------------------------- P.V issuer
    constexpr uint32_t ID = idesc_f16(128, N, true, false, true);
    const uint32_t one = elected();
    bool ok = true, any = false;
    int sv = 0;
    const uint64_t vd0 = sdesc_sw128(base + C::OFF_V, C::BLK, 1024), pd0 = sdesc_sw128(base + C::OFF_P, 16, 1024);
    for (int i = 0; i < work; ++i) {
      // (S^T of the tile, and so P, came after its blocks had landed.)
      ok = __all_sync(0xffffffffu, mbar_wait(bar(RB_PFULL + (i & 1)), (i >> 1) & 1, abort_p, kLatentWaitNs));
      if (!ok) break;
      tc_fence_after();
      const uint64_t pd = pd0 + (uint64_t)(((i & 1) * C::QBLK) >> 4);
#pragma unroll
      for (int c = 0; c < MB; ++c) {
        const uint64_t vd = vd0 + (uint64_t)((sv * 2 * C::BLK) >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ss_by(one, tm + c * N, vd + (uint64_t)((kk * 2048) >> 4), pd + kk * 2, ID, i > 0 || kk > 0 ? 1u : 0u);
        commit_by(one, vfree(sv));
        if (++sv == C::NV) sv = 0;
      }
      any = true;
      commit_by(one, bar(RB_PFREE + (i & 1)));
    }
    if (!ok && lane == 0) fail();
    if (any) {
      // After every P.V, in a failed run too.
      commit_by(one, bar(RB_OFINAL));
      drain(bar(RB_OFINAL), 0);
    }
  } else {
    // ---------------------------------------------------------------- softmax
    const int quad = warp & 3;
    // A product of 64 rows stands in the first 16 lanes of each quadrant.
    const int th = quad * 32 + lane, tt = lane < 16 ? quad * 16 + lane : kLrTile;  // thread; the tile's token
    const bool token = lane < 16;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const float c_r = p.scale_log2;
    // nm: minus the reference, kUnseen while the row has seen nothing (any score
    // then exceeds it).
    constexpr float kUnseen = 1e30f;
    float l[N], nm[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      l[n] = 0.f;
      nm[n] = n < R ? kUnseen : -INFINITY;
    }
    if (th < N) {
      const int j = th < R ? th / p.H : 0;
      bool bad_parent = false;
      see_s[th] = q.kind == 0 ? j + 1 : (int)row_mask(1, p.parent + q.row0, j, &bad_parent);
      if (bad_parent) found(VA_DEV_BAD_PARENT);
    }
    bar_sync(3, 128);
    bool ok = true;
    // A failed wait does not leave the loop: its barriers are shared by the four warps.
    for (int i = 0; i < work; ++i) {
      const int b = i & 1;
      // Whether the product that read this tile's buffer of P^T is done.
      const bool free = i < 2 || mbar_peek(bar(RB_PFREE + b), ((i - 2) >> 1) & 1);
      if (ok && !__all_sync(0xffffffffu, mbar_wait(bar(RB_SFULL + b), (i >> 1) & 1, abort_p, kLatentWaitNs))) ok = false;
      tc_fence_after();
      uint32_t sr[N];
      tmem_ld_n<N>(tm + lanes + C::COL_S + b * N, sr);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(RB_SREAD + b));
      float z[N];  // score over the reference, in log2 units
      const int t = lo + i * kLrTile + tt;
      if (lo + (i + 1) * kLrTile <= all_see) {
#pragma unroll
        for (int n = 0; n < N; ++n) z[n] = token ? __uint_as_float(sr[n]) : -INFINITY;
      } else {
        const int a = t - q.ctx;  // its place among the drafts
        const bool in = token && t < hi;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const int see = see_s[n];
          const bool vis = in && (a < 0 || (q.kind == 0 ? a < see : ((unsigned)see >> (a & 31)) & 1u));
          z[n] = vis ? __uint_as_float(sr[n]) : -INFINITY;
        }
      }
      bool over = false;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        z[n] = fmaf(z[n], c_r, nm[n]);
        over = over || z[n] > 8.f;
      }
      if (any_of_four_warps(2, over)) {
        // New references: the rows' largest scores of this tile.  (Masked is -inf alone:
        // a score that is no number stays one, and the maximum passes it over.)
        float x[N];
#pragma unroll
        for (int n = 0; n < N; ++n) x[n] = z[n] == -INFINITY ? -INFINITY : __uint_as_float(sr[n]) * c_r;
        const float top = combine_lanes<N, 16>(x, lane, [](float x, float y) { return fmaxf(x, y); });
        w_s[quad * N + lane / (32 / N)] = top;
        bar_sync(3, 128);
        if (th < N) {
          const float mx = fmaxf(fmaxf(w_s[th], w_s[N + th]), fmaxf(w_s[2 * N + th], w_s[3 * N + th]));
          const float old = m_s[th];
          const bool up = mx > old + 8.f;
          f_s[th] = up && old != -INFINITY ? exp2f(old - mx) : 1.f;
          if (up) m_s[th] = mx;
        }
        bar_sync(3, 128);
        if (i > 0) {
          if (ok && !__all_sync(0xffffffffu, mbar_wait(bar(RB_PFREE + ((i - 1) & 1)), ((i - 1) >> 1) & 1, abort_p, kLatentWaitNs))) ok = false;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < MB; ++c) {
            uint32_t o[N];
            tmem_ld_n<N>(tm + lanes + c * N, o);
            tmem_wait_ld();
#pragma unroll
            for (int n = 0; n < N; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * f_s[n]);
            tmem_st_n<N>(tm + lanes + c * N, o);
          }
          tmem_wait_st();
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
          l[n] *= f_s[n];
          nm[n] = m_s[n] == -INFINITY ? kUnseen : -m_s[n];
          // Rounded as in every other tile: a row whose reference stays has the same
          // weights whichever row made the tile come here.
          z[n] = z[n] == -INFINITY ? -INFINITY : fmaf(__uint_as_float(sr[n]), c_r, nm[n]);
        }
      }
      if (ok && !__all_sync(0xffffffffu, free || mbar_wait(bar(RB_PFREE + b), ((i - 2) >> 1) & 1, abort_p, kLatentWaitNs))) ok = false;
      unsigned char* prow = sm + C::OFF_P + b * C::QBLK;
      const int at = tt >> 3, in8 = (tt & 7) * 2;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const float w = lu_ex2(z[n]);  // masked: 0
        l[n] += w;
        // bf16, as the matrix unit takes it (2^-8 of w at most, see the 128-row kernel).
        if (token) *reinterpret_cast<__nv_bfloat16*>(prow + n * 128 + ((at ^ (n & 7)) << 4) + in8) = __float2bfloat16_rn(w);
      }
      if (i == work - 1 && token && t >= hi) {
        // Tokens behind the range may hold anything: their V is cleared (S of
        // the tile is done, its blocks have landed).
#pragma unroll 1
        for (int c = 0; c < MB * 2; ++c) {
          unsigned char* row = sm + C::OFF_V + (((i * MB + c / 2) % C::NV) * 2 + (c & 1)) * C::BLK + tt * 128;
#pragma unroll
          for (int x = 0; x < 8; ++x) *reinterpret_cast<uint4*>(row + x * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(RB_PFULL + b));
    }
    if (ok && !__all_sync(0xffffffffu, mbar_wait(bar(RB_OFINAL), 0, abort_p, kLatentWaitNs))) ok = false;
    if (!ok && lane == 0) fail();
    tc_fence_after();
    // Row sums over the threads.
    w_s[quad * N + lane / (32 / N)] = combine_lanes<N, 16>(l, lane, [](float x, float y) { return x + y; });
    bar_sync(3, 128);
    const bool bad = *abort_p != 0 || *reinterpret_cast<volatile int*>(err_s) != 0;
    auto sum_of = [&](int n) { return (w_s[n] + w_s[N + n]) + (w_s[2 * N + n] + w_s[3 * N + n]); };
    const long long item0 = (long long)q.row0 * p.H, part = latent_part(p, s, q.row0, q.n, chunk);
    if (th < R) {
      const float sum = sum_of(th), m = m_s[th];
      if (live > 1) {
        const long long si = part + item0 + th;
        p.ws_ml[2 * si] = bad ? NAN : m;
        p.ws_ml[2 * si + 1] = bad ? NAN : sum;
      } else {
        p.lse[item0 + th] = bad ? NAN : sum != 0.f ? (m + log2f(sum)) * kLn2 : -INFINITY;
      }
    }
    // O^T: a lane per value column, so a warp stores 32 of a row's at once.
    if (th < R) f_s[th] = bad ? NAN : live > 1 ? 1.f : sum_of(th) != 0.f ? 1.f / sum_of(th) : 0.f;
    bar_sync(3, 128);
    const long long first = (live > 1 ? part + item0 : item0) * C::DV + th;
#pragma unroll 1
    for (int c = 0; c < MB; ++c) {
      uint32_t o[N];
      tmem_ld_n<N>(tm + lanes + c * N, o);
      tmem_wait_ld();
      if (live > 1) {
        float* to = p.ws_acc + first + c * 128;
#pragma unroll
        for (int n = 0; n < N; ++n)
          if (n < R) to[n * C::DV] = __uint_as_float(o[n]) * f_s[n];
      } else {
        __nv_bfloat16* to = reinterpret_cast<__nv_bfloat16*>(p.o) + first + c * 128;
#pragma unroll
        for (int n = 0; n < N; ++n)
          if (n < R) to[n * C::DV] = __float2bfloat16_rn(__uint_as_float(o[n]) * f_s[n]);
      }
    }
  }

  if (work == 0) {
    // An error (a chunk holds tokens, and a sequence with rows has some).
    for (int u = tid; u < R * C::DV; u += kLrThreads) {
      const long long item = (long long)q.row0 * p.H + u / C::DV;
      const int d = u % C::DV;
      if (live > 1) {
        if (d == 0) {
          const long long si = latent_part(p, s, q.row0, q.n, chunk) + item;
          p.ws_ml[2 * si] = p.ws_ml[2 * si + 1] = NAN;
        }
      } else {
        reinterpret_cast<unsigned short*>(p.o)[item * C::DV + d] = 0x7fffu;
        if (d == 0) p.lse[item] = NAN;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*abort_p) settle();
  if (warp == 1) tmem_dealloc(tm, C::COLS);
}

template <class C>
static cudaError_t launch_rows_latent(const LatentParams& p, dim3 grid, cudaStream_t st) {
  static std::atomic<unsigned long long> ready{0ull};
  cudaError_t e = allow_smem(latent_rows_kernel<C>, C::SMEM, ready);
  if (e != cudaSuccess) return e;
  LrMaps m;
  memset(&m, 0, sizeof(m));
  if (!latent_query_map(&m.q, p, C::N) || !latent_cache_map(&m.k, p)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kLrThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, latent_rows_kernel<C>, p, m);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Rows that the kernel takes, of a launch whose sequences have at most `rows`.
int latent_rows_rows(long long rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 0; }

cudaError_t launch_latent_rows(const LatentParams& p, dim3 grid, cudaStream_t st) {
  if (p.rows_per_block == 16)
    return p.DV == 512 ? launch_rows_latent<LrCfg<512, 16>>(p, grid, st) : launch_rows_latent<LrCfg<256, 16>>(p, grid, st);
  return p.DV == 512 ? launch_rows_latent<LrCfg<512, 32>>(p, grid, st) : launch_rows_latent<LrCfg<256, 32>>(p, grid, st);
}

}  // namespace va
