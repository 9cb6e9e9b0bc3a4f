// Windowed verify attention for more than 16 query rows per KV head over bf16
// caches, up to 48 at D = 64 and 32 at D = 128: drafts and trees of a few rows
// per head group.
//
// One CTA takes a chunk of one KV head for up to RT tiles of 16 rows.  Pages
// of 16 tokens go round one ring in shared memory, filled by a warp of its
// own; page i is consumed by the RT warps of page group i mod PG, one row tile
// each, so K and V are read from memory once for all rows and a warp never
// waits for another one's products.  The groups' softmax states are joined at
// the end.  Warp MMAs (16 x 8 x 16) rather than tcgen05 because a tile of 128
// rows would stand three quarters empty and each of its steps (scores out of
// tensor memory, P back, the accumulator's rescale) waits for the one before;
// here eight or twelve warps are at different pages at any time.  What bounds
// it is a warp's chain of steps per page (some 1.5 us, issue slots 40 % used);
// with more rows, or at D = 256, fewer pages are under way and the tcgen05
// kernel wins.  Measured against it, 32 sequences of 2,052 visible tokens, one
// chunk each: D = 64 (4 KV heads) 24 rows 22.5 us against 41, 48 rows 32 against
// 42; D = 128 (8 KV heads) 32 rows 80 us against 97.  Past the limits, when they
// were set: D = 64 64 rows 44 against 42; D = 128 48 rows 136 against 101; D = 256
// (4 KV heads) 24 rows 79 against 71.
// Four warps issue the loads: one thread took 150 ns a tensor copy.
#include "va_host.h"
#include "va_window_rows.cuh"

namespace va {

template <int D, int RT, int PG>
struct TileCfg : PageCfg<D, VA_BF16> {
  using C = PageCfg<D, VA_BF16>;
  static constexpr int WARPS = RT * PG;
  static constexpr int LOADERS = 4;  // warps that load
  static constexpr int THREADS = (WARPS + LOADERS) * 32;
  static constexpr int FIT = 200 * 1024 / C::STAGE;
  static constexpr int NST = FIT > 16 ? 16 : FIT;
  static constexpr int EPI = WARPS * kTileRows * (D + 4) * 4;
  static constexpr int RING = NST * C::STAGE;
  static constexpr int SMEM = (RING > EPI ? RING : EPI) + 1024;
};

template <int D, int RT, int PG, bool EX>
__global__ void __launch_bounds__((TileCfg<D, RT, PG>::THREADS), 1)
    window_tiles_kernel(const Params p, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV) {
  using C = TileCfg<D, RT, PG>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t full[C::NST], empty[C::NST];
  __shared__ float m_s[C::WARPS][kTileRows], l_s[C::WARPS][kTileRows];
  __shared__ int err_s, abort_s;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slot = blockIdx.x, kvh = blockIdx.y, s = blockIdx.z;

  int row0, n, ctx;
  unsigned err = check_sequence(p, s, &row0, &n, &ctx);
  if (err & VA_DEV_BAD_ROWS) {
    if (tid == 0) flag(p.status, err);
    if (p.joined && slot == 0) nan_rows<D>(p, s, kvh);
    return;
  }
  const int R = n * p.G;
  if (R == 0) return;
  const int kind = seq_kind_of(p, s);
  const WinSpan ws = win_span(p, ctx, n);
  const int vctx = ctx - ws.skip;
  int lo, hi, slo, shi;
  split_range(ws.len, 1, 0, &lo, &hi);
  sub_range(lo, hi, p.slots, p.min_sub, slot, &slo, &shi);
  const int pages = err ? 0 : max(0, (shi - slo + kPage - 1) / kPage);

  if (tid == 0) {
    err_s = 0;
    abort_s = 0;
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), RT);
    }
    fence_barrier_init();
  }
  __syncthreads();

  unsigned char* ring = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  volatile int* abort_p = &abort_s;
  auto fail = [&]() {
    if (lane == 0) {
      *abort_p = 1;
      flag(p.status, VA_DEV_TIMEOUT);
    }
  };
  constexpr int LD = D + 4;
  float* os = reinterpret_cast<float*>(ring);

  if (warp >= C::WARPS) {
    // ------------------------------------------------------------- loads
    const uint64_t pol = policy_evict_first();
    const int first = warp - C::WARPS;
    int place = -1, issued = 0;
    for (int k = 0; first + k * C::LOADERS < pages; ++k) {
      const int i = first + k * C::LOADERS, st = i % C::NST;
      if ((k & 31) == 0) {
        const int mine = i + lane * C::LOADERS;
        place = mine < pages ? page_place(p, ws, s, slo / kPage + mine) : 0;
        if (place < 0) atomicOr(&err_s, (int)VA_DEV_BAD_BLOCK);
      }
      const int at = __shfl_sync(0xffffffffu, place, k & 31);
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&empty[st]), ((i / C::NST) & 1) ^ 1, abort_p, kPageWaitNs))) {
        fail();
        break;
      }
      if (lane == 0) {
        // A bad entry loads nothing; what the rows make of the stage is
        // overwritten with NaN at the end.
        if (at < 0)
          mbar_arrive(smem_u32(&full[st]));
        else {
          const uint32_t dst = smem_u32(ring + st * C::STAGE), bar = smem_u32(&full[st]);
          mbar_arrive_expect_tx(bar, 2 * C::TILE);
          load_half<D, VA_BF16>(p, &tmK, false, s, kvh, at, dst, bar, pol);
          load_half<D, VA_BF16>(p, &tmV, true, s, kvh, at, dst + C::TILE_S, bar, pol);
        }
      }
      issued = i + 1;
    }
    if (*abort_p && lane == 0) {
      // The copies still in flight land before their memory is used again.
      int dummy = 0;
      for (int i = first; i < issued; i += C::LOADERS)
        if (i >= issued - C::NST)
          mbar_wait(smem_u32(&full[i % C::NST]), (i / C::NST) & 1, &dummy, kPageWaitNs);
    }
    __syncthreads();
  } else {
    // -------------------------------------------------------------- rows
    const int tile = warp % RT, grp = warp / RT;
    const int mine = min(max(R - tile * kTileRows, 0), kTileRows);
    RowTile<D, VA_BF16, EX> rows;
    if (!rows.init(p, ws, row0, ctx, kind, kvh, tile * kTileRows, mine, !err))
      atomicOr(&err_s, (int)VA_DEV_BAD_PARENT);
    const int edge = win_low(p, ctx + n - 1) - ws.skip;
#pragma unroll 1
    for (int i = grp; i < pages; i += PG) {
      const int st = i % C::NST;
      unsigned char* ks = ring + st * C::STAGE;
      unsigned char* vs = ks + C::TILE_S;
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&full[st]), (i / C::NST) & 1, abort_p, kPageWaitNs))) {
        fail();
        break;
      }
      if (mine > 0) {
        const int u0 = slo + i * kPage, tail = min(shi - u0, kPage);
        // Every row tile's warp clears for itself: the others' writes are
        // the same zeros.
        if (tail < kPage || (u0 < ws.dead_hi && u0 + kPage > ws.dead_lo))
          clear_unseen<D, VA_BF16>(vs, u0, tail, ws.dead_lo, ws.dead_hi);
        typename RowTile<D, VA_BF16, EX>::Page pg;
        rows.scores(pg, ks);
        rows.softmax(pg, p, kind, vctx, shi, edge, u0);
        rows.values(pg, p, vs);
        __syncwarp();
      }
      if (lane == 0) mbar_arrive(smem_u32(&empty[st]));
    }
    __syncthreads();  // the ring is idle: its memory takes the O rows
    rows.store(os + (grp * RT + tile) * kTileRows * LD, LD, m_s[grp * RT + tile], l_s[grp * RT + tile]);
  }
  __syncthreads();
  err |= (unsigned)err_s;
  if (err && tid == 0) flag(p.status, err);
  join_rows<D, PG, RT>(p, slot, row0, kvh, R, err || abort_s, os, LD, m_s, l_s);
}

template <int D, int RT, int PG, bool EX>
static cudaError_t launch_tiles_t(Params& p, cudaStream_t st) {
  using C = TileCfg<D, RT, PG>;
  static_assert(C::NST >= PG && C::SMEM <= 227 * 1024, "ring");
  static std::atomic<unsigned long long> ready{0ull};
  cudaError_t e = allow_smem(window_tiles_kernel<D, RT, PG, EX>, C::SMEM, ready);
  if (e != cudaSuccess) return e;
  CUtensorMap mk, mv;
  if (!make_page_maps(p, &mk, &mv)) return cudaErrorInvalidValue;
  p.joined = chunks_join<window_tiles_kernel<D, RT, PG, EX>, kJoinMany>(p, C::THREADS, C::SMEM, st);
  WindowLaunch l(p, C::THREADS, C::SMEM, st);
  e = cudaLaunchKernelEx(&l.cfg, window_tiles_kernel<D, RT, PG, EX>, p, mk, mv);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Most rows per KV head that the row tiles take (see above).
int window_tiles_rows(int D) { return D == 64 ? 48 : D == 128 ? 32 : 0; }

template <bool EX>
static cudaError_t launch_tiles(Params& p, cudaStream_t st) {
  const int tiles = (p.max_rows * p.G + kTileRows - 1) / kTileRows;
  if (p.D == 64) return tiles <= 2 ? launch_tiles_t<64, 2, 6, EX>(p, st) : launch_tiles_t<64, 3, 4, EX>(p, st);
  if (p.D == 128) return launch_tiles_t<128, 2, 4, EX>(p, st);
  return cudaErrorInvalidValue;
}

cudaError_t launch_window_tiles(Params& p, cudaStream_t st) {
  return p.o_bf16 ? launch_tiles<false>(p, st) : launch_tiles<true>(p, st);
}

}  // namespace va
