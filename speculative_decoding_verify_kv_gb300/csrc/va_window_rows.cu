// Windowed verify attention for at most 16 query rows per KV head (direct
// rows and short drafts), bf16 and Q8_0 caches.
//
// With so few rows a call is bound by the bytes of the visible K and V: at
// G = 4, D = 128 a token of one KV head costs 512 bytes and 2 * 16 * 128
// multiply-adds, a hundredth of what the tensor cores do in that time.  So
// the work is cut for bytes in flight and for few dependent steps rather
// than for MMA size: a warp takes 16-token pages of its chunk in turn (warp
// w pages w, w + NW, ..), keeps its own ring of pages in shared memory,
// filled by TMA, and its own softmax state, and never waits for another warp
// until the end, when the warps' states are joined.  The products are warp
// MMAs of 16 x 8 x 16 with Q and the accumulator in registers (tcgen05 would
// need 128 rows and a round trip through tensor memory per tile).  64
// sequences of 4,100 visible tokens, H32/KV8/D128 bf16: 157 us, 6.8 TB/s (the
// 128-row kernel: 345).
#include "va_host.h"
#include "va_window_rows.cuh"

namespace va {

template <int D, int KVT, int NW>
struct FewCfg : PageCfg<D, KVT> {
  using C = PageCfg<D, KVT>;
  // CTAs to an SM, and as many ring stages as their share of its shared
  // memory holds, at most 6 (with two stages, one in use, too few bytes are in
  // flight: 257 us against 162 at D = 128).
  static constexpr int PER_SM = NW == 4 || D == 64 ? 2 : 1;
  static constexpr int BUDGET = 216 / PER_SM * 1024;
  static constexpr int FIT = BUDGET / (NW * C::STAGE);
  static constexpr int NST = FIT > 6 ? 6 : FIT;
  static constexpr int EPI = NW * kTileRows * (D + 4) * 4;  // the warps' O rows at the end
  static constexpr int RING = NW * NST * C::STAGE;
  static constexpr int SMEM = (RING > EPI ? RING : EPI) + 1024;
};

template <int D, int KVT, int NW, bool EX>
__global__ void __launch_bounds__(NW * 32, (FewCfg<D, KVT, NW>::PER_SM == 1 ? 0 : 2)) window_rows_kernel(const Params p, const __grid_constant__ CUtensorMap tmK,
                                                              const __grid_constant__ CUtensorMap tmV) {
  using C = FewCfg<D, KVT, NW>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[NW][C::NST];
  __shared__ float m_s[NW][kTileRows], l_s[NW][kTileRows];
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
  const int mine = pages > warp ? (pages - warp + NW - 1) / NW : 0;  // this warp's pages

  if (tid == 0) {
    err_s = 0;
    abort_s = 0;
    for (int w = 0; w < NW; ++w)
      for (int i = 0; i < C::NST; ++i) mbar_init(smem_u32(&bars[w][i]), 1);
    fence_barrier_init();
  }
  __syncthreads();

  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* ring = base + warp * C::NST * C::STAGE;
  // The pages' places, 32 of this warp's at a time, one per lane.
  auto lookup = [&](int i) {
    if (i >= mine) return -1;
    const int at = page_place(p, ws, s, slo / kPage + warp + i * NW);
    if (at < 0) atomicOr(&err_s, (int)VA_DEV_BAD_BLOCK);
    return at;
  };
  int place = lookup(lane);
  const uint64_t pol = policy_evict_first();
  auto load = [&](int i, int at) {  // page i of this warp into its stage; one lane
    const uint32_t bar = smem_u32(&bars[warp][i % C::NST]), dst = smem_u32(ring + (i % C::NST) * C::STAGE);
    mbar_arrive_expect_tx(bar, 2 * C::TILE);
    load_half<D, KVT>(p, &tmK, false, s, kvh, at, dst, bar, pol);
    load_half<D, KVT>(p, &tmV, true, s, kvh, at, dst + C::TILE_S, bar, pol);
  };
  // A bad entry loads nothing and stops the warp's loop at that page.
  int good = mine;
#pragma unroll
  for (int i = 0; i < C::NST; ++i) {
    const int at = __shfl_sync(0xffffffffu, place, i);
    if (i < good && at < 0) good = i;
    if (i < good && lane == 0) load(i, at);
  }
  RowTile<D, KVT, EX> rows;
  if (!rows.init(p, ws, row0, ctx, kind, kvh, 0, R, !err)) atomicOr(&err_s, (int)VA_DEV_BAD_PARENT);
  const int edge = win_low(p, ctx + n - 1) - ws.skip;
  volatile int* abort_p = &abort_s;

#pragma unroll 1
  for (int i = 0; i < good; ++i) {
    const int st = i % C::NST;
    unsigned char* ks = ring + st * C::STAGE;
    unsigned char* vs = ks + C::TILE_S;
    if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&bars[warp][st]), (i / C::NST) & 1, abort_p, kPageWaitNs))) {
      if (lane == 0) {
        *abort_p = 1;
        flag(p.status, VA_DEV_TIMEOUT);
      }
      break;
    }
    const int u0 = slo + (warp + i * NW) * kPage;  // the page's first span token
    const int tail = min(shi - u0, kPage);         // tokens of the chunk in it
    if (tail < kPage || (u0 < ws.dead_hi && u0 + kPage > ws.dead_lo))
      clear_unseen<D, KVT>(vs, u0, tail, ws.dead_lo, ws.dead_hi);
    typename RowTile<D, KVT, EX>::Page pg;
    rows.scores(pg, ks);
    rows.softmax(pg, p, kind, vctx, shi, edge, u0);
    rows.values(pg, p, vs);
    // The stage is free: the page NST further on.
    __syncwarp();
    const int nx = i + C::NST;
    if ((nx & 31) == 0) place = lookup(nx + lane);
    const int at = __shfl_sync(0xffffffffu, place, nx & 31);
    if (nx < good && at < 0) good = nx;
    if (nx < good && lane == 0) load(nx, at);
  }
  // A wait that gave up: the copies still in flight land before anything
  // else happens to their memory.
  if (*abort_p && lane == 0) {
    int dummy = 0;
    for (int i = 0; i < C::NST && i < good; ++i) {
      mbar_wait(smem_u32(&bars[warp][i]), 0, &dummy, kPageWaitNs);
      mbar_wait(smem_u32(&bars[warp][i]), 1, &dummy, kPageWaitNs);
    }
  }
  __syncthreads();  // every ring is idle: its memory takes the O rows
  constexpr int LD = D + 4;
  float* os = reinterpret_cast<float*>(base);
  rows.store(os + warp * kTileRows * LD, LD, m_s[warp], l_s[warp]);
  __syncthreads();
  err |= (unsigned)err_s;
  if (err && tid == 0) flag(p.status, err);
  join_rows<D, NW, 1>(p, slot, row0, kvh, R, err || abort_s, os, LD, m_s, l_s);
}

template <int D, int KVT, int NW, bool EX>
static cudaError_t launch_few_t(Params& p, cudaStream_t st) {
  using C = FewCfg<D, KVT, NW>;
  static_assert(C::NST >= 2 && C::NST <= 6, "ring depth");
  static std::atomic<unsigned long long> ready{0ull};
  cudaError_t e = allow_smem(window_rows_kernel<D, KVT, NW, EX>, C::SMEM, ready);
  if (e != cudaSuccess) return e;
  CUtensorMap mk, mv;
  memset(&mk, 0, sizeof(mk));
  memset(&mv, 0, sizeof(mv));
  if (!C::kQ8 && !make_page_maps(p, &mk, &mv)) return cudaErrorInvalidValue;
  p.joined = chunks_join<window_rows_kernel<D, KVT, NW, EX>, kJoinFew>(p, NW * 32, C::SMEM, st);
  WindowLaunch l(p, NW * 32, C::SMEM, st);
  e = cudaLaunchKernelEx(&l.cfg, window_rows_kernel<D, KVT, NW, EX>, p, mk, mv);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Warps of a CTA.  D = 64: eight, two CTAs to an SM.  D = 128: with one chunk to
// a sequence (many sequences) four, two CTAs to an SM, so that one's start and
// end hide behind the other; with several (few sequences) eight, the whole SM.
// 64 direct rows of 4,100 tokens in one chunk (H32/KV8, bf16): 157 us with four
// warps, 172 with eight; 16 of them 66 and 46 (two chunks: 50).  D = 256: what
// the registers leave.
template <int D, int KVT, bool EX>
static cudaError_t launch_few(Params& p, cudaStream_t st) {
  if constexpr (D == 128)
    if (p.slots == 1) return launch_few_t<D, KVT, 4, EX>(p, st);
  return launch_few_t<D, KVT, D == 256 && KVT == VA_BF16 ? 6 : 8, EX>(p, st);
}

cudaError_t launch_window_rows(Params& p, cudaStream_t st) {
#define VA_FEW(DD)                                                                              \
  if (p.D == DD) {                                                                              \
    if (p.kv_dtype == VA_BF16)                                                                  \
      return p.o_bf16 ? launch_few<DD, VA_BF16, false>(p, st) : launch_few<DD, VA_BF16, true>(p, st); \
    if (p.kv_dtype == VA_Q8_0) return launch_few<DD, VA_Q8_0, false>(p, st);                    \
  }
  VA_FEW(64) VA_FEW(128) VA_FEW(256)
#undef VA_FEW
  return cudaErrorInvalidValue;
}

}  // namespace va
