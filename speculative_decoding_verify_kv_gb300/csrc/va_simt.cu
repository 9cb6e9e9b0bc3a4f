// CUDA-core split-KV partial kernel.
//
// One CTA owns (sequence, KV head, split, sub-chunk, block of 16 query rows)
// and walks its token range in tiles of 32 tokens: decode K/V into shared
// memory as fp32, score every (row, token) pair, mask, update the online
// softmax (m in log2 units, l) and accumulate P.V in registers.  It writes
// one fp32 partial (m, l, acc[D]) per (row, head) into its slot of the
// workspace; the merge kernel combines the slots.
//
// This is the kernel for the fp32 cache and for row blocks too small to
// fill a tensor-core tile; it serves every dtype, so tests can also run it
// as a second implementation next to the tensor-core kernel.
//
// Restated from: hipfire PR #817 "FA2 split-KV" sections "Summary" and
// "Performance" (split partials + merge), hipfire PR #695 alpineQ comments
// (one block serves several verifier rows from one KV fetch), lucebox PR
// #686 "State and commit invariants" (tree ancestry masks).
#include <string.h>

#include "va_common.cuh"
#include "va_host.h"

namespace va {

constexpr int kSimtRows = 16;    // query rows per CTA
constexpr int kSimtTile = 32;    // tokens per tile
constexpr int kSimtThreads = 128;
// Windowed calls, whatever their size: eight warps of two rows.  Against four of
// four rows, when both were measured: 2 sequences of 200 rows, G = 4, D = 64, 19
// us against 26 (few CTAs, each waiting for its tiles' steps); 800 rows over 8 KV
// heads at D = 128, where the CTAs fill the GPU, 92 against 81.
constexpr int kSimtWinThreads = 256;

// Floats from one K row of the tile to the next: the scores are read one
// value per lane and token, or (WIN) four.
template <int D, bool WIN>
struct SimtCfg {
  static constexpr int LDK = WIN ? D + 4 : D + 1;
  static constexpr int SMEM = (kSimtRows * D + kSimtTile * LDK + kSimtTile * D + kSimtRows * kSimtTile) * 4;
};

// WIN: a windowed call; token indexes then count the span of visible tokens
// (WinSpan).  A window is a few tiles, so a CTA is bound by the latency of a
// tile's dependent steps: 2 sequences of 200 rows, G = 4, D = 64, window 100, 19
// us (issue slots 31 % used).
template <int D, int KVT, bool WIN>
__global__ void __launch_bounds__(WIN ? kSimtWinThreads : kSimtThreads) simt_partial_kernel(const Params p) {
  constexpr int TH = WIN ? kSimtWinThreads : kSimtThreads;
  constexpr int WARPS = TH / 32, RW = kSimtRows / WARPS;  // rows of a warp: warp + WARPS i
  constexpr int NK = D / 32;  // accumulator columns per lane
  constexpr int LDK = SimtCfg<D, WIN>::LDK;
  extern __shared__ float sm[];
  float* Qs = sm;                              // [16][D]
  float* Ks = Qs + kSimtRows * D;              // [32][LDK]
  float* Vs = Ks + kSimtTile * LDK;            // [32][D]
  float* Ps = Vs + kSimtTile * D;              // [16][32]
  __shared__ float alpha_s[kSimtRows];
  __shared__ unsigned mask_s[kSimtRows];
  __shared__ int wlo_s[kSimtRows];
  __shared__ int bad_s;

  // The merge kernel may launch now; it waits for this grid to finish.
  asm volatile("griddepcontrol.launch_dependents;");
  // Programmatic dependent of the preceding work on the stream: nothing is
  // read or written before that work has completed.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kvh = blockIdx.y, s = blockIdx.z;

  int row0, n, ctx;
  unsigned err = check_sequence(p, s, &row0, &n, &ctx);
  if (err & VA_DEV_BAD_ROWS) {
    if (tid == 0) flag(p.status, err);
    return;  // the rows of this sequence are unknown
  }
  // Row block and chunk (one level of chunks: split 0, slot = chunk).
  int rb, sub, nsub;
  if (!cta_work(p, n, blockIdx.x, &rb, &sub, &nsub)) return;
  const int split = 0, slot = sub;
  const int R = n * p.G;
  const int rbase = rb * kSimtRows;
  if (rbase >= R) return;
  const int nrows = min(kSimtRows, R - rbase);
  const WinSpan ws = WIN ? win_span(p, ctx, n) : WinSpan{ctx + n, 0, 0, 0, 0};
  const int L = ws.len;
  const int vctx = WIN ? ctx - ws.skip : ctx;  // where the drafts start in the span
  const int kind = seq_kind_of(p, s);
  const bool scratch = uses_scratch(p, kind);  // drafts from the tree scratch KV

  if (tid == 0) bad_s = 0;
  __syncthreads();
  if (tid < nrows) {
    int j = (rbase + tid) / p.G;
    bool bad = false;
    mask_s[tid] = row_mask(kind, p.parent + row0, j, &bad);
    if (WIN && !bad) {
      wlo_s[tid] = win_low(p, ctx + (kind == 1 ? __popc(mask_s[tid]) - 1 : j)) - ws.skip;
      if (kind == 1) mask_s[tid] = window_mask(p, p.parent + row0, j, ctx, mask_s[tid]);
    }
    if (bad) atomicOr(&bad_s, 1);
  }
  __syncthreads();
  if (bad_s) err |= VA_DEV_BAD_PARENT;

  int lo, hi, slo, shi;
  split_range(L, p.S, split, &lo, &hi);
  sub_range(lo, hi, nsub, p.min_sub, sub, &slo, &shi);

  // Q rows of this block -> shared (fp32).
  for (int i = tid; i < nrows * D; i += TH) {
    int rl = i / D, d = i % D;
    int r = rbase + rl, j = r / p.G, g = r % p.G;
    long long qi = ((long long)(row0 + j) * p.H + (kvh * p.G + g)) * D + d;
    Qs[rl * D + d] = load_q(p, qi);
  }

  float m_run[RW], l_run[RW];
  float acc[RW][NK];
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    m_run[i] = -INFINITY;
    l_run[i] = 0.f;
#pragma unroll
    for (int k = 0; k < NK; ++k) acc[i][k] = 0.f;
  }

  if constexpr (WIN) {
    // The next tile's loads are under way while a tile is worked through: four
    // elements of K and V per thread and step.
    constexpr int NR = kSimtTile * (D / 4) / TH;
    float4 kx[NR], vx[NR];
    bool lost = false;  // a bad block-table entry
    auto load = [&](int t0) {
#pragma unroll
      for (int x = 0; x < NR; ++x) {
        const int i = tid + x * TH, tok = t0 + i / (D / 4), d = 4 * (i % (D / 4));
        kx[x] = vx[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (tok >= shi || (tok >= ws.dead_lo && tok < ws.dead_hi)) continue;  // seen by no row
        const bool draft = tok >= vctx && scratch;
        const long long row = draft ? scratch_row(p, row0, kvh, tok - vctx)
                                    : kv_row(p, s, kvh, tok >= ws.head ? tok + ws.skip : tok);
        const void* kb = draft ? p.dk : p.k;
        const void* vb = draft ? p.dv : p.v;
        if (row < 0) {
          lost = true;
        } else if (KVT == VA_F32) {
          kx[x] = reinterpret_cast<const float4*>(kb)[(row * D + d) / 4];
          vx[x] = reinterpret_cast<const float4*>(vb)[(row * D + d) / 4];
        } else {
          kx[x] = make_float4(load_kv<KVT>(kb, row, p.row_bytes, d), load_kv<KVT>(kb, row, p.row_bytes, d + 1),
                              load_kv<KVT>(kb, row, p.row_bytes, d + 2), load_kv<KVT>(kb, row, p.row_bytes, d + 3));
          vx[x] = make_float4(load_kv<KVT>(vb, row, p.row_bytes, d), load_kv<KVT>(vb, row, p.row_bytes, d + 1),
                              load_kv<KVT>(vb, row, p.row_bytes, d + 2), load_kv<KVT>(vb, row, p.row_bytes, d + 3));
        }
      }
    };
    // A chain's row block sees no token past its last row, nor (but for the
    // sinks) one before its first row's window.
    const int end = kind == 0 ? min(shi, vctx + (rbase + nrows - 1) / p.G + 1) : shi;
    const int see_lo = kind == 0 ? win_low(p, ctx + rbase / p.G) - ws.skip : 0;
    auto seen = [&](int t0) {  // the first tile from t0 on that the block sees
      if (t0 >= p.sinks && t0 + kSimtTile <= see_lo) t0 += (see_lo - t0) / kSimtTile * kSimtTile;
      return t0;
    };
    int t0 = seen(slo);
    if (!err && t0 < end) load(t0);
    while (!err && t0 < end) {
      __syncthreads();
#pragma unroll
      for (int x = 0; x < NR; ++x) {
        const int i = tid + x * TH, t = i / (D / 4), d = 4 * (i % (D / 4));
        *reinterpret_cast<float4*>(Ks + t * LDK + d) = kx[x];
        *reinterpret_cast<float4*>(Vs + t * D + d) = vx[x];
      }
      if (__syncthreads_or(lost)) {
        err |= VA_DEV_BAD_BLOCK;
        break;
      }
      const int tok = t0 + lane, next = seen(t0 + kSimtTile);
      if (next < end) load(next);
      t0 = next;
      if (warp >= nrows) continue;
      // Scores: lane = token, the warp's rows from one read of K
      // (rows past the block's last hold whatever the shared memory held and
      // are masked).
      float sc[RW], m_new[RW];
#pragma unroll
      for (int i = 0; i < RW; ++i) sc[i] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(Ks + lane * LDK + d);
#pragma unroll
        for (int i = 0; i < RW; ++i) {
          const float4 q = *reinterpret_cast<const float4*>(Qs + (warp + WARPS * i) * D + d);
          sc[i] = fmaf(q.w, k4.w, fmaf(q.z, k4.z, fmaf(q.y, k4.y, fmaf(q.x, k4.x, sc[i]))));
        }
      }
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        const int rl = warp + WARPS * i;
        const bool vis = rl < nrows && tok < shi &&
                         (tok < vctx || draft_visible(kind, mask_s[rl], (rbase + rl) / p.G, tok - vctx)) &&
                         (tok < p.sinks || tok >= wlo_s[rl] || (kind == 1 && tok >= vctx));
        sc[i] = vis ? sc[i] * p.scale_log2 : -INFINITY;
        m_new[i] = sc[i];
      }
      // The rows' reductions side by side: each step waits for a shuffle.
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < RW; ++i) m_new[i] = fmaxf(m_new[i], __shfl_xor_sync(0xffffffffu, m_new[i], o));
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        m_new[i] = fmaxf(m_run[i], m_new[i]);
        const float off = m_new[i] == -INFINITY ? 0.f : m_new[i];  // nothing seen yet: every P is 0
        const float alpha = exp2f(m_run[i] - off);
        const float pr = exp2f(sc[i] - off);
        l_run[i] = fmaf(l_run[i], alpha, pr);  // this lane's tokens
        m_run[i] = m_new[i];
        Ps[(warp + WARPS * i) * kSimtTile + lane] = pr;
#pragma unroll
        for (int k = 0; k < NK; ++k) acc[i][k] *= alpha;
      }
      __syncwarp();
      // acc[row][d] += sum_t P[row][t] V[t][d]; lane owns d = lane + 32 k.
#pragma unroll 2
      for (int t = 0; t < kSimtTile; t += 4) {
        float4 pv[RW];
#pragma unroll
        for (int i = 0; i < RW; ++i) pv[i] = *reinterpret_cast<const float4*>(Ps + (warp + WARPS * i) * kSimtTile + t);
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          const float* v = Vs + t * D + lane + 32 * k;
          const float v0 = v[0], v1 = v[D], v2 = v[2 * D], v3 = v[3 * D];
#pragma unroll
          for (int i = 0; i < RW; ++i)
            acc[i][k] = fmaf(pv[i].w, v3, fmaf(pv[i].z, v2, fmaf(pv[i].y, v1, fmaf(pv[i].x, v0, acc[i][k]))));
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < RW; ++i) l_run[i] += __shfl_xor_sync(0xffffffffu, l_run[i], o);
  } else if (!err) {
    for (int t0 = slo; t0 < shi; t0 += kSimtTile) {
      __syncthreads();
      // Decode the K/V tile; tokens past the range become zeros.
      for (int i = tid; i < kSimtTile * D; i += kSimtThreads) {
        int t = i / D, d = i % D;
        int tok = t0 + t;
        float kx = 0.f, vx = 0.f;
        if (tok < shi && tok >= ctx && scratch) {
          const long long row = scratch_row(p, row0, kvh, tok - ctx);
          kx = load_kv<KVT>(p.dk, row, p.row_bytes, d);
          vx = load_kv<KVT>(p.dv, row, p.row_bytes, d);
        } else if (tok < shi) {
          long long row = kv_row(p, s, kvh, tok);
          if (row < 0) {
            atomicOr(&bad_s, 2);
          } else {
            kx = load_kv<KVT>(p.k, row, p.row_bytes, d);
            vx = load_kv<KVT>(p.v, row, p.row_bytes, d);
          }
        }
        Ks[t * (D + 1) + d] = kx;
        Vs[t * D + d] = vx;
      }
      __syncthreads();
      if (bad_s & 2) {
        err |= VA_DEV_BAD_BLOCK;
        break;
      }
      // Scores: lane = token, rows warp + 4i.
      const int tok = t0 + lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rl = warp + 4 * i;
        if (rl >= nrows) continue;
        float dot = 0.f;
#pragma unroll 8
        for (int d = 0; d < D; ++d) dot = fmaf(Qs[rl * D + d], Ks[lane * (D + 1) + d], dot);
        bool vis = tok < shi &&
                   (tok < ctx || draft_visible(kind, mask_s[rl], (rbase + rl) / p.G, tok - ctx));
        float s2 = vis ? dot * p.scale_log2 : -INFINITY;
        float mt = s2;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
        float m_new = fmaxf(m_run[i], mt);
        float alpha = (m_new == -INFINITY) ? 1.f : exp2f(m_run[i] - m_new);
        float pr = vis ? exp2f(s2 - m_new) : 0.f;
        float ps = pr;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
        l_run[i] = l_run[i] * alpha + ps;
        m_run[i] = m_new;
        Ps[rl * kSimtTile + lane] = pr;
        if (lane == 0) alpha_s[rl] = alpha;
      }
      __syncthreads();
      // acc[row][d] = alpha * acc + sum_t P[row][t] V[t][d]; lane owns d = lane + 32k.
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rl = warp + 4 * i;
        if (rl >= nrows) continue;
        const float a = alpha_s[rl];
#pragma unroll
        for (int k = 0; k < NK; ++k) acc[i][k] *= a;
        for (int t = 0; t < kSimtTile; ++t) {
          const float pv = Ps[rl * kSimtTile + t];
#pragma unroll
          for (int k = 0; k < NK; ++k) acc[i][k] = fmaf(pv, Vs[t * D + lane + 32 * k], acc[i][k]);
        }
      }
    }
  }
  if (err) {
    if (tid == 0) flag(p.status, err);
  }
  // Write this CTA's slot for its rows (an empty range writes l = 0).
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const int rl = warp + WARPS * i;
    if (rl >= nrows) continue;
    const int r = rbase + rl, j = r / p.G, g = r % p.G;
    const int grow = row0 + j, h = kvh * p.G + g;
    const long long si = slot_index(p, slot, grow, h);
    if (lane == 0) {
      p.ws_ml[2 * si] = err ? NAN : m_run[i];
      p.ws_ml[2 * si + 1] = err ? NAN : l_run[i];
    }
    float* dst = p.ws_acc + si * D;
#pragma unroll
    for (int k = 0; k < NK; ++k) dst[lane + 32 * k] = acc[i][k];
  }
}

template <int D, int KVT, bool WIN>
static cudaError_t launch_simt_t(const Params& p, dim3 grid, cudaStream_t st) {
  constexpr int smem = SimtCfg<D, WIN>::SMEM;
  static std::atomic<unsigned long long> ready{0ull};
  cudaError_t allowed = allow_smem(simt_partial_kernel<D, KVT, WIN>, smem, ready);
  if (allowed != cudaSuccess) return allowed;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3(WIN ? kSimtWinThreads : kSimtThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, simt_partial_kernel<D, KVT, WIN>, p);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

int simt_smem_bytes(int D) {
  switch (D) {
    case 64: return SimtCfg<64, false>::SMEM;
    case 128: return SimtCfg<128, false>::SMEM;
    default: return SimtCfg<256, false>::SMEM;
  }
}

cudaError_t launch_simt_partial(const Params& p, dim3 grid, cudaStream_t st) {
#define VA_SIMT_CASE(DD, KT)                                                  \
  if (p.D == DD && p.kv_dtype == KT)                                          \
    return p.window > 0 ? launch_simt_t<DD, KT, true>(p, grid, st)            \
                        : launch_simt_t<DD, KT, false>(p, grid, st);
  VA_SIMT_CASE(64, VA_F32) VA_SIMT_CASE(64, VA_BF16) VA_SIMT_CASE(64, VA_Q8_0)
  VA_SIMT_CASE(128, VA_F32) VA_SIMT_CASE(128, VA_BF16) VA_SIMT_CASE(128, VA_Q8_0)
  VA_SIMT_CASE(256, VA_F32) VA_SIMT_CASE(256, VA_BF16) VA_SIMT_CASE(256, VA_Q8_0)
#undef VA_SIMT_CASE
  return cudaErrorInvalidValue;
}

}  // namespace va
