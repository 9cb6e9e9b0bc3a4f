// CUDA-core attention over latent caches and expanded prompt keys: fp32
// products and sums, the kernel of fp32 tensors (and, asked for by flag, of
// bf16 ones).
//
// One CTA owns 16 query rows and one chunk of tokens and walks it in tiles of
// 32.  Two warps share four rows: for the scores each takes half of the tile's
// tokens (a lane: one token, half of the key's columns), for the online softmax
// (m in log2 units, l) two of the rows, for the values half of the columns, in
// registers; so a value read from shared memory serves four rows.  (Two rows to
// a warp, all tokens and columns: 32 us for the 5 x 80 rows of 320 columns over
// some 500 tokens, bound by those reads.)  Over a latent cache the values are the
// first DV of the key's own columns, so a tile is loaded once.  The next tile's
// loads are under way while a tile is worked through.
// A chunk that is a sequence's only one writes o itself; others leave (m, l,
// acc) for the merge.
#include <string.h>

#include "va_latent.cuh"

namespace va {

constexpr int kLsRows = 16;
constexpr int kLsTile = 32;
constexpr int kLsThreads = 256;

template <int DK, int DV, bool PROMPT>
struct LsCfg {
  static constexpr int LDK = DK + 4;  // lanes of a float4 read of a column hit banks of their own
  static constexpr int LDS = kLsTile + 1, LDP = kLsRows + 4;
  static constexpr int SMEM = (kLsRows * DK + kLsTile * LDK + (PROMPT ? kLsTile * DV : 0) + kLsTile * LDP + kLsRows * LDS) * 4;
};

// Four elements at index i (a multiple of 4; rows start on 16 bytes).
template <typename T>
__device__ __forceinline__ float4 load4(const void* base, long long i) {
  if constexpr (sizeof(T) == 4) {
    return *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + i);
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(reinterpret_cast<const unsigned short*>(base) + i);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xffff0000u));
  }
}

// The two warps of a row group.
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }

template <typename T, int DK, int DV, bool PROMPT>
__global__ void __launch_bounds__(kLsThreads) latent_simt_kernel(const LatentParams p) {
  using C = LsCfg<DK, DV, PROMPT>;
  constexpr int RW = 4;                            // rows that two warps share
  constexpr int NC = DV / 2 / 32;                  // value columns per lane
  constexpr int CV = NC > 1 ? 2 : 1;               // side by side
  constexpr int ROW4 = (DK + (PROMPT ? DV : 0)) / 4;  // float4 pieces of a token's key and value
  constexpr int NL = (kLsTile * ROW4 + kLsThreads - 1) / kLsThreads;
  extern __shared__ __align__(16) float lsm[];
  float* Qs = lsm;
  float* Ks = Qs + kLsRows * DK;
  float* Vs = PROMPT ? Ks + kLsTile * C::LDK : Ks;
  constexpr int LDV = PROMPT ? DV : C::LDK;
  float* Ps = Ks + kLsTile * C::LDK + (PROMPT ? kLsTile * DV : 0);  // weights, [token][row]
  float* Ss = Ps + kLsTile * C::LDP;                                // scores, [row][token]
  __shared__ float f_s[kLsRows], m_s[kLsRows], l_s[kLsRows];
  __shared__ unsigned anc_s[kLsRows];
  __shared__ int parent_s[kMaxTreeRows];
  __shared__ int bad_s;

  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int head = blockIdx.y, s = blockIdx.z;
  const LatentSeq q = latent_seq(p, s);
  if (q.err & VA_DEV_BAD_ROWS) {
    if (tid == 0) flag(p.status, q.err);
    if (blockIdx.x == 0) latent_nan_rows(p, s, PROMPT ? head : 0, PROMPT ? 1 : p.H, threadIdx.x, blockDim.x);
    return;
  }
  const int R = latent_rows(p, q.n);
  const int blocks = (R + kLsRows - 1) / kLsRows;
  if (blocks == 0) return;
  const int nchunk = latent_chunks(p, q.n);
  const int rb = blockIdx.x % blocks, chunk = blockIdx.x / blocks;
  const int live = latent_live(p, q.err ? 0 : q.len, nchunk);
  if (chunk >= live) return;
  const int rbase = rb * kLsRows, nrows = min(kLsRows, R - rbase);
  int lo, hi;
  latent_range(p, q.len, nchunk, chunk, &lo, &hi);
  const int jlast = PROMPT ? rbase + nrows - 1 : (rbase + nrows - 1) / p.H;
  hi = max(lo, min(hi, latent_end(p, q, jlast)));
  unsigned err = q.err;

  float4 x[NL];
  bool lost = false;
  auto load = [&](int t0) {
#pragma unroll
    for (int k = 0; k < NL; ++k) {
      const int i = tid + k * kLsThreads, t = t0 + i / ROW4, d = i % ROW4 * 4;
      x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i >= kLsTile * ROW4 || t >= hi) continue;
      if (PROMPT) {
        const long long row = q.key0 + t;
        constexpr int NOPE = DK - kLatentRope;
        if (d < NOPE) x[k] = load4<T>(p.kv, (row * p.H + head) * (NOPE + DV) + d);
        else if (d < DK) x[k] = load4<T>(p.k_rope, row * p.kr_stride + d - NOPE);
        else x[k] = load4<T>(p.kv, (row * p.H + head) * (NOPE + DV) + d - kLatentRope);
      } else {
        const long long row = latent_row(p, s, t);
        if (row < 0) lost = true;
        else x[k] = load4<T>(p.cache, row * DK + d);
      }
    }
  };
  if (!err && lo < hi) load(lo);  // under way while queries and masks are fetched
  if (tid == 0) bad_s = 0;
  if (q.kind == 1 && tid < q.n) parent_s[tid] = p.parent[q.row0 + tid];
  __syncthreads();
  if (tid < nrows && q.kind == 1) {
    bool bad = false;
    anc_s[tid] = row_mask(1, parent_s, (rbase + tid) / p.H, &bad);
    if (bad) atomicOr(&bad_s, (int)VA_DEV_BAD_PARENT);
  }
  for (int i = tid; i < nrows * (DK / 4); i += kLsThreads) {
    const long long item = latent_item(p, q.row0, rbase + i / (DK / 4), head);
    *reinterpret_cast<float4*>(Qs + i * 4) = load4<T>(p.q, item * DK + i % (DK / 4) * 4);
  }
  for (int i = nrows * DK + tid; i < kLsRows * DK; i += kLsThreads) Qs[i] = 0.f;

  const int rg = warp & 3, half = warp >> 2;  // row group; which half of tokens, rows and columns
  float m_run[2], l_run[2], acc[RW][NC];      // m, l: rows 4 rg + 2 half and the next
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    m_run[i] = -INFINITY;
    l_run[i] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < RW; ++i)
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[i][c] = 0.f;
  __syncthreads();
  err |= (unsigned)bad_s;
  for (int t0 = lo; t0 < hi && !err; t0 += kLsTile) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NL; ++k) {
      const int i = tid + k * kLsThreads, t = i / ROW4, d = i % ROW4 * 4;
      if (i >= kLsTile * ROW4) continue;
      if (PROMPT && d >= DK) *reinterpret_cast<float4*>(Vs + t * LDV + d - DK) = x[k];
      else *reinterpret_cast<float4*>(Ks + t * C::LDK + d) = x[k];
    }
    if (__syncthreads_or(lost)) {
      err |= VA_DEV_BAD_BLOCK;
      break;
    }
    if (t0 + kLsTile < hi) load(t0 + kLsTile);
    if (rg * RW >= nrows) continue;
    {
      const int tok = half * 16 + (lane & 15), d0 = (lane >> 4) * (DK / 2);
      const float* kr = Ks + tok * C::LDK + d0;
      const float* qr = Qs + rg * RW * DK + d0;
      float sc[RW] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
      for (int d = 0; d < DK / 2; d += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(kr + d);
#pragma unroll
        for (int i = 0; i < RW; ++i) {
          const float4 q4 = *reinterpret_cast<const float4*>(qr + i * DK + d);
          sc[i] = fmaf(q4.w, k4.w, fmaf(q4.z, k4.z, fmaf(q4.y, k4.y, fmaf(q4.x, k4.x, sc[i]))));
        }
      }
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        sc[i] += __shfl_xor_sync(0xffffffffu, sc[i], 16);
        if (lane < 16) Ss[(rg * RW + i) * C::LDS + tok] = sc[i];
      }
    }
    pair_sync(1 + rg);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int rl = rg * RW + 2 * half + i;
      const int j = PROMPT ? rbase + rl : (rbase + rl) / p.H;
      const unsigned vis = rl < nrows ? latent_bits(p, q, q.kind == 1 ? anc_s[rl] : 0u, j, hi, t0) : 0u;
      const float sc = Ss[rl * C::LDS + lane];
      float mx = (vis >> lane) & 1u ? sc * p.scale_log2 : -INFINITY;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float m_new = fmaxf(m_run[i], mx);
      // The scale in two parts: rounded to one, it would move every score alike, by
      // 2^-25 of it, and a weight by some 10 times that.
      const float w = (vis >> lane) & 1u ? exp2f(fmaf(sc, p.scale_lo, fmaf(sc, p.scale_log2, -m_new))) : 0.f;
      const float f = m_run[i] == -INFINITY ? 0.f : exp2f(m_run[i] - m_new);
      float sum = w;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l_run[i] = l_run[i] * f + sum;
      m_run[i] = m_new;
      Ps[lane * C::LDP + rl] = w;
      if (lane == 0) f_s[rl] = f;
    }
    pair_sync(1 + rg);
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const float f = f_s[rg * RW + i];
#pragma unroll
      for (int c = 0; c < NC; ++c) acc[i][c] *= f;
    }
    const float* vr = Vs + half * (DV / 2) + CV * lane;
#pragma unroll 4
    for (int t = 0; t < kLsTile; ++t) {
      const float4 w4 = *reinterpret_cast<const float4*>(Ps + t * C::LDP + rg * RW);
      const float w[RW] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
      for (int c = 0; c < NC; c += CV) {
        float v[CV];
        if constexpr (CV == 2) {
          const float2 v2 = *reinterpret_cast<const float2*>(vr + t * LDV + 32 * c);
          v[0] = v2.x;
          v[1] = v2.y;
        } else {
          v[0] = vr[t * LDV + 32 * c];
        }
#pragma unroll
        for (int i = 0; i < RW; ++i)
#pragma unroll
          for (int e = 0; e < CV; ++e) acc[i][c + e] = fmaf(w[i], v[e], acc[i][c + e]);
      }
    }
  }
  if (err && tid == 0) flag(p.status, err);
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      m_s[rg * RW + 2 * half + i] = m_run[i];
      l_s[rg * RW + 2 * half + i] = l_run[i];
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const int rl = rg * RW + i;
    if (rl >= nrows) continue;
    const long long item = latent_item(p, q.row0, rbase + rl, head);
    const float l = l_s[rl], m = m_s[rl];
    const int col = half * (DV / 2) + CV * lane;
    if (live > 1) {
      const long long si = latent_part(p, s, q.row0, q.n, chunk) + item;
      if (lane == 0 && half == 0) {
        p.ws_ml[2 * si] = err ? NAN : m;
        p.ws_ml[2 * si + 1] = err ? NAN : l;
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) p.ws_acc[si * DV + col + 32 * (c / CV * CV) + c % CV] = acc[i][c];
      continue;
    }
    const float inv = err ? NAN : l != 0.f ? 1.f / l : 0.f;
    if (lane == 0 && half == 0) p.lse[item] = err ? NAN : l != 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const long long at = item * DV + col + 32 * (c / CV * CV) + c % CV;
      const float v = acc[i][c] * inv;
      if (sizeof(T) == 4) reinterpret_cast<float*>(p.o)[at] = v;
      else reinterpret_cast<__nv_bfloat16*>(p.o)[at] = __float2bfloat16_rn(v);
    }
  }
}

// Merge of a sequence's chunks: M over the chunks, then l and o with the
// weights 2^(m - M).  Which kernel merges follows from the most rows and chunks
// that the launch allows, and the order of the sums from that and the row's own
// partials alone.  Sequences of one chunk have their o already, rows of
// inconsistent sequences their NaN.
constexpr int kLmThreads = 256;
constexpr int kLmWarps = kLmThreads / 32;

// The sequence of item's row: the last that starts at or before it (32 at a
// time); -1 where none covers it.
__device__ __forceinline__ int latent_find(const LatentParams& p, int grow, int lane) {
  int s = -1;
  for (int s0 = 0; s0 < p.num_seqs; s0 += 32) {
    const unsigned m = __ballot_sync(0xffffffffu, s0 + lane < p.num_seqs && p.cu_rows[s0 + lane] <= grow);
    if (m) s = s0 + 31 - __clz(m);
  }
  return s >= 0 && grow < p.cu_rows[s + 1] ? s : -1;
}

__device__ __forceinline__ void latent_store4(const LatentParams& p, long long at, float4 v, float inv) {
  v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
  if (p.o_bf16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    uint2 w;
    memcpy(&w.x, &a, 4);
    memcpy(&w.y, &b, 4);
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.o) + at) = w;
  } else {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.o) + at) = v;
  }
}

// Takes chunks first, first + step, .. of the partials at si0, each `apart` behind the
// one before (B of them in flight at once: m, l and a float4 of acc together), into a
// running (M, l, acc) of the calling warp's lanes, NC columns of 4 to a lane from
// column col on.
template <int DV, int NC, int B>
__device__ __forceinline__ void latent_gather(const LatentParams& p, long long si0, long long apart, int live, int first, int step, int col,
                                              bool mine, float& M, float& l, float4 (&acc)[NC], bool& nan) {
  M = -INFINITY;
  l = 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  const float2* ml = reinterpret_cast<const float2*>(p.ws_ml) + (si0 + first * apart);
  const float* part = p.ws_acc + (si0 + first * apart) * DV + col;
  for (int s0 = first; s0 < live; s0 += B * step) {
    float mm[B], ll[B];
    float4 aa[B][NC];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const bool in = s0 + k * step < live;
      const float2 v = in ? *ml : make_float2(-INFINITY, 0.f);
      mm[k] = v.x;
      ll[k] = v.y;
#pragma unroll
      for (int c = 0; c < NC; ++c)
        aa[k][c] = in && mine ? *reinterpret_cast<const float4*>(part + 128 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
      ml += step * apart;
      part += step * apart * DV;
    }
    float bm = M;
#pragma unroll
    for (int k = 0; k < B; ++k) {
      if (isnan(mm[k]) || isnan(ll[k])) nan = true;
      if (ll[k] > 0.f) bm = fmaxf(bm, mm[k]);
    }
    const float f = M == -INFINITY ? 0.f : exp2f(M - bm);
    M = bm;
    l *= f;
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[c] = make_float4(acc[c].x * f, acc[c].y * f, acc[c].z * f, acc[c].w * f);
#pragma unroll
    for (int k = 0; k < B; ++k) {
      // A chunk that a row sees nothing of: its acc is not read as data.
      const float w = ll[k] > 0.f ? exp2f(mm[k] - M) : 0.f;
      if (!(w > 0.f)) continue;
      l = fmaf(w, ll[k], l);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        acc[c].x = fmaf(w, aa[k][c].x, acc[c].x);
        acc[c].y = fmaf(w, aa[k][c].y, acc[c].y);
        acc[c].z = fmaf(w, aa[k][c].z, acc[c].z);
        acc[c].w = fmaf(w, aa[k][c].w, acc[c].w);
      }
    }
  }
}

// What a warp or CTA of a merge has before it: whether (row, head) `item` has chunks to
// merge, and where they stand.  BY_SEQ: item counts among those of sequence s that can
// have some, else among all of the launch, and the sequence is searched for.  One that
// finds nothing to do costs about as much as one that does: 300 rows of 128 heads over
// 2,300 tokens, one chunk each, 156 us by all rows of the launch, 140 by sequence, 135
// without a merge.
struct LatentMerge {
  long long item, part, apart;
  int live;
};

template <bool BY_SEQ>
__device__ __forceinline__ bool latent_to_merge(const LatentParams& p, long long item, int s, int lane, LatentMerge* w) {
  if (!BY_SEQ) {
    if (item >= (long long)p.total_rows * p.H) return false;
    s = latent_find(p, (int)(item / p.H), lane);
    if (s < 0) return false;
  }
  const LatentSeq q = latent_seq(p, s);
  if (BY_SEQ) {
    if (item >= (long long)q.n * p.H) return false;
    item += (long long)q.row0 * p.H;
  }
  w->item = item;
  w->live = latent_live(p, q.len, latent_chunks(p, q.n));
  w->part = latent_part(p, s, q.row0, q.n, 0) + item;
  w->apart = latent_apart(p, q.n);
  return !q.err && w->live > 1;
}

// Few chunks: a warp per (row, head).
template <int DV, bool BY_SEQ>
__global__ void __launch_bounds__(kLmThreads) latent_merge_kernel(const LatentParams p) {
  constexpr int NC = DV / 128 > 0 ? DV / 128 : 1;  // (DV = 64: half the lanes)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31;
  LatentMerge w;
  if (!latent_to_merge<BY_SEQ>(p, (long long)blockIdx.x * kLmWarps + threadIdx.x / 32, blockIdx.z, lane, &w)) return;
  const long long item = w.item;
  const bool mine = DV >= 128 || lane < 16;
  float M, l;
  float4 acc[NC];
  bool nan = false;
  latent_gather<DV, NC, 4>(p, w.part, w.apart, w.live, 0, 1, 4 * lane, mine, M, l, acc, nan);
  const float inv = nan ? NAN : l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
    if (mine) latent_store4(p, item * DV + 4 * lane + 128 * c, acc[c], inv);
  if (lane == 0) p.lse[item] = nan ? NAN : l > 0.f ? (M + log2f(l)) * kLn2 : -INFINITY;
}

// Many chunks (of few rows): a CTA per (row, head) and 128 columns, each of its
// eight warps every eighth chunk, then the warps' sums in warp order.  With one
// warp to a row the merge of 64 chunks was more than half of the call.
template <int DV, bool BY_SEQ>
__global__ void __launch_bounds__(kLmThreads) latent_merge_many_kernel(const LatentParams p) {
  __shared__ float4 acc_s[kLmWarps][32];
  __shared__ float m_s[kLmWarps], l_s[kLmWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  LatentMerge at;
  if (!latent_to_merge<BY_SEQ>(p, blockIdx.x, blockIdx.z, lane, &at)) return;
  const long long item = at.item;
  const int col = blockIdx.y * 128 + 4 * lane;
  float M, l;
  float4 acc[1];
  bool nan = false;
  latent_gather<DV, 1, 8>(p, at.part, at.apart, at.live, warp, kLmWarps, col, col < DV, M, l, acc, nan);
  acc_s[warp][lane] = acc[0];
  if (lane == 0) {
    m_s[warp] = M;
    l_s[warp] = l;
  }
  nan = __syncthreads_or(nan) != 0;
  if (warp != 0) return;
  float Mall = -INFINITY;
#pragma unroll
  for (int w = 0; w < kLmWarps; ++w)
    if (l_s[w] > 0.f) Mall = fmaxf(Mall, m_s[w]);
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
#pragma unroll
  for (int w = 0; w < kLmWarps; ++w) {
    const float f = l_s[w] > 0.f ? exp2f(m_s[w] - Mall) : 0.f;
    const float4 x = acc_s[w][lane];
    sum = fmaf(f, l_s[w], sum);
    t = make_float4(fmaf(f, x.x, t.x), fmaf(f, x.y, t.y), fmaf(f, x.z, t.z), fmaf(f, x.w, t.w));
  }
  const float inv = nan ? NAN : sum > 0.f ? 1.f / sum : 0.f;
  if (col < DV) latent_store4(p, item * DV + col, t, inv);
  if (lane == 0 && blockIdx.y == 0) p.lse[item] = nan ? NAN : sum > 0.f ? (Mall + log2f(sum)) * kLn2 : -INFINITY;
}

template <typename K>
static cudaError_t launch_one(K kernel, dim3 grid, int threads, int smem, cudaStream_t st, const LatentParams& p) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int DK, int DV, bool PROMPT>
static cudaError_t launch_simt_t(const LatentParams& p, dim3 grid, cudaStream_t st) {
  static std::atomic<unsigned long long> ready{0ull};
  constexpr int smem = LsCfg<DK, DV, PROMPT>::SMEM;
  cudaError_t e = allow_smem(latent_simt_kernel<T, DK, DV, PROMPT>, smem, ready);
  if (e != cudaSuccess) return e;
  return launch_one(latent_simt_kernel<T, DK, DV, PROMPT>, grid, kLsThreads, smem, st, p);
}

template <typename T>
static cudaError_t launch_simt_of(const LatentParams& p, dim3 grid, cudaStream_t st) {
  if (p.prompt)
    return p.DV == 128 ? launch_simt_t<T, 192, 128, true>(p, grid, st) : launch_simt_t<T, 128, 64, true>(p, grid, st);
  return p.DV == 512 ? launch_simt_t<T, 576, 512, false>(p, grid, st) : launch_simt_t<T, 320, 256, false>(p, grid, st);
}

int latent_simt_rows() { return kLsRows; }

cudaError_t launch_latent_simt(const LatentParams& p, dim3 grid, cudaStream_t st) {
  return p.o_bf16 ? launch_simt_of<__nv_bfloat16>(p, grid, st) : launch_simt_of<float>(p, grid, st);
}

template <int DV, bool BY_SEQ>
static cudaError_t launch_merge_of(const LatentParams& p, cudaStream_t st) {
  const long long items = BY_SEQ ? p.merge_seq : (long long)p.total_rows * p.H;
  const unsigned seqs = BY_SEQ ? (unsigned)p.num_seqs : 1u;
  if (p.many)
    return launch_one(latent_merge_many_kernel<DV, BY_SEQ>, dim3((unsigned)items, (DV + 127) / 128, seqs), kLmThreads, 0, st, p);
  return launch_one(latent_merge_kernel<DV, BY_SEQ>, dim3((unsigned)((items + kLmWarps - 1) / kLmWarps), 1u, seqs), kLmThreads, 0, st, p);
}

template <int DV>
static cudaError_t launch_merge_dv(const LatentParams& p, cudaStream_t st) {
  return p.merge_seq ? launch_merge_of<DV, true>(p, st) : launch_merge_of<DV, false>(p, st);
}

cudaError_t launch_latent_merge(const LatentParams& p, cudaStream_t st) {
  switch (p.DV) {
    case 64: return launch_merge_dv<64>(p, st);
    case 128: return launch_merge_dv<128>(p, st);
    case 256: return launch_merge_dv<256>(p, st);
    default: return launch_merge_dv<512>(p, st);
  }
}

}  // namespace va
