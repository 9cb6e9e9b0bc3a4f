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
// need 128 rows and a round trip through tensor memory per tile).
//
// Per page, in base 2 (c = scale log2 e):
//   S = Q K^T          16 rows x 16 tokens, fp32
//   m' = max(m, max S c), a = 2^(m - m'), P = 2^(S c - m')
//   l <- a l + sum P,  O <- a O + P V
// P V starts from zero for every page and is added in fp32 registers, where
// the rescaling by a costs nothing more (one fused multiply-add): tensor
// cores round their running sum towards zero, which over the pages of a
// long window is a drift of 2^-24 each (1e-5 after 4,096 tokens, measured).
//
// bf16: a page is a K and a V tile, one tiled TMA load per 64 columns, 128-
// byte swizzle; P enters as bf16 hi + lo.  Q8_0: a page is two bulk copies of
// 16 raw rows; the codes enter the MMAs as exact fp16 integers, K's scales
// multiply the fp32 sums of each 32-element block, V's elements become
// fp16(d q) (one rounding) and P is fp16.
#include <limits.h>
#include <string.h>

#include <atomic>

#include "va_common.cuh"
#include "va_sm100.cuh"

namespace va {
using namespace sm100;

constexpr int kFewRows = 16;
constexpr uint64_t kFewWaitNs = 2000000000ull;

template <int D, int KVT, int NW>
struct FewCfg {
  static constexpr bool kQ8 = KVT == VA_Q8_0;
  static constexpr int RB = kQ8 ? D / 32 * 34 : D * 2;  // bytes of a cache row
  static constexpr int TILE = kPage * RB;               // one tensor's page
  // Stage: K and V of a page, each from a 1,024-byte boundary (swizzle).
  static constexpr int TILE_S = (TILE + 1023) / 1024 * 1024;
  static constexpr int STAGE = 2 * TILE_S;
  // Ring depth: as many stages as leave the CTA its share of an SM (2 warps:
  // a quarter, or half where a quarter holds no two stages), at most 4.
  static constexpr int BUDGET = (NW > 2 ? 216 : 54 * 1024 / (NW * STAGE) >= 2 ? 54 : 108) * 1024;
  static constexpr int FIT = BUDGET / (NW * STAGE);
  static constexpr int NST = FIT > 4 ? 4 : FIT;
  static constexpr int EPI = NW * kFewRows * (D + 4) * 4;  // the warps' O rows at the end
  static constexpr int RING = NW * NST * STAGE;
  static constexpr int SMEM = (RING > EPI ? RING : EPI) + 1024;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  if (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  __half2 h = __floats2half2_rn(a, b);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}

__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b) {
  __half2 x, y;
  memcpy(&x, &a, 4);
  memcpy(&y, &b, 4);
  x = __hsub2(x, y);
  memcpy(&a, &x, 4);
  return a;
}

__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
  __half2 x, y;
  memcpy(&x, &a, 4);
  memcpy(&y, &b, 4);
  x = __hmul2(x, y);
  memcpy(&a, &x, 4);
  return a;
}

constexpr uint32_t kBias = 0x64806480u;  // fp16 1152 twice: 0x6400 | (q + 128) is 1152 + q

// The word of four codes at byte address p (even), biased to q + 128.
__device__ __forceinline__ uint32_t code_word(const unsigned char* p) {
  const uint32_t lo = *reinterpret_cast<const unsigned short*>(p);
  const uint32_t hi = *reinterpret_cast<const unsigned short*>(p + 2);
  return (lo | (hi << 16)) ^ 0x80808080u;
}

template <int D, int KVT, int NW>
__global__ void __launch_bounds__(NW * 32) window_rows_kernel(const Params p, const __grid_constant__ CUtensorMap tmK,
                                                              const __grid_constant__ CUtensorMap tmV) {
  using C = FewCfg<D, KVT, NW>;
  constexpr bool Q8 = C::kQ8;
  constexpr int KS = D / 16;  // k steps of S
  constexpr int NT = D / 8;   // column tiles of O
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t bars[NW][4];
  __shared__ float m_s[NW][kFewRows], l_s[NW][kFewRows];
  __shared__ int err_s, abort_s;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, q4 = lane & 3;  // MMA fragment row and column pair
  const int slot = blockIdx.x, kvh = blockIdx.y, s = blockIdx.z;

  int row0, n, ctx;
  unsigned err = check_sequence(p, s, &row0, &n, &ctx);
  if (err & VA_DEV_BAD_ROWS) {
    if (tid == 0) flag(p.status, err);
    // (with several chunks the merge kernel writes the NaN rows)
    if (p.slots == 1 && slot == 0) {
      const int a = max(p.cu_rows[s], 0), b = min(p.cu_rows[s + 1], p.total_rows);
      for (long long i = (long long)a * p.H * D + tid; i < (long long)b * p.H * D; i += NW * 32)
        if (i / D % p.H / p.G == kvh) {
          if (p.o_bf16) reinterpret_cast<__nv_bfloat16*>(p.o)[i] = __float2bfloat16(NAN);
          else p.o[i] = NAN;
          if (i % D == 0) p.lse[i / D] = NAN;
        }
    }
    return;
  }
  const int G = p.G, R = n * G;
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

  unsigned char* ring = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023) + warp * C::NST * C::STAGE;
  // The pages' places, 32 of this warp's at a time, one per lane: a block, or
  // (contiguous cache) the page of the sequence itself; -1 for a bad entry.
  auto lookup = [&](int i) {
    if (i >= mine) return -1;
    const int vp = slo / kPage + warp + i * NW;
    const int rp = vp * kPage >= ws.head ? vp + ws.skip / kPage : vp;
    if (p.page_size == 0) return rp;
    const int blk = p.block_table[(long long)s * p.max_blocks + rp];
    if (blk < 0 || blk >= p.num_blocks) {
      atomicOr(&err_s, (int)VA_DEV_BAD_BLOCK);
      return -1;
    }
    return blk;
  };
  int place = lookup(lane);
  const uint64_t pol = policy_evict_first();
  auto load = [&](int i, int at) {  // page i of this warp into its stage; one lane
    const uint32_t bar = smem_u32(&bars[warp][i % C::NST]);
    const uint32_t dst = smem_u32(ring + (i % C::NST) * C::STAGE);
    mbar_arrive_expect_tx(bar, 2 * C::TILE);
    if (Q8) {
      const long long row = p.page_size == 0
                                ? ((long long)s * p.KVH + kvh) * p.capacity + (long long)at * kPage
                                : ((long long)at * p.KVH + kvh) * kPage;
      bulk_g2s(dst, (const unsigned char*)p.k + row * C::RB, C::TILE, bar, pol);
      bulk_g2s(dst + C::TILE_S, (const unsigned char*)p.v + row * C::RB, C::TILE, bar, pol);
    } else {
#pragma unroll
      for (int db = 0; db < D / 64; ++db) {
        const uint32_t off = db * kPage * 128;
        if (p.page_size == 0) {
          tma_load_3d(dst + off, &tmK, db * 64, at * kPage, s * p.KVH + kvh, bar, pol);
          tma_load_3d(dst + C::TILE_S + off, &tmV, db * 64, at * kPage, s * p.KVH + kvh, bar, pol);
        } else {
          tma_load_4d(dst + off, &tmK, db * 64, 0, kvh, at, bar, pol);
          tma_load_4d(dst + C::TILE_S + off, &tmV, db * 64, 0, kvh, at, bar, pol);
        }
      }
    }
  };
  // A bad entry loads nothing and stops the warp's loop at that page.
  int good = mine;
#pragma unroll
  for (int i = 0; i < C::NST; ++i) {
    const int at = __shfl_sync(0xffffffffu, place, i);
    if (i < good && at < 0) good = i;
    if (i < good && lane == 0) load(i, at);
  }

  // This thread's two rows (g and g + 8 of the KV head's R): Q fragments,
  // masks.  Q8_0: fp16 after a power of two that brings the row's largest
  // |q| below 1 (exact), the columns of a 32-element block permuted as the
  // codes are (see below).
  uint32_t qa[KS][4];
  unsigned anc[2] = {0u, 0u};
  int jrow[2], wlo[2] = {0, 0};
  bool rvalid[2];
  float c2[2] = {p.scale_log2, p.scale_log2};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = g + 8 * h;
    rvalid[h] = r < R;
    jrow[h] = rvalid[h] ? r / G : 0;
    const unsigned short* qp = reinterpret_cast<const unsigned short*>(p.q) +
                               ((long long)(row0 + jrow[h]) * p.H + kvh * G + (rvalid[h] ? r % G : 0)) * D;
    if (Q8) {
      // Per 32-element block b this lane owns elements 32 b + 8 q4 .. + 7.
      uint4 w[D / 32];
      float amax = 0.f;
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        w[b] = rvalid[h] ? *reinterpret_cast<const uint4*>(qp + 32 * b + 8 * q4) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t u[4] = {w[b].x, w[b].y, w[b].z, w[b].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(u[k] << 16)), fabsf(__uint_as_float(u[k] & 0xFFFF0000u))));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      int e = 0;
      if (amax > 0.f) frexpf(amax, &e);
      const float qs = ldexpf(1.f, -e);
      c2[h] = ldexpf(p.scale_log2, e);
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        const uint32_t u[4] = {w[b].x, w[b].y, w[b].z, w[b].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t v = pack_f16(__uint_as_float(u[k] << 16) * qs, __uint_as_float(u[k] & 0xFFFF0000u) * qs);
          qa[2 * b + k / 2][h + 2 * (k & 1)] = v;  // steps of 4 elements per lane: (0,1 | 2,3), (4,5 | 6,7)
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint32_t* qw = reinterpret_cast<const uint32_t*>(qp + 16 * k + 2 * q4);
        qa[k][h] = rvalid[h] ? qw[0] : 0u;
        qa[k][h + 2] = rvalid[h] ? qw[4] : 0u;
      }
    }
    if (rvalid[h] && !err) {
      bool bad = false;
      anc[h] = row_mask(kind, p.parent + row0, jrow[h], &bad);
      if (bad) {
        atomicOr(&err_s, (int)VA_DEV_BAD_PARENT);
      } else {
        wlo[h] = win_low(p, ctx + (kind == 1 ? __popc(anc[h]) - 1 : jrow[h])) - ws.skip;
        if (kind == 1) anc[h] = window_mask(p, p.parent + row0, jrow[h], ctx, anc[h]);
      }
    }
  }

  float o[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  volatile int* abort_p = &abort_s;

#pragma unroll 1
  for (int i = 0; i < good; ++i) {
    const int st = i % C::NST;
    unsigned char* ks = ring + st * C::STAGE;
    unsigned char* vs = ks + C::TILE_S;
    if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&bars[warp][st]), (i / C::NST) & 1, abort_p, kFewWaitNs))) {
      if (lane == 0) {
        *abort_p = 1;
        flag(p.status, VA_DEV_TIMEOUT);
      }
      break;
    }
    const int u0 = slo + (warp + i * NW) * kPage;  // the page's first span token
    const int tail = min(shi - u0, kPage);         // tokens of the chunk in it
    if (tail < kPage || (u0 < ws.dead_hi && u0 + kPage > ws.dead_lo)) {
      // Tokens that no row sees may hold anything: their V rows are cleared
      // (Q8_0: their scales, and with K's a NaN in the scores that the mask
      // below would drop anyway).
      const int t = lane & 15, u = u0 + t;
      if (t >= tail || (u >= ws.dead_lo && u < ws.dead_hi)) {
        if (Q8) {
          if (lane < 16)
            for (int b = 0; b < D / 32; ++b) *reinterpret_cast<unsigned short*>(vs + t * C::RB + 34 * b) = 0;
        } else {
          for (int b = lane >> 4; b < D / 8; b += 2)
            *reinterpret_cast<uint4*>(vs + (b / 8) * kPage * 128 + t * 128 + (b % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
    }

    // S = Q K^T: two tiles of 8 tokens.
    float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    if (Q8) {
      // A lane's 8 codes of a block (elements 8 q4 .. + 7 of token g of the
      // tile) make two k steps; the block's sum takes the token's scale.
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const unsigned char* kr = ks + (8 * t + g) * C::RB;
        const unsigned char* d0 = ks + (8 * t + 2 * q4) * C::RB;  // this lane's score columns
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
          const uint32_t x = code_word(kr + 34 * b + 2 + 8 * q4), y = code_word(kr + 34 * b + 6 + 8 * q4);
          float cb[4] = {0.f, 0.f, 0.f, 0.f};
          mma_f16(cb, qa[2 * b], h2_sub(__byte_perm(x, 0x64646464u, 0x4140), kBias),
                  h2_sub(__byte_perm(x, 0x64646464u, 0x4342), kBias));
          mma_f16(cb, qa[2 * b + 1], h2_sub(__byte_perm(y, 0x64646464u, 0x4140), kBias),
                  h2_sub(__byte_perm(y, 0x64646464u, 0x4342), kBias));
          const float s0 = __half2float(*reinterpret_cast<const __half*>(d0 + 34 * b));
          const float s1 = __half2float(*reinterpret_cast<const __half*>(d0 + C::RB + 34 * b));
          sc[t][0] = fmaf(s0, cb[0], sc[t][0]);
          sc[t][1] = fmaf(s1, cb[1], sc[t][1]);
          sc[t][2] = fmaf(s0, cb[2], sc[t][2]);
          sc[t][3] = fmaf(s1, cb[3], sc[t][3]);
        }
      }
    } else {
      // Lane's row of the 8 x 8 matrices: tokens 0-7 (k low, k high), 8-15.
      const int tr = (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
      const uint32_t kb = smem_u32(ks) + tr * 128;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        uint32_t b[4];
        ldmatrix4<false>(b, kb + (k / 4) * kPage * 128 + ((((k % 4) * 2 + kc) ^ (tr & 7)) << 4));
        mma_bf16(sc[0], qa[k], b[0], b[1]);
        mma_bf16(sc[1], qa[k], b[2], b[3]);
      }
    }

    // Masks, running maximum, P.
    const bool plain = u0 + kPage <= min(vctx, shi) && (u0 >= win_low(p, ctx + n - 1) - ws.skip || u0 + kPage <= p.sinks);
    float a[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      unsigned vis = 0xFFFFu;
      if (!plain)
        vis = rvalid[h] ? visible_bits(kind, anc[h], jrow[h], vctx, shi, u0) & window_bits(kind, p.sinks, wlo[h], vctx, u0)
                        : 0u;
      float mx = -INFINITY;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& x = sc[t][2 * h + e];
          x = (vis >> (8 * t + 2 * q4 + e)) & 1u ? x * c2[h] : -INFINITY;
          mx = fmaxf(mx, x);
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[h], mx);
      const float off = mn == -INFINITY ? 0.f : mn;  // while nothing is visible every P is 2^-inf
      a[h] = ex2f(m[h] - off);
      m[h] = mn;
      float sum = 0.f;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& x = sc[t][2 * h + e];
          x = ex2f(x - off);
          sum += x;
        }
      l[h] = fmaf(l[h], a[h], sum);
    }
    // P as the MMA's A operand: the score fragments are its rows.
    uint32_t ph[4], pl[4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float x = sc[t][2 * h], y = sc[t][2 * h + 1];
        if (Q8) {
          ph[2 * t + h] = pack_f16(x, y);
        } else {
          const uint32_t w = pack_bf16(x, y);
          ph[2 * t + h] = w;
          pl[2 * t + h] = pack_bf16(x - __uint_as_float(w << 16), y - __uint_as_float(w & 0xFFFF0000u));
        }
      }
    if (Q8) {
      // V: a lane's word of codes (elements 4 g .. + 3 of a block) of each of
      // its four tokens; column tile i of the block takes byte i.
      const unsigned char* v0 = vs + 2 * q4 * C::RB;
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        uint32_t w[4], d2[2];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = code_word(v0 + ((k & 1) + 8 * (k >> 1)) * C::RB + 34 * b + 2 + 4 * g);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const unsigned char* d = v0 + 8 * k * C::RB + 34 * b;
          d2[k] = *reinterpret_cast<const unsigned short*>(d) |
                  ((uint32_t)*reinterpret_cast<const unsigned short*>(d + C::RB) << 16);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          // Bytes c of two tokens into the low halves of two fp16 values.
          const uint32_t sel = 0x4000u | (uint32_t)c | ((uint32_t)(c + 4) << 4);
          uint32_t f[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t pr = __byte_perm(w[2 * k], w[2 * k + 1], sel);  // bytes: q0, q1
            f[k] = h2_mul(h2_sub(__byte_perm(pr, 0x64646464u, 0x4140), kBias), d2[k]);
          }
          float cc[4] = {0.f, 0.f, 0.f, 0.f};
          mma_f16(cc, ph, f[0], f[1]);
          float(&ot)[4] = o[4 * b + c];
          ot[0] = fmaf(ot[0], a[0], cc[0]);
          ot[1] = fmaf(ot[1], a[0], cc[1]);
          ot[2] = fmaf(ot[2], a[1], cc[2]);
          ot[3] = fmaf(ot[3], a[1], cc[3]);
        }
      }
    } else {
      // Lane's row of the transposed matrices: tokens 0-7, 8-15 of columns
      // 0-7, then of columns 8-15.
      const int tr = lane & 15, dc = lane >> 4;
      const uint32_t vb = smem_u32(vs) + tr * 128;
#pragma unroll
      for (int t = 0; t < NT / 2; ++t) {
        uint32_t b[4];
        ldmatrix4<true>(b, vb + (t / 4) * kPage * 128 + ((((t % 4) * 2 + dc) ^ (tr & 7)) << 4));
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float cc[4] = {0.f, 0.f, 0.f, 0.f};
          mma_bf16(cc, pl, b[2 * c], b[2 * c + 1]);
          mma_bf16(cc, ph, b[2 * c], b[2 * c + 1]);
          float(&ot)[4] = o[2 * t + c];
          ot[0] = fmaf(ot[0], a[0], cc[0]);
          ot[1] = fmaf(ot[1], a[0], cc[1]);
          ot[2] = fmaf(ot[2], a[1], cc[2]);
          ot[3] = fmaf(ot[3], a[1], cc[3]);
        }
      }
    }
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
      mbar_wait(smem_u32(&bars[warp][i]), 0, &dummy, kFewWaitNs);
      mbar_wait(smem_u32(&bars[warp][i]), 1, &dummy, kFewWaitNs);
    }
  }

  // Join the warps: each row's states in warp order.
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    if (q4 == 0) {
      m_s[warp][g + 8 * h] = m[h];
      l_s[warp][g + 8 * h] = l[h];
    }
  }
  __syncthreads();  // every ring is idle: its memory takes the O rows
  constexpr int LD = D + 4;
  float* os = reinterpret_cast<float*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  float* mo = os + warp * kFewRows * LD;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    // Q8_0: column tile 4 b + c holds elements 32 b + 4 j + c, j the column.
    const int col = Q8 ? (t / 4) * 32 + t % 4 + 8 * q4 : 8 * t + 2 * q4;
    constexpr int next = Q8 ? 4 : 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mo[(g + 8 * h) * LD + col] = o[t][2 * h];
      mo[(g + 8 * h) * LD + col + next] = o[t][2 * h + 1];
    }
  }
  __syncthreads();
  err |= (unsigned)err_s;
  const bool fail = err || abort_s;
  if (err && tid == 0) flag(p.status, err);
  for (int r = warp; r < R; r += NW) {
    float mr = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) mr = fmaxf(mr, m_s[w][r]);
    const float off = mr == -INFINITY ? 0.f : mr;
    float f[NW], lr = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      f[w] = ex2f(m_s[w][r] - off);
      lr = fmaf(f[w], l_s[w][r], lr);
    }
    const int grow = row0 + r / G, head = kvh * G + r % G;
    const long long item = (long long)grow * p.H + head;
    const float inv = p.slots == 1 ? 1.f / lr : 1.f;
    for (int c = 2 * lane; c < D; c += 64) {
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float2 v = *reinterpret_cast<const float2*>(os + (w * kFewRows + r) * LD + c);
        x = fmaf(f[w], v.x, x);
        y = fmaf(f[w], v.y, y);
      }
      x = fail ? NAN : x * inv;
      y = fail ? NAN : y * inv;
      if (p.slots > 1)
        *reinterpret_cast<float2*>(p.ws_acc + slot_index(p, slot, grow, head) * D + c) = make_float2(x, y);
      else if (p.o_bf16)
        reinterpret_cast<uint32_t*>(p.o)[(item * D + c) / 2] = pack_bf16(x, y);
      else
        *reinterpret_cast<float2*>(p.o + item * D + c) = make_float2(x, y);
    }
    if (lane == 0) {
      if (p.slots > 1) {
        const long long si = slot_index(p, slot, grow, head);
        p.ws_ml[2 * si] = fail ? NAN : mr;
        p.ws_ml[2 * si + 1] = fail ? NAN : lr;
      } else {
        p.lse[item] = fail ? NAN : (mr + log2f(lr)) * kLn2;
      }
    }
  }
}

bool make_page_maps(const Params& p, CUtensorMap* k, CUtensorMap* v);

template <int D, int KVT, int NW>
static cudaError_t launch_few_t(const Params& p, cudaStream_t st) {
  using C = FewCfg<D, KVT, NW>;
  static_assert(C::NST >= 2 && C::NST <= 4, "ring depth");
  static std::atomic<unsigned long long> ready{0ull};  // devices whose attribute is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(window_rows_kernel<D, KVT, NW>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  CUtensorMap mk, mv;
  memset(&mk, 0, sizeof(mk));
  memset(&mv, 0, sizeof(mv));
  if (!C::kQ8 && !make_page_maps(p, &mk, &mv)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)p.slots, (unsigned)p.KVH, (unsigned)p.num_seqs);
  cfg.blockDim = dim3(NW * 32);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, window_rows_kernel<D, KVT, NW>, p, mk, mv);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// One chunk per sequence means that the sequences fill the GPU: small CTAs,
// four to an SM.  Several chunks: few sequences, the more warps to each.
cudaError_t launch_window_rows(const Params& p, cudaStream_t st) {
#define VA_FEW(DD)                                                                                          \
  if (p.D == DD) {                                                                                          \
    if (p.kv_dtype == VA_BF16)                                                                              \
      return p.slots == 1 ? launch_few_t<DD, VA_BF16, 2>(p, st)                                             \
                          : launch_few_t<DD, VA_BF16, DD == 256 ? 6 : 8>(p, st);                            \
    if (p.kv_dtype == VA_Q8_0)                                                                              \
      return p.slots == 1 ? launch_few_t<DD, VA_Q8_0, 2>(p, st) : launch_few_t<DD, VA_Q8_0, 8>(p, st);      \
  }
  VA_FEW(64) VA_FEW(128) VA_FEW(256)
#undef VA_FEW
  return cudaErrorInvalidValue;
}

}  // namespace va
