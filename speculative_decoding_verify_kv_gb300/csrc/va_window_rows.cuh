// Warp-MMA attention of 16 query rows over 16-token pages: what the windowed
// kernels for few rows (one row tile per CTA) and for row tiles share.
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
// bf16: P enters as bf16 hi + lo (16 bits), and a third part where O is fp32.
// Q8_0: the codes enter the MMAs as exact fp16 integers, K's scales multiply the
// fp32 sums of each 32-element block, V's elements become fp16(d q) (one
// rounding) and P is fp16, in fp32 outputs too: some 3e-4 of O, what the
// framework's other kernels over Q8_0 give.  (Each rounding alone moves O by
// 2.0e-4; bf16 outputs round it by 1.7e-3 anyway, of which they make 1.70e-3.)
#pragma once

#include <string.h>

#include "va_common.cuh"
#include "va_sm100.cuh"
#include "va_window_join.cuh"

namespace va {
using namespace sm100;

constexpr int kTileRows = 16;  // query rows of one warp
constexpr uint64_t kPageWaitNs = 2000000000ull;

// A page of one tensor in shared memory: bf16 [D / 64][16 tokens][128 bytes]
// with 128-byte swizzle, Q8_0 16 raw rows.
template <int D, int KVT>
struct PageCfg {
  static constexpr bool kQ8 = KVT == VA_Q8_0;
  static constexpr int RB = kQ8 ? D / 32 * 34 : D * 2;  // bytes of a cache row
  static constexpr int TILE = kPage * RB;
  static constexpr int ALIGN = kQ8 ? 128 : 1024;  // (the swizzle's period)
  static constexpr int TILE_S = (TILE + ALIGN - 1) / ALIGN * ALIGN;  // K, then V
  static constexpr int STAGE = 2 * TILE_S;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  if (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
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

// Codes 4 w .. 4 w + 3 (N words from w on) of block b of a row, biased to q +
// 128.  Blocks are 34 bytes, so the codes of odd blocks start on a word and
// those of even blocks two bytes into one.
template <int N>
__device__ __forceinline__ void code_words(uint32_t (&x)[N], const unsigned char* row, int b, int w) {
  const uint32_t* p = reinterpret_cast<const uint32_t*>(row + 34 * b + (b & 1 ? 2 : 0)) + w;
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = p[k];
  if (!(b & 1)) {
    const uint32_t last = p[N];
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = __funnelshift_r(x[k], k + 1 < N ? x[k + 1] : last, 16);
  }
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] ^= 0x80808080u;
}

// A warp's 16 rows: Q fragments, what masks them, and their softmax state.  In
// MMA fragments a lane holds rows g = lane / 4 and g + 8 and column pair
// lane % 4.  EX: O leaves in fp32 (bf16 caches).
template <int D, int KVT, bool EX>
struct RowTile {
  static constexpr bool Q8 = KVT == VA_Q8_0;
  static constexpr int KS = D / 16;  // k steps of S
  static constexpr int NT = D / 8;   // column tiles of O
  uint32_t qa[KS][4];
  unsigned anc[2];
  int jrow[2], wlo[2];
  bool rvalid[2];
  float c2[2];
  float o[NT][4];
  float m[2], l[2];

  // Rows r0 .. r0 + R - 1 (at most 16) of the KV head's; false for a bad
  // parent.
  __device__ __forceinline__ bool init(const Params& p, const WinSpan& ws, int row0, int ctx, int kind, int kvh,
                                       int r0, int R, bool check) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3, G = p.G;
    bool fine = true;
    // Q8_0: fp16 after a power of two that brings the row's largest |q| below
    // 1 (exact), the columns of a 32-element block permuted as the codes are.
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = g + 8 * h;
      rvalid[h] = r < R;
      anc[h] = 0u;
      wlo[h] = 0;
      c2[h] = p.scale_log2;
      jrow[h] = rvalid[h] ? (r0 + r) / G : 0;
      const unsigned short* qp = reinterpret_cast<const unsigned short*>(p.q) +
                                 ((long long)(row0 + jrow[h]) * p.H + kvh * G + (rvalid[h] ? (r0 + r) % G : 0)) * D;
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
      if (rvalid[h] && check) {
        bool bad = false;
        anc[h] = row_mask(kind, p.parent + row0, jrow[h], &bad);
        if (bad) {
          fine = false;
        } else {
          wlo[h] = win_low(p, ctx + (kind == 1 ? __popc(anc[h]) - 1 : jrow[h])) - ws.skip;
          if (kind == 1) anc[h] = window_mask(p, p.parent + row0, jrow[h], ctx, anc[h]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
    return fine;
  }

  // What a page leaves between its two products: the scores, then P as the
  // second MMA's A operand (in parts), and the factor of the earlier sums.
  struct Page {
    float sc[2][4];
    float a[2];
    uint32_t ph[4], pl[4], pr[4];
  };

  // Scores of one page: its K in shared memory.  (K's stage is free after
  // this.)
  __device__ __forceinline__ void scores(Page& pg, const unsigned char* ks) {
    using C = PageCfg<D, KVT>;
    const int lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
    // S = Q K^T: two tiles of 8 tokens.
    float(&sc)[2][4] = pg.sc;
#pragma unroll
    for (int t = 0; t < 2; ++t) sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.f;
    if (Q8) {
      // A lane's 8 codes of a block (elements 8 q4 .. + 7 of token g of the
      // tile) make two k steps; the block's sum takes the token's scale.
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        float cb[2][4];
        uint32_t x[2][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          code_words<2>(x[t], ks + (8 * t + g) * C::RB, b, 2 * q4);
          cb[t][0] = cb[t][1] = cb[t][2] = cb[t][3] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
          mma_f16(cb[t], qa[2 * b], h2_sub(__byte_perm(x[t][0], 0x64646464u, 0x4140), kBias),
                  h2_sub(__byte_perm(x[t][0], 0x64646464u, 0x4342), kBias));
#pragma unroll
        for (int t = 0; t < 2; ++t)
          mma_f16(cb[t], qa[2 * b + 1], h2_sub(__byte_perm(x[t][1], 0x64646464u, 0x4140), kBias),
                  h2_sub(__byte_perm(x[t][1], 0x64646464u, 0x4342), kBias));
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const unsigned char* d0 = ks + (8 * t + 2 * q4) * C::RB + 34 * b;  // this lane's score columns
          const float s0 = __half2float(*reinterpret_cast<const __half*>(d0));
          const float s1 = __half2float(*reinterpret_cast<const __half*>(d0 + C::RB));
          sc[t][0] = fmaf(s0, cb[t][0], sc[t][0]);
          sc[t][1] = fmaf(s1, cb[t][1], sc[t][1]);
          sc[t][2] = fmaf(s0, cb[t][2], sc[t][2]);
          sc[t][3] = fmaf(s1, cb[t][3], sc[t][3]);
        }
      }
    } else {
      // Lane's row of the 8 x 8 matrices: tokens 0-7 (k low, k high), 8-15.
      const int tr = (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
      const uint32_t kb = smem_u32(ks) + tr * 128;
      // Four k steps' matrices at a time, four running sums (a warp has few
      // neighbours to hide an MMA's latency behind).
      float s2[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int k0 = 0; k0 < KS; k0 += 4) {
        uint32_t b[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          ldmatrix4<false>(b[k], kb + (k0 / 4) * kPage * 128 + (((k * 2 + kc) ^ (tr & 7)) << 4));
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          mma_bf16(sc[0], qa[k0 + k], b[k][0], b[k][1]);
          mma_bf16(sc[1], qa[k0 + k], b[k][2], b[k][3]);
          mma_bf16(s2[0], qa[k0 + k + 1], b[k + 1][0], b[k + 1][1]);
          mma_bf16(s2[1], qa[k0 + k + 1], b[k + 1][2], b[k + 1][3]);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sc[0][e] += s2[0][e];
        sc[1][e] += s2[1][e];
      }
    }

  }

  // The softmax step of a page: u0 its first span token, shi the end of the
  // chunk, edge the span token from which no row's window starts any more.
  __device__ __forceinline__ void softmax(Page& pg, const Params& p, int kind, int vctx, int shi, int edge, int u0) {
    const int lane = threadIdx.x & 31, q4 = lane & 3;
    float(&sc)[2][4] = pg.sc;
    float(&a)[2] = pg.a;
    // Masks, running maximum, P.
    const bool plain = u0 + kPage <= min(vctx, shi) && (u0 >= edge || u0 + kPage <= p.sinks);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) sc[t][2 * h + e] *= c2[h];
    }
    if (!plain) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const unsigned vis =
            rvalid[h] ? visible_bits(kind, anc[h], jrow[h], vctx, shi, u0) & window_bits(kind, p.sinks, wlo[h], vctx, u0)
                      : 0u;
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (!((vis >> (8 * t + 2 * q4 + e)) & 1u)) sc[t][2 * h + e] = -INFINITY;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mx = fmaxf(fmaxf(sc[0][2 * h], sc[0][2 * h + 1]), fmaxf(sc[1][2 * h], sc[1][2 * h + 1]));
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
    uint32_t(&ph)[4] = pg.ph, (&pl)[4] = pg.pl, (&pr)[4] = pg.pr;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float x = sc[t][2 * h], y = sc[t][2 * h + 1];
        if (Q8) {
          ph[2 * t + h] = pack_f16(x, y);
        } else {
          const uint32_t w = pack_bf16(x, y);
          const float xl = x - __uint_as_float(w << 16), yl = y - __uint_as_float(w & 0xFFFF0000u);
          const uint32_t wl = pack_bf16(xl, yl);
          ph[2 * t + h] = w;
          pl[2 * t + h] = wl;
          // What is left (to 24 bits in all) counts where O leaves in fp32.
          if (EX) pr[2 * t + h] = pack_bf16(xl - __uint_as_float(wl << 16), yl - __uint_as_float(wl & 0xFFFF0000u));
        }
      }
  }

  // O <- a O + P V of a page: its V in shared memory.
  __device__ __forceinline__ void values(const Page& pg, const Params& p, const unsigned char* vs) {
    using C = PageCfg<D, KVT>;
    const int lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
    const float(&a)[2] = pg.a;
    const uint32_t(&ph)[4] = pg.ph, (&pl)[4] = pg.pl, (&pr)[4] = pg.pr;
    if (Q8) {
      // V: a lane's word of codes (elements 4 g .. + 3 of a block) of each of
      // its four tokens; column tile i of the block takes byte i.
      const unsigned char* v0 = vs + 2 * q4 * C::RB;
#pragma unroll
      for (int b = 0; b < D / 32; ++b) {
        uint32_t w[4], d2[2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t x[1];
          code_words<1>(x, v0 + ((k & 1) + 8 * (k >> 1)) * C::RB, b, g);
          w[k] = x[0];
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const unsigned char* d = v0 + 8 * k * C::RB + 34 * b;
          d2[k] = *reinterpret_cast<const unsigned short*>(d) |
                  ((uint32_t)*reinterpret_cast<const unsigned short*>(d + C::RB) << 16);
        }
        float cc[4][4];
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
          cc[c][0] = cc[c][1] = cc[c][2] = cc[c][3] = 0.f;
          mma_f16(cc[c], ph, f[0], f[1]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float(&ot)[4] = o[4 * b + c];
          ot[0] = fmaf(ot[0], a[0], cc[c][0]);
          ot[1] = fmaf(ot[1], a[0], cc[c][1]);
          ot[2] = fmaf(ot[2], a[1], cc[c][2]);
          ot[3] = fmaf(ot[3], a[1], cc[c][3]);
        }
      }
    } else {
      // Lane's row of the transposed matrices: tokens 0-7, 8-15 of columns
      // 0-7, then of columns 8-15.
      const int tr = lane & 15, dc = lane >> 4;
      const uint32_t vb = smem_u32(vs) + tr * 128;
      // Several column tiles at a time, for the same reason (fewer at D = 256,
      // whose accumulator leaves fewer registers).
      constexpr int GR = D == 256 ? 2 : 4;
#pragma unroll
      for (int t0 = 0; t0 < NT / 2; t0 += GR) {
        uint32_t b[GR][4];
        float cc[2 * GR][4];
#pragma unroll
        for (int t = 0; t < GR; ++t)
          ldmatrix4<true>(b[t], vb + ((t0 + t) / 4) * kPage * 128 + (((((t0 + t) % 4) * 2 + dc) ^ (tr & 7)) << 4));
#pragma unroll
        for (int c = 0; c < 2 * GR; ++c) {
          cc[c][0] = cc[c][1] = cc[c][2] = cc[c][3] = 0.f;
          if (EX) mma_bf16(cc[c], pr, b[c / 2][2 * (c & 1)], b[c / 2][2 * (c & 1) + 1]);
        }
#pragma unroll
        for (int c = 0; c < 2 * GR; ++c) mma_bf16(cc[c], pl, b[c / 2][2 * (c & 1)], b[c / 2][2 * (c & 1) + 1]);
#pragma unroll
        for (int c = 0; c < 2 * GR; ++c) mma_bf16(cc[c], ph, b[c / 2][2 * (c & 1)], b[c / 2][2 * (c & 1) + 1]);
#pragma unroll
        for (int c = 0; c < 2 * GR; ++c) {
          float(&ot)[4] = o[2 * t0 + c];
          ot[0] = fmaf(ot[0], a[0], cc[c][0]);
          ot[1] = fmaf(ot[1], a[0], cc[c][1]);
          ot[2] = fmaf(ot[2], a[1], cc[c][2]);
          ot[3] = fmaf(ot[3], a[1], cc[c][3]);
        }
      }
    }
  }

  // The state into shared memory: O rows of LD floats, m and l.
  __device__ __forceinline__ void store(float* os, int ld, float* ms, float* ls) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q4 = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (q4 == 0) {
        ms[g + 8 * h] = m[h];
        ls[g + 8 * h] = l[h];
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      // Q8_0: column tile 4 b + c holds elements 32 b + 4 j + c, j the column.
      const int col = Q8 ? (t / 4) * 32 + t % 4 + 8 * q4 : 8 * t + 2 * q4;
      constexpr int next = Q8 ? 4 : 1;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        os[(g + 8 * h) * ld + col] = o[t][2 * h];
        os[(g + 8 * h) * ld + col + next] = o[t][2 * h + 1];
      }
    }
  }
};

// Clears what no row sees of a page's V (its tokens may hold anything): the
// tokens from tail on and span tokens [dead_lo, dead_hi).  Q8_0: their
// scales.  One warp; its writes reach the copy engine's next fill in order.
template <int D, int KVT>
__device__ __forceinline__ void clear_unseen(unsigned char* vs, int u0, int tail, int dead_lo, int dead_hi) {
  using C = PageCfg<D, KVT>;
  const int lane = threadIdx.x & 31, t = lane & 15, u = u0 + t;
  if (t >= tail || (u >= dead_lo && u < dead_hi)) {
    if (C::kQ8) {
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

// A page of K (v false) or V into shared memory; one thread.  at: the block, or
// (contiguous cache) the page of the sequence.
template <int D, int KVT>
__device__ __forceinline__ void load_half(const Params& p, const CUtensorMap* map, bool v, int s, int kvh, int at,
                                          uint32_t dst, uint32_t bar, uint64_t pol) {
  using C = PageCfg<D, KVT>;
  if (C::kQ8) {
    const long long row = p.page_size == 0 ? ((long long)s * p.KVH + kvh) * p.capacity + (long long)at * kPage
                                           : ((long long)at * p.KVH + kvh) * kPage;
    bulk_g2s(dst, (const unsigned char*)(v ? p.v : p.k) + row * C::RB, C::TILE, bar, pol);
  } else {
    if (p.page_size == 0) tma_load_4d(dst, map, 0, at * kPage, 0, s * p.KVH + kvh, bar, pol);
    else tma_load_5d(dst, map, 0, 0, 0, kvh, at, bar, pol);
  }
}

// Place of page vp of the span: its block (-1 for a bad table entry), or in a
// contiguous cache the page of the sequence.
__device__ __forceinline__ int page_place(const Params& p, const WinSpan& ws, int s, int vp) {
  const int rp = vp * kPage >= ws.head ? vp + ws.skip / kPage : vp;
  if (p.page_size == 0) return rp;
  const int blk = p.block_table[(long long)s * p.max_blocks + rp];
  return blk < 0 || blk >= p.num_blocks ? -1 : blk;
}

// Join the states of each row's NG page groups, in order, and write the rows
// out.  State (group x, row tile y) lies at index x RT + y.  Every warp of the
// CTA.  Chunks that make a cluster are joined there, others' partials go to the
// workspace.
template <int D, int NG, int RT>
__device__ __forceinline__ void join_rows(const Params& p, int slot, int row0, int kvh, int R, bool fail, float* os,
                                          int ld, float (*ms)[kTileRows], float (*ls)[kTileRows]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const bool one = p.slots == 1, partial = !p.joined;
  // A warp takes a row, or with fewer rows than warps 64 columns of one.
  const int parts = R < warps ? D / 64 : 1;
  for (int item = warp; item < R * parts; item += warps) {
    const int r = item / parts, part = item - r * parts;
    const int tile = r / kTileRows, rt = r % kTileRows;
    float mr = -INFINITY;
#pragma unroll
    for (int w = 0; w < NG; ++w) mr = fmaxf(mr, ms[w * RT + tile][rt]);
    const float off = mr == -INFINITY ? 0.f : mr;
    float f[NG], lr = 0.f;
#pragma unroll
    for (int w = 0; w < NG; ++w) {
      f[w] = ex2f(ms[w * RT + tile][rt] - off);
      lr = fmaf(f[w], ls[w * RT + tile][rt], lr);
    }
    if (fail) mr = lr = NAN;
    const int grow = row0 + r / p.G, head = kvh * p.G + r % p.G;
    const float inv = one ? 1.f / lr : fail ? NAN : 1.f;
    float* at = os + (tile * kTileRows + rt) * ld;
    for (int c = 64 * part + 2 * lane; c < D; c += 64 * parts) {
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < NG; ++w) {
        const float2 v = *reinterpret_cast<const float2*>(at + c + w * RT * kTileRows * ld);
        x = fmaf(f[w], v.x, x);
        y = fmaf(f[w], v.y, y);
      }
      if (one || partial) put_pair<D>(p, partial, slot, grow, head, c, x * inv, y * inv);
      else *reinterpret_cast<float2*>(at + c) = make_float2(x, y);  // the first group's place
    }
    if (lane == 0 && part == 0) {
      if (one) {
        p.lse[(long long)grow * p.H + head] = (mr + log2f(lr)) * kLn2;
      } else if (partial) {
        const long long si = slot_index(p, slot, grow, head);
        p.ws_ml[2 * si] = mr;
        p.ws_ml[2 * si + 1] = lr;
      } else {  // behind the row's columns (ms and ls are still read)
        at[D] = mr;
        at[D + 1] = lr;
      }
    }
  }
  if (one || partial) return;
  join_chunks<D, (RT == 1 ? kJoinFew : kJoinMany)>(p, slot, row0, kvh, R, os, ld, os + D, os + D + 1, ld);
}

bool make_page_maps(const Params& p, CUtensorMap* k, CUtensorMap* v);

}  // namespace va
