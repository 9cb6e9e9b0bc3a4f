// Acceptance of drafted tokens against the target's logits, from given
// random numbers (chains and trees), and the token that follows.
//
// Row r of a sequence carries a token; its logits are the target's for the
// token after it.  Row 0 is known; every other row is a proposal for the
// token after its parent.  With p = softmax(logits[a] / T) at the node a
// reached so far, a's children are tried in row order.  The k-th child,
// with token x and acceptance number u, is taken iff
//     u g(x) < r(x),   r = p at the first child;
// a rejected child leaves r' = max(r - g, 0) / sum max(r - g, 0), where g
// is the drafter's distribution at a, or the indicator of x when none is
// given (r' is then r without x, renormalised).  At the node where no
// child is taken the next token is drawn from r by inversion: the lowest i
// with sum_{j <= i} r_j > v sum_j r_j.  At T = 0, p is the indicator of the
// lowest index of the row's maximum.  Taking proposals this way leaves the
// next tokens distributed exactly as p (the rejection rule of speculative
// sampling, applied to one sibling after another).
//
// Two kernels.  accept_stats_kernel reads the logits of every row that has
// a child, once, in pieces of 8,192 values (one CTA each, the whole piece
// in registers): the piece's maximum, its sum of exponentials relative to
// it, and the place of the maximum.  It is bound by the logits' bytes.
// accept_walk_kernel gives each sequence a cluster of eight CTAs: every
// CTA walks the path redundantly (the tests need one logit and one drafted
// probability per row, fetched for all rows at once), and the cluster then
// works through the one row that the next token is drawn from.
//
// Precision.  The tests compare numbers of order one: fp32 statistics
// decide them.  The draw is different: an error e in the running sum moves
// every later border by e, so that over a vocabulary the share of v that
// draws another token is e times the number of tokens that matter.  The
// weights of the last row are therefore 64-bit fixed-point numbers
// (2^43 exp(z - max), relative error about 2^-32) summed as integers: no
// order of summation changes the result, and borders move by about 1e-10.
#include <cooperative_groups.h>
#include <limits.h>
#include <math.h>
#include <string.h>

#include "va_common.cuh"
#include "va_host.h"

namespace va {
namespace cg = cooperative_groups;

constexpr int kPiece = 8192;         // values per statistics CTA
constexpr int kStatThreads = 256;
constexpr int kPerThread = kPiece / kStatThreads;
constexpr int kWalkThreads = 512;
constexpr int kWalkWarps = kWalkThreads / 32;
constexpr int kCluster = 8;          // CTAs per sequence (the portable limit)
constexpr int kSegs = kCluster * kWalkWarps;
constexpr int kMaxVocab = 1 << 20;   // 2^20 weights of 2^43 fit 63 bits
constexpr float kMinTemperature = 1e-6f;  // below it, only 0

struct AcceptParams {
  int num_seqs, total_rows, max_rows, mode;
  int vocab, pieces;
  const int* cu_rows;
  const int* parent;
  const unsigned char* seq_kind;
  const void* logits;
  long long logits_stride;
  const float* probs;
  long long probs_stride;
  const int* tokens;
  const float* accept_u;
  const float* sample_u;
  const float* temperature;
  float4* stats;  // [total_rows][pieces]: maximum, sum, bits of its index
  int* accepted_len;
  int* accepted_nodes;
  int* promote_len;
  int* next_token;
  unsigned* status;
};

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(float x) { return x; }
template <>
__device__ __forceinline__ float to_float(unsigned short x) { return bf16_bits_to_float(x); }

__device__ __forceinline__ int accept_kind(const AcceptParams& p, int s) {
  if (p.mode == VA_MODE_CHAIN) return 0;
  if (p.mode == VA_MODE_TREE) return 1;
  return p.seq_kind[s] ? 1 : 0;
}

// Rows of sequence s; false if they do not fit the launch.
__device__ __forceinline__ bool accept_rows(const AcceptParams& p, int s, int kind, int* row0, int* n) {
  const int r0 = p.cu_rows[s], r1 = p.cu_rows[s + 1];
  *row0 = r0;
  *n = r1 - r0;
  return !(r0 < 0 || r1 < r0 || r1 > p.total_rows || r1 - r0 > p.max_rows ||
           (kind == 1 && r1 - r0 > kMaxTreeRows));
}

// A sequence's temperature; negative, infinite or NaN values are refused by
// the walk kernel.
__device__ __forceinline__ float accept_temperature(const AcceptParams& p, int s) {
  return p.temperature ? p.temperature[s] : 1.f;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ---------------------------------------------------------------------------
// Statistics of one piece of one row.  grid = (pieces, max_rows, num_seqs).
// The cut into pieces depends on the vocabulary and the row's alignment
// alone, so a row's statistics do not depend on what shares the launch.
template <typename T>
__global__ void __launch_bounds__(kStatThreads) accept_stats_kernel(const AcceptParams p) {
  constexpr int VEC = 16 / (int)sizeof(T);
  constexpr int NV = kPerThread / VEC;
  __shared__ float red[kStatThreads / 32];
  __shared__ float red2[kStatThreads / 32];
  __shared__ int redi[kStatThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int s = blockIdx.z, j = blockIdx.y, piece = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kind = accept_kind(p, s);
  int row0, n;
  if (!accept_rows(p, s, kind, &row0, &n) || j >= n) return;
  bool child = j + 1 < n;
  if (kind == 1)  // n <= 32: one row per lane
    child = __any_sync(0xffffffffu, lane > j && lane < n && p.parent[row0 + lane] == j);
  if (!child) return;

  const T* row = reinterpret_cast<const T*>(p.logits) + (long long)(row0 + j) * p.logits_stride;
  // Values are counted from the 16-byte boundary at or before the row.
  const int pad = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
  const float temp = accept_temperature(p, s);
  float x[kPerThread];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = piece * kPiece + (k * kStatThreads + tid) * VEC - pad;
    if (i >= 0 && i + VEC <= p.vocab) {
      const uint4 w = __ldcs(reinterpret_cast<const uint4*>(row + i));
      const uint32_t c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (sizeof(T) == 4) x[k * VEC + e] = __uint_as_float(c[e]);
        else x[k * VEC + e] = __uint_as_float(e & 1 ? c[e / 2] & 0xFFFF0000u : c[e / 2] << 16);
      }
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        x[k * VEC + e] = i + e >= 0 && i + e < p.vocab ? to_float<T>(row[i + e]) : -INFINITY;
    }
  }
  float m = -INFINITY;
#pragma unroll
  for (int e = 0; e < kPerThread; ++e) m = fmaxf(m, x[e]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red[warp] = m;
  __syncthreads();
  m = red[0];
#pragma unroll
  for (int w = 1; w < kStatThreads / 32; ++w) m = fmaxf(m, red[w]);

  float sum = 0.f;
  int at = INT_MAX;
  if (temp > 0.f) {
    // exp((x - m) / T); a piece without a finite value (m = -inf) sums to 0.
    const float c = 1.4426950408889634f / temp;
    if (m != -INFINITY) {
#pragma unroll
      for (int e = 0; e < kPerThread; ++e) sum += exp2_fast((x[e] - m) * c);
    } else {
#pragma unroll
      for (int e = 0; e < kPerThread; ++e)
        if (x[e] != x[e]) sum = NAN;
    }
  } else {
#pragma unroll
    for (int k = NV - 1; k >= 0; --k)
#pragma unroll
      for (int e = VEC - 1; e >= 0; --e) {
        if (x[k * VEC + e] == m) at = piece * kPiece + (k * kStatThreads + tid) * VEC + e - pad;
        if (!(x[k * VEC + e] < INFINITY)) sum = NAN;  // NaN or +inf: no distribution
      }
    if (m == -INFINITY) at = INT_MAX;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    at = min(at, __shfl_xor_sync(0xffffffffu, at, o));
  }
  if (lane == 0) {
    red2[warp] = sum;
    redi[warp] = at;
  }
  __syncthreads();
  if (tid == 0) {
#pragma unroll
    for (int w = 1; w < kStatThreads / 32; ++w) {
      sum += red2[w];
      at = min(at, redi[w]);
    }
    p.stats[(long long)(row0 + j) * p.pieces + piece] = make_float4(m, sum, __int_as_float(at), 0.f);
  }
}

// ---------------------------------------------------------------------------
// Fixed-point weights: 2^(j / 64) * 2^43, rounded, for the reduction
// exp(y) = 2^(k / 64) exp(r), k = rint(64 y / ln 2), |r| <= ln 2 / 128 (the
// argument reduction in two parts of Cody and Waite; exp(r) - 1 by its
// Taylor series).
__device__ const unsigned long long kPow2[64] = {
    0x80000000000ull, 0x8164d1f3bc0ull, 0x82cd8698ac3ull, 0x843a28c3aceull,
    0x85aac367cc5ull, 0x871f61969e9ull, 0x88980e8092eull, 0x8a14d575497ull,
    0x8b95c1e3ea9ull, 0x8d1adf5b7e6ull, 0x8ea4398b45dull, 0x9031dc43146ull,
    0x91c3d373ab1ull, 0x935a2b2f13eull, 0x94f4efa8fefull, 0x96942d37202ull,
    0x9837f0518dcull, 0x99e0459320bull, 0x9b8d39b9d55ull, 0x9d3ed9a72d0ull,
    0x9ef5326091aull, 0xa0b0510fb97ull, 0xa27043030c5ull, 0xa43515ae09eull,
    0xa5fed6a9b15ull, 0xa7cd93b4e96ull, 0xa9a15ab4ea8ull, 0xab7a39b5a94ull,
    0xad583eea42aull, 0xaf3b78ad691ull, 0xb123f581d2bull, 0xb311c412a91ull,
    0xb504f333f9eull, 0xb6fd91e328dull, 0xb8fbaf47630ull, 0xbaff5ab2134ull,
    0xbd08a39f581ull, 0xbf1799b67a7ull, 0xc12c4cca667ull, 0xc346ccda249ull,
    0xc5672a11550ull, 0xc78d74c8abcull, 0xc9b9bd866e3ull, 0xcbec14fef27ull,
    0xce248c151f8ull, 0xd06333daef3ull, 0xd2a81d91f13ull, 0xd4f35aabcffull,
    0xd744fccad6aull, 0xd99d15c278bull, 0xdbfbb797dafull, 0xde60f4825e1ull,
    0xe0ccdeec2a9ull, 0xe33f8972be9ull, 0xe5b906e77c8ull, 0xe8396a503c5ull,
    0xeac0c6e7dd2ull, 0xed4f301ed99ull, 0xefe4b99bdceull, 0xf281773c5a0ull,
    0xf5257d15248ull, 0xf7d0df730adull, 0xfa83b2db723ull, 0xfd3e0c0cf48ull};

struct Weights {
  float top;              // the row's maximum
  float inv_hi, inv_lo;   // 1 / T
};

// 2^43 exp((x - top) / T), rounded.  x <= top, both finite or x = -inf.
__device__ __forceinline__ unsigned long long fixed_weight(const Weights& w, const unsigned long long* pow2,
                                                           float x) {
  // x - top exactly, as d + dl.
  const float d = x - w.top;
  const float bb = d - x;
  const float dl = (x - (d - bb)) + (-w.top - bb);
  const float y = d * w.inv_hi;
  if (!(y > -32.f)) return 0ull;  // below 2^-46 of the maximum; x = -inf
  const float yl = fmaf(d, w.inv_hi, -y) + fmaf(d, w.inv_lo, dl * w.inv_hi);
  const float kf = rintf(y * 92.332482616893656f);  // 64 / ln 2
  float r = fmaf(-kf, 0x1.62e430p-7f, y);
  r += yl - kf * -0x1.05c610p-35f;
  const int k = (int)kf;  // <= 0
  const unsigned long long t = pow2[k & 63];
  const float em1 = fmaf(r * r, fmaf(r, fmaf(r, 1.f / 24.f, 1.f / 6.f), 0.5f), r);
  const float tf = (float)(unsigned)(t >> 20) * 0x1p-23f;  // 2^(j / 64) to 24 bits
  const long long v = (long long)t + ((long long)__float2int_rn(tf * em1 * 0x1p37f) << 6);
  const int sh = -(k >> 6);
  return sh == 0 ? (unsigned long long)v : ((unsigned long long)v + (1ull << (sh - 1))) >> sh;
}

// floor(c q) up to one unit, for q in [0, 1] (NaN and negative count as 0).
__device__ __forceinline__ unsigned long long mul_prob(unsigned long long c, float q) {
  if (!(q > 0.f)) return 0ull;
  const unsigned long long f = __float2ull_rz(fminf(q, 1.f) * 0x1p63f);
  return __umul64hi(c, f) << 1;
}

constexpr int kMaxRej = kMaxTreeRows;  // rejected siblings of one node

struct WalkShared {
  unsigned long long pow2[64];
  unsigned long long seg[2][kSegs];  // a pass's sum over each warp's part of the row
  unsigned long long scale[kMaxRej + 1];  // sum of the weights before the k-th rejection
  float segmax[2][kCluster];
  unsigned segbad[2][kCluster];
  int segat[2][kCluster];
  float p[kMaxRows], q[kMaxRows], u[kMaxRows], top[kMaxRows];
  int token[kMaxRows], at[kMaxRows];
  short par[kMaxRows];
  float wmax[kWalkWarps];
  int wat[kWalkWarps];
  int rej_token[kMaxRej];
  unsigned err;
  int node, count, nrej, cmd, cursor;
  float rej_mass;
};

// One row's weights after nrej rejections: without drafted probabilities,
// the weight unless the token is one of the rejected; with them, the
// recursion s <- max(s - c g, 0) on unnormalised weights of sum c.
__device__ __forceinline__ unsigned long long weight_left(const WalkShared& sh, const Weights& w, const float* grow,
                                                          int nrej, int i, float x) {
  unsigned long long v = fixed_weight(w, sh.pow2, x);
  if (grow == nullptr) {
    for (int k = 0; k < nrej; ++k)
      if (sh.rej_token[k] == i) v = 0ull;
    return v;
  }
  if (nrej > 0 && v > 0ull) {
    const float g = grow[i];
    for (int k = 0; k < nrej; ++k) {
      const unsigned long long c = mul_prob(sh.scale[k], g);
      v = v > c ? v - c : 0ull;
    }
  }
  return v;
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ unsigned long long warp_scan(unsigned long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Walk of one sequence by a cluster.  Every CTA takes the same decisions
// from the same numbers, so the cluster's barriers always match.
template <typename T>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kWalkThreads)
    accept_walk_kernel(const AcceptParams p) {
  __shared__ WalkShared sh;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int s = blockIdx.x / kCluster;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kind = accept_kind(p, s);
  const float temp = accept_temperature(p, s);
  const bool greedy = temp == 0.f;
  int row0, n;
  const bool fits = accept_rows(p, s, kind, &row0, &n);
  if (tid < 64) sh.pow2[tid] = kPow2[tid];
  if (tid == 0) {
    sh.err = fits ? 0u : VA_DEV_BAD_ROWS;
    if (temp != 0.f && !(temp >= kMinTemperature && temp < INFINITY)) sh.err |= VA_DEV_BAD_SAMPLING;
    sh.node = 0;
    sh.count = 1;
    sh.nrej = 0;
    sh.cursor = 1;
    sh.rej_mass = 0.f;
  }
  if (!fits || n == 0) {
    // Rows unknown, or none: nothing to choose.  The same for every CTA.
    if (rank == 0 && tid == 0) {
      if (!fits) flag(p.status, VA_DEV_BAD_ROWS);
      p.accepted_len[s] = 0;
      if (p.promote_len) p.promote_len[s] = 0;
      p.next_token[s] = -1;
    }
    return;
  }
  for (int j = tid; j < n; j += kWalkThreads) sh.at[j] = -2;  // no statistics
  __syncthreads();

  // Every row's test, at once: its parent, p(x) and g(x).
  const T* logits = reinterpret_cast<const T*>(p.logits);
  for (int j = tid; j < n; j += kWalkThreads) {
    const int a = kind == 1 ? p.parent[row0 + j] : j - 1;
    if (kind == 1 && (j == 0 ? a != -1 : a < 0 || a >= j)) {
      atomicOr(&sh.err, VA_DEV_BAD_PARENT);
      continue;
    }
    if (j == 0) continue;
    const int x = p.tokens[row0 + j];
    if (x < 0 || x >= p.vocab) {
      atomicOr(&sh.err, VA_DEV_BAD_TOKEN);
      continue;
    }
    const float z = to_float<T>(logits[(long long)(row0 + a) * p.logits_stride + x]);
    const float g = p.probs ? p.probs[(long long)(row0 + a) * p.probs_stride + x] : 1.f;
    const float4* st = p.stats + (long long)(row0 + a) * p.pieces;
    float m = -INFINITY;
    int at = -1;
    for (int c = 0; c < p.pieces; ++c) {
      const float4 t = st[c];
      if (t.x > m) {
        m = t.x;
        at = __float_as_int(t.z);
      }
    }
    float sum = 0.f;
    const float inv = greedy ? 0.f : 1.4426950408889634f / temp;
    for (int c = 0; c < p.pieces; ++c) {
      const float4 t = st[c];
      // Pieces of -inf alone add nothing; a NaN in any piece stays.
      if (t.x != -INFINITY || t.y != t.y) sum += t.y * (greedy ? 1.f : exp2f((t.x - m) * inv));
    }
    const bool usable = sum == sum && m < INFINITY && m > -INFINITY;
    sh.par[j] = (short)a;
    sh.token[j] = x;
    sh.u[j] = p.accept_u[row0 + j];
    sh.q[j] = g;
    sh.p[j] = !usable ? -1.f : greedy ? (x == at ? 1.f : 0.f) : exp2f((z - m) * inv) / sum;
    sh.top[a] = usable ? m : NAN;  // siblings write the same values
    sh.at[a] = at;
  }
  __syncthreads();
  if (sh.err) {
    if (rank == 0) {
      if (tid == 0) {
        flag(p.status, sh.err);
        p.accepted_len[s] = 0;
        if (p.promote_len) p.promote_len[s] = 0;
        p.next_token[s] = -1;
      }
      for (int j = tid; j < n; j += kWalkThreads) p.accepted_nodes[row0 + j] = -1;
    }
    return;  // every CTA saw the same error and leaves here
  }

  // This warp's part of a row.
  const int seglen = ((p.vocab + kSegs - 1) / kSegs + 31) / 32 * 32;
  const int seg = rank * kWalkWarps + warp;
  const int lo = min(seg * seglen, p.vocab), hi = min(lo + seglen, p.vocab);
  Weights w;
  w.top = 0.f;
  {
    const double inv = greedy ? 1.0 : 1.0 / (double)temp;
    w.inv_hi = (float)inv;
    w.inv_lo = (float)(inv - (double)w.inv_hi);
  }
  int pass = 0;       // exchanges so far: the buffers alternate
  int have = -1;      // scale[0 .. have] hold sums at this node
  bool topped = false, bad = false;
  int best = -1;
  const T* row = logits;
  const float* grow = nullptr;

  // Sum of every segment's values in each CTA's table.
  auto exchange = [&](unsigned long long v) {
    v = warp_sum(v);
    const int b = pass & 1;
    if (lane < kCluster) *cluster.map_shared_rank(&sh.seg[b][seg], lane) = v;
    cluster.sync();
    ++pass;
    return b;
  };
  auto total_of = [&](int b) {
    unsigned long long t = 0ull;
    for (int g = lane; g < kSegs; g += 32) t += sh.seg[b][g];
    return warp_sum(t);
  };
  // The row's maximum (and its place), where the statistics kernel left
  // the row out.
  auto find_top = [&](int node) {
    topped = true;
    if (sh.at[node] != -2) {
      w.top = sh.top[node];
      best = sh.at[node];
      bad = w.top != w.top;
      return;
    }
    float m = -INFINITY;
    int at = INT_MAX;
    bool odd = false;
#pragma unroll 8
    for (int i = lo + lane; i < hi; i += 32) {
      const float x = to_float<T>(row[i]);
      odd |= !(x < INFINITY);
      if (x > m) {
        m = x;
        at = i;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float om = __shfl_xor_sync(0xffffffffu, m, o);
      const int oa = __shfl_xor_sync(0xffffffffu, at, o);
      if (om > m || (om == m && oa < at)) {
        m = om;
        at = oa;
      }
    }
    odd = __any_sync(0xffffffffu, odd);
    if (lane == 0) {
      sh.wmax[warp] = m;
      sh.wat[warp] = odd ? -1 : at;
    }
    __syncthreads();
    const int b = pass & 1;
    if (tid < kCluster) {
      float bm = -INFINITY;
      int ba = INT_MAX;
      unsigned bo = 0u;
      for (int k = 0; k < kWalkWarps; ++k) {
        if (sh.wat[k] == -1) bo = 1u;
        else if (sh.wmax[k] > bm) {
          bm = sh.wmax[k];
          ba = sh.wat[k];
        }
      }
      *cluster.map_shared_rank(&sh.segmax[b][rank], tid) = bm;
      *cluster.map_shared_rank(&sh.segat[b][rank], tid) = ba;
      *cluster.map_shared_rank(&sh.segbad[b][rank], tid) = bo;
    }
    cluster.sync();
    ++pass;
    w.top = -INFINITY;
    for (int k = 0; k < kCluster; ++k) {
      if (sh.segbad[b][k]) bad = true;
      if (sh.segmax[b][k] > w.top) {
        w.top = sh.segmax[b][k];
        best = sh.segat[b][k];
      }
    }
    if (w.top == -INFINITY) bad = true;
  };
  // The sum of the weights left after k rejections (k = 0: of all).
  auto sum_left = [&](int k) {
    unsigned long long v = 0ull;
#pragma unroll 4
    for (int i = lo + lane; i < hi; i += 32) v += weight_left(sh, w, grow, k, i, to_float<T>(row[i]));
    return exchange(v);
  };

  enum { DONE = 0, NEED_SUMS = 1 };
  for (;;) {
    if (tid == 0) {
      // Try the rows in order: a row counts when its parent is the node
      // reached so far (its siblings come later, its children after it).
      int node = sh.node, count = sh.count, nrej = sh.nrej, j = sh.cursor;
      float mass = sh.rej_mass;
      int cmd = DONE;
      for (; j < n; ++j) {
        if (sh.par[j] != node) continue;
        const float u = sh.u[j];
        bool yes;
        int x = 0;
        if (greedy) {
          yes = sh.p[j] > 0.f;
        } else if (sh.p[j] < 0.f) {
          yes = false;  // the row has no distribution
        } else if (!p.probs) {
          x = sh.token[j];
          bool again = false;
          for (int k = 0; k < nrej; ++k) again |= sh.rej_token[k] == x;
          yes = !again && u * (1.f - mass) < sh.p[j];
          if (!yes && !again) {
            sh.rej_token[nrej++] = x;
            mass += sh.p[j];
          }
        } else if (nrej == 0) {
          yes = u * sh.q[j] < sh.p[j];
          if (!yes) ++nrej;
        } else {
          // Against the weights left by the rejected siblings.
          if (have < nrej) {
            cmd = NEED_SUMS;
            break;
          }
          x = sh.token[j];
          const float* gr = p.probs + (long long)(row0 + node) * p.probs_stride;
          const unsigned long long left = weight_left(
              sh, w, gr, nrej, x, to_float<T>(logits[(long long)(row0 + node) * p.logits_stride + x]));
          yes = (double)u * (double)sh.q[j] * (double)sh.scale[nrej] < (double)left;
          if (!yes) ++nrej;
        }
        if (yes) {
          if (rank == 0) p.accepted_nodes[row0 + count] = j;
          node = j;
          ++count;
          nrej = 0;
          mass = 0.f;
          have = -1;
        }
      }
      sh.node = node;
      sh.count = count;
      sh.nrej = nrej;
      sh.cursor = j;
      sh.rej_mass = mass;
      sh.cmd = cmd;
    }
    __syncthreads();
    const int node = sh.node, cmd = sh.cmd, nrej = sh.nrej;
    const T* nrow = logits + (long long)(row0 + node) * p.logits_stride;
    if (nrow != row || !topped) {
      row = nrow;
      grow = p.probs ? p.probs + (long long)(row0 + node) * p.probs_stride : nullptr;
      have = -1;
      topped = false;
      bad = false;
      best = -1;
    }
    if (cmd == DONE) break;
    if (!topped) find_top(node);
    // Sums before each rejection so far, one exchange each.
    while (have < nrej) {
      const int b = sum_left(have + 1);
      const unsigned long long t = total_of(b);
      if (tid == 0) sh.scale[have + 1] = t;
      __syncthreads();
      ++have;
      if (t == 0ull && have > 0) break;
    }
    if (sh.scale[have] == 0ull) {  // nothing is left: the next sibling meets p itself
      have = 0;
      if (tid == 0) sh.nrej = 0;
    }
  }

  // Outputs of the walk.
  const int node = sh.node, count = sh.count;
  int nrej = sh.nrej;
  if (rank == 0) {
    if (tid == 0) {
      p.accepted_len[s] = count;
      if (p.promote_len) p.promote_len[s] = kind == 1 ? count : 0;
      p.accepted_nodes[row0] = 0;
    }
    for (int j = count + tid; j < n; j += kWalkThreads) p.accepted_nodes[row0 + j] = -1;
  }
  // The next token, from what is left at the last node.
  if (!topped) find_top(node);
  if (bad || greedy) {
    if (rank == 0 && tid == 0) {
      if (bad) flag(p.status, VA_DEV_BAD_LOGITS);
      p.next_token[s] = bad ? -1 : best;
    }
  } else {
    int b = 0;
    unsigned long long total = 0ull;
    if (grow == nullptr) {
      b = sum_left(nrej);
      total = total_of(b);
    } else {
      for (int k = have < 0 ? 0 : have; k <= nrej; ++k) {
        b = sum_left(k);
        total = total_of(b);
        if (tid == 0) sh.scale[k] = total;
        __syncthreads();
        if (total == 0ull) break;
      }
    }
    if (total == 0ull) {  // nothing is left: from p itself
      nrej = 0;
      b = sum_left(0);
      total = total_of(b);
    }
    // The lowest i whose running sum passes t = floor(v total).
    const float v = p.sample_u[s];
    unsigned long long t = v > 0.f ? __umul64hi(total, v < 1.f ? (unsigned long long)__float2ull_rz(v * 0x1p63f) << 1
                                                               : ~0ull)
                                   : 0ull;
    if (t >= total) t = total - 1;
    unsigned long long head = 0ull;
    for (int g = lane; g < seg; g += 32) head += sh.seg[b][g];
    head = warp_sum(head);
    const unsigned long long mine = sh.seg[b][seg];
    if (t >= head && t < head + mine) {
      // One warp owns the border: a lane sums a contiguous block, the block
      // that holds the border is then spread over the lanes again.
      const int blk = seglen / 32;
      const int b0 = lo + lane * blk, b1 = min(b0 + blk, hi);
      unsigned long long sum = 0ull;
#pragma unroll 4
      for (int i = b0; i < b1; ++i) sum += weight_left(sh, w, grow, nrej, i, to_float<T>(row[i]));
      const unsigned long long inc = warp_scan(sum, lane) + head;
      const int owner = __ffs(__ballot_sync(0xffffffffu, t < inc)) - 1;
      unsigned long long base = __shfl_sync(0xffffffffu, inc - sum, owner);
      const int c0 = lo + owner * blk, c1 = min(c0 + blk, hi);
      for (int i0 = c0; i0 < c1; i0 += 32) {
        const int i = i0 + lane;
        const unsigned long long wt = i < c1 ? weight_left(sh, w, grow, nrej, i, to_float<T>(row[i])) : 0ull;
        const unsigned long long c = warp_scan(wt, lane) + base;
        const unsigned hit = __ballot_sync(0xffffffffu, t < c);
        if (hit) {
          if (lane == __ffs(hit) - 1) p.next_token[s] = i;
          break;
        }
        base = __shfl_sync(0xffffffffu, c, 31);
      }
    }
  }
  cluster.sync();  // no CTA leaves while another may still write its tables
}

static int accept_pieces(int vocab) { return (vocab + 7 + kPiece - 1) / kPiece; }

static va_status check_accept(const va_problem* p, const va_draft* d, int mode) {
  if (!p || !d) return VA_ERR_INVALID_ARG;
  if (mode < VA_MODE_CHAIN || mode > VA_MODE_MIXED) return VA_ERR_INVALID_ARG;
  if (p->num_seqs < 1 || p->total_rows < 0 || p->max_rows_per_seq < 1) return VA_ERR_INVALID_ARG;
  if (!p->cu_rows) return VA_ERR_INVALID_ARG;
  if (mode != VA_MODE_CHAIN && !p->parent) return VA_ERR_INVALID_ARG;
  if (mode == VA_MODE_MIXED && !p->seq_kind) return VA_ERR_INVALID_ARG;
  if (d->vocab < 1 || d->logits_stride < d->vocab) return VA_ERR_INVALID_ARG;
  if (d->draft_probs && d->draft_stride < d->vocab) return VA_ERR_INVALID_ARG;
  if (d->logits_dtype < VA_F32 || d->logits_dtype > VA_Q8_0) return VA_ERR_INVALID_ARG;
  if (p->total_rows > 0 && (!d->logits || !d->tokens || !d->accept_u)) return VA_ERR_INVALID_ARG;
  if (!d->sample_u) return VA_ERR_INVALID_ARG;
  if (d->logits_dtype == VA_Q8_0 || d->vocab > kMaxVocab) return VA_ERR_UNSUPPORTED;
  if (p->max_rows_per_seq > kMaxRows || p->num_seqs > 65535) return VA_ERR_UNSUPPORTED;
  if (mode == VA_MODE_TREE && p->max_rows_per_seq > kMaxTreeRows) return VA_ERR_UNSUPPORTED;
  const uintptr_t esize = d->logits_dtype == VA_F32 ? 4 : 2;
  if ((uintptr_t)d->logits % esize || (uintptr_t)d->draft_probs % 4) return VA_ERR_ALIGNMENT;
  return VA_OK;
}

static size_t accept_ws_bytes(const va_problem* p, const va_draft* d) {
  if (p->max_rows_per_seq < 2) return 0;
  const size_t b = (size_t)p->total_rows * (size_t)accept_pieces(d->vocab) * sizeof(float4);
  return (b + 255) / 256 * 256;
}

template <typename K>
static cudaError_t launch_after(K kernel, dim3 grid, int threads, cudaStream_t st, const AcceptParams& q) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, q);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
static cudaError_t launch_accept(const AcceptParams& q, cudaStream_t st) {
  // A sequence of one row has no proposal: nothing to prepare.
  if (q.max_rows > 1) {
    const dim3 grid((unsigned)q.pieces, (unsigned)q.max_rows, (unsigned)q.num_seqs);
    cudaError_t e = launch_after(accept_stats_kernel<T>, grid, kStatThreads, st, q);
    if (e != cudaSuccess) return e;
  }
  return launch_after(accept_walk_kernel<T>, dim3((unsigned)(q.num_seqs * kCluster)), kWalkThreads, st, q);
}

}  // namespace va

using namespace va;

extern "C" {

size_t verify_attn_accept_workspace_size(const va_problem* p, const va_draft* d) {
  if (check_accept(p, d, VA_MODE_CHAIN) != VA_OK) return 0;
  return accept_ws_bytes(p, d);
}

va_status verify_attn_accept(const va_problem* p, const va_draft* d, int32_t mode, void* ws, size_t ws_bytes,
                             int32_t* accepted_len, int32_t* accepted_nodes, int32_t* promote_len,
                             int32_t* next_token, uint32_t* status, void* stream) {
  va_status st = check_accept(p, d, mode);
  if (st != VA_OK) return st;
  if (!accepted_len || !next_token || (p->total_rows > 0 && !accepted_nodes)) return VA_ERR_INVALID_ARG;
  const size_t need = accept_ws_bytes(p, d);
  if (need > 0 && (!ws || ws_bytes < need)) return VA_ERR_WORKSPACE_TOO_SMALL;
  if (need > 0 && ((uintptr_t)ws & 255u) != 0) return VA_ERR_ALIGNMENT;
  cudaStream_t cs = (cudaStream_t)stream;
  st = check_stream_device(cs);
  if (st != VA_OK) return st;
  AcceptParams q;
  memset(&q, 0, sizeof(q));
  q.num_seqs = p->num_seqs;
  q.total_rows = p->total_rows;
  q.max_rows = p->max_rows_per_seq;
  q.mode = mode;
  q.vocab = d->vocab;
  q.pieces = accept_pieces(d->vocab);
  q.cu_rows = p->cu_rows;
  q.parent = p->parent;
  q.seq_kind = p->seq_kind;
  q.logits = d->logits;
  q.logits_stride = d->logits_stride;
  q.probs = d->draft_probs;
  q.probs_stride = d->draft_stride;
  q.tokens = d->tokens;
  q.accept_u = d->accept_u;
  q.sample_u = d->sample_u;
  q.temperature = d->temperature;
  q.stats = (float4*)ws;
  q.accepted_len = accepted_len;
  q.accepted_nodes = accepted_nodes;
  q.promote_len = promote_len;
  q.next_token = next_token;
  q.status = (unsigned*)status;
  cudaError_t e = d->logits_dtype == VA_F32 ? launch_accept<float>(q, cs) : launch_accept<unsigned short>(q, cs);
  return e == cudaSuccess ? VA_OK : note_cuda(e);
}

}  // extern "C"
