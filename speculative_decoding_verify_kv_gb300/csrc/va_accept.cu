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
// a child, once, in pieces of 4,096 values (one warp each, the next 2 KB in
// flight while the last are summed): the piece's maximum, its sum of
// exponentials relative to it, and the place of the maximum.  It is bound
// by the logits' bytes.
// accept_walk_kernel gives each sequence a cluster of 8 or 16 CTAs: every
// CTA walks the path redundantly (the tests need one logit and one drafted
// probability per row, fetched for all rows at once), and the cluster then
// works through the one row that the next token is drawn from.
//
// Precision.  The tests compare numbers of order one: fp32 statistics
// decide them.  The draw is different: an error e in the running sum moves
// every later border by e, so that over a vocabulary the share of v that
// draws another token is e times the number of tokens that matter.  The
// weights of the last row are therefore 64-bit fixed-point numbers
// (2^39 exp(z - max) up to a vocabulary of 2^19, relative error about 2^-32)
// summed as integers: no order of summation changes the result, and borders
// move by about 1e-10 (over the share of the mass that is left, after
// rejections with drafted probabilities).
#include <cooperative_groups.h>
#include <limits.h>
#include <math.h>
#include <string.h>

#include <atomic>

#include "va_common.cuh"
#include "va_host.h"

namespace va {
namespace cg = cooperative_groups;

constexpr int kPiece = 4096;         // values per statistics warp
constexpr int kStatThreads = 256;
constexpr int kStatWarps = kStatThreads / 32;
constexpr int kMaxWalkWarps = 32;    // of a CTA: 16, or 32 (see launch_accept)
constexpr int kMaxCluster = 16;      // CTAs per sequence: 8, or 16
constexpr int kUnit = 256;           // values a warp takes at a time, 8 per lane
constexpr int kMaxVocab = 1 << 20;
// Dynamic shared memory of the walk on an SM: of one CTA of 1,024 threads or of
// two of 512.  It holds the weights of a row's part so that a pass after a
// rejection does not make them again; in five bytes a cluster of 8 with 512
// threads holds 163,000 (32 chains over 131,072 values took 68 us when
// eight-byte weights did not fit and were made again, 56 with these).
constexpr int kWalkBytes = 206 * 1024;
constexpr int kWeightBytes = 5;      // of a weight kept in shared memory
constexpr int kRowBytes = 28;        // of a row's test
constexpr float kMinTemperature = 1e-6f;  // below it, only 0

struct AcceptParams {
  int num_seqs, total_rows, max_rows, mode;
  int vocab, pieces;
  int weight_bits;        // weights are 2^weight_bits exp(..)
  int cached;             // the walk keeps its row's weights in shared memory
  int kept;               // units that a CTA has room for
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
// Four 16-byte vectors of a row per lane: values [i, i + VEC) and so on, 32
// lanes apart; values outside the row are -inf.
template <typename T>
struct RowStep {
  static constexpr int VEC = 16 / (int)sizeof(T);
  static constexpr int N = 4 * VEC;
  uint4 w[4];
  __device__ __forceinline__ void load(const T* row, int vocab, int i) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int a = i + k * 32 * VEC;
      if (a >= 0 && a + VEC <= vocab) {
        w[k] = __ldcs(reinterpret_cast<const uint4*>(row + a));
      } else {
        uint32_t c[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (sizeof(T) == 4) {
            c[e] = a + e >= 0 && a + e < vocab ? reinterpret_cast<const uint32_t*>(row)[a + e] : 0xFF800000u;
          } else {
            const unsigned short* r = reinterpret_cast<const unsigned short*>(row);
            const int b = a + 2 * e;
            c[e] = (b >= 0 && b < vocab ? r[b] : 0xFF80u) |
                   (b + 1 >= 0 && b + 1 < vocab ? (uint32_t)r[b + 1] << 16 : 0xFF800000u);
          }
        }
        w[k] = make_uint4(c[0], c[1], c[2], c[3]);
      }
    }
  }
  // Value e of vector k.
  __device__ __forceinline__ float at(int k, int e) const {
    const uint32_t c[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
    if (sizeof(T) == 4) return __uint_as_float(c[e]);
    return __uint_as_float(e & 1 ? c[e / 2] & 0xFFFF0000u : c[e / 2] << 16);
  }
};

// Statistics of one piece of one row per warp.  grid = (pieces / 8,
// max_rows, num_seqs).  The cut into pieces depends on the vocabulary and
// the row's alignment alone, so a row's statistics do not depend on what
// shares the launch.  A lane keeps its own running maximum and sum.  480 rows of
// 131,072 bf16 values: 25.6 us, 4.9 TB/s; the start of each short CTA (row
// range, then the first values) keeps it from the bandwidth, not its
// instructions (half as many took as long).
template <typename T>
__global__ void __launch_bounds__(kStatThreads) accept_stats_kernel(const AcceptParams p) {
  using S = RowStep<T>;
  constexpr int STEP = 32 * S::N;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int s = blockIdx.z, j = blockIdx.y;
  const int lane = threadIdx.x & 31, piece = blockIdx.x * kStatWarps + (threadIdx.x >> 5);
  const int kind = accept_kind(p, s);
  int row0, n;
  if (!accept_rows(p, s, kind, &row0, &n) || j >= n || piece >= p.pieces) return;
  bool child = j + 1 < n;
  if (kind == 1)  // n <= 32: one row per lane
    child = __any_sync(0xffffffffu, lane > j && lane < n && p.parent[row0 + lane] == j);
  if (!child) return;

  const T* row = reinterpret_cast<const T*>(p.logits) + (long long)(row0 + j) * p.logits_stride;
  // Values are counted from the 16-byte boundary at or before the row.
  const int pad = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
  const float temp = accept_temperature(p, s);
  const int first = piece * kPiece + lane * S::VEC - pad;
  const int steps = min(kPiece / STEP, (p.vocab + pad - piece * kPiece + STEP - 1) / STEP);
  S cur, next;
  if (steps > 0) cur.load(row, p.vocab, first);
  float m = -INFINITY, sum = 0.f;
  int at = INT_MAX;
  const float c = temp > 0.f ? 1.4426950408889634f / temp : 0.f;
  for (int t = 0; t < steps; ++t) {
    if (t + 1 < steps) next.load(row, p.vocab, first + (t + 1) * STEP);
    float tm = -INFINITY;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < S::VEC; ++e) tm = fmaxf(tm, cur.at(k, e));
    if (temp > 0.f) {
      if (tm > m) {
        sum *= exp2_fast((m - tm) * c);  // exp2(-inf) = 0 at the first
        m = tm;
      }
      // exp((x - m) / T); while nothing is finite only a NaN shows.
      const float off = m == -INFINITY ? 0.f : -m;
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < S::VEC; ++e) sum += exp2_fast((cur.at(k, e) + off) * c);
    } else {
      if (tm > m) {
        m = tm;
#pragma unroll
        for (int k = 3; k >= 0; --k)
#pragma unroll
          for (int e = S::VEC - 1; e >= 0; --e)
            if (cur.at(k, e) == m) at = first + t * STEP + k * 32 * S::VEC + e;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int e = 0; e < S::VEC; ++e)
          if (!(cur.at(k, e) < INFINITY)) sum = NAN;  // NaN or +inf: no distribution
    }
    cur = next;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, m, o), os = __shfl_xor_sync(0xffffffffu, sum, o);
    const int oa = __shfl_xor_sync(0xffffffffu, at, o);
    const float nm = fmaxf(m, om);
    if (temp > 0.f && nm != -INFINITY) {
      sum = sum * exp2_fast((m - nm) * c) + os * exp2_fast((om - nm) * c);
    } else {
      sum += os;
    }
    at = om > m ? oa : om == m ? min(at, oa) : at;
    m = nm;
  }
  if (lane == 0)
    p.stats[(long long)(row0 + j) * p.pieces + piece] = make_float4(m, sum, __int_as_float(at), 0.f);
}

// ---------------------------------------------------------------------------
// Fixed-point weights: 2^(j / 32) * 2^30, rounded, for the reduction
// exp(y) = 2^(k / 32) exp(r), k = rint(32 y / ln 2), |r| <= ln 2 / 64 (the
// argument reduction in two parts of Cody and Waite; exp(r) - 1 by its
// Taylor series).
constexpr int kPow2 = 32;
__device__ const uint32_t kPow2Fix[kPow2] = {
    0x40000000u, 0x4166c34cu, 0x42d561b4u, 0x444c0740u, 0x45cae0f2u, 0x47521cc6u, 0x48e1e9bau, 0x4a7a77d4u,
    0x4c1bf829u, 0x4dc69cddu, 0x4f7a9930u, 0x51382182u, 0x52ff6b55u, 0x54d0ad5au, 0x56ac1f75u, 0x5891fac1u,
    0x5a82799au, 0x5c7dd7a4u, 0x5e8451d0u, 0x60962665u, 0x62b39509u, 0x64dcdec3u, 0x6712460bu, 0x69540ec9u,
    0x6ba27e65u, 0x6dfddbccu, 0x70666f76u, 0x72dc8374u, 0x75606374u, 0x77f25cceu, 0x7a92be8bu, 0x7d41d96eu};

// The table in shared memory, one copy per lane: an entry's two words lie in
// the lane's own bank, so that 32 different entries are read at once.
struct Pow2Table {
  uint32_t fix[kPow2][32];
  float f[kPow2][32];  // the same value
};

struct Weights {
  float top;              // the row's maximum
  float inv_hi, inv_lo;   // 1 / T
  int drop;               // 43 - weight_bits >= 0
};

// 2^weight_bits exp((x - top) / T), rounded.  x <= top, both finite or x =
// -inf.  About 35 instructions.
template <typename T>
__device__ __forceinline__ unsigned long long fixed_weight(const Weights& w, const Pow2Table& pow2, int lane, float x) {
  // (x - top) / T as y + yl.  The difference of two bf16 values is exact but
  // for a value 2^16 times smaller than the maximum; of two fp32 values its
  // rounding error is added back.
  const float d = x - w.top;
  const float y = d * w.inv_hi;
  float yl = fmaf(d, w.inv_lo, fmaf(d, w.inv_hi, -y));
  if (sizeof(T) == 4) {
    const float bb = d - x;
    yl = fmaf((x - (d - bb)) + (-w.top - bb), w.inv_hi, yl);
  }
  // k = rint(32 y / ln 2) through the last bits of a sum with 1.5 * 2^23.
  const float yc = fmaxf(y, -33.f);  // (-inf and what rounds to 0 in the end)
  const float kt = fmaf(yc, 46.16624f, 12582912.f);
  const float kf = kt - 12582912.f;
  const int k = __float_as_int(kt) - 0x4B400000;  // <= 0
  const float r = fmaf(-kf, 0x1.62e43p-6f, yc) + fmaf(kf, 0x1.05c61p-34f, yl);
  const int j = k & (kPow2 - 1);
  const float em1 = fmaf(r * r, fmaf(r, fmaf(r, 1.f / 24.f, 1.f / 6.f), 0.5f), r);
  const uint32_t v = pow2.fix[j][lane] + __float2int_rn(pow2.f[j][lane] * em1);  // 2^30 .. 2^31
  // v 2^13 / 2^sh, rounded: sh >= 0.
  const int sh = w.drop - (k >> 5);
  const unsigned long long u = ((unsigned long long)v << 14) >> sh;
  return y > -32.f ? (u + 1) >> 1 : 0ull;  // below 2^-46 of the maximum: 0
}

// c g, rounded, for c < 2^63 and a probability g (NaN and negative count as 0,
// above 1 as 1).  All of c enters the product: what a rejection leaves is a
// difference of nearly equal numbers, which an error of the cut alone would
// move by so much over the mass that is left (c cut to 31 bits: 4e-10 over it).
__device__ __forceinline__ unsigned long long cut_times(unsigned long long c, float g) {
  const uint32_t b = __float_as_uint(fminf(fmaxf(g, 0.f), 1.f));
  const uint32_t m = b << 8 | 0x80000000u;  // g = m 2^-32 2^(e - 126); (subnormals are shifted out)
  const unsigned long long t = (unsigned long long)(uint32_t)(c >> 32) * m + __umulhi((uint32_t)c, m);
  const int sh = 126 - (int)(b >> 23);
  unsigned long long u;
  asm("shr.u64 %0, %1, %2;" : "=l"(u) : "l"(t + t), "r"(sh));  // 0 for more than 63
  return sh < 0 ? c : (u + 1) >> 1;  // (sh < 0: g = 1)
}

// The two halves of a cluster barrier.  Another CTA's shared memory may be
// touched only once that CTA has started, which being scheduled together does
// not promise: every thread says so at its start, and waits for the others'
// behind what it would wait for anyway.
__device__ __forceinline__ void cluster_started() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_met() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

constexpr int kMaxRej = kMaxTreeRows;  // rejected siblings of one node

struct WalkShared {
  Pow2Table pow2;
  unsigned long long warps[2][kMaxWalkWarps];  // sums over each warp's part of the row
  unsigned long long ctas[2][kMaxCluster];  // and over each CTA's
  unsigned long long scale[kMaxRej + 1];  // c_k: sum of the weights left by k rejections
  unsigned long long cut[kMaxRej + 2];    // c_0 + .. + c_(k-1)
  float ctamax[2][kMaxCluster];
  int ctaat[2][kMaxCluster];
  float wmax[kMaxWalkWarps];
  int wat[kMaxWalkWarps];
  int rej_token[kMaxRej];
  unsigned err;
  int node, count, nrej, cmd, cursor;
  float rej_mass;
};

// The weights of a unit, below 2^40, in shared memory: their low words, and the
// fifth bytes of a lane's values (32 apart) in two words.
struct Unit {
  uint32_t lo[kUnit];
  uint32_t hi[2][32];
  __device__ __forceinline__ unsigned long long get(int i) const {
    return ((unsigned long long)(hi[i >> 7][i & 31] >> (8 * (i >> 5 & 3)) & 0xFFu) << 32) | lo[i];
  }
  __device__ __forceinline__ void clear(int i) {
    lo[i] = 0u;
    reinterpret_cast<unsigned char*>(&hi[i >> 7][i & 31])[i >> 5 & 3] = 0;
  }
};
static_assert(sizeof(Unit) == kUnit * kWeightBytes, "room of a unit");

// The rows' tests: p(x), g(x), u, the row's own maximum, x, the place of the
// maximum (-1: no distribution, -2: not known), the parent.
struct WalkRows {
  float *p, *q, *u, *top;
  int *token, *at, *par;
  __device__ __forceinline__ WalkRows(void* base, int n)
      : p((float*)base), q(p + n), u(q + n), top(u + n), token((int*)(top + n)), at(token + n), par(at + n) {}
};

// In three parts of 22 bits, whose sums fit 32.
__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
  const unsigned a = __reduce_add_sync(0xffffffffu, (unsigned)v & 0x3FFFFFu);
  const unsigned b = __reduce_add_sync(0xffffffffu, (unsigned)(v >> 22) & 0x3FFFFFu);
  const unsigned c = __reduce_add_sync(0xffffffffu, (unsigned)(v >> 44));
  return a + ((unsigned long long)b << 22) + ((unsigned long long)c << 44);
}

__device__ __forceinline__ unsigned long long warp_scan(unsigned long long v, int lane) {
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// The largest m of the warp and its lowest place; a place of -1 anywhere wins.
__device__ __forceinline__ void best_of_lanes(float& m, int& at) {
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, m, o);
    const int oa = __shfl_xor_sync(0xffffffffu, at, o);
    at = at < 0 || oa < 0 ? -1 : om > m ? oa : om == m ? min(at, oa) : at;
    m = fmaxf(m, om);
  }
}

// The walk runs for a few microseconds and most of its code once, so the
// instructions that it has to fetch count like the work: loops stay rolled,
// and what several places need is one function out of line.

// Weights of a unit of 256 values: this lane's values i, i + 32, .. into dst;
// their sum.  i counts from the row's start.
template <typename T>
__device__ __noinline__ unsigned long long fill_unit(const WalkShared& sh, const Weights w, const T* row, int vocab,
                                                     int i, Unit* dst) {
  const int lane = threadIdx.x & 31;
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = i + 32 * e < vocab ? to_float<T>(row[i + 32 * e]) : -INFINITY;
  unsigned long long sum = 0ull;
  uint32_t hi[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const unsigned long long v = fixed_weight<T>(w, sh.pow2, lane, x[e]);
    dst->lo[lane + 32 * e] = (uint32_t)v;
    hi[e / 4] |= (uint32_t)(v >> 32) << (8 * (e % 4));
    sum += v;
  }
  dst->hi[0][lane] = hi[0];
  dst->hi[1][lane] = hi[1];
  return sum;
}

// The sum of a lane's weights of a unit, less the cut times the drafted
// probabilities.  A rejection takes s to max(s - c g, 0), c the sum of all s
// before it; a weight that reached 0 stays there, so after several of them it
// is max(v - (c_0 + c_1 + ..) g, 0).
__device__ __noinline__ unsigned long long sum_unit(const Unit* src, const float* guess, int vocab, int i,
                                                    const unsigned long long cut) {
  const int lane = threadIdx.x & 31;
  unsigned long long sum = 0ull;
  float g[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) g[e] = cut && i + 32 * e < vocab ? guess[i + 32 * e] : 0.f;
  const uint32_t hi[2] = {src->hi[0][lane], src->hi[1][lane]};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const unsigned long long c = cut_times(cut, g[e]);
    const unsigned long long v = ((unsigned long long)(hi[e / 4] >> (8 * (e % 4)) & 0xFFu) << 32) | src->lo[lane + 32 * e];
    sum += v > c ? v - c : 0ull;
  }
  return sum;
}

// Walk of one sequence by a cluster.  Every CTA takes the same decisions
// from the same numbers, so the cluster's barriers always match.  Bound by
// latency while there are few sequences (one: 11 us; 3 us more for each rejected
// sibling, a pass over the kept weights and an exchange), then by its
// instructions: 32 drawn chains over 131,072 values 35 us, issue slots 43 % used;
// 0.5 us for every further sequence that is drawn from its logits.  (Clusters of
// 4, 2 and 1 for more sequences: the same time for those, half of it for greedy
// ones, a quarter more for chains with drafted probabilities, whose weights
// then do not fit.)
template <typename T, int kCluster, int kWalkThreads>
__global__ void __launch_bounds__(kWalkThreads, 1024 / kWalkThreads) accept_walk_kernel(const AcceptParams p) {
  constexpr int kWalkWarps = kWalkThreads / 32;
  constexpr int kSegs = kCluster * kWalkWarps;
  extern __shared__ __align__(16) uint32_t dynamic[];
  __shared__ WalkShared sh;
  asm volatile("griddepcontrol.launch_dependents;");
  cluster_started();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int s = blockIdx.x / kCluster;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
#pragma unroll 1
  for (int i = tid; i < kPow2 * 32; i += kWalkThreads) {
    sh.pow2.fix[i / 32][lane] = kPow2Fix[i / 32];
    sh.pow2.f[i / 32][lane] = (float)kPow2Fix[i / 32];
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  cluster_met();  // (ahead of every return)
  const int kind = accept_kind(p, s);
  const float temp = accept_temperature(p, s);
  const bool greedy = temp == 0.f;
  const float draw_v = p.sample_u[s];  // (used at the end)
  int row0, n;
  const bool fits = accept_rows(p, s, kind, &row0, &n);
  Unit* const weights = reinterpret_cast<Unit*>(dynamic);
  const WalkRows rows(weights + p.kept, p.max_rows);
  if (tid == 0) {
    sh.err = fits ? 0u : VA_DEV_BAD_ROWS;
    if (temp != 0.f && !(temp >= kMinTemperature && temp < INFINITY)) sh.err |= VA_DEV_BAD_SAMPLING;
    sh.node = 0;
    sh.count = 1;
    sh.nrej = 0;
    sh.cursor = 1;
    sh.rej_mass = 0.f;
    sh.cut[0] = 0ull;
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
#pragma unroll 1
  for (int j = tid; j < n; j += kWalkThreads) rows.at[j] = -2;  // no statistics
  __syncthreads();

  // Every row's test, at once: its parent, p(x) and g(x).  A warp per row
  // joins the statistics of its parent's pieces.
  const T* logits = reinterpret_cast<const T*>(p.logits);
  const float inv = greedy ? 0.f : 1.4426950408889634f / temp;
#pragma unroll 1
  for (int j = warp; j < n; j += kWalkWarps) {
    const int a = kind == 1 ? p.parent[row0 + j] : j - 1;
    if (kind == 1 && (j == 0 ? a != -1 : a < 0 || a >= j)) {
      if (lane == 0) atomicOr(&sh.err, VA_DEV_BAD_PARENT);
      continue;
    }
    if (j == 0) continue;
    // Loads that wait on nothing first.
    const float4* st = p.stats + (long long)(row0 + a) * p.pieces;
    const float4 none = make_float4(-INFINITY, 0.f, __int_as_float(INT_MAX), 0.f);
    const int x = p.tokens[row0 + j];
    const float u = p.accept_u[row0 + j];
    float4 t = lane < p.pieces ? st[lane] : none;
    if (x < 0 || x >= p.vocab) {
      if (lane == 0) atomicOr(&sh.err, VA_DEV_BAD_TOKEN);
      continue;
    }
    const float z = to_float<T>(logits[(long long)(row0 + a) * p.logits_stride + x]);
    const float g = p.probs ? p.probs[(long long)(row0 + a) * p.probs_stride + x] : 1.f;
    // At temperature 0 inv is 0 and the sums are 0 or NaN: the scaling by
    // exp2(0) (or by NaN, of a sum that is NaN anyway) changes nothing.
    // Pieces of -inf alone add nothing; a NaN in any piece stays.
    float m = -INFINITY, sum = 0.f;
    int at = INT_MAX;
#pragma unroll 1
    for (int c = lane; c < p.pieces; c += 32, t = c < p.pieces ? st[c] : none) {
      if (t.x > m) {
        sum = m == -INFINITY ? sum : sum * exp2_fast((m - t.x) * inv);
        m = t.x;
        at = __float_as_int(t.z);
      }
      sum += t.x == -INFINITY ? t.y : t.y * exp2_fast((t.x - m) * inv);
    }
#pragma unroll 1
    for (int o = 16; o > 0; o >>= 1) {
      const float om = __shfl_xor_sync(0xffffffffu, m, o), os = __shfl_xor_sync(0xffffffffu, sum, o);
      const int oa = __shfl_xor_sync(0xffffffffu, at, o);
      const float nm = fmaxf(m, om);
      sum = (m == -INFINITY ? sum : sum * exp2_fast((m - nm) * inv)) +
            (om == -INFINITY ? os : os * exp2_fast((om - nm) * inv));
      at = om > m ? oa : om == m ? min(at, oa) : at;
      m = nm;
    }
    if (lane == 0) {
      const bool usable = sum == sum && m < INFINITY && m > -INFINITY;
      rows.par[j] = a;
      rows.token[j] = x;
      rows.u[j] = u;
      rows.q[j] = g;
      rows.p[j] = !usable ? -1.f : greedy ? (x == at ? 1.f : 0.f) : exp2_fast((z - m) * inv) / sum;
      rows.top[a] = m;  // siblings write the same values
      rows.at[a] = usable ? at : -1;
    }
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
#pragma unroll 1
      for (int j = tid; j < n; j += kWalkThreads) p.accepted_nodes[row0 + j] = -1;
    }
    return;  // every CTA saw the same error and leaves here
  }

  // This warp's part of a row: per units of 256 values.  Their weights are
  // kept in shared memory where the parts fit (p.cached), else a unit's are
  // made in the warp's own place each time.
  const int per = (p.vocab + kUnit * kSegs - 1) / (kUnit * kSegs);
  const int lo = (rank * kWalkWarps + warp) * per * kUnit;
  const int units = lo < p.vocab ? min(per, (p.vocab - lo + kUnit - 1) / kUnit) : 0;
  Unit* const mine = weights + warp * (p.cached ? per : 1);
  Weights w;
  w.top = 0.f;
  w.drop = 43 - p.weight_bits;
  w.inv_hi = greedy ? 1.f : 1.f / temp;  // with its rounding error
  w.inv_lo = greedy ? 0.f : fmaf(-w.inv_hi, temp, 1.f) / temp;
  int at_node = -1;     // the node that the row variables describe
  int pass = 0;         // exchanges so far: the buffers alternate
  int have = -1;        // scale[0 .. have] hold sums at this node
  int best = -1;        // place of the row's maximum, -1: no distribution
  bool filled = false;  // the table of weights is this row's
  const T* row = nullptr;
  const float* guess = nullptr;

  // The sum of this lane's weights of unit k after the rejections; the
  // weights are in the table then.  Proposals without probabilities: a
  // rejected token weighs 0 there.
  unsigned long long cut = 0ull;
  auto unit_left = [&](int k, int nrej) {
    Unit* at = mine + (p.cached ? k : 0);
    const int i = lo + k * kUnit + lane;
    if (!filled) {
      unsigned long long sum = fill_unit<T>(sh, w, row, p.vocab, i, at);
      if (!p.probs && nrej > 0) {
        __syncwarp();
        const int x = lane < nrej ? sh.rej_token[lane] - (i - lane) : -1;
        if (x >= 0 && x < kUnit) {
          sum -= at->get(x);
          at->clear(x);
        }
        __syncwarp();
      }
      if (cut == 0ull) return sum;
    }
    return sum_unit(at, guess, p.vocab, i, cut);
  };

  enum { DONE = 0, NEED_SUMS = 1 };
  int left = 0;  // the rejections behind the last sums
  unsigned long long total = 0ull;
#pragma unroll 1
  for (;;) {
    if (warp == 0) {
      // Try the children of the node reached so far in row order: a taken
      // child becomes the node, and its children come after it.
      __syncwarp();
      int node = sh.node, count = sh.count, nrej = sh.nrej, j = sh.cursor;
      float mass = sh.rej_mass;
      int cmd = DONE;
      const int up = kind == 1 && lane > 0 && lane < n ? rows.par[lane] : -1;
#pragma unroll 1
      for (;;) {
        if (kind == 1) {
          const unsigned kids = __ballot_sync(0xffffffffu, up == node && lane >= j);
          j = kids ? __ffs(kids) - 1 : n;
        } else {
          j = j <= node + 1 ? node + 1 : n;
        }
        if (j >= n) break;
        const float u = rows.u[j], pj = rows.p[j], qj = rows.q[j];
        const int x = rows.token[j];
        bool yes = false, lost = false;  // taken; rejected, with an effect
        if (greedy || pj < 0.f) {
          yes = pj > 0.f;  // below 0: the row has no distribution
        } else if (!p.probs) {
          const bool again = __any_sync(0xffffffffu, lane < nrej && sh.rej_token[lane] == x);
          yes = !again && u * (1.f - mass) < pj;
          lost = !yes && !again;
        } else if (nrej == 0) {
          yes = u * qj < pj;
          lost = !yes;
        } else if (have < nrej) {
          cmd = NEED_SUMS;  // the weights left by the rejected siblings
          break;
        } else {
          const float z = to_float<T>(logits[(long long)(row0 + node) * p.logits_stride + x]);
          const unsigned long long v = fixed_weight<T>(w, sh.pow2, lane, z);
          const unsigned long long c = cut_times(sh.cut[nrej], qj);
          yes = (double)u * (double)qj * (double)sh.scale[nrej] < (double)(v > c ? v - c : 0ull);
          lost = !yes;
        }
        if (yes) {
          if (rank == 0 && lane == 0) p.accepted_nodes[row0 + count] = j;
          node = j;
          ++count;
          nrej = 0;
          mass = 0.f;
          have = -1;
        } else if (lost) {
          if (!p.probs && lane == 0) sh.rej_token[nrej] = x;
          __syncwarp();
          ++nrej;
          mass += pj;
        }
        ++j;
      }
      __syncwarp();
      if (lane == 0) {
        sh.node = node;
        sh.count = count;
        sh.nrej = nrej;
        sh.cursor = j;
        sh.rej_mass = mass;
        sh.cmd = cmd;
      }
    }
    __syncthreads();
    const int node = sh.node, cmd = sh.cmd, nrej = sh.nrej;
    if (node != at_node) {
      at_node = node;
      row = logits + (long long)(row0 + node) * p.logits_stride;
      guess = p.probs ? p.probs + (long long)(row0 + node) * p.probs_stride : nullptr;
      have = -1;
      filled = false;
      w.top = rows.top[node];
      best = rows.at[node];
      if (best == -2) {
        // The statistics kernel left the row out (a leaf): its maximum.
        float m = -INFINITY;
        int at = INT_MAX;
        bool odd = false;
        const int end = min(lo + units * kUnit, p.vocab);
#pragma unroll 8
        for (int i = lo + lane; i < end; i += 32) {
          const float x = to_float<T>(row[i]);
          odd |= !(x < INFINITY);
          if (x > m) {
            m = x;
            at = i;
          }
        }
        if (odd) at = -1;
        best_of_lanes(m, at);
        const int b = pass++ & 1;
        if (lane == 0) {
          sh.wmax[warp] = m;
          sh.wat[warp] = at;
        }
        __syncthreads();
        if (warp == 0) {
          m = lane < kWalkWarps ? sh.wmax[lane] : -INFINITY;
          at = lane < kWalkWarps ? sh.wat[lane] : INT_MAX;
          best_of_lanes(m, at);
          if (lane < kCluster) {
            *cluster.map_shared_rank(&sh.ctamax[b][rank], lane) = m;
            *cluster.map_shared_rank(&sh.ctaat[b][rank], lane) = at;
          }
        }
        cluster.sync();
        m = lane < kCluster ? sh.ctamax[b][lane] : -INFINITY;
        at = lane < kCluster ? sh.ctaat[b][lane] : INT_MAX;
        best_of_lanes(m, at);
        w.top = m;
        best = at == INT_MAX ? -1 : at;  // nothing but -inf
      }
    }
    if (cmd == DONE && (greedy || best < 0)) break;
    // Sums of what the rejections left, one exchange each (proposals without
    // probabilities: of what all of them left, at once).
    left = nrej;
#pragma unroll 1
    for (int k = p.probs ? min(have + 1, nrej) : nrej;;) {
      unsigned long long v = 0ull;
      cut = p.probs ? sh.cut[k] : 0ull;
#pragma unroll 1
      for (int t = 0; t < units; ++t) v += unit_left(t, k);
      filled = p.cached;
      // Each warp's sum into this CTA's table, each CTA's into every CTA's.
      v = warp_sum(v);
      const int b = pass++ & 1;
      if (lane == 0) sh.warps[b][warp] = v;
      __syncthreads();
      if (warp == 0) {
        const unsigned long long c = warp_sum(lane < kWalkWarps ? sh.warps[b][lane] : 0ull);
        if (lane < kCluster) *cluster.map_shared_rank(&sh.ctas[b][rank], lane) = c;
      }
      cluster.sync();
      total = warp_sum(lane < kCluster ? sh.ctas[b][lane] : 0ull);
      if (p.probs) {
        if (tid == 0) {
          sh.scale[k] = total;
          sh.cut[k + 1] = sh.cut[k] + total;
        }
        __syncthreads();
        have = k;
      }
      if (total == 0ull && k > 0) {
        // Nothing is left: the next sibling, or the draw, meets p itself.
        left = k = 0;
        filled = filled && p.probs;
        if (cmd == DONE) continue;
        have = 0;
        if (tid == 0) sh.nrej = 0;
        break;
      }
      if (k++ == left) break;
    }
    if (cmd == DONE) break;
  }

  // Outputs of the walk.
  const int count = sh.count;
  if (rank == 0) {
    if (tid == 0) {
      p.accepted_len[s] = count;
      if (p.promote_len) p.promote_len[s] = kind == 1 ? count : 0;
      p.accepted_nodes[row0] = 0;
      if (best < 0) flag(p.status, VA_DEV_BAD_LOGITS);
      if (best < 0 || greedy) p.next_token[s] = best;
    }
#pragma unroll 1
    for (int j = count + tid; j < n; j += kWalkThreads) p.accepted_nodes[row0 + j] = -1;
  }
  // The next token, from what is left at the last node: the lowest i whose
  // running sum passes t = floor(v total).
  if (best >= 0 && !greedy) {
    const float v = draw_v;
    unsigned long long t = v > 0.f ? __umul64hi(total, v < 1.f ? (unsigned long long)__float2ull_rz(v * 0x1p63f) << 1
                                                               : ~0ull)
                                   : 0ull;
    if (t >= total) t = total - 1;
    const int b = (pass & 1) ^ 1;  // the last sums
    unsigned long long base = warp_sum(lane < rank ? sh.ctas[b][lane] : 0ull);
    base += warp_sum(lane < warp ? sh.warps[b][lane] : 0ull);
    if (t >= base && t - base < sh.warps[b][warp]) {
      // One warp owns the border: the unit that holds it, then the 32 values.
#pragma unroll 1
      for (int k = 0; k < units; ++k) {
        // (The last unit holds it if the ones before it do not.)
        if (!filled || k + 1 < units) {
          const unsigned long long sum = warp_sum(unit_left(k, left));
          if (t - base >= sum) {
            base += sum;
            continue;
          }
        }
        const Unit* at = mine + (p.cached ? k : 0);
#pragma unroll 1
        for (int i = lo + k * kUnit + lane, e = 0; e < kUnit / 32; ++e, i += 32) {
          const unsigned long long c = cut && i < p.vocab ? cut_times(cut, guess[i]) : 0ull;
          const unsigned long long w = at->get(lane + 32 * e), x = w > c ? w - c : 0ull;
          const unsigned long long sum = warp_sum(x);
          if (t - base < sum) {
            const unsigned hit = __ballot_sync(0xffffffffu, t < warp_scan(x, lane) + base);
            if (lane == __ffs(hit) - 1) p.next_token[s] = i;
            break;
          }
          base += sum;
        }
        break;
      }
    }
  }
  cluster.sync();  // no CTA leaves while another may still write its tables
}

// A row may start up to 7 values past a 16-byte boundary (so that a vocabulary of
// whole pieces has one more, which holds values of such rows only).
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

// Launch configuration of a kernel that starts early and waits for the work
// before it on the stream (programmatic dependent).
struct Launch {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  Launch(unsigned gx, unsigned gy, unsigned gz, int threads, int cluster, size_t smem, cudaStream_t st) {
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(gx, gy, gz);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
  }
};

// A walk of clusters of kCluster CTAs of kThreads threads.
constexpr int kMaxDevices = 64;

template <typename T, int kCluster, int kThreads>
struct Walk {
  static constexpr int kMaxBytes = kWalkBytes / (1024 / kThreads);

  // Sets the kernel's limits, once per device; how many clusters run at once
  // (0: none, a GPC has too few SMs).
  static cudaError_t prepare(int dev, int* at_once) {
    static std::atomic<int> known[kMaxDevices];  // one more than that
    int n = known[dev].load(std::memory_order_acquire) - 1;
    if (n < 0) {
      auto* kernel = accept_walk_kernel<T, kCluster, kThreads>;
      cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxBytes);
      if (e == cudaSuccess && kCluster > 8)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      Launch l(kCluster, 1, 1, kThreads, kCluster, kMaxBytes, nullptr);
      if (cudaOccupancyMaxActiveClusters(&n, kernel, &l.cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
      }
      known[dev].store(n + 1, std::memory_order_release);
    }
    *at_once = n;
    return cudaSuccess;
  }

  static cudaError_t launch(AcceptParams q, cudaStream_t st) {
    // The weights of a CTA's part of the row where they fit beside the rows'
    // tests, else one unit per warp.
    constexpr int W = kThreads / 32;
    const int per = (q.vocab + kUnit * kCluster * W - 1) / (kUnit * kCluster * W);
    const int tests = kRowBytes * q.max_rows;
    q.cached = per * W * (int)sizeof(Unit) + tests <= kMaxBytes;
    q.kept = (q.cached ? per : 1) * W;
    Launch l((unsigned)(q.num_seqs * kCluster), 1, 1, kThreads, kCluster,
             (size_t)(q.kept * (int)sizeof(Unit) + tests), st);
    cudaError_t e = cudaLaunchKernelEx(&l.cfg, accept_walk_kernel<T, kCluster, kThreads>, q);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
};

template <typename T>
static cudaError_t launch_accept(const AcceptParams& q, cudaStream_t st) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  // As many threads to a sequence as let all sequences run at once: clusters of
  // 16 CTAs of 1,024 threads (7 of them; 4 sequences of trees and chains over
  // 100,000 values and more 17 to 34 us against 19 to 39 with 512; up to 65,536
  // values, one unit per warp, the smaller CTAs start sooner: 7.5 us against
  // 8.0), of 512 (14), or of 8.
  int n = 0;
  int kind = 0;
  if (q.vocab > 16 * 16 * kUnit && (e = Walk<T, 16, 1024>::prepare(dev, &n)) == cudaSuccess && q.num_seqs <= n) kind = 2;
  if (e == cudaSuccess && kind == 0 && (e = Walk<T, 16, 512>::prepare(dev, &n)) == cudaSuccess && q.num_seqs <= n) kind = 1;
  if (e == cudaSuccess && kind == 0) e = Walk<T, 8, 512>::prepare(dev, &n);
  if (e != cudaSuccess) return e;
  // A sequence of one row has no proposal: nothing to prepare.
  if (q.max_rows > 1) {
    Launch l((unsigned)((q.pieces + kStatWarps - 1) / kStatWarps), (unsigned)q.max_rows, (unsigned)q.num_seqs,
             kStatThreads, 1, 0, st);
    e = cudaLaunchKernelEx(&l.cfg, accept_stats_kernel<T>, q);
    if (e != cudaSuccess) return e;
  }
  if (kind == 2) return Walk<T, 16, 1024>::launch(q, st);
  return kind == 1 ? Walk<T, 16, 512>::launch(q, st) : Walk<T, 8, 512>::launch(q, st);
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
  // The weights of a row sum to at most 2^58, the cuts of 31 rejections to 2^63; a
  // weight is at most 2^39 (kWeightBytes).
  int bits = 58;
  while (bits > 38 && (1LL << (58 - bits)) < d->vocab) --bits;
  q.weight_bits = bits < 39 ? bits : 39;
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
