// Where the rows of a windowed call go: joining the chunks of a sequence and KV
// head in one cluster, and writing rows out.
#pragma once

#include <cooperative_groups.h>
#include <string.h>

#include <atomic>

#include "va_common.cuh"

namespace va {
namespace cg = cooperative_groups;

// Chunks that may be joined in their kernel, as one cluster; otherwise they go
// through the workspace and the merge kernel.  Both take the same sums in the
// same order, so that either gives the same bits.  With at most 16 rows per KV
// head up to 16 (one token, 16 chunks at D = 64: 7.4 us against 12.5 through the
// merge kernel), with more rows 8, the portable size (96 rows of D = 256 in 16
// chunks: 29.6 us joined, 26.5 merged).
constexpr int kJoinFew = 16;
constexpr int kJoinMany = 8;

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

// Rows of a sequence whose row range is inconsistent come out NaN (called
// where no merge kernel follows).
template <int D>
__device__ __forceinline__ void nan_rows(const Params& p, int s, int kvh) {
  const int a = max(p.cu_rows[s], 0), b = min(p.cu_rows[s + 1], p.total_rows);
  for (long long i = (long long)a * p.H * D + threadIdx.x; i < (long long)b * p.H * D; i += blockDim.x)
    if (i / D % p.H / p.G == kvh) {
      if (p.o_bf16) reinterpret_cast<__nv_bfloat16*>(p.o)[i] = __float2bfloat16(NAN);
      else p.o[i] = NAN;
      if (i % D == 0) p.lse[i / D] = NAN;
    }
}

// Where a row's result goes: with one chunk the outputs, and else the chunk's
// partial for the merge kernel.
template <int D>
__device__ __forceinline__ void put_pair(const Params& p, bool partial, int slot, int grow, int head, int c, float x,
                                         float y) {
  const long long item = (long long)grow * p.H + head;
  if (partial)
    *reinterpret_cast<float2*>(p.ws_acc + slot_index(p, slot, grow, head) * D + c) = make_float2(x, y);
  else if (p.o_bf16)
    reinterpret_cast<uint32_t*>(p.o)[(item * D + c) / 2] = pack_bf16(x, y);
  else
    *reinterpret_cast<float2*>(p.o + item * D + c) = make_float2(x, y);
}

// Join the chunks of a cluster, in chunk order, through distributed shared
// memory: row r of this CTA's chunk has its unnormalised O at os + r ld and its m
// and l (in base 2) at ms[r mld] and ls[r mld].  A chunk without a visible token
// has l = 0 and weighs nothing (its O is not used), a failed one is NaN.  Every
// thread of every CTA of the cluster; a warp takes 64 columns of a row at a time,
// with the loads from all chunks in flight together (a round trip to another
// CTA's memory takes 0.6 us: one row's join 3.1 us with four of them in a row).
template <int D, int MAXC>
__device__ __forceinline__ void join_chunks(const Params& p, int slot, int row0, int kvh, int R, float* os, int ld,
                                            float* ms, float* ls, int mld) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  // Whole rows where there is one for every warp.
  const int parts = R < warps * p.slots ? D / 64 : 1;
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  for (int item = warp * p.slots + slot; item < R * parts; item += warps * p.slots) {
    const int r = item / parts, part = item - r * parts;
    // Lane k holds chunk k's m and l.
    const bool in = lane < p.slots;
    const float mk = in ? *cluster.map_shared_rank(ms + r * mld, lane) : -INFINITY;
    const float lk = in ? *cluster.map_shared_rank(ls + r * mld, lane) : 0.f;
    float2 v[MAXC];
    auto load = [&](int c) {
#pragma unroll
      for (int k = 0; k < MAXC; ++k)
        if (k < p.slots) v[k] = *reinterpret_cast<const float2*>(cluster.map_shared_rank(os + r * ld + c, k));
    };
    load(64 * part + 2 * lane);
    float mr = lk > 0.f ? mk : -INFINITY;
#pragma unroll
    for (int o = MAXC / 2; o > 0; o >>= 1) mr = fmaxf(mr, __shfl_xor_sync(0xffffffffu, mr, o));
    mr = __shfl_sync(0xffffffffu, mr, 0);
    const bool bad = __any_sync(0xffffffffu, lk != lk);
    const float fk = lk > 0.f ? ex2f(mk - mr) : 0.f;
    float lr = 0.f, w[MAXC];
#pragma unroll
    for (int k = 0; k < MAXC; ++k) {
      if (k % 8 == 0 && k >= p.slots) break;
      w[k] = __shfl_sync(0xffffffffu, fk, k);
      lr = fmaf(w[k], __shfl_sync(0xffffffffu, lk, k), lr);
    }
    const float inv = bad ? NAN : 1.f / lr;
    const int grow = row0 + r / p.G, head = kvh * p.G + r % p.G;
    for (int c = 64 * part + 2 * lane;;) {
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int k = 0; k < MAXC; ++k) {
        if (k % 8 == 0 && k >= p.slots) break;
        if (k >= p.slots || !(w[k] > 0.f)) continue;
        x = fmaf(w[k], v[k].x, x);
        y = fmaf(w[k], v[k].y, y);
      }
      put_pair<D>(p, false, slot, grow, head, c, x * inv, y * inv);
      c += 64;
      if (parts > 1 || c >= D) break;
      load(c);
    }
    if (lane == 0 && part == 0) p.lse[(long long)grow * p.H + head] = bad ? NAN : (mr + log2f(lr)) * kLn2;
  }
  cluster.sync();  // no CTA leaves while its rows are read
}

// Launch configuration of these kernels: a programmatic dependent, a sequence
// and KV head's chunks one cluster where they are joined in the kernel.
struct WindowLaunch {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  WindowLaunch(const Params& p, int threads, size_t smem, cudaStream_t st) {
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3((unsigned)p.slots, (unsigned)p.KVH, (unsigned)p.num_seqs);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.slots;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.slots > 1 && p.joined ? 2 : 1;
  }
};

// Whether a launch's chunks are joined in the kernel: where a cluster holds
// them all and the clusters need no more rounds on the GPU than the CTAs by
// themselves would (a GPC takes whole clusters only: 24 clusters of 6 CTAs
// that fill an SM each took 74 us in two rounds, 41 us apart).
template <auto KERNEL, int MAXC>
static bool chunks_join(Params p, int threads, size_t smem, cudaStream_t st) {
  // (join_chunks takes the rows of one row block.)
  if (p.slots > MAXC || p.row_blocks > 1) return false;
  if (p.slots == 1) return true;
  constexpr int kDevs = 64;
  static std::atomic<int> clusters[kDevs][MAXC + 1], ctas[kDevs];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevs) return false;
  // (Stored one higher: 0 is not known yet, 1 none.)
  int n = clusters[dev][p.slots].load(std::memory_order_relaxed) - 1;
  int c = ctas[dev].load(std::memory_order_relaxed) - 1;
  if (n < 0 || c < 0) {
    p.joined = 1;
    WindowLaunch l(p, threads, smem, st);
    int per = 0, sms = 0;
    if ((p.slots > 8 && cudaFuncSetAttribute(KERNEL, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) ||
        cudaOccupancyMaxActiveClusters(&n, KERNEL, &l.cfg) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, KERNEL, threads, smem) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    c = per * sms;
    clusters[dev][p.slots].store(n + 1, std::memory_order_relaxed);
    ctas[dev].store(c + 1, std::memory_order_relaxed);
  }
  if (n < 1 || c < 1) return false;
  const long long jobs = (long long)p.num_seqs * p.KVH;
  return (jobs + n - 1) / n <= (jobs * p.slots + c - 1) / c;
}

}  // namespace va
