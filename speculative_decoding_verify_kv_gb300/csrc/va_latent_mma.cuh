// What the tensor-core kernels over latent caches and prompt keys share: MMAs,
// commits and copies issued by an elected lane, barriers asked without waiting,
// tensor maps.
#pragma once

#include <string.h>

#include "va_latent.cuh"
#include "va_sm100.cuh"
#include "va_tma.h"

namespace va {
using namespace sm100;

constexpr uint64_t kLatentWaitNs = 2000000000ull;

__device__ __forceinline__ float lu_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Three maxima, and two products and sums, to an instruction.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t d, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// MMAs and commits that a whole warp runs through and its elected lane (e != 0)
// issues, with everything they are computed from known to be the warp's:
// descriptors then live in uniform registers.  An issuing thread of its own
// branch took some 100 cycles to an MMA, longer than one of 64 columns runs
// (64 heads x 16 rows x 4 sequences of 8,000 tokens: 142 us against 93; prompts
// of 2 x 2,048 rows, 128 heads, over 4,096 keys: 966 against 760).
__device__ __forceinline__ uint32_t elected() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(e));
  return e;
}

__device__ __forceinline__ void mma_ts_by(uint32_t e, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
      "r"(accumulate), "r"(e)
      : "memory");
}

// PAIR: one product over both CTAs of a pair (cta_group::2), issued by the first:
// each holds its own rows of A and D and half of B, and a commit arrives in both.
template <bool PAIR = false>
__device__ __forceinline__ void mma_ss_by(uint32_t e, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "r"(accumulate), "r"(e)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "r"(accumulate), "r"(e)
        : "memory");
}

template <bool PAIR = false>
__device__ __forceinline__ void commit_by(uint32_t e, uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred q;\n\t.reg .b16 m;\n\t"
        "setp.ne.b32 q, %1, 0;\n\tmov.b16 m, 3;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(bar), "r"(e)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(e)
        : "memory");
}

// Of a pair: by one warp of each CTA.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// The same place in the shared memory of the pair's first CTA, and an arrival there.
__device__ __forceinline__ uint32_t at_first(uint32_t addr) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Writes to the same place in CTA `rank` of the cluster.
__device__ __forceinline__ void store_at(uint32_t addr, int rank, int v) {
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.volatile.shared::cluster.b32 [a], %2;\n\t}" ::"r"(addr), "r"(rank),
               "r"(v)
               : "memory");
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Whether a phase has completed already.  Asked before an MMA group and used
// after it, so that the answer is there when the issuer gets to it: a wait, even
// one that passes, otherwise stands between two groups for some 150 cycles, and
// the matrix unit holds only a few MMAs in advance.
__device__ __forceinline__ bool mbar_peek(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void expect_by(uint32_t e, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %2, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes), "r"(e)
      : "memory");
}

__device__ __forceinline__ void tma_2d_by(uint32_t e, uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
      "l"(map), "r"(c0), "r"(c1), "r"(bar), "r"(e)
      : "memory");
}

// PAIR: the barrier may be the other CTA's.
template <bool PAIR = false>
__device__ __forceinline__ void tma_3d_by(uint32_t e, uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "r"(e)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n\t}" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "r"(e)
        : "memory");
}

// A kernel that gave up on a wait ends only when its copies have landed.  Each warp
// drains those whose barriers it armed; a copy counted on a barrier that another warp
// or CTA did not come to arm, or issued by a warp that saw no failure, cannot be asked
// about, so the kernel also lets the time pass (copies take some microseconds).
constexpr uint64_t kSettleNs = 2000000ull;
__device__ __forceinline__ void settle() {
  const uint64_t t0 = globaltimer();
  while (globaltimer() - t0 < kSettleNs) __nanosleep(1000);
}

// Zeros in rows from .. to - 1 of a 64-column block, by a warp.
__device__ __forceinline__ void clear_rows(unsigned char* block, int from, int to, int lane) {
  for (int x = from * 128 + lane * 16; x < to * 128; x += 512) *reinterpret_cast<uint4*>(block + x) = make_uint4(0u, 0u, 0u, 0u);
}

// ---------------------------------------------------------------------------
// Tiled map of bf16 rows in boxes of 64 columns, 128-byte swizzle.
inline bool latent_map(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                   const cuuint32_t* box) {
  const EncodeTiledFn fn = encode_fn();
  const cuuint32_t es[3] = {1, 1, 1};
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Absorbed form: all query rows of a launch, in boxes of `rows`; the cache, in
// boxes of a page.
inline bool latent_query_map(CUtensorMap* map, const LatentParams& p, int rows) {
  const cuuint64_t dk = (cuuint64_t)p.DK;
  const cuuint64_t dims[2] = {dk, (cuuint64_t)p.total_rows * (cuuint64_t)p.H}, strides[1] = {dk * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)rows};
  return latent_map(map, p.q, 2, dims, strides, box);
}

inline bool latent_cache_map(CUtensorMap* map, const LatentParams& p) {
  const cuuint64_t dk = (cuuint64_t)p.DK, rows = p.page_size ? (cuuint64_t)kPage : (cuuint64_t)p.capacity;
  const cuuint64_t dims[3] = {dk, rows, (cuuint64_t)(p.page_size ? p.num_blocks : p.num_seqs)};
  const cuuint64_t strides[2] = {dk * 2, rows * dk * 2};
  const cuuint32_t box[3] = {64, kPage, 1};
  return latent_map(map, p.cache, 3, dims, strides, box);
}

}  // namespace va
