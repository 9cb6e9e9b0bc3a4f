// Entry points of the attention over latent caches and of prompt segments:
// checks, plan, launches.
#include <math.h>
#include <string.h>

#include "va_latent.cuh"

namespace va {

struct LatentPlan {
  int kernel;          // VA_KERNEL_*
  bool few;            // the tensor-core kernel for few query rows
  bool pair;           // that of CTA pairs
  int rows_per_block;  // query rows of a CTA
  int parts;           // CTAs that share a row block's chunk
  int per_sm;          // CTAs of an SM
  int slots;
  bool many;           // more than eight chunks of a sequence of the most rows
  int part_seq;        // see latent_part
  int merge_seq;       // as in LatentParams
  size_t acc_bytes, ws_bytes;
  dim3 grid;
};

static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// What both entry points ask of the query side.
static va_status check_queries(const va_problem* p, int dtype) {
  if (p->num_seqs < 1 || p->num_heads < 1) return VA_ERR_INVALID_ARG;
  if (p->total_rows < 0 || p->num_splits < 1 || p->max_rows_per_seq < 1) return VA_ERR_INVALID_ARG;
  if (dtype < VA_F32 || dtype > VA_Q8_0 || p->q_dtype < VA_F32 || p->q_dtype > VA_Q8_0) return VA_ERR_INVALID_ARG;
  if (dtype == VA_Q8_0 || (int)p->q_dtype != dtype) return VA_ERR_UNSUPPORTED;
  if (p->num_heads > VA_MAX_LATENT_HEADS || p->num_splits > 256 || p->num_seqs > 65535) return VA_ERR_UNSUPPORTED;
  if (!(p->scale >= 0.f) || isinf(p->scale)) return VA_ERR_INVALID_ARG;
  if (p->flags & ~(uint32_t)VA_FLAG_CUDA_CORES) return VA_ERR_INVALID_ARG;
  // One launch covers every (row, head) with a warp each.
  if ((long long)p->total_rows * p->num_heads > 0x7fffffffLL) return VA_ERR_UNSUPPORTED;
  if (!p->cu_rows || (p->total_rows > 0 && !p->q)) return VA_ERR_INVALID_ARG;
  if ((uintptr_t)p->q % 16) return VA_ERR_ALIGNMENT;
  return VA_OK;
}

static va_status check_latent(const va_problem* p, const va_latent* kv, int mode) {
  if (!p || !kv || mode < VA_MODE_CHAIN || mode > VA_MODE_MIXED) return VA_ERR_INVALID_ARG;
  va_status st = check_queries(p, kv->dtype);
  if (st != VA_OK) return st;
  if (kv->latent_dim != 256 && kv->latent_dim != 512) return VA_ERR_UNSUPPORTED;
  if (kv->rope_dim != kLatentRope) return VA_ERR_UNSUPPORTED;
  if (p->max_rows_per_seq > kMaxRows) return VA_ERR_UNSUPPORTED;
  if (mode == VA_MODE_TREE && p->max_rows_per_seq > kMaxTreeRows) return VA_ERR_UNSUPPORTED;
  if (!(p->scale > 0.f) || !p->ctx_len || !kv->cache) return VA_ERR_INVALID_ARG;
  if (mode != VA_MODE_CHAIN && !p->parent) return VA_ERR_INVALID_ARG;
  if (mode == VA_MODE_MIXED && !p->seq_kind) return VA_ERR_INVALID_ARG;
  if (kv->page_size == 0) {
    if (kv->capacity < 1) return VA_ERR_INVALID_ARG;
    if (kv->capacity % kPage || kv->capacity > (1LL << 28)) return VA_ERR_UNSUPPORTED;
  } else if (kv->page_size == kPage) {
    if (!kv->block_table || kv->max_blocks_per_seq < 1 || kv->num_blocks < 1) return VA_ERR_INVALID_ARG;
    if (kv->max_blocks_per_seq > (1 << 26)) return VA_ERR_UNSUPPORTED;
  } else {
    return VA_ERR_UNSUPPORTED;
  }
  if ((uintptr_t)kv->cache % 16) return VA_ERR_ALIGNMENT;
  return VA_OK;
}

constexpr int kMaxPromptRows = 1 << 22;

static va_status check_prompt(const va_problem* p, const va_prompt* kv) {
  if (!p || !kv) return VA_ERR_INVALID_ARG;
  va_status st = check_queries(p, kv->dtype);
  if (st != VA_OK) return st;
  if (kv->nope_dim != 64 && kv->nope_dim != 128) return VA_ERR_UNSUPPORTED;
  if (kv->value_dim != kv->nope_dim || kv->rope_dim != kLatentRope) return VA_ERR_UNSUPPORTED;
  if (p->max_rows_per_seq > kMaxPromptRows || kv->total_kv > (1 << 30)) return VA_ERR_UNSUPPORTED;
  if (kv->total_kv < 0 || !kv->cu_kv || (kv->causal != 0 && kv->causal != 1)) return VA_ERR_INVALID_ARG;
  if (kv->total_kv > 0 && (!kv->kv || !kv->k_rope)) return VA_ERR_INVALID_ARG;
  if (kv->total_kv > 1 && kv->k_rope_stride < kv->rope_dim) return VA_ERR_INVALID_ARG;
  const int size = kv->dtype == VA_F32 ? 4 : 2;
  if (((uintptr_t)kv->kv | (uintptr_t)kv->k_rope) % 16 || kv->k_rope_stride * size % 16) return VA_ERR_ALIGNMENT;
  return VA_OK;
}

static LatentPlan plan_rows(const va_problem* p, int dtype, int value_dim, bool prompt) {
  LatentPlan pl;
  memset((void*)&pl, 0, sizeof(pl));
  if (dtype == VA_BF16 && !(p->flags & VA_FLAG_CUDA_CORES)) {
    pl.kernel = VA_KERNEL_TENSOR;
    const int few = prompt ? 0 : latent_rows_rows((long long)p->max_rows_per_seq * p->num_heads);
    pl.few = few > 0;
    pl.rows_per_block = prompt ? latent_prompt_rows() : few ? few : latent_umma_rows();
    // 512 latent columns: pairs of CTAs.  64 heads x 16 rows x 4 sequences of 8,000
    // tokens took the 128-row kernel, with O's columns dealt to two CTAs, 86 us
    // (64), 32 sequences of 5,100 and 64 heads 70 (55).
    pl.pair = !few && !prompt && value_dim == 512;
    if (pl.pair) pl.rows_per_block = latent_pair_rows();
    pl.parts = pl.pair ? 2 : 1;
    pl.per_sm = 1;
  } else {
    pl.kernel = VA_KERNEL_CUDA_CORES;
    pl.rows_per_block = latent_simt_rows();
    pl.parts = 1;
    pl.per_sm = 2;
  }
  pl.slots = p->num_splits;
  const long long rows = (long long)p->max_rows_per_seq * (prompt ? 1 : p->num_heads);
  const long long blocks = (rows + pl.rows_per_block - 1) / pl.rows_per_block;
  pl.many = pl.slots / (blocks > 0 ? blocks : 1) > 8;
  // A sequence of b row blocks has b max(1, slots / b) CTAs per key head.
  pl.grid = dim3((unsigned)(blocks > pl.slots ? blocks : pl.slots), (unsigned)(prompt ? p->num_heads : 1),
                 (unsigned)p->num_seqs);
  if (prompt && pl.kernel == VA_KERNEL_TENSOR) {
    // All sequences' blocks in a row; a sequence of b takes at most b + slots - 1.
    const long long most = (long long)pl.grid.x * p->num_seqs;
    const long long rows_most = p->total_rows / pl.rows_per_block + (long long)p->num_seqs * pl.slots;
    pl.grid = dim3((unsigned)(most < rows_most ? most : rows_most), (unsigned)p->num_heads, 1u);
  }
  if (pl.slots > 1) {
    const long long all = (long long)p->total_rows * p->num_heads;
    const long long seq = (rows < pl.rows_per_block ? rows : pl.rows_per_block) * (prompt ? p->num_heads : 1);
    if (seq * p->num_seqs < all) pl.part_seq = (int)seq;
    // Two chunks and more: no more row blocks than half of the slots.
    const long long cut = (long long)(pl.slots / 2) * pl.rows_per_block;
    const long long merged = (rows < cut ? rows : cut) * (prompt ? p->num_heads : 1);
    if (merged * p->num_seqs <= all) pl.merge_seq = (int)merged;
    const size_t items = (size_t)pl.slots * (size_t)(pl.part_seq ? seq * p->num_seqs : all);
    pl.acc_bytes = up256(items * (size_t)value_dim * 4);
    pl.ws_bytes = pl.acc_bytes + up256(items * 8);
  }
  return pl;
}

static LatentPlan plan_latent(const va_problem* p, const va_latent* kv) {
  return plan_rows(p, kv->dtype, kv->latent_dim, false);
}

static LatentPlan plan_prompt(const va_problem* p, const va_prompt* kv) {
  return plan_rows(p, kv->dtype, kv->value_dim, true);
}

// Chunks that fill the GPU once: a sequence's row blocks share the count out.  (More
// blocks than half of the count leave a sequence uncut; the count stays, since one with
// fewer rows than the bound is cut all the same: 4 sequences of one row, 128 heads over
// 8,000 tokens, a bound of 16 rows, 26 us, and 92 with a count of 1.  What it costs where
// all are uncut is the merge that finds nothing: 300 rows of 128 heads 140 us for 135.)
static int32_t fill(const va_problem* p, const LatentPlan& pl, int heads) {
  const long long c = (long long)pl.per_sm * sm_count() / ((long long)p->num_seqs * heads * pl.parts);
  return (int32_t)(c < 1 ? 1 : c > 256 ? 256 : c);
}

// Keys that a chunk of a prompt should have on the tensor cores before its
// partials and their merge pay.  One segment of 256 rows, us uncut and in two chunks:
// 32 heads over 1,024 keys 13.3 and 16.9, 2,048 19.9 and 20.0, 4,096 33.3 and 26.9; 16
// heads 12.8 and 14.7, 19.4 and 17.6, 32.8 and 24.4; one head 12.4 and 12.1, 19.0 and
// 15.3, 32.2 and 21.9.  Shorter chunks pay where a few blocks leave the GPU empty: one
// head over 16,384 keys 16.5 in the 16 chunks of this rule, 12.9 in 64.
constexpr int kPromptChunkKeys = 1024;

static LatentParams base_params(const va_problem* p, int mode, const LatentPlan& pl, int key_dim, int value_dim,
                                int dtype, void* ws, void* o, float* lse, uint32_t* status) {
  LatentParams q;
  memset(&q, 0, sizeof(q));
  q.num_seqs = p->num_seqs;
  q.H = p->num_heads;
  q.total_rows = p->total_rows;
  q.max_rows = p->max_rows_per_seq;
  q.mode = mode;
  q.DK = key_dim;
  q.DV = value_dim;
  const double scale = p->scale > 0.f ? (double)p->scale : 1.0 / sqrt((double)key_dim);
  q.scale_log2 = (float)(scale * 1.4426950408889634);
  q.scale_lo = (float)(scale * 1.4426950408889634 - (double)q.scale_log2);
  q.q = p->q;
  q.cu_rows = p->cu_rows;
  q.ctx_len = p->ctx_len;
  q.parent = p->parent;
  q.seq_kind = p->seq_kind;
  q.slots = pl.slots;
  q.many = pl.many;
  q.part_seq = pl.part_seq;
  q.merge_seq = pl.merge_seq;
  q.min_chunk = pl.kernel == VA_KERNEL_TENSOR ? 128 : 64;
  q.rows_per_block = pl.rows_per_block;
  q.ws_acc = (float*)ws;
  q.ws_ml = ws ? (float*)((char*)ws + pl.acc_bytes) : nullptr;
  q.o = o;
  q.lse = lse;
  q.o_bf16 = dtype == VA_BF16;
  q.status = (unsigned*)status;
  return q;
}

static va_status check_outputs(const LatentPlan& pl, const void* ws, size_t ws_bytes, const void* o, const float* lse,
                               cudaStream_t cs) {
  if (!o || !lse) return VA_ERR_INVALID_ARG;
  if ((uintptr_t)o % 16) return VA_ERR_ALIGNMENT;
  if (pl.ws_bytes > 0) {
    if (!ws || ws_bytes < pl.ws_bytes) return VA_ERR_WORKSPACE_TOO_SMALL;
    if ((uintptr_t)ws % 256) return VA_ERR_ALIGNMENT;
  }
  return check_stream_device(cs);
}

static va_status launch(const LatentParams& q, const LatentPlan& pl, cudaStream_t cs) {
  cudaError_t e = pl.few                           ? launch_latent_rows(q, pl.grid, cs)
                  : pl.pair                       ? launch_latent_pair(q, pl.grid, cs)
                  : pl.kernel != VA_KERNEL_TENSOR ? launch_latent_simt(q, pl.grid, cs)
                  : q.prompt                      ? launch_latent_prompt(q, pl.grid, cs)
                                                  : launch_latent_umma(q, pl.grid, cs);
  if (e == cudaSuccess && pl.slots > 1) e = launch_latent_merge(q, cs);
  return e == cudaSuccess ? VA_OK : note_cuda(e);
}

}  // namespace va

using namespace va;

extern "C" {

size_t va_latent_workspace_size(const va_problem* p, const va_latent* kv) {
  if (check_latent(p, kv, VA_MODE_CHAIN) != VA_OK) return 0;
  return plan_latent(p, kv).ws_bytes;
}

int32_t va_latent_splits(const va_problem* p, const va_latent* kv) {
  if (check_latent(p, kv, VA_MODE_CHAIN) != VA_OK) return 0;
  return fill(p, plan_latent(p, kv), 1);
}

va_status verify_attn_latent(const va_problem* p, const va_latent* kv, int32_t mode, void* ws, size_t ws_bytes, void* o,
                             float* lse, uint32_t* status, void* stream) {
  va_status st = check_latent(p, kv, mode);
  if (st != VA_OK) return st;
  if (p->total_rows == 0) return VA_OK;
  const LatentPlan pl = plan_latent(p, kv);
  cudaStream_t cs = (cudaStream_t)stream;
  st = check_outputs(pl, ws, ws_bytes, o, lse, cs);
  if (st != VA_OK) return st;
  LatentParams q = base_params(p, mode, pl, kv->latent_dim + kv->rope_dim, kv->latent_dim, kv->dtype, ws, o, lse, status);
  q.cache = kv->cache;
  q.page_size = kv->page_size;
  q.capacity = kv->capacity;
  q.block_table = kv->block_table;
  q.max_blocks = kv->max_blocks_per_seq;
  q.num_blocks = kv->num_blocks;
  return launch(q, pl, cs);
}

size_t va_latent_prompt_workspace_size(const va_problem* p, const va_prompt* kv) {
  if (check_prompt(p, kv) != VA_OK) return 0;
  return plan_prompt(p, kv).ws_bytes;
}

int32_t va_latent_prompt_splits(const va_problem* p, const va_prompt* kv) {
  if (check_prompt(p, kv) != VA_OK) return 0;
  const LatentPlan pl = plan_prompt(p, kv);
  const int32_t c = fill(p, pl, p->num_heads);
  if (pl.kernel != VA_KERNEL_TENSOR) return c;
  const long long blocks = ((long long)p->max_rows_per_seq + pl.rows_per_block - 1) / pl.rows_per_block;
  const long long chunks = (long long)kv->total_kv / p->num_seqs / kPromptChunkKeys;
  const long long n = c < chunks * blocks ? c : chunks * blocks;
  return (int32_t)(n / blocks < 2 ? 1 : n);
}

va_status verify_attn_latent_prompt(const va_problem* p, const va_prompt* kv, void* ws, size_t ws_bytes, void* o,
                                    float* lse, uint32_t* status, void* stream) {
  va_status st = check_prompt(p, kv);
  if (st != VA_OK) return st;
  if (p->total_rows == 0) return VA_OK;
  const LatentPlan pl = plan_prompt(p, kv);
  cudaStream_t cs = (cudaStream_t)stream;
  st = check_outputs(pl, ws, ws_bytes, o, lse, cs);
  if (st != VA_OK) return st;
  LatentParams q =
      base_params(p, VA_MODE_CHAIN, pl, kv->nope_dim + kv->rope_dim, kv->value_dim, kv->dtype, ws, o, lse, status);
  q.kv = kv->kv;
  q.k_rope = kv->k_rope;
  q.kr_stride = kv->k_rope_stride;
  q.cu_kv = kv->cu_kv;
  q.total_kv = kv->total_kv;
  q.causal = kv->causal;
  q.prompt = 1;
  return launch(q, pl, cs);
}

}  // extern "C"
