// What the attention kernels over latent caches (absorbed form) and expanded
// prompt keys share: launch parameters, the work of a CTA, visibility.
//
// Absorbed form: a sequence's n rows x H heads are one run of query rows (row
// j, head h at j H + h) over the one cache row that a token has.  Prompts:
// a head's n rows, over that head's keys; blockIdx.y is the head.  Either
// way a block of the grid is one block of query rows and one chunk of the
// sequence's tokens; blockIdx.z is the sequence (tensor-core prompts: in x).
#pragma once

#include "va_common.cuh"
#include "va_host.h"

namespace va {

constexpr int kLatentRope = 64;

struct LatentParams {
  int num_seqs, H, total_rows, max_rows, mode;
  int DK, DV;             // width of a key (rope part among it) and of a value
  float scale_log2;       // softmax scale * log2(e)
  float scale_lo;         // what its rounding left
  const void* q;          // [total_rows][H][DK]
  const int* cu_rows;
  const int* ctx_len;
  const int* parent;
  const unsigned char* seq_kind;
  // absorbed form: the cache
  const void* cache;
  int page_size;
  long long capacity;
  const int* block_table;
  int max_blocks, num_blocks;
  // prompts: expanded keys and values
  const void* kv;
  const void* k_rope;
  long long kr_stride;
  const int* cu_kv;
  int total_kv, causal;
  int prompt;
  int slots;              // largest number of chunks of a sequence
  int min_chunk;          // tokens
  int many;               // a sequence of max_rows rows may have many
  int rows_per_block;
  int part_seq;           // partials of a sequence and slot; 0: one for every row and head of the launch
  int merge_seq;          // (row, head) pairs of a sequence that may have more than one chunk; 0: any of the launch
  float* ws_acc;          // [partials][DV], see latent_part
  float* ws_ml;           // [partials][2]  (m in log2 units, l)
  void* o;                // [total_rows][H][DV]
  float* lse;             // [total_rows][H]
  int o_bf16;
  unsigned* status;
};

// A sequence: its rows, the tokens before them (negative where a prompt has
// more rows than keys), its tokens in all, and the first of its keys.
struct LatentSeq {
  int row0, n, ctx, len, kind;
  long long key0;
  unsigned err;
};

__device__ __forceinline__ int latent_kind(const LatentParams& p, int s) {
  if (p.prompt || p.mode == VA_MODE_CHAIN) return 0;
  if (p.mode == VA_MODE_TREE) return 1;
  return p.seq_kind[s] ? 1 : 0;
}

__device__ __forceinline__ LatentSeq latent_seq(const LatentParams& p, int s) {
  LatentSeq q;
  const int r0 = p.cu_rows[s], r1 = p.cu_rows[s + 1];
  q.row0 = r0;
  q.n = r1 - r0;
  q.kind = latent_kind(p, s);
  q.err = 0u;
  q.key0 = 0;
  if (r0 < 0 || r1 < r0 || r1 > p.total_rows || r1 - r0 > p.max_rows) q.err = VA_DEV_BAD_ROWS;
  if (p.prompt) {
    const int k0 = p.cu_kv[s], k1 = p.cu_kv[s + 1];
    q.key0 = k0;
    if (k0 < 0 || k1 < k0 || k1 > p.total_kv) q.err = VA_DEV_BAD_ROWS;
    q.len = k1 - k0;
    q.ctx = q.len - q.n;
  } else {
    const int c = p.ctx_len[s];
    q.ctx = c;
    q.len = c + q.n;
    if (!q.err && q.kind == 1 && q.n > kMaxTreeRows) q.err = VA_DEV_BAD_ROWS;
    const long long room = p.page_size ? (long long)p.max_blocks * kPage : p.capacity;
    if (!q.err && (c < 0 || (long long)c + q.n > room)) q.err = VA_DEV_CTX_OVERFLOW;
  }
  return q;
}

// Query rows of a sequence per key head, and its chunks: the launch's count
// shared out among its row blocks, by the sequence alone.
__device__ __forceinline__ int latent_rows(const LatentParams& p, int n) { return p.prompt ? n : n * p.H; }

__device__ __forceinline__ int latent_chunks(const LatentParams& p, int n) {
  const int b = (latent_rows(p, n) + p.rows_per_block - 1) / p.rows_per_block;
  return max(1, p.slots / max(b, 1));
}

// Chunk c of nchunk of [0, len).
__device__ __forceinline__ void latent_range(const LatentParams& p, int len, int nchunk, int c, int* lo, int* hi) {
  sub_range(0, len, nchunk, p.min_chunk, c, lo, hi);
}

// Chunks that hold tokens (they come first); 1 for a sequence of none.
__device__ __forceinline__ int latent_live(const LatentParams& p, int len, int nchunk) {
  return max(1, live_subs(0, len, nchunk, p.min_chunk));
}

// Index among [total_rows][H] of query row r of a sequence (prompts: of head).
__device__ __forceinline__ long long latent_item(const LatentParams& p, int row0, int r, int head) {
  return p.prompt ? (long long)(row0 + r) * p.H + head : (long long)row0 * p.H + r;
}

// Row (of the cache's rows) of token t of sequence s; -1 for a bad block.
__device__ __forceinline__ long long latent_row(const LatentParams& p, int s, int t) {
  if (p.page_size == 0) return (long long)s * p.capacity + t;
  const int blk = p.block_table[(long long)s * p.max_blocks + t / kPage];
  if (blk < 0 || blk >= p.num_blocks) return -1;
  return (long long)blk * kPage + t % kPage;
}

// One past the last token that rows up to j of a sequence see.
__device__ __forceinline__ int latent_end(const LatentParams& p, const LatentSeq& q, int j) {
  if (q.kind == 1 || (p.prompt && !p.causal)) return q.len;
  return min(q.len, q.ctx + j + 1);
}

// Which of the tokens t0 .. t0 + 31 query row j sees, of those below hi.
__device__ __forceinline__ unsigned latent_bits(const LatentParams& p, const LatentSeq& q, unsigned anc, int j,
                                                int hi, int t0) {
  if (p.prompt && !p.causal) return bit_range(0, hi - t0);
  if (q.kind == 0) return bit_range(0, min(hi, q.ctx + j + 1) - t0);
  return visible_bits(1, anc, j, q.ctx, hi, t0);
}

// NaN in o and lse of a sequence with inconsistent offsets (the rows of it
// that exist), by thread t of so many.  heads: first head and how many.
__device__ __forceinline__ void latent_nan_rows(const LatentParams& p, int s, int h0, int heads, int t, int threads) {
  const long long a = max(0, p.cu_rows[s]), b = min(p.total_rows, p.cu_rows[s + 1]);
  for (long long i = t; i < (b - a) * heads * p.DV; i += threads) {
    const long long item = (a + i / ((long long)heads * p.DV)) * p.H + h0 + i / p.DV % heads;
    const int d = (int)(i % p.DV);
    if (p.o_bf16) reinterpret_cast<unsigned short*>(p.o)[item * p.DV + d] = 0x7fffu;
    else reinterpret_cast<float*>(p.o)[item * p.DV + d] = NAN;
    if (d == 0) p.lse[item] = NAN;
  }
}

// Where the partials of chunk c of a sequence stand: that of (row, head) item at
// latent_part + item.  A sequence of more than one row block has no more than slots /
// blocks chunks, and so no more partials than slots for each row of one block: the
// workspace is sized by that where it is less than slots for every row of the launch
// (one sequence of 1,024 rows, 128 heads, 512 columns, 76 slots: 20 MB, not 20 GB).
__device__ __forceinline__ long long latent_part(const LatentParams& p, int s, int row0, int n, int c) {
  if (p.part_seq == 0) return (long long)c * p.total_rows * p.H;
  return (long long)s * p.part_seq * p.slots + ((long long)c * n - row0) * p.H;
}
// From one chunk's to the next one's.
__device__ __forceinline__ long long latent_apart(const LatentParams& p, int n) {
  return (long long)(p.part_seq == 0 ? p.total_rows : n) * p.H;
}

cudaError_t launch_latent_simt(const LatentParams& p, dim3 grid, cudaStream_t st);
cudaError_t launch_latent_merge(const LatentParams& p, cudaStream_t st);
int latent_simt_rows();
cudaError_t launch_latent_umma(const LatentParams& p, dim3 grid, cudaStream_t st);
int latent_umma_rows();
cudaError_t launch_latent_prompt(const LatentParams& p, dim3 grid, cudaStream_t st);
int latent_prompt_rows();
cudaError_t launch_latent_pair(const LatentParams& p, dim3 grid, cudaStream_t st);
int latent_pair_rows();
cudaError_t launch_latent_rows(const LatentParams& p, dim3 grid, cudaStream_t st);
int latent_rows_rows(long long rows);

}  // namespace va
