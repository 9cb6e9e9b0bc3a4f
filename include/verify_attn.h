/*
 * verify_attn.h — C ABI of the GB300 speculative-decoding verify-attention
 * library (libverify_attn.so, sm_103a).
 *
 * The operation: a window of draft-token query rows per sequence attends over
 * that sequence's KV cache.  Rows are causal along a chain, or follow a
 * parent array for a fixed-width tree suffix; query heads are grouped over
 * fewer KV heads; the cache is contiguous or paged in 16-token blocks and
 * holds fp32, bf16 or Q8_0 rows.  The result per (row, head) is the softmax-
 * weighted sum of the visible V rows (O) and the natural-log sum of the
 * exponentiated scaled scores (LSE).
 *
 * Sources (the pages this library restates):
 *   - hipfire PR #695 "perf(gfx11): optimize Qwen DFlash speculative verify":
 *     section "Summary" (B=16 verify through batched flash attention), the
 *     alpineQ comments (Q8 KV, one block reusing each KV fetch across several
 *     verifier rows, the batched-partials layout and its reducer).
 *   - hipfire PR #817 "speed up long-context DFlash verify 13.4% with FA2
 *     split-KV": sections "Summary", "Default and admission policy" and
 *     "Performance" (S8 split-KV partial + merge, caller-owned partial
 *     workspace, fail-closed admission, S1 equal to the unsplit result).
 *   - lucebox PR #686 "perf(qwen35): retain speculation during paged
 *     prefill": sections "Mechanism", "State and commit invariants" and
 *     "Correctness failure found during qualification" (direct rows and a
 *     fixed-width tree suffix in one step over paged KV; tree ancestry
 *     metadata; partitioning must not depend on what shares the launch).
 *
 * Conventions for every entry point:
 *   - Pointers named "device" are CUDA device memory owned by the caller;
 *     the library never allocates, frees or keeps them past the call.
 *   - Calls are asynchronous on the given CUDA stream (a cudaStream_t passed
 *     as void*; NULL = legacy default stream).  Lengths and metadata are read
 *     on the device, so the host never synchronises.
 *   - The stream must belong to the current device (the plan uses that
 *     device's SM count); outside stream capture, a stream of another
 *     device returns VA_ERR_INVALID_ARG and launches nothing (a capturing
 *     stream's device cannot be queried without ending the capture, so
 *     there the caller's word stands).
 *   - Host-checkable errors return a status and launch nothing.
 *   - Data errors found on the device (bad parent, block id, row counts,
 *     context beyond capacity) OR a VA_DEV_* bit into *status (device word,
 *     may be NULL) and the affected rows get NaN outputs (for inconsistent
 *     row offsets, VA_DEV_BAD_ROWS, every row of that sequence).
 */
#ifndef VERIFY_ATTN_H
#define VERIFY_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum va_status {
  VA_OK = 0,
  VA_ERR_INVALID_ARG = 1,         /* null pointer, negative size, bad enum */
  VA_ERR_UNSUPPORTED = 2,         /* shape/dtype outside the supported set */
  VA_ERR_ALIGNMENT = 3,           /* a pointer is not 16-byte aligned */
  VA_ERR_WORKSPACE_TOO_SMALL = 4, /* ws_bytes < va_workspace_size() */
  VA_ERR_CUDA = 5                 /* a CUDA runtime call or launch failed */
} va_status;

typedef enum va_dtype {
  VA_F32 = 0,  /* IEEE fp32 */
  VA_BF16 = 1, /* bfloat16 */
  VA_Q8_0 = 2  /* 34-byte blocks: fp16 scale d (little endian), 32 int8 codes q; value d*q */
} va_dtype;

typedef enum va_mode {
  VA_MODE_CHAIN = 0, /* every sequence is a chain: row j sees context + rows 0..j */
  VA_MODE_TREE = 1,  /* every sequence is a tree over its rows (parent array) */
  VA_MODE_MIXED = 2  /* per-sequence kind from seq_kind[] */
} va_mode;

/* Device status bits (OR-ed into *status). */
#define VA_DEV_BAD_PARENT 0x1u   /* parent[j] not in [-1, j) */
#define VA_DEV_BAD_BLOCK 0x2u    /* block_table entry outside [0, num_blocks) */
#define VA_DEV_CTX_OVERFLOW 0x4u /* ctx + n exceeds capacity / the block table */
#define VA_DEV_BAD_ROWS 0x8u     /* cu_rows not ascending, n > max_rows_per_seq, total mismatch,
                                    or a tree sequence with more than VA_MAX_TREE_ROWS rows */
#define VA_DEV_TIMEOUT 0x10u     /* a bounded pipeline wait gave up */
#define VA_DEV_BAD_SAMPLING 0x20u /* a temperature that is neither 0 nor in [1e-6, inf) */
#define VA_DEV_BAD_TOKEN 0x40u   /* a drafted token outside [0, vocab) */
#define VA_DEV_BAD_LOGITS 0x80u  /* NaN, +inf or nothing but -inf in the row the next token is drawn from */
#define VA_DEV_NO_PAGES 0x100u   /* fewer free pages than a fork needs */
#define VA_DEV_BAD_COPY 0x200u   /* a page pair outside the pool, or more pairs than the list holds */

/* Problem flags. */
#define VA_FLAG_CUDA_CORES 0x1u /* run the CUDA-core (SIMT) partial kernel for any dtype */

/*
 * The KV cache.
 *   contiguous (page_size == 0): k, v are [num_seqs][num_kv_heads][capacity][row];
 *     capacity is a multiple of 16 tokens.
 *   paged (page_size == 16): k, v are pools [num_blocks][num_kv_heads][16][row]
 *     and token t of sequence s lives in block block_table[s*max_blocks_per_seq + t/16],
 *     slot t%16 (lucebox PR #686, "Correctness failure found during
 *     qualification": 16-token blocks).
 *   row = head_dim fp32 / bf16 elements, or head_dim/32 Q8_0 blocks of 34 bytes.
 *   The draft rows' own K/V sit at positions ctx .. ctx+n-1 of the same cache,
 *   except for tree sequences when a tree scratch KV is given (draft_k,
 *   draft_v: device [total_rows][num_kv_heads][row], row r of the launch in
 *   the cache's row format, 16-byte aligned).  Then a tree sequence's draft
 *   position a reads scratch row cu_rows[s] + a, and its cache needs room
 *   for the context only (capacity, or block-table entries, for ctx_len[s]
 *   tokens).  Chain and direct sequences always read the cache: prefill and
 *   direct rows write durable KV, tree rows write scratch KV (lucebox PR
 *   #686, "State and commit invariants").  With a scratch KV, Q8_0 caches
 *   (contiguous or paged) run on the transposed tensor-core kernel and other
 *   caches on the CUDA-core kernel.
 */
typedef struct va_kv {
  va_dtype dtype;
  int32_t num_kv_heads;
  int32_t head_dim;            /* 64, 128 or 256 */
  const void *k;               /* device, 16-byte aligned */
  const void *v;               /* device, 16-byte aligned */
  int32_t page_size;           /* 0 or 16 */
  int64_t capacity;            /* contiguous only: tokens per (sequence, KV head) */
  const int32_t *block_table;  /* paged only: device [num_seqs][max_blocks_per_seq] */
  int32_t max_blocks_per_seq;  /* paged only */
  int32_t num_blocks;          /* paged only: blocks in the pool */
  const void *draft_k;         /* optional tree scratch KV (see above), or NULL */
  const void *draft_v;         /* set together with draft_k */
} va_kv;

/*
 * The query side.
 *   q: device [total_rows][num_heads][head_dim], fp32 or bf16 (bf16 for the
 *      bf16 and Q8_0 caches; fp32 or bf16 for the fp32 cache).
 *   Rows of sequence s are cu_rows[s] .. cu_rows[s+1]-1 (device array); row
 *   j of a sequence sits at KV position ctx_len[s] + j.
 *   parent: device [total_rows], the local index of each row's parent in its
 *      own sequence, -1 for a node attached to the context; must satisfy
 *      parent[j] < j.  Ignored for chain sequences (may be NULL in chain mode).
 *   seq_kind: device [num_seqs], 0 = chain (a 1-row chain is a direct/AR
 *      row), 1 = tree; read in VA_MODE_MIXED only.
 *   Query head h reads KV head h / (num_heads / num_kv_heads).
 *   scale: softmax scale; 0 selects 1/sqrt(head_dim).
 *   num_splits: S >= 1.  Sequence s's span L = ctx + n is cut into chunks
 *      of max(ceil(L/Ts), 128) tokens rounded up to a whole number of
 *      64-token tiles (at most Ts chunks).  T (>= S, <= 16 S) is fixed by S,
 *      num_kv_heads and the GPU's SM count only (one wave of CTAs per
 *      sequence and KV head); a sequence whose n * G query rows span b > 1
 *      row blocks of the partial kernel (128 rows on the tensor-core
 *      kernels, 16 on the CUDA-core kernel), each of which reads the span
 *      again, uses Ts = max(S, floor(T / b)) chunks (T otherwise); each
 *      chunk writes an fp32 online-softmax
 *      partial and a merge pass combines them in ascending order (hipfire
 *      PR #817, "Summary" and "Performance").  No choice depends on the
 *      other sequences of the launch, so a row's result depends only on
 *      its own sequence (lucebox PR #686, "Correctness failure found during
 *      qualification").
 */
/* Rows per sequence: a chain sequence (a prefill segment, a draft chain or
 * a one-row direct row; causal among its own rows) may hold up to
 * VA_MAX_ROWS_PER_SEQ rows, a tree suffix up to VA_MAX_TREE_ROWS (its
 * visibility is a 32-bit ancestor mask).  Rows beyond 128 / G per KV head
 * run as further row blocks, each reading that sequence's K/V again. */
#define VA_MAX_ROWS_PER_SEQ 1024
#define VA_MAX_TREE_ROWS 32

typedef struct va_problem {
  int32_t num_seqs;
  int32_t num_heads;
  va_dtype q_dtype;
  const void *q;
  const int32_t *cu_rows;
  const int32_t *ctx_len;
  const int32_t *parent;
  const uint8_t *seq_kind;
  int32_t total_rows;          /* host copy of cu_rows[num_seqs] */
  int32_t max_rows_per_seq;    /* host bound on rows per sequence, 1..VA_MAX_ROWS_PER_SEQ
                                  (VA_MODE_TREE: 1..VA_MAX_TREE_ROWS) */
  float scale;
  int32_t num_splits;
  uint32_t flags;              /* VA_FLAG_* */
} va_problem;

/* Library version (major*10000 + minor*100 + patch). */
int32_t va_version(void);

/*
 * Tree commit of the KV cache (the KV part of lucebox PR #686's tree commit
 * transaction, "State and commit invariants": tree rows write scratch KV;
 * the commit promotes only the accepted prefix and checks every domain
 * before it mutates any).  For each sequence s, the accepted path of m_s =
 * accepted_len[s] tree nodes, accepted_nodes[cu_rows[s] + i] for i < m_s
 * (root first), goes from the tree scratch KV (kv->draft_k / draft_v, row
 * cu_rows[s] + node) to positions ctx_len[s] + i of the cache, K and V of
 * every KV head, byte for byte.  accepted_len: device [num_seqs];
 * accepted_nodes: device [total_rows] (entries past m_s ignored).
 * Device preflight before any write, for every sequence: the row checks of
 * a verify call (VA_DEV_BAD_ROWS, VA_DEV_CTX_OVERFLOW on the context);
 * 0 <= m <= n and m = 0 unless the sequence is a tree (VA_DEV_BAD_ROWS);
 * nodes in [0, n) (VA_DEV_BAD_ROWS) forming a root path: parent[first] =
 * -1, parent[next] = previous (VA_DEV_BAD_PARENT); positions up to
 * ctx + m within capacity or the block table (VA_DEV_CTX_OVERFLOW) on
 * valid blocks (VA_DEV_BAD_BLOCK).  If the status word holds any bit after
 * the preflight, nothing is written: *status must be 0 on entry.  Host
 * checks as for the verify calls; kv->draft_k, accepted_len and status are
 * required (VA_ERR_INVALID_ARG).  The scratch must not overlap the cache.
 */
va_status verify_attn_promote(const va_problem *p, const va_kv *kv, int32_t mode,
                              const int32_t *accepted_len, const int32_t *accepted_nodes,
                              uint32_t *status, void *stream);

/* Human-readable name of a status code; never NULL. */
const char *va_status_string(va_status s);

/* Text of the CUDA error behind this thread's last VA_ERR_CUDA; never NULL. */
const char *va_last_cuda_error(void);

/*
 * Bytes of device workspace a verify call needs for this problem: the fp32
 * split partials (m, l and the unnormalised accumulator per split, row and
 * head; hipfire PR #817 "Default and admission policy": the caller-owned
 * partial workspace).  Returns 0 for an invalid problem.
 */
size_t va_workspace_size(const va_problem *p, const va_kv *kv);

/*
 * Host-only validation, no launch and no device access: the checks every
 * verify call makes before launching (fail-closed admission as in hipfire
 * PR #817 "Default and admission policy"; undersized workspace rejected).
 */
va_status va_validate(const va_problem *p, const va_kv *kv, int32_t mode, size_t ws_bytes);

/*
 * Verify attention.  o: device fp32 [total_rows][num_heads][head_dim];
 * lse: device fp32 [total_rows][num_heads] (natural log).  ws: device
 * workspace of at least va_workspace_size() bytes, 256-byte aligned;
 * its contents need no initialisation and are overwritten.
 *   verify_attn_chain: every sequence is a chain (also 1-row direct rows).
 *   verify_attn_tree:  every sequence is a tree over its rows (parent required).
 *   verify_attn_mixed: per-sequence chain or tree from seq_kind (lucebox PR
 *                      #686 "Mechanism": direct rows and tree rows in one step).
 */
va_status verify_attn_chain(const va_problem *p, const va_kv *kv, void *ws, size_t ws_bytes,
                            float *o, float *lse, uint32_t *status, void *stream);
va_status verify_attn_tree(const va_problem *p, const va_kv *kv, void *ws, size_t ws_bytes,
                           float *o, float *lse, uint32_t *status, void *stream);
va_status verify_attn_mixed(const va_problem *p, const va_kv *kv, void *ws, size_t ws_bytes,
                            float *o, float *lse, uint32_t *status, void *stream);

/*
 * Debug export of the row map and masks the kernels use: row_seq[r] is the
 * sequence of global row r; anc_mask[r] has bit a set iff draft position a
 * of that sequence is visible to row r (itself or an ancestor).  Device
 * outputs of total_rows entries each.  The mask has 32 bits: a chain row
 * j >= 31 gets every bit (the kernels decide chain visibility from j).  (lucebox PR #686 "Correctness failure
 * found during qualification": the compact row map and W8 topology checks.)
 */
va_status va_debug_row_map(const va_problem *p, int32_t mode, int32_t *row_seq,
                           uint32_t *anc_mask, uint32_t *status, void *stream);

/*
 * Debug export of the KV gather the kernels use: phys_row[s*max_len + t] is
 * the row of token t of sequence s, KV head kv_head, counted in rows of the
 * k/v array (contiguous: (s*KVH+kvh)*capacity + t; paged:
 * (block*KVH+kvh)*16 + t%16), or -1 for t >= ctx+n.  Device output of
 * num_seqs*max_len int64.
 */
va_status va_debug_gather_index(const va_problem *p, const va_kv *kv, int32_t kv_head,
                                int64_t max_len, int64_t *phys_row, uint32_t *status,
                                void *stream);

/*
 * Debug export of the KV chunks the partial kernels run (the split plan of
 * hipfire PR #817 "Summary": each sequence's span cut into chunks whose
 * partials a merge combines; lucebox PR #686 "Correctness failure found
 * during qualification": the cut must not depend on what else shares the
 * launch).  For sequence s and slot j < T (T = va_plan's slots),
 * ranges[2*(s*T + j)] and ranges[2*(s*T + j) + 1] are the first and
 * one-past-last KV position of chunk j, computed by the device functions
 * the partial kernels call: with L = ctx_len[s] + rows of s and Ts the
 * sequence's chunk count (see num_splits), a chunk has c = max(ceil(L / Ts),
 * 128) rounded up to a multiple of 64 tokens and chunk j is [min(j c, L),
 * min((j + 1) c, L)) (empty past L; slots Ts .. T - 1 are empty).  A sequence
 * whose row offsets are inconsistent gets -1, -1 and sets
 * VA_DEV_BAD_ROWS.  ranges: device int32[num_seqs * T * 2].
 */
va_status va_debug_split_ranges(const va_problem *p, const va_kv *kv, int32_t mode,
                                int32_t *ranges, uint32_t *status, void *stream);

/* Plan details for a problem (which kernel runs, splits and sub-splits). */
/* Partial kernels (va_plan_info.kernel). */
#define VA_KERNEL_CUDA_CORES 0 /* fp32 FMA, one thread block per 16 query rows */
#define VA_KERNEL_TENSOR 1     /* tcgen05, query rows on the MMA's M axis (bf16 caches) */
#define VA_KERNEL_TENSOR_Q8 2  /* tcgen05, tokens on M and query rows on N (Q8_0 caches) */

typedef struct va_plan_info {
  int32_t kernel;          /* VA_KERNEL_* */
  int32_t sub_splits;      /* T: KV chunks per sequence of one row block (equal to slots) */
  int32_t slots;           /* T partial slots per (row, head) */
  int32_t grid_x, grid_y, grid_z; /* x: max(T, S * row blocks of the longest sequence);
                                     y: KV heads; z: sequences */
  int32_t threads;
  int32_t smem_bytes;
} va_plan_info;

va_status va_plan(const va_problem *p, const va_kv *kv, int32_t mode, va_plan_info *out);

/*
 * Optional per-kernel timing for benchmarks.  While enabled (on != 0),
 * every verify_attn_chain, _tree and _mixed call records CUDA events on its
 * stream before the partial kernel, between the partial and merge kernels, and
 * after the merge;
 * enabling restarts at slot 0 (at most 4096 calls are kept).  Inside a
 * stream capture the records become event nodes of the graph, so a replay
 * refreshes them.  va_timing_read waits for the recorded events and writes
 * each recorded call's partial and merge durations in milliseconds
 * (host arrays of max_calls floats, either may be NULL).  Not thread-safe.
 */
va_status va_timing_enable(int32_t on);
va_status va_timing_read(int32_t max_calls, float *partial_ms, float *merge_ms,
                         int32_t *num_calls);

/*
 * Verify attention without a caller workspace and without any allocation
 * on the call path.  The pages have no counterpart to this entry point;
 * verify_attn_chain/tree/mixed, which take a caller workspace, are the
 * pages' route.
 *
 * For callers that cannot hand the library device memory per call: code
 * that owns no allocator (a plain C host program, a runtime whose device
 * memory budget is fixed up front), or a serving loop that must not call
 * into an allocator between steps.  The split partials go to scratch that
 * belongs to the library: a fixed array of VA_STATIC_WORKSPACE_BYTES in the
 * library's device image, reserved by the CUDA runtime when the library's
 * module is loaded on a device (one array per device).
 *
 * mode: VA_MODE_CHAIN, VA_MODE_TREE or VA_MODE_MIXED (same meaning as the
 * three entry points above).  p, kv, o, lse, status, stream: as for
 * verify_attn_chain.  Nothing needs initialising: the scratch holds no
 * state between calls and need not start at zero.
 *
 * Limits and errors:
 *   - Problems whose va_workspace_size() exceeds VA_STATIC_WORKSPACE_BYTES
 *     (16 MiB: e.g. 38 slots x 16 rows x 24 heads at D=256 fit,
 *     38 slots x 50 rows x 24 heads do not) return
 *     VA_ERR_WORKSPACE_TOO_SMALL before any launch; use the entry points
 *     with a caller workspace for those.
 *   - The scratch used is the current device's, and the stream must belong
 *     to that device (VA_ERR_INVALID_ARG otherwise, nothing launched).
 *   - The first call on each device looks the scratch address up with
 *     cudaGetSymbolAddress (VA_ERR_CUDA if that fails); make that first
 *     call, on every device it will be used on, outside any stream capture.
 *   - The scratch is shared by every call on a device: calls on one stream
 *     are ordered and safe, calls that can overlap in time (different
 *     streams without ordering between them, several host threads) race on
 *     it and must not be issued.
 */
#define VA_STATIC_WORKSPACE_BYTES (16u * 1024u * 1024u)

va_status verify_attn_noalloc(const va_problem *p, const va_kv *kv, int32_t mode, float *o,
                              float *lse, uint32_t *status, void *stream);

/*
 * Windowed verify attention: every row sees a sliding window and the first
 * few tokens of its sequence (attention sinks).
 *
 * A row at position P (a chain row j: ctx + j; a tree row: ctx + its depth,
 * 0 for a root) sees, of the tokens that verify_attn_chain / tree / mixed
 * would show it, those at positions > P - window and those at positions <
 * sinks.  A context token t stands at t, a drafted row at its own P.  With
 * window > ctx + rows the result is that of the unwindowed call.
 *   - K/V of tokens that no row of the sequence sees are not read, and their
 *     pages need not exist: block-table entries of pages that hold no
 *     visible token may be anything (pages behind the window can be given
 *     back, verify_attn_pages_free).  A page that holds visible tokens and
 *     others may hold anything in the others.
 *   - K/V that some rows see and others do not must be finite (a masked
 *     score weighs 0, and 0 times infinity is NaN).
 *   - num_splits is here the largest number of chunks that a sequence's
 *     visible tokens are cut into (whole 64-token tiles, at least 128
 *     tokens).  About c SMs / (num_seqs * num_kv_heads) chunks fill the GPU
 *     once (va_window_splits): c CTAs run on an SM, 2 where a KV head has at
 *     most 16 query rows and else 1.  Where a KV head's query rows make b > 1
 *     blocks of its kernel (of 128 rows; of 16 on the CUDA cores: fp32 caches,
 *     bf16 ones with a scratch KV, VA_FLAG_CUDA_CORES), each block takes
 *     num_splits / b chunks, rounded down, and at least m: m is 1, or on the
 *     CUDA cores a chunk per 256 tokens of window and sinks, at most
 *     num_splits (their calls with many rows may so make up to b num_splits
 *     CTAs per sequence and KV head, and num_splits partials of each row).
 *     On the 128-row kernel o_dtype VA_F32 raises num_splits and m to a
 *     chunk per 2,048 tokens, to at most 256 chunks: over more tokens the
 *     tensor cores' running sums drift visibly.  No choice depends on the other
 *     sequences of the launch: kernel and chunks follow from the types, from
 *     num_splits and max_rows_per_seq as given, and from the sequence itself.
 *   - How exactly O is summed follows from the cache and the kernel; lse is
 *     summed in fp32 by all.  On the CUDA cores: fp32 products and sums.  bf16
 *     caches: probabilities enter the products in 16 bits (2.5e-6 of O), or, for
 *     o_dtype VA_F32 and up to 16 query rows per KV head (48 at head_dim 64, 32
 *     at 128), in 24.  Q8_0 caches, as in the unwindowed calls and whatever
 *     o_dtype is: K exactly, probabilities and V elements rounded to fp16 (2^-11
 *     each), about 3e-4 of O.  fp32 sums of Q8_0 values are had with
 *     VA_FLAG_CUDA_CORES.
 *   - Rows that no sequence covers stay as they were.  Where row offsets
 *     overlap (VA_DEV_BAD_ROWS), a row claimed twice holds either result.
 *   - o: [total_rows][num_heads][head_dim] of o_dtype (VA_F32, or VA_BF16:
 *     rounded once, at the end); lse fp32.  ws of at least
 *     va_window_workspace_size() bytes, 256-byte aligned; its contents carry
 *     nothing from call to call.  Two calls that may overlap in time need
 *     two workspaces.
 * Everything else (types, layouts, tree scratch KV, errors, streams, graph
 * capture) as for verify_attn_chain / tree / mixed.
 */
typedef struct va_window {
  int32_t window;  /* >= 1: positions a row sees up to and including its own */
  int32_t sinks;   /* >= 0: first positions that stay visible */
  int32_t o_dtype; /* VA_F32 or VA_BF16 */
} va_window;

/* Bytes of device workspace; 0 for an invalid problem. */
size_t va_window_workspace_size(const va_problem *p, const va_kv *kv, const va_window *w);

/* A chunk count (num_splits) that fills the current device once with this
 * problem's sequences, at least 256 visible tokens to a chunk; 0 for an
 * invalid problem. */
int32_t va_window_splits(const va_problem *p, const va_kv *kv, const va_window *w);

va_status verify_attn_window(const va_problem *p, const va_kv *kv, int32_t mode, const va_window *w,
                             void *ws, size_t ws_bytes, void *o, float *lse, uint32_t *status,
                             void *stream);

/*
 * Acceptance of drafted tokens from given random numbers, and the token
 * that follows them: the step between a verify call (whose rows the target's
 * logits come from) and verify_attn_promote.
 *
 * Of va_problem, num_seqs, cu_rows, parent, seq_kind, total_rows and
 * max_rows_per_seq are read (kinds and row limits as for verify calls).  Row
 * 0 of a sequence is the token that is already known (a tree has one root:
 * parent[0] = -1, parent[j] in [0, j)); row j > 0 proposes tokens[row] for
 * the place after its parent.  Let p be softmax(logits[a] / temperature) at
 * the node a reached so far, starting from row 0.  The children of a are
 * tried in row order; one with token x is taken iff
 *     accept_u[row] * g(x) < r(x),
 * with r = p for the first child.  A child that is not taken leaves
 * r <- max(r - g, 0), renormalised.  g is draft_probs[a], the distribution
 * that the children of a were drawn from, or the indicator of x where
 * draft_probs is NULL (proposals that were not drawn; r then only loses x).
 * At the node where no child is taken, the next token is the lowest i with
 * r_0 + .. + r_i > sample_u[s] (r_0 + r_1 + ..).  Should r be zero
 * everywhere, p takes its place.  Temperature 0: a child is taken iff its
 * token is the lowest index of the row's maximum, and so is the next token;
 * no random number is used.
 *   accepted_len[s]: rows on the path taken, row 0 among them (>= 1);
 *   accepted_nodes[cu_rows[s] + i]: local index of its i-th row for i <
 *     accepted_len[s], -1 for the sequence's other rows;
 *   promote_len[s] (may be NULL): accepted_len[s] for a tree, 0 for a chain,
 *     as verify_attn_promote takes it;
 *   next_token[s].
 * The first child of a node, and without draft_probs every child, is tested
 * in fp32: p(x) to about 1e-5 of itself, and the mass that the rejected
 * siblings took is a sum of such numbers, so that what they left is known to
 * about 1e-7 of p's mass.  Later children with draft_probs, and the draw,
 * use fixed-point weights, which resolve 2^-40 of the row's largest p: the
 * draw's borders are off by about 1e-10 over the share of p's mass that the
 * rejections left.  A probability below that, or (in fp32) below 2^-126, may
 * count as 0, so that no number takes its child.
 * Outputs of rows that no sequence covers stay as they were.  A sequence of
 * no rows gets accepted_len 0 and next_token -1.
 * Masked vocabulary entries are -inf.  A row whose logits hold NaN, +inf or
 * nothing but -inf has no distribution: none of its children is taken, and
 * if the path ends there next_token is -1 (VA_DEV_BAD_LOGITS).  A sequence
 * with a bad row range, parent, drafted token or temperature gets
 * accepted_len 0, accepted_nodes and next_token -1 and the status bit
 * (VA_DEV_BAD_ROWS: its accepted_nodes stay as they were).  accept_u and
 * sample_u are in [0, 1), draft_probs in [0, 1].
 * The result does not depend on what else shares the launch, nor on the
 * order of any sum of the last row (its weights are summed as integers).
 */
typedef struct va_draft {
  int32_t vocab;              /* 1 .. 2^20 */
  va_dtype logits_dtype;      /* VA_F32 or VA_BF16 */
  const void *logits;         /* device [total_rows][logits_stride], element-aligned */
  int64_t logits_stride;      /* elements from row to row, >= vocab */
  const float *draft_probs;   /* device [total_rows][draft_stride] by parent row, or NULL */
  int64_t draft_stride;
  const int32_t *tokens;      /* device [total_rows]; row 0 of a sequence is not read */
  const float *accept_u;      /* device [total_rows] */
  const float *sample_u;      /* device [num_seqs] */
  const float *temperature;   /* device [num_seqs]: 0 or >= 1e-6; NULL: 1 */
} va_draft;

/* Bytes of device workspace (256-byte aligned; may be 0, ws may then be
 * NULL).  Contents carry nothing from call to call. */
size_t verify_attn_accept_workspace_size(const va_problem *p, const va_draft *d);

va_status verify_attn_accept(const va_problem *p, const va_draft *d, int32_t mode, void *ws,
                             size_t ws_bytes, int32_t *accepted_len, int32_t *accepted_nodes,
                             int32_t *promote_len, int32_t *next_token, uint32_t *status,
                             void *stream);

/*
 * Pages of a paged cache.  block_table is the table that verify calls read
 * (va_kv.block_table), here written; an entry of -1 holds no page.
 * ref_count[b] is the number of table entries that hold page b; a page is
 * free while it is 0.  Sequences may share pages; a shared page is one that
 * no sequence writes again (a full one).  An empty pool is a table of -1 and
 * counts of 0.
 * The calls run on the device in stream order, with lengths and commands in
 * device memory.  A planning call (fork, free, compact) checks everything
 * before it changes anything: a status word that is non-zero on entry, or a
 * finding of its own, leaves table and counts as they were (and num_copies
 * 0).  status may be NULL.  Two calls on one pool must not overlap in time.
 */
typedef struct va_page_pool {
  int32_t num_seqs;
  int32_t max_blocks_per_seq;
  int32_t num_blocks;
  int32_t *block_table; /* device [num_seqs][max_blocks_per_seq] */
  int32_t *ref_count;   /* device [num_blocks] */
} va_page_pool;

/* Bytes of device workspace (256-byte aligned) of a fork of num_forks
 * commands, or (num_forks = 0) of a compaction. */
size_t verify_attn_pages_workspace_size(const va_page_pool *pool, int32_t num_forks);

/*
 * Fork and grow sequences.  Command i (device arrays of num_forks):
 *   src[i] != dst[i]: the row of dst becomes a fork of the first len[i] tokens
 *     of src.  Full pages are shared; a partial last page is replaced by a
 *     fresh one and the pair (old, fresh) is written to copies; fresh pages
 *     follow up to entry pages[i], -1 beyond.  Entries of -1 below the length
 *     (pages behind a window) stay -1.  What dst's row held before is
 *     overwritten, not given back.
 *   src[i] == dst[i]: the sequence grows.  Entries from ceil(len[i] / 16) to
 *     pages[i] that hold no page get fresh ones; everything else stays.
 * Fresh pages are the free pages of lowest index, in command order and then
 * entry order.  copies: device [num_forks][2], in command order; num_copies:
 * device, the number written.  The caller then copies the pairs in every
 * pool (verify_attn_pages_copy).
 * Errors (nothing changes): a sequence out of range, named as dst twice, or a
 * src (!= dst) that is another command's dst (VA_DEV_BAD_ROWS); len or pages
 * out of range, or len > 16 pages (VA_DEV_CTX_OVERFLOW); a table entry that
 * is neither -1 nor a page in use, no page where the partial page should be,
 * a negative count (VA_DEV_BAD_BLOCK); too few free pages (VA_DEV_NO_PAGES).
 */
va_status verify_attn_pages_fork(const va_page_pool *pool, int32_t num_forks, const int32_t *src,
                                 const int32_t *dst, const int32_t *len, const int32_t *pages,
                                 int32_t *copies, int32_t *num_copies, void *ws, size_t ws_bytes,
                                 uint32_t *status, void *stream);

/*
 * Give back the table entries first[i] .. last[i] - 1 of sequence seq[i]: each
 * held page loses a reference and the entry becomes -1 (entries of -1 are
 * passed over; ranges may overlap).  With a window W and `sinks` first
 * tokens, a sequence of ctx tokens needs no entry from ceil(sinks / 16) to
 * floor((ctx - W + 1) / 16).  Errors (nothing changes): a sequence
 * (VA_DEV_BAD_ROWS) or range (VA_DEV_CTX_OVERFLOW) out of range, an entry that
 * is neither -1 nor a page in use (VA_DEV_BAD_BLOCK).  A page with fewer
 * references than entries is left at 0 and sets VA_DEV_BAD_BLOCK.
 */
va_status verify_attn_pages_free(const va_page_pool *pool, int32_t num_ranges, const int32_t *seq,
                                 const int32_t *first, const int32_t *last, uint32_t *status,
                                 void *stream);

/*
 * Pull the N pages in use together at the front of the pool: the k-th page in
 * use at or above N moves to the k-th free page below N (ascending).  Table,
 * counts and the pairs (from, to) in copies (device [num_blocks / 2][2]) are
 * written; *num_copies (device) is their number, *live_blocks (device, may be
 * NULL) is N.  No pair's target is another's source, so the pairs may be
 * copied in any order.  Errors (nothing changes): a table entry that is
 * neither -1 nor a page in use, a negative count (VA_DEV_BAD_BLOCK).
 */
va_status verify_attn_pages_compact(const va_page_pool *pool, int32_t *copies, int32_t *num_copies,
                                    int32_t *live_blocks, void *ws, size_t ws_bytes,
                                    uint32_t *status, void *stream);

/*
 * Copy pages in num_pools pools (host array of device pointers, 16-byte
 * aligned: the K and V arrays of every layer), each [num_blocks][page_bytes]:
 * for the first *num_copies (device) pairs of copies (device [max_copies][2]),
 * page copies[i][0] to page copies[i][1].  page_bytes is a multiple of 16
 * (num_kv_heads * 16 * row bytes for a cache).  No target may be another
 * pair's source or target.  Nothing is copied when *status holds a finding of
 * an earlier call other than VA_DEV_BAD_COPY; a pair outside the pool is
 * passed over and sets VA_DEV_BAD_COPY, as does *num_copies > max_copies
 * (the first max_copies pairs are copied).  With num_pools or max_copies 0
 * nothing is launched, and so no status set.
 */
va_status verify_attn_pages_copy(void *const *pools, int32_t num_pools, int64_t page_bytes,
                                 int32_t num_blocks, const int32_t *copies,
                                 const int32_t *num_copies, int32_t max_copies, uint32_t *status,
                                 void *stream);

/*
 * Block tables and slot maps of a step, from the lengths of its requests.
 *
 * Sequence s (row s of the block table) holds ctx_len[s] tokens and gets
 * rows[s] new ones (0: it sits the step out).  Its entries ceil(ctx_len / 16)
 * to ceil((ctx_len + rows) / 16) - 1 that hold no page take fresh ones, the
 * free pages of lowest index, in sequence order and then entry order; all
 * others stay.  Outputs, device:
 *   cu_rows[num_seqs + 1]: row offsets as verify calls take them; row r =
 *     cu_rows[s] + j is the j-th new row of sequence s.
 *   For each of its rows r < cu_rows[num_seqs]: row_seq[r] = s; position[r] =
 *     ctx_len[s] + j, for a tree sequence ctx_len[s] + the row's depth (0 for
 *     a root); slot[r], where the row's K/V go: block_table entry of token
 *     ctx_len[s] + j, times 16, plus (ctx_len[s] + j) % 16.
 *   Rows from there to max_rows (the padding of a captured graph of fixed
 *     size): -1 in all three.
 * mode, parent (by launch row: the caller knows the rows) and seq_kind as for
 * verify calls; a tree sequence has at most VA_MAX_TREE_ROWS rows, a chain any
 * number.  Everything is checked before anything changes, and a status word
 * that is non-zero on entry counts as a finding: table and counts then stay
 * as they were, cu_rows is 0 and the other outputs -1.  Errors: a negative
 * number of rows, more rows than max_rows, a tree of more than
 * VA_MAX_TREE_ROWS (VA_DEV_BAD_ROWS); a negative length, more tokens than the
 * table's row has entries for (VA_DEV_CTX_OVERFLOW); no page, or one that
 * other entries share, where a row goes, an entry that is neither -1 nor a
 * page in use among those, a negative count (VA_DEV_BAD_BLOCK); a parent not
 * in [-1, j) (VA_DEV_BAD_PARENT); too few free pages (VA_DEV_NO_PAGES).
 */
typedef struct va_extend {
  const int32_t *ctx_len;   /* device [num_seqs] */
  const int32_t *rows;      /* device [num_seqs] */
  const int32_t *parent;    /* device [max_rows]; VA_MODE_CHAIN: not read, may be NULL */
  const uint8_t *seq_kind;  /* device [num_seqs]; VA_MODE_MIXED only */
  int32_t max_rows;         /* entries of row_seq, position and slot */
} va_extend;

/* Bytes of device workspace (256-byte aligned). */
size_t verify_attn_pages_extend_workspace_size(const va_page_pool *pool);

va_status verify_attn_pages_extend(const va_page_pool *pool, const va_extend *x, int32_t mode,
                                   int32_t *cu_rows, int32_t *row_seq, int32_t *position,
                                   int64_t *slot, void *ws, size_t ws_bytes, uint32_t *status,
                                   void *stream);

/*
 * A latent cache: one row per token, shared by all heads, of latent_dim values
 * (c) and rope_dim rotated ones (kr).  With up-projections Wk[h] and Wv[h],
 * head h has the key [Wk[h] c; kr] and the value Wv[h] c, so a query
 * [q_nope; q_rope] scores (Wk[h]^T q_nope) . c + q_rope . kr, and the output
 * is Wv[h] applied to the weighted sum of the c.  verify_attn_latent works on
 * that absorbed form: its queries are [Wk[h]^T q_nope; q_rope], its outputs
 * are sums of c.  verify_attn_latent_prompt takes the expanded keys and values.
 *   contiguous (page_size 0): cache is [num_seqs][capacity][latent_dim +
 *     rope_dim], capacity a multiple of 16.
 *   paged (page_size 16): [num_blocks][16][latent_dim + rope_dim], block_table
 *     as in va_kv.
 */
typedef struct va_latent {
  va_dtype dtype;              /* VA_F32 or VA_BF16 */
  int32_t latent_dim;          /* 256 or 512 */
  int32_t rope_dim;            /* 64 */
  void *cache;                 /* device, 16-byte aligned */
  int32_t page_size;           /* 0 or 16 */
  int64_t capacity;            /* contiguous only */
  const int32_t *block_table;  /* paged only: device [num_seqs][max_blocks_per_seq] */
  int32_t max_blocks_per_seq;  /* paged only */
  int32_t num_blocks;          /* paged only */
} va_latent;

/*
 * Rows into a latent cache.  Row r of kv, [latent_dim + rope_dim] values as
 * the down-projection gives them, becomes the cache row slot[r]: its first
 * latent_dim values x turn into x / sqrt(mean(x^2) + norm_eps) * norm_weight
 * (or stay, norm_weight NULL), its last rope_dim are rotated by the angles of
 * position[r]: pair i (2i and 2i + 1 if interleaved, else i and i + rope_dim /
 * 2) goes from (a, b) to (a cos - b sin, a sin + b cos) with cos =
 * rope[position][i] and sin = rope[position][rope_dim / 2 + i].  With
 * num_heads > 0 the rope parts of the row's queries, q_rope, are rotated alike
 * into the last rope_dim values of each head of q, [num_rows][num_heads]
 * [latent_dim + rope_dim] (whose first latent_dim values stay); q_rope may be
 * that part of q itself.  Computed in fp32, rounded once.
 * slot[r] = -1 leaves the cache alone, position[r] = -1 skips row and queries
 * (padding, see verify_attn_pages_extend).  A slot outside [-1, num_slots)
 * (VA_DEV_BAD_BLOCK) or a position outside [-1, rope_positions)
 * (VA_DEV_CTX_OVERFLOW) sets the status bit; the row is skipped.  No two rows
 * may have the same slot.  A status word that is non-zero on entry does not
 * stop the call.  kv and q_rope must not overlap the cache.
 */
typedef struct va_latent_rows {
  int32_t num_rows;
  const void *kv;           /* device [num_rows][kv_stride], cache's dtype, element-aligned */
  int64_t kv_stride;        /* elements from row to row, >= latent_dim + rope_dim */
  const void *norm_weight;  /* device [latent_dim], cache's dtype, element-aligned, or NULL */
  float norm_eps;           /* >= 0 */
  const float *rope;        /* device [rope_positions][rope_dim], 16-byte aligned: cosines, then sines */
  int32_t rope_positions;
  int32_t interleaved;      /* 0 or 1 */
  const int32_t *position;  /* device [num_rows] */
  const int64_t *slot;      /* device [num_rows] */
  int64_t num_slots;        /* rows of the cache */
  int32_t num_heads;        /* 0 .. VA_MAX_LATENT_HEADS */
  const void *q_rope;       /* device, element-aligned; head h of row r at r q_row_stride + h q_head_stride */
  int64_t q_row_stride, q_head_stride;  /* elements, >= rope_dim (one head, one row: any) */
  void *q;                  /* device, 16-byte aligned */
} va_latent_rows;

#define VA_MAX_LATENT_HEADS 256

va_status verify_attn_latent_append(const va_latent *kv, const va_latent_rows *rows, uint32_t *status,
                                    void *stream);

/*
 * Verify attention over a latent cache, absorbed form.  p as for
 * verify_attn_chain / tree / mixed (mode), with q: [total_rows][num_heads]
 * [latent_dim + rope_dim] of the cache's dtype, num_heads <=
 * VA_MAX_LATENT_HEADS heads over the one row a token has, scale > 0 (the width
 * of the expanded keys is not known here), rows' own K at positions ctx ..
 * ctx + n - 1 of the cache.  o: [total_rows][num_heads][latent_dim] of the
 * cache's dtype, rounded once; lse: fp32 [total_rows][num_heads].
 * num_splits is the largest number of chunks (whole 64-token tiles, at least
 * 128 tokens; 64 on the CUDA cores) that a sequence is cut into; where its rows times heads make b
 * row blocks (of 128 in the tensor-core kernel, one block of up to 32 where
 * max_rows_per_seq times num_heads is no more; of 16 on the CUDA cores: fp32
 * caches, VA_FLAG_CUDA_CORES) each takes num_splits / b chunks, rounded
 * down, and at least one.  va_latent_splits gives a count that fills the
 * GPU.  No choice depends on the other sequences of the launch.  The
 * workspace holds the partials that can exist: num_splits for each row and
 * head, but no more than for one row block a sequence.
 * bf16: probabilities enter the second product rounded to bf16 (2^-8 of each at most,
 * about what rounding o costs); their sum, and lse, are of the unrounded
 * ones in fp32.  fp32: fp32 products and sums.
 * Cache rows that some rows of the sequence see and others do not must be
 * finite; others may hold anything.  A query, or a cache row that all rows
 * see, that is no number makes the rows NaN that it meets.  Scaled scores stay
 * below 2^29 in size.  Rows that no sequence covers stay as
 * they were.  At most 65,535 sequences.  Errors as for the verify calls.  ws
 * of at least va_latent_workspace_size() bytes (may be 0, ws may then be
 * NULL), 256-byte aligned; contents carry nothing from call to call, and
 * calls that may overlap in time need workspaces of their own.
 */
size_t va_latent_workspace_size(const va_problem *p, const va_latent *kv);
int32_t va_latent_splits(const va_problem *p, const va_latent *kv);
va_status verify_attn_latent(const va_problem *p, const va_latent *kv, int32_t mode, void *ws,
                             size_t ws_bytes, void *o, float *lse, uint32_t *status, void *stream);

/*
 * Attention of prompt segments over expanded keys and values.  Rows of
 * sequence s are cu_rows[s] .. of q, [total_rows][num_heads][nope_dim +
 * rope_dim]; its keys are cu_kv[s] .. cu_kv[s + 1] - 1 of kv, [total_kv]
 * [num_heads][nope_dim + value_dim] (a head's key part, then its value, as an
 * up-projection of c gives them), with the rope part k_rope[token][rope_dim]
 * shared by the heads (its rows may lie in a latent cache's: k_rope_stride).
 * causal: row j of n sees the keys up to len - n + j (its own segment's keys
 * come last); else every row sees all len keys, as for a part of the context
 * whose result is joined by lse.  A row that sees no key (len 0, or len < n)
 * gets o = 0 and lse = -inf.
 * Of p, num_seqs, num_heads (<= VA_MAX_LATENT_HEADS), q_dtype, q, cu_rows,
 * total_rows, max_rows_per_seq (any number up to 2^22), scale (0: 1 /
 * sqrt(nope_dim + rope_dim)), num_splits and flags are read.  num_splits, the
 * workspace, precision and the types of o ([total_rows][num_heads][value_dim])
 * and lse as for verify_attn_latent, with row blocks per head
 * (va_latent_prompt_splits).  Inconsistent offsets, rows beyond
 * max_rows_per_seq: VA_DEV_BAD_ROWS, NaN.  Keys that some rows of a sequence
 * see must be finite.
 */
typedef struct va_prompt {
  va_dtype dtype;         /* VA_F32 or VA_BF16 */
  int32_t nope_dim;       /* 64 or 128 */
  int32_t rope_dim;       /* 64 */
  int32_t value_dim;      /* as nope_dim */
  const void *kv;         /* device, 16-byte aligned */
  const void *k_rope;     /* device, 16-byte aligned */
  int64_t k_rope_stride;  /* elements from token to token, a multiple of 16 bytes */
  const int32_t *cu_kv;   /* device [num_seqs + 1] */
  int32_t total_kv;       /* host copy of cu_kv[num_seqs] */
  int32_t causal;         /* 0 or 1 */
} va_prompt;

size_t va_latent_prompt_workspace_size(const va_problem *p, const va_prompt *kv);
int32_t va_latent_prompt_splits(const va_problem *p, const va_prompt *kv);
va_status verify_attn_latent_prompt(const va_problem *p, const va_prompt *kv, void *ws, size_t ws_bytes,
                                    void *o, float *lse, uint32_t *status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* VERIFY_ATTN_H */
