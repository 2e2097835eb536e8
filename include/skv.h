/*
 * skv.h -- C ABI of the GB300 sparse-decode library (libskv.so).
 *
 * One decode step, for every (request b, KV head h):
 *   score   every candidate history key against the group's query      skv_score
 *   select  the exact top-k candidate positions                        skv_topk
 *   resolve the attended positions through the slot table and read
 *           their K/V rows from the GPU pool or the pinned host pool   skv_gather
 *   attend  with split-K flash decoding and a log-sum-exp merge        skv_sparse_attn
 * and all four chained on one stream                                   skv_decode_step
 *
 * Beside it: a step's new tokens, normed, rotated and appended to the pools
 * (skv_qk_norm_rope, skv_append_kv), and dense attention over a prefix that the batch
 * shares (skv_prefix_attn); the slot table kept on the GPU as requests grow and shrink
 * (skv_update_tables); and the same steps over a cache in 4 bits (skv_append_kv4,
 * skv_gather_kv4, skv_score_kv4, skv_attn_kv4, skv_decode_step_kv4).
 *
 * Conventions (every entry point):
 *  - The caller owns all memory.  Device buffers, pinned host pools and the
 *    workspace are allocated by the caller; the library allocates nothing,
 *    frees nothing and never synchronises.  Every call enqueues kernels (and,
 *    for skv_topk / skv_decode_step, one cudaMemsetAsync on the workspace) on
 *    `stream` and returns.  `stream` is a cudaStream_t passed as void*; NULL
 *    is the legacy default stream.  The device is the caller's current device.
 *  - Host rows are read by the kernels themselves through unified virtual
 *    addressing: host_k / host_v must be device-accessible pinned memory
 *    (cudaHostAlloc / cudaHostRegister).  The CPU launches no copy.
 *    (ECHO-OSDI26 wiki, core method 1: a GPU kernel reads host addresses
 *    directly; OasisKV notes, §3.3 Algorithm 1: UVA gather.)
 *  - Arguments the host can check are checked before anything is enqueued;
 *    a bad argument returns SKV_ERR_INVALID_ARGUMENT / SKV_ERR_UNSUPPORTED /
 *    SKV_ERR_WORKSPACE_TOO_SMALL and enqueues nothing.
 *  - Faults found on the device (a slot-table entry outside its pool, a
 *    selected position outside the candidate region, a wait that gave up)
 *    never trap: the kernel ORs a SKV_DEV_* bit into *dev_status, skips the
 *    offending row (a skipped key scores NaN and ranks last; a skipped
 *    attended row gets zero weight) and completes.  dev_status is a device
 *    int32 the caller zeroes and reads after the stream has drained; it may
 *    be NULL (no reporting).
 *  - All tensors are dense row-major ("C order") and 16-byte aligned (the rows of
 *    skv_tokens have a stride from token to token).
 *    Element types: SKV_DTYPE_BF16 (bf16 storage, fp32 arithmetic) or
 *    SKV_DTYPE_F32 (fp32 storage and arithmetic) for q, keys, pools and out;
 *    scores and lse are always fp32; indices and tables int32.  Softmax weights of the
 *    bf16 attentions meet V as bf16 on the tensor cores (their sum, the maximum and the
 *    accumulation are fp32), so an output is off by up to 2^-8 of the weighted |V| beside
 *    its own rounding.
 *
 * Regions of request b with history length L = seq_lens[b] (positions 0..L-1,
 * the current token included at L-1):
 *   sink        [0, s_end)            s_end   = min(n_sink, L)
 *   candidates  [s_end, l_start)      l_start = max(s_end, L - n_local)
 *   local       [l_start, L)
 * Sink and local are always attended; the top-k is taken over the candidates
 * only (ParisKV notes, §2.5: Sink and Local are attended densely on the GPU,
 * the retrieval region is the rest).
 */
#ifndef SKV_H
#define SKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t skv_status;

/* Return codes. */
#define SKV_OK 0
#define SKV_ERR_INVALID_ARGUMENT 1   /* NULL / negative / inconsistent sizes / misaligned */
#define SKV_ERR_UNSUPPORTED 2        /* valid but not built (e.g. d_idx != 128)            */
#define SKV_ERR_CUDA 3               /* a CUDA runtime call or launch failed                */
#define SKV_ERR_WORKSPACE_TOO_SMALL 4
#define SKV_ERR_DEVICE_FAULT 5       /* reserved: used by callers that map dev_status       */
#define SKV_ERR_TIMEOUT 6            /* reserved: used by callers that map dev_status       */

/* Bits of *dev_status (OR-ed by kernels). */
#define SKV_DEV_BAD_SLOT 1           /* slot-table entry names a block outside its pool     */
#define SKV_DEV_BAD_INDEX 2          /* a selected position is outside the candidate region */
#define SKV_DEV_BAD_LENGTH 4         /* seq_lens[b] outside [0, max_len] (clamped)          */
#define SKV_DEV_TIMEOUT 8            /* an internal pipeline wait gave up (never expected)  */
#define SKV_DEV_NO_BLOCK 16          /* a request got no blocks: too few are free           */

/* Element types. */
#define SKV_DTYPE_BF16 0
#define SKV_DTYPE_F32 1

/* How the scoring heads of one KV head's group combine into one score per key.
 * Each KV head ranks the context on its own (OasisKV notes, §3.2); the pages
 * leave the combination of a group's heads open, so both readings are offered,
 * and a third where every query head ranks on its own. */
#define SKV_AGG_MEAN 0               /* <q_bar, k>, q_bar the mean of the heads (orders keys like the sum) */
#define SKV_AGG_MAX 1                /* max over the heads g of <q_g, k>; bf16 with at most 16 scoring
                                        heads per KV head, else SKV_ERR_UNSUPPORTED */
/* Per query head: every query head j ranks the keys of its KV head j / G with its own
 * query, <q_j, k>, selects its own top-k and attends its own list.  The rows of scores,
 * idx and the gathered rows are then per query head (n_q_heads of them per request
 * instead of n_kv_heads); the keys are read once per KV head while scoring.  bf16,
 * n_idx_q_heads == n_q_heads (the attention query scores), at most 16 query heads per
 * KV head, paged K/V pools; skv_score, skv_topk, skv_topk_static, skv_gather,
 * skv_sparse_attn and skv_decode_step only (the block, prefetch, slot-cache and
 * ParisKV entry points return SKV_ERR_UNSUPPORTED). */
#define SKV_AGG_HEAD 2

/* Where the scored keys live. */
#define SKV_INDEX_PAGED 0            /* the K pool itself, through the slot table (block_size 16) */
#define SKV_INDEX_CONTIG 1           /* separate GPU-resident index keys [batch, n_kv_heads, max_len, d_idx] */

/*
 * Sizes of one decode step.
 *   n_q_heads      query heads; G = n_q_heads / n_kv_heads query heads share a
 *                  KV head (query head j belongs to KV head j / G).
 *   d_qk, d_v      key/query and value widths: 128/128 for paged K/V pools;
 *                  576/512 for the latent layout (gpu_v == NULL), where V is the
 *                  first d_v entries of the shared K row.
 *   d_idx          width of the scored keys and scoring query (128).
 *   n_idx_q_heads  heads of the scoring query; n_idx_q_heads / n_kv_heads of them
 *                  are averaged per KV head.  For SKV_INDEX_PAGED scoring with the
 *                  attention query itself: n_q_heads, with d_idx == d_qk.
 *   max_len        capacity: every seq_lens[b] <= max_len; sizes the scores row.
 *   topk           k: positions selected per (request, KV head) among candidates.
 *   n_sink,n_local window sizes (see regions above).
 *   block_size     tokens per slot-table entry: 16 (paged blocks) or 1 (per-token map).
 *   dtype          SKV_DTYPE_*.
 *   group_agg      SKV_AGG_MEAN, SKV_AGG_MAX or SKV_AGG_HEAD.
 *   sm_scale       softmax scale of the attention logits; <= 0 means 1/sqrt(d_qk).
 *   n_splits       split-K chunks per (request, KV head) for attention; 0 lets
 *                  the library choose from the sizes.
 *   seq_lens       device int32 [batch].
 * batch and n_kv_heads above 65535 (grid extents) return SKV_ERR_UNSUPPORTED.
 */
typedef struct skv_problem {
  int32_t batch;
  int32_t n_kv_heads;
  int32_t n_q_heads;
  int32_t d_qk;
  int32_t d_v;
  int32_t d_idx;
  int32_t n_idx_q_heads;
  int32_t max_len;
  int32_t topk;
  int32_t n_sink;
  int32_t n_local;
  int32_t block_size;
  int32_t dtype;
  int32_t group_agg;
  float sm_scale;
  int32_t n_splits;
  const int32_t *seq_lens;
} skv_problem;

/*
 * The KV pool: logical position t of request b resolves through
 *   e = slot_table[b * table_stride + t / block_size]
 *   e >= 0 : GPU block e,          rows gpu_k[e][h][t % block_size][:]
 *   e <  0 : host block (-e - 1),  rows host_k[-e-1][h][t % block_size][:]
 * (vToken notes, §3.4 Eq. (2): slot = block_id * S + offset; UlaCache article
 * §5: one logical address space, the map names the tier.)
 * Pools are [n_blocks, n_kv_heads, block_size, d] (d = d_qk for K, d_v for V).
 * gpu_v == NULL selects the latent layout: V is the first d_v entries of the K
 * row (n_kv_heads must be 1, host_v must be NULL).  host_* may be NULL when no
 * table entry is negative; n_*_blocks bound the entries (checked on device).
 * table_stride >= ceil(max_len / block_size).
 *
 * table_heads = 1 selects one table row per (request, KV head) instead (OasisKV
 * notes, §3.5, Fig. 9: each KV head keeps its own logical-block map, since different
 * heads select different blocks):
 *   e = slot_table[(b * n_kv_heads + h) * table_stride + t / block_size]
 *   e >= 0 : GPU block e holds this head's block only: gpu_k[e][t % block_size][:]
 *            (GPU pools [n_gpu_blocks, block_size, d])
 *   e <  0 : host block (-e - 1) as above (host pools keep every head).
 * Supported by skv_score, skv_gather, skv_sparse_attn, skv_decode_step, the slot cache
 * (skv_cache_*, skv_decode_step_cached) and the appends, K and V pools (not the latent layout);
 * the other entry points return SKV_ERR_UNSUPPORTED.
 * table_heads = 0 (the default of a zeroed struct) is the shared table above.
 */
typedef struct skv_kv_pool {
  const void *gpu_k;
  const void *gpu_v;
  int64_t n_gpu_blocks;
  const void *host_k;
  const void *host_v;
  int64_t n_host_blocks;
  const int32_t *slot_table;
  int32_t table_stride;
  int32_t table_heads;            /* 0: one table row per request; 1: one per (request, KV head) */
} skv_kv_pool;

/*
 * What skv_score reads.  SKV_INDEX_PAGED: the K pool through the slot table
 * (keys must be GPU-resident for candidate positions: host-resident blocks are
 * read over UVA, slowly).  SKV_INDEX_CONTIG: `keys` is a GPU-resident
 * [batch, n_kv_heads, max_len, d_idx] tensor (the indexer's key cache, kept on
 * the GPU: ECHO-OSDI26 wiki, core method 1).
 */
typedef struct skv_index_src {
  int32_t layout;
  const void *keys;
} skv_index_src;

/* Bytes of workspace skv_topk, skv_sparse_attn and skv_decode_step need for
 * this problem (the same figure serves all three). */
skv_status skv_workspace_size(const skv_problem *p, size_t *bytes);

/*
 * S0 + S1: scores[b][h][t] = <q_bar(b,h), key(b,h,t)> in fp32 for every
 * candidate t of request b; other positions of the row are left untouched.
 *   q_score  [batch, n_idx_q_heads, d_idx]; q_bar(b,h) is the mean of heads
 *            h*Gi .. h*Gi+Gi-1 with Gi = n_idx_q_heads / n_kv_heads.
 *   scores   device fp32 [batch, n_kv_heads, max_len]; with SKV_AGG_HEAD
 *            [batch, n_q_heads, max_len], row j the scores of query head j.
 * (ParisKV notes, §1 Eqs. (1)-(3): s_i = <k_i, q>; ECHO-OSDI26 wiki, core
 * method 3: the indexer scores every history key; OasisKV notes §3.2: every
 * KV head ranks the whole context on its own.)
 */
skv_status skv_score(const skv_problem *p, const void *q_score, const skv_index_src *index,
                     const skv_kv_pool *pool, float *scores, int32_t *dev_status, void *stream);

/*
 * S2: idx[b][h][0..k_eff) = the k_eff = min(topk, #candidates) candidate
 * positions with the largest scores, ascending; ties go to the lower position;
 * -0.0 equals +0.0; NaN ranks below every number.  idx[b][h][k_eff..topk) = -1.
 * Deterministic.  (ECHO-OSDI26 wiki, core method 3: the k-th score is a
 * threshold -- every key above it is in the exact top-k; core method 4 and
 * ParisKV notes §2.3: radix histograms with prefix scans instead of a sort.)
 *   scores  device fp32 [batch, n_kv_heads, max_len] (candidates read only).
 *   idx     device int32 [batch, n_kv_heads, topk].
 *   (SKV_AGG_HEAD: n_q_heads rows a request in both, one per query head.)
 *   ws      device workspace of at least skv_workspace_size() bytes.
 */
skv_status skv_topk(const skv_problem *p, const float *scores, int32_t *idx, void *ws,
                    size_t ws_bytes, int32_t *dev_status, void *stream);

/*
 * skv_topk without a workspace argument -- the pages have no counterpart; this
 * exists for callers that cannot allocate device memory when they select (a
 * plugin inside a runtime that owns the memory pool and gives it no allocator,
 * or a serving loop that must not call cudaMalloc, which can synchronise the
 * device).  Same arguments and results as skv_topk; the scratch is a fixed
 * 16 MiB device array inside the library (held on every GPU that loads the
 * library's module until the process exits), so this call allocates nothing.
 * Problems whose top-k scratch exceeds 16 MiB return SKV_ERR_WORKSPACE_TOO_SMALL
 * and enqueue nothing.  That scratch, for rows = batch * n_kv_heads (batch *
 * n_q_heads with SKV_AGG_HEAD):
 *   max_len <= 32768: none;
 *   longer rows whose segment winners fit one CTA (two stages): two arrays
 *     (winner keys, winner positions) of rows * round_up(segs * topk, 4) * 4
 *     bytes, each rounded up to 256 bytes; segs = ceil(max_len / seg), with seg
 *     16K keys, or 32K where that cuts the first stage's waves (a function of
 *     the problem alone);
 *   otherwise rows up to 128K keys: rows * 24 KB (digit histograms), 256-byte
 *     rounded; longer rows add tickets, row state and per-CTA counts, about
 *     24.1 KB per row plus 8 bytes per 2K keys of a row.
 * So roughly 680 request x KV-head rows fit when the histograms are needed.
 * The array's device address is looked up with cudaGetSymbolAddress in the
 * caller's current context on the first call in that context (that includes
 * the first call after cudaDeviceReset, which brings up a new context), and
 * cached with the context's id; make that first call before any stream
 * capture.  All calls share the array: calls whose kernels overlap on the GPU
 * race and give wrong results; serialise them (one stream, or events).
 */
skv_status skv_topk_static(const skv_problem *p, const float *scores, int32_t *idx, int32_t *dev_status,
                           void *stream);

/*
 * S3 materialised: the attended rows of every (b, h) in attended order
 *   list(b,h) = [0, s_end) ++ idx[b][h][0..topk) ++ [l_start, L)
 * resolved through the slot table.  k_out [batch, n_kv_heads, n_att, d_qk],
 * v_out [batch, n_kv_heads, n_att, d_v] with n_att = n_sink + topk + n_local
 * (SKV_AGG_HEAD: n_q_heads rows a request, query head j's list from KV head j / G);
 * list entries that are empty (idx < 0, or past the end of a short list) give
 * zero rows.  v_out may be NULL.  (vToken notes §3.4 Eq. (2); ECHO-OSDI26
 * wiki, core method 2: recall through the slot map.)
 */
skv_status skv_gather(const skv_problem *p, const skv_kv_pool *pool, const int32_t *idx,
                      void *k_out, void *v_out, int32_t *dev_status, void *stream);

/*
 * S3 + S4 + S5: for every query head j of KV head h = j / G,
 *   z_t = sm_scale * <q[b][j], K_t>,  out[b][j] = sum_t softmax(z)_t V_t,
 *   lse[b][j] = log sum_t exp(z_t)   (natural log)
 * over t in list(b,h) (idx entries < 0 are skipped; SKV_AGG_HEAD: over query
 * head j's own list(b,j), idx [batch, n_q_heads, topk]), computed as n_splits
 * fp32 online-softmax partials merged by log-sum-exp.  K/V rows are read
 * through the slot table inside the kernel (GPU pool from HBM, host pool over
 * UVA).  (ParisKV notes §2.5 and §1 Eqs. (1)-(3).)
 *   q    [batch, n_q_heads, d_qk];  out [batch, n_q_heads, d_v] (dtype);
 *   lse  fp32 [batch, n_q_heads] or NULL.
 */
skv_status skv_sparse_attn(const skv_problem *p, const void *q, const skv_kv_pool *pool,
                           const int32_t *idx, void *out, float *lse, void *ws, size_t ws_bytes,
                           int32_t *dev_status, void *stream);

/*
 * The whole step on one stream: skv_score (q_score, or q when q_score is NULL),
 * skv_topk, skv_sparse_attn.  scores and idx are outputs too.
 */
skv_status skv_decode_step(const skv_problem *p, const void *q, const void *q_score,
                           const skv_index_src *index, const skv_kv_pool *pool, float *scores,
                           int32_t *idx, void *out, float *lse, void *ws, size_t ws_bytes,
                           int32_t *dev_status, void *stream);

/* Static text of a status code. */
const char *skv_status_string(skv_status s);

/* Kernels this library has launched in this process (monotonic). */
uint64_t skv_launch_count(void);

/*
 * Check of the bounded waits (the library's failure detection; no page passage).
 * Every kernel that waits on an mbarrier gives up after a clock limit (about 2 s),
 * ORs SKV_DEV_TIMEOUT into *dev_status and returns, so a lost arrival never hangs
 * the device.  This call runs that same wait in a one-CTA kernel, on a barrier that
 * nothing completes (arrive = 0) or that one thread completes first (arrive = 1),
 * giving up after limit_cycles SM clocks.  After the stream drains, *dev_status has
 * SKV_DEV_TIMEOUT set (arrive = 0) or nothing added (arrive = 1).
 *   limit_cycles  in [1, 4e9] (4e9 clocks are about 2 s), else SKV_ERR_INVALID_ARGUMENT.
 *   arrive        0 or 1, else SKV_ERR_INVALID_ARGUMENT.
 *   dev_status    device int32, required: NULL returns SKV_ERR_INVALID_ARGUMENT.
 */
skv_status skv_check_wait_timeout(int64_t limit_cycles, int32_t arrive, int32_t *dev_status, void *stream);

/* ------------------------------------------------------------------------------------
 * Block selection from per-block key summaries (OasisKV notes, §3.2 "compressed
 * key summaries", after Quest): every 16-token block of a KV head keeps the
 * per-coordinate minimum and maximum of its keys; a KV head ranks blocks from
 * those two rows alone and attends the chosen blocks whole.
 *
 * A block's score is the largest <q, k> any key inside its per-coordinate box can
 * reach, sum_j max(q_j min_j, q_j max_j): q the group's mean query (SKV_AGG_MEAN)
 * or the largest of the heads' own bounds (SKV_AGG_MAX).  The sink and local
 * windows are rounded outward to whole blocks: blocks [0, ceil(n_sink / 16)) and
 * the blocks from floor(max(L - n_local, 0) / 16) on (none when n_local == 0);
 * the candidates are the blocks between.  The top topk_blocks candidates are
 * chosen exactly (ties to the lower block), and every token t < L of the sink,
 * chosen and local blocks is attended.
 *
 * Requirements: paged K/V pool (gpu_v != NULL) with block_size 16, d_qk = d_idx =
 * 128, n_idx_q_heads == n_q_heads (the attention group scores its blocks); else
 * SKV_ERR_UNSUPPORTED.  Errors are reported as for the token path above.
 *
 * summaries: device [batch, n_kv_heads, ceil(max_len / 16), 2, 128] of the pool's
 *            element type; per block the min row, then the max row; 16-byte
 *            aligned; caller-owned.  Blocks with no token below seq_lens[b] are
 *            not written.  A bad slot-table entry writes NaN rows (the block
 *            ranks last) and sets SKV_DEV_BAD_SLOT.
 * block_idx: device int32 [batch, n_kv_heads, topk_blocks]: chosen blocks,
 *            ascending, -1 past min(topk_blocks, candidate blocks).
 * att_idx:   device int32 [batch, n_kv_heads, list_len]: attended token
 *            positions, ascending, -1 padded; list_len from
 *            skv_block_workspace_size (16 * (ceil(n_sink/16) + topk_blocks +
 *            ceil(n_local/16) + 1)).
 * ------------------------------------------------------------------------------------ */

/* Workspace bytes for skv_block_select / skv_block_decode_step, and list_len
 * (may be NULL).  Enqueues nothing. */
skv_status skv_block_workspace_size(const skv_problem *p, int32_t topk_blocks, size_t *bytes, int32_t *list_len);

/* Writes the min / max summary rows of every block of every (request, KV head),
 * reading the K rows through the slot table (GPU pool, or the pinned host pool
 * over UVA).  Maintenance: run when blocks fill, not every decode step. */
skv_status skv_block_summaries(const skv_problem *p, const skv_kv_pool *pool, void *summaries, int32_t *dev_status,
                               void *stream);

/* Scores the candidate blocks from the summaries, chooses the top topk_blocks of
 * every (request, KV head) and writes block_idx and the attended token list att_idx. */
skv_status skv_block_select(const skv_problem *p, int32_t topk_blocks, const void *q, const void *summaries,
                            int32_t *block_idx, int32_t *att_idx, void *ws, size_t ws_bytes, int32_t *dev_status,
                            void *stream);

/* skv_block_select followed by skv_sparse_attn over att_idx (windows of width
 * zero); out / lse as for skv_decode_step. */
skv_status skv_block_decode_step(const skv_problem *p, int32_t topk_blocks, const void *q, const void *summaries,
                                 const skv_kv_pool *pool, int32_t *block_idx, int32_t *att_idx, void *out,
                                 float *lse, void *ws, size_t ws_bytes, int32_t *dev_status, void *stream);

/* ------------------------------------------------------------------------------------
 * Threshold prefetch of host rows (ECHO-OSDI26 wiki, core methods 3 and 5).  The
 * k-th largest score is a threshold; an EMA over steps of each (request, KV head)'s
 * k-th score predicts this step's.  While the indexer scores, a prefetch warp copies
 * the host rows of keys scoring above the prediction into a GPU staging area; the
 * exact top-k then runs as always, and the gather reads staged rows from HBM and
 * every other selected host row from the host pool (guaranteed recall).  A wrong
 * prediction costs speed only: the step's results are the same bits as without it.
 *
 * State, caller-owned, persistent across steps (zero-filled except tau_ema):
 *   tau_ema  device float [batch * n_kv_heads]: the EMA; NaN until a first step
 *            has selected (initialise to NaN: the first step prefetches nothing).
 *   epoch    device uint32 [1]: steps completed (initialise to 0).
 *   map      device uint64 [batch * n_kv_heads * max_len], 8-byte aligned,
 *            zero-filled once: (step tag << 32) | staging slot of a staged position.
 *   staging  device, 16-byte aligned, of the pool's element type: latent layout
 *            [batch * n_kv_heads, cap, d_qk]; paged pools [2, batch * n_kv_heads, cap, 128]
 *            (the staged K rows, then the staged V rows).
 *   count    device uint32 [batch * n_kv_heads], zero-filled once (reset by every step).
 *   stats    device uint32 [2] or NULL: running counts of attended host rows found
 *            staged / read from the host pool.
 *   cap      staging rows per (request, KV head) per step; rows past it are read
 *            from the host later.
 *   alpha    weight of the newest k-th score in the EMA, in (0, 1] (the pages: 0.5).
 * Supported, with contiguous index keys (a GPU-resident copy of the keys), bf16 and
 * SKV_AGG_MEAN: the latent layout (pool.gpu_v == NULL, block_size 1), or a paged pool
 * of 16-token blocks with d_qk = d_v = 128 whose host blocks back part of the history
 * (the 1M-context host-pool workload); else SKV_ERR_UNSUPPORTED.  The paged step ends
 * with one small kernel that advances the epoch and empties the staging counts.  One
 * step at a time per state (steps on one stream).
 * ------------------------------------------------------------------------------------ */
typedef struct skv_prefetch {
  float *tau_ema;
  uint32_t *epoch;
  uint64_t *map;
  void *staging;
  uint32_t *count;
  uint32_t *stats;
  int32_t cap;
  float alpha;
} skv_prefetch;

/* skv_decode_step with threshold prefetch of host rows; same results. */
skv_status skv_decode_step_prefetch(const skv_problem *p, const void *q, const void *q_score,
                                    const skv_index_src *index, const skv_kv_pool *pool, float *scores,
                                    int32_t *idx, void *out, float *lse, void *ws, size_t ws_bytes,
                                    const skv_prefetch *pf, int32_t *dev_status, void *stream);

/* ------------------------------------------------------------------------------------
 * GPU slot cache over a host pool that backs every token (ECHO-OSDI26 wiki, core
 * method 2).  The host pool holds token t of request b at row b * max_len + t (slot
 * table entry -(b * max_len + t) - 1); the GPU pool's rows ("slots") cache some
 * tokens (entry = the slot).  After a step's attention the cache is updated inside
 * the same enqueued work, with fixed-size state only:
 *   - attended tokens in GPU slots mark their slot used this step;
 *   - the attended tokens read from the host (misses), in (request, list position)
 *     order, take the best eviction candidates -- free slots, then the oldest last
 *     use, then the lower slot; the top `budget` of them by the exact top-k -- in
 *     ascending slot order, one each, while both last;
 *   - an evicted token's table entry returns to its host row; the promoted row is
 *     copied into its slot from the step's gathered rows (no second host read), and
 *     only then does its table entry name the slot (data, then map: UlaCache
 *     article, §8).
 * The step's own results are those of skv_decode_step; later steps find the
 * promoted tokens in HBM.
 *
 * cache.owner  device int32 [n_gpu_blocks]: b * max_len + t of the slot's token, or
 *              -1 (free).  Must agree with the slot table at the first call.
 * cache.prio   device int32 [n_gpu_blocks]: the last step that used the slot (start: -1).
 * cache.step   device int32 [1]: this step's number, advanced by every call.
 * cache.budget promotions per step, at most.
 * cache.stats  device uint64 [3] or NULL: every call adds its attended tokens found in
 *              GPU slots, those read from the host, and its promotions.
 * The call updates pool->slot_table and the rows of pool->gpu_k in place (both must be
 * writable and used by no other work meanwhile).  Slots are copies and are never written
 * back: new tokens are appended by skv_append_kv_cached.  Requirements: the latent layout
 * (pool->gpu_v == NULL, block_size 1), batch <= 64, n_host_blocks >= batch * max_len;
 * else SKV_ERR_UNSUPPORTED.
 *
 * With one table row per (request, KV head) (pool->table_heads = 1; OasisKV notes,
 * §3.5: each head keeps its own blocks resident) the same rule runs per (request, KV
 * head) u = b * n_kv_heads + h on blocks: the host pool backs block j of request b at
 * host block b * table_stride + j (every head; entry -(b * table_stride + j) - 1), a
 * slot holds one head's block, the distinct blocks of u's attended positions protect
 * their slots or miss, the misses are taken in (u, block) order, and owners are
 * u * table_stride + j.  A promoted block's K and V rows are copied from the host pool
 * into gpu_k and gpu_v.  Requirements: K and V pools, batch * n_kv_heads <= 1024,
 * n_host_blocks >= batch * table_stride, table_stride <= 262144.
 * ------------------------------------------------------------------------------------ */
typedef struct skv_slot_cache {
  int32_t *owner;
  int32_t *prio;
  int32_t *step;
  int32_t budget;
  uint64_t *stats;
} skv_slot_cache;

/* Bytes of the cache update's own workspace (cache_ws below).  Enqueues nothing. */
skv_status skv_cache_workspace_size(const skv_problem *p, const skv_kv_pool *pool, int32_t budget, size_t *bytes);

/* Creates, once per device, the library's side stream and its two events, which
 * skv_decode_step_cached uses to rank eviction candidates beside the step's attention
 * (it creates them itself on first use; call this first to keep their creation out of a
 * stream capture).  Acts on the current device. */
skv_status skv_cache_prepare(void);

/* The slot-cache update alone, for the step that skv_decode_step (or
 * skv_decode_step_prefetch) has just enqueued on `stream` with these same p, pool, idx
 * and ws: the update reads that step's selection and its gathered rows from ws, so
 * nothing may touch ws in between. */
skv_status skv_cache_update(const skv_problem *p, const skv_kv_pool *pool, const int32_t *idx, const void *ws,
                            size_t ws_bytes, const skv_slot_cache *cache, void *cache_ws, size_t cache_ws_bytes,
                            int32_t *dev_status, void *stream);

/* skv_decode_step, then the slot-cache update described above.  The ranking half of the
 * update (marking, eviction scores, their top-k) runs on the library's side stream,
 * forked from `stream` after the selection and joined back before the table changes,
 * so it overlaps the step's gather and attention; everything is ordered on `stream` when
 * the call's work there is complete (CUDA graph capture of `stream` captures both). */
skv_status skv_decode_step_cached(const skv_problem *p, const void *q, const void *q_score,
                                  const skv_index_src *index, const skv_kv_pool *pool, float *scores, int32_t *idx,
                                  void *out, float *lse, void *ws, size_t ws_bytes, const skv_slot_cache *cache,
                                  void *cache_ws, size_t cache_ws_bytes, int32_t *dev_status, void *stream);

/* ------------------------------------------------------------------------------------
 * ParisKV approximate retrieval: an alternative to exact scoring and top-k
 * (ParisKV notes, cc.laoqi.cc, arXiv 2602.07721, §2.2-§2.5).
 *
 * Per (request, KV head) row the GPU keeps compressed metadata of every key, built by
 * skv_paris_encode from the keys of the index source (contiguous index keys with
 * d_idx = 128, or the K pool through the slot table with d_qk = 128):
 *   - normalise, rotate by the SRHT R = H_128 diag(signs) / sqrt(128);
 *   - per 8-dim subspace s (16 of them): r = |k_s|, u = k_s / r; the centroid id is the
 *     sign pattern of u (bit j set iff u_j < 0), the argmax over the 256 fixed
 *     centroids (+-1/sqrt 8)^8 (§2.2, Eqs. (5)-(6));
 *   - each coordinate of u gets a 4-bit code, sign << 3 | cell, the cell from an
 *     8-level Lloyd-Max quantiser of |u_j| under u_j^2 ~ Beta(1/2, 7/2) (§2.4,
 *     Prop. 4.1; skv_paris_quantizer gives its levels and cuts); v = the decoded
 *     direction, alpha = <v, u>, w = |k| r / alpha (0 for a zero key or subspace).
 * A decode step (skv_paris_decode_step) then, per row, with n = the candidate
 * region's length:
 *   - q = the mean of the row's scoring query heads, q_t = R q / |q|;
 *   - collision (§2.3, Eq. (15)): in each subspace the centroids are ranked by
 *     <q_t,s, omega> (ties: lower id); with N = ceil(rho n / 1000) a centroid preceded
 *     by `start` keys (counted over the candidate region) earns 6..1 at the first cut
 *     ceil(P N / 100), P = 5, 15, 30, 50, 75, 100, above start, 0 from N on; a key's S
 *     sums its 16 centroids' weights;
 *   - the ceil(beta n / 1000) keys of largest S (ties: lower position) are candidates;
 *   - rerank (§2.4): s_hat = |q| sum_s w_s <v_s, q_t,s>; the exact top-k of s_hat
 *     (ties: lower position) is the selection, ascending, -1 past its end;
 *   - attention over sink U selection U local as in skv_decode_step (§2.5).
 * ------------------------------------------------------------------------------------ */
typedef struct skv_paris {
  int32_t m;            /* subspace dimension: 8 (the only one built) */
  int32_t beta_pm;      /* candidates, per mille of the candidate region: 1..1000 */
  int32_t rho_pm;       /* keys earning collision weight per subspace, per mille: beta_pm..1000 */
  const int8_t *signs;  /* device int8 [128]: the SRHT's random signs, +1 or -1 */
} skv_paris;

/* Device metadata, rows = batch * n_kv_heads, 16 subspaces, position-major: */
typedef struct skv_paris_index {
  uint8_t *cent;   /* [rows, max_len, 16] centroid ids (16-byte aligned) */
  uint32_t *rec;   /* [rows, max_len, 32] a 128-byte rerank record per key: words 0-15 the
                    * codes of subspaces 0-15 (nibble j = coordinate j), words 16-31 the
                    * fp32 weights of subspaces 0-15 (16-byte aligned) */
  int32_t *hist;   /* [rows, 16, 256] keys per centroid over positions [0, seq_len) */
} skv_paris_index;

/* The 8 levels and 7 cuts (ascending) of the magnitude quantiser for subspace dimension m
 * (3 <= m <= 64), computed on the host by Lloyd's iteration.  Enqueues nothing. */
skv_status skv_paris_quantizer(int32_t m, float *levels, float *thresholds);

/* Encodes positions [0, seq_lens[b]) of every row into *index and sets index->hist
 * (overwritten).  Positions past a row's length are left as they are.  A decode step
 * reads metadata for every position below its own seq_lens: encode with the same
 * lengths (or longer ones) first.  Errors as for skv_decode_step. */
skv_status skv_paris_encode(const skv_problem *p, const skv_paris *paris, const skv_index_src *index,
                            const skv_kv_pool *pool, const skv_paris_index *out, int32_t *dev_status, void *stream);

/* Workspace of skv_paris_decode_step (includes skv_decode_step's attention workspace). */
skv_status skv_paris_workspace_size(const skv_problem *p, const skv_paris *paris, size_t *bytes);

/* Byte offsets, inside that workspace, of the step's intermediates (for inspection):
 * out[0] rotated queries fp32 [rows, 128], [1] |q| fp32 [rows], [2] tier weights u8
 * [rows, 16, 256], [3] collision scores u8 [rows, max_len], [4] candidate counts int32
 * [batch], [5] candidate positions int32 [rows, c_cap], [6] their rerank scores fp32
 * [rows, c_cap]; out[7] = c_cap; [8] the fp32 centroid similarities <q_tilde_b, omega_c>
 * the tiers were ranked by [rows, 16, 256].  out holds 9 entries. */
skv_status skv_paris_workspace_offsets(const skv_problem *p, const skv_paris *paris, int64_t *out);

/* The retrieval alone (no attention): idx [batch, n_kv_heads, topk] receives the
 * selection.  Same arguments and requirements as skv_paris_decode_step, which is this
 * call followed by skv_sparse_attn on the same workspace. */
skv_status skv_paris_select(const skv_problem *p, const skv_paris *paris, const void *q_score,
                            const skv_index_src *index, const skv_paris_index *meta, const skv_kv_pool *pool,
                            int32_t *idx, void *ws, size_t ws_bytes, int32_t *dev_status, void *stream);

/* One decode step with ParisKV retrieval in place of S1/S2: q_score as for
 * skv_decode_step (NULL: q), idx [batch, n_kv_heads, topk] receives the selection.
 * Requirements: bf16, m = 8, retrieval dimension 128 (d_idx for contiguous index keys,
 * d_qk otherwise), batch * n_kv_heads <= 65535, and whatever the attention path
 * requires; else SKV_ERR_UNSUPPORTED. */
skv_status skv_paris_decode_step(const skv_problem *p, const skv_paris *paris, const void *q, const void *q_score,
                                 const skv_index_src *index, const skv_paris_index *meta, const skv_kv_pool *pool,
                                 int32_t *idx, void *out, float *lse, void *ws, size_t ws_bytes,
                                 int32_t *dev_status, void *stream);

/* ------------------------------------------------------------------------------------
 * New tokens: the norm and rotation of queries and keys, and their append to the cache.
 *
 * A row x of one head (d_qk entries) becomes, in fp32 and rounded once at the end,
 *   norm      y_j = gamma_j x_j / sqrt(mean_{i < norm_dim} x_i^2 + eps)   for j < norm_dim
 *             (the other entries, and every entry where gamma is NULL, are taken as they are);
 *   rotation  by the token's position t: the pairs (a, b) of the rotated span
 *             [rot_start, rot_start + rot_dim) turn by the angle t * inv_freq[i],
 *             (a, b) -> (a cos - b sin, b cos + a sin); pair i is
 *               SKV_ROPE_HALF   (rot_start + i, rot_start + i + rot_dim / 2)
 *               SKV_ROPE_PAIR   (rot_start + 2 i, rot_start + 2 i + 1).
 * inv_freq (of either sign, up to 2^14) is taken as exact and the angle is reduced to a
 * turn in 64-bit fixed point, off by less than 2^-32 of a turn at any position, before any
 * fp32 arithmetic: far positions and fast frequencies lose nothing.
 * ------------------------------------------------------------------------------------ */
#define SKV_ROPE_HALF 0
#define SKV_ROPE_PAIR 1

/*
 *   rot_start, rot_dim  the rotated span, inside [0, d_qk]; rot_dim 0: no rotation (inv_freq may be NULL).
 *   style               SKV_ROPE_HALF or SKV_ROPE_PAIR.
 *   norm_dim            entries the norm covers, in [1, d_qk]; 0: all d_qk.
 *   eps                 added to the mean square; >= 0.
 *   inv_freq            device fp32 [rot_dim / 2]: radians a position.
 *   q_gamma, k_gamma    device [norm_dim] of the element type, 16-byte aligned: the norm's
 *                       weights, shared by the heads; NULL: that side is not normed.
 * rot_start, norm_dim and d_qk multiples of 8, rot_dim a multiple of 8 (16 for SKV_ROPE_HALF),
 * d_qk and d_v at most 1024, else SKV_ERR_UNSUPPORTED.
 */
typedef struct skv_rotary {
  int32_t rot_start;
  int32_t rot_dim;
  int32_t style;
  int32_t norm_dim;
  float eps;
  const float *inv_freq;
  const void *q_gamma;
  const void *k_gamma;
} skv_rotary;

/*
 * The tokens of one call.  q, k and v are rows of n_q_heads * d_qk, n_kv_heads * d_qk and
 * n_kv_heads * d_v entries (the heads packed), q_stride / k_stride / v_stride elements
 * apart from token to token: column ranges of one fused projection output are fine.
 * Base pointers are 16-byte aligned and strides are multiples of 16 bytes (of a lone token
 * the stride is not looked at; with n_tokens 0 the pointers may be NULL).
 *   q           NULL: the call has no queries.
 *   positions   device int32 [n_tokens]; a negative one marks a padding token: its rows
 *               (which must be there) may be read, nothing is written.  NULL: token i ends
 *               its request's history, position seq_lens[request] - 1 (a history of
 *               length 0: a padding token).
 *   requests    device int32 [n_tokens]: the request (slot-table row) of each token, a
 *               negative one again padding.  NULL: token i is request i's.
 * A position outside [0, max_len) sets SKV_DEV_BAD_LENGTH and a request past the batch
 * SKV_DEV_BAD_INDEX; such tokens are skipped like padding.
 */
typedef struct skv_tokens {
  int32_t n_tokens;
  int32_t reserved;               /* 0 */
  const void *q;
  const void *k;
  const void *v;
  int64_t q_stride;
  int64_t k_stride;
  int64_t v_stride;
  const int32_t *positions;
  const int32_t *requests;
} skv_tokens;

/*
 * Norm and rotation alone: q_out [n_tokens, n_q_heads, d_qk] and k_out [n_tokens,
 * n_kv_heads, d_qk], packed -- or q_out == tokens->q and k_out == tokens->k, in place at
 * their strides; no other overlap.  tokens->v is ignored; either side may be NULL with
 * its output.  Of p, batch, the head counts, d_qk, dtype, max_len and (positions NULL)
 * seq_lens are used.  Without positions, requests NULL needs n_tokens <= batch.
 */
skv_status skv_qk_norm_rope(const skv_problem *p, const skv_rotary *rotary, const skv_tokens *tokens, void *q_out,
                            void *k_out, int32_t *dev_status, void *stream);

/*
 * Append: for every token, its K rows (normed and rotated) and its V rows (as they are)
 * of every KV head go to the pool row that the slot table names for (request, position),
 * in the GPU pool or the pinned host pool; its query rows, where tokens->q is given, are
 * normed and rotated into q_out [n_tokens, n_q_heads, d_qk] (or in place).  A table entry
 * outside its pool sets SKV_DEV_BAD_SLOT and that token's K/V rows are not written.  Rows
 * that no token names are left as they are.  The latent layout (pool->gpu_v == NULL) takes
 * no V (tokens->v is ignored).  Both table forms (table_heads 0 and 1), block sizes of any
 * length.  The pools are written (they must be writable, and read by no other work
 * meanwhile); two tokens of one call must not name the same pool row.  requests NULL
 * needs n_tokens <= batch.  n_tokens 0 enqueues nothing.
 * The pools alone are written: a score through the table (SKV_INDEX_PAGED) sees the new
 * keys, but what a selection keeps beside them -- contiguous index keys, block summaries,
 * ParisKV records -- is the caller's to renew for the new positions.
 * A row goes where the table names it and nowhere else: of a pool whose GPU slots a cache
 * manages (skv_decode_step_cached, skv_cache_update), a row written to a slot alone is lost
 * when the cache gives the slot to another -- such a pool takes skv_append_kv_cached.
 */
skv_status skv_append_kv(const skv_problem *p, const skv_rotary *rotary, const skv_tokens *tokens,
                         const skv_kv_pool *pool, void *q_out, int32_t *dev_status, void *stream);

/*
 * skv_append_kv for a pool whose GPU slots a cache manages (skv_slot_cache): K and V rows
 * whose table entry names a slot go to the host row that backs them too, so the host pool
 * keeps every token and an evicted slot loses nothing, positions written again included.
 * Both forms of the cache, with its requirements on p and pool (batch, max_len and the
 * pool are those of the cached step); the host pools must be writable.  Same arguments
 * and results as skv_append_kv otherwise.
 */
skv_status skv_append_kv_cached(const skv_problem *p, const skv_rotary *rotary, const skv_tokens *tokens,
                                const skv_kv_pool *pool, void *q_out, int32_t *dev_status, void *stream);

/* ------------------------------------------------------------------------------------
 * Attention of a batch that shares a prefix: every request attends its whole history,
 * and the keys of the shared positions [0, len) are read once for all requests.
 *   z_t = sm_scale * <q[b][j], K_t>,  out[b][j] = sum_t softmax(z)_t V_t,
 *   lse[b][j] = log sum_t exp(z_t)   over every t < L_b = seq_lens[b];
 * position t < len resolves through prefix->table[t / block_size], t >= len through the
 * request's own slot-table row (whose entries below len / block_size are not read; a
 * block that len ends inside may be shared or the request's own copy -- each side reads
 * the table it is named by).  Entries of either sign: GPU or pinned host blocks.
 *   table  device int32 [ceil(len / block_size)]; may be a row of the slot table; NULL
 *          with len 0 (every request then attends through its own row alone).
 *   len    in [0, max_len].
 * A request is of length 0 (an unused row of the batch: out 0, lse -inf) or holds the
 * whole prefix (L_b >= len); a length between, or below 0, sets SKV_DEV_BAD_LENGTH and
 * leaves out 0 and lse -inf; one past max_len sets it too and counts as max_len.  An
 * entry outside its pool sets SKV_DEV_BAD_SLOT and its rows get zero weight.  What lies in
 * a pool past a history's end or the prefix's end is never used.  Weights are bf16 at V, as
 * everywhere on bf16.
 * Of p, batch, the head counts, d_qk, d_v, max_len, block_size, dtype, sm_scale and
 * seq_lens are used.  bf16, d_qk = d_v = 128, K and V pools with one table row a request
 * (table_heads 0), at most 128 query heads per KV head, else SKV_ERR_UNSUPPORTED.
 * out [batch, n_q_heads, 128], lse fp32 [batch, n_q_heads] or NULL.  Deterministic: the
 * same inputs give the same bits.
 * ------------------------------------------------------------------------------------ */
typedef struct skv_prefix {
  const int32_t *table;
  int32_t len;
  int32_t reserved;               /* 0 */
} skv_prefix;

/* Bytes of workspace skv_prefix_attn needs for this problem and prefix length.  A call has
 * its workspace alone until it has run; calls in turn on one stream may share one. */
skv_status skv_prefix_workspace_size(const skv_problem *p, int32_t prefix_len, size_t *bytes);

skv_status skv_prefix_attn(const skv_problem *p, const void *q, const skv_kv_pool *pool, const skv_prefix *prefix,
                           void *out, float *lse, void *ws, size_t ws_bytes, int32_t *dev_status, void *stream);

/* ------------------------------------------------------------------------------------
 * Block tables and slot maps, kept on the GPU: every request grows by its new tokens or
 * gives its last ones back, blocks come off (and return to) a stack of free ones, and the
 * step's tokens learn their positions, requests and pool rows -- what skv_append_kv and
 * skv_append_kv4 take.  One call a step, nothing read back by the host; it can be captured.
 *
 * With L = seq_lens[b] before the call and n = n_new[b]:
 *   n > 0  the request takes the positions [s, s + n), s = L, or `base` where L is 0 (an
 *          unused row of the batch); its slot-table row gets free blocks for the indices
 *          that its new length needs and its old one did not; its length becomes s + n.
 *          (A request of length base, the prefix alone, has no block of its own, like one of 0.)
 *   n < 0  its last -n tokens go: the length becomes L + n, or 0 where no token past base
 *          is left; blocks that no longer hold any are free again.  (n = -max_len: all go.)
 *   n = 0  nothing.
 * Table indices below base / block_size are the caller's (a prompt that requests share):
 * they are neither read nor written; a block that base ends inside is the request's own.
 * Blocks given back in a call serve its requests first.  In order: the blocks that requests
 * need, b ascending and index ascending, come from those given back, the first request's
 * first and its lowest index first, and then off the top of the stack; of the blocks given
 * back, the rest go onto it, the last request's first and its highest index first -- so a
 * call that takes back what the call before it gave leaves the stack as it was.
 * A request is refused -- its length and table row stay, its tokens are padding, and a
 * SKV_DEV_* bit is set -- when its length is not one (L < 0, L > max_len, 0 < L < base) or
 * would pass max_len (SKV_DEV_BAD_LENGTH); when its rows would pass n_tokens
 * (SKV_DEV_BAD_INDEX); or when the blocks needed by it and the requests before it (those
 * refused for their rows or for want of blocks among them) are more than are free, and it needs any
 * (SKV_DEV_NO_BLOCK).
 *
 * Rows of the step: the tokens of request 0, then request 1's, and so on (a refused one's
 * rows stay in their place); n_tokens of them, the rows past the last token padding.
 *   positions, requests  device int32 [n_tokens]; -1 of padding.
 *   slots                device int64 [n_tokens] or NULL: the pool row of KV head 0's block,
 *                        block * block_size + position % block_size; -1 of padding.
 * The shared table form (one row a request); blocks of the GPU pool only.  An entry given
 * back that is no block below n_blocks sets SKV_DEV_BAD_SLOT and goes onto the stack all
 * the same; one that finds the stack full (of n_blocks entries) sets it and is dropped.
 *
 *   batch        requests, 1..4096 (more: SKV_ERR_UNSUPPORTED).
 *   max_len, block_size, table_stride   as in skv_problem and skv_kv_pool.
 *   base         positions that every request has before its own, in [0, max_len].
 *   n_blocks     blocks that there are; the stack's room.
 *   slot_table   device int32 [batch, table_stride], written in place.
 *   seq_lens     device int32 [batch], written in place.
 *   free_blocks  device int32 [n_blocks]: the stack, state[0] entries, the top last.
 *   state        device int32 [4]: the stack's entries; zero; zero; zero (the call's own).
 * The buffers are a call's own until it has run; calls in turn on one stream may share them.
 * ------------------------------------------------------------------------------------ */
typedef struct skv_tables {
  int32_t batch;
  int32_t max_len;
  int32_t block_size;
  int32_t base;
  int32_t table_stride;
  int32_t n_blocks;
  int32_t *slot_table;
  int32_t *seq_lens;
  int32_t *free_blocks;
  int32_t *state;
} skv_tables;

/* n_new device int32 [batch]; n_tokens 0: no rows (positions, requests and slots may be
 * NULL, and a request that grows is refused). */
skv_status skv_update_tables(const skv_tables *t, const int32_t *n_new, int32_t n_tokens, int32_t *positions,
                             int32_t *requests, int64_t *slots, int32_t *dev_status, void *stream);

/* ------------------------------------------------------------------------------------
 * A cache in 4 bits.  A row of 128 entries is held in groups of `group` (32, 64 or 128)
 * consecutive ones, each with a step s and a centre z in bf16 and a code c in 0..15 an entry:
 *   x^ = s (c - 8) + z
 * Of a row x in fp32 the append makes, per group, with lo and hi its least and largest entry,
 *   s = bf16((hi - lo) / 15),  z = bf16((hi + lo) / 2 + s / 2),
 *   c = 8 + the whole number next to (x - z) / s, ties to even, held to [-8, 7]  (8 where s is 0)
 * so |x - x^| <= s / 2, and at a group's ends up to 2^-5 s + 2^-8 |z| more, what the rounding of s
 * and z leaves them outside.  A group with an infinite or NaN entry, or whose hi - lo passes fp32, gets
 * s = z = NaN: it reads as NaN.
 *
 * Pools are those of skv_kv_pool (both table forms, GPU and pinned host blocks, K and V)
 * with bytes for elements: [n_blocks, n_kv_heads, block_size / 16, cell] (per-head tables:
 * GPU pools without n_kv_heads), block_size a multiple of 16.  A cell is 16 tokens of one
 * head, 1024 + 64 * (128 / group) bytes:
 *   token r's codes   64 bytes at 64 r: entries 2 j and 2 j + 1 share byte j, the even one
 *                     in its low half; byte j = 8 i + u stands at 64 r + 8 u + i
 *   token r's steps   a word a group at 1024 + 4 (r * (128 / group) + group): s in its low
 *                     half, z in its high half.
 *
 * d_qk = d_v = d_idx = 128, K and V pools (no latent layout), at most 16 query heads a KV
 * head, block_size a multiple of 16, max_len at most 2^30, each pool under 2^31 rows, else
 * SKV_ERR_UNSUPPORTED; a group other than the three is SKV_ERR_INVALID_ARGUMENT.  Slot caches,
 * prefetch, block summaries and ParisKV do not take these pools.
 * ------------------------------------------------------------------------------------ */

/* skv_append_kv into 4 bits: K rows normed and rotated, V rows as they are, both in fp32
 * until they are coded.  tokens and q_out of p->dtype (bf16 or fp32), as for skv_append_kv. */
skv_status skv_append_kv4(const skv_problem *p, const skv_rotary *rotary, const skv_tokens *tokens,
                          const skv_kv_pool *pool, int32_t group, void *q_out, int32_t *dev_status, void *stream);

/* skv_gather from 4 bits: the attended rows' values x^ in p->dtype, list and shapes as for
 * skv_gather.  idx may be NULL with topk 0 -- with n_sink 0 and n_local n, every request's
 * last n rows; k_out or v_out may be NULL.  SKV_AGG_HEAD as for skv_gather. */
skv_status skv_gather_kv4(const skv_problem *p, const skv_kv_pool *pool, int32_t group, const int32_t *idx,
                          void *k_out, void *v_out, int32_t *dev_status, void *stream);

/* skv_score from 4 bits: scores[b][h][t] = <q_bar, k^_t> in fp32 of the candidates, every
 * group_agg, rows and untouched positions as for skv_score.  p->dtype is bf16, q_score
 * [batch, n_idx_q_heads, 128]; SKV_AGG_MAX and SKV_AGG_HEAD: at most 16 scoring heads a KV
 * head.  A key whose entry lies outside its pool scores NaN.  Here and in the attention a query
 * head's results are of its own entries alone; one that is infinite or NaN makes them NaN,
 * and entries from 2^117 up count as infinite where their logits leave fp32. */
skv_status skv_score_kv4(const skv_problem *p, const void *q_score, const skv_kv_pool *pool, int32_t group,
                         float *scores, int32_t *dev_status, void *stream);

/* Bytes of workspace for skv_attn_kv4 and skv_decode_step_kv4 (skv_topk included). */
skv_status skv_kv4_workspace_size(const skv_problem *p, size_t *bytes);

/* Attention from 4 bits: over list(b,h) as skv_sparse_attn (SKV_AGG_HEAD: query head j's own
 * list; with topk 0 any aligned pointer, which is not read), or, with idx NULL, over every
 * position t < L_b whatever topk, n_sink and n_local.
 *   z_t = sm_scale * <q, k^_t>,  out = sum_t softmax(z)_t v^_t,  lse = log sum_t exp(z_t)
 * A request of length 0 (or an empty list) gives out 0 and lse -inf.  Entries outside their
 * pool, positions outside the candidates: flagged, zero weight.  p->dtype is bf16.  Softmax
 * weights times steps meet the codes as fp16 on the tensor cores: 11 bits, and what lies below
 * 2^-21 of the largest such product of its own query head and channel group is held to 2^-32
 * of that (value steps from 2^-75 up; smaller ones in turn to fewer bits); centres, sums and
 * the maximum are fp32, which holds the sums of values up to 2^116, or of up to 2^20 keys'
 * up to 2^126.  Deterministic: the same inputs give the same bits. */
skv_status skv_attn_kv4(const skv_problem *p, const void *q, const skv_kv_pool *pool, int32_t group,
                        const int32_t *idx, void *out, float *lse, void *ws, size_t ws_bytes, int32_t *dev_status,
                        void *stream);

/* skv_score_kv4 (of q_score, or q where it is NULL), skv_topk and skv_attn_kv4 over the
 * selection; scores and idx are outputs too. */
skv_status skv_decode_step_kv4(const skv_problem *p, const void *q, const void *q_score, const skv_kv_pool *pool,
                               int32_t group, float *scores, int32_t *idx, void *out, float *lse, void *ws,
                               size_t ws_bytes, int32_t *dev_status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SKV_H */
