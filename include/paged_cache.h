/*
 * paged_cache.h -- the cache side of libpagedattn: what a serving step does to the paged K/V
 * cache around the attention calls of paged_attn.h.
 *
 *   - rotary positions of queries and keys                      -> paged_rope_run
 *   - rotating new keys (and queries) and writing new K/V rows through the page table that
 *     the attention calls read                                  -> paged_append_run
 *   - which row owns which page: giving rows pages for new tokens, forking a row, freeing
 *     rows, compacting the live pages, copying pages            -> paged_cache_*_run
 *   - keeping rows within a budget of tokens: adding up the attention weight that every token
 *     receives, selecting the tokens to keep, cutting rows back to them
 *                              -> paged_weights_run, paged_cache_select_run, paged_cache_evict_run
 *
 * The conventions of paged_attn.h hold: *_dev are device pointers, *_host host pointers; all
 * memory is the caller's and nothing is allocated; device work goes to `stream` and nothing
 * synchronises the host, so every *_run call can be captured in a CUDA graph; arguments are
 * checked on the host before anything is enqueued; calls work on the current device.  No call
 * here keeps anything between calls but what the caller's arrays hold, and calls that share
 * tables, lengths, counts or pages have to be ordered by the caller (one stream, or events).
 * int32 arrays are 4-byte aligned, workspaces 16-byte, pools and caches 16-byte.
 *
 * Status words.  A call with a workspace clears the status word at the workspace's start and
 * ORs in what it finds (paged_attn_workspace_status reads it); the workspace belongs to one
 * launch in flight at a time.  Every call takes status_dev too, as an argument or (extend, fork,
 * compact, evict) in its params: a uint32 word that it ORs into and never clears, or NULL
 * (paged_attn_workspace_status reads such a word as well).  In both, PAGED_ATTN_ERR_METADATA
 * means that an item broke its contract and was left out, PAGED_ATTN_ERR_CAPACITY that the free
 * pages did not suffice for every item, and PAGED_ATTN_ERR_TIMEOUT that a device wait ran out and
 * rows were not written.
 */
#ifndef PAGED_CACHE_H
#define PAGED_CACHE_H

#include <stddef.h>
#include <stdint.h>

#include "paged_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- rotary positions ------------------------------------------------------------------
 * Column pair i of the first rotary_dim columns of a head (R = rotary_dim, n = R / 2) turns
 * by the angle a = p * f_i at position p:
 *     y1 = m (x1 cos a - x2 sin a),   y2 = m (x2 cos a + x1 sin a),
 * (x1, x2) = columns (i, i + n) in the half layout, (2i, 2i + 1) in the interleaved one; m is
 * attention_factor.  Columns from R on stay as they are. */
#define PAGED_ROPE_HALF 0
#define PAGED_ROPE_INTERLEAVED 1

/* Frequencies f_i = base^(-2i / R), changed for contexts longer than the original one (s =
 * factor, L = original_max_position):
 *   LINEAR      f_i / s
 *   NTK         base * s^(R / (R - 2)) in the place of base
 *   YARN        f_i (1 - g_i) + (f_i / s) g_i, where g_i rises from 0 to 1 between the pairs
 *               that make `high` (default 32) and `low` (default 1) turns over L positions:
 *               d(beta) = R ln(L / (2 pi beta)) / (2 ln base), g_i = clamp((i - d0) / max(d1 -
 *               d0, 0.001), 0, 1), d0 = max(floor(d(high)), 0), d1 = min(ceil(d(low)), R - 1);
 *               attention_factor 0.1 ln s + 1 for s > 1
 *   WAVELENGTH  with t_i = L f_i / (2 pi) turns and c_i = clamp((t_i - low) / (high - low), 0,
 *               1): (1 - c_i) f_i / s + c_i f_i (defaults: low 1, high 4) */
#define PAGED_ROPE_SCALE_NONE 0
#define PAGED_ROPE_SCALE_LINEAR 1
#define PAGED_ROPE_SCALE_NTK 2
#define PAGED_ROPE_SCALE_YARN 3
#define PAGED_ROPE_SCALE_WAVELENGTH 4

typedef struct paged_rope_scaling {
  int rotary_dim;               /* R: even, 2 to 512                                      */
  int kind;                     /* PAGED_ROPE_SCALE_*                                     */
  double base;                  /* > 1                                                    */
  double factor;                /* s > 0 (unused by NONE)                                 */
  double original_max_position; /* L > 0 (YARN and WAVELENGTH)                            */
  double low, high;             /* 0, 0 selects the defaults; else 0 < low < high         */
} paged_rope_scaling;

/* Host only: the R / 2 frequencies in radians per position and the attention factor (1 for
 * every kind but YARN). */
int paged_rope_frequencies(const paged_rope_scaling* scaling, double* freqs_host,
                           float* attention_factor_host);

/* Host only: the table that the kernels read, one entry per column pair: f / (2 pi), the turns
 * per position, as the fraction of a turn in units of 2^-64 (rounded to nearest).  A position
 * times an entry, modulo 2^64, is then the exact fraction of a turn, whatever the position, so
 * far positions lose nothing.  freqs must be at most 2^20 in magnitude.  Copy the n entries to
 * the device once. */
int paged_rope_table(const double* freqs_host, int n, uint64_t* table_host);

typedef struct paged_rope_params {
  int num_tokens;        /* T                                                             */
  int num_qo_heads;      /* heads of q                                                    */
  int num_kv_heads;      /* heads of k; 0: no k                                           */
  int head_dim;          /* D: a multiple of 8, at most 512                               */
  int rotary_dim;        /* R: even, 2 to D                                               */
  int layout;            /* PAGED_ROPE_HALF or PAGED_ROPE_INTERLEAVED                     */
  int dtype;             /* PAGED_ATTN_DTYPE_* of q, k and the outputs                    */
  int inverse;           /* 1: turn by -a, which is the transpose of the forward map and so
                            its gradient: the gradient of the input is this call on the
                            gradient of the output                                        */
  float attention_factor; /* m: finite                                                    */
  /* Strides in elements between tokens and between heads; 0, 0 selects contiguous [T, heads,
   * D].  The D columns of a head are contiguous. */
  int64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride;
  int64_t q_out_token_stride, q_out_head_stride, k_out_token_stride, k_out_head_stride;
} paged_rope_params;

/* Rotate q [T, Hq, D] and k [T, Hkv, D] (NULL with num_kv_heads = 0) at positions_dev [T]
 * (any int32), reading table_dev [R / 2].  Computed in fp32 and rounded once.  An output may
 * be its own input (same pointer and strides); otherwise outputs share no element with any
 * input.  Rows of an input may overlap or be the same (a stride of 0 beside one that is not);
 * rows of an output lie apart, the tokens within a step of the heads or the heads within a step
 * of the tokens, or the call is refused.  Pointers need the alignment of their element; accesses
 * are wide where pointers, strides and R allow 16 bytes. */
int paged_rope_run(const paged_rope_params* params, const void* q_dev, const void* k_dev,
                   const int32_t* positions_dev, const uint64_t* table_dev, void* q_out_dev,
                   void* k_out_dev, uint32_t* status_dev, void* stream);

/* ---- appending to the cache ------------------------------------------------------------- */
typedef struct paged_append_params {
  int batch;             /* B                                                             */
  int seq_len_q;         /* fixed form: SQ new tokens per request (rows b * SQ ..)        */
  int total_q;           /* packed form (qo_indptr given): rows of q, k and v              */
  int num_qo_heads;      /* heads of q; 0: no q                                            */
  int num_kv_heads, head_dim; /* D: a multiple of 8, at most 512                           */
  int page_size;         /* a multiple of 8, at most 128                                   */
  int num_pages;         /* P                                                              */
  int combined_cache;    /* 1: [P, 2, Hkv, ps, D]; 0: separate K and V pools               */
  int max_pages_per_request; /* C: columns of block_tables (unused with kv_indptr)         */
  int rotary_dim;        /* R: 0 = no rotation, else even, 2 to D                          */
  int layout;            /* PAGED_ROPE_*                                                   */
  float attention_factor; /* m: finite                                                     */
  int in_dtype;          /* PAGED_ATTN_DTYPE_* of q, k and v; the cache and q_out are bf16 */
  /* Elements between consecutive tokens (0: contiguous); heads are D apart, so q, k and v may
   * be slices of one fused projection [total_q, Hq + 2 Hkv, D]. */
  int64_t q_token_stride, k_token_stride, v_token_stride;
} paged_append_params;

/* Write the K and V rows of new tokens into the cache, keys rotated at their positions, and
 * rotate the new queries: the arrays are those of the attention call that follows.
 *   q_dev [total, Hq, D], k_dev, v_dev [total, Hkv, D];  q_out_dev [total, Hq, D] contiguous,
 *   16-byte aligned (q_dev and q_out_dev NULL with num_qo_heads = 0);
 *   qo_indptr_dev [B + 1]: packed form: request b owns rows qo_indptr[b] .. qo_indptr[b + 1]
 *   (none is fine); rows from qo_indptr[B] on are padding: q_out keeps what it holds there.
 *   NULL: the fixed form;
 *   kv_indptr_dev [B + 1]: CSR table, request b owns pages_dev[kv_indptr[b] ..]; NULL: pages_dev
 *   is block_tables [B, C];
 *   seq_lens_kv_dev [B]: lengths WITH the new tokens: token i of a request with nq new tokens
 *   and length L gets position L - nq + i, as the attention calls place query i;
 *   table_dev [R / 2] (NULL with rotary_dim = 0);
 *   k_cache_dev: combined cache or K pool; v_cache_dev: V pool (NULL with a combined cache).
 * The cache may be any page-aligned part of a larger buffer (16-byte aligned).  A token whose
 * position is negative, whose page lies past its request's entries or outside [0, num_pages)
 * is not written (metadata bit); its q_out row is.  Two requests that append to the same page
 * must not write the same slots.  No operand overlaps the cache or q_out. */
int paged_append_run(const paged_append_params* params, const void* q_dev, const void* k_dev,
                     const void* v_dev, const int32_t* qo_indptr_dev,
                     const int32_t* kv_indptr_dev, const int32_t* pages_dev,
                     const int32_t* seq_lens_kv_dev, const uint64_t* table_dev, void* q_out_dev,
                     void* k_cache_dev, void* v_cache_dev, uint32_t* status_dev, void* stream);

/* ---- which row owns which page -------------------------------------------------------------
 * Three int32 arrays say it:
 *   block_tables [rows, C]  page ids of each row, live in its first ceil(len / page_size)
 *                           entries (what later entries hold does not matter and is kept);
 *   seq_lens [rows]         tokens of each row, 0 = empty;
 *   page_refs [num_pages]   how many live entries name the page; 0 = free.
 * Block tables are the row-strided tables of paged_prefill_run; with kv_indptr = {0, C, 2C, ..}
 * they are the CSR tables of the other calls.  A page that a row has only partly filled is
 * named by that row alone, so it can be appended to; full pages may be shared.
 * Fresh pages are the lowest free ids, given to the items in the order listed. */
typedef struct paged_cache_params {
  int rows;                   /* rows of block_tables                                      */
  int max_pages_per_request;  /* C                                                         */
  int page_size;              /* a multiple of 8, at most 128                              */
  int num_pages;              /* P <= 2^24                                                 */
  uint32_t* status_dev;       /* extend, fork, compact and evict OR their findings in; or
                                 NULL                                                      */
} paged_cache_params;

/* The pools of every layer, all with the same page ids; a page is below 2^31 bytes. */
#define PAGED_CACHE_MAX_POOLS 256
typedef struct paged_cache_pools {
  int num_layers;        /* N: N pointers (combined) or 2 N (K, V of each layer in turn), at
                            most PAGED_CACHE_MAX_POOLS                                     */
  int num_pages, num_kv_heads, page_size, head_dim;
  int combined_cache;    /* 1: [P, 2, Hkv, ps, D]; 0: [P, Hkv, ps, D] pairs                */
  void* const* pools_host; /* HOST array of device pointers, 16-byte aligned, bf16         */
} paged_cache_pools;

/* Free the listed rows: each live page's count goes down by one and the row's length to 0; the
 * table's entries are kept.  An empty row stays empty, so a row listed twice is freed once.  Row
 * ids outside [0, rows), page ids outside the pool and pages whose count is already 0 are left
 * out (metadata bit). */
int paged_cache_free_run(const paged_cache_params* params, const int32_t* rows_dev, int n,
                         const int32_t* block_tables_dev, int32_t* seq_lens_dev,
                         int32_t* page_refs_dev, uint32_t* status_dev, void* stream);

/* Make each listed row longer by new_tokens[i] (>= 0) tokens, with fresh pages where its last
 * page does not hold them.  Item i is served if it needs no page or if the free pages suffice
 * for it and every item listed before it; otherwise its row stays as it is (capacity bit): its
 * length does not count the new tokens, so appending them would write over the row's last ones.
 * Rows outside [0, rows), a row listed before, negative tokens and rows that would outgrow C
 * pages are left out (metadata bit).  n <= 4096. */
size_t paged_cache_extend_workspace_size(int n);
int paged_cache_extend_run(const paged_cache_params* params, const int32_t* rows_dev,
                           const int32_t* new_tokens_dev, int n, int32_t* block_tables_dev,
                           int32_t* seq_lens_dev, int32_t* page_refs_dev, void* workspace_dev,
                           size_t workspace_bytes, void* stream);

/* Make children[i] a copy of parents[i]: the full pages are shared (their counts go up), and a
 * partly filled last page is copied, its live tokens only, into a fresh page, in every layer.
 * A parent may be listed any number of times; parents are read as they are before the call.
 * Children are distinct and empty.  Items that break this, that name rows outside [0, rows), a row
 * as its own parent or a parent whose partly filled page lies outside the pool are left out
 * (metadata bit); an item for whose fresh page the free pages do not suffice (counted as in extend)
 * leaves its child empty (capacity bit).  Ids outside the pool among the parent's full pages are
 * copied as they are and counted nowhere (metadata bit).  n <= 4096. */
size_t paged_cache_fork_workspace_size(int n);
int paged_cache_fork_run(const paged_cache_params* params, const paged_cache_pools* pools,
                         const int32_t* parents_dev, const int32_t* children_dev, int n,
                         int32_t* block_tables_dev, int32_t* seq_lens_dev,
                         int32_t* page_refs_dev, void* workspace_dev, size_t workspace_bytes,
                         void* stream);

/* Move the live pages into [0, num_live): with n = the number of live pages, the k-th live page
 * at or above n moves into the k-th free page below n, in every layer; nothing else moves.
 * block_tables_out and page_refs_out get the new tables and counts; each may be its input
 * (in place), else it overlaps none of the inputs and what does not change is copied.
 * num_live_dev [1] receives n.  Every live table entry must have a count (else it keeps its
 * id; metadata bit for ids outside the pool and rows longer than C pages). */
size_t paged_cache_compact_workspace_size(int num_pages);
int paged_cache_compact_run(const paged_cache_params* params, const paged_cache_pools* pools,
                            const int32_t* block_tables_dev, const int32_t* seq_lens_dev,
                            const int32_t* page_refs_dev, int32_t* block_tables_out_dev,
                            int32_t* page_refs_out_dev, int32_t* num_live_dev,
                            void* workspace_dev, size_t workspace_bytes, void* stream);

/* Copy page src_pages[i] of every pool of `src` to page dst_pages[i] of the same pool of `dst`,
 * i < n.  dst may be src (other page counts are fine where they differ; everything else
 * agrees).  Destinations are distinct, and with dst = src none is also a source: pages that
 * break this hold a mixture afterwards.  Pools of src and dst are the same or do not overlap.
 * Ids outside the pools are left out (metadata bit). */
int paged_cache_copy_run(const paged_cache_pools* src, const paged_cache_pools* dst,
                         const int32_t* src_pages_dev, const int32_t* dst_pages_dev, int n,
                         uint32_t* status_dev, void* stream);

/* ---- keeping rows within a budget of tokens ---------------------------------------------------
 * What the kept tokens of a row are may differ between layers and KV heads, how many there are may
 * not: each (layer, KV head) keeps a list of its own, and its kept keys and values move to the
 * row's first slots.  Keys keep the rotation of their old positions. */
typedef struct paged_weights_params {
  int batch;             /* B                                                             */
  int num_qo_heads, num_kv_heads; /* G = Hq / Hkv <= 64                                    */
  int head_dim;          /* D: 128 or 256                                                 */
  int page_size;         /* a multiple of 8, at most 128                                  */
  int num_pages;         /* P                                                             */
  int combined_cache;    /* 1: [P, 2, Hkv, ps, D]; 0: a K pool [P, Hkv, ps, D]            */
  int max_pages_per_request; /* C: columns of block_tables (unused with kv_indptr)        */
  int seq_len_q;         /* fixed form: SQ queries per request                            */
  int total_q;           /* rows of q and lse                                             */
  int last_queries;      /* n > 0: only the last n queries of each request count; 0: all  */
  int mask_type;         /* PAGED_ATTN_MASK_*, as the attention call had it               */
  int width;             /* W: weights per (request, KV head)                             */
  float sm_scale;        /* as the attention call had it; <= 0 selects 1 / sqrt(D)        */
  float decay;           /* factor on the weights before the call                         */
} paged_weights_params;

/* Add up what the queries of an attention call look at: for each request b, KV head h and key j
 *     weights[b, h, j] = decay * weights[b, h, j]
 *                        + sum over counted queries i that see j, and the G query heads of h,
 *                          of exp(sm_scale q[i, head] . k[j, h] - lse[i, head]),
 * where the old weight of the tokens that the call's queries stand for, the last nq of a request
 * with nq queries, is 0: their entries are written without being read, and so is every entry with
 * decay = 0.  Entries past a request's length are left alone, and so is a request without queries.
 * Weights belong to a row as its page table does: whoever forks a row copies them to the child.
 * Attention calls with a window are not served: keys outside it would count.
 *   q_dev [total_q, Hq, D] bf16 and lse_dev [total_q, Hq] fp32, natural logarithm: the attention
 *   call's queries and its LSE (a row with an LSE of -inf sees nothing and adds nothing);
 *   k_cache_dev: combined cache or K pool;
 *   qo_indptr_dev [B + 1]: packed form, or NULL: the fixed form;
 *   kv_indptr_dev [B + 1] with pages_dev (CSR), or NULL: pages_dev is block_tables [B, C];
 *   weights_dev [B, Hkv, W] fp32.
 * Scores, exponentials and sums are fp32.  The order of a sum depends on the batch's shape, W and
 * the device, never on timing: the same call on the same device repeats bit for bit.  Keys past W
 * or past the request's table entries get no weight, a key whose page id lies outside
 * [0, num_pages) keeps its old one, and a request whose offsets do not lie in [0, total_q] is left
 * out (metadata bit). */
int paged_weights_run(const paged_weights_params* params, const void* q_dev, const float* lse_dev,
                      const void* k_cache_dev, const int32_t* qo_indptr_dev,
                      const int32_t* kv_indptr_dev, const int32_t* pages_dev,
                      const int32_t* seq_lens_dev, float* weights_dev, uint32_t* status_dev,
                      void* stream);

typedef struct paged_cache_select_params {
  int num_layers;        /* N: layers in weights                                          */
  int rows;              /* R: rows of weights and seq_lens                               */
  int num_kv_heads;      /* Hkv                                                           */
  int width;             /* W: weights per (layer, row, KV head)                          */
  int keep;              /* K >= 1: tokens to keep of each row                            */
  int sink;              /* the first `sink` tokens are kept whatever their weight        */
  int recent;            /* and the last `recent`; sink + recent <= keep                  */
} paged_cache_select_params;

/* kept_dev [N, n, Hkv, K]: for each layer, listed row and KV head the indices of the tokens to
 * keep, in ascending order: the first `sink`, the last `recent`, and of the tokens between them
 * those with the highest weights_dev [N, R, Hkv, W] (fp32), the lower index first among equal
 * ones (0.0 and -0.0 are equal) and NaN below everything.  A row of at most K tokens keeps them
 * all: its lists are 0, 1, .. followed by -1.  A row may be listed more than once.  Rows outside
 * [0, R) and rows with a negative length or more than W tokens are left out: -1 everywhere
 * (metadata bit).  Weights past a row's length are not read. */
int paged_cache_select_run(const paged_cache_select_params* params, const int32_t* rows_dev, int n,
                           const float* weights_dev, const int32_t* seq_lens_dev,
                           int32_t* kept_dev, uint32_t* status_dev, void* stream);

/* Cut each listed row of more than `keep` tokens back to `keep`: in every layer and KV head slot j
 * gets token kept[layer, i, head, j] (key and value), and so does weights_dev[layer, row, head, j]
 * where weights_dev [N, rows, Hkv, weights_width] (fp32) is given.  Rows of at most `keep` tokens
 * stay as they are, whatever their lists hold.  The lists are ascending, kept_dev [N, n, Hkv,
 * keep], as paged_cache_select_run writes them for the rows' present lengths.
 * `sink`: the first `sink` entries of every list are 0, 1, .. sink - 1, so pages that lie wholly
 * in them do not change and stay shared (0 is always right).  Any other page among the row's first
 * ceil(keep / page_size) that other rows share is replaced by a fresh one (as in extend: the lowest
 * free ids, item by item, in the order of the row); pages past them, and replaced ones, lose a
 * count, and pages whose counts reach 0 this way are free after the call.  What the row's table
 * holds past its new length is kept, and so are the slots past it in its last page, unless that
 * page was replaced: a fresh one holds there whatever it held before.
 * The row has no more in common with others than its first `sink` tokens: behind a shared prefix
 * (paged_decode_shared_run) prefix_lens is to be cut to that.
 * Left out (metadata bit): rows outside [0, rows), a row listed before, rows with ids outside the
 * pool or more tokens than C pages or weights_width hold, lists whose first entry is negative or
 * whose last one is not in [keep - 1, length).  A slot whose entry breaks the order (below the
 * slot's own index, past the length, or another token's inside the `sink` pages) keeps what it
 * holds (metadata bit); entries that are not ascending otherwise give a mixture of tokens.  A row
 * for whose fresh pages the free ones do not suffice (counted as in extend) stays as it is
 * (capacity bit).  n <= 4096. */
size_t paged_cache_evict_workspace_size(int n, int keep, int page_size);
int paged_cache_evict_run(const paged_cache_params* params, const paged_cache_pools* pools,
                          const int32_t* rows_dev, int n, const int32_t* kept_dev, int keep,
                          int sink, float* weights_dev, int weights_width,
                          int32_t* block_tables_dev, int32_t* seq_lens_dev,
                          int32_t* page_refs_dev, void* workspace_dev, size_t workspace_bytes,
                          void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_CACHE_H */
