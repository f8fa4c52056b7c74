/*
 * gbtopk — batched variable-length exact top-K for the sparse-attention
 * (DSA) indexer decode step, on NVIDIA GB300 (sm_103a).
 *
 * C ABI.  Every pointer argument is a plain pointer; "device" means it must
 * point into CUDA device memory (or managed memory) of the current device,
 * "host" means ordinary host memory.  All buffers are owned by the caller;
 * the library allocates nothing, keeps no state between calls and never
 * reads device data on the host, so every call can be captured in a CUDA
 * graph and replayed with new seq_lens / lengths contents.
 *
 * Calls are asynchronous on `stream` (a cudaStream_t; NULL is the legacy
 * default stream).  Host-side argument checks happen before anything is
 * enqueued; a negative status means nothing was enqueued.
 */
#ifndef GBTOPK_H
#define GBTOPK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the score matrix. */
#define GBTOPK_F32 0  /* IEEE binary32 */
#define GBTOPK_BF16 1 /* bfloat16 */
#define GBTOPK_F16 2  /* IEEE binary16 */

/* Status codes. */
#define GBTOPK_OK 0
#define GBTOPK_HINT_DISCARDED 1 /* warning: pre_idx unusable, ran hint-free (result still exact) */
#define GBTOPK_EINVAL (-1)       /* shape, dtype, grouping or null-pointer error */
#define GBTOPK_EALIGN (-2)       /* an output, the score base or a decode-step array is misaligned */
#define GBTOPK_EOVERLAP (-3)     /* two output buffers, or an output and what it may not lie over, overlap */
#define GBTOPK_EUNSUPPORTED (-4) /* outside the supported envelope (e.g. top_k too large) */
#define GBTOPK_ECUDA (-5)        /* the CUDA runtime refused the launch */
#define GBTOPK_EWORKSPACE (-6)   /* workspace missing, misaligned or too small */
#define GBTOPK_ETIMEOUT (-7)     /* device flag: a bounded wait gave up (see gbtopk_device_status) */

/* Largest supported top_k. */
#define GBTOPK_MAX_TOP_K 16384

/* Flags of the `deterministic` argument (FlashInfer compact page-table PR
 * body, "SMALL/LARGE tie selection" and the deterministic output order).
 * 0 asks for none: ties at the k-th value are resolved arbitrarily and the
 * selected columns come in no particular order. */
#define GBTOPK_SORTED 1     /* each row ordered by (value descending, column ascending);
                               alone it implies GBTOPK_TIE_SMALL */
#define GBTOPK_TIE_SMALL 2  /* among values equal to the k-th, keep the smallest columns */
#define GBTOPK_TIE_LARGE 4  /* among values equal to the k-th, keep the largest columns */

/*
 * gbtopk_varlen — top-K over decode-step indexer logits.
 *
 * Defined by the FlashInfer `flashinfer.top_k_varlen` page (parameters
 * logits, seq_lens, top_k, pre_idx, compress_ratio, next_n, return_values,
 * out_indices, out_values; "returns") and the TensorRT-LLM PR #17821
 * "self-sampling (GVR V2) top-K decode kernels" (exactness, MTP window,
 * short-row and value-padding conventions).
 *
 *  logits       device, [num_rows, width] of `dtype`, inner stride 1, row
 *               stride `row_stride` elements (>= width; arena views with a
 *               padded stride are accepted).  Must be aligned to the element
 *               size.  Columns at or beyond a row's valid count are never read.
 *  seq_lens     device int32 [num_rows / next_n]: KV-token lengths.  Row r
 *               (request i = r / next_n, t = r % next_n) ranks its first
 *               n_r = max(0, (seq_lens[i] - next_n + t + 1) / compress_ratio)
 *               columns, clamped to `width`.
 *  next_n       >= 1, and num_rows % next_n == 0.
 *  compress_ratio >= 1.
 *  top_k        1 .. GBTOPK_MAX_TOP_K.
 *  pre_idx      device int32 [num_rows / next_n, top_k] or NULL: the previous
 *               step's top-K columns of each request, raw (no +1 offset),
 *               pre_idx[i][0] the argmax.  It only steers the threshold guess
 *               and never changes the result.  Entries outside [0, n_r)
 *               (including -1) and duplicates are ignored.  A pointer that
 *               is not 16-byte aligned is discarded with status
 *               GBTOPK_HINT_DISCARDED.
 *  out_indices  device int32 [num_rows, top_k], 16-byte aligned.  Row r gets
 *               min(top_k, n_r) column indices followed by -1.
 *  out_values   device, dtype of logits, [num_rows, top_k], 16-byte aligned,
 *               or NULL.  Selected values are bit copies; padding slots hold
 *               the lowest finite value of the dtype.
 *  deterministic  0 or a set of GBTOPK_SORTED / GBTOPK_TIE_SMALL /
 *               GBTOPK_TIE_LARGE (the two tie modes exclude each other;
 *               other bits are GBTOPK_EINVAL).  0: ties at the k-th value
 *               are resolved arbitrarily and the selected columns come in no
 *               particular order.  1 (GBTOPK_SORTED): ties take the smallest
 *               columns and each row is ordered by (value descending, column
 *               ascending).  A tie mode fixes the selected set; without
 *               GBTOPK_SORTED its order is unspecified.  Short rows
 *               (n_r <= top_k) come in column order unless sorted.
 *  workspace    device scratch of at least gbtopk_workspace_bytes(...) bytes,
 *               256-byte aligned.  Its first 4 bytes are a status word that
 *               should start at zero (see gbtopk_device_status); everything
 *               else is scratch that each call writes before reading (the
 *               row's guess, chunk ticket and candidate counters are written
 *               by the call's first kernel), so the contents need no
 *               initialisation and one workspace serves any sequence of
 *               calls on one stream.  Calls that may overlap in
 *               time (different streams, concurrent graph replays) need
 *               separate workspaces.
 *  stream       cudaStream_t.
 *
 * Returns GBTOPK_OK / GBTOPK_HINT_DISCARDED, or a negative status (nothing
 * enqueued).  num_rows == 0 is a no-op.
 */
int gbtopk_varlen(const void *logits, int dtype, int64_t num_rows, int64_t width,
                  int64_t row_stride, const int32_t *seq_lens, int32_t next_n,
                  int32_t compress_ratio, int32_t top_k, const int32_t *pre_idx,
                  int32_t *out_indices, void *out_values, int deterministic,
                  void *workspace, size_t workspace_bytes, void *stream);

/*
 * gbtopk_page_table_transform — top-K fused with the compact page-table
 * transform.
 *
 * Defined by the FlashInfer compact page-table PR body quoted on the SGLang
 * PR #33237 page ("--dsa-topk-backend flashinfer with fused top-k"): for a
 * selected local score index idx,
 *     page = page_table[r, pt_row_start_r + idx / page_size]
 *     out  = page * page_size + idx % page_size,     out_raw = idx,
 * with -1 padding kept in both outputs, which stay positionally aligned.
 *
 *  scores       device, [num_rows, width] of `dtype`, inner stride 1, row
 *               stride `row_stride` elements.
 *  lengths      device int32 [num_rows]: valid scores per row.
 *  row_starts   device int32 [num_rows] or NULL: offset of the row's first
 *               valid score, in score elements.  The valid window is
 *               [row_start, row_start + length) clamped to the width; a
 *               row_start outside [0, width] gives an empty row.  Indices
 *               are local to row_start.
 *  page_table   device int32 [num_rows, pt_cols], inner stride 1, row stride
 *               pt_row_stride entries (non-contiguous tables are accepted).
 *  pt_row_starts  device int32 [num_rows] or NULL: first page-table entry of
 *               each row, in page-table entries.  NULL means row_starts when
 *               page_size == 1 and 0 when row_starts is NULL; NULL together
 *               with row_starts and page_size > 1 is GBTOPK_EINVAL.
 *  page_size    1 .. 2^30.  A page-table column outside [0, pt_cols) yields
 *               -1 in `out` (out_raw still holds idx).  page * page_size +
 *               idx % page_size is computed modulo 2^32: keeping it inside
 *               int32 is the caller's responsibility.
 *  top_k        1 .. GBTOPK_MAX_TOP_K.
 *  out          device int32 [num_rows, top_k], 16-byte aligned.
 *  out_raw      device int32 [num_rows, top_k], 16-byte aligned, or NULL; must
 *               not overlap `out` (GBTOPK_EOVERLAP).
 *  deterministic, workspace, stream: as for gbtopk_varlen.
 */
int gbtopk_page_table_transform(const void *scores, int dtype, int64_t num_rows,
                                int64_t width, int64_t row_stride,
                                const int32_t *lengths, const int32_t *row_starts,
                                const int32_t *page_table, int64_t pt_cols,
                                int64_t pt_row_stride, const int32_t *pt_row_starts,
                                int32_t page_size, int32_t top_k, int32_t *out,
                                int32_t *out_raw, int deterministic, void *workspace,
                                size_t workspace_bytes, void *stream);

/*
 * gbtopk_ragged_transform — top-K fused with the ragged KV index offset.
 *
 * Defined by the SGLang TopK ops wiki, fast_topk_transform_ragged_fused (its
 * top-k indices shifted by a per-row offset for a ragged KV layout, the
 * offsets topk_indices_offset of shape (B)): the selection is the one of
 * gbtopk_page_table_transform's rows, and each selected row-local index idx
 * is written as idx + topk_indices_offset[r] (modulo 2^32); -1 padding stays
 * -1.
 *
 *  scores, lengths, row_starts, top_k, deterministic, workspace, stream:
 *               as for gbtopk_page_table_transform (valid window
 *               [row_start, row_start + length) clamped to the width).
 *  topk_indices_offset  device int32 [num_rows].
 *  out          device int32 [num_rows, top_k], 16-byte aligned.
 */
int gbtopk_ragged_transform(const void *scores, int dtype, int64_t num_rows, int64_t width,
                            int64_t row_stride, const int32_t *lengths, const int32_t *row_starts,
                            const int32_t *topk_indices_offset, int32_t top_k, int32_t *out,
                            int deterministic, void *workspace, size_t workspace_bytes, void *stream);

/*
 * gbtopk_page_table_transform_cu_seqlens — top-K fused with a page_size-1
 * page table indexed by request.
 *
 * Defined by the SGLang TopK ops wiki, fast_topk_transform_fused (page table
 * with page_size 1 and cu_seqlens_q of shape (Batch + 1)): score row r
 * belongs to request b with cu_seqlens_q[b] <= r < cu_seqlens_q[b + 1], and
 * each selected row-local index idx is written as page_table[b, idx]; an idx
 * at or beyond pt_cols gives -1, and a row that no request covers is empty
 * (all -1).
 *
 *  scores, lengths, row_starts, top_k, deterministic, workspace, stream:
 *               as for gbtopk_page_table_transform.
 *  page_table   device int32 [num_reqs, pt_cols], inner stride 1, row stride
 *               pt_row_stride entries.
 *  cu_seqlens_q device int32 [num_reqs + 1], nondecreasing.
 *  out          device int32 [num_rows, top_k], 16-byte aligned.
 */
int gbtopk_page_table_transform_cu_seqlens(const void *scores, int dtype, int64_t num_rows,
                                           int64_t width, int64_t row_stride, const int32_t *lengths,
                                           const int32_t *row_starts, const int32_t *page_table,
                                           int64_t pt_cols, int64_t pt_row_stride,
                                           const int32_t *cu_seqlens_q, int64_t num_reqs,
                                           int32_t top_k, int32_t *out, int deterministic,
                                           void *workspace, size_t workspace_bytes, void *stream);

/*
 * gbtopk_workspace_bytes — scratch needed by a call with this geometry.
 * A pure function of its arguments (capture-stable).  The workspace holds a
 * device status word plus, when rows are long enough to be split across
 * thread blocks, per-row candidate buffers, counters and histograms (the
 * multi-CTA split described on the FlashInfer `top_k_varlen` page, parameter
 * `workspace`).  Returns 0 for invalid arguments.
 */
size_t gbtopk_workspace_bytes(int64_t num_rows, int64_t width, int32_t top_k, int dtype);

/*
 * gbtopk_device_status — reads (and clears) the device status word of a
 * workspace.  Synchronises `stream`.  *flags receives a bit set:
 *   bit 0  a bounded wait on an asynchronous copy gave up; the affected rows
 *          (on the three-kernel path: every row of that call) were
 *          recomputed from global memory, so the outputs are exact;
 *   bit 1  a copy did not land even within a second bounded wait: the
 *          outputs of that call are not reliable (the shared memory the copy
 *          targets was not reused; rows whose selection needed it were left
 *          unwritten or written unsorted).
 * The waits are bounded by a poll count; the environment variable
 * GBTOPK_WAIT_POLLS (a positive integer, read once per process) lowers the
 * first wait's count, which exercises the recovery of bit 0 in tests.
 * Returns GBTOPK_OK, GBTOPK_EINVAL or GBTOPK_ECUDA.  The pages define no
 * such call.
 */
int gbtopk_device_status(void *workspace, uint32_t *flags, void *stream);

/*
 * gbtopk_plan_query — the launch plan for a geometry, for inspection and
 * tests.  `out` must hold 13 entries: out[0..12] = {columns per chunk of a
 * split row, chunks of the widest split row (1 when no row is split),
 * longest row finished by the one-block row kernel, row-kernel shared
 * memory bytes, split (0/1), candidate entries reserved per split row,
 * stream-kernel shared memory bytes (0 unless split rows take the three-
 * kernel path), finalize-kernel shared memory bytes (likewise), workspace
 * bytes, workspace bytes per row, row-kernel shared memory bytes with
 * GBTOPK_SORTED, fused (1 when split rows take the two-kernel path: the
 * row kernel's guess, then one chunk-kernel block per chunk, the row's last
 * block selecting it), chunk-kernel shared memory bytes (fused plans)}.
 * Returns GBTOPK_OK or GBTOPK_EINVAL / GBTOPK_EUNSUPPORTED (nothing is
 * written then).
 */
int gbtopk_plan_query(int64_t num_rows, int64_t width, int32_t top_k, int dtype,
                      int64_t *out);

/*
 * gbtopk_varlen_static_ws — gbtopk_varlen without a caller-provided
 * workspace.  The pages define no such call; it exists for callers that
 * cannot allocate device memory where they need top-K: code running while
 * a CUDA graph is being captured (cudaMalloc cannot be captured), engines
 * whose device memory belongs to an external allocator or planner that
 * forbids side allocations, and plugin hosts that only pass in tensors they
 * own.  It allocates nothing: the scratch is one 16 MiB buffer compiled into
 * the library (a file-scope __device__ array), reserved on every GPU that
 * loads the library and held until the process exits.
 *
 * Arguments, outputs and status codes are those of gbtopk_varlen, minus the
 * workspace.  A geometry whose workspace (gbtopk_workspace_bytes) exceeds
 * 16 MiB is refused with GBTOPK_EWORKSPACE before anything is enqueued; for
 * example a 64 x 163840 fp32 batch with top_k 2048 needs about 6.3 MiB.
 *
 * The first call on a device looks up the buffer's device address (once per
 * device); make that first call before capturing a CUDA graph.  The address
 * belongs to the device's context: after cudaDeviceReset the process must
 * not call this entry point again.  All calls on a device share the one
 * buffer and its contents carry over between calls (nothing needs clearing:
 * each call writes the scratch it reads), so calls that may overlap in time
 * on the GPU — other streams, concurrent graph replays, other host threads —
 * race on it and must be serialised by the caller.  The buffer's device
 * status word (see gbtopk_device_status) cannot be read on this path: the
 * bounded-wait flags of these calls are not reported.
 */
int gbtopk_varlen_static_ws(const void *logits, int dtype, int64_t num_rows, int64_t width,
                            int64_t row_stride, const int32_t *seq_lens, int32_t next_n,
                            int32_t compress_ratio, int32_t top_k, const int32_t *pre_idx,
                            int32_t *out_indices, void *out_values, int deterministic,
                            void *stream);

/* ------------------------------------------------------------------------
 * The decode step after the selection: attention over a paged key/value
 * cache, the weight each cached position accumulates, eviction by it, and
 * the verification of drafted tokens.
 *
 * Shared conventions (those of the calls above): row r belongs to request
 * i = r / next_n as its drafted token t = r % next_n, and seq_lens[i] counts
 * the next_n newest tokens too, whose keys and values are in the cache
 * already.  Position p of request i lies in cache slot
 *     page_table[i, p / page_size] * page_size + p % page_size,
 * the slot numbers that gbtopk_page_table_transform writes.  A position
 * whose page-table column is >= pt_cols, whose page id is negative or whose
 * slot is >= num_slots does not exist: it is never read or written.
 * Row r sees position p when p < ctx, ctx = seq_lens[i] - next_n (the
 * context), or when bit p - ctx of its tree mask is set: tree_mask[r] has
 * bit j set when drafted token j is token t itself or one of its ancestors
 * (or any other set the caller wants seen).  tree_mask NULL is a chain: row
 * t sees tokens 0 .. t.
 *
 * The cache holds one key and one value row of head_dim elements for each
 * (slot, kv head), with any slot and head strides (in elements) that are
 * multiples of 8; bases, and fp32 weights, 16-byte aligned, every other array
 * on its element's boundary (GBTOPK_EALIGN).  Query head h reads
 * kv head h / (q_heads / kv_heads).  dtype is GBTOPK_BF16 or GBTOPK_F16 for
 * queries, cache and output alike; head_dim is a multiple of 8, 8 .. 256;
 * next_n is 1 .. 64; q_heads is a multiple of kv_heads (others:
 * GBTOPK_EUNSUPPORTED for the dtype and the sizes, GBTOPK_EINVAL for the
 * grouping).
 */

#define GBTOPK_MAX_NEXT_N 64    /* drafted tokens of a request (bits of a tree mask) */
#define GBTOPK_MAX_HEAD_DIM 256

/*
 * gbtopk_tree_attention — attention of drafted tokens over a paged cache:
 *     s(r,h,p) = scale * <q[r,h], k[slot(i,p), h / group]>  over visible p,
 *     lse[r,h] = log sum_p exp s,   out[r,h] = sum_p exp(s - lse) v[slot(i,p)].
 * A row that sees nothing gives zeros and lse = -infinity.  Keys and values
 * of positions that no row of the request sees are not read, whatever they
 * hold; an infinity or NaN of a drafted token reaches the rows that see it
 * and no others.
 *
 * Arithmetic: scores, sums and the output until it is stored are 32 bits; the
 * products are the tensor core's.  Each probability is rounded to dtype for
 * its product with the value (by up to 2^-8 of itself in bf16, 2^-11 in fp16;
 * the sum it is divided by is of the unrounded ones), and the output once
 * more, so the output's error is 1.2 to 1.4 times that of its own rounding.
 * In fp16 the positions of a tile (128 consecutive ones, 64 above dimension
 * 128) have one scale: probabilities below 2^-13 of the tile's largest (2^-20
 * where that is the row's largest) are off by up to 2^-24 (2^-31) of it.
 *
 *  q            device [num_rows, q_heads, head_dim], inner stride 1, row and
 *               head strides multiples of 8, 16-byte aligned.
 *  page_table   device int32 [num_rows / next_n, pt_cols], row stride
 *               pt_row_stride.
 *  seq_lens     device int32 [num_rows / next_n].
 *  tree_mask    device uint64 [num_rows] (as int64) or NULL.
 *  out          device [num_rows, q_heads, head_dim], contiguous, 16-byte
 *               aligned.
 *  lse          device fp32 [num_rows, q_heads] or NULL.
 *  workspace    as for gbtopk_varlen, gbtopk_attention_workspace_bytes(...)
 *               bytes; its status word reports bounded waits that gave up
 *               (bit 1: outputs not reliable; GBTOPK_WAIT_POLLS, which lowers
 *               the waits' limit, makes them).  At most 2^31 - 1 slots.
 */
int gbtopk_tree_attention(const void *q, int dtype, int64_t num_rows, int64_t q_row_stride,
                          int64_t q_head_stride, int32_t q_heads, int32_t kv_heads,
                          int32_t head_dim, const void *k_cache, int64_t k_slot_stride,
                          int64_t k_head_stride, const void *v_cache, int64_t v_slot_stride,
                          int64_t v_head_stride, int64_t num_slots, const int32_t *page_table,
                          int64_t pt_cols, int64_t pt_row_stride, int32_t page_size,
                          const int32_t *seq_lens, int32_t next_n, const int64_t *tree_mask,
                          float scale, void *out, float *lse, void *workspace,
                          size_t workspace_bytes, void *stream);

/*
 * gbtopk_selected_attention — the same attention over a list of slots for
 * each row: indices device int32 [num_rows, top_k] with row stride
 * idx_row_stride, as gbtopk_page_table_transform writes them.  Entries < 0
 * or >= num_slots are skipped wherever they stand; a slot listed twice
 * counts twice.
 */
int gbtopk_selected_attention(const void *q, int dtype, int64_t num_rows, int64_t q_row_stride,
                              int64_t q_head_stride, int32_t q_heads, int32_t kv_heads,
                              int32_t head_dim, const void *k_cache, int64_t k_slot_stride,
                              int64_t k_head_stride, const void *v_cache, int64_t v_slot_stride,
                              int64_t v_head_stride, int64_t num_slots, const int32_t *indices,
                              int64_t top_k, int64_t idx_row_stride, float scale, void *out,
                              float *lse, void *workspace, size_t workspace_bytes, void *stream);

/* Scratch of the two attention calls (a pure function; 0 for invalid sizes). */
size_t gbtopk_attention_workspace_bytes(int64_t num_rows, int32_t q_heads, int32_t kv_heads,
                                        int32_t head_dim);

/*
 * gbtopk_cache_weights — adds to weights[i, w, p] the attention probability
 * that the request's rows gave position p:
 *     weights[i, w, p] += sum_{t, h} exp(s(r,h,p) - lse[r,h])
 * over the rows t whose bit in accept_mask[i] is set (all rows when it is
 * NULL) that see p, and over the query heads h of kv head w (weight_heads ==
 * kv_heads) or all query heads (weight_heads == 1).  A row with lse =
 * -infinity adds nothing.  Positions >= width are not counted.  The sum
 * over rows and heads of one position has a fixed order.
 *
 *  lse          device fp32 [num_rows, q_heads]: gbtopk_tree_attention's.
 *  accept_mask  device uint64 [num_rows / next_n] (as int64) or NULL.
 *  weights      device fp32 [num_rows / next_n, weight_heads, width],
 *               contiguous; updated in place.
 */
int gbtopk_cache_weights(const void *q, int dtype, int64_t num_rows, int64_t q_row_stride,
                         int64_t q_head_stride, int32_t q_heads, int32_t kv_heads,
                         int32_t head_dim, const void *k_cache, int64_t k_slot_stride,
                         int64_t k_head_stride, int64_t num_slots, const float *lse,
                         const int32_t *page_table, int64_t pt_cols, int64_t pt_row_stride,
                         int32_t page_size, const int32_t *seq_lens, int32_t next_n,
                         const int64_t *tree_mask, const int64_t *accept_mask, float scale,
                         float *weights, int32_t weight_heads, int64_t width, void *workspace,
                         size_t workspace_bytes, void *stream);

/*
 * gbtopk_cache_evict — keeps the positions of each request that carry the
 * most weight and packs their keys and values, in order, into new pages.
 *
 * The survivors of request i are its positions p < min(seq_lens[i], width,
 * pt_cols * page_size); with accept_mask, of the last next_n positions only
 * the drafted tokens whose bit is set (the accepted path).  When more than
 * `budget` survive, the last min(recent, budget) of them are kept and, of
 * the others, those with the largest weight (ties: the lowest position) up
 * to the budget.  The kept positions in ascending order become positions
 * 0, 1, ... of out_page_table.  weight_heads == kv_heads makes the choice
 * for each kv head by itself, weight_heads == 1 one choice for all.
 *
 *  weights      device fp32 [num_requests, weight_heads, width], contiguous;
 *               ranked by float order (-0 equals +0; NaN order unspecified).
 *  k_cache, v_cache  read at the pages of page_table and written at those of
 *               out_page_table, which must not share a slot with any page
 *               that page_table lists (pages of the source may be shared by
 *               requests).  elem_bytes 2 or 4; head_dim * elem_bytes, the
 *               strides' bytes and the bases multiples of 16 bytes.  A kept
 *               position without a source slot is written as zeros; one
 *               without a destination slot is not written.
 *  out_page_table  device int32 [num_requests, out_pt_cols], out_pt_cols *
 *               page_size >= budget.
 *  kept         device int32 [num_requests, weight_heads, budget]: the kept
 *               positions, padded with -1.
 *  new_lens     device int32 [num_requests]: positions kept.  Not overlapping
 *               seq_lens.
 *  out_weights  device fp32 like weights, not overlapping it: the kept
 *               positions' weights (-0 as +0), zeros behind them.
 */
int gbtopk_cache_evict(const float *weights, int64_t num_requests, int32_t weight_heads,
                       int64_t width, const int32_t *seq_lens, int32_t next_n,
                       const int64_t *accept_mask, int32_t budget, int32_t recent, void *k_cache,
                       int64_t k_slot_stride, int64_t k_head_stride, void *v_cache,
                       int64_t v_slot_stride, int64_t v_head_stride, int64_t num_slots,
                       int32_t kv_heads, int32_t head_dim, int32_t elem_bytes,
                       const int32_t *page_table, int64_t pt_cols, int64_t pt_row_stride,
                       const int32_t *out_page_table, int64_t out_pt_cols,
                       int64_t out_pt_row_stride, int32_t page_size, int32_t *kept,
                       int32_t *new_lens, float *out_weights, void *stream);

/*
 * gbtopk_verify_drafts — verifies a request's drafted tokens against the
 * target model's distributions, losslessly, from given random numbers.
 *
 * Row n of request i is node n of its draft tree; node 0 is the last token
 * already decided and logits row n is the target's distribution after node
 * n: p_n = softmax(logits[n] / temperature[i]), or, where the temperature is
 * <= 0, one at the largest logit (lowest index) and zero elsewhere.  The
 * parent of node n is the highest bit below n of tree_mask[n] (NULL: n - 1);
 * a node without one cannot be reached.  From node 0 the children c of the
 * current node are tried in order:
 *   draft_probs NULL:  accept when u_c * m < p(x_c), with m = 1 - the p of
 *                      the children refused before (a token refused before
 *                      has p = 0);
 *   draft_probs given: accept when u_c * q(x_c) < p(x_c), q = row of the
 *                      current node (what its child was drawn from; chains
 *                      only: tree_mask must be NULL).
 * The accepted child becomes the current node; where none is, the next token
 * is argmax_v rest(v) / noise[i, v] (lowest index), which draws from rest
 * when noise is standard exponential: rest is p without the refused tokens,
 * or max(p - q, 0) after a refusal under draft_probs, or p.  -1 where rest
 * is zero everywhere.  A token outside [0, vocab) is never accepted.
 * (A request with fewer drafts than next_n: such a token in the places left
 * over, and under draft_probs a row of zeros for the node before them.)
 * Probabilities are 32-bit numbers; the exponentials of the sums and of the
 * draw, and the draw's division by the noise, are the fast ones (relative
 * errors of about 2^-20), so of two words whose races are that close either
 * may be drawn.
 *
 *  logits       device [num_rows, vocab] of dtype (any of the three), row
 *               stride row_stride.  Logits of -infinity have p = 0.
 *  tokens       device int32 [num_rows]; node 0's is not read.
 *  uniforms     device fp32 [num_rows] in [0, 1); node 0's is not read.
 *  noise        device fp32 [num_requests, vocab], positive, contiguous.
 *  temperature  device fp32 [num_requests] or NULL (1).
 *  draft_probs  device fp32 [num_rows, vocab], contiguous, or NULL.
 *  accepted     device int32 [num_requests]: drafted tokens accepted.
 *  path         device int32 [num_rows]: the nodes from 0 to the last
 *               accepted, padded with -1.
 *  next_token   device int32 [num_requests].
 *  accept_mask  device uint64 [num_requests] (as int64): the path's bits, for
 *               gbtopk_cache_weights and gbtopk_cache_evict.
 *  workspace    gbtopk_verify_workspace_bytes(...) bytes, as for gbtopk_varlen.
 */
int gbtopk_verify_drafts(const void *logits, int dtype, int64_t num_rows, int64_t vocab,
                         int64_t row_stride, const int32_t *tokens, const float *uniforms,
                         const float *noise, int32_t next_n, const int64_t *tree_mask,
                         const float *temperature, const float *draft_probs, int32_t *accepted,
                         int32_t *path, int32_t *next_token, int64_t *accept_mask,
                         void *workspace, size_t workspace_bytes, void *stream);

/* Scratch of gbtopk_verify_drafts (a pure function; 0 for invalid sizes). */
size_t gbtopk_verify_workspace_bytes(int64_t num_rows, int64_t vocab, int32_t next_n);

/* Human-readable name of a status code (static string).  The pages define no
 * such call; the codes follow the error cases of the FlashInfer
 * `top_k_varlen` page ("Raises") and the status convention above. */
const char *gbtopk_status_str(int status);

#ifdef __cplusplus
}
#endif

#endif /* GBTOPK_H */
