/*
 * pa.h -- C ABI of libpa: paged GQA decode attention for GB300 (sm_103a).
 *
 * The library holds three things:
 *   1. a fixed-block K/V page allocator (host metadata only),
 *   2. an append kernel that scatters newly written K/V rows into their pages,
 *   3. a split-K decode kernel that reads K/V through a block table, plus the
 *      log-sum-exp merge of its splits.
 *
 * Conventions for every entry point:
 *   - Pointers marked "device" are CUDA device pointers owned by the caller
 *     (for example torch tensors); the library never frees them.  Pointers
 *     marked "host" are ordinary host memory.
 *   - Calls that take a stream are asynchronous and stream-ordered.  Errors
 *     found on the host (bad sizes, unsupported shapes, null pointers) are
 *     returned before anything is launched.  Errors found on the device (a
 *     table entry outside the pool, a bounded wait that expired) are written
 *     to the caller's device error word `err` (first error wins) and read back
 *     with pa_get_error().
 *   - No call allocates device memory.  Scratch space for pa_decode is passed
 *     in by the caller, sized by pa_decode_workspace_size().
 *
 * Data layout.  The pages describe a pool of pages plus a page table but
 * print no byte layout; this one is the library's own:
 *   K pool and V pool are separate device buffers, each
 *       pool[block][kv_head][page_size rows]
 *   with page_size a multiple of 16.  Row (seq s, position p) of kv head g
 *   lives in block block_table[s * table_stride + p / page_size] at slot
 *   p % page_size.  Each (block, kv_head) page is cut into row groups of 16
 *   consecutive slots; a group holds its 16 rows in 16 * row_bytes bytes,
 *   arranged for the decode kernel's tensor-core fragment loads:
 *     1. Q4_0/Q8_0 only: the rows' block scales (2 bytes each) in a 256-byte
 *        scale region.  K pool: scale of (row r, block b) at 16 r + 2 b.
 *        V pool: at 64 (b/2) + 16 ((r%8)/2) + 8 (b%2) + 4 (r/8) + 2 (r%2).
 *     2. The rest of each row -- an F16 row, or a quantised row's quant bytes
 *        block after block -- as 16-byte chunks, row after row; with C chunks
 *        per row, chunk c of row r sits at chunk position r C + (c XOR r%8).
 *   A row group is therefore one contiguous run that one bulk copy moves, and
 *   a whole 16-row page of every head is one run per pool.  Write pools with
 *   pa_append_rows, which takes rows in their ordinary format.
 *   Row formats are ggml's: F16 (IEEE binary16, 2*head_dim bytes), Q8_0
 *   (32-value blocks: fp16 scale d, 32 int8 q, value q*d; 34 bytes) and Q4_0
 *   (32-value blocks: fp16 d, 16 bytes whose byte j holds element j in the low
 *   nibble and element j+16 in the high nibble, value (nibble-8)*d; 18 bytes).
 */
#ifndef PA_H
#define PA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; 0 is the legacy default stream. */
typedef struct CUstream_st* pa_stream_t;

typedef enum {
  PA_OK = 0,
  PA_ERR_INVALID = 1,     /* bad argument: null pointer, size, alignment, length */
  PA_ERR_UNSUPPORTED = 2, /* shape or format this library does not implement */
  PA_ERR_OOM = 3,         /* not enough free blocks; nothing was allocated */
  PA_ERR_STALE = 4,       /* a handle is released, unknown or repeated; nothing was released */
  PA_ERR_BOUNDS = 5,      /* device: a table entry or position outside the pool or table */
  PA_ERR_TIMEOUT = 6,     /* device: a bounded wait inside a kernel expired */
  PA_ERR_CUDA = 7         /* a CUDA runtime call failed */
} pa_status;

/* Row formats, numbered as ggml numbers them. */
typedef enum { PA_F16 = 1, PA_Q4_0 = 2, PA_Q8_0 = 8 } pa_type;

/* Number types of rows outside the pools (queries, outputs, projections),
 * numbered as ggml numbers them. */
typedef enum { PA_DT_F32 = 0, PA_DT_F16 = 1, PA_DT_BF16 = 30 } pa_dtype;

typedef struct {
  uint32_t n_blocks;   /* blocks in the pool, 1 .. 2^31-1 */
  uint32_t page_size;  /* positions (rows) per block, a multiple of 16 */
  uint32_t n_kv_heads; /* KV heads per row */
  uint32_t head_dim;   /* values per row; 256 */
  int32_t k_type;      /* pa_type of K rows */
  int32_t v_type;      /* pa_type of V rows */
} pa_pool_desc;

/* A block handle: (generation << 32) | block index. */
typedef uint64_t pa_block;

typedef struct pa_pool pa_pool;

/* ------------------------------------------------------------------ allocator
 * lucebox PR #555, Summary: an exact allocator of fixed-size K/V blocks whose
 * allocations are transactional, whose stale handles are detected and whose
 * releases take effect at once.  Host metadata only; the K and V pools themselves are device buffers of
 * pa_pool_bytes() bytes that the caller allocates.  Thread-safe (one mutex
 * per pool). */

/* Create a pool's allocator state.  PA_ERR_INVALID for a zero or oversize
 * field, PA_ERR_UNSUPPORTED for an unknown type, a head_dim other than 256 or
 * a page_size that is not a multiple of 16.  *out is owned by the caller and
 * freed with pa_pool_destroy. */
pa_status pa_pool_create(const pa_pool_desc* desc, pa_pool** out);

/* Free the allocator state (not the device pools).  NULL is ignored. */
void pa_pool_destroy(pa_pool* pool);

/* Copy of the descriptor the pool was created with. */
pa_status pa_pool_get_desc(const pa_pool* pool, pa_pool_desc* out);

/* Bytes of one stored row of `head_dim` values of `type`; 0 if unsupported. */
size_t pa_row_bytes(int32_t type, uint32_t head_dim);

/* Bytes of the device K pool (which = 0) or V pool (which = 1):
 * n_blocks * n_kv_heads * page_size * row_bytes.  0 for a bad argument. */
size_t pa_pool_bytes(const pa_pool* pool, int which);

/* Allocate n blocks, all or nothing.  Writes n handles to out (host).
 * Blocks come from a LIFO free list that starts as 0, 1, 2, ...; a block
 * released earlier is handed out again first.  PA_ERR_OOM (pool unchanged)
 * when fewer than n blocks are free. */
pa_status pa_alloc_blocks(pa_pool* pool, uint32_t n, pa_block* out);

/* Release n handles (host array), all or nothing, immediately: the blocks
 * are free on return and the handles become stale (the block's generation
 * is bumped).  PA_ERR_STALE, with nothing released, if any handle is out of
 * range, not allocated, of an old generation, or repeated in the call.  The
 * caller must make sure no queued kernel still reads or writes the blocks. */
pa_status pa_release(pa_pool* pool, const pa_block* handles, uint32_t n);

/* Block index of a live handle, for building block tables.  PA_ERR_STALE
 * for a handle that is not live. */
pa_status pa_block_index(const pa_pool* pool, pa_block handle, int32_t* idx);

/* Number of free blocks. */
uint32_t pa_pool_free_count(const pa_pool* pool);

/* ------------------------------------------------------------------ prefix sharing
 * Prefix blocks shared between sequences by reference count, with
 * copy-on-write (lucebox PR #555, roadmap item 6).  A block holds one
 * reference after pa_alloc_blocks; pa_release drops one reference per
 * occurrence of a handle and frees the block (bumping its generation) when
 * the count reaches 0, so a handle may occur in one pa_release call as many
 * times as it has references (more is PA_ERR_STALE, nothing released).
 * Thread-safe; every call checks everything before it commits. */

/* Take one more reference per occurrence of each handle (a sequence that
 * forks another puts the same blocks in its own table).  PA_ERR_STALE for a
 * handle that is not live: nothing changes. */
pa_status pa_share_blocks(pa_pool* pool, const pa_block* handles, uint32_t n);

/* Reference count of a live block (PA_ERR_STALE otherwise). */
pa_status pa_block_refcount(const pa_pool* pool, pa_block handle, uint32_t* count);

/* Prepare blocks for writing.  Taking the handles in order, a block held by
 * one reference comes back unchanged in out[i]; a shared block loses the
 * caller's reference and out[i] is a freshly allocated block, with the pair
 * (old index, new index) appended to copy_src / copy_dst (host arrays of
 * capacity n; *n_copies pairs written).  The caller then copies the listed
 * blocks on the device (pa_copy_blocks) before writing to them, and puts
 * out[i] in its table.  PA_ERR_STALE (a handle not live) or PA_ERR_OOM (too
 * few free blocks for the copies): nothing changes. */
pa_status pa_cow_blocks(pa_pool* pool, const pa_block* handles, uint32_t n, pa_block* out,
                        int32_t* copy_src, int32_t* copy_dst, uint32_t* n_copies);

/* Device half of copy-on-write: copy whole blocks (every KV head's page of K
 * and of V) from block src[i] to block dst[i], i < n.  src, dst: device int32
 * arrays.  A pair with an index outside the pool is skipped and sets
 * *err = PA_ERR_BOUNDS.  Pairs that write one block twice race. */
pa_status pa_copy_blocks(const pa_pool* pool, void* k_pool, void* v_pool, const int32_t* src,
                         const int32_t* dst, uint32_t n, int32_t* err, pa_stream_t stream);

/* Bring the live blocks to the front of the pool: with m of them, those at m or behind
 * move, in order, into the free places before m (the lowest first).  Writes a
 * pair of handles for each into old_handles (ascending by index) and new_handles
 * (host arrays of `capacity`), *n_moves of them; a moved block keeps its references, its old
 * handle is stale from then on.  The free blocks are the last n_blocks - m, handed out from m
 * on.  The caller puts the new handles in the old ones' place and moves the rows
 * (pa_move_blocks, whose src and dst are the handles' indices: their low 32
 * bits) before the blocks are used again.  PA_ERR_INVALID when capacity is less than *n_moves
 * (which is written): nothing changes. */
pa_status pa_compact_blocks(pa_pool* pool, uint32_t capacity, pa_block* old_handles, pa_block* new_handles,
                            uint32_t* n_moves);

/* Device half of a compaction: copy whole blocks from src[i] to dst[i], i < n, as
 * pa_copy_blocks, and rewrite tables in the same launch: table_out[e] is dst[i]
 * where table[e] is a src[i], else table[e] (whatever it is), e < n_entries.
 * src, dst, table, table_out: device int32; table_out may be table (other overlaps
 * race), n_entries 0 for none.  With entries, src ascends (*err = PA_ERR_INVALID
 * where it does not, and then the tables are not to be used).  No block may be
 * both in src and in dst: such pairs race. */
pa_status pa_move_blocks(const pa_pool* pool, void* k_pool, void* v_pool, const int32_t* src, const int32_t* dst,
                         uint32_t n, const int32_t* table, int32_t* table_out, uint64_t n_entries, int32_t* err,
                         pa_stream_t stream);

/* ------------------------------------------------------------------ append
 * New rows are uploaded once, packed, and a kernel scatters them into their
 * page slots (colibri PR #372, Summary: one packed transfer of the newly
 * appended rows plus a scatter kernel; llama.cpp fork PR #2, KV-pool commit:
 * cache writes reach pool rows through index tensors).
 *
 * k_rows, v_rows: device, packed [n_rows][n_kv_heads][row_bytes], already in
 *                 storage format; 16-byte aligned.
 * row_seq, row_pos: device int32 [n_rows]: sequence and position of each row.
 *                 Positions are appended in order with no gap (a row is
 *                 written at the sequence's current length, lucebox PR #555,
 *                 first-token bookkeeping fix); the kernel does not check it.
 * block_table:    device int32 [n_seq][table_stride].
 * k_pool, v_pool: device pools (pa_pool_bytes each), 16-byte aligned.
 * err:            device int32 error word.
 * A row whose sequence, page or table entry is out of range is skipped and
 * sets *err = PA_ERR_BOUNDS; no out-of-range address is written.  The copy
 * is byte-exact.  Rows with the same (seq, pos) in one call race. */
pa_status pa_append_rows(const pa_pool* pool, void* k_pool, void* v_pool, const void* k_rows,
                         const void* v_rows, const int32_t* row_seq, const int32_t* row_pos,
                         uint32_t n_rows, const int32_t* block_table, uint32_t table_stride,
                         uint32_t n_seq, int32_t* err, pa_stream_t stream);

/* Quantise on append: the same scatter, from rows given as IEEE binary16
 * values, converted to the pool's K and V formats on the way in (a cache
 * write into quantised pages, as the llama.cpp fork's pool writes do; the
 * pages print no rule, so the rule is ggml's reference quantiser, a
 * reading).  Per 32-value block, in float32 with every operation rounded on
 * its own (no fused multiply-add):
 *   Q8_0: d = max|x| / 127, id = d ? 1/d : 0, q = round-half-away(x * id);
 *   Q4_0: m = the x of largest |x| (the first on ties), d = m / -8,
 *         id = d ? 1/d : 0, q = min(15, trunc(x * id + 8.5));
 *   both store fp16(d), rounded to nearest even; F16 pools take the values
 *   as they are.
 * k_rows, v_rows: device binary16 [n_rows][n_kv_heads][head_dim], 16-byte
 * aligned, finite values.  Everything else as pa_append_rows; the bytes
 * written equal those of quantising each block with the rule above and
 * appending the result with pa_append_rows. */
pa_status pa_append_rows_f16(const pa_pool* pool, void* k_pool, void* v_pool, const uint16_t* k_rows,
                             const uint16_t* v_rows, const int32_t* row_seq, const int32_t* row_pos,
                             uint32_t n_rows, const int32_t* block_table, uint32_t table_stride,
                             uint32_t n_seq, int32_t* err, pa_stream_t stream);

/* ------------------------------------------------------------------ norm and rotation
 * The pages describe no counterpart of the calls from here to "decode"; they
 * exist for users of this library.
 *
 * What a model does to the query and key heads of a projection before the
 * cache sees them.  For a head x of head_dim = 256 values at position p:
 *   norm      (only with a weight w) x_i <- x_i (w_i + weight_offset) /
 *             sqrt(mean(x^2) + eps);
 *   rotation  for pair i of rot_dim / 2: (a, b) <- (a c - b s, b c + a s) with
 *             c = attn_factor cos(p inv_freq[i]), s = attn_factor
 *             sin(p inv_freq[i]); the pair is values (i, i + rot_dim / 2), or
 *             (2i, 2i + 1) when interleaved.  Values from rot_dim on stay.
 * Arithmetic is fp32; the angle is reduced in 64-bit fixed point, so far
 * positions lose nothing.  Positions are any int32. */
typedef struct {
  uint32_t rot_dim;     /* rotated leading values of a head: a multiple of 16, 0 .. 256 */
  int32_t interleaved;  /* 0 or 1 */
  float eps;            /* >= 0 */
  float weight_offset;  /* added to every weight (1 where weights are stored as w - 1) */
  float attn_factor;    /* on cosines and sines; 1 for a plain rotation */
  double inv_freq[128]; /* radians per position of pair i; the first rot_dim / 2 are read, finite */
} pa_rope_desc;

/* Norm and rotation of query and key heads in one launch.
 *
 * rope:     host; copied by the call.
 * q, k:     device rows of n_q_heads / n_kv_heads heads of 256 values of
 *           in_type (a pa_dtype); q_stride and k_stride are elements between
 *           rows (at least heads * 256, a multiple of 16 bytes), so q and k may
 *           be parts of one projection.  A pointer is NULL exactly when its head
 *           count is 0; at most 4096 heads each.
 * q_weight, k_weight: device [256] of w_type, shared by the heads, or NULL: not
 *           normalised, only rotated.
 * row_pos:  device int32 [n_rows].
 * q_out, k_out: device rows of out_type with their own strides.  An output may
 *           be its input (same type and stride); other overlaps race.
 * Every pointer 16-byte aligned (row_pos 4).  PA_ERR_INVALID or
 * PA_ERR_UNSUPPORTED (a type, a rot_dim) before anything is launched. */
pa_status pa_norm_rope(const pa_rope_desc* rope, const void* q, int64_t q_stride, uint32_t n_q_heads, const void* k,
                       int64_t k_stride, uint32_t n_kv_heads, int32_t in_type, const void* q_weight,
                       const void* k_weight, int32_t w_type, const int32_t* row_pos, uint32_t n_rows, void* q_out,
                       int64_t q_out_stride, void* k_out, int64_t k_out_stride, int32_t out_type,
                       pa_stream_t stream);

/* Append with the norm and rotation on the way: rows straight from the
 * projection.  Keys are normalised (k_weight), rotated and stored in the
 * pool's K format, values stored in its V format as they are, both quantised
 * from fp32 by the rule of pa_append_rows_f16 (an F16 pool rounds once, to
 * nearest even), and, if q is given, queries normalised, rotated and written
 * to q_out -- one launch for all that stands between a projection and the
 * decode.
 *
 * k_rows, v_rows: device rows of n_kv_heads heads of in_type, strides as
 *           above; q, q_stride, n_q_heads, q_weight, q_out, q_out_stride,
 *           q_out_type as in pa_norm_rope (q and q_out NULL and n_q_heads 0 for
 *           none).
 * row_seq, row_pos, block_table, pools, err: as pa_append_rows; a row's
 *           position is also its rotation's.  A row whose sequence, page or
 *           table entry is out of range (the padding of a batch: row_seq -1) is
 *           not stored and sets *err = PA_ERR_BOUNDS; its query is still
 *           written.  Rows with the same (seq, pos) in one call race.  Values
 *           are finite, and in the range of their format: up to 65504 in F16, 65504
 *           times 127 in Q8_0 and times 8 in Q4_0 (past it they are stored as
 *           infinite). */
pa_status pa_append_rows_rope(const pa_pool* pool, void* k_pool, void* v_pool, const pa_rope_desc* rope,
                              const void* k_rows, int64_t k_stride, const void* v_rows, int64_t v_stride,
                              int32_t in_type, const void* k_weight, int32_t w_type, const void* q, int64_t q_stride,
                              uint32_t n_q_heads, const void* q_weight, void* q_out, int64_t q_out_stride,
                              int32_t q_out_type, const int32_t* row_seq, const int32_t* row_pos, uint32_t n_rows,
                              const int32_t* block_table, uint32_t table_stride, uint32_t n_seq, int32_t* err,
                              pa_stream_t stream);

/* Rows of the cache as floating values: the inverse of an append, for a
 * prompt whose attention runs elsewhere, and for looking at a cache.
 * k_out, v_out: device [n_rows][n_kv_heads][256] of out_type, 16-byte aligned;
 * either may be NULL (not both).  A stored value is scale * quant in fp32,
 * rounded once to out_type.  row_seq, row_pos, block_table, pools, err: as
 * pa_append_rows; a row out of range reads as zeros and sets *err =
 * PA_ERR_BOUNDS.  Rows may repeat. */
pa_status pa_read_rows(const pa_pool* pool, const void* k_pool, const void* v_pool, const int32_t* row_seq,
                       const int32_t* row_pos, uint32_t n_rows, const int32_t* block_table, uint32_t table_stride,
                       uint32_t n_seq, void* k_out, void* v_out, int32_t out_type, int32_t* err, pa_stream_t stream);

/* Rows of the cache moved to other places: row i of sequence src_seq[i], position
 * src_pos[i] (through src_table) to dst_seq[i], dst_pos[i] (through dst_table,
 * which may be src_table), K and V.  For dropping the middle of a context, keeping the accepted
 * ones of drafted tokens, giving a fork its own copy of a page's first rows, or changing the
 * frequencies of a live cache.
 *
 * All rows are read before any is written, so that rows may land where others come
 * from.  Two rows with the same destination race.  disjoint 1: the caller vouches
 * that no row's destination is another row's source (its own is fine); one launch less.
 *
 * rope:     host, or NULL: rows are copied byte for byte.  Else keys are turned by
 *           the difference of dst_pos's angles under rope and src_pos's under rope_from
 *           (NULL: rope), and multiplied by the ratio of their attn_factors where they
 *           are turned; eps and weight_offset are not used.  rope_from has rope's
 *           rot_dim and interleaved.  A turned key is dequantised, turned in fp32 and stored by
 *           the rule of pa_append_rows_f16 in blocks of 32 values; blocks from rot_dim
 *           on, keys whose position and rope stay, and V are copied byte for byte.
 * src_table, dst_table: device int32 [n_seq][stride] each.
 * workspace: 16-byte aligned scratch of ws_bytes >= pa_move_rows_workspace_size(); not
 *           used with disjoint.
 * A row of which one place is out of range is not moved and sets *err = PA_ERR_BOUNDS. */
pa_status pa_move_rows(const pa_pool* pool, void* k_pool, void* v_pool, const pa_rope_desc* rope,
                       const pa_rope_desc* rope_from, const int32_t* src_seq, const int32_t* src_pos,
                       const int32_t* dst_seq, const int32_t* dst_pos, uint32_t n_rows, const int32_t* src_table,
                       uint32_t src_stride, uint32_t src_n_seq, const int32_t* dst_table, uint32_t dst_stride,
                       uint32_t dst_n_seq, int32_t disjoint, void* workspace, size_t ws_bytes, int32_t* err,
                       pa_stream_t stream);

/* Scratch bytes pa_move_rows needs for n_rows rows that are not disjoint: 0 while they are few
 * (64 rows of 4 KV heads), else as many as the rows have. */
size_t pa_move_rows_workspace_size(const pa_pool* pool, uint32_t n_rows);

/* ------------------------------------------------------------------ decode
 * Single-step GQA decode attention over a paged cache: split-K flash decoding
 * through a block table, with a log-sum-exp merge of the splits (llama.cpp
 * fork PR #2, split-K decode commit: head size 256, GQA 6, one to four query
 * tokens for speculative verification, a later commit taking batches of up
 * to eight tokens, and the commit on ubatches of more than eight tokens, which
 * gives paged K/V of up to 96 query tokens the decode kernel's row tiles;
 * lucebox PR #555, Summary: a numerically stable merge of split softmaxes).
 * One to eight query tokens run the decode kernels; nine to 96 run row tiles
 * (128 query rows of one KV head, K and V dequantised once per tile into
 * binary16).
 *
 * For sequence s with L = seq_lens[s] cached rows (the n_qtok new rows
 * included), query token t in [0, n_qtok) sits at position L - n_qtok + t and
 * attends to keys 0 .. L - n_qtok + t.  Query head h reads KV head
 * h / (n_q_heads / n_kv_heads).  Logits are scale * q.k; the output is the
 * softmax-weighted sum of V rows, and lse the natural-log log-sum-exp of the
 * scaled, masked logits (llama.cpp fork PR #2, LSE commit: the row maximum
 * plus the log of the row sum).  A row with no visible key would give
 * out = 0 and lse = -inf.
 *
 * Supported: head_dim 256, n_q_heads / n_kv_heads = 6, n_qtok 1..96, K and V
 * each F16, Q4_0 or Q8_0 (PA_ERR_UNSUPPORTED otherwise).
 *
 * q:            device fp32 [n_seq][n_qtok][n_q_heads][head_dim], 16-byte aligned.
 * k_pool/v_pool: device pools laid out as described at the top.
 * block_table:  device int32 [n_seq][table_stride]; only entries for pages
 *               holding positions < seq_lens[s] are read.
 * seq_lens_dev / seq_lens_host: the same int32 [n_seq] lengths on the device
 *               and on the host.  Each host length must be >= n_qtok and
 *               <= table_stride * page_size (PA_ERR_INVALID otherwise).  The
 *               host copy alone sizes the launch and drives every read: the
 *               kernels walk tiles, read table entries and mask keys from it
 *               (it travels in the launch parameters).  The device copy is
 *               only compared with it: a sequence whose device length differs
 *               (whatever its value) gives out = 0 and lse = -inf for all its
 *               rows and sets *err = PA_ERR_BOUNDS (lucebox PR #555,
 *               Validation: corrupt bounds must be caught, not followed).
 * out:          device fp32 [n_seq][n_qtok][n_q_heads][head_dim], 16-byte aligned.
 * lse:          device fp32 [n_seq][n_qtok][n_q_heads], or NULL.
 * workspace:    device scratch of ws_bytes >= pa_decode_workspace_size(),
 *               256-byte aligned; its contents need no initialisation and
 *               are garbage afterwards.  Concurrent calls need separate
 *               workspaces.
 * err:          device int32 error word.  A table entry outside [0, n_blocks)
 *               sets *err = PA_ERR_BOUNDS; the rows it would have supplied are
 *               read as zeros (no out-of-range read).
 * The result depends only on the inputs and on seq_lens (not on page size or
 * page placement): a paged cache and an identity-table cache holding the same
 * rows give bit-identical outputs.
 *
 * Launches: the split kernel, then (when a sequence is split) the merge
 * kernel, on `stream`.  Both are programmatic dependent launches: each may
 * start while the previous kernel on the stream finishes, but waits for it to
 * complete before reading anything, so stream order is kept.  One launch pair
 * takes at most 128 sequences; a larger batch runs as consecutive sub-batches
 * of 128 (in order, sharing the workspace), each planned on its own lengths. */
pa_status pa_decode(const pa_pool* pool, const float* q, const void* k_pool, const void* v_pool,
                    const int32_t* block_table, uint32_t table_stride, const int32_t* seq_lens_dev,
                    const int32_t* seq_lens_host, uint32_t n_seq, uint32_t n_qtok,
                    uint32_t n_q_heads, float scale, float* out, float* lse, void* workspace,
                    size_t ws_bytes, int32_t* err, pa_stream_t stream);

/* The two passes of pa_decode as separate calls, with pa_decode's arguments.
 * pa_decode_split runs the split-K pass: sequences handled by one CTA get
 * their final out/lse, the others leave split partials in `workspace`.
 * pa_decode_merge then merges those partials into out/lse.  Calling split then
 * merge on one stream, with the same arguments and workspace and nothing in
 * between that touches the workspace, is exactly pa_decode; the split lets a
 * caller time or schedule the passes separately.  Both take at most 128
 * sequences (PA_ERR_UNSUPPORTED above that, nothing launched). */
pa_status pa_decode_split(const pa_pool* pool, const float* q, const void* k_pool, const void* v_pool,
                          const int32_t* block_table, uint32_t table_stride, const int32_t* seq_lens_dev,
                          const int32_t* seq_lens_host, uint32_t n_seq, uint32_t n_qtok, uint32_t n_q_heads,
                          float scale, float* out, float* lse, void* workspace, size_t ws_bytes, int32_t* err,
                          pa_stream_t stream);
pa_status pa_decode_merge(const pa_pool* pool, const float* q, const void* k_pool, const void* v_pool,
                          const int32_t* block_table, uint32_t table_stride, const int32_t* seq_lens_dev,
                          const int32_t* seq_lens_host, uint32_t n_seq, uint32_t n_qtok, uint32_t n_q_heads,
                          float scale, float* out, float* lse, void* workspace, size_t ws_bytes, int32_t* err,
                          pa_stream_t stream);

/* Scratch bytes pa_decode needs for up to n_seq sequences of n_qtok query
 * tokens on CUDA device `device`, whatever their lengths.  Reported up front
 * so that a caller with a fixed memory budget can reserve it before the first
 * step instead of failing in the middle of one (llama.cpp fork PR #2, scratch
 * commit).  0 for an unsupported shape. */
size_t pa_decode_workspace_size(const pa_pool* pool, uint32_t n_seq, uint32_t n_qtok, int device);

/* How pa_decode would split this batch (lucebox PR #555, Summary: the
 * context is split across the GPU by occupancy, adaptively for long
 * contexts): *n_ctas decode CTAs (the largest grid over the sub-batches),
 * *n_tiles key tiles of `*tile_keys` keys each in total, and *n_partials
 * split partials (pieces).  The tiles, laid end to end by (sequence, KV
 * head), are cut into contiguous per-CTA ranges: of equal tile counts for one
 * query token and for row tiles; for 2-8 tokens of equal cost, where the first
 * tile of each (sequence, KV head) counts two tiles more, whenever every range
 * still gets a tile.  Host only, nothing launched; for tests and tools.
 * PA_ERR_INVALID for a null pool or lengths, n_seq = 0 or a length below
 * n_qtok; PA_ERR_UNSUPPORTED for a shape pa_decode does not take. */
pa_status pa_decode_plan(const pa_pool* pool, const int32_t* seq_lens_host, uint32_t n_seq,
                         uint32_t n_qtok, int device, uint32_t* n_ctas, uint32_t* n_tiles,
                         uint32_t* tile_keys, uint32_t* n_partials);

/* ------------------------------------------------------------------ decode without allocation
 * The pages describe no counterpart of this call; it exists for users of this
 * library.  pa_decode_noalloc is pa_decode without the workspace arguments:
 * its scratch is a fixed array of PA_NOALLOC_SCRATCH_BYTES bytes that the
 * library reserves (as a static device variable) on every GPU that loads it,
 * until the process exits.  It is meant for callers that cannot allocate
 * device memory: code running under a memory budget fixed at start-up, hot
 * loops that must avoid cudaMalloc's implicit synchronisation, plain C callers
 * without an allocator.  It allocates nothing and calls no allocating routine.
 *
 * Arguments, results and device errors are those of pa_decode.  A batch whose
 * workspace (pa_decode_workspace_size) exceeds PA_NOALLOC_SCRATCH_BYTES is
 * refused with PA_ERR_UNSUPPORTED before anything is launched.  The first call
 * on a device looks up the array's device address (once per device); make
 * that first call before any stream capture.  All calls share the one array:
 * calls whose work overlaps on the GPU race and must be serialised by the
 * caller.  The array keeps the previous call's contents; the call needs no
 * clearing. */
#define PA_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)

pa_status pa_decode_noalloc(const pa_pool* pool, const float* q, const void* k_pool, const void* v_pool,
                            const int32_t* block_table, uint32_t table_stride, const int32_t* seq_lens_dev,
                            const int32_t* seq_lens_host, uint32_t n_seq, uint32_t n_qtok, uint32_t n_q_heads,
                            float scale, float* out, float* lse, int32_t* err, pa_stream_t stream);

/* ------------------------------------------------------------------ decode with shared prefixes
 * The pages describe no counterpart of this call beyond the shared blocks
 * themselves; it exists for users of this library.
 *
 * pa_decode for a batch whose sequences share prefixes: the batch is cut into
 * n_groups runs of consecutive sequences (group_sizes: host, each >= 1, summing
 * to n_seq), and the first prefix_lens[g] positions (host, >= 0) of all the
 * sequences of group g hold the same rows.  Those rows are read and multiplied
 * once for the whole group, through the table row of its first sequence; the
 * rest of each sequence as in pa_decode; the parts are merged by log-sum-exp.
 * The caller vouches for the shared rows (with pa_share_blocks the tables hold
 * the same blocks; a page that the prefix ends in may be each sequence's own
 * copy).  The result is that of pa_decode on the same batch, up to rounding;
 * a prefix length of 0 shares nothing.
 *
 * When it pays, GPU time against pa_decode on the same batch: from two sequences
 * with 1000 shared rows on in quantised pools (8.1 against 9.3 us), from four in F16
 * (8.4 against 9.1), the more the longer the prefix and the more sequences (8 of
 * 32768 + 1024 rows in Q4_0: 22.9 against 56); with four query tokens nearly always
 * (8 of 500 + 100 rows: 11.8 against 16.1).  With one token, shorter prefixes are even,
 * and sequences that share nothing take the same within an eighth, either way.
 *
 * q, out:   device [n_seq][n_qtok][n_q_heads][head_dim] of q_type / out_type (a
 *           pa_dtype), 16-byte aligned.
 *
 * Precision and range.  Queries of fp32 and bfloat16 are rounded to binary16 (fp32
 * as in pa_decode), and so is quantised K (scale * quant), which pa_decode keeps
 * exact: a logit is off by 2^-11 |q| |k| scale at most for each of the two that is
 * rounded.  Where that is not small against 1 (logits of hundreds), pa_decode is the
 * call to make.  V (scale * quant) and the softmax weights are rounded to binary16,
 * sums are fp32.  Stored keys may be of any size that a pool holds; a stored V value
 * past 65504 is infinite.  A row with a NaN logit (a NaN in its query or in a key that
 * it sees) is NaN, its lse too; so is a row with a query value of fp32 or bfloat16
 * that rounds past 65504.
 *
 * prefix_lens: at most seq_lens_host - n_qtok of every sequence of the group
 *           (PA_ERR_INVALID otherwise): the new tokens are each sequence's own.
 * workspace: ws_bytes >= pa_decode_prefix_workspace_size(), 256-byte aligned.
 * Everything else (lengths, tables, masks, lse, errors, supported shapes) as
 * pa_decode.  Launches as pa_decode; sub-batches of at most 256 sequences,
 * a group cut by a sub-batch's end being read once in each. */
pa_status pa_decode_prefix(const pa_pool* pool, const void* q, int32_t q_type, const void* k_pool,
                           const void* v_pool, const int32_t* block_table, uint32_t table_stride,
                           const int32_t* seq_lens_dev, const int32_t* seq_lens_host, uint32_t n_seq,
                           const uint32_t* group_sizes, const int32_t* prefix_lens, uint32_t n_groups,
                           uint32_t n_qtok, uint32_t n_q_heads, float scale, void* out, int32_t out_type, float* lse,
                           void* workspace, size_t ws_bytes, int32_t* err, pa_stream_t stream);

/* Scratch bytes pa_decode_prefix needs for up to n_seq sequences in up to
 * n_groups groups of n_qtok query tokens on CUDA device `device`, whatever their
 * lengths and the groups' sizes.  0 for an unsupported shape. */
size_t pa_decode_prefix_workspace_size(const pa_pool* pool, uint32_t n_seq, uint32_t n_groups, uint32_t n_qtok,
                                       int device);

/* ------------------------------------------------------------------ attention over a window
 * The pages describe no counterpart of this call; it exists for users of this library.
 *
 * Causal attention of each sequence's newest tokens over the cache, for ragged batches:
 * sequence s has n_new[s] >= 0 of them, one (a decode step), a few (verification) or many
 * (a chunk of prompt, a whole one), at positions L - n_new[s] .. L - 1 of its L =
 * seq_lens[s] cached rows.  The token at position p attends to the keys x <= p with
 * x > p - window (the window holds its own key) or x < sinks (first keys that stay
 * visible); window 0 stands for none: all keys up to p.
 *
 * q, out:   device rows of n_q_heads heads of 256 values, of q_type / out_type (a
 *           pa_dtype), a row per token: the first sequence's n_new[0], then the next's.
 *           q_stride and out_stride are values between rows (at least heads * 256, a
 *           multiple of 16 bytes), so q may be a part of a projection.  Rows after
 *           the last sequence's are neither read nor written.
 * lse:      device fp32 [tokens][n_q_heads], or NULL.
 * n_new:    host int32 [n_seq]; n_new[s] <= L.  seq_lens_dev, seq_lens_host: as pa_decode
 *           (the host's drive every read; a sequence whose device length is another gives
 *           out = 0, lse = -inf and *err = PA_ERR_BOUNDS).
 * block_table: only entries for pages that hold a row group (16 rows) with a key that
 *           some new token sees are read, so the pages outside window and sinks may
 *           have been released.  An entry outside the pool: as pa_decode.
 * workspace: ws_bytes >= pa_attend_window_workspace_size(), 256-byte aligned; contents as
 *           pa_decode's.
 *
 * Precision and range: as pa_decode_prefix, whose arithmetic it is: Q of fp32 and bfloat16,
 * quantised K, V and the softmax weights are each rounded to binary16 once, whatever out_type is;
 * sums are fp32.  Single tokens of batches that fill the device, with Q8_0 keys and quantised values, lose
 * less (K is exact there, the weights are in two parts).  So a token's last bits depend on how many
 * sequences and new tokens stand beside it.  No form of this call keeps all keys exact: for logits of
 * hundreds pa_decode is the call to make, which has no window.  It is also the faster one for single
 * tokens over long contexts that are seen whole (8 x 8192 keys: Q4_0 23.6 us against 30.1, Q8_0
 * 30.6 against 32.7, F16 45.4 against 48.5; 8 x 32768 of Q4_0 57 against 90).
 *
 * An infinite or NaN value of V (a stored one past 65504 is infinite) in a row that one of the
 * tokens sees can also reach others of the same sequence that do not see it: those whose window
 * or own position lies up to 64 tokens from it.  In a row that no token sees it has no effect, and K's
 * reach nobody who does not see them.
 *
 * Launches: one for the sequences of fewer than 64 new tokens (448 times 64 query rows, or 256
 * single tokens, at a time), and a merge when a (64 query rows, KV head) is shared by
 * CTAs; for those of more, one that turns their keys into binary16 (128 sequences at a time),
 * and one over 256 times 256 query rows at a time, with a merge when one of these is shared.  All are
 * programmatic dependent launches (pa_decode). */
pa_status pa_attend_window(const pa_pool* pool, const void* q, int64_t q_stride, int32_t q_type, const void* k_pool,
                           const void* v_pool, const int32_t* block_table, uint32_t table_stride,
                           const int32_t* seq_lens_dev, const int32_t* seq_lens_host, const int32_t* n_new,
                           uint32_t n_seq, uint32_t n_q_heads, uint32_t window, uint32_t sinks, float scale, void* out,
                           int64_t out_stride, int32_t out_type, float* lse, void* workspace, size_t ws_bytes,
                           int32_t* err, pa_stream_t stream);

/* Scratch bytes pa_attend_window needs for these lengths on CUDA device `device`; more new
 * tokens, longer sequences and windows, more first keys, or more sequences need no less, so that a
 * caller may size it once for the largest.  Sequences of 64 new tokens and more take 16 KB for
 * each KV head and 16 keys that they see, and up to three times 16 KB more for each head (131072 keys
 * of 4 heads without a window: 537 MB).  0 for an unsupported pool or lengths that the call refuses. */
size_t pa_attend_window_workspace_size(const pa_pool* pool, const int32_t* seq_lens_host, const int32_t* n_new,
                                       uint32_t n_seq, uint32_t window, uint32_t sinks, int device);

/* ------------------------------------------------------------------ errors */

/* Device-detected failures are reported, not trapped (lucebox PR #555,
 * Validation: bad block-table bounds are guarded against; llama.cpp fork
 * PR #2, SDMA copy commit: a stalled wait fails instead of hanging).  The
 * kernels record the first failure in the caller's int32 word.
 *
 * pa_get_error: synchronise `stream`, read the device error word, reset it
 * to 0 and return it as a pa_status.  PA_ERR_INVALID for a null word,
 * PA_ERR_CUDA if the read itself fails or the word holds no status. */
pa_status pa_get_error(int32_t* err, pa_stream_t stream);

/* Static, human-readable name of a status (the same failure classes; a
 * value outside pa_status gives "PA_ERR_UNKNOWN").  Never NULL. */
const char* pa_status_string(pa_status s);

/* Runs one kernel that waits, with the same bounded wait the decode kernel
 * uses, on a shared-memory barrier that nothing ever completes; after about
 * timeout_us microseconds the wait gives up and sets *err = PA_ERR_TIMEOUT.
 * Exists so tests can check the expiry path without hanging a GPU. */
pa_status pa_selftest_wait_timeout(uint32_t timeout_us, int32_t* err, pa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_H */
