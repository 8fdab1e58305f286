/*
 * tp3d_paged.h - C ABI of the paged key/value cache: serving the GPT decoder
 * layer of tp3d.h.
 *
 * The layer's attention (tp3d_layer_fwd) computes whole sequences.  A server
 * instead keeps the keys and values of earlier tokens and computes only the
 * new ones.  The cache is a pool of fixed-size pages; each request owns the
 * pages listed in its row of a block table, so requests of any length share
 * the pool without moving.  One step of a server is:
 *   tp3d_paged_plan   lengths -> pages taken from the free list, block table
 *                     rows, the slot and position of every new token;
 *   (the layer's QKV product, tp3d_linear)
 *   tp3d_paged_store  K and V of the new tokens -> their slots
 *                     (tp3d_paged_rope_store: heads normed and turned by
 *                     position on the way);
 *   tp3d_paged_attn   attention of the new tokens over the cache
 *                     (tp3d_paged_attn_window: over a sliding window and a
 *                     few first tokens).
 * Between steps pages are shared, given back and moved: tp3d_paged_fork,
 * tp3d_paged_free, tp3d_paged_compact, and tp3d_paged_copy for the contents.
 * Everything a step depends on stays on the device: no call reads a length
 * back, and a captured step replays with new lengths in the same buffers.
 *
 * Notation: request b has kv_b tokens in the cache, the last n_b of them new;
 * row q_start_b + j of Q is its new token j at position kv_b - n_b + j.
 *
 * Ownership, streams and errors are those of tp3d.h: the caller allocates
 * everything, calls are asynchronous on the given stream, arguments are
 * validated on the host before anything is launched, and calls of one
 * context must not run concurrently on different streams.  What only the
 * device can see is bounds-checked there: a length, page or slot that does
 * not fit raises TP3D_EPAGES (tp3d_sync_status reports it), and nothing is
 * read or written out of bounds.
 */
#ifndef TP3D_PAGED_H
#define TP3D_PAGED_H

#include "tp3d.h"
#include "tp3d_rope.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The cache of one layer: K and V pools of the same shape.  The head_dim
 * elements of (page p, token t, head h) start at element
 *   p * page_stride + t * token_stride + h * head_stride
 * of `k` and of `v`, so both page layouts (tokens or heads outermost inside a
 * page) are strides.  Pools may pass 2^32 elements.
 *   dtype     TP3D_BF16 (else TP3D_EDTYPE)
 *   head_dim  64 or 128, as the layer (else TP3D_EUNSUPPORTED)
 *   page      tokens per page: a power of two, 16 to 4096 (else
 *             TP3D_EUNSUPPORTED)
 *   k, v      16-byte aligned, strides multiples of 8 elements (else
 *             TP3D_EALIGN), positive, and below 2^39 (else TP3D_EUNSUPPORTED);
 *             that rows do not overlap is the caller's to keep              */
typedef struct {
  int32_t dtype, kv_heads, head_dim, page;
  int64_t pages;
  int64_t page_stride, token_stride, head_stride;
  void *k, *v;
} tp3d_kv_cache;

/* The requests of one step, in device memory.
 *   q_start      requests + 1 int32: exclusive sums of the new tokens
 *   kv_len       requests int32: tokens in the cache, the new ones included
 *   block_table  requests x table_width int32, dense rows: page of tokens
 *                [i * page, +page) at column i.  Columns past
 *                ceil(kv_b / page) are never used.
 *   tokens       rows of Q and O (>= q_start[requests])
 *   max_new      an upper bound on any request's new tokens known to the
 *                host, or <= 0 for none: it only selects the kernels to
 *                launch (a smaller bound than the truth leaves the longer
 *                requests' rows unwritten and raises TP3D_EPAGES)            */
typedef struct {
  int32_t requests, max_new;
  int64_t tokens;
  const int32_t *q_start, *kv_len, *block_table;
  int64_t table_width;
} tp3d_paged_batch;

/* Block tables and slot maps of one step from the request lengths.
 * Request b has cached[b] tokens in the cache and fresh[b] new ones:
 *   kv_len[b]   = cached[b] + fresh[b]
 *   q_start     = exclusive sums of fresh (requests + 1)
 *   block_table columns [ceil(cached/page), ceil(kv/page)) of row b get pages
 *               from the free list; the others keep their contents, and
 *               column (cached - 1) / page is read when the first new token
 *               falls into that partly filled page
 *   slots[t]    = page of the token's position * page + position % page, for
 *               t < q_start[requests]; -1 up to `tokens` (tp3d_paged_store
 *               skips it, so a padded batch needs no other marking)
 *   positions[t] likewise; 0 up to `tokens`
 * The free list is a stack: page ids free_pages[0 .. *free_count), taken from
 * the top, request by request; *free_left is the count after the step.  The
 * counts are separate buffers (as kv_len and cached are), so a call can be
 * repeated or replayed.
 * A negative length, a request longer than table_width pages or 2^31 - 4097
 * tokens, a free_count outside [0, free_cap], or too few free pages or
 * `tokens` raise TP3D_EPAGES: tokens without a page then get slot -1, pages
 * not had are entered as -1, and a request whose own lengths are bad gets no
 * new tokens.
 * requests <= 16384 (else TP3D_EUNSUPPORTED); 0 is allowed.  slots 8-byte,
 * the others 4-byte aligned.                                                 */
tp3d_status tp3d_paged_plan(tp3d_ctx* ctx, int page, int requests, int64_t tokens, const int32_t* cached,
                            const int32_t* fresh, const int32_t* free_pages, int64_t free_cap,
                            const int32_t* free_count, int32_t* block_table, int64_t table_width, int32_t* q_start,
                            int32_t* kv_len, int64_t* slots, int32_t* positions, int32_t* free_left, void* stream);

/* Writes K and V of `tokens` new tokens into their slots: row t, head h is
 * read at element t * token_stride + h * head_stride of K and of V (slices of
 * the packed QKV product's rows, for example) and its bits are written to
 * slot slots[t].  A negative slot is skipped; a slot past the pool is skipped
 * and raises TP3D_EPAGES.  Of equal slots, which token's row stays is not
 * defined.                                                                   */
tp3d_status tp3d_paged_store(tp3d_ctx* ctx, const tp3d_kv_cache* cache, int64_t tokens, const void* K, const void* V,
                             int64_t token_stride, int64_t head_stride, const int64_t* slots, void* stream);

/* tp3d_paged_store with the heads normed and turned (tp3d_rope.h) in the same
 * pass: query rows Q normed and turned into Q_out (or in place), key rows K
 * normed, turned and written to their slots, value rows V written to theirs as
 * they are.  K and V: the cache's heads.  Q rows of a token are written
 * whatever its slot; slots as in tp3d_paged_store.  rope: of the cache's dtype
 * (TP3D_EDTYPE) and head_dim (TP3D_ESHAPE).  Other checks as tp3d_qk_rope and
 * tp3d_paged_store.                                                          */
tp3d_status tp3d_paged_rope_store(tp3d_ctx* ctx, const tp3d_rope* rope, const tp3d_kv_cache* cache, int64_t tokens,
                                  int heads, const void* Q, tp3d_row_strides q_strides, const void* K,
                                  tp3d_row_strides k_strides, const void* V, tp3d_row_strides v_strides,
                                  const int32_t* positions, const int64_t* slots, void* Q_out,
                                  tp3d_row_strides qo_strides, void* stream);

/* Attention of the new tokens over the cache, causal: for new token j of
 * request b and query head i (key/value head h = i / (heads / kv_heads)),
 *   O = softmax_k(scale q . k_k) V over the keys k = 0 .. kv_b - n_b + j,
 *   lse = log(sum_k exp(scale q . k_k)).
 * A row with no key (kv_b - n_b + j < 0) gets O = 0 and lse = -infinity.  Keys and
 * values past kv_b, and whatever else lies in a page, have no effect on the
 * result (NaN and infinities among it); nor has a later token's value on the
 * rows before it in its chunk.  A row that does see a value that is not finite
 * gets NaN or an infinity in its column; one whose scores are all -infinity
 * gets NaN (0 / 0) everywhere and lse = -infinity.  Q and O rows: token t, head i at
 * element t * token_stride + i * head_stride of each; O is written in bf16,
 * lse (or NULL) as float32 [tokens][heads].  Rows from q_start[requests] on
 * are not written.  A block table entry outside the pool raises TP3D_EPAGES;
 * its tokens then read as zeros.
 * Statistics and sums are fp32; the probabilities of the second product are
 * two bf16 terms (16 bits).  The result does not depend on timing: sums that several CTAs
 * contribute to are added in a fixed order.
 * Work is counted in tiles (64 keys of a request and key/value head; 128 keys
 * for 256 rows of one); a call of 2^31 tiles or more raises TP3D_EPAGES.
 * heads a multiple of kv_heads (TP3D_ESHAPE), heads / kv_heads <= 128
 * (TP3D_EUNSUPPORTED); scale finite and positive (TP3D_EINVAL); Q, O 16-byte
 * aligned, strides positive (TP3D_EINVAL) and multiples of 8 (TP3D_EALIGN).
 * `workspace`: tp3d_paged_attn_workspace_bytes bytes, 256-byte aligned,
 * contents free.                                                             */
tp3d_status tp3d_paged_attn(tp3d_ctx* ctx, const tp3d_kv_cache* cache, const tp3d_paged_batch* batch, int heads,
                            float scale, const void* Q, tp3d_row_strides q_strides, void* O,
                            tp3d_row_strides o_strides, float* lse, void* workspace, void* stream);

/* tp3d_paged_attn with a sliding window and first tokens that stay visible: the
 * row at position p = kv_b - n_b + j sees the keys k <= p with
 *   k > p - window  or  k < sinks.
 * window >= 1, sinks >= 0 (else TP3D_EINVAL); a window longer than any request
 * is tp3d_paged_attn.  Keys between the first ones and the first new row's window are
 * not read, and pages that hold nothing else may have been given back: their
 * table entries are not used.  Everything else is as in tp3d_paged_attn: keys
 * that a row does not see, their values and scores that are not finite among them,
 * have no effect on it.                                                      */
tp3d_status tp3d_paged_attn_window(tp3d_ctx* ctx, const tp3d_kv_cache* cache, const tp3d_paged_batch* batch, int heads,
                                   float scale, int64_t window, int64_t sinks, const void* Q,
                                   tp3d_row_strides q_strides, void* O, tp3d_row_strides o_strides, float* lse,
                                   void* workspace, void* stream);

/* Bytes of tp3d_paged_attn's and tp3d_paged_attn_window's workspace for this cache and head count on the
 * context's device (it does not depend on the batch); 0 for an invalid
 * argument.  Both kernels' parts of split work, for every SM: with 152 SMs 91 MB
 * for heads of 128, 46 MB for heads of 64.                                   */
size_t tp3d_paged_attn_workspace_bytes(tp3d_ctx* ctx, const tp3d_kv_cache* cache, int heads);

/* The bookkeeping of a cache's pages, for sharing, giving back and moving them.
 * One pool serves every layer whose caches use the same block tables: these
 * calls are made once, tp3d_paged_copy for each layer.
 *   page          tokens per page, as in tp3d_kv_cache
 *   rows          rows of the block table, up to 16384 (else
 *                 TP3D_EUNSUPPORTED), one for each request that can be held
 *   block_table   rows x table_width int32, dense rows; a negative entry names
 *                 no page
 *   pages         pages of the pool
 *   shares        pages int32: the rows that name a page, less one; 0 for a page
 *                 with one owner, as tp3d_paged_plan leaves those it hands out,
 *                 and for a free one
 *   free_pages    the stack of tp3d_paged_plan, free_cap >= pages entries (else
 *                 TP3D_ESHAPE)
 * All 4-byte aligned.  What the device finds not to fit raises TP3D_EPAGES, and
 * nothing is read or written out of bounds.                                  */
typedef struct {
  int32_t page, rows;
  int64_t pages, table_width, free_cap;
  int32_t *block_table, *shares, *free_pages;
} tp3d_page_pool;

/* Forks requests (samples of one prompt, beams): for i < forks, row dst[i] of
 * the table gets the first len[i] tokens of row src[i].  Whole pages are shared:
 * their entries are copied and their shares grow by one (entries that name no
 * page, behind a window, are copied alone).  A partly filled last page, which
 * both requests will write, is the fork's own: a page from the free list, whose
 * contents the caller copies,
 *   copy_from[n] -> copy_to[n], n < *copy_count,
 * in the order of the forks (tp3d_paged_copy).  The arrays have room for `forks`
 * entries each; those from *copy_count on are not written.  Entries of row dst[i] past the
 * len[i] tokens are left as they are: pages that it names there have been given
 * back before.  *free_left is the free count after the call, as in
 * tp3d_paged_plan.  A request that is cut back into a page that it shares is
 * forked to its new length before it is written.
 * A row out of range, a dst row that is another dst or a src, a length that is
 * negative or longer than the row, a last page without a valid entry, a free
 * count out of range, too few free pages, or one to be taken that is outside the
 * pool raise TP3D_EPAGES, and nothing but *copy_count = 0 and *free_left (the free
 * count, kept within [0, free_cap]) is written.  An entry of a whole page that is
 * past the pool raises TP3D_EPAGES too, but becomes -1 in row dst[i] and holds up
 * nothing else.  That the free list names no page twice, and none that a row
 * names, is the caller's to keep.  forks <= 16384 (else TP3D_EUNSUPPORTED).    */
tp3d_status tp3d_paged_fork(tp3d_ctx* ctx, const tp3d_page_pool* pool, int forks, const int32_t* src,
                            const int32_t* dst, const int32_t* len, const int32_t* free_count, int32_t* free_left,
                            int32_t* copy_from, int32_t* copy_to, int32_t* copy_count, void* stream);

/* Gives pages back: columns [first[r], end[r]) of every row r of the table are
 * set to -1 (nothing where end <= first), and each page that they named loses an
 * owner.  Pages that have lost their last join the free list above free_count,
 * the highest first, so that the lowest are taken first again; *free_left is the
 * new count.  A request that ends gives up [0, ceil(kv / page)); one that is cut
 * back, the columns past its new length; one with a sliding window (and pages of
 * first tokens that stay), those behind the window.
 * Columns out of range (that row then gives up nothing), entries past the pool,
 * a page that loses more owners than it has (it is freed once), a free_count out
 * of range (kept within [0, free_cap]), and a free list that is full raise
 * TP3D_EPAGES.  That a row names no page which is free already is the caller's to
 * keep.                                                                       */
tp3d_status tp3d_paged_free(tp3d_ctx* ctx, const tp3d_page_pool* pool, const int32_t* first, const int32_t* end,
                            const int32_t* free_count, int32_t* free_left, void* stream);

/* Draws the used pages together at the pool's start, so that its end can be
 * given up: with F = *free_count, the n-th (in ascending order) used page past
 * pages - F moves to the n-th free page below it.  Entries of columns
 * [0, ceil(kv_len[r] / page)) of each row, and the shares, follow; the free list
 * becomes pages - 1, ..., pages - F; page_map (pages int32) tells where each used
 * page is now, -1 for a free one.  The contents move by
 *   copy_from[n] -> copy_to[n], n < *copy_count,
 * (tp3d_paged_copy, before anything else is written to the cache); the arrays
 * have room for pages / 2 entries each.  Used is every page that is not in the
 * free list, whether a row names it or not.
 * A free list with an entry out of range or twice, or a free_count out of range,
 * raises TP3D_EPAGES; the tables and the list are then left as they are, page_map is
 * the identity and *copy_count 0.  So does a row's length that does not fit (its
 * entries are left as they are), and an entry past the pool or naming a free page.  */
tp3d_status tp3d_paged_compact(tp3d_ctx* ctx, const tp3d_page_pool* pool, const int32_t* kv_len,
                               const int32_t* free_count, int32_t* page_map, int32_t* copy_from, int32_t* copy_to,
                               int32_t* copy_count, void* stream);

/* Copies whole pages of a cache, keys and values: page copy_from[n] to page
 * copy_to[n] for n < min(copies, *copy_count), or n < copies with copy_count
 * NULL.  No page may be written twice, or read and written, in one call (a fork's
 * and a compaction's lists are like that).  A page outside the pool is skipped
 * and raises TP3D_EPAGES, as does a count out of [0, copies].                 */
tp3d_status tp3d_paged_copy(tp3d_ctx* ctx, const tp3d_kv_cache* cache, int64_t copies, const int32_t* copy_from,
                            const int32_t* copy_to, const int32_t* copy_count, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TP3D_PAGED_H */
