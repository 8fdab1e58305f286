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
 *   tp3d_paged_store  K and V of the new tokens -> their slots;
 *   tp3d_paged_attn   attention of the new tokens over the cache.
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
typedef struct {
  int64_t token_stride, head_stride;
} tp3d_row_strides;
tp3d_status tp3d_paged_attn(tp3d_ctx* ctx, const tp3d_kv_cache* cache, const tp3d_paged_batch* batch, int heads,
                            float scale, const void* Q, tp3d_row_strides q_strides, void* O,
                            tp3d_row_strides o_strides, float* lse, void* workspace, void* stream);

/* Bytes of tp3d_paged_attn's workspace for this cache and head count on the
 * context's device (it does not depend on the batch); 0 for an invalid
 * argument.  Both kernels' parts of split work, for every SM: with 152 SMs 91 MB
 * for heads of 128, 46 MB for heads of 64.                                   */
size_t tp3d_paged_attn_workspace_bytes(tp3d_ctx* ctx, const tp3d_kv_cache* cache, int heads);

#ifdef __cplusplus
}
#endif

#endif /* TP3D_PAGED_H */
