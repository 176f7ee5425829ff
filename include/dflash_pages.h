/*
 * dflash_pages.h — C ABI of the pages behind the paged cache on one GB300 GPU:
 * which pages a request holds, where a step's new tokens go, and the pages that
 * rejected tokens leave, all from lengths on the device, so that a step needs
 * no host and a captured graph can be replayed.
 *
 *   dflash_pages_extend  gives a batch's requests the pages of their new tokens
 *                        and builds what the step's calls take: cu_tokens,
 *                        lens and page_table of dflash_paged_batch, and every
 *                        token's position and slot;
 *   dflash_pages_trim    shortens requests (rejected drafts, ended requests)
 *                        and takes back the pages that they no longer need.
 *
 * Conventions: as in dflash_select.h (device pointers owned by the caller,
 * asynchronous on `stream`, no aborts; a non-zero status means nothing was
 * launched and dflash_last_error() has the message). Strides count elements.
 */
#ifndef DFLASH_PAGES_H
#define DFLASH_PAGES_H

#include <stdint.h>

#include "dflash_select.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The pool. A request of n tokens holds ceil(n / page_size) pages, the first
 * entries of its row of page_table; free_pages[0 .. counters[0] - 1] is a stack
 * of the others. The calls that change a pool must not overlap on the GPU
 * (order them on one stream, any). To begin with: lens 0, the stack all pages,
 * counters {num_pages, 0}. Limits: 1 <= requests, 1 <= cols <= 2^20,
 * 1 <= page_size <= 65536, 1 <= num_pages < 2^31, cols * page_size < 2^31. */
typedef struct {
    int32_t *page_table;  /* [requests, cols], rows table_stride apart */
    int64_t table_stride;
    int32_t *lens;        /* [requests] */
    int32_t *free_pages;  /* [num_pages] */
    int32_t *counters;    /* [2]: free pages; the call's count of its blocks, 0 between calls */
    int32_t requests, cols, page_size, num_pages;
} dflash_page_pool;

/* Entry b of the batch is request rows[b] (NULL: b itself; distinct among the
 * entries with new tokens, so that others may pad a batch), which gets
 * new_tokens[b] >= 0 tokens behind those that it has. Entries are served
 * in order while pages and `tokens` last: entry b is refused, and gets nothing,
 * if the entries up to and including it need more than the free pages or have
 * more than `tokens` new tokens together (so are all after it that follow in
 * such a sum), and on its own account if its row or its number is out of range
 * or it would exceed its row of a table.
 * The i-th page taken is free_pages[counters[0] - 1 - i], in the order of the
 * entries and of their places. Changes page_table, lens and counters[0].
 * Outputs (int32 unless said; NULL = not wanted):
 *   cu_tokens  [batch + 1] the entries' first token rows, as in dflash_paged_batch
 *   lens       [batch] the requests' lengths with the new tokens (0 for a row out of range)
 *   page_table [batch, table_cols], rows table_stride apart: the entries that
 *              the lengths take, the others are left as they were
 *   positions  [tokens] each token's place in its request
 *   slots      [tokens] int64, page * page_size + place % page_size
 *   granted    [batch] 1, or 0 for a refused entry
 * Rows of positions and slots from cu_tokens[batch] on are left as they were.
 * With rows = NULL, lens and page_table may be the pool's own (the same
 * address; page_table with the same stride), and new_tokens may be the pool's
 * lens; nothing else overlaps, or the call is refused.
 * 0 <= batch <= 65536, batch <= requests; 0 <= tokens <= 2^30. Errors: INVALID_ARG, CUDA. */
dflash_status dflash_pages_extend(const dflash_page_pool *pool, const int32_t *rows, const int32_t *new_tokens,
                                  int32_t batch, int32_t tokens, int32_t *cu_tokens, int32_t *lens, int32_t *page_table,
                                  int64_t table_stride, int32_t table_cols, int32_t *positions, int64_t *slots,
                                  int32_t *granted, void *stream);

/* Request rows[b] (NULL: b itself; distinct among those that lose something)
 * loses its last d tokens, at most those that it has (none with d <= 0, or for a row out of range):
 *   d = counts[b]           with base < 0;
 *   d = base - counts[b]    with base >= 0: base = L and the accept lengths of
 *                           dflash_verify_prefix drop a block's rejected drafts;
 *   everything              with counts = NULL (a request that has ended).
 * Pages that it no longer needs return to the stack, so that an extension that
 * takes them back takes them in the same order. With rows = NULL, counts may
 * be the pool's lens; nothing else overlaps, or the call is refused.
 * 0 <= batch <= 65536, batch <= requests.
 * Errors: INVALID_ARG, CUDA. */
dflash_status dflash_pages_trim(const dflash_page_pool *pool, const int32_t *rows, const int32_t *counts, int32_t base,
                                int32_t batch, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DFLASH_PAGES_H */
