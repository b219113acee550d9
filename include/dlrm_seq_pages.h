/*
 * dlrm_seq_pages.h -- C ABI of the paged cache of user histories (MI355X, gfx950): keys and values
 * of many users in pages of one pool, the tables that say which page holds which events, kept on
 * the GPU from the lengths of each visit, and attention over such a cache.
 *
 * Conventions: as dlrm_seq.h.
 */
#ifndef DLRM_SEQ_PAGES_H
#define DLRM_SEQ_PAGES_H

#include <stddef.h>
#include <stdint.h>

#include "dlrm_seq.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * B users and the pages that they hold.  Event p of user b is row
 * table[b * table_row + p / page] * page + p % page of the pool's pages * page rows.
 *
 *   page      events of a page: a power of two, 8 to 4096
 *   pages     of the pool, >= 1; pages * page < 2^31
 *   width     most pages of a user, >= 0;  table_row: elements from one user's entries to the next's, >= width
 *   table     int32; entries past a user's pages are -1 (the update keeps them so; nothing relies on it)
 *   lengths   [B] int32: events of each user
 *   free_list [pages] int32, free_count [1] int32: a stack of the pages that nobody holds, its top at
 *             free_count - 1 (a new pool: the numbers from 0 on, and `pages`).  Only the update reads these.
 *   Contents that cannot be are brought inside (a length into [0, width * page], a page into the pool):
 *   no foreign memory is read or written.
 *   Limits: B < 2^20; width * page < 2^30.
 */
typedef struct {
    int64_t B, pages, table_row;
    int32_t width, page;
    int32_t *table, *lengths, *free_list, *free_count;
} dlrm_seq_pages;

/* Bytes of workspace dlrm_seq_pages_update needs (0 on invalid sizes). */
size_t dlrm_seq_pages_update_workspace_size(int64_t B, int64_t N);

/*
 * A visit.  Users in `leave` give their pages back and are empty; then user b's new events,
 * offsets[b+1] - offsets[b] of them, get their places:
 *
 *   leave    [B] bytes, not 0: the user leaves;  NULL: none
 *   offsets  [B+1], of index_type, non-decreasing, within [0, N] (brought inside)
 *   slots    [N] int64: new event i of user b, row offsets[b] + i, gets the pool's row; -1 where the
 *            user is refused; rows outside every user's are not written
 *   refused  [1] int32: how many users were refused: those whose events do not fit their table, and those
 *            for whom, with all that the users before them want, there are not enough pages: from the first
 *            such user on everyone who wants a page, also where fewer would do and are there.  Those who want
 *            none get their slots, and a user whose table is too short takes no part in the sum.  Nothing
 *            changes for a refused user (who may have left).
 *
 * The order is that of the users: pages that come back are put on the stack first to last (a user's in
 * the table's order), pages are taken from its top, the first user's first page first.
 * table, lengths, free_list and free_count are updated in place, `workspace` as the size says, 256-byte
 * aligned.  2^31 > N >= 0.
 */
int dlrm_seq_pages_update(const dlrm_seq_pages *p, const void *offsets, int32_t index_type, int64_t N,
                          const uint8_t *leave, int64_t *slots, int32_t *refused, void *workspace,
                          size_t workspace_bytes, dlrm_stream_t stream);

/*
 * Rows of keys and values to their slots: row slots[i] of k_pool and v_pool = row i of k and v.  Slots
 * outside [0, rows) are passed over; no two others may be equal.
 *   k, v [N][H][d], k_pool, v_pool [rows][H][d] bf16, strides and alignment as dlrm_seq_attn's;
 *   d % 8 == 0; H * d <= 2^20; N < 2^31
 */
int dlrm_seq_pages_write(const uint16_t *k, int64_t k_row, int64_t k_head, const uint16_t *v, int64_t v_row,
                         int64_t v_head, int64_t N, int32_t H, int32_t d, const int64_t *slots,
                         uint16_t *k_pool, int64_t k_pool_row, int64_t k_pool_head, uint16_t *v_pool,
                         int64_t v_pool_row, int64_t v_pool_head, int64_t rows, dlrm_stream_t stream);

/*
 * dlrm_seq_attn_fwd over the pages: `a` as there, but that k and v are the pool (Nkv == pages * page rows),
 * kv_begin and kv_end are not read, and sequence b's keys are user b's events, lengths[b] of them, the
 * new ones among them (the update has counted them, the write has put them there).  B == p->B.  (Sums over
 * keys may be taken in another order than there: the bits may differ.)
 */
int dlrm_seq_attn_paged_fwd(const dlrm_seq_attn *a, const dlrm_seq_pages *p, uint16_t *o,
                            dlrm_stream_t stream);

/* dlrm_seq_attn_decode over the pages, likewise; its workspace has the same size (256: it uses none, which may be NULL). */
int dlrm_seq_attn_paged_decode(const dlrm_seq_attn *a, const dlrm_seq_pages *p, int64_t max_kv_len,
                               uint16_t *o, void *workspace, size_t workspace_bytes,
                               dlrm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DLRM_SEQ_PAGES_H */
