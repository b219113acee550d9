/*
 * dlrm_seq_decay.h -- C ABI of linear attention with a decay (MI355X, gfx950): a layer over user
 * histories whose memory of a user is one d x d matrix a key head, however long the history.
 *
 * Key head c of a sequence has a state S, from event t - 1 to event t, and query head h of its
 * group (c = h / (Hq / Hkv)) reads it:
 *
 *     S[t] = e^g[t][c] S[t-1] + k[t][c] v[t][c]^T;    o[t][h] = scale * S[t]^T q[t][h]
 *
 * so that event j reaches event i >= j with the weight e^(g[j+1] + ... + g[i]): by the time between
 * events, or one decay for a head.  The first event decays the state that the call begins with.
 *
 * Conventions: as dlrm_seq.h (jagged sequences laid end to end with CSR offsets; bf16 activations
 * as uint16_t; caller-owned buffers; nothing allocated; arguments validated before anything is
 * enqueued; bitwise reproducible).  States, decays, their gradients and all sums are fp32 (sums of
 * decays fp64), and state_out, the single event's state and dg are right to about 2^-22 of their terms: where a
 * product takes bf16, it takes three such parts of a state.  Where only o, or dq, dk and dv of a call without dg, come of
 * a state, two parts of what is added to it are taken (2^-16), and the state's product with a row from its values
 * rounded to bf16 once (2^-8, as the outputs are).
 */
#ifndef DLRM_SEQ_DECAY_H
#define DLRM_SEQ_DECAY_H

#include <stddef.h>
#include <stdint.h>

#include "dlrm_sparse.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 *   B          sequences, >= 0;  N: rows of q, k, v
 *   Hq, Hkv    query heads, and heads of keys, values, decays and states, Hq a multiple of Hkv
 *   d          elements of a head
 *   offsets    [B+1] int64 (DLRM_INDEX_I64) or int32, non-decreasing, within [0, N].  Offsets
 *              outside are brought inside: no foreign memory is read.  Not read by the step.
 *   max_len    an upper bound of the sequences' lengths, by which a call chooses whether to cut
 *              sequences into runs that are worked on side by side, with a state for each in the workspace (up to
 *              256 MB, or as much as q, k, v and o take; twice that in the backward); N where it is not known: one sequence may then be
 *              all of them, and batches of short ones are slower.  Longer sequences give results as exact, slower.  (The bits may differ with it, and with
 *              the number of sequences and rows.)
 *   q, k, v    bf16; element e of head h of row r at r * row_stride + h * head_stride + e, strides
 *              in elements, multiples of 8, >= d; 16-byte aligned
 *   g          fp32 logarithms of the decays, <= 0: that of row r and head c at r * g_row + c; g_row >= Hkv,
 *              or 0: one decay for a head, [Hkv].  What is above 0 counts as 0 (with a gradient of 0),
 *              what is below -104, -infinity too, as -104, where e^g is 0 in fp32.
 *   Limits: d % 8 == 0, 8 <= d <= 128; Hq <= 4096; B < 2^24; N < 2^31; row strides < 2^24 elements; a
 *   sequence < 2^30 rows; (N / 64 + B + 8) * Hkv < 2^23, for d > 64 < 2^22.
 */
typedef struct {
    int64_t B, N;
    int32_t Hq, Hkv, d;
    int32_t index_type;
    const void *offsets;
    int64_t max_len;
    const uint16_t *q, *k, *v;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head; /* strides */
    const float *g;
    int64_t g_row;
    float scale;
} dlrm_seq_decay;

/* Bytes of workspace dlrm_seq_decay_fwd needs (0 on an invalid description; 256: it uses none, which may be NULL). */
size_t dlrm_seq_decay_fwd_workspace_size(const dlrm_seq_decay *a);

/*
 * Forward.  o [N][Hq][d] bf16; rows outside every sequence are not written.
 *   state_in   [B][Hkv][d][d] fp32 (key's element, value's element), or NULL: zeros
 *   state_out  the same after each sequence's last event (may be state_in, else apart from it), or NULL: not wanted.
 *              A sequence without events leaves its state as it is.
 *   What an event holds has no effect on the outputs before it, NaN and infinities included; after it,
 *   what they reach is not finite.  o takes the products within 64 events, and the state's with q,
 *   from values rounded to bf16.  (In place, the query heads of a group are not spread over workgroups while sequences
 *   are whole, and their first states are copied where they are cut: 4 sequences of up to 60, 16 heads over 2 of 128, 25 us
 *   where 14 apart.)
 */
int dlrm_seq_decay_fwd(const dlrm_seq_decay *a, const float *state_in, float *state_out, uint16_t *o,
                       void *workspace, size_t workspace_bytes, dlrm_stream_t stream);

/*
 * Bytes of workspace dlrm_seq_decay_bwd needs, with dg or without (0 on an invalid description): beside the runs'
 * states or an order, states at marks, d * d floats (d as 32, 64 or 128) for 512 rows and key head or, with one decay a head,
 * 128 (for less where sequences are cut into runs of fewer), and two floats a row and key head.
 */
size_t dlrm_seq_decay_bwd_workspace_size(const dlrm_seq_decay *a);

/*
 * Backward, of sequences that begin with a state of zeros and whose last state is not used.  With
 * w_ij = e^(g[j+1] + ... + g[i]), summed over the query heads of a group where shared:
 *
 *     dq_i = scale sum_{j<=i} w_ij <do_i, v_j> k_j;   dk_j = scale sum_{i>=j} w_ij <do_i, v_j> q_i;
 *     dv_j = scale sum_{i>=j} w_ij <q_i, k_j> do_i;   dg_t = sum_{i>=t} <q_i, dq_i> - <k_i, dk_i>
 *
 *   dout [N][Hq][d] bf16;  dq [N][Hq][d], dk, dv [N][Hkv][d] bf16 (rows of every sequence are written in
 *   full, rows outside not at all)
 *   dg   [N][Hkv] fp32 (rows outside every sequence are not written), [Hkv] where g_row == 0, or NULL:
 *        not wanted
 *   Infinities and NaN in k and v have no effect on dq before them; those of q and dout reach dk and
 *   dv of all events before them, and of up to 63 after them too; dg of a sequence that holds any means nothing (nor
 *   does that of a head).
 *   Without dg there is less to do, and dq, dk and dv come of less exact states (see above).
 */
int dlrm_seq_decay_bwd(const dlrm_seq_decay *a, const uint16_t *dout, uint16_t *dq, uint16_t *dk,
                       uint16_t *dv, float *dg, void *workspace, size_t workspace_bytes,
                       dlrm_stream_t stream);

/*
 * One event of each sequence: N == B, row b is sequence b's event.
 *   state [B][Hkv][d][d] fp32, updated in place;  o [B][Hq][d] bf16
 *   Limits: B * Hkv < 2^24.
 */
int dlrm_seq_decay_step(const dlrm_seq_decay *a, float *state, uint16_t *o, dlrm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DLRM_SEQ_DECAY_H */
