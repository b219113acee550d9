/*
 * dlrm_seq.h -- C ABI of the user-history operators (MI355X, gfx950): attention over jagged
 * sequences of events, forward, backward and for one new event over a cache; the RMS norm with the
 * residual's addition; dropout from a counter-based generator.
 *
 * A bag (dlrm_sparse.h) pools a user's ids without their order.  These calls work on the events in
 * their order: a batch is B sequences of differing lengths, laid end to end, with offsets in the
 * manner of the bags' CSR offsets.
 *
 * Conventions: as dlrm_sparse.h (device pointers unless marked, caller-owned buffers, calls enqueue
 * on `stream` and return, arguments validated before anything is enqueued, nothing allocated).
 * bf16 values are passed as uint16_t.  Activations are bf16, as between the dense layers
 * (dlrm_mlp.h); sums, softmax statistics and norms are fp32.  Every sum has a fixed order: results
 * are bitwise reproducible.
 */
#ifndef DLRM_SEQ_H
#define DLRM_SEQ_H

#include <stddef.h>
#include <stdint.h>

#include "dlrm_sparse.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most distance buckets of the attention bias. */
#define DLRM_SEQ_MAX_BUCKETS 128

/* Output type of dlrm_add_rmsnorm_fwd beside dlrm_dtype's: 8-bit floats of 4 exponent and 3
 * mantissa bits (largest value 448, no infinities), with one fp32 scale a row. */
enum { DLRM_F8_E4M3 = 2 };

/*
 * What the three attention calls share.  Query i of sequence b, 0 <= i < q_len, is row
 * q_offsets[b] + i of q and stands at position p = kv_len - q_len + i of its sequence: the queries
 * are the sequence's last events.  Key j, 0 <= j < kv_len, is row kv_begin[b] + j of k and v, with
 * kv_len = kv_end[b] - kv_begin[b].  With n = p - j the distance back to the key, query head h, its
 * key/value head h / (Hq / Hkv):
 *
 *     visible(i,j)  n >= 0 and (window == 0 or n < window or j < sinks)
 *     z[i][j]       scale * <q_i, k_j> + bias[h][bucket(n)],  bucket(n) = the last t with bounds[t] <= n
 *     lse[i]        log sum_{visible j} exp z[i][j]
 *     o[i]          sum_{visible j} exp(z[i][j] - lse[i]) v_j
 *
 * A query that sees no key (kv_len == 0, or p < 0) has o = 0 and lse = -infinity.  What k and v
 * hold for a key that a query does not see has no effect on its o and lse, NaN and infinities
 * included.  o is finite where the values that it is a mean of are, however large.
 *
 *   B          sequences, >= 0;  Nq, Nkv: rows of q, and of k and v
 *   Hq, Hkv    query and key/value heads, Hq a multiple of Hkv;  d: elements of a head
 *   q, k, v    bf16; element e of head h of row r at r * row_stride + h * head_stride + e, strides
 *              in elements, multiples of 8, >= d; 16-byte aligned
 *   q_offsets  [B+1];  kv_begin, kv_end [B] (a CSR array of B+1 offsets gives both: it, and it + 1);
 *              int64 (DLRM_INDEX_I64) or int32; non-decreasing, within [0, Nq] and [0, Nkv].
 *              Offsets outside are brought inside: no foreign memory is read.
 *   window     0: none; sinks: how many first keys every later query sees (only with a window)
 *   bias       [Hq][buckets] fp32, or NULL: no bias;  bounds (host) [buckets], bounds[0] == 0,
 *              strictly increasing: the first distance of each bucket, the last bucket open
 *   Limits: d % 8 == 0, 8 <= d <= 128; 1 <= Hq <= 4096; B < 2^24; Nq, Nkv < 2^31; row strides
 *   < 2^24 elements; a sequence < 2^30 rows; 1 <= buckets <= DLRM_SEQ_MAX_BUCKETS; Nq / 64 + B and
 *   Nkv / 64 + B below 2^25 (2^24 for d > 64) in the forward and backward, B * Hkv times the 16s of
 *   query heads that share one below 2^24 in the form for one event.
 */
typedef struct {
    int64_t B, Nq, Nkv;
    int32_t Hq, Hkv, d;
    int32_t index_type;
    const void *q_offsets, *kv_begin, *kv_end;
    const uint16_t *q, *k, *v;
    int64_t q_row, q_head, k_row, k_head, v_row, v_head; /* strides */
    int32_t window, sinks;
    float scale;
    int32_t buckets;
    const float *bias;
    const int32_t *bounds; /* (host) */
} dlrm_seq_attn;

/* Entries of the forward's `tiles` (0 on invalid sizes). */
size_t dlrm_seq_attn_tiles(int64_t B, int64_t Nq);

/*
 * Forward.  o [Nq][Hq][d] bf16; rows outside every sequence are not written.
 *   lse, tiles: NULL, or both given for a backward pass: lse [Nq][Hq] fp32, and tiles, int32
 *   [dlrm_seq_attn_tiles(B, Nq)]: the sequence that each tile of queries belongs to, which the
 *   backward would have to search for again.
 */
int dlrm_seq_attn_fwd(const dlrm_seq_attn *a, uint16_t *o, float *lse, int32_t *tiles,
                      dlrm_stream_t stream);

/* Bytes of workspace dlrm_seq_attn_bwd needs for this description (0 on an invalid one). */
size_t dlrm_seq_attn_bwd_workspace_size(const dlrm_seq_attn *a);

/*
 * Backward.  With P = exp(z - lse) on the visible pairs, dP[i][j] = <do_i, v_j> and
 * ds = P * (dP - <do_i, o_i>), summed over the query heads of a key/value head where shared:
 *
 *     dv_j = sum_i P do_i;  dk_j = scale sum_i ds q_i;  dq_i = scale sum_j ds k_j;
 *     dbias[h][t] = sum over the pairs of bucket t of ds
 *
 *   a: the forward's, with kv_begin a CSR array of B+1 offsets (kv_end == kv_begin + 1)
 *   dout [Nq][Hq][d] bf16; o, lse, tiles as the forward wrote them (not read where Nq == 0; o
 *   is read without a bias only: with one, <do, o> is summed again in fp32, as dbias needs it)
 *   dq [Nq][Hq][d], dk, dv [Nkv][Hkv][d] bf16 (rows of every sequence are written in full,
 *   rows outside every sequence not at all);
 *   dbias [Hq][buckets] fp32 (with a bias; else NULL)
 *   Infinities and NaN in a key that a query does not see have no effect on its dq, and a key that
 *   no query sees has gradients of zero; those of q, dout and lse reach every key near by.
 */
int dlrm_seq_attn_bwd(const dlrm_seq_attn *a, const uint16_t *dout, const uint16_t *o,
                      const float *lse, const int32_t *tiles, uint16_t *dq, uint16_t *dk,
                      uint16_t *dv, float *dbias, void *workspace, size_t workspace_bytes,
                      dlrm_stream_t stream);

/* Bytes of workspace dlrm_seq_attn_decode needs (0 on invalid sizes). */
size_t dlrm_seq_attn_decode_workspace_size(int64_t B, int32_t Hq, int32_t Hkv, int32_t d,
                                           int32_t window, int32_t sinks, int64_t max_kv_len);

/*
 * One new event a sequence over a cache: the forward for q_len = 1, q [B][Hq][d] (row b is sequence
 * b's query; q_offsets is not read, Nq == B), with the keys of one sequence split over workgroups
 * where B * Hkv of them do not fill the GPU.  k and v already hold the event's own row, the last.
 *   o [B][Hq][d] bf16 (written in full)
 *   max_kv_len: an upper bound of the sequences' lengths, which the split is chosen by.  Longer
 *   sequences give the same results, slower.
 */
int dlrm_seq_attn_decode(const dlrm_seq_attn *a, int64_t max_kv_len, uint16_t *o, void *workspace,
                         size_t workspace_bytes, dlrm_stream_t stream);

/*
 * Dropout's random numbers: Philox4x32-10 (Salmon, Moraes, Dror, Shaw: "Parallel random numbers:
 * as easy as 1, 2, 3", 2011) with the 64-bit key `seed`.  Element e of a row-major array takes 16
 * of the 128 bits that the counter value `offset + *offset_dev + e / 8` gives: half e % 2 (low
 * first) of word (e % 8) / 2.  It is kept when those 16 bits, as a number, are at least
 * D = floor(p * 65536 + 0.5), and is then scaled by 65536 / (65536 - D), kept as one fp32 number;
 * dropped elements are 0, whatever they held.  p is thus held to 2^-16.  No mask is stored: the backward pass makes it
 * again from the same numbers.  A step that uses n elements moves `offset` by (n + 7) / 8; kept in
 * device memory (offset_dev, NULL: 0) it moves under a captured graph.
 */
typedef struct {
    float p; /* 0 <= p <= 1; 0: no dropout */
    uint64_t seed, offset;
    const uint64_t *offset_dev;
} dlrm_dropout_spec;

/* y[e] = keep(e) ? x[e] * 65536 / (65536 - D) : 0 for e < n; x and y of `dtype` (F32 or BF16),
 * 16-byte aligned; y may be x.  Its derivative is the same call on the gradient. */
int dlrm_dropout(const void *x, int32_t dtype, int64_t n, const dlrm_dropout_spec *drop, void *y,
                 dlrm_stream_t stream);

/*
 * Between two layers of an encoder: the branch x, after dropout, is added to the residual, and the
 * sum's RMS norm goes into the next layer.
 *
 *     s = residual + dropout(x)   (element index row * D + column; rounded to res_dtype)
 *     rstd = 1 / sqrt(mean_c s[c]^2 + eps);   y = s * rstd * w
 *
 *   x [M][D] of x_dtype (F32 or BF16);  residual [M][D] of res_dtype or NULL (zeros);  w [D] fp32
 *   s [M][D] of res_dtype (may be residual), or NULL: not written;  rstd [M] fp32 or NULL
 *   y [M][D] of y_dtype: F32, BF16, or F8_E4M3 with y_scale [M] fp32: y = q * y_scale[row],
 *   y_scale = max_c |y| / 448 (1 for a row of zeros, at least 2^-149) and q the fp32 quotient
 *   y / y_scale, rounded to nearest even; y_scale is not written for the other types.
 *   The norm is taken of s as rounded, so that the backward, which has only that, agrees.
 *   Limits: 0 <= M < 2^31; D from 1 to 16384 in steps of 8, other widths to 4096; buffers 16-byte
 *   aligned.
 */
int dlrm_add_rmsnorm_fwd(const void *x, int32_t x_dtype, const void *residual, int32_t res_dtype,
                         const float *w, float eps, const dlrm_dropout_spec *drop, int64_t M, int32_t D,
                         void *s, void *y, int32_t y_dtype, float *y_scale, float *rstd,
                         dlrm_stream_t stream);

/* Bytes of workspace dlrm_add_rmsnorm_bwd needs (0 on invalid sizes). */
size_t dlrm_add_rmsnorm_bwd_workspace_size(int64_t M, int32_t D);

/*
 * Its backward.  With hat = s * rstd and g = dy * w, per row:
 *
 *     dh = ds + rstd * (g - hat * mean_c(g hat));  dresidual = dh;  dx = dropout's derivative of dh
 *     dw = sum over rows of dy * hat
 *
 *   dy [M][D] of dy_dtype (F32 or BF16);  ds [M][D] of res_dtype or NULL: the gradient that reaches
 *   s past the norm;  s, w, rstd as in the forward;  drop: the forward's
 *   dx [M][D] of x_dtype;  dresidual [M][D] of res_dtype or NULL (may be ds);  dw [D] fp32
 */
int dlrm_add_rmsnorm_bwd(const void *dy, int32_t dy_dtype, const void *ds, const void *s,
                         int32_t res_dtype, const float *w, const float *rstd,
                         const dlrm_dropout_spec *drop, int64_t M, int32_t D, void *dx, int32_t x_dtype,
                         void *dresidual, float *dw, void *workspace, size_t workspace_bytes,
                         dlrm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DLRM_SEQ_H */
