/*
 * specfold_cache.h — committed context as a paged key-value cache: what writes
 * it, reads it for one new token, and keeps it inside its capacity.
 *
 * sf_verify (specfold.h) reads the committed context of every request as
 * prefix keys (already rotary-encoded) and values, shared by all branches
 * without copies (the zero-copy strided prefix view of the onedev.kr review of
 * "SpecFold", arXiv 2610.04875v2, "How to use it").  The pages leave open where
 * that context comes from; the operators here have no counterpart in them.
 * They work, layer by layer, on pools of pages in the prefix's own layout:
 *
 *   k_pages, v_pages  device [n_pages, page_size, n_kv_heads, head_dim] dtype
 *   page_table        device int32 [S, table_cols], rows ld_table apart: entry
 *                     (s, c) is the page that holds positions
 *                     c*page_size .. (c+1)*page_size-1 of sequence s
 *   lens              device int32 [S]: cached positions of every sequence
 *
 * A layer's prefix buffer [R, P, n_kv_heads, head_dim] with P a multiple of
 * page_size is such a pool with page_table[r][c] = r * (P / page_size) + c, so
 * sf_cache_append can write the prefix that sf_verify reads: P rows a request,
 * at positions 0..P-1.
 *
 * sf_cache_attend and sf_cache_evict are a decode loop of their own beside
 * that pass.  The rows that append takes and the queries come from the
 * caller's own projections; the weights that evict goes by come from attend.
 * What an eviction leaves is read by attend, not by sf_verify: the kept keys
 * stay rotated at their original positions, lie at the front of buffers of the
 * old length and may differ in number from sequence to sequence, while
 * sf_verify takes dense keys of positions 0..P-1 with one P for all requests.
 *
 * sf_cache_attend and sf_cache_evict plan their launches for the longest
 * sequence that the call could hold, min(max_len, table_cols * page_size)
 * positions, since lengths are on the device.  Where the sequences are far
 * shorter than the table, give table_cols as the columns that they use (with
 * the same page_table and ld_table): 64 sequences of 1,000 positions and 8
 * heads evict to 500 in 60 us with 32 columns of 32, in 150 us with a table
 * for 131,072 positions and in 300 us with one for 262,144.
 *
 * Any page size >= 1 works.  Entries of page_table past a sequence's length
 * are never read.  A page may appear in several sequences (a shared prefix)
 * where it is only read; pages that a call writes must be distinct.
 *
 * Types: dtype (SF_F32 or SF_BF16) for keys, values, queries and outputs; all
 * sums, norms, softmax statistics and accumulated weights are fp32.
 *
 * Threading and streams as in specfold.h: one host thread per cache object at
 * a time, all work enqueued on the caller's stream (which belongs to the
 * object's device, the current one of the call), nothing allocated and no
 * synchronisation, so every call can be captured into a CUDA graph.
 * sf_cache_attend uses the object's workspace: attend calls (and replays of
 * graphs that captured them) that may run at the same time need an object
 * each; the other two calls keep nothing in the object.
 *
 * Device-side checks: a page id outside [0, n_pages), a length or position
 * outside its range never becomes an access.  What the offending row or
 * sequence would have written is described with each call; the other rows and
 * sequences are not affected, and the check is reported as
 * SF_ERR_DEVICE_ASSERT by sf_cache_sync_status and by later calls on the
 * object, until sf_cache_sync_status clears it.
 */
#ifndef SPECFOLD_CACHE_H
#define SPECFOLD_CACHE_H

#include <stdint.h>

#include "specfold.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct sf_cache sf_cache;

typedef struct sf_cache_shapes {
  int n_q_heads;     /* multiple of n_kv_heads */
  int n_kv_heads;
  int head_dim;      /* 64 or 128 */
  int dtype;         /* sf_dtype */
  int page_size;     /* positions of a page, 1..65536 */
  int max_seqs;      /* capacity: S <= max_seqs <= 4096 */
  int max_len;       /* capacity: cached positions of a sequence, 1..262144 */
  int max_pos;       /* rotary positions 0..max_pos-1, 1..4194304 (a table of max_pos * head_dim * 4 bytes) */
  float rms_eps;
  float rope_theta;
  int track_weights; /* nonzero: sf_cache_attend may be given weights (a workspace of
                        max_seqs * n_q_heads * max_len * 4 bytes) */
} sf_cache_shapes;

/* Create a cache object on the current CUDA device: the rotary table (angles
 * in double) and the workspace of sf_cache_attend; the pools stay the
 * caller's.  Synchronous.
 * Errors: SF_ERR_INVALID_ARG (null pointer, a non-positive size, bad dtype,
 * negative eps, rope_theta not above 0), SF_ERR_UNSUPPORTED (head_dim not
 * 64/128, n_q_heads not a multiple of n_kv_heads, more than 1024 query heads,
 * a size beyond the limits above), SF_ERR_OOM, SF_ERR_CUDA.  *out is NULL on
 * error. */
sf_status sf_cache_create(const sf_cache_shapes* shapes, sf_cache** out);

/* Norm, rotate and store the T new rows of a layer: for every row t
 *   q, k of each head:  x / sqrt(mean(x^2) + rms_eps) * gain  (where the gain is
 *                       given), then the rotate-half rotation at position
 *                       pos[t] (pairs (j, j + head_dim/2), angle
 *                       pos * rope_theta^(-2j/head_dim));
 *   q -> q_out[t]; k and v -> position index[t] of sequence seq[t].
 * Computed in fp32, rounded once to dtype.
 *   qkv      device [T] rows of dtype, ld_qkv elements apart: the row's
 *            n_q_heads query heads, n_kv_heads key heads, n_kv_heads value
 *            heads (as the packed QKV projection leaves them).
 *   q_gain, k_gain  device fp32 [head_dim], or NULL for no norm of that side.
 *   index    device int32 [T]: place of the row in its sequence; negative: the
 *            row's K and V are not stored.
 *   pos      device int32 [T]: rotary position, which after an eviction is
 *            further on than the place; NULL = index.  A row whose position is
 *            negative is padding: nothing of it is written.
 *   seq      device int32 [T]: the row's sequence; NULL = row t belongs to
 *            sequence t (one new token each; T <= S).
 *   q_out    device [T] rows of n_q_heads * head_dim elements, ld_q apart; may
 *            be the query part of qkv itself (q_out == qkv, ld_q == ld_qkv).
 * (seq, index) pairs of one call are distinct.  A row with a sequence, place,
 * position or page out of range stores no K and V; without a valid position
 * it writes no query either.
 * qkv, the pools and q_out are 16-byte aligned, ld_qkv and ld_q multiples of
 * 16 bytes, the gains 16-byte aligned, the int32 arrays 4-byte.
 * Errors (before anything is enqueued): SF_ERR_INVALID_ARG (null or misaligned
 * argument, rows closer than their width, q_out overlapping qkv otherwise than
 * as said, another device is current), SF_ERR_SHAPE
 * (S beyond max_seqs, T above 1048576, T > S without seq),
 * SF_ERR_DEVICE_ASSERT (an earlier check fired), SF_ERR_CUDA. */
sf_status sf_cache_append(sf_cache* cache, void* stream, const void* qkv, int64_t ld_qkv, int T, const float* q_gain,
                          const float* k_gain, const int32_t* index, const int32_t* pos, const int32_t* seq,
                          const int32_t* page_table, int S, int table_cols, int64_t ld_table, void* k_pages,
                          void* v_pages, int64_t n_pages, void* q_out, int64_t ld_q);

/* Attention of one new token per sequence over its cached positions (its own
 * key and value among them, stored before by sf_cache_append):
 *   p_h[j] = softmax over j < lens[s] of scale * q[s,h] . k[s,j,kv(h)]
 *   out[s,h] = sum_j p_h[j] v[s,j,kv(h)],   kv(h) = h / (n_q_heads / n_kv_heads)
 * and, where weights_out is given, for every kv head c and j < lens[s]
 *   weights_out[s,c,j] = weights_in[s,c,j] + sum over h with kv(h) = c of p_h[j]
 * A sequence of length 0 gets zeros and no weights; so does a head of which
 * every score is -infinity (a sequence with all its pages out of range, for
 * one) where its values are finite.
 *   q        device [S] rows of n_q_heads * head_dim elements, ld_q apart.
 *   out      device [S] rows likewise, ld_out apart; not overlapping q.
 *   weights_in   device fp32 [S, n_kv_heads, ld_w] or NULL (counted as 0).
 *   weights_out  the same or NULL (none wanted); may be weights_in.  Entries at
 *            j >= lens[s] are not touched.  ld_w >= min(max_len, table_cols *
 *            page_size).
 * What else is in the batch changes results by rounding only (the sums are
 * split by the batch's total length); the same call gives the same bits.
 * Values: keys, values and queries as stored; products and sums fp32.
 * NaN and infinite values, and NaN and +infinite scores, among the live
 * positions make the outputs that they enter non-finite; a score of -infinity
 * weighs nothing.  What pools hold behind a sequence's length is never read.
 * A sequence whose length is negative or beyond max_len or table_cols *
 * page_size counts as empty, a position on a page out of range as one of score
 * -infinity (device check).
 * Errors: as above; SF_ERR_INVALID_ARG for a scale that is not finite or that
 * is not once it is multiplied by log2(e) (above 2.35e38), for out overlapping
 * q, for weights_out overlapping weights_in in part, for weights on an
 * object without track_weights or weights_in without weights_out;
 * SF_ERR_SHAPE for an ld_w too small. */
sf_status sf_cache_attend(sf_cache* cache, void* stream, const void* q, int64_t ld_q, const void* k_pages,
                          const void* v_pages, int64_t n_pages, const int32_t* page_table, int S, int table_cols,
                          int64_t ld_table, const int32_t* lens, float scale, void* out, int64_t ld_out,
                          const float* weights_in, float* weights_out, int64_t ld_w);

/* Keep at most `budget` positions of every sequence, chosen per KV head by
 * accumulated attention weight, and move them to the front:
 *   kept = all positions if lens[s] <= budget, else the first n_first, the
 *          last n_recent and the budget - n_first - n_recent others with the
 *          largest weight (equal weights: the lower index first; NaN below
 *          every number, -0 equal to 0), in ascending order;
 *   position i of sequence s, head c of the output := position kept[s,c,i];
 *   weights_out[s,c,i] = weights[s,c,kept[s,c,i]] (-0 as 0), and 0 for
 *          lens_out[s] <= i < lens[s], so that tokens stored there later start
 *          from 0;
 *   lens_out[s] = min(lens[s], budget).
 *   weights, weights_out  device fp32 [S, n_kv_heads, ld_w] (may be the same).
 *   k_out, v_out, table_out  where the kept positions go: pools of n_pages_out
 *          pages with their own table.  Either the very same pools and table
 *          as the input (in place), or pages that the input does not use.
 *          Rows behind the last kept position are left as they were.
 *   lens_out  device int32 [S]; may be lens.
 *   kept   device int32 [S, n_kv_heads, budget]; entries at i >= lens_out[s]
 *          are set to -1.
 * A sequence whose length is out of range counts as empty (lens_out 0); rows
 * from or to a page out of range are not moved (device check).
 * Errors: as above; SF_ERR_INVALID_ARG for budget < 1, a negative n_first or
 * n_recent, n_first + n_recent > budget, weights_out or lens_out overlapping
 * its input in part, or k_out/v_out/table_out of which only some are the
 * input's; SF_ERR_SHAPE for ld_w too small, budget beyond
 * max_len or beyond table_out_cols * page_size. */
sf_status sf_cache_evict(sf_cache* cache, void* stream, const void* k_pages, const void* v_pages, int64_t n_pages,
                         const int32_t* page_table, int S, int table_cols, int64_t ld_table, const int32_t* lens,
                         const float* weights, int64_t ld_w, int budget, int n_first, int n_recent, void* k_out,
                         void* v_out, int64_t n_pages_out, const int32_t* table_out, int table_out_cols,
                         int64_t ld_table_out, float* weights_out, int32_t* lens_out, int32_t* kept);

/* Wait for the work on `stream` and report a device-side check that fired
 * (SF_ERR_DEVICE_ASSERT, once: it is cleared on return) or a CUDA error. */
sf_status sf_cache_sync_status(sf_cache* cache, void* stream);

/* Text of the last error recorded on this object (empty if none). */
const char* sf_cache_last_error(const sf_cache* cache);

/* Free the object (synchronises the device first). */
sf_status sf_cache_destroy(sf_cache* cache);

#ifdef __cplusplus
}
#endif
#endif /* SPECFOLD_CACHE_H */
