/*
 * specfold_cache.h — committed context as a paged key-value cache: what writes
 * it, reads it for one new token, for blocks of rows and for batches that share
 * prefixes, keeps it inside its capacity, and moves its keys to new positions.
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
 * sf_verify takes dense keys rotated at positions 0..P-1 with one P for all
 * requests.  What an eviction leaves becomes that in two steps: evict to pages
 * that are such a buffer (of P = budget positions, where every sequence had at
 * least as many), then sf_cache_reposition with its `kept` positions, since
 * the kept keys stay rotated at their original ones.  The object's rotation
 * must be sf_verify's own then (the options' defaults).
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
 * sf_cache_attend, sf_cache_attend_rows and sf_cache_attend_shared use the
 * object's workspace: such calls (and replays of graphs that captured them)
 * that may run at the same time need an object each; append, evict and
 * reposition keep nothing in the object.
 *
 * Device-side checks: a page id outside [0, n_pages), a length or position
 * outside its range never becomes an access.  What the offending row or
 * sequence would have written is described with each call; the other rows and
 * sequences are not affected, and the check is reported as
 * SF_ERR_DEVICE_ASSERT by sf_cache_sync_status and by later calls on the
 * object, until sf_cache_sync_status clears it.  A wait inside a kernel that
 * does not end within 2 s is reported the same way; the outputs of that call
 * are undefined then, and nothing else is written.
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
 * in double) and the workspaces of the attend calls; the pools stay the
 * caller's.  Synchronous.
 * Errors: SF_ERR_INVALID_ARG (null pointer, a non-positive size, bad dtype,
 * negative eps, rope_theta not above 0), SF_ERR_UNSUPPORTED (head_dim not
 * 64/128, n_q_heads not a multiple of n_kv_heads, more than 1024 query heads,
 * a size beyond the limits above), SF_ERR_OOM, SF_ERR_CUDA.  *out is NULL on
 * error. */
sf_status sf_cache_create(const sf_cache_shapes* shapes, sf_cache** out);

/* What sf_cache_create leaves at its default: zeros are the defaults. */
enum { SF_ROTARY_HALVES = 0, SF_ROTARY_NEIGHBOURS = 1 };
typedef struct sf_cache_options {
  int rotary_layout;       /* pairs (j, j + rotary_dim/2), or SF_ROTARY_NEIGHBOURS: (2j, 2j + 1) */
  int rotary_dim;          /* the first dimensions of a head that positions turn; a multiple of 16, 0 = head_dim */
  const double* inv_freq;  /* host [rotary_dim / 2]: angle of one position for every pair; NULL:
                              rope_theta^(-2j/rotary_dim).  Copied. */
  double rotary_magnitude; /* sine and cosine are multiplied by it (queries and keys alike); 0 = 1 */
  int max_rows;            /* rows of a call of sf_cache_attend_rows, sequences of one of sf_cache_attend_shared, up to
                              1048576; 0: neither is called.  A workspace of 2 * SMs * 256 * (head_dim + 2) * 4 bytes
                              (bf16; half of it for fp32), and 2 * min(max_rows, max_seqs) * n_q_heads *
                              (head_dim + 2) * 4 bytes. */
} sf_cache_options;

/* The same with options (NULL: none).
 * Errors: also SF_ERR_INVALID_ARG for an unknown layout, a magnitude that is
 * negative or not finite (nor may 1 / magnitude in fp32 be infinite), a
 * frequency that is not finite, a negative size; SF_ERR_UNSUPPORTED for a
 * rotary_dim that is not a multiple of 16 up to head_dim, max_rows beyond its
 * limit. */
sf_status sf_cache_create_with(const sf_cache_shapes* shapes, const sf_cache_options* options, sf_cache** out);

/* Norm, rotate and store the T new rows of a layer: for every row t
 *   q, k of each head:  x / sqrt(mean(x^2) + rms_eps) * gain  (where the gain is
 *                       given; the mean is the whole head's), then the
 *                       rotation at position pos[t]: pairs (a, b) =
 *                       (j, j + head_dim/2) become (a cos - b sin, b cos +
 *                       a sin) of the angle pos * rope_theta^(-2j/head_dim);
 *                       or as the options say, dimensions past rotary_dim as
 *                       they are;
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

/* Attention of blocks of rows: each sequence's rows over all of its cached
 * positions, with no mask among the rows (a denoising block over its prefix, a
 * decoder's rows over an encoder's states):
 *   rows of sequence s = starts[s] .. starts[s+1] - 1;  for each of them, t,
 *   p_h[j] = softmax over j < lens[s] of scale * q[t,h] . k[s,j,kv(h)]
 *   out[t,h] = sum_j p_h[j] v[s,j,kv(h)],   kv(h) = h / (n_q_heads / n_kv_heads)
 *   lse[t,h] = ln sum_j exp(scale * q[t,h] . k[s,j,kv(h)])
 * Rows of a sequence of length 0 get zeros and an lse of -infinity; so does a
 * head of which every score is -infinity where its values are finite.  Rows in
 * front of starts[0] and from starts[S] on are left as they were.
 *   q        device [T] rows of n_q_heads * head_dim elements, ld_q apart.
 *   starts   device int32 [S + 1], 0 <= starts[0] <= starts[1] ... <= T.  Where
 *            they do not ascend so, nothing is written (device check).
 *   out      device [T] rows likewise, ld_out apart; not overlapping q.
 *   lse      device fp32 [T, n_q_heads] or NULL; not overlapping q or out.
 * Products and sums are fp32.  In bf16, softmax weights enter their product
 * with the values as the sum of two bf16 numbers (2^-16).  Only where the
 * tensor core bounds the call, more than 128 query vectors (rows times query
 * heads of a KV head) that go together, with more than two blocks of 256 of
 * them and 128 keys for each SM, are they rounded to one, half a step of 2^-8.
 * The rest as for sf_cache_attend: what else is in the batch changes results
 * by rounding only, the same call gives the same bits; NaN and infinities;
 * lengths and pages out of range.  The workspace is the object's.
 * Errors: as above; SF_ERR_INVALID_ARG for an object without max_rows, a scale
 * as for sf_cache_attend, overlapping outputs; SF_ERR_SHAPE for T beyond
 * max_rows and, in bf16, for pools of more than 2147483646 positions. */
sf_status sf_cache_attend_rows(sf_cache* cache, void* stream, const void* q, int64_t ld_q, int T, const void* k_pages,
                               const void* v_pages, int64_t n_pages, const int32_t* page_table, int S, int table_cols,
                               int64_t ld_table, const int32_t* lens, const int32_t* starts, float scale, void* out,
                               int64_t ld_out, float* lse);

/* Attention of one new token per sequence where groups of sequences share a
 * prefix: sequences starts[g] .. starts[g+1] - 1 see the prefix_lens[g]
 * positions of prefix g, then the lens[s] positions of their own, as if these
 * lay in one table.  A prefix is read once for its group (per 256 query
 * vectors), not once per sequence.  Sequences in front of starts[0] and from
 * starts[G] on have no prefix.
 *   q, out   device [S] rows as for sf_cache_attend; lse [S, n_q_heads] or NULL.
 *   page_table, lens            the sequences' own positions, [S].
 *   prefix_table, prefix_lens   device int32 [G, prefix_cols], rows ld_prefix
 *            apart, and [G]; pages of the same pools.
 *   starts   device int32 [G + 1], 0 <= starts[0] <= ... <= S.  Where they do
 *            not ascend so, nothing is written (device check).
 * A prefix and a sequence's own positions may hold up to max_len each.
 * Arithmetic, checks and workspace as for sf_cache_attend (own positions) and
 * sf_cache_attend_rows (prefixes); the two are joined in fp32.
 * It pays for groups of some sequences: 20,000 positions shared by 2 take 28 us
 * in bf16 (105 in fp32) with 28/4 heads x 128 where sf_cache_attend over both
 * takes 18 (44), 8,192 shared by 8 take 23 (84) with 32/8 heads where that takes
 * 28 (121).  Groups without sequences are cheap, not free: 8,192 of them cost
 * 20 us, 65,536 some 200 (four times that where a group that has sequences has
 * an empty prefix).
 * Errors: as for sf_cache_attend_rows, S taking the place of T;
 * SF_ERR_INVALID_ARG for G < 1, SF_ERR_SHAPE for G > 65536 (there may be more
 * groups than sequences: empty ones). */
sf_status sf_cache_attend_shared(sf_cache* cache, void* stream, const void* q, int64_t ld_q, const void* k_pages,
                                 const void* v_pages, int64_t n_pages, const int32_t* page_table, int S,
                                 int table_cols, int64_t ld_table, const int32_t* lens, const int32_t* prefix_table,
                                 int G, int prefix_cols, int64_t ld_prefix, const int32_t* prefix_lens,
                                 const int32_t* starts, float scale, void* out, int64_t ld_out, float* lse);

/* Turn keys in the cache to other positions: the key at place i < lens[s] of
 * sequence s and KV head c, which append rotated at position pos_from[s,c,i],
 * becomes the one of position pos_to[s,c,i] (rotation by the difference, in the
 * object's layout, dimensions and frequencies; rotary_magnitude is in the key
 * already).  Computed in fp32, rounded once to dtype.
 *   pos_from, pos_to   device int32 [S, n_kv_heads, ld_pos]; pos_to NULL = the
 *            place i.  evict's `kept` is a pos_from where positions are
 *            places.  Where either is negative, or both are the same, the key
 *            stays as it is.
 * What an eviction left in dense pages becomes so a prefix for sf_verify.
 * A sequence longer than ld_pos counts as out of range (nothing of it is
 * turned, device check), so does a position from max_pos on (that key stays).
 * Pages are distinct: a key that two entries reach would be turned twice.
 * Errors: as above; ld_pos < 1. */
sf_status sf_cache_reposition(sf_cache* cache, void* stream, void* k_pages, int64_t n_pages, const int32_t* page_table,
                              int S, int table_cols, int64_t ld_table, const int32_t* lens, const int32_t* pos_from,
                              const int32_t* pos_to, int64_t ld_pos);

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

/* Failure injection for tests of the detection path: in later calls of
 * sf_cache_attend_rows and sf_cache_attend_shared on a bf16 object, one of the
 * signals between the warps of a thread block (1..13, as CacheStallAt in
 * csrc/sf_cache.h names them) is never complete.  Waits for it, and all others
 * meanwhile, give up after 50 ms; the kernels end, with the outputs undefined,
 * and the call is reported as described at the top.  0: no more.  A call that
 * does not need the signal is not affected but for the 50 ms.  No GPU fault,
 * trap or hang is involved.
 * Errors: SF_ERR_INVALID_ARG (null object, another signal). */
sf_status sf_cache_inject_stall(sf_cache* cache, int signal);

/* Text of the last error recorded on this object (empty if none). */
const char* sf_cache_last_error(const sf_cache* cache);

/* Free the object (synchronises the device first). */
sf_status sf_cache_destroy(sf_cache* cache);

#ifdef __cplusplus
}
#endif
#endif /* SPECFOLD_CACHE_H */
