/*
 * attn_paged.h -- C ABI of the paged-cache operators of libattn_decode.so:
 * appending rotated keys and values to a paged cache, and decode attention
 * over such a cache, held in 16 bits or in 8 bits with a scale per page and KV
 * head, with plain scores or with scores that are capped, biased by distance
 * and windowed.
 *
 * The conventions of attn_decode.h hold: device pointers are caller-owned and
 * 16-byte aligned (int32 arrays, scales and slopes 4-byte aligned), argument
 * errors come back synchronously before anything is launched, nothing
 * synchronises the stream, data-dependent errors set a bit of the sticky
 * device error word (attn_read_device_error), and every launch can be captured
 * in a CUDA graph and replayed while positions, tables and contents change.
 * Calls run on the current device.
 *
 * Paged cache. The rows of a sequence live in pages of page_size rows taken
 * from a pool of n_pages pages. Row j of sequence s is row j % page_size of
 * page block_table[s][j / page_size]. A dense cache [n_seq][cap][n_kv_head]
 * [head_dim] is the special case of consecutive page numbers. Only the entries
 * of pages that hold a row the call uses are read, so the others may hold
 * anything. A used entry outside [0, n_pages) sets ATTN_DEVERR_BAD_PAGE: an
 * append skips its rows, attention takes them as not there.
 *
 * Rows at or past positions[s] + 1 are never used and never change a result,
 * whatever they hold; the page that holds row positions[s] may be read to its
 * end. Rows that are seen are taken to hold finite values: NaN gives NaN, an
 * infinity among them infinity or NaN.
 */
#ifndef ATTN_PAGED_H
#define ATTN_PAGED_H

#include "attn_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A used entry of the block table is not a page of the pool. */
#define ATTN_DEVERR_BAD_PAGE 0x4u

/* Element types. Caches: F16, BF16, E4M3. New rows and queries: F32, F16, BF16. */
#define ATTN_TYPE_F32 0
#define ATTN_TYPE_F16 1
#define ATTN_TYPE_BF16 2
#define ATTN_TYPE_E4M3 3  /* 8 bits: 4 exponent, 3 fraction, no infinities, largest 448 */

/*
 * The pool. A cache element (page, row, KV head, d) is at
 *     page * page_stride + row * row_stride + head * head_stride + d
 * elements from k (v): any order of pages, rows and heads, and a pool that is
 * part of a larger allocation. Strides are in elements; page_stride,
 * row_stride and head_stride all 0 stand for the dense
 * [n_pages][page_size][n_kv_head][head_dim]. In bytes each stride is a
 * multiple of 16 and below 2^40.
 *   head_dim    64, 128 or 256 (ATTN_ERR_UNSUPPORTED otherwise)
 *   page_size   a multiple of 16, at most 1024
 *   k_scale, v_scale  E4M3 only: float [n_pages][n_kv_head], dense; the value of
 *               an element is its code times the scale of its page and head.
 *               attn_rope_append writes powers of two between 2^-60 and 2^60, or
 *               the magnitude of what it finds on a page filled elsewhere;
 *               attention takes any finite scale of magnitude up to 2^60.
 */
typedef struct {
    void *k;
    void *v;
    float *k_scale;
    float *v_scale;
    int64_t page_stride;
    int64_t row_stride;
    int64_t head_stride;
    int32_t n_pages;
    int32_t page_size;
    int32_t n_kv_head;
    int32_t head_dim;
    int32_t kv_type;       /* ATTN_TYPE_F16, _BF16 or _E4M3 */
    int32_t reserved;      /* 0 */
} attn_paged_cache;

/* How rotary frequencies are stretched for contexts longer than the trained one. */
#define ATTN_ROPE_PLAIN 0   /* f_i = base^(-2i / rot_dim) */
#define ATTN_ROPE_LINEAR 1  /* f_i / factor */
#define ATTN_ROPE_BASE 2    /* base * factor^(rot_dim / (rot_dim - 2)) in place of base */
#define ATTN_ROPE_BANDS 3   /* by turns n_i = trained_len * f_i / (2 pi): f_i where n_i >= high_turns,
                               f_i / factor where n_i <= low_turns, linear in n_i between */

/*
 * The rotation of an append. The first rot_dim dimensions of a head are
 * rotated, the rest pass through. With a_i, b_i the pair i < rot_dim / 2
 *     a' = (a cos t - b sin t) * mscale,  b' = (b cos t + a sin t) * mscale,
 * t = position * f_i; the pair is (x[i], x[i + rot_dim / 2]), or, interleaved,
 * (x[2i], x[2i + 1]).
 *   steps   device, uint64 [rot_dim / 2], 16-byte aligned: from attn_rope_steps
 *   rot_dim a multiple of 16, at most head_dim
 *   mscale  finite; 1 leaves magnitudes as they are (it scales the rotated
 *           dimensions only)
 */
typedef struct {
    const uint64_t *steps;
    int32_t rot_dim;
    int32_t interleaved;
    float mscale;
    int32_t reserved;      /* 0 */
} attn_rope;

/*
 * attn_rope_steps -- host-only: the rotation of each pair per position, as a
 * fraction of a turn in 64-bit fixed point, steps[i] = round(2^64 f_i / 2 pi),
 * written to steps[0 .. rot_dim / 2) in host memory. Position times step
 * modulo 2^64 is the angle of that position: the rounding of the step takes at
 * most |position| * pi * 2^-64 radians (4e-10 at position 2^31) beside what f_i,
 * computed in 64-bit floating point, is off by.
 *   rot_dim  as in attn_rope; base finite and >= 1; scaling ATTN_ROPE_*
 *   factor   > 0 and finite (not ATTN_ROPE_PLAIN), the enlarged base of
 *            ATTN_ROPE_BASE finite too; low_turns < high_turns and
 *            trained_len >= 1 for ATTN_ROPE_BANDS. f_i must stay below 2 pi.
 */
attn_status attn_rope_steps(int rot_dim, double base, int scaling, double factor, double low_turns,
                            double high_turns, int64_t trained_len, uint64_t *steps);

/*
 * attn_rope_append -- rotate the new tokens' queries and keys by their
 * positions and write their key and value rows into the cache, in one launch.
 *   block_table  int32 [n_seq][max_pages]
 *   positions    int32 [n_seq]: position of each sequence's LAST new token
 *   cu_tokens    int32 [n_seq + 1], non-decreasing from 0: sequence s has the tokens
 *                [cu_tokens[s], cu_tokens[s + 1]) at the positions that end at
 *                positions[s]; a sequence without tokens is left alone, and so
 *                are the rows of q_out at or past cu_tokens[n_seq] (a padded
 *                batch). NULL: n_tokens / n_seq tokens each (n_tokens must be a
 *                multiple of n_seq).
 *   q            [n_tokens][n_head][head_dim] of in_type, or NULL for none
 *   k_new, v_new [n_tokens][n_kv_head][head_dim] of in_type
 *   q_stride, k_stride, v_stride  elements from one token to the next (parts of
 *                one projection); 0: dense. A multiple of 16 bytes, at least one
 *                token's elements.
 *   in_type      ATTN_TYPE_F32, _F16 or _BF16
 *   q_out        float [n_tokens][n_head][head_dim], rotated: the q of
 *                attn_decode_paged. It may be q itself (F32, dense).
 *   rope         NULL: nothing is rotated (q is converted)
 * Sines, cosines and products are taken in 32 bits from the exact fixed-point
 * angle; each result is rounded once to the type it is stored in. E4M3: where a
 * call brings a page more rows than a sweep of its threads takes (8 or more),
 * the sines of up to three rows in four come from an earlier row's by 32-bit
 * products (within 31 * 2^-24 instead of 8 * 2^-24 of a pair's magnitude), so that an
 * element of K so near to the middle of two codes can take the other one
 * than in an append of fewer rows.
 * E4M3: the new rows of a page and head set its scale to the smallest power of
 * two s (2^-60 .. 2^60) with |x| <= 448 s, or, where the page holds rows before
 * them, to the magnitude of the scale it has if that is larger. The rows
 * before them keep their values: where the scale changes, each code becomes the
 * one nearest to its value at the new scale (with powers of two exact but for
 * values that fall below 2^-6 s; a scale of 0, negative or no power of two, of a
 * page filled elsewhere, is taken for what it is; one that is not finite counts
 * as none, and the codes stay). The first row of a page starts its scale
 * afresh. Infinite elements take the largest code, as those past 448 * 2^60
 * do, NaN stays NaN, and neither infinities nor NaN count for the scale.
 * Each page may be written by one sequence of the call only, and stand at one
 * place of its table (what a page written twice holds is not defined). A token whose
 * position lies outside [0, max_pages * page_size) is not written and sets
 * ATTN_DEVERR_POSITION_CLAMPED, except that positions[s] == -1 marks an idle
 * sequence; its q is rotated all the same.
 */
attn_status attn_rope_append(const attn_paged_cache *cache, const int32_t *block_table, int max_pages,
                             const int32_t *positions, const int32_t *cu_tokens, int n_seq,
                             int64_t n_tokens, const void *q, const void *k_new, const void *v_new,
                             int64_t q_stride, int64_t k_stride, int64_t v_stride, int in_type,
                             float *q_out, int n_head, const attn_rope *rope, attn_stream_t stream);

/*
 * What happens to a score between the product and the softmax, in this order:
 *   softcap  2^-40 .. 2^40: score = softcap * tanh(score / softcap); 0: none
 *   slopes   device, float [n_head], or NULL: score -= slopes[h] * (position of the
 *            query - j) for cache row j
 *   window   > 0: rows j <= position of the query - window are masked; 0: none
 *   starts   device, int32 [n_seq], or NULL: rows j < starts[s] are masked (left
 *            padding, or the first row of the document the queries belong to)
 * A query row that sees no cache row gives 0. Pages all of whose rows are
 * masked for every query row are not read.
 */
typedef struct {
    float softcap;
    int32_t window;
    const float *slopes;
    const int32_t *starts;
} attn_score_rules;

/*
 * attn_decode_paged -- decode attention over the paged cache.
 *   q, out       float [n_seq][n_q][n_head][head_dim]
 *   positions    int32 [n_seq]: position of each sequence's LAST query row; with
 *                nkv = clamp(positions[s] + 1, 0, max_pages * page_size) query
 *                row t has position nkv - n_q + t and sees the rows up to it.
 *                A positions[s] outside [-1, max_pages * page_size) sets
 *                ATTN_DEVERR_POSITION_CLAMPED.
 *   n_head       a multiple of n_kv_head, n_head / n_kv_head <= 64
 *   n_q          1 .. 1024
 *   scale        multiplies q.k
 *   rules        NULL: plain scores
 *   n_splits     blocks that share the call's rows, per KV head (and group of
 *                8 or 16 (query row, head) pairs): each takes an equal part of
 *                the rows of all sequences laid end to end; 0: attn_paged_plan's
 *                count, which fills the GPU once
 *   workspace    device buffer of the bytes attn_paged_plan reports, 256-byte
 *                aligned; NULL: the library-owned buffer (see attn_decode: one
 *                stream at a time, no growth while capturing, and graphs that
 *                may run at once need workspaces of their own).
 * q and the softmax weights are carried in 16-bit parts (two of binary16, 22
 * bits, or three of bfloat16, 24), sums in 32 bits, so that the result has about
 * the accuracy of 32-bit arithmetic on the values the cache stands for. Two parts
 * of binary16 (F16 and E4M3 caches) end at 2^-25: an element of q is carried to
 * 2^-22 of itself or 2^-39 of its row's largest, and a weight times the V scale
 * of its page to 2^-22 of itself or 2^-31 of the query row's largest such
 * product, whichever is more. So rows whose product lies r < 2^-9 times below
 * the largest count to 2^-31 / r of their part, which shows only in dimensions
 * where the rows of larger products hold about 0.
 */
attn_status attn_decode_paged(const attn_paged_cache *cache, const int32_t *block_table, int max_pages,
                              const int32_t *positions, const float *q, float *out, int n_seq, int n_q,
                              int n_head, float scale, const attn_score_rules *rules, int n_splits,
                              void *workspace, size_t workspace_bytes, attn_stream_t stream);

/*
 * attn_paged_plan -- host-only: n_splits and the workspace bytes (0 for one
 * split) of an attn_decode_paged call with these arguments; only the shape
 * fields of the cache are looked at. n_splits as in the call, window as in its rules (0:
 * none). sm_count <= 0 asks the current device. Either output may be NULL.
 */
attn_status attn_paged_plan(const attn_paged_cache *cache, int max_pages, int n_seq, int n_q, int n_head,
                            int window, int n_splits, int sm_count, int *n_splits_out,
                            size_t *workspace_bytes_out);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_PAGED_H */
