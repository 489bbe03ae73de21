/*
 * attn_tree.h -- C ABI of the operators of libattn_decode.so that decode with
 * drafted trees over a paged cache: several continuations of a sequence, sharing
 * their first tokens, are appended as one tree, attended in one call, and
 * the rows of the accepted path kept.
 *
 * The conventions of attn_decode.h and attn_paged.h hold: caller-owned,
 * 16-byte aligned device pointers (int32 arrays 4-byte aligned), argument errors
 * before anything is launched, data-dependent errors as bits of the sticky device
 * error word, nothing synchronises, every launch can be captured. Calls run on
 * the current device.
 *
 * Trees. Sequence s has n_s = cu_tokens[s + 1] - cu_tokens[s] nodes, tokens
 * cu_tokens[s] .. of the call; node t stands in cache row base_s + t, where
 * base_s = positions[s] + 1 - n_s rows hold the sequence up to the tree's root.
 * A node at depth d has position base_s + d. cu_tokens is int32 [n_seq + 1],
 * non-decreasing from 0; NULL: n_tokens / n_seq nodes each (n_tokens a multiple of
 * n_seq). A sequence without nodes is left alone, and so is what belongs to
 * tokens at or past cu_tokens[n_seq] (a padded batch). max_nodes (1 .. 1024)
 * bounds every n_s; a sequence with more sets ATTN_DEVERR_BAD_REQUEST and is
 * left alone.
 */
#ifndef ATTN_TREE_H
#define ATTN_TREE_H

#include "attn_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A tree, a path or a fork that is not one: it is skipped (a wrong parent: taken as a root). */
#define ATTN_DEVERR_BAD_REQUEST 0x8u

/*
 * attn_tree_rules -- which nodes each node sees, and its depth, from the parents.
 *   parents  int32 [n_tokens]: a node's parent, counted from its sequence's first
 *            node; negative: it hangs on the sequence itself (depth 0). In any
 *            order. A parent outside the tree counts as none, a node whose parents
 *            run in a circle sees what was met until then; both set
 *            ATTN_DEVERR_BAD_REQUEST.
 *   mask     uint32 [n_tokens][(max_nodes + 31) / 32]: bit j % 32 of word j / 32
 *            of a node's row is set where it sees node j: itself and its ancestors
 *   depths   int32 [n_tokens]
 */
attn_status attn_tree_rules(const int32_t *parents, const int32_t *cu_tokens, int n_seq, int64_t n_tokens,
                            int max_nodes, uint32_t *mask, int32_t *depths, attn_stream_t stream);

/*
 * attn_rope_append_tree -- attn_rope_append for the nodes of trees: rows as
 * there, node t of sequence s in row base_s + t, its q and k rotated by its
 * position base_s + depths[token]. So a node keeps its rotation when
 * attn_keep_rows moves it to the row of its depth.
 *   depths    int32 [n_tokens], or NULL: a chain, as attn_rope_append
 *   q_out     [n_tokens][n_head][head_dim] of out_type
 *   out_type  ATTN_TYPE_F32, or in_type: rounded once; of in_type, q_out may be q
 *             itself (dense)
 * E4M3: each row's angle is computed from its position.
 */
attn_status attn_rope_append_tree(const attn_paged_cache *cache, const int32_t *block_table, int max_pages,
                                  const int32_t *positions, const int32_t *cu_tokens, int n_seq,
                                  int64_t n_tokens, const void *q, const void *k_new, const void *v_new,
                                  int64_t q_stride, int64_t k_stride, int64_t v_stride, int in_type,
                                  void *q_out, int out_type, int n_head, const attn_rope *rope,
                                  const int32_t *depths, attn_stream_t stream);

/*
 * attn_decode_tree -- attention of the nodes of trees over the paged cache. Node t
 * of sequence s sees the rows before base_s and row base_s + j where bit j of its
 * mask row is set. A node that sees nothing gives 0.
 *   positions  int32 [n_seq]: the row of each sequence's LAST node. With
 *              nkv = clamp(positions[s] + 1, 0, max_pages * page_size), base_s =
 *              nkv - n_s; where that is negative, the nodes in front of row 0 have
 *              no row and are seen by none. A positions[s] outside
 *              [-1, max_pages * page_size) sets ATTN_DEVERR_POSITION_CLAMPED.
 *   q, out     [n_tokens][n_head][head_dim] of q_type (F32, F16 or BF16)
 *   mask       uint32 [n_tokens][mask_words], mask_words >= (max_nodes + 31) / 32, any
 *              bits (attn_tree_rules makes a tree's); bits at or past n_s are not
 *              looked at. NULL: a chain, node t sees nodes 0 .. t.
 *   depths     int32 [n_tokens], 0 .. max_nodes - 1 (others are taken as the
 *              nearest of these), or NULL: node t has depth t. Only slopes and
 *              window look at it.
 *   rules      as in attn_decode_paged, with distances by position: query
 *              base_s + depth, cache row j < base_s at position j, node j at base_s + its
 *              depth. starts masks rows (of nodes too), whatever their position.
 *   n_head     a multiple of n_kv_head, n_head / n_kv_head <= 64
 *   n_splits   blocks that share the call's rows, per KV head and 128 of its
 *              (node, head) pairs: each takes an equal part of the tiles (128 rows, 64
 *              at head_dim 256) of all sequences; 0: attn_tree_plan's count: as
 *              many as make a block an SM, or, where that leaves more than 15 % of
 *              the SMs without one, up to four blocks an SM, in turn
 *   workspace  device buffer of the bytes attn_tree_plan reports, 256-byte
 *              aligned; NULL: the library-owned buffer (see attn_decode). One split
 *              needs some too where F32 queries may have more than 2048 rows
 * Rows that a node does not see never change its result, whatever they hold, and
 * neither do pages that are not there (ATTN_DEVERR_BAD_PAGE). Rows that
 * are seen are taken to hold finite values, as in attn_decode_paged. A query with an
 * infinity or NaN gives NaN (0 where it sees nothing), and changes no other (with
 * a softcap: none beyond its accuracy).
 * Scores, softmax statistics and sums are 32 bits. The tensor cores, which add the
 * rows up, cut a sum off at 24 bits at every 16 rows: with F32 queries no more than
 * 2048 rows are added up so (some 5e-6 of the result), with 16-bit ones all that a
 * block has of a sequence (1e-4 of it after 30000 rows). q and the weights enter the
 * products in 16-bit parts: with F32 queries two each (of binary16, 22 bits, over F16
 * and E4M3 caches; of bfloat16, 16 bits, over BF16 ones, fewer than the 24 that
 * attn_decode_paged carries there). 16-bit queries enter as they are (F16 over a
 * BF16 cache: two parts), their weights as two parts where the query has the
 * cache's type, or is F16 over a BF16 cache, else as one of binary16: 11 bits,
 * which beside the rounding of a BF16 result adds 1 % and beside that of an F16
 * one (over E4M3) two fifths. 16-bit queries over an E4M3 cache enter as two or
 * three 8-bit parts that hold all their bits, but for what lies below 2^-17 of
 * their row's largest. So the queries' type chooses: F32 ones give weights and
 * results more bits, at up to 1.8 times the time.
 */
attn_status attn_decode_tree(const attn_paged_cache *cache, const int32_t *block_table, int max_pages,
                             const int32_t *positions, const int32_t *cu_tokens, int n_seq, int64_t n_tokens,
                             int max_nodes, const void *q, void *out, int q_type, int n_head, float scale,
                             const uint32_t *mask, int mask_words, const int32_t *depths,
                             const attn_score_rules *rules, int n_splits, void *workspace,
                             size_t workspace_bytes, attn_stream_t stream);

/*
 * attn_tree_plan -- host-only: n_splits and the workspace bytes of an
 * attn_decode_tree call with these arguments; only the shape fields of the cache are
 * looked at. sm_count <= 0 asks the current device. Either output may be NULL.
 */
attn_status attn_tree_plan(const attn_paged_cache *cache, int max_pages, int n_seq, int64_t n_tokens,
                           int max_nodes, int q_type, int n_head, int n_splits, int sm_count,
                           int *n_splits_out, size_t *workspace_bytes_out);

/*
 * attn_keep_rows -- keep some of the rows behind a sequence's row base[s], in
 * their order, and close the gaps: row base[s] + path[s][i] becomes row base[s] + i
 * for i < counts[s]. After a step with trees: the accepted path.
 *   base    int32 [n_seq]
 *   path    int32 [n_seq][max_keep], its first counts[s] entries strictly
 *           increasing from 0 or more
 *   counts  int32 [n_seq], 0 .. max_keep; 0: the sequence is left alone
 * 16-bit caches: a copy. E4M3: as if the rows' values were appended at base[s] with
 * attn_rope_append (its rules on a page's scale; rows before base[s] keep their
 * values). Rows behind the last kept one hold what they held, but an E4M3 page's
 * scale may have changed under them.
 * A path that is not increasing, or leads out of [0, max_pages * page_size), or a
 * count outside 0 .. max_keep sets ATTN_DEVERR_BAD_REQUEST, and the sequence is left
 * alone; a row on a page that is not there, or that should go to one, is not moved
 * (ATTN_DEVERR_BAD_PAGE). No other sequence may hold the pages that are written.
 */
attn_status attn_keep_rows(const attn_paged_cache *cache, const int32_t *block_table, int max_pages,
                           const int32_t *base, const int32_t *path, const int32_t *counts, int n_seq,
                           int max_keep, attn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_TREE_H */
