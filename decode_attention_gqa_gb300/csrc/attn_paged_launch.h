// attn_paged_launch.h -- internal host interface of the paged-cache operators:
// between their C-ABI layer (attn_paged_api.cu), the kernel translation units
// (attn_paged_hd*.cu, attn_rope_append.cu) and the device state that
// attn_api.cu owns. Not installed; not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace attn {

constexpr int kTypeF32 = 0, kTypeF16 = 1, kTypeBf16 = 2, kTypeE4m3 = 3;   // ATTN_TYPE_*

// Shape of the paged kernel for (head_dim, bytes of an element, slots).
struct PagedShape {
    int nsl;                  // 16-row slices of a stage
    int warps;                // compute warps: a multiple of nsl
    int stages;               // a multiple of warps / nsl, so that a stage is always the same warps'
    int blocks;               // resident blocks per SM
};

// 130 to 190 KB of stages on an SM, in as many blocks as the accumulators (head_dim / 4 registers a thread for 8
// slots, head_dim / 2 for 16) leave room for: the more warps, the better they hide each other's latency
// (head_dim 64, 8 bits, 8 slots: a ragged batch 106 us with three blocks an SM, 97 with four; 16 bits, 16 slots, 65000 rows:
// 49.6 with two, 42.1 with three). Where the registers would have to be squeezed further, it does not pay
// (head_dim 256, 8 bits, 8 slots: draft rows 22.9 with two blocks, 23.3 with three and spills).
constexpr PagedShape paged_shape(int head_dim, int es, int slots)
{
    return es == 1 ? (head_dim == 64    ? (slots == 8 ? PagedShape{4, 4, 5, 4} : PagedShape{4, 4, 6, 3})
                      : head_dim == 128 ? (slots == 8 ? PagedShape{4, 4, 4, 3} : PagedShape{4, 4, 6, 2})
                                        : (slots == 8 ? PagedShape{4, 4, 3, 2} : PagedShape{2, 6, 12, 1}))
                   : (head_dim == 64    ? (slots == 8 ? PagedShape{4, 4, 3, 4} : PagedShape{4, 4, 4, 3})
                      : head_dim == 128 ? PagedShape{4, 4, 3, 2}
                                        : PagedShape{2, 6, 6, 1});
}

constexpr int kPagedSeqs = 128;   // sequences one launch takes

// Division of 0 <= n < 2^31 by a divisor known on the host: (mulhi(n, mul) + n) >> shift.
struct FastDiv {
    unsigned mul, shift;
};

inline FastDiv fast_div(unsigned d)
{
    unsigned s = 0;
    while (s < 31 && (1u << s) < d) ++s;
    return FastDiv{(unsigned)((((uint64_t)1 << 32) * (((uint64_t)1 << s) - d)) / d + 1), s};
}

#ifdef __CUDACC__
__device__ __forceinline__ int div(const FastDiv &d, int n)
{
    return (int)((__umulhi((unsigned)n, d.mul) + (unsigned)n) >> d.shift);
}
#endif

struct PagedArgs {
    const float *q;           // [n_seq][n_q][n_head][HD]
    float *out;
    const int32_t *positions; // [n_seq]
    const int32_t *table;     // [n_seq][max_pages]
    const float *k_scale;     // [n_pages][n_kv_head], e4m3 only
    const float *v_scale;
    const float *slopes;      // [n_head] or null
    const int32_t *starts;    // [n_seq] or null
    // Partial results: row ((rank * 2 + which) * units + unit) * slots + slot, `which` 1 where the
    // sequence began in this rank's rows, 0 where it began before them
    float *ws_o;              // [rows][HD]
    float2 *ws_ml;            // [rows]
    int2 *ws_span;            // [n_seq]: first and last rank that has rows of the sequence
    unsigned *err;
    int n_seq;                // at most kPagedSeqs
    int n_head, n_kv_head, group, n_q;
    int qgroups;              // blocks per (rank, KV head) along the (query row, head) slots
    int units;                // n_kv_head * qgroups
    int ranks;                // blocks that share the rows, per unit
    int turn;                 // what going to the next sequence costs a block, in tiles
    int max_pages, n_pages, page_size;
    int cap;                  // max_pages * page_size
    int window;               // 0: none
    int box_rows;             // rows of one TMA box: a power of two that divides the page and the stage
    FastDiv by_page, by_group, by_ranks;
    float qscale;             // scale * log2 e, or scale / softcap
    float cap_log2;           // softcap * log2 e, or 0
};

struct PagedRequest {
    PagedArgs pa;
    const void *k, *v;
    int64_t page_stride, row_stride, head_stride;   // elements
    int head_dim, kv_type;
    bool rules;               // softcap or slopes
    int slots;                // (query row, head) slots of a block: 8 or 16
    cudaStream_t stream;
};

cudaError_t launch_paged_hd64_f16(const PagedRequest &r);
cudaError_t launch_paged_hd64_bf16(const PagedRequest &r);
cudaError_t launch_paged_hd64_e4m3(const PagedRequest &r);
cudaError_t launch_paged_hd128_f16(const PagedRequest &r);
cudaError_t launch_paged_hd128_bf16(const PagedRequest &r);
cudaError_t launch_paged_hd128_e4m3(const PagedRequest &r);
cudaError_t launch_paged_hd256_f16(const PagedRequest &r);
cudaError_t launch_paged_hd256_bf16(const PagedRequest &r);
cudaError_t launch_paged_hd256_e4m3(const PagedRequest &r);

struct AppendArgs {
    const void *q, *k_new, *v_new;
    void *q_out;                                    // float, or the input's type (q_in_type)
    int64_t q_stride, k_stride, v_stride;           // elements between tokens
    void *k, *v;
    float *k_scale, *v_scale;
    int64_t page_stride, row_stride, head_stride;   // elements
    const int32_t *table, *positions, *cu;
    const int32_t *depths;                          // of each token in its tree, or null: a chain
    const uint64_t *steps;                          // null: no rotation
    unsigned *err;
    float mscale;
    int rot_dim, interleaved;
    bool q_in_type;
    int n_seq, n_head, n_kv_head;
    int64_t n_tokens;
    int64_t n_each;                                 // tokens per sequence when cu is null
    int max_pages, n_pages, page_size;
    int64_t page_items;                             // (sequence, page) candidates, e4m3 only
    int64_t page_blocks;                            // blocks of page jobs, before those of token jobs
    bool kv_apart;                                  // page jobs take K or V, not both
    bool wide;                                      // every row and head starts at a multiple of 32 bytes
    int iters;                                      // head groups one warp takes for its token
    int chunks;                                     // warps per token
    // Every number of tokens, pages and jobs is below 2^31; a 64-bit division took a warp some 500 cycles, and a job's
    // place half a dozen of them (one token 4.2 -> 3.8 us)
    FastDiv by_page, by_chunks, by_each, by_item, by_seq;   // page_size, chunks, n_each; jobs of a page, pages of a sequence
};

struct AppendRequest {
    AppendArgs a;
    int head_dim, in_type, kv_type;
    cudaStream_t stream;
};

cudaError_t launch_append(const AppendRequest &r);

// Trees: rules from parents, and the rows that are kept.
struct TreeRulesArgs {
    const int32_t *parents, *cu;
    uint32_t *mask;
    int32_t *depths;
    unsigned *err;
    int64_t n_tokens, n_each;                       // n_each: nodes of a sequence when cu is null
    int n_seq, max_nodes, words;
};
cudaError_t launch_tree_rules(const TreeRulesArgs &a, cudaStream_t stream);

struct KeepArgs {
    uint8_t *k, *v;
    float *k_scale, *v_scale;
    int64_t page_stride, row_stride, head_stride;   // bytes
    const int32_t *table, *base, *path, *counts;
    unsigned *err;
    int n_seq, n_kv_head, max_keep, max_pages, n_pages, page_size;
    int row_bytes;                                  // of one head: 64 .. 512
    FastDiv by_page;
};
cudaError_t launch_keep_rows(const KeepArgs &a, bool e4m3, cudaStream_t stream);

// Attention of trees.
struct TreeArgs {
    const void *q;            // [n_tokens][n_head][HD] of q_type
    void *out;
    const void *v;            // the pool again, for rows that are added one by one
    int64_t page_stride, row_stride, head_stride;   // elements
    const int32_t *positions, *cu, *table, *starts; // of the launch's sequences
    const int32_t *depths;    // of all tokens, or null
    const uint32_t *mask;     // [n_tokens][words] or null: chains
    const float *k_scale, *v_scale, *slopes;
    // Parts: block (rank * 2 + which) * units + unit of kTreeSlots slots, `which` 1 where the sequence begins in this
    // rank's places. On the way to a part, or to an output, sums of f32 queries' (one rank: block `unit`)
    float *ws_o;              // [blocks][HD / 4][kTreeSlots][4]
    float2 *ws_ml;            // [blocks][kTreeSlots]
    int4 *ws_span;            // [units / n_kv_head][n_seq]: first place, tiles, first token, places of a rank
    unsigned *err;
    int64_t n_tokens, n_each; // n_each: nodes of a sequence when cu is null
    int64_t tok_end;          // tokens the joining kernel looks at
    int q_type, n_seq, seq0;  // sequences of the launch (at most kTreeSeqs), the first one's number
    int max_nodes, words;
    int n_head, n_kv_head, group;
    int max_pages, n_pages, page_size, cap, window;
    int units;                // n_kv_head times what max_nodes has of kTreeSlots
    int ranks;                // blocks that share a unit's tiles
    int fold;                 // tree_fold
    int q_parts;              // parts of q
    uint32_t q_bytes;         // of Q in shared memory
    int nk, nv, nrk, nrv;     // tiles of the rings of K and V, and of their 8-bit tiles that are converted
    int box_rows;             // rows of one TMA box
    bool once;                // no other block reads the same rows
    float qscale;             // scale * log2 e, or scale / softcap
    float softcap, cap_log2;  // 0: none; softcap * log2 e
    FastDiv by_page, by_group;
};

struct TreeRequest {
    TreeArgs a;
    const void *k, *v;
    int64_t page_stride, row_stride, head_stride;   // elements
    int head_dim, kv_type;
    int parts, weight_parts;  // 16-bit parts of q and of the weights
    cudaStream_t stream;
};
constexpr int kTreeSeqs = 64;     // sequences one launch of the attention of trees takes
constexpr int kTreeSlots = 128;         // (node, head) pairs of a KV head that a block serves
constexpr int tree_tile(int head_dim) { return head_dim == 256 ? 64 : 128; }
// 16-bit parts of q: one holds a 16-bit query, but for f16's in bfloat16
constexpr int tree_parts(int q_type, int kv_type) { return q_type == kTypeF32 || (q_type == kTypeF16 && kv_type == kTypeBf16) ? 2 : 1; }
// Tiles, a power of two of them, after which O is added to a sum in the workspace (see "Sums" in attn_tree.cuh)
constexpr int tree_fold(int head_dim, int q_type, int kv_type)
{
    return tree_parts(q_type, kv_type) == 1 ? 1 << 30 : (q_type == kTypeF16 ? 16384 : 2048) / tree_tile(head_dim);
}
cudaError_t launch_tree_hd64_f16(const TreeRequest &r);
cudaError_t launch_tree_hd64_bf16(const TreeRequest &r);
cudaError_t launch_tree_hd64_e4m3(const TreeRequest &r);
cudaError_t launch_tree_hd128_f16(const TreeRequest &r);
cudaError_t launch_tree_hd128_bf16(const TreeRequest &r);
cudaError_t launch_tree_hd128_e4m3(const TreeRequest &r);
cudaError_t launch_tree_hd256_f16(const TreeRequest &r);
cudaError_t launch_tree_hd256_bf16(const TreeRequest &r);
cudaError_t launch_tree_hd256_e4m3(const TreeRequest &r);

// Implemented in attn_api.cu.
// The current device's SM count and error word.
cudaError_t device_facts(int *sm_count, unsigned **err_word);
// The library-owned workspace of the current device, grown to `need` bytes
// outside capture. *ok false: it would have to grow while `stream` captures.
cudaError_t owned_workspace(size_t need, cudaStream_t stream, void **ws, bool *ok);
// A paged pool as a 4-D tensor (x = element, y = KV head, z = row, w = page) with
// a box of (box_x, 1, box_rows, 1); strides in bytes; swizzled as wide as the box's rows.
cudaError_t encode_paged_map(CUtensorMap *map, const void *base, int elem_bytes, bool bf16, int head_dim,
                             int n_kv_head, int page_size, int n_pages, int64_t head_bytes,
                             int64_t row_bytes, int64_t page_bytes, int box_x, int box_rows);
// Remembers the error for attn_last_cuda_error.
void note_cuda_error(cudaError_t e);

} // namespace attn
