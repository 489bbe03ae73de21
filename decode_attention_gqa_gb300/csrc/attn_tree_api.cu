// attn_tree_api.cu -- the C ABI of include/attn_tree.h: argument checks, the plan and the dispatch.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "attn_launch.h"
#include "attn_paged_check.h"
#include "attn_paged_launch.h"
#include "attn_tree.h"

namespace {

using namespace attn::check;

constexpr int kMaxTreeSplits = 4096;

attn_status check_trees(const int32_t *cu_tokens, int n_seq, int64_t n_tokens, int max_nodes)
{
    if (n_seq < 0 || n_seq > 65535 || n_tokens < 0 || n_tokens > kMaxRows || max_nodes < 1 || max_nodes > 1024)
        return ATTN_ERR_INVALID_ARG;
    if (n_seq == 0 && n_tokens != 0) return ATTN_ERR_INVALID_ARG;
    if (!cu_tokens && n_seq > 0 && (n_tokens % n_seq != 0 || n_tokens / n_seq > max_nodes)) return ATTN_ERR_INVALID_ARG;
    if (!aligned(cu_tokens, 4)) return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}

attn_status check_call(const attn_paged_cache *c, int q_type, int n_head, int n_splits)
{
    if (q_type != ATTN_TYPE_F32 && q_type != ATTN_TYPE_F16 && q_type != ATTN_TYPE_BF16) return ATTN_ERR_INVALID_ARG;
    if (n_head < 1 || n_head > 65535 || n_head % c->n_kv_head != 0 || n_splits < 0 || n_splits > kMaxTreeSplits)
        return ATTN_ERR_INVALID_ARG;
    if (n_head / c->n_kv_head > 64) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

struct TreePlan {
    int64_t units = 1;
    int n_splits = 1, tile = 128;
    size_t o_bytes = 0, ml_bytes = 0, workspace = 0;
};

// As many blocks for each unit (KV head, 128 slots) as make a block an SM; where that leaves more than 15 % of the SMs without
// one (units just over half of them), enough for four rounds of blocks, whose last is nearly full; no more than
// there are pairs of tiles at full capacity: the two warpgroups of a block take tiles in turn.
void make_plan(const attn_paged_cache *c, int max_pages, int n_seq, int max_nodes, int q_type, int n_head, int n_splits,
               int sm_count, TreePlan &pl)
{
    const int need = max_nodes * (n_head / c->n_kv_head);
    pl.tile = attn::tree_tile(c->head_dim);
    const int64_t mus = (need + attn::kTreeSlots - 1) / attn::kTreeSlots;
    pl.units = c->n_kv_head * mus;
    const int64_t seqs = n_seq < attn::kTreeSeqs ? n_seq : attn::kTreeSeqs;
    const int64_t tiles = ((int64_t)max_pages * c->page_size + pl.tile - 1) / pl.tile * seqs;
    const int64_t most = (tiles + 1) / 2;
    int64_t P = sm_count / pl.units;
    if (P * pl.units * 20 < (int64_t)sm_count * 17) P = 4 * (int64_t)sm_count / pl.units;
    if (P > most) P = most;
    if (P > kMaxTreeSplits) P = kMaxTreeSplits;
    pl.n_splits = n_splits > 0 ? n_splits : P < 1 ? 1 : (int)P;
    if (pl.n_splits > 1) {
        const size_t parts = (size_t)pl.n_splits * 2 * pl.units * attn::kTreeSlots;
        pl.o_bytes = align256(parts * c->head_dim * sizeof(float));
        pl.ml_bytes = align256(parts * 2 * sizeof(float));
        pl.workspace = pl.o_bytes + pl.ml_bytes + align256((size_t)(seqs * mus) * 16);
    } else if (((int64_t)max_pages * c->page_size + pl.tile - 1) / pl.tile > attn::tree_fold(c->head_dim, q_type, c->kv_type)) {
        pl.workspace = pl.o_bytes = align256((size_t)pl.units * attn::kTreeSlots * c->head_dim * sizeof(float));
    }
}

} // namespace

extern "C" {

attn_status attn_tree_rules(const int32_t *parents, const int32_t *cu_tokens, int n_seq, int64_t n_tokens,
                            int max_nodes, uint32_t *mask, int32_t *depths, attn_stream_t stream)
{
    const attn_status st = check_trees(cu_tokens, n_seq, n_tokens, max_nodes);
    if (st != ATTN_OK) return st;
    if (!aligned(parents, 4) || !aligned(mask, 4) || !aligned(depths, 4)) return ATTN_ERR_INVALID_ARG;
    if (n_tokens > 0 && (!parents || !mask || !depths)) return ATTN_ERR_INVALID_ARG;
    if (n_tokens == 0) return ATTN_OK;
    attn::TreeRulesArgs a{};
    a.parents = parents;
    a.cu = cu_tokens;
    a.mask = mask;
    a.depths = depths;
    a.n_tokens = n_tokens;
    a.n_each = cu_tokens ? 0 : n_tokens / n_seq;
    a.n_seq = n_seq;
    a.max_nodes = max_nodes;
    a.words = (max_nodes + 31) / 32;
    const cudaError_t e = attn::launch_tree_rules(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : fail(e);
}

attn_status attn_tree_plan(const attn_paged_cache *cache, int max_pages, int n_seq, int64_t n_tokens, int max_nodes,
                           int q_type, int n_head, int n_splits, int sm_count, int *n_splits_out,
                           size_t *workspace_bytes_out)
{
    Strides cs;
    const attn_status st = check_cache_shape(cache, max_pages, cs);
    if (st == ATTN_ERR_INVALID_ARG) return st;
    attn_status s2 = check_trees(nullptr, n_seq, 0, max_nodes);
    if (s2 == ATTN_OK && (n_tokens < 1 || n_tokens > kMaxRows || n_seq < 1)) s2 = ATTN_ERR_INVALID_ARG;   // nothing to plan
    if (s2 == ATTN_OK) s2 = check_call(cache, q_type, n_head, n_splits);
    if (s2 != ATTN_OK) return s2;
    if (st != ATTN_OK) return st;
    if (sm_count <= 0) {
        unsigned *err = nullptr;
        const cudaError_t e = attn::device_facts(&sm_count, &err);
        if (e != cudaSuccess) return fail(e);
    }
    TreePlan pl;
    make_plan(cache, max_pages, n_seq, max_nodes, q_type, n_head, n_splits, sm_count, pl);
    if (n_splits_out) *n_splits_out = pl.n_splits;
    if (workspace_bytes_out) *workspace_bytes_out = pl.workspace;
    return ATTN_OK;
}

attn_status attn_decode_tree(const attn_paged_cache *cache, const int32_t *block_table, int max_pages,
                             const int32_t *positions, const int32_t *cu_tokens, int n_seq, int64_t n_tokens,
                             int max_nodes, const void *q, void *out, int q_type, int n_head, float scale,
                             const uint32_t *mask, int mask_words, const int32_t *depths,
                             const attn_score_rules *rules, int n_splits, void *workspace, size_t workspace_bytes,
                             attn_stream_t stream)
{
    attn_status st = check_cache_pointers(cache);
    if (st != ATTN_OK) return st;
    if (!std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
    const attn_status tr = check_trees(cu_tokens, n_seq, n_tokens, max_nodes);
    if (tr != ATTN_OK) return tr;
    if (n_tokens > 0 && (!block_table || !positions || !q || !out)) return ATTN_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16)) return ATTN_ERR_INVALID_ARG;
    for (const void *p : {static_cast<const void *>(block_table), static_cast<const void *>(positions),
                          static_cast<const void *>(mask), static_cast<const void *>(depths)})
        if (!aligned(p, 4)) return ATTN_ERR_INVALID_ARG;
    if (mask && (mask_words < (max_nodes + 31) / 32 || mask_words > 1024)) return ATTN_ERR_INVALID_ARG;
    const float softcap = rules ? rules->softcap : 0.f;
    const int window = rules ? rules->window : 0;
    if (!(softcap == 0.f || (softcap >= 0x1p-40f && softcap <= 0x1p40f)) || window < 0) return ATTN_ERR_INVALID_ARG;
    const float qscale = softcap > 0.f ? (float)((double)scale / softcap) : (float)((double)scale * 1.4426950408889634);
    if (!std::isfinite(qscale)) return ATTN_ERR_INVALID_ARG;
    if (rules && (!aligned(rules->slopes, 4) || !aligned(rules->starts, 4))) return ATTN_ERR_INVALID_ARG;
    // distances of a tree's nodes need their depths
    if (mask && !depths && rules && (rules->slopes || window > 0)) return ATTN_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return ATTN_ERR_INVALID_ARG;
    Strides cs;
    st = check_cache_shape(cache, max_pages, cs);
    if (st == ATTN_ERR_INVALID_ARG) return st;
    const attn_status sh = check_call(cache, q_type, n_head, n_splits);
    if (sh != ATTN_OK) return sh;
    if (st != ATTN_OK) return st;
    if (n_tokens == 0) return ATTN_OK;

    attn::TreeRequest r{};
    attn::TreeArgs &a = r.a;
    int sm_count = 0;
    cudaError_t e = attn::device_facts(&sm_count, &a.err);
    if (e != cudaSuccess) return fail(e);
    TreePlan pl;
    make_plan(cache, max_pages, n_seq, max_nodes, q_type, n_head, n_splits, sm_count, pl);
    if (pl.units > 0x7fffffff) return ATTN_ERR_UNSUPPORTED;
    if (pl.workspace > 0) {
        if (!workspace) {
            bool ok = false;
            e = attn::owned_workspace(pl.workspace, reinterpret_cast<cudaStream_t>(stream), &workspace, &ok);
            if (e != cudaSuccess) return fail(e);
            if (!ok) return ATTN_ERR_WORKSPACE;
        } else if (workspace_bytes < pl.workspace) {
            return ATTN_ERR_WORKSPACE;
        }
    }
    a.q = q;
    a.out = out;
    a.v = cache->v;
    a.page_stride = cs.page;
    a.row_stride = cs.row;
    a.head_stride = cs.head;
    a.depths = depths;
    a.mask = mask;
    a.k_scale = cache->k_scale;
    a.v_scale = cache->v_scale;
    a.slopes = rules ? rules->slopes : nullptr;
    if (pl.workspace > 0) {
        uint8_t *ws = static_cast<uint8_t *>(workspace);
        a.ws_o = reinterpret_cast<float *>(ws);
        a.ws_ml = reinterpret_cast<float2 *>(ws + pl.o_bytes);
        a.ws_span = reinterpret_cast<int4 *>(ws + pl.o_bytes + pl.ml_bytes);
    }
    a.n_tokens = n_tokens;
    a.n_each = cu_tokens ? 0 : n_tokens / n_seq;
    a.q_type = q_type;
    a.max_nodes = max_nodes;
    a.words = mask ? mask_words : 0;
    a.n_head = n_head;
    a.n_kv_head = cache->n_kv_head;
    a.group = n_head / cache->n_kv_head;
    a.max_pages = max_pages;
    a.n_pages = cache->n_pages;
    a.page_size = cache->page_size;
    a.cap = max_pages * cache->page_size;
    // past every distance it masks nothing: a node may be as deep as max_nodes - 1 behind the last row
    a.window = window >= a.cap + max_nodes ? 0 : window;
    a.ranks = pl.n_splits;
    a.fold = attn::tree_fold(cache->head_dim, q_type, cache->kv_type);
    a.once = (int64_t)max_nodes * a.group <= attn::kTreeSlots;
    a.qscale = qscale;
    a.softcap = softcap;
    a.cap_log2 = (float)((double)softcap * 1.4426950408889634);
    a.by_page = attn::fast_div((unsigned)cache->page_size);
    a.by_group = attn::fast_div((unsigned)a.group);
    r.k = cache->k;
    r.v = cache->v;
    r.page_stride = cs.page;
    r.row_stride = cs.row;
    r.head_stride = cs.head;
    r.head_dim = cache->head_dim;
    r.kv_type = cache->kv_type;
    r.parts = attn::tree_parts(q_type, cache->kv_type);
    // One part of a weight carries as many bits as a result of the cache's own 16-bit type: both roundings together are off by
    // 1.4 times the result's own, by up to 2.2 where few rows weigh. Two parts leave the result's; over e4m3, where they take
    // a quarter of the time more (32 sequences of up to 32768 rows 222 -> 279 us; over 16 bits 0 to 17 %), one is kept.
    r.weight_parts = r.parts == 2 || q_type == cache->kv_type ? 2 : 1;
    r.stream = reinterpret_cast<cudaStream_t>(stream);
    using Launch = cudaError_t (*)(const attn::TreeRequest &);
    static const Launch table[3][3] = {
        {attn::launch_tree_hd64_f16, attn::launch_tree_hd64_bf16, attn::launch_tree_hd64_e4m3},
        {attn::launch_tree_hd128_f16, attn::launch_tree_hd128_bf16, attn::launch_tree_hd128_e4m3},
        {attn::launch_tree_hd256_f16, attn::launch_tree_hd256_bf16, attn::launch_tree_hd256_e4m3}};
    const Launch launch = table[cache->head_dim == 64 ? 0 : cache->head_dim == 128 ? 1 : 2][cache->kv_type - ATTN_TYPE_F16];
    a.units = (int)pl.units;
    // tiles are counted in 32 bits: fewer sequences a launch where the capacity is huge
    const int64_t per_seq = ((int64_t)a.cap + pl.tile - 1) / pl.tile + 1;
    const int batch = (int)(0x3fff0000 / per_seq < attn::kTreeSeqs ? 0x3fff0000 / per_seq : attn::kTreeSeqs);
    for (int s0 = 0; s0 < n_seq; s0 += batch) {
        a.n_seq = n_seq - s0 < batch ? n_seq - s0 : batch;
        a.seq0 = s0;
        a.positions = positions + s0;
        a.cu = cu_tokens ? cu_tokens + s0 : nullptr;
        a.table = block_table + (size_t)s0 * max_pages;
        a.starts = rules && rules->starts ? rules->starts + s0 : nullptr;
        a.tok_end = cu_tokens ? n_tokens : (s0 + a.n_seq) * a.n_each;
        e = launch(r);
        if (e != cudaSuccess) return fail(e);
    }
    return ATTN_OK;
}

attn_status attn_keep_rows(const attn_paged_cache *cache, const int32_t *block_table, int max_pages,
                           const int32_t *base, const int32_t *path, const int32_t *counts, int n_seq, int max_keep,
                           attn_stream_t stream)
{
    attn_status st = check_cache_pointers(cache);
    if (st != ATTN_OK) return st;
    if (n_seq < 0 || n_seq > 65535 || max_keep < 0 || max_keep > kMaxRows) return ATTN_ERR_INVALID_ARG;
    const bool any = n_seq > 0 && max_keep > 0;
    if (any && (!block_table || !base || !path || !counts)) return ATTN_ERR_INVALID_ARG;
    for (const int32_t *p : {block_table, base, path, counts})
        if (!aligned(p, 4)) return ATTN_ERR_INVALID_ARG;
    Strides cs;
    st = check_cache_shape(cache, max_pages, cs);
    if (st != ATTN_OK) return st;
    if (!any) return ATTN_OK;
    const int64_t es = type_bytes(cache->kv_type);
    attn::KeepArgs a{};
    a.k = static_cast<uint8_t *>(cache->k);
    a.v = static_cast<uint8_t *>(cache->v);
    a.k_scale = cache->k_scale;
    a.v_scale = cache->v_scale;
    a.page_stride = cs.page * es;
    a.row_stride = cs.row * es;
    a.head_stride = cs.head * es;
    a.table = block_table;
    a.base = base;
    a.path = path;
    a.counts = counts;
    a.n_seq = n_seq;
    a.n_kv_head = cache->n_kv_head;
    a.max_keep = max_keep;
    a.max_pages = max_pages;
    a.n_pages = cache->n_pages;
    a.page_size = cache->page_size;
    a.row_bytes = (int)(cache->head_dim * es);
    const cudaError_t e = attn::launch_keep_rows(a, cache->kv_type == ATTN_TYPE_E4M3, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : fail(e);
}

} // extern "C"
