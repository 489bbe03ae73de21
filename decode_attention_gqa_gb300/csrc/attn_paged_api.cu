// attn_paged_api.cu -- the C ABI of include/attn_paged.h: argument checks, the
// rotary steps, the split plan and the dispatch to the kernels.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "attn_launch.h"
#include "attn_paged.h"
#include "attn_paged_check.h"
#include "attn_paged_launch.h"
#include "attn_tree.h"

namespace {

using namespace attn::check;

constexpr int kMaxPagedSplits = 4096;
struct PagedPlan {
    attn::PagedShape shape{};
    int slots = 8, qgroups = 1, n_splits = 1;
    size_t o_bytes = 0, ml_bytes = 0, workspace = 0;
};

attn_status check_heads(const attn_paged_cache *c, int n_seq, int n_q, int n_head, int window, int n_splits)
{
    if (n_seq < 0 || n_seq > 65535 || n_q < 1 || n_q > 1024 || n_head < 1 || n_head % c->n_kv_head != 0 || window < 0 ||
        n_splits < 0 || n_splits > kMaxPagedSplits)
        return ATTN_ERR_INVALID_ARG;
    if (n_head / c->n_kv_head > 64) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

// How many blocks share the call's rows, per KV head and group of slots: as many as fill the SMs with
// resident blocks once, since each takes an equal part of the rows that are there (the device divides them,
// across sequences). Where that leaves much of the GPU without a block (units just over half of its
// slots), enough for four rounds of blocks, whose last is nearly full; no more than there are tiles of rows at
// full capacity.
int64_t fill_gpu(const attn::PagedShape &sh, int64_t units, int64_t rows, int64_t seqs, int sm_count)
{
    const int64_t tile = sh.nsl * 16, tiles = (rows + tile - 1) / tile * seqs;
    const int64_t blocks = (int64_t)sm_count * sh.blocks;
    int64_t P = blocks / units;
    if (P * units * 20 < blocks * 17) P = 4 * blocks / units;
    if (P > tiles) P = tiles;
    // two tiles a block, not one or a wave with idle blocks: while a third block an SM has as little to do, its start
    // costs more than it takes over (128 tiles, 4 units: P 114 8.95 us, 64 8.25; 64 tiles, 7 units: 64 8.9, 32 8.0)
    if (P * units > 2 * (int64_t)sm_count && tiles <= 2 * P) P = (tiles + 1) / 2;
    // a few tiles: one block a unit takes them in about the time that the second launch adds (a tile of 64
    // rows 0.9 us, the launch 2.5), with less work for the host
    if (tiles * tile <= 256) P = 1;
    return P < 1 ? 1 : P > kMaxPagedSplits ? kMaxPagedSplits : P;
}

void make_plan(const attn_paged_cache *c, int max_pages, int n_seq, int n_q, int n_head, int window, int n_splits,
               int sm_count, PagedPlan &pl)
{
    const int group = n_head / c->n_kv_head, es = type_bytes(c->kv_type), need = n_q * group;
    const int64_t seqs = n_seq < attn::kPagedSeqs ? n_seq : attn::kPagedSeqs;
    int64_t rows = (int64_t)max_pages * c->page_size;
    if (window > 0 && (int64_t)window + n_q + 64 < rows) rows = (int64_t)window + n_q + 64;
    auto shape = [&](int slots) { return attn::paged_shape(c->head_dim, es, slots); };
    auto units = [&](int slots) { return (int64_t)c->n_kv_head * ((need + slots - 1) / slots); };
    // 8 slots a block where a KV head has no more. Else 16 read and convert each row half as often, and 8 have
    // more blocks at work at a time and a merge half as long. With 8 bits, 8 slots
    // - while a block has few rows at full capacity (4 sequences of 8000 rows, 16 slots a KV head: head_dim 64 13.5 us
    //   with 16, 10.7 with 8; 128 15.7 and 13.4; 256 22.9 and 19.9; of 32000 rows 19.6 and 21.6, 26.2 and 28.0,
    //   44.2 and 43.5; 16-bit rows of 256 dimensions 28.4 and 33.5);
    // - where the last 16 would be half empty and 16 cost almost twice as much as 8: head_dim 256 (24, 40, 56 slots, 65000
    //   rows: 127.8 us with 16, 107.5 with 8; 183.9 and 163.7; 237.8 and 229.5), 128 up to 24 slots (64.3 and 61.0; 40
    //   slots 91.2 and 92.4), not 64 (43.1 and 47.5);
    // - at head_dim 256 for short sequences, whose merges count most, up to the capacity where 8 slots cost nothing
    //   even in a large call (1216, 1664, 2080, 2592, 4000 rows: 60 sequences, 8 KV heads, 32 slots 124.3 and 123.0, 149.6
    //   and 151.7, 173.1 and 177.7, 200.8 and 209.2, 280.9 and 297.0; 16 slots 69.0 and 64.7, 79.9 and 76.9, 92.2 and 90.2,
    //   104.5 and 105.7, 142.4 and 147.7). In small calls 8 slots gain past it too (28 sequences, 2 KV heads, 32 slots 24.6
    //   and 21.5, 29.4 and 25.3, 30.9 and 28.9, 36.0 and 32.3, 44.3 and 41.7): where blocks have few rows, the first
    //   rule takes them.
    const int64_t few = c->head_dim == 256 ? 1664 : 384;
    const bool half_empty = (need - 1) / 8 % 2 == 0;
    pl.slots = need <= 8 ? 8 : 16;
    if (need > 8 && es == 1 &&
        (rows * seqs <= few * fill_gpu(shape(8), units(8), rows, seqs, sm_count) ||
         (c->head_dim == 256 && (rows <= few || half_empty)) || (c->head_dim == 128 && need <= 24 && half_empty)))
        pl.slots = 8;
    pl.qgroups = (need + pl.slots - 1) / pl.slots;
    pl.shape = shape(pl.slots);
    pl.n_splits = n_splits > 0 ? n_splits : (int)fill_gpu(pl.shape, units(pl.slots), rows, seqs, sm_count);
    if (pl.n_splits > 1) {
        const size_t parts = (size_t)pl.n_splits * 2 * units(pl.slots) * pl.slots;
        pl.o_bytes = align256(parts * c->head_dim * sizeof(float));
        pl.ml_bytes = align256(parts * 2 * sizeof(float));
        pl.workspace = pl.o_bytes + pl.ml_bytes + align256((size_t)seqs * 8);
    }
}

} // namespace

extern "C" {

attn_status attn_rope_steps(int rot_dim, double base, int scaling, double factor, double low_turns,
                            double high_turns, int64_t trained_len, uint64_t *steps)
{
    if (!steps || rot_dim < 16 || rot_dim > 256 || rot_dim % 16 != 0) return ATTN_ERR_INVALID_ARG;
    if (!std::isfinite(base) || base < 1.0) return ATTN_ERR_INVALID_ARG;
    if (scaling < ATTN_ROPE_PLAIN || scaling > ATTN_ROPE_BANDS) return ATTN_ERR_INVALID_ARG;
    if (scaling != ATTN_ROPE_PLAIN && (!std::isfinite(factor) || factor <= 0.0)) return ATTN_ERR_INVALID_ARG;
    if (scaling == ATTN_ROPE_BANDS && (!std::isfinite(low_turns) || !std::isfinite(high_turns) ||
                                       !(low_turns < high_turns) || trained_len < 1))
        return ATTN_ERR_INVALID_ARG;
    const double two_pi = 6.283185307179586476925;
    if (scaling == ATTN_ROPE_BASE) base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
    if (!std::isfinite(base)) return ATTN_ERR_INVALID_ARG;     // every pair but the first would stand still
    uint64_t out[128];
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == ATTN_ROPE_LINEAR) f /= factor;
        if (scaling == ATTN_ROPE_BANDS) {
            const double n = (double)trained_len * f / two_pi;
            const double keep = n >= high_turns ? 1.0 : n <= low_turns ? 0.0 : (n - low_turns) / (high_turns - low_turns);
            f = keep * f + (1.0 - keep) * f / factor;
        }
        const double turns = f / two_pi;
        if (!(turns < 1.0)) return ATTN_ERR_INVALID_ARG;       // infinite and NaN too
        const double x = std::floor(turns * 18446744073709551616.0 + 0.5);
        out[i] = x >= 18446744073709551616.0 ? ~(uint64_t)0 : (uint64_t)x;
    }
    for (int i = 0; i < rot_dim / 2; ++i) steps[i] = out[i];
    return ATTN_OK;
}

attn_status attn_rope_append(const attn_paged_cache *cache, const int32_t *block_table, int max_pages,
                             const int32_t *positions, const int32_t *cu_tokens, int n_seq, int64_t n_tokens,
                             const void *q, const void *k_new, const void *v_new, int64_t q_stride,
                             int64_t k_stride, int64_t v_stride, int in_type, float *q_out, int n_head,
                             const attn_rope *rope, attn_stream_t stream)
{
    return attn_rope_append_tree(cache, block_table, max_pages, positions, cu_tokens, n_seq, n_tokens, q, k_new, v_new,
                                 q_stride, k_stride, v_stride, in_type, q_out, ATTN_TYPE_F32, n_head, rope, nullptr,
                                 stream);
}

attn_status attn_rope_append_tree(const attn_paged_cache *cache, const int32_t *block_table, int max_pages,
                                  const int32_t *positions, const int32_t *cu_tokens, int n_seq, int64_t n_tokens,
                                  const void *q, const void *k_new, const void *v_new, int64_t q_stride,
                                  int64_t k_stride, int64_t v_stride, int in_type, void *q_out, int out_type,
                                  int n_head, const attn_rope *rope, const int32_t *depths, attn_stream_t stream)
{
    attn_status st = check_cache_pointers(cache);
    if (st != ATTN_OK) return st;
    if (in_type != ATTN_TYPE_F32 && in_type != ATTN_TYPE_F16 && in_type != ATTN_TYPE_BF16) return ATTN_ERR_INVALID_ARG;
    if (out_type != ATTN_TYPE_F32 && out_type != in_type) return ATTN_ERR_INVALID_ARG;
    if (n_seq < 0 || n_seq > 65535 || n_tokens < 0 || n_tokens > kMaxRows) return ATTN_ERR_INVALID_ARG;
    if (n_seq == 0 && n_tokens != 0) return ATTN_ERR_INVALID_ARG;
    if (!cu_tokens && n_seq > 0 && n_tokens % n_seq != 0) return ATTN_ERR_INVALID_ARG;
    if (n_tokens > 0 && (!block_table || !positions || !k_new || !v_new)) return ATTN_ERR_INVALID_ARG;
    if ((q != nullptr) != (q_out != nullptr) || (q && (n_head < 1 || n_head > 65535))) return ATTN_ERR_INVALID_ARG;
    for (const void *p : {q, k_new, v_new, static_cast<const void *>(q_out)})
        if (!aligned(p, 16)) return ATTN_ERR_INVALID_ARG;
    for (const int32_t *p : {block_table, positions, cu_tokens, depths})
        if (!aligned(p, 4)) return ATTN_ERR_INVALID_ARG;
    if (rope && (!rope->steps || !aligned(rope->steps, 16) || rope->rot_dim < 16 || rope->rot_dim % 16 != 0 ||
                 rope->rot_dim > cache->head_dim || (rope->interleaved != 0 && rope->interleaved != 1) ||
                 !std::isfinite(rope->mscale) || rope->reserved != 0))
        return ATTN_ERR_INVALID_ARG;
    Strides cs;
    st = check_cache_shape(cache, max_pages, cs);
    if (st != ATTN_OK) return st;
    const int64_t hd = cache->head_dim, es = type_bytes(in_type);
    const int64_t q_dense = (int64_t)n_head * hd, kv_dense = (int64_t)cache->n_kv_head * hd;
    if (q_stride == 0 || !q) q_stride = q_dense;
    if (k_stride == 0) k_stride = kv_dense;
    if (v_stride == 0) v_stride = kv_dense;
    if ((q && q_stride < q_dense) || k_stride < kv_dense || v_stride < kv_dense) return ATTN_ERR_INVALID_ARG;
    for (int64_t x : {q ? q_stride : kv_dense, k_stride, v_stride})
        if (x >= kMaxStrideBytes / es || x * es % 16 != 0) return ATTN_ERR_INVALID_ARG;
    if (q && static_cast<const void *>(q_out) == q && (in_type != out_type || q_stride != q_dense))
        return ATTN_ERR_INVALID_ARG;
    if (n_tokens == 0) return ATTN_OK;

    attn::AppendRequest r{};
    attn::AppendArgs &a = r.a;
    a.q = q;
    a.k_new = k_new;
    a.v_new = v_new;
    a.q_out = q_out;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.k = cache->k;
    a.v = cache->v;
    a.k_scale = cache->k_scale;
    a.v_scale = cache->v_scale;
    a.page_stride = cs.page;
    a.row_stride = cs.row;
    a.head_stride = cs.head;
    a.table = block_table;
    a.positions = positions;
    a.cu = cu_tokens;
    a.depths = depths;
    a.q_in_type = out_type != ATTN_TYPE_F32;
    a.steps = rope ? rope->steps : nullptr;
    a.mscale = rope ? rope->mscale : 1.f;
    a.rot_dim = rope ? rope->rot_dim : 0;
    a.interleaved = rope ? rope->interleaved : 0;
    a.n_seq = n_seq;
    a.n_head = n_head;
    a.n_kv_head = cache->n_kv_head;
    a.n_tokens = n_tokens;
    a.n_each = cu_tokens ? 0 : n_tokens / n_seq;
    a.max_pages = max_pages;
    a.n_pages = cache->n_pages;
    a.page_size = cache->page_size;
    // (sequence, page) pairs that may be touched: the page jobs' numbering on the device
    a.page_items = cu_tokens ? n_tokens / cache->page_size + 2 * (int64_t)n_seq
                             : (int64_t)n_seq * ((a.n_each + cache->page_size - 2) / cache->page_size + 1);
    a.wide = aligned(q, 32) && aligned(k_new, 32) && aligned(v_new, 32) && aligned(q_out, 32) &&
             (q ? q_stride : 0) * es % 32 == 0 && k_stride * es % 32 == 0 && v_stride * es % 32 == 0 &&
             aligned(cache->k, 32) && aligned(cache->v, 32);
    for (int64_t x : {cs.page, cs.row, cs.head}) a.wide = a.wide && x * type_bytes(cache->kv_type) % 32 == 0;
    r.head_dim = cache->head_dim;
    r.in_type = in_type;
    r.kv_type = cache->kv_type;
    r.stream = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = attn::launch_append(r);
    return e == cudaSuccess ? ATTN_OK : fail(e);
}

attn_status attn_paged_plan(const attn_paged_cache *cache, int max_pages, int n_seq, int n_q, int n_head,
                            int window, int n_splits, int sm_count, int *n_splits_out,
                            size_t *workspace_bytes_out)
{
    Strides cs;
    attn_status st = check_cache_shape(cache, max_pages, cs);
    if (!cache) return st;
    const attn_status sh = st == ATTN_OK || st == ATTN_ERR_UNSUPPORTED
                               ? check_heads(cache, n_seq, n_q, n_head, window, n_splits) : st;
    if (sh != ATTN_OK) return sh;
    if (st != ATTN_OK) return st;
    if (n_seq == 0) return ATTN_ERR_INVALID_ARG;          // nothing to plan
    if (sm_count <= 0) {
        unsigned *err = nullptr;
        const cudaError_t e = attn::device_facts(&sm_count, &err);
        if (e != cudaSuccess) return fail(e);
    }
    PagedPlan pl;
    make_plan(cache, max_pages, n_seq, n_q, n_head, window, n_splits, sm_count, pl);
    if (n_splits_out) *n_splits_out = pl.n_splits;
    if (workspace_bytes_out) *workspace_bytes_out = pl.workspace;
    return ATTN_OK;
}

attn_status attn_decode_paged(const attn_paged_cache *cache, const int32_t *block_table, int max_pages,
                              const int32_t *positions, const float *q, float *out, int n_seq, int n_q,
                              int n_head, float scale, const attn_score_rules *rules, int n_splits,
                              void *workspace, size_t workspace_bytes, attn_stream_t stream)
{
    attn_status st = check_cache_pointers(cache);
    if (st != ATTN_OK) return st;
    if (!std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
    if (n_seq > 0 && (!block_table || !positions || !q || !out)) return ATTN_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(block_table, 4) || !aligned(positions, 4))
        return ATTN_ERR_INVALID_ARG;
    const float softcap = rules ? rules->softcap : 0.f;
    const int window = rules ? rules->window : 0;
    if (!(softcap == 0.f || (softcap >= 0x1p-40f && softcap <= 0x1p40f))) return ATTN_ERR_INVALID_ARG;
    const float qscale = softcap > 0.f ? (float)((double)scale / softcap) : (float)((double)scale * 1.4426950408889634);
    if (!std::isfinite(qscale)) return ATTN_ERR_INVALID_ARG;
    if (rules && (!aligned(rules->slopes, 4) || !aligned(rules->starts, 4))) return ATTN_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return ATTN_ERR_INVALID_ARG;
    Strides cs;
    st = check_cache_shape(cache, max_pages, cs);
    if (st == ATTN_ERR_INVALID_ARG) return st;
    const attn_status sh = check_heads(cache, n_seq, n_q, n_head, window, n_splits);
    if (sh != ATTN_OK) return sh;
    if (st != ATTN_OK) return st;
    if (n_seq == 0) return ATTN_OK;

    int sm_count = 0;
    unsigned *err = nullptr;
    cudaError_t e = attn::device_facts(&sm_count, &err);
    if (e != cudaSuccess) return fail(e);
    PagedPlan pl;
    make_plan(cache, max_pages, n_seq, n_q, n_head, window, n_splits, sm_count, pl);
    if ((int64_t)cache->n_kv_head * pl.qgroups > 0x7fffffff) return ATTN_ERR_INVALID_ARG;
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

    const int64_t units = (int64_t)cache->n_kv_head * pl.qgroups;
    attn::PagedRequest r{};
    attn::PagedArgs &a = r.pa;
    a.k_scale = cache->k_scale;
    a.v_scale = cache->v_scale;
    a.slopes = rules ? rules->slopes : nullptr;
    if (pl.workspace > 0) {
        uint8_t *ws = static_cast<uint8_t *>(workspace);
        a.ws_o = reinterpret_cast<float *>(ws);
        a.ws_ml = reinterpret_cast<float2 *>(ws + pl.o_bytes);
        a.ws_span = reinterpret_cast<int2 *>(ws + pl.o_bytes + pl.ml_bytes);
    }
    a.err = err;
    a.n_head = n_head;
    a.n_kv_head = cache->n_kv_head;
    a.group = n_head / cache->n_kv_head;
    a.n_q = n_q;
    a.qgroups = pl.qgroups;
    a.units = (int)units;
    a.ranks = pl.n_splits;
    // the merge grows with the slots and the dimensions faster than the time of a tile (places between two
    // sequences 0, 2, 3, 4: head_dim 128, 8 slots 57.8, 56.9, 57.7, 59.0 us; 256, 8 slots 38.7, 38.5, 37.5, 37.6;
    // 128, 16 slots 34.5, 32.2, 30.9, 29.8; 256, 16 slots, 16 bits 28.7, 26.8, 26.4, 25.8)
    a.turn = 2 + (pl.slots == 16 ? 2 : 0) + (cache->head_dim == 256 ? 1 : 0);
    a.max_pages = max_pages;
    a.n_pages = cache->n_pages;
    a.page_size = cache->page_size;
    a.cap = max_pages * cache->page_size;
    a.window = window > a.cap ? 0 : window;        // past the capacity it masks nothing
    const int tile = pl.shape.nsl * 16;
    a.box_rows = cache->page_size % 64 == 0 && tile >= 64 ? 64 : cache->page_size % 32 == 0 && tile >= 32 ? 32 : 16;
    a.by_page = attn::fast_div((unsigned)cache->page_size);
    a.by_group = attn::fast_div((unsigned)a.group);
    a.by_ranks = attn::fast_div((unsigned)a.ranks);
    a.qscale = qscale;
    a.cap_log2 = (float)((double)softcap * 1.4426950408889634);
    r.k = cache->k;
    r.v = cache->v;
    r.page_stride = cs.page;
    r.row_stride = cs.row;
    r.head_stride = cs.head;
    r.head_dim = cache->head_dim;
    r.kv_type = cache->kv_type;
    r.rules = softcap > 0.f || a.slopes;
    r.slots = pl.slots;
    r.stream = reinterpret_cast<cudaStream_t>(stream);
    const int ti = cache->kv_type - ATTN_TYPE_F16;
    using Launch = cudaError_t (*)(const attn::PagedRequest &);
    static const Launch table[3][3] = {
        {attn::launch_paged_hd64_f16, attn::launch_paged_hd64_bf16, attn::launch_paged_hd64_e4m3},
        {attn::launch_paged_hd128_f16, attn::launch_paged_hd128_bf16, attn::launch_paged_hd128_e4m3},
        {attn::launch_paged_hd256_f16, attn::launch_paged_hd256_bf16, attn::launch_paged_hd256_e4m3}};
    const int hi = cache->head_dim == 64 ? 0 : cache->head_dim == 128 ? 1 : 2;
    // tiles and places are counted in 32 bits, some groups past the last: fewer sequences a launch where the capacity is huge
    const int64_t per_seq = (a.cap + (int64_t)tile - 1) / tile + 1 + a.turn;
    const int batch = (int)(0x7fff0000 / per_seq < attn::kPagedSeqs ? 0x7fff0000 / per_seq : attn::kPagedSeqs);
    for (int s0 = 0; s0 < n_seq; s0 += batch) {
        const size_t rows = (size_t)s0 * n_q * n_head * cache->head_dim;
        a.n_seq = n_seq - s0 < batch ? n_seq - s0 : batch;
        a.q = q + rows;
        a.out = out + rows;
        a.positions = positions + s0;
        a.table = block_table + (size_t)s0 * max_pages;
        a.starts = rules && rules->starts ? rules->starts + s0 : nullptr;
        e = table[hi][ti](r);
        if (e != cudaSuccess) return fail(e);
    }
    return ATTN_OK;
}

} // extern "C"
