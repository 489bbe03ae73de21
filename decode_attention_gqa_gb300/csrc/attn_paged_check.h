// attn_paged_check.h -- host checks that the C-ABI units of the paged-cache operators share
// (attn_paged_api.cu, attn_tree_api.cu, attn_pages.cu). Not installed; not part of the public ABI.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "attn_paged.h"
#include "attn_paged_launch.h"

namespace attn {
namespace check {

constexpr int64_t kMaxRows = (int64_t)0x7fffffff - 16384;
constexpr int64_t kMaxStrideBytes = (int64_t)1 << 40;

inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline attn_status fail(cudaError_t e)
{
    attn::note_cuda_error(e);
    return ATTN_ERR_CUDA;
}

inline int type_bytes(int t) { return t == ATTN_TYPE_F32 ? 4 : t == ATTN_TYPE_E4M3 ? 1 : 2; }

struct Strides {
    int64_t page, row, head;
};

// Everything about the pool but its pointers.
inline attn_status check_cache_shape(const attn_paged_cache *c, int max_pages, Strides &st)
{
    if (!c || c->reserved != 0 || c->n_pages < 1 || c->n_kv_head < 1 || c->head_dim < 1 || max_pages < 1)
        return ATTN_ERR_INVALID_ARG;
    if (c->page_size < 16 || c->page_size > 1024 || c->page_size % 16 != 0) return ATTN_ERR_INVALID_ARG;
    if (c->kv_type != ATTN_TYPE_F16 && c->kv_type != ATTN_TYPE_BF16 && c->kv_type != ATTN_TYPE_E4M3)
        return ATTN_ERR_INVALID_ARG;
    if (c->n_kv_head > 65535 || (int64_t)max_pages * c->page_size > kMaxRows) return ATTN_ERR_INVALID_ARG;
    st = Strides{c->page_stride, c->row_stride, c->head_stride};
    if (st.page == 0 && st.row == 0 && st.head == 0) {
        st.head = c->head_dim;
        st.row = (int64_t)c->n_kv_head * c->head_dim;
        st.page = (int64_t)c->page_size * st.row;
    }
    const int64_t es = type_bytes(c->kv_type);
    for (int64_t x : {st.page, st.row, st.head})
        if (x < c->head_dim || x >= kMaxStrideBytes / es || x * es % 16 != 0) return ATTN_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return ATTN_ERR_UNSUPPORTED;
    return ATTN_OK;
}

inline attn_status check_cache_pointers(const attn_paged_cache *c)
{
    if (!c || !c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16)) return ATTN_ERR_INVALID_ARG;
    const bool scales = c->kv_type == ATTN_TYPE_E4M3;
    if (scales != (c->k_scale != nullptr) || scales != (c->v_scale != nullptr)) return ATTN_ERR_INVALID_ARG;
    if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)) return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

} // namespace check
} // namespace attn
