// attn_paged_impl.cuh -- instantiation and launch of the paged partial kernel
// per (head_dim, cache type). Each attn_paged_hd<N>_<type>.cu includes this once,
// so the instantiations compile in parallel.
#pragma once

#include "attn_launch.h"
#include "attn_paged.cuh"

namespace attn {

template <class C, bool RULES>
cudaError_t launch_paged_kernel(const PagedRequest &r)
{
    alignas(64) CUtensorMap kmap, vmap;
    const bool bf = std::is_same<typename C::KV, __nv_bfloat16>::value;
    const int64_t es = C::ES;
    cudaError_t e = encode_paged_map(&kmap, r.k, C::ES, bf, C::HD, r.pa.n_kv_head, r.pa.page_size, r.pa.n_pages,
                                     r.head_stride * es, r.row_stride * es, r.page_stride * es, C::CW, r.pa.box_rows);
    if (e != cudaSuccess) return e;
    e = encode_paged_map(&vmap, r.v, C::ES, bf, C::HD, r.pa.n_kv_head, r.pa.page_size, r.pa.n_pages,
                         r.head_stride * es, r.row_stride * es, r.page_stride * es, C::CW, r.pa.box_rows);
    if (e != cudaSuccess) return e;
    const void *fn = reinterpret_cast<const void *>(&attn_paged_stream<C, RULES>);
    e = ensure_smem_attr(fn, (int)C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    PagedArgs pa = r.pa;
    void *args[] = {&kmap, &vmap, &pa};
    e = launch_pdl(fn, dim3((unsigned)pa.qgroups, (unsigned)pa.n_kv_head, (unsigned)pa.ranks), dim3(C::THREADS), C::SMEM_BYTES, r.stream, args);
    if (e != cudaSuccess || pa.ranks == 1) return e;
    // The widest piece of a row a block that leaves enough of them: a piece brings its row's sums and span along, and
    // few blocks hide no latency (pieces of 32, 64, all dimensions: 64 rows of 128 47.5, 46.9, 47.5 us the
    // whole call; 256 rows of 256 21.3, 19.8, 19.9; 360 rows of 256 17.2, 15.8, 15.4; 28 rows of 128 9.0, 9.0, 9.8;
    // 16 rows of 256 14.1, 14.7, 19.0).
    const int64_t rows = (int64_t)pa.n_q * pa.n_head, pieces64 = rows * pa.n_seq * C::HD / 64;
    const int piece = rows * pa.n_seq > 256 ? C::HD : pieces64 >= 128 ? 64 : 32;
    int slots = C::SLOTS;
    const void *cf = piece == C::HD ? reinterpret_cast<const void *>(&attn_paged_combine<C::HD, C::HD>)
                     : piece == 64 ? reinterpret_cast<const void *>(&attn_paged_combine<C::HD, 64>)
                                   : reinterpret_cast<const void *>(&attn_paged_combine<C::HD, 32>);
    e = ensure_smem_attr(cf, 0);
    if (e != cudaSuccess) return e;
    void *cargs[] = {&pa, &slots};
    return launch_pdl(cf, dim3((unsigned)rows, (unsigned)pa.n_seq, (unsigned)(C::HD / piece)), dim3(128), 0, r.stream, cargs);
}

template <int HD, typename KV>
cudaError_t launch_paged_for(const PagedRequest &r)
{
    if (r.slots == 8) {
        using C = PagedCfg<HD, 8, KV>;
        return r.rules ? launch_paged_kernel<C, true>(r) : launch_paged_kernel<C, false>(r);
    }
    using C = PagedCfg<HD, 16, KV>;
    return r.rules ? launch_paged_kernel<C, true>(r) : launch_paged_kernel<C, false>(r);
}

} // namespace attn
