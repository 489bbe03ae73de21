// attn_paged_impl.cuh -- instantiation and launch of the paged partial kernel
// per (head_dim, cache type). Each attn_paged_hd<N>_<type>.cu includes this once,
// so the instantiations compile in parallel.
#pragma once

#include "attn_launch.h"
#include "attn_paged.cuh"

namespace attn {

// Stages and resident blocks per SM: about 190 KB of stages on an SM whatever
// the row size, so that enough copies are in flight for HBM, in as many blocks as
// the accumulators (head_dim / 2 registers a thread) leave room for.
template <int HD, int ES> struct PagedShape;
template <> struct PagedShape<64, 1>  { static constexpr int S = 8, MINB = 2; };
template <> struct PagedShape<128, 1> { static constexpr int S = 6, MINB = 2; };
template <> struct PagedShape<256, 1> { static constexpr int S = 6, MINB = 1; };
template <> struct PagedShape<64, 2>  { static constexpr int S = 6, MINB = 2; };
template <> struct PagedShape<128, 2> { static constexpr int S = 3, MINB = 2; };
template <> struct PagedShape<256, 2> { static constexpr int S = 3, MINB = 1; };

template <int HD, typename KV, int SLOTS>
using PagedCfgFor = PagedCfg<HD, SLOTS, KV, PagedShape<HD, std::is_same<KV, E4m3>::value ? 1 : 2>::S,
                             PagedShape<HD, std::is_same<KV, E4m3>::value ? 1 : 2>::MINB>;

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
    const void *fn = reinterpret_cast<const void *>(&attn_paged_partial<C, RULES>);
    e = ensure_smem_attr(fn, (int)C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    PagedArgs pa = r.pa;
    void *args[] = {&kmap, &vmap, &pa};
    return launch_pdl(fn, dim3(pa.n_kv_head * pa.qgroups, pa.n_splits, r.n_seq), dim3(C::THREADS), C::SMEM_BYTES,
                      r.stream, args);
}

template <int HD, typename KV>
cudaError_t launch_paged_for(const PagedRequest &r)
{
    if (paged_slots(r.pa.n_q, r.pa.group) == 8) {
        using C = PagedCfgFor<HD, KV, 8>;
        return r.rules ? launch_paged_kernel<C, true>(r) : launch_paged_kernel<C, false>(r);
    }
    using C = PagedCfgFor<HD, KV, 16>;
    return r.rules ? launch_paged_kernel<C, true>(r) : launch_paged_kernel<C, false>(r);
}

} // namespace attn
