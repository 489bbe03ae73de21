// attn_tree.cu -- attention of drafted trees over a paged cache, a warp for each (node, head).
//
// Mathematics. For a node t at position x over the cache rows j it sees -- all before its tree, and the
// tree's own as its mask has them --
//     s_j = rules(scale q.k_j),  o = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j log2 e - m),
// one pass with the running maximum m, in 32 bits.
#include <cuda_fp8.h>

#include "attn_device.cuh"
#include "attn_launch.h"
#include "attn_paged_launch.h"

namespace attn {

namespace {

struct TreePool {
    const uint8_t *k, *v;
    int64_t page, row, head;     // bytes
};

template <int KT>
__device__ __forceinline__ float element(const uint8_t *p, int d)
{
    if constexpr (KT == kTypeE4m3) {
        return (float)reinterpret_cast<const __nv_fp8_e4m3 *>(p)[d];
    } else if constexpr (KT == kTypeF16) {
        return __half2float(reinterpret_cast<const __half *>(p)[d]);
    } else {
        return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[d]);
    }
}

__device__ __forceinline__ float q_at(const TreeArgs &a, int64_t i)
{
    if (a.q_type == kTypeF32) return static_cast<const float *>(a.q)[i];
    if (a.q_type == kTypeF16) return __half2float(static_cast<const __half *>(a.q)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(a.q)[i]);
}

template <int HD, int KT>
__global__ void __launch_bounds__(128) tree_simple(const TreeArgs a, const TreePool pool)
{
    constexpr int E = HD / 32;
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t job = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t tok = job / a.n_head;
    const int h = (int)(job - tok * a.n_head), hk = h / a.group;
    if (tok >= a.n_tokens) return;
    int s = 0;
    int64_t t0 = 0, t1 = 0;
    for (; s < a.n_seq; ++s) {
        t0 = a.cu ? ld_dep(a.cu + s) : (int64_t)s * a.n_each;
        t1 = a.cu ? ld_dep(a.cu + s + 1) : t0 + a.n_each;
        if (tok < t1) break;
    }
    if (s == a.n_seq) return;
    const int n = (int)(t1 - t0), t = (int)(tok - t0);
    if (n > a.max_nodes) {
        if (t == 0 && h == 0 && lane == 0) atomicOr(a.err, 0x8u);
        return;
    }
    const int pos = ld_dep(a.positions + s);
    if ((pos < -1 || pos >= a.cap) && t == 0 && h == 0 && lane == 0) atomicOr(a.err, kErrPositionClamped);
    const int nkv = min(max(pos, -1), a.cap - 1) + 1, base = nkv - n;
    const int start = a.starts ? ld_dep(a.starts + s) : 0;
    const int x = base + (a.depths ? ld_dep(a.depths + tok) : t);
    const float slope = a.slopes ? ld_dep(a.slopes + h) * kLog2e : 0.f;
    float q[E], o[E], m = -INFINITY, l = 0.f;
    for (int e = 0; e < E; ++e) {
        q[e] = q_at(a, (tok * a.n_head + h) * HD + e * 32 + lane);
        o[e] = 0.f;
    }
    for (int j = max(start, 0); j < nkv; ++j) {
        int at = j;
        if (j >= base) {
            const int y = j - base;
            const bool sees = a.mask ? a.mask[tok * a.words + (y >> 5)] >> (y & 31) & 1 : y <= t;
            if (!sees) continue;
            at = base + (a.depths ? ld_dep(a.depths + t0 + y) : y);
        }
        if (a.window > 0 && x - at >= a.window) continue;
        const int pg = div(a.by_page, j), page = ld_dep(a.table + (size_t)s * a.max_pages + pg);
        if ((unsigned)page >= (unsigned)a.n_pages) {
            if (lane == 0) atomicOr(a.err, 0x4u);
            continue;
        }
        const int64_t off = page * pool.page + (j - pg * a.page_size) * pool.row + hk * pool.head;
        float d = 0.f;
        for (int e = 0; e < E; ++e) d = fmaf(q[e], element<KT>(pool.k + off, e * 32 + lane), d);
        d = warp_sum(d);
        float vs = 1.f;
        if (KT == kTypeE4m3) {
            d *= ld_dep(a.k_scale + (size_t)page * a.n_kv_head + hk);
            vs = ld_dep(a.v_scale + (size_t)page * a.n_kv_head + hk);
        }
        float sc = d * a.scale_log2;
        if (a.softcap > 0.f) sc = a.softcap * kLog2e * tanhf(sc / (a.softcap * kLog2e));
        sc = fmaf(-slope, (float)(x - at), sc);
        const float mn = fmaxf(m, sc), c = m == -INFINITY ? 0.f : ex2(m - mn);
        const float p = ex2(sc - (mn == -INFINITY ? 0.f : mn));
        l = fmaf(l, c, p);
        for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], c, p * vs * element<KT>(pool.v + off, e * 32 + lane));
        m = mn;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int e = 0; e < E; ++e) {
        const int64_t i = (tok * a.n_head + h) * HD + e * 32 + lane;
        const float y = o[e] * inv;
        if (a.q_type == kTypeF32) static_cast<float *>(a.out)[i] = y;
        else if (a.q_type == kTypeF16) static_cast<__half *>(a.out)[i] = __float2half_rn(y);
        else static_cast<__nv_bfloat16 *>(a.out)[i] = __float2bfloat16_rn(y);
    }
}

template <int HD, int KT>
cudaError_t launch_it(const TreeRequest &r)
{
    TreeArgs a = r.a;
    const int64_t es = KT == kTypeE4m3 ? 1 : 2;
    TreePool pool{static_cast<const uint8_t *>(r.k), static_cast<const uint8_t *>(r.v), r.page_stride * es,
                  r.row_stride * es, r.head_stride * es};
    const int64_t blocks = (a.n_tokens * a.n_head + 3) / 4;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    void *args[] = {&a, &pool};
    return launch_pdl(reinterpret_cast<const void *>(&tree_simple<HD, KT>), dim3((unsigned)blocks), dim3(128), 0, r.stream, args);
}

template <int HD>
cudaError_t launch_hd(const TreeRequest &r)
{
    return r.kv_type == kTypeF16 ? launch_it<HD, kTypeF16>(r) : r.kv_type == kTypeBf16 ? launch_it<HD, kTypeBf16>(r)
                                                                                      : launch_it<HD, kTypeE4m3>(r);
}

} // namespace

cudaError_t launch_tree(const TreeRequest &r)
{
    return r.head_dim == 64 ? launch_hd<64>(r) : r.head_dim == 128 ? launch_hd<128>(r) : launch_hd<256>(r);
}

} // namespace attn
