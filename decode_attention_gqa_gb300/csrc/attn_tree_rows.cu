// attn_tree_rows.cu -- what surrounds the attention of trees: the nodes' masks and depths from
// their parents, and the rows of the accepted path moved to where the sequence goes on.
#include <cuda_fp8.h>

#include "attn_device.cuh"
#include "attn_launch.h"
#include "attn_paged_launch.h"

namespace attn {

namespace {

constexpr unsigned kErrBadPageT = 0x4u, kErrBadRequest = 0x8u;   // ATTN_DEVERR_BAD_PAGE, _BAD_REQUEST

// ---------------------------------------------------------------------------
// Rules of a tree. A block takes a sequence: the parents lie in shared memory, and each thread walks up from its
// node, setting a bit of the node's row and counting. The chain of a call is launch, token
// numbers, parents, depth steps of some 30 cycles, store.
// 48 sequences of 7 to 26 nodes: 3.9 us alone, of which 2.5 are the launch.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) tree_rules_kernel(const TreeRulesArgs g)
{
    extern __shared__ int32_t rules_smem[];
    pdl_wait();
    const int s = blockIdx.x, tid = threadIdx.x;
    int64_t t0 = (int64_t)s * g.n_each, t1 = t0 + g.n_each;
    if (g.cu) {
        t0 = min(max((int64_t)ld_dep(g.cu + s), (int64_t)0), g.n_tokens);
        t1 = min(max((int64_t)ld_dep(g.cu + s + 1), (int64_t)0), g.n_tokens);
    }
    if (t1 <= t0) return;
    const int n = (int)min(t1 - t0, (int64_t)g.max_nodes + 1);
    if (n > g.max_nodes) {
        if (tid == 0) atomicOr(g.err, kErrBadRequest);
        return;
    }
    int32_t *par = rules_smem;
    uint32_t *rows = reinterpret_cast<uint32_t *>(rules_smem + n);
    bool bad = false;
    for (int t = tid; t < n; t += blockDim.x) {
        int p = ld_dep(g.parents + t0 + t);
        if (p >= n) {
            bad = true;
            p = -1;
        }
        par[t] = p;
    }
    for (int i = tid; i < n * g.words; i += blockDim.x) rows[i] = 0u;
    __syncthreads();
    for (int t = tid; t < n; t += blockDim.x) {
        uint32_t *row = rows + t * g.words;
        int at = t, depth = 0;
        row[at >> 5] |= 1u << (at & 31);
        for (at = par[at]; at >= 0; at = par[at]) {
            const uint32_t bit = 1u << (at & 31), w = row[at >> 5];
            if (w & bit) {                            // met before: a circle
                bad = true;
                break;
            }
            row[at >> 5] = w | bit;
            ++depth;
        }
        g.depths[t0 + t] = depth;
    }
    __syncthreads();
    for (int i = tid; i < n * g.words; i += blockDim.x) g.mask[t0 * g.words + i] = rows[i];
    if (bad) atomicOr(g.err, kErrBadRequest);
}

// ---------------------------------------------------------------------------
// Kept rows. A block takes K or V of one KV head of a sequence. A row moves towards the front, past rows that
// later ones are still to be read from only after they were: path[i] >= i increasing, so the rows
// that a chunk reads are none that an earlier chunk has written, and a barrier stands between a chunk's
// reads and its writes. What bounds it is the chain: counts, path, table, rows (and scales, the largest magnitude), store.
// In a graph: 5 rows of 4 heads of 128, e4m3 4.0 us; 64 sequences, 1 to 12 rows of 8 heads of 256, bf16 5.2 us (6.8 MB).
// ---------------------------------------------------------------------------
constexpr int kKeepThreads = 256, kKeepUnits = 4;             // 16-byte units a thread holds at a time

// The smallest power of two s in [2^-60, 2^60] with amax <= 448 s.
__device__ __forceinline__ float keep_scale(float amax)
{
    const unsigned bits = __float_as_uint(amax);
    int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    e = min(max(e, -60), 60);
    return __uint_as_float((unsigned)(e + 127) << 23);
}

__device__ __forceinline__ void codes_to_float(uint32_t w, float (&f)[4])
{
    uint32_t a, b;
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}" : "=r"(a), "=r"(b) : "r"(w));
    const float2 p = kv2_to_float2<__half>(a), q = kv2_to_float2<__half>(b);
    f[0] = p.x; f[1] = p.y; f[2] = q.x; f[3] = q.y;
}

__device__ __forceinline__ uint32_t float_to_codes(float a, float b, float c, float d)
{
    uint16_t x, y;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(x) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(y) : "f"(d), "f"(c));
    return (uint32_t)x | (uint32_t)y << 16;
}

struct KeepRow {              // of the chunk at hand
    int64_t from, to;         // bytes from the pool's first; -1: nothing to move
    float scale;
};

template <bool E8>
__global__ void __launch_bounds__(kKeepThreads) keep_rows_kernel(const KeepArgs g)
{
    __shared__ KeepRow sm_row[kKeepThreads * kKeepUnits / 4];
    __shared__ float sm_max[kKeepThreads / 32];
    pdl_wait();
    const int s = blockIdx.y, tid = threadIdx.x;
    const bool is_v = (int)blockIdx.x >= g.n_kv_head;
    const int kh = is_v ? blockIdx.x - g.n_kv_head : blockIdx.x;
    const int n = ld_dep(g.counts + s), base = ld_dep(g.base + s);
    if (n == 0) return;
    const int64_t cap = (int64_t)g.max_pages * g.page_size;
    const int32_t *path = g.path + (size_t)s * g.max_keep;
    bool bad = n < 0 || n > g.max_keep || base < 0;
    if (!bad)
        for (int i = tid; i < n; i += kKeepThreads) {
            const int p = ld_dep(path + i), before = i ? ld_dep(path + i - 1) : -1;
            bad = bad || p <= before || (int64_t)base + p >= cap;
        }
    if (__syncthreads_or(bad)) {
        if (tid == 0 && blockIdx.x == 0) atomicOr(g.err, kErrBadRequest);
        return;
    }
    uint8_t *pool = (is_v ? g.v : g.k) + (int64_t)kh * g.head_stride;
    float *scales = is_v ? g.v_scale : g.k_scale;
    const int32_t *table = g.table + (size_t)s * g.max_pages;
    const int upr = g.row_bytes / 16;                         // a power of two
    const int per_chunk = kKeepThreads * kKeepUnits / upr;    // rows
    const int lu = tid & (upr - 1), lr = tid / upr, rstep = kKeepThreads / upr;

    // pages of the destination in turn (16 bits: all at once)
    for (int i0 = 0; i0 < n;) {
        const int page_no = div(g.by_page, base + i0), at = base + i0 - page_no * g.page_size;
        const int i1 = E8 ? min(n, i0 + g.page_size - at) : n;
        int page = 0;
        float old = 0.f, now = 1.f;
        if (E8) {
            page = ld_dep(table + page_no);
            if ((unsigned)page < (unsigned)g.n_pages && at > 0) old = ld_dep(scales + (size_t)page * g.n_kv_head + kh);
        }
        // E4M3: once for the largest magnitude, once to move
        for (int pass = E8 ? 0 : 1; pass < 2; ++pass) {
            float most = 0.f;
            for (int c0 = i0; c0 < i1; c0 += per_chunk) {
                const int c1 = min(i1, c0 + per_chunk);
                __syncthreads();                              // the chunk before has read its rows' places
                for (int i = c0 + tid; i < c1; i += kKeepThreads) {
                    const int f = base + ld_dep(path + i), t = base + i;
                    const int fp = div(g.by_page, f), tp = div(g.by_page, t);
                    const int fid = ld_dep(table + fp), tid2 = ld_dep(table + tp);
                    KeepRow r{-1, -1, 1.f};
                    if ((unsigned)fid < (unsigned)g.n_pages && (unsigned)tid2 < (unsigned)g.n_pages) {
                        r.from = (int64_t)fid * g.page_stride + (int64_t)(f - fp * g.page_size) * g.row_stride;
                        r.to = (int64_t)tid2 * g.page_stride + (int64_t)(t - tp * g.page_size) * g.row_stride;
                        if (E8) r.scale = ld_dep(scales + (size_t)fid * g.n_kv_head + kh);
                    } else if (blockIdx.x == 0) {
                        atomicOr(g.err, kErrBadPageT);
                    }
                    sm_row[i - c0] = r;
                }
                __syncthreads();
                uint4 u[kKeepUnits];
#pragma unroll
                for (int x = 0; x < kKeepUnits; ++x) {
                    const int i = lr + x * rstep;
                    if (c0 + i < c1 && sm_row[i].from >= 0)
                        u[x] = ld_dep(reinterpret_cast<const uint4 *>(pool + sm_row[i].from) + lu);
                }
                if (pass == 0) {
#pragma unroll
                    for (int x = 0; x < kKeepUnits; ++x) {
                        const int i = lr + x * rstep;
                        if (c0 + i >= c1 || sm_row[i].from < 0) continue;
                        const uint32_t w[4] = {u[x].x, u[x].y, u[x].z, u[x].w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float f[4];
                            codes_to_float(w[j], f);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float m = fabsf(f[e] * sm_row[i].scale);
                                if (m < INFINITY) most = fmaxf(most, m);
                            }
                        }
                    }
                    continue;
                }
                __syncthreads();                              // every row of the chunk is read
#pragma unroll
                for (int x = 0; x < kKeepUnits; ++x) {
                    const int i = lr + x * rstep;
                    if (c0 + i >= c1 || sm_row[i].from < 0) continue;
                    if (E8 && sm_row[i].scale != now) {
                        const float sc = sm_row[i].scale;
                        uint32_t *w = &u[x].x;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float f[4];
                            codes_to_float(w[j], f);
                            w[j] = float_to_codes(__fdiv_rn(f[0] * sc, now), __fdiv_rn(f[1] * sc, now),
                                                  __fdiv_rn(f[2] * sc, now), __fdiv_rn(f[3] * sc, now));
                        }
                    }
                    reinterpret_cast<uint4 *>(pool + sm_row[i].to)[lu] = u[x];
                }
            }
            if (E8 && pass == 0) {
                most = warp_max(most);
                if ((tid & 31) == 0) sm_max[tid >> 5] = most;
                __syncthreads();
                most = sm_max[0];
#pragma unroll
                for (int w = 1; w < kKeepThreads / 32; ++w) most = fmaxf(most, sm_max[w]);
                now = keep_scale(most);
                if (at > 0 && fabsf(old) < INFINITY) now = fmaxf(now, fabsf(old));
            }
        }
        if (E8) {
            if ((unsigned)page < (unsigned)g.n_pages) {
                // rows [0, at) at the new scale
                if (at > 0 && now != old && fabsf(old) < INFINITY) {
                    const float ratio = old / now;
                    for (int i = lr; i < at; i += rstep) {
                        uint4 *p = reinterpret_cast<uint4 *>(pool + (int64_t)page * g.page_stride + (int64_t)i * g.row_stride) + lu;
                        uint4 c = *p;
                        uint32_t *w = &c.x;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float f[4];
                            codes_to_float(w[j], f);
                            w[j] = float_to_codes(f[0] * ratio, f[1] * ratio, f[2] * ratio, f[3] * ratio);
                        }
                        *p = c;
                    }
                }
                __syncthreads();                              // every row's old scale is read
                if (tid == 0) scales[(size_t)page * g.n_kv_head + kh] = now;
            }
        }
        i0 = i1;
    }
}

} // namespace

cudaError_t launch_tree_rules(const TreeRulesArgs &a, cudaStream_t stream)
{
    TreeRulesArgs g = a;
    int sms = 0;
    cudaError_t e = device_facts(&sms, &g.err);
    if (e != cudaSuccess) return e;
    const size_t smem = (size_t)g.max_nodes * (g.words + 1) * 4;
    const void *fn = reinterpret_cast<const void *>(&tree_rules_kernel);
    e = ensure_smem_attr(fn, 1024 * 33 * 4);
    if (e != cudaSuccess) return e;
    const int threads = g.max_nodes <= 64 ? 64 : g.max_nodes <= 128 ? 128 : 256;
    void *args[] = {&g};
    return launch_pdl(fn, dim3((unsigned)g.n_seq), dim3((unsigned)threads), smem, stream, args);
}

cudaError_t launch_keep_rows(const KeepArgs &a, bool e4m3, cudaStream_t stream)
{
    KeepArgs g = a;
    int sms = 0;
    cudaError_t e = device_facts(&sms, &g.err);
    if (e != cudaSuccess) return e;
    g.by_page = fast_div((unsigned)g.page_size);
    const void *fn = e4m3 ? reinterpret_cast<const void *>(&keep_rows_kernel<true>)
                          : reinterpret_cast<const void *>(&keep_rows_kernel<false>);
    void *args[] = {&g};
    return launch_pdl(fn, dim3(2u * (unsigned)g.n_kv_head, (unsigned)g.n_seq), dim3(kKeepThreads), 0, stream, args);
}

} // namespace attn
