// attn_rope_append.cu -- the append kernel: rotate the new tokens' q and k by
// position and write k and v rows into the paged cache.
//
// Mathematics. Pair i of a head turns by position * steps[i] / 2^64 of a turn;
// the 64-bit product wraps, so the angle needs no reduction and loses nothing at
// far positions. Its upper 32 bits, as a signed fraction of a turn, go to
// sincospi. A lane owns 16 elements of a head -- two 16-byte units that hold eight
// whole pairs in either layout -- and keeps their sines and cosines in registers
// for every head of its token.
//
// Two kinds of blocks in one launch. Token jobs: a warp takes one token and some
// of its heads -- q, and with a 16-bit cache k and v. Page jobs (e4m3): a block
// takes the new rows of one page of one KV head of K or V, since the scale
// they share needs their largest magnitude before the first code: one sweep for
// the maximum, rows kept in the page rescaled where the scale grows, one sweep
// for the codes (the rows come from L1 / L2 the second time).
//
// What bounds it: launch latency for a decode step, HBM for prompts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "attn_device.cuh"
#include "attn_launch.h"
#include "attn_paged_launch.h"

namespace attn {

namespace {

constexpr int kAppendThreads = 128;
constexpr unsigned kErrBadPageA = 0x4u;   // ATTN_DEVERR_BAD_PAGE

struct CacheF16 { using T = __half; };
struct CacheBf16 { using T = __nv_bfloat16; };
struct CacheE4m3 {};

// Eight consecutive elements of the input type as f32.
template <typename IN>
__device__ __forceinline__ void load8(const IN *p, float (&x)[8])
{
    if constexpr (sizeof(IN) == 4) {
        const float4 a = ld_dep(reinterpret_cast<const float4 *>(p)), b = ld_dep(reinterpret_cast<const float4 *>(p) + 1);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        const uint4 u = ld_dep(reinterpret_cast<const uint4 *>(p));
        unpack8<IN>(u, x);
    }
}

// Where a lane's two units of a head start, and whether they are rotated.
struct LaneUnits {
    int a, b;          // first elements of the two units
    bool rot;
    int pair0;         // first of the lane's eight pairs
};

template <int HD>
__device__ __forceinline__ LaneUnits lane_units(const AppendArgs &g, int l)
{
    const int h = g.rot_dim >> 4;             // lanes that rotate
    LaneUnits u;
    u.rot = l < h;
    u.pair0 = 8 * l;
    if (u.rot && !g.interleaved) {
        u.a = 8 * l;
        u.b = 8 * l + (g.rot_dim >> 1);
    } else {
        u.a = 16 * l;                         // the rest of a head starts at rot_dim = 16 h
        u.b = 16 * l + 8;
    }
    return u;
}

struct Turn {
    float c[8], s[8];
};

__device__ __forceinline__ void make_turn(const AppendArgs &g, const LaneUnits &u, int64_t pos, Turn &t)
{
    if (!u.rot) return;
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const ulonglong2 st = *reinterpret_cast<const ulonglong2 *>(g.steps + u.pair0 + j);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const unsigned long long ph = (unsigned long long)pos * (e ? st.y : st.x);
            const float half_turns = (float)(int)(ph >> 32) * 4.656612873077393e-10f;   // 2^-31
            float sn, cs;
            sincospif(half_turns, &sn, &cs);
            t.c[j + e] = cs * g.mscale;
            t.s[j + e] = sn * g.mscale;
        }
    }
}

__device__ __forceinline__ void turn(const AppendArgs &g, const Turn &t, float (&a)[8], float (&b)[8])
{
    if (!g.interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = a[j], y = b[j];
            a[j] = fmaf(x, t.c[j], -y * t.s[j]);
            b[j] = fmaf(y, t.c[j], x * t.s[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float x = a[2 * j], y = a[2 * j + 1];
            a[2 * j] = fmaf(x, t.c[j], -y * t.s[j]);
            a[2 * j + 1] = fmaf(y, t.c[j], x * t.s[j]);
            x = b[2 * j];
            y = b[2 * j + 1];
            b[2 * j] = fmaf(x, t.c[4 + j], -y * t.s[4 + j]);
            b[2 * j + 1] = fmaf(y, t.c[4 + j], x * t.s[4 + j]);
        }
    }
}

template <typename T>
__device__ __forceinline__ void store8_16(T *p, const float (&x)[8])
{
    uint4 u;
    u.x = float2_to_kv2<T>(x[0], x[1]);
    u.y = float2_to_kv2<T>(x[2], x[3]);
    u.z = float2_to_kv2<T>(x[4], x[5]);
    u.w = float2_to_kv2<T>(x[6], x[7]);
    *reinterpret_cast<uint4 *>(p) = u;
}

// Two f32 to two e4m3 codes, rounded to nearest even, at most 448 in magnitude.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// x / s: by the reciprocal where s is a power of two (exact), else by division.
struct Divisor {
    float s, r;
    bool pow2;
    explicit __device__ __forceinline__ Divisor(float v)
    {
        s = v;
        r = 1.f / v;
        pow2 = (__float_as_uint(v) & 0x7FFFFFu) == 0u;
    }
    __device__ __forceinline__ float operator()(float x) const { return pow2 ? x * r : __fdiv_rn(x, s); }
};

__device__ __forceinline__ void store8_e4m3(uint8_t *p, const float (&x)[8], const Divisor &d)
{
    uint2 u;
    u.x = to_e4m3x2(d(x[0]), d(x[1])) | to_e4m3x2(d(x[2]), d(x[3])) << 16;
    u.y = to_e4m3x2(d(x[4]), d(x[5])) | to_e4m3x2(d(x[6]), d(x[7])) << 16;
    *reinterpret_cast<uint2 *>(p) = u;
}

// The last s in [0, n) with value(s) <= x (value non-decreasing, value(0) <= x), by a warp.
template <class F>
__device__ __forceinline__ int warp_search(int n, int64_t x, int lane, F value)
{
    int lo = 0;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int i = lane * step;
        const bool le = i < n && value(lo + i) <= x;
        const int last = max(__popc(__ballot_sync(0xffffffffu, le)) - 1, 0);
        lo += last * step;
        n = min(step, n - last * step);
    }
    return lo;
}

__device__ __forceinline__ int64_t cu_at(const AppendArgs &g, int s)
{
    return g.cu ? min(max((int64_t)ld_dep(g.cu + s), (int64_t)0), g.n_tokens) : (int64_t)s * g.n_each;
}

// One head of one token.
template <int HD, typename IN, class CT>
__device__ __forceinline__ void token_jobs(const AppendArgs &g, int64_t job, int lane)
{
    constexpr int LPH = HD / 16, HPW = 32 / LPH;
    constexpr bool E8 = std::is_same<CT, CacheE4m3>::value;
    const int64_t tok = job / g.chunks;
    const int chunk = (int)(job - tok * g.chunks);
    if (tok >= g.n_tokens) return;
    const int nq = g.q ? g.n_head : 0;
    const int heads = nq + (E8 ? 0 : 2 * g.n_kv_head);
    const int s = g.cu ? warp_search(g.n_seq, tok, lane, [&](int i) { return cu_at(g, i); }) : (int)(tok / g.n_each);
    const int64_t end = cu_at(g, s + 1);
    if (tok >= end) return;                                     // behind the last sequence
    const int64_t last = ld_dep(g.positions + s);
    const int64_t pos = last + 1 - (end - tok);
    const int l = lane % LPH, hw = lane / LPH;
    const LaneUnits u = lane_units<HD>(g, l);
    Turn tr;
    make_turn(g, u, pos, tr);

    // where the token's row goes
    int64_t dst = -1;
    if constexpr (!E8) {
        const int64_t cap = (int64_t)g.max_pages * g.page_size;
        if (pos >= 0 && pos < cap) {
            const int pg = (int)(pos / g.page_size);
            const int page = ld_dep(g.table + (size_t)s * g.max_pages + pg);
            if (page >= 0 && page < g.n_pages)
                dst = page * g.page_stride + (pos - (int64_t)pg * g.page_size) * g.row_stride;
            else if (lane == 0 && chunk == 0)
                atomicOr(g.err, kErrBadPageA);
        } else if (last != -1 && lane == 0 && chunk == 0) {
            atomicOr(g.err, kErrPositionClamped);
        }
    }
    const int h1 = min((chunk + 1) * g.iters * HPW, heads);
#pragma unroll 2
    for (int hd0 = chunk * g.iters * HPW; hd0 < h1; hd0 += HPW) {
        const int h = hd0 + hw;
        if (h >= h1) continue;
        const IN *src;
        const bool is_q = h < nq, is_v = h >= nq + g.n_kv_head;
        const int kh = is_q ? h : is_v ? h - nq - g.n_kv_head : h - nq;
        if (is_q) src = static_cast<const IN *>(g.q) + tok * g.q_stride;
        else if (is_v) src = static_cast<const IN *>(g.v_new) + tok * g.v_stride;
        else src = static_cast<const IN *>(g.k_new) + tok * g.k_stride;
        src += (int64_t)kh * HD;
        float a[8], b[8];
        load8(src + u.a, a);
        load8(src + u.b, b);
        if (u.rot && !is_v) turn(g, tr, a, b);
        if (is_q) {
            float *o = g.q_out + (tok * g.n_head + kh) * HD;
            float4 *pa = reinterpret_cast<float4 *>(o + u.a), *pb = reinterpret_cast<float4 *>(o + u.b);
            pa[0] = make_float4(a[0], a[1], a[2], a[3]);
            pa[1] = make_float4(a[4], a[5], a[6], a[7]);
            pb[0] = make_float4(b[0], b[1], b[2], b[3]);
            pb[1] = make_float4(b[4], b[5], b[6], b[7]);
        } else if constexpr (!E8) {
            using T = typename CT::T;
            if (dst >= 0) {
                T *o = static_cast<T *>(is_v ? g.v : g.k) + dst + kh * g.head_stride;
                store8_16<T>(o + u.a, a);
                store8_16<T>(o + u.b, b);
            }
        }
    }
}

// The smallest power of two s in [2^-60, 2^60] with amax <= 448 s.
__device__ __forceinline__ float scale_for(float amax)
{
    const unsigned bits = __float_as_uint(amax);
    // amax = m 2^E with m in [1, 2); 448 = 1.75 x 2^8
    int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    e = min(max(e, -60), 60);
    return __uint_as_float((unsigned)(e + 127) << 23);
}

// The new rows of one page, one KV head, K or V (e4m3).
template <int HD, typename IN>
__device__ __forceinline__ void page_job(const AppendArgs &g, int64_t job)
{
    constexpr int LPH = HD / 16, TPB = kAppendThreads / LPH;      // tokens a sweep step takes
    __shared__ float sm_max[kAppendThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31;
    const int which = (int)(job % (2 * g.n_kv_head));
    const int64_t item = job / (2 * g.n_kv_head);
    const bool is_v = which >= g.n_kv_head;
    const int kh = is_v ? which - g.n_kv_head : which;

    int s;
    int64_t idx;                                                  // the item's page, counted from the first touched
    if (g.cu) {
        // sequence s may touch floor(cu[s+1] / page) - floor(cu[s] / page) + 2 pages at most
        auto first_item = [&](int i) { return cu_at(g, i) / g.page_size + 2 * (int64_t)i; };
        s = warp_search(g.n_seq, item, lane, first_item);
        idx = item - first_item(s);
    } else {
        const int64_t per = (g.n_each + g.page_size - 2) / g.page_size + 1;
        s = (int)(item / per);
        idx = item - s * per;
    }
    const int64_t tok0 = cu_at(g, s), tok1 = cu_at(g, s + 1);
    if (tok1 <= tok0) return;
    const int64_t cap = (int64_t)g.max_pages * g.page_size;
    const int64_t last = ld_dep(g.positions + s), first = last + 1 - (tok1 - tok0);
    if (idx == 0 && which == 0 && tid == 0 && last != -1 && (first < 0 || last >= cap))
        atomicOr(g.err, kErrPositionClamped);
    const int64_t pg = max(first, (int64_t)0) / g.page_size + idx;
    const int64_t r0 = max(max(first, (int64_t)0), pg * g.page_size);
    const int64_t r1 = min(min(last + 1, cap), (pg + 1) * g.page_size);
    if (r0 >= r1) return;
    const int page = ld_dep(g.table + (size_t)s * g.max_pages + pg);
    if (page < 0 || page >= g.n_pages) {
        if (which == 0 && tid == 0) atomicOr(g.err, kErrBadPageA);
        return;
    }
    const int rows = (int)(r1 - r0), at = (int)(r0 - pg * g.page_size);
    const IN *src = static_cast<const IN *>(is_v ? g.v_new : g.k_new);
    const int64_t stride = is_v ? g.v_stride : g.k_stride;
    src += (tok0 + (r0 - first)) * stride + (int64_t)kh * HD;
    uint8_t *dst = static_cast<uint8_t *>(is_v ? g.v : g.k) + page * g.page_stride + kh * g.head_stride;
    float *scale = (is_v ? g.v_scale : g.k_scale) + (size_t)page * g.n_kv_head + kh;
    const int l = tid % LPH, r = tid / LPH;
    const LaneUnits u = lane_units<HD>(g, l);

    auto row = [&](int i, float (&a)[8], float (&b)[8]) {
        load8(src + i * stride + u.a, a);
        load8(src + i * stride + u.b, b);
        if (u.rot && !is_v) {
            Turn tr;
            make_turn(g, u, r0 + i, tr);
            turn(g, tr, a, b);
        }
    };
    float amax = 0.f;
    for (int i = r; i < rows; i += TPB) {
        float a[8], b[8];
        row(i, a, b);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = fabsf(a[j]), y = fabsf(b[j]);
            if (x < INFINITY) amax = fmaxf(amax, x);
            if (y < INFINITY) amax = fmaxf(amax, y);
        }
    }
    amax = warp_max(amax);
    if (lane == 0) sm_max[tid >> 5] = amax;
    const float old = at > 0 ? ld_dep(scale) : 0.f;
    __syncthreads();                                             // also: every thread has read the old scale
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) amax = fmaxf(amax, sm_max[w]);
    const bool had = old > 0.f && old < INFINITY;
    const float now = had ? fmaxf(old, scale_for(amax)) : scale_for(amax);
    if (had && now > old) {                                      // rows [0, at) at the new scale
        const Divisor d(now);
        for (int i = r; i < at; i += TPB) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint8_t *p = dst + i * g.row_stride + 16 * l + 8 * e;
                const uint2 w = *reinterpret_cast<const uint2 *>(p);
                float x[8];
                const uint32_t h[2] = {w.x, w.y};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t f0, f1;
                    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
                        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
                        : "=r"(f0), "=r"(f1) : "r"(h[k]));
                    const float2 v0 = kv2_to_float2<__half>(f0), v1 = kv2_to_float2<__half>(f1);
                    x[4 * k] = v0.x * old; x[4 * k + 1] = v0.y * old;
                    x[4 * k + 2] = v1.x * old; x[4 * k + 3] = v1.y * old;
                }
                store8_e4m3(p, x, d);
            }
        }
    }
    if (tid == 0) *scale = now;
    const Divisor d(now);
    for (int i = r; i < rows; i += TPB) {
        float a[8], b[8];
        row(i, a, b);
        uint8_t *p = dst + (int64_t)(at + i) * g.row_stride;
        store8_e4m3(p + u.a, a, d);
        store8_e4m3(p + u.b, b, d);
    }
}

template <int HD, typename IN, class CT>
__global__ void __launch_bounds__(kAppendThreads) attn_append(const AppendArgs g)
{
    pdl_launch_dependents();
    pdl_wait();
    if constexpr (std::is_same<CT, CacheE4m3>::value) {
        if ((int64_t)blockIdx.x < g.page_blocks) {
            page_job<HD, IN>(g, blockIdx.x);
            return;
        }
    }
    const int64_t job = ((int64_t)blockIdx.x - g.page_blocks) * (kAppendThreads / 32) + (threadIdx.x >> 5);
    token_jobs<HD, IN, CT>(g, job, threadIdx.x & 31);
}

template <int HD, typename IN, class CT>
cudaError_t launch_it(AppendArgs g, cudaStream_t stream)
{
    constexpr bool E8 = std::is_same<CT, CacheE4m3>::value;
    constexpr int HPW = 32 / (HD / 16);
    int sms = 0;
    unsigned *err = nullptr;
    cudaError_t e = device_facts(&sms, &err);
    if (e != cudaSuccess) return e;
    g.err = err;
    const int heads = (g.q ? g.n_head : 0) + (E8 ? 0 : 2 * g.n_kv_head);
    const int groups = (heads + HPW - 1) / HPW;
    // A warp keeps its token's sines for every head group it takes: all of them where the tokens
    // alone fill the GPU (16 warps an SM), fewer where they do not, down to one.
    int64_t chunks = groups > 0 ? ((int64_t)sms * 16 + g.n_tokens - 1) / g.n_tokens : 0;
    if (chunks > groups) chunks = groups;
    g.iters = chunks > 0 ? (int)((groups + chunks - 1) / chunks) : 0;
    g.chunks = g.iters > 0 ? (groups + g.iters - 1) / g.iters : 0;
    g.page_blocks = E8 ? g.page_items * 2 * g.n_kv_head : 0;
    const int64_t warps = g.n_tokens * g.chunks;
    const int64_t blocks = g.page_blocks + (warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    const void *fn = reinterpret_cast<const void *>(&attn_append<HD, IN, CT>);
    void *args[] = {&g};
    return launch_pdl(fn, dim3((unsigned)blocks), dim3(kAppendThreads), 0, stream, args);
}

template <int HD, typename IN>
cudaError_t launch_in(const AppendRequest &r)
{
    switch (r.kv_type) {
    case kTypeF16: return launch_it<HD, IN, CacheF16>(r.a, r.stream);
    case kTypeBf16: return launch_it<HD, IN, CacheBf16>(r.a, r.stream);
    case kTypeE4m3: return launch_it<HD, IN, CacheE4m3>(r.a, r.stream);
    default: return cudaErrorInvalidValue;
    }
}

template <int HD>
cudaError_t launch_hd(const AppendRequest &r)
{
    switch (r.in_type) {
    case kTypeF32: return launch_in<HD, float>(r);
    case kTypeF16: return launch_in<HD, __half>(r);
    case kTypeBf16: return launch_in<HD, __nv_bfloat16>(r);
    default: return cudaErrorInvalidValue;
    }
}

} // namespace

cudaError_t launch_append(const AppendRequest &r)
{
    switch (r.head_dim) {
    case 64: return launch_hd<64>(r);
    case 128: return launch_hd<128>(r);
    case 256: return launch_hd<256>(r);
    default: return cudaErrorInvalidValue;
    }
}

} // namespace attn
