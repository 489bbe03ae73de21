// attn_rope_append.cu -- the append kernel: rotate the new tokens' q and k by
// position and write k and v rows into the paged cache.
//
// Mathematics. Pair i of a head turns by position * steps[i] / 2^64 of a turn;
// the 64-bit product wraps, so the angle needs no reduction and loses nothing at
// far positions. A lane owns 16 elements of a head -- two 16-byte units that hold eight
// whole pairs in either layout -- and keeps their sines and cosines in registers
// for every head of its token.
//
// Two kinds of blocks in one launch. Token jobs: a warp takes one token and some
// of its heads -- q, and with a 16-bit cache k and v. Page jobs (e4m3): a block
// takes the new rows of one page of one KV head, since the scale they share needs
// their largest magnitude before the first code: the rows are staged in shared memory,
// one sweep for the rotation and the maximum, rows kept in the page rescaled where the
// scale grows, one sweep for the codes.
//
// What bounds it. HBM for prompts: 7370 bfloat16 tokens of 28 + 4 heads of 128 into e4m3
// pages 30.3 us, 0.88 of the copy bandwidth (three fifths of the bytes are writes); 8399
// float32 tokens of 16 + 2 heads of 256 into bfloat16 pages 51.2 us, 0.94. Launch latency for
// a decode step: one token 3.6 us, 64 sequences of one 3.1 (a chain of position, table,
// old scale and store).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "attn_device.cuh"
#include "attn_launch.h"
#include "attn_paged_launch.h"

namespace attn {

namespace {

constexpr int kAppendMost = 256;          // threads of a block: 128, more for the page jobs of prompts
constexpr unsigned kErrBadPageA = 0x4u;   // ATTN_DEVERR_BAD_PAGE

struct CacheF16 { using T = __half; };
struct CacheBf16 { using T = __nv_bfloat16; };
struct CacheE4m3 {};

// 32 bytes, in one access where `wide` says that the address is a multiple of 32, else in two.
__device__ __forceinline__ void st32(void *p, const uint32_t *w, bool wide)
{
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     :: "l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// Where a lane's two units of a head start, and whether they are rotated. Halves: the lanes' first units
// follow each other, and their second ones; interleaved: a lane's two units do.
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
    if (g.interleaved) {
        u.a = 16 * l;
        u.b = 16 * l + 8;
    } else if (u.rot) {
        u.a = 8 * l;
        u.b = 8 * l + (g.rot_dim >> 1);
    } else {                                  // what is not rotated, in halves too
        u.a = g.rot_dim + 8 * (l - h);
        u.b = u.a + ((HD - g.rot_dim) >> 1);
    }
    return u;
}

// Head rows as they are stored, in shared memory: `kSlots` places for each group of HD / 16 lanes, which takes a
// head together. Asynchronous copies fill them, so that many loads are on their way without registers and
// with one copy of the code that uses them (unrolled over registers it no longer fitted the instruction
// cache). Lane l copies every LPH-th 16-byte part from the l-th on -- whole sectors -- and reads its own
// units, so a __syncwarp stands between a place's copies and its reads, and between those and the next copies.
template <int HD, typename IN>
struct Stage {
    static constexpr int LPH = HD / 16, ROW = HD * (int)sizeof(IN), PARTS = sizeof(IN);   // parts of a lane: 2 or 4
    static constexpr int kSlots = 16 / PARTS;                      // 256 bytes a thread
    static constexpr size_t bytes(int threads) { return (size_t)kSlots * PARTS * 16 * threads; }
    uint32_t base;                                                 // shared address of the group's first place
    uint32_t step;                                                 // bytes from a place to the next
    int l;

    __device__ __forceinline__ explicit Stage(const void *smem)
    {
        base = smem_u32(smem) + threadIdx.x / LPH * ROW;
        step = blockDim.x / LPH * ROW;
        l = threadIdx.x % LPH;
    }
    __device__ __forceinline__ void fetch(int slot, const IN *row) const
    {
#pragma unroll
        for (int p = 0; p < PARTS; ++p)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                         :: "r"(base + slot * step + (l + p * LPH) * 16),
                            "l"(reinterpret_cast<const uint8_t *>(row) + (l + p * LPH) * 16) : "memory");
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    template <int N> static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }
    __device__ __forceinline__ void values(int slot, const LaneUnits &u, float (&a)[8], float (&b)[8]) const
    {
        eight(base + slot * step + u.a * (int)sizeof(IN), a);
        eight(base + slot * step + u.b * (int)sizeof(IN), b);
    }
    static __device__ __forceinline__ void eight(uint32_t at, float (&x)[8])
    {
        const uint4 w = lds(at);
        if constexpr (PARTS == 4) {
            const uint4 v = lds(at + 16);
            x[0] = __uint_as_float(w.x); x[1] = __uint_as_float(w.y);
            x[2] = __uint_as_float(w.z); x[3] = __uint_as_float(w.w);
            x[4] = __uint_as_float(v.x); x[5] = __uint_as_float(v.y);
            x[6] = __uint_as_float(v.z); x[7] = __uint_as_float(v.w);
        } else {
            unpack8<IN>(w, x);
        }
    }
    static __device__ __forceinline__ uint4 lds(uint32_t at)
    {
        uint4 w;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at) : "memory");
        return w;
    }
};

struct Turn {
    float c[8], s[8];
};

// Sine and cosine of `pos` steps, to 4.4 2^-24 + 2 pi 2^-32. The wrapping product is the angle in 2^-64 turns; the
// quarter turn nearest to its upper half leaves r in [-1/8, 1/8] turns, an integer in 2^-32 turns without a loss
// (wrapping too, so unsigned), then rounded to 24 bits. There the Taylor series of sine
// (to x^9, remainder 2e-9) and cosine (to x^10, 1e-10) hold, and the quarter turns swap them and set signs.
// (sincospif made the rotation of a token the larger part of a warp's time.)
__device__ __forceinline__ void angle(int64_t pos, uint64_t step, float &c, float &s)
{
    const unsigned hi = (unsigned)(((uint64_t)pos * step) >> 32);
    const unsigned quarter = (hi + 0x20000000u) >> 30;
    const float x = (float)(int)(hi - (quarter << 30)) * 1.4629180792671596e-9f;   // 2 pi 2^-32
    const float z = x * x;
    float ps = 2.7557319e-6f;                        // 1 / 9!
    ps = fmaf(ps, z, -1.9841270e-4f);                // 1 / 7!
    ps = fmaf(ps, z, 8.3333333e-3f);                 // 1 / 5!
    ps = fmaf(ps, z, -1.6666667e-1f);                // 1 / 3!
    const float sn = fmaf(ps * z, x, x);
    float pc = -2.7557319e-7f;                       // 1 / 10!
    pc = fmaf(pc, z, 2.4801587e-5f);                 // 1 / 8!
    pc = fmaf(pc, z, -1.3888889e-3f);                // 1 / 6!
    pc = fmaf(pc, z, 4.1666667e-2f);                 // 1 / 4!
    pc = fmaf(pc, z, -0.5f);
    const float cn = fmaf(pc, z, 1.f);
    const float a = quarter & 1 ? cn : sn, b = quarter & 1 ? sn : cn;
    s = quarter & 2 ? -a : a;
    c = (quarter + 1) & 2 ? -b : b;
}

// The steps of a lane's eight pairs, loaded before the position is known (one token 3.8 -> 3.5 us)
struct Steps {
    ulonglong2 st[4];
    __device__ __forceinline__ void load(const uint64_t *steps, const LaneUnits &u)
    {
#pragma unroll
        for (int j = 0; j < 4; ++j) st[j] = u.rot ? reinterpret_cast<const ulonglong2 *>(steps + u.pair0)[j] : make_ulonglong2(0, 0);
    }
};

__device__ __forceinline__ void make_turn(const AppendArgs &g, const Steps &p, int64_t pos, Turn &t)
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        angle(pos, p.st[j].x, t.c[2 * j], t.s[2 * j]);
        angle(pos, p.st[j].y, t.c[2 * j + 1], t.s[2 * j + 1]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        t.c[j] *= g.mscale;
        t.s[j] *= g.mscale;
    }
}

__device__ __forceinline__ void turn_pair(float &x, float &y, float c, float s)
{
    const float a = x, b = y;
    x = fmaf(a, c, -b * s);
    y = fmaf(b, c, a * s);
}

__device__ __forceinline__ void turn(const AppendArgs &g, const Turn &t, float (&a)[8], float (&b)[8])
{
    if (!g.interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) turn_pair(a[j], b[j], t.c[j], t.s[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            turn_pair(a[2 * j], a[2 * j + 1], t.c[j], t.s[j]);
            turn_pair(b[2 * j], b[2 * j + 1], t.c[4 + j], t.s[4 + j]);
        }
    }
}

template <typename T>
__device__ __forceinline__ void store_16bit(const AppendArgs &g, T *row, const LaneUnits &u, const float (&a)[8],
                                            const float (&b)[8])
{
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        w[j] = float2_to_kv2<T>(a[2 * j], a[2 * j + 1]);
        w[4 + j] = float2_to_kv2<T>(b[2 * j], b[2 * j + 1]);
    }
    if (g.interleaved) {
        st32(row + u.a, w, g.wide);
    } else {
        *reinterpret_cast<uint4 *>(row + u.a) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4 *>(row + u.b) = make_uint4(w[4], w[5], w[6], w[7]);
    }
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

__device__ __forceinline__ uint2 e4m3x8(const float (&x)[8], const Divisor &d)
{
    return make_uint2(to_e4m3x2(d(x[0]), d(x[1])) | to_e4m3x2(d(x[2]), d(x[3])) << 16,
                      to_e4m3x2(d(x[4]), d(x[5])) | to_e4m3x2(d(x[6]), d(x[7])) << 16);
}

// The last s in [0, n) with value(s) <= x (value non-decreasing, value(0) <= x), by a warp.
template <class F>
__device__ __forceinline__ int warp_search(int n, int x, int lane, F value)
{
    int lo = 0;
    while (n > 1) {
        const int step = (n + 31) >> 5;
        const int i = lane * step;
        const bool le = i < n && value(lo + i) <= x;
        const int last = max(__popc(__ballot_sync(0xffffffffu, le)) - 1, 0);
        lo += last * step;
        n = min(step, n - last * step);
    }
    return lo;
}

// Numbers that every warp of the call looks up, through L1 (kept behind the wait for the grid before, which makes
// what it wrote visible). Through L2 thousands of warps asked for the same few sectors at once, which was half of
// the time of short prompts (52 sequences of 9 to 38 tokens 13.1 -> 7.9 us, six prompts of 7370 34 -> 31).
__device__ __forceinline__ int ld_shared_by_all(const int *p)
{
    int v;
    asm volatile("ld.global.ca.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ int cu_at(const AppendArgs &g, int s)
{
    return g.cu ? min(max(ld_shared_by_all(g.cu + s), 0), (int)g.n_tokens) : s * (int)g.n_each;
}

// One token, `iters` groups of HPW of its heads: of q, then (16-bit cache) of k and v. The loads of the next D
// groups are always on their way. Warps in order take tokens in order: a sweep over memory (with each warp at a
// place of its own, over its share of the tokens, prompts took a third longer).
template <int HD, typename IN, class CT>
__device__ __forceinline__ void token_job(const AppendArgs &g, const Stage<HD, IN> &stage, int job, int lane)
{
    constexpr int LPH = HD / 16, HPW = 32 / LPH, D = Stage<HD, IN>::kSlots;
    constexpr bool E8 = std::is_same<CT, CacheE4m3>::value;
    const int at_tok = div(g.by_chunks, job), chunk = job - at_tok * g.chunks;
    const int64_t tok = at_tok;
    if (tok >= g.n_tokens) return;
    const int nq = g.q ? g.n_head : 0;
    const int heads = nq + (E8 ? 0 : 2 * g.n_kv_head);
    const int l = lane % LPH, h0 = chunk * g.iters * HPW + lane / LPH;   // the lane's first head
    const int h1 = min((chunk + 1) * g.iters * HPW, heads);
    const LaneUnits u = lane_units<HD>(g, l);
    auto fetch = [&](int i) {                                     // always a copy group, so that waiting counts
        const int h = h0 + i * HPW;
        if (h < h1) {
            const IN *src = h < nq                 ? static_cast<const IN *>(g.q) + tok * g.q_stride + (int64_t)h * HD
                            : h < nq + g.n_kv_head ? static_cast<const IN *>(g.k_new) + tok * g.k_stride + (int64_t)(h - nq) * HD
                                                   : static_cast<const IN *>(g.v_new) + tok * g.v_stride +
                                                         (int64_t)(h - nq - g.n_kv_head) * HD;
            stage.fetch(i % D, src);
        }
        stage.commit();
    };
#pragma unroll 1
    for (int i = 0; i < D; ++i) fetch(i);                         // ... while the token's position is found
    Steps steps;
    steps.load(g.steps, u);
    const int s = g.cu ? warp_search(g.n_seq, at_tok, lane, [&](int i) { return cu_at(g, i); }) : div(g.by_each, at_tok);
    const int64_t end = cu_at(g, s + 1);
    const int64_t last = ld_shared_by_all(g.positions + s);
    const int64_t pos = last + 1 - (end - tok);
    int page = -1;
    int64_t off = -1;                                             // of the token's row in its page; -1: no row
    if (!E8 && tok < end) {
        if (pos >= 0 && pos < (int64_t)g.max_pages * g.page_size) {
            const int pg = div(g.by_page, (int)pos);
            off = (pos - (int64_t)pg * g.page_size) * g.row_stride;
            page = ld_dep(g.table + (size_t)s * g.max_pages + pg);
        } else if (last != -1 && lane == 0 && chunk == 0) {
            atomicOr(g.err, kErrPositionClamped);
        }
    }
    Turn tr;
    if (u.rot) make_turn(g, steps, pos, tr);
    const int n = tok < end ? g.iters : 0;                        // behind the last sequence: nothing
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        stage.template wait<D - 1>();
        __syncwarp();
        const int h = h0 + i * HPW;
        if (h < h1) {
            const bool is_q = h < nq, is_v = h >= nq + g.n_kv_head;
            float a[8], b[8];
            stage.values(i % D, u, a, b);
            if (u.rot && !is_v) turn(g, tr, a, b);
            if (is_q) {
                float *o = g.q_out + (tok * g.n_head + h) * HD;
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(a[j]);
                st32(o + u.a, w, g.wide);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(b[j]);
                st32(o + u.b, w, g.wide);
            } else if constexpr (!E8) {
                using T = typename CT::T;
                const int kh = is_v ? h - nq - g.n_kv_head : h - nq;
                if (off >= 0) {
                    if ((unsigned)page < (unsigned)g.n_pages)
                        store_16bit<T>(g, static_cast<T *>(is_v ? g.v : g.k) + page * g.page_stride + off + kh * g.head_stride,
                                       u, a, b);
                    else if (l == 0)
                        atomicOr(g.err, kErrBadPageA);
                }
            }
        }
        __syncwarp();
        fetch(i + D);
    }
    stage.template wait<0>();
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

// The new rows of one page and KV head, K and V or one of them (e4m3). A thread takes every TPB-th row; as many
// of its rows as the stage holds are read once, later ones (large pages) once for the maximum and once for
// the codes. K's angles are computed both times, which costs less than keeping the values.
template <int HD, typename IN>
__device__ __forceinline__ void page_job(const AppendArgs &g, const Stage<HD, IN> &stage, int job)
{
    constexpr int LPH = HD / 16;
    __shared__ float sm_max[2][kAppendMost / 32];
    const int tid = threadIdx.x, lane = tid & 31, TPB = blockDim.x / LPH;
    const int per_item = g.kv_apart ? 2 * g.n_kv_head : g.n_kv_head;
    const int item = div(g.by_item, job), which = job - item * per_item;
    const int w0 = which < g.n_kv_head ? 0 : 1, w1 = g.kv_apart ? w0 + 1 : 2;   // K: 0, V: 1
    const int kh = which - w0 * g.n_kv_head;

    int s, idx;                                                   // idx: the item's page, counted from the first touched
    if (g.cu) {
        // sequence s may touch floor(cu[s+1] / page) - floor(cu[s] / page) + 2 pages at most
        auto first_item = [&](int i) { return div(g.by_page, cu_at(g, i)) + 2 * i; };
        s = warp_search(g.n_seq, item, lane, first_item);
        idx = item - first_item(s);
    } else {
        const int per = div(g.by_page, (int)g.n_each + g.page_size - 2) + 1;
        s = div(g.by_seq, item);
        idx = item - s * per;
    }
    const int64_t tok0 = cu_at(g, s), tok1 = cu_at(g, s + 1);
    if (tok1 <= tok0) return;
    const int64_t cap = (int64_t)g.max_pages * g.page_size;
    const int64_t last = ld_shared_by_all(g.positions + s), first = last + 1 - (tok1 - tok0);
    if (idx == 0 && which == 0 && tid == 0 && last != -1 && (first < 0 || last >= cap))
        atomicOr(g.err, kErrPositionClamped);
    const int64_t pg = div(g.by_page, (int)min(max(first, (int64_t)0), cap)) + (int64_t)idx;
    const int64_t r0 = max(max(first, (int64_t)0), pg * g.page_size);
    const int64_t r1 = min(min(last + 1, cap), (pg + 1) * g.page_size);
    if (r0 >= r1) return;
    const int rows = (int)(r1 - r0), at = (int)(r0 - pg * g.page_size);
    const int l = tid % LPH, r = tid / LPH;
    const LaneUnits u = lane_units<HD>(g, l);
    const int64_t tok = tok0 + (r0 - first);
    auto source = [&](int w, int64_t token) {
        const int64_t stride = w ? g.v_stride : g.k_stride;
        return static_cast<const IN *>(w ? g.v_new : g.k_new) + token * stride + (int64_t)kh * HD;
    };
    // rows of a thread that stay in the stage, each of K and V; where there are more, the last place is for those
    const int places = Stage<HD, IN>::kSlots / (w1 - w0);
    const int kept = rows > places * TPB ? places - 1 : places;
#pragma unroll 1
    for (int w = w0; w < w1; ++w)
#pragma unroll 1
        for (int k = 0; k < kept && r + k * TPB < rows; ++k) stage.fetch((w - w0) * places + k, source(w, tok + r + k * TPB));
    __shared__ __align__(16) uint64_t sm_steps[HD / 2];
    if (w0 == 0 && tid < g.rot_dim / 4)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_u32(sm_steps + 2 * tid)), "l"(g.steps + 2 * tid) : "memory");
    stage.commit();
    const int page = ld_dep(g.table + (size_t)s * g.max_pages + pg);
    const bool there = page >= 0 && page < g.n_pages;
    if (!there && which == 0 && tid == 0) atomicOr(g.err, kErrBadPageA);
    const size_t sc = (size_t)page * g.n_kv_head + kh;
    __shared__ float sm_old[2], sm_now[2];                        // the page's scales, before and after
    if (tid >= w0 && tid < w1) sm_old[tid] = there && at > 0 ? ld_dep((tid ? g.v_scale : g.k_scale) + sc) : 0.f;
    __shared__ float2 by[HD / 2];                                 // pair i's cosine and sine of TPB positions
    if (w0 == 0 && rows > TPB)
        for (int i = tid; i < g.rot_dim / 2; i += blockDim.x) angle(TPB, g.steps[i], by[i].x, by[i].y);
    // what the sweeps need now and then, out of the registers
    __shared__ int64_t sm_tok, sm_base, sm_r0;
    if (tid == 0) {
        sm_tok = tok;
        sm_base = page * g.page_stride + kh * g.head_stride;
        sm_r0 = r0;
    }
    stage.template wait<0>();
    __syncthreads();
    if (!there) return;
    const volatile int64_t &vtok = sm_tok, &vbase = sm_base, &vr0 = sm_r0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
        for (int w = w0; w < w1; ++w) {
            const Divisor d(pass ? sm_now[w] : 1.f);
            const bool turned = u.rot && w == 0;
            float most = 0.f;
            Turn tr;
#pragma unroll 1
            for (int i = r, k = 0; i - r < rows; i += TPB, ++k) {     // together: a row past the last is not used
                const bool real = i < rows;
                int slot = (w - w0) * places + k;
                if (k >= kept) {
                    slot = (w - w0) * places + kept;
                    __syncwarp();
                    if (real) stage.fetch(slot, source(w, vtok + i));
                    stage.commit();
                    stage.template wait<0>();
                    __syncwarp();
                }
                if (!real) continue;
                float a[8], b[8];
                stage.values(slot, u, a, b);
                if (turned) {
                    // one row in four from its position, the others from the one before (three products of 32-bit
                    // rounding at most)
                    if (k % 4 == 0) {
                        Steps steps;
                        steps.load(sm_steps, u);
                        make_turn(g, steps, vr0 + i, tr);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) turn_pair(tr.c[j], tr.s[j], by[u.pair0 + j].x, by[u.pair0 + j].y);
                    }
                    turn(g, tr, a, b);
                }
                if (pass == 0) {
                    float m = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) m = fmaxf(m, fmaxf(fabsf(a[j]), fabsf(b[j])));
                    if (m == INFINITY) {                              // infinities do not count
                        m = 0.f;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float y = fabsf(a[j]), z = fabsf(b[j]);
                            if (y < INFINITY) m = fmaxf(m, y);
                            if (z < INFINITY) m = fmaxf(m, z);
                        }
                    }
                    most = fmaxf(most, m);
                } else {
                    uint8_t *p = static_cast<uint8_t *>(w ? g.v : g.k) + vbase + (int64_t)(at + i) * g.row_stride;
                    const uint2 ca = e4m3x8(a, d), cb = e4m3x8(b, d);
                    if (g.interleaved) {
                        *reinterpret_cast<uint4 *>(p + u.a) = make_uint4(ca.x, ca.y, cb.x, cb.y);
                    } else {
                        *reinterpret_cast<uint2 *>(p + u.a) = ca;
                        *reinterpret_cast<uint2 *>(p + u.b) = cb;
                    }
                }
            }
            if (pass == 0) {
                most = warp_max(most);
                if (lane == 0) sm_max[w][tid >> 5] = most;
            }
        }
        if (pass) break;
        __syncthreads();
#pragma unroll 1
        for (int w = w0; w < w1; ++w) {
            const float o = sm_old[w];
            float m = 0.f;
            for (int i = 0; i < (int)blockDim.x / 32; ++i) m = fmaxf(m, sm_max[w][i]);
            const float n = fabsf(o) < INFINITY ? fmaxf(fabsf(o), scale_for(m)) : scale_for(m);
            if (tid == 0) {
                sm_now[w] = n;
                (w ? g.v_scale : g.k_scale)[sc] = n;
            }
            if (at == 0 || n == o || !(fabsf(o) < INFINITY)) continue;
            // rows [0, at) at the new scale: exact but for the codes' rounding where n is a power of two or -o
            const float ratio = o / n;
#pragma unroll 1
            for (int i = r; i < at; i += TPB) {
                uint8_t *p = static_cast<uint8_t *>(w ? g.v : g.k) + vbase + i * g.row_stride + 16 * l;
                uint4 c = *reinterpret_cast<const uint4 *>(p);
                uint32_t *cw = &c.x;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t f0, f1;
                    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
                        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
                        : "=r"(f0), "=r"(f1) : "r"(cw[k]));
                    const float2 v0 = kv2_to_float2<__half>(f0), v1 = kv2_to_float2<__half>(f1);
                    cw[k] = to_e4m3x2(v0.x * ratio, v0.y * ratio) | to_e4m3x2(v1.x * ratio, v1.y * ratio) << 16;
                }
                *reinterpret_cast<uint4 *>(p) = c;
            }
        }
        __syncthreads();
    }
}

template <int HD, typename IN, class CT>
__global__ void __launch_bounds__(kAppendMost, 3) attn_append(const AppendArgs g)
{
    extern __shared__ uint4 stage_smem[];
    const Stage<HD, IN> stage(stage_smem);
    // no early start for the kernel after this one: it is the attention over this cache, whose blocks fill an SM and
    // would find it in pieces beside these (32 sequences, both calls: 171.7 us with an early start, 165.2 without)
    pdl_wait();
    int block = (int)blockIdx.x;
    if constexpr (std::is_same<CT, CacheE4m3>::value) {
        if (block < g.page_blocks) {
            page_job<HD, IN>(g, stage, block);
            return;
        }
        block -= (int)g.page_blocks;
    }
    token_job<HD, IN, CT>(g, stage, block * (int)(blockDim.x / 32) + (int)(threadIdx.x >> 5), threadIdx.x & 31);
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
    // A warp keeps its token's sines for every head group it takes: all of them where the tokens alone fill
    // the GPU (16 warps an SM), fewer where they do not, down to one.
    int64_t chunks = groups > 0 ? ((int64_t)sms * 16 + g.n_tokens - 1) / g.n_tokens : 0;
    if (chunks > groups) chunks = groups;
    g.iters = chunks > 0 ? (int)((groups + chunks - 1) / chunks) : 0;
    g.chunks = g.iters > 0 ? (groups + g.iters - 1) / g.iters : 0;
    // page jobs that are all resident at once even so: K and V in jobs of their own, half as long (a step of 32
    // sequences of 8 KV heads 6.2 -> 5.2 us)
    g.kv_apart = g.page_items * g.n_kv_head * 2 <= (int64_t)sms * 6;
    // threads for as many rows as a call can bring to a page, while the stage holds them
    int threads = 128;
    if (E8) {
        const int64_t most = g.cu ? g.n_tokens : g.n_each;
        const int64_t rows = most < g.page_size ? most : g.page_size;
        const int places = Stage<HD, IN>::kSlots / (g.kv_apart ? 1 : 2);
        while (threads < kAppendMost && threads * places < rows * (HD / 16)) threads *= 2;
    }
    // page jobs first: they wait more than they move, and token jobs fill in behind them (7370 tokens: 34 us;
    // token jobs first 47, evenly mixed 40)
    g.page_blocks = E8 ? g.page_items * g.n_kv_head * (g.kv_apart ? 2 : 1) : 0;
    const int64_t warps = g.n_tokens * g.chunks;
    const int64_t blocks = g.page_blocks + (warps + threads / 32 - 1) / (threads / 32);
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    g.by_page = fast_div((unsigned)g.page_size);
    g.by_chunks = fast_div((unsigned)(g.chunks > 0 ? g.chunks : 1));
    g.by_each = fast_div((unsigned)(g.n_each > 0 ? g.n_each : 1));
    g.by_item = fast_div((unsigned)(g.n_kv_head * (g.kv_apart ? 2 : 1)));
    g.by_seq = fast_div((unsigned)((g.n_each + g.page_size - 2) / g.page_size + 1));
    const void *fn = reinterpret_cast<const void *>(&attn_append<HD, IN, CT>);
    e = ensure_smem_attr(fn, (int)Stage<HD, IN>::bytes(kAppendMost));
    if (e != cudaSuccess) return e;
    void *args[] = {&g};
    return launch_pdl(fn, dim3((unsigned)blocks), dim3((unsigned)threads), Stage<HD, IN>::bytes(threads), stream, args);
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
