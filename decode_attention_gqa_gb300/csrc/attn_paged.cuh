// attn_paged.cuh -- the split partial kernel over a paged cache.
//
// Mathematics. For a (query row, head) slot at position x over the cache rows j it sees,
//     s_j = rules(scale q.k_j),  o = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j log2 e - m),
// one pass with a running reference m; a split stores (m, sum p, sum p v) and
// attn_combine merges the splits (with one split the block writes o itself).
// An e4m3 cache holds codes with one scale per page and KV head: q.k_j is the
// product with the codes times the page's K scale, one multiplication per
// score, and the V scale multiplies p before P.V. The running reference follows
// s + log2 of the V scale (rounded up), so that p times the scale stays in
// the 16-bit range whatever the scales are; sum p stays in f32.
//
// Layout. One block per (split, KV head and group of 8 or 16 slots, sequence):
// 4 compute warps and a producer warp over a ring of 64-row stages. A 16-row
// slice of a stage belongs to one compute warp and lies in one page; the
// producer looks the pages up, loads each page's piece by TMA (boxes of
// gcd(page_size, 64) rows, swizzled) and leaves the page's scales with the
// stage. Rows a block does not attend are neither waited for nor used.
//
// Tensor cores. 16x8x16 MMAs, f32 accumulation; q and p as hi + lo pairs of the
// cache's type (f16 for e4m3, whose codes f16 holds exactly). With 8 slots the
// 16 MMA rows are the hi and the lo parts, with 16 slots each part has its own
// MMA. The order of a dot product's terms is free, so a lane's share of a K row
// is contiguous: 16-byte shared loads give it whole k-steps, with no
// ldmatrix and, for 8 bits, no shuffling before the conversion. 8-bit V
// needs pairs of rows in a register: a lane reads its four rows' 16
// contiguous dimensions and pairs bytes of two rows before converting.
//
// What bounds it: HBM for long caches. The measured rates stand with the
// launch rules in attn_paged_impl.cuh.
#pragma once

#include <cuda_fp8.h>

#include "attn_device.cuh"
#include "attn_paged_launch.h"

namespace attn {

struct E4m3 {};       // tag of the 8-bit cache

template <typename KV> struct PagedMma { using T = KV; };
template <> struct PagedMma<E4m3> { using T = __half; };

constexpr unsigned kErrBadPage = 0x4u;    // ATTN_DEVERR_BAD_PAGE

// Two e4m3 codes (in 16 bits) to two f16 values, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t w)
{
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(w));
    return r;
}

__device__ __forceinline__ void e4m3x4_to_half4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
}

__device__ __forceinline__ uint4 lds128(uint32_t p)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
    return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t p)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p));
    return v;
}

__device__ __forceinline__ void ldsm_x4_trans(uint32_t (&r)[4], uint32_t p)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(p));
}

template <int HD_, int SLOTS_, typename KV_, int S_, int MINB_>
struct PagedCfg {
    static constexpr int HD = HD_, SLOTS = SLOTS_, S = S_, MIN_BLOCKS = MINB_;
    using KV = KV_;
    using MT = typename PagedMma<KV>::T;
    static constexpr bool E8 = std::is_same<KV, E4m3>::value;
    static constexpr int ES = E8 ? 1 : 2;
    static constexpr int NWC = 4, WR = 16, TILE = NWC * WR, NSL = TILE / WR;
    static constexpr int THREADS = (NWC + 1) * 32;
    static constexpr int ROWB = HD * ES;                          // bytes of a row of one head
    static constexpr int CHB = ROWB < 128 ? ROWB : 128;           // bytes of a swizzled chunk's row
    static constexpr int NCH = ROWB / CHB;
    static constexpr int CW = CHB / ES;                           // dimensions of a chunk
    static constexpr uint32_t TILE_BYTES = (uint32_t)TILE * ROWB;
    static constexpr uint32_t STAGE_BYTES = 2 * TILE_BYTES;
    static constexpr int KSTEPS = HD / 16, NTD = HD / 8;
    static constexpr int KPC = CW / 16;                           // k-steps of a chunk
    static constexpr int PARTS = SLOTS / 8;                       // Q operands: 1 (hi over lo) or 2 (hi, lo)
    static constexpr int SPL = SLOTS / 8;                         // slots a lane owns
    static constexpr bool Q_REGS = E8 && HD <= 128 && SLOTS == 8;   // else they are read per k-step (no spills)
    static constexpr uint32_t Q_BYTES = (uint32_t)PARTS * KSTEPS * 512;   // fragments, 16 bytes a lane
    static constexpr uint32_t OFF_Q = S * STAGE_BYTES;
    static constexpr uint32_t OFF_SLOT = OFF_Q + Q_BYTES;         // SlotInfo[SLOTS]
    static constexpr uint32_t OFF_INFO = OFF_SLOT + SLOTS * 16;   // SliceInfo[S][NSL]
    static constexpr uint32_t OFF_BAR = OFF_INFO + S * NSL * 16;
    static constexpr uint32_t SMEM_BYTES = OFF_BAR + 2 * S * 8 + 16 + 1024;
    static constexpr int MS = merge_stride<HD>();
    static constexpr uint32_t OFF_MO = (uint32_t)2 * NWC * SLOTS;   // floats, a multiple of 4
    static_assert((OFF_MO + (uint32_t)NWC * SLOTS * MS) * 4 <= S * STAGE_BYTES, "merge area must fit in the ring");
    static_assert(SMEM_BYTES <= 227 * 1024 && MIN_BLOCKS * (SMEM_BYTES + 1024u) <= 233472u, "shared memory");
    static_assert((TILE_BYTES / NCH) % 1024 == 0, "swizzled chunks stay 1024-aligned");

    // Rows are stored as chunks of CHB bytes, swizzled as TMA writes them. `row` is the offset of a row
    // with its swizzle bits set; `unit` adds 16-byte unit U: one exclusive or with a constant
    // (the base is 1024-aligned), so no address has to be kept in a register.
    static __device__ __forceinline__ uint32_t row(int r)
    {
        return CHB == 128 ? (uint32_t)(r * 128 + ((r & 7) << 4)) : (uint32_t)(r * 64 + (((r >> 1) & 3) << 4));
    }
    static __device__ __forceinline__ uint32_t unit(uint32_t base_row, int U)
    {
        return CHB == 128 ? (base_row ^ (uint32_t)((U & 7) << 4)) + (uint32_t)(U >> 3) * (TILE * 128)
                          : base_row ^ (uint32_t)(U << 4);
    }
};

struct __align__(16) SliceInfo {  // of one 16-row slice of a stage
    int page;             // -1: not there
    float ks, vs;
    int pad;
};

struct __align__(16) SlotInfo {   // of one (query row, head) slot of the block
    float inv;            // undoes the power of two q was scaled by
    float slope;          // times log2 e
    int t;                // query row, -1: no such slot
    int pad;
};

// The rows the slots of query rows [t0, t1] see, as [first row of t0, last row of t1]
struct SlotRows {
    int nkv, base;        // row t's position is base + t
    int start, window;
    __device__ __forceinline__ int last(int t) const { return base + t; }
    __device__ __forceinline__ int low(int t) const
    {
        const int w = window > 0 ? base + t - window + 1 : 0;
        return max(max(start, w), 0);
    }
};

template <class C, bool RULES>
struct PagedWarp {
    static constexpr float TAU = 8.f, OFF = 7.f;      // lazy rescale threshold, headroom of p (log2)
    using MT = typename C::MT;
    uint32_t qa[C::Q_REGS ? C::KSTEPS : 1][4];
    float o[C::NTD][4];
    float m[C::SPL], l[C::SPL];

    static __device__ __forceinline__ SlotInfo slot(uint32_t smem, int k, int lane)
    {
        const uint4 u = lds128(smem + C::OFF_SLOT + ((lane >> 2) + 8 * k) * 16);
        return SlotInfo{__uint_as_float(u.x), __uint_as_float(u.y), (int)u.z, 0};
    }

    __device__ __forceinline__ void init(uint32_t smem, int lane)
    {
        if constexpr (C::Q_REGS) {
#pragma unroll
            for (int kk = 0; kk < C::KSTEPS; ++kk) load_q(qa[kk], smem, 0, kk, lane);
        }
#pragma unroll
        for (int n = 0; n < C::NTD; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
#pragma unroll
        for (int k = 0; k < C::SPL; ++k) {
            m[k] = -INFINITY;
            l[k] = 0.f;
        }
    }

    static __device__ __forceinline__ void load_q(uint32_t (&f)[4], uint32_t smem, int part, int kk, int lane)
    {
        const uint4 u = lds128(smem + C::OFF_Q + ((uint32_t)(part * C::KSTEPS + kk) * 32 + lane) * 16);
        f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
    }

    // Scores of the slice at stage row r0: c[k][j], slot k of the lane, row j of
    // {2u, 2u+1, 8+2u, 9+2u}, not yet scaled back.
    __device__ __forceinline__ void scores(float (&sc)[C::SPL][4], uint32_t smem, uint32_t ks, int r0, int lane)
    {
        const int g = lane >> 2, u = lane & 3;
        float acc[2][2][4];      // [even and odd k-steps, or hi and lo][rows 0-7, 8-15]
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[e][n][i] = 0.f;
        // the lane's unit of row g of chunk 0 (its units are UPL u + v); row 8 + g lies 8 rows on
        const uint32_t kr = ks + (C::row(r0 + g) ^ (uint32_t)((C::CHB / 64) * u << 4));
        constexpr int UPL = C::CHB / 64;              // 16-byte units of a chunk's row a lane owns
        constexpr int SPU = 4 / C::ES;                // k-steps of a unit
        // unrolled over the chunks only where the Q fragments are registers (their index must be known)
#pragma unroll (C::Q_REGS ? C::NCH : 1)
        for (int c = 0; c < C::NCH; ++c)
#pragma unroll
            for (int v = 0; v < UPL; ++v) {
                uint32_t w[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const uint4 x = lds128(C::unit(kr, c * (C::CHB / 16) + v) + n * 8 * C::CHB);
                    w[n][0] = x.x; w[n][1] = x.y; w[n][2] = x.z; w[n][3] = x.w;
                }
#pragma unroll
                for (int i = 0; i < SPU; ++i) {
                    const int kk = c * C::KPC + v * SPU + i;
                    uint32_t b[2][2];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        if constexpr (C::E8) {
                            e4m3x4_to_half4(w[n][i], b[n][0], b[n][1]);
                        } else {
                            b[n][0] = w[n][2 * i];
                            b[n][1] = w[n][2 * i + 1];
                        }
                    }
                    if constexpr (C::SLOTS == 8) {
                        uint32_t f[4];
                        if constexpr (C::Q_REGS) {
#pragma unroll
                            for (int x = 0; x < 4; ++x) f[x] = qa[kk][x];
                        } else {
                            load_q(f, smem, 0, kk, lane);
                        }
                        mma_16816<MT>(acc[kk & 1][0], f, b[0][0], b[0][1]);
                        mma_16816<MT>(acc[kk & 1][1], f, b[1][0], b[1][1]);
                    } else {
                        uint32_t fh[4], fl[4];
                        load_q(fh, smem, 0, kk, lane);
                        load_q(fl, smem, 1, kk, lane);
                        mma_16816<MT>(acc[0][0], fh, b[0][0], b[0][1]);
                        mma_16816<MT>(acc[1][0], fl, b[0][0], b[0][1]);
                        mma_16816<MT>(acc[0][1], fh, b[1][0], b[1][1]);
                        mma_16816<MT>(acc[1][1], fl, b[1][0], b[1][1]);
                    }
                }
            }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = j >> 1, i = j & 1;
            if constexpr (C::SLOTS == 8) {
                sc[0][j] = (acc[0][n][i] + acc[1][n][i]) + (acc[0][n][2 + i] + acc[1][n][2 + i]);
            } else {
                sc[0][j] = acc[0][n][i] + acc[1][n][i];
                sc[1][j] = acc[0][n][2 + i] + acc[1][n][2 + i];
            }
        }
    }

    // One pair of n-tiles' worth of P.V; `ph`, `pl` are the A operands (8 slots: ph holds both parts).
    __device__ __forceinline__ void mma_pv(float (&acc)[4], const uint32_t (&ph)[4], const uint32_t (&pl)[4],
                                           uint32_t b0, uint32_t b1)
    {
        mma_16816<MT>(acc, ph, b0, b1);
        if constexpr (C::SLOTS == 16) mma_16816<MT>(acc, pl, b0, b1);
    }

    // O += P.V over the slice. EDGE: V rows whose bits in m0 (rows 2u, 2u+1) and m1 (rows 8+2u,
    // 9+2u) are clear are taken as 0.
    template <bool EDGE>
    __device__ __forceinline__ void values(uint32_t vs, int r0, const uint32_t (&ph)[4], const uint32_t (&pl)[4],
                                           uint32_t m0, uint32_t m1, int lane)
    {
        auto step = [&](int n, uint32_t b0, uint32_t b1) {
            if constexpr (EDGE) mma_pv(o[n], ph, pl, b0 & m0, b1 & m1);
            else mma_pv(o[n], ph, pl, b0, b1);
        };
        if constexpr (C::E8) {
            // n-tile n = c * TPC + j holds dimension c * CW + g * TPC + j in column g
            const int g = lane >> 2, u = lane & 3;
            constexpr int TPC = C::CW / 8;            // n-tiles of a chunk: 16, or 8 at head_dim 64
            const uint32_t in = TPC == 16 ? (uint32_t)(g << 4) : (uint32_t)((g >> 1) << 4);
            const uint32_t vr[2] = {vs + (C::row(r0 + 2 * u) ^ in), vs + (C::row(r0 + 2 * u + 1) ^ in)};
            // words of a row a lane holds at once: all of a chunk's, or half (registers)
            constexpr int NW = TPC == 16 && !(C::HD == 256 && C::SLOTS == 16) ? 4 : 2;
#pragma unroll
            for (int c = 0; c < C::NCH; ++c)
#pragma unroll
                for (int h = 0; h < TPC / 4; h += NW) {
                    uint32_t w[4][NW];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint32_t at = C::unit(vr[r & 1], c * 8) + (r >> 1) * 8 * C::CHB;
                        if constexpr (NW == 4) {
                            const uint4 x = lds128(at);
                            w[r][0] = x.x; w[r][1] = x.y; w[r][2] = x.z; w[r][3] = x.w;
                        } else {
                            const uint2 x = lds64(at + (TPC == 16 ? h * 4 : (g & 1) * 8));
                            w[r][0] = x.x; w[r][1] = x.y;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < NW; ++i) {
                        uint32_t a[4], b[4];
                        e4m3x4_to_half4(__byte_perm(w[0][i], w[1][i], 0x5140), a[0], a[1]);
                        e4m3x4_to_half4(__byte_perm(w[0][i], w[1][i], 0x7362), a[2], a[3]);
                        e4m3x4_to_half4(__byte_perm(w[2][i], w[3][i], 0x5140), b[0], b[1]);
                        e4m3x4_to_half4(__byte_perm(w[2][i], w[3][i], 0x7362), b[2], b[3]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) step(c * TPC + (h + i) * 4 + j, a[j], b[j]);
                    }
                }
        } else {
            const int i8 = lane >> 3;
            const uint32_t vr = vs + (C::row(r0 + (i8 & 1) * 8 + (lane & 7)) ^ (uint32_t)((i8 >> 1) << 4));
#pragma unroll
            for (int n = 0; n < C::NTD; n += 2) {
                uint32_t b[4];
                ldsm_x4_trans(b, C::unit(vr, n));
                step(n, b[0], b[1]);
                step(n + 1, b[2], b[3]);
            }
        }
    }

    // o += p v for slice row r alone, v that row of V, by the lanes that have `sees` set (their slot k sees it).
    __device__ __forceinline__ void add_row(uint32_t vs, int r, int k, float p, bool sees, int lane)
    {
        if (!sees) return;
        const int u = lane & 3, at = C::SLOTS == 8 ? 0 : 2 * k;
        if constexpr (C::E8) {
            constexpr int TPC = C::CW / 8;
#pragma unroll
            for (int c = 0; c < C::NCH; ++c)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int h = 0; h < TPC; h += 8) {
                        const int d = (2 * u + e) * TPC + h;       // 8 dimensions from d of the chunk
                        const uint2 x = lds64(vs + (C::row(r) ^ (uint32_t)(d >> 4 << 4)) + c * (C::TILE * 128) + (d & 15));
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t w0, w1;
                            e4m3x4_to_half4(i ? x.y : x.x, w0, w1);
                            const float2 f0 = kv2_to_float2<__half>(w0), f1 = kv2_to_float2<__half>(w1);
                            const int n = c * TPC + h + 4 * i;
                            o[n][at + e] = fmaf(p, f0.x, o[n][at + e]);
                            o[n + 1][at + e] = fmaf(p, f0.y, o[n + 1][at + e]);
                            o[n + 2][at + e] = fmaf(p, f1.x, o[n + 2][at + e]);
                            o[n + 3][at + e] = fmaf(p, f1.y, o[n + 3][at + e]);
                        }
                    }
        } else {
#pragma unroll
            for (int n = 0; n < C::NTD; ++n) {
                uint32_t x;
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(C::unit(vs + C::row(r), n) + 4 * u));
                const float2 f = kv2_to_float2<MT>(x);
                o[n][at] = fmaf(p, f.x, o[n][at]);
                o[n][at + 1] = fmaf(p, f.y, o[n][at + 1]);
            }
        }
    }

    // The slice at stage row r0, cache rows [row0, row0 + 16). edge: some slot of the block does not see all of them.
    __device__ __forceinline__ void process(uint32_t smem, uint32_t ks, uint32_t vs, int r0, int row0,
                                            const SliceInfo &info, bool edge, const SlotRows &sr, int t0, int t1,
                                            const PagedArgs &a, int lane)
    {
        const int u = lane & 3;
        const int col[4] = {2 * u, 2 * u + 1, 8 + 2 * u, 9 + 2 * u};
        float sc[C::SPL][4];
        scores(sc, smem, ks, r0, lane);
        // log2 of the V scale, rounded up: its exponent field
        float lv = 0.f;
        if constexpr (C::E8) {
            const int e = (int)((__float_as_uint(info.vs) >> 23) & 0xFFu) - 126;
            lv = (float)min(max(e, -60), 61);
        }
#pragma unroll
        for (int k = 0; k < C::SPL; ++k) {
            const SlotInfo si = slot(smem, k, lane);
            const float f = C::E8 ? si.inv * info.ks : si.inv;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float x = sc[k][j] * f;
                if constexpr (RULES) {
                    if (a.cap_log2 > 0.f) x = a.cap_log2 * tanhf(x);
                    x = fmaf(si.slope, (float)(row0 + col[j] - sr.last(si.t)), x);
                }
                sc[k][j] = x;
            }
            if (edge) {
                const int last = si.t < 0 ? -1 : sr.last(si.t), low = si.t < 0 ? 0 : sr.low(si.t);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int row = row0 + col[j];
                    if (row > last || row < low) sc[k][j] = -INFINITY;
                }
            }
        }
        bool need[C::SPL];
        float mt[C::SPL];
        bool any = false;
#pragma unroll
        for (int k = 0; k < C::SPL; ++k) {
            float x = fmaxf(fmaxf(sc[k][0], sc[k][1]), fmaxf(sc[k][2], sc[k][3]));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            mt[k] = x + lv;
            need[k] = mt[k] > m[k] + TAU;
            any |= need[k];
        }
        if (__any_sync(0xffffffffu, any)) {
            float corr[2] = {1.f, 1.f};
#pragma unroll
            for (int k = 0; k < C::SPL; ++k) {
                if (need[k]) {
                    corr[k] = ex2(m[k] - mt[k]);       // 0 while m is -inf
                    m[k] = mt[k];
                }
                l[k] *= corr[k];
            }
            if constexpr (C::SLOTS == 8) corr[1] = corr[0];
#pragma unroll
            for (int n = 0; n < C::NTD; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][i] *= corr[i >> 1];
        }
        uint32_t ph[4], pl[4];
        // A row that a slot does not see must not reach it: its weight 0 times what an unwritten or
        // unseen row holds (NaN, infinity) would. Rows that every slot of the block sees go
        // through the MMAs, with the others' V taken as 0; rows that only some query rows see (the last n_q - 1,
        // and as many at a window's start) are added one by one to the slots that see them.
        const bool some = edge && t0 != t1;
#pragma unroll
        for (int k = 0; k < C::SPL; ++k) {
            const float base = m[k] == -INFINITY ? 0.f : m[k] - OFF;     // no row seen yet: every p is 0
            float p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = ex2(sc[k][j] - base);
            l[k] += (p[0] + p[1]) + (p[2] + p[3]);
            if constexpr (C::E8) {
#pragma unroll
                for (int j = 0; j < 4; ++j) p[j] *= info.vs;
            }
            if (some) {
                const int st = slot(smem, k, lane).t;
#pragma unroll 1
                for (int r = 0; r < C::WR; ++r) {
                    const int row = row0 + r;
                    if (row > sr.last(t1) || row < sr.low(t0) || (row <= sr.last(t0) && row >= sr.low(t1))) continue;
                    const float x = r & 8 ? (r & 1 ? p[3] : p[2]) : (r & 1 ? p[1] : p[0]);
                    const float pr = __shfl_sync(0xffffffffu, x, (lane & ~3) | ((r & 7) >> 1));
                    add_row(vs, r0 + r, k, pr, st >= 0 && row <= sr.last(st) && row >= sr.low(st), lane);
                }
            }
            const uint32_t h01 = float2_to_kv2<MT>(p[0], p[1]), h23 = float2_to_kv2<MT>(p[2], p[3]);
            const float2 f01 = kv2_to_float2<MT>(h01), f23 = kv2_to_float2<MT>(h23);
            const uint32_t l01 = float2_to_kv2<MT>(p[0] - f01.x, p[1] - f01.y);
            const uint32_t l23 = float2_to_kv2<MT>(p[2] - f23.x, p[3] - f23.y);
            if constexpr (C::SLOTS == 8) {
                ph[0] = h01; ph[1] = l01; ph[2] = h23; ph[3] = l23;
                pl[0] = pl[1] = pl[2] = pl[3] = 0u;
            } else {
                ph[k] = h01; ph[2 + k] = h23;
                pl[k] = l01; pl[2 + k] = l23;
            }
        }
        if (!edge) {
            values<false>(vs, r0, ph, pl, 0u, 0u, lane);
        } else {
            uint32_t mask[2] = {0u, 0u};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = row0 + col[j];
                if (row <= sr.last(t0) && row >= sr.low(t1)) mask[j >> 1] |= 0xFFFFu << (16 * (j & 1));
            }
            values<true>(vs, r0, ph, pl, mask[0], mask[1], lane);
        }
    }

    // mm[slot] = (reference, sum), mo[slot * MS + d] = accumulator.
    __device__ __forceinline__ void publish(float2 *mm, float *mo, int lane)
    {
        const int g = lane >> 2, u = lane & 3;
#pragma unroll
        for (int k = 0; k < C::SPL; ++k) {
            float lt = l[k];
            lt += __shfl_xor_sync(0xffffffffu, lt, 1);
            lt += __shfl_xor_sync(0xffffffffu, lt, 2);
            const int i = g + 8 * k;
            if (u == 0) mm[i] = make_float2(m[k] - OFF, lt);
            auto val = [&](int n, int e) {
                return C::SLOTS == 8 ? o[n][e] + o[n][2 + e] : o[n][2 * k + e];
            };
            if constexpr (C::E8) {
                constexpr int TPC = C::CW / 8;
#pragma unroll
                for (int c = 0; c < C::NCH; ++c)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int j = 0; j < TPC; j += 4) {
                            const int n = c * TPC + j;
                            *reinterpret_cast<float4 *>(mo + i * C::MS + c * C::CW + (2 * u + e) * TPC + j) =
                                make_float4(val(n, e), val(n + 1, e), val(n + 2, e), val(n + 3, e));
                        }
            } else {
#pragma unroll
                for (int n = 0; n < C::NTD; ++n)
                    *reinterpret_cast<float2 *>(mo + i * C::MS + n * 8 + 2 * u) = make_float2(val(n, 0), val(n, 1));
            }
        }
    }
};

// Q of the block's slots as MMA A fragments in shared memory: hi = T(q sc), lo = T(q sc - hi) with a
// power of two sc per slot (exact). Slots past the last are zero.
template <class C>
__device__ __forceinline__ void paged_prepare_q(uint8_t *smem, const PagedArgs &a, int s, int hk, int qg, int tid)
{
    using MT = typename C::MT;
    const int warp = tid >> 5, lane = tid & 31;
    constexpr int NW = C::NWC;                                   // the compute warps
    constexpr int V4 = C::HD <= 128 ? 1 : 2;                     // float4 of a row a lane owns
    constexpr int ITER = C::SLOTS / NW;
    const bool active = lane * 4 < C::HD;
    float4 x[ITER][V4];
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
        const int i = warp + it * NW, qh = qg * C::SLOTS + i;
        const bool have = qh < a.n_q * a.group;
        const int t = have ? qh / a.group : 0, g = have ? qh - t * a.group : 0;
        const float *row = a.q + (((size_t)s * a.n_q + t) * a.n_head + (size_t)hk * a.group + g) * C::HD;
#pragma unroll
        for (int v = 0; v < V4; ++v) {
            x[it][v] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (have && active) x[it][v] = ld_dep(reinterpret_cast<const float4 *>(row + v * 128) + lane);
        }
    }
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
        const int i = warp + it * NW;
        float amax = 0.f;
#pragma unroll
        for (int v = 0; v < V4; ++v) {
            x[it][v].x *= a.qscale; x[it][v].y *= a.qscale; x[it][v].z *= a.qscale; x[it][v].w *= a.qscale;
            amax = fmaxf(amax, fmaxf(fmaxf(fabsf(x[it][v].x), fabsf(x[it][v].y)),
                                     fmaxf(fabsf(x[it][v].z), fabsf(x[it][v].w))));
        }
        amax = warp_max(amax);
        float sc, inv;
        pow2_scale(amax, sc, inv);
        if (lane == 0) {
            const int qh = qg * C::SLOTS + i;
            SlotInfo si;
            si.inv = inv;
            si.t = qh < a.n_q * a.group ? qh / a.group : -1;
            si.slope = a.slopes && si.t >= 0 ? ld_dep(a.slopes + hk * a.group + qh % a.group) * kLog2e : 0.f;
            si.pad = 0;
            reinterpret_cast<SlotInfo *>(smem + C::OFF_SLOT)[i] = si;
        }
        if (!active) continue;
#pragma unroll
        for (int v = 0; v < V4; ++v) {
            const int d = v * 128 + lane * 4;
            const float f[4] = {x[it][v].x * sc, x[it][v].y * sc, x[it][v].z * sc, x[it][v].w * sc};
            uint32_t hw[2], lw[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                hw[j] = float2_to_kv2<MT>(f[2 * j], f[2 * j + 1]);
                const float2 b = kv2_to_float2<MT>(hw[j]);
                lw[j] = float2_to_kv2<MT>(f[2 * j] - b.x, f[2 * j + 1] - b.y);
            }
            // dimension d is element 0 of a lane's four in k-step kk (the K loads' order)
            const int c = d / C::CW, in = d % C::CW, u = in / (C::CW / 4), w = in % (C::CW / 4) / 4;
            const int kk = c * C::KPC + w, fl = (i & 7) * 4 + u;
            uint32_t *hi, *lo;
            if constexpr (C::SLOTS == 8) {
                uint32_t *p = reinterpret_cast<uint32_t *>(smem + C::OFF_Q) + (kk * 32 + fl) * 4;
                hi = p;
                lo = p + 1;
            } else {
                hi = reinterpret_cast<uint32_t *>(smem + C::OFF_Q) + (kk * 32 + fl) * 4 + (i >> 3);
                lo = hi + C::KSTEPS * 128;
            }
            hi[0] = hw[0]; hi[2] = hw[1];
            lo[0] = lw[0]; lo[2] = lw[1];
        }
    }
}

template <class C, bool RULES>
__global__ void __launch_bounds__(C::THREADS, C::MIN_BLOCKS)
attn_paged_partial(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                   const PagedArgs a)
{
    constexpr int NWC = C::NWC, S = C::S, TILE = C::TILE, WR = C::WR, NSL = C::NSL;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    SliceInfo *info = reinterpret_cast<SliceInfo *>(smem + C::OFF_INFO);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *empty = full + S;
    volatile int *flags = reinterpret_cast<volatile int *>(empty + S);   // [0] abort, [1] tiles issued

    const int sp = blockIdx.y, s = blockIdx.z;
    const int hk = blockIdx.x / a.qgroups, qg = blockIdx.x % a.qgroups;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int P = a.n_splits;
    const size_t heads = (size_t)a.n_q * a.n_head;

    if (tid == NWC * 32) {
        for (int i = 0; i < S; ++i) {
            mbar_init(full + i, 2);          // the copies' issue, and the slices' info
            mbar_init(empty + i, NWC);
        }
        flags[0] = 0;
        flags[1] = 0;
        fence_barrier_init();
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    pdl_wait();
    pdl_launch_dependents();

    // The rows of this block's query rows [t0, t1], and its split of them
    SlotRows sr;
    {
        const int64_t n = (int64_t)ld_dep(a.positions + s) + 1;
        const bool ok = n >= 0 && n <= a.cap;
        if (!ok && sp == 0 && blockIdx.x == 0 && tid == 0) atomicOr(a.err, kErrPositionClamped);
        sr.nkv = ok ? (int)n : n < 0 ? 0 : a.cap;
        sr.base = sr.nkv - a.n_q;
        sr.start = a.starts ? ld_dep(a.starts + s) : 0;
        sr.window = a.window;
    }
    const int x1 = min((qg + 1) * C::SLOTS, a.n_q * a.group) - 1;
    const int t0 = qg * C::SLOTS / a.group, t1 = x1 / a.group;
    const int R = max(sr.last(t1) + 1, 0), L = min(sr.low(t0), R);       // rows [L, R): seen by some slot
    const int L0 = L / TILE * TILE;
    int chunk = (R - L0 + P - 1) / P;
    chunk = (chunk + TILE - 1) / TILE * TILE;
    const int64_t lo64 = (int64_t)L0 + (int64_t)sp * chunk;
    const int lo = lo64 < R ? (int)lo64 : R;
    const int hi = chunk < R - lo ? lo + chunk : R;
    if (lo >= hi || L >= R) {                                            // nothing in this split
        for (int i = tid; i < C::SLOTS; i += C::THREADS) {
            const int x = qg * C::SLOTS + i;
            if (x >= a.n_q * a.group) break;
            const int t = x / a.group;
            const size_t row = (size_t)s * heads + (size_t)t * a.n_head + hk * a.group + (x - t * a.group);
            if (P > 1) a.ws_ml[row * P + sp] = make_float2(-INFINITY, 0.f);
            else
                for (int d = 0; d < C::HD; d += 4)
                    *reinterpret_cast<float4 *>(a.out + row * C::HD + d) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        return;
    }
    const int ntiles = (hi - lo + TILE - 1) / TILE;

    if (warp != NWC) paged_prepare_q<C>(smem, a, s, hk, qg, tid);

    if (warp == NWC) {
        // ---------------- producer warp ----------------
        // Lane i keeps the page and the scales of slice i of a group of 8 tiles (32 slices); the next
        // group's entries are loaded while this one's tiles go out.
        const int32_t *table = a.table + (size_t)s * a.max_pages;
        auto load_page = [&](int grp) {
            const int64_t row = (int64_t)lo + ((int64_t)grp * 32 + lane) * WR;
            int p = -1;
            if (row < hi && row + WR > L) {
                p = ld_dep(table + (int)row / a.page_size);
                if (p < 0 || p >= a.n_pages) {
                    atomicOr(a.err, kErrBadPage);
                    p = -1;
                }
            }
            return p;
        };
        auto load_scales = [&](int p) {
            float2 f = make_float2(1.f, 1.f);
            if constexpr (C::E8) {
                if (p >= 0) {
                    f.x = ld_dep(a.k_scale + (size_t)p * a.n_kv_head + hk);
                    f.y = ld_dep(a.v_scale + (size_t)p * a.n_kv_head + hk);
                }
            }
            return f;
        };
        const int BR = a.box_rows, nbox = TILE / BR, bsl = BR / WR;
        auto issue = [&](int t, int st, int page) {        // `page`: lane i's of the tile's group
            const int row0 = lo + t * TILE;
            unsigned bytes = 0;
            for (int b = 0; b < nbox; ++b) {
                const int first = row0 + b * BR;
                // the box's page is that of any of its slices that holds a row in range
                int p = -1;
                for (int i = 0; i < bsl; ++i) p = max(p, __shfl_sync(0xffffffffu, page, (t & 7) * NSL + b * bsl + i));
                if (p >= 0 && first < hi) bytes += 2u * (unsigned)BR * C::ROWB;
            }
            if (lane == 0) mbar_arrive_expect_tx(full + st, bytes);
            __syncwarp();
            uint8_t *kst = smem + st * C::STAGE_BYTES;
            uint8_t *vst = kst + C::TILE_BYTES;
            for (int b = 0; b < nbox; ++b) {
                const int first = row0 + b * BR;
                int p = -1;
                for (int i = 0; i < bsl; ++i) p = max(p, __shfl_sync(0xffffffffu, page, (t & 7) * NSL + b * bsl + i));
                if (p >= 0 && first < hi && lane == 0) {
                    const int z = first % a.page_size;
#pragma unroll
                    for (int c = 0; c < C::NCH; ++c) {
                        const uint32_t off = c * (C::TILE_BYTES / C::NCH) + b * BR * C::CHB;
                        tma_load_4d(kst + off, &kmap, full + st, c * C::CW, hk, z, p);
                        tma_load_4d(vst + off, &vmap, full + st, c * C::CW, hk, z, p);
                    }
                }
            }
            if (lane == 0) flags[1] = t + 1;
        };
        auto inform = [&](int t, int st, int page, float2 sc) {
            const int i = lane - (t & 7) * NSL;
            if (i >= 0 && i < NSL) {
                SliceInfo f;
                f.page = page;
                f.ks = sc.x;
                f.vs = sc.y;
                f.pad = 0;
                info[st * NSL + i] = f;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(full + st);
        };
        int page = load_page(0), next = -1;
        const int early = min(min(S, 8), ntiles);
        for (int t = 0; t < early; ++t) issue(t, t, page);
        float2 sc = load_scales(page), nsc = make_float2(1.f, 1.f);
        for (int t = 0; t < early; ++t) inform(t, t, page, sc);
        next = load_page(1);
        nsc = load_scales(next);
        __syncthreads();
        for (int t = early; t < ntiles; ++t) {
            const int st = t % S;
            int ok = 1;
            if (lane == 0) {
                if (t >= S && !mbar_wait_bounded(empty + st, ((t / S) - 1) & 1)) {
                    flags[0] = 1;
                    atomicOr(a.err, kErrPipelineTimeout);
                }
                ok = !flags[0];
            }
            if (!__shfl_sync(0xffffffffu, ok, 0)) break;
            if ((t & 7) == 0) {
                page = next;
                sc = nsc;
            }
            issue(t, st, page);
            inform(t, st, page, sc);
            if ((t & 7) == 1) next = load_page((t >> 3) + 1);
            if ((t & 7) == 5) nsc = load_scales(next);
        }
    } else {
        // ---------------- compute warps ----------------
        __syncthreads();
        PagedWarp<C, RULES> w;
        const uint32_t smem_u = smem_u32(smem);
        w.init(smem_u, lane);
        const int seen_lo = sr.low(t1), seen_hi = sr.last(t0);           // rows every slot sees
#pragma unroll 1
        for (int t = 0; t < ntiles; ++t) {
            const int st = t % S;
            const bool landed = mbar_wait_bounded(full + st, (t / S) & 1);
            if (!__all_sync(0xffffffffu, landed)) {
                if (lane == 0) { flags[0] = 1; atomicOr(a.err, kErrPipelineTimeout); }
                break;
            }
            if (__shfl_sync(0xffffffffu, flags[0], 0)) break;
            const int row0 = lo + t * TILE + warp * WR;
            const SliceInfo f = info[st * NSL + warp];
            if (f.page >= 0 && row0 < hi) {
                const uint32_t kst = smem_u + st * C::STAGE_BYTES;
                const bool edge = row0 < seen_lo || row0 + WR - 1 > seen_hi;
                w.process(smem_u, kst, kst + C::TILE_BYTES, warp * WR, row0, f, edge, sr, t0, t1, a, lane);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + st);
        }
        // the merge area lies over the ring: every compute warp is done with it first
        asm volatile("bar.sync 1, %0;" :: "r"(NWC * 32) : "memory");
        if (!__shfl_sync(0xffffffffu, flags[0], 0))
            w.publish(reinterpret_cast<float2 *>(smem) + warp * C::SLOTS,
                      reinterpret_cast<float *>(smem) + C::OFF_MO + warp * C::SLOTS * C::MS, lane);
    }
    __syncthreads();

    // No copy may still be writing shared memory when the block exits; without an
    // abort every issued tile has been waited for.
    if (flags[0]) {
        if (tid == NWC * 32) {
            const int issued = flags[1];
            for (int t = issued - S > 0 ? issued - S : 0; t < issued; ++t)
                (void)mbar_wait_bounded(full + (t % S), (t / S) & 1);
        }
        return;
    }

    // Merge the warps' states; one split: the result itself
    const float2 *mm = reinterpret_cast<const float2 *>(smem);
    const float *mo = reinterpret_cast<const float *>(smem) + C::OFF_MO;
    constexpr int D4 = C::HD / 4;
    for (int i = tid; i < C::SLOTS * D4; i += C::THREADS) {
        const int g = i / D4, d = (i % D4) * 4;
        const int x = qg * C::SLOTS + g;
        if (x >= a.n_q * a.group) break;
        float2 ml[NWC];
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < NWC; ++w) {
            ml[w] = mm[w * C::SLOTS + g];
            M = fmaxf(M, ml[w].x);
        }
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < NWC; ++w) {
            const float wt = ml[w].x == -INFINITY ? 0.f : ex2(ml[w].x - M);
            const float4 v = *reinterpret_cast<const float4 *>(mo + (w * C::SLOTS + g) * C::MS + d);
            O.x = fmaf(wt, v.x, O.x);
            O.y = fmaf(wt, v.y, O.y);
            O.z = fmaf(wt, v.z, O.z);
            O.w = fmaf(wt, v.w, O.w);
            sum = fmaf(wt, ml[w].y, sum);
        }
        const int t = x / a.group;
        const size_t row = (size_t)s * heads + (size_t)t * a.n_head + hk * a.group + (x - t * a.group);
        if (P > 1) {
            *reinterpret_cast<float4 *>(a.ws_o + (row * P + sp) * C::HD + d) = O;
            if (d == 0) a.ws_ml[row * P + sp] = make_float2(M, sum);
        } else {
            if (sum == 0.f) O = make_float4(0.f, 0.f, 0.f, 0.f);
            else { O.x /= sum; O.y /= sum; O.z /= sum; O.w /= sum; }
            *reinterpret_cast<float4 *>(a.out + row * C::HD + d) = O;
        }
    }
}

} // namespace attn
