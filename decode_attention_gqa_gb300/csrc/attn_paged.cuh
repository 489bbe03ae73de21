// attn_paged.cuh -- decode attention over a paged cache: the streaming kernel and
// the merge of the parts it leaves.
//
// Mathematics. For a (query row, head) slot at position x over the cache rows j it sees,
//     s_j = rules(scale q.k_j),  o = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j log2 e - m),
// one pass with a running reference m that moves when a score passes it by 8. An e4m3
// cache holds codes with one scale per page and KV head: q.k_j is the product with the
// codes times the page's K scale, one multiplication a score, and the V scale multiplies
// p before P.V. The reference follows s + log2 of the V scale (rounded up), so that p
// times the scale stays in the 16-bit range whatever the scales are; sum p is f32.
//
// Work. The tiles (TILE rows) of all sequences that any query row sees are laid end to
// end on the device, and as many blocks as fill the GPU once ("ranks", per KV head and
// group of 8 or 16 slots) take equal runs of them, the turn to the next sequence counted
// as the few tiles whose time it takes (21.4 us against 22.9 for the draft rows below). A
// block goes through its run without a pause for the copies: at the end of a sequence its
// warps' states are merged, and written as the output where the whole sequence was the
// block's, else as a part (reference, sum, sum p v) that attn_paged_combine joins with
// the others'. A grid of (split, sequence) blocks left the tail of a ragged batch to a few
// of them: 32 sequences of 1 .. 32768 rows took 270 us that way and take 159 this way, 1.00
// of the copy bandwidth.
//
// Layout. NWC compute warps and a producer warp over a ring of S stages of one tile. A
// 16-row slice of a tile belongs to one warp and lies in one page; the producer looks the
// pages up two groups of 32 slices ahead, loads each page's piece by TMA (boxes of up to
// 64 rows of the page, swizzled, first to leave L2) and leaves page and scales beside the
// stage. Slices that nothing sees are neither loaded nor waited for.
//
// Tensor cores. 16x8x16 MMAs, f32 accumulation; q and p as two f16 parts (an f16
// or e4m3 cache; f16 holds the codes exactly) or three bf16 parts, so that
// neither loses what 32 bits hold. S = Q K^T: with 8 slots two parts lie over each
// other in the 16 MMA rows, with 16 slots each part has its own MMA. O^T = V^T P^T: the
// parts of p add up in one accumulator, 4 registers for 16 dimensions x 8 slots,
// and P is used in the registers where S was accumulated. The order of a dot
// product's terms is free, so a lane's share of a K row is contiguous: 16-byte shared
// loads give it whole k-steps, with no ldmatrix and, for 8 bits, no shuffling before the
// conversion. 8-bit V needs pairs of rows in a register: a lane reads its four rows' 16
// contiguous dimensions and pairs bytes of two rows before converting.
//
// What bounds it. HBM where there are many rows (ragged batch above; 48 sequences of
// 129 .. 4097 rows with a distance bias 57 us, 0.88 of the copy bandwidth; 131072 rows of
// 8 KV heads 47 us, 0.84: 5 to 7 us of the last two are the chain before the first tile
// -- positions, table, page --, the merges, the joining kernel and uneven ends). Latency
// where there are few: one sequence of 512 rows 6.2 us, 8192 rows of 4 KV heads 8.3; 4
// draft rows of 4 sequences of up to 8400 rows, 32 slots of 256 dimensions a KV head, 19.5
// us: the accumulators leave room for eight warps an SM, which keep the tensor pipe
// half busy.
#pragma once

#include <cuda_fp8.h>

#include "attn_device.cuh"
#include "attn_paged_launch.h"

namespace attn {

struct E4m3 {};       // tag of the 8-bit cache

template <typename KV> struct PagedMma { using T = KV; };
template <> struct PagedMma<E4m3> { using T = __half; };

constexpr unsigned kErrBadPage = 0x4u;    // ATTN_DEVERR_BAD_PAGE

// A TMA box whose lines L2 gives up first: a cache is read once a step, and what else the step works on (block
// table, scales, q, the next layers' weights) should not make room for it (a batch of 339 MB 62.3 -> 59.7
// us a call, since its small reads then hit L2).
__device__ __forceinline__ void tma_load_4d_once(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z,
                                                 int w, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;"
        :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w),
           "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

// Four e4m3 codes to four f16 values, exact.
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

template <int HD_, int SLOTS_, typename KV_>
struct PagedCfg {
    static constexpr int HD = HD_, SLOTS = SLOTS_;
    using KV = KV_;
    using MT = typename PagedMma<KV>::T;
    static constexpr bool E8 = std::is_same<KV, E4m3>::value;
    static constexpr int ES = E8 ? 1 : 2;
    static constexpr PagedShape SHAPE = paged_shape(HD, ES, SLOTS);
    static constexpr int S = SHAPE.stages, MIN_BLOCKS = SHAPE.blocks;
    static constexpr int NWC = SHAPE.warps, WR = 16, NSL = SHAPE.nsl, TILE = NSL * WR;
    static constexpr int WPT = NWC / NSL;                         // stages the warps work on at a time
    static constexpr int THREADS = (NWC + 1) * 32;
    static constexpr int TPG = 32 / NSL;                          // tiles of a descriptor group
    static constexpr int ROWB = HD * ES;                          // bytes of a row of one head
    static constexpr int CHB = ROWB < 128 ? ROWB : 128;           // bytes of a swizzled chunk's row
    static constexpr int NCH = ROWB / CHB;
    static constexpr int CW = CHB / ES;                           // dimensions of a chunk
    static constexpr uint32_t TILE_BYTES = (uint32_t)TILE * ROWB;
    static constexpr uint32_t STAGE_BYTES = 2 * TILE_BYTES;
    static constexpr int KSTEPS = HD / 16;
    static constexpr int KPC = CW / 16;                           // k-steps of a chunk
    static constexpr int SPL = SLOTS / 8;                         // slots a lane owns
    // 16-bit parts that carry q and p: two f16 (22 bits), three bf16 (24; two would keep 16)
    static constexpr int NP = std::is_same<MT, __nv_bfloat16>::value ? 3 : 2;
    // Q operands: 8 slots: parts in pairs, one over the other in the 16 rows (a third part alone: half
    // an operand); 16 slots: a part each
    static constexpr int PARTS = SLOTS == 8 ? (NP + 1) / 2 : NP;
    static constexpr bool Q_REGS = E8 && HD == 64 && SLOTS == 8;   // else they are read per k-step (no spills)
    static constexpr uint32_t Q_BYTES = (uint32_t)(SLOTS == 8 ? NP : 2 * NP) * KSTEPS * 256;
    // Row stride of the merge area: 4 floats past a multiple of 32, so that the rows of a warp's slots (2u) lie 8
    // banks apart
    static constexpr int MS = HD + 4;
    // Merge area (floats): the warps' (reference, sum) per slot, their merge, the accumulator rows
    static constexpr uint32_t OFF_RES = 2 * NWC * SLOTS, OFF_MO = OFF_RES + 2 * SLOTS;
    static constexpr int NPART = HD / 32;                         // 32-dimension parts of a row
    // q of the next sequence is loaded before the merge, where the registers are enough
    static constexpr bool Q_EARLY = !(SLOTS == 16 && (HD == 256 || (HD == 64 && !E8)));
    static constexpr uint32_t MERGE_BYTES = (OFF_MO + SLOTS * MS) * 4;
    static constexpr uint32_t OFF_Q = S * STAGE_BYTES;            // Q fragments; then the merge area
    static constexpr uint32_t OFF_SLOT = OFF_Q + (Q_BYTES > MERGE_BYTES ? Q_BYTES : MERGE_BYTES);
    static constexpr uint32_t OFF_SEG = OFF_SLOT + SLOTS * 16;    // SegInfo
    static constexpr uint32_t OFF_DESC = OFF_SEG + 48;            // SliceInfo[4][32]
    static constexpr uint32_t OFF_BAR = OFF_DESC + 4 * 32 * 16;
    static constexpr uint32_t OFF_SEQ = OFF_BAR + 2 * S * 8 + 16;
    static constexpr uint32_t SMEM_BYTES = OFF_SEQ + 16 + (3 * kPagedSeqs + 1) * 4 + kPagedSeqs;
    static_assert(NWC % NSL == 0 && S <= TPG, "descriptor buffers outlive the stages in flight");
    // a warp waits for the phases of its own stages only: if a stage changed hands, a warp could take the
    // parity of an older phase for its own
    static_assert(S % WPT == 0, "a stage belongs to the same warps throughout");
    static_assert((size_t)NWC * SLOTS * MS * 4 <= S * STAGE_BYTES, "the last merge lies over the ring");
    static_assert(SMEM_BYTES <= 227 * 1024 && MIN_BLOCKS * (SMEM_BYTES + 1024u) <= 233472u, "shared memory");
    static_assert((TILE_BYTES / NCH) % 1024 == 0 && OFF_MO % 4 == 0, "alignment");

    // Rows are stored as chunks of CHB bytes, swizzled as TMA writes them. `row` is the offset of a row
    // with its swizzle bits set; `unit` adds 16-byte unit U: one exclusive or with a constant
    // (the base is 1024-aligned), so no address has to be kept in a register.
    static __device__ __forceinline__ uint32_t row(int r)
    {
        return CHB == 128 ? (uint32_t)(r * 128 + ((r & 7) << 4)) : (uint32_t)(r * 64 + (((r >> 1) & 3) << 4));
    }
    // A row of the merge area holds 32-dimension parts; in a part, the fours of lanes g = 0..7 (two tiles of
    // accumulators) stand next to each other, so that they are written without bank conflicts. Reads
    // dimensions d .. d + 3: 8 bits, where a lane holds neighbours, one of the fours; 16 bits, where it holds
    // every eighth, an element of four of them.
    static __device__ __forceinline__ float4 merge_read(const float *row, int d)
    {
        if constexpr (E8) {
            constexpr int LD = CW / 8;                            // dimensions of a lane in a chunk
            return *reinterpret_cast<const float4 *>(row + d / CW * CW + (d % LD / 4 * 8 + d % CW / LD) * 4);
        } else {
            const float *p = row + d / 32 * 32 + d % 8 * 4 + d % 32 / 8;
            return make_float4(p[0], p[4], p[8], p[12]);
        }
    }
    static __device__ __forceinline__ uint32_t unit(uint32_t base_row, int U)
    {
        return CHB == 128 ? (base_row ^ (uint32_t)((U & 7) << 4)) + (uint32_t)(U >> 3) * (TILE * 128)
                          : base_row ^ (uint32_t)(U << 4);
    }
};

struct __align__(16) SliceInfo {  // of one 16-row slice
    int page;             // -1: not there, or nothing the stage needs
    int z;                // its first row in the page
    float ks, vs;
};

struct __align__(16) SlotInfo {   // of one (query row, head) slot of the block, for the sequence at hand
    float inv;            // undoes the power of two q was scaled by
    float slope;          // times log2 e
    int last, low;        // the rows it sees; no such slot: -1, 0
};

struct __align__(16) SegInfo {    // the sequence at hand
    int seen_lo, seen_hi; // rows every slot of the block sees
    int any_lo, any_hi;   // rows some slot sees
    int row0, tile0;      // first row of its first tile; that tile, counted from the block's first
    int seq, from, to;    // the sequence, and its tiles of this block
};
static_assert(sizeof(SegInfo) <= 48, "its place in shared memory");

// The rows the slots of query rows [t0, t1] see, as [first row of t0, last row of t1]
struct SlotRows {
    int base;             // row t's position is base + t
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
    float o[C::SPL][C::HD / 16][4];    // Oᵀ: 16 dimensions x 8 slots a tile
    float m[C::SPL], l[C::SPL];

    static __device__ __forceinline__ SlotInfo slot_at(uint32_t smem, int i)
    {
        const uint4 u = lds128(smem + C::OFF_SLOT + i * 16);
        return SlotInfo{__uint_as_float(u.x), __uint_as_float(u.y), (int)u.z, (int)u.w};
    }
    static __device__ __forceinline__ int4 seg_rows(uint32_t smem)        // seen_lo, seen_hi, any_lo, any_hi
    {
        const uint4 u = lds128(smem + C::OFF_SEG);
        return make_int4((int)u.x, (int)u.y, (int)u.z, (int)u.w);
    }

    __device__ __forceinline__ void init(uint32_t smem, int lane)
    {
        if constexpr (C::Q_REGS) {
#pragma unroll
            for (int kk = 0; kk < C::KSTEPS; ++kk) load_q(qa[kk], smem, 0, kk, lane);
        }
#pragma unroll
        for (int k = 0; k < C::SPL; ++k) {
#pragma unroll
            for (int n = 0; n < C::HD / 16; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[k][n][i] = 0.f;
            m[k] = -INFINITY;
            l[k] = 0.f;
        }
    }

    static __device__ __forceinline__ void load_q(uint32_t (&f)[4], uint32_t smem, int part, int kk, int lane)
    {
        if (C::SLOTS == 8 && C::NP == 3 && part == 1) {        // rows 8-15 have no part
            const uint2 u = lds64(smem + C::OFF_Q + C::KSTEPS * 512 + (uint32_t)(kk * 32 + lane) * 8);
            f[0] = u.x; f[2] = u.y;
            f[1] = f[3] = 0u;
        } else {
            const uint4 u = lds128(smem + C::OFF_Q + ((uint32_t)(part * C::KSTEPS + kk) * 32 + lane) * 16);
            f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
        }
    }

    // Scores of the slice at stage row r0: c[k][j], slot k of the lane, row j of
    // {2u, 2u+1, 8+2u, 9+2u}, not yet scaled back.
    __device__ __forceinline__ void scores(float (&sc)[C::SPL][4], uint32_t smem, uint32_t ks, int r0, int lane)
    {
        const int g = lane >> 2, u = lane & 3;
        float acc[2][2][4];      // [two chains][rows 0-7, 8-15]
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
#pragma unroll
                    for (int part = 0; part < C::PARTS; ++part) {
                        uint32_t f[4];
                        if constexpr (C::Q_REGS) {
#pragma unroll
                            for (int x = 0; x < 4; ++x) f[x] = qa[kk][x];
                        } else {
                            load_q(f, smem, part, kk, lane);
                        }
                        const int e = C::PARTS == 1 ? kk & 1 : part & 1;
                        mma_16816<MT>(acc[e][0], f, b[0][0], b[0][1]);
                        mma_16816<MT>(acc[e][1], f, b[1][0], b[1][1]);
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

    // Oᵀ += Vᵀ Pᵀ over the slice, V's 16 dimensions x 16 rows as the A operand, so that all parts of p add
    // up in the same accumulators. P's B fragments (slot g, rows 2u, 2u+1 and 8+2u, 9+2u) are where the
    // scores' accumulators left them. EDGE: V rows whose bits in m0 (rows 2u, 2u+1) and m1 (rows 8+2u,
    // 9+2u) are clear are taken as 0.
    template <bool EDGE>
    __device__ __forceinline__ void values(uint32_t vs, int r0, const uint32_t (&pb)[C::SPL][C::NP][2], uint32_t m0,
                                           uint32_t m1, int lane)
    {
        auto step = [&](int n, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
            uint32_t f[4] = {a0, a1, a2, a3};
            if constexpr (EDGE) {
                f[0] &= m0; f[1] &= m0; f[2] &= m1; f[3] &= m1;
            }
#pragma unroll
            for (int x = 0; x < C::NP; ++x)
#pragma unroll
                for (int k = 0; k < C::SPL; ++k) mma_16816<MT>(o[k][n], f, pb[k][x][0], pb[k][x][1]);
        };
        if constexpr (C::E8) {
            // tile n = c * TPC + j holds dimensions c * CW + g * 2 TPC + 2 j and the next in rows g and g + 8
            const int g = lane >> 2, u = lane & 3;
            constexpr int TPC = C::CW / 16;           // tiles of a chunk: 8, or 4 at head_dim 64
            const uint32_t in = TPC == 8 ? (uint32_t)(g << 4) : (uint32_t)((g >> 1) << 4);
            const uint32_t vr[2] = {vs + (C::row(r0 + 2 * u) ^ in), vs + (C::row(r0 + 2 * u + 1) ^ in)};
            // words of a row a lane holds at once: all of a chunk's, or half (registers)
            constexpr int NW = TPC == 8 && C::SLOTS == 8 ? 4 : 2;
#pragma unroll
            for (int c = 0; c < C::NCH; ++c)
#pragma unroll
                for (int h = 0; h < TPC / 2; h += NW) {
                    uint32_t w[4][NW];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const uint32_t at = C::unit(vr[r & 1], c * 8) + (r >> 1) * 8 * C::CHB;
                        if constexpr (NW == 4) {
                            const uint4 x = lds128(at);
                            w[r][0] = x.x; w[r][1] = x.y; w[r][2] = x.z; w[r][3] = x.w;
                        } else {
                            const uint2 x = lds64(at + (TPC == 8 ? h * 4 : (g & 1) * 8));
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
                        step(c * TPC + (h + i) * 2, a[0], a[1], b[0], b[1]);
                        step(c * TPC + (h + i) * 2 + 1, a[2], a[3], b[2], b[3]);
                    }
                }
        } else {
            // tile n holds dimensions 16 n + g and 16 n + 8 + g in rows g and g + 8
            const int i8 = lane >> 3;
            const uint32_t vr = vs + (C::row(r0 + (i8 & 1) * 8 + (lane & 7)) ^ (uint32_t)((i8 >> 1) << 4));
#pragma unroll
            for (int n = 0; n < C::HD / 16; ++n) {
                uint32_t b[4];
                ldsm_x4_trans(b, C::unit(vr, 2 * n));
                step(n, b[0], b[2], b[1], b[3]);
            }
        }
    }

    // o += p v for stage row r alone: p0, p1 of the lane's accumulators' slots 2u and 2u+1 (+ 8 k), each
    // only where that slot sees the row.
    __device__ __forceinline__ void add_row(uint32_t vs, int r, int k, float p0, float p1, bool s0, bool s1, int lane)
    {
        const int g = lane >> 2;
        auto add = [&](int n, float v0, float v1) {
            if (s0) {
                o[k][n][0] = fmaf(p0, v0, o[k][n][0]);
                o[k][n][2] = fmaf(p0, v1, o[k][n][2]);
            }
            if (s1) {
                o[k][n][1] = fmaf(p1, v0, o[k][n][1]);
                o[k][n][3] = fmaf(p1, v1, o[k][n][3]);
            }
        };
        if constexpr (C::E8) {
            constexpr int TPC = C::CW / 16;
#pragma unroll
            for (int c = 0; c < C::NCH; ++c)
#pragma unroll
                for (int h = 0; h < TPC; h += 4) {
                    const int d = g * 2 * TPC + 2 * h;                 // 8 dimensions from d of the chunk
                    const uint2 x = lds64(vs + (C::row(r) ^ (uint32_t)(d >> 4 << 4)) + c * (C::TILE * 128) + (d & 15));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t w0, w1;
                        e4m3x4_to_half4(i ? x.y : x.x, w0, w1);
                        const float2 f0 = kv2_to_float2<__half>(w0), f1 = kv2_to_float2<__half>(w1);
                        add(c * TPC + h + 2 * i, f0.x, f0.y);
                        add(c * TPC + h + 2 * i + 1, f1.x, f1.y);
                    }
                }
        } else {
#pragma unroll
            for (int n = 0; n < C::HD / 16; ++n) {
                uint16_t x0, x1;
                const uint32_t at = vs + C::row(r);
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x0) : "r"(C::unit(at, 2 * n) + 2 * g));
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x1) : "r"(C::unit(at, 2 * n + 1) + 2 * g));
                const float2 f = kv2_to_float2<MT>((uint32_t)x0 | (uint32_t)x1 << 16);
                add(n, f.x, f.y);
            }
        }
    }

    // The slice at stage row r0, cache rows [row0, row0 + 16). edge: some slot of the block does not see all of them.
    __device__ __forceinline__ void process(uint32_t smem, uint32_t ks, int r0, int row0, float kscale, float vscale,
                                            bool edge, float cap_log2, int lane)
    {
        const uint32_t vs = ks + C::TILE_BYTES;
        const int u = lane & 3;
        const int col[4] = {2 * u, 2 * u + 1, 8 + 2 * u, 9 + 2 * u};
        float sc[C::SPL][4];
        scores(sc, smem, ks, r0, lane);
        // log2 of the V scale, rounded up: its exponent field
        float lv = 0.f;
        if constexpr (C::E8) {
            const int e = (int)((__float_as_uint(vscale) >> 23) & 0xFFu) - 126;
            lv = (float)min(max(e, -60), 61);
        }
#pragma unroll
        for (int k = 0; k < C::SPL; ++k) {
            const SlotInfo si = slot_at(smem, (lane >> 2) + 8 * k);
            const float f = C::E8 ? si.inv * kscale : si.inv;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float x = sc[k][j] * f;
                if constexpr (RULES) {
                    if (cap_log2 > 0.f) x = cap_log2 * tanhf(x);
                    x = fmaf(si.slope, (float)(row0 + col[j] - si.last), x);
                }
                sc[k][j] = x;
            }
            if (edge) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int row = row0 + col[j];
                    if (row > si.last || row < si.low) sc[k][j] = -INFINITY;
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
#pragma unroll
            for (int k = 0; k < C::SPL; ++k) {
                float corr = 1.f;
                if (need[k]) {
                    corr = ex2(m[k] - mt[k]);          // 0 while m is -inf
                    m[k] = mt[k];
                }
                l[k] *= corr;
                // the accumulators' slots are 2u and 2u + 1
                const float c0 = __shfl_sync(0xffffffffu, corr, 8 * u), c1 = __shfl_sync(0xffffffffu, corr, 8 * u + 4);
#pragma unroll
                for (int n = 0; n < C::HD / 16; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[k][n][i] *= i & 1 ? c1 : c0;
            }
        }
        // the scores become the weights
#pragma unroll
        for (int k = 0; k < C::SPL; ++k) {
            const float base = m[k] == -INFINITY ? 0.f : m[k] - OFF;     // no row seen yet: every p is 0
#pragma unroll
            for (int j = 0; j < 4; ++j) sc[k][j] = ex2(sc[k][j] - base);
            l[k] += (sc[k][0] + sc[k][1]) + (sc[k][2] + sc[k][3]);
            if constexpr (C::E8) {
#pragma unroll
                for (int j = 0; j < 4; ++j) sc[k][j] *= vscale;
            }
        }
        // A row that a slot does not see must not reach it: its weight 0 times what an unwritten or
        // unseen row holds (NaN, infinity) would. Rows that every slot of the block sees go
        // through the MMAs, with the others' V taken as 0; rows that only some query rows see (the last n_q - 1,
        // and as many at a window's start) are added one by one to the slots that see them.
        if (edge) {
            const int4 sg = seg_rows(smem);
            if (sg.x != sg.z || sg.y != sg.w) {
#pragma unroll
                for (int k = 0; k < C::SPL; ++k) {
                    const SlotInfo sa = slot_at(smem, 2 * u + 8 * k), sb = slot_at(smem, 2 * u + 1 + 8 * k);
                    int r = max(sg.z - row0, 0);
                    const int stop = min(sg.w - row0, C::WR - 1);
#pragma unroll 1
                    for (; r <= stop; ++r) {
                        const int row = row0 + r;
                        if (row >= sg.x && row <= sg.y) {             // skip the rows every slot sees
                            r = min(sg.y - row0, stop);
                            continue;
                        }
                        const float x = r & 8 ? (r & 1 ? sc[k][3] : sc[k][2]) : (r & 1 ? sc[k][1] : sc[k][0]);
                        const float p0 = __shfl_sync(0xffffffffu, x, 8 * u + ((r & 7) >> 1));
                        const float p1 = __shfl_sync(0xffffffffu, x, 8 * u + 4 + ((r & 7) >> 1));
                        add_row(vs, r0 + r, k, p0, p1, row <= sa.last && row >= sa.low, row <= sb.last && row >= sb.low,
                                lane);
                    }
                }
            }
        }
        // p in NP parts: each the rounding of what the ones before leave
        uint32_t pb[C::SPL][C::NP][2];
#pragma unroll
        for (int k = 0; k < C::SPL; ++k)
#pragma unroll
            for (int x = 0; x < C::NP; ++x)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    pb[k][x][h] = float2_to_kv2<MT>(sc[k][2 * h], sc[k][2 * h + 1]);
                    const float2 f = kv2_to_float2<MT>(pb[k][x][h]);
                    sc[k][2 * h] -= f.x;
                    sc[k][2 * h + 1] -= f.y;
                }
        // three parts of p (bf16): one copy of the sweep, masked throughout (the second would not fit the registers)
        if (C::NP == 2 && !edge) {
            values<false>(vs, r0, pb, 0u, 0u, lane);
        } else {
            uint32_t mask[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
            if (edge) {
                const int4 sg = seg_rows(smem);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int row = row0 + col[j];
                    if (row < sg.x || row > sg.y) mask[j >> 1] &= 0xFFFFu << (16 * (1 - (j & 1)));
                }
            }
            values<true>(vs, r0, pb, mask[0], mask[1], lane);
        }
    }

    // (reference, sum) of the warp's slots. A slot that has seen no row has -inf; one whose every score is NaN
    // keeps its NaN sum.
    __device__ __forceinline__ void publish(float2 *mm, int lane)
    {
#pragma unroll
        for (int k = 0; k < C::SPL; ++k) {
            float lt = l[k];
            lt += __shfl_xor_sync(0xffffffffu, lt, 1);
            lt += __shfl_xor_sync(0xffffffffu, lt, 2);
            if ((lane & 3) == 0)
                mm[(lane >> 2) + 8 * k] = make_float2(m[k] == -INFINITY && lt != 0.f ? 0.f : m[k] - OFF, lt);
        }
    }

    // The accumulators times 2^(own reference - the largest among the warps).
    __device__ __forceinline__ void weigh(const float2 *mm, int warp, int lane)
    {
#pragma unroll
        for (int k = 0; k < C::SPL; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * (lane & 3) + e + 8 * k;
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < C::NWC; ++w) M = fmaxf(M, mm[w * C::SLOTS + i].x);
                const float x = mm[warp * C::SLOTS + i].x;
                const float wt = x == -INFINITY ? 0.f : ex2(x - M);
#pragma unroll
                for (int n = 0; n < C::HD / 16; ++n) {
                    o[k][n][e] *= wt;
                    o[k][n][2 + e] *= wt;
                }
            }
    }

    __device__ __forceinline__ float4 four(int k, int part, int e) const
    {
        return make_float4(o[k][2 * part][e], o[k][2 * part][2 + e], o[k][2 * part + 1][e], o[k][2 * part + 1][2 + e]);
    }

    // All of them into the warp's own area
    __device__ __forceinline__ void spread(float *area, int lane) const
    {
        float *at = area + 2 * (lane & 3) * C::MS + 4 * (lane >> 2);
#pragma unroll
        for (int k = 0; k < C::SPL; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int p = 0; p < C::NPART; ++p)
                    *reinterpret_cast<float4 *>(at + (e + 8 * k) * C::MS + 32 * p) = four(k, p, e);
    }

    // All warps onto one area (zeroed): in round r warp w adds part (w + r) % NPART, so that no two meet. The
    // registers are first turned by w parts, for their index to be r in every warp.
    __device__ __forceinline__ void gather(float *area, int warp, int lane)
    {
#pragma unroll
        for (int b = 1; b < C::NPART; b <<= 1) {
            const bool on = (warp & b) != 0;
#pragma unroll
            for (int k = 0; k < C::SPL; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float x[C::NPART];
#pragma unroll
                        for (int p = 0; p < C::NPART; ++p) x[p] = o[k][2 * p + h][i];
#pragma unroll
                        for (int p = 0; p < C::NPART; ++p) o[k][2 * p + h][i] = on ? x[(p + b) % C::NPART] : x[p];
                    }
        }
        float *at = area + 2 * (lane & 3) * C::MS + 4 * (lane >> 2);
#pragma unroll 1
        for (int grp = 0; grp * C::NPART < C::NWC; ++grp)          // more warps than parts: in groups
#pragma unroll
            for (int r = 0; r < C::NPART; ++r) {
                if (warp / C::NPART == grp) {
                    float *p = at + 32 * ((warp + r) & (C::NPART - 1));
                    float4 v[2 * C::SPL];
#pragma unroll
                    for (int x = 0; x < 2 * C::SPL; ++x)
                        v[x] = *reinterpret_cast<const float4 *>(p + ((x & 1) + 8 * (x >> 1)) * C::MS);
#pragma unroll
                    for (int x = 0; x < 2 * C::SPL; ++x) {
                        const float4 y = four(x >> 1, r, x & 1);
                        v[x].x += y.x; v[x].y += y.y; v[x].z += y.z; v[x].w += y.w;
                        *reinterpret_cast<float4 *>(p + ((x & 1) + 8 * (x >> 1)) * C::MS) = v[x];
                    }
                }
                asm volatile("bar.sync 1, %0;" :: "r"(C::NWC * 32) : "memory");
            }
    }
};

// Q of the block's slots as MMA A fragments in shared memory: NP parts, each the rounding of what the
// ones before leave of q sc, with a power of two sc per slot (exact). Slots past the last are zero.
template <class C>
struct PagedQ {
    static constexpr int NW = C::NWC;                            // the compute warps
    static constexpr int V4 = C::HD <= 128 ? 1 : 2;              // float4 of a row a lane owns
    static constexpr int ITER = (C::SLOTS + NW - 1) / NW;
    float4 x[ITER][V4];

    __device__ __forceinline__ void load(const PagedArgs &a, int s, int hk, int qg, int tid)
    {
        const int warp = tid >> 5, lane = tid & 31;
#pragma unroll
        for (int it = 0; it < ITER; ++it) {
            const int i = warp + it * NW, qh = qg * C::SLOTS + i;
            const bool have = i < C::SLOTS && qh < a.n_q * a.group;
            const int t = have ? div(a.by_group, qh) : 0, g = have ? qh - t * a.group : 0;
            const float *row = a.q + (((size_t)s * a.n_q + t) * a.n_head + (size_t)hk * a.group + g) * C::HD;
#pragma unroll
            for (int v = 0; v < V4; ++v) {
                x[it][v] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (have && lane * 4 < C::HD) x[it][v] = ld_dep(reinterpret_cast<const float4 *>(row + v * 128) + lane);
            }
        }
    }
    __device__ __forceinline__ void store(uint8_t *smem, const PagedArgs &a, const SlotRows &sr, int hk, int qg, int tid);
};

template <class C>
__device__ __forceinline__ void PagedQ<C>::store(uint8_t *smem, const PagedArgs &a, const SlotRows &sr, int hk, int qg,
                                                 int tid)
{
    using MT = typename C::MT;
    const int warp = tid >> 5, lane = tid & 31;
    const bool active = lane * 4 < C::HD;
#pragma unroll
    for (int it = 0; it < ITER; ++it) {
        const int i = warp + it * NW;
        if (i >= C::SLOTS) break;
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
            const bool have = qh < a.n_q * a.group;
            const int t = div(a.by_group, qh);
            si.last = have ? sr.last(t) : -1;
            si.low = have ? sr.low(t) : 0;
            si.slope = a.slopes && have ? ld_dep(a.slopes + hk * a.group + qh - t * a.group) * kLog2e : 0.f;
            reinterpret_cast<SlotInfo *>(smem + C::OFF_SLOT)[i] = si;
        }
        if (!active) continue;
#pragma unroll
        for (int v = 0; v < V4; ++v) {
            const int d = v * 128 + lane * 4;
            float f[4] = {x[it][v].x * sc, x[it][v].y * sc, x[it][v].z * sc, x[it][v].w * sc};
            // dimension d is element 0 of a lane's four in k-step kk (the K loads' order)
            const int c = d / C::CW, in = d % C::CW, u = in / (C::CW / 4), w = in % (C::CW / 4) / 4;
            const int kk = c * C::KPC + w, fl = (i & 7) * 4 + u;
            uint32_t *q0 = reinterpret_cast<uint32_t *>(smem + C::OFF_Q);
#pragma unroll
            for (int part = 0; part < C::NP; ++part) {
                uint32_t *to;
                int next = 2;                                    // words to the pair's second half
                if (C::SLOTS == 16) {
                    to = q0 + ((part * C::KSTEPS + kk) * 32 + fl) * 4 + (i >> 3);
                } else if (part < 2) {
                    to = q0 + (kk * 32 + fl) * 4 + part;
                } else {
                    to = q0 + C::KSTEPS * 128 + (kk * 32 + fl) * 2;
                    next = 1;
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t b = float2_to_kv2<MT>(f[2 * j], f[2 * j + 1]);
                    to[next * j] = b;
                    const float2 r = kv2_to_float2<MT>(b);
                    f[2 * j] -= r.x;
                    f[2 * j + 1] -= r.y;
                }
            }
        }
    }
}

__device__ __forceinline__ SlotRows seq_rows(const PagedArgs &a, int nkv, int start)
{
    return SlotRows{nkv - a.n_q, start, a.window};
}

// The sequence that tile t belongs to: the first one whose end lies past it.
__device__ __forceinline__ int find_seq(const int *cs, int n, int t)
{
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cs[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

// First row of the first tile of a sequence, and one past its last row (TILE is a power of two)
template <int TILE>
__device__ __forceinline__ int2 seq_extent(const PagedArgs &a, const SlotRows &sr)
{
    const int R = max(sr.last(a.n_q - 1) + 1, 0), L = min(sr.low(0), R);
    return make_int2(L & -TILE, R);
}

template <class C, bool RULES>
__global__ void __launch_bounds__(C::THREADS, C::MIN_BLOCKS)
attn_paged_stream(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const PagedArgs a)
{
    constexpr int NWC = C::NWC, S = C::S, TILE = C::TILE, WR = C::WR, NSL = C::NSL, TPG = C::TPG;
    extern __shared__ __align__(1024) uint8_t smem[];      // the swizzle needs the alignment (launch: no static shared memory)
    SliceInfo *desc = reinterpret_cast<SliceInfo *>(smem + C::OFF_DESC);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *empty = full + S;
    volatile int *flags = reinterpret_cast<volatile int *>(empty + S);   // [0] abort, [1] tiles issued
    int4 *srank = reinterpret_cast<int4 *>(smem + C::OFF_SEQ);   // the rank's first tile, one past its last; share, gap
    int *cs = reinterpret_cast<int *>(srank + 1);            // tiles before each sequence
    int *snkv = cs + kPagedSeqs + 1, *sstart = snkv + kPagedSeqs;
    uint8_t *behind = reinterpret_cast<uint8_t *>(sstart + kPagedSeqs);   // sequences with tiles before each

    const int hk = blockIdx.y, qg = blockIdx.x, rank = blockIdx.z;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == NWC) {
        // ---------------- producer warp ----------------
        if (lane == 0) {
            for (int i = 0; i < S; ++i) {
                mbar_init(full + i, 1);
                mbar_init(empty + i, NSL);
            }
            flags[0] = 0;
            flags[1] = 0;
            fence_barrier_init();
            prefetch_tensormap(&kmap);
            prefetch_tensormap(&vmap);
        }
        pdl_wait();
        pdl_launch_dependents();
        // rows and tiles of every sequence, and the tiles before it: lane i takes `per` of them, their positions
        // and starts loaded together
        const int per = (a.n_seq + 31) / 32;
        constexpr int MOST = kPagedSeqs / 32;
        int pos[MOST], st[MOST];
#pragma unroll
        for (int i = 0; i < MOST; ++i) {
            pos[i] = -1;
            st[i] = 0;
            if (i < per) {
                const int s = lane * per + i;
                if (s < a.n_seq) pos[i] = ld_dep(a.positions + s);
                if (a.starts && s < a.n_seq) st[i] = ld_dep(a.starts + s);
            }
        }
        int n[MOST], sum = 0, some = 0;
#pragma unroll
        for (int i = 0; i < MOST; ++i) {
            n[i] = 0;
            if (i >= per) break;
            const int s = lane * per + i;
            if (s >= a.n_seq) continue;
            const int nkv = min(max(pos[i], -1), a.cap - 1) + 1;
            if ((pos[i] < -1 || pos[i] >= a.cap) && (hk | qg) == 0 && rank == 0) atomicOr(a.err, kErrPositionClamped);
            snkv[s] = nkv;
            sstart[s] = st[i];
            const SlotRows sr = seq_rows(a, nkv, st[i]);
            const int2 x = seq_extent<TILE>(a, sr);
            if (sr.low(0) < x.y) n[i] = (int)((unsigned)(x.y - x.x + TILE - 1) / TILE);
            sum += n[i];
            some += n[i] > 0;
        }
        int before = sum, upto = some;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, before, off), z = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) {
                before += y;
                upto += z;
            }
        }
        const int total = __shfl_sync(0xffffffffu, before, 31);
        // Going from one sequence to the next costs a block the time of `turn` tiles (the merge, the next q). So the
        // ranks take equal parts not of the tiles but of places: a tile each, and `gap` between two
        // sequences with tiles (`turn`, or half of a rank's part where that is less). A sequence's own tiles
        // have no gap, so that every rank between its first and its last has some of them.
        const int turns = max(__shfl_sync(0xffffffffu, upto, 31) - 1, 0);
        const int gap = min(a.turn, div(a.by_ranks, total + a.ranks - 1) / 2);
        const int share = max(div(a.by_ranks, total + gap * turns + a.ranks - 1), 1);
        // the first tiles at or past the rank's first place and the next rank's
        const int from = rank * share;
        int first = -1, end = -1;
        before -= sum;
        upto -= some;
#pragma unroll
        for (int i = 0; i < MOST; ++i) {
            if (i >= per) break;
            const int s = lane * per + i;
            if (s >= a.n_seq) continue;
            cs[s] = before;
            behind[s] = (uint8_t)upto;
            const int shift = gap * upto;                      // a tile's place is its number and this
            if (n[i] > 0) {
                if (first < 0 && before + n[i] + shift > from) first = max(from - shift, before);
                if (end < 0 && before + n[i] + shift > from + share) end = max(from + share - shift, before);
                before += n[i];
                ++upto;
            }
        }
        const unsigned hf = __ballot_sync(0xffffffffu, first >= 0), he = __ballot_sync(0xffffffffu, end >= 0);
        first = __shfl_sync(0xffffffffu, first, __ffs(hf) - 1);
        end = __shfl_sync(0xffffffffu, end, __ffs(he) - 1);
        if (hf == 0) first = total;
        if (he == 0) end = total;
        if (lane == 0) {
            cs[a.n_seq] = total;
            *srank = make_int4(first, end, share, gap);
        }
        __syncthreads();                                       // the compute warps go on to their first q
        const int ntiles = end - first;

        // Descriptors: lane i has slice i of a group of TPG tiles. A group's pages are loaded two groups
        // ahead and its scales one ahead, so that nothing waits for them; its descriptors go to one of four
        // buffers (a buffer's tiles are consumed before it comes round again).
        int seq = find_seq(cs, a.n_seq, first + lane / NSL);   // the lane's sequence; it only moves on
        int row = 0;
        bool need = false;                                     // some row of the slice's box is attended
        // q of a sequence that is about to begin, into L2: the rows of the block's slots
        auto prefetch_q = [&](int s) {
            const int x0 = qg * C::SLOTS, x1 = min(x0 + C::SLOTS, a.n_q * a.group) - 1;
            for (int t = div(a.by_group, x0); t <= div(a.by_group, x1); ++t)
                prefetch_l2(a.q + (((size_t)s * a.n_q + t) * a.n_head + (size_t)hk * a.group) * C::HD,
                            (uint32_t)(a.group * C::HD * sizeof(float)));
        };
        auto locate = [&](int grp) {
            const int t = first + grp * TPG + lane / NSL;
            need = t < end;
            if (!need) return;
            const int was = seq;
            while (cs[seq + 1] <= t) ++seq;
            if (seq != was && lane % NSL == 0) prefetch_q(seq);
            const SlotRows sr = seq_rows(a, snkv[seq], sstart[seq]);
            const int2 x = seq_extent<TILE>(a, sr);
            row = x.x + (t - cs[seq]) * TILE + lane % NSL * WR;
            const int box = row & -a.box_rows;
            need = box < x.y && box + a.box_rows > sr.low(0);
        };
        auto load_page = [&](int &z) {                         // and the row in the page
            const int pg = div(a.by_page, row);
            z = row - pg * a.page_size;
            return need ? ld_dep(a.table + (size_t)seq * a.max_pages + pg) : -1;
        };
        auto load_scales = [&](int p) {
            float2 f = make_float2(1.f, 1.f);
            if (C::E8 && (unsigned)p < (unsigned)a.n_pages) {
                f.x = ld_dep(a.k_scale + (size_t)p * a.n_kv_head + hk);
                f.y = ld_dep(a.v_scale + (size_t)p * a.n_kv_head + hk);
            }
            return f;
        };
        auto write = [&](int grp, int p, int z, bool wanted, float2 f) {
            const bool there = (unsigned)p < (unsigned)a.n_pages;
            if (wanted && !there) atomicOr(a.err, kErrBadPage);
            desc[(grp & 3) * 32 + lane] = SliceInfo{there ? p : -1, z, f.x, f.y};
        };
        uint64_t once;
        asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
        const int BR = a.box_rows, nbox = TILE / BR, bsl = BR / WR;
        auto issue = [&](int t) {                              // by lane 0
            const int st = t % S;
            const SliceInfo *d = desc + (t / TPG & 3) * 32 + t % TPG * NSL;
            unsigned bytes = 0;
            for (int b = 0; b < nbox; ++b) bytes += d[b * bsl].page >= 0 ? 2u * (unsigned)BR * C::ROWB : 0u;
            mbar_arrive_expect_tx(full + st, bytes);
            uint8_t *kst = smem + st * C::STAGE_BYTES;
            for (int b = 0; b < nbox; ++b) {
                const SliceInfo x = d[b * bsl];
                if (x.page < 0) continue;
#pragma unroll
                for (int c = 0; c < C::NCH; ++c) {
                    uint8_t *to = kst + c * (C::TILE_BYTES / C::NCH) + b * BR * C::CHB;
                    tma_load_4d_once(to, &kmap, full + st, c * C::CW, hk, x.z, x.page, once);
                    tma_load_4d_once(to + C::TILE_BYTES, &vmap, full + st, c * C::CW, hk, x.z, x.page, once);
                }
            }
            flags[1] = t + 1;
        };
        // the first copies go out before the scales are there
        locate(0);
        int z0, z1;
        const int p0 = load_page(z0);
        const bool n0 = need;
        desc[lane] = SliceInfo{(unsigned)p0 < (unsigned)a.n_pages ? p0 : -1, z0, 1.f, 1.f};
        const float2 f0 = load_scales(p0);
        __syncwarp();
        const int early = min(1, ntiles);                      // the rest when the descriptors are complete
        if (lane == 0)
            for (int t = 0; t < early; ++t) issue(t);
        locate(1);
        int p1 = load_page(z1);
        bool n1 = need;
        __syncwarp();
        write(0, p0, z0, n0, f0);
        // group 0's descriptors are complete (without tiles nobody waits)
        if (ntiles > 0) asm volatile("bar.arrive 2, %0;" :: "r"(C::THREADS) : "memory");
        float2 f1 = load_scales(p1);
        bool dead = false;
        for (int grp = 0; grp * TPG < ntiles; ++grp) {
            locate(grp + 2);
            int z2;
            const int p2 = load_page(z2);
            const bool n2 = need;
            if (lane == 0) {
                const int stop = min((grp + 1) * TPG, ntiles);
                for (int t = grp ? grp * TPG : early; t < stop; ++t) {
                    if (t >= S && !mbar_wait_bounded(empty + t % S, ((t / S) - 1) & 1)) {
                        flags[0] = 1;
                        atomicOr(a.err, kErrPipelineTimeout);
                        dead = true;
                        break;
                    }
                    issue(t);
                }
            }
            __syncwarp();
            if (__shfl_sync(0xffffffffu, (int)dead, 0)) break;
            write(grp + 1, p1, z1, n1, f1);
            p1 = p2;
            z1 = z2;
            n1 = n2;
            f1 = load_scales(p1);
            __syncwarp();
        }
    } else {
        // ---------------- compute warps ----------------
        pdl_wait();
        pdl_launch_dependents();
        __syncthreads();
        // Values that only the ends of a sequence need are read again from shared memory there, so that the tile
        // loop's registers hold the accumulators.
        volatile SegInfo *seg = reinterpret_cast<volatile SegInfo *>(smem + C::OFF_SEG);
        auto nslots = [&] { return min(C::SLOTS, a.n_q * a.group - qg * C::SLOTS); };
        auto head_row = [&](int s, int i) {                    // of slot i of the block
            const int x = qg * C::SLOTS + i, t = div(a.by_group, x);
            return ((size_t)s * a.n_q + t) * a.n_head + hk * a.group + (x - t * a.group);
        };
        // sequences that start here: which ranks have their rows; no rows at all: 0
        const int first = srank->x, end = srank->y;
        for (int s = tid; s < a.n_seq; s += NWC * 32) {
            const int c = cs[s], n = cs[s + 1] - c;
            if (!((c >= first && c < end) || (n == 0 && c == cs[a.n_seq] && rank == 0))) continue;
            if (a.ranks > 1 && (hk | qg) == 0)
                a.ws_span[s] = make_int2(rank, n > 0 ? (c + srank->w * behind[s] + n - 1) / srank->z : rank);
            if (n == 0)
                for (int i = 0; i < nslots(); ++i)
                    for (int d = 0; d < C::HD; d += 4)
                        *reinterpret_cast<float4 *>(a.out + head_row(s, i) * C::HD + d) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const uint32_t smem_u = smem_u32(smem);
        float2 *mm = reinterpret_cast<float2 *>(smem + C::OFF_Q);
        float2 *res = reinterpret_cast<float2 *>(reinterpret_cast<float *>(smem + C::OFF_Q) + C::OFF_RES);
        float *mo = reinterpret_cast<float *>(smem + C::OFF_Q) + C::OFF_MO;
        bool begun = false;
        PagedQ<C> q;
        if (first < end && C::Q_EARLY) q.load(a, find_seq(cs, a.n_seq, first), hk, qg, tid);
        for (int at = first; at < end;) {
            {
                const int s = find_seq(cs, a.n_seq, at);
                const SlotRows sr = seq_rows(a, snkv[s], sstart[s]);
                const int t0 = div(a.by_group, qg * C::SLOTS), t1 = div(a.by_group, qg * C::SLOTS + nslots() - 1);
                if (!C::Q_EARLY) q.load(a, s, hk, qg, tid);
                q.store(smem, a, sr, hk, qg, tid);
                if (tid == 0) {
                    seg->seen_lo = sr.low(t1);
                    seg->seen_hi = sr.last(t0);
                    seg->any_lo = sr.low(t0);
                    seg->any_hi = sr.last(t1);
                    seg->row0 = seq_extent<TILE>(a, sr).x;
                    seg->tile0 = cs[s] - first;
                    seg->seq = s;
                    seg->from = at - first;
                    seg->to = min(end, cs[s + 1]) - first;
                }
            }
            if (!begun) asm volatile("bar.sync 2, %0;" :: "r"(C::THREADS) : "memory");
            else asm volatile("bar.sync 1, %0;" :: "r"(NWC * 32) : "memory");
            begun = true;
            PagedWarp<C, RULES> w;
            w.init(smem_u, lane);
            // warp w has slice w % NSL of every WPT-th stage
            int t = seg->from;
            t += (warp / NSL + C::WPT - t % C::WPT) % C::WPT;
            const int to = flags[0] ? 0 : seg->to;       // after a timeout nothing is waited for any more
#pragma unroll 1
            for (; t < to; t += C::WPT) {
                const int st = t % S;
                const bool landed = mbar_wait_bounded(full + st, (t / S) & 1);
                if (!__all_sync(0xffffffffu, landed)) {
                    if (lane == 0) { flags[0] = 1; atomicOr(a.err, kErrPipelineTimeout); }
                    break;
                }
                const int row0 = seg->row0 + (t - seg->tile0) * TILE + warp % NSL * WR;
                const int4 sg = PagedWarp<C, RULES>::seg_rows(smem_u);
                const uint4 f = lds128(smem_u + C::OFF_DESC + ((t / TPG & 3) * 32 + t % TPG * NSL + warp % NSL) * 16);
                if ((int)f.x >= 0 && row0 <= sg.w && row0 + WR > sg.z)
                    w.process(smem_u, smem_u + st * C::STAGE_BYTES, warp % NSL * WR, row0, __uint_as_float(f.z),
                              __uint_as_float(f.w), row0 < sg.x || row0 + WR - 1 > sg.y, a.cap_log2, lane);
                __syncwarp();
                if (lane == 0) mbar_arrive(empty + st);
            }
            // The next sequence's q is on its way while the warps' states are merged, over the Q fragments, which
            // are no longer read. At the block's last sequence every tile has been consumed and none is on its
            // way, so that each warp has a part of the ring to itself; before that, onto one area in rounds.
            const int from = seg->from + first, stop = seg->to + first;
            if (C::Q_EARLY && stop < end) q.load(a, find_seq(cs, a.n_seq, stop), hk, qg, tid);
            const bool over = stop == end;
            float *area = over ? reinterpret_cast<float *>(smem) : mo;
            asm volatile("bar.sync 1, %0;" :: "r"(NWC * 32) : "memory");
            w.publish(mm + warp * C::SLOTS, lane);
            if (!over)
                for (int i = tid; i < C::SLOTS * C::MS / 4; i += NWC * 32)
                    reinterpret_cast<float4 *>(mo)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            asm volatile("bar.sync 1, %0;" :: "r"(NWC * 32) : "memory");
            if (tid < C::SLOTS) {                        // (reference, sum) of the block
                float M = -INFINITY, sum = 0.f;
#pragma unroll
                for (int x = 0; x < NWC; ++x) M = fmaxf(M, mm[x * C::SLOTS + tid].x);
#pragma unroll
                for (int x = 0; x < NWC; ++x) {
                    const float2 ml = mm[x * C::SLOTS + tid];
                    if (ml.x != -INFINITY) sum = fmaf(ex2(ml.x - M), ml.y, sum);
                }
                res[tid] = make_float2(M, sum);
            }
            w.weigh(mm, warp, lane);
            if (over) {
                w.spread(area + warp * C::SLOTS * C::MS, lane);
                asm volatile("bar.sync 1, %0;" :: "r"(NWC * 32) : "memory");
            } else {
                w.gather(area, warp, lane);
            }
            const int sq = seg->seq;
            const bool begins = from == cs[sq], whole = begins && stop == cs[sq + 1];
            const size_t part = ((size_t)(rank * 2 + (begins ? 1 : 0)) * a.units + (hk * a.qgroups + qg)) * C::SLOTS;
            const bool bad = flags[0] != 0;              // left unwritten; the error word says why
            constexpr int D4 = C::HD / 4;
            for (int i = tid; i < nslots() * D4 && !bad; i += NWC * 32) {
                const int g = i / D4, d = (i % D4) * 4;
                const float2 ml = res[g];
                float4 O = C::merge_read(area + g * C::MS, d);
                if (over) {
#pragma unroll
                    for (int x = 1; x < NWC; ++x) {
                        const float4 v = C::merge_read(area + (x * C::SLOTS + g) * C::MS, d);
                        O.x += v.x; O.y += v.y; O.z += v.z; O.w += v.w;
                    }
                }
                if (whole) {
                    const float inv = ml.y == 0.f ? 0.f : 1.f / ml.y;
                    *reinterpret_cast<float4 *>(a.out + head_row(sq, g) * C::HD + d) =
                        make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv);
                } else {
                    *reinterpret_cast<float4 *>(a.ws_o + (part + g) * C::HD + d) = O;
                    if (d == 0) a.ws_ml[part + g] = ml;
                }
            }
            at = stop;
            asm volatile("bar.sync 1, %0;" :: "r"(NWC * 32) : "memory");
        }
    }
    __syncthreads();

    // No copy may still be writing shared memory when the block exits; without an abort every issued
    // tile has been waited for.
    if (flags[0] && tid == NWC * 32) {
        const int issued = flags[1];
        for (int t = issued - S > 0 ? issued - S : 0; t < issued; ++t)
            (void)mbar_wait_bounded(full + (t % S), (t / S) & 1);
    }
}

// The sequences whose rows several ranks share: o = sum w oc / sum w S over their parts, w = 2^(mx - max mx).
// One block per (row, sequence, chunk of DC dimensions); a group of DC / 4 lanes folds every NG-th part,
// BATCH of them in flight, and the groups are folded through shared memory.
template <int HD, int DC>
__global__ void __launch_bounds__(128) attn_paged_combine(const PagedArgs a, int slots)
{
    constexpr int LPS = DC / 4, NG = 128 / LPS, BATCH = 8;
    __shared__ float2 sm_ml[NG];
    __shared__ float sm_acc[NG][DC];
    // no early start for the kernel after this one: a streaming block that becomes resident beside these finds
    // the SM's shared memory and registers in pieces, and one of the blocks that should be there then waits
    // for a whole block's time (131072 rows: 54 us with one block fewer than fit, 73 with all)
    pdl_wait();
    const int s = blockIdx.y, r = blockIdx.x;
    const uint2 sp = [&] {
        uint2 v;
        asm volatile("ld.global.cg.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(a.ws_span + s) : "memory");
        return v;
    }();
    if (sp.x == sp.y) return;
    const int t = r / a.n_head, h = r - t * a.n_head, hk = h / a.group;
    const int x = t * a.group + (h - hk * a.group);
    const size_t in_rank = (size_t)(hk * a.qgroups + x / slots) * slots + x % slots;
    const size_t rank_rows = (size_t)a.units * slots;
    const int P = (int)(sp.y - sp.x) + 1;
    const int group = threadIdx.x / LPS, dl = threadIdx.x % LPS;
    auto at = [&](int j) { return ((size_t)(sp.x + j) * 2 + (j == 0 ? 1 : 0)) * rank_rows + in_rank; };

    float m = -INFINITY, S = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int base = group; base < P; base += NG * BATCH) {
        float2 ml[BATCH];
        float4 v[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int j = base + b * NG;
            ml[b] = make_float2(-INFINITY, 0.f);
            v[b] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j < P) {
                const size_t row = at(j);
                ml[b] = ld_dep(a.ws_ml + row);
                v[b] = ld_dep(reinterpret_cast<const float4 *>(a.ws_o + row * HD + blockIdx.z * DC) + dl);
            }
        }
        float mb = m;
#pragma unroll
        for (int b = 0; b < BATCH; ++b) mb = fmaxf(mb, ml[b].x);
        if (mb == -INFINITY) continue;
        const float c = m == -INFINITY ? 0.f : ex2(m - mb);
        S *= c;
        acc.x *= c; acc.y *= c; acc.z *= c; acc.w *= c;
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            if (ml[b].x == -INFINITY) continue;
            const float w = ex2(ml[b].x - mb);
            S = fmaf(w, ml[b].y, S);
            acc.x = fmaf(w, v[b].x, acc.x);
            acc.y = fmaf(w, v[b].y, acc.y);
            acc.z = fmaf(w, v[b].z, acc.z);
            acc.w = fmaf(w, v[b].w, acc.w);
        }
        m = mb;
    }
    if (dl == 0) sm_ml[group] = make_float2(m, S);
    *reinterpret_cast<float4 *>(&sm_acc[group][dl * 4]) = acc;
    __syncthreads();
    for (int d = threadIdx.x; d < DC; d += 128) {
        float M = -INFINITY;
#pragma unroll
        for (int g = 0; g < NG; ++g) M = fmaxf(M, sm_ml[g].x);
        float sum = 0.f, o = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const float2 y = sm_ml[g];
            const float w = y.x == -INFINITY ? 0.f : ex2(y.x - M);
            sum = fmaf(w, y.y, sum);
            o = fmaf(w, sm_acc[g][d], o);
        }
        const size_t row = (size_t)s * a.n_q * a.n_head + r;
        a.out[row * HD + blockIdx.z * DC + d] = sum == 0.f ? 0.f : o / sum;
    }
}

} // namespace attn
