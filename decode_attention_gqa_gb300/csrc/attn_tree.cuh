// attn_tree.cuh -- attention of drafted trees over a paged cache, on the fifth-generation tensor cores.
//
// Mathematics. For a node t at position x over the cache rows j it sees -- all before its tree, and the
// tree's own as its mask has them --
//     s_j = rules(scale q.k_j),  o = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j log2 e - m),
// one pass with a running reference m, an integer, that moves when a score passes it by 8; what was weighed before is
// then multiplied by a power of two, which rounds nothing but what falls below the 16-bit type's smallest. An
// e4m3 cache holds codes with one scale per page and KV head: the K scale multiplies a page's scores, the V scale p; the
// reference follows s + log2 of the V scale (rounded up), so that p times the scale stays in the 16-bit
// range whatever the scales are; sum p is f32.
//
// Tiles. A (node, head) pair of a KV head is a slot; 128 slots are the M rows of both products. S = Q K^T
// (128 x TR, operands in shared memory) goes to tensor memory, a warpgroup turns it into P in place, one row a
// thread, so that maxima and sums need no exchange, and O += P V takes P from tensor memory and V as an MN-major
// operand from the tile TMA brought. The two warpgroups take tiles in turn: three (four) S in tensor memory, one O, and one
// reference that a tile's warpgroup hands on to the next one's, so that the tensor cores work for one warpgroup while the
// other is at its exponentials. (With an S and an O for each of two warpgroups on alternate tiles, a tile waited 3500 cycles
// for its S. Blocks of 256 slots, two tiles of Q over the same K and V, read half as much of L2 and took 1.1 to 1.25 times as
// long, 448 slots over 8192 rows 35 us and not 28: a warpgroup waited for its own products.)
//
// Parts. 16-bit queries enter as one operand, f32 queries as two (the rounding, and the rounding of what it left), and
// then the weights too: f16 over f16 and e4m3 caches (rows of q scaled by a power of two, so that nothing is lost to
// f16's range), bf16 over bf16 caches. The weights of 16-bit queries are two as well where the result has as many bits as
// one of them (queries of the cache's type), else one. 16-bit queries over an e4m3 cache are split into e4m3 parts
// instead -- two hold the 8 bits of a bfloat16, three the 11 of a binary16 -- so that K's codes enter the products as
// they are, at twice the rate, and V alone is converted.
//
// Sums. At each step of 16 rows the tensor cores cut an accumulator off at 24 bits, always towards 0: over 30000 rows in one
// block 7e-5 of the result was lost, over 131072 3e-4. For f32 queries O is added to a sum in the workspace every 2048
// rows, at the place of the block's part (32 sequences of up to 32768 rows of 128, e4m3: 7.7e-5 of the result before, 4.6e-6 now,
// 375 and 386 us; every 1024 rows 2.5e-6 and 411 us, every 512 1.4e-6 and 432 us). Results of 16 bits are rounded at 2^-12 or
// 2^-9 of themselves; their sums run on (f16 queries over bf16, whose parts are the same code: every 16384 rows).
//
// Work. A block serves one unit -- a KV head and 128 slots of it. The tiles that a unit has in all sequences are
// laid end to end, and the unit's blocks (ranks; as many as make a block an SM, or four rounds of blocks where one would
// leave too many SMs idle) take equal runs of them, the turn to another sequence counted as some more: what a block has
// of a sequence is its output where it has all of it, else a part (reference, sum, sum p v) for attn_tree_combine. The
// KV heads of a rank run at the same time, so that the pieces of a row that they read are asked of memory together (one
// row of blocks over all units in turn took 1.9 times as long over 32 sequences of up to 32768 rows).
//
// Warps: 8 of the softmax; 4 that convert e4m3 tiles to f16, and, in tiles that some slot does not see all
// of, take infinities and NaN out of V (a weight of 0 would spread them; where a block's part of the sequence ends, the
// softmax gives them to the slots that see them); a producer of K and one of V (pages, TMA); an issuer of each product. What a
// single warp does for each tile takes some 8 cycles an instruction, and code that runs once is fetched from L2 a line at a
// time: both are written for few instructions.
//
// Measured (calls in a graph, the joining kernel among them): 32 sequences of 17 .. 32768 rows, trees of 5 to 16 nodes, 32/8 heads
// of 128, e4m3, bf16 queries 215 us (1.09 GB, 5070 GB/s, 0.75 of a copy's rate); 8192 rows, 64 nodes, 28/4 heads 24.9 us; 4
// sequences of up to 8400 rows, trees of 33 to 60 nodes, 16/2 heads of 256, capped scores, a window of 4096, bf16 35.1 us; 512
// rows, 8 nodes, 8/2 heads, f32 queries 16.3 us. Over long rows no unit alone bounds it: a tile of 128 rows and 128 slots takes
// some 1600 cycles, the tensor cores 1170 of them (every slot of 128, with a node or not), a warpgroup half of its
// 3200 for each of its own, converting V 880; with half the products, without the exponentials, the sums or the
// conversion it took 1 to 4 % less. Short calls are chains: 2500 cycles to the first table entry, 5000 for Q, a tile's
// 4000 from K to P V, 1500 to 5000 for what is stored, the joining kernel.
#pragma once

#include <cuda_fp8.h>

#include "attn_device.cuh"
#include "attn_launch.h"
#include "attn_paged.cuh"
#include "attn_paged_launch.h"
#include "attn_partial_umma.cuh"

namespace attn {

constexpr unsigned kErrBadTree = 0x8u;        // ATTN_DEVERR_BAD_REQUEST
constexpr int kTreeTurn = 7;                  // what another sequence costs a block, in tiles
constexpr int kTreeDesc = 8;                  // tiles whose descriptors are kept: K runs at most 4 tiles ahead of S, S 3 of P

// PARTS: of q; PP: of the weights
template <int HD_, typename KV_, int PARTS_, int PP_>
struct TreeCfg {
    static constexpr int HD = HD_, PARTS = PARTS_, PP = PP_;
    using KV = KV_;
    using MT = typename PagedMma<KV>::T;
    static constexpr bool E8 = std::is_same<KV, E4m3>::value;
    static constexpr int NB = HD == 256 ? 4 : 3;               // S of the warpgroups in turn
    static constexpr int TR = HD == 256 ? 64 : 128;            // cache rows of a tile
    static constexpr int NSLC = TR / 16;                       // 16-row slices
    static constexpr int TPG = 32 / NSLC;                      // tiles whose pages a warp looks up at once
    static constexpr int SM_WARPS = 8, FIX = SM_WARPS;
    // of a block of few slots the first warps have rows, those of the first scheduler: the issuers are with the others
    static constexpr int PROD_V = FIX + 4, MMA_O = FIX + 5, MMA_S = FIX + 6, PROD_K = FIX + 7;
    // whole warpgroups where registers move between them: 512 threads of 128, of which the softmax takes 176 each and
    // the others 80: the block's 65536
    static constexpr int THREADS = (PROD_K + 1) * 32;
    // 8-bit K as it is (with q in 8-bit parts), or converted
    static constexpr bool F8 = E8 && PARTS == 1, KCONV = E8 && !F8;
    static constexpr int QES = F8 ? 1 : 2;                     // bytes of an element of a part of q
    static constexpr uint32_t QPART = 128u * HD * QES;         // a part of a tile of Q
    static constexpr uint32_t SLOT = (uint32_t)TR * HD * 2;    // K or V of a tile, 16 bits
    static constexpr uint32_t RAW = (uint32_t)TR * HD;         // 8 bits
    static constexpr uint32_t KSLOT = F8 ? RAW : SLOT;
    // chunks of a row as they lie in shared memory: 128 bytes (64: 8-bit rows of 64 dimensions)
    static constexpr int RCHB = HD < 128 ? HD : 128, RNCH = HD / RCHB, NCH = HD / 64;
    static constexpr uint32_t TM_COLS = 512;                   // O first, then the S
    static constexpr uint32_t DATA = 224 * 1024;               // Q and the rings
    static constexpr uint32_t OFF_DESC = DATA;
    static constexpr uint32_t OFF_BAR = OFF_DESC + kTreeDesc * 128;
    static constexpr int NBAR = 50 + kTreeDesc;
    static constexpr uint32_t OFF_FLAG = OFF_BAR + NBAR * 8;   // TMEM slot, abort, share, the block's first tile and the one behind it, wild segments
    static constexpr uint32_t OFF_SEQ = OFF_FLAG + 32;         // before, first token, places before, rows
    static constexpr uint32_t OFF_REF = OFF_SEQ + (4 * kTreeSeqs + 4) * 4;   // references of 128 slots
    static constexpr uint32_t SMEM = OFF_REF + 128 * 4;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(NB * TR + HD <= 512, "tensor memory");
};

struct __align__(16) TileInfo {
    int row0;                 // its first cache row
    int edge;                 // some slot does not see all of it
    unsigned slices;          // 16-row slices that are there
    int live;                 // rows of it that belong to the sequence
    unsigned unused[4];       // the scales in 16-byte loads
    float ks[8], vs[8];       // scales of its slices
    float lv[8];              // log2 of the V scales, rounded up
};
static_assert(sizeof(TileInfo) == 128, "its place in shared memory");

// What a block has of a sequence: tiles [t0, t1) of its T
struct TreeSeg {
    int s, t0, t1, T;
    int n, tok0, nkv, base, start;
    int slots;                // of the unit in this sequence, at most 128
    int row0;                 // first row of tile 0
};

__device__ __forceinline__ void tmem_ld32(uint32_t t, uint32_t (&r)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(t) : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t t, const uint32_t (&r)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
                 :: "r"(t), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                    "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
                    "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
                    "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t t, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 :: "r"(t), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                    "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t t, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "r"(t), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}
__device__ __forceinline__ void tmem_st2(uint32_t t, uint32_t a, uint32_t b)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" :: "r"(t), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void tmem_ld2(uint32_t t, uint32_t &a, uint32_t &b)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(a), "=r"(b) : "r"(t) : "memory");
}
// Waits for the loads issued before, of which r is one: nothing that uses r comes before it.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                   "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :: "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p;
}
// Products by a warp, of which the lane with `one` issues: no branch.
template <bool F8>
__device__ __forceinline__ void umma_ss(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    if constexpr (F8)                                          // e4m3 operands
        asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
                     "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(one) : "memory");
    else
        asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
                     "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(one) : "memory");
}
// D += A B with A in tensor memory.
__device__ __forceinline__ void umma_ts(uint32_t one, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc)
{
    asm volatile("{\n\t.reg .pred p, e;\n\tsetp.eq.u32 p, 0, 0;\n\tsetp.ne.b32 e, %4, 0;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(one) : "memory");
}

__device__ __forceinline__ void sts128(uint32_t p, const uint4 &v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" :: "r"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// mbarriers by their 32-bit shared addresses (as in attn_device.cuh otherwise)
__device__ __forceinline__ void bar_init(uint32_t bar, unsigned count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" :: "r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void bar_arrive_expect_tx(uint32_t bar, unsigned bytes)
{
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}"
                 :: "r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, unsigned parity)
{
    unsigned ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ void bar_commit(uint32_t one, uint32_t bar)
{
    asm volatile("{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
                 :: "r"(bar), "r"(one) : "memory");
}
__device__ __forceinline__ void tree_tma(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z, int w, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;"
        :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "l"(policy)
        : "memory");
}

// 1 / x to 2^-23 (division proper is a call, with registers saved around it)
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Pairs of f32 in one instruction
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t x)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
template <typename T>
__device__ __forceinline__ uint32_t mul_kv2(uint32_t a, uint32_t b)
{
    uint32_t r;
    if constexpr (std::is_same<T, __half>::value) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Bits [a, b) of 32, for a and b of any size.
__device__ __forceinline__ unsigned bit_range(int a, int b)
{
    a = min(max(a, 0), 32);
    b = min(max(b, 0), 32);
    const unsigned hi = b == 32 ? ~0u : (1u << b) - 1u, lo = a == 32 ? ~0u : (1u << a) - 1u;
    return hi & ~lo;
}

template <class C>
struct Tree {
    static constexpr int HD = C::HD, PARTS = C::PARTS, PP = C::PP, TR = C::TR;
    using MT = typename C::MT;

    const TreeArgs &a;
    uint8_t *smem;
    uint32_t sm;

    __device__ __forceinline__ Tree(const TreeArgs &args, uint8_t *base) : a(args), smem(base), sm(smem_u32(base)) {}

    // Rings of tiles of K and of V. full: TMA's copies are there; ready: converted or looked at; empty, raw: to be
    // filled again (16-bit tiles, and K's that are used as they are; 8-bit tiles that are converted)
    __device__ __forceinline__ uint32_t bar(int i) const { return sm + C::OFF_BAR + 8 * i; }
    __device__ __forceinline__ uint32_t full(bool v, int i) const { return bar(v * 16 + i); }
    __device__ __forceinline__ uint32_t ready(bool v, int i) const { return bar(v * 16 + 4 + i); }
    __device__ __forceinline__ uint32_t empty(bool v, int i) const { return bar(v * 16 + 8 + i); }
    __device__ __forceinline__ uint32_t raw(bool v, int i) const { return bar(v * 16 + 12 + i); }
    __device__ __forceinline__ uint32_t s_full(int i) const { return bar(32 + i); }
    __device__ __forceinline__ uint32_t p_ready(int i) const { return bar(36 + i); }
    __device__ __forceinline__ uint32_t o_done(int i) const { return bar(40 + i); }
    __device__ __forceinline__ uint32_t ref_known(int quad) const { return bar(44 + quad); }
    __device__ __forceinline__ uint32_t q_ready() const { return bar(48); }
    __device__ __forceinline__ uint32_t described(unsigned tile) const { return bar(50 + (tile & (kTreeDesc - 1))); }
    __device__ __forceinline__ uint32_t met() const { return bar(49); }
    // [0] tensor memory, [1] abort, [2] places of a rank, [3], [4] its first tile and the one behind its last, [5] segments (bit
    // i: the i-th, modulo 32) of whose V infinities or NaN were taken out
    __device__ __forceinline__ volatile int *flags() const { return reinterpret_cast<volatile int *>(smem + C::OFF_FLAG); }
    __device__ __forceinline__ int *before() const { return reinterpret_cast<int *>(smem + C::OFF_SEQ); }   // tiles before each sequence
    __device__ __forceinline__ int *tok() const { return before() + kTreeSeqs + 1; }                         // first tokens
    __device__ __forceinline__ int *place() const { return tok() + kTreeSeqs + 1; }                         // place of its first tile
    __device__ __forceinline__ int *rows() const { return place() + kTreeSeqs + 1; }                        // rows
    // Q, then V's tiles, K's, and the 8-bit ones that are converted
    __device__ __forceinline__ uint32_t v_slot(int i) const { return sm + a.q_bytes + i * C::SLOT; }
    __device__ __forceinline__ uint32_t k_slot(int i) const { return v_slot(a.nv) + i * C::KSLOT; }
    __device__ __forceinline__ uint32_t raw_slot(bool v, int i) const { return k_slot(a.nk) + ((v ? 0 : a.nrv) + i) * C::RAW; }
    // Tensor memory: O, and S number b
    static __device__ __forceinline__ uint32_t s_col(int b) { return HD + b * TR; }
    // The S of a segment's tile t, and how often it was used before in the segment. `Uses` keeps the parities of all
    // segments before.
    struct Uses {
        unsigned odd = 0;
        static __device__ __forceinline__ int buffer(int t) { return t % C::NB; }
        __device__ __forceinline__ unsigned parity(int t) const { return (odd >> buffer(t) ^ t / C::NB) & 1; }
        __device__ __forceinline__ void end(int T)
        {
#pragma unroll
            for (int b = 0; b < C::NB; ++b) odd ^= ((unsigned)(T + C::NB - 1 - b) / C::NB & 1) << b;
        }
    };
    // A place in a ring of n tiles, and the parity of what is waited for there
    struct Ring {
        int at;
        unsigned phase;
        __device__ __forceinline__ void next(int n)
        {
            if (++at == n) {
                at = 0;
                phase ^= 1;
            }
        }
    };

    // By a whole warp, every lane for itself: one lane's wait that the others are told of takes 330 cycles even where there
    // is nothing to wait for, this 40. Gives up after some 2^31 cycles, a second or more; the abort flag then ends
    // every wait of the block, no more tiles are asked for, and the warps run through what is left and write nothing: no
    // branch around what follows, which would keep it out of the uniform registers. (The joining kernel does not know and joins
    // what the workspace holds; the error word tells.) LAZY: a wait that is seldom short and may end some 100 cycles late; what it
    // executes meanwhile is not taken from the scheduler's other warps. LIMIT: its logarithm, in cycles.
    template <bool LAZY = false, int LIMIT = 31>
    __device__ __forceinline__ void wait(uint32_t bar, unsigned parity)
    {
        if (!bar_try(bar, parity)) {
            const long long t0 = clock64();
#pragma unroll 1
            while (true) {
                bool done = false;
#pragma unroll 1
                for (int i = 0; i < 64 && !done; ++i) {
                    if (LAZY) __nanosleep(32);
                    done = bar_try(bar, parity);
                }
                if (done || flags()[1]) break;
                if (clock64() - t0 > (1ll << LIMIT)) {
                    flags()[1] = 1;
                    atomicOr(a.err, kErrPipelineTimeout);
                    break;
                }
            }
        }
        __syncwarp();
    }
    __device__ __forceinline__ bool ended() const { return __any_sync(0xffffffffu, flags()[1]); }
    // All warps of the softmax
    unsigned meetings = 0;
    __device__ __forceinline__ void group_sync(bool lazy = false)
    {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) bar_arrive(met());
        const unsigned parity = meetings++ & 1;
        // warps without a slot wait for all of the block's work on a sequence, which may take seconds; those that do it give up
        // for them too
        if (lazy) wait<true, 38>(met(), parity);
        else wait(met(), parity);
    }

    __device__ __forceinline__ TileInfo *tile_info(unsigned count) { return reinterpret_cast<TileInfo *>(smem + C::OFF_DESC) + (count & (kTreeDesc - 1)); }

    // The block's unit: its KV head, and the first of its slots
    __device__ __forceinline__ int hk() const { return blockIdx.x % a.n_kv_head; }
    __device__ __forceinline__ int first_slot() const { return blockIdx.x / a.n_kv_head * kTreeSlots; }

    // First row that is not masked; not below 0, so that differences to rows fit into 32 bits
    __device__ __forceinline__ int start_of(int s) const { return a.starts ? max(ld_dep(a.starts + s), 0) : 0; }

    // Rows of a sequence that some node may see: [low, high)
    __device__ __forceinline__ int low_of(int base, int start) const
    {
        return max(max(start, a.window > 0 ? base - a.window + 1 : 0), 0);
    }
    __device__ __forceinline__ int tiles_of(int n, int nkv, int start) const
    {
        if (n <= 0) return 0;
        const int lo = min(low_of(nkv - n, start), nkv) / TR;
        return max((nkv + TR - 1) / TR - lo, 1);
    }

    // The segment that begins at tile p (of the block's, up to `end`), and the tile behind it.
    __device__ __forceinline__ int segment(int p, int end, TreeSeg &g) const
    {
        int lo = 0, hi = a.n_seq - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (before()[mid + 1] > p) hi = mid;
            else lo = mid + 1;
        }
        g.s = lo;
        g.tok0 = tok()[lo];
        g.n = tok()[lo + 1] - g.tok0;
        g.nkv = rows()[lo];
        g.base = g.nkv - g.n;
        g.start = start_of(lo);
        g.T = before()[lo + 1] - before()[lo];
        g.t0 = p - before()[lo];
        g.t1 = min(g.T, g.t0 + end - p);
        g.slots = min(g.n * a.group - first_slot(), kTreeSlots);
        g.row0 = min(low_of(g.base, g.start), g.nkv) / TR * TR;
        return p + g.t1 - g.t0;
    }

    // -----------------------------------------------------------------------
    // Rows, tiles and places of every sequence, and the block's tiles; by one warp. A sequence's tiles have a place each, and
    // kTreeTurn places lie between one sequence and the next: what a block spends on another sequence (its Q, its output, the
    // pipeline's filling) is the time of as many tiles. (Without them, 4 sequences in blocks of 13 tiles: those with
    // two of the sequences took 60 thousand cycles, the others 42.)
    // -----------------------------------------------------------------------
    __device__ __forceinline__ void count(int lane)
    {
        constexpr int MOST = kTreeSeqs / 32;
        const int per = (a.n_seq + 31) / 32;
        int tiles[MOST], sum = 0, there = 0;                   // there: sequences with tiles
#pragma unroll
        for (int i = 0; i < MOST; ++i) {
            tiles[i] = 0;
            const int s = lane * per + i;
            if (i >= per || s >= a.n_seq) continue;
            const int pos = ld_dep(a.positions + s);
            int64_t c0 = (int64_t)(a.seq0 + s) * a.n_each, c1 = c0 + a.n_each;
            if (a.cu) {
                c0 = min(max((int64_t)ld_dep(a.cu + s), (int64_t)0), a.n_tokens);
                c1 = min(max((int64_t)ld_dep(a.cu + s + 1), (int64_t)0), a.n_tokens);
            }
            const int start = start_of(s);
            int n = (int)max(c1 - c0, (int64_t)0);
            tok()[s] = (int)c0;
            if (s == a.n_seq - 1) tok()[s + 1] = (int)max(c1, c0);
            const bool report = (blockIdx.x | blockIdx.y) == 0;
            if (n > a.max_nodes) {
                if (report) atomicOr(a.err, kErrBadTree);
                n = 0;
            }
            if (n > 0 && (pos < -1 || pos >= a.cap) && report) atomicOr(a.err, kErrPositionClamped);
            const int nkv = min(max(pos, -1), a.cap - 1) + 1;
            rows()[s] = nkv;
            if (n * a.group > first_slot()) tiles[i] = tiles_of(n, nkv, start);
            sum += tiles[i];
            there += tiles[i] > 0;
        }
        int upto = sum, seqs = there;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, off), z = __shfl_up_sync(0xffffffffu, seqs, off);
            if (lane >= off) {
                upto += y;
                seqs += z;
            }
        }
        const int total = __shfl_sync(0xffffffffu, upto, 31), turns = max(__shfl_sync(0xffffffffu, seqs, 31) - 1, 0);
        int at = upto - sum, turn = seqs - there;
#pragma unroll
        for (int i = 0; i < MOST; ++i) {
            const int s = lane * per + i;
            if (i >= per || s >= a.n_seq) continue;
            before()[s] = at;
            place()[s] = at + turn * kTreeTurn;
            at += tiles[i];
            turn += tiles[i] > 0;
        }
        const int places = total + turns * kTreeTurn, share = max((places + a.ranks - 1) / a.ranks, 2);   // a tile for each warpgroup
        if (lane == 0) {
            before()[a.n_seq] = total;
            flags()[2] = share;
        }
        __syncwarp();
        if (lane < 2) {                                        // tiles before the block's first place, and the one behind its last
            const int64_t p = (int64_t)(blockIdx.y + lane) * share;
            int x = total;
            if (p < places) {
                int lo = 0, hi = a.n_seq - 1;                  // the last sequence whose place is at most p (0: the first)
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (place()[mid] <= p) lo = mid;
                    else hi = mid - 1;
                }
                x = min(before()[lo] + max((int)p - place()[lo], 0), before()[lo + 1]);
            }
            flags()[3 + lane] = x;
        }
    }

    // -----------------------------------------------------------------------
    // Producer warps, one of K and one of V: pages, copies; K's writes the tiles' descriptors.
    // -----------------------------------------------------------------------
    template <bool V>
    __device__ __forceinline__ void produce(const CUtensorMap *map, int from, int end, int lane)
    {
        constexpr bool CONV = V ? C::E8 : C::KCONV;
        constexpr int NC = C::E8 ? C::RNCH : C::NCH, CB = C::E8 ? C::RCHB : 128, CW = C::E8 ? C::RCHB : 64;
        // lines that no other block reads are the first that L2 gives up
        uint64_t policy;
        if (a.once) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
        else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
        Ring ring{0, 1};                          // it is free at first
        const int n = CONV ? (V ? a.nrv : a.nrk) : (V ? a.nv : a.nk);
        unsigned tiles = 0;                       // before the segment
        const int BR = a.box_rows, lt = lane / C::NSLC, ls = lane % C::NSLC;
        const bool leads = (ls & (BR / 16 - 1)) == 0;         // the first slice of a box
        constexpr unsigned TILE_BITS = (1u << C::NSLC) - 1u;
        for (int p = from; p < end;) {
            TreeSeg g;
            p = segment(p, end, g);
            const int T = g.t1 - g.t0, low = low_of(g.base, g.start);
            const int32_t *table = a.table + (size_t)g.s * a.max_pages;
            // lane l has slice l % NSLC of tile l / NSLC of a group: its page (-2: nothing of its box is seen)
            const int row0 = g.row0 + (g.t0 + lt) * TR + ls * 16;
            auto page_of = [&](int grp) {
                const int r = row0 + grp * (C::TPG * TR), box = r & -BR;
                return grp * C::TPG + lt < T && box < g.nkv && box + BR > low ? ld_dep(table + div(a.by_page, r)) : -2;
            };
            auto scale_of = [&](int page) {
                float2 f = make_float2(1.f, 1.f);
                if (C::E8 && !V && (unsigned)page < (unsigned)a.n_pages) {
                    f.x = ld_dep(a.k_scale + (size_t)page * a.n_kv_head + hk());
                    f.y = ld_dep(a.v_scale + (size_t)page * a.n_kv_head + hk());
                }
                return f;
            };
            // pages are asked for two groups ahead, scales one
            int cur = page_of(0), next = page_of(1), far = page_of(2);
            float2 f = scale_of(cur), fnext = scale_of(next);
#pragma unroll 1
            for (int t0 = 0, grp = 0; t0 < T; t0 += C::TPG, ++grp) {
                const bool there = (unsigned)cur < (unsigned)a.n_pages;
                const unsigned slices = __ballot_sync(0xffffffffu, there), boxes = __ballot_sync(0xffffffffu, there && leads);
                const int r = row0 + grp * (C::TPG * TR), z = r - div(a.by_page, r) * a.page_size;
                const unsigned negative = V ? 0u : __ballot_sync(0xffffffffu, f.x < 0.f);
                const int count = min(C::TPG, T - t0);
#pragma unroll 1
                for (int i = 0; i < count; ++i) {
                    wait<true>(CONV ? raw(V, ring.at) : empty(V, ring.at), ring.phase);
                    if (ended()) return;
                    const unsigned mine = slices >> (i * C::NSLC) & TILE_BITS;
                    if (lt == i) {                             // a lane for each box
                        if (there && leads) {
                            const uint32_t to = (CONV ? raw_slot(V, ring.at) : V ? v_slot(ring.at) : k_slot(ring.at)) + ls * 16 * CB;
#pragma unroll
                            for (int c = 0; c < NC; ++c) tree_tma(to + c * (TR * CB), map, full(V, ring.at), c * CW, hk(), z, cur, policy);
                        }
                        if (!V) {
                            // the copies are on their way; the tile is whole once lane 0 has arrived too
                            if (cur != -2 && !there) atomicOr(a.err, kErrBadPage);
                            TileInfo *d = tile_info(tiles + i);
                            d->ks[ls] = f.x;
                            d->vs[ls] = f.y;
                            d->lv[ls] = (float)min(max((int)(__float_as_uint(f.y) >> 23 & 0xFFu) - 126, -60), 61);   // its exponent field
                            if (ls == 0) {
                                const int seen_lo = max(g.start, a.window > 0 ? g.base + a.max_nodes - a.window : 0);
                                d->row0 = r;
                                d->edge = (r < seen_lo || r + TR > g.base || mine != TILE_BITS ? 1 : 0) |
                                          (negative >> (i * C::NSLC) & TILE_BITS ? 2 : 0);
                                d->slices = mine;
                                d->live = g.nkv - r;
                            }
                        }
                    }
                    __syncwarp();
                    if (!V && lane == 0) bar_arrive(described(tiles + i));
                    if (lane == 0)
                        bar_arrive_expect_tx(full(V, ring.at), __popc(boxes >> (i * C::NSLC) & TILE_BITS) * (unsigned)BR * HD * (C::E8 ? 1 : 2));
                    ring.next(n);
                }
                tiles += count;
                cur = next;
                f = fnext;
                next = far;
                far = page_of(grp + 3);
                fnext = scale_of(next);
            }
        }
    }

    // -----------------------------------------------------------------------
    // Four warps that make tiles ready for the tensor cores: of V, and of K where it is converted.
    // -----------------------------------------------------------------------
    // A tile of codes to f16. A thread's units of 16 codes: one column, rows RSTEP (a multiple of 8) apart, so that the swizzle
    // is the same for all; their loads go out before the first conversion.
    static constexpr int UPR = HD / 16, RSTEP = 128 / UPR, NU = TR / RSTEP;
    template <bool V>
    __device__ __forceinline__ void convert(Ring &rr, Ring &sr, int tid)
    {
        constexpr int N = NU;
        // lanes of odd chunks take the next row of a pair: their units fall into other banks than those of the even ones
        const int u = tid % UPR, c = u >> 2, v = (u & 3) * 2, r = tid / UPR ^ (c & 1);
        wait<true>(full(V, rr.at), rr.phase);
        uint32_t src = raw_slot(V, rr.at);
        if constexpr (C::RCHB == 128) src += (u >> 3) * (TR * 128) + r * 128 + ((u ^ r) & 7) * 16;
        else src += r * 64 + (((u ^ (r >> 1)) & 3) << 4);
        uint4 x[N];
#pragma unroll
        for (int k = 0; k < N; ++k) x[k] = lds128(src + k * RSTEP * C::RCHB);
        wait<true>(empty(V, sr.at), sr.phase);
        const uint32_t dst = (V ? v_slot(sr.at) : k_slot(sr.at)) + c * (TR * 128) + r * 128;
        const uint32_t dst0 = dst + ((v ^ (r & 7)) << 4), dst1 = dst + (((v + 1) ^ (r & 7)) << 4);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            uint4 y0, y1;
            e4m3x4_to_half4(x[k].x, y0.x, y0.y);
            e4m3x4_to_half4(x[k].y, y0.z, y0.w);
            e4m3x4_to_half4(x[k].z, y1.x, y1.y);
            e4m3x4_to_half4(x[k].w, y1.z, y1.w);
            sts128(dst0 + k * RSTEP * 128, y0);
            sts128(dst1 + k * RSTEP * 128, y1);
        }
    }

    __device__ __forceinline__ void fix(int from, int end, int tid)
    {
        const int lane = tid & 31;
        Ring vr{0, 0}, vs{0, C::E8 ? 1u : 0u}, kr{0, 0}, ks{0, 1};
        unsigned tiles = 0, segs = 0;
        auto key = [&] {                                       // K of the next tile
            convert<false>(kr, ks, tid);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                bar_arrive(raw(false, kr.at));
                bar_arrive(ready(false, ks.at));
            }
            kr.next(a.nrk);
            ks.next(a.nk);
        };
        for (int p = from; p < end; ++segs) {
            TreeSeg g;
            p = segment(p, end, g);
            const int T = g.t1 - g.t0;
            // K as far before V as S may be before P V
            const int ahead = C::KCONV ? min(a.nk, C::NB) - 1 : 0;
#pragma unroll 1
            for (int t = -ahead; t < T; ++t) {
                if (C::KCONV && t + ahead < T) key();
                if (t < 0) continue;
                if constexpr (C::E8) {
                    convert<true>(vr, vs, tid);
                } else {
                    wait<true>(full(true, vs.at), vs.phase);
                }
                wait(described(tiles), tiles / kTreeDesc & 1);
                TileInfo *d = tile_info(tiles);
                const bool look = static_cast<volatile TileInfo *>(d)->edge & 1;
                if (look) {                                    // the units that this thread has written, where it has
                    const int u = tid % UPR * 2;
                    const uint32_t to = v_slot(vs.at) + (u >> 3) * (TR * 128);
                    bool wild = false;
#pragma unroll 1
                    for (int r = tid / UPR ^ (u >> 3 & 1); r < TR; r += RSTEP) {
                        const uint32_t p0 = to + r * 128 + (((u ^ r) & 7) << 4), p1 = to + r * 128 + ((((u + 1) ^ r) & 7) << 4);
                        uint4 y0 = lds128(p0), y1 = lds128(p1);
                        if (clean(d, r, y0, y1, wild)) {
                            sts128(p0, y0);
                            sts128(p1, y1);
                        }
                    }
                    // before V is ready, behind whose products the softmax looks
                    if (wild) atomicOr(reinterpret_cast<unsigned *>(const_cast<int *>(flags())) + 5, 1u << (segs & 31));
                }
                if (C::E8 || look) fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (C::E8) bar_arrive(raw(true, vr.at));
                    bar_arrive(ready(true, vs.at));
                }
                if (C::E8) vr.next(a.nrv);
                vs.next(a.nv);
                ++tiles;
            }
        }
    }

    // Sixteen elements of V of tile row r: what belongs to no row of the sequence, and infinities and NaN, become 0.
    // Whether anything changed; wild: whether there was an infinity or NaN.
    static __device__ __forceinline__ bool clean(const TileInfo *d, int r, uint4 &y0, uint4 &y1, bool &wild)
    {
        const volatile TileInfo *vd = d;
        if (r >= vd->live || !(vd->slices >> (r >> 4) & 1)) {
            y0 = y1 = make_uint4(0u, 0u, 0u, 0u);
            return true;
        }
        constexpr uint32_t EXP = std::is_same<MT, __half>::value ? 0x7C00u : 0x7F80u;
        uint32_t *w[8] = {&y0.x, &y0.y, &y0.z, &y0.w, &y1.x, &y1.y, &y1.z, &y1.w};
        bool found = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t keep = 0xffffffffu;
            if ((*w[i] & EXP) == EXP) keep &= 0xffff0000u;
            if ((*w[i] >> 16 & EXP) == EXP) keep &= 0x0000ffffu;
            found = found || keep != 0xffffffffu;
            *w[i] &= keep;
        }
        wild = wild || found;
        return found;
    }

    // -----------------------------------------------------------------------
    // Issuers, one of S = Q K^T and one of O += P V: warps, so that what is the same in all lanes (descriptors, addresses)
    // stays in uniform registers; one lane issues. (One warp for both was what the tensor cores waited for:
    // 2000 cycles a tile, half of them for barriers.)
    // -----------------------------------------------------------------------
    __device__ __forceinline__ void issue_s(uint32_t tm_any, int from, int end)
    {
        const uint32_t tm = __shfl_sync(0xffffffffu, tm_any, 0);
        const uint32_t one = elect_one();
        Ring kr{0, 0};
        unsigned segs = 0, used = 0;                           // used: bit b, whether S number b was used an odd number of times
        constexpr uint32_t id_s = C::F8 ? 1u << 4 | (uint32_t)(TR >> 3) << 17 | 8u << 24 : umma_idesc<MT>(128, TR, 0, 0);
        // rows of 128 bytes (swizzle 2, 8 rows 1024 bytes apart) or 64 (8-bit, head_dim 64: 4, 512)
        constexpr uint32_t SW = C::F8 && HD == 64 ? 4 : 2, SBO = SW == 4 ? 512 : 1024;
        constexpr int KK = C::F8 ? HD / 32 : HD / 16;          // steps of 32 bytes of a row
        const uint64_t q0 = umma_desc(sm, 16, SBO, SW), k0 = umma_desc(k_slot(0), 16, SBO, SW);
        for (int p = from; p < end;) {
            TreeSeg g;
            p = segment(p, end, g);
            const int T = __shfl_sync(0xffffffffu, g.t1 - g.t0, 0);
            wait<true>(q_ready(), segs++ & 1);
            int b = 0;
#pragma unroll 1
            for (int t = 0; t < T; ++t) {
                wait(C::KCONV ? ready(false, kr.at) : full(false, kr.at), kr.phase);
                // S goes over the P of a product that may still read it
                wait(o_done(b), ~used >> b & 1);
                used ^= 1u << b;
                tc_fence_after();
                const uint64_t k = k0 + (uint32_t)kr.at * (C::KSLOT >> 4);
                const uint32_t d = tm + s_col(b);
                // the last part first: a sum is cut off at 24 bits at each step, of which those of the small parts cost nothing then
                uint64_t q = q0 + (a.q_parts - 1) * (C::QPART >> 4);
#pragma unroll 1
                for (int x = 0; x < a.q_parts; ++x) {
#pragma unroll
                    for (int kk = 0; kk < KK; ++kk)
                        umma_ss<C::F8>(one, d, q + ((kk >> 2) * 16384 + (kk & 3) * 32) / 16, k + ((kk >> 2) * (TR * 128) + (kk & 3) * 32) / 16,
                                       id_s, x + kk > 0);
                    q -= C::QPART >> 4;
                }
                bar_commit(one, s_full(b));
                if (++b == C::NB) b = 0;
                bar_commit(one, empty(false, kr.at));
                kr.next(a.nk);
            }
        }
    }
    __device__ __forceinline__ void issue_o(uint32_t tm_any, int from, int end)
    {
        const uint32_t tm = __shfl_sync(0xffffffffu, tm_any, 0);
        const uint32_t one = elect_one();
        Ring vr{0, 0};
        unsigned used = 0;
        constexpr uint32_t id_o = umma_idesc<MT>(128, HD, 0, 1);
        const uint64_t v0 = umma_desc(v_slot(0), TR * 128, 1024, 2);
        for (int p = from; p < end;) {
            TreeSeg g;
            p = segment(p, end, g);
            const int T = __shfl_sync(0xffffffffu, g.t1 - g.t0, 0);
            int b = 0;
#pragma unroll 1
            for (int t = 0; t < T; ++t) {
                wait(ready(true, vr.at), vr.phase);
                wait(p_ready(b), used >> b & 1);
                used ^= 1u << b;
                tc_fence_after();
                const uint64_t v = v0 + (uint32_t)vr.at * (C::SLOT >> 4);
                const uint32_t s = tm + s_col(b);
#pragma unroll
                for (int kk = 0; kk < TR / 16; ++kk)
#pragma unroll
                    for (int x = 0; x < PP; ++x) umma_ts(one, tm, s + 32 * (kk >> 1) + 16 * x + 8 * (kk & 1), v + kk * 128, id_o);
                bar_commit(one, o_done(b));
                if (++b == C::NB) b = 0;
                bar_commit(one, empty(true, vr.at));
                vr.next(a.nv);
            }
        }
    }

    // -----------------------------------------------------------------------
    // Softmax warpgroup w: one slot a thread.
    // -----------------------------------------------------------------------
    struct Row {
        int t;                // node; -1: no slot
        int h;                // head
        int x;                // position
        float c;              // a score's factor (1 / q's scale, scale log2 e or scale / softcap)
    };
    __device__ __forceinline__ int64_t place_of(const TreeSeg &g, const Row &r) const   // of q and the output, in rows of HD
    {
        return (int64_t)(g.tok0 + r.t) * a.n_head + r.h;
    }

    __device__ __forceinline__ int depth_of(const TreeSeg &g, int t) const
    {
        return a.depths ? min(max(ld_dep(a.depths + g.tok0 + t), 0), a.max_nodes - 1) : t;
    }

    // Q of the warpgroup's slots: parts, K-major, swizzled; returns what undoes the power of two of the thread's row.
    // The rows are copied as they are, 16 bytes a lane, to where their parts will stand -- a row of
    // float is as long as its two 16-bit parts, one of 16 bits as one of those or as two 8-bit ones -- and a thread then
    // turns its own row into its parts, in place. Each of the two warpgroups copies every other 32 units and turns every other
    // unit of a row.
    __device__ __forceinline__ uint32_t q_place(int row, int part, int u) const
    {
        const uint32_t to = sm + (uint32_t)part * C::QPART;
        if (C::F8 && HD == 64) return to + row * 64 + (((u ^ (row >> 1)) & 3) << 4);
        return to + (u >> 3) * 16384 + row * 128 + (((u ^ row) & 7) << 4);
    }
    // One part of q's own type: copied only
    __device__ __forceinline__ bool as_it_is() const
    {
        return !C::F8 && PARTS == 1 && a.q_type == (std::is_same<MT, __half>::value ? kTypeF16 : kTypeBf16);
    }
    // Whether the thread's row of such a Q is finite
    __device__ __forceinline__ bool finite_q(int my) const
    {
        uint32_t m = 0;
#pragma unroll 4
        for (int u = 0; u < HD / 8; ++u) {
            const uint4 x = lds128(q_place(my, 0, u));
            m = __vmaxu2(__vmaxu2(m, x.x & 0x7fff7fffu), __vmaxu2(__vmaxu2(x.y & 0x7fff7fffu, x.z & 0x7fff7fffu), x.w & 0x7fff7fffu));
        }
        return max(m >> 16, m & 0xffffu) < (std::is_same<MT, __half>::value ? 0x7C00u : 0x7F80u);
    }
    __device__ __forceinline__ float stage_q(const TreeSeg &g, const Row &r, int w, int quad, int lane)
    {
        const int my = quad * 32 + lane;
        const bool f32 = a.q_type == kTypeF32, f16 = std::is_same<MT, __half>::value;
        const int lg = (HD == 64 ? 3 : HD == 128 ? 4 : 5) + f32, last = (1 << lg) - 1;   // log2 of a row's 16-byte units
        const int rows = min(max(g.slots - quad * 32, 0), 32);
        const int mine_at = r.t * a.n_head + r.h;                     // after the sequence's first token
        const uint8_t *src = static_cast<const uint8_t *>(a.q) + ((int64_t)g.tok0 * a.n_head << lg) * 16;
#pragma unroll 1
        for (int it = w; it * 32 < rows << lg; it += 2) {
            const int i = it * 32 + lane, row = i >> lg, u = i & last;
            const int at = __shfl_sync(0xffffffffu, mine_at, row);
            const uint32_t to = f32 || C::F8 ? q_place(quad * 32 + row, u & 1, u >> 1) : q_place(quad * 32 + row, 0, u);
            if (row < rows)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                             :: "r"(to), "l"(src + (((int64_t)at << lg) + u) * 16) : "memory");
        }
        asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
        group_sync();
        if (as_it_is()) return 1.f;
        const bool bf = a.q_type == kTypeBf16;
        const int mine = r.t >= 0 ? HD / 8 : 0;                       // units of 8 elements
        float sc = 1.f, inv = 1.f;
        if (f16) {
            // the largest magnitude, by the bits: they order as the numbers do
            uint32_t m = 0;
            if (f32) {
#pragma unroll 4
                for (int u = 0; u < 2 * mine; ++u) {
                    const uint4 x = lds128(q_place(my, u & 1, u >> 1));
                    m = max(max(m, x.x & 0x7fffffffu), max(max(x.y & 0x7fffffffu, x.z & 0x7fffffffu), x.w & 0x7fffffffu));
                }
            } else {
#pragma unroll 4
                for (int u = 0; u < mine; ++u) {
                    const uint4 x = lds128(C::F8 ? q_place(my, u & 1, u >> 1) : q_place(my, 0, u));
                    m = __vmaxu2(__vmaxu2(m, x.x & 0x7fff7fffu), __vmaxu2(__vmaxu2(x.y & 0x7fff7fffu, x.z & 0x7fff7fffu), x.w & 0x7fff7fffu));
                }
                m = max(m >> 16, m & 0xffffu);
                m = bf ? m << 16 : __float_as_uint(kv2_to_float2<__half>(m).x);
            }
            pow2_scale(__uint_as_float(m), sc, inv);
            if (C::F8) {                                              // 2^7 .. 2^8: e4m3 ends at 448
                sc *= 0.0078125f;
                inv *= 128.f;
            }
            // a row with an infinity or NaN: every score NaN (8-bit parts end at 448, and one 16-bit part of -inf hides rows)
            if (m >= 0x7f800000u) inv = __uint_as_float(0x7fffffffu);
        }
        group_sync();                                                 // the other warpgroup has read the row too
        auto pair_of = [&](uint32_t w) {                              // two elements, scaled
            const float2 x = bf ? kv2_to_float2<__nv_bfloat16>(w) : kv2_to_float2<__half>(w);
            return make_float2(x.x * sc, x.y * sc);
        };
        if constexpr (C::F8) {
#pragma unroll 1
            for (int u = w; u < mine / 2; u += 2) {       // 16 elements
                const uint4 x = lds128(q_place(my, 0, u)), y = lds128(q_place(my, 1, u));
                const uint32_t in[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
                __half2 h[8];                                         // exact: 11 bits, and 2^8 is far from f16's limits
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 f = pair_of(in[e]);
                    h[e] = __floats2half2_rn(f.x, f.y);
                }
#pragma unroll 1
                for (int part = 0; part < a.q_parts; ++part) {
                    uint32_t c[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint16_t lo, hi;
                        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lo) : "r"(*reinterpret_cast<uint32_t *>(&h[2 * e])));
                        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(*reinterpret_cast<uint32_t *>(&h[2 * e + 1])));
                        c[e] = (uint32_t)lo | (uint32_t)hi << 16;
                        uint32_t b0, b1;
                        e4m3x4_to_half4(c[e], b0, b1);
                        h[2 * e] = __hsub2(h[2 * e], *reinterpret_cast<__half2 *>(&b0));
                        h[2 * e + 1] = __hsub2(h[2 * e + 1], *reinterpret_cast<__half2 *>(&b1));
                    }
                    sts128(q_place(my, part, u), make_uint4(c[0], c[1], c[2], c[3]));
                }
            }
        } else {
#pragma unroll 1
            for (int u = w; u < mine; u += 2) {
                const uint4 x = lds128(q_place(my, 0, u));
                float2 f[4];
                if (f32) {
                    const uint4 y = lds128(q_place(my, 1, u));
                    f[0] = make_float2(__uint_as_float(x.x) * sc, __uint_as_float(x.y) * sc);
                    f[1] = make_float2(__uint_as_float(x.z) * sc, __uint_as_float(x.w) * sc);
                    f[2] = make_float2(__uint_as_float(y.x) * sc, __uint_as_float(y.y) * sc);
                    f[3] = make_float2(__uint_as_float(y.z) * sc, __uint_as_float(y.w) * sc);
                } else {
                    f[0] = pair_of(x.x);
                    f[1] = pair_of(x.y);
                    f[2] = pair_of(x.z);
                    f[3] = pair_of(x.w);
                }
#pragma unroll
                for (int part = 0; part < PARTS; ++part) {
                    uint32_t h[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        h[e] = float2_to_kv2<MT>(f[e].x, f[e].y);
                        if (part + 1 < PARTS) {
                            const float2 b = kv2_to_float2<MT>(h[e]);
                            f[e].x -= b.x;
                            f[e].y -= b.y;
                        }
                    }
                    sts128(q_place(my, part, u), make_uint4(h[0], h[1], h[2], h[3]));
                }
            }
        }
        return inv;
    }

    // tanh: near 0, |x| < 0.4, its series to x^11 (what follows is below 2^-23 of it); elsewhere 1 - 2 / (1 + e^2x), to 2^-22
    static __device__ __forceinline__ float tanh_of(float x)
    {
        const float e = ex2(2.f * kLog2e * x), z = x * x;
        const float l = e < 1e30f ? fmaf(-2.f, rcp(1.f + e), 1.f) : 1.f;
        float s = -8.8632355e-3f;                              // 1382 / 155925
        s = fmaf(s, z, 2.1869489e-2f);                         // 62 / 2835
        s = fmaf(s, z, -5.3968254e-2f);                        // 17 / 315
        s = fmaf(s, z, 1.3333333e-1f);                         // 2 / 15
        s = fmaf(s, z, -3.3333333e-1f);
        return fabsf(x) < 0.4f ? fmaf(s * z, x, x) : x == x ? l : x;
    }
    // 32 products, 16 with each factor, to capped scores: the series alone, in pairs, where no row with a slot leaves its range
    // (a cap is seldom come near, and nothing is known of rows without a slot)
    __device__ __forceinline__ void cap(const Row &r, uint32_t (&v)[32], float f0, float f1) const
    {
        uint64_t x[16];
        float k = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float f = i < 8 ? f0 : f1;
            x[i] = mul2(pack2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), pack2(f, f));
            const float2 y = unpack2(x[i]);
            k = fmaxf(fmaxf(k, fabsf(y.x)), fabsf(y.y));
        }
        if (__all_sync(0xffffffffu, k < 0.4f || r.t < 0)) {
            auto both = [](float c) { return pack2(c, c); };
            const uint64_t most = both(a.cap_log2);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint64_t z = mul2(x[i], x[i]), y = mul2(x[i], most);
                uint64_t s = fma2(both(-8.8632355e-3f), z, both(2.1869489e-2f));
                s = fma2(s, z, both(-5.3968254e-2f));
                s = fma2(s, z, both(1.3333333e-1f));
                s = fma2(s, z, both(-3.3333333e-1f));
                x[i] = fma2(mul2(s, z), y, y);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 y = unpack2(x[i]);
                x[i] = pack2(a.cap_log2 * tanh_of(y.x), a.cap_log2 * tanh_of(y.y));
            }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 y = unpack2(x[i]);
            v[2 * i] = __float_as_uint(y.x);
            v[2 * i + 1] = __float_as_uint(y.y);
        }
    }

    // Of the 32 rows from j0 on those that the thread's node sees; there: the two 16-row slices of them that are.
    __device__ __forceinline__ unsigned seen_bits(const TreeSeg &g, const Row &r, int j0, unsigned there) const
    {
        if (r.t < 0) return 0u;
        const int y0 = j0 - g.base;
        unsigned bits = bit_range(low_of(r.x, g.start) - j0, g.base - j0);
        if (y0 > -32 && y0 < g.n) {
            unsigned dr;
            if (!a.mask) {
                dr = bit_range(-y0, r.t + 1 - y0);
            } else {
                const int w = y0 >> 5;                         // -1: before the first
                const uint32_t *mask = a.mask + (int64_t)(g.tok0 + r.t) * a.words;
                const uint32_t lo = w >= 0 ? ld_mask(mask, w) : 0u;
                const uint32_t hi = w + 1 < a.words ? ld_mask(mask, w + 1) : 0u;
                dr = __funnelshift_r(lo, hi, y0 & 31);
            }
            dr &= bit_range(max(-y0, g.start - j0), g.n - y0);
            if (a.window > 0 && a.window < a.max_nodes)
                for (unsigned m = dr; m; m &= m - 1) {
                    const int c = __ffs(m) - 1;
                    if (r.x - g.base - depth_of(g, y0 + c) >= a.window) dr &= ~(1u << c);
                }
            bits |= dr;
        }
        return bits & ((there & 1u ? 0xffffu : 0u) | (there & 2u ? 0xffff0000u : 0u));
    }

    // Scores of those 32 with the rules, -inf where the node does not see the row.
    __device__ __forceinline__ void ruled(const TreeSeg &g, const Row &r, const volatile TileInfo *d, int c0, uint32_t (&v)[32]) const
    {
        float f0 = C::E8 ? r.c * d->ks[c0 >> 4] : r.c, f1 = C::E8 ? r.c * d->ks[(c0 >> 4) + 1] : r.c;
        if (a.softcap > 0.f) {
            cap(r, v, f0, f1);
            f0 = f1 = 1.f;
        }
        float s[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) s[c] = __uint_as_float(v[c]) * (c < 16 ? f0 : f1);
        if (a.slopes) {
            const float slope = ld_dep(a.slopes + r.h) * kLog2e;
            const int j0 = d->row0 + c0, y0 = j0 - g.base;
            if (y0 <= -32 || y0 >= g.n) {
                const int x0 = r.x - j0;
#pragma unroll
                for (int c = 0; c < 32; ++c) s[c] = fmaf(-slope, (float)(x0 - c), s[c]);
            } else {
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const int y = y0 + c;
                    s[c] = fmaf(-slope, (float)(r.x - (y < 0 || y >= g.n ? j0 + c : g.base + depth_of(g, y))), s[c]);
                }
            }
        }
        if (d->edge & 1) {
            const unsigned bits = seen_bits(g, r, d->row0 + c0, d->slices >> (c0 >> 4) & 3u);
#pragma unroll
            for (int c = 0; c < 32; ++c) s[c] = bits >> c & 1 ? s[c] : -INFINITY;
        }
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c] = __float_as_uint(s[c]);
    }
    static __device__ __forceinline__ uint32_t ld_mask(const uint32_t *m, int w)
    {
        uint32_t v;
        asm volatile("ld.global.ca.u32 %0, [%1];" : "=r"(v) : "l"(m + w) : "memory");
        return v;
    }

    // O of stream w times f; whole warps.
    __device__ __forceinline__ void scale_o(uint32_t o, float f)
    {
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
            uint32_t v[32];
            tmem_ld32(o + c, v);
            tmem_wait_ld(v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
            tmem_st32(o + c, v);
        }
        tmem_wait_st();
    }

    // At the end of a segment, when its products are done: infinities and NaN that were taken out of V, added to half w of O's
    // dimensions of the slots that see their rows. (A weight changes neither. Where every slot sees a tile they were left in and
    // are in O already; once more is the same.) By a scan of the segment, 32 rows at a time: it is seldom done. (A note of the rows
    // with each tile, for its softmax, needs a wait for V in every tile with an edge: 2 to 4 % of a call.)
    __device__ __forceinline__ void add_wild(const TreeSeg &g, const Row &r, uint32_t o, int w, int lane)
    {
        const uint32_t EXP = C::E8 ? 0x7F7F7F7Fu : std::is_same<MT, __half>::value ? 0x7C007C00u : 0x7F807F80u;
        constexpr int ES = C::E8 ? 1 : 2;
        const int low = low_of(g.base, g.start), end = min(g.row0 + g.t1 * TR, g.nkv);
#pragma unroll 1
        for (int j0 = g.row0 + g.t0 * TR; j0 < end; j0 += 32) {
            const int j = j0 + lane, pg = div(a.by_page, j);
            const int page = j >= low && j < end ? ld_dep(a.table + (size_t)g.s * a.max_pages + pg) : -1;
            const bool there = (unsigned)page < (unsigned)a.n_pages;
            const uint8_t *row = static_cast<const uint8_t *>(a.v) +
                                 (page * a.page_stride + (j - pg * a.page_size) * a.row_stride + hk() * a.head_stride + w * (HD / 2)) * ES;
            bool wild = false;
#pragma unroll 1
            for (int u = 0; there && u < HD / 2 * ES; u += 16) {
                const uint4 x = ld_dep(reinterpret_cast<const uint4 *>(row + u));
                const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    wild = wild || (C::E8 ? __vcmpeq4(y[i] & EXP, EXP) : __vcmpeq2(y[i] & EXP, EXP)) != 0;
            }
            const unsigned seen = seen_bits(g, r, j0, 3u);
            __syncwarp();
#pragma unroll 1
            for (unsigned m = __ballot_sync(0xffffffffu, wild); m; m &= m - 1) {
                const int at = __ffs(m) - 1;
                const uint8_t *from = reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(row), at));
                const bool sees = seen >> at & 1;
#pragma unroll 1
                for (int c = 0; c < HD / 2; c += 32) {
                    uint32_t v[32];
                    tmem_ld32(o + w * (HD / 2) + c, v);
                    tmem_wait_ld(v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float x;
                        if constexpr (C::E8) {
                            uint32_t lo, hi;
                            e4m3x4_to_half4((uint32_t)from[c + i], lo, hi);
                            x = kv2_to_float2<__half>(lo).x;
                        } else {
                            x = kv2_to_float2<MT>((uint32_t)reinterpret_cast<const uint16_t *>(from)[c + i]).x;
                        }
                        if (sees && !(fabsf(x) < INFINITY)) v[i] = __float_as_uint(x + __uint_as_float(v[i]));
                    }
                    __syncwarp();
                    tmem_st32(o + w * (HD / 2) + c, v);
                }
                tmem_wait_st();
            }
        }
    }

    static constexpr float OFF = 7.f;                          // a weight at the reference is 2^7
    __device__ __forceinline__ void softmax(uint32_t tm, int from, int end, int w, int quad, int lane, int rank)
    {
        constexpr float TAU = 8.f;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const int my = quad * 32 + lane;
        volatile float *refs = reinterpret_cast<volatile float *>(smem + C::OFF_REF);
        unsigned tiles = 0, segs = 0, refs_odd = 0;            // tiles and segments before this one; parity of the references handed on
        Uses uses;
        // Over 16-bit caches, tiles with nothing but a cap are capped on their way to weights, others with rules before (31.4 us
        // and not 33.5 for the heads of 256 dimensions above with weights in one part; over e4m3 the branch cost tiles without
        // rules 4 %).
        const bool capped = !C::E8 && a.softcap > 0.f && !a.slopes && a.qscale > 0.f;
        const bool rules = !capped && (a.softcap > 0.f || a.slopes != nullptr || a.qscale <= 0.f);
        for (int p = from; p < end;) {
            TreeSeg g;
            const int next = segment(p, end, g);
            const bool begins = g.t0 == 0, whole = begins && g.t1 == g.T;
            const int T = g.t1 - g.t0, slot = first_slot() + my;
            const uint32_t o_at = tm + lanes;
            Row r;
            r.t = my < g.slots ? div(a.by_group, slot) : -1;
            const bool any = quad * 32 < g.slots;   // some slot in this warp; warps of its group without one
            const int idle = 4 - (g.slots + 31) / 32;
            r.h = hk() * a.group + (r.t >= 0 ? slot - r.t * a.group : 0);
            r.x = g.base + depth_of(g, max(r.t, 0));
            r.c = stage_q(g, r, w, quad, lane) * a.qscale;
            fence_proxy_async_smem();                          // Q is read by the tensor cores
            __syncwarp();                                      // rows without a slot had nothing to turn
            if (any && w == 0) {
                uint32_t z[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) z[i] = 0u;
#pragma unroll 1
                for (int c = 0; c < HD; c += 32) tmem_st32(o_at + c, z);
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(q_ready());
            // while the first S is made (stage_q sees to it where it looks at the row itself)
            if (as_it_is() && r.t >= 0 && !finite_q(my)) r.c = __uint_as_float(0x7fffffffu);

            float m = -INFINITY, l = 0.f, mm = -INFINITY;      // mm: reference of the sums on the way
#pragma unroll 1
            for (int t = w; any && t < T; t += 2) {
                const int b = Uses::buffer(t);
                const uint32_t s_at = tm + s_col(b) + lanes;
                const volatile TileInfo *d = tile_info(tiles + t);
                wait(s_full(b), uses.parity(t));
                tc_fence_after();
                const int edge = __shfl_sync(0xffffffffu, d->edge, 0);
                const bool slow = edge || rules;
                if (slow) {                                    // the rules first
#pragma unroll 1
                    for (int c = 0; c < TR; c += 32) {
                        uint32_t v[32];
                        tmem_ld32(s_at + c, v);
                        tmem_wait_ld(v);
                        ruled(g, r, d, c, v);
                        __syncwarp();
                        tmem_st32(s_at + c, v);
                    }
                    tmem_wait_st();
                }
                // P, by the reference as it is: that of the tile before may be larger by now, which is seen to at the end
                const float c = slow ? 1.f : r.c;
                uint64_t sum[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) sum[i] = pack2(0.f, 0.f);
                auto gather = [&] {
                    const float2 both = unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
                    l += both.x + both.y;
#pragma unroll
                    for (int i = 0; i < 4; ++i) sum[i] = pack2(0.f, 0.f);
                };
                uint32_t u[32], v[32];
                tmem_ld32(s_at, u);
                tmem_ld32(s_at + 32, v);
#pragma unroll 1
                for (int at = 0; at < TR; at += 64) {
                    float f[4], vs[4], k[4];
                    if constexpr (C::E8) {
                        const uint32_t info = sm + C::OFF_DESC + ((tiles + t) & (kTreeDesc - 1)) * 128 + at / 4;
                        const uint4 x = lds128(info + 32), y = lds128(info + 64), z = lds128(info + 96);
                        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w}, zs[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            f[i] = slow ? 1.f : c * __uint_as_float(xs[i]);
                            vs[i] = __uint_as_float(ys[i]);
                            k[i] = __uint_as_float(zs[i]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) f[i] = c, vs[i] = 1.f, k[i] = 0.f;
                    }
                    tmem_wait_ld(u);
                    tmem_wait_ld(v);
                    if (capped && !slow) {
                        cap(r, u, f[0], f[1]);
                        cap(r, v, f[2], f[3]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) f[i] = 1.f;
                    }
                    k[0] = fmaf(most16(u, 0), f[0], k[0]);
                    k[1] = fmaf(most16(u, 16), f[1], k[1]);
                    k[2] = fmaf(most16(v, 0), f[2], k[2]);
                    k[3] = fmaf(most16(v, 16), f[3], k[3]);
                    const float mx = r.t < 0 ? -INFINITY : fmaxf(fmaxf(k[0], k[1]), fmaxf(k[2], k[3]));
                    if (__any_sync(0xffffffffu, mx > m + TAU)) {
                        const float M = mx > m + TAU ? ceilf(mx) : m, fac = M == m ? 1.f : ex2(m - M);   // 0 from -inf
                        gather();
                        l *= fac;
                        m = M;
                        if (at) scale_p(s_at, at, fac);
                    }
                    const float ref = m == -INFINITY ? 0.f : m - OFF;
                    const uint64_t nref = pack2(-ref, -ref);
                    weights(u, s_at + at, nref, f, vs, sum);
                    if (at + 64 < TR) tmem_ld32(s_at + at + 64, u);
                    weights(v, s_at + at + 32, nref, f + 2, vs + 2, sum);
                    if (at + 64 < TR) tmem_ld32(s_at + at + 96, v);
                }
                gather();
                tmem_wait_st();
                // O and P by one reference, the larger
                float mo = m;                                  // O's
                if (t > 0) {
                    wait(ref_known(quad), (refs_odd ^ (t - 1)) & 1);
                    mo = refs[my];
                }
                if (__any_sync(0xffffffffu, m != mo)) {
                    const float M = fmaxf(m, mo), fac = m == M ? 1.f : ex2(m - M);
                    if (__any_sync(0xffffffffu, m != M)) scale_p(s_at, TR, fac);
                    l *= fac;
                    if (__any_sync(0xffffffffu, mo != M)) {
                        wait(o_done(Uses::buffer(t - 1)), uses.parity(t - 1));
                        tc_fence_after();
                        scale_o(o_at, mo == M ? 1.f : fmaxf(ex2(mo - M), 1.17549435e-38f));   // not 0: it may hold infinities
                    }
                    m = M;
                }
                refs[my] = m;
                __syncwarp();
                if (lane == 0) bar_arrive(ref_known(quad));
                if (PARTS == 2 && t > 0 && (t & (a.fold - 1)) == 0) {   // the first warpgroup's
                    wait(o_done(Uses::buffer(t - 1)), uses.parity(t - 1));
                    tc_fence_after();
                    fold(o_at, part_of(rank, begins), my, r.t >= 0, t == a.fold ? -1.f : mm == m ? 1.f : fmaxf(ex2(mm - m), 1.17549435e-38f));
                    mm = m;
                }
                tc_fence_before();
                __syncwarp();
                if (lane <= (quad ? 0 : idle)) bar_arrive(p_ready(b));   // for the warps without a slot too
            }
            // Every product of the segment is done. A barrier's parity tells a phase from those next to it only, so each wait
            // is for one that the warp knows to be the last or the one under way: the warpgroup's own last tile's first
            // (the other's last tile may have used the same S as a product that is still under way, and may be done too).
            if (any && T > 1) wait(o_done(Uses::buffer(T - 2)), uses.parity(T - 2));
            if (any) wait(o_done(Uses::buffer(T - 1)), uses.parity(T - 1));
            uses.end(T);
            if (any) refs_odd ^= T & 1;
            const unsigned wild = 1u << (segs++ & 31);
            const bool is_wild = __any_sync(0xffffffffu, flags()[5] & wild);
            if (is_wild && any && !ended()) {
                tc_fence_after();
                add_wild(g, r, o_at, w, lane);
            }
            // a slot whose every score is NaN keeps its NaN sum
            finish(tm, g, r, w, quad, lane, whole, begins, rank, m == -INFINITY && l != 0.f ? 0.f : m - OFF, l, any,
                   PARTS == 2 && T > a.fold, mm);
            // for the segment 32 behind: V is never that far ahead
            if (is_wild && w == 0 && quad == 0 && lane == 0)
                atomicAnd(reinterpret_cast<unsigned *>(const_cast<int *>(flags())) + 5, ~wild);
            tiles += T;
            p = next;
        }
    }
    // 32 scores to weights, into the same columns; their sums.
    static __device__ __forceinline__ void weights(const uint32_t (&v)[32], uint32_t at, uint64_t nref, const float *f, const float *vs,
                                                   uint64_t (&sum)[4])
    {
        uint32_t h[PP][16];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint64_t f2 = pack2(f[x], f[x]), vs2 = pack2(vs[x], vs[x]);
#pragma unroll
            for (int i = 8 * x; i < 8 * x + 8; ++i) {
                const float2 s = unpack2(fma2(pack2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), f2, nref));
                uint64_t p = pack2(ex2(s.x), ex2(s.y));
                sum[i & 3] = add2(sum[i & 3], p);
                if (C::E8) p = mul2(p, vs2);
                const float2 q = unpack2(p);
                h[0][i] = float2_to_kv2<MT>(q.x, q.y);
                if (PP == 2) {
                    const float2 y = kv2_to_float2<MT>(h[0][i]);
                    h[PP - 1][i] = float2_to_kv2<MT>(q.x - y.x, q.y - y.y);
                }
            }
            if (PP == 2) {                                  // in turn: all of both parts do not fit into the registers
                tmem_st8(at + 8 * x, h[0] + 8 * x);
                tmem_st8(at + 16 + 8 * x, h[PP - 1] + 8 * x);
            }
        }
        if (PP == 1) tmem_st16(at, h[0]);
    }
    // The weights of the first n columns times f, a power of two; whole warps.
    static __device__ __forceinline__ void scale_p(uint32_t s_at, int n, float f)
    {
        const uint32_t f2 = float2_to_kv2<MT>(f, f);
        tmem_wait_st();
#pragma unroll 1
        for (int c = 0; c < n; c += 32) {
            uint32_t v[32];
            tmem_ld32(s_at + c, v);
            tmem_wait_ld(v);
#pragma unroll
            for (int i = 0; i < 16 * PP; ++i) v[i] = mul_kv2<MT>(v[i], f2);
#pragma unroll
            for (int x = 0; x < PP; ++x) tmem_st16(s_at + c + 16 * x, v + 16 * x);
        }
        tmem_wait_st();
    }
    static __device__ __forceinline__ float most16(const uint32_t (&v)[32], int at)
    {
        float k = __uint_as_float(v[at]);
#pragma unroll
        for (int i = 1; i < 15; i += 2) k = fmaxf(fmaxf(k, __uint_as_float(v[at + i])), __uint_as_float(v[at + i + 1]));
        return fmaxf(k, __uint_as_float(v[at + 15]));
    }

    // Place of the block's part of a sequence in the workspace, in slots; of one that it has all of, for sums on the way.
    __device__ __forceinline__ size_t part_of(int rank, bool begins) const
    {
        return ((size_t)(a.ranks == 1 ? 0 : rank * 2 + (begins ? 1 : 0)) * gridDim.x + blockIdx.x) * kTreeSlots;
    }
    // O of the slots to their sums on the way, those times f first (f < 0: there are none yet); O is 0 then.
    __device__ __forceinline__ void fold(uint32_t o, size_t block, int my, bool mine, float f)
    {
        float4 *to = reinterpret_cast<float4 *>(a.ws_o + block * HD) + my;
#pragma unroll 1
        for (int c = 0; c < HD; c += 32, to += 8 * kTreeSlots) {
            uint32_t v[32];
            tmem_ld32(o + c, v);
            float4 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (mine && f >= 0.f) x[i] = ld_dep(to + i * kTreeSlots);
            }
            tmem_wait_ld(v);
            if (mine) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float *y = reinterpret_cast<const float *>(v) + 4 * i;
                    to[i * kTreeSlots] = f < 0.f ? make_float4(y[0], y[1], y[2], y[3])
                                                 : make_float4(fmaf(x[i].x, f, y[0]), fmaf(x[i].y, f, y[1]), fmaf(x[i].z, f, y[2]),
                                                               fmaf(x[i].w, f, y[3]));
                }
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;
            __syncwarp();
            tmem_st32(o + c, v);
        }
        tmem_wait_st();
    }

    // The end of a segment: the output, or the block's part of it; each warpgroup writes half of the dimensions. folded: there are
    // sums on the way, by reference mm (of the first warpgroup).
    __device__ __forceinline__ void finish(uint32_t tm, const TreeSeg &g, const Row &r, int w, int quad, int lane, bool whole,
                                           bool begins, int rank, float m, float l, bool any, bool folded, float mm)
    {
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        tc_fence_after();
        const size_t block = part_of(rank, begins);
        const int in_unit = quad * 32 + lane;
        auto put = [&](int d, const float (&y)[32], float inv) {   // 32 dimensions from d on
            if (r.t < 0) return;
            if (!whole) {
                float4 *o = reinterpret_cast<float4 *>(a.ws_o + block * HD) + (size_t)(d / 4) * kTreeSlots + in_unit;
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i * kTreeSlots] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
            } else if (a.q_type == kTypeF32) {
                float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + place_of(g, r) * HD + d);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i] = make_float4(y[4 * i] * inv, y[4 * i + 1] * inv, y[4 * i + 2] * inv, y[4 * i + 3] * inv);
            } else {
                uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + place_of(g, r) * HD + d);
                const bool h = a.q_type == kTypeF16;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t u[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float y0 = y[8 * i + 2 * e] * inv, y1 = y[8 * i + 2 * e + 1] * inv;
                        u[e] = h ? float2_to_kv2<__half>(y0, y1) : float2_to_kv2<__nv_bfloat16>(y0, y1);
                    }
                    o[i] = make_uint4(u[0], u[1], u[2], u[3]);
                }
            }
        };
        // the other warpgroup's reference and sum, through this thread's lane of tensor memory; O has the larger reference
        const uint32_t box = tm + s_col(0) + lanes;
        if (any) {
            tmem_st2(box + 2 * w, __float_as_uint(m), __float_as_uint(l));
            if (folded && w == 0) tmem_st2(box + 4, __float_as_uint(mm), 0u);
            tmem_wait_st();
        }
        tc_fence_before();
        group_sync(!any);
        tc_fence_after();
        if (any) {
            uint32_t om, ol;
            tmem_ld2(box + 2 * (w ^ 1), om, ol);
            const float m1 = __uint_as_float(om), l1 = __uint_as_float(ol), M = fmaxf(m, m1);
            l = (m == -INFINITY ? 0.f : l * ex2(m - M)) + (m1 == -INFINITY ? 0.f : l1 * ex2(m1 - M));
            m = M;
        }
        float fold_f = 0.f;                                    // what the sums on the way are to be multiplied by
        if (any && folded) {
            uint32_t om, none;
            tmem_ld2(box + 4, om, none);
            mm = __uint_as_float(om) - OFF;
            fold_f = mm == m ? 1.f : fmaxf(ex2(mm - m), 1.17549435e-38f);
        }
        const int d0 = w * (HD / 2), d1 = d0 + HD / 2;
        float f = 1.f;                                         // what O is to be multiplied by
        if (any && !ended()) {
            if (!whole && r.t >= 0 && d0 == 0) a.ws_ml[block + in_unit] = make_float2(m, l);
            if (whole) f = l == 0.f ? 0.f : rcp(l);
            const uint32_t o = tm + lanes;
#pragma unroll 1
            for (int d = d0; d < d1; d += 32) {
                uint32_t u[32];
                tmem_ld32(o + d, u);
                tmem_wait_ld(u);
                float y[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(u[i]);
                if (folded && r.t >= 0) {
                    const float4 *from = reinterpret_cast<const float4 *>(a.ws_o + block * HD) + (size_t)(d / 4) * kTreeSlots + in_unit;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 x = ld_dep(from + i * kTreeSlots);
                        y[4 * i] = fmaf(x.x, fold_f, y[4 * i]);
                        y[4 * i + 1] = fmaf(x.y, fold_f, y[4 * i + 1]);
                        y[4 * i + 2] = fmaf(x.z, fold_f, y[4 * i + 2]);
                        y[4 * i + 3] = fmaf(x.w, fold_f, y[4 * i + 3]);
                    }
                }
                put(d, y, f);
                __syncwarp();
            }
        }
        // the next segment's Q and zeros go over what the other warpgroup reads, and over what its products read
        tc_fence_before();
        group_sync(!any);
        tc_fence_after();
    }
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
attn_tree_stream(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const __grid_constant__ TreeArgs a)
{
    extern __shared__ __align__(1024) uint8_t smem[];      // the swizzle needs the alignment (launch: no static shared memory)
    Tree<C> x(a, smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = blockIdx.y;
    if (warp == C::PROD_K) {
        if (lane == 0) {
            for (int i = 0; i < 32; ++i) bar_init(x.bar(i), i & 4 ? 4 : 1);   // ready and raw: a lane of each converting warp
            for (int i = 0; i < 4; ++i) {
                bar_init(x.s_full(i), 1);
                bar_init(x.p_ready(i), 4);
                bar_init(x.o_done(i), 1);
                bar_init(x.ref_known(i), 1);
            }
            bar_init(x.q_ready(), C::SM_WARPS);
            bar_init(x.met(), C::SM_WARPS);
            for (int i = 0; i < kTreeDesc; ++i) bar_init(x.described(i), 1);
            x.flags()[1] = 0;
            x.flags()[5] = 0;
            fence_barrier_init();
            prefetch_tensormap(&kmap);
            prefetch_tensormap(&vmap);
        }
        __syncwarp();
        pdl_wait();
        x.count(lane);
        if (rank == 0 && x.hk() == 0 && a.ranks > 1) {
            __syncwarp();
            for (int s = lane; s < a.n_seq; s += 32)
                a.ws_span[blockIdx.x / a.n_kv_head * a.n_seq + s] =
                    make_int4(x.place()[s], x.before()[s + 1] - x.before()[s], x.tok()[s], x.flags()[2]);
        }
    } else {
        if (warp == C::MMA_S) tmem_alloc(reinterpret_cast<uint32_t *>(const_cast<int *>(x.flags())), C::TM_COLS);
        pdl_wait();
    }
    pdl_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = (uint32_t)x.flags()[0];
    const int from = x.flags()[3], end = x.flags()[4];
    {
        if (warp < C::SM_WARPS) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    }
    if (warp < C::SM_WARPS) {
        x.softmax(tm, from, end, warp >> 2, warp & 3, lane, rank);
    } else if (warp < C::FIX + 4) {
        x.fix(from, end, tid - C::FIX * 32);
    } else if (warp == C::PROD_K) {
        x.template produce<false>(&kmap, from, end, lane);
    } else if (warp == C::PROD_V) {
        x.template produce<true>(&vmap, from, end, lane);
    } else if (warp == C::MMA_S) {
        x.issue_s(tm, from, end);
    } else if (warp == C::MMA_O) {
        x.issue_o(tm, from, end);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (x.flags()[1]) {                                      // after a timeout: copies and products under way end first
        if (tid == 0) {
            const unsigned long long t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 200000000ull) __nanosleep(1000);
        }
        __syncthreads();
    }
    tc_fence_after();
    if (warp == C::MMA_S) tmem_dealloc(tm, C::TM_COLS);
}

// Units that several blocks have tiles of: o = sum w oc / sum w S over their parts, w = 2^(mx - max mx). A warp takes a
// node, eight heads of a KV head and 16 dimensions: a part's slots lie next to each other for every four
// dimensions, as the threads of the streaming kernel store them, so the lanes read whole sectors.
template <int HD>
__global__ void __launch_bounds__(128) attn_tree_combine(const TreeArgs a)
{
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int gq = (a.group + 7) / 8, per_tok = a.n_kv_head * gq * (HD / 16);
    const int64_t job = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t tk = job / per_tok;
    if (tk >= a.tok_end) return;
    int rest = (int)(job - tk * per_tok);
    const int dq = rest % (HD / 16);
    rest /= HD / 16;
    const int hk = rest / gq, gh = (rest - hk * gq) * 8 + (lane & 7), d4 = dq * 4 + (lane >> 3);
    // its sequence: the last one that begins at or before it, of those that have places
    int s = -1;
    int4 sp = make_int4(0, 0, 0, 0);
    int64_t c1 = 0;                                            // the token behind its last
    for (int i0 = 0; i0 < a.n_seq; i0 += 32) {
        int4 q = make_int4(0, 0, 0x7fffffff, 0);
        int upto = 0;
        if (i0 + lane < a.n_seq) {
            if (a.cu) upto = ld_dep(a.cu + i0 + lane + 1);
            const uint4 u = ld_dep(reinterpret_cast<const uint4 *>(a.ws_span + i0 + lane));
            q = make_int4((int)u.x, (int)u.y, (int)u.z, (int)u.w);
        }
        const unsigned b = __ballot_sync(0xffffffffu, q.y > 0 && q.z <= tk);
        if (b) {
            const int l = 31 - __clz(b);
            s = i0 + l;
            sp = make_int4(__shfl_sync(0xffffffffu, q.x, l), __shfl_sync(0xffffffffu, q.y, l), __shfl_sync(0xffffffffu, q.z, l),
                           __shfl_sync(0xffffffffu, q.w, l));
            c1 = __shfl_sync(0xffffffffu, upto, l);
        }
    }
    if (s < 0) return;
    c1 = a.cu ? min(c1, a.n_tokens) : (int64_t)(a.seq0 + s + 1) * a.n_each;
    if (tk >= c1 || gh >= a.group) return;
    const int slot = (int)(tk - sp.z) * a.group + gh, mu = slot / kTreeSlots;
    if (mu > 0) {                                              // the unit's own places
        const uint4 u = ld_dep(reinterpret_cast<const uint4 *>(a.ws_span + mu * a.n_seq + s));
        sp = make_int4((int)u.x, (int)u.y, 0, (int)u.w);
    }
    const int r0 = sp.x / sp.w, r1 = (sp.x + sp.y - 1) / sp.w;
    if (r0 == r1) return;
    const int unit = mu * a.n_kv_head + hk;
    const int in_unit = slot - mu * kTreeSlots;
    float m = -INFINITY, S = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int BATCH = 8;
    for (int r = r0; r <= r1; r += BATCH) {
        float2 ml[BATCH];
        float4 v[BATCH];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int x = min(r + b, r1);
            const size_t block = ((size_t)(x * 2 + (x == r0 ? 1 : 0)) * a.units + unit) * kTreeSlots;   // it begins in the first one's places
            ml[b] = ld_dep(a.ws_ml + block + in_unit);
            v[b] = ld_dep(reinterpret_cast<const float4 *>(a.ws_o + block * HD) + (size_t)d4 * kTreeSlots + in_unit);
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            if (r + b > r1 || ml[b].x == -INFINITY) continue;
            const float M = fmaxf(m, ml[b].x), f = m == -INFINITY ? 0.f : ex2(m - M), w = ex2(ml[b].x - M);
            S = fmaf(S, f, w * ml[b].y);
            acc.x = fmaf(acc.x, f, w * v[b].x);
            acc.y = fmaf(acc.y, f, w * v[b].y);
            acc.z = fmaf(acc.z, f, w * v[b].z);
            acc.w = fmaf(acc.w, f, w * v[b].w);
            m = M;
        }
    }
    const float inv = S == 0.f ? 0.f : 1.f / S;
    const int64_t at = (tk * a.n_head + hk * a.group + gh) * HD + d4 * 4;
    if (a.q_type == kTypeF32) {
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    } else {
        uint2 u;
        if (a.q_type == kTypeF16) {
            u.x = float2_to_kv2<__half>(acc.x * inv, acc.y * inv);
            u.y = float2_to_kv2<__half>(acc.z * inv, acc.w * inv);
        } else {
            u.x = float2_to_kv2<__nv_bfloat16>(acc.x * inv, acc.y * inv);
            u.y = float2_to_kv2<__nv_bfloat16>(acc.z * inv, acc.w * inv);
        }
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) = u;
    }
}

template <class C>
cudaError_t launch_tree_kernel(const TreeRequest &r)
{
    alignas(64) CUtensorMap kmap, vmap;
    const bool bf = std::is_same<typename C::KV, __nv_bfloat16>::value;
    const int64_t es = C::E8 ? 1 : 2;
    TreeArgs a = r.a;
    a.box_rows = a.page_size % 64 == 0 && C::TR >= 64 ? 64 : a.page_size % 32 == 0 ? 32 : 16;
    const int box_x = C::E8 ? C::RCHB : 64;
    cudaError_t e = encode_paged_map(&kmap, r.k, (int)es, bf, C::HD, a.n_kv_head, a.page_size, a.n_pages, r.head_stride * es,
                                     r.row_stride * es, r.page_stride * es, box_x, a.box_rows);
    if (e != cudaSuccess) return e;
    e = encode_paged_map(&vmap, r.v, (int)es, bf, C::HD, a.n_kv_head, a.page_size, a.n_pages, r.head_stride * es,
                         r.row_stride * es, r.page_stride * es, box_x, a.box_rows);
    if (e != cudaSuccess) return e;
    // 8-bit parts hold 4 bits each: bfloat16 8, binary16 11
    a.q_parts = C::F8 ? (a.q_type == kTypeBf16 ? 2 : 3) : C::PARTS;
    a.q_bytes = (uint32_t)a.q_parts * C::QPART;
    // the rings share what Q leaves
    auto few = [](int x) { return x > 4 ? 4 : x; };
    const uint32_t left = C::DATA - a.q_bytes;
    a.nrk = a.nrv = 0;
    if (C::F8) {
        a.nv = left >= 2 * C::SLOT + 4 * C::RAW ? 2 : 1;
        const int raws = (int)((left - a.nv * C::SLOT) / C::RAW);
        a.nk = few(raws / 2);
        a.nrv = few(raws - a.nk);
    } else if (C::E8) {
        a.nk = left >= 5 * C::SLOT ? 2 : 1;                           // K of a tile is converted before V of the one before
        a.nv = left >= 8 * C::SLOT ? 2 : 1;
        a.nrk = a.nrv = few((int)((left - (a.nk + a.nv) * C::SLOT) / (2 * C::RAW)));
        if (a.nk + a.nrk > 4) a.nrk = 4 - a.nk;
    } else {
        const int n = (int)(left / C::SLOT);
        a.nk = few((n + (n == 3)) / 2);
        a.nv = few(n - a.nk);
    }
    const void *fn = reinterpret_cast<const void *>(&attn_tree_stream<C>);
    e = ensure_smem_attr(fn, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    void *args[] = {&kmap, &vmap, &a};
    e = launch_pdl(fn, dim3((unsigned)a.units, (unsigned)a.ranks), dim3(C::THREADS), C::SMEM, r.stream, args);
    if (e != cudaSuccess || a.ranks == 1) return e;
    const void *cf = reinterpret_cast<const void *>(&attn_tree_combine<C::HD>);
    const int64_t blocks = (a.tok_end * a.n_kv_head * ((a.group + 7) / 8) * (C::HD / 16) + 3) / 4;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    void *cargs[] = {&a};
    return launch_pdl(cf, dim3((unsigned)blocks), dim3(128), 0, r.stream, cargs);
}

template <int HD, typename KV>
cudaError_t launch_tree_for(const TreeRequest &r)
{
    if (r.parts == 2) return launch_tree_kernel<TreeCfg<HD, KV, 2, 2>>(r);
    if constexpr (!std::is_same<KV, E4m3>::value)
        if (r.weight_parts == 2) return launch_tree_kernel<TreeCfg<HD, KV, 1, 2>>(r);
    if constexpr (!std::is_same<KV, __nv_bfloat16>::value)    // bfloat16 queries over a bfloat16 cache take the form above
        return launch_tree_kernel<TreeCfg<HD, KV, 1, 1>>(r);
    return cudaErrorInvalidValue;
}

} // namespace attn
