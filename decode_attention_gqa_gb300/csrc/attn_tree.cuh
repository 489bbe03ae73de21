// attn_tree.cuh -- attention of drafted trees over a paged cache, on the fifth-generation tensor cores.
//
// Mathematics. For a node t at position x over the cache rows j it sees -- all before its tree, and the
// tree's own as its mask has them --
//     s_j = rules(scale q.k_j),  o = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j log2 e - m),
// one pass with a running reference m that moves when a score passes it by 8. An e4m3 cache holds codes
// with one scale per page and KV head: the K scale multiplies a page's scores, the V scale p; the
// reference follows s + log2 of the V scale (rounded up), so that p times the scale stays in the 16-bit
// range whatever the scales are; sum p is f32.
//
// Tiles. A (node, head) pair of a KV head is a slot; 128 slots are the M rows of both products. S = Q K^T
// (128 x TR, operands in shared memory) goes to tensor memory, a warpgroup turns it into P in place, one row a
// thread, so that maxima and sums need no exchange, and O += P V takes P from tensor memory and V as an MN-major
// operand from the tile TMA brought. With more than 128 slots a block serves 256: two tiles of Q, two
// warpgroups, each with its S and O, over the same K and V. With up to 128, the two warpgroups take tiles in
// turn, each with its own (reference, sum, O), joined at the end through tensor memory. Either way the tensor
// cores work for one while the other is at its exponentials. head_dim 256 leaves tensor memory for one O:
// one warpgroup, two S.
//
// Parts. 16-bit queries and weights enter as one operand, f32 queries as two (the rounding, and the rounding of
// what it left), and then the weights too: f16 over f16 and e4m3 caches (rows of q scaled by a power of two, so that nothing is
// lost to f16's range), bf16 over bf16 caches.
//
// Work. The tiles of all units -- (sequence, KV head, 128 or 256 slots) -- are laid end to end, and a block an
// SM takes an equal run of them: what a block has of a unit is its output where it has all of it, else a part
// (reference, sum, sum p v) for attn_tree_combine.
//
// Warps: 8 (4) of the softmax; 4 that convert an e4m3 tile to f16, and, in tiles that some slot does not see all
// of, take infinities and NaN out of V (a weight of 0 would spread them); a producer (pages, TMA); an issuer.
#pragma once

#include <cuda_fp8.h>

#include "attn_device.cuh"
#include "attn_launch.h"
#include "attn_paged.cuh"
#include "attn_paged_launch.h"
#include "attn_partial_umma.cuh"

namespace attn {

constexpr unsigned kErrBadTree = 0x8u;        // ATTN_DEVERR_BAD_REQUEST
constexpr int kTreeDesc = 8;                  // tiles whose descriptors are kept: more than the rings hold

template <int HD_, typename KV_, int PARTS_>
struct TreeCfg {
    static constexpr int HD = HD_, PARTS = PARTS_;
    using KV = KV_;
    using MT = typename PagedMma<KV>::T;
    static constexpr bool E8 = std::is_same<KV, E4m3>::value;
    static constexpr int NS = HD == 256 ? 1 : 2;               // warpgroups at the softmax
    static constexpr int TR = HD == 256 ? 64 : 128;            // cache rows of a tile
    static constexpr int NSLC = TR / 16;                       // 16-row slices
    static constexpr int TPG = 32 / NSLC;                      // tiles whose pages a warp looks up at once
    static constexpr int SM_WARPS = 4 * NS, FIX = SM_WARPS, PROD = FIX + 4, MMA = PROD + 1;
    static constexpr int THREADS = (MMA + 1) * 32;
    static constexpr int NCH = HD / 64;                        // 128-byte chunks of a 16-bit row
    static constexpr uint32_t QPART = 128u * HD * 2;           // a part of a tile of Q
    static constexpr uint32_t SLOT = (uint32_t)TR * HD * 2;    // K or V of a tile, 16 bits
    static constexpr uint32_t RAW = (uint32_t)TR * HD;         // 8 bits
    static constexpr int RCHB = HD < 128 ? HD : 128, RNCH = HD / RCHB;   // chunks of an 8-bit row
    static constexpr uint32_t TM_S = 0, TM_O = 2 * TR, TM_COLS = 512;
    static constexpr uint32_t DATA = 224 * 1024;               // Q and the rings
    static constexpr uint32_t OFF_DESC = DATA;
    static constexpr uint32_t OFF_BAR = OFF_DESC + kTreeDesc * 96;
    static constexpr int NBAR = 8 + 8 + 8 + 8 + 2 + 2 + 2 + 1;
    static constexpr uint32_t OFF_FLAG = OFF_BAR + NBAR * 8;   // TMEM slot, abort, share, total
    static constexpr uint32_t OFF_SEQ = OFF_FLAG + 16;         // before, first token, rows
    static constexpr uint32_t SMEM = OFF_SEQ + (3 * kPagedSeqs + 2) * 4;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(2 * TR + NS * HD <= 512, "tensor memory");
};

struct __align__(16) TileInfo {
    int row0;                 // its first cache row
    int edge;                 // some slot does not see all of it
    unsigned slices;          // 16-row slices that are there
    int live;                 // rows of it that belong to the sequence
    unsigned bad[4];          // rows with an infinity or NaN in V that was taken out (edge tiles)
    float ks[8], vs[8];
};
static_assert(sizeof(TileInfo) == 96, "its place in shared memory");

// A block's share of a unit: sequence s, KV head hk, slots from m * 128 NS.. on; tiles [t0, t1) of its T
struct TreeSeg {
    int s, hk, m, t0, t1, T;
    int n, tok0, nkv, base, start;
    int slots;                // of the unit, at most 256
    bool pair;                // more than 128: both warpgroups on every tile
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
__device__ __forceinline__ void tmem_st2(uint32_t t, uint32_t a, uint32_t b)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" :: "r"(t), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void tmem_ld2(uint32_t t, uint32_t &a, uint32_t &b)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=r"(a), "=r"(b) : "r"(t) : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D += A B with A in tensor memory; issued by one thread.
__device__ __forceinline__ void umma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, 0, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d), "r"(a), "l"(b), "r"(idesc) : "memory");
}

__device__ __forceinline__ void sts128(uint32_t p, const uint4 &v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" :: "r"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
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
    static constexpr int HD = C::HD, PARTS = C::PARTS, TR = C::TR, NS = C::NS;
    using MT = typename C::MT;

    const TreeArgs &a;
    uint8_t *smem;
    uint32_t sm;
    uint64_t *full, *empty, *ready, *raw_free;   // rings: full: TMA's; ready: converted or looked at; empty, raw_free: to be filled
    uint64_t *s_full, *p_ready, *o_done, *q_ready;
    volatile int *flags;                         // [0] TMEM address, [1] abort, [2] share, [3] total
    int *before, *tok, *rows;
    int nslot, nraw;
    uint32_t off_slot, off_raw;

    __device__ __forceinline__ Tree(const TreeArgs &args, uint8_t *base) : a(args), smem(base)
    {
        sm = smem_u32(smem);
        full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
        ready = full + 8;
        empty = ready + 8;
        raw_free = empty + 8;
        s_full = raw_free + 8;
        p_ready = s_full + 2;
        o_done = p_ready + 2;
        q_ready = o_done + 2;
        flags = reinterpret_cast<volatile int *>(smem + C::OFF_FLAG);
        before = reinterpret_cast<int *>(smem + C::OFF_SEQ);
        tok = before + kPagedSeqs + 1;
        rows = tok + kPagedSeqs + 1;
        nslot = a.nslot;
        nraw = a.nraw;
        off_slot = (uint32_t)(a.unit_slots / 128) * PARTS * C::QPART;
        off_raw = off_slot + nslot * C::SLOT;
    }

    __device__ __forceinline__ bool wait(uint64_t *bar, unsigned parity)
    {
        if (mbar_wait_bounded(bar, parity)) return true;
        flags[1] = 1;
        atomicOr(a.err, kErrPipelineTimeout);
        return false;
    }
    // by a whole warp
    __device__ __forceinline__ bool wait_warp(uint64_t *bar, unsigned parity)
    {
        return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
    }

    __device__ __forceinline__ TileInfo *tile_info(unsigned count) { return reinterpret_cast<TileInfo *>(smem + C::OFF_DESC) + (count & (kTreeDesc - 1)); }

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

    // The segment that begins at place p (of the block's, up to `end`), and the place behind it.
    __device__ __forceinline__ int segment(int p, int end, TreeSeg &g) const
    {
        int lo = 0, hi = a.n_seq - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (before[mid + 1] > p) hi = mid;
            else lo = mid + 1;
        }
        g.s = lo;
        g.tok0 = tok[lo];
        g.n = tok[lo + 1] - g.tok0;
        g.nkv = rows[lo];
        g.base = g.nkv - g.n;
        g.start = a.starts ? ld_dep(a.starts + lo) : 0;
        const int all = g.n * a.group, units = (all + a.unit_slots - 1) / a.unit_slots;
        g.T = (before[lo + 1] - before[lo]) / (units * a.n_kv_head);
        const int x = p - before[lo], u = x / g.T;
        g.t0 = x - u * g.T;
        g.t1 = min(g.T, g.t0 + end - p);
        g.hk = u / units;
        g.m = u - g.hk * units;
        g.slots = min(all - g.m * a.unit_slots, a.unit_slots);
        g.pair = NS == 2 && g.slots > 128;
        g.row0 = min(low_of(g.base, g.start), g.nkv) / TR * TR;
        return p + g.t1 - g.t0;
    }

    // -----------------------------------------------------------------------
    // Rows, tiles and places of every sequence; by one warp.
    // -----------------------------------------------------------------------
    __device__ __forceinline__ void count(int lane)
    {
        constexpr int MOST = kPagedSeqs / 32;
        const int per = (a.n_seq + 31) / 32;
        int places[MOST], sum = 0;
#pragma unroll
        for (int i = 0; i < MOST; ++i) {
            places[i] = 0;
            const int s = lane * per + i;
            if (i >= per || s >= a.n_seq) continue;
            const int pos = ld_dep(a.positions + s);
            int64_t c0 = (int64_t)(a.seq0 + s) * a.n_each, c1 = c0 + a.n_each;
            if (a.cu) {
                c0 = min(max((int64_t)ld_dep(a.cu + s), (int64_t)0), a.n_tokens);
                c1 = min(max((int64_t)ld_dep(a.cu + s + 1), (int64_t)0), a.n_tokens);
            }
            const int start = a.starts ? ld_dep(a.starts + s) : 0;
            int n = (int)max(c1 - c0, (int64_t)0);
            tok[s] = (int)c0;
            if (s == a.n_seq - 1) tok[s + 1] = (int)max(c1, c0);
            const bool report = blockIdx.x == 0;
            if (n > a.max_nodes) {
                if (report) atomicOr(a.err, kErrBadTree);
                n = 0;
            }
            if (n > 0 && (pos < -1 || pos >= a.cap) && report) atomicOr(a.err, kErrPositionClamped);
            const int nkv = min(max(pos, -1), a.cap - 1) + 1;
            rows[s] = nkv;
            const int units = (n * a.group + a.unit_slots - 1) / a.unit_slots * a.n_kv_head;
            places[i] = tiles_of(n, nkv, start) * units;
            sum += places[i];
        }
        int upto = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += y;
        }
        const int total = __shfl_sync(0xffffffffu, upto, 31);
        int at = upto - sum;
#pragma unroll
        for (int i = 0; i < MOST; ++i) {
            const int s = lane * per + i;
            if (i >= per || s >= a.n_seq) continue;
            before[s] = at;
            at += places[i];
        }
        if (lane == 0) {
            before[a.n_seq] = total;
            flags[2] = max((total + a.ranks - 1) / a.ranks, a.min_share);
            flags[3] = total;
        }
    }

    // K and V of tiles in the order in which the tensor cores first need them: with `lag` 1 K of the next tile
    // before V of this one.
    struct Order {
        int T, lag, m, v;
        __device__ __forceinline__ Order(const TreeSeg &g) : T(g.t1 - g.t0), lag(g.pair ? 0 : 1), m(0), v(0) {}
        // is_v, tile (from 0); false: no more
        __device__ __forceinline__ bool next(bool &is_v, int &tile)
        {
            while (m < T + lag) {
                if (v == 0) {
                    v = 1;
                    if (m < T) {
                        is_v = false;
                        tile = m;
                        return true;
                    }
                }
                v = 0;
                const int x = m++ - lag;
                if (x >= 0) {
                    is_v = true;
                    tile = x;
                    return true;
                }
            }
            return false;
        }
    };

    // -----------------------------------------------------------------------
    // Producer warp: pages, descriptors, copies.
    // -----------------------------------------------------------------------
    __device__ __forceinline__ void produce(const CUtensorMap *kmap, const CUtensorMap *vmap, int from, int end, int lane)
    {
        // lines that no other block reads are the first that L2 gives up
        uint64_t policy;
        if (a.once) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
        else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
        const int nring = C::E8 ? nraw : nslot;
        uint64_t *free = C::E8 ? raw_free : empty;
        int ring = 0;
        unsigned phase = 1;                       // the ring is free at first
        unsigned tiles = 0;                       // before the segment
        const int BR = a.box_rows, per_box = BR / 16;
        const int lt = lane / C::NSLC, ls = lane % C::NSLC;
        for (int p = from; p < end;) {
            TreeSeg g;
            p = segment(p, end, g);
            const int T = g.t1 - g.t0, low = low_of(g.base, g.start);
            const int32_t *table = a.table + (size_t)g.s * a.max_pages;
            // lane l has slice l % NSLC of tile l / NSLC of a group; -2: nothing of its box is seen
            auto page_of = [&](int grp) {
                const int t = grp * C::TPG + lt, r = g.row0 + (g.t0 + t) * TR + ls * 16, box = r & -BR;
                return t < T && box < g.nkv && box + BR > low ? ld_dep(table + div(a.by_page, r)) : -2;
            };
            auto scale_of = [&](int page) {
                float2 f = make_float2(1.f, 1.f);
                if (C::E8 && (unsigned)page < (unsigned)a.n_pages) {
                    f.x = ld_dep(a.k_scale + (size_t)page * a.n_kv_head + g.hk);
                    f.y = ld_dep(a.v_scale + (size_t)page * a.n_kv_head + g.hk);
                }
                return f;
            };
            // pages are asked for two groups ahead, scales one
            int prev = -2, cur = page_of(0), next = page_of(1), far = page_of(2), grp = 0;
            float2 f = scale_of(cur), fnext = scale_of(next);
            const int seen_lo = max(g.start, a.window > 0 ? g.base + a.max_nodes - a.window : 0);
            // A tile's descriptor goes over that of the tile kTreeDesc before it, whose V has left the rings.
            auto describe = [&](int tile) {
                const bool there = (unsigned)cur < (unsigned)a.n_pages;
                const unsigned mine = __ballot_sync(0xffffffffu, there) >> (lt * C::NSLC) & ((1u << C::NSLC) - 1u);
                if (lt != tile % C::TPG) return;
                if (cur != -2 && !there) atomicOr(a.err, kErrBadPage);
                TileInfo *d = tile_info(tiles + tile);
                d->ks[ls] = f.x;
                d->vs[ls] = f.y;
                if (ls == 0) {
                    const int r = g.row0 + (g.t0 + tile) * TR;
                    d->row0 = r;
                    d->edge = r < seen_lo || r + TR > g.base || mine != (1u << C::NSLC) - 1u;
                    d->slices = mine;
                    d->live = g.nkv - r;
                    d->bad[0] = d->bad[1] = d->bad[2] = d->bad[3] = 0u;
                }
            };
            Order order(g);
            bool is_v;
            int tile;
            while (order.next(is_v, tile)) {
                if (!is_v && tile / C::TPG != grp) {          // V of the tile before may still need the last group's
                    ++grp;
                    prev = cur;
                    cur = next;
                    f = fnext;
                    next = far;
                    far = page_of(grp + 2);
                    fnext = scale_of(next);
                }
                const int src = tile / C::TPG == grp ? cur : prev;
                int pages[C::NSLC];
#pragma unroll
                for (int i = 0; i < C::NSLC; ++i) pages[i] = __shfl_sync(0xffffffffu, src, tile % C::TPG * C::NSLC + i);
                bool ok = true;
                unsigned bytes = 0;
                if (lane == 0) {
                    ok = wait(free + ring, phase);
                    if (ok) {
                        uint8_t *to = smem + (C::E8 ? off_raw + ring * C::RAW : off_slot + ring * C::SLOT);
                        const CUtensorMap *map = is_v ? vmap : kmap;
                        constexpr int NC = C::E8 ? C::RNCH : C::NCH, CB = C::E8 ? C::RCHB : 128, CW = C::E8 ? C::RCHB : 64;
                        const int r0 = g.row0 + (g.t0 + tile) * TR;
#pragma unroll
                        for (int i = 0; i < C::NSLC; ++i) {
                            if (i % per_box != 0 || (unsigned)pages[i] >= (unsigned)a.n_pages) continue;
                            const int r = r0 + i * 16, z = r - div(a.by_page, r) * a.page_size;
                            bytes += (unsigned)BR * HD * (C::E8 ? 1 : 2);
#pragma unroll
                            for (int c = 0; c < NC; ++c)
                                tma_load_4d_once(to + c * (TR * CB) + i * 16 * CB, map, full + ring, c * CW, g.hk, z, pages[i], policy);
                        }
                    }
                }
                if (!__shfl_sync(0xffffffffu, (int)ok, 0)) return;
                // the copies are on their way; the tile is whole once this thread has arrived too
                if (!is_v) describe(tile);
                __syncwarp();
                if (lane == 0) mbar_arrive_expect_tx(full + ring, bytes);
                if (++ring == nring) {
                    ring = 0;
                    phase ^= 1;
                }
            }
            tiles += T;
        }
    }

    // -----------------------------------------------------------------------
    // Four warps that make a tile ready for the tensor cores.
    // -----------------------------------------------------------------------
    __device__ __forceinline__ void fix(int from, int end, int tid)
    {
        int ring = 0, slot = 0;
        unsigned phase = 0, sphase = 1, tiles = 0;
        const int lane = tid & 31;
        for (int p = from; p < end;) {
            TreeSeg g;
            p = segment(p, end, g);
            Order order(g);
            bool is_v;
            int tile;
            while (order.next(is_v, tile)) {
                if (!wait_warp(full + (C::E8 ? ring : slot), C::E8 ? phase : sphase ^ 1)) return;
                TileInfo *d = tile_info(tiles + tile);
                const volatile TileInfo *vd = d;
                const bool look = is_v && vd->edge;
                const uint32_t to = sm + off_slot + slot * C::SLOT;
                if constexpr (C::E8) {
                    if (!wait_warp(empty + slot, sphase)) return;
                    const uint32_t raw = sm + off_raw + ring * C::RAW;
                    constexpr int UPR = HD / 16;               // 16-byte units of a raw row
#pragma unroll 4
                    for (int i = tid; i < TR * UPR; i += 128) {
                        const int r = i / UPR, u = i % UPR;
                        uint32_t src;
                        if constexpr (C::RCHB == 128) src = raw + (u >> 3) * (TR * 128) + r * 128 + ((u ^ r) & 7) * 16;
                        else src = raw + r * 64 + (((u ^ (r >> 1)) & 3) << 4);
                        const uint4 x = lds128(src);
                        uint4 y0, y1;
                        e4m3x4_to_half4(x.x, y0.x, y0.y);
                        e4m3x4_to_half4(x.y, y0.z, y0.w);
                        e4m3x4_to_half4(x.z, y1.x, y1.y);
                        e4m3x4_to_half4(x.w, y1.z, y1.w);
                        if (look) clean(d, r, y0, y1);
                        const int c = u >> 2, v = (u & 3) * 2;
                        const uint32_t dst = to + c * (TR * 128) + r * 128;
                        // lanes of odd chunks write their second unit first: other banks than the even ones
                        const bool odd = c & 1;
                        sts128(dst + (((v + odd) ^ (r & 7)) << 4), odd ? y1 : y0);
                        sts128(dst + (((v + !odd) ^ (r & 7)) << 4), odd ? y0 : y1);
                    }
                    fence_proxy_async_smem();
                } else if (look) {
                    for (int i = tid; i < TR * (HD / 16); i += 128) {
                        const int r = i % TR, u = i / TR * 2;
                        const uint32_t at = to + (u >> 3) * (TR * 128) + r * 128;
                        const uint32_t p0 = at + ((u & 7 ^ (r & 7)) << 4), p1 = at + (((u + 1) & 7 ^ (r & 7)) << 4);
                        uint4 y0 = lds128(p0), y1 = lds128(p1);
                        if (clean(d, r, y0, y1)) {
                            sts128(p0, y0);
                            sts128(p1, y1);
                        }
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) {
                    if (C::E8) mbar_arrive(raw_free + ring);
                    mbar_arrive(ready + slot);
                }
                if (C::E8 && ++ring == nraw) {
                    ring = 0;
                    phase ^= 1;
                }
                if (++slot == nslot) {
                    slot = 0;
                    sphase ^= 1;
                }
            }
            tiles += g.t1 - g.t0;
        }
    }

    // Sixteen elements of V of tile row r: what belongs to no row of the sequence, and infinities and NaN, become 0.
    // Whether anything changed.
    static __device__ __forceinline__ bool clean(TileInfo *d, int r, uint4 &y0, uint4 &y1)
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
        if (found) atomicOr(&d->bad[r >> 5], 1u << (r & 31));
        return found;
    }

    // -----------------------------------------------------------------------
    // Issuer: one thread.
    // -----------------------------------------------------------------------
    __device__ __forceinline__ void issue(uint32_t tm, int from, int end)
    {
        int slot = 0;
        unsigned phase = 0, cnt[2] = {0, 0}, done[2] = {0, 0}, segs = 0;   // items whose S, whose P V was issued, by stream
        auto take = [&](int &got) {                            // the next entry of the ring
            if (!wait(ready + slot, phase)) return false;
            got = slot;
            if (++slot == nslot) {
                slot = 0;
                phase ^= 1;
            }
            return true;
        };
        constexpr uint32_t id_s = umma_idesc<MT>(128, TR, 0, 0), id_o = umma_idesc<MT>(128, HD, 0, 1);
        auto scores = [&](int qt, int b, int ks) {
            const uint32_t k = sm + off_slot + ks * C::SLOT, q = sm + (uint32_t)qt * PARTS * C::QPART;
            tc_fence_after();
#pragma unroll
            for (int x = 0; x < PARTS; ++x)
#pragma unroll
                for (int kk = 0; kk < HD / 16; ++kk)
                    umma_f16(tm + C::TM_S + b * TR, umma_desc(q + x * C::QPART + (kk >> 2) * 16384 + (kk & 3) * 32, 16, 1024, 2),
                             umma_desc(k + (kk >> 2) * (TR * 128) + (kk & 3) * 32, 16, 1024, 2), id_s, x + kk > 0);
            umma_commit(s_full + b);
        };
        auto values = [&](int w, int b, int vs) {
            const uint32_t v = sm + off_slot + vs * C::SLOT;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < TR / 16; ++kk)
#pragma unroll
                for (int x = 0; x < PARTS; ++x)
                    umma_f16_ts(tm + C::TM_O + w * HD, tm + C::TM_S + b * TR + 32 * (kk >> 1) + 16 * x + 8 * (kk & 1),
                                umma_desc(v + kk * 2048, TR * 128, 1024, 2), id_o);
            umma_commit(o_done + b);
        };
        for (int p = from; p < end;) {
            TreeSeg g;
            p = segment(p, end, g);
            if (!wait(q_ready, segs++ & 1)) return;
            const int T = g.t1 - g.t0, items = g.pair ? 2 * T : T;
            int kslot = 0, vslot = 0, pw = 0, pb = 0;
            for (int i = 0; i <= items; ++i) {
                int w = 0, b = 0;
                if (i < items) {
                    w = NS == 2 ? i & 1 : 0;
                    b = NS == 2 ? w : (int)(cnt[0] & 1);
                    if (!(g.pair && w == 1) && !take(kslot)) return;
                    scores(g.pair ? w : 0, b, kslot);
                    if (!g.pair || w == 1) umma_commit(empty + kslot);
                }
                if (i > 0) {                                   // the item before
                    if (!wait(p_ready + pb, NS == 2 ? done[pw] & 1 : done[0] >> 1 & 1)) return;
                    if (!(g.pair && pw == 1) && !take(vslot)) return;
                    values(pw, pb, vslot);
                    if (!g.pair || pw == 1) umma_commit(empty + vslot);
                    ++done[pw];
                }
                if (i < items) {
                    pw = w;
                    pb = b;
                    ++cnt[w];
                }
            }
        }
    }

    // -----------------------------------------------------------------------
    // Softmax warpgroup w: one slot a thread.
    // -----------------------------------------------------------------------
    struct Row {
        int t;                // node; -1: no slot
        int x, low;           // position, first context row it sees
        float c;              // a score's factor (1 / q's scale, scale log2 e or scale / softcap)
        float slope;
        const uint32_t *mask;
        int64_t at;           // of the output, in rows of HD
    };

    __device__ __forceinline__ int depth_of(const TreeSeg &g, int t) const
    {
        return a.depths ? min(max(ld_dep(a.depths + g.tok0 + t), 0), a.max_nodes - 1) : t;
    }

    // Q of the warp's 32 slots: parts, K-major, swizzled. Every lane keeps its slot's factor.
    __device__ __forceinline__ float stage_q(const TreeSeg &g, int w, int quad, int lane)
    {
        const int qt = g.pair ? w : 0, first = g.m * a.unit_slots + qt * 128 + quad * 32;
        const int count = min(max(g.slots - qt * 128 - quad * 32, 0), 32);
        const uint32_t to = sm + (uint32_t)qt * PARTS * C::QPART + quad * 32 * 128;
        const bool both = NS == 1 || g.pair;                   // else a warpgroup writes every other row
        constexpr int E = HD / 32;                             // elements of a lane: 2, 4, 8
        constexpr int B = E == 8 ? 4 : 8;                      // rows on their way at a time
        float inv = 1.f;
#pragma unroll 1
        for (int i0 = 0; i0 < count; i0 += B) {
            float f[B][E];
#pragma unroll
            for (int y = 0; y < B; ++y) {
                const int i = min(i0 + y, count - 1), slot = first + i, t = div(a.by_group, slot);
                const int64_t row = ((int64_t)(g.tok0 + t) * a.n_head + g.hk * a.group + slot - t * a.group) * HD + lane * E;
                load_q<E>(row, f[y]);
            }
#pragma unroll
            for (int y = 0; y < B; ++y) {
                const int i = i0 + y;
                if (i >= count) break;
                float m = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) m = fmaxf(m, fabsf(f[y][e]));
                m = warp_max(m);
                float sc, iv;
                if (std::is_same<MT, __half>::value) {
                    pow2_scale(m, sc, iv);
                } else {
                    sc = iv = 1.f;
                }
                if (lane == i) inv = iv;
                if (!both && (i & 1) != w) continue;
#pragma unroll
                for (int e = 0; e < E; ++e) f[y][e] *= sc;
                const int d = lane * E, u = d >> 3;            // 16-byte unit of the row
                const uint32_t at = to + (u >> 3) * 16384 + i * 128 + (((u & 7) ^ (i & 7)) << 4) + (d & 7) * 2;
#pragma unroll
                for (int x = 0; x < PARTS; ++x) {
                    uint32_t h[E / 2];
#pragma unroll
                    for (int e = 0; e < E / 2; ++e) {
                        h[e] = float2_to_kv2<MT>(f[y][2 * e], f[y][2 * e + 1]);
                        if (x + 1 < PARTS) {
                            const float2 b = kv2_to_float2<MT>(h[e]);
                            f[y][2 * e] -= b.x;
                            f[y][2 * e + 1] -= b.y;
                        }
                    }
                    if constexpr (E == 2) asm volatile("st.shared.u32 [%0], %1;" :: "r"(at + x * C::QPART), "r"(h[0]) : "memory");
                    else if constexpr (E == 4) asm volatile("st.shared.v2.u32 [%0], {%1, %2};" :: "r"(at + x * C::QPART), "r"(h[0]), "r"(h[1]) : "memory");
                    else sts128(at + x * C::QPART, make_uint4(h[0], h[1], h[2], h[3]));
                }
            }
        }
        return inv;
    }

    template <int E>
    __device__ __forceinline__ void load_q(int64_t i, float (&f)[E]) const
    {
        if (a.q_type == kTypeF32) {
            const float *p = static_cast<const float *>(a.q) + i;
            if constexpr (E == 2) {
                const float2 v = ld_dep(reinterpret_cast<const float2 *>(p));
                f[0] = v.x; f[1] = v.y;
            } else {
#pragma unroll
                for (int e = 0; e < E; e += 4) {
                    const float4 v = ld_dep(reinterpret_cast<const float4 *>(p + e));
                    f[e] = v.x; f[e + 1] = v.y; f[e + 2] = v.z; f[e + 3] = v.w;
                }
            }
        } else {
            const uint16_t *p = static_cast<const uint16_t *>(a.q) + i;
            uint32_t r[E / 2];
            if constexpr (E == 2) {
                r[0] = (uint32_t)ld_dep(reinterpret_cast<const int *>(p));
            } else if constexpr (E == 4) {
                asm volatile("ld.global.cg.v2.u32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "l"(p) : "memory");
            } else {
                const uint4 v = ld_dep(reinterpret_cast<const uint4 *>(p));
                r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
            }
#pragma unroll
            for (int e = 0; e < E / 2; ++e) {
                const float2 v = a.q_type == kTypeF16 ? kv2_to_float2<__half>(r[e]) : kv2_to_float2<__nv_bfloat16>(r[e]);
                f[2 * e] = v.x;
                f[2 * e + 1] = v.y;
            }
        }
    }

    // Scores of 32 columns from tile row c0 on, with the rules, -inf where the slot does not see the row.
    __device__ __forceinline__ void ruled(const TreeSeg &g, const Row &r, const volatile TileInfo *d, int c0, uint32_t (&v)[32])
    {
        const int j0 = d->row0 + c0, y0 = j0 - g.base;
        unsigned bits = bit_range(r.low - j0, g.base - j0);
        if (r.t >= 0 && y0 > -32 && y0 < g.n) {
            unsigned dr;
            if (!r.mask) {
                dr = bit_range(-y0, r.t + 1 - y0);
            } else {
                const int w = y0 >> 5;                         // -1: before the first
                const uint32_t lo = w >= 0 ? ld_mask(r.mask, w) : 0u;
                const uint32_t hi = w + 1 < a.words ? ld_mask(r.mask, w + 1) : 0u;
                dr = __funnelshift_r(lo, hi, y0 & 31);
            }
            dr &= bit_range(max(-y0, g.start - j0), g.n - y0) & bit_range(-j0, 32);
            if (a.window > 0 && a.window < a.max_nodes)
                for (unsigned m = dr; m; m &= m - 1) {
                    const int c = __ffs(m) - 1;
                    if (r.x - g.base - depth_of(g, y0 + c) >= a.window) dr &= ~(1u << c);
                }
            bits |= dr;
        }
        if (r.t < 0) bits = 0u;
        const unsigned there = d->slices >> (c0 >> 4) & 3u;
        bits &= (there & 1u ? 0xffffu : 0u) | (there & 2u ? 0xffff0000u : 0u);
#pragma unroll
        for (int c = 0; c < 32; ++c) {
            float s = __uint_as_float(v[c]) * (C::E8 ? r.c * d->ks[(c0 >> 4) + (c >> 4)] : r.c);
            if (a.softcap > 0.f) s = a.cap_log2 * tanhf(s);
            if (a.slopes) {
                const int y = y0 + c;
                const int x = y < 0 || y >= g.n ? j0 + c : g.base + depth_of(g, y);
                s = fmaf(-r.slope, (float)(r.x - x), s);
            }
            v[c] = __float_as_uint(bits >> c & 1 ? s : -INFINITY);
        }
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
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
            tmem_st32(o + c, v);
        }
        tmem_wait_st();
    }

    // Rows of V that hold infinities or NaN: to the slots that see them, in the dimensions that do.
    __device__ __noinline__ void add_bad(const TreeSeg &g, const volatile TileInfo *d, uint32_t s_at, uint32_t o, float ref)
    {
        for (int w = 0; w < (TR + 31) / 32; ++w)
            for (unsigned m = d->bad[w]; m; m &= m - 1) {
                const int r = w * 32 + __ffs(m) - 1, j = d->row0 + r, pg = div(a.by_page, j);
                const int page = ld_dep(a.table + (size_t)g.s * a.max_pages + pg);
                const int64_t at = page * a.page_stride + (j - pg * a.page_size) * a.row_stride + g.hk * a.head_stride;
                uint32_t sv, dummy;
                tmem_ld2(s_at + (r & ~1), sv, dummy);
                if (r & 1) sv = dummy;
                const float s = __uint_as_float(sv), p = ex2(s - ref);
                const bool sees = s != -INFINITY;
                for (int c = 0; c < HD; c += 32) {
                    uint32_t v[32];
                    tmem_ld32(o + c, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float x;
                        if constexpr (C::E8) {
                            uint32_t lo, hi;
                            e4m3x4_to_half4((uint32_t)static_cast<const uint8_t *>(a.v)[at + c + i], lo, hi);
                            x = kv2_to_float2<__half>(lo).x;
                        } else {
                            x = kv2_to_float2<MT>((uint32_t)static_cast<const uint16_t *>(a.v)[at + c + i]).x;
                        }
                        if (sees && !(fabsf(x) < INFINITY)) v[i] = __float_as_uint(fmaf(p, x, __uint_as_float(v[i])));
                    }
                    tmem_st32(o + c, v);
                }
                tmem_wait_st();
            }
    }

    __device__ __forceinline__ void softmax(uint32_t tm, int from, int end, int w, int quad, int lane, int rank)
    {
        constexpr float TAU = 8.f, OFF = 7.f;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t o_at = tm + C::TM_O + w * HD + lanes;
        bool dead = false;
        unsigned cnt = 0, tiles = 0;                           // items of this stream; tiles before the segment
        const bool rules = a.softcap > 0.f || a.slopes != nullptr;
        for (int p = from; p < end;) {
            TreeSeg g;
            const int next = segment(p, end, g);
            const bool begins = g.t0 == 0, whole = begins && g.t1 == g.T;
            const int qt = g.pair ? w : 0;
            const int in_unit = qt * 128 + quad * 32 + lane, slot = g.m * a.unit_slots + in_unit;
            Row r;
            r.t = in_unit < g.slots ? div(a.by_group, slot) : -1;
            const bool any = qt * 128 + quad * 32 < g.slots;   // some slot in this warp
            {
                const float inv = any ? stage_q(g, w, quad, lane) : 1.f;
                const int t = max(r.t, 0), h = g.hk * a.group + (r.t >= 0 ? slot - t * a.group : 0);
                r.x = g.base + depth_of(g, t);
                r.low = max(low_of(r.x, g.start), 0);
                r.c = inv * a.qscale;
                r.slope = a.slopes ? ld_dep(a.slopes + h) * kLog2e : 0.f;
                r.mask = a.mask ? a.mask + (int64_t)(g.tok0 + t) * a.words : nullptr;
                r.at = (int64_t)(g.tok0 + t) * a.n_head + h;
            }
            fence_proxy_async_smem();                          // Q is read by the tensor cores
            if (any) {
                uint32_t z[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) z[i] = 0u;
#pragma unroll 1
                for (int c = 0; c < HD; c += 32) tmem_st32(o_at + c, z);
                tmem_wait_st();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_ready);

            float m = -INFINITY, l = 0.f;
            const int step = NS == 2 && !g.pair ? 2 : 1;
            for (int t = g.pair || NS == 1 ? 0 : w; t < g.t1 - g.t0; t += step) {
                const int b = NS == 2 ? w : (int)(cnt & 1);
                const unsigned par = NS == 2 ? cnt & 1 : cnt >> 1 & 1;
                const uint32_t s_at = tm + C::TM_S + b * TR + lanes;
                const volatile TileInfo *d = tile_info(tiles + t);
                if (!dead) dead = !wait_warp(s_full + b, par);
                if (any && !dead) {
                    tc_fence_after();
                    const bool edge = d->edge || rules;
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < TR; c += 32) {
                        uint32_t v[32];
                        tmem_ld32(s_at + c, v);
                        tmem_wait_ld();
                        if (edge) {
                            ruled(g, r, d, c, v);
                            tmem_st32(s_at + c, v);
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float k = -INFINITY;
                            if (edge || !C::E8) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) k = fmaxf(k, __uint_as_float(v[16 * h + i]));
                                if (!edge) k = r.c >= 0.f ? k * r.c : lowest(v, h) * r.c;
                            } else {
                                const float f = r.c * d->ks[(c >> 4) + h];
#pragma unroll
                                for (int i = 0; i < 16; ++i) k = fmaxf(k, __uint_as_float(v[16 * h + i]) * f);
                            }
                            if (C::E8) {
                                const int e = (int)((__float_as_uint(d->vs[(c >> 4) + h]) >> 23) & 0xFFu) - 126;
                                k += (float)min(max(e, -60), 61);
                            }
                            mx = fmaxf(mx, k);
                        }
                    }
                    if (edge) tmem_wait_st();
                    const bool need = mx > m + TAU;
                    const bool bad = d->edge && (d->bad[0] | d->bad[1] | d->bad[2] | d->bad[3]) != 0u;
                    if (__any_sync(0xffffffffu, need) || bad) {
                        // one S buffer a stream: S is complete, so is what was issued before it; two: O's last product is not
                        if (NS == 1 && cnt > 0 && !wait_warp(o_done + (b ^ 1), (cnt - 1) >> 1 & 1)) dead = true;
                        tc_fence_after();
                        if (!dead && __any_sync(0xffffffffu, need)) {
                            const float f = need ? ex2(m - mx) : 1.f;      // 0 while m is -inf
                            if (need) m = mx;
                            l *= f;
                            scale_o(o_at, f);
                        }
                        if (!dead && bad) add_bad(g, d, s_at, o_at, m == -INFINITY ? 0.f : m - OFF);
                    }
                    const float ref = m == -INFINITY ? 0.f : m - OFF;
#pragma unroll 1
                    for (int c = 0; c < TR; c += 32) {
                        uint32_t v[32];
                        tmem_ld32(s_at + c, v);
                        tmem_wait_ld();
                        float sum = 0.f;
                        uint32_t h[PARTS][16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float f = edge ? 1.f : C::E8 ? r.c * d->ks[(c >> 4) + (i >> 3)] : r.c;
                            float p0 = ex2(fmaf(__uint_as_float(v[2 * i]), f, -ref));
                            float p1 = ex2(fmaf(__uint_as_float(v[2 * i + 1]), f, -ref));
                            sum += p0 + p1;
                            if (C::E8) {
                                const float vs = d->vs[(c >> 4) + (i >> 3)];
                                p0 *= vs;
                                p1 *= vs;
                            }
                            h[0][i] = float2_to_kv2<MT>(p0, p1);
                            if (PARTS == 2) {
                                const float2 q = kv2_to_float2<MT>(h[0][i]);
                                h[PARTS - 1][i] = float2_to_kv2<MT>(p0 - q.x, p1 - q.y);
                            }
                        }
                        l += sum;
#pragma unroll
                        for (int x = 0; x < PARTS; ++x) tmem_st16(s_at + c + 16 * x, h[x]);
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_ready + b);
                ++cnt;
            }
            // a slot whose every score is NaN keeps its NaN sum
            const float mref = m == -INFINITY && l != 0.f ? 0.f : m - OFF;
            finish(tm, g, r, w, quad, lane, cnt, whole, begins, rank, mref, l, any, dead);
            tiles += g.t1 - g.t0;
            p = next;
        }
    }
    static __device__ __forceinline__ float lowest(const uint32_t (&v)[32], int h)
    {
        float k = INFINITY;
#pragma unroll
        for (int i = 0; i < 16; ++i) k = fminf(k, __uint_as_float(v[16 * h + i]));
        return k;
    }

    static __device__ __forceinline__ void group_sync() { asm volatile("bar.sync 1, %0;" :: "r"(C::SM_WARPS * 32) : "memory"); }

    // The end of a segment: the output, or the block's part of it.
    __device__ __forceinline__ void finish(uint32_t tm, const TreeSeg &g, const Row &r, int w, int quad, int lane, unsigned cnt,
                                           bool whole, bool begins, int rank, float m, float l, bool any, bool &dead)
    {
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const bool mine = g.pair || NS == 1 || g.t1 - g.t0 > w;    // this stream had an item
        if (mine && !dead) {
            const unsigned last = cnt - 1;
            dead = !wait_warp(o_done + (NS == 2 ? w : (int)(last & 1)), NS == 2 ? last & 1 : last >> 1 & 1);
        }
        tc_fence_after();
        const size_t part = (size_t)(rank * 2 + (begins ? 1 : 0)) * a.unit_slots + (g.pair ? w : 0) * 128 + quad * 32 + lane;
        auto put = [&](int d, const float (&y)[32], float inv) {   // 32 dimensions from d on
            if (r.t < 0) return;
            if (!whole) {
                float4 *o = reinterpret_cast<float4 *>(a.ws_o + part * HD + d);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
            } else if (a.q_type == kTypeF32) {
                float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + r.at * HD + d);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[i] = make_float4(y[4 * i] * inv, y[4 * i + 1] * inv, y[4 * i + 2] * inv, y[4 * i + 3] * inv);
            } else {
                uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + r.at * HD + d);
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
        if (NS == 2 && !g.pair) {
            // the other warpgroup's reference and sum, through this thread's lane of tensor memory
            const uint32_t box = tm + C::TM_S + lanes;
            if (any) {
                tmem_st2(box + w * TR, __float_as_uint(m), __float_as_uint(l));
                tmem_wait_st();
            }
            tc_fence_before();
            group_sync();
            tc_fence_after();
            if (any && !dead) {
                uint32_t om, ol;
                tmem_ld2(box + (w ^ 1) * TR, om, ol);
                const float m1 = __uint_as_float(om), l1 = __uint_as_float(ol), M = fmaxf(m, m1);
                const float f = m == -INFINITY ? 0.f : ex2(m - M), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - M);
                const float L = (m == -INFINITY ? 0.f : l * f) + (m1 == -INFINITY ? 0.f : l1 * f1);
                const float inv = L == 0.f ? 0.f : 1.f / L;
                if (!whole && w == 0 && r.t >= 0) a.ws_ml[part] = make_float2(M, L);
#pragma unroll 1
                for (int d = w * (HD / 2); d < (w + 1) * (HD / 2); d += 32) {
                    uint32_t u[32], v[32];
                    tmem_ld32(tm + C::TM_O + w * HD + lanes + d, u);
                    tmem_ld32(tm + C::TM_O + (w ^ 1) * HD + lanes + d, v);
                    tmem_wait_ld();
                    float y[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float x = m == -INFINITY ? 0.f : __uint_as_float(u[i]) * f;
                        if (m1 != -INFINITY) x = fmaf(__uint_as_float(v[i]), f1, x);
                        y[i] = x;
                    }
                    put(d, y, inv);
                }
            }
        } else if (any && !dead) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            if (!whole && r.t >= 0) a.ws_ml[part] = make_float2(m, l);
#pragma unroll 1
            for (int d = 0; d < HD; d += 32) {
                uint32_t u[32];
                tmem_ld32(tm + C::TM_O + w * HD + lanes + d, u);
                tmem_wait_ld();
                float y[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) y[i] = __uint_as_float(u[i]);
                put(d, y, inv);
            }
        }
        // the next segment's Q and zeros go over what the other warpgroup reads, and over what its products read
        tc_fence_before();
        group_sync();
        tc_fence_after();
    }
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
attn_tree_stream(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const __grid_constant__ TreeArgs a)
{
    extern __shared__ __align__(1024) uint8_t smem[];      // the swizzle needs the alignment (launch: no static shared memory)
    Tree<C> x(a, smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = blockIdx.x;
    if (warp == C::PROD) {
        if (lane == 0) {
            for (int i = 0; i < 8; ++i) {
                mbar_init(x.full + i, 1);
                mbar_init(x.ready + i, 4);
                mbar_init(x.empty + i, 1);
                mbar_init(x.raw_free + i, 4);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(x.s_full + i, 1);
                mbar_init(x.p_ready + i, 4);
                mbar_init(x.o_done + i, 1);
            }
            mbar_init(x.q_ready, C::SM_WARPS);
            x.flags[1] = 0;
            fence_barrier_init();
            prefetch_tensormap(&kmap);
            prefetch_tensormap(&vmap);
        }
        __syncwarp();
        pdl_wait();
        x.count(lane);
        if (rank == 0 && a.ranks > 1) {
            __syncwarp();
            for (int s = lane; s < a.n_seq; s += 32) {
                const int n = x.tok[s + 1] - x.tok[s], units = (n * a.group + a.unit_slots - 1) / a.unit_slots;
                const int places = x.before[s + 1] - x.before[s];
                a.ws_span[s] = make_int4(x.before[s], places ? places / (units * a.n_kv_head) : 0, x.tok[s], x.flags[2]);
            }
        }
    } else {
        if (warp == C::MMA) tmem_alloc(reinterpret_cast<uint32_t *>(const_cast<int *>(x.flags)), C::TM_COLS);
        pdl_wait();
    }
    pdl_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = (uint32_t)x.flags[0];
    const int share = x.flags[2], total = x.flags[3];
    const int64_t first = (int64_t)rank * share;
    const int from = (int)min(first, (int64_t)total), end = (int)min(first + share, (int64_t)total);
    if (warp < C::SM_WARPS) {
        x.softmax(tm, from, end, warp >> 2, warp & 3, lane, rank);
    } else if (warp < C::PROD) {
        x.fix(from, end, tid - C::FIX * 32);
    } else if (warp == C::PROD) {
        x.produce(&kmap, &vmap, from, end, lane);
    } else if (lane == 0) {
        x.issue(tm, from, end);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (x.flags[1]) {                                      // after a timeout: copies and products under way end first
        if (tid == 0) {
            const unsigned long long t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 200000000ull) __nanosleep(1000);
        }
        __syncthreads();
    }
    tc_fence_after();
    if (warp == C::MMA) tmem_dealloc(tm, C::TM_COLS);
}

// Units that several blocks have tiles of: o = sum w oc / sum w S over their parts, w = 2^(mx - max mx). A warp for
// a (node, head).
template <int HD>
__global__ void __launch_bounds__(128) attn_tree_combine(const TreeArgs a)
{
    constexpr int E = HD / 32;
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t job = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t tk = job / a.n_head;
    const int h = (int)(job - tk * a.n_head), hk = h / a.group;
    if (tk >= a.tok_end) return;
    // its sequence: the last one that begins at or before it, of those that have places
    int s = -1;
    int4 sp = make_int4(0, 0, 0, 0);
    for (int i0 = 0; i0 < a.n_seq; i0 += 32) {
        int4 q = make_int4(0, 0, 0x7fffffff, 0);
        if (i0 + lane < a.n_seq) {
            const uint4 u = ld_dep(reinterpret_cast<const uint4 *>(a.ws_span + i0 + lane));
            q = make_int4((int)u.x, (int)u.y, (int)u.z, (int)u.w);
        }
        const unsigned b = __ballot_sync(0xffffffffu, q.y > 0 && q.z <= tk);
        if (b) {
            const int l = 31 - __clz(b);
            s = i0 + l;
            sp = make_int4(__shfl_sync(0xffffffffu, q.x, l), __shfl_sync(0xffffffffu, q.y, l), __shfl_sync(0xffffffffu, q.z, l),
                           __shfl_sync(0xffffffffu, q.w, l));
        }
    }
    if (s < 0) return;
    int64_t c1 = (int64_t)(a.seq0 + s + 1) * a.n_each;
    if (a.cu) c1 = min(max((int64_t)ld_dep(a.cu + s + 1), (int64_t)0), a.n_tokens);
    if (tk >= c1) return;
    const int t = (int)(tk - sp.z), slot = t * a.group + h - hk * a.group, n = (int)(c1 - sp.z);
    const int units = (n * a.group + a.unit_slots - 1) / a.unit_slots, mu = slot / a.unit_slots;
    const int p0 = sp.x + (hk * units + mu) * sp.y, r0 = p0 / sp.w, r1 = (p0 + sp.y - 1) / sp.w;
    if (r0 == r1) return;
    const int in_unit = slot - mu * a.unit_slots;
    float m = -INFINITY, S = 0.f, acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    constexpr int BATCH = 4;
    for (int r = r0; r <= r1; r += BATCH) {
        float2 ml[BATCH];
        float v[BATCH][E];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int x = min(r + b, r1);
            const size_t row = ((size_t)x * 2 + (x == r0 && p0 >= x * sp.w ? 1 : 0)) * a.unit_slots + in_unit;
            ml[b] = ld_dep(a.ws_ml + row);
            const float *p = a.ws_o + row * HD + lane * E;
            if constexpr (E == 2) {
                const float2 y = ld_dep(reinterpret_cast<const float2 *>(p));
                v[b][0] = y.x; v[b][1] = y.y;
            } else {
#pragma unroll
                for (int e = 0; e < E; e += 4) {
                    const float4 y = ld_dep(reinterpret_cast<const float4 *>(p + e));
                    v[b][e] = y.x; v[b][e + 1] = y.y; v[b][e + 2] = y.z; v[b][e + 3] = y.w;
                }
            }
        }
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            if (r + b > r1 || ml[b].x == -INFINITY) continue;
            const float M = fmaxf(m, ml[b].x), f = m == -INFINITY ? 0.f : ex2(m - M), w = ex2(ml[b].x - M);
            S = fmaf(S, f, w * ml[b].y);
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], f, w * v[b][e]);
            m = M;
        }
    }
    const float inv = S == 0.f ? 0.f : 1.f / S;
    const int64_t at = (tk * a.n_head + h) * HD + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        const float y0 = acc[e] * inv, y1 = acc[e + 1] * inv;
        if (a.q_type == kTypeF32) *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + at + e) = make_float2(y0, y1);
        else if (a.q_type == kTypeF16) *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + at + e) = float2_to_kv2<__half>(y0, y1);
        else *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + at + e) = float2_to_kv2<__nv_bfloat16>(y0, y1);
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
    // the rings share what Q leaves: 16-bit tiles alone, or three of them (two, where that is all) and 8-bit ones
    const uint32_t left = C::DATA - (uint32_t)(a.unit_slots / 128) * C::PARTS * C::QPART;
    if (!C::E8) {
        a.nslot = (int)(left / C::SLOT);
        a.nraw = 0;
    } else {
        a.nslot = left >= 3 * C::SLOT + 2 * C::RAW ? 3 : 2;
        a.nraw = (int)((left - a.nslot * C::SLOT) / C::RAW);
    }
    if (a.nslot > 8) a.nslot = 8;
    if (a.nraw > 6) a.nraw = 6;
    const void *fn = reinterpret_cast<const void *>(&attn_tree_stream<C>);
    e = ensure_smem_attr(fn, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    void *args[] = {&kmap, &vmap, &a};
    e = launch_pdl(fn, dim3((unsigned)a.ranks), dim3(C::THREADS), C::SMEM, r.stream, args);
    if (e != cudaSuccess || a.ranks == 1) return e;
    const void *cf = reinterpret_cast<const void *>(&attn_tree_combine<C::HD>);
    const int64_t blocks = (a.tok_end * a.n_head + 3) / 4;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    void *cargs[] = {&a};
    return launch_pdl(cf, dim3((unsigned)blocks), dim3(128), 0, r.stream, cargs);
}

template <int HD, typename KV>
cudaError_t launch_tree_for(const TreeRequest &r)
{
    return r.parts == 2 ? launch_tree_kernel<TreeCfg<HD, KV, 2>>(r) : launch_tree_kernel<TreeCfg<HD, KV, 1>>(r);
}

} // namespace attn
