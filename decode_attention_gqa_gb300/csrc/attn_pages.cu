// attn_pages.cu -- the page bookkeeping of include/attn_pages.h: its C ABI, the kernels that release and
// give out pages and share them between sequences, and the copy of pages.
#include <map>
#include <mutex>

#include "attn_device.cuh"
#include "attn_launch.h"
#include "attn_pages.h"
#include "attn_paged_check.h"
#include "attn_paged_launch.h"

namespace attn {

namespace {

constexpr int kBookThreads = 1024;
constexpr int kMaxResize = 8192, kMaxForks = 4096;
constexpr int kBookCluster = 16;
constexpr int kMaxBookSeqs = 65536;

struct BookArgs {
    int32_t *refs, *table;
    const int32_t *a, *b, *rows;      // resize: have, want; fork: src, dst, rows
    int4 *copies;
    unsigned *err;
    int n_pages, max_pages, page_size, n_seq, n;
    FastDiv by_page;
};

// The sum of `x` over the threads before this one in the block, and over all of them.
__device__ __forceinline__ int block_scan(int x, int *sm, int &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int y = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, off);
        if (lane >= off) y += z;
    }
    if (lane == 31) sm[warp] = y;
    __syncthreads();
    if (warp == 0) {
        int w = lane < (int)blockDim.x / 32 ? sm[lane] : 0;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, w, off);
            if (lane >= off) w += z;
        }
        sm[lane] = w;
    }
    __syncthreads();
    total = sm[blockDim.x / 32 - 1];
    const int before = y - x + (warp ? sm[warp - 1] : 0);
    __syncthreads();
    return before;
}

// Which of the 16 pages from p on are free, of those below `end`; 16 is a divisor of p.
__device__ __forceinline__ unsigned free_of(const int32_t *refs, int p, int end)
{
    unsigned free = 0;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        if (p + 4 * v + 3 < end) {
            const uint4 c = ld_dep(reinterpret_cast<const uint4 *>(refs + p) + v);
            free |= (unsigned)((c.x == 0) | (c.y == 0) << 1 | (c.z == 0) << 2 | (c.w == 0) << 3) << 4 * v;
        } else {
            for (int i = 4 * v; i < 4 * v + 4; ++i)
                if (p + i < end && ld_dep(refs + p + i) == 0) free |= 1u << i;
        }
    }
    return free;
}

// Calls give(r, page) for the free page number r < need, lowest pages first, and returns how many there were.
template <class F>
__device__ __forceinline__ int give_free(const int32_t *refs, int end, int need, int *sm, F give)
{
    int found = 0;
    for (int p0 = 0; p0 < end && found < need; p0 += kBookThreads * 16) {
        const int p = p0 + (int)threadIdx.x * 16;
        unsigned free = free_of(refs, p, end);
        int total;
        int r = found + block_scan(__popc(free), sm, total);
        for (; free && r < need; ++r) {
            const int i = __ffs(free) - 1;
            free &= free - 1;
            give(r, p + i);
        }
        found += total;
    }
    return min(found, need);
}

// All blocks of the cluster, and what they have written
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_peer(int *p, unsigned rank, int x)   // to the same place in another block
{
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("st.shared::cluster.s32 [%0], %1;" :: "r"(at), "r"(x) : "memory");
}

__device__ __forceinline__ int pages_for(const BookArgs &g, int rows) { return div(g.by_page, rows + g.page_size - 1); }

__device__ __forceinline__ int rows_of(const BookArgs &g, int rows)
{
    const int cap = g.max_pages * g.page_size;
    if (rows < 0 || rows > cap) {
        atomicOr(g.err, ATTN_DEVERR_POSITION_CLAMPED);
        rows = rows < 0 ? 0 : cap;
    }
    return rows;
}

// Lets go of what the sequences have behind the rows that stay: a warp for a sequence, four entries a lane.
__device__ __forceinline__ void release(const BookArgs &g, int warp, int warps)
{
    const int lane = threadIdx.x & 31;
    for (int s = warp; s < g.n; s += warps) {
        const int pa = pages_for(g, rows_of(g, ld_dep(g.a + s))), pb = pages_for(g, rows_of(g, ld_dep(g.b + s)));
        int32_t *row = g.table + (size_t)s * g.max_pages;
        for (int e0 = pb + lane; e0 < pa; e0 += 128) {
            int p[4], had[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = e0 + 32 * i < pa ? ld_dep(row + e0 + 32 * i) : -1;
#pragma unroll
            for (int i = 0; i < 4; ++i) had[i] = (unsigned)p[i] < (unsigned)g.n_pages ? atomicSub(g.refs + p[i], 1) : p[i] == -1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (had[i] <= 0) {                             // not a page, or one that nobody holds
                    if ((unsigned)p[i] < (unsigned)g.n_pages) atomicAdd(g.refs + p[i], 1);
                    atomicOr(g.err, ATTN_DEVERR_BAD_PAGE);
                }
                if (e0 + 32 * i < pa) row[e0 + 32 * i] = -1;
            }
        }
    }
}

// One cluster: what is released has to be known before pages are given out, and pages go out in the order of their numbers.
// Each block releases what some of the sequences let go, counts the free pages of its part of the numbers, and, once it
// knows what the blocks before it have, gives its own out. Latency bounds it: of 1000 sequences that change by 85 thousand
// pages of 356 thousand, 27 us (clusters of 8 44 us, of 1 124 us, where 64 sequences take 6 us either way; a kernel of its
// own for what is released, over the whole GPU, 25 us and 7 us).
__global__ void __launch_bounds__(kBookThreads) resize_kernel(const BookArgs g)
{
    extern __shared__ int book_smem[];                         // [n + 1] first page of each sequence, [n] first entry
    __shared__ int sm[32], counts[kBookCluster];
    __shared__ uint16_t list[kBookThreads * 16];
    int *first = book_smem, *entry = book_smem + g.n + 1;
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int blocks = (int)gridDim.x, rank = (int)blockIdx.x;
    int need = 0;
    for (int s0 = 0; s0 < g.n; s0 += kBookThreads) {
        const int s = s0 + tid;
        int x = 0;
        if (s < g.n) {
            const int a = rows_of(g, ld_dep(g.a + s)), b = rows_of(g, ld_dep(g.b + s));
            const int pa = pages_for(g, a), pb = pages_for(g, b);
            x = max(pb - pa, 0);
            entry[s] = b < a && b % g.page_size ? -pb : pa;    // the last page that is left is cut, or the first new entry
        }
        int total;
        const int before = need + block_scan(x, sm, total);
        if (s < g.n) first[s] = before;
        need += total;
    }
    if (tid == 0) first[g.n] = need;
    release(g, rank * (kBookThreads / 32) + warp, blocks * (kBookThreads / 32));
    __threadfence();
    cluster_sync();
    // cut inside a page: nobody else may hold it
    for (int s = rank * kBookThreads + tid; s < g.n; s += blocks * kBookThreads) {
        if (entry[s] < 0) {
            const int p = ld_dep(g.table + (size_t)s * g.max_pages - entry[s] - 1);
            if ((unsigned)p < (unsigned)g.n_pages && ld_dep(g.refs + p) > 1) atomicOr(g.err, ATTN_DEVERR_SHARED_PAGE);
        }
    }
    if (need == 0) return;                                     // in every block
    const int part = (g.n_pages + 16 * blocks - 1) / (16 * blocks) * 16;
    const int p0 = (int)min((int64_t)rank * part, (int64_t)g.n_pages), p1 = min(p0 + part, g.n_pages);
    int there = 0;                                             // free pages before this block's
    if (blocks > 1) {
        int mine = 0;
        for (int p = p0 + tid * 16; p < p1; p += kBookThreads * 16) mine += __popc(free_of(g.refs, p, p1));
        int total;
        (void)block_scan(mine, sm, total);
        if (tid < blocks) st_peer(counts + rank, tid, total);
        cluster_sync();
        for (int i = 0; i < rank; ++i) there += counts[i];
    }
    auto place = [&](int r) {                                  // the sequence that page number r goes to
        int lo = 0, hi = g.n - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (first[mid + 1] > r) hi = mid;
            else lo = mid + 1;
        }
        return lo;
    };
    // The free pages of 1024 x 16 numbers, in order, then a warp for a sequence that gets some of them (threads that
    // placed what they found themselves took 1.7 times as long: no two lanes wrote near each other).
    int found = there;
    for (int p = p0; p < p1 && found < need; p += kBookThreads * 16) {
        unsigned free = free_of(g.refs, p + tid * 16, p1);
        int total;
        for (int i = block_scan(__popc(free), sm, total); free; free &= free - 1, ++i) list[i] = (uint16_t)(tid * 16 + __ffs(free) - 1);
        __syncthreads();
        total = min(total, need - found);
        for (int i = tid; i < total; i += kBookThreads) g.refs[p + list[i]] = 1;
        for (int s = place(found) + warp; s < g.n && first[s] < found + total; s += kBookThreads / 32) {
            int32_t *to = g.table + (size_t)s * g.max_pages + entry[s] - first[s];
            for (int r = max(first[s], found) + lane; r < min(first[s + 1], found + total); r += 32) to[r] = p + list[r - found];
        }
        found += total;
        __syncthreads();
    }
    if (rank == blocks - 1) {
        for (int r = found + tid; r < need; r += kBookThreads) {
            const int s = place(r);
            g.table[(size_t)s * g.max_pages + entry[s] + (r - first[s])] = -1;
        }
        if (found < need && tid == 0) atomicOr(g.err, ATTN_DEVERR_NO_PAGE);
    }
}

// Blocks of the resizing cluster: 16, or where the current device (a share of one) holds no such cluster, the largest power of
// two below that it holds. The kernel takes any number. Asked once per device.
cudaError_t resize_blocks(const void *fn, unsigned *blocks)
{
    static std::mutex mu;
    static std::map<int, unsigned> known;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    const auto it = known.find(dev);
    if (it != known.end()) {
        *blocks = it->second;
        return cudaSuccess;
    }
    constexpr int smem = (2 * kMaxResize + 1) * 4;             // of the most sequences
    e = ensure_smem_attr(fn, smem);
    if (e != cudaSuccess) return e;
    unsigned n = kBookCluster;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
        (void)cudaGetLastError();
        n = 8;                                                 // the largest portable one
    }
    while (n > 1 && cluster_slots(fn, dim3(kBookThreads), smem, n) < 1) n /= 2;
    known[dev] = *blocks = n;
    return cudaSuccess;
}

__device__ __forceinline__ bool fork_at(const BookArgs &g, int i, int &src, int &dst, int &rows)
{
    src = ld_dep(g.a + i);
    dst = ld_dep(g.b + i);
    rows = ld_dep(g.rows + i);
    return (unsigned)src < (unsigned)g.n_seq && (unsigned)dst < (unsigned)g.n_seq && src != dst && rows >= 0 &&
           rows <= g.max_pages * g.page_size;
}

// Sequences that a fork may not end in: dst of two forks, or of one and src of another. Every block finds them by itself.
struct Taken {
    unsigned src[kMaxBookSeqs / 32], once[kMaxBookSeqs / 32], twice[kMaxBookSeqs / 32];

    __device__ __forceinline__ void fill(const BookArgs &g)
    {
        for (int i = threadIdx.x; i * 32 < g.n_seq; i += kBookThreads) src[i] = once[i] = twice[i] = 0u;
        __syncthreads();
        for (int i = threadIdx.x; i < g.n; i += kBookThreads) {
            int s, d, rows;
            if (!fork_at(g, i, s, d, rows)) continue;
            atomicOr(src + s / 32, 1u << s % 32);
            const unsigned bit = 1u << d % 32;
            if (atomicOr(once + d / 32, bit) & bit) atomicOr(twice + d / 32, bit);
        }
        __syncthreads();
    }
    __device__ __forceinline__ bool has(int d) const { return (src[d / 32] | twice[d / 32]) >> d % 32 & 1u; }
};

// Block 0 gives out the pages that the forks end in; the others share the full ones, which are held already, so
// that no count that block 0 looks for changes to or from 0 under it.
// With the resize before and the copy behind it, in a graph: one sequence of 1000 rows into four 10.6 us, 16 of up to 4097
// rows into 64 18.9 us (31 MB copied); each is a launch and a chain of loads.
__global__ void __launch_bounds__(kBookThreads) fork_kernel(const BookArgs g)
{
    __shared__ int sm[32];
    __shared__ uint16_t which[kMaxForks];
    __shared__ Taken taken;
    pdl_wait();
    const int tid = threadIdx.x;
    taken.fill(g);
    if (blockIdx.x == 0) {
        int need = 0;
        for (int i0 = 0; i0 < g.n; i0 += kBookThreads) {
            const int i = i0 + tid;
            int src, dst, rows, x = 0;
            if (i < g.n) {
                if (fork_at(g, i, src, dst, rows) && !taken.has(dst)) x = rows - div(g.by_page, rows) * g.page_size > 0;
                else atomicOr(g.err, ATTN_DEVERR_BAD_REQUEST);
                if (!x) g.copies[i] = make_int4(-1, -1, 0, 0);
            }
            int total;
            const int before = need + block_scan(x, sm, total);
            if (x) which[before] = (uint16_t)i;
            need += total;
        }
        __syncthreads();
        auto end = [&](int r, int page) {
            const int i = which[r];
            int src, dst, rows;
            (void)fork_at(g, i, src, dst, rows);
            const int full = div(g.by_page, rows);
            const int from = ld_dep(g.table + (size_t)src * g.max_pages + full);
            if (page >= 0) g.refs[page] = 1;
            g.table[(size_t)dst * g.max_pages + full] = page;
            const bool there = (unsigned)from < (unsigned)g.n_pages;
            if (!there) atomicOr(g.err, ATTN_DEVERR_BAD_PAGE);
            g.copies[i] = there && page >= 0 ? make_int4(from, page, rows - full * g.page_size, 0) : make_int4(-1, -1, 0, 0);
        };
        const int found = give_free(g.refs, g.n_pages, need, sm, end);
        for (int r = found + tid; r < need; r += kBookThreads) end(r, -1);
        if (found < need && tid == 0) atomicOr(g.err, ATTN_DEVERR_NO_PAGE);
        return;
    }
    // a warp for a fork
    const int warps = (gridDim.x - 1) * (kBookThreads / 32);
    for (int i = (blockIdx.x - 1) * (kBookThreads / 32) + (tid >> 5); i < g.n; i += warps) {
        int src, dst, rows;
        if (!fork_at(g, i, src, dst, rows) || taken.has(dst)) continue;
        const int full = div(g.by_page, rows);
        for (int e = tid & 31; e < full; e += 32) {
            int p = ld_dep(g.table + (size_t)src * g.max_pages + e);
            if ((unsigned)p < (unsigned)g.n_pages) {
                atomicAdd(g.refs + p, 1);
            } else {
                p = -1;
                atomicOr(g.err, ATTN_DEVERR_BAD_PAGE);
            }
            g.table[(size_t)dst * g.max_pages + e] = p;
        }
    }
}

struct CopyArgs {
    uint8_t *k, *v;
    float *k_scale, *v_scale;
    int64_t page_stride, row_stride, head_stride;              // bytes
    const int4 *copies;
    unsigned *err;
    int n_pages, page_size, n_kv_head, units;                  // 16-byte units of a head's row
    bool heads_outer;                                          // a head's rows lie together
    FastDiv by_units, by_heads, by_rows;
};

// Rows of a page, K or V, as 16-byte units in the order they lie in memory; four of a thread on their way at a time.
// Bytes and latency bound it: 64 pages of 128 rows, 8 heads of 128, f16, half full on average, 8 us from cold caches.
__global__ void __launch_bounds__(256) copy_kernel(const CopyArgs g)
{
    pdl_wait();
    uint4 c = ld_dep(reinterpret_cast<const uint4 *>(g.copies + blockIdx.x));
    const int from = (int)c.x, to = (int)c.y, rows = min((int)c.z, g.page_size);
    if (to < 0 || rows <= 0) return;
    if ((unsigned)from >= (unsigned)g.n_pages || to >= g.n_pages) {
        if (threadIdx.x == 0) atomicOr(g.err, ATTN_DEVERR_BAD_PAGE);
        return;
    }
    uint8_t *pool = blockIdx.z ? g.v : g.k;
    float *scale = blockIdx.z ? g.v_scale : g.k_scale;
    if (scale && blockIdx.y == 0)
        for (int h = threadIdx.x; h < g.n_kv_head; h += 256)
            scale[(size_t)to * g.n_kv_head + h] = ld_dep(scale + (size_t)from * g.n_kv_head + h);
    const uint8_t *src = pool + (int64_t)from * g.page_stride;
    uint8_t *dst = pool + (int64_t)to * g.page_stride;
    const int all = (g.heads_outer ? g.page_size : rows) * g.n_kv_head * g.units;
    const int step = gridDim.y * 256;
    auto at = [&](int i) -> int64_t {                          // -1: no row of the copy
        const int x = div(g.by_units, i), u = i - x * g.units;
        int row, head;
        if (g.heads_outer) {
            head = div(g.by_rows, x);
            row = x - head * g.page_size;
            if (row >= rows) return -1;
        } else {
            row = div(g.by_heads, x);
            head = x - row * g.n_kv_head;
        }
        return row * g.row_stride + head * g.head_stride + u * 16;
    };
    for (int i0 = blockIdx.y * 256 + threadIdx.x; i0 < all; i0 += 4 * step) {
        uint4 v[4];
        int64_t off[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            off[x] = i0 + x * step < all ? at(i0 + x * step) : -1;
            if (off[x] >= 0) v[x] = ld_dep(reinterpret_cast<const uint4 *>(src + off[x]));
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (off[x] >= 0) *reinterpret_cast<uint4 *>(dst + off[x]) = v[x];
    }
}

attn_status check_book(const int32_t *refs, int n_pages, const int32_t *table, int max_pages, int page_size, int n_seq)
{
    if (n_pages < 1 || max_pages < 1 || n_seq < 0 || n_seq > 65535) return ATTN_ERR_INVALID_ARG;
    if (page_size < 16 || page_size > 1024 || page_size % 16 != 0) return ATTN_ERR_INVALID_ARG;
    if (n_pages > 1 << 30) return ATTN_ERR_UNSUPPORTED;
    if ((int64_t)max_pages * page_size > check::kMaxRows) return ATTN_ERR_INVALID_ARG;
    if (!check::aligned(refs, 16) || !check::aligned(table, 4)) return ATTN_ERR_INVALID_ARG;
    return ATTN_OK;
}

} // namespace

} // namespace attn

using namespace attn;
using namespace attn::check;

extern "C" {

attn_status attn_pages_resize(int32_t *refs, int n_pages, int32_t *block_table, int max_pages, int page_size,
                              const int32_t *have, const int32_t *want, int n_seq, attn_stream_t stream)
{
    const attn_status st = check_book(refs, n_pages, block_table, max_pages, page_size, n_seq);
    if (st != ATTN_OK) return st;
    if (!aligned(have, 4) || !aligned(want, 4)) return ATTN_ERR_INVALID_ARG;
    if (n_seq > 0 && (!refs || !block_table || !have || !want)) return ATTN_ERR_INVALID_ARG;
    if (n_seq > kMaxResize || (int64_t)n_seq * max_pages > 0x7fffffff) return ATTN_ERR_UNSUPPORTED;   // 32 bits count the entries
    if (n_seq == 0) return ATTN_OK;
    BookArgs g{};
    int sms = 0;
    cudaError_t e = device_facts(&sms, &g.err);
    if (e != cudaSuccess) return fail(e);
    g.refs = refs;
    g.table = block_table;
    g.a = have;
    g.b = want;
    g.n_pages = n_pages;
    g.max_pages = max_pages;
    g.page_size = page_size;
    g.n_seq = g.n = n_seq;
    g.by_page = fast_div((unsigned)page_size);
    const void *fn = reinterpret_cast<const void *>(&resize_kernel);
    unsigned blocks = 0;
    e = resize_blocks(fn, &blocks);
    if (e != cudaSuccess) return fail(e);
    void *args[] = {&g};
    e = launch_pdl_cluster(fn, dim3(blocks), dim3(kBookThreads), (2 * (size_t)n_seq + 1) * 4, reinterpret_cast<cudaStream_t>(stream),
                           args, blocks);
    return e == cudaSuccess ? ATTN_OK : fail(e);
}

attn_status attn_pages_fork(int32_t *refs, int n_pages, int32_t *block_table, int max_pages, int page_size, int n_seq,
                            const int32_t *src, const int32_t *dst, const int32_t *rows, int n_fork, int32_t *copies,
                            attn_stream_t stream)
{
    const attn_status st = check_book(refs, n_pages, block_table, max_pages, page_size, n_seq);
    if (st != ATTN_OK) return st;
    if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(rows, 4) || !aligned(copies, 16) || n_fork < 0)
        return ATTN_ERR_INVALID_ARG;
    if (n_fork > 0 && (!refs || !block_table || !src || !dst || !rows || !copies)) return ATTN_ERR_INVALID_ARG;
    if (n_fork > kMaxForks) return ATTN_ERR_UNSUPPORTED;
    if (n_fork == 0) return ATTN_OK;
    BookArgs g{};
    int sms = 0;
    cudaError_t e = device_facts(&sms, &g.err);
    if (e != cudaSuccess) return fail(e);
    g.refs = refs;
    g.table = block_table;
    g.a = src;
    g.b = dst;
    g.rows = rows;
    g.copies = reinterpret_cast<int4 *>(copies);
    g.n_pages = n_pages;
    g.max_pages = max_pages;
    g.page_size = page_size;
    g.n_seq = n_seq;
    g.n = n_fork;
    g.by_page = fast_div((unsigned)page_size);
    const void *fn = reinterpret_cast<const void *>(&fork_kernel);
    void *args[] = {&g};
    const unsigned warps = kBookThreads / 32, sharing = ((unsigned)n_fork + warps - 1) / warps;
    e = launch_pdl(fn, dim3(1 + sharing), dim3(kBookThreads), 0, reinterpret_cast<cudaStream_t>(stream), args);
    return e == cudaSuccess ? ATTN_OK : fail(e);
}

attn_status attn_pages_copy(const attn_paged_cache *cache, const int32_t *copies, int n, attn_stream_t stream)
{
    attn_status st = check_cache_pointers(cache);
    if (st != ATTN_OK) return st;
    if (n < 0 || !aligned(copies, 16) || (n > 0 && !copies)) return ATTN_ERR_INVALID_ARG;
    Strides cs;
    st = check_cache_shape(cache, 1, cs);
    if (st != ATTN_OK) return st;
    if (n == 0) return ATTN_OK;
    CopyArgs g{};
    int sms = 0;
    cudaError_t e = device_facts(&sms, &g.err);
    if (e != cudaSuccess) return fail(e);
    const int64_t es = type_bytes(cache->kv_type);
    g.k = static_cast<uint8_t *>(cache->k);
    g.v = static_cast<uint8_t *>(cache->v);
    g.k_scale = cache->k_scale;
    g.v_scale = cache->v_scale;
    g.page_stride = cs.page * es;
    g.row_stride = cs.row * es;
    g.head_stride = cs.head * es;
    g.copies = reinterpret_cast<const int4 *>(copies);
    g.n_pages = cache->n_pages;
    g.page_size = cache->page_size;
    g.n_kv_head = cache->n_kv_head;
    g.units = (int)(cache->head_dim * es / 16);
    g.heads_outer = cs.head > cs.row;
    const int64_t units = (int64_t)cache->page_size * cache->n_kv_head * g.units;
    if (units > 0x3fffffff) return ATTN_ERR_UNSUPPORTED;
    g.by_units = fast_div((unsigned)g.units);
    g.by_heads = fast_div((unsigned)g.n_kv_head);
    g.by_rows = fast_div((unsigned)g.page_size);
    // four units a thread, until the blocks fill the GPU eight times over
    int64_t parts = (units + 1023) / 1024;
    const int64_t most = ((int64_t)sms * 64 + 2 * n - 1) / (2 * (int64_t)n);
    parts = parts < most ? parts : most;
    const void *fn = reinterpret_cast<const void *>(&copy_kernel);
    void *args[] = {&g};
    e = launch_pdl(fn, dim3((unsigned)n, (unsigned)parts, 2), dim3(256), 0, reinterpret_cast<cudaStream_t>(stream), args);
    return e == cudaSuccess ? ATTN_OK : fail(e);
}

} // extern "C"
