// pages.cu -- page operations of a paged cache: reserving, freeing, forking,
// compacting and copying pages, all on the device.
//
// The pool is one array: refs[p] is how many block-table entries name page p,
// 0 a free page.  Free pages are handed out in ascending order, so results do
// not depend on timing, and there is no free list to keep in step.  The table
// operations leave a list of moves (source page, destination page, rows), and
// one copy launch carries it out over the caches of many layers.
//
//   free     entries [from, to) of a row give their reference back, become -1
//   reserve  entries [from, to) of a row that are -1 take the lowest free pages
//   fork     row d becomes row s's first len tokens: full pages are shared, a
//            partial last page is copied into the lowest free page
//   compact  with U pages in use, the i-th page in use at or above U moves to
//            the i-th free page below U
//   copy     the listed rows of the listed pages, K, V and scales, every layer
#include <cuda_runtime.h>

#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"

namespace gqa {
namespace {

constexpr int kScanThreads = 1024;
// Pages a block looks at at a time: 16 a thread, so a pool of 16,384 is one round
// of loads; 4 a thread where the round's free pages are listed in shared memory.
constexpr int kPer = 16, kTile = kScanThreads * kPer;
constexpr int kListPer = 4, kListTile = kScanThreads * kListPer;
constexpr int kListed = 2 * kListTile;
// A fork's entries up to which one cluster copies them (16 a thread): free, fork and copy of
// 48 rows of 94 entries take 20.2 us so, 22.5 with a launch of their own, a thread each.
constexpr int kForkBlocks = 8, kForkEntries = 16 * (kForkBlocks - 1) * kScanThreads;

// Exclusive prefix of v over the block, and the block's sum in `sum`.  All
// kScanThreads threads take part.
__device__ __forceinline__ int block_scan(int v, int &sum) {
    __shared__ int warp_sum[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // warp_sum of the call before has been read
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int w = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    sum = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return x - v + (warp == 0 ? 0 : before);
}

// Which of the PER pages base + PER tid .. are free, a bit each (none past the pool).
template <int PER>
__device__ __forceinline__ uint32_t free_bits(const int32_t *refs, int base, int num_pages) {
    const int p = base + PER * (int)threadIdx.x;
    uint32_t bits = 0;
    if (p + PER <= num_pages) {
        int4 r[PER / 4];
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) r[i] = *reinterpret_cast<const int4 *>(refs + p + 4 * i);
#pragma unroll
        for (int i = 0; i < PER / 4; ++i)
            bits |= (uint32_t)((r[i].x <= 0) | (r[i].y <= 0) << 1 | (r[i].z <= 0) << 2 |
                               (r[i].w <= 0) << 3) << (4 * i);
    } else {
        for (int i = 0; i < PER; ++i)
            if (p + i < num_pages && refs[p + i] <= 0) bits |= 1u << i;
    }
    return bits;
}

// A barrier of the cluster's threads.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\t"
                 "barrier.cluster.wait.acquire;" ::: "memory");
}

// The bits of those pages that are in the pool.
template <int PER>
__device__ __forceinline__ uint32_t pool_bits(int base, int num_pages) {
    const int n = num_pages - (base + PER * (int)threadIdx.x);
    return n <= 0 ? 0u : n >= PER ? (1u << PER) - 1u : (1u << n) - 1u;
}

__global__ void __launch_bounds__(256) pages_free_kernel(int32_t *table, int max_blocks,
                                                         int table_rows, const int32_t *rows,
                                                         const int32_t *from, const int32_t *to,
                                                         int n, int per_row, int32_t *refs,
                                                         int num_pages, int32_t *err) {
    pdl_wait();
    pdl_launch_dependents();
    const int i = blockIdx.x / per_row, part = blockIdx.x - i * per_row;
    const int row = rows[i];
    if (row < 0 || row >= table_rows) {
        if (threadIdx.x == 0 && part == 0) report_error(err, ATTN_ERR_BOUNDS);
        return;
    }
    const int j = part * 256 + threadIdx.x;
    if (j < from[i] || j >= min(to[i], max_blocks)) return;
    int32_t *entry = table + (int64_t)row * max_blocks + j;
    if (*entry < 0) return;
    const int page = atomicExch(entry, -1);  // one taker, if the entry is named twice
    if (page < 0) return;
    if (page >= num_pages) {
        report_error(err, ATTN_ERR_BOUNDS);
    } else if (atomicSub(refs + page, 1) <= 0) {  // was free already
        atomicAdd(refs + page, 1);
        report_error(err, ATTN_ERR_BOUNDS);
    }
}

__global__ void __launch_bounds__(kScanThreads)
    pages_reserve_kernel(int32_t *table, int max_blocks, int table_rows, const int32_t *rows,
                         const int32_t *from, const int32_t *to, int n, int32_t *refs,
                         int num_pages, int32_t *err) {
    pdl_wait();
    pdl_launch_dependents();
    __shared__ int list[kListed];
    for (int base = 0; base < n; base += kScanThreads) {  // a row per thread
        const int i = base + threadIdx.x;
        int32_t *entries = nullptr;
        int j0 = 0, j1 = 0, need = 0;
        if (i < n) {
            const int row = rows[i];
            if (row < 0 || row >= table_rows) {
                report_error(err, ATTN_ERR_BOUNDS);
            } else {
                entries = table + (int64_t)row * max_blocks;
                j0 = max(0, from[i]);
                j1 = min(to[i], max_blocks);
                for (int j = j0; j < j1; ++j) need += entries[j] < 0 ? 1 : 0;
            }
        }
        int total;
        int rank = block_scan(need, total);  // of this row's next empty entry
        for (int done = 0; done < total;) {
            // the lowest free pages, as many as are needed and fit the list
            int listed = 0;
            for (int p = 0;
                 p < num_pages && listed < total - done && listed + kListTile <= kListed;
                 p += kListTile) {
                uint32_t bits = free_bits<kListPer>(refs, p, num_pages);
                int sum;
                int at = listed + block_scan(__popc(bits), sum);
                for (; bits != 0; bits &= bits - 1)
                    list[at++] = p + kListPer * threadIdx.x + __ffs(bits) - 1;
                listed += sum;
            }
            __syncthreads();
            const int end = done + min(listed, total - done);
            for (; j0 < j1 && rank < end; ++j0) {
                if (entries[j0] >= 0) continue;
                const int page = list[rank - done];
                entries[j0] = page;
                refs[page] = 1;
                ++rank;
            }
            __syncthreads();
            if (listed == 0) {  // the pool is exhausted
                if (threadIdx.x == 0) report_error(err, ATTN_ERR_PAGES);
                return;
            }
            done = end;
        }
    }
}

struct ForkParams {
    int32_t *table;
    int max_blocks, table_rows;
    const int32_t *src_rows, *dst_rows, *seq_lens;
    int n, block_size;
    int32_t *refs;
    int num_pages;
    int32_t *moves, *n_moves, *err;
    bool share;  // the entries have not been copied yet
};

struct ForkRow {
    int32_t *src, *dst;  // nullptr: a row outside the table
    int full, part;      // full pages, tokens of the partial one
};

__device__ __forceinline__ ForkRow fork_row(const ForkParams &p, int i, bool report) {
    ForkRow f = {};
    const int s = p.src_rows[i], d = p.dst_rows[i];
    int len = p.seq_lens[i];
    bool bad = s < 0 || s >= p.table_rows || d < 0 || d >= p.table_rows || s == d;
    if (!bad) {
        f.src = p.table + (int64_t)s * p.max_blocks;
        f.dst = p.table + (int64_t)d * p.max_blocks;
        const int64_t cap = (int64_t)p.max_blocks * p.block_size;
        if (len < 0 || len > cap) bad = true, len = len < 0 ? 0 : (int)cap;
        f.full = len / p.block_size;
        f.part = len - f.full * p.block_size;
    }
    if (bad && report) report_error(p.err, ATTN_ERR_BOUNDS);
    return f;
}

// The source's page j, -1 if there is none.  A free page is none of the source's: reported
// like one outside the pool.
__device__ __forceinline__ int fork_page(const ForkParams &p, const ForkRow &f, int j) {
    const int page = f.src[j];
    if (page < 0) return -1;
    if (page < p.num_pages && p.refs[page] > 0) return page;
    report_error(p.err, ATTN_ERR_BOUNDS);
    return -1;
}

// Entry j of request i's new row: a full page is shared, the partial last one named for
// the copy.
__device__ __forceinline__ void fork_entry(const ForkParams &p, int i, int j) {
    const ForkRow f = fork_row(p, i, j == 0);
    if (f.dst == nullptr) return;
    const int page = j < f.full + (f.part > 0 ? 1 : 0) ? fork_page(p, f, j) : -1;
    if (page >= 0 && j < f.full) atomicAdd(p.refs + page, 1);
    f.dst[j] = page;
}

// The entries of many or long rows, a thread each, before the kernel below.
__global__ void __launch_bounds__(256) pages_share_kernel(const ForkParams p, int per_row) {
    pdl_wait();
    pdl_launch_dependents();
    const int i = blockIdx.x / per_row, j = (blockIdx.x - i * per_row) * 256 + threadIdx.x;
    if (j < p.max_blocks) fork_entry(p, i, j);
}

// A cluster: block 0 hands out the pages for the partial last pages, the others copy the
// entries and count the shared pages.  Block 0 writes when they are done, so what is a free
// page is what was one before the call; until then it has read the first 1,024 requests.
__global__ void __cluster_dims__(kForkBlocks, 1, 1) __launch_bounds__(kScanThreads)
    pages_fork_kernel(const ForkParams p) {
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x > 0) {
        if (p.share)
            for (int at = (blockIdx.x - 1) * kScanThreads + threadIdx.x; at < p.n * p.max_blocks;
                 at += (kForkBlocks - 1) * kScanThreads) {
                const int i = at / p.max_blocks;
                fork_entry(p, i, at - i * p.max_blocks);
            }
        cluster_sync();
        return;
    }
    // The requests of a batch that want a page: what they copy, and the entry it becomes
    __shared__ int copied[kScanThreads], tokens[kScanThreads];
    __shared__ int32_t *entry[kScanThreads];
    int moves = 0, tile = 0;  // pages below `tile` are taken
    bool lacking = false, shared = false;
    for (int base = 0; base < p.n; base += kScanThreads) {
        const int i = base + threadIdx.x;
        ForkRow f = {};
        if (i < p.n) f = fork_row(p, i, false);
        int page = -1;
        if (f.dst != nullptr && f.part > 0)  // (the others have left it in the entry, too)
            page = base == 0 ? fork_page(p, f, f.full) : f.dst[f.full];
        const bool some = page >= 0;
        int need;
        const int at = block_scan(some ? 1 : 0, need);
        if (some) {
            copied[at] = page;
            tokens[at] = f.part;
            entry[at] = f.dst + f.full;
        }
        int given = 0;
        for (; tile < p.num_pages && given < need; tile += kTile) {
            uint32_t bits = free_bits<kPer>(p.refs, tile, p.num_pages);
            int sum;
            int to = given + block_scan(__popc(bits), sum);
            if (!shared) cluster_sync();
            shared = true;
            for (; bits != 0 && to < need; bits &= bits - 1, ++to) {
                const int page = tile + kPer * threadIdx.x + __ffs(bits) - 1;
                int32_t *move = p.moves + 3 * (moves + to);
                move[0] = copied[to];
                move[1] = page;
                move[2] = tokens[to];
                *entry[to] = page;
                p.refs[page] = 1;
            }
            given += sum;
            if (given >= need) break;  // the tile may hold pages for the next batch
        }
        given = min(given, need);
        if (!shared) cluster_sync();
        shared = true;
        __syncthreads();
        for (int to = given + threadIdx.x; to < need; to += kScanThreads) *entry[to] = -1;
        moves += given;
        lacking |= given < need;
        __syncthreads();
    }
    if (!shared) cluster_sync();  // n is 0
    if (threadIdx.x == 0) {
        *p.n_moves = moves;
        if (lacking) report_error(p.err, ATTN_ERR_PAGES);
    }
}

// One block: counts the pages in use (U), pairs pages at or above U with free
// ones below, and leaves in `to` where each page at or above U has gone.
__global__ void __launch_bounds__(kScanThreads)
    pages_plan_compact_kernel(int32_t *refs, int num_pages, int block_size, int32_t *moves,
                              int max_moves, int32_t *n_moves, int32_t *used, int32_t *to,
                              int32_t *err) {
    pdl_wait();
    pdl_launch_dependents();
    int U = 0;
    {
        int mine = 0;
        for (int base = 0; base < num_pages; base += kTile)
            mine += __popc(pool_bits<kPer>(base, num_pages) &
                           ~free_bits<kPer>(refs, base, num_pages));
        block_scan(mine, U);
    }
    int takes = 0, leaves = 0;  // free pages below U, pages in use from U on
    for (int base = 0; base < num_pages; base += kTile) {
        const int p = base + kPer * threadIdx.x;
        const uint32_t free = free_bits<kPer>(refs, base, num_pages);
        const uint32_t pool = pool_bits<kPer>(base, num_pages);
        const uint32_t low = pool & pool_bits<kPer>(base, U);
        uint32_t t = free & low, l = pool & ~low & ~free;
        int st, sl;
        int at_t = takes + block_scan(__popc(t), st), at_l = leaves + block_scan(__popc(l), sl);
        for (; t != 0; t &= t - 1, ++at_t)
            if (at_t < max_moves) moves[3 * at_t + 1] = p + __ffs(t) - 1;
        for (; l != 0; l &= l - 1, ++at_l)
            if (at_l < max_moves) moves[3 * at_l] = p + __ffs(l) - 1;
        for (uint32_t high = pool & ~low; high != 0; high &= high - 1) {
            const int page = p + __ffs(high) - 1;
            to[page] = page;
        }
        takes += st;
        leaves += sl;
    }
    __syncthreads();
    const int n = min(leaves, max_moves);
    for (int k = threadIdx.x; k < n; k += kScanThreads) {
        const int src = moves[3 * k], dst = moves[3 * k + 1];
        moves[3 * k + 2] = block_size;
        to[src] = dst;
        refs[dst] = refs[src];
        refs[src] = 0;
    }
    if (threadIdx.x == 0) {
        *n_moves = n;
        *used = U;
        if (n < leaves) report_error(err, ATTN_ERR_WORKSPACE);
    }
}

__global__ void __launch_bounds__(256) pages_rename_kernel(int32_t *table, int64_t entries,
                                                           const int32_t *to, const int32_t *used,
                                                           int num_pages, int32_t *err) {
    pdl_wait();
    pdl_launch_dependents();
    const int U = *used;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < entries;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int page = table[i];
        if (page < U) continue;
        if (page >= num_pages)
            report_error(err, ATTN_ERR_BOUNDS);
        else
            table[i] = to[page];
    }
}

constexpr int kCopyCaches = 32;  // layers of one launch
constexpr int kCopyUnroll = 4;   // 16-byte pieces a thread has in flight
constexpr int kCopyThreads = 256;

struct CopyParams {
    struct {
        uint8_t *k, *v;
        float *ks, *vs;
    } cache[kCopyCaches];
    int n_caches;
    const int32_t *moves, *n_moves;
    int max_moves, num_pages, block_size;
    int page_pieces;  // 16-byte pieces of a page of one tensor
    int run_pieces;   // pieces of the page's rows that lie together: all, or a head's
    int row_pieces;   // pieces of one row of such a run
    int scale_block, n_kv_heads;
    int segments;     // steps of a block over a page
    int32_t *err;
};

// HBM-bound copy.  A step of a block moves up to 16 KB of one tensor of one
// layer of one move, every load before the first store.
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const CopyParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int n = min(*p.n_moves, p.max_moves);
    const int per_move = p.n_caches * 2 * p.segments;
    const int64_t steps = (int64_t)max(n, 0) * per_move;
    for (int64_t s = blockIdx.x; s < steps; s += gridDim.x) {
        const int move = (int)(s / per_move);
        int rem = (int)(s - (int64_t)move * per_move);
        const int c = rem / (2 * p.segments);
        rem -= c * 2 * p.segments;
        const int tensor = rem / p.segments, seg = rem - tensor * p.segments;
        const int src = p.moves[3 * move], dst = p.moves[3 * move + 1], rows = p.moves[3 * move + 2];
        if ((unsigned)src >= (unsigned)p.num_pages || (unsigned)dst >= (unsigned)p.num_pages ||
            rows < 0 || rows > p.block_size) {
            if (threadIdx.x == 0) report_error(p.err, ATTN_ERR_BOUNDS);
            continue;
        }
        if (src == dst) continue;
        uint8_t *base = tensor == 0 ? p.cache[c].k : p.cache[c].v;
        const uint4 *from = reinterpret_cast<const uint4 *>(base) + (int64_t)src * p.page_pieces;
        uint4 *to = reinterpret_cast<uint4 *>(base) + (int64_t)dst * p.page_pieces;
        const int live = rows * p.row_pieces;  // pieces of a run to copy
        const int first = seg * kCopyThreads * kCopyUnroll + threadIdx.x;
        uint4 x[kCopyUnroll];
        bool on[kCopyUnroll];
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u) {
            const int i = first + u * kCopyThreads;
            on[u] = i < p.page_pieces &&
                    (p.run_pieces == p.page_pieces ? i : i % p.run_pieces) < live;
            if (on[u]) x[u] = from[i];
        }
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u)
            if (on[u]) to[first + u * kCopyThreads] = x[u];
        float *scales = tensor == 0 ? p.cache[c].ks : p.cache[c].vs;
        if (seg == 0 && scales != nullptr) {
            const int per_page = p.block_size / p.scale_block * p.n_kv_heads;
            const int count = (rows + p.scale_block - 1) / p.scale_block * p.n_kv_heads;
            for (int i = threadIdx.x; i < count; i += kCopyThreads)
                scales[(int64_t)dst * per_page + i] = scales[(int64_t)src * per_page + i];
        }
    }
}

int status(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

}  // namespace

int launch_pages_free(int32_t *block_table, int max_blocks, int table_rows, const int32_t *rows,
                      const int32_t *from_block, const int32_t *to_block, int n, int32_t *refs,
                      int num_pages, int32_t *err, cudaStream_t stream) {
    if (n == 0) return ATTN_OK;
    const int per_row = (max_blocks + 255) / 256;
    if ((int64_t)n * per_row >= (int64_t(1) << 31)) return ATTN_ERR_SHAPE;
    return status(launch_pdl(pages_free_kernel, dim3((unsigned)(n * per_row)), dim3(256), 0, stream,
                             block_table, max_blocks, table_rows, rows, from_block, to_block, n,
                             per_row, refs, num_pages, err));
}

int launch_pages_reserve(int32_t *block_table, int max_blocks, int table_rows,
                         const int32_t *rows, const int32_t *from_block, const int32_t *to_block,
                         int n, int32_t *refs, int num_pages, int32_t *err, cudaStream_t stream) {
    if (n == 0) return ATTN_OK;
    return status(launch_pdl(pages_reserve_kernel, dim3(1), dim3(kScanThreads), 0, stream,
                             block_table, max_blocks, table_rows, rows, from_block, to_block, n,
                             refs, num_pages, err));
}

int launch_pages_fork(int32_t *block_table, int max_blocks, int table_rows,
                      const int32_t *src_rows, const int32_t *dst_rows, const int32_t *seq_lens,
                      int n, int block_size, int32_t *refs, int num_pages, int32_t *moves,
                      int32_t *n_moves, int32_t *err, cudaStream_t stream) {
    ForkParams p = {block_table, max_blocks, table_rows, src_rows, dst_rows, seq_lens, n,
                    block_size,  refs,       num_pages,  moves,    n_moves,  err,
                    (int64_t)n * max_blocks <= kForkEntries};
    if (!p.share) {
        const int per_row = (max_blocks + 255) / 256;
        if ((int64_t)n * per_row >= (int64_t(1) << 31)) return ATTN_ERR_SHAPE;
        const int rc = status(launch_pdl(pages_share_kernel, dim3((unsigned)(n * per_row)),
                                         dim3(256), 0, stream, p, per_row));
        if (rc != ATTN_OK) return rc;
    }
    return status(launch_pdl(pages_fork_kernel, dim3(kForkBlocks), dim3(kScanThreads), 0, stream,
                             p));
}

size_t pages_workspace(int num_pages) { return (size_t)num_pages * sizeof(int32_t); }

int launch_pages_compact(int32_t *block_table, int max_blocks, int table_rows, int block_size,
                         int32_t *refs, int num_pages, int32_t *moves, int max_moves,
                         int32_t *n_moves, int32_t *used, void *workspace, int32_t *err,
                         cudaStream_t stream) {
    int32_t *to = static_cast<int32_t *>(workspace);
    const int rc = status(launch_pdl(pages_plan_compact_kernel, dim3(1), dim3(kScanThreads), 0,
                                     stream, refs, num_pages, block_size, moves, max_moves, n_moves,
                                     used, to, err));
    const int64_t entries = (int64_t)max_blocks * table_rows;
    if (rc != ATTN_OK || entries == 0) return rc;
    const int64_t blocks = std::min<int64_t>((entries + 255) / 256, (int64_t)device_sm_count() * 8);
    return status(launch_pdl(pages_rename_kernel, dim3((unsigned)blocks), dim3(256), 0, stream,
                             block_table, entries, (const int32_t *)to, (const int32_t *)used,
                             num_pages, err));
}

int launch_pages_copy(const attn_kv_cache *caches, int n_caches, int n_kv_heads, int head_dim,
                      const int32_t *moves, const int32_t *n_moves, int max_moves, int32_t *err,
                      cudaStream_t stream) {
    if (max_moves == 0) return ATTN_OK;
    const attn_kv_cache &c0 = caches[0];
    const int64_t row_bytes = head_dim * (c0.dtype == ATTN_KV_BF16 ? 2 : 1);
    CopyParams p = {};
    p.moves = moves;
    p.n_moves = n_moves;
    p.max_moves = max_moves;
    p.num_pages = (int)(c0.num_slots / c0.block_size);
    p.block_size = c0.block_size;
    p.page_pieces = (int)(c0.block_size * row_bytes * n_kv_heads / 16);
    const bool head_major = c0.layout == ATTN_LAYOUT_BHSD;
    p.run_pieces = head_major ? (int)(c0.block_size * row_bytes / 16) : p.page_pieces;
    p.row_pieces = (int)((head_major ? 1 : n_kv_heads) * row_bytes / 16);
    p.scale_block = kv_scaled(c0.dtype) ? c0.scale_block : c0.block_size;
    p.n_kv_heads = n_kv_heads;
    constexpr int kStep = kCopyThreads * kCopyUnroll;
    p.segments = (p.page_pieces + kStep - 1) / kStep;
    p.err = err;
    for (int base = 0; base < n_caches; base += kCopyCaches) {
        p.n_caches = std::min(kCopyCaches, n_caches - base);
        for (int i = 0; i < p.n_caches; ++i) {
            const attn_kv_cache &c = caches[base + i];
            const bool scaled = kv_scaled(c.dtype);
            p.cache[i] = {static_cast<uint8_t *>(c.k), static_cast<uint8_t *>(c.v),
                          scaled ? c.k_scale : nullptr, scaled ? c.v_scale : nullptr};
        }
        const int64_t steps = (int64_t)max_moves * p.n_caches * 2 * p.segments;
        const int64_t blocks = std::min<int64_t>(steps, (int64_t)device_sm_count() * 8);
        const int rc = status(launch_pdl(pages_copy_kernel, dim3((unsigned)blocks),
                                         dim3(kCopyThreads), 0, stream, p));
        if (rc != ATTN_OK) return rc;
    }
    return ATTN_OK;
}

}  // namespace gqa
