// gad_pages.cuh - page operations of the paged cache: forking, extending,
// freeing and compacting page tables over a reference-counted pool, and
// copying pages between places of the pool.
//
// State (all the caller's): a page table [rows, max_pages] with a length in
// tokens per row (negative: the row holds no request), and one reference count
// per page of the pool (0: the page is free).  Row r holds the pages
// table[r][0 .. ceil(len / page_size)).  Free pages are handed out lowest id
// first, row by row, so every result is a function of the inputs: the
// reference counts are whole numbers, and the order in which atomics reach
// them changes nothing.
//
// Handing out pages needs the k-th free page for k = 0, 1, ...: one pass counts
// the free pages per chunk of the pool (count_kernel), a second one ranks the
// free pages of each chunk behind the sum of the chunks before it and gives
// each to its row.  Both read the counts once (4 bytes a page).  Page ids
// outside [0, num_pages) are skipped everywhere.
#pragma once

#include <cooperative_groups.h>
#include <cstdint>

#include "gad_ptx.cuh"

namespace gad {
namespace pg {

constexpr int THREADS = 256;
constexpr int CHUNK = 4096;          // pages per chunk, unless the pool has more than MAX_CHUNKS of them
constexpr int MAX_CHUNKS = 1024;
constexpr int MAX_ROWS = 4096;
constexpr int COLS = 4096;           // table columns per block
constexpr int FREE_CLUSTER = 8;      // blocks that share a row in free_kernel
constexpr int MAX_CACHES = 64;       // caches per copy launch

// Pages per chunk: CHUNK, or the smallest multiple of it with at most MAX_CHUNKS chunks.
__host__ __device__ inline long long chunk_pages(long long num_pages) {
    const long long c = (num_pages + MAX_CHUNKS - 1) / MAX_CHUNKS;
    return (c + CHUNK - 1) / CHUNK * CHUNK;
}

// Workspace head: the status word at offset 0, then what one kernel of a call
// leaves for the next.
struct Head {
    int status;           // GAD_STATUS_PAGES_* bits
    int need_list;        // fork: rows that need a fresh page
    int row_overflow;     // extend: a row would outgrow the table
    int moves;            // compact: pages that move
    long long need;       // extend: pages that are needed in all
    long long total;      // compact: pages in use
};

struct Ws {
    Head* head;
    int* counts;          // [MAX_CHUNKS] free pages per chunk
    int* rows;            // [2 MAX_ROWS] per-row values
    long long* prefix;    // [MAX_ROWS + 1]
    int* rank;            // [num_pages], compact
};

struct Pool {
    int* refs;
    long long num_pages, chunk;
    int chunks;
};

__device__ __forceinline__ int pages_of(int len, int shift, int max_pages) {
    if (len <= 0) return 0;
    const long long n = (static_cast<long long>(len) + (1 << shift) - 1) >> shift;
    return n < max_pages ? static_cast<int>(n) : max_pages;
}
// Whether the row's last page is partly filled (and inside the table).
__device__ __forceinline__ bool has_partial(int len, int shift, int max_pages) {
    if (len <= 0 || (len & ((1 << shift) - 1)) == 0) return false;
    return ((static_cast<long long>(len) + (1 << shift) - 1) >> shift) <= max_pages;
}

// Exclusive prefix of v over the block's threads; *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int* total) {
    __shared__ int warp_sum[THREADS / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();  // the previous call's readers are done
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        const int s = warp_sum[w];
        if (w < warp) before += s;
        all += s;
    }
    *total = all;
    return before + x - v;
}
__device__ __forceinline__ long long block_sum(long long v) {
    __shared__ long long warp_sum[THREADS / 32];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = v;
    __syncthreads();
    long long s = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) s += warp_sum[w];
    return s;
}

// Four counts from page i on (i a multiple of 4); pages past the pool count as
// in use by `past`.
__device__ __forceinline__ int4 refs4(const Pool& p, long long i, int past) {
    if (i + 4 <= p.num_pages) return *reinterpret_cast<const int4*>(p.refs + i);
    int4 r = make_int4(past, past, past, past);
    if (i < p.num_pages) r.x = p.refs[i];
    if (i + 1 < p.num_pages) r.y = p.refs[i + 1];
    if (i + 2 < p.num_pages) r.z = p.refs[i + 2];
    return r;
}

// Free pages in the chunks before `chunk`, and in all of them.
__device__ __forceinline__ void free_before(const Ws& ws, int chunks, int chunk, long long* before,
                                            long long* total) {
    long long b = 0, t = 0;
    for (int i = threadIdx.x; i < chunks; i += THREADS) {
        const int c = ws.counts[i];
        t += c;
        if (i < chunk) b += c;
    }
    *before = block_sum(b);
    *total = block_sum(t);
}

}  // namespace pg

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------

struct ForkParams {
    const int *table, *lens, *parent;
    int *out_table, *out_lens, *copy_src, *copy_dst;
    int rows_in, rows_out, max_pages, shift;
    pg::Pool pool;
    pg::Ws ws;
};

// One block per (COLS columns, row): the row's old pages change their counts
// by its children - 1 (of a partly filled last page only the first child takes
// the page, so its count only falls when there is none), and the new row of
// that number takes its parent's entries.  The entry of a fresh last page is
// left to fork_assign_kernel.
template <bool VEC>
__global__ void __launch_bounds__(pg::THREADS) fork_kernel(const ForkParams p) {
    using namespace pg;
    __shared__ int s_kids, s_elder;
    const int y = blockIdx.y, tid = threadIdx.x;
    pdl_launch_dependents();
    if (tid == 0) s_kids = s_elder = 0;
    __syncthreads();
    const int par = y < p.rows_out ? p.parent[y] : -1;
    const bool alive = par >= 0 && par < p.rows_in;
    int kids = 0, elder = 0;
    for (int r = tid; r < p.rows_out; r += THREADS) {
        const int q = p.parent[r];
        kids += q == y;
        elder |= r < y && q == par;
    }
    if (kids) atomicAdd(&s_kids, kids);
    if (elder) s_elder = 1;
    __syncthreads();
    kids = s_kids;
    const bool fresh_last = alive && s_elder;   // and the parent's last page is partly filled (below)

    const int c0 = blockIdx.x * COLS;
    if (y < p.rows_in && kids != 1) {
        const int len = p.lens[y];
        const int n = pages_of(len, p.shift, p.max_pages);
        const int last = has_partial(len, p.shift, p.max_pages) ? n - 1 : -1;
        const int* row = p.table + static_cast<size_t>(y) * p.max_pages;
        const int end = min(n, c0 + COLS);
        for (int j = c0 + tid; j < end; j += THREADS) {
            const int page = row[j];
            const int d = (j == last ? min(kids, 1) : kids) - 1;
            if (d != 0 && page >= 0 && page < p.pool.num_pages) atomicAdd(p.pool.refs + page, d);
        }
    }
    if (y < p.rows_out) {
        const int len = alive ? p.lens[par] : -1;
        int n = pages_of(len, p.shift, p.max_pages);
        const bool fresh = fresh_last && has_partial(len, p.shift, p.max_pages);
        if (fresh) --n;
        const int* src = p.table + static_cast<size_t>(alive ? par : 0) * p.max_pages;
        int* dst = p.out_table + static_cast<size_t>(y) * p.max_pages;
        const int end = min(n, c0 + COLS);
        if (VEC) {
            const int end4 = c0 + (end > c0 ? (end - c0) / 4 * 4 : 0);
            for (int j = c0 + 4 * tid; j < end4; j += 4 * THREADS)
                *reinterpret_cast<int4*>(dst + j) = *reinterpret_cast<const int4*>(src + j);
            if (end4 + tid < end) dst[end4 + tid] = src[end4 + tid];
        } else {
            for (int j = c0 + tid; j < end; j += THREADS) dst[j] = src[j];
        }
        if (blockIdx.x == 0 && tid == 0) {
            p.out_lens[y] = len < 0 ? -1 : len;
            p.copy_src[y] = -1;
            p.copy_dst[y] = -1;
            p.ws.rows[y] = fresh ? 1 : 0;
            if (y == 0) p.ws.head->status = 0;
        }
    }
}

// Block c < chunks: free pages of chunk c.  Block `chunks`: the rows that need
// a fresh page, in order (fork).
__global__ void __launch_bounds__(pg::THREADS) fork_count_kernel(const ForkParams p) {
    using namespace pg;
    pdl_launch_dependents();
    pdl_wait_primary();
    const int tid = threadIdx.x;
    if (static_cast<int>(blockIdx.x) == p.pool.chunks) {
        int* list = p.ws.rows + MAX_ROWS;
        int at = 0;
        for (int r0 = 0; r0 < p.rows_out; r0 += THREADS) {
            const int r = r0 + tid;
            const int f = r < p.rows_out ? p.ws.rows[r] : 0;
            int total;
            const int k = block_scan(f, &total);
            if (f) list[at + k] = r;
            at += total;
        }
        if (tid == 0) p.ws.head->need_list = at;
        return;
    }
    const long long i0 = blockIdx.x * p.pool.chunk;
    const long long i1 = i0 + p.pool.chunk < p.pool.num_pages ? i0 + p.pool.chunk : p.pool.num_pages;
    long long n = 0;
    for (long long i = i0 + 4 * tid; i < i1; i += 4 * THREADS) {
        const int4 r = refs4(p.pool, i, 1);
        n += (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
    }
    n = block_sum(n);
    if (tid == 0) p.ws.counts[blockIdx.x] = static_cast<int>(n);
}

__global__ void __launch_bounds__(pg::THREADS) fork_assign_kernel(const ForkParams p, const int pool_bit) {
    using namespace pg;
    pdl_wait_primary();
    const int tid = threadIdx.x;
    const int need = p.ws.head->need_list;
    if (need == 0) return;
    const int* list = p.ws.rows + MAX_ROWS;
    long long before, total;
    free_before(p.ws, p.pool.chunks, blockIdx.x, &before, &total);
    if (blockIdx.x == 0 && total < need) {
        // the pool is used up: the rows at the end of the list keep their full pages
        for (int k = static_cast<int>(total) + tid; k < need; k += THREADS) {
            const int r = list[k];
            const int len = p.lens[p.parent[r]];
            p.out_lens[r] = len & ~((1 << p.shift) - 1);
        }
        if (tid == 0) atomicOr(&p.ws.head->status, pool_bit);
    }
    const long long i0 = blockIdx.x * p.pool.chunk;
    const long long i1 = i0 + p.pool.chunk < p.pool.num_pages ? i0 + p.pool.chunk : p.pool.num_pages;
    for (long long i = i0; i < i1 && before < need; i += 4 * THREADS) {
        const long long mine = i + 4 * tid;
        const int4 v = mine < i1 ? refs4(p.pool, mine, 1) : make_int4(1, 1, 1, 1);
        const int f[4] = {v.x == 0, v.y == 0, v.z == 0, v.w == 0};
        int sum;
        long long k = before + block_scan(f[0] + f[1] + f[2] + f[3], &sum);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (!f[u]) continue;
            if (k < need) {
                const int r = list[k], par = p.parent[r], len = p.lens[par];
                const int page = static_cast<int>(mine + u);
                const int j = pages_of(len, p.shift, p.max_pages) - 1;
                p.out_table[static_cast<size_t>(r) * p.max_pages + j] = page;
                p.copy_src[r] = p.table[static_cast<size_t>(par) * p.max_pages + j];
                p.copy_dst[r] = page;
                p.pool.refs[page] = 1;
            }
            ++k;
        }
        before += sum;
    }
}

// ---------------------------------------------------------------------------
// extend
// ---------------------------------------------------------------------------

struct ExtendParams {
    int *table, *lens;
    long long *positions, *cache_loc;
    int rows, L, max_pages, shift;
    pg::Pool pool;
    pg::Ws ws;
};

// Block c < chunks: free pages of chunk c.  Block `chunks`: each row's length
// and the pages that the rows before it need.
__global__ void __launch_bounds__(pg::THREADS) extend_count_kernel(const ExtendParams p) {
    using namespace pg;
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    if (static_cast<int>(blockIdx.x) == p.pool.chunks) {
        long long at = 0;
        bool over = false;
        for (int r0 = 0; r0 < p.rows; r0 += THREADS) {
            const int r = r0 + tid;
            int need = 0;
            if (r < p.rows) {
                const int len = p.lens[r];
                p.ws.rows[r] = len;
                if (len >= 0) {
                    const long long ps = 1 << p.shift;
                    const long long n_old = (len + ps - 1) >> p.shift;
                    const long long n_new = (static_cast<long long>(len) + p.L + ps - 1) >> p.shift;
                    need = static_cast<int>(n_new - n_old);
                    over |= n_new > p.max_pages;
                }
            }
            int total;
            const int k = block_scan(need, &total);   // at most THREADS * 65,536
            if (r < p.rows) p.ws.prefix[r] = at + k;
            at += total;
        }
        const int any = __syncthreads_or(over);
        if (tid == 0) {
            p.ws.prefix[p.rows] = at;
            p.ws.head->need = at;
            p.ws.head->row_overflow = any;
        }
        return;
    }
    const long long i0 = blockIdx.x * p.pool.chunk;
    const long long i1 = i0 + p.pool.chunk < p.pool.num_pages ? i0 + p.pool.chunk : p.pool.num_pages;
    long long n = 0;
    for (long long i = i0 + 4 * tid; i < i1; i += 4 * THREADS) {
        const int4 r = refs4(p.pool, i, 1);
        n += (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
    }
    n = block_sum(n);
    if (tid == 0) p.ws.counts[blockIdx.x] = static_cast<int>(n);
}

__global__ void __launch_bounds__(pg::THREADS)
    extend_assign_kernel(const ExtendParams p, const int pool_bit, const int row_bit) {
    using namespace pg;
    pdl_wait_primary();
    const int tid = threadIdx.x;
    const long long need = p.ws.head->need;
    const bool over = p.ws.head->row_overflow != 0;
    long long before, total;
    free_before(p.ws, p.pool.chunks, blockIdx.x, &before, &total);
    const bool ok = !over && need <= total;
    if (blockIdx.x == 0 && tid == 0)
        p.ws.head->status = (over ? row_bit : 0) | (need > total ? pool_bit : 0);

    // tokens in pages that the row has already (and those that get no place)
    const long long tokens = static_cast<long long>(p.rows) * p.L;
    const int mask = (1 << p.shift) - 1;
    for (long long t = static_cast<long long>(blockIdx.x) * THREADS + tid; t < tokens;
         t += static_cast<long long>(gridDim.x) * THREADS) {
        const int r = static_cast<int>(t / p.L), j = static_cast<int>(t % p.L);
        const int len = p.ws.rows[r];
        const long long pos = len < 0 ? 0 : static_cast<long long>(len) + j;
        p.positions[t] = pos;
        if (len < 0 || !ok) {
            p.cache_loc[t] = -1;
        } else if ((pos >> p.shift) < ((static_cast<long long>(len) + mask) >> p.shift)) {
            const int page = p.table[static_cast<size_t>(r) * p.max_pages + (pos >> p.shift)];
            p.cache_loc[t] = page < 0 || page >= p.pool.num_pages
                                 ? -1
                                 : (static_cast<long long>(page) << p.shift) + (pos & mask);
        }
    }
    if (!ok) return;
    if (blockIdx.x == 0)
        for (int r = tid; r < p.rows; r += THREADS)
            if (p.ws.rows[r] >= 0) p.lens[r] = p.ws.rows[r] + p.L;

    // fresh pages
    if (static_cast<int>(blockIdx.x) >= p.pool.chunks) return;
    const long long i0 = blockIdx.x * p.pool.chunk;
    const long long i1 = i0 + p.pool.chunk < p.pool.num_pages ? i0 + p.pool.chunk : p.pool.num_pages;
    for (long long i = i0; i < i1 && before < need; i += 4 * THREADS) {
        const long long mine = i + 4 * tid;
        const int4 v = mine < i1 ? refs4(p.pool, mine, 1) : make_int4(1, 1, 1, 1);
        const int f[4] = {v.x == 0, v.y == 0, v.z == 0, v.w == 0};
        int sum;
        long long k = before + block_scan(f[0] + f[1] + f[2] + f[3], &sum);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (!f[u]) continue;
            if (k < need) {
                int lo = 0, hi = p.rows - 1;   // the last row whose prefix is at most k
                while (lo < hi) {
                    const int mid = (lo + hi + 1) >> 1;
                    if (p.ws.prefix[mid] <= k) lo = mid;
                    else hi = mid - 1;
                }
                const int len = p.ws.rows[lo];
                const long long page = mine + u;
                const long long slot = ((static_cast<long long>(len) + mask) >> p.shift) + (k - p.ws.prefix[lo]);
                p.table[static_cast<size_t>(lo) * p.max_pages + slot] = static_cast<int>(page);
                p.pool.refs[page] = 1;
                long long j = (slot << p.shift) - len;
                if (j < 0) j = 0;
                for (; j < p.L && ((len + j) >> p.shift) == slot; ++j)
                    p.cache_loc[static_cast<long long>(lo) * p.L + j] = (page << p.shift) + ((len + j) & mask);
            }
            ++k;
        }
        before += sum;
    }
}

// ---------------------------------------------------------------------------
// free
// ---------------------------------------------------------------------------

struct FreeParams {
    const int* table;
    int* lens;
    const uint8_t* leave;
    int rows, max_pages, shift;
    int* refs;
    long long num_pages;
};

// One cluster per row: its blocks read the length, take turns at the entries
// and, once all have read it, mark the row empty.
__global__ void __cluster_dims__(pg::FREE_CLUSTER, 1, 1) __launch_bounds__(pg::THREADS)
    free_kernel(const FreeParams p) {
    using namespace pg;
    const int r = blockIdx.x / FREE_CLUSTER, part = blockIdx.x % FREE_CLUSTER;
    if (p.leave != nullptr && p.leave[r] == 0) return;   // the whole cluster
    const int n = pages_of(p.lens[r], p.shift, p.max_pages);
    cooperative_groups::this_cluster().sync();
    if (part == 0 && threadIdx.x == 0) p.lens[r] = -1;
    const int* row = p.table + static_cast<size_t>(r) * p.max_pages;
    for (int j = part * THREADS + threadIdx.x; j < n; j += FREE_CLUSTER * THREADS) {
        const int page = row[j];
        if (page >= 0 && page < p.num_pages) atomicAdd(p.refs + page, -1);
    }
}

// ---------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------

struct CompactParams {
    int* table;
    const int* lens;
    int *copy_src, *copy_dst, *used;
    int rows, max_pages, shift, max_moves;
    pg::Pool pool;
    pg::Ws ws;
};

__global__ void __launch_bounds__(pg::THREADS) compact_count_kernel(const CompactParams p) {
    using namespace pg;
    pdl_launch_dependents();
    const long long i0 = blockIdx.x * p.pool.chunk;
    const long long i1 = i0 + p.pool.chunk < p.pool.num_pages ? i0 + p.pool.chunk : p.pool.num_pages;
    long long n = 0;
    for (long long i = i0 + 4 * threadIdx.x; i < i1; i += 4 * THREADS) {
        const int4 r = refs4(p.pool, i, 1);
        n += (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
    }
    n = block_sum(n);
    if (threadIdx.x == 0) p.ws.counts[blockIdx.x] = static_cast<int>(n);
}

// With `total` pages in use, the k-th page in use at or above `total` moves to
// the k-th free page below it: sources and destinations are two disjoint
// ranges of the pool, and no page moves that need not.
__global__ void __launch_bounds__(pg::THREADS) compact_rank_kernel(const CompactParams p) {
    using namespace pg;
    pdl_launch_dependents();
    pdl_wait_primary();
    const int tid = threadIdx.x;
    long long free_base, free_all;
    free_before(p.ws, p.pool.chunks, blockIdx.x, &free_base, &free_all);
    const long long total = p.pool.num_pages - free_all;
    // free pages below `total` = pages that would move
    long long holes, unused;
    const int edge = static_cast<int>(total / p.pool.chunk);   // the chunk that `total` lies in
    free_before(p.ws, p.pool.chunks, edge, &holes, &unused);
    long long n = 0;
    for (long long i = edge * p.pool.chunk + tid; i < total; i += THREADS) n += p.pool.refs[i] == 0;
    holes += block_sum(n);
    const int moves = static_cast<int>(holes < p.max_moves ? holes : p.max_moves);
    if (blockIdx.x == 0 && tid == 0) {
        p.used[0] = static_cast<int>(total);
        p.ws.head->total = total;
        p.ws.head->moves = moves;
        p.ws.head->status = 0;
    }
    for (long long k = moves + static_cast<long long>(blockIdx.x) * THREADS + tid; k < p.max_moves;
         k += static_cast<long long>(gridDim.x) * THREADS) {
        p.copy_src[k] = -1;
        p.copy_dst[k] = -1;
    }
    // Pages in use below `total`: total - holes.
    const long long kept = total - holes;
    const long long i0 = blockIdx.x * p.pool.chunk;
    const long long i1 = i0 + p.pool.chunk < p.pool.num_pages ? i0 + p.pool.chunk : p.pool.num_pages;
    for (long long i = i0; i < i1; i += 4 * THREADS) {
        const long long mine = i + 4 * tid;
        const int4 v = mine < i1 ? refs4(p.pool, mine, 1) : make_int4(1, 1, 1, 1);
        const int f[4] = {v.x == 0, v.y == 0, v.z == 0, v.w == 0};
        int sum;
        long long k = free_base + block_scan(f[0] + f[1] + f[2] + f[3], &sum);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const long long id = mine + u;
            if (f[u]) {
                if (id < total && k < moves) p.copy_dst[k] = static_cast<int>(id);
                ++k;
            } else if (id < i1 && id >= total) {
                const long long m = id - k - kept;   // id - k pages in use come before this one
                if (m < moves) {
                    p.copy_src[m] = static_cast<int>(id);
                    p.ws.rank[id] = static_cast<int>(m);
                } else {
                    p.ws.rank[id] = -1;
                }
            }
        }
        free_base += sum;
    }
}

// Block y < rows: the row's entries follow their pages.  Block y == rows: so do
// the counts.
__global__ void __launch_bounds__(pg::THREADS) compact_apply_kernel(const CompactParams p) {
    using namespace pg;
    pdl_wait_primary();
    const int moves = p.ws.head->moves;
    const long long total = p.ws.head->total;
    if (static_cast<int>(blockIdx.y) == p.rows) {
        for (int k = blockIdx.x * THREADS + threadIdx.x; k < moves; k += gridDim.x * THREADS) {
            const int s = p.copy_src[k], d = p.copy_dst[k];
            p.pool.refs[d] = p.pool.refs[s];
            p.pool.refs[s] = 0;
        }
        return;
    }
    const int n = pages_of(p.lens[blockIdx.y], p.shift, p.max_pages);
    int* row = p.table + static_cast<size_t>(blockIdx.y) * p.max_pages;
    for (long long j = static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x; j < n;
         j += static_cast<long long>(gridDim.x) * THREADS) {
        const int page = row[j];
        if (page >= total && page < p.pool.num_pages) {
            const int k = p.ws.rank[page];
            // an entry whose page is free has no rank of this call: it stays
            if (k >= 0 && k < moves && p.copy_src[k] == page) row[j] = p.copy_dst[k];
        }
    }
}

// ---------------------------------------------------------------------------
// copy
// ---------------------------------------------------------------------------

struct CopyParams {
    uint8_t* cache[pg::MAX_CACHES];
    const int *src, *dst;
    int n, chunks, lanes;      // 16-byte chunks per page, threads per page (a power of two)
    long long num_pages;
    size_t page_bytes;
};

// A page is copied by `lanes` threads, 16 bytes each at a time, four loads of
// a thread in flight before its stores: over four pairs when a page is one
// chunk a thread (WIDE false), else over four chunks of one pair.
template <bool WIDE>
__global__ void __launch_bounds__(pg::THREADS) pages_copy_kernel(const CopyParams p) {
    using namespace pg;
    const int lane = threadIdx.x % p.lanes, group = threadIdx.x / p.lanes, groups = THREADS / p.lanes;
    uint8_t* cache = p.cache[blockIdx.y];
    if (!WIDE) {
        for (long long i0 = static_cast<long long>(blockIdx.x) * groups * 4 + group; i0 < p.n;
             i0 += static_cast<long long>(gridDim.x) * groups * 4) {
            uint4 v[4];
            uint4* to[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const long long i = i0 + static_cast<long long>(u) * groups;
                to[u] = nullptr;
                if (i < p.n && lane < p.chunks) {
                    const int s = p.src[i], d = p.dst[i];
                    if (s >= 0 && d >= 0 && s < p.num_pages && d < p.num_pages) {
                        v[u] = reinterpret_cast<const uint4*>(cache + s * p.page_bytes)[lane];
                        to[u] = reinterpret_cast<uint4*>(cache + d * p.page_bytes) + lane;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (to[u] != nullptr) *to[u] = v[u];
        }
    } else {
        for (long long i = static_cast<long long>(blockIdx.x) * groups + group; i < p.n;
             i += static_cast<long long>(gridDim.x) * groups) {
            const int s = p.src[i], d = p.dst[i];
            if (s < 0 || d < 0 || s >= p.num_pages || d >= p.num_pages) continue;
            const uint4* from = reinterpret_cast<const uint4*>(cache + s * p.page_bytes);
            uint4* to = reinterpret_cast<uint4*>(cache + d * p.page_bytes);
            for (int c0 = lane; c0 < p.chunks; c0 += 4 * p.lanes) {
                uint4 v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (c0 + u * p.lanes < p.chunks) v[u] = from[c0 + u * p.lanes];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (c0 + u * p.lanes < p.chunks) to[c0 + u * p.lanes] = v[u];
            }
        }
    }
}

}  // namespace gad
