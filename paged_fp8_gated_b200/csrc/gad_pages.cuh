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
// the free pages per chunk of the pool, a second one ranks the free pages of
// each chunk behind the sum of the chunks before it and gives each to its row.
// Both read the counts once (4 bytes a page).  A pool of at most SMALL_POOL pages
// is looked at by one cluster, which keeps the free pages as bits between the
// two and saves a launch.  Page ids outside [0, num_pages) are skipped
// everywhere.
//
// Every operation but the copy moves a few megabytes through chains of dependent
// loads (length, entry, count) over one to three launches, so latency is the
// bound: see the kernels for what they take.
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
constexpr int ROWS = 8;              // fork: table rows per block
constexpr int RUN = CHUNK / THREADS; // pages of a chunk that a thread looks at
constexpr int EARLY_CHUNKS = 16;     // chunks that extend looks at before it knows that it must
constexpr int SMALL_BLOCKS = 8, SMALL_THREADS = 512;   // the cluster for a small pool
constexpr int SMALL_POOL = SMALL_BLOCKS * SMALL_THREADS * 16;
constexpr int LIST = 2048;           // free pages that are handed out at a time
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
    int need;             // extend: pages that are needed in all (at most 2^28)
    int total;            // compact: pages in use
};

struct Ws {
    Head* head;
    unsigned* counts;     // [MAX_CHUNKS] free pages per chunk
    int* rows;            // [2 MAX_ROWS] per-row values
    int* prefix;          // [MAX_ROWS + 1]
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

// Exclusive prefix of v over the block's T threads; *total gets the sum.
template <int T>
__device__ __forceinline__ int block_scan(int v, int* total) {
    __shared__ int warp_sum[T / 32];
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
    const int s = lane < T / 32 ? warp_sum[lane] : 0;   // every warp adds the warps' sums up
    *total = __reduce_add_sync(0xffffffffu, s);
    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? s : 0);
    return before + x - v;
}
// Sums of a and b over the block's T threads (below 2^32).
template <int T>
__device__ __forceinline__ uint2 block_sum2(unsigned a, unsigned b) {
    __shared__ uint2 warp_sum[T / 32];
    const int lane = threadIdx.x & 31;
    a = __reduce_add_sync(0xffffffffu, a);
    b = __reduce_add_sync(0xffffffffu, b);
    __syncthreads();  // the previous call's readers are done
    if (lane == 0) warp_sum[threadIdx.x >> 5] = make_uint2(a, b);
    __syncthreads();
    const uint2 s = lane < T / 32 ? warp_sum[lane] : make_uint2(0, 0);
    return make_uint2(__reduce_add_sync(0xffffffffu, s.x), __reduce_add_sync(0xffffffffu, s.y));
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

// Which of the RUN pages from i on are free, as bits (i a multiple of 4).
__device__ __forceinline__ unsigned free_bits(const Pool& p, long long i, long long end) {
    unsigned bits = 0;
#pragma unroll
    for (int u = 0; u < RUN; u += 4) {
        const int4 r = i + u < end ? refs4(p, i + u, 1) : make_int4(1, 1, 1, 1);
        bits |= static_cast<unsigned>((r.x == 0) | (r.y == 0) << 1 | (r.z == 0) << 2 | (r.w == 0) << 3) << u;
    }
    return bits;
}
__device__ __forceinline__ long long chunk_end(const Pool& p, int chunk) {
    const long long e = (chunk + 1) * p.chunk;
    return e < p.num_pages ? e : p.num_pages;
}
// Free pages of a chunk (all threads get the sum).
__device__ __forceinline__ unsigned count_chunk(const Pool& p, int chunk) {
    const long long end = chunk_end(p, chunk);
    unsigned n = 0;
    for (long long i = chunk * p.chunk + RUN * threadIdx.x; i < end; i += CHUNK)
        n += __popc(free_bits(p, i, end));
    return block_sum2<THREADS>(n, 0).x;
}
// Free pages in the chunks before `chunk` (x), and in all of them (y).
__device__ __forceinline__ uint2 free_before(const Ws& ws, int chunks, int chunk) {
    unsigned b = 0, t = 0;
    for (int i = threadIdx.x; i < chunks; i += THREADS) {
        const unsigned c = ws.counts[i];
        t += c;
        if (i < chunk) b += c;
    }
    return block_sum2<THREADS>(b, t);
}

// give(page, before + q) for the first n free pages of a block's stretch of the
// pool, q = 0 .. n - 1: a thread's free pages are `bits` from page `mine` on,
// `rank` of the stretch's come before them.  The pages go through shared memory
// so that all threads give (a give is a chain of loads).
template <int T, class F>
__device__ __forceinline__ void hand_out(unsigned bits, long long mine, int rank, int n, long long before, F give) {
    __shared__ int s_list[LIST];
    for (int lo = 0; lo < n; lo += LIST) {
        __syncthreads();
        int q = rank - lo;
        for (unsigned b = bits; b != 0 && q < LIST; ++q, b &= b - 1)
            if (q >= 0) s_list[q] = static_cast<int>(mine + __ffs(b) - 1);
        __syncthreads();
        const int m = n - lo < LIST ? n - lo : LIST;
        for (int i = threadIdx.x; i < m; i += T) give(static_cast<long long>(s_list[i]), before + lo + i);
    }
}
// The same for a chunk, `before` free pages in the chunks before it, ranks below
// `need`; `bits`: those of its first CHUNK pages.
template <class F>
__device__ __forceinline__ void hand_out_chunk(const Pool& p, int chunk, unsigned bits, long long before, long long need,
                                               F give) {
    const long long end = chunk_end(p, chunk);
    for (long long i0 = chunk * p.chunk; i0 < end && before < need; i0 += CHUNK) {
        const long long mine = i0 + RUN * threadIdx.x;
        if (i0 != chunk * p.chunk) bits = mine < end ? free_bits(p, mine, end) : 0;
        int sum;
        const int rank = block_scan<THREADS>(__popc(bits), &sum);
        hand_out<THREADS>(bits, mine, rank, static_cast<int>(sum < need - before ? sum : need - before), before, give);
        before += sum;
    }
}
// A pool of at most SMALL_POOL pages as a cluster's threads see it.
struct Small {
    unsigned bits;      // the thread's free pages from page `mine` on
    int mine;
    int rank, sum;      // free pages before them in the block, and in the block
};
__device__ __forceinline__ Small look_small(const Pool& p, int block) {
    Small s;
    s.mine = (block * SMALL_THREADS + static_cast<int>(threadIdx.x)) * RUN;
    s.bits = free_bits(p, s.mine, p.num_pages);
    s.rank = block_scan<SMALL_THREADS>(__popc(s.bits), &s.sum);
    return s;
}
// What every block of the cluster has in `mine` (one value in all its threads),
// added up: over the blocks before this one (x), over all of them (y).  Each
// block stores its own in all of them, so one barrier does: behind it a block
// reads its own memory only.  Call I = 0, 1, ... of the kernel has places of its
// own; the first needs cluster_begin at the kernel's start, so that every block
// is there to be stored to.
__device__ __forceinline__ void cluster_begin() { cooperative_groups::this_cluster().barrier_arrive(); }
template <int I>
__device__ __forceinline__ uint2 cluster_sum(unsigned mine, int block) {
    __shared__ unsigned s_sums[SMALL_BLOCKS];
    const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    if (I == 0) cluster.barrier_wait();
    if (threadIdx.x < SMALL_BLOCKS) *cluster.map_shared_rank(&s_sums[block], threadIdx.x) = mine;
    cluster.sync();
    const int lane = threadIdx.x & 31;
    const unsigned v = lane < SMALL_BLOCKS ? s_sums[lane] : 0;
    return make_uint2(__reduce_add_sync(0xffffffffu, lane < block ? v : 0), __reduce_add_sync(0xffffffffu, v));
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

// One block per (U THREADS columns, ROWS rows).  An old row's pages change their
// counts by its children - 1 (of a partly filled last page only the first child
// takes the page, so its count only falls when there is none); a new row takes
// its parent's entries.  The entry of a fresh last page is left to
// fork_assign_kernel.  Rows that share pages are usually neighbours (the beams
// of a request): a thread adds up what its rows change about the page that they
// have in common in a column, and a count is touched only if something is left.
// Tables that leave the GPU with few blocks take one column a thread (U = 1),
// larger ones four, as vectors if the rows allow it (VEC).
// 128 new rows of 30,000 single-token pages (38 MB) 8.6 us, 64 of 940 pages 7.4;
// the counts' atomics, one for a page that several rows share, are its slow part.
template <int U, bool VEC>
__global__ void __launch_bounds__(pg::THREADS) fork_kernel(const ForkParams p) {
    using namespace pg;
    __shared__ int s_kids[ROWS], s_elder[ROWS], s_par[ROWS];
    // what is to be known of an old row: entries to look at (none, if its one child
    // takes them all), the partly filled last one, the changes of the counts; of a
    // new one: entries that it takes over
    __shared__ int s_n[ROWS], s_last[ROWS], s_take[ROWS];
    const int y0 = blockIdx.y * ROWS, tid = threadIdx.x;
    pdl_launch_dependents();
    int len = -1, new_len = -1;
    if (tid < ROWS) {
        const int y = y0 + tid;
        int par = y < p.rows_out ? p.parent[y] : -1;
        if (par >= p.rows_in) par = -1;
        s_kids[tid] = s_elder[tid] = 0;
        s_par[tid] = par;
        len = y < p.rows_in ? p.lens[y] : -1;
        new_len = par >= 0 ? p.lens[par] : -1;
    }
    __syncthreads();
    for (int r = tid; r < p.rows_out; r += THREADS) {
        const int q = p.parent[r];
        if (q >= y0 && q < y0 + ROWS) atomicAdd(&s_kids[q - y0], 1);
#pragma unroll
        for (int k = 0; k < ROWS; ++k)
            if (r < y0 + k && q == s_par[k]) s_elder[k] = 1;
    }
    __syncthreads();
    if (tid < ROWS) {
        const int n = pages_of(len, p.shift, p.max_pages);
        s_n[tid] = s_kids[tid] == 1 ? 0 : n;
        s_last[tid] = has_partial(len, p.shift, p.max_pages) ? n - 1 : -1;
        const bool fresh = s_elder[tid] && has_partial(new_len, p.shift, p.max_pages);
        s_take[tid] = pages_of(new_len, p.shift, p.max_pages) - fresh;
        const int y = y0 + tid;
        if (blockIdx.x == 0 && y < p.rows_out) {
            p.out_lens[y] = new_len < 0 ? -1 : new_len;
            p.copy_src[y] = -1;
            p.copy_dst[y] = -1;
            p.ws.rows[y] = fresh;
            if (y == 0) p.ws.head->status = 0;
        }
    }
    __syncthreads();

    const int c0 = blockIdx.x * (U * THREADS);
    auto col = [&](int u) { return VEC ? c0 + U * tid + u : c0 + u * THREADS + tid; };
    // the entries of a row (any value from `n` on)
    auto entries = [&](int (&e)[U], const int* row, int n) {
        if (VEC) {
            const int4 q = col(0) < n ? *reinterpret_cast<const int4*>(row + col(0)) : make_int4(-1, -1, -1, -1);
            e[0] = q.x; e[1 % U] = q.y; e[2 % U] = q.z; e[3 % U] = q.w;
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) e[u] = col(u) < n ? row[col(u)] : -1;
        }
    };
    int e[ROWS][U];   // all rows' entries at a time
    const int* old = p.table + static_cast<size_t>(y0) * p.max_pages;
#pragma unroll
    for (int k = 0; k < ROWS; ++k, old += p.max_pages) entries(e[k], old, s_n[k]);
    int page[U], left[U];
#pragma unroll
    for (int u = 0; u < U; ++u) page[u] = -1, left[u] = 0;
    auto flush = [&](int u) {
        if (left[u] != 0 && static_cast<unsigned>(page[u]) < static_cast<unsigned>(p.pool.num_pages))
            atomicAdd(p.pool.refs + page[u], left[u]);
    };
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        const int n = s_n[k], last = s_last[k], kids = s_kids[k];
        if (n <= c0) continue;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int d = col(u) >= n ? 0 : (col(u) == last ? min(kids, 1) : kids) - 1;
            if (d != 0 && e[k][u] != page[u]) {
                flush(u);
                page[u] = e[k][u];
                left[u] = 0;
            }
            left[u] += d;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) flush(u);

#pragma unroll
    for (int k = 0; k < ROWS; ++k)
        entries(e[k], p.table + static_cast<size_t>(max(s_par[k], 0)) * p.max_pages, s_take[k]);
    int* dst = p.out_table + static_cast<size_t>(y0) * p.max_pages;
#pragma unroll
    for (int k = 0; k < ROWS; ++k, dst += p.max_pages) {
        const int n = s_take[k];
        if (VEC && col(U - 1) < n) {
            *reinterpret_cast<int4*>(dst + col(0)) = make_int4(e[k][0], e[k][1 % U], e[k][2 % U], e[k][3 % U]);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (col(u) < n) dst[col(u)] = e[k][u];
        }
    }
}

// The rows that need a fresh page, in order: how many.
template <int T>
__device__ __forceinline__ int fork_list(const ForkParams& p, int* list) {
    int at = 0;
    for (int r0 = 0; r0 < p.rows_out; r0 += T) {
        const int r = r0 + threadIdx.x;
        const int f = r < p.rows_out ? p.ws.rows[r] : 0;
        int total;
        const int k = pg::block_scan<T>(f, &total);
        if (f) list[at + k] = r;
        at += total;
    }
    return at;
}
// Row r's fresh page.
__device__ __forceinline__ void fork_give(const ForkParams& p, int r, int page) {
    const int par = p.parent[r], j = pg::pages_of(p.lens[par], p.shift, p.max_pages) - 1;
    p.out_table[static_cast<size_t>(r) * p.max_pages + j] = page;
    p.copy_src[r] = p.table[static_cast<size_t>(par) * p.max_pages + j];
    p.copy_dst[r] = page;
    p.pool.refs[page] = 1;
}
// The pool is used up after `got` pages: the rows at the end of the list keep
// their full pages.
template <int T>
__device__ __forceinline__ void fork_short(const ForkParams& p, const int* list, int got, int need, int pool_bit) {
    for (int k = got + threadIdx.x; k < need; k += T) {
        const int r = list[k];
        p.out_lens[r] = p.lens[p.parent[r]] & ~((1 << p.shift) - 1);
    }
    if (threadIdx.x == 0) p.ws.head->status = pool_bit;
}

// Block c < chunks: free pages of chunk c.  Block `chunks`: the list.
__global__ void __launch_bounds__(pg::THREADS) fork_count_kernel(const ForkParams p) {
    using namespace pg;
    pdl_launch_dependents();
    pdl_wait_primary();
    const int tid = threadIdx.x;
    if (static_cast<int>(blockIdx.x) == p.pool.chunks) {
        const int n = fork_list<THREADS>(p, p.ws.rows + MAX_ROWS);
        if (tid == 0) p.ws.head->need_list = n;
        return;
    }
    const unsigned n = count_chunk(p.pool, blockIdx.x);
    if (tid == 0) p.ws.counts[blockIdx.x] = n;
}

__global__ void __launch_bounds__(pg::THREADS) fork_assign_kernel(const ForkParams p, const int pool_bit) {
    using namespace pg;
    pdl_wait_primary();
    const int chunk = blockIdx.x;
    const int need = p.ws.head->need_list;
    if (need == 0) return;
    const unsigned bits = free_bits(p.pool, chunk * p.pool.chunk + RUN * threadIdx.x, chunk_end(p.pool, chunk));
    const int* list = p.ws.rows + MAX_ROWS;
    const uint2 f = free_before(p.ws, p.pool.chunks, chunk);
    if (chunk == 0 && f.y < static_cast<unsigned>(need)) fork_short<THREADS>(p, list, f.y, need, pool_bit);
    hand_out_chunk(p.pool, chunk, bits, f.x, need,
                   [&](long long id, long long k) { fork_give(p, list[k], static_cast<int>(id)); });
}

// Both for a small pool.
__global__ void __cluster_dims__(pg::SMALL_BLOCKS, 1, 1) __launch_bounds__(pg::SMALL_THREADS)
    fork_assign_small_kernel(const ForkParams p, const int pool_bit) {
    using namespace pg;
    __shared__ int s_rows[MAX_ROWS];
    const int block = blockIdx.x;
    pdl_wait_primary();
    cluster_begin();
    const Small s = look_small(p.pool, block);
    const int need = fork_list<SMALL_THREADS>(p, s_rows);   // in every block
    const uint2 f = cluster_sum<0>(s.sum, block);
    const int before = static_cast<int>(f.x), total = static_cast<int>(f.y);
    if (block == 0 && total < need) fork_short<SMALL_THREADS>(p, s_rows, total, need, pool_bit);
    hand_out<SMALL_THREADS>(s.bits, s.mine, s.rank, min(s.sum, need - before), before,
                            [&](long long id, long long k) { fork_give(p, s_rows[k], static_cast<int>(id)); });
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

// Lengths, and the pages that the rows before each row need: put(r, len,
// before).  Returns the pages needed in all; *over: a row would outgrow the
// table.
template <int T, class F>
__device__ __forceinline__ int extend_rows(const ExtendParams& p, bool* over, F put) {
    int at = 0;
    bool big = false;
    for (int r0 = 0; r0 < p.rows; r0 += T) {
        const int r = r0 + threadIdx.x;
        int need = 0, len = -1;
        if (r < p.rows) {
            len = p.lens[r];
            if (len >= 0) {
                const long long ps = 1 << p.shift;
                const long long n_old = (len + ps - 1) >> p.shift;
                const long long n_new = (static_cast<long long>(len) + p.L + ps - 1) >> p.shift;
                need = static_cast<int>(n_new - n_old);
                big |= n_new > p.max_pages;
            }
        }
        int total;
        const int k = pg::block_scan<T>(need, &total);
        if (r < p.rows) put(r, len, at + k);
        at += total;
    }
    *over = __syncthreads_or(big) != 0;
    return at;
}
// Positions of the tokens t = first, first + stride ..., and cache rows of
// those in pages that the row has already (-1: no place).
template <class Len>
__device__ __forceinline__ void extend_tokens(const ExtendParams& p, unsigned first, unsigned stride, bool ok, Len lens) {
    const unsigned tokens = static_cast<unsigned>(p.rows) * p.L, L = p.L;   // at most 2^28
    const int mask = (1 << p.shift) - 1;
    for (unsigned t = first; t < tokens; t += stride) {
        const int r = static_cast<int>(t / L), j = static_cast<int>(t % L);
        const int len = lens(r);
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
}
// The k-th fresh page: its row is the last one with at most k pages needed
// before it.
__device__ __forceinline__ void extend_give(const ExtendParams& p, const int* prefix, const int* lens, long long page,
                                            long long k) {
    int lo = 0, hi = p.rows - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= k) lo = mid;
        else hi = mid - 1;
    }
    const int mask = (1 << p.shift) - 1;
    const long long len = lens[lo], slot = ((len + mask) >> p.shift) + (k - prefix[lo]);
    p.table[static_cast<size_t>(lo) * p.max_pages + slot] = static_cast<int>(page);
    p.pool.refs[page] = 1;
    long long j = (slot << p.shift) - len;
    if (j < 0) j = 0;
    for (; j < p.L && ((len + j) >> p.shift) == slot; ++j)
        p.cache_loc[static_cast<long long>(lo) * p.L + j] = (page << p.shift) + ((len + j) & mask);
}

// extend: 32 rows over a pool of 2.7 million pages 7.8 us in two launches, 256 rows
// over a small pool 6 in one.
// Block c < chunks: free pages of chunk c.  Block `chunks`: the rows.
__global__ void __launch_bounds__(pg::THREADS) extend_count_kernel(const ExtendParams p) {
    using namespace pg;
    pdl_launch_dependents();
    const int tid = threadIdx.x;
    if (static_cast<int>(blockIdx.x) == p.pool.chunks) {
        bool over;
        const int need = extend_rows<THREADS>(p, &over, [&](int r, int len, int before) {
            p.ws.rows[r] = len;
            p.ws.prefix[r] = before;
        });
        if (tid == 0) {
            p.ws.head->need = need;
            p.ws.head->row_overflow = over;
        }
        return;
    }
    const unsigned n = count_chunk(p.pool, blockIdx.x);
    if (tid == 0) p.ws.counts[blockIdx.x] = n;
}

__global__ void __launch_bounds__(pg::THREADS)
    extend_assign_kernel(const ExtendParams p, const int pool_bit, const int row_bit) {
    using namespace pg;
    __shared__ int s_prefix[MAX_ROWS], s_len[MAX_ROWS];
    const int tid = threadIdx.x, chunk = blockIdx.x;
    const bool pool_block = chunk < p.pool.chunks;
    // The counts change in this kernel only, a chunk by its own block.  Pages are
    // usually found in the first chunks, which look early.
    unsigned bits = 0;
    auto look = [&] { bits = free_bits(p.pool, chunk * p.pool.chunk + RUN * tid, chunk_end(p.pool, chunk)); };
    if (pool_block && chunk < EARLY_CHUNKS) look();
    pdl_wait_primary();
    const int need = p.ws.head->need;
    const bool over = p.ws.head->row_overflow != 0;
    const uint2 f = free_before(p.ws, p.pool.chunks, chunk);
    const bool enough = static_cast<unsigned>(need) <= f.y, ok = !over && enough;
    if (chunk == 0 && tid == 0) p.ws.head->status = (over ? row_bit : 0) | (enough ? 0 : pool_bit);
    extend_tokens(p, blockIdx.x * THREADS + tid, gridDim.x * THREADS, ok, [&](int r) { return p.ws.rows[r]; });
    if (!ok) return;
    if (chunk == 0)
        for (int r = tid; r < p.rows; r += THREADS)
            if (p.ws.rows[r] >= 0) p.lens[r] = p.ws.rows[r] + p.L;

    // fresh pages
    if (!pool_block || f.x >= static_cast<unsigned>(need)) return;
    if (chunk >= EARLY_CHUNKS) look();
    for (int r = tid; r < p.rows; r += THREADS) {
        s_prefix[r] = p.ws.prefix[r];
        s_len[r] = p.ws.rows[r];
    }
    hand_out_chunk(p.pool, chunk, bits, f.x, need,
                   [&](long long page, long long k) { extend_give(p, s_prefix, s_len, page, k); });
}

// Both for a small pool.
__global__ void __cluster_dims__(pg::SMALL_BLOCKS, 1, 1) __launch_bounds__(pg::SMALL_THREADS)
    extend_small_kernel(const ExtendParams p, const int pool_bit, const int row_bit) {
    using namespace pg;
    __shared__ int s_prefix[MAX_ROWS], s_len[MAX_ROWS];
    const int tid = threadIdx.x, block = blockIdx.x;
    cluster_begin();
    const Small s = look_small(p.pool, block);
    bool over;
    const int need = extend_rows<SMALL_THREADS>(p, &over, [&](int r, int len, int before) {   // in every block
        s_len[r] = len;
        s_prefix[r] = before;
    });
    const uint2 f = cluster_sum<0>(s.sum, block);   // and every block has read the lengths
    const int before = static_cast<int>(f.x);
    const bool enough = need <= static_cast<int>(f.y), ok = !over && enough;
    if (block == 0 && tid == 0) p.ws.head->status = (over ? row_bit : 0) | (enough ? 0 : pool_bit);
    extend_tokens(p, block * SMALL_THREADS + tid, SMALL_BLOCKS * SMALL_THREADS, ok, [&](int r) { return s_len[r]; });
    if (!ok) return;
    if (block == 0)
        for (int r = tid; r < p.rows; r += SMALL_THREADS)
            if (s_len[r] >= 0) p.lens[r] = s_len[r] + p.L;
    hand_out<SMALL_THREADS>(s.bits, s.mine, s.rank, min(s.sum, need - before), before,
                            [&](long long page, long long k) { extend_give(p, s_prefix, s_len, page, k); });
}

// ---------------------------------------------------------------------------
// free
// ---------------------------------------------------------------------------

struct FreeParams {
    const int* table;
    int* lens;
    const uint8_t* leave;
    int rows, max_pages, shift, parts;
    int* refs;
    long long num_pages;
};

// One cluster of `parts` blocks per row: they read the length, take turns at
// the entries and, once all have read it, mark the row empty.  8 of 32 rows, of 60,000
// entries each, 7 us (an atomic an entry), 64 of 256 short rows 3.
__global__ void free_kernel(const FreeParams p) {
    using namespace pg;
    const int r = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
    if (p.leave != nullptr && p.leave[r] == 0) return;   // the whole cluster
    const int n = pages_of(p.lens[r], p.shift, p.max_pages);
    cooperative_groups::this_cluster().barrier_arrive();   // the length has been read
    const int* row = p.table + static_cast<size_t>(r) * p.max_pages;
    const long long stride = static_cast<long long>(p.parts) * blockDim.x;
    for (long long j0 = static_cast<long long>(part) * blockDim.x + threadIdx.x; j0 < n; j0 += 4 * stride) {
        int page[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) page[u] = j0 + u * stride < n ? row[j0 + u * stride] : -1;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (page[u] >= 0 && page[u] < p.num_pages) atomicAdd(p.refs + page[u], -1);
    }
    cooperative_groups::this_cluster().barrier_wait();
    if (part == 0 && threadIdx.x == 0) p.lens[r] = -1;
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

// compact: 2^20 pages, three quarters in use, in three launches 19.0 us (196,000 pages
// move; 17.7 where none of the table's entries is left to change), half of it for the
// tables and counts (two dependent loads an entry); 16,384 in two launches 9.4.
__global__ void __launch_bounds__(pg::THREADS) compact_count_kernel(const CompactParams p) {
    using namespace pg;
    pdl_launch_dependents();
    const unsigned n = count_chunk(p.pool, blockIdx.x);
    if (threadIdx.x == 0) p.ws.counts[blockIdx.x] = n;
}

// With `total` pages in use, the k-th page in use at or above `total` moves to
// the k-th free page below it: sources and destinations are two disjoint
// ranges of the pool, and no page moves that need not.  `holes`: free pages
// below `total`, as many as pages that would move.
struct Moves {
    long long total, kept;   // pages in use; those of them below `total`
    int moves;
};
__device__ __forceinline__ Moves compact_moves(const CompactParams& p, long long total, long long holes) {
    return {total, total - holes, static_cast<int>(holes < p.max_moves ? holes : p.max_moves)};
}
// For the first thread of the first block: what the next kernel and the caller get.
__device__ __forceinline__ void compact_head(const CompactParams& p, const Moves& m) {
    p.used[0] = static_cast<int>(m.total);
    p.ws.head->total = static_cast<int>(m.total);
    p.ws.head->moves = m.moves;
    p.ws.head->status = 0;
}
// Pages id, k free ones before it.
__device__ __forceinline__ void compact_page(const CompactParams& p, const Moves& m, long long id, long long k, bool free) {
    if (free) {
        if (id < m.total && k < m.moves) p.copy_dst[k] = static_cast<int>(id);
        if (id >= m.total) p.ws.rank[id] = -1;
    } else if (id >= m.total) {
        const long long q = id - k - m.kept;   // id - k pages in use come before this one
        if (q < m.moves) p.copy_src[q] = static_cast<int>(id);
        p.ws.rank[id] = q < m.moves ? static_cast<int>(q) : -1;
    }
}

// The pages [i, end) of a block (RUN a thread), `before` free ones before them:
// neighbouring threads write neighbouring places, page by page and not run by run.
template <int T>
__device__ __forceinline__ void compact_pages(const CompactParams& p, const Moves& m, long long i, long long end,
                                              long long before, unsigned bits, int rank) {
    using namespace pg;
    __shared__ uint16_t s_bits[T];
    __shared__ int s_rank[T];
    static_assert(RUN <= 16, "a run's bits");
    s_bits[threadIdx.x] = static_cast<uint16_t>(bits);   // the last readers are behind a barrier of block_scan
    s_rank[threadIdx.x] = rank;
    __syncthreads();
#pragma unroll 4
    for (int o = threadIdx.x; o < T * RUN; o += T) {
        const unsigned b = s_bits[o / RUN], at = o % RUN;
        if (i + o < end)
            compact_page(p, m, i + o, before + s_rank[o / RUN] + __popc(b & ((1u << at) - 1)), b >> at & 1);
    }
}

__global__ void __launch_bounds__(pg::THREADS) compact_rank_kernel(const CompactParams p) {
    using namespace pg;
    const int tid = threadIdx.x, chunk = blockIdx.x;
    const long long i0 = chunk * p.pool.chunk, i1 = chunk_end(p.pool, chunk);
    unsigned bits = free_bits(p.pool, i0 + RUN * tid, i1);   // the counts change in the next kernel only
    pdl_launch_dependents();
    pdl_wait_primary();
    const uint2 f = free_before(p.ws, p.pool.chunks, chunk);
    const long long total = p.pool.num_pages - f.y;
    // the chunk that `total` lies in is counted up to it
    const int edge = static_cast<int>(total / p.pool.chunk);
    unsigned whole = 0, part = 0;
    for (int i = tid; i < edge; i += THREADS) whole += p.ws.counts[i];
    for (long long i = edge * p.pool.chunk + tid; i < total; i += THREADS) part += p.pool.refs[i] == 0;
    const uint2 h = block_sum2<THREADS>(whole, part);
    const Moves m = compact_moves(p, total, static_cast<long long>(h.x) + h.y);
    if (chunk == 0 && tid == 0) compact_head(p, m);
    for (long long k = m.moves + static_cast<long long>(chunk) * THREADS + tid; k < p.max_moves;
         k += static_cast<long long>(gridDim.x) * THREADS) {
        p.copy_src[k] = -1;
        p.copy_dst[k] = -1;
    }
    long long before = f.x;   // free pages before the next ones
    for (long long i = i0; i < i1; i += CHUNK) {
        if (i != i0) bits = free_bits(p.pool, i + RUN * tid, i1);
        int sum;
        const int rank = block_scan<THREADS>(__popc(bits), &sum);
        compact_pages<THREADS>(p, m, i, i1, before, bits, rank);
        before += sum;
    }
}
// Both for a small pool.
__global__ void __cluster_dims__(pg::SMALL_BLOCKS, 1, 1) __launch_bounds__(pg::SMALL_THREADS)
    compact_small_kernel(const CompactParams p) {
    using namespace pg;
    const int tid = threadIdx.x, block = blockIdx.x;
    pdl_launch_dependents();
    cluster_begin();
    const Small s = look_small(p.pool, block);
    const uint2 f = cluster_sum<0>(s.sum, block);
    const int total = static_cast<int>(p.pool.num_pages - f.y);
    const int below = total - s.mine;   // the thread's pages below `total`
    const unsigned low = below >= RUN ? s.bits : below > 0 ? s.bits & ((1u << below) - 1) : 0;
    const unsigned mine = block_sum2<SMALL_THREADS>(__popc(low), 0).x;
    const Moves m = compact_moves(p, total, cluster_sum<1>(mine, block).y);
    if (block == 0 && tid == 0) compact_head(p, m);
    for (long long k = m.moves + block * SMALL_THREADS + tid; k < p.max_moves; k += SMALL_BLOCKS * SMALL_THREADS)
        p.copy_src[k] = p.copy_dst[k] = -1;
    const int i = block * SMALL_THREADS * RUN;
    if (i < p.pool.num_pages) compact_pages<SMALL_THREADS>(p, m, i, p.pool.num_pages, f.x, s.bits, s.rank);
}

// Block y < rows: the row's entries follow their pages.  Block y == rows: so do
// the counts.
__global__ void __launch_bounds__(pg::THREADS) compact_apply_kernel(const CompactParams p) {
    using namespace pg;
    const bool counts = static_cast<int>(blockIdx.y) == p.rows;
    const int n = counts ? 0 : pages_of(p.lens[blockIdx.y], p.shift, p.max_pages);
    const long long stride = static_cast<long long>(gridDim.x) * THREADS, j00 = blockIdx.x * THREADS + threadIdx.x;
    if (counts) {
        pdl_wait_primary();
        const int moves = p.ws.head->moves;
        for (long long k0 = j00; k0 < moves; k0 += 8 * stride) {   // eight at a time
            int from[8], to[8], n[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const long long k = k0 + u * stride;
                from[u] = k < moves ? p.copy_src[k] : -1;
                to[u] = k < moves ? p.copy_dst[k] : -1;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) n[u] = from[u] >= 0 ? p.pool.refs[from[u]] : 0;
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (from[u] >= 0) {
                    p.pool.refs[to[u]] = n[u];
                    p.pool.refs[from[u]] = 0;
                }
        }
        return;
    }
    int* row = p.table + static_cast<size_t>(blockIdx.y) * p.max_pages;
    bool waited = false;
    for (long long j0 = j00; j0 < n; j0 += 4 * stride) {   // four chains of loads at a time
        int page[4], k[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) page[u] = j0 + u * stride < n ? row[j0 + u * stride] : -1;
        if (!waited) pdl_wait_primary();   // the tables change in this kernel only
        waited = true;
        const int total = p.ws.head->total;
        // ranks below `total` were not written: what is read there is not used
#pragma unroll
        for (int u = 0; u < 4; ++u) k[u] = page[u] >= 0 && page[u] < p.pool.num_pages ? p.ws.rank[page[u]] : -1;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (page[u] >= total && k[u] >= 0) row[j0 + u * stride] = p.copy_dst[k[u]];
    }
}

// ---------------------------------------------------------------------------
// copy
// ---------------------------------------------------------------------------

struct CopyParams {
    uint8_t* cache[pg::MAX_CACHES];
    const int *src, *dst;
    int caches, n;
    int chunks, lanes;         // 16-byte chunks per page, threads per page (a power of two)
    long long num_pages;
    size_t page_bytes;
};

// A page is copied by `lanes` threads, 16 bytes each at a time, several loads of
// a thread in flight before its stores: over four pairs in two caches when a
// page is one chunk a thread (WIDE false: K and V rows of single-token pages),
// else over four chunks of one pair in one cache.  4,096 pages of 64 tokens in four
// caches (268 MB) 46 us, 5.8 TB/s; 197,000 single tokens' rows of 128 bytes in two
// caches (101 MB) 20 us, 5.1 TB/s.
template <bool WIDE>
__global__ void __launch_bounds__(pg::THREADS) pages_copy_kernel(const CopyParams p) {
    using namespace pg;
    const int lane = threadIdx.x % p.lanes, group = threadIdx.x / p.lanes, groups = THREADS / p.lanes;
    if (!WIDE) {
        uint8_t* c0 = p.cache[2 * blockIdx.y];
        uint8_t* c1 = 2 * blockIdx.y + 1 < p.caches ? p.cache[2 * blockIdx.y + 1] : nullptr;
        for (long long i0 = static_cast<long long>(blockIdx.x) * groups * 4 + group; i0 < p.n;
             i0 += static_cast<long long>(gridDim.x) * groups * 4) {
            int s[4], d[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const long long i = i0 + static_cast<long long>(u) * groups;
                const bool in = i < p.n && lane < p.chunks;
                s[u] = in ? p.src[i] : -1;
                d[u] = in ? p.dst[i] : -1;
                if (d[u] < 0 || s[u] >= p.num_pages || d[u] >= p.num_pages) s[u] = -1;
            }
            uint4 v[4], w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (s[u] >= 0) {
                    v[u] = reinterpret_cast<const uint4*>(c0 + s[u] * p.page_bytes)[lane];
                    if (c1 != nullptr) w[u] = reinterpret_cast<const uint4*>(c1 + s[u] * p.page_bytes)[lane];
                }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (s[u] >= 0) {
                    reinterpret_cast<uint4*>(c0 + d[u] * p.page_bytes)[lane] = v[u];
                    if (c1 != nullptr) reinterpret_cast<uint4*>(c1 + d[u] * p.page_bytes)[lane] = w[u];
                }
        }
    } else {
        uint8_t* cache = p.cache[blockIdx.y];
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
