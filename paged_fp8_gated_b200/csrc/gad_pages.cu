// gad_pages.cu - C ABI of the page operations (gad_pages.cuh): argument checks,
// workspace layout and launches.  The kernels of one call are chained with
// programmatic dependent launch.
#include <cuda_runtime.h>

#include "gad_host.h"
#include "gad_pages.cuh"

using namespace gad_host;

namespace {

struct PagesWs {
    size_t head_off, counts_off, rows_off, prefix_off, rank_off, total;
};
PagesWs pages_ws(long long num_pages) {
    PagesWs w{};
    size_t off = 0;
    w.head_off = off;
    off = align_up(off + sizeof(gad::pg::Head));
    w.counts_off = off;
    off = align_up(off + gad::pg::MAX_CHUNKS * sizeof(unsigned));
    w.rows_off = off;
    off = align_up(off + 2 * gad::pg::MAX_ROWS * sizeof(int));
    w.prefix_off = off;
    off = align_up(off + (gad::pg::MAX_ROWS + 1) * sizeof(int));
    w.rank_off = off;
    off = align_up(off + static_cast<size_t>(num_pages) * sizeof(int));
    w.total = off;
    return w;
}
static_assert(gad::pg::MAX_ROWS == GAD_MAX_B, "per-row scratch holds every row a call may have");

gad::pg::Ws bind_ws(void* workspace, long long num_pages) {
    const PagesWs w = pages_ws(num_pages);
    uint8_t* b = static_cast<uint8_t*>(workspace);
    gad::pg::Ws ws;
    ws.head = reinterpret_cast<gad::pg::Head*>(b + w.head_off);
    ws.counts = reinterpret_cast<unsigned*>(b + w.counts_off);
    ws.rows = reinterpret_cast<int*>(b + w.rows_off);
    ws.prefix = reinterpret_cast<int*>(b + w.prefix_off);
    ws.rank = reinterpret_cast<int*>(b + w.rank_off);
    return ws;
}

gad::pg::Pool bind_pool(int32_t* refs, int64_t num_pages) {
    gad::pg::Pool p;
    p.refs = refs;
    p.num_pages = num_pages;
    p.chunk = gad::pg::chunk_pages(num_pages);
    p.chunks = static_cast<int>((num_pages + p.chunk - 1) / p.chunk);
    return p;
}

int check_rows(const char* name, int rows) {
    if (rows < 1 || rows > GAD_MAX_B) return fail(GAD_ERR_SHAPE, "%s=%d not in [1,%d]", name, rows, GAD_MAX_B);
    return GAD_OK;
}

int check_pool(int max_pages, int page_size, const int32_t* refs, int64_t num_pages) {
    if (page_size != 1 && page_size != 64)
        return fail(GAD_ERR_UNSUPPORTED, "page_size=%d (supported: 1, 64)", page_size);
    if (max_pages < 1) return fail(GAD_ERR_SHAPE, "max_pages=%d < 1", max_pages);
    if (static_cast<long long>(max_pages) * page_size > INT32_MAX)
        return fail(GAD_ERR_SHAPE, "max_pages * page_size exceeds 2^31");
    if (num_pages < 1 || num_pages > INT32_MAX / page_size)
        return fail(GAD_ERR_SHAPE, "num_pages=%lld: the pool holds 1 to 2^31 - 1 tokens", static_cast<long long>(num_pages));
    if (!aligned(refs, 16)) return fail(GAD_ERR_ALIGN, "refs must be 16-byte aligned");
    return GAD_OK;
}

int check_ws(const void* workspace, size_t bytes, int64_t num_pages) {
    if (!workspace) return fail(GAD_ERR_WORKSPACE, "workspace is NULL");
    if (!aligned(workspace, kAlign)) return fail(GAD_ERR_ALIGN, "workspace must be 256-byte aligned");
    const size_t need = pages_ws(num_pages).total;
    if (bytes < need) return fail(GAD_ERR_WORKSPACE, "workspace %zu B < required %zu B", bytes, need);
    return GAD_OK;
}

// A table of `rows` rows, in bytes.
size_t table_bytes(int rows, int max_pages) { return static_cast<size_t>(rows) * max_pages * 4; }
size_t row_bytes(int rows) { return static_cast<size_t>(rows) * 4; }

// Blocks read and write a call's arrays at the same time.
int check_overlap(std::initializer_list<Span> written, std::initializer_list<Span> read) {
    if (written_overlap(written, read))
        return fail(GAD_ERR_UNSUPPORTED, "an array that the call writes may not overlap another one of the call");
    return GAD_OK;
}

int check_device() {
    int sms = 0, major = 0;
    const int st = current_device_sms(&sms, &major);
    if (st != GAD_OK) return st;
    if (major != 10) return fail(GAD_ERR_DEVICE, "compute capability %d.x; this build targets sm_100a", major);
    return GAD_OK;
}

template <class... Params, class... Args>
int launch(const char* name, void (*kern)(Params...), dim3 grid, int threads, cudaStream_t s, bool pdl, Args... args) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr = pdl_attr();
    cfg.attrs = &attr;
    cfg.numAttrs = pdl ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e != cudaSuccess) return fail(GAD_ERR_CUDA, "%s launch: %s", name, cudaGetErrorString(e));
    return GAD_OK;
}

constexpr int T = gad::pg::THREADS;
// Blocks of four columns a thread below which fork takes one: 148 SMs.
constexpr long long kFewBlocks = 148;
// Most tokens that extend's cluster for a small pool places.
constexpr long long kSmallTokens = 65536;

// Whether a kernel of one cluster looks through the pool.
bool small_pool(int64_t num_pages) { return num_pages <= gad::pg::SMALL_POOL; }

int shift_of(int page_size) { return page_size == 64 ? 6 : 0; }

unsigned blocks(long long n, long long per) { return static_cast<unsigned>((n + per - 1) / per); }

}  // namespace

extern "C" {

size_t gad_pages_workspace_bytes(int rows, int64_t num_pages) {
    if (check_rows("rows", rows) != GAD_OK) return 0;
    if (num_pages < 1 || num_pages > INT32_MAX) {
        fail(GAD_ERR_SHAPE, "num_pages=%lld not in [1,2^31)", static_cast<long long>(num_pages));
        return 0;
    }
    return pages_ws(num_pages).total;
}

int gad_pages_copy(void* const* caches, int n_caches, size_t page_bytes, int64_t num_pages, const int32_t* src,
                   const int32_t* dst, int n, void* stream) {
    if (!caches || (n > 0 && (!src || !dst))) return fail(GAD_ERR_NULL, "caches, src and dst must be non-NULL");
    if (n_caches < 1 || n_caches > GAD_MAX_CACHES)
        return fail(GAD_ERR_SHAPE, "n_caches=%d not in [1,%d]", n_caches, GAD_MAX_CACHES);
    if (n < 0) return fail(GAD_ERR_SHAPE, "n=%d < 0", n);
    if (page_bytes < 16 || page_bytes % 16 != 0 || page_bytes > GAD_MAX_PAGE_BYTES)
        return fail(GAD_ERR_SHAPE, "page_bytes=%zu must be a multiple of 16 in [16,%d]", page_bytes,
                    GAD_MAX_PAGE_BYTES);
    if (num_pages < 1 || num_pages > INT32_MAX)
        return fail(GAD_ERR_SHAPE, "num_pages=%lld not in [1,2^31)", static_cast<long long>(num_pages));
    for (int i = 0; i < n_caches; ++i) {
        if (!caches[i]) return fail(GAD_ERR_NULL, "caches[%d] is NULL", i);
        if (!aligned(caches[i], 16)) return fail(GAD_ERR_ALIGN, "caches[%d] must be 16-byte aligned", i);
    }
    if (!aligned(src, 4) || !aligned(dst, 4)) return fail(GAD_ERR_ALIGN, "src and dst must be 4-byte aligned");
    int st = GAD_OK;
    for (int i = 0; i < n_caches && n > 0 && st == GAD_OK; ++i)
        st = check_overlap({{caches[i], num_pages * page_bytes}}, {{src, row_bytes(n)}, {dst, row_bytes(n)}});
    if (st == GAD_OK) st = check_device();
    if (st != GAD_OK || n == 0) return st;

    gad::CopyParams p;
    std::memset(&p, 0, sizeof(p));
    p.src = src;
    p.dst = dst;
    p.n = n;
    p.num_pages = num_pages;
    p.page_bytes = page_bytes;
    p.chunks = static_cast<int>(page_bytes / 16);
    const bool wide = p.chunks >= 128;
    const int want = wide ? (p.chunks + 3) / 4 : p.chunks;
    p.lanes = 1;
    while (p.lanes < want && p.lanes < T) p.lanes *= 2;
    const long long per_block = (T / p.lanes) * (wide ? 1 : 4);
    const unsigned gx = blocks(n, per_block) < (1u << 20) ? blocks(n, per_block) : (1u << 20);
    for (int c0 = 0; c0 < n_caches; c0 += gad::pg::MAX_CACHES) {
        const int m = n_caches - c0 < gad::pg::MAX_CACHES ? n_caches - c0 : gad::pg::MAX_CACHES;
        for (int i = 0; i < m; ++i) p.cache[i] = static_cast<uint8_t*>(caches[c0 + i]);
        p.caches = m;
        const dim3 grid(gx, static_cast<unsigned>(wide ? m : (m + 1) / 2));
        st = launch("page copy", wide ? gad::pages_copy_kernel<true> : gad::pages_copy_kernel<false>, grid, T,
                    static_cast<cudaStream_t>(stream), false, p);
        if (st != GAD_OK) return st;
    }
    return GAD_OK;
}

int gad_pages_fork(const int32_t* page_table, const int32_t* lens, int rows_in, const int32_t* parent, int rows_out,
                   int max_pages, int page_size, int32_t* refs, int64_t num_pages, int32_t* out_table,
                   int32_t* out_lens, int32_t* copy_src, int32_t* copy_dst, void* workspace, size_t workspace_bytes,
                   void* stream) {
    if (!page_table || !lens || !parent || !refs || !out_table || !out_lens || !copy_src || !copy_dst)
        return fail(GAD_ERR_NULL, "a required pointer is NULL");
    int st = check_rows("rows_in", rows_in);
    if (st == GAD_OK) st = check_rows("rows_out", rows_out);
    if (st == GAD_OK) st = check_pool(max_pages, page_size, refs, num_pages);
    if (st == GAD_OK) st = check_ws(workspace, workspace_bytes, num_pages);
    if (st != GAD_OK) return st;
    for (const void* q : {static_cast<const void*>(page_table), static_cast<const void*>(lens),
                          static_cast<const void*>(parent), static_cast<const void*>(out_table),
                          static_cast<const void*>(out_lens), static_cast<const void*>(copy_src),
                          static_cast<const void*>(copy_dst)})
        if (!aligned(q, 4)) return fail(GAD_ERR_ALIGN, "tables, lengths, parent and copy lists need 4-byte alignment");
    st = check_overlap({{out_table, table_bytes(rows_out, max_pages)},
                        {out_lens, row_bytes(rows_out)},
                        {copy_src, row_bytes(rows_out)},
                        {copy_dst, row_bytes(rows_out)},
                        {refs, static_cast<size_t>(num_pages) * 4},
                        {workspace, pages_ws(num_pages).total}},
                       {{page_table, table_bytes(rows_in, max_pages)},
                        {lens, row_bytes(rows_in)},
                        {parent, row_bytes(rows_out)}});
    if (st == GAD_OK) st = check_device();
    if (st != GAD_OK) return st;

    gad::ForkParams p;
    std::memset(&p, 0, sizeof(p));
    p.table = page_table;
    p.lens = lens;
    p.parent = parent;
    p.out_table = out_table;
    p.out_lens = out_lens;
    p.copy_src = copy_src;
    p.copy_dst = copy_dst;
    p.rows_in = rows_in;
    p.rows_out = rows_out;
    p.max_pages = max_pages;
    p.shift = shift_of(page_size);
    p.pool = bind_pool(refs, num_pages);
    p.ws = bind_ws(workspace, num_pages);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int rows = rows_in > rows_out ? rows_in : rows_out;
    const bool few = static_cast<long long>(blocks(rows, gad::pg::ROWS)) * blocks(max_pages, 4 * T) < kFewBlocks;
    const bool vec = max_pages % 4 == 0 && aligned(page_table, 16) && aligned(out_table, 16);
    const dim3 grid(blocks(max_pages, few ? T : 4 * T), blocks(rows, gad::pg::ROWS));
    st = launch("fork",
                few   ? gad::fork_kernel<1, false>
                : vec ? gad::fork_kernel<4, true>
                      : gad::fork_kernel<4, false>,
                grid, T, s, false, p);
    if (st != GAD_OK || page_size == 1) return st;   // single-token pages are never partly filled
    const int pool_bit = GAD_STATUS_PAGES_POOL;
    if (small_pool(num_pages))
        return launch("fork assign", gad::fork_assign_small_kernel, dim3(gad::pg::SMALL_BLOCKS), gad::pg::SMALL_THREADS, s, true, p, pool_bit);
    st = launch("fork count", gad::fork_count_kernel, dim3(p.pool.chunks + 1), T, s, true, p);
    if (st != GAD_OK) return st;
    return launch("fork assign", gad::fork_assign_kernel, dim3(p.pool.chunks), T, s, true, p, pool_bit);
}

int gad_pages_extend(int32_t* page_table, int32_t* lens, int rows, int L, int max_pages, int page_size, int32_t* refs,
                     int64_t num_pages, int64_t* positions, int64_t* cache_loc, void* workspace,
                     size_t workspace_bytes, void* stream) {
    if (!page_table || !lens || !refs || !positions || !cache_loc)
        return fail(GAD_ERR_NULL, "a required pointer is NULL");
    int st = check_rows("rows", rows);
    if (st != GAD_OK) return st;
    if (L < 1 || L > GAD_MAX_PREFILL_L) return fail(GAD_ERR_SHAPE, "L=%d not in [1,%d]", L, GAD_MAX_PREFILL_L);
    st = check_pool(max_pages, page_size, refs, num_pages);
    if (st == GAD_OK) st = check_ws(workspace, workspace_bytes, num_pages);
    if (st != GAD_OK) return st;
    if (!aligned(positions, 8) || !aligned(cache_loc, 8) || !aligned(page_table, 4) || !aligned(lens, 4))
        return fail(GAD_ERR_ALIGN, "positions/cache_loc need 8-byte, page_table/lens 4-byte alignment");
    const size_t token_bytes = static_cast<size_t>(rows) * L * 8;
    st = check_overlap({{page_table, table_bytes(rows, max_pages)},
                        {lens, row_bytes(rows)},
                        {refs, static_cast<size_t>(num_pages) * 4},
                        {positions, token_bytes},
                        {cache_loc, token_bytes},
                        {workspace, pages_ws(num_pages).total}},
                       {});
    if (st == GAD_OK) st = check_device();
    if (st != GAD_OK) return st;

    gad::ExtendParams p;
    std::memset(&p, 0, sizeof(p));
    p.table = page_table;
    p.lens = lens;
    p.positions = reinterpret_cast<long long*>(positions);
    p.cache_loc = reinterpret_cast<long long*>(cache_loc);
    p.rows = rows;
    p.L = L;
    p.max_pages = max_pages;
    p.shift = shift_of(page_size);
    p.pool = bind_pool(refs, num_pages);
    p.ws = bind_ws(workspace, num_pages);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int pool_bit = GAD_STATUS_PAGES_POOL, row_bit = GAD_STATUS_PAGES_ROW;
    const long long tokens = static_cast<long long>(rows) * L;
    if (small_pool(num_pages) && tokens <= kSmallTokens)
        return launch("extend", gad::extend_small_kernel, dim3(gad::pg::SMALL_BLOCKS), gad::pg::SMALL_THREADS, s, false, p, pool_bit, row_bit);
    st = launch("extend count", gad::extend_count_kernel, dim3(p.pool.chunks + 1), T, s, false, p);
    if (st != GAD_OK) return st;
    // enough blocks for the tokens' rows too
    const long long tok = (tokens + 8 * T - 1) / (8 * T);
    const long long grid = tok > 1024 ? 1024 : tok;
    return launch("extend assign", gad::extend_assign_kernel,
                  dim3(static_cast<unsigned>(grid > p.pool.chunks ? grid : p.pool.chunks)), T, s, true, p, pool_bit,
                  row_bit);
}

int gad_pages_free(const int32_t* page_table, int32_t* lens, int rows, const uint8_t* leave, int max_pages,
                   int page_size, int32_t* refs, int64_t num_pages, void* stream) {
    if (!page_table || !lens || !refs) return fail(GAD_ERR_NULL, "page_table, lens and refs must be non-NULL");
    int st = check_rows("rows", rows);
    if (st == GAD_OK) st = check_pool(max_pages, page_size, refs, num_pages);
    if (st != GAD_OK) return st;
    if (!aligned(page_table, 4) || !aligned(lens, 4))
        return fail(GAD_ERR_ALIGN, "page_table and lens need 4-byte alignment");
    st = check_overlap({{lens, row_bytes(rows)}, {refs, static_cast<size_t>(num_pages) * 4}},
                       {{page_table, table_bytes(rows, max_pages)}, {leave, static_cast<size_t>(rows)}});
    if (st == GAD_OK) st = check_device();
    if (st != GAD_OK) return st;
    gad::FreeParams p;
    std::memset(&p, 0, sizeof(p));
    p.table = page_table;
    p.lens = lens;
    p.leave = leave;
    p.rows = rows;
    p.max_pages = max_pages;
    p.shift = shift_of(page_size);
    p.refs = refs;
    p.num_pages = num_pages;
    // four entries a thread: blocks of up to 1024 threads, up to sixteen of them
    // per row (more than eight is a size that a kernel has to allow)
    int threads = 64;
    while (threads < 1024 && threads * 4 < max_pages) threads *= 2;
    p.parts = 1;
    while (p.parts < 16 && static_cast<long long>(p.parts) * threads * 4 < max_pages) p.parts *= 2;
    static OncePerContext allowed;
    int dev = 0;
    st = current_device(&dev);
    if (st != GAD_OK) return st;
    if (!allowed.is_done(dev, current_ctx_id())) {
        const cudaError_t e = cudaFuncSetAttribute(gad::free_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return fail(GAD_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        allowed.mark(dev);
    }
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>(rows) * p.parts);
    cfg.blockDim = dim3(threads);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr;
    std::memset(&attr, 0, sizeof(attr));
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = p.parts;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, gad::free_kernel, p);
    if (e != cudaSuccess) return fail(GAD_ERR_CUDA, "free launch: %s", cudaGetErrorString(e));
    return GAD_OK;
}

int gad_pages_compact(int32_t* page_table, const int32_t* lens, int rows, int max_pages, int page_size, int32_t* refs,
                      int64_t num_pages, int32_t* copy_src, int32_t* copy_dst, int max_moves, int32_t* used,
                      void* workspace, size_t workspace_bytes, void* stream) {
    if (!page_table || !lens || !refs || !copy_src || !copy_dst || !used)
        return fail(GAD_ERR_NULL, "a required pointer is NULL");
    int st = check_rows("rows", rows);
    if (st != GAD_OK) return st;
    if (max_moves < 1) return fail(GAD_ERR_SHAPE, "max_moves=%d < 1", max_moves);
    st = check_pool(max_pages, page_size, refs, num_pages);
    if (st == GAD_OK) st = check_ws(workspace, workspace_bytes, num_pages);
    if (st != GAD_OK) return st;
    if (!aligned(page_table, 4) || !aligned(lens, 4) || !aligned(copy_src, 4) || !aligned(copy_dst, 4) ||
        !aligned(used, 4))
        return fail(GAD_ERR_ALIGN, "tables, lengths, copy lists and used need 4-byte alignment");
    st = check_overlap({{page_table, table_bytes(rows, max_pages)},
                        {refs, static_cast<size_t>(num_pages) * 4},
                        {copy_src, row_bytes(max_moves)},
                        {copy_dst, row_bytes(max_moves)},
                        {used, 4},
                        {workspace, pages_ws(num_pages).total}},
                       {{lens, row_bytes(rows)}});
    if (st == GAD_OK) st = check_device();
    if (st != GAD_OK) return st;
    gad::CompactParams p;
    std::memset(&p, 0, sizeof(p));
    p.table = page_table;
    p.lens = lens;
    p.copy_src = copy_src;
    p.copy_dst = copy_dst;
    p.used = used;
    p.rows = rows;
    p.max_pages = max_pages;
    p.shift = shift_of(page_size);
    p.max_moves = max_moves;
    p.pool = bind_pool(refs, num_pages);
    p.ws = bind_ws(workspace, num_pages);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (small_pool(num_pages)) {
        st = launch("compact", gad::compact_small_kernel, dim3(gad::pg::SMALL_BLOCKS), gad::pg::SMALL_THREADS, s, false, p);
    } else {
        st = launch("compact count", gad::compact_count_kernel, dim3(p.pool.chunks), T, s, false, p);
        if (st != GAD_OK) return st;
        st = launch("compact rank", gad::compact_rank_kernel, dim3(p.pool.chunks), T, s, true, p);
    }
    if (st != GAD_OK) return st;
    const unsigned gx = blocks(max_pages, 4 * T);   // four entries a thread
    return launch("compact apply", gad::compact_apply_kernel, dim3(gx < 1024 ? gx : 1024, static_cast<unsigned>(rows) + 1), T, s, true, p);
}

}  // extern "C"
