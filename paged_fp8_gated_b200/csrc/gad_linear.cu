// gad_linear.cu - C ABI of the linear layer (gad_linear.cuh): argument checks,
// the choice of the kernel and its tiles, launches.  The kernels wait for the
// kernel before them under programmatic dependent launch, so that their set-up
// (barriers, tensor memory, descriptors) runs beside its end.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "gad_host.h"
#include "gad_linear.cuh"

using namespace gad_host;

namespace {

static_assert(gad::lin::STATUS_LINEAR_WAIT == GAD_STATUS_LINEAR_WAIT, "status bit");

// Status word of the linear layer (it has no workspace to hold it); read and
// cleared by gad_linear_status.
__device__ int g_linear_err;

int linear_status_word(int** out) {
    static OncePerContext looked_up;
    static std::atomic<void*> addr[kMaxDevices];
    int dev = 0;
    const int ds = current_device(&dev);
    if (ds != GAD_OK) return ds;
    if (!looked_up.is_done(dev, current_ctx_id())) {
        void* ea = nullptr;
        cudaError_t e = cudaGetSymbolAddress(&ea, g_linear_err);
        if (e != cudaSuccess || ea == nullptr)
            return fail(GAD_ERR_CUDA, "cudaGetSymbolAddress(linear status word): %s", cudaGetErrorString(e));
        addr[dev].store(ea, std::memory_order_release);
        looked_up.mark(dev);
    }
    *out = static_cast<int*>(addr[dev].load(std::memory_order_acquire));
    return GAD_OK;
}

// Tiles of box_cols x box_rows of a matrix of 16-bit values, box_cols of them the
// swizzle's width.
int encode_tiles(CUtensorMap* map, const void* base, bool fp16, int cols, int rows, long long ld, int box_cols,
                 int box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    const int st = tensor_map_encoder(&fn);
    if (st != GAD_OK) return st;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                    const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    box_cols == 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                    : box_cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                     : CU_TENSOR_MAP_SWIZZLE_32B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(GAD_ERR_CUDA, "cuTensorMapEncodeTiled (linear) failed (%d)", static_cast<int>(r));
    return GAD_OK;
}

// A matrix as its rows in memory, all in bytes.
struct Rows {
    const void* p;
    size_t rows, ld, width;
    Rows(const void* base, long long n, long long stride, long long cols, int elem)
        : p(base), rows(static_cast<size_t>(n)), ld(static_cast<size_t>(stride) * elem),
          width(static_cast<size_t>(cols) * elem) {}
    size_t extent() const { return (rows - 1) * ld + width; }
};
// Whether a row of one shares a byte with a row of the other.  Rows at one distance
// (a single row has any) lie side by side, as the columns of a wider matrix, where
// b's place within a's distance leaves room for both; others share none only if the
// matrices' whole extents do.
bool rows_overlap(const Rows& a, const Rows& b) {
    if (!overlap(a.p, a.extent(), b.p, b.extent())) return false;
    const size_t ld = a.rows > 1 ? a.ld : b.ld;
    if (b.rows > 1 && b.ld != ld) return true;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    const size_t at = y >= x ? (y - x) % ld : (ld - (x - y) % ld) % ld;
    return at < a.width || at + b.width > ld;
}

// Shared memory: 228 KB per SM, 1 KB of it the system's per block, 227 KB per
// block at most.  Blocks of a cluster wait for one another, so all of them must
// get their tensor memory (512 columns per SM) while others hold theirs: every
// launch takes at least the share of shared memory that its columns are of
// tensor memory, and blocks that fit side by side in the one fit in the other,
// whichever calls they belong to.
constexpr int kSmemPerSm = 228 * 1024, kSmemReserved = 1024, kSmemMax = 227 * 1024;
constexpr int smem_share(int cols) {
    return static_cast<int>(static_cast<long long>(kSmemPerSm) * cols / 512) - kSmemReserved;
}
static_assert(smem_share(512) == kSmemMax, "all of tensor memory, all of shared memory");

constexpr int kClasses = 3;   // 1, 2 or 4 blocks per SM
constexpr int kSplits = 4;    // clusters of 1, 2, 4 or 8

// How a call runs.
struct Plan {
    enum Kind { NARROW, WIDE } kind = NARROW;
    int bn = 0;        // wide: 256 or 128
    int split = 1;     // narrow: blocks of a cluster; wide: pairs of a cluster
    int cls = 0;       // narrow: 2^cls blocks per SM
    bool promote = false;
    double us = 1e30;
};

// Clusters that the GPU holds at a time: narrow[cls][log2 split], wide[log2 pairs].
struct Capacity {
    int narrow[kClasses][kSplits];
    int wide[3];
};

void cluster_config(cudaLaunchConfig_t* cfg, cudaLaunchAttribute* attr, unsigned blocks_x, unsigned blocks_y, int threads,
                    int smem, int cluster, cudaStream_t s) {
    std::memset(cfg, 0, sizeof(*cfg));
    cfg->gridDim = dim3(blocks_x, blocks_y);
    cfg->blockDim = dim3(static_cast<unsigned>(threads));
    cfg->dynamicSmemBytes = static_cast<size_t>(smem);
    cfg->stream = s;
    std::memset(attr, 0, sizeof(*attr));
    attr->id = cudaLaunchAttributeClusterDimension;
    attr->val.clusterDim.x = static_cast<unsigned>(cluster);
    attr->val.clusterDim.y = 1;
    attr->val.clusterDim.z = 1;
    cfg->attrs = attr;
    cfg->numAttrs = 1;
}

// Stands for the kernels in the question how many clusters fit: for a kernel that
// allocates tensor memory the answer counts one block per SM whatever its shared
// memory, though the blocks do run side by side (threads and registers, at most
// 64 in the four-block class, allow it).
__global__ void __launch_bounds__(256) resident_probe_kernel() {}

int capacity_of(OncePerContext& once, int smem, int cluster, int* out) {
    const int st = raise_smem(reinterpret_cast<const void*>(resident_probe_kernel), once, kSmemMax);
    if (st != GAD_OK) return st;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr;
    cluster_config(&cfg, &attr, static_cast<unsigned>(4096 * cluster), 1, 256, smem, cluster, nullptr);
    const cudaError_t e = cudaOccupancyMaxActiveClusters(out, resident_probe_kernel, &cfg);
    if (e != cudaSuccess) return fail(GAD_ERR_CUDA, "cudaOccupancyMaxActiveClusters: %s", cudaGetErrorString(e));
    if (*out < 1) *out = 1;
    return GAD_OK;
}

OncePerContext g_narrow_smem[4];

// Asked once per (device, context); two threads that ask at the same time store
// the same answers.
int capacity(Capacity* out) {
    static OncePerContext asked, raised;
    static std::atomic<int> known[kMaxDevices][kClasses * kSplits + 3];
    int dev = 0;
    const int ds = current_device(&dev);
    if (ds != GAD_OK) return ds;
    const bool ask = !asked.is_done(dev, current_ctx_id());
    int i = 0;
    auto get = [&](int smem, int cluster, int* n) {
        if (ask) {
            const int st = capacity_of(raised, smem, cluster, n);
            if (st != GAD_OK) return st;
            known[dev][i].store(*n, std::memory_order_release);
        } else {
            *n = known[dev][i].load(std::memory_order_acquire);
        }
        ++i;
        return static_cast<int>(GAD_OK);
    };
    for (int m = 0; m < kClasses; ++m)
        for (int k = 0; k < kSplits; ++k) {
            const int st = get(smem_share(512 >> m), 1 << k, &out->narrow[m][k]);
            if (st != GAD_OK) return st;
        }
    for (int k = 0; k < 3; ++k) {
        const int st = get(smem_share(512), 2 << k, &out->wide[k]);
        if (st != GAD_OK) return st;
    }
    if (ask) asked.mark(dev);
    return GAD_OK;
}

// Tokens per narrow tile: as even as tiles of at most 256 can be.
int narrow_tokens(int T) {
    const int tiles = (T + 255) / 256;
    return ((T + tiles - 1) / tiles + 15) / 16 * 16;
}

// A chain of more than this many stages is promoted: for a fp32 result, and for a
// 16-bit one, whose rounding (2^-11 of it in fp16) hides up to 5e-5 from a chain of
// 32,768 products, but not the 8e-4 that one of 524,288 loses.
constexpr int kLongChain = 768 / gad::lin::BK, kLongChain16 = 32768 / gad::lin::BK;

double larger(double a, double b) { return a > b ? a : b; }

// The plan with the least time by this model of the kernels, in microseconds.
// Its constants are fitted to every plan at T = 1 .. 2,048 over ten (K, N) from
// 256 x 32,000 to 8,192 x 32,000, weights from memory, launches one behind
// another; the plan taken is there 0.7% slower than the fastest on average, 11% at
// most:
//   narrow: a stage takes a block 0.294 (an SM draws 56 GB/s of weights), or its
//     bytes at an SM's 126 GB/s from L2, or all blocks' weights at 5.9 TB/s, or
//     a load's latency (1.48) over the stages in flight; a block's fixed part is
//     its cluster's start, its SM's share of the epilogue and the exchange with
//     the cluster.  Blocks that leave room on their SM start while the launch
//     before still runs.  Examples: 32 x 8,192 x 2,304 (18 tiles) 42 / 23 / 14 /
//     12 in clusters of 1 / 2 / 4 / 8 blocks; 32 x 1,024 x 8,192 (64 tiles) 7.2
//     in clusters of two blocks alone on their SMs, 8.3 of four, four to an SM.
//   wide: a stage of 256 x 256 takes a pair 0.37 (the tensor cores' 0.33 in a
//     long chain; 0.40 when no other tile reads the same weights), one of
//     256 x 128 0.26 (an SM's share of L2 bandwidth).  Example: 768 x 8,192 x
//     2,304 43 on 27 of 74 pairs, 27 with two pairs a tile; 1,024 x 8,192 x 2,304
//     (36 tiles, more than the 33 clusters of four blocks that fit) 43 and 52.
//   Promoted chains cost the one 17% and the other 10% (1,024 x 4,096 x 4,096 in
//     fp32 41 and 43, 4,096 x 8,192 x 14,336 980 and 898).
Plan choose(int T, int K, int N, bool f32, const Capacity& cap, int sms) {
    using namespace gad::lin;
    const int nk = (K + BK - 1) / BK, longest = f32 ? kLongChain : kLongChain16;
    Plan best;
    auto take = [&](const Plan& q) {
        if (q.us < best.us) best = q;
    };
    static constexpr double start[kClasses] = {1.88, 1.77, 1.61};
    const double dram = 2.0 * (static_cast<double>(T) * K + static_cast<double>(N) * K) / 6.4e6;
    {
        const int tt = narrow_tokens(T);
        const long long tiles = static_cast<long long>((T + tt - 1) / tt) * ((N + ROWS - 1) / ROWS);
        for (int k = 0; k < kSplits && (1 << k) <= nk; ++k) {
            const int c = 1 << k, own = (nk + c - 1) / c;
            const bool promote = own > longest;
            for (int m = 0; m < kClasses; ++m) {
                const int budget = smem_share(512 >> m);
                if (narrow_cols(tt) * (promote ? 2 : 1) > 512 >> m || narrow_smem(tt, 1) > budget) continue;
                if (promote && m > 1) continue;   // registers for two blocks
                int stages = 1;
                while (stages < own && stages < NARROW_MAX_STAGES && narrow_smem(tt, stages + 1) <= budget) ++stages;
                auto wave = [&](long long clusters) {
                    const long long blocks = clusters * c;
                    const double per_sm = static_cast<double>((blocks + sms - 1) / sms);
                    double ts = larger(0.294, per_sm * narrow_stage(tt) / 126e3);
                    ts = larger(ts, static_cast<double>(blocks * TILE) / 5.9e6);
                    if (own > stages) ts = larger(ts, 1.48 / stages);
                    const double shared = m == 1 ? larger(per_sm, 1.6) : per_sm;
                    return own * ts + 1.07 + 0.073 * c + tt * (0.0064 + 0.0206 * shared / c + 0.0029 * c);
                };
                const long long fit = cap.narrow[m][k], full = tiles / fit, rest = tiles % fit;
                Plan q;
                q.kind = Plan::NARROW;
                q.split = c;
                q.cls = m;
                q.promote = promote;
                q.us = start[m] + (full ? full * wave(fit) : 0.0) + (rest ? wave(rest) : 0.0);
                if (promote) q.us *= 1.17;
                take(q);
            }
        }
    }
    const double stage256 = T <= 256 ? 0.397 : 0.373;
    for (int bn = 256; bn >= 128; bn /= 2) {
        const long long tiles = static_cast<long long>((T + 255) / 256) * ((N + bn - 1) / bn);
        for (int k = 0; k < 3 && (1 << k) <= nk; ++k) {
            const int own = (nk + (1 << k) - 1) >> k;
            const bool promote = own > longest;
            if (promote && bn != 128) continue;
            if (bn == 256 && k == 2) continue;            // always behind 128 (512 x 8,192 x 1,024 19.3, 18.2)
            if (k > 0 && tiles > cap.wide[k]) continue;   // a second wave of clusters costs more than it saves
            Plan q;
            q.kind = Plan::WIDE;
            q.bn = bn;
            q.split = 1 << k;
            q.promote = promote;
            const double waves = static_cast<double>((tiles + cap.wide[k] - 1) / cap.wide[k]);
            if (k == 0)
                q.us = bn == 256 ? 4.4 + waves * larger(own * stage256, 2.28) : 4.58 + waves * larger(own * 0.2635, 1.4);
            else
                q.us = 3.7 + 0.6 * (k == 2) + (bn == 256 ? own * stage256 + 2.9 : own * 0.2166 + 1.5);
            if (promote) q.us *= 1.1;
            q.us = larger(q.us, 1.9 + dram);
            take(q);
        }
    }
    return best;
}

template <int ACC>
int launch_narrow(gad::lin::Params p, const void* x, long long ldx, const void* w, long long ldw, const Plan& plan,
                  cudaStream_t s) {
    using namespace gad::lin;
    auto kern = gad::linear_narrow_kernel<ACC>;
    p.tt = narrow_tokens(p.T);
    const int token_tiles = (p.T + p.tt - 1) / p.tt, nk = (p.K + BK - 1) / BK;
    const int budget = smem_share(512 >> plan.cls), own = (nk + plan.split - 1) / plan.split;
    // Small blocks find room beside those of the launch before: weights asked for
    // then 1 x 1,024 x 8,192 6.35 -> 5.95 us, 16 x 1,024 x 8,192 6.85 -> 6.25; in
    // larger blocks, which start late, 1 x 8,192 x 2,304 9.9 -> 11.2.
    p.early = plan.cls == 2;
    p.nstg = 1;
    while (p.nstg < NARROW_MAX_STAGES && p.nstg < own && narrow_smem(p.tt, p.nstg + 1) <= budget) ++p.nstg;
    if (narrow_smem(p.tt, p.nstg) > budget || narrow_cols(p.tt) * (ACC ? 2 : 1) > 512 >> plan.cls)
        return fail(GAD_ERR_SHAPE, "linear tile of %d tokens does not fit", p.tt);   // choose() plans none such
    int st = raise_smem(reinterpret_cast<const void*>(kern), g_narrow_smem[ACC / 32 > 2 ? 3 : ACC / 32], kSmemMax);
    if (st != GAD_OK) return st;
    CUtensorMap wmap, xmap;
    st = encode_tiles(&wmap, w, p.fp16 != 0, p.K, p.N, ldw, BK, ROWS);
    if (st == GAD_OK) st = encode_tiles(&xmap, x, p.fp16 != 0, p.K, p.T, ldx, BK, p.tt);
    if (st != GAD_OK) return st;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    cluster_config(&cfg, attr, static_cast<unsigned>((p.N + ROWS - 1) / ROWS * plan.split),
                   static_cast<unsigned>(token_tiles), NARROW_THREADS<ACC>, budget, plan.split, s);
    attr[1] = pdl_attr();
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, wmap, xmap, p);
    if (e != cudaSuccess) return fail(GAD_ERR_CUDA, "linear launch: %s", cudaGetErrorString(e));
    return GAD_OK;
}

template <int BN, int S, bool PROMOTE>
int launch_wide(gad::lin::Params p, const void* x, long long ldx, const void* w, long long ldw, int sms, cudaStream_t s) {
    using namespace gad::lin;
    using C = Wide<BN, S, PROMOTE>;
    auto kern = gad::linear_wide_kernel<BN, S, PROMOTE>;
    static_assert(C::SMEM <= kSmemMax, "ring and staging fit");
    static OncePerContext raised;
    int st = raise_smem(reinterpret_cast<const void*>(kern), raised, kSmemMax);
    if (st != GAD_OK) return st;
    p.mt = (p.T + 255) / 256;
    p.nt = (p.N + BN - 1) / BN;
    const long long tiles = static_cast<long long>(p.mt) * p.nt;
    CUtensorMap wmap, xmap, ymap;
    st = encode_tiles(&wmap, w, p.fp16 != 0, p.K, p.N, ldw, BK, BN / 2);
    if (st == GAD_OK) st = encode_tiles(&xmap, x, p.fp16 != 0, p.K, p.T, ldx, BK, ROWS);
    if (st == GAD_OK && p.by_tma) st = encode_tiles(&ymap, p.y, p.fp16 != 0, p.N, p.T, p.ldy, C::BOX, 32);
    else std::memset(&ymap, 0, sizeof(ymap));
    if (st != GAD_OK) return st;
    const long long pairs = S > 1 ? tiles * S : tiles < sms / 2 ? tiles : sms / 2;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    // all of an SM's shared memory: alone there, so its tensor memory is free
    cluster_config(&cfg, attr, static_cast<unsigned>(2 * pairs), 1, WIDE_THREADS, smem_share(512), 2 * S, s);
    attr[1] = pdl_attr();
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, wmap, xmap, ymap, p);
    if (e != cudaSuccess) return fail(GAD_ERR_CUDA, "linear launch: %s", cudaGetErrorString(e));
    return GAD_OK;
}

template <int BN, bool PROMOTE>
int launch_wide(const gad::lin::Params& p, const void* x, long long ldx, const void* w, long long ldw, int split, int sms,
                cudaStream_t s) {
    if (split == 1) return launch_wide<BN, 1, PROMOTE>(p, x, ldx, w, ldw, sms, s);
    if constexpr (BN == 128) {
        if (split == 4) return launch_wide<BN, 4, PROMOTE>(p, x, ldx, w, ldw, sms, s);
    }
    return launch_wide<BN, 2, PROMOTE>(p, x, ldx, w, ldw, sms, s);
}

}  // namespace

extern "C" {

int gad_linear(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias, const void* residual,
               int64_t ldr, void* y, int64_t ldy, int T, int K, int N, int dtype, int out_dtype, int activation,
               void* stream) {
    if (!x || !w || !y) return fail(GAD_ERR_NULL, "x, w and y must be non-NULL");
    if (dtype != GAD_DTYPE_BF16 && dtype != GAD_DTYPE_F16)
        return fail(GAD_ERR_DTYPE, "x and w of element type %d (bf16 or f16)", dtype);
    if (out_dtype != dtype && out_dtype != GAD_DTYPE_F32)
        return fail(GAD_ERR_DTYPE, "y of element type %d (that of x, or f32)", out_dtype);
    if (T < 1 || T > GAD_MAX_LINEAR || K < 1 || K > GAD_MAX_LINEAR || N < 1 || N > GAD_MAX_LINEAR)
        return fail(GAD_ERR_SHAPE, "T=%d, K=%d, N=%d not in [1,%d]", T, K, N, GAD_MAX_LINEAR);
    if (activation < GAD_ACT_NONE || activation > GAD_ACT_SILU)
        return fail(GAD_ERR_UNSUPPORTED, "activation %d", activation);
    if (ldx < K || ldw < K || ldx % 8 != 0 || ldw % 8 != 0 || ldx > GAD_MAX_LINEAR_LD || ldw > GAD_MAX_LINEAR_LD)
        return fail(GAD_ERR_STRIDE, "rows of x and w must be a multiple of 8 values apart, at least K (ldx=%lld, ldw=%lld)",
                    static_cast<long long>(ldx), static_cast<long long>(ldw));
    if (ldy < N || (residual && ldr < N) || ldy > GAD_MAX_LINEAR_LD || (residual && ldr > GAD_MAX_LINEAR_LD))
        return fail(GAD_ERR_STRIDE, "rows of y and residual must be at least N apart (ldy=%lld, ldr=%lld)",
                    static_cast<long long>(ldy), static_cast<long long>(ldr));
    const int oe = out_dtype == GAD_DTYPE_F32 ? 4 : 2;
    if (!aligned(x, 16) || !aligned(w, 16)) return fail(GAD_ERR_ALIGN, "x and w must be 16-byte aligned");
    if (!aligned(bias, 2) || !aligned(y, oe) || !aligned(residual, oe))
        return fail(GAD_ERR_ALIGN, "bias, residual and y must be aligned to their element size");
    const Rows out(y, T, ldy, N, oe);
    if (rows_overlap(out, Rows(x, T, ldx, K, 2)) || rows_overlap(out, Rows(w, N, ldw, K, 2)) ||
        (bias && rows_overlap(out, Rows(bias, 1, N, N, 2))))
        return fail(GAD_ERR_UNSUPPORTED, "y may not overlap x, w or bias");
    if (residual && !(residual == y && ldr == ldy) && rows_overlap(out, Rows(residual, T, ldr, N, oe)))
        return fail(GAD_ERR_UNSUPPORTED, "y may be residual itself, but not overlap it otherwise");
    int sms = 0, major = 0;
    int st = current_device_sms(&sms, &major);
    if (st != GAD_OK) return st;
    if (major != 10) return fail(GAD_ERR_DEVICE, "compute capability %d.x; this build targets sm_100a", major);

    gad::lin::Params p;
    std::memset(&p, 0, sizeof(p));
    p.bias = bias;
    p.residual = residual;
    p.y = y;
    p.ldr = ldr;
    p.ldy = ldy;
    p.T = T;
    p.K = K;
    p.N = N;
    p.fp16 = dtype == GAD_DTYPE_F16;
    p.out = out_dtype == GAD_DTYPE_F32 ? gad::lin::OUT_F32 : p.fp16 ? gad::lin::OUT_F16 : gad::lin::OUT_BF16;
    p.act = activation;
    p.vec = ldy % 4 == 0 && aligned(y, 4 * oe) && (!residual || (ldr % 4 == 0 && aligned(residual, 4 * oe)));
    const int chunk = 16 / oe;
    p.vec16 = ldy % chunk == 0 && aligned(y, 16) && (!residual || (ldr % chunk == 0 && aligned(residual, 16)));
    // (a TMA store writes a row to the end of its last 16 bytes)
    p.by_tma = oe == 2 && p.vec16 && N % 8 == 0 && !residual;
    st = linear_status_word(&p.err);
    if (st != GAD_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    Capacity cap;
    st = capacity(&cap);
    if (st != GAD_OK) return st;
    const Plan plan = choose(T, K, N, out_dtype == GAD_DTYPE_F32, cap, sms);
    if (plan.kind == Plan::WIDE)
        return plan.promote     ? launch_wide<128, true>(p, x, ldx, w, ldw, plan.split, sms, s)
               : plan.bn == 128 ? launch_wide<128, false>(p, x, ldx, w, ldw, plan.split, sms, s)
                                : launch_wide<256, false>(p, x, ldx, w, ldw, plan.split, sms, s);
    if (!plan.promote) return launch_narrow<0>(p, x, ldx, w, ldw, plan, s);
    switch (gad::lin::narrow_acc(narrow_tokens(T))) {
        case 32: return launch_narrow<32>(p, x, ldx, w, ldw, plan, s);
        case 64: return launch_narrow<64>(p, x, ldx, w, ldw, plan, s);
        default: return launch_narrow<128>(p, x, ldx, w, ldw, plan, s);
    }
}

int gad_linear_status(int* status, void* stream) {
    if (!status) return fail(GAD_ERR_NULL, "status must point to a host int");
    int* word = nullptr;
    const int st = linear_status_word(&word);
    if (st != GAD_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemcpyAsync(status, word, sizeof(int), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(word, 0, sizeof(int), s);
    if (e != cudaSuccess) return fail(GAD_ERR_CUDA, "linear status: %s", cudaGetErrorString(e));
    return GAD_OK;
}

}  // extern "C"
