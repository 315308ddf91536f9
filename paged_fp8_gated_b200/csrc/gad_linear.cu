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

// [rows, K] 16-bit matrix, rows ld apart, in boxes of 64 x box_rows.
int encode_rows(CUtensorMap* map, const void* base, bool fp16, int K, int rows, long long ld, int box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    const int st = tensor_map_encoder(&fn);
    if (st != GAD_OK) return st;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
    const cuuint32_t box[2] = {gad::lin::BK, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                    const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(GAD_ERR_CUDA, "cuTensorMapEncodeTiled (linear) failed (%d)", static_cast<int>(r));
    return GAD_OK;
}

size_t extent(long long rows, long long ld, long long cols, int elem) {
    return static_cast<size_t>((rows - 1) * ld + cols) * elem;
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

int launch_narrow(gad::lin::Params p, const void* x, long long ldx, const void* w, long long ldw, int sms,
                  cudaStream_t s) {
    using namespace gad::lin;
    const int token_tiles = (p.T + 255) / 256;
    p.tt = ((p.T + token_tiles - 1) / token_tiles + 15) / 16 * 16;
    const long long tiles = static_cast<long long>((p.N + ROWS - 1) / ROWS) * token_tiles;
    const int nk = (p.K + BK - 1) / BK;
    // Blocks that share a tile's K range: the count with the least work on the
    // busiest SM, a block's fixed part counted as four stages.
    int split = 1;
    long long best = -1;
    for (int c = 1; c <= 8 && c <= nk; c *= 2) {
        const long long cost = (tiles * c + sms - 1) / sms * ((nk + c - 1) / c + 4);
        if (best < 0 || cost < best) {
            best = cost;
            split = c;
        }
    }
    // the ring: all of an SM's shared memory when there is a block per SM at
    // most (or the partial sums need it), else half of it
    const int half = smem_share(256);
    const int budget = tiles * split <= sms || narrow_smem(p.tt, 0) > half ? kSmemMax : half;
    const int own_nk = (nk + split - 1) / split;
    p.nstg = 1;
    while (p.nstg < NARROW_MAX_STAGES && p.nstg < own_nk && narrow_smem(p.tt, p.nstg + 1) <= budget) ++p.nstg;
    int smem = narrow_smem(p.tt, p.nstg);
    const int share = smem_share(static_cast<int>(narrow_cols(p.tt)));
    if (smem < share) smem = share;
    if (smem > kSmemMax) return fail(GAD_ERR_SHAPE, "linear ring of %d bytes", smem);   // never launched

    static OncePerContext attr_done;
    int st = raise_smem(reinterpret_cast<const void*>(gad::linear_narrow_kernel), attr_done, kSmemMax);
    if (st != GAD_OK) return st;
    CUtensorMap wmap, xmap;
    st = encode_rows(&wmap, w, p.fp16 != 0, p.K, p.N, ldw, ROWS);
    if (st == GAD_OK) st = encode_rows(&xmap, x, p.fp16 != 0, p.K, p.T, ldx, p.tt);
    if (st != GAD_OK) return st;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>((p.N + ROWS - 1) / ROWS * split), static_cast<unsigned>(token_tiles));
    cfg.blockDim = dim3(NARROW_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0] = pdl_attr();
    std::memset(&attr[1], 0, sizeof(attr[1]));
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, gad::linear_narrow_kernel, wmap, xmap, p);
    if (e != cudaSuccess) return fail(GAD_ERR_CUDA, "linear launch: %s", cudaGetErrorString(e));
    return GAD_OK;
}

int launch_wide(gad::lin::Params p, const void* x, long long ldx, const void* w, long long ldw, int sms,
                cudaStream_t s) {
    using namespace gad::lin;
    static OncePerContext attr_done;
    int st = raise_smem(reinterpret_cast<const void*>(gad::linear_wide_kernel), attr_done, kSmemMax);
    if (st != GAD_OK) return st;
    p.mt = (p.T + 255) / 256;
    p.nt = (p.N + 255) / 256;
    const long long tiles = static_cast<long long>(p.mt) * p.nt;
    CUtensorMap wmap, xmap;
    st = encode_rows(&wmap, w, p.fp16 != 0, p.K, p.N, ldw, ROWS);
    if (st == GAD_OK) st = encode_rows(&xmap, x, p.fp16 != 0, p.K, p.T, ldx, ROWS);
    if (st != GAD_OK) return st;
    const long long pairs = tiles < sms / 2 ? tiles : sms / 2;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    cfg.blockDim = dim3(WIDE_THREADS);
    static_assert(WIDE_SMEM <= kSmemMax, "ring and staging fit");
    cfg.dynamicSmemBytes = smem_share(512);   // its pair holds all of tensor memory
    cfg.stream = s;
    cudaLaunchAttribute attr = pdl_attr();
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, gad::linear_wide_kernel, wmap, xmap, p);
    if (e != cudaSuccess) return fail(GAD_ERR_CUDA, "linear launch: %s", cudaGetErrorString(e));
    return GAD_OK;
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
    const size_t ny = extent(T, ldy, N, oe);
    if (overlap(y, ny, x, extent(T, ldx, K, 2)) || overlap(y, ny, w, extent(N, ldw, K, 2)) ||
        (bias && overlap(y, ny, bias, static_cast<size_t>(N) * 2)))
        return fail(GAD_ERR_UNSUPPORTED, "y may not overlap x, w or bias");
    if (residual && !(residual == y && ldr == ldy) && overlap(y, ny, residual, extent(T, ldr, N, oe)))
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
    st = linear_status_word(&p.err);
    if (st != GAD_OK) return st;
    const long long wide_tiles = static_cast<long long>((T + 255) / 256) * ((N + 255) / 256);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return T > 256 && wide_tiles >= sms / 4 ? launch_wide(p, x, ldx, w, ldw, sms, s)
                                            : launch_narrow(p, x, ldx, w, ldw, sms, s);
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
