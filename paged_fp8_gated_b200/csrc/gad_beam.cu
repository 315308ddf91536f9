// gad_beam.cu - C ABI of the beam selection (gad_beam.cuh): argument checks,
// workspace layout and the two launches, chained with programmatic dependent
// launch.
#include <cuda_runtime.h>

#include "gad_beam.cuh"
#include "gad_host.h"

using namespace gad_host;

namespace {

// Logits per thread of beam_chunk_kernel: 32 (chunks of 8,192), or 8 when that
// leaves the GPU with few blocks.
constexpr int kLongE = 32, kShortE = 8;
constexpr long long kFewBlocks = 296;

int elems(long long rows, int V) {
    const long long long_chunks = (V + kLongE * gad::bm::THREADS - 1) / (kLongE * gad::bm::THREADS);
    return rows * long_chunks < kFewBlocks ? kShortE : kLongE;
}
int splits(long long rows, int V) {
    const int chunk = elems(rows, V) * gad::bm::THREADS;
    return (V + chunk - 1) / chunk;
}

struct BeamWs {
    size_t x_off, v_off, sum_off, total;
};
BeamWs beam_ws(long long rows, int V, int K) {
    const size_t parts = static_cast<size_t>(rows) * splits(rows, V);
    BeamWs w{};
    size_t off = 0;
    w.x_off = off;
    off = align_up(off + parts * K * sizeof(float));
    w.v_off = off;
    off = align_up(off + parts * K * sizeof(int));
    w.sum_off = off;
    off = align_up(off + parts * sizeof(float2));
    w.total = off;
    return w;
}

int check_beam(int G, int W, int V, int K) {
    if (G < 1 || W < 1 || W > GAD_MAX_BEAMS || static_cast<long long>(G) * W > GAD_MAX_B)
        return fail(GAD_ERR_SHAPE, "G=%d, W=%d: 1 to %d beams per request, G W at most %d", G, W, GAD_MAX_BEAMS,
                    GAD_MAX_B);
    if (K < 1 || K > GAD_MAX_BEAMS) return fail(GAD_ERR_SHAPE, "K=%d not in [1,%d]", K, GAD_MAX_BEAMS);
    if (V < 1 || V > GAD_MAX_VOCAB) return fail(GAD_ERR_SHAPE, "V=%d not in [1,%d]", V, GAD_MAX_VOCAB);
    return GAD_OK;
}
static_assert(GAD_MAX_BEAMS == gad::bm::MAX_K, "the merge kernel's per-beam tables");

template <class T>
void (*chunk_kernel(int e))(const gad::BeamParams) {
    return e == kLongE ? gad::beam_chunk_kernel<T, kLongE> : gad::beam_chunk_kernel<T, kShortE>;
}

}  // namespace

extern "C" {

size_t gad_beam_workspace_bytes(int G, int W, int V, int K) {
    if (check_beam(G, W, V, K) != GAD_OK) return 0;
    return beam_ws(static_cast<long long>(G) * W, V, K).total;
}

int gad_beam_select(const void* logits, int dtype, int64_t row_stride, const float* scores, const uint8_t* finished,
                    int pad_token, int G, int W, int V, int K, float* out_scores, int32_t* out_parent,
                    int32_t* out_token, void* workspace, size_t workspace_bytes, void* stream) {
    if (!logits || !scores || !out_scores || !out_parent || !out_token)
        return fail(GAD_ERR_NULL, "a required pointer is NULL");
    if (dtype != GAD_DTYPE_BF16 && dtype != GAD_DTYPE_F16 && dtype != GAD_DTYPE_F32)
        return fail(GAD_ERR_DTYPE, "logits of element type %d (bf16, f16 or f32)", dtype);
    int st = check_beam(G, W, V, K);
    if (st != GAD_OK) return st;
    if (row_stride < V) return fail(GAD_ERR_STRIDE, "row_stride=%lld < V=%d", static_cast<long long>(row_stride), V);
    if (pad_token < 0 || pad_token >= V) return fail(GAD_ERR_SHAPE, "pad_token=%d not in [0,%d)", pad_token, V);
    if (!aligned(logits, dtype == GAD_DTYPE_F32 ? 4 : 2) || !aligned(scores, 4) || !aligned(out_scores, 4) ||
        !aligned(out_parent, 4) || !aligned(out_token, 4))
        return fail(GAD_ERR_ALIGN, "every array must be aligned to its element size");
    const size_t in = static_cast<size_t>(G) * W * 4, out = static_cast<size_t>(G) * K * 4;
    for (const void* o : {static_cast<const void*>(out_scores), static_cast<const void*>(out_parent),
                          static_cast<const void*>(out_token)})
        if (overlap(scores, in, o, out)) return fail(GAD_ERR_UNSUPPORTED, "the outputs may not overlap scores");
    if (!workspace) return fail(GAD_ERR_WORKSPACE, "workspace is NULL");
    if (!aligned(workspace, kAlign)) return fail(GAD_ERR_ALIGN, "workspace must be 256-byte aligned");
    const long long rows = static_cast<long long>(G) * W;
    const BeamWs w = beam_ws(rows, V, K);
    if (workspace_bytes < w.total)
        return fail(GAD_ERR_WORKSPACE, "workspace %zu B < required %zu B", workspace_bytes, w.total);
    int sms = 0, major = 0;
    st = current_device_sms(&sms, &major);
    if (st != GAD_OK) return st;
    if (major != 10) return fail(GAD_ERR_DEVICE, "compute capability %d.x; this build targets sm_100a", major);

    gad::BeamParams p;
    std::memset(&p, 0, sizeof(p));
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.logits = logits;
    p.ld = row_stride;
    p.scores = scores;
    p.finished = finished;
    p.G = G;
    p.W = W;
    p.V = V;
    p.K = K;
    p.S = splits(rows, V);
    p.pad = pad_token;
    p.cand_x = reinterpret_cast<float*>(ws + w.x_off);
    p.cand_v = reinterpret_cast<int*>(ws + w.v_off);
    p.sums = reinterpret_cast<float2*>(ws + w.sum_off);
    p.out_scores = out_scores;
    p.out_parent = out_parent;
    p.out_token = out_token;

    const int e = elems(rows, V);
    void (*kern)(const gad::BeamParams) = dtype == GAD_DTYPE_BF16  ? chunk_kernel<__nv_bfloat16>(e)
                                          : dtype == GAD_DTYPE_F16 ? chunk_kernel<__half>(e)
                                                                   : chunk_kernel<float>(e);
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>(p.S), static_cast<unsigned>(rows));
    cfg.blockDim = dim3(gad::bm::THREADS);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaError_t err = cudaLaunchKernelEx(&cfg, kern, p);
    if (err != cudaSuccess) return fail(GAD_ERR_CUDA, "beam chunk launch: %s", cudaGetErrorString(err));
    cudaLaunchAttribute attr = pdl_attr();
    cfg.gridDim = dim3(static_cast<unsigned>(G));
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, gad::beam_merge_kernel, p);
    if (err != cudaSuccess) return fail(GAD_ERR_CUDA, "beam merge launch: %s", cudaGetErrorString(err));
    return GAD_OK;
}

}  // extern "C"
