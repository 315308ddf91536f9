// gad_beam.cu - C ABI of the beam selection (gad_beam.cuh): argument checks,
// workspace layout and the two launches, chained with programmatic dependent
// launch.
#include <cuda_runtime.h>

#include "gad_beam.cuh"
#include "gad_host.h"

using namespace gad_host;

namespace {

// How a row is cut for beam_chunk_kernel: into as many segments as make kBlocks
// blocks, the ones that 148 SMs hold at a time, of NV vectors per thread.
constexpr long long kBlocks = 148 * 4;

struct Cut {
    int S, NV;
};
Cut cut_rows(long long rows, int V, int elem) {
    const int vec = 16 / elem * gad::bm::THREADS;   // elements in one vector of every thread
    const int vectors = (V + vec - 1) / vec;
    long long S = kBlocks / rows;
    if (S < 1) S = 1;
    if (S > vectors) S = vectors;
    Cut c{};
    c.NV = static_cast<int>((vectors + S - 1) / S);
    c.S = (vectors + c.NV - 1) / c.NV;
    return c;
}

struct BeamWs {
    size_t cand_off, sum_off, total;
};
// For logits of either size: the larger of the two cuts.
BeamWs beam_ws(long long rows, int V, int K) {
    const int s2 = cut_rows(rows, V, 2).S, s4 = cut_rows(rows, V, 4).S;
    const size_t parts = static_cast<size_t>(rows) * (s2 > s4 ? s2 : s4);
    BeamWs w{};
    size_t off = 0;
    w.cand_off = off;
    off = align_up(off + parts * K * sizeof(uint64_t));
    w.sum_off = off;
    off = align_up(off + parts * sizeof(gad::bm::Sum));
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
    if (!workspace) return fail(GAD_ERR_WORKSPACE, "workspace is NULL");
    if (!aligned(workspace, kAlign)) return fail(GAD_ERR_ALIGN, "workspace must be 256-byte aligned");
    const long long rows = static_cast<long long>(G) * W;
    const BeamWs w = beam_ws(rows, V, K);
    if (workspace_bytes < w.total)
        return fail(GAD_ERR_WORKSPACE, "workspace %zu B < required %zu B", workspace_bytes, w.total);
    // (a request's results are written while other requests' scores and marks are still
    // read, but behind the last read of the logits)
    const size_t in = static_cast<size_t>(rows), out = static_cast<size_t>(G) * K * 4;
    const size_t all = ((rows - 1) * static_cast<size_t>(row_stride) + V) * (dtype == GAD_DTYPE_F32 ? 4 : 2);
    if (written_overlap({{out_scores, out}, {out_parent, out}, {out_token, out}, {workspace, w.total}},
                        {{scores, in * 4}, {finished, in}}) ||
        overlap(workspace, w.total, logits, all))
        return fail(GAD_ERR_UNSUPPORTED, "outputs and workspace may not overlap scores, finished or one another, "
                                         "nor the workspace logits");
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
    const Cut cut = cut_rows(rows, V, dtype == GAD_DTYPE_F32 ? 4 : 2);
    p.S = cut.S;
    p.NV = cut.NV;
    p.pad = pad_token;
    p.cand = reinterpret_cast<uint64_t*>(ws + w.cand_off);
    p.sums = reinterpret_cast<gad::bm::Sum*>(ws + w.sum_off);
    p.out_scores = out_scores;
    p.out_parent = out_parent;
    p.out_token = out_token;

    void (*kern)(const gad::BeamParams) = dtype == GAD_DTYPE_BF16  ? gad::beam_chunk_kernel<__nv_bfloat16>
                                          : dtype == GAD_DTYPE_F16 ? gad::beam_chunk_kernel<__half>
                                                                   : gad::beam_chunk_kernel<float>;
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
