// gad_linear.cuh - the linear layer with its epilogue:
//
//   y = act(x w^T + bias) + residual
//
//   x [T, K], w [N, K] bf16 or fp16 (both the same), rows ldx / ldw apart;
//   bias [N] of their type; residual and y [T, N] of y's type (x's or fp32),
//   rows ldr / ldy apart.  fp32 accumulation, epilogue in fp32, one rounding.
//
// Two kernels, both with operands staged by TMA (128-byte swizzle, 64 values of
// K a stage, anything outside the matrices read as zero), tcgen05 MMAs and
// accumulators in tensor memory:
//
// linear_narrow_kernel: few tokens, bound by the stream of w.  D[n][t] with
// the 128 weight rows as the MMA's M and up to 256 tokens as its N, one tile a
// block.  A cluster of up to 8 blocks shares a tile's K range, so that there
// are enough blocks to keep the loads of every SM in flight; their partial
// sums meet in shared memory over the cluster, added in rank order (the result
// does not depend on timing), and each block finishes a share of the tile.
// Measured: 64 x 8,192 x 32,001 to fp32 87.6 us, 6.1 TB/s of the copy rate's 6.56
// (the weights' stream is the bound); 1 x 1,024 x 8,192 5.5 us against 2.6 of
// stream: a load's latency, two crossings of the cluster and the epilogue's
// instruction fetch.
//
// linear_wide_kernel: many tokens, bound by the tensor cores.  Pairs of blocks
// (cta_group::2) on tiles of 256 tokens x BN weight rows (each block holds 128
// tokens and BN / 2 weight rows of a stage).  Persistent, with two accumulators
// in tensor memory, so that a tile's epilogue runs beside the next tile's MMAs;
// or, where the tiles are few, one tile a cluster of S = 2 or 4 pairs that share
// its K range: each finishes BN / S of the columns, with the other pairs' partial
// sums, which they copy into its shared memory (bulk copies move 15 bytes a clock
// between an SM and the others of its cluster, loads 9.5).  Measured: 4,096 x
// 8,192 x 14,336 620 us in bursts without bias and activation, 0.96 of the tensor
// cores' measured rate, 715 for seconds on end (the power limit); 4,096 x 256 x
// 32,000 69 us, 3.9 TB/s, where writing y is the bound; 512 x 8,192 x 2,304 27 us, of which 5 after the
// last MMA, on 36 of 74 pairs (36 tiles of 128 columns would need more clusters
// of four blocks than fit).
//
// Both can PROMOTE: the tensor cores cut the partial sum off at every step of
// 16, so a chain of K products loses 1.5e-6 of its terms' magnitudes per 1,024, and
// up to 3e-6 at its start (measured on sums of positive terms; others lose a tenth).
// Chains above 768 products for a fp32 result, and above 32,768 for a 16-bit one
// (which rounds off ten times what such a chain loses), change accumulators every
// 512 products, and warps that are idle otherwise add the finished one up in
// registers, rounding to nearest.  (Of those kernels two spill: linear_narrow_kernel
// with 64 sums a thread 52 bytes, with 128 20 bytes.)
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "gad_tc.cuh"

namespace gad {
namespace lin {

constexpr int BK = 64;                       // K per stage: one 128-byte row
constexpr int ROWS = 128;                    // weight rows (narrow), tokens or weight rows of a block (wide)
constexpr int TILE = ROWS * BK * 2;          // bytes of 128 rows of a stage
constexpr int SEG = 512 / BK;                // stages of a chain that is promoted

enum Act { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };
enum Out { OUT_BF16 = 0, OUT_F16 = 1, OUT_F32 = 2 };

struct Params {
    const void* bias;        // of x's type, or null
    const void* residual;    // of y's type, or null
    void* y;
    long long ldr, ldy;
    int T, K, N;
    int fp16;                // x, w and bias are fp16 (else bf16)
    int out, act;            // Out, Act
    int vec;                 // y (and residual) take aligned stores of four values
    int vec16;               // and of 16 bytes
    int tt, nstg;            // narrow: tokens per tile, ring stages
    int early;               // narrow: the blocks start while the launch before runs
    int mt, nt;              // wide: tiles along the tokens and along N
    int by_tma;              // wide: y leaves by TMA (rows of whole 16 bytes of 16-bit values, no residual)
    int* err;                // status word: STATUS_LINEAR_WAIT when a bounded wait gave up
};
constexpr int STATUS_LINEAR_WAIT = 16;

__device__ __forceinline__ float load16(const void* p, size_t i, bool fp16) {
    return fp16 ? __half2float(static_cast<const __half*>(p)[i])
                : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// The activation over N values.
template <int ACT, int N>
__device__ __forceinline__ void activate(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (ACT == ACT_RELU) v[i] = v[i] > 0.f || v[i] != v[i] ? v[i] : 0.f;
        if (ACT == ACT_GELU) v[i] = 0.5f * v[i] * (1.f + erff(v[i] * 0.70710678118654752f));
        if (ACT == ACT_GELU_TANH) {
            const float u = 0.79788456080286536f * (v[i] + 0.044715f * v[i] * v[i] * v[i]);
            v[i] = 0.5f * v[i] * (1.f + tanhf(u));
        }
        if (ACT == ACT_SILU) v[i] = v[i] / (1.f + expf(-v[i]));
    }
}
// `act` is uniform.  (A choice costs 135 cycles, as much as sixteen values' way
// through an epilogue: long loops take it outside.)
template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
    switch (act) {
        case ACT_RELU: activate<ACT_RELU>(v); break;
        case ACT_GELU: activate<ACT_GELU>(v); break;
        case ACT_GELU_TANH: activate<ACT_GELU_TANH>(v); break;
        case ACT_SILU: activate<ACT_SILU>(v); break;
        default: break;
    }
}

template <int OUT>
struct OutType;
template <>
struct OutType<OUT_F32> {
    using type = float;
    __device__ static float widen(float x) { return x; }
    __device__ static float round(float x) { return x; }
};
template <>
struct OutType<OUT_BF16> {
    using type = __nv_bfloat16;
    __device__ static float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
    __device__ static __nv_bfloat16 round(float x) { return __float2bfloat16(x); }
};
template <>
struct OutType<OUT_F16> {
    using type = __half;
    __device__ static float widen(__half x) { return __half2float(x); }
    __device__ static __half round(float x) { return __float2half(x); }
};

// Residual and store of four values y[t][n .. n+3] (fewer at the row's end).
template <int OUT>
__device__ __forceinline__ void store4(const Params& p, long long t, int n, const float* v) {
    using E = typename OutType<OUT>::type;
    const E* res = p.residual == nullptr ? nullptr : static_cast<const E*>(p.residual) + t * p.ldr + n;
    E* y = static_cast<E*>(p.y) + t * p.ldy + n;
    if (p.vec && n + 4 <= p.N) {
        float r[4] = {v[0], v[1], v[2], v[3]};
        if (res != nullptr) {
            E q[4];
            if (OUT == OUT_F32) *reinterpret_cast<uint4*>(q) = *reinterpret_cast<const uint4*>(res);
            else *reinterpret_cast<uint2*>(q) = *reinterpret_cast<const uint2*>(res);
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] += OutType<OUT>::widen(q[i]);
        }
        E o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = OutType<OUT>::round(r[i]);
        if (OUT == OUT_F32) *reinterpret_cast<uint4*>(y) = *reinterpret_cast<const uint4*>(o);
        else *reinterpret_cast<uint2*>(y) = *reinterpret_cast<const uint2*>(o);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n + i < p.N) y[i] = OutType<OUT>::round(res != nullptr ? v[i] + OutType<OUT>::widen(res[i]) : v[i]);
}

// Eight 16-bit values to fp32, and back.
__device__ __forceinline__ void widen8(const uint4& q, bool fp16, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (fp16) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        } else {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}
__device__ __forceinline__ uint4 narrow8(const float* v, bool fp16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (fp16) {
            w[i] = pack_f16x2(v[2 * i], v[2 * i + 1]);
        } else {
            __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<uint32_t*>(&b);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight values to y's type in 16 (or 32) bytes; eight of the residual.
template <int OUT>
__device__ __forceinline__ void store8(void* y, size_t at, const float (&v)[8]) {
    if (OUT == OUT_F32) {
        float4* d = reinterpret_cast<float4*>(static_cast<float*>(y) + at);
        d[0] = make_float4(v[0], v[1], v[2], v[3]);
        d[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(y) + at) = narrow8(v, OUT == OUT_F16);
    }
}
template <int OUT>
__device__ __forceinline__ void add8(const void* r, size_t at, float (&v)[8]) {
    if (OUT == OUT_F32) {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(r) + at);
        const float4 a = q[0], b = q[1];
        v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
        v[4] += b.x; v[5] += b.y; v[6] += b.z; v[7] += b.w;
    } else {
        float q[8];
        widen8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(r) + at), OUT == OUT_F16, q);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += q[i];
    }
}

// ---- thread-block clusters ----
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
    return r;
}
// (the aligned forms need the warp converged, which code with divergent loops
// before them does not promise by itself)
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive_relaxed() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
// Without the release: nothing that the thread wrote is read behind it.  (A
// release waits for the thread's stores to y: a thousand cycles and more.)
__device__ __forceinline__ void cluster_sync_relaxed() {
    cluster_arrive_relaxed();
    cluster_wait();
}
// The address of `addr` (this block's shared memory) in block `rank` of the cluster.
__device__ __forceinline__ uint32_t in_block(uint32_t addr, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];\n"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];\n"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
// Copies `bytes` (a multiple of 16) of this block's shared memory to another
// block's; they count on a barrier there.
__device__ __forceinline__ void bulk_to_block(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(dst),
                 "r"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
// TMA tile store; a group of one.
__device__ __forceinline__ void tma_store_2d(const void* tmap, uint32_t src, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n"
        "cp.async.bulk.commit_group;\n" ::"l"(reinterpret_cast<uint64_t>(tmap)),
        "r"(x), "r"(y), "r"(src)
        : "memory");
}
__device__ __forceinline__ void tma_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory"); }
__device__ __forceinline__ void tma_store_wait() { asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory"); }
__device__ __forceinline__ void tc_ld16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// (Of the block's scope: a release over the cluster would wait for the stores to
// y, 2,700 cycles a tile of linear_wide_kernel.)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];\n" ::"r"(addr) : "memory");
}

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(addr), "r"(v) : "memory");
}
// Counts `bytes` as arrived on a barrier of this block.
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}

// ---- tcgen05 on a pair of blocks (cta_group::2) ----
__device__ __forceinline__ void tc2_alloc(uint32_t dst_smem, uint32_t ncols) {  // whole warp, in both blocks
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(dst_smem), "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tc2_relinquish() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void tc2_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(taddr), "r"(ncols) : "memory");
}
// Arrives on `bar` in both blocks of the pair (cluster ranks first_block and
// first_block + 1) when its MMAs issued so far are done.  Whole warp.
__device__ __forceinline__ void tc2_commit_both(uint32_t bar, uint32_t first_block) {
    asm volatile(
        "{\n .reg .pred e;\n .reg .b32 rx;\n elect.sync rx|e, 0xffffffff;\n"
        " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}\n" ::"r"(bar),
        "h"(static_cast<uint16_t>(3u << first_block))
        : "memory");
}
// Four MMAs of K = 64: D (+)= A(a + 32 k bytes) B(b + 32 k bytes)^T, k = 0..3.  Whole warp, one lane issues.
__device__ __forceinline__ void tc2_mma_ss4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p, e, t;\n .reg .b32 rx;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n"
        " elect.sync rx|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n setp.eq.b32 t, 0, 0;\n"
        " add.u64 a1, %1, 2;\n add.u64 a2, %1, 4;\n add.u64 a3, %1, 6;\n"
        " add.u64 b1, %2, 2;\n add.u64 b2, %2, 4;\n add.u64 b3, %2, 6;\n"
        " @e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
        " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a1, b1, %3, t;\n"
        " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a2, b2, %3, t;\n"
        " @e tcgen05.mma.cta_group::2.kind::f16 [%0], a3, b3, %3, t;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// TMA tile load into this block's shared memory whose bytes count on a barrier
// of the pair's first block (`bar`: a cluster address).
__device__ __forceinline__ void tma2_load_2d(uint32_t dst, const void* tmap, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// Brings a tile into L2.
__device__ __forceinline__ void tma_prefetch_2d(const void* tmap, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];\n" ::"l"(reinterpret_cast<uint64_t>(tmap)),
                 "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const void* tmap) {
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(tmap)) : "memory");
}
__device__ __forceinline__ uint32_t idesc(const Params& p, int m, int n) {
    return p.fp16 ? idesc_f16_f32(m, n, 0) : idesc_bf16_f32(m, n, 0);
}

// ---- linear_narrow_kernel's shared memory ----
// ACC: accumulators that a thread promotes to (columns of tensor memory that
// its warp reads), or 0.  Warps 0 and 1 load and issue; all eight read the
// accumulator at the end, or with ACC eight others all along.
template <int ACC>
constexpr int NARROW_THREADS = ACC != 0 ? 320 : 256;
constexpr int NARROW_MAX_STAGES = 12;
constexpr int NARROW_BARS = 2 * NARROW_MAX_STAGES + 5;    // full, empty, done, 2 chain full, 2 chain empty
constexpr int RED_PITCH = ROWS + 4;                       // floats per token of the partial sums
__host__ __device__ constexpr int narrow_stage(int tt) { return TILE + tt * BK * 2; }
__host__ __device__ constexpr int narrow_ring(int tt, int nstg) {  // ring, later the partial sums
    const int ring = nstg * narrow_stage(tt), red = tt * RED_PITCH * 4;
    return ring > red ? ring : red;
}
__host__ __device__ constexpr int narrow_smem(int tt, int nstg) {
    return 1024 + narrow_ring(tt, nstg) + 8 * NARROW_BARS + 8;
}
__host__ __device__ constexpr int narrow_cols(int tt) { return tt <= 32 ? 32 : tt <= 64 ? 64 : tt <= 128 ? 128 : 256; }
__host__ __device__ constexpr int narrow_acc(int tt) { return tt <= 64 ? 32 : tt <= 128 ? 64 : 128; }

// ---- linear_wide_kernel's shared memory ----
constexpr int WIDE_EPI_WARPS = 8;
constexpr int WIDE_THREADS = 32 * (4 + WIDE_EPI_WARPS);
constexpr int WIDE_GROUP = 8;                             // token tiles that share a sweep over N
// S pairs share a tile's K range; each finishes BN / S of its columns, a warp
// OWN of them for 32 tokens.  Partial sums travel in pieces of 32 tokens x CW
// columns, y leaves in boxes of 32 x BOX.  The S - 1 pairs' pieces (sent, then
// received ones) take the ring's place: it is idle by then.
template <int BN, int S, bool PROMOTE>
struct Wide {
    static constexpr int STAGES = BN == 256 ? 5 : 8;
    static constexpr int STAGE = TILE + BN / 2 * BK * 2;  // 128 tokens and BN / 2 weight rows
    static constexpr int RING = STAGES * STAGE;
    static constexpr int OWN = BN / S / 2, CW = OWN < 32 ? OWN : 32, BOX = OWN < 64 ? OWN : 64;
    static constexpr int PIECE = 32 * CW * 4, PIECES = OWN / CW;
    static constexpr int SLOT = WIDE_EPI_WARPS * PIECES * PIECE;   // what a pair's block sends another
    static constexpr int RECV = (S - 1) * SLOT;
    static constexpr int SENT = S == 1 ? 0 : (S - 1 + PROMOTE) * SLOT;   // PROMOTE: its own sums as well
    static constexpr int EPI = WIDE_EPI_WARPS * (BN == 256 ? 8192 : 4096);
    static constexpr int STAGING = RING > SENT + RECV ? RING : SENT + RECV;   // where a warp's values wait to leave
    static constexpr int STAGING_WARP = S == 1 && BN == 256 ? 8192 : 4096;
    static constexpr int STRIPS = RING + EPI;             // a warp's bias, BOX values
    static constexpr int CTRL = STRIPS + WIDE_EPI_WARPS * 128;
    static constexpr int BUFS = S > 1 && !PROMOTE ? 1 : 2;  // accumulators
    static constexpr int BARS = 2 * STAGES + 6;           // full, empty, 2 tile full, 2 tile empty, done, received
    static constexpr int SMEM = 1024 + CTRL + 8 * BARS + 8 + 4 * 2 * S;
    static_assert(STAGING + WIDE_EPI_WARPS * STAGING_WARP <= STRIPS, "the staging fits");
    static_assert(!PROMOTE || BN == 128, "64 sums a thread");
};

// Offset of 16-byte chunk `chunk` of row `row`, in rows of P bytes that a TMA box
// with the swizzle of that width has: any eight rows' chunks of one index lie in
// different banks.
template <int P>
__device__ __forceinline__ uint32_t swizzled(int row, int chunk) {
    static_assert(P == 128 || P == 64 || P == 32, "a swizzle's width");
    return static_cast<uint32_t>(row * P + ((chunk ^ (P == 128 ? row & 7 : P == 64 ? (row >> 1) & 3 : (row >> 2) & 1)) << 4));
}

// The epilogue's values for what does not leave by TMA: 32 tokens x CW columns of
// fp32 in shared memory, 8 columns of a token a lane.  Bias and activation, in place:
template <int CW>
__device__ __forceinline__ void bias_act(const Params& p, uint8_t* tile, int n0, int lane) {
    constexpr int LPR = CW / 8, RPP = 32 / LPR;   // lanes a row, rows at a time
    const int r0 = lane / LPR, c = lane % LPR * 2, j = c * 4;
    float b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        b[e] = p.bias != nullptr && n0 + j + e < p.N ? load16(p.bias, n0 + j + e, p.fp16) : 0.f;
#pragma unroll 1
    for (int r = r0; r < 32; r += RPP) {
        float4* lo = reinterpret_cast<float4*>(tile + swizzled<CW * 4>(r, c));
        float4* hi = reinterpret_cast<float4*>(tile + swizzled<CW * 4>(r, c + 1));
        float v[8] = {lo->x + b[0], lo->y + b[1], lo->z + b[2], lo->w + b[3],
                      hi->x + b[4], hi->y + b[5], hi->z + b[6], hi->w + b[7]};
        activate(v, p.act);
        *lo = make_float4(v[0], v[1], v[2], v[3]);
        *hi = make_float4(v[4], v[5], v[6], v[7]);
    }
}
// To rows t0 .. t0 + 31, columns n0 .. n0 + CW - 1 of y, with the residual: 16
// bytes of y a lane (32 in fp32), all loads before the stores.
template <int OUT, int CW>
__device__ __forceinline__ void write_tile(const Params& p, const uint8_t* tile, long long t0, int n0, int lane) {
    constexpr int LPR = CW / 8, RPP = 32 / LPR;
    const int r0 = lane / LPR, c = lane % LPR * 2, j = c * 4;
    float v[LPR][8];
#pragma unroll
    for (int i = 0; i < LPR; ++i) {
        const float4 a = *reinterpret_cast<const float4*>(tile + swizzled<CW * 4>(RPP * i + r0, c));
        const float4 b = *reinterpret_cast<const float4*>(tile + swizzled<CW * 4>(RPP * i + r0, c + 1));
        v[i][0] = a.x; v[i][1] = a.y; v[i][2] = a.z; v[i][3] = a.w;
        v[i][4] = b.x; v[i][5] = b.y; v[i][6] = b.z; v[i][7] = b.w;
    }
    const int rows = p.T - t0 < 32 ? static_cast<int>(p.T - t0) : 32;
    if (p.residual != nullptr) {
        const size_t at = (t0 + r0) * p.ldr + n0 + j;
#pragma unroll
        for (int i = 0; i < LPR; ++i)
            if (RPP * i + r0 < rows) add8<OUT>(p.residual, at + RPP * i * p.ldr, v[i]);
    }
    const size_t at = (t0 + r0) * p.ldy + n0 + j;
#pragma unroll
    for (int i = 0; i < LPR; ++i)
        if (RPP * i + r0 < rows) store8<OUT>(p.y, at + RPP * i * p.ldy, v[i]);
}
// The same at the edge of y and for rows that are not aligned: a lane a column.
template <int OUT, int CW>
__device__ __forceinline__ void write_edge(const Params& p, const uint8_t* tile, long long t0, int n0, int lane) {
    using E = typename OutType<OUT>::type;
    constexpr int RPP = 32 / CW;   // rows at a time
    const int col = lane % CW;
    if (n0 + col >= p.N) return;
    const int rows = p.T - t0 < 32 ? static_cast<int>(p.T - t0) : 32;
    const E* res = p.residual == nullptr ? nullptr : static_cast<const E*>(p.residual) + t0 * p.ldr + n0 + col;
    E* y = static_cast<E*>(p.y) + t0 * p.ldy + n0 + col;
    for (int r0 = lane / CW; r0 < rows; r0 += 8 * RPP) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)   // (rows behind the 32nd: not used)
            v[i] = *reinterpret_cast<const float*>(tile + swizzled<CW * 4>((r0 + i * RPP) & 31, col >> 2) + (col & 3) * 4);
        if (res != nullptr) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (r0 + i * RPP < rows) v[i] += OutType<OUT>::widen(res[(r0 + i * RPP) * p.ldr]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (r0 + i * RPP < rows) y[(r0 + i * RPP) * p.ldy] = OutType<OUT>::round(v[i]);
    }
}
template <int OUT, int CW>
__device__ __forceinline__ void write_piece(const Params& p, const uint8_t* tile, long long t0, int n0, int lane) {
    if (p.vec16 && n0 + CW <= p.N) write_tile<OUT, CW>(p, tile, t0, n0, lane);
    else write_edge<OUT, CW>(p, tile, t0, n0, lane);
}

// 32 tokens x BOX columns of y (columns c0 ..) as a TMA store takes them from
// shared memory, sixteen columns at a time: sums from `get(offset, v)`, bias,
// activation, one rounding.
template <int BOX, bool F16, int ACT, class Get>
__device__ __forceinline__ void fill_box(const uint16_t* strip, bool bias, uint8_t* box, int at, int lane, Get get) {
#pragma unroll 1
    for (int g = 0; g < BOX / 16; ++g) {
        float v[16];
        get(at + 16 * g, v);
        if (bias) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float b[8];
                widen8(*reinterpret_cast<const uint4*>(strip + 16 * g + 8 * h), F16, b);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[8 * h + e] += b[e];
            }
        }
        activate<ACT>(v);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            *reinterpret_cast<uint4*>(box + swizzled<BOX * 2>(lane, 2 * g + h)) = narrow8(v + 8 * h, F16);
    }
}
template <int BOX, bool F16, class Get>
__device__ __forceinline__ void fill_box(const Params& p, const uint16_t* strip, uint8_t* box, int at, int lane, Get get) {
    const bool bias = p.bias != nullptr;
    switch (p.act) {
        case ACT_RELU: fill_box<BOX, F16, ACT_RELU>(strip, bias, box, at, lane, get); break;
        case ACT_GELU: fill_box<BOX, F16, ACT_GELU>(strip, bias, box, at, lane, get); break;
        case ACT_GELU_TANH: fill_box<BOX, F16, ACT_GELU_TANH>(strip, bias, box, at, lane, get); break;
        case ACT_SILU: fill_box<BOX, F16, ACT_SILU>(strip, bias, box, at, lane, get); break;
        default: fill_box<BOX, F16, ACT_NONE>(strip, bias, box, at, lane, get); break;
    }
}

// A warp's OWN columns of 32 tokens (rows row0 .., columns col0 .. of y): sums
// from `get`, then bias, activation, residual, rounding and y.  In rolled loops:
// unrolled over the tile the activations' code is far larger than what the SM
// keeps of it.  `last` runs when the accumulator has been read.
template <int BN, int S, bool PROMOTE, class Get, class Last>
__device__ __forceinline__ void wide_finish(const Params& p, const CUtensorMap* y_map, uint8_t* stage, uint16_t* strip,
                                            long long row0, int col0, int lane, Get get, Last last) {
    using C = Wide<BN, S, PROMOTE>;
    if (row0 >= p.T) {
        last();
        return;
    }
    if (!PROMOTE && p.by_tma) {
        if (lane == 0) tma_store_wait_read();   // the tile before has left its boxes
#pragma unroll 1
        for (int blk = 0; blk < C::OWN / C::BOX; ++blk) {
            const int at = blk * C::BOX, c0 = col0 + at;
            uint8_t* box = stage + 32 * 2 * at;
            if (p.bias != nullptr) {
#pragma unroll
                for (int c = lane; c < C::BOX; c += 32)
                    strip[c] = c0 + c < p.N ? static_cast<const uint16_t*>(p.bias)[c0 + c] : static_cast<uint16_t>(0);
            }
            __syncwarp();
            if (p.fp16) fill_box<C::BOX, true>(p, strip, box, at, lane, get);
            else fill_box<C::BOX, false>(p, strip, box, at, lane, get);
            __syncwarp();   // (the strip is free)
        }
        last();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
#pragma unroll
            for (int blk = 0; blk < C::OWN / C::BOX; ++blk)
                if (col0 + blk * C::BOX < p.N)
                    tma_store_2d(y_map, smem_addr(stage + 32 * 2 * C::BOX * blk), col0 + blk * C::BOX, static_cast<int>(row0));
        }
        return;
    }
    // (PROMOTE's sums are in registers, unless they were sent)
#pragma unroll(PROMOTE && S == 1 ? C::PIECES : 1)
    for (int q = 0; q < C::PIECES; ++q) {
        const int c0 = col0 + q * C::CW;
#pragma unroll
        for (int g = 0; g < C::CW / 16; ++g) {
            float v[16];
            get(q * C::CW + 16 * g, v);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                *reinterpret_cast<float4*>(stage + swizzled<C::CW * 4>(lane, 4 * g + k)) =
                    make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        }
        if (q == C::PIECES - 1) last();
        __syncwarp();
        if (c0 < p.N) {
            if (p.bias != nullptr || p.act != ACT_NONE) {
                bias_act<C::CW>(p, stage, c0, lane);
                __syncwarp();
            }
            if (p.out == OUT_F32) write_piece<OUT_F32, C::CW>(p, stage, row0, c0, lane);
            else if (p.out == OUT_BF16) write_piece<OUT_BF16, C::CW>(p, stage, row0, c0, lane);
            else write_piece<OUT_F16, C::CW>(p, stage, row0, c0, lane);
        }
        __syncwarp();
    }
}

// The block's share (1 / S of the tokens x 128 rows) of a narrow tile: the
// cluster's partial sums, in rank order, and the epilogue.  Several items' loads
// are in flight at a time: those from other blocks take about 500 cycles.
template <int S, int THREADS>
__device__ __forceinline__ void narrow_finish(const Params& p, uint32_t red, int rank, int n0, int t0, int tn) {
    constexpr int U = S >= 4 ? 1 : S == 2 ? 2 : 4;
    uint32_t base[S];
#pragma unroll
    for (int s = 0; s < S; ++s) base[s] = in_block(red, s);
    const int items = tn * (ROWS / 4);
    const int i0 = static_cast<int>(static_cast<long long>(items) * rank / S);
    const int i1 = static_cast<int>(static_cast<long long>(items) * (rank + 1) / S);
    for (int ii = i0 + static_cast<int>(threadIdx.x); ii < i1; ii += U * THREADS) {
        float4 q[U][S];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = ii + u * THREADS;
            if (i >= i1 || n0 + i % (ROWS / 4) * 4 >= p.N) {   // not stored, so not loaded: what is
                // loaded has been used, so has arrived, when the block tells the others that it is done
#pragma unroll
                for (int s = 0; s < S; ++s) q[u][s] = make_float4(0.f, 0.f, 0.f, 0.f);
                continue;
            }
            const uint32_t at = static_cast<uint32_t>(i / (ROWS / 4) * RED_PITCH + i % (ROWS / 4) * 4) * 4u;
#pragma unroll
            for (int s = 0; s < S; ++s) q[u][s] = S == 1 ? ld_shared_f4(red + at) : ld_cluster_f4(base[s] + at);
        }
        float v[4 * U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int n = n0 + (ii + u * THREADS) % (ROWS / 4) * 4;
            v[4 * u] = q[u][0].x; v[4 * u + 1] = q[u][0].y; v[4 * u + 2] = q[u][0].z; v[4 * u + 3] = q[u][0].w;
#pragma unroll
            for (int s = 1; s < S; ++s) {
                v[4 * u] += q[u][s].x; v[4 * u + 1] += q[u][s].y; v[4 * u + 2] += q[u][s].z; v[4 * u + 3] += q[u][s].w;
            }
            if (p.bias != nullptr) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < p.N) v[4 * u + e] += load16(p.bias, n + e, p.fp16);
            }
        }
        if (p.act != ACT_NONE) activate(v, p.act);
        auto store = [&](auto out) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = ii + u * THREADS, n = n0 + i % (ROWS / 4) * 4;
                if (i < i1 && n < p.N) store4<decltype(out)::value>(p, t0 + i / (ROWS / 4), n, v + 4 * u);
            }
        };
        if (p.out == OUT_F32) store(std::integral_constant<int, OUT_F32>());
        else if (p.out == OUT_BF16) store(std::integral_constant<int, OUT_BF16>());
        else store(std::integral_constant<int, OUT_F16>());
    }
}
}  // namespace lin

template <int ACC>
__global__ void __launch_bounds__(lin::NARROW_THREADS<ACC>, ACC == 0 ? 4 : ACC == 128 ? 1 : 2)
    linear_narrow_kernel(const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map,
                         const lin::Params p) {
    using namespace lin;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    const int xs = p.tt * BK * 2, NSTG = p.nstg;
    const uint32_t ring = smem_addr(smem);                 // [NSTG] weight rows, then [NSTG] token rows
    const uint32_t xring = ring + NSTG * TILE;
    uint8_t* ctrl = smem + narrow_ring(p.tt, NSTG);
    const uint32_t bar0 = smem_addr(ctrl);
    auto FULL = [&](int s) { return bar0 + 8u * static_cast<uint32_t>(s); };
    auto EMPTY = [&](int s) { return bar0 + 8u * static_cast<uint32_t>(NSTG + s); };
    const uint32_t DONE = bar0 + 8u * (2 * NARROW_MAX_STAGES);
    auto CFULL = [&](int b) { return bar0 + 8u * static_cast<uint32_t>(2 * NARROW_MAX_STAGES + 1 + b); };
    auto CEMPTY = [&](int b) { return bar0 + 8u * static_cast<uint32_t>(2 * NARROW_MAX_STAGES + 3 + b); };
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 8 * NARROW_BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(ctrl + 8 * NARROW_BARS + 4);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int split = static_cast<int>(gridDim.x) / ((p.N + ROWS - 1) / ROWS);   // the cluster's blocks
    const int rank = static_cast<int>(cluster_rank());
    const int n0 = static_cast<int>(blockIdx.x) / split * ROWS, t0 = blockIdx.y * p.tt;
    const int nk_all = (p.K + BK - 1) / BK;
    const int k_first = static_cast<int>(static_cast<long long>(nk_all) * rank / split);
    const int nk = static_cast<int>(static_cast<long long>(nk_all) * (rank + 1) / split) - k_first;
    const uint32_t cols = static_cast<uint32_t>(narrow_cols(p.tt)), ncols = ACC != 0 ? 2 * cols : cols;

    if (tid == 0) {
        tma_prefetch_map(&w_map);
        tma_prefetch_map(&x_map);
        for (int s = 0; s < NSTG; ++s) {
            mbar_init(FULL(s), 1);
            mbar_init(EMPTY(s), 1);
        }
        mbar_init(DONE, 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(CFULL(b), 1);
            mbar_init(CEMPTY(b), 8);
        }
        *abort_flag = 0;
        mbar_fence_init();
    }
    if (warp == 1) {
        tc_alloc(smem_addr(tmem_slot), ncols);
        tc_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();
    // the first weights into L2 while the launch before still runs (it may write
    // them: L2 is where both meet)
    if (p.early && tid == 0)
        for (int kc = 0; kc < nk && kc < NSTG; ++kc) tma_prefetch_2d(&w_map, (k_first + kc) * BK, n0);
    pdl_wait_primary();

    if (warp == 0) {
        if (lane == 0) {
            const uint32_t bytes = static_cast<uint32_t>(TILE + xs);
            int issued = 0;
            for (int kc = 0; kc < nk; ++kc) {
                const int s = kc % NSTG;
                if (kc >= NSTG && !wait_bounded(EMPTY(s), (kc / NSTG - 1) & 1, abort_flag)) break;
                mbar_arrive_expect_tx(FULL(s), bytes);
                tma_load_2d(ring + s * TILE, &w_map, (k_first + kc) * BK, n0, FULL(s));
                tma_load_2d(xring + s * xs, &x_map, (k_first + kc) * BK, t0, FULL(s));
                issued = kc + 1;
            }
            // every load has landed before the shared memory is used again
            for (int kc = issued > NSTG ? issued - NSTG : 0; kc < issued; ++kc)
                wait_bounded(FULL(kc % NSTG), (kc / NSTG) & 1, abort_flag, false, TEARDOWN_LIMIT_NS);
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint32_t id = idesc(p, ROWS, p.tt);
        for (int kc = 0; kc < nk; ++kc) {
            const int s = kc % NSTG;
            const int chain = ACC != 0 ? kc / SEG : 0, first = chain * SEG, b = chain & 1;
            if (ACC != 0 && kc == first && chain >= 2) {   // the accumulator of two chains ago has been added up
                const bool free = wait_bounded(CEMPTY(b), (chain / 2 - 1) & 1, abort_flag);
                if (!__all_sync(0xffffffffu, free)) break;
            }
            const bool got = wait_bounded(FULL(s), (kc / NSTG) & 1, abort_flag);
            if (!__all_sync(0xffffffffu, got)) break;
            tc_fence_after();
            const uint32_t wa = ring + s * TILE, xa = xring + s * xs;
            const uint64_t ad[4] = {smem_desc_sw128(wa), smem_desc_sw128(wa + 32), smem_desc_sw128(wa + 64),
                                    smem_desc_sw128(wa + 96)};
            const uint64_t bd[4] = {smem_desc_sw128(xa), smem_desc_sw128(xa + 32), smem_desc_sw128(xa + 64),
                                    smem_desc_sw128(xa + 96)};
            tc_mma_ss4(tmem + b * cols, ad, bd, id, kc > first ? 1u : 0u);
            tc_commit(EMPTY(s));
            if (ACC != 0 && (kc == first + SEG - 1 || kc == nk - 1)) tc_commit(CFULL(b));
        }
        tc_commit(DONE);
    }
    // ---- promotion: warp w >= 2 adds up 32 rows of the chains' accumulators, of
    // one half of the columns (all of them, if there are 32) ----
    const int quad = warp & 3, half = ACC != 0 ? (warp - 2) >> 2 : warp >> 2;
    const uint32_t row = tmem + (static_cast<uint32_t>(32 * quad) << 16);
    float acc[ACC != 0 ? ACC : 1];
    if (ACC != 0 && warp >= 2) {
#pragma unroll
        for (int j = 0; j < ACC; ++j) acc[j] = 0.f;
        const int chains = (nk + SEG - 1) / SEG;
        for (int c = 0; c < chains; ++c) {
            const bool got = wait_bounded(CFULL(c & 1), (c / 2) & 1, abort_flag);
            if (!__all_sync(0xffffffffu, got)) break;
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < ACC / 32; ++q) {
                const uint32_t c0 = static_cast<uint32_t>(half * ACC + 32 * q);
                if (c0 >= cols) continue;
                uint32_t v[32];
                tc_ld32(row + (c & 1) * cols + c0, v);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; ++j) acc[32 * q + j] += __uint_as_float(v[j]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(CEMPTY(c & 1));
        }
    }
    const bool done = wait_bounded(DONE, 0, abort_flag, false, TEARDOWN_LIMIT_NS);
    tc_fence_after();
    __syncthreads();   // the loads have landed (warp 0) and the MMAs are done: the ring is free

    // ---- partial sums to shared memory: red[t][n], lane = weight row ----
    const int tn = p.T - t0 < p.tt ? p.T - t0 : p.tt;      // the tile's tokens
    float* red = reinterpret_cast<float*>(smem);
    if (ACC != 0) {
#pragma unroll
        for (int j = 0; j < ACC; ++j)
            if (warp >= 2 && half * ACC + j < tn) red[(half * ACC + j) * RED_PITCH + 32 * quad + lane] = acc[j];
    } else if (__all_sync(0xffffffffu, done && !*abort_flag)) {
        uint32_t v[32];
        for (int c0 = 32 * half; c0 < tn; c0 += 64) {
            tc_ld32(row + static_cast<uint32_t>(c0), v);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (c0 + j < tn) red[(c0 + j) * RED_PITCH + 32 * quad + lane] = __uint_as_float(v[j]);
        }
    }
    tc_fence_before();
    if (split > 1) cluster_sync();
    else __syncthreads();

    // ---- this block's share of the tile: sum over the cluster, epilogue ----
    switch (split) {
        case 1: narrow_finish<1, NARROW_THREADS<ACC>>(p, ring, rank, n0, t0, tn); break;
        case 2: narrow_finish<2, NARROW_THREADS<ACC>>(p, ring, rank, n0, t0, tn); break;
        case 4: narrow_finish<4, NARROW_THREADS<ACC>>(p, ring, rank, n0, t0, tn); break;
        default: narrow_finish<8, NARROW_THREADS<ACC>>(p, ring, rank, n0, t0, tn); break;
    }
    if (split > 1) cluster_sync_relaxed();   // the other blocks have read this one's sums
    if (warp == 1) {
        tc_fence_after();
        tc_dealloc(tmem, ncols);
    }
    if (tid == 0 && *abort_flag) atomicOr(p.err, STATUS_LINEAR_WAIT);
}

template <int BN, int S, bool PROMOTE>
__global__ void __launch_bounds__(lin::WIDE_THREADS, 1)
    linear_wide_kernel(const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map,
                       const __grid_constant__ CUtensorMap y_map, const lin::Params p) {
    using namespace lin;
    using C = Wide<BN, S, PROMOTE>;
    constexpr int STAGES = C::STAGES, STAGE = C::STAGE, COLS = BN * C::BUFS;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw);
    uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
    const uint32_t ring = smem_addr(smem);                 // [stage][128 tokens | BN / 2 weight rows]
    uint8_t* ctrl = smem + C::CTRL;
    const uint32_t bar0 = smem_addr(ctrl);
    auto FULL = [&](int s) { return bar0 + 8u * static_cast<uint32_t>(s); };
    auto EMPTY = [&](int s) { return bar0 + 8u * static_cast<uint32_t>(STAGES + s); };
    auto TFULL = [&](int b) { return bar0 + 8u * static_cast<uint32_t>(2 * STAGES + b); };
    auto TEMPTY = [&](int b) { return bar0 + 8u * static_cast<uint32_t>(2 * STAGES + 2 + b); };
    const uint32_t DONE = bar0 + 8u * (2 * STAGES + 4), RECEIVED = DONE + 8u;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 8 * C::BARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(ctrl + 8 * C::BARS + 4);
    // stages that each block of the cluster has asked for (bit 31: it gave up)
    uint32_t* ends = reinterpret_cast<uint32_t*>(ctrl + 8 * C::BARS + 8);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t crank = cluster_rank(), leader = crank & ~1u;   // the pair's first block
    const int rank = static_cast<int>(crank & 1);
    const int tiles = p.mt * p.nt;
    // the pair's tiles and its part of their K range
    const int pair = blockIdx.x / (2 * S), pairs = S > 1 ? tiles : gridDim.x / 2;
    const int nk_all = (p.K + BK - 1) / BK, part = S > 1 ? static_cast<int>(crank >> 1) : 0;
    const int k_first = static_cast<int>(static_cast<long long>(nk_all) * part / S);
    const int nk = static_cast<int>(static_cast<long long>(nk_all) * (part + 1) / S) - k_first;

    // tile -> (token tile, weight tile): WIDE_GROUP token tiles sweep N together,
    // so the pairs at work at one time share rows of x and of w in L2
    auto place = [&](int tile, int* m, int* n) {
        const int per = WIDE_GROUP * p.nt, g = tile / per, in = tile - g * per;
        const int gm = p.mt - g * WIDE_GROUP < WIDE_GROUP ? p.mt - g * WIDE_GROUP : WIDE_GROUP;
        *m = g * WIDE_GROUP + in % gm;
        *n = in / gm;
    };
    // S > 1: the only tile, its first token in this block, and how many of the four
    // epilogue quads have tokens (only those exchange sums)
    int m_only = 0, n_only = 0;
    if (S > 1) place(pair, &m_only, &n_only);
    const long long t_only = static_cast<long long>(m_only) * 256 + rank * ROWS;
    const int quads = t_only >= p.T ? 0 : p.T - t_only >= ROWS ? 4 : static_cast<int>(p.T - t_only + 31) / 32;

    if (tid == 0) {
        tma_prefetch_map(&w_map);
        tma_prefetch_map(&x_map);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(FULL(s), 1);    // used in the pair's first block: its expected bytes are both blocks'
            mbar_init(EMPTY(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(TFULL(b), 1);
            mbar_init(TEMPTY(b), 2 * WIDE_EPI_WARPS);
        }
        mbar_init(DONE, 1);
        mbar_init(RECEIVED, 1);
        *abort_flag = 0;
        mbar_fence_init();
        if (S > 1) mbar_arrive_expect_tx(RECEIVED, C::RECV / 4 * static_cast<uint32_t>(quads));
    }
    if (warp == 2) {
        tc2_alloc(smem_addr(tmem_slot), COLS);
        tc2_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_relaxed();   // both blocks' barriers exist (mbar_fence_init released them)
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();
    pdl_wait_primary();

    // Epilogue warps: 32 tokens, and half of the columns that the pair finishes.
    const int quad = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quad) << 16);
    uint8_t* stage = smem + C::STAGING + (warp - 4) * C::STAGING_WARP;
    uint16_t* strip = reinterpret_cast<uint16_t*>(smem + C::STRIPS + (warp - 4) * 128);
    // its pieces in slot `slot` of the sent or received ones
    auto piece = [&](uint8_t* from, int slot) { return from + slot * C::SLOT + (warp - 4) * C::PIECES * C::PIECE; };

    float acc[PROMOTE ? BN / 2 : 1];   // PROMOTE: the sums
    uint32_t src = 0;                  // the warp's first column of the first pair's share
    bool summed = true;                // they are there

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int tile = pair; tile < tiles && ok; tile += pairs) {
                int m, n;
                place(tile, &m, &n);
                const int y = m * 256 + rank * ROWS, z = n * BN + rank * (BN / 2);
                for (int kc = 0; kc < nk; ++kc, ++it) {
                    const int s = it % STAGES;
                    if (it >= STAGES && !wait_bounded(EMPTY(s), (it / STAGES - 1) & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) mbar_arrive_expect_tx(FULL(s), 2 * STAGE);
                    const uint32_t full = in_block(FULL(s), leader);
                    tma2_load_2d(ring + s * STAGE, &x_map, (k_first + kc) * BK, y, full);
                    tma2_load_2d(ring + s * STAGE + TILE, &w_map, (k_first + kc) * BK, z, full);
                }
            }
            ends[crank] = static_cast<uint32_t>(it);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t id = idesc(p, 256, BN);
            int it = 0, local = 0;
            bool ok = true;
            // `local` counts the accumulators handed to the epilogue: one a tile, or
            // with PROMOTE one a chain
            for (int tile = pair; tile < tiles && ok; tile += pairs) {
                for (int kc = 0; kc < nk; ++kc, ++it) {
                    const int s = it % STAGES, b = local & 1;
                    const bool first = PROMOTE ? kc % SEG == 0 : kc == 0;
                    if (first && local >= 2) {
                        const bool got = wait_bounded(TEMPTY(b), (local / 2 - 1) & 1, abort_flag);
                        ok = __all_sync(0xffffffffu, got);
                        if (!ok) break;
                    }
                    const bool got = wait_bounded(FULL(s), (it / STAGES) & 1, abort_flag);
                    ok = __all_sync(0xffffffffu, got);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a = ring + s * STAGE;
                    tc2_mma_ss4(tmem + static_cast<uint32_t>(BN * b), smem_desc_sw128(a), smem_desc_sw128(a + TILE), id,
                                first ? 0u : 1u);
                    tc2_commit_both(EMPTY(s), leader);
                    if (kc == nk - 1 || (PROMOTE && kc % SEG == SEG - 1)) {
                        tc2_commit_both(TFULL(b), leader);
                        ++local;
                    }
                }
            }
            tc2_commit_both(DONE, leader);
        }
    } else if (warp >= 4) {
        int local = 0;
        for (int tile = pair; tile < tiles && summed; tile += pairs) {
            const int chains = PROMOTE ? (nk + SEG - 1) / SEG : 1;
            if (PROMOTE) {
#pragma unroll
                for (int j = 0; j < BN / 2; ++j) acc[j] = 0.f;
            }
            auto release = [&] {   // the accumulator has been read
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(in_block(TEMPTY((local - 1) & 1), leader));
            };
            for (int c = 0; c < chains; ++c) {
                const int b = local & 1;
                const bool got = wait_bounded(TFULL(b), (local / 2) & 1, abort_flag);
                summed = __all_sync(0xffffffffu, got);
                if (!summed) break;
                ++local;
                tc_fence_after();
                src = lanes + static_cast<uint32_t>(BN * b + C::OWN * half);
                if (PROMOTE) {
#pragma unroll
                    for (int j = 0; j < BN / 2; j += 16) {
                        uint32_t raw[16];
                        tc_ld16(src + static_cast<uint32_t>(j / C::OWN * (BN / S) + j % C::OWN), raw);
                        tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) acc[j + e] += __uint_as_float(raw[e]);
                    }
                    release();
                }
            }
            if (!summed || S > 1) break;   // (S > 1: its only tile)
            int m, n;
            place(tile, &m, &n);
            wide_finish<BN, S, PROMOTE>(
                p, &y_map, stage, strip, static_cast<long long>(m) * 256 + rank * ROWS + quad * 32, n * BN + half * C::OWN, lane,
                [&](int at, float (&v)[16]) {
                    if (PROMOTE) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = acc[PROMOTE ? at + e : 0];
                    } else {
                        uint32_t raw[16];
                        tc_ld16(src + static_cast<uint32_t>(at), raw);
                        tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(raw[e]);
                    }
                },
                [&] {
                    if (!PROMOTE) release();
                });
        }
        if (S == 1 && lane == 0) tma_store_wait();
    }
    // ---- teardown: the MMAs are done (both blocks see it), then tensor memory goes ----
    // (one warp asks; the others would take its issue slots from the epilogue)
    if (warp == 1) wait_bounded(DONE, 0, abort_flag, false, TEARDOWN_LIMIT_NS);
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
        if (*abort_flag) ends[crank] |= 0x80000000u;
        for (uint32_t b = 0; b < 2 * S; ++b)
            if (b != crank) st_cluster_u32(in_block(smem_addr(ends + crank), b), ends[crank]);
    }
    if (warp == 0) cluster_arrive();
    else cluster_arrive_relaxed();
    if (S > 1 && warp >= 4 && summed && quad < quads) {
        // the other pairs' columns of this one's sums, for them to have; its MMAs are
        // done, so its ring is free
#pragma unroll(PROMOTE ? S : 1)
        for (int d = 0; d < S; ++d) {
            if (!PROMOTE && d == part) continue;
            uint8_t* to = piece(smem, PROMOTE ? d : d - (d > part));
#pragma unroll(PROMOTE ? C::OWN / 16 : 1)
            for (int j = 0; j < C::OWN; j += 16) {
                float v[16];
                if (PROMOTE) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = acc[PROMOTE ? d * C::OWN + j + e : 0];
                } else {
                    uint32_t raw[16];
                    tc_ld16(src + static_cast<uint32_t>(d * (BN / S) + j), raw);
                    tc_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(raw[e]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    *reinterpret_cast<float4*>(to + j / C::CW * C::PIECE + swizzled<C::CW * 4>(lane, j % C::CW / 4 + k)) =
                        make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            }
        }
        fence_proxy_async_smem();
    }
    cluster_wait();
    // All loads were used, so have landed, unless a block gave up.  Then each pair's
    // first block waits for the ones in flight, on its barriers: for a stage that
    // only one block has asked for, it makes up what the barrier still expects.
    bool gave_up = false;   // (the same answer in all blocks)
#pragma unroll
    for (int i = 0; i < S; ++i) gave_up |= ends[2 * i] != ends[2 * i + 1] || (ends[2 * i] >> 31) != 0;
    if (gave_up) {
        if (rank == 0 && tid == 0) {
            const int mine = static_cast<int>(ends[crank] & 0x7fffffffu);
            const int theirs = static_cast<int>(ends[crank + 1] & 0x7fffffffu);
            const int last = mine > theirs ? mine : theirs;
            for (int i = last > STAGES ? last - STAGES : 0; i < last; ++i) {
                if (i >= theirs) mbar_complete_tx(FULL(i % STAGES), STAGE);
                else if (i >= mine) mbar_arrive_expect_tx(FULL(i % STAGES), STAGE);
                wait_bounded(FULL(i % STAGES), (i / STAGES) & 1, abort_flag, false, TEARDOWN_LIMIT_NS);
            }
        }
        __syncthreads();
        cluster_sync();
    }
    if (S > 1) {
        // every block's ring is idle: the pieces go to the pairs that finish them (of
        // a pair that gave up too, whatever they are: none waits for what never comes)
        if (warp >= 4 && quad < quads) {
            uint8_t* received = smem + C::SENT;
            if (lane == 0) {
#pragma unroll 1
                for (int d = 0; d < S; ++d)
                    if (d != part)
                        bulk_to_block(in_block(smem_addr(piece(received, part - (part > d))), 2 * d + rank),
                                      smem_addr(piece(smem, PROMOTE ? d : d - (d > part))), C::PIECES * C::PIECE,
                                      in_block(RECEIVED, 2 * d + rank));
            }
            __syncwarp();
            const bool got = wait_bounded(RECEIVED, 0, abort_flag, false, TEARDOWN_LIMIT_NS);
            tc_fence_after();
            if (__all_sync(0xffffffffu, got && !gave_up)) {
                const int first = part * (BN / S);
                wide_finish<BN, S, PROMOTE>(
                    p, &y_map, stage, strip, t_only + quad * 32, n_only * BN + first + half * C::OWN, lane,
                    [&](int at, float (&v)[16]) {   // its own sums, then the others' by rank
                        const int q = at / C::CW * C::PIECE, chunk = at % C::CW / 4;
                        if (PROMOTE) {
                            const uint8_t* own = piece(smem, part) + q;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float4 f = *reinterpret_cast<const float4*>(own + swizzled<C::CW * 4>(lane, chunk + k));
                                v[4 * k] = f.x; v[4 * k + 1] = f.y; v[4 * k + 2] = f.z; v[4 * k + 3] = f.w;
                            }
                        } else {
                            uint32_t raw[16];
                            tc_ld16(lanes + static_cast<uint32_t>(first + half * C::OWN + at), raw);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(raw[e]);
                        }
#pragma unroll
                        for (int o = 0; o < S - 1; ++o) {
                            const uint8_t* from = piece(received, o) + q;
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float4 f = *reinterpret_cast<const float4*>(from + swizzled<C::CW * 4>(lane, chunk + k));
                                v[4 * k] += f.x; v[4 * k + 1] += f.y; v[4 * k + 2] += f.z; v[4 * k + 3] += f.w;
                            }
                        }
                    },
                    [] {});
                if (lane == 0) tma_store_wait();
            }
        }
        cluster_sync_relaxed();   // the sent pieces have left
    }
    if (warp == 2) {
        tc_fence_after();
        tc2_dealloc(tmem, COLS);
    }
    if (tid == 0 && *abort_flag) atomicOr(p.err, STATUS_LINEAR_WAIT);
}

}  // namespace gad
