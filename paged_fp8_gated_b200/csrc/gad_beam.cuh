// gad_beam.cuh - beam search's selection: the K best of all (beam, token)
// candidates of a request.
//
//   score(w, v) = s_w + (x_wv - lse_w),   lse_w = log sum_v exp(x_wv)
//
// for the logits x of beam w and its score s_w so far; a finished beam has the
// one candidate (pad token, s_w).  The K highest scores are wanted in order,
// ties by the lower w V + v.
//
// The order within a beam is that of its logits, so one pass over the logits
// suffices: each block takes a segment of a row, batch after batch through
// registers, and leaves its K best logits, its maximum m and sum of exp(x - m)
// (beam_chunk_kernel); a second kernel joins the segments' sums into lse_w and
// ranks the W S K candidates (beam_merge_kernel).  The scores that decide the
// order are held in 64 bits: candidates of different beams can be as close as
// the last bits of lse_w.  A row's elements go to threads by their index,
// whatever the row's alignment, so equal rows have equal sums and tie exactly.
//
// The K best of a segment: the K-th largest of at least K group maxima of the
// first batch is a lower bound of the K-th largest element, few elements reach
// it, and ranking those by counting leaves the K best and a threshold that
// later batches rarely pass.  If more than the buffer holds pass it (long
// ties), the block takes the batch's K best one after another.
//
// Bound: one read of the logits; beside it one MUFU exponential per logit (16 a
// cycle and SM: three quarters of the read's time for 16-bit logits) and about
// four other instructions (maxima and sums in packed pairs).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gad_ptx.cuh"

namespace gad {
namespace bm {

constexpr int THREADS = 256;
constexpr int MAX_K = 64;
constexpr int BUF = 512;        // a segment's candidates that are ranked by counting
constexpr int MERGE_BUF = 1024; // a request's
constexpr int STAGES = 3;       // batches in shared memory: one in use, two on their way
constexpr float NEG_INF = -__builtin_huge_valf();
constexpr float LOG2E = 1.4426950408889634f;

// A word of two 16-bit elements of which `left` belong to the row.
__device__ __forceinline__ uint32_t cut16(uint32_t w, int left, uint32_t lowest) {
    return left >= 2 ? w : left == 1 ? (w & 0xffffu) | (lowest & 0xffff0000u) : lowest;
}
// Element types: VEC elements in a 16-byte vector of four words.  pair(w, p) is
// elements 2p and 2p + 1 in fp32; word_max the elementwise maximum of two words
// (a NaN loses); cut keeps the first `left` elements of a word, the others are -inf.
__device__ __forceinline__ float2 f32_pair(uint32_t lo, uint32_t hi) {
    return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
template <class T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int VEC = 4;
    static constexpr uint32_t LOWEST = 0xff800000u;   // -inf in every element of a word
    __device__ static float2 pair(const uint32_t (&w)[4], int p) { return f32_pair(w[2 * p], w[2 * p + 1]); }
    __device__ static uint32_t word_max(uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }
    __device__ static float top(uint32_t w) { return fmaxf(__uint_as_float(w), NEG_INF); }
    __device__ static float one(const uint8_t* p) { return *reinterpret_cast<const float*>(p); }
    __device__ static uint32_t cut(uint32_t w, int left) { return left > 0 ? w : LOWEST; }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int VEC = 8;
    static constexpr uint32_t LOWEST = 0xff80ff80u;
    __device__ static float2 pair(const uint32_t (&w)[4], int p) { return f32_pair(w[p] << 16, w[p] & 0xffff0000u); }
    __device__ static uint32_t word_max(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.bf16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    __device__ static float top(uint32_t w) {
        return fmaxf(fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)), NEG_INF);
    }
    __device__ static float one(const uint8_t* p) { return __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p)); }
    __device__ static uint32_t cut(uint32_t w, int left) { return cut16(w, left, LOWEST); }
};
template <>
struct Elem<__half> {
    static constexpr int VEC = 8;
    static constexpr uint32_t LOWEST = 0xfc00fc00u;
    __device__ static float2 pair(const uint32_t (&w)[4], int p) {
        return __half22float2(*reinterpret_cast<const __half2*>(&w[p]));
    }
    __device__ static uint32_t word_max(uint32_t a, uint32_t b) {
        uint32_t d;
        asm("max.f16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
        return d;
    }
    __device__ static float top(uint32_t w) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
        return fmaxf(fmaxf(f.x, f.y), NEG_INF);
    }
    __device__ static float one(const uint8_t* p) { return __half2float(*reinterpret_cast<const __half*>(p)); }
    __device__ static uint32_t cut(uint32_t w, int left) { return cut16(w, left, LOWEST); }
};

// Packed fp32 pairs.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 z, x, y;\n"
        " mov.b64 {%0, %1}, z;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 z, x, y;\n"
        " mov.b64 {%0, %1}, z;\n}\n"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// Order-preserving map of floats (no NaN) to unsigned.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);   // -0 and +0 are equal
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float from_key(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

// The K-th largest of the maxima of groups of threads (8 threads a group for
// K <= 16, else 2), -inf if K groups have nothing: a lower bound of the K-th
// largest element.  Each thread brings its own maximum.  All threads call it.
__device__ __forceinline__ float group_threshold(float mine, int K, uint32_t* s_key, float* s_thr) {
    const int tid = threadIdx.x;
    uint32_t k = order_key(mine);
    const int gs = K <= 16 ? 8 : 2;
    k = max(k, __shfl_xor_sync(0xffffffffu, k, 1));
    if (gs == 8) {
        k = max(k, __shfl_xor_sync(0xffffffffu, k, 2));
        k = max(k, __shfl_xor_sync(0xffffffffu, k, 4));
    }
    if (tid % gs == 0) s_key[tid / gs] = k;
    __syncthreads();
    if (tid < 32) {
        uint32_t v[4];
        const int per = THREADS / gs / 32;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < per ? s_key[tid + 32 * i] : 0u;
        uint32_t top = 0;
        for (int r = 0; r < K; ++r) {
            const uint32_t m = max(max(v[0], v[1]), max(v[2], v[3]));
            top = __reduce_max_sync(0xffffffffu, m);
            const uint32_t who = __ballot_sync(0xffffffffu, m == top);
            if (tid == __ffs(who) - 1) {   // takes one of its values out
                if (v[0] == top) v[0] = 0;
                else if (v[1] == top) v[1] = 0;
                else if (v[2] == top) v[2] = 0;
                else v[3] = 0;
            }
        }
        if (tid == 0) *s_thr = top == 0 ? NEG_INF : from_key(top);
    }
    __syncthreads();
    return *s_thr;
}

}  // namespace bm

struct BeamParams {
    const void* logits;
    long long ld;             // elements from one row of logits to the next
    const float* scores;      // [G W]
    const uint8_t* finished;  // [G W] or null
    int G, W, V, K;
    int S, B;                 // S segments per row, of B batches
    int pad;
    float* cand_x;            // [G W S K] the segments' best logits, best first (-inf: none)
    int* cand_v;              // [G W S K] their tokens
    float2* sums;             // [G W S] maximum, sum of exp(x - maximum)
    float* out_scores;
    int *out_parent, *out_token;
};

// Rank of (x, v) among n entries: how many come before it.
__device__ __forceinline__ int beam_rank(const float* xs, const int* vs, int n, float x, int v) {
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
        const float e = xs[j];
        rank += e > x || (e == x && vs[j] < v);
    }
    return rank;
}

// One block per (segment, row).  A batch is NV vectors per thread: thread t
// holds elements v0 + (i THREADS + t) VEC + u.  Batches arrive in shared memory
// by cp.async, two ahead; a row that starts off a 16-byte boundary (by `mis`
// bytes, the same for all its vectors) is copied from the boundary before it,
// and an element vector is cut out of the two aligned ones that it lies in.
template <class T, int NV>
__global__ void __launch_bounds__(bm::THREADS, 4) beam_chunk_kernel(const BeamParams p) {
    using namespace bm;
    using E = Elem<T>;
    constexpr int VEC = E::VEC, BATCH = NV * VEC * THREADS, ESZ = static_cast<int>(sizeof(T));
    constexpr int STAGE = BATCH * ESZ + 16;
    extern __shared__ __align__(16) uint8_t ring[];   // [STAGES][STAGE]
    __shared__ float s_m[THREADS / 32], s_thr;
    __shared__ double s_sum[THREADS / 32];
    __shared__ uint32_t s_key[128];
    __shared__ float s_x[BUF], s_bx[MAX_K];
    __shared__ int s_v[BUF], s_bv[MAX_K], s_new[3];
    const int tid = threadIdx.x, lane = tid & 31, row = blockIdx.y;
    pdl_launch_dependents();
    {   // a finished beam's logits and those of a dead one are not needed
        const float s = p.scores[row];
        if ((p.finished != nullptr && p.finished[row] != 0) || !(s > NEG_INF)) return;
    }
    if (tid < 3) s_new[tid] = 0;
    const T* x = static_cast<const T*>(p.logits) + row * p.ld;
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15);
    const int first = static_cast<int>(static_cast<long long>(blockIdx.x) * p.B * BATCH);
    const int left = (p.V - first + BATCH - 1) / BATCH, batches = left < p.B ? left : p.B;
    const uint32_t ring_addr = smem_addr(ring);

    // 16-byte pieces of batch b that hold elements of the row; the others become zero
    const uint8_t* base = reinterpret_cast<const uint8_t*>(x) - mis;
    const long long row_bytes = static_cast<long long>(p.V) * ESZ + mis;
    auto fetch = [&](int b) {
        if (b < batches) {
            const long long at = (static_cast<long long>(first) + static_cast<long long>(b) * BATCH) * ESZ;
            const uint32_t dst = ring_addr + static_cast<uint32_t>(b % STAGES) * STAGE;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int off = (i * THREADS + tid) * 16;
                cp_async16(dst + off, at + off < row_bytes ? base + at + off : base, at + off < row_bytes ? 16 : 0);
            }
            if (mis != 0 && tid == 0) {
                const int off = BATCH * ESZ;
                cp_async16(dst + off, at + off < row_bytes ? base + at + off : base, at + off < row_bytes ? 16 : 0);
            }
        }
        cp_async_commit();
    };
    fetch(0);
    fetch(1);

    float m = NEG_INF, sum = 0.f;       // this thread's maximum and sum of exp(x - m)
    float thr = NEG_INF;                // elements of the K best are above it (from the second batch on)
    int held = 0;                       // entries of the buffer: at most 2 K + 15 between batches

    // What batch b left in the buffer (all threads, after a barrier behind b's
    // entries): cuts the buffer to its K best, best first, when it is long, for
    // the first batch and at the end (`last`).
    auto settle = [&](int b, bool last) {
        const int fresh = s_new[b % 3];
        if (fresh > BUF - held) {
            // more than the buffer holds: the batch's K best one after another
            const uint8_t* st = ring + (b % STAGES) * STAGE + mis;
            const int v0 = first + b * BATCH;
            float last_x = __builtin_huge_valf();
            int last_v = -1;
            for (int k = 0; k < p.K; ++k) {
                float bx = NEG_INF;
                int bv = 0x7fffffff;
                for (int o = tid; o < BATCH && v0 + o < p.V; o += THREADS) {
                    const float e = E::one(st + o * ESZ);
                    const int v = v0 + o;
                    const bool after = e < last_x || (e == last_x && v > last_v);
                    if (after && e > NEG_INF && (e > bx || (e == bx && v < bv))) {
                        bx = e;
                        bv = v;
                    }
                }
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) {
                    const float ox = __shfl_xor_sync(0xffffffffu, bx, d);
                    const int ov = __shfl_xor_sync(0xffffffffu, bv, d);
                    if (ox > bx || (ox == bx && ov < bv)) {
                        bx = ox;
                        bv = ov;
                    }
                }
                __syncthreads();   // the last round's readers are done
                if (lane == 0) {   // the buffer's end is scratch: what overflowed it is dropped
                    s_x[BUF - 1 - (tid >> 5)] = bx;
                    s_v[BUF - 1 - (tid >> 5)] = bv;
                }
                __syncthreads();
                for (int w = 0; w < THREADS / 32; ++w) {
                    const float ox = s_x[BUF - 1 - w];
                    const int ov = s_v[BUF - 1 - w];
                    if (ox > bx || (ox == bx && ov < bv)) {
                        bx = ox;
                        bv = ov;
                    }
                }
                if (tid == 0) {
                    s_x[held + k] = bx;
                    s_v[held + k] = bv;
                }
                last_x = bx;
                last_v = bv;
            }
            held += p.K;   // a batch that overflows the buffer has K elements above -inf
            __syncthreads();
        } else {
            held += fresh;
        }
        if (b == 0 || last || held >= 2 * p.K + 16) {
            for (int i = tid; i < held; i += THREADS) {
                const float e = s_x[i];
                const int v = s_v[i], rank = beam_rank(s_x, s_v, held, e, v);
                if (rank < p.K) {
                    s_bx[rank] = e;
                    s_bv[rank] = v;
                }
            }
            __syncthreads();
            if (held >= p.K) {
                held = p.K;
                thr = s_bx[p.K - 1];   // an equal element further on comes after it
            } else {
                thr = NEG_INF;
            }
            if (!last) {
                for (int k = tid; k < held; k += THREADS) {
                    s_x[k] = s_bx[k];
                    s_v[k] = s_bv[k];
                }
            }
        }
    };

    for (int b = 0; b < batches; ++b) {
        cp_async_wait<1>();
        __syncthreads();   // batch b is there, and everything of batch b - 1 is done
        if (b > 0) settle(b - 1, false);
        fetch(b + 2);
        if (tid == 0) s_new[(b + 1) % 3] = 0;

        // ---- the thread's elements; past the row's end -inf ----
        const int v0 = first + b * BATCH;
        const uint8_t* st = ring + (b % STAGES) * STAGE;
        uint32_t raw[NV][4];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint4 lo = *reinterpret_cast<const uint4*>(st + (i * THREADS + tid) * 16);
            raw[i][0] = lo.x; raw[i][1] = lo.y; raw[i][2] = lo.z; raw[i][3] = lo.w;
        }
        if (mis != 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const uint4 hi = *reinterpret_cast<const uint4*>(st + (i * THREADS + tid) * 16 + 16);
                uint32_t q[8] = {raw[i][0], raw[i][1], raw[i][2], raw[i][3], hi.x, hi.y, hi.z, hi.w};
                if (mis & 8) {
#pragma unroll
                    for (int j = 0; j < 6; ++j) q[j] = q[j + 2];
                }
                if (mis & 4) {
#pragma unroll
                    for (int j = 0; j < 5; ++j) q[j] = q[j + 1];
                }
                const int bits = 8 * (mis & 3);
#pragma unroll
                for (int j = 0; j < 4; ++j) raw[i][j] = __funnelshift_r(q[j], q[j + 1], bits);
            }
        }
        if (v0 + BATCH > p.V) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = v0 + (i * THREADS + tid) * VEC;
#pragma unroll
                for (int j = 0; j < 4; ++j) raw[i][j] = E::cut(raw[i][j], p.V - v - j * (4 / ESZ));
            }
        }

        // ---- maximum and sum of exponentials (a NaN or +inf makes the sum NaN) ----
        uint32_t wm = raw[0][0];
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) wm = E::word_max(wm, raw[i][j]);
        const float mine = E::top(wm);
        if (mine > m) {
            sum *= fast_exp2((m - mine) * LOG2E);
            m = mine;
        }
        const float ref = m > NEG_INF ? m : 0.f;
        float2 part = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < VEC / 2; ++q) {
                const float2 d = mul2(add2(E::pair(raw[i], q), make_float2(-ref, -ref)), make_float2(LOG2E, LOG2E));
                part = add2(part, make_float2(fast_exp2(d.x), fast_exp2(d.y)));
            }
        sum += part.x + part.y;

        // ---- elements that may belong to the K best: the warp looks through the
        // elements of each thread whose maximum passes, one a lane ----
        if (b == 0) thr = group_threshold(mine, p.K, s_key, &s_thr);
        uint32_t pass = __ballot_sync(0xffffffffu, mine > NEG_INF && (b == 0 ? mine >= thr : mine > thr));
        while (pass != 0) {
            const int from = __ffs(pass) - 1;
            pass &= pass - 1;
            const int o = ((lane / VEC) * THREADS + (tid - lane + from)) * VEC + lane % VEC;
            float e = NEG_INF;
            if (lane < NV * VEC && v0 + o < p.V) e = E::one(st + mis + o * ESZ);
            const bool in = e > NEG_INF && (b == 0 ? e >= thr : e > thr);
            const uint32_t who = __ballot_sync(0xffffffffu, in);
            int at = 0;
            if (lane == 0) at = atomicAdd(&s_new[b % 3], __popc(who));
            at = held + __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << lane) - 1));
            if (in && at < BUF) {
                s_x[at] = e;
                s_v[at] = v0 + o;
            }
        }
    }
    __syncthreads();
    settle(batches - 1, true);
    {
        const size_t at = (static_cast<size_t>(row) * p.S + blockIdx.x) * p.K;
        for (int k = tid; k < p.K; k += THREADS) {
            p.cand_x[at + k] = k < held ? s_bx[k] : NEG_INF;
            p.cand_v[at + k] = k < held ? s_bv[k] : -1;
        }
    }

    // ---- the segment's maximum and sum ----
    float top = m;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (lane == 0) s_m[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) top = fmaxf(top, s_m[w]);
    double total = m == top ? sum : sum * fast_exp2((m - top) * LOG2E);   // equal infinities have no difference
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    if (lane == 0) s_sum[tid >> 5] = total;
    __syncthreads();
    if (tid == 0) {
        total = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) total += s_sum[w];
        p.sums[static_cast<size_t>(row) * p.S + blockIdx.x] = make_float2(top, static_cast<float>(total));
    }
}
template <class T, int NV>
constexpr int beam_smem() {
    return bm::STAGES * (NV * bm::Elem<T>::VEC * bm::THREADS * static_cast<int>(sizeof(T)) + 16);
}

// One block per request.
__global__ void __launch_bounds__(bm::THREADS) beam_merge_kernel(const BeamParams p) {
    using namespace bm;
    __shared__ double s_lse[MAX_K], s_cum[MAX_K];   // per beam; a beam without candidates has lse NaN
    __shared__ uint8_t s_done[MAX_K];
    __shared__ uint32_t s_key[128];
    __shared__ float s_thr;
    __shared__ double s_score[MERGE_BUF];
    __shared__ int s_flat[MERGE_BUF], s_n;
    const int tid = threadIdx.x, lane = tid & 31, g = blockIdx.x;
    pdl_wait_primary();
    if (tid == 0) s_n = 0;
    for (int w = tid >> 5; w < p.W; w += THREADS / 32) {
        const int row = g * p.W + w;
        const float cum = p.scores[row];
        const bool done = p.finished != nullptr && p.finished[row] != 0;
        double lse = 0;
        if (!done && cum > NEG_INF) {
            const float2* ms = p.sums + static_cast<size_t>(row) * p.S;
            float m = NEG_INF;
            for (int s = lane; s < p.S; s += 32) m = fmaxf(m, ms[s].x);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            double sum = 0;
            for (int s = lane; s < p.S; s += 32) {
                const float2 q = ms[s];
                // a segment without a finite logit adds nothing, unless it holds a NaN
                sum += q.x > NEG_INF ? q.y * exp(static_cast<double>(q.x) - m)
                                     : static_cast<double>(q.y != q.y ? q.y : 0.f);
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            lse = m + log(sum);
        }
        if (lane == 0) {
            s_lse[w] = lse;
            s_cum[w] = cum;
            s_done[w] = done ? 2 : (cum > NEG_INF ? 0 : 1);
        }
    }
    __syncthreads();

    // candidate c of the request: list (w, s), place k
    const int SK = p.S * p.K;
    const int C = p.W * SK;
    auto score = [&](int c, int* flat) -> double {
        const int w = c / SK, q = c - w * SK;
        const int state = s_done[w];
        double key = NEG_INF;
        *flat = w * p.V;
        if (state == 2) {
            if (q == 0) {
                key = s_cum[w];
                *flat += p.pad;
            }
        } else if (state == 0) {
            const size_t at = static_cast<size_t>(g * p.W + w) * SK + q;
            const float x = p.cand_x[at];
            if (x > NEG_INF) {
                key = s_cum[w] + (x - s_lse[w]);
                *flat += p.cand_v[at];
            }
        }
        return key > NEG_INF ? key : static_cast<double>(NEG_INF);   // a NaN has no place
    };
    float mine = NEG_INF;
    for (int c = tid; c < C; c += THREADS) {
        int flat;
        mine = fmaxf(mine, static_cast<float>(score(c, &flat)));
    }
    // scores rounded to 32 bits keep their order up to ties, so the threshold
    // on them lets every candidate of the K best through
    const float thr = group_threshold(mine, p.K, s_key, &s_thr);
    if (mine >= thr)
        for (int c = tid; c < C; c += THREADS) {
            int flat;
            const double key = score(c, &flat);
            if (static_cast<float>(key) >= thr && key > NEG_INF) {
                const int k = atomicAdd(&s_n, 1);
                if (k < MERGE_BUF) {
                    s_score[k] = key;
                    s_flat[k] = flat;
                }
            }
        }
    __syncthreads();
    const int n = s_n;
    float* out_s = p.out_scores + static_cast<size_t>(g) * p.K;
    int* out_p = p.out_parent + static_cast<size_t>(g) * p.K;
    int* out_t = p.out_token + static_cast<size_t>(g) * p.K;
    auto put = [&](int k, double key, int flat) {
        const int w = flat / p.V;
        out_s[k] = static_cast<float>(key);
        out_p[k] = key > NEG_INF ? g * p.W + w : -1;
        out_t[k] = key > NEG_INF ? flat - w * p.V : -1;
    };
    if (n <= MERGE_BUF) {
        for (int i = tid; i < n; i += THREADS) {
            const double key = s_score[i];
            const int flat = s_flat[i];
            int rank = 0;
#pragma unroll 4
            for (int j = 0; j < n; ++j) rank += s_score[j] > key || (s_score[j] == key && s_flat[j] < flat);
            if (rank < p.K) put(rank, key, flat);
        }
        for (int k = n + tid; k < p.K; k += THREADS) put(k, NEG_INF, 0);
    } else {
        double last = __builtin_huge_val();
        int last_f = -1;
        for (int k = 0; k < p.K; ++k) {
            double bk = NEG_INF;
            int bf = 0x7fffffff;
            for (int c = tid; c < C; c += THREADS) {
                int flat;
                const double key = score(c, &flat);
                const bool behind = key < last || (key == last && flat > last_f);
                if (behind && key > NEG_INF && (key > bk || (key == bk && flat < bf))) {
                    bk = key;
                    bf = flat;
                }
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) {
                const double ok = __shfl_xor_sync(0xffffffffu, bk, d);
                const int of = __shfl_xor_sync(0xffffffffu, bf, d);
                if (ok > bk || (ok == bk && of < bf)) {
                    bk = ok;
                    bf = of;
                }
            }
            __syncthreads();
            if (lane == 0) {
                s_score[tid >> 5] = bk;
                s_flat[tid >> 5] = bf;
            }
            __syncthreads();
            bk = s_score[0];
            bf = s_flat[0];
            for (int w = 1; w < THREADS / 32; ++w)
                if (s_score[w] > bk || (s_score[w] == bk && s_flat[w] < bf)) {
                    bk = s_score[w];
                    bf = s_flat[w];
                }
            if (tid == 0) put(k, bk, bk > NEG_INF ? bf : 0);
            last = bk;
            last_f = bf;
        }
    }
}

}  // namespace gad
