// gad_beam.cuh - beam search's selection: the K best of all (beam, token)
// candidates of a request.
//
//   score(w, v) = s_w + (x_wv - lse_w),   lse_w = log sum_v exp(x_wv)
//
// for the logits x of beam w and its score s_w so far; a finished beam has the
// one candidate (pad token, s_w), a beam whose score is not finite none.  The K
// highest scores are wanted in order, ties by the lower w V + v.
//
// The order within a beam is that of its logits, so one pass over the logits
// suffices: each block takes a segment of a row and leaves its K best logits,
// its maximum m and its sum of exp(x - m) (beam_chunk_kernel); a second kernel
// joins the segments' sums into lse_w and ranks the W S K candidates
// (beam_merge_kernel).  The scores that decide the order are held in 64 bits, and
// all sums in 64 bits or two words of 32, but those of the at most 32 exponentials
// that a thread adds up at a time: lse_w is as good as the exponentials, however
// long the row.  Those are of fp32 differences d scaled by log2 e, each off by at
// most 2.5 2^-24 |d| (the difference's rounding, the product's and the constant's) +
// 2^-22 (the function) + 2^-24 (a product with it) of itself.  A thread's terms are
// relative to a reference that moves only when the maximum passes it by FAR, so a
// term is scaled once for its own difference, once for every FAR that the maximum
// rises behind it, and once to the segment's maximum.  With the weights p_v = exp(x_v - lse) the sum of p times the distance to the row's
// maximum is at most log V, so lse_w is off by at most
//
//   2^-24 (2.5 (log V + 2 FAR) + 5 (2 + log V / FAR) + 18),
//
// 6.6e-6 at V = 2^24, and in practice by 1e-7 (the terms' errors differ in sign).  A
// row's elements go to threads by their index, whatever the row's alignment, so
// equal rows have equal sums and tie exactly.
//
// The K best of a segment: every thread streams its elements through registers
// for its maximum and sum only, without a barrier.  The K-th largest of the
// threads' maxima is a lower bound of the K-th largest element that about K
// threads reach; their elements (K / 256 of the segment) are read again, and
// the few that pass are ranked by counting.  If more than the buffer holds pass
// (long ties), the block takes the K best one after another.
//
// Bound: one read of the logits; beside it one MUFU exponential per logit (16 a
// cycle and SM: three quarters of the read's time for 16-bit logits) and about
// four other instructions (maxima and sums in packed pairs).  Measured, both
// kernels: 32 x 8 beams over 131,072 bf16 logits, K = 16, 21.1 us with the logits
// in L2 and 23.5 from memory (a read at the copy rate 10.2, the exponentials 7.5,
// about 8 the segment's end: threshold, second look, ranks, merge); 16 x 4 over
// 32,001 fp32 10.6, 1 x 4 over 32,000 8.3, all latency.  Asking for lines ahead of
// their load into L2 gained 1.3 us from memory and lost 1.2 from L2, where a product
// has just left them: not done.
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
constexpr int GROUP = 4;        // vectors of a thread in flight
constexpr float NEG_INF = -__builtin_huge_valf();
constexpr float LOG2E = 1.4426950408889634f;
constexpr float FAR = 4.f;      // how far a maximum may pass the sum's reference

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

// A candidate as one number, larger is better: the value, then the lower index.
// 0: none.
__device__ __forceinline__ uint64_t pack(float x, uint32_t v) {
    return static_cast<uint64_t>(order_key(x)) << 32 | (0xffffffffu - v);
}
__device__ __forceinline__ float value_of(uint64_t c) { return from_key(static_cast<uint32_t>(c >> 32)); }
__device__ __forceinline__ uint32_t index_of(uint64_t c) { return 0xffffffffu - static_cast<uint32_t>(c); }

// A value that at least K of the threads' keys reach, and as far as their bits
// tell them apart no more than K + K / 4 + 2: bisection over the key's bits below
// those that all finite keys share, a counting barrier a bit (about 5 of them, 200
// cycles each; from the top bit on 12, one warp alone took 300 a bit, taking
// maxima out one by one 200 for each of the K).  All threads call it, once; its
// first barrier also covers what they wrote before.
__device__ __forceinline__ uint32_t kth_key(uint32_t key, int K) {
    constexpr uint32_t NONE = 0x007fffffu;   // order_key(-inf)
    __shared__ uint32_t s_lo[THREADS / 32], s_hi[THREADS / 32];
    const bool some = key > NONE;
    const uint32_t lo = __reduce_min_sync(0xffffffffu, some ? key : ~0u);
    const uint32_t hi = __reduce_max_sync(0xffffffffu, some ? key : 0u);
    if ((threadIdx.x & 31) == 0) {
        s_lo[threadIdx.x >> 5] = lo;
        s_hi[threadIdx.x >> 5] = hi;
    }
    int c = __syncthreads_count(some);
    if (c < K) return NONE;
    uint32_t least = s_lo[0], most = s_hi[0];
#pragma unroll
    for (int w = 1; w < THREADS / 32; ++w) {
        least = min(least, s_lo[w]);
        most = max(most, s_hi[w]);
    }
    int bit = 31 - __clz(static_cast<int>(least ^ most));   // -1: all the same
    uint32_t t = bit < 0 ? most : most & ~((2u << bit) - 1);
#pragma unroll 1
    for (; bit >= 0 && c > K + K / 4 + 2; --bit) {
        const uint32_t up = t | 1u << bit;
        const int n = __syncthreads_count(key >= up);
        if (n >= K) {
            t = up;
            c = n;
        }
    }
    return max(t, NONE);   // below it keys are no numbers'
}

}  // namespace bm

namespace bm {
struct Sum {
    double sum;   // of exp(x - top)
    float top;    // the maximum
};
}  // namespace bm

struct BeamParams {
    const void* logits;
    long long ld;             // elements from one row of logits to the next
    const float* scores;      // [G W]
    const uint8_t* finished;  // [G W] or null
    int G, W, V, K;
    int S, NV;                // S segments per row, of NV vectors per thread
    int pad;
    uint64_t* cand;           // [G W S K] the segments' best logits and their tokens, best first (see pack)
    bm::Sum* sums;            // [G W S]
    float* out_scores;
    int *out_parent, *out_token;
};

// How many of n candidates are better.
__device__ __forceinline__ int beam_rank(const uint64_t* c, int n, uint64_t mine) {
    int rank = 0;
#pragma unroll 2
    for (int j = 0; j < n; ++j) rank += c[j] > mine;
    return rank;
}

// 16 bytes of a row from element v on; elements past the row's end are -inf.  A
// row that starts off a 16-byte boundary (by `mis` bytes, the same for all its
// vectors) is read as the two aligned vectors that the elements lie in (the
// second one comes from L1).
template <class T>
__device__ __forceinline__ void beam_load(uint32_t (&w)[4], const T* x, int v, int V, int mis) {
    using E = bm::Elem<T>;
    if (v >= V) {
        w[0] = w[1] = w[2] = w[3] = E::LOWEST;
        return;
    }
    const uint4* a = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(x + v) - mis);
    const uint4 lo = __ldg(a);
    w[0] = lo.x; w[1] = lo.y; w[2] = lo.z; w[3] = lo.w;
    if (mis != 0) {
        // the second vector, unless the row ends in the first
        const int in_first = (16 - mis) / static_cast<int>(sizeof(T));
        const uint4 hi = v + in_first < V ? __ldg(a + 1) : make_uint4(0, 0, 0, 0);
        uint32_t q[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
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
        for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(q[j], q[j + 1], bits);
    }
    if (v + E::VEC > V) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = E::cut(w[j], V - v - j * (E::VEC / 4));
    }
}

// One block per (segment, row).  Thread t holds the vectors i THREADS + t of
// the segment, i < NV.
template <class T>
__global__ void __launch_bounds__(bm::THREADS, 4) beam_chunk_kernel(const BeamParams p) {
    using namespace bm;
    using E = Elem<T>;
    constexpr int VEC = E::VEC;
    __shared__ float s_m[THREADS / 32];
    __shared__ double s_sum[THREADS / 32];
    __shared__ uint64_t s_c[BUF];
    __shared__ int s_n;
    const int tid = threadIdx.x, lane = tid & 31, row = blockIdx.y;
    pdl_launch_dependents();
    {   // a finished beam's logits and those of a dead one are not needed
        const float s = p.scores[row];
        if ((p.finished != nullptr && p.finished[row] != 0) || !isfinite(s)) return;
    }
    if (tid == 0) s_n = 0;
    const T* x = static_cast<const T*>(p.logits) + row * p.ld;
    const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15);
    const int first = static_cast<int>(static_cast<long long>(blockIdx.x) * p.NV * THREADS * VEC);
    auto at = [&](int i, int t) { return first + (i * THREADS + t) * VEC; };   // below 2^25
    auto load = [&](uint32_t (&w)[GROUP][4], int i0) {
        if (mis == 0 && i0 + GROUP <= p.NV && at(i0 + GROUP, 0) <= p.V) {   // uniform: all of it inside
            const uint4* a = reinterpret_cast<const uint4*>(x + at(i0, tid));
#pragma unroll
            for (int i = 0; i < GROUP; ++i) {
                const uint4 q = __ldg(a + i * THREADS);
                w[i][0] = q.x; w[i][1] = q.y; w[i][2] = q.z; w[i][3] = q.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < GROUP; ++i) beam_load<T>(w[i], x, i0 + i < p.NV ? at(i0 + i, tid) : p.V, p.V, mis);
        }
    };

    // ---- maximum and sum of exponentials (a NaN or +inf makes the sum NaN) ----
    uint32_t raw[GROUP][4], next[GROUP][4];
    load(next, 0);
    float m = NEG_INF, ref = NEG_INF;   // maximum; what the sum's terms are relative to
    float sum = 0.f, low = 0.f;         // of exp(x - ref): sum + low
    for (int i0 = 0; i0 < p.NV; i0 += GROUP) {
#pragma unroll
        for (int i = 0; i < GROUP; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) raw[i][j] = next[i][j];
        if (i0 + GROUP < p.NV) load(next, i0 + GROUP);
        uint32_t wm = raw[0][0];
#pragma unroll
        for (int i = 0; i < GROUP; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) wm = E::word_max(wm, raw[i][j]);
        m = fmaxf(m, E::top(wm));
        if (m > ref + FAR) {
            const float f = fast_exp2((ref - m) * LOG2E);
            sum *= f;
            low *= f;
            ref = m;
        }
        const float r = ref > NEG_INF ? ref : 0.f;
        float2 part = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < GROUP; ++i)
#pragma unroll
            for (int q = 0; q < VEC / 2; ++q) {
                const float2 d = mul2(add2(E::pair(raw[i], q), make_float2(-r, -r)), make_float2(LOG2E, LOG2E));
                part = add2(part, make_float2(fast_exp2(d.x), fast_exp2(d.y)));
            }
        // the sum's rounding is kept in `low`: exactly, but where `more` is larger than all
        // before it, which doubles the sum and so happens for 2 2^-24 of it at most.  (A
        // sum in double took longer, on the exponentials' unit, which converts.)
        const float more = part.x + part.y, both = sum + more;
        low += more - (both - sum);
        sum = both;
    }

    // ---- the segment's maximum and sum ----
    float top = m;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (lane == 0) s_m[tid >> 5] = top;
    const float thr = from_key(kth_key(order_key(m), p.K));   // its barriers cover s_m and s_n
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) top = fmaxf(top, s_m[w]);
    double total = static_cast<double>(sum) + low;
    if (ref != top) total *= fast_exp2((ref - top) * LOG2E);   // equal infinities have no difference
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    if (lane == 0) s_sum[tid >> 5] = total;

    // ---- the K best: the warp reads the elements of each thread that reaches
    // the threshold again, a vector a lane ----
    uint32_t pass = __ballot_sync(0xffffffffu, m > NEG_INF && m >= thr);
#pragma unroll 1
    while (pass != 0) {
        // two threads' vectors at a time; which elements pass as bits, so that the
        // code that few elements reach is small (it is fetched when it is needed)
        const int from = tid - lane + __ffs(pass) - 1;
        pass &= pass - 1;
        const int other = pass != 0 ? tid - lane + __ffs(pass) - 1 : -1;
        pass &= pass - 1;
#pragma unroll 1
        for (int i = lane; i < p.NV; i += 32) {
            const int v0 = at(i, from), v1 = other >= 0 ? at(i, other) : p.V;
            uint32_t w[2][4];
            beam_load<T>(w[0], x, v0, p.V, mis);
            beam_load<T>(w[1], x, v1, p.V, mis);
            uint32_t bits = 0;
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                const float2 e = E::pair(w[q / (VEC / 2)], q % (VEC / 2));
                bits |= (e.x >= thr ? 1u : 0u) << 2 * q | (e.y >= thr ? 2u : 0u) << 2 * q;
            }
#pragma unroll 1
            for (; bits != 0; bits &= bits - 1) {
                const int u = __ffs(bits) - 1, v = u < VEC ? v0 + u : v1 + u - VEC;
                // past the row's end (or masked) there is nothing, whatever the threshold
                const float e = v < p.V ? E::one(reinterpret_cast<const uint8_t*>(x + v)) : NEG_INF;
                if (e > NEG_INF) {
                    const int k = atomicAdd(&s_n, 1);
                    if (k < BUF) s_c[k] = pack(e, v);
                }
            }
        }
    }
    __syncthreads();
    const size_t part = static_cast<size_t>(row) * p.S + blockIdx.x;
    if (tid >= THREADS - 32) {   // the last warp, which has no candidate to rank
        total = lane < THREADS / 32 ? s_sum[lane] : 0.0;
#pragma unroll
        for (int d = THREADS / 64; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
        if (lane == 0) p.sums[part] = {total, top};
    }
    uint64_t* out = p.cand + part * p.K;
    const int n = s_n;
    if (n <= BUF) {
        for (int i = tid; i < n; i += THREADS) {
            const uint64_t c = s_c[i];
            const int rank = beam_rank(s_c, n, c);
            if (rank < p.K) out[rank] = c;
        }
        for (int k = n + tid; k < p.K; k += THREADS) out[k] = 0;
        return;
    }
    // ---- more than the buffer holds: one after another ----
    uint64_t last = ~0ull;
    for (int k = 0; k < p.K; ++k) {
        uint64_t best = 0;
        for (int i = 0; i < p.NV; ++i) {
            const int v = at(i, tid);
            uint32_t w[4];
            beam_load<T>(w, x, v, p.V, mis);
#pragma unroll
            for (int q = 0; q < VEC / 2; ++q) {
                const float2 e = E::pair(w, q);
                const uint64_t c0 = pack(e.x, v + 2 * q), c1 = pack(e.y, v + 2 * q + 1);
                if (e.x > NEG_INF && c0 < last && c0 > best) best = c0;
                if (e.y > NEG_INF && c1 < last && c1 > best) best = c1;
            }
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            const uint64_t c = __shfl_xor_sync(0xffffffffu, best, d);
            best = c > best ? c : best;
        }
        __syncthreads();   // the last round's readers are done
        if (lane == 0) s_c[tid >> 5] = best;
        __syncthreads();
        for (int w = 0; w < THREADS / 32; ++w) best = s_c[w] > best ? s_c[w] : best;
        if (tid == 0) out[k] = best;   // more than K elements are above -inf
        last = best;
    }
}

// One block per request.
__global__ void __launch_bounds__(bm::THREADS) beam_merge_kernel(const BeamParams p) {
    using namespace bm;
    __shared__ double s_lse[MAX_K], s_cum[MAX_K];   // per beam
    __shared__ uint8_t s_done[MAX_K];               // 0: a beam that goes on, 1: without candidates, 2: finished
    __shared__ double s_score[MERGE_BUF];
    __shared__ int s_flat[MERGE_BUF], s_n;
    const int tid = threadIdx.x, lane = tid & 31, g = blockIdx.x;
    pdl_wait_primary();
    const int SK = p.S * p.K;
    const int C = p.W * SK;   // candidate c of the request: list (w, s), place k
    // the thread's first candidates, on their way while the sums are joined
    constexpr int EARLY = 4;
    uint64_t early[EARLY];
#pragma unroll
    for (int e = 0; e < EARLY; ++e) {
        const int c = tid + e * THREADS;
        early[e] = c < C ? p.cand[static_cast<size_t>(g) * C + c] : 0;
    }
    if (tid == 0) s_n = 0;
    for (int w = tid >> 5; w < p.W; w += THREADS / 32) {
        const int row = g * p.W + w;
        const Sum* ms = p.sums + static_cast<size_t>(row) * p.S;
        const Sum mine = lane < p.S ? ms[lane] : Sum{0.0, NEG_INF};   // not written for some rows
        const float cum = p.scores[row];
        const bool done = p.finished != nullptr && p.finished[row] != 0;
        double lse = 0;
        if (!done && isfinite(cum)) {
            float m = fmaxf(mine.top, NEG_INF);
            for (int s = lane + 32; s < p.S; s += 32) m = fmaxf(m, ms[s].top);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            double sum = 0;
            for (int s = lane; s < p.S; s += 32) {
                const Sum q = s == lane ? mine : ms[s];
                // a segment without a finite logit adds nothing, unless it holds a NaN
                sum += q.top > NEG_INF ? q.sum * exp(static_cast<double>(q.top) - m) : q.sum != q.sum ? q.sum : 0.0;
            }
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            lse = m + log(sum);
        }
        if (lane == 0) {
            s_lse[w] = lse;
            s_cum[w] = cum;
            s_done[w] = !isfinite(cum) ? 1 : done ? 2 : 0;
        }
    }
    __syncthreads();

    auto score = [&](int c, uint64_t cand, int* flat) -> double {
        const int w = c / SK, q = c - w * SK;
        const int state = s_done[w];
        double key = NEG_INF;
        *flat = w * p.V;
        if (state == 2) {
            if (q == 0) {
                key = s_cum[w];
                *flat += p.pad;
            }
        } else if (state == 0 && cand != 0) {
            key = s_cum[w] + (value_of(cand) - s_lse[w]);
            *flat += static_cast<int>(index_of(cand));
        }
        return key > NEG_INF ? key : static_cast<double>(NEG_INF);   // a NaN has no place
    };
    // f(key, flat) over the thread's candidates
    auto each = [&](auto f) {
#pragma unroll
        for (int e = 0; e < EARLY; ++e) {
            const int c = tid + e * THREADS;
            if (c < C) {
                int flat;
                const double key = score(c, early[e], &flat);
                f(key, flat);
            }
        }
        for (int c = tid + EARLY * THREADS; c < C; c += THREADS) {
            int flat;
            const double key = score(c, p.cand[static_cast<size_t>(g) * C + c], &flat);
            f(key, flat);
        }
    };
    float mine = NEG_INF;
    each([&](double key, int) { mine = fmaxf(mine, static_cast<float>(key)); });
    // scores rounded to 32 bits keep their order up to ties, so the threshold
    // on them lets every candidate of the K best through
    const float thr = from_key(kth_key(order_key(mine), p.K));
    if (mine >= thr)
        each([&](double key, int flat) {
            if (static_cast<float>(key) >= thr && key > NEG_INF) {
                const int k = atomicAdd(&s_n, 1);
                if (k < MERGE_BUF) {
                    s_score[k] = key;
                    s_flat[k] = flat;
                }
            }
        });
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
#pragma unroll 2
            for (int j = 0; j < n; ++j) {
                const double other = s_score[j];
                rank += (other > key) | ((other == key) & (s_flat[j] < flat));
            }
            if (rank < p.K) put(rank, key, flat);
        }
        for (int k = n + tid; k < p.K; k += THREADS) put(k, NEG_INF, 0);
    } else {
        double last = __builtin_huge_val();
        int last_f = -1;
        for (int k = 0; k < p.K; ++k) {
            double bk = NEG_INF;
            int bf = 0x7fffffff;
            each([&](double key, int flat) {
                const bool behind = key < last || (key == last && flat > last_f);
                if (behind && key > NEG_INF && (key > bk || (key == bk && flat < bf))) {
                    bk = key;
                    bf = flat;
                }
            });
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
