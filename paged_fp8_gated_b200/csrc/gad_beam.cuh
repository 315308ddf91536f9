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
// suffices: each block takes a chunk of a row into registers, and leaves its
// K best logits, its maximum m and sum of exp(x - m) (beam_chunk_kernel); a
// second kernel joins the chunks' sums into lse_w and ranks the W S K
// candidates (beam_merge_kernel).  The scores that decide the order are held
// in 64 bits: candidates of different beams can be as close as the last bits
// of lse_w.  A chunk's elements go to threads by their index, whatever the
// row's alignment, so equal rows have equal sums and tie exactly.
//
// Finding the K best of a chunk: the K-th largest of at least K group maxima
// is a lower bound of the K-th largest element, few elements reach it, and
// those are ranked by counting.  If more than the buffer holds reach it (long
// ties), the block takes the K best one after another.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gad_ptx.cuh"

namespace gad {
namespace bm {

constexpr int THREADS = 256;
constexpr int MAX_K = 64;
constexpr int BUF = 1024;       // candidates that are ranked by counting
constexpr float NEG_INF = -__builtin_huge_valf();

template <class T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int VEC = 4;
    __device__ static float get(const uint32_t (&w)[4], int i) { return __uint_as_float(w[i]); }
    __device__ static float one(const void* p, size_t i) { return static_cast<const float*>(p)[i]; }
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int VEC = 8;
    __device__ static float get(const uint32_t (&w)[4], int i) {
        return __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
    }
    __device__ static float one(const void* p, size_t i) {
        return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    }
};
template <>
struct Elem<__half> {
    static constexpr int VEC = 8;
    __device__ static float get(const uint32_t (&w)[4], int i) {
        const uint16_t h = static_cast<uint16_t>((i & 1) ? (w[i >> 1] >> 16) : (w[i >> 1] & 0xffffu));
        return __half2float(__ushort_as_half(h));
    }
    __device__ static float one(const void* p, size_t i) { return __half2float(static_cast<const __half*>(p)[i]); }
};

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

__device__ __forceinline__ float block_max(float v, float* s) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    float m = s[0];
#pragma unroll
    for (int w = 1; w < THREADS / 32; ++w) m = fmaxf(m, s[w]);
    return m;
}

}  // namespace bm

struct BeamParams {
    const void* logits;
    long long ld;             // elements from one row of logits to the next
    const float* scores;      // [G W]
    const uint8_t* finished;  // [G W] or null
    int G, W, V, K, S;        // S chunks per row
    int pad;
    float* cand_x;            // [G W S K] the chunks' best logits, best first (-inf: none)
    int* cand_v;              // [G W S K] their tokens
    float2* sums;             // [G W S] maximum, sum of exp(x - maximum)
    float* out_scores;
    int *out_parent, *out_token;
};

// One block per (chunk of E THREADS logits, row).
template <class T, int E>
__global__ void __launch_bounds__(bm::THREADS) beam_chunk_kernel(const BeamParams p) {
    using namespace bm;
    constexpr int VEC = Elem<T>::VEC, NV = E / VEC;
    static_assert(E % VEC == 0, "whole vectors");
    __shared__ float s_red[THREADS / 32], s_thr;
    __shared__ double s_sum[THREADS / 32];
    __shared__ uint32_t s_key[128];
    __shared__ float s_x[BUF];
    __shared__ int s_v[BUF], s_n;
    const int tid = threadIdx.x, row = blockIdx.y;
    pdl_launch_dependents();
    {   // a finished beam's logits and those of a dead one are not needed
        const float s = p.scores[row];
        if ((p.finished != nullptr && p.finished[row] != 0) || !(s > NEG_INF)) return;
    }
    if (tid == 0) s_n = 0;
    const T* x = static_cast<const T*>(p.logits) + row * p.ld;
    const int v0 = blockIdx.x * (E * THREADS);

    // ---- the chunk into registers: thread t holds elements (i THREADS + t) VEC + u.
    // A row that starts off a 16-byte boundary is read as the two aligned
    // vectors that an element vector lies in (the second one comes from L1).
    uint32_t raw[NV][4];
    const uintptr_t addr = reinterpret_cast<uintptr_t>(x + v0);
    const int mis = static_cast<int>(addr & 15);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = v0 + (i * THREADS + tid) * VEC;
        if (v + VEC <= p.V) {
            const uint4* a = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(x + v) - mis);
            const uint4 lo = __ldg(a);
            raw[i][0] = lo.x; raw[i][1] = lo.y; raw[i][2] = lo.z; raw[i][3] = lo.w;
            if (mis != 0) {
                const uint4 hi = __ldg(a + 1);
                uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                if (mis & 8) {
#pragma unroll
                    for (int j = 0; j < 6; ++j) w[j] = w[j + 2];
                }
                if (mis & 4) {
#pragma unroll
                    for (int j = 0; j < 5; ++j) w[j] = w[j + 1];
                }
                const int bits = 8 * (mis & 3);
#pragma unroll
                for (int j = 0; j < 4; ++j) raw[i][j] = __funnelshift_r(w[j], w[j + 1], bits);
            }
        }
    }
    auto value = [&](int i, int u) -> float { return Elem<T>::get(raw[i], u); };
    float tail[VEC];   // the vector that the row's end lies in
    int tail_i = -1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = v0 + (i * THREADS + tid) * VEC;
        if (v < p.V && v + VEC > p.V) tail_i = i;
    }
#pragma unroll
    for (int u = 0; u < VEC; ++u) {
        const int v = v0 + (tail_i * THREADS + tid) * VEC + u;
        tail[u] = tail_i >= 0 && v < p.V ? Elem<T>::one(x, v) : NEG_INF;
    }
    // f(x, v) over the thread's elements in order
    auto each = [&](auto f) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = v0 + (i * THREADS + tid) * VEC;
            if (v + VEC <= p.V) {
#pragma unroll
                for (int u = 0; u < VEC; ++u) f(value(i, u), v + u);
            }
        }
        if (tail_i >= 0) {
            const int v = v0 + (tail_i * THREADS + tid) * VEC;
#pragma unroll
            for (int u = 0; u < VEC; ++u) f(tail[u], v + u);
        }
    };

    // ---- maximum and sum of exponentials (a NaN or +inf makes the sum NaN) ----
    float mine = NEG_INF;
    each([&](float e, int) { mine = fmaxf(mine, e); });
    const float m = block_max(mine, s_red);
    float sum = 0.f;
    const float ref = m > NEG_INF ? m : 0.f;
    each([&](float e, int) { sum += fast_exp2((e - ref) * 1.4426950408889634f); });
    double total = sum;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    if ((tid & 31) == 0) s_sum[tid >> 5] = total;

    // ---- the K best logits ----
    const float thr = group_threshold(mine, p.K, s_key, &s_thr);   // its barriers cover s_sum and s_n
    if (mine >= thr)
        each([&](float e, int v) {
            if (e >= thr && e > NEG_INF) {
                const int k = atomicAdd(&s_n, 1);
                if (k < BUF) {
                    s_x[k] = e;
                    s_v[k] = v;
                }
            }
        });
    __syncthreads();
    const size_t part = static_cast<size_t>(row) * p.S + blockIdx.x;
    float* out_x = p.cand_x + part * p.K;
    int* out_v = p.cand_v + part * p.K;
    const int n = s_n;
    if (tid == 0) {
        double all = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) all += s_sum[w];
        p.sums[part] = make_float2(m, static_cast<float>(all));
    }
    if (n <= BUF) {
        for (int i = tid; i < n; i += THREADS) {
            const float e = s_x[i];
            const int v = s_v[i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += s_x[j] > e || (s_x[j] == e && s_v[j] < v);
            if (rank < p.K) {
                out_x[rank] = e;
                out_v[rank] = v;
            }
        }
        for (int k = n + tid; k < p.K; k += THREADS) {
            out_x[k] = NEG_INF;
            out_v[k] = -1;
        }
    } else {
        // one after another: the best element behind the last one taken
        float last_x = __builtin_huge_valf();
        int last_v = -1;
        for (int k = 0; k < p.K; ++k) {
            float bx = NEG_INF;
            int bv = 0x7fffffff;
            each([&](float e, int v) {
                const bool behind = e < last_x || (e == last_x && v > last_v);
                if (behind && e > NEG_INF && (e > bx || (e == bx && v < bv))) {
                    bx = e;
                    bv = v;
                }
            });
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
            if ((tid & 31) == 0) {
                s_x[tid >> 5] = bx;
                s_v[tid >> 5] = bv;
            }
            __syncthreads();
            bx = s_x[0];
            bv = s_v[0];
            for (int w = 1; w < THREADS / 32; ++w)
                if (s_x[w] > bx || (s_x[w] == bx && s_v[w] < bv)) {
                    bx = s_x[w];
                    bv = s_v[w];
                }
            if (tid == 0) {
                out_x[k] = bx;
                out_v[k] = bx > NEG_INF ? bv : -1;
            }
            last_x = bx;
            last_v = bv;
        }
    }
}

// One block per request.
__global__ void __launch_bounds__(bm::THREADS) beam_merge_kernel(const BeamParams p) {
    using namespace bm;
    __shared__ double s_lse[MAX_K], s_cum[MAX_K];   // per beam; a beam without candidates has lse NaN
    __shared__ uint8_t s_done[MAX_K];
    __shared__ uint32_t s_key[128];
    __shared__ float s_thr;
    __shared__ double s_score[BUF];
    __shared__ int s_flat[BUF], s_n;
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
                // a chunk without a finite logit adds nothing, unless it holds a NaN
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
                if (k < BUF) {
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
    if (n <= BUF) {
        for (int i = tid; i < n; i += THREADS) {
            const double key = s_score[i];
            const int flat = s_flat[i];
            int rank = 0;
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
