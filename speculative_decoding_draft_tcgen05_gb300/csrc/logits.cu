// The target's logits under penalties for repeated tokens, biases and a mask;
// from them softmax, the best token, or the logits.
//
// A cluster of C CTAs takes some positions of one sequence; each CTA has a
// slice of the vocabulary. What depends on the sequence alone is laid out once
// in shared memory, a word per token of the slice: how often it has occurred,
// and its place in the list of biases. Then one pass over the slice per
// position finds the best token and, relative to the running maximum, the sum
// of the exponentials; the CTAs exchange those through distributed shared
// memory, and a second pass, whose logits come from L2, writes the
// probabilities. So HBM sees the logits once and the outputs once, which is
// what bounds a large batch; a small one is bound by the chain history ->
// table -> logits -> exchange.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdio.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "dflash_logits.h"
#include "kernels.h"

namespace dfl {

dflash_status host_fail(dflash_status st, const char *msg);

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 8;                  // tokens of a lane in a step
constexpr int kStep = kThreads * kPer;   // tokens of a CTA in a step
constexpr int kMaxCluster = 16;
constexpr uint32_t kInPrompt = 0x80000000u;

struct LogitsParams {
    const void *logits;
    void *out;
    float *probs;
    int32_t *argmax;
    int64_t seq_stride, row_stride, out_seq_stride, out_row_stride;
    int64_t vocab;
    int batch, rows, group, groups;  // positions of a cluster, clusters of a sequence
    int slice;                       // tokens of a CTA, a multiple of 256
    int C;
    dflash_logits_rules r;
    const int32_t *draft;
    int64_t draft_stride;
    const int32_t *mask;
    int64_t mask_seq_stride, mask_row_stride;
    int counted, biased;             // there are tokens (or drafts) that penalties count; there are biases
};

struct Best {
    float m, s;   // maximum and sum of exp((x - m) / tau)
    float v;      // the largest x that is a number, and the lowest token that has it
    int id;
};

template <typename T>
__device__ __forceinline__ float to_f(T v)
{
    if constexpr (std::is_same_v<T, float>) return v;
    else if constexpr (std::is_same_v<T, __half>) return __half2float(v);
    else return __bfloat162float(v);
}

template <typename T>
__device__ __forceinline__ T from_f(float v)
{
    if constexpr (std::is_same_v<T, float>) return v;
    else if constexpr (std::is_same_v<T, __half>) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

template <typename T>
struct alignas(16) Vec {
    T v[16 / sizeof(T)];
};

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// (m, s) of two parts; scale = log2(e) / tau
__device__ __forceinline__ void join(float &m, float &s, float m2, float s2, float scale)
{
    const float top = fmaxf(m, m2);
    if (top == -INFINITY) {  // (a NaN in s or s2 stays: m is then not its maximum)
        s += s2;
        return;
    }
    s = (m == top ? s : s * exp2_fast((m - top) * scale)) + (m2 == top ? s2 : s2 * exp2_fast((m2 - top) * scale));
    m = top;
}

__device__ __forceinline__ void join_best(float &v, int &id, float v2, int id2)
{
    if (v2 > v || (v2 == v && id2 < id)) {
        v = v2;
        id = id2;
    }
}

template <typename T, bool kVec>
struct Slice {
    const LogitsParams &p;
    const uint32_t *counts, *bias;   // shared memory (or unused)
    int64_t v0, v1;                  // the CTA's tokens
    float rho, alpha, beta;
    const float *bias_values;        // the sequence's

    // Token j of this lane's step at `at` (the warp's first token).
    __device__ __forceinline__ int64_t token(int64_t at, int lane, int j) const
    {
        return kVec ? at + lane * kPer + j : at + j * 32 + lane;
    }

    __device__ __forceinline__ void load(const T *row, int64_t at, int lane, float (&x)[kPer]) const
    {
        if constexpr (kVec) {
            const int64_t t = at + lane * kPer;
            if (t < v1) {  // (v1 is a multiple of 8 where rows are)
                constexpr int N = 16 / sizeof(T);
#pragma unroll
                for (int i = 0; i < kPer / N; ++i) {
                    const Vec<T> q = *reinterpret_cast<const Vec<T> *>(row + t + i * N);
#pragma unroll
                    for (int j = 0; j < N; ++j) x[i * N + j] = to_f(q.v[j]);
                }
                return;
            }
#pragma unroll
            for (int j = 0; j < kPer; ++j) x[j] = -INFINITY;
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int64_t t = at + j * 32 + lane;
                x[j] = t < v1 ? to_f(row[t]) : -INFINITY;
            }
        }
    }

    // The rules on one value of a token that has occurred.
    __device__ __forceinline__ float repeated(float x, uint32_t word) const
    {
        x = x > 0.f ? __fdiv_rn(x, rho) : __fmul_rn(x, rho);
        const uint32_t c = word & ~kInPrompt;
        if (c) x = __fsub_rn(__fsub_rn(x, __fmul_rn(beta, static_cast<float>(c))), alpha);
        return x;
    }

    __device__ __forceinline__ void adjust(const int32_t *mask, int64_t at, int lane, float (&x)[kPer]) const
    {
        const int local = static_cast<int>(at - v0);
        if (counts) {
            uint32_t w[kPer], any = 0;
            if constexpr (kVec) {
                const uint4 a = *reinterpret_cast<const uint4 *>(counts + local + lane * kPer);
                const uint4 b = *reinterpret_cast<const uint4 *>(counts + local + lane * kPer + 4);
                w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
            } else {
#pragma unroll
                for (int j = 0; j < kPer; ++j) w[j] = counts[local + j * 32 + lane];
            }
#pragma unroll
            for (int j = 0; j < kPer; ++j) any |= w[j];
            if (any) {
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (w[j]) x[j] = repeated(x[j], w[j]);
            }
        }
        if (bias) {
            uint32_t w[kPer], any = 0;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                w[j] = bias[kVec ? local + lane * kPer + j : local + j * 32 + lane];
                any |= w[j];
            }
            if (any) {
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (w[j]) x[j] = __fadd_rn(x[j], bias_values[w[j] - 1]);
            }
        }
        if (mask) {
            if constexpr (kVec) {
                const int64_t t = at + lane * kPer;
                const uint32_t bits = t < v1 ? static_cast<uint32_t>(mask[t >> 5]) >> (t & 31) : 0u;
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (!((bits >> j) & 1u)) x[j] = -INFINITY;
            } else {
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const int64_t t = at + j * 32;  // (a multiple of 32: one word for the warp)
                    const uint32_t bits = t < v1 ? static_cast<uint32_t>(mask[t >> 5]) : 0u;
                    if (!((bits >> lane) & 1u)) x[j] = -INFINITY;
                }
            }
        }
    }
};

struct Shared {
    Best warp[kWarps];
    Best peer[2][kMaxCluster];
    Best all;
};

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads) logits_kernel(const __grid_constant__ LogitsParams p)
{
    extern __shared__ uint4 smem[];
    __shared__ Shared s;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = p.C;
    const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int b = static_cast<int>(blockIdx.x) / p.groups, g = static_cast<int>(blockIdx.x) % p.groups;
    const int t0 = g * p.group, t1 = min(p.rows, t0 + p.group);
    uint32_t *const counts = reinterpret_cast<uint32_t *>(smem);
    uint32_t *const bias = counts + (p.counted ? p.slice : 0);

    Slice<T, kVec> sl = {p, p.counted ? counts : nullptr, p.biased ? bias : nullptr, 0, 0, 1.f, 0.f, 0.f, nullptr};
    sl.v0 = min(static_cast<int64_t>(rank) * p.slice, p.vocab);
    sl.v1 = min(sl.v0 + p.slice, p.vocab);
    const int width = static_cast<int>(sl.v1 - sl.v0);
    if (p.r.repetition) sl.rho = p.r.repetition[b];
    if (p.r.presence) sl.alpha = p.r.presence[b];
    if (p.r.frequency) sl.beta = p.r.frequency[b];
    const float tau = p.r.temperature ? p.r.temperature[b] : 1.f;

    // what has occurred, and the biases' places
    const int words = ((p.counted ? p.slice : 0) + (p.biased ? p.slice : 0)) / 4;
    for (int i = tid; i < words; i += kThreads) smem[i] = make_uint4(0, 0, 0, 0);
    if (words) __syncthreads();
    auto place = [&](int32_t token) {  // the slice's index of a token, or -1
        const int64_t at = static_cast<int64_t>(token) - sl.v0;
        return at >= 0 && at < width ? static_cast<int>(at) : -1;
    };
    const int32_t *const draft = p.draft ? p.draft + b * p.draft_stride : nullptr;
    if (p.counted) {
        if (p.r.tokens) {
            const int32_t *const tokens = p.r.tokens + b * p.r.token_stride;
            const int len = min(max(p.r.lens[b], 0), p.r.token_cols);
            const int prompt = p.r.prompt_lens ? p.r.prompt_lens[b] : 0;
            for (int i0 = tid; i0 < len; i0 += 4 * kThreads) {
                int32_t w[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) w[u] = i0 + u * kThreads < len ? tokens[i0 + u * kThreads] : -1;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int at = place(w[u]);
                    if (at < 0) continue;
                    if (i0 + u * kThreads < prompt)
                        atomicOr(counts + at, kInPrompt);
                    else
                        atomicAdd(counts + at, 1u);
                }
            }
        }
        if (draft && tid < t0) {
            for (int i = tid; i < t0; i += kThreads) {
                const int at = place(draft[i]);
                if (at >= 0) atomicAdd(counts + at, 1u);
            }
        }
    }
    if (p.biased) {
        const int32_t *const ids = p.r.bias_ids + b * p.r.bias_stride;
        sl.bias_values = p.r.bias_values + b * p.r.bias_stride;
        for (int i = tid; i < p.r.bias_count; i += kThreads) {
            const int at = place(ids[i]);
            if (at >= 0) atomicMax(bias + at, static_cast<uint32_t>(i) + 1u);  // the last one counts
        }
    }
    __syncthreads();

    const bool greedy = tau == 0.f;
    float scale = greedy ? 1.f : 1.4426950408889634f / tau;
    if (scale == INFINITY) scale = 3.4028235e38f;  // (so that the best token's 0 * scale stays 0,
    if (scale == 0.f) scale = 1.1754944e-38f;      // and a masked token's -inf * scale -inf)
    const bool want_sum = p.probs && !greedy, want_best = p.argmax || (p.probs && greedy);
    for (int t = t0; t < t1; ++t) {
        const int64_t at_row = static_cast<int64_t>(b) * p.rows + t;
        const T *const row = static_cast<const T *>(p.logits) + b * p.seq_stride + t * p.row_stride;
        const int32_t *const mask = p.mask ? p.mask + b * p.mask_seq_stride + t * p.mask_row_stride : nullptr;
        T *const out = p.out ? static_cast<T *>(p.out) + b * p.out_seq_stride + t * p.out_row_stride : nullptr;
        // (a row that is written in place is written by the pass that reads it last)
        const bool out_now = out && !p.probs;

        float m = -INFINITY, sum = 0.f, best = -INFINITY;
        int best_id = 0x7FFFFFFF;
        for (int64_t at = sl.v0 + warp * (32 * kPer); at < sl.v1; at += kStep) {
            float x[kPer];
            sl.load(row, at, lane, x);
            sl.adjust(mask, at, lane, x);
            if (want_sum || want_best) {
                float top = x[0];
#pragma unroll
                for (int j = 1; j < kPer; ++j) top = fmaxf(top, x[j]);
                if (want_best && top > best) {
                    best = top;
#pragma unroll
                    for (int j = kPer - 1; j >= 0; --j)
                        if (x[j] == top) best_id = static_cast<int>(sl.token(at, lane, j));
                }
                if (want_sum) {
                    if (top > m) {
                        if (m > -INFINITY) sum *= exp2_fast((m - top) * scale);
                        m = top;
                    }
                    const float base = m == -INFINITY ? 0.f : m;  // (nothing yet: exp of -inf, or NaN)
#pragma unroll
                    for (int j = 0; j < kPer; ++j) sum += exp2_fast((x[j] - base) * scale);
                }
            }
            if (out_now) {
                if constexpr (kVec) {
                    const int64_t v = at + lane * kPer;
                    constexpr int N = 16 / sizeof(T);
                    if (v < sl.v1) {
#pragma unroll
                        for (int i = 0; i < kPer / N; ++i) {
                            Vec<T> q;
#pragma unroll
                            for (int j = 0; j < N; ++j) q.v[j] = from_f<T>(x[i * N + j]);
                            *reinterpret_cast<Vec<T> *>(out + v + i * N) = q;
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < kPer; ++j) {
                        const int64_t v = sl.token(at, lane, j);
                        if (v < sl.v1) out[v] = from_f<T>(x[j]);
                    }
                }
            }
        }
        if (want_sum || want_best) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                join(m, sum, __shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, sum, o), scale);
                join_best(best, best_id, __shfl_xor_sync(0xFFFFFFFFu, best, o), __shfl_xor_sync(0xFFFFFFFFu, best_id, o));
            }
            if (lane == 0) s.warp[warp] = {m, sum, best, best_id};
            __syncthreads();
            if (warp == 0) {
                Best q = {-INFINITY, 0.f, -INFINITY, 0x7FFFFFFF};
                if (lane < kWarps) q = s.warp[lane];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    join(q.m, q.s, __shfl_xor_sync(0xFFFFFFFFu, q.m, o), __shfl_xor_sync(0xFFFFFFFFu, q.s, o), scale);
                    join_best(q.v, q.id, __shfl_xor_sync(0xFFFFFFFFu, q.v, o), __shfl_xor_sync(0xFFFFFFFFu, q.id, o));
                }
                if (C > 1) {
                    if (lane < C) {
                        const uint32_t to = mapa_shared(smem_u32(&s.peer[t & 1][rank]), static_cast<uint32_t>(lane));
                        asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(__float_as_uint(q.m)),
                                     "r"(__float_as_uint(q.s)), "r"(__float_as_uint(q.v)), "r"(q.id)
                                     : "memory");
                    }
                } else if (lane == 0) {
                    s.all = q;
                }
                __syncwarp();
            }
            Best q;
            if (C > 1) {
                // (the next position writes the other half: a CTA that reads this one has not passed that exchange)
                cluster_sync_all();
                q = {-INFINITY, 0.f, -INFINITY, 0x7FFFFFFF};
                if (lane < C) q = s.peer[t & 1][lane];
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) {
                    join(q.m, q.s, __shfl_xor_sync(0xFFFFFFFFu, q.m, o), __shfl_xor_sync(0xFFFFFFFFu, q.s, o), scale);
                    join_best(q.v, q.id, __shfl_xor_sync(0xFFFFFFFFu, q.v, o), __shfl_xor_sync(0xFFFFFFFFu, q.id, o));
                }
                q.m = __shfl_sync(0xFFFFFFFFu, q.m, 0);
                q.s = __shfl_sync(0xFFFFFFFFu, q.s, 0);
                q.id = __shfl_sync(0xFFFFFFFFu, q.id, 0);
            } else {
                __syncthreads();
                q = s.all;
            }
            const int id = q.id == 0x7FFFFFFF ? -1 : q.id;
            if (p.argmax && rank == 0 && tid == 0) p.argmax[at_row] = id;
            if (p.probs) {
                float *const probs = p.probs + at_row * p.vocab;
                const float base = q.m == -INFINITY ? 0.f : q.m;
                const float inv = q.m == -INFINITY && q.s == 0.f ? 0.f : 1.f / q.s;
                for (int64_t at = sl.v0 + warp * (32 * kPer); at < sl.v1; at += kStep) {
                    float x[kPer], y[kPer];
                    sl.load(row, at, lane, x);
                    sl.adjust(mask, at, lane, x);
#pragma unroll
                    for (int j = 0; j < kPer; ++j)
                        y[j] = greedy ? (static_cast<int>(sl.token(at, lane, j)) == id ? 1.f : 0.f)
                                      : exp2_fast((x[j] - base) * scale) * inv;
                    if constexpr (kVec) {
                        const int64_t v = at + lane * kPer;
                        if (v < sl.v1) {
                            *reinterpret_cast<float4 *>(probs + v) = make_float4(y[0], y[1], y[2], y[3]);
                            *reinterpret_cast<float4 *>(probs + v + 4) = make_float4(y[4], y[5], y[6], y[7]);
                            if (out) {
                                constexpr int N = 16 / sizeof(T);
#pragma unroll
                                for (int i = 0; i < kPer / N; ++i) {
                                    Vec<T> o;
#pragma unroll
                                    for (int j = 0; j < N; ++j) o.v[j] = from_f<T>(x[i * N + j]);
                                    *reinterpret_cast<Vec<T> *>(out + v + i * N) = o;
                                }
                            }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < kPer; ++j) {
                            const int64_t v = sl.token(at, lane, j);
                            if (v < sl.v1) {
                                probs[v] = y[j];
                                if (out) out[v] = from_f<T>(x[j]);
                            }
                        }
                    }
                }
            }
        }
        if (p.counted && draft && t + 1 < t1) {  // the next position follows one more draft
            __syncthreads();
            if (tid == 0) {
                const int at = place(draft[t]);
                if (at >= 0) ++counts[at];
            }
            __syncthreads();
        }
    }
    if (C > 1) cluster_sync_all();  // no CTA ends while another still writes to it
}

dflash_status logits_fail(dflash_status st, const char *fmt, long long a = 0, long long b = 0)
{
    char buf[256];
    snprintf(buf, sizeof buf, fmt, a, b);
    return host_fail(st, buf);
}

bool misaligned(const void *p, uintptr_t by)
{
    return reinterpret_cast<uintptr_t>(p) % by != 0;
}

using Kernel = void (*)(LogitsParams);

Kernel kernel_of(int dtype, bool vec)
{
    if (dtype == DFLASH_BF16) return vec ? logits_kernel<__nv_bfloat16, true> : logits_kernel<__nv_bfloat16, false>;
    if (dtype == DFLASH_FP16) return vec ? logits_kernel<__half, true> : logits_kernel<__half, false>;
    return vec ? logits_kernel<float, true> : logits_kernel<float, false>;
}

// Per device, once: SMs and the shared memory of a block, and the kernels' opt-ins to it and to clusters of 16.
cudaError_t machine(int *sms, int *smem)
{
    static std::atomic<int> sms_of[64], smem_of[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (*sms = sms_of[dev].load(std::memory_order_acquire)) != 0) {
        *smem = smem_of[dev].load(std::memory_order_relaxed);
        return cudaSuccess;
    }
    int optin = 0;
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    *smem = optin - static_cast<int>(sizeof(Shared)) - 1024;
    for (int dtype : {static_cast<int>(DFLASH_BF16), static_cast<int>(DFLASH_FP16), static_cast<int>(DFLASH_FP32)})
        for (int vec = 0; vec < 2 && e == cudaSuccess; ++vec) {
            e = cudaFuncSetAttribute(kernel_of(dtype, vec != 0), cudaFuncAttributeMaxDynamicSharedMemorySize, *smem);
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(kernel_of(dtype, vec != 0), cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        }
    if (e != cudaSuccess) return e;
    if (dev < 64) {
        smem_of[dev].store(*smem, std::memory_order_relaxed);
        sms_of[dev].store(*sms, std::memory_order_release);
    }
    return cudaSuccess;
}

}  // namespace
}  // namespace dfl

using dfl::logits_fail;

extern "C" dflash_status dflash_logits_adjust(const void *logits, int64_t seq_stride, int64_t row_stride, int32_t batch,
                                              int32_t rows, int64_t vocab, int32_t dtype, const dflash_logits_rules *rules,
                                              const int32_t *draft, int64_t draft_stride, const int32_t *mask,
                                              int64_t mask_seq_stride, int64_t mask_row_stride, void *out,
                                              int64_t out_seq_stride, int64_t out_row_stride, float *probs, int32_t *argmax,
                                              void *stream)
{
    if (dtype != DFLASH_BF16 && dtype != DFLASH_FP16 && dtype != DFLASH_FP32)
        return logits_fail(DFLASH_ERR_UNSUPPORTED, "dtype must be BF16, FP16 or FP32 (got %lld)", dtype);
    if (batch < 0 || rows < 0 || static_cast<int64_t>(batch) * rows >= (int64_t(1) << 31))
        return logits_fail(DFLASH_ERR_INVALID_ARG, "batch and rows must be >= 0, their product below 2^31 (got %lld, %lld)", batch, rows);
    if (vocab < 1 || vocab >= (int64_t(1) << 31)) return logits_fail(DFLASH_ERR_INVALID_ARG, "vocab must be in [1, 2^31) (got %lld)", vocab);
    if (batch == 0 || rows == 0) return DFLASH_OK;
    if (!out && !probs && !argmax) return logits_fail(DFLASH_ERR_INVALID_ARG, "one of out, probs and argmax must be given");
    const int size = dtype == DFLASH_FP32 ? 4 : 2;
    if (!logits || dfl::misaligned(logits, size) || dfl::misaligned(out, size) || dfl::misaligned(probs, 4) ||
        dfl::misaligned(argmax, 4) || dfl::misaligned(draft, 4) || dfl::misaligned(mask, 4))
        return logits_fail(DFLASH_ERR_INVALID_ARG, "logits must be given, and all tensors aligned to their type");
    if (batch == 1) seq_stride = out_seq_stride = mask_seq_stride = draft_stride = 0;
    if (rows == 1) row_stride = out_row_stride = mask_row_stride = 0;
    if (seq_stride < 0 || row_stride < 0 || mask_seq_stride < 0 || mask_row_stride < 0 || draft_stride < 0 ||
        (out && ((batch > 1 && out_seq_stride < vocab) || (rows > 1 && out_row_stride < vocab))))
        return logits_fail(DFLASH_ERR_INVALID_ARG, "strides must not be negative, those of out at least vocab");
    if (out == logits && (seq_stride != out_seq_stride || row_stride != out_row_stride))
        return logits_fail(DFLASH_ERR_INVALID_ARG, "out can be the logits only with their strides");
    static const dflash_logits_rules none = {};
    dfl::LogitsParams p = {};
    p.r = rules ? *rules : none;
    if (p.r.tokens && (!p.r.lens || p.r.token_cols < 0 || p.r.token_stride < 0 || (batch > 1 && p.r.token_stride < p.r.token_cols)))
        return logits_fail(DFLASH_ERR_INVALID_ARG, "tokens need lens, token_cols >= 0 and a stride of at least that (got %lld, %lld)",
                           p.r.token_cols, p.r.token_stride);
    if (p.r.bias_count < 0 || (p.r.bias_count > 0 && (!p.r.bias_ids || !p.r.bias_values)) ||
        (p.r.bias_count > 0 && batch > 1 && p.r.bias_stride < p.r.bias_count))
        return logits_fail(DFLASH_ERR_INVALID_ARG, "biases need ids, values, a count >= 0 and a stride of at least that (got %lld, %lld)",
                           p.r.bias_count, p.r.bias_stride);
    for (const void *q : {static_cast<const void *>(p.r.tokens), static_cast<const void *>(p.r.lens),
                          static_cast<const void *>(p.r.prompt_lens), static_cast<const void *>(p.r.repetition),
                          static_cast<const void *>(p.r.presence), static_cast<const void *>(p.r.frequency),
                          static_cast<const void *>(p.r.temperature), static_cast<const void *>(p.r.bias_ids),
                          static_cast<const void *>(p.r.bias_values)})
        if (dfl::misaligned(q, 4)) return logits_fail(DFLASH_ERR_INVALID_ARG, "the rules' arrays must be aligned to their type");
    int sms = 0, smem_most = 0;
    cudaError_t e = dfl::machine(&sms, &smem_most);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return logits_fail(DFLASH_ERR_CUDA, "setting up the current device failed (error %lld)", e);
    }

    p.logits = logits;
    p.out = out;
    p.probs = probs;
    p.argmax = argmax;
    p.seq_stride = seq_stride;
    p.row_stride = row_stride;
    p.out_seq_stride = out_seq_stride;
    p.out_row_stride = out_row_stride;
    p.vocab = vocab;
    p.batch = batch;
    p.rows = rows;
    p.draft = rows > 1 ? draft : nullptr;
    p.draft_stride = draft_stride;
    p.mask = mask;
    p.mask_seq_stride = mask_seq_stride;
    p.mask_row_stride = mask_row_stride;
    p.counted = (p.r.repetition || p.r.presence || p.r.frequency) && (p.r.tokens || p.draft);
    p.biased = p.r.bias_count > 0;
    const int word = 4 * (p.counted + p.biased);
    // CTAs per cluster: enough that the tables leave room for two CTAs an SM and, with few positions, that all SMs
    // have work of at least a step
    const int64_t positions = static_cast<int64_t>(batch) * rows;
    auto slice_of = [&](int C) { return ((vocab + C - 1) / C + 255) / 256 * 256; };
    int C = 1;
    while (C < dfl::kMaxCluster && (slice_of(C) * word > 100 * 1024 || (positions * C < 2 * sms && slice_of(C) > dfl::kStep))) C *= 2;
    const int64_t slice = slice_of(C);
    if (slice * word > smem_most)
        return logits_fail(DFLASH_ERR_UNSUPPORTED, "a vocabulary of %lld with tokens or biases needs more shared memory than there is (%lld bytes a CTA)",
                           vocab, smem_most);
    // positions per cluster: as many as leave a few waves, since a sequence's tokens are laid out once for them
    int group = 1;
    if (p.counted || p.biased)
        while (group < rows && (positions / (2 * group)) * C >= 8 * sms) group *= 2;
    p.group = group < rows ? group : rows;
    p.groups = (rows + p.group - 1) / p.group;
    p.slice = static_cast<int>(slice);
    p.C = C;
    const int per = 16 / size;
    const bool vec = !dfl::misaligned(logits, 16) && seq_stride % per == 0 && row_stride % per == 0 && vocab % 8 == 0 &&
                     (!out || (!dfl::misaligned(out, 16) && out_seq_stride % per == 0 && out_row_stride % per == 0)) &&
                     !dfl::misaligned(probs, 16);
    const int64_t clusters = static_cast<int64_t>(batch) * p.groups;
    if (clusters >= (int64_t(1) << 31)) return logits_fail(DFLASH_ERR_INVALID_ARG, "too many positions");
    e = dfl::launch_ex(dfl::kernel_of(dtype, vec), dim3(static_cast<unsigned>(clusters), 1, C), dim3(dfl::kThreads),
                       static_cast<size_t>(slice) * word, static_cast<cudaStream_t>(stream), C, p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return logits_fail(DFLASH_ERR_CUDA, "the launch failed (error %lld)", e);
    }
    return DFLASH_OK;
}
