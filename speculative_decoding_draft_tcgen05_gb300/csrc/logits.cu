// The target's logits under penalties for repeated tokens, biases and a mask;
// from them softmax, the best token, or the logits.
//
// A cluster of C CTAs takes some positions of one sequence; its CTAs take turns
// at pieces of 2048 tokens, so that the frequent ones, which vocabularies have
// at their beginning, are everybody's. A CTA's logits come to shared memory by
// bulk copies: all of them under way at once (loads into registers, a step
// ahead, kept 20 KB an SM under way and took twice as long), and read once from
// HBM for both passes over them. Few tokens have occurred or have a bias (a
// percent), so they are a list, laid out once per sequence from a table of
// occurrences in shared memory, a thread an entry, and left out of the passes
// over all the others: the first finds the best token and, relative to each
// thread's running maximum, the sum of the exponentials; the warps of all CTAs
// send those to all CTAs (st.async, counted by an mbarrier of the receiver: a
// cluster barrier in its place cost 1.5 us a position, 120 us against 106 for 32
// sequences of 8); the second writes the probabilities. HBM sees the logits and
// the outputs once, which is what bounds a large batch (without penalties 3.9
// TB/s of 238 MB); with them the lists' chains do (106 us against 60), and a
// small call the chain history -> table -> list -> exchange (9.5 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdio.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "dflash_logits.h"
#include "kernels.h"
#include "spans.h"

namespace dfl {

dflash_status host_fail(dflash_status st, const char *msg);

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 8;                  // tokens of a lane in a step
constexpr int kLogStep = 11;
constexpr int kStep = 1 << kLogStep;     // tokens of a CTA in a step
static_assert(kStep == kThreads * kPer, "a step is a piece");
constexpr int kMaxCluster = 16;
constexpr int kMaxList = 1536;           // tokens of a CTA on its list; with more it goes by the bits

struct LogitsParams {
    const void *logits;
    void *out;
    float *probs;
    int32_t *argmax;
    int64_t seq_stride, row_stride, out_seq_stride, out_row_stride;
    int64_t vocab;
    int batch, rows, group, groups;  // positions of a cluster, clusters of a sequence
    int slice;                       // tokens of a CTA, a multiple of kStep
    int most, wide;                  // entries that a CTA's list can have; 32 bits an entry of a table, not 16
    int C, log_c;
    dflash_logits_rules r;
    const int32_t *draft;
    int64_t draft_stride;
    const int32_t *mask;
    int64_t mask_seq_stride, mask_row_stride;
    int counted, biased;             // there are tokens (or drafts) that penalties count; there are biases
    int lost_rank, lost_at;          // a CTA of the first cluster whose copies do not come, from which of its positions on; -1: none
};

struct alignas(16) Best {
    float m, s;   // maximum and sum of exp((x - m) / tau)
    float v;      // the largest x that is a number, and the lowest token that has it
    int id;
};

template <typename T>
__device__ __forceinline__ T from_f(float v)
{
    if constexpr (std::is_same_v<T, float>) return v;
    else if constexpr (std::is_same_v<T, __half>) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

// One of the two 16-bit values of a word.
template <typename T>
__device__ __forceinline__ float half_of(uint32_t w, int high)
{
    if constexpr (std::is_same_v<T, __half>)
        return __half2float(__ushort_as_half(static_cast<uint16_t>(high ? w >> 16 : w)));
    else
        return __uint_as_float(high ? w & 0xFFFF0000u : w << 16);
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void join_best(float &v, int &id, float v2, int id2)
{
    if (v2 > v || (v2 == v && id2 < id)) {
        v = v2;
        id = id2;
    }
}

// Over the warp: the maximum and the sum relative to it (a sum that is no number stays one), the best token.
__device__ __forceinline__ void reduce(Best &q, float scale, bool sum, bool best)
{
    if (sum) {
        const float m = ordered_to_f32(__reduce_max_sync(0xFFFFFFFFu, f32_to_ordered(q.m)));  // (never NaN)
        q.s = q.m == m ? q.s : q.s * exp2_fast((q.m - m) * scale);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) q.s += __shfl_xor_sync(0xFFFFFFFFu, q.s, o);
        q.m = m;
    }
    if (best) {
        const float v = ordered_to_f32(__reduce_max_sync(0xFFFFFFFFu, f32_to_ordered(q.v)));
        q.id = __reduce_min_sync(0xFFFFFFFFu, q.v == v ? q.id : 0x7FFFFFFF);
        q.v = v;
    }
}

// Shared memory in words: a position's logits; the mask's bits; bits of the tokens on the list (marks) and of those with a
// bias (listed); the list; a table of what has occurred, which the list is made from; a hash table of the listed tokens' places
// in the list of biases. Entries of the table are 32 bits (wide) or 16: the highest says that the token is in the prompt, the
// others how often it has occurred behind it. What counts is how many CTAs fit an SM. Four do with the tables of 151,936 tokens
// of 16 bits and 512 biases; a second table in place of the hash left room for three (134 us against 90 for 32 sequences of 8
// after 2000 with 300 biases), a list of 2048 for two with 32-bit logits, not three (170 us against 130), and a position's
// logits on their way beside the last one's for two (230 us against 115 for 256 positions after 8000).
struct Room {
    int logits, bits, list, counts, places, total;
};

// Slots of the hash table: a power of two, and no fewer than a CTA's tokens with a bias.
__host__ __device__ inline int slots_of(int slice, int biases)
{
    if (biases == 0) return 0;
    int n = 4;
    while (n < biases && n < slice) n *= 2;
    return n;
}

__host__ __device__ inline Room room_of(int slice, int size, int most, bool counted, int biases, bool wide)
{
    Room r = {slice / 4 * size, slice / 32, 0, 0, 0, 0};
    r.total = r.logits + r.bits;
    if (!counted && biases == 0) return r;
    r.list = ((most < kMaxList ? most : kMaxList) + 3) / 4 * (wide ? 8 : 4);
    r.counts = counted ? (wide ? slice : slice / 2) : 0;
    r.places = slots_of(slice, biases) * (wide ? 2 : 1);
    r.total += (biases > 0 ? 2 : 1) * r.bits + r.list + r.places + r.counts;
    return r;
}

// A CTA's tokens on the list. Tokens go by their index in the CTA's own.
struct Marked {
    uint32_t *marks, *listed, *list, *counts, *places;
    uint32_t slots;
    bool wide;

    __device__ __forceinline__ uint32_t occurrence(int at) const
    {
        return wide ? counts[at] : counts[at >> 1] >> (16 * (at & 1)) & 0xFFFFu;
    }
    __device__ __forceinline__ bool bit(const uint32_t *bits, int at) const { return bits[at >> 5] >> (at & 31) & 1u; }

    // One more token that has occurred (fewer than 2^15 without `wide`, so that no count runs over).
    __device__ __forceinline__ void occurred(int at, bool prompt) const
    {
        if (wide) {
            if (prompt) atomicOr(counts + at, 0x80000000u);
            else atomicAdd(counts + at, 1u);
        } else {
            const int sh = 16 * (at & 1);
            if (prompt) atomicOr(counts + (at >> 1), 0x8000u << sh);
            else atomicAdd(counts + (at >> 1), 1u << sh);
        }
    }
    // how often, of an entry that is not 0
    __device__ __forceinline__ float times(uint32_t entry) const { return static_cast<float>(entry & (wide ? 0x7FFFFFFFu : 0x7FFFu)); }

    // Where the search for a token begins (Knuth's multiplicative hashing); it goes on slot by slot.
    __device__ __forceinline__ uint32_t slot(int at) const { return static_cast<uint32_t>(at) * 0x9E3779B1u >> (__clz(slots) + 1); }

    // A slot is the token and its place by 16 bits each, or (wide) the token, 1 more, and its place.
    __device__ __forceinline__ void has_bias(int at, uint32_t place) const  // place > 0; the last one counts
    {
        atomicOr(listed + (at >> 5), 1u << (at & 31));
        for (uint32_t i = slot(at);; i = (i + 1) & (slots - 1)) {
            const uint32_t key = wide ? static_cast<uint32_t>(at) + 1u : static_cast<uint32_t>(at) << 16 | place;
            uint32_t *const word = wide ? places + 2 * i : places + i;
            const uint32_t was = atomicCAS(word, 0u, key);
            if (was != 0u && (wide ? was != key : was >> 16 != static_cast<uint32_t>(at))) continue;
            if (wide) atomicMax(word + 1, place);
            else if (was != 0u) atomicMax(word, key);
            return;
        }
    }
    __device__ __forceinline__ uint32_t place(int at) const  // of a listed token
    {
        for (uint32_t i = slot(at);; i = (i + 1) & (slots - 1)) {
            if (wide) {
                if (places[2 * i] == static_cast<uint32_t>(at) + 1u) return places[2 * i + 1];
            } else if (places[i] >> 16 == static_cast<uint32_t>(at) && places[i] != 0u) {
                return places[i] & 0xFFFFu;
            }
        }
    }

    // which of 8 tokens from `at` on have occurred, a bit each
    __device__ __forceinline__ uint32_t occurrences(int at) const
    {
        uint32_t m = 0;
        if (wide) {
#pragma unroll
            for (int j = 0; j < 8; ++j) m |= (counts[at + j] != 0u) << j;
        } else {
            const uint4 w = *reinterpret_cast<const uint4 *>(counts + (at >> 1));
            const uint32_t v[4] = {w.x, w.y, w.z, w.w};
            if (v[0] | v[1] | v[2] | v[3]) {
#pragma unroll
                for (int j = 0; j < 8; ++j) m |= ((v[j >> 1] >> (16 * (j & 1)) & 0xFFFFu) != 0u) << j;
            }
        }
        return m;
    }

    __device__ __forceinline__ void put(int e, int at, uint32_t count) const
    {
        if (wide) list[2 * e] = static_cast<uint32_t>(at), list[2 * e + 1] = count;
        else list[e] = static_cast<uint32_t>(at) | count << 16;
    }
    __device__ __forceinline__ int token(int e) const { return static_cast<int>(wide ? list[2 * e] : list[e] & 0xFFFFu); }
    __device__ __forceinline__ uint32_t count(int e) const { return wide ? list[2 * e + 1] : list[e] >> 16; }
};

// A lane's 8 tokens of a step as they are loaded. kVec: adjacent ones, by 16 bytes; else every 32nd.
template <typename T, bool kVec>
struct Raw {
    static constexpr int kWords = kVec && sizeof(T) == 2 ? 4 : 8;
    uint32_t w[kWords];

    __device__ __forceinline__ float get(int j) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
        else if constexpr (kVec) return half_of<T>(w[j >> 1], j & 1);
        else return half_of<T>(w[j], 0);
    }

    // at: the index of the lane's first token
    __device__ __forceinline__ void load(const T *logits, int at)
    {
        if constexpr (kVec) {
            const uint4 *const from = reinterpret_cast<const uint4 *>(logits + at);
#pragma unroll
            for (int q = 0; q < kWords / 4; ++q) {
                const uint4 x = from[q];
                w[4 * q] = x.x, w[4 * q + 1] = x.y, w[4 * q + 2] = x.z, w[4 * q + 3] = x.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                if constexpr (sizeof(T) == 4) w[j] = reinterpret_cast<const uint32_t *>(logits)[at + j * 32];
                else w[j] = reinterpret_cast<const uint16_t *>(logits)[at + j * 32];
            }
        }
    }

    // a bit each for the lane's tokens
    static __device__ __forceinline__ uint32_t bits(const uint32_t *from, int at)
    {
        if constexpr (kVec) return reinterpret_cast<const uint8_t *>(from)[at >> 3];
        uint32_t r = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) r |= (from[(at >> 5) + j] >> (at & 31) & 1u) << j;
        return r;
    }

    // the values; -inf for those that `keep` leaves out
    __device__ __forceinline__ void values(uint32_t keep, float2 (&x)[kPer / 2]) const
    {
#pragma unroll
        for (int j = 0; j < kPer / 2; ++j) x[j] = make_float2(get(2 * j), get(2 * j + 1));
        if (keep != 0xFFu) {
#pragma unroll
            for (int j = 0; j < kPer / 2; ++j) {
                x[j].x = keep >> (2 * j) & 1u ? x[j].x : -INFINITY;
                x[j].y = keep >> (2 * j + 1) & 1u ? x[j].y : -INFINITY;
            }
        }
    }
};

// Two fp32 operations by one instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}\n"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}\n"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

template <bool kVec, typename Y>
__device__ __forceinline__ void store8(Y *to, int v, int vocab, const float2 (&y)[kPer / 2])
{
    if constexpr (kVec) {
        if (v >= vocab) return;
        if constexpr (sizeof(Y) == 4) {
            *reinterpret_cast<float4 *>(to + v) = make_float4(y[0].x, y[0].y, y[1].x, y[1].y);
            *reinterpret_cast<float4 *>(to + v + 4) = make_float4(y[2].x, y[2].y, y[3].x, y[3].y);
        } else {
            alignas(16) Y o[kPer];
#pragma unroll
            for (int j = 0; j < kPer / 2; ++j) o[2 * j] = from_f<Y>(y[j].x), o[2 * j + 1] = from_f<Y>(y[j].y);
            *reinterpret_cast<uint4 *>(to + v) = *reinterpret_cast<const uint4 *>(o);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (v + j * 32 < vocab) to[v + j * 32] = from_f<Y>(j & 1 ? y[j >> 1].y : y[j >> 1].x);
    }
}

// x = exp2((x + less) * scale)
__device__ __forceinline__ void exponentials(float2 (&x)[kPer / 2], float2 less, float2 scale)
{
#pragma unroll
    for (int j = 0; j < kPer / 2; ++j) {
        x[j] = mul2(add2(x[j], less), scale);
        x[j] = make_float2(exp2_fast(x[j].x), exp2_fast(x[j].y));
    }
}

struct Shared {
    Best peer[2][kMaxCluster * kWarps];
    uint64_t full;     // a position's logits have arrived
    uint64_t came[2];  // the warps' results of a position have
    int abort_flag;
    int warp_n[kWarps];
    int n;  // entries of the list
};

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads, 4) logits_kernel(const __grid_constant__ LogitsParams p)
{
    extern __shared__ uint4 smem[];
    __shared__ Shared s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = p.C;
    const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const bool tables = p.counted || p.biased;
    const Room room = room_of(p.slice, sizeof(T), p.most, p.counted, p.biased ? p.r.bias_count : 0, p.wide);
    uint32_t *const words = reinterpret_cast<uint32_t *>(smem);
    T *const logits = reinterpret_cast<T *>(words);
    uint32_t *const mask = words + room.logits;
    Marked mk;
    mk.marks = mask + room.bits;
    mk.listed = mk.marks + room.bits;
    mk.list = mk.listed + (p.biased ? room.bits : 0);
    mk.places = mk.list + room.list;
    mk.counts = mk.places + room.places;
    mk.slots = static_cast<uint32_t>(room.places) >> (p.wide ? 1 : 0);
    mk.wide = p.wide;
    if (tables) {
        auto clear = [&](uint32_t *from, int n) {
            for (int i = tid; i < n / 4; i += kThreads) reinterpret_cast<uint4 *>(from)[i] = make_uint4(0, 0, 0, 0);
        };
        if (p.counted) clear(mk.counts, room.counts);
        if (p.biased) {
            clear(mk.listed, room.bits);
            clear(mk.places, room.places);
        }
    }
    if (tid == 0) {
        mbar_init(smem_u32(&s.full), 1);
        mbar_init(smem_u32(&s.came[0]), 1);
        mbar_init(smem_u32(&s.came[1]), 1);
        s.abort_flag = 0;
        s.n = 0;
        fence_mbar_init();
    }
    const int b = static_cast<int>(blockIdx.x) / p.groups, g = static_cast<int>(blockIdx.x) % p.groups;
    const int t0 = g * p.group, t1 = min(p.rows, t0 + p.group);
    // the CTA's tokens: pieces rank, rank + C, .. of kStep
    const int vocab = static_cast<int>(p.vocab), pieces = (vocab + kStep - 1) >> kLogStep;
    const int mine = (pieces - rank + C - 1) >> p.log_c;
    auto token_of = [&](int at) { return ((((at >> kLogStep) << p.log_c) + rank) << kLogStep) + (at & (kStep - 1)); };
    // this lane's first token and its index, and from one step to the next
    const int at0 = warp * (32 * kPer) + (kVec ? lane * kPer : lane), first = (rank << kLogStep) + at0, stride = C << kLogStep;
    auto row_at = [&](int t) { return static_cast<const T *>(p.logits) + b * p.seq_stride + t * p.row_stride; };
    // A position's logits on their way to shared memory (where nobody reads the last one's any more).
    auto bring = [&](int t) {
        const T *const row = row_at(t);
        if (kVec) {
            if (warp == 0) {
                const uint32_t bar = smem_u32(&s.full);
                if (lane == 0) {
                    const int end = mine > 0 ? token_of((mine - 1) * kStep) + kStep : 0;  // behind the last piece
                    mbar_arrive_expect_tx(bar, static_cast<uint32_t>((mine * kStep - max(0, end - vocab)) * sizeof(T)));
                }
                __syncwarp();
                const bool lost = rank == p.lost_rank && blockIdx.x == 0 && t - t0 == p.lost_at;
                for (int i = lane; i < mine && !lost; i += 32) {
                    const int v = token_of(i * kStep);
                    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                     smem_u32(logits + i * kStep)),
                                 "l"(row + v), "r"(static_cast<uint32_t>(min(kStep, vocab - v) * sizeof(T))), "r"(bar)
                                 : "memory");
                }
            }
        } else {  // rows that do not start on 16 bytes
            for (int i = 0; i < mine; ++i) {  // (a whole piece without looking at its end: 8 loads under way a thread)
                const int v = token_of(i * kStep) + tid;
                T x[kPer];
                if (v - tid + kStep <= vocab) {
#pragma unroll
                    for (int j = 0; j < kPer; ++j) x[j] = row[v + j * kThreads];
#pragma unroll
                    for (int j = 0; j < kPer; ++j) logits[i * kStep + tid + j * kThreads] = x[j];
                } else {
                    for (int j = 0; v + j * kThreads < vocab; ++j) logits[i * kStep + tid + j * kThreads] = row[v + j * kThreads];
                }
            }
        }
    };
    // Its mask, without what lies behind the vocabulary.
    auto bring_mask = [&](int t) {
        const int32_t *const from = p.mask ? p.mask + b * p.mask_seq_stride + t * p.mask_row_stride : nullptr;
        for (int w = tid; w < mine * (kStep / 32); w += kThreads) {
            const int v = token_of(w * 32);
            uint32_t m = v < vocab ? (from ? static_cast<uint32_t>(from[v >> 5]) : 0xFFFFFFFFu) : 0u;
            if (v < vocab && vocab - v < 32) m &= (1u << (vocab - v)) - 1u;
            mask[w] = m;
        }
    };
    __syncthreads();
    // (waited for before the first exchange: every CTA's shared memory exists before another writes to it)
    const bool exchange = C > 1 && (p.probs || p.argmax);
    if (C > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    pdl_trigger();
    pdl_wait();
    bring(t0);
    bring_mask(t0);

    const int32_t *const draft = p.draft && p.counted ? p.draft + b * p.draft_stride : nullptr;
    const float rho = p.r.repetition ? p.r.repetition[b] : 1.f, alpha = p.r.presence ? p.r.presence[b] : 0.f,
                beta = p.r.frequency ? p.r.frequency[b] : 0.f, tau = p.r.temperature ? p.r.temperature[b] : 1.f;
    const float *const bias_values = p.biased ? p.r.bias_values + b * p.r.bias_stride : nullptr;
    auto place = [&](int32_t token) {  // a token's index in its CTA's own
        return ((token >> (kLogStep + p.log_c)) << kLogStep) + (token & (kStep - 1));
    };
    auto owner = [&](int32_t token) { return token >> kLogStep & (C - 1); };
    auto known = [&](int32_t token) { return token >= 0 && token < vocab; };
    if (tables) {
        if (p.counted) {
            const int32_t *const tokens = p.r.tokens ? p.r.tokens + b * p.r.token_stride : nullptr;
            const int len = tokens ? min(max(p.r.lens[b], 0), p.r.token_cols) : 0;
            const int prompt = p.r.prompt_lens ? p.r.prompt_lens[b] : 0;
            constexpr int kAtOnce = 16;
            for (int i0 = tid; i0 < len; i0 += kAtOnce * kThreads) {
                int32_t w[kAtOnce];
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u) w[u] = i0 + u * kThreads < len ? tokens[i0 + u * kThreads] : -1;
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u)
                    if (known(w[u]) && owner(w[u]) == rank) mk.occurred(place(w[u]), i0 + u * kThreads < prompt);
            }
            if (draft)
                for (int i = tid; i < t0; i += kThreads)
                    if (known(draft[i]) && owner(draft[i]) == rank) mk.occurred(place(draft[i]), false);
        }
        if (p.biased) {
            const int32_t *const ids = p.r.bias_ids + b * p.r.bias_stride;
            for (int i = tid; i < p.r.bias_count; i += kThreads)
                if (known(ids[i]) && owner(ids[i]) == rank) mk.has_bias(place(ids[i]), static_cast<uint32_t>(i) + 1u);
        }
        __syncthreads();
        // the list: a thread has every 256th eight tokens, and its entries follow one another (an order that does not depend
        // on timing, as sums over the list then do not either)
        auto todo = [&](int w) {
            return (p.counted ? mk.occurrences(w * 8) : 0u) | (p.biased ? reinterpret_cast<const uint8_t *>(mk.listed)[w] : 0u);
        };
        int n = 0;
        for (int w = tid; w < mine * (kStep / 8); w += kThreads) {
            const uint32_t m = todo(w);
            reinterpret_cast<uint8_t *>(mk.marks)[w] = static_cast<uint8_t>(m);
            n += __popc(m);
        }
        int up = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, up, o);
            if (lane >= o) up += y;
        }
        if (lane == 31) s.warp_n[warp] = up;
        __syncthreads();
        int e = up - n;
        for (int w = 0; w < warp; ++w) e += s.warp_n[w];
        if (tid == kThreads - 1) s.n = e + n;
        for (int w = tid; n > 0; w += kThreads)
            for (uint32_t m = reinterpret_cast<const uint8_t *>(mk.marks)[w]; m; m &= m - 1, ++e, --n) {
                const int at = w * 8 + __ffs(m) - 1;
                if (e < kMaxList) mk.put(e, at, p.counted ? mk.occurrence(at) : 0u);
            }
    }
    __syncwarp();
    if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");

    const bool greedy = tau == 0.f;
    float scale = greedy ? 1.f : 1.4426950408889634f / tau;
    if (scale == INFINITY) scale = 3.4028235e38f;  // (so that the best token's 0 * scale stays 0,
    if (scale == 0.f) scale = 1.1754944e-38f;      // and a masked token's -inf * scale -inf)
    const float2 scale2 = make_float2(scale, scale);
    const bool want_sum = p.probs && !greedy, want_best = p.argmax || (p.probs && greedy);
    // With the best token alone wanted, a position's exchange passes beside the next one's pass, and who has it knows it: the
    // last one's goes to rank 0 alone.
    const bool lazy = exchange && !p.out && !p.probs;
    // What does not arrive in a second is given up. A CTA without its logits sends nothing more, so that the cluster's others
    // give up too where they need what it would have sent.
    bool arrived = true;
    int left = t1;  // the positions from here on have been given up
    // All warps' results of position t, joined.
    auto collect = [&](int t, bool read) {
        if (C > 1) {  // (who reads what other CTAs sent acquires it at cluster scope)
            const uint32_t bar = smem_u32(&s.came[t & 1]), parity = static_cast<uint32_t>((t - t0) >> 1) & 1u;
            arrived = (read ? mbar_wait_cluster(bar, parity, &s.abort_flag) : mbar_wait(bar, parity, &s.abort_flag)) && arrived;
        }
        __syncwarp();
        Best q = {-INFINITY, 0.f, -INFINITY, 0x7FFFFFFF};
        if (!read) return q;
        for (int u = lane; u < C * kWarps; u += 32) {
            const Best a = s.peer[t & 1][u];
            if (a.m > q.m) {
                q.s *= exp2_fast((q.m - a.m) * scale);
                q.m = a.m;
            }
            q.s += a.m == q.m ? a.s : a.s * exp2_fast((a.m - q.m) * scale);
            join_best(q.v, q.id, a.v, a.id);
        }
        reduce(q, scale, want_sum, want_best);
        return q;
    };
    auto best_of = [&](const Best &q) { return q.id == 0x7FFFFFFF || !arrived ? -1 : q.id; };
    auto store_best = [&](int t, const Best &q) {
        if (p.argmax && rank == 0 && tid == 0) p.argmax[static_cast<int64_t>(b) * p.rows + t] = best_of(q);
    };
    for (int t = t0; t < t1; ++t) {
        const int64_t at_row = static_cast<int64_t>(b) * p.rows + t;
        T *const out = p.out ? static_cast<T *>(p.out) + b * p.out_seq_stride + t * p.out_row_stride : nullptr;
        if (kVec) {
            arrived = mbar_wait(smem_u32(&s.full), static_cast<uint32_t>(t - t0) & 1u, &s.abort_flag) && arrived;
            if (t + 1 < t1 && tid < mine) {  // the next position's logits come to L2 beside this one's passes (mine < 256)
                const int v = token_of(tid * kStep);
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(row_at(t + 1) + v),
                             "r"(static_cast<uint32_t>(min(kStep, vocab - v) * sizeof(T)))
                             : "memory");
            }
        }
        // the list, the mask (and logits that threads have brought) are complete
        if (__syncthreads_or(!arrived)) {
            // (what has been started lands before the CTA can end)
            if (kVec && tid == 0) mbar_wait(smem_u32(&s.full), static_cast<uint32_t>(t - t0) & 1u, &s.abort_flag, false);
            __syncthreads();
            left = lazy && t > t0 ? t - 1 : t;
            break;
        }
        Best q = {-INFINITY, 0.f, -INFINITY, 0x7FFFFFFF};
        const int marked = tables ? s.n : 0;
        // all tokens but those on the list
        auto walk = [&](auto body) {
            for (int v = first, at = at0; v < vocab; v += stride, at += kStep) {
                Raw<T, kVec> r;
                r.load(logits, at);
                float2 x[kPer / 2];
                r.values(r.bits(mask, at) & ~(tables ? r.bits(mk.marks, at) : 0u), x);
                body(x, v);
            }
        };
        float2 less = make_float2(0.f, 0.f);  // what exponentials are relative to
        auto pass = [&](auto sum, auto best, auto any) {
            const bool writes = decltype(any)::value && out && !p.probs;
            walk([&](float2 (&x)[kPer / 2], int v) {
                const float top = max3(max3(max3(x[0].x, x[0].y, x[1].x), x[1].y, x[2].x), max3(x[2].y, x[3].x, x[3].y), -INFINITY);
                if (decltype(best)::value && (!decltype(any)::value || want_best) && top > q.v) {
                    q.v = top;
#pragma unroll
                    for (int j = kPer - 1; j >= 0; --j)
                        if ((j & 1 ? x[j >> 1].y : x[j >> 1].x) == top) q.id = v + (kVec ? j : j * 32);
                }
                if (decltype(sum)::value && (!decltype(any)::value || want_sum)) {
                    if (top > q.m) {
                        if (q.m > -INFINITY) q.s *= exp2_fast((q.m - top) * scale);
                        q.m = top;
                        less = make_float2(-top, -top);  // (before: nothing yet, exp of -inf or NaN)
                    }
                    exponentials(x, less, scale2);
                    const float2 e = add2(add2(x[0], x[1]), add2(x[2], x[3]));
                    q.s += e.x + e.y;
                } else if (writes) {
                    store8<kVec>(out, v, vocab, x);
                }
            });
        };
        constexpr std::true_type yes;
        constexpr std::false_type no;
        if (want_sum && !want_best)
            pass(yes, no, no);
        else if (want_best && !want_sum && !out)
            pass(no, yes, no);
        else if (want_sum || want_best || !p.probs)
            pass(yes, yes, yes);
        // the tokens on the list under the rules, each by one thread
        auto marked_tokens = [&](auto body) {
            auto one = [&](int at, uint32_t entry) {
                const int v = token_of(at);
                float x;
                if constexpr (sizeof(T) == 4) x = logits[at];
                else x = half_of<T>(reinterpret_cast<const uint16_t *>(logits)[at], 0);
                if (entry) {
                    x = x > 0.f ? __fdiv_rn(x, rho) : __fmul_rn(x, rho);
                    const float c = mk.times(entry);
                    if (c > 0.f) x = __fsub_rn(__fsub_rn(x, __fmul_rn(beta, c)), alpha);
                }
                if (p.biased && mk.bit(mk.listed, at)) x = __fadd_rn(x, bias_values[mk.place(at) - 1]);
                body(mk.bit(mask, at) ? x : -INFINITY, v);
            };
            // (by the bits if the list is too short: one loop for both, a step of which finds the next token)
            const bool listed = marked <= kMaxList;
            uint32_t m = 0;
            int w = tid - kThreads, e = tid;
            while (true) {
                int at;
                if (listed) {
                    if (e >= marked) break;
                    at = mk.token(e);
                } else {
                    while (m == 0 && (w += kThreads) < mine * (kStep / 8)) m = reinterpret_cast<const uint8_t *>(mk.marks)[w];
                    if (m == 0) break;
                    at = w * 8 + __ffs(m) - 1;
                    m &= m - 1;
                }
                one(at, listed ? mk.count(e) : p.counted ? mk.occurrence(at) : 0u);
                e += kThreads;
            }
        };
        if (want_sum || want_best) {
            if (marked > 0)
                marked_tokens([&](float x, int v) {
                    join_best(q.v, q.id, x, x > -INFINITY ? v : 0x7FFFFFFF);
                    if (want_sum) {
                        if (x > q.m) {
                            if (q.m > -INFINITY) q.s *= exp2_fast((q.m - x) * scale);
                            q.m = x;
                        }
                        q.s += exp2_fast((x - (q.m == -INFINITY ? 0.f : q.m)) * scale);
                    }
                });
            reduce(q, scale, want_sum, want_best);
            if (lazy && t > t0) store_best(t - 1, collect(t - 1, rank == 0 && warp == 0));
            Best *const here = &s.peer[t & 1][rank * kWarps + warp];
            if (C > 1) {
                // To every CTA. (A position's place is written again two positions on: by then a warp has every other warp's
                // results of the position between, and those were sent when this one's had been read.)
                const bool one = lazy && t + 1 == t1;
                if (tid == 0 && (rank == 0 || !one))
                    mbar_arrive_expect_tx(smem_u32(&s.came[t & 1]), static_cast<uint32_t>(C * kWarps * sizeof(Best)));
                if (lane < (one ? 1 : C))
                    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                                     mapa_shared(smem_u32(here), static_cast<uint32_t>(lane))),
                                 "r"(__float_as_uint(q.m)), "r"(__float_as_uint(q.s)), "r"(__float_as_uint(q.v)), "r"(q.id),
                                 "r"(mapa_shared(smem_u32(&s.came[t & 1]), static_cast<uint32_t>(lane)))
                                 : "memory");
                __syncwarp();
                if (t + 1 == t1 && (lazy || p.group == 1)) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
            } else {
                if (lane == 0) *here = q;
                __syncthreads();
            }
            if (!lazy) {
                q = collect(t, p.probs || (rank == 0 && warp == 0));
                store_best(t, q);
            }
        }
        const int id = best_of(q);
        float *const probs = p.probs ? p.probs + at_row * p.vocab : nullptr;
        const float base = q.m == -INFINITY ? 0.f : q.m;
        // (nothing above -inf: zeros. A sum that is no number makes all of them such.)
        const float inv = !arrived ? __int_as_float(0x7FFFFFFF) : q.m == -INFINITY && q.s == 0.f ? 0.f : 1.f / q.s;
        const float other = arrived ? 0.f : __int_as_float(0x7FFFFFFF);  // of a token that is not the best, with tau = 0
        if (probs) {
            less = make_float2(-base, -base);
            const float2 inv2 = make_float2(inv, inv);
            walk([&](float2 (&x)[kPer / 2], int v) {
                if (out) store8<kVec>(out, v, vocab, x);
                if (greedy) {
#pragma unroll
                    for (int j = 0; j < kPer / 2; ++j) {
                        x[j].x = v + (kVec ? 2 * j : 64 * j) == id ? 1.f : other;
                        x[j].y = v + (kVec ? 2 * j + 1 : 64 * j + 32) == id ? 1.f : other;
                    }
                } else {
                    exponentials(x, less, scale2);
#pragma unroll
                    for (int j = 0; j < kPer / 2; ++j) x[j] = mul2(x[j], inv2);
                }
                store8<kVec>(probs, v, vocab, x);
            });
        }
        const bool more = t + 1 < t1;
        if (marked > 0 && (probs || out)) {  // over what the passes wrote there
            __syncthreads();
            marked_tokens([&](float x, int v) {
                if (out) out[v] = from_f<T>(x);
                if (probs) probs[v] = greedy ? (v == id ? 1.f : other) : exp2_fast((x - base) * scale) * inv;
            });
        }
        if (more) {
            __syncthreads();  // this position's logits and mask have been read
            bring(t + 1);
            bring_mask(t + 1);
            if (draft) {  // the next position follows one more draft
                const int32_t token = draft[t];
                const bool here = known(token) && owner(token) == rank;
                const int at = here ? place(token) : 0;
                const bool old = here && mk.bit(mk.marks, at);
                if (old && marked <= kMaxList)
                    for (int e = tid; e < marked; e += kThreads)
                        if (mk.token(e) == at) mk.put(e, at, mk.count(e) + 1u);
                __syncthreads();
                if (here && tid == 0) {
                    mk.occurred(at, false);  // (for a list that is or gets too short)
                    if (!old && marked < kMaxList) mk.put(marked, at, 1u);
                    if (!old) s.n = marked + 1;
                    mk.marks[at >> 5] |= 1u << (at & 31);
                }
            }
        }
    }
    const bool together = p.group > 1 && C > 1 && !lazy;  // (see below)
    if (left < t1) {
        const float none = __int_as_float(0x7FFFFFFF);
        for (int t = left; t < t1; ++t) {
            T *const out = p.out ? static_cast<T *>(p.out) + b * p.out_seq_stride + t * p.out_row_stride : nullptr;
            float *const probs = p.probs ? p.probs + (static_cast<int64_t>(b) * p.rows + t) * p.vocab : nullptr;
            for (int at = tid; at < mine * kStep; at += kThreads) {
                const int v = token_of(at);
                if (v < vocab && out) out[v] = from_f<T>(none);
                if (v < vocab && probs) probs[v] = none;
            }
            if (p.argmax && rank == 0 && tid == 0) p.argmax[static_cast<int64_t>(b) * p.rows + t] = -1;
        }
        __syncwarp();
        if (exchange && !together) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    } else if (lazy && rank == 0) {
        store_best(t1 - 1, collect(t1 - 1, warp == 0));
    }
    // no CTA ends while another may still send to it
    __syncwarp();
    // (a cluster that ends together leaves room for one of the next call's on as many SMs: with several positions each, 32
    // sequences of 8 took 115 us otherwise, against 104; with one position each it costs 2 %)
    if (together) cluster_sync_all();
    else if (exchange) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
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
    *smem = optin - static_cast<int>(sizeof(Shared));
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

static dflash_status adjust(const void *logits, int64_t seq_stride, int64_t row_stride, int32_t batch, int32_t rows, int64_t vocab,
                            int32_t dtype, const dflash_logits_rules *rules, const int32_t *draft, int64_t draft_stride,
                            const int32_t *mask, int64_t mask_seq_stride, int64_t mask_row_stride, void *out,
                            int64_t out_seq_stride, int64_t out_row_stride, float *probs, int32_t *argmax, int32_t lost_rank,
                            int32_t lost_at, void *stream)
{
    if (dtype != DFLASH_BF16 && dtype != DFLASH_FP16 && dtype != DFLASH_FP32)
        return logits_fail(DFLASH_ERR_UNSUPPORTED, "dtype must be BF16, FP16 or FP32 (got %lld)", dtype);
    if (batch < 0 || rows < 0 || static_cast<int64_t>(batch) * rows >= (int64_t(1) << 31))
        return logits_fail(DFLASH_ERR_INVALID_ARG, "batch and rows must be >= 0, their product below 2^31 (got %lld, %lld)", batch, rows);
    if (vocab < 1) return logits_fail(DFLASH_ERR_INVALID_ARG, "vocab must be at least 1 (got %lld)", vocab);
    if (vocab > int64_t(1) << 30) return logits_fail(DFLASH_ERR_UNSUPPORTED, "a vocabulary must be at most 2^30 (got %lld)", vocab);
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
    // (the logits and out may be slices of one buffer, whose rows pass one another)
    const int64_t count = static_cast<int64_t>(batch) * rows, vector = static_cast<int64_t>(batch) * 4;
    const dfl::Rows outputs[] = {{out, vocab * size, rows, out_row_stride * size, batch, out_seq_stride * size},
                                 {probs, count * vocab * 4},
                                 {argmax, count * 4}};
    const dfl::Rows inputs[] = {{logits, vocab * size, rows, row_stride * size, batch, seq_stride * size},
                                {draft, (rows - 1) * int64_t(4), batch, draft_stride * 4},
                                {mask, (vocab + 31) / 32 * 4, rows, mask_row_stride * 4, batch, mask_seq_stride * 4},
                                {p.r.tokens, p.r.token_cols * int64_t(4), batch, p.r.token_stride * 4},
                                {p.r.bias_ids, p.r.bias_count * int64_t(4), batch, p.r.bias_stride * 4},
                                {p.r.bias_values, p.r.bias_count * int64_t(4), batch, p.r.bias_stride * 4},
                                {p.r.lens, vector},
                                {p.r.prompt_lens, vector},
                                {p.r.repetition, vector},
                                {p.r.presence, vector},
                                {p.r.frequency, vector},
                                {p.r.temperature, vector}};
    bool overlap = dfl::folds(outputs[0]) || dfl::meet(outputs[0], outputs[1]) || dfl::meet(outputs[0], outputs[2]) ||
                   dfl::meet(outputs[1], outputs[2]);
    for (const dfl::Rows &o : outputs)
        for (const dfl::Rows &i : inputs) overlap = overlap || ((o.at != i.at || &o != outputs || &i != inputs) && dfl::meet(o, i));
    if (overlap) return logits_fail(DFLASH_ERR_INVALID_ARG, "outputs must not overlap inputs or one another (but out may be the logits)");
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
    p.lost_rank = lost_rank;
    p.lost_at = lost_at;
    // CTAs per cluster: enough that the tables leave room for some CTAs an SM and, with few positions, that all SMs have
    // work of at least a piece
    const int64_t positions = static_cast<int64_t>(batch) * rows;
    const int64_t entries = (p.counted ? (p.r.tokens ? p.r.token_cols : 0) + static_cast<int64_t>(p.draft ? rows - 1 : 0) : 0) + p.r.bias_count;
    auto slice_of = [&](int C) { return ((vocab + dfl::kStep - 1) / dfl::kStep + C - 1) / C * dfl::kStep; };
    auto bytes_of = [&](int64_t slice) {
        p.wide = entries > 32767 || slice > 65536;
        p.most = static_cast<int>(entries < slice ? entries : slice);
        return static_cast<int64_t>(dfl::room_of(static_cast<int>(slice), size, p.most, p.counted, p.r.bias_count, p.wide).total) * 4;
    };
    int C = 1;
    while (C < dfl::kMaxCluster && (slice_of(C) > int64_t(1) << 24 || bytes_of(slice_of(C)) > 50 * 1024 ||
                                    (positions * C < 10 * sms && slice_of(C) > (positions * C < 2 * sms ? 1 : 4) * dfl::kStep)))
        C *= 2;
    const int64_t slice = slice_of(C);
    if (slice > int64_t(1) << 24 || bytes_of(slice) > smem_most)
        return logits_fail(DFLASH_ERR_UNSUPPORTED, "a vocabulary of %lld needs more shared memory than there is (%lld bytes a CTA)", vocab, smem_most);
    // positions per cluster: a sequence's list is laid out once for them, but three CTAs an SM have work (24 sequences of 8:
    // 77 us by 4, 84 by 8; 32: 90 by 4, 85 by 8)
    int group = 1;
    while ((p.counted || p.biased) && group < rows && static_cast<int64_t>(batch) * ((rows + 2 * group - 1) / (2 * group)) * C >= 3 * sms) group *= 2;
    p.group = group < rows ? group : rows;
    p.groups = (rows + p.group - 1) / p.group;
    p.slice = static_cast<int>(slice);
    p.C = C;
    while ((1 << p.log_c) < C) ++p.log_c;
    size_t smem = static_cast<size_t>(bytes_of(slice));
    const int per = 16 / size;
    const bool vec = !dfl::misaligned(logits, 16) && seq_stride % per == 0 && row_stride % per == 0 && vocab % 8 == 0 &&
                     (!out || (!dfl::misaligned(out, 16) && out_seq_stride % per == 0 && out_row_stride % per == 0)) &&
                     !dfl::misaligned(probs, 16);
    const int64_t clusters = static_cast<int64_t>(batch) * p.groups;
    if (clusters >= (int64_t(1) << 31)) return logits_fail(DFLASH_ERR_INVALID_ARG, "too many positions");
    // fewer CTAs than SMs: at most two of them on one (with up to four one block of 8 without penalties took 8.1 us, so 7.4)
    if (clusters * C <= sms && smem < static_cast<size_t>(smem_most) * 2 / 5) smem = static_cast<size_t>(smem_most) * 2 / 5;
    e = dfl::launch_ex(dfl::kernel_of(dtype, vec), dim3(static_cast<unsigned>(clusters), 1, C), dim3(dfl::kThreads),
                       smem, static_cast<cudaStream_t>(stream), C, p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return logits_fail(DFLASH_ERR_CUDA, "the launch failed (error %lld)", e);
    }
    return DFLASH_OK;
}

extern "C" dflash_status dflash_logits_adjust(const void *logits, int64_t seq_stride, int64_t row_stride, int32_t batch,
                                              int32_t rows, int64_t vocab, int32_t dtype, const dflash_logits_rules *rules,
                                              const int32_t *draft, int64_t draft_stride, const int32_t *mask,
                                              int64_t mask_seq_stride, int64_t mask_row_stride, void *out,
                                              int64_t out_seq_stride, int64_t out_row_stride, float *probs, int32_t *argmax,
                                              void *stream)
{
    return adjust(logits, seq_stride, row_stride, batch, rows, vocab, dtype, rules, draft, draft_stride, mask, mask_seq_stride,
                  mask_row_stride, out, out_seq_stride, out_row_stride, probs, argmax, -1, -1, stream);
}

extern "C" dflash_status dflash_selftest_logits_lost(const void *logits, int32_t batch, int32_t rows, int64_t vocab, int32_t dtype,
                                                     const dflash_logits_rules *rules, void *out, float *probs, int32_t *argmax,
                                                     int32_t rank, int32_t at, void *stream)
{
    if (rank < 0 || at < 0) return logits_fail(DFLASH_ERR_INVALID_ARG, "rank and position must be >= 0 (got %lld, %lld)", rank, at);
    return adjust(logits, rows * vocab, vocab, batch, rows, vocab, dtype, rules, nullptr, 0, nullptr, 0, 0, out, rows * vocab, vocab,
                  probs, argmax, rank, at, stream);
}
