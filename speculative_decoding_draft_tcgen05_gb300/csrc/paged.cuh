// Device helpers of the paged-attention kernels: sequences and their visible
// keys, the even split of the work over the CTAs, and small conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "paged.h"

namespace dfl {

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b)
{
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t u);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t u)
{
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t u)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}

// One sequence of the batch: first row, new tokens, length in the cache.
// Everything is clamped to what the call's arrays hold.
struct PagedSeq {
    int t0, n, len;
};

__device__ __forceinline__ PagedSeq paged_seq(const AttendParams &p, int b)
{
    PagedSeq s;
    s.t0 = min(max(__ldg(p.cu + b), 0), p.tokens);
    s.n = min(max(__ldg(p.cu + b + 1), s.t0), p.tokens) - s.t0;
    // (tiles may run past the end, so places stay clear of 2^31)
    const int64_t cap = min(static_cast<int64_t>(p.table_cols) * p.page, (int64_t(1) << 31) - 4096);
    const int len = __ldg(p.lens + b);
    s.len = len < 0 ? 0 : (len > cap ? static_cast<int>(cap) : len);
    return s;
}

// A work item is (sequence, key/value head, R consecutive rows); row r of a
// sequence's n * group rows is query head kvh * group + r % group of its new
// token r / group, so the heads that share keys share a tile. [lo, hi): keys
// that some row of the item sees (empty: lo = hi). A unit is U keys on a
// multiple of U; an item without keys still has one unit, which writes zeros.
struct PagedItem {
    int lo, hi, u0, units;
};

__device__ __forceinline__ PagedItem paged_item(const AttendParams &p, const PagedSeq &s, int rt, int R, int U)
{
    const int r0 = rt * R, r1 = min(s.n * p.group, r0 + R);
    const int ta = p.by_group.div(r0), tb = p.by_group.div(r1 - 1);
    const int base = s.len - s.n;
    PagedItem it;
    it.hi = p.causal ? min(s.len, max(0, base + tb + 1)) : s.len;
    it.lo = p.window > 0 ? max(0, base + ta - p.window + 1) : 0;
    if (it.lo >= it.hi) it.lo = it.hi = 0;
    it.u0 = it.lo / U;
    it.units = max(1, (it.hi + U - 1) / U - it.u0);
    return it;
}

__device__ __forceinline__ int paged_row_tiles(const AttendParams &p, const PagedSeq &s, int R)
{
    return (s.n * p.group + R - 1) / R;
}

// The units of all items in order (sequence, head, row tile), split evenly:
// CTA c of G takes units [total * c / G, total * (c + 1) / G), with G the grid,
// or `total` where that is less: every one of the G CTAs has a unit, so the
// CTAs that share an item are consecutive. Every CTA works
// this out for itself from the lengths on the device: the launch needs
// nothing from the host, and a captured graph stays valid when they change.
struct PagedPlan {
    int64_t total, begin, end;
    int64_t ctas;  // G
    int b;         // sequence of unit `begin`
    int per_head;  // its units per key/value head
    int64_t off;   // the offset of `begin` within that sequence's units
};

constexpr int kPlanSeqs = 512;  // sequences whose units are kept in shared memory

// Units per key/value head of a sequence, by one thread or by a whole warp.
__device__ __forceinline__ int paged_units(const AttendParams &p, const PagedSeq &s, int R, int U)
{
    const int nrt = paged_row_tiles(p, s, R);
    int u = 0;
    for (int rt = 0; rt < nrt; ++rt) u += paged_item(p, s, rt, R, U).units;
    return u;
}

__device__ __forceinline__ int paged_units_warp(const AttendParams &p, const PagedSeq &s, int R, int U, int lane)
{
    const int nrt = paged_row_tiles(p, s, R);
    int u = 0;
    for (int rt = lane; rt < nrt; rt += 32) u += paged_item(p, s, rt, R, U).units;
    return __reduce_add_sync(0xFFFFFFFFu, u);
}

// units: kPlanSeqs ints of shared memory that are free until the plan is made.
template <int NT>
__device__ PagedPlan paged_plan(const AttendParams &p, int R, int U, int *units)
{
    __shared__ int64_t warp_sum[NT / 32];
    __shared__ PagedPlan plan;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + NT - 1) / NT;
    const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    const bool kept = p.B <= kPlanSeqs;

    // Sequences of a few row tiles by a thread each, longer ones by a warp each.
    bool many = false;
    for (int b = tid; b < p.B; b += NT) {
        if (kept) {
            const PagedSeq s = paged_seq(p, b);
            const bool by_warp = paged_row_tiles(p, s, R) > 2;
            units[b] = by_warp ? -1 : paged_units(p, s, R, U);
            many |= by_warp;
        }
        if (blockIdx.x == 0) {  // what paged_seq() had to clamp
            const int len = __ldg(p.lens + b), t0 = __ldg(p.cu + b), t1 = __ldg(p.cu + b + 1);
            if (len < 0 || len > static_cast<int64_t>(p.table_cols) * p.page || t0 < 0 || t1 < t0 || t1 > p.tokens)
                atomicOr(p.err, DEV_ERR_PLACE);
        }
    }
    if (__syncthreads_or(many)) {
        for (int b = warp; b < p.B; b += NT / 32)
            if (units[b] < 0) {
                const int u = paged_units_warp(p, paged_seq(p, b), R, U, lane);
                __syncwarp();
                if (lane == 0) units[b] = u;
            }
        __syncthreads();
    }
    auto seq_units = [&](int b) {
        return static_cast<int64_t>(kept ? units[b] : paged_units(p, paged_seq(p, b), R, U)) * p.kv_heads;
    };
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += seq_units(b);
    int64_t scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    int64_t before = scan - mine, total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    const int64_t G = min(static_cast<int64_t>(gridDim.x), total), c = blockIdx.x;
    const int64_t begin = c < G ? total * c / G : 0, end = c < G ? total * (c + 1) / G : 0;
    if (begin < end ? (before <= begin && begin < before + mine) : tid == 0) {
        int64_t off = begin - before, u = 1;
        int b = b0;
        if (begin < end)
            for (; b < b1; ++b) {
                u = seq_units(b);
                if (off < u) break;
                off -= u;
            }
        plan.total = total;
        plan.begin = begin;
        plan.end = end;
        plan.ctas = G;
        plan.b = b;
        plan.per_head = static_cast<int>(u / p.kv_heads);
        plan.off = off;
    }
    __syncthreads();
    return plan;
}

// The CTA's pieces one after the other: (sequence, head, row tile) and the
// units [a, e) of it, with whether the item begins before or goes on after.
struct PagedPiece {
    PagedSeq s;
    PagedItem it;
    int b, kvh, rt;
    int a, e;  // unit range within the item
};

struct PagedWalk {
    PagedPiece pc;
    int64_t left;
    int nrt, off;

    // Whole warps call it.
    __device__ void start(const AttendParams &p, const PagedPlan &plan, int R, int U)
    {
        left = plan.end - plan.begin;
        if (left <= 0) return;
        const int lane = threadIdx.x & 31;
        pc.b = plan.b;
        pc.s = paged_seq(p, pc.b);
        nrt = paged_row_tiles(p, pc.s, R);
        pc.kvh = static_cast<int>(plan.off / plan.per_head);
        int rem = static_cast<int>(plan.off - static_cast<int64_t>(pc.kvh) * plan.per_head);
        for (int from = 0;; from += 32) {  // the row tile that holds unit `rem` of the head, 32 at a time
            const int u = from + lane < nrt ? paged_item(p, pc.s, from + lane, R, U).units : 0;
            int upto = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
                if (lane >= o) upto += v;
            }
            const int all = __shfl_sync(0xFFFFFFFFu, upto, 31);
            if (rem < all) {
                const int k = __ffs(__ballot_sync(0xFFFFFFFFu, rem < upto)) - 1;
                off = rem - __shfl_sync(0xFFFFFFFFu, upto - u, k);
                pc.rt = from + k;
                break;
            }
            rem -= all;
        }
        pc.it = paged_item(p, pc.s, pc.rt, R, U);
        cut();
    }
    __device__ void cut()
    {
        pc.a = off;
        pc.e = static_cast<int>(min(static_cast<int64_t>(pc.it.units), off + left));
    }
    // On to the next piece; false when the CTA's share is done.
    __device__ bool next(const AttendParams &p, int R, int U)
    {
        left -= pc.e - pc.a;
        if (left <= 0) return false;
        off = 0;
        if (++pc.rt == nrt) {
            pc.rt = 0;
            if (++pc.kvh == p.kv_heads) {
                pc.kvh = 0;
                do {
                    ++pc.b;
                    pc.s = paged_seq(p, pc.b);
                    nrt = paged_row_tiles(p, pc.s, R);
                } while (nrt == 0);  // ends: there are units left
            }
        }
        pc.it = paged_item(p, pc.s, pc.rt, R, U);
        cut();
        return true;
    }
};

// CTA that holds unit u of `total` over G CTAs.
__device__ __forceinline__ int paged_owner(int64_t u, int64_t total, int64_t G)
{
    return static_cast<int>(((u + 1) * G - 1) / total);
}

// The CTAs that share the current piece's item: the first, and how many.
__device__ __forceinline__ int2 paged_sharers(const PagedPlan &plan, const PagedWalk &w)
{
    const int64_t first = plan.end - w.left - w.pc.a;
    const int c0 = paged_owner(first, plan.total, plan.ctas);
    return make_int2(c0, paged_owner(first + w.pc.it.units - 1, plan.total, plan.ctas) - c0 + 1);
}

// Slot of part i of the item that CTA c0 begins.
__device__ __forceinline__ int64_t paged_slot(int c0, int i)
{
    return 2 * static_cast<int64_t>(c0 + i) + (i == 0);
}

// A warp has written its rows of a part: true if it is the last of `parts` to
// do so, and may read the others'.
__device__ __forceinline__ bool paged_last(unsigned *ticket, int parts, int lane)
{
    __threadfence();
    __syncwarp();
    unsigned got = 0;
    if (lane == 0) {
        got = atomicAdd(ticket, 1u);
        if (got == static_cast<unsigned>(parts) - 1) *ticket = 0;  // for the next call
    }
    got = __shfl_sync(0xFFFFFFFFu, got, 0);
    __threadfence();
    return got == static_cast<unsigned>(parts) - 1;
}

// True (and the counter is cleared) if all parts but this warp's are written
// already: then it need not write its own.
__device__ __forceinline__ bool paged_all_others(unsigned *ticket, int parts, int lane)
{
    unsigned got = 0;
    if (lane == 0) {
        got = atomicAdd(ticket, 0u);
        if (got == static_cast<unsigned>(parts) - 1) *ticket = 0;
    }
    got = __shfl_sync(0xFFFFFFFFu, got, 0);
    if (got != static_cast<unsigned>(parts) - 1) return false;
    __threadfence();
    return true;
}

}  // namespace dfl
