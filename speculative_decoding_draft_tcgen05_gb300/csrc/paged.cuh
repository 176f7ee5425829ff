// Device helpers of the paged-attention kernels: sequences and their visible
// keys, the even split of the work over the CTAs, and small conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

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

// The natural logarithm of a row's sum, from its maximum (log2) and the sum taken against it: -inf where it sees no key
// (both are -inf then), NaN where a score is NaN (the maximum passes those over, the sum does not) or +inf.
__device__ __forceinline__ float row_lse(float max, float sum)
{
    return (max + lg2(sum)) * 0.69314718055994531f;
}

// Four e4m3 values -> two pairs of fp16 (exact).
__device__ __forceinline__ void e4m3x4_to_h2x2(uint32_t x, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
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

// Softmax weights are rounded to the 16-bit type of the second product: with a second part for what the rounding takes
// off, that product would be two. Where many keys count, the results' error against 64 bits is then about 1.4 times that of their
// own rounding alone (relative, 0.0023 instead of 0.0017 in bf16, 0.00029 instead of 0.00021 in fp16). The sums take
// the weights unrounded. bf16 has the range of fp32; fp16 weights are taken against the running maximum less this many
// powers of two, which is then the maximum that goes with their sum. They are at most 2^15 so (a maximum may be stale by
// 2^8), and what fp16 cannot hold is 2^-32 of the largest weight a key, not 2^-25 (131,072 such keys would add up to
// 0.4 %).
template <typename CT>
constexpr float weight_lift()
{
    return std::is_same<CT, __half>::value ? 7.f : 0.f;
}

// Exponent of a query row's largest magnitude, for products in fp16 (8-bit caches): the row is scaled by 2^(8 - e), so
// that magnitude comes to [2^8, 2^9) and bf16 queries of any size fit. Values below 2^-22 of it lose bits to fp16's
// smallest step, at most 2^-33 of it each. (Zero, subnormal and infinite rows get the nearest e whose powers of two and
// their inverses are ordinary numbers.)
__device__ __forceinline__ int query_exponent(float top)
{
    return max(-118, min(127, static_cast<int>(__float_as_uint(top) >> 23) - 127));
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

// How a kernel cuts the work. A work item is (sequence, key/value head, R
// consecutive rows); row r of a sequence's n * group rows is query head
// kvh * group + r % group of its new token r / group, so the heads that share
// keys share a tile. A unit is U keys on a multiple of U. Starting and
// finishing an item costs about as much as C units.
struct PagedCut {
    int R, U, C;
};

// [lo, hi): keys that some row of the item sees (empty: lo = hi). An item
// without keys still has one unit, which writes zeros.
struct PagedItem {
    int lo, hi, u0, units;
};

__host__ __device__ __forceinline__ PagedItem paged_item(const AttendParams &p, const PagedSeq &s, int rt, PagedCut k)
{
    const int r0 = rt * k.R, r1 = r0 + min(k.R, s.n * p.group - r0);  // (a sequence has up to 2^31 - 1 rows)
    const int ta = p.by_group.div(r0), tb = p.by_group.div(r1 - 1);
    const int base = s.len - s.n;
    PagedItem it;
    it.hi = p.causal ? min(s.len, max(0, base + tb + 1)) : s.len;
    it.lo = p.window > 0 ? max(0, base + ta - p.window + 1) : 0;
    if (it.lo >= it.hi) it.lo = it.hi = 0;
    it.u0 = it.lo / k.U;
    it.units = max(1, (it.hi + k.U - 1) / k.U - it.u0);
    return it;
}

__host__ __device__ __forceinline__ int paged_row_tiles(const AttendParams &p, const PagedSeq &s, int R)
{
    return static_cast<int>((static_cast<uint32_t>(s.n * p.group) + R - 1) / R);
}

// The items' costs (units + C) of a lane's heads in order (sequence, head, row
// tile) are split evenly over its CTAs: boundary c of G lies at total * c / G,
// moved to the item's start where it falls into the C, and the lane's CTA c
// takes what is between boundaries c and c + 1. G is its CTAs, or the sum
// where that is less. Every CTA works this out
// for itself from the lengths on the device: the launch needs nothing from the
// host, and a captured graph stays valid when they change. (C, in
// the few-row kernel: 32 ragged sequences of 32 rows and 500 to 7000 keys took
// 112 us with C = 0, 102 with 5, 98 with 8, 101 with 14; 128 single tokens of an
// 8-bit cache 92 us with 0, 88 with 5, 89 with 8. In the other kernel seven
// windowed chunks took 55 us with 0, 44 with 4.)
struct PagedPlan {
    int64_t total, begin, end;
    int ctas;      // G
    int lane0, cta;  // the lane's first CTA and this one, numbered lane by lane (an idle CTA beyond them: its block)
    int64_t off;   // `begin` within its head
    int b, kvh;    // its sequence and head
    PagedSeq s;    // the sequence
};

// n / d, which the 64-bit division (some hundred cycles) is only needed for when they do not fit 32 bits.
__device__ __forceinline__ int64_t paged_quot(int64_t n, int64_t d)
{
    return (n | d) >> 32 ? n / d : static_cast<int64_t>(static_cast<uint32_t>(n) / static_cast<uint32_t>(d));
}

// Sequences whose costs are kept in shared memory. Beyond it each CTA works them out twice, a thread's sequences one
// after the other, which the work itself hides: single tokens of 512, 513, 4,096 and 65,536 sequences of 64 keys (32 / 8
// heads of 128 values, bf16) take 32, 33, 245 and 3,836 us.
constexpr int kPlanSeqs = 512;

// Cost per key/value head of a sequence, by one thread or by a whole warp. Sums of costs have 64 bits: 2^28 row tiles
// (tokens * heads < 2^31, 8 rows at least) of 2^25 units are 2^53, and their product with the number of CTAs
// (paged_sharers()) stays below 2^63.
__host__ __device__ __forceinline__ int64_t paged_cost(const AttendParams &p, const PagedSeq &s, PagedCut k)
{
    const int nrt = paged_row_tiles(p, s, k.R);
    int64_t u = 0;
    for (int rt = 0; rt < nrt; ++rt) u += paged_item(p, s, rt, k).units + k.C;
    return u;
}

__device__ __forceinline__ int64_t paged_cost_warp(const AttendParams &p, const PagedSeq &s, PagedCut k, int lane)
{
    const int nrt = paged_row_tiles(p, s, k.R);
    int64_t u = 0;
    for (int rt = lane; rt < nrt; rt += 32) u += paged_item(p, s, rt, k).units + k.C;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xFFFFFFFFu, u, o);
    return u;
}

// This CTA's share of `total`, its lane's costs.
__device__ __forceinline__ void paged_share(const AttendParams &p, PagedPlan &plan, int64_t total)
{
    const int G = static_cast<int>(min(static_cast<int64_t>(p.lane_ctas), total));
    const int c = static_cast<int>(blockIdx.x) / p.lanes, lane = static_cast<int>(blockIdx.x) - c * p.lanes;
    const bool idle = c >= p.lane_ctas;
    plan.lane0 = lane * p.lane_ctas;
    plan.cta = idle ? static_cast<int>(blockIdx.x) : plan.lane0 + c;
    plan.total = total;
    plan.ctas = G;
    plan.begin = plan.end = 0;
    if (c < G) {  // total * c / G, in parts that fit
        const int64_t q = paged_quot(total, G);
        const int rest = static_cast<int>(total - q * G);
        plan.begin = q * c + static_cast<uint32_t>(rest * c) / static_cast<uint32_t>(G);
        plan.end = q * (c + 1) + static_cast<uint32_t>(rest * (c + 1)) / static_cast<uint32_t>(G);
    }
}

// What paged_seq() had to clamp.
__device__ __forceinline__ void paged_report(const AttendParams &p, int b)
{
    const int len = __ldg(p.lens + b), t0 = __ldg(p.cu + b), t1 = __ldg(p.cu + b + 1);
    if (len < 0 || len > static_cast<int64_t>(p.table_cols) * p.page || t0 < 0 || t1 < t0 || t1 > p.tokens)
        atomicOr(p.err, DEV_ERR_PLACE);
}

// The plan of up to 32 sequences, a lane each: one round of reads, by every
// warp of the block (a call of few units is all latency). Long sequences'
// costs are shared out between the warps, through `cost`; warp 0 returns the
// plan.
template <int NT>
__device__ __forceinline__ PagedPlan paged_plan_warps(const AttendParams &p, PagedCut cut, int64_t *cost)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    PagedPlan plan = {};
    PagedSeq s = {0, 0, 0};
    int64_t head = 0;  // cost per key/value head
    bool many = false;
    if (lane < p.B) {
        s = paged_seq(p, lane);
        many = paged_row_tiles(p, s, cut.R) > 2;
        if (!many) head = paged_cost(p, s, cut);
    }
    const unsigned long_ones = __ballot_sync(0xFFFFFFFFu, many);
    if (long_ones) {
        int k = 0;
        for (unsigned m = long_ones; m; m &= m - 1, ++k) {
            if (k % (NT / 32) != warp) continue;
            const int b = __ffs(m) - 1;
            const PagedSeq of = {0, __shfl_sync(0xFFFFFFFFu, s.n, b), __shfl_sync(0xFFFFFFFFu, s.len, b)};
            const int64_t u = paged_cost_warp(p, of, cut, lane);
            if (lane == 0) cost[b] = u;
        }
        __syncthreads();
        if (many) head = cost[lane];
    }
    if (warp > 0) return plan;
    const int64_t mine = head * p.lane_heads;
    int64_t upto = mine;
    for (int o = 1; o < p.B; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += v;
    }
    paged_share(p, plan, __shfl_sync(0xFFFFFFFFu, upto, p.B - 1));
    const unsigned at = __ballot_sync(0xFFFFFFFFu, lane < p.B && plan.begin < upto);
    plan.b = max(0, __ffs(at) - 1);  // (sequences without new tokens cost nothing and are passed over)
    plan.s = {__shfl_sync(0xFFFFFFFFu, s.t0, plan.b), __shfl_sync(0xFFFFFFFFu, s.n, plan.b), __shfl_sync(0xFFFFFFFFu, s.len, plan.b)};
    const int64_t off = plan.begin - __shfl_sync(0xFFFFFFFFu, upto - mine, plan.b);
    const int64_t per_head = max(int64_t(1), __shfl_sync(0xFFFFFFFFu, head, plan.b));
    const int head_at = static_cast<int>(paged_quot(off, per_head));
    plan.off = off - head_at * per_head;
    plan.kvh = head_at * p.lanes + static_cast<int>(blockIdx.x) % p.lanes;
    if (blockIdx.x == 0 && lane < p.B) paged_report(p, lane);
    return plan;
}

// cost: kPlanSeqs numbers of shared memory that are free until the plan is made.
// The block meets in here at least once.
template <int NT>
__device__ PagedPlan paged_plan(const AttendParams &p, PagedCut cut, int64_t *cost)
{
    __shared__ int64_t warp_sum[NT / 32];
    __shared__ PagedPlan plan;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (p.B <= 32) {
        const PagedPlan small = paged_plan_warps<NT>(p, cut, cost);
        if (tid == 0) plan = small;
        __syncthreads();
        return plan;
    }
    const int per = (p.B + NT - 1) / NT;
    const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    const bool kept = p.B <= kPlanSeqs;

    // Sequences of a few row tiles by a thread each, longer ones by a warp each.
    bool many = false;
    for (int b = tid; b < p.B; b += NT) {
        if (kept) {
            const PagedSeq s = paged_seq(p, b);
            const bool by_warp = paged_row_tiles(p, s, cut.R) > 2;
            cost[b] = by_warp ? -1 : paged_cost(p, s, cut);
            many |= by_warp;
        }
        if (blockIdx.x == 0) paged_report(p, b);
    }
    if (__syncthreads_or(many)) {
        for (int b = warp; b < p.B; b += NT / 32)
            if (cost[b] < 0) {
                const int64_t u = paged_cost_warp(p, paged_seq(p, b), cut, lane);
                __syncwarp();
                if (lane == 0) cost[b] = u;
            }
        __syncthreads();
    }
    auto head_cost = [&](int b) { return kept ? cost[b] : paged_cost(p, paged_seq(p, b), cut); };
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += head_cost(b) * p.lane_heads;
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
    PagedPlan made;
    paged_share(p, made, total);
    if (made.begin < made.end ? (before <= made.begin && made.begin < before + mine) : tid == 0) {
        int64_t off = made.begin - before, per_head = 1;
        int b = b0;
        if (made.begin < made.end)
            for (; b < b1; ++b) {
                per_head = head_cost(b);
                if (off < per_head * p.lane_heads) break;
                off -= per_head * p.lane_heads;
            }
        made.b = b;
        const int at = made.begin < made.end ? static_cast<int>(paged_quot(off, per_head)) : 0;
        made.off = off - at * per_head;
        made.kvh = at * p.lanes + static_cast<int>(blockIdx.x) % p.lanes;
        made.s = paged_seq(p, min(b, p.B - 1));
        plan = made;
    }
    __syncthreads();
    return plan;
}

// The CTA's pieces one after the other: units [a, e) of an item.
struct PagedPiece {
    PagedSeq s;
    PagedItem it;
    int b, kvh, rt;
    int a, e;
};

struct PagedWalk {
    PagedPiece pc;
    int64_t at, end;  // where the item starts in the sum of costs; the CTA's end
    int nrt;
    bool more;        // pc is a piece of this CTA

    // Unit of the item that a boundary (an offset from `at`) stands for.
    __device__ __forceinline__ int unit_at(int64_t off, PagedCut k) const
    {
        return static_cast<int>(max(int64_t(0), min(off - k.C, static_cast<int64_t>(pc.it.units))));
    }
    // Whole warps call it.
    __device__ void start(const AttendParams &p, const PagedPlan &plan, PagedCut k)
    {
        end = plan.end;
        more = plan.begin < plan.end;
        if (!more) return;
        const int lane = threadIdx.x & 31;
        pc.b = plan.b;
        pc.s = plan.s;
        nrt = paged_row_tiles(p, pc.s, k.R);
        pc.kvh = plan.kvh;
        pc.rt = 0;
        int64_t rem = plan.off;
        for (int from = 0; nrt > 1; from += 32) {  // the row tile that holds cost `rem` of the head, 32 at a time
            const int u = from + lane < nrt ? paged_item(p, pc.s, from + lane, k).units + k.C : 0;
            int upto = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
                if (lane >= o) upto += v;
            }
            const int all = __shfl_sync(0xFFFFFFFFu, upto, 31);
            if (rem < all) {
                const int l = __ffs(__ballot_sync(0xFFFFFFFFu, rem < upto)) - 1;
                rem -= __shfl_sync(0xFFFFFFFFu, upto - u, l);
                pc.rt = from + l;
                break;
            }
            rem -= all;
        }
        at = plan.begin - rem;
        pc.it = paged_item(p, pc.s, pc.rt, k);
        pc.a = unit_at(rem, k);
        pc.e = unit_at(end - at, k);
        more = pc.e > pc.a;
        // (rem < units + C, so pc.a < units; a share that ends where it begins has no piece)
    }
    // On to the next piece, if the CTA's share has one.
    __device__ bool next(const AttendParams &p, PagedCut k)
    {
        at += pc.it.units + k.C;
        more = at + k.C < end;
        if (!more) return false;
        if (++pc.rt == nrt) {
            pc.rt = 0;
            pc.kvh += p.lanes;
            if (pc.kvh >= p.kv_heads) {
                pc.kvh %= p.lanes;
                do {  // there are items left (unless the lengths change while the kernel runs)
                    if (++pc.b >= p.B) return more = false;
                    pc.s = paged_seq(p, pc.b);
                    nrt = paged_row_tiles(p, pc.s, k.R);
                } while (nrt == 0);
            }
        }
        pc.it = paged_item(p, pc.s, pc.rt, k);
        pc.a = 0;
        pc.e = unit_at(end - at, k);
        return true;
    }
    // Whether another CTA has a part of the piece's item.
    __device__ __forceinline__ bool split() const { return pc.a > 0 || pc.e < pc.it.units; }
};

// The CTAs that share the piece's item: the first, and how many. Boundary c
// lies inside the item (after its first unit, before its last one's end) if
// at + C < total * c / G rounded down < at + C + units.
__device__ __forceinline__ int2 paged_sharers(const PagedPlan &plan, const PagedWalk &w, PagedCut k)
{
    const int64_t low = w.at + k.C + 1, high = w.at + k.C + w.pc.it.units;  // low <= boundary < high
    const int64_t first = paged_quot(low * plan.ctas + plan.total - 1, plan.total);  // smallest c with total * c / G >= low
    const int64_t end = paged_quot(high * plan.ctas + plan.total - 1, plan.total);   // smallest c with total * c / G >= high
    return make_int2(plan.lane0 + static_cast<int>(first - 1), static_cast<int>(end - first + 1));
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

// How many parts have been written (lane 0 reads; what they are is read after
// paged_all_others()).
__device__ __forceinline__ unsigned paged_written(const unsigned *ticket, int lane)
{
    unsigned n = 0;
    if (lane == 0) asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(n) : "l"(ticket) : "memory");
    return n;
}

// True (and the counter is cleared) if that was all parts but this warp's: then
// it need not write its own.
__device__ __forceinline__ bool paged_all_others(unsigned *ticket, unsigned written, int parts, int lane)
{
    const bool all = __shfl_sync(0xFFFFFFFFu, written, 0) == static_cast<unsigned>(parts) - 1;
    if (all && lane == 0) *ticket = 0;
    if (all) __threadfence();
    return all;
}

}  // namespace dfl
