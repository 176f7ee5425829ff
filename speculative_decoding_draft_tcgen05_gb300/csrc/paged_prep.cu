// Per-head RMS norm and position rotation of queries and keys, with the keys
// and values written to a paged cache where one is given.
#include <type_traits>

#include "paged.cuh"

namespace dfl {

namespace {

// e4m3 pair, rounded to nearest even, saturating at +-448 (NaN stays NaN).
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Index of the last entry of cu[0 .. B] (not decreasing) that is <= t; whole
// warp, 32 entries a step.
__device__ __forceinline__ int warp_find(const int32_t *cu, int B, int t, int lane)
{
    int lo = 0, size = B + 1;
    while (size > 1) {
        const int step = (size + 31) / 32, i = lo + lane * step;
        const bool below = lane * step < size && __ldg(cu + i) <= t;
        const int n = __popc(__ballot_sync(0xFFFFFFFFu, below));
        const int skip = max(0, n - 1) * step;
        lo += skip;
        size = min(step, size - skip);
    }
    return lo;
}

// ---------------------------------------------------------------------------
// A block takes up to prep_tokens() tokens. It first finds their places in the
// cache and positions (a chain of dependent small reads, once per block) and
// brings their cosines and sines to shared memory. Then its warps share the
// jobs: 32 / LPH heads of the queries, keys or values (LPH = D / 8 lanes to a
// head, 8 values each) of one token, or in a large batch of 4 consecutive
// ones, so that a job's pointers and weights are set up once for several rows.
// A lane holds four whole rotation pairs, 4 values from each half of the
// rotated part (or 8 adjacent ones where pairs are adjacent), so the rotation
// needs no exchange between lanes, and the sum of squares is a shuffle over the
// head's lanes.
//
// Each value is read and written once, so HBM would be the bound. Measured, a
// third of its rate is used and 56 to 62 % of the issue slots: what bounds it is
// the number of instructions (some 200 a warp for 256 values, near half of them
// addresses and job numbers) together with their latency, which 32 warps an SM
// do not hide (fixed-latency and long-scoreboard waits lead). Inputs come through asynchronous copies to
// shared memory, several jobs of a warp in flight: the first ones while the
// block looks up its places and angles, the others while the warp works.
// Rotation of 16001 tokens' 32 + 8 heads of 64 values, fp16: 31.6 us, 5.2 TB/s;
// 8 + 8 heads of 128 values of 16384 tokens into a cache, bf16: 34.0 us, 4.2
// TB/s; 20 + 4 heads of 128 of 4096 tokens 16.4 us, 3.2 TB/s; a block of 8
// tokens 2 to 3 us on the GPU. (Warps that keep to their heads for all tokens
// of a block have less to set up, but took 69, 45 and 19 us for the first
// three.)
// ---------------------------------------------------------------------------
constexpr int kPrepThreads = 256, kPrepWarps = kPrepThreads / 32, kPrepBlocks = 4;

// Jobs of a warp whose inputs are in flight.
constexpr int prep_ahead(int job) { return job == 1 ? 4 : 2; }

// Tokens of a block (with the copies' 32 KB, what fits 48 KB of shared memory).
template <int D>
constexpr int prep_tokens()
{
    return D <= 128 ? 16 : 8;
}

template <int D, typename T, int kPrepJob>
__global__ void __launch_bounds__(kPrepThreads, kPrepBlocks) prep_kernel(const __grid_constant__ PrepParams p, int per_block)
{
    constexpr int LPH = D / 8, HPP = 32 / LPH;
    constexpr int TOKENS = prep_tokens<D>(), kPrepAhead = prep_ahead(kPrepJob);
    __shared__ int64_t tok_row[TOKENS];        // its row of the cache (without the head)
    __shared__ int tok_pos[TOKENS], tok_is[TOKENS];  // position; 1: stored, 0: no place, -1: padding
    __shared__ float4 angles[TOKENS * D / 4];  // [token][rotary]: cosines, then sines
    __shared__ uint4 ring[kPrepWarps][kPrepAhead][kPrepJob][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane % LPH, grp = lane / LPH;
    const int pq = (p.q.heads + HPP - 1) / HPP, pk = (p.k.heads + HPP - 1) / HPP, pv = (p.v.heads + HPP - 1) / HPP;
    const int passes = pq + pk + pv, R = p.rotary;
    const int t0 = blockIdx.x * per_block, nt = min(per_block, p.tokens - t0);
    const int groups = (nt + kPrepJob - 1) / kPrepJob, stride = kPrepWarps * gridDim.y;
    const int rot_lanes = R / 8;
    pdl_trigger();
    pdl_wait();

    // Job (pass, g): the pass's heads of tokens kPrepJob * g ... A warp takes every stride-th, passes first.
    struct Job {
        int pass, g;
    };
    auto step = [&](Job &j) {
        for (j.pass += stride; j.pass >= passes; j.pass -= passes) ++j.g;
    };
    Job now = {warp + kPrepWarps * static_cast<int>(blockIdx.y), 0};
    for (; now.pass >= passes; now.pass -= passes) ++now.g;
    Job ahead = now;
    auto part_of = [&](int pass) { return pass < pq ? 0 : (pass < pq + pk ? 1 : 2); };
    auto rows_of = [&](int part) -> const PrepRows & { return part == 0 ? p.q : (part == 1 ? p.k : p.v); };
    auto head_of = [&](int pass, int part) { return (pass - (part == 0 ? 0 : (part == 1 ? pq : pq + pk))) * HPP + grp; };
    auto fetch = [&](int slot) {
        if (ahead.g < groups) {
            const int part = part_of(ahead.pass), h = head_of(ahead.pass, part), k0 = ahead.g * kPrepJob;
            const PrepRows &x = rows_of(part);
            const T *src = static_cast<const T *>(x.in) + (t0 + k0) * x.in_ts + h * x.in_hs + 8 * sub;
#pragma unroll
            for (int u = 0; u < kPrepJob; ++u, src += x.in_ts)
                if (h < x.heads && k0 + u < nt)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(&ring[warp][slot][u][lane])), "l"(src)
                                 : "memory");
            step(ahead);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int a = 0; a < kPrepAhead; ++a) fetch(a);

    // ---- places, pages and positions
    if (p.append) {
        for (int k = warp; k < nt; k += kPrepWarps) {
            const int t = t0 + k, b = warp_find(p.batch.cu_tokens, p.batch.batch, t, lane);
            int page = -1, slot = 0, place = 0;
            const bool padding = b >= p.batch.batch;
            if (!padding) {
                const int from = __ldg(p.batch.cu_tokens + b), to = __ldg(p.batch.cu_tokens + b + 1);
                place = __ldg(p.batch.lens + b) - (to - from) + (t - from);
                const int col = place / p.page;
                slot = place - col * p.page;
                if (place >= 0 && col < p.batch.table_cols) page = __ldg(p.batch.page_table + b * p.batch.table_stride + col);
                if (page < 0 || page >= p.cache.num_pages) {
                    page = -1;
                    if (lane == 0) atomicOr(p.err, DEV_ERR_PLACE);
                }
            }
            if (lane == 0) {
                tok_is[k] = padding ? -1 : page >= 0;
                tok_row[k] = page * p.cache.page_stride + slot * p.cache.slot_stride;
                tok_pos[k] = padding || !p.positions ? place : __ldg(p.positions + t);
            }
        }
        __syncthreads();
    }
    if (R > 0) {
        for (int i = tid; i < nt * (R / 4); i += kPrepThreads) {
            const int k = i / (R / 4);
            int pos = p.append ? tok_pos[k] : __ldg(p.positions + t0 + k);
            if (pos < 0 || pos >= p.positions_n) {
                if (p.append && tok_is[k] >= 0 && i % (R / 4) == 0) atomicOr(p.err, DEV_ERR_PLACE);
                pos = min(max(pos, 0), p.positions_n - 1);
            }
            angles[i] = __ldg(reinterpret_cast<const float4 *>(p.table + static_cast<int64_t>(pos) * R) + i % (R / 4));
        }
        __syncthreads();
    }

    const float k_inv = p.fp8 ? 1.f / p.cache.k_scale : 1.f, v_inv = p.fp8 ? 1.f / p.cache.v_scale : 1.f;
    for (int slot = 0; now.g < groups; step(now), slot = (slot + 1) % kPrepAhead) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kPrepAhead - 1) : "memory");
        __syncwarp();
        const int part = part_of(now.pass), h = head_of(now.pass, part), k0 = now.g * kPrepJob;
        const PrepRows &x = rows_of(part);
        const bool active = h < x.heads, cached = part > 0 && p.append, quant = cached && p.fp8;
        const T *const weight = part < 2 ? static_cast<const T *>(x.weight) : nullptr;
        const bool turn = part < 2 && R > 0;

        // Eight values of a head, in 16 or 8 bits, in two pieces of 4 (from oa and ob).
        auto store = [&](int u, int oa, int ob, uint2 ya, uint2 yb) {
            const int k = k0 + u;
            if (!active || k >= nt || (p.append && tok_is[k] < (cached ? 1 : 0))) return;
            T *to = cached ? static_cast<T *>(part == 1 ? p.cache.k : p.cache.v) + tok_row[k] + h * p.cache.head_stride
                           : static_cast<T *>(x.out) + (t0 + k) * x.out_ts + h * x.out_hs;
            if (ob == oa + 4) {
                *reinterpret_cast<uint4 *>(to + oa) = make_uint4(ya.x, ya.y, yb.x, yb.y);
            } else {
                *reinterpret_cast<uint2 *>(to + oa) = ya;
                *reinterpret_cast<uint2 *>(to + ob) = yb;
            }
        };
        auto store_e4m3 = [&](int u, int oa, int ob, const float2(&f)[4]) {
            const int k = k0 + u;
            if (!active || k >= nt || tok_is[k] < 1) return;
            uint8_t *to = static_cast<uint8_t *>(part == 1 ? p.cache.k : p.cache.v) + tok_row[k] + h * p.cache.head_stride;
            const float inv = part == 1 ? k_inv : v_inv;
            const float2 by = make_float2(inv, inv);
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 g = __fmul2_rn(f[e], by);
                y[e] = f32x2_to_e4m3x2(g.x, g.y);
            }
            if (ob == oa + 4) {
                *reinterpret_cast<uint2 *>(to + oa) = make_uint2(y[0] | y[1] << 16, y[2] | y[3] << 16);
            } else {
                *reinterpret_cast<uint32_t *>(to + oa) = y[0] | y[1] << 16;
                *reinterpret_cast<uint32_t *>(to + ob) = y[2] | y[3] << 16;
            }
        };
        // Norm and rotation: f[0], f[1] and f[2], f[3] are the lane's two pieces.
        auto transform = [&](auto halves, int oa, int ob) {
            float2 w[4];
            if (weight) {
                const uint2 wa = __ldg(reinterpret_cast<const uint2 *>(weight + oa)), wb = __ldg(reinterpret_cast<const uint2 *>(weight + ob));
                w[0] = unpack2<T>(wa.x), w[1] = unpack2<T>(wa.y), w[2] = unpack2<T>(wb.x), w[3] = unpack2<T>(wb.y);
            }
            const float4 *ang = angles + k0 * (R / 4) + sub;
            const bool turned = turn && sub < rot_lanes;
#pragma unroll
            for (int u = 0; u < kPrepJob; ++u) {
                const T *row = reinterpret_cast<const T *>(ring[warp][slot][u]) + grp * D;
                const uint2 xa = *reinterpret_cast<const uint2 *>(row + oa), xb = *reinterpret_cast<const uint2 *>(row + ob);
                float2 f[4] = {unpack2<T>(xa.x), unpack2<T>(xa.y), unpack2<T>(xb.x), unpack2<T>(xb.y)};
                if (weight) {
                    float2 s2 = __fmul2_rn(f[0], f[0]);
#pragma unroll
                    for (int e = 1; e < 4; ++e) s2 = __ffma2_rn(f[e], f[e], s2);
                    float ss = s2.x + s2.y;
#pragma unroll
                    for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
                    const float r = rsqrtf(ss * (1.f / D) + p.eps);
                    const float2 by = make_float2(r, r);
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[e] = __fmul2_rn(__fmul2_rn(f[e], by), w[e]);
                }
                if (turned) {
                    const float4 c = ang[u * (R / 4)], s = ang[u * (R / 4) + R / 8];
                    if constexpr (decltype(halves)::value) {
                        const float2 c0 = make_float2(c.x, c.y), c1 = make_float2(c.z, c.w);
                        const float2 s0 = make_float2(s.x, s.y), s1 = make_float2(s.z, s.w);
                        const float2 n0 = make_float2(-s.x, -s.y), n1 = make_float2(-s.z, -s.w);
                        const float2 a0 = f[0], a1 = f[1], b0 = f[2], b1 = f[3];
                        f[0] = __ffma2_rn(a0, c0, __fmul2_rn(b0, n0));
                        f[1] = __ffma2_rn(a1, c1, __fmul2_rn(b1, n1));
                        f[2] = __ffma2_rn(b0, c0, __fmul2_rn(a0, s0));
                        f[3] = __ffma2_rn(b1, c1, __fmul2_rn(a1, s1));
                    } else {
                        const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            f[e] = __ffma2_rn(f[e], make_float2(cs[e], cs[e]),
                                              __fmul2_rn(make_float2(f[e].y, f[e].x), make_float2(-sn[e], sn[e])));
                    }
                }
                if (quant)
                    store_e4m3(u, oa, ob, f);
                else
                    store(u, oa, ob, make_uint2(pack2<T>(f[0].x, f[0].y), pack2<T>(f[1].x, f[1].y)),
                          make_uint2(pack2<T>(f[2].x, f[2].y), pack2<T>(f[3].x, f[3].y)));
            }
        };
        if (turn && !p.interleaved) {
            // 4 values of each half; lanes past the rotated part share the rest in the same way
            const int oa = sub < rot_lanes ? 4 * sub : R + 4 * (sub - rot_lanes);
            transform(std::true_type(), oa, oa + (sub < rot_lanes ? R / 2 : (D - R) / 2));
        } else if (weight || turn) {
            transform(std::false_type(), 8 * sub, 8 * sub + 4);
        } else {
#pragma unroll
            for (int u = 0; u < kPrepJob; ++u) {
                const uint4 v = ring[warp][slot][u][lane];
                if (quant) {
                    const float2 f[4] = {unpack2<T>(v.x), unpack2<T>(v.y), unpack2<T>(v.z), unpack2<T>(v.w)};
                    store_e4m3(u, 8 * sub, 8 * sub + 4, f);
                } else {
                    store(u, 8 * sub, 8 * sub + 4, make_uint2(v.x, v.y), make_uint2(v.z, v.w));
                }
            }
        }
        __syncwarp();
        fetch(slot);
    }
}

template <int D, typename T>
cudaError_t go(const PrepParams &p, cudaStream_t s)
{
    // As many tokens a block as fill every SM's kPrepBlocks blocks once, up to prep_tokens() (a large batch then shares
    // place and angle reads between a block's warps), in jobs of 4 from 3 on; a small batch has one or two tokens a
    // block and jobs of one (272 tokens of 56 heads: 9.5 us with jobs of 4, most of them empty), spread over several
    // blocks where some are left.
    constexpr int HPP = 32 / (D / 8);
    int dev = 0, sms = 1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int slots = kPrepBlocks * sms, per = (p.tokens + slots - 1) / slots;
    const bool many = per > 2;
    int per_block = many ? (per + 3) / 4 * 4 : per;
    if (per_block > prep_tokens<D>()) per_block = prep_tokens<D>();
    const int blocks = (p.tokens + per_block - 1) / per_block;
    const int passes = (p.q.heads + HPP - 1) / HPP + (p.k.heads + HPP - 1) / HPP + (p.v.heads + HPP - 1) / HPP;
    const int jobs = passes * (many ? per_block / 4 : per_block);
    int y = slots / blocks;
    const int most = (jobs + kPrepWarps - 1) / kPrepWarps;
    y = y < 1 ? 1 : (y > most ? most : y);
    return many ? launch_ex(prep_kernel<D, T, 4>, dim3(blocks, y), dim3(kPrepThreads), 0, s, 1, p, per_block)
                : launch_ex(prep_kernel<D, T, 1>, dim3(blocks, y), dim3(kPrepThreads), 0, s, 1, p, per_block);
}

}  // namespace

cudaError_t launch_prep(const PrepParams &p, int head_dim, int dtype, cudaStream_t s)
{
    if (dtype == DFLASH_BF16) {
        if (head_dim == 64) return go<64, __nv_bfloat16>(p, s);
        if (head_dim == 128) return go<128, __nv_bfloat16>(p, s);
        return go<256, __nv_bfloat16>(p, s);
    }
    if (head_dim == 64) return go<64, __half>(p, s);
    if (head_dim == 128) return go<128, __half>(p, s);
    return go<256, __half>(p, s);
}

}  // namespace dfl
