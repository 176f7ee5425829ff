// y = residual + act(x W^T + bias) on the tcgen05 tensor cores.
//
// The weights are the products' M: 128 rows of W (256 over a CTA pair) are the
// lanes of TMEM, and a tile of NT rows of x its columns, so that a single
// token wastes 15 columns and not 127 lanes. k is streamed by TMA in stages of
// 64 or 128 columns.
//
// Few rows are bound by the stream of W: each weight is read once, from as many
// CTAs as there are (a tile's k split over a cluster of up to 8, whose CTAs
// join their sums through distributed shared memory in the order of their
// ranks, so that results do not depend on timing). Many rows are bound by the
// tensor cores: persistent CTA pairs on tiles of 256 x NT with two accumulators
// in TMEM, so that a tile's epilogue runs beside the next one's products.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdio.h>

#include <new>
#include <type_traits>

#include "common.cuh"
#include "dflash_linear.h"
#include "kernels.h"

namespace dfl {

dflash_status host_fail(dflash_status st, const char *msg);
dflash_status host_make_tmap_rows(CUtensorMap *tm, const void *ptr, int64_t rows, int64_t cols, int64_t stride, int box_rows);

struct LinearParams {
    CUtensorMap tm_w, tm_x;  // boxes of 64 columns x 128 rows, and x the tile's rows of one CTA
    const void *bias, *residual;
    void *y;
    int64_t residual_stride, y_stride;
    int rows, n;
    int NT;              // rows of x per tile
    int boxes, stages;   // 64-column boxes per stage, stages of the ring
    int KB;              // stages that k takes
    int tiles_f, tiles_t, band;
    int split;           // CTAs that share a tile's k
    int act;
    int vec;             // y and residual: 4 values at a time
    int *err;
};

namespace {

constexpr int kThreads = 320;  // TMA, products, 2 x 4 epilogue warps
constexpr int kTileF = 128;    // weight rows of one CTA
constexpr int kBox = 64;       // columns of a box: 128 bytes
constexpr uint32_t kWBox = kTileF * kBox * 2;
constexpr uint32_t kStaging = 16 * kTileF * 4;  // 16 rows of a tile's results, for each epilogue group
constexpr int kMaxSplit = 8;

struct Layout {
    uint32_t stage, staging, bars, total;
};

__host__ __device__ inline Layout layout(int NT, int boxes, int stages, bool pair, int split)
{
    Layout l;
    l.stage = static_cast<uint32_t>(boxes) * (kWBox + static_cast<uint32_t>(pair ? NT / 2 : NT) * kBox * 2);
    l.staging = static_cast<uint32_t>(stages) * l.stage;
    l.bars = l.staging + (split > 1 ? 0 : 2 * kStaging);  // (a split tile's sums go to the ring)
    l.total = l.bars + 8u * (2u * stages + 5u) + 8u;  // full, empty, tfull, tempty, drain; TMEM's address, abort flag
    return l;
}

__host__ __device__ inline int tmem_columns(int NT)
{
    int c = 32;
    while (c < 2 * NT) c <<= 1;
    return c;
}

__device__ __forceinline__ void group_sync(int id)
{
    asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory");
}

// Whether any of the group's 128 threads says so.
__device__ __forceinline__ bool group_any(int id, bool pred)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %2, 0;\n\t"
        "bar.red.or.pred q, %1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r)
        : "r"(id), "r"(static_cast<uint32_t>(pred))
        : "memory");
    return r != 0;
}

__device__ __forceinline__ float4 ld_peer(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Exponentials and quotients by the fast forms: their error is a few 2^-22 of |z| (that of exp(-z) counts only where
// it is not small against 1, and then |z| is not large), below fp32's of a product's sum.
__device__ __forceinline__ float activate(float z, int act)
{
    switch (act) {
    case DFLASH_ACT_RELU:
        return z < 0.f ? 0.f : z;
    case DFLASH_ACT_SILU:
        return __fdividef(z, 1.f + __expf(-z));
    case DFLASH_ACT_GELU:
        return 0.5f * z * (1.f + erff(z * 0.70710678f));
    case DFLASH_ACT_GELU_TANH:  // (1 + tanh u) / 2 = 1 / (1 + exp(-2u))
        return __fdividef(z, 1.f + __expf(-1.5957691f * (z + 0.044715f * z * z * z)));
    default:
        return z;
    }
}

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

// Four values of type Y, as they lie in memory.
template <typename Y>
struct alignas(sizeof(Y) * 4) Four {
    Y v[4];
};

// Results of a row of y: features n0 .. n0 + 127 of the 128 in `src` (shared memory or a sum of it), by one warp.
// A lane has four adjacent features where rows allow (vec), else every 32nd.
template <typename T, typename Y>
struct RowStore {
    const LinearParams &p;
    const int lane, n0;
    float bias[4];
    bool whole;  // all four of the lane's features exist and go as one

    __device__ __forceinline__ int feature(int i) const { return n0 + (p.vec ? lane * 4 + i : lane + 32 * i); }

    __device__ __forceinline__ RowStore(const LinearParams &p_, int lane_, int n0_) : p(p_), lane(lane_), n0(n0_)
    {
        whole = p.vec && n0 + lane * 4 + 3 < p.n;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            bias[i] = p.bias && feature(i) < p.n ? to_f(static_cast<const T *>(p.bias)[feature(i)]) : 0.f;
    }

    // this lane's values of the residual's row
    __device__ __forceinline__ void fetch(int row, Four<Y> &r) const
    {
        const Y *at = static_cast<const Y *>(p.residual) + static_cast<int64_t>(row) * p.residual_stride;
        if (whole) {
            r = *reinterpret_cast<const Four<Y> *>(at + n0 + lane * 4);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (feature(i) < p.n) r.v[i] = at[feature(i)];
        }
    }

    __device__ __forceinline__ void store(int row, const float (&acc)[4], const Four<Y> &r) const
    {
        Four<Y> o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float z = activate(acc[i] + bias[i], p.act);
            if (p.residual) z += to_f(r.v[i]);
            o.v[i] = from_f<Y>(z);
        }
        Y *at = static_cast<Y *>(p.y) + static_cast<int64_t>(row) * p.y_stride;
        if (whole) {
            *reinterpret_cast<Four<Y> *>(at + n0 + lane * 4) = o;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (feature(i) < p.n) at[feature(i)] = o.v[i];
        }
    }
};

// kPair: a cluster of two CTAs computes a tile of 256 weight rows (cta_group::2 products issued by the even CTA):
// each holds 128 weight rows and half of the tile's rows of x, and has the results of its 128 weight rows.
// Otherwise a cluster of p.split CTAs (1: none) shares the stages of one tile.
template <bool kPair, typename T, typename Y>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const __grid_constant__ LinearParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;  // 128-byte swizzled tiles start on 1024 bytes
    uint8_t *const gbase = smem_raw + (base - raw);

    const int NT = p.NT, S = p.stages, BX = p.boxes;
    const int XR = kPair ? NT / 2 : NT;
    const int split = kPair ? 1 : p.split;
    const Layout lay = layout(NT, BX, S, kPair, split);
    const uint32_t w_bytes = static_cast<uint32_t>(BX) * kWBox;
    const uint32_t bar_full = base + lay.bars, bar_empty = bar_full + 8u * S;
    const uint32_t bar_tfull = bar_empty + 8u * S, bar_tempty = bar_tfull + 16u, bar_drain = bar_tempty + 16u;
    uint32_t *const tmem_holder = reinterpret_cast<uint32_t *>(gbase + lay.bars + 8u * (2u * S + 5u));
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = kPair || split > 1 ? cluster_ctarank() : 0u;
    const int team = static_cast<int>(blockIdx.x) / (kPair ? 2 : split);  // the cluster's index, and how many there are
    const int teams = static_cast<int>(gridDim.x) / (kPair ? 2 : split);

    // work items: tiles team, team + teams, .. (a split tile: one), in bands of `band` feature tiles, within which
    // the row tiles follow one another: CTAs that run together share both operands' tiles in L2
    const int items = p.tiles_f * p.tiles_t;
    auto tile_of = [&](int item, int &tf, int &tt) {
        const int per = p.band * p.tiles_t, b = item / per, in = item - b * per;
        const int width = min(p.band, p.tiles_f - b * p.band);
        tt = in / width;
        tf = b * p.band + in - tt * width;
    };
    // this CTA's stages of a tile
    const int kb0 = kPair ? 0 : static_cast<int>(static_cast<int64_t>(p.KB) * rank / split);
    const int kb1 = kPair ? p.KB : static_cast<int>(static_cast<int64_t>(p.KB) * (rank + 1) / split);
    const int my_items = (items - team + teams - 1) / teams;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(bar_full + 8u * s, 1);
            mbar_init(bar_empty + 8u * s, 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(bar_tfull + 8u * a, 1);
            mbar_init(bar_tempty + 8u * a, kPair ? 16 : 8);  // an arrival per epilogue warp (of both CTAs)
        }
        mbar_init(bar_drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&p.tm_w);
        tma_prefetch_desc(&p.tm_x);
    }
    const uint32_t tmem_cols = static_cast<uint32_t>(tmem_columns(NT));
    if (warp == 1) {
        if constexpr (kPair) {
            tmem_alloc_pair(smem_u32(tmem_holder), tmem_cols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(tmem_holder), tmem_cols);
            tmem_relinquish();
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if constexpr (kPair) cluster_sync_all();  // the even CTA's barriers are initialised before any use
    tc_fence_after_sync();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(tmem_holder);
    // What is above overlaps the previous kernel on the stream, and so do the first loads of W, which is constant from
    // the handle's creation on. x, residual and y are touched after that kernel has finished.
    pdl_trigger();
    if (!(warp == 0 && lane == 0)) pdl_wait();

    if (warp == 0) {
        // ---------------------------------------------------------------- loads
        if (lane == 0) {
            const uint64_t pol_w = p.tiles_t == 1 ? l2_policy_evict_first() : l2_policy_evict_normal();
            const uint64_t pol_x = p.tiles_t == 1 ? l2_policy_evict_last() : l2_policy_evict_normal();
            const uint32_t tx = kPair ? 2u * lay.stage : lay.stage;  // a pair counts both CTAs' bytes on the even one's barrier
            auto load = [&](uint32_t dst, const CUtensorMap *tm, int x, int y, uint32_t bar, uint64_t pol) {
                if constexpr (kPair)
                    tma_load_2d_pair(dst, tm, x, y, mapa_shared(bar, 0), pol);
                else
                    tma_load_2d(dst, tm, x, y, bar, pol);
            };
            auto load_w = [&](int it, int tf, int kb) {
                const int s = it % S;
                if (rank == 0 || !kPair) mbar_arrive_expect_tx(bar_full + 8u * s, tx);
                const int row = kPair ? (tf * 2 + static_cast<int>(rank)) * kTileF : tf * kTileF;
                for (int b = 0; b < BX; ++b)
                    load(base + s * lay.stage + b * kWBox, &p.tm_w, (kb * BX + b) * kBox, row, bar_full + 8u * s, pol_w);
            };
            auto load_x = [&](int it, int tt, int kb) {
                const int s = it % S;
                const int row = tt * NT + (kPair ? static_cast<int>(rank) * XR : 0);
                for (int b = 0; b < BX; ++b)
                    load(base + s * lay.stage + w_bytes + b * (XR * kBox * 2), &p.tm_x, (kb * BX + b) * kBox, row,
                         bar_full + 8u * s, pol_x);
            };
            const int per = kb1 - kb0;
            int tf, tt, it = 0;
            tile_of(team, tf, tt);
            const int pre = my_items > 0 ? min(per, S) : 0;
            for (int i = 0; i < pre; ++i) load_w(i, tf, kb0 + i);
            pdl_wait();
            for (; it < pre; ++it) load_x(it, tt, kb0 + it);
            bool ok = true;
            for (int i = 0; ok && i < my_items; ++i) {
                tile_of(team + i * teams, tf, tt);
                for (int k = i == 0 ? pre : 0; k < per; ++k, ++it) {
                    if (!mbar_wait(bar_empty + 8u * (it % S), (static_cast<uint32_t>(it / S) & 1u) ^ 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    load_w(it, tf, kb0 + k);
                    load_x(it, tt, kb0 + k);
                }
            }
            if (!ok) {
                atomicOr(p.err, DEV_ERR_TIMEOUT);
                // what has been issued lands before the CTA can end
                if (rank == 0 || !kPair) {
                    for (int j = it > S ? it - S : 0; j < it; ++j)
                        mbar_wait(bar_full + 8u * (j % S), static_cast<uint32_t>(j / S) & 1u, abort_flag, false);
                } else {  // (counted on the even CTA's barriers: a copy lands within microseconds)
                    const uint64_t t0 = global_timer_ns();
                    while (global_timer_ns() - t0 < 100000ull) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- products (a pair: the even CTA's)
        if (lane == 0 && (rank == 0 || !kPair)) {
            constexpr bool kHalf = std::is_same_v<T, __half>;
            const uint32_t idesc = idesc_bf16_f32(kPair ? 2 * kTileF : kTileF, NT) & (kHalf ? ~((1u << 7) | (1u << 10)) : ~0u);
            int it = 0;
            bool ok = true;
            for (int i = 0; ok && i < my_items; ++i) {
                const int a = i & 1;
                const uint32_t u = static_cast<uint32_t>(i >> 1);
                ok = kPair ? mbar_wait_cluster(bar_tempty + 8u * a, (u & 1u) ^ 1u, abort_flag)
                           : mbar_wait(bar_tempty + 8u * a, (u & 1u) ^ 1u, abort_flag);
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t d = tmem + static_cast<uint32_t>(a * NT);
                for (int k = kb0; k < kb1; ++k, ++it) {
                    const int s = it % S;
                    const uint32_t ph = static_cast<uint32_t>(it / S) & 1u;
                    ok = kPair ? mbar_wait_cluster(bar_full + 8u * s, ph, abort_flag)
                               : mbar_wait(bar_full + 8u * s, ph, abort_flag);
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint32_t sw = base + s * lay.stage, sx = sw + w_bytes;
                    for (int b = 0; b < BX; ++b) {
#pragma unroll
                        for (int j = 0; j < kBox / 16; ++j) {
                            const uint64_t wd = smem_desc_sw128(sw + b * kWBox + 32u * j);
                            const uint64_t xd = smem_desc_sw128(sx + b * (XR * kBox * 2) + 32u * j);
                            const uint32_t acc = (k > kb0 || b > 0 || j > 0) ? 1u : 0u;
                            if constexpr (kPair)
                                umma_bf16_pair(d, wd, xd, idesc, acc);
                            else
                                umma_bf16(d, wd, xd, idesc, acc);
                        }
                    }
                    if constexpr (kPair)
                        umma_commit_pair(bar_empty + 8u * s, 3);
                    else
                        umma_commit(bar_empty + 8u * s);
                }
                if (!ok) break;
                if constexpr (kPair)
                    umma_commit_pair(bar_tfull + 8u * a, 3);
                else
                    umma_commit(bar_tfull + 8u * a);
            }
            if (!ok) atomicOr(p.err, DEV_ERR_TIMEOUT);
            // every product is over before TMEM is released
            if constexpr (kPair)
                umma_commit_pair(bar_drain, 1);
            else
                umma_commit(bar_drain);
            mbar_wait(bar_drain, 0, abort_flag, false);
        }
    } else if (split == 1) {
        // ---------------------------------------------------------------- epilogue: two groups of four warps take turns
        // at a tile's 16-row chunks: TMEM (a feature per lane) -> shared memory -> rows of y
        const int g = (warp - 2) >> 2, gw = (warp - 2) & 3, q = warp & 3;
        float *const stage = reinterpret_cast<float *>(gbase + lay.staging + g * kStaging);
        for (int i = 0; i < my_items; ++i) {
            int tf, tt;
            tile_of(team + i * teams, tf, tt);
            const int a = i & 1;
            const uint32_t u = static_cast<uint32_t>(i >> 1);
            const int n0 = kPair ? (tf * 2 + static_cast<int>(rank)) * kTileF : tf * kTileF;
            const RowStore<T, Y> out(p, lane, n0);
            const int row0 = tt * NT, valid = min(NT, p.rows - row0);
            const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(a * NT);
            bool waited = false, ok = true;
            for (int c = g * 16; c < valid || !waited; c += 32) {
                Four<Y> r[4];
                if (p.residual) {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        if (c + gw + 4 * t < valid) out.fetch(row0 + c + gw + 4 * t, r[t]);
                }
                if (!waited) {
                    const bool got = kPair ? mbar_wait_cluster(bar_tfull + 8u * a, u & 1u, abort_flag)
                                           : mbar_wait(bar_tfull + 8u * a, u & 1u, abort_flag);
                    ok = !group_any(1 + g, !got);
                    waited = true;
                    if (!ok) break;
                    tc_fence_after_sync();
                    if (c >= valid) break;  // (a tile of one chunk: the other group's)
                }
                float v[16];
                __syncwarp();
                tmem_load16(taddr + static_cast<uint32_t>(c), v);
#pragma unroll
                for (int j = 0; j < 16; ++j) stage[j * kTileF + q * 32 + lane] = v[j];
                group_sync(1 + g);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int j = gw + 4 * t;
                    if (c + j < valid) {
                        float z[4];
                        if (p.vec) {
                            const float4 f = *reinterpret_cast<const float4 *>(stage + j * kTileF + lane * 4);
                            z[0] = f.x, z[1] = f.y, z[2] = f.z, z[3] = f.w;
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e) z[e] = stage[j * kTileF + lane + 32 * e];
                        }
                        out.store(row0 + c + j, z, r[t]);
                    }
                }
                group_sync(1 + g);
            }
            if (!ok) break;
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {  // the accumulator goes back to the products' warp
                if constexpr (kPair)
                    mbar_arrive_remote(mapa_shared(bar_tempty + 8u * a, 0));
                else
                    mbar_arrive(bar_tempty + 8u * a);
            }
        }
    } else if constexpr (!kPair) {
        // ---------------------------------------------------------------- a split tile: sums to shared memory (the ring
        // is free: every product that read it is over)
        const int g = (warp - 2) >> 2, q = warp & 3;
        const bool got = mbar_wait(bar_tfull, 0, abort_flag);
        __syncwarp();
        if (__all_sync(0xFFFFFFFFu, got)) {
            tc_fence_after_sync();
            int tf, tt;
            tile_of(team, tf, tt);
            const int valid = min(NT, p.rows - tt * NT);
            float *const sums = reinterpret_cast<float *>(gbase);
            for (int c = g * 16; c < valid; c += 32) {
                float v[16];
                tmem_load16(tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(c), v);
#pragma unroll
                for (int j = 0; j < 16; ++j) sums[(c + j) * kTileF + q * 32 + lane] = v[j];
            }
        }
        tc_fence_before_sync();
    }

    __syncwarp();
    if constexpr (kPair) {
        cluster_sync_all();  // the pair's products, copies and arrivals are over
    } else if (split > 1) {
        cluster_sync_all();  // every CTA's sums are in its shared memory
        if (warp >= 2) {
            // each CTA joins its share of the tile's rows, a warp a row, in the order of the ranks
            int tf, tt;
            tile_of(team, tf, tt);
            const int valid = min(NT, p.rows - tt * NT);
            const RowStore<T, Y> out(p, lane, tf * kTileF);
            uint32_t peer[kMaxSplit];
#pragma unroll
            for (int s = 0; s < kMaxSplit; ++s) peer[s] = s < split ? mapa_shared(base, s) : 0u;
            for (int j = static_cast<int>(rank) + split * (warp - 2); j < valid; j += split * 8) {
                Four<Y> r;
                if (p.residual) out.fetch(tt * NT + j, r);
                float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < kMaxSplit; ++s) {
                    if (s >= split) continue;
                    if (p.vec) {
                        const float4 f = ld_peer(peer[s] + static_cast<uint32_t>(j * kTileF + lane * 4) * 4u);
                        z[0] += f.x, z[1] += f.y, z[2] += f.z, z[3] += f.w;
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float f;
                            asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                         : "=f"(f)
                                         : "r"(peer[s] + static_cast<uint32_t>(j * kTileF + lane + 32 * e) * 4u)
                                         : "memory");
                            z[e] += f;
                        }
                    }
                }
                out.store(tt * NT + j, z, r);
            }
        }
        __syncwarp();
        cluster_sync_all();  // no CTA ends while another reads its sums
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after_sync();
        if constexpr (kPair)
            tmem_dealloc_pair(tmem, tmem_cols);
        else
            tmem_dealloc(tmem, tmem_cols);
    }
}

// How a call is cut: tiles of NT rows, by CTA pairs or by clusters of `split` CTAs.
struct Plan {
    int pair, NT, split, boxes, stages, grid;  // grid: clusters
};

struct Machine {
    int sms = 0, smem = 0;              // SMs, dynamic shared memory of a block
    int pairs = 0;                      // CTA pairs that run at a time
    int clusters[2][kMaxSplit + 1] = {};  // clusters of that many CTAs with all of an SM's shared memory, or half of it, each
};

constexpr int kHalfSmem = 113 * 1024;  // two blocks fit an SM

int smem_of(const Plan &pl)
{
    return static_cast<int>(layout(pl.NT, pl.boxes, pl.stages, pl.pair, pl.split).total) + 1024;  // (alignment)
}

// The ring: as many stages as shared memory holds or the CTA's share of k takes. False if the plan does not fit.
bool fit_stages(Plan &pl, int KB64, const Machine &m)
{
    pl.boxes = 1;
    pl.stages = 0;
    const int fixed = smem_of(pl), stage = static_cast<int>(layout(pl.NT, 1, 1, pl.pair, pl.split).stage);
    int most = (m.smem - fixed) / (stage + 16);
    const int need = (KB64 + pl.split - 1) / pl.split;
    if (most >= 8 && need >= 8) {  // fewer, larger stages: half the barriers
        pl.boxes = 2;
        most /= 2;
    }
    const int KB = (KB64 + pl.boxes - 1) / pl.boxes;
    int use = (KB + pl.split - 1) / pl.split;
    if (use > most) use = most;
    // (a split tile's sums take NT * 512 bytes of the ring)
    while (pl.split > 1 && use * pl.boxes * stage < pl.NT * kTileF * 4) ++use;
    pl.stages = use;
    return use >= 1 && use <= most && KB >= pl.split;
}

Plan choose(int64_t rows, int64_t n, int64_t k, const Machine &m)
{
    const int KB64 = static_cast<int>((k + kBox - 1) / kBox);
    Plan best = {};
    double best_t = 0;
    for (int pair = 0; pair < 2; ++pair) {
        if (pair && (rows <= 64 || m.pairs < 1)) continue;
        const int F = pair ? 2 * kTileF : kTileF;
        const int64_t tf = (n + F - 1) / F;
        for (int split = 1; split <= (pair ? 1 : kMaxSplit); ++split) {
            const int most = static_cast<int>(rows < 256 ? (rows + 15) / 16 * 16 : 256);
            for (int NT = most; NT >= 16; NT -= 16) {
                Plan pl = {pair, NT, split, 1, 0, 0};
                const int64_t items = tf * ((rows + pl.NT - 1) / pl.NT);
                if (!fit_stages(pl, KB64, m)) continue;
                const int slots = pair ? m.pairs : m.clusters[split > 1 && smem_of(pl) <= kHalfSmem][split];
                if (slots < 1 || (split > 1 && items > slots)) continue;
                pl.grid = static_cast<int>(items < slots ? items : slots);
                const double rounds = static_cast<double>((items + slots - 1) / slots);
                // clocks: a 64-column step's products, its loads from L2, everybody's share of HBM
                const double mma = pl.NT, l2 = (kTileF + (pair ? pl.NT / 2 : pl.NT)) * 128 / 100.0;
                const double hbm = (static_cast<double>(n) * k + static_cast<double>(rows) * k) * 2 / 3500.0;
                const double steps = static_cast<double>((KB64 + split - 1) / split) * rounds;
                double t = steps * (mma > l2 ? mma : l2);
                if (hbm > t) t = hbm;
                t += 1500 + pl.NT * 12 + (split > 1 ? 2500 : 0);
                if (best_t == 0 || t < best_t) best = pl, best_t = t;
            }
        }
    }
    return best;
}

// A grid of `teams` clusters of `size` CTAs along x, which may begin while its predecessor on the stream finishes.
cudaLaunchConfig_t config(int teams, int size, int smem, cudaStream_t s, cudaLaunchAttribute (&attr)[2])
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(teams) * size);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(size);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = size > 1 ? 2 : 1;
    return cfg;
}

template <typename T, typename Y>
cudaError_t launch(const Plan &pl, const LinearParams &p, cudaStream_t s)
{
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = config(pl.grid, pl.pair ? 2 : pl.split, smem_of(pl), s, attr);
    return pl.pair ? cudaLaunchKernelEx(&cfg, linear_kernel<true, T, Y>, p) : cudaLaunchKernelEx(&cfg, linear_kernel<false, T, Y>, p);
}

template <typename T, typename Y>
cudaError_t prepare(Machine &m)
{
    cudaLaunchAttribute attr[2];
    cudaError_t e = set_max_dynamic_smem(linear_kernel<true, T, Y>, m.smem);
    if (e == cudaSuccess) e = set_max_dynamic_smem(linear_kernel<false, T, Y>, m.smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = config(1, 2, m.smem, nullptr, attr);
    e = cudaOccupancyMaxActiveClusters(&m.pairs, linear_kernel<true, T, Y>, &cfg);
    if (e != cudaSuccess) return e;
    m.clusters[0][1] = m.sms;
    for (int half = 0; half < 2; ++half)
        for (int size = 2; size <= kMaxSplit; ++size) {
            cfg = config(1, size, half ? kHalfSmem : m.smem, nullptr, attr);
            if (cudaOccupancyMaxActiveClusters(&m.clusters[half][size], linear_kernel<false, T, Y>, &cfg) != cudaSuccess) {
                cudaGetLastError();
                m.clusters[half][size] = 0;  // (such a cluster is not used)
            }
        }
    return cudaSuccess;
}

dflash_status linear_fail(dflash_status st, const char *fmt, long long a = 0, long long b = 0)
{
    char buf[256];
    snprintf(buf, sizeof buf, fmt, a, b);
    return host_fail(st, buf);
}

bool misaligned(const void *p, uintptr_t by)
{
    return reinterpret_cast<uintptr_t>(p) % by != 0;
}

// Whether rows of a (width bytes, stride bytes apart) share bytes with rows of b. Rows of two column slices of one
// buffer do not.
bool overlap(const void *a, int64_t a_rows, int64_t a_stride, int64_t a_width, const void *b, int64_t b_rows,
             int64_t b_stride, int64_t b_width)
{
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    const uintptr_t a1 = a0 + (a_rows - 1) * a_stride + a_width, b1 = b0 + (b_rows - 1) * b_stride + b_width;
    if (a1 <= b0 || b1 <= a0) return false;
    if (a_rows == 1 && b_rows == 1) return true;
    if (a_rows == 1) a_stride = b_stride;
    if (b_rows == 1) b_stride = a_stride;
    if (a_stride != b_stride) return true;
    const int64_t off = static_cast<int64_t>((b0 > a0 ? b0 - a0 : a0 - b0) % a_stride);
    const int64_t d = b0 > a0 || off == 0 ? off : a_stride - off;  // b's rows start d bytes after a's
    return d < a_width || d + b_width > a_stride;
}

}  // namespace
}  // namespace dfl

struct dflash_linear_ctx {
    dflash_linear_config cfg;
    dfl::Machine m;
    int dev = 0;
    const void *W = nullptr, *bias = nullptr;
    CUtensorMap tm_w;
    int *err = nullptr;
};

using dfl::linear_fail;

extern "C" dflash_status dflash_linear_init(const dflash_linear_config *cfg, const void *W, const void *bias, void *stream,
                                            dflash_linear_handle *out)
{
    if (!out) return linear_fail(DFLASH_ERR_INVALID_ARG, "out must not be NULL");
    *out = nullptr;
    if (!cfg || !W) return linear_fail(DFLASH_ERR_INVALID_ARG, "cfg and W must not be NULL");
    if (cfg->n < 1 || cfg->n > (1 << 30) || cfg->k < 1 || cfg->k > (1 << 30))
        return linear_fail(DFLASH_ERR_UNSUPPORTED, "n and k must be in [1, 2^30] (got %lld, %lld)", cfg->n, cfg->k);
    if (cfg->dtype != DFLASH_BF16 && cfg->dtype != DFLASH_FP16)
        return linear_fail(DFLASH_ERR_UNSUPPORTED, "dtype must be BF16 or FP16 (got %lld)", cfg->dtype);
    if (cfg->out_dtype != cfg->dtype && cfg->out_dtype != DFLASH_FP32)
        return linear_fail(DFLASH_ERR_UNSUPPORTED, "out_dtype must be dtype or FP32 (got %lld)", cfg->out_dtype);
    if (cfg->activation < DFLASH_ACT_NONE || cfg->activation > DFLASH_ACT_GELU_TANH)
        return linear_fail(DFLASH_ERR_INVALID_ARG, "no such activation: %lld", cfg->activation);
    if (dfl::misaligned(W, 16) || (cfg->n > 1 && (cfg->w_stride < cfg->k || cfg->w_stride % 8 != 0)))
        return linear_fail(DFLASH_ERR_INVALID_ARG, "W must be 16-byte aligned, its rows a multiple of 8 values and at least k = %lld apart (got %lld)",
                           cfg->k, cfg->w_stride);
    if (dfl::misaligned(bias, 2)) return linear_fail(DFLASH_ERR_INVALID_ARG, "bias must be aligned to its type");
    dflash_linear_ctx *c = new (std::nothrow) dflash_linear_ctx;
    if (!c) return linear_fail(DFLASH_ERR_CUDA, "out of host memory");
    c->cfg = *cfg;
    c->W = W;
    c->bias = bias;
    int major = 0, minor = 0, smem = 0;
    if (cudaGetDevice(&c->dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, c->dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, c->dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&c->m.sms, cudaDevAttrMultiProcessorCount, c->dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&smem, cudaDevAttrMaxSharedMemoryPerBlockOptin, c->dev) != cudaSuccess) {
        delete c;
        return linear_fail(DFLASH_ERR_CUDA, "querying the current device failed");
    }
    if (major != 10 || minor != 3) {
        delete c;
        return linear_fail(DFLASH_ERR_UNSUPPORTED, "built for sm_103 (GB300); device is sm_%lld%lld", major, minor);
    }
    c->m.smem = smem;
    const bool half = cfg->dtype == DFLASH_FP16, wide = cfg->out_dtype == DFLASH_FP32;
    cudaError_t e = half ? (wide ? dfl::prepare<__half, float>(c->m) : dfl::prepare<__half, __half>(c->m))
                         : (wide ? dfl::prepare<__nv_bfloat16, float>(c->m)
                                 : dfl::prepare<__nv_bfloat16, __nv_bfloat16>(c->m));
    dflash_status st = DFLASH_OK;
    if (e == cudaSuccess) {
        st = dfl::host_make_tmap_rows(&c->tm_w, W, cfg->n, cfg->k, cfg->n > 1 ? cfg->w_stride : (cfg->k + 7) / 8 * 8, dfl::kTileF);
        if (st != DFLASH_OK) {
            delete c;
            return st;
        }
        const auto s = static_cast<cudaStream_t>(stream);
        e = cudaMalloc(&c->err, sizeof(int));
        if (e == cudaSuccess) e = cudaMemsetAsync(c->err, 0, sizeof(int), s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        if (c->err) cudaFree(c->err);
        delete c;
        return linear_fail(DFLASH_ERR_CUDA, "setting up the layer failed (error %lld)", e);
    }
    *out = c;
    return DFLASH_OK;
}

extern "C" dflash_status dflash_linear_run(dflash_linear_handle h, const void *x, int64_t x_stride, int64_t rows,
                                           const void *residual, int64_t residual_stride, void *y, int64_t y_stride,
                                           void *stream)
{
    if (!h) return linear_fail(DFLASH_ERR_INVALID_ARG, "handle is NULL");
    if (rows < 0 || rows > (1 << 30)) return linear_fail(DFLASH_ERR_INVALID_ARG, "rows must be in [0, 2^30] (got %lld)", rows);
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return linear_fail(DFLASH_ERR_CUDA, "querying the current device failed");
    if (dev != h->dev)
        return linear_fail(DFLASH_ERR_INVALID_ARG, "the handle belongs to device %lld, the current device is %lld", h->dev, dev);
    if (rows == 0) return DFLASH_OK;
    const int64_t n = h->cfg.n, k = h->cfg.k;
    if (rows == 1) {  // (a single row may carry any stride)
        x_stride = (k + 7) / 8 * 8;
        y_stride = residual_stride = n;
    }
    if (!x || dfl::misaligned(x, 16) || x_stride < k || x_stride % 8 != 0)
        return linear_fail(DFLASH_ERR_INVALID_ARG, "x must be given and 16-byte aligned, its rows a multiple of 8 values and at least k = %lld apart (got %lld)",
                           k, x_stride);
    const int size = h->cfg.out_dtype == DFLASH_FP32 ? 4 : 2;
    if (!y || dfl::misaligned(y, size) || y_stride < n)
        return linear_fail(DFLASH_ERR_INVALID_ARG, "y must be given and aligned to its type, its rows at least n = %lld apart (got %lld)", n, y_stride);
    if (residual && (dfl::misaligned(residual, size) || residual_stride < n))
        return linear_fail(DFLASH_ERR_INVALID_ARG, "residual must be aligned to its type, its rows at least n = %lld apart (got %lld)", n,
                           residual_stride);
    if (dfl::overlap(x, rows, x_stride * 2, k * 2, y, rows, y_stride * size, n * size) ||
        dfl::overlap(h->W, n, h->cfg.w_stride * 2, k * 2, y, rows, y_stride * size, n * size) ||
        (h->bias && dfl::overlap(h->bias, 1, n * 2, n * 2, y, rows, y_stride * size, n * size)) ||
        (residual && (residual != y || residual_stride != y_stride) &&
         dfl::overlap(residual, rows, residual_stride * size, n * size, y, rows, y_stride * size, n * size)))
        return linear_fail(DFLASH_ERR_INVALID_ARG, "y must not overlap x, the weights, or a residual other than y itself");

    const dfl::Plan pl = dfl::choose(rows, n, k, h->m);
    if ((n + 127) / 128 * ((rows + pl.NT - 1) / pl.NT) >= (int64_t(1) << 31))
        return linear_fail(DFLASH_ERR_INVALID_ARG, "too many tiles: %lld rows of %lld values", rows, n);
    if (pl.grid < 1) return linear_fail(DFLASH_ERR_UNSUPPORTED, "no tiling fits this device's shared memory");
    dfl::LinearParams p;
    p.tm_w = h->tm_w;
    dflash_status st = dfl::host_make_tmap_rows(&p.tm_x, x, rows, k, x_stride, pl.pair ? pl.NT / 2 : pl.NT);
    if (st != DFLASH_OK) return st;
    p.bias = h->bias;
    p.residual = residual;
    p.y = y;
    p.residual_stride = residual_stride;
    p.y_stride = y_stride;
    p.rows = static_cast<int>(rows);
    p.n = static_cast<int>(n);
    p.NT = pl.NT;
    p.boxes = pl.boxes;
    p.stages = pl.stages;
    p.KB = static_cast<int>((k + dfl::kBox * pl.boxes - 1) / (dfl::kBox * pl.boxes));
    const int F = pl.pair ? 2 * dfl::kTileF : dfl::kTileF;
    p.tiles_f = static_cast<int>((n + F - 1) / F);
    p.tiles_t = static_cast<int>((rows + pl.NT - 1) / pl.NT);
    p.band = 8;
    p.split = pl.split;
    p.act = h->cfg.activation;
    const uintptr_t four = 4 * size;
    p.vec = !dfl::misaligned(y, four) && (rows == 1 || y_stride % 4 == 0) &&
            (!residual || (!dfl::misaligned(residual, four) && (rows == 1 || residual_stride % 4 == 0)));
    p.err = h->err;
    const auto s = static_cast<cudaStream_t>(stream);
    const bool half = h->cfg.dtype == DFLASH_FP16, wide = size == 4;
    const cudaError_t e = half ? (wide ? dfl::launch<__half, float>(pl, p, s) : dfl::launch<__half, __half>(pl, p, s))
                               : (wide ? dfl::launch<__nv_bfloat16, float>(pl, p, s)
                                       : dfl::launch<__nv_bfloat16, __nv_bfloat16>(pl, p, s));
    if (e != cudaSuccess) {
        cudaGetLastError();
        return linear_fail(DFLASH_ERR_CUDA, "the product's launch failed (error %lld)", e);
    }
    return DFLASH_OK;
}

extern "C" dflash_status dflash_linear_sync_status(dflash_linear_handle h, void *stream)
{
    if (!h) return linear_fail(DFLASH_ERR_INVALID_ARG, "handle is NULL");
    const auto s = static_cast<cudaStream_t>(stream);
    int e = 0;
    if (cudaMemcpyAsync(&e, h->err, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
        return linear_fail(DFLASH_ERR_CUDA, "reading the device error word failed");
    if (e == 0) return DFLASH_OK;
    if (cudaMemsetAsync(h->err, 0, sizeof(int), s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
        return linear_fail(DFLASH_ERR_CUDA, "clearing the device error word failed");
    return linear_fail(DFLASH_ERR_TIMEOUT, "a wait of the matrix product exceeded its time bound (error word %lld)", e);
}

extern "C" dflash_status dflash_linear_destroy(dflash_linear_handle h)
{
    if (!h) return DFLASH_OK;
    int dev = -1;
    cudaGetDevice(&dev);
    if (dev != h->dev) cudaSetDevice(h->dev);
    cudaDeviceSynchronize();
    cudaFree(h->err);
    if (dev >= 0 && dev != h->dev) cudaSetDevice(dev);
    delete h;
    return DFLASH_OK;
}
