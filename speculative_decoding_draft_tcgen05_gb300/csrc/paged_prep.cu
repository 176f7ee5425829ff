// Per-head RMS norm and position rotation of queries and keys, with the keys
// and values written to a paged cache where one is given.
#include <type_traits>

#include "paged.cuh"

namespace dfl {

namespace {

constexpr int kPrepThreads = 128;
constexpr int kPrepUnroll = 4;  // heads in flight per lane group

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
// A warp takes one token and up to kPrepUnroll * (32 / LPH) heads of its
// queries, its keys or its values; LPH = D / 8 lanes hold a head, 8 values (16
// bytes) each. The sum of squares is a shuffle over those lanes, and so is the
// partner of a half-split rotation pair (rotary % 16 = 0 puts it at the same
// place of another lane). A lane's angles do not depend on the head, so its 8
// cosines and sines are read once per warp.
//
// Bound by HBM (each value read and written once, the arithmetic is ~10
// operations a value): every load of the warp is issued before its first use.
// ---------------------------------------------------------------------------
template <int D, typename T>
__global__ void __launch_bounds__(kPrepThreads) prep_kernel(const __grid_constant__ PrepParams p)
{
    constexpr int LPH = D / 8, HPP = 32 / LPH, PER = kPrepUnroll * HPP;
    const int lane = threadIdx.x & 31, sub = lane % LPH, grp = lane / LPH;
    const int cq = (p.q.heads + PER - 1) / PER, ck = (p.k.heads + PER - 1) / PER, cv = (p.v.heads + PER - 1) / PER;
    const int chunks = cq + ck + cv;
    const unsigned id = blockIdx.x * (kPrepThreads / 32) + (threadIdx.x >> 5);
    const unsigned token = id / static_cast<unsigned>(chunks);
    int chunk = static_cast<int>(id - token * chunks);
    pdl_trigger();
    pdl_wait();
    if (token >= static_cast<unsigned>(p.tokens)) return;
    const int t = static_cast<int>(token);
    const int part = chunk < cq ? 0 : (chunk < cq + ck ? 1 : 2);
    const PrepRows &x = part == 0 ? p.q : (part == 1 ? p.k : p.v);
    chunk -= part == 0 ? 0 : (part == 1 ? cq : cq + ck);
    const int h0 = chunk * PER + grp;

    uint4 raw[kPrepUnroll];
    const T *in = static_cast<const T *>(x.in) + t * x.in_ts + 8 * sub;
#pragma unroll
    for (int u = 0; u < kPrepUnroll; ++u) {
        const int h = h0 + u * HPP;
        if (h < x.heads) raw[u] = *reinterpret_cast<const uint4 *>(in + h * x.in_hs);
        else raw[u] = make_uint4(0u, 0u, 0u, 0u);
    }

    // ---- the token's place in the cache and its position
    int place = 0, slot = 0, page = -1;
    bool bad = false;
    if (p.append) {
        const int b = warp_find(p.batch.cu_tokens, p.batch.batch, t, lane);
        if (b >= p.batch.batch) return;  // padding
        const int t0 = __ldg(p.batch.cu_tokens + b), t1 = __ldg(p.batch.cu_tokens + b + 1);
        place = __ldg(p.batch.lens + b) - (t1 - t0) + (t - t0);
        const int col = place / p.page;
        slot = place - col * p.page;
        if (place >= 0 && col < p.batch.table_cols) page = __ldg(p.batch.page_table + b * p.batch.table_stride + col);
        if (page < 0 || page >= p.cache.num_pages) {
            page = -1;
            bad = true;
        }
    }
    float w[8], cs[8], sn[8];
    if (part < 2) {
        if (x.weight) {
            const uint4 r = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(x.weight) + 8 * sub));
            const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 v = unpack2<T>(u[k]);
                w[2 * k] = v.x;
                w[2 * k + 1] = v.y;
            }
        }
        if (8 * sub < p.rotary) {
            int pos = p.positions ? __ldg(p.positions + t) : place;
            if (pos < 0 || pos >= p.positions_n) {
                bad = true;
                pos = min(max(pos, 0), p.positions_n - 1);
            }
            const int half = p.rotary / 2;
            const float *row = p.table + static_cast<int64_t>(pos) * p.rotary;
            if (p.interleaved) {  // value pair k of this lane has angle 4 sub + k
                const float4 c = __ldg(reinterpret_cast<const float4 *>(row + 4 * sub));
                const float4 s = __ldg(reinterpret_cast<const float4 *>(row + half + 4 * sub));
                cs[0] = c.x, cs[1] = c.y, cs[2] = c.z, cs[3] = c.w;
                sn[0] = s.x, sn[1] = s.y, sn[2] = s.z, sn[3] = s.w;
            } else {
                const int a = 8 * sub < half ? 8 * sub : 8 * sub - half;
#pragma unroll
                for (int k = 0; k < 8; k += 4) {
                    const float4 c = __ldg(reinterpret_cast<const float4 *>(row + a + k));
                    const float4 s = __ldg(reinterpret_cast<const float4 *>(row + half + a + k));
                    cs[k] = c.x, cs[k + 1] = c.y, cs[k + 2] = c.z, cs[k + 3] = c.w;
                    sn[k] = s.x, sn[k + 1] = s.y, sn[k + 2] = s.z, sn[k + 3] = s.w;
                }
            }
        }
    }
    if (bad && lane == 0 && p.err) atomicOr(p.err, DEV_ERR_PLACE);

    const bool turn = part < 2 && 8 * sub < p.rotary;
    const bool first = 8 * sub < p.rotary / 2;
    const int hop = p.rotary / 16;  // lanes between the halves
    const int partner = turn && !p.interleaved ? (first ? lane + hop : lane - hop) : lane;
#pragma unroll
    for (int u = 0; u < kPrepUnroll; ++u) {
        const int h = h0 + u * HPP;
        float f[8];
        const uint32_t q[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 v = unpack2<T>(q[k]);
            f[2 * k] = v.x;
            f[2 * k + 1] = v.y;
        }
        if (part < 2) {
            if (x.weight) {
                float ss = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) ss = fmaf(f[k], f[k], ss);
#pragma unroll
                for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
                const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] *= r * w[k];
            }
            if (p.rotary > 0) {
                if (p.interleaved) {
                    if (turn) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float a = f[2 * k], b = f[2 * k + 1];
                            f[2 * k] = a * cs[k] - b * sn[k];
                            f[2 * k + 1] = b * cs[k] + a * sn[k];
                        }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float o = __shfl_sync(0xFFFFFFFFu, f[k], partner);
                        if (turn) f[k] = first ? f[k] * cs[k] - o * sn[k] : f[k] * cs[k] + o * sn[k];
                    }
                }
            }
        }
        if (h >= x.heads) continue;
        if (part == 0 || !p.append) {
            T *dst = static_cast<T *>(x.out) + t * x.out_ts + h * x.out_hs + 8 * sub;
            *reinterpret_cast<uint4 *>(dst) =
                make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
        } else if (page >= 0) {
            const int64_t at = page * p.cache.page_stride + slot * p.cache.slot_stride + h * p.cache.head_stride + 8 * sub;
            void *base = part == 1 ? p.cache.k : p.cache.v;
            if (p.fp8) {
                const float scale = part == 1 ? p.cache.k_scale : p.cache.v_scale;
#pragma unroll
                for (int k = 0; k < 8; ++k) f[k] = __fdiv_rn(f[k], scale);
                *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(base) + at) =
                    make_uint2(f32x2_to_e4m3x2(f[0], f[1]) | f32x2_to_e4m3x2(f[2], f[3]) << 16,
                               f32x2_to_e4m3x2(f[4], f[5]) | f32x2_to_e4m3x2(f[6], f[7]) << 16);
            } else {
                *reinterpret_cast<uint4 *>(static_cast<T *>(base) + at) =
                    make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
            }
        }
    }
}

template <int D, typename T>
cudaError_t go(const PrepParams &p, cudaStream_t s)
{
    constexpr int PER = kPrepUnroll * (32 / (D / 8));
    const int chunks = (p.q.heads + PER - 1) / PER + (p.k.heads + PER - 1) / PER + (p.v.heads + PER - 1) / PER;
    const int64_t warps = static_cast<int64_t>(p.tokens) * chunks;
    const int64_t blocks = (warps + kPrepThreads / 32 - 1) / (kPrepThreads / 32);
    if (warps >= (int64_t(1) << 32) - kPrepThreads) return cudaErrorInvalidConfiguration;  // 32-bit warp numbers
    return launch_ex(prep_kernel<D, T>, dim3(static_cast<unsigned>(blocks)), dim3(kPrepThreads), 0, s, 1, p);
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
