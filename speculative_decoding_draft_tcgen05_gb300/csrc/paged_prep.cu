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
// A block takes up to kPrepTokens tokens. It first finds their places in the
// cache and positions (a chain of dependent small reads, once per block) and
// brings their cosines and sines to shared memory. Then its warps share the
// jobs: 32 / LPH heads of the queries, keys or values (LPH = D / 8 lanes to a
// head, 8 values each) of kPrepJob consecutive tokens, so that a job's
// pointers and weights are set up once for several rows. A lane holds four
// whole rotation pairs, 4 values from each half of the rotated part (or 8
// adjacent ones where pairs are adjacent), so the rotation needs no exchange
// between lanes, and the sum of squares is a shuffle over the head's lanes.
//
// Bound by HBM when the instructions per value stay near ten (each value is
// read and written once); a job's loads are all in flight before the first is
// used.
// ---------------------------------------------------------------------------
constexpr int kPrepThreads = 256, kPrepWarps = kPrepThreads / 32;
constexpr int kPrepTokens = 16;
constexpr int kPrepJob = 4;

template <int D, typename T>
__global__ void __launch_bounds__(kPrepThreads, 3) prep_kernel(const __grid_constant__ PrepParams p, int per_block)
{
    constexpr int LPH = D / 8, HPP = 32 / LPH;
    __shared__ int tok_page[kPrepTokens], tok_slot[kPrepTokens], tok_pos[kPrepTokens];
    __shared__ float4 angles[kPrepTokens * D / 4];  // [token][rotary]: cosines, then sines
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane % LPH, grp = lane / LPH;
    const int pq = (p.q.heads + HPP - 1) / HPP, pk = (p.k.heads + HPP - 1) / HPP, pv = (p.v.heads + HPP - 1) / HPP;
    const int passes = pq + pk + pv, R = p.rotary;
    const int t0 = blockIdx.x * per_block, nt = min(per_block, p.tokens - t0);
    const int jobs = passes * ((nt + kPrepJob - 1) / kPrepJob), stride = kPrepWarps * gridDim.y;
    const int rot_lanes = R / 8;
    pdl_trigger();
    pdl_wait();

    // What the current job is: heads of `part`, tokens k0 .. k0 + kPrepJob - 1.
    int part = 0, h = 0, k0 = 0, oa = 0, ob = 0;
    bool two = false, active = false;
    const PrepRows *x = &p.q;
    uint2 ra[kPrepJob], rb[kPrepJob];
    auto load = [&](int j) {
        if (j >= jobs) return;
        const int g = j / passes, pass = j - g * passes;
        k0 = g * kPrepJob;
        part = pass < pq ? 0 : (pass < pq + pk ? 1 : 2);
        x = part == 0 ? &p.q : (part == 1 ? &p.k : &p.v);
        h = (pass - (part == 0 ? 0 : (part == 1 ? pq : pq + pk))) * HPP + grp;
        active = h < x->heads;
        // Values oa .. oa + 3 and ob .. ob + 3 of a head: pair k of the lane is (f[k], f[4 + k]) where `two`, else
        // (f[2 k], f[2 k + 1]). Lanes past the rotated part share the rest in the same way.
        two = R > 0 && !p.interleaved && part < 2;
        oa = two ? (sub < rot_lanes ? 4 * sub : R + 4 * (sub - rot_lanes)) : 8 * sub;
        ob = two ? (sub < rot_lanes ? R / 2 + 4 * sub : R + (D - R) / 2 + 4 * (sub - rot_lanes)) : 8 * sub + 4;
        const T *src = static_cast<const T *>(x->in) + (t0 + k0) * x->in_ts + h * x->in_hs;
#pragma unroll
        for (int u = 0; u < kPrepJob; ++u, src += x->in_ts) {
            ra[u] = rb[u] = make_uint2(0u, 0u);
            if (active && k0 + u < nt) {
                if (two) {
                    ra[u] = *reinterpret_cast<const uint2 *>(src + oa);
                    rb[u] = *reinterpret_cast<const uint2 *>(src + ob);
                } else {
                    const uint4 v = *reinterpret_cast<const uint4 *>(src + oa);
                    ra[u] = make_uint2(v.x, v.y);
                    rb[u] = make_uint2(v.z, v.w);
                }
            }
        }
    };
    int j = warp + kPrepWarps * blockIdx.y;
    load(j);

    // ---- places, pages and positions
    if (p.append) {
        for (int k = warp; k < nt; k += kPrepWarps) {
            const int t = t0 + k, b = warp_find(p.batch.cu_tokens, p.batch.batch, t, lane);
            int page = -2, slot = 0, place = 0;  // -2: padding
            if (b < p.batch.batch) {
                const int from = __ldg(p.batch.cu_tokens + b), to = __ldg(p.batch.cu_tokens + b + 1);
                place = __ldg(p.batch.lens + b) - (to - from) + (t - from);
                const int col = place / p.page;
                slot = place - col * p.page;
                page = -1;
                if (place >= 0 && col < p.batch.table_cols) page = __ldg(p.batch.page_table + b * p.batch.table_stride + col);
                if (page < 0 || page >= p.cache.num_pages) {
                    page = -1;
                    if (lane == 0) atomicOr(p.err, DEV_ERR_PLACE);
                }
            }
            if (lane == 0) {
                tok_page[k] = page;
                tok_slot[k] = slot;
                tok_pos[k] = page == -2 || !p.positions ? place : __ldg(p.positions + t);
            }
        }
        __syncthreads();
    }
    if (R > 0) {
        for (int i = tid; i < nt * (R / 4); i += kPrepThreads) {
            const int k = i / (R / 4);
            int pos = p.append ? tok_pos[k] : __ldg(p.positions + t0 + k);
            if (pos < 0 || pos >= p.positions_n) {
                if (p.append && tok_page[k] != -2 && i % (R / 4) == 0) atomicOr(p.err, DEV_ERR_PLACE);
                pos = min(max(pos, 0), p.positions_n - 1);
            }
            angles[i] = __ldg(reinterpret_cast<const float4 *>(p.table + static_cast<int64_t>(pos) * R) + i % (R / 4));
        }
        __syncthreads();
    }

    for (; j < jobs; j += stride, load(j)) {
        const bool normed = part < 2 && x->weight, turned = part < 2 && sub < rot_lanes;
        const bool cached = part > 0 && p.append;
        float w[8];
        if (normed) {
            const T *wt = static_cast<const T *>(x->weight);
            const uint2 wa = __ldg(reinterpret_cast<const uint2 *>(wt + oa)), wb = __ldg(reinterpret_cast<const uint2 *>(wt + ob));
            const float2 w0 = unpack2<T>(wa.x), w1 = unpack2<T>(wa.y), w2 = unpack2<T>(wb.x), w3 = unpack2<T>(wb.y);
            w[0] = w0.x, w[1] = w0.y, w[2] = w1.x, w[3] = w1.y, w[4] = w2.x, w[5] = w2.y, w[6] = w3.x, w[7] = w3.y;
        }
        const bool plain = !normed && !(part < 2 && R > 0) && !(cached && p.fp8);  // a copy
        const float4 *ang = angles + k0 * (R / 4) + sub;
        T *dst = static_cast<T *>(x->out) + (t0 + k0) * x->out_ts + h * x->out_hs;
#pragma unroll
        for (int u = 0; u < kPrepJob; ++u, dst += x->out_ts, ang += R / 4) {
            if (k0 + u >= nt) break;
            uint2 ya = ra[u], yb = rb[u];
            float f[8];
            if (!plain) {
                const float2 a0 = unpack2<T>(ya.x), a1 = unpack2<T>(ya.y), b0 = unpack2<T>(yb.x), b1 = unpack2<T>(yb.y);
                f[0] = a0.x, f[1] = a0.y, f[2] = a1.x, f[3] = a1.y, f[4] = b0.x, f[5] = b0.y, f[6] = b1.x, f[7] = b1.y;
                if (normed) {
                    float ss = 0.f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) ss = fmaf(f[k], f[k], ss);
#pragma unroll
                    for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
                    const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
                    for (int k = 0; k < 8; ++k) f[k] = f[k] * r * w[k];
                }
                if (turned) {
                    const float4 c = ang[0], s = ang[R / 8];
                    const float cs[4] = {c.x, c.y, c.z, c.w}, sn[4] = {s.x, s.y, s.z, s.w};
                    if (two) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float a = f[k], b = f[4 + k];
                            f[k] = a * cs[k] - b * sn[k];
                            f[4 + k] = b * cs[k] + a * sn[k];
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float a = f[2 * k], b = f[2 * k + 1];
                            f[2 * k] = a * cs[k] - b * sn[k];
                            f[2 * k + 1] = b * cs[k] + a * sn[k];
                        }
                    }
                }
                ya = make_uint2(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]));
                yb = make_uint2(pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
            }
            if (!active) continue;
            T *to = dst;
            if (cached) {
                const int page = tok_page[k0 + u];
                if (page < 0) continue;
                const int64_t row = page * p.cache.page_stride + tok_slot[k0 + u] * p.cache.slot_stride + h * p.cache.head_stride;
                void *base = part == 1 ? p.cache.k : p.cache.v;
                if (p.fp8) {
                    const float scale = part == 1 ? p.cache.k_scale : p.cache.v_scale;
#pragma unroll
                    for (int k = 0; k < 8; ++k) f[k] = __fdiv_rn(f[k], scale);
                    uint8_t *c = static_cast<uint8_t *>(base) + row;
                    *reinterpret_cast<uint32_t *>(c + oa) = f32x2_to_e4m3x2(f[0], f[1]) | f32x2_to_e4m3x2(f[2], f[3]) << 16;
                    *reinterpret_cast<uint32_t *>(c + ob) = f32x2_to_e4m3x2(f[4], f[5]) | f32x2_to_e4m3x2(f[6], f[7]) << 16;
                    continue;
                }
                to = static_cast<T *>(base) + row;
            } else if (p.append && tok_page[k0 + u] == -2) {
                continue;  // padding
            }
            if (two) {
                *reinterpret_cast<uint2 *>(to + oa) = ya;
                *reinterpret_cast<uint2 *>(to + ob) = yb;
            } else {
                *reinterpret_cast<uint4 *>(to + oa) = make_uint4(ya.x, ya.y, yb.x, yb.y);
            }
        }
    }
}

template <int D, typename T>
cudaError_t go(const PrepParams &p, cudaStream_t s)
{
    // As many tokens a block as fill every SM's three blocks once, up to kPrepTokens (a large batch then shares
    // place and angle reads between a block's warps); a small batch has one token a block, and where blocks are
    // left its jobs are spread over several of them.
    constexpr int HPP = 32 / (D / 8);
    int dev = 0, sms = 1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int slots = 3 * sms, per = (p.tokens + slots - 1) / slots;
    const int per_block = per < kPrepTokens ? per : kPrepTokens, blocks = (p.tokens + per_block - 1) / per_block;
    const int passes = (p.q.heads + HPP - 1) / HPP + (p.k.heads + HPP - 1) / HPP + (p.v.heads + HPP - 1) / HPP;
    const int jobs = passes * ((per_block + kPrepJob - 1) / kPrepJob);
    int y = slots / blocks;
    const int most = (jobs + kPrepWarps - 1) / kPrepWarps;
    y = y < 1 ? 1 : (y > most ? most : y);
    return launch_ex(prep_kernel<D, T>, dim3(blocks, y), dim3(kPrepThreads), 0, s, 1, p, per_block);
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
