// Attention of many rows (chunks of a prompt, long blocks) over a paged cache
// on the tcgen05 tensor cores.
#include <type_traits>

#include "paged.cuh"

namespace dfl {

namespace {

// Warps 0-3 and 4-7 are two softmax streams (a thread per row), warp 8 issues
// the matrix products, warps 9-11 bring keys and values to shared memory.
constexpr int kTileThreads = 384;
constexpr int kLoadWarps = 3;
// Registers: 168 a thread at launch; the streams take 208, the rest keep 88
// (256 * 208 + 128 * 88 = 384 * 168).
constexpr int kStreamRegs = 208, kOtherRegs = 88;

constexpr uint32_t kTmemCols = 512;

template <int D>
struct TileShape {
    static constexpr int BOXES = D / 64;                // 64 values (128 bytes) of 128 rows each
    static constexpr uint32_t BOX = 128 * 128;          // bytes
    static constexpr uint32_t TILE = BOXES * BOX;       // 128 rows of queries, keys or values
    static constexpr int STAGES = D == 128 ? 5 : 10;    // tiles of keys or values in flight
    static constexpr uint32_t SMEM = 2 * TILE + STAGES * TILE + 1024;
    static_assert(SMEM + 2048 <= 227 * 1024, "with the static shared memory, what a block can have");
    static constexpr uint32_t O_COL = 256;              // TMEM: scores 0-127 | 128-255, results from 256
};

struct TileBars {
    uint64_t full[10], empty[10];  // ring of tiles
    uint64_t q_full[2];            // a stream's queries are in shared memory
    uint64_t s_full[2];            // its scores are in TMEM
    uint64_t p_full[2];            // its weights are in TMEM
    uint64_t o_full[2];            // its results are complete
    uint64_t x_given, x_taken;     // joining the two streams of a short item
    uint64_t done;                 // on an abort: products in flight
    uint32_t tmem;
    int abort_flag;
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *tm, int x, int y, int z, int w, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// Adds to the bytes that a barrier's phase waits for (an arrival of its own still has to follow).
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void fence_async_proxy()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// kind::f16 instruction descriptor (fp32 accumulation): bf16 or fp16 operands,
// B with its N dimension contiguous (b_mn) or its K dimension.
template <typename T>
__host__ __device__ constexpr uint32_t idesc_16(int M, int N, bool b_mn)
{
    const uint32_t f = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    return (1u << 4) | (f << 7) | (f << 10) | (static_cast<uint32_t>(b_mn) << 16) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Descriptor of a [128 rows][64 values] x BOXES tile (128-byte swizzle) read
// with the rows as K and the values as N: 8-row groups 1024 bytes apart
// (stride), the next 64 values one box on (leading).
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr, uint32_t box)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(box >> 4) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// D[tmem] (+)= A[tmem] * B[smem], A's rows in the TMEM lanes, two 16-bit K values a column.
__device__ __forceinline__ void umma_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(tmem_d),
        "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
}

#define DFL_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define DFL_W8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])

// 32 consecutive columns of this thread's lane; waits for the load.
__device__ __forceinline__ void tmem_load32(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n"
        : DFL_R8(r, 0), DFL_R8(r, 8), DFL_R8(r, 16), DFL_R8(r, 24)
        : "r"(taddr)
        : "memory");
}

// 128 consecutive columns of this thread's lane.
__device__ __forceinline__ void tmem_load128(uint32_t taddr, uint32_t (&r)[128])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x128.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63, "
        "%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
        "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95, "
        "%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, "
        "%112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%128];\n\t"
        "tcgen05.wait::ld.sync.aligned;\n"
        : DFL_R8(r, 0), DFL_R8(r, 8), DFL_R8(r, 16), DFL_R8(r, 24), DFL_R8(r, 32), DFL_R8(r, 40), DFL_R8(r, 48),
          DFL_R8(r, 56), DFL_R8(r, 64), DFL_R8(r, 72), DFL_R8(r, 80), DFL_R8(r, 88), DFL_R8(r, 96), DFL_R8(r, 104),
          DFL_R8(r, 112), DFL_R8(r, 120)
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_store32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::DFL_W8(r, 0),
        DFL_W8(r, 8), DFL_W8(r, 16), DFL_W8(r, 24), "r"(taddr)
        : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ void tmem_store_wait()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Bounded wait of a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int *abort_flag)
{
    return __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(bar), parity, abort_flag));
}

// The steps of one stream in a piece of n tiles: with rows for both streams
// every tile is a step of both; a short item (`alt`: at most 128 rows) gives
// its even tiles to stream 0 and its odd ones to stream 1, so that both still
// take turns on the tensor cores, and the two results are joined at the end.
__device__ __forceinline__ int stream_steps(int n, bool alt, int i)
{
    return alt ? (n + 1 - i) / 2 : n;
}

}  // namespace

// ---------------------------------------------------------------------------
// One persistent CTA per SM walks its even share of all (sequence, key/value
// head, 256 rows) items' keys in tiles of 128. A tile's scores are one
// 128 x 128 x D product into TMEM per stream; the stream's threads (a row
// each) read them, keep the row's running maximum and sum in registers, and
// write the weights back over the scores as 16-bit values, where they are the
// A operand of the second product, with the values as B straight from their
// [key][value] rows. Both streams share every tile of keys and values; while
// one works on its scores the other's products run, which is what keeps the
// tensor cores busy.
//
// The maximum that the weights are taken against moves only when it grew by
// more than 2^8, and then the stream rescales its result in TMEM itself: its
// previous product is complete when the scores after it are (products of one
// thread finish in order), so no other role takes part.
//
// Keys and values come by TMA in boxes of gcd(page, 128) rows x 64 values
// (128-byte swizzle); a box that reaches past the sequence's end, or lies on a
// page before the window, is written by the load warps, with zeros in the
// place of what must not be read.
// ---------------------------------------------------------------------------
struct TileParams {
    AttendParams a;
    CUtensorMap tm_k, tm_v;  // [pages][heads][slots][values], boxes of 64 values x box_rows slots
    int box_rows;
};

namespace {

template <int D, typename T>
__global__ void __launch_bounds__(kTileThreads, 1) attend_tile_kernel(const __grid_constant__ TileParams tp)
{
    using SH = TileShape<D>;
    constexpr int R = kTileRows, U = kTileUnit, S = SH::STAGES;
    const AttendParams &p = tp.a;
    extern __shared__ uint8_t smem_raw[];
    __shared__ TileBars bars;
    __shared__ float2 x_ml[128];
    uint8_t *const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t q_s = smem_u32(smem), ring = q_s + 2 * SH::TILE;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);

    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(smem_u32(&bars.full[i]), kLoadWarps);
            mbar_init(smem_u32(&bars.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars.q_full[i]), 128);
            mbar_init(smem_u32(&bars.s_full[i]), 1);
            mbar_init(smem_u32(&bars.p_full[i]), 128);
            mbar_init(smem_u32(&bars.o_full[i]), 1);
        }
        mbar_init(smem_u32(&bars.x_given), 128);
        mbar_init(smem_u32(&bars.x_taken), 128);
        mbar_init(smem_u32(&bars.done), 1);
        bars.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(&bars.tmem), kTmemCols);
        tmem_relinquish();
    }
    pdl_trigger();
    pdl_wait();
    tc_fence_before_sync();
    const PagedPlan plan = paged_plan<kTileThreads>(p, R, U, reinterpret_cast<int *>(smem));  // holds block barriers
    tc_fence_after_sync();
    const uint32_t tmem = bars.tmem;
    int *const ab = &bars.abort_flag;
    PagedWalk walk;
    walk.start(p, plan, R, U);

    if (warp < 8) {
        // ------------------------------------------------------ softmax streams
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kStreamRegs));
        const int i = warp >> 2, row = tid & 127;
        const uint32_t lane_base = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lane 32 * (warp % 4)
        const uint32_t s_col = tmem + lane_base + 128u * i, o_col = tmem + lane_base + SH::O_COL + D * i;
        uint32_t s_phase = 0, o_phase = 0, x_phase = 0;
        int4 merge0 = make_int4(0, 0, 0, 0), merge1 = merge0;
        bool ok = true;
        while (ok && walk.left > 0) {
            const PagedPiece &pc = walk.pc;
            const PagedSeq &s = pc.s;
            const int rows = min(R, s.n * p.group - pc.rt * R);
            const bool alt = rows <= 128;
            const int n = pc.e - pc.a, steps = stream_steps(n, alt, i);
            const int r = alt ? row : 128 * i + row;  // row of the item
            const bool real = r < rows;
            const int rr = pc.rt * R + r, tok = p.by_group.div(rr), head = pc.kvh * p.group + rr - tok * p.group;

            // ---- this stream's queries (of a short item, stream 0's serve both)
            if (!(alt && i == 1)) {
                const T *src = static_cast<const T *>(p.q) + (s.t0 + tok) * p.q_ts + head * p.q_hs;
                uint8_t *dst = smem + i * SH::TILE + row * 128;
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 v = real ? *reinterpret_cast<const uint4 *>(src + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4 *>(dst + (c >> 3) * SH::BOX + (((c & 7) ^ (row & 7)) * 16)) = v;
                }
                fence_async_proxy();
                mbar_arrive(smem_u32(&bars.q_full[i]));
            }

            // ---- keys that this row sees: (after, upto]
            const int place = s.len - s.n + tok;
            const int upto = real ? (p.causal ? min(place, s.len - 1) : s.len - 1) : -1;
            const int after = p.window > 0 ? place - p.window : -1;
            const int least_upto = __reduce_min_sync(0xFFFFFFFFu, real ? upto : 0x7FFFFFFF);
            const int most_after = __reduce_max_sync(0xFFFFFFFFu, real ? after : -1);
            const float factor = p.scale_log2;
            float m = -INFINITY, l = 0.f;

            for (int t = 0; t < steps; ++t) {
                const int key0 = (pc.it.u0 + pc.a + (alt ? 2 * t + i : t)) * U;
                if (!(ok = warp_wait(&bars.s_full[i], s_phase, ab))) break;
                s_phase ^= 1;
                tc_fence_after_sync();
                uint32_t sr[128];
                tmem_load128(s_col, sr);
                if (!(key0 > most_after && key0 + U - 1 <= least_upto)) {
                    const int hi = upto - key0, lo = after - key0;
#pragma unroll
                    for (int c = 0; c < 128; ++c)
                        if (c > hi || c <= lo) sr[c] = __float_as_uint(-INFINITY);
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 128; c += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        top[k] = max3(top[k], __uint_as_float(sr[c + 2 * k]), __uint_as_float(sr[c + 2 * k + 1]));
                const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * factor;
                if (t == 0) {
                    m = now;
                } else if (__any_sync(0xFFFFFFFFu, now > m + 8.f)) {
                    const float to = fmaxf(m, now);
                    const float f = to == -INFINITY ? 1.f : ex2(m - to);
                    m = to;
                    l *= f;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32];
                        tmem_load32(o_col + c, o);
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                        tmem_store32(o_col + c, o);
                    }
                    tmem_store_wait();
                }
                // weights, rounded to 16 bits for the product; the sum takes them unrounded
                const float off = m == -INFINITY ? 0.f : m;
                const float2 by = make_float2(factor, factor), less = make_float2(-off, -off);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        float2 x = __ffma2_rn(make_float2(__uint_as_float(sr[64 * h + 2 * c]), __uint_as_float(sr[64 * h + 2 * c + 1])),
                                              by, less);
                        x.x = ex2(x.x);
                        x.y = ex2(x.y);
                        sum[c & 1] = __fadd2_rn(sum[c & 1], x);
                        w[c] = pack2<T>(x.x, x.y);
                    }
                    tmem_store32(s_col + 32 * h, w);
                }
                tmem_store_wait();
                const float2 both = __fadd2_rn(sum[0], sum[1]);
                l += both.x + both.y;
                tc_fence_before_sync();
                mbar_arrive(smem_u32(&bars.p_full[i]));
            }
            if (!ok) break;
            if (steps > 0) {
                if (!(ok = warp_wait(&bars.o_full[i], o_phase, ab))) break;
                o_phase ^= 1;
                tc_fence_after_sync();
            }

            // ---- a short item: stream 1 leaves its result where the queries were, stream 0 adds it to its own
            float *const xbuf = reinterpret_cast<float *>(smem);
            float keep = 1.f, add = 0.f;
            if (alt) {
                if (i == 1) {
                    if (steps > 0) {
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32];
                            tmem_load32(o_col + c, o);
#pragma unroll
                            for (int k = 0; k < 32; k += 4)  // swizzled: a thread's row, conflict-free 16-byte pieces
                                *reinterpret_cast<uint4 *>(xbuf + row * D + (((c + k) / 4) ^ (row & 7)) * 4) =
                                    make_uint4(o[k], o[k + 1], o[k + 2], o[k + 3]);
                        }
                    }
                    x_ml[row] = make_float2(m, l);
                    tc_fence_before_sync();
                    mbar_arrive(smem_u32(&bars.x_given));
                    if (!(ok = warp_wait(&bars.x_taken, x_phase, ab))) break;
                } else {
                    if (!(ok = warp_wait(&bars.x_given, x_phase, ab))) break;
                    const float2 other = x_ml[row];
                    const float to = fmaxf(m, other.x);
                    keep = m == -INFINITY ? 0.f : ex2(m - to);
                    add = other.x == -INFINITY ? 0.f : ex2(other.x - to);
                    m = to;
                    l = l * keep + other.y * add;
                }
                x_phase ^= 1;
            }

            const bool begins = pc.a == 0, split = !begins || pc.e < pc.it.units;
            const int2 share = split ? paged_sharers(plan, walk) : make_int2(0, 1);
            if (!(alt && i == 1)) {
                T *const dst = static_cast<T *>(p.out) + (s.t0 + tok) * p.o_ts + head * p.o_hs;
                float *const part = p.part_o + (paged_slot(share.x, static_cast<int>(blockIdx.x) - share.x) * R + r) * D;
                const bool joined = alt && n > 1;
                auto store = [&](int c, const float(&v)[32]) {  // 32 finished values of the row
#pragma unroll
                    for (int k = 0; k < 32; k += 8)
                        *reinterpret_cast<uint4 *>(dst + c + k) =
                            make_uint4(pack2<T>(v[k], v[k + 1]), pack2<T>(v[k + 2], v[k + 3]), pack2<T>(v[k + 4], v[k + 5]),
                                       pack2<T>(v[k + 6], v[k + 7]));
                };
                auto store_lse = [&](float M, float L) {
                    if (p.lse)
                        p.lse[static_cast<int64_t>(s.t0 + tok) * p.kv_heads * p.group + head] =
                            M == -INFINITY ? -INFINITY : (M + lg2(L)) * 0.69314718055994531f;
                };
                const float inv = split ? 1.f : (l > 0.f || l != l ? p.v_scale / l : 0.f);
                const float f = keep * inv, g = add * inv;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[32];
                    tmem_load32(o_col + c, o);
                    float v[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(o[k]) * f;
                    if (joined) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4) {
                            const float4 x = *reinterpret_cast<const float4 *>(xbuf + row * D + (((c + k) / 4) ^ (row & 7)) * 4);
                            v[k] = fmaf(x.x, g, v[k]);
                            v[k + 1] = fmaf(x.y, g, v[k + 1]);
                            v[k + 2] = fmaf(x.z, g, v[k + 2]);
                            v[k + 3] = fmaf(x.w, g, v[k + 3]);
                        }
                    }
                    if (real && !split) store(c, v);
                    if (real && split) {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            *reinterpret_cast<float4 *>(part + c + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                    }
                }
                tc_fence_before_sync();
                if (alt) mbar_arrive(smem_u32(&bars.x_taken));
                if (real && !split) store_lse(m, l);
                if (real && split) p.part_ml[(part - p.part_o) / D] = make_float2(m, l);
                if (split && share.y <= kTicketParts &&
                    paged_last(p.ticket + share.x * kTicketWarps + warp, share.y, lane) && real) {
                    float2 ml[kTicketParts];
                    float M = -INFINITY, L = 0.f;
#pragma unroll
                    for (int k = 0; k < kTicketParts; ++k) {
                        ml[k] = k < share.y ? __ldcg(p.part_ml + paged_slot(share.x, k) * R + r) : make_float2(-INFINITY, 0.f);
                        M = fmaxf(M, ml[k].x);
                    }
#pragma unroll
                    for (int k = 0; k < kTicketParts; ++k) {
                        ml[k].x = ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - M);
                        L += ml[k].x * ml[k].y;
                    }
                    const float done = L > 0.f || L != L ? p.v_scale / L : 0.f;
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        float v[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = 0.f;
#pragma unroll 1
                        for (int k = 0; k < share.y; ++k) {
                            const float4 *src = reinterpret_cast<const float4 *>(p.part_o + (paged_slot(share.x, k) * R + r) * D + c);
                            const float w = (k == 0 ? ml[0].x : k == 1 ? ml[1].x : k == 2 ? ml[2].x : ml[3].x) * done;
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float4 x = __ldcg(src + e);
                                v[4 * e] = fmaf(x.x, w, v[4 * e]);
                                v[4 * e + 1] = fmaf(x.y, w, v[4 * e + 1]);
                                v[4 * e + 2] = fmaf(x.z, w, v[4 * e + 2]);
                                v[4 * e + 3] = fmaf(x.w, w, v[4 * e + 3]);
                            }
                        }
                        store(c, v);
                    }
                    store_lse(M, L);
                }
                __syncwarp();
            }
            if (begins && share.y > kTicketParts) {  // this CTA's last piece
                merge0 = make_int4(s.t0, pc.rt * R, rows, pc.kvh);
                merge1 = make_int4(share.y, 0, 0, 0);
            }
            walk.next(p, R, U);
        }
        if (tid == 0) {
            p.merge[2 * blockIdx.x] = merge0;
            p.merge[2 * blockIdx.x + 1] = merge1;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 8) {
            // -------------------------------------------------- matrix products
            if (lane == 0) {
                constexpr uint32_t id_s = idesc_16<T>(128, 128, false), id_o = idesc_16<T>(128, D, true);
                // (a descriptor's low bits are the address in units of 16 bytes: stepping it is an addition)
                const uint64_t q_desc = smem_desc_sw128(q_s), k_desc = smem_desc_sw128(ring), v_desc = smem_desc_mn(ring, SH::BOX);
                uint32_t seq = 0, q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
                bool ok = true;
                auto wait = [&](uint64_t *bar, uint32_t parity) {
                    ok = ok && mbar_wait(smem_u32(bar), parity, ab);
                    return ok;
                };
                while (ok && walk.left > 0) {
                    const PagedPiece &pc = walk.pc;
                    const bool alt = pc.s.n * p.group - pc.rt * R <= 128;
                    const int n = pc.e - pc.a;
                    const int steps[2] = {stream_steps(n, alt, 0), stream_steps(n, alt, 1)};
                    // tile j of the piece: keys in stage (seq + 2 j) % S, values in the next
                    auto scores = [&](int i, int t) {
                        const uint32_t k = seq + 2u * (alt ? 2 * t + i : t), st = k % S;
                        if (!wait(&bars.full[st], (k / S) & 1)) return;
                        tc_fence_after_sync();
                        const uint64_t qa = q_desc + (alt ? 0u : i * (SH::TILE >> 4)), ka = k_desc + st * (SH::TILE >> 4);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t o = ((kk >> 2) * SH::BOX + (kk & 3) * 32) >> 4;
                            umma_bf16(tmem + 128u * i, qa + o, ka + o, id_s, kk > 0);
                        }
                        umma_commit(smem_u32(&bars.s_full[i]));
                        if (alt || i == 1) umma_commit(smem_u32(&bars.empty[st]));
                    };
                    auto results = [&](int i, int t) {
                        const uint32_t k = seq + 2u * (alt ? 2 * t + i : t) + 1, st = k % S;
                        if (!wait(&bars.full[st], (k / S) & 1) || !wait(&bars.p_full[i], p_phase[i])) return;
                        p_phase[i] ^= 1;
                        tc_fence_after_sync();
                        const uint64_t va = v_desc + st * (SH::TILE >> 4);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk)
                            umma_ts(tmem + SH::O_COL + D * i, tmem + 128u * i + 8u * kk, va + kk * (2048 >> 4), id_o, t > 0 || kk > 0);
                        if (alt || i == 1) umma_commit(smem_u32(&bars.empty[st]));
                        if (t + 1 == steps[i]) umma_commit(smem_u32(&bars.o_full[i]));
                    };
                    for (int i = 0; i < 2 && ok; ++i) {
                        if (!(alt && i == 1)) {
                            if (!wait(&bars.q_full[i], q_phase[i])) break;
                            q_phase[i] ^= 1;
                        }
                        if (steps[i] > 0) scores(i, 0);
                    }
                    for (int t = 0; t < steps[0] && ok; ++t)
                        for (int i = 0; i < 2 && ok; ++i)
                            if (t < steps[i]) {
                                results(i, t);
                                if (ok && t + 1 < steps[i]) scores(i, t + 1);
                            }
                    seq += 2u * n;
                    walk.next(p, R, U);
                }
                if (!ok) {  // products in flight still write TMEM: see them off before it is freed
                    umma_commit(smem_u32(&bars.done));
                    mbar_wait(smem_u32(&bars.done), 0, ab, false);
                }
            }
            __syncwarp();
        } else {
            // -------------------------------------------------- keys and values
            const int lw = warp - 9, ltid = tid - 9 * 32;
            const int br = tp.box_rows, groups = U / br;  // row groups of a tile: 1, 2, 4 or 8
            uint32_t seq = 0, last_tma = 0;
            bool ok = true, any_tma = false;
            while (ok && walk.left > 0) {
                const PagedPiece &pc = walk.pc;
                const int n = pc.e - pc.a, len = pc.s.len, lo = pc.it.lo, hi = pc.it.hi;
                const int from = p.by_page.div(lo) * p.page;  // the first page that is used
                const int32_t *const pages = p.table + pc.b * p.table_stride;
                // lane g: the page of row group g of a tile (-1: no key of it is used)
                auto page_of = [&](int j) {
                    const int key = (pc.it.u0 + pc.a + j) * U + lane * br;
                    return lane < groups && key >= from && key < hi ? __ldg(pages + p.by_page.div(key)) : -1;
                };
                int ahead = page_of(0);
                for (int j = 0; j < n && ok; ++j) {
                    const int key0 = (pc.it.u0 + pc.a + j) * U, key = key0 + lane * br;
                    int page = ahead;
                    if (j + 1 < n) ahead = page_of(j + 1);
                    if (lane < groups && key >= from && key < hi && (page < 0 || page >= p.num_pages)) {
                        page = -1;
                        atomicOr(p.err, DEV_ERR_PLACE);
                    }
                    const int slot = key - p.by_page.div(key) * p.page;
                    // groups that TMA brings whole, and those that hold places past the end (or no key in use)
                    const unsigned tma = __ballot_sync(0xFFFFFFFFu, page >= 0 && key + br <= len);
                    const int soft = groups - __popc(tma);
#pragma unroll 1
                    for (int kv = 0; kv < 2 && ok; ++kv, ++seq) {
                        const uint32_t st = seq % S, bar = smem_u32(&bars.full[st]);
                        if (!(ok = warp_wait(&bars.empty[st], ((seq / S) & 1) ^ 1, ab))) break;
                        const uint32_t dst = ring + st * SH::TILE;
                        if (lw == 0 && tma) {
                            if (lane == 0) mbar_expect_tx(bar, __popc(tma) * br * SH::BOXES * 128u);
                            __syncwarp();
                            const int g = lane & 7, box = lane >> 3;
                            const int pg = __shfl_sync(0xFFFFFFFFu, page, g), sl = __shfl_sync(0xFFFFFFFFu, slot, g);
                            if (box < SH::BOXES && (tma >> g & 1))
                                tma_load_4d(dst + box * SH::BOX + g * br * 128, kv ? &tp.tm_v : &tp.tm_k, 64 * box, sl, pc.kvh,
                                            pg, bar);
                            any_tma = true;
                            last_tma = seq;
                        }
                        if (soft) {
                            const uint8_t *base = static_cast<const uint8_t *>(kv ? p.v : p.k);
                            constexpr int CH = D / 8;  // 16-byte pieces of a row
                            for (int g = 0; g < groups; ++g) {
                                if (tma >> g & 1) continue;
                                const int pg = __shfl_sync(0xFFFFFFFFu, page, g), sl = __shfl_sync(0xFFFFFFFFu, slot, g);
                                const int64_t at = pg * p.page_stride + sl * p.slot_stride + pc.kvh * p.head_stride;
#pragma unroll 4
                                for (int x = ltid; x < br * CH; x += 32 * kLoadWarps) {
                                    const int row = x / CH, c = x % CH, k = key0 + g * br + row;
                                    const bool in = pg >= 0 && k < len;
                                    const int64_t o = in ? at + row * p.slot_stride + 8 * c : 0;
                                    const int bytes = in ? 16 : 0;  // 0: zeros
                                    const int rw = g * br + row;
                                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                                     dst + (c >> 3) * SH::BOX + rw * 128 + (((c & 7) ^ (rw & 7)) * 16)),
                                                 "l"(base + 2 * o), "r"(bytes)
                                                 : "memory");
                                }
                            }
                            asm volatile("cp.async.wait_all;" ::: "memory");
                            fence_async_proxy();
                            __syncwarp();
                        }
                        if (lane == 0) mbar_arrive(bar);
                    }
                }
                walk.next(p, R, U);
            }
            // On an abort: wait (again with a limit) for the copies in flight. Stages are filled in order, so
            // those of the last S tiles cover them.
            if (!ok && any_tma && lane == 0) {
                const uint32_t first = last_tma >= S - 1 ? last_tma - (S - 1) : 0;
                for (uint32_t q = first; q <= last_tma; ++q)
                    mbar_wait(smem_u32(&bars.full[q % S]), (q / S) & 1, ab, false);
            }
        }
    }
    __syncthreads();
    if (warp == 8) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, kTmemCols);
    }
    if (tid == 0 && bars.abort_flag) atomicOr(p.err, DEV_ERR_TIMEOUT);
}

template <typename F>
cudaError_t tile_variant(int head_dim, int dtype, F &&f)
{
    if (head_dim == 128)
        return dtype == DFLASH_BF16 ? f(attend_tile_kernel<128, __nv_bfloat16>, TileShape<128>::SMEM)
                                    : f(attend_tile_kernel<128, __half>, TileShape<128>::SMEM);
    return dtype == DFLASH_BF16 ? f(attend_tile_kernel<64, __nv_bfloat16>, TileShape<64>::SMEM)
                                : f(attend_tile_kernel<64, __half>, TileShape<64>::SMEM);
}

}  // namespace

cudaError_t prepare_attend_tile(int smem_optin)
{
    for (int d : {64, 128})
        for (int dt : {DFLASH_BF16, DFLASH_FP16}) {
            const cudaError_t e = tile_variant(d, dt, [&](auto kern, size_t) { return set_max_dynamic_smem(kern, smem_optin); });
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}

int tile_box_rows(int page)
{
    int a = page, b = kTileUnit;
    while (b) {
        const int t = a % b;
        a = b;
        b = t;
    }
    return a;
}

cudaError_t launch_attend_tile(const AttendParams &p, const CUtensorMap &tm_k, const CUtensorMap &tm_v, int head_dim,
                               int dtype, int grid, cudaStream_t s)
{
    TileParams tp;
    tp.a = p;
    tp.tm_k = tm_k;
    tp.tm_v = tm_v;
    tp.box_rows = tile_box_rows(p.page);
    return tile_variant(head_dim, dtype, [&](auto kern, size_t smem) {
        return launch_ex(kern, dim3(grid), dim3(kTileThreads), smem, s, 1, tp);
    });
}

}  // namespace dfl
