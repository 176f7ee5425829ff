// Attention of few rows (single tokens and draft blocks) over a paged cache,
// and the merge of split items.
#include <type_traits>

#include "paged.cuh"

namespace dfl {

namespace {

constexpr int kRowsThreads = 128;  // 4 warps
constexpr int rows_cost(int R) { return R <= 16 ? 5 : 8; }  // units that starting an item costs
constexpr int kRowsWarps = kRowsThreads / 32;
// Bytes of a warp's ring: 3 (2) CTAs share an SM with it, and it holds 2 (3) steps of 16 keys of 128 16-bit values.
template <int MT> constexpr int rows_ring() { return MT == 1 ? 16 * 1024 : 24 * 1024; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid)
{
    const int n = valid ? 16 : 0;  // 0: the 16 bytes are filled with zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// A thread's pair (row lane / 4, columns 2 (lane % 4), + 1) of an 8 x 8 matrix -> the same of its transpose.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Shapes of one variant. CH: 16-byte chunks of a key's row; a stage of a
// warp's ring holds 16 keys and their values.
template <int D, int MT, bool FP8>
struct RowsShape {
    static constexpr int ROW = D * (FP8 ? 1 : 2);
    static constexpr int CH = ROW / 16;
    static constexpr int TILE = 16 * ROW;
    static constexpr int STAGE = 2 * TILE;
    static constexpr int STAGES = (rows_ring<MT>() / STAGE < 6) ? rows_ring<MT>() / STAGE : 6;
    // Physical chunk of (row, chunk): 8 rows at one chunk (an ldmatrix phase)
    // and the 16 of a half-row write fall into distinct banks.
    __device__ static uint32_t at(int row, int c)
    {
        const int x = CH >= 8 ? (c ^ (row & 7)) : (c ^ ((row >> 1) & (CH - 1)));
        return static_cast<uint32_t>(row * ROW + x * 16);
    }
    // at(row + n, c) = at(row, c) + n * ROW with this turned in the chunk's bits (n a multiple of 32 / CH > row).
    __device__ static constexpr uint32_t turn(int n) { return CH >= 8 ? (n & 7) * 16 : 0; }
};

__device__ __forceinline__ void add8(float (&acc)[8], float f, const float4 &x, const float4 &y)
{
    acc[0] = fmaf(f, x.x, acc[0]);
    acc[1] = fmaf(f, x.y, acc[1]);
    acc[2] = fmaf(f, x.z, acc[2]);
    acc[3] = fmaf(f, x.w, acc[3]);
    acc[4] = fmaf(f, y.x, acc[4]);
    acc[5] = fmaf(f, y.y, acc[5]);
    acc[6] = fmaf(f, y.z, acc[6]);
    acc[7] = fmaf(f, y.w, acc[7]);
}

template <int D, int MT>
constexpr int rows_q_bytes()
{
    return MT * 16 * D * 2;
}

constexpr int kRowsPad = 8;  // floats between merge rows

// ---------------------------------------------------------------------------
// One CTA walks its even share of all (sequence, key/value head, row tile)
// items' keys. Of every unit of 64 keys warp w takes keys 16 w .. 16 w + 15,
// with its own ring of asynchronous copies, its own running maximum and sum
// and its own accumulator over all R rows: warps meet only at the end of
// a piece, where their four results are joined in shared memory. What a CTA
// does not finish goes to the workspace for the merge kernel.
//
// For every key the rows of a group (query heads that share it, times the
// new tokens) use the same copy in shared memory, so the cache is read once.
// Up to 8 rows are the products' columns (keys or values their rows): half the
// matrix instructions and accumulators that rows of 16 would take.
//
// The floor is HBM: 2 * D * 2 bytes per key against 4 * D * rows operations,
// 32 op/byte at 32 rows, which mma.sync sustains; in tensor memory the queries
// as 128-row tiles would leave 3/4 or more of them empty (keys as the rows and
// queries as the columns would not; that form was not built). What keeps it
// from the floor is the chain of each warp's step (copy wait, scores, weights,
// values) with 8 or 12 warps an SM, and the start of each piece: over an 8-bit
// cache with 32 rows issue slots are 38 %, the tensor pipe 36 % and shared
// memory 34 % busy, and fixed-latency waits lead a warp's stalls. Heads of 128 values,
// 8 of them, a GB300 that copies 6.8 TB/s:
//   128 sequences, 1 token x 4 heads, 200 to 3800 keys   16 bit 154 us 6.6 TB/s, 8 bit 88 us 5.8 TB/s
//   32 sequences, 8 tokens x 4 heads, 500 to 7000 keys   16 bit  98 us 5.4 TB/s, 8 bit 84 us 3.2 TB/s
//   1 sequence, 8 tokens x 4 heads, 2041 keys            13.5 us with the merge, all latency
// Three CTAs an SM where their registers allow it (R <= 16): the first line
// takes 160 and 90 us with two, and 8-bit heads of 64 values 78 us, not 59.
// ---------------------------------------------------------------------------
template <int D, int R, typename QT, bool FP8>
__global__ void __launch_bounds__(kRowsThreads, R <= 16 ? 3 : 2) attend_rows_kernel(const __grid_constant__ AttendParams p)
{
    using CT = typename std::conditional<FP8, __half, QT>::type;  // type of the matrix products
    // Up to 8 rows (NARROW) are the 8 columns of the products, the 16 keys or values their rows; more rows are the
    // products' rows, in MT tiles of 16. NH: rows of a thread's state.
    constexpr bool NARROW = R == 8;
    constexpr int MT = (R + 15) / 16, NH = NARROW ? 2 : R / 8, OT = NARROW ? D / 16 : D / 8;
    constexpr int LANE0 = NARROW ? 4 : 1, LANE1 = NARROW ? 32 : 4;  // lanes that share a row differ in these bits
    using SH = RowsShape<D, MT, FP8>;
    constexpr int kRowsRing = rows_ring<MT>();
    constexpr int S = SH::STAGES, CH = SH::CH;
    constexpr int QCH = D * 2 / 16;  // chunks of a query row
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float q_undo[R];  // FP8: what a query row was scaled by, undone
    __shared__ float2 row_ml[kRowsWarps][R];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t q_s = smem_u32(smem);
    const uint32_t ring = q_s + rows_q_bytes<D, MT>() + warp * kRowsRing;
    uint8_t *const ring_ptr = smem + rows_q_bytes<D, MT>();
    auto q_at = [](int row, int c) { return static_cast<uint32_t>(row * (D * 2) + ((c ^ (row & 7)) * 16)); };

    pdl_trigger();
    pdl_wait();
    constexpr PagedCut cut = {R, kRowsUnit, rows_cost(R)};
    const PagedPlan plan = paged_plan<kRowsThreads>(p, cut, reinterpret_cast<int64_t *>(smem));
    PagedWalk walk;
    walk.start(p, plan, cut);
    int4 merge0 = make_int4(0, 0, 0, 0), merge1 = merge0;
    if (walk.more) {
        for (;;) {
            const PagedPiece &pc = walk.pc;
            const PagedSeq &s = pc.s;
            const int rows = min(R, s.n * p.group - pc.rt * R);  // real rows of this item
            const int base = s.len - s.n;

            // ---- the ring: unit j of the piece, this warp's 16 keys
            const int n_units = pc.e - pc.a, first = pc.it.u0 + pc.a;
            const int lo = pc.it.lo, hi = pc.it.hi;
            const uint8_t *kb = static_cast<const uint8_t *>(p.k);
            const uint8_t *vb = static_cast<const uint8_t *>(p.v);
            constexpr int ES = FP8 ? 1 : 2;
            // a lane copies one 16-byte piece of every RS-th key
            constexpr int RS = 32 / CH;
            const int row0 = lane / CH;
            const uint32_t x0 = SH::at(row0, lane % CH) - row0 * SH::ROW;
            const int64_t lane_off = row0 * p.slot_stride * ES + 16 * (lane % CH), row_step = RS * p.slot_stride * ES;
            int pages = -1;  // lane l: the page of unit pages_from + l
            int pages_from = -(1 << 30);
            auto issue = [&](int j) {
                if (j < n_units) {
                    if (j - pages_from >= 32) {
                        pages_from = j;
                        const int key = (first + j + lane) * kRowsUnit + 16 * warp;
                        pages = -1;
                        if (j + lane < n_units && key < hi && key + 16 > lo) {
                            pages = __ldg(p.table + pc.b * p.table_stride + p.by_page.div(key));
                            if (pages < 0 || pages >= p.num_pages) {
                                pages = -1;
                                atomicOr(p.err, DEV_ERR_PLACE);
                            }
                        }
                    }
                    const int page = __shfl_sync(0xFFFFFFFFu, pages, j - pages_from);
                    const int key = (first + j) * kRowsUnit + 16 * warp;
                    const int slot = key - p.by_page.div(key) * p.page;
                    const int64_t at = (page * p.page_stride + slot * p.slot_stride + pc.kvh * p.head_stride) * ES + lane_off;
                    const uint8_t *ks = kb + at, *vs = vb + at;
                    const uint32_t dst = ring + (j % S) * SH::STAGE + row0 * SH::ROW;
                    if (page >= 0 && key >= lo && key + 16 <= hi) {
#pragma unroll
                        for (int i = 0; i < 16 / RS; ++i, ks += row_step, vs += row_step) {
                            const uint32_t to = dst + i * RS * SH::ROW + (x0 ^ SH::turn(i * RS));
                            cp_async16(to, ks);
                            cp_async16(to + SH::TILE, vs);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16 / RS; ++i, ks += row_step, vs += row_step) {
                            const int k = key + row0 + i * RS;
                            const bool ok = page >= 0 && k >= lo && k < hi;
                            const uint32_t to = dst + i * RS * SH::ROW + (x0 ^ SH::turn(i * RS));
                            cp_async16(to, ok ? ks : kb, ok);
                            cp_async16(to + SH::TILE, ok ? vs : vb, ok);
                        }
                    }
                }
                cp_async_commit();
            };
#pragma unroll
            for (int j = 0; j < S - 1; ++j) issue(j);

            // ---- queries to shared memory, whole 16-byte pieces; rows past the item's are zero
            for (int i = tid; i < R * QCH; i += kRowsThreads) {
                const int r = i / QCH, c = i % QCH;
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (r < rows) {
                    const int rr = pc.rt * R + r, t = p.by_group.div(rr), g = rr - t * p.group;
                    v = *reinterpret_cast<const uint4 *>(static_cast<const QT *>(p.q) +
                                                         (s.t0 + t) * p.q_ts + (pc.kvh * p.group + g) * p.q_hs + 8 * c);
                }
                if constexpr (FP8) {
                    // the products run in fp16: a power of two per row (query_exponent())
                    float f[8];
                    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
                    float top = 0.f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 a = unpack2<QT>(u[k]);
                        f[2 * k] = a.x;
                        f[2 * k + 1] = a.y;
                        top = fmaxf(top, fmaxf(fabsf(a.x), fabsf(a.y)));
                    }
#pragma unroll
                    for (int o = QCH / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                    const int e = query_exponent(top);
                    const float up = __uint_as_float(static_cast<uint32_t>(127 + 8 - e) << 23);
                    if (c == 0) q_undo[r] = __uint_as_float(static_cast<uint32_t>(127 - 8 + e) << 23);
                    // of every 16 values 0, 1, 4, 5, 8, .. are k = 0 .. 7 of the product and the others 8 .. 15 (see the scores)
                    *reinterpret_cast<uint2 *>(smem + q_at(r, c & ~1) + 8 * (c & 1)) =
                        make_uint2(pack2<CT>(f[0] * up, f[1] * up), pack2<CT>(f[4] * up, f[5] * up));
                    *reinterpret_cast<uint2 *>(smem + q_at(r, c | 1) + 8 * (c & 1)) =
                        make_uint2(pack2<CT>(f[2] * up, f[3] * up), pack2<CT>(f[6] * up, f[7] * up));
                } else {
                    *reinterpret_cast<uint4 *>(smem + q_at(r, c)) = v;
                }
            }
            __syncthreads();

            // ---- limits of this thread's rows: keys in (after, upto]
            auto row_of = [&](int i) { return NARROW ? 2 * (lane & 3) + i : 8 * i + (lane >> 2); };
            int upto[NH], after[NH];
            float factor[NH];
            int most_after = -1, least_upto = 0x7FFFFFFF;
#pragma unroll
            for (int i = 0; i < NH; ++i) {
                const int r = row_of(i);
                const int place = base + p.by_group.div(pc.rt * R + r);
                upto[i] = r < rows ? (p.causal ? min(place, s.len - 1) : s.len - 1) : -1;
                after[i] = p.window > 0 ? place - p.window : -1;
                if (r < rows) {
                    least_upto = min(least_upto, upto[i]);
                    most_after = max(most_after, after[i]);
                }
                factor[i] = p.scale_log2 * (FP8 ? q_undo[r] : 1.f);
            }
            least_upto = __reduce_min_sync(0xFFFFFFFFu, least_upto);
            most_after = __reduce_max_sync(0xFFFFFFFFu, most_after);

            uint2 qf[NARROW ? D / 16 : 1];  // up to 8 rows stay in registers
            if constexpr (NARROW) {
#pragma unroll
                for (int c = 0; c < D / 16; ++c)
                    qf[c] = make_uint2(*reinterpret_cast<const uint32_t *>(smem + q_at(lane >> 2, 2 * c) + 4 * (lane & 3)),
                                       *reinterpret_cast<const uint32_t *>(smem + q_at(lane >> 2, 2 * c + 1) + 4 * (lane & 3)));
            }

            float o[MT][OT][4];
            float m[NH], l[NH];
#pragma unroll
            for (int i = 0; i < NH; ++i) {
                m[i] = -INFINITY;
                l[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int n = 0; n < OT; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[i][n][k] = 0.f;

            for (int j = 0; j < n_units; ++j) {
                cp_async_wait<S - 2>();
                __syncwarp();
                issue(j + S - 1);
                const uint32_t ks = ring + (j % S) * SH::STAGE, vs = ks + SH::TILE;
                const int key0 = (first + j) * kRowsUnit + 16 * warp;
                if (key0 >= hi || key0 + 16 <= lo) continue;  // no row sees these keys

                // ---- scores
                float sc[MT][2][4];
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k) sc[i][n][k] = 0.f;
                if constexpr (NARROW) {
                    // sc[0][n][k]: key 8 n + lane / 4, row k; two sums take turns, so that the chain of products is half as long
                    float acc[2][4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[0][k] = acc[1][k] = 0.f;
#pragma unroll
                    for (int c2 = 0; c2 < CH / 2; ++c2) {
                        uint32_t kf[4];  // keys 0-7 and 8-15 of chunk 2 c2, and of chunk 2 c2 + 1
                        ldsm4(ks + SH::at(lane & 15, 2 * c2 + (lane >> 4)), kf);
                        if constexpr (FP8) {
                            // a thread gets 4 consecutive values of a key, which stand for k = 2 j, 2 j + 1,
                            // 2 j + 8, 2 j + 9 of the product (the queries are in the same order)
#pragma unroll
                            for (int hc = 0; hc < 2; ++hc) {
                                uint32_t a[4];
                                e4m3x4_to_h2x2(kf[2 * hc], a[0], a[2]);
                                e4m3x4_to_h2x2(kf[2 * hc + 1], a[1], a[3]);
                                mma16816<CT>(acc[hc], a, qf[2 * c2 + hc].x, qf[2 * c2 + hc].y);
                            }
                        } else {
                            mma16816<CT>(acc[c2 & 1], kf, qf[c2].x, qf[c2].y);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) sc[0][k >> 1][k & 1] = acc[0][k] + acc[1][k];
                } else {
#pragma unroll
                    for (int c2 = 0; c2 < (FP8 ? D / 32 : D / 16); ++c2) {
                        uint32_t kf[4];
                        if constexpr (FP8) {
                            // matrices: keys 0-7 and 8-15 of chunks 2 c2 and 2 c2 + 1. A thread gets 4
                            // consecutive values of a key; they stand for k = 2 j, 2 j + 1, 2 j + 8, 2 j + 9
                            // of the product (the queries below are read in the same order).
                            ldsm4(ks + SH::at((lane & 7) + ((lane >> 3) & 1) * 8, 2 * c2 + (lane >> 4)), kf);
#pragma unroll
                            for (int hc = 0; hc < 2; ++hc) {
                                uint32_t b00, b01, b10, b11;
                                e4m3x4_to_h2x2(kf[2 * hc], b00, b01);
                                e4m3x4_to_h2x2(kf[2 * hc + 1], b10, b11);
#pragma unroll
                                for (int i = 0; i < MT; ++i) {
                                    uint32_t a[4];
                                    ldsm4(q_s + q_at(16 * i + (lane & 15), 2 * (2 * c2 + hc) + (lane >> 4)), a);
                                    mma16816<CT>(sc[i][0], a, b00, b01);
                                    mma16816<CT>(sc[i][1], a, b10, b11);
                                }
                            }
                        } else {
                            ldsm4(ks + SH::at((lane & 7) + (lane >> 4) * 8, 2 * c2 + ((lane >> 3) & 1)), kf);
#pragma unroll
                            for (int i = 0; i < MT; ++i) {
                                uint32_t a[4];
                                ldsm4(q_s + q_at(16 * i + (lane & 15), 2 * c2 + (lane >> 4)), a);
                                mma16816<CT>(sc[i][0], a, kf[0], kf[1]);
                                mma16816<CT>(sc[i][1], a, kf[2], kf[3]);
                            }
                        }
                    }
                }

                // ---- scale, mask, running maximum
                const bool whole = key0 > most_after && key0 + 15 <= least_upto;
                float top[NH];
#pragma unroll
                for (int i = 0; i < NH; ++i) {
                    top[i] = -INFINITY;
#pragma unroll
                    for (int n = 0; n < (NARROW ? 1 : 2); ++n)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float &x = NARROW ? sc[0][k][i] : sc[i >> 1][n][2 * (i & 1) + k];
                            x *= factor[i];
                            if (!whole) {
                                const int key = key0 + (NARROW ? 8 * k + (lane >> 2) : 8 * n + 2 * (lane & 3) + k);
                                if (key > upto[i] || key <= after[i]) x = -INFINITY;
                            }
                            top[i] = fmaxf(top[i], x);
                        }
                }
                // A row's maximum moves only when it grew by more than 2^8 (fp32 sums and the 16-bit
                // weights stand a stale one): the accumulator is then
                // hardly ever rescaled. The first unit sets it.
                bool grew = false;
#pragma unroll
                for (int i = 0; i < NH; ++i) {
#pragma unroll
                    for (int x = LANE0; x < LANE1; x *= 2) top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], x));
                    grew |= top[i] > m[i] + 8.f;
                }
                if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
                    for (int i = 0; i < NH; ++i) {
                        const float now = fmaxf(m[i], top[i]);
                        const float f = now == -INFINITY ? 1.f : ex2(m[i] - now);
                        m[i] = now;
                        l[i] *= f;
#pragma unroll
                        for (int n = 0; n < OT; ++n) {
                            o[NARROW ? 0 : i >> 1][n][NARROW ? i : 2 * (i & 1)] *= f;
                            o[NARROW ? 0 : i >> 1][n][NARROW ? 2 + i : 2 * (i & 1) + 1] *= f;
                        }
                    }
                }

                // ---- weights, rounded to the values' 16-bit type for the product (weight_lift()); the sum takes them unrounded
                uint32_t pf[MT][4];
#pragma unroll
                for (int i = 0; i < NH; ++i) {
                    const float mm = m[i] == -INFINITY ? 0.f : m[i] - weight_lift<CT>();
                    if constexpr (NARROW) {
                        sc[0][0][i] = ex2(sc[0][0][i] - mm);
                        sc[0][1][i] = ex2(sc[0][1][i] - mm);
                        l[i] += sc[0][0][i] + sc[0][1][i];
                    } else {
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const float a = ex2(sc[i >> 1][n][2 * (i & 1)] - mm);
                            const float b = ex2(sc[i >> 1][n][2 * (i & 1) + 1] - mm);
                            l[i] += a + b;
                            pf[i >> 1][2 * n + (i & 1)] = pack2<CT>(a, b);
                        }
                    }
                }
                if constexpr (NARROW) {  // keys by rows -> rows by keys
                    pf[0][0] = transpose8(pack2<CT>(sc[0][0][0], sc[0][0][1]));
                    pf[0][1] = transpose8(pack2<CT>(sc[0][1][0], sc[0][1][1]));
                }

                // ---- values
#pragma unroll
                for (int c = 0; c < CH; c += 2) {
                    uint32_t vf[4];  // keys 0-7 and 8-15 of chunks c and c + 1
                    ldsm4_t(vs + SH::at((lane & 7) + ((lane >> 3) & 1) * 8, c + (lane >> 4)), vf);
                    if constexpr (FP8) {
                        // a thread holds values 2 (lane / 4), + 1 of keys 2 j, 2 j + 1: the even values of a
                        // chunk make one 8-column tile, the odd ones the next
#pragma unroll
                        for (int hc = 0; hc < 2; ++hc) {
                            uint32_t e0, e1, d0, d1;
                            e4m3x4_to_h2x2(__byte_perm(vf[2 * hc], 0, 0x3120), e0, d0);
                            e4m3x4_to_h2x2(__byte_perm(vf[2 * hc + 1], 0, 0x3120), e1, d1);
                            if constexpr (NARROW) {  // rows 0-7 of the product: even values, 8-15: odd ones
                                const uint32_t a[4] = {e0, d0, e1, d1};
                                mma16816<CT>(o[0][c + hc], a, pf[0][0], pf[0][1]);
                            } else {
#pragma unroll
                                for (int i = 0; i < MT; ++i) {
                                    mma16816<CT>(o[i][2 * (c + hc)], pf[i], e0, e1);
                                    mma16816<CT>(o[i][2 * (c + hc) + 1], pf[i], d0, d1);
                                }
                            }
                        }
                    } else if constexpr (NARROW) {
                        const uint32_t a[4] = {vf[0], vf[2], vf[1], vf[3]};
                        mma16816<CT>(o[0][c / 2], a, pf[0][0], pf[0][1]);
                    } else {
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            mma16816<CT>(o[i][c], pf[i], vf[0], vf[1]);
                            mma16816<CT>(o[i][c + 1], pf[i], vf[2], vf[3]);
                        }
                    }
                }
            }

            // ---- join the four warps: each leaves its accumulator in its own ring
            cp_async_wait<0>();
            __syncwarp();
            constexpr int OS = D + kRowsPad;
            float *mine = reinterpret_cast<float *>(ring_ptr + warp * kRowsRing);
#pragma unroll
            for (int i = 0; i < NH; ++i) {
#pragma unroll
                for (int x = LANE0; x < LANE1; x *= 2) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], x);
                const int r = row_of(i);
                if ((lane & (LANE1 - LANE0)) == 0) row_ml[warp][r] = make_float2(m[i] - weight_lift<CT>(), l[i]);
#pragma unroll
                for (int n = 0; n < OT; ++n) {
                    if constexpr (NARROW) {  // o[0][n][k]: value lane / 4 + 8 (k / 2) of 16 (FP8: 2 (lane / 4) + k / 2), row k % 2
                        const int c = lane >> 2;
                        mine[r * OS + 16 * n + (FP8 ? 2 * c : c)] = o[0][n][i];
                        mine[r * OS + 16 * n + (FP8 ? 2 * c + 1 : c + 8)] = o[0][n][2 + i];
                        continue;
                    }
                    const float2 v = make_float2(o[i >> 1][n][2 * (i & 1)], o[i >> 1][n][2 * (i & 1) + 1]);
                    if constexpr (FP8) {  // tile 2 c + h holds values 16 c + 2 col + h
                        mine[r * OS + 16 * (n >> 1) + 4 * (lane & 3) + (n & 1)] = v.x;
                        mine[r * OS + 16 * (n >> 1) + 4 * (lane & 3) + 2 + (n & 1)] = v.y;
                    } else {
                        *reinterpret_cast<float2 *>(mine + r * OS + 8 * n + 2 * (lane & 3)) = v;
                    }
                }
            }
            __syncthreads();
            const bool begins = pc.a == 0, split = walk.split();
            const int2 share = split ? paged_sharers(plan, walk, cut) : make_int2(0, 1);
            const int64_t mine_slot = paged_slot(share.x, plan.cta - share.x);
            auto finish = [&](int r, int c, const float(&acc)[8], float M, float L) {
                const int rr = pc.rt * R + r, t = p.by_group.div(rr), hd = pc.kvh * p.group + rr - t * p.group;
                const float inv = L > 0.f || L != L ? p.v_scale / L : 0.f;
                *reinterpret_cast<uint4 *>(static_cast<QT *>(p.out) + (s.t0 + t) * p.o_ts + hd * p.o_hs + 8 * c) =
                    make_uint4(pack2<QT>(acc[0] * inv, acc[1] * inv), pack2<QT>(acc[2] * inv, acc[3] * inv),
                               pack2<QT>(acc[4] * inv, acc[5] * inv), pack2<QT>(acc[6] * inv, acc[7] * inv));
                if (c == 0 && p.lse)
                    p.lse[static_cast<int64_t>(s.t0 + t) * p.kv_heads * p.group + hd] =
                        row_lse(M, L);
            };
            // a warp always takes the same rows, so the CTAs that share an item join them warp by warp
#pragma unroll
            for (int i = tid; i < R * (D / 8); i += kRowsThreads) {
                const int r = i / (D / 8), c = i % (D / 8);
                float M = -INFINITY, L = 0.f;
#pragma unroll
                for (int w = 0; w < kRowsWarps; ++w) M = fmaxf(M, row_ml[w][r].x);
                float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < kRowsWarps; ++w) {
                    const float2 ml = row_ml[w][r];
                    const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
                    L += f * ml.y;
                    const float4 *src = reinterpret_cast<const float4 *>(
                        reinterpret_cast<const float *>(ring_ptr + w * kRowsRing) + r * OS + 8 * c);
                    add8(acc, f, src[0], src[1]);
                }
                if (r >= rows) continue;
                if (!split) {
                    finish(r, c, acc, M, L);
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(p.part_o + (mine_slot * R + r) * D + 8 * c);
                    dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
                    dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
                    if (c == 0) p.part_ml[mine_slot * R + r] = make_float2(M, L);
                }
            }
            if (split && share.y <= kTicketParts) {
                __syncwarp();
                if (paged_last(p.ticket + share.x * kTicketWarps + warp, share.y, lane))
                    for (int i = tid; i < rows * (D / 8); i += kRowsThreads) {
                        const int r = i / (D / 8), c = i % (D / 8);
                        float2 ml[kTicketParts];
                        float M = -INFINITY, L = 0.f;
#pragma unroll
                        for (int k = 0; k < kTicketParts; ++k) {
                            ml[k] = k < share.y ? __ldcg(p.part_ml + paged_slot(share.x, k) * R + r) : make_float2(-INFINITY, 0.f);
                            M = fmaxf(M, ml[k].x);
                        }
                        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int k = 0; k < kTicketParts; ++k)
                            if (k < share.y) {
                                const float f = ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - M);
                                L += f * ml[k].y;
                                const float4 *src = reinterpret_cast<const float4 *>(
                                    p.part_o + (paged_slot(share.x, k) * R + r) * D + 8 * c);
                                add8(acc, f, __ldcg(src), __ldcg(src + 1));
                            }
                        finish(r, c, acc, M, L);
                    }
            }
            if (begins && share.y > kTicketParts) {  // this CTA's last piece
                merge0 = make_int4(s.t0, pc.rt * R, rows, pc.kvh);
                merge1 = make_int4(share.y, 0, 0, 0);
            }
            if (!walk.next(p, cut)) break;
            __syncthreads();  // the rings and the queries' place are free again
        }
    }
    if (tid == 0) {
        p.merge[2 * plan.cta] = merge0;
        p.merge[2 * plan.cta + 1] = merge1;
    }
}

// Joins the items that were split over more than kTicketParts CTAs. Every
// block reads the whole list (an entry per CTA of the attention launch) and
// takes the listed items' rows in turn, a row at a time: its warps take the
// row's parts in turn, several in flight, and their sums are added in shared
// memory. Which warp adds which parts is fixed, so the result does not depend
// on the order in which anything finished. A call with few rows is all
// latency here: two dependent reads (the list; maxima and parts together), some
// 2.5 us at the end of a call.
// Value d of row r of a part is at r * row_step + d / 4 * value_step + d % 4.
constexpr int kMergeWarps = 8, kMergeMost = 1024;

template <int D, typename QT>
__global__ void __launch_bounds__(kMergeWarps * 32) attend_merge_kernel(const __grid_constant__ AttendParams p, int R, int G, int row_step, int value_step)
{
    constexpr int V = D / 32, AHEAD = 4;  // parts in flight per warp
    using F = typename std::conditional<V == 4, float4, float2>::type;
    __shared__ int4 item_of[kMergeMost];
    __shared__ int c0_of[kMergeMost], parts_of[kMergeMost], warp_n[kMergeWarps];
    __shared__ float sums[kMergeWarps];
    __shared__ __align__(16) float part[kMergeWarps][D];  // (read and written in pieces of F)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (p.merge_early) pdl_trigger();
    pdl_wait();
    if (!p.merge_early) pdl_trigger();
    int entries = 0;
    for (int from = 0; from < G; from += kMergeWarps * 32) {  // the list, without its empty entries
        const int c = from + tid;
        const int n = c < G ? p.merge[2 * c + 1].x : 0;
        const int4 item = c < G ? p.merge[2 * c] : make_int4(0, 0, 0, 0);
        const unsigned m = __ballot_sync(0xFFFFFFFFu, n > 0);
        if (lane == 0) warp_n[warp] = __popc(m);
        __syncthreads();
        int at = entries + __popc(m & ((1u << lane) - 1u));
#pragma unroll
        for (int w = 0; w < kMergeWarps; ++w) {
            if (w < warp) at += warp_n[w];
            entries += warp_n[w];
        }
        if (n > 0) {
            item_of[at] = item;
            c0_of[at] = c;
            parts_of[at] = n;
        }
        __syncthreads();
    }
    for (int64_t k = blockIdx.x; k < static_cast<int64_t>(entries) * R; k += gridDim.x) {
        const int r = static_cast<int>(k / entries), which = static_cast<int>(k - static_cast<int64_t>(r) * entries);
        const int4 item = item_of[which];
        const int c0 = c0_of[which], parts = parts_of[which];
        if (r >= item.z) continue;  // (the whole block)
        // the first parts of this warp are on their way while it finds the row's maximum
        F x[AHEAD];
        float2 ml[AHEAD];
        auto fetch = [&](int i0) {
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) {
                const int i = i0 + a * kMergeWarps;
                const int64_t at = paged_slot(c0, i < parts ? i : 0) * R + r;
                ml[a] = p.part_ml[at];
                x[a] = *reinterpret_cast<const F *>(p.part_o + (at - r) * D + r * row_step + V * lane / 4 * value_step + V * lane % 4);
                if (i >= parts) ml[a] = make_float2(-INFINITY, 0.f);
            }
        };
        fetch(warp);
        float M = -INFINITY;
        for (int i = lane; i < parts; i += 32) M = fmaxf(M, p.part_ml[paged_slot(c0, i) * R + r].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
        float L = 0.f, acc[V];
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = 0.f;
        for (int i0 = warp; i0 < parts; i0 += AHEAD * kMergeWarps) {
            if (i0 != warp) fetch(i0);
#pragma unroll
            for (int a = 0; a < AHEAD; ++a) {
                const float f = ml[a].x == -INFINITY ? 0.f : ex2(ml[a].x - M);
                L = fmaf(f, ml[a].y, L);
                const float *xs = reinterpret_cast<const float *>(&x[a]);
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] = fmaf(f, xs[v], acc[v]);
            }
        }
        F mine;
        float *ms = reinterpret_cast<float *>(&mine);
#pragma unroll
        for (int v = 0; v < V; ++v) ms[v] = acc[v];
        *reinterpret_cast<F *>(&part[warp][V * lane]) = mine;
        if (lane == 0) sums[warp] = L;
        __syncthreads();
        if (2 * tid < D) {
            float total = 0.f, a = 0.f, b = 0.f;
#pragma unroll
            for (int w = 0; w < kMergeWarps; ++w) {
                total += sums[w];
                a += part[w][2 * tid];
                b += part[w][2 * tid + 1];
            }
            const int rr = item.y + r, t = p.by_group.div(rr), hd = item.w * p.group + rr - t * p.group;
            const float inv = total > 0.f || total != total ? p.v_scale / total : 0.f;
            *reinterpret_cast<uint32_t *>(static_cast<QT *>(p.out) + (item.x + t) * p.o_ts + hd * p.o_hs + 2 * tid) =
                pack2<QT>(a * inv, b * inv);
            if (tid == 0 && p.lse)
                p.lse[static_cast<int64_t>(item.x + t) * p.kv_heads * p.group + hd] =
                    row_lse(M, total);
        }
        __syncthreads();
    }
}

template <int D, int R>
constexpr size_t rows_smem()
{
    constexpr int MT = (R + 15) / 16;
    return rows_q_bytes<D, MT>() + kRowsWarps * rows_ring<MT>();
}

// Calls f with the kernel of a variant and its shared memory.
template <typename F>
cudaError_t rows_variant(int head_dim, int dtype, int fp8, int rows, F &&f)
{
    using B = __nv_bfloat16;
    using H = __half;
#define DFL_ROWS(D, R)                                                                                       \
    if (head_dim == D && rows == R) {                                                                        \
        if (dtype == DFLASH_BF16 && !fp8) return f(attend_rows_kernel<D, R, B, false>, rows_smem<D, R>());   \
        if (dtype == DFLASH_BF16) return f(attend_rows_kernel<D, R, B, true>, rows_smem<D, R>());            \
        if (!fp8) return f(attend_rows_kernel<D, R, H, false>, rows_smem<D, R>());                           \
        return f(attend_rows_kernel<D, R, H, true>, rows_smem<D, R>());                                      \
    }
    DFL_ROWS(128, 8)
    DFL_ROWS(128, 16)
    DFL_ROWS(128, 32)
    DFL_ROWS(64, 8)
    DFL_ROWS(64, 16)
    DFL_ROWS(64, 32)
#undef DFL_ROWS
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t prepare_attend_rows(int smem_optin)
{
    for (int d : {64, 128})
        for (int dt : {DFLASH_BF16, DFLASH_FP16})
            for (int fp8 : {0, 1})
                for (int rows : {8, 16, 32}) {
                    const cudaError_t e = rows_variant(d, dt, fp8, rows, [&](auto kern, size_t) {
                        return set_max_dynamic_smem(kern, smem_optin);
                    });
                    if (e != cudaSuccess) return e;
                }
    return cudaSuccess;
}

cudaError_t launch_attend_rows(const AttendParams &p, int head_dim, int dtype, int fp8, int rows, int grid,
                               cudaStream_t s)
{
    return rows_variant(head_dim, dtype, fp8, rows, [&](auto kern, size_t smem) {
        return launch_ex(kern, dim3(grid), dim3(kRowsThreads), smem, s, 1, p);
    });
}

cudaError_t launch_attend_merge(const AttendParams &p, int head_dim, int dtype, int rows, int entries, bool by_value,
                                int grid, cudaStream_t s)
{
    if (entries > kMergeMost) return cudaErrorInvalidValue;
    const dim3 g(grid), b(kMergeWarps * 32);
    const int row_step = by_value ? 4 : head_dim, value_step = by_value ? 4 * rows : 4;
    if (head_dim == 128)
        return dtype == DFLASH_BF16
                   ? launch_ex(attend_merge_kernel<128, __nv_bfloat16>, g, b, 0, s, 1, p, rows, entries, row_step, value_step)
                   : launch_ex(attend_merge_kernel<128, __half>, g, b, 0, s, 1, p, rows, entries, row_step, value_step);
    return dtype == DFLASH_BF16
               ? launch_ex(attend_merge_kernel<64, __nv_bfloat16>, g, b, 0, s, 1, p, rows, entries, row_step, value_step)
               : launch_ex(attend_merge_kernel<64, __half>, g, b, 0, s, 1, p, rows, entries, row_step, value_step);
}

}  // namespace dfl
