// Attention of many rows (chunks of a prompt, long blocks) over a paged cache
// on the tcgen05 tensor cores.
#include <type_traits>

#include "paged.cuh"

namespace dfl {

namespace {

// Warps 0-3 and 4-7 are two softmax streams (a thread per row), warp 8 issues
// the matrix products, and the others bring keys, values and queries to shared
// memory: warps 9-11 for a 16-bit cache; warp 9, and warps 10-15 to convert,
// for an 8-bit one.
constexpr int tile_threads(bool fp8) { return fp8 ? 512 : 384; }
constexpr int load_warps(bool fp8) { return fp8 ? 6 : 3; }  // that queries and finished tiles come from
// Registers: 168 (128) a thread at launch; the streams take 200 (184) and the
// rest keep 104 (72): 256 * 200 + 128 * 104 = 384 * 168, 256 * 184 + 256 * 72 = 512 * 128.
constexpr int stream_regs(bool fp8) { return fp8 ? 184 : 200; }
constexpr int other_regs(bool fp8) { return fp8 ? 72 : 104; }

constexpr uint32_t kTmemCols = 512;
constexpr int kTileCost = 4;  // tiles that starting an item costs

template <int D, bool FP8>
struct TileShape {
    static constexpr int BOXES = D / 64;                // 64 values (128 bytes) of 128 rows each
    static constexpr uint32_t BOX = 128 * 128;          // bytes
    static constexpr uint32_t TILE = BOXES * BOX;       // 128 rows of queries, keys or values
    static constexpr int STAGES = (FP8 ? 3 : 5) * (D == 128 ? 1 : 2);  // tiles of keys or values in flight
    static constexpr int RAWS = FP8 ? 4 : 0;            // and, of an 8-bit cache, tiles as they are stored
    static constexpr uint32_t RAW = 128 * D;
    static constexpr uint32_t SMEM = 2 * TILE + STAGES * TILE + RAWS * RAW + 1024;
    static_assert(SMEM + 2048 <= 227 * 1024, "with the static shared memory, what a block can have");
    static constexpr uint32_t O_COL = 256;              // TMEM: scores 0-127 | 128-255, results from 256
};

template <int STAGES>
struct TileBars {
    uint64_t full[STAGES], empty[STAGES];  // ring of tiles
    uint64_t raw_full[4], raw_empty[4];  // ring of 8-bit tiles
    uint64_t q_full[2];            // a stream's queries are in shared memory
    uint64_t q_empty;              // the piece is done with the queries' place
    uint64_t s_full[2];            // its scores are in TMEM
    uint64_t p_full[2];            // its weights are in TMEM (an arrival per warp)
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

// The products and commits below are issued by the lane that `who` is true
// in, by predicating the instruction alone: the code around it stays
// warp-uniform and its operands in uniform registers (inside a divergent
// branch an issue took about 80 cycles, more than the product itself).
// D[tmem] (+)= A[smem] * B[smem]^T.
__device__ __forceinline__ void umma_ss(uint32_t who, uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc), "r"(who)
        : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem], A's rows in the TMEM lanes, two 16-bit K values a column.
__device__ __forceinline__ void umma_ts(uint32_t who, uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(tmem_d),
        "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(acc), "r"(who)
        : "memory");
}

// Arrives once on `bar` when every product issued so far by this lane is done.
__device__ __forceinline__ void umma_commit_if(uint32_t who, uint64_t *bar)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_u32(bar)),
        "r"(who)
        : "memory");
}

#define DFL_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
// (written before the last operand is read)
#define DFL_E8(r, i) "=&r"(r[i]), "=&r"(r[i + 1]), "=&r"(r[i + 2]), "=&r"(r[i + 3]), "=&r"(r[i + 4]), "=&r"(r[i + 5]), "=&r"(r[i + 6]), "=&r"(r[i + 7])
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

// 128 consecutive columns of this thread's lane; waits for the load (FEW: in
// four instructions, which a kernel of 128 registers a thread at launch needs).
template <bool FEW>
__device__ __forceinline__ void tmem_load128(uint32_t taddr, uint32_t (&r)[128])
{
    if constexpr (!FEW) {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x128.b32 {"
            "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
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
    } else {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
            "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%128];\n\t"
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
            "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%129];\n\t"
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, "
            "%80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95}, [%130];\n\t"
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, "
            "%112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%131];\n\t"
            "tcgen05.wait::ld.sync.aligned;\n"
            : DFL_E8(r, 0), DFL_E8(r, 8), DFL_E8(r, 16), DFL_E8(r, 24), DFL_E8(r, 32), DFL_E8(r, 40), DFL_E8(r, 48),
              DFL_E8(r, 56), DFL_E8(r, 64), DFL_E8(r, 72), DFL_E8(r, 80), DFL_E8(r, 88), DFL_E8(r, 96), DFL_E8(r, 104),
              DFL_E8(r, 112), DFL_E8(r, 120)
            : "r"(taddr), "r"(taddr + 32), "r"(taddr + 64), "r"(taddr + 96)
            : "memory");
    }
}

__device__ __forceinline__ void tmem_store32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::DFL_W8(r, 0),
        DFL_W8(r, 8), DFL_W8(r, 16), DFL_W8(r, 24), "r"(taddr)
        : "memory");
}

// The n lowest bits (n of any size).
__device__ __forceinline__ uint32_t low_bits(int n)
{
    return n <= 0 ? 0u : (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u);
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

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t is;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(is));
    return is != 0;
}

// Bounded wait of a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, int *abort_flag)
{
    return __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(bar), parity, abort_flag));
}

// One arrival of a whole warp, after what its lanes did.
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane)
{
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(bar));
}

// The steps of one stream in a piece of n tiles: with rows for both streams
// every tile is a step of both; a short item (`alt`: at most 128 rows) gives
// its even tiles to stream 0 and its odd ones to stream 1, so that both still
// take turns on the tensor cores, and the two results are joined at the end
// (32 ragged sequences of 64 rows: 106 us, 113 without; one of 40 rows over
// 131,000 keys of an 8-bit cache: 94 us, 101 without; seven windowed chunks,
// whose last row tiles are short: 44 us, 42 without).
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
//
// Bound by the tensor cores for many rows, with the exponentials (one per
// score) close behind; by HBM for few. 2048 tokens x 32 heads of 128 values (8 key/value heads) after 14336:
// 293 us, 1.76 PFLOP/s, called a few times, 326 us, 1.58 PFLOP/s, where the power
// limit holds (a plain product: 1.90 and 1.70), 346 us with an 8-bit cache; 8
// tokens x 40 heads over 131065 keys 93 us, 5.8 TB/s; seven windowed chunks of 300
// to 1100 tokens, 16 heads of 64 values, 44 us, 0.35 PFLOP/s: few, short items
// whose starts and ends are not hidden (of a CTA's cycles 7 % are the plan, 16
// to 24 % waits for a piece's first scores, 17 to 19 % the read-out of results
// and the joins, 50 to 55 % the steps themselves).
// ---------------------------------------------------------------------------
struct TileParams {
    AttendParams a;
    CUtensorMap tm_k, tm_v;  // [pages][heads][slots][values], boxes of box_rows slots
    int box_rows;
};

namespace {

template <int D, typename T, bool FP8>
__global__ void __launch_bounds__(tile_threads(FP8), 1) attend_tile_kernel(const __grid_constant__ TileParams tp)
{
    using SH = TileShape<D, FP8>;
    using CT = typename std::conditional<FP8, __half, T>::type;  // type of the matrix products
    constexpr int R = kTileRows, U = kTileUnit, S = SH::STAGES, kLoadWarps = load_warps(FP8);
    constexpr PagedCut cut = {R, U, kTileCost};
    const AttendParams &p = tp.a;
    extern __shared__ uint8_t smem_raw[];
    __shared__ TileBars<S> bars;
    __shared__ float2 x_ml[128];
    // 8-bit cache: a query row was scaled by 2^(126 - this). Pieces take the two slots in turn, since the streams read a
    // piece's before its first weights, while the queries' place (q_empty) is free once its last scores are there: in a
    // piece of one tile that is earlier, and the next piece's queries may come while the streams still finish the piece
    // before. Two are enough: a slot is written again when the scores of the piece between are complete, and those are
    // issued after the first weights of the piece that read it.
    __shared__ uint8_t q_exp[2][FP8 ? 256 : 1];
    uint8_t *const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t q_s = smem_u32(smem), ring = q_s + 2 * SH::TILE;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);

    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(smem_u32(&bars.full[i]), kLoadWarps);
            mbar_init(smem_u32(&bars.empty[i]), 1);
        }
        for (int i = 0; i < SH::RAWS; ++i) {
            mbar_init(smem_u32(&bars.raw_full[i]), 1);
            mbar_init(smem_u32(&bars.raw_empty[i]), kLoadWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars.q_full[i]), kLoadWarps);
            mbar_init(smem_u32(&bars.s_full[i]), 1);
            mbar_init(smem_u32(&bars.p_full[i]), 4);
            mbar_init(smem_u32(&bars.o_full[i]), 1);
        }
        mbar_init(smem_u32(&bars.q_empty), 1);
        mbar_init(smem_u32(&bars.x_given), 4);
        mbar_init(smem_u32(&bars.x_taken), 4);
        mbar_init(smem_u32(&bars.done), 1);
        bars.abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(&bars.tmem), kTmemCols);
        tmem_relinquish();
    }
    if (tid == 9 * 32) {
        tma_prefetch_desc(&tp.tm_k);
        tma_prefetch_desc(&tp.tm_v);
    }
    pdl_trigger();
    pdl_wait();
    tc_fence_before_sync();
    const PagedPlan plan = paged_plan<tile_threads(FP8)>(p, cut, reinterpret_cast<int64_t *>(smem));  // holds block barriers
    tc_fence_after_sync();
    const uint32_t tmem = bars.tmem;
    int *const ab = &bars.abort_flag;
    PagedWalk walk;
    walk.start(p, plan, cut);

    if (warp < 8) {
        // ------------------------------------------------------ softmax streams
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(stream_regs(FP8)));
        const int i = warp >> 2, row = tid & 127;
        const uint32_t lane_base = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lane 32 * (warp % 4)
        const uint32_t s_col = tmem + lane_base + 128u * i, o_col = tmem + lane_base + SH::O_COL + D * i;
        uint32_t s_phase = 0, o_phase = 0, x_phase = 0, q_slot = 0;
        int4 merge0 = make_int4(0, 0, 0, 0), merge1 = merge0;

        // This thread's row of a piece.
        struct Row {
            int r, tok, head;   // row of the item; row of the call and query head
            int upto, after;    // keys that it sees: (after, upto]
            int key0, steps;    // first key of the piece, steps of this stream
            bool real, alt;     // a row past the item's is not; a short item's tiles alternate
        };
        auto row_of = [&](const PagedPiece &pc) {
            Row c;
            const int rows = min(R, pc.s.n * p.group - pc.rt * R);
            c.alt = rows <= 128;
            c.r = c.alt ? row : 128 * i + row;
            c.real = c.r < rows;
            const int rr = pc.rt * R + c.r, t = p.by_group.div(rr), place = pc.s.len - pc.s.n + t;
            c.tok = pc.s.t0 + t;
            c.head = pc.kvh * p.group + rr - t * p.group;
            c.upto = c.real ? (p.causal ? min(place, pc.s.len - 1) : pc.s.len - 1) : -1;
            c.after = p.window > 0 ? place - p.window : -1;
            c.key0 = (pc.it.u0 + pc.a) * U;
            c.steps = stream_steps(pc.e - pc.a, c.alt, i);
            return c;
        };
        bool ok = true, more = walk.more;
        Row c = {};
        if (more) c = row_of(walk.pc);
        while (more) {
            const int least_upto = __reduce_min_sync(0xFFFFFFFFu, c.real ? c.upto : 0x7FFFFFFF);
            const int most_after = __reduce_max_sync(0xFFFFFFFFu, c.real ? c.after : -1);
            float m = -INFINITY, l = 0.f, factor = p.scale_log2;
            for (int t = 0; t < c.steps; ++t) {
                const int key0 = c.key0 + (c.alt ? 2 * t + i : t) * U;
                if (!(ok = warp_wait(&bars.s_full[i], s_phase, ab))) break;
                s_phase ^= 1;
                tc_fence_after_sync();
                if (FP8 && t == 0) factor *= __uint_as_float((1u + q_exp[q_slot][c.r]) << 23);
                uint32_t sr[128];
                tmem_load128<FP8>(s_col, sr);
                if (!(key0 > most_after && key0 + U - 1 <= least_upto)) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {  // a bit per key of 32
                        const uint32_t seen = low_bits(c.upto + 1 - key0 - 32 * g) & ~low_bits(c.after + 1 - key0 - 32 * g);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (!(seen & (1u << k))) sr[32 * g + k] = __float_as_uint(-INFINITY);
                    }
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < 128; k += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        top[e] = max3(top[e], __uint_as_float(sr[k + 2 * e]), __uint_as_float(sr[k + 2 * e + 1]));
                const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * factor;
                if (t == 0) {
                    m = now;
                } else if (__any_sync(0xFFFFFFFFu, now > m + 8.f)) {
                    const float to = fmaxf(m, now);
                    const float f = to == -INFINITY ? 1.f : ex2(m - to);
                    m = to;
                    l *= f;
#pragma unroll 1
                    for (int k = 0; k < D; k += 32) {
                        uint32_t o[32];
                        tmem_load32(o_col + k, o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_store32(o_col + k, o);
                    }
                    tmem_store_wait();
                }
                // weights, rounded to 16 bits for the product (weight_lift()); the sum takes them unrounded
                const float off = m == -INFINITY ? 0.f : m - weight_lift<CT>();
                const float2 by = make_float2(factor, factor), less = make_float2(-off, -off);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        float2 x = __ffma2_rn(make_float2(__uint_as_float(sr[64 * h + 2 * k]), __uint_as_float(sr[64 * h + 2 * k + 1])),
                                              by, less);
                        x.x = ex2(x.x);
                        x.y = ex2(x.y);
                        sum[k & 1] = __fadd2_rn(sum[k & 1], x);
                        w[k] = pack2<CT>(x.x, x.y);
                    }
                    tmem_store32(s_col + 32 * h, w);
                }
                tmem_store_wait();
                tc_fence_before_sync();
                warp_arrive(&bars.p_full[i], lane);
                const float2 both = __fadd2_rn(sum[0], sum[1]);
                l += both.x + both.y;
            }
            if (!ok) break;
            m -= weight_lift<CT>();

            const Row e = c;
            const bool begins = walk.pc.a == 0, split = walk.split(), joined = e.alt && walk.pc.e - walk.pc.a > 1;
            const int2 share = split ? paged_sharers(plan, walk, cut) : make_int2(0, 1);
            if (begins && share.y > kTicketParts) {  // (the CTA's last piece)
                merge0 = make_int4(walk.pc.s.t0, walk.pc.rt * R, min(R, walk.pc.s.n * p.group - walk.pc.rt * R), walk.pc.kvh);
                merge1 = make_int4(share.y, 0, 0, 0);
            }
            const bool by_ticket = split && share.y <= kTicketParts && !(e.alt && i == 1);
            unsigned *const ticket = p.ticket + share.x * kTicketWarps + warp;
            const unsigned written = by_ticket ? paged_written(ticket, lane) : 0;  // (on its way while the products end)
            more = walk.next(p, cut);
            if (more) c = row_of(walk.pc);
            q_slot ^= 1;
            if (e.steps > 0) {
                if (!(ok = warp_wait(&bars.o_full[i], o_phase, ab))) break;
                o_phase ^= 1;
                tc_fence_after_sync();
            }

            // ---- a short item: stream 1 leaves its result where the queries were, stream 0 adds it to its own
            float *const xbuf = reinterpret_cast<float *>(smem);
            float keep = 1.f, add = 0.f;
            if (e.alt) {
                if (i == 1) {
                    if (e.steps > 0) {
#pragma unroll 1
                        for (int k = 0; k < D; k += 32) {
                            uint32_t o[32];
                            tmem_load32(o_col + k, o);
#pragma unroll
                            for (int b = 0; b < 32; b += 4)  // swizzled: a thread's row, conflict-free 16-byte pieces
                                *reinterpret_cast<uint4 *>(xbuf + row * D + (((k + b) / 4) ^ (row & 7)) * 4) =
                                    make_uint4(o[b], o[b + 1], o[b + 2], o[b + 3]);
                        }
                    }
                    x_ml[row] = make_float2(m, l);
                    tc_fence_before_sync();
                    warp_arrive(&bars.x_given, lane);
                } else {
                    if (!(ok = warp_wait(&bars.x_given, x_phase, ab))) break;
                    const float2 other = x_ml[row];
                    const float to = fmaxf(m, other.x);
                    keep = m == -INFINITY ? 0.f : ex2(m - to);
                    add = other.x == -INFINITY ? 0.f : ex2(other.x - to);
                    m = to;
                    l = l * keep + other.y * add;
                }
            }

            if (!(e.alt && i == 1)) {
                T *const dst = static_cast<T *>(p.out) + e.tok * p.o_ts + e.head * p.o_hs;
                const int mine = plan.cta - share.x;  // this CTA's part of a split item
                auto own = [&](int k, float (&v)[32]) {  // 32 values of this row's result
                    uint32_t o[32];
                    tmem_load32(o_col + k, o);
#pragma unroll
                    for (int b = 0; b < 32; ++b) v[b] = __uint_as_float(o[b]) * keep;
                    if (joined) {
#pragma unroll
                        for (int b = 0; b < 32; b += 4) {
                            const float4 x = *reinterpret_cast<const float4 *>(xbuf + row * D + (((k + b) / 4) ^ (row & 7)) * 4);
                            v[b] = fmaf(x.x, add, v[b]);
                            v[b + 1] = fmaf(x.y, add, v[b + 1]);
                            v[b + 2] = fmaf(x.z, add, v[b + 2]);
                            v[b + 3] = fmaf(x.w, add, v[b + 3]);
                        }
                    }
                };
                auto store = [&](int k, const float (&v)[32], float by) {
                    if (e.real) {
#pragma unroll
                        for (int b = 0; b < 32; b += 8)
                            *reinterpret_cast<uint4 *>(dst + k + b) =
                                make_uint4(pack2<T>(v[b] * by, v[b + 1] * by), pack2<T>(v[b + 2] * by, v[b + 3] * by),
                                           pack2<T>(v[b + 4] * by, v[b + 5] * by), pack2<T>(v[b + 6] * by, v[b + 7] * by));
                    }
                };
                auto store_lse = [&](float M, float L) {
                    if (e.real && p.lse)
                        p.lse[static_cast<int64_t>(e.tok) * p.kv_heads * p.group + e.head] =
                            row_lse(M, L);
                };
                // Parts are laid out [value / 4][row]: a warp's rows are adjacent, so its accesses are whole lines.
                auto part_at = [&](int64_t slot, int k) {
                    return reinterpret_cast<float4 *>(p.part_o) + (slot * (D / 4) + k / 4) * R + e.r;
                };
                bool last = false;
                if (!split) {
                    const float inv = l > 0.f || l != l ? p.v_scale / l : 0.f;
#pragma unroll 1
                    for (int k = 0; k < D; k += 32) {
                        float v[32];
                        own(k, v);
                        store(k, v, inv);
                    }
                    store_lse(m, l);
                } else {
                    // the last to finish need not write its part down
                    if (by_ticket) last = paged_all_others(ticket, written, share.y, lane);
                    if (!last) {
                        const int64_t slot = paged_slot(share.x, mine);
#pragma unroll 1
                        for (int k = 0; k < D; k += 32) {
                            float v[32];
                            own(k, v);
                            if (e.real) {
#pragma unroll
                                for (int b = 0; b < 32; b += 4)
                                    *part_at(slot, k + b) = make_float4(v[b], v[b + 1], v[b + 2], v[b + 3]);
                            }
                        }
                        if (e.real) p.part_ml[slot * R + e.r] = make_float2(m, l);
                        if (by_ticket) last = paged_last(ticket, share.y, lane);
                    }
                }
                if (last) {  // joins the parts, in their order whoever does it
                    float2 ml[kTicketParts];
                    float M = -INFINITY, L = 0.f;
#pragma unroll
                    for (int k = 0; k < kTicketParts; ++k) {
                        ml[k] = make_float2(-INFINITY, 0.f);
                        if (k == mine) ml[k] = make_float2(m, l);
                        else if (k < share.y && e.real) ml[k] = __ldcg(p.part_ml + paged_slot(share.x, k) * R + e.r);
                        M = fmaxf(M, ml[k].x);
                    }
#pragma unroll
                    for (int k = 0; k < kTicketParts; ++k) {
                        ml[k].x = ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - M);
                        L = fmaf(ml[k].x, ml[k].y, L);
                    }
                    const float inv = L > 0.f || L != L ? p.v_scale / L : 0.f;
#pragma unroll 1
                    for (int k = 0; k < D; k += 32) {
                        float v[32], x[32];
#pragma unroll
                        for (int b = 0; b < 32; ++b) v[b] = 0.f;
#pragma unroll 1
                        for (int part = 0; part < share.y; ++part) {
                            float w = 0.f;
#pragma unroll
                            for (int b = 0; b < kTicketParts; ++b)
                                if (b == part) w = ml[b].x;
                            if (part == mine) {
                                own(k, x);
                            } else {
                                const int64_t slot = paged_slot(share.x, part);
#pragma unroll
                                for (int b = 0; b < 8; ++b) {
                                    const float4 y = e.real ? __ldcg(part_at(slot, k + 4 * b)) : make_float4(0.f, 0.f, 0.f, 0.f);
                                    x[4 * b] = y.x, x[4 * b + 1] = y.y, x[4 * b + 2] = y.z, x[4 * b + 3] = y.w;
                                }
                            }
#pragma unroll
                            for (int b = 0; b < 32; ++b) v[b] = fmaf(x[b], w, v[b]);
                        }
                        store(k, v, inv);
                    }
                    store_lse(M, L);
                }
                tc_fence_before_sync();
            }
            if (e.alt) {
                if (i == 0) warp_arrive(&bars.x_taken, lane);
                if (!(ok = warp_wait(&bars.x_taken, x_phase, ab))) break;
                x_phase ^= 1;
                if (tid == 0) mbar_arrive(smem_u32(&bars.q_empty));
            }
        }
        if (tid == 0) {
            p.merge[2 * plan.cta] = merge0;
            p.merge[2 * plan.cta + 1] = merge1;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(other_regs(FP8)));
        if (warp == 8) {
            // -------------------------------------------------- matrix products
            // (the whole warp runs this role, one lane issues)
            const uint32_t who = elect_one();
            constexpr uint32_t id_s = idesc_16<CT>(128, 128, false), id_o = idesc_16<CT>(128, D, true);
            // a descriptor's low bits are the address in units of 16 bytes: stepping it is an addition
            const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
            const uint64_t q_desc = smem_desc_sw128(q_s), k_desc = smem_desc_sw128(ring), v_desc = smem_desc_mn(ring, SH::BOX);
            uint32_t seq = 0, q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
            bool ok = true;
            while (ok && walk.more) {
                const PagedPiece &pc = walk.pc;
                const bool alt = pc.s.n * p.group - pc.rt * R <= 128;
                const int n = pc.e - pc.a;
                const int steps[2] = {stream_steps(n, alt, 0), stream_steps(n, alt, 1)};
                // tile j of the piece: keys in stage (seq + 2 j) % S, values in the next. Where both streams use a
                // tile, stream 0 waits for it and stream 1 releases it.
                auto scores = [&](int i, int t) {
                    const uint32_t k = seq + 2u * (alt ? 2 * t + i : t), st = __shfl_sync(0xFFFFFFFFu, k % S, 0);
                    if (alt || i == 0) {
                        ok = warp_wait(&bars.full[st], (k / S) & 1, ab);
                        if (!ok) return;
                        tc_fence_after_sync();
                    }
                    const uint64_t qa = q_desc + (alt ? 0u : i * (SH::TILE >> 4)), ka = k_desc + st * (SH::TILE >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t o = ((kk >> 2) * SH::BOX + (kk & 3) * 32) >> 4;
                        umma_ss(who, tm + 128u * i, qa + o, ka + o, id_s, kk > 0);
                    }
                    umma_commit_if(who, &bars.s_full[i]);
                    if (alt || i == 1) umma_commit_if(who, &bars.empty[st]);
                    if (!alt && i == 1 && t + 1 == steps[1]) umma_commit_if(who, &bars.q_empty);
                };
                auto results = [&](int i, int t) {
                    const uint32_t k = seq + 2u * (alt ? 2 * t + i : t) + 1, st = __shfl_sync(0xFFFFFFFFu, k % S, 0);
                    if (alt || i == 0) ok = warp_wait(&bars.full[st], (k / S) & 1, ab);
                    ok = ok && warp_wait(&bars.p_full[i], p_phase[i], ab);
                    if (!ok) return;
                    p_phase[i] ^= 1;
                    tc_fence_after_sync();
                    const uint64_t va = v_desc + st * (SH::TILE >> 4);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        umma_ts(who, tm + SH::O_COL + D * i, tm + 128u * i + 8u * kk, va + kk * (2048 >> 4), id_o, t > 0 || kk > 0);
                    if (alt || i == 1) umma_commit_if(who, &bars.empty[st]);
                    if (t + 1 == steps[i]) umma_commit_if(who, &bars.o_full[i]);
                };
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (ok && !(alt && i == 1)) {
                        ok = warp_wait(&bars.q_full[i], q_phase[i], ab);
                        q_phase[i] ^= 1;
                        tc_fence_after_sync();
                    }
                    if (ok && steps[i] > 0) scores(i, 0);
                }
                for (int t = 0; t < steps[0] && ok; ++t)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (ok && t < steps[i]) {
                            results(i, t);
                            if (ok && t + 1 < steps[i]) scores(i, t + 1);
                        }
                seq += 2u * n;
                walk.next(p, cut);
            }
            if (!ok) {  // products in flight still write TMEM: see them off before it is freed
                umma_commit_if(who, &bars.done);
                mbar_wait(smem_u32(&bars.done), 0, ab, false);
            }
            __syncwarp();
        } else {
            // -------------------------------------------------- keys and values
            constexpr int kFirst = FP8 ? 10 : 9;            // of the warps that queries come from
            const int ltid = tid - 32 * kFirst;             // (negative: warp 9 of an 8-bit cache's)
            const int br = tp.box_rows, groups = U / br;  // row groups of a tile: 1, 2, 4 or 8
            uint32_t seq = 0, last_tma = 0, q_phase = 1;  // (last_tma: number of the tile)
            bool ok = true, any_tma = false;
            // The piece's queries, once the one before is done with their place; rows past the item's are zero.
            auto load_q = [&](const PagedPiece &pc) {
                if (!(ok = warp_wait(&bars.q_empty, q_phase, ab))) return;
                q_phase ^= 1;  // (from 1: the first piece's slot of q_exp is 0)
                const int r0 = pc.rt * R, rows = min(R, pc.s.n * p.group - r0);
                constexpr int kQPieces = (128 * (D / 8) + 32 * kLoadWarps - 1) / (32 * kLoadWarps) * (32 * kLoadWarps);
                constexpr int CH = D / 8;  // 16-byte pieces of a row
                const int tiles = rows <= 128 ? 1 : 2;
                auto place = [&](int i, int row, int c) {
                    return i * SH::TILE + (c >> 3) * SH::BOX + row * 128 + (((c & 7) ^ (row & 7)) * 16);
                };
                for (int i = 0; i < tiles; ++i) {
#pragma unroll(FP8 ? 4 : 8)
                    for (int x = ltid; x < 128 * CH; x += 32 * kLoadWarps) {
                        const int row = x / CH, c = x % CH, r = 128 * i + row;
                        const int t = p.by_group.div(r0 + r), g = r0 + r - t * p.group;
                        const T *src = static_cast<const T *>(p.q) +
                                       (r < rows ? (pc.s.t0 + t) * p.q_ts + (pc.kvh * p.group + g) * p.q_hs + 8 * c : 0);
                        const int bytes = r < rows ? 16 : 0;  // 0: zeros
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(q_s + place(i, row, c)), "l"(src), "r"(bytes)
                                     : "memory");
                    }
                    if constexpr (!FP8) {
                        asm volatile("cp.async.wait_all;" ::: "memory");
                        fence_async_proxy();
                        warp_arrive(&bars.q_full[i], lane);
                    }
                }
                if constexpr (FP8) {
                    // In their place, by the thread that copied them: to fp16 with a power of two per row
                    // (query_exponent(); a row's lanes are neighbours).
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    for (int i = 0; i < tiles; ++i) {
#pragma unroll 2
                        for (int x = ltid; x < kQPieces; x += 32 * kLoadWarps) {
                            const int row = x / CH, c = x % CH;
                            uint4 *const at = reinterpret_cast<uint4 *>(smem + place(i, min(row, 127), c));
                            const uint4 v = *at;
                            const float2 f[4] = {unpack2<T>(v.x), unpack2<T>(v.y), unpack2<T>(v.z), unpack2<T>(v.w)};
                            float top = 0.f;
#pragma unroll
                            for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(f[e].x), fabsf(f[e].y)));
#pragma unroll
                            for (int o = CH / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                            const int e = query_exponent(top);
                            const float up = __uint_as_float(static_cast<uint32_t>(127 + 8 - e) << 23);
                            if (row < 128) {
                                *at = make_uint4(pack2<CT>(f[0].x * up, f[0].y * up), pack2<CT>(f[1].x * up, f[1].y * up),
                                                 pack2<CT>(f[2].x * up, f[2].y * up), pack2<CT>(f[3].x * up, f[3].y * up));
                                if (c == 0) q_exp[q_phase][128 * i + row] = static_cast<uint8_t>(e + 118);
                            }
                        }
                        fence_async_proxy();
                        warp_arrive(&bars.q_full[i], lane);
                    }
                }
            };
            // One tile of keys or values of `w`'s piece on its way to `dst` (16-bit: swizzled boxes; 8-bit: rows as
            // they are stored): boxes by TMA, and by the load warps those that hold places past the sequence's end
            // or no key in use. Each arrives on `full`, the first of them with the boxes' bytes too.
            struct Source {
                PagedWalk w;
                int j, page, coming;  // tile; lane g: page of its row group g, and of the next tile's
            };
            // lane g: the page of row group g of tile j (kUnused: no key of it is used)
            constexpr int kUnused = -0x7FFFFFFF - 1;
            auto page_of = [&](const PagedWalk &w, int j) {
                const int key = (w.pc.it.u0 + w.pc.a + j) * U + lane * br;
                return lane < groups && key >= p.by_page.div(w.pc.it.lo) * p.page && key < w.pc.it.hi
                           ? __ldg(p.table + w.pc.b * p.table_stride + p.by_page.div(key)) : kUnused;
            };
            auto bring = [&](Source &f, int kv, uint32_t dst, uint64_t *full, uint32_t number) {
                const uint32_t bar = smem_u32(full);
                const PagedPiece &pc = f.w.pc;
                const int key0 = (pc.it.u0 + pc.a + f.j) * U, key = key0 + lane * br, len = pc.s.len;
                if (kv == 0) {  // the values' pages are the keys'
                    f.page = f.coming;
                    if (f.j + 1 < pc.e - pc.a) f.coming = page_of(f.w, f.j + 1);
                    if (f.page != kUnused && (f.page < 0 || f.page >= p.num_pages)) {
                        f.page = -1;
                        atomicOr(p.err, DEV_ERR_PLACE);
                    }
                }
                const int slot = key - p.by_page.div(key) * p.page;
                const unsigned tma = __ballot_sync(0xFFFFFFFFu, f.page >= 0 && key + br <= len);
                constexpr int BOXES = FP8 ? 1 : SH::BOXES, ROW = FP8 ? D : 128;  // boxes of a row group; bytes of a box's row
                if (warp == 9 && tma) {
                    if (lane == 0) mbar_expect_tx(bar, __popc(tma) * br * BOXES * ROW);
                    __syncwarp();
                    const int g = lane & 7, box = lane >> 3;
                    const int pg = __shfl_sync(0xFFFFFFFFu, f.page, g), sl = __shfl_sync(0xFFFFFFFFu, slot, g);
                    if (box < BOXES && (tma >> g & 1))
                        tma_load_4d(dst + box * SH::BOX + g * br * ROW, kv ? &tp.tm_v : &tp.tm_k, 64 * box, sl, pc.kvh, pg, bar);
                    any_tma = true;
                    last_tma = number;
                }
                if (__popc(tma) < groups) {
                    const uint8_t *base = static_cast<const uint8_t *>(kv ? p.v : p.k);
                    constexpr int ES = FP8 ? 1 : 2, CH = D * ES / 16;  // 16-byte pieces of a row
                    for (int g = 0; g < groups; ++g) {
                        if (tma >> g & 1) continue;
                        const int pg = __shfl_sync(0xFFFFFFFFu, f.page, g), sl = __shfl_sync(0xFFFFFFFFu, slot, g);
                        const int64_t at = pg * p.page_stride + sl * p.slot_stride + pc.kvh * p.head_stride;
#pragma unroll(FP8 ? 2 : 4)
                        for (int x = FP8 ? lane : ltid; x < br * CH; x += FP8 ? 32 : 32 * kLoadWarps) {
                            const int row = x / CH, c = x % CH, rw = g * br + row;
                            const bool in = pg >= 0 && key0 + rw < len;
                            const int64_t o = in ? (at + row * p.slot_stride) * ES + 16 * c : 0;
                            const int bytes = in ? 16 : 0;  // 0: zeros
                            const uint32_t to = FP8 ? rw * D + 16 * c : (c >> 3) * SH::BOX + rw * 128 + (((c & 7) ^ (rw & 7)) * 16);
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + to), "l"(base + o), "r"(bytes)
                                         : "memory");
                        }
                    }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    if (!FP8) fence_async_proxy();
                }
                warp_arrive(full, lane);
            };

            if constexpr (!FP8) {
                Source f = {walk, 0, kUnused, walk.more ? page_of(walk, 0) : kUnused};
                while (ok && f.w.more) {
                    const int n = f.w.pc.e - f.w.pc.a;
                    for (f.j = 0; f.j < n && ok; ++f.j) {
#pragma unroll 1
                        for (int kv = 0; kv < 2 && ok; ++kv, ++seq) {
                            const uint32_t st = seq % S;
                            if (!(ok = warp_wait(&bars.empty[st], ((seq / S) & 1) ^ 1, ab))) break;
                            bring(f, kv, ring + st * SH::TILE, &bars.full[st], seq);
                        }
                        // (after the first keys and values: those find room in the ring while the piece before ends,
                        // which the queries have to wait for)
                        if (ok && f.j == 0) load_q(f.w.pc);
                    }
                    if (f.w.next(p, cut)) f.coming = page_of(f.w, 0);
                }
            } else {
                // An 8-bit cache: warp 9 brings tiles as they are stored, the others convert them (exactly) to fp16.
                const uint32_t raw_s = ring + S * SH::TILE;
                if (warp == 9) {
                    Source f = {walk, 0, kUnused, walk.more ? page_of(walk, 0) : kUnused};
                    while (ok && f.w.more) {
                        const int n = f.w.pc.e - f.w.pc.a;
                        for (f.j = 0; f.j < n && ok; ++f.j) {
#pragma unroll 1
                            for (int kv = 0; kv < 2 && ok; ++kv, ++seq) {
                                const uint32_t rs = seq % SH::RAWS;
                                if (!(ok = warp_wait(&bars.raw_empty[rs], ((seq / SH::RAWS) & 1) ^ 1, ab))) break;
                                bring(f, kv, raw_s + rs * SH::RAW, &bars.raw_full[rs], seq);
                            }
                        }
                        if (f.w.next(p, cut)) f.coming = page_of(f.w, 0);
                    }
                } else {
                    // a thread's pieces of a tile: 16 stored values of one row after another, STEP rows apart
                    constexpr int CH = D / 16, STEP = 32 * kLoadWarps / CH;
                    const int row0 = ltid / CH, c = 2 * (ltid % CH);
                    while (ok && walk.more) {
                        const int tiles = 2 * (walk.pc.e - walk.pc.a);
                        for (int t = 0; t < tiles && ok; ++t, ++seq) {
                            const uint32_t st = seq % S, rs = seq % SH::RAWS;
                            ok = warp_wait(&bars.raw_full[rs], (seq / SH::RAWS) & 1, ab) &&
                                 warp_wait(&bars.empty[st], ((seq / S) & 1) ^ 1, ab);
                            if (!ok) break;
                            const uint8_t *src = smem + (2 + S) * SH::TILE + rs * SH::RAW + 16 * ltid;
                            uint8_t *dst = smem + (2 + st) * SH::TILE + (c >> 3) * SH::BOX;
#pragma unroll 3
                            for (int row = row0; row < 128; row += STEP, src += 16 * 32 * kLoadWarps) {
                                const uint4 v = *reinterpret_cast<const uint4 *>(src);
                                uint4 x, y;
                                e4m3x4_to_h2x2(v.x, x.x, x.y);
                                e4m3x4_to_h2x2(v.y, x.z, x.w);
                                e4m3x4_to_h2x2(v.z, y.x, y.y);
                                e4m3x4_to_h2x2(v.w, y.z, y.w);
                                *reinterpret_cast<uint4 *>(dst + row * 128 + (((c & 7) ^ (row & 7)) * 16)) = x;
                                *reinterpret_cast<uint4 *>(dst + row * 128 + ((((c & 7) + 1) ^ (row & 7)) * 16)) = y;
                            }
                            fence_async_proxy();
                            warp_arrive(&bars.full[st], lane);
                            if (lane == 0) mbar_arrive(smem_u32(&bars.raw_empty[rs]));
                            if (t == 1) load_q(walk.pc);
                        }
                        walk.next(p, cut);
                    }
                }
            }
            // On an abort: wait (again with a limit) for the copies in flight. Stages are filled in order, so the
            // last ones' cover them.
            if (!ok && any_tma && lane == 0) {
                constexpr uint32_t N = FP8 ? SH::RAWS : S;
                const uint32_t first = last_tma >= N - 1 ? last_tma - (N - 1) : 0;
                for (uint32_t q = first; q <= last_tma; ++q)
                    mbar_wait(smem_u32(FP8 ? &bars.raw_full[q % N] : &bars.full[q % N]), (q / N) & 1, ab, false);
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
cudaError_t tile_variant(int head_dim, int dtype, int fp8, F &&f)
{
    using B = __nv_bfloat16;
    using H = __half;
#define DFL_TILE(D)                                                                                                  \
    if (head_dim == D) {                                                                                             \
        if (fp8)                                                                                                     \
            return dtype == DFLASH_BF16 ? f(attend_tile_kernel<D, B, true>, TileShape<D, true>::SMEM)                \
                                        : f(attend_tile_kernel<D, H, true>, TileShape<D, true>::SMEM);               \
        return dtype == DFLASH_BF16 ? f(attend_tile_kernel<D, B, false>, TileShape<D, false>::SMEM)                  \
                                    : f(attend_tile_kernel<D, H, false>, TileShape<D, false>::SMEM);                 \
    }
    DFL_TILE(128)
    DFL_TILE(64)
#undef DFL_TILE
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t prepare_attend_tile(int smem_optin)
{
    for (int d : {64, 128})
        for (int dt : {DFLASH_BF16, DFLASH_FP16})
            for (int fp8 : {0, 1}) {
                const cudaError_t e =
                    tile_variant(d, dt, fp8, [&](auto kern, size_t) { return set_max_dynamic_smem(kern, smem_optin); });
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
                               int dtype, int fp8, int grid, cudaStream_t s)
{
    TileParams tp;
    tp.a = p;
    tp.tm_k = tm_k;
    tp.tm_v = tm_v;
    tp.box_rows = tile_box_rows(p.page);
    return tile_variant(head_dim, dtype, fp8, [&](auto kern, size_t smem) {
        return launch_ex(kern, dim3(grid), dim3(tile_threads(fp8 != 0)), smem, s, 1, tp);
    });
}

}  // namespace dfl
