// y = residual + act(x W^T + bias) on the tcgen05 tensor cores.
//
// The weights are the products' M: up to 128 rows of W per CTA are the lanes of
// TMEM, and a tile of NT rows of x its columns, so that a single token wastes
// 15 columns and not 127 lanes. k is streamed by TMA in stages of one to four
// boxes of 64 columns.
//
// Few rows are bound by the stream of W, each weight read once. One SM takes in
// some 60 GB/s from HBM whatever it has in flight, so many of them have to
// stream: a CTA takes fewer weight rows than 128 (F, a multiple of 8), or a
// cluster of up to 8 CTAs splits a tile's k, as far as the cost of a CTA and of
// the join allows (8 rows, 2560 x 2560: 100 CTAs of 128 weight rows and a fifth
// of k). The CTAs of a cluster join their sums through distributed shared
// memory in the order of their ranks, so that results do not depend on timing.
// The products' other lanes then hold what happens to lie behind the tile, and
// nobody reads them. Many rows are bound by the tensor cores: persistent CTA
// pairs on tiles of 256 x NT with two accumulators in TMEM, so that a tile's
// epilogue runs beside the next one's products.
//
// The tensor cores' fp32 accumulator truncates, at every 16 columns its sum and
// what lies more than some 25 bits below it of their products. Values of one
// sign come out too low: by 7e-7 of the result every 512 columns that one
// accumulator takes for bf16, 2.6e-6 for fp16, whose products have more bits;
// of values of both signs two thirds and a quarter of that are left (2-norm).
// So results in 32 bits read the accumulator out every 512 columns and sum in
// registers. Results in 16 bits are rounded by up to 3.9e-3 (bf16) or 4.9e-4
// (fp16): up to 65536 columns may stay in one accumulator (off by some 3.3e-4
// at that length for fp16 of one sign, 9e-5 for bf16). Tiles whose sums fit
// registers are half as large (256 rows, n = 5120, k = 53248 take 103 us, 153
// with them), so only sums longer than that are read out, every 4096.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdio.h>

#include <atomic>
#include <new>
#include <type_traits>

#include "common.cuh"
#include "dflash_linear.h"
#include "kernels.h"

namespace dfl {

dflash_status host_fail(dflash_status st, const char *msg);
dflash_status host_make_tmap_rows(CUtensorMap *tm, const void *ptr, int64_t rows, int64_t cols, int64_t stride, int box_rows);

struct LinearParams {
    CUtensorMap tm_w, tm_x;  // boxes of 64 columns x F rows of W, and the rows of x that one CTA loads of a tile
    const void *bias, *residual;
    void *y;
    int64_t residual_stride, y_stride;
    int rows, n;
    int F, NT;           // weight rows of a CTA, rows of x of a tile
    int boxes, stages;   // 64-column boxes per stage, stages of the ring
    int KB, seg;         // stages that k takes; that one accumulator takes
    int kb_part, kb_more;  // stages of a part of k, and how many parts have one more
    int tiles_f, tiles_t, band;
    int split;           // CTAs (pairs) that share a tile's k
    int owned;           // rows of x of a split tile that one of them joins, at most
    int apart;           // their sums have a place of their own, else in the ring
    int act;
    int vec;             // y and residual: 4 values at a time
    int ahead;           // the residual's rows start on 16 bytes: they are brought to L2 while the products run
    int *err;
};

namespace {

constexpr int kThreads = 320;  // TMA, products, 8 epilogue warps
constexpr int kLanes = 128;    // of TMEM: the most weight rows of a CTA
constexpr int kBox = 64;       // columns of a box: 128 bytes
constexpr int kMaxSplit = 8;
constexpr int kPlans = 256;    // that a handle remembers
// The least shared memory of a CTA in a cluster: more than half an SM's. CTAs of a cluster wait for one another with tensor
// memory in their hands, so two clusters must never hold parts of the same two SMs and wait for the rest; one such CTA to an
// SM rules that out. (Their registers do so today, against this kernel and the library's others with tensor memory: 320
// threads of 151 take 48,640 of 65,536.)
constexpr int kAlone = 117 * 1024;
constexpr int kMaxSum = 128;   // rows of x of a tile whose results are summed in registers
constexpr int64_t kLong = 65536;  // columns, above which results in 16 bits are summed there too

struct Layout {
    uint32_t w, stage, bars, extra, total;
};

constexpr int kRows = 32;                   // rows of x that an epilogue warp finishes at a time
constexpr uint32_t kTurn = kRows * 32 * 4;  // of 32 results each, turned from a lane per column to a lane per four

__host__ __device__ inline Layout layout(int F, int NT, int boxes, int stages, bool pair, int split, int owned, int apart)
{
    Layout l;
    l.w = static_cast<uint32_t>(F) * kBox * 2;
    l.stage = static_cast<uint32_t>(boxes) * (l.w + static_cast<uint32_t>(pair ? NT / 2 : NT) * kBox * 2);
    l.bars = static_cast<uint32_t>(stages) * l.stage;
    l.extra = l.bars + ((8u * (2u * stages + 5u) + 8u + 127u) & ~127u);  // full, empty, tfull, tempty, drain; TMEM, abort flag
    // the epilogue warps' turning places, or what the parts of a split tile send: [part][row][128]
    l.total = l.extra + (split == 1 ? 8 * kTurn : apart ? static_cast<uint32_t>(split * owned) * kLanes * 4 : 0u);
    // the products read 128 rows from a box's start on
    const uint32_t read = static_cast<uint32_t>(stages > 0 ? stages - 1 : 0) * l.stage + static_cast<uint32_t>(boxes - 1) * l.w + kLanes * kBox * 2;
    if (l.total < read) l.total = read;
    return l;
}

__host__ __device__ inline int tmem_columns(int NT)
{
    int c = 32;
    while (c < 2 * NT) c <<= 1;
    return c;
}

// One lane of the calling warp.
__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t is;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(is));
    return is;
}

// The issuing instructions below act on lanes with who != 0. Whole warps run the code around them: a branch for one
// lane would cost a chain of moves to uniform registers per product (100 clocks; as it is, the tensor cores' time).
template <bool kPair>
__device__ __forceinline__ void umma_if(uint32_t who, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "setp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(who)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "setp.ne.b32 q, %5, 0;\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(who)
            : "memory");
}

// An arrival on `bar` (a pair: on that barrier of both CTAs of `both`) when the products so far are over.
template <bool kPair>
__device__ __forceinline__ void commit_if(uint32_t who, uint32_t bar, uint16_t both)
{
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %2, 0;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}\n" ::"r"(bar),
            "h"(both), "r"(who)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %1, 0;\n\t"
            "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar),
            "r"(who)
            : "memory");
}

// A box to this CTA's shared memory, its bytes counted on `bar` (a pair: a barrier of either CTA).
template <bool kPair>
__device__ __forceinline__ void load_if(uint32_t who, uint32_t dst, const CUtensorMap *tm, int x, int y, uint32_t bar, uint64_t policy)
{
    if constexpr (kPair)
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %6, 0;\n\t"
            "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            ".L2::cache_hint [%0], [%1, {%2, %3}], [%4], %5;\n\t}\n" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar), "l"(policy), "r"(who)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\t"
            "setp.ne.b32 q, %6, 0;\n\t"
            "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
            " [%0], [%1, {%2, %3}], [%4], %5;\n\t}\n" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar), "l"(policy), "r"(who)
            : "memory");
}

__device__ __forceinline__ void expect_if(uint32_t who, uint32_t bar, uint32_t bytes)
{
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}\n" ::"r"(bar),
        "r"(bytes), "r"(who)
        : "memory");
}

// A whole warp's wait (a pair's barriers are also arrived on by the other CTA).
template <bool kPair>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag)
{
    const bool got = kPair ? mbar_wait_cluster(bar, parity, abort_flag) : mbar_wait(bar, parity, abort_flag);
    return __all_sync(0xFFFFFFFFu, got);
}

__device__ __forceinline__ void st_peer(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Exponentials and quotients by the fast forms: their error is a few 2^-22 of |z| (that of exp(-z) counts only where
// it is not small against 1, and then |z| is not large), below fp32's of a product's sum.
template <int N>
__device__ __forceinline__ void activate(float (&z)[N], int act)
{
    switch (act) {
    case DFLASH_ACT_RELU:
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = z[i] < 0.f ? 0.f : z[i];
        break;
    case DFLASH_ACT_SILU:
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = __fdividef(z[i], 1.f + __expf(-z[i]));
        break;
    case DFLASH_ACT_GELU:
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = 0.5f * z[i] * (1.f + erff(z[i] * 0.70710678f));
        break;
    case DFLASH_ACT_GELU_TANH:  // (1 + tanh u) / 2 = 1 / (1 + exp(-2u))
#pragma unroll
        for (int i = 0; i < N; ++i)
            z[i] = __fdividef(z[i], 1.f + __expf(-1.5957691f * (z[i] + 0.044715f * z[i] * z[i] * z[i])));
        break;
    default:
        break;
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

// Four values of type Y as they lie in memory: whole words, taken apart only where they are used (a load whose value is
// taken apart at once holds up the loads behind it).
template <typename Y>
struct alignas(sizeof(Y) * 4) Four {
    uint32_t w[sizeof(Y)];

    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (std::is_same_v<Y, float>) {
            return __uint_as_float(w[i]);
        } else {
            const uint16_t h = static_cast<uint16_t>(i & 1 ? w[i >> 1] >> 16 : w[i >> 1]);
            if constexpr (std::is_same_v<Y, __half>) return __half2float(__ushort_as_half(h));
            else return __uint_as_float(static_cast<uint32_t>(h) << 16);
        }
    }
    __device__ __forceinline__ void put(int i, Y y)
    {
        if constexpr (std::is_same_v<Y, float>) {
            w[i] = __float_as_uint(y);
        } else {
            uint16_t h;
            if constexpr (std::is_same_v<Y, __half>) h = __half_as_ushort(y);
            else h = __bfloat16_as_ushort(y);
            w[i >> 1] = i & 1 ? (w[i >> 1] & 0xFFFFu) | static_cast<uint32_t>(h) << 16 : (w[i >> 1] & 0xFFFF0000u) | h;
        }
    }
    // what the n values at `at` are, or four of them as one
    __device__ __forceinline__ void load(const Y *at, bool whole, int n)
    {
        if (whole) {
            *this = *reinterpret_cast<const Four *>(at);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) put(i, at[i]);
        }
    }
    __device__ __forceinline__ void store(Y *at, bool whole, int n) const
    {
        if (whole) {
            *reinterpret_cast<Four *>(at) = *this;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) at[i] = from_f<Y>(get(i));
        }
    }
};

template <typename Y>
__device__ __forceinline__ Four<Y> pack(float4 z)
{
    Four<Y> o;
    if constexpr (std::is_same_v<Y, float>) {
        o.w[0] = __float_as_uint(z.x), o.w[1] = __float_as_uint(z.y), o.w[2] = __float_as_uint(z.z), o.w[3] = __float_as_uint(z.w);
    } else if constexpr (std::is_same_v<Y, __half>) {
        const __half2 a = __floats2half2_rn(z.x, z.y), b = __floats2half2_rn(z.z, z.w);
        o.w[0] = *reinterpret_cast<const uint32_t *>(&a), o.w[1] = *reinterpret_cast<const uint32_t *>(&b);
    } else {
        const __nv_bfloat162 a = __floats2bfloat162_rn(z.x, z.y), b = __floats2bfloat162_rn(z.z, z.w);
        o.w[0] = *reinterpret_cast<const uint32_t *>(&a), o.w[1] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return o;
}

// 32 consecutive columns of this thread's TMEM lane, or the first 16 of them.
__device__ __forceinline__ void tmem_load32(uint32_t taddr, float (&v)[32], bool all)
{
    uint32_t r[32];
#define DFL_LD16(at, i)                                                                                                  \
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "    \
                 "%14, %15}, [%16];\n"                                                                                    \
                 : "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]),            \
                   "=r"(r[i + 6]), "=r"(r[i + 7]), "=r"(r[i + 8]), "=r"(r[i + 9]), "=r"(r[i + 10]), "=r"(r[i + 11]),      \
                   "=r"(r[i + 12]), "=r"(r[i + 13]), "=r"(r[i + 14]), "=r"(r[i + 15])                                    \
                 : "r"(at)                                                                                               \
                 : "memory")
    __syncwarp();
    DFL_LD16(taddr, 0);
    if (all) {
        DFL_LD16(taddr + 16u, 16);
    } else {
#pragma unroll
        for (int i = 16; i < 32; ++i) r[i] = 0u;
    }
#undef DFL_LD16
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    // (what is loaded is read after the wait)
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        asm volatile("" : "+r"(r[i]));
        v[i] = __uint_as_float(r[i]);
    }
}

// A row of a tile's results by one warp, four adjacent features a lane.
template <typename T, typename Y>
struct RowStore {
    const LinearParams &p;
    const int lane, n0, n1;  // features n0 .. n1 - 1
    float bias[4];
    bool whole;  // all four of the lane's features exist and go as one

    __device__ __forceinline__ int feature(int i) const { return n0 + lane * 4 + i; }

    __device__ __forceinline__ RowStore(const LinearParams &p_, int lane_, int n0_, int n1_) : p(p_), lane(lane_), n0(n0_), n1(n1_)
    {
        whole = p.vec && n0 + lane * 4 + 3 < n1;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            bias[i] = p.bias && feature(i) < n1 ? to_f(static_cast<const T *>(p.bias)[feature(i)]) : 0.f;
    }

    // this lane's values of the residual's row
    __device__ __forceinline__ void fetch(int row, Four<Y> &r) const
    {
        r.load(static_cast<const Y *>(p.residual) + static_cast<int64_t>(row) * p.residual_stride + feature(0), whole, n1 - feature(0));
    }

    __device__ __forceinline__ void store(int row, const float (&acc)[4], const Four<Y> &r) const
    {
        float z[4] = {acc[0] + bias[0], acc[1] + bias[1], acc[2] + bias[2], acc[3] + bias[3]};
        activate(z, p.act);
        if (p.residual) {
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] += r.get(i);
        }
        pack<Y>(make_float4(z[0], z[1], z[2], z[3]))
            .store(static_cast<Y *>(p.y) + static_cast<int64_t>(row) * p.y_stride + feature(0), whole, n1 - feature(0));
    }
};

// kPair: two CTAs compute a tile of 2 F weight rows (cta_group::2 products issued by the even CTA): each holds F weight
// rows and half of the tile's rows of x, and has the results of its weight rows. A cluster of p.split CTAs or pairs
// shares the stages of one tile. kSum: the accumulator is read out every p.seg stages and summed in registers.
template <bool kPair, typename T, typename Y, bool kSum>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const __grid_constant__ LinearParams p)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;  // 128-byte swizzled tiles start on 1024 bytes
    uint8_t *const gbase = smem_raw + (base - raw);

    constexpr int kCtas = kPair ? 2 : 1;
    const int NT = p.NT, S = p.stages, BX = p.boxes, F = p.F;
    const int XR = NT / kCtas;
    const int split = p.split;
    const Layout lay = layout(F, NT, BX, S, kPair, split, p.owned, p.apart);
    const uint32_t w_bytes = static_cast<uint32_t>(BX) * lay.w, x_bytes = static_cast<uint32_t>(XR) * kBox * 2;
    const uint32_t bar_full = base + lay.bars, bar_empty = bar_full + 8u * S;
    const uint32_t bar_tfull = bar_empty + 8u * S, bar_tempty = bar_tfull + 16u, bar_drain = bar_tempty + 16u;
    uint32_t *const tmem_holder = reinterpret_cast<uint32_t *>(gbase + lay.bars + 8u * (2u * S + 5u));
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const bool clustered = kPair || split > 1;
    const uint32_t rank = clustered ? cluster_ctarank() : 0u;
    const uint32_t half = kPair ? rank & 1u : 0u;    // of a pair
    const uint32_t part = kPair ? rank >> 1 : rank;  // of a tile's k
    int team, teams;                                 // the cluster's index, and how many there are
    asm("mov.u32 %0, %%clusterid.x;" : "=r"(team));
    asm("mov.u32 %0, %%nclusterid.x;" : "=r"(teams));

    // work items: tiles team, team + teams, .. (a split tile: one), in bands of `band` feature tiles, within which
    // the row tiles follow one another: CTAs that run together share both operands' tiles in L2
    const int items = p.tiles_f * p.tiles_t;
    auto tile_of = [&](int item, int &tf, int &tt) {
        if (p.tiles_t == 1) {
            tf = item;
            tt = 0;
            return;
        }
        const int per = p.band * p.tiles_t, b = item / per, in = item - b * per;
        const int width = min(p.band, p.tiles_f - b * p.band);
        tt = in / width;
        tf = b * p.band + in - tt * width;
    };
    auto first_feature = [&](int tf) { return (tf * kCtas + static_cast<int>(half)) * F; };
    // this CTA's stages of a tile
    const int per = p.kb_part + (static_cast<int>(part) < p.kb_more ? 1 : 0);
    const int kb0 = static_cast<int>(part) * p.kb_part + min(static_cast<int>(part), p.kb_more);

    uint64_t pol_w = 0, pol_x = 0;
    uint32_t who = 0;
    const uint32_t full0 = kPair ? mapa_shared(bar_full, rank & ~1u) : bar_full;  // where the pair's bytes are counted
    const uint32_t tx = kCtas * lay.stage;
    auto load_w = [&](int s, int row, int kb) {
        if (half == 0) expect_if(who, bar_full + 8u * s, tx);
        for (int b = 0; b < BX; ++b)
            load_if<kPair>(who, base + s * lay.stage + b * lay.w, &p.tm_w, (kb * BX + b) * kBox, row, full0 + 8u * s, pol_w);
    };
    auto load_x = [&](int s, int row, int kb) {
        for (int b = 0; b < BX; ++b)
            load_if<kPair>(who, base + s * lay.stage + w_bytes + b * x_bytes, &p.tm_x, (kb * BX + b) * kBox, row, full0 + 8u * s, pol_x);
    };
    const int pre = min(per, S);  // stages whose loads of W come first of all
    int tf0, tt0;
    tile_of(team, tf0, tt0);
    if (warp == 0) {
        who = elect_one();
        if (who) {
            for (int s = 0; s < S; ++s) {
                mbar_init(bar_full + 8u * s, 1);
                mbar_init(bar_empty + 8u * s, 1);
            }
            for (int a = 0; a < 2; ++a) {
                mbar_init(bar_tfull + 8u * a, 1);
                mbar_init(bar_tempty + 8u * a, 8 * kCtas);  // an arrival per epilogue warp (of both CTAs)
            }
            mbar_init(bar_drain, 1);
            *abort_flag = 0;
            fence_mbar_init();
        }
        __syncwarp();
        pol_w = p.tiles_t == 1 ? l2_policy_evict_first() : l2_policy_evict_normal();
        pol_x = p.tiles_t == 1 ? l2_policy_evict_last() : l2_policy_evict_normal();
        // W is constant from the handle's creation on: its first loads overlap the previous kernel on the stream, on SMs
        // that have room beside it
        if constexpr (!kPair)
            for (int i = 0; i < pre; ++i) load_w(i, first_feature(tf0), kb0 + i);
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
    if (clustered) cluster_sync_all();  // the even CTA's barriers exist, and every CTA's shared memory
    tc_fence_after_sync();
    const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *reinterpret_cast<volatile uint32_t *>(tmem_holder), 0);
    if (kPair && warp == 0)
        for (int i = 0; i < pre; ++i) load_w(i, first_feature(tf0), kb0 + i);
    // x, residual and y are touched after the previous kernel has finished
    pdl_trigger();
    pdl_wait();

    if (warp == 0) {
        // ---------------------------------------------------------------- loads
        bool ok = true;
        int s = 0, it = 0;
        uint32_t ph = 1;  // of the stage's emptiness
        for (; it < pre; ++it) load_x(it, tt0 * NT + static_cast<int>(half) * XR, kb0 + it);
        s = pre;
        if (s == S) s = 0, ph ^= 1u;
        for (int i = team; ok && i < items; i += teams) {
            int tf, tt;
            tile_of(i, tf, tt);
            for (int k = i == team ? pre : 0; k < per; ++k, ++it) {
                // (the ring's first round is empty; from then on a stage is free when its products are over)
                ok = warp_wait<false>(bar_empty + 8u * s, ph, abort_flag);
                if (!ok) break;
                load_w(s, first_feature(tf), kb0 + k);
                load_x(s, tt * NT + static_cast<int>(half) * XR, kb0 + k);
                if (++s == S) s = 0, ph ^= 1u;
            }
        }
        if (!ok) {
            if (who) atomicOr(p.err, DEV_ERR_TIMEOUT);
            // what has been issued lands before the CTA can end
            if (half == 0) {
                for (int j = it > S ? it - S : 0; j < it; ++j)
                    mbar_wait(bar_full + 8u * (j % S), static_cast<uint32_t>(j / S) & 1u, abort_flag, false);
            } else {  // (counted on the even CTA's barriers: a copy lands within microseconds)
                const uint64_t t0 = global_timer_ns();
                while (global_timer_ns() - t0 < 100000ull) {
                }
            }
            __syncwarp();
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- products (a pair: the even CTA's)
        if (half == 0) {
            who = elect_one();
            constexpr bool kHalf = std::is_same_v<T, __half>;
            const uint32_t idesc = idesc_bf16_f32(kCtas * kLanes, NT) & (kHalf ? ~((1u << 7) | (1u << 10)) : ~0u);
            const uint16_t both = static_cast<uint16_t>(3u << (rank & ~1u));
            // a descriptor's low bits are the address in units of 16 bytes: stepping it is an addition
            const uint64_t w0 = smem_desc_sw128(base), x0 = smem_desc_sw128(base + w_bytes);
            int s = 0, n = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int i = team; ok && i < items; i += teams) {
                for (int k0 = 0; ok && k0 < per; k0 += p.seg, ++n) {
                    const int a = n & 1;
                    ok = warp_wait<kPair>(bar_tempty + 8u * a, (static_cast<uint32_t>(n >> 1) & 1u) ^ 1u, abort_flag);
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint32_t d = tmem + static_cast<uint32_t>(a * NT);
                    const int k1 = min(per, k0 + p.seg);
                    uint32_t more = 0;  // the accumulator holds something
                    for (int k = k0; k < k1; ++k) {
                        ok = warp_wait<kPair>(bar_full + 8u * s, ph, abort_flag);
                        if (!ok) break;
                        tc_fence_after_sync();
                        const uint32_t at = static_cast<uint32_t>(s) * (lay.stage >> 4);
                        for (int b = 0; b < BX; ++b) {
                            const uint64_t wd = w0 + at + b * (lay.w >> 4), xd = x0 + at + b * (x_bytes >> 4);
#pragma unroll
                            for (int j = 0; j < kBox / 16; ++j) {
                                umma_if<kPair>(who, d, wd + 2 * j, xd + 2 * j, idesc, more);
                                more = 1;
                            }
                        }
                        commit_if<kPair>(who, bar_empty + 8u * s, both);
                        if (++s == S) s = 0, ph ^= 1u;
                    }
                    if (ok) commit_if<kPair>(who, bar_tfull + 8u * a, both);
                }
            }
            if (!ok && who) atomicOr(p.err, DEV_ERR_TIMEOUT);
            // every product is over before TMEM is released
            commit_if<kPair>(who, bar_drain, static_cast<uint16_t>(1u << rank));
            mbar_wait(bar_drain, 0, abort_flag, false);
            __syncwarp();
        }
    } else {
        // ---------------------------------------------------------------- epilogue: a thread has a weight row's results;
        // the two warps of a lane quadrant take turns at 32 of a tile's rows of x
        const int g = (warp - 2) >> 2, q = warp & 3, f = q * 32 + lane;
        constexpr int kSteps = kMaxSum / (2 * kRows);  // of a warp, at most
        float *const turn = reinterpret_cast<float *>(gbase + lay.extra + (warp - 2) * kTurn);
        const uint32_t mail = base + (p.apart ? lay.extra : 0u);  // where the parts of a split tile arrive
        const int tr = lane >> 3, tc = (lane & 7) * 4;            // turned: rows tr + 4 t, features tc .. tc + 3
        int n = 0;
        bool ok = true;
        // A tile's residual, 32 rows a warp: whole rows of it to L2, since what the warps fetch of a row (64 bytes) is less
        // than HBM serves well (8192 rows, n = 10240, k = 2560: 350 us without)
        auto bring = [&](int i) {
            int tf, tt;
            tile_of(i, tf, tt);
            const int n0 = first_feature(tf), row = tt * NT + (warp - 2) * 32 + lane;
            const uint32_t bytes = static_cast<uint32_t>(max(0, min(p.n, n0 + F) - n0)) * sizeof(Y) & ~15u;
            if ((warp - 2) * 32 + lane < NT && row < p.rows && bytes > 0)
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const Y *>(p.residual) +
                                                                                static_cast<int64_t>(row) * p.residual_stride + n0),
                             "r"(bytes)
                             : "memory");
        };
        if (p.ahead && team < items) bring(team);
        for (int i = team; ok && i < items; i += teams) {
            int tf, tt;
            tile_of(i, tf, tt);
            if (p.ahead && i + teams < items) bring(i + teams);
            const int n0 = first_feature(tf), feature = n0 + f;
            const int end = min(p.n, n0 + F);  // behind the CTA's last feature
            const int row0 = tt * NT, valid = q * 32 < F ? min(NT, p.rows - row0) : 0;
            const float bias = p.bias && feature < end ? to_f(static_cast<const T *>(p.bias)[feature]) : 0.f;
            const bool whole = p.vec && n0 + q * 32 + tc + 3 < end;
            const int64_t col = n0 + q * 32 + tc;
            // the residual of 32 rows: as it is turned (four values of eight rows), or the thread's own column
            auto fetch = [&](int c, Four<Y> (&r)[8]) {
                if (!p.residual || split > 1) return;
                const Y *const res = static_cast<const Y *>(p.residual) + static_cast<int64_t>(row0 + c) * p.residual_stride;
                if (p.vec) {
                    const Y *const at = res + tr * p.residual_stride + col;
                    const int rows = valid - c - tr;  // (this lane's rows are 4 t < rows)
                    if (whole) {
#pragma unroll
                        for (int t = 0; t < 8; ++t)
                            if (4 * t < rows) r[t].load(at + 4 * t * p.residual_stride, true, 4);
                    } else {
#pragma unroll
                        for (int t = 0; t < 8; ++t)
                            if (4 * t < rows) r[t].load(at + 4 * t * p.residual_stride, false, end - static_cast<int>(col));
                    }
                } else if (feature < end) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c + j < valid) r[j >> 2].put(j & 3, res[j * p.residual_stride + feature]);
                }
            };
            auto finish = [&](int c, float (&v)[32], const Four<Y> (&r)[8]) {
                if (split > 1) {  // to the CTA that joins the row
                    int slot = c / split, owner = c - slot * split;
                    const uint32_t to = mail + static_cast<uint32_t>((static_cast<int>(part) * p.owned * kLanes + f) * 4);
#pragma unroll
                    for (int h = 0; h < 32; h += 8) {
                        if (c + h >= valid) break;
#pragma unroll
                        for (int j = h; j < h + 8; ++j) {
                            if (c + j < valid)
                                st_peer(mapa_shared(to + static_cast<uint32_t>(slot * kLanes * 4), static_cast<uint32_t>(owner * kCtas) + half), v[j]);
                            if (++owner == split) owner = 0, ++slot;
                        }
                    }
                    return;
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] += bias;
                activate(v, p.act);
                Y *const y = static_cast<Y *>(p.y) + static_cast<int64_t>(row0 + c) * p.y_stride;
                if (p.vec) {
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 32; ++j) turn[j * 32 + lane] = v[j];
                    __syncwarp();
                    Y *const y0 = y + tr * p.y_stride + col;
                    const int rows = valid - c - tr;  // (this lane's rows are 4 t < rows)
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        float4 z = *reinterpret_cast<const float4 *>(turn + (tr + 4 * t) * 32 + tc);
                        if (p.residual) z.x += r[t].get(0), z.y += r[t].get(1), z.z += r[t].get(2), z.w += r[t].get(3);
                        if (4 * t < rows) pack<Y>(z).store(y0 + 4 * t * p.y_stride, whole, end - static_cast<int>(col));
                    }
                } else if (feature < end) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (c + j < valid) y[j * p.y_stride + feature] = from_f<Y>(p.residual ? v[j] + r[j >> 2].get(j & 3) : v[j]);
                }
            };
            auto release = [&](int a) {  // the accumulator goes back to the products' warp
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (kPair)
                        mbar_arrive_remote(mapa_shared(bar_tempty + 8u * a, rank & ~1u));
                    else
                        mbar_arrive(bar_tempty + 8u * a);
                }
            };
            auto column = [&](int a) { return tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(a * NT); };
            if constexpr (kSum) {
                float acc[kSteps][32];
                for (int k0 = 0; ok && k0 < per; k0 += p.seg, ++n) {
                    const int a = n & 1;
                    ok = warp_wait<kPair>(bar_tfull + 8u * a, static_cast<uint32_t>(n >> 1) & 1u, abort_flag);
                    if (!ok) break;
                    tc_fence_after_sync();
#pragma unroll
                    for (int ci = 0; ci < kSteps; ++ci) {
                        const int c = (2 * ci + g) * kRows;
                        if (c < valid) {
                            float v[32];
                            tmem_load32(column(a) + static_cast<uint32_t>(c), v, c + 16 < NT);
#pragma unroll
                            for (int j = 0; j < 32; ++j) acc[ci][j] = k0 == 0 ? v[j] : acc[ci][j] + v[j];
                        }
                    }
                    release(a);
                }
                if (split > 1 && !p.apart) cluster_sync_all();  // no CTA's ring is in use
                if (!ok) break;
#pragma unroll
                for (int ci = 0; ci < kSteps; ++ci) {
                    const int c = (2 * ci + g) * kRows;
                    if (c < valid) {
                        Four<Y> r[8];
                        fetch(c, r);
                        finish(c, acc[ci], r);
                    }
                }
            } else {
                const int a = n & 1;
                Four<Y> r[8];
                if (g * kRows < valid) fetch(g * kRows, r);
                ok = warp_wait<kPair>(bar_tfull + 8u * a, static_cast<uint32_t>(n >> 1) & 1u, abort_flag);
                ++n;
                if (split > 1 && !p.apart) cluster_sync_all();  // no CTA's ring is in use
                if (!ok) break;
                tc_fence_after_sync();
                for (int c = g * kRows; c < valid; c += 2 * kRows) {
                    float v[32];
                    tmem_load32(column(a) + static_cast<uint32_t>(c), v, c + 16 < NT);
                    Four<Y> next[8];
                    if (c + 2 * kRows < valid) fetch(c + 2 * kRows, next);
                    finish(c, v, r);
#pragma unroll
                    for (int t = 0; t < 8; ++t) r[t] = next[t];
                }
                release(a);
            }
        }
    }
    if (warp < 2 && split > 1 && !p.apart) {
        __syncwarp();
        cluster_sync_all();
    }
    __syncwarp();

    if (split > 1) {
        // the CTAs that share a tile share its rows too: a warp a row, summed in the order of the parts
        const int n0 = first_feature(tf0), valid = min(NT, p.rows - tt0 * NT), end = min(p.n, n0 + F);
        const int slot0 = warp - 2, row0 = static_cast<int>(part) + slot0 * split;
        const RowStore<T, Y> out(p, lane, n0, end);
        Four<Y> r;
        if (p.residual && warp >= 2 && row0 < valid) out.fetch(tt0 * NT + row0, r);
        cluster_sync_all();  // everything has arrived, and products, copies and arrivals are over
        if (warp >= 2) {
            const float *const mine = reinterpret_cast<const float *>(gbase + (p.apart ? lay.extra : 0u)) + lane * 4;
            for (int slot = slot0; static_cast<int>(part) + slot * split < valid; slot += 8) {
                const int row = tt0 * NT + static_cast<int>(part) + slot * split;
                if (p.residual && slot != slot0) out.fetch(row, r);
                float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < kMaxSplit; ++s)
                    if (s < split) {
                        const float4 v = *reinterpret_cast<const float4 *>(mine + (s * p.owned + slot) * kLanes);
                        z[0] += v.x, z[1] += v.y, z[2] += v.z, z[3] += v.w;
                    }
                out.store(row, z, r);
            }
        }
    } else if constexpr (kPair) {
        cluster_sync_all();  // the pair's products, copies and arrivals are over
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

// Results in 16 bits of up to kLong columns do not notice the accumulator's truncation (see the top).
bool sums(const dflash_linear_config &c)
{
    return c.out_dtype == DFLASH_FP32 || c.k > kLong;
}

// How a call is cut: tiles of NT rows by F weight rows of a CTA, or of both CTAs of a pair, `split` of which share k.
struct Plan {
    int pair, F, NT, split, boxes, stages, grid;  // grid: clusters
    int apart = 0;   // a split tile's sums have a place of their own
    int owned() const { return (NT + split - 1) / split; }
};

struct Machine {
    int sms = 0, smem = 0;                // SMs, dynamic shared memory of a block
    int clusters[2][kMaxSplit + 1] = {};  // clusters of that many CTAs that run at a time: of single CTAs, of pairs
};

int smem_of(const Plan &pl)
{
    return static_cast<int>(layout(pl.F, pl.NT, pl.boxes, pl.stages, pl.pair, pl.split, pl.owned(), pl.apart).total) + 1024;  // (alignment)
}

// The ring's stages. False if the plan does not fit.
bool fit_stages(Plan &pl, int KB64, const Machine &m)
{
    const int need = (KB64 + pl.split - 1) / pl.split;
    const int box = static_cast<int>(layout(pl.F, pl.NT, 1, 1, pl.pair, pl.split, 0, 0).stage);
    // stages of up to 4 boxes and 40 KB: fewer barriers, and longer pieces of W's rows
    pl.boxes = 1;
    while (pl.boxes < 4 && 2 * pl.boxes * box <= 40 * 1024 && 4 * pl.boxes <= need) pl.boxes *= 2;
    const int KB = (KB64 + pl.boxes - 1) / pl.boxes;
    const int stage = pl.boxes * box;
    if (KB < pl.split) return false;
    // a split tile's sums have a place of their own where that is small, else in the ring
    const int sums = pl.split > 1 ? pl.split * pl.owned() * kLanes * 4 : 0;
    pl.apart = pl.split > 1 && sums <= 36 * 1024;
    pl.stages = 0;
    int most = (m.smem - smem_of(pl)) / (stage + 16);
    int use = (KB + pl.split - 1) / pl.split;
    if (use > most) use = most;
    while (pl.split > 1 && !pl.apart && use * stage < sums) ++use;
    pl.stages = use;
    return use >= 1 && smem_of(pl) <= m.smem;
}

// A plan's time in microseconds but for a constant: a fit to 3,000 plans of 35 shapes (1 to 12,000 rows, n 128 to
// 151,936, k 512 to 16,000), by which the chosen plan is 2 % slower than the fastest on average and 12 % at most. (The
// constants are what the fit gave; its timings were not kept.)
// (Above `most` only some number above it, without the roots.)
double cost(const Plan &pl, int64_t rows, int64_t n, int64_t k, int KB64, int64_t items, double most)
{
    const int ctas = pl.pair ? 2 : 1;
    const double rounds = pl.split > 1 ? 1 : static_cast<double>((items + pl.grid - 1) / pl.grid);
    const double steps = static_cast<double>((KB64 + pl.split - 1) / pl.split);  // of 64 columns
    const double xr = static_cast<double>(pl.NT / ctas < rows ? pl.NT / ctas : rows);
    const double valid = static_cast<double>(pl.NT < rows ? pl.NT : rows);
    // a step: its products, which follow one another, and what the SM takes in for them, in L4
    const double mma = pl.NT * 0.001 > 0.127 ? pl.NT * 0.001 : 0.127;
    const double in = pl.F / 940.0 + xr / 615.0;
    const double least = rounds * steps * (mma > in ? mma : in);
    if (least > most) return least;
    const double step = sqrt(sqrt(mma * mma * mma * mma + in * in * in * in));
    const double chain = rounds * steps * step, hbm = static_cast<double>(n) * k * 2 / 9e6;
    // the epilogue of the last tile; with a short k also those that the next tile's products do not cover
    const double epilogue = 0.0113 * valid, late = 1.36 * epilogue - steps * step;
    double t = sqrt(chain * chain + hbm * hbm) + 0.0084 * pl.grid * pl.split * ctas + (pl.pair ? 1.25 : 0);
    t += pl.split > 1 ? 0.375 + 0.026 * pl.split + 0.147 * ((pl.NT < rows ? pl.NT : static_cast<int>(rows)) + pl.split - 1) / pl.split + 0.5 * epilogue
                      : epilogue;
    return late > 0 ? t + late * (rounds - 1) : t;
}

Plan choose(int64_t rows, int64_t n, int64_t k, bool sum, const Machine &m)
{
    const int KB64 = static_cast<int>((k + kBox - 1) / kBox);
    Plan best = {};
    double best_t = HUGE_VAL;
    const int widest = sum ? kMaxSum : 256;
    const int most = static_cast<int>(rows < widest ? (rows + 15) / 16 * 16 : widest);
    for (int pair = 0; pair < 2; ++pair) {
        const int ctas = pair ? 2 : 1;
        if (pair && rows <= 32) continue;
        int64_t tiles_f[kLanes / 8 + 1];
        for (int F = 8; F <= kLanes; F += 8) tiles_f[F / 8] = (n + F * ctas - 1) / (F * ctas);
        for (int split = 1; split * ctas <= kMaxSplit; ++split) {
            const int slots = m.clusters[pair][split * ctas];
            if (slots < 1 || split > KB64) continue;
            for (int NT = most; NT >= 16; NT -= 16) {
                if (NT < most && rows <= 64) break;       // (more rows per weight cost nothing there)
                if (rows > 512 && NT < 64) break;
                const int64_t tiles_t = (rows + NT - 1) / NT;
                for (int F = kLanes; F >= (rows <= 256 ? 16 : kLanes); F -= 8) {
                    Plan pl = {pair, F, NT, split, 1, 0, 0};
                    const int64_t items = tiles_f[F / 8] * tiles_t;
                    if (split > 1 && items > slots) break;
                    pl.grid = static_cast<int>(items < slots ? items : slots);
                    const double t = cost(pl, rows, n, k, KB64, items, best_t);
                    if (t < best_t && fit_stages(pl, KB64, m)) best = pl, best_t = t;
                }
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

template <typename T, typename Y, bool kSum>
cudaError_t launch(const Plan &pl, const LinearParams &p, cudaStream_t s)
{
    cudaLaunchAttribute attr[2];
    const int size = (pl.pair ? 2 : 1) * pl.split, smem = smem_of(pl);
    const cudaLaunchConfig_t cfg = config(pl.grid, size, size > 1 && smem < kAlone ? kAlone : smem, s, attr);
    return pl.pair ? cudaLaunchKernelEx(&cfg, linear_kernel<true, T, Y, kSum>, p) : cudaLaunchKernelEx(&cfg, linear_kernel<false, T, Y, kSum>, p);
}

template <typename T, typename Y, bool kSum>
cudaError_t prepare(Machine &m)
{
    cudaLaunchAttribute attr[2];
    cudaError_t e = set_max_dynamic_smem(linear_kernel<true, T, Y, kSum>, m.smem);
    if (e == cudaSuccess) e = set_max_dynamic_smem(linear_kernel<false, T, Y, kSum>, m.smem);
    if (e != cudaSuccess) return e;
    m.clusters[0][1] = m.sms;
    for (int pair = 0; pair < 2; ++pair)
        for (int size = 2; size <= kMaxSplit; size += pair + 1) {
            const cudaLaunchConfig_t cfg = config(1, size, m.smem, nullptr, attr);
            int *const to = &m.clusters[pair][size];
            e = pair ? cudaOccupancyMaxActiveClusters(to, linear_kernel<true, T, Y, kSum>, &cfg)
                     : cudaOccupancyMaxActiveClusters(to, linear_kernel<false, T, Y, kSum>, &cfg);
            if (e != cudaSuccess) {
                cudaGetLastError();
                *to = 0;  // (such a cluster is not used)
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
    CUtensorMap tm_w[dfl::kLanes / 8];  // by F / 8 - 1
    int *err = nullptr;
    // plans that have been chosen, by the low bits of the rows (rows << 32 | F / 8 << 16 | NT / 16 << 8 | split << 4 | pair): a
    // server's steps come back to their row counts, and looking through the plans takes 0.5 to 25 us
    std::atomic<uint64_t> plans[dfl::kPlans] = {};
};

namespace dfl {
namespace {

Plan plan_for(dflash_linear_ctx *h, int64_t rows)
{
    std::atomic<uint64_t> &place = h->plans[rows % kPlans];
    const uint64_t last = place.load(std::memory_order_relaxed);
    const int64_t n = h->cfg.n, k = h->cfg.k;
    if (last >> 32 == static_cast<uint64_t>(rows)) {
        Plan pl = {static_cast<int>(last & 15), static_cast<int>(last >> 16 & 255) * 8, static_cast<int>(last >> 8 & 255) * 16,
                   static_cast<int>(last >> 4 & 15), 1, 0, 0};
        const int ctas = pl.pair ? 2 : 1, slots = h->m.clusters[pl.pair][pl.split * ctas];
        const int64_t items = (n + pl.F * ctas - 1) / (pl.F * ctas) * ((rows + pl.NT - 1) / pl.NT);
        fit_stages(pl, static_cast<int>((k + kBox - 1) / kBox), h->m);
        pl.grid = static_cast<int>(items < slots ? items : slots);
        return pl;
    }
    const Plan pl = choose(rows, n, k, sums(h->cfg), h->m);
    if (pl.grid > 0)
        place.store(static_cast<uint64_t>(rows) << 32 | static_cast<uint64_t>(pl.F / 8) << 16 | static_cast<uint64_t>(pl.NT / 16) << 8 |
                        static_cast<uint64_t>(pl.split) << 4 | static_cast<uint64_t>(pl.pair),
                    std::memory_order_relaxed);
    return pl;
}

}  // namespace
}  // namespace dfl

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
    const bool sum = dfl::sums(*cfg);
    using B16 = __nv_bfloat16;
    cudaError_t e = half ? (wide  ? dfl::prepare<__half, float, true>(c->m)
                            : sum ? dfl::prepare<__half, __half, true>(c->m)
                                  : dfl::prepare<__half, __half, false>(c->m))
                         : (wide  ? dfl::prepare<B16, float, true>(c->m)
                            : sum ? dfl::prepare<B16, B16, true>(c->m)
                                  : dfl::prepare<B16, B16, false>(c->m));
    dflash_status st = DFLASH_OK;
    if (e == cudaSuccess) {
        for (int i = 0; st == DFLASH_OK && i < dfl::kLanes / 8; ++i)
            st = dfl::host_make_tmap_rows(&c->tm_w[i], W, cfg->n, cfg->k, cfg->n > 1 ? cfg->w_stride : (cfg->k + 7) / 8 * 8, 8 * (i + 1));
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

    const dfl::Plan pl = dfl::plan_for(h, rows);
    if (pl.grid < 1) return linear_fail(DFLASH_ERR_UNSUPPORTED, "no tiling fits this device's shared memory");
    if ((n + pl.F - 1) / pl.F * ((rows + pl.NT - 1) / pl.NT) >= (int64_t(1) << 31))
        return linear_fail(DFLASH_ERR_INVALID_ARG, "too many tiles: %lld rows of %lld values", rows, n);
    dfl::LinearParams p;
    p.tm_w = h->tm_w[pl.F / 8 - 1];
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
    // (columns of an accumulator: 512 for results in 32 bits, 4096 for long sums in 16)
    p.seg = !dfl::sums(h->cfg) ? p.KB : (size == 4 ? 8 : 64) / pl.boxes;
    p.F = pl.F;
    const int F = pl.pair ? 2 * pl.F : pl.F;
    p.tiles_f = static_cast<int>((n + F - 1) / F);
    p.tiles_t = static_cast<int>((rows + pl.NT - 1) / pl.NT);
    p.band = 8;
    p.split = pl.split;
    p.kb_part = p.KB / pl.split;
    p.kb_more = p.KB % pl.split;
    p.owned = pl.owned();
    p.apart = pl.apart;
    p.act = h->cfg.activation;
    const uintptr_t four = 4 * size;
    p.vec = !dfl::misaligned(y, four) && (rows == 1 || y_stride % 4 == 0) &&
            (!residual || (!dfl::misaligned(residual, four) && (rows == 1 || residual_stride % 4 == 0)));
    p.ahead = residual && pl.split == 1 && !dfl::misaligned(residual, 16) && (rows == 1 || residual_stride * size % 16 == 0);
    p.err = h->err;
    const auto s = static_cast<cudaStream_t>(stream);
    const bool half = h->cfg.dtype == DFLASH_FP16, wide = size == 4, sum = dfl::sums(h->cfg);
    using B16 = __nv_bfloat16;
    const cudaError_t e = half ? (wide  ? dfl::launch<__half, float, true>(pl, p, s)
                                  : sum ? dfl::launch<__half, __half, true>(pl, p, s)
                                        : dfl::launch<__half, __half, false>(pl, p, s))
                               : (wide  ? dfl::launch<B16, float, true>(pl, p, s)
                                  : sum ? dfl::launch<B16, B16, true>(pl, p, s)
                                        : dfl::launch<B16, B16, false>(pl, p, s));
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
