// Launch interfaces of the paged-attention kernels (host side) and the launch
// parameters that they share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dflash_paged.h"
#include "kernels.h"

namespace dfl {

// Bit of the device error word beside those of kernels.h: a page id, a length
// or a position outside its table.
enum : int { DEV_ERR_PLACE = 4 };

// ---- norm + rotation (+ cache append) ----
struct PrepRows {  // [tokens, heads, head_dim] in and out; strides in elements
    const void *in = nullptr;
    void *out = nullptr;
    int64_t in_ts = 0, in_hs = 0, out_ts = 0, out_hs = 0;
    const void *weight = nullptr;
    int heads = 0;
};

struct PrepParams {
    PrepRows q, k, v;  // out of k and v unused where the cache takes them
    int tokens = 0;
    const float *table = nullptr;
    int positions_n = 0, rotary = 0, interleaved = 0;
    float eps = 0.f;
    const int32_t *positions = nullptr;
    // cache (append only)
    int append = 0, fp8 = 0;
    dflash_paged_cache cache = {};
    dflash_paged_batch batch = {};
    int page = 0;
    int *err = nullptr;
};
cudaError_t launch_prep(const PrepParams &p, int head_dim, int dtype, cudaStream_t s);

// ---- attention ----
// Division of 0 <= n < 2^31 by a constant of the launch (a product and a shift: Granlund and Montgomery, "Division by
// invariant integers using multiplication").
struct FastDiv {
    uint32_t d = 1, mul = 1, shift = 0;
    FastDiv() = default;
    explicit FastDiv(uint32_t by) : d(by)
    {
        while ((uint64_t(1) << shift) < by) ++shift;  // ceil(log2 by)
        mul = static_cast<uint32_t>((((uint64_t(1) << shift) - by) << 32) / by + 1);
    }
#ifdef __CUDACC__
    __host__ __device__ __forceinline__ int div(int n) const
    {
        const uint32_t u = static_cast<uint32_t>(n), high = static_cast<uint32_t>((static_cast<uint64_t>(u) * mul) >> 32);
        return static_cast<int>((high + u) >> shift);
    }
#endif
};

struct AttendParams {
    const void *q;
    void *out;
    float *lse;
    int64_t q_ts, q_hs, o_ts, o_hs;
    const void *k, *v;
    int64_t page_stride, slot_stride, head_stride;
    const int32_t *cu, *lens, *table;
    int64_t table_stride;
    int table_cols, num_pages;
    int B, tokens, kv_heads, group, page;  // group = query heads per key/value head
    int lanes, lane_heads, lane_ctas;      // heads walked in step, heads and CTAs of each (set_lanes())
    FastDiv by_group, by_page;
    int causal, window;            // window 0: none
    float scale_log2;              // score scale * log2(e) (* the keys' scale)
    float v_scale;
    // Workspace: CTA c's (PagedPlan::cta) partial results in slots 2c (a piece that continues an
    // earlier CTA's item) and 2c + 1 (one that a later CTA continues). An item
    // split over at most kTicketParts CTAs is joined by whichever finishes last
    // (a counter per warp's rows, at the CTA that begins the item, zero between
    // calls); one over more CTAs by the merge kernel, whose list has entry c
    // for the item that CTA c begins.
    float *part_o;     // [2 * grid][rows * head_dim]
    float2 *part_ml;   // [2 * grid][rows] running maximum (log2) and sum
    int4 *merge;       // [2 * grid]: first token row, first row, rows, key/value head | CTAs (0: nothing to do)
    unsigned *ticket;  // [grid][kTicketWarps]
    int merge_early;   // the merge kernel lets the next launch begin at once, not only when the parts are written
    int *err;
};

// Key/value heads are dealt to `lanes` groups of `lane_ctas` CTAs: group l takes heads l, l + lanes, .. and its
// CTAs split their keys, all groups in the same way, so that the CTAs of a wave read the same keys of adjacent
// heads, which lie next to each other where a slot holds all heads (128 single tokens, 8 heads, 8-bit cache: 88 us,
// 101 with the heads one after the other; 16-bit 154 and 160; heads of 64 values, 8-bit 60 and 105). The most
// lanes up to `most` that divide the heads and leave no more than 1/64 of the grid idle. The many-row kernel has
// one: its row tiles, one after the other, find a head's keys in L2 (2048 rows of 40 heads: 416 us, 429 dealt out).
inline void set_lanes(AttendParams &p, int grid, int most)
{
    p.lanes = 1;
    for (int k = 2; k <= most && k <= grid; ++k)
        if (p.kv_heads % k == 0 && grid % k <= grid / 64) p.lanes = k;
    p.lane_heads = p.kv_heads / p.lanes;
    p.lane_ctas = grid / p.lanes;
}

// Rows of a work item and keys of a work unit of the two kernels.
constexpr int kRowsUnit = 64;    // few rows: 8, 16 or 32 rows, units of 64 keys
constexpr int kTileRows = 256;   // many rows
constexpr int kTileUnit = 128;
// (Joined by tickets up to 4 CTAs: 32 ragged sequences of 32 rows take 102 us, a prompt chunk of 2048 tokens 293;
// all by the merge kernel, 115 and 461. Up to 8 CTAs was no faster.)
constexpr int kTicketParts = 4, kTicketWarps = 8;

cudaError_t prepare_attend_rows(int smem_optin);
cudaError_t launch_attend_rows(const AttendParams &p, int head_dim, int dtype, int fp8, int rows, int grid,
                               cudaStream_t s);
cudaError_t prepare_attend_tile(int smem_optin);
// Rows of one box of a page's tensor map: the most that divide a page and a tile.
int tile_box_rows(int page);
// tm_k, tm_v: host_make_tmap_pages() with boxes of tile_box_rows() slots.
cudaError_t launch_attend_tile(const AttendParams &p, const CUtensorMap &tm_k, const CUtensorMap &tm_v, int head_dim,
                               int dtype, int fp8, int grid, cudaStream_t s);
// Joins the items split over many CTAs (rows per item, `entries` CTAs of the
// attention launch); by_value: parts laid out [value / 4][row][4] instead of [row][value].
cudaError_t launch_attend_merge(const AttendParams &p, int head_dim, int dtype, int rows, int entries, bool by_value,
                                int grid, cudaStream_t s);

}  // namespace dfl
