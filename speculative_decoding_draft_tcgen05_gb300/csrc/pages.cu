// Pages, positions and slots of a step's new tokens from the requests' lengths,
// and the pages of dropped tokens given back.
//
// A page's or token's place in the batch follows from running sums over the
// entries before it. Entries are cut into ranges of 32, 256 or 1024 (a block's
// threads); the grid is ranges x parts. Every block sums the entries before its range and scans its own (a few
// hundred bytes per hundred entries, from L2), so no block waits for another,
// and the blocks of a range share its pages, table entries and tokens, found by
// binary search in the scan. Requests' lengths and the number of free pages
// change only when every block has read them: the block that finishes last (a
// counter) writes them. A call is bound by the latency of its dependent reads
// (row, length, page id), so a small batch is one warp's, without barriers.
#include <stdio.h>

#include "common.cuh"
#include "dflash_pages.h"
#include "kernels.h"
#include "spans.h"

namespace dfl {

dflash_status host_fail(dflash_status st, const char *msg);

namespace {

struct PagesParams {
    dflash_page_pool pool;
    const int32_t *rows, *counts;  // extend: new tokens; trim: what is dropped, with `base`
    int batch, ranges, parts;
    int tokens, base;
    int32_t *cu, *lens, *table;
    int64_t table_stride;
    int table_cols, room;  // columns of `table`, and those that a request may fill
    int32_t *positions;
    int64_t *slots;
    int32_t *granted;
};

// What an entry asks for.
struct Entry {
    int row, len;      // row -1: out of range
    int held, pages;   // pages taken (extend) or given (trim)
    int tokens;        // new tokens; trim: the length that is left
    bool valid;
};

// ceil(len / page)
__device__ __forceinline__ int pages_of(int len, int page)
{
    return static_cast<int>((static_cast<unsigned>(len) + static_cast<unsigned>(page) - 1u) / static_cast<unsigned>(page));
}

template <bool kTrim>
__device__ __forceinline__ Entry entry_of(const PagesParams &p, int b)
{
    Entry e = {-1, 0, 0, 0, 0, false};
    if (b >= p.batch) return e;
    const int r = p.rows ? p.rows[b] : b;
    if (r < 0 || r >= p.pool.requests) return e;
    const int most = p.pool.cols * p.pool.page_size;
    const int len = p.pool.lens[r];
    e.row = r;
    if (len < 0 || len > most) {  // (not a length of this pool)
        e.row = -1;
        return e;
    }
    e.len = len;
    e.held = pages_of(len, p.pool.page_size);
    if constexpr (kTrim) {
        int d = len;
        if (p.counts) {
            const int64_t w = p.base < 0 ? p.counts[b] : static_cast<int64_t>(p.base) - p.counts[b];
            d = w < 0 ? 0 : (w > len ? len : static_cast<int>(w));
        }
        e.valid = true;
        e.tokens = len - d;
        e.pages = e.held - pages_of(e.tokens, p.pool.page_size);
    } else {
        const int n = p.counts[b];
        const int room = p.room * p.pool.page_size;
        if (n < 0 || n > room - len) return e;
        e.valid = true;
        e.tokens = n;
        e.pages = pages_of(len + n, p.pool.page_size) - e.held;
    }
    return e;
}

__device__ __forceinline__ long long warp_scan(long long v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}

template <int R>
struct Shared {
    long long warp_a[R / 32], warp_b[R / 32];
    long long before_a, before_b;
    int first[3][R + 1];  // running sums of the range: pages, tokens, table entries
    int row[R], len[R], held[R];
    unsigned last;
};

template <int R>
__device__ __forceinline__ void block_sync()
{
    if constexpr (R > 32) __syncthreads();
    else __syncwarp();
}

template <int R>
__device__ __forceinline__ int block_count(bool pred)
{
    if constexpr (R > 32) return __syncthreads_count(pred);
    else return __popc(__ballot_sync(0xFFFFFFFFu, pred));
}

// Inclusive scans of a and b over the block.
template <int R>
__device__ __forceinline__ void block_scan(Shared<R> &s, long long &a, long long &b)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    a = warp_scan(a, lane);
    b = warp_scan(b, lane);
    if constexpr (R > 32) {
        __syncthreads();  // (the last scan's sums have been read)
        if (lane == 31) {
            s.warp_a[warp] = a;
            s.warp_b[warp] = b;
        }
        __syncthreads();
        const bool in = lane < R / 32;
        const long long wa = warp_scan(in ? s.warp_a[lane] : 0, lane), wb = warp_scan(in ? s.warp_b[lane] : 0, lane);
        const long long ea = __shfl_sync(0xFFFFFFFFu, wa, warp > 0 ? warp - 1 : 0);
        const long long eb = __shfl_sync(0xFFFFFFFFu, wb, warp > 0 ? warp - 1 : 0);
        if (warp > 0) {
            a += ea;
            b += eb;
        }
    }
}

// The last i with first[i] <= x, for x < first[n]: the entry that running index x belongs to.
__device__ __forceinline__ int find(const int *first, int n, int x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Pages and tokens of the granted entries before `range`.
template <int R>
__device__ void sums_before(Shared<R> &s, const PagesParams &p, int range, int free, long long &pages, long long &tokens)
{
    pages = tokens = 0;
    if (range == 0) return;
    long long a = 0, b = 0;
    for (int i = threadIdx.x; i < range * R; i += R) {
        const Entry e = entry_of<false>(p, i);
        if (e.valid) a += e.pages, b += e.tokens;
    }
    block_scan(s, a, b);
    if (threadIdx.x == R - 1) s.before_a = a, s.before_b = b;
    block_sync<R>();
    pages = s.before_a;
    tokens = s.before_b;
    if (pages <= free && tokens <= p.tokens) return;
    // the cut lies before this range: the sums up to it
    pages = tokens = 0;
    for (int r = 0; r < range; ++r) {
        const Entry e = entry_of<false>(p, r * R + static_cast<int>(threadIdx.x));
        long long c = e.valid ? e.pages : 0, d = e.valid ? e.tokens : 0;
        block_scan(s, c, d);
        c += pages;
        d += tokens;
        const bool fits = c <= free && d <= p.tokens;
        const int n = block_count<R>(fits);  // (sums never fall: those that fit come first)
        if (static_cast<int>(threadIdx.x) == n - 1) s.before_a = c, s.before_b = d;
        block_sync<R>();
        if (n > 0) pages = s.before_a, tokens = s.before_b;
        block_sync<R>();
        if (n < R) break;
    }
    // what follows the cut is refused: sums that nothing can be added to
    pages |= 1ll << 62;
}

template <int R>
__global__ void __launch_bounds__(R) pages_extend_kernel(const __grid_constant__ PagesParams p)
{
    __shared__ Shared<R> s;
    pdl_trigger();
    pdl_wait();
    const int t = threadIdx.x, range = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
    const int b = range * R + t, page = p.pool.page_size;
    const int free = min(max(p.pool.counters[0], 0), p.pool.num_pages);
    const Entry e = entry_of<false>(p, b);
    long long pages0, tokens0;
    sums_before(s, p, range, free, pages0, tokens0);
    const bool cut_before = (pages0 >> 62) != 0;
    pages0 &= ~(1ll << 62);
    long long a = e.valid ? e.pages : 0, c = e.valid ? e.tokens : 0;
    block_scan(s, a, c);
    const bool fits = !cut_before && pages0 + a <= free && tokens0 + c <= p.tokens;
    const bool given = fits && e.valid;
    // the granted entries' sums: those of the last one that fits
    const int n_fit = block_count<R>(fits);
    if (t == n_fit - 1) s.before_a = a, s.before_b = c;
    if (t == 0 && n_fit == 0) s.before_a = s.before_b = 0;
    block_sync<R>();
    const int my_pages = static_cast<int>(fits ? a : s.before_a), my_tokens = static_cast<int>(fits ? c : s.before_b);
    const int len = e.len + (given ? e.tokens : 0);
    int entries = 0;
    if (p.table && e.row >= 0) entries = min(pages_of(len, page), p.table_cols);
    long long f = entries, none = 0;
    if (p.table) block_scan(s, f, none);
    s.first[0][t + 1] = my_pages;
    s.first[1][t + 1] = my_tokens;
    s.first[2][t + 1] = static_cast<int>(f);
    if (t < 3) s.first[t][0] = 0;
    s.row[t] = e.row;
    s.len[t] = e.len;
    s.held[t] = e.held;
    block_sync<R>();
    // (this block has read the requests' lengths and the free pages: nobody's reads come after the last block's ticket, and
    // what blocks write is not read by others)
    if (gridDim.x > 1 && t == 0) s.last = atomicAdd(reinterpret_cast<unsigned *>(p.pool.counters + 1), 1u) == gridDim.x - 1;
    const int64_t base_page = free - 1 - pages0;  // the stack's entry of the range's first page
    const int base_token = static_cast<int>(tokens0);
    if (part == 0 && b < p.batch) {
        if (p.cu) {
            p.cu[b + 1] = base_token + my_tokens;
            if (b == 0) p.cu[0] = 0;
        }
        if (p.lens) p.lens[b] = e.row >= 0 ? len : 0;
        if (p.granted) p.granted[b] = given;
    }
    if (p.cu && p.batch == 0 && t == 0 && blockIdx.x == 0) p.cu[0] = 0;

    const int stride = p.parts * R, at0 = part * R + t;
    auto page_at = [&](int i, int col) -> int {  // page `col` of the range's entry i, new or old
        if (col >= s.held[i]) return p.pool.free_pages[base_page - (s.first[0][i] + col - s.held[i])];
        return p.pool.page_table[s.row[i] * p.pool.table_stride + col];
    };
    for (int x = at0; x < s.first[0][R]; x += stride) {
        const int i = find(s.first[0], R, x);
        const int col = s.held[i] + x - s.first[0][i];
        p.pool.page_table[s.row[i] * p.pool.table_stride + col] = p.pool.free_pages[base_page - x];
    }
    for (int x = at0; x < s.first[2][R]; x += stride) {
        const int i = find(s.first[2], R, x);
        const int col = x - s.first[2][i];
        p.table[(range * R + i) * p.table_stride + col] = page_at(i, col);
    }
    if (p.positions || p.slots) {
        for (int x = at0; x < s.first[1][R]; x += stride) {
            const int i = find(s.first[1], R, x);
            const int at = s.len[i] + x - s.first[1][i];
            if (p.positions) p.positions[base_token + x] = at;
            if (p.slots) p.slots[base_token + x] = static_cast<int64_t>(page_at(i, at / page)) * page + at % page;
        }
    }

    // the pool's lengths and free pages, when every block has read them
    block_sync<R>();
    if (gridDim.x > 1 && !s.last) return;
    long long total = 0, done = 0;
    for (int r = 0; r < p.ranges; ++r) {
        const Entry q = r == range ? e : entry_of<false>(p, r * R + t);
        long long g = q.valid ? q.pages : 0, h = q.valid ? q.tokens : 0;
        if (p.ranges > 1) {
            block_scan(s, g, h);
        } else {
            g = a;
            h = c;
        }
        const bool ok = total + g <= free && done + h <= p.tokens;
        const int n = block_count<R>(ok);
        if (t == n - 1) s.before_a = total + g, s.before_b = done + h;
        if (ok && q.valid && q.tokens > 0) p.pool.lens[q.row] = q.len + q.tokens;  // (an entry that pads the batch may name any request)
        block_sync<R>();
        if (n > 0) total = s.before_a, done = s.before_b;
        block_sync<R>();
        if (n < R) break;
    }
    if (t == 0) {
        p.pool.counters[0] = free - static_cast<int>(total);
        p.pool.counters[1] = 0;
    }
}

template <int R>
__global__ void __launch_bounds__(R) pages_trim_kernel(const __grid_constant__ PagesParams p)
{
    __shared__ Shared<R> s;
    pdl_trigger();
    pdl_wait();
    const int t = threadIdx.x, range = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
    const int free = min(max(p.pool.counters[0], 0), p.pool.num_pages);
    const Entry e = entry_of<true>(p, range * R + t);
    long long a = e.pages, none = 0;
    block_scan(s, a, none);
    // pages that the entries before this range give back, and all entries
    if (p.ranges > 1) {
        long long before = 0, all = 0;
        for (int i = t; i < p.ranges * R; i += R) {
            const Entry q = entry_of<true>(p, i);
            all += q.pages;
            if (i < range * R) before += q.pages;
        }
        block_scan(s, before, all);
        if (t == R - 1) s.before_a = before, s.before_b = all;
    } else if (t == R - 1) {
        s.before_a = 0, s.before_b = a;
    }
    block_sync<R>();
    const long long first = s.before_a;
    const int count = static_cast<int>(min(s.before_b, static_cast<long long>(p.pool.num_pages - free)));
    s.first[0][t + 1] = static_cast<int>(a);
    if (t == 0) s.first[0][0] = 0;
    s.row[t] = e.row;
    s.held[t] = e.held - e.pages;  // what is kept
    block_sync<R>();
    // (this block has read the requests' lengths and the free pages; as above)
    if (gridDim.x > 1 && t == 0) s.last = atomicAdd(reinterpret_cast<unsigned *>(p.pool.counters + 1), 1u) == gridDim.x - 1;
    for (int x = part * R + t; x < s.first[0][R]; x += p.parts * R) {
        const int i = find(s.first[0], R, x);
        const long long at = free + count - 1 - (first + x);  // (a pool that is in order has room for all)
        if (at >= free) p.pool.free_pages[at] = p.pool.page_table[s.row[i] * p.pool.table_stride + s.held[i] + x - s.first[0][i]];
    }
    block_sync<R>();
    if (gridDim.x > 1 && !s.last) return;
    for (int r = 0; r < p.ranges; ++r) {
        const Entry q = r == range ? e : entry_of<true>(p, r * R + t);
        if (q.row >= 0 && q.tokens != q.len) p.pool.lens[q.row] = q.tokens;
    }
    if (t == 0) {
        p.pool.counters[0] = free + count;
        p.pool.counters[1] = 0;
    }
}

dflash_status pages_fail(dflash_status st, const char *fmt, long long a = 0, long long b = 0)
{
    char buf[256];
    snprintf(buf, sizeof buf, fmt, a, b);
    return host_fail(st, buf);
}

bool misaligned(const void *p, uintptr_t by)
{
    return reinterpret_cast<uintptr_t>(p) % by != 0;
}

dflash_status check_pool(const dflash_page_pool *q, int32_t batch, const void *rows, const void *counts)
{
    if (!q) return pages_fail(DFLASH_ERR_INVALID_ARG, "pool must not be NULL");
    if (!q->page_table || !q->lens || !q->free_pages || !q->counters)
        return pages_fail(DFLASH_ERR_INVALID_ARG, "the pool's page_table, lens, free_pages and counters must be given");
    if (misaligned(q->page_table, 4) || misaligned(q->lens, 4) || misaligned(q->free_pages, 4) || misaligned(q->counters, 4) ||
        misaligned(rows, 4) || misaligned(counts, 4))
        return pages_fail(DFLASH_ERR_INVALID_ARG, "arrays must be aligned to their type");
    if (q->requests < 1 || q->cols < 1 || q->cols > 1 << 20 || q->page_size < 1 || q->page_size > 65536 || q->num_pages < 1)
        return pages_fail(DFLASH_ERR_INVALID_ARG, "requests and num_pages must be >= 1, cols in [1, 2^20] (got %lld), page_size in [1, 65536] (got %lld)",
                          q->cols, q->page_size);
    if (static_cast<int64_t>(q->cols) * q->page_size >= (int64_t(1) << 31))
        return pages_fail(DFLASH_ERR_INVALID_ARG, "cols * page_size must be below 2^31 (got %lld * %lld)", q->cols, q->page_size);
    if (q->requests > 1 && q->table_stride < q->cols)
        return pages_fail(DFLASH_ERR_INVALID_ARG, "the pool's table_stride must be at least cols = %lld (got %lld)", q->cols, q->table_stride);
    if (batch < 0 || batch > 65536 || batch > q->requests)
        return pages_fail(DFLASH_ERR_INVALID_ARG, "batch must be in [0, 65536] and at most requests = %lld (got %lld)", q->requests, batch);
    return DFLASH_OK;
}

// The pool's arrays, the inputs and the n outputs share nothing; but counts may be the pool's lengths without rows, when an
// entry's number is its own request's length, which is written when every block has read it.
dflash_status check_overlap(const dflash_page_pool &q, const int32_t *rows, const int32_t *counts, int32_t batch, const Rows *outputs, int n)
{
    const Rows pool[] = {{q.lens, q.requests * int64_t(4)},
                         {q.page_table, q.cols * int64_t(4), q.requests, q.table_stride * 4},
                         {q.free_pages, q.num_pages * int64_t(4)},
                         {q.counters, 8}};
    const Rows inputs[] = {{rows, batch * int64_t(4)}, {rows || counts != q.lens ? counts : nullptr, batch * int64_t(4)}};
    bool overlap = false;
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < i; ++j) overlap = overlap || meet(pool[i], pool[j]);
        for (const Rows &in : inputs) overlap = overlap || meet(pool[i], in);
    }
    for (int i = 0; i < n; ++i) {
        for (int j = 0; j < i; ++j) overlap = overlap || meet(outputs[i], outputs[j]);
        for (const Rows &in : inputs) overlap = overlap || meet(outputs[i], in);
        for (const Rows &own : pool) overlap = overlap || meet(outputs[i], own);
        overlap = overlap || folds(outputs[i]);
    }
    return overlap ? pages_fail(DFLASH_ERR_INVALID_ARG, "outputs, inputs and the pool's arrays must not overlap") : DFLASH_OK;
}

// One warp for a batch of up to 32 with little to do, else blocks of 256 or, over 256 entries, of 1024; and as many blocks
// (up to 304) as there are times 512 things to do: 32 requests that get 8192 pages each and then end took 6.3 ms by one warp,
// and take 15 us. Returns a block's threads.
int cut(PagesParams &p, int64_t work)
{
    const int R = p.batch <= 32 && work <= 1024 ? 32 : p.batch <= 256 ? 256 : 1024;
    p.ranges = p.batch > 0 ? (p.batch + R - 1) / R : 1;
    const int64_t most = 304 / p.ranges > 1 ? 304 / p.ranges : 1;
    work = work / 512 / p.ranges + 1;
    p.parts = static_cast<int>(work < most ? work : most);
    return R;
}

// Pages that a call may move if requests change by `tokens` together: rows of the table count as half filled.
int64_t pages_moved(const dflash_page_pool &q, int64_t batch, int64_t tokens)
{
    const int64_t rows = batch * q.cols / 2, by_tokens = tokens / q.page_size + batch;
    return rows < by_tokens ? rows : by_tokens;
}

}  // namespace
}  // namespace dfl

using dfl::pages_fail;

extern "C" dflash_status dflash_pages_extend(const dflash_page_pool *pool, const int32_t *rows, const int32_t *new_tokens,
                                             int32_t batch, int32_t tokens, int32_t *cu_tokens, int32_t *lens,
                                             int32_t *page_table, int64_t table_stride, int32_t table_cols,
                                             int32_t *positions, int64_t *slots, int32_t *granted, void *stream)
{
    dflash_status st = dfl::check_pool(pool, batch, rows, new_tokens);
    if (st != DFLASH_OK) return st;
    if (tokens < 0 || tokens > 1 << 30) return pages_fail(DFLASH_ERR_INVALID_ARG, "tokens must be in [0, 2^30] (got %lld)", tokens);
    if (batch > 0 && !new_tokens) return pages_fail(DFLASH_ERR_INVALID_ARG, "new_tokens must be given");
    if (page_table && (table_cols < 1 || (batch > 1 && table_stride < table_cols)))
        return pages_fail(DFLASH_ERR_INVALID_ARG, "table_cols must be >= 1 and table_stride at least that (got %lld, %lld)", table_cols, table_stride);
    if (dfl::misaligned(cu_tokens, 4) || dfl::misaligned(lens, 4) || dfl::misaligned(page_table, 4) ||
        dfl::misaligned(positions, 4) || dfl::misaligned(slots, 8) || dfl::misaligned(granted, 4))
        return pages_fail(DFLASH_ERR_INVALID_ARG, "outputs must be aligned to their type");
    if (lens == pool->lens) {
        if (rows) return pages_fail(DFLASH_ERR_INVALID_ARG, "lens can be the pool's own only without rows");
        lens = nullptr;
    }
    const int room = page_table && table_cols < pool->cols ? table_cols : pool->cols;
    if (page_table == pool->page_table) {
        if (rows || (batch > 1 && table_stride != pool->table_stride))
            return pages_fail(DFLASH_ERR_INVALID_ARG, "page_table can be the pool's own only without rows and with its stride");
        page_table = nullptr;
    }
    if (batch == 0 && !cu_tokens) return DFLASH_OK;
    const dfl::Rows outputs[] = {{cu_tokens, (batch + 1) * int64_t(4)},
                                 {lens, batch * int64_t(4)},
                                 {page_table, table_cols * int64_t(4), batch, table_stride * 4},
                                 {positions, tokens * int64_t(4)},
                                 {slots, tokens * int64_t(8)},
                                 {granted, batch * int64_t(4)}};
    st = dfl::check_overlap(*pool, rows, new_tokens, batch, outputs, 6);
    if (st != DFLASH_OK) return st;
    dfl::PagesParams p;
    p.pool = *pool;
    p.room = room;
    p.rows = rows;
    p.counts = new_tokens;
    p.batch = batch;
    p.tokens = tokens;
    p.base = -1;
    p.cu = cu_tokens;
    p.lens = lens;
    p.table = page_table;
    p.table_stride = table_stride;
    p.table_cols = page_table ? table_cols : 0;
    p.positions = positions;
    p.slots = slots;
    p.granted = granted;
    int64_t work = positions || slots ? tokens : dfl::pages_moved(*pool, batch, tokens);
    const int64_t copy = page_table ? static_cast<int64_t>(batch) * table_cols / 2 : 0;  // of a separate page table
    if (copy > work) work = copy;
    const int R = dfl::cut(p, work);
    const cudaError_t e = dfl::launch_ex(R == 32    ? dfl::pages_extend_kernel<32>
                                         : R == 256 ? dfl::pages_extend_kernel<256>
                                                    : dfl::pages_extend_kernel<1024>,
                                         dim3(p.ranges * p.parts), dim3(R), 0, static_cast<cudaStream_t>(stream), 1, p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return pages_fail(DFLASH_ERR_CUDA, "the launch failed (error %lld)", e);
    }
    return DFLASH_OK;
}

extern "C" dflash_status dflash_pages_trim(const dflash_page_pool *pool, const int32_t *rows, const int32_t *counts,
                                           int32_t base, int32_t batch, void *stream)
{
    dflash_status st = dfl::check_pool(pool, batch, rows, counts);
    if (st != DFLASH_OK) return st;
    if (batch == 0) return DFLASH_OK;
    st = dfl::check_overlap(*pool, rows, counts, batch, nullptr, 0);
    if (st != DFLASH_OK) return st;
    dfl::PagesParams p = {};
    p.pool = *pool;
    p.rows = rows;
    p.counts = counts;
    p.base = base;
    p.batch = batch;
    const int64_t most = counts && base >= 0 ? static_cast<int64_t>(base) * batch : int64_t(1) << 40;
    const int R = dfl::cut(p, dfl::pages_moved(*pool, batch, most));
    const cudaError_t e = dfl::launch_ex(R == 32    ? dfl::pages_trim_kernel<32>
                                         : R == 256 ? dfl::pages_trim_kernel<256>
                                                    : dfl::pages_trim_kernel<1024>,
                                         dim3(p.ranges * p.parts), dim3(R), 0, static_cast<cudaStream_t>(stream), 1, p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return pages_fail(DFLASH_ERR_CUDA, "the launch failed (error %lld)", e);
    }
    return DFLASH_OK;
}
