// A batch's tables from its requests' lengths: prefix sums over the requests'
// rows and pages, pages off the free list into the block tables, and a map from
// rows to requests, tokens and cache places.
//
// One launch of one thread-block cluster: the requests are shared out over its
// CTAs, whose sums meet through distributed shared memory, so the inputs may be
// overwritten by the outputs once the cluster has read them (ctx_len by
// total_len, free_count by state[1]) and a captured step needs no copies.
//
// Bound by latency: loads, three barriers, the search for a row's request.
// 64 single tokens take 5.4 us, 2,000 requests with drafts of up to 5 tokens 11.4 us, 16
// prompts of up to 4,096 tokens 13 us (of which an empty launch takes about 2.5 us).  A row's search for its
// request goes through shared memory, four rows to a thread; long runs of pages are
// copied by a warp each (by the request's own thread or warp, the 16 prompts took 29 us).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "qsa_device.cuh"
#include "qsa_internal.h"

namespace qsa {
namespace {

namespace cg = cooperative_groups;

constexpr int TB_CTAS = 8, TB_THREADS = 1024, TB_WARPS = TB_THREADS / 32;
// One CTA for small batches: it needs no barriers across the cluster, which cost 3 us
// (64 single tokens 5.4 us, 8.3 with eight CTAs; 1,000 requests with 8,192 rows 9.5, 10.9;
// 2,048 with 8,192 rows 13.0, 11.7; 16 prompts of 16,384 rows 12.1, 9.8; of 65,536 rows
// 34.6, 12.9; 1,024 single tokens 6.7, 9.4; 2,048 8.2, 10.0; 3,000 10.2, 10.5; 4,096
// 12.5, 11.4; 8,192 36, 14).
constexpr int TB_ONE_REQS = 2048, TB_ONE_ROWS = 8192;
constexpr int TB_NEAR = 8191;                    // requests whose starts and positions fit in shared memory

// Rows and pages of a run of requests.  The sums stop at 2^31 - 1, past every limit
// they are compared with.
struct Sum {
    uint32_t rows, pages;
    __device__ __forceinline__ Sum operator+(const Sum &o) const
    {
        return {min(rows + o.rows, 0x7fffffffu), min(pages + o.pages, 0x7fffffffu)};
    }
};

struct TablesShared {
    Sum warps[TB_WARPS], cta;                    // the warps' sums, and the CTA's
    int32_t used;                                // rows in use, if this CTA has the first request that does not fit, else -1
    int32_t n_runs;                              // requests that take many pages:
    int32_t request[TB_THREADS], have[TB_THREADS], fresh[TB_THREADS], from[TB_THREADS];
};

struct Need {
    int32_t n, ctx, have, fresh;                 // new tokens, tokens before, pages before and to come
    bool bad;
};

__device__ __forceinline__ Need need_of(const TablesParams &p, int32_t b)
{
    Need x;
    x.n = p.new_len[b];
    x.ctx = p.ctx_len[b];
    x.bad = x.n < 0 || x.ctx < 0 ||
            static_cast<int64_t>(x.n) + x.ctx > (static_cast<int64_t>(p.max_pages) << p.page_shift);
    if (x.bad) x.n = 0;
    // (sums below 2^31 - 1 + 256 do not pass 32 bits unsigned)
    const uint32_t up = static_cast<uint32_t>(p.page_tokens - 1);
    x.have = x.bad ? 0 : static_cast<int32_t>((static_cast<uint32_t>(x.ctx) + up) >> p.page_shift);
    x.fresh = x.bad ? 0 : static_cast<int32_t>((static_cast<uint32_t>(x.ctx) + static_cast<uint32_t>(x.n) + up) >> p.page_shift) - x.have;
    return x;
}

__device__ __forceinline__ Sum sum_of(const Need &x) { return {static_cast<uint32_t>(x.n), static_cast<uint32_t>(x.fresh)}; }

__device__ __forceinline__ Sum warp_scan_sum(Sum x, int lane)      // inclusive
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sum y = {__shfl_up_sync(0xffffffffu, x.rows, o), __shfl_up_sync(0xffffffffu, x.pages, o)};
        if (lane >= o) x = x + y;
    }
    return x;
}

__device__ __forceinline__ Sum shuffle_up(Sum x, int lane)         // 0 in the first lane
{
    const Sum y = {__shfl_up_sync(0xffffffffu, x.rows, 1), __shfl_up_sync(0xffffffffu, x.pages, 1)};
    return lane > 0 ? y : Sum{0, 0};
}

__device__ __forceinline__ void store4(int32_t *to, int32_t row, int32_t rows, bool vec, const int32_t (&x)[4])
{
    if (!to) return;
    if (vec && row + 4 <= rows) {
        *reinterpret_cast<int4 *>(to + row) = make_int4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (row + i < rows) to[row + i] = x[i];
    }
}

__global__ void __launch_bounds__(TB_THREADS, 1)
tables_kernel(const TablesParams p)
{
    extern __shared__ int32_t near_s[];          // (few requests) their starts, then their positions
    __shared__ TablesShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int ctas = static_cast<int>(cluster.num_blocks()), cta = static_cast<int>(cluster.block_rank());
    const int me = cta * TB_THREADS + t, all = ctas * TB_THREADS;
    const bool near = p.n_reqs <= TB_NEAR;
    int32_t *starts = near_s, *firsts = near_s + p.n_reqs + 1;
    // a run of requests per thread
    const int32_t run = (p.n_reqs + all - 1) / all;
    const int32_t b0 = min(me * run, p.n_reqs), b1 = min(b0 + run, p.n_reqs);
    if (t == 0) sh.used = -1;
    Sum sum = {0, 0};
    for (int32_t b = b0; b < b1; ++b) {
        const Need x = need_of(p, b);
        if (x.bad) record_error(p.status, ST_BAD_ROW);
        sum = sum + sum_of(x);
    }
    const int32_t listed = *p.free_count, avail = max(0, min(listed, p.free_capacity));
    if (me == 0 && avail != listed) record_error(p.status, ST_BAD_ROW);
    const uint32_t max_rows = static_cast<uint32_t>(p.rows), max_pages = static_cast<uint32_t>(avail);
    auto fits = [&](const Sum &x) { return x.rows <= max_rows && x.pages <= max_pages; };
    const Sum upto = warp_scan_sum(sum, lane);
    if (lane == 31) sh.warps[warp] = upto;
    __syncthreads();
    // every warp scans the warps' sums
    const Sum w_upto = warp_scan_sum(sh.warps[lane], lane), w_before = shuffle_up(w_upto, lane);
    static_assert(TB_WARPS == 32, "a lane per warp");
    if (t == 31) sh.cta = w_upto;
    Sum before = Sum{__shfl_sync(0xffffffffu, w_before.rows, warp), __shfl_sync(0xffffffffu, w_before.pages, warp)} + shuffle_up(upto, lane);
    if (ctas > 1) {
        cluster.sync();
        for (int c = 0; c < cta; ++c) before = before + cluster.map_shared_rank(&sh, c)->cta;
    }
    // the first request that does not fit
    auto end_at = [&](const Sum &x, int32_t b) {
        sh.used = static_cast<int32_t>(x.rows);
        p.state[0] = static_cast<int32_t>(x.rows);
        p.state[1] = avail - static_cast<int32_t>(x.pages);
        p.state[2] = b;
    };
    Sum at = before;
    for (int32_t b = b0; b < b1; ++b) {
        const Sum next = at + sum_of(need_of(p, b));
        if (fits(at) && !fits(next)) end_at(at, b);
        at = next;
    }
    if (b1 == p.n_reqs && (b0 < b1 || (p.n_reqs == 0 && me == 0)) && fits(at)) end_at(at, p.n_reqs);
    int32_t used;
    if (ctas > 1) {
        cluster.sync();                          // nobody reads ctx_len or free_count of others any more
        used = 0;
        for (int c = 0; c < ctas; ++c) used = max(used, cluster.map_shared_rank(&sh, c)->used);
    } else {
        __syncthreads();
        used = sh.used;
    }
    // the requests' own entries; long runs of pages by a warp each
    at = before;
    for (int32_t i = 0; i < run; ++i) {
        const int32_t b = b0 + i;
        if (t == 0) sh.n_runs = 0;
        __syncthreads();
        if (b < b1) {
            const Need x = need_of(p, b);
            const Sum next = at + sum_of(x);
            const bool in = fits(next);
            const int32_t start = in ? static_cast<int32_t>(at.rows) : used;
            p.seq_start[b] = start;
            p.pos_start[b] = x.ctx;
            if (p.total_len) p.total_len[b] = x.ctx + (in ? x.n : 0);
            if (near && ctas == 1) {
                starts[b] = start;
                firsts[b] = x.ctx;
            }
            const int32_t fresh = in ? x.fresh : 0, from = avail - 1 - static_cast<int32_t>(at.pages);
            if (fresh > 2) {
                const int32_t k = atomicAdd(&sh.n_runs, 1);
                sh.request[k] = b;
                sh.have[k] = x.have;
                sh.fresh[k] = fresh;
                sh.from[k] = from;
            } else {
                for (int32_t k = 0; k < fresh; ++k)
                    p.block_table[static_cast<int64_t>(b) * p.max_pages + x.have + k] = p.free_pages[from - k];
            }
            at = next;
        }
        __syncthreads();
        for (int32_t k = warp; k < sh.n_runs; k += TB_WARPS) {
            int32_t *to = p.block_table + static_cast<int64_t>(sh.request[k]) * p.max_pages + sh.have[k];
            const int32_t *from = p.free_pages + sh.from[k];
            const int32_t n = sh.fresh[k];
#pragma unroll 8
            for (int32_t e = lane; e < n; e += 32) to[e] = from[-e];
        }
        __syncthreads();
    }
    if (me == 0) p.seq_start[p.n_reqs] = used;
    if (near && t == 0) starts[p.n_reqs] = used;
    if (ctas > 1) {
        cluster.sync();
        if (near) {
            for (int32_t b = t; b < p.n_reqs; b += TB_THREADS) {
                starts[b] = __ldcg(p.seq_start + b);
                firsts[b] = __ldcg(p.pos_start + b);
            }
        }
    }
    __syncthreads();
    // the rows, four to a thread
    auto start_of = [&](int32_t b) { return near ? starts[b] : __ldcg(p.seq_start + b); };
    auto first_of = [&](int32_t b) { return near ? firsts[b] : __ldcg(p.pos_start + b); };
    const bool vec = ((reinterpret_cast<uintptr_t>(p.row_req) | reinterpret_cast<uintptr_t>(p.row_token) |
                       reinterpret_cast<uintptr_t>(p.row_visible) | reinterpret_cast<uintptr_t>(p.slot)) & 15) == 0;
    for (int64_t row64 = static_cast<int64_t>(me) * 4; row64 < p.rows; row64 += 4 * all) {
        const int32_t row = static_cast<int32_t>(row64);
        // the last request that starts at or before the row (padding: the last row's)
        int32_t b = 0, hi = used > 0 ? p.n_reqs : 0;
        while (hi - b > 1) {
            const int32_t mid = (b + hi) >> 1;
            if (start_of(mid) <= min(row, used - 1)) b = mid;
            else hi = mid;
        }
        int32_t req[4], tok[4], vis[4], slot[4], page[4], first = 0, end = 0;
        if (row < used) {
            first = first_of(b) - start_of(b);
            end = start_of(b + 1);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            tok[i] = page[i] = 0;
            if (row + i < used) {
                if (row + i >= end) {                    // the next request that has rows
                    do end = start_of(++b + 1);
                    while (end <= row + i);
                    first = first_of(b) - start_of(b);
                }
                tok[i] = first + row + i;
                if (p.slot) page[i] = __ldcg(p.block_table + static_cast<int64_t>(b) * p.max_pages + (tok[i] >> p.page_shift));
            }
            req[i] = b;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = row + i < used, good = page[i] >= 0 && page[i] <= (INT32_MAX >> p.page_shift);
            vis[i] = in ? static_cast<int32_t>((static_cast<uint32_t>(tok[i]) + 1u) >> 2) : 0;
            slot[i] = in && good ? (page[i] << p.page_shift) + (tok[i] & (p.page_tokens - 1)) : -1;
            if (in && !good) record_error(p.status, ST_BAD_PAGE);
        }
        store4(p.row_req, row, p.rows, vec, req);
        store4(p.row_token, row, p.rows, vec, tok);
        store4(p.row_visible, row, p.rows, vec, vis);
        store4(p.slot, row, p.rows, vec, slot);
    }
}

}  // namespace

int launch_tables(const TablesParams &p, void *stream)
{
    const size_t smem = p.n_reqs <= TB_NEAR ? (2 * static_cast<size_t>(p.n_reqs) + 1) * 4 : 0;
    if (smem > 24 * 1024) {                      // (with the 17 KB of its own, past what a kernel has without asking)
        const cudaError_t e = cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (2 * TB_NEAR + 1) * 4);
        if (e != cudaSuccess) return static_cast<int>(e);
    }
    void *args[] = {const_cast<TablesParams *>(&p)};
    const unsigned ctas = p.n_reqs <= TB_ONE_REQS && p.rows <= TB_ONE_ROWS ? 1 : TB_CTAS;
    return launch_kernel(reinterpret_cast<const void *>(&tables_kernel), dim3(ctas), dim3(TB_THREADS), smem,
                         static_cast<cudaStream_t>(stream), false, args, ctas);
}

}  // namespace qsa
