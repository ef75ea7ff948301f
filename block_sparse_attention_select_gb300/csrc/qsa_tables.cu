// A batch's tables from its requests' lengths: prefix sums over the requests'
// rows and pages, pages off the free list into the block tables, and a map from
// rows to requests, tokens and cache places.
//
// One launch of one thread-block cluster: the requests are shared out over its
// CTAs, whose sums meet through distributed shared memory, so the inputs may be
// overwritten by the outputs once the cluster has read them (ctx_len by
// total_len, free_count by state[1]) and a captured step needs no copies.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "qsa_device.cuh"
#include "qsa_internal.h"

namespace qsa {
namespace {

namespace cg = cooperative_groups;

constexpr int TB_CTAS = 8, TB_THREADS = 1024, TB_WARPS = TB_THREADS / 32;

struct TablesShared {
    int64_t rows[TB_WARPS], pages[TB_WARPS];     // the warps' sums
    int64_t cta_rows, cta_pages;                 // the CTA's
    int32_t used;                                // rows in use, if this CTA has the first request that does not fit, else -1
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

__device__ __forceinline__ int64_t warp_sum_before(int64_t x, int lane, int64_t *all)
{
    int64_t sc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, sc, o);
        if (lane >= o) sc += y;
    }
    *all = __shfl_sync(0xffffffffu, sc, 31);
    return sc - x;
}

__global__ void __cluster_dims__(TB_CTAS, 1, 1) __launch_bounds__(TB_THREADS, 1)
tables_kernel(const TablesParams p)
{
    __shared__ TablesShared sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int cta = static_cast<int>(cluster.block_rank()), me = cta * TB_THREADS + t;
    // a run of requests per thread
    const int32_t run = (p.n_reqs + TB_CTAS * TB_THREADS - 1) / (TB_CTAS * TB_THREADS);
    const int32_t b0 = min(me * run, p.n_reqs), b1 = min(b0 + run, p.n_reqs);
    if (t == 0) sh.used = -1;
    int64_t rows = 0, pages = 0;
    for (int32_t b = b0; b < b1; ++b) {
        const Need x = need_of(p, b);
        if (x.bad) record_error(p.status, ST_BAD_ROW);
        rows += x.n;
        pages += x.fresh;
    }
    const int32_t listed = *p.free_count, avail = max(0, min(listed, p.free_capacity));
    if (me == 0 && avail != listed) record_error(p.status, ST_BAD_ROW);
    int64_t warp_rows, warp_pages;
    rows = warp_sum_before(rows, lane, &warp_rows);
    pages = warp_sum_before(pages, lane, &warp_pages);
    if (lane == 0) {
        sh.rows[warp] = warp_rows;
        sh.pages[warp] = warp_pages;
    }
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        rows += sh.rows[w];
        pages += sh.pages[w];
    }
    if (t == 0) {
        int64_t r = 0, g = 0;
        for (int w = 0; w < TB_WARPS; ++w) {
            r += sh.rows[w];
            g += sh.pages[w];
        }
        sh.cta_rows = r;
        sh.cta_pages = g;
    }
    cluster.sync();
    for (int c = 0; c < cta; ++c) {
        const TablesShared *o = cluster.map_shared_rank(&sh, c);
        rows += o->cta_rows;
        pages += o->cta_pages;
    }
    // the first request that does not fit
    int64_t r = rows, g = pages;
    for (int32_t b = b0; b < b1; ++b) {
        const Need x = need_of(p, b);
        if (r <= p.rows && g <= avail && (r + x.n > p.rows || g + x.fresh > avail)) {
            sh.used = static_cast<int32_t>(r);
            p.state[0] = static_cast<int32_t>(r);
            p.state[1] = avail - static_cast<int32_t>(g);
            p.state[2] = b;
        }
        r += x.n;
        g += x.fresh;
    }
    if (b1 == p.n_reqs && (b0 < b1 || (p.n_reqs == 0 && me == 0)) && r <= p.rows && g <= avail) {
        sh.used = static_cast<int32_t>(r);
        p.state[0] = static_cast<int32_t>(r);
        p.state[1] = avail - static_cast<int32_t>(g);
        p.state[2] = p.n_reqs;
    }
    cluster.sync();
    int32_t used = 0;
    for (int c = 0; c < TB_CTAS; ++c) used = max(used, cluster.map_shared_rank(&sh, c)->used);
    // the requests' own entries; a warp takes its lanes' long runs of pages together
    r = rows;
    g = pages;
    const int32_t most = __reduce_max_sync(0xffffffffu, b1 - b0);
    for (int32_t i = 0; i < most; ++i) {
        const int32_t b = b0 + i;
        Need x{0, 0, 0, 0, false};
        bool fits = false;
        if (b < b1) {
            x = need_of(p, b);
            fits = r + x.n <= p.rows && g + x.fresh <= avail;
            p.seq_start[b] = fits ? static_cast<int32_t>(r) : used;
            p.pos_start[b] = x.ctx;
            if (p.total_len) p.total_len[b] = x.ctx + (fits ? x.n : 0);
        }
        const int32_t fresh = fits ? x.fresh : 0, at = fits ? avail - 1 - static_cast<int32_t>(g) : 0;
        if (fresh > 0 && fresh <= 2)
            for (int32_t k = 0; k < fresh; ++k)
                p.block_table[static_cast<int64_t>(b) * p.max_pages + x.have + k] = p.free_pages[at - k];
        for (uint32_t many = __ballot_sync(0xffffffffu, fresh > 2); many; many &= many - 1) {
            const int src = __ffs(many) - 1;
            const int32_t n = __shfl_sync(0xffffffffu, fresh, src), from = __shfl_sync(0xffffffffu, at, src);
            const int64_t to = static_cast<int64_t>(__shfl_sync(0xffffffffu, b, src)) * p.max_pages + __shfl_sync(0xffffffffu, x.have, src);
            for (int32_t k = lane; k < n; k += 32) p.block_table[to + k] = p.free_pages[from - k];
        }
        r += x.n;
        g += x.fresh;
    }
    if (me == 0) p.seq_start[p.n_reqs] = used;
    __threadfence();
    cluster.sync();
    // the rows
    for (int32_t row = me; row < p.rows; row += TB_CTAS * TB_THREADS) {
        int32_t tok = 0, vis = 0, slot = -1;
        int32_t b = 0, hi = used > 0 ? p.n_reqs : 0;     // the last request that starts at or before the row
        while (hi - b > 1) {
            const int32_t mid = (b + hi) >> 1;
            if (__ldcg(p.seq_start + mid) <= min(row, used - 1)) b = mid;
            else hi = mid;
        }
        if (row < used) {
            tok = __ldcg(p.pos_start + b) + (row - __ldcg(p.seq_start + b));
            vis = static_cast<int32_t>((static_cast<uint32_t>(tok) + 1u) >> 2);
            if (p.slot) {
                const int32_t page = __ldcg(p.block_table + static_cast<int64_t>(b) * p.max_pages + (tok >> p.page_shift));
                if (page >= 0 && page <= (INT32_MAX >> p.page_shift)) slot = (page << p.page_shift) + (tok & (p.page_tokens - 1));
                else record_error(p.status, ST_BAD_PAGE);
            }
        }
        if (p.row_req) p.row_req[row] = b;
        if (p.row_token) p.row_token[row] = tok;
        if (p.row_visible) p.row_visible[row] = vis;
        if (p.slot) p.slot[row] = slot;
    }
}

}  // namespace

int launch_tables(const TablesParams &p, void *stream)
{
    void *args[] = {const_cast<TablesParams *>(&p)};
    return launch_kernel(reinterpret_cast<const void *>(&tables_kernel), dim3(TB_CTAS), dim3(TB_THREADS), 0,
                         static_cast<cudaStream_t>(stream), false, args);
}

}  // namespace qsa
