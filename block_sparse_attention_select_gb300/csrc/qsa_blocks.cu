// Attention of new tokens over the blocks of 128 tokens selected for them.
//
// A unit of work is as many whole tokens of one request as have 256 (token, query
// head) pairs (16 where rows are few), for one KV head.  The kernel here turns the
// rows' selections into a list of blocks per unit, those that some row attends,
// with a row of bits per token; the kernels of dense attention then go through
// the lists instead of a run of tiles (qsa_chunk_pair.cuh, qsa_chunk_rows.cuh).
// Neighbouring tokens select much the same blocks, so a unit reads a block once
// for all of its tokens and the products stay dense; a row that does not attend a
// tile gives it zero weights.  (Reading each row's blocks for itself, the 1,616-row
// chunk would bring 3.6 GB from the L2 cache.)
//
// Bound by latency: a chunk's lists take 7 us, those of four prompts of 8,192 tokens 24
// (under the profiler, with cold caches), before attention of 140 and 1,120 us.  Single
// tokens need no lists (qsa_chunk_rows.cuh).
#include "qsa_chunk_pair.cuh"
#include "qsa_chunk_rows.cuh"

namespace qsa {
namespace {

constexpr int LS_THREADS = 128, LS_WARPS = LS_THREADS / 32;
constexpr int BLOCK_SHIFT = 7;
static_assert(1 << BLOCK_SHIFT == BLOCK_TOKENS, "block");

struct ListsParams {
    KvParams kv;
    const int32_t *sel;
    int32_t *counts, *lists;
    uint32_t *bits;
    int32_t k, recent, list_stride, words, unit_tokens;
    int32_t window;              // rows of a CTA
    int32_t map_words;           // words of a bit per block
};

// A CTA looks for the units that begin among its rows and makes their lists for
// one KV head: the union of the selections as a bitmap, its set bits in order, and
// each selection's place among them.
__global__ void __launch_bounds__(LS_THREADS)
lists_kernel(const ListsParams p)
{
    extern __shared__ uint32_t map[];                       // a bit per block, then the bits before each word
    int32_t *before = reinterpret_cast<int32_t *>(map + p.map_words);
    __shared__ int32_t n_units, u_row[LS_THREADS], u_n[LS_THREADS], u_pos[LS_THREADS];
    __shared__ int32_t late[3];                             // last visible token of the blocks from the first token's on
    __shared__ int32_t warp_sum[LS_WARPS];
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int32_t g = blockIdx.y;
    if (t == 0) n_units = 0;
    wait_prior_grid();
    allow_next_grid();                                      // the attention's CTAs wait for the lists on the device
    if (blockIdx.x == 0 && g == 0) flag_bad_requests(p.kv);
    const int32_t row0 = blockIdx.x * p.window;
    Seq s;
    const int32_t b = requests_of_rows(p.kv, row0, min(p.window, p.kv.rows - row0), &s);
    if (b >= 0 && (row0 + t - s.s0) % p.unit_tokens == 0) {
        const int32_t i = atomicAdd(&n_units, 1), tok = row0 + t - s.s0;
        u_row[i] = row0 + t;
        u_n[i] = min(p.unit_tokens, s.n - tok);
        u_pos[i] = s.p0 + tok;
    }
    __syncthreads();
    const int32_t n = n_units;
    for (int32_t i = 0; i < n; ++i) {
        const int32_t r0 = u_row[i], toks = u_n[i], p0 = u_pos[i];
        const int32_t first = p0 >> BLOCK_SHIFT, last = (p0 + toks - 1) >> BLOCK_SHIFT, words = (last >> 5) + 1;
        const int64_t unit = static_cast<int64_t>(g) * p.kv.rows + r0;
        const int32_t *sel = p.sel + (static_cast<int64_t>(r0) * p.kv.hkv + g) * p.k;
        const int64_t step = static_cast<int64_t>(p.kv.hkv) * p.k;
        const int32_t names = toks * p.k;
        const int32_t recent0 = max(0, first - p.recent + 1);                // the last blocks of some token begin here
        for (int32_t w = t; w < words; w += LS_THREADS) {
            uint32_t m = 0;
            if (p.recent > 0 && 32 * w + 31 >= recent0) {
                m = 32 * w >= recent0 ? ~0u : ~0u << (recent0 & 31);
                if (w == words - 1) m &= ~0u >> (31 - (last & 31));
            }
            map[w] = m;
        }
        if (t < 3) late[t] = -1;
        __syncthreads();
        for (int32_t e = t; e < names; e += LS_THREADS) {
            const int32_t tok = e / p.k, c = __ldg(sel + tok * step + (e - tok * p.k)), pos = p0 + tok;
            if (c >= 0 && c <= pos >> BLOCK_SHIFT) {
                atomicOr(&map[c >> 5], 1u << (c & 31));
                if (c >= first) atomicMax(&late[c - first], min(pos - (c << BLOCK_SHIFT), BLOCK_TOKENS - 1));
            } else if (c != -1) {
                record_error(p.kv.status, ST_BAD_ROW);
            }
        }
        if (p.recent > 0)
            for (int32_t tok = t; tok < toks; tok += LS_THREADS) {
                const int32_t pos = p0 + tok, own = pos >> BLOCK_SHIFT;
                for (int32_t c = max(first, own - p.recent + 1); c <= own; ++c)
                    atomicMax(&late[c - first], min(pos - (c << BLOCK_SHIFT), BLOCK_TOKENS - 1));
            }
        __syncthreads();
        // the set bits before each word
        const int32_t run = (words + LS_THREADS - 1) / LS_THREADS, w0 = min(t * run, words), w1 = min(w0 + run, words);
        int32_t sum = 0;
        for (int32_t w = w0; w < w1; ++w) sum += __popc(map[w]);
        const int32_t upto = warp_scan(sum, lane);
        if (lane == 31) warp_sum[warp] = upto;
        __syncthreads();
        int32_t at = upto - sum, count = 0;
#pragma unroll
        for (int w = 0; w < LS_WARPS; ++w) {
            if (w < warp) at += warp_sum[w];
            count += warp_sum[w];
        }
        int32_t *list = p.lists + unit * p.list_stride;
        for (int32_t w = w0; w < w1; ++w) {
            before[w] = at;
            for (uint32_t m = map[w]; m; m &= m - 1) {
                const int32_t c = 32 * w + __ffs(m) - 1;
                list[at++] = c | (c < first ? BLOCK_TOKENS - 1 : late[c - first]) << 24;
            }
        }
        if (t == 0) {
            p.counts[unit] = max(count, 1);
            if (count == 0) list[0] = NO_BLOCK;
        }
        // the tokens' bits
        const int32_t used = (max(count, 1) + 31) >> 5;
        for (int32_t e = t; e < toks * used; e += LS_THREADS) {
            const int32_t tok = e / used;
            p.bits[(unit + tok) * p.words + (e - tok * used)] = 0u;
        }
        __syncthreads();
        auto attend = [&](int32_t tok, int32_t c) {
            const int32_t at = before[c >> 5] + __popc(map[c >> 5] & ((1u << (c & 31)) - 1u));
            atomicOr(p.bits + (unit + tok) * p.words + (at >> 5), 1u << (at & 31));
        };
        for (int32_t e = t; e < names; e += LS_THREADS) {
            const int32_t tok = e / p.k, c = __ldg(sel + tok * step + (e - tok * p.k));
            if (c >= 0 && c <= (p0 + tok) >> BLOCK_SHIFT) attend(tok, c);
        }
        if (p.recent > 0)
            for (int32_t tok = t; tok < toks; tok += LS_THREADS) {
                const int32_t own = (p0 + tok) >> BLOCK_SHIFT;
                for (int32_t c = max(0, own - p.recent + 1); c <= own; ++c) attend(tok, c);
            }
        __syncthreads();
    }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// What the lists of a call take, behind the workspace of the attention kernels.
struct ListSizes {
    int32_t blocks, stride, entries, words;      // blocks of a request; entries a token, and a unit, adds at most; words of a token's bits
    size_t counts_at, lists_at, bits_at, bytes;

    ListSizes(int32_t rows, int32_t group, int32_t hkv, int32_t head_dim, int32_t k, int32_t recent, int32_t row_capacity, int32_t unit_tokens)
    {
        blocks = (row_capacity + BLOCK_TOKENS - 1) / BLOCK_TOKENS;
        stride = std::max(1, std::min(k + recent, blocks));
        entries = static_cast<int32_t>(std::min<int64_t>(static_cast<int64_t>(unit_tokens) * stride, std::max(1, blocks)));
        words = (entries + 31) / 32;
        const size_t n = static_cast<size_t>(rows) * hkv;
        counts_at = up256(std::max(chunk_workspace_bytes(rows, group, head_dim), chunk_rows_workspace_bytes(rows, group, head_dim)));
        lists_at = counts_at + up256(4 * n);
        bits_at = lists_at + up256(4 * (n * stride + entries));
        bytes = bits_at + up256(4 * n * words);
    }
};

int32_t pair_tokens(int32_t group) { return CH_ROWS / group; }

}  // namespace

size_t blocks_workspace_bytes(int32_t rows, int32_t group, int32_t hkv, int32_t head_dim, int32_t k, int32_t recent, int32_t row_capacity)
{
    return ListSizes(rows, group, hkv, head_dim, k, recent, row_capacity, pair_tokens(group)).bytes;
}

int launch_blocks(const BlocksParams &in, bool few_rows, const void *tk, const void *tv, int sms, bool overlap, void *stream,
                  int *launches)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    ChunkParams c = in.c;
    const KvParams &kv = c.kv;
    // Few rows whose units would be single tokens: no lists, no join.
    if (few_rows && in.k + in.recent <= DIRECT_BLOCKS && (c.group > CR_ROWS / 2 || kv.rows <= kv.n_reqs)) {
        const int32_t units = kv.rows * kv.hkv;              // (below 2^31: rows * hq is)
        c.sel = in.sel;
        c.sel_k = in.k;
        c.recent = in.recent;
        *launches = 1;
        if (kv.head_dim == 128)
            return kv.e4m3 ? launch_direct<128, true>(c, tk, tv, units, sms, st) : launch_direct<128, false>(c, tk, tv, units, sms, st);
        return kv.e4m3 ? launch_direct<256, true>(c, tk, tv, units, sms, st) : launch_direct<256, false>(c, tk, tv, units, sms, st);
    }
    *launches = 3;
    c.unit_tokens = few_rows ? CR_ROWS / c.group : pair_tokens(c.group);
    const int32_t capacity = kv.max_pages * kv.page_tokens;
    const ListSizes place(kv.rows, c.group, kv.hkv, kv.head_dim, in.k, in.recent, capacity, pair_tokens(c.group));
    const ListSizes z(kv.rows, c.group, kv.hkv, kv.head_dim, in.k, in.recent, capacity, c.unit_tokens);
    ListsParams l;
    l.kv = kv;
    l.sel = in.sel;
    l.k = in.k;
    l.recent = in.recent;
    l.counts = reinterpret_cast<int32_t *>(c.ws + place.counts_at);
    l.lists = reinterpret_cast<int32_t *>(c.ws + place.lists_at);
    l.bits = reinterpret_cast<uint32_t *>(c.ws + place.bits_at);
    l.list_stride = z.stride;
    l.words = z.words;
    l.unit_tokens = c.unit_tokens;
    l.map_words = (z.blocks + 31) / 32;
    // few rows to a CTA while CTAs are few
    const int64_t each = static_cast<int64_t>(kv.rows) * kv.hkv / (8 * sms);
    l.window = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>({each, c.unit_tokens, LS_THREADS})));
    c.counts = l.counts;
    c.lists = l.lists;
    c.bits = l.bits;
    c.list_stride = l.list_stride;
    c.words = l.words;
    c.max_entries = z.entries;
    c.ws_rows = few_rows ? chunk_rows_part_rows(kv.rows, c.group) : chunk_part_rows(kv.rows, c.group);

    const size_t smem = size_t{8} * l.map_words;
    if (smem > 40 * 1024) {                      // (with the 2 KB of its own, past what a kernel has without asking)
        const cudaError_t e = cudaFuncSetAttribute(lists_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(BLOCKS_MAX_TOKENS / BLOCK_TOKENS / 32 * 8));
        if (e != cudaSuccess) return static_cast<int>(e);
    }
    void *args[] = {&l};
    const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(kv.rows) + l.window - 1) / l.window), static_cast<unsigned>(kv.hkv));
    const int rc = launch_kernel(reinterpret_cast<const void *>(&lists_kernel), grid, dim3(LS_THREADS), smem, st, false, args);
    if (rc != 0) return rc;
    return few_rows ? launch_rows_for<BlockRowsGeometry>(c, tk, tv, sms, overlap, true, st)
                    : launch_pairs_for<BlockPairGeometry>(c, tk, tv, sms, overlap, true, st);
}

}  // namespace qsa
