// Attention over the paged K/V cache for few rows, decode tokens: the kernel of dense
// attention (qsa_chunk_rows.cu) and of attention over selected blocks (qsa_blocks.cu).
//
// The mathematics is that of qsa_chunk_pair.cuh; here a unit is 16 (token, query
// head) pairs of one request and KV head, so the cache's bytes are the cost and
// the work is to keep them coming.  Every CTA (one per SM) shares in the line of
// 64-token tiles (qsa_chunk.cuh); a loader warp keeps a ring of stages full by
// TMA, page piece by page piece, and eight warps compute, four to a stage, 16
// tokens each, with warp-level matrix products (m16n8k16) straight from the
// loaded bytes:
//   S[16 rows, 8 tokens] = Q . K^T,  O[16 rows, 8 dims] += P . V
// Each warp keeps its own maxima, sums and output in registers (no barrier
// inside a segment); the eight are added up at a segment's end.
//
// Why not the tcgen05 kernel: from the E4M3 cache its tiles have to be written
// back to shared memory as FP16 before the products can read them, three times
// the loaded bytes through a port that the MMA operands need too (64 requests' tokens
// over 16,384: 349 us, 177 here).  Here a thread turns the codes that it loads into operand
// registers.  The order of the dimensions inside a product is free, as long as
// both operands agree, so each thread takes 16 contiguous bytes of a token:
//   K: thread (r, q) = (lane / 4, lane % 4) reads piece 2 q + (i & 1) of 128-byte
//      chunk i / 2 of token r; its consecutive fours of dims are the four k
//      places that the thread owns in consecutive products;
//   V: thread (r, q) reads piece r of chunk i of tokens 2 q, 2 q + 1, 2 q + 8 and
//      2 q + 9; byte permutes pair up two tokens' values of a dim.
// With the 128-byte swizzle both patterns touch all banks evenly.
//
// Bound by the loads: 64 requests' tokens over up to 32,768 tokens take 290 to 299 us
// from the FP16 cache (6.5 to 6.7 TB/s) and 166 us from the E4M3 cache (6.4 TB/s; its scales
// are single bytes 2 x hkv apart).  One token over 4,096 takes 14 us: the launch,
// the search for its work, one memory latency each for table, keys and join.
//
// Over selected blocks the tiles are halves of the blocks of a unit's list, or (DIRECT)
// of one token's selection of up to 32 blocks: then the scheduler warp reads the
// selection itself, hands out whole (row, KV head) units without a search for work, and
// while units are few a cluster of CTAs shares each, its sums joined through
// distributed shared memory: no lists, no workspace, one launch.  16 of 1,440 blocks for
// one token, 24 query heads over 2 KV heads of 128: 9.3 us (through lists and a join
// 15.7).  64 tokens: 27 us (42) in a graph of equal calls, where most of their 135 MB
// stay in the L2 cache, 29 in a stream of calls, 4.5 TB/s.  200 tokens from the E4M3 cache, 256-wide heads: 92 us (125 before the
// lookups went piece by piece; 94 in a stream), 400 units in three rounds of 152.
#pragma once
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "qsa_chunk.cuh"

namespace qsa {
namespace {

constexpr int CR_ROWS = 16;
constexpr int CR_TILE = 64;                  // tokens of a stage
constexpr int CR_COMP = 8;                   // computing warps
constexpr int CR_LOAD = 8, CR_SCHED = 9, CR_SCALE = 10;   // CR_SCALE: K's scales, the next warp V's (E4M3)
constexpr int CR_WARPS = 12;
constexpr int CR_THREADS = 32 * CR_WARPS;
constexpr int CR_MAX_STAGES = 8;
constexpr int BAR_COMP = 1;

struct RowsGeometry {
    static constexpr bool BLOCKS = false;
    static constexpr bool RAW_MAX = true;    // the parts' maxima: scores before the scale
    static constexpr bool DIRECT = false;
    static constexpr int ROWS = CR_ROWS, TILE = CR_TILE, UNIT_COST = 4, MIN_SHARE = 3, THREADS = CR_THREADS, WARPS = CR_WARPS,
                         WORKERS = CHUNK_MAX_CTAS;
};
struct BlockRowsGeometry : RowsGeometry {
    static constexpr bool BLOCKS = true;
};
// Blocks taken straight from the selections: a unit is one row and KV head, on a
// cluster of p.split CTAs that share its tiles.
struct DirectRowsGeometry : BlockRowsGeometry {
    static constexpr bool DIRECT = true;
};
constexpr int DIRECT_BLOCKS = 32;            // blocks of a unit at most, a lane each
constexpr int DIRECT_SPLIT = 8;              // CTAs of a cluster at most

// A unit's list of blocks, 32 entries in the lanes and the next 32 on their way;
// a tile (two to a block) is asked for no more than 32 blocks ahead of advance().
struct ListWindow {
    const int32_t *list;
    int32_t n, base, cur, next;

    __device__ __forceinline__ void start(const ChunkParams &p, const Seg &w, int lane)
    {
        list = list_of(p, w);
        n = (w.j0 + w.n + 1) >> 1;
        base = w.j0 >> 1;
        cur = base + lane < n ? __ldg(list + base + lane) : NO_BLOCK;
        next = base + 32 + lane < n ? __ldg(list + base + 32 + lane) : NO_BLOCK;
    }
    __device__ __forceinline__ void start(int32_t entry)       // a lane's, of the whole list
    {
        n = 0;
        base = 0;
        cur = entry;
        next = NO_BLOCK;
    }
    __device__ __forceinline__ void advance(int32_t tile, int lane)
    {
        if ((tile >> 1) < base + 32) return;
        base += 32;
        cur = next;
        next = base + 32 + lane < n ? __ldg(list + base + 32 + lane) : NO_BLOCK;
    }
    __device__ __forceinline__ int32_t entry(int32_t tile) const
    {
        const int32_t e = (tile >> 1) - base;
        const int32_t a = __shfl_sync(0xffffffffu, cur, e & 31), b = __shfl_sync(0xffffffffu, next, e & 31);
        return e < 32 ? a : b;
    }
};

// Of a tile: how many of its tokens some row attends.
__device__ __forceinline__ int32_t tile_seen(int32_t entry, int32_t tile)
{
    return entry_seen(entry) - (tile & 1) * CR_TILE;
}

// Where the tiles of a segment lie in the cache, piece by piece (a piece: the tokens
// of a tile that are in one page).  The lanes look up the pieces of `batch` tiles at
// a time, the pages one batch ahead.  (Looked up tile by tile, a lane per token, the
// lookups took 1,500 clocks a stage, more than its bytes.  They have no branch around
// a load: the compiler would wait for it where the branch ends.)
template <typename G>
struct PieceRows {
    ListWindow win;
    const int32_t *bt;
    int32_t batch, off, tok, page, row;
    int sh, ld;

    // the lane's token of tiles j .. j + batch - 1, or -1: its piece is not attended
    __device__ __forceinline__ int32_t token_of(const ChunkParams &p, const Seg &w, int32_t j, int lane) const
    {
        const int32_t at = j + (lane >> ld), tile = w.j0 + at;
        if constexpr (G::BLOCKS) {
            const int32_t e = win.entry(tile), t = entry_block(e) * BLOCK_TOKENS + (tile & 1) * CR_TILE + off;
            return at < w.n && off < tile_seen(e, tile) && t >> p.kv.page_shift < p.kv.max_pages ? t : -1;
        }
        const int32_t t = tile * CR_TILE + off;
        return at < w.n && t <= w.hi_tok && t + (1 << sh) > w.lo_tok ? t : -1;
    }
    __device__ __forceinline__ void look_up(const ChunkParams &p, const Seg &w, int32_t j, int lane)
    {
        tok = token_of(p, w, j, lane);
        page = __ldg(bt + (max(tok, 0) >> p.kv.page_shift));
    }
    // (win has been started, for lists)
    __device__ __forceinline__ void start(const ChunkParams &p, const Seg &w, int lane)
    {
        sh = __ffs(min(p.kv.page_tokens, CR_TILE)) - 1;
        ld = 6 - sh;
        batch = 32 >> ld;
        off = (lane & ((1 << ld) - 1)) << sh;
        bt = p.kv.block_table + static_cast<int64_t>(w.b) * p.kv.max_pages;
        look_up(p, w, 0, lane);
    }
    // for each tile in turn, before piece() and entry(); bad pages are reported by one role
    __device__ __forceinline__ void tile(const ChunkParams &p, const Seg &w, int32_t j, int lane, bool report)
    {
        if (G::BLOCKS) win.advance(w.j0 + j, lane);
        if ((j & (batch - 1)) != 0) return;
        const bool in = static_cast<uint32_t>(page) < static_cast<uint32_t>(p.kv.num_pages);
        if (report && tok >= 0 && !in) record_error(p.kv.status, ST_BAD_PAGE);
        // the row past the cache reads zeros
        row = tok >= 0 && in ? (page << p.kv.page_shift) + (tok & (p.kv.page_tokens - 1)) : p.kv.num_pages << p.kv.page_shift;
        look_up(p, w, j + batch, lane);
    }
    // the cache row of the tile's piece d (may differ by lane)
    __device__ __forceinline__ int32_t piece(int32_t j, int32_t d) const
    {
        return __shfl_sync(0xffffffffu, row, ((j & (batch - 1)) << ld) + d);
    }
};
static_assert(CR_TILE == 64, "pieces of a tile");

template <int D, bool Q8>
struct RowShape {
    static constexpr int ES = Q8 ? 1 : 2;
    static constexpr uint32_t HALF = CR_TILE * D * ES, STAGE = 2 * HALF;   // K, then V
    static constexpr uint32_t SUM1 = CR_ROWS * D * 4;                      // an eighth of the eight warps' outputs
    // an even number of stages: a stage then belongs to one group of warps, which
    // waits for each of its phases (a parity wait must not skip one)
    static constexpr uint32_t QF = CR_ROWS * D * 2;                        // queries as A operands
    static constexpr int FIT = (227 * 1024 - 8192 - SUM1 - QF) / STAGE, NS = (FIT < CR_MAX_STAGES ? FIT : CR_MAX_STAGES) & ~1;
    // the warps' outputs are added up in 8 / SUMS steps, as few as there is room for
    static constexpr uint32_t ROOM = (227 * 1024 - 8192 - QF - NS * STAGE) / SUM1;
    static constexpr int SUMS = ROOM >= 8 ? 8 : ROOM >= 4 ? 4 : ROOM >= 2 ? 2 : 1;
    static constexpr uint32_t SUM = SUMS * SUM1;
    static constexpr int CHUNKS = D * ES / 128;                            // 128-byte chunks of a vector
    static constexpr int PD = 16 / ES;                                     // dims of a 16-byte piece
};

struct RowCtrl {
    SegRing segs;
    uint64_t full[CR_MAX_STAGES], empty[CR_MAX_STAGES];
    Share share;
    float scale[CR_MAX_STAGES][2][CR_TILE];  // K and V scales of a stage's tokens (E4M3)
    float m[CR_COMP][CR_ROWS], l[CR_COMP][CR_ROWS];
    int32_t entry[CR_MAX_STAGES];            // list entry of a stage's tile
    int32_t blocks[SEGS][DIRECT_BLOCKS];     // list of a segment of the ring (DIRECT)
    float2 part[CR_ROWS];                    // the CTA's maxima and sums, for its cluster (DIRECT)
    int32_t abort;
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint4 &a, uint32_t b0, uint32_t b1)
{
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// four codes -> two pairs of FP16
__device__ __forceinline__ void e4m3x4_to_half(uint32_t u, uint32_t *lo, uint32_t *hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(*lo), "=r"(*hi)
        : "r"(u));
}

__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

__device__ __forceinline__ uint4 lds128(const uint8_t *a) { return *reinterpret_cast<const uint4 *>(a); }

// The scheduler warp of a DIRECT kernel: units in the order (row, KV head), one
// after the other to the clusters in turn.  A lane holds one of the row's blocks.
__device__ __forceinline__ void schedule_direct(const ChunkParams &p, RowCtrl &c, int lane)
{
    const int32_t split = p.split, rank = blockIdx.x % split, clusters = gridDim.x / split;
    const int32_t units = p.kv.rows * p.kv.hkv;
    int falls = -1;                          // whether starts fall somewhere (-1: not known)
    uint32_t i = 0;
    // place: the entry's place in the list
    auto give = [&](const Seg &x, int32_t place, int32_t entry) {
        const uint32_t k = i % SEGS;
        if (i >= SEGS) mbar_wait_bounded(&c.segs.empty[k], (i / SEGS - 1) & 1u, SEG_WAIT_NS);
        __syncwarp();
        c.blocks[k][lane] = NO_BLOCK;
        __syncwarp();
        if (place >= 0) c.blocks[k][place] = entry;
        if (lane == 0) c.segs.seg[k] = x;
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.segs.full[k]);
        ++i;
    };
    Seg x;
    for (int32_t u = blockIdx.x / split; u < units; u += clusters) {
        const int32_t row = u / p.kv.hkv;
        const int32_t named = lane < p.sel_k ? __ldg(p.sel + static_cast<int64_t>(u) * p.sel_k + lane) : NO_BLOCK;
        Seq s;
        const int32_t b = request_of_by_warp(p.kv, row, lane, &falls, &s);
        if (b < 0) continue;
        x.g = u - row * p.kv.hkv;
        const int32_t tok = row - s.s0, pos = s.p0 + tok, own = pos / BLOCK_TOKENS;
        int32_t block = NO_BLOCK;
        if (lane < p.sel_k) {
            block = named;
            if (block < -1 || block > own) {
                record_error(p.kv.status, ST_BAD_ROW);
                block = NO_BLOCK;
            }
        } else if (lane < p.sel_k + p.recent) {
            block = max(NO_BLOCK, own - (lane - p.sel_k));
        }
        // each block once, without gaps
        const uint32_t same = __match_any_sync(0xffffffffu, block);
        const bool kept = block >= 0 && __ffs(same) - 1 == lane;
        const uint32_t all = __ballot_sync(0xffffffffu, kept);
        const int32_t count = max(1, __popc(all));
        // the CTA's share of the tiles: may be none
        const int32_t tiles = count * (BLOCK_TOKENS / CR_TILE);
        x.j0 = tiles * rank / split;
        x.n = tiles * (rank + 1) / split - x.j0;
        x.b = b;
        x.s0 = s.s0;
        x.p0 = s.p0;
        x.v0 = tok * p.group;
        x.rows = p.group;
        x.lo_tok = 0;
        x.hi_tok = pos;
        x.place = -1;
        give(x, kept ? __popc(all & ((1u << lane) - 1u)) : -1, block | min(pos - block * BLOCK_TOKENS, BLOCK_TOKENS - 1) << 24);
    }
    x.n = x.rows = 0;
    give(x, -1, NO_BLOCK);
}

// next_segment of a DIRECT kernel, whose segments may be empty: the last one has no
// rows.  *entry: the lane's list entry.
__device__ __forceinline__ bool next_direct(RowCtrl &c, uint32_t *i, Seg *w, int32_t *entry, int lane)
{
    const uint32_t k = *i % SEGS;
    bool got = mbar_wait_bounded(&c.segs.full[k], (*i / SEGS) & 1u, SEG_WAIT_NS);
    got = __all_sync(0xffffffffu, got);
    *w = c.segs.seg[k];
    *entry = c.blocks[k][lane];
    __syncwarp();
    if (lane == 0) mbar_arrive(&c.segs.empty[k]);
    ++*i;
    return got && w->rows > 0;
}

template <int D, bool Q8, typename G>
__global__ void __launch_bounds__(CR_THREADS, 1)
chunk_rows_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const ChunkParams p)
{
    using Sh = RowShape<D, Q8>;
    constexpr int NS = Sh::NS, PD = Sh::PD;
    constexpr uint32_t STAGE = Sh::STAGE, HALF = Sh::HALF;
    static_assert(NS >= 2 && NS % 2 == 0, "ring");
    extern __shared__ __align__(1024) uint8_t smem[];
    float4 *sum = reinterpret_cast<float4 *>(smem + NS * STAGE);
    uint4 *qf = reinterpret_cast<uint4 *>(smem + NS * STAGE + Sh::SUM);      // [product over D][lane]
    RowCtrl &c = *reinterpret_cast<RowCtrl *>(smem + NS * STAGE + Sh::SUM + Sh::QF);
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    volatile int *abort = &c.abort;
    const uint64_t lim = p.wait_limit_ns;

    if (t == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&c.full[i], Q8 ? 3 : 1);                 // the copies, and the two scale warps
            mbar_init(&c.empty[i], CR_COMP / 2);
        }
        for (int i = 0; i < SEGS; ++i) {
            mbar_init(&c.segs.full[i], 1);
            mbar_init(&c.segs.empty[i], CR_COMP + (Q8 ? 3 : 1));
        }
        c.abort = 0;
        fence_barrier_init();
    }
    if (!G::BLOCKS || G::DIRECT) wait_prior_grid();
    // (the sums' place is free until a segment's end)
    static_assert(sizeof(FindScratch<G>) <= Sh::SUM, "scratch");
    if constexpr (G::DIRECT) {
        if (blockIdx.x == 0) flag_bad_requests(p.kv);
        __syncthreads();
    } else {
        find_work<G>(p, c.share, *reinterpret_cast<FindScratch<G> *>(sum), blockIdx.x, gridDim.x, warp, lane, [&]() {
            if (G::BLOCKS) wait_prior_grid();
        });
    }
    uint32_t segs = 0;
    Seg w;
    int32_t entry = NO_BLOCK;                                  // (DIRECT) the lane's entry of w's list
    auto next = [&](Seg *x) -> bool {
        if constexpr (G::DIRECT) return next_direct(c, &segs, x, &entry, lane);
        else return next_segment(c.segs, &segs, x, lane);
    };
    auto start = [&](ListWindow &win) {
        if constexpr (G::DIRECT) win.start(entry);
        else win.start(p, w, lane);
    };

    // registers after the split: 8 x 32 x 216 + 4 x 32 x 72 = 384 x 168
    if (warp >= CR_COMP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == CR_SCHED) {
            if constexpr (G::DIRECT) schedule_direct(p, c, lane);
            else schedule<G>(p, c.share, c.segs, blockIdx.x, true, lane);
        } else if (warp == CR_LOAD) {
            // ------------------------------------------------------ K, V loads
            const int sh = __ffs(min(p.kv.page_tokens, CR_TILE)) - 1;       // log2 of a box's tokens
            const int32_t down = CR_TILE >> sh, boxes = 2 * Sh::CHUNKS * down;
            uint32_t slot = 0, phase = 0, used = 0, last = 0;
            bool ok = true;
            while (next(&w)) {
                if (!ok) continue;
                PieceRows<G> at;
                if (G::BLOCKS) start(at.win);
                at.start(p, w, lane);
                for (int32_t j = 0; j < w.n; ++j) {
                    at.tile(p, w, j, lane, true);
                    const int32_t ent = G::BLOCKS ? at.win.entry(w.j0 + j) : 0;
                    const bool some = !G::BLOCKS || tile_seen(ent, w.j0 + j) > 0;      // else nothing to load
                    if (!warp_wait(&c.empty[slot], phase ^ 1u, abort, lim)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) {
                        if (G::BLOCKS) c.entry[slot] = ent;
                        if (some) mbar_arrive_expect_tx(&c.full[slot], STAGE);
                        else mbar_arrive(&c.full[slot]);
                    }
                    __syncwarp();
                    uint8_t *dst = smem + slot * STAGE;
                    for (int32_t i0 = 0; some && i0 < boxes; i0 += 32) {
                        const int32_t i = i0 + lane;
                        const int32_t d = i & (down - 1), ch = (i >> (6 - sh)) & (Sh::CHUNKS - 1);
                        const bool v = i >= boxes / 2;
                        const int32_t y = at.piece(j, d);
                        if (i < boxes)
                            tma_load_3d(dst + (v ? HALF : 0u) + ch * (CR_TILE * 128) + (d << sh) * 128, v ? &tv : &tk, &c.full[slot], 0, y,
                                        w.g * Sh::CHUNKS + ch);
                    }
                    used |= 1u << slot;
                    last = (last & ~(1u << slot)) | (phase << slot);
                    if (++slot == NS) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
            }
            // copies still in flight (only after an abort: otherwise they were waited for)
            if (lane == 0)
                for (int i = 0; i < NS; ++i)
                    if (used & (1u << i)) mbar_wait_bounded(&c.full[i], (last >> i) & 1u, drain_limit(lim));
            __syncwarp();
        } else if (Q8) {
            // ---------------------------------------------------------- scales
            // Bytes that no one else reads come from HBM: four stages' loads go
            // out together, while the four before are written (one stage ahead,
            // each stage waited for a memory latency: 217 us on the 64-request
            // step).
            const uint8_t *scale = warp == CR_SCALE ? p.kv.k_scale : p.kv.v_scale;
            const int which = warp - CR_SCALE;
            uint32_t slot = 0, phase = 0;
            bool ok = true;
            while (next(&w)) {
                if (!ok) continue;
                PieceRows<G> at;
                if (G::BLOCKS) start(at.win);
                at.start(p, w, lane);
                // the bytes of tokens lane and lane + 32 (what tokens get that no row
                // attends does not matter)
                auto bytes_of = [&](int32_t j, uint32_t (&x)[2]) {
                    at.tile(p, w, j, lane, false);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int32_t off = lane + 32 * k, y = at.piece(j, off >> at.sh);
                        const int64_t line = y < p.kv.num_pages << p.kv.page_shift ? y + (off & ((1 << at.sh) - 1)) : 0;
                        x[k] = __ldg(scale + line * p.kv.hkv + w.g);
                    }
                };
                uint32_t byte[4][2];
#pragma unroll
                for (int u = 0; u < 4; ++u) bytes_of(u, byte[u]);
                for (int32_t j = 0; ok && j < w.n; j += 4) {
                    uint32_t next[4][2];
#pragma unroll
                    for (int u = 0; u < 4; ++u) bytes_of(j + 4 + u, next[u]);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        if (!ok || j + u >= w.n) break;
                        ok = warp_wait(&c.empty[slot], phase ^ 1u, abort, lim);
                        if (!ok) break;
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            c.scale[slot][which][lane + 32 * k] = __uint_as_float(max(112u, min(135u, byte[u][k])) << 23);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&c.full[slot]);
                        if (++slot == NS) {
                            slot = 0;
                            phase ^= 1u;
                        }
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u)
#pragma unroll
                        for (int k = 0; k < 2; ++k) byte[u][k] = next[u][k];
                }
            }
        }
    } else {
        // -------------------------------------------------------------- compute
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        constexpr int KI = D / (4 * PD);                           // 16-byte pieces of a token per thread
        constexpr int KS = D / 16;                                 // products over D
        constexpr int VI = Sh::CHUNKS;
        const int r = lane >> 2, q = lane & 3;
        const int grp = warp >> 2, sub = (warp & 3) * 16;          // stages of this parity, tokens sub .. + 15
        const float cs = p.scale * LOG2_E;
        uint32_t slot = 0, phase = 0, it = 0;
        bool ok = true;
        // The queries as A operands, in shared memory (in registers they spilled:
        // 294 us on the 64-request E4M3 step).  Product k of piece i takes dims
        // 8 PD (i / 2) + PD (2 q + i % 2) + 4 k .. + 3.  They are loaded while the
        // segment before is added up.
        uint2 xq[(KS + CR_COMP - 1) / CR_COMP][2];
        auto load_q = [&](const Seg &x) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = r + 8 * e;
                const int32_t v = x.v0 + min(row, x.rows - 1), tok = by_group(p, v), h = v - tok * p.group;
                const uint8_t *src = static_cast<const uint8_t *>(p.q) +
                                     ((static_cast<int64_t>(x.s0) + tok) * p.q_stride + (x.g * p.group + h) * D) * 2;
#pragma unroll
                for (int a = 0; a < (KS + CR_COMP - 1) / CR_COMP; ++a) {
                    const int k = warp + a * CR_COMP, i = k / (PD / 4), j = k % (PD / 4);
                    const int dim = 8 * PD * (i >> 1) + PD * (2 * q + (i & 1)) + 4 * j;
                    xq[a][e] = k < KS && row < x.rows ? __ldg(reinterpret_cast<const uint2 *>(src + dim * 2)) : make_uint2(0u, 0u);
                }
            }
        };
        auto give_q = [&]() {
#pragma unroll
            for (int a = 0; a < (KS + CR_COMP - 1) / CR_COMP; ++a)
                if (warp + a * CR_COMP < KS)
                    qf[(warp + a * CR_COMP) * 32 + lane] = make_uint4(xq[a][0].x, xq[a][1].x, xq[a][0].y, xq[a][1].y);
        };
        bool more = next(&w);
        if (more) {
            load_q(w);
            give_q();
        }
        named_barrier(BAR_COMP, 32 * CR_COMP);
        while (more) {
            const uint32_t *bits[2];                               // which entries the rows' tokens attend
            int32_t pos[2], first[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int32_t tok = by_group(p, w.v0 + min(r + 8 * e, w.rows - 1));
                pos[e] = w.p0 + tok;
                bits[e] = G::BLOCKS && !G::DIRECT ? bits_of(p, w, tok) : nullptr;
                first[e] = p.window > 0 ? max(0, pos[e] - p.window + 1) : 0;
            }
            int32_t word_at = -1;
            uint32_t words[2] = {~0u, ~0u};
            float o[VI][PD][4];
#pragma unroll
            for (int i = 0; i < VI; ++i)
#pragma unroll
                for (int d = 0; d < PD; ++d)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][d][e] = 0.0f;
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

            for (int32_t j = 0; ok && j < w.n; ++j, ++it) {
                const uint32_t sl = slot, ph = phase;
                if (++slot == NS) {
                    slot = 0;
                    phase ^= 1u;
                }
                if ((it & 1u) != static_cast<uint32_t>(grp)) continue;
                const int32_t at = (w.j0 + j) >> 1;                // (list entry)
                if (G::BLOCKS && !G::DIRECT && at >> 5 != word_at) {
                    word_at = at >> 5;
#pragma unroll
                    for (int e = 0; e < 2; ++e) words[e] = __ldg(bits[e] + word_at);
                }
                ok = warp_wait(&c.full[sl], ph, abort, lim);
                const int32_t ent = G::BLOCKS ? c.entry[sl] : 0;
                // tokens that some row attends, of a list's tile
                const int32_t seen = G::BLOCKS ? tile_seen(ent, w.j0 + j) : 0;
                const int32_t tok0 = (G::BLOCKS ? entry_block(ent) * BLOCK_TOKENS + (w.j0 + j & 1) * CR_TILE : (w.j0 + j) * CR_TILE) + sub;
                const bool att[2] = {((words[0] >> (at & 31)) & 1u) != 0, ((words[1] >> (at & 31)) & 1u) != 0};
                if (ok && (G::BLOCKS ? sub < seen : tok0 <= w.hi_tok && tok0 + 15 >= w.lo_tok)) {
                    const uint8_t *ka = smem + sl * STAGE, *va = ka + HALF;
                    // ---- scores of tokens sub + 8 n + 2 q + {0, 1}
                    float s[2][4] = {};
#pragma unroll
                    for (int i = 0; i < KI; ++i) {
                        uint4 x[2];
#pragma unroll
                        for (int n = 0; n < 2; ++n)
                            x[n] = lds128(ka + (i >> 1) * (CR_TILE * 128) + (sub + 8 * n + r) * 128 +
                                          (((2 * q + (i & 1)) ^ r) << 4));
#pragma unroll
                        for (int k = 0; k < PD / 4; ++k) {
                            const uint4 a = qf[(i * (PD / 4) + k) * 32 + lane];
#pragma unroll
                            for (int n = 0; n < 2; ++n) {
                                uint32_t b0, b1;
                                if (Q8) {
                                    e4m3x4_to_half(word(x[n], k), &b0, &b1);
                                } else {
                                    b0 = word(x[n], 2 * (k & 1));
                                    b1 = word(x[n], 2 * (k & 1) + 1);
                                }
                                mma16816(s[n], a, b0, b1);
                            }
                        }
                    }
                    // ---- softmax
                    // some token that no row attends
                    const bool edge = G::BLOCKS ? sub + 15 >= seen : tok0 < w.lo_tok || tok0 + 15 > w.hi_tok;
                    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        float2 f = make_float2(1.0f, 1.0f);
                        if (Q8) f = *reinterpret_cast<const float2 *>(&c.scale[sl][0][sub + 8 * n + 2 * q]);
                        const int32_t tk0 = tok0 + 8 * n + 2 * q;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int32_t tok = tk0 + (e & 1);
                            if (Q8) s[n][e] *= (e & 1) ? f.y : f.x;
                            if (tok > pos[e >> 1] || tok < first[e >> 1] || !att[e >> 1]) s[n][e] = -INFINITY;
                            mx[e >> 1] = fmaxf(mx[e >> 1], s[n][e]);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
                        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
                    }
                    const bool grow0 = (mx[0] - m[0]) * cs > RESCALE, grow1 = (mx[1] - m[1]) * cs > RESCALE;
                    if (__any_sync(0xffffffffu, grow0 || grow1)) {
                        const float a0 = grow0 ? exp2_approx((m[0] - mx[0]) * cs) : 1.0f;
                        const float a1 = grow1 ? exp2_approx((m[1] - mx[1]) * cs) : 1.0f;
                        if (grow0) m[0] = mx[0];
                        if (grow1) m[1] = mx[1];
                        l[0] *= a0;
                        l[1] *= a1;
#pragma unroll
                        for (int i = 0; i < VI; ++i)
#pragma unroll
                            for (int d = 0; d < PD; ++d) {
                                o[i][d][0] *= a0;
                                o[i][d][1] *= a0;
                                o[i][d][2] *= a1;
                                o[i][d][3] *= a1;
                            }
                    }
                    uint32_t pw[4];
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float mm = m[e] == -INFINITY ? 0.0f : m[e];
                            const float x = exp2_approx(fmaf(s[n][2 * e] - mm, cs, P_UP));
                            const float y = exp2_approx(fmaf(s[n][2 * e + 1] - mm, cs, P_UP));
                            l[e] += x + y;
                            const __half2 hh = __floats2half2_rn(x, y);
                            pw[2 * n + e] = *reinterpret_cast<const uint32_t *>(&hh);
                        }
                    const uint4 pa = make_uint4(pw[0], pw[1], pw[2], pw[3]);
                    // ---- O += P . V; tokens 2 q, 2 q + 1 (x), 2 q + 8, 2 q + 9 (y)
                    uint32_t fx = 0, fy = 0;
                    if (Q8) {
                        const float2 a = *reinterpret_cast<const float2 *>(&c.scale[sl][1][sub + 2 * q]);
                        const float2 b = *reinterpret_cast<const float2 *>(&c.scale[sl][1][sub + 2 * q + 8]);
                        const __half2 ha = __floats2half2_rn(a.x, a.y), hb = __floats2half2_rn(b.x, b.y);
                        fx = *reinterpret_cast<const uint32_t *>(&ha);
                        fy = *reinterpret_cast<const uint32_t *>(&hb);
                    }
#pragma unroll
                    for (int i = 0; i < VI; ++i) {
                        uint4 x[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int tr = sub + 2 * q + (e & 1) + 8 * (e >> 1);
                            x[e] = lds128(va + i * (CR_TILE * 128) + tr * 128 + ((r ^ (tr & 7)) << 4));
                            // zero weights must meet zeros
                            if (edge && (G::BLOCKS ? tr >= seen : tok0 - sub + tr < w.lo_tok || tok0 - sub + tr > w.hi_tok))
                                x[e] = make_uint4(0u, 0u, 0u, 0u);
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t xa = word(x[0], k), xb = word(x[1], k), ya = word(x[2], k), yb = word(x[3], k);
                            if (Q8) {
                                uint32_t b0[4], b1[4];
                                e4m3x4_to_half(__byte_perm(xa, xb, 0x5140), &b0[0], &b0[1]);
                                e4m3x4_to_half(__byte_perm(xa, xb, 0x7362), &b0[2], &b0[3]);
                                e4m3x4_to_half(__byte_perm(ya, yb, 0x5140), &b1[0], &b1[1]);
                                e4m3x4_to_half(__byte_perm(ya, yb, 0x7362), &b1[2], &b1[3]);
#pragma unroll
                                for (int d = 0; d < 4; ++d)
                                    mma16816(o[i][(4 * k + d) % PD], pa, half2_mul(b0[d], fx), half2_mul(b1[d], fy));
                            } else {
                                mma16816(o[i][(2 * k) % PD], pa, __byte_perm(xa, xb, 0x5410), __byte_perm(ya, yb, 0x5410));
                                mma16816(o[i][(2 * k + 1) % PD], pa, __byte_perm(xa, xb, 0x7632), __byte_perm(ya, yb, 0x7632));
                            }
                        }
                    }
                }
                __syncwarp();
                if (ok && lane == 0) mbar_arrive(&c.empty[sl]);
            }
            // ---- the next queries
            Seg w_next;
            const bool more_next = next(&w_next);
            if (more_next) load_q(w_next);
            // ---- the eight warps' sums, at the largest maximum
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
                l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
                if (q == 0) c.m[warp][r + 8 * e] = m[e];
            }
            named_barrier(BAR_COMP, 32 * CR_COMP);
            float f[2], mt[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                mt[e] = c.m[0][r + 8 * e];
#pragma unroll
                for (int k = 1; k < CR_COMP; ++k) mt[e] = fmaxf(mt[e], c.m[k][r + 8 * e]);
                f[e] = m[e] == -INFINITY ? 0.0f : exp2_approx((m[e] - mt[e]) * cs);
                if (q == 0) c.l[warp][r + 8 * e] = l[e] * f[e];
            }
            // 8 / SUMS steps; in each every warp lays down DS dims of each chunk, and
            // thread t adds up the eight warps' values of place t: chunk i, row
            // r' + 8 (e / 2), dims 8 PD i + PD (2 q' + e % 2) .., where t = (i, lane', e).
            constexpr int DS = PD * Sh::SUMS / 8, OWN = (VI * 128 + 255) / 256;    // dims per step, places per thread
            float x[OWN][PD];
#pragma unroll
            for (int st = 0; st < 8 / Sh::SUMS; ++st) {
#pragma unroll
                for (int i = 0; i < VI; ++i)
#pragma unroll
                    for (int d = 0; d < DS; ++d) {
                        const float (&v)[4] = o[i][st * DS + d];
                        sum[((warp * DS + d) * VI + i) * 32 + lane] = make_float4(v[0] * f[0], v[1] * f[0], v[2] * f[1], v[3] * f[1]);
                    }
                named_barrier(BAR_COMP, 32 * CR_COMP);
                const float *src = reinterpret_cast<const float *>(sum);
#pragma unroll
                for (int k = 0; k < OWN; ++k)
#pragma unroll
                    for (int d = 0; d < DS; ++d) {
                        float v = 0.0f;
                        if (t + 256 * k < VI * 128) {
#pragma unroll
                            for (int j = 0; j < CR_COMP; ++j) v += src[(j * DS + d) * VI * 128 + t + 256 * k];
                        }
                        x[k][st * DS + d] = v;
                    }
                named_barrier(BAR_COMP, 32 * CR_COMP);
            }
            if (G::DIRECT && p.split > 1) {
                // the CTA's sums and maxima, for its cluster
                float *mine = reinterpret_cast<float *>(sum);
#pragma unroll
                for (int k = 0; k < OWN; ++k) {
                    const int at = t + 256 * k, i = at >> 7, ln = (at >> 2) & 31, e = at & 3;
                    const int row = (ln >> 2) + 8 * (e >> 1), dim = 8 * PD * i + PD * (2 * (ln & 3) + (e & 1));
                    if (at >= VI * 128) continue;
#pragma unroll
                    for (int d = 0; d < PD; d += 4)
                        *reinterpret_cast<float4 *>(mine + row * D + dim + d) = make_float4(x[k][d], x[k][d + 1], x[k][d + 2], x[k][d + 3]);
                    if (dim == 0) {
                        float lt = 0.0f, ma = c.m[0][row];
#pragma unroll
                        for (int j = 0; j < CR_COMP; ++j) {
                            lt += c.l[j][row];
                            ma = fmaxf(ma, c.m[j][row]);
                        }
                        c.part[row] = make_float2(ma, lt);
                    }
                }
            } else
#pragma unroll
            for (int k = 0; k < OWN; ++k) {
                const int at = t + 256 * k, i = at >> 7, ln = (at >> 2) & 31, e = at & 3;
                const int row = (ln >> 2) + 8 * (e >> 1), dim = 8 * PD * i + PD * (2 * (ln & 3) + (e & 1));
                if (!ok || at >= VI * 128 || row >= w.rows) continue;
                float lt = 0.0f;
#pragma unroll
                for (int j = 0; j < CR_COMP; ++j) lt += c.l[j][row];
                if (w.place < 0) {
                    const float inv = lt > 0.0f ? 1.0f / lt : 0.0f;
                    const int32_t v = w.v0 + row, tok = by_group(p, v), h = v - tok * p.group;
                    __half *out = static_cast<__half *>(p.out) +
                                  ((static_cast<int64_t>(w.s0) + tok) * p.hq + w.g * p.group + h) * D + dim;
#pragma unroll
                    for (int d = 0; d < PD; d += 8) {
                        uint32_t u[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) u[j] = to_half2(x[k][d + 2 * j] * inv, x[k][d + 2 * j + 1] * inv);
                        *reinterpret_cast<uint4 *>(out + d) = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                } else {
                    float *out = reinterpret_cast<float *>(p.ws + ws_o<CR_ROWS, CHUNK_MAX_CTAS>()) +
                                 (static_cast<int64_t>(w.place) * p.ws_rows + row) * D + dim;
#pragma unroll
                    for (int d = 0; d < PD; d += 4)
                        *reinterpret_cast<float4 *>(out + d) = make_float4(x[k][d], x[k][d + 1], x[k][d + 2], x[k][d + 3]);
                    if (dim == 0) {
                        float ma = c.m[0][row];
#pragma unroll
                        for (int j = 1; j < CR_COMP; ++j) ma = fmaxf(ma, c.m[j][row]);
                        *reinterpret_cast<float2 *>(p.ws + WS_ML + (static_cast<int64_t>(w.place) * CR_ROWS + row) * 8) =
                            make_float2(ma, lt);
                    }
                }
            }
            if (more_next) give_q();
            w = w_next;
            more = more_next;
            named_barrier(BAR_COMP, 32 * CR_COMP);                 // sums read before the next segment's, queries in
        }
    }
    __syncthreads();
    if constexpr (G::DIRECT) {
        if (p.split > 1) {
            // The cluster had one unit at most.  Each CTA adds up an equal run of dims
            // of all rows and writes it (by the warps that have the registers for it).
            cluster_sync();
            w = c.segs.seg[0];
            if (warp >= CR_COMP) w.rows = 0;
            const float cs = p.scale * LOG2_E;
            const float *mine = reinterpret_cast<const float *>(sum);
            const int32_t per = D / p.split / 4, rank = blockIdx.x % p.split;               // float4s of a row
            for (int32_t at = t; at < w.rows * per && !c.abort; at += 32 * CR_COMP) {
                const int32_t row = at / per, dim = (rank * per + at - row * per) * 4;
                float2 ml[DIRECT_SPLIT];
                float4 y[DIRECT_SPLIT];
#pragma unroll
                for (int k = 0; k < DIRECT_SPLIT; ++k) {
                    if (k >= p.split) break;
                    ml[k] = ld_cluster_f2(&c.part[row], k);
                    y[k] = ld_cluster_f4(mine + row * D + dim, k);
                }
                float ma = -INFINITY, lt = 0.0f;
#pragma unroll
                for (int k = 0; k < DIRECT_SPLIT; ++k)
                    if (k < p.split) ma = fmaxf(ma, ml[k].x);
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int k = 0; k < DIRECT_SPLIT; ++k) {
                    if (k >= p.split) break;
                    const float wt = ml[k].x == -INFINITY ? 0.0f : exp2_approx((ml[k].x - ma) * cs);
                    lt = fmaf(ml[k].y, wt, lt);
                    v.x = fmaf(y[k].x, wt, v.x);
                    v.y = fmaf(y[k].y, wt, v.y);
                    v.z = fmaf(y[k].z, wt, v.z);
                    v.w = fmaf(y[k].w, wt, v.w);
                }
                const float inv = lt > 0.0f ? 1.0f / lt : 0.0f;
                const int32_t vr = w.v0 + row, tok = by_group(p, vr), h = vr - tok * p.group;
                __half *out = static_cast<__half *>(p.out) +
                              ((static_cast<int64_t>(w.s0) + tok) * p.hq + w.g * p.group + h) * D + dim;
                *reinterpret_cast<uint2 *>(out) = make_uint2(to_half2(v.x * inv, v.y * inv), to_half2(v.z * inv, v.w * inv));
            }
            __syncwarp();
            cluster_sync();                                      // read by the whole cluster
        }
    }
    if (t == 0 && c.abort) record_error(p.kv.status, ST_TIMEOUT);
    allow_next_grid();
}

// Lets the kernel have `smem` bytes, once per device.
inline int allow_smem(const void *kernel, size_t smem, std::mutex &mu, bool (&done)[64])
{
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return static_cast<int>(cudaErrorInvalidDevice);
    std::lock_guard<std::mutex> lk(mu);
    if (done[dev]) return 0;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    done[dev] = e == cudaSuccess;
    return static_cast<int>(e);
}

// after_lists: as in launch_pairs.
template <int D, bool Q8, typename G>
int launch_rows(const ChunkParams &p, const void *tk, const void *tv, int grid, bool overlap, bool after_lists, cudaStream_t stream)
{
    using Sh = RowShape<D, Q8>;
    constexpr size_t SMEM = Sh::NS * Sh::STAGE + Sh::SUM + Sh::QF + sizeof(RowCtrl);
    static_assert(SMEM <= 232448, "shared memory budget");
    static std::mutex mu;
    static bool done[64] = {};
    int rc = allow_smem(reinterpret_cast<const void *>(&chunk_rows_kernel<D, Q8, G>), SMEM, mu, done);
    if (rc != 0) return rc;
    void *args[] = {const_cast<void *>(tk), const_cast<void *>(tv), const_cast<ChunkParams *>(&p)};
    rc = launch_kernel(reinterpret_cast<const void *>(&chunk_rows_kernel<D, Q8, G>), dim3(grid), dim3(CR_THREADS), SMEM,
                                 stream, after_lists && overlap, args);
    if (rc != 0) return rc;
    void *join[] = {const_cast<ChunkParams *>(&p)};
    const unsigned y = static_cast<unsigned>(p.ws_rows);
    return launch_kernel(reinterpret_cast<const void *>(&chunk_join_kernel<G, D>), dim3(grid, y), dim3(256), 0, stream,
                         overlap, join);
}

// How many clusters of `size` CTAs the device runs at once (0: it cannot say).
inline int clusters_at_once(const void *kernel, size_t smem, unsigned size)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size);
    cfg.blockDim = dim3(CR_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}

// The DIRECT kernel: no lists before it, nothing to join after it.  A unit takes as
// many CTAs as leave all units running at once (8 requests of 2 KV heads: 12 us on
// clusters of 4, 18 us on clusters of 8, of which not all 16 do).
template <int D, bool Q8>
int launch_direct(const ChunkParams &in, const void *tk, const void *tv, int32_t units, int sms, cudaStream_t stream)
{
    using Sh = RowShape<D, Q8>;
    constexpr size_t SMEM = Sh::NS * Sh::STAGE + Sh::SUM + Sh::QF + sizeof(RowCtrl);
    static_assert(SMEM <= 232448, "shared memory budget");
    const void *kernel = reinterpret_cast<const void *>(&chunk_rows_kernel<D, Q8, DirectRowsGeometry>);
    static std::mutex mu;
    static bool done[64] = {};
    static int fit[64][4] = {};              // clusters of 2, 4 and 8 at once; -1: none
    const int rc = allow_smem(kernel, SMEM, mu, done);
    if (rc != 0) return rc;
    ChunkParams p = in;
    p.split = 1;
    int dev = 0;
    cudaGetDevice(&dev);
    {
        std::lock_guard<std::mutex> lk(mu);
        for (int i = 3; i > 0 && p.split == 1; --i) {
            int &n = fit[dev][i];
            if (n == 0) n = std::max(clusters_at_once(kernel, SMEM, 1u << i), 0);
            if (n == 0) n = -1;
            if (units <= n) p.split = 1 << i;
        }
    }
    static_assert(DIRECT_SPLIT == 8, "three sizes");
    const int grid = p.split > 1 ? units * p.split : std::min(units, sms);
    void *args[] = {const_cast<void *>(tk), const_cast<void *>(tv), &p};
    return launch_kernel(kernel, dim3(grid), dim3(CR_THREADS), SMEM, stream, false, args, p.split);
}

template <typename G>
int launch_rows_for(const ChunkParams &p, const void *tk, const void *tv, int sms, bool overlap, bool after_lists, cudaStream_t s)
{
    const int grid = std::min(sms, static_cast<int>(CHUNK_MAX_CTAS));
    if (p.kv.head_dim == 128)
        return p.kv.e4m3 ? launch_rows<128, true, G>(p, tk, tv, grid, overlap, after_lists, s)
                         : launch_rows<128, false, G>(p, tk, tv, grid, overlap, after_lists, s);
    return p.kv.e4m3 ? launch_rows<256, true, G>(p, tk, tv, grid, overlap, after_lists, s)
                     : launch_rows<256, false, G>(p, tk, tv, grid, overlap, after_lists, s);
}

}  // namespace
}  // namespace qsa
