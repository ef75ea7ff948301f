// Dense attention of new tokens over the paged K/V cache.
//
//   o = sum_t exp(s_t - m) v_t / sum_t exp(s_t - m),   s_t = scale * q . k_t
//
// in one pass over the visible tokens t, with the running maximum m and sum.
// Both products run on the 5th-generation tensor cores (kind::f16, FP32
// accumulators in TMEM), tile by tile of 128 tokens, each instruction spanning
// a pair of SMs (cta_group::2), so a pair shares every key and value it loads:
//   S[row, token] = Q . K^T     M = 256 rows, N = 128 tokens, K = D
//   O[row, dim]  += P . V       M = 256 rows, N = D, K = 128 tokens
// CTA r of the pair holds rows 128 r .. + 127 (Q, S, P, O), tokens 64 r .. + 63
// of the key tile and dims r D / 2 .. of the value tile.  (With one CTA per
// unit and M = 128, the ring held a quarter more than one tile of D = 256 and
// the products waited for its copies: 1,021 us on the 1,616-row chunk over
// 29,000 tokens, tensor pipe 46% busy.)
// A row of the tile is one (token, query head) pair: the query heads of a KV
// head share its keys and values, so a unit of work is 256 consecutive pairs
// (token * group + head) of one request and KV head.
//
// Work: the units' tiles, in the order (request, rows, KV head), form one line
// that the CTA pairs share out evenly (each unit a little longer than its tiles
// for what it costs besides them: without that, pairs with many short units
// ended last, 1,019 us against 8xx us on four prompts of 4,096 tokens), so one row over a long cache,
// a batch of unequal requests and a long prompt all fill the card.  A unit that
// lies across pairs leaves unnormalised FP32 partial sums with their maxima in
// the workspace (at most two per pair), which a second kernel joins.  Every
// pair finds its share itself from seq_start and pos_start: no plan kernel and
// no host knowledge of the lengths.
//
// A CTA's warps: 0-7 softmax, 8 loads K and V by TMA, one box per page piece,
// through the block table, 9 issues the MMAs (in the first CTA of the pair),
// 12-15 load the queries, clear the value rows that nothing attends and, from
// the E4M3 cache, turn the loaded codes into FP16 tiles; 10 and 11 only give
// their registers away.  K and V share a ring of slots in the order of use.
//
// Softmax warps 0-3 take the even tiles and 4-7 the odd ones (warp w: TMEM lane
// quarter w % 4, a row per thread), so that one group's exponentials run beside
// the other's waits; S has a buffer for each.  A thread takes its 128 scores
// into registers, its row's running maximum passes on from tile to tile, from
// one group to the other, before the exponentials start, and each group keeps
// its own sum.  P goes to TMEM as FP16 and is the A operand of the second
// product from there.  With D = 128, P has columns of its own, so the score
// product of the tile after next starts as soon as the scores are in registers:
//   S(0) S(1) | S(2) O(0) | S(3) O(1) | ...
// With D = 256, TMEM is full (2 x 128 for S, 256 for O): P overwrites its
// scores and the order is S(0) S(1) | O(0) S(2) | O(1) S(3) | ...
//
// The accumulator is rescaled only when a row's maximum has grown by more than
// 2^8 since the one in use: P is then at most 256, far inside FP16, and the sum
// uses the same stale maximum, so the result is the same.  Rounding P to FP16
// (2^-11 of each weight) is of the size of the output's own rounding.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "qsa_device.cuh"
#include "qsa_internal.h"
#include "qsa_seq.cuh"

namespace qsa {
namespace {

constexpr int CH_HALF = 128;                 // rows of one CTA: TMEM lanes
constexpr int CH_ROWS = 256;                 // (token, head) rows of a unit: MMA M
constexpr int CH_TILE = 128;                 // tokens of a tile
constexpr int CH_SOFT = 8;                   // softmax warps
constexpr int CH_LOAD = 8, CH_MMA = 9, CH_SCHED = 10, CH_MMA2 = 11, CH_HELP = 12;
constexpr int CH_ROLES = 15;                 // warps that read the segments: all but the scheduler

constexpr int CH_HELPERS = 4;
constexpr int CH_WARPS = CH_HELP + CH_HELPERS;
constexpr int CH_THREADS = 32 * CH_WARPS;
constexpr int RAWS = 4;                      // slots of loaded codes (E4M3)
constexpr int MAX_SLOTS = 10;                // slots of the ring at most
constexpr uint32_t RING = 229376;            // bytes for Q and the ring
constexpr float RESCALE = 8.0f;              // log2 of the growth that rescales
constexpr uint32_t TM_S = 0, TM_O = 256;     // TMEM columns: two S buffers of 128, O
constexpr int UNIT_COST = 4;                 // tiles' worth of time that a unit costs besides its tiles
constexpr int BAR_PAIR = 1, BAR_HELP = 5;    // named barriers: four softmax warp pairs, the helpers

template <int D, bool Q8>
struct Shape {
    static constexpr int QBUFS = D == 128 ? 2 : 1;                     // buffers of Q
    static constexpr uint32_t QB = CH_HALF * D * 2;                    // bytes of one
    // a CTA's half of a K tile: 64 tokens, or of a V tile: D / 2 dims of 128 tokens
    static constexpr uint32_t SLOT = 128 * D, RAW = SLOT / 2;
    static constexpr int KTOK = 64, VTOK = CH_TILE;
    static constexpr int FIT = (RING - QBUFS * QB - (Q8 ? RAWS * RAW : 0)) / SLOT, NS = FIT < MAX_SLOTS ? FIT : MAX_SLOTS;
    static constexpr bool OWN_P = D == 128;                            // P beside S, not over it
    static constexpr uint32_t TM_P = OWN_P ? 384 : TM_S, P_STRIDE = OWN_P ? 64 : 128;
    static constexpr int LEAD = OWN_P ? 3 : 2;                         // key tiles loaded before the first value tile
};

// A run of tiles of one unit, a pair's next piece of work.
struct alignas(16) Seg {
    int32_t n, j0;                           // tiles j0 .. j0 + n - 1; n = 0: no more work
    int32_t b, g;                            // request, KV head
    int32_t s0, p0, v0, rows;                // request's first row and position, unit's first (token, head) pair, pairs in use
    int32_t lo_tok, hi_tok;                  // tokens that some row attends: lo_tok .. hi_tok
    int32_t place;                           // workspace place of the partial result, -1: this is the whole unit
    int32_t pad;

    // whether tile j0 + k holds tokens that no row attends
    __device__ __forceinline__ bool cut(int32_t k) const
    {
        const int32_t t0 = (j0 + k) * CH_TILE;
        return t0 < lo_tok || t0 + CH_TILE - 1 > hi_tok;
    }
};
constexpr int SEGS = 4;                      // segments the scheduler may be ahead
constexpr uint64_t SEG_WAIT_NS = 10000000000ull;

struct Ctrl {
    Seg seg[SEGS];
    uint64_t seg_full[SEGS], seg_empty[SEGS];
    uint64_t full[MAX_SLOTS], empty[MAX_SLOTS], raw_full[RAWS], raw_empty[RAWS], bnd[8];
    uint64_t s_full[2], s_free[2], p_full[2], o_done[2], m_out[2][4], q_full[2], q_free[2], drain;
    alignas(8) float mrow[2][CH_HALF];       // [tile parity][row]: maximum in use at the group's last tile; sums at a segment's end
    alignas(8) uint16_t scale[2][CH_TILE];   // [slot parity][token]: FP16 scale (E4M3)
    int64_t w0, w1, total;                   // this pair's share of the line, the line's length
    int32_t pairs;                           // pairs that have work
    int32_t b, m, g, off;                    // the unit that w0 lies in, and w0's place in it
    uint32_t tmem;
    int32_t abort;
};

// A unit that lies across pairs, as the join kernel needs it (written by the
// pair that holds the unit's first tile).
struct Split {
    int32_t parts;                           // 0: none
    int32_t rows;                            // rows of the unit
    int32_t s0, v0, g;                       // request's first row, unit's first (token, head) pair, KV head
};

// Workspace: a Split per pair, then per place (two for each pair) the rows'
// (maximum in powers of two, sum), then their unnormalised outputs.
constexpr size_t WS_ML = 4096;
constexpr size_t WS_O = WS_ML + size_t{2} * CHUNK_MAX_PAIRS * CH_ROWS * 8;
static_assert(sizeof(Split) * CHUNK_MAX_PAIRS <= WS_ML, "workspace header");

// ------------------------------------------------------------- work sharing --

struct Unit {
    int32_t v0, rows, lo_tok, hi_tok;        // as in Seg
    int32_t lo, hi;                          // tiles lo .. hi - 1
};

// v / p.group for 0 <= v < 2^31: with s = ceil(log2 group) and group_mul =
// ceil(2^(31 + s) / group), the error of v * group_mul against v * 2^(31 + s) /
// group is below 2^31 * 2^s / group, less than one unit of the quotient's grid.
__device__ __forceinline__ int32_t by_group(const ChunkParams &p, int32_t v)
{
    return static_cast<int32_t>((static_cast<uint64_t>(static_cast<uint32_t>(v)) * p.group_mul) >> p.group_shift);
}

__device__ __forceinline__ int32_t units_of(const ChunkParams &p, const Seq &s)
{
    return (s.n * p.group + CH_ROWS - 1) / CH_ROWS;
}

__device__ __forceinline__ Unit unit_of(const ChunkParams &p, const Seq &s, int32_t m)
{
    Unit u;
    u.v0 = m * CH_ROWS;
    const int32_t end = min(s.n * p.group, u.v0 + CH_ROWS);
    u.rows = end - u.v0;
    const int32_t first = s.p0 + by_group(p, u.v0);
    u.hi_tok = s.p0 + by_group(p, end - 1);
    u.lo_tok = p.window > 0 ? max(0, first - p.window + 1) : 0;
    u.lo = u.lo_tok / CH_TILE;
    u.hi = u.hi_tok / CH_TILE + 1;
    return u;
}

template <typename T>
__device__ __forceinline__ T warp_scan(T x, int lane)      // inclusive
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// The sum of x over the threads before this one, and over all of them.
template <typename T>
__device__ __forceinline__ T block_scan(T x, T *warp_total, int warp, int lane, T *total)
{
    const T sc = warp_scan(x, lane);
    if (lane == 31) warp_total[warp] = sc;
    __syncthreads();
    T before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < CH_WARPS; ++w) {
        if (w == warp) before = all;
        all += warp_total[w];
    }
    *total = all;
    return before + sc - x;
}

// Shared memory of find_work: the queries' place, which is free until then.
struct FindScratch {
    int32_t prefix[CH_THREADS];
    int32_t units[CH_WARPS];
    int64_t costs[CH_WARPS];
};
static_assert(sizeof(FindScratch) <= Shape<128, false>::QB, "scratch");

// Finds this pair's share of the line, c.w0 .. c.w1, and the unit that w0 lies
// in (both CTAs of a pair do, alike).  Each thread counts the units of a run of
// requests, then adds up the lengths of an equal run of units.
__device__ __forceinline__ void find_work(const ChunkParams &p, Ctrl &c, FindScratch &s, int warp, int lane)
{
    const int t = threadIdx.x;
    int32_t *prefix = s.prefix;
    const int32_t run = (p.kv.n_reqs + CH_THREADS - 1) / CH_THREADS;
    const int32_t r0 = min(t * run, p.kv.n_reqs), r1 = min(r0 + run, p.kv.n_reqs);
    int32_t mine = 0, units;
    for (int32_t b = r0; b < r1; ++b) {
        bool bad;
        mine += units_of(p, seq_of(p.kv, b, &bad));
        if (bad && blockIdx.x == 0) record_error(p.kv.status, ST_BAD_ROW);
    }
    prefix[t] = block_scan(mine, s.units, warp, lane, &units);
    __syncthreads();
    const int32_t u0 = static_cast<int32_t>(static_cast<int64_t>(units) * t / CH_THREADS);
    const int32_t u1 = static_cast<int32_t>(static_cast<int64_t>(units) * (t + 1) / CH_THREADS);
    int32_t b0 = 0, m0 = 0;
    Seq s0{0, 0, 0};
    int64_t cost = 0, total;
    if (u0 < u1) {
        int lo = 0;                                          // the last run that starts at or before u0
#pragma unroll
        for (int step = CH_THREADS / 2; step > 0; step >>= 1)
            if (prefix[lo + step] <= u0) lo += step;
        b0 = lo * run;
        m0 = u0 - prefix[lo];
        bool bad;
        s0 = seq_of(p.kv, b0, &bad);
        for (int32_t n = units_of(p, s0); m0 >= n; n = units_of(p, s0)) {
            m0 -= n;
            s0 = seq_of(p.kv, ++b0, &bad);
        }
        int32_t b = b0, m = m0;
        Seq sb = s0;
        for (int32_t u = u0; u < u1; ++u, ++m) {
            while (m >= units_of(p, sb)) {
                sb = seq_of(p.kv, ++b, &bad);
                m = 0;
            }
            const Unit un = unit_of(p, sb, m);
            cost += UNIT_COST + un.hi - un.lo;
        }
        cost *= p.kv.hkv;
    }
    int64_t at = block_scan(cost, s.costs, warp, lane, &total);
    // one place each at least, so that the pairs with work are the first ones
    const int32_t pairs = static_cast<int32_t>(min(total, static_cast<int64_t>(gridDim.x >> 1)));
    const int32_t me = blockIdx.x >> 1;
    const int64_t w0 = me < pairs ? total * me / pairs : 0, w1 = me < pairs ? total * (me + 1) / pairs : 0;
    if (t == 0) {
        c.w0 = w0;
        c.w1 = w1;
        c.total = total;
        c.pairs = pairs;
    }
    if (w0 < w1 && at <= w0 && w0 < at + cost) {
        for (;; ++m0) {
            while (m0 >= units_of(p, s0)) {
                bool bad;
                s0 = seq_of(p.kv, ++b0, &bad);
                m0 = 0;
            }
            const Unit un = unit_of(p, s0, m0);
            const int32_t len = UNIT_COST + un.hi - un.lo;
            if (w0 < at + static_cast<int64_t>(len) * p.kv.hkv) {
                c.b = b0;
                c.m = m0;
                c.g = static_cast<int32_t>(w0 - at) / len;
                c.off = static_cast<int32_t>(w0 - at) % len;
                break;
            }
            at += static_cast<int64_t>(len) * p.kv.hkv;
        }
    }
    __syncthreads();
}

// The pair's share as segments.
struct Walk {
    int64_t left;
    int32_t b, m, g, off, n_units;
    Seq s;

    __device__ __forceinline__ Walk(const ChunkParams &p, const Ctrl &c)
    {
        left = c.w1 - c.w0;
        b = c.b;
        m = c.m;
        g = c.g;
        off = c.off;
        if (left > 0) load(p);
    }
    __device__ __forceinline__ void load(const ChunkParams &p)
    {
        bool bad;
        s = seq_of(p.kv, b, &bad);
        n_units = units_of(p, s);
    }
    // the next segment (n = 0 at the end of the share); *rest: tiles of the unit after it
    __device__ __forceinline__ Seg next(const ChunkParams &p, bool *head, int32_t *rest)
    {
        Seg x;
        x.n = 0;
        if (left <= 0) return x;
        while (m >= n_units) {               // empty requests have no units
            if (++b >= p.kv.n_reqs) return x;
            m = 0;
            load(p);
        }
        const Unit u = unit_of(p, s, m);
        // a unit's place in the line: UNIT_COST, then its tiles
        const int32_t len = UNIT_COST + u.hi - u.lo;
        const int32_t end = static_cast<int32_t>(min(static_cast<int64_t>(len), off + left));
        left -= end - off;
        x.j0 = u.lo + max(0, off - UNIT_COST);
        x.n = u.lo + max(0, end - UNIT_COST) - x.j0;      // 0: the share ends before the unit's first tile
        x.b = b;
        x.g = g;
        x.s0 = s.s0;
        x.p0 = s.p0;
        x.v0 = u.v0;
        x.rows = u.rows;
        x.lo_tok = u.lo_tok;
        x.hi_tok = u.hi_tok;
        *head = x.j0 == u.lo;
        *rest = u.hi - x.j0 - x.n;
        off = 0;
        if (++g == p.kv.hkv) {
            g = 0;
            ++m;
        }
        return x;
    }
};

// ------------------------------------------------------------------- pieces --

// Slot e of a segment of n tiles, in the order of use: LEAD key tiles, then
// value and key tiles in turn, then the value tiles left,
// e.g. K(0) K(1) V(0) K(2) V(1) ... K(n-1) V(n-2) V(n-1).
template <int LEAD>
__device__ __forceinline__ void slot_at(int32_t e, int32_t n, bool *is_v, int32_t *tile)
{
    const int32_t lead = min(LEAD, n), r = e - lead, turns = 2 * (n - lead);
    *is_v = r >= 0 && (r >= turns || (r & 1) == 0);
    *tile = r < 0 ? e : r >= turns ? r - (n - lead) : (r >> 1) + ((r & 1) ? lead : 0);
}

template <int LEAD>
__device__ __forceinline__ int32_t slot_of_v(int32_t tile, int32_t n)
{
    const int32_t lead = min(LEAD, n);
    return lead + (tile < n - lead ? 2 * tile : n - lead + tile);
}

__device__ __forceinline__ uint32_t sw128(uint32_t row, uint32_t c)
{
    return (row >> 3) * 1024u + (row & 7u) * 128u + ((c ^ (row & 7u)) << 4);
}

// V as the B operand [token (K)][dim (N)]: dims contiguous, 128-byte swizzle;
// chunks of 64 dims `chunk` bytes apart, groups of 8 tokens 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t smem_addr, uint32_t chunk)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(chunk >> 4) << 16;              // leading byte offset
    d |= static_cast<uint64_t>(1024 >> 4) << 32;               // stride byte offset
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// D[tmem] (+)= A * B over the CTA pair, kind::f16; A in shared memory, or in TMEM.
__device__ __forceinline__ void umma2_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void umma2_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive once on `bar` of both CTAs when every tcgen05 op issued so far is done.
__device__ __forceinline__ void umma2_commit(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// One thread of the (converged) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t x;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(x));
    return x != 0;
}

// A value that is the same in every lane, told to the compiler.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// The first CTA's copy of a shared-memory address.
__device__ __forceinline__ uint32_t of_first(const void *p)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
    return a;
}

__device__ __forceinline__ void cluster_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void cluster_arrive_expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// 2-D tiled load into this CTA, completing on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(void *dst_smem, const void *tmap, uint32_t bar, int32_t x, int32_t y)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst_smem)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t (&v)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// two FP32 lanes at once
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\t"
        "mov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ void named_barrier(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// A wait by a whole warp: true on every lane, or false on every lane.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort, uint64_t lim)
{
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, lim));
}

// ------------------------------------------------------------------- kernel --

template <int D, bool Q8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(CH_THREADS, 1)
chunk_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const ChunkParams p)
{
    using Sh = Shape<D, Q8>;
    constexpr int NS = Sh::NS;
    constexpr uint32_t SLOT = Sh::SLOT, RAW = Sh::RAW;
    static_assert(NS >= 3 && NS <= MAX_SLOTS, "10 slots hold fewer value tiles than there are barriers for cut ones");
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *q_s = smem, *ring = smem + Sh::QBUFS * Sh::QB, *raw = ring + NS * SLOT;
    Ctrl &c = *reinterpret_cast<Ctrl *>(smem + RING);
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const int rank = blockIdx.x & 1;                         // in the pair
    volatile int *abort = &c.abort;
    const uint64_t lim = p.wait_limit_ns;

    if (t == 0) {
        // full, s_free, p_full and q_full count in the first CTA, for both
        for (int i = 0; i < NS; ++i) {
            mbar_init(&c.full[i], Q8 ? 2 * CH_HELPERS : 2);
            mbar_init(&c.empty[i], 1);
        }
        for (int i = 0; i < RAWS; ++i) {
            mbar_init(&c.raw_full[i], 1);
            mbar_init(&c.raw_empty[i], CH_HELPERS);
        }
        for (int i = 0; i < 8; ++i) mbar_init(&c.bnd[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c.s_full[i], 1);
            mbar_init(&c.p_full[i], CH_SOFT);                // four warps of each CTA
            mbar_init(&c.s_free[i], CH_SOFT);
            mbar_init(&c.o_done[i], 1);
            for (int k = 0; k < 4; ++k) mbar_init(&c.m_out[i][k], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c.q_full[i], 2 * CH_HELPERS);
            mbar_init(&c.q_free[i], 1);
        }
        for (int i = 0; i < SEGS; ++i) {
            mbar_init(&c.seg_full[i], 1);
            mbar_init(&c.seg_empty[i], CH_ROLES);
        }
        mbar_init(&c.drain, 1);
        c.abort = 0;
        fence_barrier_init();
    }
    if (warp == CH_MMA) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&c.tmem)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    wait_prior_grid();
    find_work(p, c, *reinterpret_cast<FindScratch *>(q_s), warp, lane);
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                          // the pair's barriers and TMEM are ready
    tc_fence_after();
    const uint32_t tmem = c.tmem;
    const uint32_t ring_a = smem_u32(ring);
    // The next segment, false at the end.  Its wait ignores the abort flag: after
    // a time-out every role still walks through all segments, keeps to its named
    // barriers and does nothing else.
    uint32_t segs = 0;
    Seg w;
    auto next_segment = [&]() -> bool {
        const uint32_t k = segs % SEGS;
        bool got = mbar_wait_bounded(&c.seg_full[k], (segs / SEGS) & 1u, SEG_WAIT_NS);
        got = __all_sync(0xffffffffu, got);
        w = c.seg[k];
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.seg_empty[k]);
        ++segs;
        return got && w.n > 0;
    };
    // registers after the split: 8 x 32 x 200 + 8 x 32 x 56 = 65,536
    if (warp >= CH_LOAD && warp < CH_HELP) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == CH_LOAD) {
        // ---------------------------------------------------------- K, V loads
        uint8_t *dst0 = Q8 ? raw : ring;
        constexpr int NSL = Q8 ? RAWS : NS;
        constexpr uint32_t BYTES = Q8 ? RAW : SLOT;
        // elements of a box row: 128 bytes, or half a 128-wide head's 64 codes
        constexpr int CK = Q8 ? 128 : 64, CV = Q8 ? D / 2 : 64;
        constexpr int KCH = D / CK, VCH = D / 2 / CV;         // boxes across
        uint64_t *empty = Q8 ? c.raw_empty : c.empty;
        const int32_t P = p.kv.page_tokens;
        const int sh_k = __ffs(min(P, Sh::KTOK)) - 1, sh_v = __ffs(min(P, Sh::VTOK)) - 1;
        uint32_t slot = 0, phase = 0, used = 0, last = 0;     // slots loaded at least once, their latest phases
        uint32_t nb = 0;                                      // boundary tiles so far
        bool ok = true;
        // this lane's box of a slot: place in the tensor and in the slot
        int32_t x = 0, y = 0;
        uint32_t at = 0;
        bool mine = false;
        const int32_t *bt = nullptr;
        auto plan = [&](int32_t e) {
            bool v;
            int32_t tile;
            slot_at<Sh::LEAD>(e, w.n, &v, &tile);
            const int sh = v ? sh_v : sh_k;
            const int32_t toks = v ? Sh::VTOK : Sh::KTOK;
            const int lb = __ffs(toks) - 1 - sh;              // log2 of the boxes down
            const int32_t ch = lane >> lb, i = lane & ((1 << lb) - 1);
            mine = ch < (v ? VCH : KCH);
            const int32_t tok = (w.j0 + tile) * CH_TILE + (v ? 0 : rank * Sh::KTOK) + (i << sh);
            x = w.g * D + (v ? rank * (D / 2) + ch * CV : ch * CK);
            const int32_t row_bytes = v && Q8 ? CV : 128;
            at = static_cast<uint32_t>((ch * toks + (i << sh)) * row_bytes);
            // boxes without a visible token read zeros (a row past the cache)
            y = p.kv.num_pages << p.kv.page_shift;
            if (mine && tok <= w.hi_tok && tok + (1 << sh) > w.lo_tok) {
                const int32_t page = __ldg(bt + (tok >> p.kv.page_shift));
                if (page >= 0 && page < p.kv.num_pages) y = (page << p.kv.page_shift) + (tok & (P - 1));
                else record_error(p.kv.status, ST_BAD_PAGE);
            }
        };
        while (next_segment()) {
            if (!ok) continue;
            bt = p.kv.block_table + static_cast<int64_t>(w.b) * p.kv.max_pages;
            const int32_t n = w.n;
            plan(0);
            for (int32_t e = 0; e < 2 * n; ++e) {
                bool v;
                int32_t tile;
                slot_at<Sh::LEAD>(e, n, &v, &tile);
                const int32_t xx = x, yy = y;
                const uint32_t aa = at;
                const bool mm = mine;
                if (e + 1 < 2 * n) plan(e + 1);               // page lookups run under this slot's wait
                if (!warp_wait(&empty[slot], phase ^ 1u, abort, lim)) {
                    ok = false;
                    break;
                }
                uint32_t bar;
                if constexpr (Q8) {
                    bar = smem_u32(&c.raw_full[slot]);
                    if (lane == 0) mbar_arrive_expect_tx(&c.raw_full[slot], BYTES);
                } else if (v && w.cut(tile)) {
                    // the helpers clear rows of this one before the products see it
                    bar = smem_u32(&c.bnd[nb & 7u]);
                    if (lane == 0) mbar_arrive_expect_tx(&c.bnd[nb & 7u], BYTES);
                    ++nb;
                } else {
                    bar = of_first(&c.full[slot]);
                    if (lane == 0) cluster_arrive_expect_tx(bar, BYTES);
                }
                __syncwarp();
                if (mm) tma_load_2d_pair(dst0 + slot * BYTES + aa, v ? &tv : &tk, bar, xx, yy);
                used |= 1u << slot;
                last = (last & ~(1u << slot)) | (phase << slot);
                if (++slot == NSL) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
        }
        // after an abort copies may be in flight: let them land (their barriers
        // may be the other CTA's, so give them the time instead)
        if (!ok && lane == 0) {
            if (Q8)
                for (int i = 0; i < NSL; ++i)
                    if (used & (1u << i)) mbar_wait_bounded(&c.raw_full[i], (last >> i) & 1u, lim);
            const long long t0 = clock64();
            while (clock64() - t0 < 4000000) {}
        }
        __syncwarp();
    } else if (warp == CH_SCHED) {
        // ----------------------------------------------------------- segments
        Walk walk(p, c);
        Split split = {0, 0, 0, 0, 0};
        for (uint32_t i = 0;; ++i) {
            bool head = false;
            int32_t rest = 0;
            Seg x = walk.next(p, &head, &rest);
            x.place = head && rest == 0 ? -1 : 2 * static_cast<int32_t>(blockIdx.x >> 1) + (head ? 1 : 0);
            if (x.n > 0 && head && rest > 0) {
                // the unit's other tiles lie in the next pairs' shares
                split.parts = 1;
                while (c.total * ((blockIdx.x >> 1) + split.parts) / c.pairs < c.w1 + rest) ++split.parts;
                split.rows = x.rows;
                split.s0 = x.s0;
                split.v0 = x.v0;
                split.g = x.g;
            }
            const uint32_t k = i % SEGS;
            if (i >= SEGS) mbar_wait_bounded(&c.seg_empty[k], (i / SEGS - 1) & 1u, SEG_WAIT_NS);
            __syncwarp();
            if (lane == 0) {
                c.seg[k] = x;
                mbar_arrive(&c.seg_full[k]);
            }
            if (x.n == 0) break;
        }
        if (lane == 0 && rank == 0) reinterpret_cast<Split *>(p.ws)[blockIdx.x >> 1] = split;
        __syncwarp();
    } else {
        // --------------------------------------------------------------- MMAs
        // The warp runs as one and elects the issuing thread at each batch;
        // descriptors pass through a broadcast, so that their arithmetic is
        // uniform.  With P beside S, one warp issues the score products and the
        // other the second ones, so that neither waits for what the other needs;
        // else the first warp issues both.
        const bool do_s = rank == 0 && warp == CH_MMA, do_o = rank == 0 && (Sh::OWN_P ? warp == CH_MMA2 : warp == CH_MMA);
        constexpr uint32_t idesc_s = umma_idesc_f16_f32(CH_ROWS, CH_TILE);
        constexpr uint32_t idesc_o = umma_idesc_f16_f32(CH_ROWS, D) | (1u << 16);   // B: dims contiguous
        const uint64_t kd0 = sw128_kmajor_desc(0), vd0 = sw128_mn_desc(0, Sh::VTOK * 128);
        const uint32_t tm = uniform(tmem);
        uint32_t slot = 0, phase = 0, it = 0, seg = 0;
        bool ok = true;
        auto advance = [&](int32_t by) {
            slot += by;
            if (slot >= NS) {
                slot -= NS;
                phase ^= 1u;
            }
        };
        // S(i) = Q . K(i)^T
        auto scores = [&](uint32_t i, bool last) {
            ok = ok && warp_wait(&c.full[slot], phase, abort, lim);
            if (!ok) return;
            tc_fence_after();
            const uint32_t qb = Sh::QBUFS == 2 ? uniform(seg & 1u) : 0u;
            const uint64_t qd = kd0 | (uniform(smem_u32(q_s) + qb * Sh::QB) >> 4);
            const uint64_t kd = kd0 | (uniform(ring_a + slot * SLOT) >> 4);
            const uint32_t d = tm + TM_S + uniform(i & 1u) * 128u;
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t ch = kk >> 2, in = (kk & 3) * 32;
                    umma2_f16(d, qd + ((ch * (CH_HALF * 128u) + in) >> 4), kd + ((ch * (Sh::KTOK * 128u) + in) >> 4),
                              idesc_s, kk > 0 ? 1u : 0u);
                }
                umma2_commit(&c.s_full[i & 1u]);
                umma2_commit(&c.empty[slot]);
                if (last) umma2_commit(&c.q_free[qb]);
            }
            __syncwarp();
        };
        // O (+)= P(i) . V(i)
        auto values = [&](uint32_t i, bool first) {
            ok = ok && warp_wait(&c.full[slot], phase, abort, lim);
            ok = ok && warp_wait(&c.p_full[i & 1u], (i >> 1) & 1u, abort, lim);
            if (!ok) return;
            tc_fence_after();
            const uint64_t vd = vd0 | (uniform(ring_a + slot * SLOT) >> 4);
            const uint32_t pa = tm + Sh::TM_P + uniform(i & 1u) * Sh::P_STRIDE;
            const uint32_t add = uniform(first ? 0u : 1u);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < CH_TILE / 16; ++kk)
                    umma2_f16_ta(tm + TM_O, pa + kk * 8u, vd + ((kk * 2048u) >> 4), idesc_o, kk > 0 ? 1u : add);
                umma2_commit(&c.o_done[i & 1u]);
                umma2_commit(&c.empty[slot]);
            }
            __syncwarp();
        };
        while (next_segment()) {
            if (!ok || !(do_s || do_o)) continue;
            const int32_t n = w.n, lead = min(Sh::LEAD, n);
            if (do_s) ok = warp_wait(&c.q_full[Sh::QBUFS == 2 ? seg & 1u : 0u], (Sh::QBUFS == 2 ? seg >> 1 : seg) & 1u, abort, lim);
            if constexpr (Sh::OWN_P) {
                // this warp's slots of the segment's 2 n: where they are is given by slot_at
                int32_t at = 0;
                for (int32_t j = 0; ok && j < n; ++j) {
                    const int32_t e = do_s ? (j < lead ? j : 2 * j - lead + 1) : slot_of_v<Sh::LEAD>(j, n);
                    advance(e - at);
                    at = e;
                    const uint32_t i = it + j;
                    if (do_s) {
                        // the scores two tiles before are in registers (the first two tiles of a segment: those of the one before)
                        if (i > 1) ok = warp_wait(&c.s_free[i & 1u], ((i - 2) >> 1) & 1u, abort, lim);
                        scores(i, j == n - 1);
                    } else {
                        values(i, j == 0);
                    }
                }
                advance(2 * n - at);
            } else {
                scores(it, n == 1);
                advance(1);
                if (n > 1) {
                    scores(it + 1, n == 2);
                    advance(1);
                }
                for (int32_t j = 0; ok && j < n; ++j) {
                    values(it + j, j == 0);
                    advance(1);
                    if (j + 2 < n) {
                        scores(it + j + 2, j + 3 == n);
                        advance(1);
                    }
                }
            }
            it += n;
            ++seg;
        }
        if (!ok) {                                            // products still running
            if (elect_one()) {
                umma2_commit(&c.drain);
                mbar_wait_bounded(&c.drain, 0, lim);
            }
            __syncwarp();
        }
    }
    } else if (warp >= CH_HELP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        // --------------------- queries, cut value tiles, E4M3 codes to FP16 tiles
        const int ht = t - CH_HELP * 32;                      // 0 .. 127
        uint32_t seg = 0, slot = 0, phase = 0, rslot = 0, rphase = 0, ring0 = 0, nb = 0;
        bool ok = true;                                       // false: keep to the barriers, do nothing
        while (next_segment()) {
            const int32_t n = w.n;
            const uint32_t qb = Sh::QBUFS == 2 ? seg & 1u : 0u, quse = Sh::QBUFS == 2 ? seg >> 1 : seg;   // buffer, its uses before
            if (ok && quse > 0) ok = warp_wait(&c.q_free[qb], (quse - 1) & 1u, abort, lim);
            if (ok) {
                // the warp's 32 rows: a lane finds one row's queries, then
                // all lanes copy the rows, 512 bytes at a time
                constexpr int RPI = 256 / D;                   // rows per copy instruction
                const int r0 = (ht >> 5) * 32, ur = rank * CH_HALF + r0 + lane;
                const int32_t v = w.v0 + ur, tok = by_group(p, v), h = v - tok * p.group;
                const bool in = ur < w.rows;
                const uint64_t mine = in ? reinterpret_cast<uint64_t>(p.q) +
                    ((static_cast<int64_t>(w.s0) + tok) * p.q_stride + (w.g * p.group + h) * D) * 2 : 0;
                const int pc = lane & (D / 8 - 1);
                const uint32_t dst = smem_u32(q_s) + qb * Sh::QB + (pc >> 3) * (CH_HALF * 128u);
#pragma unroll 8
                for (int i = 0; i < 32 / RPI; ++i) {
                    const int k = i * RPI + lane / (D / 8);
                    const uint64_t src = __shfl_sync(0xffffffffu, mine, k);
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + sw128(r0 + k, pc & 7)),
                                 "l"((src ? src : reinterpret_cast<uint64_t>(p.q)) + (src ? pc * 16 : 0)), "r"(src ? 16 : 0)
                                 : "memory");
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) cluster_arrive(of_first(&c.q_full[qb]));
            }
            ++seg;
            if constexpr (!Q8) {
                // Rows of V that nothing attends may hold anything (the ends of
                // loaded pages): zero weights must meet zeros.
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int32_t tile = k == 0 ? 0 : n - 1;
                    if ((k == 1 && n == 1) || !w.cut(tile)) continue;
                    if (ok) ok = warp_wait(&c.bnd[nb & 7u], (nb >> 3) & 1u, abort, lim);
                    ++nb;
                    const uint32_t vs = (ring0 + slot_of_v<Sh::LEAD>(tile, n)) % NS;
                    if (ok) {
                        uint8_t *v = ring + vs * SLOT;
                        const int32_t a = w.lo_tok - (w.j0 + tile) * CH_TILE, z = w.hi_tok + 1 - (w.j0 + tile) * CH_TILE;
                        if (ht < a || ht >= z) {
#pragma unroll
                            for (int ch = 0; ch < D / 128; ++ch)
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    *reinterpret_cast<uint4 *>(v + (ch * CH_TILE + ht) * 128 + i * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async_smem();
                    }
                    named_barrier(BAR_HELP, 32 * CH_HELPERS);
                    if (ok && ht == 0) cluster_arrive(of_first(&c.full[vs]));
                }
                ring0 = (ring0 + 2 * n) % NS;
            } else {
                const int32_t *bt = p.kv.block_table + static_cast<int64_t>(w.b) * p.kv.max_pages;
                // scale bytes of the slot's tokens, one per thread, looked up two
                // slots ahead: first the page, then the byte
                auto token = [&](int32_t e) -> int32_t {       // this thread's token of slot e, -1: none
                    bool v;
                    int32_t tile;
                    if (e >= 2 * n) return -1;
                    slot_at<Sh::LEAD>(e, n, &v, &tile);
                    const int32_t tok = (w.j0 + tile) * CH_TILE + (v ? 0 : rank * Sh::KTOK) + ht;
                    return ht < (v ? Sh::VTOK : Sh::KTOK) && tok >= w.lo_tok && tok <= w.hi_tok ? tok : -1;
                };
                auto page_of = [&](int32_t tok) -> int32_t { return tok >= 0 ? __ldg(bt + (tok >> p.kv.page_shift)) : -1; };
                auto byte_of = [&](int32_t e, int32_t tok, int32_t page) -> uint32_t {
                    if (page < 0 || page >= p.kv.num_pages) return 127u;
                    bool v;
                    int32_t tile;
                    slot_at<Sh::LEAD>(e, n, &v, &tile);
                    return __ldg((v ? p.kv.v_scale : p.kv.k_scale) +
                                 ((static_cast<int64_t>(page) << p.kv.page_shift) + (tok & (p.kv.page_tokens - 1))) * p.kv.hkv + w.g);
                };
                int32_t tok1 = token(0), page1 = page_of(tok1);
                uint32_t byte = byte_of(0, tok1, page1);
                tok1 = token(1);
                page1 = page_of(tok1);
                uint32_t par = 0;
                for (int32_t e = 0; e < 2 * n; ++e) {
                    bool v;
                    int32_t tile;
                    slot_at<Sh::LEAD>(e, n, &v, &tile);
                    const int32_t tok0 = (w.j0 + tile) * CH_TILE;      // V: rows outside lo_tok .. hi_tok are cleared
                    const int32_t a = v ? w.lo_tok - tok0 : 0, z = v ? w.hi_tok + 1 - tok0 : CH_TILE;
                    // 2^(byte - 127) as FP16 (2^-15 is subnormal)
                    const int x = max(112, min(135, static_cast<int>(byte))) - 127;
                    c.scale[par][ht] = static_cast<uint16_t>(x >= -14 ? (x + 15) << 10 : 0x200);
                    byte = byte_of(e + 1, tok1, page1);                // in flight under the conversion
                    tok1 = token(e + 2);
                    page1 = page_of(tok1);
                    if (ok) ok = warp_wait(&c.raw_full[rslot], rphase, abort, lim);
                    if (ok) ok = warp_wait(&c.empty[slot], phase ^ 1u, abort, lim);
                    named_barrier(BAR_HELP, 32 * CH_HELPERS);          // the scales are in
                    if (ok) {
                        constexpr int N = RAW / 16 / (32 * CH_HELPERS); // 16-code pieces per thread
                        // a row of codes: 128 bytes, 64 for V of a 128-wide head
                        const int sh = v && D == 128 ? 2 : 3;           // log2 of its pieces
                        const int pc = ht & ((1 << sh) - 1);
                        const int toks = v ? Sh::VTOK : Sh::KTOK;
                        const uint8_t *src = raw + rslot * RAW + ht * 16;
                        uint8_t *dst = ring + slot * SLOT;
                        uint4 in[N];
#pragma unroll
                        for (int i = 0; i < N; ++i) in[i] = *reinterpret_cast<const uint4 *>(src + i * (16 * 32 * CH_HELPERS));
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            const int rr = (ht >> sh) + i * ((32 * CH_HELPERS) >> sh);
                            const int blk = rr / toks, tk2 = rr & (toks - 1);      // 128 dims, token
                            const uint32_t sc = c.scale[par][tk2] * 0x10001u;
                            const uint32_t cw[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
                            uint32_t o[8];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
                                    "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
                                    : "=r"(o[2 * k]), "=r"(o[2 * k + 1])
                                    : "r"(cw[k]));
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(o[k]) : "r"(sc));
                            if (tk2 < a || tk2 >= z) {
#pragma unroll
                                for (int k = 0; k < 8; ++k) o[k] = 0u;
                            }
                            // dims 16 pc .. of the row: chunk pc / 4, pieces 2 (pc % 4) and + 1;
                            // lanes of the upper four pieces store the odd one first, which
                            // spreads a row's eight stores over all banks
                            uint8_t *ck = dst + (2 * blk + (pc >> 2)) * (toks * 128);
                            const uint32_t p0 = 2 * (pc & 3), first = pc >> 2;
                            const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
                            *reinterpret_cast<uint4 *>(ck + sw128(tk2, p0 + first)) = first ? hi : lo;
                            *reinterpret_cast<uint4 *>(ck + sw128(tk2, p0 + 1 - first)) = first ? lo : hi;
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&c.raw_empty[rslot]);
                            cluster_arrive(of_first(&c.full[slot]));
                        }
                    }
                    par ^= 1u;
                    if (++slot == NS) {
                        slot = 0;
                        phase ^= 1u;
                    }
                    if (++rslot == RAWS) {
                        rslot = 0;
                        rphase ^= 1u;
                    }
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        // ------------------------------------------------------------- softmax
        constexpr int OC = D / 2;                              // output columns per thread
        const int lq = warp & 3, grp = warp >> 2, row = lq * 32 + lane;
        const uint32_t lane_base = static_cast<uint32_t>(lq * 32) << 16;
        const uint32_t ts = tmem + TM_S + grp * 128u + lane_base;
        const uint32_t tp = tmem + Sh::TM_P + grp * Sh::P_STRIDE + lane_base;
        const float cs = p.scale * 1.4426950408889634f;        // scores in powers of two
        const uint32_t p_full0 = of_first(&c.p_full[grp]), s_free0 = of_first(&c.s_free[grp]);
        uint32_t it = 0;                                       // tiles before the segment
        bool ok = true;                                        // false: keep to the barriers, do nothing
        while (next_segment()) {
            const int32_t n = w.n;
            // rows past the unit's last behave like it (their queries are zeros)
            const int32_t mine = w.rows - rank * CH_HALF;      // rows in use here, if positive
            const int32_t vr = w.v0 + min(rank * CH_HALF + row, w.rows - 1);
            const int32_t tok = by_group(p, vr), pos = w.p0 + tok;
            const int32_t first = p.window > 0 ? max(0, pos - p.window + 1) : 0;
            const bool live = lq * 32 < mine;                  // some row of this warp is in use
            float m = -INFINITY, l = 0.0f;
            for (int32_t j = (grp - it) & 1; ok && j < n; j += 2) {
                const uint32_t i = it + j;                     // tile i & 1 == grp
                ok = warp_wait(&c.s_full[grp], (i >> 1) & 1u, abort, lim);
                const int32_t base = (w.j0 + j) * CH_TILE;
                const int32_t hi = pos - base, lo = first - base;              // visible: lo <= column <= hi
                const bool masked = __any_sync(0xffffffffu, hi < CH_TILE - 1 || lo > 0);
                uint32_t s[4][32];
                float mx = -INFINITY;
                if (ok && live) {
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k) tmem_ld_32x32b_x32(ts + k * 32u, s[k]);
                    tmem_ld_wait();
                }
                if constexpr (Sh::OWN_P) {
                    tc_fence_before();
                    __syncwarp();
                    if (ok && lane == 0) cluster_arrive(s_free0);
                }
                if (ok && live) {
                    if (masked) {
#pragma unroll
                        for (int e = 0; e < CH_TILE; ++e)
                            if (e > hi || e < lo) s[e >> 5][e & 31] = 0xff800000u;       // -inf
                    }
                    float a[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) a[e] = fmaxf(__uint_as_float(s[0][e]), __uint_as_float(s[0][e + 4]));
#pragma unroll
                    for (int e = 8; e < CH_TILE; e += 8)
#pragma unroll
                        for (int f = 0; f < 4; ++f)
                            a[f] = fmaxf(fmaxf(a[f], __uint_as_float(s[e >> 5][(e & 31) + f])),
                                         __uint_as_float(s[e >> 5][(e & 31) + f + 4]));
                    mx = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
                }
                // the maximum in use at the tile before, and the one for this tile
                if (ok && i > 0) ok = warp_wait(&c.m_out[grp ^ 1][lq], ((i - 1) >> 1) & 1u, abort, lim);
                const float mp = j > 0 ? c.mrow[grp ^ 1][row] : -INFINITY;
                const bool grow = (mx - mp) * cs > RESCALE;
                const float mi = grow ? mx : mp;
                c.mrow[grp][row] = mi;
                __syncwarp();
                if (lane == 0) mbar_arrive(&c.m_out[grp][lq]);
                // P's columns are free when the tile before last is done with them
                if (Sh::OWN_P && ok && i > 1) ok = warp_wait(&c.o_done[grp], ((i - 2) >> 1) & 1u, abort, lim);
                if (ok && live) {
                    const float mc = mi == -INFINITY ? 0.0f : mi * cs;
                    if (m != mi) l *= exp2_approx(m * cs - mc);                // 0 at the first
                    m = mi;
                    float2 sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
                    const float2 c2 = make_float2(cs, cs), mc2 = make_float2(-mc, -mc);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t o[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 y = fma2(make_float2(__uint_as_float(s[k][2 * e]), __uint_as_float(s[k][2 * e + 1])), c2, mc2);
                            const float2 z = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                            sum[e & 1] = add2(sum[e & 1], z);
                            const __half2 h = __floats2half2_rn(z.x, z.y);
                            o[e] = *reinterpret_cast<const uint32_t *>(&h);
                        }
                        tmem_st_x16(tp + k * 16u, o);
                    }
                    l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
                }
                if (ok && i > 0) ok = warp_wait(&c.o_done[grp ^ 1], ((i - 1) >> 1) & 1u, abort, lim);
                if (ok && live && j > 0 && __any_sync(0xffffffffu, grow)) {
                    tc_fence_after();
                    const float alpha = grow ? exp2_approx((mp - mi) * cs) : 1.0f;
                    uint32_t u[32];
#pragma unroll 1
                    for (int k = 0; k < D / 32; ++k) {
                        tmem_ld_32x32b_x32(tmem + TM_O + lane_base + k * 32u, u);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * alpha);
                        tmem_st_x32(tmem + TM_O + lane_base + k * 32u, u);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (ok && lane == 0) cluster_arrive(p_full0);
            }
            it += n;
            // the segment's sums: its rows' output, or its part of it
            if (ok) ok = warp_wait(&c.o_done[(it - 1) & 1u], ((it - 1) >> 1) & 1u, abort, lim);
            named_barrier(BAR_PAIR + lq, 64);
            // both groups' sums at the last tile's maximum, exchanged in place of the maxima
            const float mlast = c.mrow[(it - 1) & 1u][row];
            l = l > 0.0f ? l * exp2_approx((m - mlast) * cs) : 0.0f;
            named_barrier(BAR_PAIR + lq, 64);
            c.mrow[grp][row] = l;
            named_barrier(BAR_PAIR + lq, 64);
            l += c.mrow[grp ^ 1][row];
            if (ok && live) {
                tc_fence_after();
                const uint32_t to = tmem + TM_O + lane_base + grp * OC;
                const bool in = row < mine, whole = w.place < 0;
                const float inv = l > 0.0f ? 1.0f / l : 0.0f;
                const int32_t h = vr - tok * p.group, ur = rank * CH_HALF + row;
                __half *out = static_cast<__half *>(p.out) +
                              ((static_cast<int64_t>(w.s0) + tok) * p.hq + w.g * p.group + h) * D + grp * OC;
                float *part = nullptr;
                if (!whole) {
                    part = reinterpret_cast<float *>(p.ws + WS_O) + (static_cast<int64_t>(w.place) * p.ws_rows + ur) * D + grp * OC;
                    if (in && grp == 0)
                        *reinterpret_cast<float2 *>(p.ws + WS_ML + (static_cast<int64_t>(w.place) * CH_ROWS + ur) * 8) =
                            make_float2(mlast == -INFINITY ? -INFINITY : mlast * cs, l);
                }
                // rolled: a unit's end is code that has left the instruction cache
#pragma unroll 1
                for (int k = 0; k < OC / 32; ++k) {
                    uint32_t u[32];
                    tmem_ld_32x32b_x32(to + k * 32u, u);
                    tmem_ld_wait();
                    if (!in) continue;
                    if (whole) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            uint32_t x[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const __half2 hh = __floats2half2_rn(__uint_as_float(u[i + 2 * e]) * inv,
                                                                     __uint_as_float(u[i + 2 * e + 1]) * inv);
                                x[e] = *reinterpret_cast<const uint32_t *>(&hh);
                            }
                            *reinterpret_cast<uint4 *>(out + 32 * k + i) = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<uint4 *>(part + 32 * k + i) = make_uint4(u[i], u[i + 1], u[i + 2], u[i + 3]);
                    }
                }
                tc_fence_before();
            }
            // sums and O are read: the other group may go on to the next tile
            named_barrier(BAR_PAIR + lq, 64);
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();                                          // nothing of the pair reaches into the other any more
    tc_fence_after();
    if (t == 0 && c.abort) record_error(p.kv.status, ST_TIMEOUT);
    if (warp == CH_MMA)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    allow_next_grid();
}

// Joins the parts of each split unit: block x the unit that pair x began (part 0
// in its second place, part i in the first place of the i-th pair after it), a
// warp per row.
template <int D>
__global__ void __launch_bounds__(256)
chunk_join_kernel(const ChunkParams p)
{
    constexpr int N = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    wait_prior_grid();
    const Split sp = reinterpret_cast<const Split *>(p.ws)[blockIdx.x];
    const int32_t n = sp.parts;
    if (n == 0) return;
    const float2 *ml = reinterpret_cast<const float2 *>(p.ws + WS_ML);
    const float *po = reinterpret_cast<const float *>(p.ws + WS_O);
    auto place = [&](int32_t i) { return 2 * (static_cast<int64_t>(blockIdx.x) + i) + (i == 0 ? 1 : 0); };
    for (int32_t row = blockIdx.y * 8 + warp; row < sp.rows; row += 8 * gridDim.y) {
        float mx = -INFINITY, sum = 0.0f;
        for (int32_t i = lane; i < n; i += 32) mx = fmaxf(mx, ml[place(i) * CH_ROWS + row].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        float acc[N];
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = 0.0f;
        for (int32_t i0 = 0; i0 < n; i0 += 32) {
            float wt = 0.0f;
            if (i0 + lane < n) {
                const float2 x = ml[place(i0 + lane) * CH_ROWS + row];
                wt = x.x == -INFINITY ? 0.0f : exp2_approx(x.x - mx);      // a part in which the row saw nothing
                sum = fmaf(x.y, wt, sum);
            }
            const int32_t k = min(32, n - i0);
#pragma unroll 4
            for (int32_t i = 0; i < k; ++i) {
                const float f = __shfl_sync(0xffffffffu, wt, i);
                const float4 *src = reinterpret_cast<const float4 *>(po + (place(i0 + i) * p.ws_rows + row) * D) + lane;
#pragma unroll
                for (int e = 0; e < N / 4; ++e) {
                    const float4 x = src[32 * e];
                    acc[4 * e] = fmaf(x.x, f, acc[4 * e]);
                    acc[4 * e + 1] = fmaf(x.y, f, acc[4 * e + 1]);
                    acc[4 * e + 2] = fmaf(x.z, f, acc[4 * e + 2]);
                    acc[4 * e + 3] = fmaf(x.w, f, acc[4 * e + 3]);
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        const int32_t v = sp.v0 + row, tok = v / p.group, h = v - tok * p.group;
        __half *out = static_cast<__half *>(p.out) +
                      ((static_cast<int64_t>(sp.s0) + tok) * p.hq + sp.g * p.group + h) * D;
#pragma unroll
        for (int e = 0; e < N / 4; ++e) {
            const __half2 a = __floats2half2_rn(acc[4 * e] * inv, acc[4 * e + 1] * inv);
            const __half2 b = __floats2half2_rn(acc[4 * e + 2] * inv, acc[4 * e + 3] * inv);
            uint2 u;
            u.x = *reinterpret_cast<const uint32_t *>(&a);
            u.y = *reinterpret_cast<const uint32_t *>(&b);
            reinterpret_cast<uint2 *>(out)[32 * e + lane] = u;
        }
    }
}

constexpr size_t CH_SMEM = RING + sizeof(Ctrl);
static_assert(CH_SMEM <= 232448, "shared memory budget");

template <int D, bool Q8>
int launch(const ChunkParams &p, const void *tk, const void *tv, int grid, bool overlap, cudaStream_t stream)
{
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return static_cast<int>(cudaErrorInvalidDevice);
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!done[dev]) {
            const cudaError_t e = cudaFuncSetAttribute(chunk_kernel<D, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       static_cast<int>(CH_SMEM));
            if (e != cudaSuccess) return static_cast<int>(e);
            done[dev] = true;
        }
    }
    void *args[] = {const_cast<void *>(tk), const_cast<void *>(tv), const_cast<ChunkParams *>(&p)};
    const int rc = launch_kernel(reinterpret_cast<const void *>(&chunk_kernel<D, Q8>), dim3(grid), dim3(CH_THREADS),
                                 CH_SMEM, stream, false, args);
    if (rc != 0) return rc;
    void *join[] = {const_cast<ChunkParams *>(&p)};
    const unsigned rows8 = static_cast<unsigned>(std::min(8, (p.ws_rows + 7) / 8));
    return launch_kernel(reinterpret_cast<const void *>(&chunk_join_kernel<D>), dim3(grid / 2, rows8), dim3(256), 0, stream,
                         overlap, join);
}

}  // namespace

int32_t chunk_part_rows(int32_t rows, int32_t group)
{
    return static_cast<int32_t>(std::min<int64_t>(CH_ROWS, static_cast<int64_t>(rows) * group));
}

size_t chunk_workspace_bytes(int32_t rows, int32_t group, int32_t head_dim)
{
    return WS_O + size_t{2} * CHUNK_MAX_PAIRS * chunk_part_rows(rows, group) * head_dim * 4;
}

// tokens per box of the K and V tensor maps
void chunk_boxes(int32_t head_dim, int32_t page_tokens, int32_t *box_k, int32_t *box_v)
{
    (void)head_dim;
    *box_k = std::min(page_tokens, CH_TILE / 2);
    *box_v = std::min(page_tokens, CH_TILE);
}

int launch_chunk(const ChunkParams &p, const void *tk, const void *tv, int sms, bool overlap, void *stream)
{
    const int grid = 2 * std::min(sms / 2, static_cast<int>(CHUNK_MAX_PAIRS));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.kv.head_dim == 128)
        return p.kv.e4m3 ? launch<128, true>(p, tk, tv, grid, overlap, s) : launch<128, false>(p, tk, tv, grid, overlap, s);
    return p.kv.e4m3 ? launch<256, true>(p, tk, tv, grid, overlap, s) : launch<256, false>(p, tk, tv, grid, overlap, s);
}

}  // namespace qsa
