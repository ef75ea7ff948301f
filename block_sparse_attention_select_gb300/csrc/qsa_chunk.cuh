// Dense attention over the paged cache: what its two kernels share, the line of
// work and its segments, and the kernel that joins partial results.
#pragma once
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qsa_device.cuh"
#include "qsa_internal.h"
#include "qsa_seq.cuh"

namespace qsa {
namespace {

// A kernel's geometry G gives ROWS ((token, query head) pairs of a unit), TILE
// (tokens of a tile), UNIT_COST (tiles' worth of time that a unit costs besides
// its tiles), THREADS and WARPS of a CTA, WORKERS (at most; a worker is a CTA or
// a pair of them).

// A run of tiles of one unit, a worker's next piece of work.
struct alignas(16) Seg {
    int32_t n, j0;                           // tiles j0 .. j0 + n - 1; n = 0: no more work
    int32_t b, g;                            // request, KV head
    int32_t s0, p0, v0, rows;                // request's first row and position, unit's first (token, head) pair, pairs in use
    int32_t lo_tok, hi_tok;                  // tokens that some row attends: lo_tok .. hi_tok
    int32_t place;                           // workspace place of the partial result, -1: this is the whole unit
    int32_t pad;

    // whether tile j0 + k holds tokens that no row attends
    __device__ __forceinline__ bool cut(int32_t k, int32_t tile) const
    {
        const int32_t t0 = (j0 + k) * tile;
        return t0 < lo_tok || t0 + tile - 1 > hi_tok;
    }
};
// A unit that lies across workers, as the join kernel needs it (written by the
// worker that holds the unit's first tile).
struct Split {
    int32_t parts;                           // 0: none
    int32_t rows;                            // rows of the unit
    int32_t s0, v0, g;                       // request's first row, unit's first (token, head) pair, KV head
};

// Workspace: a Split per worker, then per place (two for each worker: 0 for a
// unit begun before its share, 1 for one that goes on after it) the rows'
// (maximum score before the scale, sum), then their unnormalised outputs.
constexpr size_t WS_ML = 4096;
static_assert(sizeof(Split) * CHUNK_MAX_CTAS <= WS_ML && sizeof(Split) * CHUNK_MAX_PAIRS <= WS_ML, "workspace");
template <int ROWS, int WORKERS>
constexpr size_t ws_o() { return WS_ML + size_t{2} * WORKERS * ROWS * 8; }

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

template <typename G>
__device__ __forceinline__ int32_t units_of(const ChunkParams &p, const Seq &s)
{
    return (s.n * p.group + G::ROWS - 1) / G::ROWS;
}

template <typename G>
__device__ __forceinline__ Unit unit_of(const ChunkParams &p, const Seq &s, int32_t m)
{
    Unit u;
    u.v0 = m * G::ROWS;
    const int32_t end = min(s.n * p.group, u.v0 + G::ROWS);
    u.rows = end - u.v0;
    const int32_t first = s.p0 + by_group(p, u.v0);
    u.hi_tok = s.p0 + by_group(p, end - 1);
    u.lo_tok = p.window > 0 ? max(0, first - p.window + 1) : 0;
    u.lo = u.lo_tok / G::TILE;
    u.hi = u.hi_tok / G::TILE + 1;
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
template <typename G, typename T>
__device__ __forceinline__ T block_scan(T x, T *warp_total, int warp, int lane, T *total)
{
    const T sc = warp_scan(x, lane);
    if (lane == 31) warp_total[warp] = sc;
    __syncthreads();
    T before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < G::WARPS; ++w) {
        if (w == warp) before = all;
        all += warp_total[w];
    }
    *total = all;
    return before + sc - x;
}

// A worker's share of the line.
struct Share {
    int64_t w0, w1;
    int64_t each;                            // the line's length, each * workers + rest,
    int32_t workers, rest;                   // over the workers that have work, the first ones
    int32_t b, m, g, off;                    // the unit that w0 lies in, and w0's place in it

    // length * worker / workers, rounded down
    __device__ __forceinline__ int64_t start(int32_t worker) const
    {
        return each * worker + static_cast<uint32_t>(rest * worker) / static_cast<uint32_t>(workers);
    }
};

// a / b for 0 <= a, 0 < b: the 64-bit division is a call of some hundred instructions.
__device__ __forceinline__ int64_t divide(int64_t a, int32_t b)
{
    return a >> 32 ? a / b : static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

// Shared memory that find_work needs.
template <typename G>
struct FindScratch {
    int32_t prefix[G::THREADS];
    int64_t units[G::WARPS], costs[G::WARPS];
};

// Finds worker `me`'s share of the line (of `n_workers`), by the whole CTA.  Each
// thread counts the units of a run of requests, then adds up the lengths of an
// equal run of units.
template <typename G>
__device__ __forceinline__ void find_work(const ChunkParams &p, Share &c, FindScratch<G> &s, int32_t me,
                                          int32_t n_workers, int warp, int lane)
{
    const int t = threadIdx.x;
    int32_t *prefix = s.prefix;
    const int32_t run = (p.kv.n_reqs + G::THREADS - 1) / G::THREADS;
    const int32_t r0 = min(t * run, p.kv.n_reqs), r1 = min(r0 + run, p.kv.n_reqs);
    int64_t mine = 0, all;
    for (int32_t b = r0; b < r1; ++b) {
        bool bad;
        mine += units_of<G>(p, seq_of(p.kv, b, &bad));
        if (bad && blockIdx.x == 0) record_error(p.kv.status, ST_BAD_ROW);
    }
    const int64_t before = block_scan<G>(mine, s.units, warp, lane, &all);
    prefix[t] = static_cast<int32_t>(before);
    // more units than the rows allow: requests that share rows, or none in order
    const bool wrong = all > INT32_MAX;
    if (wrong && blockIdx.x == 0 && t == 0) record_error(p.kv.status, ST_BAD_ROW);
    const int32_t units = wrong ? 0 : static_cast<int32_t>(all);
    __syncthreads();
    const int32_t u0 = static_cast<int32_t>(static_cast<int64_t>(units) * t / G::THREADS);
    const int32_t u1 = static_cast<int32_t>(static_cast<int64_t>(units) * (t + 1) / G::THREADS);
    int32_t b0 = 0, m0 = 0;
    Seq s0{0, 0, 0};
    int64_t cost = 0, total;
    if (u0 < u1) {
        int lo = 0;                                          // the last run that starts at or before u0
#pragma unroll
        for (int step = 256; step > 0; step >>= 1)
            if (lo + step < G::THREADS && prefix[lo + step] <= u0) lo += step;
        b0 = lo * run;
        m0 = u0 - prefix[lo];
        bool bad;
        s0 = seq_of(p.kv, b0, &bad);
        for (int32_t n = units_of<G>(p, s0); m0 >= n; n = units_of<G>(p, s0)) {
            m0 -= n;
            s0 = seq_of(p.kv, ++b0, &bad);
        }
        int32_t b = b0, m = m0;
        Seq sb = s0;
        for (int32_t u = u0; u < u1; ++u, ++m) {
            while (m >= units_of<G>(p, sb)) {
                sb = seq_of(p.kv, ++b, &bad);
                m = 0;
            }
            const Unit un = unit_of<G>(p, sb, m);
            cost += G::UNIT_COST + un.hi - un.lo;
        }
        cost *= p.kv.hkv;
    }
    int64_t at = block_scan<G>(cost, s.costs, warp, lane, &total);
    // MIN_SHARE each at least: a smaller share costs more in the join than it saves here
    const int32_t workers = total >= static_cast<int64_t>(n_workers) * G::MIN_SHARE
                                ? n_workers : (static_cast<int32_t>(total) + G::MIN_SHARE - 1) / G::MIN_SHARE;
    Share x;
    x.workers = max(workers, 1);
    x.each = divide(total, x.workers);
    x.rest = static_cast<int32_t>(total - x.each * x.workers);
    const int64_t w0 = me < workers ? x.start(me) : 0, w1 = me < workers ? x.start(me + 1) : 0;
    if (t == 0) {
        c.w0 = w0;
        c.w1 = w1;
        c.each = x.each;
        c.workers = x.workers;
        c.rest = x.rest;
    }
    if (w0 < w1 && at <= w0 && w0 < at + cost) {
        for (;; ++m0) {
            while (m0 >= units_of<G>(p, s0)) {
                bool bad;
                s0 = seq_of(p.kv, ++b0, &bad);
                m0 = 0;
            }
            const Unit un = unit_of<G>(p, s0, m0);
            const int32_t len = G::UNIT_COST + un.hi - un.lo;
            if (w0 < at + static_cast<int64_t>(len) * p.kv.hkv) {
                c.b = b0;
                c.m = m0;
                c.g = static_cast<int32_t>(divide(w0 - at, len));
                c.off = static_cast<int32_t>(w0 - at - static_cast<int64_t>(c.g) * len);
                break;
            }
            at += static_cast<int64_t>(len) * p.kv.hkv;
        }
    }
    __syncthreads();
}

// The share as segments.
template <typename G>
struct Walk {
    int64_t left;
    int32_t b, m, g, off, n_units;
    Seq s;

    __device__ __forceinline__ Walk(const ChunkParams &p, const Share &c)
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
        n_units = units_of<G>(p, s);
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
        const Unit u = unit_of<G>(p, s, m);
        // a unit's place in the line: G::UNIT_COST, then its tiles
        const int32_t len = G::UNIT_COST + u.hi - u.lo;
        const int32_t end = static_cast<int32_t>(min(static_cast<int64_t>(len), off + left));
        left -= end - off;
        x.j0 = u.lo + max(0, off - G::UNIT_COST);
        x.n = u.lo + max(0, end - G::UNIT_COST) - x.j0;      // 0: the share ends before the unit's first tile
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


// The scheduler warp: walks through the share and hands out its segments
// through a ring; `me` writes its split unit, if any, for the join kernel.
constexpr int SEGS = 4;                      // segments it may be ahead
constexpr uint64_t SEG_WAIT_NS = 10000000000ull;
// After a time-out, what is in flight is waited for at least this long, however
// short the limit that ran out: copies and products land within microseconds.
constexpr uint64_t DRAIN_NS = 10000000ull;
__device__ __forceinline__ uint64_t drain_limit(uint64_t lim) { return lim > DRAIN_NS ? lim : DRAIN_NS; }

struct SegRing {
    Seg seg[SEGS];
    uint64_t full[SEGS], empty[SEGS];
};

template <typename G>
__device__ __forceinline__ void schedule(const ChunkParams &p, const Share &c, SegRing &ring, int32_t me, bool tell, int lane)
{
    Walk<G> walk(p, c);
    Split split = {0, 0, 0, 0, 0};
    for (uint32_t i = 0;; ++i) {
        bool head = false;
        int32_t rest = 0;
        Seg x = walk.next(p, &head, &rest);
        x.place = head && rest == 0 ? -1 : 2 * me + (head ? 1 : 0);
        if (x.n > 0 && head && rest > 0) {
            // the unit's other tiles lie in the next workers' shares
            split.parts = 1;
            while (c.start(me + split.parts) < c.w1 + rest) ++split.parts;
            split.rows = x.rows;
            split.s0 = x.s0;
            split.v0 = x.v0;
            split.g = x.g;
        }
        const uint32_t k = i % SEGS;
        if (i >= SEGS) mbar_wait_bounded(&ring.empty[k], (i / SEGS - 1) & 1u, SEG_WAIT_NS);
        __syncwarp();
        if (lane == 0) {
            ring.seg[k] = x;
            mbar_arrive(&ring.full[k]);
        }
        if (x.n == 0) break;
    }
    if (lane == 0 && tell) reinterpret_cast<Split *>(p.ws)[me] = split;
    __syncwarp();
}

// Segment number *i of the ring, false at the end.  The wait ignores the abort
// flag: after a time-out every role still walks through all segments, keeps to
// its named barriers and does nothing else.
__device__ __forceinline__ bool next_segment(SegRing &ring, uint32_t *i, Seg *w, int lane)
{
    const uint32_t k = *i % SEGS;
    bool got = mbar_wait_bounded(&ring.full[k], (*i / SEGS) & 1u, SEG_WAIT_NS);
    got = __all_sync(0xffffffffu, got);
    *w = ring.seg[k];
    __syncwarp();
    if (lane == 0) mbar_arrive(&ring.empty[k]);
    ++*i;
    return got && w->n > 0;
}

// ------------------------------------------------------------------- pieces --

__device__ __forceinline__ uint32_t sw128(uint32_t row, uint32_t c)
{
    return (row >> 3) * 1024u + (row & 7u) * 128u + ((c ^ (row & 7u)) << 4);
}

// Weights are kept as 2^P_UP exp(s - m), with m the maximum in use.  That one is
// at most RESCALE powers of two below the row's own, so a weight is at most 2^15,
// inside FP16; and one that FP16 rounds in its subnormal range is off by at most
// 2^-32 of the largest weight, so that the many small weights of a long context
// (2^20 tokens: 2^-12 of the largest) are not lost.  (Without the factor, 2^-25:
// 2^18 equal weights below that vanished from the output, though not from the sum.)
constexpr float RESCALE = 8.0f, P_UP = 7.0f;

// A weight's exponent is (s - m) * scale * log2 e.  The scores stay in the units
// that the products give, where differences near the maximum are exact: turned into
// powers of two first, each is rounded to 2^-24 of its size, at 2^23 half a power
// of two.
constexpr float LOG2_E = 1.4426950408889634f;

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two outputs as FP16, `a` in the lower half.  An output is a mean of finite values,
// but its weights are rounded and their sum is not, which can carry a mean of values
// near 65,504 past the border to infinity: it stops at 65,504.
__device__ __forceinline__ uint32_t to_half2(float a, float b)
{
    uint32_t h;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(b), "f"(a));
    return h;
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

// --------------------------------------------------------------------- join --

// Joins the parts of each split unit: block x the unit that worker x began (part
// 0 in its second place, part i in the first place of the i-th worker after it).
// A warp takes a row; with many parts and few rows (no more than blocks along y)
// the warps of a CTA share the parts of a row instead and add up through shared
// memory, for the loads of one warp would come one after another.  G: the
// geometry of the kernel that left the parts.
constexpr int JOIN_WARPS = 8;
constexpr int JOIN_PARTS = 6;                // parts that one warp takes

template <typename G, int D>
__global__ void __launch_bounds__(32 * JOIN_WARPS)
chunk_join_kernel(const ChunkParams p)
{
    constexpr int N = D / 32;
    __shared__ float part_sum[JOIN_WARPS][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    wait_prior_grid();
    const Split sp = reinterpret_cast<const Split *>(p.ws)[blockIdx.x];
    const int32_t n = sp.parts;
    if (n == 0) return;
    const float cs = G::RAW_MAX ? p.scale * LOG2_E : 1.0f;
    const float2 *ml = reinterpret_cast<const float2 *>(p.ws + WS_ML);
    const float *po = reinterpret_cast<const float *>(p.ws + ws_o<G::ROWS, G::WORKERS>());
    auto place = [&](int32_t i) { return 2 * (static_cast<int64_t>(blockIdx.x) + i) + (i == 0 ? 1 : 0); };
    const bool shared_row = n > JOIN_PARTS && sp.rows <= static_cast<int32_t>(gridDim.y);
    const int32_t step = shared_row ? gridDim.y : JOIN_WARPS * gridDim.y;
    for (int32_t row = shared_row ? blockIdx.y : blockIdx.y * JOIN_WARPS + warp; row < sp.rows; row += step) {
        float mx = -INFINITY, sum = 0.0f;
        for (int32_t i = lane; i < n; i += 32) mx = fmaxf(mx, ml[place(i) * G::ROWS + row].x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        float4 acc[N / 4];
#pragma unroll
        for (int e = 0; e < N / 4; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int32_t i0 = 0; i0 < n; i0 += 32) {
            float wt = 0.0f;
            if (i0 + lane < n) {
                const float2 x = ml[place(i0 + lane) * G::ROWS + row];
                wt = x.x == -INFINITY ? 0.0f : exp2_approx((x.x - mx) * cs);   // a part in which the row saw nothing
                sum = fmaf(x.y, wt, sum);
            }
            const int32_t k = min(32, n - i0);
#pragma unroll 8
            for (int32_t i = shared_row ? warp : 0; i < k; i += shared_row ? JOIN_WARPS : 1) {
                const float f = __shfl_sync(0xffffffffu, wt, i);
                const float4 *src = reinterpret_cast<const float4 *>(po + (place(i0 + i) * p.ws_rows + row) * D) + lane;
#pragma unroll
                for (int e = 0; e < N / 4; ++e) {
                    const float4 x = src[32 * e];
                    acc[e].x = fmaf(x.x, f, acc[e].x);
                    acc[e].y = fmaf(x.y, f, acc[e].y);
                    acc[e].z = fmaf(x.z, f, acc[e].z);
                    acc[e].w = fmaf(x.w, f, acc[e].w);
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (shared_row) {                    // uniform: n and the rows are the block's
#pragma unroll
            for (int e = 0; e < N / 4; ++e) reinterpret_cast<float4 *>(part_sum[warp])[32 * e + lane] = acc[e];
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int e = 0; e < N / 4; ++e)
#pragma unroll
                    for (int k = 1; k < JOIN_WARPS; ++k) {
                        const float4 x = reinterpret_cast<const float4 *>(part_sum[k])[32 * e + lane];
                        acc[e].x += x.x;
                        acc[e].y += x.y;
                        acc[e].z += x.z;
                        acc[e].w += x.w;
                    }
            }
            __syncthreads();
            if (warp != 0) continue;
        }
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        const int32_t v = sp.v0 + row, tok = by_group(p, v), h = v - tok * p.group;
        __half *out = static_cast<__half *>(p.out) +
                      ((static_cast<int64_t>(sp.s0) + tok) * p.hq + sp.g * p.group + h) * D;
#pragma unroll
        for (int e = 0; e < N / 4; ++e) {
            reinterpret_cast<uint2 *>(out)[32 * e + lane] =
                make_uint2(to_half2(acc[e].x * inv, acc[e].y * inv), to_half2(acc[e].z * inv, acc[e].w * inv));
        }
    }
}

}  // namespace
}  // namespace qsa
