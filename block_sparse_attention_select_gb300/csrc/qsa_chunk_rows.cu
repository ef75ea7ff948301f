// Dense attention over the paged K/V cache for few rows: decode tokens.
//
// The mathematics is that of qsa_chunk.cu; here a unit is 16 (token, query
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
// from the FP16 cache (6.5 to 6.7 TB/s) and 171 us from the E4M3 cache (6.2 TB/s; its scales
// are single bytes 2 x hkv apart).  One token over 4,096 takes 14 us: the launch,
// the search for its work, one memory latency each for table, keys and join.
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
    static constexpr bool RAW_MAX = true;    // the parts' maxima: scores before the scale
    static constexpr int ROWS = CR_ROWS, TILE = CR_TILE, UNIT_COST = 4, MIN_SHARE = 3, THREADS = CR_THREADS, WARPS = CR_WARPS,
                         WORKERS = CHUNK_MAX_CTAS;
};
using G = RowsGeometry;

template <int D, bool Q8>
struct RowShape {
    static constexpr int ES = Q8 ? 1 : 2;
    static constexpr uint32_t HALF = CR_TILE * D * ES, STAGE = 2 * HALF;   // K, then V
    static constexpr uint32_t SUM = CR_ROWS * D * 4;                       // an eighth of the eight warps' outputs
    // an even number of stages: a stage then belongs to one group of warps, which
    // waits for each of its phases (a parity wait must not skip one)
    static constexpr uint32_t QF = CR_ROWS * D * 2;                        // queries as A operands
    static constexpr int FIT = (227 * 1024 - 8192 - SUM - QF) / STAGE, NS = (FIT < CR_MAX_STAGES ? FIT : CR_MAX_STAGES) & ~1;
    static constexpr int CHUNKS = D * ES / 128;                            // 128-byte chunks of a vector
    static constexpr int PD = 16 / ES;                                     // dims of a 16-byte piece
};

struct RowCtrl {
    SegRing segs;
    uint64_t full[CR_MAX_STAGES], empty[CR_MAX_STAGES];
    Share share;
    float scale[CR_MAX_STAGES][2][CR_TILE];  // K and V scales of a stage's tokens (E4M3)
    float m[CR_COMP][CR_ROWS], l[CR_COMP][CR_ROWS];
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

template <int D, bool Q8>
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
    wait_prior_grid();
    // (the sums' place is free until a segment's end)
    static_assert(sizeof(FindScratch<G>) <= Sh::SUM, "scratch");
    find_work<G>(p, c.share, *reinterpret_cast<FindScratch<G> *>(sum), blockIdx.x, gridDim.x, warp, lane);
    uint32_t segs = 0;
    Seg w;

    // registers after the split: 8 x 32 x 216 + 4 x 32 x 72 = 384 x 168
    if (warp >= CR_COMP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == CR_SCHED) {
            schedule<G>(p, c.share, c.segs, blockIdx.x, true, lane);
        } else if (warp == CR_LOAD) {
            // ------------------------------------------------------ K, V loads
            const int32_t P = p.kv.page_tokens;
            const int sh = __ffs(min(P, CR_TILE)) - 1;             // log2 of a box's tokens
            const int32_t down = CR_TILE >> sh, boxes = 2 * Sh::CHUNKS * down;
            uint32_t slot = 0, phase = 0, used = 0, last = 0;
            bool ok = true;
            while (next_segment(c.segs, &segs, &w, lane)) {
                if (!ok) continue;
                const int32_t *bt = p.kv.block_table + static_cast<int64_t>(w.b) * p.kv.max_pages;
                // a lane looks up the cache rows of tokens lane and lane + 32, two
                // stages ahead
                const int32_t nowhere = p.kv.num_pages << p.kv.page_shift;       // past the cache: reads zeros
                auto row_of = [&](int32_t j, int k) -> int32_t {
                    const int32_t tok = (w.j0 + j) * CR_TILE + lane + 32 * k;
                    // a box is loaded when any of its tokens is attended
                    if (j >= w.n || (tok & ~((1 << sh) - 1)) > w.hi_tok || (tok | ((1 << sh) - 1)) < w.lo_tok) return nowhere;
                    const int32_t page = __ldg(bt + (tok >> p.kv.page_shift));
                    if (page >= 0 && page < p.kv.num_pages) return (page << p.kv.page_shift) + (tok & (P - 1));
                    record_error(p.kv.status, ST_BAD_PAGE);
                    return nowhere;
                };
                int32_t row[2], row1[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    row[k] = row_of(0, k);
                    row1[k] = row_of(1, k);
                }
                for (int32_t j = 0; j < w.n; ++j) {
                    if (!warp_wait(&c.empty[slot], phase ^ 1u, abort, lim)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(&c.full[slot], STAGE);
                    __syncwarp();
                    uint8_t *dst = smem + slot * STAGE;
                    for (int32_t i0 = 0; i0 < boxes; i0 += 32) {
                        const int32_t i = i0 + lane;
                        const int32_t d = i & (down - 1), ch = (i / down) % Sh::CHUNKS;
                        const bool v = i >= boxes / 2;
                        const int32_t first = d << sh;             // the box's first token, held by lane first % 32
                        const int32_t ya = __shfl_sync(0xffffffffu, row[0], first & 31);
                        const int32_t yb = __shfl_sync(0xffffffffu, row[1], first & 31);
                        if (i < boxes)
                            tma_load_3d(dst + (v ? HALF : 0u) + ch * (CR_TILE * 128) + first * 128, v ? &tv : &tk, &c.full[slot],
                                        0, first < 32 ? ya : yb, w.g * Sh::CHUNKS + ch);
                    }
                    used |= 1u << slot;
                    last = (last & ~(1u << slot)) | (phase << slot);
                    if (++slot == NS) {
                        slot = 0;
                        phase ^= 1u;
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        row[k] = row1[k];
                        row1[k] = row_of(j + 2, k);
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
            while (next_segment(c.segs, &segs, &w, lane)) {
                if (!ok) continue;
                const int32_t *bt = p.kv.block_table + static_cast<int64_t>(w.b) * p.kv.max_pages;
                auto page_of = [&](int32_t j, int k) -> int32_t {
                    const int32_t tok = (w.j0 + j) * CR_TILE + lane + 32 * k;
                    return j < w.n && tok >= w.lo_tok && tok <= w.hi_tok ? __ldg(bt + (tok >> p.kv.page_shift)) : -1;
                };
                auto byte_of = [&](int32_t j, int k, int32_t page) -> uint32_t {
                    if (page < 0 || page >= p.kv.num_pages) return 127u;
                    const int32_t tok = (w.j0 + j) * CR_TILE + lane + 32 * k;
                    return __ldg(scale + ((static_cast<int64_t>(page) << p.kv.page_shift) + (tok & (p.kv.page_tokens - 1))) * p.kv.hkv + w.g);
                };
                int32_t page[4][2];
                uint32_t byte[4][2];
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int k = 0; k < 2; ++k) page[u][k] = page_of(u, k);
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        byte[u][k] = byte_of(u, k, page[u][k]);
                        page[u][k] = page_of(u + 4, k);
                    }
                for (int32_t j = 0; ok && j < w.n; j += 4) {
                    uint32_t next[4][2];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            next[u][k] = byte_of(j + 4 + u, k, page[u][k]);
                            page[u][k] = page_of(j + 8 + u, k);
                        }
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
        while (next_segment(c.segs, &segs, &w, lane)) {
            int32_t pos[2], first[2];
            const uint8_t *qrow[2];                                // rows r and r + 8 of the unit
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = r + 8 * e;
                const int32_t v = w.v0 + min(row, w.rows - 1), tok = by_group(p, v), h = v - tok * p.group;
                pos[e] = w.p0 + tok;
                first[e] = p.window > 0 ? max(0, pos[e] - p.window + 1) : 0;
                qrow[e] = row >= w.rows ? nullptr : static_cast<const uint8_t *>(p.q) +
                          ((static_cast<int64_t>(w.s0) + tok) * p.q_stride + (w.g * p.group + h) * D) * 2;
            }
            // The queries as A operands, in shared memory (in registers they
            // spilled: 294 us on the 64-request E4M3 step).  Product k of
            // piece i takes dims 8 PD (i / 2) + PD (2 q + i % 2) + 4 k .. + 3.
            for (int k = warp; k < KS; k += CR_COMP) {
                const int i = k / (PD / 4), j = k % (PD / 4);
                const int dim = 8 * PD * (i >> 1) + PD * (2 * q + (i & 1)) + 4 * j;
                uint2 x[2];
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    x[e] = qrow[e] ? __ldg(reinterpret_cast<const uint2 *>(qrow[e] + dim * 2)) : make_uint2(0u, 0u);
                qf[k * 32 + lane] = make_uint4(x[0].x, x[1].x, x[0].y, x[1].y);
            }
            named_barrier(BAR_COMP, 32 * CR_COMP);
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
                ok = warp_wait(&c.full[sl], ph, abort, lim);
                const int32_t tok0 = (w.j0 + j) * CR_TILE + sub;
                if (ok && tok0 <= w.hi_tok && tok0 + 15 >= w.lo_tok) {
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
                    const bool edge = tok0 < w.lo_tok || tok0 + 15 > w.hi_tok;      // some token that no row attends
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
                            if (tok > pos[e >> 1] || tok < first[e >> 1]) s[n][e] = -INFINITY;
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
                            if (edge && (tok0 - sub + tr < w.lo_tok || tok0 - sub + tr > w.hi_tok)) x[e] = make_uint4(0u, 0u, 0u, 0u);
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
            // Eight steps; in each every warp lays down PD / 8 dims of each chunk, and
            // thread t adds up the eight warps' values of place t: chunk i, row
            // r' + 8 (e / 2), dims 8 PD i + PD (2 q' + e % 2) .., where t = (i, lane', e).
            constexpr int DS = PD / 8, OWN = (VI * 128 + 255) / 256;    // dims per step, places per thread
            float x[OWN][PD];
#pragma unroll
            for (int st = 0; st < 8; ++st) {
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
            named_barrier(BAR_COMP, 32 * CR_COMP);                 // read before the next segment's sums
        }
    }
    __syncthreads();
    if (t == 0 && c.abort) record_error(p.kv.status, ST_TIMEOUT);
    allow_next_grid();
}

template <int D, bool Q8>
int launch(const ChunkParams &p, const void *tk, const void *tv, int grid, bool overlap, cudaStream_t stream)
{
    using Sh = RowShape<D, Q8>;
    constexpr size_t SMEM = Sh::NS * Sh::STAGE + Sh::SUM + Sh::QF + sizeof(RowCtrl);
    static_assert(SMEM <= 232448, "shared memory budget");
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return static_cast<int>(cudaErrorInvalidDevice);
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!done[dev]) {
            const cudaError_t e = cudaFuncSetAttribute(chunk_rows_kernel<D, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       static_cast<int>(SMEM));
            if (e != cudaSuccess) return static_cast<int>(e);
            done[dev] = true;
        }
    }
    void *args[] = {const_cast<void *>(tk), const_cast<void *>(tv), const_cast<ChunkParams *>(&p)};
    const int rc = launch_kernel(reinterpret_cast<const void *>(&chunk_rows_kernel<D, Q8>), dim3(grid), dim3(CR_THREADS), SMEM,
                                 stream, false, args);
    if (rc != 0) return rc;
    void *join[] = {const_cast<ChunkParams *>(&p)};
    const unsigned y = static_cast<unsigned>(p.ws_rows);
    return launch_kernel(reinterpret_cast<const void *>(&chunk_join_kernel<G, D>), dim3(grid, y), dim3(256), 0, stream,
                         overlap, join);
}

}  // namespace

int32_t chunk_rows_part_rows(int32_t rows, int32_t group)
{
    return static_cast<int32_t>(std::min<int64_t>(CR_ROWS, static_cast<int64_t>(rows) * group));
}

size_t chunk_rows_workspace_bytes(int32_t rows, int32_t group, int32_t head_dim)
{
    return ws_o<CR_ROWS, CHUNK_MAX_CTAS>() + size_t{2} * CHUNK_MAX_CTAS * chunk_rows_part_rows(rows, group) * head_dim * 4;
}

int32_t chunk_rows_box(int32_t page_tokens) { return std::min(page_tokens, CR_TILE); }

int launch_chunk_rows(const ChunkParams &p, const void *tk, const void *tv, int sms, bool overlap, void *stream)
{
    const int grid = std::min(sms, static_cast<int>(CHUNK_MAX_CTAS));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.kv.head_dim == 128)
        return p.kv.e4m3 ? launch<128, true>(p, tk, tv, grid, overlap, s) : launch<128, false>(p, tk, tv, grid, overlap, s);
    return p.kv.e4m3 ? launch<256, true>(p, tk, tv, grid, overlap, s) : launch<256, false>(p, tk, tv, grid, overlap, s);
}

}  // namespace qsa
