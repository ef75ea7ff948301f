// K/V cache: new tokens written into their pages, as FP16 or quantised to E4M3
// with a power-of-two scale per token and head, and read back as FP16.
//
// With e the least integer of [-15, 8] that has max |x| <= 448 * 2^e, a vector
// x of head_dim values is stored as rne_e4m3(x * 2^-e) and the byte e + 127.
// Scaling by a power of two is exact in FP32, so each value is rounded once.
// The bounds of e make every stored value an FP16 number: the finest E4M3 step,
// 2^-9, times 2^-15 is FP16's finest, and at e = 8 codes stop at 240 (240 * 256
// < 65504 < 256 * 256).  A power of two costs no accuracy against a scale of
// amax / 448: E4M3 is a floating type, only its range below the maximum moves,
// by less than one binade of fourteen.
//
// Both are bound by memory: each vector is read once and written once.  A
// vector belongs to head_dim / 8 lanes, 16 bytes of FP16 in each; the lanes
// reduce the maximum by shuffles.  A warp takes up to 16 consecutive rows: its
// lanes look up one row's cache line each (request, page), then the warp walks
// through the rows' vectors, KV_BATCH of them in flight.  (With the lookups by a
// CTA for 8 rows at a time, each CTA waited for three memory latencies to move
// 12 KB: 122 us to read a 184,320-token E4M3 context back, 4.65 TB/s.)  Now that
// takes 102 us (5.6 TB/s: twice as much is written as read), writing four prompts
// of up to 4,096 tokens as FP16 22 us in a stream of calls (4.8 TB/s; 17 us where
// equal calls follow each other in a graph: most of what is written is then still in
// the L2 cache, to be overwritten there), a batch of single tokens 3 to 5 us.
//
// Starts that fall somewhere are a caller's mistake that costs only the requests
// it makes impossible: a CTA that finds a row without a request looks whether the
// starts are in order, and goes through the requests one by one where they are not.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "qsa_device.cuh"
#include "qsa_internal.h"
#include "qsa_seq.cuh"

namespace qsa {
namespace {

constexpr int KV_THREADS = 256;
constexpr int KV_BATCH = 8;        // vectors in flight per thread
constexpr int KV_MAX_ROWS = 16;    // rows per warp

// Cache line (page * page_tokens + slot) of a row of request b: -2 a page outside
// the cache.
__device__ __forceinline__ int32_t line_of(const KvParams &p, int32_t b, const Seq &s, int32_t row)
{
    const int32_t pos = s.p0 + (row - s.s0);
    const int32_t page = __ldg(p.block_table + static_cast<int64_t>(b) * p.max_pages + (pos >> p.page_shift));
    if (page >= 0 && page < p.num_pages) return (page << p.page_shift) + (pos & (p.page_tokens - 1));
    record_error(p.status, ST_BAD_PAGE);
    return -2;
}

// Cache line of `row`, a row per lane: -1 no request or skipped.
__device__ __forceinline__ int32_t find_line(const KvParams &p, int32_t row)
{
    // the last request that starts at or before the row
    int32_t lo = 0, hi = p.n_reqs;
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (__ldg(p.seq_start + mid) <= row) lo = mid;
        else hi = mid;
    }
    bool bad;
    const Seq s = seq_of(p, lo, &bad);
    return has_row(s, row) ? line_of(p, lo, s, row) : -1;
}

// The same where the starts fall somewhere, by all lanes of a warp, request by
// request: slow, but no well-formed request loses its rows to another's mistake.
__device__ __forceinline__ int32_t find_line_unsorted(const KvParams &p, int32_t row, bool wanted)
{
    int32_t line = -1;
#pragma unroll 1
    for (int32_t b = 0; b < p.n_reqs; ++b) {
        bool bad;
        const Seq s = seq_of(p, b, &bad);
        if (wanted && line == -1 && has_row(s, row)) line = line_of(p, b, s, row);
    }
    return line;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d)
{
    uint16_t lo, hi;
    // the first source operand is the upper byte
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t two)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
    return h;
}

// The scale exponent of a vector with largest magnitude a.
__device__ __forceinline__ int scale_exponent(float a)
{
    const uint32_t u = __float_as_uint(a);
    const int x = static_cast<int>(u >> 23) - 127;              // a = m * 2^x, 1 <= m < 2
    const int e = (u & 0x7fffffu) <= 0x600000u ? x - 8 : x - 7;  // 448 = 1.75 * 2^8
    return max(-15, min(8, e));
}

// LOAD false: rows k, v -> cache; true: cache -> rows.
template <int D, bool E4M3, bool LOAD>
__global__ void __launch_bounds__(KV_THREADS, 3)
kv_kernel(const KvParams p, uint8_t *kr, uint8_t *vr, int64_t k_stride, int64_t v_stride, int32_t rows_per_warp)
{
    constexpr int LPV = D / 8;                     // lanes per vector
    constexpr int VPP = 32 / LPV;                   // vectors per pass of the warp
    constexpr int ES = E4M3 ? 1 : 2;                // bytes of a cache element
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    wait_prior_grid();
    if (blockIdx.x == 0) flag_bad_requests(p);
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * (KV_THREADS / 32) + warp) * rows_per_warp;
    const int32_t row0 = static_cast<int32_t>(min(first, static_cast<int64_t>(p.rows)));
    const int32_t n_rows = min(rows_per_warp, p.rows - row0);
    int32_t mine = lane < n_rows ? find_line(p, row0 + lane) : -1;
    // No request: a row behind the last one, or of a request that is skipped; but
    // where the starts are out of order the search may have passed the row's by.
    bool lost = lane < n_rows && mine == -1;
    if (__syncthreads_or(lost)) {
        bool falls = false;
#pragma unroll 4
        for (int32_t b = threadIdx.x; b < p.n_reqs; b += KV_THREADS)
            falls = falls || __ldg(p.seq_start + b + 1) < __ldg(p.seq_start + b);
        if (__syncthreads_or(falls) && __any_sync(0xffffffffu, lost)) {
            const int32_t line = find_line_unsorted(p, row0 + lane, lost);
            if (lost) mine = line;
        }
    }
    if (n_rows <= 0) return;

    const int sub = lane / LPV, l = lane % LPV;
    const int32_t per_row = 2 * p.hkv;              // vectors of a row: K heads, then V heads
    const int32_t n = n_rows * per_row;
    // the lane's next vector as row and head, advanced without divisions
    int32_t r = sub / per_row, hv = sub - r * per_row;
    for (int32_t base = 0; base < n; base += VPP * KV_BATCH) {
        uint4 x[KV_BATCH];
        int64_t vec[KV_BATCH];                      // (line, head) vector of the cache, negative: none
        uint8_t *row[KV_BATCH];                     // this lane's 16 bytes of the row array
        uint8_t sc[KV_BATCH];
        bool is_v[KV_BATCH];
#pragma unroll
        for (int j = 0; j < KV_BATCH; ++j) {
            vec[j] = -1;
            x[j] = make_uint4(0u, 0u, 0u, 0u);
            sc[j] = 0;
            const int32_t ln = __shfl_sync(0xffffffffu, mine, r & 31);
            if (r < n_rows) {
                is_v[j] = hv >= p.hkv;
                const int32_t h = is_v[j] ? hv - p.hkv : hv;
                row[j] = (is_v[j] ? vr + (static_cast<int64_t>(row0) + r) * v_stride * 2
                                  : kr + (static_cast<int64_t>(row0) + r) * k_stride * 2) + (h * D + l * 8) * 2;
                vec[j] = ln < 0 ? ln : static_cast<int64_t>(ln) * p.hkv + h;
                if (!LOAD) {
                    if (ln >= 0) x[j] = __ldg(reinterpret_cast<const uint4 *>(row[j]));
                } else if (ln >= 0) {
                    const uint8_t *src = (is_v[j] ? p.v : p.k) + (vec[j] * D + l * 8) * ES;
                    if (E4M3) {
                        const uint2 u = *reinterpret_cast<const uint2 *>(src);
                        x[j].x = u.x;
                        x[j].y = u.y;
                        sc[j] = (is_v[j] ? p.v_scale : p.k_scale)[vec[j]];
                    } else {
                        x[j] = *reinterpret_cast<const uint4 *>(src);
                    }
                }
            }
            hv += VPP;
            while (hv >= per_row) {
                hv -= per_row;
                ++r;
            }
        }
#pragma unroll
        for (int j = 0; j < KV_BATCH; ++j) {
            if constexpr (LOAD) {
                if (vec[j] == -1) continue;
                uint4 o = x[j];
                if (E4M3 && vec[j] >= 0) {
                    // code * 2^(byte - 127), exact in FP16
                    const float s = __uint_as_float(static_cast<uint32_t>(max(112, min(135, int(sc[j])))) << 23);
                    const uint32_t in[4] = {x[j].x & 0xffffu, x[j].x >> 16, x[j].y & 0xffffu, x[j].y >> 16};
                    uint32_t w[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t h = e4m3x2_to_half2(in[c]);
                        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                        const __half2 y = __floats2half2_rn(f.x * s, f.y * s);
                        w[c] = *reinterpret_cast<const uint32_t *>(&y);
                    }
                    o = make_uint4(w[0], w[1], w[2], w[3]);
                }
                *reinterpret_cast<uint4 *>(row[j]) = o;      // zeros for a page outside the cache
            } else if constexpr (!E4M3) {
                if (vec[j] >= 0) *reinterpret_cast<uint4 *>((is_v[j] ? p.v : p.k) + (vec[j] * D + l * 8) * 2) = x[j];
            } else {
                float f[8];
                const uint32_t in[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float2 t = __half22float2(*reinterpret_cast<const __half2 *>(&in[c]));
                    f[2 * c] = t.x;
                    f[2 * c + 1] = t.y;
                }
                float a = 0.0f;
#pragma unroll
                for (int c = 0; c < 8; ++c) a = fmaxf(a, fabsf(f[c]));        // a NaN does not count
#pragma unroll
                for (int o = LPV / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
                const int e = a > 0.0f ? scale_exponent(a) : -15;
                const float s = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    f[c] *= s;
                    if (e == 8 && fabsf(f[c]) > 240.0f) f[c] = copysignf(240.0f, f[c]);
                }
                if (vec[j] >= 0) {
                    *reinterpret_cast<uint2 *>((is_v[j] ? p.v : p.k) + vec[j] * D + l * 8) =
                        make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
                    if (l == 0) (is_v[j] ? p.v_scale : p.k_scale)[vec[j]] = static_cast<uint8_t>(e + 127);
                }
            }
        }
    }
}

template <bool LOAD>
int launch(const KvParams &p, void *k, int64_t k_stride, void *v, int64_t v_stride, int sms, void *stream)
{
    // 16 rows per warp where that still gives every SM two CTAs, fewer below
    constexpr int WARPS = KV_THREADS / 32;
    const int rows_per_warp = std::max(1, std::min(KV_MAX_ROWS, p.rows / (2 * sms * WARPS)));
    const dim3 grid((p.rows + rows_per_warp * WARPS - 1) / (rows_per_warp * WARPS));
    KvParams pp = p;
    uint8_t *kr = static_cast<uint8_t *>(k), *vr = static_cast<uint8_t *>(v);
    int32_t rpw = rows_per_warp;
    void *args[] = {&pp, &kr, &vr, &k_stride, &v_stride, &rpw};
    const void *f;
    if (p.head_dim == 128)
        f = p.e4m3 ? reinterpret_cast<const void *>(&kv_kernel<128, true, LOAD>)
                   : reinterpret_cast<const void *>(&kv_kernel<128, false, LOAD>);
    else
        f = p.e4m3 ? reinterpret_cast<const void *>(&kv_kernel<256, true, LOAD>)
                   : reinterpret_cast<const void *>(&kv_kernel<256, false, LOAD>);
    return launch_kernel(f, grid, dim3(KV_THREADS), 0, static_cast<cudaStream_t>(stream), false, args);
}

}  // namespace

int launch_kv_store(const KvParams &p, const void *k, int64_t k_stride, const void *v, int64_t v_stride, int sms,
                    void *stream)
{
    return launch<false>(p, const_cast<void *>(k), k_stride, const_cast<void *>(v), v_stride, sms, stream);
}

int launch_kv_load(const KvParams &p, void *k, int64_t k_stride, void *v, int64_t v_stride, int sms, void *stream)
{
    return launch<true>(p, k, k_stride, v, v_stride, sms, stream);
}

}  // namespace qsa
