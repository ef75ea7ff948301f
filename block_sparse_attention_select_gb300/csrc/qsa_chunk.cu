// Dense attention of new tokens over the paged K/V cache.
//
// One warp per (row, query head): the lanes share the head dimension, walk the
// row's visible tokens and keep the running maximum, the sum and the weighted
// values in FP32 (o <- o * exp(m - m') + exp(s - m') * v).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qsa_device.cuh"
#include "qsa_internal.h"
#include "qsa_seq.cuh"

namespace qsa {
namespace {

constexpr int CH_WARPS = 8;

// N consecutive cache values from `src` (FP16 or E4M3 with scale s) as FP32.
template <int N, bool E4M3>
__device__ __forceinline__ void cache_values(const uint8_t *src, float s, float (&x)[N])
{
    if constexpr (E4M3) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint32_t u = __ldg(reinterpret_cast<const uint32_t *>(src + i));
            uint32_t h[2];
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[0]) : "h"(static_cast<uint16_t>(u & 0xffffu)));
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h[1]) : "h"(static_cast<uint16_t>(u >> 16)));
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[c]));
                x[i + 2 * c] = f.x * s;
                x[i + 2 * c + 1] = f.y * s;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(src + 2 * i));
            const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&u.x));
            const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&u.y));
            x[i] = a.x;
            x[i + 1] = a.y;
            x[i + 2] = b.x;
            x[i + 3] = b.y;
        }
    }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(CH_WARPS * 32)
chunk_rows_kernel(const ChunkParams p)
{
    constexpr int N = D / 32, ES = E4M3 ? 1 : 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    wait_prior_grid();
    if (blockIdx.x == 0) flag_bad_requests(p.kv);
    const int64_t task = static_cast<int64_t>(blockIdx.x) * CH_WARPS + warp;
    const int32_t row = static_cast<int32_t>(task / p.hq), h = static_cast<int32_t>(task % p.hq);
    if (row >= p.kv.rows) return;
    const int32_t b = find_request(p.kv, row, lane);
    if (b < 0) return;
    bool bad;
    const Seq s = seq_of(p.kv, b, &bad);
    if (row < s.s0 || row - s.s0 >= s.n) return;
    const int32_t pos = s.p0 + (row - s.s0);
    const int32_t first = p.window > 0 ? max(0, pos - p.window + 1) : 0;
    const int32_t g = h / p.group;
    const int32_t *bt = p.kv.block_table + static_cast<int64_t>(b) * p.kv.max_pages;

    float q[N], o[N];
    cache_values<N, false>(static_cast<const uint8_t *>(p.q) + (row * p.q_stride + h * D + lane * N) * 2, 1.0f, q);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        q[i] *= p.scale;
        o[i] = 0.0f;
    }
    float m = -INFINITY, sum = 0.0f;
    for (int32_t t = first; t <= pos; ++t) {
        const int32_t page = __ldg(bt + (t >> p.kv.page_shift));
        float k[N], v[N];
        if (page >= 0 && page < p.kv.num_pages) {
            const int64_t vec = (static_cast<int64_t>(page << p.kv.page_shift) + (t & (p.kv.page_tokens - 1))) * p.kv.hkv + g;
            float ks = 1.0f, vs = 1.0f;
            if (E4M3) {
                ks = __uint_as_float(static_cast<uint32_t>(p.kv.k_scale[vec]) << 23);
                vs = __uint_as_float(static_cast<uint32_t>(p.kv.v_scale[vec]) << 23);
            }
            cache_values<N, E4M3>(p.kv.k + (vec * D + lane * N) * ES, ks, k);
            cache_values<N, E4M3>(p.kv.v + (vec * D + lane * N) * ES, vs, v);
        } else {
            if (lane == 0) record_error(p.kv.status, ST_BAD_PAGE);
#pragma unroll
            for (int i = 0; i < N; ++i) k[i] = v[i] = 0.0f;
        }
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) dot = fmaf(q[i], k[i], dot);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
        const float m2 = fmaxf(m, dot);
        const float a = __expf(m - m2), e = __expf(dot - m2);
        m = m2;
        sum = fmaf(sum, a, e);
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = fmaf(o[i], a, e * v[i]);
    }
    const float inv = 1.0f / sum;
    __half *out = static_cast<__half *>(p.out) + (static_cast<int64_t>(row) * p.hq + h) * D + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = __float2half_rn(o[i] * inv);
}

}  // namespace

int launch_chunk(const ChunkParams &p, int sms, bool overlap, void *stream)
{
    (void)sms;
    (void)overlap;
    const int64_t tasks = static_cast<int64_t>(p.kv.rows) * p.hq;
    const dim3 grid(static_cast<unsigned>((tasks + CH_WARPS - 1) / CH_WARPS));
    void *args[] = {const_cast<ChunkParams *>(&p)};
    const void *f;
    if (p.kv.head_dim == 128)
        f = p.kv.e4m3 ? reinterpret_cast<const void *>(&chunk_rows_kernel<128, true>)
                      : reinterpret_cast<const void *>(&chunk_rows_kernel<128, false>);
    else
        f = p.kv.e4m3 ? reinterpret_cast<const void *>(&chunk_rows_kernel<256, true>)
                      : reinterpret_cast<const void *>(&chunk_rows_kernel<256, false>);
    return launch_kernel(f, grid, dim3(CH_WARPS * 32), 0, static_cast<cudaStream_t>(stream), false, args);
}

}  // namespace qsa
