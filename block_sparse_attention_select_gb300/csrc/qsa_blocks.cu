// Attention of new tokens over the blocks of 128 tokens selected for them.
//
// The simplest form: a warp per row and query head goes through the row's blocks
// token by token, its lanes sharing the dims, with a running maximum and sum.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qsa_device.cuh"
#include "qsa_internal.h"
#include "qsa_seq.cuh"

namespace qsa {
namespace {

constexpr int BL_THREADS = 128;

template <int D, bool Q8>
__device__ __forceinline__ void load_dims(const uint8_t *cache, const uint8_t *scale, int64_t vec, int lane, float (&x)[D / 32])
{
    if (Q8) {
        const int e = max(112, min(135, static_cast<int>(__ldg(scale + vec))));
        const float f = __uint_as_float(static_cast<uint32_t>(e) << 23);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            const uint16_t two = __ldg(reinterpret_cast<const uint16_t *>(cache + vec * D) + i * 32 + lane);
            uint32_t h;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            x[2 * i] = v.x * f;
            x[2 * i + 1] = v.y * f;
        }
    } else {
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            const float2 v = __half22float2(reinterpret_cast<const __half2 *>(cache + vec * D * 2)[i * 32 + lane]);
            x[2 * i] = v.x;
            x[2 * i + 1] = v.y;
        }
    }
}

template <int D, bool Q8>
__global__ void __launch_bounds__(BL_THREADS)
blocks_kernel(const BlocksParams p)
{
    __shared__ int32_t req_s;
    __shared__ Seq seq_s;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const KvParams &kv = p.c.kv;
    const int32_t row = blockIdx.x;
    wait_prior_grid();
    if (row == 0) flag_bad_requests(kv);
    Seq s;
    const int32_t b = requests_of_rows(kv, row, 1, &s);
    if (threadIdx.x == 0) {
        req_s = b;
        seq_s = s;
    }
    __syncthreads();
    if (req_s < 0) return;
    const int32_t pos = seq_s.p0 + row - seq_s.s0, last = pos / BLOCK_TOKENS;
    const int32_t *bt = kv.block_table + static_cast<int64_t>(req_s) * kv.max_pages;
    for (int32_t h = warp; h < p.c.hq; h += BL_THREADS / 32) {
        const int32_t g = h / p.c.group;
        const int32_t *sel = p.sel + (static_cast<int64_t>(row) * kv.hkv + g) * p.k;
        const __half2 *q = reinterpret_cast<const __half2 *>(static_cast<const __half *>(p.c.q) + row * p.c.q_stride + static_cast<int64_t>(h) * D);
        float qv[D / 32], o[D / 32] = {};
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            const float2 v = __half22float2(q[i * 32 + lane]);
            qv[2 * i] = v.x;
            qv[2 * i + 1] = v.y;
        }
        float m = -INFINITY, l = 0.0f;
        for (int32_t i = -p.recent; i < p.k; ++i) {
            int32_t c = i < 0 ? last + 1 + i : __ldg(sel + i);
            if (i >= 0) {
                if (c < -1 || c > last) {
                    if (lane == 0) record_error(kv.status, ST_BAD_ROW);
                    continue;
                }
                bool twice = c > last - p.recent;              // one of the last blocks, or named before
                for (int32_t j = lane; j < i; j += 32) twice = twice || __ldg(sel + j) == c;
                if (__any_sync(0xffffffffu, twice)) continue;
            }
            if (c < 0) continue;
            const int32_t end = min(pos + 1, (c + 1) * BLOCK_TOKENS);
            for (int32_t t = c * BLOCK_TOKENS; t < end; ++t) {
                const int32_t page = __ldg(bt + (t >> kv.page_shift));
                const bool in = page >= 0 && page < kv.num_pages;
                if (!in && lane == 0) record_error(kv.status, ST_BAD_PAGE);
                const int64_t vec = ((static_cast<int64_t>(page) << kv.page_shift) + (t & (kv.page_tokens - 1))) * kv.hkv + g;
                float x[D / 32] = {}, v[D / 32] = {};
                if (in) {
                    load_dims<D, Q8>(kv.k, kv.k_scale, vec, lane, x);
                    load_dims<D, Q8>(kv.v, kv.v_scale, vec, lane, v);
                }
                float sc = 0.0f;
#pragma unroll
                for (int e = 0; e < D / 32; ++e) sc = fmaf(qv[e], x[e], sc);
#pragma unroll
                for (int w = 16; w > 0; w >>= 1) sc += __shfl_xor_sync(0xffffffffu, sc, w);
                const float mn = fmaxf(m, sc), keep = exp2f((m - mn) * p.c.scale * 1.4426950408889634f);
                const float wt = exp2f((sc - mn) * p.c.scale * 1.4426950408889634f);
                l = l * keep + wt;
#pragma unroll
                for (int e = 0; e < D / 32; ++e) o[e] = o[e] * keep + wt * v[e];
                m = mn;
            }
        }
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        __half2 *out = reinterpret_cast<__half2 *>(static_cast<__half *>(p.c.out) + (static_cast<int64_t>(row) * p.c.hq + h) * D);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            uint32_t y;
            asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(o[2 * i + 1] * inv), "f"(o[2 * i] * inv));
            reinterpret_cast<uint32_t *>(out)[i * 32 + lane] = y;
        }
    }
}

template <int D, bool Q8>
int launch(const BlocksParams &p, cudaStream_t stream)
{
    void *args[] = {const_cast<BlocksParams *>(&p)};
    return launch_kernel(reinterpret_cast<const void *>(&blocks_kernel<D, Q8>), dim3(p.c.kv.rows), dim3(BL_THREADS), 0, stream,
                         false, args);
}

}  // namespace

int launch_blocks(const BlocksParams &p, int sms, bool overlap, void *stream)
{
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.c.kv.head_dim == 128) return p.c.kv.e4m3 ? launch<128, true>(p, s) : launch<128, false>(p, s);
    return p.c.kv.e4m3 ? launch<256, true>(p, s) : launch<256, false>(p, s);
}

}  // namespace qsa
