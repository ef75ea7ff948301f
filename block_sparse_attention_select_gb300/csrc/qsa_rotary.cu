// Rotary positions: the table of cosines and sines, and the rotation of queries
// and keys.
//
// Bound by memory: every value is read and written once.  A thread takes 16 dims
// of a head as two 16-byte vectors (both halves of eight pairs) and goes through
// some heads of its token with them, so that it reads its eight cosines and sines
// once for all of these; ROT_BATCH heads' loads are in flight together, the first of
// them while the rows' positions are looked up.  Four
// prompts of 4,096 tokens, 40 heads of 128: 54 us with halves paired, 53 us with
// neighbours (6.3 and 6.4 TB/s; neighbours as two 16-byte accesses 59 us; 4 or 20
// heads to a thread 57 to 60 us).  The 1,616-row chunk, 26 heads of 256 of which 64
// dims rotate: 9 us (a thread for every head or two: 11 us), 64 single tokens 4 us,
// a launch and two memory latencies.  (Times of ten equal calls in a graph, which find
// what fits in the L2 cache there; in a stream of calls on other inputs 55, 13 and 11 us.)
//
// The table is made once per model: an FP64 sine and cosine per pair and position, 17.8
// billion a second (184,320 positions of 64 dims 334 us, 2^20 of 128 3.8 ms), 50 times
// what writing it takes, bound by the few FP64 units.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "qsa_device.cuh"
#include "qsa_internal.h"
#include "qsa_seq.cuh"

namespace qsa {
namespace {

constexpr int ROT_THREADS = 256;
constexpr int ROT_ROWS = 32;                 // rows of a CTA at most
constexpr int ROT_BATCH = 4;                 // heads whose loads are in flight
constexpr int ROT_HEADS = 10;                // heads that a thread goes through (more where a row has too many for its threads)

// Eight pairs: a and b of each as FP16 halves of four words; neighbours: a0 b0 a1 b1 ...
template <bool NEIGHBOURS>
__device__ __forceinline__ void rotate8(uint4 &x, uint4 &y, const float (&cs)[8], const float (&sn)[8])
{
    uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    if (NEIGHBOURS) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            const __half2 h = __floats2half2_rn(v.x * cs[i] - v.y * sn[i], v.y * cs[i] + v.x * sn[i]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&w[4 + i]));
            const __half2 h = __floats2half2_rn(a.x * cs[2 * i] - b.x * sn[2 * i], a.y * cs[2 * i + 1] - b.y * sn[2 * i + 1]);
            const __half2 l = __floats2half2_rn(b.x * cs[2 * i] + a.x * sn[2 * i], b.y * cs[2 * i + 1] + a.y * sn[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
            w[4 + i] = *reinterpret_cast<const uint32_t *>(&l);
        }
    }
    x = make_uint4(w[0], w[1], w[2], w[3]);
    y = make_uint4(w[4], w[5], w[6], w[7]);
}

// Two 16-byte vectors, side by side and 32-byte aligned when WIDE.
template <bool WIDE>
__device__ __forceinline__ void load_two(const uint16_t *a, const uint16_t *b, uint4 &x, uint4 &y)
{
    if (WIDE) {
        asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w), "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w) : "l"(a) : "memory");
    } else {
        x = *reinterpret_cast<const uint4 *>(a);
        y = *reinterpret_cast<const uint4 *>(b);
    }
}
template <bool WIDE>
__device__ __forceinline__ void store_two(uint16_t *a, uint16_t *b, const uint4 &x, const uint4 &y)
{
    if (WIDE) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(a), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w), "r"(y.x),
                     "r"(y.y), "r"(y.z), "r"(y.w) : "memory");
    } else {
        *reinterpret_cast<uint4 *>(a) = x;
        *reinterpret_cast<uint4 *>(b) = y;
    }
}

// WIDE: neighbours, every head and its rotated part 32-byte aligned.
template <bool NEIGHBOURS, bool WIDE>
__global__ void __launch_bounds__(ROT_THREADS)
rotary_kernel(const RotaryParams p)
{
    __shared__ int32_t pos_s[ROT_ROWS];
    const int t = threadIdx.x;
    wait_prior_grid();
    const int32_t row0 = blockIdx.x * p.cta_rows, n_rows = min(p.cta_rows, p.seq.rows - row0);
    const int32_t turned = p.rope_dim / 16;                  // items of a head that rotate, then those that are copied
    const int32_t items = p.items, per_row = items * p.slices, total = n_rows * per_row;
    const int32_t heads = p.q_heads + p.k_heads;
    // a thread's work: a row, a piece of each head (as two vectors of dims), every slices-th head
    const int32_t r = t / per_row, in_row = t - r * per_row, slice = in_row / items, item = in_row - slice * items;
    const int64_t row = row0 + r;
    const bool mine = t < total, turn = item < turned;
    int32_t d0, d1;
    if (turn) {
        d0 = p.first + (NEIGHBOURS ? 16 : 8) * item;
        d1 = d0 + (NEIGHBOURS ? 8 : p.rope_dim / 2);
    } else {
        // vectors outside the rotated part, in order
        const int32_t v = 2 * (item - turned), skip = p.rope_dim / 8, before = p.first / 8;
        d0 = 8 * (v < before ? v : v + skip);
        d1 = 8 * (v + 1 < before ? v + 1 : v + 1 + skip);
    }
    auto in_of = [&](int32_t h) {
        return h < p.q_heads ? p.q + (row * p.q_stride + static_cast<int64_t>(h) * p.head_dim)
                             : p.k + (row * p.k_stride + static_cast<int64_t>(h - p.q_heads) * p.head_dim);
    };
    auto out_of = [&](int32_t h) {
        return h < p.q_heads ? p.out_q + (row * p.out_q_stride + static_cast<int64_t>(h) * p.head_dim)
                             : p.out_k + (row * p.out_k_stride + static_cast<int64_t>(h - p.q_heads) * p.head_dim);
    };
    uint4 x[ROT_BATCH], y[ROT_BATCH];
    auto load = [&](int32_t h0) {
#pragma unroll
        for (int k = 0; k < ROT_BATCH; ++k) {
            const int32_t h = h0 + k * p.slices;
            if (h >= heads) break;
            load_two<WIDE>(in_of(h) + d0, in_of(h) + d1, x[k], y[k]);
        }
    };
    // the first values are on their way while the rows' positions are looked up
    if (mine) load(slice);
    if (blockIdx.x == 0) flag_bad_requests(p.seq);
    Seq s;
    const int32_t b = requests_of_rows(p.seq, row0, n_rows, &s);
    if (t < n_rows) pos_s[t] = b < 0 ? -1 : s.p0 + (row0 + t - s.s0);
    __syncthreads();

    const int32_t at = mine ? pos_s[r] : -1;
    float cs[8], sn[8];
    if (at >= 0 && turn) {
        const float4 *tab = reinterpret_cast<const float4 *>(p.table + static_cast<int64_t>(at) * p.rope_dim + 8 * item);
        const float4 *tbs = reinterpret_cast<const float4 *>(p.table + static_cast<int64_t>(at) * p.rope_dim + p.rope_dim / 2 + 8 * item);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float4 c = __ldg(tab + k), s = __ldg(tbs + k);
            cs[4 * k] = c.x, cs[4 * k + 1] = c.y, cs[4 * k + 2] = c.z, cs[4 * k + 3] = c.w;
            sn[4 * k] = s.x, sn[4 * k + 1] = s.y, sn[4 * k + 2] = s.z, sn[4 * k + 3] = s.w;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) cs[k] = 1.0f, sn[k] = 0.0f;
    }
    for (int32_t h0 = slice; at >= 0 && h0 < heads;) {
#pragma unroll
        for (int k = 0; k < ROT_BATCH; ++k) {
            const int32_t h = h0 + k * p.slices;
            if (h >= heads) break;
            if (!turn && in_of(h) == out_of(h)) continue;     // in place
            if (turn) rotate8<NEIGHBOURS>(x[k], y[k], cs, sn);
            store_two<WIDE>(out_of(h) + d0, out_of(h) + d1, x[k], y[k]);
        }
        h0 += p.slices * ROT_BATCH;
        if (h0 < heads) load(h0);
    }
    allow_next_grid();
}

__global__ void __launch_bounds__(256)
rotary_table_kernel(float *table, int32_t n_pos, int32_t half, const RotaryAngles a)
{
    const int64_t n = static_cast<int64_t>(n_pos) * half;
    wait_prior_grid();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t pos = i / half;
        const int32_t j = static_cast<int32_t>(i - pos * half);
        double s, c;
        sincos(static_cast<double>(pos) * a.f[j], &s, &c);
        float *row = table + pos * (2 * half);
        row[j] = static_cast<float>(a.amplitude * c);
        row[half + j] = static_cast<float>(a.amplitude * s);
    }
}

}  // namespace

int launch_rotary_table(float *table, int32_t n_pos, int32_t rope_dim, const RotaryAngles &angles, int sms, void *stream)
{
    int32_t half = rope_dim / 2;
    const int64_t blocks = (static_cast<int64_t>(n_pos) * half + 255) / 256;
    const int grid = static_cast<int>(std::min<int64_t>(blocks, 8 * sms));
    void *args[] = {&table, &n_pos, &half, const_cast<RotaryAngles *>(&angles)};
    return launch_kernel(reinterpret_cast<const void *>(&rotary_table_kernel), dim3(grid), dim3(256), 0,
                         static_cast<cudaStream_t>(stream), false, args);
}

int launch_rotary(const RotaryParams &in, bool neighbours, int sms, void *stream)
{
    RotaryParams p = in;
    const int32_t heads = p.q_heads + p.k_heads;
    // ROT_HEADS heads to a thread, fewer while threads are few
    const int64_t want = static_cast<int64_t>(sms) * 1024;
    const int64_t each = static_cast<int64_t>(p.seq.rows) * p.items * heads / want;
    const int32_t mine = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(each, ROT_HEADS)));
    const int32_t most = (heads + mine - 1) / mine;
    p.slices = std::max(1, std::min(most, ROT_THREADS / p.items));
    const int32_t per_row = p.items * p.slices;
    p.cta_rows = std::max(1, std::min(ROT_ROWS, ROT_THREADS / per_row));
    const unsigned threads = static_cast<unsigned>(std::max(p.cta_rows, std::min(ROT_THREADS, p.cta_rows * per_row)) + 31) / 32 * 32;
    const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(p.seq.rows) + p.cta_rows - 1) / p.cta_rows);
    // neighbours in 32-byte pieces where all of them are aligned
    const uint64_t places = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k) | reinterpret_cast<uintptr_t>(p.out_q) |
                            reinterpret_cast<uintptr_t>(p.out_k) |
                            2 * static_cast<uint64_t>(p.q_stride | p.k_stride | p.out_q_stride | p.out_k_stride | p.first);
    const void *kernel = !neighbours ? reinterpret_cast<const void *>(&rotary_kernel<false, false>)
                         : places % 32 == 0 ? reinterpret_cast<const void *>(&rotary_kernel<true, true>)
                                            : reinterpret_cast<const void *>(&rotary_kernel<true, false>);
    void *args[] = {&p};
    return launch_kernel(kernel, dim3(grid), dim3(threads), 0, static_cast<cudaStream_t>(stream), false, args);
}

}  // namespace qsa
