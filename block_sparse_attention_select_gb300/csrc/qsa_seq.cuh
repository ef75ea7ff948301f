// Batches of requests: which request a row belongs to, and where a token lies
// in the paged cache (shared by the K/V cache kernels).
#pragma once
#include <cstdint>

#include "qsa_device.cuh"

namespace qsa {

// One request's new tokens: rows s0 .. s0 + n - 1 at positions p0 ..; n = 0
// when the request is empty or its data is out of range.
struct Seq {
    int32_t s0, n, p0;
};

__device__ __forceinline__ Seq seq_of(const KvParams &p, int32_t b, bool *bad)
{
    Seq s;
    s.s0 = __ldg(p.seq_start + b);
    s.n = 0;
    const int32_t s1 = __ldg(p.seq_start + b + 1);
    s.p0 = __ldg(p.pos_start + b);
    const int64_t n = static_cast<int64_t>(s1) - s.s0;
    const bool ok = s.s0 >= 0 && n >= 0 && s1 <= p.rows && s.p0 >= 0 &&
                    s.p0 + n <= (static_cast<int64_t>(p.max_pages) << p.page_shift);
    // a request without new tokens has no position to be wrong about
    *bad = !ok && n != 0;
    if (ok) s.n = static_cast<int32_t>(n);
    return s;
}

// Every request of the batch checked by one CTA (the rows of a bad request are
// skipped by the search below, so nothing else would notice some of them).
__device__ __forceinline__ void flag_bad_requests(const KvParams &p)
{
    for (int32_t b = threadIdx.x; b < p.n_reqs; b += blockDim.x) {
        bool bad;
        seq_of(p, b, &bad);
        if (bad) record_error(p.status, ST_BAD_ROW);
    }
}

// The request that holds `row` (same row in every lane), -1 for none: the last
// one that starts at or before it, by a 32-way search of seq_start.
__device__ __forceinline__ int32_t find_request(const KvParams &p, int32_t row, int lane)
{
    int32_t lo = 0, hi = p.n_reqs;
    while (true) {
        const int32_t step = (hi - lo + 31) >> 5;
        const int32_t i = lo + lane * step;
        const uint32_t m = __ballot_sync(0xffffffffu, i < hi && __ldg(p.seq_start + i) <= row);
        // the run of set lanes from lane 0 (all of them, in increasing starts)
        const int run = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
        if (run == 0) return -1;
        lo += (run - 1) * step;
        hi = min(hi, lo + step);
        if (step == 1) return lo;
    }
}

}  // namespace qsa
