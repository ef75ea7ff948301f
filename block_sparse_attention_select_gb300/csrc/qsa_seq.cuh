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

// Every request of the batch checked by one CTA (a search by row skips the rows of
// a bad request, so nothing else would notice some of them).
__device__ __forceinline__ void flag_bad_requests(const KvParams &p)
{
    for (int32_t b = threadIdx.x; b < p.n_reqs; b += blockDim.x) {
        bool bad;
        seq_of(p, b, &bad);
        if (bad) record_error(p.status, ST_BAD_ROW);
    }
}

}  // namespace qsa
