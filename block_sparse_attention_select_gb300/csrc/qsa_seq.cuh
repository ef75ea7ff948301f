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

__device__ __forceinline__ Seq seq_from(const KvParams &p, int32_t s0, int32_t s1, int32_t p0, bool *bad)
{
    Seq s{s0, 0, p0};
    const int64_t n = static_cast<int64_t>(s1) - s.s0;
    const bool ok = s.s0 >= 0 && n >= 0 && s1 <= p.rows && s.p0 >= 0 &&
                    s.p0 + n <= (static_cast<int64_t>(p.max_pages) << p.page_shift);
    // a request without new tokens has no position to be wrong about
    *bad = !ok && n != 0;
    if (ok) s.n = static_cast<int32_t>(n);
    return s;
}

__device__ __forceinline__ Seq seq_of(const KvParams &p, int32_t b, bool *bad)
{
    return seq_from(p, __ldg(p.seq_start + b), __ldg(p.seq_start + b + 1), __ldg(p.pos_start + b), bad);
}

// The same past the L1 cache, for a kernel that looks before it has waited for the
// kernel before it (which read them, too: they are older than both).
__device__ __forceinline__ Seq seq_of_early(const KvParams &p, int32_t b, bool *bad)
{
    return seq_from(p, __ldcg(p.seq_start + b), __ldcg(p.seq_start + b + 1), __ldcg(p.pos_start + b), bad);
}

// Whether a request has the row.  (n > 0 first: a skipped request's start may be any
// number, and the difference wrap.)
__device__ __forceinline__ bool has_row(const Seq &s, int32_t row) { return s.n > 0 && row >= s.s0 && row - s.s0 < s.n; }

// The request of a row, or -1; its tokens in *s.
__device__ __forceinline__ int32_t request_of(const KvParams &p, int32_t row, Seq *s)
{
    // the last request that starts at or before the row
    int32_t lo = 0, hi = p.n_reqs;
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) >> 1;
        if (__ldg(p.seq_start + mid) <= row) lo = mid;
        else hi = mid;
    }
    bool bad;
    *s = seq_of(p, lo, &bad);
    return has_row(*s, row) ? lo : -1;
}

// The same where the starts fall somewhere: the first request that has the row.
__device__ __forceinline__ int32_t request_of_unsorted(const KvParams &p, int32_t row, Seq *s)
{
#pragma unroll 1
    for (int32_t b = 0; b < p.n_reqs; ++b) {
        bool bad;
        *s = seq_of(p, b, &bad);
        if (has_row(*s, row)) return b;
    }
    return -1;
}

// The same for one row by a whole warp, with the same result in every lane.  Up to
// 32 requests are all looked at, after one memory latency; else each step asks 32
// places among the requests left.  *falls: whether starts fall somewhere, found out
// where it matters (-1: not yet).
__device__ __forceinline__ int32_t request_of_by_warp(const KvParams &p, int32_t row, int lane, int *falls, Seq *s)
{
    if (p.n_reqs <= 32) {
        bool bad;
        const Seq x = seq_of(p, min(lane, p.n_reqs - 1), &bad);
        const uint32_t m = __ballot_sync(0xffffffffu, has_row(x, row));
        if (m == 0) return -1;
        const int from = __ffs(m) - 1;
        s->s0 = __shfl_sync(0xffffffffu, x.s0, from);
        s->n = __shfl_sync(0xffffffffu, x.n, from);
        s->p0 = __shfl_sync(0xffffffffu, x.p0, from);
        return from;                         // (the first lane that has it: its own request)
    }
    int32_t lo = 0, n = p.n_reqs;            // among requests lo .. lo + n - 1
    while (n > 1) {
        const int32_t step = (n + 31) / 32, at = lane * step;
        const bool before = at < n && __ldg(p.seq_start + lo + at) <= row;
        const uint32_t m = __ballot_sync(0xffffffffu, before);
        const int32_t k = m ? 31 - __clz(m) : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    bool bad;
    *s = seq_of(p, lo, &bad);
    if (has_row(*s, row)) return lo;
    if (*falls < 0) {
        bool f = false;
        for (int32_t b = lane; b < p.n_reqs; b += 32) f = f || __ldg(p.seq_start + b + 1) < __ldg(p.seq_start + b);
        *falls = __any_sync(0xffffffffu, f) ? 1 : 0;
    }
    if (*falls == 0) return -1;
    for (int32_t b0 = 0; b0 < p.n_reqs; b0 += 32) {
        *s = seq_of(p, min(b0 + lane, p.n_reqs - 1), &bad);
        const uint32_t m = __ballot_sync(0xffffffffu, b0 + lane < p.n_reqs && has_row(*s, row));
        if (m == 0) continue;
        const int32_t b = b0 + __ffs(m) - 1;
        *s = seq_of(p, b, &bad);
        return b;
    }
    return -1;
}

// Requests of rows row0 .. row0 + n - 1, a row per thread of the CTA (n <= its
// threads), -1 for rows of no request; every thread of the CTA calls it.
__device__ __forceinline__ int32_t requests_of_rows(const KvParams &p, int32_t row0, int32_t n, Seq *s)
{
    const int t = threadIdx.x;
    int32_t b = -1;
    if (t < n) b = request_of(p, row0 + t, s);
    const bool lost = t < n && b < 0;
    // no request: a row behind the last one or of a request that is skipped, or the
    // search passed it by where the starts are out of order
    if (__syncthreads_or(lost)) {
        bool falls = false;
#pragma unroll 4
        for (int32_t i = t; i < p.n_reqs; i += blockDim.x)
            falls = falls || __ldg(p.seq_start + i + 1) < __ldg(p.seq_start + i);
        if (__syncthreads_or(falls) && lost) b = request_of_unsorted(p, row0 + t, s);
    }
    return b;
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
