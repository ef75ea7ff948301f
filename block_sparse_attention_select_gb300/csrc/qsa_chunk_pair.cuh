// Attention of new tokens over the paged K/V cache, on pairs of SMs: the kernel of
// dense attention (qsa_chunk.cu) and of attention over selected blocks (qsa_blocks.cu).
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
// that the CTA pairs share out evenly (each unit UNIT_COST tiles longer than it
// is, for what it costs besides them: counted as 2, 3, 4 and 5 tiles, four prompts
// of 4,096 tokens took 495, 483, 419 and 460 us on one warm card; taken over for
// 256-wide heads and E4M3, where it was not measured), so one row over
// a long cache, a batch of unequal requests and a long prompt all fill the card.  A unit that
// lies across pairs leaves unnormalised FP32 partial sums with their maxima in
// the workspace (at most two per pair), which a second kernel joins.  Every
// pair finds its share itself from seq_start and pos_start: no plan kernel and
// no host knowledge of the lengths.
//
// A CTA's warps: 0-7 softmax, 8 loads K and V by TMA, one box per page piece,
// through the block table, 9 issues the MMAs (in the first CTA of the pair; with
// D = 128 warp 11 issues the second products, so that neither product waits for
// what the other needs), 10 walks through the share and hands out its segments,
// 12-15 load the queries, clear the value rows that nothing attends and write the
// outputs or, from the E4M3 cache, turn the loaded codes into FP16 tiles (the
// softmax warps then write the outputs).  K and V share a ring of slots in the
// order of use; with D = 128 each has its own.
//
// Softmax warps 0-3 take the even tiles and 4-7 the odd ones (warp w: TMEM lane
// quarter w % 4, a row per thread), so that one group's exponentials run beside
// the other's waits; S has a buffer for each.  A thread takes its 128 scores
// into registers, its row's running maximum passes on from tile to tile, from
// one group to the other, before the exponentials start, and each group keeps
// its own sum.  P goes to TMEM as FP16, in two halves, and is the A operand of the
// second product from there.  With D = 128, P has columns of its own, so the score
// product of the tile after next starts as soon as the scores are in registers:
//   S(0) S(1) | S(2) O(0) | S(3) O(1) | ...
// With D = 256, TMEM is full (2 x 128 for S, 256 for O): P overwrites its
// scores and the order is S(0) S(1) | O(0) S(2) | O(1) S(3) | ...
//
// What bounds it (times of single calls on a cool card, in parentheses in a stream
// of calls, where the power cap takes some of the clock): with D = 256 and a long
// context the tensor cores (the 1,616-row chunk over 29,000 tokens, 12 query heads
// to a KV head: 567 us (661), 1,970 TF/s, tensor pipe 94% busy).  With D = 128 a
// tile's products take half as long and its exponentials the same, so the latency
// of two softmax warps per scheduler shows (four prompts of 4,096 tokens, 32 heads:
// 377 us (424), 1,460 TF/s; tensor pipe 69%, issue slots 48%).  From the E4M3 cache
// the turning of codes into FP16 tiles, anew for each unit of 256 pairs (three
// chunks of up to 517 over up to 12,345 tokens: 151 us (156), 1,290 TF/s, tensor pipe
// 59%).  Two chunks of up to 1,023 tokens with a window of 1,000 take 38 us (43) where
// their products need 9: the search for the work, the first loads and the last
// output are a third of it, the rest has not been taken apart.
//
// From the E4M3 cache times move by up to 8% with the place of the kernel's code:
// two groups of warps in long unrolled loops share the instruction caches.
//
// Over selected blocks (BlockPairGeometry) a unit is whole tokens, its tiles are the
// blocks of its list (qsa_chunk.cuh), and a row that does not attend a tile takes
// weights of zero; a warp none of whose rows does leaves its scores where they are.
// So the products are those of the units' lists: the 1,616-row chunk over 184,320
// tokens, 24 query heads over 2 KV heads of 128, 17 blocks to a row, has 21 tokens to
// a unit and 77 blocks to a list, 22% of them of use to a row.  It takes 150 us, of
// which the lists and the join of partial results are some 8; tensor pipe 64%, as in
// dense attention with such heads.  Four prompts of 8,192 (32 tokens, 25 blocks to a
// list, 58% of use): 1,145 to 1,190 us, 67%.  Three E4M3 chunks of up to 517 (256-wide
// heads, 34 blocks): 86 us, 46%, the helpers' codes again.  Those cost most with whole
// prompts of 128-wide heads, 2,085 us where the FP16 cache takes 1,153: each unit turns
// each block of its list anew, and reading the contexts back first (qsa_kv_load, 25 us)
// and attending the FP16 copy takes 1,158 in all, with the same bits (256-wide heads,
// 24 over 2: 1,735 and 1,336; three chunks of 512: 171 and 170).  UNIT_COST 1, 2, 6 and 8
// for lists: the prompts take 1,281, 1,231, 1,190 and 1,190 us, the E4M3 chunks 91, 89,
// 91 and 92.  (An entry and its bits are loaded a tile ahead: looked up at the tile they
// cost the softmax 180 clocks of 3,000.)
//
// The accumulator is rescaled only when a row's maximum has grown by more than
// 2^8 since the one in use: the sum uses the same stale maximum, so the result
// is the same.  Rounding P to FP16 (2^-11 of each weight, with the smallest ones
// kept by a factor, see RESCALE) is of the size of the output's own rounding.
#pragma once
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "qsa_chunk.cuh"

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
constexpr int MAX_RAWS = 4;                  // slots of loaded codes at most (E4M3)
constexpr int MAX_SLOTS = 10;                // slots of the ring at most
constexpr uint32_t RING = 229376;            // bytes for Q and the ring
constexpr uint32_t TM_S = 0, TM_O = 256;     // TMEM columns: two S buffers of 128, O
constexpr int BAR_PAIR = 1, BAR_HELP = 5;    // named barriers: four softmax warp pairs, the helpers

struct PairGeometry {
    static constexpr bool BLOCKS = false;
    static constexpr int RAWS = 4;           // slots of loaded codes (E4M3)
    static constexpr bool RAW_MAX = false;   // the parts' maxima: powers of two, or scores before the scale
    static constexpr int ROWS = CH_ROWS, TILE = CH_TILE, UNIT_COST = 4, MIN_SHARE = 4, THREADS = CH_THREADS, WARPS = CH_WARPS,
                         WORKERS = CHUNK_MAX_PAIRS;
};
struct BlockPairGeometry : PairGeometry {       // tiles are the blocks of a list
    static constexpr bool BLOCKS = true;
    // As measured, the reason has not been found: 128-wide prompts with 4, 3 and 2 slots,
    // lists (4 of 8,192, 32 heads over 4) 2,168, 2,086 and 2,181 us, dense (4 of 4,096, 32
    // over 8) 613, 619 and 657; 256-wide heads differ by 1%.
    static constexpr int RAWS = 3;
};

template <int D, bool Q8>
struct Shape {
    static constexpr int QBUFS = D == 128 ? 2 : 1;                     // buffers of Q
    static constexpr uint32_t QB = CH_HALF * D * 2;                    // bytes of one
    // a CTA's half of a K tile: 64 tokens, or of a V tile: D / 2 dims of 128 tokens
    static constexpr uint32_t SLOT = 128 * D, RAW = SLOT / 2;
    static constexpr int KTOK = 64, VTOK = CH_TILE;
    static constexpr int FIT = (RING - QBUFS * QB - (Q8 ? MAX_RAWS * RAW : 0)) / SLOT, NS = FIT < MAX_SLOTS ? FIT : MAX_SLOTS;
    static constexpr bool OWN_P = D == 128;                            // P beside S, not over it
    // With two issuing warps, keys and values have rings of their own, so that
    // each warp waits for every phase of its slots in turn.
    static constexpr int NK = OWN_P ? NS / 2 : NS, NV = OWN_P ? NS - NK : 1;   // slots 0 .. NK - 1, then the values'
    static constexpr uint32_t TM_P = OWN_P ? 384 : TM_S, P_STRIDE = OWN_P ? 64 : 128;
    static constexpr int LEAD = OWN_P ? 3 : 2;                         // key tiles loaded before the first value tile
    static constexpr bool HELP_OUT = !Q8;                              // the helpers write a unit's output
};

// A role's place in the ring of slots (one ring, or one for keys and one for
// values), and the parity of the use it is at.
template <typename Sh>
struct RingPos {
    uint32_t k = 0, kp = 0, v = 0, vp = 0;
    __device__ __forceinline__ uint32_t slot(bool is_v) const { return Sh::OWN_P && is_v ? Sh::NK + v : k; }
    __device__ __forceinline__ uint32_t phase(bool is_v) const { return Sh::OWN_P && is_v ? vp : kp; }
    __device__ __forceinline__ void next(bool is_v)
    {
        if (Sh::OWN_P && is_v) {
            if (++v == Sh::NV) {
                v = 0;
                vp ^= 1u;
            }
        } else if (++k == Sh::NK) {
            k = 0;
            kp ^= 1u;
        }
    }
};

struct Ctrl {
    SegRing segs;
    uint64_t full[MAX_SLOTS], empty[MAX_SLOTS], raw_full[MAX_RAWS], raw_empty[MAX_RAWS], bnd[8];
    uint64_t s_full[2], s_free[2], p_full[2][2], o_done[2], m_out[2][4], q_full[2], q_free[2], drain[2];
    uint64_t o_last, o_free, f_full, f_free, l_out[4];
    alignas(8) float mrow[2][CH_HALF];       // [tile parity][row]: maximum in use at the group's last tile; E4M3: sums at a segment's end
    union {
        uint32_t scale[2][CH_TILE];          // [slot parity][token]: FP16 scale, twice (E4M3)
        struct {                             // (FP16 cache)
            float factor[CH_HALF];           // [row]: what the unit's output is multiplied by
            float lrow[CH_HALF];             // [row]: the sum of the group that does not have the segment's last tile
        };
    };
    Share share;
    uint32_t tmem;
    int32_t abort;
};

// ------------------------------------------------------------------- pieces --

// Slots of a segment of n tiles, in the order of use: LEAD key tiles, then value
// and key tiles in turn, then the value tiles left,
// e.g. K(0) K(1) V(0) K(2) V(1) ... K(n-1) V(n-2) V(n-1); here that of a value tile.
template <int LEAD>
__device__ __forceinline__ int32_t slot_of_v(int32_t tile, int32_t n)
{
    const int32_t lead = min(LEAD, n);
    return lead + (tile < n - lead ? 2 * tile : n - lead + tile);
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

// 32 bytes, in one store where they are aligned.
__device__ __forceinline__ void store32(void *dst, const uint32_t *v, bool whole)
{
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                     "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
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

// Writes a word of the other CTA's shared memory.
__device__ __forceinline__ void tell_other(const void *p, uint32_t other, uint32_t value)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(other));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(value) : "memory");
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

// The same on a barrier of this CTA.
__device__ __forceinline__ void mbar_expect_tx_at(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// 3-D tiled load (from x = 0) into this CTA, completing on a barrier of either CTA
// of the pair.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void *tmap, uint32_t bar, int32_t y, int32_t z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(0), "r"(y), "r"(z)
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

// 32 columns, and their maximum in each lane.
__device__ __forceinline__ float tmem_ld_max_x32(uint32_t taddr, uint32_t (&v)[32])
{
    float m;
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, %32, [%33];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31]), "=f"(m)
        : "r"(taddr)
        : "memory");
    return m;
}

__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

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

// A slot of loaded codes as the FP16 tile that the products read, by 128
// threads: 16 codes at a time, times the token's scale; tokens outside a .. z - 1
// become zeros.  Codes lie in rows of 128 bytes (V of a 128-wide head: 64), one
// token's 128 (64) dims; a thread keeps its place in the row and steps over rows,
// so that all its addresses are one base and constants.
template <int D, bool V>
__device__ __forceinline__ void codes_to_half(const uint8_t *src, uint8_t *dst, const uint32_t *scale, int ht, int a, int z)
{
    constexpr int SH = V && D == 128 ? 2 : 3;                 // log2 of a row's 16-code pieces
    constexpr int TOKS = V ? CH_TILE : 64, STEP = 128 >> SH;  // tokens of the slot, rows per pass
    constexpr int N = 128 * D / 2 / 16 / 128;                 // pieces per thread
    const int pc = ht & ((1 << SH) - 1);
    // Dims 16 pc .. of the row go to chunk pc / 4, pieces 2 (pc % 4) and + 1.  With
    // eight pieces to a row, lanes of the upper four take the neighbouring row:
    // the eight stores then meet all banks.
    const int r0 = SH == 3 ? (ht >> 3) ^ (pc >> 2) : ht >> 2;
    const uint8_t *in = src + (r0 << (SH + 4)) + pc * 16;
    uint8_t *out = dst + (pc >> 2) * (TOKS * 128) + r0 * 128;
    const uint32_t p0 = 2 * (pc & 3), o0 = (p0 ^ (r0 & 7)) << 4, o1 = ((p0 + 1) ^ (r0 & 7)) << 4;
    const bool cut = a > 0 || z < TOKS;
    // four pieces at a time, rolled: half the code at D = 256 (unrolled, its time
    // moved by 8% with whatever else changed in the kernel's code)
    static_assert(4 * STEP == TOKS || 4 * STEP == TOKS / 2, "a pass is the tile's tokens or half of them");
    constexpr bool WHOLE = 4 * STEP == TOKS;                  // then the next pass has the next 128 dims
    const uint32_t *sc_at = scale + r0;
    int tok = r0;
#pragma unroll 1
    for (int i0 = 0; i0 < N; i0 += 4) {
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const uint4 *>(in + i * (16 * 128));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t sc = sc_at[STEP * i];
            const uint32_t cw[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            uint32_t o[8];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
                    "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
                    : "=r"(o[2 * k]), "=r"(o[2 * k + 1])
                    : "r"(cw[k]));
#pragma unroll
            for (int k = 0; k < 8; ++k) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(o[k]) : "r"(sc));
            if (cut && (tok + STEP * i < a || tok + STEP * i >= z)) {
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] = 0u;
            }
            *reinterpret_cast<uint4 *>(out + STEP * i * 128 + o0) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4 *>(out + STEP * i * 128 + o1) = make_uint4(o[4], o[5], o[6], o[7]);
        }
        in += 4 * 16 * 128;
        out += WHOLE ? 2 * TOKS * 128 : 4 * STEP * 128;
        if (!WHOLE) {
            sc_at += 4 * STEP;
            tok += 4 * STEP;
        }
    }
}

// ------------------------------------------------------------------- kernel --

template <int D, bool Q8, typename G>
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
        for (int i = 0; i < G::RAWS; ++i) {
            mbar_init(&c.raw_full[i], 1);
            mbar_init(&c.raw_empty[i], CH_HELPERS);
        }
        for (int i = 0; i < 8; ++i) mbar_init(&c.bnd[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c.s_full[i], 1);
            for (int k = 0; k < 2; ++k) mbar_init(&c.p_full[i][k], CH_SOFT);    // four warps of each CTA
            mbar_init(&c.s_free[i], CH_SOFT);
            mbar_init(&c.o_done[i], 1);
            for (int k = 0; k < 4; ++k) mbar_init(&c.m_out[i][k], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c.q_full[i], 2 * CH_HELPERS);
            mbar_init(&c.q_free[i], 1);
        }
        for (int i = 0; i < SEGS; ++i) {
            mbar_init(&c.segs.full[i], 1);
            mbar_init(&c.segs.empty[i], CH_ROLES);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&c.drain[i], 1);
        mbar_init(&c.o_last, 1);
        mbar_init(&c.o_free, 2 * CH_HELPERS);                 // in the first CTA, for both
        mbar_init(&c.f_full, 4);
        mbar_init(&c.f_free, CH_HELPERS);
        for (int i = 0; i < 4; ++i) mbar_init(&c.l_out[i], 1);
        c.abort = 0;
        fence_barrier_init();
    }
    if (warp == CH_MMA) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&c.tmem)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (!G::BLOCKS) wait_prior_grid();
    // The join's CTAs wait on the device: the windowed chunk 41 -> 38 us.  From the E4M3
    // cache that hides nothing, and this instruction's place moves the turning of codes:
    // with it, without it, dense 128-wide prompts 627 and 614 us, 256-wide chunks 154 and
    // 152; lists, 256-wide chunks 87.5 and 86.2, 128-wide prompts 2,166 and 2,257.
    if (!Q8 || (G::BLOCKS && D == 128)) allow_next_grid();
    // (the queries' place is free until the segments are known)
    static_assert(sizeof(FindScratch<G>) <= Sh::QB, "scratch");
    find_work<G>(p, c.share, *reinterpret_cast<FindScratch<G> *>(q_s), blockIdx.x >> 1, gridDim.x >> 1, warp, lane, [&]() {
        if (G::BLOCKS) wait_prior_grid();
    });
    tc_fence_before();
    __syncthreads();
    cluster_sync();                                          // the pair's barriers and TMEM are ready
    tc_fence_after();
    const uint32_t tmem = c.tmem;
    const uint32_t ring_a = smem_u32(ring);
    uint32_t segs = 0;
    Seg w;
    auto next_segment = [&]() -> bool { return qsa::next_segment(c.segs, &segs, &w, lane); };
    // registers after the split: 8 x 32 x 200 + 8 x 32 x 56 = 65,536
    if (warp >= CH_LOAD && warp < CH_HELP) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == CH_LOAD) {
        // ---------------------------------------------------------- K, V loads
        // This loop has to keep up with the products (a few hundred clocks per slot
        // with 128-wide heads), on a warp that shares its issue slots and instruction
        // cache with the softmax, so few instructions matter most: one copy per slot
        // where a page holds its tokens, page lookups for many tiles at once, one
        // thread that issues.  (With a box per 128-byte chunk, a lane each, and
        // lookups tile by tile the loop took 1,600 clocks per tile and the products
        // waited for it: 796 us on 512 new tokens of four requests over 32,768, 755 so.)
        const uint32_t dst0 = Q8 ? smem_u32(raw) : ring_a;
        constexpr uint32_t BYTES = Q8 ? RAW : SLOT;
        // elements of a box row: 128 bytes, or half a 128-wide head's 64 codes
        constexpr int CK = Q8 ? 128 : 64, CV = Q8 ? D / 2 : 64;
        constexpr int KCH = D / CK, VCH = D / 2 / CV;         // such rows of a token
        uint64_t *empty = Q8 ? c.raw_empty : c.empty;
        const int32_t P = p.kv.page_tokens;
        const int sh = __ffs(min(P, CH_TILE)) - 1;            // log2 of a piece: tokens of a tile in one page
        const int ld = 7 - sh;                                // log2 of the pieces of a tile
        const int32_t batch = 32 >> ld;                       // tiles whose pieces the lanes look up at a time
        const int32_t nowhere = p.kv.num_pages << p.kv.page_shift;      // a row past the cache: reads zeros
        const uint32_t full0 = of_first(&c.full[0]);
        RingPos<Sh> pos;
        uint32_t rslot = 0, rphase = 0, used = 0, last = 0;   // raw slots; those loaded at least once, their latest phases
        uint32_t nb = 0;                                      // boundary tiles so far
        bool ok = true;
        while (next_segment()) {
            if (!ok) continue;
            const int32_t *bt = p.kv.block_table + static_cast<int64_t>(w.b) * p.kv.max_pages;
            const int32_t n = w.n;
            const int32_t lane_tok = w.j0 * CH_TILE + (lane << sh);     // the lane's piece of the first tiles
            const int32_t lane_off = lane_tok & (CH_TILE - 1);          // its place in the tile
            const int32_t *list = G::BLOCKS ? list_of(p, w) + w.j0 : nullptr;
            auto entry_of = [&](int32_t j) -> int32_t { return j + (lane >> ld) < n ? __ldg(list + j + (lane >> ld)) : NO_BLOCK; };
            // this lane's page of tiles j .. j + batch - 1; none without a token that
            // is attended
            auto page_of = [&](int32_t j, int32_t ent) -> int32_t {
                if constexpr (G::BLOCKS) {
                    const int32_t page = (entry_block(ent) * CH_TILE + lane_off) >> p.kv.page_shift;
                    return lane_off < entry_seen(ent) && page < p.kv.max_pages ? __ldg(bt + page) : INT32_MAX;
                }
                const int32_t tok = lane_tok + j * CH_TILE;
                const bool seen = j + (lane >> ld) < n && tok <= w.hi_tok && tok + ((1 << sh) - 1) >= w.lo_tok;
                return seen ? __ldg(bt + (tok >> p.kv.page_shift)) : INT32_MAX;
            };
            auto row_of = [&](int32_t page, int32_t j, int32_t ent) -> int32_t {
                const int32_t tok = G::BLOCKS ? entry_block(ent) * CH_TILE + lane_off : lane_tok + j * CH_TILE;
                if (static_cast<uint32_t>(page) < static_cast<uint32_t>(p.kv.num_pages))
                    return (page << p.kv.page_shift) + (tok & (P - 1));
                if (page != INT32_MAX) record_error(p.kv.status, ST_BAD_PAGE);
                return nowhere;
            };
            // list entries of this batch, the next and the one after
            int32_t ent_v = NO_BLOCK, ent1_k = G::BLOCKS ? entry_of(0) : 0, ent1_v = ent1_k, ent2_k = G::BLOCKS ? entry_of(batch) : 0,
                    ent2_v = ent2_k;
            int32_t page_k = page_of(0, ent1_k), page_v = page_k, row_k = 0, row_v = 0;  // pages of the next batch, rows of this one
            auto load = [&](auto is_v, int32_t tile) {
                constexpr bool V = decltype(is_v)::value;
                constexpr int TOKS = V ? Sh::VTOK : Sh::KTOK, CH = V ? VCH : KCH;
                constexpr uint32_t ROW = V ? (Q8 ? CV : 128) : 128;      // bytes of a box row
                const uint32_t slot = Q8 ? rslot : pos.slot(V), phase = Q8 ? rphase : pos.phase(V);
                const int32_t in = tile & (batch - 1);
                if (in == 0) {
                    (V ? row_v : row_k) = row_of(V ? page_v : page_k, tile, V ? ent1_v : ent1_k);
                    if (G::BLOCKS) {
                        if (V) ent_v = ent1_v;
                        (V ? ent1_v : ent1_k) = V ? ent2_v : ent2_k;
                        (V ? ent2_v : ent2_k) = entry_of(tile + 2 * batch);
                    }
                    (V ? page_v : page_k) = page_of(tile + batch, V ? ent1_v : ent1_k);
                }
                const int32_t row = V ? row_v : row_k;
                if (!warp_wait(&empty[slot], phase ^ 1u, abort, lim)) {
                    ok = false;
                    return;
                }
                uint32_t bar;
                const bool local = Q8 || (V && (G::BLOCKS ? entry_seen(__shfl_sync(0xffffffffu, ent_v, in << ld)) < CH_TILE
                                                          : w.cut(tile, CH_TILE)));
                if (Q8) {
                    bar = smem_u32(&c.raw_full[slot]);
                } else if (local) {
                    // the helpers clear rows of this one before the products see it
                    bar = smem_u32(&c.bnd[nb & 7u]);
                    ++nb;
                } else {
                    bar = full0 + slot * 8u;
                }
                const uint32_t dst = dst0 + slot * BYTES;
                const int32_t z = V ? (w.g * D + rank * (D / 2)) / CV : w.g * (D / CK);
                // a key slot holds the rank's half of the tile: of one piece, one piece, or half of them
                if ((TOKS >> sh) <= 1) {
                    const int32_t y = __shfl_sync(0xffffffffu, row, V ? in : sh == 7 ? in : 2 * in + rank);
                    if (elect_one()) {
                        if (local) mbar_expect_tx_at(bar, BYTES);
                        else cluster_arrive_expect_tx(bar, BYTES);
                        tma_load_3d_pair(dst, V ? &tv : &tk, bar,
                                         static_cast<int32_t>(static_cast<uint32_t>(y) + (!V && sh == 7 ? rank * 64u : 0u)), z);
                    }
                } else {
                    // a lane for each piece and chunk
                    const int32_t lp = (V ? 7 : 6) - sh, ch = lane >> lp, i = lane & ((1 << lp) - 1);
                    const int32_t y = __shfl_sync(0xffffffffu, row, (in << ld) + (V ? 0 : rank << (ld - 1)) + i);
                    if (lane == 0) {
                        if (local) mbar_expect_tx_at(bar, BYTES);
                        else cluster_arrive_expect_tx(bar, BYTES);
                    }
                    __syncwarp();
                    if (ch < CH) tma_load_3d_pair(dst + (ch * TOKS + (i << sh)) * ROW, V ? &tv : &tk, bar, y, z + ch);
                }
                __syncwarp();
                if (Q8) {
                    used |= 1u << rslot;
                    last = (last & ~(1u << rslot)) | (rphase << rslot);
                    if (++rslot == G::RAWS) {
                        rslot = 0;
                        rphase ^= 1u;
                    }
                } else {
                    pos.next(V);
                }
            };
            // the order of slots
            const int32_t lead = min(Sh::LEAD, n);
            for (int32_t j = -lead; ok && j < n; ++j) {
                if (j >= 0) load(std::true_type{}, j);
                if (ok && j + lead < n) load(std::false_type{}, j + lead);
            }
        }
        // codes still in flight, whoever gave up (otherwise the helpers waited for them)
        if (Q8 && lane == 0)
            for (int i = 0; i < G::RAWS; ++i)
                if (used & (1u << i)) mbar_wait_bounded(&c.raw_full[i], (last >> i) & 1u, drain_limit(lim));
        __syncwarp();
    } else if (warp == CH_SCHED) {
        // ----------------------------------------------------------- segments
        schedule<G>(p, c.share, c.segs, blockIdx.x >> 1, rank == 0, lane);
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
        RingPos<Sh> ringpos;
        uint32_t it = 0, seg = 0;
        bool ok = true;
        // S(i) = Q . K(i)^T
        auto scores = [&](uint32_t i, bool last) {
            const uint32_t slot = ringpos.slot(false);
            ok = ok && warp_wait(&c.full[slot], ringpos.phase(false), abort, lim);
            if (!ok) return;
            ringpos.next(false);
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
        auto values = [&](uint32_t i, bool first, bool last) {
            const uint32_t slot = ringpos.slot(true);
            // the unit before has been read
            if (Sh::HELP_OUT && first && seg > 0) ok = ok && warp_wait(&c.o_free, (seg - 1) & 1u, abort, lim);
            ok = ok && warp_wait(&c.full[slot], ringpos.phase(true), abort, lim);
            ok = ok && warp_wait(&c.p_full[i & 1u][0], (i >> 1) & 1u, abort, lim);
            if (!ok) return;
            ringpos.next(true);
            const uint64_t vd = vd0 | (uniform(ring_a + slot * SLOT) >> 4);
            const uint32_t pa = tm + Sh::TM_P + uniform(i & 1u) * Sh::P_STRIDE;
            const uint32_t add = uniform(first ? 0u : 1u);
            // the first half's products start while the softmax is at the second
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (half == 1) ok = warp_wait(&c.p_full[i & 1u][1], (i >> 1) & 1u, abort, lim);
                if (!ok) return;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
                        umma2_f16_ta(tm + TM_O, pa + kk * 8u, vd + ((kk * 2048u) >> 4), idesc_o, kk > 0 ? 1u : add);
                    if (half == 1) {
                        umma2_commit(&c.o_done[i & 1u]);
                        umma2_commit(&c.empty[slot]);
                        if (Sh::HELP_OUT && last) umma2_commit(&c.o_last);
                    }
                }
                __syncwarp();
            }
        };
        while (next_segment()) {
            if (!ok || !(do_s || do_o)) continue;
            const int32_t n = w.n;
            if (do_s) ok = warp_wait(&c.q_full[Sh::QBUFS == 2 ? seg & 1u : 0u], (Sh::QBUFS == 2 ? seg >> 1 : seg) & 1u, abort, lim);
            if constexpr (Sh::OWN_P) {
                for (int32_t j = 0; ok && j < n; ++j) {
                    const uint32_t i = it + j;
                    if (do_s) {
                        // the scores two tiles before are in registers
                        if (i > 1) ok = warp_wait(&c.s_free[i & 1u], ((i - 2) >> 1) & 1u, abort, lim);
                        scores(i, j == n - 1);
                    } else {
                        values(i, j == 0, j == n - 1);
                    }
                }
            } else {
                scores(it, n == 1);
                if (n > 1) scores(it + 1, n == 2);
                for (int32_t j = 0; ok && j < n; ++j) {
                    values(it + j, j == 0, j == n - 1);
                    if (j + 2 < n) scores(it + j + 2, j + 3 == n);
                }
            }
            it += n;
            ++seg;
        }
        // the warp's own products, whoever gave up (otherwise they were waited for)
        if (do_s || do_o) {
            if (elect_one()) {
                umma2_commit(&c.drain[do_s ? 0 : 1]);
                mbar_wait_bounded(&c.drain[do_s ? 0 : 1], 0, drain_limit(lim));
            }
            __syncwarp();
        }
    }
    } else if (warp >= CH_HELP) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        // --------------------- queries, cut value tiles, E4M3 codes to FP16 tiles
        const int ht = t - CH_HELP * 32;                      // 0 .. 127
        RingPos<Sh> pos;
        uint32_t seg = 0, rslot = 0, rphase = 0, par = 0, ring0 = 0, ring_b = 0, nb = 0;  // ring0: the next segment's first slot (OWN_P: value slot), ring_b: this one's
        bool ok = true;                                       // false: keep to the barriers, do nothing
        // The limit bounds one step, a tile; waits of these warps for the end of a
        // segment span all of its tiles (and a few steps' worth around them).
        auto span = [&](const Seg &x) -> uint64_t {
            if (!Sh::HELP_OUT) return lim;                     // these are never a segment ahead
            const uint64_t step = lim < (1ull << 36) ? lim : 1ull << 36;
            const uint64_t all = step * static_cast<uint32_t>(x.n + 8);
            return all > lim ? all : lim;
        };
        // A unit's output (or its part of it), while the softmax is at the next unit
        // (by the softmax warps themselves, a unit's end took them 2,400 clocks of
        // code that had left the instruction cache).  Warp w: TMEM lane quarter w % 4.
        Seg before;
        before.n = 0;
        auto write_out = [&]() {
            if (Sh::HELP_OUT && before.n > 0 && ok) {
                const uint32_t u = seg - 1;                    // its number
                const int lq = warp & 3, ur = rank * CH_HALF + ht;
                ok = warp_wait(&c.f_full, u & 1u, abort, span(before));
                if (!ok) return;
                const float f = c.factor[ht];
                __syncwarp();
                if (lane == 0) mbar_arrive(&c.f_free);
                ok = warp_wait(&c.o_last, u & 1u, abort, span(before));
                if (!ok) return;
                tc_fence_after();
                if (rank * CH_HALF + lq * 32 < before.rows) {
                    const bool in = ur < before.rows, whole = before.place < 0;
                    const bool out_32 = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;      // (16 bytes are promised)
                    const int32_t v = before.v0 + ur, tok = by_group(p, v), h = v - tok * p.group;
                    uint8_t *dst = whole ? static_cast<uint8_t *>(p.out) +
                                               ((static_cast<int64_t>(before.s0) + tok) * p.hq + before.g * p.group + h) * D * 2
                                         : p.ws + ws_o<CH_ROWS, CHUNK_MAX_PAIRS>() +
                                               (static_cast<int64_t>(before.place) * p.ws_rows + ur) * D * 4;
                    const uint32_t to = tmem + TM_O + (static_cast<uint32_t>(lq * 32) << 16);
#pragma unroll 1
                    for (int k = 0; k < D / 16; ++k) {
                        uint32_t x[16];
                        tmem_ld_x16(to + k * 16u, x);
                        tmem_ld_wait();
                        if (k == D / 16 - 1) {                 // O is read
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) cluster_arrive(of_first(&c.o_free));
                        }
                        if (!in) continue;
                        if (whole) {
#pragma unroll
                            for (int i = 0; i < 16; i += 2)
                                x[i >> 1] = to_half2(__uint_as_float(x[i]) * f, __uint_as_float(x[i + 1]) * f);
                            store32(dst + 32 * k, x, out_32);
                        } else {
                            store32(dst + 64 * k, x, true);
                            store32(dst + 64 * k + 32, x + 8, true);
                        }
                    }
                } else if (lane == 0) {
                    cluster_arrive(of_first(&c.o_free));
                }
                __syncwarp();
            }
        };
        auto load_q = [&](uint32_t number) {
            const uint32_t qb = Sh::QBUFS == 2 ? number & 1u : 0u, quse = Sh::QBUFS == 2 ? number >> 1 : number;   // buffer, its uses before
            if (ok && quse > 0) ok = warp_wait(&c.q_free[qb], (quse - 1) & 1u, abort, span(before));
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
            }
        };
        auto q_loaded = [&](uint32_t number) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (ok) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) cluster_arrive(of_first(&c.q_full[Sh::QBUFS == 2 ? number & 1u : 0u]));
            }
        };
        // Rows of V that nothing attends may hold anything (the ends of loaded pages):
        // zero weights must meet zeros.  r0: the segment's first slot.
        auto clear = [&](const Seg &x, uint32_t r0, int32_t tile) {
            const int32_t seen = G::BLOCKS ? entry_seen(__ldg(list_of(p, x) + x.j0 + tile)) : 0;
            if (!G::BLOCKS && !x.cut(tile, CH_TILE)) return;
            if (ok) ok = warp_wait(&c.bnd[nb & 7u], (nb >> 3) & 1u, abort, span(x));
            ++nb;
            const uint32_t vs = Sh::OWN_P ? Sh::NK + (r0 + tile) % Sh::NV : (r0 + slot_of_v<Sh::LEAD>(tile, x.n)) % NS;
            if (ok) {
                uint8_t *v = ring + vs * SLOT;
                const int32_t a = G::BLOCKS ? 0 : x.lo_tok - (x.j0 + tile) * CH_TILE;
                const int32_t z = G::BLOCKS ? seen : x.hi_tok + 1 - (x.j0 + tile) * CH_TILE;
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
        };
        if constexpr (Q8) {
            while (next_segment()) {
                const int32_t n = w.n;
                load_q(seg);
                const int32_t *bt = p.kv.block_table + static_cast<int64_t>(w.b) * p.kv.max_pages;
                // Scale bytes of the slot's tokens, one per thread, looked up ahead:
                // the page two tiles, the byte one.  Keys and values have their own,
                // so that nothing depends on the order of the slots (with one chain
                // over both, finding tile and kind of the slot two ahead cost 600
                // clocks a slot, next to 950 for the codes).
                const int32_t tok_v = w.j0 * CH_TILE + ht, tok_k = tok_v + rank * Sh::KTOK;
                const int32_t *list = G::BLOCKS ? list_of(p, w) + w.j0 : nullptr;
                auto entry_of = [&](int32_t tile) -> int32_t { return G::BLOCKS && tile < n ? __ldg(list + tile) : NO_BLOCK; };
                auto page_of = [&](auto is_v, int32_t tile, int32_t ent) -> int32_t {
                    constexpr bool V = decltype(is_v)::value;
                    if constexpr (G::BLOCKS) {
                        const int32_t off = V ? ht : ht + rank * Sh::KTOK;
                        const int32_t at = (entry_block(ent) * CH_TILE + off) >> p.kv.page_shift;
                        return (V || ht < Sh::KTOK) && off < entry_seen(ent) && at < p.kv.max_pages ? __ldg(bt + at) : -1;
                    }
                    const int32_t tok = (V ? tok_v : tok_k) + tile * CH_TILE;
                    const bool seen = (V || ht < Sh::KTOK) && tile < n && tok >= w.lo_tok && tok <= w.hi_tok;
                    return seen ? __ldg(bt + (tok >> p.kv.page_shift)) : -1;
                };
                auto byte_of = [&](auto is_v, int32_t tile, int32_t page, int32_t ent) -> uint32_t {
                    constexpr bool V = decltype(is_v)::value;
                    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.kv.num_pages)) return 127u;
                    const int32_t tok = G::BLOCKS ? entry_block(ent) * CH_TILE + (V ? ht : ht + rank * Sh::KTOK)
                                                  : (V ? tok_v : tok_k) + tile * CH_TILE;
                    const int32_t at = (page << p.kv.page_shift) + (tok & (p.kv.page_tokens - 1));
                    return __ldg((V ? p.kv.v_scale : p.kv.k_scale) + (static_cast<int64_t>(at) * p.kv.hkv + w.g));
                };
                // list entries of the tile at hand, the next and the one after
                int32_t ent_v = entry_of(0), ent1_k = entry_of(1), ent1_v = ent1_k, ent2_k = entry_of(2), ent2_v = ent2_k;
                uint32_t byte_k = byte_of(std::false_type{}, 0, page_of(std::false_type{}, 0, ent_v), ent_v);
                uint32_t byte_v = byte_of(std::true_type{}, 0, page_of(std::true_type{}, 0, ent_v), ent_v);
                int32_t page_k = page_of(std::false_type{}, 1, ent1_k), page_v = page_of(std::true_type{}, 1, ent1_k);
                auto turn = [&](auto is_v, int32_t tile) {
                    constexpr bool V = decltype(is_v)::value;
                    uint32_t &byte = V ? byte_v : byte_k;
                    int32_t &page = V ? page_v : page_k;
                    // 2^(byte - 127) as FP16 (2^-15 is subnormal), twice
                    const int x = max(112, min(135, static_cast<int>(byte))) - 127;
                    c.scale[par][ht] = (x >= -14 ? (x + 15) << 10 : 0x200) * 0x10001u;
                    byte = byte_of(is_v, tile + 1, page, V ? ent1_v : ent1_k);  // in flight until the next tile
                    page = page_of(is_v, tile + 2, V ? ent2_v : ent2_k);
                    const int32_t seen = entry_seen(ent_v);    // (V)
                    if (G::BLOCKS) {
                        if (V) ent_v = ent1_v;
                        (V ? ent1_v : ent1_k) = V ? ent2_v : ent2_k;
                        (V ? ent2_v : ent2_k) = entry_of(tile + 3);
                    }
                    const uint32_t slot = pos.slot(V);
                    if (ok)
                        ok = __all_sync(0xffffffffu, mbar_wait(&c.raw_full[rslot], rphase, abort, lim) &&
                                                         mbar_wait(&c.empty[slot], pos.phase(V) ^ 1u, abort, lim));
                    named_barrier(BAR_HELP, 32 * CH_HELPERS);          // the scales are in
                    if (ok) {
                        // V: rows outside lo_tok .. hi_tok are cleared
                        const int32_t tok0 = (w.j0 + tile) * CH_TILE, a = G::BLOCKS ? 0 : w.lo_tok - tok0,
                                      z = G::BLOCKS ? seen : w.hi_tok + 1 - tok0;
                        codes_to_half<D, V>(raw + rslot * RAW, ring + slot * SLOT, c.scale[par], ht, V ? a : 0, V ? z : Sh::KTOK);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&c.raw_empty[rslot]);
                            cluster_arrive(of_first(&c.full[slot]));
                        }
                    }
                    par ^= 1u;
                    pos.next(V);
                    if (++rslot == G::RAWS) {
                        rslot = 0;
                        rphase ^= 1u;
                    }
                };
                const int32_t lead = min(Sh::LEAD, n);                 // the order of slots
                for (int32_t j = -lead; j < n; ++j) {
                    if (j >= 0) turn(std::true_type{}, j);
                    if (j + lead < n) turn(std::false_type{}, j + lead);
                    if (j == -lead) q_loaded(seg);         // landed under the first codes
                }
                ++seg;
            }
        } else {
            // a segment's cut tiles but the first one: the last tile may be cut, of a list
            // any (in order those are the last three, but see NO_BLOCK)
            auto clear_rest = [&](const Seg &x, uint32_t r0) {
                if constexpr (G::BLOCKS) {
                    const int32_t *list = list_of(p, x) + x.j0;
                    for (int32_t j0 = 0; j0 < x.n; j0 += 32) {
                        const int32_t j = j0 + lane;
                        uint32_t cut = __ballot_sync(0xffffffffu, j > 0 && j < x.n && entry_seen(__ldg(list + min(j, x.n - 1))) < CH_TILE);
                        for (; cut; cut &= cut - 1) clear(x, r0, j0 + __ffs(cut) - 1);
                    }
                } else if (x.n > 1) {
                    clear(x, r0, x.n - 1);
                }
            };
            while (true) {
                const bool more = next_segment();
                if (more) {
                    load_q(seg);
                    q_loaded(seg);
                }
                // with two buffers the next queries are loaded before the last value
                // tile of a segment, which comes late
                if (Sh::QBUFS == 2) clear_rest(before, ring_b);
                write_out();
                if (!more) break;
                before = w;
                ++seg;
                ring_b = ring0;
                ring0 = Sh::OWN_P ? (ring0 + w.n) % Sh::NV : (ring0 + 2 * w.n) % NS;
                if (!G::BLOCKS || entry_seen(__ldg(list_of(p, w) + w.j0)) < CH_TILE) clear(w, ring_b, 0);
                if (Sh::QBUFS == 1) clear_rest(w, ring_b);
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
        const float cs = p.scale * LOG2_E;
        const uint32_t p_full0 = of_first(&c.p_full[grp][0]), s_free0 = of_first(&c.s_free[grp]);
        // A weight is 2^(s cs + level(m)), m the maximum in use: one fused product-sum.
        // The level is rounded once, and what was summed at another one is scaled by
        // the difference of the two rounded levels, so that the rounding (up to one
        // power of two where m cs is 2^23) drops out of the result.  Rounded down, so
        // that no weight is above 2^15; up to m cs = 2^28 the largest is above 2^-9,
        // so FP16 holds it.  (With s - m first, right at any size, the four prompts took
        // 397 us where this takes 389, and 512 new tokens of four requests over 16,384
        // from the E4M3 cache with 128-wide heads 583 where this takes 521.)
        auto level = [&](float m) { return m == -INFINITY ? P_UP : __fmaf_rd(-m, cs, P_UP); };
        uint32_t it = 0, seg = 0;                              // tiles before the segment, segments
        // Waits until the second product of tile i is done.  A parity wait is right
        // while the barrier is in that phase or just past it.  Past the one
        // before: the product of tile i - 1 has been seen to end, and products end
        // in order.  Not past the one after: the product of tile i + 2 needs this
        // warp's own P of tile i + 1 or i + 2, which it has still to give.
        auto o_done = [&](uint32_t i) { return warp_wait(&c.o_done[i & 1u], (i >> 1) & 1u, abort, lim); };
        bool ok = true;                                        // false: keep to the barriers, do nothing
        bool zeros = false;                                    // the group's P holds zeros
        while (next_segment()) {
            const int32_t n = w.n;
            // rows past the unit's last behave like it (their queries are zeros)
            const int32_t mine = w.rows - rank * CH_HALF;      // rows in use here, if positive
            const int32_t vr = w.v0 + min(rank * CH_HALF + row, w.rows - 1);
            const int32_t tok = by_group(p, vr), pos = w.p0 + tok;
            const int32_t first = p.window > 0 ? max(0, pos - p.window + 1) : 0;
            const bool live = lq * 32 < mine;                  // some row of this warp is in use
            // tokens that all rows of the warp see
            const int32_t w_hi = __shfl_sync(0xffffffffu, pos, 0), w_lo = __shfl_sync(0xffffffffu, first, 31);
            const int32_t *list = G::BLOCKS ? list_of(p, w) + w.j0 : nullptr;
            const uint32_t *bits = G::BLOCKS ? bits_of(p, w, tok) : nullptr;
            // a list's entry and bits of the next tile, a tile ahead
            const int32_t jf = (grp - it) & 1, jl = min(jf, n - 1);
            int32_t ent_next = G::BLOCKS ? __ldg(list + jl) : 0;
            uint32_t word_next = G::BLOCKS ? __ldg(bits + ((w.j0 + jl) >> 5)) : 0u;
            float cm = 0.0f, l = 0.0f;                         // the sum, and the constant of its exponents
            for (int32_t j = jf; ok && j < n; j += 2) {
                const uint32_t i = it + j;                     // tile i & 1 == grp
                ok = warp_wait(&c.s_full[grp], (i >> 1) & 1u, abort, lim);
                const int32_t base = (G::BLOCKS ? entry_block(ent_next) : w.j0 + j) * CH_TILE;
                // whether the row attends the tile, and some row of the warp does
                const bool att = !G::BLOCKS || ((word_next >> ((w.j0 + j) & 31)) & 1u);
                const bool some = !G::BLOCKS || __any_sync(0xffffffffu, att);
                if constexpr (G::BLOCKS) {
                    const int32_t ahead = min(j + 2, n - 1);
                    ent_next = __ldg(list + ahead);
                    word_next = __ldg(bits + ((w.j0 + ahead) >> 5));
                }
                const bool load = ok && live && some;
                uint32_t s[4][32];
                float a[4];
                if (load) {
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k) a[k] = tmem_ld_max_x32(ts + k * 32u, s[k]);
                }
                // while the scores come: the maximum in use at the tile before, and
                // P's columns, free when the tile before last is done with them
                if (ok && i > 0) ok = warp_wait(&c.m_out[grp ^ 1][lq], ((i - 1) >> 1) & 1u, abort, lim);
                const float mp = j > 0 ? c.mrow[grp ^ 1][row] : -INFINITY;
                if (ok && i > 1) ok = o_done(i - 2);
                float mx = -INFINITY;
                if (load) {
                    tmem_ld_wait();
                    mx = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
                }
                if constexpr (Sh::OWN_P) {
                    tc_fence_before();
                    __syncwarp();
                    if (ok && lane == 0) cluster_arrive(s_free0);
                }
                if (load && (base + CH_TILE - 1 > w_hi || base < w_lo)) {
                    const int32_t hi = att ? pos - base : -1, lo = first - base;   // visible: lo <= column <= hi
#pragma unroll
                    for (int k = 0; k < 4; ++k) a[k] = -INFINITY;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        // bits of the visible columns (a shift past 31 gives zero)
                        uint32_t below, from;
                        asm("shl.b32 %0, 2, %1;" : "=r"(below) : "r"(min(max(hi - 32 * k, -1), 31) & 31));
                        below = hi < 32 * k ? 0u : below - 1u;
                        asm("shl.b32 %0, 0xffffffff, %1;" : "=r"(from) : "r"(max(lo - 32 * k, 0)));
                        const uint32_t bits = below & from;
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            if (!(bits & (1u << e))) s[k][e] = 0xff800000u;              // -inf
                            a[e & 3] = fmaxf(a[e & 3], __uint_as_float(s[k][e]));
                        }
                    }
                    mx = fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
                }
                if (!att) mx = -INFINITY;
                const bool grow = (mx - mp) * cs > RESCALE;
                const float mi = grow ? mx : mp;
                c.mrow[grp][row] = mi;                         // the maximum in use at this tile
                __syncwarp();
                if (lane == 0) mbar_arrive(&c.m_out[grp][lq]);
                tc_fence_after();
                if (ok && live && j > 0 && __any_sync(0xffffffffu, grow)) {
                    // only here the product before must have ended
                    ok = o_done(i - 1);
                    tc_fence_after();
                    const float alpha = grow ? exp2_approx(fminf(level(mi) - level(mp), 0.0f)) : 1.0f;
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
                // P, in two halves; the products of the first start at once
                auto give = [&](int half) {
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (ok && lane == 0) cluster_arrive(p_full0 + half * 8u);
                };
                if (ok && live && !some) {
                    // P beside S may hold zeros already
                    if (!Sh::OWN_P || !zeros) {
                        uint32_t o[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = 0u;
#pragma unroll
                        for (int k = 0; k < 4; ++k) tmem_st_x16(tp + k * 16u, o);
                    }
                    zeros = true;
                    give(0);
                }
                if (ok && live && some) {
                    zeros = false;
                    const float cn = level(mi);
                    if (cn != cm) l *= exp2_approx(fminf(cn - cm, 0.0f));      // (0 at the first)
                    cm = cn;
                    float2 sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
                    // (the scores of a tile that the row does not attend are finite, or masked)
                    const float ce = att ? cm : -INFINITY;
                    const float2 c2 = make_float2(cs, cs), cm2 = make_float2(ce, ce);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t o[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 y = fma2(make_float2(__uint_as_float(s[k][2 * e]), __uint_as_float(s[k][2 * e + 1])), c2, cm2);
                            const float2 z = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                            sum[e & 1] = add2(sum[e & 1], z);
                            const __half2 h = __floats2half2_rn(z.x, z.y);
                            o[e] = *reinterpret_cast<const uint32_t *>(&h);
                        }
                        // (by now the first half's stores are done: no wait for them)
                        if (k == 2) give(0);
                        tmem_st_x16(tp + k * 16u, o);
                    }
                    l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
                }
                if (!live) give(0);
                give(1);
            }
            it += n;
            if constexpr (Sh::HELP_OUT) {
                // The segment's sums.  The group that has the last tile adds up both and
                // hands the helpers what the output is multiplied by; the other goes on
                // at once.  (That one waits for the last tile's maximum, which its next
                // tile would wait for, so the sum before has been read.  With all eight
                // warps meeting at named barriers a unit's end took them 3,400 clocks; the
                // calls' times are the same, for the second products wait for the helpers'
                // reading of the output as long.)
                const bool ends = ((it - 1) & 1u) == static_cast<uint32_t>(grp);
                if (!ends && ok) ok = warp_wait(&c.m_out[grp ^ 1][lq], ((it - 1) >> 1) & 1u, abort, lim);
                const float mlast = c.mrow[(it - 1) & 1u][row], clast = level(mlast);
                l = l > 0.0f ? l * exp2_approx(fminf(clast - cm, 0.0f)) : 0.0f;
                if (!ends) {
                    c.lrow[row] = l;
                    __syncwarp();
                    if (ok && lane == 0) mbar_arrive(&c.l_out[lq]);
                } else {
                    if (ok) ok = warp_wait(&c.l_out[lq], seg & 1u, abort, lim);
                    l += c.lrow[row];
                    if (row < mine && w.place >= 0)
                        *reinterpret_cast<float2 *>(p.ws + WS_ML + (static_cast<int64_t>(w.place) * CH_ROWS + rank * CH_HALF + row) * 8) =
                            make_float2(mlast == -INFINITY ? -INFINITY : -clast, l);
                    if (ok && seg > 0) ok = warp_wait(&c.f_free, (seg - 1) & 1u, abort, lim);
                    if (ok) c.factor[row] = w.place >= 0 ? 1.0f : l > 0.0f ? 1.0f / l : 0.0f;
                    __syncwarp();
                    if (ok && lane == 0) mbar_arrive(&c.f_full);
                }
                ++seg;
                continue;
            }
            // the segment's sums: its rows' output, or its part of it
            if (ok) ok = (it < 2 || o_done(it - 2)) && o_done(it - 1);
            named_barrier(BAR_PAIR + lq, 64);
            // both groups' sums at the last tile's maximum, exchanged in place of the maxima
            const float mlast = c.mrow[(it - 1) & 1u][row];
            const float clast = level(mlast);
            l = l > 0.0f ? l * exp2_approx(fminf(clast - cm, 0.0f)) : 0.0f;
            named_barrier(BAR_PAIR + lq, 64);
            c.mrow[grp][row] = l;
            named_barrier(BAR_PAIR + lq, 64);
            l += c.mrow[grp ^ 1][row];
            if (grp == 0 && row < mine && w.place >= 0)
                *reinterpret_cast<float2 *>(p.ws + WS_ML + (static_cast<int64_t>(w.place) * CH_ROWS + rank * CH_HALF + row) * 8) =
                    make_float2(mlast == -INFINITY ? -INFINITY : -clast, l);
            const float inv = w.place >= 0 ? 1.0f : l > 0.0f ? 1.0f / l : 0.0f;
            if (ok && live) {
                tc_fence_after();
                const uint32_t to = tmem + TM_O + lane_base + grp * OC;
                const bool in = row < mine, whole = w.place < 0;
                const int32_t h = vr - tok * p.group, ur = rank * CH_HALF + row;
                __half *out = static_cast<__half *>(p.out) +
                              ((static_cast<int64_t>(w.s0) + tok) * p.hq + w.g * p.group + h) * D + grp * OC;
                const bool out_32 = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;      // (16 bytes are promised)
                float *part = reinterpret_cast<float *>(p.ws + ws_o<CH_ROWS, CHUNK_MAX_PAIRS>()) +
                              (static_cast<int64_t>(w.place) * p.ws_rows + ur) * D + grp * OC;
                // rolled: a unit's end is code that has left the instruction cache
#pragma unroll 1
                for (int k = 0; k < OC / 32; ++k) {
                    uint32_t u[32];
                    tmem_ld_32x32b_x32(to + k * 32u, u);
                    tmem_ld_wait();
                    if (!in) continue;
                    if (whole) {
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            u[i >> 1] = to_half2(__uint_as_float(u[i]) * inv, __uint_as_float(u[i + 1]) * inv);
                        store32(out + 32 * k, u, out_32);
                        store32(out + 32 * k + 16, u + 8, out_32);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; i += 8) store32(part + 32 * k + i, u + i, true);
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
    if (t == 0 && *abort) tell_other(&c.abort, rank ^ 1, 1u);
    __syncwarp();
    cluster_sync();                                          // nothing of the pair reaches into the other any more
    // the last commits have arrived in the first CTA; here, too
    if (rank == 1 && t == 0)
        for (int i = 0; i < (Sh::OWN_P ? 2 : 1); ++i) mbar_wait_bounded(&c.drain[i], 0, DRAIN_NS);
    __syncwarp();
    if (*abort) {
        // After a time-out in either CTA, copies may be in flight that complete on the
        // other one's barriers, whatever became of the loader itself.  Every role of
        // both has joined, so nothing new is issued: they get the time (they land
        // within microseconds).
        if (t == CH_LOAD * 32) {
            const long long t0 = clock64();
            while (clock64() - t0 < static_cast<long long>(2 * DRAIN_NS)) {}
        }
        __syncwarp();
        __syncthreads();
        cluster_sync();
    }
    tc_fence_after();
    if (t == 0 && c.abort) record_error(p.kv.status, ST_TIMEOUT);
    if (warp == CH_MMA)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

constexpr size_t CH_SMEM = RING + sizeof(Ctrl);
static_assert(CH_SMEM <= 232448, "shared memory budget");

// after_lists: the kernel waits on the device for the one before it in the stream,
// which makes the lists of blocks.
template <int D, bool Q8, typename G>
int launch_pairs(const ChunkParams &p, const void *tk, const void *tv, int grid, bool overlap, bool after_lists, cudaStream_t stream)
{
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return static_cast<int>(cudaErrorInvalidDevice);
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!done[dev]) {
            const cudaError_t e = cudaFuncSetAttribute(chunk_kernel<D, Q8, G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       static_cast<int>(CH_SMEM));
            if (e != cudaSuccess) return static_cast<int>(e);
            done[dev] = true;
        }
    }
    void *args[] = {const_cast<void *>(tk), const_cast<void *>(tv), const_cast<ChunkParams *>(&p)};
    const int rc = launch_kernel(reinterpret_cast<const void *>(&chunk_kernel<D, Q8, G>), dim3(grid), dim3(CH_THREADS),
                                 CH_SMEM, stream, after_lists && overlap, args);
    if (rc != 0) return rc;
    void *join[] = {const_cast<ChunkParams *>(&p)};
    const unsigned y = static_cast<unsigned>(std::min(CH_ROWS / JOIN_WARPS, p.ws_rows));
    return launch_kernel(reinterpret_cast<const void *>(&chunk_join_kernel<G, D>), dim3(grid / 2, y), dim3(256), 0, stream,
                         overlap, join);
}

// As many pairs as the workspace has places for.
inline int pairs_grid(int sms) { return 2 * std::min(sms / 2, static_cast<int>(CHUNK_MAX_PAIRS)); }

template <typename G>
int launch_pairs_for(const ChunkParams &p, const void *tk, const void *tv, int sms, bool overlap, bool after_lists, cudaStream_t s)
{
    const int grid = pairs_grid(sms);
    if (p.kv.head_dim == 128)
        return p.kv.e4m3 ? launch_pairs<128, true, G>(p, tk, tv, grid, overlap, after_lists, s)
                         : launch_pairs<128, false, G>(p, tk, tv, grid, overlap, after_lists, s);
    return p.kv.e4m3 ? launch_pairs<256, true, G>(p, tk, tv, grid, overlap, after_lists, s)
                     : launch_pairs<256, false, G>(p, tk, tv, grid, overlap, after_lists, s);
}

}  // namespace
}  // namespace qsa
