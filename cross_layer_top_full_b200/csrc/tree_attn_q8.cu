// tree_attn_q8.cu -- attention of a tree of drafted tokens over the quantised
// paged cache (see include/indexcache.h) on the tcgen05 tensor cores.
//
// Row (b, i), head h, over the seen positions s (before the tree, or a node of
// the row's mask; restricted to idx[b,i,:] where it is given), with g_s the
// cache row's scale and c_s its 576 scaled values:
//   p = softmax_s(scale * g_s (q . c_s)),  out = sum_s (p_s g_s) c_s[0:512].
//
// The cache's codes go into the products as they are; nothing is decoded.
//   Q K^T: a query value has 8 significant bits, an e4m3 number 4, so with a
//     power-of-two scale per row q = hi + lo exactly, two e4m3 numbers (lo's
//     floor is 2^-18 of the row's largest value).  The 64 columns that the
//     cache keeps as bfloat16 follow in the same accumulator: both operands
//     carry the same scales there.
//   P V: the weights w_s = p_s g_s go in as an e4m3 number and an e5m2 number
//     for the rest.  The running maximum is that of log2 w_s, which keeps w in
//     8-bit range whatever the scales are; the row's largest weight stands
//     between 2^4 and 2^8.5.  Weights of 2 or more are off by at most 2^-8 of
//     themselves, as in bfloat16.  Smaller ones may be very many and all alike:
//     to the nearest, with the largest weight at 2^2, 65,536 of them at 2^-19.1
//     of it (a tenth of the sum) all became 0, and at 2^-17 were off by an
//     eighth, all the same way.  So they are rounded up or down at random, right
//     on average, and of n errors the root of n of them is left: by at most 2^-7
//     of themselves down to 2^-6, then a step of 2^-13, of a quarter of the
//     weight under 2^-11, of 2^-16 at last.  That costs 1.5 %, the largest weight
//     at 2^4 instead of 2^2 (two more bits for the others, more maxima that
//     outgrow their room) another 2 %: 128 lists of 2048 over the same inputs,
//     82.7, 84.1, 85.9 us; with 2^6 89.3.  The softmax sum adds w_s / g_s in float32, before that
//     rounding.
// Two 8-bit products cost what one of bfloat16 does, without the decoding and
// with 644 bytes of cache traffic per row.
//
// A unit is 128 query rows that read the same positions: the heads of one row
// (idx given), or 128 consecutive (node, head) pairs of a sequence.  The
// units' blocks of 128 positions are shared out among the CTA pairs (see
// below); where a pair's run ends inside a unit, it leaves a float32 partial
// result and a second kernel joins them.
//
// What bounds it: the tensor core.  A block costs a pair 3,000 cycles of MMAs
// by themselves (Q K^T 1,850: 36 MMAs with N = 128, which the operand reads
// hold to 60 % of their rate; P V 1,060 at the full rate); blocks in a row
// take 2,800 to 2,900, the two products overlapping.  A unit costs 18,000
// cycles besides, for Q, the first block's latency and the results.
// 128 lists of 2048 (73 GFLOP): 102 us; 8 sequences of up to 8192 with 16 nodes,
// every position (159 GFLOP): 173 us; 32 lists: 38.5 us; one list: 17.5 us (a
// pass among others, other inputs each; over the same inputs again, as the steps
// below were compared, 88, 150 to 160, 36.3 and 17.7).
// Steps that did not help: four-row TMA gathers (about 65 cycles each, 112 a
// block, against 36 cp.async a warp), a wait of the copies' arrival by the MMA
// warp with its proxy fence there, releases at cluster scope for the arrivals
// from the other CTA (2,000 cycles each), 64-bit run arithmetic and fully
// unrolled code (the instruction fetch), query rows kept in registers over the
// end of a unit (spills: 96 -> 106 us).
//
// A pair works on one unit at a time: each CTA holds 64 of the rows, gathers
// 64 of the block's 128 keys whole (for Q K^T) and half of the value columns
// of all 128 (for P V): an M = 128 product of a pair takes its B operand in
// two halves, split by keys for the one and by columns for the other.
//   warps 0-15  softmax, two groups of eight that take the blocks in turn (each
//               with an S buffer each; thread = row x 32 keys), conversion of
//               Q, epilogue
//   warps 16-19 copy the block's rows: two K, two V, 16 bytes a lane
//               (cp.async, 128 adjacent bytes per row and eight lanes; a row
//               that nobody may see is filled with zeros), or one TMA box per
//               64 rows where a block is 128 consecutive rows; the V warps
//               look for rows of zeros and unusual scales first
//   warps 20-21 resolve positions to cache rows, scales and masks, a block
//               each in turn, ahead of the copies (a ring of three blocks)
//   warps 22-23 rank 0: issue the MMAs, 22 Q K^T as soon as a block's K is there
//               and its S buffer read, 23 P V as soon as P and V are; rank 1:
//               pass on that its own tiles have landed
// Tensor memory, all of it: O 256 columns, two S buffers of 64, three of Q's
// eight 8-bit slices and its bfloat16 columns 32 each.  Shared memory: five
// slices of Q 40 KB, K 2 x 40 KB, V 2 x 32 KB, P 2 x 16 KB, the ring 6 KB.
//
// A barrier tells only its last two phases apart.  So each wait here is for a
// phase whose predecessor is known to be over (the waiter has seen it, or what
// it has seen implies it) and whose successor cannot end before the waiter has
// gone on.
//
// Every wait is bounded (sm100.cuh); sites: 1-3 copies, 4-9 and 19 softmax,
// 10-15 and 20 MMA issue, 16 resolution.
#include <cudaTypedefs.h>

#include <algorithm>

#include "q8.cuh"
#include "sm100.cuh"

namespace ic {
namespace {

using namespace q8;
using namespace sm100;

constexpr int MROWS = 128, HROWS = 64;        // query rows of a unit, of a CTA
constexpr int NB = 128;                       // positions per block
constexpr int ATOM = 64 * 128;                // 64 rows of 128 bytes
constexpr int Q_SMEM = 5;                     // slices of Q in shared memory: hi 0-3, lo 0; the rest: TM_Q
constexpr int K_STAGE = 5 * ATOM, V_STAGE = 4 * ATOM, P_STAGE = 2 * ATOM;
constexpr int OFF_Q = 0;
constexpr int OFF_K = OFF_Q + Q_SMEM * ATOM;
constexpr int OFF_V = OFF_K + 2 * K_STAGE;
constexpr int OFF_P = OFF_V + 2 * V_STAGE;
constexpr int RING = 3;
struct Info {                                 // one block, resolved
    int rows[NB];                             // cache rows, -1: seen by nobody
    float scale[NB], lg[NB], inv[NB];         // scales, their log2 and inverse
    uint32_t seen[NB / 32];                   // bit: not -1
    int box;                                  // 128 consecutive cache rows from rows[0] on
    int pad[3];
};
constexpr int OFF_INFO = OFF_P + 2 * P_STAGE;
constexpr int OFF_XM = OFF_INFO + RING * (int)sizeof(Info);   // [2 groups][4][64] float: row maxima
constexpr int OFF_XL = OFF_XM;                        // [8][64] float: row sums, between units
constexpr int OFF_MR = OFF_XM + 2 * 4 * HROWS * 4;    // [2][64] float: running maxima after a block
constexpr int OFF_SQ = OFF_MR + 2 * HROWS * 4;        // [64] float: scales of Q's rows
constexpr int OFF_BARS = OFF_SQ + HROWS * 4;
constexpr int GROUP_WARPS = 8, SOFT_WARPS = 16, W_COPY = 16, W_RES = 20, W_S = 22;
constexpr int THREADS = 32 * 24;
constexpr uint32_t TM_O = 0, TM_S = 256, TM_Q = 384, TM_QR = TM_Q + 96;   // TM_Q: lo 1-3, the bfloat16 columns
constexpr int TMEM_COLS = 512;
constexpr int MAX_PAIRS = 74;                 // CTA pairs of 148 SMs
constexpr float LOG2E = 1.4426950408889634f;
constexpr float TOP = 4.f, SLACK = 4.5f;       // log2 of the largest weight when the maximum is
                                              // set, and how far it may grow before O is rescaled

struct __align__(8) Bars {
    uint64_t info_full[RING];        // positions, scales and masks of a block are there
    uint64_t scale_full[RING];       // and weigh_scales is through (both V warps)
    uint64_t info_free[2 * RING];    // block j % 6 has been used: always waited for by the same warp
    uint64_t q_full;                 // rank 0: Q of a unit is in place (both CTAs' warps)
    uint64_t k_full[2], v_full[2];   // own tiles have landed
    uint64_t k_peer[2], v_peer[2];   // rank 0: rank 1's tiles have landed
    uint64_t s_full[2];              // S of a block is complete: K stage free
    uint64_t s_free[2];              // rank 0: S of a block has been read (both CTAs' warps)
    uint64_t p_full[2];              // rank 0: P of a block is in place (both CTAs' warps)
    uint64_t pv_done[2];             // P V of a block is complete: V stage, P stage free
    uint64_t drain[2];
    uint32_t tmem_base;
    int abort;
    int start_b, start_u, start_t, left;
};
constexpr size_t SMEM_BYTES = 1008 + OFF_BARS + sizeof(Bars);
static_assert(SMEM_BYTES <= 232448 && OFF_BARS % 8 == 0, "shared memory budget");

struct Args {
    const __nv_bfloat16* q;
    const uint8_t* cache;
    const float* kv_scale;
    const int32_t* idx;
    const unsigned long long* tree;
    const int32_t* seq_lens;
    const int32_t* block_table;
    __nv_bfloat16* out;
    uint4* part_o;      // [2 * pairs][PART]: float32, in the order of the threads that hold them
    float2* part_ml;    // [2 * pairs][128]: running maximum, sum
    int4* joins;        // [pairs]: the unit that ends in the pair's run and began before it: its first
                        // query row (64 bits), rows, first pair (rows 0: there is none)
    uint32_t* status;
    int k, B, Lq, Hq, T_max, max_pages, page_size, num_pages;
    int units;          // per sequence
    int list_blocks;    // blocks of a list (idx given)
    int sharing;        // BY_LENGTH without lists
    float scale_log2;
};

// ------------------------------------------------------------------ the list of blocks
__device__ __forceinline__ int seq_len(const Args& a, int b) {
    const int len = __ldg(a.seq_lens + b);
    return len < a.Lq || len > a.T_max ? 0 : len;
}
__device__ __forceinline__ int blocks_of(const Args& a, int b) {
    return a.idx ? a.list_blocks : max(1, (seq_len(a, b) + NB - 1) / NB);
}

// All blocks of the call (one warp); the host has made sure that they fit.
__device__ __forceinline__ int total_blocks(const Args& a) {
    if (a.idx) return a.B * a.units * a.list_blocks;
    int n = 0;
#pragma unroll 8
    for (int b = threadIdx.x & 31; b < a.B; b += 32) n += blocks_of(a, b);
    return __reduce_add_sync(0xffffffffu, n) * a.units;
}

// How the blocks are shared out among P pairs.  In blocks' time (2,850 cycles)
// a unit costs a run about UNIT_COST (18,000 cycles for Q, the first block's
// latency and the results), and joining partial results JOIN_COST (up to 10 us
// of a second kernel).  Three ways:
//   WHOLE  the units, whole, in equal shares (nothing to join)
//   PARTS  each unit over parts_of() pairs, in proportion to its blocks; a pair
//          has one unit
//   RUNS   the list of all units' costs in equal runs, over the units' borders
// Lists are all of one length: the host takes the cheapest.  With every
// position the lengths are known on the device, which decides between PARTS
// and RUNS.  Measured: 32 lists of 2048 (16 blocks), PARTS 36 us, RUNS 44; 128
// lists, WHOLE 94, RUNS 108 (in the same run); 8 sequences of up to 8192 in RUNS of equal blocks
// 183, of equal cost 170.  Costs of 3 and 4 instead: 40 lists 50 us (in RUNS)
// against 43 (WHOLE).
enum { WHOLE, PARTS, RUNS, BY_LENGTH };
constexpr int UNIT_COST = 6, JOIN_COST = 6;
__device__ __forceinline__ int parts_of(const Args& a, int b, int n, int P) { return max(1, blocks_of(a, b) * P / n); }

// Equal shares: n things over P pairs, the first n % P one more.
__device__ __forceinline__ int pairs_of(int n, int max_pairs) { return min(n, max_pairs); }
__device__ __forceinline__ int run_begin(int n, int P, int p) { return n / P * p + min(n % P, p); }
__device__ __forceinline__ int pair_with(int n, int P, int t) {
    const int q = n / P, longer = n % P, at = longer * (q + 1);
    return t < at ? t / (q + 1) : longer + (t - at) / q;
}

// Where place v of the list of shares lies (PARTS: a unit counts as its parts,
// RUNS: as its blocks and UNIT_COST before them): sequence b (a.B: past the
// end), place o from its first, blocks before the sequence.  One warp.
struct Place {
    int b, o, blocks;
};
__device__ __forceinline__ Place locate(const Args& a, int v, bool parts, int n, int P) {
    if (a.idx) {
        const int per = a.units * (parts ? parts_of(a, 0, n, P) : a.list_blocks + UNIT_COST);
        const int b = min(v / per, a.B);
        return {b, v - b * per, b * a.units * a.list_blocks};
    }
    Place r{a.B, v, 0};
#pragma unroll 1
    for (int b0 = 0; b0 < a.B && r.b == a.B; b0 += 32) {
        const int at = b0 + (threadIdx.x & 31), nt = at < a.B ? blocks_of(a, at) : 0;
        const int c = at >= a.B ? 0 : (parts ? parts_of(a, at, n, P) : nt + UNIT_COST) * a.units;
        int x = c, y = nt * a.units;         // inclusive prefix sums
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const int x2 = __shfl_up_sync(0xffffffffu, x, o), y2 = __shfl_up_sync(0xffffffffu, y, o);
            if ((threadIdx.x & 31) >= o) { x += x2; y += y2; }
        }
        const unsigned hit = __ballot_sync(0xffffffffu, r.o < x);
        const int l = hit ? __ffs(hit) - 1 : 31;
        r.o -= __shfl_sync(0xffffffffu, hit ? x - c : x, l);
        r.blocks += __shfl_sync(0xffffffffu, hit ? y - nt * a.units : y, l);
        if (hit) r.b = b0 + l;
    }
    return r;
}

// A walk over a run: unit u of sequence b, from block t on.
struct Walk {
    int b, u, t, nt, left;
    __device__ __forceinline__ void start(const Args& a, const Bars& s) {
        b = s.start_b; u = s.start_u; t = s.start_t; left = s.left;
        nt = left > 0 ? blocks_of(a, b) : 0;
    }
    __device__ __forceinline__ int count() const { return min(left, nt - t); }
    __device__ __forceinline__ void next(const Args& a) {
        left -= count();
        t = 0;
        if (++u == a.units) {
            u = 0;
            ++b;
            if (left > 0) nt = blocks_of(a, b);
        }
    }
};

// Query rows of a unit: first + m for m in [0, rows).
struct Rows {
    int64_t first;
    int rows, node0;      // rows (at most 128); (node, head) index of the first in its sequence
};
__device__ __forceinline__ Rows unit_rows(const Args& a, int b, int u) {
    Rows r;
    if (a.idx) {
        r.node0 = u * a.Hq;
        r.rows = a.Hq;
    } else {
        r.node0 = u * MROWS;
        r.rows = min(MROWS, a.Lq * a.Hq - r.node0);
    }
    r.first = (int64_t)b * a.Lq * a.Hq + r.node0;
    return r;
}

// ------------------------------------------------------------------ small helpers
// Barriers of the softmax warps: of one group, of both, and the handing over of
// the running maxima from the group of a block to that of the next.
__device__ __forceinline__ void group_sync(int g) { asm volatile("bar.sync %0, 256;" ::"r"(1 + g) : "memory"); }
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 3, 512;" ::: "memory"); }
__device__ __forceinline__ void hand_over(int to) { asm volatile("bar.arrive %0, 512;" ::"r"(4 + to) : "memory"); }
__device__ __forceinline__ void take_over(int g) { asm volatile("bar.sync %0, 512;" ::"r"(4 + g) : "memory"); }
__device__ __forceinline__ uint64_t f2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 f2_split(uint64_t v) {
    float a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
    return make_float2(a, b);
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t bf16_pair2(uint64_t v) {
    const float2 f = f2_split(v);
    return bf16_pair(f.x, f.y);
}

// Two e4m3 numbers, and what they leave of (a, b): exactly.
__device__ __forceinline__ void split_weights(float a, float b, uint32_t& hi, float& ra, float& rb) {
    hi = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi, __NV_E4M3);
    asm("{\n\t.reg .b16 m;\n\tmov.b16 m, 0xbc00;\n\t"            // a - hi: hi * -1 + a
        "fma.rn.f32.f16 %0, %2, m, %4;\n\tfma.rn.f32.f16 %1, %3, m, %5;\n\t}"
        : "=f"(ra), "=f"(rb)
        : "h"(h.x), "h"(h.y), "f"(a), "f"(b));
}
// Four rests as e5m2 numbers (the first in the low byte), rounded up or down at
// random: up with the probability that the rest stands above the lower
// neighbour, so that the mean is the rest itself.  Each half of `random` serves
// two values, to the one with its bits in reverse order (measured; 16 bits).
__device__ __forceinline__ uint32_t round_rests(float a, float b, float c, float d, uint32_t random) {
    uint32_t r;
    asm("cvt.rs.satfinite.e5m2x4.f32 %0, {%4, %3, %2, %1}, %5;" : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d), "r"(random));
    return r;
}
constexpr uint32_t NEAREST = 0x80018001u;      // a half step, read from either end
// A number per query row and 32 positions, from which a sequence of them starts
// (multiplicative hashing; the linear congruence of a published table).
__device__ __forceinline__ uint32_t random_start(uint32_t row, uint32_t at) {
    uint32_t x = row * 0x9e3779b9u + at;
    x = (x ^ x >> 16) * 0x9e3779b9u;
    return x ^ x >> 15;
}
__device__ __forceinline__ uint32_t random_next(uint32_t x) { return x * 1664525u + 1013904223u; }
__device__ __forceinline__ float reciprocal(float a) {       // within 2^-23 of itself, subnormal results too
    float d;
    asm("rcp.approx.f32 %0, %1;" : "=f"(d) : "f"(a));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Two scaled query values (a bfloat16 pair) as e4m3 numbers and e4m3 numbers
// for what they leave.  By way of float16, which holds a bfloat16 in [-448,
// 448] down to 2^-24 exactly, as it does the rest.
__device__ __forceinline__ void split_query(uint32_t p, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u));
    hi = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(h), __NV_SATFINITE, __NV_E4M3);
    const __half2 d = __hsub2(h, __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)hi, __NV_E4M3)));
    lo = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(d), __NV_SATFINITE, __NV_E4M3);
}
// A bfloat16 pair times a power of two (a bfloat16 pair of it): exact.
__device__ __forceinline__ uint32_t mul_pair(uint32_t p, uint32_t pow2) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(p), "r"(pow2));
    return r;
}
__device__ __forceinline__ uint32_t twice(float pow2) { return (__float_as_uint(pow2) >> 16) * 0x10001u; }

// Bits of the 32 positions from s0 on that a row sees by its tree mask.
__device__ __forceinline__ uint32_t tree_bits(unsigned long long mask, int off) {   // off = s0 - ctx
    if (off <= -32) return 0xffffffffu;
    if (off >= 0) return off < 64 ? (uint32_t)(mask >> off) : 0u;
    return (uint32_t)(mask << -off) | ((1u << -off) - 1u);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {   // the rest of 16: zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A partial result of a unit: O of one thread (row (warp & 1) * 32 + lane of
// CTA rank) in 16-byte pieces i = 0..7 of 32 columns c = 0..1 from
// part_col(warp, c) on, so that a warp writes and reads 512 adjacent bytes.
constexpr int PART = MROWS * DV / 4;
__host__ __device__ constexpr int64_t part_at(int slot, int rank, int warp, int c, int i, int lane) {
    return (int64_t)slot * PART + ((((rank * 16 + warp) * 2 + c) * 8 + i) * 32 + lane);
}
__device__ __forceinline__ int part_col(int warp, int c) {
    return 256 * (warp >> 3) + 128 * ((warp >> 1) & 1) + 64 * ((warp >> 2) & 1) + 32 * c;
}

// What the resolution leaves of the scales of a block, for 64 of its keys (one
// warp, while it waits for its stage):
//
// A row whose codes are all 0 adds nothing to O, whatever its weight there.  The
// writer gives it the scale 1, far above that of small values: p_s * 1 as its
// weight would set the row's maximum and put the others under the range of 8
// bits.  It gets the weight 2^-NIL p_s instead, below p_s times any scale that the
// writer gives, and the same part in the softmax sum as ever.  Keys of scale 1
// whose first 16 codes are 0 are read whole, up to four at once, eight lanes each.
// A row of zeros with the scale 0 does as well (one that nothing was written to).
// A scale that is no power of two (another rule's) gets its logarithm and inverse.
// One that is no positive normal number makes the logits, and so the rows that
// see the key, NaN; its inverse stays finite, for the sums of the rows that do not.
//
// 128 lists, one row in a thousand zero: 85.0 -> 87.2 us.  (In the warps that
// resolve positions, a load behind the scales: 90; in the softmax warps: 98; in a
// warp of its own, with 72 registers a thread for all: 96; for rows of any scale:
// 97.)  A cache of zeros alone takes three times as long (261 us; one row at a
// time 579).
constexpr int NIL = 40;
__device__ __forceinline__ bool no_codes(uint4 v) { return ((v.x | v.y | v.z | v.w) & 0x7f7f7f7fu) == 0; }
__device__ __forceinline__ void weigh_scales(Info& info, const uint8_t* cache, int key0, int lane) {
#pragma unroll 1
    for (int i = 0; i < 64; i += 32) {
        const int key = key0 + i + lane, row = info.rows[key];
        const float g = info.scale[key];
        const uint32_t u = __float_as_uint(g);
        // a power of two that has an inverse, and not 1: ready
        if (!__any_sync(0xffffffffu, (u & 0x807fffffu) != 0 || u - 0x00800000u >= 0x7e800000u || u == 0x3f800000u)) continue;
        const bool normal = u - 0x00800000u < 0x7f000000u;
        if (normal && ((u & 0x7fffffu) != 0 || u >= 0x7f000000u)) {
            info.lg[key] = (float)((int)(u >> 23) - 127) + __log2f(__uint_as_float((u & 0x7fffffu) | 0x3f800000u));
            info.inv[key] = reciprocal(g);
        }
        bool nil = (u == 0x3f800000u || g == 0.f) && row >= 0;
        if (nil) nil = no_codes(__ldg(reinterpret_cast<const uint4*>(cache + (int64_t)row * ROW)));        // the first 16
        const uint32_t asked = __ballot_sync(0xffffffffu, nil);
#pragma unroll 1
        for (int k = 0; k < 32; k += 4) {                   // 4 rows at once
            if (!((asked >> k) & 0xfu)) continue;
            const int mine = k + lane / 8;
            bool all = true;
            if ((asked >> mine) & 1u) {
                const uint4* p = reinterpret_cast<const uint4*>(cache + (int64_t)info.rows[key0 + i + mine] * ROW) + lane % 8;
#pragma unroll 4
                for (int c = 0; c < 32; c += 8) all = no_codes(__ldg(p + c)) && all;
            }
            const uint32_t yes = __ballot_sync(0xffffffffu, all);
            if (lane >= k && lane < k + 4 && ((yes >> ((lane - k) * 8)) & 0xffu) != 0xffu) nil = false;
        }
        if (nil) {
            info.lg[key] = -(float)NIL;
            info.inv[key] = exp2_int(NIL);
        } else if (!normal) {
            info.scale[key] = __uint_as_float(0x7fffffffu);
            info.inv[key] = 1.f;
        }
    }
}

// A warp's share of a tile: 4 * GROUPS rows (rows[], -1: zeros) of ATOMS x
// 128 bytes, STEP bytes apart in the cache row, DST bytes apart in the tile;
// row0 is the first row's place in the tile.
template <int GROUPS, int ATOMS, int STEP, int DST>
__device__ __forceinline__ void copy_rows(uint32_t dst, int row0, const uint8_t* cache, const int* rows, int lane) {
    int src_row[GROUPS];
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) src_row[g] = rows[g * 4 + (lane >> 3)];
    // rows g and g + 2 are 8 apart: the same place in the swizzle
    const int r = row0 + (lane >> 3);
    const uint32_t d0 = dst + r * 128 + (((lane & 7) ^ (r & 7)) << 4);
    const uint32_t d1 = dst + (r + 4) * 128 + (((lane & 7) ^ ((r + 4) & 7)) << 4);
    cache += (lane & 7) * 16;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
        const uint32_t bytes = src_row[g] >= 0 ? 16u : 0u;
        const uint8_t* src = cache + (int64_t)max(src_row[g], 0) * ROW;
#pragma unroll
        for (int c = 0; c < ATOMS; ++c)
            copy16((g & 1 ? d1 : d0) + (g >> 1) * 1024 + c * DST, src + c * STEP, bytes);
    }
}

// ------------------------------------------------------------------ Q of a unit
// The 64 rows of this CTA, 512 threads: a warp takes 4 rows, a lane 16 of the
// coded columns and 8 of the others.  What goes to tensor memory (lane = row)
// passes through the P tiles, which are free once P V of block j - 1 is
// complete.  A row with an infinity or a NaN in its coded columns becomes NaN as
// a whole (its outputs are); in the others it goes into the logits as it is.
// Returns the scale of this thread's row.
__device__ __forceinline__ float convert_q(const Args& a, const Rows& r, uint8_t* smem, Bars& s, uint32_t rank,
                                           uint32_t tmem, uint32_t lane_base, uint32_t j, uint32_t q_bar) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* sq = reinterpret_cast<float*>(smem + OFF_SQ);
    const __nv_bfloat16* q = a.q + (r.first + rank * HROWS) * KVW;
    const int rows = r.rows - (int)rank * HROWS;
    uint4 v[4][2], rest;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = warp * 4 + i;
        const uint4* p = reinterpret_cast<const uint4*>(q + row * KVW + lane * 16);
        const bool ok = row < rows;
        v[i][0] = ok ? __ldg(p) : make_uint4(0u, 0u, 0u, 0u);
        v[i][1] = ok ? __ldg(p + 1) : make_uint4(0u, 0u, 0u, 0u);
    }
    {
        const int row = warp * 4 + (lane >> 3);
        rest = row < rows ? __ldg(reinterpret_cast<const uint4*>(q + row * KVW + DV) + (lane & 7)) : make_uint4(0u, 0u, 0u, 0u);
    }
    if (j > 0) wait_for(&s.pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, a.status, &s.abort, 8);
#pragma unroll 1                        // little code: it runs once per unit, from a cold instruction cache
    for (int i0 = 0; i0 < 4; i0 += 2) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = warp * 4 + i0 + i;
            const uint32_t u[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w, v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
            uint32_t m = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) m = __vmaxu2(m, u[k] & 0x7fff7fffu);
            m = __reduce_max_sync(0xffffffffu, max(m << 16, m & 0xffff0000u));
            const bool finite = m < 0x7f800000u;
            const int e = finite ? scale_exponent(m) : 0;
            const uint32_t inv = finite ? twice(exp2_int(-e)) : 0x7fff7fffu;
            if (lane == 0) sq[row] = exp2_int(e);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t h0, l0, h1, l1;
                split_query(mul_pair(u[2 * k], inv), h0, l0);
                split_query(mul_pair(u[2 * k + 1], inv), h1, l1);
                hi[k] = h0 | h1 << 16;
                lo[k] = l0 | l1 << 16;
            }
            const int at = row * 128 + (((lane & 7) ^ (row & 7)) << 4);
            *reinterpret_cast<uint4*>(smem + OFF_Q + (lane >> 3) * ATOM + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(smem + (lane < 8 ? OFF_Q + 4 * ATOM : OFF_P + ((lane >> 3) - 1) * ATOM) + at) =
                make_uint4(lo[0], lo[1], lo[2], lo[3]);
            v[i][0] = v[i + 2][0];
            v[i][1] = v[i + 2][1];
        }
    }
    __syncwarp();
    {
        const int row = warp * 4 + (lane >> 3);
        const uint32_t inv = twice(__uint_as_float(0x7f000000u - __float_as_uint(sq[row])));     // 1 / 2^n
        const uint32_t w[4] = {mul_pair(rest.x, inv), mul_pair(rest.y, inv), mul_pair(rest.z, inv), mul_pair(rest.w, inv)};
        *reinterpret_cast<uint4*>(smem + OFF_P + 3 * ATOM + row * 128 + (((lane & 7) ^ (row & 7)) << 4)) =
            make_uint4(w[0], w[1], w[2], w[3]);
    }
    fence_async_smem();
    soft_sync();
    // to tensor memory: warps 4t..4t+3 take tile t
    const int row = (warp & 1) * 32 + lane, tile = warp >> 2;
    uint32_t w[32];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const uint4 x = *reinterpret_cast<const uint4*>(smem + OFF_P + tile * ATOM + row * 128 + ((c ^ (row & 7)) << 4));
        w[4 * c] = x.x; w[4 * c + 1] = x.y; w[4 * c + 2] = x.z; w[4 * c + 3] = x.w;
    }
    tmem_st32(tmem + lane_base + TM_Q + 32 * tile, w);
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_remote_cta(q_bar);
    return sq[row];
}

// Sends for a unit's rows ahead of load_q: thread i of n.
__device__ __forceinline__ void prefetch_q(const Args& a, const Rows& r, uint32_t rank, int i, int n) {
    const int lines = min(HROWS, r.rows - (int)rank * HROWS) * (KVW * 2 / 128);      // 9 lines of 128 bytes a row
    const uint8_t* q = reinterpret_cast<const uint8_t*>(a.q + (r.first + rank * HROWS) * KVW);
    for (; i < lines; i += n)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(q + (int64_t)i * 128));
}

// ------------------------------------------------------------------ the kernel
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
tree_attn_kernel(const __grid_constant__ CUtensorMap map_box,     // box: 64 rows x 128 bytes
                 const __grid_constant__ Args a) {
    extern __shared__ __align__(16) uint8_t raw[];
    uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    Bars& s = *reinterpret_cast<Bars*>(smem + OFF_BARS);
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    volatile int* abort = &s.abort;
    uint32_t* status = a.status;

    if (threadIdx.x == 0) {
        mbar_init(&s.q_full, 2 * SOFT_WARPS);
        for (int i = 0; i < RING; ++i) {
            mbar_init(&s.info_full[i], 1);
            mbar_init(&s.scale_full[i], 2);
            mbar_init(&s.info_free[i], GROUP_WARPS + 4);
            mbar_init(&s.info_free[RING + i], GROUP_WARPS + 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.k_full[i], 2);
            mbar_init(&s.v_full[i], 2);
            mbar_init(&s.k_peer[i], 1);
            mbar_init(&s.v_peer[i], 1);
            mbar_init(&s.p_full[i], 2 * GROUP_WARPS);
            mbar_init(&s.s_free[i], 2 * GROUP_WARPS);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.pv_done[i], 1);
            mbar_init(&s.drain[i], 1);
        }
        s.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&map_box);
    }
    if (warp == W_S) tmem_alloc_pair<TMEM_COLS>(&s.tmem_base);
    pdl_wait();
    if (warp == W_RES) {             // this pair's run
        const int n = total_blocks(a), P = pairs_of(n, gridDim.x / 2), p = blockIdx.x / 2;
        bool parts = a.sharing == PARTS;
        if (a.sharing == BY_LENGTH && a.B * a.units <= P) {
            int used = 0, longest = 0;
            for (int i = lane; i < a.B; i += 32) {
                const int k = parts_of(a, i, n, P);
                used += k;
                longest = max(longest, (blocks_of(a, i) + k - 1) / k);
            }
            used = __reduce_add_sync(0xffffffffu, used) * a.units;
            longest = __reduce_max_sync(0xffffffffu, longest);
            parts = used <= P && longest <= (n + UNIT_COST * a.B * a.units) / P;
        }
        int b = a.B, u = 0, t = 0, left = 0, from = 0;
        bool ends = false;           // the unit that the run begins inside ends in it; `from`: its first pair
        if (a.sharing == WHOLE) {
            const int units = a.B * a.units, P1 = min(units, P), first = run_begin(units, P1, min(p, P1));
            b = first / a.units;
            u = first % a.units;
            left = p < P1 ? (run_begin(units, P1, p + 1) - first) * a.list_blocks : 0;
        } else if (parts) {
            const Place at = locate(a, p, true, n, P);
            b = at.b;
            if (b < a.B) {
                const int nt = blocks_of(a, b), k = parts_of(a, b, n, P), i = at.o % k;
                u = at.o / k;
                t = run_begin(nt, k, i);
                left = run_begin(nt, k, i + 1) - t;
                ends = k > 1 && i == k - 1;
                from = p - i;
            }
        } else if (p < P) {
            const int all = n + UNIT_COST * a.B * a.units;
            int end = n, inside = 0;         // the run's last block + 1; how far into its unit it begins
#pragma unroll 1
            for (int e = 1; e >= 0; --e) {
                const int v = run_begin(all, P, p + e);
                const Place at = locate(a, v, false, n, P);
                if (at.b == a.B) continue;
                const int nt = blocks_of(a, at.b);
                b = at.b;
                u = at.o / (nt + UNIT_COST);
                inside = at.o % (nt + UNIT_COST);
                t = max(0, inside - UNIT_COST);
                const int block = at.blocks + u * nt + t;
                if (e) end = block;
                else {
                    left = end - block;
                    ends = t > 0 && left >= nt - t;
                    if (ends) from = pair_with(all, P, v - inside + UNIT_COST);
                }
            }
        }
        if (left > 0) prefetch_q(a, unit_rows(a, b, u), rank, lane, 32);
        if (lane == 0) {
            s.start_b = min(b, a.B - 1);
            s.start_u = u;
            s.start_t = t;
            s.left = left;
            if (rank == 0) {
                const Rows r = unit_rows(a, s.start_b, u);
                a.joins[p] = make_int4((int)(uint32_t)r.first, (int)(r.first >> 32), ends ? r.rows : 0, from);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    pdl_trigger();
    const uint32_t tmem = 0;             // all of the tensor memory was allocated: it begins at column 0
    Walk w;
    w.start(a, s);

    if (warp < SOFT_WARPS) {
        // ------------------------------------------------ softmax, Q, epilogue
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const int group = warp >> 3;                // takes the blocks j with j & 1 == group
        const int cols = (warp >> 2) & 1;           // which 32 of a buffer's 64 columns
        const int half = (warp >> 1) & 1;           // which 64 of the block's keys
        const int row = (warp & 1) * 32 + lane;
        const int kw = half * 2 + cols;             // which 32 of the block's keys
        float* xm = reinterpret_cast<float*>(smem + OFF_XM) + group * (4 * HROWS) + row;
        float* xl = reinterpret_cast<float*>(smem + OFF_XL) + row;
        float* mr = reinterpret_cast<float*>(smem + OFF_MR) + row;
        uint8_t* p_hi = smem + OFF_P + group * P_STAGE + row * 128;
        // (what these arrivals at rank 0's barriers announce is read by the tensor
        // core of the SM that wrote it, after the writer's fence)
        const uint32_t q_bar = map_to_rank(smem_u32(&s.q_full), 0), p_bar = map_to_rank(smem_u32(&s.p_full[group]), 0);
        const uint32_t s_bar = map_to_rank(smem_u32(&s.s_free[group]), 0);
        const int sw = row & 7;
        uint32_t j = 0, slot = 0, turn = 0;         // block j is use `turn` of ring slot `slot`
        const int m = (int)rank * HROWS + row;      // query row of a unit
        Rows r{}, done{};
        float sq = 0.f, mref = -INFINITY, l = 0.f;
        bool whole = false;
        int part_slot = 0;
        while (true) {
            // sums of the unit before, this unit's Q, results of the unit before
            if (j > 0) {
                soft_sync();
                const float mlast = mr[((j - 1) & 1) * HROWS];
                xl[(group * 4 + kw) * HROWS] = mref == mlast ? l : l * ex2_approx(mref - mlast);
                mref = mlast;
                soft_sync();
                l = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) l += xl[i * HROWS];
            }
            if (w.left > 0) {
                r = unit_rows(a, w.b, w.u);
                sq = convert_q(a, r, smem, s, rank, tmem, lane_base, j, q_bar);
            }
            if (j > 0) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                const uint64_t inv2 = f2(inv, inv);
                const bool ok = wait_for(&s.pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, status, abort, 9);
                tc_fence_after();
                if (w.left > 0) soft_sync();            // the staging area below is that of convert_q
                uint8_t* stage = smem + OFF_P + warp * 2048;       // 32 rows x 64 bytes
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    uint32_t t[32];
                    tmem_ld32(tmem + lane_base + TM_O + 64 * (warp >> 2) + 32 * c, t);
                    tmem_ld_wait();
                    if (whole) {
                        // through shared memory, so that four lanes write 64 adjacent bytes of a row
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t u[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                u[k] = bf16_pair2(fmul2(f2(__uint_as_float(t[8 * i + 2 * k]), __uint_as_float(t[8 * i + 2 * k + 1])), inv2));
                            *reinterpret_cast<uint4*>(stage + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
                        }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int rr = 8 * i + (lane >> 2), mm = (int)rank * HROWS + (warp & 1) * 32 + rr;
                            const uint4 o = *reinterpret_cast<const uint4*>(stage + rr * 64 + (((lane & 3) ^ ((rr >> 1) & 3)) << 4));
                            if (ok && mm < done.rows)
                                *(reinterpret_cast<uint4*>(a.out + (done.first + mm) * DV + part_col(warp, c)) + (lane & 3)) = o;
                        }
                        __syncwarp();
                    } else if (ok && m < done.rows) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            a.part_o[part_at(part_slot, rank, warp, c, i, lane)] = make_uint4(t[4 * i], t[4 * i + 1], t[4 * i + 2], t[4 * i + 3]);
                    }
                }
                if (!whole && ok && m < done.rows && group == 0 && kw == 0) a.part_ml[part_slot * MROWS + m] = make_float2(mref, l);
                tc_fence_before();
                if (w.left > 0) soft_sync();            // P goes there next
            }
            if (w.left <= 0) break;
            const int n = w.count(), len = seq_len(a, w.b), ctx = len - a.Lq;
            const bool dense = a.idx == nullptr;
            unsigned long long mask = ~0ull;                // nodes that this row sees
            if (dense && m < r.rows) {
                const int i = (r.node0 + m) / a.Hq;
                mask = a.tree ? __ldg(a.tree + (int64_t)w.b * a.Lq + i) : i >= 63 ? ~0ull : (2ull << i) - 1;
            }
            const float arow = sq * a.scale_log2;
            const uint64_t a2 = f2(arow, arow);
            if (w.left > n) {
                Walk after = w;
                after.next(a);
                prefetch_q(a, unit_rows(a, after.b, after.u), rank, threadIdx.x, 32 * SOFT_WARPS);
            }
            mref = -INFINITY;       // what this group's l is relative to
            l = 0.f;
            for (int x = 0; x < n; ++x, ++j) {
                const uint32_t buf = j & 1, ph = (j >> 1) & 1;
                if (buf != (uint32_t)group) {
                    if (++slot == RING) { slot = 0; ++turn; }
                    continue;
                }
                const int s0 = (w.t + x) * NB;              // the block's first entry
                wait_for(&s.scale_full[slot], turn & 1, status, abort, 5);
                const Info& info = reinterpret_cast<const Info*>(smem + OFF_INFO)[slot];
                wait_for(&s.s_full[buf], ph, status, abort, 6);
                tc_fence_after();
                float y[32];
                {
                    uint32_t t[32];
                    tmem_ld32(tmem + lane_base + TM_S + 64 * buf + 32 * cols, t);
                    tmem_ld_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote_cta(s_bar);
                    const float4* g4 = reinterpret_cast<const float4*>(info.scale) + kw * 8;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const float4 g = g4[c], lg = g4[NB / 4 + c];
                        const float2 u = f2_split(ffma2(fmul2(f2(__uint_as_float(t[4 * c]), __uint_as_float(t[4 * c + 1])), a2),
                                                        f2(g.x, g.y), f2(lg.x, lg.y)));
                        const float2 v = f2_split(ffma2(fmul2(f2(__uint_as_float(t[4 * c + 2]), __uint_as_float(t[4 * c + 3])), a2),
                                                        f2(g.z, g.w), f2(lg.z, lg.w)));
                        y[4 * c] = u.x; y[4 * c + 1] = u.y; y[4 * c + 2] = v.x; y[4 * c + 3] = v.y;
                    }
                }
                uint32_t seen = info.seen[kw];
                if (dense && s0 + NB > ctx) seen &= tree_bits(mask, s0 + kw * 32 - ctx);
                if (seen != 0xffffffffu) {
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (!((seen >> c) & 1u)) y[c] = -INFINITY;
                }
                float mx = y[0], my = y[1];
#pragma unroll
                for (int c = 2; c < 32; c += 4) {
                    mx = max3(mx, y[c], y[c + 1]);
                    if (c + 2 < 32) my = max3(my, y[c + 2], y[c + 3]);
                }
                mx = fmaxf(mx, my);
                xm[kw * HROWS] = mx;
                group_sync(group);
                mx = fmaxf(fmaxf(xm[0], xm[HROWS]), fmaxf(xm[2 * HROWS], xm[3 * HROWS]));
                float mprev = -INFINITY;                    // the maximum that O is relative to
                if (x > 0) {
                    take_over(group);
                    mprev = mr[(buf ^ 1) * HROWS];
                } else {
                    group_sync(group);                      // as take_over: every warp has read xm
                }
                const bool grow = mx > mprev + SLACK;
                const float mnew = grow ? mx : mprev;
                if (kw == 0) mr[buf * HROWS] = mnew;
                if (x + 1 < n) hand_over(group ^ 1);
                const float off = mnew == -INFINITY ? 0.f : TOP - mnew;
                const uint64_t off2 = f2(off, off);
                uint64_t l2 = f2(0.f, 0.f);
                uint32_t hi[8], lo[8];
                uint32_t random = random_start((uint32_t)(r.first + m), (uint32_t)(s0 + kw * 32));
                const float4* inv4 = reinterpret_cast<const float4*>(info.inv) + kw * 8;
#pragma unroll
                for (int c = 0; c < 32; c += 4) {
                    const float2 u = f2_split(fadd2(f2(y[c], y[c + 1]), off2));
                    const float2 v = f2_split(fadd2(f2(y[c + 2], y[c + 3]), off2));
                    const float e0 = ex2_approx(u.x), e1 = ex2_approx(u.y), e2 = ex2_approx(v.x), e3 = ex2_approx(v.y);
                    const float4 inv = inv4[c / 4];
                    l2 = ffma2(f2(e0, e1), f2(inv.x, inv.y), l2);
                    l2 = ffma2(f2(e2, e3), f2(inv.z, inv.w), l2);
                    uint32_t h0, h1;
                    float r0, r1, r2, r3;
                    split_weights(e0, e1, h0, r0, r1);
                    split_weights(e2, e3, h1, r2, r3);
                    hi[c / 4] = h0 | h1 << 16;
                    random = random_next(random);
                    // a weight of 2 or more among the four: all of them to the nearest
                    lo[c / 4] = round_rests(r0, r1, r2, r3, hi[c / 4] & 0x40404040u ? NEAREST : random);
                }
                const float2 ls = f2_split(l2);
                l = (mref == mnew ? l : l * ex2_approx(mref - mnew)) + (ls.x + ls.y);
                mref = mnew;
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.info_free[j % (2 * RING)]);
                if (++slot == RING) { slot = 0; ++turn; }
                // P V of j - 2, and with it j - 3, before that of j - 1 (two barriers)
                if (j > 1) wait_for(&s.pv_done[buf], ((j - 2) >> 1) & 1, status, abort, 19);
                if (x > 0 && __any_sync(0xffffffffu, grow)) {
                    // O of the blocks before this one, which P V of the block has not joined yet
                    const float factor = grow ? ex2_approx(mprev - mnew) : 1.f;   // 0 from -inf
                    wait_for(&s.pv_done[buf ^ 1], ((j - 1) >> 1) & 1, status, abort, 7);
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        const uint32_t addr = tmem + lane_base + TM_O + 128 * cols + 32 * c;
                        uint32_t o[32];
                        tmem_ld32(addr, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * factor);
                        tmem_st32(addr, o);
                    }
                    tmem_st_wait();
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int at = ((kw * 2 + c) ^ sw) << 4;
                    *reinterpret_cast<uint4*>(p_hi + at) = make_uint4(hi[4 * c], hi[4 * c + 1], hi[4 * c + 2], hi[4 * c + 3]);
                    *reinterpret_cast<uint4*>(p_hi + ATOM + at) = make_uint4(lo[4 * c], lo[4 * c + 1], lo[4 * c + 2], lo[4 * c + 3]);
                }
                if (dense && s0 + NB > ctx) {
                    // A node that some of the unit's rows see and others do
                    // not: its NaN codes become 0 here, so that 0 weights
                    // leave no NaN; the weights of the rows that see it are
                    // NaN by themselves.
                    wait_for(&s.v_full[buf], ph, status, abort, 4);
                    uint4* v = reinterpret_cast<uint4*>(smem + OFF_V + buf * V_STAGE) + (threadIdx.x & 255);
#pragma unroll 1
                    for (int c = 0; c < V_STAGE / 16 / 256; ++c) {
                        const uint4 o = v[c * 256];
                        uint4 z = o;
                        z.x &= ~__vcmpeq4(o.x & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        z.y &= ~__vcmpeq4(o.y & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        z.z &= ~__vcmpeq4(o.z & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        z.w &= ~__vcmpeq4(o.w & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        if (z.x != o.x || z.y != o.y || z.z != o.z || z.w != o.w) v[c * 256] = z;
                    }
                }
                fence_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote_cta(p_bar);
            }
            done = r;
            whole = w.t == 0 && n == w.nt;
            part_slot = (blockIdx.x / 2) * 2 + (w.t > 0 ? 0 : 1);
            w.next(a);
        }
    } else if (warp < W_RES) {
        // ------------------------------------------------ copies of the tiles
        // K: this CTA's 64 keys whole, 32 rows per warp; V: its columns of all
        // keys, 64 rows per warp.
        const bool is_k = warp < W_COPY + 2;
        const int mine = (warp - W_COPY) & 1;
        const int stage_bytes = is_k ? K_STAGE : V_STAGE;
        const uint32_t stage0 = sbase + (is_k ? OFF_K : OFF_V);
        uint64_t* full = is_k ? s.k_full : s.v_full;
        uint64_t* freed = is_k ? s.s_full : s.pv_done;
        uint32_t j = 0, slot = 0, turn = 0;
        bool ok = true;
        for (int left = w.left; left > 0; --left, ++j) {
            const uint32_t buf = j & 1;
            ok = wait_for(&s.info_full[slot], turn & 1, status, abort, 1);
            if (ok && !is_k) {
                weigh_scales(reinterpret_cast<Info*>(smem + OFF_INFO)[slot], a.cache, mine * 64, lane);
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.scale_full[slot]);
            }
            if (ok && j >= 2) ok = wait_for(&freed[buf], ((j - 2) >> 1) & 1, status, abort, is_k ? 2 : 3);
            if (!ok) break;
            const Info& info = reinterpret_cast<const Info*>(smem + OFF_INFO)[slot];
            const uint32_t dst0 = stage0 + buf * stage_bytes;
            const bool box = info.box != 0;
            if (box) {
                if (lane != 0) {
                } else if (mine == 0) {
                    mbar_arrive_expect_tx(&full[buf], stage_bytes);
                    uint8_t* d = smem + (dst0 - sbase);
                    if (is_k)
                        for (int c = 0; c < 5; ++c)
                            tma_load_2d(d + c * ATOM, &map_box, &full[buf], c * 128, info.rows[0] + HROWS * (int)rank);
                    else
                        for (int c = 0; c < 4; ++c)
                            tma_load_2d(d + c * ATOM, &map_box, &full[buf], (c >> 1) * 256 + (int)rank * 128,
                                        info.rows[0] + (c & 1) * 64);
                } else {
                    mbar_arrive(&full[buf]);
                }
            } else {
                if (is_k) copy_rows<8, 5, 128, ATOM>(dst0, mine * 32, a.cache, info.rows + (int)rank * HROWS + mine * 32, lane);
                else copy_rows<16, 2, 256, 2 * ATOM>(dst0, mine * 64, a.cache + rank * 128, info.rows + mine * 64, lane);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.info_free[j % (2 * RING)]);
            if (!box) {             // the other stage is not free yet: nothing else to send meanwhile
                copy_wait_all();
                fence_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[buf]);
            }
            if (++slot == RING) { slot = 0; ++turn; }
        }
        // boxes have landed before the CTA exits, whatever happened
        for (uint32_t i = j > 2 ? j - 2 : 0; i < j; ++i) mbar_wait_drain(&full[i & 1], (i >> 1) & 1, 200000000ull);
    } else if (warp < W_S) {
        // ------------------------------------------------ positions, scales, masks
        uint32_t j = 0;
        bool ok = true;
        while (w.left > 0 && ok) {
            const int n = w.count(), len = seq_len(a, w.b), ctx = len - a.Lq;
            if (len == 0 && lane == 0) flag_status(status, IC_DEV_INDEX_RANGE);
            const int64_t qrow = (int64_t)w.b * a.Lq + w.u;           // idx given: the unit's row
            unsigned long long mask = ~0ull;
            if (a.idx) mask = a.tree ? __ldg(a.tree + qrow) : w.u >= 63 ? ~0ull : (2ull << w.u) - 1;
            const int32_t* table = a.block_table + (int64_t)w.b * a.max_pages;
            for (int x = 0; x < n && ok; ++x, ++j) {
                if ((j & 1) != (uint32_t)(warp - W_RES)) continue;
                int rows[4];
                float g[4];
                uint32_t valid = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = (w.t + x) * NB + lane * 4 + i;
                    rows[i] = a.idx ? (e < a.k ? __ldg(a.idx + qrow * a.k + e) : -1) : (e < len ? e : -1);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    int p = rows[i];
                    if (p != -1 && (p < 0 || p >= len)) {
                        if (len > 0) flag_status(status, IC_DEV_INDEX_RANGE);
                        p = -1;
                    }
                    if (a.idx && p >= ctx && (p - ctx >= 64 || !((mask >> (p - ctx)) & 1))) p = -1;
                    rows[i] = p;
                }
                int page[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = max(rows[i], 0) / a.page_size;
                    page[i] = rows[i] >= 0 ? __ldg(table + at) : -1;
                    rows[i] -= at * a.page_size;       // its place in the page (negative: seen by nobody)
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (rows[i] >= 0 && (page[i] < 0 || page[i] >= a.num_pages)) {
                        flag_status(status, IC_DEV_INDEX_RANGE);
                        page[i] = -1;
                    }
                    rows[i] = page[i] >= 0 ? page[i] * a.page_size + rows[i] : -1;
                    valid |= page[i] >= 0 ? 1u << i : 0u;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) g[i] = rows[i] >= 0 ? __ldg(a.kv_scale + rows[i]) : 1.f;
                const bool box = a.idx == nullptr && __all_sync(0xffffffffu, valid == 15u);
                uint32_t word = valid << (4 * (lane & 7));
                word |= __shfl_xor_sync(0xffffffffu, word, 1);
                word |= __shfl_xor_sync(0xffffffffu, word, 2);
                word |= __shfl_xor_sync(0xffffffffu, word, 4);
                float lg[4], inv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {          // of a power of two (others: weigh_scales)
                    const uint32_t u = __float_as_uint(g[i]);
                    lg[i] = (float)((int)(u >> 23) - 127);
                    inv[i] = __uint_as_float(0x7f000000u - u);
                }
                const uint32_t slot = j % RING, was = j - RING;       // the slot's block before
                if (j >= RING) ok = wait_for(&s.info_free[was % (2 * RING)], (was / (2 * RING)) & 1, status, abort, 16);
                if (!ok) break;
                Info& info = reinterpret_cast<Info*>(smem + OFF_INFO)[slot];
                reinterpret_cast<int4*>(info.rows)[lane] = make_int4(rows[0], rows[1], rows[2], rows[3]);
                reinterpret_cast<float4*>(info.scale)[lane] = make_float4(g[0], g[1], g[2], g[3]);
                reinterpret_cast<float4*>(info.lg)[lane] = make_float4(lg[0], lg[1], lg[2], lg[3]);
                reinterpret_cast<float4*>(info.inv)[lane] = make_float4(inv[0], inv[1], inv[2], inv[3]);
                if ((lane & 7) == 0) info.seen[lane >> 3] = word;
                if (lane == 0) info.box = box;
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.info_full[slot]);
            }
            if (ok) w.next(a);
        }
    } else {
        // ------------------------------------------------ MMA issue; rank 1 passes its readiness on
        // (counts and outcomes of waits go through votes, which keeps the
        // control flow uniform)
        const bool leader = __any_sync(0xffffffffu, rank == 0);
        const int total = __reduce_max_sync(0xffffffffu, w.left);
        uint32_t unit = 0;
        int unit_begin = 0, unit_end = 0;
        bool ok = true;
        if (warp == W_S) {
            constexpr uint32_t id_s = idesc_f32acc(0, 0, MROWS, NB), id_r = idesc_f32acc(1, 1, MROWS, NB);
            const uint64_t qd = desc_sw128(sbase + OFF_Q, 16, 1024), kd = desc_sw128(sbase + OFF_K, 16, 1024);
            const uint32_t k_peer = map_to_rank(smem_u32(&s.k_peer[0]), 0);
            for (int j = 0; j < total; ++j) {
                const uint32_t buf = j & 1, ph = (j >> 1) & 1;
                if (j == unit_end) {
                    unit_begin = unit_end;
                    unit_end += __reduce_max_sync(0xffffffffu, w.count());
                    w.next(a);
                }
                ok = wait_for(&s.k_full[buf], ph, status, abort, 10);
                if (!ok) break;
                if (!leader) {
                    if (lane == 0) mbar_arrive_remote_cta(k_peer + 8 * buf);
                    continue;
                }
                ok = wait_for(&s.k_peer[buf], ph, status, abort, 11);
                if (j > 1) ok = ok && wait_for(&s.s_free[buf], ((j - 2) >> 1) & 1, status, abort, 20);
                if (j == unit_begin) ok = ok && wait_for(&s.q_full, unit++ & 1, status, abort, 12);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t d = TM_S + 64 * buf;
                    const uint64_t kb = kd + buf * (K_STAGE >> 4);
#pragma unroll 4
                    for (int c = 0; c < 16; ++c)
                        mma_f8_pair(d, qd + (c >> 2) * (ATOM >> 4) + (c & 3) * 2, kb + (c >> 2) * (ATOM >> 4) + (c & 3) * 2, id_s, c > 0);
#pragma unroll
                    for (int c = 0; c < 4; ++c) mma_f8_pair(d, qd + 4 * (ATOM >> 4) + c * 2, kb + c * 2, id_s, 1);
#pragma unroll 4
                    for (int c = 0; c < 12; ++c)
                        mma_f8_ts_pair(d, TM_Q + 8 * c, kb + (1 + (c >> 2)) * (ATOM >> 4) + (c & 3) * 2, id_s, 1);
#pragma unroll
                    for (int c = 0; c < 4; ++c) mma_bf16_ts_pair(d, TM_QR + 8 * c, kb + 4 * (ATOM >> 4) + c * 2, id_r, 1);
                    mma_commit_pair(&s.s_full[buf]);
                }
                __syncwarp();
            }
        } else {
            constexpr uint32_t id_ph = idesc_f32acc(0, 0, MROWS, 256, 0, 1), id_pl = idesc_f32acc(1, 0, MROWS, 256, 0, 1);
            const uint64_t vd = desc_sw128(sbase + OFF_V, 16, 1024), pd = desc_sw128(sbase + OFF_P, 16, 1024);
            const uint32_t v_peer = map_to_rank(smem_u32(&s.v_peer[0]), 0);
            for (int j = 0; j < total; ++j) {
                const uint32_t buf = j & 1, ph = (j >> 1) & 1;
                if (j == unit_end) {
                    unit_begin = unit_end;
                    unit_end += __reduce_max_sync(0xffffffffu, w.count());
                    w.next(a);
                }
                ok = wait_for(&s.v_full[buf], ph, status, abort, 13);
                if (!ok) break;
                if (!leader) {
                    if (lane == 0) mbar_arrive_remote_cta(v_peer + 8 * buf);
                    continue;
                }
                ok = wait_for(&s.v_peer[buf], ph, status, abort, 14);
                ok = ok && wait_for(&s.p_full[buf], ph, status, abort, 15);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t vb = vd + buf * (V_STAGE >> 4), pb = pd + buf * (P_STAGE >> 4);
#pragma unroll 4
                    for (int c = 0; c < 8; ++c)            // hi, lo
#pragma unroll
                        for (int h = 0; h < 2; ++h)        // value columns 0-255, 256-511
                            mma_f8_pair(TM_O + 128 * h, pb + (c >> 2) * (ATOM >> 4) + (c & 3) * 2,
                                        vb + h * (2 * ATOM >> 4) + (c & 3) * (32 * 128 >> 4), c < 4 ? id_ph : id_pl,
                                        c > 0 || j != unit_begin);
                    mma_commit_pair(&s.pv_done[buf]);
                }
                __syncwarp();
            }
        }
        uint64_t* drain = &s.drain[warp - W_S];
        if (leader && elect_one()) mma_commit_pair(drain);
        __syncwarp();
        if (lane == 0) mbar_wait_drain(drain, 0, leader ? 200000000ull : 400000000ull);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == W_S) {
        tc_fence_after();
        tmem_dealloc_pair<TMEM_COLS>(tmem);
    }
}

// ------------------------------------------------------------------ joining partial results
// out = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i over the runs that share
// a unit.  A warp takes 32 rows of N 16-byte pieces (neighbours in a chunk of
// one writing warp) at a time.  The runs are read CH at a time, maxima, sums
// and pieces at once (one memory round trip per chunk); the running maximum
// rescales what earlier chunks added.  Bound by latency (31 MB of 8 runs a unit
// took 10 us as 1184 small CTAs, of which 6 to start them, and as long with a
// list entry read before each piece): one or two CTAs an SM walk over the pieces,
// and the list of what there is to join is read once.
constexpr int JOIN_THREADS = 512;
template <int N, int CH, int CTAS>
__global__ void __launch_bounds__(JOIN_THREADS, CTAS)
tree_join_kernel(const __grid_constant__ Args a, int runs) {
    const int lane = threadIdx.x & 31;
    constexpr int PIECES = 512 / N;              // of a unit
    pdl_trigger();
    pdl_wait();
    __shared__ int4 joins[MAX_PAIRS];
    __shared__ int ends[MAX_PAIRS], count;
    if (threadIdx.x < 32) {
        int n = 0;
        for (int p = lane; p - lane < runs; p += 32) {
            const int4 join = p < runs ? __ldg(a.joins + p) : make_int4(0, 0, 0, 0);
            const unsigned there = __ballot_sync(0xffffffffu, join.z > 0);
            if (join.z > 0) {
                const int at = n + __popc(there & ((1u << lane) - 1u));
                joins[at] = join;
                ends[at] = p;
            }
            n += __popc(there);
        }
        if (lane == 0) count = n;
    }
    __syncthreads();
    const int items = count * PIECES;
    for (int item = blockIdx.x * (JOIN_THREADS / 32) + (threadIdx.x >> 5); item < items;
         item += gridDim.x * (JOIN_THREADS / 32)) {
        const int piece = item % PIECES;
        const int4 join = joins[item / PIECES];
        const int p0 = join.w, p1 = ends[item / PIECES];       // the unit's runs
        const int at = piece % (8 / N) * N, c = piece / (8 / N) & 1, owner = piece / (16 / N) & 15, rank = piece / (256 / N);
        const int m = rank * HROWS + (owner & 1) * 32 + lane;
        if (m >= join.z) continue;
        float top = -INFINITY, l = 0.f;
        float4 o[N];
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p = p0; p <= p1; p += CH) {
            float2 ml[CH];
            uint4 v[CH][N];
#pragma unroll
            for (int c2 = 0; c2 < CH; ++c2) {
                // slot of a run: 1 where the unit begins in it, 0 where it continues the unit
                const bool there = p + c2 <= p1;
                const int slot = 2 * (p + c2) + (p + c2 == p0);
                ml[c2] = there ? __ldg(a.part_ml + slot * MROWS + m) : make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    v[c2][i] = there ? __ldg(a.part_o + part_at(slot, rank, owner, c, at + i, lane)) : make_uint4(0u, 0u, 0u, 0u);
            }
            float mc = top;
#pragma unroll
            for (int c2 = 0; c2 < CH; ++c2) mc = fmaxf(mc, ml[c2].x);
            const float scale = top == mc ? 1.f : ex2_approx(top - mc);
            l *= scale;
#pragma unroll
            for (int i = 0; i < N; ++i) { o[i].x *= scale; o[i].y *= scale; o[i].z *= scale; o[i].w *= scale; }
            top = mc;
#pragma unroll
            for (int c2 = 0; c2 < CH; ++c2) {
                // a run that saw nothing of the row has weight 0 (its sum is 0, or a NaN that stays)
                const float wgt = ml[c2].x == -INFINITY ? (ml[c2].y == 0.f ? 0.f : 1.f) : ex2_approx(ml[c2].x - top);
                l += wgt * ml[c2].y;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    o[i].x += wgt * __uint_as_float(v[c2][i].x); o[i].y += wgt * __uint_as_float(v[c2][i].y);
                    o[i].z += wgt * __uint_as_float(v[c2][i].z); o[i].w += wgt * __uint_as_float(v[c2][i].w);
                }
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t first = (int64_t)(((uint64_t)(uint32_t)join.y << 32) | (uint32_t)join.x);
        uint2* d = reinterpret_cast<uint2*>(a.out + (first + m) * DV + part_col(owner, c) + 4 * at);
#pragma unroll
        for (int i = 0; i < N; ++i) d[i] = make_uint2(bf16_pair(o[i].x * inv, o[i].y * inv), bf16_pair(o[i].z * inv, o[i].w * inv));
    }
}

// ------------------------------------------------------------------ host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (fn == nullptr) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }
    return fn;
}

bool make_map(CUtensorMap* map, const void* base, int64_t rows, int box_rows) {
    auto fn = encode_fn();
    if (fn == nullptr) return false;
    cuuint64_t dims[2] = {(cuuint64_t)ROW, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ROW};
    cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What the host knows of the list of blocks: at most this many.
struct Plan {
    int units, list_blocks, pairs, sharing;
    int64_t blocks;
};
Plan plan(const ic_paged_rows& pr, int k, int Hq) {
    Plan p;
    p.units = k ? pr.Lq : ceil_div(pr.Lq * Hq, MROWS);
    p.list_blocks = k ? ceil_div(k, NB) : (int)ceil_div64(pr.T_max, NB);
    p.blocks = (int64_t)pr.B * p.units * p.list_blocks;
    p.pairs = (int)std::min<int64_t>(MAX_PAIRS, p.blocks);
    p.sharing = BY_LENGTH;
    if (k && p.blocks > 0) {
        const int64_t units = p.blocks / p.list_blocks, nt = p.list_blocks, P = p.pairs;
        const int64_t parts = std::max<int64_t>(1, P / units), run = ceil_div64(units * (nt + UNIT_COST), P);
        const int64_t whole = ceil_div64(units, P) * (nt + UNIT_COST);
        const int64_t in_parts = units > P ? INT64_MAX : ceil_div64(nt, parts) + UNIT_COST + JOIN_COST;
        const int64_t in_runs = run + UNIT_COST + JOIN_COST;
        p.sharing = whole <= std::min(in_parts, in_runs) ? WHOLE : in_parts <= in_runs ? PARTS : RUNS;
    }
    return p;
}

}  // namespace

size_t tree_attn_q8_scratch_bytes(const ic_paged_rows& pr, int k, int Hq) {
    return (size_t)plan(pr, k, Hq).pairs * (2 * MROWS * (DV * sizeof(float) + sizeof(float2)) + sizeof(int4));
}

ic_status launch_tree_attn_q8(const void* q, const void* kv_q8, const float* kv_scale,
                              const int32_t* idx, int k, const uint64_t* tree, const ic_paged_rows& pr, int Hq, float scale,
                              void* out, uint32_t* status, void* scratch, cudaStream_t s) {
    const Plan p = plan(pr, k, Hq);
    if ((int64_t)pr.B * pr.Lq > 0x7fffffffLL || p.blocks >= 1 << 28) return IC_ERR_UNSUPPORTED;
    CUtensorMap map_box;
    if (!make_map(&map_box, kv_q8, (int64_t)pr.num_pages * pr.page_size, 64)) return cuda_error("tree_attn_q8");
    Args a;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.cache = static_cast<const uint8_t*>(kv_q8);
    a.kv_scale = kv_scale;
    a.idx = idx;
    a.tree = reinterpret_cast<const unsigned long long*>(tree);
    a.seq_lens = pr.seq_lens;
    a.block_table = pr.block_table;
    a.out = static_cast<__nv_bfloat16*>(out);
    a.part_o = static_cast<uint4*>(scratch);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + (size_t)p.pairs * 2 * PART);
    a.joins = reinterpret_cast<int4*>(a.part_ml + (size_t)p.pairs * 2 * MROWS);
    a.status = status;
    a.k = k;
    a.B = pr.B;
    a.Lq = pr.Lq;
    a.Hq = Hq;
    a.T_max = pr.T_max;
    a.max_pages = pr.max_pages;
    a.page_size = pr.page_size;
    a.num_pages = pr.num_pages;
    a.units = p.units;
    a.list_blocks = p.list_blocks;
    a.sharing = p.sharing;
    a.scale_log2 = scale * LOG2E;
    if (cudaFuncSetAttribute(tree_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES) != cudaSuccess)
        return cuda_error("tree_attn_q8");
    const bool pdl = pdl_rows((int64_t)pr.B * pr.Lq);
    if (launch_ex(tree_attn_kernel, dim3((unsigned)(2 * p.pairs)), dim3(THREADS), SMEM_BYTES, s, pdl, 0, map_box, a) != cudaSuccess)
        return cuda_error("tree_attn_q8");
    count_launch(IC_LK_TREE);
    ic_status st = last_launch_status();
    if (st != IC_OK || p.sharing == WHOLE || p.list_blocks == 1) return st;     // no partial results
    // Up to 32 pairs: one piece a warp and 16 runs at once, for the latency of
    // many runs of one unit.  More pairs: as for many units, more pieces a warp
    // the fewer runs a unit has (8 a unit: 9.4 us with four pieces, 5.7 with two;
    // 2 a unit: 5.3 and 7.0).  One long unit over all 74 pairs falls under the
    // second rule, where 256 warps read its runs four at a time: 60,000 positions
    // of one sequence take 57 us in all, and its bytes and operations 10.4.
    const bool few = p.pairs <= 32;
    const int64_t units = (int64_t)pr.B * p.units;
    auto join = few ? tree_join_kernel<1, 16, 1> : p.pairs / units > 2 ? tree_join_kernel<2, 4, 2> : tree_join_kernel<4, 2, 2>;
    if (launch_ex(join, dim3(few ? 148 : 2 * 148), dim3(JOIN_THREADS), 0, s, pdl, 0, a, p.pairs) != cudaSuccess)
        return cuda_error("tree_join");
    count_launch(IC_LK_COMBINE);
    return last_launch_status();
}

}  // namespace ic
