// Attention of one new token per sequence over a paged key-value cache.
//
// For query head h of sequence b, with n = lengths[b] cached tokens:
//     z_j = softmax_scale * q . k_j   for max(0, n - window) <= j < n,
//     out = sum_j exp(z_j - lse) v_j,   lse = log sum_j exp(z_j),
// in one pass over the cache: a running base m near the maximum, l = sum exp(z - m) and
// o = sum exp(z - m) v, all in 32 bits; two passes over different tokens join as
//     m = max(m1, m2),  l = l1 exp(m1 - m) + l2 exp(m2 - m),  o likewise,
// whatever the distance of each base from its largest score.
// A row with no token gives out = 0 and lse = -infinity.
//
// Bound by the cache's bytes (2 G / element size flop a byte, G query heads a
// key head), so the kernel is built around keeping loads in flight:
//  - The unit of work is a step: 16 tokens of one key head, or 32 where a row has 64
//    bytes.  All steps of all
//    sequences are numbered through (sequence, head, token) on the device, from
//    the lengths, and cut into equal contiguous ranges, one a warp of a grid
//    that fills the GPU once.  So a ragged batch, one long sequence and many
//    short ones all load every SM alike, and the host needs no length.  Each
//    (sequence, head) skips kUnitCost numbers before its first step: its query,
//    its output and the joins take about that long.
//  - A warp runs its range alone: it copies its steps' rows into its own ring
//    in shared memory (cp.async, two steps ahead and more), and no barrier is met until
//    the range is done.  Page numbers are loaded a step before their rows.
//  - Scores are K Q^T (16 tokens x 8 heads, mma.sync m16n8k16) and the output is
//    V^T P (16 dimensions x 8 heads): with the heads on the 8-wide side a group
//    of 8 query heads wastes nothing, and one head wastes less than on the
//    16-wide side.  P needs one 8x8 transpose (movmatrix) between the two.
//  - A (sequence, head) that lies in one warp's range is written by it; pieces
//    are joined per block in shared memory, and across blocks by a second
//    small kernel, in the order of the tokens: the result does not depend on timing.
// Roundings: the softmax weights meet the values in the MMA as 16 bits, BF16 for
// a BF16 cache, else FP16, and but for two shapes that exact_weights below excepts as two such
// halves wherever one rounding would show in the output: a relative 2^-16 or 2^-21 of each weight,
// where there is one half 2^-8 or 2^-11, while l keeps the 32-bit ones.  FP16 weights
// are taken 2^11 larger, so that one keeps its 11 bits down to 2^-25 of the largest (and
// below, where the values are FP16: the base follows).  E4M3 codes are exact in FP16; a
// BF16 query meets them as FP16 after a power of two that puts its largest element at
// 2^14 (elements below 2^-28 of it lose bits).  The scale of a value row is multiplied into
// its weight, whose base is taken over z + log2(scale), so that it fits FP16.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "common.cuh"
#include "kv_cache.cuh"
#include "numeric.cuh"
#include "ptx.cuh"
#include "stream_mma.cuh"

namespace nvfp4 {
namespace {

constexpr int kRows = 16;          // tokens of an MMA; a step has one or two blocks of so many
constexpr int kWholeUnit = 256;    // units of at most so many tokens are not split between blocks
// Scores may pass the base of their exponentials by so many powers of two more than the
// largest score did when it was taken, before a new one is taken: most steps need no
// maximum over the warp and no rescaling (64 x 8192 E4M3 tokens, 16 query heads a key
// head: 235 us, without 244; 16 x 16384 of 256 and 16 bits 215, 229).
constexpr float kSlack = 4.f;
// Weights that meet the values as FP16 are taken over a base 2^11 below the largest score:
// up to 2^15 with the slack, FP16's range used upwards, since downwards it ends at 2^-14
// (2^-24 with fewer bits) and l, in 32 bits, counts what is lost there.  BF16 has the
// range of 32 bits and needs none.
constexpr float kLift = 11.f;
// The scales of value rows that enter the base are at least this power of two, so that a
// row next to zero, whose weight may then be 2^(kSlack + kLift) over its scale, leaves l finite.
constexpr int kLeastScale = -84;
// With FP16 values the base also follows the scores down: a head whose weights are all
// below 2^kLow in a step takes that step's largest for its base, as far as l stays below
// 2^kMostSum.  A token far above the others with a value next to zero (the first of a long
// text, often) would else press their weights out of FP16: 24 nats above 8192 equal ones
// they came out 23 % too small.  The votes cost up to 2 %, of 16 heads a key head of 256 3 % (221
// us, 214 without).  (E4M3 values bring their scale into the base, and such a token does not
// raise it; what else is lost there, below 2^-36 of the largest weight, is less than their codes' steps.)
constexpr float kLow = -7.f;
constexpr int kMostSum = 80;
constexpr int kUnitCost = 4;       // steps' worth of time that the start and end of a unit take
constexpr size_t kMaxSmem = 227 * 1024;

struct AttnParams {
    const uint16_t* q;             // strides q_row, q_head (elements)
    int64_t q_row, q_head;
    const int32_t* block_table;    // [B, width], row stride table_stride
    int64_t table_stride;
    const int32_t* lengths;
    uint16_t* out;                 // [B, Hq, D]
    float* lse;                    // [B, Hq] or null
    float* parts;                  // workspace: partial results of blocks, then of warps
    int B, Hq, G, chunks, units;   // chunks: head groups of one key head; units = heads * chunks a sequence
    int width;
    bool whole_pages;              // sixteen tokens lie in one page (page_size a multiple of 16)
    int window;                    // 0: none
    bool whole_units;              // no unit is split between blocks
    float scale_log2;              // softmax_scale * log2(e)
    int* status;
    CacheView cache;
};

// By the bytes of a row, and the output values a lane holds: warps a block (one
// block an SM) and steps in a warp's ring.  As many bytes in flight as shared
// memory holds, and as many warps as that and the registers leave: steps of 4 KB
// need sixteen to be computed as fast as they come.  E4M3 rows of 128 with two head
// tiles take twelve warps and four steps each: 121 us for 16 x 16384 tokens, 96 query
// and 8 key heads (eight warps and six steps: 130).  Short contexts lose by it: at 4096
// tokens 42.4 against 41.9, at 2048 27.9 against 26.5, one sequence of 1000 10.7 against 9.8.
constexpr int attn_warps(int row, int values) { return row > 256 ? 4 : row > 128 ? 8 : values >= 64 ? 12 : 16; }
constexpr int attn_stages(int row, int values) { return row == 128 && values >= 64 ? 4 : 3; }

// Where a weight rounded as its values are would show beside the output's own rounding (16-bit
// values; E4M3 ones with an FP16 output, whose weights are FP16), the values are met by both
// halves of it, the larger one and what that left: the output is then as near the formula as
// 32-bit weights would bring it (64 x 16384 tokens of BF16: 1.0 times the error of a plain form
// in 32 bits, with rounded weights 1.4).  Loads hide the second product: 64 x 16384 of
// BF16 326 us with and without, of FP16 329 and 327; 32 x 16384 of 16 heads a key head 177.6 and
// 175.3; 1 x 1000 7.05 and 6.98; E4M3 16 x 4096 19.5 and 18.9, 64 x 8192 179 and 185.
// Not where two tiles of heads wait for their products: 16 heads a key head of 256 in 16 bits
// 233 us with, 214 without; E4M3 96 on 8 heads 130 and 113.  Those keep rounded weights.
constexpr bool exact_weights(bool f16, bool e4m3, int DP, int NT) { return e4m3 ? f16 && NT == 1 : DP / 4 * NT <= 64; }
// The larger half is a weight times this, rounded towards zero: what it leaves is above zero
// then, in 16 bits too (down to 2^-14 in FP16), so that an infinite value gives an infinity, not a NaN.
template <bool F16>
constexpr float kMost = F16 ? 1.f - 0x1p-10f : 1.f - 0x1p-20f;

// Shape of an instance: DP padded head size, NT tiles of 8 query heads.
template <bool E4M3, int DP, int NT>
struct Shape {
    static constexpr int kRow = DP * (E4M3 ? 1 : 2);            // bytes of a row in the ring
    static constexpr int kChunks = kRow / 16;                   // 16-byte chunks a row
    // Blocks of 16 tokens a step: 2 KB leave most of a step's instructions to finding its
    // pages and to the softmax, which a second block shares (64 x 8192 tokens, 32 query
    // and 8 key heads of 64: 99 us, one block 131; 16 x 2048 13.5 and 14.8; one sequence of
    // 1000 7.9 and 7.4).  Longer rows have no room for it.
    static constexpr int kBlocks = kRow == 64 ? 2 : 1;
    static constexpr int kStep = kRows * kBlocks;
    static constexpr int kTile = kStep * kRow;
    static constexpr int kStage = 2 * kTile + (E4M3 ? 2 * kStep * 4 : 0);
    static constexpr int kWarps = attn_warps(kRow, DP / 4 * NT);
    static constexpr int kStages = attn_stages(kRow, DP / 4 * NT);
    static constexpr int kRing = kStages * kStage;
    static constexpr size_t kSmem = (size_t)kWarps * kRing;
    template <bool F16>
    static constexpr bool kExact = exact_weights(F16, E4M3, DP, NT);
    static constexpr int kHeads = 8 * NT;
    static constexpr int kPart = kHeads * (DP + 2);             // floats of a partial result: o, m, l
    static constexpr int kPitch = DP + 4;                       // floats from head to head in shared memory
    static_assert(kSmem + 10240 <= kMaxSmem && kHeads * kPitch * 4 <= kRing && 8 * kPitch * 4 <= kStage, "ring");
};

// Partial results in the workspace: two a block, then one a warp, of whichever cache
// type has more warps (the E4M3 one, whose rows are shorter).
inline size_t workspace_for(int NT, int DP, int64_t sms) {
    const int warps = std::max(attn_warps(DP, DP / 4 * NT), attn_warps(2 * DP, DP / 4 * NT));
    return (size_t)sms * (2 + warps) * 8 * NT * (DP + 2) * sizeof(float);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool held) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(held ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool held) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(held ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t r[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t r[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float lds_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// Chunk of a row where chunk c is kept, so that the reads below meet all banks.
// 16-bit rows: ldmatrix takes one chunk of 8 rows at a time.  E4M3 keys: 8 lanes
// read 4 chunks of 2 rows; values: 8 lanes read 2 chunks of rows 0, 2, 4, 6.
template <bool E4M3, int CH>
__device__ __forceinline__ int key_chunk(int row, int c) {
    if (!E4M3) return c ^ (row & 7);
    return CH == 4 ? c : c ^ ((row & 1) << 2);
}
template <bool E4M3, int CH>
__device__ __forceinline__ int value_chunk(int row, int c) {
    if (!E4M3) return c ^ (row & 7);
    return CH == 4 ? c ^ (((row >> 1) & 1) << 1) : c ^ (row & 7);
}

// Dimension of output row `half` (0: row g, 1: row g + 8) of the 16-row tile mt.
template <bool E4M3, int DP>
__device__ __forceinline__ int out_dim(int mt, int half, int g) {
    if (!E4M3) return mt * 16 + half * 8 + g;
    if (DP == 64) return g * 8 + mt * 2 + half;
    return ((mt >> 3) * 8 + g) * 16 + (mt & 7) * 2 + half;
}

// Output tile nt (8 heads) of a warp to rows of DP + 4 floats, a head each.
template <bool E4M3, int DP, int NT>
__device__ __forceinline__ void store_heads(float* to, const float (&o)[DP / 16][NT][4], int nt, int g, int q4) {
    to += q4 * 2 * (DP + 4) + (E4M3 ? g * (DP == 64 ? 8 : 16) : g);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int mt = 0; mt < DP / 16; ++mt) {
            float* at = to + x * (DP + 4) + out_dim<E4M3, DP>(mt, 0, 0);
            if (!E4M3) {
                at[0] = o[mt][nt][x];
                at[8] = o[mt][nt][2 + x];
            } else if (mt % 2 == 0) {                           // two tiles have four dimensions in a row
                *(float4*)at = make_float4(o[mt][nt][x], o[mt][nt][2 + x], o[mt + 1][nt][x], o[mt + 1][nt][2 + x]);
            }
        }
}

__device__ __forceinline__ float reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float log_sum(float m, float l) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(l));
    return (m + y) * 0.693147180559945309f;
}
// exp2(m - top) for m <= top, and 1 for two equal infinities.
__device__ __forceinline__ float factor(float m, float top) { return m == top ? 1.f : ex2(m - top); }

// Four dimensions of the output, normalised.
template <bool F16>
__device__ __forceinline__ void store_out(uint16_t* to, float4 v, float inv) {
    *(uint2*)to = make_uint2(f32_to_act2<F16>(v.x * inv, v.y * inv), f32_to_act2<F16>(v.z * inv, v.w * inv));
}

// Tokens of sequence b that the table can hold; a length outside is recorded and clamped.
__device__ __forceinline__ int checked_length(const AttnParams& p, int b) {
    const int n = p.lengths[b], most = p.width * p.cache.page_size;
    if ((uint32_t)n > (uint32_t)most) {
        record_status(p.status, NVFP4_ERR_BAD_INDEX);
        return n < 0 ? 0 : most;
    }
    return n;
}
__device__ __forceinline__ int first_token(const AttnParams& p, int n) {
    return p.window > 0 ? max(0, n - p.window) : 0;
}
template <int STEP>
__device__ __forceinline__ int steps_of(const AttnParams& p, int n) {
    return (n + STEP - 1) / STEP - first_token(p, n) / STEP;
}

// A place in the numbering of steps: sequence, unit (key head and head group), step.
template <int STEP>
struct Place {
    int b, u, step, lo, n, s_lo, s_hi;     // tokens [lo, n), steps [s_lo, s_hi) of the sequence

    __device__ __forceinline__ void sequence(const AttnParams& p) {
        n = checked_length(p, b);
        lo = first_token(p, n);
        s_lo = lo / STEP;
        s_hi = (n + STEP - 1) / STEP;
    }
    // Only called where another step follows, so a sequence with tokens is found.
    __device__ __forceinline__ void advance(const AttnParams& p) {
        if (++step < s_hi) return;
        if (++u == p.units) {
            u = 0;
            do {
                ++b;
                sequence(p);
            } while (s_lo == s_hi);
        }
        step = s_lo;
    }
};

// The ranges of numbers: the first `rest` warps have one more than the others
// (fewer numbers than warps: one a warp, packed into the first blocks).
struct Ranges {
    int each, rest;
    __device__ __forceinline__ Ranges(int total, int warps) : each(total / warps), rest(total % warps) {}
    __device__ __forceinline__ int start(int w) const { return w * each + min(w, rest); }
    // The warp whose range holds number x.
    __device__ __forceinline__ int holder(int x) const {
        const int big = rest * (each + 1);
        return x < big ? x / (each + 1) : rest + (x - big) / each;
    }
};

// The numbering of all steps, by a block of WARPS warps: thread t takes `per`
// sequences from t * per on; sm holds the first number of each thread's.
template <int STEP>
__device__ __forceinline__ int numbers_of(const AttnParams& p, int b) {
    const int n = steps_of<STEP>(p, checked_length(p, b));
    return n > 0 ? (n + kUnitCost) * p.units : 0;
}

template <int WARPS, int STEP>
struct Numbering {
    int per, total;

    __device__ __forceinline__ void count(const AttnParams& p, int* sm, int* sums) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        per = (p.B + WARPS * 32 - 1) / (WARPS * 32);
        const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
        int mine = 0;
        for (int b = b0; b < b1; ++b) mine += numbers_of<STEP>(p, b);
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        int s = lane < WARPS ? sums[lane] : 0, before = lane < warp ? s : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s += __shfl_xor_sync(0xffffffffu, s, o);
            before += __shfl_xor_sync(0xffffffffu, before, o);
        }
        total = s;
        sm[threadIdx.x] = before + incl - mine;
        __syncthreads();
    }
    // The sequence that holds number x < total, and its first number (a whole warp asks).
    __device__ __forceinline__ int find(const AttnParams& p, const int* sm, int x, int* first) const {
        int t = -1;
        for (int k = 0, c = 32; k < WARPS * 32 && c == 32; k += 32) {       // ascending: up to the first one above
            c = __popc(__ballot_sync(0xffffffffu, sm[k + (threadIdx.x & 31)] <= x));
            t += c;
        }
        int b = t * per, at = sm[t];
        for (int n; per > 1 && x >= at + (n = numbers_of<STEP>(p, b)); ++b) at += n;
        *first = at;
        return b;
    }
};

// The first number of the unit that holds x, or of the next one if x lies behind its first.
template <int WARPS, int STEP>
__device__ __forceinline__ int unit_from(const AttnParams& p, const Numbering<WARPS, STEP>& steps, const int* sm, int x) {
    if (x >= steps.total) return steps.total;
    int first;
    const int b = steps.find(p, sm, x, &first), each = steps_of<STEP>(p, checked_length(p, b)) + kUnitCost;
    return first + (x - first + each - 1) / each * each;
}

template <bool F16, bool E4M3, int DP, int NT>
__global__ void __launch_bounds__(Shape<E4M3, DP, NT>::kWarps * 32, 1) attend_kernel(const AttnParams p) {
    using S = Shape<E4M3, DP, NT>;
    constexpr int W = S::kWarps, CH = S::kChunks, KS = DP / 16, ST = S::kStages, TB = S::kBlocks, STEP = S::kStep;
    constexpr bool H = F16 || E4M3;                             // FP16 operands in the MMAs
    constexpr bool FALLS = F16 && !E4M3;                        // the base may fall, too
    constexpr float LIFT = H ? kLift : 0.f;
    constexpr bool REST = S::template kExact<F16>;
    extern __shared__ __align__(1024) uint8_t ring_all[];
    __shared__ int first_sm[W * 32], sums[W];
    // Pieces of units, two a warp: the rest of a unit that an earlier warp began, and the last of the range.
    __shared__ int piece_unit[2 * W], piece_lo[2 * W], piece_hi[2 * W];
    __shared__ float piece_m[2 * W][S::kHeads], piece_l[2 * W][S::kHeads];

    pdl_wait_previous();
    pdl_launch_dependents();                                    // the joining kernel numbers the steps meanwhile

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, q4 = lane & 3;
    const int gw = blockIdx.x * W + warp;
    const int D = p.cache.D;

    Numbering<W, STEP> steps;
    steps.count(p, first_sm, sums);
    // This block's range and this warp's, or, where units are short, a range of whole
    // units (from the first that begins in the block's numbers on) spread over its warps.
    int a, e, block_lo, block_hi;
    if (p.whole_units) {
        const Ranges blocks(steps.total, gridDim.x);
        block_lo = unit_from(p, steps, first_sm, blocks.start(blockIdx.x));
        block_hi = unit_from(p, steps, first_sm, blocks.start(blockIdx.x + 1));
        const Ranges own(block_hi - block_lo, W);
        a = block_lo + own.start(warp);
        e = block_lo + own.start(warp + 1);
    } else {
        const Ranges ranges(steps.total, gridDim.x * W);
        block_lo = ranges.start(blockIdx.x * W);
        block_hi = ranges.start(blockIdx.x * W + W);
        a = ranges.start(gw);
        e = ranges.start(gw + 1);
    }

    // ---- sequences without a token
    for (int b = gw; b < p.B; b += gridDim.x * W) {
        if (steps_of<STEP>(p, checked_length(p, b)) > 0) continue;
        uint4* o = (uint4*)(p.out + (int64_t)b * p.Hq * D);
        for (int i = lane; i < p.Hq * D / 8; i += 32) o[i] = make_uint4(0, 0, 0, 0);
        if (p.lse)
            for (int i = lane; i < p.Hq; i += 32) p.lse[(int64_t)b * p.Hq + i] = -INFINITY;
    }

    uint8_t* const ring = ring_all + warp * S::kRing;
    const uint32_t ring_s = smem_u32(ring);
    if (D < DP) {                                               // columns that no copy fills
        for (int i = lane; i < S::kRing / 16; i += 32) ((uint4*)ring)[i] = make_uint4(0, 0, 0, 0);
        __syncwarp();
    }
    float* const warp_parts = p.parts + (size_t)gridDim.x * 2 * S::kPart;
    int head_unit = -1, tail_unit = -1;

    Place<STEP> c;                                              // the step to compute
    int at_c = e, unit_first = 0;                               // its number, and that of its unit's first step
    if (a < e) {
        c.b = steps.find(p, first_sm, a, &unit_first);
        c.sequence(p);
        const int in = a - unit_first, each = c.s_hi - c.s_lo + kUnitCost;
        c.u = in / each;
        const int x = max(in - c.u * each - kUnitCost, 0);
        unit_first += c.u * each + kUnitCost;
        c.step = c.s_lo + x;
        at_c = unit_first + x;
    }
    if (at_c < e) {
        Place<STEP> f = c;                                      // the next step to copy
        int at_f = at_c;

        // Table entries [base, base + 64) of sequence window_b, two a lane.  The second
        // half is loaded when the first is entered, long before it is needed.
        int near = 0, far = 0, base = 0, window_b = -1;
        auto load_entries = [&](int i) {
            return i <= p.cache.entry(f.n - 1) ? p.block_table[f.b * p.table_stride + i] : 0;
        };
        const int held_chunks = D * (E4M3 ? 1 : 2) / 16, r0 = lane / CH, c0 = lane % CH;
        auto copy = [&](int stage) {
            const uint32_t dst = ring_s + stage * S::kStage;
            const int s0 = f.step * STEP, i0 = p.cache.entry(max(s0, f.lo));
            if (f.b != window_b || i0 < base || i0 >= base + 64) {
                window_b = f.b;
                base = i0;
                near = load_entries(base + lane);
                far = load_entries(base + 32 + lane);
            } else if (i0 >= base + 32) {
                base += 32;
                near = far;
                far = load_entries(base + 32 + lane);
            }
            // the page and place of token lane % STEP; those not held take a neighbour's
            const int t = min(max(s0 + (lane & (STEP - 1)), f.lo), f.n - 1), i = p.cache.entry(t);
            const int n0 = __shfl_sync(0xffffffffu, near, (i - base) & 31), n1 = __shfl_sync(0xffffffffu, far, (i - base) & 31);
            int page = i - base < 32 ? n0 : n1;
            if ((uint32_t)page >= (uint32_t)p.cache.num_pages) {
                record_status(p.status, NVFP4_ERR_BAD_INDEX);
                page = 0;
            }
            const int at = t - i * p.cache.page_size, kh = p.chunks == 1 ? f.u : f.u / p.chunks;
            const int64_t off = p.cache.row(page, kh, at);
            const int r_lo = f.lo - s0, r_hi = f.n - s0;        // rows [r_lo, r_hi) are held
            if (p.whole_pages && r_lo <= 0) {                   // sixteen rows at a time evenly spaced
#pragma unroll
                for (int tb = 0; tb < TB; ++tb) {
                    const int64_t from = __shfl_sync(0xffffffffu, off, tb * kRows) + r0 * p.cache.token_bytes + c0 * 16;
                    const uint8_t *k = p.cache.k + from, *v = p.cache.v + from;
                    if (c0 >= held_chunks) continue;
#pragma unroll
                    for (int j = 0; j < CH / 2; ++j) {          // 32 / CH rows an instruction
                        const int r = tb * kRows + j * (32 / CH) + r0;
                        cp_async16(dst + r * S::kRow + key_chunk<E4M3, CH>(r, c0) * 16, k, r < r_hi);
                        cp_async16(dst + S::kTile + r * S::kRow + value_chunk<E4M3, CH>(r, c0) * 16, v, r < r_hi);
                        k += (32 / CH) * p.cache.token_bytes;
                        v += (32 / CH) * p.cache.token_bytes;
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < TB * CH / 2; ++j) {
                    const int r = j * (32 / CH) + r0;
                    const int64_t from = __shfl_sync(0xffffffffu, off, r) + c0 * 16;
                    if (c0 < held_chunks) {
                        cp_async16(dst + r * S::kRow + key_chunk<E4M3, CH>(r, c0) * 16, p.cache.k + from, r >= r_lo && r < r_hi);
                        cp_async16(dst + S::kTile + r * S::kRow + value_chunk<E4M3, CH>(r, c0) * 16, p.cache.v + from, r >= r_lo && r < r_hi);
                    }
                }
            }
            if (E4M3) {                                         // of the keys, then of the values
                const int64_t scale = p.cache.scale_at(page, kh, at);
                const int r = lane & (STEP - 1);
                const bool held = r >= r_lo && r < r_hi;
                if constexpr (TB == 1) {
                    cp_async4(dst + 2 * S::kTile + lane * 4, (lane < 16 ? p.cache.k_scale : p.cache.v_scale) + scale, held);
                } else {
                    cp_async4(dst + 2 * S::kTile + lane * 4, p.cache.k_scale + scale, held);
                    cp_async4(dst + 2 * S::kTile + (STEP + lane) * 4, p.cache.v_scale + scale, held);
                }
            }
        };

        uint32_t qf[KS][NT][2];
        float o[KS][NT][4], m[NT][2], l[NT][2], qs[NT][2];
        bool fresh = true, unscaled = true;                     // a unit begins; its query is not yet scaled
        int seg_begin = at_c, fill = 0, stage = 0;
        bool last = false;
        for (int trip = 1 - ST; !last; ++trip) {                // the first trips only fill the ring
            if (fresh) {
                fresh = false;
                unscaled = true;
                const int kh = p.chunks == 1 ? c.u : c.u / p.chunks;
                const int h0 = (c.u - kh * p.chunks) * S::kHeads;       // first head of the group
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int hg = h0 + nt * 8 + g;
                    const bool held = hg < p.G;
                    const uint16_t* qr = p.q + c.b * p.q_row + (int64_t)(kh * p.G + (held ? hg : 0)) * p.q_head + q4 * (E4M3 ? 16 : 2);
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int d = E4M3 ? (ks >> 2) * 64 + (ks & 3) * 4 + x * 2 : ks * 16 + x * 8;
                            qf[ks][nt][x] = held && d + q4 * (E4M3 ? 16 : 2) < D ? *(const uint32_t*)(qr + d) : 0u;
                        }
                    qs[nt][0] = qs[nt][1] = p.scale_log2;
                    m[nt][0] = m[nt][1] = -INFINITY;
                    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
                    for (int mt = 0; mt < KS; ++mt)
#pragma unroll
                        for (int x = 0; x < 4; ++x) o[mt][nt][x] = 0.f;
                }
            }

            // This trip's step has come, and every lane is done with the stage that is filled next.
            // (Waiting after the fill, with a third step in flight, was 2 to 3 % slower on long
            // sequences: 341 against 332 us for 64 of up to 16384 tokens.)
            cp_async_wait<ST - 2>();
            __syncwarp();
            if (at_f < e) {
                copy(fill);
                at_f += f.step + 1 == f.s_hi ? 1 + kUnitCost : 1;
                if (at_f < e) f.advance(p);
            }
            fill = fill + 1 == ST ? 0 : fill + 1;
            cp_async_commit();
            if (trip < 0) continue;

            if (E4M3 && !F16 && unscaled) {                     // BF16 to FP16, each row's largest element to 2^14
                unscaled = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    uint32_t top = 0;                       // magnitudes of BF16 are in the order of their bits
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int x = 0; x < 2; ++x) top = __vmaxu2(top, qf[ks][nt][x] & 0x7fff7fffu);
                    top = max(top & 0xffffu, top >> 16);
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const int ex = top == 0 || top >= 0x7f80u ? 0 : min(141 - (int)(top >> 7), 100);
                    const float up = __uint_as_float((uint32_t)(ex + 127) << 23), down = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const float2 v = act2_to_f32<false>(qf[ks][nt][x]);
                            qf[ks][nt][x] = f32_to_act2<true>(v.x * up, v.y * up);
                        }
                    // the accumulator's columns are heads 2 q4 and 2 q4 + 1
                    qs[nt][0] *= __shfl_sync(0xffffffffu, down, q4 * 8);
                    qs[nt][1] *= __shfl_sync(0xffffffffu, down, q4 * 8 + 4);
                }
            }
            const uint32_t ks_s = ring_s + stage * S::kStage, vs_s = ks_s + S::kTile;

            // ---- scores of 16 tokens (rows g, g + 8) x 8 heads (columns 2 q4, 2 q4 + 1)
            float z[TB][NT][4], z2[TB][NT][4];                  // one head tile: two chains of products
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 4; ++x) z[tb][nt][x] = z2[tb][nt][x] = 0.f;
                if constexpr (!E4M3) {
                    const int row = tb * kRows + (lane & 7) + (lane & 8), ch = lane >> 4;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        uint32_t af[4];
                        ldmatrix4(af, ks_s + row * S::kRow + key_chunk<E4M3, CH>(row, ks * 2 + ch) * 16);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_16816<H>(NT == 1 && ks & 1 ? z2[tb][nt] : z[tb][nt], af, qf[ks][nt][0], qf[ks][nt][1]);
                    }
                } else {
                    const int row = tb * kRows + g;
#pragma unroll
                    for (int j = 0; j < KS / 4; ++j) {
                        const uint4 w0 = lds128(ks_s + row * S::kRow + key_chunk<E4M3, CH>(row, j * 4 + q4) * 16);
                        const uint4 w1 = lds128(ks_s + (row + 8) * S::kRow + key_chunk<E4M3, CH>(row + 8, j * 4 + q4) * 16);
                        const uint32_t lo[4] = {w0.x, w0.y, w0.z, w0.w}, hi[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const uint32_t af[4] = {e4m3x2_to_f16x2((uint16_t)lo[w]), e4m3x2_to_f16x2((uint16_t)hi[w]),
                                                    e4m3x2_to_f16x2((uint16_t)(lo[w] >> 16)), e4m3x2_to_f16x2((uint16_t)(hi[w] >> 16))};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_16816<H>(NT == 1 && w & 1 ? z2[tb][nt] : z[tb][nt], af, qf[j * 4 + w][nt][0], qf[j * 4 + w][nt][1]);
                        }
                    }
                }
            }

            // ---- softmax weights; a lane has two tokens a block
            bool held[TB][2];
            float k_by[TB][2], v_by[TB][2], lv[TB][2];
#pragma unroll
            for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int row = tb * kRows + y * 8 + g, t = c.step * STEP + row;
                    held[tb][y] = t >= c.lo && t < c.n;
                    k_by[tb][y] = v_by[tb][y] = 1.f;
                    lv[tb][y] = 0.f;
                    if (E4M3) {
                        k_by[tb][y] = lds_f32(ks_s + 2 * S::kTile + row * 4);
                        v_by[tb][y] = lds_f32(ks_s + 2 * S::kTile + (STEP + row) * 4);
                        // a power of two above the scale: weights times scales stay below 2^(kSlack + kLift)
                        lv[tb][y] = (float)max((int)((__float_as_uint(v_by[tb][y]) >> 23) & 255) - 126, kLeastScale);
                    }
                }
            float top[NT][2];
            bool above = false, below = false;                  // a score far above its base; all of a head's far below it
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        float& s = z[tb][nt][x];
                        s = (NT == 1 ? s + z2[tb][nt][x] : s) * qs[nt][x & 1];
                        if (E4M3) s *= k_by[tb][x >> 1];
                        if (!held[tb][x >> 1]) s = -INFINITY;
                    }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    top[nt][x] = fmaxf(z[0][nt][x] + lv[0][0], z[0][nt][x + 2] + lv[0][1]);
                    if constexpr (TB == 2)
                        top[nt][x] = fmaxf(top[nt][x], fmaxf(z[TB - 1][nt][x] + lv[TB - 1][0], z[TB - 1][nt][x + 2] + lv[TB - 1][1]));
                    const float by = top[nt][x] - m[nt][x];
                    above |= by > kSlack + LIFT;
                    if (FALLS) below |= by < kLow;
                }
            }
            // a new base: seldom after the first steps (with both signs, one vote where there is none)
            const bool moves = __any_sync(0xffffffffu, above || below);
            if (FALLS ? moves && __any_sync(0xffffffffu, above) : moves) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float to = top[nt][x];
                        to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, 4));
                        to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, 8));
                        to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, 16));
                        to = fmaxf(m[nt][x], to - LIFT);
                        const float keep = ex2(m[nt][x] - (to == -INFINITY ? 0.f : to));
                        m[nt][x] = to;
                        l[nt][x] *= keep;
#pragma unroll
                        for (int mt = 0; mt < KS; ++mt) {
                            o[mt][nt][x] *= keep;
                            o[mt][nt][x + 2] *= keep;
                        }
                    }
            }
            if (FALLS && moves) {                               // a lower one: about once a token far above the others
                uint32_t low = 0;                               // by column: no weight of this lane reaches 2^kLow
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x) low |= (uint32_t)(top[nt][x] - m[nt][x] < kLow) << (nt * 2 + x);
                // ... and of none of the eight lanes of the same heads
#pragma unroll
                for (int lanes = 4; lanes < 32; lanes <<= 1) low &= __shfl_xor_sync(0xffffffffu, low, lanes);
                if (__any_sync(0xffffffffu, low != 0)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            float to = top[nt][x], sum = l[nt][x];
#pragma unroll
                            for (int lanes = 4; lanes < 32; lanes <<= 1) {
                                to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, lanes));
                                sum = fmaxf(sum, __shfl_xor_sync(0xffffffffu, sum, lanes));
                            }
                            // whole powers of two, by which l and o lose nothing
                            const int room = kMostSum + 126 - (int)(__float_as_uint(sum) >> 23);
                            const int by = min((int)fminf(m[nt][x] - (to - LIFT), 100.f), room);
                            if ((low >> (nt * 2 + x) & 1) && by > 0) {
                                const float up = __uint_as_float((uint32_t)(127 + by) << 23);
                                m[nt][x] -= (float)by;
                                l[nt][x] *= up;
#pragma unroll
                                for (int mt = 0; mt < KS; ++mt) {
                                    o[mt][nt][x] *= up;
                                    o[mt][nt][x + 2] *= up;
                                }
                            }
                        }
                }
            }
            uint32_t pf[TB][NT][2], pr[TB][NT][2];              // weights, or (REST) their halves
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float base[2] = {m[nt][0] == -INFINITY ? 0.f : m[nt][0], m[nt][1] == -INFINITY ? 0.f : m[nt][1]};
#pragma unroll
                for (int tb = 0; tb < TB; ++tb) {
                    float w[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) w[x] = ex2(z[tb][nt][x] - base[x & 1]);
                    l[nt][0] += w[0] + w[2];
                    l[nt][1] += w[1] + w[3];
                    // heads on the MMA's columns: transpose the 8x8 blocks
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float a = w[2 * y] * v_by[tb][y], b = w[2 * y + 1] * v_by[tb][y];
                        if constexpr (REST) {
                            const uint32_t most = f32_to_act2_down<H>(a * kMost<H>, b * kMost<H>);
                            const float2 u = act2_to_f32<H>(most);
                            pf[tb][nt][y] = movmatrix(most);
                            pr[tb][nt][y] = movmatrix(f32_to_act2<H>(a - u.x, b - u.y));
                        } else {
                            pf[tb][nt][y] = movmatrix(f32_to_act2<H>(a, b));
                        }
                    }
                }
            }

            // ---- output of 16 dimensions (rows) x 8 heads at a time
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) {
                if constexpr (!E4M3) {
                    const int row = tb * kRows + (lane & 7) + ((lane >> 4) << 3), ch = (lane >> 3) & 1;
#pragma unroll
                    for (int mt = 0; mt < KS; ++mt) {
                        uint32_t af[4];
                        ldmatrix4_trans(af, vs_s + row * S::kRow + value_chunk<E4M3, CH>(row, mt * 2 + ch) * 16);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_16816<H>(o[mt][nt], af, pf[tb][nt][0], pf[tb][nt][1]);
                            if constexpr (REST) mma_16816<H>(o[mt][nt], af, pr[tb][nt][0], pr[tb][nt][1]);
                        }
                    }
                } else {
                    // A lane takes the dimensions of chunk g (half a chunk of 64) of tokens 2 q4, 2 q4 + 1 and
                    // the two 8 on; byte permutes pair the tokens.
                    constexpr int WORDS = DP == 64 ? 2 : 4;
#pragma unroll
                    for (int j = 0; j < (DP == 64 ? 1 : DP / 128); ++j) {
                        uint32_t v[4][WORDS];
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int r = tb * kRows + 2 * q4 + (x & 1) + (x >> 1) * 8;
                            if constexpr (DP == 64) {
                                const uint2 u = lds64(vs_s + r * S::kRow + value_chunk<E4M3, CH>(r, g >> 1) * 16 + (g & 1) * 8);
                                v[x][0] = u.x; v[x][1] = u.y;
                            } else {
                                const uint4 u = lds128(vs_s + r * S::kRow + value_chunk<E4M3, CH>(r, j * 8 + g) * 16);
                                v[x][0] = u.x; v[x][1] = u.y; v[x][2] = u.z; v[x][3] = u.w;
                            }
                        }
#pragma unroll
                        for (int w = 0; w < WORDS; ++w)
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const uint32_t sel = half ? 0x7362 : 0x5140;
                                const uint32_t lo = __byte_perm(v[0][w], v[1][w], sel), hi = __byte_perm(v[2][w], v[3][w], sel);
                                const uint32_t af[4] = {e4m3x2_to_f16x2((uint16_t)lo), e4m3x2_to_f16x2((uint16_t)(lo >> 16)),
                                                        e4m3x2_to_f16x2((uint16_t)hi), e4m3x2_to_f16x2((uint16_t)(hi >> 16))};
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    mma_16816<H>(o[j * 8 + w * 2 + half][nt], af, pf[tb][nt][0], pf[tb][nt][1]);
                                    if constexpr (REST) mma_16816<H>(o[j * 8 + w * 2 + half][nt], af, pr[tb][nt][0], pr[tb][nt][1]);
                                }
                            }
                    }
                }
            }

            // ---- the end of a unit, or of the range
            const bool unit_end = c.step + 1 == c.s_hi;
            at_c += unit_end ? 1 + kUnitCost : 1;
            last = at_c >= e;
            if (unit_end || last) {
                const int unit = c.b * p.units + c.u, unit_hi = unit_first + c.s_hi - c.s_lo;
                const bool whole = unit_end && seg_begin == unit_first;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], 4);
                        l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], 8);
                        l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], 16);
                    }
                if (!whole) {
                    const int y = 2 * warp + last;
                    if (lane == 0) { piece_lo[y] = unit_first; piece_hi[y] = unit_hi; }
                    if (g == 0) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                piece_m[y][nt * 8 + q4 * 2 + x] = m[nt][x];
                                piece_l[y][nt * 8 + q4 * 2 + x] = l[nt][x];
                            }
                    }
                }
                if (!whole && last) {
                    // The last piece of the range stays in the ring: nothing is in flight any more.
                    cp_async_wait<0>();
                    __syncwarp();
                    tail_unit = unit;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) store_heads<E4M3, DP, NT>((float*)ring + nt * 8 * S::kPitch, o, nt, g, q4);
                } else {
                    // A whole unit goes out, the rest of one that an earlier warp began to the
                    // workspace: eight heads at a time through the stage just read, which is
                    // filled again after the next trip's __syncwarp.
                    if (!whole) head_unit = unit;
                    float* const buf = (float*)(ring + stage * S::kStage);
                    const int kh = p.chunks == 1 ? c.u : c.u / p.chunks, h0 = (c.u - kh * p.chunks) * S::kHeads;
                    const int64_t row = (int64_t)c.b * p.Hq + kh * p.G + h0;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        __syncwarp();
                        store_heads<E4M3, DP, NT>(buf, o, nt, g, q4);
                        __syncwarp();
                        const float inv0 = reciprocal(l[nt][0]), inv1 = reciprocal(l[nt][1]);
#pragma unroll 4
                        for (int y = 0; y < DP / 16; ++y) {
                            const int x = y * 32 + lane;
                            const int hl = x / (DP / 4), d = x % (DP / 4) * 4;
                            const float4 v = *(const float4*)(buf + hl * S::kPitch + d);
                            const float even = __shfl_sync(0xffffffffu, inv0, hl >> 1), odd = __shfl_sync(0xffffffffu, inv1, hl >> 1);
                            if (!whole) *(float4*)(warp_parts + (size_t)gw * S::kPart + (nt * 8 + hl) * DP + d) = v;
                            else if (h0 + nt * 8 + hl < p.G && d < D)
                                store_out<F16>(p.out + (row + nt * 8 + hl) * D + d, v, hl & 1 ? odd : even);
                        }
                        if (whole && p.lse && g == 0) {
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const int hl = nt * 8 + q4 * 2 + x;
                                if (h0 + hl < p.G) p.lse[row + hl] = log_sum(m[nt][x], l[nt][x]);
                            }
                        }
                    }
                    if (D < DP) {                               // the columns that no copy fills
                        __syncwarp();
                        for (int x = lane; x < S::kStage / 16; x += 32) ((uint4*)buf)[x] = make_uint4(0, 0, 0, 0);
                    }
                }
                unit_first = unit_hi + kUnitCost;
                seg_begin = at_c;
                fresh = true;
            }
            stage = stage + 1 == ST ? 0 : stage + 1;
            if (!last) c.advance(p);
        }
    }

    // ---- join the block's pieces
    if (lane == 0) {
        piece_unit[2 * warp] = head_unit;
        piece_unit[2 * warp + 1] = tail_unit;
    }
    if (!__syncthreads_or(head_unit >= 0 || tail_unit >= 0)) return;
    // Every warp makes out the block's runs of pieces of one unit: the last pieces of
    // neighbouring warps, then the first of the warp after them where the unit ends in
    // it; a first piece whose unit began in an earlier block is a run of its own.
    const int tail = lane < W ? piece_unit[2 * lane + 1] : -1, head = lane < W ? piece_unit[2 * lane] : -1;
    const int left = __shfl_up_sync(0xffffffffu, tail, 1);
    const bool joined = head >= 0 && lane > 0 && left == head;
    const uint32_t change = __ballot_sync(0xffffffffu, lane >= W || lane == 0 || tail != left);
    const uint32_t ends = __ballot_sync(0xffffffffu, joined);
    static_assert(W <= 16, "two sets of runs in 32 bits");
    uint32_t runs = __ballot_sync(0xffffffffu, tail >= 0 && (lane == 0 || tail != left)) |
                    __ballot_sync(0xffffffffu, head >= 0 && !joined) << 16;
    // A thread takes four dimensions of one head; small units side by side.
    constexpr int E = S::kHeads * DP / 4, PER = E < W * 32 ? W * 32 / E : 1;
#pragma unroll 1
    for (int rank = 0; runs != 0; ++rank, runs &= runs - 1) {
        if (PER > 1 && rank % PER != tid / E) continue;
        const int bit = __ffs(runs) - 1, w0 = bit & 15;
        const int w1 = bit >= 16 ? w0 : w0 + __ffs(change >> (w0 + 1));         // last pieces of warps [w0, w1)
        const int wh = bit >= 16 ? w0 : w1 < W && (ends >> w1 & 1) ? w1 : -1;   // the first piece of this warp
        const int y0 = bit >= 16 ? 2 * w0 : 2 * w0 + 1, unit = piece_unit[y0], lo = piece_lo[y0], hi = piece_hi[y0];
        const int b = unit / p.units, u = unit - b * p.units, kh = u / p.chunks, h0 = (u - kh * p.chunks) * S::kHeads;
#pragma unroll 1
        for (int x = PER > 1 ? tid % E : tid; x < E; x += W * 32) {
            const int hl = x / (DP / 4), d = x % (DP / 4) * 4;
            if (h0 + hl >= p.G || d >= D) continue;
            float top = wh >= 0 ? piece_m[2 * wh][hl] : -INFINITY, sum = 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int w = w0; w < w1; ++w) top = fmaxf(top, piece_m[2 * w + 1][hl]);
#pragma unroll 4
            for (int w = w0; w < w1; ++w) {
                const float t = factor(piece_m[2 * w + 1][hl], top);
                const float4 o = *(const float4*)((const float*)(ring_all + w * S::kRing) + hl * S::kPitch + d);
                sum += t * piece_l[2 * w + 1][hl];
                v.x += t * o.x; v.y += t * o.y; v.z += t * o.z; v.w += t * o.w;
            }
            if (wh >= 0) {
                const float t = factor(piece_m[2 * wh][hl], top);
                const float4 o = *(const float4*)(warp_parts + (size_t)(blockIdx.x * W + wh) * S::kPart + hl * DP + d);
                sum += t * piece_l[2 * wh][hl];
                v.x += t * o.x; v.y += t * o.y; v.z += t * o.z; v.w += t * o.w;
            }
            if (lo >= block_lo && hi <= block_hi) {
                const int64_t row = (int64_t)b * p.Hq + kh * p.G + h0 + hl;
                store_out<F16>(p.out + row * D + d, v, reciprocal(sum));
                if (p.lse && d == 0) p.lse[row] = log_sum(top, sum);
            } else {
                float* to = p.parts + ((size_t)blockIdx.x * 2 + (lo >= block_lo)) * S::kPart;
                *(float4*)(to + hl * DP + d) = v;
                if (d == 0) {
                    to[S::kHeads * DP + hl] = top;
                    to[S::kHeads * (DP + 1) + hl] = sum;
                }
            }
        }
    }
}

// Joins the units that lie in several blocks of the kernel above, each by those
// same blocks' numbers here: block x of a unit's P takes a P-th of its output, its
// threads that many elements and the pieces in turn.  The units are found from
// the lengths while that kernel still runs, so only the pieces' own loads, all at
// once, come after it.
template <bool F16, bool E4M3, int DP, int NT>
__global__ void __launch_bounds__(128, 8) join_kernel(const AttnParams p) {
    using S = Shape<E4M3, DP, NT>;
    constexpr int W = S::kWarps, N = 4;                         // pieces in flight a thread
    __shared__ int first_sm[128], sums[4];
    __shared__ float part_m[128], part_l[128];
    __shared__ float4 part_o[128];
    const int x = blockIdx.x, tid = threadIdx.x, D = p.cache.D;
    Numbering<4, S::kStep> steps;
    steps.count(p, first_sm, sums);
    const Ranges ranges(steps.total, gridDim.x * W);
    const int lo = ranges.start(x * W), hi = ranges.start(x * W + W);
    // Half the threads take the unit at the start of the block's range, if an earlier
    // block began it, the others the one at its end, if it begins here and goes on.
    const int k = tid / 64, at = k == 0 ? lo : hi - 1;
    int b = 0, u = 0, from = 0, to = -1;
    if (hi > lo) {
        int first;
        b = steps.find(p, first_sm, at, &first);
        const int each = steps_of<S::kStep>(p, checked_length(p, b)) + kUnitCost;
        u = (at - first) / each;
        const int unit_lo = first + u * each + kUnitCost, unit_hi = first + (u + 1) * each;
        if (k == 0 ? unit_lo < lo : unit_lo >= lo && unit_lo < hi && unit_hi > hi) {
            from = ranges.holder(unit_lo) / W;
            to = ranges.holder(unit_hi - 1) / W;
        }
    }
    const int kh = u / p.chunks, h0 = (u - kh * p.chunks) * S::kHeads, E = min(S::kHeads, p.G - h0) * (DP / 4);
    const int P = to - from + 1, share = to < 0 ? 0 : (E + P - 1) / P, e1 = min(E, (x - from + 1) * share);
    pdl_wait_previous();
    pdl_launch_dependents();
    if (to < 0) return;                                         // the barriers below are this half's own
    for (int base = (x - from) * share; base < e1; base += 64) {
        const int n = min(64, e1 - base), groups = min(64 / n, (P + N - 1) / N), group = tid % 64 / n, el = tid % 64 - group * n;
        const int e = base + el, hl = e / (DP / 4), d = e % (DP / 4) * 4;
        float top = -INFINITY, sum = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (group < groups && d < D) {
            for (int y0 = from + group; y0 <= to; y0 += groups * N) {
                float m[N], l[N], high = top;
                float4 o[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int y = min(y0 + i * groups, to);
                    const float* part = p.parts + ((size_t)y * 2 + (y == from)) * S::kPart;
                    m[i] = part[S::kHeads * DP + hl];
                    l[i] = part[S::kHeads * (DP + 1) + hl];
                    o[i] = *(const float4*)(part + hl * DP + d);
                }
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (y0 + i * groups <= to) high = fmaxf(high, m[i]);
                const float keep = factor(top, high);
                sum *= keep;
                v.x *= keep; v.y *= keep; v.z *= keep; v.w *= keep;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    if (y0 + i * groups > to) continue;
                    const float t = factor(m[i], high);
                    sum += t * l[i];
                    v.x += t * o[i].x; v.y += t * o[i].y; v.z += t * o[i].z; v.w += t * o[i].w;
                }
                top = high;
            }
        }
        part_m[tid] = top;
        part_l[tid] = sum;
        part_o[tid] = v;
        named_bar_sync(1 + k, 64);
        if (group == 0 && d < D) {
            for (int i = tid + n; i < k * 64 + groups * n; i += n) {
                const float high = fmaxf(top, part_m[i]), keep = factor(top, high), t = factor(part_m[i], high);
                const float4 o = part_o[i];
                sum = sum * keep + t * part_l[i];
                v.x = v.x * keep + t * o.x; v.y = v.y * keep + t * o.y; v.z = v.z * keep + t * o.z; v.w = v.w * keep + t * o.w;
                top = high;
            }
            const int64_t row = (int64_t)b * p.Hq + kh * p.G + h0 + hl;
            store_out<F16>(p.out + row * D + d, v, reciprocal(sum));
            if (p.lse && d == 0) p.lse[row] = log_sum(top, sum);
        }
        named_bar_sync(1 + k, 64);
    }
}

template <bool F16, bool E4M3, int DP, int NT>
nvfp4_status launch_attention(AttnParams p, void* workspace, cudaStream_t stream) {
    using S = Shape<E4M3, DP, NT>;
    const char* fn = "nvfp4_paged_attention";
    const int64_t most = (int64_t)p.B * p.units * (ceil_div((int64_t)p.width * p.cache.page_size, S::kStep) + 1 + kUnitCost);
    if (most > INT32_MAX)
        return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: %lld steps of tokens and heads in one call, above 2^31", fn, (long long)most);
    // Short units are not split between blocks: there is nothing to join after the
    // kernel.  (8 sequences of 128 tokens 6.3 us and one launch against 6.8 and two, of
    // 256 7.3 and 7.9; at 500 tokens, 32 steps, splitting wins, 8.8 against 9.5 us.)
    int64_t tokens = (int64_t)p.width * p.cache.page_size;
    if (p.window > 0) tokens = std::min<int64_t>(tokens, (int64_t)p.window + S::kStep);
    p.whole_units = tokens <= kWholeUnit;
    // as many blocks as the longest lengths could use, at most one wave
    const int64_t use = p.whole_units ? (int64_t)p.B * p.units : ceil_div(most, S::kWarps);
    const int ctas = (int)std::max<int64_t>(1, std::min<int64_t>(sm_count(), use));
    p.parts = (float*)workspace;
    auto kernel = attend_kernel<F16, E4M3, DP, NT>;
    static std::atomic<uint64_t> opted_in{0};                   // devices whose instance has its shared memory limit raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return check_cuda(e, fn);
    const uint64_t bit = 1ull << (dev & 63);
    if (!(opted_in.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
        if (e != cudaSuccess) return check_cuda(e, fn);
        opted_in.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(S::kWarps * 32);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, p);
    if (e != cudaSuccess) return check_cuda(e, fn);
    if (ctas == 1 || p.whole_units) return NVFP4_OK;
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    return check_cuda(cudaLaunchKernelEx(&cfg, join_kernel<F16, E4M3, DP, NT>, p), fn);
}

template <bool F16, bool E4M3>
nvfp4_status launch_shape(const AttnParams& p, int DP, int NT, void* ws, cudaStream_t s) {
    if (DP == 64) return NT == 1 ? launch_attention<F16, E4M3, 64, 1>(p, ws, s) : launch_attention<F16, E4M3, 64, 2>(p, ws, s);
    if (DP == 128) return NT == 1 ? launch_attention<F16, E4M3, 128, 1>(p, ws, s) : launch_attention<F16, E4M3, 128, 2>(p, ws, s);
    return NT == 1 ? launch_attention<F16, E4M3, 256, 1>(p, ws, s) : launch_attention<F16, E4M3, 256, 2>(p, ws, s);
}

int padded_dim(int64_t D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }
int head_tiles(int64_t G) { return G <= 8 ? 1 : 2; }

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" size_t nvfp4_paged_attention_workspace(int64_t B, int64_t Hq, int64_t heads, int64_t head_dim) {
    if (B <= 0 || heads <= 0 || Hq <= 0 || Hq % heads != 0 || head_dim <= 0 || head_dim > kMaxHeadDim) return 0;
    return workspace_for(head_tiles(Hq / heads), padded_dim(head_dim), sm_count());
}

extern "C" nvfp4_status nvfp4_paged_attention(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                                              const nvfp4_kv_cache* cache, const int32_t* block_table,
                                              int64_t table_stride, int64_t table_width, const int32_t* lengths,
                                              int64_t B, int64_t Hq, float softmax_scale, int64_t window, int f16,
                                              void* out, float* lse, void* workspace, size_t workspace_bytes,
                                              void* stream) {
    const char* fn = "nvfp4_paged_attention";
    AttnParams p{};
    if (nvfp4_status st = check_cache(fn, cache, &p.cache)) return st;
    if (B < 0 || window < 0) return fail(NVFP4_ERR_INVALID_ARG, "%s: negative size B=%lld window=%lld", fn, (long long)B, (long long)window);
    if (f16 != 0 && f16 != 1) return fail(NVFP4_ERR_INVALID_ARG, "%s: f16=%d must be 0 or 1", fn, f16);
    if (!std::isfinite(softmax_scale)) return fail(NVFP4_ERR_INVALID_ARG, "%s: softmax_scale must be finite", fn);
    if (Hq <= 0 || Hq % p.cache.heads != 0 || Hq > 65536)
        return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: Hq=%lld must be a positive multiple of the cache's %d heads (at most 65536)", fn, (long long)Hq, p.cache.heads);
    if (table_width < 0 || table_width > INT32_MAX || table_width * p.cache.page_size > INT32_MAX - 64)
        return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: a table of %lld pages of %d tokens passes 2^31 tokens", fn, (long long)table_width, p.cache.page_size);
    if (B > INT32_MAX / 2) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: B=%lld above 2^30", fn, (long long)B);
    if (B == 0) return NVFP4_OK;
    if (!q || !lengths || !out || (table_width > 0 && !block_table)) return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (q_row_stride < 0 || q_head_stride < 0 || table_stride < 0) return fail(NVFP4_ERR_INVALID_ARG, "%s: negative stride", fn);
    if (!aligned(q, 16) || q_row_stride % 8 || q_head_stride % 8 || !aligned(out, 16) || !aligned(block_table, 4) || !aligned(lengths, 4) || !aligned(lse, 4))
        return fail(NVFP4_ERR_ALIGNMENT, "%s: q's rows and out must be 16-byte aligned, block_table, lengths and lse 4-byte", fn);
    const size_t need = nvfp4_paged_attention_workspace(B, Hq, p.cache.heads, p.cache.D);
    if (workspace_bytes < need || !workspace)
        return fail(NVFP4_ERR_WORKSPACE, "%s: workspace %zu bytes, needs %zu", fn, workspace_bytes, need);
    if (!aligned(workspace, 256)) return fail(NVFP4_ERR_ALIGNMENT, "%s: workspace must be 256-byte aligned", fn);
    // out may be q: a unit's output is written once all of its steps are done, and no other unit reads its query.
    const int64_t D = p.cache.D;
    const Span o = dense_span("out", out, 2 * B * Hq * D), sums = dense_span("lse", lse, 4 * B * Hq), ws = dense_span("workspace", workspace, (int64_t)need);
    const Span qs = strided_span("q", q, 2 * D, {{B, 2 * q_row_stride}, {Hq, 2 * q_head_stride}});
    const bool in_place = q == out && (B == 1 || q_row_stride == Hq * D) && (Hq == 1 || q_head_stride == D);
    if (!in_place && overlaps(o, qs))
        return fail(NVFP4_ERR_INVALID_ARG, "%s: out overlaps q (it may be q itself where that is dense)", fn);
    const Span pages = strided_span("block_table", block_table, 4 * table_width, {{B, 4 * table_stride}}), counts = dense_span("lengths", lengths, 4 * B);
    if (const char* s = met(sums, {qs, o, ws})) return fail(NVFP4_ERR_INVALID_ARG, "%s: lse overlaps %s", fn, s);
    if (const char* s = met(ws, {qs, o})) return fail(NVFP4_ERR_INVALID_ARG, "%s: workspace overlaps %s", fn, s);
    for (const Span& to : {o, sums, ws}) {
        if (const char* s = met(to, {pages, counts})) return fail(NVFP4_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, to.name, s);
        if (const char* part = met_cache(to, p.cache)) return fail(NVFP4_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, to.name, part);
    }
    p.status = device_status_ptr();
    if (!p.status) return fail(NVFP4_ERR_CUDA, "%s: no CUDA device", fn);
    p.q = (const uint16_t*)q; p.q_row = q_row_stride; p.q_head = q_head_stride;
    p.block_table = block_table; p.table_stride = table_stride; p.width = (int)table_width;
    p.lengths = lengths; p.out = (uint16_t*)out; p.lse = lse;
    p.B = (int)B; p.Hq = (int)Hq; p.G = (int)(Hq / p.cache.heads);
    const int DP = padded_dim(p.cache.D), NT = head_tiles(p.G);
    p.chunks = (int)ceil_div(p.G, 8 * NT);
    p.units = p.cache.heads * p.chunks;
    p.window = (int)std::min<int64_t>(window, INT32_MAX);
    p.scale_log2 = softmax_scale * 1.44269504088896341f;
    p.whole_pages = p.cache.page_size % kRows == 0;
    cudaStream_t s = (cudaStream_t)stream;
    if (p.cache.e4m3) return f16 ? launch_shape<true, true>(p, DP, NT, workspace, s) : launch_shape<false, true>(p, DP, NT, workspace, s);
    return f16 ? launch_shape<true, false>(p, DP, NT, workspace, s) : launch_shape<false, false>(p, DP, NT, workspace, s);
}
