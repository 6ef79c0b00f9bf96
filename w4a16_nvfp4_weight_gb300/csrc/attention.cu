// Attention of one new token per sequence over a paged key-value cache.
//
// For query head h of sequence b, with n = lengths[b] cached tokens:
//     z_j = softmax_scale * q . k_j   for max(0, n - window) <= j < n,
//     out = sum_j exp(z_j - lse) v_j,   lse = log sum_j exp(z_j),
// in one pass over the cache: a running maximum m, l = sum exp(z - m) and
// o = sum exp(z - m) v, all in 32 bits; two passes over different tokens join as
//     m = max(m1, m2),  l = l1 exp(m1 - m) + l2 exp(m2 - m),  o likewise.
// A row with no token gives out = 0 and lse = -infinity.
//
// Bound by the cache's bytes (2 G / element size flop a byte, G query heads a
// key head), so the kernel is built around keeping loads in flight:
//  - The unit of work is a step: 16 tokens of one key head.  All steps of all
//    sequences are numbered through (sequence, head, token) on the device, from
//    the lengths, and cut into equal contiguous ranges, one a warp of a grid
//    that fills the GPU once.  So a ragged batch, one long sequence and many
//    short ones all load every SM alike, and the host needs no length.
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
// a BF16 cache (a relative 2^-8 of each weight, while l keeps the 32-bit ones),
// FP16 for FP16 and E4M3.  E4M3 codes are exact in FP16; a BF16 query meets them
// as FP16 after a power of two that puts its largest element at 2^14 (elements
// below 2^-28 of it lose bits).  The scale of a value row is multiplied into its weight,
// whose running maximum is taken over z + log2(scale), so that it fits FP16.
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

constexpr int kStep = 16;          // tokens a step
constexpr size_t kSmemPerSm = 228 * 1024, kReservedPerCta = 1024, kMaxSmem = 227 * 1024;

struct AttnParams {
    const uint16_t* q;             // strides q_row, q_head (elements)
    int64_t q_row, q_head;
    const int32_t* block_table;    // [B, width], row stride table_stride
    int64_t table_stride;
    const int32_t* lengths;
    uint16_t* out;                 // [B, Hq, D]
    float* lse;                    // [B, Hq] or null
    float* parts;                  // workspace: partial results of blocks, then of warps
    int* joins;                    // workspace: [blocks][2], unit and last block of a unit that starts here and goes on
    int B, Hq, G, chunks, units;   // chunks: head groups of one key head; units = heads * chunks a sequence
    int width;
    bool whole_pages;              // a step lies in one page (page_size a multiple of 16)
    int window;                    // 0: none
    float scale_log2;              // softmax_scale * log2(e)
    int* status;
    CacheView cache;
};

// Shape of an instance: DP padded head size, NT tiles of 8 query heads.
template <bool E4M3, int DP, int NT>
struct Shape {
    static constexpr int kRow = DP * (E4M3 ? 1 : 2);            // bytes of a row in the ring
    static constexpr int kChunks = kRow / 16;                   // 16-byte chunks a row
    static constexpr int kTile = kStep * kRow;
    static constexpr int kStage = 2 * kTile + (E4M3 ? 2 * kStep * 4 : 0);
    // Warps and ring depth: as many bytes in flight as shared memory holds; the
    // 512-byte rows of 256 dimensions leave room for four warps.
    static constexpr int kWarps = kRow == 512 ? 4 : 8;
    static constexpr int kStages = kRow == 64 ? 4 : 3;
    static constexpr int kRing = kStages * kStage;
    static constexpr size_t kSmem = (size_t)kWarps * kRing;
    static constexpr int kByRing = (int)(kSmemPerSm / (kSmem + kReservedPerCta));
    static constexpr int kCtas = kByRing < 1 ? 1 : kByRing > 2 ? 2 : kByRing;
    static constexpr int kHeads = 8 * NT;
    static constexpr int kPart = kHeads * (DP + 2);             // floats of a partial result: o, m, l
    static_assert(kSmem <= kMaxSmem && kPart * 4 <= kRing, "ring");
};

// Partial results in the workspace: two a block, then one a warp.
inline size_t workspace_for(int row, int heads, int DP, int64_t sms) {
    const int warps = row == 512 ? 4 : 8;
    const size_t ctas = 2 * (size_t)sms;
    return round_up(ctas * 8, 256) + ctas * (2 + warps) * heads * (DP + 2) * sizeof(float);
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

// Tokens of sequence b that the table can hold; a length outside is recorded and clamped.
__device__ __forceinline__ int checked_length(const AttnParams& p, int b) {
    const int n = p.lengths[b];
    const int64_t most = (int64_t)p.width * p.cache.page_size;
    if (n < 0 || n > most) {
        record_status(p.status, NVFP4_ERR_BAD_INDEX);
        return n < 0 ? 0 : (int)most;
    }
    return n;
}
__device__ __forceinline__ int first_token(const AttnParams& p, int n) {
    return p.window > 0 ? max(0, n - p.window) : 0;
}
__device__ __forceinline__ int steps_of(const AttnParams& p, int n) {
    return (n + kStep - 1) / kStep - first_token(p, n) / kStep;
}

// A place in the numbering of steps: sequence, unit (key head and head group), step.
struct Place {
    int b, u, step, lo, n, s_lo, s_hi;     // tokens [lo, n), steps [s_lo, s_hi) of the sequence

    __device__ __forceinline__ void sequence(const AttnParams& p) {
        n = checked_length(p, b);
        lo = first_token(p, n);
        s_lo = lo / kStep;
        s_hi = (n + kStep - 1) / kStep;
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

// The steps' ranges: the first `rest` warps have one step more than the others
// (fewer steps than warps: one step a warp, packed into the first blocks).
struct Ranges {
    int each, rest;
    __device__ __forceinline__ Ranges(int total, int warps) : each(total / warps), rest(total % warps) {}
    __device__ __forceinline__ int start(int w) const { return w * each + min(w, rest); }
    // The warp whose range holds step x.
    __device__ __forceinline__ int holder(int x) const {
        const int big = rest * (each + 1);
        return x < big ? x / (each + 1) : rest + (x - big) / each;
    }
};

template <bool F16, bool E4M3, int DP, int NT>
__global__ void __launch_bounds__(Shape<E4M3, DP, NT>::kWarps * 32, Shape<E4M3, DP, NT>::kCtas)
attend_kernel(const AttnParams p) {
    using S = Shape<E4M3, DP, NT>;
    constexpr int W = S::kWarps, CH = S::kChunks, KS = DP / 16;
    constexpr bool H = F16 || E4M3;                             // FP16 operands in the MMAs
    extern __shared__ __align__(1024) uint8_t ring_all[];
    __shared__ int scan_sm[W];
    __shared__ int start_sm[W][2];                              // sequence of a warp's first step, and its first step
    __shared__ int piece_unit[2 * W], piece_lo[2 * W], piece_hi[2 * W];

    pdl_wait_previous();
    pdl_launch_dependents();                                    // the joining kernel waits for this one's end

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, q4 = lane & 3;
    const int warps = gridDim.x * W, gw = blockIdx.x * W + warp;
    const int D = p.cache.D;

    // ---- number the steps: a scan over the sequences' lengths
    int total, a, e;
    {
        const int per = (p.B + W * 32 - 1) / (W * 32);
        const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
        int mine = 0;
        for (int b = b0; b < b1; ++b) mine += steps_of(p, checked_length(p, b)) * p.units;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        if (lane == 31) scan_sm[warp] = incl;
        __syncthreads();
        int before = 0;
        total = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w < warp) before += scan_sm[w];
            total += scan_sm[w];
        }
        int at = before + incl - mine;
        if (mine > 0) {
            int starts[W];
            const Ranges ranges(total, warps);
#pragma unroll
            for (int w = 0; w < W; ++w) starts[w] = ranges.start(blockIdx.x * W + w);
            if (starts[0] < at + mine && starts[W - 1] >= at) {
                for (int b = b0; b < b1; ++b) {
                    const int n = steps_of(p, checked_length(p, b)) * p.units;
#pragma unroll
                    for (int w = 0; w < W; ++w)
                        if (starts[w] >= at && starts[w] < at + n) {
                            start_sm[w][0] = b;
                            start_sm[w][1] = at;
                        }
                    at += n;
                }
            }
        }
        const Ranges ranges(total, warps);
        a = ranges.start(gw);
        e = ranges.start(gw + 1);
        __syncthreads();
    }

    // ---- sequences without a token
    for (int b = gw; b < p.B; b += warps) {
        if (steps_of(p, checked_length(p, b)) > 0) continue;
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
    int head_unit = -1, head_lo = 0, head_hi = 0, tail_unit = -1, tail_lo = 0, tail_hi = 0;

    if (a < e) {
        const int held_chunks = D * (E4M3 ? 1 : 2) / 16;
        Place f;                                                // the next step to copy
        f.b = start_sm[warp][0];
        f.sequence(p);
        {
            const int in = a - start_sm[warp][1], steps = f.s_hi - f.s_lo;
            f.u = in / steps;
            f.step = f.s_lo + in % steps;
        }
        Place c = f;                                            // the step to compute
        int unit_start = a - (c.step - c.s_lo);                 // global number of the unit's first step

        // The page of a step's tokens (lane l: of token l % 16) is loaded well before its rows.
        struct Rows { int page, at, kh, b_lo, b_n; };           // at: place in the page; token range as offsets from the step's first
        auto locate = [&](const Place& f) {
            Rows r;
            const int t = f.step * kStep + (p.whole_pages ? 0 : lane & 15);
            r.kh = p.chunks == 1 ? f.u : f.u / p.chunks;
            r.b_lo = f.lo - f.step * kStep;
            r.b_n = f.n - f.step * kStep;
            r.page = 0;
            r.at = 0;
            if (p.whole_pages || (t >= f.lo && t < f.n)) {
                const int i = p.cache.page_shift >= 0 ? t >> p.cache.page_shift : t / p.cache.page_size;
                r.at = t - i * p.cache.page_size;
                r.page = p.block_table[f.b * p.table_stride + i];
            }
            return r;
        };
        const int r0 = lane / CH, c0 = lane % CH;
        const int64_t lane_off = r0 * p.cache.token_bytes + c0 * 16;
        auto copy = [&](Rows r, int stage) {
            const uint32_t dst = ring_s + stage * S::kStage;
            if ((uint32_t)r.page >= (uint32_t)p.cache.num_pages) {
                record_status(p.status, NVFP4_ERR_BAD_INDEX);
                r.page = 0;
            }
            if (p.whole_pages) {                                // 16 rows of one page, evenly spaced
                const int64_t off = p.cache.row(r.page, r.kh, r.at) + lane_off;
                const uint8_t *k = p.cache.k + off, *v = p.cache.v + off;
                if (c0 < held_chunks) {
#pragma unroll
                    for (int i = 0; i < CH / 2; ++i) {          // 32 / CH rows an instruction
                        const int x = i * (32 / CH) + r0;
                        const bool held = x >= r.b_lo && x < r.b_n;
                        cp_async16(dst + x * S::kRow + key_chunk<E4M3, CH>(x, c0) * 16, k, held);
                        cp_async16(dst + S::kTile + x * S::kRow + value_chunk<E4M3, CH>(x, c0) * 16, v, held);
                        k += (32 / CH) * p.cache.token_bytes;
                        v += (32 / CH) * p.cache.token_bytes;
                    }
                }
                if (E4M3) {                                     // lanes 0-15 the keys' scales, 16-31 the values'
                    const int x = lane & 15;
                    cp_async4(dst + 2 * S::kTile + lane * 4,
                              (lane < 16 ? p.cache.k_scale : p.cache.v_scale) + p.cache.scale_at(r.page, r.kh, r.at) + x,
                              x >= r.b_lo && x < r.b_n);
                }
            } else {
                const int64_t off = p.cache.row(r.page, r.kh, r.at);
#pragma unroll
                for (int i = 0; i < CH / 2; ++i) {
                    const int x = i * (32 / CH) + r0;
                    const int64_t from = __shfl_sync(0xffffffffu, off, x) + c0 * 16;
                    const bool held = x >= r.b_lo && x < r.b_n;
                    if (c0 < held_chunks) {
                        cp_async16(dst + x * S::kRow + key_chunk<E4M3, CH>(x, c0) * 16, p.cache.k + from, held);
                        cp_async16(dst + S::kTile + x * S::kRow + value_chunk<E4M3, CH>(x, c0) * 16, p.cache.v + from, held);
                    }
                }
                if (E4M3)
                    cp_async4(dst + 2 * S::kTile + lane * 4,
                              (lane < 16 ? p.cache.k_scale : p.cache.v_scale) + p.cache.scale_at(r.page, r.kh, r.at),
                              (lane & 15) >= r.b_lo && (lane & 15) < r.b_n);
            }
        };
        // The first stages' pages are loaded together, then one step ahead.
        int next = a;                                           // number of the step that `ahead` belongs to
        Rows ahead;
        {
            Rows first[S::kStages];
#pragma unroll
            for (int s = 0; s < S::kStages; ++s) {
                if (next < e) {
                    first[s] = locate(f);
                    if (next + 1 < e) f.advance(p);
                    ++next;
                }
            }
#pragma unroll
            for (int s = 0; s < S::kStages - 1; ++s) {
                if (a + s < e) copy(first[s], s);
                cp_async_commit();
            }
            ahead = first[S::kStages - 1];
            next = a + S::kStages - 1;
        }

        uint32_t qf[KS][NT][2];
        float o[KS][NT][4], m[NT][2], l[NT][2], qs[NT][2];
        int stage = 0;
        bool fresh = true;                                      // a unit begins
        int seg_begin = a;
        for (int i = a; i < e; ++i) {
            if (fresh) {
                fresh = false;
                const int kh = p.chunks == 1 ? c.u : c.u / p.chunks;
                const int h0 = (c.u - kh * p.chunks) * S::kHeads;       // first head of the group
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int hg = h0 + nt * 8 + g;
                    const bool held = hg < p.G;
                    const uint16_t* qr = p.q + c.b * p.q_row + (int64_t)(kh * p.G + (held ? hg : 0)) * p.q_head;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int d = E4M3 ? ((ks >> 2) * 4 + q4) * 16 + (ks & 3) * 4 + x * 2 : ks * 16 + x * 8 + q4 * 2;
                            qf[ks][nt][x] = held && d < D ? *(const uint32_t*)(qr + d) : 0u;
                        }
                    qs[nt][0] = qs[nt][1] = p.scale_log2;
                    if (E4M3 && !F16) {
                        float top = 0.f;
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const float2 v = act2_to_f32<false>(qf[ks][nt][x]);
                                top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
                            }
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                        int ex = top > 0.f && top < INFINITY ? 14 - (int)((__float_as_uint(top) >> 23) & 255) + 127 : 0;
                        ex = min(ex, 100);
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
                    m[nt][0] = m[nt][1] = -INFINITY;
                    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
                    for (int mt = 0; mt < KS; ++mt)
#pragma unroll
                        for (int x = 0; x < 4; ++x) o[mt][nt][x] = 0.f;
                }
            }

            cp_async_wait<S::kStages - 2>();
            __syncwarp();                                       // the stage is whole, and every lane is done with the one before
            if (next < e) {
                copy(ahead, stage == 0 ? S::kStages - 1 : stage - 1);
                if (++next < e) {
                    ahead = locate(f);
                    if (next + 1 < e) f.advance(p);
                }
            }
            cp_async_commit();
            const uint32_t ks_s = ring_s + stage * S::kStage, vs_s = ks_s + S::kTile;
            stage = stage + 1 == S::kStages ? 0 : stage + 1;

            // ---- scores of 16 tokens (rows g, g + 8) x 8 heads (columns 2 q4, 2 q4 + 1)
            float z[NT][4], z2[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 4; ++x) z[nt][x] = z2[nt][x] = 0.f;
            if constexpr (!E4M3) {
                const int row = (lane & 7) + (lane & 8), ch = lane >> 4;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t af[4];
                    ldmatrix4(af, ks_s + row * S::kRow + key_chunk<E4M3, CH>(row, ks * 2 + ch) * 16);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_16816<H>(ks & 1 ? z2[nt] : z[nt], af, qf[ks][nt][0], qf[ks][nt][1]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < KS / 4; ++j) {
                    const uint4 w0 = lds128(ks_s + g * S::kRow + key_chunk<E4M3, CH>(g, j * 4 + q4) * 16);
                    const uint4 w1 = lds128(ks_s + (g + 8) * S::kRow + key_chunk<E4M3, CH>(g + 8, j * 4 + q4) * 16);
                    const uint32_t lo[4] = {w0.x, w0.y, w0.z, w0.w}, hi[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t af[4] = {e4m3x2_to_f16x2((uint16_t)lo[w]), e4m3x2_to_f16x2((uint16_t)hi[w]),
                                                e4m3x2_to_f16x2((uint16_t)(lo[w] >> 16)), e4m3x2_to_f16x2((uint16_t)(hi[w] >> 16))};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_16816<H>(w & 1 ? z2[nt] : z[nt], af, qf[j * 4 + w][nt][0], qf[j * 4 + w][nt][1]);
                    }
                }
            }

            // ---- softmax weights
            const int t0 = c.step * kStep + g;
            const bool held0 = t0 >= c.lo && t0 < c.n, held1 = t0 + 8 >= c.lo && t0 + 8 < c.n;
            float k0 = 1.f, k1 = 1.f, v0 = 1.f, v1 = 1.f, lv0 = 0.f, lv1 = 0.f;
            if (E4M3) {
                const uint32_t sc = ks_s + 2 * S::kTile;
                k0 = lds_f32(sc + g * 4); k1 = lds_f32(sc + g * 4 + 32);
                v0 = lds_f32(sc + 64 + g * 4); v1 = lds_f32(sc + 64 + g * 4 + 32);
                // a power of two above the scale: weights times scales stay below 1
                lv0 = (float)((int)((__float_as_uint(v0) >> 23) & 255) - 126);
                lv1 = (float)((int)((__float_as_uint(v1) >> 23) & 255) - 126);
            }
            uint32_t pf[NT][2];
            float keep[NT][2];
            bool grown = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float s[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    s[x] = (z[nt][x] + z2[nt][x]) * qs[nt][x & 1];
                    if (E4M3) s[x] *= x < 2 ? k0 : k1;
                    if (!(x < 2 ? held0 : held1)) s[x] = -INFINITY;
                }
                float w[4];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float top = fmaxf(s[x] + lv0, s[x + 2] + lv1);
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    const float to = fmaxf(m[nt][x], top);
                    const float base = to == -INFINITY ? 0.f : to;
                    keep[nt][x] = ex2(m[nt][x] - base);
                    grown |= to > m[nt][x];
                    m[nt][x] = to;
                    w[x] = ex2(s[x] - base);
                    w[x + 2] = ex2(s[x + 2] - base);
                    l[nt][x] = l[nt][x] * keep[nt][x] + (w[x] + w[x + 2]);
                }
                // heads on the MMA's columns: transpose the two 8x8 blocks
                pf[nt][0] = movmatrix(f32_to_act2<H>(w[0] * v0, w[1] * v0));
                pf[nt][1] = movmatrix(f32_to_act2<H>(w[2] * v1, w[3] * v1));
            }
            if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
                for (int mt = 0; mt < KS; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 4; ++x) o[mt][nt][x] *= keep[nt][x & 1];
            }

            // ---- output of 16 dimensions (rows) x 8 heads at a time
            if constexpr (!E4M3) {
                const int row = (lane & 7) + ((lane >> 4) << 3), ch = (lane >> 3) & 1;
#pragma unroll
                for (int mt = 0; mt < KS; ++mt) {
                    uint32_t af[4];
                    ldmatrix4_trans(af, vs_s + row * S::kRow + value_chunk<E4M3, CH>(row, mt * 2 + ch) * 16);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_16816<H>(o[mt][nt], af, pf[nt][0], pf[nt][1]);
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
                        const int r = 2 * q4 + (x & 1) + (x >> 1) * 8;
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
                            for (int nt = 0; nt < NT; ++nt)
                                mma_16816<H>(o[j * 8 + w * 2 + half][nt], af, pf[nt][0], pf[nt][1]);
                        }
                }
            }

            // ---- the end of a unit, or of the range
            const bool unit_end = c.step + 1 == c.s_hi, last = i + 1 == e;
            if (unit_end || last) {
                const int unit = c.b * p.units + c.u, unit_hi = unit_start + c.s_hi - c.s_lo;
                const int kh = p.chunks == 1 ? c.u : c.u / p.chunks;
                const int h0 = (c.u - kh * p.chunks) * S::kHeads;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], 4);
                        l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], 8);
                        l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], 16);
                    }
                if (unit_end && seg_begin == unit_start) {      // all of it: the result
                    const int64_t row = (int64_t)c.b * p.Hq + kh * p.G;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int hg = h0 + nt * 8 + q4 * 2 + x;
                            if (hg >= p.G) continue;
                            const float inv = 1.f / l[nt][x];
#pragma unroll
                            for (int mt = 0; mt < KS; ++mt)
#pragma unroll
                                for (int half = 0; half < 2; ++half) {
                                    const int d = out_dim<E4M3, DP>(mt, half, g);
                                    if (d < D) p.out[(row + hg) * D + d] = f32_to_act_bits<F16>(o[mt][nt][half * 2 + x] * inv);
                                }
                            if (p.lse && g == 0) p.lse[row + hg] = (m[nt][x] + log2f(l[nt][x])) * 0.693147180559945309f;
                        }
                } else {
                    // A piece of a unit.  The last one of the range goes to the ring, where
                    // nothing is in flight any more; one before (the rest of a unit that an
                    // earlier warp began) to the workspace.
                    float* part = warp_parts + (size_t)gw * S::kPart;
                    if (last) {
                        cp_async_wait<0>();
                        __syncwarp();
                        part = (float*)ring;
                        tail_unit = unit; tail_lo = unit_start; tail_hi = unit_hi;
                    } else {
                        head_unit = unit; head_lo = unit_start; head_hi = unit_hi;
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int hl = nt * 8 + q4 * 2 + x;
#pragma unroll
                            for (int mt = 0; mt < KS; ++mt)
#pragma unroll
                                for (int half = 0; half < 2; ++half)
                                    part[hl * DP + out_dim<E4M3, DP>(mt, half, g)] = o[mt][nt][half * 2 + x];
                            if (g == 0) {
                                part[S::kHeads * DP + hl] = m[nt][x];
                                part[S::kHeads * (DP + 1) + hl] = l[nt][x];
                            }
                        }
                }
                unit_start = unit_hi;
                seg_begin = i + 1;
                fresh = true;
            }
            if (!last) c.advance(p);
        }
    }

    // ---- join the block's pieces
    if (lane == 0) {
        piece_unit[2 * warp] = head_unit; piece_lo[2 * warp] = head_lo; piece_hi[2 * warp] = head_hi;
        piece_unit[2 * warp + 1] = tail_unit; piece_lo[2 * warp + 1] = tail_lo; piece_hi[2 * warp + 1] = tail_hi;
    }
    __syncthreads();
    const Ranges ranges(total, warps);
    const int block_lo = ranges.start(blockIdx.x * W), block_hi = ranges.start(blockIdx.x * W + W);
    int goes_on = -1, goes_to = 0;
    for (int i = 0; i < 2 * W;) {
        const int unit = piece_unit[i];
        if (unit < 0) { ++i; continue; }
        const int lo = piece_lo[i], hi = piece_hi[i];
        int j = i + 1;
        while (j < 2 * W && (piece_unit[j] == unit || piece_unit[j] < 0)) ++j;
        const bool whole = lo >= block_lo && hi <= block_hi;
        float* to = p.parts + ((size_t)blockIdx.x * 2 + (lo < block_lo ? 0 : 1)) * S::kPart;
        if (!whole && lo >= block_lo) {
            goes_on = unit;
            goes_to = ranges.holder(hi - 1) / W;
        }
        const int b = unit / p.units, u = unit - b * p.units, kh = u / p.chunks, h0 = (u - kh * p.chunks) * S::kHeads;
        const int64_t row = (int64_t)b * p.Hq + kh * p.G + h0;
        const int heads = min(S::kHeads, p.G - h0);
        // a thread four dimensions of one head
        for (int x = tid * 4; x < heads * DP; x += W * 32 * 4) {
            const int hl = x / DP, d = x % DP;
            if (d >= D) continue;
            float top = -INFINITY, sum = 0.f;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int y = i; y < j; ++y) {
                if (piece_unit[y] < 0) continue;
                const float* part = y & 1 ? (const float*)(ring_all + (y >> 1) * S::kRing)
                                          : warp_parts + (size_t)(blockIdx.x * W + (y >> 1)) * S::kPart;
                const float mine = part[S::kHeads * DP + hl], to_top = fmaxf(top, mine);
                const float fo = top == to_top ? 1.f : ex2(top - to_top), fn = mine == to_top ? 1.f : ex2(mine - to_top);
                const float4 o = *(const float4*)(part + x);
                sum = sum * fo + part[S::kHeads * (DP + 1) + hl] * fn;
                v.x = v.x * fo + o.x * fn; v.y = v.y * fo + o.y * fn; v.z = v.z * fo + o.z * fn; v.w = v.w * fo + o.w * fn;
                top = to_top;
            }
            if (whole) {
                const float inv = 1.f / sum;
                *(uint2*)(p.out + (row + hl) * D + d) = make_uint2(f32_to_act2<F16>(v.x * inv, v.y * inv), f32_to_act2<F16>(v.z * inv, v.w * inv));
                if (p.lse && d == 0) p.lse[row + hl] = (top + log2f(sum)) * 0.693147180559945309f;
            } else {
                *(float4*)(to + x) = v;
                if (d == 0) {
                    to[S::kHeads * DP + hl] = top;
                    to[S::kHeads * (DP + 1) + hl] = sum;
                }
            }
        }
        i = j;
    }
    if (tid == 0) {
        p.joins[2 * blockIdx.x] = goes_on;
        p.joins[2 * blockIdx.x + 1] = goes_to;
    }
}

// Joins a unit that starts in block x and goes on, up to block joins[x][1]; a
// block a head, a thread a dimension.
template <bool F16, int DP>
__global__ void __launch_bounds__(DP) join_kernel(const AttnParams p, int group) {
    pdl_wait_previous();
    const int x = blockIdx.x, hl = blockIdx.y, d = threadIdx.x, D = p.cache.D;
    const int unit = p.joins[2 * x], to = p.joins[2 * x + 1];
    if (unit < 0) return;
    const int b = unit / p.units, u = unit - b * p.units, kh = u / p.chunks, h0 = (u - kh * p.chunks) * group;
    if (h0 + hl >= p.G) return;
    const int size = group * (DP + 2), lane = threadIdx.x & 31;
    // Lane y holds the maximum and sum of piece y, 32 pieces at a time.
    const auto part = [&](int y) { return p.parts + ((size_t)y * 2 + (y == x)) * size; };
    float top = -INFINITY, sum = 0.f, v = 0.f;
    for (int y0 = x; y0 <= to; y0 += 32) {
        const int n = min(32, to + 1 - y0);
        const float mine = lane < n ? part(y0 + lane)[group * DP + hl] : -INFINITY;
        const float mass = lane < n ? part(y0 + lane)[group * (DP + 1) + hl] : 0.f;
        float high = mine;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
        high = fmaxf(high, top);
        const float fo = top == high ? 1.f : ex2(top - high), fn = mine == high ? 1.f : ex2(mine - high);
        sum *= fo;
        v *= fo;
        top = high;
#pragma unroll 8
        for (int y = 0; y < n; ++y) {
            const float f = __shfl_sync(0xffffffffu, fn, y);
            sum += f * __shfl_sync(0xffffffffu, mass, y);
            v += f * part(y0 + y)[hl * DP + d];
        }
    }
    if (d >= D) return;
    const int64_t row = (int64_t)b * p.Hq + kh * p.G + h0 + hl;
    p.out[row * D + d] = f32_to_act_bits<F16>(v / sum);
    if (p.lse && d == 0) p.lse[row] = (top + log2f(sum)) * 0.693147180559945309f;
}

template <bool F16, bool E4M3, int DP, int NT>
nvfp4_status launch_attention(AttnParams p, void* workspace, cudaStream_t stream) {
    using S = Shape<E4M3, DP, NT>;
    const char* fn = "nvfp4_paged_attention";
    const int64_t most = (int64_t)p.B * p.units * (ceil_div((int64_t)p.width * p.cache.page_size, kStep) + 1);
    if (most > INT32_MAX)
        return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: %lld steps of 16 tokens and heads in one call, above 2^31", fn, (long long)most);
    // as many blocks as the longest lengths could use, at most one wave
    const int ctas = (int)std::max<int64_t>(1, std::min<int64_t>((int64_t)sm_count() * S::kCtas, ceil_div(most, S::kWarps)));
    p.joins = (int*)workspace;
    p.parts = (float*)((uint8_t*)workspace + round_up((int64_t)ctas * 8, 256));
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
    if (ctas == 1) return NVFP4_OK;                             // nothing goes on
    cfg.gridDim = dim3((unsigned)ctas, (unsigned)std::min(S::kHeads, p.G));
    cfg.blockDim = dim3(DP);
    cfg.dynamicSmemBytes = 0;
    return check_cuda(cudaLaunchKernelEx(&cfg, join_kernel<F16, DP>, p, (int)S::kHeads), fn);
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
    const int DP = padded_dim(head_dim), group = 8 * head_tiles(Hq / heads);
    return std::max(workspace_for(2 * DP, group, DP, sm_count()), workspace_for(DP, group, DP, sm_count()));
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
    p.whole_pages = p.cache.page_size % kStep == 0;
    cudaStream_t s = (cudaStream_t)stream;
    if (p.cache.e4m3) return f16 ? launch_shape<true, true>(p, DP, NT, workspace, s) : launch_shape<false, true>(p, DP, NT, workspace, s);
    return f16 ? launch_shape<true, false>(p, DP, NT, workspace, s) : launch_shape<false, false>(p, DP, NT, workspace, s);
}
