// The next token of each row of logits, from a given random number:
//     w_i = exp((l_i - max l) / T),
// over the top_k largest logits (equal ones rank by index), of those over the shortest
// prefix in that order that holds top_p of their mass, of those over w_i >= min_p; the
// token is the first of them, by index, whose running mass passes u times their mass.
//
// A draw is a comparison of sums of up to a few hundred thousand weights with a random
// threshold: with 32-bit sums one draw in a hundred would fall on the wrong side of a
// border, another one for another order of the sums.  So weights are whole numbers of
// 2^-43 (of the largest weight), before that rounding right to 2^-29.9 of their value (2^-31.7 in the mean square), and sums of them
// are exact in 64 bits, in any order and by any block.  (top_p among many candidates of top_k is cut by sums rounded for
// each bin instead of each weight: within 2^-32 of the mass of what few candidates are cut by.)
//
// A cluster of one to eight blocks has a row, which stays in shared memory where it fits, so it is read
// once.  No sort of the row:
//  - top_k: each lane's largest logit is counted in a bin by its distance from the row's
//    largest; the bin in which that count reaches top_k has the k-th largest logit in it or
//    above, and the few logits from there up go to one block, which sorts and draws.
//  - top_p: every weight is added to its bin's mass; the values of the one bin in which the
//    running mass reaches top_p are divided by their keys, as a list or, where too many, in place.
//  - the draw: masses of warps, of blocks and of the row; the warp whose part holds the
//    target finds the step, the lane and the element.
// Bound by latency for few rows (1 x 151936 with top_k and top_p 10.4 us: the load, four meetings
// of the cluster, two sorts; greedy 3.0), by instructions for many (256 x 100003 logits of 32 bits: by top_p 92
// a logit, two additions in shared memory among them, 146 us, 0.7 TB/s; by temperature alone 49 and
// 81 us, by top_k 35 and 68; greedy rows 37 us).
#include <algorithm>

#include "common.cuh"
#include "launch.cuh"
#include "numeric.cuh"
#include "overlap.cuh"
#include "ptx.cuh"

namespace nvfp4 {
namespace {

constexpr int kSampleThreads = 512;
constexpr int kSampleWarps = kSampleThreads / 32;
constexpr int kBins = 1024;                // of the histogram
constexpr int kList = 1024;                // values of a list at most
constexpr int kMaxCluster = 8;
constexpr int kStages = 4;                 // steps of a warp in flight or in use, of rows that are not held
constexpr int64_t kHeldBytes = 86 * 1024;  // of a block's logits that stay in shared memory, with another block beside it
constexpr int kOneLog2 = 43;               // a weight of one is 2^43: 2^20 of them sum inside 63 bits
constexpr int64_t kMaxVocabulary = 1 << 20;

// 2^30 * 2^(j / 512), from the series of exp: a step of the table leaves three terms for the rest.
struct Exp2Table {
    uint32_t v[512];
    constexpr Exp2Table() : v() {
        for (int j = 0; j < 512; ++j) {
            const double x = j * (0.693147180559945309417232121458 / 512);
            double sum = 1, term = 1;
            for (int n = 1; n < 24; ++n) {
                term *= x / n;
                sum += term;
            }
            v[j] = (uint32_t)(sum * 1073741824.0 + 0.5);
        }
    }
};
__device__ const Exp2Table kExp2 = Exp2Table();
static_assert(kSampleThreads == 512, "a thread an entry of the table");

struct SampleParams {
    const void* logits;
    int64_t stride;
    const float* u;
    nvfp4_sampling how;
    int64_t* tokens;
    float* logprobs;
    int V, chunk;                          // chunk: virtual elements of a warp, a multiple of 256
};

// A number whose last bit is worth one: added to a float below 2^22, it leaves the nearest
// whole number in the low bits, at a quarter of a conversion's time.
constexpr float kWhole = 12582912.f;
constexpr int kWholeBits = 0x4B400000;

// Entry of the table: 2^30 * 2^(j / 512) less kWholeBits, and as a float.
__device__ __forceinline__ uint2 table_entry(uint32_t v) { return make_uint2(v - (uint32_t)kWholeBits, __float_as_uint((float)v)); }

// A weight of w * 2^(13 - s) units, w in [2^30, 2^31]: s factors of two below the largest.  n - kWholeBits is its
// place in 512ths of a factor of two, rounded; s and the bin go by its leading bits.
struct Weight {
    uint32_t w;
    int n;

    // The bins cut a factor of two into 16, and each belongs to one s.
    __device__ __forceinline__ int bin() const { return (kWholeBits >> 5) - (n >> 5); }
    __device__ __forceinline__ static uint32_t power(int e) {      // 2^e, zero outside [0, 31]
        uint32_t v;
        asm("shl.b32 %0, 1, %1;" : "=r"(v) : "r"(e));
        return v;
    }
    // To the nearest whole number: up to s = 13 a product, then the high word of one; either power is
    // zero where the other is not.
    __device__ __forceinline__ uint64_t units() const {
        const uint32_t down = power((n >> 9) + (45 - (kWholeBits >> 9)));
        return (uint64_t)w * power((n >> 9) + (13 - (kWholeBits >> 9))) + (uint32_t)(((uint64_t)w * down + 0x80000000u) >> 32);
    }
};
__device__ __forceinline__ int shift_of_bin(int bin) { return ((bin + 15) >> 4) - 13; }        // s - 13

// Weights of a row's logits as whole numbers, and places below the largest, in 32 bits; times
// 2^(rounding of mh), which is the same for the whole row and falls out of every ratio.
struct NearScale {
    float ch, cl;                          // log2(e) / T = ch + cl
    float mh;                              // that times the largest logit, to a 512th
    float low;                             // 47 factors of two below it: weighs nothing, and no logit is taken as less

    __device__ __forceinline__ bool set(float top, float t) {      // false: not in range
        ch = __fdiv_rn(1.44269502f, t);                            // log2(e) to 24 bits, and the rest of it
        cl = __fdiv_rn(fmaf(-ch, t, 1.44269502f) + 1.92596303e-8f, t);
        const float m = top * ch;
        mh = rintf(m * 512.f) * (1.f / 512.f);
        low = __fdiv_rn(mh - 47.f, ch);
        return fabsf(m) < 4096.f && ch > 0x1p-100f && ch < 0x1p100f;
    }
    __device__ __forceinline__ float tidy(float l) const { return fmaxf(l, low); }       // NaN, too
    __device__ __forceinline__ bool counts(float l) const { return l > low; }
    // Place below the largest in 512ths of a factor of two, as the low bits of a float: kWholeBits at
    // the largest, falling with l (each rounding keeps order).
    __device__ __forceinline__ int place(float l) const { return __float_as_int(fmaf(l, ch * 512.f, kWhole - mh * 512.f)); }
    __device__ __forceinline__ int bin(float l) const { return (kWholeBits >> 5) - (place(l) >> 5); }
    __device__ __forceinline__ float log_weight(float l) const { return fmaf(l, cl, fmaf(l, ch, -mh)) * 0.693147180559945f; }
    // 2^(l ch + l cl - mh): the nearest 512th by table, in 2^-30; the rest, below 2^-10 (and 2^-12
    // for l cl), by three terms of exp's series.  The rest itself is exact but for its last bit: mh plus a
    // 512th has no rounding.  So the table's and the product's roundings, half of 2^-30 each, are the error (2^-29.97
    // found over eight million logits).
    __device__ __forceinline__ void weights(float la, float lb, const uint2* table, Weight& wa, Weight& wb) const {
        const F2 l = make_f2(la, lb);
        const F2 whole = fma2(l, make_f2(ch * 512.f, ch * 512.f), make_f2(kWhole - mh * 512.f, kWhole - mh * 512.f));
        const F2 k = fma2(whole, make_f2(1.f, 1.f), make_f2(-kWhole, -kWhole));
        const F2 minus_s = fma2(k, make_f2(-1.f / 512.f, -1.f / 512.f), make_f2(-mh, -mh));
        const F2 rest = fma2(l, make_f2(cl, cl), fma2(l, make_f2(ch, ch), minus_s));
        constexpr float kLn2 = 0.693147180559945f;
        const F2 p = mul2(rest, fma2(rest, fma2(rest, make_f2(kLn2 * kLn2 * kLn2 / 6, kLn2 * kLn2 * kLn2 / 6), make_f2(kLn2 * kLn2 / 2, kLn2 * kLn2 / 2)),
                                     make_f2(kLn2, kLn2)));
        const float2 n = both(whole);
        wa.n = __float_as_int(n.x);
        wb.n = __float_as_int(n.y);
        const uint2 ea = table[wa.n & 511], eb = table[wb.n & 511];
        const float2 v = both(fma2(make_f2(__uint_as_float(ea.y), __uint_as_float(eb.y)), p, make_f2(kWhole, kWhole)));
        wa.w = ea.x + __float_as_uint(v.x);
        wb.w = eb.x + __float_as_uint(v.y);
    }
    __device__ __forceinline__ Weight weight(float l, const uint2* table) const {
        Weight a, b;
        weights(l, l, table, a, b);
        return a;
    }
};

// The same for rows whose products leave that range (temperatures next to zero, logits of 10^30 or
// infinity): 64-bit floating point, an exponential each.
__device__ __noinline__ double far_place(double c, float top, float l) {
    if (l == top) return 0.0;
    const double x = l == -INFINITY ? -INFINITY : ((double)l - (double)top) * c;   // zero times infinity: far below
    return fmax(x, -47.0);
}
__device__ __noinline__ Weight far_weight(double x) {
    const int k = (int)floor(x * 512.0);
    return Weight{(uint32_t)__double2ll_rn(exp2(x - (double)(k >> 9)) * 1073741824.0), kWholeBits + k};
}
struct FarScale {
    double c;
    float top;

    __device__ __forceinline__ void set(float top_, float t) {
        top = top_;
        c = 1.4426950408889634074 / (double)t;
    }
    __device__ __forceinline__ float tidy(float l) const { return fmaxf(l, -INFINITY); }
    __device__ __forceinline__ bool counts(float l) const { return far_place(c, top, l) > -47.0; }
    __device__ __forceinline__ int bin(float l) const { return -((int)floor(far_place(c, top, l) * 512.0) >> 5); }
    __device__ __forceinline__ float log_weight(float l) const { return (float)(far_place(c, top, l) * 0.69314718055994530942); }
    __device__ __forceinline__ Weight weight(float l, const uint2*) const { return far_weight(far_place(c, top, l)); }
    __device__ __forceinline__ void weights(float la, float lb, const uint2* table, Weight& wa, Weight& wb) const {
        wa = weight(la, table);
        wb = weight(lb, table);
    }
};
constexpr int kDeadBin = 16 * (kOneLog2 + 3);              // what lies in bins from here on weighs nothing

// Floats as whole numbers in the same order, the two zeros as one.
__device__ __forceinline__ uint32_t order_key(float l) {
    const uint32_t b = __float_as_uint(l + 0.f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

// Whole part of f * s for 0 <= f < 1, rounded up where asked: f is a 24-bit whole number
// and a power of two.
__device__ __forceinline__ uint64_t part_of(float f, uint64_t s, bool up) {
    if (!(f > 0.f)) return 0;
    const int e = (int)(__float_as_uint(f) >> 23);
    const uint64_t digits = e ? (__float_as_uint(f) & 0x7fffffu) | 0x800000u : __float_as_uint(f) & 0x7fffffu;
    const int shift = 150 - (e ? e : 1);                    // f = digits * 2^-shift, shift >= 24
    const uint64_t lo = digits * s, hi = __umul64hi(digits, s);
    if (shift >= 128) return up ? 1 : 0;                    // hi < 2^24, s < 2^64: the product is below 2^88
    uint64_t q, rest;
    if (shift >= 64) {
        q = shift == 64 ? hi : hi >> (shift - 64);
        rest = lo | (shift == 64 ? 0 : hi << (128 - shift));
    } else {
        q = (hi << (64 - shift)) | (lo >> shift);
        rest = lo << (64 - shift);
    }
    return q + (up && rest != 0);
}

// a / b, and what is missing from it: 0 <= a <= b < 2^63.
__device__ __forceinline__ float2 ratio(uint64_t a, uint64_t b) {
    const float ah = (float)a, bh = (float)b;
    const float al = (float)(int64_t)(a - (uint64_t)ah), bl = (float)(int64_t)(b - (uint64_t)bh);
    const float q = __fdiv_rn(ah, bh);
    return make_float2(q, __fdiv_rn(fmaf(-q, bh, ah) + fmaf(-q, bl, al), bh));
}

enum { kTypeBf16, kTypeF16, kTypeF32 };

// The row's virtual elements, in 16-byte pieces: element 0 is on a boundary of eight elements.  A warp
// takes them in steps of 256, each piece of a step (one of eight elements a lane, or two of four) as 512
// bytes side by side.
template <int TYPE>
struct Row {
    static constexpr int kSize = TYPE == kTypeF32 ? 4 : 2;
    static constexpr int kPieces = kSize / 2, kPer = 8 / kPieces;
    static constexpr int kStageBytes = 512 * kPieces;
    const uint8_t* base;
    int first, end;                        // virtual elements that are the row's

    __device__ __forceinline__ Row(const void* logits, int64_t offset, int V) {
        const uint8_t* p = (const uint8_t*)logits + offset * kSize;
        first = (int)(((uintptr_t)p & (8 * kSize - 1)) / kSize);
        base = p - first * kSize;
        end = first + V;
    }
    __device__ __forceinline__ float one(int j) const {
        return TYPE == kTypeF32 ? ((const float*)base)[j] : act_to_f32<TYPE == kTypeF16>(((const uint16_t*)base)[j]);
    }
    // Where element i of the eight lies that a lane has of the step at `at`.
    __device__ __forceinline__ static int index(int at, int i) { return at + i / kPer * 32 * kPer + (threadIdx.x & 31) * kPer + i % kPer; }

    // The piece from element j on, -infinity outside the row.
    __device__ __forceinline__ uint4 load(int j) const {
        if (j >= first && j + kPer <= end) return *(const uint4*)(base + (int64_t)j * kSize);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (TYPE == kTypeF32) {
                w[i] = j + i >= first && j + i < end ? ((const uint32_t*)base)[j + i] : 0xff800000u;
            } else {
                uint32_t h[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int at = j + 2 * i + k;
                    h[k] = at >= first && at < end ? ((const uint16_t*)base)[at] : TYPE == kTypeF16 ? 0xfc00u : 0xff80u;
                }
                w[i] = h[0] | h[1] << 16;
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // The same, to shared memory: asynchronous but at the row's ends.
    __device__ __forceinline__ void copy(int j, uint32_t to) const {
        if (j >= first && j + kPer <= end) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(base + (int64_t)j * kSize) : "memory");
            return;
        }
        const uint4 v = load(j);
        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
    }
    __device__ __forceinline__ static void widen(const uint4 (&v)[kPieces], float (&l)[8]) {
        const uint32_t* w = (const uint32_t*)v;
        if (TYPE == kTypeF32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) l[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = act2_to_f32<TYPE == kTypeF16>(w[i]);
                l[2 * i] = x.x;
                l[2 * i + 1] = x.y;
            }
        }
    }
    // This lane's eight of a step, from its warp's stage `s` in shared memory.
    __device__ __forceinline__ static void fetch(uint32_t at, int s, float (&l)[8]) {
        uint4 v[kPieces];
#pragma unroll
        for (int k = 0; k < kPieces; ++k)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[k].x), "=r"(v[k].y), "=r"(v[k].z), "=r"(v[k].w)
                         : "r"(at + s * kStageBytes + k * 512) : "memory");
        widen(v, l);
    }
    __device__ __forceinline__ void stage(int at, int j1, uint32_t to, int s) const {
        if (at < j1)
#pragma unroll
            for (int k = 0; k < kPieces; ++k) copy(index(at, k * kPer), to + s * kStageBytes + k * 512);
    }
    // f(eight logits, the step's first element) over the elements j0 to j1 (multiples of 256 after j0, or the
    // row's end) of a warp, whose stages begin at `at`.  A lane reads what it copied.  HELD: the warp's part has
    // a stage for every step, so it is copied once (`first`) and stays; else three steps are on their way
    // ahead of f, every time.
    template <bool HELD, class F>
    __device__ __forceinline__ void each(int j0, int j1, uint32_t at, bool first, F f) const {
        if (HELD) {
            const int half = (j1 - j0) / 512 * 256 + j0;
            if (first) {
                for (int j = j0; j < half; j += 256) stage(j, j1, at, (j - j0) >> 8);
                asm volatile("cp.async.commit_group;" ::: "memory");
                for (int j = half; j < j1; j += 256) stage(j, j1, at, (j - j0) >> 8);
                asm volatile("cp.async.commit_group;" ::: "memory");
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            }
            int s = 0;
            for (int j = j0; j < j1; j += 256, ++s) {
                if (first && j == half) asm volatile("cp.async.wait_group 0;" ::: "memory");
                float l[8];
                fetch(at, s, l);
                f(l, j);
            }
            return;
        }
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) {
            stage(j0 + s * 256, j1, at, s);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        int s = 0;
        for (int j = j0; j < j1; j += 256) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
            float l[8];
            fetch(at, s, l);
            stage(j + (kStages - 1) * 256, j1, at, (s + kStages - 1) % kStages);
            asm volatile("cp.async.commit_group;" ::: "memory");
            s = (s + 1) % kStages;
            f(l, j);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __device__ __forceinline__ static float largest(const float (&l)[8]) {
        return fmaxf(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])), fmaxf(fmaxf(l[4], l[5]), fmaxf(l[6], l[7])));
    }
};

// Where the kept tokens of a row end: every logit above `value`, and of those equal to it the
// first `ties`, by index.
struct Cut {
    float value;
    uint32_t ties;
};

struct Shared {
    uint2 table[512];
    uint32_t count[kBins];
    alignas(8) uint32_t lo[kBins], hi[kBins];
    union {
        uint64_t pairs[kList];             // logits with their indices, of a row with few candidates
        uint32_t list[2][kList];           // values of a bin, as keys: of this block; of the whole row
    };
    uint32_t listed, paired, few[kMaxCluster];
    uint32_t key_range[2];                 // least and largest key of a bin
    uint64_t scan[kSampleWarps];
    uint64_t found[3];
    float best[kMaxCluster];               // pushed here by every block of the row, as the next ones
    int best_at[kMaxCluster];
    uint64_t mass[kMaxCluster];
    uint32_t ties[kMaxCluster];
    float warp_best[kSampleWarps];
    int warp_at[kSampleWarps];
    uint64_t warp_mass[kSampleWarps];
    uint32_t warp_ties[kSampleWarps];
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_ranks() {
    uint32_t n;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}
__device__ __forceinline__ uint32_t remote_u32(const void* p, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_rank(smem_u32(p), rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint2 remote_u32x2(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void push_u32(void* p, uint32_t rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_rank(smem_u32(p), rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void push_u64(void* p, uint32_t rank, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(map_rank(smem_u32(p), rank)), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t remote_add(void* p, uint32_t rank, uint32_t v) {
    uint32_t old;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(map_rank(smem_u32(p), rank)), "r"(v) : "memory");
    return old;
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    cluster_arrive();
    cluster_wait();
}

template <class T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <class T>
__device__ __forceinline__ T warp_below(T v, int lane) {          // sum over lower lanes
    T x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x - v;
}

// Sum over the threads below this one; `all`: over all of them.
__device__ __forceinline__ uint64_t block_below(uint64_t v, uint64_t (&sm)[kSampleWarps], uint64_t* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t x = warp_below(v, lane);
    if (lane == 31) sm[warp] = x + v;
    __syncthreads();
    uint64_t below = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kSampleWarps; ++w) {
        if (w == warp) below = sum;
        sum += sm[w];
    }
    __syncthreads();
    *all = sum;
    return x + below;
}

// n <= kList values from the largest down, in place, by the whole block.  Up to 256 by counting what goes before
// each (100 values 0.4 us where exchanges took 2.7; 512 would take 5), more by exchanges; room for kList,
// zeros are the least.
__device__ __forceinline__ void sort_down(uint64_t* v, int n) {
    const int tid = threadIdx.x;
    if (n <= kSampleThreads / 2) {
        int each_log2 = 4;                                  // threads of a value: at most 16
        while (kSampleThreads >> each_log2 < n) --each_log2;
        const int i = tid >> each_log2, each = 1 << each_log2;
        const uint64_t mine = i < n ? v[i] : 0;
        int before = 0;
        for (int j = tid & (each - 1); j < n; j += each) {
            const uint64_t x = v[j];
            before += x > mine || (x == mine && j < i);
        }
        for (int o = each >> 1; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
        __syncthreads();
        if (i < n && (tid & (each - 1)) == 0) v[before] = mine;
        __syncthreads();
        return;
    }
    const int size = n <= kSampleThreads ? kSampleThreads : kList;
    for (int i = n + tid; i < size; i += kSampleThreads) v[i] = 0;
    __syncthreads();
    for (int k = 2; k <= size; k *= 2)
        for (int s = k / 2; s > 0; s /= 2) {
            const int a = 2 * tid - (tid & (s - 1)), b = a + s;
            if (a < size) {
                const uint64_t x = v[a], y = v[b];
                if ((x < y) == ((a & k) == 0)) {
                    v[a] = y;
                    v[b] = x;
                }
            }
            // A warp's pairs lie in 64 values of its own up to 32 apart.
            if (s <= 32 && (s > 1 || k < 64)) __syncwarp();
            else __syncthreads();
        }
}
static_assert(kList == 2 * kSampleThreads, "a pair a thread");

constexpr int kOwnBins = kBins / kSampleThreads;           // bins of a thread when they are summed

struct Bins {                              // of one thread
    uint64_t of[kOwnBins];
    __device__ __forceinline__ uint64_t& operator[](int k) { return of[k]; }
    __device__ __forceinline__ const uint64_t& operator[](int k) const { return of[k]; }
};

// A bin where a running sum reaches a target: what it holds, and what goes before it.
struct Reached {
    int bin;
    uint64_t here, before;
};

template <int TYPE, bool HELD, class SCALE>
struct Sampler {
    Shared& sm;
    Row<TYPE> row;
    uint32_t stages;                       // shared address of this lane's first piece
    uint32_t rank, ranks;
    int j0, j1;                            // virtual elements of this warp
    bool large;                            // more than 2^16 of a block
    SCALE scale;

    // f(eight logits, their largest, the step's first element) over this warp's elements.
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        row.template each<HELD>(j0, j1, stages, false, [&](float (&l)[8], int j) { f(l, scale.tidy(Row<TYPE>::largest(l)), j); });
    }
    __device__ __forceinline__ void tidy(float (&l)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) l[i] = scale.tidy(l[i]);
    }

    __device__ __forceinline__ void clear() {
        cluster_sync();                                     // all have read the last histogram
        for (int i = threadIdx.x; i < kBins; i += kSampleThreads) sm.count[i] = sm.lo[i] = sm.hi[i] = 0;
        __syncthreads();
    }
    // Sums of this thread's two bins over the blocks, after a barrier of them.
    __device__ __forceinline__ void read(const uint32_t (&bins)[kBins], Bins& sum) const {
        static_assert(kOwnBins == 2, "read in pairs");
        uint2 v[kMaxCluster];
        const uint32_t at = smem_u32(&bins[threadIdx.x * 2]);
#pragma unroll
        for (uint32_t r = 0; r < kMaxCluster; ++r) v[r] = r < ranks ? remote_u32x2(map_rank(at, r)) : make_uint2(0, 0);
        sum[0] = sum[1] = 0;
#pragma unroll
        for (uint32_t r = 0; r < kMaxCluster; ++r) {
            sum[0] += v[r].x;
            sum[1] += v[r].y;
        }
    }

    // Counts of the lanes' largest logits.
    __device__ __forceinline__ void count_lanes(float most, Bins& count) {
        most = scale.tidy(most);
        if (scale.counts(most)) atomicAdd(&sm.count[scale.bin(most)], 1u);
        cluster_sync();
        read(sm.count, count);
    }
    // Counts of all logits of the row.
    __device__ __noinline__ static Bins count_all(Sampler s) {
        s.clear();
        Bins count;
        s.count(count);
        return count;
    }
    __device__ __forceinline__ void count(Bins& count) const {
        each([&](float (&l)[8], float, int) {
            tidy(l);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (scale.counts(l[i])) atomicAdd(&sm.count[scale.bin(l[i])], 1u);
        });
        cluster_sync();
        read(sm.count, count);
    }

    // A weight's share of a sum: its high and its low 16 bits apart, so that neither sum leaves 32 bits
    // (up to 2^16 logits a block) and nothing has to come back from shared memory; larger blocks carry.
    __device__ __forceinline__ void add(int at, uint32_t w) {
        if (!large) {
            atomicAdd(&sm.hi[at], w >> 16);
            atomicAdd(&sm.lo[at], w & 0xffffu);
        } else if (atomicAdd(&sm.lo[at], w) + w < w) {
            atomicAdd(&sm.hi[at], 1u);
        }
    }
    __device__ __forceinline__ void read_sums(Bins& sum) const {
        Bins lo;
        read(sm.hi, sum);
        read(sm.lo, lo);
#pragma unroll
        for (int k = 0; k < kOwnBins; ++k) sum[k] = (sum[k] << (large ? 32 : 16)) + lo[k];
    }
    // Mass of the row's bins, of what is up to `cut`, in units.  (Whole units of a bin, not of its weights:
    // where a unit is more than a weight's last bit the one differs from the other in that.)
    __device__ __forceinline__ void weigh_bins(const Cut& cut, Bins& mass) {
        const bool all = cut.value == -INFINITY;
        each([&](float (&l)[8], float most, int) {
            if (most < cut.value) return;
            tidy(l);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                Weight w[2];
                scale.weights(l[i], l[i + 1], sm.table, w[0], w[1]);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (scale.counts(l[i + k]) && (all || l[i + k] > cut.value)) add(w[k].bin(), w[k].w);
            }
        });
        cluster_sync();
        read_sums(mass);
        const Weight last = all ? Weight{0, kWholeBits} : scale.weight(cut.value, sm.table);
#pragma unroll
        for (int k = 0; k < kOwnBins; ++k) {
            const int b = (int)threadIdx.x * kOwnBins + k, down = shift_of_bin(b);
            if (!all && b == last.bin()) mass[k] += (uint64_t)cut.ties * last.w;
            mass[k] = down > 0 ? mass[k] >> down : mass[k] << -down;
        }
    }

    // The bin in which the running sum reaches the target; bin -1 where it never does.
    __device__ __forceinline__ Reached reach(const Bins& v, uint64_t target, uint64_t* all) {
        uint64_t mine = 0;
#pragma unroll
        for (int k = 0; k < kOwnBins; ++k) mine += v[k];
        if (threadIdx.x == 0) sm.found[0] = ~0ull;
        uint64_t sum = block_below(mine, sm.scan, all);
#pragma unroll
        for (int k = 0; k < kOwnBins; ++k) {
            if (sum < target && target <= sum + v[k]) {
                sm.found[0] = threadIdx.x * kOwnBins + k;
                sm.found[1] = v[k];
                sm.found[2] = sum;
            }
            sum += v[k];
        }
        __syncthreads();
        const Reached r{(int)sm.found[0], sm.found[1], sm.found[2]};
        __syncthreads();
        return r;
    }

    // Keys of a type of 16 bits end in bits that go by the sign alone.
    static constexpr int kDrop = TYPE == kTypeF32 ? 0 : TYPE == kTypeF16 ? 13 : 16;
    __device__ __forceinline__ static uint32_t short_key(float l) { return order_key(l) >> kDrop; }
    __device__ __forceinline__ static float short_value(uint32_t k) {
        const uint32_t key = k << kDrop;
        return key_value(key & 0x80000000u ? key : key | ((1u << kDrop) - 1));
    }
    // Counts, or sums of w, of one bin's logits by their keys' distance below `top`, up to `range`, in steps
    // of 2^shift.
    __device__ __forceinline__ void digits(int bin, uint32_t top, uint32_t range, int shift, bool by_mass, Bins& sum) {
        clear();
        each([&](float (&l)[8], float most, int) {
            if (scale.bin(most) > bin) return;
            tidy(l);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t d = top - short_key(l[i]);
                if (!scale.counts(l[i]) || scale.bin(l[i]) != bin || d > range) continue;
                if (by_mass) add((int)(d >> shift), scale.weight(l[i], sm.table).w);
                else atomicAdd(&sm.count[d >> shift], 1u);
            }
        });
        cluster_sync();
        if (by_mass) read_sums(sum);
        else read(sm.count, sum);
    }
    // The cut in a bin of more values than a list has, their keys within `range` below `top`: 1024 parts of
    // that, then of one part; one round does for logits of 16 bits.
    __device__ __noinline__ static Cut cut_by_digits(Sampler s, int bin, uint32_t top, uint32_t range, bool by_mass, uint64_t want) {
        for (int shift = 32;;) {
            shift = min(shift, range < kBins ? 0 : 22 - __clz(range));       // shorter every round: it ends
            Bins sum;
            uint64_t all;
            s.digits(bin, top, range, shift, by_mass, sum);
            const Reached r = s.reach(sum, want, &all);
            if (r.bin < 0) return ended(s, top, by_mass, want);             // never: the bin holds what is wanted
            want -= r.before;
            top -= (uint32_t)r.bin << shift;
            range = min(range - ((uint32_t)r.bin << shift), (1u << shift) - 1);
            if (shift == 0) return ended(s, top, by_mass, want);
        }
    }
    // The same of the n keys in the row's list, by every block for itself: no other reads its histogram any more.
    __device__ __forceinline__ Cut cut_of_list(uint32_t n, uint32_t top, uint32_t range, bool by_mass, uint64_t want) {
        for (int shift = 32;;) {
            shift = min(shift, range < kBins ? 0 : 22 - __clz(range));
            for (int i = threadIdx.x; i < kBins; i += kSampleThreads) sm.count[i] = sm.lo[i] = sm.hi[i] = 0;
            __syncthreads();
            for (uint32_t i = threadIdx.x; i < n; i += kSampleThreads) {
                const uint32_t k = sm.list[1][i], d = top - (k >> kDrop);
                if (d > range) continue;
                if (by_mass) add((int)(d >> shift), scale.weight(key_value(k), sm.table).w);
                else atomicAdd(&sm.count[d >> shift], 1u);
            }
            __syncthreads();
            Bins sum;
#pragma unroll
            for (int k = 0; k < kOwnBins; ++k) {
                const int at = threadIdx.x * kOwnBins + k;
                sum[k] = by_mass ? ((uint64_t)sm.hi[at] << (large ? 32 : 16)) + sm.lo[at] : sm.count[at];
            }
            uint64_t all;
            const Reached r = reach(sum, want, &all);
            if (r.bin < 0) return ended(*this, top, by_mass, want);         // never: the list holds what is wanted
            want -= r.before;
            top -= (uint32_t)r.bin << shift;
            range = min(range - ((uint32_t)r.bin << shift), (1u << shift) - 1);
            if (shift == 0) return ended(*this, top, by_mass, want);
        }
    }
    // All that is left has this key.
    __device__ __forceinline__ static Cut ended(const Sampler& s, uint32_t key, bool by_mass, uint64_t want) {
        const float value = short_value(key);
        const uint32_t each = by_mass ? s.scale.weight(value, s.sm.table).w : 1;
        return Cut{value, (uint32_t)((want + each - 1) / each)};
    }

    // The cut in `bin`, where the count (or, with `by_mass`, the sum of w) of its logits from the largest
    // down reaches `want`.
    __device__ __noinline__ static Cut cut_in(Sampler s, int bin, bool by_mass, uint64_t want) { return s.cut(bin, by_mass, want); }
    __device__ __forceinline__ Cut cut(int bin, bool by_mass, uint64_t want) {
        if (threadIdx.x == 0) {
            sm.listed = 0;
            sm.key_range[0] = ~0u;
            sm.key_range[1] = 0;
        }
        __syncthreads();
        uint32_t least = ~0u, top = 0;
        each([&](float (&l)[8], float most, int) {
            if (scale.bin(most) > bin) return;              // bins rise as logits fall
            tidy(l);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (scale.bin(l[i]) != bin || !scale.counts(l[i])) continue;
                const uint32_t at = atomicAdd(&sm.listed, 1u), k = short_key(l[i]);
                least = min(least, k);
                top = max(top, k);
                if (at < kList) sm.list[0][at] = order_key(l[i]);
            }
        });
        least = __reduce_min_sync(0xffffffffu, least);
        top = __reduce_max_sync(0xffffffffu, top);
        if ((threadIdx.x & 31) == 0 && least <= top) {
            atomicMin(&sm.key_range[0], least);
            atomicMax(&sm.key_range[1], top);
        }
        cluster_sync();
        uint32_t held[kMaxCluster], low[kMaxCluster], high[kMaxCluster], n = 0;
#pragma unroll
        for (uint32_t r = 0; r < kMaxCluster; ++r) {
            held[r] = r < ranks ? remote_u32(&sm.listed, r) : 0;
            low[r] = r < ranks ? remote_u32(&sm.key_range[0], r) : ~0u;
            high[r] = r < ranks ? remote_u32(&sm.key_range[1], r) : 0;
        }
        least = ~0u;
        top = 0;
#pragma unroll
        for (uint32_t r = 0; r < kMaxCluster; ++r) {
            n += held[r];
            least = min(least, low[r]);
            top = max(top, high[r]);
        }
        if (least == top) return ended(*this, top, by_mass, want);
        if (n > kList) return cut_by_digits(*this, bin, top, top - least, by_mass, want);
        uint32_t from = 0;
#pragma unroll
        for (uint32_t r = 0; r < kMaxCluster; ++r) {
            for (uint32_t i = threadIdx.x; i < held[r]; i += kSampleThreads) sm.list[1][from + i] = remote_u32(&sm.list[0][i], r);
            from += held[r];
        }
        __syncthreads();
        return cut_of_list(n, top, top - least, by_mass, want);
    }

    // The row's logits up to the bin `last`, which the top_k largest are among, as the candidates of the
    // first block; false where they are more than a list has.
    __device__ __forceinline__ bool collect(int last) {
        uint64_t* mine = (uint64_t*)sm.lo;                  // lo and hi: this block's, before they go to the first one
        static_assert(sizeof(sm.lo) + sizeof(sm.hi) == sizeof(sm.pairs), "as many");
        if (threadIdx.x == 0) sm.listed = 0;
        __syncthreads();
        each([&](float (&l)[8], float most, int j) {
            if (scale.bin(most) > last) return;             // bins rise as logits fall
            tidy(l);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (scale.bin(l[i]) <= last && scale.counts(l[i])) {
                    const uint32_t at = atomicAdd(&sm.listed, 1u);
                    if (at < kList) mine[at] = (uint64_t)order_key(l[i]) << 32 | (uint32_t)~(Row<TYPE>::index(j, i) - row.first);
                }
        });
        __syncthreads();
        const uint32_t m = sm.listed;
        if (threadIdx.x < ranks) push_u32(&sm.few[rank], threadIdx.x, m);
        if (threadIdx.x == 0) sm.found[0] = remote_add(&sm.paired, 0, m);
        __syncthreads();
        const uint32_t to = (uint32_t)sm.found[0];
        for (uint32_t i = threadIdx.x; i < m && to + i < kList; i += kSampleThreads) push_u64(&sm.pairs[to + i], 0, mine[i]);
        cluster_sync();
        uint32_t n = 0;
        for (uint32_t r = 0; r < ranks; ++r) n += sm.few[r];
        return n <= kList;
    }
    // A draw from them.  Sorted by value, then by index, they give the kept ones; sorted by index the token.
    __device__ __forceinline__ void draw_of_few(const SampleParams& p, int64_t b, float best, int top_k, float top_p, float min_p) {
        if (rank != 0) return;
        const uint32_t n = sm.paired;
        sort_down(sm.pairs, (int)n);
        const uint32_t i = threadIdx.x * 2;
        uint64_t w[2] = {0, 0}, all;
        float l[2] = {0.f, 0.f};
        if (i < n) {
            l[0] = key_value((uint32_t)(sm.pairs[i] >> 32));
            l[1] = i + 1 < n ? key_value((uint32_t)(sm.pairs[i + 1] >> 32)) : l[0];
            Weight x[2];
            scale.weights(l[0], l[1], sm.table, x[0], x[1]);
            for (uint32_t k = 0; k < 2; ++k) w[k] = i + k < min(n, (uint32_t)top_k) ? x[k].units() : 0;
        }
        if (top_p < 1.f) {
            uint64_t m = block_below(w[0] + w[1], sm.scan, &all);
            const uint64_t target = max(part_of(top_p, all, true), (uint64_t)1);
            for (uint32_t k = 0; k < 2; ++k) {              // what begins at or behind the target is not kept
                const uint64_t here = w[k];
                if (m >= target) w[k] = 0;
                m += here;
            }
        }
        const uint64_t least = least_weight(min_p, best);
        for (uint32_t k = 0; k < 2; ++k)
            if (i + k < n) {
                if (w[k] < least && l[k] != best) w[k] = 0;
                // By index: the largest first, and its complement in order.  Weights have 44 bits, indices 20.
                sm.pairs[i + k] = (uint64_t)(0xfffffu & (uint32_t)sm.pairs[i + k]) << 44 | w[k];
            }
        __syncthreads();
        sort_down(sm.pairs, (int)n);
        constexpr uint64_t kWeightBits = (1ull << 44) - 1;
        w[0] = i < n ? sm.pairs[i] & kWeightBits : 0;
        w[1] = i + 1 < n ? sm.pairs[i + 1] & kWeightBits : 0;
        uint64_t m = block_below(w[0] + w[1], sm.scan, &all);
        const float u = p.u[b];
        const uint64_t target = u < 1.f ? part_of(u, all, false) : all - 1;
        for (uint32_t k = 0; k < 2; ++k) {
            if (target >= m && target < m + w[k]) {
                const int at = 0xfffff - (int)(sm.pairs[i + k] >> 44);
                p.tokens[b] = at;
                if (p.logprobs) p.logprobs[b] = log_share(row.one(at + row.first), w[k], all);
            }
            m += w[k];
        }
    }

    __device__ __forceinline__ uint64_t least_weight(float min_p, float best) const {
        return min_p > 0.f ? min_p < 1.f ? part_of(min_p, scale.weight(best, sm.table).units(), true) : ~0ull : 0;
    }

    // From the largest logit to the token.
    __device__ __noinline__ static void draw_far(Sampler s, const SampleParams& p, int64_t b, float best, float most, int top_k, float top_p, float min_p) {
        s.draw(p, b, best, most, top_k, top_p, min_p);
    }
    __device__ __forceinline__ void draw(const SampleParams& p, int64_t b, float best, float most, int top_k, float top_p, float min_p) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        Cut cut{-INFINITY, 0};                              // everything
        const bool by_k = top_k > 0 && top_k < p.V, by_p = top_p < 1.f;
        Bins bins;
        uint64_t all;
        if (by_k) {
            // As many lanes as top_k have a logit of this bin or above, so the top_k largest are there, too.
            count_lanes(most, bins);
            Reached r = reach(bins, (uint64_t)top_k, &all);
            if (r.bin >= 0 && r.bin < kDeadBin && collect(r.bin)) return draw_of_few(p, b, best, top_k, top_p, min_p);
            bins = count_all(*this);
            r = reach(bins, (uint64_t)top_k, &all);
            if (r.bin >= 0 && r.bin < kDeadBin) cut = cut_in(*this, r.bin, false, (uint64_t)top_k - r.before);
            if (by_p) clear();
        }
        if (by_p) {
            weigh_bins(cut, bins);
            block_below(bins[0] + bins[1], sm.scan, &all);
            const uint64_t target = max(part_of(top_p, all, true), (uint64_t)1);
            const Reached r = reach(bins, target, &all);
            // From units to w, up: as much as makes a bin's units reach it.
            const int down = shift_of_bin(r.bin);
            const uint64_t want = target - r.before;
            cut = cut_in(*this, r.bin, true, down > 0 ? want << down : (want + (1ull << -down) - 1) >> -down);
        }

        // Mass of what is kept, over warps, blocks and the row; equal values at the cut count by index.
        const uint64_t least = least_weight(min_p, best);
        const auto kept = [&](float l, uint64_t w) -> uint64_t { return w >= least || l == best ? w : 0; };
        const auto kept_weight = [&](float l) -> uint64_t { return kept(l, scale.weight(l, sm.table).units()); };
        const uint64_t tie_weight = cut.value == -INFINITY ? 0 : kept_weight(cut.value);
        uint64_t mass = 0;
        uint32_t ties = 0;
        if (cut.value == -INFINITY && least == 0) {
            each([&](float (&l)[8], float, int) {
                tidy(l);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    Weight w[2];
                    scale.weights(l[i], l[i + 1], sm.table, w[0], w[1]);
                    mass += w[0].units();
                    mass += w[1].units();
                }
            });
        } else {
            each([&](float (&l)[8], float most, int) {
                if (most < cut.value) return;
                tidy(l);
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    if (fmaxf(l[i], l[i + 1]) < cut.value) continue;
                    Weight w[2];
                    scale.weights(l[i], l[i + 1], sm.table, w[0], w[1]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if (l[i + k] > cut.value) mass += kept(l[i + k], w[k].units());
                        ties += l[i + k] == cut.value;
                    }
                }
            });
        }
        mass = warp_sum(mass);
        ties = warp_sum(ties);
        if (lane == 0) {
            sm.warp_mass[warp] = mass;
            sm.warp_ties[warp] = ties;
        }
        __syncthreads();
        if (threadIdx.x < ranks) {
            uint64_t m = 0;
            uint32_t t = 0;
            for (int w = 0; w < kSampleWarps; ++w) {
                m += sm.warp_mass[w];
                t += sm.warp_ties[w];
            }
            push_u64(&sm.mass[rank], threadIdx.x, m);
            push_u32(&sm.ties[rank], threadIdx.x, t);
        }
        cluster_sync();
        // Mass of m above the cut and the t-th to (t + n)-th values equal to it.
        const auto with_ties = [&](uint64_t m, uint32_t t, uint32_t n) { return m + (min(t + n, cut.ties) - min(t, cut.ties)) * tie_weight; };
        uint64_t whole = 0, before = 0;
        uint32_t seen = 0, seen_before = 0;
        for (uint32_t r = 0; r < ranks; ++r) {
            if (r == rank) {
                before = whole;
                seen_before = seen;
            }
            whole += with_ties(sm.mass[r], seen, sm.ties[r]);
            seen += sm.ties[r];
        }
        const float u = p.u[b];
        const uint64_t target = u < 1.f ? part_of(u, whole, false) : whole - 1;
        seen = seen_before;
        for (int w = 0; w < warp; ++w) {
            before += with_ties(sm.warp_mass[w], seen, sm.warp_ties[w]);
            seen += sm.warp_ties[w];
        }
        // The warp that holds the running mass's passage goes through its values again.
        if (target < before || target >= before + with_ties(mass, seen, ties)) return;
        // First the step of 256, then the lane and the element.
        constexpr int kPer = Row<TYPE>::kPer, kPieces = Row<TYPE>::kPieces;
        float l[8];
        uint64_t w[8];
        int at = j0;
        for (int step = 0; at < j1; at += 256, ++step) {
            if (HELD) {
                Row<TYPE>::fetch(stages, step, l);
            } else {
                uint4 v[kPieces];
#pragma unroll
                for (int k = 0; k < kPieces; ++k) v[k] = row.load(Row<TYPE>::index(at, k * kPer));
                Row<TYPE>::widen(v, l);
            }
            tidy(l);
            uint64_t m = 0;
            uint32_t n = 0;
            if (__any_sync(0xffffffffu, Row<TYPE>::largest(l) >= cut.value)) {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    Weight x[2];
                    scale.weights(l[i], l[i + 1], sm.table, x[0], x[1]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        w[i + k] = l[i + k] > cut.value ? kept(l[i + k], x[k].units()) : 0;
                        m += w[i + k];
                        n += l[i + k] == cut.value;
                    }
                }
                m = warp_sum(m);
                n = warp_sum(n);
            }
            const uint64_t here = with_ties(m, seen, n);
            if (target < before + here) break;
            before += here;
            seen += n;
        }
        if (at >= j1) return;                               // never: the warp's mass reaches the target
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            uint64_t m = 0;
            uint32_t n = 0;
#pragma unroll
            for (int i = k * kPer; i < (k + 1) * kPer; ++i) {
                m += w[i];
                n += l[i] == cut.value;
            }
            uint32_t tie = seen + warp_below(n, lane);
            const uint64_t mine = with_ties(m, tie, n);
            uint64_t sum = before + warp_below(mine, lane);
            if (target >= sum && target < sum + mine) {
#pragma unroll
                for (int i = k * kPer; i < (k + 1) * kPer; ++i) {
                    const uint64_t here = l[i] == cut.value ? (tie++ < cut.ties ? tie_weight : 0) : w[i];
                    if (target >= sum && target < sum + here) {
                        p.tokens[b] = Row<TYPE>::index(at, i) - row.first;
                        if (p.logprobs) p.logprobs[b] = log_share(l[i], here, whole);
                    }
                    sum += here;
                }
            }
            before += warp_sum(mine);
            seen += warp_sum(n);
        }
    }

    // log(w / whole): near one by what is missing, from 2^24 units on by the quotient, else by the place.  Quotients
    // with what their roundings leave, so that the logarithm's own rounding is the error.
    __device__ __forceinline__ float log_share(float l, uint64_t w, uint64_t whole) const {
        if (w > whole / 2) {
            const float2 x = ratio(whole - w, whole);
            return log1pf(-x.x) - x.y / (1.f - x.x);
        }
        if (w >= 1u << 24) {
            const float2 x = ratio(w, whole);
            return logf(x.x) + x.y / x.x;
        }
        return scale.log_weight(l) - logf((float)whole * (1.f / (float)(1ull << kOneLog2)));
    }
};

template <int TYPE, bool HELD>
__global__ void __launch_bounds__(kSampleThreads, 2) sample_kernel(const SampleParams p) {
    extern __shared__ __align__(16) uint8_t sm_stages[];
    __shared__ Shared sm;
    cluster_arrive();                                       // that every block of the row runs: before the first push
    const uint32_t rank = cluster_rank(), ranks = cluster_ranks();
    const int64_t b = blockIdx.x / ranks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    sm.table[threadIdx.x] = table_entry(kExp2.v[threadIdx.x]);
    for (int i = threadIdx.x; i < kBins; i += kSampleThreads) sm.count[i] = sm.lo[i] = sm.hi[i] = 0;
    if (threadIdx.x == 0) sm.paired = 0;
    pdl_wait_previous();
    pdl_launch_dependents();
    const float temperature = p.how.temperature ? p.how.temperature[b] : p.how.temperature_all;
    const bool greedy = !(temperature > 0.f);
    const int top_k = p.how.top_k ? p.how.top_k[b] : p.how.top_k_all;
    const float top_p = p.how.top_p ? p.how.top_p[b] : p.how.top_p_all, min_p = p.how.min_p ? p.how.min_p[b] : p.how.min_p_all;
    const Row<TYPE> row(p.logits, b * p.stride, p.V);
    const int64_t start = ((int64_t)rank * kSampleWarps + warp) * p.chunk;
    const int j0 = (int)min(start, (int64_t)row.end), j1 = (int)min(start + p.chunk, (int64_t)row.end);

    const uint32_t stages = smem_u32(sm_stages) + warp * (HELD ? p.chunk >> 8 : kStages) * Row<TYPE>::kStageBytes + lane * 16;

    // The largest logit, the first of equal ones.
    float best = -INFINITY;
    int best_at = INT32_MAX;
    row.template each<HELD>(j0, j1, stages, true, [&](const float (&l)[8], int j) {
        const float m = Row<TYPE>::largest(l);
        if (m > best) {                                     // NaN is neither
            best = m;
            if (greedy) {
#pragma unroll
                for (int i = 7; i >= 0; --i)
                    if (l[i] == m) best_at = Row<TYPE>::index(j, i);
            }
        }
    });
    const float most = best;                                // of this lane
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, best, o);
        const int at = __shfl_xor_sync(0xffffffffu, best_at, o);
        if (other > best || (other == best && at < best_at)) {
            best = other;
            best_at = at;
        }
    }
    if (lane == 0) {
        sm.warp_best[warp] = best;
        sm.warp_at[warp] = best_at;
    }
    __syncthreads();
    cluster_wait();
    if (threadIdx.x < ranks) {
        best = -INFINITY;
        best_at = INT32_MAX;
        for (int w = 0; w < kSampleWarps; ++w)
            if (sm.warp_best[w] > best) {                   // warps are in index order
                best = sm.warp_best[w];
                best_at = sm.warp_at[w];
            }
        push_u32(&sm.best[rank], threadIdx.x, __float_as_uint(best));
        push_u32(&sm.best_at[rank], threadIdx.x, (uint32_t)best_at);
    }
    cluster_sync();
    best = -INFINITY;
    best_at = INT32_MAX;
    for (uint32_t r = 0; r < ranks; ++r)
        if (sm.best[r] > best) {
            best = sm.best[r];
            best_at = sm.best_at[r];
        }
    if (greedy || best == -INFINITY) {
        if (rank == 0 && threadIdx.x == 0) {
            const bool none = best == -INFINITY;
            p.tokens[b] = none ? -1 : best_at - row.first;
            if (p.logprobs) p.logprobs[b] = none ? -INFINITY : 0.f;
        }
        return;
    }
    NearScale near;
    if (near.set(best, temperature)) {
        Sampler<TYPE, HELD, NearScale>{sm, row, stages, rank, ranks, j0, j1, p.chunk > 65536 / kSampleWarps, near}.draw(p, b, best, most, top_k, top_p, min_p);
    } else {
        FarScale far;
        far.set(best, temperature);
        const Sampler<TYPE, HELD, FarScale> s{sm, row, stages, rank, ranks, j0, j1, p.chunk > 65536 / kSampleWarps, far};
        Sampler<TYPE, HELD, FarScale>::draw_far(s, p, b, best, most, top_k, top_p, min_p);
    }
}

template <int TYPE>
const void* sample_kernel_of(bool held) { return held ? (const void*)sample_kernel<TYPE, true> : (const void*)sample_kernel<TYPE, false>; }

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status nvfp4_sample(const void* logits, int64_t row_stride, int type, int64_t B, int64_t V, const float* u,
                                     const nvfp4_sampling* how, int64_t* tokens, float* logprobs, void* stream) {
    const char* fn = "nvfp4_sample";
    if (B < 0 || row_stride < 0) return fail(NVFP4_ERR_INVALID_ARG, "%s: negative size or stride (B=%lld, stride=%lld)", fn, (long long)B, (long long)row_stride);
    if (V < 1 || V > kMaxVocabulary) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: V=%lld must be in [1, 2^20]", fn, (long long)V);
    if (B > (1 << 24)) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: B=%lld too large", fn, (long long)B);
    if (type < NVFP4_LOGITS_BF16 || type > NVFP4_LOGITS_F32) return fail(NVFP4_ERR_INVALID_ARG, "%s: type=%d must be an nvfp4_logits_type", fn, type);
    if (!how) return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (B == 0) return NVFP4_OK;
    if (!logits || !u || !tokens) return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", fn);
    const int size = type == NVFP4_LOGITS_F32 ? 4 : 2;
    if (!aligned(logits, size) || !aligned(u, 4) || !aligned(tokens, 8) || !aligned(logprobs, 4) || !aligned(how->temperature, 4) ||
        !aligned(how->top_k, 4) || !aligned(how->top_p, 4) || !aligned(how->min_p, 4))
        return fail(NVFP4_ERR_ALIGNMENT, "%s: pointers must be aligned to their elements", fn);
    const Span rows = strided_span("logits", logits, size * V, {{B, size * row_stride}}), us = dense_span("u", u, 4 * B);
    const Span t = dense_span("tokens", tokens, 8 * B), lp = dense_span("logprobs", logprobs, 4 * B);
    for (const Span& out : {t, lp})
        if (const char* s = met(out, {rows, us, dense_span("temperature", how->temperature, 4 * B), dense_span("top_k", how->top_k, 4 * B),
                                      dense_span("top_p", how->top_p, 4 * B), dense_span("min_p", how->min_p, 4 * B)}))
            return fail(NVFP4_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, out.name, s);
    if (overlaps(t, lp)) return fail(NVFP4_ERR_INVALID_ARG, "%s: logprobs overlap tokens", fn);
    if (!device_status_ptr()) return fail(NVFP4_ERR_CUDA, "%s: no CUDA device", fn);
    // Blocks of a row: enough of them for every SM, none with less than 4096 logits, or more than 65536
    // where that can be; more, where each block's part then stays in shared memory: it is read from memory once.
    const auto chunk = [&](unsigned ranks) { return round_up(ceil_div(ceil_div(V + 7, ranks), kSampleWarps), 256); };
    const auto bytes = [&](unsigned ranks) { return chunk(ranks) * kSampleWarps * size; };
    unsigned ranks = 1;
    while (ranks < kMaxCluster && ((B * ranks < sm_count() && V / (2 * ranks) >= 4096) || chunk(ranks) > 65536 / kSampleWarps)) ranks *= 2;
    unsigned more = ranks;
    while (more < kMaxCluster && bytes(more) > kHeldBytes) ++more;
    const bool held = bytes(more) <= kHeldBytes;
    if (held) ranks = more;
    // No block without logits: a share is whole steps of its warps, so fewer often hold all (16 rows of 32768 by top-p
    // 19.5 us with eight blocks a row, 16.1 with the five that have some).
    ranks = (unsigned)ceil_div(V + 7, chunk(ranks) * kSampleWarps);
    SampleParams p{};
    p.logits = logits; p.stride = row_stride; p.u = u; p.how = *how; p.tokens = tokens; p.logprobs = logprobs;
    p.V = (int)V; p.chunk = (int)chunk(ranks);
    const void* kernel = type == NVFP4_LOGITS_BF16 ? sample_kernel_of<kTypeBf16>(held)
                       : type == NVFP4_LOGITS_F16 ? sample_kernel_of<kTypeF16>(held) : sample_kernel_of<kTypeF32>(held);
    const size_t smem = held ? (size_t)bytes(ranks) : (size_t)kSampleWarps * kStages * 256 * size;
    void* args[] = {&p};
    return launch_kernel(kernel, dim3((unsigned)(B * ranks)), dim3(kSampleThreads), smem, ranks, args, (cudaStream_t)stream, fn);
}
