// The next token of each row of logits, from a given random number:
//     w_i = exp((l_i - max l) / T),
// over the top_k largest logits (equal ones rank by index), of those over the shortest
// prefix in that order that holds top_p of their mass, of those over w_i >= min_p; the
// token is the first of them, by index, whose running mass passes u times their mass.
//
// A draw is a comparison of sums of up to a few hundred thousand weights with a random
// threshold: with 32-bit sums one draw in a hundred would fall on the wrong side of a
// border, another one for another order of the sums.  So weights are whole numbers of
// 2^-43 (of the largest weight), right to about 2^-32 of their value, and sums of them
// are exact in 64 bits, in any order and by any block.  No sorting: a histogram over
// the distance to the largest logit finds the bin in which top_k or top_p ends, and
// only that bin's values are sorted.
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
constexpr int kList = 1024;                // values sorted at most
constexpr int kMaxCluster = 8;
constexpr int kOneLog2 = 43;               // a weight of one is 2^43: 2^20 of them sum inside 63 bits
constexpr int64_t kMaxVocabulary = 1 << 20;
constexpr size_t kHeldBytes = 84 * 1024;   // of a block's logits in shared memory: two blocks an SM

// 2^30 * 2^(j / 512), from the series of exp.
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
    int V, chunk;                          // chunk: virtual elements of a warp, a multiple of 8
};

// A number whose last bit is worth one: added to a float below 2^22, it leaves the nearest
// whole number in the low bits, at a quarter of a conversion's time.
constexpr float kWhole = 12582912.f;
constexpr int kWholeBits = 0x4B400000;

// Entry of the table: 2^30 * 2^(j / 512) less kWholeBits, and as a float.
__device__ __forceinline__ uint2 table_entry(uint32_t v) { return make_uint2(v - (uint32_t)kWholeBits, __float_as_uint((float)v)); }

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
    // Bin of the first histogram, 20 for each factor of two; never falls as l falls.
    __device__ __forceinline__ int bin(float l) const {
        return __float_as_int(fmaf(l, -20.f * ch, (kWhole + 1.f) + rintf(20.f * mh))) - kWholeBits;
    }
    __device__ __forceinline__ float log_weight(float l) const { return fmaf(l, cl, fmaf(l, ch, -mh)) * 0.693147180559945f; }
    // 2^(l ch + l cl - mh): the nearest 512th by table, in 2^-30; the rest, below 2^-10 (and 2^-12
    // for l cl), by three terms of exp's series, good to 2^-33 of the whole.  The rest itself is
    // exact but for its last bit: mh plus a 512th has no rounding.
    __device__ __forceinline__ void weights(float la, float lb, const uint2* table, uint64_t& wa, uint64_t& wb) const {
        const F2 l = make_f2(la, lb);
        const F2 whole = fma2(l, make_f2(ch * 512.f, ch * 512.f), make_f2(kWhole - mh * 512.f, kWhole - mh * 512.f));
        const F2 k = fma2(whole, make_f2(1.f, 1.f), make_f2(-kWhole, -kWhole));
        const F2 minus_s = fma2(k, make_f2(-1.f / 512.f, -1.f / 512.f), make_f2(-mh, -mh));
        const F2 rest = fma2(l, make_f2(cl, cl), fma2(l, make_f2(ch, ch), minus_s));
        constexpr float kLn2 = 0.693147180559945f;
        const F2 p = mul2(rest, fma2(rest, fma2(rest, make_f2(kLn2 * kLn2 * kLn2 / 6, kLn2 * kLn2 * kLn2 / 6), make_f2(kLn2 * kLn2 / 2, kLn2 * kLn2 / 2)),
                                     make_f2(kLn2, kLn2)));
        const float2 n = both(whole);
        const int na = __float_as_int(n.x), nb = __float_as_int(n.y);
        const uint2 ea = table[na & 511], eb = table[nb & 511];
        const float2 v = both(fma2(make_f2(__uint_as_float(ea.y), __uint_as_float(eb.y)), p, make_f2(kWhole, kWhole)));
        wa = shifted(ea.x + __float_as_uint(v.x), (kWholeBits >> 9) - (na >> 9));
        wb = shifted(eb.x + __float_as_uint(v.y), (kWholeBits >> 9) - (nb >> 9));
    }
    // w * 2^(13 - s), to the nearest whole number.
    __device__ __forceinline__ static uint64_t shifted(uint32_t w, int s) {
        const int d = s - (kOneLog2 - 30);                          // below 13 the product is whole
        if (d <= 0) return (uint64_t)w << -d;
        return ((w >> min(d - 1, 31)) + 1) >> 1;
    }
    __device__ __forceinline__ uint64_t weight(float l, const uint2* table) const {
        uint64_t a, b;
        weights(l, l, table, a, b);
        return a;
    }
};

// The same for rows whose products leave that range (temperatures next to zero, logits of 10^30 or
// infinity): 64-bit floating point, an exponential each.
__device__ __noinline__ double far_place(double c, float top, float l) {
    if (l == top) return 0.0;
    return l == -INFINITY ? -INFINITY : ((double)l - (double)top) * c;             // zero times infinity: not counted
}
__device__ __noinline__ uint64_t far_weight(double x) {
    return x > -47.0 ? (uint64_t)__double2ll_rn(exp2(x) * (double)(1ull << kOneLog2)) : 0;
}
struct FarScale {
    double c;
    float top;

    __device__ __forceinline__ void set(float top_, float t) {
        top = top_;
        c = 1.4426950408889634074 / (double)t;
    }
    __device__ __forceinline__ float tidy(float l) const { return fmaxf(l, -INFINITY); }
    __device__ __forceinline__ bool counts(float l) const { return place(l) > -47.0; }
    __device__ __forceinline__ double place(float l) const { return far_place(c, top, l); }
    __device__ __forceinline__ int bin(float l) const { return (int)(fmax(place(l), -47.0) * -20.0); }
    __device__ __forceinline__ float log_weight(float l) const { return (float)(place(l) * 0.69314718055994530942); }
    __device__ __forceinline__ uint64_t weight(float l, const uint2*) const {
        return far_weight(place(l));
    }
    __device__ __forceinline__ void weights(float la, float lb, const uint2* table, uint64_t& wa, uint64_t& wb) const {
        wa = weight(la, table);
        wb = weight(lb, table);
    }
};
constexpr int kDeadBin = 20 * (kOneLog2 + 1) + 2;          // what lies in bins from here on weighs nothing

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

enum { kTypeBf16, kTypeF16, kTypeF32 };

// The row's virtual elements, in 16-byte pieces: element 0 is on a boundary of eight elements.
// HELD: a block's part stays in shared memory, each lane's pieces where that lane finds them.
template <int TYPE, bool HELD>
struct Row {
    static constexpr int kSize = TYPE == kTypeF32 ? 4 : 2;
    static constexpr int kPieces = kSize / 2;              // of eight elements
    const uint8_t* base;
    uint8_t* held;
    int first, end;                        // virtual elements that are the row's

    __device__ __forceinline__ Row(const void* logits, int64_t offset, int V, uint8_t* held_) : held(held_) {
        const uint8_t* p = (const uint8_t*)logits + offset * kSize;
        first = (int)(((uintptr_t)p & (8 * kSize - 1)) / kSize);
        base = p - first * kSize;
        end = first + V;
    }
    // Elements j to j + 7 (j a multiple of 8) from memory, -infinity outside the row.
    __device__ __forceinline__ void load(int j, uint4 (&v)[kPieces]) const {
        if (j >= first && j + 8 <= end) {
#pragma unroll
            for (int k = 0; k < kPieces; ++k) v[k] = ((const uint4*)(base + (int64_t)j * kSize))[k];
            return;
        }
        if (TYPE == kTypeF32) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = j + i >= first && j + i < end ? ((const uint32_t*)base)[j + i] : 0xff800000u;
            v[0] = make_uint4(w[0], w[1], w[2], w[3]);
            v[kPieces - 1] = make_uint4(w[4], w[5], w[6], w[7]);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t h[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int at = j + 2 * i + k;
                    h[k] = at >= first && at < end ? ((const uint16_t*)base)[at] : TYPE == kTypeF16 ? 0xfc00u : 0xff80u;
                }
                w[i] = h[0] | h[1] << 16;
            }
            v[0] = make_uint4(w[0], w[1], w[2], w[3]);
        }
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
    __device__ __forceinline__ uint4* place(int step) const {
        return (uint4*)held + (step * kSampleWarps + (threadIdx.x >> 5)) * kPieces * 32 + (threadIdx.x & 31);
    }
    // Elements j to j + 7, this lane's of step `step`.
    __device__ __forceinline__ void eight(int j, int step, float (&l)[8]) const {
        uint4 v[kPieces];
        if (HELD) {
#pragma unroll
            for (int k = 0; k < kPieces; ++k) v[k] = place(step)[k * 32];
        } else {
            load(j, v);
        }
        widen(v, l);
    }
};

// Where the kept tokens of a row end: every logit above `value`, and of those equal to it the
// first `ties`, by index.  `above` is the mass of the former, `each` the weight of the latter.
struct Cut {
    float value;
    uint32_t ties;
    uint64_t above, each;
};

struct Shared {
    uint2 table[512];
    uint32_t count[kBins], lo[kBins], hi[kBins];           // a mass is lo + 2^32 hi
    uint32_t list[2][kList];               // values of a bin, as keys: of this block; of the whole row
    uint32_t listed[2];                    // of the two lists that a row may need
    int64_t scan[2][kSampleWarps];
    uint64_t found[4];
    float best[kMaxCluster];               // pushed here by every block of the row
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

// Sums over the threads below this one, of a count and a mass; returns the whole mass.
__device__ __forceinline__ uint64_t block_below(uint64_t& count, uint64_t& mass, Shared& sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t c = warp_below((uint32_t)count, lane);
    const uint64_t m = warp_below(mass, lane);
    if (lane == 31) {
        sm.scan[0][warp] = c + count;
        sm.scan[1][warp] = m + mass;
    }
    __syncthreads();
    uint64_t cs = 0, ms = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kSampleWarps; ++w) {
        if (w == warp) ms = all;
        if (w < warp) cs += sm.scan[0][w];
        all += sm.scan[1][w];
    }
    __syncthreads();
    count = c + cs;
    mass = m + ms;
    return all;
}

__device__ __forceinline__ void add_mass(Shared& sm, int bin, uint64_t w) {
    const uint32_t low = (uint32_t)w, old = atomicAdd(&sm.lo[bin], low);
    const uint32_t up = (uint32_t)(w >> 32) + (old + low < old);
    if (up) atomicAdd(&sm.hi[bin], up);
}

constexpr int kOwnBins = kBins / kSampleThreads;           // bins of a thread when they are summed

template <int TYPE, bool HELD, class SCALE>
struct Sampler {
    Shared& sm;
    const Row<TYPE, HELD>& row;
    const uint32_t rank, ranks;
    const int j0, j1;                      // virtual elements of this warp
    const SCALE& scale;

    // f(first virtual index, eight logits) over this warp's elements, in index order over lanes.
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        int step = 0;
        for (int j = j0 + (threadIdx.x & 31) * 8; j < j1; j += 256, ++step) {
            float l[8];
            row.eight(j, step, l);
#pragma unroll
            for (int i = 0; i < 8; ++i) l[i] = scale.tidy(l[i]);
            f(j, l);
        }
    }

    // Counts and masses of the whole row's bins after every block has made its own.
    __device__ __forceinline__ void gather(bool by_count, bool by_mass, uint64_t (&count)[kOwnBins], uint64_t (&mass)[kOwnBins]) {
        static_assert(kOwnBins == 2, "read in pairs");
        cluster_sync();
        uint64_t hi[kOwnBins] = {0, 0};
        count[0] = count[1] = mass[0] = mass[1] = 0;
        if (by_count) read(sm.count, count);
        if (by_mass) {
            read(sm.lo, mass);
            read(sm.hi, hi);
            mass[0] += hi[0] << 32;
            mass[1] += hi[1] << 32;
        }
    }
    // Sums of this thread's two bins over the blocks.
    __device__ __forceinline__ void read(const uint32_t (&bins)[kBins], uint64_t (&sum)[kOwnBins]) const {
        uint2 v[kMaxCluster];
        const uint32_t at = smem_u32(&bins[threadIdx.x * 2]);
#pragma unroll
        for (uint32_t r = 0; r < kMaxCluster; ++r) v[r] = r < ranks ? remote_u32x2(map_rank(at, r)) : make_uint2(0, 0);
#pragma unroll
        for (uint32_t r = 0; r < kMaxCluster; ++r) {
            sum[0] += v[r].x;
            sum[1] += v[r].y;
        }
    }

    // Histogram of the row's logits by their place, of counts and masses as asked.
    __device__ __forceinline__ void histogram(bool by_count, bool by_mass, uint64_t (&count)[kOwnBins], uint64_t (&mass)[kOwnBins]) {
        each([&](int, const float (&l)[8]) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                uint64_t w[2] = {0, 0};
                if (by_mass) scale.weights(l[i], l[i + 1], sm.table, w[0], w[1]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (!scale.counts(l[i + k])) continue;
                    const int b = scale.bin(l[i + k]);
                    if (by_count) atomicAdd(&sm.count[b], 1u);
                    if (by_mass) add_mass(sm, b, w[k]);
                }
            }
        });
        gather(by_count, by_mass, count, mass);
    }

    // The same of one bin's logits whose keys begin with the `bits` bits `known`, by their next
    // `take` bits, the largest first.
    __device__ __noinline__ void digits(int bin, uint32_t known, uint32_t bits, uint32_t take, bool by_mass, uint64_t (&count)[kOwnBins],
                                           uint64_t (&mass)[kOwnBins]) {
        cluster_sync();                                     // all have read the last histogram
        for (int i = threadIdx.x; i < kBins; i += kSampleThreads) sm.count[i] = sm.lo[i] = sm.hi[i] = 0;
        __syncthreads();
        each([&](int, const float (&l)[8]) {
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                const uint32_t k = order_key(l[i]);
                if (!scale.counts(l[i]) || scale.bin(l[i]) != bin || (bits && k >> (32 - bits) != known)) continue;
                const int d = (int)((1u << take) - 1 - ((k >> (32 - bits - take)) & ((1u << take) - 1)));
                atomicAdd(&sm.count[d], 1u);
                if (by_mass) add_mass(sm, d, scale.weight(l[i], sm.table));
            }
        });
        gather(true, by_mass, count, mass);
    }

    // The bin in which `count` or `mass` reaches the target; false where the sum never does.
    // Leaves the bin, its count, and the count and mass before it in `out`.
    __device__ __forceinline__ bool bin_of(const uint64_t (&count)[kOwnBins], const uint64_t (&mass)[kOwnBins], bool by_mass, uint64_t target,
                                           uint64_t (&out)[4]) {
        uint64_t c = 0, m = 0;
#pragma unroll
        for (int k = 0; k < kOwnBins; ++k) {
            c += count[k];
            m += mass[k];
        }
        if (threadIdx.x == 0) sm.found[0] = ~0ull;
        block_below(c, m, sm);
#pragma unroll
        for (int k = 0; k < kOwnBins; ++k) {
            const uint64_t before = by_mass ? m : c, here = by_mass ? mass[k] : count[k];
            if (before < target && target <= before + here) {
                sm.found[0] = threadIdx.x * kOwnBins + k;
                sm.found[1] = count[k];
                sm.found[2] = c;
                sm.found[3] = m;
            }
            c += count[k];
            m += mass[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 4; ++k) out[k] = sm.found[k];
        __syncthreads();
        return out[0] != ~0ull;
    }

    // The cut at which the count or the mass of the logits, from the largest down, reaches the
    // target, which lies in `bin` of the first histogram.  `which` list: the row's first or second.
    __device__ __noinline__ Cut cut_in(uint64_t (&bin)[4], bool by_mass, bool with_mass, uint64_t target, int which) {
        uint32_t known = 0, bits = 0;                       // leading bits of the keys in question
        const int b0 = (int)bin[0];
        while (bin[1] > kList && bits < 32) {
            // More values than can be sorted: their keys' next bits, 10, 10, 10 and 2 of them.
            const uint32_t take = min(32 - bits, 10u);
            uint64_t count[kOwnBins], mass[kOwnBins];
            const uint64_t count0 = bin[2], mass0 = bin[3];
            digits(b0, known, bits, take, with_mass, count, mass);
            bin_of(count, mass, by_mass, target - (by_mass ? mass0 : count0), bin);
            known = (known << take) | ((1u << take) - 1 - (uint32_t)bin[0]);
            bits += take;
            bin[2] += count0;
            bin[3] += mass0;
        }
        Cut cut;
        if (bits == 32) {                                   // all values left are equal
            cut.value = key_value(known);
            cut.above = bin[3];
            cut.each = scale.weight(cut.value, sm.table);
            cut.ties = (uint32_t)(by_mass ? (target - bin[3] + cut.each - 1) / cut.each : target - bin[2]);
            return cut;
        }
        // The bin's keys, from every block.
        if (which) {
            __syncthreads();
            cluster_sync();                                 // all have read the first list
        }
        each([&](int, const float (&l)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (!scale.counts(l[i]) || scale.bin(l[i]) != b0) continue;
                const uint32_t k = order_key(l[i]);
                if (bits && k >> (32 - bits) != known) continue;
                sm.list[0][atomicAdd(&sm.listed[which], 1u)] = k;
            }
        });
        cluster_sync();
        const uint64_t want = target - (by_mass ? bin[3] : bin[2]);
        int n = 0;
        const auto weight_of = [&](uint32_t k) { return scale.weight(key_value(k), sm.table); };
        if (bin[1] <= 32) {
            // A value a lane, in every warp alike: what goes before each, and the one that reaches the target.
            const int lane = threadIdx.x & 31;
            uint32_t key = 0;
            for (uint32_t r = 0; r < ranks; ++r) {
                const int m = (int)remote_u32(&sm.listed[which], r);
                if (lane >= n && lane < n + m) key = remote_u32(&sm.list[0][lane - n], r);
                n += m;
            }
            const uint64_t w = lane < n && with_mass ? weight_of(key) : 0;
            uint32_t c = 0, greater = 0;                    // before it: larger ones, and equal ones of lower lanes
            uint64_t m = 0, above = 0;
            for (int o = 0; o < n; ++o) {
                const uint32_t k = __shfl_sync(0xffffffffu, key, o);
                const uint64_t v = __shfl_sync(0xffffffffu, w, o);
                const bool over = k > key, ahead = over || (k == key && o < lane);
                c += ahead;
                greater += over;
                m += ahead ? v : 0;
                above += over ? v : 0;
            }
            const uint64_t before = by_mass ? m : c, here = by_mass ? w : 1;
            const uint32_t reaches = __ballot_sync(0xffffffffu, lane < n && before < want && want <= before + here);
            const int at = __ffs(reaches) - 1;
            cut.value = key_value(__shfl_sync(0xffffffffu, key, at));
            cut.above = bin[3] + __shfl_sync(0xffffffffu, above, at);
            cut.each = __shfl_sync(0xffffffffu, w, at);
            cut.ties = (uint32_t)(by_mass ? (target - cut.above + cut.each - 1) / cut.each : want - __shfl_sync(0xffffffffu, greater, at));
            return cut;
        }
        for (uint32_t r = 0; r < ranks; ++r) {
            const int m = (int)remote_u32(&sm.listed[which], r);
            for (int i = threadIdx.x; i < m; i += kSampleThreads) sm.list[1][n + i] = remote_u32(&sm.list[0][i], r);
            n += m;
        }
        int size = 64;
        while (size < n) size *= 2;
        for (int i = n + threadIdx.x; i < size; i += kSampleThreads) sm.list[1][i] = 0;      // below every key
        __syncthreads();
        for (int k = 2; k <= size; k *= 2)                  // from the largest down, in place
            for (int s = k / 2; s > 0; s /= 2) {
                const int i = threadIdx.x;
                if (i < size / 2) {
                    const int a = 2 * i - (i & (s - 1)), b = a + s;
                    const uint32_t x = sm.list[1][a], y = sm.list[1][b];
                    if ((x < y) == ((a & k) == 0)) {
                        sm.list[1][a] = y;
                        sm.list[1][b] = x;
                    }
                }
                __syncthreads();
            }
        // The value where the target is reached, then what lies above it.
        const int i = threadIdx.x * 2;
        uint64_t w[2] = {0, 0};
        for (int k = 0; k < 2; ++k)
            if (i + k < n && with_mass) w[k] = weight_of(sm.list[1][i + k]);
        uint64_t c = (i < n) + (i + 1 < n), m = w[0] + w[1];
        block_below(c, m, sm);
        for (int k = 0; k < 2; ++k)
            if (i + k < n) {
                const uint64_t before = by_mass ? m + (k ? w[0] : 0) : c + k, here = by_mass ? w[k] : 1;
                if (before < want && want <= before + here) sm.found[0] = sm.list[1][i + k];
            }
        __syncthreads();
        const uint32_t key = (uint32_t)sm.found[0];
        for (int k = 0; k < 2; ++k) {                       // its first place in the list
            const int at = i + k;
            if (at < n && sm.list[1][at] == key && (at == 0 || sm.list[1][at - 1] != key)) {
                sm.found[1] = c + k;
                sm.found[2] = m + (k ? w[0] : 0);
            }
        }
        __syncthreads();
        cut.value = key_value(key);
        cut.above = bin[3] + sm.found[2];
        cut.each = weight_of(key);
        cut.ties = (uint32_t)(by_mass ? (target - cut.above + cut.each - 1) / cut.each : want - sm.found[1]);
        __syncthreads();
        return cut;
    }

    // From the largest logit to the token.
    __device__ __forceinline__ void draw(const SampleParams& p, int64_t b, float best, int top_k, float top_p, float min_p) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        Cut cut{-INFINITY, 0, 0, 0};                        // everything
        const bool by_k = top_k > 0 && top_k < p.V, by_p = top_p < 1.f;
        if (by_k || by_p) {
            uint64_t count[kOwnBins], mass[kOwnBins], bin[4], total = ~0ull;
            histogram(true, by_p, count, mass);
            if (by_k && bin_of(count, mass, false, (uint64_t)top_k, bin) && bin[0] < kDeadBin) {
                cut = cut_in(bin, false, by_p, (uint64_t)top_k, 0);
                total = cut.above + cut.ties * cut.each;
            }
            if (by_p) {
                if (total == ~0ull) {
                    uint64_t c = 0, m = 0;
#pragma unroll
                    for (int k = 0; k < kOwnBins; ++k) m += mass[k];
                    total = block_below(c, m, sm);
                }
                const uint64_t target = max(part_of(top_p, total, true), (uint64_t)1);
                if (bin_of(count, mass, true, target, bin)) cut = cut_in(bin, true, true, target, 1);
            }
        }

        // Mass of what is kept, over warps, blocks and the row; equal values at the cut count by index.
        const uint64_t least = min_p > 0.f ? min_p < 1.f ? part_of(min_p, scale.weight(best, sm.table), true) : ~0ull : 0;
        const auto kept = [&](float l, uint64_t w) -> uint64_t { return w >= least || l == best ? w : 0; };
        const auto kept_weight = [&](float l) -> uint64_t { return kept(l, scale.weight(l, sm.table)); };
        cut.each = cut.value == -INFINITY ? 0 : kept_weight(cut.value);
        uint64_t mass = 0;
        uint32_t ties = 0;
        each([&](int, const float (&l)[8]) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                if (l[i] > cut.value || l[i + 1] > cut.value) {
                    uint64_t w[2];
                    scale.weights(l[i], l[i + 1], sm.table, w[0], w[1]);
                    mass += (l[i] > cut.value ? kept(l[i], w[0]) : 0) + (l[i + 1] > cut.value ? kept(l[i + 1], w[1]) : 0);
                }
                ties += (l[i] == cut.value) + (l[i + 1] == cut.value);
            }
        });
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
        const auto with_ties = [&](uint64_t m, uint32_t t, uint32_t n) { return m + (min(t + n, cut.ties) - min(t, cut.ties)) * cut.each; };
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
        int step = 0;
        for (int j = j0 + lane * 8; j - lane * 8 < j1; j += 256, ++step) {
            float l[8];
            uint64_t w[8], m = 0;
            uint32_t n = 0;
            if (j < j1) {
                row.eight(j, step, l);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    l[i] = scale.tidy(l[i]);
                    w[i] = l[i] > cut.value ? kept_weight(l[i]) : 0;
                    m += w[i];
                    n += l[i] == cut.value;
                }
            }
            uint32_t at = seen + warp_below(n, lane);
            const uint64_t mine = with_ties(m, at, n);
            uint64_t sum = before + warp_below(mine, lane);
            if (target >= sum && target < sum + mine) {
                for (int i = 0; i < 8; ++i) {
                    const uint64_t here = l[i] == cut.value ? (at++ < cut.ties ? cut.each : 0) : w[i];
                    if (target >= sum && target < sum + here) {
                        p.tokens[b] = j + i - row.first;
                        if (p.logprobs) p.logprobs[b] = log_share(l[i], here, whole);
                    }
                    sum += here;
                }
            }
            before += warp_sum(mine);
            seen += warp_sum(n);
        }
    }

    // log(w / whole): near one by what is missing, from 2^24 units on by the quotient, else by the place.
    __device__ __forceinline__ float log_share(float l, uint64_t w, uint64_t whole) const {
        if (w > whole / 2) return log1pf(-((float)(whole - w) / (float)whole));
        if (w >= 1u << 24) return logf((float)w / (float)whole);
        return scale.log_weight(l) - logf((float)whole * (1.f / (float)(1ull << kOneLog2)));
    }
};

template <int TYPE, bool HELD>
__global__ void __launch_bounds__(kSampleThreads, 2) sample_kernel(const SampleParams p) {
    extern __shared__ __align__(16) uint8_t sm_held[];
    __shared__ Shared sm;
    cluster_arrive();                                       // that every block of the row runs: before the first push
    const uint32_t rank = cluster_rank(), ranks = cluster_ranks();
    const int64_t b = blockIdx.x / ranks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    sm.table[threadIdx.x] = table_entry(kExp2.v[threadIdx.x]);
    for (int i = threadIdx.x; i < kBins; i += kSampleThreads) sm.count[i] = sm.lo[i] = sm.hi[i] = 0;
    if (threadIdx.x < 2) sm.listed[threadIdx.x] = 0;
    pdl_wait_previous();
    pdl_launch_dependents();
    const float temperature = p.how.temperature ? p.how.temperature[b] : p.how.temperature_all;
    const bool greedy = !(temperature > 0.f);
    const int top_k = p.how.top_k ? p.how.top_k[b] : p.how.top_k_all;
    const float top_p = p.how.top_p ? p.how.top_p[b] : p.how.top_p_all, min_p = p.how.min_p ? p.how.min_p[b] : p.how.min_p_all;
    const Row<TYPE, HELD> row(p.logits, b * p.stride, p.V, sm_held);
    const int64_t start = ((int64_t)rank * kSampleWarps + warp) * p.chunk;
    const int j0 = (int)min(start, (int64_t)row.end), j1 = (int)min(start + p.chunk, (int64_t)row.end);

    // The largest logit, the first of equal ones; four loads in flight.
    constexpr int U = 4 / Row<TYPE, HELD>::kPieces;
    float best = -INFINITY;
    int best_at = INT32_MAX, step = 0;
    for (int j = j0 + lane * 8; j < j1; j += 256 * U, step += U) {
        uint4 v[U][Row<TYPE, HELD>::kPieces];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (j + u * 256 < j1) row.load(j + u * 256, v[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (j + u * 256 >= j1) break;
            if (HELD)
#pragma unroll
                for (int k = 0; k < Row<TYPE, HELD>::kPieces; ++k) row.place(step + u)[k * 32] = v[u][k];
            float l[8];
            row.widen(v[u], l);
            float m = fmaxf(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])), fmaxf(fmaxf(l[4], l[5]), fmaxf(l[6], l[7])));
            if (m > best) {                                 // NaN is neither
                best = m;
                if (greedy) {
#pragma unroll
                    for (int i = 7; i >= 0; --i)
                        if (l[i] == m) best_at = j + u * 256 + i;
                }
            }
        }
    }
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
        Sampler<TYPE, HELD, NearScale>{sm, row, rank, ranks, j0, j1, near}.draw(p, b, best, top_k, top_p, min_p);
    } else {
        FarScale far;
        far.set(best, temperature);
        Sampler<TYPE, HELD, FarScale>{sm, row, rank, ranks, j0, j1, far}.draw(p, b, best, top_k, top_p, min_p);
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
    // Blocks of a row: enough of them to fill the SMs with two each, none with less than 4096 logits;
    // more where a block's part then stays in shared memory beside another block's.
    const auto part = [&](unsigned ranks) { return round_up(ceil_div(ceil_div(V + 7, ranks), kSampleWarps), 8); };      // of a warp
    const auto bytes = [&](unsigned ranks) { return (size_t)ceil_div(part(ranks), 256) * 256 * kSampleWarps * size; };
    unsigned ranks = 1;
    while (ranks < kMaxCluster && ((B * ranks < sm_count() && V / (2 * ranks) >= 4096) || bytes(ranks) > kHeldBytes)) ranks *= 2;
    const bool held = bytes(ranks) <= kHeldBytes;
    SampleParams p{};
    p.logits = logits; p.stride = row_stride; p.u = u; p.how = *how; p.tokens = tokens; p.logprobs = logprobs;
    p.V = (int)V; p.chunk = (int)part(ranks);
    const void* kernel = type == NVFP4_LOGITS_BF16 ? sample_kernel_of<kTypeBf16>(held)
                       : type == NVFP4_LOGITS_F16 ? sample_kernel_of<kTypeF16>(held) : sample_kernel_of<kTypeF32>(held);
    void* args[] = {&p};
    return launch_kernel(kernel, dim3((unsigned)(B * ranks)), dim3(kSampleThreads), held ? bytes(ranks) : 0, ranks, args, (cudaStream_t)stream, fn);
}
