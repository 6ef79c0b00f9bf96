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
constexpr int kBins = 2048;                // of the histogram; 64 for each factor of two in weight
constexpr int kList = 1024;                // values sorted at most
constexpr int kMaxCluster = 8;
constexpr int kOneLog2 = 43;               // a weight of one is 2^43: 2^20 of them sum inside 63 bits
constexpr int64_t kMaxVocabulary = 1 << 20;

// 2^31 * 2^(j / 512), from the series of exp.
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
            v[j] = (uint32_t)(sum * 2147483648.0 + 0.5);
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
    int V, slice;                          // slice: virtual elements of a block, a multiple of 8 * warps
};

// A logit's place below the row's largest, in factors of two, and its weight.
struct Scale {
    double c, m;                           // log2(e) / T, and that times the largest logit
    float ch, cl, mh, ml;                  // c = ch + cl, m = mh + ml with mh a multiple of 2^-9
    float shift;                           // ml in 512ths, the other way
    float top;                             // the largest logit
    bool wide;                             // m too large for mh, or infinite: in 64-bit floating point

    __device__ __forceinline__ void set(float top_, float t) {
        top = top_;
        c = 1.4426950408889634074 / (double)t;
        m = (double)top * c;
        wide = !(fabs(m) < 4096.0 && c < 0x1p100);
        ch = (float)c;
        cl = (float)(c - (double)ch);
        mh = wide ? 0.f : rintf((float)(m * 512.0)) * (1.f / 512.f);
        ml = wide ? 0.f : (float)(m - (double)mh);
        shift = -512.f * ml;
    }
    // Falls with l, never rises (each rounding keeps order); l is not -infinity.
    __device__ __forceinline__ float place(float l) const {
        if (wide) return l == top ? 0.f : (float)(((double)l - (double)top) * c);
        return fmaf(l, ch, -mh);
    }
    // The same but for its last bits: what place() leaves out.
    __device__ __forceinline__ float exact_place(float l) const { return wide ? place(l) : place(l) + fmaf(l, cl, -ml); }
    // Whole number of 2^-43.  2^place: the nearest 512th by table, in 2^-31; the rest, below
    // 2^-10 (and 2^-12 for l * cl), by three terms of exp's series, good to 2^-33 of the
    // whole.  The rest itself is exact but for its own last bit: mh plus a 512th has no rounding.
    __device__ __forceinline__ uint64_t weight(float l, float t, const uint2* table) const {
        if (wide) {
            if (l == top) return 1ull << kOneLog2;
            const double x = ((double)l - (double)top) * c;
            return x > -46.0 ? (uint64_t)__double2ll_rn(exp2(x) * (double)(1ull << kOneLog2)) : 0;
        }
        if (!(t > -46.f)) return 0;
        const float k = rintf(fmaf(t, 512.f, shift));
        const float rest = fmaf(l, ch, -fmaf(k, 1.f / 512.f, mh)) + fmaf(l, cl, -ml);
        const float y = rest * 0.693147180559945f;
        const float p = fmaf(y * y, fmaf(y, 1.f / 6.f, 0.5f), y);
        const int n = (int)k;
        const uint2 e = table[n & 511];
        const uint32_t w = e.x + (uint32_t)__float2int_rn(__uint_as_float(e.y) * p);
        return ((uint64_t)w << (kOneLog2 - 31)) >> (-(n >> 9));
    }
    __device__ __forceinline__ int bin(float t) const { return t > -(float)(kBins - 1) / 64.f ? (int)fmaxf(t * -64.f, 0.f) : kBins - 1; }
};

// Floats as whole numbers in the same order.
__device__ __forceinline__ uint32_t order_key(float l) {
    const uint32_t b = __float_as_uint(l);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

// Whole part of f * s for 0 <= f < 1, rounded up where asked: f is a 24-bit whole number
// and a power of two.
__device__ __forceinline__ uint64_t part_of(float f, uint64_t s, bool up) {
    if (!(f > 0.f)) return 0;
    int e = (int)(__float_as_uint(f) >> 23);
    const uint64_t digits = e ? (__float_as_uint(f) & 0x7fffffu) | 0x800000u : __float_as_uint(f) & 0x7fffffu;
    const int shift = 150 - (e ? e : 1);                    // f = digits * 2^-shift, shift >= 24
    const uint64_t lo = digits * s, hi = __umul64hi(digits, s);
    if (shift >= 128) return up ? 1 : 0;                    // hi < 2^24, s < 2^63: the product is below 2^87
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

template <int TYPE>
struct Row {
    const uint8_t* base;                   // of virtual element 0, on a 32- or 16-byte boundary
    int first, end;                        // virtual elements that are the row's

    static constexpr int kSize = TYPE == kTypeF32 ? 4 : 2;

    __device__ __forceinline__ Row(const void* logits, int64_t offset, int V) {
        const uint8_t* p = (const uint8_t*)logits + offset * kSize;
        first = (int)(((uintptr_t)p & (8 * kSize - 1)) / kSize);
        base = p - first * kSize;
        end = first + V;
    }
    // NaN as -infinity, and one zero.
    __device__ __forceinline__ static float tidy(float l) { return l == l ? l + 0.f : -INFINITY; }
    __device__ __forceinline__ float one(int j) const {
        if (TYPE == kTypeF32) return tidy(((const float*)base)[j]);
        return tidy(act_to_f32<TYPE == kTypeF16>(((const uint16_t*)base)[j]));
    }
    // Elements j to j + 7 (j a multiple of 8), -infinity outside the row.
    __device__ __forceinline__ void eight(int j, float (&l)[8]) const {
        if (j >= first && j + 8 <= end) {
            if (TYPE == kTypeF32) {
                const float4 a = ((const float4*)base)[j / 4], b = ((const float4*)base)[j / 4 + 1];
                l[0] = a.x; l[1] = a.y; l[2] = a.z; l[3] = a.w;
                l[4] = b.x; l[5] = b.y; l[6] = b.z; l[7] = b.w;
            } else {
                const uint4 w = ((const uint4*)base)[j / 8];
                const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 v = act2_to_f32<TYPE == kTypeF16>(in[i]);
                    l[2 * i] = v.x;
                    l[2 * i + 1] = v.y;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) l[i] = tidy(l[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) l[i] = j + i >= first && j + i < end ? one(j + i) : -INFINITY;
        }
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
    uint2 table[512];                      // 2^31 * 2^(j/512), and the same as a float
    uint32_t count[kBins], lo[kBins], hi[kBins];
    uint32_t list[2][kList];               // values of a bin, as keys: of this block; of the whole row
    uint32_t listed;
    int64_t scan[2][kSampleWarps + 1];
    uint64_t found[4];
    Cut cut;
    float best[kMaxCluster];               // pushed here by every block of the row
    int best_at[kMaxCluster];
    uint64_t mass[kMaxCluster];
    uint32_t ties[kMaxCluster];
    uint64_t warp_mass[kSampleWarps];
    uint32_t warp_ties[kSampleWarps];
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t remote_u32(const void* p, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_rank(smem_u32(p), rank)) : "memory");
    return v;
}
__device__ __forceinline__ void push_u32(void* p, uint32_t rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_rank(smem_u32(p), rank)), "r"(v) : "memory");
}
__device__ __forceinline__ void push_u64(void* p, uint32_t rank, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(map_rank(smem_u32(p), rank)), "l"(v) : "memory");
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

// Sums over the threads below this one, of a count and a mass.
__device__ __forceinline__ void block_below(uint64_t& count, uint64_t& mass, Shared& sm) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint64_t c = warp_below(count, lane), m = warp_below(mass, lane);
    if (lane == 31) {
        sm.scan[0][warp] = c + count;
        sm.scan[1][warp] = m + mass;
    }
    __syncthreads();
    uint64_t cs = 0, ms = 0;
    for (int w = 0; w < warp; ++w) {
        cs += sm.scan[0][w];
        ms += sm.scan[1][w];
    }
    __syncthreads();
    count = c + cs;
    mass = m + ms;
}

template <int TYPE>
struct Sampler {
    Shared& sm;
    const Row<TYPE> row;
    const uint32_t rank, ranks;
    const int j0, j1;                      // virtual elements of this warp
    Scale scale;

    // f(first virtual index, eight logits) over this warp's elements, in index order over lanes.
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        const int lane = threadIdx.x & 31;
        for (int j = j0 + lane * 8; j < j1; j += 256) {
            float l[8];
            row.eight(j, l);
            f(j, l);
        }
    }

    __device__ __forceinline__ void cluster_sync() const {
        __syncwarp();
        cluster_arrive();
        cluster_wait();
    }

    // Histogram of the logits for which `digit` is not negative, of masses too where asked, over
    // the whole row: afterwards each thread holds four bins' counts and masses.
    template <class D>
    __device__ __forceinline__ void histogram(bool with_mass, D digit, uint64_t (&count)[4], uint64_t (&mass)[4]) {
        for (int i = threadIdx.x; i < kBins; i += kSampleThreads) sm.count[i] = sm.lo[i] = sm.hi[i] = 0;
        __syncthreads();
        uint32_t rest = 0;                                  // the last bin, in registers: most of a row may lie there
        uint64_t rest_mass = 0;
        each([&](int, const float (&l)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (l[i] == -INFINITY) continue;
                const float t = scale.place(l[i]);
                const int d = digit(l[i], t);
                if (d < 0) continue;
                const uint64_t w = with_mass ? scale.weight(l[i], t, sm.table) : 0;
                if (d == kBins - 1) {
                    ++rest;
                    rest_mass += w;
                    continue;
                }
                atomicAdd(&sm.count[d], 1u);
                if (with_mass) {
                    const uint32_t old = atomicAdd(&sm.lo[d], (uint32_t)w);
                    const uint32_t up = (uint32_t)(w >> 32) + (old + (uint32_t)w < old);
                    if (up) atomicAdd(&sm.hi[d], up);
                }
            }
        });
        rest = warp_sum(rest);
        rest_mass = warp_sum(rest_mass);
        if ((threadIdx.x & 31) == 0 && rest) {
            atomicAdd(&sm.count[kBins - 1], rest);
            const uint32_t old = atomicAdd(&sm.lo[kBins - 1], (uint32_t)rest_mass);
            const uint32_t up = (uint32_t)(rest_mass >> 32) + (old + (uint32_t)rest_mass < old);
            if (up) atomicAdd(&sm.hi[kBins - 1], up);
        }
        cluster_sync();
#pragma unroll
        for (int k = 0; k < 4; ++k) count[k] = mass[k] = 0;
        for (uint32_t r = 0; r < ranks; ++r)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int b = threadIdx.x * 4 + k;
                count[k] += remote_u32(&sm.count[b], r);
                if (with_mass) mass[k] += remote_u32(&sm.lo[b], r) + ((uint64_t)remote_u32(&sm.hi[b], r) << 32);
            }
    }

    // The bin in which `count` or `mass` reaches the target; false where the sum never does.
    // Leaves the bin, its count, and the count and mass before it in `out`.
    __device__ __forceinline__ bool bin_of(const uint64_t (&count)[4], const uint64_t (&mass)[4], bool by_mass, uint64_t target, uint64_t (&out)[4]) {
        uint64_t c = count[0] + count[1] + count[2] + count[3], m = mass[0] + mass[1] + mass[2] + mass[3];
        if (threadIdx.x == 0) sm.found[0] = ~0ull;
        block_below(c, m, sm);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint64_t before = by_mass ? m : c, here = by_mass ? mass[k] : count[k];
            if (before < target && target <= before + here) {
                sm.found[0] = threadIdx.x * 4 + k;
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
    // target, which lies in `bin` of the first histogram.
    __device__ Cut cut_in(uint64_t (&bin)[4], bool by_mass, bool with_mass, uint64_t target) {
        uint32_t known = 0, bits = 0;                       // leading bits of the keys in question
        const int b0 = (int)bin[0];
        while (bin[1] > kList && bits < 32) {
            // A bin with more values than can be sorted: its keys' next bits, 11, 11 and 10 of them.
            // Bins run from the largest digit down; the last of the 2048 is a digit as any other.
            const uint32_t take = bits < 22 ? 11 : 10, low = 32 - bits - take;
            uint64_t count[4], mass[4];
            const uint64_t count0 = bin[2], mass0 = bin[3];
            cluster_sync();                                 // all have read the last histogram
            histogram(with_mass, [&](float l, float t) -> int {
                const uint32_t k = order_key(l);
                if (scale.bin(t) != b0 || (bits && k >> (32 - bits) != known)) return -1;
                return (int)((1u << take) - 1 - ((k >> low) & ((1u << take) - 1)));
            }, count, mass);
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
            cut.each = scale.weight(cut.value, scale.place(cut.value), sm.table);
            cut.ties = (uint32_t)(by_mass ? (target - bin[3] + cut.each - 1) / cut.each : target - bin[2]);
            return cut;
        }
        // The bin's keys, from every block, sorted from the largest down.
        if (threadIdx.x == 0) sm.listed = 0;
        __syncthreads();
        each([&](int, const float (&l)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (l[i] == -INFINITY || scale.bin(scale.place(l[i])) != b0) continue;
                const uint32_t k = order_key(l[i]);
                if (bits && k >> (32 - bits) != known) continue;
                sm.list[0][atomicAdd(&sm.listed, 1u)] = k;
            }
        });
        cluster_sync();
        int n = 0;
        for (uint32_t r = 0; r < ranks; ++r) {
            const int m = (int)remote_u32(&sm.listed, r);
            for (int i = threadIdx.x; i < m; i += kSampleThreads) sm.list[1][n + i] = remote_u32(&sm.list[0][i], r);
            n += m;
        }
        int size = 2;
        while (size < n) size *= 2;
        for (int i = n + threadIdx.x; i < size; i += kSampleThreads) sm.list[1][i] = 0;      // below every key
        cluster_sync();                                     // lists may be written again
        for (int k = 2; k <= size; k *= 2)
            for (int s = k / 2; s > 0; s /= 2) {
                const int i = threadIdx.x;
                if (i < size / 2) {
                    const int a = (i / s) * 2 * s + i % s, b = a + s;
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
            if (i + k < n && with_mass) {
                const float l = key_value(sm.list[1][i + k]);
                w[k] = scale.weight(l, scale.place(l), sm.table);
            }
        uint64_t c = (i < n) + (i + 1 < n), m = w[0] + w[1];
        block_below(c, m, sm);
        const uint64_t want = target - (by_mass ? bin[3] : bin[2]);
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
        cut.each = scale.weight(cut.value, scale.place(cut.value), sm.table);
        cut.ties = (uint32_t)(by_mass ? (target - cut.above + cut.each - 1) / cut.each : target - bin[2] - sm.found[1]);
        __syncthreads();
        return cut;
    }
};

template <int TYPE>
__global__ void __launch_bounds__(kSampleThreads, 2) sample_kernel(const SampleParams p) {
    __shared__ Shared sm;
    cluster_arrive();                                       // that every block of the row runs: before the first push
    const uint32_t rank = cluster_rank(), ranks = [] {
        uint32_t n;
        asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
        return n;
    }();
    const int64_t b = blockIdx.x / ranks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t entry = kExp2.v[threadIdx.x];
    sm.table[threadIdx.x] = make_uint2(entry, __float_as_uint((float)entry));
    pdl_wait_previous();
    pdl_launch_dependents();
    const float temperature = p.how.temperature ? p.how.temperature[b] : p.how.temperature_all;
    const bool greedy = !(temperature > 0.f);
    const int top_k = p.how.top_k ? p.how.top_k[b] : p.how.top_k_all;
    const float top_p = p.how.top_p ? p.how.top_p[b] : p.how.top_p_all, min_p = p.how.min_p ? p.how.min_p[b] : p.how.min_p_all;
    const int chunk = p.slice / kSampleWarps, slice0 = (int)rank * p.slice + warp * chunk;
    const Row<TYPE> row(p.logits, b * p.stride, p.V);
    Sampler<TYPE> s{sm, row, rank, ranks, min(slice0, row.end), min(slice0 + chunk, row.end), Scale{}};

    // The largest logit, the first of equal ones.
    float best = -INFINITY;
    int best_at = INT32_MAX;
    s.each([&](int j, const float (&l)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (l[i] > best) {
                best = l[i];
                best_at = j + i;
            }
    });
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
        sm.list[0][warp] = __float_as_uint(best);
        sm.list[1][warp] = (uint32_t)best_at;
    }
    __syncthreads();
    cluster_wait();
    if (threadIdx.x < ranks) {
        best = -INFINITY;
        best_at = INT32_MAX;
        for (int w = 0; w < kSampleWarps; ++w) {
            const float other = __uint_as_float(sm.list[0][w]);
            if (other > best) {                             // warps are in index order
                best = other;
                best_at = (int)sm.list[1][w];
            }
        }
        push_u32(&sm.best[rank], threadIdx.x, __float_as_uint(best));
        push_u32(&sm.best_at[rank], threadIdx.x, (uint32_t)best_at);
    }
    s.cluster_sync();
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
    s.scale.set(best, temperature);

    Cut cut{-INFINITY, 0, 0, 0};                            // everything
    const bool by_k = top_k > 0 && top_k < p.V, by_p = top_p < 1.f;
    if (by_k || by_p) {
        uint64_t count[4], mass[4], bin[4];
        s.histogram(by_p, [&](float, float t) { return s.scale.bin(t); }, count, mass);
        uint64_t total = ~0ull;
        if (by_k && s.bin_of(count, mass, false, (uint64_t)top_k, bin)) {
            cut = s.cut_in(bin, false, by_p, (uint64_t)top_k);
            total = cut.above + cut.ties * cut.each;
        }
        if (by_p) {
            if (total == ~0ull) {
                uint64_t c = 0, m = mass[0] + mass[1] + mass[2] + mass[3];
                const uint64_t mine = m;
                block_below(c, m, sm);
                if (threadIdx.x == kSampleThreads - 1) sm.found[0] = m + mine;
                __syncthreads();
                total = sm.found[0];
                __syncthreads();
            }
            const uint64_t target = max(part_of(top_p, total, true), (uint64_t)1);
            if (s.bin_of(count, mass, true, target, bin)) cut = s.cut_in(bin, true, true, target);
        }
    }

    // Mass of what is kept, over warps, blocks and the row; equal values at the cut count by index.
    const uint64_t least = min_p > 0.f ? part_of(fminf(min_p, 0x1.fffffep-1f), 1ull << kOneLog2, true) : 0;
    const bool only_best = min_p >= 1.f;
    const auto kept_weight = [&](float l) -> uint64_t {     // of a value above the cut
        const uint64_t w = s.scale.weight(l, s.scale.place(l), sm.table);
        return l == best || (w >= least && !only_best) ? w : 0;
    };
    cut.each = cut.value == -INFINITY ? 0 : kept_weight(cut.value);
    uint64_t mass = 0;
    uint32_t ties = 0;
    s.each([&](int, const float (&l)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (l[i] > cut.value) mass += kept_weight(l[i]);
            ties += l[i] == cut.value;
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
    s.cluster_sync();
    // Mass of m above the cut and the t-th to (t + n)-th values equal to it.
    const auto with_ties = [&](uint64_t m, uint32_t t, uint32_t n) { return m + (min(t + n, cut.ties) - min(t, cut.ties)) * cut.each; };
    uint64_t whole = 0;
    uint32_t seen = 0;
    for (uint32_t r = 0; r < ranks; ++r) {
        whole += with_ties(sm.mass[r], seen, sm.ties[r]);
        seen += sm.ties[r];
    }
    const float u = p.u[b];
    const uint64_t target = u < 1.f ? part_of(u, whole, false) : whole - 1;
    uint64_t before = 0;
    seen = 0;
    for (uint32_t r = 0; r < rank; ++r) {
        before += with_ties(sm.mass[r], seen, sm.ties[r]);
        seen += sm.ties[r];
    }
    for (int w = 0; w < warp; ++w) {
        before += with_ties(sm.warp_mass[w], seen, sm.warp_ties[w]);
        seen += sm.warp_ties[w];
    }
    // The warp that holds the running mass's passage goes through its values again.
    if (target < before || target >= before + with_ties(mass, seen, ties)) return;
    for (int j = s.j0 + lane * 8; j - lane * 8 < s.j1; j += 256) {
        float l[8];
        if (j < s.j1) row.eight(j, l);
        else
            for (int i = 0; i < 8; ++i) l[i] = -INFINITY;
        uint64_t m = 0;
        uint32_t n = 0;
        if (j < s.j1)
            for (int i = 0; i < 8; ++i) {
                if (l[i] > cut.value) m += kept_weight(l[i]);
                n += l[i] == cut.value;
            }
        uint32_t at = seen + warp_below(n, lane);
        const uint64_t mine = with_ties(m, at, n);
        uint64_t sum = before + warp_below(mine, lane);
        if (target >= sum && target < sum + mine) {
            for (int i = 0; i < 8; ++i) {
                const uint64_t w = l[i] > cut.value ? kept_weight(l[i]) : l[i] == cut.value && at++ < cut.ties ? cut.each : 0;
                if (target >= sum && target < sum + w) {
                    p.tokens[b] = j + i - row.first;
                    if (p.logprobs) {
                        // log(w / whole): near one by what is missing, else by the exact place.
                        const float all = (float)whole;
                        p.logprobs[b] = w > whole / 2 ? log1pf(-(float)(whole - w) / all)
                                                      : s.scale.exact_place(l[i]) * 0.693147180559945f - logf(all * (1.f / (float)(1ull << kOneLog2)));
                    }
                }
                sum += w;
            }
        }
        before += warp_sum(mine);
        seen += warp_sum(n);
    }
}

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
    // Blocks of a row: enough of them to fill the SMs with two each, none with less than 4096 logits.
    unsigned ranks = 1;
    while (ranks < kMaxCluster && B * ranks < sm_count() && V / (2 * ranks) >= 4096) ranks *= 2;
    SampleParams p{};
    p.logits = logits; p.stride = row_stride; p.u = u; p.how = *how; p.tokens = tokens; p.logprobs = logprobs;
    p.V = (int)V;
    p.slice = (int)round_up(ceil_div(V + 7, ranks), 8 * kSampleWarps);
    const void* kernel = type == NVFP4_LOGITS_BF16 ? (const void*)sample_kernel<kTypeBf16>
                       : type == NVFP4_LOGITS_F16 ? (const void*)sample_kernel<kTypeF16> : (const void*)sample_kernel<kTypeF32>;
    void* args[] = {&p};
    return launch_kernel(kernel, dim3((unsigned)(B * ranks)), dim3(kSampleThreads), 0, ranks, args, (cudaStream_t)stream, fn);
}
