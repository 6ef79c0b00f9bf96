// The paged key-value cache as the kernels see it, and the host checks that the
// entry points taking one share.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "overlap.cuh"

namespace nvfp4 {

constexpr int kMaxHeadDim = 256;

struct CacheView {
    uint8_t *k, *v;                // 16-bit activations or E4M3 codes
    float *k_scale, *v_scale;      // [pages, heads, page_size], E4M3 only
    int64_t num_pages, num_slots;  // slots = pages * page_size
    int64_t page_bytes, head_bytes, token_bytes;
    int page_size, heads, D;
    int page_shift;                // log2(page_size), or -1
    uint32_t page_mul;             // where that is -1: 2^(32 + page_mul_shift) / page_size, rounded up
    int page_mul_shift;
    bool e4m3;

    // t / page_size for t < 2^31, by a product (Granlund and Montgomery, PLDI 1994): page_mul
    // is above the quotient by less than page_size <= 2^(page_mul_shift + 1), in units of
    // 2^-(32 + page_mul_shift) / page_size, which t < 2^31 cannot carry to the next integer.
    __device__ int entry(int t) const {
        return page_shift >= 0 ? t >> page_shift : (int)(__umulhi((uint32_t)t, page_mul) >> page_mul_shift);
    }

    // Page and place of a slot below num_slots (a 64-bit division only where nothing shorter will do).
    __device__ void split(int64_t slot, int64_t* page, int* at) const {
        if (page_shift >= 0) *page = slot >> page_shift;
        else if (num_slots <= INT32_MAX) *page = entry((int32_t)slot);
        else *page = slot / page_size;
        *at = (int)(slot - *page * page_size);
    }

    // Byte offset of token `at` of `page`, head h: 64-bit, a cache passes 4 GB.
    __host__ __device__ int64_t row(int64_t page, int h, int at) const {
        return page * page_bytes + (int64_t)h * head_bytes + (int64_t)at * token_bytes;
    }
    __host__ __device__ int64_t scale_at(int64_t page, int h, int at) const {
        return (page * heads + h) * page_size + at;
    }
};

// The cache's rows, keys or values, and scales.
inline Span cache_span(const char* name, const CacheView& c, const void* rows) {
    return strided_span(name, rows, (int64_t)c.D * (c.e4m3 ? 1 : 2), {{c.num_pages, c.page_bytes}, {c.heads, c.head_bytes}, {c.page_size, c.token_bytes}});
}
inline Span scale_span(const char* name, const CacheView& c, const float* scale) {
    return dense_span(name, scale, 4 * c.num_slots * c.heads);
}
// The cache's part that `out` overlaps, or null.
inline const char* met_cache(const Span& out, const CacheView& c) {
    return met(out, {cache_span("the cache's keys", c, c.k), cache_span("the cache's values", c, c.v),
                     scale_span("the cache's scales", c, c.k_scale), scale_span("the cache's scales", c, c.v_scale)});
}

// Checks `c` and fills `view`.
nvfp4_status check_cache(const char* fn, const nvfp4_kv_cache* c, CacheView* view);

}  // namespace nvfp4
