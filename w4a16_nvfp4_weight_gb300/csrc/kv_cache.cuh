// The paged key-value cache as the kernels see it, and the host checks that the
// entry points taking one share.
#pragma once

#include <cstdint>

#include "common.cuh"

namespace nvfp4 {

constexpr int kMaxHeadDim = 256;

struct CacheView {
    uint8_t *k, *v;                // 16-bit activations or E4M3 codes
    float *k_scale, *v_scale;      // [pages, heads, page_size], E4M3 only
    int64_t num_pages, num_slots;  // slots = pages * page_size
    int64_t page_bytes, head_bytes, token_bytes;
    int page_size, heads, D;
    int page_shift;                // log2(page_size), or -1
    bool e4m3;

    // Page and place of a slot below num_slots (a 64-bit division only where nothing shorter will do).
    __device__ void split(int64_t slot, int64_t* page, int* at) const {
        if (page_shift >= 0) *page = slot >> page_shift;
        else if (num_slots <= INT32_MAX) *page = (int32_t)slot / page_size;
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

// Checks `c` and fills `view`.
nvfp4_status check_cache(const char* fn, const nvfp4_kv_cache* c, CacheView* view);

}  // namespace nvfp4
