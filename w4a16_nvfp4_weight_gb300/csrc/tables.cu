// Page tables of a batch, kept on the device: pages taken from a stack of free ones
// as requests grow, with the positions and slots of their new tokens, and pages given
// back as they shrink or end.
//
// Request b holds n tokens in ceil(n / page_size) pages.  With m new ones it needs
// ceil((n + m) / page_size) - ceil(n / page_size) more, taken from the top of the
// stack in the order of the requests: exclusive sums of the needs say where.  Whole
// numbers throughout, so nothing depends on the order of anything.
//
// Bound by latency: a chain of loads (lengths, table or stack), two sums over the
// block and a search, against bytes that take a tenth of a microsecond (64 requests by a token 3.5
// us, 16384 rows of 48 prompts 6.1, 1000 requests of which 600 end 4.2).  So every block sums all
// requests for itself, and one launch does everything.
#include <algorithm>

#include "common.cuh"
#include "launch.cuh"
#include "overlap.cuh"
#include "ptx.cuh"

namespace nvfp4 {
namespace {

constexpr int kMaxRequests = 16384;        // 12 bytes each of shared memory
constexpr int kTableThreads = 1024;

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}

// Sum over the threads below this one, and over all; `sm` holds 33 values, free
// again when the call returns in every thread.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sm, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sm[warp] = x;
    __syncthreads();
    int64_t w = lane < warps ? sm[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int64_t below = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    __syncthreads();
    return x - v + (warp ? below : 0);
}

// Pages of n tokens, 0 <= n < 2^31: by 32 bits, which n + page - 1 does not leave (64 took 13.9 us of
// 64 requests' extension where this takes 3.7).
__device__ __forceinline__ int pages_of(int n, int page) { return (int)((uint32_t)(n + (uint32_t)page - 1u) / (uint32_t)page); }

struct ExtendParams {
    const int32_t *lengths, *fresh;        // tokens cached, and new ones, of each request
    int32_t* table;
    const int32_t *pages, *count;          // the stack of free pages
    int64_t *positions, *slots;
    int32_t *request, *starts, *lengths_out, *count_out, *row_lengths;
    int64_t table_stride;
    int B, rows, width, P, page;
    int* status;
};

// Blocks of one cluster; each holds every request's first row, cached tokens and place
// in the stack, and takes its share of the rows.  All have read the lengths and the
// count before the first block writes them (they may be the same tensors).
__global__ void __launch_bounds__(kTableThreads) extend_kernel(const ExtendParams p) {
    extern __shared__ int32_t sm_requests[];
    __shared__ int64_t sm_scan[33];
    int32_t* start = sm_requests;                  // [B + 1]
    int32_t* held = start + p.B + 1;               // [B]
    int32_t* place = held + p.B;                   // [B]: pages taken by the requests before, -1: not served
    pdl_wait_previous();
    pdl_launch_dependents();
    const int tid = threadIdx.x, per = (p.B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    const uint32_t rank = blockIdx.x, ranks = gridDim.x;
    bool bad = false;
    int count = *p.count;
    if (count < 0 || count > p.P) {
        bad = true;
        count = min(max(count, 0), p.P);
    }
    int64_t rows = 0, total;
    for (int b = b0; b < b1; ++b) {
        const int m = p.fresh[b], n = p.lengths[b];
        bad |= m < 0 || n < 0;
        rows += max(m, 0);
    }
    int64_t at = block_scan(rows, sm_scan, &total);
    if (tid == 0) start[p.B] = (int)min(total, (int64_t)p.rows);
    int64_t needs = 0;
    const auto need_of = [&](int n, int m, int64_t row) {                     // -1: does not fit
        if (n < 0 || m < 0 || m > INT32_MAX - n || row + m > p.rows) return -1;
        const int last = pages_of(n + m, p.page);
        return last > p.width ? -1 : last - pages_of(n, p.page);
    };
    {
        int64_t row = at;
        for (int b = b0; b < b1; ++b) {
            const int m = p.fresh[b];
            needs += max(need_of(p.lengths[b], m, row), 0);
            row += max(m, 0);
        }
    }
    int64_t asked = block_scan(needs, sm_scan, &total);
    int64_t served_pages = 0;
    bool several = false;
    for (int b = b0; b < b1; ++b) {
        const int n = p.lengths[b], m = p.fresh[b];
        const int need = need_of(n, m, at);
        const bool served = need == 0 || (need > 0 && asked + need <= count);
        start[b] = (int)min(at, (int64_t)p.rows);
        held[b] = n;
        place[b] = !served ? -1 : need > 0 ? (int)asked : 0;
        if (served) served_pages += need;
        several |= served && need > 1;
        asked += max(need, 0);
        at += max(m, 0);
    }
    block_scan(served_pages, sm_scan, &total);
    if (bad) record_status(p.status, NVFP4_ERR_BAD_INDEX);
    several = __syncthreads_or(several);
    if (ranks > 1) {
        cluster_arrive();
        cluster_wait();
    }
    const int gthreads = ranks * blockDim.x, gid = rank * blockDim.x + tid;
    // The first page of a request by a thread, more of them by a warp.
    for (int b = gid; b < p.B; b += gthreads) {
        const int n = held[b];
        const int m = max(start[b + 1] - start[b], 0);      // all its rows where it is served
        p.starts[b] = start[b];
        p.lengths_out[b] = place[b] >= 0 ? n + m : n;
        if (place[b] >= 0) {
            const int first = pages_of(n, p.page);
            if (pages_of(n + m, p.page) > first) p.table[b * p.table_stride + first] = p.pages[count - 1 - place[b]];
        }
    }
    if (gid == 0) {
        p.starts[p.B] = start[p.B];
        *p.count_out = count - (int)total;
    }
    for (int b = several ? gid >> 5 : p.B; b < p.B; b += gthreads >> 5) {
        if (place[b] < 0) continue;
        const int n = held[b], first = pages_of(n, p.page);
        const int last = pages_of(n + start[b + 1] - start[b], p.page);
        for (int j = first + 1 + (tid & 31); j < last; j += 32)
            p.table[b * p.table_stride + j] = p.pages[count - 1 - place[b] - (j - first)];
    }
    for (int64_t t = gid; t < p.rows; t += gthreads) {
        int lo = 0, hi = p.B;                               // the last request that starts at or before t
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start[mid] <= t) lo = mid;
            else hi = mid;
        }
        int64_t position = 0, slot = -1;
        int request = -1, length = 0;
        if (t < start[p.B]) {
            const int n = max(held[lo], 0);
            request = lo;
            position = (int64_t)n + (t - start[lo]);
            if (place[lo] >= 0) {
                const int j = (int)((uint32_t)position / (uint32_t)p.page), first = pages_of(n, p.page);
                const int32_t page = j < first ? p.table[lo * p.table_stride + j] : p.pages[count - 1 - place[lo] - (j - first)];
                slot = (int64_t)page * p.page + (position - (int64_t)j * p.page);
                length = (int)position + 1;
            }
        }
        p.positions[t] = position;
        p.slots[t] = slot;
        p.request[t] = request;
        if (p.row_lengths) p.row_lengths[t] = length;
    }
}

struct RowTableParams {
    const int32_t *table, *request, *row_lengths;
    int32_t* out;                          // [rows, width]
    int64_t table_stride;
    int rows, width, page;
};

// Each row's table: its request's pages up to its own length, then zeros.  A warp takes
// 128 entries of a row.
__global__ void __launch_bounds__(256) row_tables_kernel(const RowTableParams p) {
    pdl_wait_previous();
    pdl_launch_dependents();
    const int parts = (p.width + 127) / 128;
    const int64_t total = (int64_t)p.rows * parts;
    for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += (int64_t)gridDim.x * 8) {
        const int64_t t = i / parts;
        const int j0 = (int)(i - t * parts) * 128 + (threadIdx.x & 31);
        const int b = p.request[t];
        const int used = pages_of(p.row_lengths[t], p.page);
        int32_t v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = j0 + 32 * k < used ? p.table[b * p.table_stride + j0 + 32 * k] : 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (j0 + 32 * k < p.width) p.out[t * p.width + j0 + 32 * k] = v[k];
    }
}

struct TrimParams {
    const int32_t *lengths, *keep, *table, *count;
    int32_t *pages, *lengths_out, *count_out;
    int64_t table_stride;
    int B, width, P, page;
    int copy, commit;                      // give pages back; write lengths and count
    int* status;
};

// Every block sums all requests; each gives back the pages of its share of them.
__global__ void __launch_bounds__(kTableThreads) trim_kernel(const TrimParams p) {
    extern __shared__ int32_t sm_requests[];
    __shared__ int64_t sm_scan[33];
    int32_t* after = sm_requests;                  // [B]: length from now on
    int32_t* gone = after + p.B;                   // [B]: pages given back
    int32_t* place = gone + p.B;                   // [B]: where on the stack
    pdl_wait_previous();
    pdl_launch_dependents();
    const int tid = threadIdx.x, per = (p.B + blockDim.x - 1) / blockDim.x;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    bool bad = false;
    int count = *p.count;
    if (count < 0 || count > p.P) {
        bad = true;
        count = min(max(count, 0), p.P);
    }
    int64_t sum = 0, total;
    for (int b = b0; b < b1; ++b) {
        const int n = p.lengths[b], k = p.keep[b];
        bad |= n < 0 || k < 0;
        const int a = n < 0 || k < 0 ? n : min(n, k);
        int first = 0, last = 0;
        if (a < n) {
            first = pages_of(a, p.page);
            last = pages_of(n, p.page);
            bad |= last > p.width;
            last = max(min(last, p.width), first);
        }
        after[b] = a;
        gone[b] = last - first;
        sum += last - first;
    }
    int64_t at = block_scan(sum, sm_scan, &total);
    for (int b = b0; b < b1; ++b) {
        at = min(at, (int64_t)p.P);                // beyond the stack: dropped
        place[b] = (int)at;
        at += gone[b];
    }
    if (count + total > p.P) {
        bad = true;
        total = p.P - count;
    }
    if (bad) record_status(p.status, NVFP4_ERR_BAD_INDEX);
    if (p.copy && p.commit && gridDim.x > 1 && cluster_size() == gridDim.x) {     // every block has read what the first ones write
        __syncwarp();
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    const int gthreads = gridDim.x * blockDim.x, gid = blockIdx.x * blockDim.x + tid;
    for (int b = gid; b < p.B; b += gthreads) {
        if (p.commit) p.lengths_out[b] = after[b];
        if (p.copy && gone[b] > 0) {
            const int64_t to = (int64_t)count + place[b];
            if (to < p.P) p.pages[to] = p.table[b * p.table_stride + pages_of(after[b], p.page)];
        }
    }
    if (p.commit && gid == 0) *p.count_out = count + (int)total;
    if (!p.copy) return;
    for (int b = gid >> 5; b < p.B; b += gthreads >> 5) {
        const int n = gone[b];
        if (n <= 1) continue;
        const int32_t* from = p.table + b * p.table_stride + pages_of(after[b], p.page);
        const int64_t to = (int64_t)count + place[b];
        const int m = (int)min((int64_t)n, p.P - to);
        for (int j0 = 1 + (tid & 31); j0 < m; j0 += 128) {
            int32_t v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = j0 + 32 * k < m ? from[j0 + 32 * k] : 0;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (j0 + 32 * k < m) p.pages[to + j0 + 32 * k] = v[k];
        }
    }
}

// What both entry points ask of the requests, the table and the stack.
nvfp4_status check_pool(const char* fn, int64_t B, int64_t width, int64_t table_stride, int64_t P, int64_t page) {
    if (B < 0 || width < 0 || P < 0 || table_stride < 0)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: negative size or stride (B=%lld, width=%lld, stride=%lld, pages=%lld)", fn, (long long)B,
                    (long long)width, (long long)table_stride, (long long)P);
    if (B > kMaxRequests) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: B=%lld must be at most %d", fn, (long long)B, kMaxRequests);
    if (width > INT32_MAX || P > INT32_MAX) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: table width or stack beyond 2^31 entries", fn);
    if (page < 1 || page > INT32_MAX) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: page_size=%lld must be in [1, 2^31)", fn, (long long)page);
    if (B > 1 && table_stride < width)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: rows of the table %lld apart overlap (width %lld)", fn, (long long)table_stride, (long long)width);
    return NVFP4_OK;
}

// Block and cluster for B requests and `work` independent items: a block for up to 1024.
void shape_of(int64_t B, int64_t work, int* threads, int* blocks) {
    const int64_t most = std::max(B, work);
    *threads = (int)std::min<int64_t>(kTableThreads, round_up(std::max<int64_t>(most, 1), 32));
    *blocks = 1;
    while (*blocks < 8 && (int64_t)*blocks * kTableThreads < work) *blocks *= 2;
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status nvfp4_extend_tables(const int32_t* lengths, const int32_t* new_tokens, int64_t B, int32_t* block_table,
                                            int64_t table_stride, int64_t table_width, const int32_t* free_pages, int64_t num_free,
                                            const int32_t* free_count, int64_t page_size, int64_t rows, int64_t* positions,
                                            int64_t* slots, int32_t* request, int32_t* starts, int32_t* lengths_out,
                                            int32_t* free_count_out, int32_t* row_tables, int32_t* row_lengths, void* stream) {
    const char* fn = "nvfp4_extend_tables";
    if (nvfp4_status st = check_pool(fn, B, table_width, table_stride, num_free, page_size)) return st;
    if (rows < 0) return fail(NVFP4_ERR_INVALID_ARG, "%s: negative size rows=%lld", fn, (long long)rows);
    if (rows > INT32_MAX) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: rows=%lld too large", fn, (long long)rows);
    if (!free_count || !starts || !free_count_out || (B > 0 && (!lengths || !new_tokens || !lengths_out)) || (B > 0 && table_width > 0 && !block_table) ||
        (num_free > 0 && !free_pages) || (rows > 0 && (!positions || !slots || !request)))
        return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", fn);
    if ((row_tables != nullptr) && !row_lengths) return fail(NVFP4_ERR_INVALID_ARG, "%s: row_tables needs row_lengths", fn);
    for (const void* q : {(const void*)lengths, (const void*)new_tokens, (const void*)block_table, (const void*)free_pages, (const void*)free_count,
                          (const void*)request, (const void*)starts, (const void*)lengths_out, (const void*)free_count_out, (const void*)row_tables, (const void*)row_lengths})
        if (!aligned(q, 4)) return fail(NVFP4_ERR_ALIGNMENT, "%s: pointers must be aligned to their elements", fn);
    if (!aligned(positions, 8) || !aligned(slots, 8)) return fail(NVFP4_ERR_ALIGNMENT, "%s: positions and slots must be 8-byte aligned", fn);
    const Span n = dense_span("lengths", lengths, 4 * B), m = dense_span("new_tokens", new_tokens, 4 * B);
    const Span tab = strided_span("block_table", block_table, 4 * table_width, {{B, 4 * table_stride}});
    const Span stack = dense_span("free_pages", free_pages, 4 * num_free), top = dense_span("free_count", free_count, 4);
    const Span outs[] = {dense_span("positions", positions, 8 * rows), dense_span("slots", slots, 8 * rows), dense_span("request", request, 4 * rows),
                         dense_span("starts", starts, 4 * (B + 1)), dense_span("lengths_out", lengths_out, 4 * B),
                         dense_span("free_count_out", free_count_out, 4), dense_span("row_tables", row_tables, 4 * rows * table_width),
                         dense_span("row_lengths", row_lengths, 4 * rows)};
    for (const Span& in : {n, m, stack, top})
        if (overlaps(in, tab)) return fail(NVFP4_ERR_INVALID_ARG, "%s: block_table overlaps %s", fn, in.name);
    for (const Span& out : outs) {
        if (const char* s = met(out, {m, tab, stack})) return fail(NVFP4_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, out.name, s);
        if (overlaps(out, n) && out.at != (uintptr_t)lengths_out) return fail(NVFP4_ERR_INVALID_ARG, "%s: %s overlaps lengths", fn, out.name);
        if (overlaps(out, top) && out.at != (uintptr_t)free_count_out) return fail(NVFP4_ERR_INVALID_ARG, "%s: %s overlaps free_count", fn, out.name);
        for (const Span& other : outs)
            if (&other < &out && overlaps(out, other)) return fail(NVFP4_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, out.name, other.name);
    }
    // In place these are their inputs, element for element.
    if (overlaps(outs[4], n) && lengths_out != lengths) return fail(NVFP4_ERR_INVALID_ARG, "%s: lengths_out overlaps lengths (it may be lengths itself)", fn);
    if (overlaps(outs[4], top) || overlaps(outs[5], n)) return fail(NVFP4_ERR_INVALID_ARG, "%s: lengths and free_count overlap", fn);
    ExtendParams p{};
    p.status = device_status_ptr();
    if (!p.status) return fail(NVFP4_ERR_CUDA, "%s: no CUDA device", fn);
    p.lengths = lengths; p.fresh = new_tokens; p.table = block_table; p.pages = free_pages; p.count = free_count;
    p.positions = positions; p.slots = slots; p.request = request; p.starts = starts; p.lengths_out = lengths_out;
    p.count_out = free_count_out; p.row_lengths = row_lengths; p.table_stride = table_stride;
    p.B = (int)B; p.rows = (int)rows; p.width = (int)table_width; p.P = (int)num_free; p.page = (int)page_size;
    int threads, blocks;
    shape_of(B, rows, &threads, &blocks);
    void* args[] = {&p};
    if (nvfp4_status st = launch_kernel((const void*)extend_kernel, dim3(blocks), dim3(threads), 4 * (3 * B + 1), blocks, args, (cudaStream_t)stream, fn)) return st;
    if (!row_tables || rows == 0 || table_width == 0) return NVFP4_OK;
    RowTableParams q{block_table, request, row_lengths, row_tables, table_stride, p.rows, p.width, p.page};
    void* qargs[] = {&q};
    const int64_t warps = rows * ceil_div(table_width, 128);
    return launch_kernel((const void*)row_tables_kernel, dim3((unsigned)std::min<int64_t>(ceil_div(warps, 8), (int64_t)sm_count() * 16)), dim3(256), 0,
                         1, qargs, (cudaStream_t)stream, fn);
}

extern "C" nvfp4_status nvfp4_trim_tables(const int32_t* lengths, const int32_t* keep, int64_t B, const int32_t* block_table,
                                          int64_t table_stride, int64_t table_width, int32_t* free_pages, int64_t num_free,
                                          const int32_t* free_count, int64_t page_size, int32_t* lengths_out, int32_t* free_count_out,
                                          void* stream) {
    const char* fn = "nvfp4_trim_tables";
    if (nvfp4_status st = check_pool(fn, B, table_width, table_stride, num_free, page_size)) return st;
    if (!free_count || !free_count_out || (B > 0 && (!lengths || !keep || !lengths_out)) || (B > 0 && table_width > 0 && !block_table) ||
        (num_free > 0 && !free_pages))
        return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", fn);
    for (const void* q : {(const void*)lengths, (const void*)keep, (const void*)block_table, (const void*)free_pages, (const void*)free_count,
                          (const void*)lengths_out, (const void*)free_count_out})
        if (!aligned(q, 4)) return fail(NVFP4_ERR_ALIGNMENT, "%s: pointers must be aligned to their elements", fn);
    const Span n = dense_span("lengths", lengths, 4 * B), k = dense_span("keep", keep, 4 * B), top = dense_span("free_count", free_count, 4);
    const Span tab = strided_span("block_table", block_table, 4 * table_width, {{B, 4 * table_stride}});
    const Span stack = dense_span("free_pages", free_pages, 4 * num_free);
    const Span after = dense_span("lengths_out", lengths_out, 4 * B), count = dense_span("free_count_out", free_count_out, 4);
    if (const char* s = met(stack, {n, k, tab, top, after, count})) return fail(NVFP4_ERR_INVALID_ARG, "%s: free_pages overlaps %s", fn, s);
    if (const char* s = met(after, {k, tab, top, count})) return fail(NVFP4_ERR_INVALID_ARG, "%s: lengths_out overlaps %s", fn, s);
    if (const char* s = met(count, {n, k, tab})) return fail(NVFP4_ERR_INVALID_ARG, "%s: free_count_out overlaps %s", fn, s);
    if (overlaps(after, n) && lengths_out != lengths) return fail(NVFP4_ERR_INVALID_ARG, "%s: lengths_out overlaps lengths (it may be lengths itself)", fn);
    TrimParams p{};
    p.status = device_status_ptr();
    if (!p.status) return fail(NVFP4_ERR_CUDA, "%s: no CUDA device", fn);
    p.lengths = lengths; p.keep = keep; p.table = block_table; p.count = free_count; p.pages = free_pages; p.lengths_out = lengths_out;
    p.count_out = free_count_out; p.table_stride = table_stride; p.B = (int)B; p.width = (int)table_width; p.P = (int)num_free;
    p.page = (int)page_size; p.copy = 1; p.commit = 1;
    void* args[] = {&p};
    const size_t smem = 4 * 3 * (size_t)B;
    const bool in_place = lengths_out == lengths || free_count_out == free_count;
    const int64_t entries = std::min(B * table_width, num_free);           // that can come back
    int threads, blocks;
    if (entries <= 65536) {
        shape_of(B, std::max(B, entries / 8), &threads, &blocks);
        return launch_kernel((const void*)trim_kernel, dim3(blocks), dim3(threads), smem, blocks, args, (cudaStream_t)stream, fn);
    }
    // More pages than the eight SMs of a cluster move quickly: a block an SM, and in place the
    // lengths and the count by a launch of their own, after every block has read them.
    blocks = (int)std::min<int64_t>(ceil_div(entries, 4096), sm_count());
    p.commit = !in_place;
    if (nvfp4_status st = launch_kernel((const void*)trim_kernel, dim3(blocks), dim3(kTableThreads), smem, 1, args, (cudaStream_t)stream, fn)) return st;
    if (!in_place) return NVFP4_OK;
    p.copy = 0; p.commit = 1;
    return launch_kernel((const void*)trim_kernel, dim3(1), dim3(kTableThreads), smem, 1, args, (cudaStream_t)stream, fn);
}
