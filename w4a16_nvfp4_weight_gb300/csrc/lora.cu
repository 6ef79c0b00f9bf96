// Low-rank adapters of many requests at once, beside a projection that all share:
//     out_t = RN(y_t + s_a B_a (A_a x_t)),  a = adapters[t]  (a < 0: out_t = y_t).
// x, y, A and B are 16-bit; A x and its sums are held in 32 bits and meet B as two 16-bit halves, right
// to 2^-16 of a value for BF16, for FP16 to 2^-22 of it or 2^-39 of the row's largest, whichever is more.
//
// Rows are grouped by adapter into items of up to 16 or 64 rows of one adapter (rows of a
// request need not lie side by side): by every block for itself, or of more than 128 rows by
// one block ahead.  The down kernels multiply an item's rows with A, the long axis K split
// over blocks and warps; the up kernels add the splits' sums in their order (no atomics: the
// same bits every time), multiply with B onto y.  Both products are mma.sync m16n8k16: at
// rank r they do r flop for each byte of x or y that they read or write, far below what would
// need tcgen05.  An order of k that is the same for both operands lets a lane load 16 bytes of each row, and
// an order of the columns 16 bytes of y.
// Few rows are bound by latency (1 x 4096 x 4096, rank 16, 4.7 us; 64 x 4096 x 28672 16.5, 2.5
// TB/s), many by memory and the products (8192 x 4096 x 4096, rank 64, 65.7 us, 3.1 TB/s).
#include <algorithm>

#include "common.cuh"
#include "launch.cuh"
#include "numeric.cuh"
#include "overlap.cuh"
#include "ptx.cuh"
#include "stream_mma.cuh"

namespace nvfp4 {
namespace {

constexpr int kMaxAdapters = 4096;
constexpr int kMaxRank = 256;
constexpr int kLoraThreads = 128;
constexpr int kMaxSplits = 16;
constexpr int kSelfRows = kLoraThreads;    // up to so many rows every block finds its item for itself

struct Item { int32_t adapter, first, rows, pad; };      // rows order[first .. first + rows)

struct LoraParams {
    const uint16_t *x, *a, *b, *y;
    const int32_t* adapters;
    const float* scales;                   // null: 1
    uint16_t* out;
    int64_t T, K, N, x_stride, y_stride;
    int n, r, rp;                          // adapters, rank, padded_rank(r)
    int splits, k_split;                   // of K, and its elements a split (a multiple of 32)
    int rows_item;                         // 16 or 64
    int copy_rest;                         // rows without an adapter are copied
    int32_t* num_items;                    // null: every block finds its item for itself
    Item* items;
    int32_t* order;                        // [T] rows by adapter
    float* low;                            // [splits, T, rp] A x
    int* status;
};

// Rows by adapter, and items of them.  One block; eight rows a thread at a time, and one addition
// for neighbours of the same adapter (8192 rows 13.2 us with an addition and a load a row).
__global__ void __launch_bounds__(1024) lora_group_kernel(const LoraParams p) {
    extern __shared__ int32_t sm_groups[];
    __shared__ int32_t warp_sum[2][32];
    int32_t* count = sm_groups;            // [n + 1] rows of each adapter; the last: without one
    int32_t* place = count + p.n + 1;      // [n + 1] where the next of them goes
    pdl_wait_previous();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, groups = p.n + 1;
    for (int g = tid; g < groups; g += blockDim.x) count[g] = 0;
    __syncthreads();
    constexpr int kEach = 8;
    const int64_t round = (int64_t)blockDim.x * kEach;
    int group[kEach];
    const auto read = [&](int64_t t0) {                     // of this round; -1 behind the last row
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int64_t t = t0 + i * blockDim.x + tid;
            group[i] = t < p.T ? p.adapters[t] : INT32_MIN;
        }
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            if (group[i] >= p.n) record_status(p.status, NVFP4_ERR_BAD_INDEX);
            group[i] = group[i] == INT32_MIN && t0 + i * blockDim.x + tid >= p.T ? -1 : group[i] < 0 || group[i] >= p.n ? p.n : group[i];
        }
    };
    for (int64_t t0 = 0; t0 < p.T; t0 += round) {
        read(t0);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const uint32_t same = __match_any_sync(0xffffffffu, group[i]);
            if (group[i] >= 0 && lane == __ffs(same) - 1) atomicAdd(&count[group[i]], __popc(same));
        }
    }
    __syncthreads();
    // Exclusive sums of rows and items over the groups, a run of groups a thread.
    const int per = (groups + blockDim.x - 1) / blockDim.x, g0 = min(tid * per, groups), g1 = min(g0 + per, groups);
    int rows = 0, items = 0;
    for (int g = g0; g < g1; ++g) {
        rows += count[g];
        items += (count[g] + p.rows_item - 1) / p.rows_item;
    }
    int r = rows, i = items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, r, o), v = __shfl_up_sync(0xffffffffu, i, o);
        if (lane >= o) {
            r += u;
            i += v;
        }
    }
    if (lane == 31) {
        warp_sum[0][warp] = r;
        warp_sum[1][warp] = i;
    }
    __syncthreads();
    r -= rows;
    i -= items;
    for (int w = 0; w < warp; ++w) {
        r += warp_sum[0][w];
        i += warp_sum[1][w];
    }
    for (int g = g0; g < g1; ++g) {
        place[g] = r;
        const int adapter = g == p.n ? -1 : g;
        for (int at = 0; at < count[g]; at += p.rows_item)
            p.items[i++] = Item{adapter, r + at, min(p.rows_item, count[g] - at), 0};
        r += count[g];
    }
    if (tid == blockDim.x - 1) *p.num_items = i;            // the threads past the last group hold the sum, too
    __syncthreads();
    for (int64_t t0 = 0; t0 < p.T; t0 += round) {
        if (p.T > round) read(t0);                          // else they are still here
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const uint32_t same = __match_any_sync(0xffffffffu, group[i]);
            const int leader = __ffs(same) - 1;
            int at = 0;
            if (group[i] >= 0 && lane == leader) at = atomicAdd(&place[group[i]], __popc(same));
            at = __shfl_sync(0xffffffffu, at, leader) + __popc(same & ((1u << lane) - 1));
            if (group[i] >= 0) p.order[at] = (int32_t)(t0 + i * blockDim.x + tid);
        }
    }
}

// The rows of a block's item.
template <int ROWS>
struct ItemRows {
    int32_t row[ROWS];
    alignas(16) int32_t ids[kSelfRows];
    int32_t warp_starts[kLoraThreads / 32];
    int32_t adapter, first;

    // Item `it`, its adapter and number of rows; false where there is none.  Of the few rows that have no list,
    // each 16th of an adapter begins an item, in the order of the rows.
    __device__ __forceinline__ bool find(const LoraParams& p, int it, int* adapter_out, int* rows_out) {
        const int tid = threadIdx.x;
        if (p.num_items) {
            if (it >= *p.num_items) return false;
            const Item item = p.items[it];
            *adapter_out = item.adapter;
            *rows_out = item.rows;
            if (tid < item.rows) row[tid] = p.order[item.first + tid];
            __syncthreads();
            return true;
        }
        int id = INT32_MIN;                                 // behind the last row
        if (tid < p.T) {
            id = p.adapters[tid];
            if (id >= p.n && it == 0) record_status(p.status, NVFP4_ERR_BAD_INDEX);
            if (id < 0 || id >= p.n) id = -1;
        }
        ids[tid] = id;
        if (tid == 0) first = -1;
        __syncthreads();
        int rank = 0;
#pragma unroll 4
        for (int t = 0; t < (int)p.T; t += 4) {             // what follows the last row is no adapter's
            const int4 v = *(const int4*)(ids + t);
            rank += (t < tid && v.x == id) + (t + 1 < tid && v.y == id) + (t + 2 < tid && v.z == id) + (t + 3 < tid && v.w == id);
        }
        const bool starts = id >= (p.copy_rest ? -1 : 0) && rank % ROWS == 0;
        const uint32_t mine = __ballot_sync(0xffffffffu, starts);
        if ((tid & 31) == 0) warp_starts[tid >> 5] = __popc(mine);
        __syncthreads();
        int index = __popc(mine & ((1u << (tid & 31)) - 1));
        for (int w = 0; w < tid >> 5; ++w) index += warp_starts[w];
        if (starts && index == it) {
            adapter = id;
            first = rank;
        }
        __syncthreads();
        if (first < 0) return false;
        const bool in = id == adapter && rank >= first && rank < first + ROWS;
        if (in) row[rank - first] = tid;
        *adapter_out = adapter;
        *rows_out = __syncthreads_count(in);
        return true;
    }
};

// Eight 16-bit elements, zero where they are outside; VEC: all or none, 16-byte aligned.
template <bool VEC>
__device__ __forceinline__ uint4 eight(const uint16_t* p, int64_t left) {
    if (VEC) return left > 0 ? *(const uint4*)p : make_uint4(0, 0, 0, 0);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) w[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One item's rows times 8 * NT rows of A over one split of K.  A warp takes MT * 16 rows and 32 k of a
// step, four lanes 16 bytes each of a row; RW warps take the rows, and the others of four the next k.
// Rows of 64 share their A through L1.
template <bool F16, int RW, int MT, int NT, bool VEC>
__global__ void __launch_bounds__(kLoraThreads) lora_down_kernel(const LoraParams p) {
    constexpr int kRows = 16 * MT * RW, kCols = 8 * NT, kKWarps = kLoraThreads / 32 / RW;
    __shared__ float sm[kKWarps][kRows][kCols + 4];
    __shared__ ItemRows<kRows> item;
    pdl_wait_previous();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    const int row_warp = warp % RW, k_warp = warp / RW;
    const int split = blockIdx.y, col0 = blockIdx.z * kCols;
    int adapter, rows;
    if (!item.find(p, blockIdx.x, &adapter, &rows) || adapter < 0) return;
    const int64_t k_begin = (int64_t)split * p.k_split, k_end = min(k_begin + p.k_split, p.K);
    const uint16_t* xr[MT][2];
    bool held[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = (row_warp * MT + m) * 16 + h * 8 + g;
            held[m][h] = row < rows;
            xr[m][h] = p.x + (held[m][h] ? item.row[row] : 0) * p.x_stride;
        }
    const uint16_t* a = p.a + ((int64_t)adapter * p.r + col0 + g) * p.K;
    float acc[MT][NT][4] = {};
    constexpr int U = MT * 2 + NT <= 4 ? 4 : MT * 2 + NT <= 6 ? 2 : 1;         // steps whose loads go out together
    for (int64_t k0 = k_begin + k_warp * 32; k0 < k_end; k0 += kKWarps * 32 * U) {
        uint4 xv[U][MT][2], av[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t k = k0 + u * kKWarps * 32 + q * 8, left = k_end - k;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) xv[u][m][h] = held[m][h] ? eight<VEC>(xr[m][h] + k, left) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < NT; ++j) av[u][j] = col0 + j * 8 + g < p.r ? eight<VEC>(a + (int64_t)j * 8 * p.K + k, left) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint32_t lo[4] = {xv[u][m][0].x, xv[u][m][1].x, xv[u][m][0].y, xv[u][m][1].y};
                const uint32_t hi[4] = {xv[u][m][0].z, xv[u][m][1].z, xv[u][m][0].w, xv[u][m][1].w};
#pragma unroll
                for (int j = 0; j < NT; ++j) mma_16816<F16>(acc[m][j], lo, av[u][j].x, av[u][j].y);
#pragma unroll
                for (int j = 0; j < NT; ++j) mma_16816<F16>(acc[m][j], hi, av[u][j].z, av[u][j].w);
            }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *(float2*)&sm[k_warp][(row_warp * MT + m) * 16 + h * 8 + g][j * 8 + q * 2] = make_float2(acc[m][j][2 * h], acc[m][j][2 * h + 1]);
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * kCols / 4; i += kLoraThreads) {
        const int row = i / (kCols / 4), c = i % (kCols / 4) * 4;
        if (row >= rows || col0 + c >= p.rp) continue;
        float4 v = *(const float4*)&sm[0][row][c];
#pragma unroll
        for (int w = 1; w < kKWarps; ++w) {
            const float4 u = *(const float4*)&sm[w][row][c];
            v.x += u.x;
            v.y += u.y;
            v.z += u.z;
            v.w += u.w;
        }
        *(float4*)(p.low + ((int64_t)split * p.T + item.row[row]) * p.rp + col0 + c) = v;
    }
}

constexpr int kRingStages = 4;

// The same for items of 64 rows and 16-byte rows: stages of 64 k of x and A through a ring in shared memory
// (cp.async, three in flight; straight to registers the loads of a step waited for the products before
// it: 8192 rows of 4096, rank 64, 42 us).  Two warps by two: 32 rows and 32 of the 64 k each.  The four
// 16-byte pieces of a lane group lie in the halves of a 128-byte row by turns, so eight lanes meet no bank twice.
template <bool F16, int NT>
__global__ void __launch_bounds__(kLoraThreads) lora_down_ring_kernel(const LoraParams p) {
    constexpr int kRows = 64, kCols = 8 * NT, kStage = (kRows + kCols) * 128;
    extern __shared__ __align__(128) uint8_t sm_ring[];
    __shared__ ItemRows<kRows> item;
    pdl_wait_previous();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
    const int split = blockIdx.y, col0 = blockIdx.z * kCols;
    int adapter, rows;
    if (!item.find(p, blockIdx.x, &adapter, &rows) || adapter < 0) return;
    const int k_begin = split * p.k_split, k_end = min(k_begin + p.k_split, (int)p.K);
    const uint32_t ring = smem_u32(sm_ring);
    // A thread copies piece tid % 8 of rows tid / 8, + 16 and so on; zeros behind the rows, columns and K.
    const int piece = tid & 7, row0 = tid >> 3;
    const uint32_t to = ring + row0 * 128 + (piece ^ (row0 & 1) * 4) * 16;
    const uint16_t *from_x[4], *from_a[(kCols + 15) / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) from_x[i] = p.x + (row0 + i * 16 < rows ? item.row[row0 + i * 16] : 0) * p.x_stride + piece * 8;
#pragma unroll
    for (int i = 0; i < (kCols + 15) / 16; ++i) {
        const int c = col0 + row0 + i * 16;
        from_a[i] = p.a + ((int64_t)adapter * p.r + (c < p.r ? c : 0)) * p.K + piece * 8;
    }
    const auto copy = [&](uint32_t dst, const uint16_t* src, bool held) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(held ? 16 : 0) : "memory");
    };
    const auto stage = [&](int k0, int s) {
        if (k0 < k_end) {
            const bool in = k0 + piece * 8 < k_end;
            const int k = in ? k0 : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) copy(to + s * kStage + i * 16 * 128, from_x[i] + k, in && row0 + i * 16 < rows);
#pragma unroll
            for (int i = 0; i < (kCols + 15) / 16; ++i)
                if (row0 + i * 16 < kCols) copy(to + s * kStage + (kRows + i * 16) * 128, from_a[i] + k, in && col0 + row0 + i * 16 < p.r);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const int row_warp = warp & 1, k_warp = warp >> 1;
    float acc[2][NT][4] = {};
#pragma unroll
    for (int s = 0; s < kRingStages - 1; ++s) stage(k_begin + s * 64, s);
    int s = 0;
    for (int k0 = k_begin; k0 < k_end; k0 += 64) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kRingStages - 2) : "memory");
        __syncthreads();                                    // this stage is there, and the last one is read
        stage(k0 + (kRingStages - 1) * 64, (s + kRingStages - 1) % kRingStages);
        const uint8_t* at = sm_ring + s * kStage + ((k_warp * 4 + q) ^ (g & 1) * 4) * 16 + g * 128;
        uint4 xv[2][2];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) xv[m][h] = *(const uint4*)(at + ((row_warp * 2 + m) * 16 + h * 8) * 128);
        uint4 av[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) av[j] = *(const uint4*)(at + (kRows + j * 8) * 128);
        // Both products of a sum are far apart: one waits for the other.
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const uint32_t lo[4] = {xv[m][0].x, xv[m][1].x, xv[m][0].y, xv[m][1].y};
#pragma unroll
            for (int j = 0; j < NT; ++j) mma_16816<F16>(acc[m][j], lo, av[j].x, av[j].y);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const uint32_t hi[4] = {xv[m][0].z, xv[m][1].z, xv[m][0].w, xv[m][1].w};
#pragma unroll
            for (int j = 0; j < NT; ++j) mma_16816<F16>(acc[m][j], hi, av[j].z, av[j].w);
        }
        s = (s + 1) % kRingStages;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    float* sums = (float*)sm_ring;                          // [2][kRows][kCols + 4]
    constexpr int kPitch = kCols + 4;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                *(float2*)&sums[(k_warp * kRows + (row_warp * 2 + m) * 16 + h * 8 + g) * kPitch + j * 8 + q * 2] = make_float2(acc[m][j][2 * h], acc[m][j][2 * h + 1]);
    __syncthreads();
    for (int i = tid; i < kRows * kCols / 4; i += kLoraThreads) {
        const int row = i / (kCols / 4), c = i % (kCols / 4) * 4;
        if (row >= rows || col0 + c >= p.rp) continue;
        const float4 u = *(const float4*)&sums[row * kPitch + c], v = *(const float4*)&sums[(kRows + row) * kPitch + c];
        *(float4*)(p.low + ((int64_t)split * p.T + item.row[row]) * p.rp + col0 + c) = make_float4(u.x + v.x, u.y + v.y, u.z + v.z, u.w + v.w);
    }
}

// 2 * KP elements of a row of B, zero from `left` on; VEC: all or none, on boundaries of as many.
template <int KP, bool VEC>
__device__ __forceinline__ void part(const uint16_t* p, int left, uint32_t (&w)[KP]) {
    if (VEC && KP == 4) {
        const uint4 v = left > 0 ? *(const uint4*)p : make_uint4(0, 0, 0, 0);
        w[0] = v.x; w[1] = v.y; w[KP - 2] = v.z; w[KP - 1] = v.w;
    } else if (VEC) {
        const uint2 v = left > 0 ? *(const uint2*)p : make_uint2(0, 0);
        w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < KP; ++i) w[i] = 0;
#pragma unroll
        for (int i = 0; i < 2 * KP; ++i)
            if (i < left) w[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
    }
}

// s A x of an item's rows, the splits' sums in order, as two 16-bit halves in shared memory: four rows a warp at
// a time, eight lanes each.  FP16 holds them divided by a power of two (`sm_up`) that puts a row's largest
// into [2^14, 2^15), the top of its range: the halves' last bit is then 2^-24 of an absolute 1, so what is 2^17 times
// smaller than the largest still has 22 bits, and B may be zero at the large ones (with the largest in [1, 2) a value 2^14
// times smaller was off by 2^-11).  The products are added to y over that power, and the end takes it back.  BF16 needs none.
template <bool F16>
__device__ __forceinline__ void sum_splits(const LoraParams& p, const int32_t* order, int adapter, int rows, int all, int pitch, uint32_t* sm_hi,
                                           uint32_t* sm_lo, float* sm_up) {
    const float s = p.scales ? p.scales[adapter] : 1.f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int row = warp * 4 + (lane >> 3); row < all; row += kLoraThreads / 8) {
        const bool held = row < rows;
        const float* low = p.low + (int64_t)(held ? order[row] : 0) * p.rp;
        const int64_t apart = p.T * p.rp;
        const auto sum = [&](int c) {                   // of four; behind r zeros, where x or s is infinite, too
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (held && c < p.r) {
                const float* at = low + c;
#pragma unroll 4
                for (int sp = 0; sp < p.splits; ++sp, at += apart) {
                    const float4 u = *(const float4*)at;
                    v.x += u.x;
                    v.y += u.y;
                    v.z += u.z;
                    v.w += u.w;
                }
                v.x *= s;
                v.y = c + 1 < p.r ? v.y * s : 0.f;
                v.z = c + 2 < p.r ? v.z * s : 0.f;
                v.w = c + 3 < p.r ? v.w * s : 0.f;
            }
            return v;
        };
        float down = 1.f, up = 1.f;
        if (F16) {
            float most = 0.f;                               // of what is finite
            const auto meet = [&](float x) { most = fmaxf(most, fabsf(x) < INFINITY ? fabsf(x) : 0.f); };
            for (int c = (lane & 7) * 4; c < p.rp; c += 32) {
                const float4 v = sum(c);
                meet(v.x);
                meet(v.y);
                meet(v.z);
                meet(v.w);
            }
            __syncwarp();
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
            // From 2^-60 on (less is nothing beside 2^-25, the half of FP16's smallest): either power is a normal number.
            const uint32_t e = max(__float_as_uint(most) & 0x7f800000u, (127u - 60u) << 23) - (14u << 23);
            up = __uint_as_float(e);
            down = __uint_as_float(0x7f000000u - e);                // 1 / up
        }
        if (F16 && (lane & 7) == 0) sm_up[row] = up;
        const auto halves = [&](float a, float b, uint32_t* hi, uint32_t* lo) {
            *hi = f32_to_act2<F16>(a, b);
            const float2 back = act2_to_f32<F16>(*hi);
            // An infinity (or one that the type cannot hold) is its own first half.
            *lo = f32_to_act2<F16>(fabsf(back.x) < INFINITY ? a - back.x : 0.f, fabsf(back.y) < INFINITY ? b - back.y : 0.f);
        };
        for (int c = (lane & 7) * 4; c < p.rp; c += 32) {
            const float4 v = sum(c);
            uint2 hi, lo;
            halves(v.x * down, v.y * down, &hi.x, &lo.x);
            halves(v.z * down, v.w * down, &hi.y, &lo.y);
            *(uint2*)(sm_hi + row * pitch + c / 2) = hi;
            *(uint2*)(sm_lo + row * pitch + c / 2) = lo;
        }
    }
}

constexpr int kUpStages = 3;
constexpr int kUpRingRank = 128;           // where a row of B is a multiple of 128 bytes it is 128 or 256 (`turn`)
constexpr int kFewBlocks = 5;              // of the up kernel of 16 rows, on an SM

// One item's rows of A x times B, and y, over a range of N: stages of columns of B and y through a ring in
// shared memory (with loads to registers a step ahead, 8192 rows, 4096 columns, rank 64: 75 us for the
// 43 here; 64 rows, 28672 columns, rank 16: 20.9 for the 16.5
// here, with the down kernel).  RW warps by 4 / RW: MT * 16 rows
// and 32 columns each; items of 64 rows are two by two warps of 32, of 16 rows one by four.  Tile j of
// four holds columns 8 (c / 2) + 2 j + c % 2, so that a lane's eight outputs of a row lie side by side: the
// 16 bytes of y that it copies itself.  KS: 16s of the rank, or 8 for any number of them.  EXACT: it is
// a multiple of a step's k.
template <bool F16, int RW, int MT, int KS, bool EXACT>
__global__ void __launch_bounds__(kLoraThreads, RW == 2 ? 3 : kFewBlocks) lora_up_ring_kernel(const LoraParams p, const int cols_block) {
    constexpr int kRows = 16 * MT * RW, kStep = 32 * (kLoraThreads / 32 / RW), kYBytes = kLoraThreads * MT * 2 * 16;
    constexpr int KP = KS == 1 ? 2 : 4;
    constexpr bool kHeld = KS <= 4;
    extern __shared__ __align__(128) uint8_t sm_up[];
    __shared__ ItemRows<kRows> item;
    __shared__ float sm_power[kRows];
    const int pitch = p.rp / 2 + 4;                         // words of two values
    const int b_bytes = kStep * p.r * 2;
    uint8_t* sm_y = sm_up;                                  // [kUpStages][2 * MT][kLoraThreads] pieces of 16 bytes
    uint8_t* sm_b = sm_y + kUpStages * kYBytes;             // [kUpStages][kStep][r]
    uint32_t* sm_hi = (uint32_t*)(sm_b + kUpStages * b_bytes);      // [kRows][pitch] halves of A x
    uint32_t* sm_lo = sm_hi + kRows * pitch;
    if (p.n == 0) pdl_wait_previous();                      // else the down kernel has, for all but its own sums
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
    int adapter, rows;
    if (!item.find(p, blockIdx.x, &adapter, &rows) || (adapter < 0 && !p.copy_rest)) {
        if (blockIdx.x == 0 && blockIdx.y == 0) pdl_wait_previous();        // the grid ends behind the down kernel, whatever its items
        return;
    }
    const int64_t n_begin = (int64_t)blockIdx.y * cols_block, n_end = min(n_begin + cols_block, p.N);
    const int steps = adapter < 0 ? 0 : p.rp / (8 * KP);
    const int row_warp = warp % RW, col_warp = warp / RW;
    bool held[MT][2];
    const uint16_t* y[MT][2];
    uint16_t* out[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = (row_warp * MT + m) * 16 + h * 8 + g;
            held[m][h] = row < rows;
            const int64_t t = held[m][h] ? item.row[row] : 0;
            y[m][h] = p.y + t * p.y_stride + col_warp * 32 + q * 8;
            out[m][h] = p.out + t * p.N + col_warp * 32 + q * 8;
        }
    const uint16_t* b = p.b + (int64_t)max(adapter, 0) * p.N * p.r;
    const uint32_t y0 = smem_u32(sm_y) + tid * 16, b0 = smem_u32(sm_b);
    // Rows of 128 and of 256 bytes: the four pieces of a lane group lie in the halves of 128 bytes by turns, which
    // go by the row's last bit (bit 3 or 4 of a piece's number).
    const int turn = p.r % 64 == 0 ? 4 : 0, row_bit = p.r == 128 ? 4 : 3, pieces = p.r / 8;
    const auto stage = [&](int64_t n0, int s) {
        const int64_t left = n_end - n0;
        if (left > 0) {
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i)
                if (held[i >> 1][i & 1] && left > col_warp * 32 + q * 8)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(y0 + s * kYBytes + i * kLoraThreads * 16),
                                 "l"(y[i >> 1][i & 1] + n0) : "memory");
            if (steps) {
                const int all = (int)min(left, (int64_t)kStep) * pieces;
                const uint16_t* from = b + n0 * p.r;
                for (int i = tid; i < all; i += kLoraThreads) {
                    const int to = i ^ (i >> row_bit & 1) * turn;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(b0 + s * b_bytes + to * 16), "l"(from + i * 8) : "memory");
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int s = 0; s < kUpStages - 1; ++s) stage(n_begin + s * kStep, s);
    pdl_wait_previous();
    pdl_launch_dependents();
    if (steps) sum_splits<F16>(p, item.row, adapter, rows, kRows, pitch, sm_hi, sm_lo, sm_power);
    __syncthreads();
    const uint32_t *hi0 = sm_hi + (row_warp * MT * 16 + g) * pitch + q * KP, *lo0 = sm_lo + (row_warp * MT * 16 + g) * pitch + q * KP;
    // Halves of A x of a lane's rows: words w and w + 1 of step st are the k of one product.
    const auto low_words = [&](const uint32_t* from, int m, int st, uint32_t (&w0)[KP], uint32_t (&w1)[KP]) {
        const int at = m * 16 * pitch + st * 4 * KP, at8 = at + 8 * pitch;
        if (KP == 4) {
            *(uint4*)w0 = *(const uint4*)(from + at);
            *(uint4*)w1 = *(const uint4*)(from + at8);
        } else {
            *(uint2*)w0 = *(const uint2*)(from + at);
            *(uint2*)w1 = *(const uint2*)(from + at8);
        }
    };
    // They are the same for all columns: up to rank 64 they stay in registers.
    constexpr int kHeldSteps = kHeld ? KS * 2 / KP : 1;
    uint32_t kept[2][MT][kHeldSteps][2][KP];                 // [half][m][step][row or row + 8]
    if (kHeld && steps)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int st = 0; st < kHeldSteps; ++st) {
                low_words(hi0, m, st, kept[0][m][st][0], kept[0][m][st][1]);
                low_words(lo0, m, st, kept[1][m][st][0], kept[1][m][st][1]);
            }
    float up[MT][2], down[MT][2];                             // FP16: of sum_splits, and its reciprocal
    if (F16)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                up[m][h] = steps ? sm_power[(row_warp * MT + m) * 16 + h * 8 + g] : 1.f;
                down[m][h] = __uint_as_float(0x7f000000u - __float_as_uint(up[m][h]));
            }
    const int first = col_warp * 32 + 8 * (g >> 1) + (g & 1), odd = (g & 1) * turn * 16;     // of a row's pieces: 64 bytes on, or back
    int s = 0;
    for (int64_t n0 = n_begin; n0 < n_end; n0 += kStep) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kUpStages - 2) : "memory");
        __syncthreads();                                    // this stage is there, and the last one is read
        stage(n0 + (kUpStages - 1) * kStep, (s + kUpStages - 1) % kUpStages);
        const uint8_t* bs = sm_b + s * b_bytes + first * p.r * 2;
        // The products are added to y.
        float acc[MT][4][4];
        uint4 yv[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                yv[m][h] = make_uint4(0, 0, 0, 0);
                if (MT > 1 || h * 8 < rows)                 // of few rows the second eight are often not there
                    yv[m][h] = *(const uint4*)(sm_y + s * kYBytes + ((m * 2 + h) * kLoraThreads + tid) * 16);
                const uint32_t w[4] = {yv[m][h].x, yv[m][h].y, yv[m][h].z, yv[m][h].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 u = act2_to_f32<F16>(w[j]);
                    acc[m][j][2 * h] = F16 ? u.x * down[m][h] : u.x;
                    acc[m][j][2 * h + 1] = F16 ? u.y * down[m][h] : u.y;
                }
            }
        const auto products = [&](int st, const auto& words) {
            const bool in = EXACT || st * 8 * KP + q * 2 * KP < p.r;
            const int at_b = (st * 8 * KP + q * 2 * KP) * 2 ^ odd;
            uint32_t bv[4][KP];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (KP == 4) *(uint4*)bv[j] = in ? *(const uint4*)(bs + 2 * j * p.r * 2 + at_b) : make_uint4(0, 0, 0, 0);
                else *(uint2*)bv[j] = in ? *(const uint2*)(bs + 2 * j * p.r * 2 + at_b) : make_uint2(0, 0);
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                uint32_t w0[MT][KP], w1[MT][KP];
#pragma unroll
                for (int m = 0; m < MT; ++m) words(half, m, w0[m], w1[m]);
                // Products of one sum as far apart as they go: one waits for the other.
#pragma unroll
                for (int k = 0; k < KP; k += 2)
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const uint32_t a[4] = {w0[m][k], w1[m][k], w0[m][k + 1], w1[m][k + 1]};
#pragma unroll
                        for (int j = 0; j < 4; ++j) mma_16816<F16>(acc[m][j], a, bv[j][k], bv[j][k + 1]);
                    }
            }
        };
        if (kHeld) {
            if (steps)
#pragma unroll
                for (int st = 0; st < kHeldSteps; ++st)
                    products(st, [&](int half, int m, uint32_t (&w0)[KP], uint32_t (&w1)[KP]) {
#pragma unroll
                        for (int k = 0; k < KP; ++k) {
                            w0[k] = kept[half][m][st][0][k];
                            w1[k] = kept[half][m][st][1][k];
                        }
                    });
        } else {
            for (int st = 0; st < steps; ++st)
                products(st, [&](int half, int m, uint32_t (&w0)[KP], uint32_t (&w1)[KP]) { low_words(half ? lo0 : hi0, m, st, w0, w1); });
        }
        if (n_end - n0 > col_warp * 32 + q * 8)
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) {
                const int m = i >> 1, h = i & 1;
                if (!held[m][h]) continue;
                uint32_t w[4] = {yv[m][h].x, yv[m][h].y, yv[m][h].z, yv[m][h].w};      // without an adapter: as it is
                if (steps)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        w[j] = F16 ? f32_to_act2<F16>(acc[m][j][2 * h] * up[m][h], acc[m][j][2 * h + 1] * up[m][h])
                                   : f32_to_act2<F16>(acc[m][j][2 * h], acc[m][j][2 * h + 1]);
                *(uint4*)(out[m][h] + n0) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        s = (s + 1) % kUpStages;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// One item's rows of A x times B, and y, over a range of N.  A warp takes MT * 16 rows and 32 columns
// of a step, whose y it asks for first; tile j of four holds columns 8 (c / 2) + 2 j + c % 2, so that a
// lane's eight outputs of a row lie side by side.  A lane takes KP words of a row of B: four k for
// each 16, or (KP = 4) eight for each 32.  The first step's y and B are asked for while the down kernel
// still runs, each further one's a step ahead (64 rows of 4096 and 28672 columns,
// rank 16: 22.8 us without, 20.9 with, for both kernels).  For what the ring does not take: rows of B or y
// off 16-byte boundaries, ranks that are no multiple of 8 or beyond its room.
template <bool F16, int RW, int MT, int KP, bool VEC_B, bool VEC_Y>
__global__ void __launch_bounds__(kLoraThreads, MT == 1 ? kFewBlocks : 1) lora_up_kernel(const LoraParams p, const int cols_block) {
    constexpr int kRows = 16 * MT * RW, kColWarps = kLoraThreads / 32 / RW;
    extern __shared__ __align__(16) uint8_t sm_up[];
    __shared__ ItemRows<kRows> item;
    __shared__ float sm_power[kRows];
    const int pitch = p.rp / 2 + 4;                         // words of two values
    uint32_t* sm_hi = (uint32_t*)sm_up;                     // [kRows][pitch] halves of A x
    uint32_t* sm_lo = sm_hi + kRows * pitch;
    if (p.n == 0) pdl_wait_previous();                      // else the down kernel has, for all but its own sums
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    int adapter, rows;
    if (!item.find(p, blockIdx.x, &adapter, &rows) || (adapter < 0 && !p.copy_rest)) {
        if (blockIdx.x == 0 && blockIdx.y == 0) pdl_wait_previous();        // the grid ends behind the down kernel, whatever its items
        return;
    }
    const int64_t n_begin = (int64_t)blockIdx.y * cols_block, n_end = min(n_begin + cols_block, p.N);
    const int steps = adapter < 0 ? 0 : p.rp / (8 * KP);
    const int row_warp = warp % RW, col_warp = warp / RW;
    bool held[MT][2];
    const uint16_t* y[MT][2];
    uint16_t* out[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = (row_warp * MT + m) * 16 + h * 8 + g;
            held[m][h] = row < rows;
            const int64_t t = held[m][h] ? item.row[row] : 0;
            y[m][h] = p.y + t * p.y_stride + q * 8;
            out[m][h] = p.out + t * p.N + q * 8;
        }
    const uint16_t* b = p.b + (int64_t)max(adapter, 0) * p.N * p.r + q * 2 * KP;
    const uint32_t *hi0 = sm_hi + (row_warp * MT * 16 + g) * pitch + q * KP, *lo0 = sm_lo + (row_warp * MT * 16 + g) * pitch + q * KP;
    const int r = p.r, first = 8 * (g >> 1) + (g & 1);
    // y of the step at n0.  `whole`: all of its columns are there.
    const auto ask = [&](int64_t n0, bool whole, uint4 (&v)[MT][2]) {
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                v[m][h] = make_uint4(0, 0, 0, 0);
                if (held[m][h]) v[m][h] = eight<VEC_Y>(y[m][h] + n0, whole ? 8 : n_end - n0 - q * 8);
            }
    };
    // B of the step at n0, its k from `st` on.
    const auto ask_b = [&](int64_t n0, bool whole, int st, uint32_t (&v)[4][KP]) {
        const uint16_t* bn = b + (n0 + first) * r + st * 8 * KP;
        const int left = r - st * 8 * KP - q * 2 * KP;
        if (whole) {
#pragma unroll
            for (int j = 0; j < 4; ++j) part<KP, VEC_B>(bn + 2 * j * r, left, v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) part<KP, VEC_B>(bn + 2 * j * r, n0 + first + 2 * j < n_end ? left : 0, v[j]);
        }
    };
    constexpr int kStep = 32;
    uint4 next[MT][2];
    uint32_t b_next[4][KP];                             // a step's first k, asked for with its y
    int64_t n0 = n_begin + col_warp * kStep;
    if (n0 < n_end) {
        ask(n0, n0 + kStep <= n_end, next);
        if (steps) ask_b(n0, n0 + kStep <= n_end, 0, b_next);
    }
    pdl_wait_previous();
    pdl_launch_dependents();
    if (steps) sum_splits<F16>(p, item.row, adapter, rows, kRows, pitch, sm_hi, sm_lo, sm_power);
    __syncthreads();
    float up[MT][2], down[MT][2];                           // FP16: of sum_splits, and its reciprocal
    if (F16)
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                up[m][h] = steps ? sm_power[(row_warp * MT + m) * 16 + h * 8 + g] : 1.f;
                down[m][h] = __uint_as_float(0x7f000000u - __float_as_uint(up[m][h]));
            }
    for (; n0 < n_end; n0 += kColWarps * kStep) {
        const bool whole = n0 + kStep <= n_end;
        uint4 now[MT][2];
        uint32_t bv[4][KP];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) now[m][h] = next[m][h];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < KP; ++k) bv[j][k] = b_next[j][k];
        const int64_t n1 = n0 + kColWarps * kStep;
        if (n1 < n_end) {
            ask(n1, n1 + kStep <= n_end, next);
            if (steps) ask_b(n1, n1 + kStep <= n_end, 0, b_next);
        }
        float acc[MT][4][4];                                // the products are added to y
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t w[4] = {now[m][h].x, now[m][h].y, now[m][h].z, now[m][h].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 v = act2_to_f32<F16>(w[j]);
                    acc[m][j][2 * h] = F16 ? v.x * down[m][h] : v.x;
                    acc[m][j][2 * h + 1] = F16 ? v.y * down[m][h] : v.y;
                }
            }
        for (int st = 0; st < steps; ++st) {
            if (st) ask_b(n0, whole, st, bv);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int at = m * 16 * pitch + st * 4 * KP, at8 = at + 8 * pitch;
                uint32_t h0[KP], h1[KP], l0[KP], l1[KP];
                if (KP == 4) {
                    *(uint4*)h0 = *(const uint4*)(hi0 + at); *(uint4*)h1 = *(const uint4*)(hi0 + at8);
                    *(uint4*)l0 = *(const uint4*)(lo0 + at); *(uint4*)l1 = *(const uint4*)(lo0 + at8);
                } else {
                    *(uint2*)h0 = *(const uint2*)(hi0 + at); *(uint2*)h1 = *(const uint2*)(hi0 + at8);
                    *(uint2*)l0 = *(const uint2*)(lo0 + at); *(uint2*)l1 = *(const uint2*)(lo0 + at8);
                }
#pragma unroll
                for (int k = 0; k < KP; k += 2) {
                    const uint32_t hi[4] = {h0[k], h1[k], h0[k + 1], h1[k + 1]}, lo[4] = {l0[k], l1[k], l0[k + 1], l1[k + 1]};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        mma_16816<F16>(acc[m][j], hi, bv[j][k], bv[j][k + 1]);
                        mma_16816<F16>(acc[m][j], lo, bv[j][k], bv[j][k + 1]);
                    }
                }
            }
        }
        const int64_t left = n_end - n0 - q * 8;
        if (left <= 0) continue;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!held[m][h]) continue;
                uint32_t w[4] = {now[m][h].x, now[m][h].y, now[m][h].z, now[m][h].w};
                if (steps)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        w[j] = F16 ? f32_to_act2<F16>(acc[m][j][2 * h] * up[m][h], acc[m][j][2 * h + 1] * up[m][h])
                                   : f32_to_act2<F16>(acc[m][j][2 * h], acc[m][j][2 * h + 1]);
                uint16_t* to = out[m][h] + n0;
                if (VEC_Y) {
                    *(uint4*)to = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i < left) to[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
                }
            }
    }
}

// The rank that A x is held with: whole steps of the products, zeros behind r.
int64_t padded_rank(int64_t r) { return r <= 16 ? 16 : r <= 32 ? 32 : r <= 64 ? 64 : round_up(r, 32); }

// How a call of these sizes is cut up.
struct LoraPlan {
    int rows_item, splits, k_split, nt;
    bool listed;                           // items from the grouping kernel
    int64_t items;                         // at most
    size_t bytes, order_at, low_at;
};

LoraPlan plan_lora(int64_t T, int64_t n, int64_t r, int64_t K) {
    LoraPlan pl{};
    pl.rows_item = T >= 64 * (n + 1) ? 64 : 16;
    pl.listed = T > kSelfRows;
    pl.items = std::min(T, T / pl.rows_item + n + 1);
    pl.nt = r <= 8 ? 1 : r <= 16 ? 2 : r <= 32 ? 4 : 8;
    const int64_t blocks = pl.items * ceil_div(r, pl.nt * 8);
    int64_t splits = std::max<int64_t>(1, 3 * (int64_t)sm_count() / blocks);
    splits = std::min<int64_t>({splits, kMaxSplits, ceil_div(K, 256)});
    pl.k_split = (int)round_up(ceil_div(K, std::max<int64_t>(splits, 1)), 32);
    pl.splits = (int)ceil_div(K, pl.k_split);
    pl.order_at = 256 + (pl.listed ? (size_t)round_up(sizeof(Item) * pl.items, 256) : 0);
    pl.low_at = pl.order_at + (pl.listed ? (size_t)round_up(4 * T, 256) : 0);
    pl.bytes = pl.low_at + (size_t)round_up(4 * pl.splits * T * padded_rank(r), 256);
    return pl;
}

template <bool F16, int RW, int MT, bool VEC>
const void* down_kernel(int nt) {
    return nt == 1   ? (const void*)lora_down_kernel<F16, RW, MT, 1, VEC>
           : nt == 2 ? (const void*)lora_down_kernel<F16, RW, MT, 2, VEC>
           : nt == 4 ? (const void*)lora_down_kernel<F16, RW, MT, 4, VEC>
                     : (const void*)lora_down_kernel<F16, RW, MT, 8, VEC>;
}

template <bool F16>
const void* down_kernel(int rows, int nt, bool vec) {
    if (rows == 16) return vec ? down_kernel<F16, 1, 1, true>(nt) : down_kernel<F16, 1, 1, false>(nt);
    return down_kernel<F16, 2, 2, false>(nt);               // with vector loads: ring_kernel
}

template <bool F16>
const void* ring_kernel(int nt) {
    return nt == 1   ? (const void*)lora_down_ring_kernel<F16, 1>
           : nt == 2 ? (const void*)lora_down_ring_kernel<F16, 2>
           : nt == 4 ? (const void*)lora_down_ring_kernel<F16, 4>
                     : (const void*)lora_down_ring_kernel<F16, 8>;
}

// wide: B in 16-byte pieces of eight k.  (Without vector loads there is one form of each.)
template <bool F16, int RW, int MT>
const void* up_kernel(bool wide, bool vec_b, bool vec_y) {
    if (!vec_b) return vec_y ? (const void*)lora_up_kernel<F16, RW, MT, 2, false, true> : (const void*)lora_up_kernel<F16, RW, MT, 2, false, false>;
    if (wide) return vec_y ? (const void*)lora_up_kernel<F16, RW, MT, 4, true, true> : (const void*)lora_up_kernel<F16, RW, MT, 4, true, false>;
    return vec_y ? (const void*)lora_up_kernel<F16, RW, MT, 2, true, true> : (const void*)lora_up_kernel<F16, RW, MT, 2, true, false>;
}

template <bool F16, int RW, int KS>
const void* up_ring_kernel_of(bool exact) {
    return exact ? (const void*)lora_up_ring_kernel<F16, RW, RW, KS, true> : (const void*)lora_up_ring_kernel<F16, RW, RW, KS, false>;
}
template <bool F16, int RW>
const void* up_ring_kernel(int64_t r) {
    if (r <= 16) return up_ring_kernel_of<F16, RW, 1>(r == 16);
    if (r <= 32) return up_ring_kernel_of<F16, RW, 2>(r == 32);
    if (r <= 64) return up_ring_kernel_of<F16, RW, 4>(r == 64);
    return up_ring_kernel_of<F16, RW, 8>(r % 32 == 0);
}

nvfp4_status check_sizes(const char* fn, int64_t T, int64_t n, int64_t r, int64_t K, int64_t N) {
    if (T < 0 || N < 0 || n < 0) return fail(NVFP4_ERR_INVALID_ARG, "%s: negative size T=%lld N=%lld adapters=%lld", fn, (long long)T, (long long)N, (long long)n);
    if (r < 1 || r > kMaxRank) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: rank %lld must be in [1, %d]", fn, (long long)r, kMaxRank);
    if (n > kMaxAdapters) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: %lld adapters, at most %d", fn, (long long)n, kMaxAdapters);
    if (K < 1 || K > (1 << 24) || N > (1 << 24) || T > (1 << 24))
        return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: T=%lld, K=%lld and N=%lld must be at most 2^24, K positive", fn, (long long)T, (long long)K, (long long)N);
    return NVFP4_OK;
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" size_t nvfp4_lora_workspace(int64_t T, int64_t adapters, int64_t r, int64_t K) {
    if (check_sizes("nvfp4_lora_workspace", T, adapters, r, K, 0) != NVFP4_OK || T == 0) return 0;
    return plan_lora(T, adapters, r, K).bytes;
}

extern "C" nvfp4_status nvfp4_lora_add(const void* y, int64_t y_stride, const void* x, int64_t x_stride, const void* A, const void* B,
                                       const float* scales, const int32_t* adapters, int64_t T, int64_t num_adapters, int64_t r, int64_t K,
                                       int64_t N, int f16, void* out, void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "nvfp4_lora_add";
    if (nvfp4_status st = check_sizes(fn, T, num_adapters, r, K, N)) return st;
    if (f16 != 0 && f16 != 1) return fail(NVFP4_ERR_INVALID_ARG, "%s: f16=%d must be 0 or 1", fn, f16);
    if (x_stride < 0 || y_stride < 0) return fail(NVFP4_ERR_INVALID_ARG, "%s: negative stride", fn);
    if (T == 0 || N == 0) return NVFP4_OK;
    if (!y || !x || !adapters || !out || (num_adapters > 0 && (!A || !B))) return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(y, 2) || !aligned(x, 2) || !aligned(A, 2) || !aligned(B, 2) || !aligned(out, 2) || !aligned(adapters, 4) || !aligned(scales, 4))
        return fail(NVFP4_ERR_ALIGNMENT, "%s: pointers must be aligned to their elements", fn);
    const LoraPlan pl = plan_lora(T, num_adapters, r, K);
    if (!workspace || workspace_bytes < pl.bytes) return fail(NVFP4_ERR_WORKSPACE, "%s: workspace %zu bytes, needs %zu", fn, workspace ? workspace_bytes : 0, pl.bytes);
    if (!aligned(workspace, 256)) return fail(NVFP4_ERR_ALIGNMENT, "%s: workspace must be 256-byte aligned", fn);
    const Span to = dense_span("out", out, 2 * T * N), ws = dense_span("workspace", workspace, (int64_t)pl.bytes);
    const Span ys = strided_span("y", y, 2 * N, {{T, 2 * y_stride}}), xs = strided_span("x", x, 2 * K, {{T, 2 * x_stride}});
    const Span as = dense_span("a", A, 2 * num_adapters * r * K), bs = dense_span("b", B, 2 * num_adapters * N * r);
    const Span ids = dense_span("adapters", adapters, 4 * T), ss = dense_span("scales", scales, 4 * num_adapters);
    if (overlaps(to, ys) && !same_place(to, ys)) return fail(NVFP4_ERR_INVALID_ARG, "%s: out overlaps y (it may be y itself where that is dense)", fn);
    if (const char* s = met(to, {xs, as, bs, ids, ss, ws})) return fail(NVFP4_ERR_INVALID_ARG, "%s: out overlaps %s", fn, s);
    if (const char* s = met(ws, {ys, xs, as, bs, ids, ss})) return fail(NVFP4_ERR_INVALID_ARG, "%s: workspace overlaps %s", fn, s);
    LoraParams p{};
    p.status = device_status_ptr();
    if (!p.status) return fail(NVFP4_ERR_CUDA, "%s: no CUDA device", fn);
    uint8_t* w = (uint8_t*)workspace;
    p.x = (const uint16_t*)x; p.a = (const uint16_t*)A; p.b = (const uint16_t*)B; p.y = (const uint16_t*)y;
    p.adapters = adapters; p.scales = scales; p.out = (uint16_t*)out;
    p.T = T; p.K = K; p.N = N; p.x_stride = x_stride; p.y_stride = y_stride;
    p.n = (int)num_adapters; p.r = (int)r; p.rp = (int)padded_rank(r);
    p.splits = pl.splits; p.k_split = pl.k_split; p.rows_item = pl.rows_item; p.copy_rest = out != y;
    p.num_items = (int32_t*)w; p.items = (Item*)(w + 256); p.order = (int32_t*)(w + pl.order_at); p.low = (float*)(w + pl.low_at);
    cudaStream_t s = (cudaStream_t)stream;
    void* args[] = {&p};
    if (pl.listed) {
        if (nvfp4_status st = launch_kernel((const void*)lora_group_kernel, dim3(1), dim3(1024), 8 * (p.n + 1), 1, args, s, fn)) return st;
    } else {
        p.num_items = nullptr;
    }
    const bool vec_x = K % 8 == 0 && x_stride % 8 == 0 && aligned(x, 16) && aligned(A, 16);
    const bool vec_b = r % 4 == 0 && aligned(B, 8), wide = p.rp % 32 == 0 && r % 8 == 0 && aligned(B, 16);
    const bool vec_y = N % 8 == 0 && y_stride % 8 == 0 && aligned(y, 16) && aligned(out, 16);
    if (num_adapters > 0) {
        const bool ring = vec_x && pl.rows_item == 64;
        const void* kernel = ring ? (f16 ? ring_kernel<true>(pl.nt) : ring_kernel<false>(pl.nt))
                                  : (f16 ? down_kernel<true>(pl.rows_item, pl.nt, vec_x) : down_kernel<false>(pl.rows_item, pl.nt, vec_x));
        const dim3 grid((unsigned)pl.items, (unsigned)pl.splits, (unsigned)ceil_div(r, pl.nt * 8));
        const size_t smem = ring ? kRingStages * (64 + 8 * pl.nt) * 128 : 0;
        if (nvfp4_status st = launch_kernel(kernel, grid, dim3(kLoraThreads), smem, 1, args, s, fn)) return st;
    }
    // Stages of 64 or 128 columns of B and y: as far as two blocks an SM have room for them (rank 256: 147 KB
    // for 64 rows).
    const int step = pl.rows_item == 16 ? 128 : 64;
    const size_t halves = (size_t)pl.rows_item * (p.rp / 2 + 4) * 8, stage = (size_t)kLoraThreads * (pl.rows_item == 16 ? 32 : 64) + (size_t)step * 2 * r;
    const bool up_ring = vec_y && vec_b && r % 8 == 0 && r <= kUpRingRank && aligned(B, 16) && halves + kUpStages * stage <= 110 * 1024;
    const void* kernel;
    if (up_ring) {
        kernel = pl.rows_item == 16 ? (f16 ? up_ring_kernel<true, 1>(r) : up_ring_kernel<false, 1>(r))
                                    : (f16 ? up_ring_kernel<true, 2>(r) : up_ring_kernel<false, 2>(r));
    } else {
        kernel = pl.rows_item == 16 ? (f16 ? up_kernel<true, 1, 1>(wide, vec_b, vec_y) : up_kernel<false, 1, 1>(wide, vec_b, vec_y))
                                    : (f16 ? up_kernel<true, 2, 2>(wide, vec_b, vec_y) : up_kernel<false, 2, 2>(wide, vec_b, vec_y));
    }
    // Columns of a block: as many steps of its warps as leave one wave of blocks, so that an item's sums over
    // the splits are not read more often than that needs.  Of 64 rows three an SM fit by their registers, two
    // by the shared memory of ranks beyond 64 (4096 x 4096 x 4096, rank 128: 76 us, with three counted 94; rank 80 67 and 79;
    // 2048 x 5120 x 5120, rank 96, 53.4 and 52.8).  Of few rows nine for each item that there may be, of which fewer are (six / nine /
    // twelve: 64 x 4096 x 28672, rank 16, 32 adapters 17.5 / 15.9 / 18.2 us, 16 x 4096 x 28672 8.4 / 7.7 / 9.8, 300 x 4096 x
    // 4096 12.0 / 12.1 / 13.5, 64 x 4096 x 4096 8.5 / 9.4 / 9.4, 1000 x 4096 x 8192, rank 32, 33.7 / 35.1 / 34.7).
    const size_t smem = halves + (up_ring ? kUpStages * stage : 0);
    const int64_t fit = std::min<int64_t>(3, (227 * 1024) / (int64_t)(smem + 2 * 1024));       // with what is static, and reserved
    const int64_t waves = (pl.rows_item == 16 ? 9 : fit) * sm_count();
    const int64_t blocks = std::min<int64_t>(std::max<int64_t>(1, waves / pl.items), 65535);        // of an item
    int cols_block = (int)round_up(ceil_div(N, blocks), step);
    const int64_t cols = cols_block;
    void* up_args[] = {&p, &cols_block};
    return launch_kernel(kernel, dim3((unsigned)pl.items, (unsigned)ceil_div(N, cols)), dim3(kLoraThreads), smem, 1, up_args, s, fn);
}
