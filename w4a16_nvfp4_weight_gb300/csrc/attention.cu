// Attention of one new token per sequence over a paged key-value cache.
//
// For query head h of sequence b, with n = lengths[b] cached tokens:
//     z_j = softmax_scale * q . k_j   for max(0, n - window) <= j < n,
//     out = sum_j exp(z_j - lse) v_j,   lse = log sum_j exp(z_j),
// in one pass over the cache with the running maximum and sum of the softmax
// in 32 bits.  A row with no token gives out = 0 and lse = -infinity.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kv_cache.cuh"
#include "numeric.cuh"
#include "ptx.cuh"

namespace nvfp4 {
namespace {

struct AttnParams {
    const uint16_t* q;             // strides q_row, q_head (elements)
    int64_t q_row, q_head;
    const int32_t* block_table;    // [B, width], row stride table_stride
    int64_t table_stride;
    const int32_t* lengths;
    uint16_t* out;                 // [B, Hq, D]
    float* lse;                    // [B, Hq] or null
    int B, Hq, G, width;           // G query heads a key head
    int window;                    // 0: none
    float scale_log2;              // softmax_scale * log2(e)
    int* status;
    CacheView cache;
};

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

constexpr int kDims = kMaxHeadDim / 32;

// A block takes one query head of one sequence; its warps take every fourth
// token, a lane every 32nd dimension.
template <bool F16>
__global__ void __launch_bounds__(128) attend_any_kernel(AttnParams p) {
    __shared__ float sm_m[4], sm_l[4], sm_o[4][kMaxHeadDim];
    const int b = blockIdx.y, hq = blockIdx.x, h = hq / p.G;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, D = p.cache.D;
    const int n = checked_length(p, b);
    const int first = p.window > 0 ? max(0, n - p.window) : 0;
    float q[kDims], o[kDims], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < kDims; ++i) {
        const int d = lane + 32 * i;
        q[i] = d < D ? act_to_f32<F16>(p.q[b * p.q_row + hq * p.q_head + d]) : 0.f;
        o[i] = 0.f;
    }
    for (int t = first + warp; t < n; t += 4) {
        int64_t page = p.block_table[b * p.table_stride + t / p.cache.page_size];
        if (page < 0 || page >= p.cache.num_pages) {
            if (lane == 0) record_status(p.status, NVFP4_ERR_BAD_INDEX);
            page = 0;
        }
        const int at = t % p.cache.page_size;
        const int64_t row = p.cache.row(page, h, at);
        const int64_t sc = p.cache.e4m3 ? p.cache.scale_at(page, h, at) : 0;
        const float ks = p.cache.e4m3 ? p.cache.k_scale[sc] : 1.f, vs = p.cache.e4m3 ? p.cache.v_scale[sc] : 1.f;
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < kDims; ++i) {
            const int d = lane + 32 * i;
            if (d >= D) continue;
            z += q[i] * (p.cache.e4m3 ? act2_to_f32<true>(e4m3x2_to_f16x2(p.cache.k[row + d])).x
                                      : act_to_f32<F16>(((const uint16_t*)(p.cache.k + row))[d]));
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
        z *= ks * p.scale_log2;
        const float m_new = fmaxf(m, z), base = m_new == -INFINITY ? 0.f : m_new;
        const float keep = exp2f(m - base), w = exp2f(z - base);
        l = l * keep + w;
        m = m_new;
#pragma unroll
        for (int i = 0; i < kDims; ++i) {
            const int d = lane + 32 * i;
            if (d >= D) continue;
            const float v = p.cache.e4m3 ? vs * act2_to_f32<true>(e4m3x2_to_f16x2(p.cache.v[row + d])).x
                                         : act_to_f32<F16>(((const uint16_t*)(p.cache.v + row))[d]);
            o[i] = o[i] * keep + w * v;
        }
    }
    if (lane == 0) { sm_m[warp] = m; sm_l[warp] = l; }
#pragma unroll
    for (int i = 0; i < kDims; ++i)
        if (lane + 32 * i < D) sm_o[warp][lane + 32 * i] = o[i];
    __syncthreads();
    float top = sm_m[0];
    for (int w = 1; w < 4; ++w) top = fmaxf(top, sm_m[w]);
    float part[4], total = 0.f;
    for (int w = 0; w < 4; ++w) {
        part[w] = sm_m[w] == -INFINITY ? (top == -INFINITY ? 1.f : 0.f) : exp2f(sm_m[w] - top);
        total += part[w] * sm_l[w];
    }
    for (int d = threadIdx.x; d < D; d += blockDim.x) {
        float v = 0.f;
        for (int w = 0; w < 4; ++w) v += part[w] * sm_o[w][d];
        p.out[((int64_t)b * p.Hq + hq) * D + d] = n > 0 ? f32_to_act_bits<F16>(v / total) : 0;
    }
    if (p.lse && threadIdx.x == 0)
        p.lse[(int64_t)b * p.Hq + hq] = n > 0 ? (top + log2f(total)) * 0.693147180559945309f : -INFINITY;
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" size_t nvfp4_paged_attention_workspace(int64_t B, int64_t Hq, int64_t heads, int64_t head_dim) {
    (void)B; (void)Hq; (void)heads; (void)head_dim;
    return 0;
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
    if (table_width < 0 || table_width * p.cache.page_size > INT32_MAX - 64 || table_width > INT32_MAX)
        return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: a table of %lld pages of %d tokens passes 2^31 tokens", fn, (long long)table_width, p.cache.page_size);
    if (B > 65535) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: B=%lld above 65535", fn, (long long)B);
    if (B == 0) return NVFP4_OK;
    if (!q || !lengths || !out || (table_width > 0 && !block_table)) return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (q_row_stride < 0 || q_head_stride < 0 || table_stride < 0) return fail(NVFP4_ERR_INVALID_ARG, "%s: negative stride", fn);
    if (!aligned(q, 16) || q_row_stride % 8 || q_head_stride % 8 || !aligned(out, 16) || !aligned(block_table, 4) || !aligned(lengths, 4) || !aligned(lse, 4))
        return fail(NVFP4_ERR_ALIGNMENT, "%s: q's rows and out must be 16-byte aligned, block_table, lengths and lse 4-byte", fn);
    const size_t need = nvfp4_paged_attention_workspace(B, Hq, p.cache.heads, p.cache.D);
    if (workspace_bytes < need || (need > 0 && !workspace))
        return fail(NVFP4_ERR_WORKSPACE, "%s: workspace %zu bytes, needs %zu", fn, workspace_bytes, need);
    if (need > 0 && !aligned(workspace, 256)) return fail(NVFP4_ERR_ALIGNMENT, "%s: workspace must be 256-byte aligned", fn);
    p.status = device_status_ptr();
    if (!p.status) return fail(NVFP4_ERR_CUDA, "%s: no CUDA device", fn);
    p.q = (const uint16_t*)q; p.q_row = q_row_stride; p.q_head = q_head_stride;
    p.block_table = block_table; p.table_stride = table_stride; p.width = (int)table_width;
    p.lengths = lengths; p.out = (uint16_t*)out; p.lse = lse;
    p.B = (int)B; p.Hq = (int)Hq; p.G = (int)(Hq / p.cache.heads);
    p.window = (int)std::min<int64_t>(window, INT32_MAX);
    p.scale_log2 = softmax_scale * 1.44269504088896341f;
    const dim3 grid((unsigned)Hq, (unsigned)B);
    if (f16) attend_any_kernel<true><<<grid, 128, 0, (cudaStream_t)stream>>>(p);
    else attend_any_kernel<false><<<grid, 128, 0, (cudaStream_t)stream>>>(p);
    return check_cuda(cudaGetLastError(), fn);
}
