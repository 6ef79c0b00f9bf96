// Root-mean-square norm of rows, with the residual's addition before it and a
// 16-bit or an E4M3 output:
//     r = RN16(x + residual)  (or x),   y = r * rsqrt(mean(r^2) + eps) * w,
//     out = RN16(y),  or  s = max(amax(|y|) / 448, 2^-100), code = E4M3(y / s)
// with s per row or per group of columns.  r is rounded before it is normalised:
// the norm is the norm of the stream that is stored, whoever reads it back.
// Squares and their sum, y and s are held in 32 bits.
#include <algorithm>

#include "common.cuh"
#include "numeric.cuh"
#include "ptx.cuh"

namespace nvfp4 {
namespace {

struct NormParams {
    const uint16_t* x;
    const uint16_t* residual;      // null: no addition
    const uint16_t* weight;
    uint16_t* residual_out;
    void* y;
    float* scales;                 // null: 16-bit output
    int64_t T, H, x_stride, res_stride;
    int64_t group;                 // columns of one scale (H: one a row)
    float eps;
};

template <bool MAX>
__device__ __forceinline__ float warp_reduce(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float u = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? fmaxf(v, u) : v + u;
    }
    return v;
}

// Reduction over the block; every thread gets the result.
template <bool MAX>
__device__ float block_reduce(float v, float* sm) {
    v = warp_reduce<MAX>(v);
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    __syncthreads();                                   // the last use of sm is over
    if ((threadIdx.x & 31) == 0) sm[warp] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < warps ? sm[threadIdx.x & 31] : 0.f;     // sums and magnitudes: 0 is neutral
    return warp_reduce<MAX>(v);
}

// Any width, stride and alignment: a block walks a row element by element, and
// reads it again (from L1/L2) for the output.
template <bool F16>
__global__ void __launch_bounds__(256) norm_any_kernel(NormParams p) {
    __shared__ float sm[32];
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const uint16_t* x = p.x + t * p.x_stride;
        const uint16_t* r = x;
        float sum = 0.f;
        for (int64_t i = threadIdx.x; i < p.H; i += blockDim.x) {
            float v = act_to_f32<F16>(x[i]);
            if (p.residual) {
                const uint16_t b = f32_to_act_bits<F16>(v + act_to_f32<F16>(p.residual[t * p.res_stride + i]));
                p.residual_out[t * p.H + i] = b;
                v = act_to_f32<F16>(b);
            }
            sum += v * v;
        }
        if (p.residual) r = p.residual_out + t * p.H;
        sum = block_reduce<false>(sum, sm);            // its barriers make the block's r visible, too
        const float rstd = rsqrtf(sum / (float)p.H + p.eps);
        if (!p.scales) {
            uint16_t* y = (uint16_t*)p.y + t * p.H;
            for (int64_t i = threadIdx.x; i < p.H; i += blockDim.x)
                y[i] = f32_to_act_bits<F16>(act_to_f32<F16>(r[i]) * rstd * act_to_f32<F16>(p.weight[i]));
            continue;
        }
        uint8_t* y = (uint8_t*)p.y + t * p.H;
        const int64_t groups = p.H / p.group;
        for (int64_t g = 0; g < groups; ++g) {
            const int64_t end = (g + 1) * p.group;
            float amax = 0.f;
            for (int64_t i = g * p.group + threadIdx.x; i < end; i += blockDim.x)
                amax = fmaxf(amax, fabsf(act_to_f32<F16>(r[i]) * rstd * act_to_f32<F16>(p.weight[i])));
            const float s = e4m3_scale(block_reduce<true>(amax, sm));
            if (threadIdx.x == 0) p.scales[t * groups + g] = s;
            for (int64_t i = g * p.group + threadIdx.x; i < end; i += blockDim.x)
                y[i] = (uint8_t)f32_to_e4m3x2(
                    __fdiv_rn(act_to_f32<F16>(r[i]) * rstd * act_to_f32<F16>(p.weight[i]), s), 0.f);
        }
    }
}

nvfp4_status launch_norm(const NormParams& p, bool f16, cudaStream_t s) {
    const int grid = (int)std::min<int64_t>(p.T, (int64_t)sm_count() * 8);
    if (f16) norm_any_kernel<true><<<grid, 256, 0, s>>>(p);
    else norm_any_kernel<false><<<grid, 256, 0, s>>>(p);
    return check_cuda(cudaGetLastError(), "nvfp4_rms_norm");
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status nvfp4_rms_norm(const void* X, int64_t x_stride, const void* residual, int64_t residual_stride,
                                       const void* weight, int64_t T, int64_t H, float eps, int out_type, int64_t group,
                                       int f16, void* Y, float* scales, void* residual_out, void* stream) {
    const char* fn = "nvfp4_rms_norm";
    if (T < 0) return fail(NVFP4_ERR_INVALID_ARG, "%s: negative size T=%lld", fn, (long long)T);
    if (H <= 0 || H > (1 << 24)) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: H=%lld must be in [1, 2^24]", fn, (long long)H);
    if (f16 != 0 && f16 != 1) return fail(NVFP4_ERR_INVALID_ARG, "%s: f16=%d must be 0 or 1", fn, f16);
    if (out_type != NVFP4_OUT_16 && out_type != NVFP4_OUT_E4M3)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: out_type=%d must be NVFP4_OUT_16 or NVFP4_OUT_E4M3", fn, out_type);
    if (!(eps >= 0.f) || eps > 3.4e38f) return fail(NVFP4_ERR_INVALID_ARG, "%s: eps must be finite and not negative", fn);
    const bool e4m3 = out_type == NVFP4_OUT_E4M3;
    const bool known = group == 0 || group == 16 || group == 32 || group == 64 || group == 128 || group == 256;
    if (!known || (!e4m3 && group != 0) || (group != 0 && H % group != 0))
        return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: group=%lld must be 0, or (E4M3 output) 16, 32, 64, 128 or 256 and divide H=%lld",
                    fn, (long long)group, (long long)H);
    if (T == 0) return NVFP4_OK;
    if (!X || !weight || !Y || (e4m3 && !scales)) return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", fn);
    if ((residual == nullptr) != (residual_out == nullptr))
        return fail(NVFP4_ERR_INVALID_ARG, "%s: residual and residual_out go together", fn);
    if (x_stride < 0 || residual_stride < 0) return fail(NVFP4_ERR_INVALID_ARG, "%s: negative stride", fn);
    if (!aligned(X, 2) || !aligned(weight, 2) || (!e4m3 && !aligned(Y, 2)) || !aligned(residual, 2) ||
        !aligned(residual_out, 2) || !aligned(scales, 4))
        return fail(NVFP4_ERR_ALIGNMENT, "%s: pointers must be aligned to their elements", fn);
    if (sm_count() <= 0 || device_status_ptr() == nullptr) return fail(NVFP4_ERR_CUDA, "%s: no CUDA device", fn);
    NormParams p{};
    p.x = (const uint16_t*)X; p.residual = (const uint16_t*)residual; p.weight = (const uint16_t*)weight;
    p.residual_out = (uint16_t*)residual_out; p.y = Y; p.scales = e4m3 ? scales : nullptr;
    p.T = T; p.H = H; p.x_stride = x_stride; p.res_stride = residual_stride;
    p.group = group ? group : H; p.eps = eps;
    return launch_norm(p, f16 != 0, (cudaStream_t)stream);
}
