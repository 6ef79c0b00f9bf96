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
#include "overlap.cuh"
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
    int64_t group, groups;         // columns of one scale (H: one a row), scales a row
    int lanes_log2;                // groups of 16 to 256 columns: threads of one, eight columns each
    float eps;
};

template <bool MAX>
__device__ __forceinline__ float join(float a, float b) { return MAX ? fmaxf(a, b) : a + b; }

// Reduction over a warp.
template <bool MAX>
__device__ __forceinline__ float lane_reduce(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = join<MAX>(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The largest of each of V values over groups of 2^log2 neighbouring lanes.
template <int V>
__device__ __forceinline__ void group_max(float (&v)[V], int log2) {
#pragma unroll
    for (int k = 0; k < 5; ++k) {
        if (k >= log2) break;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = fmaxf(v[i], __shfl_xor_sync(0xffffffffu, v[i], 1 << k));
    }
}

// Reduction over the threads of a row; every thread gets the result.  `sm` holds
// a float a warp and is used once.
template <bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* sm) {
    v = lane_reduce<MAX>(v);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    v = (threadIdx.x & 31) < warps ? sm[threadIdx.x & 31] : 0.f;     // sums and magnitudes: 0 is neutral
    return lane_reduce<MAX>(v);
}

// Threads of a row at most: V pieces a thread have to fit in the registers.
constexpr int norm_threads(int V) { return V == 1 ? 1024 : 512; }
// Blocks of so many that an SM holds at least, by 64 registers a thread for four pieces
// (69 without the limit: 8192x8192 to E4M3 74.4 us, with it 71.7).
constexpr int norm_blocks(int V) { return V == 4 ? 2 : 1; }

// Rows of 16-byte pieces: a row's threads keep it in registers, V pieces of 8
// elements each, so that it is read once.
// Bound by memory: 2 or 3 passes' worth of bytes a row (x, residual in; r, y
// out), all loads issued before the first use, and the weights' (from L2) before
// the one barrier of the sum: 8192x8192 in 79.2 us (6.8 TB/s), 4096x5120 to E4M3 in
// 22.9 (6.4).  The E4M3 output is not far from its instructions' time: values are kept
// for both of its passes, and computed in pairs.
template <bool F16, bool E4M3, int V>
__global__ void __launch_bounds__(norm_threads(V), norm_blocks(V)) norm_rows_kernel(const NormParams p) {
    __shared__ float sm[2][32];
    pdl_wait_previous();
    pdl_launch_dependents();
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= p.T) return;                              // whole warps: several rows a block have a warp each
    const int pieces = (int)(p.H / 8);
    uint4 x[V], w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        x[i] = c < pieces ? ldg_once(p.x + t * p.x_stride + c * 8) : make_uint4(0, 0, 0, 0);
    }
    if (p.residual) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            w[i] = c < pieces ? ldg_once(p.residual + t * p.res_stride + c * 8) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            uint32_t* a = &x[i].x;
            const uint32_t* b = &w[i].x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 u = act2_to_f32<F16>(a[j]), v = act2_to_f32<F16>(b[j]);
                a[j] = f32_to_act2<F16>(u.x + v.x, u.y + v.y);
            }
            if (c < pieces) *(uint4*)(p.residual_out + t * p.H + c * 8) = x[i];
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        w[i] = c < pieces ? *(const uint4*)(p.weight + c * 8) : make_uint4(0, 0, 0, 0);
    }
    F2 sums = make_f2(0.f, 0.f), y[V][4];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t* a = &x[i].x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y[i][j] = widen2<F16>(a[j]);
            sums = fma2(y[i][j], y[i][j], sums);
        }
    }
    const float2 sum = both(sums);
    const float rstd = rsqrtf(row_reduce<false>(sum.x + sum.y, sm[0]) / (float)p.H + p.eps);
    const F2 rstd2 = make_f2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t* b = &w[i].x;
#pragma unroll
        for (int j = 0; j < 4; ++j) y[i][j] = mul2(mul2(y[i][j], rstd2), widen2<F16>(b[j]));
    }
    if constexpr (!E4M3) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 u = both(y[i][j]);
                o[j] = f32_to_act2<F16>(u.x, u.y);
            }
            if (c < pieces) *(uint4*)((uint16_t*)p.y + t * p.H + c * 8) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    } else {
        const bool by_row = p.group == p.H;
        float amax[V], top = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            amax[i] = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 u = both(y[i][j]);
                amax[i] = fmaxf(fmaxf(amax[i], fabsf(u.x)), fabsf(u.y));
            }
            top = fmaxf(top, amax[i]);
        }
        if (by_row) top = row_reduce<true>(top, sm[1]);
        else group_max<V>(amax, p.lanes_log2);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            const float s = e4m3_scale(by_row ? top : amax[i]), inv = e4m3_inverse(s);
            if (c >= pieces) continue;
            if (by_row ? c == 0 : (threadIdx.x & ((1 << p.lanes_log2) - 1)) == 0)
                p.scales[t * p.groups + (by_row ? 0 : c >> p.lanes_log2)] = s;
            const F2 minus_s = make_f2(-s, -s), inv2 = make_f2(inv, inv);
            const uint32_t o0 = e4m3_codes(y[i][0], minus_s, inv2), o1 = e4m3_codes(y[i][1], minus_s, inv2);
            const uint32_t o2 = e4m3_codes(y[i][2], minus_s, inv2), o3 = e4m3_codes(y[i][3], minus_s, inv2);
            *(uint2*)((uint8_t*)p.y + t * p.H + c * 8) = make_uint2(o0 | o1 << 16, o2 | o3 << 16);
        }
    }
}

// Rows of any width up to 8192, element by element (VEC 1), or up to 16384 in twos
// where width, strides and pointers are even: kept in registers like the rows above,
// V elements or twos a thread, as 16-bit values.  Such loads are narrow but many
// in flight: 8000 x 4098 53 us (4.9 TB/s), 8000 x 4097 94 us, bound by the number of
// loads; sixteen a thread were slower (64 and 160).  One E4M3 scale a row.
template <bool F16, bool E4M3, int VEC, int V>
__global__ void __launch_bounds__(1024) norm_narrow_kernel(const NormParams p) {
    __shared__ float sm[2][32];
    pdl_wait_previous();
    pdl_launch_dependents();
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (t >= p.T) return;                              // whole warps, as above
    const int n = (int)p.H / VEC;
    auto load = [](const uint16_t* from) -> uint32_t { return VEC == 2 ? *(const uint32_t*)from : *from; };
    uint32_t r[V], w[V];
    const uint16_t* x = p.x + t * p.x_stride;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        r[i] = c < n ? load(x + c * VEC) : 0u;
    }
    if (p.residual) {
        const uint16_t* a = p.residual + t * p.res_stride;
        uint16_t* to = p.residual_out + t * p.H;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            w[i] = c < n ? load(a + c * VEC) : 0u;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = i * blockDim.x + threadIdx.x;
            const float2 u = act2_to_f32<F16>(r[i]), v = act2_to_f32<F16>(w[i]);
            r[i] = f32_to_act2<F16>(u.x + v.x, u.y + v.y);
            if (c >= n) continue;
            if (VEC == 2) *(uint32_t*)(to + c * 2) = r[i];
            else to[c] = (uint16_t)r[i];
        }
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        w[i] = c < n ? load(p.weight + c * VEC) : 0u;
        const float2 u = act2_to_f32<F16>(r[i]);
        sum += u.x * u.x + (VEC == 2 ? u.y * u.y : 0.f);
    }
    const float rstd = rsqrtf(row_reduce<false>(sum, sm[0]) / (float)p.H + p.eps);
    auto value = [&](int i) {
        const float2 u = act2_to_f32<F16>(r[i]), v = act2_to_f32<F16>(w[i]);
        return make_float2(u.x * rstd * v.x, VEC == 2 ? u.y * rstd * v.y : 0.f);
    };
    float s = 1.f, inv = 1.f;
    if (E4M3) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float2 y = value(i);
            amax = fmaxf(amax, fmaxf(fabsf(y.x), fabsf(y.y)));
        }
        s = e4m3_scale(row_reduce<true>(amax, sm[1]));
        inv = e4m3_inverse(s);
        if (threadIdx.x == 0) p.scales[t] = s;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        if (c >= n) continue;
        const float2 y = value(i);
        if (E4M3) {
            const uint16_t o = f32_to_e4m3x2(quotient(y.x, s, inv), quotient(y.y, s, inv));
            if (VEC == 2) *(uint16_t*)((uint8_t*)p.y + t * p.H + c * 2) = o;
            else ((uint8_t*)p.y)[t * p.H + c] = (uint8_t)o;
        } else if (VEC == 2) {
            *(uint32_t*)((uint16_t*)p.y + t * p.H + c * 2) = f32_to_act2<F16>(y.x, y.y);
        } else {
            ((uint16_t*)p.y)[t * p.H + c] = f32_to_act_bits<F16>(y.x);
        }
    }
}

// Any width, stride and alignment: a block walks a row element by element, and
// reads it again (from L1/L2) for the output.
template <bool F16>
__global__ void __launch_bounds__(1024) norm_any_kernel(const NormParams p) {
    __shared__ float sm[2][32];
    pdl_wait_previous();
    pdl_launch_dependents();
    const int64_t t = blockIdx.x;
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
    sum = row_reduce<false>(sum, sm[0]);               // its barrier makes the block's r visible, too
    const float rstd = rsqrtf(sum / (float)p.H + p.eps);
    auto value = [&](int64_t i) { return act_to_f32<F16>(r[i]) * rstd * act_to_f32<F16>(p.weight[i]); };
    if (!p.scales) {
        uint16_t* y = (uint16_t*)p.y + t * p.H;
        for (int64_t i = threadIdx.x; i < p.H; i += blockDim.x) y[i] = f32_to_act_bits<F16>(value(i));
        return;
    }
    uint8_t* y = (uint8_t*)p.y + t * p.H;
    if (p.group == p.H) {
        float amax = 0.f;
        for (int64_t i = threadIdx.x; i < p.H; i += blockDim.x) amax = fmaxf(amax, fabsf(value(i)));
        const float s = e4m3_scale(row_reduce<true>(amax, sm[1])), inv = e4m3_inverse(s);
        if (threadIdx.x == 0) p.scales[t] = s;
        for (int64_t i = threadIdx.x; i < p.H; i += blockDim.x) y[i] = e4m3_code(value(i), s, inv);
        return;
    }
    const int lane = threadIdx.x & 31;                 // a warp takes a group at a time
    for (int64_t g = threadIdx.x >> 5; g < p.groups; g += blockDim.x >> 5) {
        float amax = 0.f;
        for (int64_t i = g * p.group + lane; i < (g + 1) * p.group; i += 32) amax = fmaxf(amax, fabsf(value(i)));
        const float s = e4m3_scale(lane_reduce<true>(amax)), inv = e4m3_inverse(s);
        if (lane == 0) p.scales[t * p.groups + g] = s;
        for (int64_t i = g * p.group + lane; i < (g + 1) * p.group; i += 32)
            y[i] = e4m3_code(value(i), s, inv);
    }
}

template <bool F16>
const void* rows_kernel(bool e4m3, int V) {
    switch (V) {
        case 1: return e4m3 ? (const void*)norm_rows_kernel<F16, true, 1> : (const void*)norm_rows_kernel<F16, false, 1>;
        case 4: return e4m3 ? (const void*)norm_rows_kernel<F16, true, 4> : (const void*)norm_rows_kernel<F16, false, 4>;
        default: return e4m3 ? (const void*)norm_rows_kernel<F16, true, 8> : (const void*)norm_rows_kernel<F16, false, 8>;
    }
}

template <bool F16, bool E4M3, int VEC>
const void* narrow_kernel(int V) {
    return V == 4 ? (const void*)norm_narrow_kernel<F16, E4M3, VEC, 4> : (const void*)norm_narrow_kernel<F16, E4M3, VEC, 8>;
}
template <bool F16>
const void* narrow_kernel(bool e4m3, bool twos, int V) {
    if (e4m3) return twos ? narrow_kernel<F16, true, 2>(V) : narrow_kernel<F16, true, 1>(V);
    return twos ? narrow_kernel<F16, false, 2>(V) : narrow_kernel<F16, false, 1>(V);
}

nvfp4_status launch_norm(const NormParams& p, bool f16, cudaStream_t stream) {
    const char* fn = "nvfp4_rms_norm";
    const bool e4m3 = p.scales != nullptr;
    const int64_t pieces = p.H / 8;
    const bool rows = p.H % 8 == 0 && pieces <= 4096 && p.x_stride % 8 == 0 && p.res_stride % 8 == 0 && aligned(p.x, 16) &&
                      aligned(p.residual, 16) && aligned(p.weight, 16) && aligned(p.residual_out, 16) && aligned(p.y, e4m3 ? 8 : 16);
    const void* kernel = f16 ? (const void*)norm_any_kernel<true> : (const void*)norm_any_kernel<false>;
    dim3 block(p.H > 4096 ? 1024 : 256);
    if (rows) {
        // Rows that fill the GPU take four pieces a thread: loads in flight, few threads
        // to join and few scales' quotients (8192x8192: one 84.9 us, four 79.1; 500x4096 3.12
        // and 2.95; 8192x8192 to E4M3 91.5 and 71.5).  Few rows take as many threads as they
        // have pieces: that is for narrow ones (1x1024 1.41 us with one, 1.49 with four; to
        // E4M3 with groups of 128 1.56 and 1.90); wide ones lose by it (1x8192 2.31 and 2.01).
        int V = p.T <= sm_count() * 2 ? 1 : 4;
        while (pieces > norm_threads(V) * V) V = V == 1 ? 4 : 8;
        block = dim3((unsigned)round_up(ceil_div(pieces, V), 32));
        kernel = f16 ? rows_kernel<true>(e4m3, V) : rows_kernel<false>(e4m3, V);
    } else if (p.group == p.H) {
        const bool twos = p.H % 2 == 0 && p.x_stride % 2 == 0 && p.res_stride % 2 == 0 && aligned(p.x, 4) && aligned(p.residual, 4) &&
                          aligned(p.weight, 4) && aligned(p.residual_out, 4) && aligned(p.y, e4m3 ? 2 : 4);
        const int64_t n = twos ? p.H / 2 : p.H;
        if (n <= 8192) {
            const int V = p.T > sm_count() * 2 || n > 4096 ? 8 : 4;
            block = dim3((unsigned)round_up(ceil_div(n, V), 32));
            kernel = f16 ? narrow_kernel<true>(e4m3, twos, V) : narrow_kernel<false>(e4m3, twos, V);
        }
    }
    if (block.x == 32) block.y = p.T > sm_count() * 2 ? 8 : 1;        // a warp a row
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ceil_div(p.T, block.y));
    cfg.blockDim = block;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {const_cast<NormParams*>(&p)};
    return check_cuda(cudaLaunchKernelExC(&cfg, kernel, args), fn);
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status nvfp4_rms_norm(const void* X, int64_t x_stride, const void* residual, int64_t residual_stride,
                                       const void* weight, int64_t T, int64_t H, float eps, int out_type, int64_t group,
                                       int f16, void* Y, float* scales, void* residual_out, void* stream) {
    const char* fn = "nvfp4_rms_norm";
    if (T < 0) return fail(NVFP4_ERR_INVALID_ARG, "%s: negative size T=%lld", fn, (long long)T);
    if (T > INT32_MAX) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: T=%lld too large", fn, (long long)T);
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
    // A thread reads its elements of X and residual before it writes them, so an output of
    // their type may be one of them; anything else would be read by others after that.
    const Span x = strided_span("X", X, 2 * H, {{T, 2 * x_stride}}), res = strided_span("residual", residual, 2 * H, {{T, 2 * residual_stride}});
    const Span y = dense_span("Y", Y, T * H * (e4m3 ? 1 : 2)), sums = dense_span("residual_out", residual_out, 2 * T * H);
    const Span by = dense_span("scales", e4m3 ? scales : nullptr, 4 * T * (group ? H / group : 1)), w = dense_span("weight", weight, 2 * H);
    for (const Span& in : {x, res})
        for (const Span& out : {y, sums})
            if (overlaps(out, in) && !same_place(out, in))
                return fail(NVFP4_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, out.name, in.name);
    if (const char* s = met(by, {x, res, w})) return fail(NVFP4_ERR_INVALID_ARG, "%s: scales overlap %s", fn, s);
    if (const char* s = met(sums, {w, by})) return fail(NVFP4_ERR_INVALID_ARG, "%s: residual_out overlaps %s", fn, s);
    if (const char* s = met(y, {w, by, sums})) return fail(NVFP4_ERR_INVALID_ARG, "%s: Y overlaps %s", fn, s);
    if (sm_count() <= 0 || device_status_ptr() == nullptr) return fail(NVFP4_ERR_CUDA, "%s: no CUDA device", fn);
    NormParams p{};
    p.x = (const uint16_t*)X; p.residual = (const uint16_t*)residual; p.weight = (const uint16_t*)weight;
    p.residual_out = (uint16_t*)residual_out; p.y = Y; p.scales = e4m3 ? scales : nullptr;
    p.T = T; p.H = H; p.x_stride = x_stride; p.res_stride = residual_stride;
    p.group = group ? group : H; p.groups = H / p.group; p.eps = eps;
    for (p.lanes_log2 = 0; group > 8 << p.lanes_log2;) ++p.lanes_log2;
    return launch_norm(p, f16 != 0, (cudaStream_t)stream);
}
