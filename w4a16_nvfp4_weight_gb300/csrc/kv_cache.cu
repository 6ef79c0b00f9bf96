// Rotary positions with the write into a paged key-value cache, and the read of
// cached rows.
//
// Rotation: frequency i of R/2 belongs to the position axis whose section holds
// it; with (c, s) = (table[p, i], table[p, R/2 + i]) of that axis's position p,
//     (x1, x2) -> (x1 c - x2 s, x2 c + x1 s)
// for the pair (x[i], x[i + R/2]), or (x[2i], x[2i+1]) when interleaved; elements
// from R on pass through.  The products and their sum are separate 32-bit
// roundings (no fused multiply-add), so that a key is the same bits, and gets
// the same 8-bit code, in whatever kernel it is computed.
// Write: keys (rotated) and values rounded once, to the activation type or to
// E4M3 with s = max(amax / 448, 2^-100) per token and head.
#include <algorithm>

#include "common.cuh"
#include "kv_cache.cuh"
#include "numeric.cuh"
#include "ptx.cuh"

namespace nvfp4 {

nvfp4_status check_cache(const char* fn, const nvfp4_kv_cache* c, CacheView* view) {
    if (!c) return fail(NVFP4_ERR_INVALID_ARG, "%s: null cache", fn);
    if (c->type != NVFP4_CACHE_16 && c->type != NVFP4_CACHE_E4M3)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: cache type %lld must be NVFP4_CACHE_16 or NVFP4_CACHE_E4M3", fn, (long long)c->type);
    const bool e4m3 = c->type == NVFP4_CACHE_E4M3;
    const int64_t es = e4m3 ? 1 : 2;
    if (c->num_pages <= 0 || c->num_pages > INT32_MAX || c->page_size <= 0 || c->page_size > (1 << 20) || c->heads <= 0 || c->heads > 4096)
        return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: cache of %lld pages of %lld tokens, %lld heads (limits 2^31-1, 2^20, 4096)", fn,
                    (long long)c->num_pages, (long long)c->page_size, (long long)c->heads);
    if (c->head_dim <= 0 || c->head_dim % 16 != 0 || c->head_dim > kMaxHeadDim)
        return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: head_dim=%lld must be a multiple of 16 up to %d", fn, (long long)c->head_dim, kMaxHeadDim);
    if (!c->k || !c->v || (e4m3 && (!c->k_scale || !c->v_scale)))
        return fail(NVFP4_ERR_INVALID_ARG, "%s: null cache pointer", fn);
    if (c->page_stride <= 0 || c->head_stride <= 0 || c->token_stride < c->head_dim)
        return fail(NVFP4_ERR_INVALID_ARG, "%s: cache strides (%lld, %lld, %lld) must be positive and hold a row", fn,
                    (long long)c->page_stride, (long long)c->head_stride, (long long)c->token_stride);
    if (c->page_stride * es % 16 || c->head_stride * es % 16 || c->token_stride * es % 16 || !aligned(c->k, 16) || !aligned(c->v, 16))
        return fail(NVFP4_ERR_ALIGNMENT, "%s: cache rows must start on 16-byte boundaries", fn);
    if (e4m3 && (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)))
        return fail(NVFP4_ERR_ALIGNMENT, "%s: cache scales must be 4-byte aligned", fn);
    view->k = (uint8_t*)c->k; view->v = (uint8_t*)c->v;
    view->k_scale = e4m3 ? c->k_scale : nullptr; view->v_scale = e4m3 ? c->v_scale : nullptr;
    view->num_pages = c->num_pages; view->num_slots = c->num_pages * c->page_size;
    view->page_bytes = c->page_stride * es; view->head_bytes = c->head_stride * es; view->token_bytes = c->token_stride * es;
    view->page_size = (int)c->page_size; view->heads = (int)c->heads; view->D = (int)c->head_dim;
    view->page_shift = -1;
    for (int i = 0; i <= 20; ++i)
        if (view->page_size == 1 << i) view->page_shift = i;
    for (view->page_mul_shift = 0; 2 << view->page_mul_shift < view->page_size;) ++view->page_mul_shift;
    view->page_mul = (uint32_t)(((1ull << (32 + view->page_mul_shift)) + c->page_size - 1) / c->page_size);
    view->e4m3 = e4m3;
    return NVFP4_OK;
}

namespace {

constexpr int kMaxAxes = 4;
constexpr int kRopeThreads = 128;

struct RopeParams {
    const uint16_t *q, *k, *v;
    int64_t q_token, q_head, k_token, k_head, v_token, v_head;   // strides, elements
    const int64_t* positions;      // [axes, T]
    const float* table;            // [rows, rot]: cosines, then sines
    const int64_t* slots;
    uint16_t* q_out;               // [T, Hq, D]
    int64_t T, rows;
    int Hq, Hkv, D, rot, axes;
    int end[kMaxAxes];             // frequencies [end[a-1], end[a]) belong to axis a
    int* status;
    CacheView cache;
};

// The position of frequency f's axis, or -1 (recorded) outside the table.
__device__ __forceinline__ int64_t axis_position(const RopeParams& p, int64_t t, int f) {
    int a = 0;
    while (a + 1 < p.axes && f >= p.end[a]) ++a;
    const int64_t pos = p.positions[a * p.T + t];
    if ((uint64_t)pos < (uint64_t)p.rows) return pos;
    record_status(p.status, NVFP4_ERR_BAD_INDEX);
    return -1;
}

// Any rot: a warp takes one head of one token, a lane every 32nd element.
template <bool F16, bool INTER>
__global__ void __launch_bounds__(256) rope_write_any_kernel(const RopeParams p) {
    pdl_wait_previous();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int heads = p.Hq + 2 * p.Hkv;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
    const int half = p.rot / 2;
    for (int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); w < p.T * heads; w += warps) {
        const int64_t t = w / heads;
        int h = (int)(w % heads);
        const int kind = h < p.Hq ? 0 : h < p.Hq + p.Hkv ? 1 : 2;       // query, key, value
        h -= kind == 0 ? 0 : kind == 1 ? p.Hq : p.Hq + p.Hkv;
        const int64_t slot = p.slots[t];
        if (kind > 0 && slot < 0) continue;
        if (kind > 0 && slot >= p.cache.num_slots) {
            if (lane == 0) record_status(p.status, NVFP4_ERR_BAD_INDEX);
            continue;
        }
        const uint16_t* x = kind == 0 ? p.q + t * p.q_token + h * p.q_head
                          : kind == 1 ? p.k + t * p.k_token + h * p.k_head : p.v + t * p.v_token + h * p.v_head;
        float y[kMaxHeadDim / 32];
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < kMaxHeadDim / 32; ++i) {
            const int d = lane + 32 * i;
            y[i] = 0.f;
            if (d >= p.D) continue;
            float v = act_to_f32<F16>(x[d]);
            if (kind < 2 && d < p.rot) {
                const int f = INTER ? d / 2 : d % half;
                const bool first = INTER ? d % 2 == 0 : d < half;
                const float other = act_to_f32<F16>(x[INTER ? d ^ 1 : first ? d + half : d - half]);
                const int64_t pos = axis_position(p, t, f);
                const float c = pos < 0 ? 1.f : p.table[pos * p.rot + f], s = pos < 0 ? 0.f : p.table[pos * p.rot + half + f];
                v = first ? __fsub_rn(__fmul_rn(v, c), __fmul_rn(other, s)) : __fadd_rn(__fmul_rn(v, c), __fmul_rn(other, s));
            }
            y[i] = v;
            amax = fmaxf(amax, fabsf(v));
        }
        __syncwarp();                                  // q_out may be q: no store before every lane has read its pair
        if (kind == 0) {
#pragma unroll
            for (int i = 0; i < kMaxHeadDim / 32; ++i)
                if (lane + 32 * i < p.D) p.q_out[(t * p.Hq + h) * p.D + lane + 32 * i] = f32_to_act_bits<F16>(y[i]);
            continue;
        }
        int64_t page;
        int at;
        p.cache.split(slot, &page, &at);
        uint8_t* row = (kind == 1 ? p.cache.k : p.cache.v) + p.cache.row(page, h, at);
        if (!p.cache.e4m3) {
#pragma unroll
            for (int i = 0; i < kMaxHeadDim / 32; ++i)
                if (lane + 32 * i < p.D) ((uint16_t*)row)[lane + 32 * i] = f32_to_act_bits<F16>(y[i]);
            continue;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float s = e4m3_scale(amax), inv = e4m3_inverse(s);
        if (lane == 0) (kind == 1 ? p.cache.k_scale : p.cache.v_scale)[p.cache.scale_at(page, h, at)] = s;
#pragma unroll
        for (int i = 0; i < kMaxHeadDim / 32; ++i)
            if (lane + 32 * i < p.D) row[lane + 32 * i] = e4m3_code(y[i], s, inv);
    }
}

// A piece of PE elements of a row (8: 16 bytes, 4: 8 bytes) as words.
template <int PE>
__device__ __forceinline__ void load_piece(uint32_t* w, const uint16_t* from) {
    if constexpr (PE == 8) {
        const uint4 v = ldg_once(from);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else {
        asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(from) : "memory");
    }
}
template <int WORDS>
__device__ __forceinline__ void store_words(void* to, const uint32_t* w) {
    if constexpr (WORDS == 4) *(uint4*)to = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (WORDS == 2) *(uint2*)to = make_uint2(w[0], w[1]);
    else *(uint32_t*)to = w[0];
}

// rot a multiple of 2 PE: a thread takes 2 PE elements of several heads of one
// token, both sides of PE pairs, so that nothing is exchanged: pieces j and
// j + rot/(2 PE) of PE elements (INTER: 2j and 2j + 1), past rot two neighbouring
// pieces as they are.  PE is 8 where rot allows it, else 4.  L threads a head (a
// power of two), `per` heads a token at a time, `tokens` a block of at most kRopeThreads.
// Bound by memory (q, k, v in, q and the cache rows out) and not far from it by
// instructions: 20.4 us (5.9 TB/s) for 4096 tokens of 40 + 2 * 8 heads of 128
// with three axes, where a piece of 8 a thread with its mate's by shuffle (176
// instructions a warp for two heads) took 30.  The rows of U heads are loaded first;
// then the block fetches its tokens' cosines and sines into shared memory, a
// thread a frequency (each thread fetching its own through L1: 40 us), whose addresses
// wait for the positions: those are asked for before the rows.
template <bool F16, bool INTER, bool E4M3, int U, int PE>
__global__ void __launch_bounds__(kRopeThreads, (E4M3 && U > 1 ? 768 : 896) / kRopeThreads)
rope_write_kernel(const RopeParams p, int log2_L, int per, int tokens) {
    constexpr int PW = PE / 2;                         // words of a piece, pairs of frequencies
    pdl_wait_previous();
    pdl_launch_dependents();
    const int L = 1 << log2_L, j = threadIdx.x & (L - 1), group = threadIdx.x >> log2_L;
    const int own = tokens == 1 ? 0 : group / per;                 // the thread's of the block's tokens
    const int64_t t = (int64_t)blockIdx.x * tokens + own;
    const bool live = t < p.T && j * 2 * PE < p.D;
    const int heads = p.Hq + 2 * p.Hkv, stride = per * gridDim.y;
    const int first = blockIdx.y * per + group - own * per;
    const bool turns = j * 2 * PE < p.rot;
    const int half = p.rot / 2;
    const int e0 = INTER || !turns ? j * 2 * PE : j * PE;          // first element of the two pieces
    const int e1 = INTER || !turns ? j * 2 * PE + PE : half + j * PE;
    const uint32_t same = (L == 32 ? 0xffffffffu : (1u << L) - 1) << (threadIdx.x & 31 & ~(L - 1));     // the lanes of this head
    F2 cs[PW], sn[PW];
    int64_t row = -1, scale_row = 0;                   // byte offset of the token's cache row of head 0

    __shared__ __align__(16) float turn[kRopeThreads * 2 * PE];    // [token][cosines, sines]: kRopeThreads / L tokens of 2 PE L at most
    // Frequency i of the block's tokens: its place in `turn`, and its row of the table (-2: none such).
    auto locate = [&](int i, int* at) -> int64_t {
        if (i >= tokens * half) return -2;
        const int n = tokens == 1 ? 0 : i / half, f = i - n * half;
        const int64_t u = (int64_t)blockIdx.x * tokens + n;
        *at = n * p.rot + f;
        return u < p.T ? axis_position(p, u, f) : -2;
    };
    int turn_at = 0;
    const int64_t slot = live ? p.slots[t] : -1;
    int64_t pos = locate(threadIdx.x, &turn_at);
    uint32_t x[U][2 * PW];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int h = i * stride + first;
#pragma unroll
        for (int n = 0; n < 2 * PW; ++n) x[i][n] = 0;          // lanes past D join in the row's amax
        if (!live || h >= heads) continue;
        const uint16_t* from = h < p.Hq ? p.q + t * p.q_token + h * p.q_head
                             : h < p.Hq + p.Hkv ? p.k + t * p.k_token + (h - p.Hq) * p.k_head
                                                : p.v + t * p.v_token + (h - p.Hq - p.Hkv) * p.v_head;
        load_piece<PE>(x[i], from + e0);
        load_piece<PE>(x[i] + PW, from + e1);
    }
    for (int i = threadIdx.x; pos > -2;) {
        const int f = tokens == 1 ? turn_at : turn_at % p.rot;
        turn[turn_at] = pos < 0 ? 1.f : p.table[pos * p.rot + f];
        turn[turn_at + half] = pos < 0 ? 0.f : p.table[pos * p.rot + half + f];
        i += blockDim.x;
        pos = locate(i, &turn_at);
    }
    __syncthreads();
    if (slot >= p.cache.num_slots) {
        record_status(p.status, NVFP4_ERR_BAD_INDEX);
    } else if (slot >= 0) {
        int64_t page;
        int at;
        p.cache.split(slot, &page, &at);
        row = p.cache.row(page, 0, at);
        scale_row = p.cache.scale_at(page, 0, at);
    }
    if (turns) {
        const float4* from = (const float4*)(turn + own * p.rot + j * PE);
#pragma unroll
        for (int i = 0; i < PE / 4; ++i) {
            const float4 u = from[i], w = from[half / 4 + i];
            cs[2 * i] = make_f2(u.x, u.y); cs[2 * i + 1] = make_f2(u.z, u.w);
            sn[2 * i] = make_f2(w.x, w.y); sn[2 * i + 1] = make_f2(w.z, w.w);
        }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int h = i * stride + first;
        if (h >= heads) break;                     // all lanes of a head together
        const bool value = h >= p.Hq + p.Hkv, codes = E4M3 && h >= p.Hq, moves = !value && turns;
        uint32_t* w = x[i];
        F2 a[PW], b[PW];                           // the first and second sides of the pairs
        if (moves || codes) {
#pragma unroll
            for (int n = 0; n < PW; ++n) {
                const float2 u = act2_to_f32<F16>(w[INTER ? 2 * n : n]), v = act2_to_f32<F16>(w[INTER ? 2 * n + 1 : n + PW]);
                a[n] = INTER ? make_f2(u.x, v.x) : make_f2(u.x, u.y);
                b[n] = INTER ? make_f2(u.y, v.y) : make_f2(v.x, v.y);
                if (moves) {
                    const F2 c = a[n];
                    a[n] = sub2(mul2(c, cs[n]), mul2(b[n], sn[n]));
                    b[n] = add2(mul2(b[n], cs[n]), mul2(c, sn[n]));
                }
            }
        }
        if (!codes) {
            if (moves) {
#pragma unroll
                for (int n = 0; n < PW; ++n) {
                    const float2 u = both(a[n]), v = both(b[n]);
                    w[INTER ? 2 * n : n] = INTER ? f32_to_act2<F16>(u.x, v.x) : f32_to_act2<F16>(u.x, u.y);
                    w[INTER ? 2 * n + 1 : n + PW] = INTER ? f32_to_act2<F16>(u.y, v.y) : f32_to_act2<F16>(v.x, v.y);
                }
            }
            if (!live || (h >= p.Hq && row < 0)) continue;
            uint16_t* to = h < p.Hq ? p.q_out + (t * p.Hq + h) * p.D
                         : (uint16_t*)((value ? p.cache.v + (h - p.Hq - p.Hkv) * p.cache.head_bytes
                                              : p.cache.k + (h - p.Hq) * p.cache.head_bytes) + row);
            store_words<PW>(to + e0, w);
            store_words<PW>(to + e1, w + PW);
            continue;
        }
        float amax = 0.f;
#pragma unroll
        for (int n = 0; n < PW; ++n) {
            const float2 u = both(a[n]), v = both(b[n]);
            amax = fmaxf(fmaxf(amax, fmaxf(fabsf(u.x), fabsf(u.y))), fmaxf(fabsf(v.x), fabsf(v.y)));
        }
#pragma unroll
        for (int k = 0; k < 5; ++k) {
            if (k >= log2_L) break;
            amax = fmaxf(amax, __shfl_xor_sync(same, amax, 1 << k));
        }
        if (!live || row < 0) continue;
        const float s = e4m3_scale(amax), inv = e4m3_inverse(s);
        const int kh = h - p.Hq - (value ? p.Hkv : 0);
        const F2 minus_s = make_f2(-s, -s), inv2 = make_f2(inv, inv);
        uint32_t o[PW];                            // codes of the pieces at e0 and e1
#pragma unroll
        for (int n = 0; n < PW; ++n) {
            F2 one = a[n], two = b[n];             // in the order of the elements
            if (INTER) {
                const float2 u = both(a[n]), v = both(b[n]);
                one = make_f2(u.x, v.x);
                two = make_f2(u.y, v.y);
            }
            const uint32_t c0 = e4m3_codes(one, minus_s, inv2), c1 = e4m3_codes(two, minus_s, inv2);
            if (INTER) {
                o[n] = c0 | c1 << 16;
            } else {
                o[n >> 1] = n & 1 ? o[n >> 1] | c0 << 16 : c0;
                o[PW / 2 + (n >> 1)] = n & 1 ? o[PW / 2 + (n >> 1)] | c1 << 16 : c1;
            }
        }
        uint8_t* to = (value ? p.cache.v : p.cache.k) + kh * p.cache.head_bytes + row;
        store_words<PW / 2>(to + e0, o);
        store_words<PW / 2>(to + e1, o + PW / 2);
        if (j == 0) (value ? p.cache.v_scale : p.cache.k_scale)[scale_row + (int64_t)kh * p.cache.page_size] = s;
    }
}

constexpr int kManyHeads = 4;      // heads a thread takes where there are many tokens

template <bool F16, bool INTER, bool E4M3>
const void* rope_kernel(bool one, int PE) {
    if (PE == 8) return one ? (const void*)rope_write_kernel<F16, INTER, E4M3, 1, 8> : (const void*)rope_write_kernel<F16, INTER, E4M3, kManyHeads, 8>;
    return one ? (const void*)rope_write_kernel<F16, INTER, E4M3, 1, 4> : (const void*)rope_write_kernel<F16, INTER, E4M3, kManyHeads, 4>;
}
template <bool F16>
const void* rope_kernel(bool inter, bool e4m3, bool one, int PE) {
    if (inter) return e4m3 ? rope_kernel<F16, true, true>(one, PE) : rope_kernel<F16, true, false>(one, PE);
    return e4m3 ? rope_kernel<F16, false, true>(one, PE) : rope_kernel<F16, false, false>(one, PE);
}

nvfp4_status launch_after(const void* kernel, dim3 grid, dim3 block, void** args, cudaStream_t stream, const char* fn) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return check_cuda(cudaLaunchKernelExC(&cfg, kernel, args), fn);
}

nvfp4_status launch_rope(RopeParams p, bool f16, bool inter, cudaStream_t stream, const char* fn) {
    const int heads = p.Hq + 2 * p.Hkv;
    if (p.rot % 8 != 0) {
        const void* kernel = f16 ? (inter ? (const void*)rope_write_any_kernel<true, true> : (const void*)rope_write_any_kernel<true, false>)
                                 : (inter ? (const void*)rope_write_any_kernel<false, true> : (const void*)rope_write_any_kernel<false, false>);
        void* args[] = {&p};
        return launch_after(kernel, dim3((unsigned)std::min<int64_t>(ceil_div(p.T * heads, 8), (int64_t)sm_count() * 8)), dim3(256), args, stream, fn);
    }
    const int PE = p.rot % 16 == 0 ? 8 : 4;
    int log2_L = 0;
    while ((2 * PE << log2_L) < p.D) ++log2_L;
    const int L = 1 << log2_L;
    // Many tokens: four heads a thread, all in flight (4096 tokens of 40 + 2 * 8 heads: 20.4
    // us; three 26.6, two 24.6).  Few tokens: one head a thread over as many blocks
    // as that takes, for the shortest way through.
    const bool one = p.T * heads * L <= (int64_t)sm_count() * 1024;
    const int U = one ? 1 : kManyHeads, blocks = (int)ceil_div(heads, U * (kRopeThreads / L));
    int per = (int)ceil_div(heads, U * blocks), tokens = std::max(1, kRopeThreads / (L * per));
    const dim3 grid((unsigned)ceil_div(p.T, tokens), (unsigned)blocks), block(L * per * tokens);
    const void* kernel = f16 ? rope_kernel<true>(inter, p.cache.e4m3, one, PE) : rope_kernel<false>(inter, p.cache.e4m3, one, PE);
    void* args[] = {&p, &log2_L, &per, &tokens};
    return launch_after(kernel, grid, block, args, stream, fn);
}

struct ReadParams {
    CacheView cache;
    const int64_t* slots;
    uint16_t *k_out, *v_out;       // [T, heads, D]
    int64_t T;
    int* status;
};

// A thread takes 16 elements of a key and of a value, or of one of the two (blockIdx.y).
// Bound by memory, and by the threads that wait for it: 65536 tokens of 8 heads of 128
// E4M3 64.6 us (6.3 TB/s) with 32 registers and 8 blocks an SM, 71 with two more
// registers; several rows' loads ahead of the first store did not help (68 to 81).
template <bool F16, bool E4M3>
__global__ void __launch_bounds__(256, 8) cache_read_kernel(const ReadParams p) {
    pdl_wait_previous();
    pdl_launch_dependents();
    const int per = p.cache.D / 16, each = p.cache.heads * per;
    const int64_t total = p.T * each;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t t = total <= INT32_MAX ? (int32_t)i / each : i / each;
        const int x = (int)(i - t * each), h = x / per, c = x - h * per;
        const int64_t row = t * p.cache.heads + h;
        const int64_t slot = p.slots[t];
        const bool held = slot >= 0 && slot < p.cache.num_slots;
        if (slot >= p.cache.num_slots) record_status(p.status, NVFP4_ERR_BAD_INDEX);
#pragma unroll 1
        for (int kv = blockIdx.y; kv < 2; kv += gridDim.y) {
            uint4 out[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
            if (held) {
                int64_t page;
                int at;
                p.cache.split(slot, &page, &at);
                const uint8_t* src = (kv == 0 ? p.cache.k : p.cache.v) + p.cache.row(page, h, at) + c * (E4M3 ? 16 : 32);
                if (!E4M3) {
                    out[0] = ((const uint4*)src)[0];
                    out[1] = ((const uint4*)src)[1];
                } else {
                    const float s = (kv == 0 ? p.cache.k_scale : p.cache.v_scale)[p.cache.scale_at(page, h, at)];
                    const uint4 w = *(const uint4*)src;
                    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
                    uint32_t* o = (uint32_t*)out;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 a = act2_to_f32<true>(e4m3x2_to_f16x2((uint16_t)in[j]));
                        const float2 b = act2_to_f32<true>(e4m3x2_to_f16x2((uint16_t)(in[j] >> 16)));
                        o[2 * j] = f32_to_act2<F16>(a.x * s, a.y * s);
                        o[2 * j + 1] = f32_to_act2<F16>(b.x * s, b.y * s);
                    }
                }
            }
            uint4* dst = (uint4*)((kv == 0 ? p.k_out : p.v_out) + row * p.cache.D + c * 16);
            dst[0] = out[0];
            dst[1] = out[1];
        }
    }
}

bool no_device(int** status) {
    *status = device_status_ptr();
    return *status == nullptr;
}

}  // namespace
}  // namespace nvfp4

using namespace nvfp4;

extern "C" nvfp4_status nvfp4_rope_cache_write(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                               const void* k, int64_t k_token_stride, int64_t k_head_stride,
                                               const void* v, int64_t v_token_stride, int64_t v_head_stride,
                                               int64_t T, int64_t Hq, const int64_t* positions, int axes,
                                               const int32_t* sections, const float* table, int64_t table_rows, int64_t rot,
                                               int interleaved, int f16, const int64_t* slots,
                                               const nvfp4_kv_cache* cache, void* q_out, void* stream) {
    const char* fn = "nvfp4_rope_cache_write";
    RopeParams p{};
    if (nvfp4_status st = check_cache(fn, cache, &p.cache)) return st;
    if (T < 0 || Hq < 0) return fail(NVFP4_ERR_INVALID_ARG, "%s: negative size T=%lld Hq=%lld", fn, (long long)T, (long long)Hq);
    if (T > INT32_MAX || Hq > 65536) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: T=%lld or Hq=%lld too large", fn, (long long)T, (long long)Hq);
    if ((f16 != 0 && f16 != 1) || (interleaved != 0 && interleaved != 1))
        return fail(NVFP4_ERR_INVALID_ARG, "%s: f16=%d and interleaved=%d must be 0 or 1", fn, f16, interleaved);
    const int64_t D = p.cache.D;
    if (rot < 0 || rot % 2 != 0 || rot > D) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: rot=%lld must be even and at most head_dim=%lld", fn, (long long)rot, (long long)D);
    if (axes < 1 || axes > kMaxAxes) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: axes=%d must be 1 to %d", fn, axes, kMaxAxes);
    if (axes > 1 && !sections) return fail(NVFP4_ERR_INVALID_ARG, "%s: %d axes need their sections", fn, axes);
    int64_t sum = 0;
    for (int a = 0; a < axes; ++a) {
        const int64_t n = sections ? sections[a] : rot / 2;
        if (n < 0) return fail(NVFP4_ERR_INVALID_ARG, "%s: negative section", fn);
        sum += n;
        p.end[a] = (int)std::min<int64_t>(sum, kMaxHeadDim);
    }
    if (sum != rot / 2) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: the sections sum to %lld, not to rot/2=%lld", fn, (long long)sum, (long long)(rot / 2));
    if (T == 0) return NVFP4_OK;
    if ((Hq > 0 && (!q || !q_out)) || !k || !v || !positions || !slots || (rot > 0 && !table))
        return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (rot > 0 && table_rows <= 0) return fail(NVFP4_ERR_INVALID_ARG, "%s: table_rows=%lld must be positive", fn, (long long)table_rows);
    const int64_t strides[] = {q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride, v_head_stride};
    for (int64_t s : strides) {
        if (s < 0) return fail(NVFP4_ERR_INVALID_ARG, "%s: negative stride", fn);
        if (s % 8) return fail(NVFP4_ERR_ALIGNMENT, "%s: strides must be multiples of 8 elements", fn);
    }
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(table, 16) || !aligned(positions, 8) || !aligned(slots, 8))
        return fail(NVFP4_ERR_ALIGNMENT, "%s: q, k, v, q_out and table must be 16-byte aligned, positions and slots 8-byte", fn);
    // q_out may be q: a thread reads both sides of its pairs before it writes them.
    const Span to = dense_span("q_out", q_out, 2 * T * Hq * D);
    const Span qs = strided_span("q", q, 2 * D, {{T, 2 * q_token_stride}, {Hq, 2 * q_head_stride}});
    const bool in_place = q == q_out && (T == 1 || q_token_stride == Hq * D) && (Hq == 1 || q_head_stride == D);
    if (!in_place && overlaps(to, qs)) return fail(NVFP4_ERR_INVALID_ARG, "%s: q_out overlaps q (it may be q itself where that is dense)", fn);
    if (const char* in = met(to, {strided_span("k", k, 2 * D, {{T, 2 * k_token_stride}, {p.cache.heads, 2 * k_head_stride}}),
                                  strided_span("v", v, 2 * D, {{T, 2 * v_token_stride}, {p.cache.heads, 2 * v_head_stride}}),
                                  dense_span("positions", positions, 8 * axes * T), dense_span("slots", slots, 8 * T),
                                  dense_span("table", table, 4 * table_rows * rot)}))
        return fail(NVFP4_ERR_INVALID_ARG, "%s: q_out overlaps %s", fn, in);
    if (const char* part = met_cache(to, p.cache)) return fail(NVFP4_ERR_INVALID_ARG, "%s: q_out overlaps %s", fn, part);
    if (no_device(&p.status)) return fail(NVFP4_ERR_CUDA, "%s: no CUDA device", fn);
    p.q = (const uint16_t*)q; p.k = (const uint16_t*)k; p.v = (const uint16_t*)v;
    p.q_token = q_token_stride; p.q_head = q_head_stride; p.k_token = k_token_stride; p.k_head = k_head_stride;
    p.v_token = v_token_stride; p.v_head = v_head_stride;
    p.positions = positions; p.table = table; p.slots = slots; p.q_out = (uint16_t*)q_out;
    p.T = T; p.rows = table_rows; p.Hq = (int)Hq; p.Hkv = p.cache.heads; p.D = (int)D; p.rot = (int)rot; p.axes = axes;
    cudaStream_t s = (cudaStream_t)stream;
    return launch_rope(p, f16 != 0, interleaved != 0, s, fn);
}

extern "C" nvfp4_status nvfp4_kv_cache_read(const nvfp4_kv_cache* cache, const int64_t* slots, int64_t T, int f16,
                                            void* k_out, void* v_out, void* stream) {
    const char* fn = "nvfp4_kv_cache_read";
    ReadParams p{};
    if (nvfp4_status st = check_cache(fn, cache, &p.cache)) return st;
    if (T < 0) return fail(NVFP4_ERR_INVALID_ARG, "%s: negative size T=%lld", fn, (long long)T);
    if (f16 != 0 && f16 != 1) return fail(NVFP4_ERR_INVALID_ARG, "%s: f16=%d must be 0 or 1", fn, f16);
    if (T > INT32_MAX) return fail(NVFP4_ERR_UNSUPPORTED_SHAPE, "%s: T=%lld too large", fn, (long long)T);
    if (T == 0) return NVFP4_OK;
    if (!slots || !k_out || !v_out) return fail(NVFP4_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(slots, 8) || !aligned(k_out, 16) || !aligned(v_out, 16))
        return fail(NVFP4_ERR_ALIGNMENT, "%s: slots must be 8-byte aligned, k_out and v_out 16-byte", fn);
    const int64_t bytes = 2 * T * p.cache.heads * p.cache.D;
    const Span ko = dense_span("k_out", k_out, bytes), vo = dense_span("v_out", v_out, bytes);
    for (const Span& out : {ko, vo}) {
        if (overlaps(out, dense_span("slots", slots, 8 * T))) return fail(NVFP4_ERR_INVALID_ARG, "%s: %s overlaps slots", fn, out.name);
        if (const char* part = met_cache(out, p.cache)) return fail(NVFP4_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, out.name, part);
    }
    if (overlaps(ko, vo)) return fail(NVFP4_ERR_INVALID_ARG, "%s: k_out overlaps v_out", fn);
    if (no_device(&p.status)) return fail(NVFP4_ERR_CUDA, "%s: no CUDA device", fn);
    p.slots = slots; p.k_out = (uint16_t*)k_out; p.v_out = (uint16_t*)v_out; p.T = T;
    cudaStream_t s = (cudaStream_t)stream;
    const int64_t threads = T * p.cache.heads * (p.cache.D / 16);
    // Keys and values by threads of their own: 300 E4M3 tokens of 8 heads of 128 1.75 us
    // (else 2.12), 4000 5.4 (6.2), 65536 70.1 (64.6); with 16 bits 3000 4.6 (6.4), 65536 83.6 (93.6).
    const bool apart = !p.cache.e4m3 || threads <= (int64_t)sm_count() * 4096;
    const dim3 grid((unsigned)std::min<int64_t>(ceil_div(threads, 256), (int64_t)sm_count() * 16), apart ? 2 : 1);
    const void* kernel = !p.cache.e4m3 ? (const void*)cache_read_kernel<false, false>       // a copy: the type does not matter
                       : f16 ? (const void*)cache_read_kernel<true, true> : (const void*)cache_read_kernel<false, true>;
    void* args[] = {&p};
    return launch_after(kernel, grid, dim3(256), args, s, fn);
}
