// Per-head norms of queries and keys, the position rotation and the cache
// append of the new keys and values, in one pass over the projections.
//
// The math, for a head row x of head_dim values (fp32, one rounding at the end):
//     y = x * rsqrt(mean(x^2) + eps) * weight             (no weight: y = x)
//     y_a' = y_a cos - y_b sin,  y_b' = y_b cos + y_a sin  for each rotated pair
// It is bound by memory: every row is read once and written once (q to q_out,
// k and v into the cache), a few operations an element.  16411 packed tokens of
// the Llama-7B layer (815 MB) take 125 us, 6.5 TB/s (96 % of the copy rate);
// 2043 tokens of the Llama-70B layer (80 MB) 18.4 us into E4M3 pages, 17.7 us into
// 16-bit ones, 1.55 and 1.44 times their bytes at that rate: 6129 CTAs, four and a
// half waves of them, each of which loads, waits and stores once; 32 tokens 2 us, a
// launch's least.
//
// A group of head_dim / 8 lanes takes a row, two blocks of 4 dims a
// lane, chosen so that a lane has both halves of its pairs (halves: 4 l and
// rotary_dim / 2 + 4 l; interleaved pairs and dims that are not rotated: 8 l
// and 8 l + 4): the rotation needs no exchange between lanes, and the mean is
// the group's only one.  A CTA takes rows of one token, of q or of k and v, so a
// lane reads its cosines, sines and weights once for all of its rows.
#include <algorithm>
#include <climits>
#include <cmath>

#include <cuda_fp8.h>

#include "pkv_common.cuh"
#include "pkv_device.cuh"

namespace pkv {

struct RopeParams {
    void* q_out;
    const void* q;
    const void* k;
    const void* v;
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    const void* q_weight;                  // nullable
    const void* k_weight;                  // nullable
    const float* cos_sin;                  // [max_position][rotary_dim]
    const int32_t* positions;
    void* k_cache;
    void* v_cache;
    const int64_t* slot_mapping;
    int64_t num_slots;
    int32_t* err_flag;
    float eps;
    float k_scale, v_scale;                // E4M3 caches
    int max_position;
    int rotary_dim;
    int num_q_heads, num_kv_heads;
    int block_size;
    int block_shift;                       // log2 of the block size
    int rows_per_cta;                      // head rows of a token per CTA
    int q_blocks;                          // CTAs of a token with q rows; then k and v rows
    bool interleaved;
    bool hnd;
};

constexpr int kRopeThreads = 128;
// A group's rows, all in flight at once, and the CTAs an SM that the registers
// leave room for.  The rows come by cp.async: held in registers as plain loads
// they leave seven or eight CTAs an SM.  16411 packed tokens of the Llama-7B layer
// and 2043 tokens of the Llama-70B layer into E4M3 pages: 124 and 18.3 us (plain
// loads: 130 and 20.6); for 8, 10 and 12 CTAs 124 and 18.7, 128 and 17.8, 122 and
// 19.2; with 2 and 8 rows 139 and 19.1, 131 and 19.6.
constexpr int kRopeBatch = 4;
constexpr int kRopeCtas = 9;
// CTAs an SM below which a group takes fewer rows: 32 tokens of the Llama-70B
// layer 2.0 us, with four rows a group all the same 2.3 us.
constexpr int kRopeMinCtas = 8;

template <typename T>
__device__ __forceinline__ void widen4(uint2 w, float2 (&x)[2], T) {
    x[0] = pair_to_float2(w.x, T());
    x[1] = pair_to_float2(w.y, T());
}

template <typename T, int D, bool F8, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas)
norm_rope_append_kernel(const RopeParams p) {
    constexpr int LPR = D / 8;                    // lanes per row
    constexpr int kGroups = kRopeThreads / LPR;   // rows a CTA holds at a time
    __shared__ uint4 s_rows[kRopeBatch][kGroups][LPR];
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int64_t i = blockIdx.x;
    const int lane = threadIdx.x % LPR;
    const int group = threadIdx.x / LPR;
    const int half = p.rotary_dim / 2;
    const bool turns = lane * 8 < p.rotary_dim;
    // the lane's two blocks of 4 dims
    const int d0 = !INTER && turns ? 4 * lane : 8 * lane;
    const int d1 = !INTER && turns ? half + 4 * lane : 8 * lane + 4;
    const bool kv = (int)blockIdx.y >= p.q_blocks;  // k, then v rows; else q rows
    const int first = (kv ? blockIdx.y - p.q_blocks : blockIdx.y) * p.rows_per_cta;
    const int r_end = min(kv ? 2 * p.num_kv_heads : p.num_q_heads, first + p.rows_per_cta);
    const int r0 = first + group;

    // every load that depends on no other first: the slot, the position, the
    // group's rows
    const int64_t slot = __ldg(p.slot_mapping + i);
    const int pos = __ldg(p.positions + i);
    const T* qk = static_cast<const T*>(kv ? p.k : p.q) + i * (kv ? p.k_stride : p.q_stride);
    const T* vv = static_cast<const T*>(p.v) + i * p.v_stride - (int64_t)p.num_kv_heads * D;
#pragma unroll
    for (int u = 0; u < kRopeBatch; ++u) {
        const int r = r0 + u * kGroups;
        if (r < r_end)
            ptx::cp_async_16(ptx::smem_addr(&s_rows[u][group][lane]),
                             (kv && r >= p.num_kv_heads ? vv : qk) + r * D + 8 * lane, true);
    }
    const T* weight = static_cast<const T*>(kv ? p.k_weight : p.q_weight);
    float2 wl[2], wh[2];
    wl[0] = wl[1] = wh[0] = wh[1] = make_float2(1.f, 1.f);
    if (weight != nullptr) {
        widen4(__ldg(reinterpret_cast<const uint2*>(weight + d0)), wl, T());
        widen4(__ldg(reinterpret_cast<const uint2*>(weight + d1)), wh, T());
    }
    if (slot < 0) {  // padding
        ptx::cp_async_wait_all();
        return;
    }
    if (slot >= p.num_slots || pos < 0 || pos >= p.max_position) {
        ptx::cp_async_wait_all();
        if (threadIdx.x == 0 && blockIdx.y == 0)
            flag_error(p.err_flag, (slot >= p.num_slots ? PKV_EFLAG_SLOT : 0) |
                                       (pos < 0 || pos >= p.max_position ? PKV_EFLAG_POSITION : 0));
        return;
    }
    // the lane's 4 pairs' cosines and sines
    float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (turns && !(kv && first >= p.num_kv_heads)) {
        const float* row = p.cos_sin + (int64_t)pos * p.rotary_dim + 4 * lane;
        c = __ldg(reinterpret_cast<const float4*>(row));
        s = __ldg(reinterpret_cast<const float4*>(row + half));
    }
    const int64_t blk = slot >> p.block_shift;
    const int off = (int)(slot & ((1 << p.block_shift) - 1));
    // elements from a head's row to the next head's in the cache, and the first
    const int64_t head_step = (p.hnd ? (int64_t)1 << p.block_shift : 1) * D;
    const int64_t cell0 =
        p.hnd ? (((blk * p.num_kv_heads) << p.block_shift) + off) * D : slot * p.num_kv_heads * D;
    ptx::cp_async_wait_all();
    __syncwarp();
#pragma unroll 1
    for (int u = 0; u < kRopeBatch; ++u) {
        const int r = r0 + u * kGroups;
        if (r - group >= r_end) break;  // the same for the whole CTA
        const T* row_in = reinterpret_cast<const T*>(s_rows[u][group]);
        const uint2 lo = *reinterpret_cast<const uint2*>(row_in + d0);
        const uint2 hi = *reinterpret_cast<const uint2*>(row_in + d1);
        const bool is_v = kv && r >= p.num_kv_heads;
        float2 x[2], y[2];  // the blocks at d0 and d1
        widen4(lo, x, T());
        widen4(hi, y, T());
        if (weight != nullptr && !(kv && r - group >= p.num_kv_heads)) {
            // (whole warps take part in the shuffles)
            float2 q = ptx::mul2(x[0], x[0]);
            q = ptx::fma2(x[1], x[1], q);
            q = ptx::fma2(y[0], y[0], q);
            q = ptx::fma2(y[1], y[1], q);
            float sq = q.x + q.y;
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o, LPR);
            if (!is_v) {
                const float inv = rsqrtf(sq * (1.f / D) + p.eps);
                const float2 inv2 = make_float2(inv, inv);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    x[e] = ptx::mul2(ptx::mul2(x[e], inv2), wl[e]);
                    y[e] = ptx::mul2(ptx::mul2(y[e], inv2), wh[e]);
                }
            }
        }
        if (turns && !is_v) {
            if constexpr (INTER) {
                // pairs (x, y) of each float2: a cos - b sin, b cos + a sin
                auto turn = [](float2 v, float cc, float ss) {
                    return make_float2(v.x * cc - v.y * ss, v.y * cc + v.x * ss);
                };
                x[0] = turn(x[0], c.x, s.x);
                x[1] = turn(x[1], c.y, s.y);
                y[0] = turn(y[0], c.z, s.z);
                y[1] = turn(y[1], c.w, s.w);
            } else {
                // pairs (x element, y element)
                const float2 cc[2] = {make_float2(c.x, c.y), make_float2(c.z, c.w)};
                const float2 ss[2] = {make_float2(s.x, s.y), make_float2(s.z, s.w)};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float2 a = x[e], b = y[e];
                    x[e] = ptx::fma2(make_float2(-b.x, -b.y), ss[e], ptx::mul2(a, cc[e]));
                    y[e] = ptx::fma2(a, ss[e], ptx::mul2(b, cc[e]));
                }
            }
        }
        if (r >= r_end) continue;
        if (!kv || !F8) {
            uint2 out0 = lo, out1 = hi;  // v: bit-exact, NaN payloads included
            if (!is_v) {
                out0 = make_uint2(pack2(x[0].x, x[0].y, T()), pack2(x[1].x, x[1].y, T()));
                out1 = make_uint2(pack2(y[0].x, y[0].y, T()), pack2(y[1].x, y[1].y, T()));
            }
            T* dst = !kv ? static_cast<T*>(p.q_out) + (i * p.num_q_heads + r) * D
                   : is_v ? static_cast<T*>(p.v_cache) + cell0 + (r - p.num_kv_heads) * head_step
                          : static_cast<T*>(p.k_cache) + cell0 + r * head_step;
            if constexpr (INTER) {
                *reinterpret_cast<uint4*>(dst + d0) = make_uint4(out0.x, out0.y, out1.x, out1.y);
            } else {
                *reinterpret_cast<uint2*>(dst + d0) = out0;
                *reinterpret_cast<uint2*>(dst + d1) = out1;
            }
        } else {
            const float sc = is_v ? p.v_scale : p.k_scale;
            auto code4 = [sc](const float2 (&v)[2]) {
                const uint32_t a = __nv_cvt_float2_to_fp8x2(
                    make_float2(__fdiv_rn(v[0].x, sc), __fdiv_rn(v[0].y, sc)), __NV_SATFINITE,
                    __NV_E4M3);
                const uint32_t b = __nv_cvt_float2_to_fp8x2(
                    make_float2(__fdiv_rn(v[1].x, sc), __fdiv_rn(v[1].y, sc)), __NV_SATFINITE,
                    __NV_E4M3);
                return a | (b << 16);
            };
            uint8_t* dst =
                is_v ? static_cast<uint8_t*>(p.v_cache) + cell0 + (r - p.num_kv_heads) * head_step
                     : static_cast<uint8_t*>(p.k_cache) + cell0 + r * head_step;
            *reinterpret_cast<uint32_t*>(dst + d0) = code4(x);
            *reinterpret_cast<uint32_t*>(dst + d1) = code4(y);
        }
    }
}

template <typename T, int D, bool F8, bool INTER>
static cudaError_t launch_rope_t(const RopeParams& p, dim3 grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_rope_append_kernel<T, D, F8, INTER>, p);
}

template <typename T, int D, bool F8>
static cudaError_t launch_rope(RopeParams p, int num_tokens, int sms, cudaStream_t stream) {
    constexpr int kGroups = kRopeThreads / (D / 8);
    // As many rows a group as leave kRopeMinCtas CTAs an SM: few tokens spread over
    // the SMs, many share a token's cosines among more rows.
    auto blocks = [](int batch, int rows) {
        return (rows + batch * kGroups - 1) / (batch * kGroups);
    };
    const int kv_rows = 2 * p.num_kv_heads;
    int batch = kRopeBatch;
    while (batch > 1 &&
           (int64_t)num_tokens * (blocks(batch, p.num_q_heads) + blocks(batch, kv_rows)) <
               (int64_t)sms * kRopeMinCtas)
        batch /= 2;
    p.rows_per_cta = batch * kGroups;
    p.q_blocks = blocks(batch, p.num_q_heads);
    const dim3 grid(num_tokens, p.q_blocks + blocks(batch, kv_rows));
    return p.interleaved ? launch_rope_t<T, D, F8, true>(p, grid, stream)
                         : launch_rope_t<T, D, F8, false>(p, grid, stream);
}

static pkv_status norm_rope_impl(RopeParams p, int num_tokens, int num_blocks, int head_dim,
                                 pkv_dtype dtype, bool f8, void* stream) {
    p.hnd = take_layout(dtype);
    const int hq = p.num_q_heads, hkv = p.num_kv_heads, bs = p.block_size;
    if (num_tokens < 0 || num_blocks <= 0 || bs <= 0 || hq <= 0 || hkv <= 0 || head_dim <= 0 ||
        (dtype != PKV_FP16 && dtype != PKV_BF16) || !std::isfinite(p.eps) || p.eps < 0.f ||
        p.max_position <= 0 || hq % hkv != 0)
        return PKV_ERR_INVALID_ARG;
    if (f8 && (!std::isfinite(p.k_scale) || !std::isfinite(p.v_scale) || p.k_scale <= 0.f ||
               p.v_scale <= 0.f))
        return PKV_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim) || !supported_block_size(bs) || hq > 65535 || hkv > 65535)
        return PKV_ERR_UNSUPPORTED;
    if (p.rotary_dim < 16 || p.rotary_dim > head_dim || p.rotary_dim % 16 != 0)
        return PKV_ERR_UNSUPPORTED;
    if (p.q_stride < (int64_t)hq * head_dim || p.k_stride < (int64_t)hkv * head_dim ||
        p.v_stride < (int64_t)hkv * head_dim || p.q_stride % 8 || p.k_stride % 8 || p.v_stride % 8)
        return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    if (!p.q_out || !p.q || !p.k || !p.v || !p.cos_sin || !p.positions || !p.k_cache ||
        !p.v_cache || !p.slot_mapping)
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(p.q_out) || !aligned16(p.q) || !aligned16(p.k) || !aligned16(p.v) ||
        !aligned16(p.q_weight) || !aligned16(p.k_weight) || !aligned16(p.cos_sin) ||
        !aligned16(p.k_cache) || !aligned16(p.v_cache) ||
        (reinterpret_cast<uintptr_t>(p.positions) & 3u) ||
        (reinterpret_cast<uintptr_t>(p.slot_mapping) & 7u))
        return PKV_ERR_INVALID_ARG;
    // q_out is q itself, row for row, or apart from everything that is read:
    // a row is read whole before it is written, but rows have no order.
    const int64_t last = num_tokens - 1;
    const int64_t q_bytes = (last * p.q_stride + (int64_t)hq * head_dim) * 2;
    const int64_t out_bytes = (int64_t)num_tokens * hq * head_dim * 2;
    const bool in_place = p.q_out == p.q && p.q_stride == (int64_t)hq * head_dim;
    if ((!in_place && overlap(p.q_out, out_bytes, p.q, q_bytes)) ||
        overlap(p.q_out, out_bytes, p.k, (last * p.k_stride + (int64_t)hkv * head_dim) * 2) ||
        overlap(p.q_out, out_bytes, p.v, (last * p.v_stride + (int64_t)hkv * head_dim) * 2))
        return PKV_ERR_INVALID_ARG;
    const int64_t cache_bytes = (int64_t)num_blocks * bs * hkv * head_dim * (f8 ? 1 : 2);
    const auto over = [&](const void* a, int64_t bytes) {
        return a != nullptr && overlap(p.q_out, out_bytes, a, bytes);
    };
    if (over(p.q_weight, head_dim * 2) || over(p.k_weight, head_dim * 2) ||
        over(p.cos_sin, (int64_t)p.max_position * p.rotary_dim * 4) ||
        over(p.positions, (int64_t)num_tokens * 4) ||
        over(p.slot_mapping, (int64_t)num_tokens * 8) || over(p.k_cache, cache_bytes) ||
        over(p.v_cache, cache_bytes))
        return PKV_ERR_INVALID_ARG;
    const int sms = current_sm_count();
    if (sms <= 0) return PKV_ERR_CUDA;
    p.num_slots = (int64_t)num_blocks * bs;
    p.block_shift = 0;
    while ((1 << p.block_shift) < bs) ++p.block_shift;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    const bool half = dtype == PKV_FP16;
    if (head_dim == 64)
        e = half ? (f8 ? launch_rope<__half, 64, true>(p, num_tokens, sms, s)
                       : launch_rope<__half, 64, false>(p, num_tokens, sms, s))
                 : (f8 ? launch_rope<__nv_bfloat16, 64, true>(p, num_tokens, sms, s)
                       : launch_rope<__nv_bfloat16, 64, false>(p, num_tokens, sms, s));
    else
        e = half ? (f8 ? launch_rope<__half, 128, true>(p, num_tokens, sms, s)
                       : launch_rope<__half, 128, false>(p, num_tokens, sms, s))
                 : (f8 ? launch_rope<__nv_bfloat16, 128, true>(p, num_tokens, sms, s)
                       : launch_rope<__nv_bfloat16, 128, false>(p, num_tokens, sms, s));
    if (e != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_norm_rope_append(
    void* q_out, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
    int64_t v_stride, const void* q_weight, const void* k_weight, float eps, const float* cos_sin,
    int max_position, int rotary_dim, int interleaved, const int32_t* positions, void* k_cache,
    void* v_cache, const int64_t* slot_mapping, int num_tokens, int num_blocks, int block_size,
    int num_q_heads, int num_kv_heads, int head_dim, pkv_dtype dtype, int32_t* err_flag,
    void* stream) {
    RopeParams p = {};
    p.q_out = q_out;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_weight = q_weight;
    p.k_weight = k_weight;
    p.eps = eps;
    p.cos_sin = cos_sin;
    p.max_position = max_position;
    p.rotary_dim = rotary_dim;
    p.interleaved = interleaved != 0;
    p.positions = positions;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.slot_mapping = slot_mapping;
    p.block_size = block_size;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.err_flag = err_flag;
    p.k_scale = p.v_scale = 1.f;
    return norm_rope_impl(p, num_tokens, num_blocks, head_dim, dtype, false, stream);
}

extern "C" pkv_status pkv_norm_rope_append_fp8(
    void* q_out, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
    int64_t v_stride, const void* q_weight, const void* k_weight, float eps, const float* cos_sin,
    int max_position, int rotary_dim, int interleaved, const int32_t* positions, void* k_cache,
    void* v_cache, const int64_t* slot_mapping, int num_tokens, int num_blocks, int block_size,
    int num_q_heads, int num_kv_heads, int head_dim, float k_scale, float v_scale, pkv_dtype dtype,
    int32_t* err_flag, void* stream) {
    RopeParams p = {};
    p.q_out = q_out;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_weight = q_weight;
    p.k_weight = k_weight;
    p.eps = eps;
    p.cos_sin = cos_sin;
    p.max_position = max_position;
    p.rotary_dim = rotary_dim;
    p.interleaved = interleaved != 0;
    p.positions = positions;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.slot_mapping = slot_mapping;
    p.block_size = block_size;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.err_flag = err_flag;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    return norm_rope_impl(p, num_tokens, num_blocks, head_dim, dtype, true, stream);
}
