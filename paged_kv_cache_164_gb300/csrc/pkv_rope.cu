// Per-head norms of queries and keys, the position rotation and the cache
// append of the new keys and values, in one pass over the projections.
//
// The math, for a head row x of head_dim values (fp32, one rounding at the end):
//     y = x * rsqrt(mean(x^2) + eps) * weight             (no weight: y = x)
//     y_a' = y_a cos - y_b sin,  y_b' = y_b cos + y_a sin  for each rotated pair
// It is bound by memory: every row is read once and written once (q to q_out,
// k and v into the cache), a few operations an element.
//
// A group of head_dim / 8 lanes holds a row in registers, 8 consecutive dims
// (one 16-byte load and store) a lane: the mean is a few shuffles inside the
// group, and a pair's other half is in the same lane (interleaved pairs) or in
// a fixed partner lane (halves).  A CTA takes rows of one token, so a lane
// reads its cosines and sines once for all of its rows.
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
    int rows_per_cta;                      // head rows (q, then k, then v) of a token per CTA
    bool interleaved;
    bool hnd;
};

constexpr int kRopeThreads = 128;

template <typename T, int D, bool F8>
__global__ void __launch_bounds__(kRopeThreads) norm_rope_append_kernel(const RopeParams p) {
    constexpr int LPR = D / 8;                    // lanes per row
    constexpr int kGroups = kRopeThreads / LPR;   // rows a CTA holds at a time
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int64_t i = blockIdx.x;
    const int64_t slot = __ldg(p.slot_mapping + i);
    if (slot < 0) return;  // padding
    const int pos = __ldg(p.positions + i);
    if (slot >= p.num_slots || pos < 0 || pos >= p.max_position) {
        if (threadIdx.x == 0 && blockIdx.y == 0)
            flag_error(p.err_flag, (slot >= p.num_slots ? PKV_EFLAG_SLOT : 0) |
                                       (pos < 0 || pos >= p.max_position ? PKV_EFLAG_POSITION : 0));
        return;
    }
    const int lane = threadIdx.x % LPR;
    const int group = threadIdx.x / LPR;
    const int half = p.rotary_dim / 2;
    const int e0 = lane * 8;                      // this lane's first dim
    const bool turns = e0 < p.rotary_dim;

    // this lane's cosines and sines: of dims e0.. (halves: 8 of each, the same
    // for both halves), or of the 4 pairs that start at e0
    float cs[8], sn[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        cs[u] = 1.f;
        sn[u] = 0.f;
    }
    if (turns) {
        const float* row = p.cos_sin + (int64_t)pos * p.rotary_dim;
        const int j0 = p.interleaved ? e0 / 2 : (e0 < half ? e0 : e0 - half);
#pragma unroll
        for (int u = 0; u < 8; u += 4) {
            if (u >= 4 && p.interleaved) break;
            const float4 c = __ldg(reinterpret_cast<const float4*>(row + j0 + u));
            const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + j0 + u));
            cs[u] = c.x; cs[u + 1] = c.y; cs[u + 2] = c.z; cs[u + 3] = c.w;
            sn[u] = s.x; sn[u + 1] = s.y; sn[u + 2] = s.z; sn[u + 3] = s.w;
        }
    }
    const int partner = e0 < half ? lane + half / 8 : lane - half / 8;

    const int rows = p.num_q_heads + 2 * p.num_kv_heads;
    const int r_end = min(rows, (int)(blockIdx.y + 1) * p.rows_per_cta);
    const int r_begin = blockIdx.y * p.rows_per_cta;
    const int64_t blk = slot / p.block_size;
    const int off = (int)(slot - blk * p.block_size);
    // whole warps stay in the loop (the shuffles name all lanes)
    for (int base = r_begin; base < r_end; base += kGroups) {
        const int r = base + group;
        const bool live = r < r_end;
        const bool is_q = r < p.num_q_heads;
        const bool is_v = r >= p.num_q_heads + p.num_kv_heads;
        const int head = is_q ? r : is_v ? r - p.num_q_heads - p.num_kv_heads : r - p.num_q_heads;
        const T* src = static_cast<const T*>(is_q ? p.q : is_v ? p.v : p.k) +
                       i * (is_q ? p.q_stride : is_v ? p.v_stride : p.k_stride) + head * D + e0;
        uint4 raw = make_uint4(0u, 0u, 0u, 0u);
        if (live) raw = *reinterpret_cast<const uint4*>(src);
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
        float x[8];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float2 f = pair_to_float2(w[u], T());
            x[2 * u] = f.x;
            x[2 * u + 1] = f.y;
        }
        float sq = 0.f;
#pragma unroll
        for (int u = 0; u < 8; ++u) sq = fmaf(x[u], x[u], sq);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o, LPR);
        const void* weight = is_q ? p.q_weight : is_v ? nullptr : p.k_weight;
        if (weight != nullptr) {
            const float inv = rsqrtf(sq * (1.f / D) + p.eps);
            const uint4 wr = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(weight) + e0));
            const uint32_t ww[4] = {wr.x, wr.y, wr.z, wr.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float2 f = pair_to_float2(ww[u], T());
                x[2 * u] = x[2 * u] * inv * f.x;
                x[2 * u + 1] = x[2 * u + 1] * inv * f.y;
            }
        }
        if (p.interleaved) {
            if (!is_v) {
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float a = x[2 * u], b = x[2 * u + 1];
                    x[2 * u] = a * cs[u] - b * sn[u];
                    x[2 * u + 1] = b * cs[u] + a * sn[u];
                }
            }
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float other = __shfl_sync(0xffffffffu, x[u], partner, LPR);
                if (turns && !is_v)
                    x[u] = e0 < half ? x[u] * cs[u] - other * sn[u] : x[u] * cs[u] + other * sn[u];
            }
        }
        if (!live) continue;
        if (is_q || !F8) {
            uint4 y;
            y.x = pack2(x[0], x[1], T());
            y.y = pack2(x[2], x[3], T());
            y.z = pack2(x[4], x[5], T());
            y.w = pack2(x[6], x[7], T());
            if (is_v) y = raw;  // bit-exact, NaN payloads included
            T* dst;
            if (is_q)
                dst = static_cast<T*>(p.q_out) + (i * p.num_q_heads + head) * D + e0;
            else
                dst = static_cast<T*>(is_v ? p.v_cache : p.k_cache) +
                      (p.hnd ? (blk * p.num_kv_heads + head) * p.block_size + off
                             : slot * p.num_kv_heads + head) * D + e0;
            *reinterpret_cast<uint4*>(dst) = y;
        } else {
            const float sc = is_v ? p.v_scale : p.k_scale;
            uint32_t codes[2] = {0u, 0u};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float2 f = make_float2(__fdiv_rn(x[2 * u], sc), __fdiv_rn(x[2 * u + 1], sc));
                const uint32_t two = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
                codes[u / 2] |= two << (16 * (u % 2));
            }
            uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) +
                           (p.hnd ? (blk * p.num_kv_heads + head) * p.block_size + off
                                  : slot * p.num_kv_heads + head) * D + e0;
            *reinterpret_cast<uint2*>(dst) = make_uint2(codes[0], codes[1]);
        }
    }
}

template <typename T, int D, bool F8>
static cudaError_t launch_rope(RopeParams p, int num_tokens, int sms, cudaStream_t stream) {
    constexpr int kGroups = kRopeThreads / (D / 8);
    const int rows = p.num_q_heads + 2 * p.num_kv_heads;
    // Enough CTAs for about eight an SM; then each takes more of a token's rows.
    const int passes = (rows + kGroups - 1) / kGroups;  // CTAs of one row a group
    const int64_t want = std::max<int64_t>(1, (int64_t)sms * 8 / num_tokens);
    const int splits = (int)std::min<int64_t>(passes, want);
    p.rows_per_cta = (passes + splits - 1) / splits * kGroups;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_tokens, (rows + p.rows_per_cta - 1) / p.rows_per_cta);
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, norm_rope_append_kernel<T, D, F8>, p);
}

// Whether [a, a + an) and [b, b + bn) share a byte.
static bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
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
    const int sms = current_sm_count();
    if (sms <= 0) return PKV_ERR_CUDA;
    p.num_slots = (int64_t)num_blocks * bs;
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
