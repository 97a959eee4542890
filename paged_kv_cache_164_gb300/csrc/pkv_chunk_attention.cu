// Attention of a ragged step's new tokens over a paged KV cache.
//
// The math: token i of sequence b, which brings t_b tokens to n_b, has position
// m = n_b - t_b + i and sees lo <= t < hi,
//     lo = max(0, m + 1 - window), hi = max(m + 1, min(prefix_b, n_b));
//     z_t = scale <q_i, K_t>, capped by softcap tanh(z / softcap), plus slope_h (t - m);
//     out_i = softmax(z) V over those t.
//
// The simplest form: a warp takes one (token, query head), 32 positions at a time, a
// lane a position for the scores and D / 32 columns of V for the sum.
#include <algorithm>
#include <climits>
#include <cmath>

#include "pkv_common.cuh"
#include "pkv_device.cuh"

namespace pkv {

struct ChunkParams {
    void* out;
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const int32_t* block_tables;
    const int32_t* query_starts;
    const int32_t* context_lens;
    const int32_t* prefix_lens;
    const float* slopes;
    int32_t* err_flag;
    int max_blocks_per_seq;
    int num_seqs;
    int num_tokens;
    int num_blocks;
    int block_size;
    int num_q_heads;
    int num_kv_heads;
    int group;
    int cap;
    int window;
    bool hnd;
    float scale;
    float softcap;
};

template <typename T, int D>
__global__ void __launch_bounds__(128) chunk_attention_kernel(const ChunkParams p) {
    constexpr int E = D / 32;
    __shared__ float s_q[4][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int token = blockIdx.x, h = blockIdx.y * 4 + warp;
    if (h >= p.num_q_heads) return;
    if (token == 0 && h == 0)
        for (int i = lane; i <= p.num_seqs; i += 32) {
            const int here = p.query_starts[i];
            if (here < 0 || here > p.num_tokens || (i > 0 && here < p.query_starts[i - 1]))
                flag_error(p.err_flag, PKV_EFLAG_QUERY);
        }
    int lo_b = 0, hi_b = p.num_seqs;  // the first sequence that ends behind the token
    while (lo_b < hi_b) {
        const int mid = (lo_b + hi_b) / 2;
        if (p.query_starts[mid + 1] > token)
            hi_b = mid;
        else
            lo_b = mid + 1;
    }
    const int b = lo_b;
    if (b == p.num_seqs || p.query_starts[b] > token) return;
    const int first = max(0, p.query_starts[b]);
    const int t_b = min(p.num_tokens, p.query_starts[b + 1]) - first;
    const int n_raw = p.context_lens[b], n = clamped_len(n_raw, p.cap);
    if (lane == 0 && h == 0 && (n_raw != n || n < t_b)) flag_error(p.err_flag, PKV_EFLAG_CONTEXT_LEN);
    const int m = n - t_b + token - first;
    const int prefix = p.prefix_lens != nullptr ? min(p.prefix_lens[b], n) : 0;
    const int hi = m < 0 ? 0 : max(m + 1, prefix);
    const int lo = p.window > 0 ? max(0, m + 1 - p.window) : 0;
    const T* q = static_cast<const T*>(p.q) + ((int64_t)token * p.num_q_heads + h) * D;
    for (int e = lane; e < D; e += 32) s_q[warp][e] = (float)q[e];
    __syncwarp();
    const int g = h / p.group;
    const float slope = p.slopes != nullptr ? p.slopes[h] : 0.f;
    float top = -INFINITY, sum = 0.f, acc[E] = {};
    auto row = [&](const void* cache, int t) -> const T* {
        const int blk = p.block_tables[(int64_t)b * p.max_blocks_per_seq + t / p.block_size];
        if (blk < 0 || blk >= p.num_blocks) return nullptr;
        const int off = t % p.block_size;
        return static_cast<const T*>(cache) +
               (p.hnd ? ((int64_t)blk * p.num_kv_heads + g) * p.block_size + off
                      : ((int64_t)blk * p.block_size + off) * p.num_kv_heads + g) * D;
    };
    for (int t0 = lo; t0 < hi; t0 += 32) {
        const int t = t0 + lane;
        float z = -INFINITY;
        const T* k = t < hi ? row(p.k_cache, t) : nullptr;
        if (t < hi && k == nullptr) flag_error(p.err_flag, PKV_EFLAG_BLOCK_ID);
        if (k != nullptr) {
            z = 0.f;
            for (int e = 0; e < D; e += 2) {
                const float2 x = pair_to_float2(*reinterpret_cast<const uint32_t*>(k + e), T());
                z = fmaf(s_q[warp][e], x.x, z);
                z = fmaf(s_q[warp][e + 1], x.y, z);
            }
            z *= p.scale;
            if (p.softcap > 0.f) z = p.softcap * tanhf(z / p.softcap);
            z += slope * (float)(t - m);
        }
        float mx = z;
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float next = fmaxf(top, mx);
        const float ref = next == -INFINITY ? 0.f : next;
        const float alpha = expf(top - ref), w = expf(z - ref);
        top = next;
        float ws = w;
        for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, o);
        sum = sum * alpha + ws;
        for (int e = 0; e < E; ++e) acc[e] *= alpha;
        for (int j = 0; j < 32; ++j) {
            const float wj = __shfl_sync(0xffffffffu, w, j);
            const T* v = t0 + j < hi ? row(p.v_cache, t0 + j) : nullptr;
            if (v == nullptr) continue;
            for (int e = 0; e < E; ++e) {
                const float x = (float)v[e * 32 + lane];
                // (a weight that underflows does not make an infinity that it sees a NaN)
                acc[e] = isinf(x) ? acc[e] + x : fmaf(wj, x, acc[e]);
            }
        }
    }
    T* out = static_cast<T*>(p.out) + ((int64_t)token * p.num_q_heads + h) * D;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    for (int e = 0; e < E; ++e) out[e * 32 + lane] = from_float(acc[e] * inv, T());
}

// Sizes that the workspace and the launch share.
constexpr int kChunkMaxContext = INT_MAX - 1024;  // positions of the last tile fit an int
static pkv_status check_chunk(int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads,
                              int head_dim, int block_size, int max_context_len) {
    const pkv_status st = check_shapes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                       max_context_len, 0);
    if (st != PKV_OK) return st;
    if (num_tokens < 0) return PKV_ERR_INVALID_ARG;
    if (max_context_len > kChunkMaxContext) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

template <typename T, int D>
static cudaError_t launch_chunk_t(const ChunkParams& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.num_tokens, (p.num_q_heads + 3) / 4);
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, chunk_attention_kernel<T, D>, p);
}

template <typename T>
static cudaError_t launch_chunk(const ChunkParams& p, int head_dim, cudaStream_t stream) {
    return head_dim == 64 ? launch_chunk_t<T, 64>(p, stream) : launch_chunk_t<T, 128>(p, stream);
}

}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_chunk_attention_workspace_size(int num_seqs, int num_tokens, int num_q_heads,
                                                     int num_kv_heads, int head_dim,
                                                     int block_size, int max_context_len) {
    if (check_chunk(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size,
                    max_context_len) != PKV_OK)
        return SIZE_MAX;
    return 256;
}

extern "C" pkv_status pkv_chunk_attention(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* query_starts,
    const int32_t* context_lens, int max_context_len, const int32_t* prefix_lens,
    const float* slopes, int num_seqs, int num_tokens, int num_blocks, int block_size,
    int num_q_heads, int num_kv_heads, int head_dim, float scale, float softcap, int window,
    void* workspace, size_t workspace_bytes, pkv_dtype dtype, int32_t* err_flag, void* stream) {
    const bool hnd = take_layout(dtype);
    if ((dtype != PKV_FP16 && dtype != PKV_BF16) || max_blocks_per_seq <= 0 || num_blocks <= 0 ||
        !std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f || window < 0)
        return PKV_ERR_INVALID_ARG;
    pkv_status st = check_chunk(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim,
                                block_size, max_context_len);
    if (st != PKV_OK) return st;
    if ((int64_t)max_blocks_per_seq * block_size > kChunkMaxContext) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || num_tokens == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !query_starts || !context_lens ||
        !workspace)
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
        !aligned16(workspace) ||
        ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(context_lens) |
          reinterpret_cast<uintptr_t>(query_starts) | reinterpret_cast<uintptr_t>(prefix_lens) |
          reinterpret_cast<uintptr_t>(slopes)) & 3u))
        return PKV_ERR_INVALID_ARG;
    // the output is q itself, or apart from everything that is read
    const int64_t seqs = num_seqs;
    const int64_t q_bytes = (int64_t)num_tokens * num_q_heads * head_dim * 2;
    const int64_t cache_bytes = (int64_t)num_blocks * block_size * num_kv_heads * head_dim * 2;
    const size_t need = 256;
    const auto over = [&](const void* a, int64_t bytes) {
        return a != nullptr && overlap(out, q_bytes, a, bytes);
    };
    if ((out != q && over(q, q_bytes)) || over(block_tables, seqs * max_blocks_per_seq * 4) ||
        over(context_lens, seqs * 4) || over(query_starts, (seqs + 1) * 4) ||
        over(prefix_lens, seqs * 4) || over(slopes, (int64_t)num_q_heads * 4) ||
        over(k_cache, cache_bytes) || over(v_cache, cache_bytes))
        return PKV_ERR_INVALID_ARG;
    if (workspace_bytes < need) return PKV_ERR_WORKSPACE;
    if (over(workspace, (int64_t)need)) return PKV_ERR_INVALID_ARG;
    ChunkParams p = {};
    p.out = out;
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.query_starts = query_starts;
    p.context_lens = context_lens;
    p.prefix_lens = prefix_lens;
    p.slopes = slopes;
    p.err_flag = err_flag;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = num_q_heads / num_kv_heads;
    p.cap = std::min(max_blocks_per_seq * block_size, max_context_len);
    p.window = window;
    p.hnd = hnd;
    p.scale = scale;
    p.softcap = softcap;
    cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = dtype == PKV_FP16 ? launch_chunk<__half>(p, head_dim, s)
                                            : launch_chunk<__nv_bfloat16>(p, head_dim, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}
