// Attention of a tree's drafted nodes over a paged KV cache.
//
// The math: node i of sequence b attends to the committed positions
// t < base = n - tree_len and to the nodes j (position base + j) of its mask:
//     s_t = scale * <q_i, K_t>,  out_i = softmax(s) V      over those t
// with the online softmax (running maximum m, sum l, accumulator O; one
// division at the end).
#include <algorithm>
#include <climits>
#include <cmath>

#include "pkv_common.cuh"
#include "pkv_device.cuh"

namespace pkv {

struct TreeParams {
    void* out;
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* tree_mask;
    int64_t mask_stride;
    int32_t* err_flag;
    int max_blocks_per_seq;
    int num_blocks;
    int block_size;
    int num_q_heads;
    int num_kv_heads;
    int tree_len;
    int cap;
    bool hnd;
    float scale_log2;
};

constexpr int kTreeWarps = 4;

// One CTA per (query head, node, sequence): its warps take every fourth
// token, D / 32 dims a lane, and meet at the end.
template <typename T, int D>
__global__ void __launch_bounds__(kTreeWarps * 32) tree_attention_kernel(const TreeParams p) {
    constexpr int E = D / 32;
    __shared__ float s_o[kTreeWarps][D];
    __shared__ float s_m[kTreeWarps], s_l[kTreeWarps];
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int h = blockIdx.x, i = blockIdx.y, b = blockIdx.z;
    const int g = h / (p.num_q_heads / p.num_kv_heads);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n_raw = __ldg(p.context_lens + b);
    if (h == 0 && i == 0 && threadIdx.x == 0 &&
        (n_raw < 0 || n_raw > p.cap || (n_raw != 0 && n_raw < p.tree_len)))
        flag_error(p.err_flag, PKV_EFLAG_CONTEXT_LEN);
    const int n = clamped_len(n_raw, p.cap);
    const int base = n - p.tree_len;
    const int64_t row = ((int64_t)b * p.tree_len + i) * p.num_q_heads + h;
    float q[E], o[E];
    load_as_float<T, E>(static_cast<const T*>(p.q) + row * D + lane * E, q);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    float m = -INFINITY, l = 0.f;
    const int32_t* mask = p.tree_mask + b * p.mask_stride + (int64_t)i * ((p.tree_len + 31) / 32);
    for (int t = warp; t < n; t += kTreeWarps) {
        const int j = t - base;
        if (j >= 0 && !((__ldg(mask + (j >> 5)) >> (j & 31)) & 1)) continue;
        const int blk = __ldg(p.block_tables + (int64_t)b * p.max_blocks_per_seq + t / p.block_size);
        if (blk < 0 || blk >= p.num_blocks) {
            if (lane == 0) flag_error(p.err_flag, PKV_EFLAG_BLOCK_ID);
            continue;
        }
        const int off = t % p.block_size;
        const int64_t at =
            (p.hnd ? ((int64_t)blk * p.num_kv_heads + g) * p.block_size + off
                   : ((int64_t)blk * p.block_size + off) * p.num_kv_heads + g) * D + lane * E;
        float k[E], v[E];
        load_as_float<T, E>(static_cast<const T*>(p.k_cache) + at, k);
        load_as_float<T, E>(static_cast<const T*>(p.v_cache) + at, v);
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= p.scale_log2;
        const float mn = fmaxf(m, s);
        const float alpha = exp2f(m - mn), w = exp2f(s - mn);
        m = mn;
        l = l * alpha + w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(w, v[e], o[e] * alpha);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
    __syncthreads();
    float mx = -INFINITY;
    for (int w = 0; w < kTreeWarps; ++w) mx = fmaxf(mx, s_m[w]);
    for (int d = threadIdx.x; d < D; d += kTreeWarps * 32) {
        float num = 0.f, den = 0.f;
        for (int w = 0; w < kTreeWarps; ++w) {
            const float f = s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - mx);
            if (f != 0.f) {
                num = fmaf(f, s_o[w][d], num);
                den = fmaf(f, s_l[w], den);
            }
        }
        static_cast<T*>(p.out)[row * D + d] = from_float(den == 0.f ? 0.f : num / den, T());
    }
}

// Arguments that the workspace size and the launch share.
static pkv_status check_tree(int num_seqs, int tree_len, int num_q_heads, int num_kv_heads,
                             int head_dim, int block_size, int max_context_len) {
    const pkv_status st = check_shapes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                       max_context_len, 0);
    if (st != PKV_OK) return st;
    if (tree_len <= 0) return PKV_ERR_INVALID_ARG;
    if (tree_len > PKV_MAX_TREE_LEN || (int64_t)num_seqs * num_kv_heads > 65535)
        return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_tree_attention_workspace_size(int num_seqs, int tree_len, int num_q_heads,
                                                    int num_kv_heads, int head_dim,
                                                    int block_size, int max_context_len) {
    if (check_tree(num_seqs, tree_len, num_q_heads, num_kv_heads, head_dim, block_size,
                   max_context_len) != PKV_OK)
        return SIZE_MAX;
    return 256;
}

extern "C" pkv_status pkv_tree_attention(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens,
    int max_context_len, const int32_t* tree_mask, int64_t mask_stride, int num_seqs, int tree_len,
    int num_blocks, int block_size, int num_q_heads, int num_kv_heads, int head_dim, float scale,
    void* workspace, size_t workspace_bytes, pkv_dtype dtype, int32_t* err_flag, void* stream) {
    const bool hnd = take_layout(dtype);
    if ((dtype != PKV_FP16 && dtype != PKV_BF16) || max_blocks_per_seq <= 0 || num_blocks <= 0 ||
        !std::isfinite(scale))
        return PKV_ERR_INVALID_ARG;
    const pkv_status st = check_tree(num_seqs, tree_len, num_q_heads, num_kv_heads, head_dim,
                                     block_size, max_context_len);
    if (st != PKV_OK) return st;
    const int64_t mask_words = (int64_t)tree_len * ((tree_len + 31) / 32);
    if (mask_stride != 0 && mask_stride < mask_words) return PKV_ERR_INVALID_ARG;
    if (num_seqs == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !tree_mask ||
        !workspace)
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
        !aligned16(workspace) ||
        ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(context_lens) |
          reinterpret_cast<uintptr_t>(tree_mask)) & 3u))
        return PKV_ERR_INVALID_ARG;
    if ((int64_t)max_blocks_per_seq * block_size > INT_MAX) return PKV_ERR_UNSUPPORTED;
    if (workspace_bytes < 256) return PKV_ERR_WORKSPACE;

    TreeParams p = {};
    p.out = out;
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.tree_mask = tree_mask;
    p.mask_stride = mask_stride;
    p.err_flag = err_flag;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.tree_len = tree_len;
    p.cap = std::min(max_blocks_per_seq * block_size, max_context_len);
    p.hnd = hnd;
    p.scale_log2 = scale * kLog2e;
    cudaStream_t s = (cudaStream_t)stream;
    const dim3 grid(num_q_heads, tree_len, num_seqs);
    if (head_dim == 64) {
        if (dtype == PKV_FP16)
            tree_attention_kernel<__half, 64><<<grid, kTreeWarps * 32, 0, s>>>(p);
        else
            tree_attention_kernel<__nv_bfloat16, 64><<<grid, kTreeWarps * 32, 0, s>>>(p);
    } else {
        if (dtype == PKV_FP16)
            tree_attention_kernel<__half, 128><<<grid, kTreeWarps * 32, 0, s>>>(p);
        else
            tree_attention_kernel<__nv_bfloat16, 128><<<grid, kTreeWarps * 32, 0, s>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
