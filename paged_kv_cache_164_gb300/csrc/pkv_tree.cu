// A step over trees of drafted tokens: the plan (ancestor masks, rotary
// positions, cache slots) and the commit of an accepted path.  The attention of
// the nodes is in pkv_tree_attention.cu.
#include <algorithm>
#include <climits>
#include <cmath>

#include "pkv_common.cuh"
#include "pkv_device.cuh"

namespace pkv {

// ---------------------------------------------------------------------------
// The plan
// ---------------------------------------------------------------------------
// A thread per node, a CTA per kPlanRows nodes of a sequence.  A node's
// ancestors are its parent chain, whose indices fall.  The nodes of one mask word
// belong to one warp, which finds their ancestors among themselves by doubling
// (five rounds of shuffles: the bits, and the first ancestor before the word, if
// the chain is sound); then a thread hops from word to word instead of from node
// to node, and the bits it gathers count its depth.  The rows go through shared
// memory, so that their stores are dense: a row is 4 to 128 bytes.
// Latency is all it costs.  One sequence's 64 nodes: 2 us, a launch's least; 256
// sequences of 250 nodes, some 55 deep: 5.5 us a call, 4.3 in a graph of such calls.
// (A walk of the whole chain for its soundness, another for its bits, and each
// thread storing its row: 8.7 us where this form took 5.1, by the same clock.)

struct TreePlanParams {
    int32_t* tree_mask;
    int32_t* positions;
    int64_t* slot_mapping;
    const int32_t* parents;
    const int32_t* context_lens;
    const int32_t* block_tables;
    int32_t* err_flag;
    int max_blocks_per_seq;
    int cap;
    int tree_len;
    int num_blocks;
    int block_size;
};

constexpr int kPlanRows = 256;

// Shared memory: {next ancestor before the node's word, bits in its word} of each
// node, then the CTA's rows of the mask, an odd number of words apart.
static int plan_smem_bytes(int tree_len) {
    const int words = (tree_len + 31) / 32;
    return words * 32 * (int)sizeof(int2) + std::min(tree_len, kPlanRows) * (words | 1) * 4;
}

__global__ void __launch_bounds__(kPlanRows) tree_plan_kernel(const TreePlanParams p) {
    extern __shared__ int2 s_link[];
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int t = p.tree_len;
    const int words = (t + 31) / 32;
    const int parts = (t + kPlanRows - 1) / kPlanRows;
    const int b = blockIdx.x / parts;
    const int r0 = (blockIdx.x - b * parts) * kPlanRows;
    const int nrows = min(kPlanRows, t - r0);
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int i = r0 + threadIdx.x;  // this thread's node
    const int n_raw = __ldg(p.context_lens + b);
    const bool n_ok = n_raw >= t && n_raw <= p.cap;
    const int base = clamped_len(n_raw, p.cap) - t;
    const int pos = base + i;
    const int bs_shift = __ffs(p.block_size) - 1;

    // The links of the words up to the CTA's last one; a warp's last word is its
    // own (words of rows are kPlanRows / 32 apart, which is the warps of a CTA
    // where a sequence has several).
    int par = PKV_TREE_ABSENT, up = PKV_TREE_ABSENT, blk = -1;
    uint32_t bits = 0;
    for (int w = warp; w * 32 < r0 + nrows; w += warps) {
        const int node = w * 32 + lane;
        par = node < t ? __ldg(p.parents + (int64_t)b * t + node) : PKV_TREE_ABSENT;
        if (node == i && i < t && n_ok)  // (read while the links settle)
            blk = __ldg(p.block_tables + (int64_t)b * p.max_blocks_per_seq + (pos >> bs_shift));
        up = par < -1 || par >= node ? PKV_TREE_ABSENT : par;
        bits = 1u << lane;
#pragma unroll
        for (int round = 0; round < 5; ++round) {
            const uint32_t more = __shfl_sync(0xffffffffu, bits, up & 31);
            const int next = __shfl_sync(0xffffffffu, up, up & 31);
            if (up >= w * 32) {
                bits |= more;
                up = next;
            }
        }
        s_link[node] = make_int2(up, (int)bits);
    }
    __syncthreads();

    uint32_t* s_mask = reinterpret_cast<uint32_t*>(s_link + words * 32);
    if (i < t) {
        uint32_t* row = s_mask + threadIdx.x * (words | 1);
        int depth = __popc(bits) - 1;
        int w = words - 1;
        for (; w > i >> 5; --w) row[w] = 0;
        row[w--] = bits;
        while (up >= 0) {
            const int2 link = s_link[up];
            for (; w > up >> 5; --w) row[w] = 0;
            row[w--] = (uint32_t)link.y;
            depth += __popc(link.y);
            up = link.x;
        }
        for (; w >= 0; --w) row[w] = 0;
        // every link of the chain is sound: an earlier, present node, or the context
        const bool there = n_raw != 0 && up == -1;
        if (!there)
            for (w = 0; w < words; ++w) row[w] = 0;
        if (n_raw != 0 && !there && par != PKV_TREE_ABSENT)
            flag_error(p.err_flag, PKV_EFLAG_TREE);
        if (i == 0 && !n_ok && n_raw != 0) flag_error(p.err_flag, PKV_EFLAG_CONTEXT_LEN);
        const int64_t at = (int64_t)b * t + i;
        p.positions[at] = there ? max(0, base + depth) : 0;
        int64_t slot = -1;
        if (there && n_ok) {
            if (blk < 0 || blk >= p.num_blocks)
                flag_error(p.err_flag, PKV_EFLAG_BLOCK_ID);
            else
                slot = ((int64_t)blk << bs_shift) + (pos & (p.block_size - 1));
        }
        p.slot_mapping[at] = slot;
    }
    __syncthreads();
    int32_t* mask = p.tree_mask + ((int64_t)b * t + r0) * words;
    for (int k = threadIdx.x; k < nrows * words; k += blockDim.x) {
        const int r = k / words;
        mask[k] = (int32_t)s_mask[r * (words | 1) + k - r * words];
    }
}

// ---------------------------------------------------------------------------
// The commit
// ---------------------------------------------------------------------------
// Each accepted row is read once and written once.  In place and without a
// buffer: the path is strictly increasing, so path[j] >= j, and a thread that
// moves its own 16-byte column of the rows in increasing j never overwrites a
// row it still has to read (a later source path[j'] >= j' > j).  Threads share
// no bytes, so there is nothing to wait for; kMoveBatch loads are in flight
// before the first store.  Bound by memory where there is much to move, else by
// the chain of length, path, table and row.  256 sequences' 5.5 rows of 16 KB on
// average, 45.6 MB: 9.7 us, with 32 registers a thread, so that the 2048 CTAs are
// all there at once; 10.4 with 8 loads in flight and nine CTAs an SM, 11.3 and
// 13.5 where a thread moves two or four columns after one reading of the path.

struct TreeCommitParams {
    uint4* k_cache;
    uint4* v_cache;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* accepted;
    const int32_t* accepted_lens;
    int32_t* new_context_lens;  // nullable
    int32_t* err_flag;
    int max_blocks_per_seq;
    int tree_len;
    int max_accepted;
    int num_blocks;
    int block_size;
    int num_kv_heads;
    int head_vecs;              // 16-byte vectors of a head row
    int cap;
    bool hnd;
};

constexpr int kCommitThreads = 128;
constexpr int kMoveBatch = 4;
constexpr int kCommitCtas = 14;  // an SM

__global__ void __launch_bounds__(kCommitThreads, kCommitCtas)
tree_commit_kernel(const TreeCommitParams p) {
    // cache rows (slots) of the path's sources and destinations
    extern __shared__ int64_t s_src[];
    int64_t* s_dst = s_src + min(p.max_accepted, p.tree_len);
    __shared__ int s_bad;
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int b = blockIdx.y;
    const int tid = threadIdx.x;
    if (tid == 0) s_bad = 0;
    const int n_raw = __ldg(p.context_lens + b);
    const int a_raw = __ldg(p.accepted_lens + b);
    // (the first entries need not wait for the count)
    const int32_t* path = p.accepted + (int64_t)b * p.max_accepted;
    const int node0 = tid < p.max_accepted ? __ldg(path + tid) : 0;
    const int before0 = tid > 0 && tid < p.max_accepted ? __ldg(path + tid - 1) : -1;
    const int base = max(0, clamped_len(n_raw, p.cap) - p.tree_len);
    const bool n_ok = n_raw >= p.tree_len && n_raw <= p.cap;
    const bool a_ok = a_raw >= 0 && a_raw <= min(p.max_accepted, p.tree_len);
    const int a = n_ok && a_ok ? a_raw : 0;
    __syncthreads();
    int bad = 0;
    if (!n_ok && n_raw != 0) bad |= PKV_EFLAG_CONTEXT_LEN;
    if (n_raw != 0 && !a_ok) bad |= PKV_EFLAG_TREE;
    const int32_t* table = p.block_tables + (int64_t)b * p.max_blocks_per_seq;
    for (int j = tid; j < a; j += kCommitThreads) {
        const int node = j == tid ? node0 : __ldg(path + j);
        const int before = j == tid ? before0 : __ldg(path + j - 1);
        if (node <= before || node < 0 || node >= p.tree_len) {
            bad |= PKV_EFLAG_TREE;
            continue;
        }
        const int from = base + node, to = base + j;
        const int sb = __ldg(table + from / p.block_size), db = __ldg(table + to / p.block_size);
        if (sb < 0 || sb >= p.num_blocks || db < 0 || db >= p.num_blocks) {
            bad |= PKV_EFLAG_BLOCK_ID;
            continue;
        }
        s_src[j] = (int64_t)sb * p.block_size + from % p.block_size;
        s_dst[j] = (int64_t)db * p.block_size + to % p.block_size;
    }
    if (bad) atomicOr(&s_bad, bad);
    __syncthreads();
    const int fault = s_bad;
    if (blockIdx.x == 0 && tid == 0) {
        if (fault) flag_error(p.err_flag, fault);
        if (p.new_context_lens != nullptr) p.new_context_lens[b] = base + (fault ? 0 : a);
    }
    if (fault) return;

    const int row_vecs = p.num_kv_heads * p.head_vecs;
    const int c = blockIdx.x * kCommitThreads + tid;  // column of K, then of V
    if (c >= 2 * row_vecs) return;
    uint4* cache = c < row_vecs ? p.k_cache : p.v_cache;
    const int col = c < row_vecs ? c : c - row_vecs;
    const int head = col / p.head_vecs;
    auto vec = [&](int64_t slot) -> uint4* {
        if (!p.hnd) return cache + slot * row_vecs + col;
        const int64_t blk = slot / p.block_size;
        return cache + ((blk * p.num_kv_heads + head) * p.block_size + slot - blk * p.block_size) *
                           p.head_vecs + (col - head * p.head_vecs);
    };
    for (int j0 = 0; j0 < a; j0 += kMoveBatch) {
        uint4 x[kMoveBatch];
#pragma unroll
        for (int u = 0; u < kMoveBatch; ++u)
            if (j0 + u < a && s_src[j0 + u] != s_dst[j0 + u]) x[u] = *vec(s_src[j0 + u]);
#pragma unroll
        for (int u = 0; u < kMoveBatch; ++u)
            if (j0 + u < a && s_src[j0 + u] != s_dst[j0 + u]) *vec(s_dst[j0 + u]) = x[u];
    }
}

template <typename P>
static pkv_status launch_pdl(void (*kern)(const P), const P& p, dim3 grid, int threads,
                             void* stream, int smem_bytes = 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem_bytes;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_tree_plan(int32_t* tree_mask, int32_t* positions, int64_t* slot_mapping,
                                    const int32_t* parents, const int32_t* context_lens,
                                    const int32_t* block_tables, int max_blocks_per_seq,
                                    int max_context_len, int num_seqs, int tree_len,
                                    int num_blocks, int block_size, int32_t* err_flag,
                                    void* stream) {
    if (num_seqs < 0 || tree_len <= 0 || max_blocks_per_seq <= 0 || max_context_len < 0 ||
        num_blocks <= 0 || block_size <= 0)
        return PKV_ERR_INVALID_ARG;
    if (tree_len > PKV_MAX_TREE_LEN || !supported_block_size(block_size) ||
        (int64_t)max_blocks_per_seq * block_size > INT_MAX)
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!tree_mask || !positions || !slot_mapping || !parents || !context_lens || !block_tables)
        return PKV_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(tree_mask) | reinterpret_cast<uintptr_t>(positions) |
          reinterpret_cast<uintptr_t>(parents) | reinterpret_cast<uintptr_t>(context_lens) |
          reinterpret_cast<uintptr_t>(block_tables)) & 3u) ||
        (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
        return PKV_ERR_INVALID_ARG;
    // a sequence of more than kPlanRows nodes has several CTAs, which all read its
    // parents, length and table and each write their own rows
    const int64_t seqs = num_seqs, nodes = seqs * tree_len;
    const int64_t out_bytes[3] = {nodes * ((tree_len + 31) / 32) * 4, nodes * 4, nodes * 8};
    const void* outs[3] = {tree_mask, positions, slot_mapping};
    for (int i = 0; i < 3; ++i)
        if (overlap(outs[i], out_bytes[i], parents, nodes * 4) ||
            overlap(outs[i], out_bytes[i], context_lens, seqs * 4) ||
            overlap(outs[i], out_bytes[i], block_tables, seqs * max_blocks_per_seq * 4))
            return PKV_ERR_INVALID_ARG;
    TreePlanParams p = {};
    p.tree_mask = tree_mask;
    p.positions = positions;
    p.slot_mapping = slot_mapping;
    p.parents = parents;
    p.context_lens = context_lens;
    p.block_tables = block_tables;
    p.err_flag = err_flag;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.cap = std::min(max_blocks_per_seq * block_size, max_context_len);
    p.tree_len = tree_len;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    const int parts = (tree_len + kPlanRows - 1) / kPlanRows;
    if (num_seqs > INT_MAX / parts) return PKV_ERR_UNSUPPORTED;
    return launch_pdl(tree_plan_kernel, p, dim3(num_seqs * parts),
                      std::min((tree_len + 31) / 32 * 32, kPlanRows), stream,
                      plan_smem_bytes(tree_len));
}

extern "C" pkv_status pkv_tree_commit_within(
    void* k_cache, void* v_cache, const int32_t* block_tables, int max_blocks_per_seq,
    const int32_t* context_lens, int max_context_len, int tree_len, const int32_t* accepted,
    const int32_t* accepted_lens, int max_accepted, int32_t* new_context_lens, int num_seqs,
    int num_blocks, int block_size, int num_kv_heads, int head_dim, pkv_dtype dtype,
    int32_t* err_flag, void* stream) {
    const bool hnd = take_layout(dtype);
    if (num_seqs < 0 || max_context_len < 0 || tree_len <= 0 || max_accepted <= 0 || max_blocks_per_seq <= 0 ||
        num_blocks <= 0 || block_size <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        (dtype != PKV_FP16 && dtype != PKV_BF16))
        return PKV_ERR_INVALID_ARG;
    if (tree_len > PKV_MAX_TREE_LEN || !supported_block_size(block_size) ||
        !supported_head_dim(head_dim) || num_seqs > 65535 || num_kv_heads > 65535 ||
        (int64_t)max_blocks_per_seq * block_size > INT_MAX)
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!k_cache || !v_cache || !block_tables || !context_lens || !accepted || !accepted_lens)
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(k_cache) || !aligned16(v_cache) ||
        ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(context_lens) |
          reinterpret_cast<uintptr_t>(accepted) | reinterpret_cast<uintptr_t>(accepted_lens) |
          reinterpret_cast<uintptr_t>(new_context_lens)) & 3u))
        return PKV_ERR_INVALID_ARG;
    // every CTA of a sequence reads its length, its count, its path and its table, and
    // the first writes the new length when it is through with them: that goes elsewhere
    const int64_t lens_bytes = (int64_t)num_seqs * 4;
    const int64_t cache_bytes = (int64_t)num_blocks * block_size * num_kv_heads * head_dim * 2;
    const auto over = [&](const void* a, int64_t bytes) {
        return new_context_lens != nullptr && overlap(new_context_lens, lens_bytes, a, bytes);
    };
    if (over(context_lens, lens_bytes) || over(accepted_lens, lens_bytes) ||
        over(accepted, lens_bytes * max_accepted) ||
        over(block_tables, lens_bytes * max_blocks_per_seq) || over(k_cache, cache_bytes) ||
        over(v_cache, cache_bytes))
        return PKV_ERR_INVALID_ARG;
    TreeCommitParams p = {};
    p.k_cache = static_cast<uint4*>(k_cache);
    p.v_cache = static_cast<uint4*>(v_cache);
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.accepted = accepted;
    p.accepted_lens = accepted_lens;
    p.new_context_lens = new_context_lens;
    p.err_flag = err_flag;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.tree_len = tree_len;
    p.max_accepted = max_accepted;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.num_kv_heads = num_kv_heads;
    p.head_vecs = head_dim / 8;
    p.cap = std::min(max_blocks_per_seq * block_size, max_context_len);
    p.hnd = hnd;
    const int cols = 2 * num_kv_heads * p.head_vecs;
    return launch_pdl(tree_commit_kernel, p,
                      dim3((cols + kCommitThreads - 1) / kCommitThreads, num_seqs), kCommitThreads,
                      stream,
                      2 * std::min(max_accepted, tree_len) * (int)sizeof(int64_t));
}

extern "C" pkv_status pkv_tree_commit(void* k_cache, void* v_cache, const int32_t* block_tables,
                                      int max_blocks_per_seq, const int32_t* context_lens,
                                      int tree_len, const int32_t* accepted,
                                      const int32_t* accepted_lens, int max_accepted,
                                      int32_t* new_context_lens, int num_seqs, int num_blocks,
                                      int block_size, int num_kv_heads, int head_dim,
                                      pkv_dtype dtype, int32_t* err_flag, void* stream) {
    return pkv_tree_commit_within(k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                                  INT_MAX, tree_len, accepted, accepted_lens, max_accepted,
                                  new_context_lens, num_seqs, num_blocks, block_size, num_kv_heads,
                                  head_dim, dtype, err_flag, stream);
}
