// Verification of drafted tokens: the accepted path of a chain or a tree, and the
// token drawn from what is left of the target's distribution.
#include <algorithm>
#include <climits>

#include "pkv_common.cuh"
#include "pkv_device.cuh"

namespace pkv {

// ---------------------------------------------------------------------------
// The math: at a node with target row p and draft row q the children are tried in
// order, with what earlier ones left of p (unnormalised):
//     R_0 = p, Z_0 = 1;  child of token x and number u: accepted if u q(x) Z_j < R_j(x),
//     else R_{j+1} = max(R_j - Z_j q, 0), Z_{j+1} = sum R_{j+1}
// A child that is accepted starts anew with its own rows; the next token is drawn
// from R where no child was.  A node comes behind its parent, so one walk over the
// nodes in order meets all of it.  Every value that the first test of a node takes is
// known beforehand and fetched by a thread a node; a pass over the vocabulary is made
// only where a child is rejected, and the last one's sums already say where the next
// token lies.
// Sums: 64-bit whole numbers of 2^-60, so that they are the same in any order and a
// draw at a border does not depend on the split of the work (a sum in fp32 is off by
// more than the probability of a token of a flat distribution).
// ---------------------------------------------------------------------------

struct VerifyParams {
    int32_t* accepted;
    int32_t* accepted_lens;
    int32_t* next_tokens;
    int32_t* new_context_lens;
    const float* target;
    const float* draft;
    const int32_t* tokens;
    const int32_t* parents;
    const int32_t* row_starts;
    const float* uniforms;
    const int32_t* context_lens;
    int32_t* err_flag;
    int num_rows;
    int vocab;
    int max_accepted;
};

constexpr int kVerifyThreads = 1024;
constexpr int kVerifyWarps = kVerifyThreads / 32;

// x in [0, 1] as a multiple of 2^-60, cut (exact from 2^-37 on); NaN and negative
// values are 0, larger ones 1.
constexpr int kFixedBits = 60;
__device__ __forceinline__ uint64_t to_fixed(float x) {
    if (!(x > 0.f)) return 0;
    const uint32_t b = __float_as_uint(fminf(x, 1.f));
    const int shift = (int)(b >> 23) - (127 + 23 - kFixedBits);
    const uint64_t m = (b & 0x7fffffu) | 0x800000u;  // (a subnormal vanishes either way)
    return shift >= 0 ? m << shift : shift > -32 ? m >> -shift : 0;
}
__device__ __forceinline__ double from_fixed(uint64_t x) { return (double)x * 0x1p-60; }
// x z, both in 2^-60
__device__ __forceinline__ uint64_t fixed_product(uint64_t x, uint64_t z) {
    return (__umul64hi(x, z) << (64 - kFixedBits)) | ((x * z) >> kFixedBits);
}
// x within [0, top]; NaN: 0
__device__ __forceinline__ float within(float x, float top) { return x > 0.f ? fminf(x, top) : 0.f; }

__device__ __forceinline__ uint64_t warp_sum64(uint64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The rejected children of the node that the walk has reached.
struct Rest {
    const float* p;
    const float* q;          // null: a draft has all its mass on its token
    const uint64_t* mass;    // Z_0 .. of the rejections
    const int32_t* tokens;   // their tokens
    int count;

    // What is left of element k, of target p_k and draft q_k.
    __device__ __forceinline__ uint64_t left(int k, float p_k, float q_k) const {
        uint64_t r = to_fixed(p_k);
        if (q != nullptr) {
            const uint64_t f = to_fixed(q_k);
            for (int j = 0; j < count; ++j) {
                const uint64_t gone = j == 0 ? f : fixed_product(f, mass[j]);
                r = r > gone ? r - gone : 0;
            }
        } else {
            for (int j = 0; j < count; ++j)
                if (tokens[j] == k) r = 0;
        }
        return r;
    }
    __device__ __forceinline__ uint64_t at(int k) const {
        return left(k, __ldg(p + k), q != nullptr ? __ldg(q + k) : 0.f);
    }
};

__global__ void __launch_bounds__(kVerifyThreads, 1) verify_kernel(const VerifyParams p) {
    __shared__ int s_parent[PKV_MAX_TREE_LEN], s_token[PKV_MAX_TREE_LEN];
    __shared__ float s_u[PKV_MAX_TREE_LEN], s_p[PKV_MAX_TREE_LEN], s_q[PKV_MAX_TREE_LEN];
    __shared__ uint64_t s_mass[PKV_MAX_TREE_LEN];
    __shared__ int32_t s_gone[PKV_MAX_TREE_LEN];
    __shared__ uint64_t s_warp[kVerifyWarps + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x;
    const int v = p.vocab;
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    int bad = 0;
    int first = p.row_starts[b];
    const int end = p.row_starts[b + 1];
    int count = 0;
    if (first < 0 || end < first || end > p.num_rows || end - first > PKV_MAX_TREE_LEN) {
        bad |= PKV_EFLAG_QUERY;
        first = 0;
    } else {
        count = end - first;
    }
    if (tid < count) {  // (a node a thread)
        int parent = tid - 1;
        const int token = tid > 0 ? p.tokens[first + tid] : 0;
        if (p.parents != nullptr && tid > 0) {
            parent = p.parents[first + tid];
            if (parent < 0 || parent >= tid) {
                if (parent != -1 && parent != PKV_TREE_ABSENT) bad |= PKV_EFLAG_TREE;
                parent = -1;
            }
        }
        if (token < 0 || token >= v) {
            bad |= PKV_EFLAG_TOKEN;
            parent = -1;
        }
        s_parent[tid] = parent;
        s_token[tid] = token;
        s_u[tid] = within(p.uniforms[first + tid], 0x1.fffffep-1f);
        if (parent >= 0) {
            const int64_t at = (int64_t)(first + parent) * v + token;
            s_p[tid] = within(p.target[at], 1.f);
            s_q[tid] = p.draft != nullptr ? within(p.draft[at], 1.f) : 1.f;
        }
    }
    int32_t* path = p.accepted + (int64_t)b * p.max_accepted;
    if (bad) flag_error(p.err_flag, bad);
    __syncthreads();

    // Sums of what is left over the warps' parts of the vocabulary, in s_warp; their total.
    const int per = ((v + kVerifyWarps - 1) / kVerifyWarps + 31) & ~31;  // elements of a warp
    Rest rest = {nullptr, nullptr, s_mass, s_gone, 0};
    auto pass = [&]() {
        uint64_t mine = 0;
        const int hi = min(v, (warp + 1) * per);
#pragma unroll 4
        for (int k = warp * per + lane; k < hi; k += 32) mine += rest.at(k);
        mine = warp_sum64(mine);
        __syncthreads();  // (the sums before these are used)
        if (lane == 0) s_warp[warp] = mine;
        __syncthreads();
        uint64_t total = 0;
        for (int w = 0; w < kVerifyWarps; ++w) total += s_warp[w];
        return total;
    };
    auto reach = [&](int node) {
        rest.p = p.target + (int64_t)(first + node) * v;
        rest.q = p.draft != nullptr ? p.draft + (int64_t)(first + node) * v : nullptr;
        rest.count = 0;
    };

    int cur = 0, length = 0;
    uint64_t total = 0;  // of the rest, where a child was rejected
    if (count > 0) {
        reach(0);
        if (tid == 0) path[0] = 0;
        length = 1;
    }
    for (int i = 1; i < count && length < p.max_accepted; ++i) {
        if (s_parent[i] != cur) continue;
        const int token = s_token[i];
        bool taken;
        if (rest.count == 0) {
            taken = (double)s_u[i] * (double)s_q[i] < (double)s_p[i];
        } else {
            const uint64_t r = rest.left(token, s_p[i], s_q[i]);
            taken = (double)s_u[i] * (double)s_q[i] * from_fixed(total) < from_fixed(r);
        }
        if (taken) {
            cur = i;
            reach(i);
            if (tid == 0) path[length] = i;
            ++length;
            continue;
        }
        __syncthreads();  // (the last pass's readers of these are through)
        if (tid == 0) {
            s_mass[rest.count] = total;  // (of the first, which is 1, nothing is read)
            s_gone[rest.count] = token;
        }
        ++rest.count;
        __syncthreads();
        total = pass();
    }

    int next = -1;
    if (count > 0) {
        if (rest.count == 0 || total == 0) {
            rest.count = 0;
            total = pass();
        }
        if (total == 0) {
            if (tid == 0) flag_error(p.err_flag, PKV_EFLAG_TOKEN);
        } else {
            // the first element whose running sum is above u times the total: the warp's
            // part that holds it, then of that the warp's share, then of that the lane
            const uint64_t u = (uint64_t)((double)s_u[0] * 0x1p64);
            uint64_t aim = __umul64hi(u, total);
            int w = 0;
            while (w + 1 < kVerifyWarps && s_warp[w] <= aim) aim -= s_warp[w++];
            const int lo = w * per, hi = min(v, lo + per);
            const int share = (hi - lo + kVerifyWarps - 1) / kVerifyWarps;
            uint64_t mine = 0;
            for (int k = lo + warp * share + lane; k < min(hi, lo + (warp + 1) * share); k += 32)
                mine += rest.at(k);
            mine = warp_sum64(mine);
            __syncthreads();
            if (lane == 0) s_warp[warp] = mine;
            __syncthreads();
            if (warp == 0) {
                int part = 0;
                while (part + 1 < kVerifyWarps && s_warp[part] <= aim) aim -= s_warp[part++];
                const int last = min(hi, lo + (part + 1) * share);
                for (int k0 = lo + part * share; k0 < last; k0 += 32) {
                    uint64_t r = k0 + lane < last ? rest.at(k0 + lane) : 0;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const uint64_t x = __shfl_up_sync(0xffffffffu, r, o);
                        if (lane >= o) r += x;
                    }
                    const uint32_t over = __ballot_sync(0xffffffffu, r > aim);
                    if (over != 0) {
                        next = k0 + __ffs(over) - 1;
                        break;
                    }
                    aim -= __shfl_sync(0xffffffffu, r, 31);
                }
                if (next < 0 && lane == 0) flag_error(p.err_flag, PKV_EFLAG_TOKEN);
            }
        }
    }
    for (int i = length + tid; i < p.max_accepted; i += kVerifyThreads) path[i] = -1;
    if (tid == 0) {
        p.accepted_lens[b] = length;
        p.next_tokens[b] = next;
        if (p.new_context_lens != nullptr)
            p.new_context_lens[b] = p.context_lens[b] - count + length;
    }
}

}  // namespace pkv

using namespace pkv;

extern "C" pkv_status pkv_verify_drafts(int32_t* accepted, int32_t* accepted_lens,
                                        int32_t* next_tokens, int32_t* new_context_lens,
                                        const float* target_probs, const float* draft_probs,
                                        const int32_t* tokens, const int32_t* parents,
                                        const int32_t* row_starts, const float* uniforms,
                                        const int32_t* context_lens, int num_seqs, int num_rows,
                                        int vocab, int max_accepted, int32_t* err_flag,
                                        void* stream) {
    if (num_seqs < 0 || num_rows < 0 || vocab <= 0 || max_accepted <= 0 ||
        (context_lens == nullptr) != (new_context_lens == nullptr))
        return PKV_ERR_INVALID_ARG;
    if (vocab > (1 << 24) || num_seqs == INT_MAX) return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!accepted || !accepted_lens || !next_tokens || !row_starts ||
        (num_rows > 0 && (!target_probs || !tokens || !uniforms)))
        return PKV_ERR_INVALID_ARG;
    const void* all[] = {accepted, accepted_lens, next_tokens, new_context_lens, target_probs,
                         draft_probs, tokens, parents, row_starts, uniforms, context_lens};
    for (const void* a : all)
        if (reinterpret_cast<uintptr_t>(a) & 3u) return PKV_ERR_INVALID_ARG;
    const int64_t seqs = num_seqs, rows = num_rows;
    const int64_t bytes[] = {seqs * max_accepted * 4, seqs * 4, seqs * 4, seqs * 4,
                             rows * vocab * 4, rows * vocab * 4, rows * 4, rows * 4,
                             (seqs + 1) * 4, rows * 4, seqs * 4};
    for (int i = 0; i < 4; ++i)  // what is written, against everything behind it
        for (int j = i + 1; j < 11; ++j) {
            if (all[i] == nullptr || all[j] == nullptr || bytes[j] == 0) continue;
            if (i == 3 && j == 10 && all[i] == all[j]) continue;
            if (overlap(all[i], bytes[i], all[j], bytes[j])) return PKV_ERR_INVALID_ARG;
        }
    VerifyParams p = {};
    p.accepted = accepted;
    p.accepted_lens = accepted_lens;
    p.next_tokens = next_tokens;
    p.new_context_lens = new_context_lens;
    p.target = target_probs;
    p.draft = draft_probs;
    p.tokens = tokens;
    p.parents = parents;
    p.row_starts = row_starts;
    p.uniforms = uniforms;
    p.context_lens = context_lens;
    p.err_flag = err_flag;
    p.num_rows = num_rows;
    p.vocab = vocab;
    p.max_accepted = max_accepted;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_seqs);
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, verify_kernel, p) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}
