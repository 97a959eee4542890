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
// token lies.  A cluster of CTAs shares a sequence's vocabulary: each takes the walk by
// itself, holds its part of the rest in registers (16 elements a thread) and exchanges
// its sum with the others' through their shared memory.
// Sums: 64-bit whole numbers of 2^-45, so that they are the same in any order and a
// draw at a border does not depend on the split of the work (a sum in fp32 is off by
// more than the probability of a token of a flat distribution).  Two additions of fp32
// take a probability apart into them (to_fixed); 2^-60, by shifts of the fraction, took
// twice the instructions, which are what a pass over registers costs.
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
    int slice;  // of the vocabulary, a CTA's
};

constexpr int kVerifyThreads = 1024;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyEach = 16;  // elements that a thread holds
constexpr int kVerifyBlock = kVerifyThreads * kVerifyEach;
constexpr int kVerifyCluster = 8;  // CTAs of a sequence at most

// x in [0, 1] as a multiple of 2^-45, to nearest: a sum with 2 has the bits of x down to
// 2^-22 as its fraction, and what is left of x, 2^23 times as large, beside 3 the next 23
// (every step but the last is exact).  NaN and negative values are 0, larger ones 1.
constexpr int kFixedBits = 45;
constexpr int kFixedHigh = 0x40000000, kFixedLow = 0x40400000;  // the bits of 2 and of 3
__device__ __forceinline__ int64_t fixed_of(int hi, int lo) {
    return (int64_t)hi * (1 << (kFixedBits - 22)) + lo;
}
__device__ __forceinline__ uint64_t to_fixed(float x) {
    x = __saturatef(x);
    const float a = __fadd_rn(x, 2.f);
    const float r = __fsub_rn(x, __fsub_rn(a, 2.f));  // at most 2^-23
    const float c = __fmaf_rn(r, 0x1p23f, 3.f);
    return (uint64_t)fixed_of(__float_as_int(a) - kFixedHigh, __float_as_int(c) - kFixedLow);
}
// to_fixed(x) - to_fixed(y), at least 0: both taken apart at once.
__device__ __forceinline__ uint64_t fixed_rest(float x, float y) {
    const float2 v = make_float2(__saturatef(x), __saturatef(y));
    const float2 a = ptx::add2(v, make_float2(2.f, 2.f));
    const float2 t = ptx::add2(a, make_float2(-2.f, -2.f));
    const float2 r = ptx::fma2(t, make_float2(-1.f, -1.f), v);
    const float2 c = ptx::fma2(r, make_float2(0x1p23f, 0x1p23f), make_float2(3.f, 3.f));
    const int64_t d = fixed_of(__float_as_int(a.x) - __float_as_int(a.y),
                               __float_as_int(c.x) - __float_as_int(c.y));
    return (uint64_t)(d > 0 ? d : 0);
}
// x z, both in 2^-45, x at most 1
__device__ __forceinline__ uint64_t fixed_product(uint64_t x, uint64_t z) {
    return __umul64hi(x << (64 - kFixedBits - 1), z << 1);
}
// u q < p without a rounding: their product as two terms.
__device__ __forceinline__ bool product_below(float u, float q, float p) {
    const float hi = __fmul_rn(u, q);
    return hi < p || (hi == p && __fmaf_rn(u, q, -hi) < 0.f);
}
// x within [0, top]; NaN: 0
__device__ __forceinline__ float within(float x, float top) { return x > 0.f ? fminf(x, top) : 0.f; }

__device__ __forceinline__ uint64_t warp_sum64(uint64_t x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// What is left of an element once the first `count` of a node's children were rejected:
// `mass` holds Z_0 .., `gone` their tokens (of a draft without a distribution).
__device__ __forceinline__ uint64_t fixed_less(uint64_t r, uint64_t gone) {
    return r > gone ? r - gone : 0;
}
__device__ __forceinline__ uint64_t rest_of(uint64_t p, uint64_t q, bool draft, int k,
                                            const uint64_t* mass, const int32_t* gone, int count) {
    for (int j = 0; j < count; ++j) {
        if (draft)
            p = fixed_less(p, j == 0 ? q : fixed_product(q, mass[j]));
        else if (gone[j] == k)
            p = 0;
    }
    return p;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Writes x where `local` lies in CTA `rank` of the cluster.
__device__ __forceinline__ void store_cluster(uint64_t* local, uint32_t rank, uint64_t x) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_addr(local)), "r"(rank));
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(x) : "memory");
}

// VEC: elements that a thread loads at a time (4 where rows and their parts are 16-byte
// aligned, else 1).  A block of a slice: kVerifyEach / VEC groups of VEC a thread, so that
// the order of the elements is (group, thread, element).
template <int VEC>
__global__ void __launch_bounds__(kVerifyThreads, 1) verify_kernel(const VerifyParams p) {
    constexpr int G = kVerifyEach / VEC;
    __shared__ int s_parent[PKV_MAX_TREE_LEN], s_token[PKV_MAX_TREE_LEN];
    __shared__ float s_u[PKV_MAX_TREE_LEN], s_p[PKV_MAX_TREE_LEN], s_q[PKV_MAX_TREE_LEN];
    __shared__ uint64_t s_mass[PKV_MAX_TREE_LEN];
    __shared__ int32_t s_gone[PKV_MAX_TREE_LEN];
    __shared__ uint64_t s_warp[G][kVerifyWarps];
    __shared__ uint64_t s_cta[2][kVerifyCluster];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = cluster_rank(), ctas = cluster_size();
    const int b = blockIdx.x / ctas;
    const int v = p.vocab;
    const int lo = min(v, rank * p.slice), hi = min(v, lo + p.slice);  // this CTA's elements
    const bool once = p.slice <= kVerifyBlock;  // they stay in registers
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
    if (bad && rank == 0) flag_error(p.err_flag, bad);
    __syncthreads();

    // The rest of this CTA's block of elements from `base` on, and the draft's part of it.
    uint64_t left[kVerifyEach] = {};
    float draft[kVerifyEach];
    const bool has_draft = p.draft != nullptr;
    auto element = [&](int base, int i) {  // (of this thread's i-th)
        return base + (i / VEC) * kVerifyThreads * VEC + tid * VEC + i % VEC;
    };
    // (what lies beyond the slice is 0)
    float target[kVerifyEach];
    auto fetch = [&](int node, int base, bool with_draft) {
        const float* tp = p.target + (int64_t)(first + node) * v;
        const float* dp = with_draft ? p.draft + (int64_t)(first + node) * v : nullptr;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int k = element(base, g * VEC);
            if constexpr (VEC == 4) {
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f), d = a;
                if (k < hi) {
                    a = __ldg(reinterpret_cast<const float4*>(tp + k));
                    if (with_draft) d = __ldg(reinterpret_cast<const float4*>(dp + k));
                }
                target[4 * g] = a.x, target[4 * g + 1] = a.y;
                target[4 * g + 2] = a.z, target[4 * g + 3] = a.w;
                draft[4 * g] = d.x, draft[4 * g + 1] = d.y;
                draft[4 * g + 2] = d.z, draft[4 * g + 3] = d.w;
            } else {
                target[g] = k < hi ? __ldg(tp + k) : 0.f;
                draft[g] = with_draft && k < hi ? __ldg(dp + k) : 0.f;
            }
        }
    };
    // f(i) for this thread's elements of a block, group by group while there are any.
    auto each = [&](int base, auto f) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (base + g * kVerifyThreads * VEC >= hi) break;
#pragma unroll
            for (int i = 0; i < VEC; ++i) f(g * VEC + i);
        }
    };
    auto cta_sum = [&](uint64_t mine) {  // of all threads, for all
        mine = warp_sum64(mine);
        __syncthreads();  // (the sums before these are used)
        if (lane == 0) s_warp[0][warp] = mine;
        __syncthreads();
        return warp_sum64(s_warp[0][lane]);
    };
    int passes = 0;
    // What is left of block `base` at the node that was fetched, into `left`, and its sum.
    auto start = [&](int base, int rejected) {
        uint64_t mine = 0;
        each(base, [&](int i) {
            if (has_draft && rejected > 0)
                left[i] = fixed_rest(target[i], draft[i]);
            else
                left[i] = rest_of(to_fixed(target[i]), 0, false, element(base, i), s_mass, s_gone,
                                  rejected);
            if (has_draft && rejected > 1) {
                const uint64_t f = to_fixed(draft[i]);
                for (int j = 1; j < rejected; ++j)
                    left[i] = fixed_less(left[i], fixed_product(f, s_mass[j]));
            }
            mine += left[i];
        });
        return mine;
    };
    // What is left at `node` after `rejected` children, its sum over the cluster.
    auto pass = [&](int node, int rejected) {
        uint64_t mine = 0;
        if (!once) {
            for (int base = lo; base < hi; base += kVerifyBlock) {
                fetch(node, base, has_draft && rejected > 0);
                mine += start(base, rejected);
            }
        } else if (rejected <= 1) {
            fetch(node, lo, has_draft && rejected > 0);
            mine = start(lo, rejected);
        } else {  // (the rest is there)
            const uint64_t z = s_mass[rejected - 1];
            const int token = s_gone[rejected - 1];
            each(lo, [&](int i) {
                if (has_draft)
                    left[i] = fixed_less(left[i], fixed_product(to_fixed(draft[i]), z));
                else if (element(lo, i) == token)
                    left[i] = 0;
                mine += left[i];
            });
        }
        const uint64_t sum = cta_sum(mine);
        const int par = passes++ & 1;
        if (tid < ctas) store_cluster(&s_cta[par][rank], tid, sum);
        cluster_sync();
        uint64_t total = 0;
        for (int c = 0; c < ctas; ++c) total += s_cta[par][c];
        return total;
    };

    int cur = 0, length = 0, rejected = 0;
    uint64_t total = 0;  // of the rest, where a child was rejected
    if (count > 0) {
        if (tid == 0 && rank == 0) path[0] = 0;
        length = 1;
    }
    for (int i = 1; i < count && length < p.max_accepted; ++i) {
        if (s_parent[i] != cur) continue;
        bool taken;
        if (rejected == 0) {
            taken = product_below(s_u[i], s_q[i], s_p[i]);
        } else {
            const uint64_t r = rest_of(to_fixed(s_p[i]), to_fixed(s_q[i]), has_draft, s_token[i],
                                       s_mass, s_gone, rejected);
            taken = fixed_product(fixed_product(to_fixed(s_u[i]), to_fixed(s_q[i])), total) < r;
        }
        if (taken) {
            cur = i;
            rejected = 0;
            if (tid == 0 && rank == 0) path[length] = i;
            ++length;
            continue;
        }
        __syncthreads();  // (the last pass's readers of these are through)
        if (tid == 0) {
            s_mass[rejected] = total;  // (of the first, which is 1, nothing is read)
            s_gone[rejected] = s_token[i];
        }
        ++rejected;
        __syncthreads();
        total = pass(cur, rejected);
    }

    if (count > 0 && (rejected == 0 || total == 0)) {
        rejected = 0;
        total = pass(cur, 0);
    }
    // The first element whose running sum is above u times the total: the CTA that holds
    // it, the block, the warp's part of a group, and there the lane's element.
    bool found = false;
    if (total > 0) {
        uint64_t aim = fixed_product(to_fixed(s_u[0]), total);
        int owner = 0;
        const int par = (passes - 1) & 1;
        while (owner + 1 < ctas && s_cta[par][owner] <= aim) aim -= s_cta[par][owner++];
        for (int base = lo; owner == rank && base < hi && !found; base += kVerifyBlock) {
            if (!once) {
                fetch(cur, base, has_draft && rejected > 0);
#pragma unroll
                for (int i = 0; i < kVerifyEach; ++i) left[i] = 0;
                const uint64_t sum = cta_sum(start(base, rejected));
                if (sum <= aim && base + kVerifyBlock < hi) {
                    aim -= sum;
                    continue;
                }
            }
            found = true;  // in this block
            __syncthreads();
#pragma unroll
            for (int g = 0; g < G; ++g) {
                uint64_t x = 0;
#pragma unroll
                for (int i = 0; i < VEC; ++i) x += left[g * VEC + i];
                x = warp_sum64(x);
                if (lane == 0) s_warp[g][warp] = x;
            }
            __syncthreads();
            // every warp finds the part, a group at a time; the part's own goes on
            int group = 0, owns = 0;
            for (; group < G; ++group) {
                uint64_t incl = s_warp[group][lane];
                const uint64_t own = incl;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint64_t x = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += x;
                }
                const uint32_t over = __ballot_sync(0xffffffffu, incl > aim);
                if (over != 0) {
                    owns = __ffs(over) - 1;
                    aim -= __shfl_sync(0xffffffffu, incl - own, owns);
                    break;
                }
                aim -= __shfl_sync(0xffffffffu, incl, 31);
            }
            if (warp == owns) {
                uint64_t mine[VEC] = {};
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        if (g == group) mine[i] = left[g * VEC + i];
                uint64_t sum = 0;
#pragma unroll
                for (int i = 0; i < VEC; ++i) sum += mine[i];
                uint64_t incl = sum;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint64_t x = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += x;
                }
                const uint32_t over = __ballot_sync(0xffffffffu, incl > aim);
                if (over == 0) {  // (a row whose sum is no distribution's)
                    if (lane == 0) {
                        flag_error(p.err_flag, PKV_EFLAG_TOKEN);
                        p.next_tokens[b] = -1;
                    }
                } else if (lane == __ffs(over) - 1) {
                    aim -= incl - sum;
                    int i = 0;
#pragma unroll
                    for (int j = 0; j + 1 < VEC; ++j)
                        if (i == j && mine[j] <= aim) {
                            aim -= mine[j];
                            ++i;
                        }
                    p.next_tokens[b] = base + group * kVerifyThreads * VEC +
                                       tid * VEC + i;
                }
            }
        }
    }
    if (rank == 0) {
        for (int i = length + tid; i < p.max_accepted; i += kVerifyThreads) path[i] = -1;
        if (tid == 0) {
            p.accepted_lens[b] = length;
            if (total == 0) {
                p.next_tokens[b] = -1;
                if (count > 0) flag_error(p.err_flag, PKV_EFLAG_TOKEN);
            }
            if (p.new_context_lens != nullptr)
                p.new_context_lens[b] = p.context_lens[b] - count + length;
        }
    }
    cluster_sync();  // (no CTA leaves while another may still write its sum there)
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
    // CTAs of a sequence: as many as hold its vocabulary in registers, and more while the
    // sequences leave SMs idle
    const int sms = current_sm_count();
    if (sms <= 0) return PKV_ERR_CUDA;
    int ctas = 1;
    while (ctas < kVerifyCluster && ((int64_t)ctas * kVerifyBlock < vocab ||
                                     (ctas * 1024 < vocab && num_seqs * 2ll * ctas <= sms)))
        ctas *= 2;
    if (num_seqs > INT_MAX / ctas) return PKV_ERR_UNSUPPORTED;
    p.slice = ((vocab + ctas - 1) / ctas + 3) & ~3;
    const bool vec = vocab % 4 == 0 && aligned16(target_probs) && aligned16(draft_probs);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_seqs * ctas);
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, vec ? verify_kernel<4> : verify_kernel<1>, p) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}
