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
// itself, sums its part of the rest (from L2 where a node has a second pass) and
// exchanges its sum with the others' through their shared memory.
// Sums: 64-bit whole numbers of 2^-44, so that they are the same in any order and a
// draw at a border does not depend on the split of the work (a sum in fp32 is off by
// more than the probability of a token of a flat distribution).  Two additions of fp32
// take a probability apart into them (to_fixed); 2^-60, by shifts of the fraction, took
// twice the instructions, which are what a pass over registers costs.
// Measured (a call in a graph): a chain of 5 over 32000 tokens 6.2 us, 64 chains of up to 7
// 9.0 us, 32 trees of 16 nodes over 128000 tokens 35.5 us, of 4.8 that the bytes of the rows
// passed over would take: one sequence's passes follow one another, some 3 us each (its
// eight CTAs' share of two rows, a sum over the cluster), and the most rejected sequence
// has the last word.  Memory reads 9 % of its rate, 0.4 instructions a cycle.
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

// (32 trees over 128000 tokens: 35 us, with 256 threads and four CTAs an SM 45, with 1024
// and one 39)
constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyCtas = 2;     // an SM
constexpr int kVerifyCluster = 8;  // CTAs of a sequence at most

// x in [0, 1] as a multiple of 2^-44, to nearest: a sum with 2 has the bits of x down to
// 2^-22 as its fraction, and what is left of x, 2^22 times as large, beside 3 the next 22
// (every step but the last is exact).  NaN and negative values are 0, larger ones 1.
constexpr int kFixedBits = 44;
constexpr int kFixedHigh = 0x40000000, kFixedLow = 0x40400000;  // the bits of 2 and of 3
__device__ __forceinline__ int64_t fixed_of(int hi, int lo) {
    return (int64_t)hi * (1 << (kFixedBits - 22)) + lo;
}
__device__ __forceinline__ uint64_t to_fixed(float x) {
    x = __saturatef(x);
    const float a = __fadd_rn(x, 2.f);
    const float r = __fsub_rn(x, __fsub_rn(a, 2.f));  // at most 2^-23
    const float c = __fmaf_rn(r, 0x1p22f, 3.f);
    return (uint64_t)fixed_of(__float_as_int(a) - kFixedHigh, __float_as_int(c) - kFixedLow);
}
// to_fixed(x) - to_fixed(y), at least 0: both taken apart at once.
__device__ __forceinline__ uint64_t fixed_rest(float x, float y) {
    const float2 v = make_float2(__saturatef(x), __saturatef(y));
    const float2 a = ptx::add2(v, make_float2(2.f, 2.f));
    const float2 t = ptx::add2(a, make_float2(-2.f, -2.f));
    const float2 r = ptx::fma2(t, make_float2(-1.f, -1.f), v);
    const float2 c = ptx::fma2(r, make_float2(0x1p22f, 0x1p22f), make_float2(3.f, 3.f));
    const int64_t d = fixed_of(__float_as_int(a.x) - __float_as_int(a.y),
                               __float_as_int(c.x) - __float_as_int(c.y));
    return (uint64_t)(d > 0 ? d : 0);
}
// x z, both in 2^-44, x at most 1
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

__device__ __forceinline__ uint64_t fixed_less(uint64_t r, uint64_t gone) {
    return r > gone ? r - gone : 0;
}
// Z as two fp32 terms, and Z q for two q: exact to 2^-47 before it is a multiple of 2^-44.
__device__ __forceinline__ float2 mass_terms(uint64_t z) {
    const float hi = __ull2float_rn(z);
    const int64_t rest = (int64_t)(z - __float2ull_rn(hi));
    return make_float2(hi * 0x1p-44f, __ll2float_rn(rest) * 0x1p-44f);
}
__device__ __forceinline__ void fixed_products(float2 z, float2 q, uint64_t& first,
                                               uint64_t& second) {
    const float2 zh = make_float2(z.x, z.x), zl = make_float2(z.y, z.y);
    const float2 hi = ptx::mul2(zh, q);
    const float2 lo =
        ptx::fma2(zl, q, ptx::fma2(zh, q, make_float2(-hi.x, -hi.y)));
    const float2 a = ptx::add2(hi, make_float2(2.f, 2.f));
    const float2 t = ptx::add2(a, make_float2(-2.f, -2.f));
    const float2 r = ptx::add2(ptx::fma2(t, make_float2(-1.f, -1.f), hi), lo);
    const float2 c = ptx::fma2(r, make_float2(0x1p22f, 0x1p22f), make_float2(3.f, 3.f));
    first = (uint64_t)fixed_of(__float_as_int(a.x) - kFixedHigh, __float_as_int(c.x) - kFixedLow);
    second = (uint64_t)fixed_of(__float_as_int(a.y) - kFixedHigh, __float_as_int(c.y) - kFixedLow);
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

// VEC: elements that a lane loads at a time (4 where rows and their parts are 16-byte
// aligned, else 1).  A warp takes a run of its CTA's elements.
template <int VEC>
__global__ void __launch_bounds__(kVerifyThreads, kVerifyCtas)
verify_kernel(const VerifyParams p) {
    __shared__ int s_parent[PKV_MAX_TREE_LEN], s_token[PKV_MAX_TREE_LEN];
    __shared__ float s_u[PKV_MAX_TREE_LEN], s_p[PKV_MAX_TREE_LEN], s_q[PKV_MAX_TREE_LEN];
    __shared__ float2 s_mass[PKV_MAX_TREE_LEN];  // Z of the rejections
    __shared__ int32_t s_gone[PKV_MAX_TREE_LEN];
    __shared__ uint64_t s_warp[kVerifyWarps];
    __shared__ uint64_t s_cta[2][kVerifyCluster];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = cluster_rank(), ctas = cluster_size();
    const int b = blockIdx.x / ctas;
    const int v = p.vocab;
    const int lo = min(v, rank * p.slice), hi = min(v, lo + p.slice);  // this CTA's elements
    const int run = (p.slice / 4 + kVerifyWarps - 1) / kVerifyWarps * 4;  // of a warp
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
    for (int i = tid; i < count; i += kVerifyThreads) {  // (a node a thread)
        int parent = i - 1;
        const int token = i > 0 ? p.tokens[first + i] : 0;
        if (p.parents != nullptr && i > 0) {
            parent = p.parents[first + i];
            if (parent < 0 || parent >= i) {
                if (parent != -1 && parent != PKV_TREE_ABSENT) bad |= PKV_EFLAG_TREE;
                parent = -1;
            }
        }
        if (token < 0 || token >= v) {
            bad |= PKV_EFLAG_TOKEN;
            parent = -1;
        }
        s_parent[i] = parent;
        s_token[i] = token;
        s_u[i] = within(p.uniforms[first + i], 0x1.fffffep-1f);
        if (parent >= 0) {
            const int64_t at = (int64_t)(first + parent) * v + token;
            s_p[i] = within(p.target[at], 1.f);
            s_q[i] = p.draft != nullptr ? within(p.draft[at], 1.f) : 1.f;
        }
    }
    int32_t* path = p.accepted + (int64_t)b * p.max_accepted;
    if (bad && rank == 0) flag_error(p.err_flag, bad);
    __syncthreads();

    const bool has_draft = p.draft != nullptr;
    const float *tp = nullptr, *dp = nullptr;  // the rows of the pass
    int rejected = 0;
    // What is left of two elements, k of target x.x and draft y.x and k2 of x.y and y.y,
    // after `rejected` children.
    auto rest2 = [&](int k, int k2, float2 x, float2 y, uint64_t& r, uint64_t& r2) {
        if (!has_draft || rejected == 0) {
            r = to_fixed(x.x);
            r2 = to_fixed(x.y);
            for (int j = 0; j < rejected; ++j) {
                if (s_gone[j] == k) r = 0;
                if (s_gone[j] == k2) r2 = 0;
            }
            return;
        }
        r = fixed_rest(x.x, y.x);
        r2 = fixed_rest(x.y, y.y);
        if (rejected > 1) {
            const float2 q = make_float2(__saturatef(y.x), __saturatef(y.y));
            for (int j = 1; j < rejected; ++j) {
                uint64_t g, g2;
                fixed_products(s_mass[j], q, g, g2);
                r = fixed_less(r, g);
                r2 = fixed_less(r2, g2);
            }
        }
    };
    auto rest = [&](int k, float x, float y) {
        uint64_t r, r2;
        rest2(k, -1, make_float2(x, 0.f), make_float2(y, 0.f), r, r2);
        return r;
    };
    // The sum of elements from .. to - 1 over a warp; kSteps loads of a lane in flight.
    constexpr int kSteps = 16 / VEC;
    auto warp_run = [&](int from, int to) {
        uint64_t mine = 0;
        for (int k0 = from + lane * VEC; k0 < to; k0 += 32 * VEC * kSteps) {
            float x[kSteps * VEC], y[kSteps * VEC];
#pragma unroll
            for (int u = 0; u < kSteps; ++u) {
                const int k = k0 + u * 32 * VEC;
                if constexpr (VEC == 4) {
                    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), d = a;
                    if (k < to) {
                        a = __ldg(reinterpret_cast<const float4*>(tp + k));
                        if (dp != nullptr) d = __ldg(reinterpret_cast<const float4*>(dp + k));
                    }
                    x[4 * u] = a.x, x[4 * u + 1] = a.y, x[4 * u + 2] = a.z, x[4 * u + 3] = a.w;
                    y[4 * u] = d.x, y[4 * u + 1] = d.y, y[4 * u + 2] = d.z, y[4 * u + 3] = d.w;
                } else {
                    x[u] = k < to ? __ldg(tp + k) : 0.f;
                    y[u] = k < to && dp != nullptr ? __ldg(dp + k) : 0.f;
                }
            }
#pragma unroll
            for (int u = 0; u < kSteps; ++u) {
                const int k = k0 + u * 32 * VEC;
                if (k >= to) break;
                if constexpr (VEC == 4) {
                    uint64_t r[4];
                    rest2(k, k + 1, make_float2(x[4 * u], x[4 * u + 1]),
                          make_float2(y[4 * u], y[4 * u + 1]), r[0], r[1]);
                    rest2(k + 2, k + 3, make_float2(x[4 * u + 2], x[4 * u + 3]),
                          make_float2(y[4 * u + 2], y[4 * u + 3]), r[2], r[3]);
                    mine += (r[0] + r[1]) + (r[2] + r[3]);
                } else {
                    mine += rest(k, x[u], y[u]);
                }
            }
        }
        return warp_sum64(mine);
    };
    int passes = 0;
    // What is left at `node`, its sum over the cluster; the warps' parts in s_warp.
    auto pass = [&](int node) {
        tp = p.target + (int64_t)(first + node) * v;
        dp = has_draft && rejected > 0 ? p.draft + (int64_t)(first + node) * v : nullptr;
        const int from = lo + warp * run;
        const uint64_t mine = warp_run(from, min(hi, from + run));
        __syncthreads();  // (the sums before these are used)
        if (lane == 0) s_warp[warp] = mine;
        __syncthreads();
        const int par = passes++ & 1;
        if (warp == 0) {
            const uint64_t sum = warp_sum64(lane < kVerifyWarps ? s_warp[lane] : 0);
            if (lane < ctas) store_cluster(&s_cta[par][rank], lane, sum);
        }
        cluster_sync();
        uint64_t total = 0;
        for (int c = 0; c < ctas; ++c) total += s_cta[par][c];
        return total;
    };

    int cur = 0, length = 0;
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
            const uint64_t r = rest(s_token[i], s_p[i], s_q[i]);
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
            s_mass[rejected] = mass_terms(total);  // (of the first, which is 1, nothing is read)
            s_gone[rejected] = s_token[i];
        }
        ++rejected;
        __syncthreads();
        total = pass(cur);
    }

    if (count > 0 && (rejected == 0 || total == 0)) {
        rejected = 0;
        total = pass(cur);
    }
    // The first element whose running sum is above u times the total: the CTA that holds
    // it, the warp's run, of that a warp's share, there the element.
    if (total > 0) {
        uint64_t aim = fixed_product(to_fixed(s_u[0]), total);
        int owner = 0;
        const int par = (passes - 1) & 1;
        while (owner + 1 < ctas && s_cta[par][owner] <= aim) aim -= s_cta[par][owner++];
        if (owner == rank) {
            // the first of the warps' sums that the aim lies in, and what is left of it there
            auto narrow = [&]() {
                const uint64_t own = lane < kVerifyWarps ? s_warp[lane] : 0;
                uint64_t incl = own;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint64_t x = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += x;
                }
                const uint32_t over = __ballot_sync(0xffffffffu, incl > aim);
                const int at = over != 0 ? __ffs(over) - 1 : kVerifyWarps - 1;
                aim -= __shfl_sync(0xffffffffu, incl - own, at);
                return at;
            };
            const int from = lo + narrow() * run, to = min(hi, from + run);
            const int share = (run + kVerifyWarps - 1) / kVerifyWarps;
            uint64_t mine = 0;
            for (int k = from + warp * share + lane; k < min(to, from + (warp + 1) * share); k += 32)
                mine += rest(k, __ldg(tp + k), dp != nullptr ? __ldg(dp + k) : 0.f);
            mine = warp_sum64(mine);
            __syncthreads();
            if (lane == 0) s_warp[warp] = mine;
            __syncthreads();
            if (warp == 0) {
                const int part = narrow();
                const int last = min(to, from + (part + 1) * share);
                int next = -1;
                for (int k0 = from + part * share; k0 < last && next < 0; k0 += 32) {
                    const int k = k0 + lane;
                    uint64_t r = k < last ? rest(k, __ldg(tp + k), dp != nullptr ? __ldg(dp + k) : 0.f)
                                          : 0;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const uint64_t x = __shfl_up_sync(0xffffffffu, r, o);
                        if (lane >= o) r += x;
                    }
                    const uint32_t over = __ballot_sync(0xffffffffu, r > aim);
                    if (over != 0) next = k0 + __ffs(over) - 1;
                    aim -= __shfl_sync(0xffffffffu, r, 31);
                }
                if (lane == 0) {
                    p.next_tokens[b] = next;
                    if (next < 0)  // a row whose sum is no distribution's
                        flag_error(p.err_flag, PKV_EFLAG_TOKEN);
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
    // CTAs of a sequence: while there are elements for them, as many as run at once
    const int sms = current_sm_count();
    if (sms <= 0) return PKV_ERR_CUDA;
    int ctas = 1;
    while (ctas < kVerifyCluster && ctas * 1024 < vocab &&
           num_seqs * 2ll * ctas <= (int64_t)sms * kVerifyCtas)
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
