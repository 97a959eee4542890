// The plan of a ragged step: pages given back and taken, block tables, positions
// and cache slots, from the requests' lengths.
#include <algorithm>
#include <climits>

#include "pkv_common.cuh"
#include "pkv_device.cuh"

namespace pkv {

// ---------------------------------------------------------------------------
// One CTA does all that has an order: sums over the sequences place each one's
// released pages on the free list, the pages it takes and its tokens.  Pages and
// tokens are then handled one a thread, whichever sequence they belong to (found by
// bisection in the sums), so that one sequence's thousand pages take no longer than
// a thousand sequences' one.  Steps of many tokens write their positions and slots
// in a second kernel (batch_slots_kernel), which only reads what the first left.
// Latency is all that it costs (a call in a graph: 4.5 us for 256 sequences of single
// tokens, 7.9 us for 200 of which 24 bring some 15000 together, whose positions the second
// kernel writes): a launch, three rounds of loads that depend on one another and a scan.
// What is known to need no sum is not summed (no page given back, everyone served), a
// batch of one run is read once, and the tokens' bisections run in shared memory: without
// these 6.3 and 8.9 us.
// ---------------------------------------------------------------------------

struct BatchPlanParams {
    int32_t* query_starts;
    int32_t* positions;
    int64_t* slot_mapping;
    int32_t* new_context_lens;
    int32_t* new_free_count;
    const int32_t* context_lens;
    const int32_t* new_lens;
    const int32_t* keep_lens;
    const int32_t* shared_pages;
    int32_t* block_tables;
    int32_t* free_blocks;
    const int32_t* free_count;
    int32_t* err_flag;
    int max_blocks_per_seq;
    int free_capacity;
    int num_seqs;
    int max_tokens;
    int num_blocks;
    int block_size;
    int cap;  // tokens of a block table
};

// (With 1024 threads 256 single tokens took 0.6 us longer, with 256 24 chunks of 15000
// tokens 1.2 us.)
constexpr int kBatchThreads = 512;
constexpr int kBatchWarps = kBatchThreads / 32;
// Up to this many token places the first kernel writes them itself.
constexpr int kBatchOwnTokens = 8 * kBatchThreads;

// A sequence's part of the step, before the free list is asked.
struct BatchSeq {
    int keep;     // tokens kept
    int first;    // the first released entry of its table
    int back;     // pages released
    int add;      // new tokens asked for
    int need;     // pages for them
};

__device__ __forceinline__ BatchSeq batch_seq(const BatchPlanParams& p, int b, int& bad) {
    BatchSeq s;
    const int c = p.context_lens[b], a = p.new_lens[b];
    const int k = p.keep_lens != nullptr ? p.keep_lens[b] : c;
    const int shared = p.shared_pages != nullptr ? p.shared_pages[b] : 0;
    const int shift = __ffs(p.block_size) - 1;
    auto pages = [&](int n) { return n == 0 ? 0 : ((n - 1) >> shift) + 1; };
    if (c < 0 || c > p.cap || k < 0 || k > c) {
        bad |= PKV_EFLAG_CONTEXT_LEN;
        s.keep = clamped_len(c, p.cap);
        s.first = s.back = s.add = s.need = 0;
        return s;
    }
    s.keep = k;
    const int kept = pages(k), held = pages(c);
    s.first = max(kept, shared);
    s.back = max(0, held - s.first);
    s.add = a;
    if (a < 0 || a > p.cap - k) {
        bad |= PKV_EFLAG_CONTEXT_LEN;
        s.add = 0;
    }
    s.need = pages(k + s.add) - kept;
    return s;
}

// Inclusive sums of two numbers over the CTA's threads, and their totals.
struct Sums {
    int64_t a, b, total_a, total_b;
};
__device__ __forceinline__ Sums block_sums(int64_t a, int64_t b, int64_t (*s_warp)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
            a += x;
            b += y;
        }
    }
    __syncthreads();  // (the last sums' readers are through)
    if (lane == 31) {
        s_warp[warp][0] = a;
        s_warp[warp][1] = b;
    }
    __syncthreads();
    if (warp == 0) {
        const bool has = lane < kBatchWarps;
        int64_t x = has ? s_warp[lane][0] : 0, y = has ? s_warp[lane][1] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, x, o),
                          v = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) {
                x += u;
                y += v;
            }
        }
        if (has) {
            s_warp[lane][0] = x;
            s_warp[lane][1] = y;
        }
    }
    __syncthreads();
    if (warp > 0) {
        a += s_warp[warp - 1][0];
        b += s_warp[warp - 1][1];
    }
    return {a, b, s_warp[kBatchWarps - 1][0], s_warp[kBatchWarps - 1][1]};
}

// The first of n nondecreasing sums above x (n if none is).
template <typename I>
__device__ __forceinline__ int first_above(const I* sums, int n, int64_t x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)sums[mid] > x)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// Position and slot of token place j of the step, whose row starts and new lengths are
// `starts` and `lens`.
__device__ __forceinline__ void batch_token(const BatchPlanParams& p, const int32_t* starts,
                                            const int32_t* lens, int j) {
    int pos = 0;
    int64_t slot = -1;
    if (j < starts[p.num_seqs]) {
        const int b = first_above(starts + 1, p.num_seqs, j);
        const int first = starts[b], count = starts[b + 1] - first;
        pos = lens[b] - count + (j - first);
        const int shift = __ffs(p.block_size) - 1;
        const int blk = p.block_tables[(int64_t)b * p.max_blocks_per_seq + (pos >> shift)];
        if (blk < 0 || blk >= p.num_blocks)
            flag_error(p.err_flag, PKV_EFLAG_BLOCK_ID);
        else
            slot = ((int64_t)blk << shift) + (pos & (p.block_size - 1));
    }
    p.positions[j] = pos;
    p.slot_mapping[j] = slot;
}

__global__ void __launch_bounds__(kBatchThreads, 1) batch_plan_kernel(const BatchPlanParams p) {
    __shared__ int64_t s_warp[kBatchWarps][2];
    __shared__ int64_t s_sum[kBatchThreads];
    __shared__ int s_first[kBatchThreads];
    __shared__ int32_t s_starts[kBatchThreads + 1], s_lens[kBatchThreads];
    const int tid = threadIdx.x;
    const bool one_run = p.num_seqs <= kBatchThreads;
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    int bad = 0;
    const int count = p.free_count[0];
    if (count < 0 || count > p.free_capacity) bad |= PKV_EFLAG_POOL;
    int64_t top = min(max(count, 0), p.free_capacity);

    // the released pages, a run of sequences at a time
    BatchSeq s = {};
    for (int b0 = 0; b0 < p.num_seqs; b0 += kBatchThreads) {
        const int b = b0 + tid;
        s = {};
        if (b < p.num_seqs) s = batch_seq(p, b, bad);
        if (!__syncthreads_or(s.back)) continue;  // (none, in most decode steps)
        const Sums sum = block_sums(s.back, 0, s_warp);
        s_sum[tid] = sum.a;
        s_first[tid] = s.first;
        __syncthreads();
        for (int64_t i = tid; i < sum.total_a; i += kBatchThreads) {
            const int w = first_above(s_sum, kBatchThreads, i);
            const int64_t before = w > 0 ? s_sum[w - 1] : 0;
            const int blk = p.block_tables[(int64_t)(b0 + w) * p.max_blocks_per_seq + s_first[w] +
                                           (i - before)];
            if (blk < 0 || blk >= p.num_blocks) bad |= PKV_EFLAG_BLOCK_ID;
            if (top + i < p.free_capacity)
                p.free_blocks[top + i] = blk;
            else
                bad |= PKV_EFLAG_POOL;
        }
        top = min(top + sum.total_a, (int64_t)p.free_capacity);
    }
    __syncthreads();  // the list is whole

    // tokens and pages, in order while both last
    int64_t pages = 0, tokens = 0;  // asked for before this run of sequences
    int64_t taken = 0;              // pages that the served ones take
    int given = 0;                  // tokens that they receive
    for (int b0 = 0; b0 < p.num_seqs; b0 += kBatchThreads) {
        const int b = b0 + tid;
        if (!one_run) {
            int again = 0;
            s = {};
            if (b < p.num_seqs) s = batch_seq(p, b, again);
        }
        const Sums ask = block_sums(s.need, s.add, s_warp);
        const bool served = pages + ask.a <= top && tokens + ask.b <= p.max_tokens;
        if (!served && s.add > 0) bad |= PKV_EFLAG_POOL;
        // (the last one served: all are)
        const bool all = pages + ask.total_a <= top && tokens + ask.total_b <= p.max_tokens;
        const Sums sum =
            all ? ask : block_sums(served ? s.need : 0, served ? s.add : 0, s_warp);
        s_sum[tid] = sum.a;
        s_first[tid] = s.keep == 0 ? 0 : (s.keep - 1) / p.block_size + 1;
        if (b < p.num_seqs) {
            const int next = given + (int)sum.b, len = s.keep + (served ? s.add : 0);
            p.query_starts[b + 1] = next;
            p.new_context_lens[b] = len;
            if (one_run) {  // (the tokens' bisection reads them from here)
                s_starts[tid + 1] = next;
                s_lens[tid] = len;
            }
        }
        __syncthreads();
        for (int64_t i = tid; i < sum.total_a; i += kBatchThreads) {
            const int w = first_above(s_sum, kBatchThreads, i);
            const int64_t before = w > 0 ? s_sum[w - 1] : 0;
            const int blk = p.free_blocks[top - 1 - taken - i];
            if (blk < 0 || blk >= p.num_blocks) bad |= PKV_EFLAG_BLOCK_ID;
            p.block_tables[(int64_t)(b0 + w) * p.max_blocks_per_seq + s_first[w] + (i - before)] =
                blk;
        }
        pages += ask.total_a;
        tokens += ask.total_b;
        taken += sum.total_a;
        given += (int)sum.total_b;
    }
    if (tid == 0) {
        p.query_starts[0] = 0;
        s_starts[0] = 0;
        p.new_free_count[0] = (int)(top - taken);
    }
    if (bad) flag_error(p.err_flag, bad);
    if (p.max_tokens > kBatchOwnTokens) return;
    __syncthreads();
    const int32_t* starts = one_run ? s_starts : p.query_starts;
    const int32_t* lens = one_run ? s_lens : p.new_context_lens;
    for (int j = tid; j < p.max_tokens; j += kBatchThreads) batch_token(p, starts, lens, j);
}

// The row starts are read once, not at every step of a bisection.
constexpr int kSlotsStarts = 2047;
__global__ void __launch_bounds__(256) batch_slots_kernel(const BatchPlanParams p) {
    __shared__ int32_t s_starts[kSlotsStarts + 1];
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const bool few = p.num_seqs <= kSlotsStarts;
    if (few) {
        for (int i = threadIdx.x; i <= p.num_seqs; i += 256) s_starts[i] = p.query_starts[i];
        __syncthreads();
    }
    const int j = blockIdx.x * 256 + threadIdx.x;
    if (j < p.max_tokens)
        batch_token(p, few ? s_starts : p.query_starts, p.new_context_lens, j);
}

static pkv_status launch_batch(void (*kern)(const BatchPlanParams), const BatchPlanParams& p,
                               int ctas, int threads, void* stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
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

extern "C" pkv_status pkv_batch_plan(int32_t* query_starts, int32_t* positions,
                                     int64_t* slot_mapping, int32_t* new_context_lens,
                                     int32_t* new_free_count, const int32_t* context_lens,
                                     const int32_t* new_lens, const int32_t* keep_lens,
                                     const int32_t* shared_pages, int32_t* block_tables,
                                     int max_blocks_per_seq, int32_t* free_blocks,
                                     int free_capacity, const int32_t* free_count, int num_seqs,
                                     int max_tokens, int num_blocks, int block_size,
                                     int32_t* err_flag, void* stream) {
    if (num_seqs < 0 || max_tokens < 0 || max_blocks_per_seq <= 0 || free_capacity < 0 ||
        num_blocks <= 0 || block_size <= 0)
        return PKV_ERR_INVALID_ARG;
    if (!supported_block_size(block_size) || (int64_t)max_blocks_per_seq * block_size > INT_MAX ||
        num_seqs == INT_MAX)
        return PKV_ERR_UNSUPPORTED;
    if (!query_starts || !new_free_count || !free_count ||
        (max_tokens > 0 && (!positions || !slot_mapping)) || (free_capacity > 0 && !free_blocks) ||
        (num_seqs > 0 && (!new_context_lens || !context_lens || !new_lens || !block_tables)))
        return PKV_ERR_INVALID_ARG;
    // everything that is written lies apart from everything else, but for the two
    // that may be updated in place
    const int64_t seqs = num_seqs;
    struct Part {
        const void* at;
        int64_t bytes;
        bool written;
        int place;  // of the pair that may be one
    };
    const Part parts[] = {{query_starts, (seqs + 1) * 4, true, -1},
                          {positions, (int64_t)max_tokens * 4, true, -1},
                          {slot_mapping, (int64_t)max_tokens * 8, true, -1},
                          {new_context_lens, seqs * 4, true, 0},
                          {new_free_count, 4, true, 1},
                          {block_tables, seqs * max_blocks_per_seq * 4, true, -1},
                          {free_blocks, (int64_t)free_capacity * 4, true, -1},
                          {context_lens, seqs * 4, false, 0},
                          {new_lens, seqs * 4, false, -1},
                          {keep_lens, keep_lens ? seqs * 4 : 0, false, -1},
                          {shared_pages, shared_pages ? seqs * 4 : 0, false, -1},
                          {free_count, 4, false, 1}};
    for (const Part& a : parts)
        if (reinterpret_cast<uintptr_t>(a.at) & (a.at == slot_mapping ? 7u : 3u))
            return PKV_ERR_INVALID_ARG;
    for (const Part& a : parts)
        for (const Part& b : parts) {
            if (&a == &b || !a.written || a.bytes == 0 || b.bytes == 0) continue;
            if (a.at == b.at && a.place >= 0 && a.place == b.place) continue;
            if (overlap(a.at, a.bytes, b.at, b.bytes)) return PKV_ERR_INVALID_ARG;
        }
    BatchPlanParams p = {};
    p.query_starts = query_starts;
    p.positions = positions;
    p.slot_mapping = slot_mapping;
    p.new_context_lens = new_context_lens;
    p.new_free_count = new_free_count;
    p.context_lens = context_lens;
    p.new_lens = new_lens;
    p.keep_lens = keep_lens;
    p.shared_pages = shared_pages;
    p.block_tables = block_tables;
    p.free_blocks = free_blocks;
    p.free_count = free_count;
    p.err_flag = err_flag;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.free_capacity = free_capacity;
    p.num_seqs = num_seqs;
    p.max_tokens = max_tokens;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.cap = max_blocks_per_seq * block_size;
    const pkv_status st = launch_batch(batch_plan_kernel, p, 1, kBatchThreads, stream);
    if (st != PKV_OK || max_tokens <= kBatchOwnTokens) return st;
    return launch_batch(batch_slots_kernel, p, (int)(((int64_t)max_tokens + 255) / 256), 256,
                        stream);
}
