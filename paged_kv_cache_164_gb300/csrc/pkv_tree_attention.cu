// Attention of a tree's drafted nodes over a paged KV cache (tcgen05).
//
// The math: node i of sequence b attends to the committed positions
// t < base = n - tree_len and to the nodes j (position base + j) of its mask:
//     s_t = scale * <q_i, K_t>,  out_i = softmax(s) V      over those t
// The (node, query head) rows of one KV head form a dense matrix that meets
// every cached token once, so the two products run on the tensor cores
// (tcgen05, fp32 accumulators in tensor memory), with the online softmax
// between them: running reference m, sum l and accumulator O per row, one
// division at the end.
//
// Tiles: 128 rows x 64 tokens.  Two softmax warpgroups, one thread per row, each
// with two S tiles and an O of its own in tensor memory (all 512 columns):
//   S_w = Q K^T     tcgen05.mma 128 x 64 x D, Q and K from shared memory
//   softmax         a thread reads its row of S, writes P over it
//   O_w += P V      P from tensor memory, as hi + lo 16-bit terms (a single
//                   16-bit P would cost the outputs of short contexts half
//                   their precision), V from shared memory
// A warpgroup's next S is made while it is at its softmax, and the other's
// products run meanwhile: with one S of 128 tokens a warpgroup, which its P
// frees only for the step after, the step was a chain of S, softmax and P V
// (32 nodes over 8 contexts of 82000 tokens, Llama-70B layer: 702 us; so 621 us).
// ROWS: the warpgroups take 128 rows each of the same tokens, so 256 rows meet a
// K/V tile that was read once.  Otherwise they take the same rows and every
// other tile, and meet at the end.  (The rule and both sides' times: plan_tree.)
// Four warps stream the K and V tiles by TMA through the block table into a ring
// of tile slots (a warp takes about 95 cycles to issue a box, and the HBM rate
// leaves 88 for the 2 KB boxes of 16-token pages), and one warp each issues a
// warpgroup's products.
//
// Work: the (sequence, KV head, row block) units' stretches of 128 tokens lie on
// one line, and each of the persistent CTAs (one an SM) takes an equal part of
// it, so ragged contexts and few long ones fill the SMs alike.  A unit inside
// one part is written to the output at once; one that is cut leaves a partial
// (normalised O and its log-sum-exp) per CTA, at most two a CTA, and
// tree_merge_kernel joins them.
//
// What bounds it (times of a few dozen calls, then of calls that go on for seconds,
// where the power cap lowers the clock):
// Up to 128 rows per KV head, memory: 16 nodes on the Llama-70B layer over 8 ragged
// contexts of 33000 to 131000 tokens take 390 to 412 us, then 450, for 2.69 GB (96
// to 102 % of the copy rate, then 88 %), 8 nodes on the Llama-7B layer (16 contexts
// of 520 to 4096) 97 to 101 us, then 100, for 607 MB (89 to 92 %).
// With 256 rows, 32 nodes on the Llama-70B layer (32 x 4096 tokens), 147 us, then
// 166.  No unit is full: the tensor pipe is active 63 % of the time, the memory 48 %.
// The products alone, with P twice, would take 109 at the dense rate (a single 16-bit
// P would take 129 in all); the softmax threads take about as long beside them, and
// the join of the cut units 16.
// Head dim 64 takes as long at the softmax of a score for half the products: the same
// 256 rows 126 us, 128 rows (16 nodes) 75, for floors of 42 and 41; tensor pipe 34 %
// active, 0.53 instructions a cycle and scheduler from its two softmax warps, and a
// token-major cache's rows of 128 bytes read 1.5 times (410 MB of 268).
//
// Every wait is bounded, as in the decode kernels.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <type_traits>

#include "pkv_common.cuh"
#include "pkv_device.cuh"
#include "pkv_tree_parts.cuh"

namespace pkv {

struct TreeParams {
    void* out;
    const void* q;
    const void* v_cache;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* tree_mask;
    int64_t mask_stride;
    int32_t* err_flag;
    int2* unit_ctas;     // per unit: the first and last CTA of its tiles; null: no unit is cut
    float* partial_o;    // [tree_partials(ctas)][rows per unit][D]
    float* partial_lse;  // [tree_partials(ctas)][rows per unit], base 2
    int ctas;            // of the attention kernel
    int max_blocks_per_seq;
    int num_blocks;
    int block_size;
    int num_seqs;
    int num_q_heads;
    int num_kv_heads;
    int group;           // query heads per KV head
    int tree_len;
    int cap;
    int row_blocks;      // units per (sequence, KV head)
    bool hnd;
    float scale_log2;    // |scale| * log2(e) (of 1 where scale is 0)
    float scale_sign;    // 1, -1 or 0
};

constexpr int kTreeRows = 128;                     // rows of a tile (MMA M)
constexpr int kTreeTokens = 64;                    // tokens of a tile
constexpr int kTreePair = 2 * kTreeTokens;         // tokens of a place on the line of work
constexpr int kTreeSoftmaxWarps = 8;               // two warpgroups
constexpr int kTreeTmaWarp = kTreeSoftmaxWarps;    // four producers: K and V of even and odd tiles
constexpr int kTreeMmaWarp = kTreeTmaWarp + 4;     // an issuer for each softmax warpgroup
constexpr int kTreeThreads = (kTreeSoftmaxWarps + 8) * 32;  // the last two warps only fill up
// Registers: the other warpgroups hand over what they do not need, so that a
// softmax thread's row of S and its copies stay in registers (the shares add up
// to the 128 a thread of the launch).
constexpr int kTreeLaunchRegs = 128, kTreeSoftmaxRegs = 184, kTreeOtherRegs = 72;
static_assert(2 * kTreeSoftmaxRegs + 2 * kTreeOtherRegs <= 4 * kTreeLaunchRegs, "register shares");
// Scores may exceed a row's reference by this much (base 2) before it moves: P
// stays below 2^8, and O / l and the log-sum-exp come out the same.
constexpr float kTreeLazyLog2 = 8.f;
constexpr int kTreeBoxes = kTreeTokens / kStageTokens;  // TMA boxes along a tile's tokens
// Marks of stretches with a V that is not finite, a ring of them.  With ROWS the slots
// alone hold the warpgroups together: while one has yet to read the mark of a stretch
// whose slots are free, the other may be at the V of as many stretches further on as
// the ring has room for, two tiles (four slots) each at least.
constexpr int kTreeMarks = 8;

template <int D>
struct TreeTileCfg {
    static constexpr int kRegions = D / 64;                     // 128-byte column blocks
    static constexpr int kQRegionBytes = kTreeRows * 128;
    static constexpr int kQTileBytes = kRegions * kQRegionBytes;
    static constexpr int kRegionBytes = kTreeTokens * 128;
    static constexpr int kSlotBytes = kRegions * kRegionBytes;  // K or V of a tile
    static constexpr int kSlots = D == 128 ? 10 : 16;
    // The output's way through shared memory, 32 rows x 32 columns a warp.  D =
    // 128 leaves no room for it: it takes the Q tile that the stretch is done with.
    static constexpr int kStageBytes = D == 128 ? 0 : kTreeSoftmaxWarps * 4096;
    static constexpr int kXchBytes = 2 * kTreeRows * 8;         // (m, l) of each half and row
    // full[slots], empty[slots], s_full[2][2], p_ready[2][2], pv_done[2][2], drain[2],
    // q_ready[2], met, o_free
    static constexpr int kBarriers = 2 * kSlots + 18;
    static constexpr int kSmemBytes = 2 * kQTileBytes + kSlots * kSlotBytes + kStageBytes +
                                      kXchBytes + kBarriers * 8 + 256;
    static constexpr uint32_t kColO = 4 * kTreeTokens;  // S of (warpgroup, buffer), then O
    static_assert(kSlots / 4 < kTreeMarks, "marks of the stretches that may be under way");
    static_assert(kColO + 2 * D <= 512, "tensor memory layout");
    static_assert(kSmemBytes <= 232448, "shared memory of a CTA");
};

__host__ __device__ inline int tree_tiles(int n) {
    // places on the line (pairs of tiles); an empty context has one of nothing
    return n <= 0 ? 1 : (n - 1) / kTreePair + 1;
}

// A unit costs more than its places: its queries, the first products with
// nothing to run beside, the masked tiles of its nodes, its output.  It counts
// this many places ahead of its own on the line.  Measured for 0, 2, 3 and 4:
// 8 nodes on the Llama-7B layer with ragged contexts 131, 116, 102 and 109 us,
// 63 nodes on a ragged mix of 48 contexts (300 to 9000 tokens) 303, 262, 250 and
// 253 us, 32 nodes on the Llama-70B layer 155, 150, 149 and 152 us.
constexpr int kTreeUnitCost = 3;
__host__ __device__ inline int tree_cost(int n) { return kTreeUnitCost + tree_tiles(n); }

__device__ __forceinline__ int warp_scan(int x) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, x, o);
        if ((threadIdx.x & 31) >= o) x += v;
    }
    return x;
}

// A stretch of one unit's places.
struct TreeSeg {
    int b, g, rb;        // sequence, KV head, row block
    int n;               // context length
    int tile0, tiles;    // first place and places of the stretch
    int unit_tiles;      // the unit's places
};

// Walks a CTA's part of the line of places (sequence, KV head, row block,
// place; the last fastest).  Every thread that takes part walks it by itself.
struct TreeWalk {
    int64_t at, end;
    int b, unit, pos, n;  // pos: in the unit's cost, its places from kTreeUnitCost on

    __device__ __forceinline__ bool next(const TreeParams& p, TreeSeg& s) {
        while (at < end) {
            s.b = b;
            s.n = n;
            s.unit_tiles = tree_tiles(n);
            const int u = unit;
            const int take = (int)min((int64_t)(kTreeUnitCost + s.unit_tiles - pos), end - at);
            s.tile0 = max(0, pos - kTreeUnitCost);
            s.tiles = max(0, pos + take - kTreeUnitCost) - s.tile0;
            at += take;
            pos += take;
            if (pos == kTreeUnitCost + s.unit_tiles) {
                pos = 0;
                if (++unit == p.num_kv_heads * p.row_blocks) {
                    unit = 0;
                    ++b;
                    if (at < end) n = clamped_len(__ldg(p.context_lens + b), p.cap);
                }
            }
            if (s.tiles > 0) {
                s.g = u / p.row_blocks;
                s.rb = u - s.g * p.row_blocks;
                return true;
            }
        }
        return false;
    }
};

// Where tile j of a stretch of nt tiles lies in the ring of slots.  ROWS: one
// ring, which both warpgroups' issuers walk; else a ring for each warpgroup,
// half of the slots (tile j belongs to warpgroup j % 2).  A ring's places are in
// the order in which its issuer takes them, S two steps ahead: K0 K1 V0 K2 V1
// ....  An issuer that took every other place of one ring could meet a slot
// whose fill before the one it waits for is still to come, and a wait by the
// phase's parity would not tell the two apart.
struct TreePlace {
    int slot, phase;
};
template <bool ROWS, int NS>
__device__ __forceinline__ TreePlace tree_place(bool is_v, int place0, int j, int nt) {
    constexpr int kRing = ROWS ? NS : NS / 2;
    const int k = ROWS ? j : j >> 1, n = ROWS ? nt : nt >> 1;  // tile k of the ring's n
    const int at = place0 + (is_v ? min(k + 2, n) + k : (k < 2 ? k : 2 * k - 1));
    return {at % kRing + (ROWS ? 0 : (j & 1) * kRing), at / kRing};
}
// A ring's places in a stretch (a K and a V for each of its tiles).
template <bool ROWS>
__device__ __forceinline__ int tree_places(int nt) { return ROWS ? 2 * nt : nt; }

template <typename T, int D, bool ROWS>
__global__ void __launch_bounds__(kTreeThreads, 1)
tree_attention_kernel(const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const TreeParams p) {
    using Cfg = TreeTileCfg<D>;
    constexpr int R = Cfg::kRegions;
    constexpr int NS = Cfg::kSlots;
    constexpr int TR = kTreeRows;
    constexpr int TT = kTreeTokens;
    constexpr int kUnitRows = ROWS ? 2 * TR : TR;

    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* sq = smem;  // two Q tiles [region][128 rows][128 B], swizzled
    uint8_t* ring = sq + 2 * Cfg::kQTileBytes;
    uint8_t* stage = ring + NS * Cfg::kSlotBytes;
    float2* xch = reinterpret_cast<float2*>(stage + Cfg::kStageBytes);
    uint64_t* full_bar = reinterpret_cast<uint64_t*>(stage + Cfg::kStageBytes + Cfg::kXchBytes);
    uint64_t* empty_bar = full_bar + NS;
    uint64_t* s_full = empty_bar + NS;  // [warpgroup][buffer]
    uint64_t* p_ready = s_full + 4;     // [warpgroup][buffer]
    uint64_t* pv_done = p_ready + 4;    // [warpgroup][buffer]
    uint64_t* drain = pv_done + 4;      // [warpgroup]
    uint64_t* q_ready = drain + 2;      // Q is in place (ROWS: [warpgroup], its rows)
    uint64_t* met = q_ready + 2;        // both warpgroups are through the stretch (not ROWS)
    uint64_t* o_free = met + 1;         // both have read O_0 and O_1 (not ROWS)
    int* words = reinterpret_cast<int*>(full_bar + Cfg::kBarriers);
    volatile int* abort_flag = words;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(words + 1);
    int* s_start = words + 2;           // first sequence, and the first place in its part
    volatile int* s_bad = words + 6;    // [kTreeMarks]: 1 + the stretch (its place: the
                                        // remainder) with a bad V
    int* s_scan = words + 6 + kTreeMarks;  // [16]

    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane = tid & 31;
    const int bs = p.block_size;
    const int bs_shift = __ffs(bs) - 1;
    const int rows = p.tree_len * p.group;

    ptx::launch_dependents();
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            ptx::mbar_init(ptx::smem_addr(&full_bar[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&empty_bar[i]), ROWS ? 2 : 1);  // readers of a tile
        }
        for (int i = 0; i < 4; ++i) {
            ptx::mbar_init(ptx::smem_addr(&s_full[i]), 1);
            ptx::mbar_init(ptx::smem_addr(&p_ready[i]), TR);
            ptx::mbar_init(ptx::smem_addr(&pv_done[i]), 1);
        }
        ptx::mbar_init(ptx::smem_addr(&drain[0]), 1);
        ptx::mbar_init(ptx::smem_addr(&drain[1]), 1);
        ptx::mbar_init(ptx::smem_addr(&q_ready[0]), ROWS ? TR : 2 * TR);
        ptx::mbar_init(ptx::smem_addr(&q_ready[1]), TR);
        ptx::mbar_init(ptx::smem_addr(met), 2 * TR);
        ptx::mbar_init(ptx::smem_addr(o_free), 2 * TR);
        *abort_flag = 0;
        for (int i = 0; i < kTreeMarks; ++i) s_bad[i] = 0;
        ptx::fence_barrier_init();
        ptx::prefetch_tensormap(&tm_k);
        ptx::prefetch_tensormap(&tm_v);
    }
    if (warp == kTreeMmaWarp) {
        ptx::tmem_alloc(ptx::smem_addr(tmem_slot), 512);
        ptx::tmem_relinquish_alloc_permit();
    }
#ifdef PKV_DEBUG
    poison_smem(ring, NS * Cfg::kSlotBytes, tid, kTreeThreads);
#endif
    ptx::grid_dependency_wait();

    // The line of places, and the sequence and the place in it where this CTA's part
    // starts.  Up to 32 sequences a warp scans by itself, a lane a sequence: without
    // the exchange of the block-wide scan a call of two sequences of 50 tokens takes
    // 5.6 us instead of 6.1.
    const int units = p.num_kv_heads * p.row_blocks;
    int64_t line, ctas, start, stop;
    auto parts = [&](int total) {
        line = (int64_t)total * units;
        ctas = min((int64_t)gridDim.x, line);  // with a place at least; the rest idle
        const int64_t x = min((int64_t)blockIdx.x, ctas), y = min((int64_t)blockIdx.x + 1, ctas);
        if (y * line <= UINT_MAX) {  // (a 64-bit division takes several times as long)
            start = (uint32_t)(x * line) / (uint32_t)ctas;
            stop = (uint32_t)(y * line) / (uint32_t)ctas;
        } else {
            start = x * line / ctas;
            stop = y * line / ctas;
        }
    };
    TreeWalk walk;
    int in_seq = 0;  // the first place in its sequence's part of the line
    if (p.num_seqs <= 32) {
        const int n = lane < p.num_seqs ? clamped_len(__ldg(p.context_lens + lane), p.cap) : 0;
        const int mine = lane < p.num_seqs ? tree_cost(n) : 0;
        const int incl = warp_scan(mine);
        parts(__shfl_sync(0xffffffffu, incl, 31));
        // the sequences that end at or before the start (a later CTA than the last has none)
        const uint32_t over =
            __ballot_sync(0xffffffffu, lane < p.num_seqs && (int64_t)incl * units <= start);
        walk.b = min(__popc(over), p.num_seqs - 1);
        walk.n = __shfl_sync(0xffffffffu, n, walk.b);
        in_seq = (int)(start - (int64_t)__shfl_sync(0xffffffffu, incl - mine, walk.b) * units);
        ptx::tc_fence_before_sync();
        __syncthreads();
        ptx::tc_fence_after_sync();
    } else {
        // a thread sums those of a run of sequences, a scan places the runs, and the
        // thread whose run holds this CTA's first place finds its sequence
        const int per = (p.num_seqs + kTreeThreads - 1) / kTreeThreads;
        const int b_lo = min(p.num_seqs, tid * per), b_hi = min(p.num_seqs, b_lo + per);
        int mine = 0;  // the host checks that all sequences' costs fit an int
        for (int b = b_lo; b < b_hi; ++b)
            mine += tree_cost(clamped_len(__ldg(p.context_lens + b), p.cap));
        const int incl = warp_scan(mine);
        if (lane == 31) s_scan[warp] = incl;
        ptx::tc_fence_before_sync();
        __syncthreads();
        ptx::tc_fence_after_sync();
        int total = 0, before = incl - mine;
        for (int w = 0; w < kTreeThreads / 32; ++w) {
            if (w < warp) before += s_scan[w];
            total += s_scan[w];
        }
        parts(total);
        if (start >= (int64_t)before * units && start < (int64_t)(before + mine) * units) {
            int b = b_lo;
            int64_t first = (int64_t)before * units;
            while (true) {
                const int64_t next = first + (int64_t)units * tree_cost(clamped_len(
                                                 __ldg(p.context_lens + b), p.cap));
                if (start < next) break;
                first = next;
                ++b;
            }
            s_start[0] = b;
            s_start[1] = (int)(start - first);
        }
        __syncthreads();
        if (start < stop) {
            walk.b = s_start[0];
            walk.n = clamped_len(__ldg(p.context_lens + walk.b), p.cap);
            in_seq = s_start[1];
        }
    }
    const uint32_t tmem = *tmem_slot;
    const uint32_t ring_addr = ptx::smem_addr(ring);
    const uint32_t q_addr = ptx::smem_addr(sq);

    walk.at = start;
    walk.end = stop;
    if (start < stop) {
        const int cost = tree_cost(walk.n);
        walk.unit = in_seq / cost;
        walk.pos = in_seq - walk.unit * cost;
    }

    if (warp >= kTreeSoftmaxWarps) {
        ptx::reg_dec<kTreeOtherRegs>();
        TreeSeg seg;
        if (warp < kTreeMmaWarp) {
            // ------------------------------------------------------------ producers
            // A warp loads the K or the V of every other tile; a lane issues one box
            // (16 tokens x 64 dims).
            const bool is_v = warp & 1;
            const int odd = (warp - kTreeTmaWarp) >> 1;
            const CUtensorMap* map = is_v ? &tm_v : &tm_k;
            const uint64_t policy =
                p.row_blocks > 1 ? ptx::l2_policy_evict_last() : ptx::l2_policy_evict_first();
            const int bx = lane / R, rr = lane % R;
            const bool loads = lane < kTreeBoxes * R;
            int place0 = 0;      // a ring's places of the stretches before this one
            uint64_t filled = 0; // slots with a copy of this warp's that may be in flight,
            uint64_t parity = 0; // and its phase's parity
            bool ok = true;
            while (ok && walk.next(p, seg)) {
                const int nt = 2 * seg.tiles;
                const int32_t* table = p.block_tables + (int64_t)seg.b * p.max_blocks_per_seq;
                if (p.unit_ctas != nullptr && warp == kTreeTmaWarp && lane == 0 &&
                    seg.tile0 == 0) {
                    // the unit's first and last CTA: cost position u of the line belongs to
                    // the last CTA c with c * line < (u + 1) * CTAs.  The unit's first
                    // place may lie behind this CTA's first position in it.
                    const int64_t last = walk.at + (seg.unit_tiles - seg.tiles);  // one past it
                    p.unit_ctas[((int64_t)seg.b * p.num_kv_heads + seg.g) * p.row_blocks +
                                seg.rb] =
                        make_int2(blockIdx.x, (int)((last * ctas - 1) / line));
                }
                if (warp == kTreeTmaWarp + 1 && lane == 0 && seg.tile0 == 0 && seg.g == 0 &&
                    seg.rb == 0) {
                    const int n_raw = __ldg(p.context_lens + seg.b);
                    if (n_raw < 0 || n_raw > p.cap || (n_raw != 0 && n_raw < p.tree_len))
                        flag_error(p.err_flag, PKV_EFLAG_CONTEXT_LEN);
                }
                // the block of this lane's box of tile j, as the table has it (-1: none)
                auto box_block = [&](int j) {
                    const int tok = seg.tile0 * kTreePair + j * TT + bx * kStageTokens;
                    return loads && j < nt && tok < seg.n ? __ldg(table + (tok >> bs_shift)) : -1;
                };
                auto load = [&](int j, int blk) {
                    const int tok = seg.tile0 * kTreePair + j * TT + bx * kStageTokens;
                    if (blk < 0 || blk >= p.num_blocks) {
                        if (!is_v && loads && tok < seg.n)
                            flag_error(p.err_flag, PKV_EFLAG_BLOCK_ID);
                        blk = -1;
                    }
                    const auto [slot, phase] = tree_place<ROWS, NS>(is_v, place0, j, nt);
                    if (phase > 0 && !warp_wait_phase(ptx::smem_addr(&empty_bar[slot]),
                                                      (phase - 1) & 1, abort_flag, p.err_flag))
                        return false;
#ifdef PKV_DEBUG
                    if (phase > 0) {
                        ptx::tc_fence_after_sync();
                        poison_smem(ring + slot * Cfg::kSlotBytes, Cfg::kSlotBytes, lane, 32);
                        __syncwarp();
                    }
#endif
                    const uint32_t fb = ptx::smem_addr(&full_bar[slot]);
                    const uint32_t boxes = __ballot_sync(0xffffffffu, blk >= 0);
                    if (lane == 0) {
                        if (boxes == 0)
                            ptx::mbar_arrive(fb);  // every token of the tile is masked
                        else
                            ptx::mbar_arrive_expect_tx(fb, __popc(boxes) * kStageTokens * 128);
                    }
                    __syncwarp();
                    if (blk >= 0) {
                        load_kv_box(ring_addr + slot * Cfg::kSlotBytes + rr * Cfg::kRegionBytes +
                                        bx * kStageTokens * 128,
                                    map, fb, rr * 64, seg.g, tok & (bs - 1), blk, p.hnd, policy);
                    }
                    filled |= 1ull << slot;
                    parity = (parity & ~(1ull << slot)) | ((uint64_t)(phase & 1) << slot);
                    return true;
                };
                // read a turn ahead: a table entry takes about as long as a tile's turn
                int blk = box_block(odd), blk_next = box_block(odd + 2);
                for (int j = odd; j < nt && ok; j += 2) {
                    const int far = box_block(j + 4);
                    ok = load(j, blk);
                    blk = blk_next;
                    blk_next = far;
                }
                place0 += tree_places<ROWS>(nt);
            }
            if (lane == 0 && *abort_flag) {
                // wait (bounded) for this warp's copies in flight before leaving
                const uint64_t t0 = ptx::globaltimer();
                for (int i = 0; i < NS; ++i) {
                    if (!((filled >> i) & 1)) continue;
                    while (!ptx::mbar_try_wait(ptx::smem_addr(&full_bar[i]),
                                               (uint32_t)(parity >> i) & 1u) &&
                           ptx::globaltimer() - t0 < kWaitLimitNs) {
                    }
                }
            }
        } else if (warp < kTreeMmaWarp + 2) {
            // ------------------------------------------------------------ MMA issuers
            // One warp per softmax warpgroup.  The whole warp walks the steps, so
            // that addresses and descriptors are uniform values; one elected lane
            // issues.  (One lane alone walking them took 110 cycles a product to
            // issue, of the 64 that it runs.)
            constexpr uint32_t fmt = F16Format<T>::value;
            constexpr uint32_t idesc_s = mma_idesc(fmt, TR, TT, false);
            constexpr uint32_t idesc_o = mma_idesc(fmt, TR, D, true);
            const int w = __shfl_sync(0xffffffffu, warp - kTreeMmaWarp, 0);
            // descriptors of the first slots: a byte offset adds its sixteenth (the
            // address field stays within its 14 bits: shared memory is 228 KB)
            const uint64_t qdesc = ptx::smem_desc_sw128(q_addr, 16, 1024);
            const uint64_t kdesc = ptx::smem_desc_sw128(ring_addr, 16, 1024);
            const uint64_t vdesc = ptx::smem_desc_sw128(ring_addr, Cfg::kRegionBytes, 1024);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t acc_o = tm + Cfg::kColO + w * D;
            int place0 = 0, nseg = 0;
            int step0 = 0;  // this warpgroup's steps before the stretch
            bool ok = true;
            while (ok && walk.next(p, seg)) {
                const int nt = __shfl_sync(0xffffffffu, 2 * seg.tiles, 0);
                const int steps = ROWS ? nt : nt / 2;  // step k: tile k, or tile 2k + w
                auto wait = [&](uint64_t* bar, int parity) {
                    return warp_wait_phase(ptx::smem_addr(bar), parity & 1, abort_flag,
                                           p.err_flag);
                };
                auto issue_s = [&](int k) {
                    const auto [slot, phase] =
                        tree_place<ROWS, NS>(false, place0, ROWS ? k : 2 * k + w, nt);
                    const int buf = (step0 + k) & 1;
                    if (!wait(&full_bar[slot], phase)) return false;
                    ptx::tc_fence_after_sync();
                    const uint64_t kd = kdesc + (uint32_t)(slot * (Cfg::kSlotBytes / 16));
                    const uint64_t qd =
                        qdesc + (uint32_t)((ROWS ? w : nseg & 1) * (Cfg::kQTileBytes / 16));
                    const uint32_t acc = tm + (2 * w + buf) * TT;
                    if (ptx::elect_one()) {
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks)
                            ptx::tc_mma_f16(
                                acc, qd + (ks / 4) * (Cfg::kQRegionBytes / 16) + (ks % 4) * 2,
                                kd + (ks / 4) * (Cfg::kRegionBytes / 16) + (ks % 4) * 2, idesc_s,
                                ks > 0 ? 1u : 0u);
                        ptx::tc_commit(ptx::smem_addr(&s_full[2 * w + buf]));
                        ptx::tc_commit(ptx::smem_addr(&empty_bar[slot]));
                    }
                    __syncwarp();
                    return true;
                };
                auto issue_pv = [&](int k) {
                    const auto [slot, phase] =
                        tree_place<ROWS, NS>(true, place0, ROWS ? k : 2 * k + w, nt);
                    const int buf = (step0 + k) & 1;
                    if (!wait(&full_bar[slot], phase) ||
                        !wait(&p_ready[2 * w + buf], (step0 + k) >> 1))
                        return false;
                    ptx::tc_fence_after_sync();
                    const uint64_t vd = vdesc + (uint32_t)(slot * (Cfg::kSlotBytes / 16));
                    const uint32_t pt = tm + (2 * w + buf) * TT;
                    if (ptx::elect_one()) {
#pragma unroll
                        for (int kt = 0; kt < TT / 16; ++kt) {
                            // tokens 16 kt ..: of each 32 tokens of P, 16 columns of hi
                            // pairs, then 16 of lo pairs
                            const uint32_t a = pt + (kt / 2) * 32 + (kt % 2) * 8;
                            const uint64_t v = vd + (uint32_t)(kt * 16 * 128 / 16);
                            ptx::tc_mma_f16_ts(acc_o, a, v, idesc_o, (k > 0 || kt > 0) ? 1u : 0u);
                            ptx::tc_mma_f16_ts(acc_o, a + 16, v, idesc_o, 1u);
                        }
                        ptx::tc_commit(ptx::smem_addr(&pv_done[2 * w + buf]));
                        ptx::tc_commit(ptx::smem_addr(&empty_bar[slot]));
                    }
                    __syncwarp();
                    return true;
                };
                // The tensor core runs a warp's products in the order of their issue:
                // S over a buffer's P comes after the O += P V that reads it.
                // ROWS: a warpgroup's rows of Q are its own, and it need not wait for the other's
                ok = wait(&q_ready[ROWS ? w : 0], nseg) && issue_s(0) && (steps < 2 || issue_s(1));
                for (int k = 0; k < steps && ok; ++k)
                    ok = issue_pv(k) && (k + 2 >= steps || issue_s(k + 2));
                place0 += tree_places<ROWS>(nt);
                step0 += steps;
                ++nseg;
            }
            // every product has completed before the tensor memory is released
            if (ptx::elect_one()) ptx::tc_commit(ptx::smem_addr(&drain[w]));
            __syncwarp();
            const uint64_t t0 = ptx::globaltimer();
            while (!ptx::mbar_try_wait(ptx::smem_addr(&drain[w]), 0) &&
                   ptx::globaltimer() - t0 < kWaitLimitNs) {
            }
        }
    } else {
        // ------------------------------------------------------------ softmax rows
        ptx::reg_inc<kTreeSoftmaxRegs>();
        const int wg = warp / 4;                  // warpgroup
        const int srow = 32 * (warp % 4) + lane;  // row of the tile = tensor-memory lane
        const uint32_t lane_base = (uint32_t)(32 * (warp % 4)) << 16;
        const uint32_t o_col = tmem + lane_base + Cfg::kColO;
        const int urow = ROWS ? wg * TR + srow : srow;  // row of the unit
        int place0 = 0, nseg = 0;
        int step = 0;  // this warpgroup's steps so far
        bool ok = true;

        // Query row r of the unit: node r / group, head g * group + r % group; its
        // place in the (node, query head) rows of the sequence, or -1 past them.
        auto row_of = [&](const TreeSeg& s, int& node) {
            const int r = s.rb * kUnitRows + urow;
            if (r >= rows) {
                node = 0;
                return -1;
            }
            node = r / p.group;
            return node * p.num_q_heads + s.g * p.group + r - node * p.group;
        };
        auto q_row = [&](const TreeSeg& s, int rel) {
            return reinterpret_cast<const uint4*>(
                static_cast<const T*>(p.q) +
                ((int64_t)s.b * p.tree_len * p.num_q_heads + max(rel, 0)) * D);
        };
        // where 16-byte chunk c of this thread's row lies in a Q tile
        auto q_chunk = [&](int c) {
            return (c / 8) * Cfg::kQRegionBytes + srow * 128 + (((c % 8) ^ (srow & 7)) << 4);
        };
        // not ROWS: this thread's half of its row of Q into the Q tile of stretch `which`
        auto load_q_half = [&](const TreeSeg& s, int which) {
            int node;
            const int rel = row_of(s, node);
            const uint4* src = q_row(s, rel);
            const uint32_t dst = q_addr + (which & 1) * Cfg::kQTileBytes;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const int c = wg * (D / 16) + k;
                ptx::cp_async_16(dst + q_chunk(c), src + c, rel >= 0);
            }
        };
        // ROWS: its row of Q into Q tile wg.  Where the output leaves by way of the Q
        // tile's first region, that region's part waits in registers until it has.
        constexpr int QH = ROWS && D == 128 ? 8 : 1;
        uint4 held[QH];
        auto load_q_row = [&](const TreeSeg& s) {
            int node;
            const int rel = row_of(s, node);
            const uint4* src = q_row(s, rel);
#pragma unroll
            for (int c = D == 128 ? 8 : 0; c < D / 8; ++c)
                ptx::cp_async_16(q_addr + wg * Cfg::kQTileBytes + q_chunk(c), src + c, rel >= 0);
            if constexpr (QH > 1) {
#pragma unroll
                for (int c = 0; c < QH; ++c)
                    held[c] = rel >= 0 ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
            }
        };
        auto q_loaded = [&] {
            if constexpr (QH > 1) {
#pragma unroll
                for (int c = 0; c < QH; ++c)
                    *reinterpret_cast<uint4*>(sq + wg * Cfg::kQTileBytes + q_chunk(c)) = held[c];
            }
            ptx::cp_async_wait_all();
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(ptx::smem_addr(&q_ready[ROWS ? wg : 0]));
        };

        TreeSeg s, next;
        bool have = walk.next(p, s);
        if (have) {
            if constexpr (ROWS)
                load_q_row(s);
            else
                load_q_half(s, 0);
            q_loaded();
        }
        while (have && ok) {
            const int base = s.n - p.tree_len;
            int node;
            const int rel = row_of(s, node);
            const bool live = rel >= 0;
            const bool warp_live = __any_sync(0xffffffffu, live);
            // the next stretch's Q is on its way long before it is needed (its tile
            // belonged to the stretch before this one)
            const bool have_next = walk.next(p, next);
            if (!ROWS && have_next) load_q_half(next, nseg + 1);
            const int mask_words = (p.tree_len + 31) / 32;
            const int32_t* mask = p.tree_mask + s.b * p.mask_stride + (int64_t)node * mask_words;
            // bits of nodes jb .. jb + 31 (below 0: committed positions)
            auto tree_bits = [&](int jb) -> uint32_t {
                if (jb <= -32) return ~0u;
                const int w = jb >> 5;
                const uint32_t lo = w < 0 ? ~0u : w < mask_words ? (uint32_t)__ldg(mask + w) : 0u;
                const uint32_t hi = w + 1 < 0 ? ~0u
                                    : w + 1 < mask_words ? (uint32_t)__ldg(mask + w + 1)
                                                         : 0u;
                return __funnelshift_r(lo, hi, jb & 31);
            };
            const int nt = 2 * s.tiles;
            const int tok0 = s.tile0 * kTreePair;
            const int32_t* table = p.block_tables + (int64_t)s.b * p.max_blocks_per_seq;
            // lanes 0-3: the block of box `lane` of tile j, as the table has it (-1: none)
            auto box_block = [&](int j) {
                const int tok = tok0 + j * TT + lane * kStageTokens;
                return lane < kTreeBoxes && j < nt && tok < s.n ? __ldg(table + (tok >> bs_shift))
                                                                : -1;
            };

            float m_ref = -INFINITY, l = 0.f;
            constexpr int kStep = ROWS ? 1 : 2;
            const int j0 = ROWS ? 0 : wg;
            int blk = box_block(j0), blk_next = box_block(j0 + kStep);  // two steps ahead
            for (int j = j0; j < nt; j += kStep, ++step) {
                const uint32_t boxes = __ballot_sync(0xffffffffu, blk >= 0 && blk < p.num_blocks);
                blk = blk_next;
                blk_next = box_block(j + 2 * kStep);
                const int buf = step & 1;
                const uint32_t s_col = tmem + lane_base + (2 * wg + buf) * TT;
                const int t0 = tok0 + j * TT;
                const bool plain = boxes == (1u << kTreeBoxes) - 1u && t0 + TT <= s.n &&
                                   t0 + TT <= base;
                if (!warp_wait_phase(ptx::smem_addr(&s_full[2 * wg + buf]), (step >> 1) & 1,
                                     abort_flag, p.err_flag)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after_sync();
                if (!plain) {
                    // V rows of absent tokens hold stale bytes, and a node's V may hold
                    // infinities or NaN that only some rows attend to: zeroed in
                    // shared memory, so that 0 * V is 0; the rows that do attend to
                    // such a value get it back at the end.
                    const auto [slot, phase] = tree_place<ROWS, NS>(true, place0, j, nt);
                    if (!warp_wait_phase(ptx::smem_addr(&full_bar[slot]), phase & 1, abort_flag,
                                         p.err_flag)) {
                        ok = false;
                        break;
                    }
                    uint8_t* vst = ring + slot * Cfg::kSlotBytes;
                    const int row0 = boxes == (1u << kTreeBoxes) - 1u
                                         ? min(max(0, min(base, s.n) - t0), TT)
                                         : 0;
                    for (int idx = row0 * R * 8 + srow; idx < TT * R * 8; idx += TR) {
                        const int row = idx / (R * 8), rem = idx - row * (R * 8);
                        uint4* cell = reinterpret_cast<uint4*>(
                            vst + (rem / 8) * Cfg::kRegionBytes + row * 128 + (rem % 8) * 16);
                        if (t0 + row >= s.n || !((boxes >> (row / kStageTokens)) & 1u)) {
                            *cell = make_uint4(0u, 0u, 0u, 0u);
                        } else if (t0 + row >= base) {
                            uint4 x = *cell;
                            const uint32_t bad = drop_not_finite(x.x, T()) |
                                                 drop_not_finite(x.y, T()) |
                                                 drop_not_finite(x.z, T()) |
                                                 drop_not_finite(x.w, T());
                            if (bad) {
                                s_bad[nseg % kTreeMarks] = nseg + 1;
                                __threadfence_block();  // before the value is gone
                                *cell = x;
                            }
                        }
                    }
                    ptx::fence_proxy_async_smem();
                }
                if (!ROWS && j == j0 && nseg > 0 &&
                    !warp_wait_phase(ptx::smem_addr(o_free), (nseg - 1) & 1, abort_flag,
                                     p.err_flag)) {
                    // both warpgroups read O_0, O_1 and the exchanged (m, l) of the
                    // stretch before; neither is written anew until both have
                    ok = false;
                    break;
                }
                if (warp_live) {
                    float sc[TT];
                    {
                        uint32_t(&r0)[32] = *reinterpret_cast<uint32_t(*)[32]>(sc);
                        uint32_t(&r1)[32] = *reinterpret_cast<uint32_t(*)[32]>(sc + 32);
                        __syncwarp();
                        ptx::tmem_ld32_async(s_col, r0);
                        ptx::tmem_ld32_async(s_col + 32, r1);
                        ptx::tmem_wait_ld();
                        ptx::tmem_loaded(r0);
                        ptx::tmem_loaded(r1);
                    }
                    if (p.scale_sign != 1.f) {
#pragma unroll
                        for (int i = 0; i < TT; ++i) sc[i] *= p.scale_sign;
                    }
                    if (!plain) {
#pragma unroll
                        for (int c = 0; c < TT / 32; ++c) {
                            const int tc = t0 + c * 32;
                            const int left = s.n - tc;
                            uint32_t allow = left >= 32 ? ~0u : left <= 0 ? 0u : (1u << left) - 1u;
                            const uint32_t bb = boxes >> (2 * c);
                            allow &= ((bb & 1u) ? 0x0000ffffu : 0u) |
                                     ((bb & 2u) ? 0xffff0000u : 0u);
                            allow &= tree_bits(tc - base);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!((allow >> i) & 1u)) sc[c * 32 + i] = -INFINITY;
                        }
                    }
                    float mx[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) mx[c] = fmaxf(sc[2 * c], sc[2 * c + 1]);
#pragma unroll
                    for (int i = 8; i < TT; i += 2)
                        mx[(i / 2) % 4] = fmaxf(fmaxf(mx[(i / 2) % 4], sc[i]), sc[i + 1]);
                    const float top =
                        fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
                    float alpha = 1.f;
                    if (m_ref == -INFINITY) {
                        m_ref = top;  // O and l are still zero for this row
                    } else if (top > m_ref + kTreeLazyLog2) {
                        alpha = ptx::ex2_approx(m_ref - top);
                        m_ref = top;
                    }
                    const float ref = (m_ref == -INFINITY ? 0.f : m_ref) - WeightBias<T>::value;
                    // O is rescaled when a reference moved, once the last O += P V has
                    // completed (that of the step before it has: S of this step is
                    // complete, and was issued behind it)
                    if (__any_sync(0xffffffffu, alpha != 1.f)) {
                        if (!warp_wait_phase(ptx::smem_addr(&pv_done[2 * wg + (buf ^ 1)]),
                                             ((step - 1) >> 1) & 1, abort_flag, p.err_flag)) {
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after_sync();
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t ov[32];
                            __syncwarp();
                            ptx::tmem_ld32(o_col + wg * D + c * 32, ov);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                            ptx::tmem_st32(o_col + wg * D + c * 32, ov);
                        }
                        l *= alpha;
                    }
                    const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
                    const float2 ref2 = make_float2(-ref, -ref);
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int c = 0; c < TT / 32; ++c) {
                        uint32_t pv[32];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int i = c * 32 + 2 * e;
                            float2 y = ptx::fma2(make_float2(sc[i], sc[i + 1]), scale2, ref2);
                            y.x = ptx::ex2_approx(y.x);
                            y.y = ptx::ex2_approx(y.y);
                            sum[e % 2] = ptx::add2(sum[e % 2], y);
                            split_pair(y, pv[e], pv[16 + e], T());
                        }
                        ptx::tmem_st32_async(s_col + c * 32, pv);
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                    ptx::tmem_wait_st();
                }
                ptx::tc_fence_before_sync();
                ptx::mbar_arrive(ptx::smem_addr(&p_ready[2 * wg + buf]));
            }
            if (!ok) break;
            place0 += tree_places<ROWS>(nt);
            if (have_next) {
                if constexpr (ROWS)
                    load_q_row(next);
                else
                    q_loaded();
            }

            // the stretch's last O += P V
            if (!warp_wait_phase(ptx::smem_addr(&pv_done[2 * wg + ((step - 1) & 1)]),
                                 ((step - 1) >> 1) & 1, abort_flag, p.err_flag))
                break;
            float fa, fb = 0.f, lse;  // out = O_0 fa + O_1 fb (ROWS: O_w fa)
            if constexpr (ROWS) {
                fa = l == 0.f ? 0.f : 1.f / l;
                lse = l == 0.f ? -INFINITY : m_ref - WeightBias<T>::value + log2f(l);
            } else {
                // both warpgroups are through: their halves of the softmax meet
                xch[wg * TR + srow] = make_float2(m_ref, l);
                ptx::mbar_arrive(ptx::smem_addr(met));
                if (!warp_wait_phase(ptx::smem_addr(met), nseg & 1, abort_flag, p.err_flag)) break;
                const float2 ha = xch[srow], hb = xch[TR + srow];
                const float mm = fmaxf(ha.x, hb.x);
                fa = ha.x == -INFINITY ? 0.f : ptx::ex2_approx(ha.x - mm);
                fb = hb.x == -INFINITY ? 0.f : ptx::ex2_approx(hb.x - mm);
                const float sum = ha.y * fa + hb.y * fb;
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                fa *= inv;
                fb *= inv;
                lse = sum == 0.f ? -INFINITY : mm - WeightBias<T>::value + log2f(sum);
            }
            ptx::tc_fence_after_sync();
            const bool direct = s.tiles == s.unit_tiles;
            const int slot = tree_partial(blockIdx.x, s.tile0 == 0);
            const bool bad_v = s_bad[nseg % kTreeMarks] == nseg + 1;
            // Columns: ROWS: the whole row; else this warpgroup's half.  They leave
            // through shared memory, 32 at a time, so that a warp writes whole lines
            // (a row a thread: 4 cycles of the load/store unit for every one).
            constexpr int kCols = ROWS ? D : D / 2;
            const int col0 = ROWS ? 0 : wg * kCols;
            uint8_t* tray = D == 128
                                ? sq + (ROWS ? wg : nseg & 1) * Cfg::kQTileBytes +
                                      (ROWS ? 0 : wg) * Cfg::kQRegionBytes + (warp % 4) * 4096
                                : stage + warp * 4096;
#pragma unroll 1
            for (int c = 0; c < kCols; c += 32) {
                if (!warp_live) break;
                float v[32];
                uint32_t ov[32];
                __syncwarp();
                ptx::tmem_ld32(o_col + (ROWS ? wg * D : 0) + col0 + c, ov);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(ov[i]) * fa;
                if constexpr (!ROWS) {
                    ptx::tmem_ld32(o_col + D + col0 + c, ov);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = fmaf(__uint_as_float(ov[i]), fb, v[i]);
                }
                if (live && bad_v) {
                    // infinities and NaN in the V of nodes that this row attends to
                    const int t_hi = min(s.n, tok0 + nt * TT);
                    for (int t = max(max(0, base), tok0); t < t_hi; ++t) {
                        const int j = t - base;
                        if (!((__ldg(mask + (j >> 5)) >> (j & 31)) & 1)) continue;
                        const int blk = __ldg(table + (t >> bs_shift));
                        if (blk < 0 || blk >= p.num_blocks) continue;
                        const int off = t & (bs - 1);
                        const uint16_t* vr =
                            static_cast<const uint16_t*>(p.v_cache) +
                            (p.hnd ? ((int64_t)blk * p.num_kv_heads + s.g) * bs + off
                                   : ((int64_t)blk * bs + off) * p.num_kv_heads + s.g) * D +
                            col0 + c;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const uint16_t e = __ldg(vr + i);
                            if (not_finite(e, T())) v[i] += unpack2(e, T()).x;
                        }
                    }
                }
                // row `lane` of the tray, 16-byte chunk i at i ^ (row % 8)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<float4*>(tray + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                        make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                __syncwarp();
                auto chunk = [&](int row, int i) {
                    return *reinterpret_cast<const float4*>(tray + row * 128 +
                                                            ((i ^ (row & 7)) << 4));
                };
                // everything is read before the first store, which might alias it for all
                // that the compiler knows (900 cycles a turn of partials, so 650 to 700;
                // 32 nodes on the Llama-70B layer 154 us, so 148, of a few dozen calls)
                if (direct) {
                    const int64_t first = (int64_t)s.b * p.tree_len * p.num_q_heads;
                    uint4 x[4];
                    int rr[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {  // 8 rows of 32 columns at a time
                        const int row = i * 8 + lane / 4, q4 = lane % 4;
                        rr[i] = __shfl_sync(0xffffffffu, rel, row);
                        const float4 lo = chunk(row, 2 * q4), hi = chunk(row, 2 * q4 + 1);
                        x[i] = make_uint4(pack2(lo.x, lo.y, T()), pack2(lo.z, lo.w, T()),
                                          pack2(hi.x, hi.y, T()), pack2(hi.z, hi.w, T()));
                    }
                    uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + first * D +
                                                          col0 + c) + lane % 4;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (rr[i] >= 0) out[(int64_t)rr[i] * (D / 8)] = x[i];
                } else {
                    float4* part = reinterpret_cast<float4*>(
                                       p.partial_o +
                                       ((int64_t)slot * kUnitRows + urow - lane) * D + col0 + c) +
                                   lane % 8;
                    float4 x[8];
                    int rr[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {  // 4 rows
                        const int row = i * 4 + lane / 8;
                        rr[i] = __shfl_sync(0xffffffffu, rel, row);
                        x[i] = chunk(row, lane % 8);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (rr[i] >= 0) part[(i * 4 + lane / 8) * (D / 4)] = x[i];
                }
            }
            if (live && !direct && (ROWS || wg == 0))
                p.partial_lse[(int64_t)slot * kUnitRows + urow] = lse;
            if constexpr (ROWS) {
                __syncwarp();
                if (have_next) q_loaded();
            } else {
                ptx::tc_fence_before_sync();
                ptx::mbar_arrive(ptx::smem_addr(o_free));
            }
            ++nseg;
            s = next;
            have = have_next;
        }
        // a warp that gave up a wait may have the next stretch's queries on their way
        ptx::cp_async_wait_all();
    }

    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == kTreeMmaWarp) {
        __syncwarp();
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// Joins the partials of the units that were cut: w_c = 2^(lse_c - max),
// out = sum_c w_c O_c / sum_c w_c over the CTAs of the unit, with a running
// maximum.  Eight lanes take a row's columns, all of two partials' loads in flight
// at once (a warp a row, one partial after another, took 20 us for the 65536 rows
// of 32 nodes on the Llama-70B layer), and G such groups share a row's partials
// where rows are few: launch_tree_t has the rule.
constexpr int kTreeMergeThreads = 128;
constexpr int kTreeMergeGroups = kTreeMergeThreads / 8;

template <int E>
struct TreeSum {  // of partials: O's 4 E columns of a lane, weights to base 2^m
    float m, den;
    float4 acc[E];

    __device__ __forceinline__ void scale(float f) {
        den *= f;
#pragma unroll
        for (int e = 0; e < E; ++e)  // a zero weight adds nothing, whatever it weighs
            acc[e] = f == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                              : make_float4(acc[e].x * f, acc[e].y * f, acc[e].z * f,
                                            acc[e].w * f);
    }
    __device__ __forceinline__ void add(float w, const float4 (&x)[E]) {
        den += w;
        if (w == 0.f) return;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            acc[e].x = fmaf(w, x[e].x, acc[e].x);
            acc[e].y = fmaf(w, x[e].y, acc[e].y);
            acc[e].z = fmaf(w, x[e].z, acc[e].z);
            acc[e].w = fmaf(w, x[e].w, acc[e].w);
        }
    }
};

template <typename T, int D, int G>
__global__ void __launch_bounds__(kTreeMergeThreads)
tree_merge_kernel(const TreeParams p, int unit_rows) {
    constexpr int E = D / 32;  // float4 columns of a lane: 8 k + lane % 8
    static_assert(G == 1 || G == 4 || G == kTreeMergeGroups, "a group, a warp or a CTA a row");
    ptx::launch_dependents();
    const int q8 = threadIdx.x & 7;
    const int group = threadIdx.x >> 3;
    // (rows fit 30 bits: 65535 sequences and KV heads, 1024 nodes, groups of 16)
    const uint32_t row = blockIdx.x * (kTreeMergeGroups / G) + group / G;
    const uint32_t bi = row / p.num_q_heads, h = row - bi * p.num_q_heads;
    const uint32_t b = bi / p.tree_len, node = bi - b * p.tree_len;
    const uint32_t g = h / p.group;
    const uint32_t r = node * p.group + h - g * p.group;
    const uint32_t rb = r / unit_rows;
    const int urow = (int)(r - rb * unit_rows);
    ptx::grid_dependency_wait();
    if (b >= (uint32_t)p.num_seqs) return;
    const int2 ctas = __ldg(p.unit_ctas + ((int64_t)b * p.num_kv_heads + g) * p.row_blocks + rb);
    if (ctas.x == ctas.y) return;  // written whole
    if (!tree_parts_valid(ctas.x, ctas.y, p.ctas)) return;  // a wait expired: flagged there
    TreeSum<E> sum;
    sum.m = -INFINITY;
    sum.den = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) sum.acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = ctas.x + 2 * (group % G); c <= ctas.y; c += 2 * G) {
        // a unit's first CTA leaves its last partial, the others their first
        const bool two = c < ctas.y;
        const int64_t at0 = (int64_t)tree_partial(c, c == ctas.x) * unit_rows + urow;
        const int64_t at1 = two ? (int64_t)tree_partial(c + 1, false) * unit_rows + urow : at0;
        const float lse0 = __ldg(p.partial_lse + at0);
        const float lse1 = two ? __ldg(p.partial_lse + at1) : -INFINITY;
        const float4* o0 = reinterpret_cast<const float4*>(p.partial_o + at0 * D) + q8;
        const float4* o1 = reinterpret_cast<const float4*>(p.partial_o + at1 * D) + q8;
        float4 x[E], y[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] = __ldg(o0 + 8 * e);
            y[e] = __ldg(o1 + 8 * e);
        }
        const float mn = fmaxf(sum.m, fmaxf(lse0, lse1));
        const float ref = mn == -INFINITY ? 0.f : mn;
        sum.scale(exp2f(sum.m - ref));
        sum.m = mn;
        sum.add(exp2f(lse0 - ref), x);
        sum.add(exp2f(lse1 - ref), y);
    }
    if constexpr (G > 1) {  // a warp's four groups
        const float mw = fmaxf(sum.m, __shfl_xor_sync(0xffffffffu, sum.m, 8));
        const float mn = fmaxf(mw, __shfl_xor_sync(0xffffffffu, mw, 16));
        sum.scale(exp2f(sum.m - (mn == -INFINITY ? 0.f : mn)));
        sum.m = mn;
#pragma unroll
        for (int o = 8; o <= 16; o *= 2) {
            sum.den += __shfl_xor_sync(0xffffffffu, sum.den, o);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                sum.acc[e].x += __shfl_xor_sync(0xffffffffu, sum.acc[e].x, o);
                sum.acc[e].y += __shfl_xor_sync(0xffffffffu, sum.acc[e].y, o);
                sum.acc[e].z += __shfl_xor_sync(0xffffffffu, sum.acc[e].z, o);
                sum.acc[e].w += __shfl_xor_sync(0xffffffffu, sum.acc[e].w, o);
            }
        }
    }
    if constexpr (G == kTreeMergeGroups) {  // the CTA's four warps
        constexpr int kWarps = kTreeMergeThreads / 32;
        __shared__ float4 s_acc[kWarps][E][8];
        __shared__ float2 s_mden[kWarps];
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) < 8) {
#pragma unroll
            for (int e = 0; e < E; ++e) s_acc[warp][e][q8] = sum.acc[e];
            if (q8 == 0) s_mden[warp] = make_float2(sum.m, sum.den);
        }
        __syncthreads();
        if (threadIdx.x >= 8) return;
        float mn = sum.m;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) mn = fmaxf(mn, s_mden[w].x);
        const float ref = mn == -INFINITY ? 0.f : mn;
        sum.scale(exp2f(sum.m - ref));
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            const float f = exp2f(s_mden[w].x - ref);
            const float den = sum.den + s_mden[w].y * f;
            float4 x[E];
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = s_acc[w][e][q8];
            sum.add(f, x);
            sum.den = den;
        }
    }
    if (group % G % 4 != 0) return;
    const float inv = sum.den == 0.f ? 0.f : 1.f / sum.den;
    uint2* out = reinterpret_cast<uint2*>(static_cast<T*>(p.out) + (int64_t)row * D) + q8;
#pragma unroll
    for (int e = 0; e < E; ++e)
        out[8 * e] = make_uint2(pack2(sum.acc[e].x * inv, sum.acc[e].y * inv, T()),
                                pack2(sum.acc[e].z * inv, sum.acc[e].w * inv, T()));
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Arguments that the workspace size and the launch share, and the plan of a
// call: the rows' split, the CTAs and the workspace.
constexpr int kTreeMaxContext = INT_MAX - 1024;  // positions of the last tile fit an int
struct TreeCallPlan {
    bool two_row_tiles;  // ROWS
    int row_blocks;
    int unit_rows;
    int ctas;
    int max_tiles;       // of a unit, in places
    bool cut;            // a unit may be cut: partials and a merge
    size_t units_bytes;
    size_t workspace_bytes;
};

static pkv_status plan_tree(int num_seqs, int tree_len, int num_q_heads, int num_kv_heads,
                            int head_dim, int block_size, int max_context_len,
                            TreeCallPlan* plan) {
    const pkv_status st = check_shapes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                       max_context_len, 0);
    if (st != PKV_OK) return st;
    if (tree_len <= 0) return PKV_ERR_INVALID_ARG;
    if (tree_len > PKV_MAX_TREE_LEN || (int64_t)num_seqs * num_kv_heads > 65535)
        return PKV_ERR_UNSUPPORTED;
    if (max_context_len > kTreeMaxContext) return PKV_ERR_UNSUPPORTED;
    const int tiles = tree_tiles(max_context_len);
    if ((int64_t)num_seqs * tree_cost(max_context_len) > INT_MAX) return PKV_ERR_UNSUPPORTED;
    const int sms = current_sm_count();
    if (sms <= 0) return PKV_ERR_CUDA;
    const int rows = tree_len * (num_q_heads / num_kv_heads);
    // ROWS or 128-row units (each reading the K/V again, mostly from L2).  32 x 4096
    // tokens on the Llama-70B layer, ROWS against 128-row units: 136 rows per KV
    // head 143 / 180 us, 256 rows 151 / 187, 512 rows 299 / 359; of three blocks of
    // 128 rows ROWS would compute four: 320 rows 280 / 268 us, 384 rows 285 / 274.
    const int blocks = (rows + kTreeRows - 1) / kTreeRows;
    plan->two_row_tiles = blocks > 1 && blocks != 3;
    plan->unit_rows = plan->two_row_tiles ? 2 * kTreeRows : kTreeRows;
    plan->row_blocks = (rows + plan->unit_rows - 1) / plan->unit_rows;
    const int64_t units = (int64_t)num_seqs * num_kv_heads * plan->row_blocks;
    if ((int64_t)num_kv_heads * plan->row_blocks * tree_cost(max_context_len) > INT_MAX)
        return PKV_ERR_UNSUPPORTED;
    plan->ctas = (int)std::max<int64_t>(1, std::min<int64_t>(sms, units * tiles));
    plan->max_tiles = tiles;
    plan->cut = tiles > 1;
    plan->units_bytes = ((size_t)units * sizeof(int2) + 255) & ~size_t(255);
    plan->workspace_bytes =
        256 + (plan->cut ? plan->units_bytes + (size_t)tree_partials(plan->ctas) *
                                                   plan->unit_rows * (head_dim + 1) * sizeof(float)
                         : 0);
    return PKV_OK;
}

template <typename T, int D, bool ROWS>
static cudaError_t launch_tree_t(const CUtensorMap& mk, const CUtensorMap& mv, const TreeParams& p,
                                 const TreeCallPlan& plan, cudaStream_t stream) {
    using Cfg = TreeTileCfg<D>;
    auto kern = tree_attention_kernel<T, D, ROWS>;
    // the attribute belongs to a device's copy of the kernel
    static std::atomic<bool> set[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !set[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Cfg::kSmemBytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) set[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(plan.ctas);
    cfg.blockDim = dim3(kTreeThreads);
    cfg.dynamicSmemBytes = Cfg::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, mk, mv, p);
    if (e != cudaSuccess || !plan.cut) return e;
    const int64_t rows = (int64_t)p.num_seqs * p.tree_len * p.num_q_heads;
    // Groups a row: while few rows leave the SMs room (about 20000 groups run at a
    // time) and a unit may have partials for them.  1, 4 and 16 groups, the whole call
    // in a graph (bf16, head dim 128, 16-token pages):
    //   9 nodes, 4/1 heads, 1 x 12579 tokens (36 rows of 99 partials)     40, 19.5, 13.1
    //   63 nodes, 4/1 heads, 1 x 17963 tokens (252 rows of 141)           61, 34, 27.8
    //   16 nodes, 8/1 heads, 14 x 4016 tokens (1792 rows of some 11)    24.8, 19.2, 19.7
    //   60 nodes, 8/4 heads, 27 x 2060 tokens (12960 rows of two or three)  34, 37, 51
    const int partials = std::min(plan.ctas, plan.max_tiles);
    const int groups = rows * 16 <= 32768 && partials > 8 ? kTreeMergeGroups
                       : rows * 4 <= 32768 && partials > 2 ? 4
                                                           : 1;
    const int64_t ctas = (rows * groups + kTreeMergeGroups - 1) / kTreeMergeGroups;
    if (ctas > INT_MAX) return cudaErrorInvalidValue;
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kTreeMergeThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg,
                              groups == 1   ? tree_merge_kernel<T, D, 1>
                              : groups == 4 ? tree_merge_kernel<T, D, 4>
                                            : tree_merge_kernel<T, D, kTreeMergeGroups>,
                              p, plan.unit_rows);
}

template <typename T>
static cudaError_t launch_tree(const CUtensorMap& mk, const CUtensorMap& mv, const TreeParams& p,
                               const TreeCallPlan& plan, int head_dim, cudaStream_t stream) {
    if (head_dim == 64)
        return plan.two_row_tiles ? launch_tree_t<T, 64, true>(mk, mv, p, plan, stream)
                                  : launch_tree_t<T, 64, false>(mk, mv, p, plan, stream);
    return plan.two_row_tiles ? launch_tree_t<T, 128, true>(mk, mv, p, plan, stream)
                              : launch_tree_t<T, 128, false>(mk, mv, p, plan, stream);
}

}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_tree_attention_workspace_size(int num_seqs, int tree_len, int num_q_heads,
                                                    int num_kv_heads, int head_dim,
                                                    int block_size, int max_context_len) {
    TreeCallPlan plan;
    if (plan_tree(num_seqs, tree_len, num_q_heads, num_kv_heads, head_dim, block_size,
                  max_context_len, &plan) != PKV_OK)
        return SIZE_MAX;
    return plan.workspace_bytes;
}

extern "C" pkv_status pkv_tree_attention(
    void* out, const void* q, const void* k_cache, const void* v_cache,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* context_lens,
    int max_context_len, const int32_t* tree_mask, int64_t mask_stride, int num_seqs, int tree_len,
    int num_blocks, int block_size, int num_q_heads, int num_kv_heads, int head_dim, float scale,
    void* workspace, size_t workspace_bytes, pkv_dtype dtype, int32_t* err_flag, void* stream) {
    const bool hnd = take_layout(dtype);
    if ((dtype != PKV_FP16 && dtype != PKV_BF16) || max_blocks_per_seq <= 0 || num_blocks <= 0 ||
        !std::isfinite(scale) || tree_len <= 0)
        return PKV_ERR_INVALID_ARG;
    const int64_t mask_words = (int64_t)tree_len * (((int64_t)tree_len + 31) / 32);
    if (mask_stride != 0 && mask_stride < mask_words) return PKV_ERR_INVALID_ARG;
    pkv_status st = check_shapes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                 max_context_len, 0);
    if (st != PKV_OK) return st;
    if (tree_len > PKV_MAX_TREE_LEN || (int64_t)num_seqs * num_kv_heads > 65535)
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PKV_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !tree_mask ||
        !workspace)
        return PKV_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
        !aligned16(workspace) ||
        ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(context_lens) |
          reinterpret_cast<uintptr_t>(tree_mask)) & 3u))
        return PKV_ERR_INVALID_ARG;
    if ((int64_t)max_blocks_per_seq * block_size > kTreeMaxContext ||
        max_context_len > kTreeMaxContext)
        return PKV_ERR_UNSUPPORTED;
    // the output is q itself (a unit's rows are read by its CTAs alone, and written when
    // they are through), or apart from everything that is read
    const int64_t seqs = num_seqs;
    const int64_t q_bytes = seqs * tree_len * num_q_heads * head_dim * 2;
    const int64_t mask_bytes = ((seqs - 1) * mask_stride + mask_words) * 4;
    const int64_t cache_bytes = (int64_t)num_blocks * block_size * num_kv_heads * head_dim * 2;
    const auto over = [&](const void* a, int64_t bytes) { return overlap(out, q_bytes, a, bytes); };
    if ((out != q && over(q, q_bytes)) || over(block_tables, seqs * max_blocks_per_seq * 4) ||
        over(context_lens, seqs * 4) || over(tree_mask, mask_bytes) ||
        over(k_cache, cache_bytes) || over(v_cache, cache_bytes))
        return PKV_ERR_INVALID_ARG;
    TreeCallPlan plan;
    st = plan_tree(num_seqs, tree_len, num_q_heads, num_kv_heads, head_dim, block_size,
                   max_context_len, &plan);
    if (st != PKV_OK) return st;
    if (workspace_bytes < plan.workspace_bytes) return PKV_ERR_WORKSPACE;
    if (over(workspace, (int64_t)plan.workspace_bytes)) return PKV_ERR_INVALID_ARG;

    CUtensorMap mk, mv;
    if (!make_cache_map(&mk, k_cache, dtype, num_blocks, block_size, num_kv_heads, head_dim, hnd) ||
        !make_cache_map(&mv, v_cache, dtype, num_blocks, block_size, num_kv_heads, head_dim, hnd))
        return PKV_ERR_CUDA;
    TreeParams p = {};
    p.out = out;
    p.q = q;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.tree_mask = tree_mask;
    p.mask_stride = mask_stride;
    p.err_flag = err_flag;
    if (plan.cut) {
        p.unit_ctas = static_cast<int2*>(workspace);
        p.partial_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan.units_bytes);
        p.partial_lse =
            p.partial_o + (size_t)tree_partials(plan.ctas) * plan.unit_rows * head_dim;
        p.ctas = plan.ctas;
    }
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.num_seqs = num_seqs;
    p.num_q_heads = num_q_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = num_q_heads / num_kv_heads;
    p.tree_len = tree_len;
    p.cap = std::min(max_blocks_per_seq * block_size, max_context_len);
    p.row_blocks = plan.row_blocks;
    p.hnd = hnd;
    p.scale_log2 = (scale == 0.f ? 1.f : std::fabs(scale)) * kLog2e;
    p.scale_sign = scale > 0.f ? 1.f : scale < 0.f ? -1.f : 0.f;
    cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = dtype == PKV_FP16
                              ? launch_tree<__half>(mk, mv, p, plan, head_dim, s)
                              : launch_tree<__nv_bfloat16>(mk, mv, p, plan, head_dim, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}
