// Attention of a ragged step's new tokens over a paged KV cache (tcgen05).
//
// The math: token i of sequence b, which brings t_b tokens to n_b, has position
// m = n_b - t_b + i and sees lo <= t < hi,
//     lo = max(0, m + 1 - window), hi = max(m + 1, min(prefix_b, n_b));
//     z_t = scale <q_i, K_t>, capped by softcap tanh(z / softcap), plus slope_h (t - m);
//     out_i = softmax(z) V over those t.
// The (token, query head) rows of a KV head form a dense matrix that meets every
// position once: the two products run on the tensor cores (fp32 accumulators in tensor
// memory), with the online softmax between them: running reference m, sum l and
// accumulator O per row, one division at the end.
//
// Tiles: 128 rows x 128 positions.  Two softmax warpgroups, a thread a row, each with
// an S and an O of its own in tensor memory (all 512 columns at head dim 128):
//   S_w = Q_w K^T   tcgen05.mma 128 x 128 x D, Q and K from shared memory
//   softmax         a thread reads its row of S, writes P over it
//   O_w += P_w V    P from tensor memory, V from shared memory
// One warp issues everything in the order PV_0(j) S_0(j+1) PV_1(j) S_1(j+1), so that a
// warpgroup is at its softmax while the other's two products run; the order keeps them
// apart (with an issuer for each, both fell into step, and a chunk of 4096 tokens behind
// 61440, 64/8 heads, took a fifth longer).  The tensor core runs the products in that order: S over a
// P comes after the product that reads it, and where S(j) is complete so is PV(j-1).  P
// goes over in two halves of 64 positions: the first is multiplied while the second is
// made.
// A unit (row block of a KV head, pkv_chunk_line.cuh) of more than 128 rows gives each
// warpgroup 128 of its rows, which meet the same tiles; a smaller one (single tokens,
// drafted tails) gives both the same rows and every other tile, and they meet at the
// end.  Four warps stream K and V by TMA through the block table into a ring of tiles.
// Two warps clean the V of tiles that some rows see only in part (below), once for all.
// One warp walks the segments and leaves what the others need of a unit in a ring in
// shared memory, a few units ahead: walked by every warp for itself, the reads of a new
// sequence and its tables stood before each unit's first softmax, 6 to 7 us a unit.
//
// A softmax weight meets V as one 16-bit term in the larger units, where the products
// are what takes the time (a second term costs half as much again), and as two in the
// smaller ones, which wait for memory: a single token's output is as precise as
// pkv_decode_attention's, a chunk's row has its weights' rounding beside its own.
//
// Work: the units' places lie on one line, cut into equal segments; a persistent CTA an
// SM takes one of them, or one in each of a few rounds where the line is long (so that
// the CTAs are near one another on the line, and what they read of K and V together
// stays in L2).  A unit inside a segment is written to the output at once; one that is
// cut leaves a partial (normalised O and its log-sum-exp) per segment, which
// chunk_merge_kernel joins.
//
// Measured (64/8 heads, bf16, d 128, a call in a graph): single tokens of 64 sequences over
// 2500 positions 117 us, 85 % of the copy rate; whole prompts of 4096 tokens 925 us, 1026
// TFLOP/s; 4096 tokens behind 61440 6.9 ms, 1231 TFLOP/s, 65 % of the rate of library
// products.  What bounds the large ones is a warpgroup's chain: of the 3900 cycles a tile of
// both takes, 500 go into the maximum, 1900 into the weights, 750 into the wait for P V and
// the next S; the tensor pipe is active 44 % of the time.  Twice the softmax warps (a row's
// halves in two threads) took as long or longer; so did every form with more instructions:
// beside eight other warps' loops it is the instruction cache that the softmax runs out of.
//
// Every wait is bounded, as in the decode kernels.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>

#include "pkv_chunk_line.cuh"
#include "pkv_common.cuh"
#include "pkv_device.cuh"

namespace pkv {

struct ChunkParams {
    void* out;
    const void* q;
    const void* v_cache;
    const int32_t* block_tables;
    const int32_t* query_starts;
    const int32_t* context_lens;
    const int32_t* prefix_lens;
    const float* slopes;
    int32_t* err_flag;
    ChunkRecord* records;  // [rounds * ctas]
    int32_t* has;          // [chunk_partials]: whether a stretch of tiles left a partial
    float* partial_o;      // [chunk_partials][D / 4][2 kChunkRows][4]
    float* partial_lse;    // [chunk_partials][2 kChunkRows], base 2
    ChunkShape shape;
    int rounds;            // at most
    int max_blocks_per_seq;
    int num_seqs;
    int num_tokens;
    int num_blocks;
    int block_size;
    int num_q_heads;
    int cap;
    bool hnd;
    float scale_log2;      // scale * log2(e)
    float softcap;
    float tanh_log2;       // 2 log2(e) scale / softcap
};

constexpr int kChunkSoftmaxWarps = 8;                 // two warpgroups
constexpr int kChunkTmaWarp = kChunkSoftmaxWarps;     // four producers
constexpr int kChunkTmaWarps = 4;
constexpr int kChunkMmaWarp = kChunkTmaWarp + kChunkTmaWarps;
constexpr int kChunkWalkWarp = kChunkMmaWarp + 1;
constexpr int kChunkCleanWarp = kChunkWalkWarp + 1;
constexpr int kChunkCleanWarps = 2;
constexpr int kChunkThreads = (kChunkCleanWarp + kChunkCleanWarps) * 32;
static_assert(kChunkThreads == 512, "four warpgroups");
constexpr int kChunkReaders =  // of a unit's notes
    kChunkSoftmaxWarps + kChunkTmaWarps + 1 + kChunkCleanWarps;
// Registers: the other warpgroups hand over what they do not need, so that a softmax
// thread's half row of S stays in registers.  Nothing is spilled at this split (at 184 and
// 72 the walker's and the issuer's values were, and a chunk behind 61440 tokens took 7.0 ms
// instead of 6.5: beside 226 KB of shared memory little is left to cache a stack in).
constexpr int kChunkLaunchRegs = 128, kChunkSoftmaxRegs = 168, kChunkOtherRegs = 88;
static_assert(2 * kChunkSoftmaxRegs + 2 * kChunkOtherRegs <= 4 * kChunkLaunchRegs, "register shares");
// Scores may exceed a row's reference by this much (base 2) before it moves.
constexpr float kChunkLazyLog2 = 8.f;
constexpr int kChunkBoxes = kChunkTile / kStageTokens;  // TMA boxes along a tile
constexpr int kChunkMaxRounds = 4;
// Notes of units, a ring of them; with each the mark of a V that is not finite in it.
constexpr int kChunkNotes = 4;
// A segment has at least this many places, no more than the smallest unit, so that each
// unit of a small batch has a CTA (two sequences of 40 tokens: 8.6 us, 10.7 at 512), and
// more rounds are taken only where theirs have this many (whole prompts of 4096 tokens:
// 924 us, 939 at 24576 and 966 at 12288, where more units are cut).
constexpr int kChunkLeastSegment = kChunkUnitCost;
constexpr int kChunkRoundSegment = 49152;

// What the walking warp notes of a unit's stretch.
struct ChunkNote {
    int b, g;
    int q_row;           // row of q of the row block's first token
    int tokens;          // of the row block
    int m;               // the first one's position
    int prefix;
    int lo, hi;          // positions that any row sees
    int lo_all, hi_all;  // that all rows see
    int tile, tiles;     // tiles of the stretch; -1 tiles: the end
    int partial;         // the stretch's partial, or -1: it is the whole unit
    int flags;
    int bad_from, bad_to;  // tiles of the stretch whose V was not finite (by the cleaners)
    int blocks[2 * kChunkBoxes];  // of the first two tiles' boxes, as the table has them
};
constexpr int kNotePagesThere = 1;  // every page of the stretch is within the pool
constexpr int kNoteAgain = 2;       // other row blocks read the same tiles
// The stretch's tiles that every row sees whole, where all pages are there: from .. to - 1.
__device__ __forceinline__ int chunk_plain_from(const ChunkNote& t) {
    return t.flags & kNotePagesThere ? (t.lo_all + kChunkTile - 1) / kChunkTile - t.tile : 0;
}
__device__ __forceinline__ int chunk_plain_to(const ChunkNote& t) {
    return t.flags & kNotePagesThere ? t.hi_all / kChunkTile - t.tile : 0;
}
static_assert(sizeof(ChunkNote) == 128, "notes in shared memory");

// A segment's start, as one thread found it for all.
struct ChunkStart {
    int64_t at;
    int b, g, rb, pos;
};

template <int D>
struct ChunkTileCfg {
    static constexpr int kRegions = D / 64;                      // 128-byte column blocks
    static constexpr int kRegionBytes = kChunkTile * 128;        // of a tile, and of Q
    static constexpr int kTileBytes = kRegions * kRegionBytes;   // K or V of a tile; Q
    static constexpr int kSlots = D == 128 ? 5 : 10;
    static constexpr int kXchBytes = 2 * kChunkRows * 8;         // (m, l) of each half and row
    // full[slots], empty[slots], clean[slots], s_full[2], p_half[2], p_ready[2], o_done[2],
    // q_ready[2], met, o_free, drain, noted[notes], read[notes], cleaned[notes]
    static constexpr int kBarriers = 3 * kSlots + 13 + 3 * kChunkNotes;
    static constexpr int kSmemBytes = (2 + kSlots) * kTileBytes + kXchBytes + kBarriers * 8 + 24 +
                                      kChunkMaxRounds * (int)sizeof(ChunkStart) +
                                      kChunkNotes * (int)sizeof(ChunkNote);
    static constexpr uint32_t kColO = 2 * kChunkTile;  // S of each warpgroup, then O
    static_assert(kColO + 2 * D <= 512, "tensor memory layout");
    static_assert(kSmemBytes <= 232448, "shared memory of a CTA");
};

// A bounded wait of a whole warp, as warp_wait_phase, in a few instructions: a dozen warps
// wait at any time here, and what they execute meanwhile takes instruction cache from the
// softmax.  Every wait has its limit, so no flag between the warps ends them.
constexpr unsigned kChunkWaitCycles = 3800000000u;  // about 2 s
__device__ __forceinline__ bool chunk_wait(uint32_t bar, uint32_t parity) {
    const unsigned t0 = clock();
    bool ok;
    while (!(ok = ptx::mbar_try_wait(bar, parity)))
        if ((unsigned)clock() - t0 > kChunkWaitCycles) break;
    return __all_sync(0xffffffffu, ok);
}

// What lies at place i of the ring, counted from the first of a stretch of nt tiles: the
// order in which the issuer takes them.  Both warpgroups on every tile: K0 V0 K1 V1 ..;
// every other tile (split): K0 K1 V0 K2 V1 K3 ..
__device__ __forceinline__ int chunk_place_tile(bool split, int i, int nt, bool& is_v) {
    is_v = split ? (i > 1 && i % 2 == 0) || i == 2 * nt - 1 : i % 2 == 1;
    if (!split) return i / 2;
    return i == 2 * nt - 1 ? nt - 1 : i < 2 ? i : is_v ? i / 2 - 1 : (i + 1) / 2;
}

__device__ __forceinline__ ChunkSeq chunk_load(const ChunkParams& p, int b) {
    const int from = __ldg(p.query_starts + b), to = __ldg(p.query_starts + b + 1);
    const int n = __ldg(p.context_lens + b);
    const int prefix = p.prefix_lens != nullptr ? __ldg(p.prefix_lens + b) : 0;
    ChunkSeq s;
    s.first = clamped_len(from, p.num_tokens);
    s.tokens = max(0, clamped_len(to, p.num_tokens) - s.first);
    s.n = clamped_len(n, p.cap);
    s.prefix = clamped_len(prefix, s.n);
    return s;
}

__device__ __forceinline__ int64_t warp_scan64(int64_t x) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, x, o);
        if ((threadIdx.x & 31) >= o) x += v;
    }
    return x;
}

// Adds to a finished row what it sees of the V that the cleaners took out: infinities and
// NaN, but for positions lo_all .. hi_all - 1, whose V was left alone.  (Whatever finite
// value stands there, the sum is the same.)
struct ChunkSeen {
    const int32_t* table;
    int from, to;  // positions of the stretch that the row sees
    int lo_all, hi_all;
    int g;
};
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T, int D, typename At>
__device__ __forceinline__ void add_not_finite(const ChunkParams& p, const ChunkSeen& s, int col0,
                                               int cols, At at) {
    const int bs = p.block_size;
#pragma unroll 1
    for (int x = s.from; x < s.to; ++x) {
        if (x >= s.lo_all && x < s.hi_all) {
            x = min(s.hi_all, s.to) - 1;
            continue;
        }
        const int blk = __ldg(s.table + x / bs);
        if (blk < 0 || blk >= p.num_blocks) continue;
        const int off = x % bs;
        const uint16_t* v =
            static_cast<const uint16_t*>(p.v_cache) +
            (p.hnd ? ((int64_t)blk * p.shape.heads + s.g) * bs + off
                   : ((int64_t)blk * bs + off) * p.shape.heads + s.g) * D;
#pragma unroll 1
        for (int c = col0; c < col0 + cols; ++c) {
            const uint16_t e = __ldg(v + c);
            if (not_finite(e, T())) at(c, unpack2(e, T()).x);
        }
    }
}

// Four lanes with four 16-byte pieces each: lane k's piece i becomes lane i's piece k.
__device__ __forceinline__ uint4 shfl_xor4(uint4 x, int o) {
    return make_uint4(__shfl_xor_sync(0xffffffffu, x.x, o), __shfl_xor_sync(0xffffffffu, x.y, o),
                      __shfl_xor_sync(0xffffffffu, x.z, o), __shfl_xor_sync(0xffffffffu, x.w, o));
}
__device__ __forceinline__ void trade_pieces(uint4 (&x)[4], int lane) {
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & o) continue;
            const bool up = lane & o;
            const uint4 got = shfl_xor4(up ? x[i] : x[i + o], o);
            if (up)
                x[i] = got;
            else
                x[i + o] = got;
        }
}

template <typename T, int D, bool MOD>
__global__ void __launch_bounds__(kChunkThreads, 1)
chunk_attention_kernel(const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const ChunkParams p) {
    using Cfg = ChunkTileCfg<D>;
    constexpr int R = Cfg::kRegions;
    constexpr int NS = Cfg::kSlots;
    constexpr int TR = kChunkRows;
    constexpr int TT = kChunkTile;

    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* sq = smem;  // two Q tiles [region][128 rows][128 B], swizzled
    uint8_t* ring = sq + 2 * Cfg::kTileBytes;
    float2* xch = reinterpret_cast<float2*>(ring + NS * Cfg::kTileBytes);
    uint64_t* full_bar = reinterpret_cast<uint64_t*>(ring + NS * Cfg::kTileBytes + Cfg::kXchBytes);
    uint64_t* empty_bar = full_bar + NS;
    uint64_t* clean_bar = empty_bar + NS;  // of a V that is cleaned
    uint64_t* s_full = clean_bar + NS;  // [warpgroup]
    uint64_t* p_half = s_full + 2;      // [warpgroup]: the first 64 positions' weights
    uint64_t* p_ready = p_half + 2;     // [warpgroup]: all of them
    uint64_t* o_done = p_ready + 2;   // [warpgroup]: a unit's last product is complete
    uint64_t* q_ready = o_done + 2;     // [warpgroup]
    uint64_t* met = q_ready + 2;        // both are through a split unit
    uint64_t* o_free = met + 1;         // both have read O_0, O_1 and the exchange of one
    uint64_t* drain = o_free + 1;
    uint64_t* noted = drain + 1;        // [notes]
    uint64_t* read = noted + kChunkNotes;  // [notes]: by all readers
    uint64_t* cleaned = read + kChunkNotes;  // [notes]: every tile of the unit
    int64_t* s_line = reinterpret_cast<int64_t*>(full_bar + Cfg::kBarriers);
    int* words = reinterpret_cast<int*>(s_line + 1);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(words);
    int* s_segments = words + 1;
    ChunkStart* s_start = reinterpret_cast<ChunkStart*>(words + 4);
    ChunkNote* notes = reinterpret_cast<ChunkNote*>(s_start + kChunkMaxRounds);
    int64_t* s_scan = reinterpret_cast<int64_t*>(xch);  // [16], before the first exchange

    const int tid = threadIdx.x;
    const int warp = tid >> 5;
    const int lane = tid & 31;
    const int bs = p.block_size;
    const int bs_shift = __ffs(bs) - 1;

    ptx::launch_dependents();
    if (tid < Cfg::kBarriers) {  // a thread a barrier, in their order
        const int i = tid;
        const int count =
            i < NS                ? kChunkTmaWarps
            : i < 2 * NS          ? 1 + kChunkCleanWarps
            : i < 3 * NS          ? kChunkCleanWarps
            : i < 3 * NS + 2      ? 1            // s_full
            : i < 3 * NS + 6      ? TR / 32      // p_half, p_ready
            : i < 3 * NS + 8      ? 1            // o_done
            : i < 3 * NS + 10     ? TR           // q_ready
            : i < 3 * NS + 12     ? 2 * TR       // met, o_free
            : i < 3 * NS + 13     ? 1            // drain
            : i < 3 * NS + 13 + kChunkNotes     ? 1  // noted
            : i < 3 * NS + 13 + 2 * kChunkNotes ? kChunkReaders
                                                : kChunkCleanWarps;
        ptx::mbar_init(ptx::smem_addr(&full_bar[i]), count);
        ptx::fence_barrier_init();
    }
    if (tid == 0) {
        ptx::prefetch_tensormap(&tm_k);
        ptx::prefetch_tensormap(&tm_v);
    }
    if (warp == kChunkMmaWarp) {
        ptx::tmem_alloc(ptx::smem_addr(tmem_slot), 512);
        ptx::tmem_relinquish_alloc_permit();
    }
#ifdef PKV_DEBUG
    poison_smem(ring, NS * Cfg::kTileBytes, tid, kChunkThreads);
#endif
    ptx::grid_dependency_wait();

    auto load = [&](int b) { return chunk_load(p, b); };
    auto chunk_ctas = [&](int64_t line) {
        return (int)min((int64_t)gridDim.x, (line + kChunkLeastSegment - 1) / kChunkLeastSegment);
    };

    // The line, and where on it this CTA's segments start: a thread sums the places of a
    // run of sequences, a scan puts the runs in order, and the thread whose run holds a
    // segment's first place stands there for all.  Up to 32 sequences the walking warp
    // does it by itself, a lane a sequence, and the others go on meanwhile.
    const bool few = p.num_seqs <= 32;
    if (few) {
        ptx::tc_fence_before_sync();
        __syncthreads();
        ptx::tc_fence_after_sync();
    }
    if (!few || warp == kChunkWalkWarp) {
        const int me = few ? lane : tid;
        const int runs = few ? 32 : kChunkThreads;
        const int per = (p.num_seqs + runs - 1) / runs;
        const int b_lo = min(p.num_seqs, me * per);
        const int b_hi = min(p.num_seqs, b_lo + per);
        int64_t mine = 0;
        for (int b = b_lo; b < b_hi; ++b) {
            mine += chunk_places(load(b), p.shape);
            if (blockIdx.x == 0) {
                const int from = __ldg(p.query_starts + b), to = __ldg(p.query_starts + b + 1);
                if (from < 0 || to < from || to > p.num_tokens)
                    flag_error(p.err_flag, PKV_EFLAG_QUERY);
            }
        }
        const int64_t incl = warp_scan64(mine);
        int64_t before = incl - mine;
        int64_t line = __shfl_sync(0xffffffffu, incl, 31);
        if (!few) {
            if (lane == 31) s_scan[warp] = line;
            __syncthreads();
            line = 0;
            for (int w = 0; w < kChunkThreads / 32; ++w) {
                if (w < warp) before += s_scan[w];
                line += s_scan[w];
            }
        }
        {
            const int ctas = chunk_ctas(line);
            const int64_t long_ones =
                ctas > 0 ? line / ((int64_t)ctas * kChunkRoundSegment) : 0;
            const int rounds = (int)max((int64_t)1, min((int64_t)p.rounds, long_ones));
            const int segments = rounds * ctas;
            if (me == 0) {
                *s_line = line;
                *s_segments = segments;
            }
            for (int r = 0; r < rounds && (int)blockIdx.x < ctas; ++r) {
                const int seg = r * ctas + blockIdx.x;
                const int64_t at = chunk_segment_start(line, segments, seg);
                if (at < before || at >= before + mine) continue;
                int64_t first = before;
                int b = b_lo;
                ChunkSeq s;
                while (true) {
                    s = load(b);
                    const int64_t places = chunk_places(s, p.shape);
                    if (at < first + places) break;
                    first += places;
                    ++b;
                }
                ChunkWalk w;
                w.enter(s, p.shape, b, at - first);
                s_start[r] = ChunkStart{at, w.b, w.g, w.rb, w.pos};
            }
        }
        __syncwarp();
    }
    if (!few) {
        ptx::tc_fence_before_sync();
        __syncthreads();
        ptx::tc_fence_after_sync();
    }
    const uint32_t tmem = *tmem_slot;
    const uint32_t ring_addr = ptx::smem_addr(ring);
    const uint32_t q_addr = ptx::smem_addr(sq);
    bool gave_up = false;
    auto wait_for = [&](uint32_t bar, int parity) {
        const bool done = chunk_wait(bar, parity);
        gave_up |= !done;
        return done;
    };
    // A reader's wait for note i of the CTA's, and its leave of it.
    auto note_there = [&](int i) {
        return wait_for(ptx::smem_addr(&noted[i % kChunkNotes]), (i / kChunkNotes) & 1);
    };
    auto note_read = [&](int i) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&read[i % kChunkNotes]));
    };
    const int group = p.shape.group;

    if (warp >= kChunkSoftmaxWarps) {
        ptx::reg_dec<kChunkOtherRegs>();
        if (warp < kChunkMmaWarp) {
            // ------------------------------------------------------------ producers
            // A warp loads a quarter of every tile; a lane issues one box (16 positions x
            // 64 dims).
            constexpr int kMine = kChunkBoxes * R / kChunkTmaWarps;
            const int box = (warp - kChunkTmaWarp) * kMine + lane;
            const int bx = box / R, rr = box % R;
            const bool loads = lane < kMine;
            const uint64_t keep = ptx::l2_policy_evict_last();
            const uint64_t once = ptx::l2_policy_evict_first();
            int place = 0;       // of the ring, since the start
            uint32_t filled = 0; // slots with a copy of this warp's that may be in flight,
            uint32_t parity = 0; // and its phase's parity
            bool ok = true;
            for (int u = 0; ok && note_there(u); ++u) {
                const ChunkNote& note = notes[u % kChunkNotes];
                const int nt = note.tiles, g = note.g, lo = note.lo, hi = note.hi;
                const int base = note.tile * TT + bx * kStageTokens;
                const bool split = note.tokens * group <= TR;
                const int32_t* table = p.block_tables + (int64_t)note.b * p.max_blocks_per_seq;
                const uint64_t policy = note.flags & kNoteAgain ? keep : once;
                const int first0 = loads ? note.blocks[bx] : -1;
                const int first1 = loads ? note.blocks[kChunkBoxes + bx] : -1;
                note_read(u);
                if (nt < 0) break;
                // the block of this lane's box of tile j, as the table has it (-1: none)
                auto box_block = [&](int j) {
                    const int at = base + j * TT;
                    return loads && j < nt && at + kStageTokens > lo && at < hi
                               ? __ldg(table + (at >> bs_shift))
                               : -1;
                };
                auto fill = [&](bool is_v, int j, int blk) {
                    const int at = base + j * TT;
                    if (blk < 0 || blk >= p.num_blocks) {
                        if (!is_v && loads && at + kStageTokens > lo && at < hi)
                            flag_error(p.err_flag, PKV_EFLAG_BLOCK_ID);
                        blk = -1;
                    }
                    const int slot = place % NS, phase = place / NS;
                    ++place;
                    if (phase > 0 && !wait_for(ptx::smem_addr(&empty_bar[slot]),
                                                      (phase - 1) & 1))
                        return false;
                    const uint32_t fb = ptx::smem_addr(&full_bar[slot]);
                    const uint32_t dst = ring_addr + slot * Cfg::kTileBytes +
                                         rr * Cfg::kRegionBytes + bx * kStageTokens * 128;
#ifdef PKV_DEBUG
                    if (phase > 0) {
                        ptx::tc_fence_after_sync();
                        for (int i = 0; i < kMine; ++i) {
                            const uint32_t d = __shfl_sync(0xffffffffu, dst, i);
                            poison_smem(ring + (d - ring_addr), kStageTokens * 128, lane, 32);
                        }
                        __syncwarp();
                    }
#endif
                    const uint32_t boxes = __ballot_sync(0xffffffffu, blk >= 0);
                    if (lane == 0) {
                        if (boxes == 0)
                            ptx::mbar_arrive(fb);  // every position of the quarter is masked
                        else
                            ptx::mbar_arrive_expect_tx(fb, __popc(boxes) * kStageTokens * 128);
                    }
                    __syncwarp();
                    if (blk >= 0)
                        load_kv_box(dst, is_v ? &tm_v : &tm_k, fb, rr * 64, g, at & (bs - 1),
                                    blk, p.hnd, policy);
                    filled |= 1u << slot;
                    parity = (parity & ~(1u << slot)) | ((uint32_t)(phase & 1) << slot);
                    return true;
                };
                // table entries are read two tiles ahead
                int b0 = first0, b1 = first1, b2 = box_block(2);
                if (split) ok = fill(false, 0, b0) && (nt < 2 || fill(false, 1, b1));
                for (int j = 0; j < nt && ok; ++j) {
                    const int far = box_block(j + 3);
                    if (split)
                        ok = fill(true, j, b0) && (j + 2 >= nt || fill(false, j + 2, b2));
                    else
                        ok = fill(false, j, b0) && fill(true, j, b0);
                    b0 = b1;
                    b1 = b2;
                    b2 = far;
                }
            }
            if (lane == 0) {
                // this warp's copies have arrived (they are still in flight where a reader
                // gave up) before the CTA leaves
                const uint64_t t0 = ptx::globaltimer();
                for (int i = 0; i < NS; ++i) {
                    if (!((filled >> i) & 1u)) continue;
                    while (!ptx::mbar_try_wait(ptx::smem_addr(&full_bar[i]), (parity >> i) & 1u) &&
                           ptx::globaltimer() - t0 < kWaitLimitNs) {
                    }
                }
            }
        } else if (warp == kChunkMmaWarp) {
            // ------------------------------------------------------------ MMA issuer
            // The whole warp walks the steps, so that addresses and descriptors are
            // uniform values; one elected lane issues.
            constexpr uint32_t fmt = F16Format<T>::value;
            constexpr uint32_t idesc_s = mma_idesc(fmt, TR, TT, false);
            constexpr uint32_t idesc_o = mma_idesc(fmt, TR, D, true);
            // descriptors of the first slots: a byte offset adds its sixteenth
            const uint64_t qdesc = ptx::smem_desc_sw128(q_addr, 16, 1024);
            const uint64_t kdesc = ptx::smem_desc_sw128(ring_addr, 16, 1024);
            const uint64_t vdesc = ptx::smem_desc_sw128(ring_addr, Cfg::kRegionBytes, 1024);
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            int slot = 0, phase = 0;  // of the ring's next place
            int step[2] = {0, 0};     // tiles of each warpgroup so far
            int unit[2] = {0, 0};     // units with tiles for it
            uint32_t cleans = 0;      // parity of the slots' cleanings
            bool ok = true;
            auto wait = [&](uint64_t* bar, int parity) {
                return wait_for(ptx::smem_addr(bar), parity & 1);
            };
            // the ring's next place, once it is full; -1: a wait gave up
            auto take = [&] {
                if (!wait(&full_bar[slot], phase)) return -1;
                const int at = slot;
                if (++slot == NS) {
                    slot = 0;
                    phase ^= 1;
                }
                return at;
            };
            // S of warpgroup w from the K in slot `at`; `last`: its last reader
            auto issue_s = [&](int w, int at, bool last) {
                ptx::tc_fence_after_sync();
                const uint64_t kd = kdesc + (uint32_t)(at * (Cfg::kTileBytes / 16));
                const uint64_t qd = qdesc + (uint32_t)(w * (Cfg::kTileBytes / 16));
                if (ptx::elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        ptx::tc_mma_f16(
                            tm + w * TT, qd + (ks / 4) * (Cfg::kRegionBytes / 16) + (ks % 4) * 2,
                            kd + (ks / 4) * (Cfg::kRegionBytes / 16) + (ks % 4) * 2, idesc_s,
                            ks > 0 ? 1u : 0u);
                    ptx::tc_commit(ptx::smem_addr(&s_full[w]));
                    if (last) ptx::tc_commit(ptx::smem_addr(&empty_bar[at]));
                }
                __syncwarp();
            };
            // the V there, once it is clean where it has to be
            auto take_v = [&](bool cleaned_first) {
                const int at = take();
                if (at < 0 || !cleaned_first) return at;
                const int parity = (cleans >> at) & 1;
                cleans ^= 1u << at;
                return wait(&clean_bar[at], parity) ? at : -1;
            };
            // O += P V of warpgroup w from the V in slot `at`
            auto issue_pv = [&](int w, int at, bool split, bool first, bool ends, bool last) {
                const uint64_t vd = vdesc + (uint32_t)(at * (Cfg::kTileBytes / 16));
                const uint32_t pt = tm + w * TT;
                const uint32_t acc = tm + Cfg::kColO + w * D;
                auto half = [&](int h) {
#pragma unroll
                    for (int i = 0; i < TT / 32; ++i) {
                        const int kt = h * (TT / 32) + i;
                        const uint64_t v = vd + (uint32_t)(kt * 16 * 128 / 16);
                        // of each 32 positions of P, 16 columns of pairs and 16 of their
                        // second terms, which a split unit's weights have
                        const uint32_t a = pt + (kt / 2) * 32 + (kt % 2) * 8;
                        ptx::tc_mma_f16_ts(acc, a, v, idesc_o, (!first || kt > 0) ? 1u : 0u);
                        if (split) ptx::tc_mma_f16_ts(acc, a + 16, v, idesc_o, 1u);
                    }
                };
                if (!wait(&p_half[w], step[w])) return false;
                ptx::tc_fence_after_sync();
                if (ptx::elect_one()) half(0);
                __syncwarp();
                if (!wait(&p_ready[w], step[w])) return false;
                ++step[w];
                ptx::tc_fence_after_sync();
                if (ptx::elect_one()) {
                    half(1);
                    if (ends) ptx::tc_commit(ptx::smem_addr(&o_done[w]));
                    if (last) ptx::tc_commit(ptx::smem_addr(&empty_bar[at]));
                }
                __syncwarp();
                return true;
            };
            for (int u = 0; ok && note_there(u); ++u) {
                const ChunkNote& note = notes[u % kChunkNotes];
                const int nt = __shfl_sync(0xffffffffu, note.tiles, 0);
                const bool split =
                    __shfl_sync(0xffffffffu, note.tokens * group <= TR ? 1 : 0, 0);
                // tiles of the stretch that every row sees, of pages that are there
                const int plain0 = __shfl_sync(0xffffffffu, chunk_plain_from(note), 0);
                const int plain1 = __shfl_sync(0xffffffffu, chunk_plain_to(note), 0);
                auto dirty = [&](int j) { return j < plain0 || j >= plain1; };
                note_read(u);
                if (nt < 0) break;
                ok = wait(&q_ready[0], unit[0]++);
                int at = ok ? take() : -1;
                if (at < 0) break;
                issue_s(0, at, split);
                if (split) {
                    // K0 K1 V0 K2 V1 K3 ..
                    if (nt > 1) {
                        ok = wait(&q_ready[1], unit[1]++) && (at = take()) >= 0;
                        if (!ok) break;
                        issue_s(1, at, true);
                    }
                    for (int j = 0; j < nt && ok; ++j) {
                        const int w = j & 1;
                        at = take_v(dirty(j));
                        ok = at >= 0 && issue_pv(w, at, true, j < 2, j + 2 >= nt, true);
                        if (ok && j + 2 < nt) {
                            at = take();
                            ok = at >= 0;
                            if (ok) issue_s(w, at, true);
                        }
                    }
                } else {
                    // K0 V0 K1 V1 ..
                    ok = wait(&q_ready[1], unit[1]++);
                    if (!ok) break;
                    issue_s(1, at, true);
                    for (int j = 0; j < nt && ok; ++j) {
                        const bool more = j + 1 < nt;
                        const int v = take_v(dirty(j));
                        ok = v >= 0 && issue_pv(0, v, false, j == 0, !more, false);
                        int k = -1;
                        if (ok && more) {
                            k = take();
                            ok = k >= 0;
                            if (ok) issue_s(0, k, false);
                        }
                        ok = ok && issue_pv(1, v, false, j == 0, !more, true);
                        if (ok && more) issue_s(1, k, true);
                    }
                }
            }
            // every product has completed before the tensor memory is released
            if (ptx::elect_one()) ptx::tc_commit(ptx::smem_addr(drain));
            __syncwarp();
            const uint64_t t0 = ptx::globaltimer();
            while (!ptx::mbar_try_wait(ptx::smem_addr(drain), 0) &&
                   ptx::globaltimer() - t0 < kWaitLimitNs) {
            }
        } else if (warp == kChunkWalkWarp) {
            // ------------------------------------------------------------ the walk
            const int64_t line = *s_line;
            const int segments = *s_segments;
            const int ctas = chunk_ctas(line);
            const int rounds = (int)blockIdx.x < ctas ? segments / ctas : 0;
            if (p.records != nullptr)  // segments that the line has not
                for (int i = segments + blockIdx.x * 32 + lane; i < p.rounds * (int)gridDim.x;
                     i += gridDim.x * 32)
                    p.records[i].first = -1;
            ChunkWalk walk;
            ChunkStretch t;
            int u = 0;
            bool ok = true;
            auto place = [&](int i) {  // where note i is written, once it was read
                return i < kChunkNotes ||
                       wait_for(ptx::smem_addr(&read[i % kChunkNotes]),
                                       (i / kChunkNotes - 1) & 1);
            };
            for (int round = 0; round < rounds && ok; ++round) {
                const ChunkStart start = s_start[round];
                const int segment = round * ctas + blockIdx.x;
                walk.at = start.at;
                walk.end = chunk_segment_start(line, segments, segment + 1);
                walk.b = start.b;
                walk.g = start.g;
                walk.rb = start.rb;
                walk.pos = start.pos;
                walk.seq = load(start.b);
                while (walk.next_any(p.shape, load, t)) {
                    const bool cut = t.tiles < t.unit_tiles;
                    if (p.records != nullptr && lane == 0) {
                        // what the join reads: whether this stretch leaves a partial, and,
                        // once a segment, the unit whose partials it joins: one that was cut
                        // by the segment's start and ends here
                        p.has[chunk_partial(segment, t.begins)] = cut && t.tiles > 0;
                        if (t.at == start.at) {
                            const bool joins =
                                !t.begins && cut && t.skipped + t.tiles == t.unit_tiles;
                            p.records[segment] = ChunkRecord{
                                joins ? chunk_segment_of(line, segments, t.unit_at) : -1, t.b,
                                t.g, t.rb};
                        }
                    }
                    if (t.tiles == 0) continue;
                    if (t.skipped == 0 && t.g == 0 && t.rb == 0 && lane == 0) {
                        const int n_raw = __ldg(p.context_lens + t.b);
                        if (n_raw != t.seq.n || n_raw < t.seq.tokens)
                            flag_error(p.err_flag, PKV_EFLAG_CONTEXT_LEN);
                    }
                    const int32_t* table = p.block_tables + (int64_t)t.b * p.max_blocks_per_seq;
                    // lanes 0-15: boxes of the first two tiles
                    const int at = t.tile * TT + lane * kStageTokens;
                    const int end = min(t.hi, (t.tile + t.tiles) * TT);
                    const int blk = lane < 2 * kChunkBoxes && at + kStageTokens > t.lo && at < end
                                        ? __ldg(table + (at >> bs_shift))
                                        : -1;
                    // whether all pages are there: where one is not, the others look at each
                    // tile's
                    const int page0 = max(t.lo, t.tile * TT) >> bs_shift;
                    const int pages = ((end - 1) >> bs_shift) - page0 + 1;
                    bool there = end > t.lo;
#pragma unroll 1
                    for (int i0 = lane; there && i0 < pages; i0 += 8 * 32) {
                        int x[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            x[i] = i0 + i * 32 < pages ? __ldg(table + page0 + i0 + i * 32) : 0;
#pragma unroll
                        for (int i = 0; i < 8; ++i) there &= x[i] >= 0 && x[i] < p.num_blocks;
                    }
                    there = __all_sync(0xffffffffu, there);
                    if (!place(u)) {
                        ok = false;
                        break;
                    }
                    ChunkNote& note = notes[u % kChunkNotes];
                    if (lane < 2 * kChunkBoxes) note.blocks[lane] = blk;
                    if (lane == 0) {
                        note.b = t.b;
                        note.g = t.g;
                        note.q_row = t.seq.first + t.token0;
                        note.tokens = t.tokens;
                        note.m = t.seq.n - t.seq.tokens + t.token0;
                        note.prefix = t.seq.prefix;
                        note.lo = t.lo;
                        note.hi = t.hi;
                        note.lo_all = t.lo_all;
                        note.hi_all = t.hi_all;
                        note.tile = t.tile;
                        note.tiles = t.tiles;
                        note.partial = cut ? chunk_partial(segment, t.begins) : -1;
                        note.flags = (there ? kNotePagesThere : 0) |
                                     (t.seq.tokens > p.shape.block_tokens ? kNoteAgain : 0);
                        note.bad_from = INT_MAX;
                        note.bad_to = 0;
                    }
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&noted[u % kChunkNotes]));
                    ++u;
                }
            }
            if (ok && place(u) && lane == 0) {
                notes[u % kChunkNotes].tiles = -1;
                ptx::mbar_arrive(ptx::smem_addr(&noted[u % kChunkNotes]));
            }
        } else {
            // ------------------------------------------------------------ cleaners
            // V rows that are not there hold stale bytes, and one that only some rows see may
            // hold infinities or NaN: zeroed in shared memory, so that 0 * V is 0; the rows
            // that do see such a value get it back at the end.  They pass every place of
            // the ring in its order and release it like the issuer (a reader that kept to
            // the tiles it has work in could not tell a slot's fills apart by their parity).
            const int half = warp - kChunkCleanWarp;
            constexpr int kCells = R * 8;                    // 16-byte cells of a row
            constexpr int kRowsEach = TT / kChunkCleanWarps;
            int slot = 0, phase = 0;
            bool ok = true;
            auto leave = [&] {
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&empty_bar[slot]));
                if (++slot == NS) {
                    slot = 0;
                    phase ^= 1;
                }
            };
            for (int u = 0; ok && note_there(u); ++u) {
                ChunkNote& t = notes[u % kChunkNotes];
                const int nt = t.tiles, tile = t.tile;
                if (nt < 0) break;
                const bool split = t.tokens * group <= TR;
                const bool there = t.flags & kNotePagesThere;
                const int lo = t.lo, hi = t.hi, lo_all = t.lo_all, hi_all = t.hi_all;
                const int plain0 = chunk_plain_from(t), plain1 = chunk_plain_to(t);
                const int32_t* table = p.block_tables + (int64_t)t.b * p.max_blocks_per_seq;
                auto box_block = [&](int j) {  // lanes 0-7
                    const int at = (tile + j) * TT + lane * kStageTokens;
                    return !there && lane < kChunkBoxes && j < nt && at + kStageTokens > lo &&
                                   at < hi
                               ? __ldg(table + (at >> bs_shift))
                               : -1;
                };
                int blk = box_block(0);
                for (int i = 0; i < 2 * nt; ++i) {
                    bool is_v;
                    const int j = chunk_place_tile(split, i, nt, is_v);
                    uint32_t boxes = (1u << kChunkBoxes) - 1u;
                    if (is_v && !there) {
                        boxes = __ballot_sync(0xffffffffu, blk >= 0 && blk < p.num_blocks);
                        blk = box_block(j + 1);
                    }
                    ok = wait_for(ptx::smem_addr(&full_bar[slot]), phase);
                    if (!ok) break;
                    if (!is_v || (j >= plain0 && j < plain1)) {
                        leave();
                        continue;
                    }
                    const int t0 = (tile + j) * TT;
                    // a lane keeps to its 16-byte column of every (32 / kCells)-th row
                    uint8_t* column = ring + slot * Cfg::kTileBytes +
                                      (lane % kCells / 8) * Cfg::kRegionBytes + (lane % 8) * 16;
                    constexpr int kStep = 32 / kCells;
                    auto zero = [&](int row0, int row1) {
                        row1 = min(row1, (half + 1) * kRowsEach);
                        for (int r = max(row0, half * kRowsEach) + lane / kCells; r < row1; r += kStep)
                            *reinterpret_cast<uint4*>(column + r * 128) = make_uint4(0u, 0u, 0u, 0u);
                    };
                    auto look_through = [&](int row0, int row1) {
                        row1 = min(row1, (half + 1) * kRowsEach);
                        for (int r = max(row0, half * kRowsEach) + lane / kCells; r < row1;
                             r += 4 * kStep) {
                            uint4 x[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                x[k] = r + k * kStep < row1 ? *reinterpret_cast<const uint4*>(
                                                                  column + (r + k * kStep) * 128)
                                                            : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (any_not_finite(x[k], T())) {
                                    drop_not_finite(x[k].x, T());
                                    drop_not_finite(x[k].y, T());
                                    drop_not_finite(x[k].z, T());
                                    drop_not_finite(x[k].w, T());
                                    atomicMin(&t.bad_from, j);
                                    atomicMax(&t.bad_to, j + 1);
                                    *reinterpret_cast<uint4*>(column + (r + k * kStep) * 128) = x[k];
                                }
                        }
                    };
                    // rows of the tile: none sees those before `a` and from `d` on, all see
                    // those from `b` to `c`
                    auto in_tile = [&](int x) { return min(max(x - t0, 0), TT); };
                    const int a = in_tile(lo), d = max(in_tile(hi), a);
                    const int b = min(max(in_tile(lo_all), a), d);
                    const int c = min(max(in_tile(hi_all), b), d);
                    zero(0, a);
                    look_through(a, b);
                    look_through(c, d);
                    zero(d, TT);
                    if (boxes != (1u << kChunkBoxes) - 1u)
                        for (int x = 0; x < kChunkBoxes; ++x)
                            if (!((boxes >> x) & 1u)) zero(x * kStageTokens, (x + 1) * kStageTokens);
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&clean_bar[slot]));
                    leave();
                }
                if (!ok) break;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_addr(&cleaned[u % kChunkNotes]));
                note_read(u);
            }
        }
    } else {
        // ------------------------------------------------------------ softmax rows
        ptx::reg_inc<kChunkSoftmaxRegs>();
        const int wg = warp / 4;                  // warpgroup
        const int srow = 32 * (warp % 4) + lane;  // row of the tile = tensor-memory lane
        const uint32_t lane_base = (uint32_t)(32 * (warp % 4)) << 16;
        const uint32_t s_col = tmem + lane_base + wg * TT;
        const uint32_t o_col = tmem + lane_base + Cfg::kColO;
        int step = 0;                     // this warpgroup's tiles so far
        int own = 0;                      // units with tiles for it
        int splits = 0;                   // split units so far
        bool free_due = false;            // O and the exchange of the last one may be read
        bool ok = true;

        auto is_split = [&](const ChunkNote& t) { return t.tokens * group <= TR; };
        auto tiles_of = [&](const ChunkNote& t) {
            return t.tiles < 0 ? 0 : is_split(t) ? (t.tiles + 1 - wg) / 2 : t.tiles;
        };
        // this thread's row of a unit: (token of the row block, query head), or a token
        // of -1 past its rows
        auto row_of = [&](const ChunkNote& t, int& head) {
            const int r = is_split(t) ? srow : wg * TR + srow;
            const int token = r / group;
            head = t.g * group + r - token * group;
            return r < t.tokens * group ? token : -1;
        };
        // its row of Q into this warpgroup's tile
        auto load_q = [&](const ChunkNote& t) {
            int head;
            const int token = row_of(t, head);
            const bool live = token >= 0;
            const uint4* src = reinterpret_cast<const uint4*>(
                static_cast<const T*>(p.q) +
                ((int64_t)(t.q_row + max(token, 0)) * p.num_q_heads + (live ? head : 0)) * D);
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
                ptx::cp_async_16(q_addr + wg * Cfg::kTileBytes + (c / 8) * Cfg::kRegionBytes +
                                     srow * 128 + (((c % 8) ^ (srow & 7)) << 4),
                                 src + c, live);
        };
        auto q_loaded = [&] {
            ptx::cp_async_wait_all();
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(ptx::smem_addr(&q_ready[wg]));
        };
        if (note_there(0)) {
            if (tiles_of(notes[0]) > 0) {
                load_q(notes[0]);
                q_loaded();
            }
        } else {
            ok = false;
        }
        for (int u = 0; ok && notes[u % kChunkNotes].tiles >= 0; ++u) {
            ChunkNote& t = notes[u % kChunkNotes];
            const ChunkNote& ahead = notes[(u + 1) % kChunkNotes];
            const bool split = is_split(t);
            const int nt = t.tiles, mine = tiles_of(t), tile = t.tile;
            const int lo_all = t.lo_all, hi_all = t.hi_all;
            int head;
            const int token = row_of(t, head);
            const bool live = token >= 0;
            const uint32_t live_lanes = __ballot_sync(0xffffffffu, live);
            const bool warp_live = live_lanes != 0;
            const int m = t.m + max(token, 0);
            const int lo = chunk_lo(p.shape, m), hi = live && m >= 0 ? max(m + 1, t.prefix) : 0;
            const bool look = !(t.flags & kNotePagesThere);
            const int32_t* table = p.block_tables + (int64_t)t.b * p.max_blocks_per_seq;
            const float slope =
                MOD && p.slopes != nullptr && live ? __ldg(p.slopes + head) * kLog2e : 0.f;
            // lanes 0-7, where the notes do not say that all pages are there: the block of
            // box `lane` of tile j, as the table has it (-1: none)
            auto box_block = [&](int j) {
                const int at = (tile + j) * TT + lane * kStageTokens;
                return look && lane < kChunkBoxes && j < nt && at + kStageTokens > t.lo && at < t.hi
                           ? __ldg(table + (at >> bs_shift))
                           : -1;
            };
            float m_ref = -INFINITY, l = 0.f;
            const int j0 = split ? wg : 0, by = split ? 2 : 1;
            int blk = box_block(j0), blk_next = box_block(j0 + by);  // two steps ahead
            for (int j = j0; j < nt; j += by, ++step) {
                const int t0 = (tile + j) * TT;
                uint32_t boxes = (1u << kChunkBoxes) - 1u;  // (beyond lo and hi all is masked)
                if (look) {
                    boxes = __ballot_sync(0xffffffffu, blk >= 0 && blk < p.num_blocks);
                    blk = blk_next;
                    blk_next = box_block(j + 2 * by);
                }
                // every row of the unit sees the whole tile
                const bool plain = boxes == (1u << kChunkBoxes) - 1u && t0 >= lo_all &&
                                   t0 + TT <= hi_all;
                if (!wait_for(ptx::smem_addr(&s_full[wg]), step & 1)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after_sync();
                if (j + by >= nt) {  // (the last reader of Q's tile is done)
                    if (!note_there(u + 1)) {
                        ok = false;
                        break;
                    }
                    if (tiles_of(ahead) > 0) load_q(ahead);
                }
                if (free_due) {
                    // both warpgroups have read O_0, O_1 and the exchange of the split unit
                    // before; neither is written anew until then
                    if (!wait_for(ptx::smem_addr(o_free), (splits - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    free_due = false;
                }
                if (warp_live) {
                    const float scale = MOD ? 1.f : p.scale_log2;
                    // Two small loops over the row's scores, which are read twice, 32 at a
                    // time: unrolled further, the instructions did not stay in their cache
                    // beside the other warps' (single tokens of 64 sequences of 2500: 123
                    // us, 142 with 64 at a time, 188 with the tile in one piece).

                    // f over the pairs of neighbouring scores
                    auto pairs = [](auto& r, auto f) {
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const float2 y =
                                f(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), i);
                            r[i] = __float_as_uint(y.x);
                            r[i + 1] = __float_as_uint(y.y);
                        }
                    };
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int c = 0; c < TT / 32; ++c) {
                        uint32_t r[32];
                        __syncwarp();
                        ptx::tmem_ld32(s_col + c * 32, r);
                        const int at = t0 + c * 32;
                        if constexpr (MOD) {
                            // the scores themselves, in base-2 units
                            if (p.softcap > 0.f) {
                                // cap tanh(x) = cap - 2 cap / (1 + e^(2x))
                                const float cap2 = p.softcap * kLog2e;
                                pairs(r, [&](float2 y, int) {
                                    y = ptx::mul2(y, make_float2(p.tanh_log2, p.tanh_log2));
                                    y = ptx::add2(
                                        make_float2(ptx::ex2_approx(y.x), ptx::ex2_approx(y.y)),
                                        make_float2(1.f, 1.f));
                                    return ptx::fma2(make_float2(-2.f * cap2, -2.f * cap2),
                                                     make_float2(ptx::rcp_approx(y.x),
                                                                 ptx::rcp_approx(y.y)),
                                                     make_float2(cap2, cap2));
                                });
                            } else if (p.slopes == nullptr) {
                                const float k = p.scale_log2;
                                pairs(r, [&](float2 y, int) {
                                    return ptx::mul2(y, make_float2(k, k));
                                });
                            }
                            if (p.slopes != nullptr) {
                                const float k = p.softcap > 0.f ? 1.f : p.scale_log2;
                                const float base = slope * (float)(at - m);
                                pairs(r, [&](float2 y, int i) {
                                    return ptx::fma2(y, make_float2(k, k),
                                                     make_float2(fmaf(slope, (float)i, base),
                                                                 fmaf(slope, (float)(i + 1), base)));
                                });
                            }
                        }
                        if (!plain) {
                            const int from = lo - at, to = hi - at;
                            uint32_t allow = to >= 32 ? ~0u : to <= 0 ? 0u : (1u << to) - 1u;
                            allow &= from <= 0 ? ~0u : from >= 32 ? 0u : ~0u << from;
                            const uint32_t bb = boxes >> (2 * c);
                            allow &= ((bb & 1u) ? 0x0000ffffu : 0u) |
                                     ((bb & 2u) ? 0xffff0000u : 0u);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!((allow >> i) & 1u)) r[i] = __float_as_uint(-INFINITY);
                        }
                        if (MOD || !plain) ptx::tmem_st32_async(s_col + c * 32, r);
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mx[k] = fmaxf(fmaxf(mx[k], __uint_as_float(r[i + 2 * k])),
                                              __uint_as_float(r[i + 2 * k + 1]));
                    }
                    if (MOD || !plain) ptx::tmem_wait_st();
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
                    float alpha = 1.f;
                    if (m_ref == -INFINITY) {
                        m_ref = top;  // O and l are still zero for this row
                    } else if (top > m_ref + kChunkLazyLog2) {
                        alpha = ptx::ex2_approx(m_ref - top);
                        m_ref = top;
                    }
                    // O is rescaled where a reference moved (the product of the tile before is
                    // complete: S of this one is, and was issued behind it)
                    if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t ov[16];
                            __syncwarp();
                            ptx::tmem_ld16(o_col + wg * D + c * 16, ov);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                            ptx::tmem_st16_async(o_col + wg * D + c * 16, ov);
                        }
                        l *= alpha;
                    }
                    const float ref = (m_ref == -INFINITY ? 0.f : m_ref) - WeightBias<T>::value;
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
                    for (int c = 0; c < TT / 32; ++c) {
                        uint32_t r[32];
                        const uint32_t col = s_col + c * 32;
                        __syncwarp();
                        ptx::tmem_ld32(col, r);
                        pairs(r, [&](float2 y, int i) {
                            y = ptx::fma2(y, make_float2(scale, scale), make_float2(-ref, -ref));
                            y = make_float2(ptx::ex2_approx(y.x), ptx::ex2_approx(y.y));
                            sum[i / 2 % 2] = ptx::add2(sum[i / 2 % 2], y);
                            return y;
                        });
                        if (split) {
                            uint32_t pp[32];
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                split_pair(make_float2(__uint_as_float(r[2 * e]),
                                                       __uint_as_float(r[2 * e + 1])),
                                           pp[e], pp[16 + e], T());
                            ptx::tmem_st32_async(col, pp);
                        } else {
                            uint32_t ph[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                ph[e] = pack2(__uint_as_float(r[2 * e]),
                                              __uint_as_float(r[2 * e + 1]), T());
                            ptx::tmem_st16_async(col, ph);
                        }
                        if (c % 2 == 1) {  // half a tile, or all of it
                            ptx::tmem_wait_st();
                            ptx::tc_fence_before_sync();
                            __syncwarp();
                            if (lane == 0)
                                ptx::mbar_arrive(
                                    ptx::smem_addr(c < TT / 64 ? &p_half[wg] : &p_ready[wg]));
                        }
                    }
                    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                } else if (lane == 0) {
                    ptx::mbar_arrive(ptx::smem_addr(&p_half[wg]));
                    ptx::mbar_arrive(ptx::smem_addr(&p_ready[wg]));
                }
            }
            if (!ok) break;
            if (mine == 0 && !note_there(u + 1)) break;
            const bool load_ahead = tiles_of(ahead) > 0;
            if (load_ahead) {
                if (mine == 0) load_q(ahead);
                q_loaded();
            }

            // the unit's last O += P V
            if (mine > 0) {
                if (!wait_for(ptx::smem_addr(&o_done[wg]), own & 1)) break;
                ++own;
            }
            float fa, fb = 0.f;  // out = O_0 fa + O_1 fb (not split: O_w fa)
            float sum, top;      // of the weights; their reference
            const bool two = split && nt > 1;  // O_1 has something
            if (!split) {
                sum = l;
                top = m_ref;
                fa = 1.f;
            } else {
                // both warpgroups are through: their parts of the softmax meet
                if (free_due) {
                    if (!wait_for(ptx::smem_addr(o_free), (splits - 1) & 1)) break;
                    free_due = false;
                }
                xch[wg * TR + srow] = make_float2(m_ref, l);
                ptx::tc_fence_before_sync();
                ptx::mbar_arrive(ptx::smem_addr(met));
                if (!wait_for(ptx::smem_addr(met), splits & 1)) break;
                const float2 ha = xch[srow], hb = xch[TR + srow];
                top = fmaxf(ha.x, hb.x);
                fa = ha.x == -INFINITY ? 0.f : ptx::ex2_approx(ha.x - top);
                fb = hb.x == -INFINITY ? 0.f : ptx::ex2_approx(hb.x - top);
                sum = ha.y * fa + hb.y * fb;
            }
            // (a sum is 0 or 1 at least: the score that set the reference is in it)
            const float inv = sum == 0.f ? 0.f : ptx::rcp_approx(sum);
            fa *= inv;
            fb *= inv;
            ptx::tc_fence_after_sync();
            const int partial = t.partial;
            const bool direct = partial < 0;
            if (!wait_for(ptx::smem_addr(&cleaned[u % kChunkNotes]), (u / kChunkNotes) & 1))
                break;
            const bool bad_v = t.bad_to != 0;
            // Columns: the whole row; of a split unit this warpgroup's half.
            const int cols = split ? D / 2 : D;
            const int col0 = split ? wg * cols : 0;
            const int64_t out_row =
                (int64_t)(t.q_row + max(token, 0)) * p.num_q_heads + (live ? head : 0);
            const int urow = split ? srow : wg * TR + srow;
            // where columns 4 c .. of row r of the partial lie
            auto partial_at = [&](int c, int r) {
                return reinterpret_cast<float4*>(p.partial_o) +
                       ((int64_t)partial * (D / 4) + c) * 2 * TR + r;
            };
#pragma unroll 1
            for (int c = 0; c < cols; c += 32) {
                if (!warp_live) break;
                float v[32];
                uint32_t ov[32];
                __syncwarp();
                ptx::tmem_ld32(o_col + (split ? 0 : wg * D) + col0 + c, ov);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(ov[i]) * fa;
                if (two) {
                    ptx::tmem_ld32(o_col + D + col0 + c, ov);
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = fmaf(__uint_as_float(ov[i]), fb, v[i]);
                }
                if (direct && t.tokens * group <= 32) {
                    // few rows: each lane its own, in fewer instructions
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + out_row * D +
                                                          col0 + c);
                    if (live)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            dst[i] = make_uint4(pack2(v[8 * i], v[8 * i + 1], T()),
                                                pack2(v[8 * i + 2], v[8 * i + 3], T()),
                                                pack2(v[8 * i + 4], v[8 * i + 5], T()),
                                                pack2(v[8 * i + 6], v[8 * i + 7], T()));
                } else if (direct) {
                    // Four lanes trade 16-byte pieces of their rows, so that a store writes
                    // 64 bytes of each of eight rows, not 16 of 32
                    const int quad = lane & ~3, piece = lane & 3;
                    uint4 x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[i] = make_uint4(pack2(v[8 * i], v[8 * i + 1], T()),
                                          pack2(v[8 * i + 2], v[8 * i + 3], T()),
                                          pack2(v[8 * i + 4], v[8 * i + 5], T()),
                                          pack2(v[8 * i + 6], v[8 * i + 7], T()));
                    trade_pieces(x, lane);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int64_t row = __shfl_sync(0xffffffffu, out_row, quad + i);
                        if ((live_lanes >> (quad + i)) & 1u)
                            reinterpret_cast<uint4*>(static_cast<T*>(p.out) + row * D + col0 +
                                                     c)[piece] = x[i];
                    }
                } else if (live) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *partial_at((col0 + c) / 4 + i, urow) =
                            make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                }
            }
            __syncwarp();  // (what the lanes wrote of each other's rows is there)
            if (bad_v && live) {
                const ChunkSeen seen = {table, max(lo, (tile + t.bad_from) * TT),
                                        min(hi, (tile + t.bad_to) * TT), lo_all, hi_all, t.g};
                add_not_finite<T, D>(p, seen, col0, cols, [&](int c, float x) {
                    if (direct) {
                        T* o = static_cast<T*>(p.out) + out_row * D + c;
                        *o = from_float(as_float(*o) + x, T());
                    } else {
                        reinterpret_cast<float*>(partial_at(c / 4, urow))[c % 4] += x;
                    }
                });
            }
            if (live && !direct && (!split || wg == 0))
                p.partial_lse[(int64_t)partial * 2 * TR + urow] =
                    sum == 0.f ? -INFINITY : top - WeightBias<T>::value + log2f(sum);
            if (split) {
                ptx::tc_fence_before_sync();
                ptx::mbar_arrive(ptx::smem_addr(o_free));
                free_due = true;
                ++splits;
            }
            note_read(u);
        }
        // a warp that gave up a wait may have the next unit's queries on their way
        ptx::cp_async_wait_all();
    }

    if (gave_up && lane == 0) flag_error(p.err_flag, PKV_EFLAG_TIMEOUT);
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == kChunkMmaWarp) {
        __syncwarp();
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// Joins the partials of the units that were cut: w_c = 2^(lse_c - max),
// out = sum_c w_c O_c / sum_c w_c over the unit's segments, with a running maximum.  The
// segment that ends a unit has its record; a CTA takes 16 of its rows, eight lanes a row.
constexpr int kChunkMergeThreads = 128;
constexpr int kChunkMergeRows = kChunkMergeThreads / 8;

template <typename T, int D>
__global__ void __launch_bounds__(kChunkMergeThreads) chunk_merge_kernel(const ChunkParams p) {
    constexpr int E = D / 32;  // float4 columns of a lane: 8 k + lane % 8
    constexpr int F = 4;       // partials in flight
    ptx::launch_dependents();
    ptx::grid_dependency_wait();
    const int segment = blockIdx.x;
    const int row = blockIdx.y * kChunkMergeRows + (threadIdx.x >> 3), q8 = threadIdx.x & 7;
    const int4 words = __ldg(reinterpret_cast<const int4*>(p.records) + segment);
    const ChunkRecord r = {words.x, words.y, words.z, words.w};
    if (!chunk_record_valid(r, segment, p.num_seqs, p.shape.heads)) return;
    const ChunkSeq s = chunk_load(p, r.b);
    const int64_t token0 = (int64_t)r.rb * p.shape.block_tokens;
    const int token = row / p.shape.group;
    if (token >= p.shape.block_tokens || token0 + token >= s.tokens) return;
    float m = -INFINITY, den = 0.f;
    float4 acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = r.first; c <= segment; c += F) {
        float lse[F];
        float4 x[F][E];
#pragma unroll
        for (int f = 0; f < F; ++f) {
            // a unit's first segment leaves the partial that it begins, the others that
            // which was begun before them
            const int slot = chunk_partial(min(c + f, segment), c + f == r.first);
            const int64_t at = (int64_t)slot * 2 * kChunkRows + row;
            const bool has = c + f <= segment && __ldg(p.has + slot) == 1;
            lse[f] = has ? __ldg(p.partial_lse + at) : -INFINITY;
            const float4* o = reinterpret_cast<const float4*>(p.partial_o) +
                              ((int64_t)slot * (D / 4) + q8) * 2 * kChunkRows + row;
#pragma unroll
            for (int e = 0; e < E; ++e)
                x[f][e] = has ? __ldg(o + e * 16 * kChunkRows) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float mn = m;
#pragma unroll
        for (int f = 0; f < F; ++f) mn = fmaxf(mn, lse[f]);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float old = exp2f(m - ref);
        m = mn;
        den *= old;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            acc[e].x *= old;
            acc[e].y *= old;
            acc[e].z *= old;
            acc[e].w *= old;
        }
#pragma unroll
        for (int f = 0; f < F; ++f) {
            const float w = exp2f(lse[f] - ref);
            den += w;
            if (w == 0.f) continue;  // adds nothing, whatever it weighs
#pragma unroll
            for (int e = 0; e < E; ++e) {
                acc[e].x = fmaf(w, x[f][e].x, acc[e].x);
                acc[e].y = fmaf(w, x[f][e].y, acc[e].y);
                acc[e].z = fmaf(w, x[f][e].z, acc[e].z);
                acc[e].w = fmaf(w, x[f][e].w, acc[e].w);
            }
        }
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    const int64_t out_row = (s.first + token0 + token) * p.num_q_heads + r.g * p.shape.group + row -
                            token * p.shape.group;
    uint2* out = reinterpret_cast<uint2*>(static_cast<T*>(p.out) + out_row * D) + q8;
#pragma unroll
    for (int e = 0; e < E; ++e)
        out[8 * e] = make_uint2(pack2(acc[e].x * inv, acc[e].y * inv, T()),
                                pack2(acc[e].z * inv, acc[e].w * inv, T()));
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// The plan of a call: the CTAs, the rounds at most, and the workspace.
constexpr int kChunkMaxContext = INT_MAX - 1024;  // positions of the last tile fit an int
struct ChunkCallPlan {
    int ctas;
    int rounds;
    bool cut;  // a unit may be cut: partials and a join
    size_t records_bytes;
    size_t has_bytes;
    size_t workspace_bytes;
};

static pkv_status check_chunk(int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads,
                              int head_dim, int block_size, int max_context_len) {
    const pkv_status st = check_shapes(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size,
                                       max_context_len, 0);
    if (st != PKV_OK) return st;
    if (num_tokens < 0) return PKV_ERR_INVALID_ARG;
    if (max_context_len > kChunkMaxContext) return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

static pkv_status plan_chunk(int num_seqs, int num_tokens, int num_q_heads, int num_kv_heads,
                             int head_dim, int block_size, int max_context_len,
                             ChunkCallPlan* plan) {
    const pkv_status st = check_chunk(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim,
                                      block_size, max_context_len);
    if (st != PKV_OK) return st;
    const int sms = current_sm_count();
    if (sms <= 0) return PKV_ERR_CUDA;
    // the line at most: every unit as long as the longest context
    const int block_tokens = 2 * kChunkRows / (num_q_heads / num_kv_heads);
    const double units = (double)num_kv_heads *
                         ((double)num_tokens / block_tokens + std::min(num_seqs, num_tokens));
    const double places = units * ((double)kChunkUnitCost + max_context_len);
    if (places > 1e15) return PKV_ERR_UNSUPPORTED;  // (times the segments, within 64 bits)
    plan->ctas = (int)std::max(1.0, std::min((double)sms, std::ceil(places / kChunkLeastSegment)));
    plan->rounds = (int)std::max(
        1.0, std::min((double)kChunkMaxRounds, places / ((double)plan->ctas * kChunkRoundSegment)));
    plan->cut = max_context_len > kChunkTile;
    const size_t segments = (size_t)plan->ctas * plan->rounds;
    plan->records_bytes = (segments * sizeof(ChunkRecord) + 255) & ~size_t(255);
    plan->has_bytes = (chunk_partials((int)segments) * sizeof(int32_t) + 255) & ~size_t(255);
    plan->workspace_bytes =
        256 + (plan->cut ? plan->records_bytes + plan->has_bytes +
                               (size_t)chunk_partials((int)segments) * 2 * kChunkRows *
                                   (head_dim + 1) * sizeof(float)
                         : 0);
    return PKV_OK;
}

template <typename T, int D, bool MOD>
static cudaError_t launch_chunk_t(const CUtensorMap& mk, const CUtensorMap& mv,
                                  const ChunkParams& p, const ChunkCallPlan& plan,
                                  cudaStream_t stream) {
    using Cfg = ChunkTileCfg<D>;
    auto kern = chunk_attention_kernel<T, D, MOD>;
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
    cfg.blockDim = dim3(kChunkThreads);
    cfg.dynamicSmemBytes = Cfg::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, mk, mv, p);
    if (e != cudaSuccess || !plan.cut) return e;
    const int64_t rows = std::min<int64_t>(2 * kChunkRows, (int64_t)p.num_tokens * p.shape.group);
    cfg.gridDim = dim3(plan.ctas * plan.rounds,
                       (unsigned)((rows + kChunkMergeRows - 1) / kChunkMergeRows));
    cfg.blockDim = dim3(kChunkMergeThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, chunk_merge_kernel<T, D>, p);
}

template <typename T>
static cudaError_t launch_chunk(const CUtensorMap& mk, const CUtensorMap& mv, const ChunkParams& p,
                                const ChunkCallPlan& plan, int head_dim, cudaStream_t stream) {
    // the plain kernel takes the largest score before it multiplies by the scale
    const bool mod = p.softcap > 0.f || p.slopes != nullptr || !(p.scale_log2 > 0.f);
    if (head_dim == 64)
        return mod ? launch_chunk_t<T, 64, true>(mk, mv, p, plan, stream)
                   : launch_chunk_t<T, 64, false>(mk, mv, p, plan, stream);
    return mod ? launch_chunk_t<T, 128, true>(mk, mv, p, plan, stream)
               : launch_chunk_t<T, 128, false>(mk, mv, p, plan, stream);
}

}  // namespace pkv

using namespace pkv;

extern "C" size_t pkv_chunk_attention_workspace_size(int num_seqs, int num_tokens, int num_q_heads,
                                                     int num_kv_heads, int head_dim,
                                                     int block_size, int max_context_len) {
    ChunkCallPlan plan;
    if (plan_chunk(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size,
                   max_context_len, &plan) != PKV_OK)
        return SIZE_MAX;
    return plan.workspace_bytes;
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
    const auto over = [&](const void* a, int64_t bytes) {
        return a != nullptr && overlap(out, q_bytes, a, bytes);
    };
    if ((out != q && over(q, q_bytes)) || over(block_tables, seqs * max_blocks_per_seq * 4) ||
        over(context_lens, seqs * 4) || over(query_starts, (seqs + 1) * 4) ||
        over(prefix_lens, seqs * 4) || over(slopes, (int64_t)num_q_heads * 4) ||
        over(k_cache, cache_bytes) || over(v_cache, cache_bytes))
        return PKV_ERR_INVALID_ARG;
    ChunkCallPlan plan;
    st = plan_chunk(num_seqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size,
                    max_context_len, &plan);
    if (st != PKV_OK) return st;
    if (workspace_bytes < plan.workspace_bytes) return PKV_ERR_WORKSPACE;
    if (over(workspace, (int64_t)plan.workspace_bytes)) return PKV_ERR_INVALID_ARG;

    CUtensorMap mk, mv;
    if (!make_cache_map(&mk, k_cache, dtype, num_blocks, block_size, num_kv_heads, head_dim, hnd) ||
        !make_cache_map(&mv, v_cache, dtype, num_blocks, block_size, num_kv_heads, head_dim, hnd))
        return PKV_ERR_CUDA;
    ChunkParams p = {};
    p.out = out;
    p.q = q;
    p.v_cache = v_cache;
    p.block_tables = block_tables;
    p.query_starts = query_starts;
    p.context_lens = context_lens;
    p.prefix_lens = prefix_lens;
    p.slopes = slopes;
    p.err_flag = err_flag;
    if (plan.cut) {
        char* at = static_cast<char*>(workspace);
        p.records = reinterpret_cast<ChunkRecord*>(at);
        p.has = reinterpret_cast<int32_t*>(at + plan.records_bytes);
        p.partial_o = reinterpret_cast<float*>(at + plan.records_bytes + plan.has_bytes);
        p.partial_lse = p.partial_o + (size_t)chunk_partials(plan.ctas * plan.rounds) * 2 *
                                          kChunkRows * head_dim;
    }
    p.shape.group = num_q_heads / num_kv_heads;
    p.shape.block_tokens = 2 * kChunkRows / p.shape.group;
    p.shape.heads = num_kv_heads;
    p.shape.window = window;
    p.rounds = plan.rounds;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.num_q_heads = num_q_heads;
    p.cap = std::min(max_blocks_per_seq * block_size, max_context_len);
    p.hnd = hnd;
    p.scale_log2 = scale * kLog2e;
    p.softcap = softcap;
    p.tanh_log2 = softcap > 0.f ? 2.f * kLog2e * scale / softcap : 0.f;
    cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = dtype == PKV_FP16 ? launch_chunk<__half>(mk, mv, p, plan, head_dim, s)
                                            : launch_chunk<__nv_bfloat16>(mk, mv, p, plan, head_dim, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
    }
    return PKV_OK;
}
