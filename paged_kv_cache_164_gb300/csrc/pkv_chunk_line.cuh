// The work of a ragged step's attention as one line, cut into equal segments.  Plain
// C++ on the host too, so that it is tested there.
//
// A sequence's new tokens are taken in row blocks of `block_tokens`; a unit is a row
// block of one KV head, and meets the 128-position tiles that any of its rows sees.
// On the line (sequence, KV head, row block; the last fastest) a unit has as many
// places as it sees positions, and kChunkUnitCost more for what it costs besides: its
// queries, its first products with nothing to run beside, its masked tiles and its
// output.  Places are linear in the row block, so that the sum over a sequence's
// blocks is a closed form and a segment's start is found without walking there.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define PKV_LINE __host__ __device__ __forceinline__
#else
#define PKV_LINE inline
#endif

namespace pkv {

constexpr int kChunkRows = 128;      // rows of a softmax warpgroup
constexpr int kChunkTile = 128;      // positions of a tile
constexpr int kChunkUnitCost = 384;  // places of a unit beside its positions

PKV_LINE int line_min(int a, int b) { return a < b ? a : b; }
PKV_LINE int line_max(int a, int b) { return a > b ? a : b; }

// A sequence's part of the step: its first row of q, its new tokens, its context and
// the positions of its prefix, each within its limits.
struct ChunkSeq {
    int first, tokens, n, prefix;
};

// What the call says, the same for all of its sequences.
struct ChunkShape {
    int block_tokens;  // of a row block
    int group;         // query heads of a KV head
    int heads;         // KV heads
    int window;        // 0: none
};

// Positions seen by the token at position m: lo .. hi - 1.
PKV_LINE int chunk_hi(const ChunkSeq& s, int m) { return m < 0 ? 0 : line_max(m + 1, s.prefix); }
PKV_LINE int chunk_lo(const ChunkShape& c, int m) {
    return c.window > 0 && m >= 0 ? line_max(0, m + 1 - c.window) : 0;
}

PKV_LINE int chunk_blocks(const ChunkSeq& s, const ChunkShape& c) {
    return (s.tokens + c.block_tokens - 1) / c.block_tokens;
}

// Places of row block rb of a head.
PKV_LINE int chunk_width(const ChunkSeq& s, const ChunkShape& c, int rb) {
    const int before = s.n - s.tokens;
    const int hi = line_max(s.prefix, line_min(s.n, before + (rb + 1) * c.block_tokens));
    const int lo = c.window > 0 ? line_max(0, before + rb * c.block_tokens + 1 - c.window) : 0;
    return kChunkUnitCost + line_max(0, hi - lo);
}

// The sum of max(floor, start + i step) over i < k.
PKV_LINE int64_t chunk_sum(int floor, int start, int step, int k) {
    int64_t below = 0;  // terms that are the floor
    if (start < floor) below = ((int64_t)floor - start + step - 1) / step;
    if (below > k) below = k;
    const int64_t rest = k - below;
    return below * floor + rest * start + step * ((int64_t)k * (k - 1) - below * (below - 1)) / 2;
}

// Places of a head's row blocks before block k.
PKV_LINE int64_t chunk_before(const ChunkSeq& s, const ChunkShape& c, int k) {
    const int before = s.n - s.tokens, q = c.block_tokens;
    int64_t sum = (int64_t)kChunkUnitCost * k + chunk_sum(s.prefix, before + q, q, k);
    if (k > 0 && k == chunk_blocks(s, c))  // the last block ends at n
        sum -= line_max(s.prefix, before + k * q) - line_max(s.prefix, s.n);
    if (c.window > 0) sum -= chunk_sum(0, before + 1 - c.window, q, k);
    return sum;
}

// Places of a sequence.
PKV_LINE int64_t chunk_places(const ChunkSeq& s, const ChunkShape& c) {
    return s.tokens <= 0 ? 0 : c.heads * chunk_before(s, c, chunk_blocks(s, c));
}

// A segment's part of a unit.
struct ChunkStretch {
    ChunkSeq seq;
    int b, g, rb;
    int token0, tokens;  // of the row block, within the sequence's new ones
    int lo, hi;          // positions that any of its rows sees
    int lo_all, hi_all;  // that all of them see: lo_all .. hi_all - 1
    int tile;            // first tile (of the sequence's) of the stretch
    int tiles;           // of the stretch; may be none
    int skipped;         // the unit's tiles before it
    int unit_tiles;
    bool begins;         // the segment meets the unit's first place
    int64_t unit_at;     // that place on the line
    int64_t at;          // the stretch's first place
    int segment;         // (the caller's)
};

// Walks a segment's part of the line.
struct ChunkWalk {
    int64_t at, end;
    ChunkSeq seq;
    int b, g, rb, pos;  // pos: within the unit's places

    // Stands at place `x` of sequence b's part of the line.
    PKV_LINE void enter(const ChunkSeq& s, const ChunkShape& c, int b_, int64_t x) {
        seq = s;
        b = b_;
        const int blocks = chunk_blocks(s, c);
        const int64_t head = chunk_before(s, c, blocks);
        g = (int)(x / head);
        x -= g * head;
        int lo = 0, hi = blocks - 1;  // the last block that begins at or before x
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (chunk_before(s, c, mid) <= x)
                lo = mid;
            else
                hi = mid - 1;
        }
        rb = lo;
        pos = (int)(x - chunk_before(s, c, lo));
    }

    // The next unit's stretch, empty ones too.  load(b) reads a sequence.
    template <typename Load>
    PKV_LINE bool next_any(const ChunkShape& c, Load load, ChunkStretch& t) {
        if (at >= end) return false;
        const int width = chunk_width(seq, c, rb);
        const int64_t left = end - at;
        const int take = left < width - pos ? (int)left : width - pos;
        t.seq = seq;
        t.b = b;
        t.g = g;
        t.rb = rb;
        t.token0 = rb * c.block_tokens;
        t.tokens = line_min(seq.tokens - t.token0, c.block_tokens);
        const int m = seq.n - seq.tokens + t.token0;  // the first row's position
        t.lo = chunk_lo(c, m);
        t.hi = chunk_hi(seq, m + t.tokens - 1);
        t.lo_all = chunk_lo(c, m + t.tokens - 1);
        t.hi_all = chunk_hi(seq, m);
        const int tile0 = t.lo / kChunkTile;
        t.unit_tiles = line_max(1, (t.hi + kChunkTile - 1) / kChunkTile - tile0);
        const int upto = pos + take;
        t.skipped = part(pos, width, t.unit_tiles);
        t.tiles = part(upto, width, t.unit_tiles) - t.skipped;
        t.tile = tile0 + t.skipped;
        t.begins = pos == 0;
        t.unit_at = at - pos;
        t.at = at;
        at += take;
        pos = upto;
        if (upto == width) {
            pos = 0;
            if (t.token0 + t.tokens < seq.tokens) {
                ++rb;
            } else {
                rb = 0;
                if (++g == c.heads) {
                    g = 0;
                    do {
                        ++b;
                        if (at >= end) break;
                        seq = load(b);
                    } while (seq.tokens <= 0);
                }
            }
        }
        return true;
    }
    template <typename Load>
    PKV_LINE bool next(const ChunkShape& c, Load load, ChunkStretch& t) {
        do {
            if (!next_any(c, load, t)) return false;
        } while (t.tiles == 0);
        return true;
    }

    // Tiles of a unit before its place `pos`.
    static PKV_LINE int part(int pos, int width, int tiles) {
        if (pos == width) return tiles;
        return pos <= kChunkUnitCost ? 0 : line_min(tiles, (pos - kChunkUnitCost) / kChunkTile);
    }
};

// A unit that is cut leaves partials: a segment at most two, that of the unit which one
// before it began, then that of the unit which it begins itself.
PKV_LINE int chunk_partials(int segments) { return 2 * segments; }
PKV_LINE int chunk_partial(int segment, bool begins) { return 2 * segment + (begins ? 1 : 0); }

// The first place of a segment, and the segment of a place, of a line of `line` places.
PKV_LINE int64_t chunk_segment_start(int64_t line, int segments, int segment) {
    return line * segment / segments;
}
PKV_LINE int chunk_segment_of(int64_t line, int segments, int64_t place) {
    return (int)(((place + 1) * segments - 1) / line);
}

// What the segment that ends a cut unit leaves for the join of its partials: the
// segments first .. itself.  -1 where there is none.
struct ChunkRecord {
    int first;
    int b, g, rb;
};
// Whether a record, which a CTA that gave up a wait leaves as the workspace came, names
// what the launch has.
PKV_LINE bool chunk_record_valid(const ChunkRecord& r, int segment, int num_seqs, int heads) {
    return r.first >= 0 && r.first < segment && r.b >= 0 && r.b < num_seqs && r.g >= 0 &&
           r.g < heads && r.rb >= 0;
}

}  // namespace pkv
