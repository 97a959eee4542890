"""The line of work of a ragged step's attention, cut into segments (CPU)."""
import ctypes
import os
import random
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "paged_kv_cache_164_gb300", "csrc")
SOURCE = """#include "pkv_chunk_line.cuh"
using namespace pkv;
static ChunkSeq seq(const int* s) { return {s[0], s[1], s[2], s[3]}; }
static ChunkShape shape(const int* c) { return {c[0], c[1], c[2], c[3]}; }
extern "C" long long places(const int* s, const int* c) { return chunk_places(seq(s), shape(c)); }
extern "C" long long before(const int* s, const int* c, int k) { return chunk_before(seq(s), shape(c), k); }
extern "C" int width(const int* s, const int* c, int rb) { return chunk_width(seq(s), shape(c), rb); }
extern "C" int blocks(const int* s, const int* c) { return chunk_blocks(seq(s), shape(c)); }
extern "C" int segment_of(long long line, int segments, long long at) { return chunk_segment_of(line, segments, at); }
extern "C" long long start_of(long long line, int segments, int s) { return chunk_segment_start(line, segments, s); }
extern "C" int valid(int first, int b, int g, int rb, int segment, int seqs, int heads) {
    return chunk_record_valid({first, b, g, rb}, segment, seqs, heads);
}
// walks a segment: 14 numbers a stretch into out
extern "C" int walk(const int* seqs, const int* c, int b, long long in_seq, long long at,
                    long long end, long long* out, int room) {
    const ChunkShape sh = shape(c);
    ChunkWalk w;
    w.at = at;
    w.end = end;
    w.enter(seq(seqs + 4 * b), sh, b, in_seq);
    ChunkStretch t;
    int n = 0;
    while (n < room && w.next_any(sh, [&](int i) { return seq(seqs + 4 * i); }, t)) {
        const long long x[14] = {t.b, t.g, t.rb, t.token0, t.tokens, t.lo, t.hi, t.lo_all, t.hi_all,
                                 t.tile, t.tiles, t.skipped, t.unit_tiles, t.begins};
        for (int i = 0; i < 14; ++i) out[14 * n + i] = x[i];
        ++n;
    }
    return n;
}
"""
TILE, COST = 128, 384


@pytest.fixture(scope="module")
def line(tmp_path_factory):
    folder = tmp_path_factory.mktemp("line")
    (folder / "line.cpp").write_text(SOURCE)
    out = folder / "line.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=undefined",
                    "-fno-sanitize-recover", "-shared", "-fPIC", "-I", CSRC, "-o", str(out),
                    str(folder / "line.cpp")], check=True)
    lib = ctypes.CDLL(str(out))
    for n in ("places", "before", "start_of"):
        getattr(lib, n).restype = ctypes.c_longlong
    return lib


def _ints(v):
    return (ctypes.c_int * len(v))(*v)


def _batch(r):
    group = r.choice([1, 2, 3, 4, 5, 7, 8, 11, 16])
    shape = [256 // group, group, r.choice([1, 2, 3]), r.choice([0, 0, 1, 50, 128, 1000])]
    seqs, first = [], 0
    for _ in range(r.randint(1, 8)):
        t = r.choice([0, 1, 1, r.randint(1, 40), r.randint(1, 900)])
        n = t + r.choice([0, 0, r.randint(0, 200), r.randint(0, 3500)])
        if r.random() < 0.1:
            n = max(0, t - r.randint(1, 50))  # flagged: rows without a position
        seqs.append([first, t, n, min(n, r.choice([0, 0, r.randint(0, 1000)]))])
        first += t
    return shape, seqs


def test_sums_of_places_are_those_of_the_blocks(line):
    r = random.Random(1)
    for _ in range(400):
        shape, seqs = _batch(r)
        for s in seqs:
            total = 0
            c, cs = _ints(s), _ints(shape)
            for k in range(line.blocks(c, cs)):
                assert line.before(c, cs, k) == total
                total += line.width(c, cs, k)
            if s[1]:
                assert line.before(c, cs, line.blocks(c, cs)) == total
            assert line.places(c, cs) == (total * shape[2] if s[1] else 0)
    # the largest numbers stay within 64 bits
    s, c = [0, 2 ** 27, 2 ** 31 - 1025, 0], [16, 16, 8, 0]
    assert 0 < line.places(_ints(s), _ints(c)) < 2 ** 62


def test_segments_take_every_tile_of_every_unit_once(line):
    r = random.Random(2)
    for _ in range(300):
        shape, seqs = _batch(r)
        cs, flat = _ints(shape), _ints([x for s in seqs for x in s])
        parts = [line.places(_ints(s), cs) for s in seqs]
        total = sum(parts)
        if total == 0:
            continue
        segments = min(r.choice([1, 2, 3, 7, 40]), total)
        seen, partials, ended = {}, {}, {}
        for seg in range(segments):
            at, end = line.start_of(total, segments, seg), line.start_of(total, segments, seg + 1)
            if at == end:
                continue
            b, rest = 0, at
            while rest >= parts[b]:
                rest -= parts[b]
                b += 1
            out = (ctypes.c_longlong * (14 * 5000))()
            n = line.walk(flat, cs, b, ctypes.c_longlong(rest), ctypes.c_longlong(at),
                          ctypes.c_longlong(end), out, 5000)
            assert 0 < n < 5000
            for i in range(n):
                (b, g, rb, token0, tokens, lo, hi, lo_all, hi_all, tile, tiles, skipped, unit_tiles,
                 begins) = out[14 * i:14 * i + 14]
                _, t, ctx, prefix = seqs[b]
                assert 0 <= g < shape[2] and token0 == rb * shape[0]
                assert tokens == min(shape[0], t - token0) > 0
                ms = [ctx - t + token0 + x for x in (0, tokens - 1)]
                his = [0 if m < 0 else max(m + 1, prefix) for m in ms]
                los = [max(0, m + 1 - shape[3]) if shape[3] and m >= 0 else 0 for m in ms]
                assert (lo, hi, lo_all, hi_all) == (los[0], his[1], los[1], his[0])
                key = (b, g, rb)
                done = seen.setdefault(key, 0)
                assert skipped == done and tile == lo // TILE + done
                assert unit_tiles == max(1, -(-hi // TILE) - lo // TILE)
                assert bool(begins) == (key not in partials)
                seen[key] = done + tiles
                # the segments of a unit are consecutive, each with a partial of its own
                slot = 2 * seg + (1 if begins else 0)
                partials.setdefault(key, []).append((slot, tiles))
                first = partials[key][0][0] // 2
                assert seg - first == len(partials[key]) - 1
                if skipped + tiles == unit_tiles:
                    ended.setdefault(key, seg)
        assert set(seen) == set(ended)  # each to its last tile
        expect = {(b, g, rb) for b, s in enumerate(seqs) for g in range(shape[2])
                  for rb in range(-(-s[1] // shape[0]))}
        assert set(seen) == expect
        slots = [x for p in partials.values() for x, _ in p]
        cut = [x for p in partials.values() if len(p) > 1 for x, _ in p]
        assert len(set(cut)) == len(cut) and max(slots) < 2 * segments


def test_the_segment_of_a_place(line):
    r = random.Random(3)
    for _ in range(300):
        total, segments = r.randint(1, 10 ** 6), r.randint(1, 700)
        starts = [line.start_of(ctypes.c_longlong(total), segments, s) for s in range(segments + 1)]
        for _ in range(20):
            x = r.randrange(total)
            s = line.segment_of(ctypes.c_longlong(total), segments, ctypes.c_longlong(x))
            assert starts[s] <= x < starts[s + 1]


def test_records_that_lead_out_of_the_launch_are_not_followed(line):
    words = [0, 1, 5, 6, -1, -2 ** 31, 2 ** 31 - 1, 0x7F7F7F7F]
    for first in words:
        for b in words:
            for g in words:
                if line.valid(first, b, g, 0, 5, 6, 2):
                    assert 0 <= first < 5 and 0 <= b < 6 and 0 <= g < 2
    assert line.valid(0, 5, 1, 3, 5, 6, 2) and not line.valid(0, 0, 0, -1, 5, 6, 2)
