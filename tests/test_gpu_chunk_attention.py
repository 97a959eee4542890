"""Attention of a ragged step's new tokens against the definition in 64 bits (GPU)."""
import math

import pytest
import torch

import paged_kv_cache_164_gb300 as pkv
import ragged_reference as ref

pytestmark = pytest.mark.gpu


def _call(c, out=None, **kw):
    return pkv.chunk_attention(c["q"], c["k"], c["v"], c["tables"], c["starts"], c["lens"],
                               c["max_len"], scale=c["scale"], softcap=c["softcap"],
                               window=c["window"], slopes=c["slopes"], prefix_lens=c["prefix"],
                               out=out, layout=c["layout"], **kw)


def _check(c, flags=0, skip_blocks=(), expect=None):
    out, bound = ref.attention(c, skip_blocks) if expect is None else expect
    g = ref.on_gpu(c)
    before = torch.full_like(g["q"], 7.0)
    got = before.clone()
    flag = pkv.new_error_flag("cuda")
    _call(g, out=got, err_flag=flag)
    assert pkv.check_error(flag) == flags
    return ref.assert_close(got, out, bound, before)


# (context, new tokens) of sequences: one token to a few hundred, empty ones between
SHORT = [(1, 1), (0, 0), (16, 3), (17, 17), (50, 1), (33, 0), (64, 5)]
MIXED = [(700, 1), (300, 130), (129, 129), (1, 1), (515, 2), (257, 1)]
LONG = [(900, 400), (2300, 1)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("h_q,h_kv,d", [(4, 2, 64), (8, 1, 128), (3, 3, 128), (16, 1, 64)])
def test_short_sequences(dtype, h_q, h_kv, d):
    _check(ref.make_chunk(1, SHORT, h_q, h_kv, d, 16, dtype, lead=2))


@pytest.mark.parametrize("bs,layout", [(16, "hnd"), (32, "nhd"), (64, "hnd"), (128, "nhd")])
@pytest.mark.parametrize("h_q,h_kv,d", [(5, 1, 128), (8, 2, 64)])
def test_pages_and_layouts(bs, layout, h_q, h_kv, d):
    _check(ref.make_chunk(2, MIXED, h_q, h_kv, d, bs, "bf16", layout))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("h_q,h_kv,d", [(1, 1, 128), (6, 2, 128), (8, 1, 64), (16, 1, 128),
                                        (11, 1, 64)])
def test_chunks_of_several_row_blocks(dtype, h_q, h_kv, d):
    _check(ref.make_chunk(3, LONG, h_q, h_kv, d, 16, dtype))


@pytest.mark.parametrize("window", [1, 2, 31, 64, 65, 200, 5000])
@pytest.mark.parametrize("h_q,h_kv,d", [(4, 1, 64), (2, 2, 128)])
def test_sliding_windows(window, h_q, h_kv, d):
    _check(ref.make_chunk(4, MIXED, h_q, h_kv, d, 32, "fp16", window=window))


@pytest.mark.parametrize("window", [0, 40])
def test_prefixes_that_every_token_sees(window):
    _check(ref.make_chunk(5, MIXED, 8, 2, 64, 16, "bf16", window=window,
                          prefix=[650, 300, 5000, 1, 514, -3]))


@pytest.mark.parametrize("softcap,bias,q_scale", [(30.0, False, 1.0), (5.0, False, 20.0),
                                                  (0.0, True, 1.0), (20.0, True, 8.0)])
@pytest.mark.parametrize("d", [64, 128])
def test_capped_scores_and_bias(softcap, bias, q_scale, d):
    _check(ref.make_chunk(6, MIXED, 8, 2, d, 16, "bf16", softcap=softcap, bias=bias,
                          q_scale=q_scale))


def test_everything_at_once():
    _check(ref.make_chunk(7, MIXED, 8, 2, 128, 16, "fp16", "hnd", window=77, softcap=25.0,
                          bias=True, prefix=[100, 290, 60, 0, 400, 9]))


def test_slopes_of_either_sign_and_a_scale_of_either_sign():
    c = ref.make_chunk(8, MIXED, 4, 1, 64, 16, "bf16", bias=True)
    c["slopes"] = torch.tensor([0.5, -0.01, 0.0, -0.5])
    _check(c)
    for scale in (-0.2, 0.0):
        c = ref.make_chunk(9, SHORT, 4, 1, 64, 16, "bf16")
        c["scale"] = scale
        _check(c)


def test_scores_that_differ_by_far():
    """Weights that underflow, and a maximum that moves up at every page."""
    c = ref.make_chunk(10, MIXED, 4, 1, 128, 16, "bf16", q_scale=30.0)
    _check(c)
    c = ref.make_chunk(11, [(600, 3)], 4, 4, 64, 16, "fp16")
    for j in range(38):
        c["k"][c["tables"][0, j].long()] *= 1 + 0.25 * j
    _check(c)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("seqs", [[(300, 130), (40, 9), (200, 1)], [(700, 600)]])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(d, value, seqs):
    c = ref.make_chunk(12, seqs, 4, 2, d, 16, "bf16", window=100)
    for s, (n, t) in enumerate(seqs):
        for p in (n - 1, n - max(1, t // 2)):
            blk, off = int(c["tables"][s, p // 16]), p % 16
            c["v"][blk, off, 0, 3] = value
        p = n - t - 100  # before every window
        if p >= 0:
            c["v"][int(c["tables"][s, p // 16]), p % 16] = value
            c["k"][int(c["tables"][s, p // 16]), p % 16] = value
    _check(c)


def test_keys_that_are_not_finite_reach_only_the_rows_that_see_them():
    c = ref.make_chunk(13, [(150, 140)], 2, 1, 64, 16, "bf16")
    out, bound = ref.attention(c)
    blk = int(c["tables"][0, 120 // 16])
    c["k"][blk, 120 % 16] = math.nan
    g = ref.on_gpu(c)
    got = _call(g).cpu()
    ref.assert_close(got[:110], out[:110], bound[:110])
    assert torch.isnan(got[110:140]).all()


def test_pages_that_are_not_there():
    c = ref.make_chunk(14, [(300, 130), (90, 2)], 4, 2, 64, 16, "bf16")
    gone = int(c["tables"][0, 5])
    expect = ref.attention(c, skip_blocks=(gone,))
    for bad in (-1, c["k"].shape[0], 2 ** 31 - 1):
        c["tables"][0, 5] = bad
        _check(c, flags=pkv.EFLAG_BLOCK_ID, expect=expect)


def test_contexts_out_of_range():
    c = ref.make_chunk(15, [(40, 3), (60, 4), (20, 2)], 4, 2, 64, 16, "bf16")
    out, bound = ref.attention(c)
    c["lens"] = torch.tensor([40, -5, 10 ** 6], dtype=torch.int32)
    c["tables"][2] = c["tables"][0]
    g = ref.on_gpu(c)
    flag = pkv.new_error_flag("cuda")
    got = _call(g, err_flag=flag).cpu()
    assert pkv.check_error(flag) & pkv.EFLAG_CONTEXT_LEN
    ref.assert_close(got[:3], out[:3], bound[:3])
    assert (got[3:7] == 0).all()
    # a context shorter than the chunk: its first rows have no position
    c = ref.make_chunk(16, [(5, 5)], 4, 2, 64, 16, "bf16")
    out, bound = ref.attention(c)
    c["starts"] = torch.tensor([0, 8], dtype=torch.int32)
    c["q"] = torch.cat([c["q"][:3], c["q"][:5]])
    g = ref.on_gpu(c)
    flag = pkv.new_error_flag("cuda")
    got = _call(g, err_flag=flag).cpu()
    assert pkv.check_error(flag) == pkv.EFLAG_CONTEXT_LEN
    assert (got[:3] == 0).all()
    ref.assert_close(got[3:], out[:5], bound[:5])


@pytest.mark.parametrize("starts", [[0, 5, 3, 9], [-2, 3, 3, 9], [0, 5, 9, 500], [20, 10, 0, 9]])
def test_starts_out_of_range_are_flagged(starts):
    c = ref.on_gpu(ref.make_chunk(17, [(40, 3), (60, 3), (20, 3)], 4, 2, 64, 16, "bf16"))
    c["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    flag = pkv.new_error_flag("cuda")
    got = _call(c, out=torch.zeros_like(c["q"]), err_flag=flag)
    assert pkv.check_error(flag) & pkv.EFLAG_QUERY
    assert torch.isfinite(got).all()


def test_in_place_and_the_same_bits_each_time():
    c = ref.make_chunk(18, MIXED, 8, 2, 128, 16, "bf16")
    g = ref.on_gpu(c)
    first = _call(g, out=torch.zeros_like(g["q"]))
    for _ in range(3):
        assert torch.equal(_call(g, out=torch.zeros_like(g["q"])), first)
    end = int(c["starts"][-1])
    same = _call(g, out=g["q"])
    assert same is g["q"] and torch.equal(same[:end], first[:end])


def test_a_sequence_gives_the_same_alone_as_in_a_batch_within_rounding():
    c = ref.make_chunk(19, MIXED, 8, 2, 128, 16, "bf16")
    out, bound = ref.attention(c)
    for s in range(len(MIXED)):
        one = dict(c, starts=c["starts"][s:s + 2], lens=c["lens"][s:s + 1],
                   tables=c["tables"][s:s + 1])
        lo, hi = int(c["starts"][s]), int(c["starts"][s + 1])
        got = _call(ref.on_gpu(one)).cpu()
        ref.assert_close(got[lo:hi], out[lo:hi], bound[lo:hi])


def test_many_sequences():
    seqs = [(1 + (37 * i) % 90, 1 + (5 * i) % 3 if (37 * i) % 90 > 3 else 1) for i in range(300)]
    _check(ref.make_chunk(20, seqs, 2, 1, 64, 16, "fp16"))


def test_other_streams_and_captured_graphs_that_share_a_workspace():
    a = ref.make_chunk(21, MIXED, 8, 2, 64, 16, "bf16")
    b = ref.make_chunk(22, LONG, 8, 2, 64, 16, "bf16")
    expect = [ref.attention(a), ref.attention(b)]
    ga, gb = ref.on_gpu(a), ref.on_gpu(b)
    need = max(pkv.chunk_attention_workspace_size(len(c["lens"]), c["q"].shape[0], 8, 2, 64, 16,
                                                  c["max_len"]) for c in (a, b))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros_like(ga["q"]), torch.zeros_like(gb["q"])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _call(ga, out=outs[0], stream=side)
    side.synchronize()
    ref.assert_close(outs[0], *expect[0])
    graphs = []
    for c, o in ((ga, outs[0]), (gb, outs[1])):
        _call(c, out=o, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _call(c, out=o, workspace=ws)
        graphs.append(graph)
    for o in outs:
        o.zero_()
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for o, e in zip(outs, expect):
        ref.assert_close(o, *e)


def test_a_graph_follows_the_lengths_that_its_buffers_hold():
    """Captured for a batch's bounds, replayed with other lengths and empty places."""
    big = ref.make_chunk(23, [(400, 100), (300, 1), (200, 60)], 8, 2, 64, 16, "bf16", tail=0)
    g = ref.on_gpu(big)
    out = torch.zeros_like(g["q"])
    _call(g, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(g, out=out)
    for starts, lens in (([0, 100, 101, 161], [400, 300, 200]), ([0, 1, 1, 3], [17, 0, 33]),
                         ([0, 0, 161, 161], [0, 300, 0]), ([0, 1, 2, 3], [1, 1, 1])):
        c = dict(big, starts=torch.tensor(starts, dtype=torch.int32),
                 lens=torch.tensor(lens, dtype=torch.int32))
        g["starts"].copy_(c["starts"])
        g["lens"].copy_(c["lens"])
        out.fill_(3.0)
        before = out.clone()
        graph.replay()
        torch.cuda.synchronize()
        ref.assert_close(out, *ref.attention(c), before)


def test_scores_that_jump_within_a_tile():
    """A largest score in either half of a tile, far above what the row had before."""
    for dtype, jump in (("fp16", 3.0), ("bf16", 3.0), ("bf16", 40.0)):
        for at in (5, 70, 130, 200, 300):
            c = ref.make_chunk(24, [(400, 130), (400, 1)], 4, 1, 64, 16, dtype)
            for s in range(2):
                c["k"][int(c["tables"][s, at // 16]), at % 16] *= jump
            _check(c)


@pytest.mark.parametrize("softcap,bias", [(20.0, False), (0.0, True), (15.0, True)])
def test_masked_keys_that_are_not_finite_beside_seen_ones(softcap, bias):
    """NaN at every other position from the first one that no row sees on, and before windows."""
    c = ref.make_chunk(25, [(151, 20), (77, 1)], 4, 1, 64, 16, "bf16", window=33, softcap=softcap,
                       bias=bias)
    for s, (n, t) in enumerate(((151, 20), (77, 1))):
        for p in range(n - t - 33, -1, -2):
            c["k"][int(c["tables"][s, p // 16]), p % 16] = math.nan
            c["v"][int(c["tables"][s, p // 16]), p % 16] = math.inf
    _check(c)


def test_a_nan_key_makes_every_row_that_sees_it_nan_under_a_cap():
    c = ref.make_chunk(26, [(150, 140)], 2, 1, 64, 16, "bf16", softcap=10.0)
    out, bound = ref.attention(c)
    c["k"][int(c["tables"][0, 120 // 16]), 120 % 16] = math.nan
    got = _call(ref.on_gpu(c)).cpu()
    ref.assert_close(got[:110], out[:110], bound[:110])
    assert torch.isnan(got[110:140]).all()
