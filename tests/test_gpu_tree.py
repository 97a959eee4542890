"""Tree plan, tree attention and tree commit on the GPU vs plain 64-bit references."""
import pytest
import torch

import paged_kv_cache_164_gb300 as pkv
import tree_reference as ref

pytestmark = pytest.mark.gpu


def _same_bits(a, b):
    return torch.equal(a.cpu().view(torch.int16), b.cpu().view(torch.int16))


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("t,lens,bs", [
    (1, [1], 16), (1, [17, 40], 16), (7, [7, 23, 64], 16), (32, [33, 32, 100], 32),
    (33, [500, 33, 0, 47], 64), (250, [250, 1000, 700], 128), (1024, [1024, 3000], 16),
])
def test_plan_matches_the_definition(t, lens, bs):
    c = ref.make_case(t * 3 + bs, lens, t, 2, 1, 64, bs, "fp16")
    parents = c["parents"].clone()
    for s in range(len(lens)):  # ragged: the last nodes of every other tree are not there
        if s % 2:
            parents[s, max(1, t - s - 1):] = ref.ABSENT
    nb = c["k"].shape[0]
    bits, positions, slots, flags = ref.plan(parents, c["lens"], c["tables"], bs, c["max_len"], nb)
    assert flags == 0
    flag = pkv.new_error_flag("cuda")
    mask, pos, slot = pkv.tree_plan(parents.cuda(), c["lens"].cuda(), c["tables"].cuda(), nb, bs,
                                    c["max_len"], err_flag=flag)
    assert pkv.check_error(flag) == 0
    assert torch.equal(mask.cpu(), ref.pack(bits))
    assert torch.equal(pos.cpu(), positions) and torch.equal(slot.cpu(), slots)


def test_plan_of_a_chain_and_a_star():
    t = 40
    chain = torch.arange(-1, t - 1, dtype=torch.int32)
    star = torch.zeros(t, dtype=torch.int32)
    star[0] = -1
    parents = torch.stack([chain, star, torch.full((t,), -1, dtype=torch.int32)])
    lens = torch.tensor([t + 5, t, t + 100], dtype=torch.int32)
    tables = torch.arange(3 * 16, dtype=torch.int32).view(3, 16)
    bits, positions, slots, _ = ref.plan(parents, lens, tables, 16, 256, 48)
    mask, pos, slot = pkv.tree_plan(parents.cuda(), lens.cuda(), tables.cuda(), 48, 16, 256)
    assert torch.equal(mask.cpu(), ref.pack(bits))
    assert torch.equal(pos.cpu(), positions) and torch.equal(slot.cpu(), slots)
    assert bits[0].sum() == t * (t + 1) // 2 and bits[1].sum() == 2 * t - 1 and bits[2].sum() == t


def test_plan_of_more_sequences_than_a_grid_dimension_of_65535():
    b, t = 66001, 2
    parents = torch.tensor([[-1, 0]], dtype=torch.int32).repeat(b, 1)
    parents[-1, 1] = -1
    tables = torch.arange(b, dtype=torch.int32)[:, None].contiguous()
    lens = torch.full((b,), 5, dtype=torch.int32)
    mask, pos, slot = pkv.tree_plan(parents.cuda(), lens.cuda(), tables.cuda(), b, 16, 16)
    assert mask[:-1, 0, 0].eq(1).all() and mask[:-1, 1, 0].eq(3).all()
    assert mask[-1, :, 0].tolist() == [1, 2] and pos[-1].tolist() == [3, 3]
    assert pos[:-1].eq(torch.tensor([3, 4], device="cuda")).all()
    want = torch.arange(b)[:, None] * 16 + torch.tensor([3, 4])
    assert torch.equal(slot.cpu(), want)


@pytest.mark.parametrize("t", [31, 64, 100, 257, 513, 1000])
def test_plan_of_random_chains_with_unsound_links(t):
    """Links to the parent just before, to nodes far before, to nothing, to the node itself,
    behind it and out of range."""
    gen = torch.Generator().manual_seed(t)
    b = 9
    i = torch.arange(t)
    parents = torch.empty(b, t, dtype=torch.int32)
    for s in range(b):
        near = i - 1 - (torch.rand(t, generator=gen) * (1, 3, 40)[s % 3]).to(torch.int64)
        far = (torch.rand(t, generator=gen) * i).to(torch.int64)
        parents[s] = torch.where(torch.rand(t, generator=gen) < 0.1, far, near).clamp(min=-1)
    odd = torch.rand(b, t, generator=gen) < torch.linspace(0, 0.02, b)[:, None]
    kind = torch.randint(0, 6, (b, t), generator=gen)
    bad = torch.stack([i, i + 1, torch.full((t,), 2 ** 31 - 1), torch.full((t,), -3),
                       torch.full((t,), ref.ABSENT), torch.full((t,), -2 ** 31)])
    parents = torch.where(odd, bad[kind, i.expand(b, t)], parents.long()).to(torch.int32)
    lens = torch.randint(t, t + 200, (b,), generator=gen, dtype=torch.int32)
    width = (t + 200 + 15) // 16
    tables = torch.randperm(b * width, generator=gen).to(torch.int32).view(b, width)
    bits, positions, slots, flags = ref.plan(parents, lens, tables, 16, t + 200, b * width)
    flag = pkv.new_error_flag("cuda")
    mask, pos, slot = pkv.tree_plan(parents.cuda(), lens.cuda(), tables.cuda(), b * width, 16,
                                    t + 200, err_flag=flag)
    torch.cuda.synchronize()
    assert int(flag.item()) == flags
    assert torch.equal(mask.cpu(), ref.pack(bits))
    assert torch.equal(pos.cpu(), positions) and torch.equal(slot.cpu(), slots)


@pytest.mark.parametrize("what", ["forward", "self", "below", "orphan", "block", "short", "long",
                                  "negative"])
def test_plan_flags_and_leaves_out_what_is_malformed(what):
    t, bs = 12, 16
    c = ref.make_case(5, [30, 50], t, 2, 1, 64, bs, "fp16")
    parents, lens, tables = c["parents"].clone(), c["lens"].clone(), c["tables"].clone()
    nb, want = c["k"].shape[0], pkv.EFLAG_TREE
    if what == "forward":
        parents[0, 3] = 7
    elif what == "self":
        parents[0, 4] = 4
    elif what == "below":
        parents[0, 2] = -3
    elif what == "orphan":
        parents[0, 5], parents[0, 6] = ref.ABSENT, 5
    elif what == "block":
        tables[1, (50 - t) // bs] = nb
        want = pkv.EFLAG_BLOCK_ID
    else:
        lens[0] = {"short": t - 1, "long": 51, "negative": -4}[what]
        want = pkv.EFLAG_CONTEXT_LEN
    bits, positions, slots, flags = ref.plan(parents, lens, tables, bs, 50, nb)
    assert flags == want
    flag = pkv.new_error_flag("cuda")
    mask, pos, slot = pkv.tree_plan(parents.cuda(), lens.cuda(), tables.cuda(), nb, bs, 50,
                                    err_flag=flag)
    assert pkv.check_error(flag) == want
    assert torch.equal(mask.cpu(), ref.pack(bits))
    assert torch.equal(pos.cpu(), positions) and torch.equal(slot.cpu(), slots)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

ATTENTION = {
    "tiny_gqa2_d64_fp16": dict(lens=[38, 51], t=4, h_q=4, h_kv=2, d=64, bs=16, dtype="fp16"),
    "one_token": dict(lens=[1, 2, 129, 300], t=1, h_q=2, h_kv=2, d=128, bs=16, dtype="bf16"),
    "nothing_committed": dict(lens=[9, 9], t=9, h_q=6, h_kv=2, d=64, bs=16, dtype="fp16"),
    "nothing_committed_rows_of_none": dict(lens=[40, 40], t=40, h_q=4, h_kv=1, d=128, bs=16,
                                           dtype="bf16", mask="random"),
    "two_mask_words_hnd_bs32": dict(lens=[33, 161, 700], t=33, h_q=16, h_kv=2, d=128, bs=32,
                                    dtype="bf16", layout="hnd"),
    "tile_edges": dict(lens=[64 + x for x in (63, 64, 65, 127, 128, 129, 255, 256, 257)], t=64,
                       h_q=4, h_kv=1, d=128, bs=16, dtype="bf16"),
    "tile_edges_random_bits_d64": dict(lens=[20 + x for x in (107, 108, 109, 236, 500)], t=20,
                                       h_q=3, h_kv=3, d=64, bs=64, dtype="fp16", mask="random"),
    "rows_300": dict(lens=[100, 230, 801], t=100, h_q=6, h_kv=2, d=128, bs=16, dtype="fp16"),
    "group16_rows_144": dict(lens=[30, 555], t=9, h_q=32, h_kv=2, d=128, bs=128, dtype="bf16",
                             layout="hnd"),
    "long_tree": dict(lens=[300, 421], t=300, h_q=1, h_kv=1, d=64, bs=16, dtype="bf16"),
    "rows_1024_and_more": dict(lens=[170, 300], t=150, h_q=8, h_kv=1, d=64, bs=32, dtype="fp16",
                               mask="random"),
    "full_mask": dict(lens=[70, 333], t=17, h_q=8, h_kv=2, d=128, bs=16, dtype="bf16",
                      mask="full"),
    "group5": dict(lens=[19, 77, 410], t=13, h_q=10, h_kv=2, d=128, bs=16, dtype="bf16"),
    "empty_places": dict(lens=[0, 90, 0, 0, 260, 0], t=11, h_q=4, h_kv=2, d=64, bs=16,
                         dtype="bf16"),
    "many_ragged": dict(lens=[8 + 37 * i % 900 for i in range(70)], t=8, h_q=4, h_kv=2, d=64,
                        bs=16, dtype="fp16"),
    "split_over_many": dict(lens=[20000], t=5, h_q=4, h_kv=1, d=64, bs=16, dtype="bf16"),
    "many_sequences": dict(lens=[1 + 7 * i % 40 for i in range(1400)], t=1, h_q=2, h_kv=2, d=64,
                           bs=16, dtype="bf16"),
    "peaked": dict(lens=[40, 900], t=16, h_q=8, h_kv=1, d=128, bs=16, dtype="bf16", q_scale=6.0),
}


def _run(c, **kw):
    g = ref.on_gpu(c)
    flag = pkv.new_error_flag("cuda")
    out = pkv.tree_attention(g["q"], g["k"], g["v"], g["tables"], g["lens"], c["max_len"],
                             g["mask"], scale=c["scale"], err_flag=flag, layout=c["layout"], **kw)
    return out, pkv.check_error(flag)


@pytest.mark.parametrize("key", ATTENTION)
def test_attention_matches_the_definition(key):
    c = ref.make_case(len(key), **ATTENTION[key])
    out, err = _run(c)
    assert err == 0
    ref.assert_close(out, *ref.attention(c), key)


@pytest.mark.parametrize("t,group", [(6, 2), (40, 4)])
@pytest.mark.parametrize("b", [31, 32, 33, 64])
def test_attention_of_about_a_warp_of_sequences(b, t, group):
    """Ragged, with empty places at the start, in the middle and at the end."""
    lens = [0 if i in (0, b // 2, b - 1) else t + 131 * i % 700 for i in range(b)]
    c = ref.make_case(b + t, lens, t, 2 * group, 2, 64, 16, "fp16")
    out, err = _run(c)
    assert err == 0
    ref.assert_close(out, *ref.attention(c), f"{b} sequences")


@pytest.mark.parametrize("scale", [0.0, -0.11, 2.0])
def test_attention_scales(scale):
    c = ref.make_case(3, **ATTENTION["rows_300"]) | {"scale": scale}
    out, err = _run(c)
    assert err == 0
    ref.assert_close(out, *ref.attention(c), str(scale))


def test_attention_of_ancestor_chains_is_multi_query_attention():
    c = ref.make_case(9, [400, 77], 12, 8, 2, 128, 16, "bf16")
    t = 12
    bits = torch.tril(torch.ones((t, t), dtype=torch.bool)).expand(2, t, t).clone()
    c |= dict(bits=bits, mask=ref.pack(bits))
    g = ref.on_gpu(c)
    out, err = _run(c)
    assert err == 0
    causal = pkv.multi_query_attention(g["q"], g["k"], g["v"], g["tables"], g["lens"], 400,
                                       scale=c["scale"])
    o, bound = ref.attention(c)
    ref.assert_close(out, o, bound)
    ref.assert_close(causal, o, bound)


def test_attention_with_one_mask_for_all_sequences():
    c = ref.make_case(10, [60, 300, 45], 40, 4, 2, 64, 16, "fp16")
    c["bits"] = c["bits"][:1].expand(3, 40, 40).clone()
    c["mask"] = ref.pack(c["bits"])
    g = ref.on_gpu(c)
    whole, err = _run(c)
    assert err == 0
    ref.assert_close(whole, *ref.attention(c))
    for mask in (g["mask"][:1], g["mask"][:1].expand(3, 40, 2)):
        one = pkv.tree_attention(g["q"], g["k"], g["v"], g["tables"], g["lens"], 300, mask,
                                 scale=c["scale"])
        assert _same_bits(one, whole)
    apart = torch.zeros((3, 3, 40, 2), dtype=torch.int32, device="cuda")
    apart[:, 1] = g["mask"]  # a batch stride of its own
    far = pkv.tree_attention(g["q"], g["k"], g["v"], g["tables"], g["lens"], 300, apart[:, 1],
                             scale=c["scale"])
    assert _same_bits(far, whole)


def test_attention_ignores_bits_past_the_tree():
    c = ref.make_case(11, [50, 200], 20, 4, 1, 128, 16, "bf16")
    clean, _ = _run(c)
    c["mask"] = c["mask"] | (-1 << 20)
    noisy, err = _run(c)
    assert err == 0 and _same_bits(clean, noisy)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("which", ["k", "v", "kv"])
@pytest.mark.parametrize("key", ["rows_300", "tile_edges", "tiny_gqa2_d64_fp16", "group5"])
def test_attention_rows_see_nothing_of_what_they_do_not_attend_to(key, which, value):
    c = ref.make_case(21, **ATTENTION[key])
    clean, _ = _run(c)
    t = c["q"].shape[1]
    bad = [t // 3, t - 1]  # nodes whose rows hold the value in one dim or all
    for s in range(len(c["lens"])):
        for node in bad:
            p = int(c["lens"][s]) - t + node
            blk, off = int(c["tables"][s, p // c["bs"]]), p % c["bs"]
            for x in which:
                if node == t - 1:
                    c[x][blk, off] = value
                else:
                    c[x][blk, off, :, 3] = value
    got, err = _run(c)
    assert err == 0
    hit = c["bits"][:, :, bad].any(-1)  # rows that attend to such a node
    assert hit.any() and not hit.all()
    keep = ~hit
    assert _same_bits(got.cpu()[keep], clean.cpu()[keep])
    spoilt = got.cpu()[hit].float()
    if which == "v":  # weights above zero: the value itself comes out where it is
        col = spoilt[..., 3]
        assert (col.isnan() if value != value else (col == value)).all()
    elif value != value:
        assert spoilt[..., 3].isnan().all()


def test_attention_skips_and_flags_bad_blocks():
    for case in (dict(lens=[700, 90], t=10, h_q=8, h_kv=2, d=128, bs=16, dtype="bf16"),
                 dict(lens=[300, 90], t=90, h_q=4, h_kv=1, d=64, bs=32, dtype="fp16",
                      mask="full")):
        c = ref.make_case(31, **case)
        nb = c["k"].shape[0]
        c["tables"][0, 3], c["tables"][0, 5] = nb, -7
        c["tables"][1, 2] = 2 ** 30
        got, err = _run(c)
        assert err == pkv.EFLAG_BLOCK_ID
        fixed = dict(c, tables=torch.where((c["tables"] < 0) | (c["tables"] >= nb), nb,
                                           c["tables"]))
        for n in ("k", "v"):
            fixed[n] = torch.cat([c[n], torch.zeros_like(c[n][:1])])
        ref.assert_close(got, *ref.attention(fixed, skip_blocks=(nb,)))


def test_attention_flags_lengths_out_of_range():
    c = ref.make_case(32, [200, 120, 64], 10, 4, 2, 64, 16, "fp16")
    for lens, n in (([200, 9, 64], 9), ([200, -5, 64], 0), ([200, 100000, 64], None)):
        d = dict(c, lens=torch.tensor(lens, dtype=torch.int32))
        got, err = _run(d)
        # (cut to max_context_len, the longest runs into table entries that hold no block)
        assert err == pkv.EFLAG_CONTEXT_LEN | (pkv.EFLAG_BLOCK_ID if n is None else 0)
        o, bound = ref.attention(c, seqs=[0, 2])
        keep = [0, 2]
        ref.assert_close(got[keep], o[keep], bound[keep])
        if n == 0:
            assert (got[1] == 0).all()
        if n == 9:  # the last nine nodes are there, node j at position j - 1
            rows = dict(c, lens=torch.tensor([0, 9, 0], dtype=torch.int32))
            o, bound = ref.attention(rows)
            ref.assert_close(got[1:2], o[1:2], bound[1:2])


@pytest.mark.parametrize("rows", [(8, 2), (40, 8)])
def test_attention_on_a_long_context_with_large_offsets(rows):
    # a pool whose last pages start beyond 2^31 elements
    t, grp = rows
    bs, h_kv, d = 16, 8, 128
    nb = 2 ** 31 // (bs * h_kv * d) + 40
    n = 130 + t
    g = torch.Generator(device="cuda").manual_seed(4)
    k = torch.empty((nb, bs, h_kv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    pages = (n + bs - 1) // bs
    table = torch.arange(nb - pages, nb, dtype=torch.int32, device="cuda")[None]
    for x in (k, v):
        x[nb - pages:] = torch.randn((pages, bs, h_kv, d), generator=g, device="cuda").bfloat16()
    small = ref.make_case(33, [n], t, h_kv * grp, h_kv, d, bs, "bf16")
    q = small["q"].cuda()
    out = pkv.tree_attention(q, k, v, table, small["lens"].cuda(), n, small["mask"].cuda(),
                             scale=small["scale"])
    small |= dict(k=k[nb - pages:].cpu(), v=v[nb - pages:].cpu(),
                  tables=(table - (nb - pages)).cpu())
    del k, v
    ref.assert_close(out, *ref.attention(small))


def test_attention_is_the_same_every_time():
    c = ref.make_case(34, [5000, 300, 2100], 24, 16, 2, 128, 16, "bf16")
    first, _ = _run(c)
    for _ in range(4):
        again, _ = _run(c)
        assert _same_bits(first, again)


def test_attention_workspace_contents_do_not_matter():
    c = ref.make_case(35, [3000, 450], 9, 8, 1, 128, 16, "bf16")
    first, _ = _run(c)
    need = pkv.tree_attention_workspace_size(2, 9, 8, 1, 128, 16, 3000)
    for fill in (0, 255, 0x7F):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        got, err = _run(c, workspace=ws)
        assert err == 0 and _same_bits(first, got)
    with pytest.raises(pkv.PkvError, match="WORKSPACE"):
        _run(c, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


def test_attention_on_another_stream():
    c = ref.make_case(36, [900, 450], 20, 8, 2, 64, 16, "fp16")
    g = ref.on_gpu(c)
    want, _ = _run(c)
    side = torch.cuda.Stream()
    for _ in range(5):
        q = torch.zeros_like(g["q"])
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
            q.copy_(g["q"])
        out = pkv.tree_attention(q, g["k"], g["v"], g["tables"], g["lens"], 900, g["mask"],
                                 scale=c["scale"], stream=side)
        junk = torch.full_like(want, 7.0)  # the allocator must not hand out the call's workspace
        side.synchronize()
        assert _same_bits(out, want) and (junk == 7).all()


def test_graphs_that_share_a_workspace_and_replay_on_new_inputs():
    a = ref.make_case(37, [700, 310], 16, 8, 2, 128, 16, "bf16")
    b = ref.make_case(38, [333, 640], 16, 8, 2, 128, 16, "bf16", spare_pages=10)
    ws = torch.empty(pkv.tree_attention_workspace_size(2, 16, 8, 2, 128, 16, 700),
                     dtype=torch.uint8, device="cuda")
    calls = []
    for c in (a, b):
        g = ref.on_gpu(c)
        out = torch.zeros_like(g["q"])
        args = (g["q"], g["k"], g["v"], g["tables"], g["lens"], 700, g["mask"])
        pkv.tree_attention(*args, scale=c["scale"], out=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pkv.tree_attention(*args, scale=c["scale"], out=out, workspace=ws)
        calls.append((c, g, out, graph))
    want = [ref.attention(c) for c in (a, b)]
    for order in ((0, 1), (1, 0), (0, 0)):
        for i in order:
            calls[i][2].zero_()
            calls[i][3].replay()
        torch.cuda.synchronize()
        for i in set(order):
            ref.assert_close(calls[i][2], *want[i])
    # other lengths and trees in the captured tensors
    c, g, out, graph = calls[0]
    new = ref.make_case(39, [700, 310], 16, 8, 2, 128, 16, "bf16", mask="random")
    new["lens"] = torch.tensor([250, 0], dtype=torch.int32)
    new["tables"], new["k"], new["v"] = c["tables"], c["k"], c["v"]
    for n in ("q", "lens", "mask"):
        g[n].copy_(new[n])
    graph.replay()
    ref.assert_close(out, *ref.attention(new))


# ---------------------------------------------------------------------------
# commit
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,layout,d", [("fp16", "nhd", 128), ("bf16", "hnd", 64)])
@pytest.mark.parametrize("t,paths", [
    (1, [[0], [], [0]]),
    (16, [[0, 1, 5, 15], [3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15], list(range(16))]),
    (60, [[59], [0] + list(range(20, 60)), [1, 2, 3, 58, 59]]),
])
def test_commit_moves_the_accepted_rows(t, paths, dtype, layout, d):
    lens = [t, t + 29, t + 200]
    c = ref.make_case(t + d, lens, t, 4, 2, d, 16, dtype, layout=layout)
    most = max(1, max(len(p) for p in paths))
    accepted = torch.tensor([p + [-9] * (most - len(p)) for p in paths], dtype=torch.int32)
    counts = torch.tensor([len(p) for p in paths], dtype=torch.int32)
    k, v, new = ref.commit(c, t, accepted, counts)
    g = ref.on_gpu(c)
    flag = pkv.new_error_flag("cuda")
    got = pkv.tree_commit(g["k"], g["v"], g["tables"], g["lens"], t, accepted.cuda(),
                          counts.cuda(), err_flag=flag, layout=layout)
    assert pkv.check_error(flag) == 0
    assert torch.equal(got.cpu(), new)
    for name, want in (("k", k), ("v", v)):
        have = g[name].transpose(1, 2).contiguous() if layout == "hnd" else g[name]
        assert _same_bits(have, want)


@pytest.mark.parametrize("what", ["order", "twice", "beyond", "count", "negative_count", "block",
                                  "short", "long"])
def test_commit_flags_and_moves_nothing_of_a_malformed_path(what):
    t, bs = 24, 16
    c = ref.make_case(41, [60, 100, 80], t, 4, 2, 64, bs, "fp16")
    accepted = torch.tensor([[0, 2, 9, 20], [0, 5, 8, 22], [1, 3, 10, 23]], dtype=torch.int32)
    counts = torch.tensor([4, 4, 3], dtype=torch.int32)
    lens, tables = c["lens"].clone(), c["tables"].clone()
    want, new1 = pkv.EFLAG_TREE, 100 - t
    if what == "order":
        accepted[1, 2] = 4
    elif what == "twice":
        accepted[1, 2] = 5
    elif what == "beyond":
        accepted[1, 3] = t
    elif what == "count":
        counts[1] = 5
    elif what == "negative_count":
        counts[1] = -1
    elif what == "block":
        tables[1, (100 - t + 22) // bs] = c["k"].shape[0]
        want = pkv.EFLAG_BLOCK_ID
    else:
        lens[1] = t - 1 if what == "short" else 16 * tables.shape[1] + 1
        want = pkv.EFLAG_CONTEXT_LEN
        new1 = 0 if what == "short" else 16 * tables.shape[1] - t
    good = dict(c, lens=torch.tensor([60, 0, 80], dtype=torch.int32))
    k, v, new = ref.commit(good, t, accepted, counts)
    new[1] = new1
    g = ref.on_gpu(c)
    flag = pkv.new_error_flag("cuda")
    got = pkv.tree_commit(g["k"], g["v"], tables.cuda(), lens.cuda(), t, accepted.cuda(),
                          counts.cuda(), err_flag=flag)
    assert pkv.check_error(flag) == want
    assert torch.equal(got.cpu(), new)
    assert _same_bits(g["k"], k) and _same_bits(g["v"], v)


def test_plan_and_commit_on_another_stream():
    t = 16
    c = ref.make_case(61, [40, 200], t, 4, 2, 64, 16, "bf16")
    accepted = torch.tensor([[0, 3, 15], [2, 3, 9]], dtype=torch.int32)
    counts = torch.tensor([3, 2], dtype=torch.int32)
    nb = c["k"].shape[0]
    bits, positions, slots, _ = ref.plan(c["parents"], c["lens"], c["tables"], 16, 200, nb)
    k, v, new = ref.commit(c, t, accepted, counts)
    g = ref.on_gpu(c)
    acc, cnt = accepted.cuda(), counts.cuda()
    lens = torch.zeros_like(g["lens"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        lens.copy_(g["lens"])
    mask, pos, slot = pkv.tree_plan(g["parents"], lens, g["tables"], nb, 16, 200, stream=side)
    got = pkv.tree_commit(g["k"], g["v"], g["tables"], lens, t, acc, cnt, stream=side)
    junk = [torch.full_like(x, 7) for x in (mask, pos, slot, got)]  # not the calls' outputs
    side.synchronize()
    assert torch.equal(mask.cpu(), ref.pack(bits)) and torch.equal(pos.cpu(), positions)
    assert torch.equal(slot.cpu(), slots) and torch.equal(got.cpu(), new)
    assert _same_bits(g["k"], k) and _same_bits(g["v"], v) and all((x == 7).all() for x in junk)


# ---------------------------------------------------------------------------
# a step
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_a_whole_step_captured_and_followed_by_a_decode(layout):
    """plan -> norm + rotation + append -> attention -> commit -> decode, in one
    graph, replayed over the state that it leaves."""
    t, h_q, h_kv, d, bs, cap = 10, 8, 2, 64, 16, 160
    start, accept = [41, 100], [4, 1]
    c = ref.make_case(51, [cap, cap], t, h_q, h_kv, d, bs, "bf16", layout=layout)
    gen = torch.Generator().manual_seed(52)
    x = torch.randn((2 * t, h_q + 2 * h_kv, d), generator=gen).bfloat16()
    wq, wk = (1 + 0.1 * torch.randn((2, d), generator=gen)).bfloat16()
    angle = torch.arange(cap).double()[:, None] * 100.0 ** (-torch.arange(0, d, 2).double() / d)
    table = torch.cat([angle.cos(), angle.sin()], 1).float()
    parents = torch.tensor([ref.random_parents(t, gen) for _ in range(2)], dtype=torch.int32)
    parents[1, 7:] = ref.ABSENT
    paths = []
    for s in range(2):  # the last node of a chain of `accept` nodes
        best = [0]
        for i in range(t):
            chain, up = [i], i
            while parents[s, up] >= 0:
                up = int(parents[s, up])
                chain.append(up)
            if parents[s, i] != ref.ABSENT and len(chain) <= accept[s] and \
                    len(chain) > len(best):
                best = chain[::-1]
        paths.append(best)
    counts = [len(p) for p in paths]
    accepted = torch.tensor([p + [0] * (4 - len(p)) for p in paths], dtype=torch.int32)

    g = ref.on_gpu(c)
    lens = torch.tensor([n + t for n in start], dtype=torch.int32, device="cuda")
    xs, tab, par = x.cuda(), table.cuda(), parents.cuda()
    acc, cnt = accepted.cuda(), torch.tensor(counts, dtype=torch.int32, device="cuda")
    q_w, k_w = wq.cuda(), wk.cuda()
    nb = c["k"].shape[0]
    flag = pkv.new_error_flag("cuda")
    ws = torch.empty(pkv.tree_attention_workspace_size(2, t, h_q, h_kv, d, bs, cap),
                     dtype=torch.uint8, device="cuda")
    out = {}

    def step():
        mask, pos, slots = pkv.tree_plan(par, lens, g["tables"], nb, bs, cap, err_flag=flag)
        q = pkv.norm_rope_append(xs[:, :h_q], xs[:, h_q:h_q + h_kv], xs[:, h_q + h_kv:],
                                 pos.view(-1), tab, g["k"], g["v"], slots.view(-1),
                                 q_weight=q_w, k_weight=k_w, eps=1e-5, q_out=out.get("q"),
                                 err_flag=flag, layout=layout)
        o = pkv.tree_attention(q.view(2, t, h_q, d), g["k"], g["v"], g["tables"], lens, cap, mask,
                               workspace=ws, err_flag=flag, layout=layout)
        new = pkv.tree_commit(g["k"], g["v"], g["tables"], lens, t, acc, cnt, err_flag=flag,
                              layout=layout)
        dec = pkv.decode_attention(q.view(2, t, h_q, d)[:, 0].contiguous(), g["k"], g["v"],
                                   g["tables"], new, cap, num_splits=1, err_flag=flag,
                                   layout=layout)
        lens.copy_(new + t)
        return o, new, dec, q

    def expect(state):
        base = [int(n) - t for n in state["lens"]]
        bits, pos, slots, flags = ref.plan(parents, state["lens"], c["tables"], bs, cap, nb)
        assert flags == 0
        yq, yk, yv, _, _ = ref.norm_rope(x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:],
                                         pos.view(-1), table, wq, wk, 1e-5, "half")
        for i, s in enumerate(slots.view(-1).tolist()):
            if s >= 0:
                state["k"][s // bs, s % bs] = yk[i].bfloat16()
                state["v"][s // bs, s % bs] = yv[i].bfloat16()
        state |= dict(q=yq.bfloat16().view(2, t, h_q, d), bits=bits)
        o, bound = ref.attention(state)
        state["k"], state["v"], new = ref.commit(state, t, accepted, counts)
        assert new.tolist() == [b + n for b, n in zip(base, counts)]
        one = dict(state, q=state["q"][:, :1], lens=new,
                   bits=torch.ones((2, 1, 1), dtype=torch.bool))
        do, dbound = ref.attention(one)
        state["lens"] = new + t
        return o, bound, new, do, dbound, slots.view(2, t) >= 0

    state = dict(c, k=c["k"].clone(), v=c["v"].clone(), lens=lens.cpu())
    # absent nodes' rows of q are left as they were: give them something finite
    out["q"] = torch.zeros((2 * t, h_q, d), dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    expect(state)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, new, dec, q = step()
    for _ in range(3):
        graph.replay()
        assert pkv.check_error(flag) == 0
        eo, bound, enew, edo, edb, there = expect(state)
        assert torch.equal(new.cpu(), enew)
        # q and k themselves may differ from the reference's by a rounding to
        # bf16 here and there; scores of |q||k| sum them up: a few 2^-8 steps
        slack = 6 * 2.0 ** -8
        d1 = (o.cpu().double() - eo).abs()[there]
        assert (d1 <= bound[there] + slack).all(), d1.max()
        d2 = (dec.cpu().double() - edo[:, 0]).abs()
        assert (d2 <= edb[:, 0] + slack).all(), d2.max()
