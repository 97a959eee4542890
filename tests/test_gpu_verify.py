"""Verification of drafted tokens against the definition in exact fractions (GPU)."""
import math

import pytest
import torch

import paged_kv_cache_164_gb300 as pkv
import ragged_reference as ref

pytestmark = pytest.mark.gpu


def _case(seed, counts, vocab, tree=False, draft=True, noise=0.7, sharp=2.0):
    g = torch.Generator().manual_seed(seed)
    starts = [0]
    for n in counts:
        starts.append(starts[-1] + n)
    rows = starts[-1]
    logits = torch.randn((rows, vocab), generator=g) * sharp
    p = torch.softmax(logits, -1)
    q = torch.softmax(logits + noise * torch.randn((rows, vocab), generator=g), -1)
    parents, tokens = [], []
    for s, n in enumerate(counts):
        for i in range(n):
            lo = max(0, i - 3)
            par = -1 if i == 0 else int(torch.randint(lo, i, (1,), generator=g)) if tree else i - 1
            parents.append(par)
            dist = q[starts[s] + max(0, par)]
            tokens.append(int(torch.multinomial(dist, 1, generator=g)))
    return dict(p=p, q=q if draft else None, tokens=torch.tensor(tokens, dtype=torch.int32),
                starts=torch.tensor(starts, dtype=torch.int32),
                u=torch.rand(rows, generator=g), most=max([1] + list(counts)),
                parents=torch.tensor(parents, dtype=torch.int32) if tree else None,
                context=torch.tensor([50 + n for n in counts], dtype=torch.int32))


def _call(c, **kw):
    g = {n: x.cuda() if isinstance(x, torch.Tensor) else x for n, x in c.items()}
    return pkv.verify_drafts(g["p"], g["q"], g["tokens"], g["starts"], g["u"], g["most"],
                             parents=g["parents"], context_lens=g["context"], **kw)


def _check(c):
    expect = ref.verify(c["p"], c["q"], c["tokens"], c["starts"], c["u"], c["most"], c["parents"],
                        c["context"])
    flag = pkv.new_error_flag("cuda")
    got = _call(c, err_flag=flag)
    names = ("accepted", "accepted_lens", "next_tokens", "new_context_lens")
    for n, t in zip(names, got):
        assert t.tolist() == expect[n], n
    assert pkv.check_error(flag) == expect["flags"]
    return expect


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("vocab", [1, 2, 31, 100, 1001])
def test_chains_and_trees(vocab, tree, draft):
    lens = []
    for seed in range(3):
        c = _case(seed, [5, 1, 9, 0, 3, 12, 2, 7], vocab, tree, draft)
        lens += _check(c)["accepted_lens"]
    assert not draft or vocab < 100 or (min(x for x in lens if x) == 1 and max(lens) > 2)


@pytest.mark.parametrize("vocab", [4096, 33000, 50001])
def test_large_vocabularies(vocab):
    _check(_case(11, [4, 6], vocab, True, sharp=1.0))


@pytest.mark.parametrize("vocab,draft", [(140001, True), (200000, True), (140001, False)])
def test_vocabularies_beyond_what_a_cluster_holds_in_registers(vocab, draft):
    c = _case(15, [3], vocab, True, draft, sharp=1.0)
    c["parents"] = torch.tensor([-1, 0, 0], dtype=torch.int32)
    for u in (0.02, 0.97):
        c["u"] = torch.tensor([u, 0.9999, 0.9999])
        _check(c)


@pytest.mark.parametrize("batch", [1, 2, 5, 19, 40, 90, 200])
def test_batches_that_take_clusters_of_every_size(batch):
    _check(_case(16, [4] * batch, 2056, True))


def test_flat_distributions_at_many_borders():
    """Tokens of probability 1 / V each: a sum in 32 bits would miss its neighbour."""
    n, v = 200, 3000
    g = torch.Generator().manual_seed(4)
    c = _case(5, [1] * n, v)
    c["p"] = (1 + 1e-3 * torch.rand((n, v), generator=g)) / v
    c["u"] = torch.rand(n, generator=g)
    _check(c)


def test_a_star_whose_children_are_all_rejected_but_one():
    c = _case(6, [40], 64, True, noise=3.0)
    c["parents"] = torch.tensor([-1] + [0] * 39, dtype=torch.int32)
    c["u"][1:] = 0.999
    _check(c)
    c["q"] = None
    c["tokens"][1:] = torch.arange(39, dtype=torch.int32) // 2  # (each twice)
    _check(c)


def test_random_numbers_at_their_borders_and_outside():
    for u in (0.0, 1 - 2.0 ** -24, 1.0, 7.0, -1.0, math.nan):
        c = _case(7, [4, 1, 6], 50)
        c["u"][:] = u
        _check(c)


def test_rests_of_nothing_and_rows_of_nothing():
    c = _case(8, [3, 2], 40)
    c["q"] = c["p"].clone()
    c["q"][0] = 1.0  # more than p everywhere: nothing is left, p itself is drawn from
    c["u"][1] = 0.9
    _check(c)
    c["p"][3] = 0.0
    c["q"][3] = 0.5
    assert _check(c)["next_tokens"][1] == -1
    c["p"][3, 7] = math.nan
    c["p"][3, 9] = -0.5
    _check(c)
    c["p"][3, 30] = 2.0  # taken as 1
    _check(c)


def test_bad_parents_tokens_and_rows():
    c = _case(9, [6, 4, 5], 40, True)
    c["parents"][2], c["parents"][3], c["parents"][8] = 5, -7, pkv.TREE_ABSENT
    _check(c)
    c["tokens"][4], c["tokens"][12] = -1, 40
    _check(c)
    for starts in ([0, 6, 4, 15], [0, 6, 10, 16], [-1, 6, 10, 15], [0, 2 ** 31 - 1, 10, 15]):
        d = dict(c, starts=torch.tensor(starts, dtype=torch.int32))
        _check(d)


def test_fewer_places_than_nodes():
    for most in (1, 2):
        c = _case(10, [6, 3], 30)
        c["q"] = c["p"].clone()  # every draft is accepted
        c["most"] = most
        assert _check(c)["accepted_lens"] == [most, most]


def test_the_longest_chain_and_one_beyond_it():
    for n, flags in ((1024, 0), (1025, pkv.EFLAG_QUERY)):
        c = _case(12, [n, 2], 5)
        c["q"] = c["p"].clone()
        c["p"][:-2] = c["p"][0]
        c["q"][:-2] = c["p"][0]
        assert _check(c)["flags"] == flags


def test_without_lengths_on_another_stream_and_captured():
    c = _case(13, [5, 3, 8], 500, True)
    g = {n: x.cuda() if isinstance(x, torch.Tensor) else x for n, x in c.items()}
    args = (g["p"], g["q"], g["tokens"], g["starts"], g["u"], g["most"])
    plain = pkv.verify_drafts(*args, parents=g["parents"])
    assert plain[3] is None
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = pkv.verify_drafts(*args, parents=g["parents"], stream=side)
    side.synchronize()
    outs = dict(accepted=torch.zeros_like(plain[0]), accepted_lens=torch.zeros_like(plain[1]),
                next_tokens=torch.zeros_like(plain[2]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.verify_drafts(*args, parents=g["parents"], **outs)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, d in zip(plain[:3], other[:3], outs.values()):
        assert torch.equal(a, b) and torch.equal(a, d)


def test_lengths_in_place():
    c = _case(14, [5, 3, 8], 300)
    expect = _call(c)[3]
    lens = c["context"].cuda()
    got = pkv.verify_drafts(c["p"].cuda(), c["q"].cuda(), c["tokens"].cuda(), c["starts"].cuda(),
                            c["u"].cuda(), c["most"], context_lens=lens, new_context_lens=lens)
    assert got[3] is lens and torch.equal(lens, expect)
