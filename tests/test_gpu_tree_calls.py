"""Calls of the tree step that are easily made and were once answered wrongly or refused (GPU)."""
import pytest
import torch

import paged_kv_cache_164_gb300 as pkv
import tree_reference as ref

pytestmark = pytest.mark.gpu


def _same_bits(a, b):
    return torch.equal(a.cpu().view(torch.int16), b.cpu().view(torch.int16))


def _commit_case(t, lens, paths, seed=5, bs=16, dtype="bf16", **kw):
    c = ref.make_case(seed, lens, t, 8, 8, 128, bs, dtype, **kw)
    most = max(len(p) for p in paths)
    accepted = torch.tensor([p + [0] * (most - len(p)) for p in paths], dtype=torch.int32)
    counts = torch.tensor([len(p) for p in paths], dtype=torch.int32)
    return c, accepted, counts


@pytest.mark.parametrize("quick", [True, False])
def test_commit_refuses_the_counts_as_the_place_of_the_new_lengths(quick, monkeypatch):
    pkv.load()
    if not quick:
        monkeypatch.setattr(pkv, "_quick", None)
    c, accepted, counts = _commit_case(6, [40, 90], [[0, 3, 5], [1, 2]])
    g, acc, cnt = ref.on_gpu(c), accepted.cuda(), counts.cuda()
    packed = torch.zeros(4, dtype=torch.int32, device="cuda")
    packed[1:3] = cnt
    before = g["k"].clone()
    for new, count in ((cnt, cnt), (packed[:2], packed[1:3]), (acc.view(-1)[:2], cnt),
                       (g["tables"].view(-1)[:2], cnt), (g["lens"], cnt)):
        with pytest.raises(pkv.PkvError, match="INVALID_ARG"):
            pkv.tree_commit(g["k"], g["v"], g["tables"], g["lens"], 6, acc, count,
                            new_context_lens=new)
    assert torch.equal(g["k"].view(torch.int16), before.view(torch.int16))
    # beside them is fine
    pkv.tree_commit(g["k"], g["v"], g["tables"], g["lens"], 6, acc, packed[1:3],
                    new_context_lens=torch.empty_like(cnt))
    want = ref.commit(c, 6, accepted, counts)
    assert _same_bits(g["k"], want[0]) and _same_bits(g["v"], want[1])
