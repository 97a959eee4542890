"""The quick form of the tree step's Python calls against the form checked in Python:
the same outputs, bit for bit, and the same refusals."""
import pytest
import torch

import paged_kv_cache_164_gb300 as pkv

pytestmark = pytest.mark.gpu

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _step(seed, dtype, layout, b, t, h_q, h_kv, d, bs, f8=False):
    gen = torch.Generator().manual_seed(seed)
    dt = DTYPES[dtype]
    pages = (150 + t + bs - 1) // bs
    lens = torch.randint(t, 150 + t, (b,), generator=gen, dtype=torch.int32)
    tables = torch.randperm(b * pages, generator=gen).to(torch.int32).view(b, pages)
    shape = (b * pages, bs, h_kv, d) if layout == "nhd" else (b * pages, h_kv, bs, d)
    parents = torch.stack([torch.randint(-1, max(i, 1), (b,), generator=gen) if i else
                           torch.full((b,), -1) for i in range(t)], 1).to(torch.int32)
    angles = torch.rand(400, d // 2, generator=gen) * 6
    c = dict(lens=lens, tables=tables, parents=parents,
             k_cache=torch.randn(shape, generator=gen).to(dt),
             v_cache=torch.randn(shape, generator=gen).to(dt),
             qkv=torch.randn(b * t, h_q + 2 * h_kv, d, generator=gen).to(dt),
             table=torch.cat([angles.cos(), angles.sin()], 1),
             weight=torch.rand(d, generator=gen).to(dt),
             accepted=torch.zeros(b, 2, dtype=torch.int32),
             counts=torch.randint(0, 2, (b,), generator=gen, dtype=torch.int32))
    c = {k: v.cuda() for k, v in c.items()}
    if f8:
        c["k8"], c["v8"] = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in "kv")
    return c, dict(b=b, t=t, h_q=h_q, h_kv=h_kv, d=d, bs=bs, layout=layout, f8=f8,
                   cap=pages * bs, nb=b * pages)


def _calls(c, p):
    """One step with every output given: what it wrote."""
    b, t, h_q, h_kv, d = (p[n] for n in ("b", "t", "h_q", "h_kv", "d"))
    mask = torch.full((b, t, (t + 31) // 32), -7, dtype=torch.int32, device="cuda")
    pos = torch.full((b, t), -7, dtype=torch.int32, device="cuda")
    slots = torch.full((b, t), -7, dtype=torch.int64, device="cuda")
    flag = pkv.new_error_flag("cuda")
    kc, vc = c["k_cache"].clone(), c["v_cache"].clone()
    got = pkv.tree_plan(c["parents"], c["lens"], c["tables"], p["nb"], p["bs"], p["cap"],
                        tree_mask=mask, positions=pos, slot_mapping=slots, err_flag=flag)
    assert got[0] is mask and got[1] is pos and got[2] is slots
    q, k, v = c["qkv"].split([h_q, h_kv, h_kv], 1)
    q_out = torch.empty(b * t, h_q, d, dtype=q.dtype, device="cuda")
    kw = dict(q_weight=c["weight"], q_out=q_out, err_flag=flag, layout=p["layout"])
    if p["f8"]:
        k8, v8 = c["k8"].clone(), c["v8"].clone()
        pkv.norm_rope_append_fp8(q, k, v, pos.view(-1), c["table"], k8, v8, slots.view(-1), 0.02,
                                 0.03, style="interleaved", **kw)
    assert pkv.norm_rope_append(q, k, v, pos.view(-1), c["table"], kc, vc, slots.view(-1),
                                **kw) is q_out
    out = torch.empty(b, t, h_q, d, dtype=q.dtype, device="cuda")
    ws = _workspace(p)
    both = []
    for scale in (None, 0.21):
        assert pkv.tree_attention(q_out.view(b, t, h_q, d), kc, vc, c["tables"], c["lens"],
                                  p["cap"], mask, scale=scale, out=out, workspace=ws,
                                  err_flag=flag, layout=p["layout"]) is out
        both.append(out.clone())
    lens = torch.empty_like(c["lens"])
    assert pkv.tree_commit(kc, vc, c["tables"], c["lens"], t, c["accepted"], c["counts"],
                           new_context_lens=lens, err_flag=flag, layout=p["layout"]) is lens
    assert pkv.check_error(flag) == 0
    return [mask, pos, slots, q_out, kc, vc, lens, *both, *((k8, v8) if p["f8"] else ())]


def _workspace(p):
    need = pkv.tree_attention_workspace_size(p["b"], p["t"], p["h_q"], p["h_kv"], p["d"],
                                             p["bs"], p["cap"])
    return torch.empty(need, dtype=torch.uint8, device="cuda")


class _Spy:
    """The quick module, with the results of its calls kept."""

    def __init__(self, module):
        self.module, self.results = module, []

    def __getattr__(self, name):
        call = getattr(self.module, name)

        def run(*args):
            self.results.append(call(*args))
            return self.results[-1]
        return run


@pytest.mark.parametrize("case", [
    ("fp16", "nhd", 3, 7, 4, 2, 64, 16, False), ("bf16", "hnd", 2, 33, 8, 1, 128, 32, True),
    ("bf16", "nhd", 1, 1, 2, 2, 64, 128, True), ("fp16", "hnd", 4, 40, 32, 8, 128, 16, False),
])
def test_both_forms_of_a_step_write_the_same(case, monkeypatch):
    pkv.load()
    assert pkv._quick is not None, "pkv_binding.so is not built"
    c, p = _step(sum(map(ord, str(case))), *case)
    spy = _Spy(pkv._quick)
    monkeypatch.setattr(pkv, "_quick", spy)
    quick = _calls(c, p)
    assert spy.results == [0] * len(spy.results) and len(spy.results) == 5 + p["f8"]
    monkeypatch.setattr(pkv, "_quick", None)
    for a, b in zip(quick, _calls(c, p)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_other_forms_are_left_to_python(monkeypatch):
    """Outputs to allocate, another stream, a wider integer or float type: the same call."""
    pkv.load()
    c, p = _step(5, "fp16", "nhd", 2, 5, 4, 2, 64, 16)
    spy = _Spy(pkv._quick)
    monkeypatch.setattr(pkv, "_quick", spy)
    plan = (c["parents"], c["lens"], c["tables"], p["nb"], p["bs"], p["cap"])
    first = pkv.tree_plan(*plan)
    again = pkv.tree_plan(*plan, tree_mask=torch.empty_like(first[0]))
    assert spy.results == [None, None]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    third = pkv.tree_plan(*plan, *(torch.empty_like(x) for x in first), stream=side)
    side.synchronize()
    assert spy.results == [None, None]
    for a, b, d in zip(first, again, third):
        assert torch.equal(a, b) and torch.equal(a, d)
    q = c["qkv"][:, :4].contiguous().view(2, 5, 4, 64)
    attend = (q, c["k_cache"], c["v_cache"], c["tables"], c["lens"])
    a = pkv.tree_attention(*attend, p["cap"], first[0])
    ws = _workspace(p)
    b = pkv.tree_attention(*attend, p["cap"], first[0], scale=1 / 8, out=torch.empty_like(q),
                           workspace=ws)
    assert spy.results[2:] == [None, 0] and torch.equal(a, b)
    # the current stream is the one that torch has current at the call
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d = pkv.tree_attention(*attend, p["cap"], first[0], scale=1 / 8, out=torch.empty_like(q),
                               workspace=ws)
    side.synchronize()
    assert spy.results[-1] == 0 and torch.equal(a, d)


def test_one_mask_of_all_sequences_and_a_mask_with_a_stride(monkeypatch):
    pkv.load()
    c, p = _step(6, "bf16", "nhd", 3, 35, 4, 2, 64, 16)
    mask = pkv.tree_plan(c["parents"], c["lens"], c["tables"], p["nb"], p["bs"], p["cap"])[0]
    q = torch.randn(3, 35, 4, 64, device="cuda").bfloat16()
    out, ws = torch.empty_like(q), _workspace(p)
    wide = torch.stack([mask, mask], 1)[:, 0]
    spy = _Spy(pkv._quick)
    for m in (mask[:1], wide, mask):
        monkeypatch.setattr(pkv, "_quick", spy)
        a = pkv.tree_attention(q, c["k_cache"], c["v_cache"], c["tables"], c["lens"], p["cap"], m,
                               out=out, workspace=ws).clone()
        assert spy.results[-1] == 0
        monkeypatch.setattr(pkv, "_quick", None)
        b = pkv.tree_attention(q, c["k_cache"], c["v_cache"], c["tables"], c["lens"], p["cap"], m)
        assert torch.equal(a, b)


@pytest.mark.parametrize("quick", [True, False])
def test_refusals_are_the_same(quick, monkeypatch):
    pkv.load()
    if not quick:
        monkeypatch.setattr(pkv, "_quick", None)
    c, p = _step(7, "fp16", "nhd", 2, 5, 4, 2, 64, 16)
    mask = torch.zeros(2, 5, 1, dtype=torch.int32, device="cuda")
    pos = torch.zeros(2, 5, dtype=torch.int32, device="cuda")
    slots = torch.zeros(2, 5, dtype=torch.int64, device="cuda")
    outs = dict(tree_mask=mask, positions=pos, slot_mapping=slots)
    good = dict(parents=c["parents"], context_lens=c["lens"], block_tables=c["tables"],
                num_blocks=p["nb"], block_size=16, max_context_len=p["cap"])
    for bad, error in ((dict(context_lens=c["lens"].long()), TypeError),
                       (dict(context_lens=c["lens"][:1]), ValueError),
                       (dict(block_tables=c["tables"].t()), ValueError),
                       (dict(block_tables=c["tables"].cpu()), ValueError),
                       (dict(max_context_len=2 ** 32 + 64), ValueError),
                       (dict(num_blocks=2 ** 40), ValueError),
                       (dict(block_size=48), pkv.PkvError),
                       (dict(max_context_len=-1), pkv.PkvError),
                       (dict(tree_mask=mask[:, :4]), ValueError),
                       (dict(slot_mapping=pos), TypeError),
                       (dict(err_flag=slots), TypeError)):
        with pytest.raises(error):
            pkv.tree_plan(**{**good, **outs, **bad})
    q = torch.zeros(2, 5, 4, 64, dtype=torch.float16, device="cuda")
    ws = _workspace(p)
    good = dict(q=q, k_cache=c["k_cache"], v_cache=c["v_cache"], block_tables=c["tables"],
                context_lens=c["lens"], max_context_len=p["cap"], tree_mask=mask,
                out=torch.empty_like(q), workspace=ws)
    for bad, error in ((dict(out=torch.empty_like(q).bfloat16()), TypeError),
                       (dict(out=q[:, :4]), ValueError),
                       (dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), ValueError),
                       (dict(v_cache=c["v_cache"][:-1]), ValueError),
                       (dict(k_cache=c["k_cache"].float()), TypeError),
                       (dict(tree_mask=mask.long()), TypeError),
                       (dict(tree_mask=mask.expand(2, 5, 2)), ValueError),
                       (dict(tree_mask=mask[:, :1].expand(2, 5, 1)), ValueError),
                       (dict(workspace=ws[:16]), pkv.PkvError),
                       (dict(layout="nhdd"), ValueError),
                       (dict(scale=float("nan")), pkv.PkvError),
                       (dict(max_context_len=2 ** 31), ValueError)):
        with pytest.raises(error):
            pkv.tree_attention(**{**good, **bad})
    lens = torch.empty_like(c["lens"])
    good = dict(k_cache=c["k_cache"], v_cache=c["v_cache"], block_tables=c["tables"],
                context_lens=c["lens"], tree_len=5, accepted=c["accepted"],
                accepted_lens=c["counts"], new_context_lens=lens)
    for bad, error in ((dict(accepted=c["accepted"].t().contiguous().t()), ValueError),
                       (dict(accepted_lens=c["counts"].long()), TypeError),
                       (dict(new_context_lens=lens[:1]), ValueError),
                       (dict(new_context_lens=c["lens"]), pkv.PkvError),
                       (dict(tree_len=0), pkv.PkvError), (dict(tree_len=2 ** 33 + 5), ValueError),
                       (dict(k_cache=c["k_cache"].float(), v_cache=c["v_cache"].float()),
                        TypeError)):
        with pytest.raises(error):
            pkv.tree_commit(**{**good, **bad})
    rows, kv = c["qkv"][:, :4], c["qkv"][:, 4:6]
    good = dict(q=rows, k=kv, v=kv, positions=pos.view(-1), cos_sin=c["table"],
                k_cache=c["k_cache"], v_cache=c["v_cache"],
                slot_mapping=torch.full((10,), -1, device="cuda"),
                q_out=torch.empty(10, 4, 64, dtype=torch.float16, device="cuda"))
    pkv.norm_rope_append(**good)
    for bad, error in ((dict(positions=pos.view(-1).long()), TypeError),
                       (dict(positions=pos.view(-1)[:9]), ValueError),
                       (dict(q_weight=torch.ones(32, device="cuda").half()), ValueError),
                       (dict(q_weight=torch.ones(64, device="cuda")), TypeError),
                       (dict(cos_sin=c["table"].half()), TypeError),
                       (dict(style="none"), ValueError), (dict(eps=-1.0), pkv.PkvError),
                       (dict(q=c["qkv"][:, :4, :32]), ValueError),
                       (dict(k=c["qkv"][:, 1:6:2][:, :2]), ValueError),
                       (dict(q_out=torch.empty(10, 4, 64, device="cuda")), TypeError)):
        with pytest.raises(error):
            pkv.norm_rope_append(**{**good, **bad})
    torch.cuda.synchronize()
