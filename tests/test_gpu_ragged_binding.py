"""The quick form of the ragged step's Python calls against the form checked in Python: the
same outputs, bit for bit, and the same refusals."""
import pytest
import torch

import paged_kv_cache_164_gb300 as pkv
import ragged_reference as ref

pytestmark = pytest.mark.gpu


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


@pytest.fixture
def spy(monkeypatch):
    pkv.load()
    assert pkv._quick is not None, "pkv_binding.so is not built"
    s = _Spy(pkv._quick)
    monkeypatch.setattr(pkv, "_quick", s)
    return s


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _empty(*shape, dtype=torch.int32):
    return torch.full(shape, -7, dtype=dtype, device="cuda")


def _plan_args(flag=None):
    """A plan with every output given, its inputs new each time (it updates them)."""
    return dict(context_lens=_i32(20, 0, 33), new_lens=_i32(3, 17, 1),
                block_tables=_i32(4, 1, -1, -1, -1, -1, 0, 3, 5).view(3, 3),
                free_blocks=_i32(2, 6, 7, 8, -1, -1, -1, -1, -1, -1), free_count=_i32(4),
                num_blocks=9, block_size=16, max_tokens=25, keep_lens=_i32(15, 0, 33),
                shared_pages=_i32(0, 0, 1), query_starts=_empty(4), positions=_empty(25),
                slot_mapping=_empty(25, dtype=torch.int64), new_context_lens=_empty(3),
                new_free_count=_empty(1), err_flag=flag)


def _chunk_args(layout="nhd", bias=True, flag=None, **kw):
    c = ref.on_gpu(ref.make_chunk(3, [(70, 20), (0, 0), (33, 1), (200, 130)], 8, 2, 64, 16, "bf16",
                                  layout, window=90, prefix=[30, 0, 0, 150], softcap=20.0,
                                  bias=bias, lead=1))
    need = pkv.chunk_attention_workspace_size(4, c["q"].shape[0], 8, 2, 64, 16, c["max_len"])
    return dict(q=c["q"], k_cache=c["k"], v_cache=c["v"], block_tables=c["tables"],
                query_starts=c["starts"], context_lens=c["lens"], max_context_len=c["max_len"],
                scale=c["scale"], softcap=c["softcap"], window=c["window"], slopes=c["slopes"],
                prefix_lens=c["prefix"], out=torch.full_like(c["q"], 7.0),
                workspace=torch.empty(need, dtype=torch.uint8, device="cuda"), err_flag=flag,
                layout=layout) | kw


def _verify_args(tree=True, draft=True, lens=True, flag=None):
    g = torch.Generator().manual_seed(9)
    p = torch.softmax(torch.randn(7, 300, generator=g) * 2, -1).cuda()
    q = torch.softmax(torch.randn(7, 300, generator=g) * 2, -1).cuda()
    return dict(target_probs=p, draft_probs=q if draft else None,
                tokens=torch.randint(0, 300, (7,), generator=g).int().cuda(),
                row_starts=_i32(0, 4, 4, 7), uniforms=torch.rand(7, generator=g).cuda(),
                max_accepted=4, parents=_i32(-1, 0, 0, 1, -1, 0, 1) if tree else None,
                context_lens=_i32(50, 60, 70) if lens else None, accepted=_empty(3, 4),
                accepted_lens=_empty(3), next_tokens=_empty(3),
                new_context_lens=_empty(3) if lens else None, err_flag=flag)


def _bits(args):
    """What a call read and wrote (a workspace's bytes mean nothing afterwards)."""
    return [t.clone().view(torch.uint8) for n, t in args.items()
            if isinstance(t, torch.Tensor) and n != "workspace"]


CASES = [(pkv.batch_plan, _plan_args, {}), (pkv.chunk_attention, _chunk_args, {}),
         (pkv.chunk_attention, _chunk_args, dict(layout="hnd", bias=False)),
         (pkv.chunk_attention, _chunk_args, dict(scale=None)),
         (pkv.verify_drafts, _verify_args, {}),
         (pkv.verify_drafts, _verify_args, dict(tree=False, draft=False, lens=False))]


@pytest.mark.parametrize("call,make,kw", CASES)
def test_both_forms_write_the_same(call, make, kw, spy, monkeypatch):
    both = []
    for quick in (True, False):
        if not quick:
            monkeypatch.setattr(pkv, "_quick", None)
        flag = pkv.new_error_flag("cuda")
        args = make(**kw, flag=flag)
        got = call(**args)
        first = got if isinstance(got, torch.Tensor) else got[0]
        assert any(first is x for x in args.values())
        both.append(_bits(args))
        assert pkv.check_error(flag) == 0
    assert spy.results == [0]
    for a, b in zip(*both):
        assert torch.equal(a, b)


OUTS = {pkv.batch_plan: ("query_starts", "positions", "slot_mapping", "new_context_lens",
                         "new_free_count"),
        pkv.chunk_attention: ("out",),
        pkv.verify_drafts: ("accepted", "accepted_lens", "next_tokens", "new_context_lens")}


@pytest.mark.parametrize("call,make", [c[:2] for c in (CASES[0], CASES[1], CASES[4])])
def test_other_forms_are_left_to_python(call, make, spy):
    """Outputs to allocate, another stream: the same call.  A current stream that is not the
    default one: the quick form, on it."""
    def result(**change):
        got = call(**{**make(), **change})
        return [got] if isinstance(got, torch.Tensor) else list(got)
    full = result()
    rows = slice(1, 152) if call is pkv.chunk_attention else slice(None)  # (written ones)
    for name in OUTS[call]:
        if call is pkv.verify_drafts and name == "new_context_lens":
            continue
        for a, b in zip(full, result(**{name: None})):
            assert torch.equal(a[rows], b[rows])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    args = make()
    torch.cuda.synchronize()
    got = call(**args, stream=side)
    side.synchronize()
    assert torch.equal(full[0], got if isinstance(got, torch.Tensor) else got[0])
    assert spy.results[0] == 0 and not any(r is not None for r in spy.results[1:])
    with torch.cuda.stream(side):
        got = result()
    side.synchronize()
    assert spy.results[-1] == 0 and torch.equal(full[0], got[0])


@pytest.mark.parametrize("quick", [True, False])
def test_refusals_are_the_same(quick, monkeypatch):
    pkv.load()
    if not quick:
        monkeypatch.setattr(pkv, "_quick", None)
    good = _plan_args()
    for bad, error in ((dict(context_lens=good["context_lens"].long()), TypeError),
                       (dict(new_lens=good["new_lens"][:2]), ValueError),
                       (dict(new_lens=None), (TypeError, ValueError, pkv.PkvError)),
                       (dict(block_tables=good["block_tables"].t()), ValueError),
                       (dict(block_tables=good["block_tables"][:2]), ValueError),
                       (dict(free_blocks=good["free_blocks"][::2]), ValueError),
                       (dict(free_count=good["free_blocks"]), ValueError),
                       (dict(positions=good["positions"][:24]), ValueError),
                       (dict(slot_mapping=good["positions"]), TypeError),
                       (dict(max_tokens=2 ** 33 + 25), ValueError),
                       (dict(max_tokens=-1), ValueError), (dict(block_size=48), pkv.PkvError),
                       (dict(num_blocks=-1), pkv.PkvError),
                       (dict(query_starts=good["new_lens"]), ValueError),
                       (dict(positions=good["block_tables"].view(-1)[:25]), ValueError),
                       (dict(new_context_lens=good["new_lens"]), pkv.PkvError)):
        with pytest.raises(error):
            pkv.batch_plan(**{**good, **bad})
    good = _chunk_args()
    for bad, error in ((dict(out=good["out"].half()), TypeError),
                       (dict(out=good["out"][:, :4]), ValueError),
                       (dict(q=good["q"].transpose(0, 1).contiguous().transpose(0, 1)), ValueError),
                       (dict(v_cache=good["v_cache"][:-1]), ValueError),
                       (dict(k_cache=good["k_cache"].float()), TypeError),
                       (dict(query_starts=good["context_lens"]), ValueError),
                       (dict(context_lens=good["context_lens"][:3]), ValueError),
                       (dict(slopes=good["slopes"][:4]), ValueError),
                       (dict(slopes=good["slopes"].double()), TypeError),
                       (dict(prefix_lens=good["prefix_lens"].long()), TypeError),
                       (dict(workspace=good["workspace"][:16]), pkv.PkvError),
                       (dict(scale=float("nan")), pkv.PkvError),
                       (dict(softcap=-1.0), pkv.PkvError), (dict(window=-1), pkv.PkvError),
                       (dict(window=2 ** 31), ValueError), (dict(layout="nhdd"), ValueError),
                       (dict(max_context_len=2 ** 31), ValueError),
                       (dict(err_flag=good["slopes"]), TypeError)):
        with pytest.raises(error):
            pkv.chunk_attention(**{**good, **bad})
    good = _verify_args()
    for bad, error in ((dict(draft_probs=good["draft_probs"][:, :299]), ValueError),
                       (dict(target_probs=good["target_probs"].half()), TypeError),
                       (dict(tokens=good["tokens"].long()), TypeError),
                       (dict(parents=good["parents"][:6]), ValueError),
                       (dict(uniforms=good["uniforms"].double()), TypeError),
                       (dict(accepted=good["accepted"][:, :3]), ValueError),
                       (dict(max_accepted=0), ValueError), (dict(max_accepted=5), ValueError),
                       (dict(context_lens=None), ValueError),
                       (dict(next_tokens=good["accepted_lens"]), pkv.PkvError),
                       (dict(row_starts=good["row_starts"].view(2, 2)), ValueError)):
        with pytest.raises(error):
            pkv.verify_drafts(**{**good, **bad})
    torch.cuda.synchronize()
