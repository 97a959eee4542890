"""Refusals of a ragged step's entry points on the host, before any launch, and the
plain references against each other (CPU)."""
import ctypes
import random
from fractions import Fraction

import pytest
import torch

import paged_kv_cache_164_gb300 as pkv
import ragged_reference as ref
from paged_kv_cache_164_gb300 import build as pkv_build

NULL = ctypes.c_void_p(0)


def at(i, offset=0):  # far apart, 16-byte aligned, never dereferenced
    return ctypes.c_void_p(((i + 2) << 34) + offset)


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.load()


PLAN = ("qs", "pos", "slots", "ncl", "nfc", "cl", "nl", "kl", "sp", "bt", "mb", "fb", "fcap", "fc",
        "b", "mt", "nb", "bs")


def _plan(lib, **kw):
    a = {n: at(i) for i, n in enumerate(("qs", "pos", "slots", "ncl", "nfc", "cl", "nl", "kl", "sp",
                                         "bt", "fb", "fc"))}
    a.update(mb=4, fcap=8, b=2, mt=16, nb=8, bs=16)
    a.update(kw)
    return lib.pkv_batch_plan(*[a[n] for n in PLAN], NULL, NULL)


def test_batch_plan_refuses(lib):
    for n in ("qs", "pos", "slots", "ncl", "nfc", "cl", "nl", "bt", "fb", "fc"):
        assert _plan(lib, **{n: NULL}) == 1, n
    for n in PLAN:
        if n not in ("mb", "fcap", "b", "mt", "nb", "bs"):
            assert _plan(lib, **{n: at(3, 2)}) == 1, n
    assert _plan(lib, slots=at(2, 4)) == 1
    for n, v in (("b", -1), ("mt", -1), ("mb", 0), ("nb", 0), ("bs", 0), ("fcap", -1)):
        assert _plan(lib, **{n: v}) == 1, n
    assert _plan(lib, bs=48) == 2 and _plan(lib, mb=2 ** 28) == 2
    # what is written, over something else
    for out in ("qs", "pos", "slots", "bt", "fb"):
        for other in ("cl", "nl", "kl", "sp", "fc", "ncl"):
            assert _plan(lib, **{out: at(20), other: at(20, 8)}) == 1, (out, other)
    assert _plan(lib, ncl=at(20), cl=at(20, 4)) == 1  # in place is all or nothing
    assert _plan(lib, ncl=at(20), kl=at(20)) == 1
    assert _plan(lib, nfc=at(20), cl=at(20)) == 1


CHUNK = ("out", "q", "k", "v", "bt", "mb", "qs", "cl", "mcl", "pl", "sl", "b", "t", "nb", "bs", "hq",
         "hkv", "d", "scale", "cap", "window", "ws", "wsb", "dt")


def _chunk(lib, **kw):
    a = {n: at(i) for i, n in enumerate(("out", "q", "k", "v", "bt", "qs", "cl", "pl", "sl", "ws"))}
    a.update(mb=4, mcl=64, b=2, t=10, nb=8, bs=16, hq=8, hkv=2, d=64, scale=0.125, cap=0.0,
             window=0, wsb=0, dt=1)
    a.update(kw)
    return lib.pkv_chunk_attention(*[a[n] for n in CHUNK], NULL, NULL)


def test_chunk_attention_refuses(lib):
    for n in ("out", "q", "k", "v", "bt", "qs", "cl", "ws"):
        assert _chunk(lib, **{n: NULL}) == 1, n
    for n in ("out", "q", "k", "v", "bt", "qs", "cl", "pl", "sl", "ws"):
        assert _chunk(lib, **{n: at(5, 2)}) == 1, n
    for n, v in (("b", -1), ("t", -1), ("mb", 0), ("nb", 0), ("bs", 0), ("mcl", -1), ("hq", 9),
                 ("dt", 2), ("window", -1), ("cap", -1.0), ("cap", float("nan")),
                 ("cap", float("inf")), ("scale", float("inf")), ("scale", float("nan"))):
        assert _chunk(lib, **{n: v}) == 1, (n, v)
    for n, v in (("bs", 24), ("d", 96), ("hq", 64), ("mb", 2 ** 28), ("mcl", 2 ** 31 - 100)):
        assert _chunk(lib, **{n: v}) == 2, (n, v)
    assert _chunk(lib, b=0, q=NULL) == 0 and _chunk(lib, t=0, q=NULL) == 0
    for other in ("k", "v", "bt", "qs", "cl", "pl", "sl"):
        assert _chunk(lib, out=at(20), **{other: at(20, 16)}) == 1, other
    assert _chunk(lib, out=at(20), q=at(20, 128)) == 1
    size = lib.pkv_chunk_attention_workspace_size
    for bad in ((-1, 10, 8, 2, 64, 16, 64), (2, -1, 8, 2, 64, 16, 64), (2, 10, 7, 2, 64, 16, 64),
                (2, 10, 8, 2, 80, 16, 64), (2, 10, 8, 2, 64, 8, 64)):
        assert size(*bad) == pkv.SIZE_MAX


VERIFY = ("acc", "al", "nt", "ncl", "tp", "dp", "tok", "par", "rs", "u", "cl", "b", "n", "v", "ma")


def _verify(lib, **kw):
    a = {n: at(i) for i, n in enumerate(VERIFY[:11])}
    a.update(b=2, n=10, v=100, ma=5)
    a.update(kw)
    return lib.pkv_verify_drafts(*[a[n] for n in VERIFY], NULL, NULL)


def test_verify_drafts_refuses(lib):
    for n in ("acc", "al", "nt", "tp", "tok", "rs", "u", "cl", "ncl"):
        assert _verify(lib, **{n: NULL}) == 1, n
    for n in VERIFY[:11]:
        assert _verify(lib, **{n: at(5, 2)}) == 1, n
    for n, v in (("b", -1), ("n", -1), ("v", 0), ("ma", 0)):
        assert _verify(lib, **{n: v}) == 1, n
    assert _verify(lib, v=2 ** 24 + 1) == 2
    assert _verify(lib, b=0, tp=NULL) == 0
    for out in ("acc", "al", "nt", "ncl"):
        for other in ("tp", "dp", "tok", "par", "rs", "u"):
            assert _verify(lib, **{out: at(20), other: at(20, 4)}) == 1, (out, other)
    assert _verify(lib, ncl=at(20), cl=at(20, 4)) == 1
    assert _verify(lib, acc=at(20), al=at(20, 4)) == 1


def test_python_calls_refuse_what_is_not_on_a_gpu(lib):
    i32 = torch.zeros(3, dtype=torch.int32)
    x = torch.zeros((3, 4, 64), dtype=torch.float16)
    kv = torch.zeros((2, 16, 2, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.batch_plan(i32, i32, torch.zeros((3, 2), dtype=torch.int32), i32, i32[:1], 4, 16, 8)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.chunk_attention(x, kv, kv, torch.zeros((2, 2), dtype=torch.int32), i32, i32[:2], 16)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.verify_drafts(torch.zeros((3, 9)), None, i32, i32, torch.zeros(3), 3)


def test_the_reference_of_the_plan_keeps_every_page_once():
    """Over random steps no page is lost, and none has two holders."""
    r = random.Random(5)
    bs, b, blocks = 16, 9, 120
    state = dict(context=[0] * b, tables=[[-1] * 40 for _ in range(b)],
                 free=list(range(blocks)), count=blocks)
    for _ in range(200):
        keep = [r.choice([n, n, n, 0, r.randint(0, n)]) for n in state["context"]]
        new = [r.choice([0, 1, r.randint(0, 70)]) for _ in range(b)]
        new = [min(a, 640 - k) for a, k in zip(new, keep)]
        out = ref.batch_plan(new=new, keep=keep, num_blocks=blocks, bs=bs, max_tokens=300, **state)
        assert out["flags"] in (0, 0x100)
        state = dict(context=out["new_context_lens"], tables=out["block_tables"],
                     free=out["free_blocks"], count=out["new_free_count"][0])
        held = [blk for n, row in zip(state["context"], state["tables"]) for blk in row[:-(-n // bs)]]
        assert sorted(held + state["free"][:state["count"]]) == list(range(blocks))
        live = [s for s in out["slot_mapping"] if s >= 0]
        assert len(set(live)) == len(live) == out["query_starts"][-1]


def test_the_reference_of_the_verification_draws_from_the_target():
    """Averaged over the random numbers, the first new token of a chain or of siblings has
    the target's distribution: with fractions, over a grid of numbers, exactly."""
    p = torch.tensor([[0.5, 0.25, 0.125, 0.125]])
    q = torch.tensor([[0.25, 0.25, 0.25, 0.25]])
    grid = 64
    for kids in (1, 2):
        mass = [Fraction(0)] * 4
        drafts = [[x] for x in range(4)] if kids == 1 else [[x, y] for x in range(4) for y in range(4)]
        for d in drafts:
            reach, left, z = Fraction(1, 4 ** kids), [Fraction(v) for v in p[0].tolist()], Fraction(1)
            for x in d:
                take = min(Fraction(1), left[x] / (z * Fraction(1, 4)))
                if z == 1:  # the reference decides as this share of its numbers says
                    hits = 0
                    for i in range(grid):
                        c = ref.verify(torch.cat([p] * 2), torch.cat([q] * 2),
                                       torch.tensor([0, x]), [0, 2],
                                       torch.tensor([0.0, (i + 0.5) / grid]), 2)
                        hits += c["accepted_lens"][0] - 1
                    assert Fraction(hits, grid) == take
                mass[x] += reach * take
                reach *= 1 - take
                left = [max(a - z * Fraction(1, 4), Fraction(0)) for a in left]
                z = sum(left)
                if reach == 0:
                    break
            if reach:
                for k in range(4):
                    mass[k] += reach * left[k] / z
        assert [float(m) for m in mass] == p[0].tolist()


def test_quick_binding_leaves_what_it_does_not_know_to_python(lib):
    if pkv._quick is None:
        pytest.skip("built without the headers of Python and torch")
    i = torch.zeros((1, 1), dtype=torch.int32)
    k = torch.zeros((4, 16, 2, 64), dtype=torch.float16)
    quick = pkv._quick
    for call, n in ((quick.batch_plan, 16), (quick.chunk_attention, 16), (quick.verify_drafts, 13)):
        for args in ((), (i,) * n, (i[0],) * n, (k,) * n, (k[0],) * n, (None,) * n, (1,) * n,
                     ("nhd",) * n, (object(),) * (n + 1), (i.to_sparse(),) * n,
                     (k[0].to("meta"),) * n):
            assert call(*args) is None
    with pytest.raises(TypeError):
        quick.bind_ragged(1, 2)
    with pytest.raises(ValueError):
        quick.bind_ragged(0, 0, 0)
