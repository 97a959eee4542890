"""The plan of a ragged step against the plain one, sequence after sequence (GPU)."""
import random

import pytest
import torch

import paged_kv_cache_164_gb300 as pkv
import ragged_reference as ref

pytestmark = pytest.mark.gpu

OUTS = ("query_starts", "positions", "slot_mapping", "new_context_lens", "new_free_count",
        "block_tables", "free_blocks")


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _run(a, in_place=False, **kw):
    c = dict(context_lens=_ints(a["context"]), new_lens=_ints(a["new"]),
             block_tables=_ints(a["tables"]), free_blocks=_ints(a["free"]),
             free_count=_ints([a["count"]]))
    flag = pkv.new_error_flag("cuda")
    extra = dict(keep_lens=None if a.get("keep") is None else _ints(a["keep"]),
                 shared_pages=None if a.get("shared") is None else _ints(a["shared"]))
    if in_place:
        extra.update(new_context_lens=c["context_lens"], new_free_count=c["free_count"])
    got = pkv.batch_plan(*c.values(), a["num_blocks"], a["bs"], a["max_tokens"], err_flag=flag,
                         **extra, **kw)
    out = dict(zip(OUTS, got), block_tables=c["block_tables"], free_blocks=c["free_blocks"])
    return {n: t.tolist() for n, t in out.items()} | {"flags": pkv.check_error(flag)}


def _check(a, **kw):
    expect = ref.batch_plan(**a)
    got = _run(a, **kw)
    for n in OUTS + ("flags",):
        assert got[n] == expect[n], n


def _case(seed, b, bs, most_past, most_new, keep=True, shared=False, spare=20, max_tokens=None):
    r = random.Random(seed)
    context = [r.choice([0, 1, bs, r.randint(0, most_past)]) for _ in range(b)]
    kept = [r.choice([n, n, n, 0, r.randint(0, n)]) if keep else n for n in context]
    new = [r.choice([0, 1, 1, r.randint(0, most_new)]) for _ in range(b)]
    width = max([1] + [-(-(max(n, k + a)) // bs) for n, k, a in zip(context, kept, new)])
    held = [-(-n // bs) for n in context]
    need = sum(max(0, -(-(k + a) // bs) + 1) for k, a in zip(kept, new))
    num_blocks = sum(held) + need + 40
    pool = list(range(num_blocks))
    r.shuffle(pool)
    tables, at = [], 0
    for h in held:
        tables.append(pool[at:at + h] + [-1] * (width - h))
        at += h
    free = pool[at:]
    count = min(len(free), spare if spare is not None else len(free))
    free = free[:count] + [-1] * (num_blocks - count)
    return dict(context=context, new=new, keep=kept if keep else None, tables=tables, free=free,
                count=count, num_blocks=num_blocks, bs=bs,
                max_tokens=sum(new) + 5 if max_tokens is None else max_tokens,
                shared=[r.randint(0, 3) for _ in range(b)] if shared else None)


@pytest.mark.parametrize("b,bs,past,new", [(1, 16, 0, 40), (1, 128, 5000, 300), (7, 32, 200, 90),
                                           (64, 16, 500, 20), (300, 64, 900, 50)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plans(b, bs, past, new, in_place):
    _check(_case(b, b, bs, past, new, spare=None), in_place=in_place)


@pytest.mark.parametrize("seed", range(4))
def test_pages_that_run_out(seed):
    _check(_case(100 + seed, 40, 16, 300, 60, spare=seed))


@pytest.mark.parametrize("tokens", [0, 1, 17, 200])
def test_places_that_run_out(tokens):
    _check(_case(7, 40, 16, 300, 60, spare=None, max_tokens=tokens))


def test_more_sequences_than_threads_and_shared_pages():
    _check(_case(8, 2500, 16, 60, 4, spare=None, shared=True))
    _check(_case(9, 2500, 16, 60, 4, spare=300), in_place=True)
    _check(_case(10, 2500, 16, 60, 4, keep=False, spare=None, max_tokens=2000))


def test_many_tokens_go_through_the_second_kernel():
    _check(_case(11, 30, 32, 2000, 1500, spare=None))
    _check(_case(12, 1500, 16, 20, 9, spare=None, max_tokens=9000))


def test_one_sequence_gives_back_a_thousand_pages():
    n = 16 * 1000 + 3
    a = dict(context=[n, 5], new=[0, 700], keep=[0, 5],
             tables=[list(range(1001)), [1001] + [-1] * 1000], free=[-1] * 1002, count=0,
             num_blocks=1002, bs=16, max_tokens=700)
    _check(a)


def test_bad_inputs_are_flagged_and_leave_the_rest_in_order():
    a = _case(13, 12, 16, 100, 30, spare=None)
    for name, i, value in (("context", 2, -1), ("context", 3, 10 ** 6), ("keep", 4, -2),
                           ("new", 6, -7), ("new", 7, 2 ** 31 - 1)):
        bad = {n: list(x) if isinstance(x, list) else x for n, x in a.items()}
        bad[name][i] = value
        _check(bad)
    bad = dict(a, keep=list(a["context"]))
    bad["keep"][5] += 1
    _check(bad)
    for count in (-1, len(a["free"]) + 1):
        _check(dict(a, count=count))
    # a list too short for what comes back
    _check(dict(a, free=a["free"][:a["count"] + 1], keep=[0] * 12, new=[0] * 12))
    # a block that is none: on the list, and in a table
    _check(dict(a, free=[a["num_blocks"]] * len(a["free"])))
    tables = [list(r) for r in a["tables"]]
    tables[1][0] = -9
    _check(dict(a, tables=tables, context=[40] * 12, keep=[0] * 12))


def test_no_sequences_and_no_tokens():
    got = pkv.batch_plan(_ints([]), _ints([]), torch.zeros((0, 4), dtype=torch.int32, device="cuda"),
                         _ints([3, 1]), _ints([2]), 4, 16, 3)
    assert [t.tolist() for t in got] == [[0], [0, 0, 0], [-1, -1, -1], [], [2]]
    a = _case(14, 5, 16, 100, 30, spare=None, max_tokens=0)
    a["new"] = [0] * 5
    _check(a)


def test_steps_in_a_graph_that_updates_its_own_buffers():
    """Captured once, replayed with the lengths that the last replay left."""
    bs, b = 16, 6
    r = random.Random(3)
    a = _case(15, b, bs, 40, 0, spare=None)
    a.update(new=[1] * b, keep=None, max_tokens=64, tables=[x + [-1] * 20 for x in a["tables"]])
    c = [_ints(a["context"]), _ints(a["new"]), _ints(a["tables"]), _ints(a["free"]),
         _ints([a["count"]])]
    outs = dict(query_starts=_ints([0] * (b + 1)), positions=_ints([0] * 64),
                slot_mapping=_ints([0] * 64, torch.int64))
    call = lambda: pkv.batch_plan(*c, a["num_blocks"], bs, 64, new_context_lens=c[0],  # noqa: E731
                                  new_free_count=c[4], **outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(5):
        a["new"] = [r.randint(0, 9) for _ in range(b)]
        c[1].copy_(_ints(a["new"]))
        expect = ref.batch_plan(**a)
        graph.replay()
        for n, t in dict(outs, new_context_lens=c[0], new_free_count=c[4], block_tables=c[2],
                         free_blocks=c[3]).items():
            assert t.tolist() == expect[n], n
        a.update(context=expect["new_context_lens"], tables=expect["block_tables"],
                 free=expect["free_blocks"], count=expect["new_free_count"][0])
