"""The ragged step's operators at the sizes where their kernels change form, and two calls at
once (GPU)."""
import random

import pytest
import torch

import paged_kv_cache_164_gb300 as pkv
import ragged_reference as ref

pytestmark = pytest.mark.gpu


def _plan(b, max_tokens, seed, release):
    """b sequences of a few tokens; with `release` some of them give pages back."""
    r = random.Random(seed)
    context = [r.randint(0, 40) for _ in range(b)]
    keep = [r.choice([n, n, r.randint(0, n)]) if release else n for n in context]
    new = [r.choice([0, 1, 1, 3, 5]) for _ in range(b)]
    held = [-(-n // 16) for n in context]
    blocks = list(range(sum(held) + 2 * b))
    r.shuffle(blocks)
    tables = [[blocks.pop() for _ in range(h)] + [-1] * (4 - h) for h in held]
    free = blocks + [-1] * sum(held)
    return dict(context=context, new=new, tables=tables, free=free, count=len(blocks),
                num_blocks=sum(held) + 2 * b, bs=16, max_tokens=max_tokens, keep=keep)


def _run_plan(a):
    i32 = dict(dtype=torch.int32, device="cuda")
    tables, free = torch.tensor(a["tables"], **i32), torch.tensor(a["free"], **i32)
    flag = pkv.new_error_flag("cuda")
    got = pkv.batch_plan(torch.tensor(a["context"], **i32), torch.tensor(a["new"], **i32), tables,
                         free, torch.tensor([a["count"]], **i32), a["num_blocks"], a["bs"],
                         a["max_tokens"], keep_lens=torch.tensor(a["keep"], **i32), err_flag=flag)
    names = ("query_starts", "positions", "slot_mapping", "new_context_lens", "new_free_count")
    out = dict(zip(names, (t.tolist() for t in got)))
    return out | dict(block_tables=tables.tolist(), free_blocks=free.tolist(),
                      flags=pkv.check_error(flag))


@pytest.mark.parametrize("release", [False, True])
@pytest.mark.parametrize("b,max_tokens", [(512, 4096), (513, 4096), (512, 4097), (1, 4097),
                                          (2047, 9000), (2048, 9000), (2048, 4096), (3000, 12000),
                                          (600, 700)])
def test_plans_where_the_kernels_change(b, max_tokens, release):
    a = _plan(b, max_tokens, b + max_tokens, release)
    expect, got = ref.batch_plan(**a), _run_plan(a)
    for name in got:
        assert got[name] == expect[name], name


@pytest.mark.parametrize("b", [32, 33, 511, 513, 1300])
def test_attention_of_as_many_sequences_as_threads_and_more(b):
    seqs = [(1 + (37 * i) % 50, 1 if i % 3 else 0) for i in range(b)]
    c = ref.make_chunk(b, seqs, 2, 1, 64, 16, "bf16")
    out, bound = ref.attention(c)
    g = ref.on_gpu(c)
    before = torch.full_like(g["q"], 7.0)
    got = before.clone()
    flag = pkv.new_error_flag("cuda")
    pkv.chunk_attention(g["q"], g["k"], g["v"], g["tables"], g["starts"], g["lens"], g["max_len"],
                        scale=g["scale"], out=got, err_flag=flag)
    assert pkv.check_error(flag) == 0
    ref.assert_close(got, out, bound, before)


@pytest.mark.parametrize("rows", [31, 32, 33, 127, 128, 129, 255, 256, 257])
def test_units_of_every_kind_of_row_count(rows):
    """One sequence of `rows` tokens of one head: few rows, one warpgroup's, both's, two units."""
    for d, dtype in ((128, "bf16"), (64, "fp16")):
        c = ref.make_chunk(rows, [(rows + 300, rows), (rows, rows)], 1, 1, d, 16, dtype)
        out, bound = ref.attention(c)
        g = ref.on_gpu(c)
        before = torch.full_like(g["q"], 7.0)
        got = before.clone()
        pkv.chunk_attention(g["q"], g["k"], g["v"], g["tables"], g["starts"], g["lens"],
                            g["max_len"], scale=g["scale"], out=got)
        ref.assert_close(got, out, bound, before)


def test_calls_at_once_on_two_streams():
    """Both with workspaces of their own, again and again: what each gives by itself."""
    cases = [ref.on_gpu(ref.make_chunk(s, seqs, 8, 2, 128, 16, "bf16"))
             for s, seqs in ((1, [(900, 1)] * 9 + [(400, 300)]), (2, [(700, 500), (30, 2)]))]
    probs = torch.softmax(torch.randn(60, 5000, device="cuda"), -1)
    tokens = torch.randint(0, 5000, (60,), device="cuda", dtype=torch.int32)
    starts = torch.arange(0, 61, 6, device="cuda", dtype=torch.int32)
    uniforms = torch.rand(60, device="cuda")

    def attend(c, stream=None):
        return pkv.chunk_attention(c["q"], c["k"], c["v"], c["tables"], c["starts"], c["lens"],
                                   c["max_len"], scale=c["scale"], out=torch.zeros_like(c["q"]),
                                   stream=stream)

    def verify(stream=None):
        return pkv.verify_drafts(probs, probs, tokens, starts, uniforms, 6, stream=stream)[:3]
    alone = [attend(c).clone() for c in cases]
    told = [t.clone() for t in verify()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got.append((i, attend(cases[i]), verify()))
    torch.cuda.synchronize()
    for i, out, path in got:
        assert torch.equal(out, alone[i])
        for a, b in zip(path, told):
            assert torch.equal(a, b)


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_pages_behind_32_bit_offsets(layout):
    """The last pages of caches of 2.3e9 values each, an infinity among them that only some
    rows see."""
    c = ref.make_chunk(77, [(300, 40), (65, 1)], 16, 8, 128, 16, "bf16", layout)
    c["v"][c["tables"][0, 290 // 16], 290 % 16, 3, 5] = float("inf")
    out, bound = ref.attention(c)
    g = ref.on_gpu(c)
    used, blocks = c["k"].shape[0], 140000
    big = [torch.empty((blocks, *g[n].shape[1:]), dtype=torch.bfloat16, device="cuda")
           for n in "kv"]
    assert big[0].numel() > 2 ** 31
    for x, n in zip(big, "kv"):
        x[blocks - used:] = g[n]
    tables = torch.where(g["tables"] >= 0, g["tables"] + (blocks - used), -1).int()
    before = torch.full_like(g["q"], 7.0)
    got = before.clone()
    flag = pkv.new_error_flag("cuda")
    pkv.chunk_attention(g["q"], *big, tables, g["starts"], g["lens"], g["max_len"],
                        scale=g["scale"], out=got, layout=layout, err_flag=flag)
    assert pkv.check_error(flag) == 0
    ref.assert_close(got, out, bound, before)
