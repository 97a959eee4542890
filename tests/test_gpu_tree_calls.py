"""Calls of the tree step that are easily made and were once answered wrongly or refused (GPU)."""
import ctypes
import subprocess
import threading
import time

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


def test_outputs_made_for_another_stream_lie_in_no_memory_that_is_in_use():
    """Blocks that are freed on the current stream, where work that writes them is still
    queued, while the calls run at once on another stream."""
    t, h_q, h_kv, d, bs = 40, 4, 2, 64, 16
    c = ref.make_case(71, [60, 300], t, h_q, h_kv, d, bs, "fp16")
    g, nb = ref.on_gpu(c), c["k"].shape[0]
    accepted = torch.tensor([[0, 3, 15], [2, 3, 9]], dtype=torch.int32, device="cuda")
    counts = torch.tensor([3, 2], dtype=torch.int32, device="cuda")
    x = torch.randn(2 * t, h_q + 2 * h_kv, d, device="cuda").half()
    pos = torch.arange(2 * t, dtype=torch.int32, device="cuda")
    slots = pos.long()
    angle = torch.rand(2 * t, d // 2, device="cuda")
    table = torch.cat([angle.cos(), angle.sin()], 1)
    kc, vc = g["k"].clone(), g["v"].clone()

    def plan(stream):
        return pkv.tree_plan(g["parents"], g["lens"], g["tables"], nb, bs, 300, stream=stream)

    def rope(stream):
        return [pkv.norm_rope_append(x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:], pos,
                                     table, kc, vc, slots, stream=stream)]

    def attention(stream):
        return [pkv.tree_attention(g["q"], g["k"], g["v"], g["tables"], g["lens"], 300, g["mask"],
                                   scale=c["scale"], stream=stream)]

    def commit(stream):  # (the same rows each time: nothing moves twice)
        return [pkv.tree_commit(kc, vc, g["tables"], g["lens"], t, accepted, counts,
                                stream=stream)]

    need = pkv.tree_attention_workspace_size(2, t, h_q, h_kv, d, bs, 300)
    side = torch.cuda.Stream()
    for call in (plan, rope, attention, commit):
        want = [y.clone() for y in call(None)]
        torch.cuda.synchronize()
        old = [torch.empty_like(y) for y in want for _ in range(3)]
        old += [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda._sleep(50_000_000)
        for y in old:
            y.fill_(7)
        del old, y
        got = call(side)
        side.synchronize()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), call.__name__


@pytest.mark.parametrize("quick", [True, False])
def test_a_context_beyond_the_steps_longest_is_not_committed(quick, monkeypatch):
    """Longer than max_context_len and shorter than the block table: the plan gives its nodes
    no slots and the attention leaves them out, so that the commit has no rows to move."""
    pkv.load()
    if not quick:
        monkeypatch.setattr(pkv, "_quick", None)
    t, cap = 6, 80
    c, accepted, counts = _commit_case(t, [40, 96, 80], [[0, 3, 5], [1, 2], [2]])
    assert 16 * c["tables"].shape[1] > 96
    g, acc, cnt = ref.on_gpu(c), accepted.cuda(), counts.cuda()
    nb = c["k"].shape[0]
    flag = pkv.new_error_flag("cuda")
    slots = pkv.tree_plan(g["parents"], g["lens"], g["tables"], nb, 16, cap, err_flag=flag)[2]
    assert pkv.check_error(flag) == pkv.EFLAG_CONTEXT_LEN
    assert (slots[1] == -1).all() and (slots[[0, 2]] >= 0).all()
    flag.zero_()
    new = torch.empty_like(cnt)
    pkv.tree_commit(g["k"], g["v"], g["tables"], g["lens"], t, acc, cnt, new_context_lens=new,
                    err_flag=flag, max_context_len=cap)
    assert pkv.check_error(flag) == pkv.EFLAG_CONTEXT_LEN
    empty = dict(c, lens=torch.tensor([40, 0, 80], dtype=torch.int32))
    k, v, want = ref.commit(empty, t, accepted, counts)
    want[1] = cap - t
    assert torch.equal(new.cpu(), want) and _same_bits(g["k"], k) and _same_bits(g["v"], v)
    # without it the block table alone bounds a context
    again = ref.on_gpu(c)
    flag.zero_()
    pkv.tree_commit(again["k"], again["v"], again["tables"], again["lens"], t, acc, cnt,
                    new_context_lens=new, err_flag=flag)
    k, v, want = ref.commit(c, t, accepted, counts)
    assert pkv.check_error(flag) == 0
    assert torch.equal(new.cpu(), want) and _same_bits(again["k"], k)
    for bad, error in ((-1, pkv.PkvError), (2 ** 31, ValueError)):
        with pytest.raises(error):
            pkv.tree_commit(g["k"], g["v"], g["tables"], g["lens"], t, acc, cnt,
                            new_context_lens=new, max_context_len=bad)


@pytest.mark.parametrize("quick", [True, False])
def test_a_launch_that_waits_for_the_queue_lets_other_threads_run(quick, monkeypatch):
    """Plans queued behind a kernel of about half a second, more of them than the device's
    queue holds: a thread that ticks every millisecond goes on meanwhile."""
    pkv.load()
    if not quick:
        monkeypatch.setattr(pkv, "_quick", None)
    t = 4
    c, _, _ = _commit_case(t, [40, 90], [[0], [0]])
    g, nb = ref.on_gpu(c), c["k"].shape[0]
    args = (g["parents"], g["lens"], g["tables"], nb, 16, 100)
    outs = pkv.tree_plan(*args)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    torch.cuda._sleep(100_000_000)
    end.record()
    end.synchronize()
    cycles = int(100_000_000 * 500 / start.elapsed_time(end))
    gaps, stop = [], threading.Event()

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now

    thread = threading.Thread(target=tick)
    thread.start()
    begun = time.perf_counter()
    torch.cuda._sleep(cycles)
    for _ in range(6000):
        pkv.tree_plan(*args, *outs)
    queued = time.perf_counter() - begun
    stop.set()
    thread.join()
    torch.cuda.synchronize()
    assert queued > 0.3, "the queue took every launch: nothing was tested"
    assert max(gaps) < 0.15, f"the other thread stood still for {max(gaps):.2f} s"


@pytest.mark.parametrize("key", ["one_tile_d64", "one_tile", "whole_units", "cut", "cut_256_rows",
                                 "three_blocks"])
def test_attention_in_place(key):
    """The output over the queries, where a unit is written at once and where it is cut."""
    c = ref.make_case(len(key), **{
        "one_tile_d64": dict(lens=[20, 33, 9], t=9, h_q=6, h_kv=3, d=64, bs=16, dtype="fp16"),
        "one_tile": dict(lens=[90, 77], t=40, h_q=8, h_kv=1, d=128, bs=16, dtype="bf16"),
        "whole_units": dict(lens=[300] * 40, t=5, h_q=8, h_kv=8, d=128, bs=16, dtype="bf16"),
        "cut": dict(lens=[9000, 40, 2500], t=7, h_q=8, h_kv=2, d=64, bs=32, dtype="bf16"),
        "cut_256_rows": dict(lens=[2000, 130], t=32, h_q=16, h_kv=2, d=128, bs=16, dtype="bf16"),
        "three_blocks": dict(lens=[700, 64], t=48, h_q=8, h_kv=1, d=128, bs=16, dtype="fp16"),
    }[key])
    g = ref.on_gpu(c)
    args = (g["k"], g["v"], g["tables"], g["lens"], c["max_len"], g["mask"])
    want = pkv.tree_attention(g["q"], *args, scale=c["scale"])
    ref.assert_close(want, *ref.attention(c), key)
    q = g["q"].clone()
    assert pkv.tree_attention(q, *args, scale=c["scale"], out=q) is q
    assert _same_bits(q, want)
    both = torch.empty(2 * q.numel() + 8, dtype=q.dtype, device="cuda")
    shifted = both[8:8 + q.numel()].view(q.shape)
    with pytest.raises(pkv.PkvError, match="INVALID_ARG"):
        pkv.tree_attention(both[:q.numel()].view(q.shape), *args, out=shifted)


def test_empty_batches_and_norms_of_one_side():
    t = 5
    c, accepted, counts = _commit_case(t, [40, 30], [[0], [1]])
    g, nb = ref.on_gpu(c), c["k"].shape[0]
    none = pkv.tree_plan(g["parents"][:0], g["lens"][:0], g["tables"][:0], nb, 16, 64)
    assert [tuple(x.shape) for x in none] == [(0, t, 1), (0, t), (0, t)]
    out = pkv.tree_attention(g["q"][:0], g["k"], g["v"], g["tables"][:0], g["lens"][:0], 64,
                             g["mask"][:0])
    assert out.shape == (0, t, 8, 128)
    new = pkv.tree_commit(g["k"], g["v"], g["tables"][:0], g["lens"][:0], t, accepted[:0].cuda(),
                          counts[:0].cuda())
    assert new.shape == (0,)
    x = torch.randn(7, 12, 128, device="cuda").bfloat16()
    w = (1 + 0.1 * torch.randn(128, device="cuda")).bfloat16()
    angle = torch.rand(50, 64, device="cuda")
    table = torch.cat([angle.cos(), angle.sin()], 1)
    pos = torch.arange(7, dtype=torch.int32, device="cuda") * 7
    slots = torch.arange(7, device="cuda") * 3
    for wq, wk in ((w, None), (None, w), (None, None), (w, w)):
        kc, vc = (torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        q = pkv.norm_rope_append(x[:, :8], x[:, 8:10], x[:, 10:], pos, table, kc, vc, slots,
                                 q_weight=wq, k_weight=wk)
        cpu = [y.cpu() if y is not None else None for y in (wq, wk)]
        eq, ek, ev, bq, bk = ref.norm_rope(x[:, :8].cpu(), x[:, 8:10].cpu(), x[:, 10:].cpu(),
                                           pos.cpu(), table.cpu(), *cpu, 1e-6, "half")
        for got, exact, lost in ((q, eq, bq), (kc.view(-1, 2, 128)[slots], ek, bk),
                                 (vc.view(-1, 2, 128)[slots], ev, 0 * ev)):
            off = (got.cpu().double() - exact).abs()
            assert (off <= 2.0 ** -8 * (exact.abs() + lost) + lost).all()


THROWS = """#include <stdexcept>
extern "C" int throws() { throw std::runtime_error("no"); }
"""


def test_an_exception_in_a_call_gives_the_lock_back(tmp_path, monkeypatch):
    """The quick form answers "not mine" and Python's lock is held again: the call in Python
    that follows needs it."""
    lib = pkv.load()
    if pkv._quick is None:
        pytest.skip("built without the headers of Python and torch")
    (tmp_path / "throws.cpp").write_text(THROWS)
    out = str(tmp_path / "throws.so")
    subprocess.run(["g++", "-shared", "-fPIC", "-o", out, str(tmp_path / "throws.cpp")], check=True)
    fake = ctypes.cast(ctypes.CDLL(out).throws, ctypes.c_void_p).value
    real = [ctypes.cast(getattr(lib, "pkv_" + n), ctypes.c_void_p).value
            for n in ("norm_rope_append", "norm_rope_append_fp8", "tree_plan", "tree_attention",
                      "tree_commit_within")]
    c, _, _ = _commit_case(4, [40, 90], [[0], [0]])
    g, nb = ref.on_gpu(c), c["k"].shape[0]
    args = (g["parents"], g["lens"], g["tables"], nb, 16, 100)
    want = pkv.tree_plan(*args)
    outs = [torch.full_like(x, -9) for x in want]
    pkv._quick.bind(*[fake] * 5)
    try:
        assert pkv._quick.tree_plan(*args, *outs, None) is None
        for _ in range(50):
            pkv.tree_plan(*args, *outs)
    finally:
        pkv._quick.bind(*real)
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_outputs_made_on_a_forked_stream_in_a_graph():
    """Captured on a stream that joins the capture, outputs and workspace allocated there;
    other tensors are made and written between the replays."""
    t = 9
    c = ref.make_case(77, [700, 90], t, 8, 2, 128, 16, "bf16")
    g, nb = ref.on_gpu(c), c["k"].shape[0]

    def step(stream):
        mask, pos, slots = pkv.tree_plan(g["parents"], g["lens"], g["tables"], nb, 16, 700,
                                         stream=stream)
        out = pkv.tree_attention(g["q"], g["k"], g["v"], g["tables"], g["lens"], 700, mask,
                                 scale=c["scale"], stream=stream)
        return mask, pos, slots, out

    want = [x.clone() for x in step(None)]
    torch.cuda.synchronize()
    graph, fork = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        fork.wait_stream(torch.cuda.current_stream())
        got = step(fork)
        torch.cuda.current_stream().wait_stream(fork)
    for _ in range(3):
        junk = [torch.full((1 << 16,), 7, dtype=torch.int64, device="cuda") for _ in range(20)]
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all((x == 7).all() for x in junk)
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
