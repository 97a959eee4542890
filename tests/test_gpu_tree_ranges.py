"""The tree step's calls over the ranges that they accept: the longest trees and paths, caches
and strides beyond 2^31 elements, E4M3 caches read back, several threads at once (GPU)."""
import threading

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_164_gb300 as pkv
import test_gpu_norm_rope as rope
import tree_reference as ref
from helpers import assert_attention_close
from workloads import bits

pytestmark = pytest.mark.gpu


def _same_bits(a, b):
    return torch.equal(a.cpu().view(torch.int16), b.cpu().view(torch.int16))


# ---------------------------------------------------------------------------
# long trees and paths
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("key", ["one_head", "group16", "any_bits", "d64_hnd"])
def test_attention_of_the_longest_trees(key):
    t = pkv.MAX_TREE_LEN
    c = ref.make_case(81, **{
        "one_head": dict(lens=[t, t + 77], t=t, h_q=1, h_kv=1, d=128, bs=16, dtype="bf16"),
        "group16": dict(lens=[t + 300], t=t, h_q=16, h_kv=1, d=128, bs=32, dtype="bf16"),
        "any_bits": dict(lens=[t + 5, 0, t], t=t, h_q=4, h_kv=2, d=64, bs=128, dtype="fp16",
                         mask="random"),
        "d64_hnd": dict(lens=[t + 130], t=t, h_q=6, h_kv=2, d=64, bs=64, dtype="fp16",
                        layout="hnd"),
    }[key])
    g = ref.on_gpu(c)
    flag = pkv.new_error_flag("cuda")
    out = pkv.tree_attention(g["q"], g["k"], g["v"], g["tables"], g["lens"], c["max_len"],
                             g["mask"], scale=c["scale"], err_flag=flag, layout=c["layout"])
    assert pkv.check_error(flag) == 0
    ref.assert_close(out, *ref.attention(c), key)


@pytest.mark.parametrize("layout,d", [("nhd", 128), ("hnd", 64)])
@pytest.mark.parametrize("t", [200, 257, 1024])
def test_commit_of_paths_longer_than_a_cta(t, layout, d):
    lens = [t, t + 29, t + 300, t + 1]
    c = ref.make_case(t, lens, t, 2, 2, d, 16, "bf16", layout=layout, mask="full")
    paths = [list(range(t)), list(range(1, t, 2)) + ([t - 1] if t % 2 else []),
             [0, 2] + list(range(t - 150, t)), list(range(t - 129, t))]
    most = t
    accepted = torch.tensor([p + [-1] * (most - len(p)) for p in paths], dtype=torch.int32)
    counts = torch.tensor([len(p) for p in paths], dtype=torch.int32)
    g = ref.on_gpu(c)
    flag = pkv.new_error_flag("cuda")
    new = pkv.tree_commit(g["k"], g["v"], g["tables"], g["lens"], t, accepted.cuda(),
                          counts.cuda(), err_flag=flag, layout=layout)
    assert pkv.check_error(flag) == 0
    k, v, want = ref.commit(c, t, accepted, counts)
    assert torch.equal(new.cpu(), want)
    for name, rows in (("k", k), ("v", v)):
        have = g[name].transpose(1, 2).contiguous() if layout == "hnd" else g[name]
        assert _same_bits(have, rows)


@pytest.mark.parametrize("at", [130, 199])
def test_commit_flags_a_break_late_in_a_path(at):
    t = 220
    c = ref.make_case(t, [t + 29, t + 300], t, 2, 2, 64, 16, "fp16", mask="full")
    accepted = torch.arange(10, 210, dtype=torch.int32).repeat(2, 1)
    accepted[1, at] = accepted[1, at - 1]
    counts = torch.tensor([200, 200], dtype=torch.int32)
    g = ref.on_gpu(c)
    flag = pkv.new_error_flag("cuda")
    new = pkv.tree_commit(g["k"], g["v"], g["tables"], g["lens"], t, accepted.cuda(),
                          counts.cuda(), err_flag=flag)
    assert pkv.check_error(flag) == pkv.EFLAG_TREE
    k, v, want = ref.commit(dict(c, lens=torch.tensor([t + 29, 0], dtype=torch.int32)), t,
                            accepted, counts)
    want[1] = 300
    assert torch.equal(new.cpu(), want) and _same_bits(g["k"], k) and _same_bits(g["v"], v)


# ---------------------------------------------------------------------------
# offsets beyond 2^31 elements
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_commit_in_a_cache_beyond_2_31_elements(layout):
    t, bs, h, d = 20, 16, 8, 128
    c = ref.make_case(83, [130, 40], t, h, h, d, bs, "bf16", layout=layout)
    small = ref.on_gpu(c)
    pages = small["k"].shape[0]
    nb = 2 ** 31 // (bs * h * d) + pages
    big = []
    for n in ("k", "v"):
        x = torch.empty((nb, *small[n].shape[1:]), dtype=torch.bfloat16, device="cuda")
        x[nb - pages:] = small[n]
        big.append(x)
    accepted = torch.tensor([[0, 4, 5, 19], [3, 7, 0, 0]], dtype=torch.int32)
    counts = torch.tensor([4, 2], dtype=torch.int32)
    tables = torch.where(small["tables"] >= 0, small["tables"] + (nb - pages), -1).to(torch.int32)
    new = pkv.tree_commit(*big, tables, small["lens"], t, accepted.cuda(), counts.cuda(),
                          layout=layout)
    k, v, want = ref.commit(c, t, accepted, counts)
    assert torch.equal(new.cpu(), want)
    for x, rows in zip(big, (k, v)):
        have = x[nb - pages:]
        assert _same_bits(have.transpose(1, 2).contiguous() if layout == "hnd" else have, rows)


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_norm_rope_append_beyond_2_31_elements(layout, f8):
    """The cache's last pages, and tokens 2^30 elements apart."""
    c = rope._make(t=3, h_q=4, h_kv=2, d=64, layout=layout, f8=f8)
    args, kw = rope._gpu(c)
    stride = 2 ** 30 + 8
    wide = torch.empty(2 * stride + 8 * 64, dtype=c["dt"], device="cuda")
    far = wide.as_strided((3, 8, 64), (stride, 64, 1))
    far.copy_(c["x"].cuda())
    q, k, v = far[:, :4], far[:, 4:6], far[:, 6:]
    small = args[5]
    pages = small.shape[0]
    nb = 2 ** 31 // (16 * 2 * 64) + pages
    caches = [torch.empty((nb, *small.shape[1:]), dtype=small.dtype, device="cuda")
              for _ in "kv"]
    for x in caches:
        x[nb - pages:] = small
    slots = args[7] + (nb - pages) * 16
    if f8:
        want = pkv.norm_rope_append_fp8(*args, 0.02, 0.03, **kw)
        got = pkv.norm_rope_append_fp8(q, k, v, *args[3:5], *caches, slots, 0.02, 0.03, **kw)
    else:
        want = pkv.norm_rope_append(*args, **kw)
        got = pkv.norm_rope_append(q, k, v, *args[3:5], *caches, slots, **kw)
        rope._check(c, want, args[5], args[6])
    assert _same_bits(got, want)
    for x, y in zip(caches, args[5:7]):
        assert torch.equal(x[nb - pages:].contiguous().view(torch.uint8), y.view(torch.uint8))


# ---------------------------------------------------------------------------
# E4M3 caches
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("key", ["partial_half", "partial_interleaved", "partial_odd_partner",
                                 "interleaved_d64", "no_norm", "one_head"])
def test_e4m3_cache_with_other_rotations(key):
    rope.test_e4m3_cache(key)


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_e4m3_append_and_the_decode_that_reads_it(layout):
    """Three steps of one token each: the decode against the oracle on the codes written."""
    b, h_q, h_kv, d, bs, k_scale, v_scale = 4, 8, 2, 128, 16, 0.02, 0.015
    gen = torch.Generator().manual_seed(84)
    lens = torch.tensor([1, 15, 16, 130], dtype=torch.int32)
    tables = torch.randperm(4 * 9, generator=gen).to(torch.int32).view(4, 9)
    shape = (36, bs, h_kv, d) if layout == "nhd" else (36, h_kv, bs, d)
    kc, vc = (torch.randint(0, 120, shape, generator=gen, dtype=torch.uint8).cuda()
              for _ in "kv")
    angle = torch.rand(200, d // 2, generator=gen) * 6
    table = torch.cat([angle.cos(), angle.sin()], 1).cuda()
    weight = (1 + 0.1 * torch.randn(d, generator=gen)).bfloat16().cuda()
    flag = pkv.new_error_flag("cuda")
    for step in range(3):
        x = torch.randn(b, h_q + 2 * h_kv, d, generator=gen).bfloat16().cuda()
        at = (lens - 1).long()
        slots = tables.long().gather(1, at[:, None] // bs)[:, 0] * bs + at % bs
        q = pkv.norm_rope_append_fp8(x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:],
                                     at.to(torch.int32).cuda(), table, kc, vc, slots.cuda(),
                                     k_scale, v_scale, q_weight=weight, k_weight=weight,
                                     err_flag=flag, layout=layout)
        out = pkv.decode_attention_fp8(q, kc, vc, tables.cuda(), lens.cuda(), 140, k_scale,
                                       v_scale, err_flag=flag, layout=layout)
        assert pkv.check_error(flag) == 0
        codes = [(y.transpose(1, 2).contiguous() if layout == "hnd" else y).cpu().numpy()
                 for y in (kc, vc)]
        # the new token's codes are there (checked one by one elsewhere)
        vals = oracle.decode_e4m3(codes[1].reshape(-1, h_kv, d)[slots.numpy()]) * v_scale
        assert np.abs(vals - x[:, h_q + h_kv:].float().cpu().numpy()).max() < 0.3
        expect = oracle.decode_attention_fp8(bits(q), *codes, tables.numpy(), lens.numpy(),
                                             d ** -0.5, k_scale, v_scale, "bf16")
        assert_attention_close(out, expect, f"step {step}")
        lens = lens + 1


# ---------------------------------------------------------------------------
# several threads
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("quick", [True, False])
def test_threads_with_streams_of_their_own(quick, monkeypatch):
    pkv.load()
    if not quick:
        monkeypatch.setattr(pkv, "_quick", None)
    t, wrong = 12, []
    jobs = []
    for i in range(4):
        c = ref.make_case(90 + i, [60 + 200 * i, 300], t, 8, 2, (64, 128)[i % 2], 16,
                          ("fp16", "bf16")[i // 2])
        g = ref.on_gpu(c)
        need = pkv.tree_attention_workspace_size(2, t, 8, 2, g["q"].shape[-1], 16, c["max_len"])
        jobs.append((c, g, torch.empty_like(g["q"]), torch.empty(need, dtype=torch.uint8,
                                                                 device="cuda")))

    def run(c, g, out, ws):
        return pkv.tree_attention(g["q"], g["k"], g["v"], g["tables"], g["lens"], c["max_len"],
                                  g["mask"], scale=c["scale"], out=out, workspace=ws)

    want = [run(*j).clone() for j in jobs]
    torch.cuda.synchronize()
    start = threading.Barrier(len(jobs))

    def work(i):
        c, g, out, ws = jobs[i]
        stream = torch.cuda.Stream()
        start.wait()
        with torch.cuda.stream(stream):
            for _ in range(60):
                out.fill_(float("nan"))
                run(c, g, out, ws)
                mask, pos, _ = pkv.tree_plan(g["parents"], g["lens"], g["tables"],
                                             g["k"].shape[0], 16, c["max_len"])
                stream.synchronize()
                if not _same_bits(out, want[i]) or not torch.equal(mask, g["mask"]):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not wrong
