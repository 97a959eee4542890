"""norm_rope_append on the GPU vs a plain 64-bit reference.

The kernel computes in fp32 and rounds once, so an element may be off by half a
step of its type plus the fp32 arithmetic's share (tree_reference.norm_rope).
"""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_164_gb300 as pkv
import tree_reference as ref
from workloads import bits

pytestmark = pytest.mark.gpu

CASES = {
    "one_token": dict(t=1, h_q=8, h_kv=2, d=128),
    "tokens_33_d64": dict(t=33, h_q=4, h_kv=4, d=64, dtype="fp16", layout="hnd"),
    "interleaved": dict(t=70, h_q=8, h_kv=1, d=128, style="interleaved", dtype="fp16", bs=64),
    "interleaved_d64": dict(t=19, h_q=2, h_kv=2, d=64, style="interleaved"),
    "partial_half": dict(t=40, h_q=6, h_kv=2, d=128, rd=32),
    "partial_interleaved": dict(t=40, h_q=6, h_kv=2, d=64, rd=48, style="interleaved",
                                dtype="fp16"),
    "partial_odd_partner": dict(t=9, h_q=2, h_kv=1, d=128, rd=80),
    "no_norm": dict(t=50, h_q=4, h_kv=2, d=128, norm=False, layout="hnd", bs=32),
    "packed": dict(t=61, h_q=10, h_kv=2, d=128, packed=True),
    "one_head": dict(t=5, h_q=1, h_kv=1, d=64, packed=True, bs=128),
    "wide": dict(t=300, h_q=64, h_kv=8, d=128, pads=17),
    "more_tokens_than_65535": dict(t=65600, h_q=1, h_kv=1, d=64, bs=128),
    "mha": dict(t=260, h_q=32, h_kv=32, d=128, dtype="fp16", packed=True, style="interleaved"),
}


def _make(t, h_q, h_kv, d, dtype="bf16", bs=16, layout="nhd", style="half", rd=None, norm=True,
          packed=False, pads=0, seed=1, f8=False):
    g = torch.Generator().manual_seed(seed + t)
    dt = ref.TORCH[dtype]
    rd = rd or d
    x = (torch.randn((t, h_q + 2 * h_kv, d), generator=g) * 2).to(dt)
    wq, wk = (1 + 0.2 * torch.randn((2, d), generator=g)).to(dt) if norm else (None, None)
    npos = 5000
    ang = torch.arange(npos).double()[:, None] * 10000.0 ** (-torch.arange(0, rd, 2).double() / rd)
    nb = (t + bs - 1) // bs + 2
    slots = torch.randperm(nb * bs, generator=g)[:t]
    where = torch.randperm(t, generator=g)[:pads]
    slots[where] = -1
    shape = (nb, bs, h_kv, d) if layout == "nhd" else (nb, h_kv, bs, d)
    fill = torch.full(shape, 0x5A, dtype=torch.uint8) if f8 else \
        torch.full(shape, 0x7E5A, dtype=torch.int16).view(dt)
    return dict(x=x, q=x[:, :h_q], k=x[:, h_q:h_q + h_kv], v=x[:, h_q + h_kv:], wq=wq, wk=wk,
                pos=torch.randint(0, npos, (t,), generator=g, dtype=torch.int32),
                table=torch.cat([ang.cos(), ang.sin()], 1).float(), slots=slots, fill=fill, bs=bs,
                layout=layout, style=style, packed=packed, dt=dt, h_q=h_q, h_kv=h_kv)


def _gpu(c):
    x, h_q, h_kv = c["x"].cuda(), c["h_q"], c["h_kv"]
    q, k, v = x[:, :h_q], x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:]
    if not c["packed"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    w = [None if y is None else y.cuda() for y in (c["wq"], c["wk"])]
    return (q, k, v, c["pos"].cuda(), c["table"].cuda(), c["fill"].cuda(), c["fill"].cuda(),
            c["slots"].cuda()), dict(q_weight=w[0], k_weight=w[1], eps=1e-6, style=c["style"],
                                     layout=c["layout"])


def _slot_rows(cache, c):
    """[nb * bs, H_kv, d] rows by slot."""
    x = cache.cpu()
    if c["layout"] == "hnd":
        x = x.transpose(1, 2)
    return x.reshape(-1, x.shape[2], x.shape[3])


def _near(got, exact, bound, dt, what):
    tol = ref.half_step(dt) * (exact.abs() + bound) + bound + \
        (2.0 ** -25 if dt == torch.float16 else 0.0)  # fp16: half a subnormal step
    err = (got.double() - exact).abs()
    assert (err <= tol).all(), f"{what}: {(err / tol).max():.3f} of the bound"


def _check(c, q_out, kc, vc, live=None):
    live = c["slots"] >= 0 if live is None else live
    pos = torch.where(live, c["pos"], 0)
    eq, ek, ev, bq, bk = ref.norm_rope(c["q"], c["k"], c["v"], pos, c["table"], c["wq"], c["wk"],
                                       1e-6, c["style"])
    s = c["slots"][live]
    _near(q_out.cpu()[live], eq[live], bq[live], c["dt"], "q")
    kr, vr = _slot_rows(kc, c), _slot_rows(vc, c)
    _near(kr[s], ek[live], bk[live], c["dt"], "k")
    assert torch.equal(vr[s].view(torch.int16), c["v"][live].contiguous().view(torch.int16))
    rest = torch.ones(kr.shape[0], dtype=torch.bool)
    rest[s] = False
    for r in (kr, vr):
        assert (r[rest].view(torch.int16) == 0x7E5A).all()


@pytest.mark.parametrize("key", CASES)
def test_matches_the_definition(key):
    c = _make(**CASES[key])
    args, kw = _gpu(c)
    flag = pkv.new_error_flag("cuda")
    q_out = torch.full((c["x"].shape[0], c["h_q"], c["x"].shape[2]), 9.0, dtype=c["dt"],
                       device="cuda")
    assert pkv.norm_rope_append(*args, q_out=q_out, err_flag=flag, **kw) is q_out
    assert pkv.check_error(flag) == 0
    _check(c, q_out, args[5], args[6])
    assert (q_out.cpu()[c["slots"] < 0] == 9.0).all()  # padding is left as it was


@pytest.mark.parametrize("key", ["one_token", "tokens_33_d64", "interleaved", "packed", "wide"])
def test_e4m3_cache(key):
    c = _make(**CASES[key], f8=True)
    args, kw = _gpu(c)
    k_scale, v_scale = 0.011, 0.004  # the second saturates some of V
    flag = pkv.new_error_flag("cuda")
    q_out = pkv.norm_rope_append_fp8(*args, k_scale, v_scale, err_flag=flag, **kw)
    assert pkv.check_error(flag) == 0
    eq, ek, _, bq, bk = ref.norm_rope(c["q"], c["k"], c["v"], c["pos"], c["table"], c["wq"],
                                      c["wk"], 1e-6, c["style"])
    live = c["slots"] >= 0
    s = c["slots"][live]
    _near(q_out.cpu()[live], eq[live], bq[live], c["dt"], "q")
    kr = torch.from_numpy(oracle.decode_e4m3(_slot_rows(args[5], c).numpy()))[s].double()
    want = (ek[live] / k_scale).clamp(-448, 448)
    slack = bk[live] / k_scale + want.abs() * 2.0 ** -23  # the fp32 scale and quotient
    tol = torch.maximum(want.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10)) * (1 + 2.0 ** -10) + slack
    assert ((kr - want).abs() <= tol).all()
    # V's codes are pkv_append_fp8's, bit for bit; the other slots keep their bytes
    ko = np.full(c["fill"].shape if c["layout"] == "nhd" else
                 tuple(c["fill"].transpose(1, 2).shape), 0x5A, dtype=np.uint8)
    vo = ko.copy()
    assert oracle.append_fp8(ko, vo, bits(c["v"]), bits(c["v"]), c["slots"].numpy(), v_scale,
                             v_scale, "fp16" if c["dt"] == torch.float16 else "bf16") == 0
    have = args[6].cpu()
    have = have.transpose(1, 2).contiguous() if c["layout"] == "hnd" else have
    assert np.array_equal(have.numpy(), vo)
    rest = np.ones(_slot_rows(args[5], c).shape[0], dtype=bool)
    rest[s.numpy()] = False
    assert (_slot_rows(args[5], c).numpy()[rest] == 0x5A).all()


def test_in_place_and_on_views():
    c = _make(t=37, h_q=8, h_kv=2, d=128)
    args, kw = _gpu(c)
    want = pkv.norm_rope_append(*args, **kw)
    q = args[0].clone()
    assert pkv.norm_rope_append(q, *args[1:], q_out=q, **kw) is q
    assert torch.equal(q, want)
    # a packed buffer's own q part is not a place to write to: rows have no order
    x = c["x"].cuda()
    with pytest.raises(ValueError, match="contiguous"):
        pkv.norm_rope_append(x[:, :8], *args[1:], q_out=x[:, :8], **kw)
    with pytest.raises(pkv.PkvError, match="INVALID_ARG"):
        pkv.norm_rope_append(x[:, :8], *args[1:], q_out=x.view(-1)[:37 * 8 * 128].view(37, 8, 128),
                             **kw)


@pytest.mark.parametrize("what", ["slot", "position", "negative_position", "both"])
def test_flags_and_skips_bad_indices(what):
    c = _make(t=20, h_q=4, h_kv=2, d=64)
    want, bad = 0, [3, 11]
    if what in ("slot", "both"):
        c["slots"][bad] = c["fill"].shape[0] * 16 + torch.tensor([0, 2 ** 40])
        want |= pkv.EFLAG_SLOT
    if what != "slot":
        c["pos"][bad] = torch.tensor([5000, 2 ** 31 - 1] if what != "negative_position"
                                     else [-1, -2 ** 31], dtype=torch.int32)
        want |= pkv.EFLAG_POSITION
    args, kw = _gpu(c)
    flag = pkv.new_error_flag("cuda")
    q_out = torch.full((20, 4, 64), 9.0, dtype=c["dt"], device="cuda")
    pkv.norm_rope_append(*args, q_out=q_out, err_flag=flag, **kw)
    assert pkv.check_error(flag) == want
    live = torch.ones(20, dtype=torch.bool)
    live[bad] = False
    _check(c, q_out, args[5], args[6], live)
    assert (q_out.cpu()[~live] == 9.0).all()


def test_padding_with_garbage_positions_is_not_read():
    c = _make(t=12, h_q=2, h_kv=1, d=64)
    c["slots"][4:9] = -1
    c["pos"][4:9] = -77
    args, kw = _gpu(c)
    flag = pkv.new_error_flag("cuda")
    q_out = pkv.norm_rope_append(*args, err_flag=flag, **kw)
    assert pkv.check_error(flag) == 0
    _check(c, q_out, args[5], args[6])


def test_zero_rows_and_values_that_are_not_finite():
    c = _make(t=6, h_q=2, h_kv=1, d=128)
    c["x"][0] = 0
    c["x"][1, 0, 5] = float("nan")
    c["x"][2, 2, 7] = float("inf")
    args, kw = _gpu(c)
    q_out = pkv.norm_rope_append(*args, **kw).cpu()
    assert (q_out[0] == 0).all() and (_slot_rows(args[5], c)[c["slots"][0]] == 0).all()
    assert q_out[1, 0].isnan().all() and q_out[1, 1].isfinite().all()  # its own head only
    assert _slot_rows(args[5], c)[c["slots"][2]].isnan().any() and q_out[2].isfinite().all()


def test_strided_and_empty_calls_are_refused_or_do_nothing():
    c = _make(t=8, h_q=4, h_kv=2, d=64)
    args, kw = _gpu(c)
    empty = [a[:0] if i in (0, 1, 2, 3, 7) else a for i, a in enumerate(args)]
    assert pkv.norm_rope_append(*empty, **kw).shape == (0, 4, 64)
    with pytest.raises(ValueError, match="dense"):
        pkv.norm_rope_append(args[0].transpose(0, 1).contiguous().transpose(0, 1), *args[1:], **kw)
    with pytest.raises(TypeError, match="bfloat16"):
        pkv.norm_rope_append(args[0], args[1].half(), *args[2:], **kw)
    with pytest.raises(TypeError, match="int32"):
        pkv.norm_rope_append(*args[:3], args[3].long(), *args[4:], **kw)


def test_on_another_stream():
    c = _make(t=50, h_q=8, h_kv=2, d=128, packed=True)
    args, kw = _gpu(c)
    slots = torch.full_like(args[7], -1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        slots.copy_(args[7])
    q_out = pkv.norm_rope_append(*args[:7], slots, stream=side, **kw)
    junk = torch.full_like(q_out, 7.0)  # the allocator must not hand out the call's output
    side.synchronize()
    _check(c, q_out, args[5], args[6])
    assert (junk == 7).all()


def test_captured_in_a_graph_with_the_append_and_decode_it_replaces():
    """norm_rope_append + decode_attention as one captured step, replayed."""
    c = _make(t=4, h_q=8, h_kv=2, d=128, norm=False)
    args, kw = _gpu(c)
    nb = c["fill"].shape[0]
    kc = torch.randn((nb + 8, 16, 2, 128), device="cuda").bfloat16()
    vc = torch.randn_like(kc)
    tables = torch.randperm(nb + 8, device="cuda")[:8].view(4, 2).to(torch.int32)
    lens = torch.tensor([5, 17, 32, 1], dtype=torch.int32, device="cuda")
    slots = tables.long().gather(1, ((lens - 1) // 16).long()[:, None])[:, 0] * 16 + (lens - 1) % 16
    k0, v0 = kc.clone(), vc.clone()
    rot = pkv.norm_rope_append(*args[:5], args[5], args[6], args[7], **kw)
    k_rot = args[5].view(-1, 2, 128)[args[7]]
    pkv.append(k_rot.contiguous(), args[2], k0, v0, slots)
    want = pkv.decode_attention(rot, k0, v0, tables, lens, 32)

    def step():
        q = pkv.norm_rope_append(*args[:5], kc, vc, slots, **kw)
        return pkv.decode_attention(q, kc, vc, tables, lens, 32)

    keep = (kc.clone(), vc.clone())
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    kc.copy_(keep[0])
    vc.copy_(keep[1])
    graph.replay()
    assert torch.equal(out, want) and torch.equal(kc, k0) and torch.equal(vc, v0)
