"""Refusals of the tree-speculation entry points on the host, before any launch (CPU)."""
import ctypes

import pytest
import torch

import paged_kv_cache_164_gb300 as pkv
from paged_kv_cache_164_gb300 import build as pkv_build

NULL = ctypes.c_void_p(0)
FAKE = ctypes.c_void_p(1 << 20)  # 16-byte aligned, never dereferenced: the call rejects first
ODD = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.load()


def _rope(lib, f8=False, **kw):
    far = [ctypes.c_void_p((i + 2) << 30) for i in range(4)]
    a = dict(out=far[0], q=far[1], qs=8 * 64, k=far[2], ks=2 * 64, v=far[3], vs=2 * 64, wq=FAKE,
             wk=FAKE, eps=1e-6, table=FAKE, npos=100, rd=64, inter=0, pos=FAKE, kc=FAKE, vc=FAKE,
             slots=FAKE, t=4, nb=8, bs=16, hq=8, hkv=2, d=64, sc=(0.1, 0.1), dt=1)
    a.update(kw)
    head = [a[n] for n in ("out", "q", "qs", "k", "ks", "v", "vs", "wq", "wk", "eps", "table",
                           "npos", "rd", "inter", "pos", "kc", "vc", "slots", "t", "nb", "bs",
                           "hq", "hkv", "d")]
    if f8:
        return lib.pkv_norm_rope_append_fp8(*head, *a["sc"], a["dt"], NULL, NULL)
    return lib.pkv_norm_rope_append(*head, a["dt"], NULL, NULL)


@pytest.mark.parametrize("f8", [False, True])
def test_norm_rope_append_refuses(lib, f8):
    for name in ("out", "q", "k", "v", "table", "pos", "kc", "vc", "slots"):
        assert _rope(lib, f8, **{name: NULL}) == 1
    for name in ("out", "q", "k", "v", "wq", "wk", "table", "pos", "kc", "vc", "slots"):
        assert _rope(lib, f8, **{name: ODD}) == 1
    assert _rope(lib, f8, t=-1) == 1 and _rope(lib, f8, nb=0) == 1
    assert _rope(lib, f8, eps=-1.0) == 1 and _rope(lib, f8, eps=float("nan")) == 1
    assert _rope(lib, f8, npos=0) == 1 and _rope(lib, f8, hq=5) == 1 and _rope(lib, f8, dt=2) == 1
    assert _rope(lib, f8, d=96) == 2 and _rope(lib, f8, bs=24) == 2
    for rd in (0, 8, 24, 80):
        assert _rope(lib, f8, rd=rd) == 2
    assert _rope(lib, f8, qs=8 * 64 - 8) == 1 and _rope(lib, f8, ks=2 * 64 + 4) == 1
    assert _rope(lib, f8, vs=64) == 1
    assert _rope(lib, f8, t=0, q=NULL) == 0
    # q_out over q (rows of another stride), k or v
    base = 1 << 31
    at = lambda n: ctypes.c_void_p(base + n)  # noqa: E731
    assert _rope(lib, f8, out=at(0), q=at(0), qs=12 * 64) == 1
    assert _rope(lib, f8, out=at(0), q=at(512)) == 1
    assert _rope(lib, f8, out=at(0), k=at(4 * 8 * 64 * 2 - 16)) == 1
    assert _rope(lib, f8, out=at(256), v=at(0)) == 1
    if f8:
        for bad in (0.0, -1.0, float("inf"), float("nan")):
            assert _rope(lib, True, sc=(bad, 0.1)) == 1 and _rope(lib, True, sc=(0.1, bad)) == 1


def _plan(lib, **kw):
    a = dict(mask=FAKE, pos=FAKE, slots=FAKE, par=FAKE, cl=FAKE, bt=FAKE, mb=4, mcl=64, b=2, t=5,
             nb=8, bs=16)
    a.update(kw)
    return lib.pkv_tree_plan(*[a[n] for n in ("mask", "pos", "slots", "par", "cl", "bt", "mb",
                                              "mcl", "b", "t", "nb", "bs")], NULL, NULL)


def test_tree_plan_refuses(lib):
    for name in ("mask", "pos", "slots", "par", "cl", "bt"):
        assert _plan(lib, **{name: NULL}) == 1 and _plan(lib, **{name: ODD}) == 1
    assert _plan(lib, b=-1) == 1 and _plan(lib, t=0) == 1 and _plan(lib, mb=0) == 1
    assert _plan(lib, mcl=-1) == 1 and _plan(lib, nb=0) == 1 and _plan(lib, bs=0) == 1
    assert _plan(lib, t=1025) == 2 and _plan(lib, bs=48) == 2 and _plan(lib, mb=2 ** 28) == 2
    assert _plan(lib, b=0, par=NULL) == 0


def _attention(lib, **kw):
    a = dict(out=FAKE, q=FAKE, k=FAKE, v=FAKE, bt=FAKE, mb=4, cl=FAKE, mcl=64, mask=FAKE, ms=5,
             b=2, t=5, nb=8, bs=16, hq=8, hkv=2, d=64, scale=0.1, ws=FAKE, wsb=1 << 40, dt=1)
    a.update(kw)
    return lib.pkv_tree_attention(*[a[n] for n in ("out", "q", "k", "v", "bt", "mb", "cl", "mcl",
                                                   "mask", "ms", "b", "t", "nb", "bs", "hq",
                                                   "hkv", "d", "scale", "ws", "wsb", "dt")],
                                  NULL, NULL)


def test_tree_attention_refuses(lib):
    for name in ("out", "q", "k", "v", "bt", "cl", "mask", "ws"):
        assert _attention(lib, **{name: NULL}) == 1 and _attention(lib, **{name: ODD}) == 1
    assert _attention(lib, t=0) == 1 and _attention(lib, b=-1) == 1 and _attention(lib, mb=0) == 1
    assert _attention(lib, hq=7) == 1 and _attention(lib, dt=5) == 1 and _attention(lib, nb=0) == 1
    assert _attention(lib, scale=float("inf")) == 1 and _attention(lib, mcl=-1) == 1
    assert _attention(lib, ms=4) == 1 and _attention(lib, ms=-5) == 1
    assert _attention(lib, d=80) == 2 and _attention(lib, bs=8) == 2 and _attention(lib, hq=34) == 2
    assert _attention(lib, t=1025, ms=0) == 2 and _attention(lib, b=40000) == 2
    assert _attention(lib, mb=2 ** 28) == 2 and _attention(lib, mb=2 ** 27) == 2
    assert _attention(lib, mcl=2 ** 31 - 1) == 2
    assert _attention(lib, b=0, q=NULL) == 0
    size = lib.pkv_tree_attention_workspace_size
    assert size(2, 0, 8, 2, 64, 16, 64) == pkv.SIZE_MAX
    assert size(2, 5, 8, 2, 96, 16, 64) == pkv.SIZE_MAX
    assert size(2, 1025, 8, 2, 64, 16, 64) == pkv.SIZE_MAX
    assert size(2, 5, 8, 2, 64, 16, 2 ** 31 - 1) == pkv.SIZE_MAX


def _commit(lib, **kw):
    a = dict(k=FAKE, v=FAKE, bt=FAKE, mb=4, cl=FAKE, t=5, acc=FAKE, al=FAKE, ma=3,
             new=ctypes.c_void_p(1 << 21), b=2, nb=8, bs=16, hkv=2, d=64, dt=1)
    a.update(kw)
    return lib.pkv_tree_commit(*[a[n] for n in ("k", "v", "bt", "mb", "cl", "t", "acc", "al",
                                                "ma", "new", "b", "nb", "bs", "hkv", "d", "dt")],
                               NULL, NULL)


def test_tree_commit_refuses(lib):
    for name in ("k", "v", "bt", "cl", "acc", "al"):
        assert _commit(lib, **{name: NULL}) == 1 and _commit(lib, **{name: ODD}) == 1
    assert _commit(lib, new=FAKE) == 1                                  # over context_lens
    assert _commit(lib, new=ctypes.c_void_p((1 << 20) + 4)) == 1
    assert _commit(lib, t=0) == 1 and _commit(lib, ma=0) == 1 and _commit(lib, b=-1) == 1
    assert _commit(lib, nb=0) == 1 and _commit(lib, mb=0) == 1 and _commit(lib, dt=9) == 1
    assert _commit(lib, t=1025) == 2 and _commit(lib, bs=20) == 2 and _commit(lib, d=72) == 2
    assert _commit(lib, b=70000) == 2
    assert _commit(lib, b=0, k=NULL) == 0


def test_bindings_refuse_cpu_tensors(lib):
    i = torch.zeros((1, 1), dtype=torch.int32)
    k = torch.zeros((4, 16, 2, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.tree_plan(i, i[0], i, 4, 16, 64)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.tree_attention(k[:1], k, k, i, i[0], 64, i[None])
    with pytest.raises(ValueError, match="CUDA"):
        pkv.tree_commit(k, k, i, i[0], 1, i, i[0])
    with pytest.raises(ValueError, match="CUDA"):
        pkv.norm_rope_append(k[0], k[0], k[0], i[0], k[0], k, k, i[0])


def test_quick_binding_leaves_what_it_does_not_know_to_python(lib):
    if pkv._quick is None:
        pytest.skip("built without the headers of Python and torch")
    i = torch.zeros((1, 1), dtype=torch.int32)
    k = torch.zeros((4, 16, 2, 64), dtype=torch.float16)
    quick = pkv._quick
    for call, n in ((quick.norm_rope_append, 15), (quick.norm_rope_append, 17),
                    (quick.tree_plan, 10), (quick.tree_attention, 12), (quick.tree_commit, 10)):
        for args in ((), (i,) * n, (k,) * n, (k[0],) * n, (None,) * n, (1,) * n, ("nhd",) * n,
                     (object(),) * (n + 1), (i.to_sparse(),) * n, (k.to("meta"),) * n):
            assert call(*args) is None
    with pytest.raises(TypeError):
        quick.bind(1, 2)
    with pytest.raises(ValueError):
        quick.bind(0, 0, 0, 0, 0)
