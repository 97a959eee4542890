"""Outputs of the tree step's calls that lie over what the call reads are refused before any
launch (CPU): the CTAs of a sequence have no order among them."""
import ctypes

import pytest

import paged_kv_cache_164_gb300 as pkv
from paged_kv_cache_164_gb300 import build as pkv_build

NULL = ctypes.c_void_p(0)


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.load()


def _at(place, offset=0):
    """Addresses a gigabyte apart that nothing dereferences."""
    return ctypes.c_void_p((place + 1 << 30) + offset)


B, T, WIDTH, MOST, NB, BS, H_KV, D = 3, 5, 4, 3, 8, 16, 2, 64
CACHE = NB * BS * H_KV * D * 2
COMMIT = {"k": (0, CACHE), "v": (1, CACHE), "tables": (2, B * WIDTH * 4), "lens": (3, B * 4),
          "accepted": (4, B * MOST * 4), "counts": (5, B * 4)}


def _commit(lib, new):
    k, v, tables, lens, accepted, counts = (_at(i) for i in range(6))
    return lib.pkv_tree_commit(k, v, tables, WIDTH, lens, T, accepted, counts, MOST, new, B, NB,
                               BS, H_KV, D, 1, NULL, NULL)


PLAN_IN = {"parents": (3, B * T * 4), "lens": (4, B * 4), "tables": (5, B * WIDTH * 4)}
PLAN_OUT = {"mask": (0, B * T * 4), "positions": (1, B * T * 4), "slots": (2, B * T * 8)}


@pytest.mark.parametrize("name", PLAN_IN)
@pytest.mark.parametrize("out", PLAN_OUT)
def test_plan_refuses_outputs_over_what_it_reads(lib, out, name):
    place, size = PLAN_IN[name]
    for offset in (0, (size - 4) // 8 * 8, -((PLAN_OUT[out][1] - 4) // 8 * 8)):
        mask, positions, slots = (_at(place, offset) if n == out else _at(at)
                                  for n, (at, _) in PLAN_OUT.items())
        parents, lens, tables = (_at(at) for at, _ in PLAN_IN.values())
        assert lib.pkv_tree_plan(mask, positions, slots, parents, lens, tables, WIDTH, 64, B, T,
                                 NB, BS, NULL, NULL) == 1


@pytest.mark.parametrize("name", COMMIT)
def test_commit_refuses_new_lengths_over_what_it_reads(lib, name):
    place, size = COMMIT[name]
    for offset in (0, size - 4, -4 * (B - 1)):
        assert _commit(lib, _at(place, offset)) == 1


TOKENS, H_Q, NPOS = 4, 6, 100
ROPE = {"q": (1, TOKENS * H_Q * D * 2), "k": (2, TOKENS * H_KV * D * 2),
        "v": (3, TOKENS * H_KV * D * 2), "q_weight": (4, D * 2), "k_weight": (5, D * 2),
        "cos_sin": (6, NPOS * D * 4), "positions": (7, TOKENS * 4), "k_cache": (8, CACHE),
        "v_cache": (9, CACHE), "slots": (10, TOKENS * 8)}


@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("name", ROPE)
def test_norm_rope_append_refuses_its_output_over_what_it_reads(lib, name, f8):
    place, size = ROPE[name]
    if f8 and "cache" in name:
        size //= 2
    q, k, v, wq, wk, table, pos, kc, vc, slots = (_at(i) for i in range(1, 11))
    before = TOKENS * H_Q * D * 2 - 16
    for offset in ([0] if name != "q" else []) + [16 * ((size - 1) // 16), -before]:
        head = (_at(place, offset), q, H_Q * D, k, H_KV * D, v, H_KV * D, wq, wk, 1e-6, table,
                NPOS, D, 0, pos, kc, vc, slots, TOKENS, NB, BS, H_Q, H_KV, D)
        if f8:
            assert lib.pkv_norm_rope_append_fp8(*head, 0.1, 0.1, 1, NULL, NULL) == 1
        else:
            assert lib.pkv_norm_rope_append(*head, 1, NULL, NULL) == 1


Q_BYTES = B * T * H_Q * D * 2
ATTENTION = {"q": (1, Q_BYTES), "k": (2, CACHE), "v": (3, CACHE), "tables": (4, B * WIDTH * 4),
             "lens": (5, B * 4), "mask": (6, 4 * ((B - 1) * 9 + T))}


@pytest.mark.parametrize("name", ATTENTION)
def test_attention_refuses_its_output_over_what_it_reads(lib, name):
    place, size = ATTENTION[name]
    q, k, v, tables, lens, mask, ws = (_at(i) for i in range(1, 8))
    for offset in ([0] if name != "q" else []) + [16 * ((size - 1) // 16), -(Q_BYTES - 16)]:
        assert lib.pkv_tree_attention(_at(place, offset), q, k, v, tables, WIDTH, lens, 64, mask,
                                      9, B, T, NB, BS, H_Q, H_KV, D, 0.1, ws, 1 << 29, 1, NULL,
                                      NULL) == 1
