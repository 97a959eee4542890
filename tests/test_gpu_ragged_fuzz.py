"""Seeded cases of the ragged step's attention over its whole range against the definition in
64 bits (GPU): what no other test puts together."""
import random

import pytest
import torch

import paged_kv_cache_164_gb300 as pkv
import ragged_reference as ref

pytestmark = pytest.mark.gpu


def _drawn(seed):
    r = random.Random(seed)
    h_kv = r.choice([1, 1, 2, 3, 4])
    group = r.choice([1, 2, 3, 4, 5, 7, 8, 11, 16])
    d, bs = r.choice([64, 128]), r.choice([16, 32, 64, 128])
    seqs = []
    for _ in range(r.choice([1, 2, 5, 9, 40])):
        t = r.choice([0, 1, 1, 1, 2, r.randint(1, 9), r.randint(1, 70)])
        if r.random() < 0.15 and len(seqs) < 8:
            t = r.randint(60, 260)
        past = r.choice([0, 0, r.randint(0, 40), r.randint(0, 300), r.randint(0, 1500)])
        seqs.append((past + t, t))
    n_max = max(n for n, _ in seqs)
    window = r.choice([0, 0, 0, 1, r.randint(1, 200), r.randint(1, 2 * n_max + 1)])
    prefix = [r.choice([-1, 0, n // 2, n - t, n, n + 50]) for n, t in seqs] \
        if r.random() < 0.3 else None
    c = ref.make_chunk(seed, seqs, h_kv * group, h_kv, d, bs, r.choice(["fp16", "bf16"]),
                       r.choice(["nhd", "hnd"]), window=window, prefix=prefix,
                       softcap=r.choice([0.0, 0.0, 0.0, 8.0, 50.0]), bias=r.random() < 0.25,
                       q_scale=r.choice([0.1, 1.0, 1.0, 4.0]), lead=r.choice([0, 0, 3]),
                       tail=r.choice([0, 1, 20]))
    c["scale"] *= r.choice([1.0, 1.0, 1.0, 0.5, -1.0])
    c["max_len"] = r.choice([c["max_len"], c["max_len"], 5000])
    return c


@pytest.mark.parametrize("seed", range(48))
def test_drawn_cases(seed):
    c = _drawn(1000 + seed)
    out, bound = ref.attention(c)
    g = ref.on_gpu(c)
    before = torch.full_like(g["q"], 7.0)
    got = before.clone()
    flag = pkv.new_error_flag("cuda")
    pkv.chunk_attention(g["q"], g["k"], g["v"], g["tables"], g["starts"], g["lens"], g["max_len"],
                        scale=g["scale"], softcap=g["softcap"], window=g["window"],
                        slopes=g["slopes"], prefix_lens=g["prefix"], out=got, layout=g["layout"],
                        err_flag=flag)
    assert pkv.check_error(flag) == 0
    ref.assert_close(got, out, bound, before)
