"""The softmax weights of tree attention as two 16-bit terms, held to what rounded terms keep."""
import math

import pytest
import torch

import paged_kv_cache_164_gb300 as pkv
import tree_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b,t,group", [(32, 1, 1), (4, 20, 8)])
def test_bf16_weights_are_rounded_and_not_cut(b, t, group):
    """32 committed tokens whose weight beside the row's own node, whose weight is 1, is
    (1 + 2^-7 - 2^-20) / 2: its fraction bits from the 8th to the 20th are all set, so a
    bf16 term that is cut, with a second one that is cut, holds 2^-15 of it too little.

    Values lie in [1, 2), so an output may be off by half a step, 2^-8, and by what the
    arithmetic loses of it (below 2): of a weight, whose first term is cut to 8 bits and
    leaves less than 2^-7, the second's rounding, 2^-9 of that: 2^-16; the numerator's 66
    products in fp32 and the denominator's 33 weights (99 * 2^-24); exp2 and its argument,
    of numerator and denominator (4 * 2^-22).  Scores are whole numbers, exact.  Two terms
    that are cut exceed this by 2^-15 * 16.1 / 17.1 - 2^-16 - 2^-17.4 - 2^-20 > 2^-18 of
    the outputs.
    """
    committed, h_kv, d, bs = 32, 8, 128, 16
    c = ref.make_case(7 + t, [committed + t] * b, t, h_kv * group, h_kv, d, bs, "bf16")
    bits = torch.eye(t, dtype=torch.bool).expand(b, t, t).contiguous()
    c |= dict(bits=bits, mask=ref.pack(bits))
    c["q"].zero_()
    c["q"][..., 0] = -1
    for s in range(b):
        for p in range(committed + t):
            blk, off = int(c["tables"][s, p // bs]), p % bs
            c["k"][blk, off] = 0
            c["k"][blk, off, :, 0] = float(p < committed)  # scores -1, and 0 of the nodes
    gen = torch.Generator().manual_seed(11)
    value = 1 + torch.randint(0, 128, c["v"].shape, generator=gen) / 128
    c["v"] = torch.where(c["held"][:, :, None, None], value, math.nan).bfloat16()
    weight = (1 + 2.0 ** -7 - 2.0 ** -20) / 2
    c["scale"] = float(torch.tensor(-math.log(weight), dtype=torch.float32))
    g = ref.on_gpu(c)
    out = pkv.tree_attention(g["q"], g["k"], g["v"], g["tables"], g["lens"], c["max_len"],
                             g["mask"], scale=c["scale"])
    exact, _ = ref.attention(c)
    assert (exact >= 1).all() and (exact < 2).all()
    lost = exact * (2.0 ** -16 + 99 * 2.0 ** -24 + 4 * 2.0 ** -22)
    off = (out.cpu().double() - exact).abs() - (2.0 ** -8 + lost)
    assert (off <= 0).all(), f"{int((off > 0).sum())} of {off.numel()} outputs beyond the bound"
