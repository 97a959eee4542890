"""Plain 64-bit references of the tree-speculation operators, and their inputs.

Nothing here uses the library: torch on the CPU in float64, token by token.
"""
import math

import torch

ABSENT = -2
TORCH = {"fp16": torch.float16, "bf16": torch.bfloat16}
# What P = hi + lo keeps of a softmax weight: bf16 terms are cut, not rounded
# (2^-7 of a weight each, twice), fp16 terms rounded (2^-11 each).
P_REL = {torch.bfloat16: 2.0 ** -14, torch.float16: 2.0 ** -22}


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def random_parents(t, gen, reach=6, roots=1):
    out = []
    for i in range(t):
        if i < roots:
            out.append(-1)
        else:
            lo = max(0, i - reach)
            out.append(lo + int(torch.randint(0, i - lo, (1,), generator=gen)))
    return out


def plan(parents, context_lens, block_tables, block_size, cap, num_blocks):
    """(mask bits [B, T, T], positions, slots, flags) from the definitions."""
    b, t = parents.shape
    bits = torch.zeros((b, t, t), dtype=torch.bool)
    positions = torch.zeros((b, t), dtype=torch.int32)
    slots = torch.full((b, t), -1, dtype=torch.int64)
    flags = 0
    for s in range(b):
        n = int(context_lens[s])
        if n == 0:
            continue
        n_ok = t <= n <= cap
        if not n_ok:
            flags |= 0x4
        base = max(0, min(n, cap)) - t
        for i in range(t):
            p = int(parents[s, i])
            up, chain, ok = i, [i], True
            while int(parents[s, up]) != -1:
                nxt = int(parents[s, up])
                if nxt < -1 or nxt >= up:
                    ok = False
                    break
                up = nxt
                chain.append(up)
            if not ok:
                if p != ABSENT:
                    flags |= 0x40
                continue
            bits[s, i, chain] = True
            positions[s, i] = max(0, base + len(chain) - 1)
            if n_ok:
                blk = int(block_tables[s, (base + i) // block_size])
                if 0 <= blk < num_blocks:
                    slots[s, i] = blk * block_size + (base + i) % block_size
                else:
                    flags |= 0x1
    return bits, positions, slots, flags


def pack(bits):
    b, t, _ = bits.shape
    words = (t + 31) // 32
    out = torch.zeros((b, t, words), dtype=torch.int64)
    for j in range(t):
        out[:, :, j // 32] |= bits[:, :, j].long() << (j % 32)
    return torch.where(out >= 2 ** 31, out - 2 ** 32, out).to(torch.int32)


def make_case(seed, lens, t, h_q, h_kv, d, bs, dtype, layout="nhd", mask="ancestors",
              spare_pages=2, max_blocks=None, q_scale=1.0):
    """Seeded inputs on the CPU; slots that no sequence holds are NaN.

    lens: positions per sequence, the t nodes' included (0: an empty place).
    """
    g = torch.Generator().manual_seed(seed)
    b = len(lens)
    pages = [(n + bs - 1) // bs for n in lens]
    nb = sum(pages) + spare_pages
    width = max_blocks or max(1, max(pages) + 1)
    pool = torch.randperm(nb, generator=g).tolist()
    tables = torch.full((b, width), -1, dtype=torch.int32)
    held = torch.zeros((nb, bs), dtype=torch.bool)
    for s in range(b):
        for j in range(pages[s]):
            blk = pool.pop()
            tables[s, j] = blk
            held[blk, :min(bs, lens[s] - j * bs)] = True
    dt = TORCH[dtype]
    k = torch.randn((nb, bs, h_kv, d), generator=g).to(dt)
    v = torch.randn((nb, bs, h_kv, d), generator=g).to(dt)
    k[~held] = float("nan")
    v[~held] = float("nan")
    parents = torch.tensor([random_parents(t, g) for _ in range(b)], dtype=torch.int32)
    if mask == "ancestors":
        bits = plan(parents, torch.full((b,), t), torch.zeros((b, 1 + t // bs)), bs, t, 1)[0]
    elif mask == "random":  # any bits, rows of none among them
        bits = torch.rand((b, t, t), generator=g) < 0.4
        bits[:, ::3] = False
    elif mask == "full":
        bits = torch.ones((b, t, t), dtype=torch.bool)
    else:
        raise ValueError(mask)
    return dict(q=(torch.randn((b, t, h_q, d), generator=g) * q_scale).to(dt), k=k, v=v,
                tables=tables, lens=torch.tensor(lens, dtype=torch.int32), bits=bits,
                mask=pack(bits), parents=parents, scale=1.0 / math.sqrt(d), layout=layout, bs=bs,
                held=held, max_len=max(max(lens), 1))


def on_gpu(c):
    """The case's tensors on the GPU, the caches in its layout."""
    out = {n: x.cuda() if isinstance(x, torch.Tensor) else x for n, x in c.items()}
    if c["layout"] == "hnd":
        for n in ("k", "v"):
            out[n] = out[n].transpose(1, 2).contiguous()
    return out


def attention(c, seqs=None, skip_blocks=()):
    """(out, bound) float64 [B, T, H_q, d]: the definition, and how far a kernel may be off.

    The bound: the output's own rounding (half a step), and of
    a = sum_t p_t |v_t| the share that the arithmetic may lose: scores in fp32
    (d products and sums: (d + 2) 2^-24 of sum |q||k|, an absolute error of the
    exponent), exp2 and the rescales (2^-20), the weights' hi + lo terms, and n
    sums in fp32; numerator and denominator alike.
    """
    q, k, v = c["q"].double(), c["k"], c["v"]
    b, t, h_q, d = q.shape
    h_kv = k.shape[2]
    grp = h_q // h_kv
    out = torch.zeros_like(q)
    bound = torch.zeros_like(q)
    half = half_step(c["q"].dtype)
    for s in range(b) if seqs is None else seqs:
        n = int(c["lens"][s])
        if n == 0:
            continue
        base = n - t
        at = torch.arange(n)
        blk = c["tables"][s].long()[at // c["bs"]]
        ok = torch.tensor([int(x) not in skip_blocks for x in blk])
        kk, vv = k[blk, at % c["bs"]].double(), v[blk, at % c["bs"]].double()
        seen = torch.ones((t, n), dtype=torch.bool)
        for p in range(max(0, base), n):
            seen[:, p] = c["bits"][s, :, p - base]
        seen &= ok
        for h in range(h_q):
            g = h // grp
            qs, ks, vs = q[s, :, h], kk[:, g], vv[:, g]
            kz = torch.where(seen.any(0)[:, None], ks, 0.0)
            logit = (qs @ kz.T) * c["scale"]
            size = (qs.abs() @ kz.abs().T) * abs(c["scale"])
            size = torch.where(seen, size, 0.0).amax(1, keepdim=True)
            logit = torch.where(seen, logit, -math.inf)
            any_ = seen.any(1, keepdim=True)
            m = torch.where(any_, logit.amax(1, keepdim=True), 0.0)
            p = torch.exp(logit - m)
            den = p.sum(1, keepdim=True)
            p = torch.where(any_, p / torch.where(any_, den, 1.0), 0.0)
            vz = torch.where(seen.any(0)[:, None], vs, 0.0)
            o = p @ vz
            a = p @ vz.abs()
            lost = a * (2 * ((d + 2) * 2.0 ** -24 * size + 2.0 ** -20 + n * 2.0 ** -24) +
                        P_REL[c["q"].dtype])
            out[s, :, h] = o
            bound[s, :, h] = half * (o.abs() + lost) + lost + 2.0 ** -25
    return out, bound


def assert_close(got, out, bound, what=""):
    g = got.detach().cpu().double()
    assert torch.isfinite(g).all(), f"{what}: non-finite outputs"
    worst = ((g - out).abs() / bound.clamp(min=1e-30)).max().item() if g.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"
    return worst


def norm_rope(q, k, v, positions, cos_sin, q_weight, k_weight, eps, style):
    """(q, k, v, bound of q, bound of k) in float64 before any rounding.

    The bounds: fp32 arithmetic on an element, 16 roundings (2^-24 each) of the
    magnitudes that meet in it: the mean's sum (at most 12 in a chain, halved by
    the root), the root, two products, the rotation's two products and sum.
    """
    half = cos_sin.shape[1] // 2
    table = cos_sin.double()[positions.long()]
    cos, sin = table[:, None, :half], table[:, None, half:]

    def one(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
        y, size = x.clone(), x.abs()
        idx = torch.arange(half)
        a, b = (idx, idx + half) if style == "half" else (2 * idx, 2 * idx + 1)
        y[..., a] = x[..., a] * cos - x[..., b] * sin
        y[..., b] = x[..., b] * cos + x[..., a] * sin
        size[..., a] = (x[..., a] * cos).abs() + (x[..., b] * sin).abs()
        size[..., b] = (x[..., b] * cos).abs() + (x[..., a] * sin).abs()
        return y, 16 * 2.0 ** -24 * size

    yq, bq = one(q, q_weight)
    yk, bk = one(k, k_weight)
    return yq, yk, v.double(), bq, bk


def commit(c, t, accepted, accepted_lens):
    """(k, v, new lengths): the accepted rows moved, one after another."""
    k, v = c["k"].clone(), c["v"].clone()
    new = c["lens"].clone()
    for s in range(len(new)):
        n = int(c["lens"][s])
        if n == 0:
            continue
        base, a = n - t, int(accepted_lens[s])
        rows = []
        for j in range(a):
            p = base + int(accepted[s, j])
            blk, off = int(c["tables"][s, p // c["bs"]]), p % c["bs"]
            rows.append((c["k"][blk, off].clone(), c["v"][blk, off].clone()))
        for j, (kr, vr) in enumerate(rows):
            p = base + j
            blk, off = int(c["tables"][s, p // c["bs"]]), p % c["bs"]
            k[blk, off], v[blk, off] = kr, vr
        new[s] = base + a
    return k, v, new
