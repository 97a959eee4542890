"""Plain references of a ragged step's operators, and their inputs.

Nothing here uses the library: Python's whole numbers, and torch on the CPU in
float64, sequence by sequence.
"""
import math
from fractions import Fraction

import torch

TORCH = {"fp16": torch.float16, "bf16": torch.bfloat16}


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


# ---------------------------------------------------------------------------
# batch_plan
# ---------------------------------------------------------------------------

def batch_plan(context, new, tables, free, count, num_blocks, bs, max_tokens, keep=None,
               shared=None):
    """Lists in, a dict of lists out (tables and free are copied), one sequence after another."""
    tables, free = [list(r) for r in tables], list(free)
    b, cap = len(context), (len(tables[0]) if tables else 0) * bs
    keep = list(context) if keep is None else keep
    shared = [0] * b if shared is None else shared
    up = lambda n: -(-n // bs)  # noqa: E731
    flags = 0
    if not 0 <= count <= len(free):
        flags |= 0x100
    top = max(0, min(count, len(free)))
    sound = []
    for s in range(b):
        ok = 0 <= context[s] <= cap and 0 <= keep[s] <= context[s]
        sound.append(ok)
        if not ok:
            flags |= 0x4
            continue
        for j in range(max(up(keep[s]), shared[s]), up(context[s])):
            blk = tables[s][j]
            if not 0 <= blk < num_blocks:
                flags |= 0x1
            if top < len(free):
                free[top] = blk
                top += 1
            else:
                flags |= 0x100
    starts, positions, slots, lens = [0], [], [], []
    pages = tokens = 0
    serving = True
    for s in range(b):
        if not sound[s]:
            lens.append(max(0, min(context[s], cap)))
            starts.append(starts[-1])
            continue
        a = new[s]
        if not 0 <= a <= cap - keep[s]:
            flags |= 0x4
            a = 0
        need = up(keep[s] + a) - up(keep[s])
        if pages + need > top or tokens + a > max_tokens:
            serving = False
        if not serving:
            if a > 0:
                flags |= 0x100
            a = need = 0
        for j in range(need):
            blk = free[top - 1 - pages - j]
            if not 0 <= blk < num_blocks:
                flags |= 0x1
            tables[s][up(keep[s]) + j] = blk
        pages, tokens = pages + need, tokens + a
        for i in range(a):
            p = keep[s] + i
            blk = tables[s][p // bs]
            positions.append(p)
            if not 0 <= blk < num_blocks:
                flags |= 0x1
            slots.append(blk * bs + p % bs if 0 <= blk < num_blocks else -1)
        lens.append(keep[s] + a)
        starts.append(starts[-1] + a)
    spare = max_tokens - len(slots)
    return dict(query_starts=starts, positions=positions + [0] * spare,
                slot_mapping=slots + [-1] * spare, new_context_lens=lens, new_free_count=[top - pages],
                block_tables=tables, free_blocks=free, flags=flags)


# ---------------------------------------------------------------------------
# chunk_attention
# ---------------------------------------------------------------------------

def make_chunk(seed, seqs, h_q, h_kv, d, bs, dtype, layout="nhd", window=0, prefix=None,
               softcap=0.0, bias=False, q_scale=1.0, lead=0, tail=3, spare_pages=2):
    """Seeded inputs on the CPU; cache slots that no sequence holds are NaN.

    seqs: (context, new tokens) of each sequence; lead, tail: rows of q before the
    first and behind the last sequence's.
    """
    g = torch.Generator().manual_seed(seed)
    pages = [(n + bs - 1) // bs for n, _ in seqs]
    nb = sum(pages) + spare_pages
    tables = torch.full((len(seqs), max(1, max(pages) + 1)), -1, dtype=torch.int32)
    pool = torch.randperm(nb, generator=g).tolist()
    held = torch.zeros((nb, bs), dtype=torch.bool)
    for s, (n, _) in enumerate(seqs):
        for j in range(pages[s]):
            blk = pool.pop()
            tables[s, j] = blk
            held[blk, :min(bs, n - j * bs)] = True
    dt = TORCH[dtype]
    k = torch.randn((nb, bs, h_kv, d), generator=g).to(dt)
    v = torch.randn((nb, bs, h_kv, d), generator=g).to(dt)
    k[~held] = float("nan")
    v[~held] = float("nan")
    starts = [lead]
    for _, t in seqs:
        starts.append(starts[-1] + t)
    q = (torch.randn((starts[-1] + tail, h_q, d), generator=g) * q_scale).to(dt)
    slopes = None
    if bias:
        slopes = torch.exp2(-8.0 * torch.arange(1, h_q + 1, dtype=torch.float32) / h_q)
    return dict(q=q, k=k, v=v, tables=tables, starts=torch.tensor(starts, dtype=torch.int32),
                lens=torch.tensor([n for n, _ in seqs], dtype=torch.int32),
                prefix=None if prefix is None else torch.tensor(prefix, dtype=torch.int32),
                slopes=slopes, softcap=softcap, window=window, bs=bs, layout=layout,
                scale=1.0 / math.sqrt(d), max_len=max([1] + [n for n, _ in seqs]))


def on_gpu(c):
    """The case's tensors on the GPU, the caches in its layout."""
    out = {n: x.cuda() if isinstance(x, torch.Tensor) else x for n, x in c.items()}
    if c["layout"] == "hnd":
        for n in ("k", "v"):
            out[n] = out[n].transpose(1, 2).contiguous()
    return out


def attention(c, skip_blocks=()):
    """(out, bound) float64 [T, H_q, d]: the definition, and how far a kernel may be off.
    Rows that no sequence holds are NaN.

    The bound, with w the weights and a = sum w |v|:
      scores: an absolute error dz_t of the exponent of d products and sums in fp32,
        (d + 2) 2^-24 sum |q||k|; the tanh (taken as accurate to 2^-20 of the cap), the
        bias and the sums with it, 4 2^-24 of what meets there; this changes a weight by
        w_t dz_t, the numerator by sum w_t dz_t |v_t|, the denominator by sum w_t dz_t;
      exp2, the rescales and the division: 2^-19 of a; n sums in fp32, twice;
      a weight's rounding to the 16-bit type before it meets V: half a step of it;
      the output's own rounding: half a step.
    """
    q, k, v = c["q"].double(), c["k"].double(), c["v"].double()
    rows, h_q, d = q.shape
    h_kv, bs = k.shape[2], c["bs"]
    out = torch.full_like(q, float("nan"))
    bound = torch.full_like(q, float("nan"))
    half = half_step(c["q"].dtype)
    eps = 2.0 ** -24
    for s in range(len(c["lens"])):
        n, first, end = int(c["lens"][s]), int(c["starts"][s]), int(c["starts"][s + 1])
        t = end - first
        if t <= 0:
            continue
        at = torch.arange(n)
        blk = c["tables"][s].long()[at // bs]
        there = torch.tensor([int(x) not in skip_blocks for x in blk], dtype=torch.bool)
        kk, vv = k[blk.clamp(min=0), at % bs], v[blk.clamp(min=0), at % bs]
        pos = torch.arange(n - t, n)[:, None]
        seen = at <= pos
        if c["prefix"] is not None:
            seen = seen | ((at < int(c["prefix"][s])) & (pos >= 0))
        if c["window"]:
            seen = seen & (at > pos - c["window"])
        seen = seen & there
        for h in range(h_q):
            g = h // (h_q // h_kv)
            # (what no row sees may hold anything)
            some = seen.any(0)[:, None]
            ks, vs = torch.where(some, kk[:, g], 0.0), torch.where(some, vv[:, g], 0.0)
            z = (q[first:end, h] @ ks.T) * c["scale"]
            dz = (d + 2) * eps * (q[first:end, h].abs() @ ks.abs().T) * abs(c["scale"])
            if c["softcap"]:
                z = torch.tanh(z / c["softcap"]) * c["softcap"]
                dz = dz + 2.0 ** -20 * c["softcap"]
            if c["slopes"] is not None:
                far = float(c["slopes"][h]) * (at - pos).double()
                z = z + far
                dz = dz + 4 * eps * far.abs()
            dz = dz + 4 * eps * z.abs()
            z = torch.where(seen, z, -math.inf)
            any_ = seen.any(1, keepdim=True)
            w = torch.exp(z - torch.where(any_, z.amax(1, keepdim=True), 0.0)) if n else z
            den = w.sum(1, keepdim=True)
            w = torch.where(any_, w / torch.where(any_, den, 1.0), 0.0)
            w = torch.where(seen, w, 0.0)
            # a product with a weight of nothing is nothing, whatever the value
            fine = torch.where(torch.isfinite(vs), vs, 0.0)
            o = w @ fine
            a = w @ fine.abs()
            wdz = torch.where(seen, w * dz, 0.0)
            lost = wdz @ fine.abs() + o.abs() * wdz.sum(1, keepdim=True)
            lost = lost + a * (2.0 ** -19 + 2 * n * eps + half)
            if not torch.isfinite(vs).all():
                for i in range(t):
                    x = vs[seen[i]]
                    o[i] = o[i] + torch.where(torch.isfinite(x), 0.0, x).sum(0)
            out[first:end, h] = o
            bound[first:end, h] = half * (o.abs() + lost) + lost + 2.0 ** -25
    return out, bound


def assert_close(got, out, bound, before=None):
    """got against the definition; what is not finite must be the same, and rows that no
    sequence holds what they were before."""
    g = got.detach().cpu()
    rows = torch.isnan(bound).all(-1).all(-1)
    if before is not None:
        assert torch.equal(g[rows].view(torch.int16), before.cpu()[rows].view(torch.int16)), \
            "rows outside the batch changed"
    g, out, bound = g[~rows].double(), out[~rows], bound[~rows]
    if not g.numel():
        return 0.0
    fine = torch.isfinite(out)
    assert torch.equal(torch.isnan(g), torch.isnan(out))
    assert torch.equal(g[~fine & ~torch.isnan(out)], out[~fine & ~torch.isnan(out)])
    err = (g - out).abs()[fine] / bound[fine].clamp(min=1e-30)
    worst = err.max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"{worst:.3f} of the bound"
    return worst


# ---------------------------------------------------------------------------
# verify_drafts
# ---------------------------------------------------------------------------

def _exact(row):
    return [Fraction(x) if 0 < x <= 1 else Fraction(1) if x > 1 else Fraction(0)
            for x in row.tolist()]


def verify(p, q, tokens, starts, u, most, parents=None, context=None):
    """The definition in exact fractions, sequence by sequence."""
    n, vocab = p.shape
    out = dict(accepted=[], accepted_lens=[], next_tokens=[], new_context_lens=[], flags=0)
    top = Fraction(1) - Fraction(1, 2 ** 24)
    uu = [Fraction(0) if not x > 0 else top if x >= 1 else Fraction(x) for x in u.tolist()]
    for s in range(len(starts) - 1):
        first, count = int(starts[s]), int(starts[s + 1]) - int(starts[s])
        path, token = [], -1
        if first < 0 or count < 0 or first + count > n or count > 1024:
            out["flags"] |= 0x80
            count = 0
        if count > 0:
            row = lambda i: _exact(p[first + i])  # noqa: E731
            cur, left, mass, path = 0, row(0), Fraction(1), [0]
            for i in range(1, count):
                par = i - 1 if parents is None else int(parents[first + i])
                x = int(tokens[first + i])
                if not 0 <= par < i and par not in (-1, -2):
                    out["flags"] |= 0x40
                if not 0 <= x < vocab:
                    out["flags"] |= 0x200
                    continue
                if par != cur or len(path) >= most or not 0 <= par < i:
                    continue
                draft = _exact(q[first + cur]) if q is not None else \
                    [Fraction(int(k == x)) for k in range(vocab)]
                if uu[first + i] * draft[x] * mass < left[x]:
                    cur, left, mass = i, row(i), Fraction(1)
                    path.append(i)
                else:
                    left = [max(a - mass * d, Fraction(0)) for a, d in zip(left, draft)]
                    mass = sum(left)
            if sum(left) == 0:
                left = row(cur)
            total = sum(left)
            if total == 0:
                out["flags"] |= 0x200
            else:
                aim, run = uu[first] * total, Fraction(0)
                for k in range(vocab):
                    run += left[k]
                    if run > aim:
                        token = k
                        break
        out["accepted"].append(path + [-1] * (most - len(path)))
        out["accepted_lens"].append(len(path))
        out["next_tokens"].append(token)
        if context is not None:
            out["new_context_lens"].append(int(context[s]) - count + len(path))
    return out
