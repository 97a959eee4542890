"""Cases of the tree-speculation operators over the paged KV cache.

One speculative step of a serving loop drafts a tree of tokens per sequence and
has the large model score all of them in one pass:

  tree_plan         parents of the drafted nodes -> packed ancestor masks,
                    rotary positions and cache slots
  norm_rope_append  per-head norms of queries and keys, the position rotation,
                    and the write of the new keys and values into their slots
                    (16-bit or E4M3 caches)
  tree_attention    every node's queries against the committed context and the
                    node's own ancestors
  tree_commit       the accepted path's cache rows moved to consecutive
                    positions, and the new context lengths

Head counts, page sizes and contexts follow this repository's layer workloads
(Llama-7B: 32/32 heads, Llama-70B: 64/8, the continuous-batching mix: 32/8).

``own`` False: ``run`` computes the plain form in elementary torch operations;
True: it calls the library.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
ABSENT = -2  # parents entry of a node that is not there


def listed():
    return [
        # the plan of one sequence's tree: a latency-bound call
        _plan("plan_one_tree", batch=1, nodes=64, block_size=16, context=(500, 500)),
        # the plans of a full batch of ragged trees
        _plan("plan_batch_256", batch=256, nodes=250, block_size=32, context=(100, 16000), ragged=True),
        # one plain decode step of the Llama-70B layer's batch: 32 tokens
        _norm("rope_decode_32", tokens=32, q_heads=64, kv_heads=8, block_size=16, dtype="bf16"),
        # 32 sequences' trees of 64 nodes into an E4M3 cache, head-major pages
        _norm("rope_trees_e4m3", tokens=2043, q_heads=64, kv_heads=8, block_size=32, dtype="bf16",
              cache="e4m3", layout="hnd", pads=5),
        # a prefill chunk of the Llama-7B layer: packed projections, interleaved
        # pairs, no norm
        _norm("rope_chunk_packed", tokens=16411, q_heads=32, kv_heads=32, block_size=16,
              dtype="fp16", style="interleaved", norm=False, packed=True),
        # the smallest call: two short sequences with four drafted tokens
        _tree("tree_tiny", batch=2, nodes=4, q_heads=4, kv_heads=2, head_dim=64, block_size=16,
              dtype="fp16", context=(34, 47)),
        # the Llama-7B layer (one query head per KV head) verifying 8 tokens
        _tree("tree_mha_8", batch=16, nodes=8, q_heads=32, kv_heads=32, head_dim=128,
              block_size=16, dtype="fp16", context=(512, 4088)),
        # the Llama-70B layer verifying trees of 32 nodes: 256 rows per KV head
        _tree("tree_gqa8_32", batch=32, nodes=32, q_heads=64, kv_heads=8, head_dim=128,
              block_size=16, dtype="bf16", context=(4064, 4064)),
        # the continuous-batching mix, 63 nodes, head-major 32-token pages
        _tree("tree_mix_63", batch=48, nodes=63, q_heads=32, kv_heads=8, head_dim=128,
              block_size=32, dtype="bf16", layout="hnd", context=(300, 9000), ragged=True),
        # long contexts, 16 nodes: 128 rows per KV head
        _tree("tree_long_16", batch=8, nodes=16, q_heads=64, kv_heads=8, head_dim=128,
              block_size=16, dtype="bf16", context=(32768, 131056)),
        # one sequence accepts a few of its drafted tokens
        _commit("commit_one", batch=1, nodes=16, kv_heads=8, block_size=16, dtype="bf16",
                accept=5),
        # a full batch of the Llama-7B layer commits up to 12 of 64 nodes each
        _commit("commit_batch_256", batch=256, nodes=64, kv_heads=32, block_size=16, dtype="fp16",
                accept=12),
    ]


def _plan(name, **kw):
    lo, hi = kw.pop("context")
    return dict(name=name, op="tree_plan", ragged=False, context_lo=lo, context_hi=hi) | kw


def _norm(name, **kw):
    return dict(name=name, op="norm_rope_append", head_dim=128, rotary_dim=128, style="half",
                norm=True, packed=False, cache="16bit", layout="nhd", max_position=131072,
                pads=0) | kw


def _tree(name, **kw):
    lo, hi = kw.pop("context")
    return dict(name=name, op="tree_attention", layout="nhd", ragged=False, context_lo=lo,
                context_hi=hi) | kw


def _commit(name, **kw):
    return dict(name=name, op="tree_commit", head_dim=128, layout="nhd", context_lo=40,
                context_hi=400) | kw


def _between(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree_plan", "norm_rope_append", "norm_rope_append", "tree_attention",
                     "tree_attention", "tree_attention", "tree_commit"])
    block_size = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["fp16", "bf16"])
    layout = rng.choice(["nhd", "hnd"])
    head_dim = rng.choice([64, 128, 128])
    if op == "tree_plan":
        hi = _between(rng, 16, 16000)
        c = _plan("", batch=_between(rng, 1, 256), nodes=_between(rng, 1, 250),
                  block_size=block_size, context=(_between(rng, 1, hi), hi),
                  ragged=rng.random() < 0.5)
    elif op == "norm_rope_append":
        kv = rng.choice([1, 2, 4, 8, 32])
        group = rng.choice([1, 2, 4, 5, 8]) if kv <= 8 else 1
        most = 16411 * 96 // (kv * (group + 2))
        tokens = _between(rng, 1, min(16411, most))
        c = _norm("", tokens=tokens, q_heads=kv * group, kv_heads=kv, block_size=block_size,
                  dtype=dtype, layout=layout, head_dim=head_dim,
                  rotary_dim=rng.choice([head_dim, head_dim, head_dim // 2]),
                  style=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.7,
                  packed=rng.random() < 0.5, cache=rng.choice(["16bit", "16bit", "e4m3"]),
                  pads=rng.choice([0, min(3, tokens - 1)]))
        if c["cache"] == "e4m3":
            c["tokens"] = max(1, min(tokens, 3_000_000 // (kv * head_dim)))
            c["pads"] = min(c["pads"], c["tokens"] - 1)
    elif op == "tree_attention":
        kv = rng.choice([1, 2, 4, 8, 32])
        group = rng.choice([1, 3, 4, 8, 16]) if kv <= 8 else 1
        nodes = _between(rng, 1, 128)
        batch = _between(rng, 1, 64)
        # at most the work of the largest listed case, and plain forms that fit the card
        most = 6.5e8 / (batch * nodes * kv * group)
        most = min(most, 5.2e6 / (batch * kv), 131056)
        hi = _between(rng, 16, max(17, int(most)))
        c = _tree("", batch=batch, nodes=nodes, q_heads=kv * group, kv_heads=kv,
                  head_dim=head_dim, block_size=block_size, dtype=dtype, layout=layout,
                  context=(_between(rng, 1, hi), hi), ragged=rng.random() < 0.5)
    else:
        nodes = _between(rng, 1, 64)
        c = _commit("", batch=_between(rng, 1, 256), nodes=nodes, kv_heads=rng.choice([1, 4, 8]),
                    block_size=block_size, dtype=dtype, layout=layout, head_dim=head_dim,
                    accept=rng.randint(1, min(nodes, 16)))
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lengths(case):
    """Committed tokens per sequence: evenly spread between the case's bounds."""
    b, lo, hi = case["batch"], case["context_lo"], case["context_hi"]
    return [lo + (hi - lo) * i // max(1, b - 1) if b > 1 else hi for i in range(b)]


def _sizes(case):
    """Nodes of each sequence's tree: all of them, or (ragged) from half of them up."""
    b, t = case["batch"], case["nodes"]
    return [max(1, t - i % (t // 2 + 1)) if case.get("ragged") else t for i in range(b)]


def _structure(case, seed):
    """Committed lengths, trees, block tables and pool size: whole numbers, on the host."""
    r = random.Random(seed * 1009 + 7)
    b, t, bs = case["batch"], case["nodes"], case["block_size"]
    committed = _lengths(case)
    sizes = _sizes(case)
    order = list(range(b))
    r.shuffle(order)
    committed, sizes = [committed[i] for i in order], [sizes[i] for i in order]
    parents = []
    for s in sizes:
        # a drafter grows the tree level by level: a node hangs on one of the few before it
        row = [-1] + [r.randrange(max(0, i - 8), i) for i in range(1, s)]
        parents.append(row + [ABSENT] * (t - s))
    pages = [(n + t + bs - 1) // bs for n in committed]
    num_blocks = sum(pages) + 3
    pool = list(range(num_blocks))
    r.shuffle(pool)
    width, at = max(pages) + 1, 0
    tables = []
    for p in pages:
        tables.append(pool[at:at + p] + [-1] * (width - p))
        at += p
    return committed, parents, tables, num_blocks


def _cache(case, num_blocks, gen):
    bs, h, d = case["block_size"], case["kv_heads"], case["head_dim"]
    shape = (num_blocks, bs, h, d) if case["layout"] == "nhd" else (num_blocks, h, bs, d)
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(DTYPES[case["dtype"]])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 3)
    s = {"case": case}

    def ints(v, dtype=torch.int32):
        return torch.tensor(v, dtype=dtype, device="cuda")

    if case["op"] == "norm_rope_append":
        r = random.Random(seed * 1009 + 7)
        t, hq, h, d = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
        dt, bs, rd = DTYPES[case["dtype"]], case["block_size"], case["rotary_dim"]
        if case["packed"]:  # one projection's output, taken apart without a copy
            x = (torch.randn((t, hq + 2 * h, d), generator=gen, device="cuda") * 2).to(dt)
            s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + h], x[:, hq + h:]
        else:
            for name, heads in (("q", hq), ("k", h), ("v", h)):
                s[name] = (torch.randn((t, heads, d), generator=gen, device="cuda") * 2).to(dt)
        s["q_weight"] = s["k_weight"] = None
        if case["norm"]:
            s["q_weight"] = (1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(dt)
            s["k_weight"] = (1 + 0.1 * torch.randn(d, generator=gen, device="cuda")).to(dt)
        angle = torch.arange(case["max_position"], device="cuda", dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, rd, 2, device="cuda", dtype=torch.float64) / rd)
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        first = r.randrange(case["max_position"] - t + 1)
        s["positions"] = torch.arange(first, first + t, device="cuda", dtype=torch.int32)
        num_blocks = (t + bs - 1) // bs + 2
        slots = torch.randperm(num_blocks * bs, generator=gen, device="cuda")[:t]
        if case["pads"]:
            slots[t - case["pads"]:] = -1
        s["slots"] = slots
        shape = (num_blocks, bs, h, d) if case["layout"] == "nhd" else (num_blocks, h, bs, d)
        cdt = torch.uint8 if case["cache"] == "e4m3" else dt
        s["k_cache"] = torch.zeros(shape, dtype=cdt, device="cuda")
        s["v_cache"] = torch.zeros(shape, dtype=cdt, device="cuda")
        s["k_scale"], s["v_scale"] = 6.0 / 448, 9.0 / 448
        s["q_out"] = torch.zeros((t, hq, d), dtype=dt, device="cuda")
        return s

    committed, parents, tables, num_blocks = _structure(case, seed)
    b, t = case["batch"], case["nodes"]
    s["context_lens"] = ints([n + t for n in committed])
    s["block_tables"] = ints(tables)
    s["parents"] = ints(parents)
    s["num_blocks"] = num_blocks
    s["max_context_len"] = case["context_hi"] + t
    if case["op"] == "tree_plan":
        s["mask"] = torch.zeros((b, t, (t + 31) // 32), dtype=torch.int32, device="cuda")
        s["positions"] = torch.zeros((b, t), dtype=torch.int32, device="cuda")
        s["slots"] = torch.zeros((b, t), dtype=torch.int64, device="cuda")
        return s
    s["k_cache"], s["v_cache"] = _cache(case, num_blocks, gen), _cache(case, num_blocks, gen)
    if case["op"] == "tree_attention":
        shape = (b, t, case["q_heads"], case["head_dim"])
        s["q"] = (torch.randn(shape, generator=gen, device="cuda") * 2).to(DTYPES[case["dtype"]])
        s["out"] = torch.zeros_like(s["q"])
        s["scale"] = 1.0 / math.sqrt(case["head_dim"])
        s["mask"] = _pack(_ancestors(s["parents"]))
        return s
    r = random.Random(seed * 1013 + 11)
    accept = [case["accept"] - i % case["accept"] for i in range(b)]
    r.shuffle(accept)
    paths = []
    for a in accept:
        path = [0] + sorted(r.sample(range(1, t), a - 1)) if t > 1 else [0]
        paths.append(path + [-1] * (case["accept"] - len(path)))
    s["accepted"] = ints(paths)
    s["accepted_lens"] = ints(accept)
    s["new_lens"] = torch.zeros_like(s["context_lens"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        import paged_kv_cache_164_gb300 as pkv
        return _OWN[op](pkv, state)
    return _PLAIN[op](state)


def _own_plan(pkv, s):
    pkv.tree_plan(s["parents"], s["context_lens"], s["block_tables"], s["num_blocks"],
                  s["case"]["block_size"], s["max_context_len"], tree_mask=s["mask"],
                  positions=s["positions"], slot_mapping=s["slots"])
    return {"mask": s["mask"], "positions": s["positions"], "slots": s["slots"]}


def _own_norm(pkv, s):
    c = s["case"]
    if c["cache"] == "e4m3":
        pkv.norm_rope_append_fp8(s["q"], s["k"], s["v"], s["positions"], s["cos_sin"],
                                 s["k_cache"], s["v_cache"], s["slots"], s["k_scale"],
                                 s["v_scale"], q_weight=s["q_weight"], k_weight=s["k_weight"],
                                 eps=1e-6, style=c["style"], q_out=s["q_out"], layout=c["layout"])
        e4m3 = torch.float8_e4m3fn
        return {"q": s["q_out"], "k_cache": s["k_cache"].view(e4m3),
                "v_cache": s["v_cache"].view(e4m3)}
    pkv.norm_rope_append(s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["k_cache"],
                         s["v_cache"], s["slots"], q_weight=s["q_weight"],
                         k_weight=s["k_weight"], eps=1e-6, style=c["style"], q_out=s["q_out"],
                         layout=c["layout"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_tree(pkv, s):
    c = s["case"]
    if "workspace" not in s:  # a serving loop keeps its workspace
        need = pkv.tree_attention_workspace_size(c["batch"], c["nodes"], c["q_heads"],
                                                 c["kv_heads"], c["head_dim"], c["block_size"],
                                                 s["max_context_len"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return pkv.tree_attention(s["q"], s["k_cache"], s["v_cache"], s["block_tables"],
                              s["context_lens"], s["max_context_len"], s["mask"],
                              scale=s["scale"], out=s["out"], workspace=s["workspace"],
                              layout=c["layout"])


def _own_commit(pkv, s):
    pkv.tree_commit(s["k_cache"], s["v_cache"], s["block_tables"], s["context_lens"],
                    s["case"]["nodes"], s["accepted"], s["accepted_lens"],
                    new_context_lens=s["new_lens"], layout=s["case"]["layout"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "context_lens": s["new_lens"]}


_OWN = {"tree_plan": _own_plan, "norm_rope_append": _own_norm, "tree_attention": _own_tree,
        "tree_commit": _own_commit}


def _ancestors(parents):
    """[B, T, T] truth values: node j is node i or one of its ancestors; no node that is absent."""
    b, t = parents.shape
    node = torch.arange(t, device=parents.device)
    there = parents != ABSENT
    reach = (parents[:, :, None] == node) | (node[:, None] == node)
    for _ in range((t - 1).bit_length()):  # twice as far up with every product
        reach = reach.float() @ reach.float() > 0
    return reach & there[:, :, None]


def _pack(bits):
    """Truth values [B, T, T] as int32 words [B, T, ceil(T / 32)], bit j % 32 of word j // 32."""
    b, t, _ = bits.shape
    words = (t + 31) // 32
    wide = torch.zeros((b, t, words * 32), dtype=torch.int64, device=bits.device)
    wide[:, :, :t] = bits.long()
    place = 2 ** torch.arange(32, dtype=torch.int64, device=bits.device)
    word = (wide.view(b, t, words, 32) * place).sum(-1)
    return ((word + 2 ** 31) % 2 ** 32 - 2 ** 31).to(torch.int32)


def _unpack(mask, t):
    place = torch.arange(32, dtype=torch.int32, device=mask.device)
    bits = (mask[..., None] >> place) & 1
    return bits.flatten(-2)[..., :t] != 0


def _plain_plan(s):
    bs = s["case"]["block_size"]
    parents, n = s["parents"], s["context_lens"]
    b, t = parents.shape
    reach = _ancestors(parents)
    there = parents != ABSENT
    base = (n - t)[:, None]
    positions = torch.where(there, base + reach.sum(-1) - 1, 0).to(torch.int32)
    at = base + torch.arange(t, device=n.device)
    blocks = torch.gather(s["block_tables"], 1, at // bs).long()
    slots = torch.where(there, blocks * bs + at % bs, -1)
    return {"mask": _pack(reach), "positions": positions, "slots": slots}


def _rotate(x, cos, sin, style):
    """x [T, H, d] with its first 2 * cos.shape[1] dims rotated in pairs."""
    half = cos.shape[1]
    rd = 2 * half
    c, n = cos[:, None], sin[:, None]
    if style == "half":
        a, b = x[..., :half], x[..., half:rd]
        turned = torch.cat([a * c - b * n, b * c + a * n], -1)
    else:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        turned = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    return torch.cat([turned, x[..., rd:]], -1)


def _plain_norm(s):
    c = s["case"]
    bs, half = c["block_size"], c["rotary_dim"] // 2
    at = s["positions"].long()
    cos, sin = s["cos_sin"][at, :half], s["cos_sin"][at, half:]
    made = []
    for x, w in ((s["q"], s["q_weight"]), (s["k"], s["k_weight"])):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        made.append(_rotate(x, cos, sin, c["style"]))
    live = c["tokens"] - c["pads"]
    slots = s["slots"][:live]
    s["q_out"][:live] = made[0][:live].to(s["q_out"].dtype)
    e4m3 = c["cache"] == "e4m3"
    for cache, x, scale in ((s["k_cache"], made[1][:live], s["k_scale"]),
                            (s["v_cache"], s["v"][:live].float(), s["v_scale"])):
        if e4m3:
            x = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            x = x.to(cache.dtype)
        if c["layout"] == "nhd":
            cache[slots // bs, slots % bs] = x
        else:
            cache[slots // bs, :, slots % bs] = x
    if e4m3:
        return {"q": s["q_out"], "k_cache": s["k_cache"].view(torch.float8_e4m3fn),
                "v_cache": s["v_cache"].view(torch.float8_e4m3fn)}
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_tree(s):
    c = s["case"]
    b, t, hq, d = s["q"].shape
    h, n = c["kv_heads"], s["context_lens"]

    def rows(cache):  # [B, H_kv, tokens, d]
        x = cache[s["block_tables"].clamp(min=0).long()]
        x = x.permute(0, 3, 1, 2, 4) if c["layout"] == "nhd" else x.permute(0, 2, 1, 3, 4)
        return x.reshape(b, h, -1, d).float()

    q = s["q"].float().view(b, t, h, hq // h, d).permute(0, 2, 1, 3, 4).reshape(b, h, -1, d)
    scores = (q @ rows(s["k_cache"]).transpose(-1, -2)) * s["scale"]
    at = torch.arange(scores.shape[-1], device=n.device)
    node = at[None] - (n - t)[:, None]  # [B, tokens]: which node a position holds
    seen = torch.gather(_unpack(s["mask"], t), 2,
                        node.clamp(0, t - 1)[:, None].expand(b, t, -1))
    seen = torch.where((node < 0)[:, None], True, seen & (node < t)[:, None])
    seen = seen[:, None, :, None].expand(b, 1, t, hq // h, -1).reshape(b, 1, t * (hq // h), -1)
    scores.masked_fill_(~seen, -math.inf)
    scores -= scores.amax(-1, keepdim=True)
    p = scores.exp_()
    out = (p @ rows(s["v_cache"])) / p.sum(-1, keepdim=True)
    out = out.view(b, h, t, hq // h, d).permute(0, 2, 1, 3, 4).reshape(b, t, hq, d)
    return out.to(s["q"].dtype)


def _plain_commit(s):
    c = s["case"]
    b, t, bs = c["batch"], c["nodes"], c["block_size"]
    base = (s["context_lens"] - t)[:, None]
    node = torch.arange(t, device="cuda")[None]
    path = torch.nn.functional.pad(s["accepted"], (0, t - s["accepted"].shape[1]))
    source = torch.where(node < s["accepted_lens"][:, None], path, node)  # the rest stay

    def places(i):
        at = base + i
        return torch.gather(s["block_tables"], 1, at // bs).long(), at % bs

    (src_block, src_off), (dst_block, dst_off) = places(source), places(node)
    for cache in (s["k_cache"], s["v_cache"]):
        if c["layout"] == "nhd":
            cache[dst_block, dst_off] = cache[src_block, src_off]
        else:
            cache[dst_block, :, dst_off] = cache[src_block, :, src_off]
    s["new_lens"].copy_(s["context_lens"] - t + s["accepted_lens"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "context_lens": s["new_lens"]}


_PLAIN = {"tree_plan": _plain_plan, "norm_rope_append": _plain_norm,
          "tree_attention": _plain_tree, "tree_commit": _plain_commit}


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its exact values
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "tree_plan":
        b, t = case["batch"], case["nodes"]
        words = (t + 31) // 32
        pages = (t + case["block_size"] - 1) // case["block_size"]
        return {"bytes": b * (4 + 4 * t + 4 * pages + t * (4 * words + 4 + 8)), "flops": 0}
    d = case["head_dim"]
    if case["op"] == "norm_rope_append":
        t, hq, h = case["tokens"] - case["pads"], case["q_heads"], case["kv_heads"]
        out = 1 if case["cache"] == "e4m3" else 2
        moved = t * d * (2 * hq * 2 + 2 * h * 2 + 2 * h * out)
        return {"bytes": moved + t * (4 * case["rotary_dim"] + 4 + 8),
                "flops": t * (hq + h) * (4 * d * bool(case["norm"]) + 3 * case["rotary_dim"])}
    b, t, h = case["batch"], case["nodes"], case["kv_heads"]
    if case["op"] == "tree_attention":
        committed = sum(_lengths(case))
        hq, bs = case["q_heads"], case["block_size"]
        tokens = committed + b * t
        moved = tokens * h * d * 2 * 2 + b * t * hq * d * 2 * 2
        moved += tokens // bs * 4 + b * t * ((t + 31) // 32) * 4
        # a node sees the committed context and its few ancestors (itself, at least)
        return {"bytes": moved, "flops": 4 * d * hq * t * (committed + b)}
    moved = sum(case["accept"] - 1 - i % case["accept"] for i in range(b))  # the root stays
    return {"bytes": moved * h * d * 2 * 2 * 2 + b * 12, "flops": 0}


def exact(case, seed):
    """The definitions in 64 bits, token by token and sequence by sequence."""
    if case["op"] == "norm_rope_append":
        return _exact_norm(case, prepare(case, seed))
    if case["op"] == "tree_attention":
        return _exact_tree(case, prepare(case, seed))
    return None  # whole numbers and rows that are moved


def _exact_norm(case, s):
    half, bs = case["rotary_dim"] // 2, case["block_size"]
    i = torch.arange(half, device="cuda")
    first, second = (i, i + half) if case["style"] == "half" else (2 * i, 2 * i + 1)
    table = s["cos_sin"].double()[s["positions"].long()]
    turn = torch.complex(table[:, :half], table[:, half:])[:, None]

    def one(x, w):
        y = x.double()
        if w is not None:
            y = y / (y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + 1e-6).sqrt() * w.double()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    live = s["slots"] >= 0
    q = torch.zeros(s["q_out"].shape, dtype=torch.float64, device="cuda")
    q[live] = one(s["q"], s["q_weight"])[live]
    e4m3 = case["cache"] == "e4m3"
    caches = []
    for x, scale in ((one(s["k"], s["k_weight"]), s["k_scale"]), (s["v"].double(), s["v_scale"])):
        nb = s["k_cache"].shape[0]
        flat = torch.zeros((nb * bs, case["kv_heads"], case["head_dim"]), dtype=torch.float64,
                           device="cuda")
        flat[s["slots"][live]] = (x / scale).clamp(-448, 448)[live] if e4m3 else x[live]
        flat = flat.view(nb, bs, case["kv_heads"], case["head_dim"])
        caches.append(flat if case["layout"] == "nhd" else flat.transpose(1, 2).contiguous())
    return {"q": q, "k_cache": caches[0], "v_cache": caches[1]}


def _exact_tree(case, s):
    b, t, hq, d = s["q"].shape
    h, bs = case["kv_heads"], case["block_size"]
    if 4.0 * d * hq * t * (sum(_lengths(case)) + b * t) > 1.2e12:
        return None
    parents, lens, tables = s["parents"].tolist(), s["context_lens"].tolist(), s["block_tables"]
    out = torch.zeros((b, t, hq, d), dtype=torch.float64, device="cuda")
    for i in range(b):
        n = lens[i]
        at = torch.arange(n, device="cuda")
        block = tables[i].long()[at // bs]
        if case["layout"] == "nhd":
            k, v = s["k_cache"][block, at % bs], s["v_cache"][block, at % bs]
        else:
            k, v = s["k_cache"][block, :, at % bs], s["v_cache"][block, :, at % bs]
        hidden = torch.ones((t, n), dtype=torch.bool)
        hidden[:, :n - t] = False
        for node in range(t):
            up = node if parents[i][node] != ABSENT else -1
            while up >= 0:
                hidden[node, n - t + up] = False
                up = parents[i][up]
        hidden = hidden.cuda()
        for g in range(h):
            heads = slice(g * (hq // h), (g + 1) * (hq // h))
            logits = torch.einsum("thd,nd->thn", s["q"][i, :, heads].double(), k[:, g].double())
            logits = (logits * s["scale"]).masked_fill(hidden[:, None], -math.inf)
            out[i, :, heads] = torch.einsum("thn,nd->thd", torch.softmax(logits, -1),
                                            v[:, g].double())
    return out
