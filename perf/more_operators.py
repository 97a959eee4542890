"""Cases of the operators of a ragged step over the paged KV cache.

A serving loop's step brings a different number of new tokens for every
sequence: chunks of prompts, single tokens, drafted tails.

  batch_plan        request lengths -> pages taken from and given back to the
                    free list, block tables, positions and cache slots
  chunk_attention   the new tokens' queries, packed, against their sequences'
                    pages: causal, with a sliding window, a prefix that every
                    row sees, capped scores and a bias by distance
  verify_drafts     drafted tokens (chains or trees) accepted or rejected by
                    the target's and the draft's probabilities and given random
                    numbers, and the token that follows

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


def listed():
    return [
        # a decode step of a full batch: one new token each, a page now and then
        _plan("plan_decode_256", batch=256, prompts=0, new=(1, 1), past=(100, 16000),
              block_size=16),
        # chunks of prompts beside running and finished sequences
        _plan("plan_prompts_200", batch=200, prompts=24, new=(64, 1311), past=(0, 4000),
              finished=16, block_size=32),
        # the smallest call: two short sequences with a few tokens each
        _chunk("chunk_tiny", batch=2, prompts=2, new=(3, 5), past=(31, 42), q_heads=4, kv_heads=2,
               head_dim=64, block_size=16, dtype="fp16"),
        # single tokens on the Llama-70B layer, capped scores
        _chunk("chunk_decode_64", batch=64, prompts=0, new=(1, 1), past=(1023, 4095), q_heads=64,
               kv_heads=8, block_size=16, dtype="bf16", softcap=30.0),
        # two chunks of prompts among running sequences of the continuous-batching mix
        _chunk("chunk_mixed_32", batch=32, prompts=2, new=(1000, 1048), past=(300, 9000),
               q_heads=32, kv_heads=8, block_size=32, dtype="bf16", layout="hnd"),
        # whole prompts, nothing before them
        _chunk("chunk_prompts_4", batch=4, prompts=4, new=(3500, 4096), past=(0, 0), q_heads=64,
               kv_heads=8, block_size=16, dtype="bf16"),
        # a chunk at the end of a long document
        _chunk("chunk_long_document", batch=1, prompts=1, new=(4096, 4096), past=(61440, 61440),
               q_heads=64, kv_heads=8, block_size=64, dtype="bf16"),
        # the Llama-7B layer (one query head per KV head) with a sliding window
        _chunk("chunk_window_mha", batch=5, prompts=5, new=(900, 2048), past=(0, 6000),
               q_heads=32, kv_heads=32, block_size=16, dtype="fp16", window=1024),
        # prompts with a part that every token sees (an image, instructions), bias by distance
        _chunk("chunk_prefix_bias", batch=12, prompts=10, new=(77, 900), past=(0, 300),
               q_heads=16, kv_heads=4, head_dim=64, block_size=16, dtype="bf16", prefix=257,
               bias=True),
        # one sequence's four drafted tokens
        _verify("verify_chain", batch=1, nodes=5, vocab=32000, tree=False),
        # drafted tails of a batch
        _verify("verify_chains_64", batch=64, nodes=7, vocab=32000, tree=False, ragged=True),
        # trees over a large vocabulary
        _verify("verify_trees_32", batch=32, nodes=16, vocab=128000, tree=True),
    ]


def _plan(name, **kw):
    (new_lo, new_hi), (past_lo, past_hi) = kw.pop("new"), kw.pop("past")
    return dict(name=name, op="batch_plan", new_lo=new_lo, new_hi=new_hi, past_lo=past_lo,
                past_hi=past_hi, finished=0, short=0) | kw


def _chunk(name, **kw):
    (new_lo, new_hi), (past_lo, past_hi) = kw.pop("new"), kw.pop("past")
    return dict(name=name, op="chunk_attention", head_dim=128, layout="nhd", new_lo=new_lo,
                new_hi=new_hi, past_lo=past_lo, past_hi=past_hi, window=0, prefix=0, softcap=0.0,
                bias=False) | kw


def _verify(name, **kw):
    return dict(name=name, op="verify_drafts", ragged=False, draft=True) | kw


def _between(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["batch_plan", "chunk_attention", "chunk_attention", "chunk_attention",
                     "verify_drafts"])
    if op == "batch_plan":
        batch = _between(rng, 1, 256)
        prompts = rng.randint(0, min(batch, 32))
        hi, past = _between(rng, 1, 2000), _between(rng, 1, 16000)
        c = _plan("", batch=batch, prompts=prompts, new=(_between(rng, 1, hi), hi),
                  past=(rng.choice([0, _between(rng, 1, past)]), past),
                  finished=rng.randint(0, (batch - prompts) // 2),
                  short=rng.choice([0, 0, rng.randint(1, 3)]),
                  block_size=rng.choice([16, 32, 64, 128]))
    elif op == "chunk_attention":
        kv = rng.choice([1, 2, 4, 8, 32])
        group = rng.choice([1, 3, 4, 5, 8, 16]) if kv <= 4 else rng.choice([1, 4, 8]) if kv == 8 else 1
        batch = _between(rng, 1, 64)
        prompts = rng.choice([0, min(batch, 1), rng.randint(0, min(batch, 6)), min(batch, 6)])
        hi = _between(rng, 1, 4096)
        # at most the work of the largest listed case, and plain forms that fit the card
        most = min(1.6e10 / (kv * group * (prompts * hi + batch)), 4e9 / (kv * group * hi),
                   4e6 / (batch * kv), 131000)
        past = _between(rng, 1, max(1, int(most)))
        c = _chunk("", batch=batch, prompts=prompts, new=(_between(rng, 1, hi), hi),
                   past=(rng.choice([0, _between(rng, 1, past)]), past), q_heads=kv * group,
                   kv_heads=kv, head_dim=rng.choice([64, 128, 128]),
                   block_size=rng.choice([16, 32, 64, 128]), dtype=rng.choice(["fp16", "bf16"]),
                   layout=rng.choice(["nhd", "hnd"]),
                   window=rng.choice([0, 0, _between(rng, 1, 4096)]),
                   prefix=rng.choice([0, 0, _between(rng, 1, 1000)]),
                   softcap=rng.choice([0.0, 0.0, 30.0, 50.0]), bias=rng.random() < 0.3)
    else:
        vocab = _between(rng, 1000, 128000)
        nodes = _between(rng, 1, 24)
        c = _verify("", batch=min(_between(rng, 1, 128), max(1, int(6.5e7 / (vocab * nodes)))),
                    nodes=nodes, vocab=vocab, tree=rng.random() < 0.5, ragged=rng.random() < 0.5,
                    draft=rng.random() < 0.8)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _spread(lo, hi, count):
    return [lo + (hi - lo) * i // (count - 1) if count > 1 else hi for i in range(count)]


def _lengths(case):
    """(tokens before the step, new tokens) of each sequence, before they are shuffled."""
    b, prompts = case["batch"], case["prompts"]
    new = _spread(case["new_lo"], case["new_hi"], prompts) + [1] * (b - prompts)
    return _spread(case["past_lo"], case["past_hi"], b), new


def _structure(case, seed):
    r = random.Random(seed * 1009 + 7)
    past, new = _lengths(case)
    order = list(range(case["batch"]))
    r.shuffle(past)
    r.shuffle(order)
    return r, past, [new[i] for i in order], order


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _tables(r, pages, spare):
    """Block tables over a shuffled pool, and the pool's unused blocks."""
    num_blocks = sum(pages) + spare
    pool = list(range(num_blocks))
    r.shuffle(pool)
    tables, at = [], 0
    width = max(pages) + 1
    for n in pages:
        tables.append(pool[at:at + n] + [-1] * (width - n))
        at += n
    return tables, pool[at:], num_blocks


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 7919 + 3)
    return {"batch_plan": _prepare_plan, "chunk_attention": _prepare_chunk,
            "verify_drafts": _prepare_verify}[case["op"]](case, seed, gen)


def _prepare_plan(case, seed, gen):
    r, past, new, order = _structure(case, seed)
    bs, b = case["block_size"], case["batch"]
    done = {i for i, o in enumerate(order) if o >= b - case["finished"]}
    new = [0 if i in done else x for i, x in enumerate(new)]
    held = [(n + bs - 1) // bs for n in past]
    more = [(n + a + bs - 1) // bs - h for n, a, h in zip(past, new, held)]
    back = sum(held[i] for i in done)
    # as many free blocks as the step takes and some, or a few too few for its last sequences
    free = max(0, sum(more) - back + (40 if not case["short"] else -case["short"]))
    num_blocks = sum(held) + sum((a + bs - 1) // bs + 1 for a in new) + 40
    tables, pool, _ = _tables(r, held, num_blocks - sum(held))
    width = (case["past_hi"] + case["new_hi"]) // bs + 3
    tables = [row[:width] + [-1] * (width - len(row)) for row in tables]
    tokens = max(1, sum(new))
    tokens = (tokens + 63) // 64 * 64  # a captured step's room
    stack = pool[:free] + [-1] * (num_blocks - free)
    return {"case": case, "context_lens": _ints(past), "new_lens": _ints(new),
            "keep_lens": _ints([0 if i in done else n for i, n in enumerate(past)]),
            "block_tables": _ints(tables), "free_blocks": _ints(stack),
            "free_count": _ints([free]), "num_blocks": num_blocks,
            "max_tokens": tokens,
            "query_starts": _ints([0] * (b + 1)), "positions": _ints([0] * tokens),
            "slots": _ints([0] * tokens, torch.int64), "new_context_lens": _ints([0] * b),
            "new_free_count": _ints([0])}


def _prepare_chunk(case, seed, gen):
    r, past, new, _ = _structure(case, seed)
    bs, h, d, dt = case["block_size"], case["kv_heads"], case["head_dim"], DTYPES[case["dtype"]]
    lens = [n + a for n, a in zip(past, new)]
    tables, _, num_blocks = _tables(r, [(n + bs - 1) // bs for n in lens], 3)
    shape = (num_blocks, bs, h, d) if case["layout"] == "nhd" else (num_blocks, h, bs, d)
    starts = [0]
    for a in new:
        starts.append(starts[-1] + a)
    s = {"case": case, "new": new, "lens": lens, "context_lens": _ints(lens),
         "query_starts": _ints(starts), "block_tables": _ints(tables),
         "max_context_len": max(lens), "scale": 1.0 / math.sqrt(d)}
    for name in ("k_cache", "v_cache"):
        s[name] = torch.randn(shape, generator=gen, device="cuda").to(dt)
    q = torch.randn((starts[-1], case["q_heads"], d), generator=gen, device="cuda") * 2
    s["q"] = q.to(dt)
    s["out"] = torch.zeros_like(s["q"])
    s["slopes"] = s["prefix_lens"] = None
    if case["bias"]:  # a geometric row of slopes, one per query head
        at = torch.arange(1, case["q_heads"] + 1, device="cuda", dtype=torch.float32)
        s["slopes"] = torch.exp2(-8.0 * at / case["q_heads"])
    if case["prefix"]:
        s["prefix_lens"] = _ints([case["prefix"] - i % case["prefix"] // 2 for i in range(len(new))])
    return s


def _nodes(case):
    """Rows of each sequence: all of them, or (ragged) from one up."""
    t = case["nodes"]
    return [t - i % t if case["ragged"] else t for i in range(case["batch"])]


def _prepare_verify(case, seed, gen):
    r = random.Random(seed * 1009 + 7)
    nodes, v = _nodes(case), case["vocab"]
    r.shuffle(nodes)
    starts, parents, rows = [0], [], []
    for n in nodes:
        tree = [-1] + [r.randrange(max(0, (i - 1) // 3), i) if case["tree"] else i - 1
                       for i in range(1, n)]
        rows += [starts[-1] + max(0, p) for p in tree]
        parents += tree
        starts.append(starts[-1] + n)
    total = starts[-1]
    logits = torch.randn((total, v), generator=gen, device="cuda") * 2.5
    p = torch.softmax(logits, -1)
    # a small model's distribution, near the large one's
    q = torch.softmax(logits + torch.randn((total, v), generator=gen, device="cuda"), -1)
    drawn = torch.multinomial(q, 8, replacement=True, generator=gen)
    # every node draws from its parent's row; siblings independently of each other
    order, seen = [], {}
    for row in rows:
        order.append(seen.setdefault(row, 0) % 8)
        seen[row] += 1
    rows = _ints(rows, torch.int64)
    tokens = drawn[rows, _ints(order, torch.int64)].to(torch.int32)
    if not case["draft"]:  # deterministic drafts: the likeliest tokens, siblings the next ones
        tokens = q.topk(8, -1).indices[rows, _ints(order, torch.int64)].to(torch.int32)
    b, most = case["batch"], case["nodes"]
    return {"case": case, "target_probs": p, "draft_probs": q if case["draft"] else None,
            "tokens": tokens, "parents": _ints(parents) if case["tree"] else None,
            "row_starts": _ints(starts), "max_rows": max(nodes),
            "uniforms": torch.rand(total, generator=gen, device="cuda"),
            "context_lens": _ints([100 + 7 * i + n for i, n in enumerate(nodes)]),
            "accepted": _ints([[0] * most] * b), "accepted_lens": _ints([0] * b),
            "next_tokens": _ints([0] * b), "new_context_lens": _ints([0] * b)}


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
    pkv.batch_plan(s["context_lens"], s["new_lens"], s["block_tables"], s["free_blocks"],
                   s["free_count"], s["num_blocks"], s["case"]["block_size"], s["max_tokens"],
                   keep_lens=s["keep_lens"], query_starts=s["query_starts"],
                   positions=s["positions"], slot_mapping=s["slots"],
                   new_context_lens=s["new_context_lens"], new_free_count=s["new_free_count"])
    return _planned(s)


def _planned(s):
    return {n: s[n] for n in ("query_starts", "positions", "slots", "block_tables", "free_blocks",
                              "new_context_lens", "new_free_count")}


def _own_chunk(pkv, s):
    c = s["case"]
    if "workspace" not in s:  # a serving loop keeps its workspace
        need = pkv.chunk_attention_workspace_size(c["batch"], s["q"].shape[0], c["q_heads"],
                                                  c["kv_heads"], c["head_dim"], c["block_size"],
                                                  s["max_context_len"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return pkv.chunk_attention(s["q"], s["k_cache"], s["v_cache"], s["block_tables"],
                               s["query_starts"], s["context_lens"], s["max_context_len"],
                               scale=s["scale"], softcap=c["softcap"], window=c["window"],
                               slopes=s["slopes"], prefix_lens=s["prefix_lens"], out=s["out"],
                               workspace=s["workspace"], layout=c["layout"])


def _own_verify(pkv, s):
    pkv.verify_drafts(s["target_probs"], s["draft_probs"], s["tokens"], s["row_starts"],
                      s["uniforms"], s["accepted"].shape[1], parents=s["parents"],
                      context_lens=s["context_lens"], accepted=s["accepted"],
                      accepted_lens=s["accepted_lens"], next_tokens=s["next_tokens"],
                      new_context_lens=s["new_context_lens"])
    return _verified(s)


def _verified(s):
    return {n: s[n] for n in ("accepted", "accepted_lens", "next_tokens", "new_context_lens")}


_OWN = {"batch_plan": _own_plan, "chunk_attention": _own_chunk, "verify_drafts": _own_verify}


def _plain_plan(s):
    bs = s["case"]["block_size"]
    tables, stack = s["block_tables"], s["free_blocks"]
    up = lambda n: (n + bs - 1) // bs  # noqa: E731
    keep, new = s["keep_lens"].long(), s["new_lens"].long()
    held, kept = up(s["context_lens"].long()), up(keep)
    col = torch.arange(tables.shape[1], device=tables.device)
    # pages behind the kept tokens go onto the stack
    back = held - kept
    at = s["free_count"].long() + (back.cumsum(0) - back)[:, None] + col - kept[:, None]
    gone = (col >= kept[:, None]) & (col < held[:, None])
    room = torch.cat([stack, stack.new_zeros(1)])  # its last place takes what is not written
    room[torch.where(gone, at, stack.numel())] = tables
    stack.copy_(room[:-1])
    top = s["free_count"].long() + back.sum()
    # in order, while pages and tokens last
    need = up(keep + new) - kept
    served = (need.cumsum(0) <= top) & (new.cumsum(0) <= s["max_tokens"])
    need, new = need * served, new * served
    from_top = (need.cumsum(0) - need)[:, None] + col - kept[:, None]
    taken = (col >= kept[:, None]) & (col < (kept + need)[:, None])
    fresh = stack[(top - 1 - from_top).clamp(0, stack.numel() - 1)]
    tables.copy_(torch.where(taken, fresh, tables))
    s["new_free_count"].copy_(top - need.sum())
    s["new_context_lens"].copy_(keep + new)
    ends = new.cumsum(0)
    s["query_starts"][1:] = ends
    token = torch.arange(s["max_tokens"], device=tables.device)
    seq = torch.searchsorted(ends, token, right=True)
    there = seq < ends.numel()
    seq = seq.clamp(max=ends.numel() - 1)
    pos = torch.where(there, keep[seq] + token - (ends - new)[seq], 0)
    s["positions"].copy_(pos)
    s["slots"].copy_(torch.where(there, tables[seq, pos // bs].long() * bs + pos % bs, -1))
    return _planned(s)


def _plain_chunk(s):
    c = s["case"]
    hq, h, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    group = hq // h
    by_length = {}  # sequences with as many new tokens go together
    for i, t in enumerate(s["new"]):
        by_length.setdefault(t, []).append(i)
    for t, seqs in by_length.items():
        b = len(seqs)
        seqs = torch.tensor(seqs, device="cuda")
        longest = max(s["lens"][i] for i in by_length[t])
        tables = s["block_tables"][seqs, :(longest + c["block_size"] - 1) // c["block_size"]]
        tables = tables.clamp(min=0).long()

        def rows(cache):  # [b, H_kv, tokens, d]
            x = cache[tables]
            x = x.permute(0, 3, 1, 2, 4) if c["layout"] == "nhd" else x.permute(0, 2, 1, 3, 4)
            return x.reshape(b, h, -1, d).float()

        new = s["query_starts"].long()[seqs][:, None] + torch.arange(t, device="cuda")
        q = s["q"][new].float().view(b, t, h, group, d).permute(0, 2, 3, 1, 4)
        z = q.reshape(b, h, group * t, d) @ rows(s["k_cache"]).transpose(-1, -2)
        z = z.view(b, h, group, t, -1).mul_(s["scale"])
        if c["softcap"]:
            z.div_(c["softcap"]).tanh_().mul_(c["softcap"])
        n = s["context_lens"][seqs].long()[:, None, None]
        at = torch.arange(z.shape[-1], device="cuda")
        pos = n - t + torch.arange(t, device="cuda")[:, None]
        if s["slopes"] is not None:
            away = (at - pos).float()[:, None, None]
            z.add_(s["slopes"].view(1, h, group, 1, 1) * away)
        seen = at <= pos
        if s["prefix_lens"] is not None:
            seen = seen | (at < torch.minimum(s["prefix_lens"][seqs].long()[:, None, None], n))
        if c["window"]:
            seen = seen & (at > pos - c["window"])
        z.masked_fill_(~seen[:, None, None], -math.inf)
        z.sub_(z.amax(-1, keepdim=True)).exp_()
        total = z.sum(-1).view(b, h, group * t, 1)
        o = (z.view(b, h, group * t, -1) @ rows(s["v_cache"])) / total
        o = o.view(b, h, group, t, d).permute(0, 3, 1, 2, 4)
        s["out"][new] = o.reshape(b, t, hq, d).to(s["out"].dtype)
    return s["out"]


def _plain_verify(s):
    p, tokens, u = s["target_probs"], s["tokens"].long(), s["uniforms"].double()
    first, q = s["row_starts"].long()[:-1], s["draft_probs"]
    count = s["row_starts"].long()[1:] - first
    b = first.numel()
    at = torch.arange(b, device="cuda")
    cur = torch.zeros_like(first)
    left, mass = p[first].double(), torch.ones(b, 1, dtype=torch.float64, device="cuda")
    path, length = s["accepted"].fill_(-1), torch.ones_like(first)
    path[:, 0] = 0
    # a node comes behind its parent, so one walk meets every child of an accepted node
    for i in range(1, s["max_rows"]):
        row = (first + i).clamp(max=tokens.numel() - 1)
        parent = s["parents"][row] if s["parents"] is not None else i - 1
        tried = ((parent == cur) & (i < count))[:, None]
        token = tokens[row][:, None]
        if q is not None:
            draft = q[first + cur].double()
        else:
            draft = torch.zeros_like(left).scatter_(1, token, 1.0)
        taken = tried & (u[row][:, None] * draft.gather(1, token) * mass < left.gather(1, token))
        rest = (left - mass * draft).clamp_(min=0)
        left = torch.where(taken, p[row].double(), torch.where(tried, rest, left))
        mass = torch.where(taken, 1.0, torch.where(tried, rest.sum(1, keepdim=True), mass))
        taken = taken[:, 0]
        cur = torch.where(taken, i, cur)
        path[at, length.clamp(max=path.shape[1] - 1)] = torch.where(
            taken, i, path[at, length.clamp(max=path.shape[1] - 1)]).to(torch.int32)
        length = length + taken
    left = torch.where(left.sum(1, keepdim=True) > 0, left, p[first + cur].double())
    total = left.cumsum(1)
    s["next_tokens"].copy_((total > u[first][:, None] * total[:, -1:]).int().argmax(1))
    s["accepted_lens"].copy_(length)
    s["new_context_lens"].copy_(s["context_lens"] - count + length)
    return _verified(s)


_PLAIN = {"batch_plan": _plain_plan, "chunk_attention": _plain_chunk,
          "verify_drafts": _plain_verify}


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its exact values
# ---------------------------------------------------------------------------

def _limits(case, past, new, prefix):
    """(positions that the new tokens see in all, the union's length) of a sequence."""
    n, w = past + new, case["window"]
    first = max(0, past + 1 - w) if w else 0
    if not w and not prefix:
        return new * past + new * (new + 1) // 2, n
    pos = torch.arange(past, n, dtype=torch.int64)
    hi = torch.maximum(pos + 1, torch.tensor(min(prefix, n)))
    lo = (pos + 1 - w).clamp(min=0) if w else torch.zeros_like(pos)
    return int((hi - lo).clamp(min=0).sum()), int(hi.max()) - first


def work(case):
    if case["op"] == "batch_plan":
        past, new = _lengths(case)
        b, bs = case["batch"], case["block_size"]
        pages = sum(new) // bs  # read from the stack, written into the tables
        return {"bytes": b * 5 * 4 + sum(new) * (4 + 8) + pages * 8, "flops": 0}
    if case["op"] == "verify_drafts":
        # the rows that the next token is drawn from (nearly every sequence ends in a
        # rejection, whose rest takes the target's and the draft's)
        rows = case["batch"] * (2 if case["draft"] and case["nodes"] > 1 else 1)
        return {"bytes": rows * case["vocab"] * 4 + sum(_nodes(case)) * 16, "flops": 0}
    d, hq, h = case["head_dim"], case["q_heads"], case["kv_heads"]
    seen = union = 0
    past, new = _lengths(case)
    for n, a in zip(past, new):
        x, y = _limits(case, n, a, case["prefix"])
        seen, union = seen + x, union + y
    moved = 2 * sum(new) * hq * d * 2 + 2 * union * h * d * 2 + union // case["block_size"] * 4
    return {"bytes": moved, "flops": 4 * d * hq * seen}


def exact(case, seed):
    """The definition in 64 bits, sequence by sequence and head by head."""
    if case["op"] != "chunk_attention" or work(case)["flops"] > 2e12:
        return None  # (whole numbers)
    s = prepare(case, seed)
    hq, h, bs = case["q_heads"], case["kv_heads"], case["block_size"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    starts = s["query_starts"].tolist()
    for i, n in enumerate(s["lens"]):
        t = s["new"][i]
        at = torch.arange(n, device="cuda")
        block = s["block_tables"][i].long()[at // bs]
        if case["layout"] == "nhd":
            k, v = s["k_cache"][block, at % bs], s["v_cache"][block, at % bs]
        else:
            k, v = s["k_cache"][block, :, at % bs], s["v_cache"][block, :, at % bs]
        pos = torch.arange(n - t, n, device="cuda")[:, None]
        hidden = at > pos
        if case["prefix"]:
            hidden &= at >= int(s["prefix_lens"][i])
        if case["window"]:
            hidden |= at <= pos - case["window"]
        for head in range(hq):
            g = head // (hq // h)
            q = s["q"][starts[i]:starts[i + 1], head].double()
            z = torch.einsum("td,nd->tn", q, k[:, g].double()) * s["scale"]
            if case["softcap"]:
                z = torch.tanh(z / case["softcap"]) * case["softcap"]
            if case["bias"]:
                z = z - float(s["slopes"][head]) * (pos - at)
            w = torch.softmax(z.masked_fill(hidden, -math.inf), -1)
            out[starts[i]:starts[i + 1], head] = torch.einsum("tn,nd->td", w, v[:, g].double())
    return out
