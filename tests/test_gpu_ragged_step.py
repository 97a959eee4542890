"""A ragged step as a serving loop runs it: the plan takes pages, the new tokens' K and V are
appended, they attend, the drafts among them are verified, and the next plan keeps what was
accepted (GPU)."""
import pytest
import torch

import paged_kv_cache_164_gb300 as pkv
import ragged_reference as ref

pytestmark = pytest.mark.gpu

H_Q, H_KV, D, BS, VOCAB, MOST = 8, 2, 64, 16, 257, 6


class _Loop:
    """The buffers of a loop over b sequences and its one step, which neither allocates nor
    reads anything back: a step's inputs are written into the buffers before it."""

    def __init__(self, b, room, max_tokens, dtype=torch.bfloat16):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.b, self.room, self.max_tokens = b, room, max_tokens
        self.blocks = b * room // BS
        self.context = torch.zeros(b, **i32)
        self.keep = torch.zeros(b, **i32)
        self.new = torch.zeros(b, **i32)
        self.tables = torch.full((b, room // BS), -1, **i32)
        self.free = torch.arange(self.blocks, **i32).flip(0).contiguous()
        self.count = torch.tensor([self.blocks], **i32)
        self.starts = torch.zeros(b + 1, **i32)
        self.positions = torch.zeros(max_tokens, **i32)
        self.slots = torch.zeros(max_tokens, dtype=torch.int64, device="cuda")
        shape = (self.blocks, BS, H_KV, D)
        self.k, self.v = (torch.full(shape, float("nan"), dtype=dtype, device="cuda")
                          for _ in "kv")
        self.qkv = torch.zeros(max_tokens, H_Q + 2 * H_KV, D, dtype=dtype, device="cuda")
        angles = torch.rand(room, D // 2, generator=torch.Generator().manual_seed(1)) * 6
        self.cos_sin = torch.cat([angles.cos(), angles.sin()], 1).cuda()
        self.q = torch.zeros(max_tokens, H_Q, D, dtype=dtype, device="cuda")
        self.out = torch.zeros_like(self.q)
        self.workspace = torch.empty(pkv.chunk_attention_workspace_size(
            b, max_tokens, H_Q, H_KV, D, BS, room), dtype=torch.uint8, device="cuda")
        self.p = torch.zeros(max_tokens, VOCAB, device="cuda")
        self.p_draft = torch.zeros(max_tokens, VOCAB, device="cuda")
        self.tokens = torch.zeros(max_tokens, **i32)
        self.uniforms = torch.zeros(max_tokens, device="cuda")
        self.accepted = torch.zeros(b, MOST, **i32)
        self.accepted_lens = torch.zeros(b, **i32)
        self.next = torch.zeros(b, **i32)
        self.flag = pkv.new_error_flag("cuda")

    def step(self):
        pkv.batch_plan(self.context, self.new, self.tables, self.free, self.count, self.blocks,
                       BS, self.max_tokens, keep_lens=self.keep, query_starts=self.starts,
                       positions=self.positions, slot_mapping=self.slots,
                       new_context_lens=self.context, new_free_count=self.count,
                       err_flag=self.flag)
        q, k, v = self.qkv.split([H_Q, H_KV, H_KV], 1)
        pkv.norm_rope_append(q, k, v, self.positions, self.cos_sin, self.k, self.v, self.slots,
                             q_out=self.q, err_flag=self.flag)
        pkv.chunk_attention(self.q, self.k, self.v, self.tables, self.starts, self.context,
                            self.room, out=self.out, workspace=self.workspace,
                            err_flag=self.flag)
        pkv.verify_drafts(self.p, self.p_draft, self.tokens, self.starts, self.uniforms, MOST,
                          context_lens=self.context, accepted=self.accepted,
                          accepted_lens=self.accepted_lens, next_tokens=self.next,
                          new_context_lens=self.keep, err_flag=self.flag)

    def feed(self, g, new):
        """Seeded inputs of a step of `new` tokens of each sequence."""
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        rows = self.max_tokens
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=g))
        logits = torch.randn(rows, VOCAB, generator=g) * 2
        draft = torch.softmax(logits + torch.randn(rows, VOCAB, generator=g) * 0.5, -1)
        self.p.copy_(torch.softmax(logits, -1))
        self.p_draft.copy_(draft)
        tokens = torch.multinomial(draft, 1, generator=g).view(-1).roll(1).int()
        self.tokens.copy_(tokens)
        self.uniforms.copy_(torch.rand(rows, generator=g))

    def state(self):
        return {n: x.clone() for n, x in vars(self).items() if isinstance(x, torch.Tensor)}


# new tokens of each sequence, step by step: prompts, then drafts of several lengths, a
# sequence that waits, one that takes a second chunk of its prompt meanwhile
STEPS = [[150, 40, 0, 1], [5, 6, 130, 3], [1, 4, 2, 0], [6, 1, 5, 200], [2, 2, 2, 2]]


def _check(loop, before, new):
    plan = ref.batch_plan(before["context"].tolist(), new, before["tables"].tolist(),
                          before["free"].tolist(), int(before["count"]), loop.blocks, BS,
                          loop.max_tokens, keep=before["keep"].tolist())
    assert plan["flags"] == 0 == pkv.check_error(loop.flag)
    for name, got in (("query_starts", loop.starts), ("positions", loop.positions),
                      ("slot_mapping", loop.slots), ("new_context_lens", loop.context),
                      ("new_free_count", loop.count), ("block_tables", loop.tables),
                      ("free_blocks", loop.free)):
        assert got.tolist() == plan[name], name
    c = dict(q=loop.q.cpu(), k=loop.k.cpu(), v=loop.v.cpu(), tables=loop.tables.cpu(),
             starts=loop.starts.cpu(), lens=loop.context.cpu(), prefix=None, slopes=None,
             softcap=0.0, window=0, bs=BS, layout="nhd", scale=D ** -0.5)
    ref.assert_close(loop.out, *ref.attention(c), before["out"])
    told = ref.verify(loop.p.cpu(), loop.p_draft.cpu(), loop.tokens.cpu(), loop.starts.cpu(),
                      loop.uniforms.cpu(), MOST, None, loop.context.cpu())
    assert loop.accepted.tolist() == told["accepted"]
    assert loop.accepted_lens.tolist() == told["accepted_lens"]
    assert loop.next.tolist() == told["next_tokens"]
    assert loop.keep.tolist() == told["new_context_lens"]


def _prompt_keeps_all(loop):
    # (a chunk of a prompt is no draft: the loop keeps all of it)
    long = loop.new > MOST
    loop.keep.copy_(torch.where(long, loop.context, loop.keep))


def test_steps_against_the_definitions_and_in_a_captured_graph():
    g = torch.Generator().manual_seed(21)
    loop = _Loop(4, 512, 400)
    states = []
    for new in STEPS:
        loop.feed(g, new)
        before = loop.state()
        loop.step()
        _check(loop, before, new)
        states.append(loop.state())
        _prompt_keeps_all(loop)
    # the same steps as one graph that is replayed
    g = torch.Generator().manual_seed(21)
    again = _Loop(4, 512, 400)
    again.step()  # (no tokens: nothing changes)
    assert pkv.check_error(again.flag) == 0 and int(again.count) == again.blocks
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again.step()
    for new, expect in zip(STEPS, states):
        again.feed(g, new)
        graph.replay()
        torch.cuda.synchronize()
        got = again.state()
        got.pop("workspace")
        for name, x in got.items():
            assert torch.equal(x.cpu().view(torch.uint8), expect[name].cpu().view(torch.uint8)), name
        _prompt_keeps_all(again)
    assert pkv.check_error(again.flag) == 0


def test_a_sequence_that_finds_no_pages_leaves_its_rows_alone():
    loop = _Loop(2, 64, 80)
    g = torch.Generator().manual_seed(3)
    loop.count.fill_(2)  # pages for 32 tokens
    loop.feed(g, [30, 20])
    loop.out.fill_(7.0)
    loop.step()
    assert pkv.check_error(loop.flag) == pkv.EFLAG_POOL
    assert loop.context.tolist() == [30, 0] and loop.starts.tolist() == [0, 30, 30]
    assert (loop.out[30:] == 7.0).all() and not (loop.out[:30] == 7.0).all()
    assert loop.accepted_lens.tolist()[1] == 0 and loop.keep.tolist()[1] == 0


def test_a_line_of_several_rounds():
    """One sequence whose units fill two rounds of segments: rows here and there against the
    definition in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(4)
    n, t, h_q, d = 66000, 9000, 8, 64
    pages = (n + 127) // 128
    k = torch.randn(pages, 128, 1, d, generator=g, device="cuda").half()
    v = torch.randn(pages, 128, 1, d, generator=g, device="cuda").half()
    q = torch.randn(t, h_q, d, generator=g, device="cuda").half()
    tables = torch.randperm(pages, generator=torch.Generator().manual_seed(4)).int().cuda()[None]
    starts = torch.tensor([0, t], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    flag = pkv.new_error_flag("cuda")
    out = pkv.chunk_attention(q, k, v, tables, starts, lens, n, err_flag=flag)
    assert pkv.check_error(flag) == 0
    rows = torch.tensor([0, 1, 31, 32, 1000, 2047, 2048, 6333, t - 33, t - 1])
    order = tables[0].long()
    kk = k[order].view(-1, d)[:n].double()
    vv = v[order].view(-1, d)[:n].double()
    half, eps = ref.half_step(torch.float16), 2.0 ** -24
    for i in rows.tolist():
        z = q[i].double() @ kk.T * d ** -0.5
        z[:, n - t + i + 1:] = -float("inf")
        w = torch.softmax(z, -1)
        o, a = w @ vv, w @ vv.abs()
        # as the definition's tolerance in the reference: scores, exponents, sums, roundings
        dz = (d + 2) * eps * (q[i].double().abs() @ kk.abs().T) * d ** -0.5 + 4 * eps * z.abs()
        wdz = torch.where(w > 0, w * dz, 0.0)
        lost = wdz @ vv.abs() + o.abs() * wdz.sum(1, keepdim=True)
        lost = lost + a * (2.0 ** -19 + 2 * n * eps + half)
        bound = half * (o.abs() + lost) + lost + 2.0 ** -25
        worst = ((out[i].double() - o).abs() / bound).max().item()
        assert worst <= 1.0, (i, worst)
