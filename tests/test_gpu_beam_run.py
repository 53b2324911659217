"""Beam search over grouped-query pools as a server runs it: prompts, shared pages, decoding steps, the end; each step's
attention against histories kept as plain lists in 64 bits."""
import math

import pytest
import torch

from gpu_common import kvq_module
from gqa_common import close, encode_rows, select

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    return kvq_module()


HEADS, KV, DIM, LAYERS, VOCAB = 8, 2, 64, 2, 997


def plain_attention(q, k, v):
    """q [heads][dim], k and v [rows][kv][dim] in f64."""
    g = HEADS // KV
    z = torch.einsum("hgd,thd->hgt", q.double().view(KV, g, DIM), k) / math.sqrt(DIM)
    return torch.einsum("hgt,thd->hgd", torch.softmax(z, -1), v).reshape(HEADS, DIM)


class Server:
    """A batch of `n` requests of `b` beams; every layer has its own pool, all share tables and lengths."""

    def __init__(self, kvq, n, b, page, prompts, steps, dtype):
        g = torch.Generator().manual_seed(page)
        self.kvq, self.n, self.b, self.page, self.dtype = kvq, n, b, page, dtype
        rows = max(prompts) + steps + 1
        self.width = -(-rows // page)
        self.n_pages = n * b * self.width + n * b
        i32 = dict(dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(n * b, dtype=torch.int64, device="cuda")
        self.table = torch.zeros(n * b, self.width, **i32)
        self.free, self.n_free = torch.randperm(self.n_pages, generator=g).to(**i32), torch.tensor([self.n_pages], **i32)
        self.k = [torch.zeros(self.n_pages, KV, page, DIM, dtype=torch.uint8, device="cuda") for _ in range(LAYERS)]
        self.v = [torch.zeros_like(k) for k in self.k]
        self.s = [torch.zeros(self.n_pages, KV, page, 2, device="cuda") for _ in range(LAYERS)]
        self.embed = torch.randn(VOCAB, LAYERS, HEADS + 2 * KV, DIM, generator=g).to(dtype).cuda()
        self.head = (torch.randn(VOCAB, HEADS * DIM, generator=g) / 4).to(dtype).cuda()
        self.rope = kvq.rope_layout([100.0 ** (-i / 16) for i in range(16)])
        # the encoder's rows: a request's beams list the same pages
        self.source = [11, 64, 130][:n]
        x = torch.randn(2, sum(-(-t // 16) for t in self.source), KV, 16, DIM, generator=g).cuda()
        (self.xk, ks), (self.xv, vs) = encode_rows(x[0]), encode_rows(x[1])
        self.xs = torch.stack([ks, vs], -1).contiguous()
        self.xt, at = torch.zeros(n * b, 9, **i32), 0
        for i, t in enumerate(self.source):
            m = -(-t // 16)
            self.xt[i * b:(i + 1) * b, :m] = torch.arange(at, at + m, **i32)
            at += m
        self.xlens = torch.tensor([t for t in self.source for _ in range(b)], dtype=torch.int64, device="cuda")
        size = kvq.kv_gqa_attn_paged_workspace_size(n * b, HEADS, KV, DIM, sum(prompts), bf16=dtype == torch.bfloat16)
        u8 = dict(dtype=torch.uint8, device="cuda")
        self.ws = torch.zeros(size, **u8)
        self.pages_ws = torch.zeros(kvq.kv_pages_workspace_size(), **u8)
        self.beam_ws = torch.zeros(kvq.kv_beam_workspace_size(n, b, VOCAB, b), **u8)
        self.fork_ws = torch.zeros(kvq.kv_pages_fork_workspace_size(n * b, self.width, self.n_pages), **u8)
        self.scores, self.next_scores = torch.zeros(n, b, device="cuda"), torch.zeros(n, b, device="cuda")
        self.parents, self.tokens = torch.zeros(n, b, **i32), torch.zeros(n, b, **i32)
        self.copies = torch.zeros(n * b, 2, **i32)
        self.cu = torch.zeros(n * b + 1, dtype=torch.int64, device="cuda")

    def errors(self):
        return [self.kvq.read_device_error(w) for w in (self.ws, self.pages_ws, self.fork_ws)]

    def forward(self, ids, new):
        """Appends `new` tokens of each sequence and attends; the outputs of all layers and of the last cross attention."""
        n = len(ids)
        self.slots = torch.full((n,), -1, dtype=torch.int64, device="cuda")
        self.pos = torch.zeros(n, dtype=torch.int64, device="cuda")
        self.kvq.kv_pages_reserve(self.lens, new, self.table, self.free, self.n_free, self.page, self.lens, self.cu, self.slots,
                                  self.pos, self.pages_ws)
        fused = self.embed[ids.long()]
        self.q, self.out = [], []
        for i in range(LAYERS):
            q, k, v = (t.contiguous() for t in fused[:, i].split([HEADS, KV, KV], 1))
            turned, out = torch.empty_like(q), torch.empty_like(q)
            self.kvq.kv_gqa_append(self.rope, k, v, self.pos, self.slots, q, turned, self.k[i], self.v[i], self.s[i],
                                   self.pages_ws)
            self.kvq.kv_gqa_attn_paged(turned, self.cu, self.k[i], self.v[i], self.s[i], self.table, self.lens, out, self.ws,
                                       1 / math.sqrt(DIM))
            self.q.append(turned)
            self.out.append(out)
        self.cross = torch.empty_like(out)
        self.kvq.kv_gqa_attn_paged(self.out[-1], self.cu, self.xk, self.xv, self.xs, self.xt, self.xlens, self.cross, self.ws,
                                   1 / math.sqrt(DIM), causal=False)

    def choose(self, last):
        """The best continuations from the tokens `last` of the cross attention; pages and lengths follow."""
        self.logits = (self.cross[last].view(-1, HEADS * DIM) @ self.head.T).view(self.n, self.b, VOCAB)
        self.kvq.kv_beam_select(self.logits, self.scores, self.next_scores, self.parents, self.tokens, self.beam_ws)
        self.kvq.kv_pages_fork(self.parents.view(-1), self.lens, self.table, self.free, self.n_free, self.page, self.copies,
                               self.fork_ws)
        self.kvq.kv_pages_copy(self.copies, [*self.k, *self.v, *self.s], self.fork_ws)


class Histories:
    """Every sequence's rows as the append left them, in lists."""

    def __init__(self, n):
        self.rows = [[[] for _ in range(LAYERS)] for _ in range(n)]

    def append(self, sv, new):
        slots, at = sv.slots.tolist(), 0
        for b, m in enumerate(new):
            for slot in slots[at:at + m]:
                pg, r = divmod(slot, sv.page)
                for i in range(LAYERS):
                    kv = [c[i][pg, :, r].view(torch.float8_e4m3fn).double() * sv.s[i][pg, :, r, j, None].double()
                          for j, c in enumerate((sv.k, sv.v))]
                    self.rows[b][i].append(kv)
            at += m

    def fork(self, parents):
        self.rows = [[list(r) for r in self.rows[f]] if f >= 0 else [[] for _ in range(LAYERS)] for f in parents]

    def check(self, sv, new):
        """Every token's output against the lists."""
        at = 0
        for b, m in enumerate(new):
            for i in range(LAYERS):
                k, v = (torch.stack([r[j] for r in self.rows[b][i]]) for j in (0, 1)) if self.rows[b][i] else (None, None)
                for t in range(m):
                    n = len(k) - m + t + 1
                    ref = plain_attention(sv.q[i][at + t], k[:n], v[:n])
                    # many vectors go the tensor cores' way: weights off by 2^-11, of bf16 queries
                    mass = plain_attention(sv.q[i][at + t], k[:n], v[:n].abs()) if m > 1 and sv.dtype == torch.bfloat16 else None
                    close(sv.out[i][at + t], ref, f"sequence {b}, layer {i}, token {t}", mass)
            at += m

    def check_cross(self, sv, new):
        at = 0
        for b, m in enumerate(new):
            n = sv.source[b // sv.b]
            pg, r = sv.xt[b].long()[torch.arange(n, device="cuda") // 16], torch.arange(n, device="cuda") % 16
            k, v = (c[pg, :, r].view(torch.float8_e4m3fn).double() * sv.xs[pg, :, r, j, None].double()
                    for j, c in enumerate((sv.xk, sv.xv)))
            for t in range(m):
                mass = plain_attention(sv.out[-1][at + t], k, v.abs()) if m > 1 and sv.dtype == torch.bfloat16 else None
                close(sv.cross[at + t], plain_attention(sv.out[-1][at + t], k, v), f"cross {b}", mass)
            at += m


def held(sv):
    """Pages that the sequences list, each once; checks that the stack holds the others."""
    lens, table = sv.lens.tolist(), sv.table.tolist()
    pages = {p for n, row in zip(lens, table) for p in row[:-(-n // sv.page)]}
    free = sv.free.tolist()[:int(sv.n_free)]
    assert sorted(free + list(pages)) == list(range(sv.n_pages))
    return pages


def prompt(sv, prompts):
    """The prompts go to the first beam of each request, whose best continuations are the beams."""
    g = torch.Generator().manual_seed(7)
    new = [t if j == 0 else 0 for t in prompts for j in range(sv.b)]
    sv.forward(torch.randint(0, VOCAB, (sum(new),), generator=g).cuda(), torch.tensor(new, dtype=torch.int64, device="cuda"))
    last = torch.tensor([sum(prompts[:i + 1]) - 1 for i in range(sv.n) for _ in range(sv.b)], device="cuda")
    sv.scores.fill_(-math.inf)
    sv.scores[:, 0] = 0.0
    return new, last


@pytest.mark.parametrize("dtype,page", [(torch.bfloat16, 16), (torch.float32, 16), (torch.bfloat16, 32)])
def test_prompts_steps_and_the_end(kvq, dtype, page):
    n, b, prompts, steps = 3, 4, [5, 47, 16], 14
    sv, hist = Server(kvq, n, b, page, prompts, steps, dtype), Histories(n * b)
    new, last = prompt(sv, prompts)
    ones = torch.ones(n * b, dtype=torch.int64, device="cuda")
    branched = 0
    for step in range(steps):
        if step:
            new, last = [1] * (n * b), torch.arange(n * b, device="cuda")
            if step % 5 == 2:   # a token that is taken back
                sv.forward(sv.tokens.view(-1).flip(0).contiguous(), ones)
                kvq.kv_pages_trim(sv.lens, sv.lens - 1, sv.table, sv.free, sv.n_free, page, sv.pages_ws)
                held(sv)
            sv.forward(sv.tokens.view(-1), ones)
        hist.append(sv, new)
        hist.check(sv, new)
        hist.check_cross(sv, new)
        sv.choose(last)
        best = select(sv.logits.double().cpu().numpy(), sv.scores.cpu().numpy(), b)
        assert sv.parents.tolist() == best[1].tolist() and sv.tokens.tolist() == best[2].tolist()
        parents = sv.parents.view(-1).tolist()
        branched += len(set(parents)) < len(parents)
        hist.fork(parents)
        assert sv.lens.tolist() == [len(r[0]) for r in hist.rows]
        held(sv)
        sv.scores.copy_(sv.next_scores)
        assert sv.errors() == [0, 0, 0]
    assert branched > steps // 2
    # request 1 ends, the others go on with two beams each twice; then all end
    sv.parents.view(-1).copy_(torch.tensor([0, 0, 2, 2] + [-1] * 4 + [9, 8, 9, 8], dtype=torch.int32))
    kvq.kv_pages_fork(sv.parents.view(-1), sv.lens, sv.table, sv.free, sv.n_free, page, sv.copies, sv.fork_ws)
    kvq.kv_pages_copy(sv.copies, [*sv.k, *sv.v, *sv.s], sv.fork_ws)
    hist.fork(sv.parents.view(-1).tolist())
    held(sv)
    new = [1] * 4 + [0] * 4 + [1] * 4
    sv.forward(torch.arange(8, device="cuda"), torch.tensor(new, dtype=torch.int64, device="cuda"))
    hist.append(sv, new)
    hist.check(sv, new)
    sv.parents.fill_(-1)
    kvq.kv_pages_fork(sv.parents.view(-1), sv.lens, sv.table, sv.free, sv.n_free, page, sv.copies, sv.fork_ws)
    assert sv.errors() == [0, 0, 0] and held(sv) == set() and sv.lens.tolist() == [0] * 12


def test_a_step_captured_and_replayed(kvq):
    n, b, prompts, steps = 3, 4, [5, 47, 16], 12
    runs = []
    for captured in (False, True):
        sv = Server(kvq, n, b, 16, prompts, steps, torch.bfloat16)
        _, last = prompt(sv, prompts)
        sv.choose(last)
        sv.scores.copy_(sv.next_scores)
        ones, last = torch.ones(n * b, dtype=torch.int64, device="cuda"), torch.arange(n * b, device="cuda")

        def step():
            sv.forward(sv.tokens.view(-1), ones)
            sv.choose(last)
            sv.scores.copy_(sv.next_scores)

        step()   # libraries' first calls are made outside the capture
        run = step
        if captured:
            graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
            st.wait_stream(torch.cuda.current_stream())
            with torch.cuda.graph(graph, stream=st):
                step()
            run = graph.replay
        trace = []
        for _ in range(steps - 2):
            run()
            trace += [t.clone() for t in (sv.parents, sv.tokens, sv.scores, sv.lens, sv.cross)]
        held(sv)
        assert sv.errors() == [0, 0, 0]
        runs.append(trace)
    for x, y in zip(*runs):
        assert torch.equal(x, y)
