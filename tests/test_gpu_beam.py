"""Beam search's selection, page sharing and page copies on the GPU against plain implementations."""
import math

import numpy as np
import pytest
import torch

from gpu_common import kvq_module
from gqa_common import fork, select

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    return kvq_module()


DTYPES = [torch.bfloat16, torch.float32]


def run_select(kvq, logits, scores, keep, ws=None):
    n, b, v = logits.shape
    ws = torch.zeros(kvq.kv_beam_workspace_size(n, b, v, keep), dtype=torch.uint8, device="cuda") if ws is None else ws
    o = torch.full((n, keep), 3.0, device="cuda")
    p, t = (torch.full((n, keep), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    kvq.kv_beam_select(logits, scores, o, p, t, ws)
    return o, p, t


def check_select(kvq, logits, scores, keep):
    o, p, t = run_select(kvq, logits, scores, keep)
    with np.errstate(over="ignore"):
        ro, rp, rt = select(logits.double().cpu().numpy(), scores.cpu().numpy(), keep)
    assert np.array_equal(p.cpu().numpy(), rp) and np.array_equal(t.cpu().numpy(), rt)
    got = o.double().cpu().numpy()
    # the mass in f32: 2^-22 of each term and one rounding for each of at most 129 terms a
    # partial sum, 8e-6; then the result's rounding
    assert np.array_equal(np.isneginf(got), np.isneginf(ro))
    ok = ~np.isneginf(ro)
    assert np.all(np.abs(got[ok] - ro[ok]) <= 1e-5 + 2.0 ** -24 * np.abs(ro[ok]))


def random_logits(n, b, v, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, b, v, generator=g) * 3).to(dtype).cuda(), (-4 * torch.rand(n, b, generator=g)).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,b,v,keep", [(1, 1, 1, 1), (1, 1, 5, 8), (3, 4, 1000, 8), (2, 5, 4099, 10), (1, 8, 50001, 16),
                                        (2, 32, 9000, 64), (1, 1, 200003, 64), (9, 2, 32768, 4), (1, 16, 70000, 32),
                                        (300, 1, 777, 2)])
def test_random(kvq, dtype, n, b, v, keep):
    check_select(kvq, *random_logits(n, b, v, dtype, seed=v), keep)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ties_and_orders(kvq, dtype):
    v = 30011
    x, s = random_logits(2, 3, v, dtype)
    check_select(kvq, torch.zeros_like(x), s, 8)                                # equal logits
    check_select(kvq, torch.zeros_like(x), torch.zeros_like(s), 8)              # equal beams
    check_select(kvq, x.round(), torch.zeros_like(s), 64)                       # many ties
    check_select(kvq, x[:, :1].expand(2, 3, v).contiguous(), torch.zeros_like(s), 16)   # the same beam three times
    up = (torch.arange(v, device="cuda") // 64 / 64.0).to(dtype)
    check_select(kvq, up.expand(2, 3, v).contiguous(), s, 16)                   # ascending
    check_select(kvq, up.flip(0).expand(2, 3, v).contiguous(), s, 16)
    z = torch.zeros_like(x)
    z[..., ::2] = -0.0                                                          # -0 and 0 are one value
    check_select(kvq, z, s, 8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masks(kvq, dtype):
    v = 20000
    x, s = random_logits(3, 4, v, dtype)
    low = torch.finfo(dtype).min
    y = torch.full_like(x, low)                      # a grammar: three tokens may come
    y[..., [7, 9000, 19999]] = x[..., [7, 9000, 19999]]
    check_select(kvq, y, s, 8)
    y = torch.full_like(x, -math.inf)
    y[..., [7, 9000, 19999]] = x[..., [7, 9000, 19999]]
    check_select(kvq, y, s, 16)                      # 12 continuations of 16
    y[1] = -math.inf                                 # none
    y[2, 0] = -math.inf
    check_select(kvq, y, s, 16)
    y = x.clone()
    y[:, :, 100:200] = math.nan
    check_select(kvq, y, s, 8)
    check_select(kvq, torch.full_like(x, math.nan), s, 4)
    y = x.clone()
    y[0, 1, [5, 15000]] = math.inf                   # infinite logits share the mass
    y[2] = math.inf
    check_select(kvq, y, s, 8)
    y = x.clone()
    y[0, 0, 3] = torch.finfo(dtype).max
    y[0, 1, :] = torch.finfo(dtype).max
    check_select(kvq, y, s, 8)
    for dead in (-math.inf, math.inf, math.nan):
        d = s.clone()
        d[0, 1:] = dead                              # the first step: one beam
        d[1] = dead
        check_select(kvq, x, d, 8)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fill", ["lowest", -1e30, -1e4])
def test_masks_of_the_lowest_value_with_few_tokens_left(kvq, dtype, fill):
    """Masked tokens of a finite logit come once the others have: of the beam with the largest cum - lse, in order."""
    fill = torch.finfo(dtype).min if fill == "lowest" else float(torch.tensor(fill, dtype=dtype))
    for v, keep in ((40, 12), (1000, 16), (30011, 20)):
        x, s = torch.full((2, 3, v), fill, dtype=dtype, device="cuda"), torch.tensor([[-3.0, -1.0, -2.0], [0.0, -9.0, 1.0]], device="cuda")
        g = torch.Generator().manual_seed(v)
        free = torch.tensor([5, 17])
        x[:, :, free] = torch.randn(2, 3, 2, generator=g).to(dtype).cuda()
        o, p, t = (a.cpu().numpy() for a in run_select(kvq, x, s, keep))
        z = x[:, :, free].double().cpu().numpy()
        lse = np.logaddexp(z[..., 0], z[..., 1])
        base = s.double().cpu().numpy() - lse
        for i in range(2):
            order = sorted((-(base[i, b] + z[i, b, k]), b, int(free[k])) for b in range(3) for k in range(2))
            b = int(base[i].argmax())
            rest = [t_ for t_ in range(v) if t_ not in free.tolist()][:keep - 6]
            assert p[i].tolist() == [3 * i + c[1] for c in order] + [3 * i + b] * (keep - 6)
            assert t[i].tolist() == [c[2] for c in order] + rest
            ref = np.array([-c[0] for c in order] + [fill + base[i, b]] * (keep - 6))
            assert np.all(np.abs(o[i] - ref) <= 1e-5 + 2.0 ** -24 * np.abs(ref))   # as check_select


def test_sizes_of_logits(kvq):
    x, s = random_logits(1, 3, 5000, torch.float32)
    for scale in (1e-20, 1e3, 1e10, 1e30, 1e38 / 12):
        check_select(kvq, x * scale, s, 8)
        check_select(kvq, x + scale, s, 8)


def test_scores_that_cannot_tell_logits_apart(kvq):
    # one beam: whatever the sums round to, the larger logit is better
    x, _ = random_logits(3, 1, 150001, torch.float32)
    for scores in (0.0, -1e6, 1e30, -3e38):
        check_select(kvq, x * 1e-9, torch.full((3, 1), scores, device="cuda"), 64)


def test_rows_at_a_distance_and_unaligned(kvq):
    x, s = random_logits(2, 3, 5001, torch.bfloat16)
    wide = torch.full((2, 3, 6007), 50.0, dtype=torch.bfloat16, device="cuda")
    wide[..., 5:5006] = x
    a, b = run_select(kvq, wide[..., 5:5006], s, 8), run_select(kvq, x, s, 8)
    assert all(torch.equal(i, j) for i, j in zip(a, b))
    check_select(kvq, wide[..., 5:5006], s, 8)


def test_the_workspace_is_left_ready_and_graphs_replay(kvq):
    x, s = random_logits(4, 4, 30000, torch.float32)
    ws = torch.zeros(kvq.kv_beam_workspace_size(4, 4, 30000, 8), dtype=torch.uint8, device="cuda")
    first = run_select(kvq, x, s, 8, ws)
    assert all(torch.equal(i, j) for i, j in zip(first, run_select(kvq, x, s, 8, ws)))
    o, p, t = (torch.zeros_like(i) for i in first)
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=st):
        kvq.kv_beam_select(x, s, o, p, t, ws)
    for k in range(3):
        x.copy_(x.roll(k, -1))
        graph.replay()
        assert all(torch.equal(i, j) for i, j in zip((o, p, t), run_select(kvq, x, s, 8)))


def test_one_workspace_for_calls_of_different_sizes(kvq):
    sizes = [(40, 4, 30000, 8), (2, 4, 30000, 8), (40, 4, 100, 8), (1, 4, 30000, 8), (33, 2, 9000, 3)]
    ws = torch.zeros(kvq.kv_beam_workspace_size(*sizes[0]), dtype=torch.uint8, device="cuda")
    for i, (n, b, v, keep) in enumerate(sizes + sizes):
        x, s = random_logits(n, b, v, DTYPES[i % 2], seed=i)
        assert all(torch.equal(i, j) for i, j in zip(run_select(kvq, x, s, keep, ws), run_select(kvq, x, s, keep)))


# -- page sharing ------------------------------------------------------------------

class Batch:
    def __init__(self, lens, page, width, n_pages, seed=0, shared=()):
        """Sequences with pages of their own, but for (a, b, k): b lists a's first k pages."""
        r = np.random.default_rng(seed)
        order = list(map(int, r.permutation(n_pages)))
        self.page, self.lens, at = page, list(lens), 0
        self.table = [[int(i) for i in r.integers(0, n_pages, width)] for _ in lens]
        for s, t in enumerate(lens):
            n = -(-t // page)
            self.table[s][:n] = order[at:at + n]
            at += n
        loose = []
        for a, b, k in shared:
            loose += self.table[b][:k]
            self.table[b][:k] = self.table[a][:k]
        rest = order[at:] + loose
        self.n_free, self.free = len(rest), rest + [0] * (n_pages - len(rest))

    def device(self):
        i32 = dict(dtype=torch.int32, device="cuda")
        return dict(lens=torch.tensor(self.lens, device="cuda"), table=torch.tensor(self.table, **i32),
                    free=torch.tensor(self.free, **i32), n_free=torch.tensor([self.n_free], **i32),
                    copies=torch.full((len(self.lens), 2), 55, **i32))

    def step(self, parents):
        self.lens, self.table, self.free, self.n_free, copies = fork(parents, self.lens, self.table, self.free, self.n_free,
                                                                     self.page)
        return copies


def run_fork(kvq, d, parents, page, ws=None):
    n, w = d["table"].shape
    if ws is None:
        ws = torch.zeros(kvq.kv_pages_fork_workspace_size(n, w, d["free"].numel()), dtype=torch.uint8, device="cuda")
    kvq.kv_pages_fork(torch.tensor(parents, dtype=torch.int32, device="cuda"), d["lens"], d["table"], d["free"], d["n_free"],
                      page, d["copies"], ws)
    return ws


def same(d, batch, copies):
    assert d["lens"].tolist() == batch.lens
    assert d["table"].tolist() == batch.table
    assert d["n_free"].tolist() == [batch.n_free]
    assert d["free"].tolist()[:batch.n_free] == batch.free[:batch.n_free]
    assert d["copies"].tolist() == [list(c) for c in copies]


@pytest.mark.parametrize("page", [1, 16, 256])
@pytest.mark.parametrize("n,seed", [(1, 0), (2, 1), (7, 2), (64, 3), (1000, 4), (1025, 5), (4096, 6)])
def test_fork_steps(kvq, page, n, seed):
    r = np.random.default_rng(seed)
    top = 40 * page if n < 2000 else 3 * page
    lens = [int(x) for x in r.integers(0, top, n)]
    width = -(-top // page) + 2
    batch = Batch(lens, page, width, n * width + n, seed)
    d = batch.device()
    ws = None
    for k in range(4):
        parents = [int(x) for x in r.integers(0, n, n)]
        if k % 2:
            parents = [-1 if r.random() < 0.3 else p for p in parents]
        copies = batch.step(parents)
        ws = run_fork(kvq, d, parents, page, ws)
        same(d, batch, copies)
        assert kvq.read_device_error(ws) == 0
        marks = ws[256:256 + 4 * len(batch.free)].view(torch.int32)
        assert int(marks.abs().sum()) == 0


def test_fork_ends_everything(kvq):
    batch = Batch([100, 100, 100, 37], 16, 9, 40, shared=[(0, 1, 6), (0, 2, 4)])
    d = batch.device()
    copies = batch.step([-1] * 4)
    run_fork(kvq, d, [-1] * 4, 16)
    same(d, batch, copies)
    assert batch.n_free == 40 and sorted(batch.free) == list(range(40))


def test_fork_refuses_all_or_nothing(kvq):
    def fresh():
        return Batch([33, 40, 5], 16, 4, 12)   # two copies are needed, five pages are free

    for name, status in (("parent", 1), ("low parent", 1), ("length", 1), ("long", 1), ("page", 1), ("free count", 1),
                         ("free page", 1), ("few", 3)):
        batch = fresh()
        d = batch.device()
        parents = [0, 0, 0]
        if name == "parent":
            parents[1] = 3
        elif name == "low parent":
            parents[1] = -2
        elif name == "length":
            d["lens"][2] = -1
        elif name == "long":
            d["lens"][2] = 65
        elif name == "page":
            d["table"][1, 0] = 12
        elif name == "free count":
            d["n_free"][0] = 13
        elif name == "free page":
            d["free"][batch.n_free - 2] = -1
        else:
            d["n_free"][0] = 1
        before = {k: v.clone() for k, v in d.items()}
        ws = run_fork(kvq, d, parents, 16)
        assert kvq.read_device_error(ws) == status, name
        for k in ("lens", "table", "free", "n_free"):
            assert torch.equal(d[k], before[k]), (name, k)
        assert d["copies"].tolist() == [[-1, -1]] * 3, name
        good = fresh()
        e = good.device()
        copies = good.step([0, 0, 0])
        run_fork(kvq, e, [0, 0, 0], 16, ws)   # the workspace serves on
        same(e, good, copies)
        assert kvq.read_device_error(ws) == 0


def test_operands_aligned_to_their_elements_only(kvq):
    def odd(t):   # the same values, one element behind a 16-byte boundary
        return torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)

    batch = Batch([33, 40, 5, 64], 16, 5, 30, seed=4)
    d = {k: odd(v) for k, v in batch.device().items()}
    assert all(v.data_ptr() % 16 for v in d.values())
    for parents in ([0, 0, 1, 3], [2, 2, 2, -1]):
        copies = batch.step(parents)
        ws = torch.zeros(kvq.kv_pages_fork_workspace_size(4, 5, 30), dtype=torch.uint8, device="cuda")
        kvq.kv_pages_fork(odd(torch.tensor(parents, dtype=torch.int32, device="cuda")), d["lens"], d["table"], d["free"], d["n_free"], 16,
                          d["copies"], ws)
        same(d, batch, copies)
    pool = torch.arange(30 * 7, dtype=torch.int32, device="cuda").view(30, 7)
    kvq.kv_pages_copy(odd(torch.tensor([[3, 9]], dtype=torch.int32, device="cuda")), [odd(pool)])
    x, s = random_logits(3, 4, 5000, torch.float32)
    want = run_select(kvq, x, s, 8)
    got = [odd(torch.zeros_like(w)) for w in want]
    kvq.kv_beam_select(odd(x), odd(s), *got, torch.zeros(kvq.kv_beam_workspace_size(3, 4, 5000, 8), dtype=torch.uint8, device="cuda"))
    assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_copy(kvq):
    g = torch.Generator().manual_seed(0)
    pools = [torch.randint(0, 255, (12, 2, 16, 64), generator=g, dtype=torch.uint8).cuda(),
             torch.randn(12, 2, 16, 2, generator=g).cuda(), torch.randint(0, 255, (12, 7), generator=g, dtype=torch.uint8).cuda(),
             torch.randint(0, 255, (12, 70001), generator=g, dtype=torch.uint8).cuda(),
             torch.randint(0, 255, (12 * 16, 576), generator=g, dtype=torch.uint8).cuda()] + \
        [torch.randn(12, 3, generator=g).cuda() for _ in range(200)]   # more pools than one launch takes
    before = [p.clone() for p in pools]
    copies = torch.tensor([[3, 1], [-1, -1], [3, 0], [5, 11], [-1, 4]], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.kv_pages_copy(copies, pools, err)
    assert int(err) == 0
    for p, b in zip(pools, before):
        x, y = p.view(12, -1), b.view(12, -1).clone()
        for f, t in ((3, 1), (3, 0), (5, 11)):
            y[t] = y[f]
        assert torch.equal(x, y)
    kvq.kv_pages_copy(torch.tensor([[3, 12], [2, 7]], dtype=torch.int32, device="cuda"), pools[:1], err)
    assert int(err) == 1 and torch.equal(pools[0][7], before[0][2])
