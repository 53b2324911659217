"""Plain implementations in 64 bits for the grouped-query pools, beam search and page sharing."""
import math

import numpy as np
import torch


def encode_rows(x):
    """(codes, scales) of f32 rows [..., D]: amax / 448, nearest e4m3."""
    s = x.abs().amax(-1) / torch.tensor(448.0, device=x.device)
    y = x / torch.where(s > 0, s, torch.ones_like(s))[..., None]
    return y.to(torch.float8_e4m3fn).view(torch.uint8), s


class Pool:
    """A pool with random rows, block tables over shuffled pages."""

    def __init__(self, kv_heads, dim, page, lens, seed=0, spare=3, gain=1.0, scale_spread=0.0):
        g = torch.Generator().manual_seed(seed)
        need = [-(-int(t) // page) for t in lens]
        self.page, self.dim, self.heads = page, dim, kv_heads
        self.n_pages = sum(need) + spare
        order = torch.randperm(self.n_pages, generator=g)
        self.width = max(1, max(need, default=1))
        table, at = torch.zeros(max(1, len(lens)), self.width, dtype=torch.int32), 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n].to(torch.int32)
            at += n
        self.table = table[:len(lens)].cuda().contiguous()
        shape = (self.n_pages, kv_heads, page, dim)
        k, v = torch.randn(shape, generator=g) * gain, torch.randn(shape, generator=g)
        if scale_spread:
            v *= torch.exp2(torch.randn(shape[:3], generator=g) * scale_spread)[..., None]
        (kc, ks), (vc, vs) = encode_rows(k), encode_rows(v)
        self.k, self.v = kc.cuda(), vc.cuda()
        self.scales = torch.stack([ks, vs], -1).cuda().contiguous()
        self.lens = torch.tensor([int(t) for t in lens], dtype=torch.int64, device="cuda")

    def rows(self, b, n):
        """(keys, values) of sequence b in f64: [heads][n][dim]."""
        t = torch.arange(n, device="cuda")
        pg, at = self.table[b].long()[t // self.page], t % self.page
        s = self.scales[pg, :, at].double()
        k = self.k[pg, :, at].view(torch.float8_e4m3fn).double() * s[..., :1]
        v = self.v[pg, :, at].view(torch.float8_e4m3fn).double() * s[..., 1:]
        return k.transpose(0, 1), v.transpose(0, 1)


def attention(q, pool, lens, new, sm, causal, absolute=False):
    """Outputs in f64, [tokens][heads][dim]; absolute: sums of the values' sizes."""
    n_tok, heads, dim = q.shape
    group = heads // pool.heads
    out = torch.zeros(n_tok, heads, dim, dtype=torch.float64, device="cuda")
    at = 0
    for b, (t, n) in enumerate(zip(lens, new)):
        if n and t:
            k, v = pool.rows(b, t)
            v = v.abs() if absolute else v
            x = q[at:at + n].double().view(n, pool.heads, group, dim)
            z = torch.einsum("nhgd,htd->nhgt", x, k) * sm
            if causal:
                late = torch.arange(t, device="cuda")[None] > t - n + torch.arange(n, device="cuda")[:, None]
                z = z.masked_fill(late[:, None, None], -math.inf)
            p = torch.softmax(z, -1)
            p = torch.where(torch.isneginf(z.amax(-1, keepdim=True)), 0.0, p)   # a token that sees no row
            w = torch.einsum("nhgt,htd->nhgd", p, v)
            out[at:at + n] = w.reshape(n, heads, dim)
        at += n
    return out


def close(got, ref, what="", mass=None):
    """1e-5 of a vector's largest before the rounding to the output's type (half a step of it); mass (sums of the
    values' sizes): each weight besides off by half a step of f16, which holds 11 bits: 2^-11 of itself."""
    half = torch.finfo(got.dtype).eps / 2
    top = ref.abs().amax(-1, keepdim=True)
    own = 1e-5 * top if mass is None else 1e-5 * top + 2.0 ** -11 * mass
    bad = (got.double() - ref).abs() - (half * ref.abs() + (1 + half) * own)
    assert not torch.isnan(got).any(), what + ": NaN"
    assert bool((bad <= 0).all()), f"{what}: off by {float((got.double() - ref).abs().div(top.clamp(min=1e-300)).max()):.3g} of the largest"


def select(logits, scores, keep):
    """(scores, parents, tokens) of one batch: logits [n][b][v] and scores [n][b] as numpy f64 / f32 arrays."""
    n, b, v = logits.shape
    out = np.full((n, keep), -np.inf), np.full((n, keep), -1, np.int64), np.full((n, keep), -1, np.int64)
    for i in range(n):
        cand = []
        for j in range(b):
            if not np.isfinite(scores[i, j]):
                continue
            x = np.where(np.isnan(logits[i, j]), -np.inf, logits[i, j])
            top = x.max()
            if top == -np.inf:
                continue
            with np.errstate(invalid="ignore"):
                d = np.where(x == top, 0.0, x - top)
            mass = math.log(math.fsum(np.exp(d)))
            for t in np.argsort(-x, kind="stable")[:keep]:
                s = float(scores[i, j]) + (d[t] - mass)
                if s > -np.inf:
                    cand.append((-s, j, -x[t], t))
        for k, (s, j, _, t) in enumerate(sorted(cand)[:keep]):
            out[0][i, k], out[1][i, k], out[2][i, k] = -s, i * b + j, t
    return out


def fork(parents, lens, table, free, n_free, page):
    """The sharing of pages on lists; returns (lens, table, free, n_free, copies)."""
    n = len(parents)
    pages = [-(-t // page) for t in lens]
    first = {}
    for i, f in enumerate(parents):
        if f >= 0:
            first.setdefault(f, i)
    new, copies, taken = [list(r) for r in table], [(-1, -1)] * n, 0
    for i, f in enumerate(parents):
        if f < 0:
            continue
        new[i][:pages[f]] = table[f][:pages[f]]
        if first[f] != i and lens[f] % page:
            to = free[n_free - 1 - taken]
            taken += 1
            copies[i] = (table[f][pages[f] - 1], to)
            new[i][pages[f] - 1] = to
    kept = {p for f in first for p in table[f][:pages[f]]}
    gone = {}
    for s in range(n):
        if s not in first:
            for p in table[s][:pages[s]]:
                if p not in kept and p not in gone:
                    gone[p] = True
    free = list(free)
    n_free -= taken
    for k, p in enumerate(gone):
        free[n_free + len(gone) - 1 - k] = p
    return [lens[f] if f >= 0 else 0 for f in parents], new, free, n_free + len(gone), copies
