"""What is measured of the paged-cache operators: cases, inputs and plain forms.

Three operators that a serving loop over a paged quantized MLA cache calls one
after another:

* pages   kv_pages_reserve / kv_pages_trim: pages for the new rows of a batch
          taken from a free list, block tables extended, one pool slot and one
          position per new row; then the rows given back (a refused step).
* rope    kv_rope_append: rotary positions with one or several axes on the
          queries' and the new rows' rotary dims, the rows quantized into their
          slots.
* attn    kv_attn_paged: causal attention of every sequence's new tokens over
          its paged quantized rows (one token per sequence is the decode step).

A row has 576 dims: 512 latent (also the value) and 64 rotary.
"""
import math
import random

import numpy as np
import torch

own = False

D, DL, DR = 576, 512, 64
SM = 1.0 / math.sqrt(192.0)
SEED = 4   # sign seed of the 4-bit rotation
# positive levels of the 16-level Lloyd-Max quantizer of N(0, 1)
LEVELS = (0.12839503586292267, 0.38804829120635986, 0.6567591488361359, 0.9423404335975647,
          1.2562311887741089, 1.6180464029312134, 2.069017171859741, 2.7325894832611084)


# -- cases ---------------------------------------------------------------------

def listed():
    return [
        # a decode step's bookkeeping: 64 sequences, one new row each
        dict(name="pages_decode_64", kind="pages", n_seq=64, page=64, past_lo=1, past_hi=8192, new_lo=1, new_hi=1),
        # chunked prefill among many sequences: up to 64 rows each, small pages
        dict(name="pages_mixed_1024", kind="pages", n_seq=1024, page=16, past_lo=0, past_hi=4096, new_lo=0, new_hi=63),
        # a decode step's queries and rows, far positions
        dict(name="rope_decode_8", kind="rope", n=8, heads=128, dtype="bf16", axes=1, spread="sections",
             adjacent=True, far=131072),
        # a prefill chunk with image positions on three axes
        dict(name="rope_chunk_2048", kind="rope", n=2048, heads=128, dtype="bf16", axes=3, spread="sections",
             adjacent=False, far=126976),
        # an odd batch in f32, video positions interleaved over the pairs
        dict(name="rope_odd_333_f32", kind="rope", n=333, heads=20, dtype="f32", axes=3, spread="interleaved",
             adjacent=False, far=1000003),
        # the decode step of 8 sequences of 4096 rows, KV8 and 4 bits
        dict(name="attn_decode_8x4096_kv8", kind="attn", fmt="kv8", dtype="bf16", heads=128, n_seq=8, page=64,
             past_lo=4095, past_hi=4095, new_lo=1, new_hi=1),
        dict(name="attn_decode_8x4096_tq4", kind="attn", fmt="tq4", dtype="bf16", heads=128, n_seq=8, page=64,
             past_lo=4095, past_hi=4095, new_lo=1, new_hi=1),
        # ragged long-context decode: 32 sequences of 1024 to 131072 rows
        dict(name="attn_decode_ragged_32", kind="attn", fmt="kv8", dtype="bf16", heads=128, n_seq=32, page=64,
             past_lo=1024, past_hi=131071, new_lo=1, new_hi=1),
        # a prefill chunk of 512 tokens over a long prefix
        dict(name="attn_chunk_512_past_32768", kind="attn", fmt="kv8", dtype="bf16", heads=128, n_seq=1, page=128,
             past_lo=32768, past_hi=32768, new_lo=512, new_hi=512),
        # a first chunk of a new prompt, 4 bits, odd length, small pages
        dict(name="attn_first_chunk_777_tq4", kind="attn", fmt="tq4", dtype="bf16", heads=128, n_seq=1, page=32,
             past_lo=0, past_hi=0, new_lo=777, new_hi=777),
        # decode tokens, speculative windows and prompt chunks in one batch, 16 heads
        dict(name="attn_mixed_24", kind="attn", fmt="kv8", dtype="bf16", heads=16, n_seq=24, page=16,
             past_lo=0, past_hi=8000, new_lo=1, new_hi=120),
        # the exact path that results are checked against, f32 queries
        dict(name="attn_exact_4_f32", kind="attn", fmt="kv8", dtype="f32", heads=16, n_seq=4, page=64,
             past_lo=100, past_hi=700, new_lo=1, new_hi=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    kind = rng.choice(["pages", "rope", "attn", "attn"])
    if kind == "pages":
        n_seq = _log(rng, 1, 1500)
        return dict(kind="pages", n_seq=n_seq, page=rng.choice([16, 32, 64, 128, 256]), past_lo=rng.choice([0, 1, 100]),
                    past_hi=_log(rng, 200, 8192), new_lo=rng.choice([0, 1]), new_hi=_log(rng, 1, max(1, 60000 // n_seq)))
    if kind == "rope":
        heads = rng.choice([1, 8, 16, 20, 32, 64, 128])
        axes = rng.choice([1, 2, 3])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        return dict(kind="rope", n=_log(rng, 1, 2048 if dtype == "bf16" else 1024), heads=heads, dtype=dtype, axes=axes,
                    spread=rng.choice(["sections", "interleaved"]), adjacent=rng.random() < 0.5, far=_log(rng, 100, 1 << 20))
    heads = rng.choice([8, 16, 20, 32, 48, 64, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    fmt = rng.choice(["kv8", "kv8", "tq4"])
    form = rng.choice(["decode", "decode", "chunk", "mixed", "exact"])
    if form == "exact":
        return dict(kind="attn", fmt=fmt, dtype="f32", heads=rng.choice([8, 16, 20]), n_seq=_log(rng, 1, 6), page=page,
                    past_lo=0, past_hi=_log(rng, 20, 700), new_lo=1, new_hi=rng.choice([1, 2]))
    if form == "decode":
        n_seq = _log(rng, 1, 64)
        hi = _log(rng, 64, min(131071, 4000000 // n_seq))
        return dict(kind="attn", fmt=fmt, dtype="bf16", heads=heads, n_seq=n_seq, page=page, past_lo=max(1, hi // 16),
                    past_hi=hi, new_lo=1, new_hi=1)
    if form == "chunk":
        new = _log(rng, 2, 1024)
        past = rng.choice([0, _log(rng, 16, max(17, 16000000 // (new * heads // 128 + 256) - new))])
        return dict(kind="attn", fmt=fmt, dtype="bf16", heads=heads, n_seq=1, page=page, past_lo=min(past, 65536),
                    past_hi=min(past, 65536), new_lo=new, new_hi=new)
    n_seq = _log(rng, 2, 32)
    return dict(kind="attn", fmt=fmt, dtype="bf16", heads=rng.choice([8, 16, 20, 32]), n_seq=n_seq, page=page, past_lo=0,
                past_hi=_log(rng, 64, 8192), new_lo=0, new_hi=_log(rng, 2, 128))


def _lengths(case):
    """(past, new) rows of every sequence, from the case alone."""
    r = random.Random("%s" % sorted((k, v) for k, v in case.items() if k != "name"))
    past = [r.randint(case["past_lo"], case["past_hi"]) for _ in range(case["n_seq"])]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["n_seq"])]
    if sum(new) == 0:
        new[0] = 1
    return past, new


def _spread(case):
    """(axis, inverse frequency) of each of the 32 rotary pairs."""
    n, a = DR // 2, case["axes"]
    inv = [10000.0 ** (-2.0 * i / DR) for i in range(n)]
    if case["spread"] == "interleaved":
        axis = [i % a for i in range(n)]
    else:
        first = n - (a - 1) * (n * 3 // 8) if a > 1 else n
        axis = [0 if i < first else 1 + (i - first) * (a - 1) // (n - first) for i in range(n)]
    return axis, inv


def _signs(dims):
    """+1 / -1 of each dim: splitmix64 words from state SEED, a block starting at a fresh word."""
    m, state, out = (1 << 64) - 1, SEED, []
    for n in dims:
        bits = []
        while len(bits) < n:
            state = (state + 0x9E3779B97F4A7C15) & m
            z = state
            z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & m
            z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & m
            z ^= z >> 31
            bits += [(z >> i) & 1 for i in range(64)]
        out += [-1.0 if v else 1.0 for v in bits[:n]]
    return out


def _hadamard(n):
    h = torch.ones(1, 1)
    while h.shape[0] < n:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h / math.sqrt(n)


# -- inputs --------------------------------------------------------------------

def _table(past, new, page, g, extra=0):
    """Block tables over a shuffled pool: every sequence's pages for past (+ new) rows."""
    need = [-(-(p + n) // page) for p, n in zip(past, new)]
    width = max(1, max(need) + extra)
    n_pages = sum(need) + 7
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    cols = torch.arange(width, device="cuda")[None]
    needed = torch.tensor(need, device="cuda")[:, None]
    first = torch.cumsum(needed, 0) - needed
    table = torch.where(cols < needed, order[(first + cols).clamp(max=n_pages - 1)], 0).to(torch.int32)
    return table.contiguous(), order, sum(need), n_pages


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 11)
    s = dict(case=case)
    if case["kind"] == "pages":
        past, new = _lengths(case)
        page = case["page"]
        held = [-(-p // page) * page for p in past]
        table, order, used, n_pages = _table(held, [0] * len(past), page, g, extra=-(-case["new_hi"] // page) + 1)
        n_need = sum(-(-(p + n) // page) - -(-p // page) for p, n in zip(past, new))
        pool = n_pages + n_need + 50
        free = torch.zeros(pool, dtype=torch.int32, device="cuda")
        rest = torch.cat([order[used:], torch.arange(n_pages, pool, dtype=torch.int32, device="cuda")])
        rest = rest[torch.randperm(rest.numel(), generator=g, device="cuda")]
        free[:rest.numel()] = rest
        n = sum(new)
        s.update(lens=torch.tensor(past, device="cuda"), new=torch.tensor(new, device="cuda"), table=table, free=free,
                 n_free=torch.tensor([rest.numel()], dtype=torch.int32, device="cuda"), page=page, n=n,
                 lens_out=torch.zeros(len(past), dtype=torch.int64, device="cuda"),
                 cu=torch.zeros(len(past) + 1, dtype=torch.int64, device="cuda"),
                 slots=torch.zeros(n, dtype=torch.int64, device="cuda"),
                 positions=torch.zeros(n, dtype=torch.int64, device="cuda"))
        if own:
            from quantized_kv_cache_kv8_gb300 import kvq
            s["ws"] = torch.zeros(kvq.kv_pages_workspace_size(), dtype=torch.uint8, device="cuda")
        return s
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    gain = torch.exp(torch.randn(D, generator=g, device="cuda"))
    if case["kind"] == "rope":
        n, H = case["n"], case["heads"]
        pool = n + 37
        axis, inv = _spread(case)
        pos = torch.randint(0, case["far"] + 1, (case["axes"], n), generator=g, device="cuda")
        s.update(x=(torch.randn(n, D, generator=g, device="cuda") * gain).to(dt), positions=pos,
                 slots=torch.randperm(pool, generator=g, device="cuda")[:n].contiguous(),
                 q_pe=torch.randn(n, H, 192, generator=g, device="cuda").to(dt)[..., 128:],
                 q=torch.randn(n, H, D, generator=g, device="cuda").to(dt),
                 codes=torch.zeros(pool, D, dtype=torch.uint8, device="cuda"),
                 scales=torch.zeros(pool, 2, dtype=torch.float32, device="cuda"),
                 axis=torch.tensor(axis, device="cuda"), inv=torch.tensor(inv, dtype=torch.float64, device="cuda"))
        if own:
            from quantized_kv_cache_kv8_gb300 import kvq
            s["rope"] = kvq.rope_layout(inv, axis, n_axes=case["axes"], adjacent=case["adjacent"])
            s["layout"] = kvq.mla_layout()
        return s
    past, new = _lengths(case)
    total = [p + n for p, n in zip(past, new)]
    table, _, _, n_pages = _table(past, new, case["page"], g)
    rows, n_tok, H = n_pages * case["page"], sum(new), case["heads"]
    tq4 = case["fmt"] == "tq4"
    codes = torch.empty(rows, D // 2 if tq4 else D, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, 2, dtype=torch.float32, device="cuda")
    th = torch.tensor([(a + b) / 2 for a, b in zip(LEVELS, LEVELS[1:])], device="cuda")
    th = torch.cat([-th.flip(0), torch.zeros(1, device="cuda"), th])
    step = 1 << 18
    for r in range(0, rows, step):
        m = min(step, rows - r)
        x = torch.randn(m, D, generator=g, device="cuda")
        if tq4:   # the rotated, normalized row is close to N(0, 1); its radius varies from row to row
            c = torch.bucketize(x, th).to(torch.uint8)
            codes[r:r + m] = c[:, 0::2] | (c[:, 1::2] << 4)
            scales[r:r + m] = 1.6 * torch.exp(0.2 * torch.randn(m, 2, generator=g, device="cuda"))
        else:
            x *= gain
            sc = torch.stack([x[:, :DL].abs().amax(1), x[:, DL:].abs().amax(1)], 1) / 448.0
            x[:, :DL] /= sc[:, :1]
            x[:, DL:] /= sc[:, 1:]
            codes[r:r + m] = x.to(torch.float8_e4m3fn).view(torch.uint8)
            scales[r:r + m] = sc
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    seq = [b for b, n in enumerate(new) for _ in range(n)]
    place = [i for n in new for i in range(n)]
    s.update(q=torch.randn(n_tok, H, D, generator=g, device="cuda").to(dt), codes=codes, scales=scales, table=table,
             kv_lens=torch.tensor(total, device="cuda"), cu=torch.tensor(cu, device="cuda"),
             seq=torch.tensor(seq, device="cuda"), place=torch.tensor(place, device="cuda"),
             out=torch.zeros(n_tok, H, DL, dtype=dt, device="cuda"), t_max=max(total), n_max=max(new))
    if tq4:
        s.update(signs=torch.tensor(_signs((DL, DR)), device="cuda"), h=(_hadamard(DL).cuda(), _hadamard(DR).cuda()),
                 levels=torch.tensor([-v for v in LEVELS[::-1]] + list(LEVELS), device="cuda"))
    if own:
        from quantized_kv_cache_kv8_gb300 import kvq
        s["fmt"] = kvq.KVQ_TQ4 if tq4 else kvq.KVQ_KV8
        s["layout"] = kvq.mla_layout(seed=SEED)
        s["ws"] = torch.zeros(kvq.kv_attn_paged_workspace_size(s["fmt"], len(past), H, n_tok, s["layout"],
                                                               bf16=case["dtype"] == "bf16"),
                              dtype=torch.uint8, device="cuda")
    return s


# -- one pass --------------------------------------------------------------------

def _plain_pages(s):
    P, lens, new, table, free = s["page"], s["lens"], s["new"], s["table"], s["free"]
    old, tot = (lens + P - 1) // P, (lens + new + P - 1) // P
    need = tot - old
    off = torch.cumsum(need, 0) - need
    cu = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(new, 0)])
    # reserve: the top of the free list first
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), new, output_size=s["n"])
    pos = lens[seq] + torch.arange(s["n"], device="cuda") - cu[seq]
    pg = pos // P
    last = len(free) - 1
    top = s["n_free"] - 1
    fresh = free[(top - off[seq] - (pg - old[seq])).clamp(0, last)]
    held = table[seq, pg]
    slots = torch.where(pg >= old[seq], fresh, held).long() * P + pos % P
    cols = torch.arange(table.shape[1], device="cuda")[None]
    mine = (cols >= old[:, None]) & (cols < tot[:, None])
    rank = off[:, None] + cols - old[:, None]
    table.copy_(torch.where(mine, free[(top - rank).clamp(0, last)], table))
    total = need.sum()
    s["n_free"] -= total.to(torch.int32)
    # trim back to the old lengths: the same pages return to the same places
    dst = torch.where(mine, s["n_free"] + total - 1 - rank, len(free))
    wide = torch.cat([free, free[:1]])
    wide[dst.flatten()] = table.flatten()
    free.copy_(wide[:-1])
    s["n_free"] += total.to(torch.int32)
    s["lens_out"].copy_(lens)
    s["cu"].copy_(cu)
    s["slots"].copy_(slots)
    s["positions"].copy_(pos)


def _plain_turn(x, cos, sin, adjacent):
    x = x.float()
    a, b = (x[..., 0::2], x[..., 1::2]) if adjacent else (x[..., :DR // 2], x[..., DR // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    return torch.stack([u, v], -1).flatten(-2) if adjacent else torch.cat([u, v], -1)


def _plain_rope(s):
    angle = s["positions"][s["axis"]].double() * s["inv"][:, None]   # [32, n]
    cos, sin = torch.cos(angle).float().T, torch.sin(angle).float().T
    adjacent = s["case"]["adjacent"]
    s["q"][..., DL:] = _plain_turn(s["q_pe"], cos[:, None], sin[:, None], adjacent).to(s["q"].dtype)
    left = s["x"][:, :DL].float()
    right = _plain_turn(s["x"][:, DL:], cos, sin, adjacent)
    sc = torch.stack([left.abs().amax(1), right.abs().amax(1)], 1) / 448.0
    safe = torch.where(sc > 0, sc, 1.0)
    y = torch.cat([left / safe[:, :1], right / safe[:, 1:]], 1)
    s["codes"][s["slots"]] = y.to(torch.float8_e4m3fn).view(torch.uint8)
    s["scales"][s["slots"]] = sc


def _plain_rotate(x, signs, h, inverse):
    left, right = h
    if inverse:   # the context lies in the latent block
        return (x @ left) * signs[:DL]
    y = x * signs
    return torch.cat([y[..., :DL] @ left, y[..., DL:] @ right], -1)


def _plain_attn(s):
    case, H, B = s["case"], s["case"]["heads"], s["case"]["n_seq"]
    P, T, N = case["page"], s["t_max"], s["n_max"]
    tq4 = case["fmt"] == "tq4"
    t = torch.arange(T, device="cuda")
    inside = t[None] < s["kv_lens"][:, None]
    slot = torch.where(inside, s["table"][:, t // P].long() * P + t % P, 0)
    if tq4:
        c = s["codes"][slot]
        x = s["levels"][torch.stack([c & 15, c >> 4], -1).flatten(-2).int()]
    else:
        x = s["codes"][slot].view(torch.float8_e4m3fn).float()
    sc = s["scales"][slot]
    x[..., :DL] *= sc[..., :1]
    x[..., DL:] *= sc[..., 1:]
    q = torch.zeros(B, N, H, D, device="cuda")
    q[s["seq"], s["place"]] = s["q"].float()
    if tq4:
        q = _plain_rotate(q, s["signs"], s["h"], False)
    z = torch.bmm(q.view(B, N * H, D), x.transpose(1, 2)).view(B, N, H, T).mul_(SM)
    past = s["kv_lens"] - (s["cu"][1:] - s["cu"][:-1])
    seen = t <= (past[:, None] + torch.arange(N, device="cuda"))[:, :, None]
    z.masked_fill_(~(seen & inside[:, None])[:, :, None], float("-inf"))
    z -= z.amax(-1, keepdim=True).clamp(min=-3e38)
    z.exp_()
    o = torch.bmm(z.view(B, N * H, T), x[..., :DL]).view(B, N, H, DL)
    o /= z.sum(-1, keepdim=True).clamp(min=1e-30)
    if tq4:
        o = _plain_rotate(o, s["signs"], s["h"], True)
    s["out"].copy_(o[s["seq"], s["place"]])


def run(state):
    s = state
    kind = s["case"]["kind"]
    if own:
        from quantized_kv_cache_kv8_gb300 import kvq
        if kind == "pages":
            kvq.kv_pages_reserve(s["lens"], s["new"], s["table"], s["free"], s["n_free"], s["page"], s["lens_out"],
                                 s["cu"], s["slots"], s["positions"], s["ws"])
            kvq.kv_pages_trim(s["lens_out"], s["lens"], s["table"], s["free"], s["n_free"], s["page"], s["ws"])
        elif kind == "rope":
            kvq.kv_rope_append(kvq.KVQ_KV8, s["rope"], s["x"], s["positions"], s["slots"], s["q_pe"], s["q"],
                               s["codes"], s["scales"], s["layout"])
        else:
            kvq.kv_attn_paged(s["fmt"], s["q"], s["cu"], s["codes"], s["scales"], s["table"], s["kv_lens"],
                              s["case"]["page"], s["out"], s["ws"], SM, s["layout"])
    elif kind == "pages":
        _plain_pages(s)
    elif kind == "rope":
        _plain_rope(s)
    else:
        _plain_attn(s)
    if kind == "pages":
        return dict(slots=s["slots"], positions=s["positions"], cu=s["cu"], lens=s["lens_out"], table=s["table"],
                    free=s["free"], n_free=s["n_free"])
    if kind == "rope":
        return dict(q=s["q"], codes=s["codes"].view(torch.float8_e4m3fn), scales=s["scales"])
    return s["out"]


# -- the definition in 64 bits ---------------------------------------------------

def exact(case, seed):
    if case["kind"] == "pages":
        return None   # whole numbers only
    s = prepare(case, seed)
    if case["kind"] == "rope":
        axis, inv = _spread(case)
        pos = s["positions"].cpu().numpy().astype(np.float64)
        ang = pos[axis] * np.array(inv)[:, None]
        cos, sin = np.cos(ang).T, np.sin(ang).T

        def turn(v, c, z):
            out = np.empty_like(v)
            i, j = (slice(0, None, 2), slice(1, None, 2)) if case["adjacent"] else (slice(0, 32), slice(32, 64))
            out[..., i] = v[..., i] * c - v[..., j] * z
            out[..., j] = v[..., j] * c + v[..., i] * z
            return out

        q = s["q"].double().cpu().numpy()
        q[..., DL:] = turn(s["q_pe"].double().cpu().numpy(), cos[:, None], sin[:, None])
        x = s["x"].double().cpu().numpy()
        x[:, DL:] = turn(x[:, DL:], cos, sin)
        scales = np.zeros(s["scales"].shape)
        scales[s["slots"].cpu().numpy()] = np.stack([np.abs(x[:, :DL]).max(1), np.abs(x[:, DL:]).max(1)], 1) / 448.0
        return dict(q=q, codes=None, scales=scales)
    past, new = _lengths(case)
    H, page = case["heads"], case["page"]
    cost = sum((p + n) * n for p, n in zip(past, new)) * H * 4.0 * D
    if cost > 6e12:
        return None
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b in range(len(past)):
        n, T = new[b], past[b] + new[b]
        if n:
            rows = (s["table"][b].long()[:, None] * page + torch.arange(page, device="cuda")).flatten()[:T]
            c = s["codes"][rows]
            if case["fmt"] == "tq4":
                y = torch.empty(T, D, dtype=torch.float64, device="cuda")
                y[:, 0::2], y[:, 1::2] = s["levels"].double()[(c & 15).long()], s["levels"].double()[(c >> 4).long()]
                sign = s["signs"].double()
                y[:, :DL] = sign[:DL] * (y[:, :DL] @ (s["h"][0].double() * math.sqrt(DL)).round() / math.sqrt(DL))
                y[:, DL:] = sign[DL:] * (y[:, DL:] @ (s["h"][1].double() * math.sqrt(DR)).round() / math.sqrt(DR))
            else:
                y = c.view(torch.float8_e4m3fn).double()
            scale = s["scales"][rows].double()
            y = y * torch.cat([scale[:, :1].expand(T, DL), scale[:, 1:].expand(T, DR)], 1)
            for i0 in range(0, n, 64):
                i1 = min(n, i0 + 64)
                z = torch.einsum("nhd,td->nht", s["q"][at + i0:at + i1].double(), y) * SM
                late = torch.arange(T, device="cuda")[None] > past[b] + torch.arange(i0, i1, device="cuda")[:, None]
                z[late[:, None].expand_as(z)] = -math.inf
                out[at + i0:at + i1] = torch.einsum("nht,td->nhd", torch.softmax(z, -1), y[:, :DL])
        at += n
    return out.cpu().numpy()


# -- what a pass cannot do without -------------------------------------------------

def work(case):
    if case["kind"] == "pages":
        past, new = _lengths(case)
        n, B, P = sum(new), len(past), case["page"]
        pages = sum(-(-(p + m) // P) - -(-p // P) for p, m in zip(past, new))
        held = sum(1 for p, m in zip(past, new) if m and p % P)
        return {"bytes": 8 * (4 * B + 1) + 16 * n + 4 * (4 * pages + held) + 8, "flops": 4 * n + 8 * B}
    if case["kind"] == "rope":
        n, H, e = case["n"], case["heads"], 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * (2 * H * DR * e + D * e + 8 * case["axes"] + 8 + D + 8), "flops": n * ((H + 1) * 3 * DR + 3 * D)}
    past, new = _lengths(case)
    H, e = case["heads"], 2 if case["dtype"] == "bf16" else 4
    row = (D // 2 if case["fmt"] == "tq4" else D) + 8
    seen = sum(n * p + n * (n + 1) // 2 for p, n in zip(past, new))
    rows = sum(p + n for p, n in zip(past, new) if n)
    return {"bytes": rows * row + sum(new) * H * (D + DL) * e + 4 * (rows // case["page"]), "flops": seen * H * 2 * (D + DL)}
