"""What is measured of the beam-search step over KV8 caches with separate keys and values: cases, inputs, plain forms.

A model with grouped query heads keeps a key row and a value row per token and
key-value head, each in e4m3 codes with one f32 scale, in pages of a pool
[n_pages][n_kv_heads][page_rows][head_dim].  Four operators of its serving step,
with beam search or without:

* append  kv_gqa_append: rotary positions on the queries and the new keys, keys
          and values quantized into their slots.
* attn    kv_gqa_attn_paged: every new token over its sequence's rows; causal, or
          unmasked over an encoder's states of another length (cross attention).
* select  kv_beam_select: the best continuations of every request over its beams
          and the vocabulary.
* fork    kv_pages_fork / kv_pages_copy: block tables follow the chosen parents,
          full pages shared, the page in progress copied, dropped pages freed.
"""
import math
import random

import torch

own = False

TILE = 512   # tokens of one sequence that the plain forms take at once


# -- cases ---------------------------------------------------------------------

def listed():
    return [
        # a decode step's queries and rows, far positions
        dict(name="append_decode_64", kind="append", n=64, heads=32, kv_heads=8, dim=128, rot=128, dtype="bf16",
             axes=1, adjacent=False, page=64, far=131072),
        # an odd prefill chunk, wide heads of which a part turns
        dict(name="append_chunk_1999", kind="append", n=1999, heads=16, kv_heads=2, dim=256, rot=64, dtype="bf16",
             axes=1, adjacent=True, page=32, far=32768),
        # one short request: latency
        dict(name="attn_decode_1x300", kind="attn", causal=True, dtype="bf16", heads=32, kv_heads=8, dim=128, n_seq=1,
             page=16, past_lo=299, past_hi=299, new_lo=1, new_hi=1),
        # the decode step of 4 sequences of 32768 rows, 2 wide heads
        dict(name="attn_decode_4x32768", kind="attn", causal=True, dtype="bf16", heads=16, kv_heads=2, dim=256, n_seq=4,
             page=64, past_lo=32767, past_hi=32767, new_lo=1, new_hi=1),
        # ragged long-context decode
        dict(name="attn_decode_ragged_32", kind="attn", causal=True, dtype="bf16", heads=32, kv_heads=8, dim=128,
             n_seq=32, page=64, past_lo=1024, past_hi=65535, new_lo=1, new_hi=1),
        # a prefill chunk over a prefix
        dict(name="attn_chunk_512_past_8192", kind="attn", causal=True, dtype="bf16", heads=32, kv_heads=8, dim=128,
             n_seq=1, page=64, past_lo=8192, past_hi=8192, new_lo=512, new_hi=512),
        # 4 beams of 16 requests read their encoder's states
        dict(name="cross_beams_16x4", kind="attn", causal=False, dtype="bf16", heads=16, kv_heads=16, dim=64, n_seq=16,
             page=64, past_lo=100, past_hi=1500, new_lo=4, new_hi=4),
        # decoder prompts over encoder states, f32, odd lengths, some encoders empty
        dict(name="cross_prompts_8_f32", kind="attn", causal=False, dtype="f32", heads=32, kv_heads=8, dim=128, n_seq=8,
             page=32, past_lo=0, past_hi=1501, new_lo=1, new_hi=77),
        # a few requests, small vocabulary: latency
        dict(name="select_8x4_32768", kind="select", n_seq=8, beams=4, keep=8, vocab=32768, dtype="f32", dead=0.0),
        # a large batch over a large vocabulary
        dict(name="select_64x8_131072", kind="select", n_seq=64, beams=8, keep=16, vocab=131072, dtype="bf16", dead=0.05),
        # 16 requests of 4 beams, one layer's pools
        dict(name="fork_16x4", kind="fork", n_req=16, beams=4, prompt_lo=500, prompt_hi=4000, gen=150, page=64,
             kv_heads=8, dim=128, layers=1),
        # 64 requests of 8 beams, 8 layers' pools, small pages
        dict(name="fork_64x8", kind="fork", n_req=64, beams=8, prompt_lo=100, prompt_hi=1500, gen=99, page=16,
             kv_heads=2, dim=256, layers=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _heads(rng):
    kv = rng.choice([1, 2, 4, 8, 16])
    return kv * rng.choice([1, 2, 3, 4, 5, 8] if kv > 2 else [1, 4, 7, 8, 16]), kv


def draw(rng):
    kind = rng.choice(["append", "attn", "attn", "cross", "select", "fork"])
    page = rng.choice([16, 32, 64, 128, 256])
    dim = rng.choice([64, 128, 128, 256])
    heads, kv = _heads(rng)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "append":
        return dict(kind="append", n=_log(rng, 1, 2048 * 16 * 128 // (heads * dim) if heads * dim > 2048 else 2048),
                    heads=heads, kv_heads=kv, dim=dim, rot=rng.choice([16, 64, min(dim, 128)]), dtype=dtype,
                    axes=rng.choice([1, 1, 3]), adjacent=rng.random() < 0.5, page=page, far=_log(rng, 100, 1 << 20))
    if kind == "cross":
        new = _log(rng, 1, 128)
        return dict(kind="attn", causal=False, dtype=dtype, heads=heads, kv_heads=kv, dim=dim, n_seq=_log(rng, 1, 32),
                    page=page, past_lo=rng.choice([0, 1, 50]), past_hi=_log(rng, 60, 3000), new_lo=rng.choice([1, new]),
                    new_hi=new)
    if kind == "attn":
        form = rng.choice(["decode", "decode", "window", "chunk"])
        if form == "decode":
            n_seq = _log(rng, 1, 128)
            hi = _log(rng, 64, max(64, min(131071, 120000000 // (n_seq * kv * dim))))
            lo, new = max(1, hi // 16), 1
        elif form == "window":
            n_seq, hi, new = _log(rng, 1, 48), _log(rng, 64, 6000), _log(rng, 2, 16)
            lo = 0
        else:
            n_seq, new = 1, _log(rng, 16, 600)
            lo = hi = rng.choice([0, _log(rng, 16, 6000)])
        return dict(kind="attn", causal=True, dtype=dtype, heads=heads, kv_heads=kv, dim=dim, n_seq=n_seq, page=page,
                    past_lo=lo, past_hi=hi, new_lo=new if form != "window" else 0, new_hi=new)
    if kind == "select":
        beams = rng.choice([1, 2, 3, 4, 5, 8, 16])
        n_seq, vocab = _log(rng, 1, 64), _log(rng, 50, 140001)
        n_seq = max(1, min(n_seq, (1 << 26) // (beams * vocab)))
        return dict(kind="select", n_seq=n_seq, beams=beams, keep=rng.choice([1, beams, 2 * beams]), vocab=vocab,
                    dtype=dtype, dead=rng.choice([0.0, 0.3]))
    beams = rng.choice([1, 2, 3, 4, 8, 16])
    return dict(kind="fork", n_req=_log(rng, 1, 512 // beams), beams=beams, prompt_lo=rng.choice([0, 1, 100]),
                prompt_hi=_log(rng, 100, 4000), gen=_log(rng, 1, 300), page=page, kv_heads=rng.choice([1, 2]), dim=dim,
                layers=rng.choice([1, 2, 4]))


def _rng(case):
    return random.Random("%s" % sorted((k, v) for k, v in case.items() if k != "name"))


def _lengths(case):
    """(rows, new tokens) of every sequence, from the case alone; a causal sequence's rows end with its new tokens."""
    r = _rng(case)
    past = [r.randint(case["past_lo"], case["past_hi"]) for _ in range(case["n_seq"])]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["n_seq"])]
    if sum(new) == 0:
        new[0] = 1
    return ([p + n for p, n in zip(past, new)] if case["causal"] else past), new


def _spread(case):
    """(axis, inverse frequency) of each rotary pair."""
    n, a = case["rot"] // 2, case["axes"]
    return [min(a - 1, i * a // n) for i in range(n)], [10000.0 ** (-i / n) for i in range(n)]


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


# -- inputs --------------------------------------------------------------------

def _encode(x):
    """(codes, scale) of rows: amax / 448 and the nearest e4m3."""
    sc = x.abs().amax(-1) / 448.0
    y = x / torch.where(sc > 0, sc, 1.0)[..., None]
    return y.to(torch.float8_e4m3fn).view(torch.uint8), sc


def _prepare_fork(case, seed, g):
    r = _rng(case)
    n_req, beams, page = case["n_req"], case["beams"], case["page"]
    n = n_req * beams
    prompt = [r.randint(case["prompt_lo"], case["prompt_hi"]) for _ in range(n_req)]
    gen = [r.randint(0, case["gen"]) for _ in range(n_req)]
    width = max(-(-(p + q) // page) for p, q in zip(prompt, gen)) + 1
    most = n * width + n + 5
    r = _rng(dict(case, seed=seed))   # sizes are the case's, the rest the seed's
    order = list(range(most))
    r.shuffle(order)
    table, at = [[0] * width for _ in range(n)], 0
    for i in range(n_req):   # full pages of the prompt shared, the rest each beam's own
        shared, total = prompt[i] // page, -(-(prompt[i] + gen[i]) // page)
        for b in range(beams):
            table[i * beams + b][:shared] = order[at:at + shared]
        at += shared
        for b in range(beams):
            table[i * beams + b][shared:total] = order[at:at + total - shared]
            at += total - shared
    n_free = min(most - at, 2 * n + 5)
    # the pool: the pages in use and the free ones, renumbered without gaps
    used = sorted(order[:at + n_free])
    number = {p: k for k, p in enumerate(used)}
    table = [[number.get(p, 0) for p in row] for row in table]
    n_pages = len(used)
    free = [number[p] for p in order[at:at + n_free]] + [0] * (n_pages - n_free)
    parents = []
    for i in range(n_req):   # the best beams have several children
        ps = [min(int(r.expovariate(0.8)), beams - 1) for _ in range(beams)]
        parents += [i * beams + p for p in ps]
    if n_req > 3:   # a finished request
        parents[-beams:] = [-1] * beams
    H, D = case["kv_heads"], case["dim"]
    pools = []
    for _ in range(case["layers"]):
        pools += [torch.randint(0, 127, (n_pages, H, page, D), generator=g, device="cuda", dtype=torch.uint8),
                  torch.randint(0, 127, (n_pages, H, page, D), generator=g, device="cuda", dtype=torch.uint8),
                  torch.rand(n_pages, H, page, 2, generator=g, device="cuda")]
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(parents=torch.tensor(parents, **i32), table=torch.tensor(table, **i32),
                lens=torch.tensor([prompt[i // beams] + gen[i // beams] for i in range(n)], device="cuda"),
                free=torch.tensor(free, **i32), n_free=torch.tensor([n_free], **i32), pools=pools, n_pages=n_pages,
                copies=torch.full((n, 2), -1, **i32))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 11)
    s = dict(case=case)
    kind = case["kind"]
    if own:
        from quantized_kv_cache_kv8_gb300 import kvq
    if kind == "fork":
        s.update(_prepare_fork(case, seed, g))
        if own:
            s["ws"] = torch.zeros(kvq.kv_pages_fork_workspace_size(s["table"].shape[0], s["table"].shape[1], s["n_pages"]),
                                  dtype=torch.uint8, device="cuda")
        return s
    dt = _dtype(case)
    if kind == "select":
        n, b, v = case["n_seq"], case["beams"], case["vocab"]
        logits = torch.randn(n, b, v, generator=g, device="cuda", dtype=torch.float32)
        logits = (logits * 2.5 + torch.randn(v, generator=g, device="cuda")).to(dt)
        scores = -5.0 * torch.rand(n, b, generator=g, device="cuda")
        scores[torch.rand(n, b, generator=g, device="cuda") < case["dead"]] = -math.inf
        # tokens that may not come next
        logits[..., torch.randint(0, v, (max(1, v // 100),), generator=g, device="cuda")] = -math.inf
        s.update(logits=logits, scores=scores, out_scores=torch.zeros(n, case["keep"], device="cuda"),
                 parents=torch.zeros(n, case["keep"], dtype=torch.int32, device="cuda"),
                 tokens=torch.zeros(n, case["keep"], dtype=torch.int32, device="cuda"))
        if own:
            s["ws"] = torch.zeros(kvq.kv_beam_workspace_size(n, b, v, case["keep"]), dtype=torch.uint8, device="cuda")
        return s
    H, D, P, Hq = case["kv_heads"], case["dim"], case["page"], case["heads"]
    gain = torch.exp(0.5 * torch.randn(D, generator=g, device="cuda"))
    if kind == "append":
        n = case["n"]
        pages = -(-(n + 37) // P)
        axis, inv = _spread(case)
        s.update(q=torch.randn(n, Hq, D, generator=g, device="cuda").to(dt), q_out=torch.zeros(n, Hq, D, dtype=dt, device="cuda"),
                 k=(torch.randn(n, H, D, generator=g, device="cuda") * gain).to(dt),
                 v=torch.randn(n, H, D, generator=g, device="cuda").to(dt),
                 positions=torch.randint(0, case["far"] + 1, (case["axes"], n), generator=g, device="cuda"),
                 slots=torch.randperm(pages * P, generator=g, device="cuda")[:n].contiguous(),
                 k_codes=torch.zeros(pages, H, P, D, dtype=torch.uint8, device="cuda"),
                 v_codes=torch.zeros(pages, H, P, D, dtype=torch.uint8, device="cuda"),
                 scales=torch.zeros(pages, H, P, 2, device="cuda"),
                 axis=torch.tensor(axis, device="cuda"), inv=torch.tensor(inv, dtype=torch.float64, device="cuda"))
        if own:
            s["rope"] = kvq.rope_layout(inv, axis, n_axes=case["axes"], adjacent=case["adjacent"])
        return s
    lens, new = _lengths(case)
    need = [-(-t // P) for t in lens]
    n_pages, width = sum(need) + 7, max(1, max(need))
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    cols, needed = torch.arange(width, device="cuda")[None], torch.tensor(need, device="cuda")[:, None]
    first = torch.cumsum(needed, 0) - needed
    table = torch.where(cols < needed, order[(first + cols).clamp(max=n_pages - 1)], 0).to(torch.int32).contiguous()
    k_codes = torch.empty(n_pages, H, P, D, dtype=torch.uint8, device="cuda")
    v_codes, scales = torch.empty_like(k_codes), torch.empty(n_pages, H, P, 2, device="cuda")
    step = max(1, (1 << 26) // (H * P * D))
    for i in range(0, n_pages, step):
        m = min(step, n_pages - i)
        k_codes[i:i + m], scales[i:i + m, ..., 0] = _encode(torch.randn(m, H, P, D, generator=g, device="cuda") * gain)
        v_codes[i:i + m], scales[i:i + m, ..., 1] = _encode(torch.randn(m, H, P, D, generator=g, device="cuda"))
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    n_tok = sum(new)
    s.update(q=torch.randn(n_tok, Hq, D, generator=g, device="cuda").to(dt), k_codes=k_codes, v_codes=v_codes, scales=scales,
             table=table, kv_lens=torch.tensor(lens, device="cuda"), cu=torch.tensor(cu, device="cuda"), lens=lens, new=new,
             out=torch.zeros(n_tok, Hq, D, dtype=dt, device="cuda"), sm=1.0 / math.sqrt(D))
    if own:
        s["ws"] = torch.zeros(kvq.kv_gqa_attn_paged_workspace_size(len(new), Hq, H, D, n_tok, bf16=dt == torch.bfloat16),
                              dtype=torch.uint8, device="cuda")
    return s


# -- one pass --------------------------------------------------------------------

def _plain_turn(x, cos, sin, adjacent):
    a, b = (x[..., 0::2], x[..., 1::2]) if adjacent else x.chunk(2, -1)
    u, v = a * cos - b * sin, b * cos + a * sin
    return torch.stack([u, v], -1).flatten(-2) if adjacent else torch.cat([u, v], -1)


def _plain_append(s):
    case = s["case"]
    rot, adjacent, P = case["rot"], case["adjacent"], case["page"]
    angle = s["positions"][s["axis"]].double() * s["inv"][:, None]   # [pairs, n]
    cos, sin = torch.cos(angle).float().T[:, None], torch.sin(angle).float().T[:, None]
    q, k = s["q"].float(), s["k"].float()
    q = torch.cat([_plain_turn(q[..., :rot], cos, sin, adjacent), q[..., rot:]], -1)
    k = torch.cat([_plain_turn(k[..., :rot], cos, sin, adjacent), k[..., rot:]], -1)
    s["q_out"].copy_(q)
    page, place = s["slots"] // P, s["slots"] % P
    kc, ks = _encode(k)
    vc, vs = _encode(s["v"].float())
    s["k_codes"][page, :, place] = kc
    s["v_codes"][page, :, place] = vc
    s["scales"][page, :, place] = torch.stack([ks, vs], -1)


def _plain_attn(s):
    case = s["case"]
    H, D, P, G = case["kv_heads"], case["dim"], case["page"], case["heads"] // case["kv_heads"]
    at = 0
    for b, (T, n) in enumerate(zip(s["lens"], s["new"])):
        if n and not T:
            s["out"][at:at + n] = 0
        if n and T:
            pages = s["table"][b, :-(-T // P)].long()
            sc = s["scales"][pages].transpose(0, 1).reshape(H, -1, 2)[:, :T]
            k = s["k_codes"][pages].transpose(0, 1).reshape(H, -1, D)[:, :T].view(torch.float8_e4m3fn).float()
            v = s["v_codes"][pages].transpose(0, 1).reshape(H, -1, D)[:, :T].view(torch.float8_e4m3fn).float()
            k *= sc[..., :1]
            v *= sc[..., 1:]
            for i in range(0, n, TILE):
                m = min(TILE, n - i)
                q = s["q"][at + i:at + i + m].float().view(m, H, G, D).permute(1, 0, 2, 3).reshape(H, m * G, D)
                z = torch.bmm(q, k.transpose(1, 2)).view(H, m, G, T) * s["sm"]
                if case["causal"]:
                    t, last = torch.arange(T, device="cuda"), T - n + i + torch.arange(m, device="cuda")
                    z.masked_fill_((t[None] > last[:, None])[None, :, None], -math.inf)
                z = torch.exp(z - z.amax(-1, keepdim=True)).view(H, m * G, T)
                o = torch.bmm(z, v) / z.sum(-1, keepdim=True)
                s["out"][at + i:at + i + m] = o.view(H, m, G, D).permute(1, 0, 2, 3).reshape(m, H * G, D)
        at += n


def _plain_select(s):
    case = s["case"]
    n, b, v, keep = case["n_seq"], case["beams"], case["vocab"], case["keep"]
    per = min(keep, v)
    x = s["logits"].float()
    x = torch.where(torch.isnan(x), -math.inf, x)
    top = x.amax(-1, keepdim=True)
    # the score of a beam's token is compared with other beams': in 64 bits
    mass = torch.where(x == top, 1.0, torch.exp(x - top)).sum(-1, dtype=torch.float64)
    val, tok = torch.sort(x, dim=-1, descending=True, stable=True)
    val, tok = val[..., :per], tok[..., :per]
    own_part = torch.where(val == top, 0.0, val.double() - top.double()) - torch.log(mass)[..., None]
    scores = s["scores"].double()[..., None] + own_part
    ok = torch.isfinite(s["scores"])[..., None] & (val > -math.inf)
    scores = torch.where(ok, scores, -math.inf).view(n, b * per)
    if b * per < keep:
        scores = torch.cat([scores, torch.full((n, keep - b * per), -math.inf, dtype=torch.float64, device="cuda")], 1)
    best, at = torch.sort(scores, dim=-1, descending=True, stable=True)
    best, at = best[:, :keep], at[:, :keep]
    found = best > -math.inf
    at = at.clamp(max=b * per - 1)
    first = torch.arange(n, device="cuda")[:, None] * b
    s["out_scores"].copy_(best)
    s["parents"].copy_(torch.where(found, first + at // per, -1))
    s["tokens"].copy_(torch.where(found, torch.gather(tok.reshape(n, b * per), 1, at), -1))


def _plain_fork(s):
    par, lens, table, free, P, N = s["parents"].long(), s["lens"], s["table"], s["free"], s["case"]["page"], s["n_pages"]
    n, width = table.shape
    rows = torch.arange(n, device="cuda")
    cols = torch.arange(width, device="cuda")[None]
    live = par >= 0
    src = par.clamp(min=0)
    held = cols < ((lens + P - 1) // P)[:, None]
    children = torch.zeros(n, dtype=torch.int64, device="cuda").scatter_add_(0, src, live.long())
    first = torch.full((n,), n, device="cuda").scatter_reduce_(0, src, torch.where(live, rows, n), "amin")
    # a page in progress stays with its sequence's first child; the others get a copy
    need = live & (first[src] != rows) & (lens[src] % P != 0)
    rank = torch.cumsum(need.long(), 0) - 1
    top = s["n_free"].long()
    fresh = free[(top - 1 - rank).clamp(0, N - 1)]
    last = (lens[src] // P).clamp(max=width - 1)
    s["copies"].copy_(torch.where(need[:, None], torch.stack([table[src, last], fresh], 1), -1))
    # pages that no sequence holds any more, at their first holder's place
    id_ = torch.where(held, table, N).long()
    kept = torch.zeros(N + 1, dtype=torch.int64, device="cuda")
    kept.scatter_reduce_(0, torch.where((children > 0)[:, None], id_, N).flatten(), torch.ones(n * width, dtype=torch.int64,
                                                                                            device="cuda"), "amax")
    kept[N] = 1
    flat = torch.arange(n * width, device="cuda")
    owner = torch.full((N + 1,), n * width, device="cuda").scatter_reduce_(0, id_.flatten(), flat, "amin")
    gone = ((kept[id_] == 0) & (owner[id_] == flat.view(n, width))).flatten()
    total, copied = gone.long().sum(), need.long().sum()
    where = torch.where(gone, top - copied + total - torch.cumsum(gone.long(), 0), N)
    wide = torch.cat([free, free[:1]])
    wide[where] = table.flatten()
    new = torch.where((live[:, None] & (cols < ((lens[src] + P - 1) // P)[:, None])), table[src], table)
    new = torch.where(need[:, None] & (cols == last[:, None]), fresh[:, None], new)
    free.copy_(wide[:N])
    table.copy_(new)
    s["n_free"] += (total - copied).to(torch.int32)
    lens.copy_(torch.where(live, lens[src], 0))
    pairs = s["copies"][need].long()
    for pool in s["pools"]:
        pool[pairs[:, 1]] = pool[pairs[:, 0]]


def run(state):
    s = state
    case = s["case"]
    kind = case["kind"]
    if own:
        from quantized_kv_cache_kv8_gb300 import kvq
        if kind == "append":
            kvq.kv_gqa_append(s["rope"], s["k"], s["v"], s["positions"], s["slots"], s["q"], s["q_out"], s["k_codes"],
                              s["v_codes"], s["scales"])
        elif kind == "attn":
            kvq.kv_gqa_attn_paged(s["q"], s["cu"], s["k_codes"], s["v_codes"], s["scales"], s["table"], s["kv_lens"],
                                  s["out"], s["ws"], s["sm"], causal=case["causal"])
        elif kind == "select":
            kvq.kv_beam_select(s["logits"], s["scores"], s["out_scores"], s["parents"], s["tokens"], s["ws"])
        else:
            kvq.kv_pages_fork(s["parents"], s["lens"], s["table"], s["free"], s["n_free"], case["page"], s["copies"], s["ws"])
            kvq.kv_pages_copy(s["copies"], s["pools"], s["ws"])
    else:
        dict(append=_plain_append, attn=_plain_attn, select=_plain_select, fork=_plain_fork)[kind](s)
    if kind == "append":
        return dict(q=s["q_out"], k=s["k_codes"].view(torch.float8_e4m3fn), v=s["v_codes"].view(torch.float8_e4m3fn),
                    scales=s["scales"])
    if kind == "attn":
        return s["out"]
    if kind == "select":
        return dict(scores=s["out_scores"], parents=s["parents"], tokens=s["tokens"])
    return dict(table=s["table"], lens=s["lens"], free=s["free"], n_free=s["n_free"], copies=s["copies"],
                pools=[p.view(torch.float8_e4m3fn) if p.dtype == torch.uint8 else p for p in s["pools"]])


# -- the definition in 64 bits ---------------------------------------------------

def exact(case, seed):
    kind = case["kind"]
    if kind == "fork":
        return None   # whole numbers, and values moved as they are
    if kind == "attn":
        lens, new = _lengths(case)
        if sum(t * n for t, n in zip(lens, new)) * case["heads"] * 4.0 * case["dim"] > 2e12:
            return None
    s = prepare(case, seed)
    if kind == "append":
        axis, inv = _spread(case)
        w = torch.tensor(inv, dtype=torch.float64, device="cuda")
        phase = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["positions"].double()[axis].T * w)[:, None]
        rot = case["rot"]

        def turn(x):
            x = x.double().clone()
            pairs = x[..., :rot].unflatten(-1, (rot // 2, 2)) if case["adjacent"] else \
                x[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * phase)
            x[..., :rot] = (y if case["adjacent"] else y.transpose(-1, -2)).flatten(-2)
            return x

        q, k, v = turn(s["q"]), turn(s["k"]), s["v"].double()
        scales = torch.zeros(s["scales"].shape, dtype=torch.float64, device="cuda")
        at = s["slots"]
        for i, x in enumerate((k, v)):
            scales.select(-1, i)[at // case["page"], :, at % case["page"]] = x.abs().amax(-1) / 448.0
        return dict(q=q.cpu().numpy(), k=None, v=None, scales=scales.cpu().numpy())
    if kind == "select":
        n, b, keep = case["n_seq"], case["beams"], case["keep"]
        out = torch.full((n, keep), -math.inf, dtype=torch.float64)
        for i in range(n):
            alive = torch.isfinite(s["scores"][i])
            if alive.any():
                p = s["logits"][i][alive].double()
                p = p - torch.logsumexp(p, -1, keepdim=True) + s["scores"][i][alive].double()[:, None]
                best = torch.topk(p.flatten(), min(keep, p.numel())).values
                out[i, :best.numel()] = best.cpu()
        return dict(scores=out.numpy(), parents=None, tokens=None)
    H, D, P = case["kv_heads"], case["dim"], case["page"]
    G = case["heads"] // H
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (T, n) in enumerate(zip(lens, new)):
        row = torch.arange(T, device="cuda")
        page, place = s["table"][b].long()[row // P], row % P
        for h in range(H if n and T else 0):
            sc = s["scales"][page, h, place].double()
            k = s["k_codes"][page, h, place].view(torch.float8_e4m3fn).double() * sc[:, :1]
            v = s["v_codes"][page, h, place].view(torch.float8_e4m3fn).double() * sc[:, 1:]
            for i in range(0, n, 128):
                j = min(n, i + 128)
                z = torch.einsum("ngd,td->ngt", s["q"][at + i:at + j, h * G:(h + 1) * G].double(), k) * s["sm"]
                if case["causal"]:
                    late = row[None] > T - n + torch.arange(i, j, device="cuda")[:, None]
                    z[late[:, None].expand_as(z)] = -math.inf
                out[at + i:at + j, h * G:(h + 1) * G] = torch.einsum("ngt,td->ngd", torch.softmax(z, -1), v)
        at += n
    return out.cpu().numpy()


# -- what a pass cannot do without -------------------------------------------------

def work(case):
    kind = case["kind"]
    if kind == "fork":
        n = case["n_req"] * case["beams"]
        rows = (case["prompt_lo"] + case["prompt_hi"] + case["gen"]) // 2
        pages = n * -(-rows // case["page"])
        page = case["kv_heads"] * case["page"] * (2 * case["dim"] + 8) * case["layers"]
        copies = n // 2   # about: a parent's further children
        return {"bytes": 8 * pages + 8 * n + 2 * copies * page, "flops": pages}
    e = 2 if case["dtype"] == "bf16" else 4
    if kind == "select":
        n = case["n_seq"] * case["beams"] * case["vocab"]
        return {"bytes": n * e + 12 * case["n_seq"] * case["keep"], "flops": 4 * n}
    H, Hq, D = case["kv_heads"], case["heads"], case["dim"]
    if kind == "append":
        n = case["n"]
        return {"bytes": n * (2 * Hq * D * e + 2 * H * D * e + 8 * case["axes"] + 8 + H * (2 * D + 8)),
                "flops": n * ((Hq + H) * 3 * case["rot"] + 6 * H * D)}
    lens, new = _lengths(case)
    seen = sum(n * t - (n * (n - 1) // 2 if case["causal"] else 0) for t, n in zip(lens, new))
    rows = sum(t for t, n in zip(lens, new) if n)
    return {"bytes": rows * H * (2 * D + 8) + 2 * sum(new) * Hq * D * e + 4 * (rows // case["page"]), "flops": seen * Hq * 4 * D}
