"""Paged pools on the GPU: page bookkeeping against a plain list simulation, the
rotary append against f64 rotation and the oracle's encoders, attention against
f64 softmax attention over the oracle's reconstruction, and the three together."""
import math

import numpy as np
import pytest
import torch

from gpu_common import SIMT_TOL, TENSOR_TOL, gpu_encode, kvq_module, rel_err, to_dev
from quantized_kv_cache_kv8_gb300 import synth

pytestmark = pytest.mark.gpu
SM = 1.0 / math.sqrt(192.0)
# an output rounded once to bf16 is off by at most half a step, 2^-8 of its value
BF16_STEP = 2.0 ** -8


@pytest.fixture(scope="module")
def kvq():
    return kvq_module()


# -- pages ----------------------------------------------------------------------

class Pages:
    """Sequences' pages as plain lists."""

    def __init__(self, kvq, lens, page, stride, n_pages, seed=0):
        rng = np.random.default_rng(seed)
        self.kvq, self.page, self.n_pages = kvq, page, n_pages
        order = rng.permutation(n_pages).tolist()
        self.lens = list(lens)
        self.pages = []
        for n in lens:
            k = -(-n // page)
            self.pages.append(order[:k])
            order = order[k:]
        self.stack = order
        table = np.full((len(lens), stride), -9, np.int32)
        for s, p in enumerate(self.pages):
            table[s, :len(p)] = p
        free = np.full(n_pages, -1, np.int32)
        free[:len(order)] = order
        self.d_lens, self.d_table, self.d_free = to_dev(np.array(lens, np.int64)), to_dev(table), to_dev(free)
        self.d_n = to_dev(np.array([len(order)], np.int32))
        self.ws = torch.zeros(kvq.kv_pages_workspace_size(), dtype=torch.uint8, device="cuda")

    def reserve(self, new, max_new=None, in_place=True, want_pos=True):
        B = len(self.lens)
        m = sum(new) if max_new is None else max_new
        out = self.d_lens if in_place else torch.empty_like(self.d_lens)
        cu = torch.full((B + 1,), 77, dtype=torch.int64, device="cuda")
        slots = torch.full((m,), 77, dtype=torch.int64, device="cuda")
        pos = torch.full((m,), 77, dtype=torch.int64, device="cuda") if want_pos else None
        self.kvq.kv_pages_reserve(self.d_lens, to_dev(np.array(new, np.int64)), self.d_table, self.d_free, self.d_n,
                                  self.page, out, cu, slots, pos, self.ws)
        return out, cu.cpu().numpy(), slots.cpu().numpy(), None if pos is None else pos.cpu().numpy()

    def model_reserve(self, new):
        slots, pos = [], []
        for s, n in enumerate(new):
            for i in range(n):
                t = self.lens[s] + i
                if t // self.page == len(self.pages[s]):
                    self.pages[s].append(self.stack.pop())
                slots.append(self.pages[s][t // self.page] * self.page + t % self.page)
                pos.append(t)
            self.lens[s] += n
        return slots, pos

    def model_trim(self, keep):
        for s in reversed(range(len(keep))):
            k = self.lens[s] if keep[s] < 0 or keep[s] > self.lens[s] else keep[s]
            while len(self.pages[s]) > -(-k // self.page):
                self.stack.append(self.pages[s].pop())
            self.lens[s] = k

    def check(self):
        n = int(self.d_n.item())
        assert n == len(self.stack)
        assert self.d_free.cpu().numpy()[:n].tolist() == self.stack
        table = self.d_table.cpu().numpy()
        for s, p in enumerate(self.pages):
            assert table[s, :len(p)].tolist() == p
        assert self.d_lens.cpu().numpy().tolist() == self.lens
        assert int(self.ws[4:8].view(torch.int32).item()) == 0


@pytest.mark.parametrize("n_seq,page,past,new", [
    (1, 16, 0, 1), (1, 64, 130, 5000), (3, 1, 5, 4), (64, 64, 500, 1), (513, 16, 100, 9), (1500, 32, 60, 40),
    (512, 128, 1000, 0),
])
def test_pages_follow_the_list_model(kvq, n_seq, page, past, new):
    rng = np.random.default_rng(n_seq)
    lens = rng.integers(0, past + 1, n_seq).tolist()
    lens[0] = page * (past // page)          # a full last page (or none)
    n_pages = sum(-(-n // page) for n in lens) + n_seq * (3 * new // page + 3)
    p = Pages(kvq, lens, page, (past + 3 * new) // page + 3, n_pages)
    for step in range(3):
        add = rng.integers(0, new + 1, n_seq).tolist()
        pad = 0 if step == 0 else 37 * step
        before = list(p.lens)
        out, cu, slots, pos = p.reserve(add, max_new=sum(add) + pad, in_place=step != 1)
        ref_slots, ref_pos = p.model_reserve(add)
        assert cu.tolist() == np.concatenate([[0], np.cumsum(add)]).tolist()
        assert slots.tolist() == ref_slots + [-1] * pad
        assert pos.tolist() == ref_pos + [0] * pad
        assert out.cpu().numpy().tolist() == p.lens
        if step == 1:
            assert p.d_lens.cpu().numpy().tolist() == before
            p.d_lens.copy_(out)
        p.check()
        keep = [b + int(rng.integers(0, a + 1)) if rng.random() < 0.7 else -1 for a, b in zip(add, before)]
        keep[int(rng.integers(0, n_seq))] = 0
        p.kvq.kv_pages_trim(p.d_lens, to_dev(np.array(keep, np.int64)), p.d_table, p.d_free, p.d_n, page, p.ws)
        p.model_trim(keep)
        p.check()
        assert kvq.read_device_error(p.ws) == 0


def test_pages_trim_undoes_a_reservation(kvq):
    p = Pages(kvq, [100, 0, 64, 31], 32, 40, 64)
    free, lens = p.d_free.clone(), p.d_lens.clone()
    p.reserve([70, 200, 1, 0], in_place=True)
    kvq.kv_pages_trim(p.d_lens, lens, p.d_table, p.d_free, p.d_n, 32, p.ws)
    assert torch.equal(p.d_free, free) and torch.equal(p.d_lens, lens)
    p.check()


@pytest.mark.parametrize("new,max_new,stride,status", [
    ([400, 400], None, 40, 3),      # more pages than are free
    ([10, 700], 5, 40, 1),          # more rows than the slot map holds
    ([10, 700], None, 8, 1),        # a table row too short
    ([-1, 10], 20, 40, 1),
])
def test_pages_reserve_is_all_or_nothing(kvq, new, max_new, stride, status):
    p = Pages(kvq, [100, 3], 16, stride, 40)
    table, free = p.d_table.clone(), p.d_free.clone()
    out, cu, slots, pos = p.reserve(new, max_new=max_new, in_place=False)
    assert np.all(cu == 0) and np.all(slots == -1) and np.all(pos == 0)
    assert torch.equal(out, p.d_lens) and torch.equal(p.d_table, table) and torch.equal(p.d_free, free)
    assert kvq.read_device_error(p.ws) == status
    p.check()
    p.reserve([1, 1])                # and the next call works
    p.model_reserve([1, 1])
    p.check()
    assert kvq.read_device_error(p.ws) == 0


def test_pages_report_broken_state(kvq):
    p = Pages(kvq, [20, 3], 16, 8, 10)
    p.d_table[0, 1] = 99                                       # the last, partly filled page
    _, _, slots, _ = p.reserve([1, 1])
    assert slots[0] == -1 and slots[1] >= 0 and kvq.read_device_error(p.ws) == 1
    p = Pages(kvq, [20, 3], 16, 8, 10)
    p.d_n.fill_(9)                                             # 9 free + 3 held > 10
    lens = p.d_lens.clone()
    kvq.kv_pages_trim(p.d_lens, torch.zeros_like(lens), p.d_table, p.d_free, p.d_n, 16, p.ws)
    assert torch.equal(p.d_lens, lens) and kvq.read_device_error(p.ws) == 1
    empty = torch.zeros(0, dtype=torch.int64, device="cuda")   # no sequences, padded rows only
    cu, slots = torch.full((1,), 5, dtype=torch.int64, device="cuda"), torch.full((3,), 5, dtype=torch.int64, device="cuda")
    kvq.kv_pages_reserve(empty, empty, p.d_table[:0], p.d_free, p.d_n, 16, empty, cu, slots, None, p.ws)
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 3


def test_pages_refuse_bad_tensors(kvq):
    p = Pages(kvq, [20, 3], 16, 8, 10)
    with pytest.raises(ValueError):
        kvq.kv_pages_trim(p.d_lens, p.d_lens[:1], p.d_table, p.d_free, p.d_n, 16, p.ws)
    with pytest.raises(ValueError):
        kvq.kv_pages_trim(p.d_lens, p.d_lens.int(), p.d_table, p.d_free, p.d_n, 16, p.ws)
    with pytest.raises(ValueError):
        kvq.kv_pages_trim(p.d_lens, p.d_lens.clone(), p.d_table[:1], p.d_free, p.d_n, 16, p.ws)
    with pytest.raises(ValueError):
        kvq.kv_pages_trim(p.d_lens, p.d_lens.cpu(), p.d_table, p.d_free, p.d_n, 16, p.ws)


# -- rotary append ----------------------------------------------------------------

def turn64(v, pos, inv, axis, adjacent):
    ang = np.asarray(pos, np.float64)[axis] * np.asarray(inv)[:, None]     # [pairs][n]
    c, s = np.cos(ang).T, np.sin(ang).T
    while c.ndim < v.ndim:
        c, s = c[:, None], s[:, None]
    n = v.shape[-1] // 2
    i, j = (slice(0, None, 2), slice(1, None, 2)) if adjacent else (slice(0, n), slice(n, 2 * n))
    out = np.empty(v.shape, np.float64)
    out[..., i] = v[..., i] * c - v[..., j] * s
    out[..., j] = v[..., j] * c + v[..., i] * s
    return out


def freqs(dim):
    return [10000.0 ** (-2.0 * i / dim) for i in range(dim // 2)]


# a rotation: two products and a sum rounded to f32, cos and sin within 2 units in
# the last place of values up to 1, the phase within 2^-24 turns of pi: every
# term is a multiple of 2^-24 of |u| + |v|, 8 in all
F32_TURN = 8 * 2.0 ** -24


@pytest.mark.parametrize("n,heads,dim,dtype,axes,adjacent,far", [
    (1, 1, 64, "bf16", 1, True, 0), (8, 128, 64, "bf16", 1, True, 131072), (8, 128, 64, "f32", 2, False, 1 << 20),
    (37, 20, 64, "bf16", 3, False, 1 << 28), (300, 5, 64, "f32", 3, True, 5000), (700, 1, 64, "bf16", 4, False, 99),
    (5, 3, 6, "f32", 1, False, 1000), (9, 7, 128, "bf16", 2, True, 1000), (4, 2, 2, "bf16", 1, True, 10),
])
def test_rope_queries_match_f64(kvq, n, heads, dim, dtype, axes, adjacent, far):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(n + heads)
    pos = torch.randint(-3, far + 1, (axes, n), generator=g, device="cuda")
    axis = [i % axes for i in range(dim // 2)]
    rope = kvq.rope_layout(freqs(dim), axis, n_axes=axes, adjacent=adjacent)
    whole = torch.randn(n, heads, dim + 48, generator=g, device="cuda").to(dt)
    ref = turn64(whole[..., 48:].double().cpu().numpy(), pos.cpu().numpy(), freqs(dim), axis, adjacent)
    size = np.abs(whole[..., 48:].double().cpu().numpy())
    half = dim // 2
    pair = (size[..., 0::2] + size[..., 1::2]).repeat(2, -1) if adjacent else np.tile(size[..., :half] + size[..., half:], 2)
    tol = F32_TURN * pair + (BF16_STEP if dt == torch.bfloat16 else 0.0) * (np.abs(ref) + F32_TURN * pair)
    out = torch.full((n, heads, dim + 16), 3.0, device="cuda", dtype=dt)
    kvq.kv_rope_append(kvq.KVQ_KV8, rope, None, pos, None, whole[..., 48:], out[..., 16:], None, None)
    got = out.double().cpu().numpy()
    assert np.all(np.abs(got[..., 16:] - ref) <= tol)
    assert np.all(got[..., :16] == 3.0)
    # in place, and on views that start off 16 bytes: the same bits
    same = whole.clone()
    kvq.kv_rope_append(kvq.KVQ_KV8, rope, None, pos, None, same[..., 48:], same[..., 48:], None, None)
    assert torch.equal(same[..., 48:], out[..., 16:]) and torch.equal(same[..., :48], whole[..., :48])
    off = torch.zeros(n, heads, dim + 49, device="cuda", dtype=dt)
    off[..., 49:] = whole[..., 48:]
    kvq.kv_rope_append(kvq.KVQ_KV8, rope, None, pos, None, off[..., 49:], off[..., 49:], None, None)
    assert torch.equal(off[..., 49:], out[..., 16:])


@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("n,dims,dim,dtype,adjacent", [
    (1, (512, 64), 64, "f32", True), (45, (512, 64), 64, "bf16", False), (9, (256, 32), 32, "f32", False),
    (7, (64,), 16, "bf16", True), (3, (1024,), 128, "f32", True),
])
def test_rope_rows_are_the_oracles_codes(kvq, oracle, fmt, n, dims, dim, dtype, adjacent):
    D = sum(dims)
    layout = kvq.mla_layout(dims, v_dim=dims[0], seed=9)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = to_dev(synth.mla_rows(n, n, D)).to(dt)
    pos = torch.randint(0, 100000, (2, n), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    axis = [i % 2 for i in range(dim // 2)]
    rope = kvq.rope_layout(freqs(dim), axis, adjacent=adjacent)
    pool = n + 11
    slots = torch.randperm(pool, generator=torch.Generator().manual_seed(2))[:n].cuda()
    row = kvq.row_bytes(fmt, layout)
    codes = torch.full((pool, row), 171, dtype=torch.uint8, device="cuda")
    scales = torch.full((pool, len(dims)), -7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    skip = slots.clone()
    if n > 2:
        skip[1] = -1
    wide = torch.zeros(n, D + 24, device="cuda", dtype=dt)      # rows inside a wider tensor
    wide[:, :D] = x
    kvq.kv_rope_append(fmt, rope, wide[:, :D], pos, skip, None, None, codes, scales, layout, err_word=err)
    # the rotated dims exactly as the kernel rounds them: through the query side, in f32
    turned = torch.empty(n, 1, dim, device="cuda")
    kvq.kv_rope_append(fmt, rope, None, pos, None, x[:, None, D - dim:].float().contiguous(), turned, None, None, layout)
    rows = x.float().cpu().numpy().copy()
    rows[:, D - dim:] = turned[:, 0].cpu().numpy()
    oc, os_ = oracle.kv8_encode(rows, dims) if fmt == 1 else oracle.tq4_encode(rows, dims, seed=9)
    got_c, got_s = codes.cpu().numpy(), scales.cpu().numpy()
    sl = skip.cpu().numpy()
    for i in range(n):
        if sl[i] >= 0:
            assert np.array_equal(got_c[sl[i]], oc[i]) and np.array_equal(got_s[sl[i]], os_[i]), i
    untouched = np.setdiff1d(np.arange(pool), sl[sl >= 0])
    assert np.all(got_c[untouched] == 171) and np.all(got_s[untouched] == -7.0)
    assert err.item() == 0


def test_rope_append_reports_bad_rows(kvq):
    rope = kvq.rope_layout(freqs(64))
    pos = torch.zeros(3, dtype=torch.int64, device="cuda")
    codes, scales = torch.zeros(4, 576, dtype=torch.uint8, device="cuda"), torch.zeros(4, 2, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = torch.ones(3, 576, device="cuda")
    kvq.kv_rope_append(1, rope, x, pos, to_dev(np.array([0, 4, 2])), None, None, codes, scales, err_word=err)
    assert err.item() == 1 and bool((scales[[0, 2]] > 0).all()) and bool((scales[[1, 3]] == 0).all())
    err.zero_()
    x[1, 5] = float("nan")
    kvq.kv_rope_append(1, rope, x, pos, to_dev(np.array([0, 1, 2])), None, None, codes, scales, err_word=err)
    assert err.item() == 9
    for bad in (dict(x_new=x[:, :575]), dict(positions=pos[:2]), dict(slot_map=pos.int()), dict(codes=codes[:, :500])):
        a = dict(fmt=1, rope=rope, x_new=x, positions=pos, slot_map=pos, q_in=None, q_out=None, codes=codes, scales=scales)
        a.update(bad)
        with pytest.raises(ValueError):
            kvq.kv_rope_append(**a)
    q = torch.zeros(3, 2, 64, device="cuda")
    with pytest.raises(ValueError):
        kvq.kv_rope_append(1, rope, None, pos, None, q, q.bfloat16(), None, None)
    with pytest.raises(ValueError):
        kvq.kv_rope_append(1, rope, None, pos, None, q.transpose(1, 2), q, None, None)


def test_rope_one_token_one_head_any_stride(kvq):
    """Dimensions of size one have strides that say nothing."""
    rope = kvq.rope_layout(freqs(64))
    pos = torch.tensor([5], device="cuda")
    q = torch.randn(64, device="cuda")
    x = torch.randn(576, device="cuda")
    out = torch.zeros(2, 1, 1, 64, device="cuda")
    codes, scales = torch.zeros(2, 576, dtype=torch.uint8, device="cuda"), torch.zeros(2, 2, device="cuda")
    for i, (qs, xs) in enumerate([((64, 64, 1), (576, 1)), ((0, 3, 1), (0, 1))]):
        kvq.kv_rope_append(1, rope, x.as_strided((1, 576), xs), pos, torch.tensor([i], device="cuda"),
                           q.as_strided((1, 1, 64), qs), out[i].as_strided((1, 1, 64), qs), codes, scales)
    assert torch.equal(out[0], out[1]) and bool((out[0] != 0).any())
    assert torch.equal(codes[0], codes[1]) and torch.equal(scales[0], scales[1]) and bool((scales > 0).all())


# -- attention --------------------------------------------------------------------

class Paged:
    """A paged pool of encoded rows, every sequence's pages scattered over it."""

    def __init__(self, kvq, oracle, fmt, past, new, page, seed, x=None, dims=(512, 64), spare=3):
        self.kvq, self.fmt, self.page, self.new = kvq, fmt, page, list(new)
        self.layout = kvq.mla_layout(dims, seed=seed)
        self.total = [p + n for p, n in zip(past, new)]
        need = [-(-t // page) for t in self.total]
        self.n_pages = sum(need) + spare
        rng = np.random.default_rng(seed)
        order = rng.permutation(self.n_pages).tolist()
        self.table = np.full((len(past), max(max(need), 1) + 2), 12345678, np.int32)   # entries past the end: garbage
        rows = []
        for s, k in enumerate(need):
            ids, order = order[:k], order[k:]
            self.table[s, :k] = ids
            rows.append(np.array([ids[t // page] * page + t % page for t in range(self.total[s])], np.int64))
        n = sum(self.total)
        self.x = synth.mla_rows(seed, n) if x is None else x
        codes, scales = gpu_encode(kvq, fmt, self.x, self.layout)
        # rows of no sequence hold NaN codes and scales: reading one shows
        self.codes = torch.full((self.n_pages * page, codes.shape[1]), 0x7F, dtype=torch.uint8, device="cuda")
        self.scales = torch.full((self.n_pages * page, scales.shape[1]), float("nan"), device="cuda")
        flat = to_dev(np.concatenate(rows) if n else np.zeros(0, np.int64))
        self.codes[flat], self.scales[flat] = codes, scales
        self.cu = synth.cu_seqlens(new)
        self.lens = np.array(self.total, np.int64)
        xh = oracle.reconstruct(fmt, codes.cpu().numpy(), scales.cpu().numpy(), dims, seed)
        off = synth.cu_seqlens(self.total)
        self.xh = [np.asarray(xh[off[b]:off[b + 1]], np.float64) for b in range(len(past))]
        self.rotate = lambda v: np.asarray(oracle.tq4_rotate(np.ascontiguousarray(v, np.float32), dims, seed), np.float64)

    def run(self, q, path, n_tok=None, sm=SM, fill=float("nan"), stream=None):
        kvq, H = self.kvq, q.shape[1]
        bf16 = q.dtype == torch.bfloat16
        out = torch.full((q.shape[0], H, 512), fill, dtype=q.dtype, device="cuda")
        ws = torch.full((kvq.kv_attn_paged_workspace_size(self.fmt, len(self.new), H, q.shape[0], self.layout, bf16, path),),
                        0xFF, dtype=torch.uint8, device="cuda")
        ws[:256] = 0
        kvq.kv_attn_paged(self.fmt, q, to_dev(self.cu), self.codes, self.scales, to_dev(self.table), to_dev(self.lens),
                          self.page, out, ws, sm, self.layout, path, stream)
        torch.cuda.synchronize()
        self.err = kvq.read_device_error(ws)
        return out

    def check(self, q, out, tol, sm=SM, q_rounded=False):
        """tol: of the largest output of a vector.  q_rounded: the rotated query was rounded to f16 (4-bit rows on the
        tensor cores), each element off by at most 2^-11 of itself, so by 2^-11 / sqrt(3) in the root mean square of a
        uniform rounding error.  A score sm sum_i q'_i x'_i is then off by sigma = sm 2^-11 / sqrt(3)
        sqrt(sum_i (q'_i x'_i)^2), and the output, d out = sum_t w_t dz_t (x_t - out), by at most
        8 sigma_t w_t |x_t - out| summed over the rows (8 sigma: once in 10^15)."""
        qv, got = q.double().cpu().numpy(), out.double().cpu().numpy()
        worst = 0.0
        for b, n in enumerate(self.new):
            T = int(self.lens[b])
            for i in range(n):
                at, seen = int(self.cu[b]) + i, T - n + i + 1
                if seen <= 0:
                    assert np.all(got[at] == 0.0)
                    continue
                K = self.xh[b][:seen]
                z = qv[at] @ K.T * sm
                w = np.exp(z - z.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                ref = w @ K[:, :512]
                allowed = tol * np.max(np.abs(ref), 1)
                if q_rounded:
                    sigma = sm * 2.0 ** -11 / math.sqrt(3.0) * np.sqrt(self.rotate(qv[at]) ** 2 @ self.rotate(K).T ** 2)
                    for h in range(len(allowed)):
                        allowed[h] += np.max((8 * sigma[h] * w[h]) @ np.abs(K[:, :512] - ref[h]))
                e = np.max(np.abs(got[at] - ref), 1) / allowed
                worst = max(worst, float(e.max()))
                assert e.max() <= 1.0, (b, i, int(e.argmax()), float(e.max()))
        return worst


def query(n, H, seed, bf16, scale=1.0):
    q = torch.randn(n, H, 576, generator=torch.Generator().manual_seed(seed)) * scale
    return (q.bfloat16() if bf16 else q).cuda()


def tolerance(fmt, path, bf16):
    if path == 2:
        return TENSOR_TOL + BF16_STEP
    return SIMT_TOL + (BF16_STEP if bf16 else 0.0)


PATHS = [(1, False), (1, True), (2, True)]


@pytest.mark.parametrize("path,bf16", PATHS)
@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("past,new,H,page", [
    ([0], [1], 1, 16), ([0, 31, 32, 33], [1, 1, 1, 1], 16, 32), ([300, 0, 17, 1000, 5], [1, 7, 0, 3, 40], 20, 16),
    ([127, 128, 129, 0], [2, 1, 130, 129], 5, 64), ([70, 260], [9, 3], 128, 128), ([500], [33], 65, 256),
    ([4000, 1, 90], [1, 2, 70], 64, 64),
])
def test_attn_paged_matches_f64(kvq, oracle, fmt, path, bf16, past, new, H, page):
    p = Paged(kvq, oracle, fmt, past, new, page, seed=len(past) + H)
    q = query(sum(new), H, H, bf16)
    out = p.run(q, path)
    assert p.err == 0
    p.check(q, out, tolerance(fmt, path, bf16), q_rounded=fmt == 2 and path == 2)
    assert torch.equal(out.view(torch.int16 if bf16 else torch.int32),
                       p.run(q, path).view(torch.int16 if bf16 else torch.int32))   # the same bits every time


@pytest.mark.parametrize("path,bf16", PATHS)
def test_attn_paged_one_scale_layout(kvq, oracle, path, bf16):
    p = Paged(kvq, oracle, 1, [150, 20], [3, 1], 32, seed=3, dims=(576,))
    q = query(4, 16, 5, bf16)
    p.check(q, p.run(q, path), tolerance(1, path, bf16))


@pytest.mark.parametrize("path,bf16", PATHS)
@pytest.mark.parametrize("fmt", [1, 2])
def test_attn_paged_rows_without_anything_to_see(kvq, oracle, fmt, path, bf16):
    """Fewer cached rows than new tokens, none at all, padded tokens behind the batch."""
    p = Paged(kvq, oracle, fmt, [10, 0, 5], [40, 9, 3], 16, seed=8)
    p.lens[0], p.lens[1] = 17, 0       # tokens 0..22 of sequence 0 and all of sequence 1 see nothing
    q = query(sum(p.new) + 6, 20, 8, bf16)
    out = p.run(q, path, fill=7.0)
    assert p.err == 0 and bool((out[52:] == 7.0).all())
    p.check(q, out, tolerance(fmt, path, bf16), q_rounded=fmt == 2 and path == 2)


@pytest.mark.parametrize("path,bf16", PATHS)
@pytest.mark.parametrize("fmt", [1, 2])
def test_attn_paged_long_and_split(kvq, oracle, fmt, path, bf16):
    """One long sequence spread over every CTA, next to short ones."""
    p = Paged(kvq, oracle, fmt, [30000, 2, 700], [1, 3, 2], 64, seed=12)
    q = query(6, 16, 12, bf16)
    p.check(q, p.run(q, path), tolerance(fmt, path, bf16), q_rounded=fmt == 2 and path == 2)


@pytest.mark.parametrize("path,bf16", PATHS)
def test_attn_paged_scores_that_climb(kvq, oracle, path, bf16):
    """Scores that pass every earlier one by far, tile after tile, and latent scales over many binades."""
    T = 1500
    x = synth.mla_rows(5, T)
    ramp = np.exp2(np.linspace(-12.0, 3.0, T)).astype(np.float32)
    x *= ramp[:, None]
    x[::97] *= np.float32(2.0 ** -10)
    p = Paged(kvq, oracle, 1, [T - 8, ], [8], 32, seed=5, x=x)
    q = query(8, 16, 6, bf16, scale=3.0)
    q[:, 3] *= 2.0 ** -20          # heads of very different size share a tile
    q[:, 4] *= 2.0 ** 9
    q[:, 5] = 0
    p.check(q, p.run(q, path), tolerance(1, path, bf16))


@pytest.mark.parametrize("path,bf16", PATHS)
def test_attn_paged_zero_rows(kvq, oracle, path, bf16):
    x = synth.mla_rows(5, 300)
    x[:200, :512] = 0               # inert latent blocks first
    x[250:] = 0
    p = Paged(kvq, oracle, 1, [299], [1], 16, seed=5, x=x)
    q = query(1, 8, 6, bf16)
    p.check(q, p.run(q, path), tolerance(1, path, bf16))


@pytest.mark.parametrize("path,bf16", PATHS)
def test_attn_paged_nan_query_stays_alone(kvq, oracle, path, bf16):
    p = Paged(kvq, oracle, 1, [200, 40], [1, 5], 32, seed=4)
    q = query(6, 16, 4, bf16)
    clean = p.run(q, path)
    q[2, 7, 100] = float("nan")
    q[3, 2, 550] = float("inf")
    out = p.run(q, path)
    hit = torch.zeros(6, 16, dtype=torch.bool, device="cuda")
    hit[2, 7] = hit[3, 2] = True
    assert bool(torch.isnan(out[2, 7]).all()) and not bool(torch.isfinite(out[3, 2]).any())
    p.check(torch.where(hit[..., None], torch.zeros_like(q), q), torch.where(hit[..., None], p.run(torch.where(
        hit[..., None], torch.zeros_like(q), q), path), out), tolerance(1, path, bf16))
    assert bool(torch.isfinite(clean).all())


@pytest.mark.parametrize("path,bf16", PATHS)
def test_attn_paged_reports_bad_batches(kvq, oracle, path, bf16):
    def fresh():
        return Paged(kvq, oracle, 1, [100, 60], [2, 2], 32, seed=4, spare=2)
    q = query(4, 16, 4, bf16)
    p = fresh()
    p.codes.copy_(torch.zeros_like(p.codes))
    p.scales.fill_(1.0)
    p.table[0, 1] = p.n_pages                     # a page outside the pool: reported, page 0 read instead
    assert bool(torch.isfinite(p.run(q, path)).all()) and p.err == 1
    p = fresh()
    p.lens[1] = -5                                # no rows: zeros
    out = p.run(q, path)
    assert p.err == 1 and bool((out[2:] == 0).all())
    p = fresh()
    p.cu[2] = 5                                   # past the tokens: the sequence is left out
    out = p.run(q, path, fill=7.0)
    assert p.err == 1 and bool((out[2:] == 7.0).all()) and bool(torch.isfinite(out[:2]).all())
    p = fresh()
    p.lens[0] = 1 << 40                           # more than its table row can list
    p.table[:] = 0
    p.codes.zero_()
    p.scales.fill_(1.0)
    p.run(q, path)
    assert p.err == 1


def test_attn_paged_refuses_bad_tensors(kvq, oracle):
    p = Paged(kvq, oracle, 1, [100], [2], 32, seed=4)
    q = query(2, 16, 4, True)
    with pytest.raises(kvq.KvqError):
        p.run(q.float(), 2)                       # f32 queries on the tensor path: no workspace, no kernel
    with pytest.raises(ValueError):
        p.run(q[..., :512].contiguous(), 0)
    p.page = 48
    with pytest.raises((kvq.KvqError, ValueError)):
        p.run(q, 0)


def test_attn_paged_on_its_own_stream_and_twice_at_once(kvq, oracle):
    p = Paged(kvq, oracle, 1, [900, 60], [4, 2], 32, seed=4)
    q = query(6, 64, 4, True)
    want = p.run(q, 0)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    cu, table, lens = to_dev(p.cu), to_dev(p.table), to_dev(p.lens)
    size = kvq.kv_attn_paged_workspace_size(1, 2, 64, 6, p.layout)
    ws = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in streams]
    outs = [torch.zeros_like(want) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(4):
        for st, w, o in zip(streams, ws, outs):
            kvq.kv_attn_paged(1, q, cu, p.codes, p.scales, table, lens, 32, o, w, SM, p.layout, stream=st)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


@pytest.mark.parametrize("path,bf16", PATHS)
@pytest.mark.parametrize("fmt", [1, 2])
def test_attn_paged_rows_that_are_no_numbers(kvq, oracle, fmt, path, bf16):
    """NaN codes and NaN or infinite scales in a late row: tokens before it do not notice, those that see it are NaN."""
    p = Paged(kvq, oracle, fmt, [100, 30], [40, 3], 32, seed=14)
    q = query(43, 16, 4, bf16)
    want = p.run(q, path)
    for what in ("code", "nan", "inf", "rope"):
        if what == "code" and fmt == 2:
            continue
        r = p.table[0, 110 // 32] * 32 + 110 % 32           # row 110: tokens 10 .. 39 of sequence 0 see it
        keep = p.codes[r].clone(), p.scales[r].clone()
        if what == "code":
            p.codes[r, 7] = 0xFF
        else:
            p.scales[r, 1 if what == "rope" else 0] = float("inf") if what == "inf" else float("nan")
        out = p.run(q, path)
        p.codes[r], p.scales[r] = keep
        assert bool(torch.isnan(out[10:40]).all()), what
        rest = torch.cat([out[:10], want[10:40], out[40:]])
        p.check(q, rest, tolerance(fmt, path, bf16), q_rounded=fmt == 2 and path == 2)


@pytest.mark.parametrize("path,bf16", PATHS)
@pytest.mark.parametrize("fmt", [1, 2])
@pytest.mark.parametrize("n_seq,H,every", [(700, 4, 7), (1400, 2, 200), (300, 128, 1)])
def test_attn_paged_padded_batches(kvq, oracle, fmt, path, bf16, n_seq, H, every):
    """Many sequences, most of them without tokens; many short tiles to a walker."""
    rng = np.random.default_rng(n_seq)
    new = [int(rng.integers(1, 3)) if s % every == every - 1 else 0 for s in range(n_seq)]
    past = [int(rng.integers(0, 40)) for _ in range(n_seq)]
    p = Paged(kvq, oracle, fmt, past, new, 16, seed=2)
    q = query(sum(new), H, 4, bf16)
    out = p.run(q, path)
    assert p.err == 0
    p.check(q, out, tolerance(fmt, path, bf16), q_rounded=fmt == 2 and path == 2)


@pytest.mark.parametrize("path,bf16", PATHS)
@pytest.mark.parametrize("page", [16, 4096, 65536])
def test_attn_paged_page_sizes(kvq, oracle, path, bf16, page):
    p = Paged(kvq, oracle, 1, [4090, 5], [20, 2], page, seed=2, spare=1)
    q = query(22, 8, 4, bf16)
    out = p.run(q, path)
    assert p.err == 0
    p.check(q, out, tolerance(1, path, bf16))


@pytest.mark.parametrize("path,bf16", PATHS)
@pytest.mark.parametrize("fmt", [1, 2])
def test_attn_paged_offset_buffers(kvq, oracle, fmt, path, bf16):
    """Queries, output and workspace that start on 16 bytes and no more."""
    p = Paged(kvq, oracle, fmt, [300, 5], [9, 2], 32, seed=2)
    q = query(11, 24, 4, bf16)
    want = p.run(q, path)
    pad = 16 // q.element_size()
    q2 = torch.empty(q.numel() + pad, dtype=q.dtype, device="cuda")[pad:].view(q.shape).copy_(q)
    o2 = torch.zeros(want.numel() + pad, dtype=q.dtype, device="cuda")[pad:].view(want.shape)
    size = kvq.kv_attn_paged_workspace_size(fmt, 2, 24, 11, p.layout, bf16, path)
    ws = torch.zeros(size + 16, dtype=torch.uint8, device="cuda")[16:]
    kvq.kv_attn_paged(fmt, q2, to_dev(p.cu), p.codes, p.scales, to_dev(p.table), to_dev(p.lens), 32, o2, ws, SM, p.layout, path)
    assert torch.equal(o2, want) and kvq.read_device_error(ws) == 0


@pytest.mark.parametrize("path,bf16", PATHS)
def test_attn_paged_shared_prefix(kvq, oracle, path, bf16):
    """Three sequences over the same first pages."""
    p = Paged(kvq, oracle, 1, [128, 128, 128], [5, 1, 40], 32, seed=2)
    p.table[1, :4] = p.table[2, :4] = p.table[0, :4]
    for b in (1, 2):
        p.xh[b][:128] = p.xh[0][:128]
    q = query(46, 20, 4, bf16)
    p.check(q, p.run(q, path), tolerance(1, path, bf16))


def test_attn_paged_counts_rescales_and_time(kvq, oracle):
    """The diagnostics of the other attention calls: steps on the exact path, launch times."""
    T = 1500
    x = synth.mla_rows(5, T)
    # 30 tiles of 12 steps: a walker has several steps of a tile
    flat = Paged(kvq, oracle, 1, [T - 30], [30], 32, seed=5, x=x)
    climb = Paged(kvq, oracle, 1, [T - 30], [30], 32, seed=5, x=x * np.exp2(np.linspace(-12.0, 3.0, T)).astype(np.float32)[:, None])
    counts = []
    kvq.timing_enable(4)
    try:
        for p in (flat, climb):
            q = query(30, 128, 6, True, scale=0.1 if p is flat else 3.0)
            ws = torch.zeros(kvq.kv_attn_paged_workspace_size(1, 1, 128, 30, p.layout), dtype=torch.uint8, device="cuda")
            out = torch.empty(30, 128, 512, dtype=torch.bfloat16, device="cuda")
            kvq.kv_attn_paged(1, q, to_dev(p.cu), p.codes, p.scales, to_dev(p.table), to_dev(p.lens), 32, out, ws, SM, p.layout)
            counts.append(kvq.read_exact_rescales(ws))
        partial, merge, calls = kvq.timing_read()
    finally:
        kvq.timing_enable(0)
    assert calls == 2 and partial > 0 and merge > 0
    assert counts[0] == 0 and counts[1] > 0


@pytest.mark.parametrize("path,bf16", PATHS)
@pytest.mark.parametrize("fmt", [1, 2])
def test_attn_paged_offsets_past_32_bits(kvq, oracle, fmt, path, bf16):
    """A pool of 8 (16) million rows, 4.8 GB: pages at its end, and rows appended there."""
    page, n_pages = 64, (1 << 17) * fmt
    p = Paged(kvq, oracle, fmt, [300, 70], [5, 1], page, seed=2)
    q = query(6, 16, 4, bf16)
    want = p.run(q, path)
    codes = torch.empty(n_pages * page, p.codes.shape[1], dtype=torch.uint8, device="cuda")
    scales = torch.empty(n_pages * page, p.scales.shape[1], device="cuda")
    assert codes.numel() > 1 << 32
    far = p.n_pages * page
    codes[-far:], scales[-far:] = p.codes, p.scales
    small = p.codes, p.scales, p.table
    p.codes, p.scales = codes, scales
    p.table = np.where(p.table < p.n_pages, p.table + n_pages - p.n_pages, p.table).astype(np.int32)
    assert torch.equal(p.run(q, path).view(torch.int16), want.view(torch.int16)) and p.err == 0
    rope, pos = kvq.rope_layout(freqs(64)), torch.arange(3, device="cuda")
    x = torch.randn(3, 576, generator=torch.Generator().manual_seed(1)).cuda()
    near = torch.zeros(3, codes.shape[1], dtype=torch.uint8, device="cuda"), torch.zeros(3, scales.shape[1], device="cuda")
    kvq.kv_rope_append(fmt, rope, x, pos, torch.arange(3, device="cuda"), None, None, *near, p.layout)
    last = torch.tensor([n_pages * page - 1, n_pages * page - 70, n_pages * page - 3], device="cuda")
    kvq.kv_rope_append(fmt, rope, x, pos, last, None, None, codes, scales, p.layout)
    assert torch.equal(codes[last], near[0]) and torch.equal(scales[last], near[1])


@pytest.mark.parametrize("path,bf16", PATHS)
def test_attn_paged_empty_pool(kvq, path, bf16):
    layout = kvq.mla_layout()
    q = query(3, 4, 1, bf16)
    out = torch.full((3, 4, 512), 7.0, dtype=q.dtype, device="cuda")
    ws = torch.zeros(kvq.kv_attn_paged_workspace_size(1, 2, 4, 3, layout, bf16, path), dtype=torch.uint8, device="cuda")
    for stride in (0, 2):
        kvq.kv_attn_paged(1, q, to_dev(np.array([0, 1, 3])), torch.zeros(0, 576, dtype=torch.uint8, device="cuda"),
                          torch.zeros(0, 2, device="cuda"), torch.zeros(2, stride, dtype=torch.int32, device="cuda"),
                          to_dev(np.zeros(2, np.int64)), 16, out, ws, SM, layout, path)
        assert bool((out == 0).all()) and kvq.read_device_error(ws) == 0


def test_attn_paged_query_outliers(kvq, oracle):
    """One query element 2^12 times the others, against rows that are small there.  The others keep an absolute error of
    2^-17 of the largest (uniform, so 2^-17 / sqrt(3) in the root mean square): a score is off by
    sigma = sm 2^-17 / sqrt(3) max|q| |x|, the output by at most 8 sigma_t w_t |x_t - out| summed over the rows."""
    T, H = 600, 8
    x = synth.mla_rows(7, T)
    x[:, 33] = 0.0
    p = Paged(kvq, oracle, 1, [T - 2], [2], 32, seed=2, x=x)
    q = query(2, H, 4, True)
    q[:, :4, 33] = 4096.0
    out = p.run(q, 0).double().cpu().numpy()
    qv = q.double().cpu().numpy()
    for i in range(2):
        K = p.xh[0][:T - 1 + i]
        z = qv[i] @ K.T * SM
        w = np.exp(z - z.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        ref = w @ K[:, :512]
        for h in range(H):
            sigma = SM * 2.0 ** -17 / math.sqrt(3.0) * np.abs(qv[i, h]).max() * np.linalg.norm(K, axis=1)
            allowed = tolerance(1, 2, True) * np.abs(ref[h]).max() + np.max((8 * sigma * w[h]) @ np.abs(K[:, :512] - ref[h]))
            assert np.max(np.abs(out[i, h] - ref[h])) <= allowed, (i, h)


@pytest.mark.parametrize("fmt", [1, 2])
def test_attn_paged_wait_that_runs_out(kvq, oracle, fmt):
    """The products held back until their wait gives up: an error word, and the next call runs."""
    p = Paged(kvq, oracle, fmt, [900, 60], [4, 2], 32, seed=4)
    q = query(6, 64, 4, True)
    try:
        kvq.test_stall_waits(2000)
        p.run(q, 0)
        assert p.err == 10
    finally:
        kvq.test_stall_waits(0)
    out = p.run(q, 0)
    assert p.err == 0
    p.check(q, out, tolerance(fmt, 2, True), q_rounded=fmt == 2)


def test_attn_paged_two_graphs_share_a_workspace(kvq, oracle):
    a = Paged(kvq, oracle, 1, [900, 60], [4, 2], 32, seed=4)
    b = Paged(kvq, oracle, 2, [10, 700, 3], [1, 1, 9], 64, seed=5)
    qs = [query(6, 64, 4, True), query(11, 16, 5, True)]
    want = [p.run(q, 0) for p, q in zip((a, b), qs)]
    size = max(kvq.kv_attn_paged_workspace_size(p.fmt, len(p.new), q.shape[1], q.shape[0], p.layout) for p, q in zip((a, b), qs))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for p, q, w in zip((a, b), qs, want):
        args = (p.fmt, q, to_dev(p.cu), p.codes, p.scales, to_dev(p.table), to_dev(p.lens), p.page)
        outs.append((torch.zeros_like(w), args))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kvq.kv_attn_paged(*args, outs[-1][0], ws, SM, p.layout)
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (o, _), w in zip(outs, want):
        assert torch.equal(o, w)
    assert kvq.read_device_error(ws) == 0


# -- a serving loop -----------------------------------------------------------------

@pytest.mark.parametrize("fmt", [1, 2])
def test_a_captured_step_replays_a_serving_loop(kvq, oracle, fmt):
    """reserve -> append -> attend, captured once and replayed with new tokens, against the same rows in a contiguous
    pool: a prompt of 50, 3 and 0 rows first, then six steps of one token a sequence, one of them taken back."""
    B, H, page, seed = 3, 16, 16, 6
    layout = kvq.mla_layout(seed=seed)
    rope = kvq.rope_layout(freqs(64), adjacent=True)
    n_pages, stride = 24, 8
    free = torch.arange(n_pages, dtype=torch.int32, device="cuda").flip(0).contiguous()
    n_free = torch.tensor([n_pages], dtype=torch.int32, device="cuda")
    table = torch.zeros(B, stride, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int64, device="cuda")
    codes = torch.zeros(n_pages * page, kvq.row_bytes(fmt, layout), dtype=torch.uint8, device="cuda")
    scales = torch.zeros(n_pages * page, 2, device="cuda")
    pws = torch.zeros(kvq.kv_pages_workspace_size(), dtype=torch.uint8, device="cuda")
    size = kvq.kv_attn_paged_workspace_size(fmt, B, H, 64, layout)
    aws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)

    class Buffers:
        def __init__(self, m):
            self.new = torch.zeros(B, dtype=torch.int64, device="cuda")
            self.cu = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
            self.slots = torch.zeros(m, dtype=torch.int64, device="cuda")
            self.pos = torch.zeros(m, dtype=torch.int64, device="cuda")
            self.x = torch.zeros(m, 576, device="cuda", dtype=torch.bfloat16)
            self.pe = torch.zeros(m, H, 64, device="cuda", dtype=torch.bfloat16)
            self.q = torch.zeros(m, H, 576, device="cuda", dtype=torch.bfloat16)
            self.out = torch.zeros(m, H, 512, device="cuda", dtype=torch.bfloat16)

        def fill(self, new):
            self.new.copy_(torch.tensor(new))
            for t in (self.x, self.pe, self.q):
                t.copy_(torch.randn(t.shape, generator=g, device="cuda"))

        def step(self):
            kvq.kv_pages_reserve(lens, self.new, table, free, n_free, page, lens, self.cu, self.slots, self.pos, pws)
            kvq.kv_rope_append(fmt, rope, self.x, self.pos, self.slots, self.pe, self.q, codes, scales, layout,
                               err_word=aws)
            kvq.kv_attn_paged(fmt, self.q, self.cu, codes, scales, table, lens, page, self.out, aws, SM, layout)

    held = [np.zeros((0, 576)) for _ in range(B)]
    tol = tolerance(fmt, 2, True) + (2.0 ** -7 if fmt == 2 else 0.0)   # 4 bits: room for the rounded query

    def check(buf, new, keep=True):
        turned = torch.empty(buf.x.shape[0], 1, 64, device="cuda")
        kvq.kv_rope_append(fmt, rope, None, buf.pos, None, buf.x[:, None, 512:].float().contiguous(), turned, None, None,
                           layout)
        rows = buf.x.float().cpu().numpy().copy()
        rows[:, 512:] = turned[:, 0].cpu().numpy()
        oc, os_ = oracle.kv8_encode(rows) if fmt == 1 else oracle.tq4_encode(rows, seed=seed)
        xh = np.asarray(oracle.reconstruct(fmt, oc, os_, seed=seed), np.float64)
        q, out = buf.q.double().cpu().numpy(), buf.out.double().cpu().numpy()
        at = 0
        for b, n in enumerate(new):
            rows_b = np.concatenate([held[b], xh[at:at + n]])
            for i in range(n):
                K = rows_b[:len(held[b]) + i + 1]
                z = q[at + i] @ K.T * SM
                w = np.exp(z - z.max(1, keepdims=True))
                ref = (w / w.sum(1, keepdims=True)) @ K[:, :512]
                for h in range(H):
                    assert rel_err(out[at + i, h], ref[h]) <= tol, (b, i, h)
            if keep:
                held[b] = rows_b
            at += n

    prompt = Buffers(60)
    prompt.fill([50, 3, 0])
    prompt.step()
    check(prompt, [50, 3, 0])
    one = Buffers(B)
    one.fill([1, 1, 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    state = [t.clone() for t in (lens, table, free, n_free, codes, scales)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        one.step()
    for t, v in zip((lens, table, free, n_free, codes, scales), state):
        assert torch.equal(t, v)        # capturing runs nothing
    for step in range(6):
        one.fill([1, 1, 1])
        before = lens.clone()
        graph.replay()
        check(one, [1, 1, 1], keep=step != 3)
        if step == 3:
            kvq.kv_pages_trim(lens, before, table, free, n_free, page, pws)
            assert torch.equal(lens, before)
    assert kvq.read_device_error(pws) == 0 and kvq.read_device_error(aws) == 0
    assert lens.tolist() == [len(h) for h in held] == [55, 8, 5]
    kvq.kv_pages_trim(lens, torch.zeros_like(lens), table, free, n_free, page, pws)
    assert n_free.item() == n_pages and sorted(free.tolist()) == list(range(n_pages))


@pytest.mark.parametrize("fmt,path", [(1, 0), (2, 0), (1, 1)])
def test_steps_back_to_back_equal_steps_waited_for(kvq, fmt, path):
    """Each launch begins while the one before it runs and waits for its results: the bits of calls waited for one by
    one, over steps of changing lengths in which every call reads what the one before it wrote."""
    B, H, page, m = 5, 8, 16, 96
    layout, rope = kvq.mla_layout(seed=3), kvq.rope_layout(freqs(64))
    rng = np.random.default_rng(7)
    new = [to_dev(rng.integers(0, 2 if i % 3 else 19, B).astype(np.int64)) for i in range(12)]
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(12, m, 576, generator=g, device="cuda")
    dt = torch.float32 if path == 1 else torch.bfloat16
    q = torch.randn(12, m, H, 576, generator=g, device="cuda").to(dt)

    def run(wait):
        n_pages = 40
        free = torch.arange(n_pages, dtype=torch.int32, device="cuda")
        n_free = torch.tensor([n_pages], dtype=torch.int32, device="cuda")
        table = torch.zeros(B, 20, dtype=torch.int32, device="cuda")
        lens, keep = torch.zeros(B, dtype=torch.int64, device="cuda"), torch.zeros(B, dtype=torch.int64, device="cuda")
        codes = torch.zeros(n_pages * page, kvq.row_bytes(fmt, layout), dtype=torch.uint8, device="cuda")
        scales = torch.zeros(n_pages * page, 2, device="cuda")
        cu = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
        slots, pos = torch.zeros(m, dtype=torch.int64, device="cuda"), torch.zeros(m, dtype=torch.int64, device="cuda")
        pws = torch.zeros(kvq.kv_pages_workspace_size(), dtype=torch.uint8, device="cuda")
        aws = torch.zeros(kvq.kv_attn_paged_workspace_size(fmt, B, H, m, layout, dt == torch.bfloat16, path),
                          dtype=torch.uint8, device="cuda")
        out = torch.zeros(12, m, H, 512, dtype=dt, device="cuda")
        w = q.clone()
        torch.cuda.synchronize()
        pause = torch.cuda.synchronize if wait else lambda: None
        for i in range(12):
            kvq.kv_pages_reserve(lens, new[i], table, free, n_free, page, lens, cu, slots, pos, pws)
            pause()
            kvq.kv_rope_append(fmt, rope, x[i], pos, slots, w[i][..., 512:], w[i][..., 512:], codes, scales, layout)
            pause()
            kvq.kv_attn_paged(fmt, w[i], cu, codes, scales, table, lens, page, out[i], aws, SM, layout, path)
            pause()
            if i % 4 == 3:
                kvq.kv_pages_trim(lens, keep, table, free, n_free, page, pws)      # ends every sequence
                pause()
        torch.cuda.synchronize()
        assert kvq.read_device_error(pws) == 0 and kvq.read_device_error(aws) == 0
        return out, w, codes, scales, lens, table, free, n_free

    want = run(True)
    for _ in range(5):
        for a, b in zip(run(False), want):
            assert torch.equal(a, b)
