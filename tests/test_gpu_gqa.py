"""Grouped-query KV8 pools on the GPU: append and attention against plain implementations in 64 bits."""
import math

import pytest
import torch

from gpu_common import kvq_module
from gqa_common import Pool, attention, close, encode_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    return kvq_module()


def workspace(kvq, heads, kv, dim, bf16):
    return torch.zeros(kvq.kv_gqa_attn_paged_workspace_size(1, heads, kv, dim, 1, bf16=bf16), dtype=torch.uint8, device="cuda")


def offsets(new):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, device="cuda")


def queries(n, heads, dim, dtype, seed=1, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, heads, dim, generator=g) * gain).to(dtype).cuda()


def attend(kvq, pool, q, lens, new, causal=True, sm=None, ws=None, extra=0, stream=None):
    """(out, workspace); `extra` rows behind the last sequence hold 7."""
    n, heads, dim = q.shape
    ws = workspace(kvq, heads, pool.heads, dim, q.dtype == torch.bfloat16) if ws is None else ws
    out = torch.full((n, heads, dim), 7.0, dtype=q.dtype, device="cuda")
    kvq.kv_gqa_attn_paged(q, offsets(new), pool.k, pool.v, pool.scales, pool.table,
                          torch.tensor(lens, dtype=torch.int64, device="cuda"), out, ws,
                          1 / math.sqrt(dim) if sm is None else sm, causal=causal, stream=stream)
    if extra:
        assert bool((out[n - extra:] == 7.0).all()), "rows behind the last sequence"
    return out, ws


def check(out, q, pool, lens, new, sm, causal, what=""):
    """Against 64 bits; bf16 queries with many vectors of a kv head go the tensor cores' way, with weights in f16."""
    wide = q.dtype == torch.bfloat16 and len(q) * (q.shape[1] // pool.heads) > 24 * len(lens)
    mass = attention(q, pool, lens, new, sm, causal, absolute=True) if wide else None
    close(out, attention(q, pool, lens, new, sm, causal), what, mass)


DT = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("dim,heads,kv", [(64, 1, 1), (64, 16, 16), (128, 32, 8), (128, 7, 1), (256, 16, 2), (256, 36, 4)])
def test_decode(kvq, dtype, dim, heads, kv):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 0, 127, 128, 129, 1000, 3001]
    new = [1] * len(lens)
    pool = Pool(kv, dim, 16, lens, seed=dim + heads)
    q = queries(len(lens) + 2, heads, dim, dtype)
    out, ws = attend(kvq, pool, q, lens, new, extra=2)
    close(out[:-2], attention(q[:-2], pool, lens, new, 1 / math.sqrt(dim), True))
    assert kvq.read_device_error(ws) == 0


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim,heads,kv,page", [(64, 12, 4, 64), (128, 32, 8, 32), (128, 40, 8, 256), (256, 8, 2, 16)])
def test_mixtures_of_lengths(kvq, dtype, causal, dim, heads, kv, page):
    new = [3, 0, 1, 40, 17, 1, 200, 0, 5]
    lens = [3, 9, 700, 300, 5, 1, 260, 0, 2] if causal else [0, 9, 700, 1, 5, 64, 1501, 3, 16]
    pool = Pool(kv, dim, page, lens, seed=page)
    q = queries(sum(new), heads, dim, dtype)
    out, ws = attend(kvq, pool, q, lens, new, causal)   # causal: 17 tokens on 5 rows, 5 on 2: the first see none
    check(out, q, pool, lens, new, 1 / math.sqrt(dim), causal)
    assert kvq.read_device_error(ws) == 0


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("past,new", [(0, 1), (0, 333), (1000, 130), (4097, 64), (31, 515)])
def test_chunks(kvq, dtype, past, new):
    for dim in (64, 128, 256):
        pool = Pool(2, dim, 64, [past + new], seed=past)
        q = queries(new, 10, dim, dtype)
        out, ws = attend(kvq, pool, q, [past + new], [new])
        check(out, q, pool, [past + new], [new], 1 / math.sqrt(dim), True, f"dim {dim}")
        assert kvq.read_device_error(ws) == 0


@pytest.mark.parametrize("dtype", DT)
def test_spread_of_scales_and_scores(kvq, dtype):
    lens, new = [5000, 4000, 90], [1, 9, 2]
    pool = Pool(4, 128, 64, lens, seed=5, gain=4.0, scale_spread=8.0)
    q = queries(12, 16, 128, dtype, gain=3.0)
    out, _ = attend(kvq, pool, q, lens, new, sm=0.25)
    ref = attention(q, pool, lens, new, 0.25, True)
    # scores reach 500: f32 holds a score to 2^-24 of its size several times over, a weight to
    # 500 * 2^-21 = 2.4e-4 then; in the type's own rounding besides
    half = torch.finfo(dtype).eps / 2
    top = ref.abs().amax(-1, keepdim=True)
    assert bool(((out.double() - ref).abs() <= half * ref.abs() + 5e-4 * top).all())


def test_small_weights_and_small_scales_add_up(kvq):
    """131,072 rows some 20 binades below one row, by score and by scale: they weigh a third of it."""
    n = 131073
    pool = Pool(1, 64, 256, [n])
    one = torch.zeros(1, 64)
    one[0, 0] = 1.0
    codes, _ = encode_rows(one)
    pool.k[:] = codes.cuda()[0]
    pool.v[:] = 0
    pool.v[..., 1] = codes.cuda()[0, 0]
    for by_scale in (False, True):
        pool.scales[..., 0] = 0.0 if by_scale else -20 * math.log(2) / 448 / 1.0
        pool.scales[..., 1] = 2.0 ** -20 / 448 if by_scale else 1 / 448
        pg = int(pool.table[0, 0])
        pool.scales[pg, 0, 0, 0] = 0.0
        if by_scale:
            pool.scales[pg, 0, 0, 1] = 1 / 448
        q = torch.zeros(1, 1, 64, device="cuda")
        q[..., 0] = 1.0
        out, _ = attend(kvq, pool, q, [n], [1], sm=1.0)
        close(out, attention(q, pool, [n], [1], 1.0, True), f"by_scale={by_scale}")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_many_vectors_and_rows_that_are_no_numbers(kvq, dim, causal):
    """Tiles of 128 vectors: NaN codes and scales reach the tokens that see them, and no other."""
    lens, new = [400, 150], [70, 20]
    for dtype in DT if dim < 256 else DT[:1]:
        for bad in ("k", "v", "sk", "sv", "inf"):
            pool = Pool(2, dim, 16, lens, seed=9)
            q = queries(90, 8, dim, dtype)
            clean = Pool(2, dim, 16, lens, seed=9)
            row = 371   # seen by sequence 0's tokens from the 41st on
            pg, last = int(pool.table[0, row // 16]), int(pool.table[1, 150 // 16])
            for p_, a in ((pg, slice(row % 16, row % 16 + 1)), (last, slice(150 % 16, 16))):
                if bad in "kv":
                    (pool.k if bad == "k" else pool.v)[p_, :, a, 5] = 0x7f
                else:
                    pool.scales[p_, :, a, 0 if bad == "sk" else 1] = math.inf if bad == "inf" else math.nan
            out, ws = attend(kvq, pool, q, lens, new, causal, sm=0.1)
            sees = [i for i in range(70) if not causal or 330 + i >= row]
            rest = [i for i in range(90) if i not in sees]
            assert bool(torch.isnan(out[sees]).any(-1).all()), bad
            ref, mass = attention(q, clean, lens, new, 0.1, causal), attention(q, clean, lens, new, 0.1, causal, absolute=True)
            close(out[rest], ref[rest], f"{bad} {dtype}", mass[rest])
            assert kvq.read_device_error(ws) == 0


@pytest.mark.parametrize("dtype", DT)
def test_many_vectors_over_spread_scales(kvq, dtype):
    """References rise again and again, by scores and by scales; rows of large scale and no weight change nothing."""
    lens, new = [3000], [64]
    pool = Pool(2, 128, 64, lens, seed=5, scale_spread=6.0)
    rise = torch.linspace(0, 30, 3000, device="cuda").exp2()   # values 2^30 apart along the rows
    t = torch.arange(3000, device="cuda")
    pg = pool.table[0].long()[t // 64]
    pool.scales[pg, :, t % 64, 1] *= rise[:, None]
    q = queries(64, 8, 128, dtype, gain=3.0)
    out, ws = attend(kvq, pool, q, lens, new)
    check(out, q, pool, lens, new, 1 / math.sqrt(128), True)
    assert kvq.read_device_error(ws) == 0


def test_many_vectors_long_sums(kvq):
    """More than 256 steps by one walker: the totals in the workspace, to f32's 1e-5."""
    n, b = 70000, 304
    pool = Pool(1, 64, 1024, [n], seed=3)
    pool.table = pool.table.expand(b, -1).contiguous()
    q = queries(40 * b, 1, 64, torch.float32)
    q[40:] = q[:40].repeat(b - 1, 1, 1)
    out, ws = attend(kvq, pool, q, [n] * b, [40] * b, causal=False)
    ref = attention(q[:40], pool, [n], [40], 0.125, False)
    for i in (0, 1, 150, 303):
        close(out[40 * i:40 * i + 40], ref, f"sequence {i}")
    pool.v[:] = 0x35
    pool.scales[..., 1] = 0.3
    out, _ = attend(kvq, pool, q, [n] * b, [40] * b, causal=False, ws=ws)
    ref = attention(q[:1], pool, [n], [1], 0.125, False)
    assert float((out.double() - float(ref[0, 0, 0])).abs().max()) <= 1e-5 * float(ref[0, 0, 0])
    assert kvq.read_device_error(ws) == 0


@pytest.mark.parametrize("binades", [12, 20, 26])
def test_many_vectors_small_weights_add_up(kvq, binades):
    """131,072 rows that far below one row, by score and by scale, in tiles of 128 vectors."""
    n = 131073
    pool = Pool(1, 64, 256, [n])
    one = torch.zeros(1, 64)
    one[0, 0] = 1.0
    codes, _ = encode_rows(one)
    pool.k[:] = codes.cuda()[0]
    pool.v[:] = 0
    pool.v[..., 1] = codes.cuda()[0, 0]
    pg = int(pool.table[0, 0])
    for by_scale in (False, True):
        pool.scales[..., 0] = 0.0 if by_scale else -binades * math.log(2) / 448
        pool.scales[..., 1] = 2.0 ** -binades / 448 if by_scale else 1 / 448
        pool.scales[pg, 0, 0, 0] = 0.0
        pool.scales[pg, 0, 0, 1] = 1 / 448
        for dtype in DT:
            q = torch.zeros(64, 1, 64, dtype=dtype, device="cuda")
            q[..., 0] = 1.0
            out, _ = attend(kvq, pool, q, [n], [64], causal=False, sm=1.0)
            check(out, q, pool, [n], [64], 1.0, False, f"{dtype} by_scale={by_scale}")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("most", [3, 60])
def test_many_sequences(kvq, causal, most):
    """More sequences than one warp deals out; `most` tokens each: with few and with many vectors."""
    g = torch.Generator().manual_seed(most)
    new = torch.randint(0, most + 1, (700,), generator=g).tolist()
    lens = [max(0, int(t) + (n if causal else 0) - 2) for t, n in zip(torch.randint(0, 300, (700,), generator=g), new)]
    pool = Pool(2, 64, 32, lens, seed=most)
    for dtype in DT:
        q = queries(sum(new), 6, 64, dtype)
        out, ws = attend(kvq, pool, q, lens, new, causal)
        check(out, q, pool, lens, new, 0.125, causal, f"{dtype}")
        assert kvq.read_device_error(ws) == 0


@pytest.mark.parametrize("heads", [128, 200, 300])
def test_groups_wider_than_a_tile(kvq, heads):
    """A token's vectors fill a tile, or more than one."""
    lens, new = [700, 33, 5], [3, 1, 7]
    pool = Pool(1, 64, 16, lens, seed=heads)
    for dtype in DT:
        q = queries(11, heads, 64, dtype)
        out, ws = attend(kvq, pool, q, lens, new)
        check(out, q, pool, lens, new, 0.125, True, f"{dtype}")
        assert kvq.read_device_error(ws) == 0


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("new", [1, 70])
def test_scales_of_scores_and_queries_that_are_no_numbers(kvq, dtype, new):
    pool = Pool(2, 128, 32, [500])
    q = queries(new, 8, 128, dtype)
    for sm in (0.0, -0.3):
        out, _ = attend(kvq, pool, q, [500], [new], sm=sm)
        check(out, q, pool, [500], [new], sm, True, f"sm {sm}")
    ref = attention(q, pool, [500], [new], 0.1, True)
    mass = attention(q, pool, [500], [new], 0.1, True, absolute=True) if new > 1 and dtype == torch.bfloat16 else None
    bad = q.clone()
    bad[0, 1, 5], bad[-1, 7, 100] = math.nan, math.inf
    out, _ = attend(kvq, pool, bad, [500], [new], sm=0.1)
    rest = torch.ones(new, 8, dtype=torch.bool, device="cuda")
    rest[0, 1] = rest[-1, 7] = False
    assert bool(torch.isnan(out[~rest]).any(-1).all())
    close(out[rest], ref[rest], "the other vectors", None if mass is None else mass[rest])


def test_tensors_and_calls_on_a_stream(kvq):
    """The stream that is given takes the call, whichever is current."""
    pool = Pool(2, 128, 32, [900])
    q = queries(40, 8, 128, torch.bfloat16)
    st = torch.cuda.Stream()
    turned = torch.zeros_like(q)
    rope = kvq.rope_layout([100.0 ** (-i / 64) for i in range(64)])
    pos = torch.arange(40, device="cuda")
    ref = torch.zeros_like(q)
    kvq.kv_gqa_append(rope, None, None, pos, None, q, ref, None, None, None)
    want, _ = attend(kvq, pool, ref, [900], [40])
    ws, out, lens, cu = workspace(kvq, 8, 2, 128, True), torch.zeros_like(q), torch.tensor([900], device="cuda"), offsets([40])
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
    kvq.kv_gqa_append(rope, None, None, pos, None, q, turned, None, None, None, stream=st)
    kvq.kv_gqa_attn_paged(turned, cu, pool.k, pool.v, pool.scales, pool.table, lens, out, ws, 1 / math.sqrt(128), stream=st)
    assert not st.query()
    st.synchronize()
    assert torch.equal(turned, ref) and torch.equal(out, want)


def test_more_than_2_to_31_elements_of_queries(kvq):
    n, heads, dim = 70001, 128, 256
    pool = Pool(4, dim, 16, [20], seed=4)
    q = torch.zeros(n, heads, dim, dtype=torch.bfloat16, device="cuda")
    q[-9:] = queries(9, heads, dim, torch.bfloat16)
    out, ws = attend(kvq, pool, q, [20], [n], causal=False)
    ref, mass = (attention(q[-9:], pool, [20], [9], 1 / 16, False, absolute=a) for a in (False, True))
    close(out[-9:], ref, "the last", mass)
    assert torch.equal(out[0], out[-10]) and kvq.read_device_error(ws) == 0
    last = q[-9:].clone()
    rope, pos = kvq.rope_layout([0.5 ** i for i in range(64)]), torch.arange(n, device="cuda")
    kvq.kv_gqa_append(rope, None, None, pos, None, q, q, None, None, None)
    few = torch.empty_like(last)
    kvq.kv_gqa_append(rope, None, None, pos[-9:].contiguous(), None, last, few, None, None, None)
    assert torch.equal(q[-9:], few) and not bool(q[:-9].any())


def test_wait_that_runs_out(kvq):
    pool = Pool(2, 128, 64, [300])
    q = queries(64, 4, 128, torch.bfloat16)
    ws = workspace(kvq, 4, 2, 128, True)
    kvq.test_stall_waits(2000)
    try:
        attend(kvq, pool, q, [300], [64], ws=ws)
        torch.cuda.synchronize()
    finally:
        kvq.test_stall_waits(0)
    assert kvq.read_device_error(ws) == 10
    out, _ = attend(kvq, pool, q, [300], [64], ws=ws)
    check(out, q, pool, [300], [64], 1 / math.sqrt(128), True)
    assert kvq.read_device_error(ws) == 0


def test_a_million_rows(kvq):
    """Long sums whose roundings point one way, by as few walkers as the grid has."""
    n, kv = 1 << 20, 1
    pool = Pool(kv, 64, 1024, [n], seed=3)
    b = 456   # sequences that list the same pages
    pool.table = pool.table.expand(b, -1).contiguous()
    pool.v[:] = 0x35
    pool.scales[..., 1] = 0.3
    q = queries(b, 1, 64, torch.float32)
    out, _ = attend(kvq, pool, q, [n] * b, [1] * b)
    ref = attention(q[:1], pool, [n], [1], 0.125, True)
    close(out[:1], ref)
    assert float((out.double() - float(ref[0, 0, 0])).abs().max()) <= 1e-5 * float(ref[0, 0, 0])


@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_are_no_numbers(kvq, causal):
    """NaN codes and scales reach the tokens that see them, and no other; rows behind the last are never seen."""
    lens, new, dim = [70, 33], [6, 2], 128
    for bad in ("k", "v", "sk", "sv", "inf"):
        pool = Pool(2, dim, 16, lens, seed=9)
        q = queries(8, 6, dim, torch.float32)
        ref = attention(q, pool, lens, new, 0.1, causal)
        pg, at = int(pool.table[0, 4]), 67 - 64   # row 67 of sequence 0, seen by its last three tokens
        last, end = int(pool.table[1, 2]), 33 - 32   # behind sequence 1's end
        for p_, a in ((pg, slice(at, at + 1)), (last, slice(end, 16))):
            if bad in "kv":
                (pool.k if bad == "k" else pool.v)[p_, :, a, 5] = 0xff
            else:
                pool.scales[p_, :, a, 0 if bad == "sk" else 1] = math.inf if bad == "inf" else math.nan
        out, ws = attend(kvq, pool, q, lens, new, causal, sm=0.1)
        sees = [i for i in range(6) if not causal or 64 + i >= 67]
        for i in range(8):
            if i in sees:
                hit = torch.isnan(out[i]) if bad != "k" else torch.isnan(out[i])
                assert bool(hit.any(-1).all()), (bad, i)
            else:
                close(out[i], ref[i], f"{bad} {i}")


def test_zero_queries_and_zero_rows(kvq):
    pool = Pool(1, 64, 16, [20])
    pool.scales[..., 1] = 0.0
    out, _ = attend(kvq, pool, queries(1, 2, 64, torch.float32), [20], [1])
    assert float(out.abs().max()) == 0.0
    pool = Pool(1, 64, 16, [20])
    q = torch.zeros(1, 2, 64, device="cuda")
    out, _ = attend(kvq, pool, q, [20], [1])
    close(out, attention(q, pool, [20], [1], 0.125, True))


@pytest.mark.parametrize("gain", [1e-30, 1e-8, 1e8, 1e30])
def test_sizes_of_queries(kvq, gain):
    pool = Pool(2, 128, 32, [300])
    for dtype in DT:
        q = queries(1, 4, 128, dtype, gain=gain)
        out, _ = attend(kvq, pool, q, [300], [1], sm=0.1 / gain)
        close(out, attention(q, pool, [300], [1], 0.1 / gain, True), f"{dtype}")


def test_the_same_bits_again(kvq):
    for new in ([2, 3, 1, 40], [100, 20, 1, 400]):
        lens = [9000, 20, 1, 3000]
        pool = Pool(4, 128, 64, lens)
        q = queries(sum(new), 8, 128, torch.bfloat16)
        a, ws = attend(kvq, pool, q, lens, new)
        for _ in range(3):
            b, _ = attend(kvq, pool, q, lens, new, ws=ws)
            assert torch.equal(a, b)


def test_offsets_past_32_bits(kvq):
    dim, kv, page = 256, 8, 256
    n_pages = (1 << 32) // (dim * kv * page) * 2 + 5   # codes of 8 GB each
    k = torch.empty(n_pages, kv, page, dim, dtype=torch.uint8, device="cuda")
    v, scales = torch.empty_like(k), torch.empty(n_pages, kv, page, 2, device="cuda")
    small = Pool(kv, dim, page, [600], seed=2, spare=0)
    ids = torch.tensor([[n_pages - 1, n_pages - 4, n_pages // 2 + 1]], dtype=torch.int32, device="cuda")
    for i in range(3):
        for big, little in ((k, small.k), (v, small.v), (scales, small.scales)):
            big[ids[0, i]] = little[small.table[0, i]]
    q = queries(1, 16, dim, torch.bfloat16)
    ref = attention(q, small, [600], [1], 1 / 16, True)
    small.k, small.v, small.scales, small.table = k, v, scales, ids
    out, ws = attend(kvq, small, q, [600], [1])
    close(out, ref)
    rows = queries(1, kv, dim, torch.bfloat16, seed=8)
    slot = torch.tensor([(n_pages - 1) * page + 255], device="cuda")
    kvq.kv_gqa_append(None, rows, rows, None, slot, None, None, k, v, scales, ws)
    c, s = encode_rows(rows[0].float())
    assert torch.equal(k[-1, :, 255], c) and torch.equal(v[-1, :, 255], c) and torch.equal(scales[-1, :, 255, 1], s)


def test_broken_tables_and_lengths_are_reported(kvq):
    lens, new = [40, 50], [1, 1]
    pool = Pool(2, 64, 16, lens)
    q = queries(2, 4, 64, torch.float32)
    ref = attention(q, pool, lens, new, 0.125, True)
    pool.table[1, 1] = pool.n_pages
    out, ws = attend(kvq, pool, q, lens, new)
    assert kvq.read_device_error(ws) == 1
    close(out[:1], ref[:1])
    for bad in ([-1, 50], [40, 17 * 16]):
        pool = Pool(2, 64, 16, lens)
        out, ws = attend(kvq, pool, q, bad, new, ws=ws)
        assert kvq.read_device_error(ws) == 1
        out, ws = attend(kvq, pool, q, lens, new, ws=ws)   # the workspace serves on
        assert kvq.read_device_error(ws) == 0
        close(out, ref)
    cu = torch.tensor([0, 3, 2], device="cuda")
    kvq.kv_gqa_attn_paged(q, cu, pool.k, pool.v, pool.scales, pool.table, pool.lens, out, ws, 0.125)
    assert kvq.read_device_error(ws) == 1


def test_captured_on_another_stream_and_replayed(kvq):
    lens, new = [200, 1000, 64], [1, 1, 1]
    pool = Pool(2, 128, 64, [256, 1088, 128])   # room for every length below
    q = queries(3, 8, 128, torch.bfloat16)
    kv_lens, cu = torch.tensor(lens, device="cuda"), offsets(new)
    graphs = []
    for _ in range(2):   # two graphs, a workspace each
        ws, out = workspace(kvq, 8, 2, 128, True), torch.zeros_like(q)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            kvq.kv_gqa_attn_paged(q, cu, pool.k, pool.v, pool.scales, pool.table, kv_lens, out, ws, 0.1)
        graphs.append((graph, out, ws))
    for shift in (0, 1, 50, -60):
        kv_lens.copy_(torch.tensor([t + shift for t in lens], device="cuda"))
        ref = attention(q, pool, [t + shift for t in lens], new, 0.1, True)
        for graph, _, _ in graphs:
            graph.replay()
        for _, out, _ in graphs:
            close(out, ref)


def test_a_captured_chunk_with_other_lengths(kvq):
    """Many vectors: offsets and lengths may change between replays, rows behind the last sequence stay."""
    pool = Pool(2, 128, 32, [900, 1200, 500], seed=2)
    q = queries(220, 8, 128, torch.bfloat16)
    cu, lens = offsets([100, 20, 100]), torch.tensor([900, 1200, 500], device="cuda")
    ws, out = workspace(kvq, 8, 2, 128, True), torch.zeros_like(q)
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=st):
        kvq.kv_gqa_attn_paged(q, cu, pool.k, pool.v, pool.scales, pool.table, lens, out, ws, 0.1)
    for new, rows in (([100, 20, 100], [900, 1200, 500]), ([1, 0, 200], [20, 0, 400]), ([220, 0, 0], [300, 5, 5]), ([0, 0, 0], [1, 1, 1])):
        cu.copy_(offsets(new))
        lens.copy_(torch.tensor(rows, device="cuda"))
        out.fill_(7.0)
        graph.replay()
        n = sum(new)
        mass = attention(q[:n], pool, rows, new, 0.1, True, absolute=True)
        close(out[:n], attention(q[:n], pool, rows, new, 0.1, True), f"{new}", mass)
        assert bool((out[n:] == 7.0).all()) and kvq.read_device_error(ws) == 0


@pytest.mark.parametrize("new", [1, 100])
def test_entries_behind_a_sequence_are_not_read(kvq, new):
    lens = [33, 0, 500, 16]
    pool = Pool(2, 64, 16, lens, seed=3)
    for b, t in enumerate(lens):
        pool.table[b, -(-t // 16):] = -7
    q = queries(4 * new, 4, 64, torch.bfloat16)
    for causal in (True, False):
        out, ws = attend(kvq, pool, q, lens, [new] * 4, causal)
        check(out, q, pool, lens, [new] * 4, 0.125, causal)
        assert kvq.read_device_error(ws) == 0


@pytest.mark.parametrize("new", [1, 100])
def test_a_pool_without_pages(kvq, new):
    q = queries(2 * new, 4, 64, torch.bfloat16)
    codes = torch.empty(0, 2, 16, 64, dtype=torch.uint8, device="cuda")
    for width in (0, 3):
        ws, out = workspace(kvq, 4, 2, 64, True), torch.full_like(q, 7.0)
        kvq.kv_gqa_attn_paged(q, offsets([new, new]), codes, codes, torch.empty(0, 2, 16, 2, device="cuda"),
                              torch.zeros(2, width, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda"),
                              out, ws, 0.1)
        assert not bool(out.any()) and kvq.read_device_error(ws) == 0


def test_timed_calls(kvq):
    pool = Pool(2, 128, 32, [900])
    kvq.timing_enable(4)
    try:
        for new in (1, 100):
            attend(kvq, pool, queries(new, 8, 128, torch.bfloat16), [900], [new])
        partial, merge, calls = kvq.timing_read()
        assert calls == 2 and 0 < partial < 100 and 0 < merge < 100
    finally:
        kvq.timing_enable(0)


# -- append ----------------------------------------------------------------------

def turn(x, positions, inv, axis, adjacent):
    """Rotation of the leading dims in f64."""
    rot = 2 * len(inv)
    angle = positions.double()[axis].T * torch.tensor(inv, dtype=torch.float64, device="cuda")   # [n][pairs]
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    y = x.double().clone()
    i = torch.arange(rot // 2, device="cuda")
    a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + rot // 2)
    y[..., a], y[..., b] = x[..., a].double() * c - x[..., b].double() * s, x[..., b].double() * c + x[..., a].double() * s
    return y


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("dim,heads,kv,pairs,axes", [(64, 5, 5, 32, 1), (128, 32, 8, 64, 3), (256, 16, 2, 32, 1), (128, 6, 2, 3, 2),
                                                     (64, 4, 1, 1, 1), (256, 3, 1, 64, 4)])
def test_append(kvq, dtype, adjacent, dim, heads, kv, pairs, axes):
    n, page, n_pages = 37, 16, 5
    g = torch.Generator().manual_seed(dim + pairs)
    fused = torch.randn(n, heads + 2 * kv, dim, generator=g).to(dtype).cuda()   # strided slices of one projection
    q, k, v = fused[:, :heads], fused[:, heads:heads + kv], fused[:, heads + kv:]
    inv = [10000.0 ** (-i / pairs) for i in range(pairs)]
    axis = [i % axes for i in range(pairs)]
    rope = kvq.rope_layout(inv, axis, n_axes=axes, adjacent=adjacent)
    pos = torch.randint(0, 1 << 20, (axes, n), generator=g).cuda()
    slots = torch.randperm(page * n_pages, generator=g)[:n].cuda()
    slots[3] = -1
    kc = torch.full((n_pages, kv, page, dim), 9, dtype=torch.uint8, device="cuda")
    vc, sc = kc.clone(), torch.full((n_pages, kv, page, 2), 5.0, device="cuda")
    out = torch.zeros(n, heads, dim, dtype=dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.kv_gqa_append(rope, k, v, pos, slots, q, out, kc, vc, sc, err)
    assert int(err) == 0
    # products, sum and cos / sin in f32: 2^-22 of the two elements, then the type's rounding
    half = torch.finfo(dtype).eps / 2
    ref = turn(q, pos, inv, axis, adjacent)
    size = turn(q.abs().float() * 0 + q.abs(), pos * 0, inv, axis, adjacent).amax(-1, keepdim=True)
    assert bool(((out.double() - ref).abs() <= half * ref.abs() + 2.0 ** -22 * size * 2).all())
    rk, rv = turn(k, pos, inv, axis, adjacent), v.double()
    wrote = torch.zeros(n_pages, page, dtype=torch.bool, device="cuda")
    for i in range(n):
        if i == 3:
            continue
        p, a = int(slots[i]) // page, int(slots[i]) % page
        wrote[p, a] = True
        for codes, x, j in ((kc, rk[i], 0), (vc, rv[i], 1)):
            s = sc[p, :, a, j].double()
            amax = x.abs().amax(-1)
            assert bool(((s - amax / 448).abs() <= 2.0 ** -21 * amax / 448).all())
            got = codes[p, :, a].view(torch.float8_e4m3fn).double() * s[:, None]
            # half a step of e4m3: 2^-4 of the value, or 2^-10 scales below its normals
            assert bool(((got - x).abs() <= (2.0 ** -4 + 1e-5) * x.abs() + (2.0 ** -10 + 1e-6) * s[:, None] + 1e-6 * amax[:, None]).all())
    if True:   # values are not rotated: the encoder's very bytes
        c, s = encode_rows(v.float())
        keep = [i for i in range(n) if i != 3]
        assert torch.equal(vc[slots[keep] // page, :, slots[keep] % page], c[keep])
        assert torch.equal(sc[slots[keep] // page, :, slots[keep] % page, 1], s[keep])
    rest = ~wrote
    assert bool((kc.transpose(1, 2)[rest] == 9).all()) and bool((sc.transpose(1, 2)[rest] == 5.0).all())


def test_append_in_place_without_rotation_and_parts(kvq):
    n, dim = 9, 128
    q = queries(n, 4, dim, torch.bfloat16)
    rope = kvq.rope_layout([0.5 ** i for i in range(64)])
    pos = torch.arange(n, device="cuda") * 1001
    out = torch.zeros_like(q)
    kvq.kv_gqa_append(rope, None, None, pos, None, q, out, None, None, None)
    again = q.clone()
    kvq.kv_gqa_append(rope, None, None, pos, None, again, again, None, None, None)
    assert torch.equal(out, again)
    odd = torch.zeros(n * 4 * dim + 1, dtype=torch.bfloat16, device="cuda")[1:].view(n, 4, dim)   # not 16-byte aligned
    kvq.kv_gqa_append(rope, None, None, pos, None, q, odd, None, None, None)
    assert torch.equal(out, odd)
    pool = Pool(4, dim, 16, [32])
    kvq.kv_gqa_append(None, q, q, None, torch.arange(n, device="cuda"), None, None, pool.k, pool.v, pool.scales)
    c, s = encode_rows(q.float())
    assert torch.equal(pool.k[0, :, :n].transpose(0, 1), c) and torch.equal(pool.scales[0, :, :n, 0].T, s)


@pytest.mark.parametrize("dtype", DT)
def test_operands_aligned_to_their_elements_only(kvq, dtype):
    def odd(t):
        return torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)

    pool, twin = Pool(2, 128, 16, [40, 60]), Pool(2, 128, 16, [40, 60])
    k, v, q = (queries(5, h, 128, dtype, seed=h + i) for i, h in enumerate((2, 2, 6)))
    rope = kvq.rope_layout([0.7 ** i for i in range(20)], [i % 2 for i in range(20)], n_axes=2)
    pos, slots = torch.arange(10, device="cuda").view(2, 5), torch.tensor([3, 50, 17, 0, 64], device="cuda")
    outs, errs = [torch.zeros_like(q), odd(torch.zeros_like(q))], [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2)]
    kvq.kv_gqa_append(rope, k, v, pos, slots, q, outs[0], pool.k, pool.v, pool.scales, errs[0])
    kvq.kv_gqa_append(rope, odd(k), odd(v), odd(pos), odd(slots), odd(q), outs[1], twin.k, twin.v, twin.scales, odd(errs[1]))
    assert torch.equal(*outs) and all(torch.equal(getattr(pool, a), getattr(twin, a)) for a in ("k", "v", "scales"))
    for new in (1, 40):
        q = queries(2 * new, 6, 128, dtype)
        want, ws = attend(kvq, pool, q, [40, 60], [new, new])
        out = torch.zeros_like(q)
        kvq.kv_gqa_attn_paged(q, odd(offsets([new, new])), pool.k, pool.v, pool.scales, odd(pool.table), odd(pool.lens), out, ws,
                              1 / math.sqrt(128))
        assert torch.equal(out, want)


def test_append_reports_what_is_no_number_and_what_is_no_slot(kvq):
    pool = Pool(2, 64, 16, [16], spare=0)
    x = queries(3, 2, 64, torch.float32)
    x[1, 0, 7] = math.nan
    x[2, 1, 9] = math.inf
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    v = torch.ones_like(x)
    kvq.kv_gqa_append(None, x, v, None, torch.tensor([0, 1, 2], device="cuda"), None, None, pool.k, pool.v, pool.scales, err)
    assert int(err) == 9
    assert torch.isnan(pool.scales[0, :, :3, 0]).tolist() == [[False, True, False], [False, False, True]]
    assert not bool(torch.isnan(pool.scales[0, :, :3, 1]).any())
    err.zero_()
    kvq.kv_gqa_append(None, v, v, None, torch.tensor([16, -1, 99], device="cuda"), None, None, pool.k, pool.v, pool.scales, err)
    assert int(err) == 1


# -- the binding -------------------------------------------------------------------

def test_refusals_of_the_binding(kvq):
    pool = Pool(2, 64, 16, [20, 30])
    q = queries(2, 4, 64, torch.bfloat16)
    ws = workspace(kvq, 4, 2, 64, True)
    good = dict(q=q, cu_q=offsets([1, 1]), k_codes=pool.k, v_codes=pool.v, scales=pool.scales, block_table=pool.table,
                kv_lens=pool.lens, out=torch.zeros_like(q), workspace=ws, sm_scale=0.1)
    kvq.kv_gqa_attn_paged(**good)
    for bad in (dict(q=q.half()), dict(q=q.cpu()), dict(q=q[:, :, :32]), dict(q=q[:, :3]), dict(q=None), dict(out=good["out"].float()),
                dict(cu_q=good["cu_q"].int()), dict(cu_q=good["cu_q"][:2]), dict(k_codes=pool.k.int()), dict(v_codes=pool.v[1:]),
                dict(scales=pool.scales[..., :1]), dict(block_table=pool.table.long()), dict(block_table=pool.table[:1]),
                dict(kv_lens=pool.lens.int()), dict(kv_lens=pool.lens.cpu()), dict(workspace=ws[:1024]), dict(workspace=ws.int()),
                dict(sm_scale=math.nan), dict(sm_scale="x"), dict(q=q.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises((ValueError, TypeError, kvq.KvqError)):
            kvq.kv_gqa_attn_paged(**{**good, **bad})
    rope, pos, slots = kvq.rope_layout([1.0] * 32), torch.arange(2, device="cuda"), torch.arange(2, device="cuda")
    k = queries(2, 2, 64, torch.bfloat16)
    good = dict(rope=rope, k_new=k, v_new=k.clone(), positions=pos, slot_map=slots, q_in=q, q_out=torch.zeros_like(q),
                k_codes=pool.k, v_codes=pool.v, scales=pool.scales)
    kvq.kv_gqa_append(**good)
    for bad in (dict(v_new=None), dict(k_new=None, v_new=None, q_in=None), dict(k_new=k.float()), dict(k_new=k[:, :1]), dict(k_new=k[:1]),
                dict(q_out=None), dict(q_out=good["q_out"].float()), dict(q_out=q[:1]), dict(positions=None), dict(positions=pos.int()),
                dict(positions=pos[:1]), dict(slot_map=None), dict(slot_map=slots[:1]), dict(slot_map=slots.int()),
                dict(rope=kvq.rope_layout([1.0] * 33)), dict(rope=kvq.mla_layout()), dict(k_codes=None), dict(q_in=q[:, :3]),
                dict(err_word=torch.zeros(1, device="cuda")), dict(q_in=q.permute(0, 2, 1))):
        with pytest.raises((ValueError, TypeError, kvq.KvqError)):
            kvq.kv_gqa_append(**{**good, **bad})
    x, s = torch.zeros(2, 3, 100, device="cuda"), torch.zeros(2, 3, device="cuda")
    o, i = torch.zeros(2, 4, device="cuda"), torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    good = dict(logits=x, scores=s, out_scores=o, parents=i, tokens=i.clone(),
                workspace=torch.zeros(kvq.kv_beam_workspace_size(2, 3, 100, 4), dtype=torch.uint8, device="cuda"))
    kvq.kv_beam_select(**good)
    for bad in (dict(logits=x.half()), dict(logits=x[:, :, ::2]), dict(logits=x[0]), dict(logits=x.expand(2, 3, 100)[:, :1].expand(2, 3, 100)),
                dict(logits=torch.zeros(2, 5, 100, device="cuda")[:, :3]), dict(scores=s[:1]), dict(scores=s.double()), dict(parents=i.long()),
                dict(tokens=i[:, :3]), dict(out_scores=o.cpu()), dict(workspace=good["workspace"][:4096])):
        with pytest.raises((ValueError, TypeError, kvq.KvqError)):
            kvq.kv_beam_select(**{**good, **bad})
    free, n_free = torch.arange(pool.n_pages, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    good = dict(parents=torch.arange(2, dtype=torch.int32, device="cuda"), kv_lens=pool.lens, block_table=pool.table, free_pages=free,
                n_free=n_free, page_rows=16, copies=torch.zeros(2, 2, dtype=torch.int32, device="cuda"),
                workspace=torch.zeros(kvq.kv_pages_fork_workspace_size(2, pool.width, pool.n_pages), dtype=torch.uint8, device="cuda"))
    kvq.kv_pages_fork(**good)
    for bad in (dict(parents=good["parents"].long()), dict(parents=good["parents"][:1]), dict(kv_lens=pool.lens.int()),
                dict(block_table=pool.table[:, :1]), dict(n_free=free), dict(page_rows=24), dict(page_rows=0),
                dict(copies=good["copies"].view(-1)), dict(workspace=good["workspace"][:256])):
        with pytest.raises((ValueError, TypeError, kvq.KvqError)):
            kvq.kv_pages_fork(**{**good, **bad})
    copies = torch.full((2, 2), -1, dtype=torch.int32, device="cuda")
    kvq.kv_pages_copy(copies, [pool.k, pool.v, pool.scales])
    for bad in (dict(copies=copies.long()), dict(copies=copies[:, :1]), dict(pools=[pool.k, pool.v[1:]]), dict(pools=[pool.k.cpu()]),
                dict(pools=[pool.k.transpose(1, 2)]), dict(pools=7), dict(pools=[None])):
        with pytest.raises((ValueError, TypeError, kvq.KvqError)):
            kvq.kv_pages_copy(**{**dict(copies=copies, pools=[pool.k]), **bad})


def test_calls_side_by_side(kvq):
    """Two streams, a workspace each."""
    jobs = []
    for i, (new, dtype) in enumerate(((1, torch.bfloat16), (300, torch.bfloat16), (90, torch.float32))):
        pool = Pool(4, 128, 64, [6000 + i], seed=i)
        q = queries(new, 16, 128, dtype, seed=i)
        jobs.append((pool, q, offsets([new]), torch.zeros_like(q), workspace(kvq, 16, 4, 128, dtype == torch.bfloat16), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for pool, q, cu, out, ws, st in jobs:
            kvq.kv_gqa_attn_paged(q, cu, pool.k, pool.v, pool.scales, pool.table, pool.lens, out, ws, 0.1, stream=st)
    torch.cuda.synchronize()
    for i, (pool, q, cu, out, ws, st) in enumerate(jobs):
        check(out, q, pool, [6000 + i], [len(q)], 0.1, True, f"job {i}")
        assert kvq.read_device_error(ws) == 0


@pytest.mark.parametrize("page", [1024, 65536])
def test_large_pages(kvq, page):
    """Rows appended into pages larger than a tile's steps and attended; the second sequence's page is partly filled."""
    kv, dim, lens, new = 2, 64, [page + 3, 100], [70, 1]
    for dtype in DT:
        pool = Pool(kv, dim, page, lens, seed=2)
        t = torch.cat([torch.arange(n - m, n, device="cuda") for n, m in zip(lens, new)])
        b = torch.repeat_interleave(torch.arange(2, device="cuda"), torch.tensor(new, device="cuda"))
        slots = pool.table[b, t // page].long() * page + t % page
        k, v = queries(71, kv, dim, dtype, seed=3), queries(71, kv, dim, dtype, seed=4)
        kvq.kv_gqa_append(None, k, v, None, slots, None, None, pool.k, pool.v, pool.scales)
        (kc, ks), (vc, vs) = encode_rows(k.float()), encode_rows(v.float())
        pg, at = slots // page, slots % page
        assert torch.equal(pool.k[pg, :, at], kc) and torch.equal(pool.v[pg, :, at], vc)
        assert torch.allclose(pool.scales[pg, :, at], torch.stack([ks, vs], -1), rtol=2.0 ** -23, atol=0.0)
        q = queries(71, 8, dim, dtype)
        for causal in (True, False):
            out, ws = attend(kvq, pool, q, lens, new, causal)
            check(out, q, pool, lens, new, 1 / math.sqrt(dim), causal, f"{dtype} {causal}")
            assert kvq.read_device_error(ws) == 0
